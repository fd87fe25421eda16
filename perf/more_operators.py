"""The operators around attention of a decoding step with drafted tokens, as they are measured: rotary positions
with several axes (`turn`), the page tables, slots, positions and tree masks of a step made from the requests'
lengths (`plan`), the choice of the drafted tokens that stay, by the target's probabilities and given random numbers
(`verify`), and the cache rows, lengths and pages that stay with them (`keep`).

    turn    pair i of a head turned by positions[axis[i]][t] * f_i
    plan    sequence b gets counts[b] rows behind its lens[b] tokens; new pages come off the top of a list
    verify  from a row's target p and draft q: a child x stays iff u S q(x) < p(x) - a q(x), else a += S and
            S = sum (p - a q)+ (a = 0, S = 1 at first); q a point mass where no draft is given; then the first i with
            cumsum(w)_i > u sum(w), w what is left of p
    keep    the kept rows moved behind the sequence's tokens, the pages behind them put back on the list

`own = False`: elementary torch operations. `own = True`: the library's calls.
"""

import math

import numpy as np
import torch

own = False

DTYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
BITS = {4: 2, 8: 3, 16: 4, 256: 8}


# ---- cases --------------------------------------------------------------------------------

def listed():
    def turn(name, **kw):
        return {"name": name, "op": "turn", "dtype": "bf16", "tokens": 1, "heads": 40, "dim": 128, "time": 16, "height": 24,
                "width": 24, "cycle": False, "restart": False, "interleaved": False, "backward": False, **kw}

    def plan(name, **kw):
        return {"name": name, "op": "plan", "seqs": 16, "rows": 1, "ragged": False, "longest": 8000, "page": 64,
                "tree": False, "short": False, **kw}

    def verify(name, **kw):
        return {"name": name, "op": "verify", "target": "bf16", "draft": "bf16", "probabilities": False, "seqs": 1, "rows": 4,
                "ragged": False, "tree": False, "vocab": 32000, "greedy": False, **kw}

    def keep(name, **kw):
        return {"name": name, "op": "keep", "seqs": 16, "rows": 5, "longest": 8000, "page": 64, "tree": False, "heads": 8,
                "dim": 128, "klevels": 256, "vlevels": 8, "group": 64, **kw}

    return [
        # one decoded token of a model that reads images: 32 query and 8 key heads, pairs in three blocks
        turn("turn_token"),
        # a prompt of text and images, the three axes taking pairs in turn
        turn("turn_prompt", tokens=8192, time=24, height=20, width=20, cycle=True),
        # the patches of an image (an odd grid) by height and width, each axis with frequencies of its own; the gradient
        turn("turn_patches_gradient", dtype="fp32", tokens=1369, heads=16, dim=80, time=0, height=20, width=20, restart=True,
             interleaved=True, backward=True),
        # a decoding step of 16 sequences, one token each
        plan("plan_step"),
        # trees of 24 drafted tokens for 192 sequences, with their masks
        plan("plan_trees", seqs=192, rows=24, tree=True),
        # chunks of five prompts of uneven length, the list too short for the last one
        plan("plan_prompts", seqs=5, rows=16001, ragged=True, longest=30000, page=32, short=True),
        # one sequence with three drafted tokens, a small vocabulary: the smallest verification
        verify("verify_short"),
        # a large batch with eight drafted tokens each over a large vocabulary (the largest call)
        verify("verify_batch", seqs=64, rows=9, vocab=131072),
        # trees of drafted tokens without a distribution, an odd vocabulary, some sequences greedy
        verify("verify_trees", target="fp16", draft="none", seqs=8, rows=24, tree=True, vocab=50257, greedy=True),
        # probabilities that the sampler has filtered already, uneven numbers of drafted tokens
        verify("verify_filtered", target="fp32", draft="fp32", probabilities=True, seqs=32, rows=6, ragged=True, vocab=100003),
        # 16 sequences with chains of drafted tokens: lengths and pages only
        keep("keep_chains"),
        # 192 sequences with trees: accepted branches moved together in the cache
        keep("keep_trees", seqs=192, rows=24, tree=True),
    ]


def draw(rng):
    def spread(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["turn", "plan", "verify", "keep"])
    page = rng.choice([16, 32, 64, 256])
    if op == "turn":
        dim = rng.choice([64, 80, 96, 128, 256])
        heads = rng.randint(1, 48)
        used = rng.choice([dim // 2, dim // 2, dim // 4])     # pairs that turn
        time = rng.choice([0, used // 4, used // 3])
        height = (used - time) // 2
        return {"op": op, "dtype": rng.choice(list(DTYPES)), "tokens": spread(1, max(2, 8192 * 40 * 128 // (2 * heads * dim))),
                "heads": heads, "dim": dim, "time": time, "height": height, "width": used - time - height,
                "cycle": rng.random() < 0.5, "restart": rng.random() < 0.3, "interleaved": rng.random() < 0.4,
                "backward": rng.random() < 0.3}
    if op == "plan":
        tree = rng.random() < 0.4
        seqs = spread(1, 256)
        rows = rng.randint(2, 60) if tree else spread(1, max(2, 60000 // seqs))
        return {"op": op, "seqs": seqs, "rows": rows, "ragged": rng.random() < 0.5, "longest": spread(10, 40000), "page": page,
                "tree": tree, "short": rng.random() < 0.3}
    if op == "verify":
        tree, probabilities = rng.random() < 0.4, rng.random() < 0.3
        seqs, vocab = spread(1, 64), spread(1000, 131072)
        rows = rng.randint(1, max(1, min(20 if tree else 9, 64 * 9 * 131072 // (2 * seqs * vocab))))
        return {"op": op, "target": rng.choice(list(DTYPES)), "draft": rng.choice(["none"] + 2 * list(DTYPES)),
                "probabilities": probabilities, "seqs": seqs, "rows": rows, "ragged": rng.random() < 0.5, "tree": tree,
                "vocab": vocab, "greedy": rng.random() < 0.3}
    dim = rng.choice([64, 128, 256])
    return {"op": op, "seqs": spread(1, 192), "rows": rng.randint(2, 40), "longest": spread(10, 8000), "page": page,
            "tree": rng.random() < 0.7, "heads": rng.randint(1, 8), "dim": dim, "klevels": rng.choice([256, 256, 16]),
            "vlevels": rng.choice([8, 16, 256, 4]), "group": rng.choice([g for g in (32, 64, 128) if g <= dim])}


def _counts(case):
    """Rows of each sequence in the step."""
    n, q = case["seqs"], case["rows"]
    return [max(1, q * (i + 1) // n) for i in range(n)] if case.get("ragged") else [q] * n


def _row(case):
    """Bytes of a token of one head in the cache, keys and values."""
    return sum(case["dim"] * BITS[case[k]] // 8 + case["dim"] // case["group"] * 2 for k in ("klevels", "vlevels"))


def work(case):
    op = case["op"]
    if op == "turn":
        size = 4 if case["dtype"] == "fp32" else 2
        pairs = case["time"] + case["height"] + case["width"]
        n = case["tokens"] * case["heads"]
        axes = (case["time"] > 0) + 2
        return {"bytes": 2 * n * case["dim"] * size + case["tokens"] * 4 * axes, "flops": 6 * n * pairs}
    B, M = case["seqs"], sum(_counts(case))
    if op == "plan":
        tree = 4 + 4 * (-(-case["rows"] // 32)) if case["tree"] else 0
        return {"bytes": B * 24 + M * (12 + tree) + M // case["page"] * 8, "flops": 4 * M}
    if op == "verify":
        size = {"fp32": 4, "bf16": 2, "fp16": 2}
        V = case["vocab"]
        rows = B if case["probabilities"] else M          # probabilities: one row and single values; logits: each row
        drafts = 0 if case["draft"] == "none" else B if case["probabilities"] else max(0, M - B)
        return {"bytes": V * (rows * size[case["target"]] + drafts * size.get(case["draft"], 0)) + M * 16,
                "flops": 10 * V * (rows + drafts)}
    kept = B * min(5, max(1, case["rows"] // 2))
    return {"bytes": B * 24 + M * 4 + (2 * kept * case["heads"] * _row(case) if case["tree"] else 0), "flops": 4 * B}


# ---- inputs -------------------------------------------------------------------------------

def _sections(case):
    return [n for n in (case["time"], case["height"], case["width"]) if n]


def _pairs(case):
    """Axis of each pair, and its radians per position."""
    sections = _sections(case)
    axis = []
    left = list(sections)
    if case["cycle"]:
        while sum(left):
            for a in range(len(left)):
                if left[a]:
                    axis.append(a)
                    left[a] -= 1
    else:
        axis = [a for a, n in enumerate(sections) for _ in range(n)]
    seen, freq = [0] * len(sections), []
    for i, a in enumerate(axis):
        freq.append(10000.0 ** (-seen[a] / sections[a]) if case["restart"] else 10000.0 ** (-i / len(axis)))
        seen[a] += 1
    return axis, freq


def _parents(counts, rng):
    """Each drafted row hangs on one of the four rows before it."""
    out = []
    for n in counts:
        out += [0] + [int(rng.randint(max(0, i - 4), i)) for i in range(1, n)]
    return out


def _pool(case, lens, counts, gen, dev):
    """Page tables of `lens` tokens, the list of the free pages, and how many of them are free."""
    page = case["page"]
    held = [-(-n // page) for n in lens]
    want = [-(-(n + c) // page) - h for n, c, h in zip(lens, counts, held)]
    width = max(h + w for h, w in zip(held, want)) + 1
    free = sum(want) + 3
    if case.get("short"):
        free = max(0, sum(want) - max(1, want[-1] // 2))
    pages = sum(held) + sum(-(-c // page) + 1 for c in counts) + 7      # the same for every seed
    order = torch.randperm(pages, generator=gen, device=dev).to(torch.int32)
    table = torch.full((len(lens), width), -1, dtype=torch.int32, device=dev)
    at = 0
    for b, h in enumerate(held):
        table[b, :h] = order[at:at + h]
        at += h
    stack = torch.full((pages,), -1, dtype=torch.int32, device=dev)
    stack[:free] = order[at:at + free]
    return {"pages": pages, "table": table, "stack": stack, "free": free}


def _filtered(x, temperature):
    """What a sampler leaves: probabilities below a thousandth of the largest are taken out."""
    p = torch.softmax(x / temperature, -1)
    p = torch.where(p >= p.amax(-1, keepdim=True) * 1e-3, p, torch.zeros_like(p))
    return p / p.sum(-1, keepdim=True)


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    rng = np.random.RandomState(seed % (2 ** 31))
    op, st = case["op"], {"case": case}
    if op == "turn":
        axis, freq = _pairs(case)
        st["axis"] = torch.tensor(axis, dtype=torch.uint8, device=dev)
        st["freq"] = torch.tensor(freq, dtype=torch.float64, device=dev)
        axes, T = len(_sections(case)), case["tokens"]
        # images of 37 x 37 patches one after another; the time axis goes on from image to image
        t = torch.arange(T, device=dev) + int(rng.randint(0, 30000))
        st["positions"] = torch.stack(([t // 1369] if axes == 3 else []) + [t % 1369 // 37, t % 37]).to(torch.int32)
        wide = torch.randn((T, case["heads"] + max(1, case["heads"] // 5), case["dim"]), generator=gen, device=dev)
        st["x"] = wide.to(DTYPES[case["dtype"]])[:, :case["heads"]]    # the value heads lie behind the turned ones
        return st
    counts = _counts(case)
    B, M = len(counts), sum(counts)
    offsets = np.concatenate([[0], np.cumsum(counts)])
    st["counts"] = torch.tensor(counts, dtype=torch.int32, device=dev)
    st["most"] = max(counts)
    st["parents"] = None
    if case["tree"]:
        st["parents"] = torch.tensor(_parents(counts, rng), dtype=torch.int32, device=dev)
    if op in ("plan", "keep"):
        lens = [int((case["longest"] + 1.0) ** ((b + 1) / B)) - 1 for b in rng.permutation(B - 1)] + [case["longest"]]
        st["lens"] = torch.tensor(lens, dtype=torch.int32, device=dev)
        pool = _pool(case, lens, counts, gen, dev)
        st.update(pages=pool["pages"], table=pool["table"], stack=pool["stack"])
        st["shift"] = torch.randint(-50, 50, (B,), generator=gen, device=dev, dtype=torch.int32) if op == "plan" else None
        st["left"] = torch.tensor([pool["free"], 0], dtype=torch.int32, device=dev)
        st["words"] = (st["most"] + 31) // 32 if case["tree"] else 0
        if op == "plan":
            return st
        # the step's pages are taken: off the list and in the tables
        st["offsets"] = torch.tensor(offsets, dtype=torch.int32, device=dev)
        page, at = case["page"], pool["free"]
        for b, (n, c) in enumerate(zip(lens, counts)):
            h, w = -(-n // page), -(-(n + c) // page)
            if w > h:
                st["table"][b, h:w] = st["stack"][at - (w - h):at].flip(0)
                at -= w - h
        st["left"][0] = at
        kept = rng.randint(1, min(5, max(1, case["rows"] // 2)) + 1, B)
        st["kept"] = torch.tensor(kept, dtype=torch.int32, device=dev)
        if case["tree"]:
            path = np.full(M, -1, dtype=np.int32)
            for b in range(B):     # a branch whose rows all lie behind the places that they move to
                k = int(kept[b])
                path[offsets[b]] = 0
                rows = np.sort(rng.choice(np.arange(k, counts[b]), k - 1, replace=False)) if k > 1 else []
                path[offsets[b] + 1:offsets[b] + k] = rows
            st["path"] = torch.tensor(path, dtype=torch.int32, device=dev)
            rows = case["heads"] * page
            for name, levels in (("k", case["klevels"]), ("v", case["vlevels"])):
                words = case["dim"] * BITS[levels] // 32
                st[name] = torch.randint(-2 ** 31, 2 ** 31 - 1, (st["pages"], rows, words), generator=gen, device=dev,
                                         dtype=torch.int32)
                st[name + "s"] = torch.exp(0.5 * torch.randn((st["pages"], rows, case["dim"] // case["group"]), generator=gen,
                                                             device=dev)).to(torch.float16)
            st["signs"] = torch.randint(-2 ** 31, 2 ** 31 - 1, (case["dim"] // 32,), generator=gen, device=dev, dtype=torch.int32)
        return st
    # verification: the draft model's values are the target's with some noise; drafted tokens drawn from its distribution
    V = case["vocab"]
    st["offsets"] = torch.tensor(offsets, dtype=torch.int32, device=dev)
    temperature = torch.rand((B,), generator=gen, device=dev) * 0.6 + 0.6
    row_seq = torch.repeat_interleave(torch.arange(B, device=dev), torch.tensor(counts, device=dev))
    parents = st["parents"] if case["tree"] else torch.cat([torch.arange(-1, n - 1, device=dev).clamp(min=0) for n in counts])
    target = torch.empty((M, V), dtype=DTYPES[case["target"]], device=dev)
    draft = None if case["draft"] == "none" else torch.empty((M, V), dtype=DTYPES[case["draft"]], device=dev)
    tokens = torch.empty((M,), dtype=torch.int32, device=dev)
    for b in range(B):
        a, e = int(offsets[b]), int(offsets[b + 1])
        x = torch.randn((e - a, V), generator=gen, device=dev) * 3.0
        y = x + torch.randn((e - a, V), generator=gen, device=dev) * 0.6
        if case["probabilities"]:
            x, y = _filtered(x, temperature[b]), _filtered(y, temperature[b])
        target[a:e] = x.to(target.dtype)
        if draft is not None:
            y = y.to(draft.dtype)
            draft[a:e] = y
        z = torch.log(y.float()) if case["probabilities"] else y.float() / temperature[b]
        noise = -torch.log(-torch.log(torch.rand((e - a, V), generator=gen, device=dev).clamp(1e-7, 1 - 1e-7)))
        tokens[a:e] = (z[parents[a:e].long()] + noise).argmax(-1).to(torch.int32)
    if case["greedy"]:
        temperature[::3] = 0.0
    st.update(target=target, draft=draft, tokens=tokens, row_seq=row_seq,
              temperature=temperature if case["greedy"] or not case["probabilities"] else None,
              uniforms=torch.rand((M,), generator=gen, device=dev))
    return st


# ---- the plain forms ----------------------------------------------------------------------

def _plain_turn(st):
    case = st["case"]
    rot = 2 * st["axis"].numel()
    pos = st["positions"][st["axis"].long()].t().to(torch.float64)       # [tokens, pairs]
    a = pos * st["freq"]
    cos, sin = torch.cos(a)[:, None], torch.sin(a)[:, None]
    if case["backward"]:
        sin = -sin
    x = st["x"].to(torch.float64)
    head, rest = x[..., :rot], x[..., rot:]
    if case["interleaved"]:
        p, q = head[..., 0::2], head[..., 1::2]
        turned = torch.stack((p * cos - q * sin, q * cos + p * sin), dim=-1).flatten(-2)
    else:
        p, q = head[..., :rot // 2], head[..., rot // 2:]
        turned = torch.cat((p * cos - q * sin, q * cos + p * sin), dim=-1)
    return torch.cat((turned, rest), dim=-1).to(st["x"].dtype)


def _plain_plan(st):
    case, page, table = st["case"], st["case"]["page"], st["table"]
    B, width = table.shape
    lens, counts = st["lens"].to(torch.int64), st["counts"].to(torch.int64)
    dev = lens.device
    M = sum(_counts(case))
    offsets = torch.cat([torch.zeros(1, dtype=torch.int64, device=dev), torch.cumsum(counts, 0)])
    held = (lens + page - 1) // page
    want = (lens + counts + page - 1) // page - held
    total = torch.cumsum(want, 0)
    ok = (want == 0) | (total <= st["left"][0])
    status = torch.where(ok, 0, 1)
    row = torch.arange(M, device=dev)
    b = torch.searchsorted(offsets, row, right=True) - 1
    i = row - offsets[b]
    # new pages into the tables: entry j of a sequence's new ones is the list's number left - 1 - (those before + j)
    j = torch.arange(width, device=dev)[None] - held[:, None]
    new = (j >= 0) & (j < want[:, None]) & ok[:, None]
    at = (st["left"][0] - 1 - (total - want)[:, None] - j).clamp(0, st["stack"].numel() - 1)
    table.copy_(torch.where(new, st["stack"][at], table))
    place = lens[b] + i
    slots = table[b, (place // page).clamp(max=width - 1)].to(torch.int64) * page + place % page
    slots = torch.where(ok[b], slots, -1)
    depth, mask = i, None
    if case["tree"]:
        # a row's mask: its parent's and itself, row by row of the sequences
        most, words = st["most"], st["words"]
        bits = torch.zeros((B, most, words * 32), dtype=torch.bool, device=dev)
        dep = torch.zeros((B, most), dtype=torch.int64, device=dev)
        seq = torch.arange(B, device=dev)
        for r in range(most):
            at = (offsets[:-1] + r).clamp(max=M - 1)
            up = st["parents"][at].to(torch.int64)
            if r:
                live = r < counts
                up = torch.where(live, up, 0)
                bits[:, r] = bits[seq, up] & live[:, None]
                dep[:, r] = dep[seq, up] + 1
            bits[:, r, r] = r < counts
        depth = dep[b, i]
        flat = (bits[b, i] & ok[b][:, None]).view(M, words, 32).to(torch.int64)
        mask = (flat << torch.arange(32, device=dev)).sum(-1)
        mask = torch.where(mask >= 2 ** 31, mask - 2 ** 32, mask).to(torch.int32)
    positions = torch.where(ok[b], lens[b] + depth + st["shift"][b], 0)
    left = st["left"][0] - (want * ok).sum()
    return (slots, positions.to(torch.int32), offsets.to(torch.int32), torch.where(ok, lens + counts, 0).to(torch.int32),
            status.to(torch.int32), mask, table, left.to(torch.int32).view(1))


def _plain_verify(st):
    case, V = st["case"], st["case"]["vocab"]
    dev = st["tokens"].device
    first, n = st["offsets"][:-1].to(torch.int64), st["counts"].to(torch.int64)
    B, M = first.numel(), st["tokens"].numel()
    temperature = st["temperature"]
    greedy = temperature <= 0 if temperature is not None else torch.zeros(B, dtype=torch.bool, device=dev)

    def distribution(x):
        x = x.to(torch.float64)
        if case["probabilities"]:
            return x
        x = x / torch.where(greedy, 1.0, temperature.to(torch.float64))[st["row_seq"]][:, None]
        e = torch.exp(x - x.amax(-1, keepdim=True))
        return e / e.sum(-1, keepdim=True)

    P = distribution(st["target"])
    if case["greedy"]:
        rows = greedy[st["row_seq"]]
        one = torch.zeros_like(P).scatter_(1, st["target"].to(torch.float64).argmax(-1, keepdim=True), 1.0)
        P = torch.where(rows[:, None], one, P)
    Q = distribution(st["draft"]) if st["draft"] is not None else None
    drafted = Q is not None and st["most"] > 1
    seq = torch.arange(B, device=dev)
    cur = torch.zeros(B, dtype=torch.int64, device=dev)
    kept = torch.ones(B, dtype=torch.int64, device=dev)
    a, S = torch.zeros(B, dtype=torch.float64, device=dev), torch.ones(B, dtype=torch.float64, device=dev)
    gone = torch.zeros((B, V), dtype=torch.bool, device=dev) if Q is None else None
    path = torch.full((M + 1,), -1, dtype=torch.int64, device=dev)
    path[first] = 0
    for r in range(1, st["most"]):
        row = (first + r).clamp(max=M - 1)
        up = st["parents"][row].to(torch.int64) if case["tree"] else torch.full((B,), r - 1, dtype=torch.int64, device=dev)
        x = st["tokens"][row].to(torch.int64)
        here = (r < n) & (up == cur)
        u = st["uniforms"][row].to(torch.float64)
        at = first + cur
        if Q is None:
            px = torch.where(gone[seq, x], 0.0, P[at, x])
            yes = here & (u * S < px)
            S = torch.where(here & ~yes, S - px, S)
            gone[seq, x] |= here & ~yes
            gone &= ~yes[:, None]
        else:
            q = torch.where(greedy, 0.0, Q[at, x])
            yes = here & (u * S * q < P[at, x] - a * q)
            no = here & ~yes
            a = torch.where(no, a + S, a)
            if case["tree"]:
                rest = (P[at] - a[:, None] * torch.where(greedy[:, None], 0.0, Q[at])).clamp(min=0).sum(-1)
                S = torch.where(no, rest, S)
        path[torch.where(yes, first + kept, M)] = r
        cur = torch.where(yes, r, cur)
        kept = kept + yes
        a, S = torch.where(yes, 0.0, a), torch.where(yes, 1.0, S)
    path = path[:M]
    p = P[first + cur]
    if drafted:
        w = (p - torch.where(greedy, 0.0, a)[:, None] * Q[first + cur]).clamp(min=0)
    else:
        w = p if gone is None else torch.where(gone, 0.0, p)
    w = torch.where(w.sum(-1, keepdim=True) > 0, w, p)
    c = torch.cumsum(w, -1)
    u = st["uniforms"][first].to(torch.float64) * c[:, -1]
    last = V - 1 - (w > 0).flip(-1).to(torch.int8).argmax(-1)
    new = torch.minimum((c <= u[:, None]).sum(-1), last)
    out = torch.full((M + 1,), -1, dtype=torch.int64, device=dev)
    row = torch.arange(M, device=dev)
    i = row - first[st["row_seq"]]
    accepted = i < kept[st["row_seq"]] - 1
    step = torch.where(accepted, torch.cat([path[1:], path[:1]]), 0)      # the row of the token that follows path[i]
    out[:M] = torch.where(accepted, st["tokens"][first[st["row_seq"]] + step.clamp(min=0)].to(torch.int64), -1)
    out[first + kept - 1] = new
    return kept.to(torch.int32), out[:M].to(torch.int32), path.to(torch.int32)


def _plain_keep(st):
    case, page, table = st["case"], st["case"]["page"], st["table"]
    B, width = table.shape
    lens, counts, kept = (st[k].to(torch.int64) for k in ("lens", "counts", "kept"))
    dev = lens.device
    if case["tree"]:
        M = st["path"].numel()
        row = torch.arange(M, device=dev)
        b = torch.searchsorted(st["offsets"].to(torch.int64), row, right=True) - 1
        i = row - st["offsets"][b].to(torch.int64)
        moves = (i > 0) & (i < kept[b])
        # a row that stays where it is is written onto itself
        source = lens[b] + torch.where(moves, st["path"].to(torch.int64), i)
        target = lens[b] + i
        head = torch.arange(case["heads"], device=dev)[None] * page
        src_page, src = table[b, source // page].to(torch.int64)[:, None], head + (source % page)[:, None]
        dst_page, dst = table[b, target // page].to(torch.int64)[:, None], head + (target % page)[:, None]
        # rows behind the kept ones may be sources of moves: only the moved ones are written
        for name in ("k", "ks", "v", "vs"):
            data = st[name][src_page, src]
            old = st[name][dst_page, dst]
            st[name][dst_page, dst] = torch.where(moves[:, None, None], data, old)
    end = lens + kept
    have, want = (lens + counts + page - 1) // page, (end + page - 1) // page
    back = have - want
    total = torch.cumsum(back, 0)
    left = st["left"][0] + total[-1]
    j = torch.arange(width, device=dev)[None] - want[:, None]
    ours = (j >= 0) & (j < back[:, None])
    size = st["stack"].numel()
    at = torch.where(ours, left - 1 - (total - back)[:, None] - j, size)
    longer = torch.cat([st["stack"], st["stack"][:1]])
    longer[at.flatten()] = table.flatten()
    st["stack"].copy_(longer[:size])
    return end.to(torch.int32), left.to(torch.int32).view(1)


# ---- one pass -----------------------------------------------------------------------------

def _cache(st):
    """The cache's handle: descriptors around tensors in hand."""
    import rotation_lloyd_max_amd as tq
    case, halves = st["case"], []
    for name, levels in (("k", case["klevels"]), ("v", case["vlevels"])):
        halves.append(tq.QWeight(st[name], st[name + "s"], st["signs"], levels, case["group"], case["dim"], st[name].shape[1],
                                 st["pages"], 0))
    return tq.KVCache(halves[0], halves[1], case["heads"], case["page"])


def _own(st):
    import rotation_lloyd_max_amd as tq
    case, op = st["case"], st["case"]["op"]
    if op == "turn":
        rope = tq.Rope(st["freq"], 2 * st["axis"].numel(), interleaved=case["interleaved"], axis=st["axis"])
        return tq.rope(st["x"], st["positions"], rope, transposed=case["backward"])
    if op == "verify":
        kind = "probabilities" if case["probabilities"] else "logits"
        out = tq.verify(st["target"], st["tokens"], st["uniforms"], st["offsets"], draft=st["draft"], parents=st["parents"],
                        temperature=st["temperature"], target_kind=kind, draft_kind=kind)
        return out.kept, out.tokens, out.path
    pool = tq.KVPool(st["stack"], st["left"])
    left = torch.empty_like(st["left"][:1])
    if op == "plan":
        p = tq.kv_plan(pool, st["lens"], st["counts"], st["table"], sum(_counts(case)), case["page"], parents=st["parents"],
                       tree_words=st["words"], shift=st["shift"], left=left)
        return p.slots, p.positions, p.q_offsets, p.kv_lens, p.status, p.tree, st["table"], left
    cache = _cache(st) if case["tree"] else None
    end = tq.kv_keep(pool, st["lens"], st["kept"], st["table"], case["page"], q_offsets=st["offsets"],
                     path=st["path"] if case["tree"] else None, cache=cache, out=torch.empty_like(st["lens"]), left=left)
    return end, left


def run(state):
    op = state["case"]["op"]
    if own:
        out = _own(state)
    else:
        out = {"turn": _plain_turn, "plan": _plain_plan, "verify": _plain_verify, "keep": _plain_keep}[op](state)
    if op == "keep":
        out = (*out, state["stack"], *(state[name] for name in ("k", "v", "ks", "vs") if name in state))
    return out if torch.is_tensor(out) else tuple(x for x in out if x is not None)


# ---- the definition in 64 bits --------------------------------------------------------------

def _exact_turn(st):
    case = st["case"]
    x = st["x"].double()
    y = x.clone()
    h = st["axis"].numel()
    axis = st["axis"].tolist()
    for i in range(h):
        angle = st["positions"][axis[i]].double() * float(st["freq"][i]) * (-1.0 if case["backward"] else 1.0)
        turn = torch.polar(torch.ones_like(angle), angle)[:, None]
        c, d = (2 * i, 2 * i + 1) if case["interleaved"] else (i, i + h)
        z = torch.complex(x[..., c], x[..., d]) * turn
        y[..., c], y[..., d] = z.real, z.imag
    return y


def _exact_plan(st):
    case, page = st["case"], st["case"]["page"]
    table = st["table"].cpu().numpy().copy()
    stack, left = st["stack"].tolist(), int(st["left"][0])
    lens, counts, shift = st["lens"].tolist(), st["counts"].tolist(), st["shift"].tolist()
    parents = st["parents"].tolist() if case["tree"] else None
    slots, positions, tree, offsets, ends, status = [], [], [], [0], [], []
    refused = False
    for b, (n, c) in enumerate(zip(lens, counts)):
        held, full = -(-n // page), -(-(n + c) // page)
        refused = refused or full - held > left
        ok = full == held or not refused
        status.append(0 if ok else 1)
        ends.append(n + c if ok else 0)
        if ok:
            for j in range(held, full):
                left -= 1
                table[b, j] = stack[left]
        seen, depth = [], []
        for i in range(c):
            if parents is not None:
                up = parents[offsets[-1] + i]
                seen.append((seen[up] if i else 0) | 1 << i)
                depth.append(depth[up] + 1 if i else 0)
                word = seen[-1] if ok else 0
                words = [(word >> 32 * k) & 0xffffffff for k in range(st["words"])]
                tree.append([w - 2 ** 32 if w >= 2 ** 31 else w for w in words])
            else:
                depth.append(i)
            slots.append(int(table[b, (n + i) // page]) * page + (n + i) % page if ok else -1)
            positions.append(n + depth[i] + shift[b] if ok else 0)
        offsets.append(offsets[-1] + c)
    dev = st["lens"].device
    put = lambda v, t=torch.int32: torch.tensor(v, dtype=t, device=dev)  # noqa: E731
    return (put(slots, torch.int64), put(positions), put(offsets), put(ends), put(status), put(tree) if tree else None,
            torch.from_numpy(table).to(dev), put([left]))


def _exact_verify(st):
    case = st["case"]
    offsets, tokens = st["offsets"].tolist(), st["tokens"].tolist()
    parents = st["parents"].tolist() if case["tree"] else None
    u = st["uniforms"].double().tolist()
    T = st["temperature"].double().tolist() if st["temperature"] is not None else None

    def distribution(x, b):
        x = x.double()
        if T is not None and T[b] <= 0:
            return torch.zeros_like(x).index_fill_(0, torch.nonzero(x == x.max())[0], 1.0)
        if case["probabilities"]:
            return x
        z = x / T[b]
        return torch.exp(z - torch.logsumexp(z, 0))

    kept, out, path = [], [-1] * len(tokens), [-1] * len(tokens)
    for b, (first, end) in enumerate(zip(offsets[:-1], offsets[1:])):
        greedy = T is not None and T[b] <= 0
        path[first], at, k = 0, 0, 1
        while True:
            p0 = distribution(st["target"][first + at], b)
            q = distribution(st["draft"][first + at], b) if st["draft"] is not None and not greedy else None
            children = [r for r in range(at + 1, end - first) if (parents[first + r] if parents else r - 1) == at]
            p, found = p0.clone(), None
            for r in children:
                x = tokens[first + r]
                px = float(p[x])
                if (u[first + r] * float(q[x]) if q is not None else u[first + r]) < px:
                    found = r
                    break
                if q is not None:
                    p = (p - q).clamp(min=0)
                    total = float(p.sum())
                    p = p / total if total > 0 else p
                else:
                    p[x] = 0.0
                    p = p / (1.0 - px) if px < 1.0 else p
            if found is None:
                break
            out[first + k - 1] = tokens[first + found]
            path[first + k] = found
            at, k = found, k + 1
        p = p if float(p.sum()) > 0 else p0
        c = torch.cumsum(p, 0)
        hit = torch.nonzero(c > u[first] * c[-1])
        out[first + k - 1] = int(hit[0]) if hit.numel() else int(torch.nonzero(p)[-1])
        kept.append(k)
    put = lambda v: torch.tensor(v, dtype=torch.int32, device=st["tokens"].device)  # noqa: E731
    return put(kept), put(out), put(path)


def _exact_keep(st):
    case, page = st["case"], st["case"]["page"]
    table, stack, left = st["table"].tolist(), st["stack"].tolist(), int(st["left"][0])
    lens, counts, kept = st["lens"].tolist(), st["counts"].tolist(), st["kept"].tolist()
    offsets = st["offsets"].tolist()
    cache = {name: st[name].clone() for name in ("k", "v", "ks", "vs") if name in st}
    back, end = [], []
    for b, (n, c, k) in enumerate(zip(lens, counts, kept)):
        if case["tree"]:
            path = st["path"][offsets[b]:offsets[b] + k].tolist()
            for i in range(1, k):
                (sp, s), (dp, d) = ((table[b][(n + r) // page], (n + r) % page) for r in (path[i], i))
                for name in cache:
                    cache[name][dp, d::page] = st[name][sp, s::page]
        end.append(n + k)
        back += table[b][-(-(n + k) // page):-(-(n + c) // page)]
    for page_number in reversed(back):
        stack[left] = page_number
        left += 1
    put = lambda v: torch.tensor(v, dtype=torch.int32, device=st["lens"].device)  # noqa: E731
    return (put(end), put([left]), put(stack), *cache.values())


def exact(case, seed):
    st = prepare(case, seed)
    out = {"turn": _exact_turn, "plan": _exact_plan, "verify": _exact_verify, "keep": _exact_keep}[case["op"]](st)
    return out if torch.is_tensor(out) else tuple(x for x in out if x is not None)
