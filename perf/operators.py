"""The operators of a compressed, paged KV cache, as they are measured: rotary positions (`rope`), the
write of new tokens into the cache and their reading back (`store`), the reading back of many tokens
(`load`), and attention of single tokens, prompt chunks and trees of drafted tokens over the cache (`attend`).

A cache row is one token's key (or value) of one head, D elements x. It is held as
    w = R x,  R = H_D diag(s) / sqrt(D)   (s = +-1 signs, H_D the Sylvester Hadamard matrix),
    scale_g = fp16(rms of group g of w),  code_j = #{k : w_j / rms > t_k},
with the thresholds t and centroids c of the Lloyd-Max quantizer of N(0,1), the codes packed little-endian
into 32-bit words. It stands for R^T (c[code] * scale). Pages hold [heads][page_tokens] such rows.

`own = False`: elementary torch operations. `own = True`: the library's calls.
"""

import functools
import math

import numpy as np
import torch

own = False

PAGE = 64          # tokens of a page, unless a case says otherwise
DTYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
BITS = {4: 2, 8: 3, 16: 4, 256: 8}


# ---- cases --------------------------------------------------------------------------------

def listed():
    def rope(name, **kw):
        return {"name": name, "op": "rope", "dtype": "bf16", "tokens": 1, "heads": 40, "dim": 128, "rot": 128,
                "interleaved": False, "backward": False, "stretch": 1.0, "farthest": 32768, **kw}

    def store(name, **kw):
        return {"name": name, "op": "store", "dtype": "bf16", "tokens": 1, "heads": 8, "dim": 128, "klevels": 256,
                "vlevels": 8, "group": 64, "rot": 128, "interleaved": False, "farthest": 32768, **kw}

    def load(name, **kw):
        return {"name": name, "op": "load", "dtype": "bf16", "tokens": 1, "heads": 8, "dim": 128, "klevels": 256,
                "vlevels": 8, "group": 64, **kw}

    def attend(name, **kw):
        return {"name": name, "op": "attend", "dtype": "bf16", "seqs": 1, "queries": 1, "shortest": 1, "longest": 1,
                "heads": 8, "share": 4, "dim": 128, "klevels": 256, "vlevels": 8, "group": 64, "tree": False,
                "ragged": False, "page": PAGE, **kw}

    return [
        # one decoded token: its 32 query and 8 key heads turned where they lie, between the value heads
        rope("rope_token"),
        # a long prompt with stretched frequencies at far positions (the largest call)
        rope("rope_prompt", tokens=8192, stretch=8.0, farthest=131072),
        # interleaved pairs, part of the head, an odd token count, the gradient's direction
        rope("rope_part_gradient", dtype="fp32", tokens=1021, heads=12, dim=64, rot=32, interleaved=True, backward=True),
        # a decode step of 16 sequences: keys turned and both halves quantized into scattered slots, read back
        store("store_step", tokens=16),
        # a prompt of odd length, wide heads, 4-bit keys and values
        store("store_prompt_wide", dtype="fp16", tokens=3001, heads=4, dim=256, klevels=16, vlevels=16, group=128,
              rot=128, interleaved=True),
        # some tokens of a small-headed cache in fp32 (inspection, moving a sequence to another cache)
        load("load_few", dtype="fp32", tokens=301, heads=5, dim=64, klevels=8, vlevels=4, group=32),
        # every token of a long sequence, for a computation outside the cache
        load("load_long", tokens=32768),
        # the smallest attention: one token after a short text
        attend("attend_token_short", longest=337, shortest=337),
        # a serving batch of uneven lengths, one token each
        attend("attend_batch", seqs=32, shortest=61, longest=8191),
        # one token after a very long text
        attend("attend_token_long", shortest=131071, longest=131071),
        # trees of 24 drafted tokens for four sequences, fp16, 4-bit values
        attend("attend_tree", dtype="fp16", seqs=4, queries=24, shortest=1500, longest=6007, tree=True, vlevels=16),
        # chunks of two prompts of unequal length
        attend("attend_prompt", seqs=2, queries=2047, shortest=4095, longest=8190, ragged=True),
    ]


def draw(rng):
    def spread(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["rope", "store", "load", "attend"])
    dim = rng.choice([64, 128, 256])
    cache = {"dim": dim, "klevels": rng.choice([256, 256, 16]), "vlevels": rng.choice([8, 16, 256, 4]),
             "group": rng.choice([g for g in (32, 64, 128) if g <= dim])}
    if op == "rope":
        heads = rng.randint(1, 48)
        return {"op": op, "dtype": rng.choice(list(DTYPES)), "tokens": spread(1, max(2, 8192 * 40 * 128 // (2 * heads * dim))),
                "heads": heads, "dim": dim, "rot": rng.choice([dim, dim // 2, dim // 4]), "interleaved": rng.random() < 0.5,
                "backward": rng.random() < 0.3, "stretch": rng.choice([1.0, 4.0, 16.0]), "farthest": spread(2048, 262144)}
    if op == "store":
        return {"op": op, "dtype": rng.choice(list(DTYPES)), "tokens": spread(1, 2500 * 128 // dim), "heads": rng.randint(1, 8),
                "rot": rng.choice([0, dim, dim // 2]), "interleaved": rng.random() < 0.5, "farthest": spread(2048, 262144), **cache}
    if op == "load":
        return {"op": op, "dtype": rng.choice(list(DTYPES)), "tokens": spread(1, 16384 * 128 // dim), "heads": rng.randint(1, 8), **cache}
    kind = rng.choice(["token", "token", "tree", "prompt"])
    heads, share = rng.choice([1, 2, 4, 8]), rng.choice([1, 3, 4, 8])
    seqs = spread(1, 32) if kind != "prompt" else rng.randint(1, 3)
    queries = 1 if kind == "token" else rng.randint(2, 60) if kind == "tree" else spread(64, 1500)
    if kind == "token":
        longest = spread(1, max(2, min(100000, 131072 * 8 * 64 // (heads * seqs * dim))))
        shortest = 1 + int(longest * rng.random() * 0.9)
    else:
        shortest = queries + spread(1, 1000)
        longest = shortest + spread(1, 3000 if kind == "prompt" else 5000)
    return {"op": op, "dtype": rng.choice(["bf16", "fp16"]), "seqs": seqs, "queries": queries, "shortest": min(shortest, longest),
            "longest": longest, "heads": heads, "share": share, "tree": kind == "tree", "ragged": rng.random() < 0.5 and kind != "token",
            "page": rng.choice([16, 32, 64, 256]), **cache}


def _lens(case):
    """Tokens in the cache of each sequence, the queries among them."""
    n = case["seqs"]
    lo, hi = math.log(case["shortest"]), math.log(case["longest"])
    return [int(round(math.exp(lo + (hi - lo) * (i / (n - 1) if n > 1 else 1)))) for i in range(n)]


def _counts(case):
    n, q = case["seqs"], case["queries"]
    return [max(1, q * (i + 1) // n) for i in range(n)] if case["ragged"] else [q] * n


def work(case):
    op, dim = case["op"], case["dim"]
    size = 4 if case["dtype"] == "fp32" else 2
    if op == "rope":
        n = case["tokens"] * case["heads"]
        return {"bytes": n * case["rot"] * size * 2 + n * (dim - case["rot"]) * size * 2 + case["tokens"] * 4,
                "flops": 3 * n * case["rot"]}
    row = sum(dim * BITS[case[k]] // 8 + dim // case["group"] * 2 for k in ("klevels", "vlevels"))
    fwht = dim * int(math.log2(dim))
    if op == "load":
        n = case["tokens"] * case["heads"]
        return {"bytes": n * (row + 2 * dim * size) + case["tokens"] * 8, "flops": 2 * n * (fwht + 2 * dim)}
    if op == "store":
        n = case["tokens"] * case["heads"]
        return {"bytes": n * (2 * row + 4 * dim * size) + case["tokens"] * 12, "flops": 2 * n * (2 * fwht + 8 * dim) + 3 * n * case["rot"]}
    lens, counts = _lens(case), _counts(case)
    qh = case["heads"] * case["share"]
    pairs = 0
    for n, q in zip(lens, counts):
        pairs += q * (n - q) + (q * (q + 1) // 2)
    return {"bytes": sum(lens) * case["heads"] * row + 2 * sum(counts) * qh * dim * size, "flops": 4 * pairs * qh * dim}


# ---- the codebook: Lloyd-Max quantizer of N(0,1) --------------------------------------------

@functools.lru_cache(None)
def _book(levels):
    """(centroids, thresholds), float32 numpy: each centroid the mean of N(0,1) over its cell, each threshold
    the midpoint of its neighbours. Newton's method on that fixed point over the positive half; cell integrals
    by Gauss-Legendre, the last (infinite) cell by erfc."""
    half = levels // 2
    gx, gw = np.polynomial.legendre.leggauss(24)
    phi = lambda x: np.exp(-0.5 * x * x) / math.sqrt(2 * math.pi)  # noqa: E731
    c = np.array([(k + 0.5) * 2.5 / half for k in range(half)])
    for _ in range(4000):
        t = np.concatenate([[0.0], (c[1:] + c[:-1]) / 2])
        mass, mean = np.empty(half), np.empty(half)
        w = np.diff(t)
        x = t[:-1, None] + w[:, None] * (gx + 1) / 2
        mass[:-1] = (phi(x) @ gw) * w / 2
        mean[:-1] = ((x - t[:-1, None]) * phi(x)) @ gw * w / 2 / mass[:-1] + t[:-1]
        mass[-1] = 0.5 * math.erfc(t[-1] / math.sqrt(2))
        mean[-1] = phi(t[-1]) / mass[-1]
        if _ < 400:        # plain iteration towards the basin of Newton's method
            c = mean
            continue
        J = np.zeros((half, half))
        for k in range(half):
            if k:
                da = phi(t[k]) * (mean[k] - t[k]) / mass[k] / 2
                J[k, k] += da
                J[k, k - 1] += da
            if k + 1 < half:
                db = phi(t[k + 1]) * (t[k + 1] - mean[k]) / mass[k] / 2
                J[k, k] += db
                J[k, k + 1] += db
        d = np.linalg.solve(J - np.eye(half), c - mean)
        c = c + d
        if np.max(np.abs(d)) < 1e-14:
            break
    full = np.concatenate([-c[::-1], c])
    return full.astype(np.float32), ((full[1:] + full[:-1]) / 2).astype(np.float32)


@functools.lru_cache(None)
def _tables(levels, device):
    c, t = _book(levels)
    return torch.from_numpy(c).to(device), torch.from_numpy(t).to(device)


# ---- inputs -----------------------------------------------------------------------------------

def _signs(seed, dim):
    """Bit i set: s_i = -1 (the top bit of SplitMix64's output i)."""
    bits = []
    for i in range(dim):
        z = (seed + (i + 1) * 0x9E3779B97F4A7C15) & (2 ** 64 - 1)
        z = ((z ^ (z >> 30)) * 0xBF58476D1CE4E5B9) & (2 ** 64 - 1)
        z = ((z ^ (z >> 27)) * 0x94D049BB133111EB) & (2 ** 64 - 1)
        bits.append((z ^ (z >> 31)) >> 63)
    return np.array(bits, dtype=np.uint8)


def _pack(idx, bits):
    """[..., D] codes (uint8) -> int32 words, code j in bits [b j, b j + b) of the row."""
    if bits == 8:
        return idx.contiguous().view(torch.int32)
    one = (idx.unsqueeze(-1) >> torch.arange(bits, device=idx.device, dtype=torch.uint8)) & 1
    one = one.reshape(*idx.shape[:-1], -1, 8)
    byte = (one << torch.arange(8, device=idx.device, dtype=torch.uint8)).sum(-1, dtype=torch.uint8)
    return byte.contiguous().view(torch.int32)


def _frequencies(rot, stretch, device):
    """Radians per position (64 bits) and the gain: base 10000, and for a stretch > 1 the frequencies blended by
    their number of turns in the original 4096 positions (fewer than one: divided by the stretch; more than 32:
    as they are) with the gain 0.1 ln(stretch) + 1."""
    i = np.arange(0, rot, 2, dtype=np.float64)
    f = 10000.0 ** (-i / rot)
    if stretch > 1.0:
        turns = 4096.0 * f / (2 * math.pi)
        keep = np.clip((np.log(turns) / math.log(32.0)), 0.0, 1.0)
        f = f * keep + f / stretch * (1 - keep)
    gain = 0.1 * math.log(stretch) + 1.0 if stretch > 1.0 else 1.0
    return torch.from_numpy(f).to(device), gain


def _cache_rows(rows, dim, levels, group, gen, device):
    """Codes and scales of `rows` stored rows: the codes of N(0,1) values, lognormal group scales."""
    bits = BITS[levels]
    _, t = _tables(levels, device)
    codes = torch.empty((rows, dim * bits // 32), dtype=torch.int32, device=device)
    for a in range(0, rows, 1 << 19):
        n = min(1 << 19, rows - a)
        u = torch.randn((n, dim), generator=gen, device=device)
        codes[a:a + n] = _pack(torch.bucketize(u, t).to(torch.uint8), bits)
    scales = torch.exp(0.5 * torch.randn((rows, dim // group), generator=gen, device=device)).to(torch.float16)
    return codes, scales


def _cache(case, pages, page, gen, device, filled):
    st = {"pages": pages, "page": page}
    for part, levels, seed in (("k", case["klevels"], 11), ("v", case["vlevels"], 12)):
        dim, rows = case["dim"], pages * case["heads"] * page
        if filled:
            codes, scales = _cache_rows(rows, dim, levels, case["group"], gen, device)
        else:
            codes = torch.zeros((rows, dim * BITS[levels] // 32), dtype=torch.int32, device=device)
            scales = torch.zeros((rows, dim // case["group"]), dtype=torch.float16, device=device)
        bits = _signs(seed, dim)
        words = torch.from_numpy(np.packbits(bits, bitorder="little").view(np.int32).copy()).to(device)
        st[part] = {"codes": codes.view(pages, case["heads"] * page, -1), "scales": scales.view(pages, case["heads"] * page, -1),
                    "signs": words, "sign": torch.from_numpy(1.0 - 2.0 * bits.astype(np.float64)).to(device),
                    "levels": levels, "group": case["group"], "dim": dim, "seed": seed}
    return st


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    op, dt = case["op"], DTYPES[case["dtype"]]
    st = {"case": case}
    if op in ("rope", "store"):
        st["freq"], st["gain"] = _frequencies(case["rot"], case.get("stretch", 1.0), dev) if case["rot"] else (None, 1.0)
        st["positions"] = torch.randint(0, case["farthest"], (case["tokens"],), generator=gen, device=dev, dtype=torch.int32)
    if op == "rope":
        # the turned heads lie in a wider buffer, as in a fused projection's output (the value heads follow them)
        wide = torch.randn((case["tokens"], case["heads"] + max(1, case["heads"] // 5), case["dim"]), generator=gen, device=dev).to(dt)
        st["x"] = wide[:, :case["heads"]]
        return st
    if op in ("store", "load"):
        T, page = case["tokens"], PAGE
        pages = -(-T // page) + 2
        st["cache"] = _cache(case, pages, page, gen, dev, filled=op == "load")
        st["slots"] = torch.randperm(pages * page, generator=gen, device=dev)[:T].to(torch.int64)
        if op == "load" or T > 256:    # a prompt's tokens follow one another through scattered pages
            order = torch.randperm(pages, generator=gen, device=dev)[:, None] * page + torch.arange(page, device=dev)
            st["slots"] = order.reshape(-1)[:T].to(torch.int64).contiguous()
        if op == "store":
            for part in "kv":     # keys have a few channels far larger than the others
                x = torch.randn((T, case["heads"], case["dim"]), generator=gen, device=dev)
                if part == "k":
                    x[:, :, torch.randperm(case["dim"], generator=gen, device=dev)[:4]] *= 20.0
                st[part] = x.to(dt)
        return st
    lens, counts = _lens(case), _counts(case)
    page, qh = case["page"], case["heads"] * case["share"]
    need = [-(-n // page) for n in lens]
    pages = sum(need) + 1
    st["cache"] = _cache(case, pages, page, gen, dev, filled=True)
    order = torch.randperm(pages, generator=gen, device=dev).to(torch.int32)
    table = torch.full((len(lens), max(need)), -1, dtype=torch.int32, device=dev)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    st["table"] = table
    st["lens"] = torch.tensor(lens, dtype=torch.int32, device=dev)
    offsets = np.concatenate([[0], np.cumsum(counts)])
    st["offsets"] = torch.tensor(offsets, dtype=torch.int32, device=dev)
    st["most"] = max(counts)          # plain sizes, as a program that made the batch knows them
    st["q"] = torch.randn((int(offsets[-1]), qh, case["dim"]), generator=gen, device=dev).to(dt)
    st["scale"] = 1.0 / math.sqrt(case["dim"])
    st["tree"] = None
    if case["tree"]:
        # drafted token i hangs on an earlier one and sees itself and its ancestors
        words = (max(counts) + 31) // 32
        bits = np.zeros((int(offsets[-1]), words * 32), dtype=np.uint8)
        r = np.random.RandomState(seed % (2 ** 31))
        for b, n in enumerate(counts):
            for i in range(n):
                row = offsets[b] + i
                if i:
                    bits[row] = bits[offsets[b] + int(r.randint(max(0, i - 4), i))]
                bits[row, i] = 1
        st["tree"] = torch.from_numpy(np.packbits(bits, axis=1, bitorder="little").view(np.int32).copy()).to(dev)
    return st


# ---- the plain forms --------------------------------------------------------------------------

def _turn(x, positions, freq, gain, rot, interleaved, backward=False):
    """[T, heads, D] in 64 bits: pairs of the first `rot` elements turned by position * frequency."""
    a = positions.to(torch.float64)[:, None] * freq
    cos, sin = (torch.cos(a) * gain)[:, None], (torch.sin(a) * gain)[:, None]
    if backward:
        sin = -sin
    head, rest = x[..., :rot], x[..., rot:]
    if interleaved:
        p, q = head[..., 0::2], head[..., 1::2]
        turned = torch.stack((p * cos - q * sin, q * cos + p * sin), dim=-1).flatten(-2)
    else:
        p, q = head[..., :rot // 2], head[..., rot // 2:]
        turned = torch.cat((p * cos - q * sin, q * cos + p * sin), dim=-1)
    return torch.cat((turned, rest), dim=-1)


@functools.lru_cache(None)
def _hadamard(dim, dtype, device):
    h = torch.ones((1, 1), dtype=dtype, device=device)
    while h.shape[0] < dim:
        h = torch.cat((torch.cat((h, h), 1), torch.cat((h, -h), 1)), 0)
    return h / math.sqrt(dim)


def _decode(part, codes, scales):
    """Packed rows [..., words] -> c[code] * scale, fp32, in the rotated basis."""
    c, _ = _tables(part["levels"], codes.device)
    bits = BITS[part["levels"]]
    byte = codes.contiguous().view(torch.uint8)
    if bits == 8:
        idx = byte
    elif bits == 3:
        three = byte.view(*byte.shape[:-1], -1, 3).to(torch.int32)
        word = three[..., 0] | three[..., 1] << 8 | three[..., 2] << 16
        idx = (word.unsqueeze(-1) >> torch.arange(0, 24, 3, device=codes.device, dtype=torch.int32)) & 7
        idx = idx.flatten(-2)
    else:
        shift = torch.arange(0, 8, bits, device=codes.device, dtype=torch.uint8)
        idx = ((byte.unsqueeze(-1) >> shift) & ((1 << bits) - 1)).flatten(-2)
    w = c[idx.to(torch.int32)]
    return (w.unflatten(-1, (-1, part["group"])) * scales.to(torch.float32).unsqueeze(-1)).flatten(-2)


def _rows(cache, heads, slots):
    """Page of each slot and its rows [T, heads] inside the page."""
    page = slots // cache["page"]
    inside = torch.arange(heads, device=slots.device) * cache["page"] + (slots % cache["page"])[:, None]
    return page[:, None], inside


def _plain_store(st):
    case, cache = st["case"], st["cache"]
    at = _rows(cache, case["heads"], st["slots"])
    for name in "kv":
        part = cache[name]
        x = st[name].to(torch.float64)
        if name == "k" and case["rot"]:
            x = _turn(x, st["positions"], st["freq"], st["gain"], case["rot"], case["interleaved"])
        # 64 bits: a value next to a threshold must fall on the same side everywhere
        w = torch.matmul(x * part["sign"], _hadamard(case["dim"], torch.float64, x.device))
        g = w.unflatten(-1, (-1, part["group"]))
        r = g.square().mean(-1, keepdim=True).sqrt()
        u = torch.where(r > 0, g / r, torch.zeros_like(g)).flatten(-2).to(torch.float32)
        _, t = _tables(part["levels"], x.device)
        part["codes"][at] = _pack(torch.bucketize(u, t).to(torch.uint8), BITS[part["levels"]])
        part["scales"][at] = r.squeeze(-1).clamp(max=65504.0).to(torch.float16)


def _plain_load(st):
    case, cache = st["case"], st["cache"]
    at, out = _rows(cache, case["heads"], st["slots"]), []
    for name in "kv":
        part = cache[name]
        w = _decode(part, part["codes"][at], part["scales"][at])
        x = torch.matmul(w, _hadamard(case["dim"], torch.float32, w.device)) * part["sign"].to(torch.float32)
        out.append(x.to(DTYPES[case["dtype"]]))
    return tuple(out)


def _plain_attend(st):
    case, cache, q = st["case"], st["cache"], st["q"]
    seqs, heads, share, dim, most = case["seqs"], case["heads"], case["share"], case["dim"], st["most"]
    page, pages = case["page"], st["table"].shape[1]
    table = st["table"].clamp(min=0).to(torch.int64)
    L = pages * page
    kv = []
    for name in "kv":
        part = cache[name]
        codes = part["codes"].view(cache["pages"], heads, page, -1)[table]      # [seqs, pages, heads, page, words]
        scales = part["scales"].view(cache["pages"], heads, page, -1)[table]
        w = _decode(part, codes, scales).transpose(1, 2).reshape(seqs, heads, L, dim)
        kv.append(w)
    k, v = kv
    had = _hadamard(dim, torch.float32, q.device)
    # queries padded to the longest count of the batch
    i = torch.arange(most, device=q.device)
    n = (st["offsets"][1:] - st["offsets"][:-1]).to(torch.int64)
    row = (st["offsets"][:-1, None] + torch.minimum(i, n[:, None] - 1)).to(torch.int64)
    qr = torch.matmul(q.to(torch.float32) * cache["k"]["sign"].to(torch.float32), had)[row]
    qr = qr.view(seqs, most, heads, share, dim).permute(0, 2, 3, 1, 4).reshape(seqs, heads, share * most, dim)
    s = torch.matmul(qr, k.transpose(-1, -2).contiguous()).view(seqs, heads, share, most, L) * st["scale"]
    j = torch.arange(L, device=q.device)
    before = (st["lens"].to(torch.int64) - n)[:, None, None]
    if st["tree"] is None:
        seen = j <= before + i[None, :, None]
    else:
        own_j = (j - before).clamp(0, st["tree"].shape[1] * 32 - 1).expand(seqs, most, L)
        word = torch.gather(st["tree"][row], 2, own_j // 32)
        seen = (j < before) | ((word >> (own_j % 32).to(torch.int32)) & 1).bool()
    seen = seen & (j < st["lens"][:, None, None])
    s = s.masked_fill(~seen[:, None, None], -math.inf)
    top = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(top == -math.inf, torch.zeros_like(top), top))
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(seqs, heads, share * most, L), v).view(seqs, heads, share, most, dim)
    o = o / torch.where(total > 0, total, torch.ones_like(total))
    o = torch.matmul(o, had) * cache["v"]["sign"].to(torch.float32)
    o = o.permute(0, 3, 1, 2, 4).reshape(seqs * most, heads * share, dim)
    m = torch.arange(q.shape[0], device=q.device, dtype=st["offsets"].dtype)
    b = torch.searchsorted(st["offsets"], m, right=True) - 1
    return o[b * most + m - st["offsets"][b]].to(q.dtype)


# ---- one pass ---------------------------------------------------------------------------------

def _kv(st):
    """The cache's handle: descriptors around tensors in hand."""
    import rotation_lloyd_max_amd as tq
    parts = []
    for name in "kv":
        p = st["cache"][name]
        parts.append(tq.QWeight(p["codes"], p["scales"], p["signs"], p["levels"], p["group"], p["dim"],
                                p["codes"].shape[1], st["cache"]["pages"], p["seed"]))
    return tq.KVCache(parts[0], parts[1], st["case"]["heads"], st["cache"]["page"])


def run(state):
    case, op = state["case"], state["case"]["op"]
    if own:
        import rotation_lloyd_max_amd as tq
        rope = None
        if op in ("rope", "store") and case["rot"]:
            rope = tq.Rope(state["freq"], case["rot"], interleaved=case["interleaved"], gain=state["gain"])
        if op == "rope":
            return tq.rope(state["x"], state["positions"], rope, transposed=case["backward"])
        cache = _kv(state)
        if op == "attend":
            return tq.kv_attend(cache, state["q"], state["lens"], state["table"], q_offsets=state["offsets"],
                                tree=state["tree"], scale=state["scale"])
        if op == "store":
            tq.kv_store(cache, state["k"], state["v"], state["slots"], rope=rope,
                        positions=state["positions"] if rope is not None else None)
        return tq.kv_load(cache, state["slots"], out_dtype=DTYPES[case["dtype"]])
    if op == "rope":
        return _turn(state["x"].to(torch.float64), state["positions"], state["freq"], state["gain"], case["rot"],
                     case["interleaved"], case["backward"]).to(state["x"].dtype)
    if op == "attend":
        return _plain_attend(state)
    if op == "store":
        _plain_store(state)
    return _plain_load(state)


# ---- the definition in 64 bits ----------------------------------------------------------------

def _butterflies(x):
    """H x / sqrt(D) along the last axis by its log2(D) stages."""
    D, h = x.shape[-1], 1
    x = x.clone()
    while h < D:
        y = x.view(*x.shape[:-1], D // (2 * h), 2, h)
        x = torch.stack((y[..., 0, :] + y[..., 1, :], y[..., 0, :] - y[..., 1, :]), dim=-2).reshape(x.shape)
        h *= 2
    return x / math.sqrt(D)


def _values(part, codes, scales):
    """Rows in 64 bits from the bitstream, bit by bit."""
    bits, D = BITS[part["levels"]], part["dim"]
    idx = torch.zeros((*codes.shape[:-1], D), dtype=torch.int64, device=codes.device)
    for q in range(bits):
        p = torch.arange(D, device=codes.device) * bits + q
        idx += ((codes[..., p // 32].to(torch.int64) >> (p % 32)) & 1) << q
    c = torch.from_numpy(_book(part["levels"])[0].astype(np.float64)).to(codes.device)
    return c[idx] * scales.to(torch.float64).repeat_interleave(part["group"], dim=-1)


def _angle_pairs(x, st, back):
    """Each pair as a complex number times gain * exp(+-i position frequency)."""
    case = st["case"]
    rot = case["rot"]
    turn = torch.polar(torch.full((case["tokens"], rot // 2), st["gain"], dtype=torch.float64, device=x.device),
                       torch.outer(st["positions"].double(), st["freq"]) * (-1.0 if back else 1.0))[:, None]
    y = x.clone()
    first, second = (slice(0, rot, 2), slice(1, rot, 2)) if case["interleaved"] else (slice(0, rot // 2), slice(rot // 2, rot))
    z = torch.complex(x[..., first], x[..., second]) * turn
    y[..., first], y[..., second] = z.real, z.imag
    return y


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "rope":
        return _angle_pairs(st["x"].double(), st, case["backward"])
    cache, heads, D = st["cache"], case["heads"], case["dim"]
    if op in ("store", "load"):
        out = []
        for name in "kv":
            part = cache[name]
            if op == "load":
                page, inside = st["slots"] // cache["page"], st["slots"] % cache["page"]
                pick = [part[f].view(cache["pages"], heads, cache["page"], -1)[page, :, inside] for f in ("codes", "scales")]
                w = _values(part, *pick)
            else:
                x = st[name].double()
                if name == "k" and case["rot"]:
                    x = _angle_pairs(x, st, False)
                w = _butterflies(x * part["sign"])
                g = w.view(*w.shape[:-1], -1, part["group"])
                r = torch.sqrt((g * g).sum(-1, keepdim=True) / part["group"])
                u = torch.where(r > 0, g / r, 0.0 * g).reshape(w.shape).float()
                c, t = _book(part["levels"])
                idx = torch.searchsorted(torch.from_numpy(t).to(u.device), u)
                s = r.clamp(max=65504.0).half().double()
                w = (torch.from_numpy(c.astype(np.float64)).to(u.device)[idx].view(g.shape) * s).reshape(w.shape)
            out.append(_butterflies(w) * part["sign"])
        return tuple(out)
    lens, counts = _lens(case), _counts(case)
    if sum(n * q for n, q in zip(lens, counts)) * heads * case["share"] > 1 << 30:
        return None
    rows, at = [], 0
    for b, (n, q) in enumerate(zip(lens, counts)):
        need = -(-n // case["page"])
        pages = st["table"][b, :need].long()
        k, v = (_values(cache[p], *[cache[p][f].view(cache["pages"], heads, case["page"], -1)[pages].transpose(0, 1)
                                    .reshape(heads, need * case["page"], -1)[:, :n] for f in ("codes", "scales")]) for p in "kv")
        k, v = (_butterflies(x) * cache[p]["sign"] for x, p in ((k, "k"), (v, "v")))
        seen = torch.ones((q, n), dtype=torch.bool, device=k.device)
        for i in range(q) if case["tree"] else ():
            word = st["tree"][at + i].cpu().numpy().view(np.uint32)
            seen[i, n - q:] = torch.tensor([bool(word[j // 32] >> (j % 32) & 1) for j in range(q)], device=k.device)
        if not case["tree"]:
            seen[:, n - q:] = torch.tril(torch.ones((q, q), dtype=torch.bool, device=k.device))
        qq = st["q"][at:at + q].double().view(q, heads, case["share"], D)
        one = torch.empty((q, heads, case["share"], D), dtype=torch.float64, device=k.device)
        for h in range(heads):
            s = (qq[:, h].reshape(-1, D) @ k[h].t().contiguous()).view(q, case["share"], n) * st["scale"]
            s = s.masked_fill(~seen[:, None], -math.inf)
            one[:, h] = (torch.softmax(s, dim=-1).view(-1, n) @ v[h]).view(q, case["share"], D)
        rows.append(one.view(q, heads * case["share"], D))
        at += q
    return torch.cat(rows)
