"""Binding of include/tq_step.h: a decoding step's tables from the requests' lengths, the
verification of drafted tokens, and what stays of the step in the paged cache. Argument
marshalling only; like the calls of kv.py these run once per step, so their host side is short.
"""

import ctypes
import functools
from typing import NamedTuple, Optional

import torch

import rotation_lloyd_max_amd as _tq

from .kv import _KV, _apart, _as, _call

_P, _I32, _I64, _U32, _SZ = (ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_uint32,
                             ctypes.c_size_t)
_INT = ctypes.c_int


class _KVPool(ctypes.Structure):
    _fields_ = [("free_pages", ctypes.c_void_p), ("state", ctypes.c_void_p), ("pages", ctypes.c_int32)]


_PL = ctypes.POINTER(_KVPool)

# (name, restype, argtypes) for every function declared in include/tq_step.h
SIGNATURES = [
    ("tq_kv_plan", _INT,
     [_PL, _I32, _I32, _P, _P, _P, _I32, _I64, _P, _P, _P, _P, _P, _P, _P, _P, _I32, _P, _P]),
    ("tq_kv_keep", _INT, [_PL, _KV, _I32, _I32, _P, _P, _P, _P, _P, _I64, _P, _I32, _P, _P, _P]),
    ("tq_verify", _INT,
     [_P, _INT, _I64, _P, _INT, _I64, _U32, _I64, _I32, _P, _I64, _P, _P, _P, _P, _P, _P, _P, _P, _SZ, _P]),
    ("tq_verify_workspace", _SZ, [_I64, _I32, _I64, _I32, _U32]),
]

_KINDS = {"logits": 0, "probabilities": 1}
_NONE = ctypes.c_size_t(-1).value


def _same(t, dtype, device, name, shape=None):
    """t itself, checked to be what the call writes to or reads in place."""
    if t.get_device() != (-1 if device.index is None else device.index):
        raise ValueError(f"{name} is on {t.device}, the call runs on {device}")
    if t.dtype != dtype or not t.is_contiguous() or shape is not None and tuple(t.shape) != shape:
        raise ValueError(f"{name} must be a contiguous {dtype} tensor" + (f" of shape {shape}" if shape else ""))
    return t.data_ptr()


class KVPool:
    """The pages of a cache that no sequence holds: the first state[0] entries of `free` (int32
    [pages] on the device), the last of them given out first; state: int32 [2], the number of
    free pages and 0. The handle is of the tensors that it was made with."""

    def __init__(self, free, state):
        _same(free, torch.int32, free.device, "free")
        _same(state, torch.int32, free.device, "state", (2,))
        self.desc = _KVPool(free.data_ptr(), state.data_ptr(), free.numel())
        self.free, self.state, self.pages, self.device = free, state, free.numel(), free.device


def kv_pool(pages, device="cuda"):
    """A KVPool of all pages of a cache of `pages` pages, page 0 given out first."""
    free = torch.arange(pages - 1, -1, -1, dtype=torch.int32, device=device)
    return KVPool(free, torch.tensor([pages, 0], dtype=torch.int32, device=free.device))


class KVPlan(NamedTuple):
    """A step's tables (see kv_plan), in one allocation: clone what is kept for long."""
    slots: torch.Tensor
    positions: torch.Tensor
    q_offsets: torch.Tensor
    kv_lens: torch.Tensor
    status: torch.Tensor
    tree: Optional[torch.Tensor]


def _table(page_table, B, dev):
    if page_table.dim() != 2 or page_table.shape[0] != B:
        raise ValueError(f"page_table must be [{B}, pages of a sequence]")
    return _same(page_table, torch.int32, dev, "page_table"), page_table.shape[1]


def _left(left, dev):
    if left is None:
        return None
    if left.numel() != 1:
        raise ValueError("left= must be one element")
    return _same(left, torch.int32, dev, "left=")


def kv_plan(pool, lens, counts, page_table, rows, page_tokens, parents=None, tree_words=0, shift=None,
            left=None):
    """The tables of a step in which sequence b, with lens[b] tokens in the cache, gets counts[b]
    rows: new pages come off the pool into page_table (int32 [B, width], changed in place), and the
    KVPlan holds, on the device, slots (int64 [rows], for kv_store), positions (int32 [rows]),
    q_offsets and kv_lens (for kv_attend and verify), status (0: served; 1: too few pages; 2: too
    long for the table; 3: more rows than `rows`) and tree (int32 [rows, tree_words], for
    kv_attend, with tree_words > 0; else None). Rows without a sequence that is served have slot -1.
    rows: the size of the step's tensors, at least the sum of the counts that is to be served.
    parents (int [rows]): row i of a sequence follows its row parents[i] < i (drafted trees: the
    position is the depth's); None: chains. shift (int [B]): added to the positions. left (int32
    [1]): receives the free pages that are left, and the pool stays as it is (a look ahead)."""
    dev = pool.device
    B = lens.numel()
    lens = _as(lens, torch.int32, dev, "lens", (B,))
    counts = _as(counts, torch.int32, dev, "counts", (B,))
    table, width = _table(page_table, B, dev)
    if parents is not None:
        parents = _as(parents, torch.int32, dev, "parents", (rows,))
    if shift is not None:
        shift = _as(shift, torch.int32, dev, "shift", (B,))
    if rows < 0 or tree_words < 0:
        raise ValueError("rows and tree_words must not be negative")
    left = _left(left, dev)
    # one allocation for all of them (5 us less than one each, a quarter of the call)
    sizes = [2 * rows, rows, B + 1, B, B]
    if tree_words:
        sizes.append(rows * tree_words)
    parts = pool.free.new_empty((sum(sizes),)).split_with_sizes(sizes)
    p = KVPlan(parts[0].view(torch.int64), parts[1], parts[2], parts[3], parts[4],
               parts[5].view(rows, tree_words) if tree_words else None)
    _call(dev, _tq.lib().tq_kv_plan, pool.desc, page_tokens, B, lens.data_ptr(), counts.data_ptr(), table,
          width, rows, parents.data_ptr() if parents is not None else None,
          shift.data_ptr() if shift is not None else None, p.slots.data_ptr(), p.positions.data_ptr(),
          p.q_offsets.data_ptr(), p.kv_lens.data_ptr(), p.status.data_ptr(),
          p.tree.data_ptr() if tree_words and rows else None, tree_words if rows else 0, left)
    return p


def kv_keep(pool, lens, kept, page_table, page_tokens, q_offsets=None, status=None, path=None, cache=None,
            out=None, left=None):
    """What stays of a planned step: kept[b] of sequence b's rows (negative: the sequence ends and
    none of its tokens stays). Returns the new lengths, int32 [B] (out=: written there; it may be
    lens, int32, itself); pages behind them go back to the pool. q_offsets and status: the plan's
    (None: no rows were planned, none refused). path (verify's): the rows that stay, moved together
    in `cache`; None: the first kept[b] ones stay where they are. left: as in kv_plan."""
    dev = pool.device
    B = lens.numel()
    given = lens
    lens = _as(lens, torch.int32, dev, "lens", (B,))
    kept = _as(kept, torch.int32, dev, "kept", (B,))
    table, width = _table(page_table, B, dev)
    if q_offsets is not None:
        q_offsets = _as(q_offsets, torch.int32, dev, "q_offsets", (B + 1,))
    if status is not None:
        status = _as(status, torch.int32, dev, "status", (B,))
    if path is not None:
        if cache is None or q_offsets is None:
            raise ValueError("path= needs cache= and q_offsets=")
        if cache.device != dev:
            raise ValueError(f"the cache is on {cache.device}, the pool on {dev}")
        path = _as(path, torch.int32, dev, "path", (path.numel(),))
    if out is None:
        out = pool.free.new_empty((B,))
    else:
        at = _same(out, torch.int32, dev, "out=", (B,)) - given.data_ptr()
        if (at or given is not lens) and -4 * B < at < given.numel() * given.element_size() and not _apart(out, given):
            raise ValueError("out= must be lens itself (int32) or not overlap it")
    left = _left(left, dev)
    _call(dev, _tq.lib().tq_kv_keep, pool.desc, cache.desc if path is not None else None, page_tokens, B,
          lens.data_ptr(), q_offsets.data_ptr() if q_offsets is not None else None,
          status.data_ptr() if status is not None else None, kept.data_ptr(),
          path.data_ptr() if path is not None else None, path.numel() if path is not None else 0, table, width,
          out.data_ptr(), left)
    return out


class Verified(NamedTuple):
    """What verify found: kept [B] rows of each sequence that stay, the root among them; tokens
    [M], from offsets[b] the drafted tokens that stay and the new one (kept[b] in all), -1 behind
    them; path [M], from offsets[b] the rows that stay, -1 behind them. tokens and path behind the
    last sequence's rows hold anything. The three share one allocation, up to 64 KiB larger than
    they are: clone what is kept for long."""
    kept: torch.Tensor
    tokens: torch.Tensor
    path: torch.Tensor


@functools.lru_cache(maxsize=256)
def _verify_bytes(vocab, seqs, rows, drafted, flags):
    n = _tq.lib().tq_verify_workspace(vocab, seqs, rows, drafted, flags)
    if n == _NONE:
        raise _tq.TqError(-1, _tq.lib().tq_last_error().decode())
    return n


def verify_workspace(vocab, seqs, rows, drafted=False, target_kind="logits", draft_kind="logits"):
    """Bytes of workspace verify needs for `rows` rows of `seqs` sequences."""
    return _verify_bytes(vocab, seqs, rows, 1 if drafted else 0, _KINDS[target_kind] | _KINDS[draft_kind] << 1)


def _rows(t, M, V, dev, name):
    """Row stride of a distribution tensor [M, V] whose rows are contiguous."""
    if t.shape != (M, V):
        raise ValueError(f"{name} must be [{M}, {V}], got {tuple(t.shape)}")
    if t.device != dev:
        raise ValueError(f"{name} is on {t.device}, the call runs on {dev}")
    if V > 1 and t.stride(1) != 1 and M:  # (an empty tensor's strides may be anything)
        raise ValueError(f"the elements of a row of {name} must be contiguous")
    return t.stride(0)


def verify(target, tokens, uniforms, offsets, draft=None, parents=None, temperature=None,
           target_kind="logits", draft_kind="logits", ws=None):
    """Which drafted tokens stay, and the token after them, so that the tokens are distributed as the
    target's own (speculative sampling). Rows offsets[b] .. offsets[b + 1] are sequence b's: row 0
    its last token, the others drafted `tokens`, each following its row parents[i] < i (None: the row
    before). Row r of target ([M, vocab], float32 / bfloat16 / float16, "logits" or "probabilities")
    is the target's distribution of the token after r, row r of draft the one that the tokens of r's
    children were drawn from; without draft the drafted tokens are fixed ones. uniforms: float32 [M]
    numbers in [0, 1), a row's own for its test, the root's for the new token. temperature: float32
    [B] of the logits (None: 1); not above 0: greedy. Returns a Verified (see tq_step.h)."""
    dev = target.device
    if target.dim() != 2:
        raise ValueError("target must be [rows, vocab]")
    M, V = target.shape
    B = offsets.numel() - 1
    if B < 0:
        raise ValueError("offsets must hold the sequences' bounds")
    ts = _rows(target, M, V, dev, "target")
    ds, dd, dp = 0, 0, None
    if draft is not None:
        ds, dd, dp = _rows(draft, M, V, dev, "draft"), _tq._dt(draft), draft.data_ptr()
    offsets = _as(offsets, torch.int32, dev, "offsets", (B + 1,))
    tokens = _as(tokens, torch.int32, dev, "tokens", (M,))
    if parents is not None:
        parents = _as(parents, torch.int32, dev, "parents", (M,))
    up = _same(uniforms, torch.float32, dev, "uniforms", (M,))
    tp = _same(temperature, torch.float32, dev, "temperature", (B,)) if temperature is not None else None
    try:
        flags = _KINDS[target_kind] | _KINDS[draft_kind] << 1
    except KeyError:
        raise ValueError(f"target_kind and draft_kind must be one of {list(_KINDS)}") from None
    nbytes = _verify_bytes(V, B, M, 1 if draft is not None else 0, flags)
    if ws is not None and (ws.device != dev or not ws.is_contiguous() or ws.numel() * ws.element_size() < nbytes):
        raise ValueError(f"ws= must be a contiguous tensor of at least {nbytes} bytes on {dev}")
    words = 0
    if ws is None and nbytes <= 1 << 16:     # in one allocation with the outputs (1 us of 16), which keep it
        words = nbytes >> 2
    elif ws is None:
        ws = torch.empty(nbytes, dtype=torch.uint8, device=dev)
    whole = tokens.new_empty((words + B + 2 * M,))
    at = whole.data_ptr() + 4 * words
    _call(dev, _tq.lib().tq_verify, target.data_ptr(), _tq._dt(target), ts, dp, dd, ds, flags, V, B,
          offsets.data_ptr(), M, tokens.data_ptr(), parents.data_ptr() if parents is not None else None, up, tp,
          at, at + 4 * B, at + 4 * (B + M), ws.data_ptr() if ws is not None else whole.data_ptr(), nbytes)
    return Verified(*whole.split_with_sizes((words, B, M, M))[1:])
