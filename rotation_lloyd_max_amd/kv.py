"""Binding of include/tq_kv.h: rotary positions, and the paged compressed KV cache with its
write, read-back and attention. Argument marshalling only, like the package's other calls.

These calls run once per layer and decoded token, so what a call does on the host is kept
short: the cache's descriptor is checked and built once, in KVCache, and the device guard
is entered only where the tensors' device is not the current one.
"""

import ctypes
from dataclasses import dataclass

import numpy as np
import torch

import rotation_lloyd_max_amd as _tq

_P, _I32, _I64, _U32, _SZ = (ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_uint32,
                             ctypes.c_size_t)
_INT, _F32, _F64 = ctypes.c_int, ctypes.c_float, ctypes.c_double


class _KVCache(ctypes.Structure):
    _fields_ = [("k", _tq._QWeight), ("v", _tq._QWeight),
                ("heads", ctypes.c_int32), ("page_tokens", ctypes.c_int32)]


class _RopeParams(ctypes.Structure):
    _fields_ = [("inv_freq", ctypes.c_void_p), ("rot_dim", ctypes.c_int32),
                ("interleaved", ctypes.c_int32), ("gain", ctypes.c_double)]


_KV, _RP = ctypes.POINTER(_KVCache), ctypes.POINTER(_RopeParams)

# (name, restype, argtypes) for every function declared in include/tq_kv.h
SIGNATURES = [
    ("tq_rope_frequencies", _INT, [_I32, _F64, _I32, _F64, _F64, _P, _P]),
    ("tq_rope", _INT, [_P, _INT, _I64, _I32, _I32, _I64, _I64, _P, _RP, _U32, _P, _I64, _I64, _P]),
    ("tq_kv_store", _INT, [_KV, _P, _P, _INT, _I64, _I64, _I64, _I64, _I64, _P, _RP, _P, _P]),
    ("tq_kv_load", _INT, [_KV, _P, _I64, _P, _P, _INT, _P]),
    ("tq_kv_attend", _INT, [_KV, _P, _INT, _I32, _I64, _I32, _P, _I64, _P, _P, _I32, _P, _I32, _F32,
                            _P, _INT, _P, _SZ, _P]),
    ("tq_kv_attend_workspace", _SZ, [_KV, _I32, _I32, _I64]),
]

ROPE_SCALING = {None: 0, "linear": 1, "ntk": 2, "yarn": 3}
_TRANSPOSED = 1
_BITS = {4: 2, 8: 3, 16: 4, 256: 8}


def _call(device, fn, *args):
    """fn(*args, stream) on `device`'s current stream, with that device current."""
    if device.type != "cuda":
        raise ValueError(f"the tensors must be on a GPU, not on {device}")
    if device.index == torch.cuda.current_device():
        _tq._check(fn(*args, _stream(device)))
    else:
        with torch.cuda.device(device):
            _tq._check(fn(*args, _stream(device)))


# the current stream's handle; torch's own short cut where it has it (2 us less than by the Stream
# object, a sixth of a small call)
if hasattr(torch._C, "_cuda_getCurrentRawStream"):
    def _stream(device):
        return torch._C._cuda_getCurrentRawStream(device.index)
else:
    def _stream(device):
        return torch.cuda.current_stream(device).cuda_stream


def _as(t, dtype, device, name, shape=None):
    """t as a contiguous tensor of dtype on device (the call's index arrays). Values that dtype does not
    hold become its nearest: a page or a length far outside stays outside, where plain conversion
    would wrap it to another page's."""
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, the call runs on {device}")
    if shape is not None and tuple(t.shape) != shape:
        raise ValueError(f"{name} must have shape {shape}, got {tuple(t.shape)}")
    if t.dtype != dtype:
        if t.dtype.is_floating_point or t.dtype.is_complex or t.dtype == torch.bool:
            raise TypeError(f"{name} must hold integers, got {t.dtype}")
        if t.dtype == torch.uint64:     # (from 2^63 on it would turn negative; elementwise calls do not take it)
            t = t.view(torch.int64)
            t = torch.where(t < 0, torch.iinfo(torch.int64).max, t)
        if dtype == torch.int32 and t.dtype in (torch.int64, torch.uint32):
            t = t.to(torch.int64).clamp(-2 ** 31, 2 ** 31 - 1)
        t = t.to(dtype)
    return t if t.is_contiguous() else t.contiguous()


def _no_gradient(name):
    """The library's calls are outside autograd: refuse rather than return a detached result."""
    if torch.is_grad_enabled():
        raise ValueError(f"{name} records no gradient: call it on detached tensors or under torch.no_grad()")


@dataclass
class Rope:
    """Rotary positions: inv_freq float64 [rot_dim / 2] on the device (radians per position),
    pairs (i, i + rot_dim / 2) or, interleaved, (2i, 2i + 1), the turned pair scaled by gain."""
    inv_freq: torch.Tensor
    rot_dim: int
    interleaved: bool = False
    gain: float = 1.0

    def desc(self, device):
        f = self.inv_freq
        if f.dtype != torch.float64 or f.numel() * 2 != self.rot_dim or not f.is_contiguous():
            raise ValueError("inv_freq must be a contiguous float64 tensor of rot_dim / 2 elements")
        if f.device != device:
            raise ValueError(f"inv_freq is on {f.device}, the call runs on {device}")
        return _RopeParams(f.data_ptr(), self.rot_dim, 1 if self.interleaved else 0, self.gain)


def rope_frequencies(rot_dim, base=10000.0, scaling=None, stretch=1.0, original=4096,
                     interleaved=False, device="cuda"):
    """A Rope of the frequencies base^(-2i / rot_dim), stretched for texts `stretch` times as
    long as `original` positions: scaling None, "linear", "ntk" or "yarn" (see tq_kv.h)."""
    if scaling not in ROPE_SCALING:
        raise ValueError(f"scaling must be one of {list(ROPE_SCALING)}")
    f = np.zeros(max(1, rot_dim // 2), dtype=np.float64)
    gain = ctypes.c_double(1.0)
    _tq._check(_tq.lib().tq_rope_frequencies(rot_dim, base, ROPE_SCALING[scaling], stretch,
                                             original, f.ctypes.data, ctypes.addressof(gain)))
    return Rope(torch.from_numpy(f).to(device), rot_dim, interleaved, gain.value)


def _head_strides(t, name):
    """(token, head) strides of a [tokens, heads, dim] tensor with contiguous heads."""
    if t.dim() != 3:
        raise ValueError(f"{name} must be [tokens, heads, head_dim]")
    s = t.stride()
    if s[2] != 1 and t.shape[2] > 1 and t.numel():  # (an empty tensor's strides may be anything)
        raise ValueError(f"the elements of a head of {name} must be contiguous")
    return s[0], s[1]


def _overlaps_itself(t):
    """Whether two (token, head) vectors of t can share an element."""
    (n, h, d), (a, b, _) = t.shape, t.stride()
    if n * h <= 1:
        return False
    if n == 1:
        return b < d
    if h == 1:
        return a < d
    inner, outer, count = (b, a, h) if b <= a else (a, b, n)
    return inner < d or outer < inner * (count - 1) + d


def _span(t):
    """(first, last + 1) byte that the elements of t lie between."""
    n = 1 + sum((d - 1) * s for d, s in zip(t.shape, t.stride()))
    return t.data_ptr(), t.data_ptr() + n * t.element_size()


def _apart(a, b):
    """Whether the memory between a's first and last element and that of b's do not meet."""
    if not a.numel() or not b.numel():
        return True
    (a0, a1), (b0, b1) = _span(a), _span(b)
    return a1 <= b0 or b1 <= a0


def _vectors_meet(x, y):
    """Whether a (token, head) vector of x and one of y, of one shape and type, share a byte."""
    (n, h, d), size = x.shape, x.element_size()
    if _apart(x, y):
        return False
    width, step, first = d * size, y.data_ptr() - x.data_ptr(), lambda t: tuple(s * size for s in t.stride()[:2])
    (xt, xh), (yt, yh) = first(x), first(y)
    if (n == 1 or xt == yt) and (h == 1 or xh == yh):
        # one grid moved by `step`: the differences of its vectors' places, i tokens and j heads
        j = step + np.arange(1 - h, h, dtype=np.int64) * xh
        i = np.clip(-j // xt, 1 - n, n - 1) if xt else np.zeros_like(j)
        near = np.minimum(np.abs(j + i * xt), np.abs(j + np.minimum(i + 1, n - 1) * xt))
        return bool((near < width).any())
    a = np.sort((np.arange(n, dtype=np.int64)[:, None] * xt + np.arange(h, dtype=np.int64) * xh).ravel())
    b = (step + np.arange(n, dtype=np.int64)[:, None] * yt + np.arange(h, dtype=np.int64) * yh).ravel()
    k = np.searchsorted(a, b)
    above = a[np.minimum(k, len(a) - 1)] - b
    below = b - a[np.maximum(k - 1, 0)]
    return bool(((np.abs(above) < width) | (np.abs(below) < width)).any())


def rope(x, positions, rope, transposed=False, out=None):
    """x ([tokens, heads, head_dim], the elements of a head contiguous, any token and head
    strides) with rotary positions applied. out=x turns it in place; another out= must not
    overlap x. transposed: the negative angle (the gradient of the call). Not recorded by
    autograd: refused where x requires grad, unless under torch.no_grad() (as in the forward of an
    autograd.Function, whose backward is the transposed call)."""
    if x.requires_grad or out is not None and out.requires_grad:
        _no_gradient("rope")
    xs = _head_strides(x, "x")
    dev = x.device
    positions = _as(positions, torch.int32, dev, "positions", (x.shape[0],))
    if out is None:
        out = torch.empty_like(x)  # (half a microsecond less than torch.empty)
        if not out.is_contiguous():
            out = torch.empty(x.shape, dtype=x.dtype, device=dev)
        os_ = out.stride()
    elif out.shape != x.shape or out.dtype != x.dtype or out.device != dev:
        raise ValueError("out= must have x's shape, dtype and device")
    elif _overlaps_itself(out):
        raise ValueError("out= must not overlap itself")
    elif (out.data_ptr() != x.data_ptr() or out.stride() != x.stride()) and _vectors_meet(x, out):
        raise ValueError("out= must be x itself or not overlap it")
    else:
        os_ = _head_strides(out, "out")
    r = rope.desc(dev)
    _call(dev, _tq.lib().tq_rope, x.data_ptr(), _tq._dt(x), x.shape[0], x.shape[1], x.shape[2],
          xs[0], xs[1], positions.data_ptr(), r, _TRANSPOSED if transposed else 0, out.data_ptr(),
          os_[0], os_[1])
    return out


def _half(w, name, index):
    """The descriptor of a cache's half. The library reads and writes E * N rows through its
    pointers: its tensors must hold them, on the device `index`."""
    codes, scales, sg, K = w.codes, w.scales, w.signs, w.K
    n = w.E * w.N * K
    if (codes.dtype != torch.int32 or codes.numel() * 32 != n * _BITS.get(w.levels, 0)
            or not codes.is_contiguous()):
        raise ValueError(f"{name}.codes must be a contiguous int32 tensor of {w.E * w.N} packed rows")
    if scales.dtype != torch.float16 or scales.numel() * w.group != n or not scales.is_contiguous():
        raise ValueError(f"{name}.scales must be a contiguous float16 tensor of {w.E * w.N} rows "
                         "of K / group scales")
    if sg.dtype != torch.int32 or sg.numel() * 32 < K or not sg.is_contiguous():
        raise ValueError(f"{name}.signs must hold {K} sign bits")
    if not codes.get_device() == scales.get_device() == sg.get_device() == index:
        raise ValueError(f"the tensors of a cache must be on one device ({name} is not on {index})")
    return _tq._QWeight(codes.data_ptr(), scales.data_ptr(), sg.data_ptr(), w.levels, w.group, K, w.N, w.E)


class KVCache:
    """A paged compressed cache: k and v are QWeights of E = pages experts of N = heads *
    page_tokens rows of head_dim K; row h * page_tokens + t of a page is its token t of head h.
    Slot page * page_tokens + t names a token's place. The handle is of the tensors that k
    and v held when it was made."""

    def __init__(self, k, v, heads, page_tokens):
        index = k.codes.get_device()
        self.desc = _KVCache(_half(k, "k", index), _half(v, "v", index), heads, page_tokens)
        self.device = k.codes.device
        self._keep = (k.codes, k.scales, k.signs, v.codes, v.scales, v.signs)
        self.k, self.v, self.heads, self.page_tokens = k, v, heads, page_tokens
        self.head_dim = k.K


def kv_cache(pages, heads, head_dim, page_tokens=64, k_levels=256, v_levels=8, k_group=64,
             v_group=64, k_seed=0, v_seed=0, device="cuda"):
    """A KVCache of zero rows."""
    halves = []
    for levels, group, seed in ((k_levels, k_group, k_seed), (v_levels, v_group, v_seed)):
        rows = heads * page_tokens
        codes = torch.zeros((pages, rows, _tq.words_per_row(head_dim, levels)), dtype=torch.int32,
                            device=device)
        scales = torch.zeros((pages, rows, head_dim // group), dtype=torch.float16, device=device)
        with torch.cuda.device(codes.device):
            sg = _tq.signs(seed, head_dim, codes.device)
        halves.append(_tq.QWeight(codes, scales, sg, levels, group, head_dim, rows, pages, seed))
    return KVCache(halves[0], halves[1], heads, page_tokens)


def kv_store(cache, k, v, slots, rope=None, positions=None):
    """Quantize the new tokens' keys and values ([tokens, heads, head_dim], the elements of a
    head contiguous) into their slots of the cache (a slot outside it, such as -1, is skipped;
    each other one at most once); with rope, the keys are turned at `positions` first."""
    dev = cache.device
    n = k.shape[0]
    shape = (n, cache.heads, cache.head_dim)
    if tuple(k.shape) != shape or tuple(v.shape) != shape or v.dtype != k.dtype:
        raise ValueError(f"k and v must be [tokens, {cache.heads}, {cache.head_dim}] of one dtype")
    if k.device != dev or v.device != dev:
        raise ValueError(f"k and v must be on the cache's device {dev}")
    ks, vs = _head_strides(k, "k"), _head_strides(v, "v")
    slots = _as(slots, torch.int64, dev, "slots", (n,))
    r = pos = None
    if rope is not None:
        if positions is None:
            raise ValueError("rope needs the tokens' positions")
        positions = _as(positions, torch.int32, dev, "positions", (n,))
        r, pos = rope.desc(dev), positions.data_ptr()
    _call(dev, _tq.lib().tq_kv_store, cache.desc, k.data_ptr(), v.data_ptr(), _tq._dt(k), n, ks[0],
          ks[1], vs[0], vs[1], slots.data_ptr(), r, pos)


def kv_load(cache, slots, out_dtype=torch.bfloat16, k_out=None, v_out=None, keys=True, values=True):
    """(keys, values) of the tokens in `slots`, [tokens, heads, head_dim] each, dequantized and
    rotated back; a slot outside the cache gives NaN rows. keys=False or values=False leaves
    that half out (None)."""
    dev = cache.device
    slots = _as(slots, torch.int64, dev, "slots", (slots.numel(),))
    shape = (slots.numel(), cache.heads, cache.head_dim)
    for o in (k_out, v_out):
        if o is not None and o.dtype != out_dtype:
            raise ValueError(f"k_out= and v_out= must be {out_dtype}")
    k = _tq._out(k_out, shape, out_dtype, dev) if keys else None
    if values:
        v = torch.empty_like(k) if keys and k_out is None and v_out is None else _tq._out(v_out, shape, out_dtype, dev)
    else:
        v = None
    if k_out is not None and v_out is not None and keys and values and not _apart(k, v):
        raise ValueError("k_out= and v_out= must not overlap")
    if out_dtype not in _tq._DT:
        raise TypeError(f"unsupported dtype {out_dtype}")
    _call(dev, _tq.lib().tq_kv_load, cache.desc, slots.data_ptr(), shape[0],
          k.data_ptr() if keys else None, v.data_ptr() if values else None, _tq._DT[out_dtype])
    return k, v


def kv_attend_workspace(cache, q_heads, seqs, rows):
    """Bytes of workspace kv_attend needs for `rows` queries of `seqs` sequences."""
    n = _tq.lib().tq_kv_attend_workspace(cache.desc, q_heads, seqs, rows)
    if n == ctypes.c_size_t(-1).value:
        raise _tq.TqError(-1, _tq.lib().tq_last_error().decode())
    return n


def kv_attend(cache, q, kv_lens, page_table, q_offsets=None, tree=None, scale=None,
              out_dtype=None, out=None, ws=None):
    """Attention of q ([M, q_heads, head_dim], bf16 or fp16, the heads of a row contiguous)
    over the cache: sequence b has kv_lens[b] tokens in the pages page_table[b], the last of
    them its queries' own; q_offsets [B + 1] bounds the sequences' rows of q (None: M / B rows
    each). Causal, or with tree (int32 words [M, words]) bit j of a row's mask for each of the
    sequence's own tokens j. scale: 1 / sqrt(head_dim) by default. Returns [M, q_heads,
    head_dim] in out_dtype (q's by default; out= may be q itself, and must not overlap it otherwise); rows behind q_offsets[B] are not written (without
    out= they hold whatever the memory held). Not recorded by autograd: refused where q requires
    grad, unless under torch.no_grad()."""
    if q.requires_grad or out is not None and out.requires_grad:
        _no_gradient("kv_attend")
    dev = cache.device
    if q.dim() != 3 or q.shape[2] != cache.head_dim:
        raise ValueError(f"q must be [M, q_heads, {cache.head_dim}]")
    M, H, D = q.shape
    stride = q.stride()
    if M and (stride[2] != 1 or (H > 1 and stride[1] != D)):
        raise ValueError("the heads of a query row must be contiguous")
    if q.device != dev:
        raise ValueError(f"q is on {q.device}, the cache on {dev}")
    B = kv_lens.numel()
    kv_lens = _as(kv_lens, torch.int32, dev, "kv_lens", (B,))
    if page_table.dim() != 2:
        raise ValueError("page_table must be [sequences, pages of a sequence]")
    width = page_table.shape[1]
    page_table = _as(page_table, torch.int32, dev, "page_table", (B, width))
    if q_offsets is not None:
        q_offsets = _as(q_offsets, torch.int32, dev, "q_offsets", (B + 1,))
    words = 0
    if tree is not None:
        if tree.dim() != 2 or tree.dtype != torch.int32:
            raise ValueError("tree must be int32 words [M, words]")
        words = tree.shape[1]
        tree = _as(tree, torch.int32, dev, "tree", (M, words))
    if out is None:
        if q.is_contiguous() and (out_dtype is None or out_dtype == q.dtype):
            out = torch.empty_like(q)
        else:
            out = torch.empty((M, H, D), dtype=out_dtype or q.dtype, device=dev)
    else:
        if out_dtype is not None and out.dtype != out_dtype:
            raise ValueError(f"out= must be {out_dtype}")
        out = _tq._out(out, (M, H, D), out.dtype, dev)
        same = out.data_ptr() == q.data_ptr() and out.dtype == q.dtype and q.is_contiguous()
        if not same and not _apart(out, q):
            raise ValueError("out= must be q itself (contiguous, of its type) or not overlap it")
    nbytes = kv_attend_workspace(cache, H, B, M)
    if ws is None:
        ws = torch.empty(nbytes, dtype=torch.uint8, device=dev) if nbytes else None
    elif ws.device != dev or not ws.is_contiguous() or ws.numel() * ws.element_size() < nbytes:
        raise ValueError(f"ws= must be a contiguous tensor of at least {nbytes} bytes on {dev}")
    _call(dev, _tq.lib().tq_kv_attend, cache.desc, q.data_ptr(), _tq._dt(q), H,
          stride[0] if M > 1 else H * D, B, q_offsets.data_ptr() if q_offsets is not None else None, M,
          kv_lens.data_ptr(), page_table.data_ptr(), width,
          tree.data_ptr() if tree is not None else None, words, D ** -0.5 if scale is None else scale,
          out.data_ptr(), _tq._dt(out), ws.data_ptr() if ws is not None else None, nbytes)
    return out
