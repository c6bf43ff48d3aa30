"""The operators around the routed experts in a decoder layer (the C ABI in
include/moe_layer.h): residual addition with root-mean-square norm, projections
with NVFP4 weights, the paged 8-bit key/value cache with its append (rotation
included) and the attention over it; and what speculative decoding and several samples
of a prompt ask of them (include/moe_speculate.h): trees of new tokens, the compaction
of the cache to the accepted ones, the fork of sequences, the sampling of tokens
from logits.

Argument marshalling only, as in `binding`: every step of the computation runs
in the library's sm_103a kernels, on `stream` or the current stream; outputs
that the caller does not pass are allocated on that stream.  Tensors and stream
belong to the current device.  A call that fails raises MoeError; there is no
fallback.
"""
from __future__ import annotations

import ctypes as C
import math

import torch

from . import binding
from .binding import MOE_ERR_INVALID_ARG, MOE_OK, MoeError, _check, _need

PAGE = 64        # tokens of a cache page
MAX_SEQS = 512   # sequences of a step
MAX_TREE = 256   # new tokens of a sequence that are a tree
MAX_VOCAB = 262144  # logits of a row that tokens are sampled from
_BF16 = (torch.bfloat16,)

_P, _I, _S, _L, _F = C.c_void_p, C.c_int, C.c_size_t, C.c_int64, C.c_float


class moe_kv_desc(C.Structure):
    _fields_ = [("n_pages", _I), ("q_heads", _I), ("kv_heads", _I), ("head_dim", _I), ("k_dev", _P), ("v_dev", _P),
                ("k_scale_dev", _P), ("v_scale_dev", _P), ("rot_dim", _I), ("rot_interleaved", _I),
                ("rope_positions", _I), ("rope_dev", _P), ("device", _I)]


class moe_kv_batch(C.Structure):
    _fields_ = [("q_off_dev", _P), ("kv_len_dev", _P), ("pages_dev", _P), ("max_pages", _I), ("B", _I), ("N", _I),
                ("max_q", _I)]


class moe_sample_desc(C.Structure):
    _fields_ = [("logits_dev", _P), ("stride", _L), ("bf16", _I), ("T", _I), ("V", _I), ("u_dev", _P),
                ("temperature_dev", _P), ("temperature", _F), ("top_k_dev", _P), ("top_k", _I), ("top_p_dev", _P),
                ("top_p", _F), ("min_p_dev", _P), ("min_p", _F), ("token_dev", _P), ("prob_dev", _P)]


# Every function include/moe_layer.h declares: name -> (restype, argtypes).
SIGNATURES = {
    "moe_norm": (_I, [_P, _I, _L, _P, _P, _P, _F, _P, _P, _P, _I, _I, _P]),
    "moe_linear": (_I, [_P, _P, _P, _I, _I, _P, _L, _P, _I, _I, _P]),
    "moe_kv_create": (_I, [C.POINTER(moe_kv_desc), C.POINTER(C.c_void_p)]),
    "moe_kv_destroy": (None, [_P]),
    "moe_kv_workspace_bytes": (_S, [_P]),
    "moe_kv_workspace_init": (_I, [_P, _P, _S, _P]),
    "moe_kv_append": (_I, [_P, _P, _L, _P, _L, _P, _L, _P, C.POINTER(moe_kv_batch), _P, _P]),
    "moe_kv_attend": (_I, [_P, _P, _L, _F, _P, C.POINTER(moe_kv_batch), _P, _P]),
    "moe_kv_check": (_I, [_P, _P, _P]),
}
# And include/moe_speculate.h.
SPECULATE_SIGNATURES = {
    "moe_kv_append_tree": (_I, [_P, _P, _L, _P, _L, _P, _L, _P, C.POINTER(moe_kv_batch), _P, _P, _P]),
    "moe_kv_attend_tree": (_I, [_P, _P, _L, _F, _P, C.POINTER(moe_kv_batch), _P, _P, _P]),
    "moe_kv_compact": (_I, [_P, _P, _P, _I, _P, C.POINTER(moe_kv_batch), _P, _P]),
    "moe_kv_fork": (_I, [_P, _P, _P, _I, _P, _P, _I, _I, _P, _P, _P, _P]),
    "moe_sample": (_I, [C.POINTER(moe_sample_desc), _P]),
}
_ready = None


def _library():
    """The library, with both headers' functions prototyped."""
    global _ready
    lib = binding.load_library()
    if _ready is not lib:
        for name, (res, args) in {**SIGNATURES, **SPECULATE_SIGNATURES}.items():
            fn = getattr(lib, name)
            fn.restype, fn.argtypes = res, args
        _ready = lib
    return lib


def _bad(msg):
    return MoeError(MOE_ERR_INVALID_ARG, msg)


# The checks below run on every call, and the host bounds the small ones: what is
# right passes in one expression of few lookups, and the reason is looked for where
# that fails.
_Tensor, _INT32, _FLOAT32 = torch.Tensor, torch.int32, torch.float32


def _rows(t, dtypes, tail, name, n=None):
    """Row stride, in elements, of a CUDA tensor [n, *tail] (one or two dimensions of
    tail) whose rows are contiguous (only dimension 0 may be strided)."""
    if type(t) is _Tensor and t.is_cuda and t.dtype in dtypes:
        shape, stride = t.shape, t.stride()
        if len(tail) == 2:
            if len(shape) == 3 and shape[1:] == tail and stride[2] == 1 and stride[1] == tail[1] and (n is None or shape[0] == n):
                return stride[0] if shape[0] > 1 else tail[0] * tail[1]
        elif len(shape) == 2 and shape[1] == tail[0] and stride[1] == 1 and (n is None or shape[0] == n):
            return stride[0] if shape[0] > 1 else max(tail[0], 1)
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise _bad(f"{name} must be a CUDA tensor")
    if t.dtype not in dtypes:
        raise _bad(f"{name} must be {' or '.join(map(str, dtypes))}, got {t.dtype}")
    shape = t.shape
    if len(shape) != len(tail) + 1 or shape[1:] != tail or (n is not None and shape[0] != n):
        raise _bad(f"{name} {tuple(shape)} is not {('T' if n is None else n, *tail)}")
    stride, row = t.stride(), 1
    for d in range(len(tail), 0, -1):
        if stride[d] != row and shape[d] != 1:
            raise _bad(f"a row of {name} must be contiguous (strides {stride})")
        row *= shape[d]
    return stride[0] if shape[0] > 1 else max(row, 1)


def _need_out(t, dtype, shape, device, name):
    if not (isinstance(t, _Tensor) and t.dtype is dtype and t.shape == shape and t.device == device and t.is_contiguous()):
        _need(t, dtype, name)
        raise _bad(f"{name} {tuple(t.shape)} on {t.device} is not {tuple(shape)} on {device}")


def _empty(shape, dtype, device, stream):
    """Allocated on the stream that the call runs on, so that its memory is not
    handed out again while the work queued there may still use it."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _handle(stream, device):
    """cudaStream_t of `stream`, or of the device's current stream.  The kernels
    launch on the current device, which has to be the tensors'."""
    if device.index != torch.cuda.current_device():
        raise _bad(f"tensors on {device}, but the current device is cuda:{torch.cuda.current_device()}")
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(device.index)
    if stream.device != device:
        raise _bad(f"a stream of {stream.device} for tensors on {device}")
    return stream.cuda_stream


def _ptr(t):
    return None if t is None else t.data_ptr()


def _same_device(device, **tensors):
    for name, t in tensors.items():
        if t is not None and t.device != device:
            raise _bad(f"{name} is on {t.device}, expected {device}")


def add_rms_norm(x, weight, residual=None, eps: float = 1e-6, residual_out=None, out=None, outputs: str = "bf16",
                 out_q=None, out_scale=None, stream=None):
    """s = x + residual, y = s / sqrt(mean(s^2) + eps) * weight over the last
    dimension (moe_norm).  x: float32 or bfloat16 [T, H] (rows may be strided),
    such as an expert step's output; weight: bfloat16 [H]; residual: bfloat16
    [T, H], replaced by bf16(s) unless residual_out takes it.  outputs: "bf16"
    returns y, "e4m3" returns (codes as float8_e4m3fn [T, H], scales float32
    [T, H / 128]), "both" returns (y, codes, scales)."""
    if outputs not in ("bf16", "e4m3", "both"):
        raise _bad(f"outputs={outputs!r} is not bf16, e4m3 or both")
    if not isinstance(x, torch.Tensor) or x.dim() != 2:
        raise _bad("x must be a CUDA tensor [T, H]")
    T, H = x.shape
    stride = _rows(x, (torch.float32, torch.bfloat16), (H,), "x")
    dev = x.device
    handle = _handle(stream, dev)
    _need_out(weight, torch.bfloat16, (H,), dev, "weight")
    if residual is None:
        if residual_out is not None:
            raise _bad("residual_out without a residual")
    else:
        _need_out(residual, torch.bfloat16, (T, H), dev, "residual")
        if residual_out is None:
            residual_out = residual
        else:
            _need_out(residual_out, torch.bfloat16, (T, H), dev, "residual_out")
    if outputs == "e4m3":
        if out is not None:
            raise _bad("out with outputs='e4m3'")
    elif out is None:
        out = _empty((T, H), torch.bfloat16, dev, stream)
    else:
        _need_out(out, torch.bfloat16, (T, H), dev, "out")
    if outputs == "bf16":
        if out_q is not None or out_scale is not None:
            raise _bad("out_q or out_scale with outputs='bf16'")
    else:
        if out_q is None:
            out_q = _empty((T, H), torch.float8_e4m3fn, dev, stream)
        if out_scale is None:
            out_scale = _empty((T, H // 128), torch.float32, dev, stream)
        _need_out(out_q, torch.float8_e4m3fn, (T, H), dev, "out_q")
        _need_out(out_scale, torch.float32, (T, H // 128), dev, "out_scale")
    st = _library().moe_norm(x.data_ptr(), x.dtype == torch.float32, stride, _ptr(residual), _ptr(residual_out),
                             weight.data_ptr(), eps, _ptr(out), _ptr(out_q), _ptr(out_scale), T, H, handle)
    if st != MOE_OK:
        _check(st)
    return out if outputs == "bf16" else ((out_q, out_scale) if outputs == "e4m3" else (out, out_q, out_scale))


class Nvfp4Linear:
    """y = x W^T for NVFP4 weights (moe_linear): q uint8 [N, K/2], s uint8
    [N, K/16], ts float32 [N] (a tensor scale for each row; one for the whole
    weight may be given as [1]).  Keeps the tensors alive."""

    def __init__(self, q, s, ts):
        _need(q, torch.uint8, "q")
        _need(s, torch.uint8, "s")
        _need(ts, torch.float32, "ts")
        if q.dim() != 2 or s.dim() != 2 or q.shape[0] != s.shape[0] or q.shape[1] != 8 * s.shape[1]:
            raise _bad(f"q {tuple(q.shape)} and s {tuple(s.shape)} are not [N, K/2] and [N, K/16]")
        if tuple(ts.shape) not in ((1,), (q.shape[0],)):
            raise _bad(f"ts {tuple(ts.shape)} is not [N] or [1]")
        _same_device(q.device, s=s, ts=ts)
        self.q, self.s = q, s
        self.ts = ts.expand(q.shape[0]).contiguous()
        self.N, self.K = q.shape[0], 2 * q.shape[1]
        self._weights = (q.data_ptr(), s.data_ptr(), self.ts.data_ptr(), self.N, self.K)

    def __call__(self, x, dtype=torch.float32, out=None, stream=None):
        """x bfloat16 [T, K] (rows may be strided) -> [T, N] float32 or bfloat16."""
        dev = self.q.device
        stride = _rows(x, _BF16, (self.K,), "x")
        if x.device != dev:
            _same_device(dev, x=x)
        handle = _handle(stream, dev)
        T = x.shape[0]
        if out is not None:
            dtype = out.dtype
        if dtype not in (torch.float32, torch.bfloat16):
            raise _bad(f"dtype {dtype} is not float32 or bfloat16")
        if out is None:
            out = _empty((T, self.N), dtype, dev, stream)
        else:
            _need_out(out, dtype, (T, self.N), dev, "out")
        st = _library().moe_linear(*self._weights, x.data_ptr(), stride, out.data_ptr(), dtype == torch.bfloat16, T,
                                   handle)
        if st != MOE_OK:
            _check(st)
        return out


def rope_table(positions: int, rot_dim: int, theta: float = 10000.0, inv_freq=None, magnitude: float = 1.0,
               device="cuda") -> torch.Tensor:
    """(cos, sin) pairs of every position, float32 [positions, rot_dim], from
    angles in 64 bits.  inv_freq: the rot_dim / 2 frequencies where they are not
    theta^(-2j / rot_dim) (scaled for long contexts); magnitude scales both."""
    if inv_freq is None:
        inv_freq = theta ** (-torch.arange(0, rot_dim, 2, dtype=torch.float64, device=device) / max(rot_dim, 1))
    inv_freq = torch.as_tensor(inv_freq, dtype=torch.float64, device=device)
    if tuple(inv_freq.shape) != (rot_dim // 2,):
        raise _bad(f"inv_freq {tuple(inv_freq.shape)} is not [rot_dim / 2 = {rot_dim // 2}]")
    ang = torch.arange(positions, dtype=torch.float64, device=device)[:, None] * inv_freq[None, :]
    return (torch.stack((ang.cos(), ang.sin()), -1) * magnitude).reshape(positions, rot_dim).float()


class KVCache:
    """A paged key/value cache in 8 bits (moe_kv_create): k uint8 [n_pages,
    kv_heads, PAGE, head_dim], v uint8 [n_pages, kv_heads, head_dim, PAGE] (E4M3
    codes, v transposed), k_scale and v_scale float32 [n_pages, kv_heads].
    Allocated zeroed, or taken from `buffers` (dict of k, v, k_scale, v_scale; v
    must hold no NaN code, 0x7F or 0xFF, in unused slots either: zero it once).
    rope: float32 [positions, rot_dim] (rope_table) or None for no rotation.

    A step's sequences are q_off int32 [B + 1] (offsets of each one's new tokens),
    kv_len int32 [B] (tokens in the cache, the new ones included) and pages int32
    [B, max_pages], all on the device; max_q is the host's bound on a sequence's
    new tokens."""

    def __init__(self, n_pages: int, q_heads: int, kv_heads: int, head_dim: int, rope=None, interleaved: bool = False,
                 device=None, buffers: dict = None):
        if buffers is None:
            device = torch.device("cuda" if device is None else device)
            buffers = dict(k=torch.zeros((n_pages, kv_heads, PAGE, head_dim), dtype=torch.uint8, device=device),
                           v=torch.zeros((n_pages, kv_heads, head_dim, PAGE), dtype=torch.uint8, device=device),
                           k_scale=torch.zeros((n_pages, kv_heads), dtype=torch.float32, device=device),
                           v_scale=torch.zeros((n_pages, kv_heads), dtype=torch.float32, device=device))
        self.k, self.v = buffers["k"], buffers["v"]
        self.k_scale, self.v_scale = buffers["k_scale"], buffers["v_scale"]
        _need(self.k, torch.uint8, "k")
        dev = self.k.device
        _need_out(self.k, torch.uint8, (n_pages, kv_heads, PAGE, head_dim), dev, "k")
        _need_out(self.v, torch.uint8, (n_pages, kv_heads, head_dim, PAGE), dev, "v")
        _need_out(self.k_scale, torch.float32, (n_pages, kv_heads), dev, "k_scale")
        _need_out(self.v_scale, torch.float32, (n_pages, kv_heads), dev, "v_scale")
        if rope is not None:
            _need(rope, torch.float32, "rope")
            if rope.dim() != 2:
                raise _bad(f"rope {tuple(rope.shape)} is not [positions, rot_dim]")
            _same_device(dev, rope=rope)
        self.rope, self.device = rope, dev
        self.n_pages, self.q_heads, self.kv_heads, self.head_dim = n_pages, q_heads, kv_heads, head_dim
        d = moe_kv_desc(n_pages, q_heads, kv_heads, head_dim, self.k.data_ptr(), self.v.data_ptr(),
                        self.k_scale.data_ptr(), self.v_scale.data_ptr(), 0 if rope is None else rope.shape[1],
                        int(bool(interleaved)), 0 if rope is None else rope.shape[0],
                        None if rope is None else rope.data_ptr(), dev.index)
        self.handle = C.c_void_p()
        _check(_library().moe_kv_create(C.byref(d), C.byref(self.handle)))
        self._ws_bytes = int(_library().moe_kv_workspace_bytes(self.handle))
        self._q_row, self._kv_row = (q_heads, head_dim), (kv_heads, head_dim)
        self._scale = 1.0 / math.sqrt(head_dim)

    def __del__(self):
        h = getattr(self, "handle", None)
        if h and _ready is not None:
            _ready.moe_kv_destroy(h)
            self.handle = None

    def new_workspace(self, stream=None) -> torch.Tensor:
        """Zeroed workspace for append and attend: one per concurrent stream."""
        handle = _handle(stream, self.device)
        ws = _empty((self._ws_bytes,), torch.uint8, self.device, stream)
        _check(_library().moe_kv_workspace_init(self.handle, ws.data_ptr(), self._ws_bytes, handle))
        return ws

    def _step(self, q_off, kv_len, pages, ws, N, max_q):
        """The batch description; checks the step's arrays and the workspace."""
        dev = self.device
        if isinstance(kv_len, _Tensor) and isinstance(q_off, _Tensor) and isinstance(pages, _Tensor):
            one, two = kv_len.shape, pages.shape
            if (len(one) == 1 and len(two) == 2 and one[0] == two[0] and q_off.shape == (one[0] + 1,) and
                    kv_len.dtype is _INT32 and q_off.dtype is _INT32 and pages.dtype is _INT32 and
                    kv_len.device == dev and q_off.device == dev and pages.device == dev and
                    kv_len.is_contiguous() and q_off.is_contiguous() and pages.is_contiguous()):
                self._need_ws(ws)
                return C.byref(moe_kv_batch(q_off.data_ptr(), kv_len.data_ptr(), pages.data_ptr(), two[1], one[0], N, max_q))
        for name, t in (("q_off", q_off), ("kv_len", kv_len), ("pages", pages)):
            _need(t, torch.int32, name)
            _same_device(dev, **{name: t})
        raise _bad(f"shapes q_off {tuple(q_off.shape)}, kv_len {tuple(kv_len.shape)}, pages {tuple(pages.shape)} "
                   "are not [B + 1], [B], [B, max_pages]")

    def _need_ws(self, ws):
        if not (isinstance(ws, _Tensor) and ws.dtype is torch.uint8 and ws.device == self.device and
                ws.is_contiguous() and ws.numel() >= self._ws_bytes):
            _need(ws, torch.uint8, "ws")
            _same_device(self.device, ws=ws)
            raise _bad("ws is smaller than this cache's workspace (new_workspace)")

    def append(self, k, v, q_off, kv_len, pages, ws, max_q: int, q=None, q_out=None, stream=None, parents=None):
        """Rotate and append the new tokens' k and v (bfloat16 [N, kv_heads,
        head_dim], tokens may be strided), and rotate q (bfloat16 [N, q_heads,
        head_dim]) into q_out, which is returned (None without q) and may be q.
        Rows outside every sequence (before q_off[0], from q_off[B] on) are not
        read and not written: a q_out allocated here holds anything there.  parents
        (int32 [N]) makes each sequence's new tokens a tree of up to MAX_TREE: the token
        before each, counted inside the sequence's new ones, or -1 at a root; a token
        turns by its depth (moe_kv_append_tree), and is stored in the order given."""
        dev = self.device
        ks = _rows(k, _BF16, self._kv_row, "k")
        N = k.shape[0]
        vs = _rows(v, _BF16, self._kv_row, "v", N)
        qs = 0
        if k.device != dev or v.device != dev:
            _same_device(dev, k=k, v=v)
        handle = _handle(stream, dev)
        if q is not None:
            qs = _rows(q, _BF16, self._q_row, "q", N)
            if q.device != dev:
                _same_device(dev, q=q)
            if q_out is None:
                q_out = _empty((N, *self._q_row), torch.bfloat16, dev, stream)
            else:
                _need_out(q_out, torch.bfloat16, (N, *self._q_row), dev, "q_out")
        elif q_out is not None:
            raise _bad("q_out without q")
        args = (self.handle, _ptr(q), qs, k.data_ptr(), ks, v.data_ptr(), vs, _ptr(q_out),
                self._step(q_off, kv_len, pages, ws, N, max_q))
        if parents is None:
            st = _library().moe_kv_append(*args, ws.data_ptr(), handle)
        else:
            self._need_int32(parents, (N,), "parents")
            st = _library().moe_kv_append_tree(*args, parents.data_ptr(), ws.data_ptr(), handle)
        if st != MOE_OK:
            _check(st)
        return q_out

    def attend(self, q, q_off, kv_len, pages, ws, max_q: int, scale: float = None, out=None, stream=None, parents=None):
        """Causal attention of q (bfloat16 [N, q_heads, head_dim], tokens may be
        strided) over the cache: bfloat16 [N, q_heads, head_dim].  scale: 1 /
        sqrt(head_dim) unless given.  A token that sees nothing gets 0; rows
        outside every sequence (before q_off[0], from q_off[B] on) are not written:
        an out allocated here holds anything there, so give a zeroed one where
        what follows reads padded rows.  parents as in append: a token then sees the
        tokens before the tree and the way to its root (moe_kv_attend_tree)."""
        dev = self.device
        qs = _rows(q, _BF16, self._q_row, "q")
        if q.device != dev:
            _same_device(dev, q=q)
        handle = _handle(stream, dev)
        if out is None:
            out = _empty(q.shape, torch.bfloat16, dev, stream)
        else:
            _need_out(out, torch.bfloat16, q.shape, dev, "out")
        args = (self.handle, q.data_ptr(), qs, self._scale if scale is None else scale, out.data_ptr(),
                self._step(q_off, kv_len, pages, ws, q.shape[0], max_q))
        if parents is None:
            st = _library().moe_kv_attend(*args, ws.data_ptr(), handle)
        else:
            self._need_int32(parents, (q.shape[0],), "parents")
            st = _library().moe_kv_attend_tree(*args, parents.data_ptr(), ws.data_ptr(), handle)
        if st != MOE_OK:
            _check(st)
        return out

    def compact(self, keep, n_keep, q_off, kv_len, pages, ws, max_q: int = 0, kv_len_out=None, stream=None):
        """Keep the accepted ones of each sequence's newest tokens (moe_kv_compact),
        those that a step appended with the same q_off, kv_len and pages: of sequence
        b's n the ones keep[b, :n_keep[b]] (int32 [B, K], ascending; n_keep int32 [B]),
        which move up to follow the tokens before them.  Returns the new lengths, int32
        [B]; kv_len is left as it is (and kv_len_out is another array).  max_q may be given, so
        that a step's arguments go to append, attend and compact alike; nothing depends on it."""
        dev = self.device
        handle = _handle(stream, dev)
        # (offsets are only subtracted here, no row is read by them: the most rows that a step can have bound them)
        step = self._step(q_off, kv_len, pages, ws, (1 << 30) // self.q_heads, 0)
        B = kv_len.shape[0]
        if not isinstance(keep, torch.Tensor) or keep.dim() != 2:
            raise _bad("keep must be a CUDA tensor [B, K]")
        K = keep.shape[1]
        self._need_int32(keep, (B, K), "keep")
        self._need_int32(n_keep, (B,), "n_keep")
        if kv_len_out is None:
            kv_len_out = _empty((B,), torch.int32, dev, stream)
        else:
            self._need_int32(kv_len_out, (B,), "kv_len_out")
        st = _library().moe_kv_compact(self.handle, keep.data_ptr(), n_keep.data_ptr(), K, kv_len_out.data_ptr(), step,
                                       ws.data_ptr(), handle)
        if st != MOE_OK:
            _check(st)
        return kv_len_out

    def fork(self, src, fresh, kv_len, pages, ws, pages_out=None, kv_len_out=None, stream=None):
        """Sequences that go on from others (moe_kv_fork): child c has the tokens of
        sequence src[c] (int32 [C]) of kv_len [B] and pages [B, max_pages].  fresh[c]
        (int32 [C]) is a free page that becomes the child's own for the tokens to come,
        with a copy of what the sequence's last page holds; -1 leaves the child the
        sequence's own page (for one child at most: a second one that is left a partly
        filled page is flagged, and gets no pages).  Full pages are shared.
        Returns (pages, kv_len) of the children, int32 [C, max_pages] and [C]."""
        dev = self.device
        handle = _handle(stream, dev)
        B = kv_len.shape[0] if isinstance(kv_len, torch.Tensor) and kv_len.dim() == 1 else -1
        width = pages.shape[1] if isinstance(pages, torch.Tensor) and pages.dim() == 2 else -1
        C_ = src.shape[0] if isinstance(src, torch.Tensor) and src.dim() == 1 else -1
        self._need_int32(kv_len, (B,), "kv_len")
        self._need_int32(pages, (B, width), "pages")
        self._need_int32(src, (C_,), "src")
        self._need_int32(fresh, (C_,), "fresh")
        self._need_ws(ws)
        if pages_out is None:
            pages_out = _empty((C_, width), torch.int32, dev, stream)
        else:
            self._need_int32(pages_out, (C_, width), "pages_out")
        if kv_len_out is None:
            kv_len_out = _empty((C_,), torch.int32, dev, stream)
        else:
            self._need_int32(kv_len_out, (C_,), "kv_len_out")
        st = _library().moe_kv_fork(self.handle, src.data_ptr(), fresh.data_ptr(), C_, kv_len.data_ptr(), pages.data_ptr(),
                                    width, B, kv_len_out.data_ptr(), pages_out.data_ptr(), ws.data_ptr(), handle)
        if st != MOE_OK:
            _check(st)
        return pages_out, kv_len_out

    def _need_int32(self, t, shape, name):
        _need_out(t, _INT32, shape, self.device, name)

    def check(self, ws, stream=None) -> int:
        """Synchronise and return the device status (0 = MOE_OK); clears it."""
        self._need_ws(ws)
        return int(_library().moe_kv_check(self.handle, ws.data_ptr(), _handle(stream, self.device)))


def sample(logits, u, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0, out=None, prob=None, return_prob: bool = False,
           stream=None):
    """A token for each row of logits (float32 or bfloat16 [T, V], rows may be
    strided), by the random numbers u (float32 [T], in [0, 1)): int32 [T]
    (moe_sample).  temperature, top_p and min_p are numbers or float32 [T], top_k a
    number or int32 [T]; temperature 0 gives the token of the largest logit, top_k 0,
    top_p 1 and min_p 0 set no limit.  A row of -inf gives -1.  With return_prob (or
    prob, float32 [T], to write to): (tokens, the probability that each was chosen with)."""
    if not isinstance(logits, torch.Tensor) or logits.dim() != 2:
        raise _bad("logits must be a CUDA tensor [T, V]")
    T, V = logits.shape
    stride = _rows(logits, (_FLOAT32, torch.bfloat16), (V,), "logits")
    dev, one = logits.device, (T,)
    handle = _handle(stream, dev)
    _need_out(u, _FLOAT32, one, dev, "u")
    if type(top_k) is int and not 0 < top_k <= V:
        top_k = 0  # (no limit, also past 32 bits)
    settings = []
    for v, dtype, name in ((temperature, _FLOAT32, "temperature"), (top_k, _INT32, "top_k"), (top_p, _FLOAT32, "top_p"),
                           (min_p, _FLOAT32, "min_p")):
        if isinstance(v, _Tensor):
            _need_out(v, dtype, one, dev, name)
            settings += (v.data_ptr(), 0)
        else:
            settings += (None, v)
    if out is None:
        out = _empty(one, _INT32, dev, stream)
    else:
        _need_out(out, _INT32, one, dev, "out")
    if prob is not None:
        _need_out(prob, _FLOAT32, one, dev, "prob")
    elif return_prob:
        prob = _empty(one, _FLOAT32, dev, stream)
    d = moe_sample_desc(logits.data_ptr(), stride, logits.dtype == torch.bfloat16, T, V, u.data_ptr(), *settings,
                        out.data_ptr(), _ptr(prob))
    st = _library().moe_sample(C.byref(d), handle)
    if st != MOE_OK:
        _check(st)
    return out if prob is None else (out, prob)
