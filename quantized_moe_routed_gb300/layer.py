"""The operators around the routed experts in a decoder layer (the C ABI in
include/moe_layer.h): residual addition with root-mean-square norm, projections
with NVFP4 weights, the paged 8-bit key/value cache with its append (rotation
included) and the attention over it.

Argument marshalling only, as in `binding`: every step of the computation runs
in the library's sm_103a kernels, on `stream` or the current stream; outputs
that the caller does not pass are allocated on that stream.  A call that fails
raises MoeError; there is no fallback.
"""
from __future__ import annotations

import ctypes as C
import math

import torch

from . import binding
from .binding import MOE_ERR_INVALID_ARG, MoeError, _check, _need, _ptr, _stream

PAGE = 64        # tokens of a cache page
MAX_SEQS = 512   # sequences of a step

_P, _I, _S, _L, _F = C.c_void_p, C.c_int, C.c_size_t, C.c_int64, C.c_float


class moe_kv_desc(C.Structure):
    _fields_ = [("n_pages", _I), ("q_heads", _I), ("kv_heads", _I), ("head_dim", _I), ("k_dev", _P), ("v_dev", _P),
                ("k_scale_dev", _P), ("v_scale_dev", _P), ("rot_dim", _I), ("rot_interleaved", _I),
                ("rope_positions", _I), ("rope_dev", _P), ("device", _I)]


class moe_kv_batch(C.Structure):
    _fields_ = [("q_off_dev", _P), ("kv_len_dev", _P), ("pages_dev", _P), ("max_pages", _I), ("B", _I), ("N", _I),
                ("max_q", _I)]


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
_ready = None


def _library():
    """The library, with this header's functions prototyped."""
    global _ready
    lib = binding.load_library()
    if _ready is not lib:
        for name, (res, args) in SIGNATURES.items():
            fn = getattr(lib, name)
            fn.restype, fn.argtypes = res, args
        _ready = lib
    return lib


def _bad(msg):
    return MoeError(MOE_ERR_INVALID_ARG, msg)


def _need_rows(t, dtypes, shape, name):
    """A CUDA tensor whose rows are contiguous; returns its row stride in
    elements.  Only dimension 0 may be strided."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise _bad(f"{name} must be a CUDA tensor")
    if t.dtype not in dtypes:
        raise _bad(f"{name} must be {' or '.join(map(str, dtypes))}, got {t.dtype}")
    if t.dim() != len(shape) or any(s is not None and s != d for s, d in zip(shape, t.shape)):
        raise _bad(f"{name} {tuple(t.shape)} is not {['any' if s is None else s for s in shape]}")
    row = 1
    for d in range(t.dim() - 1, 0, -1):
        if t.shape[d] != 1 and t.stride(d) != row:
            raise _bad(f"a row of {name} must be contiguous (strides {t.stride()})")
        row *= t.shape[d]
    return t.stride(0) if t.shape[0] > 1 else max(row, 1)


def _need_out(t, dtype, shape, device, name):
    _need(t, dtype, name)
    if tuple(t.shape) != tuple(shape) or t.device != device:
        raise _bad(f"{name} {tuple(t.shape)} on {t.device} is not {tuple(shape)} on {device}")


def _on(stream, device):
    return torch.cuda.current_stream(device) if stream is None else stream


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
    stride = _need_rows(x, (torch.float32, torch.bfloat16), (None, None), "x")
    T, H = x.shape
    dev = x.device
    _need_out(weight, torch.bfloat16, (H,), dev, "weight")
    if residual is None:
        if residual_out is not None:
            raise _bad("residual_out without a residual")
    else:
        _need_out(residual, torch.bfloat16, (T, H), dev, "residual")
        if residual_out is None:
            residual_out = residual
        _need_out(residual_out, torch.bfloat16, (T, H), dev, "residual_out")
    st = _on(stream, dev)
    quant = outputs != "bf16"
    with torch.cuda.stream(st):
        if outputs != "e4m3" and out is None:
            out = torch.empty((T, H), dtype=torch.bfloat16, device=dev)
        if quant and out_q is None:
            out_q = torch.empty((T, H), dtype=torch.float8_e4m3fn, device=dev)
        if quant and out_scale is None:
            out_scale = torch.empty((T, H // 128), dtype=torch.float32, device=dev)
    if outputs == "e4m3":
        if out is not None:
            raise _bad("out with outputs='e4m3'")
    else:
        _need_out(out, torch.bfloat16, (T, H), dev, "out")
    if quant:
        _need_out(out_q, torch.float8_e4m3fn, (T, H), dev, "out_q")
        _need_out(out_scale, torch.float32, (T, H // 128), dev, "out_scale")
    elif out_q is not None or out_scale is not None:
        raise _bad("out_q or out_scale with outputs='bf16'")
    _check(_library().moe_norm(_ptr(x), int(x.dtype == torch.float32), stride, _ptr(residual), _ptr(residual_out),
                               _ptr(weight), eps, _ptr(out), _ptr(out_q), _ptr(out_scale), T, H, _stream(st)))
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

    def __call__(self, x, dtype=torch.float32, out=None, stream=None):
        """x bfloat16 [T, K] (rows may be strided) -> [T, N] float32 or bfloat16."""
        stride = _need_rows(x, (torch.bfloat16,), (None, self.K), "x")
        _same_device(self.q.device, x=x)
        if out is not None:
            dtype = out.dtype
        if dtype not in (torch.float32, torch.bfloat16):
            raise _bad(f"dtype {dtype} is not float32 or bfloat16")
        st = _on(stream, x.device)
        if out is None:
            with torch.cuda.stream(st):
                out = torch.empty((x.shape[0], self.N), dtype=dtype, device=x.device)
        _need_out(out, dtype, (x.shape[0], self.N), x.device, "out")
        _check(_library().moe_linear(_ptr(self.q), _ptr(self.s), _ptr(self.ts), self.N, self.K, _ptr(x), stride,
                                     _ptr(out), int(dtype == torch.bfloat16), x.shape[0], _stream(st)))
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
    Allocated zeroed, or taken from `buffers` (dict of k, v, k_scale, v_scale).
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

    def __del__(self):
        h = getattr(self, "handle", None)
        if h and _ready is not None:
            _ready.moe_kv_destroy(h)
            self.handle = None

    def new_workspace(self, stream=None) -> torch.Tensor:
        """Zeroed workspace for append and attend: one per concurrent stream."""
        n = int(_library().moe_kv_workspace_bytes(self.handle))
        st = _on(stream, self.device)
        with torch.cuda.stream(st):
            ws = torch.empty(n, dtype=torch.uint8, device=self.device)
        _check(_library().moe_kv_workspace_init(self.handle, _ptr(ws), n, _stream(st)))
        return ws

    def _batch(self, q_off, kv_len, pages, N, max_q):
        for name, t in (("q_off", q_off), ("kv_len", kv_len), ("pages", pages)):
            _need(t, torch.int32, name)
            _same_device(self.device, **{name: t})
        B = kv_len.shape[0] if kv_len.dim() == 1 else -1
        if B < 0 or tuple(q_off.shape) != (B + 1,) or pages.dim() != 2 or pages.shape[0] != B:
            raise _bad(f"shapes q_off {tuple(q_off.shape)}, kv_len {tuple(kv_len.shape)}, pages {tuple(pages.shape)} "
                       "are not [B + 1], [B], [B, max_pages]")
        return moe_kv_batch(q_off.data_ptr(), kv_len.data_ptr(), pages.data_ptr(), pages.shape[1], B, N, max_q)

    def _need_ws(self, ws):
        _need(ws, torch.uint8, "ws")
        _same_device(self.device, ws=ws)
        if ws.numel() < int(_library().moe_kv_workspace_bytes(self.handle)):
            raise _bad("ws is smaller than this cache's workspace (new_workspace)")

    def append(self, k, v, q_off, kv_len, pages, ws, max_q: int, q=None, q_out=None, stream=None):
        """Rotate and append the new tokens' k and v (bfloat16 [N, kv_heads,
        head_dim], tokens may be strided), and rotate q (bfloat16 [N, q_heads,
        head_dim]) into q_out, which is returned (None without q)."""
        ks = _need_rows(k, (torch.bfloat16,), (None, self.kv_heads, self.head_dim), "k")
        N = k.shape[0]
        vs = _need_rows(v, (torch.bfloat16,), (N, self.kv_heads, self.head_dim), "v")
        _same_device(self.device, k=k, v=v)
        qs = 0
        st = _on(stream, self.device)
        if q is not None:
            qs = _need_rows(q, (torch.bfloat16,), (N, self.q_heads, self.head_dim), "q")
            _same_device(self.device, q=q)
            if q_out is None:
                with torch.cuda.stream(st):
                    q_out = torch.empty((N, self.q_heads, self.head_dim), dtype=torch.bfloat16, device=self.device)
            _need_out(q_out, torch.bfloat16, (N, self.q_heads, self.head_dim), self.device, "q_out")
        elif q_out is not None:
            raise _bad("q_out without q")
        self._need_ws(ws)
        batch = self._batch(q_off, kv_len, pages, N, max_q)
        _check(_library().moe_kv_append(self.handle, _ptr(q), qs, _ptr(k), ks, _ptr(v), vs, _ptr(q_out),
                                        C.byref(batch), _ptr(ws), _stream(st)))
        return q_out

    def attend(self, q, q_off, kv_len, pages, ws, max_q: int, scale: float = None, out=None, stream=None):
        """Causal attention of q (bfloat16 [N, q_heads, head_dim], tokens may be
        strided) over the cache: bfloat16 [N, q_heads, head_dim].  scale: 1 /
        sqrt(head_dim) unless given."""
        qs = _need_rows(q, (torch.bfloat16,), (None, self.q_heads, self.head_dim), "q")
        _same_device(self.device, q=q)
        st = _on(stream, self.device)
        if out is None:
            with torch.cuda.stream(st):
                out = torch.empty((q.shape[0], self.q_heads, self.head_dim), dtype=torch.bfloat16, device=self.device)
        _need_out(out, torch.bfloat16, (q.shape[0], self.q_heads, self.head_dim), self.device, "out")
        self._need_ws(ws)
        batch = self._batch(q_off, kv_len, pages, q.shape[0], max_q)
        _check(_library().moe_kv_attend(self.handle, _ptr(q), qs,
                                        1.0 / math.sqrt(self.head_dim) if scale is None else scale, _ptr(out),
                                        C.byref(batch), _ptr(ws), _stream(st)))
        return out

    def check(self, ws, stream=None) -> int:
        """Synchronise and return the device status (0 = MOE_OK); clears it."""
        self._need_ws(ws)
        return int(_library().moe_kv_check(self.handle, _ptr(ws), _stream(_on(stream, self.device))))
