"""Binding of the paged-cache operators of libmoe_int4.so: moe_kv_plan,
moe_rope_append, moe_attn_decode and moe_block_norm (include/moe_int4.h).

Argument checks and marshalling only, as in the rest of the package.  The
argument structs are packed with struct.Struct: these calls sit in a decode
loop, where filling a ctypes.Structure of thirty fields costs more than the
call itself.  A class's calls go to one stream at a time.
"""
from __future__ import annotations

import ctypes
import math
import struct

import torch

from . import _check, _destroy, _lib, _stream

MOE_F32, MOE_F16, MOE_BF16, MOE_E4M3 = 0, 1, 2, 3
MOE_PLAN_NO_PAGES, MOE_PLAN_ROW_FULL, MOE_PLAN_NO_ROOM, MOE_PLAN_NEGATIVE = 1, 2, 4, 8
MOE_ROPE_SCALINGS = {"none": 0, "linear": 1, "ntk": 2, "parts": 3, "parts_by_index": 4}

_ACT = {torch.float32: MOE_F32, torch.float16: MOE_F16, torch.bfloat16: MOE_BF16}
_CACHE = {torch.float16: MOE_F16, torch.bfloat16: MOE_BF16, torch.float8_e4m3fn: MOE_E4M3}

_vp, _ci, _i64 = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64


class MoeRopeDesc(ctypes.Structure):
    _fields_ = [("rot_dim", _ci), ("base", ctypes.c_double), ("scaling", _ci), ("factor", ctypes.c_double),
                ("original_len", _ci), ("beta_fast", ctypes.c_double), ("beta_slow", ctypes.c_double)]


class MoeAttnDesc(ctypes.Structure):
    _fields_ = [(n, _ci) for n in ("max_requests", "n_heads", "n_kv_heads", "k_dim", "v_dim")]


# the host structs of the header, field by field ("@": the C compiler's alignment)
_ROPE_ARGS = struct.Struct("@11iP3f2Pq6P14q")
_ATTN_ARGS = struct.Struct("@6i3f2P2q5P10q")
_NORM_ARGS = struct.Struct("@4i3f7P6q")

for _name, _args in {
        "moe_kv_plan": [_vp, _vp, _ci, _vp, _ci, _vp, _ci, _vp, _i64, _ci, _ci, _vp, _vp, _vp, _vp, _vp, _vp],
        "moe_rope_turns": [ctypes.POINTER(MoeRopeDesc), _vp, _vp],
        "moe_rope_append": [_vp, _vp],
        "moe_attn_create": [ctypes.POINTER(MoeAttnDesc), ctypes.POINTER(_vp)],
        "moe_attn_destroy": [_vp],
        "moe_attn_decode": [_vp, _vp, _vp],
        "moe_block_norm": [_vp, _vp],
}.items():
    getattr(_lib, _name).argtypes = _args
    getattr(_lib, _name).restype = _ci


_UNPACKABLE = (struct.error, OverflowError)


def _refuse(error):
    raise ValueError(f"an argument is out of range or of another kind: {error}") from None


def _device(device) -> int:
    d = torch.device(device)
    if d.type != "cuda":
        raise ValueError("expected a CUDA device (the library has no CPU path)")
    return torch.cuda.current_device() if d.index is None else d.index


def _here(dev: int, *tensors) -> None:
    """Every tensor (None: absent) on CUDA device `dev`, which has to be the current one."""
    for t in tensors:
        if t is not None and t.get_device() != dev:
            raise ValueError(f"expected every tensor on cuda:{max(dev, 0)}, got one on {t.device} "
                             "(the library has no CPU path)")
    if dev < 0:
        raise ValueError("expected CUDA tensors (the library has no CPU path)")
    if torch._C._cuda_getDevice() != dev:
        raise ValueError(f"cuda:{dev} has to be the current device")


def _raw(stream, dev: int) -> int:
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(dev)
    return _stream(stream).value or 0


def _empty(shape, like, dtype, dev: int, stream):
    """A new contiguous tensor that belongs to the stream the call runs on."""
    if stream is None:
        if like is not None and like.is_contiguous():
            return torch.empty_like(like)  # the cheapest way
        return torch.empty(shape, dtype=dtype, device=dev)
    s = stream if isinstance(stream, torch.cuda.Stream) else torch.cuda.ExternalStream(int(stream), device=dev)
    with torch.cuda.stream(s):
        return torch.empty(shape, dtype=dtype, device=dev)


def _ints(name, t, shape, dtype=torch.int32):
    if t.dtype is not dtype or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name}: expected a contiguous {dtype} tensor of shape {tuple(shape)}, "
                         f"got {t.dtype} {tuple(t.shape)}")


def _table(t, rows):
    """Entries of a row of a block table, and their distance between rows."""
    shape = t.shape
    if t.dtype is not torch.int32 or len(shape) != 2 or shape[0] < rows or (shape[1] > 1 and t.stride(1) != 1):
        raise ValueError(f"block_table: expected int32 [>= {rows}, pages] with contiguous rows, "
                         f"got {t.dtype} {tuple(shape)}")
    return shape[1], t.stride(0)


def _caches(k_cache, v_cache, heads, k_dim, v_dim):
    """Of a pair of caches [pages, page_size, heads, dim] (any strides, contiguous
    rows; v_cache None: no values): MOE_* type, strides, pages and page size."""
    dt, ks, kst = k_cache.dtype, k_cache.shape, k_cache.stride()
    kind, vst = _CACHE.get(dt), (0, 0, 0, 1) if v_cache is None else v_cache.stride()
    if kind is None or len(ks) != 4 or ks[2] != heads or ks[3] != k_dim or kst[3] != 1 or (
            v_cache is not None and (v_cache.dtype is not dt or v_cache.shape != (ks[0], ks[1], heads, v_dim) or
                                     vst[3] != 1)):
        raise ValueError(f"expected caches [pages, page_size, {heads}, {k_dim}] and [.., .., {heads}, {v_dim}] of one "
                         f"type (float16, bfloat16 or float8_e4m3fn) with contiguous rows, got "
                         f"{[None if c is None else (c.dtype, tuple(c.shape)) for c in (k_cache, v_cache)]}")
    return kind, kst, vst, ks[0], ks[1]


class KvPlan:
    """Pages, positions and cache slots of the tokens a batch brings (moe_kv_plan).

    Owns the outputs of `update`: q_start [n + 1], seq_len [n], positions
    [max_new_tokens] int32, slots [max_new_tokens] int64 (-1: no token, or no
    page for it) and info [4] int32 (new tokens, list head after the call,
    MOE_PLAN_* flags, largest seq_len).  To go on, copy info[1:2] to free_head and
    seq_len to past_len: the plan's own outputs are refused as its inputs.
    """

    def __init__(self, max_requests, max_new_tokens, page_size, device="cuda"):
        self.max_requests, self.max_new_tokens = int(max_requests), int(max_new_tokens)
        self.page_size, self._dev = int(page_size), _device(device)
        new = lambda n, dt: torch.empty(n, dtype=dt, device=self._dev)  # noqa: E731
        self._start, self._len = new(self.max_requests + 1, torch.int32), new(self.max_requests, torch.int32)
        self.positions, self.slots = new(self.max_new_tokens, torch.int32), new(self.max_new_tokens, torch.int64)
        self.info = new(4, torch.int32)
        self.q_start, self.seq_len = self._start, self._len
        self._out = tuple(t.data_ptr() for t in (self._start, self._len, self.positions, self.slots, self.info))

    def update(self, past_len, new_len, free_pages, free_head, block_table, stream=None):
        """past_len, new_len int32 [n]; free_pages int32 [n_free]; free_head
        int32 [1]; block_table int32 [>= n, pages], updated in place."""
        n, dev = past_len.shape[0] if past_len.dim() else -1, self._dev
        if n > self.max_requests:
            raise ValueError(f"{n} requests: the plan holds {self.max_requests}")
        _here(dev, past_len, new_len, free_pages, free_head, block_table)
        _ints("past_len", past_len, (n,))
        _ints("new_len", new_len, (n,))
        _ints("free_pages", free_pages, (free_pages.numel(),))
        _ints("free_head", free_head, (1,))
        cols, row = _table(block_table, n)
        if self.q_start.shape[0] != n + 1:
            self.q_start, self.seq_len = self._start[:n + 1], self._len[:n]
        _check(_lib.moe_kv_plan(past_len.data_ptr(), new_len.data_ptr(), n, free_pages.data_ptr(), free_pages.shape[0],
                                free_head.data_ptr(), self.page_size, block_table.data_ptr(), row, cols,
                                self.max_new_tokens, *self._out, _raw(stream, dev)))
        return self


class Rope:
    """Rotary positions for dimensions [rot_offset, rot_offset + rot_dim) of a
    head (moe_rope_turns, moe_rope_append).

    interleaved: pairs (2i, 2i+1), else (i, i + rot_dim/2).  scaling: "none",
    "linear", "ntk", "parts" or "parts_by_index" (with factor; parts also
    original_len, beta_fast, beta_slow), for contexts longer than the trained
    one: "parts" goes from kept to divided frequencies linearly in a pair's
    turns, "parts_by_index" in its index.  amplitude: factor on cos and sin,
    that of the scaling unless given (parts: 0.1 ln(factor) + 1, else 1).
    """

    def __init__(self, rot_dim, base=10000.0, interleaved=False, rot_offset=0, scaling="none", factor=1.0,
                 original_len=4096, beta_fast=32.0, beta_slow=1.0, device="cuda", amplitude=None):
        if scaling not in MOE_ROPE_SCALINGS:
            raise ValueError(f"scaling {scaling!r}: expected one of {sorted(MOE_ROPE_SCALINGS)}")
        self.rot_dim, self.rot_offset, self.interleaved = int(rot_dim), int(rot_offset), bool(interleaved)
        desc = MoeRopeDesc(self.rot_dim, float(base), MOE_ROPE_SCALINGS[scaling], float(factor), int(original_len),
                           float(beta_fast), float(beta_slow))
        turns = torch.zeros(max(1, self.rot_dim // 2), dtype=torch.int64)
        own = ctypes.c_float(0)
        _check(_lib.moe_rope_turns(ctypes.byref(desc), turns.data_ptr(), ctypes.byref(own)))
        self.amplitude, self._dev = own.value if amplitude is None else float(amplitude), _device(device)
        self.turns = turns.to(torch.device("cuda", self._dev))
        self._turns_ptr = self.turns.data_ptr()

    def append(self, q, k, v, positions, slots, k_cache, v_cache, q_out=None, k_scale=1.0, v_scale=1.0, stream=None):
        """q [n, heads, dim] -> rotated (q_out, or a new tensor, returned);
        k [n, kv_heads, dim] rotated and v [n, kv_heads, v_dim] (None: no
        values) into the caches [pages, page_size, kv_heads, dim] at `slots`
        (int64 [>= n]; < 0: not cached), positions int32 [>= n].  Token and
        head strides are free.  E4M3 caches hold x / scale."""
        dev = self._dev
        _here(dev, q, k, v, positions, slots, k_cache, v_cache, q_out)
        if q.dim() != 3 or k.dim() != 3 or (v is not None and v.dim() != 3) or (q_out is not None and q_out.dim() != 3):
            raise ValueError("q, k, v and q_out: expected [n, heads, dim]")
        shape, dt, kv_heads = q.shape, q.dtype, k.shape[1]
        n, heads, dim = shape
        act, v_dim = _ACT.get(dt), 0 if v is None else v.shape[2]
        if act is None:
            raise ValueError(f"q: expected float32, float16 or bfloat16, got {dt}")
        if q_out is None:
            q_out = _empty((n, heads, dim), q, dt, dev, stream)
        qs, ks, os, vs = q.stride(), k.stride(), q_out.stride(), (0, 0, 1) if v is None else v.stride()
        if k.dtype is not dt or k.shape != (n, kv_heads, dim) or q_out.dtype is not dt or q_out.shape != shape or \
                qs[2] != 1 or ks[2] != 1 or os[2] != 1 or vs[2] != 1 or \
                (v is not None and (v.dtype is not dt or v.shape != (n, kv_heads, v_dim))):
            raise ValueError(f"expected q, q_out {(n, heads, dim)}, k {(n, kv_heads, dim)} and v of {dt} with contiguous "
                             f"rows, got {[None if t is None else (t.dtype, tuple(t.shape)) for t in (q, q_out, k, v)]}")
        if positions.dtype is not torch.int32 or slots.dtype is not torch.int64 or positions.dim() != 1 or \
                slots.dim() != 1 or positions.shape[0] < n or slots.shape[0] < n or \
                not positions.is_contiguous() or not slots.is_contiguous():
            raise ValueError(f"expected contiguous positions int32 and slots int64 of at least {n} entries")
        if (v is None) != (v_cache is None):
            raise ValueError("v and v_cache go together")
        cache, kcs, vcs, pages, page = _caches(k_cache, v_cache, kv_heads, dim, v_dim)
        try:
            args = _ROPE_ARGS.pack(
                n, heads, kv_heads, dim, v_dim, self.rot_dim, self.rot_offset, self.interleaved, act, cache,
                page, self._turns_ptr, self.amplitude, k_scale, v_scale, positions.data_ptr(), slots.data_ptr(), pages,
                q.data_ptr(), k.data_ptr(), 0 if v is None else v.data_ptr(), q_out.data_ptr(), k_cache.data_ptr(),
                0 if v is None else v_cache.data_ptr(), qs[0], qs[1], ks[0], ks[1], vs[0], vs[1], os[0], os[1], kcs[0],
                kcs[1], kcs[2], vcs[0], vcs[1], vcs[2])
        except _UNPACKABLE as e:
            _refuse(e)
        _check(_lib.moe_rope_append(args, _raw(stream, dev)))
        return q_out


class PagedAttention:
    """Attention of one new token per request over a paged cache (an owned
    handle of moe_attn_create; one stream at a time).  Keep it as long as a CUDA
    graph that captured its calls."""

    def __init__(self, max_requests, n_heads, n_kv_heads, head_dim, v_dim=None, device="cuda"):
        self.n_heads, self.n_kv_heads = int(n_heads), int(n_kv_heads)
        self.head_dim, self.v_dim = int(head_dim), int(head_dim if v_dim is None else v_dim)
        self._dev, self._scale = _device(device), 1.0 / math.sqrt(self.head_dim)
        desc = MoeAttnDesc(int(max_requests), self.n_heads, self.n_kv_heads, self.head_dim, self.v_dim)
        h = ctypes.c_void_p()
        with torch.cuda.device(self._dev):
            _check(_lib.moe_attn_create(ctypes.byref(desc), ctypes.byref(h)))
        self.handle = h

    def close(self):
        if getattr(self, "handle", None) is not None and self.handle.value:
            handle, self.handle = self.handle, None
            _destroy(_lib.moe_attn_destroy, handle)

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def decode(self, q, k_cache, v_cache, block_table, seq_len, scale=None, window=0, k_scale=1.0, v_scale=1.0,
               out=None, lse=None, stream=None):
        """q [n, heads, dim]; caches [pages, page_size, kv_heads, dim] (any
        strides of 16 bytes, contiguous rows); block_table int32 [>= n, pages];
        seq_len int32 [>= n], the new token's own key included.  scale: 1 /
        sqrt(dim) unless given; window > 0: the last `window` tokens only.
        Keys and values that are read are finite (an infinity among the values
        makes NaN of outputs that the formula gives as infinite).  Returns (out [n, heads, v_dim], lse [n, heads] fp32); a request that
        sees no token gets 0 and -inf."""
        dev, heads, v_dim, dt = self._dev, self.n_heads, self.v_dim, q.dtype
        _here(dev, q, k_cache, v_cache, block_table, seq_len, out, lse)
        shape, act, qs = q.shape, _ACT.get(dt), q.stride()
        n = shape[0] if shape else 0
        if act is None or shape != (n, heads, self.head_dim) or qs[2] != 1:
            raise ValueError(f"q: expected float32, float16 or bfloat16 [n, {heads}, {self.head_dim}] with contiguous "
                             f"rows, got {dt} {tuple(shape)}")
        cache, ks, vs, pages, page = _caches(k_cache, v_cache, self.n_kv_heads, self.head_dim, v_dim)
        cols, row = _table(block_table, n)
        if seq_len.dtype is not torch.int32 or seq_len.dim() != 1 or seq_len.shape[0] < n or \
                not seq_len.is_contiguous():
            raise ValueError(f"seq_len: expected a contiguous int32 tensor of at least {n} entries")
        if out is None:
            out = _empty((n, heads, v_dim), q if v_dim == self.head_dim else None, dt, dev, stream)
        elif out.dtype is not dt or out.shape != (n, heads, v_dim) or out.stride(2) != 1:
            raise ValueError(f"out: expected {dt} {(n, heads, v_dim)} with contiguous rows")
        if lse is None:
            lse = _empty((n, heads), None, torch.float32, dev, stream)
        else:
            _ints("lse", lse, (n, heads), torch.float32)
        os = out.stride()
        try:
            args = _ATTN_ARGS.pack(
                n, act, cache, page, cols, window, self._scale if scale is None else scale, k_scale,
                v_scale, seq_len.data_ptr(), block_table.data_ptr(), row, pages, q.data_ptr(), k_cache.data_ptr(),
                v_cache.data_ptr(), out.data_ptr(), lse.data_ptr(), qs[0], qs[1], os[0], os[1], ks[0], ks[1], ks[2],
                vs[0], vs[1], vs[2])
        except _UNPACKABLE as e:
            _refuse(e)
        _check(_lib.moe_attn_decode(self.handle, args, _raw(stream, dev)))
        return out, lse


def block_norm(x, y=None, w_post=None, gate=None, w_pre=None, alpha=1.0, beta=1.0, eps=1e-5, gate_act="sigmoid",
               norm=None, out=None, normed=None, stream=None):
    """moe_block_norm: r = alpha x + beta act(gate) * norm(y; w_post) and the
    next block's input norm(r; w_pre), in one pass -> (r, normed).

    x, y [n, dim] with contiguous rows; w_post, w_pre fp32 [dim] (w_post None:
    y as it is); gate [n or 1, dim or 1], act "sigmoid" or "none".  norm: take
    the second norm (default: when w_pre or `normed` is given; with w_pre None
    its weight is 1); without it normed is None.  out may be x, normed may be y."""
    dev = x.get_device()
    _here(dev, x, y, w_post, gate, w_pre, out, normed)
    act = _ACT.get(x.dtype)
    if act is None or x.dim() != 2:
        raise ValueError(f"x: expected float32, float16 or bfloat16 [n, dim], got {x.dtype} {tuple(x.shape)}")
    if gate_act not in ("sigmoid", "none"):
        raise ValueError(f"gate_act {gate_act!r}: expected 'sigmoid' or 'none'")
    n, dim = x.shape
    if norm is None:
        norm = w_pre is not None or normed is not None
    if not norm and (w_pre is not None or normed is not None):
        raise ValueError("norm=False takes neither w_pre nor normed")
    if out is None:
        out = _empty((n, dim), x, x.dtype, dev, stream)
    if normed is None and norm:
        normed = _empty((n, dim), x, x.dtype, dev, stream)
    shape, dt = x.shape, x.dtype
    for t in (x, y, out, normed):
        if t is not None and (t.dtype is not dt or t.shape != shape or (dim > 1 and t.stride(1) != 1)):
            raise ValueError(f"expected x, y, out and normed {dt} {(n, dim)} with contiguous rows, got {t.dtype} "
                             f"{tuple(t.shape)}")
    for w in (w_post, w_pre):
        if w is not None and (w.dtype is not torch.float32 or w.shape != (dim,) or not w.is_contiguous()):
            raise ValueError(f"expected w_post and w_pre float32 [{dim}], got {w.dtype} {tuple(w.shape)}")
    gt = gd = 0
    if gate is not None:
        if gate.dtype is not x.dtype or gate.dim() != 2 or gate.shape[0] not in (1, n) or gate.shape[1] not in (1, dim):
            raise ValueError(f"gate: expected {x.dtype} [{n} or 1, {dim} or 1], got {gate.dtype} {tuple(gate.shape)}")
        gt = 0 if gate.shape[0] == 1 else gate.stride(0)
        gd = 0 if gate.shape[1] == 1 else gate.stride(1)
    ptr = lambda t: 0 if t is None else t.data_ptr()  # noqa: E731
    try:
        args = _NORM_ARGS.pack(n, dim, act, gate_act == "sigmoid", alpha, beta, eps, x.data_ptr(), ptr(y), ptr(w_post),
                               ptr(w_pre), ptr(gate), out.data_ptr(), ptr(normed), x.stride(0),
                               0 if y is None else y.stride(0), out.stride(0), 0 if normed is None else normed.stride(0),
                               gt, gd)
    except _UNPACKABLE as e:
        _refuse(e)
    _check(_lib.moe_block_norm(args, _raw(stream, dev)))
    return out, normed
