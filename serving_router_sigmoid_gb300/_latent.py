"""Binding of the FP8 products and the latent attention of libmoe_int4.so:
moe_quant_act_fp8, moe_fp8_linear, moe_latent_decode and moe_latent_prompt
(include/moe_int4.h).  Argument checks and marshalling only."""
from __future__ import annotations

import ctypes
import struct

import torch

from . import _check, _destroy, _lib, _stream
from ._paged import (_ACT, _UNPACKABLE, MOE_BF16, MOE_E4M3, MOE_F16, _device, _empty, _here, _ints, _raw, _refuse,
                     _table)

_HALF = {torch.float16: MOE_F16, torch.bfloat16: MOE_BF16}
_E4M3 = torch.float8_e4m3fn

_vp, _ci, _i64 = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64


class MoeLatentDesc(ctypes.Structure):
    _fields_ = [(n, _ci) for n in ("max_requests", "n_heads", "latent_dim", "rope_dim")]


# the host structs of the header, field by field ("@": the C compiler's alignment)
_LINEAR_ARGS = struct.Struct("@4i5P3q")
_LATENT_ARGS = struct.Struct("@5i2f2P2q4P6q")
_PROMPT_ARGS = struct.Struct("@9if8P9q")

for _name, _args in {
        "moe_quant_act_fp8": [_vp, _ci, _i64, _ci, _ci, _vp, _i64, _vp, _vp],
        "moe_fp8_linear": [_vp, _vp],
        "moe_latent_create": [ctypes.POINTER(MoeLatentDesc), ctypes.POINTER(_vp)],
        "moe_latent_destroy": [_vp],
        "moe_latent_decode": [_vp, _vp, _vp],
        "moe_latent_prompt": [_vp, _vp],
        "moe_dense_status": [_vp, ctypes.POINTER(_ci)],
}.items():
    getattr(_lib, _name).argtypes = _args
    getattr(_lib, _name).restype = _ci


_templates = {}  # (shape, type, device) -> a tensor of that shape over one element


def _out(shape, dtype, dev, stream):
    """A new contiguous tensor that belongs to the stream the call runs on.

    torch.empty_like is the cheapest way to one (2 us next to a launch, torch.empty 3
    to 4), so shapes that were asked for before stand by as expanded single elements."""
    if stream is not None:
        return _empty(shape, None, dtype, dev, stream)
    like = _templates.get((shape, dtype, dev))
    if like is None:
        if torch.cuda.is_current_stream_capturing():  # nothing of a graph's memory stays here
            return torch.empty(shape, dtype=dtype, device=dev)
        if len(_templates) >= 256:
            _templates.clear()
        like = _templates[shape, dtype, dev] = torch.empty(1, dtype=dtype, device=dev).expand(shape)
    return torch.empty_like(like)


def _rows(name, t, dtypes):
    """A matrix with contiguous rows -> its shape and row stride (0: one row)."""
    shape = t.shape
    if t.dtype in dtypes and len(shape) == 2:
        rs, cs = t.stride()
        if cs == 1 or shape[1] <= 1:
            return shape[0], shape[1], rs if shape[0] > 1 else 0
    raise ValueError(f"{name}: expected a matrix of {' or '.join(str(d) for d in dtypes)} with contiguous rows, got "
                     f"{t.dtype} {tuple(shape)}")


_CODES = (_E4M3, torch.uint8)


def quant_act_fp8(x, x8=None, scale=None, stream=None):
    """moe_quant_act_fp8: x [n, dim] (float32, float16 or bfloat16, contiguous
    rows) as E4M3 codes and one scale for each 128 of a row -> (x8 [n, dim]
    float8_e4m3fn, scale [n, ceil(dim / 128)] float32).  dim is a multiple of 16."""
    dev = x.get_device()
    _here(dev, x, x8, scale)
    n, dim, xs = _rows("x", x, _ACT)
    groups = (dim + 127) // 128
    if x8 is None:
        x8, row = _out((n, dim), _E4M3, dev, stream), dim
    else:
        row = _rows("x8", x8, _CODES)[2]
        if x8.shape != (n, dim):
            raise ValueError(f"x8: expected {(n, dim)}, got {tuple(x8.shape)}")
    if scale is None:
        scale = _out((n, groups), torch.float32, dev, stream)
    else:
        _ints("scale", scale, (n, groups), torch.float32)
    _check(_lib.moe_quant_act_fp8(x.data_ptr(), _ACT[x.dtype], xs, n, dim, x8.data_ptr(), row, scale.data_ptr(),
                                  _raw(stream, dev)))
    return x8, scale


def fp8_linear(x8, x_scale, w8, scale_inv, out=None, dtype=torch.bfloat16, stream=None):
    """moe_fp8_linear: the product of activations as quant_act_fp8 gives them,
    x8 [n, I] and x_scale [n, ceil(I / 128)], with a checkpoint's matrix w8 [O, I]
    (float8_e4m3fn or its codes) and scale_inv [ceil(O / 128), ceil(I / 128)] ->
    out [n, O] of `dtype` (float32, float16 or bfloat16; that of `out` if given)."""
    dev = x8.get_device()
    _here(dev, x8, x_scale, w8, scale_inv, out)
    n, inner, xs = _rows("x8", x8, _CODES)
    outer, w_inner, ws = _rows("w8", w8, _CODES)
    if w_inner != inner:
        raise ValueError(f"x8 has rows of {inner}, w8 of {w_inner}")
    blocks = (inner + 127) // 128
    _ints("x_scale", x_scale, (n, blocks), torch.float32)
    _ints("scale_inv", scale_inv, ((outer + 127) // 128, blocks), torch.float32)
    if out is None:
        if dtype not in _ACT:
            raise ValueError(f"dtype: expected float32, float16 or bfloat16, got {dtype}")
        out, os = _out((n, outer), dtype, dev, stream), outer
    else:
        dtype, os = out.dtype, _rows("out", out, _ACT)[2]
        if out.shape != (n, outer):
            raise ValueError(f"out: expected {(n, outer)}, got {tuple(out.shape)}")
    try:
        args = _LINEAR_ARGS.pack(n, inner, outer, _ACT[dtype], x8.data_ptr(), x_scale.data_ptr(), w8.data_ptr(),
                                 scale_inv.data_ptr(), out.data_ptr(), xs, ws, os)
    except _UNPACKABLE as e:
        _refuse(e)
    _check(_lib.moe_fp8_linear(args, _raw(stream, dev)))
    return out


class LatentAttention:
    """Attention of one new token per request over a paged cache of latent rows
    (latent part, then rotary part) that all heads share: an owned handle of
    moe_latent_create, one stream at a time.  Keep it as long as a CUDA graph that
    captured its calls."""

    def __init__(self, max_requests, n_heads, latent_dim=512, rope_dim=64, device="cuda"):
        self.n_heads, self.latent_dim, self.rope_dim = int(n_heads), int(latent_dim), int(rope_dim)
        self.dim, self._dev = self.latent_dim + self.rope_dim, _device(device)
        desc = MoeLatentDesc(int(max_requests), self.n_heads, self.latent_dim, self.rope_dim)
        h = ctypes.c_void_p()
        with torch.cuda.device(self._dev):
            _check(_lib.moe_latent_create(ctypes.byref(desc), ctypes.byref(h)))
        self.handle = h

    def close(self):
        if getattr(self, "handle", None) is not None and self.handle.value:
            handle, self.handle = self.handle, None
            _destroy(_lib.moe_latent_destroy, handle)

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def decode(self, q, cache, block_table, seq_len, scale, k_scale=1.0, out=None, lse=None, stream=None):
        """q [n, heads, latent + rope] float16 or bfloat16: each head's query with
        the key expansion absorbed, then its rotary part; cache [pages, page_size,
        1, latent + rope] (or without the 1) of q's type or float8_e4m3fn, as
        Rope.append writes it; block_table int32 [>= n, pages]; seq_len int32 [>= n],
        the new token's own row included; scale: on q . row (1 / sqrt of the
        expanded head's size).  Returns (out [n, heads, latent], lse [n, heads] fp32);
        the value expansion is the caller's.  A request that sees no token gets 0
        and -inf."""
        dev, heads, dim, dt = self._dev, self.n_heads, self.dim, q.dtype
        _here(dev, q, cache, block_table, seq_len, out, lse)
        act, shape = _HALF.get(dt), q.shape
        n = shape[0] if shape else 0
        if act is None or shape != (n, heads, dim) or q.stride(2) != 1:
            raise ValueError(f"q: expected float16 or bfloat16 [n, {heads}, {dim}] with contiguous rows, got {dt} "
                             f"{tuple(shape)}")
        cs, ct, qt, cd = cache.shape, cache.stride(), q.stride(), cache.dtype
        if (cd is not dt and cd is not _E4M3) or len(cs) not in (3, 4) or cs[-1] != dim or ct[-1] != 1 or (
                len(cs) == 4 and cs[2] != 1):
            raise ValueError(f"cache: expected {dt} or float8_e4m3fn [pages, page_size, 1, {dim}] with contiguous rows, got "
                             f"{cd} {tuple(cs)}")
        cols, row = _table(block_table, n)
        if seq_len.dtype is not torch.int32 or seq_len.dim() != 1 or seq_len.shape[0] < n or \
                not seq_len.is_contiguous():
            raise ValueError(f"seq_len: expected a contiguous int32 tensor of at least {n} entries")
        latent = self.latent_dim
        if out is None:
            out, os = _out((n, heads, latent), dt, dev, stream), (heads * latent, latent)
        elif out.dtype is not dt or out.shape != (n, heads, latent) or out.stride(2) != 1:
            raise ValueError(f"out: expected {dt} {(n, heads, latent)} with contiguous rows")
        else:
            os = out.stride()
        if lse is None:
            lse = _out((n, heads), torch.float32, dev, stream)
        else:
            _ints("lse", lse, (n, heads), torch.float32)
        many, many_h = n > 1, heads > 1  # a stride counts where there is something to step to
        try:
            args = _LATENT_ARGS.pack(
                n, act, act if cd is dt else MOE_E4M3, cs[1], cols, scale, k_scale, seq_len.data_ptr(),
                block_table.data_ptr(), row, cs[0], q.data_ptr(), cache.data_ptr(), out.data_ptr(), lse.data_ptr(),
                qt[0] * many, qt[1] * many_h, os[0] * many, os[1] * many_h, ct[0] if cs[0] > 1 else 0,
                ct[1] if cs[1] > 1 else 0)
        except _UNPACKABLE as e:
            _refuse(e)
        _check(_lib.moe_latent_decode(self.handle, args, _raw(stream, dev)))
        return out, lse


def latent_prompt(q, k, k_rope, v, q_start, kv_start, scale, causal=True, out=None, lse=None, stream=None):
    """moe_latent_prompt: attention of the new tokens of ragged prompts over keys
    and values expanded a head, the rotary part of the keys shared by the heads.

    q [queries, heads, nope + rope], k [keys, heads, nope], k_rope [keys, rope]
    (None: no rotary part), v [keys, heads, v_dim], all float16 or all bfloat16 with
    contiguous rows and free strides (k and v may be views of one projection);
    q_start, kv_start int32 [requests + 1] as KvPlan.q_start: request b holds queries
    q_start[b] .. q_start[b + 1] and keys kv_start[b] .. kv_start[b + 1].  causal: a
    request's queries are its last tokens, each sees the keys up to its own.
    Returns (out [queries, heads, v_dim], lse [queries, heads] fp32); rows behind
    the last request are left as they were, a query that sees no key gets 0 and -inf."""
    dev = q.get_device()
    _here(dev, q, k, k_rope, v, q_start, kv_start, out, lse)
    dt, qs, ks, vs = q.dtype, q.shape, k.shape, v.shape
    act = _HALF.get(dt)
    rs = None if k_rope is None else k_rope.shape
    rope = rs[1] if rs is not None and len(rs) == 2 else 0
    if act is None or len(qs) != 3 or len(ks) != 3 or len(vs) != 3 or k.dtype is not dt or v.dtype is not dt or \
            ks[1] != qs[1] or vs[1] != qs[1] or vs[0] != ks[0] or qs[2] != ks[2] + rope or \
            (rs is not None and (len(rs) != 2 or rs[0] != ks[0] or k_rope.dtype is not dt)):
        raise ValueError("expected float16 or bfloat16 q [queries, heads, nope + rope], k [keys, heads, nope], k_rope [keys, rope] "
                         f"and v [keys, heads, v_dim] of one type, got "
                         f"{[None if t is None else (t.dtype, tuple(t.shape)) for t in (q, k, k_rope, v)]}")
    nq, heads, _ = qs
    nk, _, nope = ks
    v_dim = vs[2]
    if out is None:
        out, os = _out((nq, heads, v_dim), dt, dev, stream), (heads * v_dim, v_dim, 1)
    elif out.dtype is not dt or out.shape != (nq, heads, v_dim):
        raise ValueError(f"out: expected {dt} {(nq, heads, v_dim)}, got {out.dtype} {tuple(out.shape)}")
    else:
        os = out.stride()
    if lse is None:
        lse = _out((nq, heads), torch.float32, dev, stream)
    else:
        _ints("lse", lse, (nq, heads), torch.float32)
    qt, kt, vt, rt = q.stride(), k.stride(), v.stride(), (0, 1) if rs is None else k_rope.stride()
    if qt[2] != 1 or kt[2] != 1 or vt[2] != 1 or rt[1] != 1 or os[2] != 1:
        raise ValueError("expected q, k, k_rope, v and out with contiguous rows")
    n = q_start.shape[0] - 1 if q_start.dim() == 1 else 0
    _ints("q_start", q_start, (n + 1,))
    _ints("kv_start", kv_start, (n + 1,))
    many_q, many_k, many_h = nq > 1, nk > 1, heads > 1  # a stride counts where there is something to step to
    try:
        args = _PROMPT_ARGS.pack(
            n, heads, nq, nk, nope, rope, v_dim, act, bool(causal), scale, q_start.data_ptr(), kv_start.data_ptr(),
            q.data_ptr(), k.data_ptr(), 0 if rs is None else k_rope.data_ptr(), v.data_ptr(), out.data_ptr(),
            lse.data_ptr(), qt[0] * many_q, qt[1] * many_h, kt[0] * many_k, kt[1] * many_h, rt[0] * many_k, vt[0] * many_k,
            vt[1] * many_h, os[0] * many_q, os[1] * many_h)
    except _UNPACKABLE as e:
        _refuse(e)
    _check(_lib.moe_latent_prompt(args, _raw(stream, dev)))
    return out, lse


def dense_status(stream=None) -> int:
    """Reads and clears the error flags that the calls of this module left on the
    current device (0 when none); synchronises the stream."""
    v = _ci(0)
    rc = _lib.moe_dense_status(_stream(stream), ctypes.byref(v))
    if rc != -5:  # MOE_ERR_DEVICE: the flags are the answer
        _check(rc)
    return int(v.value)
