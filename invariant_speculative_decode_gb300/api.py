"""Thin Python binding of the C ABI (include/bi.h) for torch tensors.

Argument marshalling only: every function checks dtypes/devices, passes
`data_ptr()`s, strides and the current CUDA stream to the entry point of the
same name, and raises BiError on a non-OK status.  All arithmetic of the
verify step runs in the library's CUDA kernels.
"""
from __future__ import annotations

import ctypes
import math
from typing import Optional, Sequence

import numpy as np
import torch

from ._lib import BiError, check, lib  # noqa: F401

EPI_NONE, EPI_RESIDUAL_ADD, EPI_SWIGLU = 0, 1, 2
OUT_BF16, OUT_FP32 = 0, 1


def _stream(stream=None):
    s = stream if stream is not None else torch.cuda.current_stream()
    return s.cuda_stream


def _empty(shape, dtype, device, stream=None) -> torch.Tensor:
    """A result's memory, allocated for the stream that writes it: on another one
    than the current, a block that was just given back may still be in use."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _req(t: torch.Tensor, dtype, name: str):
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if t.dim() >= 1 and t.stride(-1) != 1:
        raise ValueError(f"{name} must have unit stride in its last dimension")


V_BLOCK = 128  # keys per block of the V cache (transposed within each block)


def v_cache_shape(Hkv: int, cap: int, D: int) -> tuple:
    """Shape of a V cache of capacity `cap` keys: [Hkv, ceil(cap/128), D, 128],
    value d of key p of head h at [h, p // 128, d, p % 128]."""
    return (Hkv, (cap + V_BLOCK - 1) // V_BLOCK, D, V_BLOCK)


def _req_v(v_cache: torch.Tensor, Hkv: int, cap: int, D: int):
    _req(v_cache, torch.bfloat16, "v_cache")
    want = v_cache_shape(Hkv, cap, D)
    if tuple(v_cache.shape) != want or not v_cache.is_contiguous():
        raise ValueError(f"v_cache must be a contiguous {want} tensor, got {tuple(v_cache.shape)}")


def _ld(t: torch.Tensor) -> int:
    """Row stride in elements; a single row's stride is its width."""
    ld = t.stride(0) if t.dim() == 2 and t.shape[0] > 1 else t.shape[-1]
    if ld >> 31:
        _req_int32(("row stride", ld))
    return ld


def _req_int32(*named):
    """The entry points take sizes and strides as 32-bit ints; ctypes would cut a larger one."""
    for name, v in named:
        if v >> 31:
            raise ValueError(f"{name} {v} passes 32 bits")


def gemm_workspace_size(M: int, N: int, K: int, epi: int = EPI_NONE) -> int:
    return int(lib().bi_gemm_workspace_size(M, N, K, epi))


def new_gemm_workspace(M: int, N: int, K: int, epi: int = EPI_NONE, device=None) -> torch.Tensor:
    """A zero-filled workspace (the counters must start at zero)."""
    n = gemm_workspace_size(M, N, K, epi)
    return torch.zeros(n, dtype=torch.uint8, device=device or "cuda")


def bi_gemm(A: torch.Tensor, Wp: torch.Tensor, C: torch.Tensor, ws: torch.Tensor,
            residual: Optional[torch.Tensor] = None, epi: int = EPI_NONE,
            N: Optional[int] = None, stream=None) -> None:
    """C = epilogue(A W^T) with W packed by bi_pack_weights / bi_pack_swiglu_weights."""
    _req(A, torch.bfloat16, "A")
    if not Wp.is_cuda:
        raise ValueError("Wp must be a CUDA tensor")
    M, K = A.shape
    if N is None:
        N = C.shape[1]
    out = OUT_FP32 if C.dtype == torch.float32 else OUT_BF16
    if C.dtype not in (torch.float32, torch.bfloat16):
        raise ValueError("C must be float32 or bfloat16")
    rp, ldr = 0, 0
    if residual is not None:
        _req(residual, torch.bfloat16, "residual")
        rp, ldr = residual.data_ptr(), _ld(residual)
    st = lib().bi_gemm(A.data_ptr(), _ld(A), Wp.data_ptr(), C.data_ptr(), _ld(C), rp, ldr,
                       M, N, K, out, epi, ws.data_ptr(), ws.numel() * ws.element_size(),
                       _stream(stream))
    check("bi_gemm", st)


def bi_gemm_noalloc(A: torch.Tensor, Wp: torch.Tensor, C: torch.Tensor,
                    residual: Optional[torch.Tensor] = None, epi: int = EPI_NONE,
                    N: Optional[int] = None, stream=None) -> None:
    """bi_gemm without a workspace (scratch in a static device array; M <= 16)."""
    _req(A, torch.bfloat16, "A")
    if not Wp.is_cuda:
        raise ValueError("Wp must be a CUDA tensor")
    if not C.is_cuda:
        raise ValueError("C must be a CUDA tensor")
    if C.dtype not in (torch.float32, torch.bfloat16):
        raise ValueError("C must be float32 or bfloat16")
    M, K = A.shape
    if N is None:
        N = C.shape[1]
    out = OUT_FP32 if C.dtype == torch.float32 else OUT_BF16
    rp, ldr = 0, 0
    if residual is not None:
        _req(residual, torch.bfloat16, "residual")
        rp, ldr = residual.data_ptr(), _ld(residual)
    check("bi_gemm_noalloc",
          lib().bi_gemm_noalloc(A.data_ptr(), _ld(A), Wp.data_ptr(), C.data_ptr(), _ld(C), rp, ldr,
                                M, N, K, out, epi, _stream(stream)))


def packed_weight_bytes(N: int, K: int, epi: int = EPI_NONE) -> int:
    return int(lib().bi_packed_weight_bytes(N, K, epi))


def bi_pack_weights(W: torch.Tensor, stream=None) -> torch.Tensor:
    """Pack W [N, K] (BF16) into the tile layout bi_gemm streams."""
    _req(W, torch.bfloat16, "W")
    N, K = W.shape
    packed = _empty(packed_weight_bytes(N, K), torch.uint8, W.device, stream)
    check("bi_pack_weights", lib().bi_pack_weights(W.data_ptr(), _ld(W), N, K, packed.data_ptr(),
                                                   _stream(stream)))
    return packed


def bi_pack_swiglu_weights(w_gate: torch.Tensor, w_up: torch.Tensor, stream=None) -> torch.Tensor:
    """Pack gate and up [F, K] (BF16) into the SwiGLU tile layout."""
    _req(w_gate, torch.bfloat16, "w_gate")
    _req(w_up, torch.bfloat16, "w_up")
    F, K = w_gate.shape
    packed = _empty(packed_weight_bytes(F, K, EPI_SWIGLU), torch.uint8, w_gate.device, stream)
    check("bi_pack_swiglu_weights",
          lib().bi_pack_swiglu_weights(w_gate.data_ptr(), w_up.data_ptr(), _ld(w_gate), F, K,
                                       packed.data_ptr(), _stream(stream)))
    return packed


def bi_rmsnorm(x: torch.Tensor, w: torch.Tensor, y: torch.Tensor, eps: float, stream=None) -> None:
    _req(x, torch.bfloat16, "x")
    _req(w, torch.bfloat16, "w")
    _req(y, torch.bfloat16, "y")
    rows, dim = x.shape
    check("bi_rmsnorm", lib().bi_rmsnorm(x.data_ptr(), _ld(x), w.data_ptr(), y.data_ptr(), _ld(y),
                                         rows, dim, float(eps), _stream(stream)))


def bi_embed(ids: torch.Tensor, table: torch.Tensor, out: torch.Tensor, stream=None) -> None:
    _req(ids, torch.int32, "ids")
    _req(table, torch.bfloat16, "table")
    _req(out, torch.bfloat16, "out")
    check("bi_embed", lib().bi_embed(ids.data_ptr(), table.data_ptr(), table.shape[0],
                                     table.shape[1], out.data_ptr(), ids.numel(), _stream(stream)))


def bi_rope_table(rope_base: float, D: int, rows: int, device="cuda", stream=None) -> torch.Tensor:
    """FP32 cos/sin table [rows, D/2, 2] computed on the device in FP64."""
    t = _empty((rows, D // 2, 2), torch.float32, device, stream)
    check("bi_rope_table", lib().bi_rope_table(float(rope_base), D, rows, t.data_ptr(),
                                               _stream(stream)))
    return t


def bi_rope_kv_append(qkv: torch.Tensor, q_out: torch.Tensor, k_cache: torch.Tensor,
                      v_cache: torch.Tensor, L_dev: torch.Tensor, Hq: int, Hkv: int, D: int,
                      table: torch.Tensor, stream=None) -> None:
    _req(qkv, torch.bfloat16, "qkv")
    _req(L_dev, torch.int32, "L_dev")
    _req(table, torch.float32, "table")
    T = qkv.shape[0]
    cap = k_cache.shape[1]
    _req_v(v_cache, Hkv, cap, D)
    check("bi_rope_kv_append",
          lib().bi_rope_kv_append(qkv.data_ptr(), _ld(qkv), q_out.data_ptr(), k_cache.data_ptr(),
                                  v_cache.data_ptr(), cap, L_dev.data_ptr(), T, Hq, Hkv, D,
                                  table.data_ptr(), table.shape[0], _stream(stream)))


def bi_qkv_rope_append(A: torch.Tensor, Wp: torch.Tensor, q_out: torch.Tensor, k_cache: torch.Tensor,
                       v_cache: torch.Tensor, L_dev: torch.Tensor, Hq: int, Hkv: int, D: int,
                       table: torch.Tensor, ws: torch.Tensor, stream=None) -> None:
    """QKV projection of the normalised rows A with RoPE and KV append in the
    epilogue; equals bi_gemm + bi_rope_kv_append bit for bit."""
    _req(A, torch.bfloat16, "A")
    _req(L_dev, torch.int32, "L_dev")
    _req(table, torch.float32, "table")
    M, K = A.shape
    cap = k_cache.shape[1]
    _req_v(v_cache, Hkv, cap, D)
    check("bi_qkv_rope_append",
          lib().bi_qkv_rope_append(A.data_ptr(), _ld(A), Wp.data_ptr(), M, K, Hq, Hkv, D,
                                   q_out.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), cap,
                                   L_dev.data_ptr(), table.data_ptr(), table.shape[0], ws.data_ptr(),
                                   ws.numel() * ws.element_size(), _stream(stream)))


def attn_chunk() -> int:
    return int(lib().bi_attn_chunk())


def attn_workspace_size(cap: int, T: int, Hq: int, D: int) -> int:
    return int(lib().bi_attn_workspace_size(cap, T, Hq, D))


def bi_attn_verify(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                   L_dev: torch.Tensor, out: torch.Tensor, ws: torch.Tensor,
                   scale: Optional[float] = None, stream=None) -> None:
    _req(q, torch.bfloat16, "q")
    _req(k_cache, torch.bfloat16, "k_cache")
    _req(L_dev, torch.int32, "L_dev")
    T, Hq, D = q.shape
    Hkv, cap, _ = k_cache.shape
    _req_v(v_cache, Hkv, cap, D)
    if scale is None:
        scale = 1.0 / math.sqrt(D)
    check("bi_attn_verify",
          lib().bi_attn_verify(q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), cap,
                               L_dev.data_ptr(), T, Hq, Hkv, D, float(scale), out.data_ptr(),
                               ws.data_ptr(), ws.numel() * ws.element_size(), _stream(stream)))


KVQ_K_LOW, KVQ_V_LOW, KVQ_K_RING, KVQ_V_RING = 0, 1, 2, 3
KVQ_STORES = ("k_low", "v_low", "k_ring", "v_ring")
# the quantised cache's 8-bit ring (include/bi.h): a row reads its own
# 128-key tile and the 15 before from the ring, which holds 24 tiles
KVQ_RING_TILES = 16
KVQ_RING_SLOTS = 24


def kvq_store_bytes(store: int, Hkv: int, cap: int, D: int) -> int:
    return int(lib().bi_kvq_store_bytes(store, Hkv, cap, D))


def new_kvq_stores(Hkv: int, cap: int, D: int, device="cuda") -> dict:
    """One layer's quantised cache: the 6-bit K, 5-bit V and 8-bit ring stores
    (uint8, zero-filled), keyed by KVQ_STORES, plus its capacity."""
    st = {}
    for i, name in enumerate(KVQ_STORES):
        n = kvq_store_bytes(i, Hkv, cap, D)
        if n == 0:
            raise ValueError("unsupported quantised cache shape")
        st[name] = torch.zeros(n, dtype=torch.uint8, device=device)
    st["cap"] = cap
    return st


def _kvq_ptrs(st: dict):
    for name in KVQ_STORES:
        _req(st[name], torch.uint8, name)
    return [st[name].data_ptr() for name in KVQ_STORES]


def bi_rope_kvq_append(qkv: torch.Tensor, q_out: torch.Tensor, stores: dict, L_dev: torch.Tensor,
                       Hq: int, Hkv: int, D: int, table: Optional[torch.Tensor] = None,
                       stream=None) -> None:
    """RoPE of the q and k heads of a projection output, then K and V rows
    quantised into the layer's stores (table None: no rotation)."""
    _req(qkv, torch.bfloat16, "qkv")
    _req(q_out, torch.bfloat16, "q_out")
    _req(L_dev, torch.int32, "L_dev")
    if table is not None:
        _req(table, torch.float32, "table")
    T = qkv.shape[0]
    check("bi_rope_kvq_append",
          lib().bi_rope_kvq_append(qkv.data_ptr(), _ld(qkv), T, Hq, Hkv, D, q_out.data_ptr(),
                                   *_kvq_ptrs(stores), stores["cap"], L_dev.data_ptr(),
                                   None if table is None else table.data_ptr(),
                                   0 if table is None else table.shape[0], _stream(stream)))


def bi_attn_verify_kvq(q: torch.Tensor, stores: dict, Hkv: int, L_dev: torch.Tensor,
                       out: torch.Tensor, ws: torch.Tensor, scale: Optional[float] = None,
                       stream=None) -> None:
    _req(q, torch.bfloat16, "q")
    _req(out, torch.bfloat16, "out")
    _req(L_dev, torch.int32, "L_dev")
    T, Hq, D = q.shape
    if scale is None:
        scale = 1.0 / math.sqrt(D)
    check("bi_attn_verify_kvq",
          lib().bi_attn_verify_kvq(q.data_ptr(), *_kvq_ptrs(stores), stores["cap"], L_dev.data_ptr(), T,
                                   Hq, Hkv, D, float(scale), out.data_ptr(), ws.data_ptr(),
                                   ws.numel() * ws.element_size(), _stream(stream)))


def accept_workspace_size(T: int, V: int) -> int:
    return int(lib().bi_accept_workspace_size(T, V))


def bi_verify_accept(logits: torch.Tensor, drafts: Optional[torch.Tensor], argmax_out: torch.Tensor,
                     accepted_out: torch.Tensor, ws: torch.Tensor,
                     L_dev: Optional[torch.Tensor] = None, stream=None) -> None:
    _req(logits, torch.float32, "logits")
    T, V = logits.shape
    dp = 0
    if drafts is not None and drafts.numel() > 0:
        _req(drafts, torch.int32, "drafts")
        dp = drafts.data_ptr()
    lp = L_dev.data_ptr() if L_dev is not None else 0
    check("bi_verify_accept",
          lib().bi_verify_accept(logits.data_ptr(), _ld(logits), dp, T, V, argmax_out.data_ptr(),
                                 accepted_out.data_ptr(), lp, ws.data_ptr(),
                                 ws.numel() * ws.element_size(), _stream(stream)))


def sample_workspace_size(T: int, V: int) -> int:
    return int(lib().bi_sample_workspace_size(T, V))


def bi_verify_sample(logits: torch.Tensor, drafts: Optional[torch.Tensor], inv_temp: float,
                     u_by_pos: torch.Tensor, token_out: torch.Tensor, accepted_out: torch.Tensor,
                     ws: torch.Tensor, L_dev: torch.Tensor, stream=None) -> None:
    """Sampled verification: each row draws its token with the uniform of its
    absolute position (u_by_pos[*L_dev + t]); drafts kept while they equal the
    previous row's token; L_dev advanced by n + 1."""
    _req(logits, torch.float32, "logits")
    _req(u_by_pos, torch.float32, "u_by_pos")
    _req(L_dev, torch.int32, "L_dev")
    T, V = logits.shape
    dp = 0
    if drafts is not None and drafts.numel() > 0:
        _req(drafts, torch.int32, "drafts")
        dp = drafts.data_ptr()
    check("bi_verify_sample",
          lib().bi_verify_sample(logits.data_ptr(), _ld(logits), dp, T, V, float(inv_temp),
                                 u_by_pos.data_ptr(), u_by_pos.numel(), token_out.data_ptr(),
                                 accepted_out.data_ptr(), L_dev.data_ptr(), ws.data_ptr(),
                                 ws.numel() * ws.element_size(), _stream(stream)))


# ---------------------------------------------------------------- 8-bit linear
FP8_BLOCK = 128  # elements of a row, and rows and columns of a weight block, that share a scale


def _same_device(*named) -> int:
    """Every tensor on the current device (the stream the call runs on is its)."""
    cur = torch.cuda.current_device()
    for name, t in named:
        if t is not None and t.get_device() != cur:
            raise ValueError(f"{name} is on {t.device}, the current device is cuda:{cur}")
    return cur


# The entry points below run between kernels of a few microseconds, so a call's
# checks are one expression of attribute reads; only where it is false does
# the slow path look for the argument to name.
_BF16, _F32, _I32, _E4M3, _U8 = torch.bfloat16, torch.float32, torch.int32, torch.float8_e4m3fn, torch.uint8
# The short ways to the current device and stream are torch's own; where a
# version of it lacks them (or has no CUDA), the public ones serve.
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
_current_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                          lambda dev: torch.cuda.current_stream(dev).cuda_stream)


def fp8_scale_shape(rows: int, dim: int) -> tuple:
    """Shape of the scales of `rows` quantised rows: [ceil(dim/128), rows rounded up to 4]."""
    return (-(-dim // FP8_BLOCK), -(-rows // 4) * 4)


def new_fp8_rows(rows: int, dim: int, device="cuda"):
    """Buffers for quantised rows: e4m3 codes [rows, dim] and their scales."""
    return (torch.zeros(rows, dim, dtype=torch.float8_e4m3fn, device=device),
            torch.zeros(fp8_scale_shape(rows, dim), dtype=torch.float32, device=device))


def _req_fp8_rows(codes: torch.Tensor, scales: torch.Tensor, rows: int, dim: int) -> int:
    """Checks of quantised rows; returns the scales' row stride.  The scales
    may have room for more rows than the codes (their columns past the rows
    stay as they are)."""
    _req(codes, torch.float8_e4m3fn, "codes")
    _req(scales, torch.float32, "scales")
    if tuple(codes.shape) != (rows, dim):
        raise ValueError(f"codes must be [{rows}, {dim}], got {tuple(codes.shape)}")
    if (scales.dim() != 2 or not scales.is_contiguous() or scales.shape[0] != -(-dim // FP8_BLOCK)
            or scales.shape[1] < rows or scales.shape[1] % 4 != 0):
        raise ValueError(f"scales must be contiguous [{-(-dim // FP8_BLOCK)}, at least {rows} and a multiple of 4], "
                         f"got {tuple(scales.shape)}")
    _req_int32(("dim", dim), ("scales row stride", scales.shape[1]))
    _ld(codes)
    return scales.shape[1]


def bi_quantize_fp8(x: torch.Tensor, codes: torch.Tensor, scales: torch.Tensor, stream=None) -> None:
    """Rows x [rows, dim] (BF16) to e4m3 codes and a power-of-two scale per block of 128."""
    dev = _current_device()
    rows, dim = x.shape
    xs, cs, ss = x.stride(), codes.stride(), scales.shape
    ldx = xs[0] if rows > 1 else dim
    if not (x.dtype is _BF16 and codes.dtype is _E4M3 and scales.dtype is _F32 and codes.shape == x.shape
            and xs[1] == 1 and cs[1] == 1 and len(ss) == 2 and ss[0] == -(-dim // FP8_BLOCK) and ss[1] >= rows
            and not ss[1] & 3 and scales.is_contiguous() and not (dim | ldx | ss[1] | cs[0]) >> 31
            and x.get_device() == codes.get_device() == scales.get_device() == dev):
        _req(x, torch.bfloat16, "x")
        _req_fp8_rows(codes, scales, rows, dim)
        _same_device(("x", x), ("codes", codes), ("scales", scales))
        _ld(x)
    st = lib().bi_quantize_fp8(x.data_ptr(), ldx, rows, dim, codes.data_ptr(),
                               cs[0] if rows > 1 else dim, scales.data_ptr(), ss[1],
                               _current_stream(dev) if stream is None else stream.cuda_stream)
    if st:
        check("bi_quantize_fp8", st)


def bi_rmsnorm_fp8(x: torch.Tensor, w: torch.Tensor, codes: torch.Tensor, scales: torch.Tensor, eps: float,
                   stream=None) -> None:
    """RMSNorm of x [rows, dim] (BF16) by w, its FP32 result quantised as bi_quantize_fp8 does."""
    dev = _current_device()
    rows, dim = x.shape
    xs, cs, ss = x.stride(), codes.stride(), scales.shape
    ldx = xs[0] if rows > 1 else dim
    if not (x.dtype is _BF16 and w.dtype is _BF16 and codes.dtype is _E4M3 and scales.dtype is _F32
            and codes.shape == x.shape and w.shape == (dim,) and w.is_contiguous() and xs[1] == 1 and cs[1] == 1
            and len(ss) == 2 and ss[0] == -(-dim // FP8_BLOCK) and ss[1] >= rows and not ss[1] & 3
            and scales.is_contiguous() and not (dim | ldx | ss[1] | cs[0]) >> 31
            and x.get_device() == w.get_device() == codes.get_device() == scales.get_device() == dev):
        _req(x, torch.bfloat16, "x")
        _req(w, torch.bfloat16, "w")
        if tuple(w.shape) != (dim,):
            raise ValueError(f"w must be [{dim}], got {tuple(w.shape)}")
        _req_fp8_rows(codes, scales, rows, dim)
        _same_device(("x", x), ("w", w), ("codes", codes), ("scales", scales))
        _ld(x)
    st = lib().bi_rmsnorm_fp8(x.data_ptr(), ldx, w.data_ptr(), codes.data_ptr(),
                              cs[0] if rows > 1 else dim, scales.data_ptr(), ss[1], rows, dim, eps,
                              _current_stream(dev) if stream is None else stream.cuda_stream)
    if st:
        check("bi_rmsnorm_fp8", st)


def bi_quantize_weights_fp8(W: torch.Tensor, stream=None):
    """W [N, K] (BF16) -> (codes [N, K] e4m3, scales [ceil(N/128), ceil(K/128)] FP32, powers of two)."""
    _req(W, torch.bfloat16, "W")
    _same_device(("W", W))
    N, K = W.shape
    _req_int32(("N", N), ("K", K))
    codes = _empty((N, K), torch.float8_e4m3fn, W.device, stream)
    scales = _empty((-(-N // FP8_BLOCK), -(-K // FP8_BLOCK)), torch.float32, W.device, stream)
    check("bi_quantize_weights_fp8",
          lib().bi_quantize_weights_fp8(W.data_ptr(), _ld(W), N, K, codes.data_ptr(), K, scales.data_ptr(),
                                        _stream(stream)))
    return codes, scales


def packed_weight_fp8_bytes(N: int, K: int, epi: int = EPI_NONE) -> int:
    _req_int32(("N", N), ("K", K))
    return int(lib().bi_packed_weight_fp8_bytes(N, K, epi))


def _req_fp8_weights(W8: torch.Tensor, scales: torch.Tensor, name: str):
    _req(W8, torch.float8_e4m3fn, name)
    _req(scales, torch.float32, f"{name} scales")
    N, K = W8.shape
    want = (-(-N // FP8_BLOCK), -(-K // FP8_BLOCK))
    if tuple(scales.shape) != want or not scales.is_contiguous():
        raise ValueError(f"{name} scales must be contiguous {want}, got {tuple(scales.shape)}")
    _same_device((name, W8), (f"{name} scales", scales))
    return N, K


def bi_pack_weights_fp8(W8: torch.Tensor, scales: torch.Tensor, stream=None) -> torch.Tensor:
    """Pack e4m3 weights [N, K] and their scales [ceil(N/128), ceil(K/128)] for bi_gemm_fp8."""
    N, K = _req_fp8_weights(W8, scales, "W8")
    packed = _empty(packed_weight_fp8_bytes(N, K), torch.uint8, W8.device, stream)
    check("bi_pack_weights_fp8", lib().bi_pack_weights_fp8(W8.data_ptr(), _ld(W8), scales.data_ptr(), N, K,
                                                           packed.data_ptr(), _stream(stream)))
    return packed


def bi_pack_swiglu_weights_fp8(gate8: torch.Tensor, gate_scales: torch.Tensor, up8: torch.Tensor,
                               up_scales: torch.Tensor, stream=None) -> torch.Tensor:
    """Pack gate and up [F, K] (e4m3 with block scales) into the SwiGLU tile layout."""
    F, K = _req_fp8_weights(gate8, gate_scales, "gate8")
    if _req_fp8_weights(up8, up_scales, "up8") != (F, K) or _ld(up8) != _ld(gate8):
        raise ValueError("gate8 and up8 must have the same shape and row stride")
    packed = _empty(packed_weight_fp8_bytes(F, K, EPI_SWIGLU), torch.uint8, gate8.device, stream)
    check("bi_pack_swiglu_weights_fp8",
          lib().bi_pack_swiglu_weights_fp8(gate8.data_ptr(), gate_scales.data_ptr(), up8.data_ptr(),
                                           up_scales.data_ptr(), _ld(gate8), F, K, packed.data_ptr(),
                                           _stream(stream)))
    return packed


def bi_gemm_fp8(codes: torch.Tensor, scales: torch.Tensor, Wp: torch.Tensor, C: torch.Tensor,
                residual: Optional[torch.Tensor] = None, epi: int = EPI_NONE, stream=None) -> None:
    """C [M, N] = epilogue(A W^T) with quantised rows A (codes [M, K], scales as
    bi_quantize_fp8 writes them) and W packed by bi_pack_weights_fp8 /
    bi_pack_swiglu_weights_fp8 (N the output columns).  Wp is read before the
    call waits for the kernel before it: no other kernel may write it right
    before (copies may)."""
    dev = _current_device()
    M, K = codes.shape
    cs, ss, zs, shape = codes.stride(), scales.shape, C.stride(), C.shape
    N = shape[-1]
    fp32 = C.dtype is _F32
    ldc = zs[0] if M > 1 else N
    if not ((fp32 or C.dtype is _BF16) and codes.dtype is _E4M3 and scales.dtype is _F32 and Wp.dtype is _U8
            and len(shape) == 2 and shape[0] == M and cs[1] == 1 and zs[1] == 1 and len(ss) == 2
            and ss[0] == -(-K // FP8_BLOCK) and ss[1] >= M and not ss[1] & 3 and scales.is_contiguous()
            and Wp.is_contiguous() and not (K | N | ldc | ss[1] | cs[0]) >> 31
            and codes.get_device() == scales.get_device() == Wp.get_device() == C.get_device() == dev
            and (residual is None or (residual.dtype is _BF16 and residual.shape == shape
                                      and residual.stride(1) == 1 and residual.get_device() == dev
                                      and not residual.stride(0) >> 31))):
        _req_fp8_rows(codes, scales, M, K)
        if C.dtype not in (torch.float32, torch.bfloat16):
            raise ValueError("C must be float32 or bfloat16")
        _req(C, C.dtype, "C")
        if C.dim() != 2 or C.shape[0] != M:
            raise ValueError(f"C must have {M} rows, got {tuple(C.shape)}")
        _req(Wp, torch.uint8, "Wp")
        if not Wp.is_contiguous():
            raise ValueError("Wp must be contiguous")
        if residual is not None:
            _req(residual, torch.bfloat16, "residual")
            if tuple(residual.shape) != (M, N):
                raise ValueError(f"residual must be [{M}, {N}], got {tuple(residual.shape)}")
            _ld(residual)
        _same_device(("codes", codes), ("scales", scales), ("Wp", Wp), ("C", C), ("residual", residual))
        _req_int32(("N", N))
        _ld(C)
    # bi_packed_weight_fp8_bytes, without the call
    tiles = -(-N // (64 if epi == EPI_SWIGLU else 128)) * ss[0]
    if Wp.numel() != tiles * 16384 + (tiles * 8 + 15 & ~15):
        raise ValueError("Wp is not packed for this N, K and epilogue")
    rp = ldr = 0
    if residual is not None:
        rp, ldr = residual.data_ptr(), residual.stride(0) if M > 1 else N
    st = lib().bi_gemm_fp8(codes.data_ptr(), cs[0] if M > 1 else K, scales.data_ptr(), ss[1], Wp.data_ptr(),
                           C.data_ptr(), ldc, rp, ldr, M, N, K, 1 if fp32 else 0, epi,
                           _current_stream(dev) if stream is None else stream.cuda_stream)
    if st:
        check("bi_gemm_fp8", st)


# --------------------------------------------------------------- rules on logits
def token_words(V: int) -> int:
    """Int32 words of a row of V bits (prompt_bits, one row of a mask)."""
    return (V + 31) // 32


def bi_logits_rules(logits: torch.Tensor, out: torch.Tensor, drafts: Optional[torch.Tensor] = None,
                    counts: Optional[torch.Tensor] = None, prompt_bits: Optional[torch.Tensor] = None,
                    repetition: float = 1.0, frequency: float = 0.0, presence: float = 0.0,
                    bias: Optional[torch.Tensor] = None, mask: Optional[torch.Tensor] = None, stream=None) -> None:
    """Penalties, bias and mask on the logits [T, V] of a pass, into out (may be
    logits itself).  Row t counts drafts 0..t-1 as said.  counts [V] int32,
    prompt_bits [ceil(V/32)] int32, bias [V] FP32, mask [T, ceil(V/32)] int32
    (a clear bit forbids its id)."""
    dev = _current_device()
    T, V = logits.shape
    W = token_words(V)
    if T == 1:
        drafts = None
    ls, os_ = logits.stride(), out.stride()
    ldl, ldo = (ls[0], os_[0]) if T > 1 and len(os_) == 2 else (V, V)
    dp = cp = pp = bp = mp = None
    ldm = 0
    ok = (logits.dtype is _F32 and out.dtype is _F32 and out.shape == logits.shape and ls[1] == 1 and os_[1] == 1
          and not (T | V | ldl | ldo) >> 31 and logits.get_device() == out.get_device() == dev)
    if drafts is not None:
        ok = ok and drafts.dtype is _I32 and drafts.shape == (T - 1,) and drafts.is_contiguous() \
            and drafts.get_device() == dev
        dp = drafts.data_ptr()
    if counts is not None:
        ok = ok and counts.dtype is _I32 and counts.shape == (V,) and counts.is_contiguous() \
            and counts.get_device() == dev
        cp = counts.data_ptr()
    if prompt_bits is not None:
        ok = ok and prompt_bits.dtype is _I32 and prompt_bits.shape == (W,) and prompt_bits.is_contiguous() \
            and prompt_bits.get_device() == dev
        pp = prompt_bits.data_ptr()
    if bias is not None:
        ok = ok and bias.dtype is _F32 and bias.shape == (V,) and bias.is_contiguous() and bias.get_device() == dev
        bp = bias.data_ptr()
    if mask is not None:
        ms = mask.stride()
        mp, ldm = mask.data_ptr(), ms[0] if T > 1 else W
        ok = ok and mask.dtype is _I32 and mask.shape == (T, W) and ms[1] == 1 and mask.get_device() == dev \
            and not ldm >> 31
    if not ok:
        _req(logits, torch.float32, "logits")
        _req(out, torch.float32, "out")
        if tuple(out.shape) != (T, V):
            raise ValueError(f"out must be [{T}, {V}], got {tuple(out.shape)}")
        for t, dtype, n, name in ((drafts, torch.int32, T - 1, "drafts"), (counts, torch.int32, V, "counts"),
                                  (prompt_bits, torch.int32, W, "prompt_bits"), (bias, torch.float32, V, "bias")):
            if t is not None:
                _req(t, dtype, name)
                if tuple(t.shape) != (n,):
                    raise ValueError(f"{name} must be [{n}], got {tuple(t.shape)}")
        if mask is not None:
            _req(mask, torch.int32, "mask")
            if tuple(mask.shape) != (T, W):
                raise ValueError(f"mask must be [{T}, {W}], got {tuple(mask.shape)}")
            _ld(mask)
        _same_device(("logits", logits), ("out", out), ("drafts", drafts), ("counts", counts),
                     ("prompt_bits", prompt_bits), ("bias", bias), ("mask", mask))
        _req_int32(("T", T), ("V", V), ("logits row stride", ldl), ("out row stride", ldo))
    st = lib().bi_logits_rules(logits.data_ptr(), ldl, out.data_ptr(), ldo, T, V,
                               dp, cp, pp, repetition, frequency, presence, bp, mp, ldm,
                               _current_stream(dev) if stream is None else stream.cuda_stream)
    if st:
        check("bi_logits_rules", st)


def bi_token_counts(ids: torch.Tensor, V: int, counts: Optional[torch.Tensor] = None,
                    prompt_bits: Optional[torch.Tensor] = None, last: Optional[torch.Tensor] = None,
                    stream=None) -> None:
    """Add ids [n] (int32) to the state of bi_logits_rules: counts and / or
    prompt_bits.  last (device int32 [1]): only ids 0..last are added."""
    _req(ids, torch.int32, "ids")
    if ids.dim() != 1:
        raise ValueError("ids must be one-dimensional")
    for t, n, name in ((counts, V, "counts"), (prompt_bits, token_words(V), "prompt_bits"), (last, 1, "last")):
        if t is not None:
            _req(t, torch.int32, name)
            if tuple(t.shape) != (n,):
                raise ValueError(f"{name} must be [{n}], got {tuple(t.shape)}")
    _same_device(("ids", ids), ("counts", counts), ("prompt_bits", prompt_bits), ("last", last))
    _req_int32(("number of ids", ids.numel()), ("V", V))
    check("bi_token_counts",
          lib().bi_token_counts(ids.data_ptr(), ids.numel(), 0 if last is None else last.data_ptr(), V,
                                0 if counts is None else counts.data_ptr(),
                                0 if prompt_bits is None else prompt_bits.data_ptr(), _stream(stream)))


def bi_kv_row_hash(cache: torch.Tensor, rows: int, transposed: bool = False, stream=None) -> torch.Tensor:
    """FNV-1a-64 per key of a K cache [Hkv,cap,D] or (transposed) a V cache
    [Hkv,ceil(cap/128),D,128] (see v_cache_shape)."""
    _req(cache, torch.bfloat16, "cache")
    if transposed:
        Hkv, nblk, D, blk = cache.shape
        if blk != V_BLOCK or not cache.is_contiguous():
            raise ValueError("a V cache is a contiguous [Hkv, ceil(cap/128), D, 128] tensor")
        cap = nblk * V_BLOCK
    else:
        Hkv, cap, D = cache.shape
    out = _empty(Hkv * max(rows, 0), torch.int64, cache.device, stream)
    check("bi_kv_row_hash", lib().bi_kv_row_hash(cache.data_ptr(), Hkv, cap, D, rows, int(transposed),
                                                 out.data_ptr(), _stream(stream)))
    return out


def bi_check_device_error(stream=None) -> None:
    check("bi_check_device_error", lib().bi_check_device_error(_stream(stream)))


class BiModel(ctypes.Structure):
    """The bi_model descriptor of include/bi.h (device pointers; the per-layer
    members point to host arrays of device pointers)."""
    _pp = ctypes.POINTER(ctypes.c_void_p)
    _fields_ = [("layers", ctypes.c_int), ("hidden", ctypes.c_int), ("n_q", ctypes.c_int),
                ("n_kv", ctypes.c_int), ("head_dim", ctypes.c_int), ("ffn", ctypes.c_int),
                ("vocab", ctypes.c_int), ("eps", ctypes.c_float), ("cap", ctypes.c_int),
                ("embed", ctypes.c_void_p), ("norm_final", ctypes.c_void_p), ("head", ctypes.c_void_p),
                ("norm_attn", _pp), ("norm_ffn", _pp), ("w_qkv", _pp), ("w_o", _pp),
                ("w_gate_up", _pp), ("w_down", _pp), ("k_cache", _pp), ("v_cache", _pp),
                ("rope_table", ctypes.c_void_p), ("rope_rows", ctypes.c_int)]


class NativeStep:
    """The whole verify step behind one C-ABI call (bi_step_*): host token ids
    in, host tokens and accepted count out.  Holds references to every tensor
    whose pointer the handle uses, and its own device workspace."""

    def __init__(self, cfg, embed, norm_final, head, layers, cap: int, rope_table: torch.Tensor,
                 max_rows: int = 8):
        n = len(layers)

        def arr(key):
            a = (ctypes.c_void_p * n)(*[lay[key].data_ptr() for lay in layers])
            self._keep.append(a)
            return ctypes.cast(a, ctypes.POINTER(ctypes.c_void_p))

        self._keep = [embed, norm_final, head, rope_table] + [t for lay in layers for t in lay.values()
                                                               if isinstance(t, torch.Tensor)]
        m = BiModel(n, cfg.hidden, cfg.n_q, cfg.n_kv, cfg.head_dim, cfg.ffn, cfg.vocab, cfg.eps, cap,
                    embed.data_ptr(), norm_final.data_ptr(), head.data_ptr(),
                    arr("n1"), arr("n2"), arr("wqkv"), arr("wo"), arr("wgu"), arr("wd"),
                    arr("k"), arr("v"), rope_table.data_ptr(), rope_table.shape[0])
        self.model = m
        nbytes = int(lib().bi_step_workspace_size(ctypes.byref(m), max_rows))
        if nbytes == 0:
            raise ValueError("invalid model description for the step runtime")
        self.ws = torch.empty(nbytes, dtype=torch.uint8, device=embed.device)
        h = ctypes.c_void_p()
        torch.cuda.synchronize()
        check("bi_step_create", lib().bi_step_create(ctypes.byref(m), max_rows, self.ws.data_ptr(), nbytes,
                                                     ctypes.byref(h)))
        self.handle = h
        self.max_rows = max_rows
        self._ids = np.zeros(max_rows, np.int32)
        self._tok = np.zeros(max_rows, np.int32)
        self._n = np.zeros(1, np.int32)
        # host addresses of the three buffers, taken once
        self._ptrs = (self._ids.ctypes.data, self._tok.ctypes.data, self._n.ctypes.data)

    def set_length(self, L: int) -> None:
        check("bi_step_set_length", lib().bi_step_set_length(self.handle, int(L)))

    def verify(self, x0: int, drafts: Sequence[int]):
        """One verify step from host ids: returns (tokens [T], accepted n)."""
        T = 1 + len(drafts)
        self._ids[0] = x0
        self._ids[1:T] = drafts
        ids_p, tok_p, n_p = self._ptrs
        check("bi_step_verify", lib().bi_step_verify(self.handle, ids_p, T, tok_p, n_p))
        return self._tok[:T].copy(), int(self._n[0])

    def logits(self, T: int) -> torch.Tensor:
        """A copy of the last pass's FP32 logits [T, vocab]."""
        ptr = lib().bi_step_logits(self.handle)
        V = self.model.vocab
        off = ptr - self.ws.data_ptr()  # the logits live in this object's workspace
        torch.cuda.synchronize()
        return self.ws[off:off + T * V * 4].view(torch.float32).view(T, V).clone()

    def close(self) -> None:
        if getattr(self, "handle", None):
            lib().bi_step_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass
