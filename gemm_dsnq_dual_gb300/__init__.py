"""GB300-native decode-step MLA latent pre-projection.

Thin PyTorch binding over libdsnq (include/dsnq.h).  Tensors supply device
memory and the current CUDA stream; every step runs in the library's CUDA
kernels.  Output tensors are allocated here with torch when not supplied.

  fused_dual_rmsnorm_group_quant  -- dual RMSNorm + per-1x128 FP8 quant (one kernel)
  block_scaled_fp8_gemm           -- W8A8 block-scaled GEMM on the pre-quantized pair
  block_scaled_fp8_gemm_dual      -- both wq_b consumers in one launch
  quantize_weight_block128        -- load-time 128x128 weight-block quantization
  dual_rmsnorm_bf16, group_quant_bf16 -- the unfused baseline sequence
  extend_block_tables             -- block tables, positions and slots of a step
  head_rmsnorm_rope               -- per-head RMSNorm and rotary positions in one pass
  latent_cache_write              -- normalized, rotated latent rows into the paged cache
  paged_latent_attention          -- one new token per request over the paged latent cache

Method: vLLM PR #53540 (fused_qk_rmsnorm_group_quant feeding
apply_pre_quantized_block_scaled_mm for the attention and indexer wq_b) and
sglang PR #27289 (transpose_scale: column-major activation scales).
"""

from __future__ import annotations

import ctypes as C
import functools
import math
import threading

import torch

from ._native import DsnqError, check, lib  # noqa: F401

ROW_MAJOR = 0
COL_MAJOR = 1
GROUP = 128
ROPE_INTERLEAVED = 0
ROPE_HALF = 1

__all__ = [
    "ROW_MAJOR", "COL_MAJOR", "DsnqError",
    "fused_dual_rmsnorm_group_quant", "rmsnorm_group_quant", "dual_rmsnorm_bf16", "group_quant_bf16",
    "quantize_weight_block128", "block_scaled_fp8_gemm", "block_scaled_fp8_gemm_dual",
    "block_scaled_fp8_gemm_dual_bf16a", "block_scaled_fp8_gemm_dual_bf16a_static", "fused_quant_fits",
    "bf16a_workspace_bytes", "gemm_plan",
    "fused_norm_quant_gemm_dual",
    "ROPE_INTERLEAVED", "ROPE_HALF", "rope_frequencies", "extend_block_tables", "head_rmsnorm_rope",
    "latent_cache_write", "paged_latent_attention", "paged_latent_attention_workspace_bytes",
    "release_workspaces",
    "quant_output_sizes", "debug_status", "debug_set", "set_launch_overlap", "scale_layout_of", "scale_ld_for",
    "empty_scales",
]


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream, dev) -> int:
    """The stream handle for a call on tensors of device `dev`.  The library
    launches on the current CUDA device (and picks per-device state by it), so
    tensors on another device are refused rather than silently mixed."""
    if dev.type != "cuda":
        raise ValueError(f"tensors must be CUDA tensors, got {dev}")
    cur = torch.cuda.current_device()
    if dev.index is not None and dev.index != cur:
        raise ValueError(f"tensors are on {dev} but the current CUDA device is cuda:{cur}; "
                         f"call under torch.cuda.device({dev})")
    if stream is None:
        if _raw_stream is not None:          # the handle alone, without a Stream object around it
            return _raw_stream(cur)
        stream = torch.cuda.current_stream(cur)
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _layout(layout) -> int:
    if layout in (ROW_MAJOR, "row", "row_major"):
        return ROW_MAJOR
    if layout in (COL_MAJOR, "col", "col_major", "column_major"):
        return COL_MAJOR
    raise ValueError(f"unknown scale layout {layout!r}")


def _row_view_ok(t: torch.Tensor, name: str) -> int:
    """Row stride of a 2-D tensor whose rows are contiguous."""
    if t.dim() != 2 or (t.stride(1) != 1 and t.shape[1] > 1):
        raise ValueError(f"{name} must be 2-D with contiguous rows")
    return t.stride(0) if t.shape[0] > 1 else max(t.stride(0), t.shape[1])


def quant_output_sizes(M: int, Kq: int, group: int = GROUP, layout=ROW_MAJOR):
    """(n_scale_elems, default_ld_scale) of the scale buffer."""
    n, ld = C.c_int64(), C.c_int64()
    check(lib().dsnq_quant_output_sizes(M, Kq, group, _layout(layout), C.byref(n), C.byref(ld)),
          "dsnq_quant_output_sizes")
    return n.value, ld.value


def empty_scales(M: int, G: int, layout, device) -> torch.Tensor:
    """Logical [M, G] fp32 scale tensor in the requested memory layout
    (column-major = the transposed buffer viewed with strides (1, M))."""
    if _layout(layout) == ROW_MAJOR:
        return torch.empty(M, G, dtype=torch.float32, device=device)
    return torch.empty(G, M, dtype=torch.float32, device=device).t()


def scale_ld_for(scale: torch.Tensor, layout) -> int:
    """Leading dimension of a logical [M, G] scale tensor read in `layout`;
    raises if its memory does not have that layout."""
    M, G = scale.shape
    if _layout(layout) == ROW_MAJOR:
        if G > 1 and scale.stride(1) != 1:
            raise ValueError("scale tensor is not row-major")
        return scale.stride(0) if M > 1 else G
    if M > 1 and scale.stride(0) != 1:
        raise ValueError("scale tensor is not column-major")
    return scale.stride(1) if G > 1 else M


def scale_layout_of(scale: torch.Tensor):
    """(layout, ld) of a logical [M, G] scale tensor."""
    M, G = scale.shape
    if scale.stride(1) == 1 and (M <= 1 or scale.stride(0) >= G):
        return ROW_MAJOR, (scale.stride(0) if M > 1 else G)
    if scale.stride(0) == 1 and (G <= 1 or scale.stride(1) >= M):
        return COL_MAJOR, (scale.stride(1) if G > 1 else M)
    raise ValueError("scale tensor is neither row-major nor column-major")


def fused_dual_rmsnorm_group_quant(q, kv, gamma_q, gamma_kv, eps: float = 1e-6, group: int = GROUP,
                                   scale_layout=ROW_MAJOR, q_out=None, q_scale=None, kv_out=None,
                                   stream=None):
    """RMSNorm q [M,Kq] and kv [M,Kkv] (bf16, rows may be strided split views),
    quantize the normalized q per 1x128 group to E4M3FN.
    Returns (q_fp8 [M,Kq] float8_e4m3fn, q_scale [M,Kq/128] fp32, kv_out [M,Kkv] bf16)."""
    M, Kq = q.shape
    Kkv = kv.shape[1]
    dev = q.device
    lay = _layout(scale_layout)
    if q_out is None:
        q_out = torch.empty(M, Kq, dtype=torch.float8_e4m3fn, device=dev)
    if q_scale is None:
        q_scale = empty_scales(M, Kq // group, lay, dev)
    if kv_out is None:
        kv_out = torch.empty(M, Kkv, dtype=torch.bfloat16, device=dev)
    ld = scale_ld_for(q_scale, lay)
    check(lib().dsnq_fused_dual_rmsnorm_group_quant(
        M, Kq, Kkv, q.data_ptr(), _row_view_ok(q, "q"), kv.data_ptr(), _row_view_ok(kv, "kv"),
        gamma_q.data_ptr(), gamma_kv.data_ptr(), float(eps), group,
        q_out.data_ptr(), _row_view_ok(q_out, "q_out"), q_scale.data_ptr(), lay, ld,
        kv_out.data_ptr(), _row_view_ok(kv_out, "kv_out"), _stream(stream, q.device)),
        "dsnq_fused_dual_rmsnorm_group_quant")
    return q_out, q_scale, kv_out


def rmsnorm_group_quant(x, gamma, eps: float = 1e-6, group: int = GROUP, scale_layout=ROW_MAJOR,
                        x_out=None, x_scale=None, stream=None):
    """RMSNorm one latent x [M,K] (bf16, rows may be a strided view) and
    quantize it per 1x128 group to E4M3FN.  Returns (x_fp8, x_scale)."""
    M, K = x.shape
    lay = _layout(scale_layout)
    if x_out is None:
        x_out = torch.empty(M, K, dtype=torch.float8_e4m3fn, device=x.device)
    if x_scale is None:
        x_scale = empty_scales(M, K // group, lay, x.device)
    ld = scale_ld_for(x_scale, lay)
    check(lib().dsnq_rmsnorm_group_quant(
        M, K, x.data_ptr(), _row_view_ok(x, "x"), gamma.data_ptr(), float(eps), group,
        x_out.data_ptr(), _row_view_ok(x_out, "x_out"), x_scale.data_ptr(), lay, ld, _stream(stream, x.device)),
        "dsnq_rmsnorm_group_quant")
    return x_out, x_scale


def dual_rmsnorm_bf16(q, kv, gamma_q, gamma_kv, eps: float = 1e-6, q_out=None, kv_out=None, stream=None):
    """Unfused baseline step 1: both latents normalized to bf16."""
    M, Kq = q.shape
    Kkv = kv.shape[1]
    if q_out is None:
        q_out = torch.empty(M, Kq, dtype=torch.bfloat16, device=q.device)
    if kv_out is None:
        kv_out = torch.empty(M, Kkv, dtype=torch.bfloat16, device=q.device)
    check(lib().dsnq_dual_rmsnorm_bf16(
        M, Kq, Kkv, q.data_ptr(), _row_view_ok(q, "q"), kv.data_ptr(), _row_view_ok(kv, "kv"),
        gamma_q.data_ptr(), gamma_kv.data_ptr(), float(eps),
        q_out.data_ptr(), _row_view_ok(q_out, "q_out"), kv_out.data_ptr(), _row_view_ok(kv_out, "kv_out"),
        _stream(stream, q.device)), "dsnq_dual_rmsnorm_bf16")
    return q_out, kv_out


def group_quant_bf16(x, group: int = GROUP, scale_layout=ROW_MAJOR, x_out=None, x_scale=None, stream=None):
    """Unfused baseline step 2: per-1x128 quant of a bf16 [M,K] tensor."""
    M, K = x.shape
    lay = _layout(scale_layout)
    if x_out is None:
        x_out = torch.empty(M, K, dtype=torch.float8_e4m3fn, device=x.device)
    if x_scale is None:
        x_scale = empty_scales(M, K // group, lay, x.device)
    ld = scale_ld_for(x_scale, lay)
    check(lib().dsnq_group_quant_bf16(
        M, K, x.data_ptr(), _row_view_ok(x, "x"), group, x_out.data_ptr(), _row_view_ok(x_out, "x_out"),
        x_scale.data_ptr(), lay, ld, _stream(stream, x.device)), "dsnq_group_quant_bf16")
    return x_out, x_scale


def quantize_weight_block128(w, w_out=None, w_scale=None, stream=None):
    """fp32 weight [N,K] -> (E4M3FN codes [N,K], fp32 block scales [ceil(N/128), K/128])."""
    N, K = w.shape
    if w_out is None:
        w_out = torch.empty(N, K, dtype=torch.float8_e4m3fn, device=w.device)
    if w_scale is None:
        w_scale = torch.empty((N + 127) // 128, K // 128, dtype=torch.float32, device=w.device)
    check(lib().dsnq_quantize_weight_block128(
        N, K, w.data_ptr(), _row_view_ok(w, "w"), w_out.data_ptr(), _row_view_ok(w_out, "w_out"),
        w_scale.data_ptr(), _row_view_ok(w_scale, "w_scale"), _stream(stream, w.device)),
        "dsnq_quantize_weight_block128")
    return w_out, w_scale


def block_scaled_fp8_gemm(a_fp8, a_scale, w_fp8, w_scale, out=None, stream=None):
    """out[M,N] bf16 = block-scaled (a_fp8, a_scale) x (w_fp8, w_scale)^T."""
    M, K = a_fp8.shape
    N = w_fp8.shape[0]
    if out is None:
        out = torch.empty(M, N, dtype=torch.bfloat16, device=a_fp8.device)
    lay, ld = scale_layout_of(a_scale)
    check(lib().dsnq_block_scaled_fp8_gemm(
        M, N, K, a_fp8.data_ptr(), _row_view_ok(a_fp8, "a_fp8"), a_scale.data_ptr(), lay, ld,
        w_fp8.data_ptr(), _row_view_ok(w_fp8, "w_fp8"), w_scale.data_ptr(), _row_view_ok(w_scale, "w_scale"),
        out.data_ptr(), _row_view_ok(out, "out"), _stream(stream, a_fp8.device)), "dsnq_block_scaled_fp8_gemm")
    return out


def block_scaled_fp8_gemm_dual(a_fp8, a_scale, w1_fp8, w1_scale, w2_fp8, w2_scale,
                               out1=None, out2=None, stream=None):
    """Both consumers (e.g. attention wq_b and indexer wq_b) in one launch."""
    M, K = a_fp8.shape
    N1, N2 = w1_fp8.shape[0], w2_fp8.shape[0]
    dev = a_fp8.device
    if out1 is None:
        out1 = torch.empty(M, N1, dtype=torch.bfloat16, device=dev)
    if out2 is None:
        out2 = torch.empty(M, N2, dtype=torch.bfloat16, device=dev)
    lay, ld = scale_layout_of(a_scale)
    check(lib().dsnq_block_scaled_fp8_gemm_dual(
        M, K, a_fp8.data_ptr(), _row_view_ok(a_fp8, "a_fp8"), a_scale.data_ptr(), lay, ld,
        N1, w1_fp8.data_ptr(), _row_view_ok(w1_fp8, "w1_fp8"), w1_scale.data_ptr(),
        _row_view_ok(w1_scale, "w1_scale"), out1.data_ptr(), _row_view_ok(out1, "out1"),
        N2, w2_fp8.data_ptr(), _row_view_ok(w2_fp8, "w2_fp8"), w2_scale.data_ptr(),
        _row_view_ok(w2_scale, "w2_scale"), out2.data_ptr(), _row_view_ok(out2, "out2"),
        _stream(stream, a_fp8.device)), "dsnq_block_scaled_fp8_gemm_dual")
    return out1, out2


def bf16a_workspace_bytes(M: int, K: int):
    """(code_bytes, scale_bytes) of the workspace block_scaled_fp8_gemm_dual_bf16a
    needs for M rows of K bf16 activations; (0, 0) when it quantizes inside
    the GEMM (the library's own rule, dsnq_bf16a_workspace_bytes)."""
    c, s = C.c_int64(), C.c_int64()
    check(lib().dsnq_bf16a_workspace_bytes(M, K, C.byref(c), C.byref(s)), "dsnq_bf16a_workspace_bytes")
    return c.value, s.value


def fused_quant_fits(M: int, K: int) -> bool:
    """True when block_scaled_fp8_gemm_dual_bf16a quantizes inside the GEMM
    (one launch, no workspace)."""
    return M > 0 and bf16a_workspace_bytes(M, K) == (0, 0)


def gemm_plan(M: int, K: int):
    """(variant, dynamic shared memory bytes) of the GEMM kernel that
    block_scaled_fp8_gemm(_dual) launches for M rows and reduction length K
    (host-only query, dsnq_gemm_plan)."""
    v, b = C.c_int32(), C.c_int64()
    check(lib().dsnq_gemm_plan(M, K, C.byref(v), C.byref(b)), "dsnq_gemm_plan")
    return v.value, b.value


def block_scaled_fp8_gemm_dual_bf16a(a_bf16, w1_fp8, w1_scale, w2_fp8, w2_scale,
                                     out1=None, out2=None, workspace=None, stream=None):
    """The dual GEMM on bf16 activations, quantized per 1x128 on the fly.
    `workspace` = (a_fp8 [M,K] uint8/e4m3, a_scale [M*K/128] fp32) is only
    needed outside fused_quant_fits(M, K); it is allocated here if omitted."""
    M, K = a_bf16.shape
    N1, N2 = w1_fp8.shape[0], w2_fp8.shape[0]
    dev = a_bf16.device
    if out1 is None:
        out1 = torch.empty(M, N1, dtype=torch.bfloat16, device=dev)
    if out2 is None:
        out2 = torch.empty(M, N2, dtype=torch.bfloat16, device=dev)
    ws_a = ws_s = 0
    code_bytes, scale_bytes = bf16a_workspace_bytes(M, K)
    if code_bytes:
        if workspace is None:
            workspace = (torch.empty(code_bytes, dtype=torch.uint8, device=dev),
                         torch.empty(scale_bytes // 4, dtype=torch.float32, device=dev))
        ws_a, ws_s = workspace[0].data_ptr(), workspace[1].data_ptr()
    check(lib().dsnq_block_scaled_fp8_gemm_dual_bf16a(
        M, K, a_bf16.data_ptr(), _row_view_ok(a_bf16, "a_bf16"),
        N1, w1_fp8.data_ptr(), _row_view_ok(w1_fp8, "w1_fp8"), w1_scale.data_ptr(),
        _row_view_ok(w1_scale, "w1_scale"), out1.data_ptr(), _row_view_ok(out1, "out1"),
        N2, w2_fp8.data_ptr(), _row_view_ok(w2_fp8, "w2_fp8"), w2_scale.data_ptr(),
        _row_view_ok(w2_scale, "w2_scale"), out2.data_ptr(), _row_view_ok(out2, "out2"),
        ws_a, ws_s, _stream(stream, a_bf16.device)), "dsnq_block_scaled_fp8_gemm_dual_bf16a")
    return out1, out2


def block_scaled_fp8_gemm_dual_bf16a_static(a_bf16, w1_fp8, w1_scale, w2_fp8, w2_scale,
                                            out1=None, out2=None, stream=None):
    """block_scaled_fp8_gemm_dual_bf16a with the library's own device scratch
    (M, K <= 2048): nothing is allocated for the quantized pair."""
    M, K = a_bf16.shape
    N1, N2 = w1_fp8.shape[0], w2_fp8.shape[0]
    dev = a_bf16.device
    if out1 is None:
        out1 = torch.empty(M, N1, dtype=torch.bfloat16, device=dev)
    if out2 is None:
        out2 = torch.empty(M, N2, dtype=torch.bfloat16, device=dev)
    check(lib().dsnq_block_scaled_fp8_gemm_dual_bf16a_static(
        M, K, a_bf16.data_ptr(), _row_view_ok(a_bf16, "a_bf16"),
        N1, w1_fp8.data_ptr(), _row_view_ok(w1_fp8, "w1_fp8"), w1_scale.data_ptr(),
        _row_view_ok(w1_scale, "w1_scale"), out1.data_ptr(), _row_view_ok(out1, "out1"),
        N2, w2_fp8.data_ptr(), _row_view_ok(w2_fp8, "w2_fp8"), w2_scale.data_ptr(),
        _row_view_ok(w2_scale, "w2_scale"), out2.data_ptr(), _row_view_ok(out2, "out2"),
        _stream(stream, a_bf16.device)), "dsnq_block_scaled_fp8_gemm_dual_bf16a_static")
    return out1, out2


def fused_norm_quant_gemm_dual(q, kv, gamma_q, gamma_kv, eps, w1_fp8, w1_scale, w2_fp8, w2_scale,
                               out1=None, out2=None, kv_out=None, q_fp8=None, q_scale=None, stream=None):
    """RMSNorm + per-1x128 quant of the q latent (kv latent normalized to
    bf16), then the dual GEMM, in one call.  Returns (out1, out2, kv_out,
    q_fp8, q_scale); the last two are None when the rows were quantized
    inside the GEMM and no buffers were passed."""
    M, Kq = q.shape
    Kkv = kv.shape[1]
    N1, N2 = w1_fp8.shape[0], w2_fp8.shape[0]
    dev = q.device
    if out1 is None:
        out1 = torch.empty(M, N1, dtype=torch.bfloat16, device=dev)
    if out2 is None:
        out2 = torch.empty(M, N2, dtype=torch.bfloat16, device=dev)
    if kv_out is None:
        kv_out = torch.empty(M, Kkv, dtype=torch.bfloat16, device=dev)
    one_launch = fused_quant_fits(M, Kq) and Kkv <= 2048 and N1 + N2 > 0
    if not one_launch and M > 0:
        if q_fp8 is None:
            q_fp8 = torch.empty(M, Kq, dtype=torch.float8_e4m3fn, device=dev)
        if q_scale is None:
            q_scale = empty_scales(M, Kq // GROUP, COL_MAJOR, dev)
    if q_fp8 is not None and not q_fp8.is_contiguous():
        raise ValueError("q_fp8 must be contiguous [M, Kq]")
    if q_scale is not None and M > 1 and q_scale.stride() != (1, M):
        raise ValueError("q_scale must be column-major [M, Kq/128] (strides (1, M))")
    check(lib().dsnq_fused_norm_quant_gemm_dual(
        M, Kq, Kkv, q.data_ptr(), _row_view_ok(q, "q"), kv.data_ptr(), _row_view_ok(kv, "kv"),
        gamma_q.data_ptr(), gamma_kv.data_ptr(), float(eps), kv_out.data_ptr(), _row_view_ok(kv_out, "kv_out"),
        N1, w1_fp8.data_ptr(), _row_view_ok(w1_fp8, "w1_fp8"), w1_scale.data_ptr(),
        _row_view_ok(w1_scale, "w1_scale"), out1.data_ptr(), _row_view_ok(out1, "out1"),
        N2, w2_fp8.data_ptr(), _row_view_ok(w2_fp8, "w2_fp8"), w2_scale.data_ptr(),
        _row_view_ok(w2_scale, "w2_scale"), out2.data_ptr(), _row_view_ok(out2, "out2"),
        0 if q_fp8 is None else q_fp8.data_ptr(), 0 if q_scale is None else q_scale.data_ptr(),
        _stream(stream, q.device)), "dsnq_fused_norm_quant_gemm_dual")
    return out1, out2, kv_out, q_fp8, q_scale


_BF16, _F32, _F64, _I32, _I64 = torch.bfloat16, torch.float32, torch.float64, torch.int32, torch.int64


def _refuse(t, name: str, dtype, dim: int, dev, why: str):
    """Says what is wrong with a tensor argument."""
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.dim() != dim:
        raise ValueError(f"{name} must have {dim} dimensions, got {t.dim()}")
    if t.device != dev:
        raise ValueError(f"{name} is on {t.device}, expected {dev}")
    raise ValueError(f"{name} {why}, got shape {tuple(t.shape)}, strides {t.stride()}")


# One function per rank checks a tensor and gives what the library takes of
# it: small calls are bound by this host work.

def _vec(t, name: str, dtype, n: int, dev) -> int:
    """The address of a contiguous 1-D tensor of n elements."""
    if t.dtype is not dtype or t.dim() != 1 or t.numel() != n or not t.is_contiguous() or t.device != dev:
        _refuse(t, name, dtype, 1, dev, f"must be contiguous with {n} elements")
    return t.data_ptr()


def _mat(t, name: str, dtype, dev):
    """(rows, columns, row stride, address) of a 2-D tensor with contiguous
    rows (a lone row's stride is its length, whatever the view's is)."""
    if t.dtype is not dtype or t.dim() != 2 or t.device != dev:
        _refuse(t, name, dtype, 2, dev, "")
    n0, n1 = t.shape
    s0, s1 = t.stride()
    if s1 != 1 and n1 > 1:
        _refuse(t, name, dtype, 2, dev, "must have contiguous rows")
    return n0, n1, (s0 if n0 > 1 else n1), t.data_ptr()


def _cube(t, name: str, dtype, dev):
    """(three sizes, two outer strides, address) of a 3-D tensor with
    contiguous rows (a dimension of size 1 gets the stride it would have if
    packed)."""
    if t.dtype is not dtype or t.dim() != 3 or t.device != dev:
        _refuse(t, name, dtype, 3, dev, "")
    n0, n1, n2 = t.shape
    s0, s1, s2 = t.stride()
    if s2 != 1 and n2 > 1:
        _refuse(t, name, dtype, 3, dev, "must have contiguous rows")
    if n1 == 1:
        s1 = n2
    return n0, n1, n2, (n1 * s1 if n0 == 1 else s0), s1, t.data_ptr()


def _new(shape, dtype, dev, stream):
    """An uninitialized tensor for a call on `stream`, of that stream's
    memory: memory of another one may still be in use there."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=dev)
    with torch.cuda.stream(stream if hasattr(stream, "cuda_stream") else torch.cuda.ExternalStream(int(stream))):
        return torch.empty(shape, dtype=dtype, device=dev)


_kept = threading.local()


def _workspace(size: int, dev, stream, handle: int):
    """A uint8 tensor of at least `size` bytes for one call on the stream
    `handle`.  Calls of one thread on one stream run one after the other, so
    outside a capture the last such tensor serves again (an allocation took 5
    of a small call's 19 us on the host); on each device, the four streams
    that the thread used last keep theirs.  A capture gets a tensor of its
    graph's pool, a call with an explicit stream one of that stream."""
    if stream is not None or torch.cuda.is_current_stream_capturing():
        return _new(size, torch.uint8, dev, stream)
    kept = _kept.__dict__.setdefault(dev.index, {})          # in the order of their last use
    t = kept.pop(handle, None)
    if t is None or t.numel() < size:
        t = None
        while len(kept) >= 4:
            kept.pop(next(iter(kept)))
        t = torch.empty(size, dtype=torch.uint8, device=dev)
    kept[handle] = t
    return t


def release_workspaces() -> None:
    """Gives the workspaces that paged_latent_attention keeps for the calling
    thread (up to 42 MB for each of four streams of a device) back to torch's
    allocator.  Calls still running may go on using theirs: the memory goes to
    later work of the same stream only."""
    _kept.__dict__.clear()


def _rope_layout(layout) -> int:
    if layout == "interleaved" or layout == ROPE_INTERLEAVED:
        return ROPE_INTERLEAVED
    if layout == "half" or layout == ROPE_HALF:
        return ROPE_HALF
    raise ValueError(f"unknown rotary layout {layout!r}")


def rope_frequencies(rope_dim: int, base: float = 10000.0, factor: float = 1.0, original_length: int = 4096,
                     beta_fast: float = 32.0, beta_slow: float = 1.0, device="cuda"):
    """(inv_freq [rope_dim/2] float64, rope_scale) of head_rmsnorm_rope and
    latent_cache_write.  With factor > 1 (a context `factor` times
    original_length) the frequencies of fewer than beta_slow turns over the
    original length are divided by it, those of more than beta_fast kept, the
    ones between blended (the YaRN scheme), and rope_scale is its attention
    factor 0.1 ln(factor) + 1.  Any other table serves as well.  Those two take
    rope_dim = 2 * len(inv_freq) of multiples of 16 up to 256."""
    if rope_dim <= 0 or rope_dim % 2:
        raise ValueError(f"rope_dim must be even and positive, got {rope_dim}")
    i = torch.arange(0, rope_dim, 2, dtype=torch.float64)
    freq = torch.pow(torch.tensor(float(base), dtype=torch.float64), -i / rope_dim)
    if factor <= 1.0:
        return freq.to(device), 1.0

    def pair_of(turns):                  # the (fractional) pair that makes so many turns
        return rope_dim * math.log(original_length / (turns * 2 * math.pi)) / (2 * math.log(base))

    low = max(math.floor(pair_of(beta_fast)), 0)
    high = min(math.ceil(pair_of(beta_slow)), rope_dim - 1)
    ramp = ((i / 2 - low) / max(high - low, 1e-3)).clamp(0, 1)
    return (freq / factor * ramp + freq * (1 - ramp)).to(device), 0.1 * math.log(factor) + 1.0


def extend_block_tables(seq_lens, new_tokens, free_pages, block_table, page_size: int, rows: int, out=None, stream=None):
    """Gives each request (int32 lengths seq_lens [B]) new_tokens [B] more
    tokens (None: one each): takes the pages they need from free_pages in
    order, enters them in block_table [B, width] (in place; only new entries
    are written) and lays the tokens out as `rows` rows of the step.
    Returns (new_lens [B] int32, row_starts [B+1] int32, positions [rows]
    int64, slots [rows] int64, counts [2] int32 = pages taken and wanted);
    `out` supplies those five.  Padded rows and tokens without a place have
    slot -1."""
    B, dev = seq_lens.shape[0], seq_lens.device
    tb, width, ld, table = _mat(block_table, "block_table", _I32, dev)
    if tb != B:
        raise ValueError(f"block_table has {tb} rows for {B} requests")
    if out is None:
        out = (_new(B, _I32, dev, stream), _new(B + 1, _I32, dev, stream), _new(rows, _I64, dev, stream),
               _new(rows, _I64, dev, stream), _new(2, _I32, dev, stream))
    new_lens, row_starts, positions, slots, counts = out
    F = free_pages.shape[0]
    check(lib().dsnq_extend_block_tables(
        B, rows, page_size, _vec(seq_lens, "seq_lens", _I32, B, dev),
        None if new_tokens is None else _vec(new_tokens, "new_tokens", _I32, B, dev),
        _vec(free_pages, "free_pages", _I32, F, dev), F, table, width, ld,
        _vec(new_lens, "new_lens", _I32, B, dev), _vec(row_starts, "row_starts", _I32, B + 1, dev),
        _vec(positions, "positions", _I64, rows, dev), _vec(slots, "slots", _I64, rows, dev),
        _vec(counts, "counts", _I32, 2, dev), _stream(stream, dev)), "dsnq_extend_block_tables")
    return new_lens, row_starts, positions, slots, counts


def head_rmsnorm_rope(x, positions, inv_freq, gamma=None, eps: float = 1e-6, normalize: bool = True, rope_offset=None,
                      layout="interleaved", rope_scale: float = 1.0, inverse: bool = False, out=None, stream=None):
    """RMSNorm of each head of x [M,H,D] (bf16; token and head strides are
    free multiples of 8, at least D) and rotation of its columns [rope_offset,
    rope_offset + 2 * len(inv_freq)) (default: the last ones; an offset that is
    a multiple of 8, a width that is one of 16, up to 256) by positions [M]
    int64 times inv_freq float64, one rounding.  `out` may be x.  Returns out
    [M,H,D]."""
    dev = x.device
    M, H, D, xt, xh, xp = _cube(x, "x", _BF16, dev)
    if out is None:
        out = _new((M, H, D), _BF16, dev, stream)
    oM, oH, oD, ot, oh, op = _cube(out, "out", _BF16, dev)
    if oM != M or oH != H or oD != D:
        raise ValueError(f"out has shape {tuple(out.shape)}, expected {(M, H, D)}")
    pairs = inv_freq.shape[0]
    check(lib().dsnq_head_rmsnorm_rope(
        M, H, D, xp, xt, xh, 1 if normalize else 0, None if gamma is None else _vec(gamma, "gamma", _BF16, D, dev), float(eps),
        _vec(positions, "positions", _I64, M, dev), _vec(inv_freq, "inv_freq", _F64, pairs, dev),
        D - 2 * pairs if rope_offset is None else rope_offset, 2 * pairs, _rope_layout(layout), float(rope_scale),
        1 if inverse else 0, op, ot, oh, _stream(stream, dev)), "dsnq_head_rmsnorm_rope")
    return out


def latent_cache_write(kv, pe, positions, slots, inv_freq, cache, gamma=None, eps: float = 1e-6, normalize: bool = False,
                       rope_offset=None, layout="interleaved", rope_scale: float = 1.0, stream=None):
    """Stores row m = [kv[m] | pe[m]] (bf16; pe [M,P] or None) at slots[m] of
    the paged cache [pages, page_size, K+P], kv RMSNormed first when
    `normalize`, columns [rope_offset, + 2 * len(inv_freq)) of the row
    (default: the last ones; multiples of 8 and 16 as above) rotated.
    Negative slots are skipped; the slots of a call must be distinct.  Returns
    cache."""
    dev = kv.device
    M, K, ldkv, kvp = _mat(kv, "kv", _BF16, dev)
    P = ldpe = 0
    pep = None
    if pe is not None:
        rows, P, ldpe, pep = _mat(pe, "pe", _BF16, dev)
        if rows != M:
            raise ValueError(f"pe has {rows} rows, kv {M}")
    pages, page_size, W, ld_page, ld_row, cp = _cube(cache, "cache", _BF16, dev)
    if W != K + P:
        raise ValueError(f"cache rows have {W} columns, kv and pe {K + P}")
    pairs = inv_freq.shape[0]
    check(lib().dsnq_latent_cache_write(
        M, K, P, kvp, ldkv, pep, ldpe, 1 if normalize else 0, None if gamma is None else _vec(gamma, "gamma", _BF16, K, dev),
        float(eps), _vec(positions, "positions", _I64, M, dev), _vec(inv_freq, "inv_freq", _F64, pairs, dev),
        W - 2 * pairs if rope_offset is None else rope_offset, 2 * pairs, _rope_layout(layout), float(rope_scale),
        _vec(slots, "slots", _I64, M, dev), cp, pages, page_size, ld_page, ld_row, _stream(stream, dev)),
        "dsnq_latent_cache_write")
    return cache


@functools.lru_cache(maxsize=256)
def paged_latent_attention_workspace_bytes(B: int, H: int, v_dim: int, table_width: int, page_size: int) -> int:
    """Bytes of paged_latent_attention's workspace (host-only query)."""
    n = C.c_int64()
    check(lib().dsnq_paged_latent_attention_workspace_bytes(B, H, v_dim, table_width, page_size, C.byref(n)),
          "dsnq_paged_latent_attention_workspace_bytes")
    return n.value


def paged_latent_attention(q, cache, block_table, seq_lens, v_dim: int, scale: float, out=None, lse=None, workspace=None,
                           stream=None):
    """Attention of q [B,H,DK] (bf16, one new token per request) over the
    first seq_lens[b] (int32) tokens of each request in the paged cache
    [pages, page_size, DK], whose pages block_table [B, width] (int32) names.
    The value of a row is its first v_dim columns.  Returns (out [B,H,v_dim]
    bf16, lse [B,H] fp32).  The uint8 `workspace` is the binding's own if
    omitted: one per thread and stream, kept until release_workspaces(), and
    one of its own in a capture (with streams that are destroyed while work is
    pending, pass one)."""
    dev = q.device
    B, H, DK, qt, qh, qp = _cube(q, "q", _BF16, dev)
    pages, page_size, W, ld_page, ld_row, cp = _cube(cache, "cache", _BF16, dev)
    if W != DK:
        raise ValueError(f"cache rows have {W} columns, q {DK}")
    tb, width, ldt, table = _mat(block_table, "block_table", _I32, dev)
    if tb != B:
        raise ValueError(f"block_table has {tb} rows for {B} requests")
    if out is None:
        out = _new((B, H, v_dim), _BF16, dev, stream)
    oB, oH, oD, ot, oh, op = _cube(out, "out", _BF16, dev)
    if oB != B or oH != H or oD != v_dim:
        raise ValueError(f"out has shape {tuple(out.shape)}, expected {(B, H, v_dim)}")
    if lse is None:
        lse = _new((B, H), _F32, dev, stream)
    lB, lH, ldl, lp = _mat(lse, "lse", _F32, dev)
    if lB != B or lH != H:
        raise ValueError(f"lse has shape {tuple(lse.shape)}, expected {(B, H)}")
    handle = _stream(stream, dev)
    if workspace is None:
        workspace = _workspace(paged_latent_attention_workspace_bytes(B, H, v_dim, width, page_size), dev, stream, handle)
    size = workspace.numel()
    check(lib().dsnq_paged_latent_attention(
        B, H, DK, v_dim, qp, qt, qh, cp, pages, page_size, ld_page, ld_row, table, width, ldt,
        _vec(seq_lens, "seq_lens", _I32, B, dev), float(scale), op, ot, oh, lp, ldl,
        _vec(workspace, "workspace", torch.uint8, size, dev), size, handle), "dsnq_paged_latent_attention")
    return out, lse


def debug_status(stream=None) -> int:
    """Synchronizes the stream and returns (and clears) the device status."""
    return lib().dsnq_debug_status(_stream(stream, torch.device("cuda", torch.cuda.current_device())))


def debug_set(inject_flags: int = 0, wait_timeout_ns: int = 0) -> None:
    lib().dsnq_debug_set(inject_flags, wait_timeout_ns)


def set_launch_overlap(enable: bool = True) -> None:
    """Programmatic dependent launch for every later call (on by default):
    a kernel may be scheduled while the previous kernel of its stream runs,
    and waits in hardware for that kernel's writes before reading inputs."""
    lib().dsnq_set_launch_overlap(1 if enable else 0)
