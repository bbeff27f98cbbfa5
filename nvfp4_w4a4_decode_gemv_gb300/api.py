"""Python face of the C ABI: the same names as include/nvfp4.h, taking torch
CUDA tensors.  Argument marshalling only -- allocation of outputs and
workspaces with torch, then one call into libnvfp4_gb300.so on the current
stream.  Every computation runs in the library's CUDA kernels.
"""
import ctypes
import weakref

import torch

from ._lib import (DTYPES, MOE_SCORES, ROPE_STYLES, THRESHOLD_FIXED, THRESHOLD_RESET, THRESHOLD_WINDOW, KVCacheDesc,
                   MoERouter, ResetParams, check, lib, ptr, stream_handle)

__all__ = [
    "nvfp4_quantize_act", "nvfp4_quantize_f32", "nvfp4_silu_mul_quantize", "nvfp4_gemv_smallm",
    "nvfp4_gemv_smallm_cudacore", "DEVERR_FLAG_TIMEOUT", "nvfp4_gemm_packed", "nvfp4_gemm_workspace_bytes",
    "nvfp4_gemv_workspace_bytes", "nvfp4_packed_weight_bytes", "nvfp4_pack_weights", "nvfp4_gemv_smallm_packed",
    "NVFP4PackedWeight", "nvfp4_quantize_gemv_packed", "nvfp4_quantize_gemv_workspace_bytes",
    "nvfp4_quantize_gemv_launches", "nvfp4_bf16_gemv", "nvfp4_bf16_gemv_tc", "nvfp4_bf16_gemv_workspace_bytes",
    "nvfp4_rms_norm_bf16", "nvfp4_rms_norm_quantize", "nvfp4_f32_to_bf16",
    "reset_state_bytes",
    "reset_state_init", "reset_workspace_bytes", "reset_sample", "reset_sample_noalloc", "device_status", "GemvWorkspace",
    "NVFP4Tensor", "ResetSampler",
    "NVFP4KVCache", "KVPlan", "nvfp4_kv_page_bytes", "nvfp4_kv_release", "nvfp4_kv_plan", "nvfp4_kv_append",
    "nvfp4_kv_read", "nvfp4_kv_attention", "nvfp4_kv_attention_workspace_bytes", "nvfp4_process_logits",
    "DEVERR_KV_RANGE", "DEVERR_NO_TOKEN",
    "rope_table", "nvfp4_kv_append_rope",
    "MoERouting", "NVFP4MoEWeight", "nvfp4_moe_route", "nvfp4_moe_plan", "nvfp4_moe_packed_weight_bytes",
    "nvfp4_moe_pack_weights", "nvfp4_moe_gate_up", "nvfp4_moe_gate_up_workspace_bytes", "nvfp4_moe_down",
    "nvfp4_moe_down_workspace_bytes", "DEVERR_NO_EXPERT", "DEVERR_MOE_RANGE",
]


class NVFP4Tensor:
    """codes uint8 [rows, K/2], scales uint8 [rows, K/16], global float32 [1] (all on the device)."""

    def __init__(self, codes, scales, global_scale):
        self.codes, self.scales, self.global_scale = codes, scales, global_scale

    @classmethod
    def empty(cls, rows: int, K: int, device="cuda"):
        return cls(torch.empty((rows, K // 2), dtype=torch.uint8, device=device),
                   torch.empty((rows, K // 16), dtype=torch.uint8, device=device),
                   torch.empty((1,), dtype=torch.float32, device=device))

    @property
    def rows(self):
        return self.codes.shape[0]

    @property
    def K(self):
        return self.codes.shape[1] * 2


def _need_cuda(*ts):
    for t in ts:
        if t is not None and (not t.is_cuda or not t.is_contiguous()):
            raise ValueError("expected contiguous CUDA tensors")


def nvfp4_quantize_act(x_bf16: torch.Tensor, out: NVFP4Tensor | None = None, stream=None) -> NVFP4Tensor:
    """BF16 [rows, K] -> NVFP4 (codes, scales, global)."""
    _need_cuda(x_bf16)
    if x_bf16.dtype != torch.bfloat16 or x_bf16.dim() != 2:
        raise ValueError("x must be a 2-D bfloat16 tensor")
    rows, K = x_bf16.shape
    out = out or NVFP4Tensor.empty(rows, K, x_bf16.device)
    check(lib().nvfp4_quantize_act(ptr(x_bf16), rows, K, ptr(out.codes), ptr(out.scales), ptr(out.global_scale),
                                   stream_handle(stream)), "nvfp4_quantize_act")
    return out


def nvfp4_quantize_f32(x: torch.Tensor, K: int | None = None, out: NVFP4Tensor | None = None,
                       stream=None) -> NVFP4Tensor:
    """FP32 rows (first K columns of a row-major [rows, ld] tensor) -> BF16 (RNE) -> NVFP4."""
    _need_cuda(x)
    if x.dtype != torch.float32 or x.dim() != 2:
        raise ValueError("x must be a 2-D float32 tensor")
    rows, ld = x.shape
    K = ld if K is None else K
    out = out or NVFP4Tensor.empty(rows, K, x.device)
    check(lib().nvfp4_quantize_f32(ptr(x), rows, K, ld, ptr(out.codes), ptr(out.scales), ptr(out.global_scale),
                                   stream_handle(stream)), "nvfp4_quantize_f32")
    return out


def nvfp4_silu_mul_quantize(gate_up: torch.Tensor, out: NVFP4Tensor | None = None, stream=None) -> NVFP4Tensor:
    """FP32 [rows, 2I] -> BF16(SiLU(gate) * up) -> NVFP4 [rows, I]."""
    _need_cuda(gate_up)
    rows, two_i = gate_up.shape
    inter = two_i // 2
    out = out or NVFP4Tensor.empty(rows, inter, gate_up.device)
    check(lib().nvfp4_silu_mul_quantize(ptr(gate_up), rows, inter, ptr(out.codes), ptr(out.scales),
                                        ptr(out.global_scale), stream_handle(stream)), "nvfp4_silu_mul_quantize")
    return out


def nvfp4_gemv_workspace_bytes(M: int, N: int, K: int) -> int:
    return int(lib().nvfp4_gemv_workspace_bytes(M, N, K))


# Device error bit of a GEMV CTA whose wait for another CTA's partial sum gave up
# (nvfp4_device_status); the GEMV workspaces must be zeroed again after it.
DEVERR_FLAG_TIMEOUT = 4

_live_workspaces = weakref.WeakSet()


class GemvWorkspace:
    """A zero-initialised GEMV workspace that grows on demand (re-zeroed when it
    grows, and by device_status() after a GEMV wait gave up)."""

    def __init__(self, device="cuda"):
        self.device = device
        self.buf = torch.zeros(0, dtype=torch.uint8, device=device)
        _live_workspaces.add(self)

    def get(self, M, N, K) -> torch.Tensor:
        need = nvfp4_gemv_workspace_bytes(M, N, K)
        if need == 0:
            raise ValueError(f"unsupported GEMV shape M={M} N={N} K={K}")
        return self.get_bytes(need)

    def get_bytes(self, need: int) -> torch.Tensor:
        if self.buf.numel() < need:
            self.buf = torch.zeros(need + 4096, dtype=torch.uint8, device=self.device)
        return self.buf

    def rezero(self) -> None:
        self.buf.zero_()


_default_ws: dict = {}


def _ws_for(device) -> GemvWorkspace:
    key = torch.device(device).index if torch.device(device).index is not None else torch.cuda.current_device()
    if key not in _default_ws:
        _default_ws[key] = GemvWorkspace(device)
    return _default_ws[key]


def nvfp4_gemv_smallm(x: NVFP4Tensor, w: NVFP4Tensor, y: torch.Tensor | None = None,
                      workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Y[M, N] = dequant(x) @ dequant(w)^T in FP32."""
    M, N, K = x.rows, w.rows, x.K
    if w.K != K:
        raise ValueError("x and w disagree on K")
    y = y if y is not None else torch.empty((M, N), dtype=torch.float32, device=x.codes.device)
    ws = workspace if workspace is not None else _ws_for(x.codes.device).get(M, N, K)
    check(lib().nvfp4_gemv_smallm(ptr(x.codes), ptr(x.scales), ptr(x.global_scale), M, ptr(w.codes), ptr(w.scales),
                                  ptr(w.global_scale), N, K, ptr(y), ptr(ws), ws.numel(), stream_handle(stream)),
          "nvfp4_gemv_smallm")
    return y


def nvfp4_gemv_smallm_cudacore(x: NVFP4Tensor, w: NVFP4Tensor, y: torch.Tensor | None = None,
                               workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """nvfp4_gemv_smallm on the library's second, CUDA-core kernel (a cross-check, not the fast path)."""
    M, N, K = x.rows, w.rows, x.K
    if w.K != K:
        raise ValueError("x and w disagree on K")
    y = y if y is not None else torch.empty((M, N), dtype=torch.float32, device=x.codes.device)
    ws = workspace if workspace is not None else _ws_for(x.codes.device).get(M, N, K)
    check(lib().nvfp4_gemv_smallm_cudacore(ptr(x.codes), ptr(x.scales), ptr(x.global_scale), M, ptr(w.codes),
                                           ptr(w.scales), ptr(w.global_scale), N, K, ptr(y), ptr(ws), ws.numel(),
                                           stream_handle(stream)), "nvfp4_gemv_smallm_cudacore")
    return y


class NVFP4PackedWeight:
    """An NVFP4 weight [N, K] in the packed layout of nvfp4_pack_weights: packed uint8 [bytes], global float32 [1]."""

    def __init__(self, packed, global_scale, N: int, K: int):
        self.packed, self.global_scale, self.N, self.K = packed, global_scale, N, K


def nvfp4_packed_weight_bytes(N: int, K: int) -> int:
    return int(lib().nvfp4_packed_weight_bytes(N, K))


def nvfp4_pack_weights(w: NVFP4Tensor, out: torch.Tensor | None = None, stream=None) -> NVFP4PackedWeight:
    """Row-major NVFP4 weight -> packed layout (same bytes, tile-chunk blocks of 18432 B)."""
    N, K = w.rows, w.K
    need = nvfp4_packed_weight_bytes(N, K)
    if need == 0:
        raise ValueError(f"unsupported weight shape N={N} K={K}")
    out = out if out is not None else torch.empty(need, dtype=torch.uint8, device=w.codes.device)
    check(lib().nvfp4_pack_weights(ptr(w.codes), ptr(w.scales), N, K, ptr(out), out.numel(), stream_handle(stream)),
          "nvfp4_pack_weights")
    return NVFP4PackedWeight(out, w.global_scale, N, K)


def nvfp4_gemv_smallm_packed(x: NVFP4Tensor, w: NVFP4PackedWeight, y: torch.Tensor | None = None,
                             workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """nvfp4_gemv_smallm with the weight packed."""
    M, N, K = x.rows, w.N, x.K
    if w.K != K:
        raise ValueError("x and w disagree on K")
    y = y if y is not None else torch.empty((M, N), dtype=torch.float32, device=x.codes.device)
    ws = workspace if workspace is not None else _ws_for(x.codes.device).get(M, N, K)
    check(lib().nvfp4_gemv_smallm_packed(ptr(x.codes), ptr(x.scales), ptr(x.global_scale), M, ptr(w.packed),
                                         ptr(w.global_scale), N, K, ptr(y), ptr(ws), ws.numel(),
                                         stream_handle(stream)), "nvfp4_gemv_smallm_packed")
    return y


def nvfp4_quantize_gemv_workspace_bytes(M: int, N: int, K: int) -> int:
    return int(lib().nvfp4_quantize_gemv_workspace_bytes(M, N, K))


def nvfp4_quantize_gemv_launches(M: int, N: int, K: int) -> int:
    """1 or 2: how nvfp4_quantize_gemv_packed runs the shape; 0 invalid shape, -1 no device."""
    return int(lib().nvfp4_quantize_gemv_launches(M, N, K))


def nvfp4_quantize_gemv_packed(x_bf16: torch.Tensor, w: NVFP4PackedWeight, y: torch.Tensor | None = None,
                               xg_out: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                               stream=None) -> torch.Tensor:
    """nvfp4_quantize_act(x_bf16) then nvfp4_gemv_smallm_packed, as one call (one launch where it fits)."""
    _need_cuda(x_bf16, y, xg_out)
    if x_bf16.dtype != torch.bfloat16 or x_bf16.dim() != 2:
        raise ValueError("x_bf16 must be a 2-D bfloat16 tensor")
    M, K = x_bf16.shape
    N = w.N
    if w.K != K:
        raise ValueError("x and w disagree on K")
    y = y if y is not None else torch.empty((M, N), dtype=torch.float32, device=x_bf16.device)
    if workspace is None:
        need = nvfp4_quantize_gemv_workspace_bytes(M, N, K)
        if need == 0:
            raise ValueError(f"unsupported shape M={M} N={N} K={K}")
        workspace = _ws_for(x_bf16.device).get_bytes(need)
    check(lib().nvfp4_quantize_gemv_packed(ptr(x_bf16), M, ptr(w.packed), ptr(w.global_scale), N, K, ptr(y),
                                           ptr(xg_out), ptr(workspace),
                                           workspace.numel(), stream_handle(stream)), "nvfp4_quantize_gemv_packed")
    return y


def nvfp4_gemm_workspace_bytes(M: int, N: int, K: int) -> int:
    return int(lib().nvfp4_gemm_workspace_bytes(M, N, K))


_gemm_ws: dict = {}


def nvfp4_gemm_packed(x: NVFP4Tensor, w: NVFP4PackedWeight, y: torch.Tensor | None = None,
                      workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Y[M, N] = dequant(x) @ dequant(w)^T for a prefill-sized batch (M <= 128) on packed weights."""
    M, N, K = x.rows, w.N, x.K
    if w.K != K:
        raise ValueError("x and w disagree on K")
    y = y if y is not None else torch.empty((M, N), dtype=torch.float32, device=x.codes.device)
    if workspace is None:
        dev = x.codes.device
        key = dev.index if dev.index is not None else torch.cuda.current_device()
        need = nvfp4_gemm_workspace_bytes(M, N, K)
        if need == 0:
            raise ValueError(f"unsupported GEMM shape M={M} N={N} K={K}")
        if key not in _gemm_ws or _gemm_ws[key].numel() < need:
            _gemm_ws[key] = torch.zeros(need, dtype=torch.uint8, device=dev)
        workspace = _gemm_ws[key]
    check(lib().nvfp4_gemm_packed(ptr(x.codes), ptr(x.scales), ptr(x.global_scale), M, ptr(w.packed),
                                  ptr(w.global_scale), N, K, ptr(y), ptr(workspace), workspace.numel(),
                                  stream_handle(stream)), "nvfp4_gemm_packed")
    return y


def nvfp4_bf16_gemv(x: torch.Tensor, w: torch.Tensor, y: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """y[M, N] = x[M, K] @ w[N, K]^T for BF16 x, w; FP32 result."""
    _need_cuda(x, w)
    M, K = x.shape
    N = w.shape[0]
    y = y if y is not None else torch.empty((M, N), dtype=torch.float32, device=x.device)
    check(lib().nvfp4_bf16_gemv(ptr(x), M, ptr(w), N, K, ptr(y), stream_handle(stream)), "nvfp4_bf16_gemv")
    return y


def nvfp4_bf16_gemv_workspace_bytes(M: int, N: int, K: int) -> int:
    return int(lib().nvfp4_bf16_gemv_workspace_bytes(M, N, K))


def nvfp4_bf16_gemv_tc(x: torch.Tensor, w: torch.Tensor, y: torch.Tensor | None = None,
                       workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """y[M, N] = x[M, K] @ w[N, K]^T for BF16 x, w on the tensor cores; FP32 result.  `workspace`: a zeroed
    uint8 device tensor of at least nvfp4_bf16_gemv_workspace_bytes(M, N, K) bytes (a GEMV workspace serves)."""
    _need_cuda(x, w)
    M, K = x.shape
    N = w.shape[0]
    y = y if y is not None else torch.empty((M, N), dtype=torch.float32, device=x.device)
    if workspace is None:            # the per-device GEMV workspace (its records region is what this call uses)
        workspace = _ws_for(x.device).get(M, N, 256)
    check(lib().nvfp4_bf16_gemv_tc(ptr(x), M, ptr(w), N, K, ptr(y), ptr(workspace), workspace.numel(),
                                   stream_handle(stream)), "nvfp4_bf16_gemv_tc")
    return y


def nvfp4_rms_norm_bf16(x: torch.Tensor, K: int | None = None, eps: float = 1e-6, out: torch.Tensor | None = None,
                        stream=None) -> torch.Tensor:
    """FP32 rows (first K columns of a row-major [rows, ld] tensor) -> BF16 RMS-normalized [rows, K]."""
    _need_cuda(x)
    if x.dtype != torch.float32 or x.dim() != 2:
        raise ValueError("x must be a 2-D float32 tensor")
    rows, ld = x.shape
    K = ld if K is None else K
    out = out if out is not None else torch.empty((rows, K), dtype=torch.bfloat16, device=x.device)
    check(lib().nvfp4_rms_norm_bf16(ptr(x), rows, K, ld, float(eps), ptr(out), stream_handle(stream)),
          "nvfp4_rms_norm_bf16")
    return out


def nvfp4_rms_norm_quantize(x: torch.Tensor, K: int | None = None, eps: float = 1e-6, out: NVFP4Tensor | None = None,
                            r_out: torch.Tensor | None = None, stream=None) -> NVFP4Tensor:
    """FP32 rows (first K columns of a row-major [rows, ld] tensor) -> BF16 RMS-normalized -> NVFP4, one launch;
    the BF16 rows also go to r_out when it is given."""
    _need_cuda(x)
    if x.dtype != torch.float32 or x.dim() != 2:
        raise ValueError("x must be a 2-D float32 tensor")
    rows, ld = x.shape
    K = ld if K is None else K
    if r_out is not None and (r_out.dtype != torch.bfloat16 or tuple(r_out.shape) != (rows, K)
                              or not r_out.is_contiguous()):
        raise ValueError("r_out must be a contiguous [rows, K] bfloat16 tensor")
    out = out or NVFP4Tensor.empty(rows, K, x.device)
    check(lib().nvfp4_rms_norm_quantize(ptr(x), rows, K, ld, float(eps), ptr(out.codes), ptr(out.scales),
                                        ptr(out.global_scale), ptr(r_out), stream_handle(stream)),
          "nvfp4_rms_norm_quantize")
    return out


def nvfp4_f32_to_bf16(x: torch.Tensor, y: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    _need_cuda(x)
    y = y if y is not None else torch.empty(x.shape, dtype=torch.bfloat16, device=x.device)
    check(lib().nvfp4_f32_to_bf16(ptr(x), x.numel(), ptr(y), stream_handle(stream)), "nvfp4_f32_to_bf16")
    return y


# Device error bit of a KV cache kernel that met a slot, page, length or row range outside its cache or
# tables and skipped it (nvfp4_device_status).
DEVERR_KV_RANGE = 8
# Device error bit of a reset_sample row without a distribution (all -inf, a NaN, +inf): its token is -1.
DEVERR_NO_TOKEN = 16
# Bytes at the start of an nvfp4_kv_attention workspace that are zeroed before its first use.
ATTENTION_WS_ZEROED = 4096


def _need(t, dtype, name, dim=None):
    """A contiguous CUDA tensor of one type (and rank), or ValueError."""
    if t.dtype is not dtype or not t.is_cuda or not t.is_contiguous() or (dim is not None and t.dim() != dim):
        raise ValueError(f"{name} must be a contiguous CUDA tensor of {dtype}" + (f" with {dim} dimensions" if dim else ""))


def _need_all(dtype, dim, names, *ts):
    """_need of several tensors (None is left out); a name is looked up for the message only."""
    for i, t in enumerate(ts):
        if t is not None and (t.dtype is not dtype or t.dim() != dim or not t.is_cuda or not t.is_contiguous()):
            _need(t, dtype, names.split()[i], dim)


def _empty(shape, dtype, device, stream) -> torch.Tensor:
    """An output of a call on `stream` (None: the current one): that stream's memory, so that nothing else is at work
    in it, given back when the current stream, on which the caller holds it, has come so far, too."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    current = torch.cuda.current_stream(device)
    with torch.cuda.stream(stream):
        t = torch.empty(shape, dtype=dtype, device=device)
    t.record_stream(current)
    return t


def nvfp4_kv_page_bytes(page_size: int, kv_heads: int, head_dim: int) -> int:
    return int(lib().nvfp4_kv_page_bytes(page_size, kv_heads, head_dim))


class NVFP4KVCache:
    """A paged KV cache in NVFP4: pages uint8 [num_pages, kv_heads, page_size / 16, 18 * head_dim] (layout:
    nvfp4_kv_cache in nvfp4.h) and one FP32 global scale [1] each for K and V, all on the device."""

    def __init__(self, pages: torch.Tensor, k_global: torch.Tensor, v_global: torch.Tensor):
        _need(pages, torch.uint8, "pages", 4)
        _need(k_global, torch.float32, "k_global")
        _need(v_global, torch.float32, "v_global")
        self.pages, self.k_global, self.v_global = pages, k_global, v_global
        self.num_pages, self.kv_heads, groups, group_bytes = pages.shape
        self.page_size, self.head_dim = 16 * groups, group_bytes // 18
        if (k_global.numel() != 1 or v_global.numel() != 1 or group_bytes != 18 * self.head_dim
                or nvfp4_kv_page_bytes(self.page_size, self.kv_heads, self.head_dim) == 0):
            raise ValueError(f"unsupported cache shape {tuple(pages.shape)}")
        self.desc = KVCacheDesc(pages.data_ptr(), k_global.data_ptr(), v_global.data_ptr(), self.num_pages,
                                self.page_size, self.kv_heads, self.head_dim)
        self.desc_ptr = ctypes.addressof(self.desc)

    @classmethod
    def empty(cls, num_pages: int, page_size: int, kv_heads: int, head_dim: int, k_global: float = 1.0,
              v_global: float = 1.0, device="cuda"):
        if nvfp4_kv_page_bytes(page_size, kv_heads, head_dim) == 0:
            raise ValueError(f"unsupported cache shape: page_size {page_size}, kv_heads {kv_heads}, head_dim {head_dim}")
        return cls(torch.empty((num_pages, kv_heads, page_size // 16, 18 * head_dim), dtype=torch.uint8, device=device),
                   torch.tensor([k_global], dtype=torch.float32, device=device),
                   torch.tensor([v_global], dtype=torch.float32, device=device))


class KVPlan:
    """Outputs of nvfp4_kv_plan, int32 on the device: slots and positions [max_tokens] of the packed new tokens,
    cu_q [batch + 1], kv_lens [batch], free_count [1] (pages left), info [2] (requests refused, tokens planned)."""

    __slots__ = ("slots", "positions", "cu_q", "kv_lens", "free_count", "info")

    def __init__(self, slots, positions, cu_q, kv_lens, free_count, info):
        self.slots, self.positions, self.cu_q = slots, positions, cu_q
        self.kv_lens, self.free_count, self.info = kv_lens, free_count, info

    @classmethod
    def empty(cls, batch: int, max_tokens: int, device="cuda", free_count: torch.Tensor | None = None, stream=None):
        i32 = lambda n: _empty(n, torch.int32, device, stream)
        return cls(i32(max_tokens), i32(max_tokens), i32(batch + 1), i32(batch),
                   i32(1) if free_count is None else free_count, i32(2))


def nvfp4_kv_release(lens: torch.Tensor, ended: torch.Tensor, block_table: torch.Tensor, free_pages: torch.Tensor,
                     free_count: torch.Tensor, page_size: int, free_count_out: torch.Tensor | None = None,
                     stream=None) -> torch.Tensor:
    """Pushes the pages of the requests with ended[b] != 0 (lens[b] tokens each) onto the free stack; returns the
    new count (in place unless free_count_out is given)."""
    out = free_count if free_count_out is None else free_count_out
    i32 = torch.int32
    _need_all(i32, 1, "lens free_pages free_count free_count_out", lens, free_pages, free_count, out)
    _need(block_table, i32, "block_table", 2)
    _need(ended, torch.uint8, "ended", 1)
    batch, width = block_table.shape
    if lens.numel() != batch or ended.numel() != batch or free_count.numel() != 1 or out.numel() != 1:
        raise ValueError("lens and ended need one entry a row of block_table, the counts one entry")
    check(lib().nvfp4_kv_release(lens.data_ptr(), ended.data_ptr(), batch, page_size, block_table.data_ptr(), width,
                                 free_pages.data_ptr(), free_pages.numel(), free_count.data_ptr(), out.data_ptr(),
                                 stream_handle(stream)), "nvfp4_kv_release")
    return out


def nvfp4_kv_plan(ctx_lens: torch.Tensor, new_lens: torch.Tensor, block_table: torch.Tensor, free_pages: torch.Tensor,
                  free_count: torch.Tensor, page_size: int, max_tokens: int | None = None,
                  out: KVPlan | None = None, stream=None) -> KVPlan:
    """Takes pages for new_lens[b] tokens behind ctx_lens[b] (block_table updated in place) and maps every new token
    to its slot.  Without `out`, the outputs are new tensors for max_tokens tokens and free_count is updated in
    place; out.free_count may be free_count, out.kv_lens may be ctx_lens."""
    i32 = torch.int32
    _need(block_table, i32, "block_table", 2)
    _need_all(i32, 1, "ctx_lens new_lens free_pages free_count", ctx_lens, new_lens, free_pages, free_count)
    batch, width = block_table.shape
    if out is None:
        if max_tokens is None:
            raise ValueError("max_tokens is needed to allocate the outputs")
        out = KVPlan.empty(batch, max_tokens, ctx_lens.device, free_count, stream)
    _need_all(i32, 1, "slots positions cu_q kv_lens free_count info", out.slots, out.positions, out.cu_q, out.kv_lens,
              out.free_count, out.info)
    if (ctx_lens.numel() != batch or new_lens.numel() != batch or out.kv_lens.numel() != batch
            or out.cu_q.numel() != batch + 1 or out.positions.numel() != out.slots.numel()
            or free_count.numel() != 1 or out.free_count.numel() != 1 or out.info.numel() != 2):
        raise ValueError("the lengths and outputs do not fit a batch of the block_table's rows")
    check(lib().nvfp4_kv_plan(ctx_lens.data_ptr(), new_lens.data_ptr(), batch, page_size, block_table.data_ptr(), width,
                              free_pages.data_ptr(), free_pages.numel(), free_count.data_ptr(),
                              out.free_count.data_ptr(), out.kv_lens.data_ptr(), out.cu_q.data_ptr(),
                              out.slots.data_ptr(), out.positions.data_ptr(), out.slots.numel(), out.info.data_ptr(),
                              stream_handle(stream)), "nvfp4_kv_plan")
    return out


def _need_rows(t, name, heads, dim):
    """CUDA rows [tokens, heads, dim] with adjacent elements in a row: their NVFP4_DTYPE_* code."""
    code = DTYPES.get(t.dtype)
    if code is None or not t.is_cuda or t.dim() != 3 or t.shape[1] != heads or t.shape[2] != dim or t.stride(2) != 1:
        raise ValueError(f"{name} must be a CUDA tensor [tokens, {heads}, {dim}] of float32 or bfloat16 with adjacent "
                         "elements")
    return code


def nvfp4_kv_append(k: torch.Tensor, v: torch.Tensor, slots: torch.Tensor, cache: NVFP4KVCache, stream=None) -> None:
    """Quantizes rows k, v [tokens, kv_heads, head_dim] (any token and head strides) into the cache's slots (-1: skip)."""
    code = _need_rows(k, "k", cache.kv_heads, cache.head_dim)
    if _need_rows(v, "v", cache.kv_heads, cache.head_dim) != code or v.shape[0] != k.shape[0]:
        raise ValueError("k and v must have the same type and number of tokens")
    _need(slots, torch.int32, "slots", 1)
    tokens = k.shape[0]
    if slots.numel() != tokens:
        raise ValueError("slots needs one entry a token")
    ks, vs = k.stride(), v.stride()
    check(lib().nvfp4_kv_append(k.data_ptr(), v.data_ptr(), code, tokens, ks[0], ks[1], vs[0], vs[1], slots.data_ptr(),
                                cache.desc_ptr, stream_handle(stream)), "nvfp4_kv_append")


def rope_table(max_positions: int, rotated: int, base: float = 10000.0, scale: float = 1.0, device="cuda") -> torch.Tensor:
    """Cosines and sines of position * scale * base^(-2 m / rotated), m < rotated / 2, for nvfp4_kv_append_rope: float32
    [max_positions, rotated / 2, 2], computed in 64 bits."""
    f64 = dict(dtype=torch.float64, device=device)
    angle = (torch.arange(max_positions, **f64) * scale)[:, None] * base ** (torch.arange(rotated // 2, **f64) * (-2.0 / rotated))
    return torch.stack([angle.cos(), angle.sin()], -1).float()


def nvfp4_kv_append_rope(q: torch.Tensor | None, k: torch.Tensor, v: torch.Tensor, positions: torch.Tensor,
                         slots: torch.Tensor, cache: NVFP4KVCache, table: torch.Tensor, style: str = "halves",
                         q_out: torch.Tensor | None = None, stream=None) -> torch.Tensor | None:
    """Rows q [tokens, heads, head_dim] and k [tokens, kv_heads, head_dim] rotated by their positions (int32 [tokens]) with
    the cosines and sines of table (float32 [max_positions, rotated / 2, 2], rope_table); k and v go quantized into the
    cache's slots (-1: skip, q zero), q comes back in BF16 (None: k and v alone).  style: the rotated part's "halves" form
    the pairs, or neighbours do ("pairs")."""
    if style not in ROPE_STYLES:
        raise ValueError(f"style must be one of {sorted(ROPE_STYLES)}")
    dim, tokens = cache.head_dim, k.shape[0]
    code = _need_rows(k, "k", cache.kv_heads, dim)
    if _need_rows(v, "v", cache.kv_heads, dim) != code or v.shape[0] != tokens:
        raise ValueError("k and v must have the same type and number of tokens")
    _need_all(torch.int32, 1, "positions slots", positions, slots)
    _need(table, torch.float32, "table", 3)
    if positions.numel() != tokens or slots.numel() != tokens or table.shape[2] != 2:
        raise ValueError("positions and slots need one entry a token, table two numbers a pair")
    heads, qs = 0, (0, 0)
    if q is not None:
        heads, qs = q.shape[1] if q.dim() == 3 else 0, q.stride()
        if _need_rows(q, "q", heads, dim) != code or q.shape[0] != tokens:
            raise ValueError("q must have the type and number of tokens of k and v")
        if q_out is None:
            q_out = _empty((tokens, heads, dim), torch.bfloat16, q.device, stream)
        else:
            _need(q_out, torch.bfloat16, "q_out")
            if q_out.shape != q.shape:
                raise ValueError(f"q_out must have shape {tuple(q.shape)}")
    elif q_out is not None:
        raise ValueError("q_out goes with q")
    ks, vs = k.stride(), v.stride()
    check(lib().nvfp4_kv_append_rope(ptr(q), k.data_ptr(), v.data_ptr(), code, tokens, heads, qs[0], qs[1], ks[0], ks[1],
                                     vs[0], vs[1], positions.data_ptr(), table.data_ptr(), table.shape[0],
                                     2 * table.shape[1], ROPE_STYLES[style], slots.data_ptr(), cache.desc_ptr,
                                     ptr(q_out), stream_handle(stream)), "nvfp4_kv_append_rope")
    return q_out


def nvfp4_kv_read(cache: NVFP4KVCache, slots: torch.Tensor, k_out: torch.Tensor | None = None,
                  v_out: torch.Tensor | None = None, stream=None):
    """The cached rows of the slots as BF16 [tokens, kv_heads, head_dim] (k, v); zeros where a slot is -1."""
    _need(slots, torch.int32, "slots", 1)
    shape = (slots.numel(), cache.kv_heads, cache.head_dim)
    k_out = k_out if k_out is not None else _empty(shape, torch.bfloat16, slots.device, stream)
    v_out = v_out if v_out is not None else _empty(shape, torch.bfloat16, slots.device, stream)
    for t, n in ((k_out, "k_out"), (v_out, "v_out")):
        _need(t, torch.bfloat16, n)
        if t.shape != shape:
            raise ValueError(f"{n} must have shape {shape}")
    check(lib().nvfp4_kv_read(cache.desc_ptr, slots.data_ptr(), shape[0], k_out.data_ptr(), v_out.data_ptr(),
                              stream_handle(stream)), "nvfp4_kv_read")
    return k_out, v_out


def nvfp4_kv_attention_workspace_bytes(batch: int, tokens: int, heads: int, kv_heads: int, head_dim: int) -> int:
    return int(lib().nvfp4_kv_attention_workspace_bytes(batch, tokens, heads, kv_heads, head_dim))


_attention_ws: dict = {}


def _new_attention_workspace(need: int, device) -> torch.Tensor:
    ws = torch.empty(need, dtype=torch.uint8, device=device)
    ws[:ATTENTION_WS_ZEROED].zero_()
    return ws


def _attention_workspace(need: int, device, stream) -> torch.Tensor:
    """A workspace of the stream's own (calls on different streams may overlap), cleared on that stream.  A captured
    call gets one of its graph's memory, cleared by each replay."""
    if stream is not None:
        with torch.cuda.stream(stream):                  # its memory, its order, and whether it is being captured
            return _attention_workspace(need, device, None)
    if torch.cuda.is_current_stream_capturing():
        return _new_attention_workspace(need, device)
    key = (device, stream_handle())
    ws = _attention_ws.get(key)
    if ws is None or ws.numel() < need:
        ws = _attention_ws[key] = _new_attention_workspace(need, device)
    return ws


def nvfp4_kv_attention(q: torch.Tensor, cache: NVFP4KVCache, block_table: torch.Tensor, kv_lens: torch.Tensor,
                       cu_q: torch.Tensor | None = None, max_q: int | None = None, scale: float | None = None,
                       window: int = 0, out: torch.Tensor | None = None, lse: torch.Tensor | None = None,
                       workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """softmax(scale q K^T) V of packed query rows q [tokens, heads, head_dim] over the cache, causal from the
    bottom right (BF16).  kv_lens [batch]: keys of each request, its new tokens among them; cu_q [batch + 1]: first
    row of each request, None: one row each; max_q: most rows of a request; scale: 1 / sqrt(head_dim) by default;
    window: a row sees its last `window` keys only (0: all); lse [tokens, heads] FP32 receives log sum exp; workspace:
    uint8, its first ATTENTION_WS_ZEROED bytes zeroed once (the stream's own by default)."""
    if q.dim() != 3:
        raise ValueError("q must be [tokens, heads, head_dim]")
    tokens, heads = q.shape[0], q.shape[1]
    code = _need_rows(q, "q", heads, cache.head_dim)
    _need(block_table, torch.int32, "block_table", 2)
    _need(kv_lens, torch.int32, "kv_lens", 1)
    batch, width = block_table.shape
    if kv_lens.numel() != batch:
        raise ValueError("kv_lens needs one entry a row of block_table")
    if cu_q is not None:
        _need(cu_q, torch.int32, "cu_q", 1)
        if cu_q.numel() != batch + 1:
            raise ValueError("cu_q needs batch + 1 entries")
    shape = (tokens, heads, cache.head_dim)
    if out is None:
        out = _empty(shape, torch.bfloat16, q.device, stream)
    else:
        _need(out, torch.bfloat16, "out")
        if out.shape != shape:
            raise ValueError(f"out must have shape {shape}")
    if lse is not None:
        _need(lse, torch.float32, "lse", 2)
        if lse.shape != shape[:2]:
            raise ValueError(f"lse must have shape {shape[:2]}")
    if workspace is None:
        workspace = _attention_workspace(
            nvfp4_kv_attention_workspace_bytes(batch, tokens, heads, cache.kv_heads, cache.head_dim), q.device, stream)
    else:
        _need(workspace, torch.uint8, "workspace")
    qs = q.stride()
    if max_q is None:
        max_q = 1 if cu_q is None else max(1, tokens)
    check(lib().nvfp4_kv_attention(q.data_ptr(), code, tokens, qs[0], qs[1], heads, cache.desc_ptr,
                                   block_table.data_ptr(), width, kv_lens.data_ptr(), ptr(cu_q), batch, max_q,
                                   scale if scale is not None else cache.head_dim ** -0.5, window, out.data_ptr(),
                                   ptr(lse), workspace.data_ptr(), workspace.numel(), stream_handle(stream)),
          "nvfp4_kv_attention")
    return out


# Device error bit of a token whose router logits give no choice (a NaN; with softmax +inf, or -inf alone): its ids are -1.
DEVERR_NO_EXPERT = 32
# Device error bit of an expert kernel that met an expert, offset, pair or place outside its tables and skipped it.
DEVERR_MOE_RANGE = 64


class MoERouting:
    """Which experts take which tokens, on the device: ids int32 and weights float32 [tokens, top_k] (weights may be
    None), and the plan of the pairs (token t's j-th expert is pair t top_k + j): offsets int32 [experts + 1] (where an
    expert's pairs begin), pairs int32 [tokens * top_k] (the pair at each place, -1 behind the last) and places int32
    [tokens, top_k] (where each pair stands, -1: nowhere)."""

    __slots__ = ("ids", "weights", "offsets", "pairs", "places", "tokens", "top_k", "experts")

    def __init__(self, ids, weights, offsets, pairs, places):
        i32 = torch.int32
        _need_all(i32, 2, "ids places", ids, places)
        _need_all(i32, 1, "offsets pairs", offsets, pairs)
        _need_all(torch.float32, 2, "weights", weights)
        if (places.shape != ids.shape or pairs.numel() != ids.numel() or offsets.numel() < 2
                or (weights is not None and weights.shape != ids.shape)):
            raise ValueError("weights and places have the shape of ids [tokens, top_k], pairs its entries, offsets an "
                             "entry an expert and one more")
        self.ids, self.weights, self.offsets, self.pairs, self.places = ids, weights, offsets, pairs, places
        (self.tokens, self.top_k), self.experts = ids.shape, offsets.numel() - 1

    @classmethod
    def empty(cls, tokens: int, top_k: int, experts: int, device="cuda", stream=None):
        i32 = torch.int32
        return cls(_empty((tokens, top_k), i32, device, stream), _empty((tokens, top_k), torch.float32, device, stream),
                   _empty(experts + 1, i32, device, stream), _empty(tokens * top_k, i32, device, stream),
                   _empty((tokens, top_k), i32, device, stream))


def _scratch(need: int, device, stream) -> torch.Tensor | None:
    """Workspace of a call that keeps no state: memory of its stream, or none."""
    return _empty(need, torch.uint8, device, stream) if need else None


def nvfp4_moe_route(logits: torch.Tensor, top_k: int, score: str = "softmax", bias: torch.Tensor | None = None,
                    groups: int = 1, top_groups: int = 1, group_best: int = 1, renormalize: bool = True,
                    scale: float = 1.0, rows: torch.Tensor | None = None, out: MoERouting | None = None,
                    stream=None) -> MoERouting:
    """Router logits [tokens, experts] (float32 or bfloat16, adjacent elements in a row) -> the top_k experts of each
    token, their weights and the plan by expert.  score: "softmax" or "sigmoid"; bias [experts] float32: added to the
    scores for the choice alone; groups: only the top_groups groups of experts with the largest sums of their group_best
    (1 or 2) best values stay; renormalize: a token's weights sum to `scale`, else they are its scores times `scale`; rows
    (uint8 or bool [tokens]): tokens with 0 get no expert (ids -1)."""
    code = DTYPES.get(logits.dtype)
    if code is None or not logits.is_cuda or logits.dim() != 2 or (logits.shape[1] > 1 and logits.stride(1) != 1):
        raise ValueError("logits must be a CUDA tensor [tokens, experts] of float32 or bfloat16 with adjacent elements")
    tokens, experts = logits.shape
    if score not in MOE_SCORES:
        raise ValueError(f"score must be one of {sorted(MOE_SCORES)}")
    if bias is not None:
        _need(bias, torch.float32, "bias", 1)
        if bias.numel() != experts:
            raise ValueError("bias needs one entry an expert")
    if rows is not None:
        _need_row_mask(rows, tokens)
    if out is None:
        if experts < 1 or top_k < 1:
            raise ValueError("experts and top_k must be positive")
        out = MoERouting.empty(tokens, top_k, experts, logits.device, stream)
    elif out.tokens != tokens or out.top_k != top_k or out.experts != experts or out.weights is None:
        raise ValueError("out does not fit the tokens, experts and top_k")
    router = MoERouter(top_k, MOE_SCORES[score], groups, top_groups, group_best, renormalize, scale)
    ws = _scratch(int(lib().nvfp4_moe_route_workspace_bytes(tokens, experts)), logits.device, stream)
    check(lib().nvfp4_moe_route(logits.data_ptr(), code, tokens, experts, logits.stride(0) if tokens > 1 else experts,
                                ctypes.byref(router), ptr(bias), ptr(rows), out.ids.data_ptr(), out.weights.data_ptr(),
                                out.offsets.data_ptr(), out.pairs.data_ptr(), out.places.data_ptr(), ptr(ws),
                                ws.numel() if ws is not None else 0, stream_handle(stream)), "nvfp4_moe_route")
    return out


def nvfp4_moe_plan(ids: torch.Tensor, experts: int, weights: torch.Tensor | None = None, stream=None) -> MoERouting:
    """The plan of a choice made elsewhere: ids int32 [tokens, top_k] (-1: no expert), with its weights."""
    _need(ids, torch.int32, "ids", 2)
    if experts < 1:
        raise ValueError("experts must be positive")
    i32, dev = torch.int32, ids.device
    out = MoERouting(ids, weights, _empty(experts + 1, i32, dev, stream), _empty(ids.numel(), i32, dev, stream),
                     _empty(tuple(ids.shape), i32, dev, stream))
    ws = _scratch(int(lib().nvfp4_moe_route_workspace_bytes(out.tokens, experts)), dev, stream)
    check(lib().nvfp4_moe_plan(ids.data_ptr(), out.tokens, out.top_k, experts, out.offsets.data_ptr(),
                               out.pairs.data_ptr(), out.places.data_ptr(), ptr(ws), ws.numel() if ws is not None else 0,
                               stream_handle(stream)), "nvfp4_moe_plan")
    return out


def nvfp4_moe_packed_weight_bytes(experts: int, N: int, K: int, gated: bool) -> int:
    return int(lib().nvfp4_moe_packed_weight_bytes(experts, N, K, int(gated)))


class NVFP4MoEWeight:
    """The NVFP4 weights [experts, N, K] of all experts in the packed layout of nvfp4_moe_pack_weights: packed uint8
    [bytes], global_scale float32 [experts].  gated: gate and up in one, N = 2 * inter."""

    def __init__(self, packed, global_scale, experts: int, N: int, K: int, gated: bool):
        _need(packed, torch.uint8, "packed", 1)
        _need(global_scale, torch.float32, "global_scale", 1)
        need = nvfp4_moe_packed_weight_bytes(experts, N, K, gated)
        if need == 0 or packed.numel() < need or global_scale.numel() != experts:
            raise ValueError(f"unsupported expert weights: experts {experts}, N {N}, K {K}, {packed.numel()} bytes")
        self.packed, self.global_scale = packed, global_scale
        self.experts, self.N, self.K, self.gated = experts, N, K, bool(gated)


def nvfp4_moe_pack_weights(codes: torch.Tensor, scales: torch.Tensor, global_scale: torch.Tensor, gated: bool,
                           out: torch.Tensor | None = None, stream=None) -> NVFP4MoEWeight:
    """Row-major NVFP4 codes [experts, N, K/2], scales [experts, N, K/16] and global scales [experts] -> packed.  gated:
    rows [0, N/2) are the gate's, [N/2, N) the up's."""
    _need(codes, torch.uint8, "codes", 3)
    _need(scales, torch.uint8, "scales", 3)
    experts, N, half = codes.shape
    if scales.shape != (experts, N, half // 8) or half % 8:
        raise ValueError("codes and scales disagree on their shapes")
    need = nvfp4_moe_packed_weight_bytes(experts, N, 2 * half, gated)
    if need == 0:
        raise ValueError(f"unsupported expert weights: experts {experts}, N {N}, K {2 * half}, gated {bool(gated)}")
    if out is None:
        out = _empty(need, torch.uint8, codes.device, stream)
    w = NVFP4MoEWeight(out, global_scale, experts, N, 2 * half, gated)
    check(lib().nvfp4_moe_pack_weights(codes.data_ptr(), scales.data_ptr(), experts, N, 2 * half, int(gated),
                                       out.data_ptr(), out.numel(), stream_handle(stream)), "nvfp4_moe_pack_weights")
    return w


def _need_nvfp4(x: NVFP4Tensor, rows: int, K: int, name: str):
    for t in (x.codes, x.scales):
        _need(t, torch.uint8, name, 2)
    _need(x.global_scale, torch.float32, name)
    if x.codes.shape != (rows, K // 2) or x.scales.shape != (rows, K // 16) or x.global_scale.numel() != 1:
        raise ValueError(f"{name} must have {rows} rows of {K}")


def nvfp4_moe_gate_up_workspace_bytes(tokens: int, top_k: int, experts: int, K: int) -> int:
    return int(lib().nvfp4_moe_gate_up_workspace_bytes(tokens, top_k, experts, K))


def nvfp4_moe_down_workspace_bytes(tokens: int, top_k: int, experts: int, N: int, K: int) -> int:
    return int(lib().nvfp4_moe_down_workspace_bytes(tokens, top_k, experts, N, K))


def nvfp4_moe_gate_up(x: NVFP4Tensor, w: NVFP4MoEWeight, routing: MoERouting, out: torch.Tensor | None = None,
                      workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """BF16(SiLU(gate) * up) of the chosen experts on x [tokens, K]: rows by place [tokens * top_k, inter], zero behind
    the last pair.  `workspace`: a uint8 tensor of at least nvfp4_moe_gate_up_workspace_bytes bytes (the stream's memory
    by default)."""
    r = routing
    if not w.gated or r.experts != w.experts:
        raise ValueError("w must hold gate and up of the routing's experts")
    _need_nvfp4(x, r.tokens, w.K, "x")
    shape = (r.tokens * r.top_k, w.N // 2)
    if out is None:
        out = _empty(shape, torch.bfloat16, x.codes.device, stream)
    else:
        _need(out, torch.bfloat16, "out")
        if out.shape != shape:
            raise ValueError(f"out must have shape {shape}")
    if workspace is None:
        workspace = _scratch(nvfp4_moe_gate_up_workspace_bytes(r.tokens, r.top_k, w.experts, w.K), x.codes.device, stream)
    else:
        _need(workspace, torch.uint8, "workspace")
    check(lib().nvfp4_moe_gate_up(x.codes.data_ptr(), x.scales.data_ptr(), x.global_scale.data_ptr(), r.tokens, r.top_k,
                                  r.offsets.data_ptr(), r.pairs.data_ptr(), w.packed.data_ptr(),
                                  w.global_scale.data_ptr(), w.experts, w.N // 2, w.K, out.data_ptr(), ptr(workspace),
                                  workspace.numel() if workspace is not None else 0, stream_handle(stream)),
          "nvfp4_moe_gate_up")
    return out


def nvfp4_moe_down(h: NVFP4Tensor, w: NVFP4MoEWeight, routing: MoERouting, y: torch.Tensor | None = None,
                   workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Y[tokens, N] FP32 = sum over a token's experts of weight * dequant(h) @ dequant(w)^T, h [tokens * top_k, K] by
    place.  `workspace`: a uint8 tensor of at least nvfp4_moe_down_workspace_bytes bytes (the stream's memory by
    default)."""
    r = routing
    if w.gated or r.experts != w.experts or r.weights is None:
        raise ValueError("w must hold plain matrices of the routing's experts, and the routing weights")
    _need_nvfp4(h, r.tokens * r.top_k, w.K, "h")
    shape, dev = (r.tokens, w.N), h.codes.device
    if y is None:
        y = _empty(shape, torch.float32, dev, stream)
    else:
        _need(y, torch.float32, "y")
        if y.shape != shape:
            raise ValueError(f"y must have shape {shape}")
    if workspace is None:
        workspace = _scratch(nvfp4_moe_down_workspace_bytes(r.tokens, r.top_k, w.experts, w.N, w.K), dev, stream)
    else:
        _need(workspace, torch.uint8, "workspace")
    check(lib().nvfp4_moe_down(h.codes.data_ptr(), h.scales.data_ptr(), h.global_scale.data_ptr(), r.tokens, r.top_k,
                               r.offsets.data_ptr(), r.pairs.data_ptr(), r.places.data_ptr(), r.weights.data_ptr(),
                               w.packed.data_ptr(), w.global_scale.data_ptr(), w.experts, w.N, w.K, y.data_ptr(),
                               ptr(workspace), workspace.numel() if workspace is not None else 0, stream_handle(stream)),
          "nvfp4_moe_down")
    return y


def nvfp4_process_logits(logits: torch.Tensor, tokens: torch.Tensor | None = None, n_tokens: torch.Tensor | None = None,
                         n_prompt: torch.Tensor | None = None, repetition: torch.Tensor | None = None,
                         presence: torch.Tensor | None = None, frequency: torch.Tensor | None = None,
                         bias_ids: torch.Tensor | None = None, bias_values: torch.Tensor | None = None,
                         mask: torch.Tensor | None = None, mask_rows: torch.Tensor | None = None,
                         fill: float = float("-inf"), out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Penalties, biases and grammar masks on logits [rows, V] (float32 or bfloat16, adjacent elements in a row);
    FP32 result.  tokens [rows, history] int32 with n_tokens, n_prompt [rows] int32; repetition, presence, frequency
    [rows] float32; bias_ids [rows, n] int32 (-1: unused) with bias_values float32; mask [masks, ceil(V / 32)] int32,
    bit v % 32 of word v / 32 set where token v is allowed, mask_rows [rows] int32 (-1: no mask)."""
    code = DTYPES.get(logits.dtype)
    if code is None or not logits.is_cuda or logits.dim() != 2 or (logits.shape[1] > 1 and logits.stride(1) != 1):
        raise ValueError("logits must be a CUDA tensor [rows, V] of float32 or bfloat16 with adjacent elements")
    rows, V = logits.shape
    i32, f32 = torch.int32, torch.float32
    _need_all(i32, 1, "n_tokens n_prompt mask_rows", n_tokens, n_prompt, mask_rows)
    _need_all(f32, 1, "repetition presence frequency", repetition, presence, frequency)
    _need_all(i32, 2, "tokens bias_ids", tokens, bias_ids)
    _need_all(f32, 2, "bias_values", bias_values)
    for t in (tokens, n_tokens, n_prompt, repetition, presence, frequency, bias_ids, bias_values, mask_rows):
        if t is not None and t.shape[0] != rows:
            raise ValueError("tokens, biases and the rows' parameters need one entry a row of logits")
    if (tokens is None) != (n_tokens is None) or (bias_ids is None) != (bias_values is None):
        raise ValueError("tokens and n_tokens, bias_ids and bias_values go together")
    if bias_ids is not None and bias_ids.shape != bias_values.shape:
        raise ValueError("bias_ids and bias_values must have the same shape")
    if mask is not None:
        _need(mask, torch.int32, "mask", 2)
        if mask.shape[1] != (V + 31) // 32 or (mask_rows is None and mask.shape[0] < rows):
            raise ValueError("mask needs ceil(V / 32) words a row, and a row for each row of logits without mask_rows")
    if out is None:
        out = _empty((rows, V), torch.float32, logits.device, stream)
    else:
        _need(out, torch.float32, "out", 2)
        if out.shape != logits.shape:
            raise ValueError("out must have the shape of logits")
    check(lib().nvfp4_process_logits(
        logits.data_ptr(), code, rows, V, logits.stride(0) if rows > 1 else V, ptr(tokens),
        tokens.shape[1] if tokens is not None else 0, ptr(n_tokens), ptr(n_prompt), ptr(repetition), ptr(presence),
        ptr(frequency), ptr(bias_ids), ptr(bias_values), bias_ids.shape[1] if bias_ids is not None else 0, ptr(mask),
        mask.shape[0] if mask is not None else 0, ptr(mask_rows), fill, out.data_ptr(), stream_handle(stream)),
        "nvfp4_process_logits")
    return out


def reset_state_bytes(M: int, w: int) -> int:
    return int(lib().reset_state_bytes(M, w))


def reset_workspace_bytes(M: int, V: int) -> int:
    return int(lib().reset_workspace_bytes(M, V))


def reset_state_init(state: torch.Tensor, M: int, w: int, stream=None, rows: torch.Tensor | None = None) -> None:
    """Every row at sequence position 0; with `rows` (uint8 or bool [M]) those rows alone."""
    if rows is None:
        check(lib().reset_state_init(ptr(state), M, w, stream_handle(stream)), "reset_state_init")
    else:
        _need_row_mask(rows, M)
        check(lib().reset_state_init_rows(ptr(state), M, w, ptr(rows), stream_handle(stream)), "reset_state_init_rows")


def _need_row_mask(rows: torch.Tensor, M: int) -> None:
    if rows.dtype not in (torch.uint8, torch.bool) or not rows.is_cuda or not rows.is_contiguous() or rows.shape != (M,):
        raise ValueError(f"rows must be a contiguous CUDA tensor [{M}] of uint8 or bool")


def reset_sample(logits, step_start, u, state, params: ResetParams, token, H_out, T_out, workspace, stream=None, rows=None):
    """One position of every row; with `rows` (uint8 or bool [M]) of those rows alone, the others' state and outputs
    stay as they are."""
    M, V = logits.shape
    if rows is not None:
        _need_row_mask(rows, M)
        check(lib().reset_sample_rows(ptr(logits), M, V, ptr(step_start), ptr(u), ptr(rows), ptr(state),
                                      ctypes.byref(params), ptr(token), ptr(H_out), ptr(T_out), ptr(workspace),
                                      workspace.numel(), stream_handle(stream)), "reset_sample_rows")
        return
    check(lib().reset_sample(ptr(logits), M, V, ptr(step_start), ptr(u), ptr(state), ctypes.byref(params),
                             ptr(token), ptr(H_out), ptr(T_out), ptr(workspace), workspace.numel(),
                             stream_handle(stream)), "reset_sample")


def reset_sample_noalloc(logits, step_start, u, state, params: ResetParams, token, H_out, T_out, stream=None):
    """reset_sample with its scratch in the library's static device array (no
    workspace): for callers that may not allocate device memory.  Limit
    M * ceil(V / 2048) <= 4096; calls that overlap on the GPU race."""
    M, V = logits.shape
    check(lib().reset_sample_noalloc(ptr(logits), M, V, ptr(step_start), ptr(u), ptr(state), ctypes.byref(params),
                                     ptr(token), ptr(H_out), ptr(T_out), stream_handle(stream)),
          "reset_sample_noalloc")


class ResetSampler:
    """Owns the per-row state, the workspace and the outputs of reset_sample for M rows x V logits.

    threshold: "reset" (ReSET's step-aware threshold), "fixed" (tau0 at every
    position) or "window" (the mean of the last w entropies); top_p in (0, 1)
    samples from the nucleus only (1 keeps every token)."""

    THRESHOLDS = {"reset": THRESHOLD_RESET, "fixed": THRESHOLD_FIXED, "window": THRESHOLD_WINDOW}

    def __init__(self, M: int, V: int, tau0=0.6, t_low=0.3, t_high=1.0, w=8, device="cuda", threshold="reset",
                 top_p=1.0):
        self.M, self.V = M, V
        self.params = ResetParams(tau0, t_low, t_high, w, self.THRESHOLDS[threshold], top_p)
        self.state = torch.zeros(reset_state_bytes(M, w), dtype=torch.uint8, device=device)
        self.workspace = torch.zeros(reset_workspace_bytes(M, V), dtype=torch.uint8, device=device)
        self.token = torch.zeros(M, dtype=torch.int32, device=device)
        self.H = torch.zeros(M, dtype=torch.float32, device=device)
        self.T = torch.zeros(M, dtype=torch.float32, device=device)
        reset_state_init(self.state, M, w)

    def __call__(self, logits, step_start, u, stream=None, rows=None):
        reset_sample(logits, step_start, u, self.state, self.params, self.token, self.H, self.T, self.workspace,
                     stream, rows)
        return self.token, self.H, self.T

    def restart(self, rows: torch.Tensor, stream=None):
        """The rows with rows[r] != 0 (uint8 or bool [M]) get new sequences."""
        reset_state_init(self.state, self.M, self.params.w, stream, rows)


def device_status() -> int:
    """Reads and clears the library's device error bits (synchronous).  After a
    GEMV wait gave up (DEVERR_FLAG_TIMEOUT), a late partial sum may sit in a
    workspace: every GemvWorkspace of this process is zeroed again; a caller's
    own workspace tensors must be zeroed by the caller."""
    code = ctypes.c_uint(0)
    check(lib().nvfp4_device_status(ctypes.byref(code)), "nvfp4_device_status")
    if code.value & DEVERR_FLAG_TIMEOUT:
        torch.cuda.synchronize()
        for ws in list(_live_workspaces):
            ws.rezero()
        torch.cuda.synchronize()
    return int(code.value)
