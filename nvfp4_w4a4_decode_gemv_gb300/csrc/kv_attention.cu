// Attention over the NVFP4 KV cache:
//   out[r, h] = sum_j p_j V[j] / sum_j p_j,  p_j = exp(scale * q[r, h] . K[j] - m),  m the running maximum,
// over the keys j that row r sees (causal from the bottom right, optionally a
// window), in one pass with the running maximum and sum.
#include <math.h>

#include "kv_layout.cuh"

NVFP4_DEFINE_ERROR_READER(nvfp4_internal_read_error_kv_attention)

namespace {

struct AttnArgs {
  const void* q;
  int64_t q_ts, q_hs;
  const uint8_t* pages;
  const float *k_global, *v_global;
  const int32_t *table, *kv_lens, *cu_q;
  uint16_t* out;
  float* lse;
  int tokens, heads, kv_heads, group, page_size, num_pages, width, batch, window;
  float scale;
};

NVFP4_DEVINL float e2m1_to_f32(uint32_t c) {
  return __uint_as_float(__float_as_uint(__fmul_rn(__uint_as_float((c & 7u) << 22), 0x1p126f)) | ((c & 8u) << 28));
}

NVFP4_DEVINL float load_q(const float* p) { return __bfloat162float(__float2bfloat16_rn(*p)); }
NVFP4_DEVINL float load_q(const uint16_t* p) { return __uint_as_float((uint32_t)*p << 16); }

// One warp per (row, head); a lane holds D / 32 elements.
template <int D, class T>
__global__ void __launch_bounds__(128) kv_attention_kernel(const AttnArgs a) {
  using L = KvLayout<D>;
  constexpr int E = D / 32;
  const int lane = threadIdx.x & 31;
  const long long item = (long long)blockIdx.x * 4 + (threadIdx.x >> 5);
  if (item >= (long long)a.tokens * a.heads) return;
  const int row = (int)(item / a.heads), h = (int)(item % a.heads), kvh = h / a.group;
  int b = row, first = row, last = row + 1;
  if (a.cu_q) {
    int lo = 0, hi = a.batch;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (a.cu_q[mid] <= row) lo = mid; else hi = mid;
    }
    b = lo;
    first = a.cu_q[b];
    last = a.cu_q[b + 1];
    if (row < first || row >= last) return;       // a row of no request
  }
  int len = max(a.kv_lens[b], 0);
  if (len > (long long)a.width * a.page_size) {
    len = a.width * a.page_size;
    atomicOr(&g_nvfp4_device_error, NVFP4_DEVERR_KV_RANGE);
  }
  const int p = len - (last - first) + (row - first);
  const int j_end = min(p + 1, len);
  const int j_begin = a.window > 0 ? max(p - a.window + 1, 0) : 0;
  const int blk = lane / (32 / L::kBlocks), e0 = (lane % (32 / L::kBlocks)) * E;   // first element in its block
  float q[E], o[E];
  const float qs = a.scale * *a.k_global;
#pragma unroll
  for (int i = 0; i < E; ++i) {
    q[i] = load_q(static_cast<const T*>(a.q) + row * a.q_ts + h * a.q_hs + blk * 16 + e0 + i) * qs;
    o[i] = 0.0f;
  }
  float m = -INFINITY, l = 0.0f;
  for (int j = j_begin; j < j_end; ++j) {
    const int page = a.table[(size_t)b * a.width + j / a.page_size];
    if (page < 0 || page >= a.num_pages) {
      if (lane == 0) atomicOr(&g_nvfp4_device_error, NVFP4_DEVERR_KV_RANGE);
      continue;
    }
    const uint8_t* g = a.pages + kv_group_offset<D>(page * a.page_size + j % a.page_size, kvh, a.page_size, a.kv_heads);
    const int t = j % kKvGroup;
    const float ks = e4m3_to_f32(g[L::k_scale(t, blk)]), vs = e4m3_to_f32(g[L::v_scale(t, blk)]);
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < E; ++i) {
      const int e = e0 + i;
      const uint32_t byte = g[L::k_codes(t, blk) + e / 2];
      s = fmaf(q[i], e2m1_to_f32(byte >> (4 * (e & 1))) * ks, s);
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
    const float mn = fmaxf(m, s);
    const float f = expf(m - mn), w = expf(s - mn);
    m = mn;
    l = fmaf(l, f, w);
#pragma unroll
    for (int i = 0; i < E; ++i) {
      const int e = e0 + i;
      const uint32_t byte = g[L::v_codes(t, blk, e / 8) + e % 8 / 2];
      o[i] = fmaf(o[i], f, w * (e2m1_to_f32(byte >> (4 * (e & 1))) * vs));
    }
  }
  const float inv = l > 0.0f ? *a.v_global / l : 0.0f;
#pragma unroll
  for (int i = 0; i < E; ++i)
    a.out[((size_t)row * a.heads + h) * D + blk * 16 + e0 + i] = __bfloat16_as_ushort(__float2bfloat16_rn(o[i] * inv));
  if (a.lse && lane == 0) a.lse[(size_t)row * a.heads + h] = l > 0.0f ? m + logf(l) : -INFINITY;
}

}  // namespace

nvfp4_status nvfp4_internal_cuda_status(cudaError_t e);
bool nvfp4_internal_aligned(const void* p, size_t a);
nvfp4_status nvfp4_internal_check_device();

extern "C" size_t nvfp4_kv_attention_workspace_bytes(int batch, int tokens, int heads, int kv_heads, int head_dim) {
  if (batch < 1 || tokens < 0 || nvfp4_kv_page_bytes(16, kv_heads, head_dim) == 0) return 0;
  if (heads < kv_heads || heads % kv_heads != 0 || heads / kv_heads > 64) return 0;
  return 256;
}

extern "C" nvfp4_status nvfp4_kv_attention(const void* q, int dtype, int tokens, int64_t q_token_stride,
                                           int64_t q_head_stride, int heads, const nvfp4_kv_cache* cache,
                                           const int32_t* block_table, int table_width, const int32_t* kv_lens,
                                           const int32_t* cu_q, int batch, int max_q, float scale, int window,
                                           uint16_t* out, float* lse, void* workspace, size_t workspace_bytes,
                                           cudaStream_t stream) {
  const nvfp4_status cs = nvfp4_internal_check_kv_cache(cache);
  if (cs != NVFP4_OK) return cs;
  if (dtype != NVFP4_DTYPE_F32 && dtype != NVFP4_DTYPE_BF16) return NVFP4_ERR_RANGE;
  if (!(scale > 0.0f) || isinf(scale) || window < 0 || max_q < 1) return NVFP4_ERR_RANGE;
  if (tokens < 0 || batch < 0 || table_width < 1 || (!cu_q && tokens != batch)) return NVFP4_ERR_SHAPE;
  if (heads < cache->kv_heads || heads % cache->kv_heads != 0 || heads / cache->kv_heads > 64) return NVFP4_ERR_SHAPE;
  if ((long long)batch * table_width > 0x7FFFFFFFll) return NVFP4_ERR_SHAPE;
  if (tokens == 0 || batch == 0) return NVFP4_OK;
  if (!q || !block_table || !kv_lens || !out || !workspace) return NVFP4_ERR_NULL;
  const int per = dtype == NVFP4_DTYPE_F32 ? 4 : 8;
  if (q_token_stride % per || q_head_stride % per) return NVFP4_ERR_ALIGN;
  if (!nvfp4_internal_aligned(q, 16) || !nvfp4_internal_aligned(out, 16) || !nvfp4_internal_aligned(workspace, 256))
    return NVFP4_ERR_ALIGN;
  for (const void* p : {(const void*)block_table, (const void*)kv_lens, (const void*)cu_q, (const void*)lse})
    if (!nvfp4_internal_aligned(p, 4)) return NVFP4_ERR_ALIGN;
  if (workspace_bytes < nvfp4_kv_attention_workspace_bytes(batch, tokens, heads, cache->kv_heads, cache->head_dim))
    return NVFP4_ERR_SHAPE;
  const nvfp4_status ds = nvfp4_internal_check_device();
  if (ds != NVFP4_OK) return ds;
  const AttnArgs a = {q, q_token_stride, q_head_stride, cache->pages, cache->k_global, cache->v_global,
                      block_table, kv_lens, cu_q, out, lse, tokens, heads, cache->kv_heads,
                      heads / cache->kv_heads, cache->page_size, cache->num_pages, table_width, batch, window, scale};
  const unsigned grid = (unsigned)(((long long)tokens * heads + 3) / 4);
  if (cache->head_dim == 128) {
    if (dtype == NVFP4_DTYPE_F32) kv_attention_kernel<128, float><<<grid, 128, 0, stream>>>(a);
    else kv_attention_kernel<128, uint16_t><<<grid, 128, 0, stream>>>(a);
  } else {
    if (dtype == NVFP4_DTYPE_F32) kv_attention_kernel<64, float><<<grid, 128, 0, stream>>>(a);
    else kv_attention_kernel<64, uint16_t><<<grid, 128, 0, stream>>>(a);
  }
  return nvfp4_internal_cuda_status(cudaGetLastError());
}
