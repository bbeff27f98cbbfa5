// Rows of K and V into the NVFP4 KV cache and back.
//
// Append: one thread per 16-element block (the unit of the format): 32 bytes
// of BF16 in, 8 code bytes and a scale byte out, by the quantizer's own recipe
// (quant_block), so a cached row has the codes nvfp4_quantize_act would give it
// under the cache's global scale.  Bound by HBM: 2 bytes an element in, 9/16 out.
// Read: the reverse, 8.5 bytes in, 32 bytes out a thread.
#include "kv_layout.cuh"
#include "quant_block.cuh"

NVFP4_DEFINE_ERROR_READER(nvfp4_internal_read_error_kv_cache)

namespace {

constexpr int kThreads = 256;

struct AppendArgs {
  const void* x[2];             // K, V
  int64_t ts[2], hs[2];         // token and head strides in elements
  const int32_t* slots;
  uint8_t* pages;
  const float* glob[2];
  int tokens, heads, page_size;
  long long num_slots;
};

NVFP4_DEVINL void load16(const float* p, float (&v)[16]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float4 f = __ldcg(reinterpret_cast<const float4*>(p) + i);
    const float r[4] = {f.x, f.y, f.z, f.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) v[4 * i + j] = __bfloat162float(__float2bfloat16_rn(r[j]));
  }
}

NVFP4_DEVINL void load16(const uint16_t* p, float (&v)[16]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint4 u = __ldcg(reinterpret_cast<const uint4*>(p) + i);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[8 * i + 2 * j] = bf16_lo(w[j]);
      v[8 * i + 2 * j + 1] = bf16_hi(w[j]);
    }
  }
}

// Item = ((token * heads + head) * 2 + {K, V}) * (D / 16) + block.
template <int D, class T>
__global__ void __launch_bounds__(kThreads) kv_append_kernel(const AppendArgs a) {
  using L = KvLayout<D>;
  griddep_launch_dependents();
  griddep_wait();
  const long long items = (long long)a.tokens * a.heads * 2 * L::kBlocks;
  for (long long it = (long long)blockIdx.x * kThreads + threadIdx.x; it < items; it += (long long)gridDim.x * kThreads) {
    const int b = (int)(it % L::kBlocks);
    const int which = (int)(it / L::kBlocks & 1);
    const long long th = it / (2 * L::kBlocks);
    const int token = (int)(th / a.heads), head = (int)(th - (long long)token * a.heads);
    const int slot = a.slots[token];
    if (slot == -1) continue;
    if (slot < 0 || slot >= a.num_slots) {
      atomicOr(&g_nvfp4_device_error, NVFP4_DEVERR_KV_RANGE);
      continue;
    }
    float v[16];
    load16(static_cast<const T*>(a.x[which]) + token * a.ts[which] + head * a.hs[which] + b * 16, v);
    uint2 codes;
    const uint32_t s = quant_block(v, block_absmax(v), __ldg(a.glob[which]), codes);
    uint8_t* g = a.pages + kv_group_offset<D>(slot / a.page_size, slot % a.page_size, head, a.page_size, a.heads);
    const int t = slot % kKvGroup;
    if (which == 0) {
      *reinterpret_cast<uint2*>(g + L::k_codes(t, b)) = codes;
      g[L::k_scale(t, b)] = (uint8_t)s;
    } else {
      *reinterpret_cast<uint32_t*>(g + L::v_codes(t, b, 0)) = codes.x;
      *reinterpret_cast<uint32_t*>(g + L::v_codes(t, b, 1)) = codes.y;
      g[L::v_scale(t, b)] = (uint8_t)s;
    }
  }
}

struct ReadArgs {
  const uint8_t* pages;
  const int32_t* slots;
  const float* glob[2];
  uint16_t* out[2];
  int tokens, heads, page_size;
  long long num_slots;
};

// E2M1 code (4 bits) -> float: the three low bits at FP32 bits 24..22 are 2^-126 times the magnitude, exactly
// (also for the subnormal code 1); the multiply by 2^126 is exact.
NVFP4_DEVINL float e2m1_to_f32(uint32_t c) {
  return __uint_as_float(__float_as_uint(__fmul_rn(__uint_as_float((c & 7u) << 22), 0x1p126f)) | ((c & 8u) << 28));
}

template <int D>
__global__ void __launch_bounds__(kThreads) kv_read_kernel(const ReadArgs a) {
  using L = KvLayout<D>;
  griddep_launch_dependents();
  griddep_wait();
  const long long items = (long long)a.tokens * a.heads * 2 * L::kBlocks;
  for (long long it = (long long)blockIdx.x * kThreads + threadIdx.x; it < items; it += (long long)gridDim.x * kThreads) {
    const int b = (int)(it % L::kBlocks);
    const int which = (int)(it / L::kBlocks & 1);
    const long long th = it / (2 * L::kBlocks);
    const int token = (int)(th / a.heads), head = (int)(th - (long long)token * a.heads);
    const int slot = a.slots[token];
    uint4 o[2] = {make_uint4(0u, 0u, 0u, 0u), make_uint4(0u, 0u, 0u, 0u)};
    if (slot >= 0 && slot < a.num_slots) {
      const uint8_t* g = a.pages + kv_group_offset<D>(slot / a.page_size, slot % a.page_size, head, a.page_size, a.heads);
      const int t = slot % kKvGroup;
      uint2 c;
      uint32_t s;
      if (which == 0) {
        c = __ldcg(reinterpret_cast<const uint2*>(g + L::k_codes(t, b)));
        s = __ldcg(g + L::k_scale(t, b));
      } else {
        c.x = __ldcg(reinterpret_cast<const uint32_t*>(g + L::v_codes(t, b, 0)));
        c.y = __ldcg(reinterpret_cast<const uint32_t*>(g + L::v_codes(t, b, 1)));
        s = __ldcg(g + L::v_scale(t, b));
      }
      const float S = __fmul_rn(e4m3_to_f32(s), __ldg(a.glob[which]));
      uint32_t w[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint32_t byte = ((i < 4 ? c.x : c.y) >> (8 * (i & 3))) & 0xFFu;
        const __nv_bfloat162 p = __floats2bfloat162_rn(__fmul_rn(e2m1_to_f32(byte & 15u), S),
                                                       __fmul_rn(e2m1_to_f32(byte >> 4), S));
        w[i] = *reinterpret_cast<const uint32_t*>(&p);
      }
      o[0] = make_uint4(w[0], w[1], w[2], w[3]);
      o[1] = make_uint4(w[4], w[5], w[6], w[7]);
    } else if (slot != -1) {
      atomicOr(&g_nvfp4_device_error, NVFP4_DEVERR_KV_RANGE);
    }
    uint4* out = reinterpret_cast<uint4*>(a.out[which] + th * D + b * 16);
    out[0] = o[0];
    out[1] = o[1];
  }
}

template <class Args>
cudaError_t launch(void (*kern)(Args), long long items, const Args& a, cudaStream_t stream) {
  long long grid = (items + kThreads - 1) / kThreads;
  if (grid > 1 << 20) grid = 1 << 20;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, a);
}

}  // namespace

nvfp4_status nvfp4_internal_cuda_status(cudaError_t e);
bool nvfp4_internal_aligned(const void* p, size_t a);
nvfp4_status nvfp4_internal_check_device();

nvfp4_status nvfp4_internal_check_kv_cache(const nvfp4_kv_cache* c) {
  if (!c || !c->pages || !c->k_global || !c->v_global) return NVFP4_ERR_NULL;
  if (nvfp4_kv_page_bytes(c->page_size, c->kv_heads, c->head_dim) == 0) return NVFP4_ERR_SHAPE;
  if (c->num_pages < 1 || (long long)c->num_pages * c->page_size > 0x7FFFFFFFll) return NVFP4_ERR_SHAPE;
  if (!nvfp4_internal_aligned(c->pages, 16) || !nvfp4_internal_aligned(c->k_global, 4) ||
      !nvfp4_internal_aligned(c->v_global, 4))
    return NVFP4_ERR_ALIGN;
  return NVFP4_OK;
}

extern "C" size_t nvfp4_kv_page_bytes(int page_size, int kv_heads, int head_dim) {
  if (page_size < 16 || page_size > 1024 || page_size % 16 != 0) return 0;
  if (kv_heads < 1 || kv_heads > 1024 || (head_dim != 64 && head_dim != 128)) return 0;
  return (size_t)page_size / 16 * kv_heads * 18 * head_dim;
}

extern "C" nvfp4_status nvfp4_kv_append(const void* k, const void* v, int dtype, int tokens, int64_t k_token_stride,
                                        int64_t k_head_stride, int64_t v_token_stride, int64_t v_head_stride,
                                        const int32_t* slots, const nvfp4_kv_cache* cache, cudaStream_t stream) {
  const nvfp4_status cs = nvfp4_internal_check_kv_cache(cache);
  if (cs != NVFP4_OK) return cs;
  if (dtype != NVFP4_DTYPE_F32 && dtype != NVFP4_DTYPE_BF16) return NVFP4_ERR_RANGE;
  if (tokens < 0) return NVFP4_ERR_SHAPE;
  if (tokens == 0) return NVFP4_OK;
  if (!k || !v || !slots) return NVFP4_ERR_NULL;
  const int per = dtype == NVFP4_DTYPE_F32 ? 4 : 8;          // elements of 16 bytes
  if (k_token_stride % per || k_head_stride % per || v_token_stride % per || v_head_stride % per)
    return NVFP4_ERR_ALIGN;
  if (!nvfp4_internal_aligned(k, 16) || !nvfp4_internal_aligned(v, 16) || !nvfp4_internal_aligned(slots, 4))
    return NVFP4_ERR_ALIGN;
  const nvfp4_status ds = nvfp4_internal_check_device();
  if (ds != NVFP4_OK) return ds;
  AppendArgs a = {};
  a.x[0] = k, a.x[1] = v;
  a.ts[0] = k_token_stride, a.ts[1] = v_token_stride;
  a.hs[0] = k_head_stride, a.hs[1] = v_head_stride;
  a.slots = slots;
  a.pages = cache->pages;
  a.glob[0] = cache->k_global, a.glob[1] = cache->v_global;
  a.tokens = tokens, a.heads = cache->kv_heads, a.page_size = cache->page_size;
  a.num_slots = (long long)cache->num_pages * cache->page_size;
  const long long items = (long long)tokens * a.heads * 2 * (cache->head_dim / 16);
  cudaError_t e;
  if (cache->head_dim == 128)
    e = dtype == NVFP4_DTYPE_F32 ? launch(kv_append_kernel<128, float>, items, a, stream)
                                 : launch(kv_append_kernel<128, uint16_t>, items, a, stream);
  else
    e = dtype == NVFP4_DTYPE_F32 ? launch(kv_append_kernel<64, float>, items, a, stream)
                                 : launch(kv_append_kernel<64, uint16_t>, items, a, stream);
  return nvfp4_internal_cuda_status(e);
}

extern "C" nvfp4_status nvfp4_kv_read(const nvfp4_kv_cache* cache, const int32_t* slots, int tokens, uint16_t* k_out,
                                      uint16_t* v_out, cudaStream_t stream) {
  const nvfp4_status cs = nvfp4_internal_check_kv_cache(cache);
  if (cs != NVFP4_OK) return cs;
  if (tokens < 0) return NVFP4_ERR_SHAPE;
  if (tokens == 0) return NVFP4_OK;
  if (!slots || !k_out || !v_out) return NVFP4_ERR_NULL;
  if (!nvfp4_internal_aligned(slots, 4) || !nvfp4_internal_aligned(k_out, 16) || !nvfp4_internal_aligned(v_out, 16))
    return NVFP4_ERR_ALIGN;
  const nvfp4_status ds = nvfp4_internal_check_device();
  if (ds != NVFP4_OK) return ds;
  ReadArgs a = {};
  a.pages = cache->pages;
  a.slots = slots;
  a.glob[0] = cache->k_global, a.glob[1] = cache->v_global;
  a.out[0] = k_out, a.out[1] = v_out;
  a.tokens = tokens, a.heads = cache->kv_heads, a.page_size = cache->page_size;
  a.num_slots = (long long)cache->num_pages * cache->page_size;
  const long long items = (long long)tokens * a.heads * 2 * (cache->head_dim / 16);
  const cudaError_t e = cache->head_dim == 128 ? launch(kv_read_kernel<128>, items, a, stream)
                                               : launch(kv_read_kernel<64>, items, a, stream);
  return nvfp4_internal_cuda_status(e);
}
