// Rows of K and V into the NVFP4 KV cache and back.
//
// A 16-element block is the unit of work: 32 bytes of BF16, 8 code bytes and a
// scale byte, by the quantizer's own recipe (quant_block), so a cached row has the
// codes nvfp4_quantize_act would give it under the cache's global scale.  Bound by
// HBM: 2 bytes an element on one side, 9/16 on the other.
//
// The cache's order scatters a token's bytes over its 16-token group, and writes
// of 1, 4 and 8 bytes cost L2 a 32-byte sector each (one thread a block, every
// block on its own: 12.3 M sectors for 16384 tokens of 8 heads, 50 us).  So a warp
// takes the K or V rows of one head for a window of 16 tokens.  Where the 16 tokens
// of a whole group follow one another (prompts) and the first of them is in the
// window, it quantizes the group's half into shared memory and moves it in 16-byte
// pieces.  Other tokens (single new tokens, the ragged ends of prompts) go block by
// block.  A warp finds out by itself, with ballots: with a CTA looking together, its
// barriers took a third of the time (16384 tokens of 8 heads of 128: append 27 us instead
// of 31, read 17.5 instead of 22; 12.6 each at the copy rate).
#include <cuda_fp16.h>

#include "kv_rows.cuh"

NVFP4_DEFINE_ERROR_READER(nvfp4_internal_read_error_kv_cache)

namespace {

constexpr int kThreads = 256;

struct AppendArgs {
  const void *k, *v;
  int64_t k_ts, k_hs, v_ts, v_hs;   // token and head strides in elements
  const int32_t* slots;
  uint8_t* pages;
  const float *k_global, *v_global;
  int tokens, heads, page_size;
  long long num_slots;
  uint64_t inv_heads;               // 2^32 / heads, rounded up: a quotient where it times heads is below 2^32
};

// One block of a token on its own.
template <int D, class T>
NVFP4_DEVINL void append_block(const AppendArgs& a, long long token, int slot, int head, int which, int b) {
  using M = Map<D>;
  Raw<T> raw;
  raw.load(which == 0 ? static_cast<const T*>(a.k) + token * a.k_ts + head * a.k_hs + b * 16
                      : static_cast<const T*>(a.v) + token * a.v_ts + head * a.v_hs + b * 16);
  const int page = slot / a.page_size, in = slot - page * a.page_size, t = slot % kKvGroup;
  float v[16];
  raw.values(v);
  uint2 c;
  const uint32_t s = kv_quant_block(v, *(which == 0 ? a.k_global : a.v_global), c);
  uint8_t* g = a.pages + kv_group_offset<D>(page, in, head, a.page_size, a.heads) + which * M::kHalf;
  *reinterpret_cast<uint32_t*>(g + M::codes(which, t, b, 0)) = c.x;
  *reinterpret_cast<uint32_t*>(g + M::codes(which, t, b, 1)) = c.y;
  g[M::scale(which, t, b)] = (uint8_t)s;
}

constexpr int kWarps = kThreads / 32;

// A warp's task: window, head, K or V, in this order.
struct Task {
  long long i0;
  int head, which;
  bool there;
  NVFP4_DEVINL Task(int tokens, int heads) {
    const long long n = (long long)blockIdx.x * kWarps + (threadIdx.x >> 5), per = 2 * heads;
    const long long window = n / per;
    const int rest = (int)(n - window * per);
    i0 = window * kKvGroup;
    head = rest >> 1;
    which = rest & 1;
    there = i0 < tokens;
  }
};

template <int D, class T>
__global__ void __launch_bounds__(kThreads, 3) kv_append_kernel(const AppendArgs a) {
  using M = Map<D>;
  __shared__ __align__(16) uint8_t s_half[kWarps][M::kHalf];
  griddep_launch_dependents();
  griddep_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const Task k(a.tokens, a.heads);
  if (!k.there) return;
  const Window w = look_at_window(SlotsOf{a.slots}, a.tokens, k.i0, a.num_slots, lane, k.head == 0 && k.which == 0);
  const float glob = *(k.which == 0 ? a.k_global : a.v_global);
  const int64_t ts = k.which == 0 ? a.k_ts : a.v_ts;
  const T* rows = (k.which == 0 ? static_cast<const T*>(a.k) + k.head * a.k_hs : static_cast<const T*>(a.v) + k.head * a.v_hs) +
                  k.i0 * ts;
  const int b = lane % KvLayout<D>::kBlocks, t_lane = lane / KvLayout<D>::kBlocks;
  for (uint32_t lead = w.leads; lead != 0u; lead &= lead - 1u) {
    const int first = __ffs(lead) - 1;
    Raw<T> raw[M::kPasses];
#pragma unroll
    for (int p = 0; p < M::kPasses; ++p) raw[p].load(rows + (first + p * M::kPerPass + t_lane) * ts + b * 16);
    const int slot = __shfl_sync(0xffffffffu, w.slot, 16 + first), page = slot / a.page_size, in = slot - page * a.page_size;
#pragma unroll
    for (int p = 0; p < M::kPasses; ++p) {
      const int t = p * M::kPerPass + t_lane;
      float v[16];
      raw[p].values(v);
      uint2 c;
      const uint32_t s = kv_quant_block(v, glob, c);
      *reinterpret_cast<uint32_t*>(&s_half[warp][M::codes(k.which, t, b, 0)]) = c.x;
      *reinterpret_cast<uint32_t*>(&s_half[warp][M::codes(k.which, t, b, 1)]) = c.y;
      s_half[warp][M::scale(k.which, t, b)] = (uint8_t)s;
    }
    __syncwarp();
    uint8_t* g = a.pages + kv_group_offset<D>(page, in, k.head, a.page_size, a.heads) + k.which * M::kHalf;
    for (int i = lane; i < M::kHalf / 16; i += 32)
      reinterpret_cast<uint4*>(g)[i] = reinterpret_cast<const uint4*>(s_half[warp])[i];
    __syncwarp();
  }
  if (w.alone == 0u) return;
  // the other tokens, block by block
#pragma unroll 1
  for (int p = 0; p < M::kPasses; ++p) {
    const int t = p * M::kPerPass + t_lane;
    const int slot = __shfl_sync(0xffffffffu, w.slot, 16 + t);
    if ((w.alone >> t) & 1u) append_block<D, T>(a, k.i0 + t, slot, k.head, k.which, b);
  }
}

// Few tokens: a thread for every block, no look at the neighbours.
template <int D, class T>
__global__ void __launch_bounds__(kThreads) kv_append_few_kernel(const AppendArgs a) {
  griddep_launch_dependents();
  griddep_wait();
  const int it = blockIdx.x * kThreads + threadIdx.x;
  const int b = it % KvLayout<D>::kBlocks, which = it / KvLayout<D>::kBlocks & 1, at = it / (2 * KvLayout<D>::kBlocks);
  const int token = (int)((uint64_t)at * a.inv_heads >> 32), head = at - token * a.heads;
  if (token >= a.tokens) return;
  const int slot = a.slots[token];
  if (slot >= 0 && slot < a.num_slots) append_block<D, T>(a, token, slot, head, which, b);
  else if (slot != -1) atomicOr(&g_nvfp4_device_error, NVFP4_DEVERR_KV_RANGE);
}

struct ReadArgs {
  const uint8_t* pages;
  const int32_t* slots;
  const float *k_global, *v_global;
  uint16_t *k_out, *v_out;
  int tokens, heads, page_size;
  long long num_slots;
  uint64_t inv_heads;               // 2^32 / heads, rounded up: a quotient where it times heads is below 2^32
};

// 4 code bytes times S -> 8 BF16 values, 16 bytes.
NVFP4_DEVINL uint4 half_block(uint32_t c, float S) {
  uint32_t f[4], w[4];
  e2m1x8_to_f16(c, f);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&f[i]));
    const __nv_bfloat162 p = __floats2bfloat162_rn(__fmul_rn(x.x, S), __fmul_rn(x.y, S));
    w[i] = *reinterpret_cast<const uint32_t*>(&p);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// Half a block (h 0, 1) of a token on its own; slot -1: zeros.
template <int D>
NVFP4_DEVINL void read_half(const ReadArgs& a, long long token, int slot, int head, int which, int b, int h) {
  using M = Map<D>;
  uint32_t c = 0u;
  float S = 0.0f;
  if (slot >= 0) {
    const int page = slot / a.page_size, in = slot - page * a.page_size, t = slot % kKvGroup;
    const uint8_t* g = a.pages + kv_group_offset<D>(page, in, head, a.page_size, a.heads) + which * M::kHalf;
    c = __ldcg(reinterpret_cast<const uint32_t*>(g + M::codes(which, t, b, h)));
    S = __fmul_rn(e4m3_to_f32(__ldcg(g + M::scale(which, t, b))), *(which == 0 ? a.k_global : a.v_global));
  }
  *reinterpret_cast<uint4*>((which == 0 ? a.k_out : a.v_out) + (token * a.heads + head) * D + b * 16 + h * 8) =
      half_block(c, S);
}

template <int D>
__global__ void __launch_bounds__(kThreads, 6) kv_read_kernel(const ReadArgs a) {
  using M = Map<D>;
  __shared__ __align__(16) uint8_t s_half[kWarps][M::kHalf];
  griddep_launch_dependents();
  griddep_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const Task k(a.tokens, a.heads);
  if (!k.there) return;
  const Window w = look_at_window(SlotsOf{a.slots}, a.tokens, k.i0, a.num_slots, lane, k.head == 0 && k.which == 0);
  const float glob = *(k.which == 0 ? a.k_global : a.v_global);
  // a lane takes half a block, so that a store of the warp is whole rows
  constexpr int kHalves = 2 * KvLayout<D>::kBlocks, kTokens = 32 / kHalves;
  const int hb = lane % kHalves, b = hb >> 1, h = hb & 1;
  uint16_t* rows = (k.which == 0 ? a.k_out : a.v_out) + (k.i0 * a.heads + k.head) * D + hb * 8;
  for (uint32_t lead = w.leads; lead != 0u; lead &= lead - 1u) {
    const int first = __ffs(lead) - 1;
    const int slot = __shfl_sync(0xffffffffu, w.slot, 16 + first), page = slot / a.page_size, in = slot - page * a.page_size;
    const uint8_t* g = a.pages + kv_group_offset<D>(page, in, k.head, a.page_size, a.heads) + k.which * M::kHalf;
    for (int i = lane; i < M::kHalf / 16; i += 32)
      reinterpret_cast<uint4*>(s_half[warp])[i] = __ldcg(reinterpret_cast<const uint4*>(g) + i);
    __syncwarp();
#pragma unroll
    for (int p = 0; p < kKvGroup / kTokens; ++p) {
      const int t = p * kTokens + lane / kHalves;
      const uint32_t c = *reinterpret_cast<const uint32_t*>(&s_half[warp][M::codes(k.which, t, b, h)]);
      const float S = __fmul_rn(e4m3_to_f32(s_half[warp][M::scale(k.which, t, b)]), glob);
      *reinterpret_cast<uint4*>(rows + (long long)(first + t) * a.heads * D) = half_block(c, S);
    }
    __syncwarp();
  }
  // tokens outside whole groups, padding among them (zeros)
  if ((w.alone | w.rest) == 0u) return;
#pragma unroll 1
  for (int p = 0; p < kKvGroup / kTokens; ++p) {
    const int t = p * kTokens + lane / kHalves;
    const int slot = __shfl_sync(0xffffffffu, w.slot, 16 + t);
    if (((w.alone | w.rest) >> t) & 1u)
      read_half<D>(a, k.i0 + t, ((w.alone >> t) & 1u) ? slot : -1, k.head, k.which, b, h);
  }
}

template <int D>
__global__ void __launch_bounds__(kThreads) kv_read_few_kernel(const ReadArgs a) {
  griddep_launch_dependents();
  griddep_wait();
  const int it = blockIdx.x * kThreads + threadIdx.x;
  const int hb = it % (2 * KvLayout<D>::kBlocks), which = it / (2 * KvLayout<D>::kBlocks) & 1;
  const int at = it / (4 * KvLayout<D>::kBlocks), token = (int)((uint64_t)at * a.inv_heads >> 32);
  const int head = at - token * a.heads;
  if (token >= a.tokens) return;
  int slot = a.slots[token];
  if (slot < 0 || slot >= a.num_slots) {
    if (slot != -1) atomicOr(&g_nvfp4_device_error, NVFP4_DEVERR_KV_RANGE);
    slot = -1;
  }
  read_half<D>(a, token, slot, head, which, hb >> 1, hb & 1);
}

// Up to so many elements of K every (half) block gets a thread of its own at once, and the shorter chain of loads wins.
// Own threads / windows, BF16, 8 heads of 128, us:  append 2.2 / 3.0 (256 tokens), 4.5 / 4.9 (2048), 7.3 / 6.6 (4096);
// read 2.1 / 2.6, 4.7 / 4.5, 8.0 / 5.6.  One head: append 1.9 / 2.9, 2.1 / 3.0, 3.0 / 3.2.
constexpr long long kFew = 1 << 21;

// per_thread: elements of K or V that a thread of `few` has, twice over.
template <int D, class Args>
cudaError_t launch(void (*window)(Args), void (*few)(Args), Args a, int per_thread, cudaStream_t stream) {
  const long long tasks = (a.tokens + (long long)kKvGroup - 1) / kKvGroup * a.heads * 2;
  const bool is_few = (long long)a.tokens * a.heads * D <= kFew;   // (heads <= 1024)
  a.inv_heads = ((1ull << 32) + a.heads - 1) / a.heads;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(is_few ? ((long long)a.tokens * a.heads * (D / per_thread) + kThreads - 1) / kThreads
                                       : (tasks + kWarps - 1) / kWarps));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, is_few ? few : window, a);
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
  // (the stride of a single token or head is used in no address)
  if (tokens > 1 && (k_token_stride % per || v_token_stride % per)) return NVFP4_ERR_ALIGN;
  if (cache->kv_heads > 1 && (k_head_stride % per || v_head_stride % per)) return NVFP4_ERR_ALIGN;
  if (!nvfp4_internal_aligned(k, 16) || !nvfp4_internal_aligned(v, 16) || !nvfp4_internal_aligned(slots, 4))
    return NVFP4_ERR_ALIGN;
  const nvfp4_status ds = nvfp4_internal_check_device();
  if (ds != NVFP4_OK) return ds;
  AppendArgs a = {};
  a.k = k, a.v = v;
  a.k_ts = k_token_stride, a.k_hs = k_head_stride;
  a.v_ts = v_token_stride, a.v_hs = v_head_stride;
  a.slots = slots;
  a.pages = cache->pages;
  a.k_global = cache->k_global, a.v_global = cache->v_global;
  a.tokens = tokens, a.heads = cache->kv_heads, a.page_size = cache->page_size;
  a.num_slots = (long long)cache->num_pages * cache->page_size;
  cudaError_t e;
  if (cache->head_dim == 128)
    e = dtype == NVFP4_DTYPE_F32 ? launch<128>(kv_append_kernel<128, float>, kv_append_few_kernel<128, float>, a, 8, stream)
                                 : launch<128>(kv_append_kernel<128, uint16_t>, kv_append_few_kernel<128, uint16_t>, a, 8, stream);
  else
    e = dtype == NVFP4_DTYPE_F32 ? launch<64>(kv_append_kernel<64, float>, kv_append_few_kernel<64, float>, a, 8, stream)
                                 : launch<64>(kv_append_kernel<64, uint16_t>, kv_append_few_kernel<64, uint16_t>, a, 8, stream);
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
  a.k_global = cache->k_global, a.v_global = cache->v_global;
  a.k_out = k_out, a.v_out = v_out;
  a.tokens = tokens, a.heads = cache->kv_heads, a.page_size = cache->page_size;
  a.num_slots = (long long)cache->num_pages * cache->page_size;
  const cudaError_t e = cache->head_dim == 128 ? launch<128>(kv_read_kernel<128>, kv_read_few_kernel<128>, a, 4, stream)
                                               : launch<64>(kv_read_kernel<64>, kv_read_few_kernel<64>, a, 4, stream);
  return nvfp4_internal_cuda_status(e);
}
