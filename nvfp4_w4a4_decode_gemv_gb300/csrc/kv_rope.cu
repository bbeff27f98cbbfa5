// Rows of q and k rotated by their positions on the way: q to BF16, k and v into the NVFP4 KV cache.
//
// A pair of elements (a, b) of a rotated row becomes (a c - b s, b c + a s), c and s from a table by position; each product
// and each sum rounds to FP32 (no fused multiply-add, so that the bits are those of the formula step by step), the results
// to BF16, and k goes on to the cache as in nvfp4_kv_append.
//
// A thread takes two 16-element blocks of a row that are turned together: blocks j and j + rotated/32 where the halves of
// the rotated part form the pairs, 2 j and 2 j + 1 where neighbours do; either way the pair needs the 16 table entries from
// 16 j on.  Bound by HBM: the rows in, q and the cache out.
#include <cuda_fp16.h>

#include "kv_rows.cuh"

NVFP4_DEFINE_ERROR_READER(nvfp4_internal_read_error_kv_rope)

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kHeadsOfTask = 8;           // heads of q that a thread turns with one load of the table

struct RopeArgs {
  const void *q, *k, *v;
  int64_t q_ts, q_hs, k_ts, k_hs, v_ts, v_hs;      // token and head strides in elements
  const int32_t *positions, *slots;
  const float2* table;                             // [max_positions][rotated / 2] of (cos, sin)
  uint16_t* q_out;
  uint8_t* pages;
  const float *k_global, *v_global;
  int tokens, heads, kv_heads, page_size, max_positions, rotated, neighbours;
  long long num_slots;
  unsigned kv_ctas;                                // CTAs of the windows' tasks; the others turn q
};

// The slot of a token: as given; outside the cache where its position is outside the table; -1 stays -1 (padding).
struct SlotsAndPositions {
  const RopeArgs& a;
  NVFP4_DEVINL int operator()(long long i) const {
    const int s = a.slots[i];
    return s == -1 || (unsigned)a.positions[i] < (unsigned)a.max_positions ? s : -2;
  }
};

// Pair j of the blocks of a row.
template <bool ROTATE>
struct Pair {
  int b0, b1;
  bool turned;
  NVFP4_DEVINL Pair(const RopeArgs& a, int j) {
    turned = ROTATE && 32 * j < a.rotated;
    const bool halves = turned && !a.neighbours;
    b0 = halves ? j : 2 * j;
    b1 = halves ? j + a.rotated / 32 : 2 * j + 1;
  }
};

NVFP4_DEVINL void load_table(const RopeArgs& a, int position, int j, float2 (&cs)[16]) {
  const float4* p = reinterpret_cast<const float4*>(a.table + (size_t)position * (a.rotated / 2) + 16 * j);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float4 x = __ldg(p + i);
    cs[2 * i] = make_float2(x.x, x.y);
    cs[2 * i + 1] = make_float2(x.z, x.w);
  }
}

NVFP4_DEVINL void turn(float& a, float& b, float2 cs) {
  const float x = __fsub_rn(__fmul_rn(a, cs.x), __fmul_rn(b, cs.y));
  b = __fadd_rn(__fmul_rn(b, cs.x), __fmul_rn(a, cs.y));
  a = x;
}

NVFP4_DEVINL void turn_blocks(float (&v0)[16], float (&v1)[16], const float2 (&cs)[16], int neighbours) {
  if (neighbours) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      turn(v0[2 * i], v0[2 * i + 1], cs[i]);
      turn(v1[2 * i], v1[2 * i + 1], cs[8 + i]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i) turn(v0[i], v1[i], cs[i]);
  }
}

// 16 FP32 or BF16 elements, not rounded.
template <class T>
NVFP4_DEVINL void exact_values(const Raw<T>& r, float (&v)[16]) {
#pragma unroll
  for (int i = 0; i < Raw<T>::kPieces; ++i) {
    const uint32_t u[4] = {r.w[i].x, r.w[i].y, r.w[i].z, r.w[i].w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if constexpr (sizeof(T) == 4) {
        v[4 * i + j] = __uint_as_float(u[j]);
      } else {
        v[8 * i + 2 * j] = bf16_lo(u[j]);
        v[8 * i + 2 * j + 1] = bf16_hi(u[j]);
      }
    }
  }
}

NVFP4_DEVINL void round_bf16(float (&v)[16]) {
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = __bfloat162float(__float2bfloat16_rn(v[i]));
}

NVFP4_DEVINL void store_bf16(uint16_t* dst, const float (&v)[16]) {
  uint32_t w[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const __nv_bfloat162 p = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&p);
  }
  reinterpret_cast<uint4*>(dst)[0] = make_uint4(w[0], w[1], w[2], w[3]);
  reinterpret_cast<uint4*>(dst)[1] = make_uint4(w[4], w[5], w[6], w[7]);
}

// Block b of token t of a group, into the group's K or V half (offsets of Map).
template <int D>
NVFP4_DEVINL void store_block(uint8_t* half, int which, int t, int b, float (&v)[16], float glob) {
  using M = Map<D>;
  uint2 c;
  const uint32_t s = kv_quant_block(v, glob, c);
  *reinterpret_cast<uint32_t*>(half + M::codes(which, t, b, 0)) = c.x;
  *reinterpret_cast<uint32_t*>(half + M::codes(which, t, b, 1)) = c.y;
  half[M::scale(which, t, b)] = (uint8_t)s;
}

// A token's pair j of one kv head on its own.
template <int D, class T>
NVFP4_DEVINL void append_pair(const RopeArgs& a, long long token, int slot, int head, int which, int j) {
  const T* row = which == 0 ? static_cast<const T*>(a.k) + token * a.k_ts + head * a.k_hs
                            : static_cast<const T*>(a.v) + token * a.v_ts + head * a.v_hs;
  float v0[16], v1[16];
  int b0 = 2 * j, b1 = 2 * j + 1;
  Raw<T> r0, r1;
  if (which == 0) {
    const Pair<true> p(a, j);
    b0 = p.b0, b1 = p.b1;
    r0.load(row + b0 * 16);
    r1.load(row + b1 * 16);
    exact_values(r0, v0);
    exact_values(r1, v1);
    if (p.turned) {
      float2 cs[16];
      load_table(a, a.positions[token], j, cs);
      turn_blocks(v0, v1, cs, a.neighbours);
    }
    round_bf16(v0);
    round_bf16(v1);
  } else {
    r0.load(row + b0 * 16);
    r1.load(row + b1 * 16);
    r0.values(v0);
    r1.values(v1);
  }
  const int page = slot / a.page_size, in = slot - page * a.page_size, t = slot % kKvGroup;
  uint8_t* half = a.pages + kv_group_offset<D>(page, in, head, a.page_size, a.kv_heads) + which * Map<D>::kHalf;
  const float glob = *(which == 0 ? a.k_global : a.v_global);
  store_block<D>(half, which, t, b0, v0, glob);
  store_block<D>(half, which, t, b1, v1, glob);
}

// Pair j of heads [h0, h1) of a token's q.
template <int D, class T>
NVFP4_DEVINL void turn_q(const RopeArgs& a, long long token, int slot, int position, int h0, int h1, int j) {
  const Pair<true> p(a, j);
  uint16_t* out = a.q_out + (token * a.heads + h0) * D;
  if (slot < 0 || slot >= a.num_slots) {
    for (int h = h0; h < h1; ++h, out += D) {
      reinterpret_cast<uint4*>(out + p.b0 * 16)[0] = reinterpret_cast<uint4*>(out + p.b0 * 16)[1] = make_uint4(0u, 0u, 0u, 0u);
      reinterpret_cast<uint4*>(out + p.b1 * 16)[0] = reinterpret_cast<uint4*>(out + p.b1 * 16)[1] = make_uint4(0u, 0u, 0u, 0u);
    }
    return;
  }
  float2 cs[16];
  if (p.turned) load_table(a, position, j, cs);
  const T* row = static_cast<const T*>(a.q) + token * a.q_ts + h0 * a.q_hs;
  for (int h = h0; h < h1; ++h, row += a.q_hs, out += D) {
    Raw<T> r0, r1;
    r0.load(row + p.b0 * 16);
    r1.load(row + p.b1 * 16);
    float v0[16], v1[16];
    exact_values(r0, v0);
    exact_values(r1, v1);
    if (p.turned) turn_blocks(v0, v1, cs, a.neighbours);
    store_bf16(out + p.b0 * 16, v0);
    store_bf16(out + p.b1 * 16, v1);
  }
}

// Few tokens: a thread for each pair of blocks of each row, q first.
template <int D, class T>
__global__ void __launch_bounds__(kThreads) kv_rope_few_kernel(const RopeArgs a) {
  griddep_launch_dependents();
  griddep_wait();
  constexpr int kPairs = D / 32;
  const int rows = a.heads + 2 * a.kv_heads;
  const long long at = (long long)blockIdx.x * kThreads + threadIdx.x;
  const int j = (int)(at % kPairs), row = (int)(at / kPairs % rows);
  const long long token = at / kPairs / rows;
  if (token >= a.tokens) return;
  const int slot = SlotsAndPositions{a}(token);
  if (row == 0 && j == 0 && slot != -1 && (slot < 0 || slot >= a.num_slots))
    atomicOr(&g_nvfp4_device_error, NVFP4_DEVERR_KV_RANGE);
  if (row < a.heads) {
    turn_q<D, T>(a, token, slot, a.positions[token], row, row + 1, j);
  } else if (slot >= 0 && slot < a.num_slots) {
    const int n = row - a.heads;
    append_pair<D, T>(a, token, slot, n >> 1, n & 1, j);
  }
}

// Many tokens: warps of the first CTAs take a window of 16 tokens of K or V of one head (whole groups through shared
// memory in 16-byte pieces), warps of the others a few tokens of kHeadsOfTask heads of q.
template <int D, class T>
__global__ void __launch_bounds__(kThreads, 2) kv_rope_kernel(const RopeArgs a) {
  using M = Map<D>;
  constexpr int kPairs = D / 32, kPerPass = 32 / kPairs, kPasses = kKvGroup / kPerPass;
  __shared__ __align__(16) uint8_t s_half[kWarps][M::kHalf];
  griddep_launch_dependents();
  griddep_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int j = lane % kPairs, t_lane = lane / kPairs;
  if (blockIdx.x >= a.kv_ctas) {
    const int groups = (a.heads + kHeadsOfTask - 1) / kHeadsOfTask;
    const long long n = (long long)(blockIdx.x - a.kv_ctas) * kWarps + warp;
    const int g = (int)(n % groups);
    const long long token = n / groups * kPerPass + t_lane;
    if (token >= a.tokens) return;
    turn_q<D, T>(a, token, SlotsAndPositions{a}(token), a.positions[token], g * kHeadsOfTask,
                 min(a.heads, (g + 1) * kHeadsOfTask), j);
    return;
  }
  const long long n = (long long)blockIdx.x * kWarps + warp, per = 2 * a.kv_heads, window = n / per;
  const int rest = (int)(n - window * per), head = rest >> 1, which = rest & 1;
  const long long i0 = window * kKvGroup;
  if (i0 >= a.tokens) return;
  const Window w = look_at_window(SlotsAndPositions{a}, a.tokens, i0, a.num_slots, lane, head == 0 && which == 0);
  const float glob = *(which == 0 ? a.k_global : a.v_global);
  const int64_t ts = which == 0 ? a.k_ts : a.v_ts;
  const T* rows = (which == 0 ? static_cast<const T*>(a.k) + head * a.k_hs : static_cast<const T*>(a.v) + head * a.v_hs) + i0 * ts;
  const Pair<true> pk(a, j);
  const int b0 = which == 0 ? pk.b0 : 2 * j, b1 = which == 0 ? pk.b1 : 2 * j + 1;
  const bool turned = which == 0 && pk.turned;
  for (uint32_t lead = w.leads; lead != 0u; lead &= lead - 1u) {
    const int first = __ffs(lead) - 1;
    Raw<T> raw[kPasses][2];
#pragma unroll
    for (int p = 0; p < kPasses; ++p) {
      const T* row = rows + (first + p * kPerPass + t_lane) * ts;
      raw[p][0].load(row + b0 * 16);
      raw[p][1].load(row + b1 * 16);
    }
    const int slot = __shfl_sync(0xffffffffu, w.slot, 16 + first), page = slot / a.page_size, in = slot - page * a.page_size;
#pragma unroll
    for (int p = 0; p < kPasses; ++p) {
      const int t = p * kPerPass + t_lane;
      float v0[16], v1[16];
      exact_values(raw[p][0], v0);
      exact_values(raw[p][1], v1);
      if (turned) {
        float2 cs[16];
        load_table(a, a.positions[i0 + first + t], j, cs);
        turn_blocks(v0, v1, cs, a.neighbours);
      }
      round_bf16(v0);
      round_bf16(v1);
      store_block<D>(s_half[warp], which, t, b0, v0, glob);
      store_block<D>(s_half[warp], which, t, b1, v1, glob);
    }
    __syncwarp();
    uint8_t* g = a.pages + kv_group_offset<D>(page, in, head, a.page_size, a.kv_heads) + which * M::kHalf;
    for (int i = lane; i < M::kHalf / 16; i += 32)
      reinterpret_cast<uint4*>(g)[i] = reinterpret_cast<const uint4*>(s_half[warp])[i];
    __syncwarp();
  }
  if (w.alone == 0u) return;
#pragma unroll 1
  for (int p = 0; p < kPasses; ++p) {
    const int t = p * kPerPass + t_lane;
    const int slot = __shfl_sync(0xffffffffu, w.slot, 16 + t);
    if ((w.alone >> t) & 1u) append_pair<D, T>(a, i0 + t, slot, head, which, j);
  }
}

// Up to so many elements of K every pair of blocks gets a thread of its own (as in nvfp4_kv_append).
constexpr long long kFew = 1 << 20;

template <int D, class T>
cudaError_t launch(RopeArgs a, cudaStream_t stream) {
  constexpr int kPairs = D / 32, kPerPass = 32 / kPairs;
  const long long rows = a.heads + 2ll * a.kv_heads;
  const bool few = (long long)a.tokens * a.kv_heads * D <= kFew;
  long long grid;
  if (few) {
    grid = (a.tokens * rows * kPairs + kThreads - 1) / kThreads;
  } else {
    const long long windows = (a.tokens + kKvGroup - 1) / kKvGroup * a.kv_heads * 2;
    const long long q_tasks = (a.tokens + kPerPass - 1) / kPerPass * ((a.heads + kHeadsOfTask - 1) / kHeadsOfTask);
    a.kv_ctas = (unsigned)((windows + kWarps - 1) / kWarps);
    grid = a.kv_ctas + (q_tasks + kWarps - 1) / kWarps;
  }
  if (grid > 0x7FFFFFFFll) return cudaErrorInvalidConfiguration;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, few ? kv_rope_few_kernel<D, T> : kv_rope_kernel<D, T>, a);
}

}  // namespace

nvfp4_status nvfp4_internal_cuda_status(cudaError_t e);
bool nvfp4_internal_aligned(const void* p, size_t a);
nvfp4_status nvfp4_internal_check_device();

extern "C" nvfp4_status nvfp4_kv_append_rope(const void* q, const void* k, const void* v, int dtype, int tokens, int heads,
                                             int64_t q_token_stride, int64_t q_head_stride, int64_t k_token_stride,
                                             int64_t k_head_stride, int64_t v_token_stride, int64_t v_head_stride,
                                             const int32_t* positions, const float* table, int max_positions, int rotated,
                                             int style, const int32_t* slots, const nvfp4_kv_cache* cache, uint16_t* q_out,
                                             cudaStream_t stream) {
  const nvfp4_status cs = nvfp4_internal_check_kv_cache(cache);
  if (cs != NVFP4_OK) return cs;
  if (dtype != NVFP4_DTYPE_F32 && dtype != NVFP4_DTYPE_BF16) return NVFP4_ERR_RANGE;
  if (style != NVFP4_ROPE_HALVES && style != NVFP4_ROPE_PAIRS) return NVFP4_ERR_RANGE;
  if (tokens < 0 || heads < 0 || heads > 65536 || max_positions < 1 || rotated < 32 || rotated > cache->head_dim ||
      rotated % 32 != 0)
    return NVFP4_ERR_SHAPE;
  if (tokens == 0) return NVFP4_OK;
  if (!k || !v || !positions || !table || !slots || (heads > 0 && (!q || !q_out))) return NVFP4_ERR_NULL;
  const int per = dtype == NVFP4_DTYPE_F32 ? 4 : 8;          // elements of 16 bytes
  // (the stride of a single token or head is used in no address)
  if (tokens > 1 && ((heads > 0 && q_token_stride % per) || k_token_stride % per || v_token_stride % per))
    return NVFP4_ERR_ALIGN;
  if (heads > 1 && q_head_stride % per) return NVFP4_ERR_ALIGN;
  if (cache->kv_heads > 1 && (k_head_stride % per || v_head_stride % per)) return NVFP4_ERR_ALIGN;
  if (!nvfp4_internal_aligned(q, 16) || !nvfp4_internal_aligned(k, 16) || !nvfp4_internal_aligned(v, 16) ||
      !nvfp4_internal_aligned(table, 16) || !nvfp4_internal_aligned(q_out, 16) || !nvfp4_internal_aligned(slots, 4) ||
      !nvfp4_internal_aligned(positions, 4))
    return NVFP4_ERR_ALIGN;
  const nvfp4_status ds = nvfp4_internal_check_device();
  if (ds != NVFP4_OK) return ds;
  RopeArgs a = {};
  a.q = q, a.k = k, a.v = v;
  a.q_ts = q_token_stride, a.q_hs = q_head_stride;
  a.k_ts = k_token_stride, a.k_hs = k_head_stride;
  a.v_ts = v_token_stride, a.v_hs = v_head_stride;
  a.positions = positions, a.slots = slots;
  a.table = reinterpret_cast<const float2*>(table);
  a.q_out = q_out;
  a.pages = cache->pages;
  a.k_global = cache->k_global, a.v_global = cache->v_global;
  a.tokens = tokens, a.heads = heads, a.kv_heads = cache->kv_heads, a.page_size = cache->page_size;
  a.max_positions = max_positions, a.rotated = rotated, a.neighbours = style == NVFP4_ROPE_PAIRS;
  a.num_slots = (long long)cache->num_pages * cache->page_size;
  cudaError_t e;
  if (cache->head_dim == 128)
    e = dtype == NVFP4_DTYPE_F32 ? launch<128, float>(a, stream) : launch<128, uint16_t>(a, stream);
  else
    e = dtype == NVFP4_DTYPE_F32 ? launch<64, float>(a, stream) : launch<64, uint16_t>(a, stream);
  return nvfp4_internal_cuda_status(e);
}
