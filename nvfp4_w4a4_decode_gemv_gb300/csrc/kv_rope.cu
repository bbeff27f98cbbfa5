// Rows of q and k rotated by their positions on the way: q to BF16, k and v into the NVFP4 KV cache.
//
// A pair of elements (a, b) of a rotated row becomes (a c - b s, b c + a s), c and s from a table by position; each product
// and each sum rounds to FP32 (no fused multiply-add, so that the bits are those of the formula step by step), the results
// to BF16, and k goes on to the cache as in nvfp4_kv_append.
//
// A thread takes a 16-element block of K or V, which the quantizer wants whole, and reads the block that a block of K is
// turned with beside it (from L1, where that block's own thread has it too).  Of q it takes 8 pairs of elements.  Bound by
// HBM: the rows in, q and the cache out.  8192 tokens of 40 heads of q and 8 of K and V, BF16, D 128: 211 MB in 41 us
// (5.1 TB/s), 54 with their read back; 8 tokens of 32 and 8 heads, FP32: 6.7 us cold, the loads' latency one after another.
// That prompt with the read back, with both blocks of a pair turned by one thread 60 us (its registers left too few warps to
// cover the loads), with q in a launch of its own 70, with all windows before q 58.
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
  unsigned kv_ctas;                                // CTAs of the windows' tasks (1 or more); the others turn q
};

// The slot of a token: as given; outside the cache where its position is outside the table; -1 stays -1 (padding).
struct SlotsAndPositions {
  const RopeArgs& a;
  NVFP4_DEVINL int operator()(long long i) const {
    const int s = a.slots[i];
    return s == -1 || (unsigned)a.positions[i] < (unsigned)a.max_positions ? s : -2;
  }
};

NVFP4_DEVINL void turn(float& a, float& b, float2 cs) {
  const float x = __fsub_rn(__fmul_rn(a, cs.x), __fmul_rn(b, cs.y));
  b = __fadd_rn(__fmul_rn(b, cs.x), __fmul_rn(a, cs.y));
  a = x;
}

// Element i of a block as it is given.
template <class T>
NVFP4_DEVINL float value_of(const Raw<T>& r, int i) {
  const uint4& q = r.w[i * (int)sizeof(T) / 16];
  const int w = i * (int)sizeof(T) / 4 % 4;
  const uint32_t u = w == 0 ? q.x : w == 1 ? q.y : w == 2 ? q.z : q.w;
  return sizeof(T) == 4 ? __uint_as_float(u) : (i & 1) ? bf16_hi(u) : bf16_lo(u);
}

// Block b of a row of K, turned and rounded to BF16.
template <class T>
NVFP4_DEVINL void turned_block(const RopeArgs& a, const T* row, int position, int b, float (&v)[16]) {
  Raw<T> own;
  own.load(row + b * 16);
  const int blocks = a.rotated / 16, half = blocks / 2;
  const float2* table = a.table + (size_t)position * (a.rotated / 2);
  if (b >= blocks) {
    own.values(v);
    return;
  }
  if (a.neighbours) {
    const float4* p = reinterpret_cast<const float4*>(table + 8 * b);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float4 cs = __ldg(p + i);
      v[4 * i] = value_of(own, 4 * i), v[4 * i + 1] = value_of(own, 4 * i + 1);
      v[4 * i + 2] = value_of(own, 4 * i + 2), v[4 * i + 3] = value_of(own, 4 * i + 3);
      turn(v[4 * i], v[4 * i + 1], make_float2(cs.x, cs.y));
      turn(v[4 * i + 2], v[4 * i + 3], make_float2(cs.z, cs.w));
    }
  } else {
    const bool first = b < half;
    Raw<T> other;
    other.load(row + (first ? b + half : b - half) * 16);
    const float4* p = reinterpret_cast<const float4*>(table + 16 * (first ? b : b - half));
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float4 cs = __ldg(p + i);
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        // a c - b s of the first half, b c + a s of the second (x + -y rounds as x - y)
        const float x = __fmul_rn(value_of(own, 2 * i + k), k == 0 ? cs.x : cs.z);
        const float y = __fmul_rn(value_of(other, 2 * i + k), k == 0 ? cs.y : cs.w);
        v[2 * i + k] = __fadd_rn(x, first ? -y : y);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = __bfloat162float(__float2bfloat16_rn(v[i]));
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

// A block of a token of one kv head on its own.
template <int D, class T>
NVFP4_DEVINL void append_block(const RopeArgs& a, long long token, int slot, int head, int which, int b) {
  float v[16];
  if (which == 0) {
    turned_block(a, static_cast<const T*>(a.k) + token * a.k_ts + head * a.k_hs, a.positions[token], b, v);
  } else {
    Raw<T> raw;
    raw.load(static_cast<const T*>(a.v) + token * a.v_ts + head * a.v_hs + b * 16);
    raw.values(v);
  }
  const int page = slot / a.page_size, in = slot - page * a.page_size, t = slot % kKvGroup;
  uint8_t* half = a.pages + kv_group_offset<D>(page, in, head, a.page_size, a.kv_heads) + which * Map<D>::kHalf;
  store_block<D>(half, which, t, b, v, *(which == 0 ? a.k_global : a.v_global));
}

// Rows of q go in smaller units than those of K: 8 pairs of elements, the 8 table entries from 8 u on, so that a thread keeps
// several heads' loads in flight.  first, second: where its two pieces of 8 elements stand.
struct Unit {
  int first, second;
  bool turned;
  NVFP4_DEVINL Unit(const RopeArgs& a, int u) {
    turned = 16 * u < a.rotated;
    const bool halves = turned && !a.neighbours;
    first = halves ? 8 * u : 16 * u;
    second = halves ? 8 * u + a.rotated / 2 : 16 * u + 8;
  }
};

template <class T>
struct Raw8 {                                // 8 FP32 or BF16 elements
  static constexpr int kPieces = sizeof(T) == 4 ? 2 : 1;
  uint4 w[kPieces];
  NVFP4_DEVINL void load(const T* p) {
#pragma unroll
    for (int i = 0; i < kPieces; ++i) w[i] = __ldcs(reinterpret_cast<const uint4*>(p) + i);
  }
  NVFP4_DEVINL void values(float (&v)[8]) const {
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      const uint32_t u[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if constexpr (sizeof(T) == 4) {
          v[4 * i + j] = __uint_as_float(u[j]);
        } else {
          v[2 * j] = bf16_lo(u[j]);
          v[2 * j + 1] = bf16_hi(u[j]);
        }
      }
    }
  }
};

NVFP4_DEVINL uint4 pack8(const float (&v)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 p = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&p);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// Unit u of heads [h0, h1) of a token's q, AT_ONCE heads' loads in flight.
template <int D, class T, int AT_ONCE>
NVFP4_DEVINL void turn_q(const RopeArgs& a, long long token, int slot, int h0, int h1, int u) {
  const Unit un(a, u);
  uint16_t* out = a.q_out + (token * a.heads + h0) * D;
  if (slot < 0 || slot >= a.num_slots) {
    for (int h = h0; h < h1; ++h, out += D)
      *reinterpret_cast<uint4*>(out + un.first) = *reinterpret_cast<uint4*>(out + un.second) = make_uint4(0u, 0u, 0u, 0u);
    return;
  }
  float2 cs[8];
  if (un.turned) {
    const float4* p = reinterpret_cast<const float4*>(a.table + (size_t)a.positions[token] * (a.rotated / 2) + 8 * u);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float4 x = __ldg(p + i);
      cs[2 * i] = make_float2(x.x, x.y);
      cs[2 * i + 1] = make_float2(x.z, x.w);
    }
  }
  const T* row = static_cast<const T*>(a.q) + token * a.q_ts + h0 * a.q_hs;
  for (int h = h0; h < h1; h += AT_ONCE) {
    Raw8<T> raw[AT_ONCE][2];
#pragma unroll
    for (int i = 0; i < AT_ONCE; ++i)
      if (h + i < h1) {
        raw[i][0].load(row + i * a.q_hs + un.first);
        raw[i][1].load(row + i * a.q_hs + un.second);
      }
#pragma unroll
    for (int i = 0; i < AT_ONCE; ++i)
      if (h + i < h1) {
        float v0[8], v1[8];
        raw[i][0].values(v0);
        raw[i][1].values(v1);
        if (un.turned) {
          if (a.neighbours) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              turn(v0[2 * j], v0[2 * j + 1], cs[j]);
              turn(v1[2 * j], v1[2 * j + 1], cs[4 + j]);
            }
          } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) turn(v0[j], v1[j], cs[j]);
          }
        }
        *reinterpret_cast<uint4*>(out + i * D + un.first) = pack8(v0);
        *reinterpret_cast<uint4*>(out + i * D + un.second) = pack8(v1);
      }
    row += AT_ONCE * a.q_hs;
    out += AT_ONCE * D;
  }
}

// Few tokens: a thread for each unit of each row of q, and for each block of each row of K and V.
template <int D, class T>
__global__ void __launch_bounds__(kThreads) kv_rope_few_kernel(const RopeArgs a) {
  griddep_launch_dependents();
  griddep_wait();
  constexpr int kUnits = D / 16, kBlocks = KvLayout<D>::kBlocks;
  const int of_q = a.heads * kUnits, per = of_q + 2 * a.kv_heads * kBlocks;   // threads of a token
  const long long at = (long long)blockIdx.x * kThreads + threadIdx.x;
  const long long token = at / per;
  const int in = (int)(at - token * per);
  if (token >= a.tokens) return;
  const int slot = SlotsAndPositions{a}(token);
  if (in == 0 && slot != -1 && (slot < 0 || slot >= a.num_slots)) atomicOr(&g_nvfp4_device_error, NVFP4_DEVERR_KV_RANGE);
  if (in < of_q) {
    turn_q<D, T, 1>(a, token, slot, in / kUnits, in / kUnits + 1, in % kUnits);
  } else if (slot >= 0 && slot < a.num_slots) {
    const int n = in - of_q, row = n / kBlocks;
    append_block<D, T>(a, token, slot, row >> 1, row & 1, n % kBlocks);
  }
}

// Many tokens: every so many CTAs one whose warps take a window of 16 tokens of K or V of one head (whole groups through
// shared memory in 16-byte pieces); warps of the others take a few tokens of kHeadsOfTask heads of q.  The two kinds are
// dealt in turn: a window waits for its loads, quantizes and writes little, and q streams past it meanwhile.
template <int D, class T>
__global__ void __launch_bounds__(kThreads, 4) kv_rope_kernel(const RopeArgs a) {
  using M = Map<D>;
  __shared__ __align__(16) uint8_t s_half[kWarps][M::kHalf];
  griddep_launch_dependents();
  griddep_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const unsigned every = gridDim.x / a.kv_ctas, mine = blockIdx.x / every;
  const bool of_kv = mine < a.kv_ctas && blockIdx.x - mine * every == 0u;
  if (!of_kv) {
    constexpr int kUnits = D / 16, kTokens = 32 / kUnits;
    const int groups = (a.heads + kHeadsOfTask - 1) / kHeadsOfTask;
    const long long n = (long long)(blockIdx.x - min(mine + 1u, a.kv_ctas)) * kWarps + warp;
    const int g = (int)(n % groups);
    const long long token = n / groups * kTokens + lane / kUnits;
    if (token >= a.tokens) return;
    turn_q<D, T, 2>(a, token, SlotsAndPositions{a}(token), g * kHeadsOfTask,
                    min(a.heads, (g + 1) * kHeadsOfTask), lane % kUnits);
    return;
  }
  const int b = lane % KvLayout<D>::kBlocks, t_lane = lane / KvLayout<D>::kBlocks;
  const long long n = (long long)mine * kWarps + warp, per = 2 * a.kv_heads, window = n / per;
  const int rest = (int)(n - window * per), head = rest >> 1, which = rest & 1;
  const long long i0 = window * kKvGroup;
  if (i0 >= a.tokens) return;
  const Window w = look_at_window(SlotsAndPositions{a}, a.tokens, i0, a.num_slots, lane, head == 0 && which == 0);
  const float glob = *(which == 0 ? a.k_global : a.v_global);
  const int64_t ts = which == 0 ? a.k_ts : a.v_ts;
  const T* rows = (which == 0 ? static_cast<const T*>(a.k) + head * a.k_hs : static_cast<const T*>(a.v) + head * a.v_hs) + i0 * ts;
  for (uint32_t lead = w.leads; lead != 0u; lead &= lead - 1u) {
    const int first = __ffs(lead) - 1;
    const int slot = __shfl_sync(0xffffffffu, w.slot, 16 + first), page = slot / a.page_size, in = slot - page * a.page_size;
    if (which == 0) {
#pragma unroll 1
      for (int p = 0; p < M::kPasses; ++p) {
        const int t = p * M::kPerPass + t_lane;
        float v[16];
        turned_block(a, rows + (first + t) * ts, a.positions[i0 + first + t], b, v);
        store_block<D>(s_half[warp], 0, t, b, v, glob);
      }
    } else {
      Raw<T> raw[M::kPasses];
#pragma unroll
      for (int p = 0; p < M::kPasses; ++p) raw[p].load(rows + (first + p * M::kPerPass + t_lane) * ts + b * 16);
#pragma unroll
      for (int p = 0; p < M::kPasses; ++p) {
        float v[16];
        raw[p].values(v);
        store_block<D>(s_half[warp], 1, p * M::kPerPass + t_lane, b, v, glob);
      }
    }
    __syncwarp();
    uint8_t* g = a.pages + kv_group_offset<D>(page, in, head, a.page_size, a.kv_heads) + which * M::kHalf;
    for (int i = lane; i < M::kHalf / 16; i += 32)
      reinterpret_cast<uint4*>(g)[i] = reinterpret_cast<const uint4*>(s_half[warp])[i];
    __syncwarp();
  }
  if (w.alone == 0u) return;
#pragma unroll 1
  for (int p = 0; p < M::kPasses; ++p) {
    const int t = p * M::kPerPass + t_lane;
    const int slot = __shfl_sync(0xffffffffu, w.slot, 16 + t);
    if ((w.alone >> t) & 1u) append_block<D, T>(a, i0 + t, slot, head, which, b);
  }
}

// Up to so many elements of K every block gets a thread of its own (40 and 8 heads of 128: 1024 tokens 8.3 us, by windows
// 12.1; 2048 tokens 14.3 and 13.8).
constexpr long long kFew = 1 << 20;

template <int D, class T>
cudaError_t launch(RopeArgs a, cudaStream_t stream) {
  constexpr int kUnits = D / 16, kTokens = 32 / kUnits;
  const bool few = (long long)a.tokens * a.kv_heads * D <= kFew;
  long long grid;
  if (few) {
    grid = (a.tokens * ((long long)a.heads * kUnits + 2ll * a.kv_heads * KvLayout<D>::kBlocks) + kThreads - 1) / kThreads;
  } else {
    const long long windows = (a.tokens + kKvGroup - 1ll) / kKvGroup * a.kv_heads * 2;
    const long long q_tasks = (a.tokens + kTokens - 1ll) / kTokens * ((a.heads + kHeadsOfTask - 1) / kHeadsOfTask);
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
