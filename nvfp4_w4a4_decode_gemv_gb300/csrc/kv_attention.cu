// Attention over the NVFP4 KV cache, for few query rows a request (decode,
// drafted tokens):
//   out[r, h] = sum_j p_j V[j] / sum_j p_j,  p_j = 2^(f q[r, h] . K[j] - m),  m a running maximum,
// over the keys j that row r sees, f = scale * log2 e, in one pass over the cache.
//
// Bound by HBM: 18 D / 16 bytes a token and kv head, each read once for all the
// query heads (and rows) that share it.  What could stop it from getting there
// is the instruction rate: a token of one kv head (D = 128) is 256 elements, and
// at the copy rate an SM has about 6 cycles (24 issue slots) for it.  So:
//  - the matrix instructions (mma.m16n8k16, FP16 in, FP32 out) have the tokens or
//    the elements of V on their 16-row side and the query rows on the 8-column
//    side: no half-empty tiles at 8 query heads a kv head;
//  - a code and its scale multiply exactly in FP16 (2 + 4 significant bits, 2^-10
//    .. 2688), so dequantization is one conversion and one multiply for two
//    elements; V's two tokens of an operand register are put together on the 4-bit
//    codes (half an instruction an operand) instead of on the FP16 values;
//  - the cache's own layout is that of the operands, so a lane's loads are whole
//    16-byte pieces without bank conflicts.
// Queries enter as FP16 of q / 2^e, 2^e the power of two at the row's maximum:
// exact for BF16 queries down to 2^-14 of it.  Weights are rounded to FP16 for
// the product with V (2^-11 of each, 0 below 2^-25 of the maximum); their sum is of
// the FP32 weights, so up to n 2^-25 of it may have no part in the product: less than
// what n additions in FP32 may lose.
//
// Work split: units of 64 or 32 tokens (D = 64: 128 or 64) of one (request, kv head, row tile),
// Stream-K over all of them, so that any mix of lengths fills the GPU; the split
// is made on the GPU from the lengths (a captured call follows them).  A CTA of
// four warps takes a contiguous range; its warps take every fourth unit of a
// segment, each with its own ring of bulk copies (no CTA barrier while it
// streams) and its own running maximum, and are merged in shared memory at the
// segment's end.  Segments that several CTAs share go through records in the
// workspace; the last CTA to arrive merges them in CTA order (the same bits
// every time) and resets the counter.  Nothing waits for another CTA.
//
// 8 requests of 131000 keys, 64/8 heads of 128: 204 us, 5.9 TB/s (0.87 of the copy rate), 60 % of the issue slots.
// 8 rows over 1000 keys: 9.7 us, a chain of set-up, first copy, products and merge.
#include <math.h>

#include "kv_attention.cuh"

NVFP4_DEFINE_ERROR_READER(nvfp4_internal_read_error_kv_attention)

namespace {

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
// Pieces of a segment when there are few: more cost more to merge than they save.  8 query heads on each of 1 / 8 kv
// heads, one request of 4000 keys, us with 4, 8, 16, 32 pieces:  16.1, 12.8, 12.4, 15.3 / 16.3, 12.8, 13.8, 17.6;
// 16000 keys on one kv head: 37, 23, 17.9, 17.9.
constexpr int kMaxSplits = 16;
// Where there are many: a piece of K / s keys and a merge of s pieces take time a K / s + b s, least at s = sqrt(a K / b).
// One request, 64/8 heads, us with 16, 24, 32, 48, 64 pieces:  8000 keys 16.0, 16.5, 18.3, 23.3, 23.2;  16000 keys 20.8,
// 20.1, 21.5, 24.3, 25.8;  64000 keys 48, 37, 40, 35, 35;  131000 keys 74, 59, 62, 53, 50.
constexpr int kMaxShares = 64;
constexpr float kShareRate = 1.0f / 6.0f;   // s / sqrt(K)
// More query rows of a kv head than this, and more rows x keys (kv heads x keys there is room for, and what segments
// cost besides), take the other kernel (kv_attention_tc.cu).  Here / there, D = 128, 8 kv heads, us:  32 rows: 36 / 44
// (4 requests of 8000 keys), 53 / 58 (16 of 4000), 93 / 135 (16 of 500 to 16384);  64 rows: 15 / 28 (one of 2000),
// 35 / 48 (one of 16000), 49 / 45, 77 / 60, 142 / 137;  128 rows: 19 / 31, 59 / 52, 96 / 48, 145 / 62, 275 / 142;
// prompts of 200 and 400 tokens, 4 query heads a kv head:  19 / 24, 35 / 26.
constexpr int kTcRows = 48;
constexpr long long kTcProducts = 10 << 20;
// Keys that the fixed cost of a segment (queries, first copies, merge) stands for in the split.  With 256, 512, 1024:
// 64 requests x 16 heads with a window of 1024 keys 33.6, 30.1, 30.1 us; 16 requests of 500 to 16384 keys, 32 rows 93,
// 84.6, 86.5 us.
constexpr int kSegmentCost = 512;
// Rounds for a warp below which units are halved; the same cases with 4, 8, 32: 30.9, 30.1, 30.1 and 84.7, 84.6, 94 us.
constexpr int kShortUnits = 8;

NVFP4_DEVINL int shares_of(int keys) {
  return min(max((int)(sqrtf((float)keys) * kShareRate), kMaxSplits), kMaxShares);
}

NVFP4_DEVINL uint32_t transpose8x8(uint32_t a) {
  uint32_t d;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}

// d = a b, and d += a b.
NVFP4_DEVINL void mma16816_first(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.0f));
}
NVFP4_DEVINL void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// ---- shapes --------------------------------------------------------------------
template <int D, int NT>
struct Shape {
  static constexpr int kRows = 8 * NT;                     // query rows of a tile
  static constexpr int kUnitGroups = 512 / D;              // most groups of a unit: 64 tokens at D = 128, 128 at D = 64
  static constexpr int kUnitLog = D == 128 ? 6 : 7;        // log2 of its tokens; short work has units of half of that
  static constexpr int kUnitBytes = kUnitGroups * KvLayout<D>::kGroupBytes;
  static constexpr int kPair = 2;                          // groups whose scores are formed together (latency)
  static constexpr int kStages = 2;
  static constexpr int kMergeStride = D + 4;               // floats a row in the merge buffer (bank spread)
  static constexpr int kRecord = kRows * (D + 2);          // floats of a record: O, then M, then L
  // shared memory
  static constexpr int kOffRing = 0;
  static constexpr int kOffQ = kWarps * kStages * kUnitBytes;             // FP16 query operands
  static constexpr int kOffMerge = 0;                      // [kWarps][8][kMergeStride] floats, in the ring: idle then
  static_assert(kWarps * 8 * kMergeStride * 4 <= kOffQ, "the merge buffer");
  static constexpr int kOffML = kOffQ + kRows * D * 2;                    // [kWarps][kRows] maxima, then sums
  static constexpr int kOffF = kOffML + 2 * kWarps * kRows * 4;           // [kRows] score factors
  static constexpr int kOffBar = kOffF + kRows * 4;                       // [kWarps][kStages] barriers
  static constexpr int kOffScan = kOffBar + kWarps * kStages * 8;         // 32 words for the split
  static constexpr int kSmem = (kOffScan + 32 * 4 + 15) / 16 * 16;
};

// Units of a segment (one row tile of one kv head); at least one, so that rows without keys are written too.
NVFP4_DEVINL int segment_units(const Request& r, int unit_log) {
  const int n = ((r.len + (1 << unit_log) - 1) >> unit_log) - (r.begin >> unit_log);
  return n > 0 ? n : 1;
}
template <class S>
NVFP4_DEVINL int request_tiles(const AttnArgs& a, const Request& r) {
  return (r.rows * a.group + S::kRows - 1) / S::kRows;
}

// How the segments are laid end to end for the split: each stands for `head` units of overhead, its own units,
// and padding to a multiple of `align`.
struct Split {
  int head, align;
  NVFP4_DEVINL int length(int n) const { return head + (n + align - 1) / align * align; }
};

// G equal shares of U units, the first U % G one longer.
struct Shares {
  int size, longer;
  Shares() = default;
  NVFP4_DEVINL Shares(int U, int G) : size(U / G), longer(U - size * G) {}
  NVFP4_DEVINL int start(int q) const { return q * size + min(q, longer); }
  NVFP4_DEVINL int owner(int x) const {
    const int head = longer * (size + 1);
    return x < head ? x / (size + 1) : longer + (x - head) / size;
  }
};

// ---- one unit of keys ---------------------------------------------------------------
// Scores, weights and output of one 16-token group.  `masked`: rows see part of it only.
template <int D, int NT>
struct WarpState {
  float o[D / 16][NT][4];               // [row tile][column tile]: elements (2i, 2i + 1 of the lane's) x rows 2c, 2c + 1
  float m[NT][2], l[NT][2];             // running maximum (log2 units), the lane's part of the sum
};

template <int D, int NT>
NVFP4_DEVINL void scores(const uint8_t* g, int lane, const uint32_t (&qreg)[NT * (D / 16)][2], float (&s)[NT][4]) {
  using L = KvLayout<D>;
  constexpr int W = D / 32;             // code words of the lane's D/4 elements of a row
  uint32_t raw[2][W];
  const int r = lane >> 2, c = lane & 3;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint8_t* p = g + (8 * i + r) * (D / 2) + c * (D / 8);
    if constexpr (D == 128) {
      const uint4 v = lds128(p);
      raw[i][0] = v.x, raw[i][1] = v.y, raw[i][2] = v.z, raw[i][3] = v.w;
    } else {
      const uint2 v = lds64(p);
      raw[i][0] = v.x, raw[i][1] = v.y;
    }
  }
  uint32_t sc[2][D / 64];               // FP16 pairs of the lane's block scales
  if constexpr (D == 128) {
    const uint32_t w = *reinterpret_cast<const uint32_t*>(g + L::kOffKScale + lane * 4);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t h = e4m3x2_to_f16(w >> (16 * i));
      sc[i][0] = __byte_perm(h, h, 0x1010);
      sc[i][1] = __byte_perm(h, h, 0x3232);
    }
  } else {
    const uint32_t h = e4m3x2_to_f16(*reinterpret_cast<const uint16_t*>(g + L::kOffKScale + lane * 2));
    sc[0][0] = __byte_perm(h, h, 0x1010);
    sc[1][0] = __byte_perm(h, h, 0x3232);
  }
#pragma unroll
  for (int w = 0; w < W; ++w) {         // a word: 8 elements, two contraction steps
    uint32_t h[2][4];
    e2m1x8_to_f16(raw[0][w], h[0]);
    e2m1x8_to_f16(raw[1][w], h[1]);
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const uint32_t a[4] = {hmul2(h[0][2 * u], sc[0][w / 2]), hmul2(h[1][2 * u], sc[1][w / 2]),
                             hmul2(h[0][2 * u + 1], sc[0][w / 2]), hmul2(h[1][2 * u + 1], sc[1][w / 2])};
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const uint32_t(&b)[2] = qreg[t * (D / 16) + 2 * w + u];
        if (w == 0 && u == 0) mma16816_first(s[t], a, b[0], b[1]);
        else mma16816(s[t], a, b[0], b[1]);
      }
    }
  }
}

// O += V^T P for one group; p[t]: FP16 weights as B operands; live: how many of the lane's four tokens exist.
template <int D, int NT>
NVFP4_DEVINL void weigh(const uint8_t* g, int lane, const uint32_t (&p)[NT][2], int live, WarpState<D, NT>& st) {
  using L = KvLayout<D>;
  const int r = lane >> 2, c = lane & 3;
  uint32_t sw = *reinterpret_cast<const uint32_t*>(g + L::kOffVScale + (D == 128 ? r : r >> 1) * 16 + 4 * c);
  if (live < 4) sw &= live > 0 ? (1u << (8 * live)) - 1u : 0u;      // what lies behind the last key may be NaN
  const uint32_t s01 = e4m3x2_to_f16(sw), s23 = e4m3x2_to_f16(sw >> 16);
  constexpr int W = D / 64;             // code words of a token: the lane's D/8 elements
  uint32_t x[4][W];                     // [token]
  if constexpr (D == 128) {
    const uint8_t* q = g + L::kOffV + (r >> 1) * 256 + (r & 1) * 64 + c * 16;
    const uint4 v0 = lds128(q), v1 = lds128(q + 128);
    x[0][0] = v0.x, x[0][1] = v0.y, x[1][0] = v0.z, x[1][1] = v0.w;
    x[2][0] = v1.x, x[2][1] = v1.y, x[3][0] = v1.z, x[3][1] = v1.w;
  } else {
    const uint4 v = lds128(g + L::kOffV + r * 64 + c * 16);
    x[0][0] = v.x, x[1][0] = v.y, x[2][0] = v.z, x[3][0] = v.w;
  }
#pragma unroll
  for (int w = 0; w < W; ++w) {
    // even and odd elements of two tokens side by side in a byte
    uint32_t h[4][4];
    constexpr uint32_t kLo = 0x0F0F0F0Fu;
    e2m1x8_to_f16((x[0][w] & kLo) | ((x[1][w] << 4) & ~kLo), h[0]);
    e2m1x8_to_f16(((x[0][w] >> 4) & kLo) | (x[1][w] & ~kLo), h[1]);
    e2m1x8_to_f16((x[2][w] & kLo) | ((x[3][w] << 4) & ~kLo), h[2]);
    e2m1x8_to_f16(((x[2][w] >> 4) & kLo) | (x[3][w] & ~kLo), h[3]);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t a[4] = {hmul2(h[0][i], s01), hmul2(h[1][i], s01), hmul2(h[2][i], s23), hmul2(h[3][i], s23)};
#pragma unroll
      for (int t = 0; t < NT; ++t) mma16816(st.o[4 * w + i][t], a, p[t][0], p[t][1]);
    }
  }
}

// ---- the kernel -----------------------------------------------------------------------
template <int D, int NT, class T>
__global__ void __launch_bounds__(kThreads, NT == 1 ? 3 : 2) kv_attention_kernel(const AttnArgs a) {
  using S = Shape<D, NT>;
  using L = KvLayout<D>;
  extern __shared__ __align__(128) uint8_t smem[];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + S::kOffBar) + warp * S::kStages;
  uint8_t* ring = smem + S::kOffRing + warp * S::kStages * S::kUnitBytes;
  float* s_f = reinterpret_cast<float*>(smem + S::kOffF);
  float* s_m = reinterpret_cast<float*>(smem + S::kOffML);
  float* s_l = s_m + kWarps * S::kRows;
  float* s_merge = reinterpret_cast<float*>(smem + S::kOffMerge);
  if (lane == 0)
    for (int i = 0; i < S::kStages; ++i) mbar_init(&bars[i], 1);
  fence_mbar_init();
  griddep_launch_dependents();
  griddep_wait();
  fence_proxy_async_global();

  // ---- the split: this CTA's range and the request it starts in (all counts fit 31 bits: the host checks).
  // Up to 32 requests every warp works it out by itself, a request a lane; more are shared by the CTA's threads.
  int b, base, u, u_end, n_ctas, unit_log;
  Split split;
  Shares shares;
  {
    const bool small = a.batch <= 32;
    int* s_scan = reinterpret_cast<int*>(smem + S::kOffScan);
    const int per = small ? 1 : (a.batch + kThreads - 1) / kThreads, me = small ? lane : tid;
    const int b0 = min(per * me, a.batch), b1 = min(b0 + per, a.batch);
    // units of the two sizes, each segment's padded to one for every warp
    int units4 = 0, units4_half = 0, n_segs = 0, longest = 0;
    Request own = {};                                   // the thread's request, where it has one only
    bool bad = false;
    for (int i = b0; i < b1; ++i) {
      own = get_request(a, i, blockIdx.x == 0);
      bad = bad || own.bad;
      const int segs = request_tiles<S>(a, own) * a.kv_heads, n = segment_units(own, S::kUnitLog - 1);
      units4 += segs * ((segment_units(own, S::kUnitLog) + kWarps - 1) / kWarps);
      units4_half += segs * ((n + kWarps - 1) / kWarps);
      n_segs += segs;
      if (segs > 0) longest = max(longest, n);          // in halves
    }
    units4 = __reduce_add_sync(0xffffffffu, units4);
    units4_half = __reduce_add_sync(0xffffffffu, units4_half);
    n_segs = __reduce_add_sync(0xffffffffu, n_segs);
    longest = __reduce_max_sync(0xffffffffu, longest);
    if (!small) {
      if (lane == 0) {
        s_scan[warp] = units4;
        s_scan[4 + warp] = longest;
        s_scan[8 + warp] = n_segs;
        s_scan[20 + warp] = units4_half;
      }
      bad = __syncthreads_or(bad);
      units4 = s_scan[0] + s_scan[1] + s_scan[2] + s_scan[3];
      longest = max(max(s_scan[4], s_scan[5]), max(s_scan[6], s_scan[7]));
      n_segs = s_scan[8] + s_scan[9] + s_scan[10] + s_scan[11];
      units4_half = s_scan[20] + s_scan[21] + s_scan[22] + s_scan[23];
    }
    // Ranges that never fall add up to no more than the rows there are, and the host's bound on the units holds.
    // Where one falls, the others may overlap: the call is given up if they do.
    if (small ? __any_sync(0xffffffffu, bad) : bad) {
      float rows = 0.0f;
      for (int i = b0; i < b1; ++i) rows += (float)get_request(a, i, false).rows;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) rows += __shfl_xor_sync(0xffffffffu, rows, o);
      if (!small) {
        if (lane == 0) s_scan[24 + warp] = __float_as_int(rows);
        __syncthreads();
        rows = __int_as_float(s_scan[24]) + __int_as_float(s_scan[25]) + __int_as_float(s_scan[26]) + __int_as_float(s_scan[27]);
      }
      if (rows > 1.001f * (float)a.tokens) return;
    }
    if (units4 == 0) return;
    // less than kShortUnits rounds for a warp: halves of units divide more evenly, and their latency is shorter
    unit_log = units4 < kShortUnits * (int)gridDim.x ? S::kUnitLog - 1 : S::kUnitLog;
    if (unit_log != S::kUnitLog) units4 = units4_half;
    else longest = (longest + 1) / 2;
    // Few units: every CTA a piece of one segment, one unit a warp or as many as keep a segment's pieces under
    // kMaxSplits.  Many: equal ranges, where a segment's fixed cost counts as kSegmentCost keys, and at most
    // shares_of its keys of them a segment.
    const bool few = units4 <= (int)gridDim.x;
    const int piece = kWarps * max(1, (longest + kWarps * kMaxSplits - 1) / (kWarps * kMaxSplits));
    split = few ? Split{0, piece} : Split{kSegmentCost >> unit_log, 1};
    int mine = 0;
    for (int i = b0; i < b1; ++i) {
      const Request r = per == 1 ? own : get_request(a, i, false);
      mine += split.length(segment_units(r, unit_log)) * request_tiles<S>(a, r) * a.kv_heads;
    }
    int inc = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += v;
    }
    int U = __shfl_sync(0xffffffffu, inc, 31);
    if (!small) {
      if (lane == 31) s_scan[12 + warp] = inc;
      __syncthreads();
      U = 0;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        if (w < warp) inc += s_scan[12 + w];
        U += s_scan[12 + w];
      }
    }
    const int excl = inc - mine;
    n_ctas = few ? min((int)gridDim.x, U / piece) : (int)min((long long)gridDim.x, (long long)shares_of(longest << unit_log) * n_segs);
    if ((int)blockIdx.x >= n_ctas) return;
    shares = Shares(U, n_ctas);
    u = shares.start(blockIdx.x);
    u_end = shares.start(blockIdx.x + 1);
    const bool here = excl <= u && u < excl + mine;
    if (small) {
      const int l = __ffs(__ballot_sync(0xffffffffu, here)) - 1;
      b = l;
      base = __shfl_sync(0xffffffffu, excl, l);
    } else {
      if (here) {
        int at = excl;
        for (int i = b0; i < b1; ++i) {
          const Request r = per == 1 ? own : get_request(a, i, false);
          const int n = split.length(segment_units(r, unit_log)) * request_tiles<S>(a, r) * a.kv_heads;
          if (u < at + n) {
            s_scan[16] = i;
            s_scan[17] = at;
            break;
          }
          at += n;
        }
      }
      __syncthreads();
      b = s_scan[16];
      base = s_scan[17];
    }
  }
  const int cta = blockIdx.x;

  const float kg = *a.k_global, vg = *a.v_global;
  uint32_t slot = 0, phase = 0;                         // of the next copy that this warp waits for
  auto advance = [&]() {
    if (++slot == S::kStages) {
      slot = 0;
      phase ^= 1u;
    }
  };
  bool gave_up = false;
  while (u < u_end) {
    const Request rq = get_request(a, b, false);
    const int n_seg = segment_units(rq, unit_log), tiles = request_tiles<S>(a, rq), len_seg = split.length(n_seg);
    const int n_req = len_seg * tiles * a.kv_heads;
    if (u >= base + n_req) {
      base += n_req;
      ++b;
      continue;
    }
    const int seg = (u - base) / len_seg;
    const int seg0 = base + seg * len_seg;              // where it stands; its own units from seg0 + head on
    const int s0 = max(u - seg0 - split.head, 0);
    const int s1 = min(min(len_seg, u_end - seg0) - split.head, n_seg);
    u = min(seg0 + len_seg, u_end);
    if (s1 <= s0) continue;                             // overhead or padding only
    const int kvh = seg / tiles, tile = seg - kvh * tiles;
    const int row0 = tile * S::kRows;                   // row = query row * group + query head of the kv head
    const int n_rows = min(S::kRows, rq.rows * a.group - row0);
    // positions of the tile's first and last row: every row sees [lo_all, hi_all], some row [lo_any, hi_any]
    const int hi_all = rq.len - rq.rows + row0 / a.group;
    const int hi_any = rq.len - rq.rows + (row0 + n_rows - 1) / a.group;
    const int lo_any = a.window > 0 ? max(hi_all - a.window + 1, 0) : 0;
    const int lo_all = a.window > 0 ? max(hi_any - a.window + 1, 0) : 0;

    // ---- the queries' loads first: they and the page table's are in flight together
    constexpr int E = D / 32;
    float v[S::kRows / kWarps][E];
#pragma unroll
    for (int i = 0; i < S::kRows / kWarps; ++i) {
      const int row = warp + i * kWarps;
      const int rr = row0 + min(row, n_rows - 1), tok = rq.first + rr / a.group, h = kvh * a.group + rr % a.group;
      const T* q = static_cast<const T*>(a.q) + tok * a.q_ts + h * a.q_hs + lane * E;
#pragma unroll
      for (int e = 0; e < E; ++e) v[i][e] = row < n_rows ? load_q(q + e) : 0.0f;
    }

    // ---- this warp's units, and its first copies
    const int unit0 = rq.begin >> unit_log;             // the segment's first unit
    const int u_lo = max(s0, (lo_any >> unit_log) - unit0);
    const int u_hi = hi_any < 0 ? u_lo : min(s1, (hi_any >> unit_log) + 1 - unit0);
    const int my_n = u_lo + warp < u_hi ? (u_hi - u_lo - warp + kWarps - 1) / kWarps : 0;
    const int32_t* trow = a.table + (size_t)b * a.width;
    const int u_groups = 1 << (unit_log - 4), u_all = (1 << u_groups) - 1;
    const bool whole = (a.page_size & ((1 << unit_log) - 1)) == 0;   // a unit lies in one page
    const int t_first = (unit0 + u_lo + warp) << unit_log, t_step = kWarps << unit_log;
    const uint8_t* src_head = a.pages + (size_t)kvh * (a.page_size / kKvGroup) * L::kGroupBytes;
    const size_t page_bytes = (size_t)a.kv_heads * (a.page_size / kKvGroup) * L::kGroupBytes;
    // The pages of the groups of `ahead` units are looked up with one load, a lane a group (-1: not there, or not to be
    // read), `ahead` units before the first of them is needed.
    const int ahead = 32 >> (unit_log - 4);
    const int my_group = lane & (u_groups - 1);
    auto look_up = [&](int k0) -> int {
      const int k = k0 + (lane >> (unit_log - 4)), t = t_first + k * t_step + my_group * kKvGroup;
      if (k >= my_n || t > hi_any || t + kKvGroup <= lo_any) return -1;
      const int page = trow[t / a.page_size];
      if (page >= 0 && page < a.num_pages) return page;
      atomicOr(&g_nvfp4_device_error, NVFP4_DEVERR_KV_RANGE);
      return -1;
    };
    int pages_now = look_up(0), pages_next = look_up(ahead);
    int issued = 0;                                     // units whose copies have been started
    // where the lane's group of the next unit lies in its page, advanced without a division
    int g_off = (t_first + my_group * kKvGroup) % a.page_size;
    const int step_off = t_step % a.page_size;
    // Starts the copies of the next unit into ring slot `to`; returns which of its groups come.
    auto issue = [&](uint32_t to) -> uint32_t {
      const int at = issued & (ahead - 1);
      int page = __shfl_sync(0xffffffffu, pages_now, (at << (unit_log - 4)) + my_group);
      if (lane >= u_groups) page = -1;
      const uint32_t have = __ballot_sync(0xffffffffu, page >= 0);
      const bool one = whole && have == (uint32_t)u_all;
      if (lane == 0) mbar_arrive_expect_tx(&bars[to], __popc(have) * L::kGroupBytes);
      __syncwarp();
      if (page >= 0 && (lane == 0 || !one))
        bulk_g2s(ring + to * S::kUnitBytes + lane * L::kGroupBytes,
                 src_head + page * page_bytes + (g_off / kKvGroup) * L::kGroupBytes, one ? u_groups * L::kGroupBytes : L::kGroupBytes,
                 &bars[to]);
      ++issued;
      if (at == ahead - 1) {
        pages_now = pages_next;
        pages_next = look_up(issued + ahead);
      }
      g_off += step_off;
      if (g_off >= a.page_size) g_off -= a.page_size;
      return have;
    };
    // the ring held the last segment's merge: order those accesses before the copies
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    uint32_t coming[S::kStages];                        // groups of the units in flight, oldest first
#pragma unroll
    for (int k = 0; k < S::kStages; ++k) {
      coming[k] = 0;
      if (k < my_n) coming[k] = issue(slot + k < S::kStages ? slot + k : slot + k - S::kStages);
    }

    // ---- the queries (while the first copies fly): FP16 of q / 2^e in operand order, and the factors of the scores
#pragma unroll
    for (int i = 0; i < S::kRows / kWarps; ++i) {
      const int row = warp + i * kWarps;
      float big = 0.0f;
#pragma unroll
      for (int e = 0; e < E; ++e) big = fmaxf(big, fabsf(v[i][e]));
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, o));
      float down, up;
      power_of_two(big, down, up);
      uint8_t* sq = smem + S::kOffQ;
      const int cq = lane >> 3;
      if constexpr (D == 128) {
        *reinterpret_cast<uint2*>(sq + (((row >> 3) * 8 + (lane & 7)) * 32 + (row & 7) * 4 + cq) * 8) =
            make_uint2(pack_f16(v[i][0] * down, v[i][1] * down), pack_f16(v[i][2] * down, v[i][3] * down));
      } else {
        *reinterpret_cast<uint32_t*>(sq + (((row >> 3) * 4 + ((lane & 7) >> 1)) * 32 + (row & 7) * 4 + cq) * 8 +
                                     (lane & 1) * 4) = pack_f16(v[i][0] * down, v[i][1] * down);
      }
      if (lane == 0) s_f[row] = score_factor(a.scale * kLog2e * kg * up);
    }
    __syncthreads();

    WarpState<D, NT> st;
#pragma unroll
    for (int t = 0; t < NT; ++t) {
#pragma unroll
      for (int i = 0; i < D / 16; ++i)
#pragma unroll
        for (int k = 0; k < 4; ++k) st.o[i][t][k] = 0.0f;
      st.m[t][0] = st.m[t][1] = -INFINITY;
      st.l[t][0] = st.l[t][1] = 0.0f;
    }
    uint32_t qreg[NT * (D / 16)][2];
#pragma unroll
    for (int i = 0; i < NT * (D / 16); ++i) {
      const uint2 v = lds64(smem + S::kOffQ + (i * 32 + lane) * 8);
      qreg[i][0] = v.x, qreg[i][1] = v.y;
    }
    float f[NT][2], neg_m[NT][2];                       // factors; minus the maximum, 0 while there is none
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      neg_m[t][0] = neg_m[t][1] = 0.0f;
      f[t][0] = s_f[t * 8 + (lane & 3) * 2];
      f[t][1] = s_f[t * 8 + (lane & 3) * 2 + 1];
    }
    int t_unit = t_first;
    for (int k = 0; k < my_n; ++k, t_unit += t_step) {
      gave_up = !mbar_wait(&bars[slot], phase) || gave_up;
      const uint32_t have = coming[0];
      const uint8_t* unit = ring + slot * S::kUnitBytes;
      for (int gi = 0; gi < u_groups; gi += S::kPair) {
        const uint32_t there = (have >> gi) & ((1u << S::kPair) - 1u);
        if (there == 0u) continue;
        const uint8_t* g = unit + gi * L::kGroupBytes;
        const int t0 = t_unit + gi * kKvGroup;
        float s[S::kPair][NT][4];
#pragma unroll
        for (int h = 0; h < S::kPair; ++h) scores<D, NT>(g + h * L::kGroupBytes, lane, qreg, s[h]);
        int live[S::kPair];
#pragma unroll
        for (int h = 0; h < S::kPair; ++h) live[h] = 4;
        if (t0 + S::kPair * kKvGroup - 1 > hi_all || t0 < lo_all || there != (1u << S::kPair) - 1u) {
#pragma unroll
          for (int h = 0; h < S::kPair; ++h) {
            // token of score row pos = r + 8 i: 4 (r / 2) + 2 i + r % 2; a group that is not there is hidden too
            const int th = t0 + h * kKvGroup;
            const bool gone = !((there >> h) & 1u);
            live[h] = gone ? 0 : min(max(rq.len - th - 4 * (lane & 3), 0), 4);
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const int tok = th + 4 * (lane >> 3) + 2 * (i >> 1) + ((lane >> 2) & 1);
                const int rr = t * 8 + (lane & 3) * 2 + (i & 1);
                const int hi = rq.len - rq.rows + (row0 + rr) / a.group;
                if (gone || tok > hi || (a.window > 0 && tok <= hi - a.window)) s[h][t][i] = -INFINITY;
              }
          }
        }
        // a larger score than any before moves the maximum and rescales what has been summed
        bool grew = false;
        float top[NT][2];
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int k2 = 0; k2 < 2; ++k2) {
            float x = fmaxf(s[0][t][k2], s[0][t][k2 + 2]);
            x = fmaxf(x, fmaxf(s[S::kPair - 1][t][k2], s[S::kPair - 1][t][k2 + 2]));
            top[t][k2] = x * f[t][k2];
            grew = grew || top[t][k2] > st.m[t][k2];
          }
        if (__any_sync(0xffffffffu, grew)) {
#pragma unroll
          for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int k2 = 0; k2 < 2; ++k2) {
              float mx = fmaxf(st.m[t][k2], top[t][k2]);
#pragma unroll
              for (int o = 4; o < 32; o <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
              const float back = mx == -INFINITY ? 1.0f : ex2(st.m[t][k2] - mx);
              st.m[t][k2] = mx;
              neg_m[t][k2] = mx == -INFINITY ? 0.0f : -mx;
              st.l[t][k2] *= back;
#pragma unroll
              for (int i = 0; i < D / 16; ++i) {
                st.o[i][t][k2] *= back;
                st.o[i][t][k2 + 2] *= back;
              }
            }
        }
#pragma unroll
        for (int h = 0; h < S::kPair; ++h) {
          uint32_t p[NT][2];
#pragma unroll
          for (int t = 0; t < NT; ++t) {
            float w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) w[i] = ex2(fmaf(s[h][t][i], f[t][i & 1], neg_m[t][i & 1]));
            st.l[t][0] += w[0] + w[2];
            st.l[t][1] += w[1] + w[3];
            p[t][0] = transpose8x8(pack_f16(w[0], w[1]));
            p[t][1] = transpose8x8(pack_f16(w[2], w[3]));
          }
          weigh<D, NT>(g + h * L::kGroupBytes, lane, p, live[h], st);
        }
      }
      __syncwarp();                                     // the slot has been read
#pragma unroll
      for (int i = 0; i + 1 < S::kStages; ++i) coming[i] = coming[i + 1];
      coming[S::kStages - 1] = 0;
      if (k + S::kStages < my_n && !gave_up) {
        coming[S::kStages - 1] = issue(slot);
      }
      advance();
      if (gave_up) {
        // wait for the copies still in flight, then leave the units that are not loaded
        for (int j = 1; j < S::kStages && k + j < my_n; ++j) {
          mbar_wait(&bars[slot], phase);
          advance();
        }
        break;
      }
    }

    // ---- the four warps together
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int k2 = 0; k2 < 2; ++k2) {
        float l = st.l[t][k2];
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
        if (lane < 4) {
          s_m[warp * S::kRows + t * 8 + lane * 2 + k2] = st.m[t][k2];
          s_l[warp * S::kRows + t * 8 + lane * 2 + k2] = l;
        }
      }
    __syncthreads();
    const bool all = s0 == 0 && s1 == n_seg;
    const int c_first = shares.owner(seg0 + split.head), c_last = shares.owner(seg0 + split.head + n_seg - 1);
    float* rec = a.records + (size_t)(2 * cta + (cta == c_first ? 1 : 0)) * S::kRecord;
#pragma unroll
    for (int t = 0; t < NT; ++t) {
#pragma unroll
      for (int k2 = 0; k2 < 2; ++k2) {
        const int row = t * 8 + (lane & 3) * 2 + k2;
        float mx = -INFINITY;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) mx = fmaxf(mx, s_m[w * S::kRows + row]);
        const float fw = st.m[t][k2] == -INFINITY ? 0.0f : ex2(st.m[t][k2] - mx);
        float* dst = s_merge + (warp * 8 + (lane & 3) * 2 + k2) * S::kMergeStride + (lane >> 2) * (D / 8);
#pragma unroll
        for (int i = 0; i < D / 16; i += 2)
          *reinterpret_cast<float4*>(dst + 2 * i) = make_float4(st.o[i][t][k2] * fw, st.o[i][t][k2 + 2] * fw,
                                                                st.o[i + 1][t][k2] * fw, st.o[i + 1][t][k2 + 2] * fw);
      }
      __syncthreads();
      for (int e = tid; e < 8 * D / 4; e += kThreads) {
        const int row = e / (D / 4), d = e % (D / 4) * 4;
        if (t * 8 + row >= n_rows) continue;
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
        float mx = -INFINITY, l = 0.0f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
          const float4 y = *reinterpret_cast<const float4*>(s_merge + (w * 8 + row) * S::kMergeStride + d);
          x.x += y.x, x.y += y.y, x.z += y.z, x.w += y.w;
          mx = fmaxf(mx, s_m[w * S::kRows + t * 8 + row]);
        }
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
          const float mw = s_m[w * S::kRows + t * 8 + row];
          l += s_l[w * S::kRows + t * 8 + row] * (mw == -INFINITY ? 1.0f : ex2(mw - mx));   // (0 or NaN without a maximum)
        }
        if (all) {
          const int rr = row0 + t * 8 + row, tok = rq.first + rr / a.group, h = kvh * a.group + rr % a.group;
          const float inv = l == 0.0f ? 0.0f : vg / l;
          const __nv_bfloat162 lo = __floats2bfloat162_rn(x.x * inv, x.y * inv), hi = __floats2bfloat162_rn(x.z * inv, x.w * inv);
          *reinterpret_cast<uint2*>(a.out + ((size_t)tok * a.heads + h) * D + d) =
              make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
          if (a.lse && d == 0) a.lse[(size_t)tok * a.heads + h] = l == 0.0f ? -INFINITY : (mx + log2f(l)) / kLog2e;
        } else {
          __stcg(reinterpret_cast<float4*>(rec + (t * 8 + row) * D + d), x);
          if (d == 0) {
            __stcg(rec + S::kRows * D + t * 8 + row, mx);
            __stcg(rec + S::kRows * (D + 1) + t * 8 + row, l);
          }
        }
      }
      __syncthreads();
    }

    // ---- a segment that several CTAs share: the last one to arrive merges the records
    if (!all) {
      __threadfence();
      __syncthreads();
      unsigned int* flag = reinterpret_cast<unsigned int*>(smem + S::kOffScan + 124);
      if (tid == 0) *flag = atomicAdd(&a.counters[c_first], 1u);
      __syncthreads();
      if (*flag == (unsigned)(c_last - c_first)) {
        __threadfence();
        for (int e = tid; e < n_rows * (D / 4); e += kThreads) {
          const int row = e / (D / 4), d = e % (D / 4) * 4;
          float mx = -INFINITY, l = 0.0f;
          float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
          constexpr int kBatch = 8;                     // records whose loads are in flight together
          for (int q0 = c_first; q0 <= c_last; q0 += kBatch) {
            float m[kBatch], lq[kBatch];
            float4 y[kBatch];
#pragma unroll
            for (int j = 0; j < kBatch; ++j) {
              const int q = min(q0 + j, c_last);
              const float* r = a.records + (size_t)(2 * q + (q == c_first ? 1 : 0)) * S::kRecord;
              m[j] = __ldcg(r + S::kRows * D + row);
              lq[j] = __ldcg(r + S::kRows * (D + 1) + row);
              y[j] = __ldcg(reinterpret_cast<const float4*>(r + row * D + d));
            }
#pragma unroll
            for (int j = 0; j < kBatch; ++j) {
              if (q0 + j > c_last || no_keys(m[j], lq[j])) continue;
              const float mn = fmaxf(mx, m[j]), back = ex2(mx - mn), w = ex2(m[j] - mn);
              mx = mn;
              l = fmaf(lq[j], w, l * back);
              x.x = fmaf(y[j].x, w, x.x * back), x.y = fmaf(y[j].y, w, x.y * back);
              x.z = fmaf(y[j].z, w, x.z * back), x.w = fmaf(y[j].w, w, x.w * back);
            }
          }
          const int rr = row0 + row, tok = rq.first + rr / a.group, h = kvh * a.group + rr % a.group;
          const float inv = l == 0.0f ? 0.0f : vg / l;
          const __nv_bfloat162 lo = __floats2bfloat162_rn(x.x * inv, x.y * inv), hi = __floats2bfloat162_rn(x.z * inv, x.w * inv);
          *reinterpret_cast<uint2*>(a.out + ((size_t)tok * a.heads + h) * D + d) =
              make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
          if (a.lse && d == 0) a.lse[(size_t)tok * a.heads + h] = l == 0.0f ? -INFINITY : (mx + log2f(l)) / kLog2e;
        }
        if (tid == 0) a.counters[c_first] = 0u;
      }
      __syncthreads();
    }
  }
}


// CTAs of a variant: as many as are resident at once.
template <int D, int NT, class T>
cudaError_t launch(const AttnArgs& a, cudaStream_t stream) {
  using S = Shape<D, NT>;
  static PerDeviceInt grid_cache;
  cudaError_t err = cudaSuccess;
  const int grid = grid_cache.get([](int dev, cudaError_t* e_out) -> int {
    int sms = 0, per = 0;
    cudaError_t e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e == cudaSuccess)
      e = cudaFuncSetAttribute(kv_attention_kernel<D, NT, T>, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmem);
    if (e == cudaSuccess)
      e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per, kv_attention_kernel<D, NT, T>, kThreads, S::kSmem);
    if (e != cudaSuccess) {
      *e_out = e;
      return 0;
    }
    const int g = sms * (per > 0 ? per : 1);
    return g < kMaxCtas ? g : kMaxCtas;
  }, &err);
  if (grid == 0) return err;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = S::kSmem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kv_attention_kernel<D, NT, T>, a);
}

// Tiles of 8 query rows or of 16 (`keys`: kv heads x keys there is room for).  More rows share a dequantized key, but a
// tile has fewer CTAs at work at a time (two an SM instead of three) and takes longer to set up and merge: with D = 128
// and 8 kv heads, us with 8 / 16:  16 rows: 13 / 16 (2000 keys), 50 / 53 (16 requests of 8000);  32 rows: 14 / 17,
// 20 / 25 (8000 keys), 36 / 34 (4 of 8000), 110 / 88 (16 of 8000);  48 rows: 22 / 24, 39 / 37, 123 / 106.  Tiles of 32
// rows gained 3 % at the largest of these and took up to twice as long at the others.
constexpr long long kSmallKeys = 1 << 18;

template <int D, class T>
cudaError_t dispatch(const AttnArgs& a, int rows, long long keys, cudaStream_t stream) {
  return rows <= 16 || keys <= kSmallKeys ? launch<D, 1, T>(a, stream) : launch<D, 2, T>(a, stream);
}

// Whether a workspace has the many-row kernel's records: calls of fewer rows hardly reach it.
bool room_for_pieces(int tokens, int group) { return (long long)tokens * group > kTcRows; }

}  // namespace

nvfp4_status nvfp4_internal_cuda_status(cudaError_t e);
bool nvfp4_internal_aligned(const void* p, size_t a);
nvfp4_status nvfp4_internal_check_device();

extern "C" size_t nvfp4_kv_attention_workspace_bytes(int batch, int tokens, int heads, int kv_heads, int head_dim) {
  if (batch < 1 || tokens < 0 || nvfp4_kv_page_bytes(16, kv_heads, head_dim) == 0) return 0;
  if (heads < kv_heads || heads % kv_heads != 0 || heads / kv_heads > 64) return 0;
  const size_t decode = (size_t)2 * kMaxCtas * Shape<128, 2>::kRecord, many = (size_t)kTcPieces * kTcRecord;
  return kCounterBytes + (room_for_pieces(tokens, heads / kv_heads) && many > decode ? many : decode) * sizeof(float);
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
  if ((long long)batch * table_width > 0x7FFFFFFFll || (long long)tokens * heads > 0x7FFFFFFFll ||
      (long long)table_width * cache->page_size > 0x7FFFFFFFll)
    return NVFP4_ERR_SHAPE;
  if (tokens == 0 || batch == 0) return NVFP4_OK;
  if (!q || !block_table || !kv_lens || !out || !workspace) return NVFP4_ERR_NULL;
  const int per = dtype == NVFP4_DTYPE_F32 ? 4 : 8;
  if ((tokens > 1 && q_token_stride % per) || (heads > 1 && q_head_stride % per)) return NVFP4_ERR_ALIGN;
  if (!nvfp4_internal_aligned(q, 16) || !nvfp4_internal_aligned(out, 16) || !nvfp4_internal_aligned(workspace, 256))
    return NVFP4_ERR_ALIGN;
  for (const void* p : {(const void*)block_table, (const void*)kv_lens, (const void*)cu_q, (const void*)lse})
    if (!nvfp4_internal_aligned(p, 4)) return NVFP4_ERR_ALIGN;
  if (workspace_bytes < nvfp4_kv_attention_workspace_bytes(batch, tokens, heads, cache->kv_heads, cache->head_dim))
    return NVFP4_ERR_SHAPE;
  const nvfp4_status ds = nvfp4_internal_check_device();
  if (ds != NVFP4_OK) return ds;
  const int group = heads / cache->kv_heads;
  if (window >= table_width * cache->page_size) window = 0;   // no request is longer: nothing to hide
  const AttnArgs a = {q, q_token_stride, q_head_stride, cache->pages, cache->k_global, cache->v_global,
                      block_table, kv_lens, cu_q, out, lse, static_cast<unsigned int*>(workspace),
                      reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + kCounterBytes), tokens, heads,
                      cache->kv_heads, group, cache->page_size, cache->num_pages, table_width, batch, window,
                      room_for_pieces(tokens, group) ? kTcPieces : 0, scale};
  const int rows = cu_q ? (int)((long long)max_q * group < 1 << 20 ? max_q * group : 1 << 20) : group;
  // the decode kernel counts its units (32 keys of a row tile, with their overhead) in 31 bits; this is the most there
  // can be, whatever kv_lens hold, with row ranges that do not overlap (the kernel looks)
  const long long keys = (long long)batch * cache->kv_heads * table_width * cache->page_size;
  const long long most_units = ((long long)tokens * group / 8 + batch) * cache->kv_heads *
                               ((long long)table_width * cache->page_size / 32 + 2 + kSegmentCost / 32 + kWarps);
  cudaError_t e;
  const long long segment_keys = (long long)batch * cache->kv_heads * kSegmentCost;
  if ((rows > kTcRows && rows * (keys + segment_keys) > kTcProducts) || most_units > 0x7F000000ll)
    e = nvfp4_internal_kv_attention_tc(a, cache->head_dim, dtype, stream);
  else if (cache->head_dim == 128)
    e = dtype == NVFP4_DTYPE_F32 ? dispatch<128, float>(a, rows, keys, stream) : dispatch<128, uint16_t>(a, rows, keys, stream);
  else
    e = dtype == NVFP4_DTYPE_F32 ? dispatch<64, float>(a, rows, keys, stream) : dispatch<64, uint16_t>(a, rows, keys, stream);
  return nvfp4_internal_cuda_status(e);
}
