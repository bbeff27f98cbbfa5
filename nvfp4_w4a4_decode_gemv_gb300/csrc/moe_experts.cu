// The chosen experts' NVFP4 products (tcgen05, sm_103a), on a plan of the pairs by expert:
//   gate_up  h[p, i] = BF16(SiLU(g) u),  g = xg wg[e] x[t(p)] . w[e, gate row i],  u the same with up row i
//   down     y[t, n] = sum_j weight[t, j] hg wg[e] h[place(t, j)] . w[e, n]
//
// As in the projections, 128 weight rows are the wide side of the MMA (kind::mxf4nvf4) and an expert's rows of x its narrow
// side, N chosen at run time: the work of a tile is the bytes of its weights however few rows the expert got.
//
// Weights are packed (nvfp4_moe_pack_weights) in blocks of 128 rows x 256 K, one bulk copy each; a block's scales stand as
// tcgen05.cp wants them, so that they go from the block to TMEM without a thread's help.  Rows of gate and up alternate: a
// TMEM lane and its neighbour hold both halves of an h.
//
// Three modes:
//   UP    items (expert, row tile, up to NT of its pairs) dealt out to the CTAs in turn; with fewer items than SMs a cluster
//         splits an item's K and adds the parts over distributed shared memory.
//   SUM   (down, few tokens) a cluster takes a tile of y's columns and shares out all the experts' K for it: every token's sum
//         over its experts stays in shared memory and meets the other CTAs' there.  No workspace, one launch.
//   PART  (down, many tokens) items as in UP; products go to a workspace, and a second kernel adds a token's products with
//         its weights.
// No CTA waits for another but at cluster barriers, and no state is left behind.
//
// Measured (128 experts where not said; in brackets the share of the time that the bytes a call cannot do without would take
// at the copy rate, 6.76 TB/s):
//   up, few places an expert   1 token of 8, K 4096, 2048 rows: 10.5 us, 8.9 in a graph (53 %): a launch, the experts' table
//                              (1.7 us) and the ramp of the copies; 8 tokens of 8, K 5120, 1536 rows: 36 us (86 %);
//                              33 tokens of 2 of 8 experts, K 4096, 16384 rows: 48.6 us (92 %)
//   up, many                   2048 tokens of 8, K 4096, 1536 rows: 134 us (1.54 PFLOP/s; 53 %); without its loads and
//                              stores 103, 15 to 20 of them for laying the rows out; with one MMA a stage in place of four 74.
//                              Stages of 400 to 700 cycles add up to 35 to 65
//   down, few tokens           1 token of 8, K 1024, 4096 rows: 8.2 us (34 %); 64 tokens of 8, K 768, 5120 rows: 54 us
//                              (71 %), on the 120 SMs that 40 row tiles of 3 CTAs fill.  N 256, 1024, 2880, 7168, 9856: 23,
//                              25, 33, 78, 141 us on 16, 64, 138, 112, 77 SMs
//   down, many                 2048 tokens of 8, K 768, 4096 rows: 154 us (26 %): 268 MB of FP32 products written and read
//                              again; without the writes 124
#include <cuda.h>
#include <cudaTypedefs.h>
#include <string.h>

#include "common.cuh"
#include "tcgen05.cuh"

NVFP4_DEFINE_ERROR_READER(nvfp4_internal_read_error_moe_experts)

namespace {

constexpr int kTR = 128;                     // weight rows of a tile: MMA M
constexpr int kChunk = 256;                  // K of a stage
constexpr int kWCodes = kTR * 128;           // 16384
constexpr int kBlock = kWCodes + kTR * 16;   // 18432
constexpr int kXBlock = 2048;                // scales of 128 places and a chunk, as tcgen05.cp takes them
constexpr int kMaxExperts = 512;
constexpr int kMaxTop = 32;
constexpr int kMaxCluster = 8;
constexpr uint32_t kTmemCols = 512;

// The experts that have pairs, as a kernel keeps them: first places, counts, tiles of NT and of 128 places before, experts;
// sums.  The offsets as given stand elsewhere while the table is built.
constexpr int kTableBytes = kMaxExperts * (4 * 4 + 2) + 16;
constexpr int kOffsetsBytes = (kMaxExperts + 1) * 4;

enum Mode { UP, SUM, PART };

// NT places to a tile, in halves of 128 at most.  FEW: rows of x by asynchronous copies of the loader warps, and sums of y
// in shared memory with SUM; else by TMA from rows in the order of the plan.
template <int NT, int MODE, bool FEW>
struct Shape {
  static constexpr int kHalves = NT > 128 ? 2 : 1;
  static constexpr int kHalf = NT > 128 ? 128 : NT;                   // columns of an accumulator buffer
  static constexpr int kOffX = kBlock;
  static constexpr int kOffXS = kOffX + NT * 128;
  static constexpr int kSlot = kOffXS + kHalves * kXBlock;
  static constexpr int kSums = MODE == SUM ? NT * kTR * 4 : 0;        // y of up to NT tokens
  static constexpr int kStages = FEW ? (MODE == SUM ? 6 : 7) : 4;
  static constexpr uint32_t kColSF = 2u * kHalf;                      // first scale column, behind two buffers
  static constexpr uint32_t kSFStage = 16u + 16u * kHalves;           // weights' 4 x 4, tokens' 4 x 4 a half
  static constexpr int kOffSums = kStages * kSlot;
  static constexpr int kOffTables = kOffSums + kSums;
  static constexpr int kOffBars = kOffTables + kTableBytes;
  static constexpr size_t kBytes = 1024 + kOffBars + (2 * kStages + 4) * 8 + 16;
  static_assert(kColSF + kSFStage * kStages <= kTmemCols, "scale columns must fit the TMEM allocation");
  static_assert(kBytes <= 227 * 1024 && kSlot % 1024 == 0 && kOffX % 1024 == 0, "shared memory");
};

struct ExpertArgs {
  const uint8_t *xc, *xs;                    // rows of x: codes [.., K/2], scales [.., K/16]
  const uint8_t* x_blocks;                   // !FEW: scales in kXBlock blocks [tile of 128 places][C]
  const float* xg;
  const uint8_t* w;                          // [experts][RT][C] blocks
  const float* wg;                           // [experts]
  const int32_t *offsets, *pairs;
  const float* weights;                      // SUM
  uint16_t* h;                               // UP: [n_pairs, inter]
  float* out;                                // SUM: y [tokens, N]; PART: [rts][n_pairs][kTR]
  int tokens, top, experts, N, K, C, RT;     // N: columns of y, or of h
  int rt0, rts;                              // row tiles of the call
  int n_pairs;
  int cluster;
};

// A stretch of K of one tile: what a pass of the ring's roles works on.
struct Segment {
  int e, p0, n, rt, c0, nc;                  // expert, first place, places, row tile, first chunk, chunks
  int block;                                 // first tile of 128 places
};

// The experts that have pairs, in order.
struct Table {
  int *first, *count, *tiles_before, *blocks, *offsets;  // tiles of up to NT places, and of 128, of the experts before
  int* sums;
  uint16_t* expert;
  int used, total, tiles;                                // entries; pairs; tiles of up to NT places
  NVFP4_DEVINL Table(uint8_t* mem, uint8_t* scratch) {   // kTableBytes, and kOffsetsBytes until it is built; 16-byte aligned
    first = reinterpret_cast<int*>(mem);
    count = first + kMaxExperts;
    tiles_before = count + kMaxExperts;
    blocks = tiles_before + kMaxExperts;
    sums = blocks + kMaxExperts;                         // 4
    expert = reinterpret_cast<uint16_t*>(sums + 4);
    offsets = reinterpret_cast<int*>(scratch);
  }
};

// Built by the whole CTA; ends with a __syncthreads.  HEAVY: experts of more than 128 places come first, so that items dealt
// out in turn cost about the same (a stage of more than 128 places takes twice the MMAs).
template <int NT, bool HEAVY>
NVFP4_DEVINL void build_table(const ExpertArgs& a, Table& tb) {
  for (int i = threadIdx.x; i <= a.experts; i += blockDim.x) tb.offsets[i] = __ldcg(a.offsets + i);
  __syncthreads();
  if (threadIdx.x < 32) {
    // a lane looks at `per` experts that follow one another
    const int lane = threadIdx.x, per = (a.experts + 31) / 32;
    int used[2] = {0, 0}, tiles[2] = {0, 0}, blocks = 0;      // [0]: of heavy experts
    bool bad = false;
    auto look = [&](auto take) {
      for (int i = 0; i < per; ++i) {
        const int e = lane * per + i;
        if (e >= a.experts) break;
        const int f = tb.offsets[e], l = tb.offsets[e + 1];
        const int lo = min(max(f, 0), a.n_pairs), hi = min(max(l, 0), a.n_pairs);
        bad = bad || f != lo || l != hi || hi < lo || (e == 0 && f != 0);
        if (hi > lo) take(e, lo, hi - lo, HEAVY && hi - lo <= 128);
      }
    };
    look([&](int, int, int n, bool light) {
      const int t = (n + NT - 1) / NT;
      used[0] += light ? 0 : 1;
      used[1] += light ? 1 : 0;
      tiles[0] += light ? 0 : t;
      tiles[1] += light ? t : 0;
      blocks += (n + 127) / 128;
    });
    // Ranges that fall or leave the pairs have more tiles between them than the workspace and the grid are made for: no pairs.
    // A first place that is no one's would be left as it is: no pairs either.
    bad = __any_sync(0xffffffffu, bad);
    if (bad) used[0] = used[1] = tiles[0] = tiles[1] = blocks = 0;
    int at[5] = {used[0], used[1], tiles[0], tiles[1], blocks};
#pragma unroll
    for (int o = 1; o < 32; o <<= 1)
#pragma unroll
      for (int i = 0; i < 5; ++i) {
        if (!HEAVY && (i == 1 || i == 3)) continue;
        const int x = __shfl_up_sync(0xffffffffu, at[i], o);
        if (lane >= o) at[i] += x;
      }
    const int heavy = __shfl_sync(0xffffffffu, at[0], 31), heavy_tiles = __shfl_sync(0xffffffffu, at[2], 31);
    if (lane == 31) {
      tb.sums[0] = heavy_tiles + at[3];
      tb.sums[1] = heavy + at[1];
      tb.sums[2] = bad ? 0 : tb.offsets[a.experts];
    }
    at[0] -= used[0];
    at[1] += heavy - used[1];
    at[2] -= tiles[0];
    at[3] += heavy_tiles - tiles[1];
    at[4] -= blocks;
    if (!bad) look([&](int e, int lo, int n, bool light) {
      const int i = light ? at[1] : at[0], t = (n + NT - 1) / NT;
      tb.first[i] = lo;
      tb.count[i] = n;
      tb.blocks[i] = at[4];
      tb.tiles_before[i] = light ? at[3] : at[2];
      tb.expert[i] = (uint16_t)e;
      at[0] += light ? 0 : 1;
      at[1] += light ? 1 : 0;
      at[2] += light ? 0 : t;
      at[3] += light ? t : 0;
      at[4] += (n + 127) / 128;
    });
    if (bad && lane == 0 && blockIdx.x == 0) atomicOr(&g_nvfp4_device_error, NVFP4_DEVERR_MOE_RANGE);
  }
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");   // (the ring's copies may come where the offsets stood)
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  tb.tiles = tb.sums[0];
  tb.used = tb.sums[1];
  tb.total = tb.sums[2];
}

// Every role's warp walks the CTA's segments by itself, in the same order.  UP, PART: its lanes look up the next 32 items, one
// each, and hand them out one by one (looked up when they were wanted, by the warp together, each took 700 cycles, as long as
// a stage).
template <int NT, int MODE>
struct Walk {
  const Table& tb;
  const ExpertArgs& a;
  int it, end;                               // UP, PART: item; SUM: unit (tile of places, chunk)
  int used, tile;                            // SUM: the entry and its tile that `it` stands in, -1: to be looked up
  int rank, step;
  int c0, nc;                                // UP, PART: the rank's chunks
  Segment mine;                              // UP, PART: the lane's of the 32 items, and how many of them are handed out
  int handed;
  NVFP4_DEVINL Walk(const Table& t, const ExpertArgs& args) : tb(t), a(args), used(-1), tile(0), handed(32) {
    rank = args.cluster > 1 ? (int)cluster_ctarank() : 0;
    if (MODE == SUM) {
      const long long units = (long long)t.tiles * a.C;
      it = (int)(units * rank / a.cluster);
      end = (int)(units * (rank + 1) / a.cluster);
      step = 0;
    } else {
      it = blockIdx.x / a.cluster;
      end = t.tiles * a.rts;
      step = gridDim.x / a.cluster;
      c0 = a.C * rank / a.cluster;
      nc = a.C * (rank + 1) / a.cluster - c0;
    }
  }
  // The last entry whose tiles begin at x or before, by a whole warp.
  NVFP4_DEVINL int entry_of(int x) const {
    const int lane = threadIdx.x & 31, per = (tb.used + 31) / 32, at = lane * per;
    const int piece = __popc(__ballot_sync(0xffffffffu, at < tb.used && tb.tiles_before[at] <= x)) - 1;
    const int i = piece * per + lane;
    return piece * per + __popc(__ballot_sync(0xffffffffu, lane < per && i < tb.used && tb.tiles_before[i] <= x)) - 1;
  }
  NVFP4_DEVINL void place(Segment& s, int u, int t) const {   // tile t of entry u
    s.e = tb.expert[u];
    s.p0 = tb.first[u] + t * NT;
    s.n = min(NT, tb.count[u] - t * NT);
    s.block = tb.blocks[u] + t * (NT / 128);
  }
  NVFP4_DEVINL void look_up(int item) {
    int u = 0;                               // the last entry whose items begin at `item` or before
    for (int hi = tb.used; hi - u > 1;) {
      const int mid = (u + hi) >> 1;
      if (tb.tiles_before[mid] * a.rts <= item) u = mid; else hi = mid;
    }
    const int in = item - tb.tiles_before[u] * a.rts, tt = (tb.count[u] + NT - 1) / NT;
    mine.rt = tt == 1 ? in : in / tt;        // an expert's items: the tiles of places of a row tile follow one another
    place(mine, u, in - mine.rt * tt);
    mine.rt += a.rt0;
  }
  // By a whole warp.
  NVFP4_DEVINL bool next(Segment& s) {
    if (it >= end) return false;
    if (MODE == SUM) {
      if (used < 0) {
        const int at = it / a.C;
        used = entry_of(at);
        tile = at - tb.tiles_before[used];
        s.c0 = it - at * a.C;
      } else {
        s.c0 = 0;
        if (++tile == (tb.count[used] + NT - 1) / NT) {
          tile = 0;
          ++used;
        }
      }
      place(s, used, tile);
      s.rt = blockIdx.x / a.cluster;
      s.nc = min(a.C - s.c0, end - it);
      it += s.nc;
    } else {
      if (handed == 32) {
        const int lane = threadIdx.x & 31;
        if ((long long)lane * step < end - it) look_up(it + lane * step);
        handed = 0;
        __syncwarp();
      }
      s.e = __shfl_sync(0xffffffffu, mine.e, handed);
      s.p0 = __shfl_sync(0xffffffffu, mine.p0, handed);
      s.n = __shfl_sync(0xffffffffu, mine.n, handed);
      s.rt = __shfl_sync(0xffffffffu, mine.rt, handed);
      s.block = __shfl_sync(0xffffffffu, mine.block, handed);
      s.c0 = c0;
      s.nc = nc;
      ++handed;
      it = step < end - it ? it + step : end;
    }
    return true;
  }
};

// Which of the two accumulator buffers a segment takes: one in turn, or both (more than 128 places), and how often each has
// been taken; a role counts along.
struct Buffers {
  uint32_t uses0 = 0u, uses1 = 0u;
  int turn = 0;
  NVFP4_DEVINL int first(bool both) const { return both ? 0 : turn; }
  NVFP4_DEVINL uint32_t uses(int buf) const { return buf ? uses1 : uses0; }
  NVFP4_DEVINL void took(bool both) {
    uses0 += both || turn == 0;
    uses1 += both || turn == 1;
    if (!both) turn ^= 1;
  }
};

// One look, without waiting.
NVFP4_DEVINL bool mbar_test_wait(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}

// 32 rows of 16 bytes, one behind the other, to 4 columns of every lane quadrant: word w of row i to lane i, column w.
NVFP4_DEVINL void copy_scales(uint32_t tmem, uint64_t desc) {
  asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(tmem), "l"(desc) : "memory");
}
// Rows of 16 bytes without a swizzle: groups of 8 rows 128 bytes apart.
NVFP4_DEVINL uint64_t smem_desc_rows16(uint32_t saddr) {
  return (uint64_t)((saddr & 0x3FFFFu) >> 4) | ((uint64_t)(128 >> 4) << 16) | ((uint64_t)(128 >> 4) << 32) |
         ((uint64_t)1 << 46);
}

// E2M1 x E2M1, UE4M3 scales, K-major operands, M = 128 and N = n rounded up to 16, 32, 64, 128, 192 or 256 (an MMA takes 64
// cycles whatever its N up to 128).
NVFP4_DEVINL uint32_t idesc_for(int n) {
  const uint32_t eighths = n <= 16 ? 2u : n <= 32 ? 4u : n <= 64 ? 8u : n <= 128 ? 16u : n <= 192 ? 24u : 32u;
  return (1u << 7) | (1u << 10) | (eighths << 17) | ((uint32_t)(kTR >> 4) << 24);
}

NVFP4_DEVINL void async_copy16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
NVFP4_DEVINL void async_copy4(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
NVFP4_DEVINL void async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
NVFP4_DEVINL void async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
NVFP4_DEVINL float ld_dsmem_f32(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}
NVFP4_DEVINL float4 ld_dsmem_f32x4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}

// g / (1 + e^-g) u of g4 = g / 4.  An approximate power (off by 2^-22, its argument by 1.25 2^-24 |g|) and quotient (2^-22):
// 2^-16 of the result, far below the 2^-8 of its BF16.  Both sides of the quotient are a quarter: __fdividef gives 0 for a
// divisor above 2^126, which 1 + e^-g reaches at g = -87.3.  Below g = -88.72 e^-g overflows and the result is 0.
NVFP4_DEVINL float silu_mul(float g4, float u) {
  return __fdividef(g4, 0.25f + ex2(fmaf(g4, -5.77078016f, -2.0f))) * u;    // e^-g / 4 = 2^(-4 log2(e) g4 - 2)
}

// 16 columns of the accumulator, even lanes gates and odd lanes ups, to h: 16 bytes a lane, 8 values of one place.
// Halves of what a lane holds go to the lane whose bit differs, bit by bit: first gates meet ups, then lanes 2, 4 and 8
// apart trade places for values of h.
NVFP4_DEVINL void store_h16(const ExpertArgs& a, const Segment& sg, int quad, int m0, const float (&v)[16], float scale) {
  const int lane = threadIdx.x & 31;
  const bool odd = lane & 1, b1 = lane & 2, b2 = lane & 4, b3 = lane & 8;
  const float f = odd ? scale : 0.25f * scale;
  float h[8];                                // place 2 j + odd
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float a0 = v[2 * j] * f, a1 = v[2 * j + 1] * f;
    const float other = __shfl_xor_sync(0xffffffffu, odd ? a0 : a1, 1);
    h[j] = odd ? silu_mul(other, a1) : silu_mul(a0, other);
  }
  uint32_t w[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float keep = b1 ? h[2 * j + 1] : h[2 * j];
    const float other = __shfl_xor_sync(0xffffffffu, b1 ? h[2 * j] : h[2 * j + 1], 2);
    const __nv_bfloat162 p = __floats2bfloat162_rn(b1 ? other : keep, b1 ? keep : other);
    w[j] = *reinterpret_cast<const uint32_t*>(&p);
  }
  uint32_t x[2][2];
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const uint32_t keep = b2 ? w[2 * j + 1] : w[2 * j];
    const uint32_t other = __shfl_xor_sync(0xffffffffu, b2 ? w[2 * j] : w[2 * j + 1], 4);
    x[j][0] = b2 ? other : keep;
    x[j][1] = b2 ? keep : other;
  }
  uint32_t o[2];
#pragma unroll
  for (int j = 0; j < 2; ++j) o[j] = __shfl_xor_sync(0xffffffffu, b3 ? x[0][j] : x[1][j], 8);
  const uint4 out = b3 ? make_uint4(o[0], o[1], x[1][0], x[1][1]) : make_uint4(x[0][0], x[0][1], o[0], o[1]);
  const int m = m0 + 2 * ((lane >> 1) & 7) + (lane & 1), i = sg.rt * 64 + quad * 16 + 8 * (lane >> 4);
  if (m < sg.n) *reinterpret_cast<uint4*>(a.h + (size_t)(sg.p0 + m) * a.N + i) = out;
}

// The parts of a kernel that all roles need.
template <int NT, int MODE, bool FEW>
struct Smem {
  using S = Shape<NT, MODE, FEW>;
  uint8_t* base;
  uint64_t *full, *empty, *acc_full, *acc_empty;
  uint32_t* tmem_slot;
  float* sums;
  NVFP4_DEVINL explicit Smem(uint8_t* raw) {
    base = raw + ((1024u - (smem_u32(raw) & 1023u)) & 1023u);
    sums = reinterpret_cast<float*>(base + S::kOffSums);
    full = reinterpret_cast<uint64_t*>(base + S::kOffBars);
    empty = full + S::kStages;
    acc_full = empty + S::kStages;
    acc_empty = acc_full + 2;
    tmem_slot = reinterpret_cast<uint32_t*>(acc_empty + 2);
  }
  NVFP4_DEVINL Table table() const { return Table(base + S::kOffTables, base); }
  // By the first thread; `arrivals`: on a stage, `readers`: warps that read an accumulator.
  NVFP4_DEVINL void init_barriers(int arrivals, int readers) const {
    for (int s = 0; s < S::kStages; ++s) {
      mbar_init(&full[s], arrivals);
      mbar_init(&empty[s], 1);
    }
    for (int d = 0; d < 2; ++d) {
      mbar_init(&acc_full[d], 1);
      mbar_init(&acc_empty[d], readers);
    }
    fence_mbar_init();
  }
  // By warp 1.
  NVFP4_DEVINL void alloc_tmem() const {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)),
                 "r"(kTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  static NVFP4_DEVINL void free_tmem(uint32_t tmem) {
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols));
  }
};

// Stages of a CTA's segments that one lane of a warp fills: fill(sg, c, slot, bar) for each, once its last use is over.
template <int NT, int MODE, bool FEW, class F>
NVFP4_DEVINL void fill_stages(const Smem<NT, MODE, FEW>& sm, Walk<NT, MODE> walk, const F& fill) {
  using S = Shape<NT, MODE, FEW>;
  constexpr int kS = S::kStages;
  Segment sg;
  int s = 0, k = 0, ok = 1;
  uint32_t phase = 0;
  while (ok && walk.next(sg)) {
    if ((threadIdx.x & 31) == 0) {
      for (int c = sg.c0; c < sg.c0 + sg.nc; ++c) {
        if (k >= kS && !mbar_wait(&sm.empty[s], phase ^ 1u)) {
          ok = 0;
          break;
        }
        fill(sg, c, sm.base + s * S::kSlot, &sm.full[s]);
        ++k;
        if (++s == kS) { s = 0; phase ^= 1u; }
      }
    }
    ok = __shfl_sync(0xffffffffu, ok, 0);
  }
  // Not to leave with copies in flight: the last ones' waits (bounded; on the normal path long over).
  if ((threadIdx.x & 31) == 0)
    for (int j = k > kS ? k - kS : 0; j < k; ++j) mbar_wait(&sm.full[j % kS], (j / kS) & 1);
  __syncwarp();
}

template <int NT, int MODE, bool FEW>
NVFP4_DEVINL void copy_weights(const Smem<NT, MODE, FEW>& sm, const ExpertArgs& a, const Walk<NT, MODE>& walk) {
  fill_stages(sm, walk, [&](const Segment& sg, int c, uint8_t* slot, uint64_t* bar) {
    mbar_arrive_expect_tx(bar, kBlock);
    bulk_g2s(slot, a.w + (((size_t)sg.e * a.RT + sg.rt) * a.C + c) * kBlock, kBlock, bar);
  });
}

// Scales to TMEM and products, by one warp: it looks a segment up and waits for its accumulator together; one lane then takes
// all of the segment's stages, with the others held until it is through.  (Instructions predicated lane by lane, with the
// other lanes free to run ahead, faulted once several stages were ready: operands are in uniform registers, which the lanes
// that run ahead overwrite.  A vote and a branch for each stage cost 2 % more than one for a segment.)  The next stage's
// barrier is looked at before a stage's instructions are issued: behind them, the look would wait until the tensor core has
// taken them (300 cycles).
template <int NT, int MODE, bool FEW>
NVFP4_DEVINL void multiply(const Smem<NT, MODE, FEW>& sm, const ExpertArgs& a, Walk<NT, MODE> walk, uint32_t tmem) {
  using S = Shape<NT, MODE, FEW>;
  constexpr int kS = S::kStages;
  const bool lead = elect_one() != 0u;
  // operands of the first stage; another stage's are an addition to the address field
  const uint64_t da0 = smem_desc_sw128(smem_u32(sm.base)), db0 = smem_desc_sw128(smem_u32(sm.base + S::kOffX));
  const uint64_t dwa0 = smem_desc_rows16(smem_u32(sm.base + kWCodes)), dxa0 = smem_desc_rows16(smem_u32(sm.base + S::kOffXS));
  Segment sg;
  Buffers bufs;
  int s = 0, k = 0;                          // of the lane that issues
  uint32_t phase = 0;
  bool ok = true, ready = false;
  while (ok && walk.next(sg)) {
    const bool both = S::kHalves == 2 && sg.n > 128;
    const int buf = bufs.first(both);
    if (bufs.uses(buf) > 0 && !mbar_wait_warp(&sm.acc_empty[buf], (bufs.uses(buf) - 1) & 1)) break;
    if (both && bufs.uses1 > 0 && !mbar_wait_warp(&sm.acc_empty[1], (bufs.uses1 - 1) & 1)) break;
    bufs.took(both);
    const uint32_t idesc = idesc_for(sg.n), d = tmem + (uint32_t)(buf * S::kHalf);
    int good = 1;
    if (lead) {
      for (int c = 0; c < sg.nc; ++c) {
        if (!ready && !mbar_wait(&sm.full[s], phase)) {
          good = 0;
          break;
        }
        const int next = s + 1 == kS ? 0 : s + 1;
        const uint32_t next_phase = next == 0 ? phase ^ 1u : phase;
        ready = mbar_test_wait(&sm.full[next], next_phase);
        tc_fence_after();
        const uint64_t at = (uint64_t)(s * (S::kSlot >> 4));
        const uint64_t da = da0 + at, db = db0 + at, dwa = dwa0 + at, dxa = dxa0 + at;
        const uint32_t sfa = tmem + S::kColSF + S::kSFStage * (uint32_t)s, sfb = sfa + 16u;
        const int mmas = min(4, (a.K - (sg.c0 + c) * kChunk) / 64);
#pragma unroll
        for (int q = 0; q < 4; ++q)
          if (q < mmas) {
            copy_scales(sfa + 4u * q, dwa + (uint64_t)(32 * q));
            copy_scales(sfb + 4u * S::kHalves * q, dxa + (uint64_t)(32 * q));
            if (both) copy_scales(sfb + 8u * q + 4u, dxa + (uint64_t)(128 + 32 * q));
          }
#pragma unroll
        for (int q = 0; q < 4; ++q)
          if (q < mmas) {
            const uint32_t acc = c > 0 || q > 0 ? 1u : 0u;
            mma_mxf4nvf4(d, da + 2 * q, db + 2 * q, idesc, sfa + 4u * q, sfb + 4u * S::kHalves * q, acc);
          }
        mma_commit(&sm.empty[s]);
        if (c == sg.nc - 1) {
          mma_commit(&sm.acc_full[buf]);
          if (both) mma_commit(&sm.acc_full[1]);
        }
        ++k;
        s = next;
        phase = next_phase;
      }
    }
    ok = __all_sync(0xffffffffu, good);
  }
  if (k > 0) mbar_wait(&sm.empty[(k - 1) % kS], ((k - 1) / kS) & 1);   // not to leave with MMAs in flight
  __syncwarp();
}

extern __shared__ __align__(1024) uint8_t smem_raw[];

// ---- few places: UP, SUM ------------------------------------------------------------
constexpr int kFewWarps = 10;               // 0 weights, 1 products, 2-5 rows of x, 6-9 the accumulator
constexpr int kFewThreads = 32 * kFewWarps;
constexpr int kLoaders = 4;                  // warps 2-5

template <int NT, int MODE>
__global__ void __launch_bounds__(kFewThreads, 1) moe_few_kernel(const ExpertArgs a) {
  using S = Shape<NT, MODE, true>;
  constexpr int kS = S::kStages;
  static_assert(S::kHalves == 1 && kLoaders <= kS && (kLoaders & (kLoaders - 1)) == 0,
                "one buffer a segment; a loader looks at a stage's release when those of two rounds before are over");
  const Smem<NT, MODE, true> sm(smem_raw);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) sm.init_barriers(2, 4);
  if (warp == 1) sm.alloc_tmem();
  griddep_launch_dependents();
  griddep_wait();                            // the plan comes from a preceding kernel
  fence_proxy_async_global();                // (and the weights may)
  Table tb = sm.table();
  build_table<NT, false>(a, tb);
  const uint32_t tmem = *sm.tmem_slot;
  Walk<NT, MODE> walk(tb, a);
  Segment sg;

  if (MODE == UP) {
    // rows of no pair are zero: one scale over all rows is taken of h
    const size_t per = (size_t)a.N / 8, end = (size_t)a.n_pairs * per;
    for (size_t i = tb.total * per + blockIdx.x * kFewThreads + threadIdx.x; i < end; i += (size_t)gridDim.x * kFewThreads)
      reinterpret_cast<uint4*>(a.h)[i] = make_uint4(0u, 0u, 0u, 0u);
  }
  __syncwarp();

  if (warp == 0) {
    copy_weights(sm, a, walk);
  } else if (warp == 1) {
    multiply(sm, a, walk, tmem);
  } else if (warp < 6) {
    // ---------------- rows of x ----------------
    // A warp a stage: the fence that hands a stage over waits for all that its warp has under way, so a warp has no other
    // (with all four on a stage, each fenced every stage: 64 tokens of 8 of 128 experts, N 5120, K 768 took 62 us).
    const int mine = warp - 2, piece = lane & 7, q = lane & 3;
    const size_t row_codes = (size_t)a.K / 2, row_scales = (size_t)a.K / 16;
    constexpr int kCols = (NT + 31) / 32;
    int row[kCols];                            // rows of x of places lane, lane + 32 (the lowest one for a place of no pair)
    bool ok = true;
    for (int k = 0; ok && walk.next(sg); k += sg.nc) {
      int c = (mine - k) & (kLoaders - 1);
      if (c >= sg.nc) continue;
#pragma unroll
      for (int i = 0; i < kCols; ++i) {
        const int place = lane + 32 * i;
        row[i] = place < sg.n ? sg.p0 + place : 0;
        if (MODE == UP && place < sg.n) {
          const int pair = __ldcg(a.pairs + row[i]);
          const bool in = pair >= 0 && pair < a.n_pairs;
          if (!in) atomicOr(&g_nvfp4_device_error, NVFP4_DEVERR_MOE_RANGE);
          row[i] = in ? pair / a.top : 0;
        }
      }
      auto row_of = [&](int r) {               // of place r < NT, by the whole warp
        int x = __shfl_sync(0xffffffffu, row[0], r & 31);
        if (kCols > 1) {
          const int y = __shfl_sync(0xffffffffu, row[kCols - 1], r & 31);
          x = r >= 32 ? y : x;
        }
        return x;
      };
      for (; c < sg.nc; c += kLoaders) {
        const int s = (k + c) % kS, chunk = sg.c0 + c;
        // (the release before that one, two rounds ago, is over: stages are released in order, and this warp has waited for
        // that of kLoaders stages ago)
        if (k + c >= kS && !mbar_wait_warp(&sm.empty[s], (uint32_t)((k + c) / kS - 1) & 1u)) {
          ok = false;
          break;
        }
        const uint32_t slot = smem_u32(sm.base) + (uint32_t)(s * S::kSlot);
        const bool in_c = chunk * 128 + piece * 16 < (int)row_codes, in_s = chunk * 16 + q * 4 < (int)row_scales;
#pragma unroll 4
        for (int r0 = 0; r0 < sg.n; r0 += 4) {
          const int r = r0 + (lane >> 3), from = row_of(r);
          if (in_c && r < sg.n)
            async_copy16(slot + S::kOffX + r * 128 + ((piece ^ (r & 7)) << 4), a.xc + from * row_codes + chunk * 128 + piece * 16);
        }
#pragma unroll 2
        for (int r0 = 0; r0 < sg.n; r0 += 8) {
          const int r = r0 + (lane >> 2), from = row_of(r);
          if (in_s && r < sg.n)
            async_copy4(slot + S::kOffXS + q * 512 + (r & 31) * 16 + (r >> 5) * 4, a.xs + from * row_scales + chunk * 16 + q * 4);
        }
        async_commit();
        async_wait<0>();
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");   // the MMAs read through the asynchronous proxy
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.full[s]);
      }
    }
  } else {
    // ---------------- the accumulator ----------------
    const int p = warp & 3, row = p * 32 + lane;
    const float xg = __ldcg(a.xg);
    if (MODE == SUM)
      for (int t = 0; t < a.tokens; ++t) sm.sums[t * kTR + row] = 0.0f;
    Buffers bufs;
    // The pairs of a segment's places lane, lane + 32 and their weights are read a segment ahead.
    constexpr int kCols = (NT + 31) / 32;
    auto load_pairs = [&](int (&pair)[kCols]) {
#pragma unroll
      for (int i = 0; i < kCols; ++i) {
        const int m = lane + 32 * i;
        pair[i] = m < sg.n ? __ldcg(a.pairs + sg.p0 + m) : 0;
        if (pair[i] < 0 || pair[i] >= a.n_pairs) {
          if (p == 0) atomicOr(&g_nvfp4_device_error, NVFP4_DEVERR_MOE_RANGE);
          pair[i] = -1;
        }
      }
    };
    int pair[kCols], next_pair[kCols];
    float wgt[kCols];
    bool more = walk.next(sg);
    float wg = more ? __ldcg(a.wg + sg.e) : 0.0f;
    if (MODE == SUM && more) {
      load_pairs(pair);
#pragma unroll
      for (int i = 0; i < kCols; ++i) wgt[i] = pair[i] >= 0 ? __ldcg(a.weights + pair[i]) : 0.0f;
    }
    while (more) {
      const Segment cur = sg;
      const float scale = __fmul_rn(xg, wg);
      more = walk.next(sg);
      if (more) wg = __ldcg(a.wg + sg.e);
      if (MODE == SUM && more) load_pairs(next_pair);
      const int buf = bufs.first(false);
      if (!mbar_wait_warp(&sm.acc_full[buf], bufs.uses(buf) & 1)) break;
      tc_fence_after();
      bufs.took(false);
      const uint32_t d = tmem + ((uint32_t)(p * 32) << 16) + (uint32_t)(buf * S::kHalf);
#pragma unroll 1
      for (int m0 = 0; m0 < cur.n; m0 += 16) {
        float v[16];
        __syncwarp();
        read16(d + (uint32_t)m0, v);
        if (MODE == UP && a.cluster > 1) {
          // raw sums to the ring's memory (free: every MMA of the CTA's one item is done)
          float* stage = reinterpret_cast<float*>(sm.base);
#pragma unroll
          for (int i = 0; i < 16; ++i) stage[(m0 + i) * kTR + row] = v[i];
        } else if (MODE == UP) {
          store_h16(a, cur, p, m0, v, scale);
        } else {
          const int at = m0 >> 5, l0 = m0 & 31;
          int pr = pair[0];
          float wt = wgt[0];
          if (kCols > 1 && at == 1) pr = pair[kCols - 1], wt = wgt[kCols - 1];
          const int t_lane = pr >= 0 ? pr / a.top : -1;
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            if (i % 4 == 0 && m0 + i >= cur.n) break;         // (most segments of a decode batch have a few places)
            const int t = __shfl_sync(0xffffffffu, t_lane, l0 + i);
            const float w = __shfl_sync(0xffffffffu, wt, l0 + i);
            if (m0 + i < cur.n && t >= 0) {
              float* y = &sm.sums[t * kTR + row];
              *y = fmaf(w, v[i] * scale, *y);
            }
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.acc_empty[buf]);
      if (MODE == SUM && more) {
#pragma unroll
        for (int i = 0; i < kCols; ++i) {
          pair[i] = next_pair[i];
          wgt[i] = pair[i] >= 0 ? __ldcg(a.weights + pair[i]) : 0.0f;
        }
      }
    }
  }

  // ---------------- the cluster's parts ----------------
  __syncwarp();
  if (a.cluster > 1) cluster_sync(); else __syncthreads();
  if (MODE == SUM) {
    // a warp a token; all ranks' parts are read together (one by one, 64 tokens of 3 ranks took 10 us) and added in their order
    const int n = blockIdx.x / a.cluster * kTR + 4 * lane;
    for (int t = walk.rank + a.cluster * warp; t < a.tokens; t += a.cluster * kFewWarps) {
      float4 x[kMaxCluster];
#pragma unroll
      for (int r = 0; r < kMaxCluster; ++r)
        if (r < a.cluster) x[r] = ld_dsmem_f32x4(dsmem_addr(&sm.sums[t * kTR + 4 * lane], (uint32_t)r));
      float4 y = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
      for (int r = 0; r < kMaxCluster; ++r)
        if (r < a.cluster) y.x += x[r].x, y.y += x[r].y, y.z += x[r].z, y.w += x[r].w;
      float* dst = a.out + (size_t)t * a.N + n;
      if (a.N % 4 == 0) {
        if (n < a.N) *reinterpret_cast<float4*>(dst) = y;
      } else {
        if (n < a.N) dst[0] = y.x;
        if (n + 1 < a.N) dst[1] = y.y;
        if (n + 2 < a.N) dst[2] = y.z;
        if (n + 3 < a.N) dst[3] = y.w;
      }
    }
  }
  if (MODE == UP && a.cluster > 1 && warp >= 6) {
    // a cluster has one item at most: its parts are in every CTA's stage; the ranks take its places in turn
    Walk<NT, MODE> again(tb, a);
    if (again.next(sg)) {
      const int row = (warp & 3) * 32 + lane, i = sg.rt * 64 + row / 2;
      const float scale = __fmul_rn(__ldcg(a.xg), __ldcg(a.wg + sg.e));
      const float* stage = reinterpret_cast<const float*>(sm.base);
      for (int m = walk.rank; m < sg.n; m += a.cluster) {
        float x[kMaxCluster], v = 0.0f;
#pragma unroll
        for (int r = 0; r < kMaxCluster; ++r)
          if (r < a.cluster) x[r] = ld_dsmem_f32(dsmem_addr(&stage[m * kTR + row], (uint32_t)r));
#pragma unroll
        for (int r = 0; r < kMaxCluster; ++r)
          if (r < a.cluster) v += x[r];
        v *= lane & 1 ? scale : 0.25f * scale;
        const float other = __shfl_xor_sync(0xffffffffu, v, 1);
        if (!(lane & 1) && i < a.N)
          a.h[(size_t)(sg.p0 + m) * a.N + i] = __bfloat16_as_ushort(__float2bfloat16_rn(silu_mul(v, other)));
      }
    }
  }
  tc_fence_before();
  __syncwarp();
  if (a.cluster > 1) cluster_sync();                              // (the others have read this CTA's memory)
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    sm.free_tmem(tmem);
  }
}

// ---- many places: UP, PART -----------------------------------------------------------
// 0 weights, 1 products, 2 rows of x, 4-19 the accumulator: with 16 of them a warp holds all its columns of a buffer in
// registers, so that the buffer is free before they are stored (2048 tokens of 8 of 128 experts, K 4096 and 1536 rows up,
// K 768 and 4096 rows down: 135 and 155 us; 8 warps, 16 columns at a time: 137 and 157).
constexpr int kManyWarps = 20;
constexpr int kReaders = kManyWarps - 4;
constexpr int kManyThreads = 32 * kManyWarps;
constexpr int kBoxRows = 64;                 // rows of x of a copy (2048 tokens, up: 137 us; 32: 141)

template <int NT, int MODE>
__global__ void __launch_bounds__(kManyThreads, 1) moe_many_kernel(const __grid_constant__ CUtensorMap tm_x,
                                                                   const ExpertArgs a) {
  using S = Shape<NT, MODE, false>;
  const Smem<NT, MODE, false> sm(smem_raw);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    prefetch_tmap(&tm_x);
    sm.init_barriers(2, kReaders);
  }
  if (warp == 1) sm.alloc_tmem();
  griddep_launch_dependents();
  griddep_wait();
  fence_proxy_async_global();                // rows and scales were laid out by a preceding kernel
  Table tb = sm.table();
  build_table<NT, (NT > 128)>(a, tb);
  const uint32_t tmem = *sm.tmem_slot;
  Walk<NT, MODE> walk(tb, a);
  Segment sg;
  if (MODE == UP) {
    const size_t per = (size_t)a.N / 8, end = (size_t)a.n_pairs * per;
    for (size_t i = tb.total * per + blockIdx.x * kManyThreads + threadIdx.x; i < end; i += (size_t)gridDim.x * kManyThreads)
      reinterpret_cast<uint4*>(a.h)[i] = make_uint4(0u, 0u, 0u, 0u);
  }
  __syncwarp();

  if (warp == 0) {
    copy_weights(sm, a, walk);
  } else if (warp == 1) {
    multiply(sm, a, walk, tmem);
  } else if (warp == 2) {
    // ---------------- rows of x, in the order of the plan, and their scales ----------------
    fill_stages(sm, walk, [&](const Segment& sg, int c, uint8_t* slot, uint64_t* bar) {
      const int boxes = (sg.n + kBoxRows - 1) / kBoxRows, halves = (sg.n + 127) / 128;
      mbar_arrive_expect_tx(bar, (uint32_t)(boxes * kBoxRows * 128 + halves * kXBlock));
      for (int b = 0; b < boxes; ++b)
        tma_load_2d(slot + S::kOffX + b * (kBoxRows * 128), &tm_x, c * 128, sg.p0 + b * kBoxRows, bar);
      for (int h = 0; h < halves; ++h)
        bulk_g2s(slot + S::kOffXS + h * kXBlock, a.x_blocks + ((size_t)(sg.block + h) * a.C + c) * kXBlock, kXBlock, bar);
    });
  } else if (warp >= 4) {
    // ---------------- the accumulator: four warps a lane quadrant, 16 columns in turn ----------------
    const int p = warp & 3, row = p * 32 + lane, part = (warp - 4) >> 2;
    const float xg = __ldcg(a.xg);
    Buffers bufs;
    bool ok = true;
    while (ok && walk.next(sg)) {
      const float scale = __fmul_rn(xg, __ldcg(a.wg + sg.e));
      const bool both = S::kHalves == 2 && sg.n > 128;
      const int halves = both ? 2 : 1;
#pragma unroll 1
      for (int half = 0; half < halves; ++half) {
        const int buf = both ? half : bufs.first(false);
        if (!mbar_wait_warp(&sm.acc_full[buf], bufs.uses(buf) & 1)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t d = tmem + ((uint32_t)(p * 32) << 16) + (uint32_t)(buf * S::kHalf);
        // All of the warp's columns to registers first, so that the buffer is free while they are stored.
        constexpr int kGroups = (S::kHalf + 16 * (kReaders / 4) - 1) / (16 * (kReaders / 4));
        const int end = min(sg.n - half * 128, S::kHalf);
        float v[kGroups][16];
        __syncwarp();
#pragma unroll
        for (int g = 0; g < kGroups; ++g)
          if (16 * part + 4 * kReaders * g < end) read16(d + (uint32_t)(16 * part + 4 * kReaders * g), v[g]);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.acc_empty[buf]);
#pragma unroll
        for (int g = 0; g < kGroups; ++g) {
          const int m = half * 128 + 16 * part + 4 * kReaders * g;
          if (m >= sg.n) break;
          if (MODE == UP) {
            store_h16(a, sg, p, m, v[g], scale);
          } else {
            float* dst = a.out + ((size_t)(sg.rt - a.rt0) * a.n_pairs + sg.p0 + m) * kTR + row;
#pragma unroll
            for (int i = 0; i < 16; ++i)
              if (m + i < sg.n) dst[i * kTR] = v[g][i] * scale;
          }
        }
      }
      bufs.took(both);
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    sm.free_tmem(tmem);
  }
}

// Rows of x in the order of the plan, and their scales in blocks of 128 places and 256 of K: a CTA a tile of 128 places of
// an expert and kArrangeChunks chunks.  codes NULL: the rows stand so already (down), only the scales are laid out.  Bound by
// the latency of the table, the pairs and the rows, one behind the other: 2048 tokens of 8 of 128 experts, K 4096, 38 MB
// written: 20 us (scales alone, K 768: 7).
struct ArrangeArgs {
  ExpertArgs x;
  uint8_t *codes, *blocks;
  int* last;                                 // down: the number of pairs that get products (0: a plan that is refused); or NULL
};
constexpr int kArrangeThreads = 256;
constexpr int kArrangeChunks = 4;

__global__ void __launch_bounds__(kArrangeThreads) moe_arrange_kernel(const ArrangeArgs g) {
  __shared__ __align__(16) uint8_t s_table[kTableBytes], s_offsets[kOffsetsBytes];
  __shared__ int s_row[128];
  griddep_launch_dependents();
  griddep_wait();
  const ExpertArgs& a = g.x;
  Table tb(s_table, s_offsets);
  build_table<128, false>(a, tb);
  if (g.last && blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) *g.last = tb.total;
  if ((int)blockIdx.x >= tb.tiles) return;
  int used = 0;                              // the last entry whose tiles begin at blockIdx.x or before
  for (int hi = tb.used; hi - used > 1;) {
    const int mid = (used + hi) >> 1;
    if (tb.blocks[mid] <= (int)blockIdx.x) used = mid; else hi = mid;
  }
  const int in = blockIdx.x - tb.blocks[used], p0 = tb.first[used] + 128 * in, n = min(128, tb.count[used] - 128 * in);
  for (int r = threadIdx.x; r < n; r += kArrangeThreads) {
    int row = p0 + r;
    if (g.codes) {
      const int pair = __ldcg(a.pairs + row);
      const bool there = pair >= 0 && pair < a.n_pairs;
      if (!there) atomicOr(&g_nvfp4_device_error, NVFP4_DEVERR_MOE_RANGE);
      row = there ? pair / a.top : 0;
    }
    s_row[r] = row;
  }
  __syncthreads();
  const int c0 = blockIdx.y * kArrangeChunks, c1 = min(a.C, c0 + kArrangeChunks);
  const int row_codes = a.K / 2, row_scales = a.K / 16;
  // scales: word q of chunk c of rows i, i + 32, i + 64, i + 96 in 16 bytes
  for (int x = threadIdx.x; x < (c1 - c0) * 128; x += kArrangeThreads) {
    const int c = c0 + (x >> 7), q = (x >> 5) & 3, i = x & 31, at = c * 16 + q * 4;
    uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
    for (int p = 0; p < 4; ++p)
      if (i + 32 * p < n && at < row_scales)
        w[p] = __ldcg(reinterpret_cast<const uint32_t*>(a.xs + (size_t)s_row[i + 32 * p] * row_scales + at));
    *reinterpret_cast<uint4*>(g.blocks + ((size_t)blockIdx.x * a.C + c) * kXBlock + q * 512 + i * 16) =
        make_uint4(w[0], w[1], w[2], w[3]);
  }
  if (!g.codes) return;
  // a warp a row's codes of the CTA's chunks
  constexpr int kPieces = kArrangeChunks * 8;
  const int b0 = c0 * 128, b1 = min(row_codes, c1 * 128);
  for (int x = threadIdx.x; x < n * kPieces; x += 4 * kArrangeThreads) {
    uint4 v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int y = x + i * kArrangeThreads, r = y / kPieces, at = b0 + y % kPieces * 16;
      if (r < n && at < b1) v[i] = __ldcg(reinterpret_cast<const uint4*>(a.xc + (size_t)s_row[r] * row_codes + at));
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int y = x + i * kArrangeThreads, r = y / kPieces, at = b0 + y % kPieces * 16;
      if (r < n && at < b1) *reinterpret_cast<uint4*>(g.codes + (size_t)(p0 + r) * row_codes + at) = v[i];
    }
  }
}

// y[t, n] = sum_j weights[t, j] part[places[t, j], n], in the order of j: a thread has V columns of a token.  Bound by HBM:
// 2048 tokens of 8, N 4096: 302 MB in 54 us (5.6 TB/s).
struct CombineArgs {
  const float *part, *weights;               // part: [column / 128][n_pairs][128], columns [n0, n1) of y
  const int32_t *places, *last;              // last: places from *last on have no product (what stands there was never written)
  float* y;
  int tokens, top, N, n_pairs, n0, n1;
};

constexpr int kAtOnce = 8;                   // products of a token that are read together
constexpr int kCombineCtas = 16;             // CTAs an SM, each goes through several tokens (2048 tokens of 8, N 4096: 162 us
                                             // with the products; 8: 163, 4: 178, 2: 233)

template <int V>
__global__ void __launch_bounds__(256) moe_combine_kernel(const CombineArgs a) {
  griddep_launch_dependents();
  griddep_wait();
  const int n = a.n0 + (blockIdx.x * 256 + threadIdx.x) * V;
  if (n >= a.n1) return;
  const size_t column = (size_t)((n - a.n0) / kTR) * a.n_pairs;
  // places and weights are read a token ahead
  auto look = [&](int t, int j0, int (&place)[kAtOnce], float (&w)[kAtOnce]) {
#pragma unroll
    for (int j = 0; j < kAtOnce; ++j) {
      const bool there = t < a.tokens && j0 + j < a.top;
      place[j] = there ? __ldcg(a.places + (size_t)t * a.top + j0 + j) : -1;
      w[j] = there ? __ldcg(a.weights + (size_t)t * a.top + j0 + j) : 0.0f;
    }
  };
  int place[kAtOnce];
  float w[kAtOnce];
  look(blockIdx.y, 0, place, w);
  const int last = __ldcg(a.last);
  for (int t = blockIdx.y; t < a.tokens; t += gridDim.y) {
    float y[V] = {};
    for (int j0 = 0; j0 < a.top; j0 += kAtOnce) {
      float x[kAtOnce][V];
      bool there[kAtOnce];
#pragma unroll
      for (int j = 0; j < kAtOnce; ++j) {
        there[j] = place[j] >= 0 && place[j] < last;
        if (!there[j] && place[j] != -1) atomicOr(&g_nvfp4_device_error, NVFP4_DEVERR_MOE_RANGE);
        const float* src = a.part + (column + (there[j] ? place[j] : 0)) * kTR + n % kTR;
        if constexpr (V == 4) {
          const float4 v = there[j] ? __ldcg(reinterpret_cast<const float4*>(src)) : make_float4(0.f, 0.f, 0.f, 0.f);
          x[j][0] = v.x, x[j][1] = v.y, x[j][2] = v.z, x[j][3] = v.w;
        } else {
          x[j][0] = there[j] ? __ldcg(src) : 0.0f;
        }
      }
      float wj[kAtOnce];
#pragma unroll
      for (int j = 0; j < kAtOnce; ++j) wj[j] = w[j];
      const bool more = j0 + kAtOnce < a.top;
      look(more ? t : t + gridDim.y, more ? j0 + kAtOnce : 0, place, w);
#pragma unroll
      for (int j = 0; j < kAtOnce; ++j)
        if (there[j]) {
#pragma unroll
          for (int v = 0; v < V; ++v) y[v] = fmaf(wj[j], x[j][v], y[v]);
        }
    }
    float* dst = a.y + (size_t)t * a.N + n;
    if constexpr (V == 4)
      *reinterpret_cast<float4*>(dst) = make_float4(y[0], y[1], y[2], y[3]);
    else
      *dst = y[0];
  }
}

// Row-major codes and scales of all experts into blocks: a thread a 16-byte piece of codes, or a row's scales of a block.
struct PackArgs {
  const uint8_t *codes, *scales;
  uint8_t* packed;
  int N, K, C, RT, gated;
  long long blocks;
};

__global__ void __launch_bounds__(256) moe_pack_kernel(const PackArgs a) {
  griddep_launch_dependents();
  griddep_wait();
  constexpr int kPieces = kTR * 9;                 // 8 of codes and the scales of each row
  for (long long b = blockIdx.x; b < a.blocks; b += gridDim.x) {
    const int c = (int)(b % a.C);
    const long long et = b / a.C;
    const int rt = (int)(et % a.RT);
    const long long e = et / a.RT;
    uint8_t* dst = a.packed + (size_t)b * kBlock;
    for (int i = threadIdx.x; i < kPieces; i += 256) {
      const int r = i / 9, j = i - r * 9, g = rt * kTR + r;
      const int n = a.gated ? (g & 1) * (a.N / 2) + g / 2 : g;     // the row of the matrix
      const bool there = g < a.N;
      const size_t row = (size_t)e * a.N + (there ? n : 0);
      if (j < 8) {
        uint4 v = make_uint4(0u, 0u, 0u, 0u);
        if (there && c * 128 + j * 16 < a.K / 2)
          v = __ldcg(reinterpret_cast<const uint4*>(a.codes + row * (a.K / 2) + c * 128 + j * 16));
        *reinterpret_cast<uint4*>(dst + r * 128 + ((j ^ (r & 7)) << 4)) = v;
      } else {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          uint32_t v = 0u;
          if (there && c * 16 + q * 4 < a.K / 16)
            v = __ldcg(reinterpret_cast<const uint32_t*>(a.scales + row * (a.K / 16) + c * 16 + q * 4));
          *reinterpret_cast<uint32_t*>(dst + kWCodes + q * 512 + (r & 31) * 16 + (r >> 5) * 4) = v;
        }
      }
    }
  }
}

int device_sms() {
  static PerDeviceInt sms;
  cudaError_t err = cudaSuccess;
  const int n = sms.get([](int dev, cudaError_t* e) -> int {
    int v = 0;
    *e = cudaDeviceGetAttribute(&v, cudaDevAttrMultiProcessorCount, dev);
    return v;
  }, &err);
  return n > 0 ? n : 152;
}

template <class... Args>
cudaError_t launch(void (*kern)(Args...), dim3 grid, int threads, size_t smem, int cluster, cudaStream_t stream,
                   const Args&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kern, args...);
}

// Allows a kernel its dynamic shared memory, once a device.
template <auto KERNEL>
cudaError_t allow_smem(size_t bytes) {
  static PerDeviceInt done;
  cudaError_t err = cudaSuccess;
  done.get([bytes](int, cudaError_t* e) -> int {
    *e = cudaFuncSetAttribute(KERNEL, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
    return *e == cudaSuccess ? 1 : 0;
  }, &err);
  return err;
}

template <int NT, int MODE>
cudaError_t run_few(long long grid, const ExpertArgs& a, cudaStream_t stream) {
  constexpr size_t bytes = Shape<NT, MODE, true>::kBytes;
  const cudaError_t e = allow_smem<moe_few_kernel<NT, MODE>>(bytes);
  if (e != cudaSuccess) return e;
  return launch(moe_few_kernel<NT, MODE>, dim3((unsigned)grid), kFewThreads, bytes, a.cluster, stream, a);
}

template <int NT, int MODE>
cudaError_t run_many(long long grid, const CUtensorMap& map, const ExpertArgs& a, cudaStream_t stream) {
  constexpr size_t bytes = Shape<NT, MODE, false>::kBytes;
  const cudaError_t e = allow_smem<moe_many_kernel<NT, MODE>>(bytes);
  if (e != cudaSuccess) return e;
  return launch(moe_many_kernel<NT, MODE>, dim3((unsigned)grid), kManyThreads, bytes, 1, stream, map, a);
}

// Places of a tile: with few 64 (16 places are no faster for 1, 8 or 16 tokens: a stage's time is that of its weights), with
// many 256 (1024 tokens of 8 of 128 experts, up: 112 us, with 64 places 136; with 16 places an expert as fast).
constexpr int kFewTile = 64, kManyTile = 256;

// Tokens up to which y is summed in shared memory, which holds no more.  Both sides, us: 128 experts, 8 a token, N 5120, K 768:
// 16 tokens 40, by products and sums 49; 32 tokens 47, 57; 64 tokens 55, 64.  2 of 8 experts, N 4096, K 2048: 64 tokens 14, 20.
// Beyond 76 row tiles a tile has one CTA and the sums lose (N 9856: 141, 109).  For h, where all places are those of few
// experts: 64 tokens of 2 of 2, K 4096, 8192 rows 14, laid out 18.
constexpr int kFewTokens = 64;

long long used_experts(const ExpertArgs& a) { return a.n_pairs < a.experts ? a.n_pairs : a.experts; }

// Most stretches of up to nt pairs that any plan of the pairs has.
long long most_tiles(const ExpertArgs& a, int nt) {
  const long long used = used_experts(a);
  return used + (a.n_pairs - used) / nt;
}

// Whether h goes without rows laid out first: few tokens, or few places an expert on average, which is what the host knows
// (K 4096, 1536 rows, 512 tokens of 8 of 128 experts, 32 places each: 85 us, laid out 101; K 4096, 16384 rows, 2 of 8
// experts, 32 places each: 55 and 67, 64 places: 84 and 76).
bool few_places(const ExpertArgs& a) { return a.tokens <= kFewTokens || a.n_pairs <= 32 * used_experts(a); }

size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }
size_t codes_bytes(const ExpertArgs& a) { return align256((size_t)a.n_pairs * a.K / 2); }
size_t blocks_bytes(const ExpertArgs& a) { return align256((size_t)most_tiles(a, 128) * a.C * kXBlock); }

}  // namespace

// Defined in gemv.cu.
bool nvfp4_internal_encode_2d(CUtensorMap* map, const void* base, uint64_t inner_bytes, uint64_t rows,
                              uint32_t box_inner, uint32_t box_rows, bool swizzle128);

namespace {

// Rows of x by place (codes: where they go, NULL: they stand so) and their scales' blocks, and the map of the rows.
cudaError_t arrange(const ExpertArgs& a, uint8_t* codes, uint8_t* blocks, int* last, CUtensorMap* map, cudaStream_t stream) {
  memset(map, 0, sizeof(*map));
  if (!nvfp4_internal_encode_2d(map, codes ? codes : a.xc, (uint64_t)a.K / 2, (uint64_t)a.n_pairs, 128, kBoxRows, true))
    return cudaErrorInvalidValue;
  ArrangeArgs g = {a, codes, blocks, last};
  const dim3 grid((unsigned)most_tiles(a, 128), (unsigned)((a.C + kArrangeChunks - 1) / kArrangeChunks));
  return launch(moe_arrange_kernel, grid, kArrangeThreads, 0, 1, stream, g);
}

// Most bytes of products that wait for their sum: above, y is done in slabs of columns.  Smaller slabs that stay in L2 (129 MB)
// cost their launches and gained nothing (2048 tokens of 8 experts, N 4096, K 768: 32 MB 206 us, 64 184, 128 177, 512 170).
constexpr long long kSlabBytes = 512ll << 20;

constexpr size_t kLastBytes = 256;           // the number of pairs that get products, behind the products

int slab_tiles(const ExpertArgs& a) {
  const long long per = (long long)a.n_pairs * kTR * 4, fit = kSlabBytes / per;
  return (int)(fit < 1 ? 1 : fit < a.RT ? fit : a.RT);
}

size_t products_bytes(const ExpertArgs& a) { return (size_t)a.n_pairs * slab_tiles(a) * kTR * sizeof(float); }

// Whether a call's items and units are counted in 31 bits.
bool too_many_items(const ExpertArgs& a) {
  const long long tiles = most_tiles(a, kFewTile);
  return tiles * a.RT > 0x7FFFFFFFll || tiles * a.C > 0x7FFFFFFFll;
}

bool bad_matrix(int experts, int N, int K, bool gated) {
  return experts < 1 || experts > kMaxExperts || N < 1 || N > (1 << 20) || K < 64 || K > (1 << 20) || K % 64 != 0 ||
         (gated && N % 128 != 0);
}

}  // namespace

nvfp4_status nvfp4_internal_cuda_status(cudaError_t e);
bool nvfp4_internal_aligned(const void* p, size_t a);
nvfp4_status nvfp4_internal_check_device();

extern "C" size_t nvfp4_moe_packed_weight_bytes(int experts, int N, int K, int gated) {
  if (bad_matrix(experts, N, K, gated != 0)) return 0;
  return (size_t)experts * ((N + kTR - 1) / kTR) * ((K + kChunk - 1) / kChunk) * kBlock;
}

extern "C" nvfp4_status nvfp4_moe_pack_weights(const uint8_t* wq, const uint8_t* ws, int experts, int N, int K, int gated,
                                               uint8_t* packed, size_t packed_bytes, cudaStream_t stream) {
  if (!wq || !ws || !packed) return NVFP4_ERR_NULL;
  const size_t need = nvfp4_moe_packed_weight_bytes(experts, N, K, gated);
  if (need == 0 || packed_bytes < need) return NVFP4_ERR_SHAPE;
  if (!nvfp4_internal_aligned(wq, 16) || !nvfp4_internal_aligned(ws, 4) || !nvfp4_internal_aligned(packed, 16))
    return NVFP4_ERR_ALIGN;
  const nvfp4_status ds = nvfp4_internal_check_device();
  if (ds != NVFP4_OK) return ds;
  PackArgs a = {};
  a.codes = wq, a.scales = ws, a.packed = packed;
  a.N = N, a.K = K, a.C = (K + kChunk - 1) / kChunk, a.RT = (N + kTR - 1) / kTR, a.gated = gated != 0;
  a.blocks = (long long)(need / kBlock);
  const long long grid = a.blocks < 65536 ? a.blocks : 65536;
  return nvfp4_internal_cuda_status(launch(moe_pack_kernel, dim3((unsigned)grid), 256, 0, 1, stream, a));
}

namespace {

nvfp4_status check_experts(const uint8_t* xq, const uint8_t* xs, const float* xg, const ExpertArgs& a, const void* out) {
  if (a.tokens < 0 || a.top < 1 || a.top > kMaxTop || (long long)a.tokens * a.top > 0x7FFFFFFFll) return NVFP4_ERR_SHAPE;
  if (a.tokens == 0) return NVFP4_OK;
  if (!xq || !xs || !xg || !a.w || !a.wg || !a.offsets || !a.pairs || !out) return NVFP4_ERR_NULL;
  if (!nvfp4_internal_aligned(xq, 16) || !nvfp4_internal_aligned(xs, 4) || !nvfp4_internal_aligned(xg, 4) ||
      !nvfp4_internal_aligned(a.w, 16) || !nvfp4_internal_aligned(a.wg, 4) || !nvfp4_internal_aligned(a.offsets, 4) ||
      !nvfp4_internal_aligned(a.pairs, 4) || !nvfp4_internal_aligned(out, 16))
    return NVFP4_ERR_ALIGN;
  return NVFP4_OK;
}

ExpertArgs experts_args(const uint8_t* xq, const uint8_t* xs, const float* xg, int tokens, int top_k, const int32_t* offsets,
                        const int32_t* pairs, const uint8_t* w, const float* wg, int experts, int rows, int K) {
  ExpertArgs a;
  memset(&a, 0, sizeof(a));
  a.xc = xq, a.xs = xs, a.xg = xg, a.w = w, a.wg = wg, a.offsets = offsets, a.pairs = pairs;
  a.tokens = tokens, a.top = top_k, a.experts = experts, a.K = K;
  a.C = (K + kChunk - 1) / kChunk, a.RT = a.rts = (rows + kTR - 1) / kTR;
  a.n_pairs = tokens * top_k;                // (checked to fit by check_experts before it is used)
  a.cluster = 1;
  return a;
}

}  // namespace

extern "C" size_t nvfp4_moe_gate_up_workspace_bytes(int tokens, int top_k, int experts, int K) {
  if (tokens < 1 || top_k < 1 || top_k > kMaxTop || (long long)tokens * top_k > 0x7FFFFFFFll ||
      bad_matrix(experts, 128, K, false))
    return 0;
  const ExpertArgs a = experts_args(nullptr, nullptr, nullptr, tokens, top_k, nullptr, nullptr, nullptr, nullptr, experts, 128, K);
  return few_places(a) ? 0 : codes_bytes(a) + blocks_bytes(a);
}

extern "C" nvfp4_status nvfp4_moe_gate_up(const uint8_t* xq, const uint8_t* xs, const float* xg, int tokens, int top_k,
                                          const int32_t* offsets, const int32_t* pairs, const uint8_t* wpacked,
                                          const float* wg, int experts, int inter, int K, uint16_t* h, void* workspace,
                                          size_t workspace_bytes, cudaStream_t stream) {
  if (inter < 64 || inter > (1 << 19) || bad_matrix(experts, 2 * inter, K, true)) return NVFP4_ERR_SHAPE;
  if (tokens < 0 || top_k < 1 || top_k > kMaxTop || (long long)tokens * top_k > 0x7FFFFFFFll) return NVFP4_ERR_SHAPE;
  ExpertArgs a = experts_args(xq, xs, xg, tokens, top_k, offsets, pairs, wpacked, wg, experts, 2 * inter, K);
  a.h = h, a.N = inter;
  if (too_many_items(a)) return NVFP4_ERR_SHAPE;
  const nvfp4_status cs = check_experts(xq, xs, xg, a, h);
  if (cs != NVFP4_OK || tokens == 0) return cs;
  const size_t need = nvfp4_moe_gate_up_workspace_bytes(tokens, top_k, experts, K);
  if (need > 0 && !workspace) return NVFP4_ERR_NULL;
  if (!nvfp4_internal_aligned(workspace, 256)) return NVFP4_ERR_ALIGN;
  if (workspace_bytes < need) return NVFP4_ERR_SHAPE;
  const nvfp4_status ds = nvfp4_internal_check_device();
  if (ds != NVFP4_OK) return ds;
  const int sms = device_sms();
  if (need == 0) {
    const long long items = most_tiles(a, kFewTile) * a.RT;
    while (a.cluster < kMaxCluster && items * a.cluster * 2 <= sms && a.C >= a.cluster * 2) a.cluster *= 2;
    const long long grid = items * a.cluster < sms ? items * a.cluster : sms;
    return nvfp4_internal_cuda_status(run_few<kFewTile, UP>(grid, a, stream));
  }
  uint8_t *codes = static_cast<uint8_t*>(workspace), *blocks = codes + codes_bytes(a);
  CUtensorMap map;
  const cudaError_t e = arrange(a, codes, blocks, nullptr, &map, stream);
  if (e != cudaSuccess) return nvfp4_internal_cuda_status(e);
  a.x_blocks = blocks;
  const long long items = most_tiles(a, kManyTile) * a.RT, grid = items < sms ? items : sms;
  return nvfp4_internal_cuda_status(run_many<kManyTile, UP>(grid, map, a, stream));
}

extern "C" size_t nvfp4_moe_down_workspace_bytes(int tokens, int top_k, int experts, int N, int K) {
  if (tokens <= kFewTokens || top_k < 1 || top_k > kMaxTop || (long long)tokens * top_k > 0x7FFFFFFFll ||
      bad_matrix(experts, N, K, false))
    return 0;
  const ExpertArgs a = experts_args(nullptr, nullptr, nullptr, tokens, top_k, nullptr, nullptr, nullptr, nullptr, experts, N, K);
  return blocks_bytes(a) + products_bytes(a) + kLastBytes;
}

extern "C" nvfp4_status nvfp4_moe_down(const uint8_t* hq, const uint8_t* hs, const float* hg, int tokens, int top_k,
                                       const int32_t* offsets, const int32_t* pairs, const int32_t* places,
                                       const float* weights, const uint8_t* wpacked, const float* wg, int experts, int N,
                                       int K, float* y, void* workspace, size_t workspace_bytes, cudaStream_t stream) {
  if (bad_matrix(experts, N, K, false)) return NVFP4_ERR_SHAPE;
  if (tokens < 0 || top_k < 1 || top_k > kMaxTop || (long long)tokens * top_k > 0x7FFFFFFFll) return NVFP4_ERR_SHAPE;
  ExpertArgs a = experts_args(hq, hs, hg, tokens, top_k, offsets, pairs, wpacked, wg, experts, N, K);
  a.N = N, a.weights = weights;
  if (too_many_items(a)) return NVFP4_ERR_SHAPE;
  const nvfp4_status cs = check_experts(hq, hs, hg, a, y);
  if (cs != NVFP4_OK || tokens == 0) return cs;
  if (!places || !weights) return NVFP4_ERR_NULL;
  const size_t need = nvfp4_moe_down_workspace_bytes(tokens, top_k, experts, N, K);
  if (need > 0 && !workspace) return NVFP4_ERR_NULL;
  if (!nvfp4_internal_aligned(places, 4) || !nvfp4_internal_aligned(weights, 4) || !nvfp4_internal_aligned(workspace, 256))
    return NVFP4_ERR_ALIGN;
  if (workspace_bytes < need) return NVFP4_ERR_SHAPE;
  const nvfp4_status ds = nvfp4_internal_check_device();
  if (ds != NVFP4_OK) return ds;
  const int sms = device_sms();
  if (need == 0) {
    a.out = y;
    while (a.cluster < kMaxCluster && a.RT * (a.cluster + 1) <= sms) ++a.cluster;
    return nvfp4_internal_cuda_status(run_few<kFewTile, SUM>((long long)a.RT * a.cluster, a, stream));
  }
  uint8_t* blocks = static_cast<uint8_t*>(workspace);
  uint8_t* products = blocks + blocks_bytes(a);
  int* last = reinterpret_cast<int*>(products + products_bytes(a));
  CUtensorMap map;
  cudaError_t e = arrange(a, nullptr, blocks, last, &map, stream);
  if (e != cudaSuccess) return nvfp4_internal_cuda_status(e);
  a.x_blocks = blocks;
  a.out = reinterpret_cast<float*>(products);
  const int slab = slab_tiles(a);
  for (a.rt0 = 0; a.rt0 < a.RT; a.rt0 += slab) {
    a.rts = a.RT - a.rt0 < slab ? a.RT - a.rt0 : slab;
    const long long items = most_tiles(a, kManyTile) * a.rts, grid = items < sms ? items : sms;
    e = run_many<kManyTile, PART>(grid, map, a, stream);
    if (e != cudaSuccess) break;
    const int n0 = a.rt0 * kTR, n1 = (a.rt0 + a.rts) * kTR < N ? (a.rt0 + a.rts) * kTR : N;
    const CombineArgs c = {a.out, weights, places, last, y, tokens, top_k, N, a.n_pairs, n0, n1};
    const int per = N % 4 == 0 ? 1024 : 256;
    const int across = (n1 - n0 + per - 1) / per, down = (kCombineCtas * sms + across - 1) / across;
    const dim3 grid2((unsigned)across, (unsigned)(tokens < down ? tokens : down));
    e = N % 4 == 0 ? launch(moe_combine_kernel<4>, grid2, 256, 0, 1, stream, c)
                   : launch(moe_combine_kernel<1>, grid2, 256, 0, 1, stream, c);
    if (e != cudaSuccess) break;
  }
  return nvfp4_internal_cuda_status(e);
}
