// The chosen experts' NVFP4 products (tcgen05, sm_103a), on a plan of the pairs by expert:
//   gate_up  h[p, i] = BF16(SiLU(g) u),  g = xg wg[e] x[t(p)] . w[e, gate row i],  u the same with up row i
//   down     y[t, n] = sum_j weight[t, j] hg wg[e] h[place(t, j)] . w[e, n]
//
// As in the projections, 128 weight rows are the wide side of the MMA (kind::mxf4nvf4) and an expert's rows of x its
// narrow side, here up to NT of them, N chosen at run time: the work of a tile is the bytes of its weights
// however few rows the expert got.  Bound by HBM (each chosen expert's weights once) until an expert has some hundreds
// of rows.
//
// Weights are packed (nvfp4_moe_pack_weights) in blocks of 128 rows x 256 K, one bulk copy each; a block's scales stand
// as tcgen05.cp wants them, so that they go from the block to TMEM without a thread's help.  Rows of gate and up
// alternate: a TMEM lane and its neighbour hold both halves of an h.
//
// Roles of a CTA (one an SM):
//   warp 0     weight blocks into a ring of S stages
//   warp 1     scales to TMEM, 4 MMAs of K = 64 a stage, commits
//   warps 2-5  rows of x into the stage: 16-byte asynchronous copies of the rows that the plan names, in the order of
//              the 128-byte swizzle; their scales in the order of tcgen05.cp
//   warps 6-9  the accumulator (two buffers up to 128 columns) to h, or to sums of y
//
// Three modes:
//   UP    items (expert, row tile, up to NT of its pairs) dealt out to the CTAs in turn; with fewer items than SMs a
//         cluster splits an item's K and adds the parts over distributed shared memory.
//   SUM   (down, few tokens) a cluster takes a tile of y's columns and shares out all the experts' K for it: every
//         token's sum over its experts stays in shared memory and meets the other CTAs' there.  No workspace, one launch.
//   PART  (down, many tokens) items as in UP; products go to a workspace [places, N], and a second kernel adds a
//         token's products with its weights.
// Nothing here waits for another CTA but at cluster barriers, and no state is left behind.
#include <string.h>

#include "common.cuh"
#include "tcgen05.cuh"

NVFP4_DEFINE_ERROR_READER(nvfp4_internal_read_error_moe_experts)

namespace {

constexpr int kTR = 128;                     // weight rows of a tile: MMA M
constexpr int kChunk = 256;                  // K of a stage
constexpr int kWCodes = kTR * 128;           // 16384
constexpr int kBlock = kWCodes + kTR * 16;   // 18432
constexpr int kWarps = 10;
constexpr int kThreads = 32 * kWarps;
constexpr int kLoaders = 128;                // warps 2-5
constexpr int kLag = 2;                      // stages whose row copies are in flight behind the one that is issued
constexpr int kMaxExperts = 512;
constexpr int kMaxTop = 32;
constexpr int kMaxCluster = 8;
constexpr uint32_t kTmemCols = 512;

enum Mode { UP, SUM, PART };

template <int NT, int MODE>
struct Shape {
  static constexpr int kXCodes = NT * 128;
  static constexpr int kHalves = NT > 128 ? 2 : 1;                    // of 128 tokens
  static constexpr int kOffX = kBlock;
  static constexpr int kOffXS = kOffX + kXCodes;
  static constexpr int kSlot = kOffXS + kHalves * 2048;
  static constexpr int kSums = MODE == SUM ? NT * kTR * 4 : 0;        // y of up to NT tokens
  static constexpr int kStages = NT == 16 ? 9 : NT == 64 ? (MODE == SUM ? 6 : 7) : NT == 128 ? 6 : 4;
  static constexpr int kBufs = NT > 128 ? 1 : 2;
  static constexpr uint32_t kColSF = (uint32_t)(kBufs * NT);          // first scale column
  static constexpr uint32_t kSFStage = 16u + 16u * kHalves;           // weights' 4 x 4, tokens' 4 x 4 a half
  static constexpr int kOffSums = kStages * kSlot;
  static constexpr int kOffTables = kOffSums + kSums;                 // first places, counts, experts
  static constexpr int kOffBars = kOffTables + kMaxExperts * 10;
  static constexpr size_t kBytes = 1024 + kOffBars + (2 * kStages + 4) * 8 + 16;
  static_assert(kColSF + kSFStage * kStages <= kTmemCols, "scale columns must fit the TMEM allocation");
  static_assert(kBytes <= 227 * 1024 && kSlot % 1024 == 0 && kOffX % 1024 == 0, "shared memory");
  static_assert(kLag < kStages, "a stage must be handed over before the ring comes round");
};

struct ExpertArgs {
  const uint8_t *xc, *xs;                    // rows of x: codes [.., K/2], scales [.., K/16]
  const float* xg;
  const uint8_t* w;                          // [experts][RT][C] blocks
  const float* wg;                           // [experts]
  const int32_t *offsets, *pairs;
  const float* weights;                      // SUM
  uint16_t* h;                               // UP: [n_pairs, inter]
  float* out;                                // SUM: y [tokens, N]; PART: [n_pairs, N]
  int tokens, top, experts, N, K, C, RT;     // N: columns of y, or of h
  int n_pairs;
  int cluster;
};

// A stretch of K of one tile: what a pass of the ring's roles works on.
struct Segment {
  int e, p0, n, rt, c0, nc;                  // expert, first place, places, row tile, first chunk, chunks
};

// The experts that have pairs, in order.
struct Table {
  const int *first, *count;
  const uint16_t* expert;
  int used;
  long long tiles;                           // stretches of up to NT pairs
};

// Every role walks the CTA's segments by itself, in the same order.
template <int NT, int MODE>
struct Walk {
  const Table& tb;
  const ExpertArgs& a;
  long long it, end, base;                   // UP, PART: item; SUM: unit (tile of pairs, chunk)
  int used;                                  // the table's entry that `base` belongs to
  int rank, step;
  NVFP4_DEVINL Walk(const Table& t, const ExpertArgs& args) : tb(t), a(args), base(0), used(0) {
    rank = args.cluster > 1 ? (int)cluster_ctarank() : 0;
    if (MODE == SUM) {
      const long long units = t.tiles * a.C;
      it = units * rank / a.cluster;
      end = units * (rank + 1) / a.cluster;
      step = 0;
    } else {
      it = blockIdx.x / a.cluster;
      end = t.tiles * a.RT;
      step = gridDim.x / a.cluster;
    }
  }
  NVFP4_DEVINL bool next(Segment& s) {
    if (it >= end) return false;
    int tt, t;
    if (MODE == SUM) {
      const long long tile = it / a.C;
      while (tile >= base + (tt = (tb.count[used] + NT - 1) / NT)) {
        base += tt;
        ++used;
      }
      t = (int)(tile - base);
      s.rt = blockIdx.x / a.cluster;
      s.c0 = (int)(it - tile * a.C);
      s.nc = (int)min((long long)(a.C - s.c0), end - it);
      it += s.nc;
    } else {
      while (it >= base + (long long)(tt = (tb.count[used] + NT - 1) / NT) * a.RT) {
        base += (long long)tt * a.RT;
        ++used;
      }
      const long long in = it - base;        // an expert's items: the tiles of pairs of a row tile follow one another
      s.rt = (int)(in / tt);
      t = (int)(in - (long long)s.rt * tt);
      s.c0 = a.C * rank / a.cluster;
      s.nc = a.C * (rank + 1) / a.cluster - s.c0;
      it += step;
    }
    s.e = tb.expert[used];
    s.p0 = tb.first[used] + t * NT;
    s.n = min(NT, tb.count[used] - t * NT);
    return true;
  }
};

// 32 rows of 16 bytes, one behind the other, to 4 columns of every lane quadrant: word w of row i to lane i, column w.
NVFP4_DEVINL void copy_scales(uint32_t tmem, uint64_t desc) {
  asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(tmem), "l"(desc) : "memory");
}
// Rows of 16 bytes without a swizzle: groups of 8 rows 128 bytes apart.
NVFP4_DEVINL uint64_t smem_desc_rows16(uint32_t saddr) {
  return (uint64_t)((saddr & 0x3FFFFu) >> 4) | ((uint64_t)(128 >> 4) << 16) | ((uint64_t)(128 >> 4) << 32) |
         ((uint64_t)1 << 46);
}

// E2M1 x E2M1, UE4M3 scales, K-major operands, M = 128 and N = n rounded up to 16, 32, 64 or 128 (an MMA takes 64 cycles
// whatever its N up to 128).
NVFP4_DEVINL uint32_t idesc_for(int n) {
  const uint32_t eighths = n <= 16 ? 2u : n <= 32 ? 4u : n <= 64 ? 8u : 16u;
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

NVFP4_DEVINL float silu_mul(float g, float u) { return __fdividef(g, 1.0f + __expf(-g)) * u; }

template <int NT, int MODE>
__global__ void __launch_bounds__(kThreads, 1) moe_experts_kernel(const ExpertArgs a) {
  using S = Shape<NT, MODE>;
  constexpr int kS = S::kStages;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  float* sums = reinterpret_cast<float*>(smem + S::kOffSums);
  int* t_first = reinterpret_cast<int*>(smem + S::kOffTables);
  int* t_count = t_first + kMaxExperts;
  uint16_t* t_expert = reinterpret_cast<uint16_t*>(t_count + kMaxExperts);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + S::kOffBars);
  uint64_t* empty = full + kS;
  uint64_t* acc_full = empty + kS;
  uint64_t* acc_empty = acc_full + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(acc_empty + 2);
  __shared__ int s_used, s_total;
  __shared__ long long s_tiles;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < kS; ++s) {
      mbar_init(&full[s], 1 + kLoaders / 32);
      mbar_init(&empty[s], 1);
    }
    for (int d = 0; d < 2; ++d) {
      mbar_init(&acc_full[d], 1);
      mbar_init(&acc_empty[d], 4);
    }
    fence_mbar_init();
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)),
                 "r"(kTmemCols));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  griddep_launch_dependents();
  griddep_wait();                            // the plan comes from a preceding kernel
  if (warp == 0) {
    // the experts that have pairs: a lane looks at `per` experts that follow one another
    const int per = (a.experts + 31) / 32;
    int used = 0;
    long long tiles = 0;
    bool bad = false;
    auto look = [&](auto take) {
      for (int i = 0; i < per; ++i) {
        const int e = lane * per + i;
        if (e >= a.experts) break;
        const int f = __ldcg(a.offsets + e), l = __ldcg(a.offsets + e + 1);
        const int lo = min(max(f, 0), a.n_pairs), hi = min(max(l, 0), a.n_pairs);
        bad = bad || f != lo || l != hi || hi < lo;
        if (hi > lo) take(e, lo, hi - lo);
      }
    };
    look([&](int, int, int n) {
      ++used;
      tiles += (n + NT - 1) / NT;
    });
    int at = used;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, at, o);
      if (lane >= o) at += x;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) tiles += __shfl_xor_sync(0xffffffffu, tiles, o);
    if (lane == 31) {
      s_used = at;
      s_tiles = tiles;
      s_total = min(max(__ldcg(a.offsets + a.experts), 0), a.n_pairs);
    }
    at -= used;
    look([&](int e, int lo, int n) {
      t_first[at] = lo;
      t_count[at] = n;
      t_expert[at] = (uint16_t)e;
      ++at;
    });
    if (bad) atomicOr(&g_nvfp4_device_error, NVFP4_DEVERR_MOE_RANGE);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const Table tb = {t_first, t_count, t_expert, s_used, s_tiles};
  Walk<NT, MODE> walk(tb, a);
  Segment sg;

  if (MODE == UP) {
    // rows of no pair are zero: one scale over all rows is taken of h
    const size_t per = (size_t)a.N / 8, end = (size_t)a.n_pairs * per;
    for (size_t i = s_total * per + blockIdx.x * kThreads + threadIdx.x; i < end; i += (size_t)gridDim.x * kThreads)
      reinterpret_cast<uint4*>(a.h)[i] = make_uint4(0u, 0u, 0u, 0u);
  }

  if (warp == 0) {
    // ---------------- weight blocks ----------------
    if (lane == 0) {
      int s = 0, k = 0;
      uint32_t phase = 0;
      bool ok = true;
      while (ok && walk.next(sg)) {
        const uint8_t* src = a.w + (((size_t)sg.e * a.RT + sg.rt) * a.C + sg.c0) * kBlock;
        for (int c = 0; c < sg.nc; ++c, src += kBlock) {
          if (k >= kS && !mbar_wait(&empty[s], phase ^ 1u)) {
            ok = false;
            break;
          }
          mbar_arrive_expect_tx(&full[s], kBlock);
          bulk_g2s(smem + s * S::kSlot, src, kBlock, &full[s]);
          ++k;
          if (++s == kS) { s = 0; phase ^= 1u; }
        }
      }
      // Not to leave with copies in flight: the last ones' waits (bounded; on the normal path long over).
      for (int j = k > kS ? k - kS : 0; j < k; ++j) mbar_wait(&full[j % kS], (j / kS) & 1);
    }
  } else if (warp == 1) {
    // ---------------- scales and products ----------------
    // The warp waits together; one lane then issues a stage's copies, products and commit in one branch, with the others
    // held at its end.  (Predicated one by one, with the other lanes free to run ahead, they faulted once several stages
    // were ready: operands are in uniform registers, which the lanes that run ahead overwrite.)
    const bool lead = elect_one() != 0u;
    const uint32_t base = smem_u32(smem);
    int s = 0, k = 0, seg = 0;
    uint32_t phase = 0;
    bool ok = true;
    while (ok && walk.next(sg)) {
      const int buf = seg % S::kBufs;
      if (seg >= S::kBufs && !mbar_wait_warp(&acc_empty[buf], (seg / S::kBufs - 1) & 1)) break;
      for (int c = 0; c < sg.nc; ++c) {
        if (!mbar_wait_warp(&full[s], phase)) {
          ok = false;
          break;
        }
        if (lead) {
          tc_fence_after();
          const uint32_t d = tmem + (uint32_t)(buf * NT), slot = base + (uint32_t)(s * S::kSlot);
          const uint64_t da = smem_desc_sw128(slot), db = smem_desc_sw128(slot + S::kOffX);
          const uint64_t dwa = smem_desc_rows16(slot + kWCodes), dxa = smem_desc_rows16(slot + S::kOffXS);
          const uint32_t sfa = tmem + S::kColSF + S::kSFStage * (uint32_t)s, sfb = sfa + 16u;
          const uint32_t idesc = idesc_for(sg.n);          // of the first 128 places; the others are another MMA's
          const int mmas = min(4, (a.K - (sg.c0 + c) * kChunk) / 64);
#pragma unroll
          for (int q = 0; q < 4; ++q)
            if (q < mmas) {
              copy_scales(sfa + 4u * q, dwa + (uint64_t)(32 * q));
              copy_scales(sfb + 4u * S::kHalves * q, dxa + (uint64_t)(32 * q));
              if (S::kHalves == 2 && sg.n > 128) copy_scales(sfb + 8u * q + 4u, dxa + (uint64_t)(128 + 32 * q));
            }
#pragma unroll
          for (int q = 0; q < 4; ++q)
            if (q < mmas) {
              const uint32_t acc = c > 0 || q > 0 ? 1u : 0u;
              mma_mxf4nvf4(d, da + 2 * q, db + 2 * q, idesc, sfa + 4u * q, sfb + 4u * S::kHalves * q, acc);
              if (S::kHalves == 2 && sg.n > 128)
                mma_mxf4nvf4(d + 128u, da + 2 * q, db + (uint64_t)(128 * 128 / 16 + 2 * q), idesc_for(sg.n - 128),
                             sfa + 4u * q, sfb + 8u * q + 4u, acc);
            }
          mma_commit(&empty[s]);
          if (c == sg.nc - 1) mma_commit(&acc_full[buf]);
        }
        __syncwarp();
        ++k;
        if (++s == kS) { s = 0; phase ^= 1u; }
      }
      ++seg;
    }
    if (k > 0) mbar_wait_warp(&empty[(k - 1) % kS], ((k - 1) / kS) & 1);   // not to leave with MMAs in flight
  } else if (warp < 6) {
    // ---------------- rows of x ----------------
    const int lt = threadIdx.x - 64;
    const size_t row_codes = (size_t)a.K / 2, row_scales = (size_t)a.K / 16;
    int s = 0, k = 0;
    uint32_t phase = 0;
    bool ok = true;
    // stage j's copies of this warp are in place: the MMAs read them through the asynchronous proxy
    auto hand_over = [&](int j) {
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncwarp();
      if (lane == 0) mbar_arrive(&full[j % kS]);
    };
    // the row of x at a place (the lowest one for a place of no pair)
    auto row_at = [&](int place) {
      if (MODE != UP) return place;
      const int pair = __ldcg(a.pairs + place);
      const bool in = pair >= 0 && pair < a.n_pairs;
      if (!in) atomicOr(&g_nvfp4_device_error, NVFP4_DEVERR_MOE_RANGE);
      return in ? pair / a.top : 0;
    };
    // a thread copies piece lt % 8 of rows lt / 8 + 16 i, and scale word lt % 4 of rows lt / 4 + 32 i
    constexpr int kRC = NT / 16, kRS = (NT + 31) / 32;
    const int piece = lt & 7, q = lt & 3, rc = lt >> 3, rs = lt >> 2;
    while (ok && walk.next(sg)) {
      int row_c[kRC], row_s[kRS];
#pragma unroll
      for (int i = 0; i < kRC; ++i) row_c[i] = rc + 16 * i < sg.n ? row_at(sg.p0 + rc + 16 * i) : -1;
#pragma unroll
      for (int i = 0; i < kRS; ++i) row_s[i] = rs + 32 * i < sg.n ? row_at(sg.p0 + rs + 32 * i) : -1;
      for (int c = sg.c0; c < sg.c0 + sg.nc; ++c) {
        if (k >= kS && !mbar_wait_warp(&empty[s], phase ^ 1u)) {
          ok = false;
          break;
        }
        const uint32_t slot = smem_u32(smem) + (uint32_t)(s * S::kSlot);
        if (c * 128 + piece * 16 < (int)row_codes) {
          const uint32_t dst = slot + S::kOffX + rc * 128 + ((piece ^ (rc & 7)) << 4);     // (16 i does not move the swizzle)
          const uint8_t* src = a.xc + c * 128 + piece * 16;
#pragma unroll
          for (int i = 0; i < kRC; ++i)
            if (row_c[i] >= 0) async_copy16(dst + 2048 * i, src + row_c[i] * row_codes);
        }
        if (c * 16 + q * 4 < (int)row_scales) {
          const uint32_t dst = slot + S::kOffXS + q * 512 + rs * 16;                         // row rs + 32 i: word i % 4
          const uint8_t* src = a.xs + c * 16 + q * 4;
#pragma unroll
          for (int i = 0; i < kRS; ++i)
            if (row_s[i] >= 0) async_copy4(dst + (i / 4) * 2048 + (i % 4) * 4, src + row_s[i] * row_scales);
        }
        async_commit();
        if (k >= kLag) {
          async_wait<kLag>();
          hand_over(k - kLag);
        }
        ++k;
        if (++s == kS) { s = 0; phase ^= 1u; }
      }
    }
    async_wait<0>();
    for (int j = k > kLag ? k - kLag : 0; j < k; ++j) hand_over(j);
  } else {
    // ---------------- the accumulator ----------------
    const int p = warp & 3, row = p * 32 + lane;
    const float xg = __ldcg(a.xg);
    if (MODE == SUM)
      for (int t = 0; t < a.tokens; ++t) sums[t * kTR + row] = 0.0f;
    int seg = 0;
    while (walk.next(sg)) {
      const int buf = seg % S::kBufs;
      const float scale = __fmul_rn(xg, __ldcg(a.wg + sg.e));
      if (!mbar_wait_warp(&acc_full[buf], (seg / S::kBufs) & 1)) break;
      tc_fence_after();
      const uint32_t d = tmem + ((uint32_t)(p * 32) << 16) + (uint32_t)(buf * NT);
      for (int m0 = 0; m0 < sg.n; m0 += 16) {
        float v[16];
        __syncwarp();
        read16(d + (uint32_t)m0, v);
        if (MODE == UP && a.cluster > 1) {
          // raw sums to the ring's memory (free: every MMA of the CTA's one item is done)
          float* stage = reinterpret_cast<float*>(smem);
#pragma unroll
          for (int i = 0; i < 16; ++i) stage[(m0 + i) * kTR + row] = v[i];
        } else if (MODE == UP) {
          // even lanes hold gates, odd ones ups: an even lane takes the even places of h row `row / 2`, an odd one the others
          const int i = sg.rt * 64 + row / 2;
#pragma unroll
          for (int j = 0; j < 16; j += 2) {
            const float a0 = v[j] * scale, a1 = v[j + 1] * scale;
            const float other = __shfl_xor_sync(0xffffffffu, lane & 1 ? a0 : a1, 1);
            const float hv = lane & 1 ? silu_mul(other, a1) : silu_mul(a0, other);
            const int m = m0 + j + (lane & 1);
            if (m < sg.n && i < a.N)
              a.h[(size_t)(sg.p0 + m) * a.N + i] = __bfloat16_as_ushort(__float2bfloat16_rn(hv));
          }
        } else if (MODE == SUM) {
          int pair[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) pair[i] = m0 + i < sg.n ? __ldcg(a.pairs + sg.p0 + m0 + i) : -1;
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            if (m0 + i >= sg.n) continue;
            if (pair[i] < 0 || pair[i] >= a.n_pairs) {
              if (row == 0) atomicOr(&g_nvfp4_device_error, NVFP4_DEVERR_MOE_RANGE);
              continue;
            }
            float* y = &sums[pair[i] / a.top * kTR + row];
            *y = fmaf(__ldcg(a.weights + pair[i]), v[i] * scale, *y);
          }
        } else {
          const int n = sg.rt * kTR + row;
          if (n < a.N) {
#pragma unroll
            for (int i = 0; i < 16; ++i)
              if (m0 + i < sg.n) a.out[(size_t)(sg.p0 + m0 + i) * a.N + n] = v[i] * scale;
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&acc_empty[buf]);
      ++seg;
    }
  }

  // ---------------- the cluster's parts ----------------
  __syncwarp();
  if (MODE != PART && a.cluster > 1) cluster_sync();
  if (MODE == SUM && warp >= 6) {
    const int row = (warp & 3) * 32 + lane, n = blockIdx.x / a.cluster * kTR + row;
    for (int t = walk.rank; t < a.tokens; t += a.cluster) {
      float y = 0.0f;
      for (int r = 0; r < a.cluster; ++r)                       // in the order of the ranks
        y += r == walk.rank ? sums[t * kTR + row] : ld_dsmem_f32(dsmem_addr(&sums[t * kTR + row], (uint32_t)r));
      if (n < a.N) a.out[(size_t)t * a.N + n] = y;
    }
  }
  if (MODE == UP && a.cluster > 1 && warp >= 6) {
    // a cluster has one item at most: its parts are in every CTA's stage; the ranks take its places in turn
    Walk<NT, MODE> again(tb, a);
    if (again.next(sg)) {
      const int row = (warp & 3) * 32 + lane, i = sg.rt * 64 + row / 2;
      const float scale = __fmul_rn(__ldcg(a.xg), __ldcg(a.wg + sg.e));
      const float* stage = reinterpret_cast<const float*>(smem);
      for (int m = walk.rank; m < sg.n; m += a.cluster) {
        float v = 0.0f;
        for (int r = 0; r < a.cluster; ++r) v += ld_dsmem_f32(dsmem_addr(&stage[m * kTR + row], (uint32_t)r));
        v *= scale;
        const float other = __shfl_xor_sync(0xffffffffu, v, 1);
        if (!(lane & 1) && i < a.N)
          a.h[(size_t)(sg.p0 + m) * a.N + i] = __bfloat16_as_ushort(__float2bfloat16_rn(silu_mul(v, other)));
      }
    }
  }
  tc_fence_before();
  __syncwarp();
  if (MODE != PART && a.cluster > 1) cluster_sync();              // (the others have read this CTA's memory)
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols));
  }
}

// y[t, n] = sum_j weights[t, j] part[places[t, j], n], in the order of j: a thread has V columns of a token.
struct CombineArgs {
  const float *part, *weights;
  const int32_t* places;
  float* y;
  int tokens, top, N, n_pairs;
};

template <int V>
__global__ void __launch_bounds__(256) moe_combine_kernel(const CombineArgs a) {
  griddep_launch_dependents();
  griddep_wait();
  const int n = (blockIdx.x * 256 + threadIdx.x) * V;
  if (n >= a.N) return;
  for (int t = blockIdx.y; t < a.tokens; t += gridDim.y) {
    float y[V] = {};
#pragma unroll 4
    for (int j = 0; j < a.top; ++j) {
      const int place = __ldcg(a.places + (size_t)t * a.top + j);
      if (place < 0 || place >= a.n_pairs) {
        if (place != -1) atomicOr(&g_nvfp4_device_error, NVFP4_DEVERR_MOE_RANGE);
        continue;
      }
      const float w = __ldcg(a.weights + (size_t)t * a.top + j);
      const float* src = a.part + (size_t)place * a.N + n;
      if constexpr (V == 4) {
        const float4 x = __ldcg(reinterpret_cast<const float4*>(src));
        y[0] = fmaf(w, x.x, y[0]);
        y[1] = fmaf(w, x.y, y[1]);
        y[2] = fmaf(w, x.z, y[2]);
        y[3] = fmaf(w, x.w, y[3]);
      } else {
        y[0] = fmaf(w, __ldcg(src), y[0]);
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

template <class Args>
cudaError_t launch(void (*kern)(Args), dim3 grid, int threads, size_t smem, int cluster, const Args& a, cudaStream_t stream) {
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
  return cudaLaunchKernelEx(&cfg, kern, a);
}

template <int NT, int MODE>
cudaError_t run(int grid, const ExpertArgs& a, cudaStream_t stream) {
  static PerDeviceInt done;
  cudaError_t err = cudaSuccess;
  done.get([](int, cudaError_t* e) -> int {
    *e = cudaFuncSetAttribute(moe_experts_kernel<NT, MODE>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              (int)Shape<NT, MODE>::kBytes);
    return *e == cudaSuccess ? 1 : 0;
  }, &err);
  if (err != cudaSuccess) return err;
  return launch(moe_experts_kernel<NT, MODE>, dim3((unsigned)grid), kThreads, Shape<NT, MODE>::kBytes, a.cluster, a, stream);
}

// Tokens up to which y is summed in shared memory.
constexpr int kSumTokens = 64;

// Most stretches of up to nt pairs that any plan of the pairs has.
long long most_tiles(const ExpertArgs& a, int nt) {
  const long long used = a.n_pairs < a.experts ? a.n_pairs : a.experts;
  return used + (a.n_pairs - used) / nt;
}

// Places of a tile: an expert of few tokens has few places; of many tokens, about the mean.
int tile_for(const ExpertArgs& a) {
  const long long used = a.n_pairs < a.experts ? a.n_pairs : a.experts;
  const long long mean = used > 0 ? a.n_pairs / used : 0;
  if (a.tokens <= 16) return 16;
  if (a.tokens <= 64 || mean <= 24) return 64;
  return mean <= 64 ? 128 : 256;
}

cudaError_t run_items(bool up, ExpertArgs a, cudaStream_t stream) {
  const int nt = tile_for(a), sms = device_sms();
  const long long items = most_tiles(a, nt) * a.RT;
  a.cluster = 1;
  if (up)
    while (a.cluster < kMaxCluster && items * a.cluster * 2 <= sms && a.C >= a.cluster * 2) a.cluster *= 2;
  long long grid = items * a.cluster;
  if (grid > sms) grid = sms;
  if (grid < 1) grid = 1;
  if (up) return nt == 16 ? run<16, UP>(grid, a, stream) : nt == 64 ? run<64, UP>(grid, a, stream)
                 : nt == 128 ? run<128, UP>(grid, a, stream) : run<256, UP>(grid, a, stream);
  return nt == 16 ? run<16, PART>(grid, a, stream) : nt == 64 ? run<64, PART>(grid, a, stream)
         : nt == 128 ? run<128, PART>(grid, a, stream) : run<256, PART>(grid, a, stream);
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
  return nvfp4_internal_cuda_status(launch(moe_pack_kernel, dim3((unsigned)grid), 256, 0, 1, a, stream));
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
  a.C = (K + kChunk - 1) / kChunk, a.RT = (rows + kTR - 1) / kTR;
  a.n_pairs = tokens * top_k;                // (checked to fit by check_experts before it is used)
  a.cluster = 1;
  return a;
}

}  // namespace

extern "C" nvfp4_status nvfp4_moe_gate_up(const uint8_t* xq, const uint8_t* xs, const float* xg, int tokens, int top_k,
                                          const int32_t* offsets, const int32_t* pairs, const uint8_t* wpacked,
                                          const float* wg, int experts, int inter, int K, uint16_t* h, cudaStream_t stream) {
  if (inter < 64 || inter > (1 << 19) || bad_matrix(experts, 2 * inter, K, true)) return NVFP4_ERR_SHAPE;
  if (tokens < 0 || top_k < 1 || top_k > kMaxTop || (long long)tokens * top_k > 0x7FFFFFFFll) return NVFP4_ERR_SHAPE;
  ExpertArgs a = experts_args(xq, xs, xg, tokens, top_k, offsets, pairs, wpacked, wg, experts, 2 * inter, K);
  a.h = h, a.N = inter;
  const nvfp4_status cs = check_experts(xq, xs, xg, a, h);
  if (cs != NVFP4_OK || tokens == 0) return cs;
  const nvfp4_status ds = nvfp4_internal_check_device();
  if (ds != NVFP4_OK) return ds;
  return nvfp4_internal_cuda_status(run_items(true, a, stream));
}

extern "C" size_t nvfp4_moe_down_workspace_bytes(int tokens, int top_k, int N) {
  if (tokens <= kSumTokens || top_k < 1 || top_k > kMaxTop || N < 1 || N > (1 << 20)) return 0;
  return (size_t)tokens * top_k * N * sizeof(float);
}

extern "C" nvfp4_status nvfp4_moe_down(const uint8_t* hq, const uint8_t* hs, const float* hg, int tokens, int top_k,
                                       const int32_t* offsets, const int32_t* pairs, const int32_t* places,
                                       const float* weights, const uint8_t* wpacked, const float* wg, int experts, int N,
                                       int K, float* y, void* workspace, size_t workspace_bytes, cudaStream_t stream) {
  if (bad_matrix(experts, N, K, false)) return NVFP4_ERR_SHAPE;
  if (tokens < 0 || top_k < 1 || top_k > kMaxTop || (long long)tokens * top_k > 0x7FFFFFFFll) return NVFP4_ERR_SHAPE;
  ExpertArgs a = experts_args(hq, hs, hg, tokens, top_k, offsets, pairs, wpacked, wg, experts, N, K);
  a.N = N, a.weights = weights;
  const nvfp4_status cs = check_experts(hq, hs, hg, a, y);
  if (cs != NVFP4_OK || tokens == 0) return cs;
  if (!places || !weights) return NVFP4_ERR_NULL;
  const size_t need = nvfp4_moe_down_workspace_bytes(tokens, top_k, N);
  if (need > 0 && !workspace) return NVFP4_ERR_NULL;
  if (!nvfp4_internal_aligned(places, 4) || !nvfp4_internal_aligned(weights, 4) || !nvfp4_internal_aligned(workspace, 16))
    return NVFP4_ERR_ALIGN;
  if (workspace_bytes < need) return NVFP4_ERR_SHAPE;
  const nvfp4_status ds = nvfp4_internal_check_device();
  if (ds != NVFP4_OK) return ds;
  if (need == 0) {
    a.out = y;
    const int sms = device_sms();
    while (a.cluster < kMaxCluster && a.RT * (a.cluster + 1) <= sms) ++a.cluster;
    return nvfp4_internal_cuda_status(tokens <= 16 ? run<16, SUM>(a.RT * a.cluster, a, stream)
                                                   : run<64, SUM>(a.RT * a.cluster, a, stream));
  }
  a.out = static_cast<float*>(workspace);
  cudaError_t e = run_items(false, a, stream);
  if (e != cudaSuccess) return nvfp4_internal_cuda_status(e);
  CombineArgs c = {a.out, weights, places, y, tokens, top_k, N, a.n_pairs};
  const int per = N % 4 == 0 ? 1024 : 256;
  const dim3 grid((unsigned)((N + per - 1) / per), (unsigned)(tokens < 65535 ? tokens : 65535));
  e = N % 4 == 0 ? launch(moe_combine_kernel<4>, grid, 256, 0, 1, c, stream)
                 : launch(moe_combine_kernel<1>, grid, 256, 0, 1, c, stream);
  return nvfp4_internal_cuda_status(e);
}
