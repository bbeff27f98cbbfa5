// Attention over the NVFP4 KV cache for many query rows a request (prompt
// chunks), on the 5th-generation tensor cores:
//   S = Q K^T,  P = 2^(f S - m),  O += P V,  out = O / sum P
// for tiles of 2 x 128 query rows of one (request, kv head), 128 keys a step.
//
// With R query rows a kv head a key costs 4 R D operations and 18 D / 16 bytes:
// bound by the matrix units (2048 cycles a step of 256 rows at D = 128), close
// behind by shared memory, which feeds them 128 bytes a cycle (about 2300 cycles),
// and by the exponentials (32768 a step).  An instruction with 128 rows takes 64
// cycles or more whatever its N, so a step has 128 keys: both products have N = 128.
// The weights are an operand in TMEM (no trip through shared memory), the queries
// (FP16 of q / 2^e, as in the decode kernel) one in shared memory, because scores
// and output of both halves fill the TMEM:
//   half h: S at columns 256 h [128, FP32], O at 256 h + 128 [D], P [FP16] over each thread's own scores: keys 0-63
//   at 256 h [32], keys 64-127 at 256 h + 64 [32].
// K and V are dequantized once a step for both halves, as [token][element] in
// 128-byte swizzled panels of 64 elements: K is then a K-major operand, V one whose
// rows are contiguous (no transposition on the way).
//
// Warps: 0-7 and 8-15 softmax of the two halves (two threads a row, 64 keys each: one thread
// for all 128 took 2900 cycles, more than the products under which it should hide), 16-19
// dequantize (two 16-token groups each), 20 copies the cache's groups in, 21 issues the
// products; one half's softmax runs under the other's products.  A tile of 128 rows
// or fewer stands in both halves, which take every second step and are put together at
// the end (with one half at work alone, its softmax and its products in turn, 64 rows
// over 4 x 8000 keys took 52 us instead of 44).  The maximum that the
// weights refer to moves only when a row's scores exceed it by 2^13 (then O is
// rescaled in TMEM); up to there FP16 holds the weights as exactly as below 1.
// Every wait is bounded and an abort flag ends the others.
// Tiles are handed out from a counter, the longest of a request first.  Where they are fewer than fill the SMs, or
// their lengths differ, their keys are cut into pieces of one size, kMinSteps steps or more, which go through records
// in the workspace (128 KB each), and a second launch merges them, all SMs at work on it (merged by the last piece to
// arrive instead, one CTA read up to 32 records: 115 us for 128 rows over 16000 keys, 64/8 heads, now 52).  With as
// many pieces for every tile instead of one size, 64 rows over 16 requests of 500 to 16384 keys took 179 us, not 137.
// 2 x 1024 prompt tokens over 4096 and 8192 keys (64/8 heads, D = 128: 377 GFLOP): 422 us, 890 TFLOP/s, a step of 256
// rows in 4400 cycles, of which a half's softmax has 1800 and the products 2050.
#include <math.h>

#include "kv_attention.cuh"
#include "tcgen05.cuh"

NVFP4_DEFINE_ERROR_READER(nvfp4_internal_read_error_kv_attention_tc)

namespace {

constexpr int kHalfRows = 128;          // query rows of a half: a thread each
constexpr int kRows = 2 * kHalfRows;    // of a tile
constexpr int kKeys = 128;              // keys of a step
constexpr int kGroups = kKeys / kKvGroup;
constexpr int kRing = 3;                // raw steps in flight
constexpr int kDequantWarps = 4;        // each takes kGroups / kDequantWarps groups
constexpr int kSoftWarps = 16;
constexpr int kThreads = (kSoftWarps + kDequantWarps + 2) * 32;
constexpr int kCopyWarp = kSoftWarps + kDequantWarps, kMmaWarp = kCopyWarp + 1;
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kColHalf = 256, kColO = 128;
constexpr uint32_t kSpinLimit = 1u << 22;  // polls of a wait (each suspends for a while): far beyond any step
constexpr float kSlack = 13.0f;         // log2 units a score may exceed the maximum in use (FP16 holds 2^15)

template <int D>
struct Shape {
  static constexpr int kRaw = kGroups * KvLayout<D>::kGroupBytes;
  static constexpr int kPanel = kKeys * 128;              // 128 rows x 64 elements
  static constexpr int kTile = kKeys * D * 2;             // Q of a half, K or V of a step, FP16
  static constexpr int kOffQ = 0;                         // [2] halves
  static constexpr int kOffK = 2 * kTile;
  static constexpr int kOffV = 3 * kTile;                 // [2] steps
  static constexpr int kOffRaw = 5 * kTile;               // [kRing]
  static constexpr int kOffBar = kOffRaw + kRing * kRaw;
  static constexpr int kBars = 2 * kRing + 2 + 4 + 6 + 1;
  static constexpr int kOffWords = kOffBar + kBars * 8;   // TMEM address, abort flag, two tiles (5 each), groups
                                                          // present (kRing + 4), pieces
  static constexpr int kOffMax = kOffWords + 32 * 4;      // [2 steps][2 halves][2 threads][kHalfRows] maxima, then sums
  static constexpr int kOffF = kOffMax + 8 * kHalfRows * 4;   // [2][kHalfRows] score factors
  static constexpr int kRecord = kRows * (D + 2);         // floats of a piece's record: O, then the maxima in use, then the sums
  static_assert(kRecord <= kTcRecord, "the workspace");
  static constexpr int kSmem = kOffF + kRows * 4 + 1024; // + alignment of the swizzled panels
  // instruction descriptors: FP32 accumulator, FP16 operands, M = 128; N = keys, and N = D with B's rows contiguous
  static constexpr uint32_t kIdescS = (1u << 4) | ((uint32_t)(kKeys >> 3) << 17) | ((uint32_t)(kHalfRows >> 4) << 24);
  static constexpr uint32_t kIdescO =
      (1u << 4) | (1u << 16) | ((uint32_t)(D >> 3) << 17) | ((uint32_t)(kHalfRows >> 4) << 24);
};

// The products are issued by one lane of a warp that stays together: what the instructions take is then uniform
// over the warp and is kept in uniform registers (issued from a branch of one lane, 32 of them took 3700 cycles).
// D (+)= A . B^T, A in shared memory.
NVFP4_DEVINL void mma_f16_ss(uint32_t lead, uint32_t d_tmem, uint64_t da, uint64_t db, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(da), "l"(db), "r"(idesc), "r"(acc), "r"(lead)
      : "memory");
}
// A in TMEM (two FP16 of the contraction to a column).
NVFP4_DEVINL void mma_f16_ts(uint32_t lead, uint32_t d_tmem, uint32_t a_tmem, uint64_t db, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(db), "r"(idesc), "r"(acc), "r"(lead)
      : "memory");
}
NVFP4_DEVINL void commit(uint32_t lead, uint64_t* bar) {
  asm volatile(
      "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %1, 0;\n\t"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(smem_u32(bar)),
      "r"(lead)
      : "memory");
}

// Operand whose rows (N) are contiguous, 128-byte swizzle: 64-element panels `panel` bytes apart, groups of 8
// contraction indices 1024 bytes apart.
NVFP4_DEVINL uint64_t smem_desc_mn_sw128(uint32_t saddr, uint32_t panel) {
  return (uint64_t)((saddr & 0x3FFFFu) >> 4) | ((uint64_t)(panel >> 4) << 16) | ((uint64_t)(1024 >> 4) << 32) |
         ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}

#define R4(a, i) "=r"(a[i]), "=r"(a[i + 1]), "=r"(a[i + 2]), "=r"(a[i + 3])
#define W4(a, i) "r"(a[i]), "r"(a[i + 1]), "r"(a[i + 2]), "r"(a[i + 3])
// 32 columns of this warp's lane quadrant; the loaded values may be used after tmem_wait_ld.
NVFP4_DEVINL void tmem_ld32(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,"
      "%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : R4(r, 0), R4(r, 4), R4(r, 8), R4(r, 12), R4(r, 16), R4(r, 20), R4(r, 24), R4(r, 28)
      : "r"(taddr));
}
NVFP4_DEVINL void tmem_st32(uint32_t taddr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,"
      "%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31};" ::W4(r, 0),
      W4(r, 4), W4(r, 8), W4(r, 12), W4(r, 16), W4(r, 20), W4(r, 24), W4(r, 28), "r"(taddr)
      : "memory");
}
NVFP4_DEVINL void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15};" ::W4(r, 0),
      W4(r, 4), W4(r, 8), W4(r, 12), "r"(taddr)
      : "memory");
}
#undef R4
#undef W4
// The values pass through the wait, so that nothing uses them before it.
NVFP4_DEVINL void tmem_wait_ld(uint32_t (&r)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int i = 0; i < 32; ++i) asm volatile("" : "+r"(r[i]));
}
NVFP4_DEVINL void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Waits for the phase of `bar` with this parity: bounded; false, and the abort flag up, when it gives up, or when
// another wait has.
NVFP4_DEVINL bool wait(uint64_t* bar, uint32_t parity, volatile uint32_t* abort_flag) {
  for (uint32_t i = 0; i < kSpinLimit; ++i) {
    if (mbar_try_wait(bar, parity & 1u)) return true;
    if ((i & 1023u) == 1023u && *abort_flag) return false;
  }
  atomicOr(&g_nvfp4_device_error, NVFP4_DEVERR_MBAR_TIMEOUT);
  *abort_flag = 1u;
  return false;
}

constexpr int kMinSteps = 4;            // below this a record costs more than the piece saves

struct Tile {
  int b, kvh, row0, piece, number;
};

// Row tiles of a request.
NVFP4_DEVINL int request_tiles(const AttnArgs& a, const Request& r) {
  return (int)(((long long)r.rows * a.group + kRows - 1) / kRows);
}

// Steps of a request's tiles, at most.
NVFP4_DEVINL int request_steps(const AttnArgs& a, const Request& r) {
  const int all = (r.len + kKeys - 1) / kKeys;
  // the keys that the rows of a tile see: a window's and one more for each of its further tokens
  const long long seen = (long long)a.window + min(kRows / a.group + 1, r.rows);
  return a.window > 0 ? (int)min((long long)all, seen / kKeys + 2) : all;
}

// Pieces of a tile of a request, at most, for pieces of about `size` steps (0: not cut).
NVFP4_DEVINL int request_pieces(const AttnArgs& a, const Request& r, int size) {
  return size > 0 ? max((request_steps(a, r) + size - 1) / size, 1) : 1;
}

// The steps of a piece, 0 if no tile is cut: the smallest size with as many pieces as SMs, or twice as many where that
// is much shorter, so that lengths that differ fill the SMs too.  One warp.
NVFP4_DEVINL int piece_size(const AttnArgs& a, int sms, int lane, bool report) {
  long long tiles_all = 0;
  float sum = 0.0f;                                       // (an estimate is enough)
  int longest = 0, n0 = 0, s0 = 0;                        // tiles and steps of request `lane`
  for (int b = lane; b < a.batch; b += 32) {
    const Request r = get_request(a, b, report);
    const long long n = (long long)request_tiles(a, r) * a.kv_heads;
    if (n == 0) continue;
    const int s = request_steps(a, r);
    tiles_all += n;
    sum += (float)n * (float)s;
    longest = max(longest, s);
    if (b == lane) n0 = (int)min(n, (long long)kTcPieces), s0 = s;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    tiles_all += __shfl_xor_sync(0xffffffffu, tiles_all, o);
    sum += __shfl_xor_sync(0xffffffffu, sum, o);
  }
  longest = __reduce_max_sync(0xffffffffu, longest);
  if (tiles_all >= a.pieces || longest <= kMinSteps) return 0;
  // sum / target will do where the tiles' last pieces are whole, sum / (target - tiles) always, and often one between
  const int tiles = (int)tiles_all;
  int best = 0, best_cost = (tiles + sms - 1) / sms * longest;
#pragma unroll 1
  for (int rounds = 1; rounds <= 2; ++rounds) {
    const int target = min(rounds * sms, a.pieces);
    if (tiles >= target) continue;
#pragma unroll 1
    for (int j = 0; j <= 4; ++j) {
      const int parts = target - tiles * j / 4;
      const int size = max((int)min(ceilf(__fdividef(sum, (float)parts)), 1e9f), kMinSteps);
      int pieces = 0, most = 0;                           // of all; steps of the longest one
      auto add = [&](int n, int s) {
        const int p = (s + size - 1) / size;
        pieces = min(pieces + n * min(p, kTcPieces + 1), kTcPieces + 1);
        most = max(most, (s + p - 1) / p);
      };
      if (n0 > 0 && s0 > 0) add(n0, s0);
      else pieces = n0;
      for (int b = lane + 32; b < a.batch; b += 32) {
        const Request r = get_request(a, b, false);
        const int n = request_tiles(a, r) * a.kv_heads, s = request_steps(a, r);
        if (n > 0 && s > 0) add(n, s);
        else pieces = min(pieces + n, kTcPieces + 1);
      }
      pieces = (int)__reduce_add_sync(0xffffffffu, (uint32_t)pieces);
      if (pieces > target) continue;
      const int cost = rounds * max((int)__reduce_max_sync(0xffffffffu, (uint32_t)most), kMinSteps);
      // a second round has to gain a fifth: its pieces have queries to load and records to write, too
      if (rounds == 1 ? cost < best_cost : 5ll * cost < 4ll * best_cost) {
        best = size;
        best_cost = cost;
      }
      break;
    }
  }
  return best;
}

// The steps of a tile and how many of them a piece has.
struct Steps {
  int lo, hi, first, all, piece;                          // keys [lo, hi]; first step, steps, steps of a piece
  NVFP4_DEVINL Steps(const AttnArgs& a, const Request& rq, int row0, int n_rows, int size) {
    const int p_first = rq.len - rq.rows + row0 / a.group;
    hi = rq.len - rq.rows + (row0 + n_rows - 1) / a.group;
    lo = a.window > 0 ? max(p_first - a.window + 1, 0) : 0;
    first = lo / kKeys;
    all = hi < 0 ? 0 : max(hi / kKeys + 1 - first, 0);
    // (the same for every tile of the request, so that none has more pieces than are counted for it)
    const int pieces = request_pieces(a, rq, size);
    piece = size > 0 ? max(kMinSteps, (request_steps(a, rq) + pieces - 1) / pieces) : all;
  }
};

// Piece number t, or the first piece of tile number t, -> request, kv head, first row, piece of the tile and its number
// (b = -1: there is no such piece).  One warp; the requests are summed 32 at a time.  The last rows of a request, which
// see most keys, come first.
template <bool TILES>
NVFP4_DEVINL Tile find(const AttnArgs& a, int t, int size, int lane) {
  long long before = 0, numbers = 0;                      // tiles are few where TILES: some are cut
  for (int b0 = 0; b0 < a.batch; b0 += 32) {
    int tiles = 0, pieces = 1;
    if (b0 + lane < a.batch) {
      const Request r = get_request(a, b0 + lane, false);
      tiles = request_tiles(a, r);
      if (size > 0 && tiles > 0) pieces = request_pieces(a, r, size);
    }
    const int each = TILES ? 1 : pieces;
    long long inc = (long long)tiles * a.kv_heads * each;
    int inc_n = TILES ? (int)inc * pieces : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long v = __shfl_up_sync(0xffffffffu, inc, o);
      const int w = TILES ? __shfl_up_sync(0xffffffffu, inc_n, o) : 0;
      if (lane >= o) inc += v, inc_n += w;
    }
    const uint32_t past = __ballot_sync(0xffffffffu, before + inc > t);
    if (past) {
      const int l = __ffs(past) - 1;
      const int n = __shfl_sync(0xffffffffu, tiles, l), p = __shfl_sync(0xffffffffu, pieces, l);
      const int per = TILES ? 1 : p;
      const int i = (int)(t - before - (__shfl_sync(0xffffffffu, inc, l) - (long long)n * a.kv_heads * per));
      const int tile = per > 1 ? i / per : i, piece = i - tile * per;
      const int number = TILES ? (int)numbers + __shfl_sync(0xffffffffu, inc_n, l) - n * a.kv_heads * p + tile * p : t;
      return Tile{b0 + l, tile % a.kv_heads, (n - 1 - tile / a.kv_heads) * kRows, piece, number};
    }
    before += __shfl_sync(0xffffffffu, inc, 31);
    if (TILES) numbers += __shfl_sync(0xffffffffu, inc_n, 31);
  }
  return Tile{-1, 0, 0, 0, 0};
}

// Dequantizes the keys of one 16-token group into rows [16 g, 16 g + 16) of the K tile.
template <int D>
NVFP4_DEVINL void dequantize_keys(const uint8_t* raw, uint8_t* k_tile, int g, int lane) {
  using L = KvLayout<D>;
  const int r = lane >> 2, c = lane & 3;
  constexpr int kPanel = kKeys * 128;
  // lane (r, c) has D/4 elements of the tokens at pos r and r + 8
  uint32_t sc[2][D / 64];
  if constexpr (D == 128) {
    const uint32_t w = *reinterpret_cast<const uint32_t*>(raw + L::kOffKScale + lane * 4);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t h = e4m3x2_to_f16(w >> (16 * i));
      sc[i][0] = __byte_perm(h, h, 0x1010);
      sc[i][1] = __byte_perm(h, h, 0x3232);
    }
  } else {
    const uint32_t h = e4m3x2_to_f16(*reinterpret_cast<const uint16_t*>(raw + L::kOffKScale + lane * 2));
    sc[0][0] = __byte_perm(h, h, 0x1010);
    sc[1][0] = __byte_perm(h, h, 0x3232);
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int row = g * kKvGroup + 4 * (r >> 1) + 2 * i + (r & 1);
    const uint8_t* p = raw + (8 * i + r) * (D / 2) + c * (D / 8);
    if constexpr (D == 128) {
      // a word is an 8-element piece; lanes with c >= 2 (the second panel) take theirs in another order, so that
      // the pieces a quarter warp stores together lie in different banks
      uint4 v = lds128(p);
      const bool swap = c >= 2;
      const uint32_t w[4] = {swap ? v.z : v.x, swap ? v.w : v.y, swap ? v.x : v.z, swap ? v.y : v.w};
      const uint32_t s_lo = swap ? sc[i][1] : sc[i][0], s_hi = swap ? sc[i][0] : sc[i][1];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        uint32_t h[4];
        e2m1x8_to_f16(w[j], h);
        const uint32_t s = j < 2 ? s_lo : s_hi;
        const int piece = ((c & 1) * 4 + (j ^ (swap ? 2 : 0))) ^ (row & 7);
        *reinterpret_cast<uint4*>(k_tile + (c >> 1) * kPanel + row * 128 + piece * 16) =
            make_uint4(hmul2(h[0], s), hmul2(h[1], s), hmul2(h[2], s), hmul2(h[3], s));
      }
    } else {
      const uint2 v = lds64(p);
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        uint32_t h[4];
        e2m1x8_to_f16(j == 0 ? v.x : v.y, h);
        const int piece = (2 * c + j) ^ (row & 7);
        *reinterpret_cast<uint4*>(k_tile + row * 128 + piece * 16) =
            make_uint4(hmul2(h[0], sc[i][0]), hmul2(h[1], sc[i][0]), hmul2(h[2], sc[i][0]), hmul2(h[3], sc[i][0]));
      }
    }
  }
}

// And its values into the V tile.  live: tokens that exist.
template <int D>
NVFP4_DEVINL void dequantize_values(const uint8_t* raw, uint8_t* v_tile, int g, int live, int lane) {
  using L = KvLayout<D>;
  const int r = lane >> 2, c = lane & 3;
  constexpr int kPanel = kKeys * 128;
  // lane (r, c) has D/8 elements of tokens 4 c .. 4 c + 3
  uint32_t sw = *reinterpret_cast<const uint32_t*>(raw + L::kOffVScale + (D == 128 ? r : r >> 1) * 16 + 4 * c);
  const int mine = live - 4 * c;
  if (mine < 4) sw &= mine > 0 ? (1u << (8 * mine)) - 1u : 0u;      // what lies behind the last key may be NaN
  const uint32_t s01 = e4m3x2_to_f16(sw), s23 = e4m3x2_to_f16(sw >> 16);
  const uint32_t vs[4] = {__byte_perm(s01, s01, 0x1010), __byte_perm(s01, s01, 0x3232), __byte_perm(s23, s23, 0x1010),
                          __byte_perm(s23, s23, 0x3232)};
  uint32_t x[4][D / 64];
  if constexpr (D == 128) {
    const uint8_t* q = raw + L::kOffV + (r >> 1) * 256 + (r & 1) * 64 + c * 16;
    const uint4 v0 = lds128(q), v1 = lds128(q + 128);
    const bool swap = c >= 2;             // as above
    x[0][0] = swap ? v0.y : v0.x, x[0][1] = swap ? v0.x : v0.y, x[1][0] = swap ? v0.w : v0.z, x[1][1] = swap ? v0.z : v0.w;
    x[2][0] = swap ? v1.y : v1.x, x[2][1] = swap ? v1.x : v1.y, x[3][0] = swap ? v1.w : v1.z, x[3][1] = swap ? v1.z : v1.w;
  } else {
    const uint4 v = lds128(raw + L::kOffV + r * 64 + c * 16);
    x[0][0] = v.x, x[1][0] = v.y, x[2][0] = v.z, x[3][0] = v.w;
  }
#pragma unroll
  for (int t = 0; t < 4; ++t) {
    const int row = g * kKvGroup + 4 * c + t;
#pragma unroll
    for (int j = 0; j < D / 64; ++j) {
      uint32_t h[4];
      e2m1x8_to_f16(x[t][j], h);
      const int piece = D == 128 ? (((r & 3) * 2 + (j ^ (c >> 1))) ^ (row & 7)) : (r ^ (row & 7));
      *reinterpret_cast<uint4*>(v_tile + (D == 128 ? (r >> 2) * kPanel : 0) + row * 128 + piece * 16) =
          make_uint4(hmul2(h[0], vs[t]), hmul2(h[1], vs[t]), hmul2(h[2], vs[t]), hmul2(h[3], vs[t]));
    }
  }
}

template <int D, class T>
__global__ void __launch_bounds__(kThreads, 1) kv_attention_tc_kernel(const AttnArgs a) {
  using S = Shape<D>;
  using L = KvLayout<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + (1024u - (smem_u32(smem_raw) & 1023u)) % 1024u;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + S::kOffBar);
  uint64_t *raw_full = bars, *raw_free = raw_full + kRing, *k_full = raw_free + kRing, *k_free = k_full + 1;
  uint64_t *v_full = k_free + 1, *v_free = v_full + 2;                  // [2] steps
  uint64_t *s_full = v_free + 2, *p_full = s_full + 2, *pv_done = p_full + 2, *q_full = pv_done + 2;   // [2] halves
  volatile uint32_t* words = reinterpret_cast<volatile uint32_t*>(smem + S::kOffWords);
  volatile uint32_t* abort_flag = words + 1;
  volatile int* s_tile = reinterpret_cast<volatile int*>(words + 2);
  volatile uint32_t* raw_have = words + 12;              // [kRing] groups that a raw step brings
  volatile uint32_t* kv_have = words + 12 + kRing;       // [4] steps
  if (tid == 0) {
    for (int i = 0; i < kRing; ++i) {
      mbar_init(&raw_full[i], 1);
      mbar_init(&raw_free[i], kDequantWarps);
    }
    mbar_init(k_full, kDequantWarps);
    mbar_init(k_free, 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&v_full[i], kDequantWarps);
      mbar_init(&v_free[i], 1);
      mbar_init(&s_full[i], 1);
      mbar_init(&p_full[i], kSoftWarps / 2);
      mbar_init(&pv_done[i], 1);
    }
    mbar_init(q_full, kSoftWarps);
    *abort_flag = 0u;
  }
  fence_mbar_init();
  griddep_wait();
  fence_proxy_async_global();
  if (warp == kMmaWarp) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32(const_cast<uint32_t*>(words))),
                 "r"(kTmemCols));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = words[0];
  // only now: a dependent kernel that came first to the TMEM would wait for this one, and this one for it
  griddep_launch_dependents();
  const float kg = *a.k_global, vg = *a.v_global;
  // steps of this CTA so far (they give ring slot, operand buffer and the parities of their barriers), those of the
  // two halves, tiles
  uint32_t step = 0, step_a = 0, step_b = 0, tiles = 0;
  uint32_t copied = 0;                                  // steps whose copies this warp has started

  volatile uint32_t* s_size = words + 12 + kRing + 4;   // steps of a piece, 0 if no tile is cut
  // the copy warp takes the pieces of tiles from the counter, each while the one before it is worked on
  auto take_tile = [&](uint32_t n) {
    uint32_t t = 0;
    if (lane == 0) t = atomicAdd(&a.counters[kTileCounter], 1u);
    t = __shfl_sync(0xffffffffu, t, 0);
    const Tile tile = find<false>(a, (int)t, (int)*s_size, lane);
    if (lane == 0) {
      volatile int* to = s_tile + 5 * (n & 1u);
      to[0] = tile.b, to[1] = tile.kvh, to[2] = tile.row0, to[3] = tile.piece, to[4] = (int)t;
    }
  };
  if (warp == kCopyWarp) {
    const int size = piece_size(a, gridDim.x, lane, blockIdx.x == 0);
    if (lane == 0) {
      *s_size = (uint32_t)size;
      if (blockIdx.x == 0) a.counters[kTileCounter + 2] = (uint32_t)size;   // for the merge
    }
    __syncwarp();
    take_tile(0);
  }
  __syncthreads();
  const int size = (int)*s_size;
  for (;;) {
    const volatile int* from = s_tile + 5 * (tiles & 1u);
    const int b = from[0], kvh = from[1], row0 = from[2], piece = from[3], record = from[4];
    if (b < 0) break;
    const Request rq = get_request(a, b, false);
    const int n_rows = (int)min((long long)kRows, (long long)rq.rows * a.group - row0);
    const bool both = n_rows > kHalfRows;
    // a tile of one piece (also one without keys) is written at once
    const Steps steps(a, rq, row0, n_rows, size);
    const int lo = steps.lo, hi = steps.hi;               // keys that some row of the tile sees
    const bool whole = steps.all <= steps.piece, idle = piece > 0 && piece * steps.piece >= steps.all;
    const int step0 = steps.first + piece * steps.piece;
    const int n = idle ? 0 : min(steps.piece, steps.all - piece * steps.piece);

    if (warp < kSoftWarps) {
      // ================ softmax of a half: two threads a row, `part` 0 and 1 ================
      const int half = warp >> 3, part = (warp >> 2) & 1, r = (warp & 3) * 32 + lane, row_h = both ? half * kHalfRows : 0;
      const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
      const uint32_t col_s = tmem + kColHalf * half + 64 * part + lanes, col_o = tmem + kColHalf * half + kColO + lanes;
      const int row = row0 + row_h + r;
      const bool mine = row_h + r < n_rows;
      const int tok = rq.first + row / a.group, head = kvh * a.group + row % a.group;
      float* s_max = reinterpret_cast<float*>(smem + S::kOffMax) + half * 2 * kHalfRows + r;   // + part, + step
      constexpr int kStepMax = 4 * kHalfRows;
      auto meet = [&]() {                               // the half's 8 warps
        asm volatile("bar.sync %0, %1;" ::"r"(1 + half), "r"(kSoftWarps / 2 * 32) : "memory");
      };
      auto meet_all = [&]() {                           // both halves
        asm volatile("bar.sync 3, %0;" ::"r"(kSoftWarps * 32) : "memory");
      };
      // queries: a warp a row at a time (whole rows a load), eight in flight
      float* s_f = reinterpret_cast<float*>(smem + S::kOffF);
      if (!idle) {
        constexpr int E = D / 32, kBatch = 8;
        const int warp_rows = (both ? kRows : kHalfRows) / kSoftWarps;
#pragma unroll 1
        for (int j0 = 0; j0 < warp_rows; j0 += kBatch) {
          float v[kBatch][E];
#pragma unroll
          for (int j = 0; j < kBatch; ++j) {
            const int rt = warp * warp_rows + j0 + j, rr = row0 + rt;
            const bool there = rt < n_rows;
            const T* q = static_cast<const T*>(a.q) +
                         (there ? (rq.first + rr / a.group) * a.q_ts + (kvh * a.group + rr % a.group) * a.q_hs : 0) + lane * E;
#pragma unroll
            for (int e = 0; e < E; ++e) v[j][e] = there ? load_q(q + e) : 0.0f;
          }
#pragma unroll
          for (int j = 0; j < kBatch; ++j) {
            const int rt = warp * warp_rows + j0 + j, rh = rt % kHalfRows;
            float big = 0.0f;
#pragma unroll
            for (int e = 0; e < E; ++e) big = fmaxf(big, fabsf(v[j][e]));
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, o));
            float down, up;
            power_of_two(big, down, up);
            if (lane == 0) s_f[rt] = score_factor(a.scale * kLog2e * kg * up);
            // element lane * E: panel, 16-byte piece, place in it
            const int e0 = lane * E;
            uint8_t* sq = smem + S::kOffQ + rt / kHalfRows * S::kTile + (e0 / 64) * S::kPanel + rh * 128 +
                          (((e0 / 8) & 7) ^ (rh & 7)) * 16 + (e0 & 7) * 2;
            if constexpr (E == 4)
              *reinterpret_cast<uint2*>(sq) = make_uint2(pack_f16(v[j][0] * down, v[j][1] * down),
                                                         pack_f16(v[j][2] * down, v[j][3] * down));
            else
              *reinterpret_cast<uint32_t*>(sq) = pack_f16(v[j][0] * down, v[j][1] * down);
          }
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        if (both) meet();                               // the factors are there
        else meet_all();
      }
      const float f = idle ? 1.0f : s_f[row_h + r];
      __syncwarp();
      if (lane == 0) mbar_arrive(q_full);
      const int nh = both ? n : (n + 1 - half) / 2;     // steps of the half
      const uint32_t first = half == 0 ? step_a : step_b;
      // every row of the half sees [lo_all, hi_all]
      const int hi_all = rq.len - rq.rows + (row0 + row_h) / a.group;
      const int hi_any = rq.len - rq.rows + (row0 + min(row_h + kHalfRows, n_rows) - 1) / a.group;
      const int lo_all = a.window > 0 ? max(hi_any - a.window + 1, 0) : 0;
      const int pos = rq.len - rq.rows + row / a.group, low = a.window > 0 ? pos - a.window : -1;
      float m = -INFINITY, l = 0.0f;                    // the same m in both threads of a row
      bool ok = true;
      for (int k = 0; k < nh; ++k) {                    // (an abort ends the waits, not the meetings)
        ok = ok && wait(&s_full[half], first + k, abort_flag);
        tc_fence_after();
        const int i = both ? k : 2 * k + half;
        const int t0 = (step0 + i) * kKeys + 64 * part;
        const uint32_t have = (kv_have[(step + i) & 3u] >> (4 * part)) & 15u;
        const bool some = t0 + 63 > hi_all || t0 < lo_all || have != 15u;
        auto hide = [&](uint32_t (&s)[32], int c) {
          if (some) {
#pragma unroll
            for (int j = 0; j < 32; ++j) {
              const int t = t0 + 32 * c + j;
              if (t > pos || t <= low || !((have >> (2 * c + j / kKvGroup)) & 1u)) s[j] = 0xFF800000u;   // -inf
            }
          }
        };
        // the scores are read twice, 32 columns at a time: for the maximum, and for the weights
        uint32_t s[32];
        float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          tmem_ld32(col_s + 32 * c, s);
          tmem_wait_ld(s);
          hide(s, c);
#pragma unroll
          for (int j = 0; j < 32; ++j) top[j & 3] = fmaxf(top[j & 3], __uint_as_float(s[j]));
        }
        const float mine_top = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
        float* at = s_max + (k & 1) * kStepMax;
        at[part * kHalfRows] = mine_top;
        meet();
        const float mt = fmaxf(mine_top, at[(part ^ 1) * kHalfRows]) * f;
        float back = 1.0f;
        if (mt > m + kSlack) {                          // (also the first finite one)
          back = ex2(m - mt);
          m = mt;
          l *= back;
        }
        const float neg_m = m == -INFINITY ? 0.0f : -m;
        const float2 f2 = make_float2(f, f), neg_m2 = make_float2(neg_m, neg_m);
        float2 sum[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
        uint32_t keep[16];                              // weights of the second 32 keys, whose scores are still here:
#pragma unroll
        for (int cc = 0; cc < 2; ++cc) {                // they would stand over the first 32's, to be read again
          if (cc == 1) {
            tmem_ld32(col_s, s);
            tmem_wait_ld(s);
            hide(s, 0);
          }
          uint32_t p[16];
#pragma unroll
          for (int j = 0; j < 32; j += 2) {
            const float2 x = __ffma2_rn(make_float2(__uint_as_float(s[j]), __uint_as_float(s[j + 1])), f2, neg_m2);
            const float2 w = make_float2(ex2(x.x), ex2(x.y));
            sum[(j >> 1) & 1] = __fadd2_rn(sum[(j >> 1) & 1], w);
            p[j / 2] = pack_f16(w.x, w.y);
          }
          if (cc == 0) {
#pragma unroll
            for (int j = 0; j < 16; ++j) keep[j] = p[j];
          } else {
            tmem_st16(col_s, p);
            tmem_st16(col_s + 16, keep);
          }
        }
        l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
        if (k > 0 && __any_sync(0xffffffffu, back != 1.0f)) {
          ok = ok && wait(&pv_done[half], first + k - 1, abort_flag);   // O is at rest until these weights are multiplied
          tc_fence_after();
#pragma unroll 1
          for (int i = part * (D / 2); i < (part + 1) * (D / 2); i += 32) {
            tmem_ld32(col_o + i, s);
            tmem_wait_ld(s);
#pragma unroll
            for (int j = 0; j < 32; ++j) s[j] = __float_as_uint(__uint_as_float(s[j]) * back);
            tmem_st32(col_o + i, s);
          }
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[half]);
      }
      // ---- output: each thread of a row its share of the elements, 32 at a time
      if (!idle) {
        float* at = s_max + (nh & 1) * kStepMax;        // not the last step's
        at[part * kHalfRows] = l;
        meet();
        l += at[(part ^ 1) * kHalfRows];
        if (nh > 0 && ok) ok = wait(&pv_done[half], first + nh - 1, abort_flag);
        float back = 1.0f, back_o = 0.0f;               // factors of this half's O and, of the same rows, the other's
        const int nh_o = both ? 0 : (n + half) / 2;
        if (!both) {
          // (the buffer of this half's last step, whose maxima have been read)
          at = s_max + ((nh + 1) & 1) * kStepMax;
          if (part == 0) {
            at[0] = m;
            at[kHalfRows] = l;
          }
          meet_all();
          at = s_max + (1 - 2 * half) * 2 * kHalfRows + ((nh_o + 1) & 1) * kStepMax;
          const float m_o = at[0], l_o = at[kHalfRows], top = fmaxf(m, m_o);
          back = m == -INFINITY ? 0.0f : ex2(m - top);
          back_o = m_o == -INFINITY ? 0.0f : ex2(m_o - top);
          const float mine_l = l * back, others = l_o * back_o;
          l = __fadd_rn(mine_l, others);
          m = top;
          if (nh_o > 0 && ok) wait(&pv_done[half ^ 1], (half == 0 ? step_b : step_a) + nh_o - 1, abort_flag);
        }
        tc_fence_after();
        const float inv = l == 0.0f ? 0.0f : vg / l;
        uint16_t* out = a.out + ((size_t)tok * a.heads + head) * D;
        float* rec = a.records + (size_t)record * S::kRecord;
        const int rt = row_h + r;                       // row in the tile
        // columns of a thread: half a row's, or a quarter (D = 64: half of them of every second thread)
        const int i0 = both ? part * (D / 2) : D == 128 ? (2 * half + part) * 32 : half * 32;
        const int i1 = both ? i0 + D / 2 : D == 128 || part == 0 ? i0 + 32 : i0;
#pragma unroll 1
        for (int i = i0; i < i1; i += 32) {
          uint32_t o[32];
          if (nh > 0) {
            tmem_ld32(col_o + i, o);
            tmem_wait_ld(o);
          } else {
#pragma unroll
            for (int j = 0; j < 32; ++j) o[j] = 0u;
          }
          if (!both) {
            uint32_t x[32];
            if (nh_o > 0) {
              tmem_ld32(col_o + (half == 0 ? kColHalf : -kColHalf) + i, x);
              tmem_wait_ld(x);
            } else {
#pragma unroll
              for (int j = 0; j < 32; ++j) x[j] = 0u;
            }
#pragma unroll
            for (int j = 0; j < 32; ++j)
              o[j] = __float_as_uint(__fadd_rn(__uint_as_float(o[j]) * back, __uint_as_float(x[j]) * back_o));
          }
          if (mine && !whole) {
#pragma unroll
            for (int j = 0; j < 32; j += 4)
              __stcg(reinterpret_cast<float4*>(rec + (size_t)rt * D + i + j),
                     make_float4(__uint_as_float(o[j]), __uint_as_float(o[j + 1]), __uint_as_float(o[j + 2]),
                                 __uint_as_float(o[j + 3])));
          } else if (mine) {
#pragma unroll
            for (int j = 0; j < 32; j += 8) {
              uint32_t w[4];
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const __nv_bfloat162 x = __floats2bfloat162_rn(__uint_as_float(o[j + 2 * e]) * inv,
                                                               __uint_as_float(o[j + 2 * e + 1]) * inv);
                w[e] = *reinterpret_cast<const uint32_t*>(&x);
              }
              *reinterpret_cast<uint4*>(out + i + j) = make_uint4(w[0], w[1], w[2], w[3]);
            }
          }
        }
        const bool says = mine && part == 0 && (both || half == 0);
        if (says && whole && a.lse)
          a.lse[(size_t)tok * a.heads + head] = l == 0.0f ? -INFINITY : (m + log2f(l)) / kLog2e;
        if (says && !whole) {
          __stcg(rec + kRows * D + rt, m);
          __stcg(rec + kRows * (D + 1) + rt, l);
        }
      }
      tc_fence_before();
    } else if (warp < kCopyWarp) {
      // ================ dequantize ================
      constexpr int kMine = kGroups / kDequantWarps;
      const int g0 = (warp - kSoftWarps) * kMine;
      bool ok = true;
      for (int k = 0; k < n && ok; ++k) {
        const uint32_t i = step + k, slot = i % kRing, buf = i & 1u;
        ok = wait(&raw_full[slot], i / kRing, abort_flag);
        const uint32_t have = raw_have[slot];
        const uint8_t* raw = smem + S::kOffRaw + slot * S::kRaw;
        if (i >= 1) ok = wait(k_free, i - 1, abort_flag) && ok;          // the last step's keys have been multiplied
#pragma unroll
        for (int g = g0; g < g0 + kMine; ++g) dequantize_keys<D>(raw + g * L::kGroupBytes, smem + S::kOffK, g, lane);
        if (g0 == 0 && lane == 0) kv_have[i & 3u] = have;
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (lane == 0) mbar_arrive(k_full);
        if (i >= 2) ok = wait(&v_free[buf], i / 2 - 1, abort_flag) && ok;
#pragma unroll
        for (int g = g0; g < g0 + kMine; ++g) {
          const int t0 = (step0 + k) * kKeys + g * kKvGroup;
          const int live = ((have >> g) & 1u) ? min(max(rq.len - t0, 0), kKvGroup) : 0;
          dequantize_values<D>(raw + g * L::kGroupBytes, smem + S::kOffV + buf * S::kTile, g, live, lane);
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&raw_free[slot]);
          mbar_arrive(&v_full[buf]);
        }
      }
    } else if (warp == kCopyWarp) {
      // ================ copies ================
      const int32_t* trow = a.table + (size_t)b * a.width;
      const uint8_t* src_head = a.pages + (size_t)kvh * (a.page_size / kKvGroup) * L::kGroupBytes;
      const size_t page_bytes = (size_t)a.kv_heads * (a.page_size / kKvGroup) * L::kGroupBytes;
      // lane g < kGroups: the page of group g of step k (-1: not there, or not to be read)
      auto look_up = [&](int k) {
        const int t0 = (step0 + k) * kKeys + lane * kKvGroup;
        if (k >= n || lane >= kGroups || t0 > hi || t0 + kKvGroup <= lo) return -1;
        const int page = trow[t0 / a.page_size];
        if (page >= 0 && page < a.num_pages) return page;
        atomicOr(&g_nvfp4_device_error, NVFP4_DEVERR_KV_RANGE);
        return -1;
      };
      bool ok = true;
      int next = look_up(0);
      bool taken = false;
      for (int k = 0; k < n && ok; ++k) {
        const uint32_t i = step + k, slot = i % kRing;
        const int page = next;
        next = look_up(k + 1);
        if (i >= kRing) ok = wait(&raw_free[slot], i / kRing - 1, abort_flag);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        const uint32_t have = __ballot_sync(0xffffffffu, page >= 0);
        if (lane == 0) {
          raw_have[slot] = have;
          mbar_arrive_expect_tx(&raw_full[slot], __popc(have) * L::kGroupBytes);
        }
        __syncwarp();
        const int t0 = (step0 + k) * kKeys + lane * kKvGroup;
        if (page >= 0)
          bulk_g2s(smem + S::kOffRaw + slot * S::kRaw + lane * L::kGroupBytes,
                   src_head + page * page_bytes + (t0 % a.page_size / kKvGroup) * L::kGroupBytes, L::kGroupBytes,
                   &raw_full[slot]);
        copied = i + 1;
        if (k == kRing - 1) {                           // the ring is full: time for the next tile
          take_tile(tiles + 1);
          taken = true;
        }
      }
      if (!taken) take_tile(tiles + 1);
    } else {
      // ================ products ================
      const uint32_t lead = elect_one();
      bool ok = wait(q_full, tiles, abort_flag);
      // descriptors of the operands' starts; everything else is an addition to their address field
      const uint64_t q_desc = smem_desc_sw128(smem_u32(smem + S::kOffQ)), k_desc = smem_desc_sw128(smem_u32(smem + S::kOffK));
      const uint64_t v_desc = smem_desc_mn_sw128(smem_u32(smem + S::kOffV), S::kPanel);
      // item j: half j % 2's next step, which is step j / 2 where the halves have their own rows, and step j where they
      // share the rows
      const int items = both ? 2 * n : n;
      auto step_of = [&](int j) { return both ? j >> 1 : j; };
      auto multiply_scores = [&](int item) {
        const int h = item & 1;
        if (!both || h == 0) ok = wait(k_full, step + step_of(item), abort_flag) && ok;
        if (!ok) return;
        tc_fence_after();
        const uint64_t dq = q_desc + (uint64_t)(both ? h * (S::kTile >> 4) : 0);
#pragma unroll
        for (int j = 0; j < D / 16; ++j) {
          constexpr int kPanel16 = S::kPanel >> 4;
          const uint64_t at = (uint64_t)((j >> 2) * kPanel16 + (j & 3) * 2);
          mma_f16_ss(lead, tmem + kColHalf * h, dq + at, k_desc + at, S::kIdescS, j > 0 ? 1u : 0u);
        }
        commit(lead, &s_full[h]);
        if (!both || h == 1) commit(lead, k_free);
      };
      for (int item = 0; item < min(items, 2); ++item) multiply_scores(item);
      for (int item = 0; item < items && ok; ++item) {
        const int h = item & 1;
        const uint32_t i = step + step_of(item), buf = i & 1u, u = (h == 0 ? step_a : step_b) + (item >> 1);
        const uint64_t dv = v_desc + (uint64_t)(buf * (S::kTile >> 4));
        if (!both || h == 0) ok = wait(&v_full[buf], i / 2, abort_flag);
        ok = ok && wait(&p_full[h], u, abort_flag);
        if (!ok) break;
        tc_fence_after();
        const uint32_t col = tmem + kColHalf * h;
#pragma unroll
        for (int j = 0; j < kKeys / 16; ++j)
          mma_f16_ts(lead, col + kColO, col + (j >> 2) * 64 + 8 * (j & 3), dv + (uint64_t)(j * (2048 >> 4)), S::kIdescO,
                     (item > 1 || j > 0) ? 1u : 0u);
        commit(lead, &pv_done[h]);
        if (!both || h == 1) commit(lead, &v_free[buf]);
        if (item + 2 < items) {
          ok = wait(&pv_done[h], u, abort_flag);        // the next scores stand where these weights are
          multiply_scores(item + 2);
        }
      }
    }
    step += (uint32_t)n;
    step_a += (uint32_t)(both ? n : (n + 1) / 2);
    step_b += (uint32_t)(both ? n : n / 2);
    ++tiles;
    __syncthreads();                                    // the tile's numbers and the TMEM are free again
    const bool aborted = *abort_flag != 0u;
    __syncthreads();
    if (aborted) break;
  }
  if (*abort_flag && warp == kCopyWarp) {
    // copies may still be in flight after a wait has given up: let every started one land (bounded)
    for (uint32_t i = copied > kRing ? copied - kRing : 0u; i < copied; ++i)
      for (uint32_t j = 0; j < (1u << 16); ++j)
        if (mbar_try_wait(&raw_full[i % kRing], (i / kRing) & 1u)) break;
  }
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols));
  }
  // the last CTA to leave resets the tile counter
  if (tid == 0) {
    __threadfence();
    if (atomicAdd(&a.counters[kTileCounter + 1], 1u) == gridDim.x - 1u) {
      a.counters[kTileCounter] = 0u;
      a.counters[kTileCounter + 1] = 0u;
    }
  }
}

// Merges the records of tiles that were cut, kMergeRows rows of a tile at a time.
constexpr int kMergeRows = 32, kMergeThreads = 256;

template <int D>
__global__ void __launch_bounds__(kMergeThreads) kv_attention_merge_kernel(const AttnArgs a) {
  using S = Shape<D>;
  __shared__ int s_info[4];
  griddep_launch_dependents();
  griddep_wait();
  const int tid = threadIdx.x, lane = tid & 31;
  const int size = (int)__ldcg(&a.counters[kTileCounter + 2]);
  if (size == 0) return;
  constexpr int kParts = kRows / kMergeRows;
  const float vg = *a.v_global;
  for (int item = blockIdx.x; ; item += gridDim.x) {
    const int r0 = item % kParts * kMergeRows;
    __syncthreads();
    if (tid < 32) {
      const Tile tile = find<true>(a, item / kParts, size, lane);
      if (lane == 0) s_info[0] = tile.b, s_info[1] = tile.kvh, s_info[2] = tile.row0, s_info[3] = tile.number;
    }
    __syncthreads();
    const int b = s_info[0], kvh = s_info[1], row0 = s_info[2], number = s_info[3];
    if (b < 0) break;
    const Request rq = get_request(a, b, false);
    const int n_rows = (int)min((long long)kRows, (long long)rq.rows * a.group - row0);
    const Steps steps(a, rq, row0, n_rows, size);
    if (steps.all <= steps.piece) continue;
    const int n_rec = (steps.all + steps.piece - 1) / steps.piece;
    for (int e = tid; e < kMergeRows * (D / 4); e += kMergeThreads) {
      const int rt = r0 + e / (D / 4), d = e % (D / 4) * 4;
      if (rt >= n_rows) break;
      const float* rec = a.records + (size_t)number * S::kRecord;
      float mx = -INFINITY, l = 0.0f;
      float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
      for (int q = 0; q < n_rec; ++q, rec += S::kRecord) {
        const float m = __ldcg(rec + kRows * D + rt), lq = __ldcg(rec + kRows * (D + 1) + rt);
        const float4 y = __ldcg(reinterpret_cast<const float4*>(rec + (size_t)rt * D + d));
        if (no_keys(m, lq)) continue;
        const float mn = fmaxf(mx, m), back = ex2(mx - mn), w = ex2(m - mn);
        mx = mn;
        l = fmaf(lq, w, l * back);
        x.x = fmaf(y.x, w, x.x * back), x.y = fmaf(y.y, w, x.y * back);
        x.z = fmaf(y.z, w, x.z * back), x.w = fmaf(y.w, w, x.w * back);
      }
      const int row = row0 + rt, tok = rq.first + row / a.group, head = kvh * a.group + row % a.group;
      const float inv = l == 0.0f ? 0.0f : vg / l;
      const __nv_bfloat162 x0 = __floats2bfloat162_rn(x.x * inv, x.y * inv), x1 = __floats2bfloat162_rn(x.z * inv, x.w * inv);
      *reinterpret_cast<uint2*>(a.out + ((size_t)tok * a.heads + head) * D + d) =
          make_uint2(*reinterpret_cast<const uint32_t*>(&x0), *reinterpret_cast<const uint32_t*>(&x1));
      if (a.lse && d == 0) a.lse[(size_t)tok * a.heads + head] = l == 0.0f ? -INFINITY : (mx + log2f(l)) / kLog2e;
    }
  }
}

template <int D, class T>
cudaError_t launch(const AttnArgs& a, cudaStream_t stream) {
  using S = Shape<D>;
  static PerDeviceInt grid_cache;
  cudaError_t err = cudaSuccess;
  const int grid = grid_cache.get([](int dev, cudaError_t* e_out) -> int {
    int sms = 0;
    cudaError_t e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e == cudaSuccess)
      e = cudaFuncSetAttribute(kv_attention_tc_kernel<D, T>, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmem);
    if (e != cudaSuccess) {
      *e_out = e;
      return 0;
    }
    return sms > 0 ? sms : 1;
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
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kv_attention_tc_kernel<D, T>, a);
  if (e != cudaSuccess || a.pieces == 0) return e;
  // whether anything was cut only the GPU knows: the launch ends at once if not
  cfg.gridDim = dim3((unsigned)(4 * grid));
  cfg.blockDim = dim3(kMergeThreads);
  cfg.dynamicSmemBytes = 0;
  return cudaLaunchKernelEx(&cfg, kv_attention_merge_kernel<D>, a);
}

}  // namespace

cudaError_t nvfp4_internal_kv_attention_tc(const AttnArgs& a, int head_dim, int dtype, cudaStream_t stream) {
  if (head_dim == 128)
    return dtype == NVFP4_DTYPE_F32 ? launch<128, float>(a, stream) : launch<128, uint16_t>(a, stream);
  return dtype == NVFP4_DTYPE_F32 ? launch<64, float>(a, stream) : launch<64, uint16_t>(a, stream);
}
