// What the kernels that write rows of K and V into the NVFP4 cache share: a block's loads and its quantization, and a
// warp's look at a window of 16 tokens.
#pragma once

#include "kv_layout.cuh"
#include "quant_block.cuh"

namespace {

// Raw words of a block: 16 FP32 or BF16 elements.
template <class T>
struct Raw {
  static constexpr int kPieces = sizeof(T) == 4 ? 4 : 2;
  uint4 w[kPieces];
  NVFP4_DEVINL void load(const T* p) {
#pragma unroll
    for (int i = 0; i < kPieces; ++i) w[i] = reinterpret_cast<const uint4*>(p)[i];   // L1 keeps the sectors' other halves
  }
  NVFP4_DEVINL void values(float (&v)[16]) const {
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      const uint32_t u[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if constexpr (sizeof(T) == 4) {
          v[4 * i + j] = __bfloat162float(__float2bfloat16_rn(__uint_as_float(u[j])));
        } else {
          v[8 * i + 2 * j] = bf16_lo(u[j]);
          v[8 * i + 2 * j + 1] = bf16_hi(u[j]);
        }
      }
    }
  }
};

// quant_block's recipe, the same bits where S is finite: s = E4M3(bm / (6 g)), S = dec(s) g, code = E2M1(RN(x / S)).
// The quotient is the correctly rounded one by Markstein's theorem (P. Markstein, "Computation of elementary functions
// on the IBM RISC System/6000 processor", 1990): with y = RN(1/S) and p = RN(x y), RN(p + y RN(x - p S)) = RN(x / S)
// while nothing underflows or overflows; NaN passes through bm and t into the branch, which costs no look of its own
// then (a cut of every quotient: 23.4 us for 16384 tokens of 8 heads instead of 21.1).  quant_block divides where x y
// is too close to a decision point to tell; with a global scale that is a power of two BF16 values meet those points
// exactly, in some lane of nearly every warp.
NVFP4_DEVINL uint32_t kv_quant_block(float (&v)[16], float g, uint2& codes) {
  float bm = 0.0f;
#pragma unroll
  for (int i = 0; i < 16; i += 2) asm("max.NaN.abs.f32 %0, %0, %1, %2;" : "+f"(bm) : "f"(v[i]), "f"(v[i + 1]));
  const float d = __fmul_rn(6.0f, g);
  const float t = d > 0.0f ? __fdiv_rn(bm, d) : 0.0f;
  uint32_t s = f32x2_to_e4m3x2(0.0f, t) & 0xFFu;
  float S = __fmul_rn(e4m3_to_f32(s), g);
  if (!(S > 0x1p-80f && S < 0x1p80f && t <= 464.0f)) {
    if (isnan(bm)) {                    // the scale is that of the other values
      s = f32x2_to_e4m3x2(0.0f, d > 0.0f ? __fdiv_rn(block_absmax(v), d) : 0.0f) & 0xFFu;
      S = __fmul_rn(e4m3_to_f32(s), g);
    }
    // far out: the quotient of x f and S f, f a power of two, is the same (what x f loses below 2^-149 is far
    // below the first decision point).  Where the scale saturates (t > 464; else |x| <= 16 S), quotients are cut to
    // 8, so that none overflows: like infinities and NaN, such values get the largest code and their own sign.
    // S = 0 gives zeros with the values' signs
    const float f = S > 0x1p-80f && S < 0x1p80f ? 1.0f : S < 1.0f ? 0x1p100f : 0x1p-100f;
    const float most = 8.0f * (S * f);
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = copysignf(fminf(fabsf(v[i]) * f, most), v[i]);
    S *= f;
  }
  const float y = S != 0.0f ? __frcp_rn(S) : 0.0f;
  uint32_t w[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    float q[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float x = v[8 * h + i], p = __fmul_rn(x, y);
      q[i] = copysignf(__fmaf_rn(__fmaf_rn(-p, S, x), y, p), x);   // a zero keeps its sign
    }
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
        "mov.b32 %0, {a, b, c, d};\n\t}"
        : "=r"(w[h])
        : "f"(q[0]), "f"(q[1]), "f"(q[2]), "f"(q[3]), "f"(q[4]), "f"(q[5]), "f"(q[6]), "f"(q[7]));
  }
  codes = make_uint2(w[0], w[1]);
  return s;
}

// ---- a window of 16 tokens --------------------------------------------------------
struct Window {
  int slot;                     // lane 16 + k: the slot of the window's token k
  uint32_t leads, alone, rest;  // bit k: token k is the first of a whole group, by itself, padding or bad
};

// The slot of token i, as given.
struct SlotsOf {
  const int32_t* slots;
  NVFP4_DEVINL int operator()(long long i) const { return slots[i]; }
};

// One warp looks at tokens i0 .. i0 + 15 and their neighbours; slot_of(i): token i's slot, -1: padding.
template <class F>
NVFP4_DEVINL Window look_at_window(const F& slot_of, int tokens, long long i0, long long num_slots, int lane, bool report) {
  const long long i = i0 - 16 + lane;
  const int s = i >= 0 && i < tokens ? slot_of(i) : -1;
  const int after = i + 32 < tokens ? slot_of(i + 32) : -1;
  // bit j: token i0 - 16 + j's slot is followed by the next one
  int next = __shfl_down_sync(0xffffffffu, s, 1);
  const int first_after = __shfl_sync(0xffffffffu, after, 0), next_after = __shfl_down_sync(0xffffffffu, after, 1);
  if (lane == 31) next = first_after;
  const uint64_t run = (uint64_t)__ballot_sync(0xffffffffu, (uint32_t)next == (uint32_t)s + 1u) |
                       (uint64_t)__ballot_sync(0xffffffffu, lane < 31 && (uint32_t)next_after == (uint32_t)after + 1u) << 32;
  const bool in_window = lane >= 16 && i < tokens, valid = in_window && s >= 0 && s < num_slots;
  const int t = s & (kKvGroup - 1);
  const bool whole = valid && ((run >> (lane - t)) & 0x7FFFu) == 0x7FFFu;
  if (in_window && !valid && s != -1 && report) atomicOr(&g_nvfp4_device_error, NVFP4_DEVERR_KV_RANGE);
  Window w;
  w.slot = s;
  w.leads = __ballot_sync(0xffffffffu, whole && t == 0) >> 16;
  w.alone = __ballot_sync(0xffffffffu, valid && !whole) >> 16;
  w.rest = __ballot_sync(0xffffffffu, in_window && !valid) >> 16;
  return w;
}

template <int D>
struct Map {
  using L = KvLayout<D>;
  static constexpr int kHalf = 9 * D;                     // bytes of a group's K or V half
  static constexpr int kPerPass = 32 / L::kBlocks;        // tokens a warp has a block each of
  static constexpr int kPasses = kKvGroup / kPerPass;
  // offsets in the half
  static NVFP4_DEVINL int codes(int which, int t, int b, int h) {
    return which == 0 ? L::k_codes(t, b) + 4 * h : L::v_codes(t, b, h) - kHalf;
  }
  static NVFP4_DEVINL int scale(int which, int t, int b) { return which == 0 ? L::k_scale(t, b) : L::v_scale(t, b) - kHalf; }
};

}  // namespace
