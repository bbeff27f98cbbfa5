// What the two attention kernels over the NVFP4 KV cache share: the arguments of
// a call, conversions, and a request's rows and keys.
#pragma once

#include <math.h>

#include "kv_layout.cuh"

constexpr int kMaxCtas = 640;           // most CTAs of a launch
constexpr size_t kCounterBytes = 4096;  // start of a workspace: counters, zero between calls (what a caller zeroes)
constexpr int kTileCounter = kMaxCtas;  // counters behind those of the segments: next piece, CTAs done; steps of a piece
static_assert((kTileCounter + 3) * 4 <= kCounterBytes, "the counters");
constexpr int kTcPieces = 304;          // records of the many-row kernel: two a SM
constexpr int kTcRecord = 256 * 130;    // floats of one
constexpr float kLog2e = 1.4426950408889634f;

struct AttnArgs {
  const void* q;
  int64_t q_ts, q_hs;
  const uint8_t* pages;
  const float *k_global, *v_global;
  const int32_t *table, *kv_lens, *cu_q;
  uint16_t* out;
  float* lse;
  unsigned int* counters;               // kCounterBytes, zero between calls
  float* records;                       // [2 kMaxCtas][rows][D + 2] (decode kernel)
  int tokens, heads, kv_heads, group, page_size, num_pages, width, batch, window;
  int pieces;                           // records that the many-row kernel has room for (0: none)
  float scale;
};

// The cache's rows may come from the preceding kernel's ordinary stores: order them before this thread's bulk copies.
NVFP4_DEVINL void fence_proxy_async_global() { asm volatile("fence.proxy.async.global;" ::: "memory"); }

// ---- instructions ------------------------------------------------------------
NVFP4_DEVINL float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Two E4M3 scale bytes -> an FP16 pair.
NVFP4_DEVINL uint32_t e4m3x2_to_f16(uint32_t s) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((unsigned short)s));
  return h;
}

NVFP4_DEVINL uint32_t hmul2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

NVFP4_DEVINL uint32_t pack_f16(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}

NVFP4_DEVINL uint4 lds128(const uint8_t* p) { return *reinterpret_cast<const uint4*>(p); }
NVFP4_DEVINL uint2 lds64(const uint8_t* p) { return *reinterpret_cast<const uint2*>(p); }

NVFP4_DEVINL float load_q(const float* p) { return __bfloat162float(__float2bfloat16_rn(*p)); }
NVFP4_DEVINL float load_q(const uint16_t* p) { return __uint_as_float((uint32_t)*p << 16); }

// Four query elements, as BF16 values.
NVFP4_DEVINL void load4(const float* p, float (&v)[4]) {
  const float4 f = *reinterpret_cast<const float4*>(p);
  v[0] = load_q(&f.x), v[1] = load_q(&f.y), v[2] = load_q(&f.z), v[3] = load_q(&f.w);
}
NVFP4_DEVINL void load4(const uint16_t* p, float (&v)[4]) {
  const uint2 u = *reinterpret_cast<const uint2*>(p);
  v[0] = bf16_lo(u.x), v[1] = bf16_hi(u.x), v[2] = bf16_lo(u.y), v[3] = bf16_hi(u.y);
}

// ---- requests --------------------------------------------------------------------
struct Request {
  int first, rows, len;                 // query rows [first, first + rows), keys [0, len)
  int begin;                            // first key that any row sees
  bool bad;                             // its row range is none
};

NVFP4_DEVINL Request get_request(const AttnArgs& a, int b, bool report) {
  Request r;
  r.first = b;
  r.rows = 1;
  r.bad = false;
  bool bad = false;
  if (a.cu_q) {
    r.first = a.cu_q[b];
    const int last = a.cu_q[b + 1];
    bad = r.first < 0 || last < r.first || last > a.tokens;
    r.rows = bad ? 0 : last - r.first;
    r.bad = bad;
  }
  r.len = max(a.kv_lens[b], 0);
  const long long most = (long long)a.width * a.page_size;
  if (r.len > most) {
    r.len = (int)most;
    bad = true;
  }
  if (bad && report) atomicOr(&g_nvfp4_device_error, NVFP4_DEVERR_KV_RANGE);
  r.begin = a.window > 0 ? (int)max((long long)r.len - r.rows - a.window + 1, 0ll) : 0;
  return r;
}

// A score's factor is never 0: a hidden score, -inf, times it has to stay -inf.
NVFP4_DEVINL float score_factor(float f) { return fmaxf(f, 1.2e-38f); }

// Whether a partial sum l with maximum m counts nothing.  A row of NaN scores has no maximum either; its NaN sum is
// carried on, so that the row's output is NaN however its keys are cut.
NVFP4_DEVINL bool no_keys(float m, float l) { return m == -INFINITY && l == 0.0f; }

// 2^-e and 2^e of the power of two at `big` (1 for 0), within FP32's normal range.
NVFP4_DEVINL void power_of_two(float big, float& down, float& up) {
  int e = (int)(__float_as_uint(big) >> 23) - 127;
  e = big > 0.0f ? min(max(e, -126), 126) : 0;
  down = __uint_as_float((uint32_t)(127 - e) << 23);
  up = __uint_as_float((uint32_t)(127 + e) << 23);
}

// Host: the kernel for many query rows a request (kv_attention_tc.cu).
cudaError_t nvfp4_internal_kv_attention_tc(const AttnArgs& a, int head_dim, int dtype, cudaStream_t stream);
