// Memory layout of the NVFP4 KV cache (see nvfp4_kv_cache in nvfp4.h): pages of
// 16-token groups, a group of one kv head being K codes, K scales, V codes and
// V scales, 18 D bytes.
//
// Why this order.  The attention kernel multiplies 16 tokens at a time with
// mma.m16n8k16, lane = 4 r + c (r 0..7, c 0..3), and each lane should find its
// operands in whole 16-byte pieces without bank conflicts:
//   K (scores, A operand, rows = tokens): lane (r, c) holds rows r and r + 8,
//     the D/4 elements from c D/4 on -- the order of the contraction index is
//     free, as long as the queries use the same one;
//   V (output, A operand, rows = elements): lane (r, c) holds the D/8 elements
//     from r D/8 on for four tokens, 4c .. 4c + 3;
//   score row pos and token t go together as pos = 8 (t/2 % 2) + 2 (t/4) + t % 2,
//     so that the scores a lane gets back are those of its four V tokens.
#pragma once

#include "common.cuh"

constexpr int kKvGroup = 16;            // tokens of a group

template <int D>
struct KvLayout {
  static constexpr int kGroupBytes = 18 * D;
  static constexpr int kOffKScale = 8 * D;
  static constexpr int kOffV = 9 * D;
  static constexpr int kOffVScale = 17 * D;
  static constexpr int kBlocks = D / 16;

  static NVFP4_DEVINL int pos(int t) { return 8 * ((t >> 1) & 1) + 2 * (t >> 2) + (t & 1); }
  // The 8 bytes of K block b of token t, and its scale byte.
  static NVFP4_DEVINL int k_codes(int t, int b) { return pos(t) * (D / 2) + b * 8; }
  static NVFP4_DEVINL int k_scale(int t, int b) {
    const int p = pos(t);
    return kOffKScale + (((p & 7) * 4 + b / (D / 64)) * 2 + (p >> 3)) * (D / 64) + b % (D / 64);
  }
  // Bytes 4 h .. 4 h + 3 (h 0, 1) of V block b of token t; D = 128: h = 1 follows h = 0.
  static NVFP4_DEVINL int v_codes(int t, int b, int h) {
    if (D == 128) return kOffV + (b >> 1) * 256 + ((t >> 1) & 1) * 128 + (b & 1) * 64 + (t >> 2) * 16 + (t & 1) * 8 + 4 * h;
    return kOffV + (2 * b + h) * 64 + t * 4;
  }
  static NVFP4_DEVINL int v_scale(int t, int b) { return kOffVScale + b * 16 + t; }
};

// Byte offset of the group that holds token `in` of page `page` for kv head `head`.
template <int D>
NVFP4_DEVINL size_t kv_group_offset(int page, int in, int head, int page_size, int kv_heads) {
  return (((size_t)page * kv_heads + head) * (page_size / kKvGroup) + in / kKvGroup) * KvLayout<D>::kGroupBytes;
}

// Four code bytes (two E2M1 codes each) -> four FP16 pairs.
NVFP4_DEVINL void e2m1x8_to_f16(uint32_t w, uint32_t (&h)[4]) {
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "mov.b32 {a, b, c, d}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, a;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, c;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(w));
}

// Host: the checks of an nvfp4_kv_cache descriptor that every entry point makes.
nvfp4_status nvfp4_internal_check_kv_cache(const nvfp4_kv_cache* c);
