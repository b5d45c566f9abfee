// The 4-bit key/value cache: where a page's bytes lie (include/fa.h gives the
// format in words) and how its codes are made and read.
#pragma once

#include <cstdint>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "fa.h"

namespace fa {

constexpr int kKv4Block = 16;  // tokens stored together (a page holds whole blocks)
constexpr int kKv4Group = 32;  // channels that share a scale

template <int D>
struct Kv4 {
  static constexpr int kGroups = D / kKv4Group;                  // NG
  static constexpr int kRowBytes = D / 2;                        // codes of one token's key (or value)
  static constexpr int kValues = kKv4Block * kRowBytes;          // offset of the values in a block
  static constexpr int kScales = 2 * kValues;                    // offset of the scales
  static constexpr int kScaleBytes = 4 * kGroups;                // scales of one token, key and value
  static constexpr int kBlockBytes = kScales + kKv4Block * kScaleBytes;
  static constexpr int kQuad = kGroups < 4 ? kGroups : 4;        // words a lane reads at once

  // Byte offset of the word with channels 32 g + 8 t + 0..7 of token p's key.
  __host__ __device__ static constexpr int key_word(int p, int g, int t) {
    const int b = ((g / 4) * 16 + t * kQuad + g % 4) * 4;
    return p * kRowBytes + (D == 256 ? (b ^ (64 * (p & 1))) : b);
  }
  // Row of the values section that holds token p.
  __host__ __device__ static constexpr int value_row(int p) { return 4 * ((p & 1) + 2 * (p >> 3)) + ((p >> 1) & 3); }
  // What the byte offsets within value row r are xor'd with.
  __host__ __device__ static constexpr int value_xor(int r) {
    return D == 128 ? 32 * ((r >> 1) & 1) : (D == 256 ? 32 * (r & 3) : 0);
  }
  // Byte offset of the unit with channels 32 g + 4 u + 0..3 of token p's value.
  __host__ __device__ static constexpr int value_unit(int p, int g, int u) {
    const int r = value_row(p);
    return kValues + r * kRowBytes + (((u * kGroups + g) * 2) ^ value_xor(r));
  }
  // Byte offset of the scale of group g of token p's key (which = 0) or value (1).
  __host__ __device__ static constexpr int scale(int p, int which, int g) {
    return kScales + p * kScaleBytes + (which * kGroups + g) * 2;
  }
};

static_assert(Kv4<64>::kBlockBytes == 18 * 64 && Kv4<96>::kBlockBytes == 18 * 96 && Kv4<128>::kBlockBytes == 18 * 128 &&
                  Kv4<256>::kBlockBytes == 18 * 256,
              "a block holds 16 tokens of keys and values at 4.5 bits a value");

// Sizes and index arrays that the kernels over the cache share.
struct Kv4Cache {
  uint8_t* pages;        // [num_pages, Hkv, page bytes]
  const int* table;      // [B, max_pages]
  int num_pages;
  int max_pages;
  int Hkv;
  int page_shift;        // log2(page_size)
  int B;
  unsigned int* status;  // words of fa_poll_status
};

namespace dev {

// Records that an index out of range was skipped.
__device__ __forceinline__ void kv4_bad_index(const Kv4Cache& c) { atomicExch(c.status + 1, (unsigned)FA_ERR_BAD_INDEX); }

// The eight e2m1 codes of a word as four pairs of fp16 (exact).
__device__ __forceinline__ void kv4_decode8(uint32_t w, uint32_t* h) {
  asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, a;\n\tcvt.rn.f16x2.e2m1x2 %1, b;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, c;\n\tcvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(w));
}

// Eight fp32 to e2m1 codes (nearest, ties to even, saturating), x[0] lowest.
__device__ __forceinline__ uint32_t kv4_encode8(const float2* x) {
  uint32_t w;
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\tcvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\tcvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
      "mov.b32 %0, {a, b, c, d};\n\t}"
      : "=r"(w)
      : "f"(x[0].x), "f"(x[0].y), "f"(x[1].x), "f"(x[1].y), "f"(x[2].x), "f"(x[2].y), "f"(x[3].x), "f"(x[3].y));
  return w;
}

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

}  // namespace dev
}  // namespace fa
