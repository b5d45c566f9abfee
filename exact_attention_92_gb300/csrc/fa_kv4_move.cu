// Writing tokens into the 4-bit key/value cache and reading them back
// (fa_kv4_write, fa_kv4_read).
//
// A CTA takes the tokens of one call that share a 16-token block of the cache
// (of one head), so that sequence, page and block are worked out once for it; a
// thread takes 8 channels of a token's key and value.  Both kernels move each
// byte once, straight between global memory and registers, and are bound by
// that traffic (a token-head of d channels is 4 d bytes of bf16 and 9 d / 8 of
// cache) as long as a value costs few enough instructions.
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "fa_common.h"
#include "sm103_primitives.cuh"
#include "kv4_format.cuh"

namespace fa {

using namespace dev;

struct Kv4MoveParams {
  Kv4Cache c;
  const int* start;   // [B]
  const int* count;   // [B] or null
  const uint4* k_in;  // [B, Hkv, N, d] (write)
  const uint4* v_in;
  uint4* k_out;       // (read)
  uint4* v_out;
  int N;
  int blocks;         // 16-token blocks that N tokens can touch: (N + 30) / 16
};

// The token of this thread: its row of [B, Hkv, N], its place in the block, and
// the block, or null where there is none.
template <int D>
__device__ __forceinline__ uint8_t* kv4_token(const Kv4MoveParams& p, size_t* row, int* place) {
  constexpr int kPer = D / 8;  // threads a token
  pdl_wait();
  pdl_trigger();
  const int bh = (int)(blockIdx.x / (unsigned)p.blocks), nth = (int)(blockIdx.x - (unsigned)bh * p.blocks);
  const int b = bh / p.c.Hkv;
  const int start = p.start[b];
  int n = p.N;
  if (p.count != nullptr) {
    n = p.count[b];
    if (n < 0 || n > p.N) {
      if (threadIdx.x == 0) kv4_bad_index(p.c);
      n = n < 0 ? 0 : p.N;
    }
  }
  *place = threadIdx.x / kPer;
  // Positions may be far out of range: 64 bits, rounded down for negative ones.
  const long long pos = (((long long)start >> 4) + nth) * 16 + *place;
  const long long i = pos - start;
  if (i < 0 || i >= n) return nullptr;
  *row = (size_t)bh * p.N + (size_t)i;
  if (pos < 0 || pos >= ((long long)p.c.max_pages << p.c.page_shift)) {
    kv4_bad_index(p.c);
    return nullptr;
  }
  const int page = kv4_page(p.c, b, (int)pos);
  if (page < 0) return nullptr;
  return kv4_block<D>(p.c, page, bh - b * p.c.Hkv, (int)pos);
}

// Both halves of a word of 16-bit magnitudes at once.
__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) { return __vmaxu2(a, b); }

// Largest magnitude of 8 bf16, as bits, in the low half.
__device__ __forceinline__ uint32_t top_bits(uint4 w) {
  const uint32_t k = 0x7fff7fffu;
  const uint32_t m = max_u16x2(max_u16x2(w.x & k, w.y & k), max_u16x2(w.z & k, w.w & k));
  return max_u16x2(m, m >> 16) & 0xffffu;
}

// Scale bits and the factor 1 / scale of a group whose largest magnitude has
// the bits `top`; the factor is 0 where all codes are 0.
//
// The scale is top / 6 rounded to bf16.  top has 8 significant bits, so top / 6
// is never the middle of two bf16 (that has 9 bits, and 6 times it 10 or more)
// and lies 2^-12 of itself away from any: top * (1/6 in fp32) rounds alike.
__device__ __forceinline__ float kv4_scale(uint32_t top, uint32_t* bits) {
  const float s = __bfloat162float(__float2bfloat16_rn(__uint_as_float(top << 16) * 0.16666667163372040f));
  const bool finite = top < 0x7f80u;
  const bool held = finite && s >= 1.17549435e-38f;
  *bits = held ? __float_as_uint(s) >> 16 : (finite ? 0u : 0x7fffu);
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(s));
  return held ? r : 0.f;
}

// Codes of 8 channels whose group has the factor r = 1 / s.
//
// The codes are those of the exact quotients x / s.  x has 8 significant bits
// and s has 8, so a quotient that is not one of the rounding borders
// (multiples of 1/4 up to 5) differs from each by more than 2^-13 of it (x
// and border * s are then different multiples of one unit, of which border * s
// holds at most 20 * 255).  r is within 2^-23 of 1 / s (the bound that PTX
// gives), so x r is within 7 * 2^-23 of the quotient, at most 7 or so, and the
// addition of 96 rounds it, once, to a multiple of 2^-17.  So a quotient on a
// border lands on it exactly, and any other stays on its side: one reciprocal a
// group in place of 32 divisions.
__device__ __forceinline__ uint32_t kv4_codes8(uint4 raw, float r) {
  const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
  float2 x[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[i] = __ffma2_rn(make_float2(bf16_lo(w[i]), bf16_hi(w[i])), make_float2(r, r), make_float2(96.f, 96.f));
    x[i] = __fadd2_rn(x[i], make_float2(-96.f, -96.f));
  }
  return kv4_encode8(x);
}

// Two 16-bit units of the values that lanes 4 apart (groups g and g ^ 1) hold
// for the same channels u, u + 1: the even group's lane gets unit u of both as
// one word, the odd one's unit u + 1.  Its own inverse.
__device__ __forceinline__ uint32_t exchange_units(uint32_t w, bool odd) {
  const uint32_t other = __shfl_xor_sync(0xffffffffu, w, 4);
  return odd ? __byte_perm(other, w, 0x7632) : __byte_perm(w, other, 0x5410);
}

template <int D>
__global__ void __launch_bounds__(2 * D) kv4_write_kernel(const Kv4MoveParams p) {
  using F = Kv4<D>;
  constexpr int kPer = D / 8;
  const int c8 = threadIdx.x % kPer, g = c8 / 4, t = c8 % 4;
  int place = 0;
  size_t row = 0;
  uint8_t* const block = kv4_token<D>(p, &row, &place);
  uint4 kr = make_uint4(0, 0, 0, 0), vr = kr;
  if (block != nullptr) {
    kr = p.k_in[row * kPer + c8];
    vr = p.v_in[row * kPer + c8];
  }
  // A group's 32 channels are a quad of lanes: key and value in one word.
  uint32_t top = top_bits(kr) | (top_bits(vr) << 16);
  top = max_u16x2(top, __shfl_xor_sync(0xffffffffu, top, 1));
  top = max_u16x2(top, __shfl_xor_sync(0xffffffffu, top, 2));
  uint32_t ks, vs;
  const float rk = kv4_scale(top & 0xffffu, &ks), rv = kv4_scale(top >> 16, &vs);
  uint32_t kw = kv4_codes8(kr, rk), vw = kv4_codes8(vr, rv);
  // A group without a scale: zeros, whatever 0 * inf and the like gave.
  kw = rk == 0.f ? 0u : kw;
  vw = rv == 0.f ? 0u : vw;
  if constexpr (F::kGroups % 2 == 0) {
    vw = exchange_units(vw, g & 1);
    if (block != nullptr) *reinterpret_cast<uint32_t*>(block + F::value_unit(place, g & ~1, 2 * t + (g & 1))) = vw;
  } else if (block != nullptr) {
    *reinterpret_cast<uint16_t*>(block + F::value_unit(place, g, 2 * t)) = (uint16_t)vw;
    *reinterpret_cast<uint16_t*>(block + F::value_unit(place, g, 2 * t + 1)) = (uint16_t)(vw >> 16);
  }
  if (block == nullptr) return;
  *reinterpret_cast<uint32_t*>(block + F::key_word(place, g, t)) = kw;
  if (t < 2) *reinterpret_cast<uint16_t*>(block + F::scale(place, t, g)) = (uint16_t)(t == 0 ? ks : vs);
}

// 8 held values as bf16: code * scale has at most 10 significant bits, exact
// in fp32, so this rounds once.
__device__ __forceinline__ uint4 kv4_values8(uint32_t w, float s) {
  uint32_t h[4], o[4];
  kv4_decode8(w, h);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = __fmul2_rn(__half22float2(*reinterpret_cast<const __half2*>(&h[i])), make_float2(s, s));
    o[i] = pack_bf16(f.x, f.y);
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
}

template <int D>
__global__ void __launch_bounds__(2 * D) kv4_read_kernel(const Kv4MoveParams p) {
  using F = Kv4<D>;
  constexpr int kPer = D / 8;
  const int c8 = threadIdx.x % kPer, g = c8 / 4, t = c8 % 4;
  int place = 0;
  size_t row = 0;
  const uint8_t* const block = kv4_token<D>(p, &row, &place);
  uint32_t kw = 0, vw = 0, ks = 0, vs = 0;
  if (block != nullptr) {
    kw = *reinterpret_cast<const uint32_t*>(block + F::key_word(place, g, t));
    ks = *reinterpret_cast<const uint16_t*>(block + F::scale(place, 0, g));
    vs = *reinterpret_cast<const uint16_t*>(block + F::scale(place, 1, g));
    if constexpr (F::kGroups % 2 == 0)
      vw = *reinterpret_cast<const uint32_t*>(block + F::value_unit(place, g & ~1, 2 * t + (g & 1)));
    else
      vw = *reinterpret_cast<const uint16_t*>(block + F::value_unit(place, g, 2 * t)) |
           ((uint32_t)*reinterpret_cast<const uint16_t*>(block + F::value_unit(place, g, 2 * t + 1)) << 16);
  }
  if constexpr (F::kGroups % 2 == 0) vw = exchange_units(vw, g & 1);
  if (block == nullptr) return;
  p.k_out[row * kPer + c8] = kv4_values8(kw, bf16_lo(ks));
  p.v_out[row * kPer + c8] = kv4_values8(vw, bf16_lo(vs));
}

template <int D>
static cudaError_t launch_move_t(bool write, const Kv4MoveParams& p, unsigned grid, cudaStream_t stream) {
  return launch_pdl(write ? kv4_write_kernel<D> : kv4_read_kernel<D>, dim3(grid), dim3(2 * D), 0, stream, p);
}

cudaError_t launch_kv4_move(int d, bool write, const Kv4Cache& c, const int* start, const int* count, const void* k_in,
                            const void* v_in, void* k_out, void* v_out, int N, cudaStream_t stream) {
  Kv4MoveParams p;
  p.c = c;
  p.start = start;
  p.count = count;
  p.k_in = static_cast<const uint4*>(k_in);
  p.v_in = static_cast<const uint4*>(v_in);
  p.k_out = static_cast<uint4*>(k_out);
  p.v_out = static_cast<uint4*>(v_out);
  p.N = N;
  p.blocks = (int)(((long long)N + 30) / 16);
  const unsigned grid = (unsigned)c.B * c.Hkv * p.blocks;
  switch (d) {
    case 64: return launch_move_t<64>(write, p, grid, stream);
    case 96: return launch_move_t<96>(write, p, grid, stream);
    case 128: return launch_move_t<128>(write, p, grid, stream);
    case 256: return launch_move_t<256>(write, p, grid, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace fa
