// Writing tokens into the 4-bit key/value cache and reading them back
// (fa_kv4_write, fa_kv4_read).
//
// A CTA takes 16 rows of [B * Hkv * N], a thread 8 channels of a row's key and
// value.  Both kernels move each byte once, straight between global memory
// and registers, and are bound by that traffic (a token-head of d channels is
// 4 d bytes of bf16 and 9 d / 8 of cache).
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
  int rows;           // B * Hkv * N
};

// Where the row of this thread is held: the block and the place in it, or
// null if the row takes no part.  One thread of a row records bad indices.
template <int D>
__device__ __forceinline__ uint8_t* kv4_row(const Kv4MoveParams& p, unsigned r, int* place) {
  if (r >= (unsigned)p.rows) return nullptr;  // unsigned: the last CTA's rows may pass 2^31 - 1
  const int row = (int)r;
  const int bh = row / p.N, i = row - bh * p.N;
  const int b = bh / p.c.Hkv;
  int n = p.N;
  if (p.count != nullptr) {
    n = p.count[b];
    if (n < 0 || n > p.N) {
      kv4_bad_index(p.c);
      n = n < 0 ? 0 : p.N;
    }
  }
  if (i >= n) return nullptr;
  const long long at = (long long)p.start[b] + i;
  if (at < 0 || at >= ((long long)p.c.max_pages << p.c.page_shift)) {
    kv4_bad_index(p.c);
    return nullptr;
  }
  const int page = kv4_page(p.c, b, (int)at);
  if (page < 0) return nullptr;
  *place = (int)at & 15;
  return kv4_block<D>(p.c, page, bh - b * p.c.Hkv, (int)at);
}

// Scale and codes of the 8 channels of this thread, whose group of 32 is held
// by a quad of lanes.
//
// The codes are those of the exact quotients x / s.  x has 8 significant bits
// and s has 8, so a quotient that is not one of the rounding borders
// (multiples of 1/4 up to 5) differs from each by more than 2^-13 of it (x
// and border * s are then different multiples of one unit, of which border * s
// holds at most 20 * 255).  x * (1 / s), two roundings, is within 2^-22 of the
// quotient, at most 7; adding and taking away 96 rounds it to a multiple of
// 2^-17.  So a quotient on a border lands on it exactly, and any other stays
// on its side: one reciprocal a group in place of 32 divisions.
__device__ __forceinline__ uint32_t kv4_quantise8(uint4 raw, uint32_t* scale_bits) {
  const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
  float x[8], top = 0.f;
  bool odd = false;  // a NaN or an infinity
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = bf16_lo(w[i]);
    x[2 * i + 1] = bf16_hi(w[i]);
    odd |= (w[i] & 0x7f80u) == 0x7f80u || (w[i] & 0x7f800000u) == 0x7f800000u;
    top = fmaxf(top, fmaxf(fabsf(x[2 * i]), fabsf(x[2 * i + 1])));
  }
  if (odd) top = INFINITY;
  top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
  top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
  const __nv_bfloat16 s16 = __float2bfloat16_rn(__fdiv_rn(top, 6.0f));
  float s = __bfloat162float(s16);
  const bool held = s >= 1.17549435e-38f && top < INFINITY;  // else all codes are 0
  *scale_bits = held ? __bfloat16_as_ushort(s16) : (top < INFINITY ? 0u : 0x7fffu);
  const float r = held ? __frcp_rn(s) : 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] = held ? fmaf(x[i], r, 96.0f) - 96.0f : 0.f;
  return kv4_encode8(x);
}

template <int D>
__global__ void __launch_bounds__(2 * D) kv4_write_kernel(const Kv4MoveParams p) {
  using F = Kv4<D>;
  constexpr int kPer = D / 8;  // threads a row
  const unsigned row = blockIdx.x * 16 + threadIdx.x / kPer;
  const int c8 = threadIdx.x % kPer;
  int place = 0;
  uint8_t* block = kv4_row<D>(p, row, &place);
  const size_t at = (size_t)row * kPer + c8;
  // Rows that take no part go through the shuffles with zeros.
  uint4 kr = make_uint4(0, 0, 0, 0), vr = kr;
  if (block != nullptr) {
    kr = p.k_in[at];
    vr = p.v_in[at];
  }
  const int g = c8 / 4, t = c8 % 4;
  uint32_t ks, vs;
  const uint32_t kw = kv4_quantise8(kr, &ks);
  const uint32_t vw = kv4_quantise8(vr, &vs);
  if (block == nullptr) return;
  *reinterpret_cast<uint32_t*>(block + F::key_word(place, g, t)) = kw;
  *reinterpret_cast<uint16_t*>(block + F::value_unit(place, g, 2 * t)) = (uint16_t)vw;
  *reinterpret_cast<uint16_t*>(block + F::value_unit(place, g, 2 * t + 1)) = (uint16_t)(vw >> 16);
  if (t == 0) {
    *reinterpret_cast<uint16_t*>(block + F::scale(place, 0, g)) = (uint16_t)ks;
    *reinterpret_cast<uint16_t*>(block + F::scale(place, 1, g)) = (uint16_t)vs;
  }
}

// 8 held values as bf16: code * scale has at most 10 significant bits, exact
// in fp32, so this rounds once.
__device__ __forceinline__ uint4 kv4_values8(uint32_t w, float s) {
  uint32_t h[4], o[4];
  kv4_decode8(w, h);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h[i]));
    o[i] = pack_bf16(f.x * s, f.y * s);
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
}

template <int D>
__global__ void __launch_bounds__(2 * D) kv4_read_kernel(const Kv4MoveParams p) {
  using F = Kv4<D>;
  constexpr int kPer = D / 8;
  const unsigned row = blockIdx.x * 16 + threadIdx.x / kPer;
  const int c8 = threadIdx.x % kPer;
  int place = 0;
  const uint8_t* block = kv4_row<D>(p, row, &place);
  if (block == nullptr) return;
  const int g = c8 / 4, t = c8 % 4;
  const uint32_t kw = *reinterpret_cast<const uint32_t*>(block + F::key_word(place, g, t));
  const uint32_t v0 = *reinterpret_cast<const uint16_t*>(block + F::value_unit(place, g, 2 * t));
  const uint32_t v1 = *reinterpret_cast<const uint16_t*>(block + F::value_unit(place, g, 2 * t + 1));
  const float ks = bf16_lo(*reinterpret_cast<const uint16_t*>(block + F::scale(place, 0, g)));
  const float vs = bf16_lo(*reinterpret_cast<const uint16_t*>(block + F::scale(place, 1, g)));
  const size_t at = (size_t)row * kPer + c8;
  p.k_out[at] = kv4_values8(kw, ks);
  p.v_out[at] = kv4_values8(v0 | (v1 << 16), vs);
}

template <int D>
static cudaError_t launch_move_t(bool write, const Kv4MoveParams& p, cudaStream_t stream) {
  const int grid = (int)(((long long)p.rows + 15) / 16);
  if (write)
    kv4_write_kernel<D><<<grid, 2 * D, 0, stream>>>(p);
  else
    kv4_read_kernel<D><<<grid, 2 * D, 0, stream>>>(p);
  return cudaGetLastError();
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
  p.rows = c.B * c.Hkv * N;
  switch (d) {
    case 64: return launch_move_t<64>(write, p, stream);
    case 96: return launch_move_t<96>(write, p, stream);
    case 128: return launch_move_t<128>(write, p, stream);
    case 256: return launch_move_t<256>(write, p, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace fa
