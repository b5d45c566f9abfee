// Writing tokens into the 4-bit key/value cache and reading them back
// (fa_kv4_write, fa_kv4_read).
//
// A CTA takes the tokens of one call that share a 16-token block of the cache
// (of one head), so that sequence, page and block are worked out once for it; a
// thread takes 8 channels of a token's key and value.  Both kernels move each
// byte once, straight between global memory and registers, and are bound by
// that traffic (a token-head of d channels is 4 d bytes of bf16 and 9 d / 8 of
// cache) as long as a value costs few enough instructions: writing takes 163 for
// 16 values a lane (issue slots 70% taken).  Writing 4 x 8192 tokens of 8 heads
// at d = 128 and reading them back takes 56 us, 90% of what a copy moves;
// reading 2 x 32768 tokens 54 us, 94%.  CTAs past a sequence's tokens end at once:
// 24 pieces of up to 1000 tokens, half of that on average, at d = 64 take 13.3 us to
// write (16.6 with the work done on no tokens), 11.9 without such CTAs.
#include <cstdint>
#include <type_traits>

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
  int groups;         // CTAs that the N tokens of a sequence and head can touch
};

// Where a CTA's tokens are: U blocks of one sequence and head, thread `place`
// having a token in each.
template <int D, int U>
struct Kv4Tokens {
  size_t row;         // of the token in block 0, in [B, Hkv, N] (block u: 16 u rows on)
  int place;          // in the block
  uint32_t has;       // bit u: this thread has a row for block u
  bool all;           // of the CTA: every thread has one for every block
  int blocks;         // of the CTA: those before the tokens' end, 0 or less: none
  int page[U];        // of block u; -1: none, or out of range
  int in_page;        // 16-token blocks of a page before block 0
  int head;
};

template <int D, int U>
__device__ __forceinline__ Kv4Tokens<D, U> kv4_tokens(const Kv4MoveParams& p) {
  pdl_wait();
  pdl_trigger();
  Kv4Tokens<D, U> w;
  w.place = threadIdx.x / (D / 8);
  const int bh = (int)(blockIdx.x / (unsigned)p.groups), nth = (int)(blockIdx.x - (unsigned)bh * p.groups) * U;
  const int b = bh / p.c.Hkv;
  w.head = bh - b * p.c.Hkv;
  const int start = p.start[b];
  int n = p.N;
  if (p.count != nullptr) {
    n = p.count[b];
    if (n < 0 || n > p.N) {
      if (threadIdx.x == 0) kv4_bad_index(p.c);
      n = n < 0 ? 0 : p.N;
    }
  }
  // Block of the sequence (rounded down, where `start` is negative) and the
  // row of its first token.
  const int block0 = (start >> 4) + nth;
  const int i0 = nth * 16 - (start & 15);
  const int blocks = (int)(((long long)p.c.max_pages << p.c.page_shift) >> 4);
  const int* const table = p.c.table + (size_t)b * p.c.max_pages;
  const int shift = p.c.page_shift - 4;
  w.row = (size_t)bh * p.N + (ptrdiff_t)(i0 + w.place);
  w.has = 0;
  w.all = true;
  w.blocks = (n - i0 + 15) >> 4;
  w.in_page = block0;
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int i = i0 + 16 * u + w.place;
    w.page[u] = -1;
    if (i0 + 16 * u < n && i0 + 16 * u > -16) {  // for the whole CTA: some row is a token
      if ((unsigned)(block0 + u) < (unsigned)blocks) w.page[u] = table[(block0 + u) >> shift];
    }
    w.has |= (i >= 0 && i < n ? 1u : 0u) << u;
    w.all = w.all && i0 + 16 * u >= 0 && i0 + 16 * u + 16 <= n;
  }
  return w;
}

// Whether block u's page is in range; a thread with a row for it records that
// it is not.
template <int D, int U>
__device__ __forceinline__ bool kv4_there(const Kv4MoveParams& p, const Kv4Tokens<D, U>& w, int u) {
  if ((unsigned)w.page[u] < (unsigned)p.c.num_pages) return true;
  if ((w.has >> u) & 1) kv4_bad_index(p.c);
  return false;
}

// Block u of the CTA's tokens.
template <int D, int U>
__device__ __forceinline__ uint8_t* kv4_block_of(const Kv4MoveParams& p, const Kv4Tokens<D, U>& w, int u) {
  const int shift = p.c.page_shift - 4;
  const size_t first = ((size_t)w.page[u] * p.c.Hkv + w.head) << shift;
  return p.c.pages + (first + ((w.in_page + u) & ((1 << shift) - 1))) * Kv4<D>::kBlockBytes;
}

// Larger magnitudes of two pairs of bf16, with some sign; a NaN wins.
__device__ __forceinline__ uint32_t max_abs(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.NaN.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// Scales (as bf16 bits, the key's low) and the factors 1 / scale of a key's and
// a value's group whose largest magnitudes `top` holds (the key's low).  A
// factor is 0 where all codes are 0.
//
// The scale is top / 6 rounded to bf16.  top has 8 significant bits, so top / 6
// is never the middle of two bf16 (that has 9 bits, and 6 times it 10 or more)
// and lies 2^-12 of itself away from any: top * (1/6 in fp32) rounds alike.  It
// is at least 2^-126 from top = 6 * 2^-126 on, bits 0x01c0.
__device__ __forceinline__ uint32_t kv4_scales(uint32_t top, float* rk, float* rv) {
  uint32_t s = pack_bf16(bf16_lo(top) * 0.16666667163372040f, bf16_hi(top) * 0.16666667163372040f);
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(*rk) : "f"(bf16_lo(s)));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(*rv) : "f"(bf16_hi(s)));
  const uint32_t k = top & 0xffffu, v = top >> 16;
  if (k - 0x01c0u >= 0x7f80u - 0x01c0u || v - 0x01c0u >= 0x7f80u - 0x01c0u) {
    if (k < 0x01c0u || k >= 0x7f80u) {
      s = (s & 0xffff0000u) | (k < 0x01c0u ? 0u : 0x7fffu);
      *rk = 0.f;
    }
    if (v < 0x01c0u || v >= 0x7f80u) {
      s = (s & 0xffffu) | (v < 0x01c0u ? 0u : 0x7fff0000u);
      *rv = 0.f;
    }
  }
  return s;
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

template <int D, int U>
__global__ void __launch_bounds__(2 * D) kv4_write_kernel(const Kv4MoveParams p) {
  using F = Kv4<D>;
  constexpr int kPer = D / 8;
  const int c8 = threadIdx.x % kPer, g = c8 / 4, t = c8 % 4;
  const Kv4Tokens<D, U> w = kv4_tokens<D, U>(p);
  if (w.blocks <= 0) return;
  const uint4* const k_in = p.k_in + (ptrdiff_t)w.row * kPer + c8;
  const uint4* const v_in = p.v_in + (ptrdiff_t)w.row * kPer + c8;
  const int at_key = F::key_word(w.place, g, t), at_scale = F::scale(w.place, t & 1, g);
  const int at_value = F::kGroups % 2 == 0 ? F::value_unit(w.place, g & ~1, 2 * t + (g & 1))
                                           : F::value_unit(w.place, g, 2 * t);
  // ALL: every thread has a token in every block (most CTAs of a prompt).
  auto body = [&](auto all) {
    constexpr bool ALL = decltype(all)::value;
    uint4 kr[U], vr[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      kr[u] = vr[u] = make_uint4(0, 0, 0, 0);
      if (ALL || (w.has >> u) & 1) {
        kr[u] = k_in[u * 16 * kPer];
        vr[u] = v_in[u * 16 * kPer];
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (!ALL && u >= w.blocks) break;
      // A group's 32 channels are a quad of lanes: key and value in one word.
      const uint32_t km = max_abs(max_abs(kr[u].x, kr[u].y), max_abs(kr[u].z, kr[u].w));
      const uint32_t vm = max_abs(max_abs(vr[u].x, vr[u].y), max_abs(vr[u].z, vr[u].w));
      uint32_t top = max_abs(__byte_perm(km, vm, 0x5410), __byte_perm(km, vm, 0x7632));
      top = max_abs(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = max_abs(top, __shfl_xor_sync(0xffffffffu, top, 2)) & 0x7fff7fffu;
      float rk, rv;
      const uint32_t scales = kv4_scales(top, &rk, &rv);
      uint32_t kw = kv4_codes8(kr[u], rk), vw = kv4_codes8(vr[u], rv);
      kw = rk == 0.f ? 0u : kw;
      vw = rv == 0.f ? 0u : vw;
      if constexpr (F::kGroups % 2 == 0) vw = exchange_units(vw, g & 1);
      if ((!ALL && !((w.has >> u) & 1)) || !kv4_there<D, U>(p, w, u)) continue;
      uint8_t* const block = kv4_block_of<D, U>(p, w, u);
      *reinterpret_cast<uint32_t*>(block + at_key) = kw;
      if constexpr (F::kGroups % 2 == 0) {
        *reinterpret_cast<uint32_t*>(block + at_value) = vw;
      } else {
        *reinterpret_cast<uint16_t*>(block + at_value) = (uint16_t)vw;
        *reinterpret_cast<uint16_t*>(block + F::value_unit(w.place, g, 2 * t + 1)) = (uint16_t)(vw >> 16);
      }
      if (t < 2) *reinterpret_cast<uint16_t*>(block + at_scale) = (uint16_t)(t == 0 ? scales : scales >> 16);
    }
  };
  if (w.all)
    body(std::true_type{});
  else
    body(std::false_type{});
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

template <int D, int U>
__global__ void __launch_bounds__(2 * D) kv4_read_kernel(const Kv4MoveParams p) {
  using F = Kv4<D>;
  constexpr int kPer = D / 8;
  const int c8 = threadIdx.x % kPer, g = c8 / 4, t = c8 % 4;
  Kv4Tokens<D, U> w = kv4_tokens<D, U>(p);
  if (w.blocks <= 0) return;
#pragma unroll
  for (int u = 0; u < U; ++u)
    if (!kv4_there<D, U>(p, w, u)) {
      w.has &= ~(1u << u);
      w.all = false;
    }
  uint4* const k_out = p.k_out + (ptrdiff_t)w.row * kPer + c8;
  uint4* const v_out = p.v_out + (ptrdiff_t)w.row * kPer + c8;
  auto body = [&](auto all) {
    constexpr bool ALL = decltype(all)::value;
    uint32_t kw[U], vw[U], ks[U], vs[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      kw[u] = vw[u] = ks[u] = vs[u] = 0;
      if (ALL || (w.has >> u) & 1) {
        const uint8_t* const block = kv4_block_of<D, U>(p, w, u);
        kw[u] = *reinterpret_cast<const uint32_t*>(block + F::key_word(w.place, g, t));
        ks[u] = *reinterpret_cast<const uint16_t*>(block + F::scale(w.place, 0, g));
        vs[u] = *reinterpret_cast<const uint16_t*>(block + F::scale(w.place, 1, g));
        if constexpr (F::kGroups % 2 == 0)
          vw[u] = *reinterpret_cast<const uint32_t*>(block + F::value_unit(w.place, g & ~1, 2 * t + (g & 1)));
        else
          vw[u] = *reinterpret_cast<const uint16_t*>(block + F::value_unit(w.place, g, 2 * t)) |
                  ((uint32_t)*reinterpret_cast<const uint16_t*>(block + F::value_unit(w.place, g, 2 * t + 1)) << 16);
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if constexpr (F::kGroups % 2 == 0) vw[u] = exchange_units(vw[u], g & 1);
      if (!ALL && !((w.has >> u) & 1)) continue;
      k_out[u * 16 * kPer] = kv4_values8(kw[u], bf16_lo(ks[u]));
      v_out[u * 16 * kPer] = kv4_values8(vw[u], bf16_lo(vs[u]));
    }
  };
  if (w.all)
    body(std::true_type{});
  else
    body(std::false_type{});
}

template <int D, int U>
static cudaError_t launch_move_u(void (*kernel)(Kv4MoveParams), Kv4MoveParams& p, cudaStream_t stream) {
  // N tokens touch (N + 30) / 16 blocks at most, wherever they begin.
  p.groups = (int)((((long long)p.N + 30) / 16 + U - 1) / U);
  const unsigned grid = (unsigned)p.c.B * p.c.Hkv * p.groups;
  return launch_pdl(kernel, dim3(grid), dim3(2 * D), 0, stream, p);
}

template <int D>
static cudaError_t launch_move_t(bool write, Kv4MoveParams& p, int sm_count, cudaStream_t stream) {
  // Several blocks a CTA keep enough loads in flight (writing and reading 4 x 8192
  // tokens of 8 heads at d = 128: 57.0 us, with one block 67.1); where that leaves
  // SMs without a CTA, one block each is sooner done (100 tokens of 12 heads at
  // d = 96, read: 1.66 us, with two blocks 1.86).  Writing takes four (4 x 8192 tokens
  // 27.7 us, with two 28.8).  Reading takes two (28.1 us, with four 28.8; 24 pieces
  // of up to 1000 tokens at d = 96 20.3 and 21.0), but four at d = 64, whose CTAs
  // have half the threads (such pieces written and read back 28.7 us, with two 30.6;
  // read alone 14.2 and 14.6, all of them full 22.4 and 21.7).
  constexpr int R = D == 64 ? 4 : 2;
  const bool many = (long long)p.c.B * p.c.Hkv * (p.N / 64) >= 2ll * sm_count;
  if (write)
    return many ? launch_move_u<D, 4>(kv4_write_kernel<D, 4>, p, stream)
                : launch_move_u<D, 1>(kv4_write_kernel<D, 1>, p, stream);
  return many ? launch_move_u<D, R>(kv4_read_kernel<D, R>, p, stream)
              : launch_move_u<D, 1>(kv4_read_kernel<D, 1>, p, stream);
}

cudaError_t launch_kv4_move(int d, bool write, const Kv4Cache& c, const int* start, const int* count, const void* k_in,
                            const void* v_in, void* k_out, void* v_out, int N, int sm_count, cudaStream_t stream) {
  Kv4MoveParams p;
  p.c = c;
  p.start = start;
  p.count = count;
  p.k_in = static_cast<const uint4*>(k_in);
  p.v_in = static_cast<const uint4*>(v_in);
  p.k_out = static_cast<uint4*>(k_out);
  p.v_out = static_cast<uint4*>(v_out);
  p.N = N;
  switch (d) {
    case 64: return launch_move_t<64>(write, p, sm_count, stream);
    case 96: return launch_move_t<96>(write, p, sm_count, stream);
    case 128: return launch_move_t<128>(write, p, sm_count, stream);
    case 256: return launch_move_t<256>(write, p, sm_count, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace fa
