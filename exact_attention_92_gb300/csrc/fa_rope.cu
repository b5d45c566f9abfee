// Rotary positions (include/fa.h, fa_rope): the channel pairs of queries and
// keys turned by angles that grow with the position.
//
// Pair i of a row at position t turns by theta = t * f_i:
//   (a, b) -> mscale * (a cos theta - b sin theta, b cos theta + a sin theta)
// and by -theta for gradients (the transpose of the rotation).  A pair is
// channels (i, i + rot/2), or (2i, 2i + 1) interleaved; channels from rot on
// are passed through.
//
// Angles.  t f_i in fp32 is off by t f_i 2^-24 radians: 0.008 at position
// 131072, more than the rounding to bf16.  So frequencies are held as the
// fraction of a turn a position in 64-bit fixed point, f_i / (2 pi) * 2^64: the
// product with the integer t, modulo 2^64, is the fraction of a turn itself,
// off by |t| 2^-65 turns (2^-33 at most: fa_rope_phases rounds to the nearest), and
// whole turns fall out of the integer arithmetic.  Its upper 32 bits, as a float, go
// to sincospif: in all an angle is off by less than 2^-24 of a half turn.
//
// Bound: memory, two bytes read and two written a channel.  A thread keeps the
// cosines and sines of eight pairs (16-byte loads) and walks the heads of its
// row with them, so that a row's angles are worked out once for all heads where
// there are rows enough to fill the GPU, and by more threads, a head or a few
// each, where there are not.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "sm103_primitives.cuh"

namespace fa {

int internal_device_setup(unsigned int** status, int* sm_count);
cudaError_t internal_timed_launch(int kernel, cudaStream_t stream, cudaError_t (*launch)(void*), void* ctx);

using namespace dev;

struct RopeSide {
  const __nv_bfloat16* x;
  __nv_bfloat16* y;
  long long xb, xr, xh;  // strides of batch, row, head in elements
  long long yb, yr, yh;
  int heads;
};

struct RopeParams {
  RopeSide s[2];  // queries, keys (heads = 0: none)
  const unsigned long long* phases;
  const int* positions;
  const int* start;
  long long rows;  // B * N
  int N, d, rot;
  int items;        // threads a row: turned pieces, then pieces passed through
  int turned;       // of these, the turned ones
  int chunk;        // heads a thread walks
  int chunks;       // ceil((heads of queries + of keys) / chunk)
  float mscale;     // times cos and sin
  float sign;       // -1: gradients
};

// VW: channels a piece, 8 (16 bytes) or 1 where rot does not divide so.  In the
// half layout a turned piece is VW pairs (VW channels of each half); interleaved
// it is VW/2 pairs, or one pair with VW = 1.
template <int VW, bool INTERLEAVED>
__global__ void __launch_bounds__(256) fa_rope_kernel(const RopeParams p) {
  constexpr int kPairs = VW == 1 ? 1 : (INTERLEAVED ? VW / 2 : VW);
  pdl_trigger();
  const long long task = (long long)blockIdx.x * 256 + threadIdx.x;
  const long long per_chunk = p.rows * p.items;
  if (task >= per_chunk * p.chunks) {
    pdl_wait();
    return;
  }
  const int hc = (int)(task / per_chunk);
  const long long rest = task - hc * per_chunk;
  const long long row = rest / p.items;
  const int item = (int)(rest - row * p.items);
  const int b = (int)(row / p.N), i = (int)(row - (long long)b * p.N);
  pdl_wait();

  const bool turn = item < p.turned;
  // First channel of the piece, and how far its partner channels are.
  const int c0 = turn ? item * (INTERLEAVED ? (VW == 1 ? 2 : VW) : VW) : p.rot + (item - p.turned) * VW;
  float cs[kPairs], sn[kPairs];
  if (turn) {
    const long long t = p.positions ? p.positions[row] : (p.start ? (long long)p.start[b] + i : i);
    const int pair0 = INTERLEAVED ? c0 / 2 : c0;
#pragma unroll
    for (int e = 0; e < kPairs; ++e) {
      const unsigned long long turns = p.phases[pair0 + e] * (unsigned long long)t;
      sincospif((float)(int)(turns >> 32) * 4.656612873077392578125e-10f, &sn[e], &cs[e]);  // 2^-31: half turns
      cs[e] *= p.mscale;
      sn[e] *= p.mscale * p.sign;
    }
  }
  const int h0 = hc * p.chunk, h1 = min(h0 + p.chunk, p.s[0].heads + p.s[1].heads);
#pragma unroll 1
  for (int side = 0; side < 2; ++side) {
    const RopeSide& s = p.s[side];
    const int lo = max(0, h0 - (side ? p.s[0].heads : 0)), hi = min(s.heads, h1 - (side ? p.s[0].heads : 0));
    if (lo >= hi) continue;
    const __nv_bfloat16* x = s.x + b * s.xb + i * s.xr + lo * s.xh + c0;
    __nv_bfloat16* y = s.y + b * s.yb + i * s.yr + lo * s.yh + c0;
    const int half = p.rot / 2;
    if (!turn) {
      if (s.x == s.y) continue;  // in place: already there
      for (int h = lo; h < hi; ++h, x += s.xh, y += s.yh) {
        if constexpr (VW == 1)
          *y = *x;
        else
          *reinterpret_cast<uint4*>(y) = *reinterpret_cast<const uint4*>(x);
      }
      continue;
    }
    if constexpr (VW == 1) {
      const int other = INTERLEAVED ? 1 : half;
      for (int h = lo; h < hi; ++h, x += s.xh, y += s.yh) {
        const float a = __bfloat162float(x[0]), c = __bfloat162float(x[other]);
        y[0] = __float2bfloat16_rn(fmaf(a, cs[0], -c * sn[0]));
        y[other] = __float2bfloat16_rn(fmaf(c, cs[0], a * sn[0]));
      }
    } else {
      // Four heads' loads are in flight at a time.
      constexpr int kU = 4;
      constexpr int kParts = INTERLEAVED ? 1 : 2;
      for (int h = lo; h < hi; h += kU, x += kU * s.xh, y += kU * s.yh) {
        uint4 v[kU][kParts];
#pragma unroll
        for (int u = 0; u < kU; ++u)
          if (h + u < hi) {
#pragma unroll
            for (int q = 0; q < kParts; ++q) v[u][q] = *reinterpret_cast<const uint4*>(x + u * s.xh + q * half);
          }
#pragma unroll
        for (int u = 0; u < kU; ++u) {
          if (h + u >= hi) continue;
          uint32_t* w0 = reinterpret_cast<uint32_t*>(&v[u][0]);
          if constexpr (INTERLEAVED) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float a = __uint_as_float(w0[e] << 16), c = __uint_as_float(w0[e] & 0xffff0000u);
              w0[e] = pack_bf16(fmaf(a, cs[e], -c * sn[e]), fmaf(c, cs[e], a * sn[e]));
            }
          } else {
            uint32_t* w1 = reinterpret_cast<uint32_t*>(&v[u][kParts - 1]);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float a0 = __uint_as_float(w0[e] << 16), a1 = __uint_as_float(w0[e] & 0xffff0000u);
              const float c0v = __uint_as_float(w1[e] << 16), c1v = __uint_as_float(w1[e] & 0xffff0000u);
              w0[e] = pack_bf16(fmaf(a0, cs[2 * e], -c0v * sn[2 * e]), fmaf(a1, cs[2 * e + 1], -c1v * sn[2 * e + 1]));
              w1[e] = pack_bf16(fmaf(c0v, cs[2 * e], a0 * sn[2 * e]), fmaf(c1v, cs[2 * e + 1], a1 * sn[2 * e + 1]));
            }
          }
#pragma unroll
          for (int q = 0; q < kParts; ++q) *reinterpret_cast<uint4*>(y + u * s.yh + q * half) = v[u][q];
        }
      }
    }
  }
}

}  // namespace fa

namespace {

struct Launch {
  fa::RopeParams p;
  bool wide, interleaved;
  long long blocks;
  cudaStream_t st;
};

cudaError_t run(void* ctx) {
  const Launch& l = *static_cast<const Launch*>(ctx);
  const dim3 grid((unsigned)l.blocks), block(256);
  auto* kern = l.wide ? (l.interleaved ? fa::fa_rope_kernel<8, true> : fa::fa_rope_kernel<8, false>)
                      : (l.interleaved ? fa::fa_rope_kernel<1, true> : fa::fa_rope_kernel<1, false>);
  return fa::launch_pdl(kern, grid, block, 0, l.st, l.p);
}

bool side(const fa_rows_t* x, const fa_rows_t* y, int heads, fa::RopeSide* s) {
  if (x == nullptr) return false;
  for (const fa_rows_t* t : {x, y})
    if (t == nullptr || t->ptr == nullptr || (reinterpret_cast<uintptr_t>(t->ptr) & 15u) != 0 ||
        t->batch_stride % 8 != 0 || t->row_stride % 8 != 0 || t->head_stride % 8 != 0)
      return false;
  s->x = static_cast<const __nv_bfloat16*>(x->ptr);
  s->y = static_cast<__nv_bfloat16*>(y->ptr);
  s->xb = x->batch_stride, s->xr = x->row_stride, s->xh = x->head_stride;
  s->yb = y->batch_stride, s->yr = y->row_stride, s->yh = y->head_stride;
  s->heads = heads;
  return true;
}

// The fraction of |x| (its distance from the integer below) in 128-bit fixed point,
// negated modulo 1 where x is negative.  Each step is exact down to 2^-128.
unsigned __int128 fraction(double x) {
  const double a = std::fabs(x);
  const double part = (a - std::floor(a)) * 18446744073709551616.0;  // 2^64
  const double hi = std::floor(part);
  const unsigned __int128 f =
      ((unsigned __int128)(uint64_t)hi << 64) + (uint64_t)((part - hi) * 18446744073709551616.0);
  return x < 0 ? 0 - f : f;
}

}  // namespace

extern "C" {

int fa_rope_phases(const double* inv_freq, int n, uint64_t* phases) {
  if (inv_freq == nullptr || phases == nullptr || n < 1) return FA_ERR_INVALID_ARG;
  for (int i = 0; i < n; ++i) {
    if (!std::isfinite(inv_freq[i])) return FA_ERR_INVALID_ARG;
    // 1 / (2 pi) in three doubles is off by 2^-164; their products with a frequency
    // below 2^64, as exact pairs, leave the nearest phase (a double's quotient alone
    // would be off by 2^-53 of itself, 2^-24 of a turn at position 2^31).
    const double x = std::fabs(inv_freq[i]);
    constexpr double kTurn[3] = {0x1.45f306dc9c883p-3, -0x1.6b01ec5417056p-57, -0x1.6447e493ad4cep-111};
    const double p0 = x * kTurn[0], p1 = x * kTurn[1];
    const unsigned __int128 turns = fraction(p0) + fraction(std::fma(x, kTurn[0], -p0)) + fraction(p1) +
                                    fraction(std::fma(x, kTurn[1], -p1)) + fraction(x * kTurn[2]);
    const uint64_t f = (uint64_t)((turns + ((unsigned __int128)1 << 63)) >> 64);
    phases[i] = inv_freq[i] < 0 ? 0 - f : f;
  }
  return FA_OK;
}

int fa_rope(const fa_rows_t* q, const fa_rows_t* k, const fa_rows_t* q_out, const fa_rows_t* k_out,
            const uint64_t* phases, const int* positions, const int* start, int B, int N, int H, int Hkv, int d, int rot,
            int interleaved, float mscale, int inverse, void* stream) {
  if (B < 1 || N < 1 || H < 1 || (k != nullptr && Hkv < 1) || !std::isfinite(mscale)) return FA_ERR_INVALID_ARG;
  if (d != 64 && d != 96 && d != 128 && d != 256) return FA_ERR_UNSUPPORTED;
  if (rot < 2 || rot > d || rot % 2 != 0) return FA_ERR_INVALID_ARG;
  if (phases == nullptr || (reinterpret_cast<uintptr_t>(phases) & 7u) != 0 ||
      (reinterpret_cast<uintptr_t>(positions) & 3u) != 0 || (reinterpret_cast<uintptr_t>(start) & 3u) != 0 ||
      (positions != nullptr && start != nullptr))
    return FA_ERR_INVALID_ARG;
  if ((long long)B * N > 0x7fffffffLL || (long long)H + (k ? Hkv : 0) > (1 << 20)) return FA_ERR_INVALID_ARG;
  Launch l;
  l.p.s[1] = {};
  if (!side(q, q_out, H, &l.p.s[0]) || (k != nullptr && !side(k, k_out, Hkv, &l.p.s[1]))) return FA_ERR_INVALID_ARG;
  unsigned int* status = nullptr;
  int sm_count = 0;
  const int e = fa::internal_device_setup(&status, &sm_count);
  if (e) return e;
  l.p.phases = reinterpret_cast<const unsigned long long*>(phases);
  l.p.positions = positions;
  l.p.start = start;
  l.p.rows = (long long)B * N;
  l.p.N = N;
  l.p.d = d;
  l.p.rot = rot;
  l.p.mscale = mscale;
  l.p.sign = inverse ? -1.f : 1.f;
  l.interleaved = interleaved != 0;
  l.wide = rot % (interleaved ? 8 : 16) == 0;
  const int piece = l.wide ? 8 : 1;
  l.p.turned = interleaved ? rot / (l.wide ? 8 : 2) : rot / 2 / piece;
  l.p.items = l.p.turned + (d - rot) / piece;
  // Heads a thread: the more, the fewer times an angle is worked out, as long as
  // there are threads for the GPU: 2048 an SM (8191 tokens, 12 + 4 heads of d = 96
  // 12.8 us; with 1024 an SM 14.1, with 4096 17.1).
  const int heads = H + l.p.s[1].heads;
  const long long room = (long long)sm_count * 2048;
  l.p.chunk = (int)std::max(1LL, std::min((long long)heads, l.p.rows * l.p.items * heads / room));
  l.p.chunks = (heads + l.p.chunk - 1) / l.p.chunk;
  const long long tasks = l.p.rows * l.p.items * l.p.chunks;
  l.blocks = (tasks + 255) / 256;
  if (l.blocks > 0x7fffffffLL) return FA_ERR_INVALID_ARG;
  l.st = static_cast<cudaStream_t>(stream);
  return fa::internal_timed_launch(FA_KERNEL_ROPE, l.st, run, &l) == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

}  // extern "C"
