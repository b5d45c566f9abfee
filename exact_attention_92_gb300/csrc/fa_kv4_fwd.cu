// Attention over the 4-bit key/value cache (fa_kv4_fwd): one query row a CTA,
// tiles of 128 keys, fp32 throughout.
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "fa_common.h"
#include "sm103_primitives.cuh"
#include "kv4_format.cuh"
#include "kv4_fwd.h"

namespace fa {

using namespace dev;

template <int D>
__global__ void __launch_bounds__(128) kv4_fwd_kernel(const Kv4FwdParams p) {
  using F = Kv4<D>;
  constexpr int kT = 128;
  __shared__ float qs[D], sc[kT], red[4];
  const int tid = threadIdx.x, row = blockIdx.x;  // row of [B, H, Nq]
  const int qi = row % p.Nq, h = (row / p.Nq) % p.H, b = row / p.Nq / p.H;
  const int head = h / (p.H / p.c.Hkv);
  for (int c = tid; c < D; c += kT) qs[c] = __bfloat162float(p.q[(size_t)row * D + c]);
  __syncthreads();
  const int len = kv4_length(p.c, p.lens, b);
  const int seen = kv4_seen(p, len, qi);  // keys this row sees
  float m = -INFINITY, l = 0.f, acc[(D + kT - 1) / kT] = {};
  for (int j0 = 0; j0 < seen; j0 += kT) {
    const int j = j0 + tid;
    float s = -INFINITY;
    if (j < seen) {
      const int page = kv4_page(p.c, b, j);
      if (page >= 0) {
        const uint8_t* blk = kv4_block<D>(p.c, page, head, j);
        s = 0.f;
        for (int g = 0; g < F::kGroups; ++g) {
          float part = 0.f;
          for (int t = 0; t < 4; ++t) {
            uint32_t x[4];
            kv4_decode8(*reinterpret_cast<const uint32_t*>(blk + F::key_word(j & 15, g, t)), x);
            for (int i = 0; i < 4; ++i) {
              const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&x[i]));
              part = fmaf(qs[32 * g + 8 * t + 2 * i], f.x, fmaf(qs[32 * g + 8 * t + 2 * i + 1], f.y, part));
            }
          }
          s = fmaf(part, bf16_lo(*reinterpret_cast<const uint16_t*>(blk + F::scale(j & 15, 0, g))), s);
        }
        s *= p.scale_log2;
      }
    }
    float mx = s;
    for (int o = 16; o; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    if (tid % 32 == 0) red[tid / 32] = mx;
    __syncthreads();
    const float mn = fmaxf(m, fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3])));
    const float pr = s == -INFINITY ? 0.f : exp2f(s - mn);
    sc[tid] = pr;
    __syncthreads();
    const float f = m == -INFINITY ? 0.f : exp2f(m - mn);
    l *= f;
    for (int k = 0; k < kT; ++k) l += sc[k];
    for (int c = tid, a = 0; c < D; c += kT, ++a) {
      acc[a] *= f;
      for (int k = 0; k < kT; ++k) {
        if (sc[k] == 0.f) continue;  // keys not seen, pages out of range
        const int jj = j0 + k;
        const uint8_t* blk = kv4_block<D>(p.c, kv4_page(p.c, b, jj), head, jj);
        const int g = c / 32, u = c % 32 / 4;
        uint32_t x[4];
        kv4_decode8(*reinterpret_cast<const uint16_t*>(blk + F::value_unit(jj & 15, g, u)), x);
        const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&x[c % 4 / 2]));
        acc[a] = fmaf(sc[k] * bf16_lo(*reinterpret_cast<const uint16_t*>(blk + F::scale(jj & 15, 1, g))),
                      c % 2 ? v.y : v.x, acc[a]);
      }
    }
    m = mn;
    __syncthreads();
  }
  const float inv = l > 0.f ? 1.0f / l : 0.f;
  for (int c = tid, a = 0; c < D; c += kT, ++a) p.o[(size_t)row * D + c] = __float2bfloat16_rn(acc[a] * inv);
  if (tid == 0) p.lse[row] = l > 0.f ? (m + log2f(l)) * 0.69314718055994530942f : -INFINITY;
}

cudaError_t launch_kv4_fwd(int d, const Kv4FwdParams& p, cudaStream_t stream) {
  const int grid = p.c.B * p.H * p.Nq;
  switch (d) {
    case 64: kv4_fwd_kernel<64><<<grid, 128, 0, stream>>>(p); break;
    case 96: kv4_fwd_kernel<96><<<grid, 128, 0, stream>>>(p); break;
    case 128: kv4_fwd_kernel<128><<<grid, 128, 0, stream>>>(p); break;
    case 256: kv4_fwd_kernel<256><<<grid, 128, 0, stream>>>(p); break;
    default: return cudaErrorInvalidValue;
  }
  return cudaGetLastError();
}

}  // namespace fa
