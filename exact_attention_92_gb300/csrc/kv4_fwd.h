// Parameters of attention over the 4-bit cache, shared by the host call and
// the kernels.
#pragma once

#include <cuda_bf16.h>

#include "kv4_format.cuh"

namespace fa {

struct Kv4FwdParams {
  Kv4Cache c;
  const __nv_bfloat16* q;  // [B, H, Nq, d]
  const int* lens;         // [B]
  __nv_bfloat16* o;        // [B, H, Nq, d]
  float* lse;              // [B, H, Nq]
  int H;
  int Nq;
  int causal;              // FA_CAUSAL_*
  float scale_log2;        // scale * log2(e)
};

namespace dev {

// Length of sequence b, clamped to what the table can hold.
__device__ __forceinline__ int kv4_length(const Kv4Cache& c, const int* lens, int b) {
  const int most = c.max_pages << c.page_shift, n = lens[b];
  if (n >= 0 && n <= most) return n;
  kv4_bad_index(c);
  return n < 0 ? 0 : most;
}

// Keys that the row at query position qi sees, from the first on.
__device__ __forceinline__ int kv4_seen(const Kv4FwdParams& p, int len, int qi) {
  if (p.causal == FA_CAUSAL_NONE) return len;
  const int last = p.causal == FA_CAUSAL_BOTTOM_RIGHT ? qi + len - p.Nq : qi;
  return last < 0 ? 0 : (last + 1 < len ? last + 1 : len);
}

}  // namespace dev
}  // namespace fa
