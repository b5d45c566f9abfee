// Parameters of attention over the 4-bit cache, shared by the host call and
// the kernels.
#pragma once

#include <cuda_bf16.h>

#include "kv4_format.cuh"

namespace fa {

// Query rows of a tile: the N of the m16n8k16 matrix instructions.
constexpr int kKv4Rows = 8;

// A unit that more than one CTA works on: written by the CTA that holds its
// first step, for the merge.
struct Kv4Cut {
  int row;    // first of its rows in [B, H, Nq]; -1: none starts here
  int rows;
  int last;   // the last CTA that holds a part of it
  int pad;
};

struct Kv4FwdParams {
  Kv4Cache c;
  const __nv_bfloat16* q;  // [B, H, Nq, d]
  const int* lens;         // [B]
  __nv_bfloat16* o;        // [B, H, Nq, d]
  float* lse;              // [B, H, Nq]
  int Nq;
  int rows;                // (H / Hkv) * Nq: query rows that share a key/value head
  int row_blocks;          // ceil(rows / rows of a unit)
  int causal;              // FA_CAUSAL_*
  float scale_pow2;        // scale * log2(e): a power of two,
  float scale_rest;        // and what is left, 1 to 2 (more if the power is at its largest)
  int whole;               // 1: units are not cut
  int single;              // 1: nor does a CTA have more than one
  float* part_o;           // [2 * grid][rows of a unit][d]: partial sums (not whole)
  float2* part_ml;         // [2 * grid][rows of a unit]: reference and sum
  Kv4Cut* cuts;            // [grid]
  unsigned long long timeout_ns;
  uint32_t missing;        // bytes that every copy is announced with and does not bring (self-test; else 0)
};

namespace dev {

// A length, clamped to what the table can hold.
__device__ __forceinline__ int kv4_length(const Kv4Cache& c, int n) {
  const int most = c.max_pages << c.page_shift;
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
