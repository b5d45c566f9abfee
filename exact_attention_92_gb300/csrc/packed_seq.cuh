// What the planning kernels of packed sequences share: a sequence's bounds, sums
// over a CTA, and which sequence the i-th block is of.
#pragma once

#include "packed.h"
#include "sm103_primitives.cuh"

namespace fa {
namespace {

constexpr int kPlanThreads = 1024;

struct Seq {
  int q, q_len, k, k_len;
};

// Where sequence b starts, as far as it is within the rows (0 otherwise).  A sequence
// is out of order where one before it starts further on: taken all the same, such
// sequences would overlap and have more blocks than there is room for.
__device__ __forceinline__ int start_of(const int* cu, int b, int rows) {
  const int x = cu[b];
  return x >= 0 && x <= rows ? x : 0;
}

// Sequence b; one whose bounds are out of order or out of the tensors is empty
// (and reported).  first_q: the furthest start of the sequences up to this one.
__device__ __forceinline__ Seq load_seq(const PackedSeqs& s, int b, int first_q, int first_k = 0) {
  const int q0 = s.cu_q[b], q1 = s.cu_q[b + 1], k0 = s.cu_k[b], k1 = s.cu_k[b + 1];
  bool bad = q0 < first_q || q0 < 0 || q1 < q0 || q1 > s.Tq || k0 < first_k || k0 < 0 || k1 < k0 || k1 > s.Tk;
  int n = k1 - k0;
  if (!bad && s.used_k != nullptr) {
    const int used = s.used_k[b];
    bad = used < 0 || used > n;
    n = used;
  }
  if (bad) {
    atomicCAS(s.status + 1, 0u, (unsigned int)FA_ERR_BAD_INDEX);
    return Seq{0, 0, 0, 0};
  }
  return Seq{q0, q1 - q0, k0, n};
}

// Sums (or, MAX, largest values) over a CTA: of the threads up to this one, and of
// all.  Two sets of words taken in turn, so that one barrier a scan is enough.
template <typename T, bool MAX = false>
struct Scan {
  T (*warps)[32];
  int turn;
  __device__ __forceinline__ explicit Scan(T (*w)[32]) : warps(w), turn(0) {}
  __device__ __forceinline__ static T join(T a, T b) { return MAX ? (a > b ? a : b) : a + b; }
  __device__ __forceinline__ T operator()(T v, T* total) {
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    T* sums = warps[turn];
    turn ^= 1;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const T x = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) v = join(v, x);
    }
    if (lane == 31) sums[w] = v;
    __syncthreads();
    T x = sums[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const T y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x = join(x, y);
    }
    *total = __shfl_sync(0xffffffffu, x, 31);
    const T before = __shfl_sync(0xffffffffu, x, w > 0 ? w - 1 : 0);
    return w > 0 ? join(v, before) : v;
  }
};

// The sequence of block i, with base[b] the first block of sequence b: the last
// that starts at or before it.
__device__ __forceinline__ int seq_of(const int* base, int B, int i) {
  int lo = 0, hi = B;
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (base[mid] <= i) lo = mid; else hi = mid;
  }
  return lo;
}

// Blocks of a sequence, by list: whole ones, and at most one small one behind them.
__device__ __forceinline__ int2 blocks_of(const Seq& s, int tile_tokens) {
  const int block = 2 * tile_tokens, rest = s.q_len % block;
  return make_int2(s.q_len / block + (rest > tile_tokens), rest > 0 && rest <= tile_tokens);
}

// The block of a sequence that starts at its token t0, behind `prefix` tiles.
__device__ __forceinline__ PackedEntry block_at(const Seq& s, int t0, int block, int prefix, int causal) {
  PackedEntry x;
  x.q_row = s.q + t0;
  x.q_len = min(block, s.q_len - t0);
  x.k_row = s.k;
  x.k_len = s.k_len;
  x.prefix = prefix;
  x.pos = t0 + (causal == FA_CAUSAL_BOTTOM_RIGHT ? s.k_len - s.q_len : 0);
  const int seen = causal == FA_CAUSAL_NONE ? s.k_len : min(s.k_len, max(0, x.pos + x.q_len));
  x.tiles = prefix + (seen + kTileN - 1) / kTileN;
  x.kind = 0;
  return x;
}

}  // namespace
}  // namespace fa
