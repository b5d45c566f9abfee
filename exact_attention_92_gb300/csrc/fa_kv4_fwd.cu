// Attention over the 4-bit key/value cache (fa_kv4_fwd).
//
// A unit is a (sequence, key/value head, block of 4, 8, 16 or 24 of the
// group's query rows); its keys are walked in steps of 32.  The steps of all units form
// one list, in the order of the units, of which every CTA takes an equal stretch
// whatever the sequences' lengths, and every warp of it an equal stretch of
// that.  Where a border cuts a unit, the warps of a CTA join their fp32 results
// at the CTA's end, and a second kernel merges those of the CTAs, both in the
// order of the list, so the results do not change from run to run.  (Warps that
// took a CTA's steps in turn and joined at each unit's end, in an earlier form of
// the kernel: 64 ragged sequences 127 us in place of 109.)
//
// Each warp fetches its own steps: bulk copies of whole 16-token blocks into a
// ring in shared memory, ahead of use, so no warp waits for another within a
// unit.  A step computes S^T = K Q^T and O^T += V^T P^T with m16n8k16
// instructions on fp16 (16 keys, or 16 channels, by 8 query rows): the keys and
// values are the row operand, so the decoding of 8 query rows wastes nothing,
// and their codes go from shared memory through one conversion instruction per
// two values into the operand's registers.  With up to 4 query rows (PACK) the
// two 16-key blocks of a step share the 8 columns, which halves the softmax's
// share of the instructions (100.5 -> 94.6 us in the case below).
// (A tcgen05 product would want the 128-row operand in shared memory, decoded:
// 512 bytes written and read back a token for 144 bytes of cache.)
//
// What bounds it (d = 128, 64 sequences of up to 16384 tokens, 8 heads, 4 rows,
// 552 MB): 94.6 us, 5.8 TB/s of DRAM reads, 86% of what a copy moves.  512
// instructions a step and warp, 58% of the issue slots while SMs are busy; 128 of
// them are conversions from e2m1 and about 100 others of the same half-rate pipe,
// which so is in use 61% of the time; the matrix pipe 29%.  Scores, weights and
// their sums are packed fp32 (20 instructions a step fewer; an earlier form of the
// step took 94.3 us with them and 96.7 without).
// Of a call of 8 sequences of 8192 tokens (22.4 us, 11.2 us of traffic) 3.4 us
// go before the first copies are on the way (lengths 0.9, place in the list 1.3,
// page and issue 1.2) and 2.3 until their bytes are there; the warps end their
// steps (9 or 10 each) between 14 and 19.6 us, 1.2 us go for the join and about 2
// for the merge.
//
// Numbers.  Codes are exact in fp16.  A query row is scaled by a power of two
// to lie just below 2^16, where fp16 holds its bf16 values exactly down to
// 2^-29 of the row's largest; the products of one group of 32 channels are
// summed by the matrix instruction in fp32, multiplied by the group's scale over
// that power of two (and times that of the softmax's scale) in fp32 and added, so
// scores are those of the exact held values.  The weights
// p = 2^(s - ref) are multiplied by the values' scale in fp32 and rounded once
// to fp16 (11 bits) for the P V product: bf16 would lose three bits, and 8 bits
// of weight are what the output's own rounding costs.  To keep p * scale within
// fp16 the running reference is that of s + log2(the largest scale of the
// token's value), not of s: p * scale starts at 2^4 for the largest key seen and
// may grow to 2^14 before the reference is moved (and the sums rescaled); what
// falls below 2^-14 of that loses relative, not absolute, precision.  A weight is
// 2^((x - ref) - log2(scale)) of the same rounded x = s + log2(scale) that moves
// the reference, so it keeps that bound where fp32 holds scores in steps of 4 and
// more.  The sum of p is fp32.  The scale is taken at 2^-80 at least: p stays below
// 2^94, and the sum over the 2^30 positions that a table may have below 2^124.
#include <atomic>
#include <cstdint>
#include <type_traits>

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "fa_common.h"
#include "sm103_primitives.cuh"
#include "kv4_format.cuh"
#include "kv4_fwd.h"

namespace fa {

using namespace dev;

namespace {

template <int D, int NR, bool PACK>
struct Cfg {
  // One CTA an SM, its warps a multiple of the four schedulers and as many as
  // their registers allow without spilling more than a few words outside the main
  // loop's sums (65536 over 16, 12 or 8 warps: 128, 168 or 255 each).  16 warps at
  // d = 128 spill and take 102.4 us in place of 94.7 in the case above.  At d = 96
  // 12 warps are a little sooner done than 16 (9 ragged sequences, two units of 8
  // rows 14.4 us and 14.9; 8 rows, 32 sequences of up to 4000 tokens 23.7 and 24.1,
  // 16 of 8192 33.5 and 33.5), and with two row tiles 12 spill: long calls are 2%
  // faster (16 rows, 16 sequences of 8192 47.0 and 48.1), short ones 6% slower (15
  // rows, 9 ragged ones 16.7 and 15.7).
  static constexpr int kWarps = D == 256 || NR == 3 || (NR == 2 && D > 64) ? 8 : NR == 1 && D == 64 ? 16 : 12;
  static constexpr int kThreads = kWarps * 32;
  static constexpr int kBlocks = 2;                             // 16-token blocks a step
  static constexpr int kKeys = kBlocks * kKv4Block;
  static constexpr int kStages = D == 256 || (D == 128 && NR == 1) ? 2 : 3;
  static constexpr int kStageBytes = kBlocks * Kv4<D>::kBlockBytes;
  static constexpr int kRows = PACK ? kKv4Rows / 2 : NR * kKv4Rows;  // query rows of a unit
  static_assert(!PACK || (NR == 1 && kBlocks == 2), "two blocks share the columns of a tile");
  // Shared memory: a ring of steps and the sums of a unit's head for each
  // warp (the sums of a tail go to the ring, which is empty by then).
  static constexpr int kRing = kStages * kStageBytes;
  static constexpr int kSums = kRows * D * 4;
  static constexpr int kSmem = kWarps * (kRing + kSums);
  static_assert(kSmem + 8 * 1024 <= 227 * 1024, "shared memory of an SM, 8 KB of it static");
  static_assert(kRing >= kSums, "a tail's sums go where the ring was");
  static_assert(kWarps <= 30, "a lane for each warp's results, and one for a tail's");
};

// Places of the list that a unit takes besides one for each of its steps: what
// it costs a warp, its query rows among it.
constexpr int kUnitCost = 2;

// A unit, or a stretch of its steps, that a warp has to do.
struct Piece {
  int b, u, head;  // sequence; unit within it; key/value head
  int len, steps;  // of the sequence, of each of its units
  int lo, hi;      // steps to do
  int place;       // of the unit in the list
};

// A part of a unit that a warp leaves to be joined with its neighbours'.
struct Part {
  int row, rows;   // the unit's rows in [B, H, Nq]
  int place;       // of the unit in the list
  int steps;       // of the unit
};
struct Left {
  int kinds;       // bit 0: a unit's beginning (tail); bits 1, 2: a middle or an end (head), an end
  Part head, tail;
};

__device__ __forceinline__ void mma16816(float* c, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Transpose of an 8 x 8 matrix of 16-bit values held by a warp.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                   smem_u32(dst)),
               "l"(src), "r"(bytes), "r"(smem_u32(bar))
               : "memory");
}

// N consecutive words of shared memory (N words are N * 4 bytes aligned for
// N = 1, 2, 4, else 4).
template <int N>
__device__ __forceinline__ void load_words(const uint8_t* p, uint32_t* w) {
  if constexpr (N % 4 == 0) {
#pragma unroll
    for (int i = 0; i < N; i += 4) *reinterpret_cast<uint4*>(w + i) = *reinterpret_cast<const uint4*>(p + 4 * i);
  } else if constexpr (N == 2) {
    *reinterpret_cast<uint2*>(w) = *reinterpret_cast<const uint2*>(p);
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) w[i] = *reinterpret_cast<const uint32_t*>(p + 4 * i);
  }
}

// Words g = 0..NG-1 of lane t of the key in row `slot` of a block.
template <int D>
__device__ __forceinline__ void load_key(const uint8_t* block, int slot, int t, uint32_t* w) {
  using F = Kv4<D>;
  if constexpr (D == 256) {
    load_words<4>(block + F::key_word(slot, 0, t), w);
    load_words<4>(block + F::key_word(slot, 4, t), w + 4);
  } else {
    load_words<F::kQuad>(block + F::key_word(slot, 0, t), w);
  }
}

// Channels 4 u .. 4 u + 3 of every group of row `row` of the values: group g in
// half g % 2 of word g / 2.
template <int D>
__device__ __forceinline__ void load_value(const uint8_t* block, int row, int u, uint32_t* w) {
  using F = Kv4<D>;
  const uint8_t* p = block + F::kValues + row * F::kRowBytes + ((u * F::kGroups * 2) ^ F::value_xor(row));
  if constexpr (D == 96) {
    const uint16_t* h = reinterpret_cast<const uint16_t*>(p);
    w[0] = h[0] | ((uint32_t)h[1] << 16);
    w[1] = h[2];
  } else {
    load_words<F::kGroups / 2>(p, w);
  }
}

// Scales of a token: NG of the key, NG of the value, as bf16 pairs.
template <int D>
__device__ __forceinline__ void load_scales(const uint8_t* block, int token, uint32_t* w) {
  load_words<Kv4<D>::kGroups>(block + Kv4<D>::kScales + token * Kv4<D>::kScaleBytes, w);
}
// The largest scale of a token's value, 2^-80 at least; NaN does not count.
template <int NG>
__device__ __forceinline__ float largest_scale(const uint32_t* w) {
  constexpr float kLeast = 8.271806125530277e-25f;
  if constexpr (NG % 2 == 0) {
    uint32_t m = w[NG / 2];
#pragma unroll
    for (int i = NG / 2 + 1; i < NG; ++i) asm("max.bf16x2 %0, %0, %1;" : "+r"(m) : "r"(w[i]));
    return fmax3(bf16_lo(m), bf16_hi(m), kLeast);
  } else {
    float m = kLeast;
#pragma unroll
    for (int i = NG; i < 2 * NG; ++i) m = fmaxf(m, i & 1 ? bf16_hi(w[i / 2]) : bf16_lo(w[i / 2]));
    return m;
  }
}
__device__ __forceinline__ float scale_of(const uint32_t* w, int i) { return i & 1 ? bf16_hi(w[i / 2]) : bf16_lo(w[i / 2]); }

// Place of the n-th bit that is set (n from 0).
__device__ __forceinline__ int nth_bit(uint32_t x, int n) {
  for (; n > 0; --n) x &= x - 1;
  return __ffs(x) - 1;
}

}  // namespace

template <int D, int NR, bool PACK>
__global__ void __launch_bounds__(Cfg<D, NR, PACK>::kThreads, 1) kv4_fwd_kernel(const Kv4FwdParams p) {
  using F = Kv4<D>;
  using C = Cfg<D, NR, PACK>;
  constexpr int NG = F::kGroups, W = C::kWarps;
  constexpr int kQueue = 8;  // pieces between the copies and the products
  static_assert(kQueue >= C::kStages + 2, "a piece has a step at least");
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ uint64_t bars[W * C::kStages];
  __shared__ Piece queue[W * kQueue];
  __shared__ Left left[W];
  __shared__ float2 stats[2][W * C::kRows];  // reference and sum of heads, of tails
  __shared__ int lims[W * C::kRows];

  // Through a shuffle, so that what follows from it stays in uniform registers.
  auto uniform = [](int x) { return __shfl_sync(0xffffffffu, x, 0); };
  const int tid = threadIdx.x, warp = uniform(tid / 32), lane = tid % 32, g = lane / 4, t = lane % 4;
  // Columns col0, col0 + 1 of a tile are this lane's query rows; where two blocks
  // share a tile, they are those of block my_blk.
  const int col0 = PACK ? 2 * (t & 1) : 2 * t, my_blk = PACK ? t >> 1 : 0;
  const int units = p.c.Hkv * p.row_blocks;  // of a sequence
  const WaitCtl ctl{p.c.status, p.timeout_ns};

  if (lane < C::kStages) {  // each warp its own
    mbar_init(&bars[warp * C::kStages + lane], 1);
    fence_barrier_init();
  }
  pdl_wait();
  pdl_trigger();

  // Steps of a unit of a sequence of n tokens; one at least, so that its rows
  // are written.
  auto steps_of = [&](int n) {
    if (p.causal == FA_CAUSAL_TOP_LEFT && n > p.Nq) n = p.Nq;
    return n == 0 ? 1 : (n + C::kKeys - 1) / C::kKeys;
  };

  auto length = [&](int b) { return kv4_length(p.c, p.lens[b]); };
  Piece ahead;
  ahead.lo = ahead.hi = 0;
  const int* row = nullptr;  // of the block table
  auto sequence = [&] {
    ahead.len = uniform(length(ahead.b));
    ahead.steps = steps_of(ahead.len);
    row = p.c.table + (size_t)ahead.b * p.c.max_pages;
  };

  // ---- the list (the host has checked that its places fit 31 bits).  Every
  // warp works it out for itself, each lane adding up a run of sequences: the
  // warps need not wait for each other before their copies are on the way.
  const int run = (p.c.B + 31) / 32;
  int upto = 0, total = 0;
  if (!p.single) {
    const int b_end = min(p.c.B, lane * run + run);
    for (int b = lane * run; b < b_end; b += 4) {
      int n[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) n[i] = b + i < b_end ? p.lens[b + i] : 0;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (b + i < b_end) upto += kUnitCost + steps_of(kv4_length(p.c, n[i]));
    }
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += x;
    }
    total = __shfl_sync(0xffffffffu, upto, 31) * units;
  }
  if (tid == 0 && !p.whole) p.cuts[blockIdx.x].row = -1;
  // Sequence, unit, place within it and places of the unit at list place x.
  struct Found {
    int b, u, off, places;
  };
  auto find = [&](int x) {
    Found f;
    const int r = __ffs(__ballot_sync(0xffffffffu, upto * units > x)) - 1;
    int rest = x - (r > 0 ? __shfl_sync(0xffffffffu, upto, r - 1) * units : 0);
    f.b = r * run;
    f.places = kUnitCost + steps_of(length(f.b));
    while (rest >= f.places * units && f.b + 1 < p.c.B) {
      rest -= f.places * units;
      f.places = kUnitCost + steps_of(length(++f.b));
    }
    f.u = rest / f.places;
    f.off = rest - f.u * f.places;
    return f;
  };
  // This CTA's stretch of the list: [first, end).  CTAs that take part: a place
  // for every warp, or a unit each; the first `more` have a place more than the
  // others.  Where every unit has a CTA of its own, the list need not be known.
  int each = 1, more = 0, first = 0, end = 0;
  if (p.single) {
    ahead.b = (int)blockIdx.x / units;
    ahead.u = (int)blockIdx.x - ahead.b * units;
    sequence();
    end = kUnitCost + ahead.steps;
  } else {
    const int active = min((int)gridDim.x, max(total / W, p.c.B * units));
    if ((int)blockIdx.x >= active) return;
    each = total / active;
    more = total - each * active;
    first = (int)blockIdx.x * each + min((int)blockIdx.x, more);
    end = first + each + ((int)blockIdx.x < more ? 1 : 0);
    if (p.whole) {  // the units that begin in the stretch
      const Found f = find(first);
      if (f.off > 0) first += f.places - f.off;
      if (end < total) {
        const Found e = find(end);
        if (e.off > 0) end += e.places - e.off;
      }
    }
    if (first >= end) return;
  }
  auto cta_of = [&](int place) {
    return place < more * (each + 1) ? place / (each + 1) : more + (place - more * (each + 1)) / each;
  };
  // ---- this warp's stretch of it, walked by the copies
  const int warp_each = (end - first) / W, warp_more = (end - first) - warp_each * W;
  int at = first + warp * warp_each + min(warp, warp_more);
  const int my_end = at + warp_each + (warp < warp_more ? 1 : 0);
  int made = 0, taken = 0;  // pieces put into the queue, and taken out
  auto enter = [&](int off) {
    ahead.head = p.row_blocks == 1 ? ahead.u : ahead.u / p.row_blocks;
    const int upto_off = min(ahead.steps + kUnitCost, off + my_end - at);
    ahead.lo = max(0, off - kUnitCost);
    ahead.hi = max(ahead.lo, upto_off - kUnitCost);
    ahead.place = at - off;
    at += upto_off - off;
    if (ahead.lo < ahead.hi) {
      if (lane == 0) queue[warp * kQueue + made % kQueue] = ahead;
      ++made;
      // Its query rows, nearer before they are wanted (1% of a decoding step).
      const int row0 = (ahead.u - ahead.head * p.row_blocks) * C::kRows;
      const int n_rows = min(C::kRows, p.rows - row0);
      const size_t row_at = ((size_t)ahead.b * p.c.Hkv + ahead.head) * p.rows + row0;
      if (lane * 64 < n_rows * D)
        asm volatile("prefetch.global.L2 [%0];" ::"l"(p.q + row_at * D + lane * 64) : "memory");
    }
  };
  // To the next unit; where the stretch is at its end, lo = hi.
  auto next_unit = [&] {
    ahead.lo = ahead.hi;
    if (at >= my_end) return;
    if (++ahead.u == units) {
      ahead.u = 0;
      if (++ahead.b == p.c.B) {
        at = my_end;
        return;
      }
      sequence();
    }
    enter(0);
  };
  if (at < my_end) {
    if (p.single) {
      enter(at);
    } else {
      const Found f = find(at);
      ahead.b = f.b;
      ahead.u = f.u;
      sequence();
      enter(f.off);
    }
  }

  // A copy takes the blocks of a step that lie in one page, all of them where
  // pages are long enough; lane i issues the step's copy i, whose page it has
  // looked up a step before.
  uint8_t* const ring = smem + warp * C::kRing;
  uint64_t* const bar = bars + warp * C::kStages;
  const int copy_blocks = min(C::kBlocks, 1 << (p.c.page_shift - 4));
  const uint32_t copy_bytes = copy_blocks * F::kBlockBytes;
  const int my_key = lane * copy_blocks * kKv4Block;  // of this lane's copy in a step; past the step: no copy
  const uint32_t have_all = (1u << (C::kBlocks / copy_blocks)) - 1;
  const int page_mask = (1 << p.c.page_shift) - 1;
  const uint32_t page_bytes = (uint32_t)F::kBlockBytes << (p.c.page_shift - 4);
  uint32_t have = 0;  // copies that were made, kBlocks bits a stage, the newest stage in the lowest
  int page = -1;      // of this lane's copy of the step at ahead.lo, -1: none
  auto look_up = [&] {
    const int pos = ahead.lo * C::kKeys + my_key;
    page = -1;
    if (my_key < C::kKeys && pos < ahead.len && ahead.lo < ahead.hi) page = row[pos >> p.c.page_shift];
  };
  auto issue = [&](int stage) {
    if (ahead.lo == ahead.hi) return;
    const int pos = ahead.lo * C::kKeys + my_key;
    bool good = (unsigned)page < (unsigned)p.c.num_pages;
    if (!good && my_key < C::kKeys && pos < ahead.len) kv4_bad_index(p.c);
    const uint32_t ones = __ballot_sync(0xffffffffu, good);
    have = (have << C::kBlocks) | ones;
    if (lane == 0) mbar_arrive_expect_tx(&bar[stage], __popc(ones) * copy_bytes + p.missing);
    __syncwarp();
    if (good)
      bulk_load(ring + stage * C::kStageBytes + lane * copy_bytes,
                p.c.pages + ((size_t)page * p.c.Hkv + ahead.head) * page_bytes +
                    ((pos & page_mask) / kKv4Block) * F::kBlockBytes,
                copy_bytes, &bar[stage]);
    if (++ahead.lo == ahead.hi) next_unit();
    look_up();
  };
  look_up();
  int in_flight = 0;  // stages issued and not yet waited for
#pragma unroll 1
  for (int s = 0; s < C::kStages; ++s) {
    in_flight += ahead.lo < ahead.hi ? 1 : 0;
    issue(s);
  }

  bool ok = true;
  int stage = 0;
  uint32_t phase = 0;
  Left mine = {};

  // ---- units
  while (taken < made) {
    __syncwarp();
    const Piece& now = queue[warp * kQueue + taken % kQueue];
    const int s0 = uniform(now.lo), s1 = uniform(now.hi), len = uniform(now.len);
    const bool starts = s0 == 0, ends = s1 == uniform(now.steps);
    const int row0 = uniform((now.u - now.head * p.row_blocks) * C::kRows);
    const int n_rows = min(C::kRows, p.rows - row0);
    const int row_at = uniform((now.b * p.c.Hkv + now.head) * p.rows + row0);  // in [B, H, Nq]
    ++taken;

    uint32_t q[PACK ? 2 : NR][NG][4];  // as the column operand (PACK: for each block, in its half of the columns)
    float2 cc[NR];          // powers of two that columns 2 t, 2 t + 1 lack: their rows' and the scale's
    int low = len;          // keys that all rows see
#pragma unroll
    for (int r = 0; r < NR; ++r) {
      // Query rows g (and g + 8), channels 32 i + 8 t .. + 7.
      uint4 raw[NG];
#pragma unroll
      for (int i = 0; i < NG; ++i) {
        raw[i] = make_uint4(0, 0, 0, 0);
        const int row = PACK ? g & 3 : r * 8 + g;
        if (row < n_rows) raw[i] = *reinterpret_cast<const uint4*>(p.q + (size_t)(row_at + row) * D + 32 * i + 8 * t);
      }
      float top = 0.f;
#pragma unroll
      for (int i = 0; i < NG; ++i) {
        const uint32_t w[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
#pragma unroll
        for (int k = 0; k < 4; ++k) top = fmax3(top, fabsf(bf16_lo(w[k])), fabsf(bf16_hi(w[k])));
      }
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
      // 2^15 over the power of two of the row's largest value (at most 2^126).
      const int e = (int)(__float_as_uint(top) >> 23);
      const int f = min(127 + 126, 127 + 15 + 127 - e);
      const float up = top > 0.f ? __uint_as_float((uint32_t)f << 23) : 1.f;
#pragma unroll
      for (int i = 0; i < NG; ++i) {
        const uint32_t w[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const uint32_t x = pack_f16(bf16_lo(w[k]) * up, bf16_hi(w[k]) * up);
          if constexpr (PACK) {
            q[0][i][k] = g < 4 ? x : 0u;
            q[1][i][k] = g < 4 ? 0u : x;
          } else {
            q[r][i][k] = x;
          }
        }
      }
      const float back = __uint_as_float((uint32_t)(top > 0.f ? 254 - f : 127) << 23) * p.scale_pow2;  // 1 / up: exact
      cc[r].x = __shfl_sync(0xffffffffu, back, 4 * col0);
      cc[r].y = __shfl_sync(0xffffffffu, back, 4 * col0 + 4);
    }
    // Keys that each row sees; padding rows see all.
    if (p.causal != FA_CAUSAL_NONE) {
      if (lane < C::kRows) {
        const int lim = lane < n_rows ? kv4_seen(p, len, (row0 + lane) % p.Nq) : len;
        lims[warp * C::kRows + lane] = lim;
        low = lim;
      }
      low = __reduce_min_sync(0xffffffffu, low);
    } else if (lane < C::kRows) {
      lims[warp * C::kRows + lane] = len;
    }
    __syncwarp();

    float o[NR][NG][2][4];
    float ref[NR][2], l[NR][2];
#pragma unroll
    for (int r = 0; r < NR; ++r) {
#pragma unroll
      for (int i = 0; i < NG; ++i)
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int k = 0; k < 4; ++k) o[r][i][h][k] = 0.f;
      ref[r][0] = ref[r][1] = -3.402823466e38f;
      l[r][0] = l[r][1] = 0.f;
    }

    // One step: MASK where some row does not see some of the keys.
    auto step = [&](auto mask, const uint8_t* const st, int key0, uint32_t there) {
      constexpr bool MASK = decltype(mask)::value;
      // Keys g and g + 8 of a block, this lane's columns.  PACK: tile 0 holds both
      // blocks, the query rows once in its columns 0-3 for block 0 and once in
      // 4-7 for block 1, so that a lane has scores of one block only.
      constexpr int NS = PACK ? 1 : C::kBlocks;
      float2 sc[NS][NR][2];  // keys g, g + 8: scores but for the factor `rest`, then base-2 ones + vl, then weights
      float vl[NS][2];       // log2(largest scale of the value)
      float top[NR][2];
      const float2 rest = make_float2(p.scale_rest, p.scale_rest);
#pragma unroll
      for (int r = 0; r < NR; ++r) top[r][0] = top[r][1] = -INFINITY;
      auto seen = [&](int s, int r, int x) {
        const int k = PACK ? my_blk : s;
        return key0 + k * kKv4Block + g + (x & 2) * 4 < lims[warp * C::kRows + r * 8 + col0 + (x & 1)] &&
               ((there >> (k / copy_blocks)) & 1) != 0;
      };
#pragma unroll
      for (int s = 0; s < NS; ++s) {
        const uint8_t* const blk = st + (PACK ? my_blk : s) * F::kBlockBytes;
        uint32_t wa[NG], wb[NG];
        load_scales<D>(blk, g, wa);
        load_scales<D>(blk, g + 8, wb);
        constexpr int NK = PACK ? C::kBlocks : 1;  // blocks of the tile
        uint32_t ka[NK][NG], kb[NK][NG];
#pragma unroll
        for (int k = 0; k < NK; ++k) {
          load_key<D>(st + (PACK ? k : s) * F::kBlockBytes, g, t, ka[k]);
          load_key<D>(st + (PACK ? k : s) * F::kBlockBytes, g + 8, t, kb[k]);
        }
#pragma unroll
        for (int r = 0; r < NR; ++r)
          for (int x = 0; x < 2; ++x) sc[s][r][x] = make_float2(0.f, 0.f);
#pragma unroll
        for (int i = 0; i < NG; ++i) {
          float c[NR][4];
#pragma unroll
          for (int r = 0; r < NR; ++r) c[r][0] = c[r][1] = c[r][2] = c[r][3] = 0.f;
#pragma unroll
          for (int k = 0; k < NK; ++k) {
            uint32_t ha[4], hb[4];
            kv4_decode8(ka[k][i], ha);
            kv4_decode8(kb[k][i], hb);
#pragma unroll
            for (int r = 0; r < NR; ++r) {
              const uint32_t* const b = q[PACK ? k : r][i];
              mma16816(c[r], ha[0], hb[0], ha[1], hb[1], b[0], b[1]);
              mma16816(c[r], ha[2], hb[2], ha[3], hb[3], b[2], b[3]);
            }
          }
          const float fa_ = scale_of(wa, i), fb_ = scale_of(wb, i);
#pragma unroll
          for (int r = 0; r < NR; ++r) {
            // The powers of two go to the key's scale first (exact): c times that
            // scale, or q k, may overflow where the score does not.
            const float2 fa2 = __fmul2_rn(make_float2(fa_, fa_), cc[r]), fb2 = __fmul2_rn(make_float2(fb_, fb_), cc[r]);
            sc[s][r][0] = __ffma2_rn(fa2, make_float2(c[r][0], c[r][1]), sc[s][r][0]);
            sc[s][r][1] = __ffma2_rn(fb2, make_float2(c[r][2], c[r][3]), sc[s][r][1]);
          }
        }
        const float va = vl[s][0] = lg2_approx(largest_scale<NG>(wa)), vb = vl[s][1] = lg2_approx(largest_scale<NG>(wb));
#pragma unroll
        for (int r = 0; r < NR; ++r) {
          float2 &x = sc[s][r][0], &y = sc[s][r][1];
          x = __ffma2_rn(x, rest, make_float2(va, va));
          y = __ffma2_rn(y, rest, make_float2(vb, vb));
          if constexpr (MASK) {
            x.x = seen(s, r, 0) ? x.x : -INFINITY;
            x.y = seen(s, r, 1) ? x.y : -INFINITY;
            y.x = seen(s, r, 2) ? y.x : -INFINITY;
            y.y = seen(s, r, 3) ? y.y : -INFINITY;
          }
          top[r][0] = fmax3(top[r][0], x.x, y.x);
          top[r][1] = fmax3(top[r][1], x.y, y.y);
        }
      }

      // Move the references of columns that have outgrown them.  The same
      // difference is the weight's exponent below, whatever it was rounded from:
      // from 2^25 on fp32 holds multiples of 4 only, and ref + 14 may be ref + 16.
      bool grow = false;
#pragma unroll
      for (int r = 0; r < NR; ++r) grow |= top[r][0] - ref[r][0] > 14.f || top[r][1] - ref[r][1] > 14.f;
      if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
        for (int r = 0; r < NR; ++r) {
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            float x = top[r][c];
            x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
            x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
            x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
            const float next = x - ref[r][c] > 14.f ? x - 4.f : ref[r][c];
            const float f = ex2_approx(ref[r][c] - next);
            ref[r][c] = next;
            l[r][c] *= f;
#pragma unroll
            for (int i = 0; i < NG; ++i) {
              o[r][i][0][c] *= f;
              o[r][i][0][c + 2] *= f;
              o[r][i][1][c] *= f;
              o[r][i][1][c + 2] *= f;
            }
          }
        }
      }

      // Weights, and O^T += V^T P^T.  PACK: columns 4-7 of O gather what block 1
      // gives the same rows, and are added at the end.
#pragma unroll
      for (int s = 0; s < NS; ++s) {
        const uint8_t* const blk = st + (PACK ? my_blk : s) * F::kBlockBytes;
        uint32_t wa[NG], wb[NG];
        load_scales<D>(blk, g, wa);
        load_scales<D>(blk, g + 8, wb);
#pragma unroll
        for (int r = 0; r < NR; ++r)
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            float2 y = __fadd2_rn(sc[s][r][x], make_float2(-ref[r][0], -ref[r][1]));
            y = __fadd2_rn(y, make_float2(-vl[s][x], -vl[s][x]));
            y = make_float2(ex2_approx(y.x), ex2_approx(y.y));  // of a key that the row does not see: 0
            sc[s][r][x] = y;
            const float2 sum = __fadd2_rn(make_float2(l[r][0], l[r][1]), y);
            l[r][0] = sum.x;
            l[r][1] = sum.y;
          }
        constexpr int NW = (NG + 1) / 2, NK = PACK ? C::kBlocks : 1;
        uint32_t v[NK][4][NW];  // tokens 2 t, 2 t + 1, 2 t + 8, 2 t + 9
#pragma unroll
        for (int k = 0; k < NK; ++k)
#pragma unroll
          for (int x = 0; x < 4; ++x) load_value<D>(st + (PACK ? k : s) * F::kBlockBytes, 4 * x + t, g, v[k][x]);
#pragma unroll
        for (int j = 0; j < NW; ++j) {
          // Weights times the scales of this word's groups, as the column operand.
          uint32_t b0[2][NR], b1[2][NR];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int i = 2 * j + h;
            if (i >= NG) continue;
            const float fa_ = scale_of(wa, NG + i), fb_ = scale_of(wb, NG + i);
#pragma unroll
            for (int r = 0; r < NR; ++r) {
              float2 x = __fmul2_rn(sc[s][r][0], make_float2(fa_, fa_)), y = __fmul2_rn(sc[s][r][1], make_float2(fb_, fb_));
              if constexpr (MASK) {  // whatever the scale is
                x.x = seen(s, r, 0) ? x.x : 0.f;
                x.y = seen(s, r, 1) ? x.y : 0.f;
                y.x = seen(s, r, 2) ? y.x : 0.f;
                y.y = seen(s, r, 3) ? y.y : 0.f;
              }
              b0[h][r] = transpose8(pack_f16(x.x, x.y));
              b1[h][r] = transpose8(pack_f16(y.x, y.y));
            }
          }
#pragma unroll
          for (int k = 0; k < NK; ++k) {
            // Bytes of two tokens' codes for one channel: even channels, odd channels.
            const uint32_t w0 = v[k][0][j], w1 = v[k][1][j], w2 = v[k][2][j], w3 = v[k][3][j];
            const uint32_t lo01 = (w0 & 0x0f0f0f0fu) | ((w1 << 4) & 0xf0f0f0f0u);
            const uint32_t hi01 = ((w0 >> 4) & 0x0f0f0f0fu) | (w1 & 0xf0f0f0f0u);
            const uint32_t lo23 = (w2 & 0x0f0f0f0fu) | ((w3 << 4) & 0xf0f0f0f0u);
            const uint32_t hi23 = ((w2 >> 4) & 0x0f0f0f0fu) | (w3 & 0xf0f0f0f0u);
            uint32_t a0[4], a1[4], a2[4], a3[4];
            kv4_decode8(lo01, a0);
            kv4_decode8(hi01, a1);
            kv4_decode8(lo23, a2);
            kv4_decode8(hi23, a3);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const int i = 2 * j + h;
              if (i >= NG) continue;
              const int y = 2 * h;
#pragma unroll
              for (int r = 0; r < NR; ++r) {
                const bool its = !PACK || g / 4 == k;  // column g is of this block
                const uint32_t c0 = its ? b0[h][r] : 0u, c1 = its ? b1[h][r] : 0u;
                mma16816(o[r][i][0], a0[y], a1[y], a2[y], a3[y], c0, c1);
                mma16816(o[r][i][1], a0[y + 1], a1[y + 1], a2[y + 1], a3[y + 1], c0, c1);
              }
            }
          }
        }
      }
    };
#pragma unroll 1
    for (int s = s0; s < s1; ++s) {
      if (!ok) break;
      ok = __all_sync(0xffffffffu, mbar_wait(&bar[stage], phase, ctl, kWaitKvFull));
      if (!ok) break;
      const uint8_t* const st = ring + stage * C::kStageBytes;
      const uint32_t there = (have >> (C::kBlocks * --in_flight)) & ((1u << C::kBlocks) - 1);
      const int key0 = s * C::kKeys;
      if (key0 + C::kKeys <= low && there == have_all)
        step(std::false_type{}, st, key0, there);
      else
        step(std::true_type{}, st, key0, there);
      __syncwarp();  // every lane has read the stage
      in_flight += ahead.lo < ahead.hi ? 1 : 0;
      issue(stage);
      if (++stage == C::kStages) {
        stage = 0;
        phase ^= 1;
      }
    }

    // ---- results
#pragma unroll
    for (int r = 0; r < NR; ++r)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        l[r][c] += __shfl_xor_sync(0xffffffffu, l[r][c], 4);
        l[r][c] += __shfl_xor_sync(0xffffffffu, l[r][c], 8);
        l[r][c] += __shfl_xor_sync(0xffffffffu, l[r][c], 16);
      }
    if constexpr (PACK) {  // columns 4-7 to 0-3
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const float m = fmaxf(ref[0][c], __shfl_xor_sync(0xffffffffu, ref[0][c], 2));
        const float f = ex2_approx(ref[0][c] - m);
        ref[0][c] = m;
        l[0][c] *= f;
        l[0][c] += __shfl_xor_sync(0xffffffffu, l[0][c], 2);
#pragma unroll
        for (int i = 0; i < NG; ++i)
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int k = c; k < 4; k += 2) {
              o[0][i][h][k] *= f;
              o[0][i][h][k] += __shfl_xor_sync(0xffffffffu, o[0][i][h][k], 2);
            }
      }
    }
    if (starts && ends) {
#pragma unroll
      for (int r = 0; r < NR; ++r)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const int col = r * 8 + col0 + c;
          if (col >= n_rows || (PACK && t >= 2)) continue;
          const float inv = l[r][c] == 0.f ? 0.f : 1.0f / l[r][c];
          __nv_bfloat16* dst = p.o + (size_t)(row_at + col) * D + 4 * g;
#pragma unroll
          for (int i = 0; i < NG; ++i)
            *reinterpret_cast<uint2*>(dst + 32 * i) =
                make_uint2(pack_bf16(o[r][i][0][c] * inv, o[r][i][0][c + 2] * inv),
                           pack_bf16(o[r][i][1][c] * inv, o[r][i][1][c + 2] * inv));
          if (g == 0)
            p.lse[row_at + col] = l[r][c] == 0.f ? -INFINITY : (ref[r][c] + lg2_approx(l[r][c])) * 0.69314718055994530942f;
        }
    } else {
      // A part of a unit: [row][channel / 4], the quads of a row exchanged so
      // that a store meets no bank twice.
      float4* const dst = reinterpret_cast<float4*>(starts ? ring : smem + W * C::kRing + warp * C::kSums);
#pragma unroll
      for (int r = 0; r < NR; ++r)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const int col = r * 8 + col0 + c;
          if (PACK && t >= 2) continue;
#pragma unroll
          for (int i = 0; i < NG; ++i)
            dst[col * (D / 4) + ((8 * i + g) ^ col0)] =
                make_float4(o[r][i][0][c], o[r][i][0][c + 2], o[r][i][1][c], o[r][i][1][c + 2]);
          if (g == 0) stats[starts ? 1 : 0][warp * C::kRows + col] = make_float2(ref[r][c], l[r][c]);
        }
      const Part part{row_at, n_rows, uniform(now.place), uniform(now.steps)};
      if (starts) {
        mine.kinds |= 1;
        mine.tail = part;
      } else {
        mine.kinds |= ends ? 6 : 2;
        mine.head = part;
      }
    }
  }
  if (lane == 0) left[warp] = mine;
  __syncthreads();

  // ---- join what the warps have left.  A chain begins with a warp's tail, or
  // goes on from the CTA before, and takes the heads of the warps behind it
  // until the unit's end.  Lane c of every warp works out chain c: that from
  // warp c - 1's tail, or for lane 0 the one from the CTA before.
  const int kinds = lane < W ? left[lane].kinds : 0;
  const uint32_t tails = __ballot_sync(0xffffffffu, kinds & 1), heads = __ballot_sync(0xffffffffu, kinds & 2),
                 stops = __ballot_sync(0xffffffffu, kinds & 4);
  const int first_left = __ffs(heads | tails) - 1;
  bool is = lane > 0 ? lane <= W && ((tails >> (lane - 1)) & 1) : first_left >= 0 && ((heads >> first_left) & 1);
  const int from = lane;                                     // warps [from, past): their heads belong to it
  const uint32_t ahead_stops = from < W ? stops >> from : 0u;
  const bool stopped = ahead_stops != 0;
  const int past = stopped ? from + __ffs(ahead_stops) : W;
  Part whose{};
  if (is) whose = lane > 0 ? left[lane - 1].tail : left[first_left].head;
  const uint32_t chains = __ballot_sync(0xffffffffu, is);
  // The chains that other CTAs have parts of: from the one before, into the next.
  const uint32_t open = __ballot_sync(0xffffffffu, is && (lane == 0 || !stopped));

  // A warp takes a row of a chain at a time.
  for (int j = warp; j < __popc(chains) * C::kRows; j += W) {
    const int chain = nth_bit(chains, j / C::kRows), col = j % C::kRows;
    const int c_rows = __shfl_sync(0xffffffffu, whose.rows, chain);
    if (col >= c_rows) continue;
    const int c_row = __shfl_sync(0xffffffffu, whose.row, chain);
    const int c_past = __shfl_sync(0xffffffffu, past, chain);
    const uint32_t parts = heads & ((1u << c_past) - 1) & ~((1u << chain) - 1);
    // Lane w has warp w's reference, sum and factor; lane 31 the tail's.
    float2 ml = make_float2(-3.402823466e38f, 0.f);
    if ((parts >> lane) & 1) ml = stats[0][lane * C::kRows + col];
    if (lane == 31 && chain > 0) ml = stats[1][(chain - 1) * C::kRows + col];
    float m = ml.x;
#pragma unroll
    for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    const float f = ex2_approx(ml.x - m);
    float sum = ml.y * f;
#pragma unroll
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    constexpr int kMany = (D / 4 + 31) / 32;
    float4 x[kMany];
    auto add = [&](const uint8_t* part, float by) {
      const float4* const src = reinterpret_cast<const float4*>(part) + col * (D / 4);
#pragma unroll
      for (int i = 0; i < kMany; ++i) {
        const float4 y = src[min(32 * i + lane, D / 4 - 1) ^ (col & 6)];
        x[i].x = fmaf(y.x, by, x[i].x);
        x[i].y = fmaf(y.y, by, x[i].y);
        x[i].z = fmaf(y.z, by, x[i].z);
        x[i].w = fmaf(y.w, by, x[i].w);
      }
    };
#pragma unroll
    for (int i = 0; i < kMany; ++i) x[i] = make_float4(0.f, 0.f, 0.f, 0.f);
    if (chain > 0) add(smem + (chain - 1) * C::kRing, __shfl_sync(0xffffffffu, f, 31));
    for (uint32_t todo = parts; todo != 0; todo &= todo - 1) {
      const int w = __ffs(todo) - 1;
      add(smem + W * C::kRing + w * C::kSums, __shfl_sync(0xffffffffu, f, w));
    }
    if (!((open >> chain) & 1)) {
      const float inv = sum == 0.f ? 0.f : 1.0f / sum;
#pragma unroll
      for (int i = 0; i < kMany; ++i)
        if (32 * i + lane < D / 4)
          *reinterpret_cast<uint2*>(p.o + (size_t)(c_row + col) * D + 4 * (32 * i + lane)) =
              make_uint2(pack_bf16(x[i].x * inv, x[i].y * inv), pack_bf16(x[i].z * inv, x[i].w * inv));
      if (lane == 0) p.lse[c_row + col] = sum == 0.f ? -INFINITY : (m + lg2_approx(sum)) * 0.69314718055994530942f;
    } else {
      const size_t slot = (size_t)(2 * blockIdx.x + (chain > 0 ? 1 : 0)) * C::kRows + col;
#pragma unroll
      for (int i = 0; i < kMany; ++i)
        if (32 * i + lane < D / 4) reinterpret_cast<float4*>(p.part_o + slot * D)[32 * i + lane] = x[i];
      if (lane == 0) p.part_ml[slot] = make_float2(m, sum);
      if (chain > 0 && col == 0) {
        const int place = __shfl_sync(0xffffffffu, whose.place, chain), steps = __shfl_sync(0xffffffffu, whose.steps, chain);
        if (lane == 0) p.cuts[blockIdx.x] = Kv4Cut{c_row, c_rows, cta_of(place + kUnitCost + steps - 1), 0};
      }
    }
  }

  // After a wait that gave up, copies may still be on their way into this CTA's
  // shared memory: wait for them, bounded, before it is given back.
  if (!ok) {
    const unsigned long long limit = max(p.timeout_ns, 100000000ull);  // however short the waits' limit is
    const uint64_t t0 = globaltimer_ns();
    for (; in_flight > 0; --in_flight) {
      while (!mbar_try_wait(smem_u32(&bar[stage]), phase) && globaltimer_ns() - t0 < limit) {
      }
      if (++stage == C::kStages) {
        stage = 0;
        phase ^= 1;
      }
    }
  }
}

// Merge of the parts of the units that CTA borders cut: a CTA per main CTA, a
// warp per row.  O = sum_k 2^(ref_k - m) O_k / sum_k 2^(ref_k - m) l_k, the parts in
// the order of the CTAs.  Bound by its chain of loads (which CTAs, their
// references and sums): about 2 us with its launch.  Merging in the main kernel
// instead, by the CTA that brings a unit's last part, cost more (two barriers,
// fences and an atomic in every CTA: 8 sequences of 8192 tokens 24.9 us in place of
// 22.6).
template <int D, int kRows>
__global__ void __launch_bounds__(256) kv4_merge_kernel(const Kv4FwdParams p) {
  constexpr int kMany = (D / 4 + 31) / 32, kBatch = 8 / kMany;
  pdl_wait();
  const Kv4Cut cut = p.cuts[blockIdx.x];
  if (cut.row < 0) return;
  const int lane = threadIdx.x % 32;
  const int parts = cut.last - (int)blockIdx.x + 1;
  for (int row = threadIdx.x / 32; row < cut.rows; row += 8) {
    // Part k: the tail of this CTA, then the heads of those behind it.
    auto at = [&](int k) { return (size_t)(2 * (blockIdx.x + k) + (k == 0 ? 1 : 0)) * kRows + row; };
    float4 acc[kMany], next[kBatch][kMany];
    auto fetch = [&](int k0) {
#pragma unroll
      for (int k = 0; k < kBatch; ++k)
#pragma unroll
        for (int i = 0; i < kMany; ++i)
          if (k0 + k < parts && 32 * i + lane < D / 4)
            next[k][i] = reinterpret_cast<const float4*>(p.part_o + at(k0 + k) * D)[32 * i + lane];
    };
    fetch(0);
    float m = -3.402823466e38f, l = 0.f;
#pragma unroll
    for (int i = 0; i < kMany; ++i) acc[i] = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int k0 = 0; k0 < parts; k0 += 32) {  // references of 32 parts at a time
      const float2 ml = k0 + lane < parts ? p.part_ml[at(k0 + lane)] : make_float2(-3.402823466e38f, 0.f);
      float top = fmaxf(m, ml.x);
#pragma unroll
      for (int x = 16; x; x >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
      const float back = ex2_approx(m - top), f = ex2_approx(ml.x - top);
      m = top;
      float sum = ml.y * f;
#pragma unroll
      for (int x = 16; x; x >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, x);
      l = fmaf(l, back, sum);
#pragma unroll
      for (int i = 0; i < kMany; ++i) {
        acc[i].x *= back;
        acc[i].y *= back;
        acc[i].z *= back;
        acc[i].w *= back;
      }
      for (int k = k0; k < min(k0 + 32, parts); k += kBatch) {
        float4 now[kBatch][kMany];
#pragma unroll
        for (int x = 0; x < kBatch; ++x)
#pragma unroll
          for (int i = 0; i < kMany; ++i) now[x][i] = next[x][i];
        fetch(k + kBatch);
#pragma unroll
        for (int x = 0; x < kBatch; ++x) {
          const float by = __shfl_sync(0xffffffffu, f, k - k0 + x);
          if (k + x < parts) {
#pragma unroll
            for (int i = 0; i < kMany; ++i) {
              acc[i].x = fmaf(now[x][i].x, by, acc[i].x);
              acc[i].y = fmaf(now[x][i].y, by, acc[i].y);
              acc[i].z = fmaf(now[x][i].z, by, acc[i].z);
              acc[i].w = fmaf(now[x][i].w, by, acc[i].w);
            }
          }
        }
      }
    }
    const float inv = l == 0.f ? 0.f : 1.0f / l;
#pragma unroll
    for (int i = 0; i < kMany; ++i)
      if (32 * i + lane < D / 4)
        *reinterpret_cast<uint2*>(p.o + ((size_t)cut.row + row) * D + 4 * (32 * i + lane)) =
            make_uint2(pack_bf16(acc[i].x * inv, acc[i].y * inv), pack_bf16(acc[i].z * inv, acc[i].w * inv));
    if (lane == 0) p.lse[cut.row + row] = l == 0.f ? -INFINITY : (m + lg2_approx(l)) * 0.69314718055994530942f;
  }
}

namespace {

template <int D, int NR, bool PACK>
cudaError_t launch_fwd_t(const Kv4FwdParams& p, int grid, cudaStream_t stream) {
  using C = Cfg<D, NR, PACK>;
  // The kernel's shared memory is allowed once on each device.
  static std::atomic<unsigned long long> allowed{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const unsigned long long bit = 1ull << (dev & 63);
  if (!(allowed.load(std::memory_order_relaxed) & bit)) {
    e = cudaFuncSetAttribute(kv4_fwd_kernel<D, NR, PACK>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
    if (e != cudaSuccess) return e;
    allowed.fetch_or(bit, std::memory_order_relaxed);
  }
  return launch_pdl(kv4_fwd_kernel<D, NR, PACK>, dim3(grid), dim3(C::kThreads), C::kSmem, stream, p);
}

template <int D>
cudaError_t launch_fwd_d(int unit_rows, const Kv4FwdParams& p, int grid, cudaStream_t stream) {
  if (unit_rows == kKv4Rows / 2) return launch_fwd_t<D, 1, true>(p, grid, stream);
  if (unit_rows == kKv4Rows) return launch_fwd_t<D, 1, false>(p, grid, stream);
  if constexpr (D != 256) {
    if (unit_rows == 2 * kKv4Rows) return launch_fwd_t<D, 2, false>(p, grid, stream);
  }
  if constexpr (D <= 96) {
    if (unit_rows == 3 * kKv4Rows) return launch_fwd_t<D, 3, false>(p, grid, stream);
  }
  return cudaErrorInvalidValue;
}

template <int D>
cudaError_t launch_merge_d(int unit_rows, const Kv4FwdParams& p, int grid, cudaStream_t stream) {
  const dim3 g(grid), b(256);
  if (unit_rows == kKv4Rows / 2) return launch_pdl(kv4_merge_kernel<D, kKv4Rows / 2>, g, b, 0, stream, p);
  if (unit_rows == kKv4Rows) return launch_pdl(kv4_merge_kernel<D, kKv4Rows>, g, b, 0, stream, p);
  if constexpr (D != 256) {
    if (unit_rows == 2 * kKv4Rows) return launch_pdl(kv4_merge_kernel<D, 2 * kKv4Rows>, g, b, 0, stream, p);
  }
  if constexpr (D <= 96) {
    if (unit_rows == 3 * kKv4Rows) return launch_pdl(kv4_merge_kernel<D, 3 * kKv4Rows>, g, b, 0, stream, p);
  }
  return cudaErrorInvalidValue;
}

}  // namespace

// Query rows of a unit for head dim d and `rows` query rows a key/value head.
// Up to four rows leave half of a tile's columns free for a second block of
// keys, which halves what a step spends on softmax (PACK).  Above eight, two row
// tiles a unit read and decode each key once for 16 rows, but leave room for
// fewer warps: where there are few steps to an SM (`sm_steps`, with one tile a
// unit), one tile is sooner done (d = 128, 16 rows, 8 heads: 4 sequences of 2000
// tokens, 26 steps an SM, 12.2 us and 13.7 with two; 8 of 4000, 105 steps, 22.0
// and 22.6; 16 of 4000, 210 steps, 35.4 and 32.2; d = 64 and 96 24.4 and 23.5, 32.8
// and 30.1).  The steps are those that the table has room for: a wider one takes
// the two tiles however short the sequences are.  Not at
// d = 256, whose sums take 64 registers a tile.
// At d = 64 and 96, 17 to 24 rows are one unit of three tiles (24 rows, 16
// sequences of 8000 tokens: d = 96 57.2 us, with three units of one tile 76.9 and
// two of two tiles 81.4; d = 64 45.6, 54.0 and 55.9), at d = 64 from more steps on
// (9 of 4000, 178 steps an SM: d = 96 26.8 us and 27.9 with one tile a unit, d = 64
// 22.7 and 21.5; 14 of 4000, 276 steps: d = 64 28.1 and 28.6).  Three tiles for more
// rows there gain nothing (48 rows 77.7 us, 77.9 with two), nor did four for 32 rows
// (an earlier form: 55.8, 54.3 with two).
int kv4_fwd_unit_rows(int d, int rows, long long sm_steps) {
  if (rows <= kKv4Rows / 2) return kKv4Rows / 2;
  if (rows <= kKv4Rows || d == 256) return kKv4Rows;
  const bool three = rows > 2 * kKv4Rows && rows <= 3 * kKv4Rows && d <= 96;
  if (sm_steps < (three && d == 64 ? 280 : 160)) return kKv4Rows;
  return three ? 3 * kKv4Rows : 2 * kKv4Rows;
}

template <int D>
static int warps_d(int unit_rows) {
  if (unit_rows == kKv4Rows / 2) return Cfg<D, 1, true>::kWarps;
  if constexpr (D != 256) {
    if (unit_rows == 2 * kKv4Rows) return Cfg<D, 2, false>::kWarps;
  }
  if constexpr (D <= 96) {
    if (unit_rows == 3 * kKv4Rows) return Cfg<D, 3, false>::kWarps;
  }
  return Cfg<D, 1, false>::kWarps;
}

// Warps of a CTA.
int kv4_fwd_warps(int d, int unit_rows) {
  switch (d) {
    case 64: return warps_d<64>(unit_rows);
    case 96: return warps_d<96>(unit_rows);
    case 128: return warps_d<128>(unit_rows);
    default: return warps_d<256>(unit_rows);
  }
}

int kv4_fwd_step_keys() { return Cfg<64, 1, false>::kKeys; }
int kv4_fwd_unit_cost() { return kUnitCost; }

cudaError_t launch_kv4_fwd(int d, int unit_rows, const Kv4FwdParams& p, int grid, cudaStream_t stream) {
  switch (d) {
    case 64: return launch_fwd_d<64>(unit_rows, p, grid, stream);
    case 96: return launch_fwd_d<96>(unit_rows, p, grid, stream);
    case 128: return launch_fwd_d<128>(unit_rows, p, grid, stream);
    case 256: return launch_fwd_d<256>(unit_rows, p, grid, stream);
    default: return cudaErrorInvalidValue;
  }
}

cudaError_t launch_kv4_merge(int d, int unit_rows, const Kv4FwdParams& p, int grid, cudaStream_t stream) {
  switch (d) {
    case 64: return launch_merge_d<64>(unit_rows, p, grid, stream);
    case 96: return launch_merge_d<96>(unit_rows, p, grid, stream);
    case 128: return launch_merge_d<128>(unit_rows, p, grid, stream);
    case 256: return launch_merge_d<256>(unit_rows, p, grid, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace fa
