// Forward pass over packed sequences on sm_103a (include/fa.h: fa_packed_fwd,
// fa_prefix_fwd): the products, online softmax and roles of fa_fwd.cu over the
// list of units of packed.h.  What differs:
//
//  * A CTA walks stretches of the two lists of units that the planning kernel gave
//    it, and may start and end within a unit.  It takes the whole blocks first,
//    as fa_fwd.cu does; then each element-wise warpgroup takes small blocks on its
//    own, with its own loading and issuing warp, its Q buffer and half of the ring.
//  * A unit's key tiles are those of the shared prefix (all visible), then the
//    sequence's own (causal or not, up to its length).
//  * Rows of a tile are (token, query head) pairs, so that the query heads of a
//    key/value head share its K and V.
//  * A warp whose 32 rows lie past the block's skips the element-wise work (its
//    rows of P stay what they were; they reach only rows of O that are not kept).
//
// Both warpgroups, registers, tensor memory columns and the rounding of P are as
// described there.
#include <cuda_runtime.h>

#include <type_traits>

#include "packed.h"
#include "packed_seq.cuh"
#include "sm103_primitives.cuh"

namespace fa {

using namespace dev;

namespace pk {

// A stretch's part of one unit.
struct Piece {
  PackedEntry e;
  int hk, g0;    // key/value head, first query head of the group's
  int lo, hi;    // tiles of this part
  int n0;        // steps of tile 0 of a whole block (tile 1, and a small block, take all)
  bool cut;      // not the whole unit
};

// Steps of a whole block's first tile of rows: the second holds the block's last
// token, the first may see less.
__device__ __forceinline__ int first_steps(const PackedFwd& p, const Piece& w) {
  const int own = p.causal ? min(w.e.k_len, max(0, w.e.pos + p.tile_tokens)) : w.e.k_len;
  const int seen = w.e.kind ? w.e.prefix : w.e.prefix + (own + kTileN - 1) / kTileN;
  return max(0, min(w.hi, seen) - w.lo);
}

// A call without a plan: the sequences, and the first unit of each, by list.
struct DirectSeqs {
  Seq seq[kDirectSeqs];
  int base[2][kDirectSeqs + 1];
  // By the threads of one warp.
  __device__ __forceinline__ void fill(const PackedFwd& p) {
    const int lane = threadIdx.x & 31;
    Seq x{0, 0, 0, 0};
    int first_q = lane < p.s.B ? start_of(p.s.cu_q, lane, p.s.Tq) : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int a = __shfl_up_sync(0xffffffffu, first_q, o);
      if (lane >= o) first_q = max(first_q, a);
    }
    if (lane < p.s.B) x = load_seq(p.s, lane, first_q);
    seq[lane] = x;
    int2 n = blocks_of(x, p.tile_tokens);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int a = __shfl_up_sync(0xffffffffu, n.x, o), b = __shfl_up_sync(0xffffffffu, n.y, o);
      if (lane >= o) n.x += a, n.y += b;
    }
    base[kWhole][lane + 1] = n.x;
    base[kSmall][lane + 1] = n.y;
    if (lane == 0) base[kWhole][0] = base[kSmall][0] = 0;
  }
};
static_assert(kDirectSeqs == 32, "a lane each");

// The units of a CTA (of its warpgroup t, of the small ones) without a plan: every
// grid-th; the small ones from the CTAs on that have the fewest whole ones.  Where
// there are no more small ones than CTAs (dual), the warpgroups of a CTA halve the
// keys of one.
struct DirectWalk {
  const PackedFwd& p;
  const DirectSeqs* q;
  int list, t, u;
  // (Read again at each unit: the issuing warps have few registers.)
  __device__ __forceinline__ int units() const { return q->base[list][kDirectSeqs] * p.head_groups; }
  __device__ __forceinline__ bool dual() const { return list == kSmall && p.halves && units() <= (int)gridDim.x; }
  __device__ __forceinline__ DirectWalk(const PackedFwd& params, const DirectSeqs* seqs, int which, int wg)
      : p(params), q(seqs), list(which), t(wg) {
    const int grid = gridDim.x, c = blockIdx.x;
    u = list == kSmall ? (dual() ? 0 : t * grid) + (grid - 1 - c) : c;
  }
  __device__ __forceinline__ bool get(Piece& w) {
    if (u >= units()) return false;
    const int entries = q->base[list][kDirectSeqs];
    const int hg = u / entries, i = u - hg * entries;
    const int b = seq_of(q->base[list], kDirectSeqs, i);
    const int block = 2 * p.tile_tokens;
    const int t0 = (list == kSmall ? q->base[kWhole][b + 1] - q->base[kWhole][b] : i - q->base[kWhole][b]) * block;
    w.e = block_at(q->seq[b], t0, block, p.prefix_tiles, p.s.causal);
    w.hk = hg / p.chunks;
    w.g0 = (hg - w.hk * p.chunks) * p.group_heads;
    const bool dual = this->dual();
    const int half = dual ? (w.e.tiles + 1) / 2 : w.e.tiles;
    w.lo = t > 0 && dual ? half : 0;
    w.hi = t > 0 && dual ? w.e.tiles : half;
    w.cut = false;
    w.n0 = first_steps(p, w);
    u += list == kSmall ? 2 * gridDim.x : gridDim.x;
    return true;
  }
};

template <int D>
struct Cfg {
  static_assert(D == 64 || D == 96 || D == 128, "head dim");
  static constexpr int kChunks = (D + 63) / 64;
  static constexpr int kChunkBytes = kTileM * 128;
  static constexpr int kTileBytes = kChunks * kChunkBytes;
  static constexpr int kStages = (D == 64) ? 8 : 4;
  static constexpr int kOCols = kChunks * 64;
  static constexpr int kThreads = 384;
  __host__ __device__ static constexpr uint32_t col_s(int t) { return 128u * t; }
  __host__ __device__ static constexpr uint32_t col_o(int t) { return 256u + (uint32_t)kOCols * t; }
  // The weights P take the place of S in tensor memory, or columns of their own where
  // there is room (d = 64): then S of the next keys is worked out while the
  // element-wise warps still have this one (64 sequences' steps over 4096 keys 173 ->
  // 165 us, 4 prompts of 4096 without a mask 533 -> 519).
  static constexpr bool kOwnP = D == 64;
  __host__ __device__ static constexpr uint32_t col_p(int t) { return kOwnP ? 256u + 2 * kOCols + 64u * t : col_s(t); }
  static constexpr uint32_t kTmemCols = 512;
  static constexpr int kOffQ = 0;
  static constexpr int kOffKV = 2 * kTileBytes;
  // Room of 4 KB for each element-wise warp, from which its rows of O are stored
  // (32 rows of 128 bytes, swizzled).
  static constexpr int kOffOut = kOffKV + kStages * kTileBytes;
  static constexpr int kOffBar = kOffOut + 8 * 4096;
  static constexpr int kPhaseBars = 2 + 2 + 2 * kStages + 2 + 2 + 2 + 2;
  static constexpr int kNumBars = 2 * kPhaseBars + 1 + 2 + 1;
  static constexpr int kOffSeqs = (kOffBar + kNumBars * 8 + 16 + 15) / 16 * 16;
  static constexpr int kSmemBytes = kOffSeqs + (int)sizeof(DirectSeqs);
  static_assert(kSmemBytes <= 232448, "shared memory");
  static constexpr float kRescaleThreshold = 24.0f;  // log2 units, as in fa_fwd.cu
  static constexpr int kRegsAtLaunch = 168;
  static constexpr int kRegsCtl = 72;
  static constexpr int kRegsMath = 216;
  static_assert(128 * kRegsCtl + 256 * kRegsMath <= kThreads * kRegsAtLaunch, "register split exceeds the launch");
  static_assert(kRegsCtl % 8 == 0 && kRegsMath % 8 == 0, "setmaxnreg counts are multiples of 8");
};

// The units of a stretch of a list, in order.  AHEAD: the next entry is fetched a
// unit ahead (not by the issuing warps, whose registers are few: they come to a
// unit while the element-wise warps still end the one before).
template <bool AHEAD>
struct PlannedWalk {
  const PackedFwd& p;
  PackedStart s0, s1;
  const PackedEntry* list;
  int entries;
  int u, u_last, at, hk, chunk;
  PackedEntry next;

  __device__ __forceinline__ static PackedEntry fetch(const PackedEntry* e) {
    const int4* w = reinterpret_cast<const int4*>(e);
    const int4 a = w[0], b = w[1];
    return PackedEntry{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
  }
  __device__ __forceinline__ PlannedWalk(const PackedFwd& params, const DirectSeqs*, int which, int t) : p(params) {
    const int stretch = which == kSmall ? 2 * (int)blockIdx.x + t : (int)blockIdx.x;
    const PackedStart* s = p.starts[which] + stretch;
    s0 = s[0];
    s1 = s[1];
    list = p.entries[which];
    entries = p.header->entries[which];
    u = s0.unit;
    u_last = s1.tile > 0 ? s1.unit : s1.unit - 1;
    if (s0.unit == s1.unit && s0.tile == s1.tile) u_last = u - 1;
    hk = chunk = at = 0;
    if (u <= u_last) {
      const int hg = u / entries;
      at = u - hg * entries;
      hk = hg / p.chunks;
      chunk = hg - hk * p.chunks;
      if (AHEAD) next = fetch(list + at);
    }
  }
  __device__ __forceinline__ bool get(Piece& w) {
    if (u > u_last) return false;
    w.e = AHEAD ? next : fetch(list + at);
    w.hk = hk;
    w.g0 = chunk * p.group_heads;
    w.lo = u == s0.unit ? s0.tile : 0;
    w.hi = u == s1.unit ? s1.tile : w.e.tiles;
    w.cut = w.lo > 0 || w.hi < w.e.tiles;
    ++u;
    if (++at == entries) {
      at = 0;
      if (++chunk == p.chunks) {
        chunk = 0;
        ++hk;
      }
    }
    if (AHEAD && u <= u_last) next = fetch(list + at);
    w.n0 = first_steps(p, w);
    return true;
  }
};

template <bool AHEAD, bool DIRECT>
using Walk = std::conditional_t<DIRECT, DirectWalk, PlannedWalk<AHEAD>>;

// Barriers of one way of taking units: of whole blocks (list 0), or of small ones.
template <int D, int LIST>
struct Bars {
  static constexpr int kStages = Cfg<D>::kStages;
  uint64_t* b;
  __device__ __forceinline__ explicit Bars(uint64_t* all) : b(all + LIST * Cfg<D>::kPhaseBars) {}
  __device__ __forceinline__ uint64_t* q_full(int t) const { return b + t; }
  __device__ __forceinline__ uint64_t* q_empty(int t) const { return b + 2 + t; }
  __device__ __forceinline__ uint64_t* kv_full(int s) const { return b + 4 + s; }
  __device__ __forceinline__ uint64_t* kv_empty(int s) const { return b + 4 + kStages + s; }
  __device__ __forceinline__ uint64_t* s_full(int t) const { return b + 4 + 2 * kStages + t; }
  __device__ __forceinline__ uint64_t* p_full(int t) const { return b + 6 + 2 * kStages + t; }
  __device__ __forceinline__ uint64_t* s_read(int t) const { return b + 8 + 2 * kStages + t; }
  __device__ __forceinline__ uint64_t* o_full(int t) const { return b + 10 + 2 * kStages + t; }
};

// Key tile x of a unit, K or V, into a ring slot (ONCE: own keys under a policy).
template <int D, bool ONCE = false>
__device__ __forceinline__ void load_keys(uint8_t* dst, uint64_t* bar, const Piece& w, int x, const CUtensorMap* own,
                                          const CUtensorMap* prefix, uint64_t policy = 0) {
  using C = Cfg<D>;
  mbar_arrive_expect_tx(bar, C::kTileBytes);
  if (x < w.e.prefix) {
#pragma unroll
    for (int c = 0; c < C::kChunks; ++c) tma_load_3d(dst + c * C::kChunkBytes, prefix, bar, c * 64, x * kTileN, w.hk);
  } else {
    const int row = (x - w.e.prefix) * kTileN;
    const int n = min(kTileN, w.e.k_len - row);  // keys of the sequence in the tile
#pragma unroll
    for (int c = 0; c < C::kChunks; ++c) {
      if constexpr (ONCE)
        tma_load_4d_policy(dst + c * C::kChunkBytes, own, bar, c * 64, n - kTileN, w.e.k_row + row, w.hk, policy);
      else
        tma_load_4d(dst + c * C::kChunkBytes, own, bar, c * 64, n - kTileN, w.e.k_row + row, w.hk);
    }
  }
}

// Tile t of a block's queries.  (Rows past the block's are another one's: they
// reach no row but their own.)
template <int D>
__device__ __forceinline__ void load_queries(uint8_t* dst, uint64_t* bar, const PackedFwd& p, const Piece& w, int t,
                                             const CUtensorMap* m) {
  using C = Cfg<D>;
  mbar_arrive_expect_tx(bar, (uint32_t)(p.group_heads * p.tile_tokens) * 128u * C::kChunks);
#pragma unroll
  for (int c = 0; c < C::kChunks; ++c)
    tma_load_4d(dst + c * C::kChunkBytes, m, bar, c * 64, w.g0, w.e.q_row + t * p.tile_tokens, w.hk);
}

template <int D>
__device__ __forceinline__ void issue_qk(uint32_t tmem_s, uint32_t q_lo, uint32_t k_lo, uint32_t hi) {
  using C = Cfg<D>;
  constexpr uint32_t idesc = idesc_bf16(kTileM, kTileN, false, false);
#pragma unroll
  for (int kk = 0; kk < D / 16; ++kk) {
    const uint32_t off = ((kk / 4) * C::kChunkBytes + (kk % 4) * 32) >> 4;
    mma_ss_lh_w(tmem_s, q_lo + off, hi, k_lo + off, hi, idesc, kk > 0 ? 1u : 0u);
  }
}

template <int D>
__device__ __forceinline__ void issue_pv(uint32_t tmem_o, uint32_t tmem_p, uint32_t v_lo, uint32_t hi,
                                         bool accumulate) {
  constexpr uint32_t idesc = idesc_bf16(kTileM, D, false, true);
#pragma unroll
  for (int kk = 0; kk < kTileN / 16; ++kk)
    mma_ts_lh_w(tmem_o, tmem_p + kk * 8, v_lo + ((kk * 2048) >> 4), hi, idesc, (accumulate || kk > 0) ? 1u : 0u);
}

}  // namespace pk

template <int D, bool DIRECT>
__global__ void __launch_bounds__(384, 1)
    fa_packed_fwd_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                         const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_kp,
                         const __grid_constant__ CUtensorMap tm_vp, const __grid_constant__ CUtensorMap tm_o,
                         const PackedFwd p) {
  using namespace pk;
  using C = Cfg<D>;
  extern __shared__ __align__(1024) uint8_t smem[];
  if ((smem_u32(smem) & 1023u) != 0u) {
    if (threadIdx.x == 0) atomicCAS(p.status, 0u, (unsigned int)FA_ERR_CUDA);
    pdl_wait();
    return;
  }
  uint8_t* sQ = smem + C::kOffQ;
  uint8_t* sKV = smem + C::kOffKV;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::kOffBar);
  const Bars<D, kWhole> wb(bars);
  const Bars<D, kSmall> sb(bars);
  uint64_t* whole_done = bars + 2 * C::kPhaseBars;    // every product of the whole blocks is complete
  uint64_t* drain = whole_done + 1;                   // [2]: of each issuing warp
  uint64_t* half_done = drain + 2;                    // a unit's second half is complete (DirectWalk)
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(half_done + 1);
  constexpr int kHalf = C::kStages / 2;               // ring slots of a warpgroup with small blocks

  const int warp = threadIdx.x / 32;
  const int lane = threadIdx.x % 32;

  if (threadIdx.x == 0) {
    for (int i = 0; i < C::kNumBars; ++i) {
      const int k = i % C::kPhaseBars;
      const bool of_warps = i < 2 * C::kPhaseBars && k >= 6 + 2 * C::kStages && k < 10 + 2 * C::kStages;
      mbar_init(&bars[i], of_warps || i == C::kNumBars - 1 ? 4 : 1);  // p_full, s_read, half_done: a warpgroup's warps
    }
    fence_barrier_init();
  }
  if (warp == 8) {
    tmem_alloc(tmem_slot, C::kTmemCols);
    tmem_relinquish();
  }
  if (warp == 9 && lane == 0) {
    tma_prefetch_desc(&tm_q);
    tma_prefetch_desc(&tm_k);
    tma_prefetch_desc(&tm_v);
    tma_prefetch_desc(&tm_kp);
    tma_prefetch_desc(&tm_vp);
    tma_prefetch_desc(&tm_o);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const WaitCtl ctl{p.status, p.timeout_ns};
  // The plan, and whatever wrote the tensors, is complete.
  pdl_wait();
  pdl_trigger();
  DirectSeqs* const seqs = reinterpret_cast<DirectSeqs*>(smem + C::kOffSeqs);
  if constexpr (DIRECT) {
    if (warp == 0) seqs->fill(p);
    __syncthreads();
  }
  // What an issuing warp does for the small blocks of warpgroup t.
  auto issue_small = [&](auto which_t, bool ok) {
    constexpr uint32_t hi = sdesc_hi(1024);
    constexpr uint32_t kTileStep = C::kTileBytes >> 4;
    const uint32_t q_lo0 = sdesc_lo(smem_u32(sQ), 16);
    const uint32_t k_lo0 = sdesc_lo(smem_u32(sKV), 16);
    const uint32_t v_lo0 = sdesc_lo(smem_u32(sKV), C::kChunkBytes);
    auto wait = [&](uint64_t* bar, uint32_t parity, uint32_t where) -> bool {
      return __all_sync(0xffffffffu, mbar_wait(bar, parity, ctl, where));
    };
    Piece w;
    constexpr int t = decltype(which_t)::value;
    const uint32_t q_lo = q_lo0 + t * kTileStep, t_s = tmem + C::col_s(t), t_o = tmem + C::col_o(t);
    const uint32_t t_p = tmem + C::col_p(t);
    uint32_t pos = 0, qn = 0, pn = 0, sn = 0;  // pos: the unit's first ring place
    auto key_slot = [&](uint32_t i) { return t * kHalf + i % kHalf; };
    auto wait_kv = [&](uint32_t i) -> bool { return wait(sb.kv_full(key_slot(i)), (i / kHalf) & 1, kWaitKvFull); };
    auto issue_s = [&](int j, bool last) -> bool {  // S of the unit's key tile j
      const uint32_t at = pos + 2 * j;
      if (!wait_kv(at) || (C::kOwnP && sn > 0 && !wait(sb.s_read(t), (sn - 1) & 1, kWaitPFull))) return false;
      ++sn;
      tc_fence_after();
      issue_qk<D>(t_s, q_lo, k_lo0 + key_slot(at) * kTileStep, hi);
      mma_commit_w(sb.s_full(t));
      if (last) mma_commit_w(sb.q_empty(t));
      mma_commit_w(sb.kv_empty(key_slot(at)));
      return true;
    };
    Walk<false, DIRECT> walk(p, seqs, kSmall, t);
    while (ok && walk.get(w)) {
      const int n = w.hi - w.lo;
      if (n == 0) continue;
      // (The loads wait for the whole blocks' products.)
      ok = wait(sb.q_full(t), qn & 1, kWaitQFull) && issue_s(0, n == 1);
      ++qn;
      for (int j = 0; ok && j < n; ++j) {
        const uint32_t at = pos + 2 * j + 1;
        if (C::kOwnP && j + 1 < n) ok = issue_s(j + 1, j + 2 == n);
        ok = ok && wait_kv(at) && wait(sb.p_full(t), pn & 1, kWaitPFull);
        ++pn;
        if (!ok) break;
        tc_fence_after();
        issue_pv<D>(t_o, t_p, v_lo0 + key_slot(at) * kTileStep, hi, j > 0);
        mma_commit_w(sb.kv_empty(key_slot(at)));
        if (C::kOwnP || j + 1 == n) mma_commit_w(sb.o_full(t));
        if (!C::kOwnP && j + 1 < n) ok = issue_s(j + 1, j + 2 == n);
      }
      pos += 2 * n;
    }
    // Every MMA this warp issued completes before TMEM is released.
    mma_commit_w(&drain[t]);
    (void)wait(&drain[t], 0, kWaitDrain);
  };
  // What a producer does for the small blocks of warpgroup t.
  auto load_small = [&](auto which_t, bool ok) {
    Piece w;
    constexpr int t = decltype(which_t)::value;
    Walk<true, DIRECT> walk(p, seqs, kSmall, t);
    uint32_t pos = 0, qn = 0;
    // Their own keys are mostly read once (decoding): the L2 cache gives them up first
    // and keeps what blocks share (64 steps behind a prefix 50.6 -> 47.7 us, a server's
    // batch 217.6 -> 214.1, both over changing inputs).
    const uint64_t once = evict_first_policy();
    bool first = true;
    while (ok && walk.get(w)) {
      if (w.hi == w.lo) continue;
      // The products of the whole blocks have read Q and the ring.
      if (first) ok = mbar_wait(whole_done, 0, ctl, kWaitKvEmpty);
      first = false;
      ok = ok && mbar_wait(sb.q_empty(t), (qn & 1) ^ 1, ctl, kWaitQEmpty);
      if (!ok) break;
      load_queries<D>(sQ + t * C::kTileBytes, sb.q_full(t), p, w, 0, &tm_q);
      ++qn;
      for (int x = w.lo; ok && x < w.hi; ++x) {
#pragma unroll
        for (int which = 0; which < 2; ++which) {
          const uint32_t slot = t * kHalf + pos % kHalf;
          ok = ok && mbar_wait(sb.kv_empty(slot), ((pos / kHalf) & 1) ^ 1, ctl, kWaitKvEmpty);
          if (!ok) continue;
          load_keys<D, true>(sKV + slot * C::kTileBytes, sb.kv_full(slot), w, x, which ? &tm_v : &tm_k,
                             which ? &tm_vp : &tm_kp, once);
          ++pos;
        }
      }
    }
    for (uint32_t i = pos > (uint32_t)kHalf ? pos - kHalf : 0u; i < pos; ++i)
      mbar_wait(sb.kv_full(t * kHalf + i % kHalf), (i / kHalf) & 1, ctl, kWaitDrain);
    if (qn > 0) mbar_wait(sb.q_full(t), (qn - 1) & 1, ctl, kWaitDrain);
  };
  if (warp == 9) {
    reg_dealloc<C::kRegsCtl>();
    // ----------------------------------------------------------- producers
    if (lane == 0) {
      bool ok = true;
      Piece w;
      uint32_t rc = 0, qc[2] = {0, 0};
      // Whole blocks.
      Walk<true, DIRECT> walk(p, seqs, kWhole, 0);
      while (ok && walk.get(w)) {
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          if (!ok || (t ? w.hi == w.lo : w.n0 == 0)) continue;
          ok = mbar_wait(wb.q_empty(t), (qc[t] & 1) ^ 1, ctl, kWaitQEmpty);
          if (!ok) continue;
          load_queries<D>(sQ + t * C::kTileBytes, wb.q_full(t), p, w, t, &tm_q);
          ++qc[t];
        }
        for (int x = w.lo; ok && x < w.hi; ++x) {
#pragma unroll
          for (int which = 0; which < 2; ++which) {
            const uint32_t slot = rc % C::kStages;
            ok = ok && mbar_wait(wb.kv_empty(slot), ((rc / C::kStages) & 1) ^ 1, ctl, kWaitKvEmpty);
            if (!ok) continue;
            load_keys<D>(sKV + slot * C::kTileBytes, wb.kv_full(slot), w, x, which ? &tm_v : &tm_k,
                         which ? &tm_vp : &tm_kp);
            ++rc;
          }
        }
      }
      // Let every copy this thread started land before the CTA can exit.
      for (uint32_t pos = rc > (uint32_t)C::kStages ? rc - C::kStages : 0u; pos < rc; ++pos)
        mbar_wait(wb.kv_full(pos % C::kStages), (pos / C::kStages) & 1, ctl, kWaitDrain);
      for (int t = 0; t < 2; ++t)
        if (qc[t] > 0) mbar_wait(wb.q_full(t), (qc[t] - 1) & 1, ctl, kWaitDrain);
      load_small(std::integral_constant<int, 0>{}, ok);
    }
    __syncwarp();
  } else if (warp == 11) {
    reg_dealloc<C::kRegsCtl>();
    if (lane == 0) load_small(std::integral_constant<int, 1>{}, true);
    __syncwarp();
  } else if (warp == 8) {
    reg_dealloc<C::kRegsCtl>();
    // --------------------------------------------------------- MMA issuers
    bool ok = true;
    {
      constexpr uint32_t hi = sdesc_hi(1024);
      constexpr uint32_t kTileStep = C::kTileBytes >> 4;
      const uint32_t q_lo0 = sdesc_lo(smem_u32(sQ), 16);
      const uint32_t k_lo0 = sdesc_lo(smem_u32(sKV), 16);
      const uint32_t v_lo0 = sdesc_lo(smem_u32(sKV), C::kChunkBytes);
      auto wait = [&](uint64_t* bar, uint32_t parity, uint32_t where) -> bool {
        return __all_sync(0xffffffffu, mbar_wait(bar, parity, ctl, where));
      };
      Piece w;
      // Whole blocks: the order of fa_fwd.cu.
      uint32_t rc = 0, qc[2] = {0, 0}, pc[2] = {0, 0}, sc[2] = {0, 0};
      auto wait_kv = [&](uint32_t pos) -> bool {
        return wait(wb.kv_full(pos % C::kStages), (pos / C::kStages) & 1, kWaitKvFull);
      };
      Walk<false, DIRECT> walk(p, seqs, kWhole, 0);
      while (ok && walk.get(w)) {
        const int n1 = w.hi - w.lo;
        if (n1 == 0) continue;
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          if (!ok || (t ? n1 : w.n0) == 0) continue;
          ok = wait(wb.q_full(t), qc[t] & 1, kWaitQFull);
          ++qc[t];
        }
        if constexpr (C::kOwnP) {
          // S of the unit's key tile j for one tile of rows.
          auto issue_s = [&](int t, int j) {
            const int nt = t ? n1 : w.n0;
            const uint32_t slot = (rc + 2 * j) % C::kStages;
            if (sc[t] > 0) ok = wait(wb.s_read(t), (sc[t] - 1) & 1, kWaitPFull);
            ++sc[t];
            ok = ok && wait_kv(rc + 2 * j);
            if (!ok) return;
            tc_fence_after();
            issue_qk<D>(tmem + C::col_s(t), q_lo0 + t * kTileStep, k_lo0 + slot * kTileStep, hi);
            mma_commit_w(wb.s_full(t));
            if (j + 1 == nt) mma_commit_w(wb.q_empty(t));  // Q_t's last product
          };
#pragma unroll
          for (int t = 0; t < 2; ++t)
            if (ok && (t ? n1 : w.n0) > 0) issue_s(t, 0);
          if (ok) mma_commit_w(wb.kv_empty(rc % C::kStages));
          // A tile's next S goes ahead of its product with V, and all of one tile ahead of
          // the other's: that keeps the warpgroups half a step apart, one in the maxima
          // while the other is in the exponentials.
          for (int j = 0; ok && j < n1; ++j) {
            const uint32_t slot = (rc + 2 * j + 1) % C::kStages;
#pragma unroll
            for (int t = 0; t < 2; ++t) {
              const int nt = t ? n1 : w.n0;
              if (!ok || j >= nt) continue;
              if (j + 1 < nt) issue_s(t, j + 1);
              ok = ok && wait_kv(rc + 2 * j + 1) && wait(wb.p_full(t), pc[t] & 1, kWaitPFull);
              ++pc[t];
              if (!ok) continue;
              tc_fence_after();
              issue_pv<D>(tmem + C::col_o(t), tmem + C::col_p(t), v_lo0 + slot * kTileStep, hi, j > 0);
              mma_commit_w(wb.o_full(t));
            }
            if (!ok) break;
            if (j + 1 < n1) mma_commit_w(wb.kv_empty((rc + 2 * j + 2) % C::kStages));
            mma_commit_w(wb.kv_empty(slot));
          }
          if (!ok) break;
        } else {
          ok = ok && wait_kv(rc);
          if (!ok) break;
          tc_fence_after();
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            const int nt = t ? n1 : w.n0;
            if (nt == 0) continue;
            issue_qk<D>(tmem + C::col_s(t), q_lo0 + t * kTileStep, k_lo0 + (rc % C::kStages) * kTileStep, hi);
            mma_commit_w(wb.s_full(t));
            if (nt == 1) mma_commit_w(wb.q_empty(t));  // Q_t's last product
          }
          mma_commit_w(wb.kv_empty(rc % C::kStages));
          for (int j = 0; ok && j < n1; ++j) {
            const uint32_t pos_v = rc + 2 * j + 1;
            const uint32_t pos_k = pos_v + 1;
            const uint32_t slot_v = pos_v % C::kStages;
            const uint32_t slot_k = pos_k % C::kStages;
            ok = wait_kv(pos_v);
            if (!ok) break;
            tc_fence_after();
            bool k_ready = false;
#pragma unroll
            for (int t = 0; t < 2; ++t) {
              const int nt = t ? n1 : w.n0;
              if (!ok || j >= nt) continue;
              ok = wait(wb.p_full(t), pc[t] & 1, kWaitPFull);
              ++pc[t];
              if (!ok) continue;
              tc_fence_after();
              issue_pv<D>(tmem + C::col_o(t), tmem + C::col_p(t), v_lo0 + slot_v * kTileStep, hi, j > 0);
              if (j + 1 < nt) {
                if (!k_ready) {
                  ok = wait_kv(pos_k);
                  if (!ok) continue;
                  tc_fence_after();
                  k_ready = true;
                }
                issue_qk<D>(tmem + C::col_s(t), q_lo0 + t * kTileStep, k_lo0 + slot_k * kTileStep, hi);
                mma_commit_w(wb.s_full(t));
                if (j + 2 == nt) mma_commit_w(wb.q_empty(t));  // Q_t's last product
              } else {
                mma_commit_w(wb.o_full(t));
              }
            }
            if (!ok) break;
            mma_commit_w(wb.kv_empty(slot_v));
            if (j + 1 < n1) mma_commit_w(wb.kv_empty(slot_k));
          }
        }
        rc += 2 * n1;
      }
      mma_commit_w(whole_done);
    }
    issue_small(std::integral_constant<int, 0>{}, ok);
    __syncwarp();
  } else if (warp == 10) {
    reg_dealloc<C::kRegsCtl>();
    issue_small(std::integral_constant<int, 1>{}, true);
    __syncwarp();
  } else if (warp < 8) {
    reg_alloc<C::kRegsMath>();
    // ------------------------------------------------------------- softmax
    const int t = warp >> 2;
    const int wq = warp & 3;  // rows [32 wq, 32 wq + 32) of the tile
    const uint32_t lane_off = (uint32_t)(32 * wq) << 16;
    const uint32_t tS = tmem + lane_off + C::col_s(t);
    const uint32_t tO = tmem + lane_off + C::col_o(t);
    const uint32_t tP = tmem + lane_off + C::col_p(t);
    const int r_in_tile = 32 * wq + lane;
    const int tok = r_in_tile / p.group_heads;      // token within the tile
    const int gh = r_in_tile - tok * p.group_heads;  // query head within the group's run
    const int warp_tok = 32 * wq / p.group_heads;    // the warp's first token
    const float sl2 = p.scale_log2;
    uint8_t* const out = smem + C::kOffOut + warp * 4096;
    bool storing = false;  // a store from `out` may still be reading it
    bool ok = true;
    // The units of a list: one copy of the code for each.
    auto take = [&](auto which) {
      constexpr int kList = decltype(which)::value;
      constexpr bool small = kList == kSmall;
      const Bars<D, kList> bar(bars);
      uint64_t *const s_full = bar.s_full(t), *const p_full = bar.p_full(t), *const s_read = bar.s_read(t);
      uint64_t* const o_full = bar.o_full(t);
      uint32_t sc = 0, oc = 0;
      Walk<true, DIRECT> walk(p, seqs, kList, t);
      Piece w;
      while (ok && walk.get(w)) {
        const int steps = t || small ? w.hi - w.lo : w.n0;
        const int first = small ? 0 : t * p.tile_tokens;         // the tile's first token in the block
        const int here = min(p.tile_tokens, w.e.q_len - first);  // its tokens
        const bool live = warp_tok < here;                       // the warp has rows
        const bool row_ok = tok < here && tok < p.tile_tokens && w.g0 + gh < p.group;
        float m_ref = -INFINITY;  // reference max of this row, log2 units
        // Sum of the fp32 weights: L = m + log l, and O is divided by it.  The product with V
        // has their roundings to bf16, which cancel less than in fa_fwd.cu, where O is divided
        // by the sum of the rounded ones: a third of a step's instructions (16 prompts 208 us
        // with that sum, 202 without), for an error of O that is 0.0001 of 0.0020 larger.
        float l = 0.f;
        for (int j = 0; j < steps; ++j) {
          ok = __all_sync(0xffffffffu, mbar_wait(s_full, sc & 1, ctl, kWaitSFull));
          ++sc;
          if (!ok) break;
          // With columns of its own, P is free (and O complete) once the product before
          // this one is done.
          auto wait_pv = [&]() -> bool {
            if (!C::kOwnP || j == 0) return true;
            const bool done = __all_sync(0xffffffffu, mbar_wait(o_full, oc & 1, ctl, kWaitOFull));
            ++oc;
            tc_fence_after();
            return done;
          };
          if (!live) {
            if (C::kOwnP) mbar_arrive_warp(s_read);
            ok = wait_pv();
            if (!ok) break;
            mbar_arrive_warp(p_full);
            continue;
          }
          tc_fence_after();
          uint32_t s[kTileN];
#pragma unroll
          for (int c = 0; c < kTileN / 32; ++c) tmem_ld32(tS + 32 * c, s + 32 * c);
          tmem_ld_wait<kTileN>(s);
          if (C::kOwnP) {
            tc_fence_before();
            mbar_arrive_warp(s_read);
          }
          float x[kTileN];
#pragma unroll
          for (int c = 0; c < kTileN; ++c) x[c] = __uint_as_float(s[c]);
          const int tile = w.lo + j;
          const bool pre = tile < w.e.prefix;
          const int row = (pre ? tile : tile - w.e.prefix) * kTileN;
          const int len = pre ? p.prefix_len : w.e.k_len;
          const bool causal = p.causal && !pre;
          // Column c is key kv0 + c; a sequence's last tile has its keys at the end.
          const int skip = pre ? 0 : max(0, row + kTileN - len);
          const int kv0 = row - skip;
          if (skip > 0 || kv0 + kTileN > len || (causal && kv0 + kTileN > w.e.pos + first + warp_tok + 1)) {
            const int lim = (causal ? min(len, w.e.pos + first + tok + 1) : len) - kv0;
            // A word of bits for 32 columns, then one select a column (compares of
            // every column took 2500 cycles where this takes 700).
#pragma unroll
            for (int h = 0; h < kTileN / 32; ++h) {
              const int n = lim - 32 * h, z = skip - 32 * h;
              uint32_t see = n >= 32 ? ~0u : n <= 0 ? 0u : (1u << n) - 1u;
              if (z > 0) see &= z >= 32 ? 0u : ~0u << z;
#pragma unroll
              for (int c = 0; c < 32; ++c)
                if (!(see & (1u << c))) x[32 * h + c] = -INFINITY;
            }
          }
          float mx0 = x[0], mx1 = x[1], mx2 = x[2], mx3 = x[3];
#pragma unroll
          for (int c = 4; c + 8 <= kTileN; c += 8) {
            mx0 = fmax3(mx0, x[c], x[c + 1]);
            mx1 = fmax3(mx1, x[c + 2], x[c + 3]);
            mx2 = fmax3(mx2, x[c + 4], x[c + 5]);
            mx3 = fmax3(mx3, x[c + 6], x[c + 7]);
          }
          mx0 = fmax3(mx0, x[kTileN - 4], x[kTileN - 3]);
          mx1 = fmax3(mx1, x[kTileN - 2], x[kTileN - 1]);
          const float m_tile = fmax3(fmaxf(mx0, mx1), mx2, mx3) * sl2;
          float f = 1.f;
          bool rescale = false;
          if (j == 0) {
            m_ref = m_tile;
          } else if (__any_sync(0xffffffffu, row_ok && m_tile > m_ref + C::kRescaleThreshold)) {
            // (A lane without a row holds another sequence's, or what shared memory held before:
            // it has no vote, since rescaling moves the roundings of the warp's other rows.  With
            // its m_ref at +inf instead 32 sentences of d = 96 take 56.0 us, so 55.4.)
            const float m_new = fmaxf(m_ref, m_tile);
            f = (m_new == -INFINITY) ? 1.f : ex2_approx(m_ref - m_new);
            l *= f;
            m_ref = m_new;
            rescale = true;
          }
          ok = wait_pv();
          if (!ok) break;
          const float m_exp = (m_ref == -INFINITY) ? 0.f : m_ref;
          const float2 sl2v = make_float2(sl2, sl2);
          const float2 negv = make_float2(-m_exp, -m_exp);
          float2 ls0 = make_float2(0.f, 0.f), ls1 = ls0;
#pragma unroll
          for (int h = 0; h < kTileN / 32; ++h) {
            uint32_t pk_[16];
#pragma unroll
            for (int e = 0; e < 32; e += 2) {
              const float2 a = __ffma2_rn(make_float2(x[32 * h + e], x[32 * h + e + 1]), sl2v, negv);
              const float p0 = ex2_approx(a.x);
              const float p1 = ex2_approx(a.y);
              const uint32_t pp = pack_bf16(p0, p1);
              if ((e >> 1) & 1) {
                ls1 = __fadd2_rn(ls1, make_float2(p0, p1));
              } else {
                ls0 = __fadd2_rn(ls0, make_float2(p0, p1));
              }
              pk_[e / 2] = pp;
            }
            tmem_st16(tP + 16 * h, pk_);
          }
          l += (ls0.x + ls0.y) + (ls1.x + ls1.y);
          if (rescale) {
#pragma unroll 1
            for (int c = 0; c < D / 32; ++c) {
              uint32_t o[32];
              tmem_ld32(tO + 32 * c, o);
              tmem_ld_wait<32>(o);
#pragma unroll
              for (int i = 0; i < 32; i += 2) {
                const float2 v = __fmul2_rn(make_float2(__uint_as_float(o[i]), __uint_as_float(o[i + 1])),
                                            make_float2(f, f));
                o[i] = __float_as_uint(v.x);
                o[i + 1] = __float_as_uint(v.y);
              }
              tmem_st32(tO + 32 * c, o);
            }
          }
          tmem_st_wait();
          tc_fence_before();
          mbar_arrive_warp(p_full);
        }
        if (!ok) break;
        // ---- the rows' results.  What does not need O is worked out while the last
        // product runs; then all of the row is read at once.
        const int token = w.e.q_row + first + tok;
        const int head = w.hk * p.group + w.g0 + gh;
        const int stretch = small ? 2 * (int)blockIdx.x + t : (int)blockIdx.x;
        const int sl = 2 * stretch + (w.lo > 0 ? 0 : 1);
        const int slot_row = (small ? 0 : kTileM * t) + r_in_tile;
        uint8_t* orow = reinterpret_cast<uint8_t*>(p.o) + ((long long)token * p.o_row + (long long)head * p.o_head) * 2;
        if (steps > 0) {
          ok = __all_sync(0xffffffffu, mbar_wait(o_full, oc & 1, ctl, kWaitOFull));
          ++oc;
          if (!ok) break;
          tc_fence_after();
        }
        bool dual = false;
        if constexpr (DIRECT) dual = walk.dual();
        if (!live) {
          if (dual && t == 1) mbar_arrive_warp(half_done);
          continue;
        }
        // Halves of a unit: the first one's warps find the second's rows of O in the same
        // lanes of tensor memory, its maxima and sums in its room for O.
        if (dual) {
          uint32_t none;  // keeps the addresses from being worked out ahead of the steps, which have no register over
          asm volatile("mov.u32 %0, 0;" : "=r"(none));
          float2* const stats = reinterpret_cast<float2*>(smem + C::kOffOut + (4 + wq) * 4096) + lane + none;
          if (t == 1) {
            if (storing) {  // from that room, rows of a whole block
              if (lane == 0) bulk_wait_read();
              __syncwarp();
            }
            *stats = make_float2(m_ref, l);
            tc_fence_before();
            mbar_arrive_warp(half_done);
            continue;
          }
          ok = __all_sync(0xffffffffu, mbar_wait(half_done, 0, ctl, kWaitOFull));
          if (!ok) break;
          tc_fence_after();
          const float2 other = *stats;
          const float m_new = fmaxf(m_ref, other.x);
          const float keep = m_ref == -INFINITY ? 0.f : ex2_approx(m_ref - m_new);
          const float add = other.x == -INFINITY ? 0.f : ex2_approx(other.x - m_new);
          m_ref = m_new;
          l = l * keep + other.y * add;
          // (Of one tile the second half has nothing, and its columns hold anything.)
#pragma unroll 1
          for (int c = 0; c < D / 16; ++c) {
            uint32_t a[16], b[16];
            tmem_ld16(tO + 16 * c + none, a);
            tmem_ld16(tO + (C::col_o(1) - C::col_o(0)) + 16 * c + none, b);
            tmem_ld_wait<16>(a);
            tmem_ld_wait<16>(b);
#pragma unroll
            for (int i = 0; i < 16; ++i)
              a[i] = __float_as_uint(__uint_as_float(a[i]) * keep + (add > 0.f ? __uint_as_float(b[i]) * add : 0.f));
            tmem_st16(tO + 16 * c, a);
          }
          tmem_st_wait();
        }
        uint32_t o[D];
        if (steps > 0) {
#pragma unroll
          for (int c = 0; c < D / 32; ++c) tmem_ld32(tO + 32 * c, o + 32 * c);
          tmem_ld_wait<D>(o);
        } else {
#pragma unroll
          for (int i = 0; i < D; ++i) o[i] = 0u;
        }
        // A row that saw no key has l = 0: O = 0, L = -inf.  One with a score of NaN or
        // +inf has l = NaN, and O and L with it: the merges drop parts by L = -inf.
        const float inv_l = l == 0.f ? 0.f : 1.0f / l;
        const float lse = l == 0.f ? -INFINITY : (m_ref + lg2_approx(l)) * 0.69314718055994530942f;
        const float2 il = make_float2(inv_l, inv_l);
        if (DIRECT || (!w.cut && !p.shared)) {
#pragma unroll
          for (int i = 0; i < D / 2; ++i) {
            const float2 a = __fmul2_rn(make_float2(__uint_as_float(o[2 * i]), __uint_as_float(o[2 * i + 1])), il);
            o[i] = pack_bf16(a.x, a.y);
          }
          if (p.tile_store && warp_tok + 32 / p.group_heads <= here) {
            // All 32 rows: 64 channels at a time through shared memory, stored by the
            // copy engine.  (Stores from registers, a row a lane, touch 32 lines each: 2800
            // cycles a unit at d = 128, during which the other warps' barriers queue behind
            // them; with rows exchanged between lanes first, 3300.)
#pragma unroll
            for (int h = 0; h < (D + 63) / 64; ++h) {
              if (storing) {
                if (lane == 0) bulk_wait_read();
                __syncwarp();
              }
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                if (64 * h + 8 * i >= D) continue;  // (past d = 96 nothing is stored)
                const uint32_t* x = o + 32 * h + 4 * i;
                *reinterpret_cast<uint4*>(out + lane * 128 + ((i ^ (lane & 7)) << 4)) = make_uint4(x[0], x[1], x[2], x[3]);
              }
              fence_async_shared();
              __syncwarp();
              if (lane == 0) {
                tma_store_4d(&tm_o, out, 64 * h, w.g0, w.e.q_row + first + warp_tok, w.hk);
                bulk_commit();
              }
              storing = true;
            }
          } else if (row_ok) {
            if (p.store32) {
#pragma unroll
              for (int i = 0; i < D / 16; ++i) st_global_v8(orow + 32 * i, o + 8 * i);
            } else {
#pragma unroll
              for (int i = 0; i < D / 8; ++i)
                reinterpret_cast<uint4*>(orow)[i] = make_uint4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
            }
          }
          if (row_ok) p.lse[(size_t)head * p.Tq + token] = lse;
          continue;
        }
#pragma unroll
        for (int i = 0; i < D / 2; ++i) {
          const float2 a = __fmul2_rn(make_float2(__uint_as_float(o[2 * i]), __uint_as_float(o[2 * i + 1])), il);
          o[2 * i] = __float_as_uint(a.x);
          o[2 * i + 1] = __float_as_uint(a.y);
        }
        if (w.cut) {
          const int rows = small ? kSlotRows / 2 : kSlotRows;
          float4* dst = reinterpret_cast<float4*>(p.o_slot[small]) + (size_t)sl * (D / 4) * rows + slot_row;
          if (row_ok) {
#pragma unroll
            for (int i = 0; i < D / 4; ++i)
              dst[i * rows] = make_float4(__uint_as_float(o[4 * i]), __uint_as_float(o[4 * i + 1]),
                                               __uint_as_float(o[4 * i + 2]), __uint_as_float(o[4 * i + 3]));
            p.lse_slot[small][(size_t)sl * rows + slot_row] = lse;
          }
        } else {
          float* prow = p.o_part + (((size_t)(1 - w.e.kind) * p.Tq + token) * p.H + head) * D;
          if (row_ok) {
#pragma unroll
            for (int i = 0; i < D / 8; ++i) st_global_v8(prow + 8 * i, o + 8 * i);
            p.lse_part[((size_t)(1 - w.e.kind) * p.H + head) * p.Tq + token] = lse;
          }
        }
      }
    };
    take(std::integral_constant<int, kWhole>{});
    take(std::integral_constant<int, kSmall>{});
    // The stores have reached the tensor (and read shared memory) before the CTA ends.
    if (lane == 0) bulk_wait();
    __syncwarp();
  } else {
    reg_dealloc<C::kRegsCtl>();
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 8) {
    tc_fence_after();
    tmem_dealloc(tmem, C::kTmemCols);
  }
}

// ------------------------------------------------------------------ launch

template <int D>
static cudaError_t load_t() {
  constexpr auto kWhat = cudaFuncAttributeMaxDynamicSharedMemorySize;
  const cudaError_t e = cudaFuncSetAttribute(fa_packed_fwd_kernel<D, true>, kWhat, pk::Cfg<D>::kSmemBytes);
  return e != cudaSuccess ? e : cudaFuncSetAttribute(fa_packed_fwd_kernel<D, false>, kWhat, pk::Cfg<D>::kSmemBytes);
}

template <int D, bool DIRECT>
static cudaError_t launch_t(const CUtensorMap* tm, const PackedFwd& p, cudaStream_t stream) {
  using C = pk::Cfg<D>;
  // Two CTAs of a cluster run on a pair of SMs.  Where one of a pair takes whole
  // blocks and the other small ones, each in code of its own, the first takes 5 to
  // 8 % longer; so pairs stay together, and the plan gives both the same list.
  return launch_pdl_clusters(!DIRECT && p.grid % 2 == 0 ? 2 : 1, fa_packed_fwd_kernel<D, DIRECT>, dim3(p.grid),
                             dim3(C::kThreads), C::kSmemBytes, stream, tm[0], tm[1], tm[2], tm[3], tm[4], tm[5], p);
}

// Loads the kernels of a head dim on the current device; ahead of their launches.
cudaError_t load_packed_fwd(int d) { return d == 64 ? load_t<64>() : d == 96 ? load_t<96>() : load_t<128>(); }

// tm: Q, K, V, K and V of the prefix (any map where there is none), O (any map
// without tile_store).
cudaError_t launch_packed_fwd(int d, const CUtensorMap* tm, const PackedFwd& p, cudaStream_t stream) {
  switch (d) {
    case 64: return p.direct ? launch_t<64, true>(tm, p, stream) : launch_t<64, false>(tm, p, stream);
    case 96: return p.direct ? launch_t<96, true>(tm, p, stream) : launch_t<96, false>(tm, p, stream);
    case 128: return p.direct ? launch_t<128, true>(tm, p, stream) : launch_t<128, false>(tm, p, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace fa
