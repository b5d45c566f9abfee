// Forward pass over packed sequences on sm_103a (include/fa.h: fa_packed_fwd,
// fa_prefix_fwd): the products, online softmax and roles of fa_fwd.cu over the
// list of units of packed.h.  What differs:
//
//  * A CTA walks a stretch of the list that the planning kernel gave it, and may
//    start and end within a unit.
//  * A unit's key tiles are those of the shared prefix (all visible), then the
//    sequence's own (causal or not, up to its length).
//  * Rows of a tile are (token, query head) pairs, so that the query heads of a
//    key/value head share its K and V.
//  * A block of at most one tile of rows (decoding, the ends of sequences) is
//    taken by both warpgroups: both hold the same rows, warpgroup t takes the key
//    tiles lo + t, lo + t + 2, ..., and at the end the second hands its maximum,
//    sums and O to the first through shared memory.  One tile a step then keeps
//    two chains of S, softmax and P V going.
//  * A warp whose 32 rows lie past the block's skips the element-wise work (its
//    rows of P stay what they were; they reach only rows of O that are not kept).
//
// Both warpgroups, registers, tensor memory columns and the rounding of P are as
// described there.
#include <cuda_runtime.h>

#include "packed.h"
#include "sm103_primitives.cuh"

namespace fa {

using namespace dev;

namespace pk {

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
  static constexpr uint32_t kTmemCols = 512;
  static constexpr int kOffQ = 0;
  static constexpr int kOffKV = 2 * kTileBytes;
  // Room of 4 KB for each element-wise warp, from which its rows of O are stored
  // (32 rows of 128 bytes, swizzled).  That of the second warpgroup also takes
  // what it hands over: 16 KB of O, [warp][column / 4][lane] float4; (m, l, l_bf) of
  // 128 rows lie apart.
  static constexpr int kOffOut = kOffKV + kStages * kTileBytes;
  static constexpr int kOffEx = kOffOut + 4 * 4096;
  static constexpr int kOffStat = kOffEx + 4 * 4096;
  static constexpr int kOffBar = kOffStat + 3 * 128 * 4;
  static constexpr int kNumBars = 2 + 2 + 2 * kStages + 2 + 2 + 2 + 4 + 4 + 1;
  static constexpr int kSmemBytes = kOffBar + kNumBars * 8 + 16;
  static_assert(kSmemBytes <= 232448, "shared memory");
  static constexpr float kRescaleThreshold = 24.0f;  // log2 units, as in fa_fwd.cu
  static constexpr int kRegsAtLaunch = 168;
  static constexpr int kRegsCtl = 72;
  static constexpr int kRegsMath = 216;
  static_assert(128 * kRegsCtl + 256 * kRegsMath <= kThreads * kRegsAtLaunch, "register split exceeds the launch");
  static_assert(kRegsCtl % 8 == 0 && kRegsMath % 8 == 0, "setmaxnreg counts are multiples of 8");
};

// A CTA's part of one unit.
struct Piece {
  PackedEntry e;
  int hk, g0;    // key/value head, first query head of the group's
  int lo, hi;    // tiles of this part
  int n0, n1;    // steps of warpgroup 0 and 1
  bool dual;     // both warpgroups on the block's one tile
  bool cut;      // not the whole unit
};

// The units of a CTA, in order.  The next entry is fetched a unit ahead.
struct Walk {
  const PackedFwd& p;
  PackedStart s0, s1;
  int entries;
  int u, u_last, at, hk, chunk;
  PackedEntry next;

  __device__ __forceinline__ static PackedEntry fetch(const PackedEntry* e) {
    const int4* w = reinterpret_cast<const int4*>(e);
    const int4 a = w[0], b = w[1];
    return PackedEntry{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
  }
  __device__ __forceinline__ explicit Walk(const PackedFwd& params) : p(params) {
    s0 = p.starts[blockIdx.x];
    s1 = p.starts[blockIdx.x + 1];
    entries = p.header[0];
    u = s0.unit;
    u_last = s1.tile > 0 ? s1.unit : s1.unit - 1;
    if (s0.unit == s1.unit && s0.tile == s1.tile) u_last = u - 1;
    hk = chunk = at = 0;
    if (u <= u_last) {
      const int hg = u / entries;
      at = u - hg * entries;
      hk = hg / p.chunks;
      chunk = hg - hk * p.chunks;
      next = fetch(p.entries + at);
    }
  }
  __device__ __forceinline__ bool get(Piece& w) {
    if (u > u_last) return false;
    w.e = next;
    w.hk = hk;
    w.g0 = chunk * p.group_heads;
    w.lo = u == s0.unit ? s0.tile : 0;
    w.hi = u == s1.unit ? s1.tile : w.e.tiles;
    w.cut = w.lo > 0 || w.hi < w.e.tiles;
    w.dual = w.e.q_len <= p.tile_tokens;
    ++u;
    if (++at == entries) {
      at = 0;
      if (++chunk == p.chunks) {
        chunk = 0;
        ++hk;
      }
    }
    if (u <= u_last) next = fetch(p.entries + at);
    if (w.dual) {
      const int nk = max(0, w.hi - w.lo);
      w.n0 = (nk + 1) / 2;
      w.n1 = nk / 2;
    } else {
      // The second tile holds the block's last token; the first may see less.
      const int own = p.causal ? min(w.e.k_len, max(0, w.e.pos + p.tile_tokens)) : w.e.k_len;
      const int seen = w.e.kind ? w.e.prefix : w.e.prefix + (own + kTileN - 1) / kTileN;
      w.n0 = max(0, min(w.hi, seen) - w.lo);
      w.n1 = max(0, w.hi - w.lo);
    }
    return true;
  }
};

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

template <int D>
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
  uint64_t* q_full = bars;
  uint64_t* q_empty = bars + 2;
  uint64_t* kv_full = bars + 4;
  uint64_t* kv_empty = kv_full + C::kStages;
  uint64_t* s_full = kv_empty + C::kStages;
  uint64_t* p_full = s_full + 2;
  uint64_t* o_full = p_full + 2;
  uint64_t* ex_full = o_full + 2;   // [4]: warp w's columns handed over
  uint64_t* ex_free = ex_full + 4;  // [4]: ... and read
  uint64_t* drain = ex_free + 4;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);

  const int warp = threadIdx.x / 32;
  const int lane = threadIdx.x % 32;

  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&q_full[i], 1);
      mbar_init(&q_empty[i], 1);
      mbar_init(&s_full[i], 1);
      mbar_init(&p_full[i], 4);
      mbar_init(&o_full[i], 1);
    }
    for (int i = 0; i < C::kStages; ++i) {
      mbar_init(&kv_full[i], 1);
      mbar_init(&kv_empty[i], 1);
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(&ex_full[i], 1);
      mbar_init(&ex_free[i], 1);
    }
    mbar_init(drain, 1);
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
  if (warp == 9) {
    reg_dealloc<C::kRegsCtl>();
    // ------------------------------------------------------------ producer
    if (lane == 0) {
      const uint32_t q_bytes = (uint32_t)(p.group_heads * p.tile_tokens) * 128u * C::kChunks;
      uint32_t rc = 0;
      uint32_t qc[2] = {0, 0};
      bool ok = true;
      Walk walk(p);
      Piece w;
      while (ok && walk.get(w)) {
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          if (!ok || (t ? w.dual || w.n1 == 0 : w.n0 == 0)) continue;
          ok = mbar_wait(&q_empty[t], (qc[t] & 1) ^ 1, ctl, kWaitQEmpty);
          if (!ok) continue;
          // (Rows past the block's are another one's: they reach no row but their own.)
          mbar_arrive_expect_tx(&q_full[t], q_bytes);
          for (int c = 0; c < C::kChunks; ++c)
            tma_load_4d(sQ + t * C::kTileBytes + c * C::kChunkBytes, &tm_q, &q_full[t], c * 64, w.g0,
                        w.e.q_row + t * p.tile_tokens, w.hk);
          ++qc[t];
        }
        for (int x = w.lo; ok && x < w.hi; ++x) {
          const bool pre = x < w.e.prefix;
          const int row = (pre ? x : x - w.e.prefix) * kTileN;
          const int n = min(kTileN, w.e.k_len - row);  // keys of the sequence in an own tile
          for (int which = 0; which < 2; ++which) {
            const uint32_t slot = rc % C::kStages;
            ok = mbar_wait(&kv_empty[slot], ((rc / C::kStages) & 1) ^ 1, ctl, kWaitKvEmpty);
            if (!ok) break;
            mbar_arrive_expect_tx(&kv_full[slot], C::kTileBytes);
            uint8_t* dst = sKV + slot * C::kTileBytes;
            for (int c = 0; c < C::kChunks; ++c) {
              if (pre)
                tma_load_3d(dst + c * C::kChunkBytes, which ? &tm_vp : &tm_kp, &kv_full[slot], c * 64, row, w.hk);
              else
                tma_load_4d(dst + c * C::kChunkBytes, which ? &tm_v : &tm_k, &kv_full[slot], c * 64, n - kTileN,
                            w.e.k_row + row, w.hk);
            }
            ++rc;
          }
        }
      }
      // Let every copy this thread started land before the CTA can exit.
      const uint32_t first = rc > (uint32_t)C::kStages ? rc - C::kStages : 0u;
      for (uint32_t pos = first; pos < rc; ++pos)
        mbar_wait(&kv_full[pos % C::kStages], (pos / C::kStages) & 1, ctl, kWaitDrain);
      for (int t = 0; t < 2; ++t)
        if (qc[t] > 0) mbar_wait(&q_full[t], (qc[t] - 1) & 1, ctl, kWaitDrain);
    }
  } else if (warp == 8) {
    reg_dealloc<C::kRegsCtl>();
    // ---------------------------------------------------------- MMA issuer
    {
      constexpr uint32_t hi = sdesc_hi(1024);
      constexpr uint32_t kTileStep = C::kTileBytes >> 4;
      const uint32_t q_lo0 = sdesc_lo(smem_u32(sQ), 16);
      const uint32_t k_lo0 = sdesc_lo(smem_u32(sKV), 16);
      const uint32_t v_lo0 = sdesc_lo(smem_u32(sKV), C::kChunkBytes);
      uint32_t rc = 0;
      uint32_t qc[2] = {0, 0}, pc[2] = {0, 0};
      bool ok = true;
      auto wait = [&](uint64_t* bar, uint32_t parity, uint32_t where) -> bool {
        return __all_sync(0xffffffffu, mbar_wait(bar, parity, ctl, where));
      };
      auto wait_kv = [&](uint32_t pos) -> bool {
        return wait(&kv_full[pos % C::kStages], (pos / C::kStages) & 1, kWaitKvFull);
      };
      Walk walk(p);
      Piece w;
      while (ok && walk.get(w)) {
        const int nmax = max(w.n0, w.n1);
        if (nmax == 0) continue;
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          if (!ok || (t ? w.dual || w.n1 == 0 : w.n0 == 0)) continue;
          ok = wait(&q_full[t], qc[t] & 1, kWaitQFull);
          ++qc[t];
        }
        if (!ok) break;
        if (w.dual) {
          // Warpgroup t's step j reads key tile 2j + t (K at position rc + 2
          // (2j + t), V one after it); each K and V has one reader and is
          // released after its product.
          const int nk = w.n0 + w.n1;
          auto qk = [&](int t, int j) -> bool {
            const int tile = 2 * j + t;
            const uint32_t pos_k = rc + 2 * tile;
            if (!wait_kv(pos_k)) return false;
            tc_fence_after();
            issue_qk<D>(tmem + C::col_s(t), q_lo0, k_lo0 + (pos_k % C::kStages) * kTileStep, hi);
            mma_commit_w(&s_full[t]);
            if (tile + 1 == nk) mma_commit_w(&q_empty[0]);  // the block's last product with Q
            mma_commit_w(&kv_empty[pos_k % C::kStages]);
            return true;
          };
          ok = qk(0, 0);
          if (ok && w.n1 > 0) ok = qk(1, 0);
          for (int j = 0; ok && j < nmax; ++j) {
#pragma unroll
            for (int t = 0; t < 2; ++t) {
              const int nt = t ? w.n1 : w.n0;
              if (!ok || j >= nt) continue;
              const uint32_t pos_v = rc + 2 * (2 * j + t) + 1;
              ok = wait_kv(pos_v) && wait(&p_full[t], pc[t] & 1, kWaitPFull);
              ++pc[t];
              if (!ok) continue;
              tc_fence_after();
              issue_pv<D>(tmem + C::col_o(t), tmem + C::col_s(t), v_lo0 + (pos_v % C::kStages) * kTileStep, hi, j > 0);
              mma_commit_w(&kv_empty[pos_v % C::kStages]);
              if (j + 1 < nt)
                ok = qk(t, j + 1);
              else
                mma_commit_w(&o_full[t]);
            }
          }
          rc += 2 * nk;
          continue;
        }
        {
          const uint32_t slot_k = rc % C::kStages;
          ok = wait_kv(rc);
          if (!ok) break;
          tc_fence_after();
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            const int nt = t ? w.n1 : w.n0;
            if (nt == 0) continue;
            issue_qk<D>(tmem + C::col_s(t), q_lo0 + t * kTileStep, k_lo0 + slot_k * kTileStep, hi);
            mma_commit_w(&s_full[t]);
            if (nt == 1) mma_commit_w(&q_empty[t]);  // Q_t's last product
          }
          mma_commit_w(&kv_empty[slot_k]);
        }
        for (int j = 0; ok && j < nmax; ++j) {
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
            const int nt = t ? w.n1 : w.n0;
            if (!ok || j >= nt) continue;
            ok = wait(&p_full[t], pc[t] & 1, kWaitPFull);
            ++pc[t];
            if (!ok) continue;
            tc_fence_after();
            issue_pv<D>(tmem + C::col_o(t), tmem + C::col_s(t), v_lo0 + slot_v * kTileStep, hi, j > 0);
            if (j + 1 < nt) {
              if (!k_ready) {
                ok = wait_kv(pos_k);
                if (!ok) continue;
                tc_fence_after();
                k_ready = true;
              }
              issue_qk<D>(tmem + C::col_s(t), q_lo0 + t * kTileStep, k_lo0 + slot_k * kTileStep, hi);
              mma_commit_w(&s_full[t]);
              if (j + 2 == nt) mma_commit_w(&q_empty[t]);  // Q_t's last product
            } else {
              mma_commit_w(&o_full[t]);
            }
          }
          if (!ok) break;
          mma_commit_w(&kv_empty[slot_v]);
          if (j + 1 < nmax) mma_commit_w(&kv_empty[slot_k]);
        }
        rc += 2 * nmax;
      }
      // Every MMA this warp issued completes before TMEM is released.
      mma_commit_w(drain);
      (void)wait(drain, 0, kWaitDrain);
    }
    __syncwarp();
  } else if (warp < 8) {
    reg_alloc<C::kRegsMath>();
    // ------------------------------------------------------------- softmax
    const int t = warp >> 2;
    const int wq = warp & 3;  // rows [32 wq, 32 wq + 32) of the tile
    const uint32_t lane_off = (uint32_t)(32 * wq) << 16;
    const uint32_t tS = tmem + lane_off + C::col_s(t);
    const uint32_t tO = tmem + lane_off + C::col_o(t);
    const int r_in_tile = 32 * wq + lane;
    const int tok = r_in_tile / p.group_heads;      // token within the tile
    const int gh = r_in_tile - tok * p.group_heads;  // query head within the group's run
    const int warp_tok = 32 * wq / p.group_heads;    // the warp's first token
    const float sl2 = p.scale_log2;
    float4* const ex0 = reinterpret_cast<float4*>(smem + C::kOffEx);
    uint8_t* const out = smem + C::kOffOut + warp * 4096;
    bool storing = false;  // a store from `out` may still be reading it
    float* stat = reinterpret_cast<float*>(smem + C::kOffStat);
    uint32_t sc = 0, oc = 0, xc = 0;
    bool ok = true;
    Walk walk(p);
    Piece w;
    while (ok && walk.get(w)) {
      const int steps = t ? w.n1 : w.n0;
      const int first = w.dual ? 0 : t * p.tile_tokens;     // the tile's first token in the block
      const int here = min(p.tile_tokens, w.e.q_len - first);  // its tokens (<= 0: none)
      const bool live = warp_tok < here;                       // the warp has rows
      const bool row_ok = tok < here && tok < p.tile_tokens && w.g0 + gh < p.group;
      const bool mine = !w.dual || t == 0;                     // this warpgroup writes the rows
      const int token = w.e.q_row + first + tok;
      const int head = w.hk * p.group + w.g0 + gh;
      float m_ref = -INFINITY;  // reference max of this row, log2 units
      float l = 0.f;     // sum of the fp32 weights: L = m + log l
      float l_bf = 0.f;  // sum of the bf16-rounded weights the PV MMA takes: O = O~ / l_bf
      for (int j = 0; j < steps; ++j) {
        ok = __all_sync(0xffffffffu, mbar_wait(&s_full[t], sc & 1, ctl, kWaitSFull));
        ++sc;
        if (!ok) break;
        if (j == 0 && storing) {
          // Before this warp's first arrival of the unit: so whoever writes `out` after
          // the unit's products finds it read.
          if (lane == 0) bulk_wait_read();
          __syncwarp();
          storing = false;
        }
        if (!live) {
          mbar_arrive_warp(&p_full[t]);
          continue;
        }
        tc_fence_after();
        uint32_t s[kTileN];
#pragma unroll
        for (int c = 0; c < kTileN / 32; ++c) tmem_ld32(tS + 32 * c, s + 32 * c);
        tmem_ld_wait<kTileN>(s);
        float x[kTileN];
#pragma unroll
        for (int c = 0; c < kTileN; ++c) x[c] = __uint_as_float(s[c]);
        const int tile = w.lo + (w.dual ? 2 * j + t : j);
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
        } else if (__any_sync(0xffffffffu, m_tile > m_ref + C::kRescaleThreshold)) {
          const float m_new = fmaxf(m_ref, m_tile);
          f = (m_new == -INFINITY) ? 1.f : ex2_approx(m_ref - m_new);
          l *= f;
          l_bf *= f;
          m_ref = m_new;
          rescale = true;
        }
        const float m_exp = (m_ref == -INFINITY) ? 0.f : m_ref;
        const float2 sl2v = make_float2(sl2, sl2);
        const float2 negv = make_float2(-m_exp, -m_exp);
        float2 ls0 = make_float2(0.f, 0.f), ls1 = ls0;
        float lr0 = 0.f, lr1 = 0.f, lr2 = 0.f, lr3 = 0.f;
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
              lr2 = add_bf16_lo(lr2, pp);
              lr3 = add_bf16_hi(lr3, pp);
            } else {
              ls0 = __fadd2_rn(ls0, make_float2(p0, p1));
              lr0 = add_bf16_lo(lr0, pp);
              lr1 = add_bf16_hi(lr1, pp);
            }
            pk_[e / 2] = pp;
          }
          tmem_st16(tS + 16 * h, pk_);
        }
        l += (ls0.x + ls0.y) + (ls1.x + ls1.y);
        l_bf += (lr0 + lr1) + (lr2 + lr3);
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
        mbar_arrive_warp(&p_full[t]);
      }
      if (!ok) break;
      // ---- the rows' results.  What does not need O is worked out while the last
      // product runs; then all of the row is read at once.
      const bool joined = w.dual && w.n1 > 0;                // the second warpgroup hands over
      const int live_warps = (here * p.group_heads + 31) / 32;
      // Groups of columns handed over at a time: the four warps' room is for all who have rows.
      const int group = live_warps <= 1 ? 4 : live_warps == 2 ? 2 : 1;
      float4* ex = ex0 + wq * group * 256;
      const int sl = 2 * (int)blockIdx.x + (w.lo > 0 ? 0 : 1);
      const int slot_row = (w.dual ? 0 : kTileM * t) + r_in_tile;
      uint8_t* orow = reinterpret_cast<uint8_t*>(p.o) + ((long long)token * p.o_row + (long long)head * p.o_head) * 2;
      if (steps > 0) {
        ok = __all_sync(0xffffffffu, mbar_wait(&o_full[t], oc & 1, ctl, kWaitOFull));
        ++oc;
        if (!ok) break;
        tc_fence_after();
      }
      if (!live || (!mine && !joined)) continue;
      uint32_t o[D];
      if (steps > 0) {
#pragma unroll
        for (int c = 0; c < D / 32; ++c) tmem_ld32(tO + 32 * c, o + 32 * c);
        tmem_ld_wait<D>(o);
      } else {
#pragma unroll
        for (int i = 0; i < D; ++i) o[i] = 0u;
      }
      if (!mine) {
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
          const int place = c & (group - 1);
          if (place == 0) {
            ok = ok && __all_sync(0xffffffffu, mbar_wait(&ex_free[wq], (xc & 1) ^ 1, ctl, kWaitPFull));
            ++xc;
          }
          if (!ok) continue;
          if (c == 0) {
            stat[r_in_tile] = m_ref;
            stat[128 + r_in_tile] = l;
            stat[256 + r_in_tile] = l_bf;
          }
#pragma unroll
          for (int i = 0; i < 8; ++i)
            ex[(8 * place + i) * 32 + lane] =
                make_float4(__uint_as_float(o[32 * c + 4 * i]), __uint_as_float(o[32 * c + 4 * i + 1]),
                            __uint_as_float(o[32 * c + 4 * i + 2]), __uint_as_float(o[32 * c + 4 * i + 3]));
          if (place == group - 1 || c == D / 32 - 1) mbar_arrive_warp(&ex_full[wq]);
        }
        continue;
      }
      if (joined) {
        float a0 = 1.f, a1 = 0.f;
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
          const int place = c & (group - 1);
          if (place == 0) {
            ok = ok && __all_sync(0xffffffffu, mbar_wait(&ex_full[wq], xc & 1, ctl, kWaitPFull));
            ++xc;
          }
          if (!ok) continue;
          if (c == 0) {
            const float m1 = stat[r_in_tile], l1 = stat[128 + r_in_tile], b1 = stat[256 + r_in_tile];
            const float m = fmaxf(m_ref, m1);
            a0 = m_ref == -INFINITY ? 0.f : ex2_approx(m_ref - m);
            a1 = m1 == -INFINITY ? 0.f : ex2_approx(m1 - m);
            l = l * a0 + l1 * a1;
            l_bf = l_bf * a0 + b1 * a1;
            m_ref = m;
          }
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float4 y = ex[(8 * place + i) * 32 + lane];
            uint32_t* x = o + 32 * c + 4 * i;
            x[0] = __float_as_uint(__uint_as_float(x[0]) * a0 + y.x * a1);
            x[1] = __float_as_uint(__uint_as_float(x[1]) * a0 + y.y * a1);
            x[2] = __float_as_uint(__uint_as_float(x[2]) * a0 + y.z * a1);
            x[3] = __float_as_uint(__uint_as_float(x[3]) * a0 + y.w * a1);
          }
          if (place == group - 1 || c == D / 32 - 1) mbar_arrive_warp(&ex_free[wq]);
        }
        if (!ok) break;
      }
      // A row that saw no key has l = 0: O = 0, L = -inf.
      const float inv_l = l_bf > 0.f ? 1.0f / l_bf : 0.f;
      const float lse = l > 0.f ? (m_ref + lg2_approx(l)) * 0.69314718055994530942f : -INFINITY;
      const float2 il = make_float2(inv_l, inv_l);
      if (!w.cut && !p.shared) {
#pragma unroll
        for (int i = 0; i < D / 2; ++i) {
          const float2 a = __fmul2_rn(make_float2(__uint_as_float(o[2 * i]), __uint_as_float(o[2 * i + 1])), il);
          o[i] = pack_bf16(a.x, a.y);
        }
        // (The second warpgroup's room may hold what the first still reads of the unit
        // before; the first has read it once it has a product in this unit.)
        if (p.tile_store && warp_tok + 32 / p.group_heads <= here && (t == 0 || w.n0 > 0)) {
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
        float4* dst = reinterpret_cast<float4*>(p.o_slot) + (size_t)sl * (D / 4) * kSlotRows + slot_row;
        if (row_ok) {
#pragma unroll
          for (int i = 0; i < D / 4; ++i)
            dst[i * kSlotRows] = make_float4(__uint_as_float(o[4 * i]), __uint_as_float(o[4 * i + 1]),
                                             __uint_as_float(o[4 * i + 2]), __uint_as_float(o[4 * i + 3]));
          p.lse_slot[(size_t)sl * kSlotRows + slot_row] = lse;
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
static cudaError_t launch_t(const CUtensorMap* tm, const PackedFwd& p, cudaStream_t stream) {
  using C = pk::Cfg<D>;
  const cudaError_t e =
      cudaFuncSetAttribute(fa_packed_fwd_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmemBytes);
  if (e != cudaSuccess) return e;
  return launch_pdl(fa_packed_fwd_kernel<D>, dim3(p.grid), dim3(C::kThreads), C::kSmemBytes, stream, tm[0], tm[1], tm[2],
                    tm[3], tm[4], tm[5], p);
}

// tm: Q, K, V, K and V of the prefix (any map where there is none), O (any map
// without tile_store).
cudaError_t launch_packed_fwd(int d, const CUtensorMap* tm, const PackedFwd& p, cudaStream_t stream) {
  switch (d) {
    case 64: return launch_t<64>(tm, p, stream);
    case 96: return launch_t<96>(tm, p, stream);
    case 128: return launch_t<128>(tm, p, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace fa
