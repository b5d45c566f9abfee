// Backward pass over packed sequences (include/fa.h: fa_packed_bwd): the kernels
// of fa_bwd.cu and fa_bwd_pair.cu over units of sequences.  Here: the planning
// kernel, the D preprocess for rows with strides, and the host side.
//
// A unit is a key tile (at d = 128 two) of a sequence for one key/value head,
// or a query tile for one query head; its work is the tiles of the other operand
// that it meets.  Units cannot be cut (dK, dV and dQ are summed in tensor memory,
// in one order), so the list is sorted, heaviest first, and dealt in rounds of
// alternating direction: a CTA with a heavy unit gets a light one next.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstring>

#include "packed.h"
#include "packed_host.h"
#include "packed_seq.cuh"
#include "sm103_primitives.cuh"

namespace fa {

using namespace dev;

cudaError_t launch_bwd_packed_dkdv(int d, const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                                   const CUtensorMap& tdo, const BwdParams& p, int grid, cudaStream_t stream);
cudaError_t launch_bwd_packed_pair(const CUtensorMap& tq64, const CUtensorMap& tq, const CUtensorMap& tk,
                                   const CUtensorMap& tv, const CUtensorMap& tdo64, const CUtensorMap& tdo,
                                   const BwdParams& p, long long units, int sm_count, cudaStream_t stream);
cudaError_t launch_bwd_packed_dq(int d, const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                                 const CUtensorMap& tdo, const BwdParams& p, int grid, cudaStream_t stream);

struct PackedBwdPlan {
  PackedSeqs s;
  int kv_block;       // keys of a dK/dV unit: 128 or 256
  int* seq_base[2];   // [B + 1] first entry of each sequence, of either list (where it does not fit shared memory)
  BwdEntry* entries_kv;
  BwdEntry* entries_q;
  int* counts;        // entries of the two lists
};

namespace {

constexpr int kBuckets = 2048;
constexpr int kPlanShared = 1024;  // sequences up to this number have their places in shared memory

struct BwdPlanShared {
  long long warps[2][32];
  int starts[2][2][32];
  Seq seq[kPlanShared];
  int base[kPlanShared + 1];
  int bucket[kBuckets];
  int most;
};

// Entry i of a list: KV, the i-th key block, else the i-th query tile.
template <bool KV>
__device__ __forceinline__ BwdEntry make_entry(const PackedBwdPlan& p, const Seq* seq, const int* base, int i) {
  const int b = seq_of(base, p.s.B, i);
  const Seq s = seq != nullptr ? seq[b] : load_seq(p.s, b, 0);  // (one with entries is in order)
  BwdEntry e{s.q, s.q_len, s.k, s.k_len, i - base[b], 0, 0, 0};
  e.off = p.s.causal == FA_CAUSAL_BOTTOM_RIGHT ? s.k_len - s.q_len : 0;
  const bool causal = p.s.causal != FA_CAUSAL_NONE;
  if (KV) {
    const int first_row = e.tile * p.kv_block - e.off;  // the first query that sees the block
    e.first = causal && first_row > 0 ? first_row / kTileM : 0;
    e.count = max(0, (s.q_len + kTileM - 1) / kTileM - e.first);
  } else {
    const int tiles = (s.k_len + kTileN - 1) / kTileN;
    const int last_key = min(s.q_len, (e.tile + 1) * kTileM) - 1 + e.off;
    e.count = !causal ? tiles : last_key < 0 ? 0 : min(tiles, last_key / kTileN + 1);
  }
  return e;
}

// One list, heaviest entries first (a counting sort; entries of equal count in any order).
template <bool KV>
__device__ void make_list(const PackedBwdPlan& p, int* far_base, BwdEntry* out, int* count, BwdPlanShared& sh) {
  const int tid = threadIdx.x;
  const int block = KV ? p.kv_block : kTileM;
  const bool few = p.s.B <= kPlanShared;
  int* const base = few ? sh.base : far_base;
  const Seq* const seq = few ? sh.seq : nullptr;
  Scan<long long> scan(sh.warps);
  Scan<int, true> furthest_q(sh.starts[0]), furthest_k(sh.starts[1]);
  if (tid == 0) sh.most = 0;
  for (int i = tid; i < kBuckets; i += kPlanThreads) sh.bucket[i] = 0;
  long long n_all = 0, more;
  int most = 0;  // no entry has more steps: those of a sequence without a mask
  int first_q = 0, first_k = 0, next_q, next_k;
  for (int b0 = 0; b0 < p.s.B; b0 += kPlanThreads) {
    const int b = b0 + tid;
    int tiles = 0;
    const int at_q = max(first_q, furthest_q(b < p.s.B ? start_of(p.s.cu_q, b, p.s.Tq) : 0, &next_q));
    const int at_k = max(first_k, furthest_k(b < p.s.B ? start_of(p.s.cu_k, b, p.s.Tk) : 0, &next_k));
    first_q = max(first_q, next_q);
    first_k = max(first_k, next_k);
    if (b < p.s.B) {
      const Seq s = load_seq(p.s, b, at_q, at_k);
      if (few) sh.seq[b] = s;
      tiles = ((KV ? s.k_len : s.q_len) + block - 1) / block;
      if (tiles > 0) most = max(most, ((KV ? s.q_len : s.k_len) + kTileM - 1) / kTileM);
    }
    const long long sum = n_all + scan(tiles, &more);
    if (b < p.s.B) base[b + 1] = (int)sum;
    n_all += more;
  }
  const int n = (int)n_all;
  if (tid == 0) {
    base[0] = 0;
    *count = n;
  }
  most = __reduce_max_sync(0xffffffffu, most);
  if ((tid & 31) == 0) atomicMax(&sh.most, most);
  __syncthreads();
  most = sh.most;
  // Bucket 0 holds the heaviest.
  auto bucket = [&](int c) { return most < kBuckets ? most - c : (int)((long long)(most - c) * (kBuckets - 1) / most); };
  for (int i = tid; i < n; i += kPlanThreads) atomicAdd(&sh.bucket[bucket(make_entry<KV>(p, seq, base, i).count)], 1);
  __syncthreads();
  // Where each bucket starts: two buckets a thread.
  const int a0 = sh.bucket[2 * tid], a1 = sh.bucket[2 * tid + 1];
  const int end = (int)scan(a0 + a1, &more);
  sh.bucket[2 * tid] = end - a1 - a0;
  sh.bucket[2 * tid + 1] = end - a1;
  __syncthreads();
  for (int i = tid; i < n; i += kPlanThreads) {
    const BwdEntry e = make_entry<KV>(p, seq, base, i);
    out[atomicAdd(&sh.bucket[bucket(e.count)], 1)] = e;
  }
}
static_assert(kBuckets == 2 * kPlanThreads, "two buckets a thread");

}  // namespace

// A CTA for each list.
__global__ void __launch_bounds__(kPlanThreads) fa_packed_bwd_plan_kernel(const PackedBwdPlan p) {
  __shared__ BwdPlanShared sh;
  pdl_trigger();
  if (blockIdx.x == 0) make_list<true>(p, p.seq_base[0], p.entries_kv, p.counts, sh);
  else make_list<false>(p, p.seq_base[1], p.entries_q, p.counts + 1, sh);
}

// D = rowsum(dO * O) for rows of any strides, [H, Tq]: as fa_bwd_preprocess, the
// rows of a head one after another.  It runs beside the planning kernel, which is
// launched in stream order proper, so that what came before is complete; the
// kernel behind it waits for this one alone, so this one ends after the plan.
template <int D>
__global__ void __launch_bounds__(256) fa_packed_pre_kernel(const __nv_bfloat16* __restrict__ o, long long o_row,
                                                            long long o_head, const __nv_bfloat16* __restrict__ dout,
                                                            long long do_row, long long do_head, float* __restrict__ dvec,
                                                            int rows) {
  pdl_trigger();
  constexpr int kVec = (D == 96) ? 3 : 1;
  constexpr int kLanes = D / (8 * kVec);
  constexpr int kSlots = 256 / kLanes;
  constexpr int kRowsPerThread = 4;
  const int part = threadIdx.x % kLanes;
  const int slot = threadIdx.x / kLanes;
  const int base = blockIdx.x * kSlots * kRowsPerThread;
  o += blockIdx.y * o_head;
  dout += blockIdx.y * do_head;
  uint4 a[kRowsPerThread][kVec], b[kRowsPerThread][kVec];
#pragma unroll
  for (int r = 0; r < kRowsPerThread; ++r) {
    const int row = base + r * kSlots + slot;
#pragma unroll
    for (int v = 0; v < kVec; ++v) {
      a[r][v] = b[r][v] = make_uint4(0u, 0u, 0u, 0u);
      if (row < rows) {
        a[r][v] = reinterpret_cast<const uint4*>(o + row * o_row)[part * kVec + v];
        b[r][v] = reinterpret_cast<const uint4*>(dout + row * do_row)[part * kVec + v];
      }
    }
  }
#pragma unroll
  for (int r = 0; r < kRowsPerThread; ++r) {
    float acc = 0.f;
#pragma unroll
    for (int v = 0; v < kVec; ++v) {
      const __nv_bfloat162* a2 = reinterpret_cast<const __nv_bfloat162*>(&a[r][v]);
      const __nv_bfloat162* b2 = reinterpret_cast<const __nv_bfloat162*>(&b[r][v]);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 x = __bfloat1622float2(a2[i]);
        const float2 y = __bfloat1622float2(b2[i]);
        acc = fmaf(x.x, y.x, acc);
        acc = fmaf(x.y, y.y, acc);
      }
    }
#pragma unroll
    for (int off = kLanes / 2; off > 0; off >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, off);
    const int row = base + r * kSlots + slot;
    if (row < rows && part == 0) dvec[(size_t)blockIdx.y * rows + row] = acc;
  }
  pdl_wait();
}

}  // namespace fa

namespace {

using namespace fa::packed_host;

struct Call {
  int d, H, Tq, sm_count;
  long long kv_units, q_units;
  fa::PackedBwdPlan plan;
  fa::BwdParams p;
  CUtensorMap q_clip, q_clip64, do_clip, do_clip64, k_rows, v_rows, q_rows, do_rows, k_clip, v_clip;
  const fa_rows_t *o, *dout;
  float* dvec;
  cudaStream_t st;
};

cudaError_t run_plan(void* ctx) {
  const Call& c = *static_cast<const Call*>(ctx);
  fa::fa_packed_bwd_plan_kernel<<<2, fa::kPlanThreads, 0, c.st>>>(c.plan);
  return cudaGetLastError();
}
template <int D>
cudaError_t pre_t(const Call& c) {
  constexpr int kVec = (D == 96) ? 3 : 1;
  const int per_block = (256 / (D / (8 * kVec))) * 4;
  const long long hs = c.H > 1 ? 1 : 0, rs = c.Tq > 1 ? 1 : 0;
  return fa::launch_pdl(fa::fa_packed_pre_kernel<D>, dim3((c.Tq + per_block - 1) / per_block, c.H), dim3(256), 0, c.st,
                        static_cast<const __nv_bfloat16*>(c.o->ptr), rs * c.o->row_stride, hs * c.o->head_stride,
                        static_cast<const __nv_bfloat16*>(c.dout->ptr), rs * c.dout->row_stride,
                        hs * c.dout->head_stride, c.dvec, c.Tq);
}
cudaError_t run_pre(void* ctx) {
  const Call& c = *static_cast<const Call*>(ctx);
  return c.d == 64 ? pre_t<64>(c) : c.d == 96 ? pre_t<96>(c) : pre_t<128>(c);
}
cudaError_t run_kv(void* ctx) {
  const Call& c = *static_cast<const Call*>(ctx);
  if (c.d == 128)
    return fa::launch_bwd_packed_pair(c.q_clip64, c.q_clip, c.k_rows, c.v_rows, c.do_clip64, c.do_clip, c.p, c.kv_units,
                                      c.sm_count, c.st);
  return fa::launch_bwd_packed_dkdv(c.d, c.q_clip, c.k_rows, c.v_rows, c.do_clip, c.p,
                                    (int)std::min<long long>(c.kv_units, c.sm_count), c.st);
}
cudaError_t run_dq(void* ctx) {
  const Call& c = *static_cast<const Call*>(ctx);
  return fa::launch_bwd_packed_dq(c.d, c.q_rows, c.k_clip, c.v_clip, c.do_rows, c.p,
                                  (int)std::min<long long>(c.q_units, c.sm_count), c.st);
}

}  // namespace

extern "C" int fa_packed_bwd(const fa_rows_t* q, const fa_rows_t* k, const fa_rows_t* v, const fa_rows_t* o,
                             const float* lse, const fa_rows_t* dout, const fa_rows_t* dq, const fa_rows_t* dk,
                             const fa_rows_t* dv, const int* cu_q, const int* cu_k, int B, int Tq, int Tk, int H, int Hkv,
                             int d, int causal, float scale, void* stream) {
  if (B < 1 || Tq < 1 || Tk < 1 || H < 1 || Hkv < 1 || H % Hkv != 0 || B > kMost || Tq > kMost || Tk > kMost ||
      H > 65535)
    return FA_ERR_INVALID_ARG;
  if (!head_dim(d)) return FA_ERR_UNSUPPORTED;
  if (causal < FA_CAUSAL_NONE || causal > FA_CAUSAL_BOTTOM_RIGHT) return FA_ERR_INVALID_ARG;
  if (!(std::isfinite(scale) && scale > 0.f)) return FA_ERR_INVALID_ARG;
  for (const fa_rows_t* r : {q, o, dout, dq})
    if (!rows_ok(r, Tq, H)) return FA_ERR_INVALID_ARG;
  for (const fa_rows_t* r : {k, v, dk, dv})
    if (!rows_ok(r, Tk, Hkv)) return FA_ERR_INVALID_ARG;
  if (!rows_apart(dq, Tq, H, d) || !rows_apart(dk, Tk, Hkv, d) || !rows_apart(dv, Tk, Hkv, d)) return FA_ERR_INVALID_ARG;
  if (!array_ok(lse, 16) || !array_ok(cu_q, 4) || !array_ok(cu_k, 4)) return FA_ERR_INVALID_ARG;
  Call c;
  std::memset(&c, 0, sizeof(c));
  const int kv_block = d == 128 ? 256 : 128;
  const long long kv_most = Tk / kv_block + (long long)std::min(B, Tk), q_most = Tq / 128 + (long long)std::min(B, Tq);
  c.kv_units = kv_most * Hkv;
  c.q_units = q_most * H;
  if (c.kv_units > 0x7fffffffLL || c.q_units > 0x7fffffffLL) return FA_ERR_INVALID_ARG;
  unsigned int* status = nullptr;
  int sm_count = 0;
  const int e = fa::internal_device_setup(&status, &sm_count);
  if (e) return e;

  if (encode_tile(&c.q_clip, q, Tq, H, d, 128) || encode_tile(&c.do_clip, dout, Tq, H, d, 128) ||
      encode_tile(&c.k_clip, k, Tk, Hkv, d, 128) || encode_tile(&c.v_clip, v, Tk, Hkv, d, 128) ||
      encode_plain(&c.q_rows, q, Tq, H, d) || encode_plain(&c.do_rows, dout, Tq, H, d) ||
      encode_plain(&c.k_rows, k, Tk, Hkv, d) || encode_plain(&c.v_rows, v, Tk, Hkv, d))
    return FA_ERR_CUDA;
  if (d == 128 && (encode_tile(&c.q_clip64, q, Tq, H, d, 64) || encode_tile(&c.do_clip64, dout, Tq, H, d, 64)))
    return FA_ERR_CUDA;

  const size_t n_kv = up((size_t)kv_most * sizeof(fa::BwdEntry)), n_q = up((size_t)q_most * sizeof(fa::BwdEntry));
  const size_t n_base = up((2 * ((size_t)B + 1) + 2) * sizeof(int)), n_d = (size_t)H * Tq * sizeof(float);
  c.st = static_cast<cudaStream_t>(stream);
  void* ws = nullptr;
  if (fa::internal_workspace(&ws, n_kv + n_q + n_base + n_d, c.st) != cudaSuccess) {
    cudaGetLastError();
    return FA_ERR_NO_MEMORY;
  }
  char* at = static_cast<char*>(ws);
  c.plan.entries_kv = reinterpret_cast<fa::BwdEntry*>(at);
  c.plan.entries_q = reinterpret_cast<fa::BwdEntry*>(at += n_kv);
  c.plan.counts = reinterpret_cast<int*>(at += n_q);
  c.plan.seq_base[0] = c.plan.counts + 2;
  c.plan.seq_base[1] = c.plan.seq_base[0] + B + 1;
  c.dvec = reinterpret_cast<float*>(at + n_base);
  c.plan.s = fa::PackedSeqs{cu_q, cu_k, nullptr, B, Tq, Tk, causal, status};
  c.plan.kv_block = kv_block;
  c.d = d;
  c.H = H;
  c.Tq = Tq;
  c.sm_count = sm_count;
  c.o = o;
  c.dout = dout;
  fa::BwdParams& p = c.p;
  p.B = 1;
  p.H = H;
  p.Hkv = Hkv;
  p.Nq = Tq;
  p.Nk = Tk;
  p.causal = causal != FA_CAUSAL_NONE ? 1 : 0;
  p.scale = scale;
  p.scale_log2 = scale * 1.4426950408889634f;
  p.lse = lse;
  p.dvec = c.dvec;
  p.dq = dq->ptr;
  p.dk = dk->ptr;
  p.dv = dv->ptr;
  p.dq_row = dq->row_stride, p.dq_head = dq->head_stride;
  p.dk_row = dk->row_stride, p.dk_head = dk->head_stride;
  p.dv_row = dv->row_stride, p.dv_head = dv->head_stride;
  if (Tq == 1) p.dq_row = 0;
  if (H == 1) p.dq_head = 0;
  if (Tk == 1) p.dk_row = p.dv_row = 0;
  if (Hkv == 1) p.dk_head = p.dv_head = 0;
  p.store32 = aligned32(dq->ptr, p.dq_row, p.dq_head) && aligned32(dk->ptr, p.dk_row, p.dk_head) &&
                      aligned32(dv->ptr, p.dv_row, p.dv_head)
                  ? 1
                  : 0;
  p.group = H / Hkv;
  p.status = status;
  p.timeout_ns = fa::internal_wait_timeout_ns();
  p.entries_kv = c.plan.entries_kv;
  p.entries_q = c.plan.entries_q;
  p.entry_counts = c.plan.counts;

  cudaError_t ce = fa::internal_timed_launch(FA_KERNEL_PACKED_PLAN, c.st, run_plan, &c);
  if (ce == cudaSuccess) ce = fa::internal_timed_launch(FA_KERNEL_BWD_PRE, c.st, run_pre, &c);
  if (ce == cudaSuccess) ce = fa::internal_timed_launch(FA_KERNEL_BWD, c.st, run_kv, &c);
  if (ce == cudaSuccess) ce = fa::internal_timed_launch(FA_KERNEL_BWD_DQ, c.st, run_dq, &c);
  cudaFreeAsync(ws, c.st);
  return ce == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}
