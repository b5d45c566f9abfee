// Attention over packed sequences: the planning kernel, the merge of partial
// results and the host side (include/fa.h: fa_packed_fwd, fa_prefix_fwd).  The
// forward kernel is fa_packed_fwd.cu, what all share packed.h.
//
// The lengths are on the device, so the list of units is made there, by one CTA
// ahead of the forward kernel: a scan over the sequences numbers their blocks, a
// scan over the blocks adds up their tiles, and a search for each CTA's share of
// the total gives where it starts.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdint>
#include <cstring>

#include "packed.h"
#include "packed_host.h"
#include "packed_seq.cuh"
#include "sm103_primitives.cuh"

namespace fa {

using namespace dev;

cudaError_t launch_packed_fwd(int d, const CUtensorMap* tm, const PackedFwd& p, cudaStream_t stream);

namespace {

__device__ __forceinline__ bool before(const PackedStart& a, const PackedStart& b) {
  return a.unit < b.unit || (a.unit == b.unit && a.tile < b.tile);
}

}  // namespace

__global__ void __launch_bounds__(kPlanThreads) fa_packed_plan_kernel(const PackedPlan p) {
  __shared__ long long s_warps[32];
  __shared__ long long s_carry;
  const int tid = threadIdx.x;
  pdl_trigger();
  pdl_wait();
  const int block = 2 * p.tile_tokens;
  // Entries of the sequences: [seq_base[b], seq_base[b + 1]) after those of the prefix.
  int own = 0;
  for (int b0 = 0; b0 < p.s.B; b0 += kPlanThreads) {
    const int b = b0 + tid;
    int n = 0;
    if (b < p.s.B) n = (load_seq(p.s, b).q_len + block - 1) / block;
    const int sum = (int)scan_block<long long>(n, s_warps);
    if (b < p.s.B) p.seq_base[b + 1] = own + sum;
    if (tid == kPlanThreads - 1) s_carry = own + sum;
    __syncthreads();
    own = (int)s_carry;
    __syncthreads();
  }
  if (tid == 0) p.seq_base[0] = 0;
  // Blocks over the prefix alone: all rows from the first sequence's first to
  // the last one's last, whatever sequence they are of.
  int first = 0, over = 0, rows = 0;
  if (p.shared) {
    first = min(max(p.s.cu_q[0], 0), p.s.Tq);
    rows = max(0, min(p.s.cu_q[p.s.B], p.s.Tq) - first);
    over = (rows + block - 1) / block;
  }
  const int entries = over + own;
  __syncthreads();  // seq_base
  long long total = 0;
  for (int e0 = 0; e0 < entries; e0 += kPlanThreads) {
    const int e = e0 + tid;
    long long places = 0;
    if (e < entries) {
      PackedEntry x;
      if (e < over) {
        x = PackedEntry{first + e * block, min(block, rows - e * block), 0, 0, p.prefix_tiles, p.prefix_tiles, 0, 1};
      } else {
        const int i = e - over;
        const int lo = seq_of(p.seq_base, p.s.B, i);
        const Seq s = load_seq(p.s, lo);
        const int t0 = (i - p.seq_base[lo]) * block;
        x.q_row = s.q + t0;
        x.q_len = min(block, s.q_len - t0);
        x.k_row = s.k;
        x.k_len = s.k_len;
        x.prefix = p.shared ? 0 : p.prefix_tiles;
        x.pos = t0 + (p.s.causal == FA_CAUSAL_BOTTOM_RIGHT ? s.k_len - s.q_len : 0);
        const int seen = p.s.causal == FA_CAUSAL_NONE ? s.k_len : min(s.k_len, max(0, x.pos + x.q_len));
        x.tiles = x.prefix + (seen + kTileN - 1) / kTileN;
        x.kind = 0;
      }
      p.entries[e] = x;
      places = x.tiles + kUnitTiles;
    }
    const long long sum = scan_block<long long>(places, s_warps);
    if (e < entries) p.cum[e + 1] = total + sum;
    if (tid == kPlanThreads - 1) s_carry = total + sum;
    __syncthreads();
    total = s_carry;
    __syncthreads();
  }
  if (tid == 0) {
    p.cum[0] = 0;
    p.header[0] = entries;
    p.header[1] = over;
  }
  __syncthreads();
  for (int c = tid; c <= p.grid; c += kPlanThreads) {
    PackedStart s{0, 0};
    if (c == p.grid) {
      s.unit = p.head_groups * entries;
    } else if (total > 0) {
      const long long at = total * p.head_groups / p.grid * c + total * p.head_groups % p.grid * c / p.grid;
      const int hg = (int)(at / total);
      const long long r = at - hg * total;
      int lo = 0, hi = entries;  // cum[lo] <= r < cum[hi]
      while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (p.cum[mid] <= r) lo = mid; else hi = mid;
      }
      int x = (int)(r - p.cum[lo]);
      const int n = (int)(p.cum[lo + 1] - p.cum[lo]) - kUnitTiles;
      if (p.whole)
        x = 2 * x < n + kUnitTiles ? 0 : n;
      else if (x < p.min_tiles)
        x = 0;
      if (x > n - (p.whole ? 1 : p.min_tiles) && x > 0) {
        ++lo;
        x = 0;
      }
      s.unit = hg * entries + lo;
      s.tile = x;
    }
    p.starts[c] = s;
  }
}

// Partial results of a unit, merged for one row and 16 channels at a time:
// L = log sum exp(L_s), O = sum exp(L_s - L) O_s.
namespace {

struct Merge {
  float m, tot;
  float acc[16];
  __device__ __forceinline__ Merge() : m(-INFINITY), tot(0.f) {
#pragma unroll
    for (int i = 0; i < 16; ++i) acc[i] = 0.f;
  }
  // A part with logsumexp ls whose 16 channels are float4s `step` apart.
  __device__ __forceinline__ void add(float ls, const float4* o, size_t step) {
    if (ls == -INFINITY) return;
    float4 v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = o[i * step];
    const float m_new = fmaxf(m, ls);
    const float keep = m == -INFINITY ? 0.f : exp2f((m - m_new) * 1.4426950408889634f);
    const float wgt = exp2f((ls - m_new) * 1.4426950408889634f);
    m = m_new;
    tot = tot * keep + wgt;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      acc[4 * i] = acc[4 * i] * keep + wgt * v[i].x;
      acc[4 * i + 1] = acc[4 * i + 1] * keep + wgt * v[i].y;
      acc[4 * i + 2] = acc[4 * i + 2] * keep + wgt * v[i].z;
      acc[4 * i + 3] = acc[4 * i + 3] * keep + wgt * v[i].w;
    }
  }
};

// The parts of `unit` in slots: its first CTA is c (which holds its tile 0).
template <int D>
__device__ __forceinline__ void add_slots(const PackedFwd& p, const PackedStart* starts, Merge& m, int unit, int c, int row,
                                          int c16) {
  int slot = 2 * c + 1;
  while (true) {
    const float4* o = reinterpret_cast<const float4*>(p.o_slot) + ((size_t)slot * (D / 4) + 4 * c16) * kSlotRows + row;
    m.add(p.lse_slot[(size_t)slot * kSlotRows + row], o, kSlotRows);
    // The next CTA that starts within the unit and has some of it.
    do {
      ++c;
      if (c >= p.grid || starts[c].unit != unit || starts[c].tile == 0) return;
    } while (starts[c + 1].unit == unit && starts[c + 1].tile == starts[c].tile);
    slot = 2 * c;
  }
}

template <int D>
__device__ __forceinline__ void write_row(const PackedFwd& p, const Merge& m, int token, int head, int c16) {
  const float inv = m.tot > 0.f ? 1.0f / m.tot : 0.f;
  uint32_t w[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) w[i] = pack_bf16(m.acc[2 * i] * inv, m.acc[2 * i + 1] * inv);
  uint4* dst = reinterpret_cast<uint4*>(reinterpret_cast<__nv_bfloat16*>(p.o) + token * p.o_row + head * p.o_head + 16 * c16);
  dst[0] = make_uint4(w[0], w[1], w[2], w[3]);
  dst[1] = make_uint4(w[4], w[5], w[6], w[7]);
  if (c16 == 0) p.lse[(size_t)head * p.Tq + token] = m.tot > 0.f ? m.m + logf(m.tot) : -INFINITY;
}

// Query token and head of row r of a block's tile; false if it is none of them.
__device__ __forceinline__ bool row_of(const PackedFwd& p, const PackedEntry& e, int hg, int r, int* token, int* head) {
  const int tile = r / kTileM, rr = r % kTileM;
  const int tok = rr / p.group_heads, gh = rr - tok * p.group_heads;
  const int hk = hg / p.chunks, g = (hg % p.chunks) * p.group_heads + gh;
  const int j = tile * p.tile_tokens + tok;
  *token = e.q_row + j;
  *head = hk * p.group + g;
  return tok < p.tile_tokens && j < e.q_len && g < p.group;
}

}  // namespace

// Units that were cut: one for each CTA that starts within a unit that no CTA
// before it starts within.
template <int D>
__global__ void __launch_bounds__(256) fa_packed_merge_kernel(const PackedFwd p) {
  pdl_wait();
  const int c = blockIdx.x + 1;
  const PackedStart s = p.starts[c], before_s = p.starts[c - 1];
  if (s.tile == 0 || (before_s.unit == s.unit && before_s.tile > 0)) return;
  const int entries = p.header[0];
  const int hg = s.unit / entries;
  const PackedEntry e = p.entries[s.unit - hg * entries];
  for (int i = blockIdx.y * 256 + threadIdx.x; i < kSlotRows * (D / 16); i += 256 * gridDim.y) {
    const int row = i % kSlotRows, c16 = i / kSlotRows;
    int token, head;
    if (!row_of(p, e, hg, row, &token, &head)) continue;
    Merge m;
    add_slots<D>(p, p.starts, m, s.unit, c - 1, row, c16);
    write_row<D>(p, m, token, head, c16);
  }
}

// The last CTA that starts at or before the unit's first tile.
__device__ __forceinline__ int first_cta(const PackedStart* starts, int grid, int unit) {
  const PackedStart want{unit, 0};
  int lo = 0, hi = grid;
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (before(want, starts[mid])) hi = mid; else lo = mid;
  }
  return lo;
}

// All rows of the sequences, each from its part over the prefix and its part
// over the sequence's own keys (one row each where the unit was not cut).  A
// thread takes 16 channels of a row; rows are taken token by token, so that the
// threads of a CTA are of few units and find them in the same places.
constexpr int kJoinStarts = 320;  // CTAs' starts kept in shared memory
template <int D>
__global__ void __launch_bounds__(256) fa_packed_join_kernel(const PackedFwd p) {
  __shared__ PackedStart s_starts[kJoinStarts];
  pdl_wait();
  const PackedStart* starts = p.starts;
  if (p.grid < kJoinStarts) {
    for (int i = threadIdx.x; i <= p.grid; i += 256) s_starts[i] = p.starts[i];
    starts = s_starts;
  }
  const int entries = p.header[0], over = p.header[1];
  __syncthreads();
  if (over == 0 || entries == over) return;
  const int block = 2 * p.tile_tokens;
  const int q0 = p.entries[0].q_row;
  const int rows = p.entries[over - 1].q_row + p.entries[over - 1].q_len - q0;
  constexpr int kPer = D / 16;
  const long long tasks = (long long)rows * p.H * kPer;
  for (long long i = (long long)blockIdx.x * 256 + threadIdx.x; i < tasks; i += 256LL * gridDim.x) {
    const int c16 = (int)(i % kPer);
    const long long r = i / kPer;
    const int at = (int)(r / p.H), head = (int)(r - (long long)at * p.H);
    const int token = q0 + at;
    // The own block: the last that starts at or before the token.  (A token of no
    // sequence is behind that block's last.)
    int lo = over, hi = entries;
    while (hi - lo > 1) {
      const int mid = (lo + hi) / 2;
      if (p.entries[mid].q_row <= token) lo = mid; else hi = mid;
    }
    const int tok = token - p.entries[lo].q_row;
    if (tok < 0 || tok >= p.entries[lo].q_len) continue;
    const int hk = head / p.group, g = head - hk * p.group;
    const int hg = hk * p.chunks + g / p.group_heads, gh = g % p.group_heads;
    const int pe = at / block, ptok = at - pe * block;
    Merge m;
    for (int part = 0; part < 2; ++part) {
      const int unit = hg * entries + (part ? lo : pe), t = part ? tok : ptok;
      const int c = first_cta(starts, p.grid, unit);
      if (starts[c + 1].unit == unit && starts[c + 1].tile > 0) {
        const int row = t / p.tile_tokens * kTileM + t % p.tile_tokens * p.group_heads + gh;
        add_slots<D>(p, starts, m, unit, c, row, c16);
      } else {
        const float4* o = reinterpret_cast<const float4*>(p.o_part + (((size_t)part * p.Tq + token) * p.H + head) * D) + 4 * c16;
        m.add(p.lse_part[((size_t)part * p.H + head) * p.Tq + token], o, 1);
      }
    }
    write_row<D>(p, m, token, head, c16);
  }
}

}  // namespace fa

namespace {

using fa::PackedFwd;
using fa::PackedPlan;
using namespace fa::packed_host;

struct Call {
  int d;
  PackedPlan plan;
  PackedFwd p;
  CUtensorMap tm[6];
  int join_grid;
  cudaStream_t st;
};

cudaError_t run_plan(void* ctx) {
  const Call& c = *static_cast<const Call*>(ctx);
  return fa::launch_pdl(fa::fa_packed_plan_kernel, dim3(1), dim3(fa::kPlanThreads), 0, c.st, c.plan);
}
cudaError_t run_fwd(void* ctx) {
  const Call& c = *static_cast<const Call*>(ctx);
  return fa::launch_packed_fwd(c.d, c.tm, c.p, c.st);
}
template <int D>
cudaError_t merge_t(const Call& c) {
  if (c.p.shared)
    return fa::launch_pdl(fa::fa_packed_join_kernel<D>, dim3(c.join_grid), dim3(256), 0, c.st, c.p);
  return fa::launch_pdl(fa::fa_packed_merge_kernel<D>, dim3(c.p.grid - 1, D / 16), dim3(256), 0, c.st, c.p);
}
cudaError_t run_merge(void* ctx) {
  const Call& c = *static_cast<const Call*>(ctx);
  return c.d == 64 ? merge_t<64>(c) : c.d == 96 ? merge_t<96>(c) : merge_t<128>(c);
}

// Queries: [channel, head of the group, token, key/value head].
int encode_queries(CUtensorMap* m, const fa_rows_t* r, int rows, int heads, int group, int d, int box_heads, int box_rows) {
  const uint64_t rs = step_bytes(r->row_stride, rows), hs = step_bytes(r->head_stride, heads);
  const uint64_t dims[4] = {(uint64_t)d, (uint64_t)group, (uint64_t)rows, (uint64_t)(heads / group)};
  const uint64_t strides[3] = {hs, rs, hs * group};
  const uint32_t box[4] = {64, (uint32_t)box_heads, (uint32_t)box_rows, 1};
  return fa::internal_encode_tiled(m, r->ptr, 4, dims, strides, box);
}

// Kernels are loaded at their first use; those of a head dim all before the
// first of them runs, so that nothing is loaded behind kernels in flight.
template <int D>
cudaError_t load_t() {
  cudaFuncAttributes a;
  cudaError_t e = cudaFuncGetAttributes(&a, fa::fa_packed_merge_kernel<D>);
  if (e == cudaSuccess) e = cudaFuncGetAttributes(&a, fa::fa_packed_join_kernel<D>);
  if (e == cudaSuccess) e = cudaFuncGetAttributes(&a, fa::fa_packed_plan_kernel);
  return e;
}
cudaError_t load(int d) {
  constexpr int kMaxDevices = 64;
  static std::atomic<unsigned> loaded[kMaxDevices];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess || dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
  const unsigned bit = 1u << (d / 32);
  if (loaded[dev].load(std::memory_order_relaxed) & bit) return cudaSuccess;
  e = d == 64 ? load_t<64>() : d == 96 ? load_t<96>() : load_t<128>();
  if (e == cudaSuccess) loaded[dev].fetch_or(bit, std::memory_order_relaxed);
  return e;
}

int forward(const fa_rows_t* q, const fa_rows_t* kp, const fa_rows_t* vp, const fa_rows_t* k, const fa_rows_t* v,
            const fa_rows_t* o, float* lse, const int* cu_q, const int* cu_k, const int* used_k, int B, int P, int Tq,
            int Tk, int H, int Hkv, int d, int causal, float scale, void* stream) {
  if (B < 1 || Tq < 1 || Tk < 0 || P < 0 || H < 1 || Hkv < 1 || H % Hkv != 0 || B > kMost || Tq > kMost || Tk > kMost ||
      P > kMost)
    return FA_ERR_INVALID_ARG;
  if (!head_dim(d)) return FA_ERR_UNSUPPORTED;
  if (causal < FA_CAUSAL_NONE || causal > FA_CAUSAL_BOTTOM_RIGHT) return FA_ERR_INVALID_ARG;
  if (!(std::isfinite(scale) && scale > 0.f)) return FA_ERR_INVALID_ARG;
  if (!rows_ok(q, Tq, H) || !rows_ok(o, Tq, H) || !rows_apart(o, Tq, H, d)) return FA_ERR_INVALID_ARG;
  if (Tk > 0 && (!rows_ok(k, Tk, Hkv) || !rows_ok(v, Tk, Hkv))) return FA_ERR_INVALID_ARG;
  if (P > 0 && (!rows_ok(kp, P, Hkv) || !rows_ok(vp, P, Hkv))) return FA_ERR_INVALID_ARG;
  if (!array_ok(lse, 16) || !array_ok(cu_q, 4) || !array_ok(cu_k, 4) || (used_k != nullptr && !array_ok(used_k, 4)))
    return FA_ERR_INVALID_ARG;

  Call c;
  std::memset(&c, 0, sizeof(c));
  PackedFwd& p = c.p;
  PackedPlan& pl = c.plan;
  p.H = H;
  p.Hkv = Hkv;
  p.group = H / Hkv;
  p.group_heads = std::min(p.group, fa::kTileM);
  p.chunks = (p.group + p.group_heads - 1) / p.group_heads;
  p.tile_tokens = fa::kTileM / p.group_heads;
  const int block = 2 * p.tile_tokens;
  const long long hgs = (long long)Hkv * p.chunks;
  const int prefix_tiles = (P + fa::kTileN - 1) / fa::kTileN;
  const long long own_most = Tq / block + (long long)std::min(B, Tq);

  unsigned int* status = nullptr;
  int sm_count = 0;
  int e = fa::internal_device_setup(&status, &sm_count);
  if (e) return e;

  // Blocks of their own over the prefix pay where the sequences' blocks are not
  // full: half a block each, on average, would walk the prefix for nothing.  They
  // cost a second partial result of every row, written and read in fp32.
  if (prefix_tiles > 0) {
    const double step_us = 1.4 * d / 128;  // a block's key tile
    const double spared = 0.5 * std::min(B, Tq) * prefix_tiles * hgs / sm_count * step_us;
    const double parts_us = 16.0 * Tq * H * d / 6.8e6 + 3.0;
    p.shared = spared > parts_us ? 1 : 0;
  }
  const long long entries = own_most + (p.shared ? Tq / block + 1 : 0);
  if (entries * hgs > 0x7fffffffLL) return FA_ERR_INVALID_ARG;
  const long long key_tiles = prefix_tiles + (Tk + fa::kTileN - 1) / fa::kTileN;
  pl.min_tiles = 2;
  pl.whole = key_tiles <= 4 && !p.shared ? 1 : 0;
  p.grid = (int)std::min<long long>(sm_count, entries * hgs * (pl.whole ? 1 : std::max(1LL, key_tiles / pl.min_tiles)));

  // Workspace: the list, then partial results.
  const size_t n_entries = up((size_t)entries * sizeof(fa::PackedEntry));
  const size_t n_cum = up((size_t)(entries + 1) * sizeof(long long));
  const size_t n_base = up(((size_t)B + 1) * sizeof(int));
  const size_t n_starts = up(((size_t)p.grid + 1) * sizeof(fa::PackedStart) + 2 * sizeof(int));
  const bool cuts = !pl.whole && p.grid > 1;
  const size_t slot_rows = cuts ? (size_t)2 * p.grid * fa::kSlotRows : 0;
  const size_t part_rows = p.shared ? (size_t)2 * Tq * H : 0;
  const size_t bytes = n_entries + n_cum + n_base + n_starts + up(slot_rows * (d + 1) * 4) + part_rows * (d + 1) * 4;
  c.st = static_cast<cudaStream_t>(stream);
  c.d = d;

  const fa_rows_t* kk = Tk > 0 ? k : q;  // never read without keys
  const fa_rows_t* vv = Tk > 0 ? v : q;
  const int own_rows = Tk > 0 ? Tk : 1;
  if (encode_queries(&c.tm[0], q, Tq, H, p.group, d, p.group_heads, p.tile_tokens) ||
      encode_tile(&c.tm[1], kk, own_rows, Hkv, d, 128) || encode_tile(&c.tm[2], vv, own_rows, Hkv, d, 128))
    return FA_ERR_CUDA;
  c.tm[3] = c.tm[1];
  c.tm[4] = c.tm[2];
  if (P > 0 && (encode_plain(&c.tm[3], kp, P, Hkv, d) || encode_plain(&c.tm[4], vp, P, Hkv, d))) return FA_ERR_CUDA;

  if (load(d) != cudaSuccess) {
    cudaGetLastError();
    return FA_ERR_CUDA;
  }
  // A warp's 32 rows of O are a box of tokens and heads where the heads divide 32.
  c.tm[5] = c.tm[0];
  if (32 % p.group_heads == 0) {
    p.tile_store = 1;
    if (encode_queries(&c.tm[5], o, Tq, H, p.group, d, p.group_heads, 32 / p.group_heads)) return FA_ERR_CUDA;
  }
  void* ws = nullptr;
  if (fa::internal_workspace(&ws, bytes, c.st) != cudaSuccess) {
    cudaGetLastError();
    return FA_ERR_NO_MEMORY;
  }
  char* at = static_cast<char*>(ws);
  pl.entries = reinterpret_cast<fa::PackedEntry*>(at);
  pl.cum = reinterpret_cast<long long*>(at += n_entries);
  pl.seq_base = reinterpret_cast<int*>(at += n_cum);
  pl.starts = reinterpret_cast<fa::PackedStart*>(at += n_base);
  pl.header = reinterpret_cast<int*>(pl.starts + p.grid + 1);
  at += n_starts;
  if (slot_rows > 0) {
    p.o_slot = reinterpret_cast<float*>(at);
    p.lse_slot = p.o_slot + slot_rows * d;
    at += up(slot_rows * (d + 1) * 4);
  }
  if (part_rows > 0) {
    p.o_part = reinterpret_cast<float*>(at);
    p.lse_part = p.o_part + part_rows * d;
  }
  pl.s = fa::PackedSeqs{cu_q, cu_k, used_k, B, Tq, Tk, causal, status};
  pl.tile_tokens = p.tile_tokens;
  pl.prefix_tiles = prefix_tiles;
  pl.shared = p.shared;
  pl.head_groups = (int)hgs;
  pl.grid = p.grid;
  p.Tq = Tq;
  p.prefix_len = P;
  p.causal = causal != FA_CAUSAL_NONE ? 1 : 0;
  p.scale_log2 = scale * 1.4426950408889634f;
  p.entries = pl.entries;
  p.starts = pl.starts;
  p.header = pl.header;
  p.o = o->ptr;
  p.o_row = Tq > 1 ? o->row_stride : 0;
  p.o_head = H > 1 ? o->head_stride : 0;
  p.lse = lse;
  p.store32 = aligned32(o->ptr, p.o_row, p.o_head) ? 1 : 0;
  p.status = status;
  p.timeout_ns = fa::internal_wait_timeout_ns();
  c.join_grid = (int)std::min<long long>(((long long)Tq * H * (d / 16) + 255) / 256, 8LL * sm_count);

  cudaError_t ce = fa::internal_timed_launch(FA_KERNEL_PACKED_PLAN, c.st, run_plan, &c);
  if (ce == cudaSuccess) ce = fa::internal_timed_launch(FA_KERNEL_PACKED_FWD, c.st, run_fwd, &c);
  if (ce == cudaSuccess && (cuts || p.shared)) ce = fa::internal_timed_launch(FA_KERNEL_PACKED_MERGE, c.st, run_merge, &c);
  cudaFreeAsync(ws, c.st);
  return ce == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

}  // namespace

extern "C" {

int fa_packed_fwd(const fa_rows_t* q, const fa_rows_t* k, const fa_rows_t* v, const fa_rows_t* o, float* lse,
                  const int* cu_q, const int* cu_k, const int* used_k, int B, int Tq, int Tk, int H, int Hkv, int d,
                  int causal, float scale, void* stream) {
  return forward(q, nullptr, nullptr, k, v, o, lse, cu_q, cu_k, used_k, B, 0, Tq, Tk, H, Hkv, d, causal, scale, stream);
}

int fa_prefix_fwd(const fa_rows_t* q, const fa_rows_t* k_prefix, const fa_rows_t* v_prefix, const fa_rows_t* k,
                  const fa_rows_t* v, const fa_rows_t* o, float* lse, const int* cu_q, const int* cu_k,
                  const int* used_k, int B, int P, int Tq, int Tk, int H, int Hkv, int d, int causal, float scale,
                  void* stream) {
  if (P < 1) return FA_ERR_INVALID_ARG;
  return forward(q, k_prefix, v_prefix, k, v, o, lse, cu_q, cu_k, used_k, B, P, Tq, Tk, H, Hkv, d, causal, scale, stream);
}

}  // extern "C"
