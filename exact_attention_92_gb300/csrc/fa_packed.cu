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

cudaError_t load_packed_fwd(int d);
cudaError_t launch_packed_fwd(int d, const CUtensorMap* tm, const PackedFwd& p, cudaStream_t stream);

namespace {

__device__ __forceinline__ bool before(const PackedStart& a, const PackedStart& b) {
  return a.unit < b.unit || (a.unit == b.unit && a.tile < b.tile);
}

}  // namespace

// Sequences and entries up to this number have their places in shared memory.
constexpr int kPlanShared = 1024;

// Where the CTAs' stretches start, once the entries' places are summed up: cum[e]
// is what lies ahead of entry e, the small blocks' behind the whole ones'.  T: an
// unsigned word where the places of all head groups fit, else 64 bits, whose
// divisions take 2000 cycles more.
template <typename T>
__device__ __forceinline__ void plan_starts(const PackedPlan& p, const long long* cum, const int (&entries)[2]) {
  const int tid = threadIdx.x;
  const T total[2] = {(T)cum[entries[0]], (T)(cum[entries[0] + entries[1]] - cum[entries[0]])};
  // Place `at` of a list as unit and tile.  A cut near a unit's border moves there.
  auto locate = [&](int list, T at) -> PackedStart {
    const T all = list ? total[1] : total[0];
    const int n_entries = list ? entries[1] : entries[0], base = list ? entries[0] : 0;
    if (at >= all * (T)p.head_groups) return PackedStart{p.head_groups * n_entries, 0};
    const int hg = (int)(at / all);
    const long long r = (long long)(at - (T)hg * all) + cum[base];
    int lo = base, hi = base + n_entries;  // cum[lo] <= r < cum[hi]
    while (hi - lo > 1) {
      const int mid = (lo + hi) / 2;
      if (cum[mid] <= r) lo = mid; else hi = mid;
    }
    const int size = (int)(cum[lo + 1] - cum[lo]), in = (int)(r - cum[lo]);
    const int n = (size - unit_places(list)) / tile_places(list);
    int x = in / tile_places(list);
    const int least = p.whole ? n + 1 : least_tiles(list);
    if (x < least && 2 * in < size) x = 0;
    else if (x < least || x > n - least) x = 0, ++lo;
    return PackedStart{hg * n_entries + lo - base, x};
  };
  const T whole = total[0] * (T)p.head_groups, all = whole + total[1] * (T)p.head_groups;
  // A CTA that takes of both lists fills its pipeline twice (10 to 25 us more at
  // d = 128), and a pair of SMs that runs both slows down: pairs of CTAs take one
  // list where that makes no stretch longer by a 16th.
  const int apart = all > 0 ? 2 * (int)((float)whole / (float)all * 0.5f * (float)p.grid + 0.5f) : 0;
  const int behind = p.grid - apart;
  const T even = all / (T)p.grid;
  const bool split = whole > 0 && all > whole && apart > 0 && behind > 0 &&
                     max(whole / (T)apart, (all - whole) / (T)behind) <= even + even / 16;
  auto part = [](T sum, T n, T c) { return sum / n * c + sum % n * c / n; };
  auto edge = [&](int c) -> T {
    if (c >= p.grid) return all;
    if (!split) return part(all, p.grid, c);
    return c < apart ? part(whole, apart, c) : whole + part(all - whole, behind, c - apart);
  };
  auto behind_whole = [&](T x) { return x > whole ? x - whole : T(0); };
  for (int i = tid; i < 3 * p.grid + 2; i += kPlanThreads) {
    if (i <= p.grid) {
      p.starts[kWhole][i] = locate(kWhole, min(edge(i), whole));
    } else {
      const int v = i - p.grid - 1;
      const T a = behind_whole(edge(v / 2)), b = behind_whole(edge(v / 2 + 1));
      p.starts[kSmall][v] = locate(kSmall, v & 1 ? a + (b - a) / 2 : a);
    }
  }
}

__global__ void __launch_bounds__(kPlanThreads) fa_packed_plan_kernel(const PackedPlan p) {
  __shared__ long long s_warps[2][32];
  __shared__ int s_starts[2][32];
  __shared__ Seq s_seq[kPlanShared];
  __shared__ int s_base[2][kPlanShared + 1];
  __shared__ long long s_cum[kPlanShared + 1];
  __shared__ int s_span[2];  // the first and the end of the rows that sequences have
  const int tid = threadIdx.x;
  pdl_trigger();
  pdl_wait();
  const int block = 2 * p.tile_tokens;
  const bool few = p.s.B <= kPlanShared;
  if (tid == 0) s_span[0] = p.s.Tq, s_span[1] = 0;
  int from = p.s.Tq, to = 0;  // of this thread's sequences
  int* const base0 = few ? s_base[0] : p.seq_base[0];
  int* const base1 = few ? s_base[1] : p.seq_base[1];
  Scan<long long> scan(s_warps);
  Scan<int, true> furthest(s_starts);
  // Entries of the sequences, by list: [base[b], base[b + 1]).  Both numbers in one sum.
  long long own = 0, more;
  int first_q = 0, next_q;
  for (int b0 = 0; b0 < p.s.B; b0 += kPlanThreads) {
    const int b = b0 + tid;
    long long n = 0;
    const int at_q = max(first_q, furthest(b < p.s.B ? start_of(p.s.cu_q, b, p.s.Tq) : 0, &next_q));
    first_q = max(first_q, next_q);
    if (b < p.s.B) {
      const Seq s = load_seq(p.s, b, at_q);
      if (few) s_seq[b] = s;
      if (s.q_len > 0) from = min(from, s.q), to = max(to, s.q + s.q_len);
      const int2 blocks = blocks_of(s, p.tile_tokens);
      n = ((long long)blocks.y << 32) + blocks.x;
    }
    const long long sum = own + scan(n, &more);
    if (b < p.s.B) {
      base0[b + 1] = (int)(sum & 0xffffffffLL);
      base1[b + 1] = (int)(sum >> 32);
    }
    own += more;
  }
  if (tid == 0) base0[0] = base1[0] = 0;
  // Blocks over the prefix alone: all rows from the first sequence's first to the
  // last one's last, whatever sequence they are of.  (Of those that were not skipped:
  // cu_q[0] or cu_q[B] may be the bound that is out of order.)
  int first = 0, rows = 0;
  if (p.shared) {
    from = __reduce_min_sync(0xffffffffu, from);
    to = __reduce_max_sync(0xffffffffu, to);
    if ((tid & 31) == 0 && from < to) {
      atomicMin(&s_span[0], from);
      atomicMax(&s_span[1], to);
    }
    __syncthreads();
    first = s_span[0];
    rows = max(0, s_span[1] - first);
  }
  const int rest = rows % block;
  int over[2], entries[2];
  over[kWhole] = rows / block + (rest > p.tile_tokens);
  over[kSmall] = rest > 0 && rest <= p.tile_tokens;
  entries[kWhole] = over[kWhole] + (int)(own & 0xffffffffLL);
  entries[kSmall] = over[kSmall] + (int)(own >> 32);
  const int both = entries[kWhole] + entries[kSmall];
  long long* const cum = both <= kPlanShared ? s_cum : p.cum;
  __syncthreads();  // base
  long long places_all = 0;
  for (int e0 = 0; e0 < both; e0 += kPlanThreads) {
    const int at = e0 + tid;
    long long places = 0;
    if (at < both) {
      const int list = at >= entries[kWhole];
      const int e = list ? at - entries[kWhole] : at, n_over = list ? over[kSmall] : over[kWhole];
      PackedEntry x;
      if (e < n_over) {
        const int t0 = (list ? over[kWhole] : e) * block;
        x = PackedEntry{first + t0, min(block, rows - t0), 0, 0, p.prefix_tiles, p.prefix_tiles, 0, 1};
      } else {
        const int* base = list ? base1 : base0;
        const int i = e - n_over;
        const int b = seq_of(base, p.s.B, i);
        const Seq s = few ? s_seq[b] : load_seq(p.s, b, 0);  // (one with blocks is in order)
        const int t0 = (list ? base0[b + 1] - base0[b] : i - base[b]) * block;
        x = block_at(s, t0, block, p.shared ? 0 : p.prefix_tiles, p.s.causal);
      }
      (list ? p.entries[kSmall] : p.entries[kWhole])[e] = x;
      places = (long long)x.tiles * tile_places(list) + unit_places(list);
    }
    const long long sum = places_all + scan(places, &more);
    if (at < both) cum[at + 1] = sum;
    places_all += more;
  }
  if (tid == 0) {
    cum[0] = 0;
    *p.header = PackedHeader{{entries[0], entries[1]}, {over[0], over[1]}, first, rows};
  }
  __syncthreads();  // cum
  if (places_all * p.head_groups < 0x7fffffffLL) plan_starts<unsigned>(p, cum, entries);
  else plan_starts<unsigned long long>(p, cum, entries);
}

// Partial results of a unit, merged for one row and 16 channels at a time:
// L = log sum exp(L_s), O = sum exp(L_s - L) O_s.  A part that holds NaN has L_s = NaN:
// the maximum passes over it (fmaxf), its weight and so the sum `tot` and O are NaN, and
// stay so.
namespace {

struct Merge {
  float m, tot;
  float acc[16];
  __device__ __forceinline__ Merge() : m(-INFINITY), tot(0.f) {
#pragma unroll
    for (int i = 0; i < 16; ++i) acc[i] = 0.f;
  }
  // A part with logsumexp ls; a row without keys has none, and nothing in v.
  __device__ __forceinline__ void add(float ls, const float4 (&v)[4]) {
    if (ls == -INFINITY) return;
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

// Rows of a slot of the list.
__device__ __forceinline__ int slot_rows(int list) { return list ? kSlotRows / 2 : kSlotRows; }
__device__ __forceinline__ int stretches(const PackedFwd& p, int list) { return list ? 2 * p.grid : p.grid; }

__device__ __forceinline__ bool same(const PackedStart& a, const PackedStart& b) {
  return a.unit == b.unit && a.tile == b.tile;
}

// Parts first, first + step, ... of `unit` in slots: its tile 0 is in stretch c, and
// each stretch that starts within the unit and has some of it (starts[0] is that
// of c) has a part.
template <int D>
__device__ __forceinline__ void add_slots(const PackedFwd& p, int list, const PackedStart* starts, Merge& m, int unit, int c,
                                          int first, int step, int row, int c16) {
  const int rows = slot_rows(list), left = stretches(p, list) - c;
  const float4* o = reinterpret_cast<const float4*>(p.o_slot[list]) + (size_t)4 * c16 * rows + row;
  const float* lse = p.lse_slot[list] + row;
  for (int k = first; k < left && (k == 0 || (starts[k].unit == unit && starts[k].tile > 0)); k += step) {
    if (k > 0 && same(starts[k], starts[k + 1])) continue;
    const size_t slot = k == 0 ? 2 * c + 1 : 2 * (c + k);
    float4 v[4];
#pragma unroll
    for (int x = 0; x < 4; ++x) v[x] = o[(slot * (D / 4) + x) * rows];
    m.add(lse[slot * rows], v);
  }
}

// Rows of a CTA of the merges: thread tid works on row tid % n_rows (a power of
// two), and where that leaves threads over, they take a share of the row's parts
// each: a step of one sequence over 128 Ki keys and 8 heads, cut in 300, took
// 112 us with one thread for 16 channels of a row, and 12 us so.
constexpr int kMergeThreads = 256;

struct MergeShared {
  float m[kMergeThreads], tot[kMergeThreads];
  float acc[kMergeThreads][17];
};

// Writes the CTA's rows; `shares` threads have parts of a row.
template <int D>
__device__ __forceinline__ void write_rows(const PackedFwd& p, MergeShared& sh, Merge& m, int n_rows, int shares, bool ok,
                                           int token, int head, int c16) {
  const int tid = threadIdx.x;
  if (shares > 1) {
    sh.m[tid] = m.m;
    sh.tot[tid] = m.tot;
#pragma unroll
    for (int i = 0; i < 16; ++i) sh.acc[tid][i] = m.acc[i];
    __syncthreads();
    // A halving of the shares at a time.
    int width = 1;
    while (width < shares) width *= 2;
    const int share = tid / n_rows;
    for (int half = width / 2; half > 0; half /= 2) {
      if (share < half && share + half < shares) {
        const int x = tid + half * n_rows;
        const float m_x = sh.m[x];
        if (sh.tot[x] != 0.f) {  // (0: it found no part; with m_x = -inf alone its parts may be NaN)
          const float m_new = fmaxf(m.m, m_x);
          const float keep = m.m == -INFINITY ? 0.f : exp2f((m.m - m_new) * 1.4426950408889634f);
          const float wgt = exp2f((m_x - m_new) * 1.4426950408889634f);
          m.m = m_new;
          m.tot = m.tot * keep + wgt * sh.tot[x];
#pragma unroll
          for (int i = 0; i < 16; ++i) m.acc[i] = m.acc[i] * keep + wgt * sh.acc[x][i];
          sh.m[tid] = m.m;
          sh.tot[tid] = m.tot;
#pragma unroll
          for (int i = 0; i < 16; ++i) sh.acc[tid][i] = m.acc[i];
        }
      }
      shares = min(shares, half);
      __syncthreads();
    }
    ok = ok && share == 0;
  }
  if (!ok) return;
  const float inv = m.tot == 0.f ? 0.f : 1.0f / m.tot;
  uint32_t w[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) w[i] = pack_bf16(m.acc[2 * i] * inv, m.acc[2 * i + 1] * inv);
  __nv_bfloat16* row = reinterpret_cast<__nv_bfloat16*>(p.o) + token * p.o_row + head * p.o_head;
  uint4* dst = reinterpret_cast<uint4*>(row + 16 * c16);
  dst[0] = make_uint4(w[0], w[1], w[2], w[3]);
  dst[1] = make_uint4(w[4], w[5], w[6], w[7]);
  if (c16 == 0) p.lse[(size_t)head * p.Tq + token] = m.tot == 0.f ? -INFINITY : m.m + logf(m.tot);
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

// What the plan wrote may be read ahead of the wait for the forward kernel: that
// lets its dependents start only once it has seen the plan.  (Past the L1 cache,
// which no launch has emptied for it.)
__device__ __forceinline__ PackedStart read_start(const PackedStart* s) {
  const int2 v = __ldcg(reinterpret_cast<const int2*>(s));
  return PackedStart{v.x, v.y};
}
__device__ __forceinline__ PackedEntry read_entry(const PackedEntry* e) {
  const int4 a = __ldcg(reinterpret_cast<const int4*>(e)), b = __ldcg(reinterpret_cast<const int4*>(e) + 1);
  return PackedEntry{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
}

// Units that were cut: one for each stretch that starts within a unit that no
// stretch before it starts within.  A CTA takes 16 channels of a unit, or all of
// a small block in few parts.
template <int D>
__global__ void __launch_bounds__(kMergeThreads, 4) fa_packed_merge_kernel(const PackedFwd p) {
  __shared__ PackedStart s_starts[2 * kMostGrid + 2];
  __shared__ MergeShared sh;
  __shared__ int s_parts;
  constexpr int kPer = D / 16;
  const int tid = threadIdx.x;
  const int list = (int)blockIdx.x >= p.grid - 1 ? kSmall : kWhole;
  const int c = (int)blockIdx.x - (list ? p.grid - 1 : 0);  // the unit starts in stretch c
  const PackedStart* starts = p.starts[list];
  const PackedStart before_s = read_start(starts + c), s = read_start(starts + c + 1);
  if (s.tile == 0 || (before_s.unit == s.unit && before_s.tile > 0)) {
    if (blockIdx.x == 0 && blockIdx.y == 0) pdl_wait();  // one waits: this grid does not end ahead of the one before it
    return;
  }
  const int end = stretches(p, list);
  if (tid == 0) s_parts = end - c;
  __syncthreads();
  for (int i = c + tid; i <= end; i += kMergeThreads) {
    const PackedStart x = read_start(starts + i);
    s_starts[i - c] = x;
    if (i > c && (x.unit != s.unit || x.tile == 0)) atomicMin(&s_parts, i - c);
  }
  const int entries = __ldcg(&p.header->entries[list]);
  const int hg = s.unit / entries;
  const PackedEntry e = read_entry(p.entries[list] + (s.unit - hg * entries));
  const int used = e.q_len > p.tile_tokens ? 2 * kTileM : e.q_len * p.group_heads;
  int n_rows = 1;
  while (n_rows < used) n_rows *= 2;
  __syncthreads();
  const bool few = s_parts <= 4;
  const bool all = list && few;
  if (all && blockIdx.y > 0) return;  // (the first of these waits)
  const int per = all ? min(kPer, kMergeThreads / n_rows) : 1;  // of 16 channels, at a time
  const int row = tid & (n_rows - 1), channels = tid / n_rows % per, share = tid / (n_rows * per);
  const int shares = few ? 1 : min(kMergeThreads / n_rows, s_parts);
  int token, head;
  const bool row_ok = row_of(p, e, hg, row, &token, &head) && share < shares;
  pdl_wait();
  for (int at = blockIdx.y; at < (all ? kPer : (int)blockIdx.y + 1); at += per) {
    const int c16 = at + channels;
    const bool ok = row_ok && c16 < kPer;
    Merge m;
    if (ok) add_slots<D>(p, list, s_starts, m, s.unit, c, share, shares, row, c16);
    write_rows<D>(p, sh, m, n_rows * per, shares, ok, token, head, c16);
    if (shares > 1) __syncthreads();  // sh
  }
}

// The last stretch that starts at or before the unit's first tile.
__device__ __forceinline__ int stretch_of(const PackedStart* starts, int number, int unit) {
  const PackedStart want{unit, 0};
  int lo = 0, hi = number;
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (before(want, starts[mid])) hi = mid; else lo = mid;
  }
  return lo;
}

// All rows of the sequences, each from its part over the prefix and its part
// over the sequence's own keys (one row each where the unit was not cut).  A
// CTA takes rows / H tokens at a time (or `rows` heads of one) and 16 channels,
// blockIdx.y; heads come first, so that a group's rows are read side by side.
template <int D>
__global__ void __launch_bounds__(kMergeThreads, 4) fa_packed_join_kernel(const PackedFwd p, int tokens, int n_rows) {
  __shared__ PackedStart s_starts[3 * kMostGrid + 2];
  __shared__ MergeShared sh;
  __shared__ int s_own[kMergeThreads];  // the token's own block: entry and list; -1: of no sequence
  __shared__ int s_row[kMergeThreads];  // and the block's first token
  const int tid = threadIdx.x;
  const int c16 = blockIdx.y;
  const int shares = kMergeThreads / n_rows, share = tid / n_rows;
  for (int i = tid; i < 3 * p.grid + 2; i += kMergeThreads)
    s_starts[i] = read_start(i <= p.grid ? p.starts[0] + i : p.starts[1] + (i - p.grid - 1));
  __shared__ PackedHeader h;
  static_assert(sizeof(PackedHeader) == 6 * sizeof(int), "copied as words");
  if (tid < 6) reinterpret_cast<int*>(&h)[tid] = __ldcg(reinterpret_cast<const int*>(p.header) + tid);
  __syncthreads();
  bool waited = false;
  const int block = 2 * p.tile_tokens;
  for (int at0 = blockIdx.x * tokens; at0 < h.rows; at0 += gridDim.x * tokens) {
    const int n = min(tokens, h.rows - at0), t0 = h.first + at0;
    if (tid < n) s_own[tid] = -1;
    __syncthreads();
    // Every thread looks whether an entry of its has one of the tokens.
#pragma unroll
    for (int list = 0; list < 2; ++list) {
      const PackedEntry* e = p.entries[list];
      int lo = h.over[list], hi = h.entries[list];
      while (hi - lo > 1024) {  // the entry of t0, if there is one, stays within [lo, hi)
        const int mid = (lo + hi) / 2;
        if (__ldcg(&e[mid].q_row) <= t0) lo = mid; else hi = mid;
      }
      hi = min(hi + n, h.entries[list]);
      for (int i = lo + tid; i < hi; i += kMergeThreads) {
        const int2 row_len = __ldcg(reinterpret_cast<const int2*>(e + i));
        const int a = max(row_len.x - t0, 0), b = min(row_len.x + row_len.y - t0, n);
        for (int x = a; x < b; ++x) {
          s_own[x] = 2 * i + list;
          s_row[x] = row_len.x;
        }
      }
    }
    __syncthreads();
    for (int r0 = 0; r0 < n * p.H; r0 += n_rows) {
      const int r = r0 + (tid & (n_rows - 1));
      const int x = r / p.H, head = r - x * p.H;
      const int at = at0 + x, token = t0 + x;
      const bool ok = x < n && s_own[x] >= 0;
      // Where the two parts are: in the slots from stretch c on, or as a row of their own (c < 0).
      int c[2] = {-1, -1}, unit[2], row[2];
      const int own_list = ok ? s_own[x] & 1 : 0;
      const int over_list = at / block >= h.over[kWhole];
      if (ok) {
        const int own = s_own[x] >> 1;
        const int hk = head / p.group, g = head - hk * p.group;
        const int hg = hk * p.chunks + g / p.group_heads, gh = g % p.group_heads;
#pragma unroll
        for (int part = 0; part < 2; ++part) {
          const int list = part ? own_list : over_list;
          const int e = part ? own : list ? 0 : at / block;
          const int t = part ? token - s_row[x] : at % block;
          unit[part] = hg * h.entries[list] + e;
          row[part] = t / p.tile_tokens * kTileM + t % p.tile_tokens * p.group_heads + gh;
          const PackedStart* starts = s_starts + (list ? p.grid + 1 : 0);
          const int at_c = stretch_of(starts, stretches(p, list), unit[part]);
          const PackedStart next = starts[at_c + 1];
          if (next.unit == unit[part] && next.tile > 0) c[part] = at_c;
        }
      }
      if (!waited) pdl_wait();
      waited = true;
      Merge m;
      if (ok) {
#pragma unroll
        for (int part = 0; part < 2; ++part) {
          const int list = part ? own_list : over_list;
          const int turn = part ? shares - 1 - share : share;  // the prefix's parts from the first share on
          if (c[part] >= 0) {
            const PackedStart* starts = s_starts + (list ? p.grid + 1 : 0);
            add_slots<D>(p, list, starts + c[part], m, unit[part], c[part], turn, shares, row[part], c16);
          } else if (turn == 0) {
            const float* rows = p.o_part + (((size_t)part * p.Tq + token) * p.H + head) * D;
            const float4* o = reinterpret_cast<const float4*>(rows) + 4 * c16;
            const float4 v[4] = {o[0], o[1], o[2], o[3]};
            m.add(p.lse_part[((size_t)part * p.H + head) * p.Tq + token], v);
          }
        }
      }
      write_rows<D>(p, sh, m, n_rows, shares, ok, token, head, c16);
      if (shares > 1) __syncthreads();  // sh
    }
    __syncthreads();  // s_own
  }
  if (!waited) pdl_wait();
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
  int join_grid, join_tokens, join_rows;
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
  const dim3 block(fa::kMergeThreads);
  if (c.p.shared)
    return fa::launch_pdl(fa::fa_packed_join_kernel<D>, dim3(c.join_grid, D / 16), block, 0, c.st, c.p, c.join_tokens,
                          c.join_rows);
  return fa::launch_pdl(fa::fa_packed_merge_kernel<D>, dim3(3 * c.p.grid - 2, D / 16), block, 0, c.st, c.p);
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
  if (e == cudaSuccess) e = fa::load_packed_fwd(d);
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
  // cost a second partial result of every row, written and read in fp32.  (A block's
  // key tile takes 1.4 us at d = 128, and 1.3 and 1.2 at 96 and 64, where the rule
  // reckons with 1.05 and 0.7: there it shares later than these steps ask for.)
  if (prefix_tiles > 0) {
    const double step_us = 1.4 * d / 128;
    const double spared = 0.5 * std::min(B, Tq) * prefix_tiles * hgs / sm_count * step_us;
    const double parts_us = 16.0 * Tq * H * d / 6.8e6 + 3.0;
    p.shared = spared > parts_us ? 1 : 0;
  }
  const long long entries = own_most + (p.shared ? Tq / block + 1 : 0);
  if (entries * hgs > 0x7fffffffLL) return FA_ERR_INVALID_ARG;
  const long long key_tiles = prefix_tiles + (Tk + fa::kTileN - 1) / fa::kTileN;
  // Few keys of few sequences: each CTA finds its units itself, and none is cut, so
  // that the forward kernel is all there is.  One token, 8 key/value heads of d = 128:
  // 1 sequence of 1024, 1536, 2048 and 4096 keys 10.6, 13.3, 15.7 and 26 us, planned,
  // cut and merged 15.3, 15.1, 15.6 and 18; 4 of 1024 keys 11.1 and 19.8, 8 of 512 8.5
  // and 17.6; 4 prompts of 1024, 4 heads, 16.6 and 23.2.  (Of several sequences one may
  // have all the keys: 26 us in place of 18, at worst.)
  const bool direct = B <= fa::kDirectSeqs && key_tiles <= (std::min(B, Tq) > 1 ? 40 : 16) && !p.shared &&
                      entries * hgs <= 4LL * sm_count;
  // Of many sequences: no cuts (and no merge) where the cuts would be of single tiles.
  pl.whole = key_tiles <= 4 && !p.shared ? 1 : 0;
  const long long parts = pl.whole || direct ? 1 : std::max(1LL, key_tiles / fa::least_tiles(fa::kWhole));
  p.grid = (int)std::min<long long>(std::min(sm_count, fa::kMostGrid), entries * hgs * parts);

  // Workspace: the lists, then partial results.  Small blocks are the last of
  // their sequences (and one over the prefix).
  const long long small = (long long)std::min(B, Tq) + 1;
  const size_t n_entries[2] = {up((size_t)entries * sizeof(fa::PackedEntry)), up((size_t)small * sizeof(fa::PackedEntry))};
  const size_t n_cum = up((size_t)(entries + small + 1) * sizeof(long long));
  const size_t n_base = up(((size_t)B + 1) * sizeof(int));
  const size_t n_starts[2] = {up(((size_t)p.grid + 1) * sizeof(fa::PackedStart)),
                              up(((size_t)2 * p.grid + 1) * sizeof(fa::PackedStart))};
  const bool cuts = !pl.whole && !direct;
  size_t slot_rows[2] = {0, 0};
  if (cuts) {
    slot_rows[0] = (size_t)2 * p.grid * fa::kSlotRows;
    slot_rows[1] = (size_t)4 * p.grid * (fa::kSlotRows / 2);
  }
  const size_t part_rows = p.shared ? (size_t)2 * Tq * H : 0;
  const size_t bytes = n_entries[0] + n_entries[1] + n_cum + 2 * n_base + n_starts[0] + n_starts[1] +
                       up(sizeof(fa::PackedHeader)) + up(slot_rows[0] * (d + 1) * 4) + up(slot_rows[1] * (d + 1) * 4) +
                       part_rows * (d + 1) * 4;
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
  if (!direct && fa::internal_workspace(&ws, bytes, c.st) != cudaSuccess) {
    cudaGetLastError();
    return FA_ERR_NO_MEMORY;
  }
  if (!direct) {
    char* at = static_cast<char*>(ws);
    pl.cum = reinterpret_cast<long long*>(at);
    at += n_cum;
    for (int list = 0; list < 2; ++list) {
      p.entries[list] = pl.entries[list] = reinterpret_cast<fa::PackedEntry*>(at);
      at += n_entries[list];
      pl.seq_base[list] = reinterpret_cast<int*>(at);
      at += n_base;
      p.starts[list] = pl.starts[list] = reinterpret_cast<fa::PackedStart*>(at);
      at += n_starts[list];
      if (slot_rows[list] > 0) {
        p.o_slot[list] = reinterpret_cast<float*>(at);
        p.lse_slot[list] = p.o_slot[list] + slot_rows[list] * d;
        at += up(slot_rows[list] * (d + 1) * 4);
      }
    }
    p.header = pl.header = reinterpret_cast<fa::PackedHeader*>(at);
    at += up(sizeof(fa::PackedHeader));
    if (part_rows > 0) {
      p.o_part = reinterpret_cast<float*>(at);
      p.lse_part = p.o_part + part_rows * d;
    }
  }
  p.s = pl.s = fa::PackedSeqs{cu_q, cu_k, used_k, B, Tq, Tk, causal, status};
  p.direct = direct ? 1 : 0;
  // (One token, 8 heads of d = 128 over 600 and 1024 keys: 10.5 and 13.7 us by one
  // warpgroup, 9.5 and 10.7 by two; 4 sequences of 150 tokens in all 6.6, and 7.2.)
  p.halves = key_tiles >= 4 ? 1 : 0;
  p.head_groups = (int)hgs;
  p.prefix_tiles = prefix_tiles;
  pl.tile_tokens = p.tile_tokens;
  pl.prefix_tiles = prefix_tiles;
  pl.shared = p.shared;
  pl.head_groups = (int)hgs;
  pl.grid = p.grid;
  p.Tq = Tq;
  p.prefix_len = P;
  p.causal = causal != FA_CAUSAL_NONE ? 1 : 0;
  p.scale_log2 = scale * 1.4426950408889634f;
  p.o = o->ptr;
  p.o_row = Tq > 1 ? o->row_stride : 0;
  p.o_head = H > 1 ? o->head_stride : 0;
  p.lse = lse;
  p.store32 = aligned32(o->ptr, p.o_row, p.o_head) ? 1 : 0;
  p.status = status;
  p.timeout_ns = fa::internal_wait_timeout_ns();
  // Rows of a CTA of the join: all its threads', or fewer where these leave SMs
  // over (not many more CTAs than that: twice as many take 3 us longer).
  c.join_rows = fa::kMergeThreads;
  while (c.join_rows > 8 && (long long)Tq * H / c.join_rows * (d / 16) < sm_count) c.join_rows /= 2;
  c.join_tokens = std::max(1, c.join_rows / H);
  c.join_grid = (Tq + c.join_tokens - 1) / c.join_tokens;
  c.join_grid = std::min(c.join_grid, sm_count);

  cudaError_t ce = cudaSuccess;
  if (!direct) ce = fa::internal_timed_launch(FA_KERNEL_PACKED_PLAN, c.st, run_plan, &c);
  if (ce == cudaSuccess) ce = fa::internal_timed_launch(FA_KERNEL_PACKED_FWD, c.st, run_fwd, &c);
  if (ce == cudaSuccess && (cuts || p.shared)) ce = fa::internal_timed_launch(FA_KERNEL_PACKED_MERGE, c.st, run_merge, &c);
  if (ws != nullptr) cudaFreeAsync(ws, c.st);
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
