// Host side of the 4-bit key/value cache calls (include/fa.h): argument
// checks and launches.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstring>

#include "fa_common.h"
#include "kv4_fwd.h"

namespace fa {
int internal_device_setup(unsigned int** status, int* sm_count);
cudaError_t internal_timed_launch(int kernel, cudaStream_t stream, cudaError_t (*launch)(void*), void* ctx);
cudaError_t launch_kv4_move(int d, bool write, const Kv4Cache& c, const int* start, const int* count, const void* k_in,
                            const void* v_in, void* k_out, void* v_out, int N, int sm_count, cudaStream_t stream);
int kv4_fwd_unit_rows(int d, int rows, long long sm_steps);
int kv4_fwd_step_keys();
int kv4_fwd_warps(int d, int unit_rows);
int kv4_fwd_unit_cost();
cudaError_t launch_kv4_fwd(int d, int unit_rows, const Kv4FwdParams& p, int grid, cudaStream_t stream);
cudaError_t launch_kv4_merge(int d, int unit_rows, const Kv4FwdParams& p, int grid, cudaStream_t stream);
cudaError_t internal_workspace(void** ptr, size_t bytes, cudaStream_t st);
unsigned long long internal_wait_timeout_ns();
}  // namespace fa

namespace {

constexpr int kMinPage = 16, kMaxPage = 1024;
// Units of at most this many steps are not cut between CTAs: a second launch
// costs more than it gains (32 sequences, 8 heads of d = 128: 16 steps 10.0 us
// whole, 11.6 us cut; 24 steps 12.2 and 13.1; 32 steps 15.5 and 16.3, but the
// lengths ragged 13.4 and 12.7).  The host knows the table's width and not the
// lengths, so this goes by what the table has room for.
constexpr int kWholeSteps = 24;
constexpr int kMaxRows = 128;  // query rows of a key/value head's group (fa_kv4_fwd)

bool aligned(const void* p, uintptr_t n) { return p != nullptr && (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

bool head_dim(int d) { return d == 64 || d == 96 || d == 128 || d == 256; }

// Sizes that every call over a cache has; `rows` counts the rows of its bf16
// tensors per (batch, head).
int check_sizes(int B, int heads, int Hkv, int rows, int d, int num_pages, int page_size, int max_pages) {
  if (B < 1 || heads < 1 || Hkv < 1 || rows < 1 || num_pages < 1 || max_pages < 1) return FA_ERR_INVALID_ARG;
  if (page_size < kMinPage || page_size > kMaxPage || (page_size & (page_size - 1)) != 0) return FA_ERR_INVALID_ARG;
  if (!head_dim(d)) return FA_ERR_UNSUPPORTED;
  const long long most = 0x7fffffffLL;
  // Positions and rows stay below 2^30, so that a step past one fits an int.
  if ((long long)max_pages * page_size > (1 << 30) || rows > (1 << 30)) return FA_ERR_INVALID_ARG;
  if ((long long)B * heads > most || (long long)B * heads * rows > most) return FA_ERR_INVALID_ARG;
  return FA_OK;
}

fa::Kv4Cache view(const void* cache, const int* table, int B, int Hkv, int num_pages, int page_size, int max_pages,
                  unsigned int* status) {
  fa::Kv4Cache c;
  c.pages = static_cast<uint8_t*>(const_cast<void*>(cache));
  c.table = table;
  c.num_pages = num_pages;
  c.max_pages = max_pages;
  c.Hkv = Hkv;
  c.page_shift = 0;
  while ((1 << c.page_shift) < page_size) ++c.page_shift;
  c.B = B;
  c.status = status;
  return c;
}

struct Move {
  int d;
  bool write;
  fa::Kv4Cache c;
  const int *start, *count;
  const void *k_in, *v_in;
  void *k_out, *v_out;
  int N;
  int sm_count;
  cudaStream_t st;
};

cudaError_t run_move(void* ctx) {
  const Move& m = *static_cast<const Move*>(ctx);
  return fa::launch_kv4_move(m.d, m.write, m.c, m.start, m.count, m.k_in, m.v_in, m.k_out, m.v_out, m.N, m.sm_count, m.st);
}

int move(bool write, const void* k_in, const void* v_in, void* k_out, void* v_out, const void* cache,
         const int* block_table, const int* start, const int* count, int B, int Hkv, int N, int d, int num_pages,
         int page_size, int max_pages, void* stream) {
  const void* k = write ? k_in : k_out;
  const void* v = write ? v_in : v_out;
  if (!aligned(k, 16) || !aligned(v, 16) || !aligned(cache, 16) || !aligned(block_table, 4) || !aligned(start, 4) ||
      (count != nullptr && !aligned(count, 4)))
    return FA_ERR_INVALID_ARG;
  int e = check_sizes(B, Hkv, Hkv, N, d, num_pages, page_size, max_pages);
  if (e) return e;
  unsigned int* status = nullptr;
  int sm_count = 0;
  e = fa::internal_device_setup(&status, &sm_count);
  if (e) return e;
  Move m{d, write, view(cache, block_table, B, Hkv, num_pages, page_size, max_pages, status), start, count, k_in, v_in,
         k_out, v_out, N, sm_count, static_cast<cudaStream_t>(stream)};
  const int id = write ? FA_KERNEL_KV4_WRITE : FA_KERNEL_KV4_READ;
  return fa::internal_timed_launch(id, m.st, run_move, &m) == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

struct Fwd {
  int d;
  int unit_rows;
  fa::Kv4FwdParams p;
  int grid;
  cudaStream_t st;
};

cudaError_t run_fwd(void* ctx) {
  const Fwd& f = *static_cast<const Fwd*>(ctx);
  return fa::launch_kv4_fwd(f.d, f.unit_rows, f.p, f.grid, f.st);
}

cudaError_t run_merge(void* ctx) {
  const Fwd& f = *static_cast<const Fwd*>(ctx);
  return fa::launch_kv4_merge(f.d, f.unit_rows, f.p, f.grid, f.st);
}

int units_of(int rows, int unit_rows) { return (rows + unit_rows - 1) / unit_rows; }

// How a call is carried out (fa_kv4_plan_t), but for what depends on the
// device.  The lengths are known on the device only, so this goes by what the
// table can hold; FA_ERR_INVALID_ARG where the list of steps might then not fit
// 31 bits.
int plan_units(int B, int H, int Hkv, int Nq, int d, int num_pages, int page_size, int max_pages, int causal,
               fa_kv4_plan_t* pl) {
  const int e = check_sizes(B, H, Hkv, Nq, d, num_pages, page_size, max_pages);
  if (e) return e;
  if (H % Hkv != 0 || causal < FA_CAUSAL_NONE || causal > FA_CAUSAL_BOTTOM_RIGHT) return FA_ERR_INVALID_ARG;
  if ((long long)(H / Hkv) * Nq > kMaxRows) return FA_ERR_UNSUPPORTED;
  std::memset(pl, 0, sizeof(*pl));
  pl->rows = (H / Hkv) * Nq;
  pl->step_keys = fa::kv4_fwd_step_keys();
  const long long held = (long long)max_pages * page_size;
  pl->max_steps = (int)((held + pl->step_keys - 1) / pl->step_keys);
  // With the fewest rows a unit may have.
  const long long places = (long long)B * Hkv * units_of(pl->rows, fa::kv4_fwd_unit_rows(d, pl->rows, 0)) *
                           (pl->max_steps + fa::kv4_fwd_unit_cost());
  return places > 0x7fffffffLL ? FA_ERR_INVALID_ARG : FA_OK;
}

void plan_grid(int B, int Hkv, int d, int sm_count, fa_kv4_plan_t* pl) {
  const long long steps = (long long)B * Hkv * units_of(pl->rows, fa::kv4_fwd_unit_rows(d, pl->rows, 0)) * pl->max_steps;
  pl->unit_rows = fa::kv4_fwd_unit_rows(d, pl->rows, steps / sm_count);
  pl->row_blocks = units_of(pl->rows, pl->unit_rows);
  pl->units = B * Hkv * pl->row_blocks;
  // Where every unit has a CTA of its own, up to three steps a warp, and four if
  // that keeps half the SMs busy (8 heads of d = 128: one sequence of 1000 tokens
  // 8.3 us, cut 9.2, of 1500 9.7 and 9.2; 16 of 1500 10.5 and 13.2; alike at
  // d = 64 and 256 with their 16 and 8 warps).
  const int warps = fa::kv4_fwd_warps(d, pl->unit_rows);
  const int single = pl->units > sm_count ? 0 : (2 * pl->units >= sm_count ? 4 : 3) * warps;
  pl->whole = pl->max_steps <= std::max(kWholeSteps, single) ? 1 : 0;
  pl->launches = pl->whole ? 1 : 2;
  const long long most = (long long)pl->units * (pl->whole ? 1 : pl->max_steps);
  pl->grid = (int)std::min<long long>(most, sm_count);
  if (!pl->whole)
    pl->workspace_bytes = (uint64_t)pl->grid * (2ull * pl->unit_rows * (d * sizeof(float) + sizeof(float2)) +
                                                sizeof(fa::Kv4Cut));
}

// fa_kv4_fwd, its waits limited to `timeout_ns`; `missing`: see Kv4FwdParams.
int forward(const void* q, const void* cache, const int* block_table, const int* lens, void* o, float* lse, int B, int H,
            int Hkv, int Nq, int d, int num_pages, int page_size, int max_pages, int causal, float scale,
            unsigned long long timeout_ns, uint32_t missing, void* stream) {
  if (!aligned(q, 16) || !aligned(cache, 16) || !aligned(o, 16) || !aligned(lse, 16) || !aligned(block_table, 4) ||
      !aligned(lens, 4))
    return FA_ERR_INVALID_ARG;
  if (!(std::isfinite(scale) && scale > 0.f)) return FA_ERR_INVALID_ARG;
  fa_kv4_plan_t pl;
  int e = plan_units(B, H, Hkv, Nq, d, num_pages, page_size, max_pages, causal, &pl);
  if (e) return e;
  unsigned int* status = nullptr;
  int sm_count = 0;
  e = fa::internal_device_setup(&status, &sm_count);
  if (e) return e;
  plan_grid(B, Hkv, d, sm_count, &pl);
  Fwd f;
  f.d = d;
  f.unit_rows = pl.unit_rows;
  f.grid = pl.grid;
  f.p.c = view(cache, block_table, B, Hkv, num_pages, page_size, max_pages, status);
  f.p.q = static_cast<const __nv_bfloat16*>(q);
  f.p.lens = lens;
  f.p.o = static_cast<__nv_bfloat16*>(o);
  f.p.lse = lse;
  f.p.Nq = Nq;
  f.p.rows = pl.rows;
  f.p.row_blocks = pl.row_blocks;
  f.p.causal = causal;
  int power = 0;
  const double rest = std::frexp((double)scale * 1.4426950408889634, &power);
  power = std::min(power - 1, 127);
  f.p.scale_pow2 = std::ldexp(1.f, power);
  f.p.scale_rest = (float)(power == 127 ? (double)scale * 1.4426950408889634 / std::ldexp(1.0, 127) : 2 * rest);
  f.p.whole = pl.whole;
  f.p.single = pl.whole && pl.grid == pl.units ? 1 : 0;
  f.p.part_o = nullptr;
  f.p.part_ml = nullptr;
  f.p.cuts = nullptr;
  f.p.timeout_ns = timeout_ns;
  f.p.missing = missing;
  f.st = static_cast<cudaStream_t>(stream);
  void* ws = nullptr;
  if (pl.workspace_bytes > 0) {
    if (fa::internal_workspace(&ws, pl.workspace_bytes, f.st) != cudaSuccess) {
      cudaGetLastError();
      return FA_ERR_NO_MEMORY;
    }
    const size_t parts = (size_t)2 * pl.grid * pl.unit_rows;
    f.p.part_o = static_cast<float*>(ws);
    f.p.part_ml = reinterpret_cast<float2*>(f.p.part_o + parts * d);
    f.p.cuts = reinterpret_cast<fa::Kv4Cut*>(f.p.part_ml + parts);
  }
  cudaError_t ce = fa::internal_timed_launch(FA_KERNEL_KV4_FWD, f.st, run_fwd, &f);
  if (ce == cudaSuccess && ws != nullptr) ce = fa::internal_timed_launch(FA_KERNEL_KV4_MERGE, f.st, run_merge, &f);
  if (ws != nullptr) cudaFreeAsync(ws, f.st);
  return ce == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

}  // namespace

extern "C" {

int fa_kv4_cache_bytes(int num_pages, int Hkv, int page_size, int d, uint64_t* bytes) {
  if (bytes == nullptr) return FA_ERR_INVALID_ARG;
  const int e = check_sizes(1, 1, Hkv, 1, d, num_pages, page_size, 1);
  if (e) return e;
  // A page of a head is below 2^19 bytes; pages and heads are below 2^31 each.
  const uint64_t page = (uint64_t)page_size * (9 * d / 8), pages = (uint64_t)num_pages * Hkv;
  if (pages > INT64_MAX / page) return FA_ERR_INVALID_ARG;
  *bytes = pages * page;
  return FA_OK;
}

int fa_kv4_write(const void* k, const void* v, void* cache, const int* block_table, const int* start,
                 const int* count, int B, int Hkv, int N, int d, int num_pages, int page_size, int max_pages,
                 void* stream) {
  return move(true, k, v, nullptr, nullptr, cache, block_table, start, count, B, Hkv, N, d, num_pages, page_size,
              max_pages, stream);
}

int fa_kv4_read(const void* cache, const int* block_table, const int* start, const int* count, void* k, void* v,
                int B, int Hkv, int N, int d, int num_pages, int page_size, int max_pages, void* stream) {
  return move(false, nullptr, nullptr, k, v, cache, block_table, start, count, B, Hkv, N, d, num_pages, page_size,
              max_pages, stream);
}

int fa_kv4_fwd(const void* q, const void* cache, const int* block_table, const int* lens, void* o, float* lse,
               int B, int H, int Hkv, int Nq, int d, int num_pages, int page_size, int max_pages, int causal,
               float scale, void* stream) {
  return forward(q, cache, block_table, lens, o, lse, B, H, Hkv, Nq, d, num_pages, page_size, max_pages, causal, scale,
                 fa::internal_wait_timeout_ns(), 0, stream);
}

int fa_selftest_kv4_timeout(const void* q, const void* cache, const int* block_table, const int* lens, void* o,
                            float* lse, int B, int H, int Hkv, int Nq, int d, int num_pages, int page_size,
                            int max_pages, uint64_t timeout_ns, void* stream) {
  if (timeout_ns > 2000000000ull) return FA_ERR_INVALID_ARG;
  return forward(q, cache, block_table, lens, o, lse, B, H, Hkv, Nq, d, num_pages, page_size, max_pages,
                 FA_CAUSAL_NONE, 1.f, timeout_ns, 16, stream);
}

int fa_kv4_fwd_plan(int B, int H, int Hkv, int Nq, int d, int page_size, int max_pages, int sm_count,
                    fa_kv4_plan_t* plan) {
  if (plan == nullptr || sm_count < 1) return FA_ERR_INVALID_ARG;
  fa_kv4_plan_t pl;
  const int e = plan_units(B, H, Hkv, Nq, d, 1, page_size, max_pages, FA_CAUSAL_NONE, &pl);
  if (e) return e;
  plan_grid(B, Hkv, d, sm_count, &pl);
  *plan = pl;
  return FA_OK;
}

}  // extern "C"
