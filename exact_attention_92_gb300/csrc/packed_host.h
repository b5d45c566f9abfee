// Host helpers of the calls over packed sequences: checks of their arguments and
// the tensor maps of rows with strides.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "fa_common.h"

namespace fa {

int internal_device_setup(unsigned int** status, int* sm_count);
int internal_encode_tiled(CUtensorMap* m, const void* ptr, int rank, const uint64_t* dims, const uint64_t* strides,
                          const uint32_t* box);
cudaError_t internal_workspace(void** ptr, size_t bytes, cudaStream_t st);
cudaError_t internal_timed_launch(int kernel, cudaStream_t stream, cudaError_t (*launch)(void*), void* ctx);
unsigned long long internal_wait_timeout_ns();

namespace packed_host {

constexpr long long kMost = 1 << 30;  // tokens, sequences

inline bool head_dim(int d) { return d == 64 || d == 96 || d == 128; }
inline bool array_ok(const void* p, uintptr_t n) { return p != nullptr && (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
inline bool aligned32(const void* p, long long row, long long head) {
  return (reinterpret_cast<uintptr_t>(p) & 31u) == 0 && row % 16 == 0 && head % 16 == 0;
}

// Rows that a tensor map can say: strides above zero (but where there is only
// one), multiples of 16 bytes, below 2^40.
inline bool rows_ok(const fa_rows_t* r, long long rows, int heads) {
  if (r == nullptr || r->ptr == nullptr || (reinterpret_cast<uintptr_t>(r->ptr) & 15u) != 0) return false;
  const long long most = 1LL << 38;
  if (rows > 1 && (r->row_stride <= 0 || r->row_stride % 8 != 0 || r->row_stride >= most)) return false;
  if (heads > 1 && (r->head_stride <= 0 || r->head_stride % 8 != 0 || r->head_stride >= most)) return false;
  return true;
}
// ... and that do not overlap, for outputs.
inline bool rows_apart(const fa_rows_t* r, long long rows, int heads, int d) {
  const long long rs = rows > 1 ? r->row_stride : 0, hs = heads > 1 ? r->head_stride : 0;
  if (rows == 1) return heads == 1 || hs >= d;
  if (heads == 1) return rs >= d;
  return (hs >= d && rs >= (long double)(heads - 1) * hs + d) || (rs >= d && hs >= (long double)(rows - 1) * rs + d);
}

inline uint64_t step_bytes(int64_t stride, long long n) { return n > 1 ? (uint64_t)stride * 2 : 16; }

// Rows of a tile that may start before its sequence's (see packed.h): [channel,
// row of the tile, first row, head].
inline int encode_tile(CUtensorMap* m, const fa_rows_t* r, int rows, int heads, int d, int box_rows) {
  const uint64_t rs = step_bytes(r->row_stride, rows), hs = step_bytes(r->head_stride, heads);
  const uint64_t dims[4] = {(uint64_t)d, (uint64_t)kTileN, (uint64_t)rows, (uint64_t)heads};
  const uint64_t strides[3] = {rs, rs, hs};
  const uint32_t box[4] = {64, (uint32_t)box_rows, 1, 1};
  return internal_encode_tiled(m, r->ptr, 4, dims, strides, box);
}

// Rows as they lie, 128 at a time: [channel, row, head].
inline int encode_plain(CUtensorMap* m, const fa_rows_t* r, int rows, int heads, int d) {
  const uint64_t dims[3] = {(uint64_t)d, (uint64_t)rows, (uint64_t)heads};
  const uint64_t strides[2] = {step_bytes(r->row_stride, rows), step_bytes(r->head_stride, heads)};
  const uint32_t box[3] = {64, 128, 1};
  return internal_encode_tiled(m, r->ptr, 3, dims, strides, box);
}

inline size_t up(size_t n) { return (n + 255) & ~(size_t)255; }

}  // namespace packed_host
}  // namespace fa
