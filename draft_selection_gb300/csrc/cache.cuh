// What the paged-cache and tree translation units share: argument checks on the
// host and the view of a cache that their kernels take.  Not public.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "dfl2.h"
#include "dfl2_internal.cuh"

namespace dfl2 {

struct PtrArg {
  const void* p;
  const char* name;
  int align;
  bool optional = false;
};
dfl2_status report_errorf(dfl2_status st, const char* fmt, ...);
dfl2_status report_cuda_error(cudaError_t e, const char* what);
// Non-NULL and aligned (no CUDA call); then: device memory (sets up the device's state).
dfl2_status check_args_host(const PtrArg* a, int n);
dfl2_status check_args_device(const PtrArg* a, int n);
// The fields of a cache, its pointers included (no CUDA call).
dfl2_status check_cache_host(const dfl2_cache* c);
dfl2_status check_cache_device(const dfl2_cache* c);

constexpr int kMaxTree = 256;   // nodes of a tree
constexpr int kMaxSeqs = 4096;  // sequences of one call that takes pages
constexpr int kMaxBatch = 65535;  // and of any other: a grid's second dimension
constexpr int kMaxLen = 1 << 30;  // a sequence's length

inline int elem_bytes(int dtype) { return dtype == DFL2_F32 ? 4 : 2; }
inline int log2_of(int v) {
  int s = 0;
  while ((1 << s) < v) ++s;
  return s;
}

// Where a cache's sequences are, as kernels see it.
struct TableView {
  int32_t* table;
  int rows, cols, pages, page_shift;
  int32_t* refs;
  uint32_t* free_bits;
  const int32_t* seq;     // table row of sequence b, or NULL
  const int32_t* length;  // [B]
  const int32_t* count;   // [B], or NULL: T each
  int T;
  uint32_t* err;

  // The table row of sequence b; -1 (recorded) if out of range.
  __device__ __forceinline__ int row_of(int b) const { return checked_row(seq ? seq[b] : b); }
  __device__ __forceinline__ int checked_row(int r) const {
    if (static_cast<unsigned>(r) < static_cast<unsigned>(rows)) return r;
    record_error(err, kDevErrBadIndex);
    return -1;
  }
  // Whether a sequence can be that long; if not, recorded.  (Positions behind a length near
  // the largest integers would wrap round to entries before the table.)
  __device__ __forceinline__ bool checked_length(int len) const {
    if (static_cast<unsigned>(len) <= static_cast<unsigned>(kMaxLen)) return true;
    record_error(err, kDevErrBadIndex);
    return false;
  }
  __device__ __forceinline__ bool in_range(int row, int len) const {
    return static_cast<unsigned>(row) < static_cast<unsigned>(rows) &&
           static_cast<unsigned>(len) <= static_cast<unsigned>(kMaxLen);
  }
  __device__ __forceinline__ int count_of(int b) const {
    return count ? max(0, min(T, count[b])) : T;
  }
  // Entry i of a row as it stands, -1 past its end.
  __device__ __forceinline__ int entry(int row, int i) const {
    return static_cast<unsigned>(i) < static_cast<unsigned>(cols)
               ? table[static_cast<int64_t>(row) * cols + i]
               : -1;
  }
  // An entry that is a page number, or -1 (recorded, unless it is the plain "none" that
  // may_lack allows).
  __device__ __forceinline__ int checked(int p, bool may_lack = false) const {
    if (static_cast<unsigned>(p) < static_cast<unsigned>(pages)) return p;
    if (!may_lack || p != -1) record_error(err, kDevErrBadIndex);
    return -1;
  }
  // Both.
  __device__ __forceinline__ int page_at(int row, int i, bool may_lack = false) const {
    return checked(entry(row, i), may_lack);
  }
};

// One holder of page p fewer.
__device__ __forceinline__ void drop_page(const TableView& t, int p) {
  if (static_cast<unsigned>(p) >= static_cast<unsigned>(t.pages)) {
    record_error(t.err, kDevErrBadIndex);
    return;
  }
  const int old = atomicSub(&t.refs[p], 1);
  if (old == 1) {
    atomicOr(&t.free_bits[p >> 5], 1u << (p & 31));
  } else if (old < 1) {  // nobody held it: the state is not a cache's
    atomicAdd(&t.refs[p], 1);
    record_error(t.err, kDevErrBadIndex);
  }
}

inline TableView table_view(const dfl2_cache* c, const int32_t* seq, const int32_t* length,
                            const int32_t* count, int T) {
  return TableView{c->table, c->rows, c->cols,  c->pages, log2_of(c->page_size), c->refs,
                   c->free_bits, seq, length, count, T, device_error_word()};
}

}  // namespace dfl2
