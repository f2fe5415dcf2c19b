// The paged key/value cache: taking, sharing and giving back pages, and moving
// rows of keys and values (include/dfl2.h, "The cache").
//
// Bookkeeping.  A page is free iff its count is 0, and the free pages are kept
// as a bit map besides: finding the N lowest free pages is then one scan of
// pages/8 bytes by one CTA, and giving a page back is one atomicOr, whose order
// does not matter.  So a call's result is a function of the state before it.
//
// Moving rows.  All copies are pure traffic: a position's row in one layer is
// kv_heads pieces of head_dim elements for K and as many for V, each at least
// 16 bytes and 16-byte aligned.  One warp takes one position's row with eight
// 16-byte loads a lane in flight (four of K, four of V) before the stores.
#include <cuda_runtime.h>

#include <algorithm>

#include "cache.cuh"

namespace dfl2 {
namespace {

constexpr int kBookThreads = 1024;
constexpr int kListCap = 4096;  // pages handed out per round of the list below
constexpr unsigned kAll = 0xffffffffu;

// Sum over the threads before this one, and over all of them.
__device__ __forceinline__ int block_scan(int v, int& total, int* warp_sums) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int x = v;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int y = __shfl_up_sync(kAll, x, off);
    if (lane >= off) x += y;
  }
  __syncthreads();  // warp_sums may still be read from the scan before
  if (lane == 31) warp_sums[warp] = x;
  __syncthreads();
  if (warp == 0) {
    int w = warp_sums[lane];
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int y = __shfl_up_sync(kAll, w, off);
      if (lane >= off) w += y;
    }
    warp_sums[lane] = w;
  }
  __syncthreads();
  total = warp_sums[31];
  return x - v + (warp ? warp_sums[warp - 1] : 0);
}

struct TakeArgs {
  TableView t;  // reserve: seq = table_rows; fork: seq = dst
  const int32_t* src;
  int32_t* served;
  int B;
};

// The table entries sequence b may need pages for: [c0, c1) of its row.
struct Span {
  int row, c0, c1;
  bool ok;
};
template <bool kFork>
__device__ __forceinline__ Span span_of(const TakeArgs& a, int b) {
  Span s;
  const int len = a.t.length[b], ps = 1 << a.t.page_shift;  // beside the row's
  s.row = a.t.row_of(b);
  const int64_t end = static_cast<int64_t>(len) + (kFork ? 0 : a.t.count_of(b));
  s.ok = s.row >= 0 && len >= 0 && len <= kMaxLen &&
         end <= static_cast<int64_t>(a.t.cols) << a.t.page_shift;
  s.c0 = s.ok ? len >> a.t.page_shift : 0;
  s.c1 = s.ok ? static_cast<int>((end + ps - 1) >> a.t.page_shift) : 0;
  return s;
}

// One CTA: which sequences get their pages, and the pages themselves.  Bound by its
// dependent steps (lengths, table entries, two scans, the table again), not by the
// pages/8 bytes of the map: 5.2 us for one sequence, 5.9 for 64 with 33 nodes each, 7.4
// for 128 forks (ncu, caches flushed), less in a turn, where PDL hides its start.  Loads
// that do not need each other are issued together (four forks with their copies: 9.9 us,
// 10.9 one after the other).
//
// kWidth lanes of a warp look after a sequence: all 32 while the 32 warps hold every
// sequence at once, else 8, so that up to 128 still go at once.  With a warp to each in
// any case, 128 forks take 143.6 us instead of 135.7 and a turn of 64 sequences 62.6
// instead of 60.9; with 8 lanes in any case, a long prompt's entries take four times the
// steps.
template <bool kFork, int kWidth>
__global__ void __launch_bounds__(kBookThreads) take_kernel(const __grid_constant__ TakeArgs a) {
  __shared__ int offs[kMaxSeqs];  // a sequence's need; then its first page's rank, -1 if unserved
  __shared__ int list[kListCap];
  __shared__ int warp_sums[32];
  __shared__ int taken_s;
  const int tid = threadIdx.x, lane = tid & 31;
  pdl_wait();
  pdl_launch_dependents();
  if (tid == 0) taken_s = 0;

  constexpr int kGroups = kBookThreads / kWidth;
  constexpr unsigned kGroupBits = kAll >> (32 - kWidth);
  const int group = tid / kWidth, gl = lane % kWidth, g0 = lane - gl;  // g0: the group's lane 0
  const int first = (tid - lane) / kWidth;  // the warp's first group
  // the free pages: each thread the words [w0, w1) of the bit map (bits past the pages
  // are none), the first of them on its way beside the tables
  const int words = (a.t.pages - 1) / 32 + 1;
  auto free_word = [&](int w) {
    const uint32_t x = a.t.free_bits[w];
    return w < words - 1 ? x : x & (0xffffffffu >> (31 - ((a.t.pages - 1) & 31)));
  };
  const int wper = (words + kBookThreads - 1) / kBookThreads;
  const int w0 = min(words, tid * wper), w1 = min(words, w0 + wper);
  uint32_t left = w0 < w1 ? free_word(w0) : 0u;
  // the needs (the collectives are the warp's, so its groups take the same steps)
  for (int b0 = 0; b0 + first < a.B; b0 += kGroups) {
    const int b = b0 + group;
    const bool there = b < a.B;
    Span s{-1, 0, 0, false};
    const int src = kFork && there ? a.src[b] : -1;
    if (there) s = span_of<kFork>(a, b);
    int need = 0;
    bool good = s.ok;
    if (kFork && there) good &= a.t.checked_row(src) >= 0;
    if (good) {
      const int32_t* row = a.t.table + static_cast<int64_t>(s.row) * a.t.cols;
      if (kFork) {
        good = src != s.row;
        if (good) {
#pragma unroll 4
          for (int c = gl; c < s.c1; c += kWidth) good &= a.t.page_at(src, c, true) >= 0;
          // (to the row's end: pages past the fork's last would be the next reserve's)
#pragma unroll 8
          for (int c = gl; c < a.t.cols; c += kWidth) good &= row[c] < 0;
        }
      }
#pragma unroll 4
      for (int c = s.c0 + gl; c < s.c1; c += kWidth) need += row[c] < 0;
    }
    __syncwarp();
    const bool ok = ((__ballot_sync(kAll, good) >> g0) & kGroupBits) == kGroupBits;
    if (kWidth == 32)
      need = __reduce_add_sync(kAll, need);
    else
#pragma unroll
      for (int off = kWidth >> 1; off; off >>= 1) need += __shfl_xor_sync(kAll, need, off);
    if (there && gl == 0) offs[b] = ok ? need : -1;
  }
  int mine = __popc(left);
  for (int w = w0 + 1; w < w1; ++w) mine += __popc(free_word(w));
  int n_free, total;
  int rank = block_scan(mine, n_free, warp_sums);  // rank of this thread's first free page
  // served in order while the pages last
  const int bper = (a.B + kBookThreads - 1) / kBookThreads;
  const int b0 = min(a.B, tid * bper), b1 = min(a.B, b0 + bper);
  int need = 0;
  for (int b = b0; b < b1; ++b) need += max(0, offs[b]);
  int cum = block_scan(need, total, warp_sums);
  int reach = 0;
  for (int b = b0; b < b1; ++b) {
    const int n = offs[b];
    const bool ok = n >= 0 && (n == 0 || n <= n_free - cum);
    a.served[b] = ok;
    offs[b] = ok ? cum : -1;
    cum += max(0, n);
    if (ok && n > 0) reach = cum;
  }
  if (reach) atomicMax(&taken_s, reach);
  __syncthreads();
  const int taken = taken_s;

  int w = w0;
  for (int r0 = 0; r0 < taken; r0 += kListCap) {
    const int r1 = min(taken, r0 + kListCap);
    // the pages of ranks [r0, r1), each from the thread that holds its word
    while (w < w1 && rank < r1) {
      uint32_t gone = 0;
      while (left && rank < r1) {
        const int bit = __ffs(left) - 1;
        left &= left - 1;
        gone |= 1u << bit;
        const int page = w * 32 + bit;
        list[rank - r0] = page;
        a.t.refs[page] = 1;
        ++rank;
      }
      if (gone) a.t.free_bits[w] &= ~gone;
      if (!left) {
        ++w;
        left = w < w1 ? free_word(w) : 0u;
      }
    }
    __syncthreads();
    for (int b0 = 0; b0 + first < a.B; b0 += kGroups) {
      const int b = b0 + group;
      const bool takes = b < a.B && offs[b] >= 0 && offs[b] < r1;
      Span s{-1, 0, 0, false};
      if (takes) s = span_of<kFork>(a, b);
      int32_t* row = a.t.table + static_cast<int64_t>(s.row) * a.t.cols;
      // entries of lower rank were filled in the rounds before
      int r = takes ? max(offs[b], r0) : r1;
      for (int c = s.c0; __any_sync(kAll, c < s.c1 && r < r1); c += kWidth) {
        const bool miss = r < r1 && c + gl < s.c1 && row[c + gl] < 0;
        const unsigned m = (__ballot_sync(kAll, miss) >> g0) & kGroupBits;
        const int at = r + __popc(m & ((1u << gl) - 1));
        if (miss && at < r1) row[c + gl] = list[at - r0];
        r += __popc(m);
      }
    }
    __syncthreads();
  }
  if (kFork) {  // the whole pages, shared
    for (int b = group; b < a.B; b += kGroups) {
      if (offs[b] < 0) continue;
      const Span s = span_of<kFork>(a, b);
      const int32_t* from = a.t.table + static_cast<int64_t>(a.src[b]) * a.t.cols;
      int32_t* row = a.t.table + static_cast<int64_t>(s.row) * a.t.cols;
      for (int c = gl; c < s.c0; c += kWidth) {
        const int p = from[c];
        row[c] = p;
        atomicAdd(&a.t.refs[p], 1);
      }
    }
  }
}

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

__global__ void __launch_bounds__(256) free_kernel(const __grid_constant__ TableView t) {
  pdl_wait();
  pdl_launch_dependents();
  const int row = t.row_of(blockIdx.x);
  if (row < 0) return;
  int32_t* r = t.table + static_cast<int64_t>(row) * t.cols;
  for (int c = threadIdx.x; c < t.cols; c += blockDim.x) {
    const int p = r[c] == -1 ? -1 : atomicExch(&r[c], -1);
    if (p != -1) drop_page(t, p);
  }
}

// ---- rows of keys and values ------------------------------------------------

// x / d for 0 <= x < 2^16, 1 <= d < 2^16: with m = ceil(2^32 / d), x m / 2^32
// exceeds x / d by less than x / 2^32 < 1 / d, so its floor is right.
struct SmallDiv {
  uint32_t m, d;
  __device__ __forceinline__ uint32_t div(uint32_t x) const { return m ? __umulhi(x, m) : x; }
};
SmallDiv small_div(int d) {
  return SmallDiv{d == 1 ? 0u : static_cast<uint32_t>(((1ull << 32) + d - 1) / d),
                  static_cast<uint32_t>(d)};
}

// Strides in 16-byte units.
struct RowView {
  uint4* k;
  uint4* v;
  int64_t layer, page, head, slot;
  int chunks;  // 16-byte pieces of a position's row: kv_heads * per_head
  SmallDiv per_head;
};
RowView row_view(const dfl2_cache* c) {
  const int per = 16 / elem_bytes(c->dtype);
  return RowView{static_cast<uint4*>(c->k), static_cast<uint4*>(c->v), c->layer_stride / per,
                 c->page_stride / per, c->head_stride / per, c->slot_stride / per,
                 c->kv_heads * (c->head_dim / per), small_div(c->head_dim / per)};
}

// One warp copies a position's row of K and of V; fh, th: head strides.
__device__ __forceinline__ void copy_row(const uint4* fk, const uint4* fv, int64_t fh, uint4* tk,
                                         uint4* tv, int64_t th, int chunks, SmallDiv per_head,
                                         int lane) {
  for (int c0 = lane; c0 < chunks; c0 += 128) {
    uint4 x[4], y[4];
    int64_t to[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int c = c0 + 32 * i;
      if (c >= chunks) break;
      const uint32_t h = per_head.div(c), r = c - h * per_head.d;
      x[i] = fk[h * fh + r];
      y[i] = fv[h * fh + r];
      to[i] = h * th + r;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (c0 + 32 * i >= chunks) break;
      tk[to[i]] = x[i];
      tv[to[i]] = y[i];
    }
  }
}

struct WriteArgs {
  TableView t;
  RowView r;
  const uint4* k_new;
  const uint4* v_new;
  int64_t nl, nb, nt, nh;  // strides of the new rows, 16-byte units
  int layer, n_layers, B;
};

// Bound by HBM: 8 prompts of 300 to 2000 tokens into 24 layers, 8 heads x 128 channels,
// 0.97 GB read and as much written, in 271 us: 7.2 TB/s (the copy peak is 6.8).
__global__ void __launch_bounds__(256) write_kernel(const __grid_constant__ WriteArgs a) {
  pdl_wait();
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int64_t items = static_cast<int64_t>(a.n_layers) * a.B * a.t.T;
  const int64_t step = static_cast<int64_t>(gridDim.x) * 8;
  for (int64_t it = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5); it < items;
       it += step) {
    const int t = static_cast<int>(it % a.t.T);
    const int64_t lb = it / a.t.T;
    const int b = static_cast<int>(lb % a.B), l = static_cast<int>(lb / a.B);
    const int r = a.t.seq ? a.t.seq[b] : b, len = a.t.length[b];  // beside the count
    if (t >= a.t.count_of(b)) continue;
    const int row = a.t.checked_row(r);
    if (row < 0 || !a.t.checked_length(len)) continue;
    const int pos = len + t;  // t is below 2^30
    const int page = a.t.page_at(row, pos >> a.t.page_shift);
    if (page < 0) continue;
    const int64_t from = l * a.nl + b * a.nb + t * a.nt;
    const int64_t to = (a.layer + l) * a.r.layer + page * a.r.page +
                       (pos & ((1 << a.t.page_shift) - 1)) * a.r.slot;
    copy_row(a.k_new + from, a.v_new + from, a.nh, a.r.k + to, a.r.v + to, a.r.head, a.r.chunks,
             a.r.per_head, lane);
  }
}

struct ForkCopyArgs {
  TableView t;
  RowView r;
  const int32_t* src;
  const int32_t* served;
  int layers, n;
};

// The positions of the partly filled last page, every layer.  Bound by HBM: 128 forks
// of 32 sequences, pages of 64, 32 layers, 617 MB written and a quarter of it read (a
// parent's four children share it in L2), in 124 us: 6.2 TB/s.
__global__ void __launch_bounds__(256) fork_copy_kernel(const __grid_constant__ ForkCopyArgs a) {
  pdl_wait();
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31, ps = 1 << a.t.page_shift;
  const int64_t items = (static_cast<int64_t>(a.layers) * a.n) << a.t.page_shift;
  const int64_t step = static_cast<int64_t>(gridDim.x) * 8;
  for (int64_t it = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5); it < items;
       it += step) {
    const int slot = static_cast<int>(it & (ps - 1));
    const int64_t li = it >> a.t.page_shift;
    const int i = static_cast<int>(li % a.n), l = static_cast<int>(li / a.n);
    const int served = a.served[i], len = a.t.length[i], src = a.src[i], dst = a.t.seq[i];
    if (!served) continue;
    if (slot >= (len & (ps - 1))) continue;
    const int c = len >> a.t.page_shift;
    const int64_t from_page = a.t.page_at(src, c), to_page = a.t.page_at(dst, c);
    if (from_page < 0 || to_page < 0) continue;
    const int64_t at = l * a.r.layer + slot * a.r.slot;
    const int64_t from = at + from_page * a.r.page, to = at + to_page * a.r.page;
    copy_row(a.r.k + from, a.r.v + from, a.r.head, a.r.k + to, a.r.v + to, a.r.head, a.r.chunks,
             a.r.per_head, lane);
  }
}

struct CompactArgs {
  TableView t;
  RowView r;
  const int32_t* path;
  const int32_t* n_path;
  int32_t* new_length;
  int layers, B;
};

// A cluster of blocks to a sequence.  Each block works out where the moving rows come
// from and go to once, a thread to a node; then a thread owns one 16-byte column of K or
// V in one layer and moves it down that list, eight rows in flight.  The path ascends
// strictly, so path[i] >= i and a row that is written has been read before: reading ahead
// is safe.  When every block of the cluster has read the table, the first one gives the
// pages behind the kept rows back.
// Bound by the chain of dependent reads (path, table, rows).  The turn of 64 sequences,
// 16 layers: 61.1 us (60.0 since the path is read beside the count); with as many blocks
// as columns ask for and the pages given back by a kernel of their own 61.3, which costs
// the host 1.9 us more a call; blocks of 1024 threads 61.7; every thread looking its rows
// up for itself 1.8 more.
constexpr int kMoveThreads = 512, kMoveBlocks = 8;
__global__ void __launch_bounds__(kMoveThreads)
    compact_kernel(const __grid_constant__ CompactArgs a) {
  __shared__ int64_t from_s[kMaxTree], to_s[kMaxTree];
  __shared__ int warp_sums[kMaxTree / 32];
  constexpr int kBatch = 8;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, b = blockIdx.y;
  pdl_wait();
  pdl_launch_dependents();
  const int from = tid < a.t.T ? a.path[static_cast<int64_t>(b) * a.t.T + tid] : 0;
  const int len = a.t.length[b], count = a.t.count_of(b), n = min(a.n_path[b], count);
  int row = a.t.row_of(b);
  if (!a.t.checked_length(len)) row = -1;
  const int slots = (1 << a.t.page_shift) - 1;
  bool moves = false;
  int64_t src = 0, dst = 0;
  if (row >= 0 && tid < n) {
    if (from != tid) {
      const int64_t pf = from > tid && from < count
                             ? a.t.page_at(row, (len + from) >> a.t.page_shift)
                             : -1;
      const int64_t pt = a.t.page_at(row, (len + tid) >> a.t.page_shift);
      if (from < tid || from >= count) record_error(a.t.err, kDevErrBadIndex);
      moves = pf >= 0 && pt >= 0;
      src = pf * a.r.page + ((len + from) & slots) * a.r.slot;
      dst = pt * a.r.page + ((len + tid) & slots) * a.r.slot;
    }
  }
  const unsigned mine = __ballot_sync(kAll, moves);
  if (lane == 0 && warp < kMaxTree / 32) warp_sums[warp] = __popc(mine);
  __syncthreads();
  int at = 0, total = 0;
#pragma unroll
  for (int w = 0; w < kMaxTree / 32; ++w) {
    if (w < warp) at += warp_sums[w];
    total += warp_sums[w];
  }
  if (moves) {
    at += __popc(mine & ((1u << lane) - 1));
    from_s[at] = src;
    to_s[at] = dst;
  }
  __syncthreads();
  cluster_arrive_release();  // this block has read the table and the length
  const int columns = total > 0 ? a.layers * 2 * a.r.chunks : 0;
  for (int c = blockIdx.x * kMoveThreads + tid; c < columns; c += gridDim.x * kMoveThreads) {
    const int l = c / (2 * a.r.chunks);
    uint32_t col = c - l * 2 * a.r.chunks;
    const bool is_v = col >= static_cast<uint32_t>(a.r.chunks);
    if (is_v) col -= a.r.chunks;
    const uint32_t h = a.r.per_head.div(col);
    uint4* base = (is_v ? a.r.v : a.r.k) + l * a.r.layer + h * a.r.head +
                  (col - h * a.r.per_head.d);
    for (int i = 0; i < total; i += kBatch) {
      uint4 x[kBatch];
#pragma unroll
      for (int j = 0; j < kBatch; ++j)
        if (i + j < total) x[j] = base[from_s[i + j]];
#pragma unroll
      for (int j = 0; j < kBatch; ++j)
        if (i + j < total) base[to_s[i + j]] = x[j];
    }
  }
  __syncwarp();
  cluster_wait_acquire();
  if (blockIdx.x > 0) return;
  if (tid == 0) a.new_length[b] = row < 0 ? len : len + max(0, n);
  if (row < 0) return;
  const int ps = 1 << a.t.page_shift;
  const int c1 = min(a.t.cols, (len + count + ps - 1) >> a.t.page_shift);
  int32_t* r = a.t.table + static_cast<int64_t>(row) * a.t.cols;
  for (int c = ((len + max(0, n) + ps - 1) >> a.t.page_shift) + tid; c < c1; c += kMoveThreads) {
    const int p = atomicExch(&r[c], -1);
    if (p != -1) drop_page(a.t, p);
  }
}

dfl2_status check_batch(int B, int T, int max_t, int max_b = kMaxBatch) {
  if (B < 1) return report_errorf(DFL2_ERR_INVALID_ARG, "B=%d must be >= 1", B);
  if (B > max_b)
    return report_errorf(DFL2_ERR_UNSUPPORTED, "B=%d: at most %d sequences a call", B, max_b);
  if (T < 0) return report_errorf(DFL2_ERR_INVALID_ARG, "T=%d must be >= 0", T);
  if (T > max_t) return report_errorf(DFL2_ERR_UNSUPPORTED, "T=%d: at most %d", T, max_t);
  return DFL2_OK;
}

template <bool kFork>
cudaError_t launch_take(const TakeArgs& a, cudaStream_t s) {
  const auto kernel = a.B <= kBookThreads / 32 ? take_kernel<kFork, 32> : take_kernel<kFork, 8>;
  return launch_k(kernel, dim3(1), dim3(kBookThreads), 0, s, true, a);
}

int copy_blocks(int64_t items, int per_block) {
  const int64_t want = (items + per_block - 1) / per_block;
  return static_cast<int>(std::min<int64_t>(want, int64_t(1) << 20));
}

}  // namespace

dfl2_status check_cache_host(const dfl2_cache* c) {
  if (!c) return report_errorf(DFL2_ERR_INVALID_ARG, "cache is NULL");
  const PtrArg ptrs[] = {{c->k, "cache k", 16},         {c->v, "cache v", 16},
                         {c->table, "cache table", 4},  {c->refs, "cache refs", 4},
                         {c->free_bits, "cache free_bits", 4}};
  const dfl2_status st = check_args_host(ptrs, 5);
  if (st != DFL2_OK) return st;
  if (c->dtype != DFL2_F32 && c->dtype != DFL2_BF16 && c->dtype != DFL2_F16)
    return report_errorf(DFL2_ERR_UNSUPPORTED, "cache dtype %d", c->dtype);
  if (c->layers < 1 || c->pages < 1 || c->kv_heads < 1 || c->head_dim < 1 || c->rows < 1 ||
      c->cols < 1)
    return report_errorf(DFL2_ERR_INVALID_ARG, "every size of the cache must be >= 1");
  if (c->layers > 4096)
    return report_errorf(DFL2_ERR_UNSUPPORTED, "layers=%d: at most 4096", c->layers);
  if (c->page_size < 8 || c->page_size > 256 || (c->page_size & (c->page_size - 1)))
    return report_errorf(DFL2_ERR_UNSUPPORTED, "page_size %d: a power of two, 8 to 256",
                         c->page_size);
  const int per = 16 / elem_bytes(c->dtype);
  if (c->head_dim % per)
    return report_errorf(DFL2_ERR_UNSUPPORTED, "head_dim %d: a multiple of 16 bytes", c->head_dim);
  if (static_cast<int64_t>(c->kv_heads) * c->head_dim >= 65536)
    return report_errorf(DFL2_ERR_UNSUPPORTED, "kv_heads * head_dim must be below 65536");
  for (int64_t s : {c->layer_stride, c->page_stride, c->head_stride, c->slot_stride})
    if (s < 0 || s % per)
      return report_errorf(DFL2_ERR_INVALID_ARG,
                           "cache stride %lld: non-negative multiples of 16 bytes", (long long)s);
  return DFL2_OK;
}

dfl2_status check_cache_device(const dfl2_cache* c) {
  const PtrArg ptrs[] = {{c->k, "cache k", 16},         {c->v, "cache v", 16},
                         {c->table, "cache table", 4},  {c->refs, "cache refs", 4},
                         {c->free_bits, "cache free_bits", 4}};
  return check_args_device(ptrs, 5);
}

}  // namespace dfl2

#define DFL2_TRY(expr)              \
  do {                              \
    dfl2_status _st = (expr);       \
    if (_st != DFL2_OK) return _st; \
  } while (0)

using dfl2::PtrArg;

namespace {
template <int N>
dfl2_status check_all_host(const dfl2_cache* c, const PtrArg (&p)[N]) {
  DFL2_TRY(dfl2::check_cache_host(c));
  return dfl2::check_args_host(p, N);
}
template <int N>
dfl2_status check_all_device(const dfl2_cache* c, const PtrArg (&p)[N]) {
  DFL2_TRY(dfl2::check_cache_device(c));
  return dfl2::check_args_device(p, N);
}
dfl2_status launched(cudaError_t e, const char* what) {
  return e == cudaSuccess ? DFL2_OK : dfl2::report_cuda_error(e, what);
}
cudaStream_t cu(dfl2_stream s) { return reinterpret_cast<cudaStream_t>(s); }
}  // namespace

extern "C" {

dfl2_status dfl2_cache_reserve(const dfl2_cache* cache, int B, int T, const int32_t* table_rows,
                               const int32_t* length, const int32_t* count, int32_t* served,
                               dfl2_stream stream) {
  const PtrArg ptrs[] = {{table_rows, "table_rows", 4, true}, {length, "length", 4},
                         {count, "count", 4, true}, {served, "served", 4}};
  DFL2_TRY(dfl2::check_batch(B, T, 1 << 30, dfl2::kMaxSeqs));
  DFL2_TRY(check_all_host(cache, ptrs));
  // (the pages that all sequences lack are counted in 32 bits)
  if (int64_t(B) * std::min<int64_t>(cache->cols, T / cache->page_size + 2) > INT32_MAX)
    return dfl2::report_errorf(DFL2_ERR_UNSUPPORTED, "B=%d rows of %d entries: at most 2^31 - 1", B,
                               cache->cols);
  DFL2_TRY(check_all_device(cache, ptrs));
  const dfl2::TakeArgs a{dfl2::table_view(cache, table_rows, length, count, T), nullptr, served, B};
  return launched(dfl2::launch_take<false>(a, cu(stream)), "cache reserve launch");
}

dfl2_status dfl2_cache_write(const dfl2_cache* cache, int layer, int n_layers, const void* k_new,
                             const void* v_new, const int64_t* new_strides, int B, int T,
                             const int32_t* table_rows, const int32_t* length,
                             const int32_t* count, dfl2_stream stream) {
  const PtrArg ptrs[] = {{k_new, "k_new", 16, T == 0}, {v_new, "v_new", 16, T == 0},
                         {table_rows, "table_rows", 4, true}, {length, "length", 4},
                         {count, "count", 4, true}};
  DFL2_TRY(dfl2::check_batch(B, T, 1 << 30));
  DFL2_TRY(check_all_host(cache, ptrs));
  if (layer < 0 || n_layers < 1 || layer > cache->layers - n_layers)
    return dfl2::report_errorf(DFL2_ERR_INVALID_ARG, "layers %d .. %d of %d", layer,
                               layer + n_layers - 1, cache->layers);
  if (!new_strides) return dfl2::report_errorf(DFL2_ERR_INVALID_ARG, "new_strides is NULL");
  const int per = 16 / dfl2::elem_bytes(cache->dtype);
  const int dims[4] = {n_layers, B, T, cache->kv_heads};
  for (int i = 0; i < 4; ++i)
    if (dims[i] > 1 && (new_strides[i] < 0 || new_strides[i] % per))
      return dfl2::report_errorf(DFL2_ERR_INVALID_ARG,
                                 "new_strides[%d] = %lld: non-negative multiples of 16 bytes", i,
                                 (long long)new_strides[i]);
  DFL2_TRY(check_all_device(cache, ptrs));
  if (T == 0) return DFL2_OK;
  const dfl2::WriteArgs a{dfl2::table_view(cache, table_rows, length, count, T),
                          dfl2::row_view(cache),
                          static_cast<const uint4*>(k_new),
                          static_cast<const uint4*>(v_new),
                          new_strides[0] / per,
                          new_strides[1] / per,
                          new_strides[2] / per,
                          new_strides[3] / per,
                          layer,
                          n_layers,
                          B};
  const int blocks = dfl2::copy_blocks(static_cast<int64_t>(n_layers) * B * T, 8);
  return launched(
      dfl2::launch_k(dfl2::write_kernel, dim3(blocks), dim3(256), 0, cu(stream), true, a),
      "cache write launch");
}

dfl2_status dfl2_cache_compact(const dfl2_cache* cache, int B, int T, const int32_t* table_rows,
                               const int32_t* length, const int32_t* count, const int32_t* path,
                               const int32_t* n_path, int32_t* new_length, dfl2_stream stream) {
  const PtrArg ptrs[] = {{table_rows, "table_rows", 4, true}, {length, "length", 4},
                         {count, "count", 4, true}, {path, "path", 4}, {n_path, "n_path", 4},
                         {new_length, "new_length", 4}};
  DFL2_TRY(dfl2::check_batch(B, T, dfl2::kMaxTree));
  DFL2_TRY(check_all_host(cache, ptrs));
  DFL2_TRY(check_all_device(cache, ptrs));
  const dfl2::CompactArgs a{dfl2::table_view(cache, table_rows, length, count, T),
                            dfl2::row_view(cache), path, n_path, new_length, cache->layers, B};
  // (at most 4096 layers of 2 x 16384 columns of a sequence: an int holds them; clusters
  // of more than 8 blocks are not portable)
  const int64_t columns = static_cast<int64_t>(cache->layers) * 2 * a.r.chunks;
  int blocks = 1;
  while (blocks < dfl2::kMoveBlocks && int64_t(blocks) * dfl2::kMoveThreads < columns) blocks *= 2;
  const cudaError_t e = dfl2::launch_kc(dfl2::compact_kernel, dim3(blocks, B),
                                        dim3(dfl2::kMoveThreads), 0, cu(stream), true, blocks, a);
  return launched(e, "cache compact launch");
}

dfl2_status dfl2_cache_fork(const dfl2_cache* cache, int n, const int32_t* src, const int32_t* dst,
                            const int32_t* length, int32_t* served, dfl2_stream stream) {
  const PtrArg ptrs[] = {{src, "src", 4}, {dst, "dst", 4}, {length, "length", 4},
                         {served, "served", 4}};
  DFL2_TRY(dfl2::check_batch(n, 0, 0, dfl2::kMaxSeqs));
  DFL2_TRY(check_all_host(cache, ptrs));
  DFL2_TRY(check_all_device(cache, ptrs));
  const dfl2::TakeArgs a{dfl2::table_view(cache, dst, length, nullptr, 0), src, served, n};
  cudaError_t e = dfl2::launch_take<true>(a, cu(stream));
  if (e == cudaSuccess) {
    const dfl2::ForkCopyArgs f{a.t, dfl2::row_view(cache), src, served, cache->layers, n};
    const int64_t items = static_cast<int64_t>(cache->layers) * n * cache->page_size;
    e = dfl2::launch_k(dfl2::fork_copy_kernel, dim3(dfl2::copy_blocks(items, 8)), dim3(256), 0,
                       cu(stream), true, f);
  }
  return launched(e, "cache fork launch");
}

dfl2_status dfl2_cache_free(const dfl2_cache* cache, int n, const int32_t* table_rows,
                            dfl2_stream stream) {
  const PtrArg ptrs[] = {{table_rows, "table_rows", 4}};
  DFL2_TRY(dfl2::check_batch(n, 0, 0));
  DFL2_TRY(check_all_host(cache, ptrs));
  DFL2_TRY(check_all_device(cache, ptrs));
  const dfl2::TableView t = dfl2::table_view(cache, table_rows, nullptr, nullptr, 0);
  return launched(dfl2::launch_k(dfl2::free_kernel, dim3(n), dim3(256), 0, cu(stream), true, t),
                  "cache free launch");
}

}  // extern "C"
