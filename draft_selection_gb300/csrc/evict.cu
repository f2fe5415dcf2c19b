// Eviction from the paged cache by accumulated attention weight (include/dfl2.h,
// dfl2_cache_evict).
//
// evict_select_kernel, a block to a sequence: of the positions that are neither sinks nor
// recent, those with the m largest weights stay.  The m-th largest is found by its bits, 11
// at a time from the top, with a histogram in shared memory; equal weights stay from the
// lowest position on.  A position's new place is the number of those that stay before it,
// so it is known from two counts: of larger weights, and of equal ones.  The block checks
// that every page is there and that no page it would write is shared, moves the weights, and
// leaves the rows' old and new places for the second kernel.
//
// evict_move_kernel moves the rows of keys and values, as 16-byte columns: a warp's lanes
// are 32 columns of one layer's K or V, its block's warps share the rows of these columns,
// 8 rows a warp at a time.  A row's new place is at or before its old one, and a place that
// is written holds either nothing that stays or a row of the same step or an earlier one; so
// reading a step ahead is safe, and one barrier a step keeps a row from being overwritten
// before another warp has read it.  The first block gives the pages behind the rows back.
// Bound by HBM: each row that moves is read and written once (16 sequences of up to 4000
// positions at 2000, 16 layers, 8 heads x 128 channels, 2.6 GB: 419 us, 6.3 TB/s).  One
// sequence at 1024 positions, 32 layers: 44 us, 6.1 TB/s, with 16 warps a block (8: 50), after
// 10 us of selection: a chain of two or three histograms, a scan and a look at the pages.
#include <cuda_runtime.h>

#include <algorithm>

#include "cache.cuh"

namespace dfl2 {
namespace {

constexpr unsigned kAll = 0xffffffffu;
constexpr int kSelThreads = 1024, kSelWarps = kSelThreads / 32;
constexpr int kPer = 8;                          // positions a thread holds at most
constexpr int kBins = 2048;

struct Move {
  int64_t from, to;  // of a row, in 16-byte units from the layer and head's first
};
struct alignas(16) Plan {
  int moves;        // rows that move, to the places keep - moves ..
  int row, len, new_len;  // row < 0: nothing to do
};

struct EvictArgs {
  TableView t;
  int keep, sinks, recent;
  float* weight;
  int32_t* kept;
  int32_t* new_length;
  int32_t* served;
  Move* moves;  // [B][keep], of place i at i
  Plan* plans;  // [B]
  int64_t page_stride, slot_stride;  // 16-byte units
};

// Larger for larger weights; NaN counts as -inf.
__device__ __forceinline__ uint32_t weight_key(float w) {
  return ord_f32(w == w ? w : __uint_as_float(0xFF800000u));
}

__global__ void __launch_bounds__(kSelThreads)
    evict_select_kernel(const __grid_constant__ EvictArgs a) {
  __shared__ int hist[kBins];
  __shared__ uint32_t sums[2][kSelWarps];
  __shared__ int digit_s, left_s, all_s, first_s;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, b = blockIdx.x;
  pdl_wait();
  pdl_launch_dependents();
  const int len = a.t.length[b], row = a.t.row_of(b);
  const bool fits = row >= 0 && a.t.checked_length(len) &&
                    len <= static_cast<int64_t>(a.t.cols) << a.t.page_shift;
  int32_t* kept = a.kept + static_cast<int64_t>(b) * a.keep;
  const int ps = 1 << a.t.page_shift;
  const int32_t* table = a.t.table + static_cast<int64_t>(max(0, row)) * a.t.cols;
  // Whether (for this thread) every page of the sequence is there, and none shared that is
  // written, which are those of places `first` .. keep - 1.
  auto pages_good = [&](int first) {
    bool good = true;
    for (int c = tid; c < (len + ps - 1) >> a.t.page_shift; c += kSelThreads) {
      const int p = table[c];
      if (static_cast<unsigned>(p) >= static_cast<unsigned>(a.t.pages))
        good = false;
      else if (first < a.keep && c >= first >> a.t.page_shift &&
               c <= (a.keep - 1) >> a.t.page_shift)
        good &= a.t.refs[p] == 1;
    }
    return good;
  };
  if (!fits || len <= a.keep) {  // (the block as one)
    const bool good = __syncthreads_and(fits && pages_good(a.keep));
    for (int i = tid; i < a.keep; i += kSelThreads) kept[i] = good && i < len ? i : -1;
    if (tid == 0) {
      a.plans[b] = Plan{0, -1, len, len};
      a.served[b] = good;
      a.new_length[b] = len;
    }
    return;
  }
  float* weight = a.weight + (static_cast<int64_t>(row) * a.t.cols << a.t.page_shift);
  const int recent0 = len - a.recent;  // the first recent position
  // A block holds kSelThreads times `per` positions at a time, so that short sequences too
  // are spread over all warps (1041 positions: 11 us with eight to a thread in any case).
  const int per = min(kPer, (len - a.sinks - 1) / kSelThreads + 1);
  const int chunk = kSelThreads * per, chunks = (len - a.sinks - 1) / chunk + 1;

  // A thread's positions of a chunk: a warp's are contiguous, so that ballots give their order.
  float w[kPer];
  auto pos_of = [&](int c, int j) { return a.sinks + c * chunk + (warp * per + j) * 32 + lane; };
  auto load = [&](int c) {
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      const int p = pos_of(c, j);
      w[j] = j < per && p < len ? weight[p] : 0.f;
    }
  };
  load(0);

  // ---- the smallest weight that stays (its key), and how many of that stay ----
  int m = a.keep - a.sinks - a.recent;
  uint32_t key = 0xFFFFFFFEu;  // (m = 0: above every weight's)
  if (m > 0) {
    key = 0;
#pragma unroll 1
    for (int shift : {21, 10, 0}) {
      const uint32_t digits = shift == 0 ? 1024u : 2048u, mask = digits - 1;
      const uint32_t above = shift == 21 ? 0u : shift == 10 ? 0xFFE00000u : 0xFFFFFC00u;
      for (int i = tid; i < kBins; i += kSelThreads) hist[i] = 0;
      __syncthreads();
      for (int c = 0; c < chunks; ++c) {
        if (chunks > 1) load(c);
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
          const uint32_t k = weight_key(w[j]);
          if (j < per && pos_of(c, j) < recent0 && (k & above) == key)
            atomicAdd(&hist[mask - (k >> shift & mask)], 1);
        }
      }
      __syncthreads();
      // two bins a thread, the largest digits first
      const int x0 = hist[2 * tid], x1 = hist[2 * tid + 1];
      int sum = x0 + x1;
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const int y = __shfl_up_sync(kAll, sum, off);
        if (lane >= off) sum += y;
      }
      if (lane == 31) sums[0][warp] = sum;
      __syncthreads();
      int before = static_cast<int>(sums[0][lane]);
      before = __reduce_add_sync(kAll, lane < warp ? before : 0) + sum - x0 - x1;
      // (exactly one bin holds the m-th)
      if (before < m && m <= before + x0) {
        digit_s = 2 * tid;
        left_s = m - before;
        all_s = x0;
      } else if (before + x0 < m && m <= before + x0 + x1) {
        digit_s = 2 * tid + 1;
        left_s = m - before - x0;
        all_s = x1;
      }
      __syncthreads();
      key |= (mask - static_cast<uint32_t>(digit_s)) << shift;
      m = left_s;
      if (m == all_s) break;  // every weight of these digits stays: they need no further ones
    }
  }

  // The positions of chunk c that stay: a bit for each of a warp's (gt: of larger weights, eq:
  // of equal ones), and the numbers of both (g, e) before the warp's first; larger, equal: in
  // the chunks before.
  int larger = 0, equal = 0;
  unsigned gt[kPer], eq[kPer];
  int g = 0, e = 0;
  auto stay = [&](int c) {
    uint32_t n = 0;  // larger ones, and equal ones << 16
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      gt[j] = eq[j] = 0;
      if (j >= per) continue;
      const int p = pos_of(c, j);
      const uint32_t k = p >= recent0 ? 0xFFFFFFFFu : weight_key(w[j]);
      gt[j] = __ballot_sync(kAll, p < len && k > key);
      eq[j] = __ballot_sync(kAll, p < len && k == key);
      n += __popc(gt[j]) + (__popc(eq[j]) << 16);
    }
    if (lane == 0) sums[c & 1][warp] = n;
    __syncthreads();
    const uint32_t x = sums[c & 1][lane];
    const uint32_t before = __reduce_add_sync(kAll, lane < warp ? x : 0u);
    const uint32_t all = __reduce_add_sync(kAll, x);
    g = larger + static_cast<int>(before & 0xFFFF);
    e = equal + static_cast<int>(before >> 16);
    larger += static_cast<int>(all & 0xFFFF);
    equal += static_cast<int>(all >> 16);
  };
  const unsigned lower = (1u << lane) - 1;

  // ---- the first place whose row moves: the first position that goes ----
  if (tid == 0) first_s = len;
  int first = len;
  for (int c = 0; c < chunks && first == len; ++c) {
    if (chunks > 1) load(c);
    stay(c);
    int gone = len;
#pragma unroll
    for (int j = kPer - 1; j >= 0; --j) {
      const int p = pos_of(c, j);
      int eb = e;
#pragma unroll
      for (int z = 0; z < kPer; ++z)
        if (z < j) eb += __popc(eq[z]);
      const bool stays = gt[j] >> lane & 1 ||
                         (eq[j] >> lane & 1 && eb + __popc(eq[j] & lower) < m);
      if (j < per && p < len && !stays) gone = p;
    }
    gone = __reduce_min_sync(kAll, gone);
    if (lane == 0 && gone < len) atomicMin(&first_s, gone);
    __syncthreads();
    first = first_s;
  }

  // ---- every page there, and none shared that is written ----
  const bool good = __syncthreads_and(pages_good(first));
  if (tid == 0) {
    a.plans[b] = Plan{good ? a.keep - min(first, a.keep) : 0, good ? row : -1, len, a.keep};
    a.served[b] = good;
    a.new_length[b] = good ? a.keep : len;
  }
  if (!good) {
    for (int i = tid; i < a.keep; i += kSelThreads) kept[i] = -1;
    return;
  }

  // ---- the new places ----
  for (int i = tid; i < a.sinks; i += kSelThreads) kept[i] = i;
  larger = equal = 0;
  Move* moves = a.moves + static_cast<int64_t>(b) * a.keep;
  auto place = [&](int p) {
    return table[p >> a.t.page_shift] * a.page_stride + (p & (ps - 1)) * a.slot_stride;
  };
  for (int c = 0; c < chunks; ++c) {
    if (chunks > 1) {
      load(c);
      stay(c);  // (its barrier: every weight of the chunk has been read)
    }
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      if (j >= per) break;
      const int p = pos_of(c, j);
      const int eb = e + __popc(eq[j] & lower);
      const bool is_eq = eq[j] >> lane & 1;
      if (gt[j] >> lane & 1 || (is_eq && eb < m)) {
        const int i = a.sinks + g + __popc(gt[j] & lower) + min(eb, m);
        kept[i] = p;
        if (i != p) {
          weight[i] = w[j];
          moves[i] = Move{place(p), place(i)};
        }
      }
      g += __popc(gt[j]);
      e += __popc(eq[j]);
    }
    __syncthreads();  // (a chunk's sums are read before the one after the next writes them)
  }
}

struct EvictMoveArgs {
  TableView t;
  uint4* k;
  uint4* v;
  int64_t layer, head;     // strides, 16-byte units
  int columns, chunks, per_head;  // of all layers' K and V; of a position's K in one; of a head's
  int keep;
  const Move* moves;
  const Plan* plans;
};

constexpr int kRows = 8;  // of a warp at a time

template <int kWarps>
__global__ void __launch_bounds__(kWarps * 32)
    evict_move_kernel(const __grid_constant__ EvictMoveArgs a) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, b = blockIdx.y;
  const int c = blockIdx.x * 32 + lane;
  const int l = c / (2 * a.chunks), in = c - l * 2 * a.chunks;
  const bool is_v = in >= a.chunks;
  const int x = in - (is_v ? a.chunks : 0), h = x / a.per_head;
  uint4* base = (is_v ? a.v : a.k) + l * a.layer + h * a.head + (x - h * a.per_head);
  const bool mine = c < a.columns;
  pdl_wait();
  pdl_launch_dependents();
  const Plan plan = a.plans[b];
  if (plan.row < 0) return;
  const Move* moves = a.moves + static_cast<int64_t>(b) * a.keep + (a.keep - plan.moves);
  constexpr int kStep = kWarps * kRows;
  // lane j < 8: row j of the warp's next step
  auto look = [&](int i) {
    return lane < kRows && i + lane < plan.moves ? moves[i + lane] : Move{0, 0};
  };
  int i = warp * kRows;
  Move at = look(i);
  uint4 y[kRows];
  auto read = [&](int i0, const Move& m) {
#pragma unroll
    for (int j = 0; j < kRows; ++j) {
      const int64_t from = __shfl_sync(kAll, m.from, j);
      if (mine && i0 + j < plan.moves) y[j] = base[from];
    }
  };
  const int steps = (plan.moves + kStep - 1) / kStep;
  for (int s = 0; s < steps; ++s, i += kStep) {
    read(i, at);
    const Move next = look(i + kStep);
    __syncthreads();  // every warp has read its rows of this step
#pragma unroll
    for (int j = 0; j < kRows; ++j) {
      const int64_t to = __shfl_sync(kAll, at.to, j);
      if (mine && i + j < plan.moves) base[to] = y[j];
    }
    at = next;
  }
  if (blockIdx.x > 0) return;
  const int ps = 1 << a.t.page_shift;
  int32_t* r = a.t.table + static_cast<int64_t>(plan.row) * a.t.cols;
  for (int e = ((plan.new_len + ps - 1) >> a.t.page_shift) + threadIdx.x;
       e < (plan.len + ps - 1) >> a.t.page_shift; e += kWarps * 32) {
    const int p = atomicExch(&r[e], -1);
    if (p != -1) drop_page(a.t, p);
  }
}

size_t plans_bytes(int B) { return align_up(size_t(B) * sizeof(Plan), 256); }

dfl2_status check_sizes(int B, int keep) {
  if (B < 1 || keep < 1)
    return report_errorf(DFL2_ERR_INVALID_ARG, "B=%d and keep=%d must be >= 1", B, keep);
  if (B > kMaxBatch || keep > kMaxLen)
    return report_errorf(DFL2_ERR_UNSUPPORTED, "B=%d, keep=%d: at most %d sequences, 2^30 positions",
                         B, keep, kMaxBatch);
  return DFL2_OK;
}

}  // namespace
}  // namespace dfl2

#define DFL2_TRY(expr)              \
  do {                              \
    dfl2_status _st = (expr);       \
    if (_st != DFL2_OK) return _st; \
  } while (0)

extern "C" {

size_t dfl2_cache_evict_workspace_size(int B, int keep) {
  if (dfl2::check_sizes(B, keep) != DFL2_OK) return 0;
  return dfl2::plans_bytes(B) + size_t(B) * keep * sizeof(dfl2::Move) + 256;  // (to align the base)
}

dfl2_status dfl2_cache_evict(const dfl2_cache* cache, int B, const int32_t* table_rows,
                             const int32_t* length, int keep, int sinks, int recent, float* weight,
                             int32_t* kept, int32_t* new_length, int32_t* served, void* ws,
                             size_t ws_bytes, dfl2_stream stream) {
  const dfl2::PtrArg ptrs[] = {{table_rows, "table_rows", 4, true}, {length, "length", 4},
                               {weight, "weight", 4}, {kept, "kept", 4},
                               {new_length, "new_length", 4}, {served, "served", 4}};
  DFL2_TRY(dfl2::check_sizes(B, keep));
  DFL2_TRY(dfl2::check_cache_host(cache));
  DFL2_TRY(dfl2::check_args_host(ptrs, 6));
  if (sinks < 0 || recent < 0 || int64_t(sinks) + recent > keep)
    return dfl2::report_errorf(DFL2_ERR_INVALID_ARG,
                               "sinks=%d and recent=%d: at least 0, together at most keep=%d", sinks,
                               recent, keep);
  const size_t need = dfl2::plans_bytes(B) + size_t(B) * keep * sizeof(dfl2::Move) + 256;
  if (!ws || ws_bytes < need)
    return dfl2::report_errorf(DFL2_ERR_WORKSPACE, "workspace of %zu bytes < %zu needed",
                               ws ? ws_bytes : size_t(0), need);
  DFL2_TRY(dfl2::check_args_device(ptrs, 6));
  DFL2_TRY(dfl2::check_cache_device(cache));
  const dfl2::PtrArg wsp[] = {{ws, "workspace", 1}};
  DFL2_TRY(dfl2::check_args_device(wsp, 1));
  uint8_t* w = reinterpret_cast<uint8_t*>(dfl2::align_up(reinterpret_cast<uintptr_t>(ws), 256));
  const int per = 16 / dfl2::elem_bytes(cache->dtype);
  dfl2::EvictArgs a{};
  a.t = dfl2::table_view(cache, table_rows, length, nullptr, 0);
  a.keep = keep;
  a.sinks = sinks;
  a.recent = recent;
  a.weight = weight;
  a.kept = kept;
  a.new_length = new_length;
  a.served = served;
  a.plans = reinterpret_cast<dfl2::Plan*>(w);
  a.moves = reinterpret_cast<dfl2::Move*>(w + dfl2::plans_bytes(B));
  a.page_stride = cache->page_stride / per;
  a.slot_stride = cache->slot_stride / per;
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e = dfl2::launch_k(dfl2::evict_select_kernel, dim3(B), dim3(dfl2::kSelThreads), 0, s,
                                 true, a);
  if (e == cudaSuccess) {
    dfl2::EvictMoveArgs m{};
    m.t = a.t;
    m.k = static_cast<uint4*>(cache->k);
    m.v = static_cast<uint4*>(cache->v);
    m.layer = cache->layer_stride / per;
    m.head = cache->head_stride / per;
    m.per_head = cache->head_dim / per;
    m.chunks = cache->kv_heads * m.per_head;
    m.columns = cache->layers * 2 * m.chunks;  // (below 4096 x 2 x 16384)
    m.keep = keep;
    m.moves = a.moves;
    m.plans = a.plans;
    // Few columns: more warps share the rows, so that enough of them are on their way.  Both
    // launches, with 8, 16 and 32 warps, 1041 positions at 1024, and 8192 at 4096: 64 blocks 30,
    // 31, 27 us and 89, 73, 64; 128 blocks 47, 41, 39 and 115, 102, 103; 256 blocks 74, 67, 61
    // and 184, 194, 184; 384 blocks 99, 87, 88 and 278, 283, 261; 1024 blocks 205, 202, 209.  So
    // it matters below a block an SM; past two 8 warps are within 12% of the best.
    const dim3 grid((m.columns + 31) / 32, B);
    const int64_t blocks = int64_t(grid.x) * B;
    if (blocks < dfl2::device_info().sms)
      e = dfl2::launch_k(dfl2::evict_move_kernel<32>, grid, dim3(1024), 0, s, true, m);
    else if (blocks < 2 * dfl2::device_info().sms)
      e = dfl2::launch_k(dfl2::evict_move_kernel<16>, grid, dim3(512), 0, s, true, m);
    else
      e = dfl2::launch_k(dfl2::evict_move_kernel<8>, grid, dim3(256), 0, s, true, m);
  }
  return e == cudaSuccess ? DFL2_OK : dfl2::report_cuda_error(e, "cache evict launch");
}

}  // extern "C"
