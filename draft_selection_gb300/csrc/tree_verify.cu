// Acceptance of a tree of sampled tokens (include/dfl2.h, dfl2_tree_verify).
//
// At a node the target's distribution is p and the children were drawn, one after the
// other, from q (16 candidates).  Each child in turn: x is kept with probability
// min(1, r(x) / d(x)) with r = p and d = q at first; a miss leaves r = max(0, r - d),
// normalised, and takes x out of d where the children were drawn without replacement.
// When no child is kept the next token is drawn from r.  Off the candidates r is p times
// one factor, so a test needs 16 numbers, and only the last draw a whole row of p.
//
// A cluster of blocks to a sequence.  Every block looks the candidates of all nodes up at
// once (two dependent loads, however deep the tree is) and walks the tree in its first
// warp, a lane to a candidate, in double precision; so the blocks need not exchange the
// path.  The row of the last draw is then cut into one range a warp.  The warps' sums are
// exchanged through distributed shared memory, and the warp whose range the drawn number
// falls in looks for the element.
// Sums of the row are pairs of floats (the exact error of every addition is kept, Knuth's
// two-sum): this GPU adds two doubles a cycle and SM, and the drawn index has to be that
// of the exact sums.
#include <cuda_runtime.h>

#include <algorithm>

#include "cache.cuh"

namespace dfl2 {
namespace {

constexpr unsigned kAll = 0xffffffffu;
constexpr int kThreads = 512, kWarps = kThreads / 32, kMaxCluster = 8;

struct TreeVerifyArgs {
  const float* p;
  const int32_t* tokens;
  const int32_t* parents;
  const int32_t* count;
  const int32_t* cand;
  const float* q;
  const float* u;
  int32_t* path;
  int32_t* n_path;
  int32_t* next;
  int T, V, replace;
  uint32_t* err;
};

// hi + lo += x, the rounding error of every addition kept in lo.
__device__ __forceinline__ void add_exact(float& hi, float& lo, float x) {
  const float s = __fadd_rn(hi, x);
  const float b = __fsub_rn(s, hi);
  lo = __fadd_rn(lo, __fadd_rn(__fsub_rn(hi, __fsub_rn(s, b)), __fsub_rn(x, b)));
  hi = s;
}
__device__ __forceinline__ double sum16(double x) {  // over the lanes of a half-warp
#pragma unroll
  for (int off = 8; off; off >>= 1) x += __shfl_xor_sync(kAll, x, off);
  return x;
}
__device__ __forceinline__ double scan32(double x) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const double y = __shfl_up_sync(kAll, x, off);
    if (lane >= off) x += y;
  }
  return x;
}

// The row of the last draw.  Rows need not begin on 16 bytes: elements are numbered from
// the 16-byte boundary at or before the row, `off` elements early.
struct Row {
  const float4* base;
  int off, V, vecs;
  // Elements 4 v - off .. + 3; 0 outside the row.
  __device__ __forceinline__ float4 at(int v) const {
    const int e = 4 * v - off;
    if (e >= 0 && e + 3 < V) return __ldg(base + v);
    const float* f = reinterpret_cast<const float*>(base + v);
    float4 x;
    x.x = e >= 0 && e < V ? f[0] : 0.f;
    x.y = e + 1 >= 0 && e + 1 < V ? f[1] : 0.f;
    x.z = e + 2 >= 0 && e + 2 < V ? f[2] : 0.f;
    x.w = e + 3 >= 0 && e + 3 < V ? f[3] : 0.f;
    return x;
  }
};

// What is drawn from: the row with the candidates' values replaced.  These are doubles
// (their rounding to float would move the borders of all later elements by 2^-25 of them),
// so they are added beside the row's, whose own values there count as 0.
struct Left {
  Row row;
  int vec;    // of this lane's candidate (lanes 0 .. 15; -1: none)
  int place;  // and which of the four
  double val;
  __device__ __forceinline__ bool within(int v0, int v1) const { return vec >= v0 && vec < v1; }
};
__device__ __forceinline__ void set4(float4& x, int e, float y) {
  if (e == 0) x.x = y;
  if (e == 1) x.y = y;
  if (e == 2) x.z = y;
  if (e == 3) x.w = y;
}

// The sum of vectors [v0, v1) by a warp, in every lane.
__device__ __forceinline__ double range_sum(const Left& a, int v0, int v1, int lane) {
  constexpr int kBatch = 8;
  float hi[4] = {0.f, 0.f, 0.f, 0.f}, lo[4] = {0.f, 0.f, 0.f, 0.f};
  for (int v = v0; v < v1; v += 32 * kBatch) {
    float4 x[kBatch];
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      const int at = v + 32 * j + lane;
      x[j] = at < v1 ? a.row.at(at) : make_float4(0.f, 0.f, 0.f, 0.f);
    }
    unsigned hit = __ballot_sync(kAll, a.within(v, min(v1, v + 32 * kBatch)));
    while (hit) {
      const int k = __ffs(hit) - 1;
      hit &= hit - 1;
      const int at = __shfl_sync(kAll, a.vec, k) - v, e = __shfl_sync(kAll, a.place, k);
      if ((at & 31) == lane)
#pragma unroll
        for (int j = 0; j < kBatch; ++j)
          if (j == at >> 5) set4(x[j], e, 0.f);
    }
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      add_exact(hi[0], lo[0], x[j].x);
      add_exact(hi[1], lo[1], x[j].y);
      add_exact(hi[2], lo[2], x[j].z);
      add_exact(hi[3], lo[3], x[j].w);
    }
  }
  float h = hi[0], l = lo[0];
#pragma unroll
  for (int j = 1; j < 4; ++j) {
    add_exact(h, l, hi[j]);
    l += lo[j];
  }
  double s = static_cast<double>(h) + static_cast<double>(l);
  if (a.within(v0, v1)) s += a.val;
#pragma unroll
  for (int off = 16; off; off >>= 1) s += __shfl_xor_sync(kAll, s, off);
  return s;
}

// The first element of vectors [v0, v1) whose running sum exceeds t, by a warp; the last
// one with mass if there is none, -1 if that is none either.
__device__ __noinline__ int range_find(const Left& a, int v0, int v1, double t, int lane) {
  double before = 0.;
  int last = -1;
  for (int v = v0; v < v1; v += 32) {
    const float4 x =
        v + lane < v1 ? a.row.at(v + lane) : make_float4(0.f, 0.f, 0.f, 0.f);
    double y[4] = {x.x, x.y, x.z, x.w};
    unsigned cand = __ballot_sync(kAll, a.within(v, min(v1, v + 32)));
    while (cand) {
      const int k = __ffs(cand) - 1;
      cand &= cand - 1;
      const int at = __shfl_sync(kAll, a.vec, k) - v, e = __shfl_sync(kAll, a.place, k);
      const double val = __shfl_sync(kAll, a.val, k);
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (at == lane && e == j) y[j] = val;
    }
    const double s = (y[0] + y[1]) + (y[2] + y[3]);
    const double to = before + scan32(s);
    const int e0 = 4 * (v + lane) - a.row.off;
    int m = -1;  // the lane's last element with mass, and the first past t
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (y[j] > 0.) m = j;
    const unsigned hit = __ballot_sync(kAll, to > t && m >= 0);
    if (hit) {
      double c = to - s;
      int e = m;
      bool found = false;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        c += y[j];
        if (!found && y[j] > 0. && c > t) {
          found = true;
          e = j;
        }
      }
      return __shfl_sync(kAll, e0 + e, __ffs(hit) - 1);
    }
    if (m >= 0) last = e0 + m;
    before = __shfl_sync(kAll, to, 31);
  }
  return __reduce_max_sync(kAll, last);
}

__global__ void __launch_bounds__(kThreads)
    tree_verify_kernel(const __grid_constant__ TreeVerifyArgs a) {
  __shared__ float r_s[kMaxTree][kCand], d_s[kMaxTree][kCand];
  __shared__ int8_t slot_s[kMaxTree];  // of a node's token among its parent's candidates
  __shared__ double val_s[kCand];      // the candidates' part of what is left
  __shared__ int vec_s[kCand];
  __shared__ float u_s[kMaxTree];
  __shared__ int node_s, got_s, owner_s;
  __shared__ double sums_s[kMaxCluster * kWarps];  // every warp of the cluster's
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int b = blockIdx.y, rank = blockIdx.x, ranks = gridDim.x;
  const int T = a.T, V = a.V;
  const int64_t at = static_cast<int64_t>(b) * T;
  cluster_arrive_relaxed();  // every block of the cluster has begun before one writes to another
  pdl_wait();
  pdl_launch_dependents();
  const int n = a.count ? max(0, min(T, a.count[b])) : T;

  // ---- every node's candidates: p and q, 0 for one out of range or named before ----
  for (int x = tid; x - lane < n * kCand; x += kThreads) {
    const bool in = x < n * kCand;
    const int c = in ? a.cand[at * kCand + x] : -1;
    float q = in ? a.q[at * kCand + x] : 0.f;
    const bool ok = static_cast<unsigned>(c) < static_cast<unsigned>(V);
    if (in && !ok) record_error(a.err, kDevErrBadIndex);
    float p = ok ? a.p[(at + x / kCand) * V + c] : 0.f;
    bool again = false;
#pragma unroll
    for (int k = 1; k < kCand; ++k) {
      const int y = __shfl_up_sync(kAll, c, k, kCand);
      again |= (lane & 15) >= k && y == c;
    }
    if (!ok || again) p = q = 0.f;
    if (in) {
      r_s[x / kCand][x % kCand] = p;
      d_s[x / kCand][x % kCand] = q > 0.f ? q : 0.f;
    }
  }
  int8_t slot = -1;
  if (tid < n) {
    const int up = a.parents[at + tid], x = a.tokens[at + tid];
    if (up >= 0 && up < tid) {
      const int4* c = reinterpret_cast<const int4*>(a.cand + (at + up) * kCand);
#pragma unroll
      for (int j = 3; j >= 0; --j) {
        const int4 y = __ldg(c + j);
        if (y.w == x) slot = 4 * j + 3;
        if (y.z == x) slot = 4 * j + 2;
        if (y.y == x) slot = 4 * j + 1;
        if (y.x == x) slot = 4 * j;
      }
    }
  }
  if (tid < kMaxTree) {
    slot_s[tid] = slot;
    if (tid < n) u_s[tid] = a.u[at + tid];
  }
  __syncthreads();

  // ---- the walk: lanes 0 .. 15 a candidate each (16 .. 31 do the same) ----
  if (warp == 0) {
    int par[kMaxTree / 32];
#pragma unroll
    for (int j = 0; j < kMaxTree / 32; ++j) {
      const int i = lane + 32 * j;
      par[j] = i < n && slot_s[i] >= 0 ? a.parents[at + i] : -1;
    }
    const int k = lane & 15;
    int cur = 0, len = 0;
    double r = 0., g = 1.;
    while (n > 0) {
      if (rank == 0 && lane == 0) a.path[at + len] = cur;
      ++len;
      const double p = r_s[cur][k];
      double d = d_s[cur][k];
      r = p;
      g = 1.;
      const double whole = fmax(0., 1. - sum16(p));
      double rest = whole;
      int took = -1;
      bool over = false;
#pragma unroll
      for (int j = 0; j < kMaxTree / 32; ++j) {
        unsigned kids = __ballot_sync(kAll, par[j] == cur);
        while (kids && took < 0 && !over) {
          const int i = 32 * j + __ffs(kids) - 1;
          kids &= kids - 1;
          const int s = slot_s[i];
          const double dk = __shfl_sync(kAll, d, s);
          if (!(dk > 0.)) continue;  // (its mass was taken by a sibling before)
          const double R = rest + sum16(r), D = sum16(d), rk = __shfl_sync(kAll, r, s);
          const double u = u_s[i];
          if (u * dk * R < rk * D) {
            took = i;
            break;
          }
          const double ir = 1. / R, id = 1. / D;
          r = fmax(0., r * ir - d * id);
          rest *= ir;
          g *= ir;
          if (!a.replace && k == s) d = 0.;
          if (!(rest + sum16(r) > 0.)) {  // p never exceeds q: p itself
            r = p;
            rest = whole;
            g = 1.;
            over = true;
          }
        }
      }
      if (took < 0) break;
      cur = took;
    }
    if (rank == 0) {
      for (int i = len + lane; i < T; i += 32) a.path[at + i] = -1;
      if (lane == 0) a.n_path[b] = len;
    }
    if (lane < kCand) {
      const int c = n > 0 ? a.cand[(at + cur) * kCand + k] : -1;
      bool again = false;
#pragma unroll
      for (int z = 1; z < kCand; ++z) {
        const int y = __shfl_up_sync(0xffffu, c, z, kCand);
        again |= k >= z && y == c;
      }
      vec_s[k] = again || static_cast<unsigned>(c) >= static_cast<unsigned>(V) ? -1 : c;
      val_s[k] = r / g;
    }
    if (lane == 0) node_s = cur;
  }
  __syncthreads();

  // ---- the last draw ----
  Left left;
  const int64_t start = (at + node_s) * V;
  left.row.off = static_cast<int>(start & 3);
  left.row.base = reinterpret_cast<const float4*>(a.p + (start - left.row.off));
  left.row.V = V;
  left.row.vecs = (V + left.row.off + 3) / 4;
  const int c = lane < kCand ? vec_s[lane] : -1;
  left.vec = c < 0 ? -1 : (c + left.row.off) >> 2;
  left.place = (c + left.row.off) & 3;
  left.val = lane < kCand ? val_s[lane] : 0.;
  const int total_warps = ranks * kWarps;
  cluster_wait();
  auto range_at = [&](int w) {
    return static_cast<int>(static_cast<int64_t>(left.row.vecs) * w / total_warps);
  };
  for (int pass = 0; pass < 2 && n > 0; ++pass) {
    const int w = rank * kWarps + warp;
    const double s = range_sum(left, range_at(w), range_at(w + 1), lane);
    if (lane < ranks) {  // to every block of the cluster
      const uint32_t to = dsmem_addr(&sums_s[w], lane);
      asm volatile("st.shared::cluster.f64 [%0], %1;" ::"r"(to), "d"(s) : "memory");
    }
    cluster_sync_all();
    if (warp == 0) {
      constexpr int kEach = kMaxCluster * kWarps / 32;
      double x[kEach], sum = 0.;
#pragma unroll
      for (int j = 0; j < kEach; ++j) {
        const int i = lane * kEach + j;
        x[j] = i < total_warps ? sums_s[i] : 0.;
        sum += x[j];
      }
      const double to = scan32(sum);
      const double total = __shfl_sync(kAll, to, 31), t = u_s[0] * total;
      double run = to - sum;
      int mine = -1, last = -1;
      double rel = 0., rel_last = 0.;
#pragma unroll
      for (int j = 0; j < kEach; ++j) {
        if (x[j] > 0.) {
          last = lane * kEach + j;
          rel_last = t - run;
          if (mine < 0 && run + x[j] > t) {
            mine = last;
            rel = rel_last;
          }
        }
        run += x[j];
      }
      unsigned hit = __ballot_sync(kAll, mine >= 0);
      int src = hit ? __ffs(hit) - 1 : 0;
      if (!hit) {  // rounding left none: the last range with mass
        hit = __ballot_sync(kAll, last >= 0);
        src = hit ? 31 - __clz(hit) : 0;
        mine = last;
        rel = rel_last;
      }
      const int owner = hit ? __shfl_sync(kAll, mine, src) : -1;
      rel = __shfl_sync(kAll, rel, src);
      int got = -1;
      if (owner >= 0 && owner / kWarps == rank)
        got = range_find(left, range_at(owner), range_at(owner + 1), rel, lane);
      if (lane == 0) {
        owner_s = owner;
        got_s = got;
      }
    }
    __syncthreads();
    if (owner_s >= 0) break;
    left.vec = -1;  // what is left sums to nothing: the row itself
    cluster_sync_all();
  }
  if (tid == 0) {
    const int owner = n > 0 ? owner_s : -1;
    if (owner < 0 ? rank == 0 : owner / kWarps == rank) a.next[b] = owner < 0 ? -1 : got_s;
  }
  cluster_sync_all();  // no block ends while another may still write to it
}

}  // namespace
}  // namespace dfl2

#define DFL2_TRY(expr)              \
  do {                              \
    dfl2_status _st = (expr);       \
    if (_st != DFL2_OK) return _st; \
  } while (0)

extern "C" dfl2_status dfl2_tree_verify(const float* p, int B, int T, int V, const int32_t* tokens,
                                        const int32_t* parents, const int32_t* count,
                                        const int32_t* cand_idx, const float* q, const float* u,
                                        int replace, int32_t* path, int32_t* n_path,
                                        int32_t* next_token, dfl2_stream stream) {
  const dfl2::PtrArg ptrs[] = {{p, "p", 16}, {tokens, "tokens", 4}, {parents, "parents", 4},
                               {count, "count", 4, true}, {cand_idx, "cand_idx", 16}, {q, "q", 4},
                               {u, "u", 4}, {path, "path", 4}, {n_path, "n_path", 4},
                               {next_token, "next_token", 4}};
  if (B < 1 || T < 1 || V < 1)
    return dfl2::report_errorf(DFL2_ERR_INVALID_ARG, "B=%d, T=%d and V=%d must be >= 1", B, T, V);
  if (B > dfl2::kMaxBatch || T > dfl2::kMaxTree || V > (1 << 30))
    return dfl2::report_errorf(DFL2_ERR_UNSUPPORTED,
                               "B=%d, T=%d, V=%d: at most %d trees of %d nodes, 2^30 tokens", B, T,
                               V, dfl2::kMaxBatch, dfl2::kMaxTree);
  DFL2_TRY(dfl2::check_args_host(ptrs, 10));
  DFL2_TRY(dfl2::check_args_device(ptrs, 10));
  const dfl2::TreeVerifyArgs a{p,    tokens, parents, count,      cand_idx, q, u,
                               path, n_path, next_token, T, V, replace != 0,
                               dfl2::device_error_word()};
  // as many blocks a sequence as are resident at once (four an SM), and have 4096 elements
  const int most = 4 * dfl2::device_info().sms;
  int ranks = dfl2::kMaxCluster;
  while (ranks > 1 && (int64_t(ranks) * B > most || V / ranks < 4096)) ranks /= 2;
  const cudaError_t e =
      dfl2::launch_kc(dfl2::tree_verify_kernel, dim3(ranks, B), dim3(dfl2::kThreads), 0,
                      reinterpret_cast<cudaStream_t>(stream), true, ranks, a);
  return e == cudaSuccess ? DFL2_OK : dfl2::report_cuda_error(e, "tree verify launch");
}
