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
// Numbers are unevaluated sums of two floats (about 46 bits): decisions and the drawn index
// have to be those of the exact sums, and this GPU's doubles are slow (two additions a cycle
// and SM, 60 cycles each).
#include <cuda_runtime.h>

#include <algorithm>

#include "cache.cuh"

namespace dfl2 {
namespace {

constexpr unsigned kAll = 0xffffffffu;
constexpr int kThreads = 512, kWarps = kThreads / 32, kCtas = 2, kMaxCluster = 8;

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

// A number as the sum of two floats, the second at most half a unit of the first's last
// place.  Additions and products by Knuth's two-sum and the fused remainder of a product.
struct Pair {
  float hi, lo;
};
__device__ __forceinline__ Pair quick(float a, float b) {  // |a| >= |b|
  const float s = __fadd_rn(a, b);
  return {s, __fsub_rn(b, __fsub_rn(s, a))};
}
__device__ __forceinline__ Pair two_sum(float a, float b) {
  const float s = __fadd_rn(a, b), c = __fsub_rn(s, a);
  return {s, __fadd_rn(__fsub_rn(a, __fsub_rn(s, c)), __fsub_rn(b, c))};
}
__device__ __forceinline__ Pair operator+(Pair a, Pair b) {
  const Pair s = two_sum(a.hi, b.hi);
  return quick(s.hi, __fadd_rn(s.lo, __fadd_rn(a.lo, b.lo)));
}
__device__ __forceinline__ Pair operator-(Pair a, Pair b) { return a + Pair{-b.hi, -b.lo}; }
__device__ __forceinline__ Pair operator*(Pair a, Pair b) {
  const float p = __fmul_rn(a.hi, b.hi);
  const float e = __fmaf_rn(a.hi, b.hi, -p);
  return quick(p, __fmaf_rn(a.hi, b.lo, __fmaf_rn(a.lo, b.hi, e)));
}
__device__ __forceinline__ Pair operator*(Pair a, float b) { return a * Pair{b, 0.f}; }
__device__ __forceinline__ Pair scaled(Pair a, float f) { return {a.hi * f, a.lo * f}; }  // f = 2^n
__device__ __forceinline__ Pair operator/(Pair a, Pair b) {
  const float q = __fdiv_rn(a.hi, b.hi);
  const Pair r = a - b * q;
  return quick(q, __fdiv_rn(r.hi, b.hi));
}
__device__ __forceinline__ bool operator<(Pair a, Pair b) {
  return a.hi < b.hi || (a.hi == b.hi && a.lo < b.lo);
}
__device__ __forceinline__ Pair shfl(Pair x, int lane) {
  return {__shfl_sync(kAll, x.hi, lane), __shfl_sync(kAll, x.lo, lane)};
}
__device__ __forceinline__ Pair shfl_xor(Pair x, int bit) {
  return {__shfl_xor_sync(kAll, x.hi, bit), __shfl_xor_sync(kAll, x.lo, bit)};
}
__device__ __forceinline__ Pair sum16(Pair x) {  // over the lanes of a half-warp
#pragma unroll
  for (int off = 8; off; off >>= 1) x = x + shfl_xor(x, off);
  return x;
}
__device__ __forceinline__ Pair scan32(Pair x) {  // over this lane and those before it
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const Pair y = {__shfl_up_sync(kAll, x.hi, off), __shfl_up_sync(kAll, x.lo, off)};
    if (lane >= off) x = x + y;
  }
  return x;
}
// 2^-e for x in [2^e, 2^(e+1)), x normal and e within -125 .. 125; 1 otherwise.
__device__ __forceinline__ float to_one(float x) {
  const int e = static_cast<int>(__float_as_uint(x) >> 23);  // (x >= 0)
  return e < 2 || e > 252 ? 1.f : __uint_as_float(static_cast<uint32_t>(254 - e) << 23);
}

// The row of the last draw.  Rows need not begin on 16 bytes: elements are numbered from
// the 16-byte boundary at or before the row, `off` elements early.
struct Row {
  const float4* base;
  int off, V, vecs;
  // Elements 4 v - off .. + 3 of a row, 0 where v is past `end` or not wholly inside.
  __device__ __forceinline__ float4 inner(int v, int end) const {
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
    const int e = 4 * v - off;
    if (v < end && e >= 0 && e + 3 < V) x = __ldg(base + v);
    return x;
  }
  // The row's first and last vectors where they are cut, else x.
  __device__ __forceinline__ float4 ends(float4 x, int v) const {
    const int e = 4 * v - off;
    if (e < 0 || (e < V && e + 3 >= V)) {
      const float* f = reinterpret_cast<const float*>(base + v);
      x.x = e >= 0 ? f[0] : 0.f;
      x.y = e + 1 >= 0 && e + 1 < V ? f[1] : 0.f;
      x.z = e + 2 >= 0 && e + 2 < V ? f[2] : 0.f;
      x.w = e + 3 < V ? f[3] : 0.f;
    }
    return x;
  }
};

// Two floats in one register pair, for the two-sums of the row.
__device__ __forceinline__ uint64_t pack(float x, float y) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
  return r;
}
__device__ __forceinline__ void unpack(uint64_t r, float& x, float& y) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(r));
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t sub2(uint64_t a, uint64_t b) {  // a - b, as b (-1) + a
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(b), "l"(0xBF800000BF800000ull), "l"(a));
  return r;
}
// hi + lo += x, twice.
__device__ __forceinline__ void add_exact2(uint64_t& hi, uint64_t& lo, uint64_t x) {
  const uint64_t s = add2(hi, x), c = sub2(s, hi);
  lo = add2(lo, add2(sub2(hi, sub2(s, c)), sub2(x, c)));
  hi = s;
}

// What is drawn from: the row with the candidates' values replaced.  These are pairs (their
// rounding to a float would move the borders of all later elements by 2^-25 of them), so
// they are added beside the row's, whose own values there count as 0.
struct Left {
  Row row;
  const int* at;    // [16], the candidates' elements; -1: none
  const Pair* val;
  // The candidates in vectors [v0, v1), by a warp.
  __device__ __forceinline__ unsigned among(int v0, int v1) const {
    const int lane = threadIdx.x & 31, c = lane < kCand ? at[lane] : -1;
    const int v = (c + row.off) >> 2;
    return __ballot_sync(kAll, c >= 0 && v >= v0 && v < v1);
  }
  // The sum of vectors v, v + step, .. below v1; cand: the candidates that may be there.
  __device__ __forceinline__ Pair sum(int v, int v1, int step, unsigned cand) const {
    constexpr int kBatch = 8;
    uint64_t hi[2] = {0, 0}, lo[2] = {0, 0};
#pragma unroll 1
    for (; v < v1; v += step * kBatch) {
      float4 x[kBatch];
#pragma unroll
      for (int j = 0; j < kBatch; ++j) x[j] = row.inner(v + step * j, v1);
      if (cand || v < step || v + step * kBatch >= row.vecs)
#pragma unroll
        for (int j = 0; j < kBatch; ++j)
          if (v + step * j < v1) x[j] = odd(x[j], v + step * j, cand);
#pragma unroll
      for (int j = 0; j < kBatch; ++j) {
        if (v + step * j >= v1) break;
        add_exact2(hi[0], lo[0], pack(x[j].x, x[j].y));
        add_exact2(hi[1], lo[1], pack(x[j].z, x[j].w));
      }
    }
    float h[4], l[4];
    unpack(hi[0], h[0], h[1]);
    unpack(hi[1], h[2], h[3]);
    unpack(lo[0], l[0], l[1]);
    unpack(lo[1], l[2], l[3]);
    return (quick(h[0], l[0]) + quick(h[1], l[1])) + (quick(h[2], l[2]) + quick(h[3], l[3]));
  }
  // Vector v where the row is cut, and without the candidates among `which`.
  __device__ __noinline__ float4 odd(float4 x, int v, unsigned which) const {
    x = row.ends(x, v);
    for (; which; which &= which - 1) {
      const int c = at[__ffs(which) - 1] + row.off;
      if (c >> 2 != v) continue;
      if ((c & 3) == 0) x.x = 0.f;
      if ((c & 3) == 1) x.y = 0.f;
      if ((c & 3) == 2) x.z = 0.f;
      if ((c & 3) == 3) x.w = 0.f;
    }
    return x;
  }
};

// By a warp: which of the lanes' values, in order, the running sum first exceeds t at (the
// last one above 0 if none, -1 if that is none either), and t less what comes before it.
__device__ __forceinline__ int find32(Pair x, Pair& t, bool above) {
  const Pair to = scan32(x);
  unsigned hit = __ballot_sync(kAll, above && t < to);
  if (!hit) {
    hit = __ballot_sync(kAll, above);
    if (!hit) return -1;
    hit = 1u << (31 - __clz(hit));
  }
  const int w = __ffs(hit) - 1;
  t = shfl(t - (to - x), w);
  return w;
}

// The element of vectors [v0, v1) at which the running sum first exceeds t, by a warp:
// 32 parts a step, down to a vector a lane.
__device__ __noinline__ int find(const Left& a, int v0, int v1, Pair t, int lane) {
  while (true) {
    const int each = (v1 - v0 + 31) / 32;
    const int w0 = min(v1, v0 + lane * each), w1 = min(v1, w0 + each);
    const unsigned cand = a.among(v0, v1);
    Pair s = a.sum(w0, w1, 1, cand);
    for (unsigned c = cand; c; c &= c - 1) {
      const int k = __ffs(c) - 1, v = (a.at[k] + a.row.off) >> 2;
      if (v >= w0 && v < w1) s = s + a.val[k];
    }
    const int w = find32(s, t, s.hi > 0.f);
    if (w < 0) return -1;
    if (each > 1) {
      v1 = __shfl_sync(kAll, w1, w);
      v0 = __shfl_sync(kAll, w0, w);
      continue;
    }
    // an element a lane
    const int e = 4 * (v0 + w) - a.row.off + lane;
    Pair x = {0.f, 0.f};
    if (lane < 4 && e >= 0 && e < a.row.V) {
      x.hi = __ldg(reinterpret_cast<const float*>(a.row.base) + a.row.off + e);
      for (unsigned c = cand; c; c &= c - 1)
        if (a.at[__ffs(c) - 1] == e) x = a.val[__ffs(c) - 1];
    }
    const int z = find32(x, t, x.hi > 0.f);
    return z < 0 ? -1 : __shfl_sync(kAll, e, z);
  }
}

__global__ void __launch_bounds__(kThreads, kCtas)
    tree_verify_kernel(const __grid_constant__ TreeVerifyArgs a) {
  __shared__ float r_s[kMaxTree][kCand], d_s[kMaxTree][kCand];
  __shared__ int8_t slot_s[kMaxTree];  // of a node's token among its parent's candidates
  __shared__ int16_t up_s[kMaxTree];   // its parent; -1: no child
  __shared__ float u_s[kMaxTree];
  __shared__ int at_s[kCand];          // the last node's candidates, and their part of what
  __shared__ Pair val_s[kCand];        // is left
  __shared__ int node_s, got_s, owner_s;
  __shared__ uint64_t sums_s[kMaxCluster * kWarps];  // every warp of the cluster's (a Pair)
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int b = blockIdx.y, rank = blockIdx.x, ranks = gridDim.x;
  const int T = a.T, V = a.V;
  const int64_t at = static_cast<int64_t>(b) * T;
  cluster_arrive_relaxed();  // every block of the cluster has begun before one writes to another
  pdl_wait();
  pdl_launch_dependents();
  const int n = a.count ? max(0, min(T, a.count[b])) : T;

  // ---- every node's candidates: p and q, 0 for one out of range or named before ----
  // (loads that do not need each other first: a node's number, token and parent beside them)
  int up = -1, token = -1;
  float u = 0.f;
  if (tid < n) {
    up = a.parents[at + tid];
    token = a.tokens[at + tid];
    u = a.u[at + tid];
  }
  constexpr int kBatch = 2;
  for (int x0 = tid; x0 - lane < n * kCand; x0 += kBatch * kThreads) {
    int c[kBatch];
    float p[kBatch], q[kBatch];
#pragma unroll
    for (int z = 0; z < kBatch; ++z) {
      const int x = x0 + z * kThreads;
      c[z] = x < n * kCand ? a.cand[at * kCand + x] : -1;
      q[z] = x < n * kCand ? a.q[at * kCand + x] : 0.f;
    }
#pragma unroll
    for (int z = 0; z < kBatch; ++z) {
      const int x = x0 + z * kThreads;
      const bool ok = static_cast<unsigned>(c[z]) < static_cast<unsigned>(V);
      if (x < n * kCand && !ok) record_error(a.err, kDevErrBadIndex);
      p[z] = ok ? a.p[(at + x / kCand) * V + c[z]] : 0.f;
      if (!ok || !(q[z] > 0.f)) q[z] = 0.f;
    }
#pragma unroll
    for (int z = 0; z < kBatch; ++z) {
      const int x = x0 + z * kThreads;
      bool again = false;
#pragma unroll
      for (int k = 1; k < kCand; ++k) {
        const int y = __shfl_up_sync(kAll, c[z], k, kCand);
        again |= (lane & 15) >= k && y == c[z];
      }
      if (x < n * kCand) {
        r_s[x / kCand][x % kCand] = again ? 0.f : p[z];
        d_s[x / kCand][x % kCand] = again ? 0.f : q[z];
      }
    }
  }
  if (tid < kMaxTree) {
    int slot = -1;
    if (tid < n && up >= 0 && up < tid) {
      const int4* c = reinterpret_cast<const int4*>(a.cand + (at + up) * kCand);
#pragma unroll
      for (int j = 3; j >= 0; --j) {
        const int4 y = __ldg(c + j);
        if (y.w == token) slot = 4 * j + 3;
        if (y.z == token) slot = 4 * j + 2;
        if (y.y == token) slot = 4 * j + 1;
        if (y.x == token) slot = 4 * j;
      }
    }
    slot_s[tid] = static_cast<int8_t>(slot);
    up_s[tid] = static_cast<int16_t>(slot < 0 ? -1 : up);
    u_s[tid] = u;
  }
  __syncthreads();

  // ---- the walk: lanes 0 .. 15 a candidate each ----
  if (warp == 0) {
    const int k = lane & 15;
    // Lanes 0 .. 15 hold r, 16 .. 31 d, so that one reduction sums both.  Nothing is
    // divided: r/|r| - d/|d| is r |d| - d |r| but for a factor, which g keeps (what r off
    // the candidates is, relative to p).  |r| and |d| are held in [1, 2) by powers of two.
    const bool low = lane < kCand;
    int cur = 0, len = 0;
    Pair x = {0.f, 0.f}, g = {1.f, 0.f};
    while (n > 0) {
      if (rank == 0 && lane == 0) a.path[at + len] = cur;
      ++len;
      const Pair p = {r_s[cur][k], 0.f};
      x = low ? p : Pair{d_s[cur][k], 0.f};
      g = {1.f, 0.f};
      Pair sum = sum16(x);
      const Pair P = shfl(sum, 0);
      Pair rest = Pair{1.f, 0.f} - P;
      if (rest.hi < 0.f) rest = {0.f, 0.f};
      const Pair whole = rest;
      Pair R = rest + P, D = shfl(sum, 16);
      if (!low) x = scaled(x, to_one(D.hi));
      D = scaled(D, to_one(D.hi));
      int took = -1;
      bool over = false;
#pragma unroll 1
      for (int j = cur >> 5; j <= (n - 1) >> 5 && took < 0 && !over; ++j) {
        unsigned kids = __ballot_sync(kAll, up_s[32 * j + lane] == cur);
#pragma unroll 1
        while (kids && !over) {
          const int i = 32 * j + __ffs(kids) - 1;
          kids &= kids - 1;
          const int s = slot_s[i];
          const Pair dk = shfl(x, 16 + s);
          if (!(dk.hi > 0.f)) continue;  // (its mass was taken by a sibling before)
          const Pair rk = shfl(x, s);
          if (dk * u_s[i] * R < rk * D) {
            took = i;
            break;
          }
          const Pair d = shfl_xor(x, 16);
          if (low) {
            x = x * D - d * R;
            if (x.hi < 0.f) x = {0.f, 0.f};
          } else if (!a.replace && k == s) {
            x = {0.f, 0.f};
          }
          rest = rest * D;
          g = g * D;
          sum = sum16(x);
          R = rest + shfl(sum, 0);
          D = shfl(sum, 16);
          if (!(R.hi > 0.f)) {  // p never exceeds q: p itself
            x = p;
            g = {1.f, 0.f};
            over = true;
          } else {
            const float e = to_one(R.hi), f = to_one(D.hi);
            x = scaled(x, low ? e : f);
            rest = scaled(rest, e);
            g = scaled(g, e);
            R = scaled(R, e);
            D = scaled(D, f);
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
      at_s[k] = again || static_cast<unsigned>(c) >= static_cast<unsigned>(V) ? -1 : c;
      val_s[k] = x / g;
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
  left.at = at_s;
  left.val = val_s;
  const int total_warps = ranks * kWarps;
  cluster_wait();
  auto range_at = [&](int w) {
    return static_cast<int>(static_cast<int64_t>(left.row.vecs) * w / total_warps);
  };
  for (int pass = 0; pass < 2 && n > 0; ++pass) {
    const int w = rank * kWarps + warp;
    const int v0 = range_at(w), v1 = range_at(w + 1);
    const unsigned cand = left.among(v0, v1);
    Pair s = left.sum(v0 + lane, v1, 32, cand);
    if (cand >> lane & 1) s = s + val_s[lane];
#pragma unroll
    for (int off = 16; off; off >>= 1) s = s + shfl_xor(s, off);
    if (lane < ranks) {  // to every block of the cluster
      const uint32_t to = dsmem_addr(&sums_s[w], lane);
      asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(to), "f"(s.hi), "f"(s.lo)
                   : "memory");
    }
    cluster_sync_all();
    if (warp == 0) {
      constexpr int kEach = kMaxCluster * kWarps / 32;
      Pair sum = {0.f, 0.f};
#pragma unroll
      for (int j = 0; j < kEach; ++j) {
        const int i = lane * kEach + j;
        if (i < total_warps) sum = sum + *reinterpret_cast<const Pair*>(&sums_s[i]);
      }
      const Pair total = shfl(scan32(sum), 31);
      Pair t = total * u_s[0];
      const int group = find32(sum, t, sum.hi > 0.f);
      int owner = -1;
      if (group >= 0) {
        const Pair y = lane < kEach && group * kEach + lane < total_warps
                           ? *reinterpret_cast<const Pair*>(&sums_s[group * kEach + lane])
                           : Pair{0.f, 0.f};
        owner = group * kEach + find32(y, t, y.hi > 0.f);
      }
      int got = -1;
      if (owner >= 0 && owner / kWarps == rank)
        got = find(left, range_at(owner), range_at(owner + 1), t, lane);
      if (lane == 0) {
        owner_s = owner;
        got_s = got;
      }
    }
    __syncthreads();
    if (owner_s >= 0) break;
    if (tid < kCand) at_s[tid] = -1;  // what is left sums to nothing: the row itself
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
  // as many blocks a sequence as are resident at once, and have 4096 elements each
  const int most = dfl2::kCtas * dfl2::device_info().sms;
  int ranks = dfl2::kMaxCluster;
  while (ranks > 1 && (int64_t(ranks) * B > most || V / ranks < 4096)) ranks /= 2;
  const cudaError_t e =
      dfl2::launch_kc(dfl2::tree_verify_kernel, dim3(ranks, B), dim3(dfl2::kThreads), 0,
                      reinterpret_cast<cudaStream_t>(stream), true, ranks, a);
  return e == cudaSuccess ? DFL2_OK : dfl2::report_cuda_error(e, "tree verify launch");
}
