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
// warp, a lane to a candidate; so the blocks need not exchange the path.  The row of the last
// draw is then cut into one range a warp.  The warps' sums are exchanged through distributed
// shared memory, and the block that has the range the drawn number falls in looks for the
// element with all its threads.
// Numbers are unevaluated sums of two floats (about 46 bits): decisions and the drawn index
// have to be those of the exact sums, and this GPU's doubles are slow (two additions a cycle
// and SM, 60 cycles each).
//
// One tree is bound by the latency of its dependent steps: a candidate's number and its p
// (2 us), the tests of the walk (about 1000 cycles each), the row's elements, and the search for
// the drawn one (9.8 us a pass for 33 nodes and 151,936 tokens).  64 trees: the longest walk of
// them, and 39 MB of rows (19.0 us a pass; 5.7 at HBM's rate).
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>

#include "cache.cuh"

namespace dfl2 {
namespace {

constexpr unsigned kAll = 0xffffffffu;
constexpr int kThreads = 512, kWarps = kThreads / 32, kCtas = 2, kMaxCluster = 16;

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
// 2^-e for x in [2^e, 2^(e+1)), so that x times it is in [1, 2); for x below the smallest normal
// number 2^127 (then x times it is at least 2^-22), from 2^127 on 2^-126.
__device__ __forceinline__ float to_one(float x) {
  const int e = static_cast<int>(__float_as_uint(x) >> 23);  // (x >= 0)
  return __uint_as_float(static_cast<uint32_t>(254 - min(e, 253)) << 23);
}

// a times g, g > 0: not 0 if a is not.
__device__ __forceinline__ Pair times(Pair a, Pair g) {
  const Pair x = a * g;
  return x.hi > 0.f || !(a.hi > 0.f) ? x : Pair{__uint_as_float(1u), 0.f};
}

// The row of the last draw.  Rows need not begin on 16 bytes: its vectors are numbered from
// the 16-byte boundary at or before the row, `off` elements early.
struct Row {
  const float* p;  // element 0
  int off, V, vecs;
  __device__ __forceinline__ float4 vec(int v) const {
    return __ldg(reinterpret_cast<const float4*>(p - off) + v);
  }
  // Whether vector v holds elements of other rows (and may lie outside the tensor).
  __device__ __forceinline__ bool cut(int v) const { return 4 * v < off || 4 * v + 4 - off > V; }
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
// hi + lo += x, twice: the two-sum, what hi loses of each addition goes into lo.
__device__ __forceinline__ void add2_with_rest(uint64_t& hi, uint64_t& lo, uint64_t x) {
  const uint64_t s = add2(hi, x), c = sub2(s, hi);
  lo = add2(lo, add2(sub2(hi, sub2(s, c)), sub2(x, c)));
  hi = s;
}

// The sum of vectors v, v + step, .. below v1 (step = 2^lg), without those that are cut and
// without the elements at[k] of the bits k of `cand`.  Nothing that was added is taken out
// again: a sum is 0 if and only if every element in it is.
// Off by at most 2^-38 of itself for each of its 32 vectors' sums (32 additions, which leave lo
// up to 2^-24 of the sum each, and round it as often) and 2^-46 for adding each of these.
__device__ __noinline__ Pair row_sum(const Row row, int v, int v1, int lg, const int* at,
                                     unsigned cand) {
  // Vectors on their way at a time: 32 of the 64 registers that two blocks on an SM leave a
  // thread (64 trees of 151,936 tokens, 19 vectors a lane: 18.7 us with 5, 19.0 with 8, and
  // with 10 and 12, which spill, 22.5 and 23.3).
  constexpr int kBatch = 8;
  constexpr int kFold = 4;  // batches that are added up in floats and their remainders
  Pair sum = {0.f, 0.f};
#pragma unroll 1
  while (v < v1) {
    uint64_t hi[2] = {0, 0}, lo[2] = {0, 0};
#pragma unroll 1
    for (int f = 0; f < kFold && v < v1; ++f, v += kBatch << lg) {
      uint32_t gone = 0;  // bit 4 j + z: element z of vector j
#pragma unroll 1
      for (unsigned c = cand; c; c &= c - 1) {
        const int e = at[__ffs(c) - 1] + row.off, d = (e >> 2) - v;
        if (d >= 0 && d < kBatch << lg && (d & ((1 << lg) - 1)) == 0)
          gone |= 1u << (4 * (d >> lg) + (e & 3));
      }
      float4 x[kBatch];
#pragma unroll
      for (int j = 0; j < kBatch; ++j) {
        const int i = v + (j << lg);
        x[j] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (i < v1 && !row.cut(i)) x[j] = row.vec(i);
      }
      if (gone) {
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
          if (gone >> (4 * j) & 1) x[j].x = 0.f;
          if (gone >> (4 * j + 1) & 1) x[j].y = 0.f;
          if (gone >> (4 * j + 2) & 1) x[j].z = 0.f;
          if (gone >> (4 * j + 3) & 1) x[j].w = 0.f;
        }
      }
#pragma unroll
      for (int j = 0; j < kBatch; ++j) {
        if (v + (j << lg) >= v1) break;
        add2_with_rest(hi[0], lo[0], pack(x[j].x, x[j].y));
        add2_with_rest(hi[1], lo[1], pack(x[j].z, x[j].w));
      }
    }
    float h[4], l[4];
    unpack(hi[0], h[0], h[1]);
    unpack(hi[1], h[2], h[3]);
    unpack(lo[0], l[0], l[1]);
    unpack(lo[1], l[2], l[3]);
    sum = sum + ((quick(h[0], l[0]) + quick(h[1], l[1])) + (quick(h[2], l[2]) + quick(h[3], l[3])));
  }
  return sum;
}

// What is drawn from: the row times g, and in the candidates' places other values.
struct Left {
  Row row;
  Pair g;
  const int* at;    // [16], the candidates' elements; -1: none
  const Pair* val;  // [16]
  // The candidates in vectors [v0, v1), by a warp.
  __device__ __forceinline__ unsigned among(int v0, int v1) const {
    const int lane = threadIdx.x & 31, c = lane < kCand ? at[lane] : -1;
    const int v = (c + row.off) >> 2;
    return __ballot_sync(kAll, c >= 0 && v >= v0 && v < v1);
  }
  // This lane's sum of vectors v, v + 2^lg, .. below v1; cand: the candidates that may be
  // among them.
  __device__ __forceinline__ Pair sum(int v, int v1, int lg, unsigned cand) const {
    auto mine = [&](int i) { return i >= v && i < v1 && ((i - v) & ((1 << lg) - 1)) == 0; };
    Pair s = times(row_sum(row, v, v1, lg, at, cand), g);
    const int last = row.vecs - 1;
    if (v < v1 && (v == 0 || v1 > last)) {  // the elements of the cut vectors
#pragma unroll 1
      for (int j = 0; j < (last ? 8 : 4); ++j) {
        const int i = j < 4 ? 0 : last, e = 4 * i + (j & 3) - row.off;
        if (row.cut(i) && e >= 0 && e < row.V && mine(i) && slot(e, cand) < 0)
          s = s + times({row.p[e], 0.f}, g);
      }
    }
#pragma unroll 1
    for (; cand; cand &= cand - 1) {
      const int k = __ffs(cand) - 1;
      if (mine((at[k] + row.off) >> 2)) s = s + val[k];
    }
    return s;
  }
  // Which of the candidates in `cand` element e is; -1: none.
  __device__ __forceinline__ int slot(int e, unsigned cand) const {
    int k = -1;
#pragma unroll 1
    for (; cand; cand &= cand - 1)
      if (at[__ffs(cand) - 1] == e) k = __ffs(cand) - 1;
    return k;
  }
  __device__ __forceinline__ Pair element(int e, unsigned cand) const {
    const int k = slot(e, cand);
    return k < 0 ? times({row.p[e], 0.f}, g) : val[k];
  }
};

// By a warp: which of the lanes' values x, in order, the running sum `to` first exceeds t at
// (the last one above 0 if none, -1 if that is none either), and t less what comes before it.
__device__ __forceinline__ int find32(Pair x, Pair to, Pair& t) {
  const bool above = x.hi > 0.f;
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

__global__ void __launch_bounds__(kThreads, kCtas)
    tree_verify_kernel(const __grid_constant__ TreeVerifyArgs a) {
  __shared__ float r_s[kMaxTree][kCand], d_s[kMaxTree][kCand];
  __shared__ int8_t slot_s[kMaxTree];  // of a node's token among its parent's candidates
  __shared__ int16_t up_s[kMaxTree];   // its parent; -1: no child
  __shared__ float u_s[kMaxTree];
  __shared__ int at_s[kCand];          // the last node's candidates, and their part of what
  __shared__ Pair val_s[kCand], g_s;   // is left, and of the row's other elements
  __shared__ int node_s, owner_s, who_s, last_s;
  __shared__ Pair t_s, warp_s[kWarps];
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
      // (c is below 2^30; the halves of a warp are different nodes)
      const unsigned same = __match_any_sync(kAll, c[z] ^ (lane >> 4 << 30));
      const bool again = same >> (lane & 16) & ((1u << (lane & 15)) - 1);
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
    // the candidates is, relative to p).  |r| and |d| are held near 1 by powers of two.
    const bool low = lane < kCand;
    int cur = 0, len = 0, cand = -1;
    Pair x = {0.f, 0.f}, g = {1.f, 0.f};
    while (n > 0) {
      cand = a.cand[(at + cur) * kCand + k];  // (looked at after the walk)
      if (rank == 0 && lane == 0) a.path[at + len] = cur;
      ++len;
      const Pair p = {r_s[cur][k], 0.f};
      x = low ? p : Pair{d_s[cur][k], 0.f};
      g = {1.f, 0.f};
      Pair sum = sum16(x);
      const Pair P = shfl(sum, 0);
      Pair rest = Pair{1.f, 0.f} - P;
      if (rest.hi < 0.f) rest = {0.f, 0.f};
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
    bool again = static_cast<unsigned>(cand) >= static_cast<unsigned>(V);
    again |= (__match_any_sync(kAll, cand) & ((1u << k) - 1)) != 0;
    if (low) {
      at_s[k] = again ? -1 : cand;
      val_s[k] = x;
    }
    if (lane == 0) g_s = g.hi < 0x1p100f ? g : Pair{0x1p100f, 0.f};
    if (lane == 0) node_s = cur;
  }
  __syncthreads();

  // ---- the last draw ----
  Left left;
  const int64_t start = (at + node_s) * V;
  left.row.p = a.p + start;
  left.row.off = static_cast<int>(start & 3);
  left.row.V = V;
  left.row.vecs = (V + left.row.off + 3) / 4;
  left.g = g_s;
  left.at = at_s;
  left.val = val_s;
  const int total_warps = ranks * kWarps;
  const int each = (left.row.vecs + total_warps - 1) / total_warps;
  cluster_wait();
  auto range_at = [&](int w) { return min(left.row.vecs, w * each); };
  for (int pass = 0; pass < 2 && n > 0; ++pass) {
    const int w = rank * kWarps + warp;
    const int v0 = range_at(w), v1 = range_at(w + 1);
    Pair s = left.sum(v0 + lane, v1, 5, left.among(v0, v1));
#pragma unroll 1
    for (int off = 16; off; off >>= 1) s = s + shfl_xor(s, off);
    if (lane < ranks) {  // to every block of the cluster
      const uint32_t to = dsmem_addr(&sums_s[w], lane);
      asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(to), "f"(s.hi), "f"(s.lo)
                   : "memory");
    }
    cluster_sync_all();
    if (warp == 0) {
      constexpr int kEach = kMaxCluster * kWarps / 32;
      Pair x[kEach], sum = {0.f, 0.f};
#pragma unroll
      for (int j = 0; j < kEach; ++j) {
        const int i = lane * kEach + j;
        x[j] = i < total_warps ? *reinterpret_cast<const Pair*>(&sums_s[i]) : Pair{0.f, 0.f};
        sum = sum + x[j];
      }
      const Pair to = scan32(sum);
      Pair t = shfl(to, 31) * u_s[0];
      int owner = find32(sum, to, t);
      if (owner >= 0) {  // every lane looks in its own kEach
        int mine = 0;
        Pair before = {0.f, 0.f}, run = {0.f, 0.f};
        bool found = false;
#pragma unroll
        for (int j = 0; j < kEach; ++j)
          if (!found && x[j].hi > 0.f) {
            mine = j;
            before = run;
            run = run + x[j];
            found = t < run;
          }
        t = shfl(t - before, owner);
        owner = owner * kEach + __shfl_sync(kAll, mine, owner);
      }
      if (lane == 0) {
        owner_s = owner;
        t_s = t;
        who_s = kThreads;
        last_s = -1;
      }
    }
    __syncthreads();
    if (owner_s >= 0) break;
    if (tid < kCand) at_s[tid] = -1;  // what is left sums to nothing: the row itself
    left.g = {1.f, 0.f};
    cluster_sync_all();
  }

  // ---- the element, by the block that has its range: a run of vectors a thread ----
  const int owner = n > 0 ? owner_s : -1;
  if (owner >= 0 && owner / kWarps == rank) {
    const int v0 = range_at(owner), v1 = range_at(owner + 1);
    const int run = (v1 - v0 + kThreads - 1) / kThreads;
    const int w0 = min(v1, v0 + tid * run), w1 = min(v1, w0 + run);
    const unsigned cand = left.among(v0, v1);
    const Pair x = left.sum(w0, w1, 0, cand);
    const Pair to = scan32(x);
    if (lane == 31) warp_s[warp] = to;
    __syncthreads();
    const Pair sums = scan32(lane < kWarps ? warp_s[lane] : Pair{0.f, 0.f});
    Pair before = shfl(sums, max(0, warp - 1));
    if (warp == 0) before = {0.f, 0.f};
    const unsigned hit = __ballot_sync(kAll, x.hi > 0.f && t_s < before + to);
    const unsigned some = __ballot_sync(kAll, x.hi > 0.f);
    if (lane == 0) {
      if (hit) atomicMin(&who_s, tid + __ffs(hit) - 1);
      if (some) atomicMax(&last_s, tid + 31 - __clz(some));
    }
    __syncthreads();
    // (the first thread where none has a sum above 0, which rows with values below 0 can do)
    if (tid == (who_s < kThreads ? who_s : max(0, last_s))) {
      const int e0 = max(0, 4 * w0 - left.row.off), e1 = min(V, 4 * w1 - left.row.off);
      const Pair t = t_s - (before + (to - x));
      Pair c = {0.f, 0.f};
      int got = -1;
#pragma unroll 1
      for (int e = e0; e < e1; ++e) {
        const Pair y = left.element(e, cand);
        if (!(y.hi > 0.f)) continue;
        c = c + y;
        got = e;
        if (t < c) break;
      }
      a.next[b] = got;
    }
  } else if (owner < 0 && rank == 0 && tid == 0) {
    a.next[b] = -1;
  }
  cluster_sync_all();  // no block ends while another may still write to it
}

// Whether the current device can hold a cluster of 16 blocks of the kernel.
bool wide_clusters() {
  static std::atomic<int> known[64];  // (ordinals are below 64: ensured with the device's state)
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return false;
  int k = known[dev].load();
  if (k == 0) {
    int n = 0;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(kMaxCluster);
    cfg.blockDim = dim3(kThreads);
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = kMaxCluster;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const bool ok =
        cudaFuncSetAttribute(tree_verify_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed,
                             1) == cudaSuccess &&
        cudaOccupancyMaxActiveClusters(&n, tree_verify_kernel, &cfg) == cudaSuccess && n > 0;
    if (!ok) cudaGetLastError();
    k = ok ? 2 : 1;
    known[dev].store(k);
  }
  return k == 2;
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
  // As many blocks a sequence as are resident at once, and have 4096 elements each; 16, which
  // a device may refuse, where it takes them.
  const int most = dfl2::kCtas * dfl2::device_info().sms;
  int ranks = dfl2::wide_clusters() ? dfl2::kMaxCluster : 8;
  while (ranks > 1 && (int64_t(ranks) * B > most || V / ranks < 4096)) ranks /= 2;
  const cudaError_t e =
      dfl2::launch_kc(dfl2::tree_verify_kernel, dim3(ranks, B), dim3(dfl2::kThreads), 0,
                      reinterpret_cast<cudaStream_t>(stream), true, ranks, a);
  return e == cudaSuccess ? DFL2_OK : dfl2::report_cuda_error(e, "tree verify launch");
}
