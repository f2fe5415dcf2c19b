// Attention of a tree of drafted tokens over the paged cache (include/dfl2.h,
// dfl2_tree_attn):
//   o_i = sum_j p_ij v_j,  p_ij = exp(s_ij) / sum_j exp(s_ij),  s_ij = scale <q_i, k_j>
// over the positions j that node i sees.
//
// The G = q_heads / kv_heads query heads that share a key head read the same
// keys, so the T nodes and G heads make one matrix of M = T G rows against the
// keys of (sequence, key head): row r is node r / G, head h G + r % G.  Each key
// and value is then read once per kRows rows and used 2 kRows times, and the
// work is two matrix products around an exponential.
//
// Split.  Lengths live on the device and differ by sequence, so the host
// cannot cut the work.  A unit is one tile of keys of one (sequence, key head,
// row tile); every CTA takes an equal, contiguous range of the units, whatever
// sequences it spans.  A CTA that covers all tiles of a row tile writes its
// output; one that covers a part writes its running maximum, sum and
// unnormalised output to the workspace (a range has at most two such ends), and
// combine_kernel adds the parts in the order of the keys.
//
// Softmax in one pass: with the running maximum m and sum l of a row, a tile
// with row maximum m' multiplies l and o by 2^(m - m') before adding its own
// terms (scores are kept times log2 e, so that exp is exp2).
#include <algorithm>
#include <cmath>

#include "tree_attn.cuh"

namespace dfl2 {
namespace {

template <typename E>
__device__ __forceinline__ void mma16816(float d[4], const uint32_t a[4], const uint32_t b0,
                                         const uint32_t b1) {
  if constexpr (std::is_same_v<E, __half>)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void ldsm_x4_t(uint32_t addr, uint32_t r[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}
// ---------------------------------------------------------------------------
// Warp-level kernel.  Four warps, tiles of 64 keys, 16 keys to a warp: each warp
// keeps its own maximum, sum and output for all rows and the four are added at
// the end of a row tile, so no warp waits for another inside a tile but for its
// keys' arrival.
// ---------------------------------------------------------------------------
constexpr int kWThreads = 128;

template <int D, int kRows>
struct WarpCfg {
  static constexpr int kStages = D == 64 ? 4 : D == 128 ? 3 : 2;
  static constexpr int kTile = kKeys * D * 2;  // bytes of K (or V) in a stage
  static constexpr int kQBytes = kRows * D * 2;
  static constexpr int kJoin = kRows == 16 ? 64 : 32;  // channels added per round at the end
  static constexpr int kJoinBytes = kRows * kJoin * 4;
  static constexpr size_t kSmem =
      size_t(kStages) * 2 * kTile + kQBytes + kJoinBytes + 4 * kRows * 8 + 16;
};

template <typename E, int D, int kRows>
__global__ void __launch_bounds__(kWThreads, D == 256 ? 1 : 2)
    attn_warp_kernel(const __grid_constant__ AttnArgs a) {
  using C = WarpCfg<D, kRows>;
  constexpr int kMT = kRows / 16;        // 16-row MMA tiles
  constexpr int kCPR = D / 8;            // 16-byte pieces of a key
  constexpr int kRowStep = kWThreads / kCPR;
  constexpr int kPer = kKeys / kRowStep;  // keys each thread copies a piece of, per tile
  extern __shared__ __align__(128) uint8_t smem[];
  uint8_t* ring = smem;
  uint8_t* qs = smem + C::kStages * 2 * C::kTile;
  float* join = reinterpret_cast<float*>(qs + C::kQBytes);
  float2* ml_s = reinterpret_cast<float2*>(reinterpret_cast<uint8_t*>(join) + C::kJoinBytes);
  int* bad_s = reinterpret_cast<int*>(ml_s + 4 * kRows);

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const E* K = static_cast<const E*>(a.k);
  const E* V = static_cast<const E*>(a.v);
  const int ps1 = (1 << a.t.page_shift) - 1;
  pdl_wait();
  pdl_launch_dependents();

  const Range g = find_range(a, blockIdx.x);
  const int64_t u0 = g.u0, u1 = g.u1;
  if (tid == 0) a.cuts[blockIdx.x].b = -1;
  if (u0 == u1) return;
  Cursor cur = g.first;
  Cursor ld = cur;

  // ---- loads: thread -> piece cp of keys kr0, kr0 + kRowStep, .. ----
  const int cp = tid % kCPR, kr0 = tid / kCPR;
  int pages[kPer];
  auto look_up = [&]() {  // the pages of the tile at ld
    if (ld.u >= u1) return;
    const int end = ld.s.len + ld.s.n;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int pos = ld.tile * kKeys + kr0 + i * kRowStep;
      pages[i] = pos < end ? a.t.page_at(ld.s.row, pos >> a.t.page_shift) : -1;
    }
  };
  auto issue = [&](int stage) {  // the copies of the tile at ld
    if (ld.u < u1) {
      uint8_t* st = ring + stage * 2 * C::kTile;
      const int h = ld.hr / a.row_tiles;
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const int r = kr0 + i * kRowStep;
        const int pos = ld.tile * kKeys + r;
        const bool ok = pages[i] >= 0;
        const int64_t at = static_cast<int64_t>(ok ? pages[i] : 0) * a.page_stride +
                           h * a.head_stride + (ok ? pos & ps1 : 0) * a.slot_stride + cp * 8;
        uint8_t* dst = st + r * (D * 2) + ((cp ^ (r & 7)) << 4);
        cp_async16(dst, K + at, ok);
        cp_async16(dst + C::kTile, V + at, ok);
      }
      ld.next(a);
    }
    cp_async_commit();
  };
  look_up();
#pragma unroll
  for (int s = 0; s < C::kStages - 1; ++s) {
    issue(s);
    look_up();
  }

  float o[kMT][D / 8][4];
  float m[kMT][2], l[kMT][2];
  int stage = 0;
  bool fresh = true;
  int tile_lo = 0;  // first tile of this CTA's part of the row tile
  int bad = 0;

  for (; cur.u < u1;) {
    const Seq s = cur.s;
    const int h = cur.hr / a.row_tiles, r0 = (cur.hr % a.row_tiles) * kRows;
    const int rows = min(kRows, a.t.T * a.G - r0);
    if (fresh) {
      fresh = false;
      tile_lo = cur.tile;
      bad = 0;
      const E* Q = static_cast<const E*>(a.q) + cur.b * a.qb;
      for (int x = tid; x < kRows * kCPR; x += kWThreads) {
        const int r = x / kCPR, c = x % kCPR;
        uint4 val = make_uint4(0, 0, 0, 0);
        if (r < rows)
          val = *reinterpret_cast<const uint4*>(Q + (r0 + r) / a.G * a.qt +
                                                (h * a.G + (r0 + r) % a.G) * a.qh + c * 8);
        *reinterpret_cast<uint4*>(qs + r * (D * 2) + ((c ^ (r & 7)) << 4)) = val;
      }
#pragma unroll
      for (int i = 0; i < kMT; ++i) {
        m[i][0] = m[i][1] = -INFINITY;
        l[i][0] = l[i][1] = 0.f;
#pragma unroll
        for (int j = 0; j < D / 8; ++j) o[i][j][0] = o[i][j][1] = o[i][j][2] = o[i][j][3] = 0.f;
      }
    }
    cp_async_wait<C::kStages - 2>();
    __syncthreads();  // the tile (and a new q) is here; everyone is done with the stage before
    issue((stage + C::kStages - 1) % C::kStages);
    look_up();

    uint8_t* kst = ring + stage * 2 * C::kTile + warp * 16 * (D * 2);
    uint8_t* vst = kst + C::kTile;
    const int p0 = cur.tile * kKeys + warp * 16;  // this warp's first position
    const bool edge = p0 + 16 > s.len;             // has nodes, or lies past the end

    // scores: rows x 16 keys
    float sc[kMT][2][4];
#pragma unroll
    for (int i = 0; i < kMT; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j) sc[i][j][0] = sc[i][j][1] = sc[i][j][2] = sc[i][j][3] = 0.f;
#pragma unroll
    for (int kk = 0; kk < D / 16; ++kk) {
      uint32_t kb[4];  // keys 0..7 and 8..15, channels 16 kk .. + 7 and + 8 ..
      {
        const int r = (lane & 7) + ((lane >> 4) << 3), c = 2 * kk + ((lane >> 3) & 1);
        ldsm_x4(smem_u32(kst + r * (D * 2) + ((c ^ (r & 7)) << 4)), kb);
      }
#pragma unroll
      for (int i = 0; i < kMT; ++i) {
        uint32_t qa[4];
        const int r = i * 16 + (lane & 15), c = 2 * kk + (lane >> 4);
        ldsm_x4(smem_u32(qs + r * (D * 2) + ((c ^ (r & 7)) << 4)), qa);
        mma16816<E>(sc[i][0], qa, kb[0], kb[1]);
        mma16816<E>(sc[i][1], qa, kb[2], kb[3]);
      }
    }
    // what a row does not see
#pragma unroll
    for (int i = 0; i < kMT; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float x = sc[i][j][e] * a.scale_log2;
          if (edge) {
            const int node = p0 + j * 8 + (lane & 3) * 2 + (e & 1) - s.len;
            const int r = r0 + i * 16 + (lane >> 2) + (e >> 1) * 8;
            if (node >= 0 && (r - r0 >= rows || !sees(a, cur.b, s.n, r / a.G, node)))
              x = -INFINITY;
          }
          sc[i][j][e] = x;
        }
    // running maximum, weights, sum
    bool moved = false;
    float al[kMT][2];
#pragma unroll
    for (int i = 0; i < kMT; ++i)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float x = fmaxf(fmaxf(sc[i][0][2 * e], sc[i][0][2 * e + 1]),
                        fmaxf(sc[i][1][2 * e], sc[i][1][2 * e + 1]));
        x = fmaxf(x, __shfl_xor_sync(kAll, x, 1));
        x = fmaxf(x, __shfl_xor_sync(kAll, x, 2));
        const float mn = fmaxf(m[i][e], x);
        const float safe = mn == -INFINITY ? 0.f : mn;
        al[i][e] = ex2(m[i][e] - safe);
        moved |= mn != m[i][e];
        m[i][e] = mn;
        float sum = 0.f;
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int z = 0; z < 2; ++z) {
            const float p = ex2(sc[i][j][2 * e + z] - safe);
            sc[i][j][2 * e + z] = p;
            sum += p;
          }
        l[i][e] = l[i][e] * al[i][e] + sum;
      }
    if (__any_sync(kAll, moved)) {
#pragma unroll
      for (int i = 0; i < kMT; ++i)
#pragma unroll
        for (int j = 0; j < D / 8; ++j) {
          o[i][j][0] *= al[i][0];
          o[i][j][1] *= al[i][0];
          o[i][j][2] *= al[i][1];
          o[i][j][3] *= al[i][1];
        }
    }
    if (edge) {  // Inf and NaN of nodes stay out of the product (unseen_safe_sum)
      bool found = false;
      for (int x = lane; x < 16 * kCPR; x += 32) {
        if (p0 + x / kCPR < s.len) continue;
        uint4* at = reinterpret_cast<uint4*>(vst) + x;
        uint4 y = *at;
        bool b4 = false;
        y.x = finite2<E>(y.x, b4);
        y.y = finite2<E>(y.y, b4);
        y.z = finite2<E>(y.z, b4);
        y.w = finite2<E>(y.w, b4);
        if (b4) *at = y;
        found |= b4;
      }
      bad |= __any_sync(kAll, found);
      __syncwarp();
    }
    // the weights (rounded to E: they multiply values of E, and their own rounding
    // errors average out over the keys) times V
    uint32_t pa[kMT][4];
#pragma unroll
    for (int i = 0; i < kMT; ++i) {
      pa[i][0] = pack2<E>(sc[i][0][0], sc[i][0][1]);
      pa[i][1] = pack2<E>(sc[i][0][2], sc[i][0][3]);
      pa[i][2] = pack2<E>(sc[i][1][0], sc[i][1][1]);
      pa[i][3] = pack2<E>(sc[i][1][2], sc[i][1][3]);
    }
#pragma unroll
    for (int j = 0; j < D / 16; ++j) {
      uint32_t vb[4];  // keys 0..7 / 8..15 of channels 16 j .. + 7, then of + 8 ..
      const int r = lane & 15, c = 2 * j + (lane >> 4);
      ldsm_x4_t(smem_u32(vst + r * (D * 2) + ((c ^ (r & 7)) << 4)), vb);
#pragma unroll
      for (int i = 0; i < kMT; ++i) {
        mma16816<E>(o[i][2 * j], pa[i], vb[0], vb[1]);
        mma16816<E>(o[i][2 * j + 1], pa[i], vb[2], vb[3]);
      }
    }
    if (++stage == C::kStages) stage = 0;

    // ---- the end of this CTA's part of the row tile ----
    const bool last = cur.tile + 1 == s.tiles;
    if (last || cur.u + 1 == u1) {
      const bool whole = last && tile_lo == 0;
      const int slot = tile_lo == 0 && !whole && cur.u + 1 == u1 &&
                               cur.u - cur.tile > u0 ? 1 : 0;
      const int tile_hi = cur.tile + 1;
      if (cur.u + 1 == u1 && tid == 0) {
        Cursor at = cur;
        at.u -= cur.tile;  // the row tile's first unit
        a.cuts[blockIdx.x] = make_cut(g, at, tile_lo, tile_hi, slot);
      }
#pragma unroll
      for (int i = 0; i < kMT; ++i)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          l[i][e] += __shfl_xor_sync(kAll, l[i][e], 1);
          l[i][e] += __shfl_xor_sync(kAll, l[i][e], 2);
          if ((lane & 3) == 0)
            ml_s[warp * kRows + i * 16 + e * 8 + (lane >> 2)] = make_float2(m[i][e], l[i][e]);
        }
      if (lane == 0) bad_s[warp] = bad;
      __syncthreads();
      const bool any_bad = bad_s[0] | bad_s[1] | bad_s[2] | bad_s[3];
      // this warp's factor to the common maximum
      float f[kMT][2];
#pragma unroll
      for (int i = 0; i < kMT; ++i)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int r = i * 16 + e * 8 + (lane >> 2);
          float mm = -INFINITY;
#pragma unroll
          for (int w = 0; w < 4; ++w) mm = fmaxf(mm, ml_s[w * kRows + r].x);
          f[i][e] = ex2(m[i][e] - (mm == -INFINITY ? 0.f : mm));
        }
#pragma unroll
      for (int c0 = 0; c0 < D; c0 += C::kJoin) {
        for (int w = 0; w < 4; ++w) {  // the four warps' outputs, in their order
          if (warp == w) {
#pragma unroll
            for (int i = 0; i < kMT; ++i)
#pragma unroll
              for (int j = 0; j < C::kJoin / 8; ++j)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                  float2* at = reinterpret_cast<float2*>(
                      join + (i * 16 + e * 8 + (lane >> 2)) * C::kJoin + j * 8 + (lane & 3) * 2);
                  float2 x = make_float2(o[i][c0 / 8 + j][2 * e] * f[i][e],
                                         o[i][c0 / 8 + j][2 * e + 1] * f[i][e]);
                  if (w) {
                    const float2 y = *at;
                    x.x += y.x;
                    x.y += y.y;
                  }
                  *at = x;
                }
          }
          __syncthreads();
        }
        for (int x = tid; x < rows * (C::kJoin / 4); x += kWThreads) {
          const int r = x / (C::kJoin / 4), c = c0 + x % (C::kJoin / 4) * 4;
          float mm = -INFINITY, ll = 0.f;
#pragma unroll
          for (int w = 0; w < 4; ++w) mm = fmaxf(mm, ml_s[w * kRows + r].x);
          const float safe = mm == -INFINITY ? 0.f : mm;
#pragma unroll
          for (int w = 0; w < 4; ++w)
            ll += ml_s[w * kRows + r].y * ex2(ml_s[w * kRows + r].x - safe);
          float4 y = *reinterpret_cast<const float4*>(join + r * C::kJoin + (c - c0));
          const int node = (r0 + r) / a.G, head = h * a.G + (r0 + r) % a.G;
          if (any_bad) {
            float* yy = reinterpret_cast<float*>(&y);
            for (int z = 0; z < 4; ++z)
              yy[z] += unseen_safe_sum<E>(a, cur.b, s, h, node, c + z, tile_lo * kKeys,
                                          tile_hi * kKeys);
          }
          if (whole) {
            if (node < s.n) {
              const float inv = ll == 0.f ? 0.f : 1.f / ll;
              E* out = static_cast<E*>(a.out) + cur.b * a.ob + node * a.ot + head * a.oh + c;
              *reinterpret_cast<uint2*>(out) = make_uint2(pack2<E>(y.x * inv, y.y * inv),
                                                          pack2<E>(y.z * inv, y.w * inv));
              if (a.lse && c == 0)
                a.lse[(static_cast<int64_t>(cur.b) * a.t.T + node) * (a.H * a.G) + head] =
                    safe * kLn2 + logf(ll);
            }
          } else {
            const int64_t p = (static_cast<int64_t>(blockIdx.x) * 2 + slot) * kRows + r;
            *reinterpret_cast<float4*>(a.part_o + p * D + c) = y;
            if (c == 0) a.part_ml[p] = make_float2(mm, ll);
          }
        }
        __syncthreads();
      }
      fresh = true;
    }
    cur.next(a);
  }
}

// The parts that the CTAs left of a row tile, added in the order of the keys, a warp
// to a row: block column c takes the row tile that CTA c began and did not end (its
// Cut), block rows divide the tile's rows, and the last B block columns zero what
// lies past a sequence's count.
// (A warp to every output row, looking up whether it was cut, took 76 us after the
// 1.28 ms of 32 sequences of 64 nodes: most rows are whole.)
constexpr int kCombineWarps = 8;
template <typename E, int D>
__global__ void __launch_bounds__(kCombineWarps * 32)
    combine_kernel(const __grid_constant__ AttnArgs a) {
  pdl_wait();
  pdl_launch_dependents();
  constexpr int kPer = D / 32;  // channels per lane
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int step = gridDim.y * kCombineWarps;
  const int Hq = a.H * a.G;
  if (static_cast<int>(blockIdx.x) >= a.grid) {
    const int b = blockIdx.x - a.grid;
    for (int x = load_seq(a, b).n * Hq + blockIdx.y * kCombineWarps + warp; x < a.t.T * Hq;
         x += step) {
      const int node = x / Hq, head = x - node * Hq;
      uint32_t* out = reinterpret_cast<uint32_t*>(static_cast<E*>(a.out) + b * a.ob + node * a.ot +
                                                  head * a.oh + lane * kPer);
#pragma unroll
      for (int i = 0; i < kPer / 2; ++i) out[i] = 0;
      if (a.lse && lane == 0)
        a.lse[(static_cast<int64_t>(b) * a.t.T + node) * Hq + head] = -INFINITY;
    }
    return;
  }
  const Cut cut = a.cuts[blockIdx.x];
  if (cut.b < 0) return;
  const int b = cut.b, c0 = blockIdx.x, c1 = cut.last_cta, slot0 = cut.slot;
  const int h = cut.hr / a.row_tiles, r0 = (cut.hr - h * a.row_tiles) * a.rows;
  const int n = load_seq(a, b).n;
  const int rows = min(a.rows, n * a.G - r0);  // (rows past the count are zeroed above)
  for (int r = blockIdx.y * kCombineWarps + warp; r < rows; r += step) {
    auto part = [&](int c) {
      return (static_cast<int64_t>(c) * 2 + (c == c0 ? slot0 : 0)) * a.rows + r;
    };
    float mm = -INFINITY;
    for (int c = c0 + lane; c <= c1; c += 32) mm = fmaxf(mm, a.part_ml[part(c)].x);
#pragma unroll
    for (int off = 16; off; off >>= 1) mm = fmaxf(mm, __shfl_xor_sync(kAll, mm, off));
    const float safe = mm == -INFINITY ? 0.f : mm;
    float y[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) y[i] = 0.f;
    float ll = 0.f;
#pragma unroll 8
    for (int c = c0; c <= c1; ++c) {
      const float2 ml = a.part_ml[part(c)];
      const float w = ex2(ml.x - safe);
      const float* p = a.part_o + part(c) * D + lane * kPer;
      ll += ml.y * w;
#pragma unroll
      for (int i = 0; i < kPer; ++i) y[i] += p[i] * w;
    }
    const float inv = ll == 0.f ? 0.f : 1.f / ll;
    const int node = (r0 + r) / a.G, head = h * a.G + (r0 + r) - node * a.G;
    uint32_t* out = reinterpret_cast<uint32_t*>(static_cast<E*>(a.out) + b * a.ob + node * a.ot +
                                                head * a.oh + lane * kPer);
#pragma unroll
    for (int i = 0; i < kPer / 2; ++i) out[i] = pack2<E>(y[2 * i] * inv, y[2 * i + 1] * inv);
    if (a.lse && lane == 0)  // log 0 = -inf: nothing seen
      a.lse[(static_cast<int64_t>(b) * a.t.T + node) * Hq + head] = safe * kLn2 + logf(ll);
  }
}

// ---- plan ---------------------------------------------------------------------
struct AttnPlan {
  bool tc;    // the tensor-core kernel
  int rows;   // rows of a row tile
  int row_tiles, grid;
  size_t o_off, ml_off, cut_off, ws_bytes;
};

// The warp-level kernel for a few rows (one 16-row MMA tile while they fit it, two
// up to 32 rows, so that a key is loaded half as often), the tensor cores' 128-row
// tiles above; 256 channels, and strides that no tensor map takes, stay with the
// warp-level kernel.
AttnPlan attn_plan(int M, int D, bool tc_takes, int sms) {
  AttnPlan p;
  p.tc = tc_takes && M > 16;
  p.rows = p.tc ? attn_tc_rows(M) : M <= 16 || D == 256 ? 16 : 32;
  p.row_tiles = (M + p.rows - 1) / p.rows;
  p.grid = p.tc ? attn_tc_grid(p.rows, sms) : sms * (D == 256 ? 1 : 2);
  p.o_off = 0;
  p.ml_off = align_up(size_t(p.grid) * 2 * p.rows * D * sizeof(float), 256);
  p.cut_off = p.ml_off + align_up(size_t(p.grid) * 2 * p.rows * sizeof(float2), 256);
  p.ws_bytes = p.cut_off + align_up(size_t(p.grid) * sizeof(Cut), 256);
  return p;
}

template <typename E, int D, int kRows>
cudaError_t launch_warp(const AttnArgs& a, cudaStream_t s) {
  auto kernel = attn_warp_kernel<E, D, kRows>;
  constexpr size_t smem = WarpCfg<D, kRows>::kSmem;
  const cudaError_t e = cudaFuncSetAttribute(
      kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
  if (e != cudaSuccess) return e;
  return launch_k(kernel, dim3(a.grid), dim3(kWThreads), smem, s, true, a);
}

template <typename E, int D>
cudaError_t launch_attn(const AttnArgs& a, const AttnPlan& p, const dfl2_cache* c,
                        cudaStream_t s) {
  cudaError_t e;
  if (p.tc)
    e = launch_attn_tc(a, c, s);
  else if (D == 256 || p.rows == 16)
    e = launch_warp<E, D, 16>(a, s);
  else
    e = launch_warp<E, D, D == 256 ? 16 : 32>(a, s);
  if (e != cudaSuccess) return e;
  const int rows = std::min(a.rows, a.t.T * a.G);
  return launch_k(combine_kernel<E, D>, dim3(a.grid + a.B, (rows + kCombineWarps - 1) / kCombineWarps),
                  dim3(kCombineWarps * 32), 0, s, true, a);
}

template <typename E>
cudaError_t launch_attn_d(const AttnArgs& a, const AttnPlan& p, const dfl2_cache* c,
                          cudaStream_t s) {
  return c->head_dim == 64    ? launch_attn<E, 64>(a, p, c, s)
         : c->head_dim == 128 ? launch_attn<E, 128>(a, p, c, s)
                              : launch_attn<E, 256>(a, p, c, s);
}

dfl2_status check_shapes(int B, int T, int q_heads, int kv_heads, int head_dim, int dtype) {
  if (B < 1 || T < 1 || q_heads < 1 || kv_heads < 1)
    return report_errorf(DFL2_ERR_INVALID_ARG, "B=%d, T=%d, q_heads=%d, kv_heads=%d must be >= 1",
                         B, T, q_heads, kv_heads);
  if (q_heads % kv_heads)
    return report_errorf(DFL2_ERR_INVALID_ARG, "q_heads=%d is no multiple of kv_heads=%d", q_heads,
                         kv_heads);
  if (B > 65535 || T > kMaxTree || q_heads > 65535)
    return report_errorf(DFL2_ERR_UNSUPPORTED, "B=%d, T=%d, q_heads=%d: at most 65535, %d, 65535",
                         B, T, q_heads, kMaxTree);
  if (head_dim != 64 && head_dim != 128 && head_dim != 256)
    return report_errorf(DFL2_ERR_UNSUPPORTED, "head_dim=%d: 64, 128 or 256", head_dim);
  if (dtype != DFL2_BF16 && dtype != DFL2_F16)
    return report_errorf(DFL2_ERR_UNSUPPORTED, "dtype %d: the attention takes bf16 and fp16", dtype);
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

size_t dfl2_tree_attn_workspace_size(int B, int T, int q_heads, int kv_heads, int head_dim,
                                     dfl2_dtype dtype) {
  if (dfl2::check_shapes(B, T, q_heads, kv_heads, head_dim, dtype) != DFL2_OK) return 0;
  if (dfl2::check_args_device(nullptr, 0) != DFL2_OK) return 0;
  // (whichever kernel the cache's strides will allow)
  const int M = T * (q_heads / kv_heads), sms = dfl2::device_info().sms;
  const bool tc = head_dim != 256;
  return std::max(dfl2::attn_plan(M, head_dim, false, sms).ws_bytes,
                  dfl2::attn_plan(M, head_dim, tc, sms).ws_bytes);
}

dfl2_status dfl2_tree_attn(const void* q, const int64_t* q_strides, const dfl2_cache* cache,
                           int layer, int B, int T, int q_heads, const int32_t* table_rows,
                           const int32_t* length, const int32_t* count, const uint32_t* mask,
                           float scale, void* out, const int64_t* out_strides, float* lse,
                           void* ws, size_t ws_bytes, dfl2_stream stream) {
  const dfl2::PtrArg ptrs[] = {{q, "q", 16}, {table_rows, "table_rows", 4, true},
                               {length, "length", 4}, {count, "count", 4, true},
                               {mask, "mask", 4, true}, {out, "out", 16}, {lse, "lse", 4, true}};
  DFL2_TRY(dfl2::check_cache_host(cache));
  DFL2_TRY(dfl2::check_shapes(B, T, q_heads, cache->kv_heads, cache->head_dim, cache->dtype));
  DFL2_TRY(dfl2::check_args_host(ptrs, 7));
  if (layer < 0 || layer >= cache->layers)
    return dfl2::report_errorf(DFL2_ERR_INVALID_ARG, "layer %d of %d", layer, cache->layers);
  if (!q_strides || !out_strides)
    return dfl2::report_errorf(DFL2_ERR_INVALID_ARG, "q_strides and out_strides are needed");
  for (int i = 0; i < 3; ++i)
    if (q_strides[i] < 0 || q_strides[i] % 8 || out_strides[i] < 0 || out_strides[i] % 8)
      return dfl2::report_errorf(DFL2_ERR_INVALID_ARG,
                                 "strides of q and out: non-negative multiples of 8");
  if (!std::isfinite(scale))
    return dfl2::report_errorf(DFL2_ERR_INVALID_ARG, "scale %g must be finite", double(scale));
  DFL2_TRY(dfl2::check_args_device(ptrs, 7));
  DFL2_TRY(dfl2::check_cache_device(cache));
  const int G = q_heads / cache->kv_heads, D = cache->head_dim;
  const dfl2::AttnPlan p = dfl2::attn_plan(T * G, D, dfl2::attn_tc_takes(cache), dfl2::device_info().sms);
  if (!ws || ws_bytes < p.ws_bytes)
    return dfl2::report_errorf(DFL2_ERR_WORKSPACE, "workspace of %zu bytes < %zu needed",
                               ws ? ws_bytes : size_t(0), p.ws_bytes);
  const dfl2::PtrArg wsp[] = {{ws, "workspace", 16}};
  DFL2_TRY(dfl2::check_args_host(wsp, 1));
  DFL2_TRY(dfl2::check_args_device(wsp, 1));
  uint8_t* w = static_cast<uint8_t*>(ws);
  const int64_t at = layer * cache->layer_stride * 2;
  dfl2::AttnArgs a{};
  a.t = dfl2::table_view(cache, table_rows, length, count, T);
  a.q = q;
  a.qb = q_strides[0];
  a.qt = q_strides[1];
  a.qh = q_strides[2];
  a.k = static_cast<const uint8_t*>(cache->k) + at;
  a.v = static_cast<const uint8_t*>(cache->v) + at;
  a.page_stride = cache->page_stride;
  a.head_stride = cache->head_stride;
  a.slot_stride = cache->slot_stride;
  a.mask = mask;
  a.W = (T + 31) / 32;
  a.B = B;
  a.H = cache->kv_heads;
  a.G = G;
  a.scale_log2 = scale * dfl2::kLog2e;
  a.out = out;
  a.ob = out_strides[0];
  a.ot = out_strides[1];
  a.oh = out_strides[2];
  a.lse = lse;
  a.part_o = reinterpret_cast<float*>(w + p.o_off);
  a.part_ml = reinterpret_cast<float2*>(w + p.ml_off);
  a.cuts = reinterpret_cast<dfl2::Cut*>(w + p.cut_off);
  a.grid = p.grid;
  a.rows = p.rows;
  a.row_tiles = p.row_tiles;
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e = cache->dtype == DFL2_F16
                            ? dfl2::launch_attn_d<__half>(a, p, cache, s)
                            : dfl2::launch_attn_d<__nv_bfloat16>(a, p, cache, s);
  return e == cudaSuccess ? DFL2_OK : dfl2::report_cuda_error(e, "tree attention launch");
}

}  // extern "C"
