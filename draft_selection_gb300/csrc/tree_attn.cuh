// The attention kernels' arguments, the division of their work into units, what a
// node sees, and small conversions.  Not public.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <type_traits>

#include "cache.cuh"

namespace dfl2 {
namespace {  // each translation unit its own copy

constexpr unsigned kAll = 0xffffffffu;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr int kKeys = 64;  // keys of a tile

}  // namespace

// The keys of a sequence and head that several ranges have parts of, as each CTA
// leaves it for combine_kernel (b < 0: none): the ranges c0 .. c1, in the order of
// the keys, and which of its two places c0's part is in (the others': the first).
struct alignas(16) Cut {
  int b;
  int h_n;      // h * 1024 + the sequence's nodes (at most kMaxTree)
  int c0;
  int c1_slot;  // c1 * 2 + slot
};

struct AttnArgs {
  TableView t;
  const void* q;
  int64_t qb, qt, qh;  // element strides
  const void* k;       // the layer's keys and values
  const void* v;
  int64_t page_stride, head_stride, slot_stride;
  const uint32_t* mask;  // [B][T][W], or NULL: a chain
  int W;
  int B, H, G;           // sequences, key heads, query heads per key head
  float scale_log2;      // scale * log2 e
  void* out;
  int64_t ob, ot, oh;
  bool out32;      // every row of out begins on 32 bytes: stored so (143 us, 16 at a time 146:
                   // 64 trees of 33 nodes)
  float* lse;      // nullable
  float* part_o;   // [CTAs][2][streams][128 rows x D] unnormalised outputs (part_at)
  float2* part_ml; // [CTAs][2][rows] (maximum, sum)
  Cut* cuts;       // [CTAs][2]: of the row tiles a CTA goes on with, and begins
  int grid;        // ranges that the units are cut into; row_tiles CTAs share one
  int stream_rows; // rows of a stream: whole nodes, at most 128
  int rows;        // rows of a row tile
  int row_tiles;   // ceil(T G / rows)
  // with a window (kernels with kWin): a node sees, of what it would see without, the first
  // `sinks` positions and those less than `window` before its own
  int sinks, window;
  const int32_t* depth;  // [B][T] a node's own position behind the length, or NULL: its number
};
// What the attention's entry points and dfl2_cache_weigh take.
dfl2_status check_attn_shapes(int B, int T, int q_heads, int kv_heads, int head_dim, int dtype);
cudaError_t launch_window_attn(const AttnArgs& a, const dfl2_cache* c, cudaStream_t s);

namespace {

// What a row of length `len` and `n` nodes amounts to; n == 0: no units.
struct Seq {
  int row, len, n, tiles;
};
// With a window the units are the tiles that a node may see something of: those of the
// sinks, and those from the first one that reaches into the first node's window on.
struct Gap {
  int at, size;  // tiles at, .. at + size - 1 are left out
};
__device__ __forceinline__ Gap gap_of(const AttnArgs& a, int len, int tiles) {
  Gap g;
  g.at = min(tiles, (a.sinks + kKeys - 1) / kKeys);
  g.size = max(0, max(0, len - a.window + 1) / kKeys - g.at);
  return g;
}
// The tile of keys that a sequence's unit is.
template <bool kWin>
__device__ __forceinline__ int key_tile(const AttnArgs& a, const Seq& s, int tile) {
  if (!kWin) return tile;
  const Gap g = gap_of(a, s.len, (s.len + s.n + kKeys - 1) / kKeys);
  return tile < g.at ? tile : tile + g.size;
}
// Whether a node may miss something of a tile of keys (that of position p0 on): it has nodes,
// or positions past the end, or reaches out of the sinks or a node's window.
template <bool kWin>
__device__ __forceinline__ bool is_edge(const AttnArgs& a, const Seq& s, int key) {
  if (!kWin) return key >= s.len / kKeys;
  const int p0 = key * kKeys;
  return p0 + kKeys > s.len ||
         (p0 + kKeys > a.sinks && p0 < s.len + a.t.T - a.window);  // (depths are below T)
}
template <bool kWin>
__device__ __forceinline__ Seq load_seq(const AttnArgs& a, int b) {
  Seq s;
  s.len = a.t.length[b];
  s.n = a.t.count_of(b);
  s.row = a.t.seq ? a.t.seq[b] : b;
  if (!a.t.in_range(s.row, s.len)) {  // (one branch, behind all the loads)
    record_error(a.t.err, kDevErrBadIndex);
    s.n = 0;
  }
  s.tiles = s.n > 0 ? (s.len + s.n + kKeys - 1) / kKeys : 0;
  if (kWin && s.n > 0) s.tiles -= gap_of(a, s.len, s.tiles).size;
  return s;
}

// Where range c of `units` units in `n` ranges begins, and which range unit u is in.
// (32-bit divisions where they do: a 64-bit one is a chain of some 100 instructions.)
__device__ __forceinline__ int64_t range_start(int64_t units, int n, int c) {
  if (units < (1 << 20))  // n and c are at most a few thousand
    return static_cast<uint32_t>(units) * static_cast<uint32_t>(c) / static_cast<uint32_t>(n);
  return units * c / n;
}
__device__ __forceinline__ int range_of(int64_t units, int n, int64_t u) {
  if (units < (1 << 20))
    return ((static_cast<uint32_t>(u) + 1) * static_cast<uint32_t>(n) - 1) /
           static_cast<uint32_t>(units);
  return static_cast<int>(((u + 1) * n - 1) / units);
}

// A place in a range of units.
template <bool kWin>
struct Cursor {
  int64_t u;
  int b, h, tile;  // sequence, key head, tile
  Seq s;
  // On to tile `hi` of this head, or, where that is its end, to the next one.
  __device__ __forceinline__ void to(const AttnArgs& a, int hi) {
    u += hi - 1 - tile;
    tile = hi - 1;
    next(a);
  }
  __device__ __forceinline__ void next(const AttnArgs& a) {
    ++u;
    if (++tile < s.tiles) return;
    tile = 0;
    if (++h < a.H) return;
    h = 0;
    do {
      if (++b >= a.B) return;
      s = load_seq<kWin>(a, b);
    } while (s.tiles == 0);
  }
};

// 2^x to two units in the last place; results below 2^-126 become 0.
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// Range `cta` [u0, u1) of the units in n_cta ranges, and the place where it begins, by a
// warp together.  Up to 32 sequences need one load of their lengths.
template <bool kWin>
struct Range {
  int64_t units, u0, u1;
  int n_cta;
  Cursor<kWin> first;  // if u0 < u1
};
template <bool kWin>
__device__ __forceinline__ Range<kWin> find_range(const AttnArgs& a, int cta) {
  const int lane = threadIdx.x & 31;
  Range<kWin> g;
  Seq own;
  int sum;  // tiles of the sequences up to this lane's: 32 times 2^24 at most
  auto load = [&](int b0) {
    own = b0 + lane < a.B ? load_seq<kWin>(a, b0 + lane) : Seq{0, 0, 0, 0};
    sum = own.tiles;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int y = __shfl_up_sync(kAll, sum, off);
      if (lane >= off) sum += y;
    }
  };
  load(0);
  g.units = static_cast<int64_t>(__shfl_sync(kAll, sum, 31)) * a.H;
  if (a.B > 32) {
    int64_t x = 0;
    for (int b = lane + 32; b < a.B; b += 32) x += load_seq<kWin>(a, b).tiles;
#pragma unroll
    for (int off = 16; off; off >>= 1) x += __shfl_xor_sync(kAll, x, off);
    g.units += x * a.H;
  }
  g.n_cta = static_cast<int>(min(static_cast<int64_t>(a.grid), g.units));
  g.u0 = g.u1 = 0;
  if (cta >= g.n_cta) return g;
  g.u0 = range_start(g.units, g.n_cta, cta);
  g.u1 = range_start(g.units, g.n_cta, cta + 1);
  // the sequence that u0 falls in
  int64_t base = 0;
  for (int b0 = 0; b0 < a.B; b0 += 32) {
    if (b0 > 0) load(b0);
    const unsigned hit = __ballot_sync(kAll, g.u0 < base + static_cast<int64_t>(sum) * a.H);
    if (hit) {
      const int w = __ffs(hit) - 1;
      const int64_t before =
          base + static_cast<int64_t>(__shfl_sync(kAll, sum - own.tiles, w)) * a.H;
      g.first.u = g.u0;
      g.first.b = b0 + w;
      g.first.s = Seq{__shfl_sync(kAll, own.row, w), __shfl_sync(kAll, own.len, w),
                      __shfl_sync(kAll, own.n, w), __shfl_sync(kAll, own.tiles, w)};
      // within one sequence: at most 2^24 tiles of each of its heads
      const int64_t in = g.u0 - before;
      g.first.h = in < (1ll << 32)
                       ? static_cast<int>(static_cast<uint32_t>(in) /
                                          static_cast<uint32_t>(g.first.s.tiles))
                       : static_cast<int>(in / g.first.s.tiles);
      g.first.tile = static_cast<int>(in - static_cast<int64_t>(g.first.h) * g.first.s.tiles);
      return g;
    }
    base += static_cast<int64_t>(__shfl_sync(kAll, sum, 31)) * a.H;
  }
  g.u1 = g.u0;  // the lengths changed in between: no work, and no endless search
  return g;
}

// Of the head whose first unit is v0.
template <bool kWin>
__device__ __forceinline__ Cut make_cut(const Range<kWin>& g, int64_t v0, int b, int h, const Seq& s) {
  const int c0 = range_of(g.units, g.n_cta, v0), c1 = range_of(g.units, g.n_cta, v0 + s.tiles - 1);
  return Cut{b, h * 1024 + s.n, c0, c1 * 2 + (range_start(g.units, g.n_cta, c0) < v0 ? 1 : 0)};
}

template <typename E>
__device__ __forceinline__ uint32_t pack2(float x, float y) {  // x in the low half
  if constexpr (std::is_same_v<E, __half>) {
    const __half2 h = __floats2half2_rn(x, y);
    return *reinterpret_cast<const uint32_t*>(&h);
  } else {
    const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
}
template <typename E>
__device__ __forceinline__ float to_f32(E x) {
  if constexpr (std::is_same_v<E, __half>)
    return __half2float(x);
  else
    return __bfloat162float(x);
}
template <typename E>
constexpr uint32_t kExpMask = std::is_same_v<E, __half> ? 0x7C00u : 0x7F80u;

// Two elements with those that are Inf or NaN set to 0.
template <typename E>
__device__ __forceinline__ uint32_t finite2(uint32_t x) {
  constexpr uint32_t lo = kExpMask<E>, hi = lo << 16;
  if ((x & lo) == lo) x &= 0xFFFF0000u;
  if ((x & hi) == hi) x &= 0x0000FFFFu;
  return x;
}
// Whether one of eight elements is Inf or NaN: an exponent of all ones and one more
// in its last place carries into the place of the sign, and no further.
template <typename E>
__device__ __forceinline__ bool not_finite(uint4 x) {
  constexpr uint32_t m = kExpMask<E> * 0x10001u, one = (kExpMask<E> & -kExpMask<E>) * 0x10001u;
  return (((x.x & m) + one) | ((x.y & m) + one) | ((x.z & m) + one) | ((x.w & m) + one)) &
         0x80008000u;
}

}  // namespace

}  // namespace dfl2
