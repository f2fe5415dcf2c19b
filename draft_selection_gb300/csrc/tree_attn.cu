// Attention of a tree of drafted tokens over the paged cache (include/dfl2.h,
// dfl2_tree_attn):
//   o_i = sum_j p_ij v_j,  p_ij = exp(s_ij) / sum_j exp(s_ij),  s_ij = scale <q_i, k_j>
// over the positions j that node i sees.
//
// The G = q_heads / kv_heads query heads that share a key head read the same
// keys, so the T nodes and G heads make one matrix of M = T G rows against the
// keys of (sequence, key head): row r is node r / G, head h G + r % G.  Each key
// and value is then read once per row tile of up to 256 rows, and the work is two
// matrix products around an exponential.
//
// Split.  Lengths live on the device and differ by sequence, so the host
// cannot cut the work.  A unit is one tile of keys of one sequence and key head;
// the units are cut into equal, contiguous ranges, whatever sequences they span, as
// many as the GPU holds CTAs, or where the M rows need several row tiles, as many
// as it holds groups of one CTA for each row tile: the CTAs of a group walk the
// same keys side by side, so that HBM is read once and L2 serves the rest (with
// each row tile a range of its own, 32 sequences of 16 to 32 thousand positions and
// 512 rows read their keys twice: 1.37 ms instead of 1.20).  A CTA that covers
// all tiles of a head writes its output; one that covers a part writes its running
// maximum, sum and unnormalised output to the workspace (a range has at most two
// such ends), and combine_kernel adds the parts in the order of the keys.
//
// Softmax in one pass: with the running maximum m and sum l of a row, a tile
// with row maximum m' multiplies l and o by 2^(m - m') before adding its own
// terms (scores are kept times log2 e, so that exp is exp2).
//
// For a row tile of 128 rows (node, head) and tiles of 64 keys:
//   S = Q K^T   tcgen05.mma, 128 x 64, Q and K in shared memory, S (float32) in TMEM
//   P = 2^(scale log2 e S - m)   a thread to a row: its 64 scores come from TMEM,
//               its weights go back there, rounded to the cache's type (float16: times
//               2^7, and so is l: kLift)
//   O += P V    tcgen05.mma, 128 x D, P in TMEM, V in shared memory as it lies in
//               the cache (keys x channels: the channel-major operand), O in TMEM
// A row's statistics never leave its thread, so the softmax has no exchange at
// all.  O is rescaled only when a row's maximum has risen by more than 2^8 since
// the reference m was taken: weights up to 2^8 lose nothing in float32 sums or in
// rounding to a floating type, and the rescaling (TMEM -> registers -> TMEM, after
// the products in flight) then almost never happens past a row's first tiles.
//
// A page that a sequence lacks is read as NaN in K and as zeros in V.  A row's maximum is NaN
// then, and only in that case does it look for such positions, which it leaves out.  (A word
// of each tile's missing pages read with its scores, or the scores replaced in place, cost
// every tile: 64 trees of 33 nodes 142.8 and 141.5 us instead of 141.0, 9 trees of 61 nodes
// and 64 channels 34.0 and 33.5 instead of 32.8.)
//
// Roles: warp 0 loads K and V (TMA boxes of one page's rows x 64 channels,
// 128-byte swizzle, into a ring of slots of one tile's K or V); a stream, 128
// rows, has one warp that issues its MMAs and four that do its softmax.  A row's
// scores are in registers soon after they are in TMEM, so one S is enough: the
// scores of tile i+1 are computed over those of tile i while its softmax runs.  P
// has two buffers, so neither product ever waits for the other one (with two S
// and P written over S, tile i+1's scores waited for tile i-1's output: 1830 cycles
// a tile of two streams instead of 1450).
// With M = T G rows up to 128: one stream, two CTAs on an SM.  Above: one CTA with
// two streams (256 rows), which share each K and V tile, so that a tile crosses L2
// and fills shared memory once for 256 rows.
//
// Bounds.  A tile of 64 keys of 128 channels is 32 KB: 1400 cycles of one SM's share
// of HBM.  Its MMAs take a stream 384 + 256 cycles (measured: 48 for 128 x 64 x 16
// with both operands in shared memory, which reads 6 KB at 128 bytes a cycle, 64 for
// 128 x 128 x 16 with A in TMEM).  Its softmax is a chain of 1350 to 1600 cycles a tile
// for a warp that shares its scheduler with the other stream's: the scores from TMEM 125,
// their maximum 190, the exponentials 540 alone and 640 to 770 beside the other warp's
// (their unit: 256 each), barriers and the weights' store the rest.  So HBM bounds up to
// 128 rows, all three meet at 256 (about 1400 cycles a tile), the tensor cores bound what
// has more rows of 128 channels, and the softmax what has more of 64.
#include <cuda.h>
#include <cudaTypedefs.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <mutex>

#include "tree_attn.cuh"

namespace dfl2 {
namespace {

constexpr int kLanes = 128;                // rows of a stream: the TMEM lanes
constexpr float kRise = 8.f;               // log2 of the rise that O is rescaled at
// log2 of what the weights are taken times: with kRise they stay below float16's largest
// number, 2^16, and a long tail of small ones that much above its smallest, 2^-24 (60,000
// weights of 2^-19 beside one of 1 were 1.6% too large).  bfloat16 has float32's exponents.
template <typename E>
constexpr float kLift = std::is_same_v<E, __half> ? 7.f : 0.f;
template <typename E>
constexpr float kUnlift = std::is_same_v<E, __half> ? 1.f / 128.f : 1.f;
constexpr uint32_t kColP = kKeys, kColO = 2 * kKeys;

template <int D, int NS>
struct TcCfg {
  // 256 channels fill the SM with one stream: O alone is half of TMEM
  static constexpr int kCtas = NS == 1 && D < 256 ? 2 : 1;     // on an SM
  static constexpr uint32_t kStreamCols = D < 256 ? 256 : 512;  // TMEM columns: S, P, P, O
  static constexpr int kSlot = kKeys * D * 2;                  // bytes of a tile's K (or V)
  static constexpr int kRing = 163840 / kCtas / kSlot;
  static constexpr int kSlots = kRing < 16 ? kRing : 16;
  static constexpr int kQ = kLanes * D * 2;                    // bytes of a stream's Q
  static constexpr int kThreads = 32 * (1 + NS) + NS * kLanes;
  static constexpr int kBars = 2 * kSlots + NS * 8;
  static constexpr int kBadSegs = 16;
  static constexpr int kHoles = 16;
  static constexpr size_t kSmem = size_t(NS) * kQ + size_t(kSlots) * kSlot + kBars * 8 +
                                  (1 + kBadSegs + 4 + 2 * kHoles) * 4;
  static_assert(kBadSegs > kSlots / 2 + 1, "a head's mark outlives its last reader");
  static_assert(kHoles > kSlots / 2 + 3, "a tile's holes outlive their last reader");
  static_assert(NS * kStreamCols * kCtas <= 512, "TMEM");
  static_assert((kSmem + 1024) * kCtas <= 233472, "shared memory");
};

// A wait whose first look nearly always succeeds; the rest is out of line, which
// keeps the loops that wait short (mbar_wait in place, with a vote, took 85 cycles
// when there was nothing to wait for, and more once its code had left the cache).
// Lanes that wait together give up together: one that went on alone would wait at the
// warp's next barrier for ever.
__device__ __noinline__ bool wait_on(uint64_t* bar, uint32_t parity, uint32_t* err) {
  const unsigned lanes = __activemask();
  const long long t0 = clock64();
  while (!__any_sync(lanes, mbar_try_wait(bar, parity)))
    if (__any_sync(lanes, wait_expired(t0, err))) {
      record_error(err, kDevErrAttn);
      return false;
    }
  return true;
}
__device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity, uint32_t* err) {
  if (mbar_try_wait(bar, parity)) return true;
  return wait_on(bar, parity, err);
}

// One lane of a converged warp, the same one each time.
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(r));
  return r != 0;
}
// Operand of 128-byte rows in the 128-byte swizzle whose contiguous dimension is
// not the summed one: 64-element blocks along it `block` bytes apart, groups of
// eight summed indices 1024 bytes apart.
__device__ __forceinline__ uint64_t umma_desc_sw128_mn(const void* smem_tile, uint32_t block) {
  uint64_t d = (static_cast<uint64_t>(smem_u32(smem_tile)) >> 4) & 0x3FFFull;
  d |= static_cast<uint64_t>(block >> 4) << 16;  // leading byte offset
  d |= uint64_t(1024 >> 4) << 32;                // stride byte offset
  d |= uint64_t(1) << 46;
  d |= uint64_t(2) << 61;
  return d;
}
// kind::f16, float32 accumulator; b_mn: B's contiguous dimension is N.
template <typename E>
__host__ __device__ constexpr uint32_t idesc_f16(int M, int N, bool b_mn) {
  const uint32_t f = std::is_same_v<E, __half> ? 0u : 1u;
  return (1u << 4) | (f << 7) | (f << 10) | ((b_mn ? 1u : 0u) << 16) |
         (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(M >> 4) << 24);
}
// As umma_bf16 with A in TMEM.
__device__ __forceinline__ void umma_f16_ts(uint32_t tmem_d, uint32_t tmem_a, uint64_t bdesc,
                                            uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(tmem_d),
      "r"(tmem_a), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}

__device__ __forceinline__ void tmem_ld32_issue(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, "
      "%11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, "
      "%28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]),
        "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]),
        "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]),
        "=r"(r[31])
      : "r"(taddr)
      : "memory");
}
// Waits for this thread's tcgen05.ld; names r so that nothing reads it before.
__device__ __forceinline__ void tmem_ld32_wait(uint32_t* r) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]),
                 "+r"(r[6]), "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]),
                 "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]), "+r"(r[16]), "+r"(r[17]),
                 "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]),
                 "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]),
                 "+r"(r[30]), "+r"(r[31])
               :
               : "memory");
}
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, "
      "%10, %11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, "
      "%27, %28, %29, %30, %31};" ::"r"(r[0]),
      "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
      "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]),
      "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]),
      "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]),
      "r"(r[30]), "r"(r[31]), "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_st_wait() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tma_load_4d(void* dst, const void* tmap, int x, int y, int z,
                                            int w, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(smem_u32(dst)),
      "l"(tmap), "r"(x), "r"(y), "r"(z), "r"(w), "r"(smem_u32(bar))
      : "memory");
}

// Two float32 operations in one instruction, and a maximum of three.
__device__ __forceinline__ uint64_t pack_f32x2(float x, float y) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
  return r;
}
__device__ __forceinline__ uint64_t pack_u32x2(uint32_t x, uint32_t y) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "r"(x), "r"(y));
  return r;
}
__device__ __forceinline__ void unpack_f32x2(uint64_t r, float& x, float& y) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(r));
}
__device__ __forceinline__ uint64_t fma_f32x2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add_f32x2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ float max3(float a, float b, float c) {  // NaN if one is
  float r;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ float max64(const uint32_t* x) {
  float mx[4];
#pragma unroll
  for (int c = 0; c < 4; ++c) mx[c] = __uint_as_float(x[c]);
#pragma unroll
  for (int c = 4; c < 60; c += 8)
#pragma unroll
    for (int z = 0; z < 4; ++z)
      mx[z] = max3(mx[z], __uint_as_float(x[c + z]), __uint_as_float(x[c + 4 + z]));
  return max3(max3(mx[0], __uint_as_float(x[60]), __uint_as_float(x[61])),
              max3(mx[1], __uint_as_float(x[62]), __uint_as_float(x[63])),
              max3(mx[2], mx[3], mx[3]));
}

// 32 bytes: a whole sector a thread, where rows lie apart (a store of 16 costs as many
// passes for half the bytes)
__device__ __forceinline__ void st_v8(void* p, const uint32_t* r) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(r[0]),
               "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}
__device__ __forceinline__ void prefetch_l1(const void* p) {
  asm volatile("prefetch.global.L1 [%0];" ::"l"(p));
}
__device__ __forceinline__ void tma_prefetch_4d(const void* tmap, int x, int y, int z, int w) {
  asm volatile("cp.async.bulk.prefetch.tensor.4d.L2.global.tile [%0, {%1, %2, %3, %4}];" ::"l"(
                   tmap),
               "r"(x), "r"(y), "r"(z), "r"(w)
               : "memory");
}

// Where 8 channels, from 8 c on, of a row of a stream's part are in part_o.  The 32 bytes
// of four rows lie side by side, so a warp's store of 32 bytes a thread is of 8 whole
// lines, not of 32 quarters (9 trees of 61 nodes, 7 heads of 64 channels a key head: 33.7
// us, row by row 35.3; 64 trees of 33 nodes 143.3 and 144.1; 0.2 more for one token).
constexpr int kPartStep = 4 * 8;  // floats from 8 channels to the next 8
template <int D>
__device__ __forceinline__ int part_at(int stream, int row, int c) {
  return stream * (kLanes * D) + (row >> 2) * (4 * D) + c * kPartStep + (row & 3) * 8;
}

// Which of the 64 positions from p0 on node i of sequence b sees (0 past the end).
__device__ __forceinline__ uint64_t seen64(const AttnArgs& a, int b, const Seq& s, int i, int p0) {
  if (i >= s.n) return 0;
  const int ctx = max(0, min(64, s.len - p0));  // committed positions of the tile
  uint64_t vis = ctx == 64 ? ~0ull : (1ull << ctx) - 1;
  if (ctx == 64) return vis;
  const int j0 = p0 + ctx - s.len;              // first node of the tile
  if (j0 >= s.n) return vis;
  uint64_t nodes;
  if (a.mask) {
    const uint32_t* w = a.mask + (static_cast<int64_t>(b) * a.t.T + i) * a.W;
    const int w0 = j0 >> 5;
    const uint64_t lo = w[w0], mid = w0 + 1 < a.W ? w[w0 + 1] : 0,
                   hi = w0 + 2 < a.W ? w[w0 + 2] : 0;
    const int sh = j0 & 31;
    nodes = ((lo | mid << 32) >> sh) | (sh ? hi << (64 - sh) : 0);
  } else {
    nodes = i < j0 ? 0 : i - j0 >= 63 ? ~0ull : (2ull << (i - j0)) - 1;
  }
  const int left = s.n - j0;
  if (left < 64) nodes &= (1ull << left) - 1;
  return vis | nodes << ctx;
}

// A row's 64 scores at TMEM address `at`: those of positions whose pages are among `hole`
// (bit z * kBlk: the tile's z-th page) are NaN and become -inf.  The row's maximum.
template <int kBlk>
__device__ __noinline__ float leave_out(uint32_t at, uint32_t hole, int page_shift) {
  uint32_t x[64];
  tmem_ld32_issue(at, x);
  tmem_ld32_issue(at + 32, x + 32);
  tmem_ld32_wait(x);
  tmem_ld32_wait(x + 32);
#pragma unroll
  for (int c = 0; c < 64; ++c)
    if (hole >> (c >> page_shift) * kBlk & 1) x[c] = 0xFF800000u;
  tmem_st32(at, x);
  tmem_st32(at + 32, x + 32);
  tmem_st_wait();
  return max64(x);
}

// The Inf and NaN values, of the nodes of positions [p0, p1), that node i (-1: none) sees,
// added to this row's O at TMEM address `to`, by a warp together.  Such values are kept out
// of the matrix product, where a weight of 0 would spread them to the nodes that do not see
// them; their sum decides its channel of the output.  Only called when there are any; a
// node's mask bit and page are looked up once for 32 channels (64 trees of 256 nodes, 8
// heads, one NaN in each tree: 2.7 ms, channel by channel 50).
template <typename E, int D>
__device__ __noinline__ void add_unseen(const AttnArgs& a, uint32_t to, int b, const Seq& s, int h,
                                        int i, int p0, int p1) {
  const int j0 = max(0, p0 - s.len), j1 = i < 0 ? 0 : min(p1 - s.len, s.n);
  const uint32_t* mask =
      a.mask ? a.mask + (static_cast<int64_t>(b) * a.t.T + max(0, i)) * a.W : nullptr;
  for (int c0 = 0; c0 < D; c0 += 32) {
    float y[32];
#pragma unroll
    for (int c = 0; c < 32; ++c) y[c] = 0.f;
    uint32_t word = 0;
    for (int j = j0; j < j1; ++j) {
      if (mask) {
        if (j == j0 || (j & 31) == 0) word = mask[j >> 5];
        if (!(word >> (j & 31) & 1u)) continue;
      } else if (j > i) {
        break;
      }
      const int pos = s.len + j;
      const int64_t page = a.t.page_at(s.row, pos >> a.t.page_shift);
      if (page < 0) continue;
      const E* v = static_cast<const E*>(a.v) + page * a.page_stride + h * a.head_stride +
                   (pos & ((1 << a.t.page_shift) - 1)) * a.slot_stride + c0;
#pragma unroll
      for (int c = 0; c < 32; c += 8) {
        const uint4 x = *reinterpret_cast<const uint4*>(v + c);
        if (!not_finite<E>(x)) continue;
        const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int z = 0; z < 8; ++z) {
          const uint16_t bits = static_cast<uint16_t>(w[z / 2] >> (z % 2 * 16));
          const float f = to_f32(*reinterpret_cast<const E*>(&bits));
          if (!isfinite(f)) y[c + z] += f;
        }
      }
    }
    __syncwarp();
    uint32_t o[32];
    tmem_ld32_issue(to + c0, o);
    tmem_ld32_wait(o);
#pragma unroll
    for (int c = 0; c < 32; ++c) o[c] = __float_as_uint(__uint_as_float(o[c]) + y[c]);
    tmem_st32(to + c0, o);
  }
  tmem_st_wait();
}

template <typename E, int D, int NS>
__global__ void __launch_bounds__(TcCfg<D, NS>::kThreads, TcCfg<D, NS>::kCtas)
    attn_kernel(const __grid_constant__ AttnArgs a, const __grid_constant__ CUtensorMap tmQ,
                const __grid_constant__ CUtensorMap tmK,
                const __grid_constant__ CUtensorMap tmV) {
  using C = TcCfg<D, NS>;
  constexpr int kBlk = D / 64;          // 64-channel blocks of a row
  constexpr int kBlkBytes = kKeys * 128;  // one block of a K or V slot
  extern __shared__ __align__(1024) uint8_t smem[];
  uint8_t* qs = smem;                   // [NS][kBlk][128 rows][128 B]
  uint8_t* ring = smem + NS * C::kQ;    // [slots][kBlk][64 keys][128 B]
  uint64_t* full = reinterpret_cast<uint64_t*>(ring + C::kSlots * C::kSlot);
  uint64_t* empty = full + C::kSlots;
  uint64_t* q_full = empty + C::kSlots;  // [NS] a row tile's Q is in place
  uint64_t* s_full = q_full + NS;        // [NS] scores are in TMEM
  uint64_t* s_read = s_full + NS;        // [NS] and in registers
  // The weights of tile i, and the output product that took them, have a barrier for
  // even and one for odd tiles, as P has: each side may be a tile ahead of the other,
  // and a barrier's parity tells only two neighbouring phases apart.
  uint64_t* p_ready = s_read + NS;       // [NS][2] weights are in TMEM
  uint64_t* pv_done = p_ready + 2 * NS;  // [NS][2] the output product is in O
  uint64_t* all_done = pv_done + 2 * NS; // [NS]
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(all_done + NS);
  // Heads of this CTA's range, counted up, that met Inf or NaN in V.  Stream 0, which looks,
  // may be as many tiles, so heads, ahead of stream 1 as half the ring has slots.
  int* bad_seg = reinterpret_cast<int*>(tmem_slot + 1);  // [kBadSegs]
  // Edge tiles whose V each of stream 0's warps has cleaned, counted up: stream 0 may be
  // several tiles ahead of stream 1, more than a barrier's parity can tell apart, and one
  // of its warps a tile ahead of another, so that a sum over them would not say which
  // tile is clean.
  uint32_t* v_clean = reinterpret_cast<uint32_t*>(bad_seg + C::kBadSegs);  // [4]
  // A tile that lacks pages: its number in this CTA's range, and a bit for each of the loads'
  // lanes.  The loads may be as many tiles ahead of the softmax as half the ring has slots,
  // and those of the products in flight.
  int* hole_tile = reinterpret_cast<int*>(v_clean + 4);  // [kHoles]
  uint32_t* holes = v_clean + 4 + C::kHoles;             // [kHoles]

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid == 0) {
    for (int i = 0; i < C::kSlots; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], NS);
    }
    for (int s = 0; s < NS; ++s) {
      mbar_init(&q_full[s], 1);
      mbar_init(&s_full[s], 1);
      mbar_init(&s_read[s], 4);
      for (int z = 0; z < 2; ++z) {
        mbar_init(&p_ready[2 * s + z], 4);
        mbar_init(&pv_done[2 * s + z], 1);
      }
      mbar_init(&all_done[s], 1);
    }
    for (int i = 0; i < 4; ++i) v_clean[i] = 0;
    for (int i = 0; i < C::kBadSegs; ++i) bad_seg[i] = -1;
    for (int i = 0; i < C::kHoles; ++i) hole_tile[i] = -1;
    fence_mbar_init();
    tma_prefetch_desc(&tmQ);
    tma_prefetch_desc(&tmK);
    tma_prefetch_desc(&tmV);
  }
  if (warp == 1) tmem_alloc(tmem_slot, NS * C::kStreamCols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  pdl_wait();
  pdl_launch_dependents();

  // this CTA's range of units, and where it begins (each warp for itself)
  const int range = blockIdx.x / a.row_tiles, row_tile = blockIdx.x - range * a.row_tiles;
  const Range g = find_range(a, range);
  const int64_t u0 = g.u0;
  Cursor cur = g.first;
  int N = static_cast<int>(g.u1 - u0);
  if (smem_u32(smem) & 1023u) {  // the swizzle counts on it
    record_error(a.t.err, kDevErrAttn);
    N = 0;
  }
  constexpr int kFirst = 32 * (1 + NS);  // the first softmax thread
  if (tid == kFirst) {  // (it alone writes the cuts, below)
    a.cuts[2 * blockIdx.x].b = -1;
    a.cuts[2 * blockIdx.x + 1].b = -1;
  }
  // The ring's order is K(0), K(1), V(0), K(2), V(1), ..: as the MMAs read them.  V(i)'s place:
  auto seq_v = [N](int i) { return i + 1 < N ? 2 * i + 2 : 2 * i + 1; };

  if (warp == 0) {
    // ---- loads ----
    const int ps = 1 << a.t.page_shift;
    const int box = min(ps, kKeys);           // positions of a TMA box
    const int n_page = kKeys / box;           // pages of a tile
    const int my_page = lane / kBlk, my_blk = lane % kBlk;
    const bool mine = my_page < n_page;
    // A tile, and the table entry of this lane's page of it (unless past the end).  The
    // entry is read two tiles before it is looked at, so its latency is not the loop's
    // (decode of 64 x 8192 positions, 64 channels, pages of 16: 179 us, 206 with the entry
    // of the next tile looked at once; pages of 64: level).
    struct Tile {
      int h, tile, entry;
      bool past;
    };
    auto tile_at = [&](const Cursor& c) {
      const int pos = c.tile * kKeys + my_page * box;
      const bool past = !mine || pos >= c.s.len + c.s.n;
      return Tile{c.h, c.tile, past ? -1 : a.t.entry(c.s.row, pos >> a.t.page_shift), past};
    };
    // One page too far for none: V's rows are then zeros and K's NaN (map_4d).
    auto page_of = [&](const Tile& t, int i) {
      const bool in = static_cast<unsigned>(t.entry) < static_cast<unsigned>(a.t.pages);
      const uint32_t hole = __ballot_sync(kAll, !in && !t.past);
      if (hole && lane == 0) {  // before the arrival on K's barrier
        record_error(a.t.err, kDevErrBadIndex);
        hole_tile[i % C::kHoles] = i;
        holes[i % C::kHoles] = hole;
      }
      return in ? t.entry : a.t.pages;
    };
    int issued = 0;
    bool ok = true;
    int slot = 0, ph = 0;  // the next slot, and the phase of its last use
    auto load = [&](const CUtensorMap* tm, int h, int tile, int page) {
      if (issued >= C::kSlots && !wait(&empty[slot], ph ^ 1, a.t.err)) {
        ok = false;
        return;
      }
      if (lane == 0) mbar_arrive_expect_tx(&full[slot], C::kSlot);
      __syncwarp();
      if (mine) {
        uint8_t* dst = ring + slot * C::kSlot + my_blk * kBlkBytes + my_page * box * 128;
        const int at = (tile * kKeys) & (ps - 1);
        tma_load_4d(dst, tm, my_blk * 64, at, h, page, &full[slot]);
      }
      ++issued;
      if (++slot == C::kSlots) {
        slot = 0;
        ph ^= 1;
      }
    };
    Tile t{}, t1{}, t2{};  // this tile and the next two
    int v_h = 0, v_tile = 0, v_page = 0;
    if (N > 0) {
      t1 = tile_at(cur);
      cur.next(a);
    }
    if (N > 1) {
      t2 = tile_at(cur);
      cur.next(a);
    }
    for (int i = 0; i <= N && ok; ++i) {
      t = t1;
      t1 = t2;
      if (i + 2 < N) {
        t2 = tile_at(cur);
        cur.next(a);
      }
      int page = 0;
      if (i < N) {
        page = page_of(t, i);
        load(&tmK, t.h, t.tile, page);
      }
      if (i > 0 && ok) load(&tmV, v_h, v_tile, v_page);
      v_h = t.h;
      v_tile = t.tile;
      v_page = page;
    }
    // the copies still in flight land before the CTA ends
    for (int j = max(0, issued - C::kSlots); j < issued; ++j)
      mbar_wait(&full[j % C::kSlots], (j / C::kSlots) & 1, a.t.err);
  } else if (warp <= NS) {
    // ---- a stream's MMAs ----
    // The whole warp walks the loop and one elected lane issues: the descriptors are
    // then warp-uniform, which the MMA's operands have to be (from a single lane's
    // loop each MMA cost about 100 cycles of moves to uniform registers).
    constexpr uint32_t id_qk = idesc_f16<E>(kLanes, kKeys, false);
    constexpr uint32_t id_pv = idesc_f16<E>(kLanes, D, true);
    const int st = __shfl_sync(kAll, warp, 0) - 1;
    const uint32_t tb = __shfl_sync(kAll, tmem, 0) + st * C::kStreamCols;
    const uint64_t ad = umma_desc_sw128(qs + st * C::kQ);
    const uint64_t bd_qk = umma_desc_sw128(ring);
    const uint64_t bd_pv = umma_desc_sw128_mn(ring, kBlkBytes);
    const int n = __shfl_sync(kAll, N, 0);
    int slot = 0, ph = 0;  // the ring's next slot in MMA order, and its phase
    auto advance = [&]() {
      if (++slot == C::kSlots) {
        slot = 0;
        ph ^= 1;
      }
    };
    auto scores = [&](int i, int slot, int ph) {  // of tile i
      if (i > 0 && !wait(&s_read[st], (i - 1) & 1, a.t.err)) return false;
      if (!wait(&full[slot], ph, a.t.err)) return false;
      __syncwarp();
      tc_fence_after();
      if (elect_one()) {
        const uint64_t bd = bd_qk + slot * (C::kSlot >> 4);
#pragma unroll
        for (int kb = 0; kb < kBlk; ++kb)
#pragma unroll
          for (int k = 0; k < 4; ++k)
            umma_bf16(tb, ad + kb * (kLanes * 128 >> 4) + 2 * k, bd + kb * (kBlkBytes >> 4) + 2 * k,
                      id_qk, kb > 0 || k > 0);
        umma_commit(&s_full[st]);
        umma_commit(&empty[slot]);
      }
      __syncwarp();
      return true;
    };
    // This stream's rows of Q: G heads of the nodes from node0 on, row by row
    const int node0 = (row_tile * NS + st) * a.stream_rows / a.G;
    const uint32_t q_bytes = kBlk * 128 * a.stream_rows;
    int q_loads = 0;
    auto load_q = [&](const Cursor& c) {
      ++q_loads;
      if (elect_one()) {
        mbar_arrive_expect_tx(&q_full[st], q_bytes);
#pragma unroll
        for (int kb = 0; kb < kBlk; ++kb)
          tma_load_4d(qs + st * C::kQ + kb * (kLanes * 128), &tmQ, kb * 64, c.h * a.G, node0, c.b,
                      &q_full[st]);
      }
      __syncwarp();
    };
    if (n > 0) load_q(cur);
    uint32_t edges = 0;
    bool first_prev = false, edge_prev = false;  // of the tile whose output is next
    auto output = [&](int i, int slot, int ph) {  // of tile i
      const int odd = i & 1;
      if (!wait(&full[slot], ph, a.t.err)) return false;
      if (!wait(&p_ready[2 * st + odd], (i >> 1) & 1, a.t.err)) return false;
      if (edge_prev) {  // stream 0's softmax cleans V; the others' products wait for it
        ++edges;
        if (st > 0 &&
            !__all_sync(kAll, wait_count_above(v_clean + (lane & 3), edges - 1, a.t.err))) {
          record_error(a.t.err, kDevErrAttn);
          return false;
        }
      }
      __syncwarp();
      tc_fence_after();
      if (elect_one()) {
        const uint64_t bd = bd_pv + slot * (C::kSlot >> 4);
        const uint32_t pa = tb + kColP + odd * (kKeys / 2);
#pragma unroll
        for (int k = 0; k < kKeys / 16; ++k)  // 16 keys: 8 TMEM columns, 2 KB of V
          umma_f16_ts(tb + kColO, pa + 8 * k, bd + k * (2048 >> 4), id_pv, !first_prev || k > 0);
        umma_commit(&pv_done[2 * st + odd]);
        umma_commit(&empty[slot]);
      }
      __syncwarp();
      return true;
    };
    bool ok = true;
    int i = 0;
    for (int seg = 0; i < n && ok; ++seg) {
      const int tile_lo = cur.tile, tile_hi = min(cur.s.tiles, tile_lo + (n - i));
      const int edge_from = cur.s.len / kKeys;
      // A new head's Q replaces the old one as soon as the last scores with that are
      // done, and comes while the softmax and the output of that tile go on.
      const int k_slot = slot, k_ph = ph;
      advance();
      if (i > 0) {
        ok = wait(&s_read[st], (i - 1) & 1, a.t.err);
        __syncwarp();
        if (ok) load_q(cur);
        ok = ok && output(i - 1, slot, ph);
        advance();
      }
      if (i + tile_hi - tile_lo < n) {  // the next head's Q on its way into L2
        Cursor next = cur;
        next.to(a, tile_hi);
        if (elect_one())
#pragma unroll
          for (int kb = 0; kb < kBlk; ++kb)
            tma_prefetch_4d(&tmQ, kb * 64, next.h * a.G, node0, next.b);
        __syncwarp();
      }
      ok = ok && wait(&q_full[st], seg & 1, a.t.err) && scores(i, k_slot, k_ph);
      ++i;
      first_prev = true;
      edge_prev = tile_lo >= edge_from;
      for (int tile = tile_lo + 1; tile < tile_hi && ok; ++tile, ++i) {
        ok = scores(i, slot, ph);
        advance();
        ok = ok && output(i - 1, slot, ph);
        advance();
        first_prev = false;
        edge_prev = tile >= edge_from;
      }
      cur.to(a, tile_hi);
    }
    if (n > 0 && ok) output(n - 1, slot, ph);
    // Q's last copy has landed, also where a wait ran out before the look at it, and every
    // MMA issued is complete before TMEM is freed
    if (q_loads > 0) mbar_wait(&q_full[st], (q_loads - 1) & 1, a.t.err);
    if (elect_one()) umma_commit(&all_done[st]);
    mbar_wait(&all_done[st], 0, a.t.err);
    __syncwarp();
  } else if (N > 0) {
    // ---- softmax: a thread to a row ----
    const int stream = (tid - kFirst) / kLanes;
    const int quarter = warp & 3;  // the TMEM lanes a warp may read: 32 (warp % 4) ..
    const int row_l = quarter * 32 + lane;
    const uint32_t tbase =
        tmem + stream * C::kStreamCols + (static_cast<uint32_t>(quarter * 32) << 16);
    const uint32_t to = tbase + kColO;
    const int M = a.t.T * a.G;
    const int r0 = (row_tile * NS + stream) * a.stream_rows;
    // (a warp without rows only keeps in step)
    const bool live = quarter * 32 < a.stream_rows && r0 + quarter * 32 < M;
    const int r = row_l < a.stream_rows ? r0 + row_l : M, node = r / a.G;
    const float sl = fmaxf(fabsf(a.scale_log2), 1e-37f);
    const bool negative = a.scale_log2 < 0.f;
    bool ok = true;
    int i = 0;  // tile of this CTA's range
    for (int seg = 0; i < N && ok; ++seg) {
      // this CTA's part [tile_lo, tile_hi) of a row tile
      const Cursor at = cur;
      const Seq s = at.s;
      const int tile_lo = at.tile, tile_hi = min(s.tiles, tile_lo + (N - i));
      const int h = at.h;
      float m = -INFINITY, l = 0.f;

      // One tile.  kEdge: it has nodes, or positions past the end.
      auto tile_step = [&](auto edge_tag, int tile) {
        constexpr bool kEdge = decltype(edge_tag)::value;
        const int p0 = tile * kKeys;
        const int odd = i & 1;
        const uint64_t vis = kEdge && r < M ? seen64(a, at.b, s, node, p0) : 0;
        // (the MMA warp issued tile i - 2's output before these scores, so it is complete
        // too, and its weights' buffer free for tile i's)
        if (!wait(&s_full[stream], odd, a.t.err)) return false;
        __syncwarp();
        tc_fence_after();
        if (!live) {
          if (lane == 0) mbar_arrive(&s_read[stream]);
        } else {
          uint32_t x[64];
          tmem_ld32_issue(tbase, x);
          tmem_ld32_issue(tbase + 32, x + 32);
          tmem_ld32_wait(x);
          tmem_ld32_wait(x + 32);
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&s_read[stream]);
          if (negative)
#pragma unroll
            for (int c = 0; c < 64; ++c) x[c] ^= 0x80000000u;
          if (kEdge) {
#pragma unroll
            for (int c = 0; c < 64; ++c)
              if (!(vis >> c & 1)) x[c] = 0xFF800000u;  // -inf
          }
          float top = r < M ? max64(x) * sl : -INFINITY;  // NaN if a score is
          if (__any_sync(kAll, !(top <= m + kRise))) {  // (m = -inf: anything above)
            if (__any_sync(kAll, top != top)) {
              // the scores of positions without a page, which are NaN, become -inf
              if (*reinterpret_cast<volatile int*>(&hole_tile[i % C::kHoles]) == i) {
                // (out of line, by way of P's columns: in place it slows every tile)
                const uint32_t hole = *reinterpret_cast<volatile uint32_t*>(&holes[i % C::kHoles]);
                if (i > 0 && !wait(&pv_done[2 * stream + (odd ^ 1)], ((i - 1) >> 1) & 1, a.t.err))
                  return false;
                __syncwarp();
                tc_fence_after();
                tmem_st32(tbase + kColP, x);
                tmem_st32(tbase + kColP + 32, x + 32);
                tmem_st_wait();
                top = leave_out<kBlk>(tbase + kColP, hole, a.t.page_shift) * sl;
                if (r >= M) top = -INFINITY;
                tmem_ld32_issue(tbase + kColP, x);
                tmem_ld32_issue(tbase + kColP + 32, x + 32);
                tmem_ld32_wait(x);
                tmem_ld32_wait(x + 32);
              }
            }
            if (tile == tile_lo) {
              m = top == top ? top : 0.f;  // (NaN is in l, and need not rescale every tile)
            } else {
              if (!wait(&pv_done[2 * stream + (odd ^ 1)], ((i - 1) >> 1) & 1, a.t.err))
                return false;
              __syncwarp();
              tc_fence_after();
              const float mn = top > m + kRise ? top : m;
              const float f = mn == -INFINITY ? 1.f : ex2(m - mn);
              l *= f;
              m = mn;
#pragma unroll 1
              for (int c = 0; c < D; c += 32) {
                uint32_t o[32];
                tmem_ld32_issue(to + c, o);
                tmem_ld32_wait(o);
#pragma unroll
                for (int j = 0; j < 32; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * f);
                tmem_st32(to + c, o);
              }
            }
          }
          const float safe = m == -INFINITY ? 0.f : m;
          const float off = kLift<E> - safe;
          const uint64_t sl2 = pack_f32x2(sl, sl), off2 = pack_f32x2(off, off);
          uint64_t sum[2] = {0, 0};
          uint32_t p[32];
#pragma unroll
          for (int c = 0; c < 32; ++c) {
            const uint64_t y2 = fma_f32x2(pack_u32x2(x[2 * c], x[2 * c + 1]), sl2, off2);
            float y, z;
            unpack_f32x2(y2, y, z);
            y = ex2(y);
            z = ex2(z);
            sum[c & 1] = add_f32x2(sum[c & 1], pack_f32x2(y, z));
            p[c] = pack2<E>(y, z);
          }
          float s0, s1;
          unpack_f32x2(add_f32x2(sum[0], sum[1]), s0, s1);
          l += s0 + s1;
          tmem_st32(tbase + kColP + odd * (kKeys / 2), p);
          tmem_st_wait();
        }
        if (kEdge && stream == 0) {
          // V's rows past the end are zeroed and Inf and NaN of nodes set aside
          // (add_unseen): a weight of 0 would not keep them out of the product
          const int sq = seq_v(i), slot = sq % C::kSlots;
          if (!wait(&full[slot], (sq / C::kSlots) & 1, a.t.err)) return false;
          constexpr int kPieces = C::kSlot / 16 / kLanes;
          uint4* v = reinterpret_cast<uint4*>(ring + slot * C::kSlot) + (tid - kFirst);
          uint4 y[kPieces];
#pragma unroll
          for (int z = 0; z < kPieces; ++z) y[z] = v[z * kLanes];
          // (with two branches a piece the 64 trees of 33 nodes took 142.8 us, so 141.0)
          unsigned bad = 0;
#pragma unroll
          for (int z = 0; z < kPieces; ++z) {
            // 512 pieces to a 64-channel block, 8 to a key
            const int pos = p0 + ((tid - kFirst + z * kLanes) & 511) / 8;
            const bool past = pos >= s.len + s.n;
            if (past) v[z * kLanes] = make_uint4(0, 0, 0, 0);
            bad |= static_cast<unsigned>(!past & (pos >= s.len) & not_finite<E>(y[z])) << z;
          }
          if (bad) {
#pragma unroll
            for (int z = 0; z < kPieces; ++z)
              if (bad >> z & 1)
                v[z * kLanes] = make_uint4(finite2<E>(y[z].x), finite2<E>(y[z].y),
                                           finite2<E>(y[z].z), finite2<E>(y[z].w));
            bad_seg[seg % C::kBadSegs] = seg;
          }
          fence_proxy_async_smem();
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&p_ready[2 * stream + odd]);
          if (kEdge && stream == 0 && NS > 1) add_release_cta(v_clean + quarter, 1);
        }
        ++i;
        return true;
      };
      if (a.mask && r < M && tile_hi * kKeys > s.len)  // read at the head's last tiles
        prefetch_l1(a.mask + (static_cast<int64_t>(at.b) * a.t.T + node) * a.W);
      const int plain_hi = max(tile_lo, min(tile_hi, s.len / kKeys));
      int tile = tile_lo;
      for (; tile < plain_hi && ok; ++tile) ok = tile_step(std::false_type{}, tile);
      for (; tile < tile_hi && ok; ++tile) ok = tile_step(std::true_type{}, tile);
      if (!ok) break;

      // ---- the end of this CTA's part of the row tile ----
      cur.to(a, tile_hi);
      if (!wait(&pv_done[2 * stream + ((i - 1) & 1)], ((i - 1) >> 1) & 1, a.t.err)) break;
      __syncwarp();
      tc_fence_after();
      const bool whole = tile_hi == s.tiles && tile_lo == 0;
      const int slot = tile_lo == 0 && !whole && at.u > u0 ? 1 : 0;
      if (!whole && tid == kFirst)
        a.cuts[2 * blockIdx.x + (tile_lo == 0)] =
            make_cut(g, at.u - tile_lo, at.b, h, s);
      if (live) {
        const int head = h * a.G + r - node * a.G;
        const bool bad = *reinterpret_cast<volatile int*>(&bad_seg[seg % C::kBadSegs]) == seg;
        const float inv = l == 0.f ? 0.f : 1.f / l;
        const int64_t part = static_cast<int64_t>(blockIdx.x) * 2 + slot;
        float* part_o = a.part_o + part * (NS * kLanes * D) + part_at<D>(stream, row_l, 0);
        E* out = static_cast<E*>(a.out) + at.b * a.ob + node * a.ot + head * a.oh;
        const bool mine = r < M && node < s.n;
        if (__any_sync(kAll, bad))
          add_unseen<E, D>(a, to, at.b, s, h, mine ? node : -1, tile_lo * kKeys, tile_hi * kKeys);
#pragma unroll 1
        for (int c = 0; c < D; c += 32) {
          uint32_t o[32];
          tmem_ld32_issue(to + c, o);
          tmem_ld32_wait(o);
          if (mine && whole) {
            if (l == 0.f)  // no score above -inf, whatever the values: 0 times Inf is NaN
#pragma unroll
              for (int j = 0; j < 32; ++j) o[j] = 0;
            uint32_t y[16];
#pragma unroll
            for (int j = 0; j < 16; ++j)
              y[j] = pack2<E>(__uint_as_float(o[2 * j]) * inv, __uint_as_float(o[2 * j + 1]) * inv);
            if (a.out32) {
              st_v8(out + c, y);
              st_v8(out + c + 16, y + 8);
            } else {
#pragma unroll
              for (int j = 0; j < 4; ++j)
                *reinterpret_cast<uint4*>(out + c + 8 * j) =
                    make_uint4(y[4 * j], y[4 * j + 1], y[4 * j + 2], y[4 * j + 3]);
            }
          } else if (mine) {
#pragma unroll
            for (int j = 0; j < 4; ++j)
              st_v8(part_o + (c / 8 + j) * kPartStep, o + 8 * j);
          }
          __syncwarp();  // the next load is the whole warp's
        }
        if (mine && !whole)
          a.part_ml[part * a.rows + stream * a.stream_rows + row_l] = make_float2(m, l);
        if (mine && whole && a.lse)
          a.lse[(static_cast<int64_t>(at.b) * a.t.T + node) * (a.H * a.G) + head] =
              (m == -INFINITY ? 0.f : m) * kLn2 + logf(l * kUnlift<E>);
      }
      tc_fence_before();  // O is read before the next row tile's first product
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, NS * C::kStreamCols);
}

__device__ __forceinline__ float4 scaled(float4 x, float f) {
  return make_float4(x.x * f, x.y * f, x.z * f, x.w * f);
}
__device__ __forceinline__ void add_scaled(float4& y, float4 x, float f) {
  y.x = fmaf(x.x, f, y.x);
  y.y = fmaf(x.y, f, y.y);
  y.z = fmaf(x.z, f, y.z);
  y.w = fmaf(x.w, f, y.w);
}

// The parts that the CTAs left of a row tile, added in the order of the keys.  The
// P ranges that have parts of it lend it P block columns of gridDim.y blocks, so the
// more parts there are to add, the more blocks add them.  A warp takes 512 / D rows
// at once, 16 channels a lane, and four parts at once, whose loads are all in flight
// together; with more than four parts, 2, 4 or 8 warps share the rows.  The last B
// block columns zero what lies past a sequence's count.
constexpr int kCombineWarps = 8, kCombineParts = 4;
template <typename E, int D>
__global__ void __launch_bounds__(kCombineWarps * 32)
    combine_kernel(const __grid_constant__ AttnArgs a) {
  constexpr int kLanesRow = D / 16, kRows = 32 / kLanesRow;  // lanes of a row, rows of a warp
  __shared__ float4 y_s[kCombineWarps][4][32];
  __shared__ float2 ml_s[kCombineWarps][kRows];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int Hq = a.H * a.G;
  pdl_wait();
  pdl_launch_dependents();
  const int ctas = a.grid * a.row_tiles;
  if (static_cast<int>(blockIdx.x) >= 2 * ctas) {
    const int b = blockIdx.x - 2 * ctas;
    const int done = load_seq(a, b).n * Hq;
    for (int x = done + blockIdx.y * kCombineWarps + warp; x < a.t.T * Hq;
         x += gridDim.y * kCombineWarps) {
      const int node = x / Hq, head = x - node * Hq;
      uint32_t* out = reinterpret_cast<uint32_t*>(static_cast<E*>(a.out) + b * a.ob + node * a.ot +
                                                  head * a.oh);
#pragma unroll
      for (int i = 0; i < D / 64; ++i) out[lane + 32 * i] = 0;
      if (a.lse && lane == 0)
        a.lse[(static_cast<int64_t>(b) * a.t.T + node) * Hq + head] = -INFINITY;
    }
    return;
  }
  const Cut cut = a.cuts[blockIdx.x];
  if (cut.b < 0) return;
  const int b = cut.b, c0 = cut.c0, c1 = cut.c1_slot >> 1, slot0 = cut.c1_slot & 1;
  const int parts = c1 - c0 + 1;
  const int range = blockIdx.x / 2 / a.row_tiles, row_tile = blockIdx.x / 2 - range * a.row_tiles;
  const int h = cut.h_n >> 10, r0 = row_tile * a.rows;
  const int part_size = (a.rows > a.stream_rows ? 2 : 1) * (kLanes * D);
  const int rows = min(a.rows, (cut.h_n & 1023) * a.G - r0);  // (past the count: zeroed above)
  const int wide = parts <= kCombineParts       ? 1
                   : parts <= 2 * kCombineParts ? 2
                   : parts <= 4 * kCombineParts ? 4
                                                : 8;  // warps that share rows
  const int per_block = kCombineWarps / wide * kRows, part0 = warp % wide;
  const int id = (range - c0) * gridDim.y + blockIdx.y;
  for (int rb = id * per_block; rb < rows; rb += parts * gridDim.y * per_block) {
    const int r = rb + warp / wide * kRows + lane / kLanesRow, j = lane % kLanesRow;
    const int stream = r >= a.stream_rows;
    const int at = part_at<D>(stream, r - stream * a.stream_rows, j / 2) / 4 + j % 2;
    float m = -INFINITY, l = 0.f;
    float4 y[4];  // channels 4 (j + kLanesRow q) .. + 3
#pragma unroll
    for (int q = 0; q < 4; ++q) y[q] = make_float4(0.f, 0.f, 0.f, 0.f);
    if (r < rows)
      for (int c = c0 + part0; c <= c1; c += kCombineParts * wide) {
        float2 ml[kCombineParts];
        float4 o[kCombineParts][4];
#pragma unroll
        for (int z = 0; z < kCombineParts; ++z) {
          const int cz = c + z * wide;
          ml[z] = make_float2(-INFINITY, 0.f);
          if (cz <= c1) {
            const int64_t part = (cz * a.row_tiles + row_tile) * 2 + (cz == c0 ? slot0 : 0);
            ml[z] = a.part_ml[part * a.rows + r];
            const float4* p = reinterpret_cast<const float4*>(a.part_o + part * part_size) + at;
#pragma unroll
            for (int q = 0; q < 4; ++q) o[z][q] = p[q * (kLanesRow / 2 * kPartStep / 4)];
          } else {
#pragma unroll
            for (int q = 0; q < 4; ++q) o[z][q] = make_float4(0.f, 0.f, 0.f, 0.f);
          }
        }
        float mn = m;
#pragma unroll
        for (int z = 0; z < kCombineParts; ++z) mn = fmaxf(mn, ml[z].x);
        const float safe = mn == -INFINITY ? 0.f : mn;
        const float f = ex2(m - safe);
        m = mn;
        l *= f;
#pragma unroll
        for (int q = 0; q < 4; ++q) y[q] = scaled(y[q], f);
#pragma unroll
        for (int z = 0; z < kCombineParts; ++z) {
          const float w = ex2(ml[z].x - safe);
          l += ml[z].y * w;
#pragma unroll
          for (int q = 0; q < 4; ++q) add_scaled(y[q], o[z][q], w);
        }
      }
    if (wide > 1) {
#pragma unroll
      for (int q = 0; q < 4; ++q) y_s[warp][q][lane] = y[q];
      if (j == 0) ml_s[warp][lane / kLanesRow] = make_float2(m, l);
      __syncthreads();
      if (part0 == 0) {
        float mn = m;
        for (int w = warp + 1; w < warp + wide; ++w) mn = fmaxf(mn, ml_s[w][lane / kLanesRow].x);
        const float safe = mn == -INFINITY ? 0.f : mn;
        const float f = ex2(m - safe);
        l *= f;
#pragma unroll
        for (int q = 0; q < 4; ++q) y[q] = scaled(y[q], f);
        for (int w = warp + 1; w < warp + wide; ++w) {
          const float2 ml = ml_s[w][lane / kLanesRow];
          const float g = ex2(ml.x - safe);
          l += ml.y * g;
#pragma unroll
          for (int q = 0; q < 4; ++q) add_scaled(y[q], y_s[w][q][lane], g);
        }
        m = mn;
      }
      __syncthreads();
    }
    if (r < rows && part0 == 0) {
      if (l == 0.f)  // (as in attn_kernel)
#pragma unroll
        for (int q = 0; q < 4; ++q) y[q] = make_float4(0.f, 0.f, 0.f, 0.f);
      const float inv = l == 0.f ? 0.f : 1.f / l;
      const int node = (r0 + r) / a.G, head = h * a.G + (r0 + r) - node * a.G;
      uint2* out = reinterpret_cast<uint2*>(static_cast<E*>(a.out) + b * a.ob + node * a.ot +
                                            head * a.oh) + j;
#pragma unroll
      for (int q = 0; q < 4; ++q)
        out[q * kLanesRow] = make_uint2(pack2<E>(y[q].x * inv, y[q].y * inv),
                                        pack2<E>(y[q].z * inv, y[q].w * inv));
      if (a.lse && j == 0)  // log 0 = -inf: nothing seen
        a.lse[(static_cast<int64_t>(b) * a.t.T + node) * Hq + head] =
            (m == -INFINITY ? 0.f : m) * kLn2 + logf(l * kUnlift<E>);
    }
  }
}

// ---- host -------------------------------------------------------------------------
PFN_cuTensorMapEncodeTiled_v12000 encoder() {
  static std::mutex mu;
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  std::lock_guard<std::mutex> lock(mu);
  if (!fn) {
    cudaDriverEntryPointQueryResult q;
    void* p = nullptr;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                         &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  }
  return fn;
}

// A tensor map of 16-bit elements [n3, n2, n1, D] with element strides, boxes of
// 64 channels x b1 x b2, 128-byte swizzle.  What lies outside is read as zeros, or as NaN:
// so K is, whose page may be none, and the softmax need not look for that in every tile, only
// where a row's maximum is NaN.
bool map_4d(const void* base, bool f16, int D, const int64_t (&n)[3], const int64_t (&stride)[3],
            int b1, int b2, bool nan, CUtensorMap* out) {
  const PFN_cuTensorMapEncodeTiled_v12000 encode = encoder();
  if (!encode) return false;
  cuuint64_t dims[4] = {static_cast<cuuint64_t>(D)}, strides[3];
  for (int i = 0; i < 3; ++i) {
    dims[1 + i] = static_cast<cuuint64_t>(n[i]);
    // (the stride of a dimension of one entry is never used, but has to be one)
    strides[i] = static_cast<cuuint64_t>(n[i] > 1 ? stride[i] : D) * 2;
  }
  const cuuint32_t box[4] = {64, static_cast<cuuint32_t>(b1), static_cast<cuuint32_t>(b2), 1};
  const cuuint32_t one[4] = {1, 1, 1, 1};
  return encode(out, f16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4,
                const_cast<void*>(base), dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
                CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                nan ? CU_TENSOR_MAP_FLOAT_OOB_FILL_NAN_REQUEST_ZERO_FMA
                    : CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// ---- plan ---------------------------------------------------------------------
struct AttnPlan {
  int stream_rows, rows;  // rows of a stream and of a row tile
  int row_tiles, grid;
  size_t o_off, ml_off, cut_off, ws_bytes;
};

// A stream has as many whole nodes as 128 rows hold.  One stream while it is enough
// (or 256 channels leave room for no second one), two above: see the top of this
// file.
AttnPlan attn_plan(int T, int G, int D, int sms) {
  AttnPlan p;
  const int M = T * G;
  p.stream_rows = kLanes / G * G;
  const int streams = M <= p.stream_rows || D == 256 ? 1 : 2;
  p.rows = streams * p.stream_rows;
  p.row_tiles = (M + p.rows - 1) / p.rows;
  p.grid = std::max(1, (streams == 1 && D < 256 ? 2 * sms : sms) / p.row_tiles);
  const size_t ctas = size_t(p.grid) * p.row_tiles;
  const size_t parts = p.grid > 1 ? ctas * 2 : 0;  // one range cuts nothing
  p.o_off = 0;
  p.ml_off = align_up(parts * streams * kLanes * D * sizeof(float), 256);
  p.cut_off = p.ml_off + align_up(parts * p.rows * sizeof(float2), 256);
  p.ws_bytes = p.cut_off + align_up(ctas * 2 * sizeof(Cut), 256) + 256;  // (to align the base)
  return p;
}

template <typename E, int D, int NS>
cudaError_t launch_main(const AttnArgs& a, const CUtensorMap& q, const CUtensorMap& k,
                        const CUtensorMap& v, cudaStream_t s) {
  auto kernel = attn_kernel<E, D, NS>;
  constexpr size_t smem = TcCfg<D, NS>::kSmem;
  static std::atomic<uint64_t> ready{0};  // devices on which the kernel may use that much
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (!(ready.load() >> dev & 1)) {  // (ordinals are below 64: ensured with the device's state)
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(smem));
    if (e != cudaSuccess) return e;
    ready.fetch_or(uint64_t(1) << dev);
  }
  return launch_k(kernel, dim3(a.grid * a.row_tiles), dim3(TcCfg<D, NS>::kThreads), smem, s, true,
                  a, q, k, v);
}

template <typename E, int D>
cudaError_t launch_attn(const AttnArgs& a, const dfl2_cache* c, cudaStream_t s) {
  alignas(64) CUtensorMap tq, tk, tv;
  const bool f16 = std::is_same_v<E, __half>;
  const int64_t qn[3] = {a.H * a.G, a.t.T, a.B}, qs[3] = {a.qh, a.qt, a.qb};
  const int64_t n[3] = {c->page_size, c->kv_heads, c->pages};
  const int64_t st[3] = {c->slot_stride, c->head_stride, c->page_stride};
  const int box = std::min(c->page_size, kKeys);
  if (!map_4d(a.q, f16, D, qn, qs, a.G, a.stream_rows / a.G, false, &tq) ||
      !map_4d(a.k, f16, D, n, st, box, 1, true, &tk) ||
      !map_4d(a.v, f16, D, n, st, box, 1, false, &tv))
    return cudaErrorInvalidValue;
  cudaError_t e;
  if constexpr (D == 256)
    e = launch_main<E, D, 1>(a, tq, tk, tv, s);
  else
    e = a.rows == a.stream_rows ? launch_main<E, D, 1>(a, tq, tk, tv, s)
                                : launch_main<E, D, 2>(a, tq, tk, tv, s);
  if (e != cudaSuccess) return e;
  // (measured: four block rows to 256 rows; sixteen cost a decode step, whose blocks
  // have next to nothing to do, 7 us of 10, one costs 427 rows in 61 nodes 14 of 46)
  const int blocks = std::max(1, std::min(a.rows, a.t.T * a.G) / 64);
  return launch_k(combine_kernel<E, D>, dim3(2 * a.grid * a.row_tiles + a.B, blocks),
                  dim3(kCombineWarps * 32), 0, s, true, a);
}

template <typename E>
cudaError_t launch_attn_d(const AttnArgs& a, const dfl2_cache* c, cudaStream_t s) {
  return c->head_dim == 64    ? launch_attn<E, 64>(a, c, s)
         : c->head_dim == 128 ? launch_attn<E, 128>(a, c, s)
                              : launch_attn<E, 256>(a, c, s);
}

dfl2_status check_shapes(int B, int T, int q_heads, int kv_heads, int head_dim, int dtype) {
  if (B < 1 || T < 1 || q_heads < 1 || kv_heads < 1)
    return report_errorf(DFL2_ERR_INVALID_ARG, "B=%d, T=%d, q_heads=%d, kv_heads=%d must be >= 1",
                         B, T, q_heads, kv_heads);
  if (q_heads % kv_heads)
    return report_errorf(DFL2_ERR_INVALID_ARG, "q_heads=%d is no multiple of kv_heads=%d", q_heads,
                         kv_heads);
  if (B > kMaxBatch || T > kMaxTree || q_heads / kv_heads > kLanes)
    return report_errorf(DFL2_ERR_UNSUPPORTED,
                         "B=%d, T=%d, q_heads/kv_heads=%d: at most %d, %d, %d", B, T,
                         q_heads / kv_heads, kMaxBatch, kMaxTree, kLanes);
  if (head_dim != 64 && head_dim != 128 && head_dim != 256)
    return report_errorf(DFL2_ERR_UNSUPPORTED, "head_dim=%d: 64, 128 or 256", head_dim);
  if (dtype != DFL2_BF16 && dtype != DFL2_F16)
    return report_errorf(DFL2_ERR_UNSUPPORTED, "dtype %d: the attention takes bf16 and fp16",
                         dtype);
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
  return dfl2::attn_plan(T, q_heads / kv_heads, head_dim, dfl2::device_info().sms).ws_bytes;
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
  // a tensor map's strides are positive, under 2^40 bytes and multiples of 16
  const int64_t most = int64_t(1) << 38;
  const int dims[3] = {B, T, q_heads};
  for (int i = 0; i < 3; ++i)
    for (const int64_t st : {q_strides[i], out_strides[i]})
      if (dims[i] > 1 && (st < 1 || st > most || st % 8))
        return dfl2::report_errorf(DFL2_ERR_INVALID_ARG,
                                   "strides of q and out: multiples of 8 from 8 to 2^38");
  const int cdims[3] = {cache->page_size, cache->kv_heads, cache->pages};
  const int64_t cst[3] = {cache->slot_stride, cache->head_stride, cache->page_stride};
  for (int i = 0; i < 3; ++i)
    if (cdims[i] > 1 && (cst[i] < 1 || cst[i] > most))
      return dfl2::report_errorf(DFL2_ERR_UNSUPPORTED,
                                 "the attention needs cache strides of 8 .. 2^38 elements");
  if (!std::isfinite(scale))
    return dfl2::report_errorf(DFL2_ERR_INVALID_ARG, "scale %g must be finite", double(scale));
  DFL2_TRY(dfl2::check_args_device(ptrs, 7));
  DFL2_TRY(dfl2::check_cache_device(cache));
  const int G = q_heads / cache->kv_heads, D = cache->head_dim;
  const dfl2::AttnPlan p = dfl2::attn_plan(T, G, D, dfl2::device_info().sms);
  if (!ws || ws_bytes < p.ws_bytes)
    return dfl2::report_errorf(DFL2_ERR_WORKSPACE, "workspace of %zu bytes < %zu needed",
                               ws ? ws_bytes : size_t(0), p.ws_bytes);
  const dfl2::PtrArg wsp[] = {{ws, "workspace", 16}};
  DFL2_TRY(dfl2::check_args_host(wsp, 1));
  DFL2_TRY(dfl2::check_args_device(wsp, 1));
  uint8_t* w = reinterpret_cast<uint8_t*>(
      dfl2::align_up(reinterpret_cast<uintptr_t>(ws), 256));  // parts are stored 32 bytes at a time
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
  a.out32 = reinterpret_cast<uintptr_t>(out) % 32 == 0;
  for (int i = 0; i < 3; ++i)
    if (dims[i] > 1 && out_strides[i] % 16) a.out32 = false;
  a.part_o = reinterpret_cast<float*>(w + p.o_off);
  a.part_ml = reinterpret_cast<float2*>(w + p.ml_off);
  a.cuts = reinterpret_cast<dfl2::Cut*>(w + p.cut_off);
  a.grid = p.grid;
  a.rows = p.rows;
  a.stream_rows = p.stream_rows;
  a.row_tiles = p.row_tiles;
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e = cache->dtype == DFL2_F16
                            ? dfl2::launch_attn_d<__half>(a, cache, s)
                            : dfl2::launch_attn_d<__nv_bfloat16>(a, cache, s);
  return e == cudaSuccess ? DFL2_OK : dfl2::report_cuda_error(e, "tree attention launch");
}

}  // extern "C"
