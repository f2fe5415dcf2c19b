// The attention weight that cached positions receive (include/dfl2.h, dfl2_cache_weigh):
//   weight_j += sum over kept queries i and heads h of 2^(scale log2 e <q_ih, k_j> - lse_ih log2 e)
//
// The logarithms of the rows' sums are known, so there is no maximum to look for, and the sum
// over queries and heads needs no exchange if a thread owns a key: the product is taken the
// other way round, S^T = K Q^T, 128 keys by the (query, head) columns, so that a key is a
// lane of TMEM, and a thread adds up its key's columns.
//
// Split.  A step is 128 keys of one key head against up to NC columns; the steps of all
// sequences (lengths are on the device) are cut into equal, contiguous ranges, one a CTA.
// A tile of keys whose steps (all heads, all columns) lie in one range is added to the
// weights by it; of one that several ranges share each leaves its part in the workspace,
// and weigh_add_kernel adds the parts in order.  So the result does not depend on timing.
//
// Roles: warp 0 loads K (TMA boxes of one page, 128-byte swizzle); warp 1 issues the MMAs; four
// warps gather the columns' rows of Q, which path may order anyhow, with 16-byte cp.async; and
// two groups of four take turns with the two accumulators.
//
// Bounds.  A step reads 32 KB of K (128 channels): 1400 cycles of an SM's share of HBM.  With
// 128 columns its MMAs take 512 cycles, and its 16,384 exponentials as many.  So HBM bounds
// up to some 300 columns a key head, and beyond that the tensor cores and the exponentials.
#include "tree_attn_kernel.cuh"

namespace dfl2 {
namespace {

constexpr int kTile = 128;   // keys of a tile: lanes of TMEM
constexpr int kInfos = 4;    // steps whose columns' numbers are held

struct alignas(16) WeighCut {  // a tile that range c0 begins and c1 ends; b < 0: none
  int b, tile, c0, c1;
};

struct WeighArgs {
  TableView t;  // count: how many queries were kept
  const void* q;
  int64_t qb, qt, qh;  // element strides
  const float* lse;    // [B][T][H G]
  const int32_t* path; // [B][T] or NULL
  float* weight;
  int first;
  int B, H, G;
  float scale_log2;
  float* parts;        // [grid][2][kTile]
  WeighCut* cuts;      // [grid]
  int grid;
};

template <int D>
struct WeighCfg {
  static constexpr int kCols = D == 256 ? 64 : 128;  // columns of a step
  static constexpr int kSlotK = kTile * D * 2, kSlotQ = kCols * D * 2;
  static constexpr int kSlotsK = D == 64 ? 6 : D == 128 ? 3 : 2;
  static constexpr int kSlotsQ = D == 64 ? 4 : D == 128 ? 3 : 2;
  static constexpr int kBars = 2 * (kSlotsK + kSlotsQ + kInfos + 2 + 2) + 1;
  static constexpr int kThreads = 14 * 32;
  static constexpr size_t kSmem = size_t(kSlotsK) * kSlotK + size_t(kSlotsQ) * kSlotQ +
                                  kInfos * kCols * 8 + 2 * kTile * 4 + kBars * 8 + 8;
  static_assert(kSmem + 1024 <= 232448, "shared memory");
};

struct WSeq {
  int row, len, n, tiles, chunks;
  __device__ __forceinline__ int64_t steps(int H) const {
    return static_cast<int64_t>(tiles) * H * chunks;
  }
};
template <int kCols>
__device__ __forceinline__ WSeq load_wseq(const WeighArgs& a, int b) {
  WSeq s;
  s.len = a.t.length[b];
  s.n = a.t.count_of(b);
  s.row = a.t.seq ? a.t.seq[b] : b;
  // (and the weights of a row hold no more than its entries' positions)
  if (!a.t.in_range(s.row, s.len)) {
    record_error(a.t.err, kDevErrBadIndex);
    s.n = 0;
  }
  const int64_t room = static_cast<int64_t>(a.t.cols) << a.t.page_shift;
  if (s.n > 0 && s.len + s.n > room) {  // positions that can have no page
    record_error(a.t.err, kDevErrBadIndex);
    s.n = 0;
  }
  s.tiles = s.n > 0 ? (s.len + s.n + kTile - 1) / kTile : 0;
  s.chunks = (s.n * a.G + kCols - 1) / kCols;
  return s;
}

template <int kCols>
struct WCursor {
  int b, tile, h, chunk;
  WSeq s;
  __device__ __forceinline__ void next(const WeighArgs& a) {
    if (++chunk < s.chunks) return;
    chunk = 0;
    if (++h < a.H) return;
    h = 0;
    if (++tile < s.tiles) return;
    tile = 0;
    do {
      if (++b >= a.B) return;
      s = load_wseq<kCols>(a, b);
    } while (s.tiles == 0);
  }
};

// Range `cta` [u0, u1) of the steps, and where it begins, by a warp.
template <int kCols>
struct WRange {
  int64_t units, u0, u1;
  int n_cta;
  WCursor<kCols> first;  // if u0 < u1
};
template <int kCols>
__device__ __forceinline__ WRange<kCols> find_wrange(const WeighArgs& a, int cta) {
  const int lane = threadIdx.x & 31;
  WRange<kCols> g;
  WSeq own;
  int64_t sum;
  auto load = [&](int b0) {
    own = b0 + lane < a.B ? load_wseq<kCols>(a, b0 + lane) : WSeq{0, 0, 0, 0, 0};
    sum = own.steps(a.H);
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int64_t y = __shfl_up_sync(kAll, sum, off);
      if (lane >= off) sum += y;
    }
  };
  load(0);
  g.units = __shfl_sync(kAll, sum, 31);
  if (a.B > 32) {
    int64_t x = 0;
    for (int b = lane + 32; b < a.B; b += 32) x += load_wseq<kCols>(a, b).steps(a.H);
#pragma unroll
    for (int off = 16; off; off >>= 1) x += __shfl_xor_sync(kAll, x, off);
    g.units += x;
  }
  g.n_cta = static_cast<int>(min(static_cast<int64_t>(a.grid), g.units));
  g.u0 = g.u1 = 0;
  if (cta >= g.n_cta) return g;
  g.u0 = range_start(g.units, g.n_cta, cta);
  g.u1 = range_start(g.units, g.n_cta, cta + 1);
  int64_t base = 0;
  for (int b0 = 0; b0 < a.B; b0 += 32) {
    if (b0 > 0) load(b0);
    const unsigned hit = __ballot_sync(kAll, g.u0 < base + sum);
    if (hit) {
      const int w = __ffs(hit) - 1;
      const int64_t in = g.u0 - base - __shfl_sync(kAll, sum - own.steps(a.H), w);
      WCursor<kCols>& c = g.first;
      c.b = b0 + w;
      c.s = WSeq{__shfl_sync(kAll, own.row, w), __shfl_sync(kAll, own.len, w),
                 __shfl_sync(kAll, own.n, w), __shfl_sync(kAll, own.tiles, w),
                 __shfl_sync(kAll, own.chunks, w)};
      const int64_t hc = in / c.s.chunks;
      c.chunk = static_cast<int>(in - hc * c.s.chunks);
      c.tile = static_cast<int>(hc / a.H);
      c.h = static_cast<int>(hc - static_cast<int64_t>(c.tile) * a.H);
      return g;
    }
    base += __shfl_sync(kAll, sum, 31);
  }
  g.u1 = g.u0;  // the lengths changed in between
  return g;
}

// What a position received, added to its weight.
__device__ __forceinline__ void put(const WeighArgs& a, const WSeq& s, int pos, float sum) {
  if (pos >= s.len + s.n || a.t.page_at(s.row, pos >> a.t.page_shift) < 0) return;
  float* w = a.weight + (static_cast<int64_t>(s.row) * a.t.cols << a.t.page_shift) + pos;
  *w = (a.first && pos >= s.len ? 0.f : *w) + sum;
}

template <typename E, int D>
__global__ void __launch_bounds__(WeighCfg<D>::kThreads, 1)
    weigh_kernel(const __grid_constant__ WeighArgs a, const __grid_constant__ CUtensorMap tmK) {
  using C = WeighCfg<D>;
  constexpr int kBlk = D / 64, kCols = C::kCols;
  extern __shared__ __align__(1024) uint8_t smem[];
  uint8_t* ks = smem;                             // [slots][kBlk][128 keys][128 B]
  uint8_t* qs = ks + C::kSlotsK * C::kSlotK;      // [slots][kBlk][kCols][128 B]
  float* lse_s = reinterpret_cast<float*>(qs + C::kSlotsQ * C::kSlotQ);  // [kInfos][kCols], negated
  int* pos_s = reinterpret_cast<int*>(lse_s + kInfos * kCols);  // [kInfos][kCols]
  float* acc_s = reinterpret_cast<float*>(pos_s + kInfos * kCols);  // [2][kTile]
  uint64_t* k_full = reinterpret_cast<uint64_t*>(acc_s + 2 * kTile);
  uint64_t* k_empty = k_full + C::kSlotsK;
  uint64_t* q_full = k_empty + C::kSlotsK;
  uint64_t* q_empty = q_full + C::kSlotsQ;
  uint64_t* i_full = q_empty + C::kSlotsQ;   // a step's columns are described
  uint64_t* i_empty = i_full + kInfos;
  uint64_t* s_full = i_empty + kInfos;       // [2] scores are in TMEM
  uint64_t* s_empty = s_full + 2;
  uint64_t* acc_full = s_empty + 2;          // [2] the second group's sums are in place
  uint64_t* acc_empty = acc_full + 2;
  uint64_t* all_done = acc_empty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(all_done + 1);

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid == 0) {
    for (int i = 0; i < C::kSlotsK; ++i) {
      mbar_init(&k_full[i], 1);
      mbar_init(&k_empty[i], 1);
    }
    for (int i = 0; i < C::kSlotsQ; ++i) {
      mbar_init(&q_full[i], 128);
      mbar_init(&q_empty[i], 1);
    }
    for (int i = 0; i < kInfos; ++i) {
      mbar_init(&i_full[i], 4);
      mbar_init(&i_empty[i], 4);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&s_empty[i], 4);
      mbar_init(&acc_full[i], 4);
      mbar_init(&acc_empty[i], 4);
    }
    mbar_init(all_done, 1);
    fence_mbar_init();
    tma_prefetch_desc(&tmK);
  }
  if (warp == 1) tmem_alloc(tmem_slot, 2 * kCols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  pdl_wait();
  pdl_launch_dependents();

  const WRange<kCols> g = find_wrange<kCols>(a, blockIdx.x);
  WCursor<kCols> cur = g.first;
  int64_t N = g.u1 - g.u0;
  if (smem_u32(smem) & 1023u) {  // the swizzle counts on it
    record_error(a.t.err, kDevErrAttn);
    N = 0;
  }

  // A wait that ran out (ok false) is the last one of its warp: what follows is only counted.
  bool ok = true;
  if (warp == 0) {
    // ---- K: a tile of a head at a time ----
    const int ps = 1 << a.t.page_shift, box = min(ps, kTile);
    const int boxes = kTile / box * kBlk;  // at most 64
    int slot = 0, ph = 0, issued = 0, page[2] = {0, 0};
    bool fresh = true;
    for (int64_t i = 0; i < N && ok;) {
      const WSeq s = cur.s;
      if (fresh)
#pragma unroll
        for (int z = 0; z < 2; ++z) {  // this lane's pages of the tile; one too far for none
          const int x = lane + 32 * z, pos = cur.tile * kTile + x / kBlk * box;
          page[z] = a.t.pages;
          if (x < boxes && pos < s.len + s.n) {
            const int p = a.t.page_at(s.row, pos >> a.t.page_shift);
            if (p >= 0) page[z] = p;
          }
        }
      if (issued >= C::kSlotsK) ok = wait(&k_empty[slot], ph ^ 1, a.t.err);
      ok = __all_sync(kAll, ok);
      if (ok) {
        if (lane == 0) mbar_arrive_expect_tx(&k_full[slot], C::kSlotK);
        __syncwarp();
#pragma unroll
        for (int z = 0; z < 2; ++z) {
          const int x = lane + 32 * z;
          if (x < boxes)
            tma_load_4d(ks + slot * C::kSlotK + x % kBlk * (kTile * 128) + x / kBlk * box * 128, &tmK,
                        x % kBlk * 64, cur.tile * kTile & (ps - 1), cur.h, page[z], &k_full[slot]);
        }
        ++issued;
        if (++slot == C::kSlotsK) {
          slot = 0;
          ph ^= 1;
        }
      }
      const int tile = cur.tile, b = cur.b;
      const int64_t here = min(N - i, static_cast<int64_t>(s.chunks - cur.chunk));
      i += here;
      cur.chunk = s.chunks - 1;  // (on to the next head's tile)
      cur.next(a);
      fresh = cur.tile != tile || cur.b != b;
    }
    // the copies still in flight land before the CTA ends
    for (int j = max(0, issued - C::kSlotsK); j < issued; ++j)
      mbar_wait(&k_full[j % C::kSlotsK], (j / C::kSlotsK) & 1, a.t.err);
  } else if (warp == 1) {
    // ---- MMAs (the whole warp walks, one elected lane issues: descriptors stay uniform) ----
    const uint32_t tb = __shfl_sync(kAll, tmem, 0);
    const uint64_t ad = umma_desc_sw128(ks), bd = umma_desc_sw128(qs);
    int k_slot = 0, k_ph = 0, q_slot = 0, q_ph = 0;
    for (int64_t i = 0; i < N && ok; ++i) {
      const int buf = static_cast<int>(i & 1);
      const int cols = min(kCols, cur.s.n * a.G - cur.chunk * kCols);
      if (i == 0 || cur.chunk == 0) ok = wait(&k_full[k_slot], k_ph, a.t.err);
      ok = ok && wait(&q_full[q_slot], q_ph, a.t.err);
      if (i > 1) ok = ok && wait(&s_empty[buf], ((i >> 1) - 1) & 1, a.t.err);
      ok = __all_sync(kAll, ok);
      if (!ok) break;
      tc_fence_after();
      const bool last = cur.chunk == cur.s.chunks - 1 || i == N - 1;
      if (elect_one()) {
        const uint32_t id = idesc_f16<E>(kTile, (cols + 15) & ~15, false);
        const uint64_t ak = ad + k_slot * (C::kSlotK >> 4), bq = bd + q_slot * (C::kSlotQ >> 4);
#pragma unroll
        for (int kb = 0; kb < kBlk; ++kb)
#pragma unroll
          for (int k = 0; k < 4; ++k)
            umma_bf16(tb + buf * kCols, ak + kb * (kTile * 128 >> 4) + 2 * k,
                      bq + kb * (kCols * 128 >> 4) + 2 * k, id, kb > 0 || k > 0);
        umma_commit(&s_full[buf]);
        umma_commit(&q_empty[q_slot]);
        if (last) umma_commit(&k_empty[k_slot]);
      }
      __syncwarp();
      if (++q_slot == C::kSlotsQ) {
        q_slot = 0;
        q_ph ^= 1;
      }
      if (last && ++k_slot == C::kSlotsK) {
        k_slot = 0;
        k_ph ^= 1;
      }
      cur.next(a);
    }
    if (elect_one()) umma_commit(all_done);  // every MMA complete before TMEM is freed
    mbar_wait(all_done, 0, a.t.err);
    __syncwarp();
  } else if (warp < 6) {
    // ---- Q: a warp a quarter of the columns, a lane to a column's numbers ----
    const int w = warp - 2;
    constexpr int kMine = kCols / 4, kPieces = D / 8;  // columns of a warp, 16-byte pieces
    int slot = 0, ph = 0, before = 0;
    int64_t i = 0;
    for (; i < N && ok; ++i) {
      const WSeq s = cur.s;
      const int info = static_cast<int>(i & (kInfos - 1));
      const int col = cur.chunk * kCols + w * kMine + lane;  // (of kMine lanes)
      int64_t from = -1;
      float l = 0.f;
      int pos = INT32_MIN;  // seen by no key
      if (lane < kMine && col < s.n * a.G) {
        const int x = col / a.G, head = cur.h * a.G + col - x * a.G;
        const int node = a.path ? a.path[static_cast<int64_t>(cur.b) * a.t.T + x] : x;
        if (static_cast<unsigned>(node) < static_cast<unsigned>(a.t.T)) {
          l = a.lse[(static_cast<int64_t>(cur.b) * a.t.T + node) * (a.H * a.G) + head];
          if (isfinite(l)) pos = x;
          from = cur.b * a.qb + node * a.qt + head * a.qh;
        } else {
          record_error(a.t.err, kDevErrBadIndex);
        }
      }
      if (i >= kInfos) ok = wait(&i_empty[info], ((i / kInfos) - 1) & 1, a.t.err);
      if (i >= C::kSlotsQ) ok = ok && wait(&q_empty[slot], ph ^ 1, a.t.err);
      ok = __all_sync(kAll, ok);
      if (!ok) break;
      if (lane < kMine) {
        lse_s[info * kCols + w * kMine + lane] = -l * kLog2e;
        pos_s[info * kCols + w * kMine + lane] = pos;
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&i_full[info]);
      // 32 / kPieces columns at a time
      uint8_t* dst = qs + slot * C::kSlotQ;
      const int mine = min(kMine, s.n * a.G - cur.chunk * kCols - w * kMine);
#pragma unroll 4
      for (int z = 0; z < mine * kPieces; z += 32) {
        const int c = (z + lane) / kPieces, p = (z + lane) % kPieces, at = w * kMine + c;
        const int64_t f = __shfl_sync(kAll, from, c & 31);
        if (c < mine)
          cp_async16(dst + (p >> 3) * (kCols * 128) + at * 128 + (((p & 7) ^ (at & 7)) << 4),
                     static_cast<const E*>(a.q) + (f < 0 ? 0 : f) + p * 8, f >= 0);
      }
      cp_async_commit();
      if (i > 0) {
        cp_async_wait<1>();
        fence_proxy_async_smem();
        mbar_arrive(&q_full[before]);
      }
      before = slot;
      if (++slot == C::kSlotsQ) {
        slot = 0;
        ph ^= 1;
      }
      cur.next(a);
    }
    cp_async_wait<0>();
    fence_proxy_async_smem();
    if (i > 0) mbar_arrive(&q_full[before]);
  } else {
    // ---- sums: a thread to a key, two groups by turns ----
    const int group = (warp - 6) >> 2, quarter = warp & 3, key = quarter * 32 + lane;
    const uint32_t tbase =
        tmem + group * kCols + (static_cast<uint32_t>(quarter * 32) << 16);
    const uint64_t sl2 = pack_f32x2(a.scale_log2, a.scale_log2);
    if (group == 0 && key == 0) a.cuts[blockIdx.x].b = -1;
    int seg = 0;
    for (int64_t i = 0; i < N && ok; ++seg) {
      // this CTA's steps of a tile
      const WSeq s = cur.s;
      const int b = cur.b, tile = cur.tile;
      const int per = a.H * s.chunks, at0 = cur.h * s.chunks + cur.chunk;
      const int64_t i1 = min(N, i + per - at0);
      const int64_t v0 = g.u0 + i - at0;  // the tile's first step
      const int rel = tile * kTile + key - s.len;  // < 0: committed
      const bool plain = (tile + 1) * kTile <= s.len;
      uint64_t sum[2] = {0, 0};
      float more = 0.f;
      int chunk = cur.chunk;
      for (; i < i1; ++i) {
        if ((i & 1) == group && ok) {
          const int info = static_cast<int>(i & (kInfos - 1));
          const int cols = min(kCols, s.n * a.G - chunk * kCols);
          ok = wait(&i_full[info], (i / kInfos) & 1, a.t.err) &&
               wait(&s_full[group], (i >> 1) & 1, a.t.err);
          ok = __all_sync(kAll, ok);
          if (ok) {
            tc_fence_after();
            const float* l = lse_s + info * kCols;
            const int* p = pos_s + info * kCols;
#pragma unroll 1
            for (int c = 0; c < cols; c += 32) {
              uint32_t x[32];
              tmem_ld32_issue(tbase + c, x);
              // (a column that is left out, or past the last, is seen by no key)
              const bool whole = plain && __all_sync(kAll, p[c + lane] >= 0);
              tmem_ld32_wait(x);
              if (whole) {
#pragma unroll
                for (int j = 0; j < 32; j += 4) {
                  const float4 y = *reinterpret_cast<const float4*>(l + c + j);
                  float e0, e1, e2, e3;
                  unpack_f32x2(fma_f32x2(pack_u32x2(x[j], x[j + 1]), sl2, pack_f32x2(y.x, y.y)), e0,
                               e1);
                  unpack_f32x2(fma_f32x2(pack_u32x2(x[j + 2], x[j + 3]), sl2, pack_f32x2(y.z, y.w)),
                               e2, e3);
                  sum[0] = add_f32x2(sum[0], pack_f32x2(ex2(e0), ex2(e1)));
                  sum[1] = add_f32x2(sum[1], pack_f32x2(ex2(e2), ex2(e3)));
                }
              } else {
#pragma unroll
                for (int j = 0; j < 32; ++j) {
                  const float e = ex2(fmaf(__uint_as_float(x[j]), a.scale_log2, l[c + j]));
                  if (rel <= p[c + j]) more += e;
                }
              }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
              mbar_arrive(&s_empty[group]);
              mbar_arrive(&i_empty[info]);
            }
          }
        }
        if (++chunk == s.chunks) chunk = 0;
      }
      // ---- the end of this CTA's part of the tile ----
      float s0, s1;
      unpack_f32x2(add_f32x2(sum[0], sum[1]), s0, s1);
      float all = (s0 + s1) + more;
      const int half = seg & 1;
      if (group == 1) {
        if (seg > 1 && ok) ok = wait(&acc_empty[half], ((seg >> 1) - 1) & 1, a.t.err);
        ok = __all_sync(kAll, ok);
        if (ok) {
          acc_s[half * kTile + key] = all;
          __syncwarp();
          if (lane == 0) mbar_arrive(&acc_full[half]);
        }
      } else {
        if (ok) ok = wait(&acc_full[half], (seg >> 1) & 1, a.t.err);
        ok = __all_sync(kAll, ok);
        if (ok) {
          all += acc_s[half * kTile + key];
          __syncwarp();
          if (lane == 0) mbar_arrive(&acc_empty[half]);
          const bool begins = at0 == 0, ends = g.u0 + i == v0 + per;
          if (begins && ends) {
            put(a, s, tile * kTile + key, all);
          } else {
            a.parts[(static_cast<int64_t>(blockIdx.x) * 2 + (begins ? 1 : 0)) * kTile + key] = all;
            if (begins && key == 0)
              a.cuts[blockIdx.x] = WeighCut{b, tile, static_cast<int>(blockIdx.x),
                                            range_of(g.units, g.n_cta, v0 + per - 1)};
          }
        }
      }
      cur.h = a.H - 1;  // on to the next tile
      cur.chunk = s.chunks - 1;
      cur.next(a);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, 2 * kCols);
}

// The parts of the tiles that several ranges share, in order.
template <int kCols>
__global__ void __launch_bounds__(kTile) weigh_add_kernel(const __grid_constant__ WeighArgs a) {
  pdl_wait();
  pdl_launch_dependents();
  const WeighCut cut = a.cuts[blockIdx.x];
  if (cut.b < 0) return;
  const int key = threadIdx.x;
  const WSeq s = load_wseq<kCols>(a, cut.b);
  float sum = a.parts[(static_cast<int64_t>(cut.c0) * 2 + 1) * kTile + key];
#pragma unroll 8
  for (int c = cut.c0 + 1; c <= cut.c1; ++c)
    sum += a.parts[static_cast<int64_t>(c) * 2 * kTile + key];
  put(a, s, cut.tile * kTile + key, sum);
}

struct WeighPlan {
  int grid;
  size_t cut_off, ws_bytes;
};
WeighPlan weigh_plan() {
  WeighPlan p;
  p.grid = device_info().sms;
  p.cut_off = align_up(size_t(p.grid) * 2 * kTile * sizeof(float), 256);
  p.ws_bytes = p.cut_off + p.grid * sizeof(WeighCut) + 256;  // (to align the base)
  return p;
}

template <typename E, int D>
cudaError_t launch_weigh(const WeighArgs& a, const dfl2_cache* c, const void* k, cudaStream_t s) {
  alignas(64) CUtensorMap tk;
  const int64_t n[3] = {c->page_size, c->kv_heads, c->pages};
  const int64_t st[3] = {c->slot_stride, c->head_stride, c->page_stride};
  if (!map_4d(k, std::is_same_v<E, __half>, D, n, st, std::min(c->page_size, kTile), 1, false, &tk))
    return cudaErrorInvalidValue;
  auto kernel = weigh_kernel<E, D>;
  using C = WeighCfg<D>;
  static std::atomic<uint64_t> ready{0};  // devices on which the kernel may use that much
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (!(ready.load() >> dev & 1)) {
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(C::kSmem));
    if (e != cudaSuccess) return e;
    ready.fetch_or(uint64_t(1) << dev);
  }
  e = launch_k(kernel, dim3(a.grid), dim3(C::kThreads), C::kSmem, s, true, a, tk);
  if (e != cudaSuccess) return e;
  return launch_k(weigh_add_kernel<C::kCols>, dim3(a.grid), dim3(kTile), 0, s, true, a);
}
template <typename E>
cudaError_t launch_weigh_d(const WeighArgs& a, const dfl2_cache* c, const void* k, cudaStream_t s) {
  return c->head_dim == 64    ? launch_weigh<E, 64>(a, c, k, s)
         : c->head_dim == 128 ? launch_weigh<E, 128>(a, c, k, s)
                              : launch_weigh<E, 256>(a, c, k, s);
}

}  // namespace
}  // namespace dfl2

#define DFL2_TRY(expr)              \
  do {                              \
    dfl2_status _st = (expr);       \
    if (_st != DFL2_OK) return _st; \
  } while (0)

extern "C" {

size_t dfl2_cache_weigh_workspace_size(void) {
  if (dfl2::check_args_device(nullptr, 0) != DFL2_OK) return 0;
  return dfl2::weigh_plan().ws_bytes;
}

dfl2_status dfl2_cache_weigh(const void* q, const int64_t* q_strides, const float* lse,
                             const dfl2_cache* cache, int layer, int B, int T, int q_heads,
                             const int32_t* table_rows, const int32_t* length, const int32_t* path,
                             const int32_t* n_path, float scale, int first, float* weight, void* ws,
                             size_t ws_bytes, dfl2_stream stream) {
  const dfl2::PtrArg ptrs[] = {{q, "q", 16}, {lse, "lse", 4}, {table_rows, "table_rows", 4, true},
                               {length, "length", 4}, {path, "path", 4, true},
                               {n_path, "n_path", 4, true}, {weight, "weight", 4}};
  DFL2_TRY(dfl2::check_cache_host(cache));
  DFL2_TRY(dfl2::check_attn_shapes(B, T, q_heads, cache->kv_heads, cache->head_dim, cache->dtype));
  DFL2_TRY(dfl2::check_args_host(ptrs, 7));
  if (layer < 0 || layer >= cache->layers)
    return dfl2::report_errorf(DFL2_ERR_INVALID_ARG, "layer %d of %d", layer, cache->layers);
  if (!q_strides) return dfl2::report_errorf(DFL2_ERR_INVALID_ARG, "q_strides is needed");
  const int dims[3] = {B, T, q_heads};
  for (int i = 0; i < 3; ++i)
    if (dims[i] > 1 && (q_strides[i] < 0 || q_strides[i] % 8))
      return dfl2::report_errorf(DFL2_ERR_INVALID_ARG,
                                 "strides of q: non-negative multiples of 8");
  const int64_t most = int64_t(1) << 38;  // a tensor map's strides are positive, under 2^40 bytes
  const int cdims[3] = {cache->page_size, cache->kv_heads, cache->pages};
  const int64_t cst[3] = {cache->slot_stride, cache->head_stride, cache->page_stride};
  for (int i = 0; i < 3; ++i)
    if (cdims[i] > 1 && (cst[i] < 1 || cst[i] > most))
      return dfl2::report_errorf(DFL2_ERR_UNSUPPORTED, "cache strides of 8 .. 2^38 elements");
  if (!std::isfinite(scale))
    return dfl2::report_errorf(DFL2_ERR_INVALID_ARG, "scale %g must be finite", double(scale));
  DFL2_TRY(dfl2::check_args_device(ptrs, 7));
  DFL2_TRY(dfl2::check_cache_device(cache));
  const dfl2::WeighPlan p = dfl2::weigh_plan();
  if (!ws || ws_bytes < p.ws_bytes)
    return dfl2::report_errorf(DFL2_ERR_WORKSPACE, "workspace of %zu bytes < %zu needed",
                               ws ? ws_bytes : size_t(0), p.ws_bytes);
  const dfl2::PtrArg wsp[] = {{ws, "workspace", 1}};
  DFL2_TRY(dfl2::check_args_device(wsp, 1));
  uint8_t* w = reinterpret_cast<uint8_t*>(dfl2::align_up(reinterpret_cast<uintptr_t>(ws), 256));
  dfl2::WeighArgs a{};
  a.t = dfl2::table_view(cache, table_rows, length, n_path, T);
  a.q = q;
  a.qb = q_strides[0];
  a.qt = q_strides[1];
  a.qh = q_strides[2];
  a.lse = lse;
  a.path = path;
  a.weight = weight;
  a.first = first != 0;
  a.B = B;
  a.H = cache->kv_heads;
  a.G = q_heads / cache->kv_heads;
  a.scale_log2 = scale * dfl2::kLog2e;
  a.parts = reinterpret_cast<float*>(w);
  a.cuts = reinterpret_cast<dfl2::WeighCut*>(w + p.cut_off);
  a.grid = p.grid;
  const void* k = static_cast<const uint8_t*>(cache->k) + layer * cache->layer_stride * 2;
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e = cache->dtype == DFL2_F16
                            ? dfl2::launch_weigh_d<__half>(a, cache, k, s)
                            : dfl2::launch_weigh_d<__nv_bfloat16>(a, cache, k, s);
  return e == cudaSuccess ? DFL2_OK : dfl2::report_cuda_error(e, "cache weigh launch");
}

}  // extern "C"
