// The attention weight that cached positions receive (include/dfl2.h, dfl2_cache_weigh):
//   weight_j += sum over kept queries i and heads h of 2^(scale log2 e <q_ih, k_j> - lse_ih log2 e)
//
// The logarithms of the rows' sums are known, so there is no maximum to look for, and the sum
// over queries and heads needs no exchange if a thread owns a key: the product is taken the
// other way round, S^T = K Q^T, 128 keys by the (query, head) columns, so that a key is a
// lane of TMEM, and a thread adds up its key's columns.
//
// Split.  A step is a group of up to kt tiles of 128 keys of one key head against up to
// kCols columns; the steps of all sequences (lengths are on the device) are cut into equal,
// contiguous ranges, one a CTA.  A group whose steps (all heads, all columns) lie in one range
// is added to the weights by it; of one that several ranges share each leaves its part in
// the workspace, and weigh_add_kernel adds the parts in order.  So the result does not depend
// on timing.  A group's tiles stay in shared memory while all columns pass by: an SM takes in
// about 26 bytes a cycle from L2, and with the 32 KB of 128 columns (128 channels) brought
// again for every 128 keys the gather of Q bounded everything (2700 cycles a tile).  kt is the
// largest of 4, 2 and 1 that leaves every CTA four steps.  Measured with two, four, eight and
// sixteen: 8 sequences of 2500 positions, four kept tokens, 17.9, 16.6, 19.3, 19.4 us; 12 of them
// 21.0, 20.0, 23.9, 23.9; 24 31.3, 31.1, 30.2, 38.4; a chunk of 256 tokens, 7 heads a key head,
// at 3000 positions 18.7, 19.3, 26.2, 26.3, at 12,000 35.4, 35.4, 35.4, 45.6.
//
// Roles: warp 0 loads K (TMA boxes of one page, 128-byte swizzle); warp 1 issues the MMAs; four
// warps gather the columns' rows of Q, which path may order anyhow, with 16-byte cp.async; and
// four warps for each tile of a group add up (a warp's 128 columns take 2,000 cycles, most of
// them latency, so a scheduler wants four of them).  Four accumulators take turns, so MMAs,
// exponentials and gather overlap.
//
// Bounds.  A tile of K is 32 KB (128 channels): 1400 cycles of an SM's share of HBM.  With
// 128 columns its MMAs take 512 cycles, and its 16,384 exponentials as many.  So HBM bounds
// up to some 300 columns a key head, and beyond that the tensor cores and the exponentials.
// Measured: 64 sequences of 900 to 4100 positions, 8 key heads, one to 15 kept tokens: 62 us,
// 76% of measured HBM.  A chunk of 256 tokens, 7 heads a key head, behind 3000 to 12,345
// positions, 4 sequences: 71 us, 43% of the tensor cores' rate: a step of four tiles takes 4900
// cycles, 640 for each tile's MMAs and 3300 for its sums, which the next step's MMAs into the
// same accumulator wait for.
#include "tree_attn_kernel.cuh"

namespace dfl2 {
namespace {

constexpr int kTile = 128;   // keys of a tile: lanes of TMEM
constexpr int kInfos = 4;    // steps whose columns' numbers are held
constexpr int kAccs = 4;     // accumulators
constexpr int kMaxGroup = 4; // tiles of a group

struct alignas(32) WeighCut {  // a group that range c0 begins and c1 ends; b < 0: none
  int b, c0, c1;
  int pos;       // the group's first position
  int row, len, n;
  int keys;      // positions of the group
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
  float* parts;        // [grid][2][kMaxGroup][kTile]
  WeighCut* cuts;      // [grid]
  int grid;
};

template <int D>
struct WeighCfg {
  static constexpr int kCols = D == 256 ? 64 : 128;  // columns of a step
  static constexpr int kSlotK = kTile * D * 2, kSlotQ = kCols * D * 2;
  static constexpr int kSlotsK = D == 64 ? 8 : D == 128 ? 4 : 2;
  static constexpr int kSlotsQ = D == 64 ? 4 : 2;
  static constexpr int kGroup = kSlotsK < kMaxGroup ? kSlotsK : kMaxGroup;  // most tiles of a group
  static constexpr int kBars = 2 * (kSlotsK + kSlotsQ + kInfos + kAccs) + 1;
  static constexpr int kThreads = (6 + 4 * kMaxGroup) * 32;
  static constexpr size_t kSmem = size_t(kSlotsK) * kSlotK + size_t(kSlotsQ) * kSlotQ +
                                  kInfos * kCols * 8 + kCols * 8 + kBars * 8 + 8;
  static_assert(kSmem + 1024 <= 232448, "shared memory");
};

struct WSeq {
  int row, len, n, tiles, chunks;
  __device__ __forceinline__ int groups(int kt) const { return (tiles + kt - 1) / kt; }
  __device__ __forceinline__ int64_t steps(int H, int kt) const {
    return static_cast<int64_t>(groups(kt)) * H * chunks;
  }
};
template <int kCols>
__device__ __forceinline__ WSeq load_wseq(const WeighArgs& a, int b) {
  WSeq s;
  s.len = a.t.length[b];
  s.n = a.t.count_of(b);
  s.row = a.t.seq ? a.t.seq[b] : b;
  const int64_t room = static_cast<int64_t>(a.t.cols) << a.t.page_shift;
  // (the weights of a row hold no more than its entries' positions)
  if (!a.t.in_range(s.row, s.len) || (s.n > 0 && s.len + s.n > room)) {
    record_error(a.t.err, kDevErrBadIndex);
    s.n = 0;
  }
  s.tiles = s.n > 0 ? (s.len + s.n + kTile - 1) / kTile : 0;
  s.chunks = (s.n * a.G + kCols - 1) / kCols;
  return s;
}

template <int kCols>
struct WCursor {
  int b, group, h, chunk;
  WSeq s;
  __device__ __forceinline__ void next(const WeighArgs& a, int kt) {
    if (++chunk < s.chunks) return;
    chunk = 0;
    if (++h < a.H) return;
    h = 0;
    if (++group < s.groups(kt)) return;
    group = 0;
    do {
      if (++b >= a.B) return;
      s = load_wseq<kCols>(a, b);
    } while (s.tiles == 0);
  }
  // Tiles of this group.
  __device__ __forceinline__ int here(int kt) const { return min(kt, s.tiles - group * kt); }
};

// Range `cta` [u0, u1) of the steps, and where it begins, by a warp.
template <int kCols>
struct WRange {
  int64_t units, u0, u1;
  int n_cta, kt;
  WCursor<kCols> first;  // if u0 < u1
};
template <int kCols, int kGroup>
__device__ __forceinline__ WRange<kCols> find_wrange(const WeighArgs& a, int cta) {
  const int lane = threadIdx.x & 31;
  WRange<kCols> g;
  // each lane's sequences' steps for groups of 4, 2 and 1
  WSeq own = lane < a.B ? load_wseq<kCols>(a, lane) : WSeq{0, 0, 0, 0, 0};
  int64_t x[3] = {own.steps(a.H, 4), own.steps(a.H, 2), own.steps(a.H, 1)};
  for (int b = lane + 32; b < a.B; b += 32) {
    const WSeq s = load_wseq<kCols>(a, b);
    x[0] += s.steps(a.H, 4);
    x[1] += s.steps(a.H, 2);
    x[2] += s.steps(a.H, 1);
  }
#pragma unroll
  for (int off = 16; off; off >>= 1)
#pragma unroll
    for (int z = 0; z < 3; ++z) x[z] += __shfl_xor_sync(kAll, x[z], off);
  const int64_t enough = 4ll * a.grid;
  const int pick = kGroup >= 4 && x[0] >= enough ? 0 : x[1] >= enough ? 1 : 2;
  g.kt = 4 >> pick;
  g.units = x[pick];
  g.n_cta = static_cast<int>(min(static_cast<int64_t>(a.grid), g.units));
  g.u0 = g.u1 = 0;
  if (cta >= g.n_cta) return g;
  g.u0 = range_start(g.units, g.n_cta, cta);
  g.u1 = range_start(g.units, g.n_cta, cta + 1);
  int64_t base = 0;
  for (int b0 = 0; b0 < a.B; b0 += 32) {
    if (b0 > 0) own = b0 + lane < a.B ? load_wseq<kCols>(a, b0 + lane) : WSeq{0, 0, 0, 0, 0};
    const int64_t mine = own.steps(a.H, g.kt);
    int64_t sum = mine;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int64_t y = __shfl_up_sync(kAll, sum, off);
      if (lane >= off) sum += y;
    }
    const unsigned hit = __ballot_sync(kAll, g.u0 < base + sum);
    if (hit) {
      const int w = __ffs(hit) - 1;
      const int64_t in = g.u0 - base - __shfl_sync(kAll, sum - mine, w);
      WCursor<kCols>& c = g.first;
      c.b = b0 + w;
      c.s = WSeq{__shfl_sync(kAll, own.row, w), __shfl_sync(kAll, own.len, w),
                 __shfl_sync(kAll, own.n, w), __shfl_sync(kAll, own.tiles, w),
                 __shfl_sync(kAll, own.chunks, w)};
      const int64_t hc = in / c.s.chunks;
      c.chunk = static_cast<int>(in - hc * c.s.chunks);
      c.group = static_cast<int>(hc / a.H);
      c.h = static_cast<int>(hc - static_cast<int64_t>(c.group) * a.H);
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
  int64_t* from_s = reinterpret_cast<int64_t*>(qs + C::kSlotsQ * C::kSlotQ);  // [kCols] rows of Q
  float* lse_s = reinterpret_cast<float*>(from_s + kCols);      // [kInfos][kCols], negated
  int* pos_s = reinterpret_cast<int*>(lse_s + kInfos * kCols);  // [kInfos][kCols]
  uint64_t* k_full = reinterpret_cast<uint64_t*>(pos_s + kInfos * kCols);
  uint64_t* k_empty = k_full + C::kSlotsK;
  uint64_t* q_full = k_empty + C::kSlotsK;
  uint64_t* q_empty = q_full + C::kSlotsQ;
  uint64_t* i_full = q_empty + C::kSlotsQ;   // a step's columns are described
  uint64_t* i_empty = i_full + kInfos;
  uint64_t* s_full = i_empty + kInfos;       // [kAccs] scores are in TMEM
  uint64_t* s_empty = s_full + kAccs;
  uint64_t* all_done = s_empty + kAccs;
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
      mbar_init(&i_empty[i], 4 * kMaxGroup);
    }
    for (int i = 0; i < kAccs; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&s_empty[i], 4);
    }
    mbar_init(all_done, 1);
    fence_mbar_init();
    tma_prefetch_desc(&tmK);
  }
  if (warp == 1) tmem_alloc(tmem_slot, kAccs * kCols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  pdl_wait();
  pdl_launch_dependents();

  const WRange<kCols> g = find_wrange<kCols, C::kGroup>(a, blockIdx.x);
  const int kt = g.kt;
  WCursor<kCols> cur = g.first;
  int64_t N = g.u1 - g.u0;
  if (smem_u32(smem) & 1023u) {  // the swizzle counts on it
    record_error(a.t.err, kDevErrAttn);
    N = 0;
  }

  // A wait that ran out (ok false) is the last one of its warp: what follows is only counted.
  bool ok = true;
  if (warp == 0) {
    // ---- K: the tiles of a group, a head at a time ----
    const int ps = 1 << a.t.page_shift, box = min(ps, kTile);
    const int boxes = kTile / box * kBlk;  // at most 64
    int slot = 0, ph = 0, issued = 0;
    for (int64_t i = 0; i < N && ok;) {
      const WSeq s = cur.s;
      const int here = cur.here(kt);
#pragma unroll 1
      for (int t = 0; t < here && ok; ++t) {
        const int tile = cur.group * kt + t;
        int page[2];
#pragma unroll
        for (int z = 0; z < 2; ++z) {  // this lane's pages of the tile; one too far for none
          const int x = lane + 32 * z, pos = tile * kTile + x / kBlk * box;
          page[z] = a.t.pages;
          if (x < boxes && pos < s.len + s.n) {
            const int p = a.t.page_at(s.row, pos >> a.t.page_shift);
            if (p >= 0) page[z] = p;
          }
        }
        if (issued >= C::kSlotsK) ok = wait(&k_empty[slot], ph ^ 1, a.t.err);
        ok = __all_sync(kAll, ok);
        if (!ok) break;
        if (lane == 0) mbar_arrive_expect_tx(&k_full[slot], C::kSlotK);
        __syncwarp();
#pragma unroll
        for (int z = 0; z < 2; ++z) {
          const int x = lane + 32 * z;
          if (x < boxes)
            tma_load_4d(ks + slot * C::kSlotK + x % kBlk * (kTile * 128) + x / kBlk * box * 128, &tmK,
                        x % kBlk * 64, tile * kTile & (ps - 1), cur.h, page[z], &k_full[slot]);
        }
        ++issued;
        if (++slot == C::kSlotsK) {
          slot = 0;
          ph ^= 1;
        }
      }
      i += min(N - i, static_cast<int64_t>(s.chunks - cur.chunk));
      cur.chunk = s.chunks - 1;  // (on to the next head's tiles)
      cur.next(a, kt);
    }
    // the copies still in flight land before the CTA ends
    for (int j = max(0, issued - C::kSlotsK); j < issued; ++j)
      mbar_wait(&k_full[j % C::kSlotsK], (j / C::kSlotsK) & 1, a.t.err);
  } else if (warp == 1) {
    // ---- MMAs (the whole warp walks, one elected lane issues: descriptors stay uniform) ----
    const uint32_t tb = __shfl_sync(kAll, tmem, 0);
    const uint64_t ad = umma_desc_sw128(ks), bd = umma_desc_sw128(qs);
    int k_slot = 0, k_ph = 0, q_slot = 0, q_ph = 0;  // (of a group's first tile)
    uint32_t m = 0;  // rounds so far: kt a step, so that an accumulator is always the same warps'
    for (int64_t i = 0; i < N && ok; ++i) {
      const int cols = min(kCols, cur.s.n * a.G - cur.chunk * kCols);
      const int here = cur.here(kt);
      const bool fresh = i == 0 || cur.chunk == 0;
      const bool last = cur.chunk == cur.s.chunks - 1 || i == N - 1;
      const uint32_t id = idesc_f16<E>(kTile, (cols + 15) & ~15, false);
      const uint64_t bq = bd + q_slot * (C::kSlotQ >> 4);
      ok = wait(&q_full[q_slot], q_ph, a.t.err);
      int slot = k_slot, ph = k_ph;
#pragma unroll 1
      for (int t = 0; t < kt && ok; ++t, ++m) {
        const uint32_t acc = m % kAccs;
        if (fresh && t < here) ok = wait(&k_full[slot], ph, a.t.err);
        if (m >= kAccs) ok = ok && wait(&s_empty[acc], (m / kAccs - 1) & 1, a.t.err);
        ok = __all_sync(kAll, ok);
        if (!ok) break;
        tc_fence_after();
        if (elect_one()) {
          if (t < here) {
            const uint64_t ak = ad + slot * (C::kSlotK >> 4);
#pragma unroll
            for (int kb = 0; kb < kBlk; ++kb)
#pragma unroll
              for (int k = 0; k < 4; ++k)
                umma_bf16(tb + acc * kCols, ak + kb * (kTile * 128 >> 4) + 2 * k,
                          bq + kb * (kCols * 128 >> 4) + 2 * k, id, kb > 0 || k > 0);
          }
          umma_commit(&s_full[acc]);
          if (t == here - 1) umma_commit(&q_empty[q_slot]);
          if (last && t < here) umma_commit(&k_empty[slot]);
        }
        __syncwarp();
        if (t < here && ++slot == C::kSlotsK) {
          slot = 0;
          ph ^= 1;
        }
      }
      if (last) {
        k_slot = slot;
        k_ph = ph;
      }
      if (++q_slot == C::kSlotsQ) {
        q_slot = 0;
        q_ph ^= 1;
      }
      cur.next(a, kt);
    }
    if (elect_one()) umma_commit(all_done);  // every MMA complete before TMEM is freed
    mbar_wait(all_done, 0, a.t.err);
    __syncwarp();
  } else if (warp < 6) {
    // ---- Q: a warp a quarter of the columns, a lane to a column's numbers ----
    // A step's numbers are looked up a step before its rows are asked for.  With four slots
    // its rows are waited for two steps later; with two at once, since the next step's slot
    // is only free when the MMAs that wait for these rows are next.
    constexpr int kLag = C::kSlotsQ > 2 ? 2 : 0;
    const int w = warp - 2;
    constexpr int kMine = kCols / 4;       // columns of a warp
    constexpr int kPieces = D / 8;         // 16-byte pieces of a row
    constexpr int kAtOnce = 32 / kPieces;  // columns that a warp's lanes copy a piece each of
    struct Column {
      int64_t from;  // of q; -1: none
      float l;
      int pos;  // of the positions behind the length, the last one that it sees
    };
    auto look = [&](const WCursor<kCols>& c) {
      Column x{-1, 0.f, INT32_MIN};
      const int col = c.chunk * kCols + w * kMine + lane;
      if (lane < kMine && col < c.s.n * a.G) {
        const int i = col / a.G, head = c.h * a.G + col - i * a.G;
        const int node = a.path ? a.path[static_cast<int64_t>(c.b) * a.t.T + i] : i;
        if (static_cast<unsigned>(node) < static_cast<unsigned>(a.t.T)) {
          x.l = a.lse[(static_cast<int64_t>(c.b) * a.t.T + node) * (a.H * a.G) + head];
          x.pos = i;
          x.from = c.b * a.qb + node * a.qt + head * a.qh;
        } else {
          record_error(a.t.err, kDevErrBadIndex);
        }
      }
      return x;
    };
    int64_t* from = from_s + w * kMine;
    const int piece = lane % kPieces, c0 = lane / kPieces;  // this lane's, of kAtOnce columns
    // a row's piece p lies at p ^ (row % 8) of its 128 bytes; 8 rows are 1024 bytes
    const int dst0 = (piece >> 3) * (kCols * 128) + w * kMine * 128;
    int slot = 0, ph = 0, before[2] = {0, 0};  // the slots of the steps before
    int64_t i = 0;
    Column next{};
    if (N > 0) next = look(cur);
    for (; i < N; ++i) {
      const Column x = next;
      const int mine = min(kMine, cur.s.n * a.G - cur.chunk * kCols - w * kMine);
      if (i + 1 < N) {
        cur.next(a, kt);
        next = look(cur);
      }
      const int info = static_cast<int>(i & (kInfos - 1));
      if (i >= kInfos) ok = wait(&i_empty[info], ((i / kInfos) - 1) & 1, a.t.err);
      if (i >= C::kSlotsQ) ok = ok && wait(&q_empty[slot], ph ^ 1, a.t.err);
      ok = __all_sync(kAll, ok);
      if (!ok) break;
      if (lane < kMine) {
        lse_s[info * kCols + w * kMine + lane] = -x.l * kLog2e;
        pos_s[info * kCols + w * kMine + lane] = isfinite(x.l) ? x.pos : INT32_MIN;
        from[lane] = x.from;
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&i_full[info]);
      uint8_t* dst = qs + slot * C::kSlotQ + dst0;
#pragma unroll 4
      for (int c = c0; c < mine; c += kAtOnce) {
        const int64_t f = from[c];
        cp_async16(dst + c * 128 + (((piece & 7) ^ (c & 7)) << 4),
                   static_cast<const E*>(a.q) + (f < 0 ? 0 : f) + piece * 8, f >= 0);
      }
      cp_async_commit();
      __syncwarp();  // (the next step's numbers replace these)
      if (i >= kLag) {
        cp_async_wait<kLag>();
        fence_proxy_async_smem();
        mbar_arrive(&q_full[kLag ? before[1] : slot]);
      }
      before[1] = before[0];
      before[0] = slot;
      if (++slot == C::kSlotsQ) {
        slot = 0;
        ph ^= 1;
      }
    }
    cp_async_wait<0>();
    fence_proxy_async_smem();
    if (kLag && i > 1) mbar_arrive(&q_full[before[1]]);
    if (kLag && i > 0) mbar_arrive(&q_full[before[0]]);
  } else {
    // ---- sums: a thread to a key, four warps to a tile of the group ----
    const int t = (warp - 6) >> 2, quarter = warp & 3, key = quarter * 32 + lane;
    const uint32_t tbase = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
    const uint64_t sl2 = pack_f32x2(a.scale_log2, a.scale_log2);
    if (t == 0 && key == 0) a.cuts[blockIdx.x].b = -1;
    uint32_t m = t;  // the round of this tile in this step
    for (int64_t i = 0; i < N && ok;) {
      // this CTA's steps of a group
      const WSeq s = cur.s;
      const int here = cur.here(kt), tile = cur.group * kt + t;
      const int per = a.H * s.chunks, at0 = cur.h * s.chunks + cur.chunk;
      const int64_t i1 = min(N, i + per - at0);
      const int64_t v0 = g.u0 + i - at0;  // the group's first step
      const int rel = tile * kTile + key - s.len;  // < 0: committed
      const bool plain = (tile + 1) * kTile <= s.len;
      int chunk = cur.chunk;
      uint64_t sum[2] = {0, 0};
      for (; i < i1; ++i, m += kt) {
        const int info = static_cast<int>(i & (kInfos - 1));
        if (ok) ok = wait(&i_full[info], (i / kInfos) & 1, a.t.err);  // (an idle warp keeps in step)
        ok = __all_sync(kAll, ok);
        if (t < kt) {
          const int cols = t < here ? min(kCols, s.n * a.G - chunk * kCols) : 0;
          const float* l = lse_s + info * kCols;
          const int* p = pos_s + info * kCols;
          const uint32_t acc = m % kAccs;
          if (ok) ok = wait(&s_full[acc], m / kAccs & 1, a.t.err);
          ok = __all_sync(kAll, ok);
          if (ok) {
            tc_fence_after();
            uint64_t step[2] = {0, 0};
#pragma unroll 1
            for (int c = 0; c < cols; c += 32) {
              uint32_t x[32];
              tmem_ld32_issue(tbase + acc * kCols + c, x);
              // (a column that is left out, or past the last, is seen by no key)
              const bool whole = plain && __all_sync(kAll, p[c + lane] >= 0);
              tmem_ld32_wait(x);
              if (whole) {
#pragma unroll
                for (int j = 0; j < 32; j += 4) {
                  const float4 y = *reinterpret_cast<const float4*>(l + c + j);
                  float e[4];
                  unpack_f32x2(fma_f32x2(pack_u32x2(x[j], x[j + 1]), sl2, pack_f32x2(y.x, y.y)), e[0],
                               e[1]);
                  unpack_f32x2(fma_f32x2(pack_u32x2(x[j + 2], x[j + 3]), sl2, pack_f32x2(y.z, y.w)),
                               e[2], e[3]);
                  step[0] = add_f32x2(step[0], pack_f32x2(ex2(e[0]), ex2(e[1])));
                  step[1] = add_f32x2(step[1], pack_f32x2(ex2(e[2]), ex2(e[3])));
                }
              } else {
#pragma unroll
                for (int j = 0; j < 32; j += 4) {
                  const float4 y = *reinterpret_cast<const float4*>(l + c + j);
                  const int4 at = *reinterpret_cast<const int4*>(p + c + j);
                  float e[4] = {ex2(fmaf(__uint_as_float(x[j]), a.scale_log2, y.x)),
                                ex2(fmaf(__uint_as_float(x[j + 1]), a.scale_log2, y.y)),
                                ex2(fmaf(__uint_as_float(x[j + 2]), a.scale_log2, y.z)),
                                ex2(fmaf(__uint_as_float(x[j + 3]), a.scale_log2, y.w))};
                  e[0] = rel <= at.x ? e[0] : 0.f;
                  e[1] = rel <= at.y ? e[1] : 0.f;
                  e[2] = rel <= at.z ? e[2] : 0.f;
                  e[3] = rel <= at.w ? e[3] : 0.f;
                  step[0] = add_f32x2(step[0], pack_f32x2(e[0], e[1]));
                  step[1] = add_f32x2(step[1], pack_f32x2(e[2], e[3]));
                }
              }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&s_empty[acc]);
            sum[0] = add_f32x2(sum[0], step[0]);
            sum[1] = add_f32x2(sum[1], step[1]);
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&i_empty[info]);
        if (++chunk == s.chunks) chunk = 0;
      }
      // ---- the end of this CTA's part of the group ----
      const bool begins = at0 == 0, ends = g.u0 + i == v0 + per;
      if (t < here && ok) {
        float s0, s1;
        unpack_f32x2(add_f32x2(sum[0], sum[1]), s0, s1);
        if (begins && ends)
          put(a, s, tile * kTile + key, s0 + s1);
        else
          a.parts[((static_cast<int64_t>(blockIdx.x) * 2 + (begins ? 1 : 0)) * kMaxGroup + t) * kTile +
                  key] = s0 + s1;
      }
      if (begins && !ends && t == 0 && key == 0)
        a.cuts[blockIdx.x] = WeighCut{cur.b, static_cast<int>(blockIdx.x),
                                      range_of(g.units, g.n_cta, v0 + per - 1), tile * kTile, s.row,
                                      s.len, s.n, min(here * kTile, s.len + s.n - tile * kTile)};
      cur.h = a.H - 1;  // on to the next group
      cur.chunk = s.chunks - 1;
      cur.next(a, kt);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, kAccs * kCols);
}

// The parts of the groups that several ranges share, in order.
__global__ void __launch_bounds__(kMaxGroup * kTile)
    weigh_add_kernel(const __grid_constant__ WeighArgs a) {
  pdl_wait();
  pdl_launch_dependents();
  const WeighCut cut = a.cuts[blockIdx.x];
  const int x = threadIdx.x;
  if (cut.b < 0 || x >= cut.keys) return;
  constexpr int kPart = kMaxGroup * kTile;
  const int pos = cut.pos + x;
  float* w = a.weight + (static_cast<int64_t>(cut.row) * a.t.cols << a.t.page_shift) + pos;
  const float old = *w;  // (beside the parts and the page's number)
  const int page = a.t.entry(cut.row, pos >> a.t.page_shift);
  float sum = a.parts[(static_cast<int64_t>(cut.c0) * 2 + 1) * kPart + x];
#pragma unroll 8
  for (int c = cut.c0 + 1; c <= cut.c1; ++c) sum += a.parts[static_cast<int64_t>(c) * 2 * kPart + x];
  if (a.t.checked(page) >= 0) *w = (a.first && pos >= cut.len ? 0.f : old) + sum;
}

struct WeighPlan {
  int grid;
  size_t cut_off, ws_bytes;
};
WeighPlan weigh_plan() {
  WeighPlan p;
  p.grid = device_info().sms;
  p.cut_off = align_up(size_t(p.grid) * 2 * kMaxGroup * kTile * sizeof(float), 256);
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
  return launch_k(weigh_add_kernel, dim3(a.grid), dim3(kMaxGroup * kTile), 0, s, true, a);
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
