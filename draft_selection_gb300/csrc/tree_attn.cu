// The attention's entry points, dfl2_tree_attn and dfl2_window_attn, and its plan; the
// kernels are tree_attn_kernel.cuh's, instantiated here without a window.
#include <algorithm>
#include <cmath>

#include "tree_attn_kernel.cuh"

#define DFL2_TRY(expr)              \
  do {                              \
    dfl2_status _st = (expr);       \
    if (_st != DFL2_OK) return _st; \
  } while (0)

namespace dfl2 {

dfl2_status check_attn_shapes(int B, int T, int q_heads, int kv_heads, int head_dim, int dtype) {
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

namespace {

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

// Both entry points; `windowed`: with sinks, window and depth.
dfl2_status attend(const void* q, const int64_t* q_strides, const dfl2_cache* cache, int layer,
                   int B, int T, int q_heads, const int32_t* table_rows, const int32_t* length,
                   const int32_t* count, const uint32_t* mask, bool windowed, const int32_t* depth,
                   int sinks, int window, float scale, void* out, const int64_t* out_strides,
                   float* lse, void* ws, size_t ws_bytes, dfl2_stream stream) {
  const PtrArg ptrs[] = {{q, "q", 16}, {table_rows, "table_rows", 4, true},
                               {length, "length", 4}, {count, "count", 4, true},
                               {mask, "mask", 4, true}, {out, "out", 16}, {lse, "lse", 4, true},
                          {depth, "depth", 4, true}};
  DFL2_TRY(check_cache_host(cache));
  DFL2_TRY(check_attn_shapes(B, T, q_heads, cache->kv_heads, cache->head_dim, cache->dtype));
  DFL2_TRY(check_args_host(ptrs, 8));
  if (layer < 0 || layer >= cache->layers)
    return report_errorf(DFL2_ERR_INVALID_ARG, "layer %d of %d", layer, cache->layers);
  if (!q_strides || !out_strides)
    return report_errorf(DFL2_ERR_INVALID_ARG, "q_strides and out_strides are needed");
  // a tensor map's strides are positive, under 2^40 bytes and multiples of 16
  const int64_t most = int64_t(1) << 38;
  const int dims[3] = {B, T, q_heads};
  for (int i = 0; i < 3; ++i)
    for (const int64_t st : {q_strides[i], out_strides[i]})
      if (dims[i] > 1 && (st < 1 || st > most || st % 8))
        return report_errorf(DFL2_ERR_INVALID_ARG,
                                   "strides of q and out: multiples of 8 from 8 to 2^38");
  const int cdims[3] = {cache->page_size, cache->kv_heads, cache->pages};
  const int64_t cst[3] = {cache->slot_stride, cache->head_stride, cache->page_stride};
  for (int i = 0; i < 3; ++i)
    if (cdims[i] > 1 && (cst[i] < 1 || cst[i] > most))
      return report_errorf(DFL2_ERR_UNSUPPORTED,
                                 "the attention needs cache strides of 8 .. 2^38 elements");
  if (!std::isfinite(scale))
    return report_errorf(DFL2_ERR_INVALID_ARG, "scale %g must be finite", double(scale));
  if (windowed) {
    if (window < 1 || sinks < 0)
      return report_errorf(DFL2_ERR_INVALID_ARG, "window=%d must be >= 1, sinks=%d >= 0", window,
                           sinks);
    if (window > kMaxLen || sinks > kMaxLen)
      return report_errorf(DFL2_ERR_UNSUPPORTED, "window=%d, sinks=%d: at most 2^30", window, sinks);
    if (mask && !depth)
      return report_errorf(DFL2_ERR_INVALID_ARG, "a mask needs the nodes' depths");
  }
  DFL2_TRY(check_args_device(ptrs, 8));
  DFL2_TRY(check_cache_device(cache));
  const int G = q_heads / cache->kv_heads, D = cache->head_dim;
  const AttnPlan p = attn_plan(T, G, D, device_info().sms);
  if (!ws || ws_bytes < p.ws_bytes)
    return report_errorf(DFL2_ERR_WORKSPACE, "workspace of %zu bytes < %zu needed",
                               ws ? ws_bytes : size_t(0), p.ws_bytes);
  const PtrArg wsp[] = {{ws, "workspace", 16}};
  DFL2_TRY(check_args_host(wsp, 1));
  DFL2_TRY(check_args_device(wsp, 1));
  uint8_t* w = reinterpret_cast<uint8_t*>(
      align_up(reinterpret_cast<uintptr_t>(ws), 256));  // parts are stored 32 bytes at a time
  const int64_t at = layer * cache->layer_stride * 2;
  AttnArgs a{};
  a.t = table_view(cache, table_rows, length, count, T);
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
  a.scale_log2 = scale * kLog2e;
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
  a.cuts = reinterpret_cast<Cut*>(w + p.cut_off);
  a.grid = p.grid;
  a.rows = p.rows;
  a.stream_rows = p.stream_rows;
  a.row_tiles = p.row_tiles;
  a.sinks = sinks;
  a.window = window;
  a.depth = depth;
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e = windowed                    ? launch_window_attn(a, cache, s)
                        : cache->dtype == DFL2_F16 ? launch_attn_d<__half, false>(a, cache, s)
                                                   : launch_attn_d<__nv_bfloat16, false>(a, cache, s);
  return e == cudaSuccess ? DFL2_OK : report_cuda_error(e, "tree attention launch");
}

}  // namespace
}  // namespace dfl2

extern "C" {

size_t dfl2_tree_attn_workspace_size(int B, int T, int q_heads, int kv_heads, int head_dim,
                                     dfl2_dtype dtype) {
  if (dfl2::check_attn_shapes(B, T, q_heads, kv_heads, head_dim, dtype) != DFL2_OK) return 0;
  if (dfl2::check_args_device(nullptr, 0) != DFL2_OK) return 0;
  return dfl2::attn_plan(T, q_heads / kv_heads, head_dim, dfl2::device_info().sms).ws_bytes;
}

dfl2_status dfl2_tree_attn(const void* q, const int64_t* q_strides, const dfl2_cache* cache,
                           int layer, int B, int T, int q_heads, const int32_t* table_rows,
                           const int32_t* length, const int32_t* count, const uint32_t* mask,
                           float scale, void* out, const int64_t* out_strides, float* lse,
                           void* ws, size_t ws_bytes, dfl2_stream stream) {
  return dfl2::attend(q, q_strides, cache, layer, B, T, q_heads, table_rows, length, count, mask,
                      false, nullptr, 0, 0, scale, out, out_strides, lse, ws, ws_bytes, stream);
}

dfl2_status dfl2_window_attn(const void* q, const int64_t* q_strides, const dfl2_cache* cache,
                             int layer, int B, int T, int q_heads, const int32_t* table_rows,
                             const int32_t* length, const int32_t* count, const uint32_t* mask,
                             const int32_t* depth, int sinks, int window, float scale, void* out,
                             const int64_t* out_strides, float* lse, void* ws, size_t ws_bytes,
                             dfl2_stream stream) {
  return dfl2::attend(q, q_strides, cache, layer, B, T, q_heads, table_rows, length, count, mask,
                      true, depth, sinks, window, scale, out, out_strides, lse, ws, ws_bytes,
                      stream);
}

}  // extern "C"
