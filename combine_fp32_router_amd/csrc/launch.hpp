// Host-side launchers of the gfx950 kernels.  Arguments are validated by the
// C ABI (abi.cpp) before any of these is called; each returns the HIP error
// of its launch(es).
#pragma once

#include <hip/hip_runtime_api.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/moe_route.h"

namespace moe {

hipError_t launch_route_topk(const float *logits, int64_t T, int E, int k,
                             int32_t *idx, float *w, hipStream_t stream);
// Workgroups of kRouteThreads threads that launch_route_topk runs for T tokens.
constexpr int kRouteThreads = 256;
int64_t route_topk_blocks(int64_t T, int E);

// A HIP launch counts the work-items of each grid dimension in 32 bits: a
// dimension of `blocks` workgroups of `threads` work-items must stay below
// 2^32.  The C ABI refuses calls whose grid would not (MOE_ERR_SHAPE).
inline bool grid_fits(int64_t blocks, int threads)
{
    return blocks <= int64_t(0xFFFFFFFF) / threads;
}

// Tiling of the layout: `tile_slots` slots per wave-tile, `ntiles` tiles.
struct LayoutTiling {
    int tile_slots;
    int ntiles;
};
LayoutTiling layout_tiling(int64_t slots, int E);
// Chunks of a batched layout: ceil(T / chunk_tokens) (1 when T == 0).
int layout_chunks(int64_t T, int64_t chunk_tokens);
size_t layout_workspace_bytes(int64_t T, int64_t chunk_tokens, int E, int k);

// Layout of every chunk of chunk_tokens tokens (the last may be shorter) in
// one pair of launches.  Capacity of chunk c: cap_chunk[c] (device array)
// when cap_chunk is not NULL, else cap_all (<= 0: unlimited).
hipError_t launch_dispatch_layout(const int32_t *idx, int64_t T, int64_t chunk_tokens, int E,
                                  int k, int R, const int32_t *cap_chunk, int cap_all,
                                  int32_t *expert_counts, int32_t *expert_offsets,
                                  int32_t *rank_counts, int32_t *rank_offsets, int32_t *pos,
                                  int32_t *row_src, void *workspace, hipStream_t stream);

// Router fused with the layout's histogram pass (two launches; falls back to
// route + layout when a layout tile does not hold whole router groups).
// Tokens per router group (one histogram row) of a fused call over T tokens.
int route_group_tokens(int E, int64_t T);
hipError_t launch_route_hist(const float *logits, int64_t T, int64_t chunk_tokens, int chunks,
                             int E, int k, int hrows, int32_t *idx, float *w, int32_t *hist,
                             hipStream_t stream);
size_t route_layout_workspace_bytes(int64_t T, int64_t chunk_tokens, int E, int k);
hipError_t launch_route_layout(const float *logits, int64_t T, int64_t chunk_tokens, int E,
                               int k, int R, const int32_t *cap_chunk, int cap_all,
                               int32_t *idx, float *w, int32_t *expert_counts,
                               int32_t *expert_offsets, int32_t *rank_counts,
                               int32_t *rank_offsets, int32_t *pos, int32_t *row_src,
                               void *workspace, hipStream_t stream);

// Device address of the static histogram scratch (MOE_NOALLOC_SCRATCH_BYTES)
// on the device of `stream` (the current device for the null stream), looked
// up on the first call on each device.
hipError_t static_scratch(hipStream_t stream, void **ptr);

// Quantised payloads (quant != 0) write / read one fp32 scale per row in
// `scales` (send / recv rows at the same index); bf16 ignores it.
// stream_stores: the send rows are written with streaming device-scope
// stores (not kept in the last-level cache) instead of device-scope stores.
hipError_t launch_dispatch_pack(const void *x, int64_t T, int H, int k,
                                const int32_t *pos, int quant, bool stream_stores, void *send,
                                float *scales, hipStream_t stream);

hipError_t launch_combine(const void *recv, const float *scales, int quant, const int32_t *pos,
                          const float *w, int64_t T, int H, int k, void *out,
                          hipStream_t stream);

// Combine of Tc tokens (blocks first) and pack of Tp tokens in one grid;
// stream_stores applies to the pack half, as for launch_dispatch_pack.
hipError_t launch_combine_pack(const void *recv, const float *rscales, const int32_t *pos_c,
                               const float *w, int64_t Tc, void *out, const void *x,
                               const int32_t *pos_p, int64_t Tp, void *send, float *sscales,
                               int H, int k, int quant, bool stream_stores, hipStream_t stream);

// Receiver side: segment offsets, expert-major starts and the two row maps
// (group_pos: receive row -> grouped row, group_src: the inverse; -1 past N).
hipError_t launch_recv_layout(const int32_t *src_offsets, int E, int R, int64_t max_rows,
                              int32_t *recv_offsets, int32_t *group_offsets, int32_t *group_seg,
                              int32_t *group_pos, int32_t *group_src, hipStream_t stream);

// out[i] = in[map[i]] for i < max_rows, rows of row_bytes(H, quant) bytes
// (and their scales for quant != 0); rows whose map entry is outside
// [0, max_rows) are not written.
hipError_t launch_gather_rows(const void *in, const float *in_scales, void *out, float *out_scales,
                              int64_t max_rows, int H, int quant, const int32_t *map,
                              hipStream_t stream);

// Balance loss over segments of `seg` tokens, and the router's gradient.
size_t balance_workspace_bytes(int64_t T, int64_t seg, int E);
hipError_t launch_balance_loss(const float *logits, const int32_t *idx, const uint8_t *mask,
                               int64_t T, int64_t seg, int E, int k, float *loss, int32_t *counts,
                               float *prob_sums, int32_t *live, void *workspace,
                               hipStream_t stream);
int64_t route_grad_blocks(int64_t seg, int E);  // of a segment, of kRouteThreads threads
hipError_t launch_route_grad(const float *logits, const int32_t *idx, const float *w,
                             const float *dw, const uint8_t *mask, const float *dloss,
                             const int32_t *counts, const int32_t *live, int64_t T, int64_t seg,
                             int E, int k, bool masked_gates, float *dlogits, hipStream_t stream);

// Gradient of the combine; d_rows or d_w may be null.
hipError_t launch_combine_grad(const void *d_out, const void *rows, const float *scales, int quant,
                               const int32_t *pos, const float *w, int64_t T, int H, int k,
                               void *d_rows, float *d_w, hipStream_t stream);

// Blocks of values with one scale, along a row.
constexpr int kCodeBlock = 128;
constexpr int code_blocks(int n) { return (n + kCodeBlock - 1) / kCodeBlock; }

// The residual's addition with the norm, and its gradient; codes and scales of
// rows and of weights.
hipError_t launch_add_norm(const void *x, const void *residual, const float *weight, float eps, int64_t T, int H,
                           void *sum, void *y, bool blocks, void *codes, float *scales, hipStream_t stream);
size_t norm_grad_workspace_bytes(int64_t T, int H);
hipError_t launch_add_norm_grad(const void *d_y, const void *d_sum, const void *sum, const float *weight, float eps,
                                int64_t T, int H, void *d_x, float *d_weight, bool accumulate, void *workspace,
                                hipStream_t stream);
hipError_t launch_quant_rows(const void *x, const int32_t *offsets, int E, int64_t max_rows, int n, int halves,
                             void *codes, float *scales, hipStream_t stream);
hipError_t launch_quant_wide_rows(const float *x, const int32_t *offsets, int E, int64_t max_rows, int n, int halves,
                                  void *codes, float *scales, hipStream_t stream);  // of fp32 values
int64_t quant_weights_groups(int E, int N, int K, int halves);  // of kRouteThreads threads
hipError_t launch_quant_weights(const void *w, int E, int N, int K, int halves, void *codes, float *scales,
                                void *codes_t, float *scales_t, hipStream_t stream);

// The experts' products of E4M3 rows and weights, and the gradient of their rows.
hipError_t launch_expert_fp8(const void *x, const float *xs, int xs_cols, const int32_t *offsets, const void *w,
                             const float *ws, const float *bias, int act, const void *residual, int E, int64_t max_rows,
                             int K, int N, void *out, void *codes, float *scales, void *preact, void *workspace,
                             hipStream_t stream);
size_t expert_fp8_workspace_bytes(int act, int E, int64_t max_rows, int K, int N);
size_t expert_fp8_dx_workspace_bytes(int halves, int act, int E, int64_t max_rows, int K, int N);
hipError_t launch_expert_fp8_dx(const void *dy, const float *dys, const int32_t *offsets, const void *wt,
                                const float *wts, int halves, int act, const void *z, int E, int64_t max_rows, int K,
                                int N, void *dx, void *codes, float *scales, void *workspace, hipStream_t stream);

// The experts' products over their runs of rows, and their gradients.
hipError_t launch_expert_matmul(const void *x, const int32_t *offsets, const void *w,
                                const float *bias, int act, const void *residual, int E,
                                int64_t max_rows, int K, int N, void *out, void *preact,
                                void *workspace, hipStream_t stream);
// The same for few rows an expert, and whether it pays.
bool few_rows_pay(int act, int E, int64_t max_rows, int K, int N, int parts);
hipError_t launch_expert_few(const void *x, const int32_t *offsets, const void *w, const float *bias,
                             int act, const void *residual, int E, int64_t max_rows, int K, int N,
                             void *out, void *preact, hipStream_t stream);
hipError_t launch_expert_matmul_dx(const void *dy, const int32_t *offsets, const void *w, int act,
                                   const void *z, int E, int64_t max_rows, int K, int N, void *dx,
                                   void *workspace, hipStream_t stream);
// The products walk lists of 256 x 256 tiles counted in 32 bits.
inline bool product_tiles_fit(int64_t row_tiles, int cols) { return row_tiles * ((cols + 127) / 128) < (int64_t(1) << 30); }
hipError_t launch_expert_matmul_dw(const void *dy, const void *x, const int32_t *offsets, int E,
                                   int64_t max_rows, int K, int N, int flags, void *dw, float *db,
                                   void *workspace, hipStream_t stream);
// In how many parts a product's reduced length is taken (1: whole), its tiles
// then, and the workspace for them.  row_parts: products of rows with reduced
// length R and C output columns, `unit` of which make 128 of a tile.
struct Parts {
    int parts;
    int64_t tiles, bytes;
};
Parts row_parts(int E, int64_t max_rows, int R, int C, int unit);
Parts forward_parts(int act, int E, int64_t max_rows, int K, int N);
Parts dw_parts(int E, int64_t max_rows, int K, int N);

// Most tiles of `height` rows that E runs of together max_rows rows can have.
inline int64_t max_row_tiles(int64_t max_rows, int E, int height)
{
    const int64_t live = max_rows < E ? max_rows : E;
    return (max_rows - live) / height + live;
}

constexpr int kCus = 256;  // of the card
constexpr int64_t kCacheBytes = 256 << 20;  // of its last-level cache

// Rows and columns of the tiles of a product whose outputs have C columns,
// `unit` of which make 128 of a tile.  256 x 256 has the best rate; smaller ones
// serve a call that all of them fit the card at once, where larger ones would
// leave more of it idle.  Cost in percent of 256 x 256's, as measured: 72 with
// half the columns (K = N = 2048, 4096 rows: 38 us against 51; 4352 rows, more
// than fit: 64 against 51), 49 and 38 with half or a quarter of the rows too
// (K = N = 1024, 2048 rows: 11.9 us against 20.7; 8192 rows, K = 16384, N =
// 256: 121 against 218).
struct TileShape {
    int rows, cols, percent;
    int64_t tiles;
};
inline TileShape tile_shape(int E, int64_t max_rows, int C, int unit)
{
    const TileShape shapes[6] = {{64, 128, 38, 0},  {64, 256, 44, 0},  {128, 128, 49, 0},
                                 {128, 256, 63, 0}, {256, 128, 72, 0}, {256, 256, 100, 0}};
    TileShape s{};
    for (const TileShape &each : shapes) {
        s = each;
        const int cols = s.cols / 128 * unit;
        s.tiles = max_row_tiles(max_rows, E, s.rows) * ((C + cols - 1) / cols);
        if (s.tiles <= kCus)
            break;
    }
    return s;
}

// Threads per block and 16-byte vectors per thread covering one row of
// `vecs` 16-byte vectors with one block (<= 1024 threads, a whole number of
// 64-lane waves): one vector per thread up to 1024 vectors, then 2, 4, 8.
struct RowTiling {
    int threads;
    int vpt;
};
// The int8 / fp8 / int4 kernels tile 16-element groups: G = H / 16 <= 4096
// groups, so their vpt is at most 4 and only 1, 2 and 4 are built (the bf16
// kernels tile H / 8 <= 8192 vectors and take up to 8).
static_assert(MOE_MAX_HIDDEN / 16 <= 4 * 1024, "16-element groups: at most four per thread");
inline RowTiling row_tiling(int vecs)
{
    RowTiling r;
    r.vpt = 1;
    while (r.vpt < 8 && (vecs + r.vpt - 1) / r.vpt > 1024)
        r.vpt *= 2;
    int thr = (vecs + r.vpt - 1) / r.vpt;
    thr = ((thr + 63) / 64) * 64;
    r.threads = thr < 64 ? 64 : thr;
    return r;
}

// Threads of the one-workgroup-per-token pack, combine and combine+pack
// kernels: the bf16 kernels tile H / 8 vectors, the others H / 16 groups.
inline int token_threads(int H, int quant)
{
    return row_tiling(quant == MOE_QUANT_BF16 ? H / 8 : H / 16).threads;
}

}  // namespace moe
