// C ABI of the dispatch/combine library: host-side validation of every
// argument, then the kernel launchers.  Nothing is launched and no output is
// touched when validation fails; no call aborts, exits or throws.
#include <hip/hip_runtime_api.h>

#include <stdint.h>

#include "../../include/moe_recv.h"
#include "../../include/moe_route.h"
#include "checks.hpp"
#include "launch.hpp"

using namespace moe;

namespace {

// A byte range [p, p + bytes); a null pointer is an empty range.
struct Extent {
    const void *p;
    int64_t bytes;
};

bool overlap(const Extent &a, const Extent &b)
{
    if (!a.p || !b.p || a.bytes <= 0 || b.bytes <= 0)
        return false;
    const uintptr_t a0 = reinterpret_cast<uintptr_t>(a.p), b0 = reinterpret_cast<uintptr_t>(b.p);
    return a0 < b0 + static_cast<uintptr_t>(b.bytes) && b0 < a0 + static_cast<uintptr_t>(a.bytes);
}

// Segments of the balance loss: seg_tokens is clamped to T (one segment).
int check_segments(int64_t T, int64_t &seg_tokens, int E, int k)
{
    if (T < 0 || check_ek(E, k) != MOE_OK || too_many_slots(T, k) || seg_tokens < 0 ||
        (T > 0 && seg_tokens < 1))
        return MOE_ERR_SHAPE;
    if (seg_tokens > T)
        seg_tokens = T;
    return moe::layout_chunks(T, seg_tokens) > 65535 ? MOE_ERR_SHAPE : MOE_OK;  // grid y dimension
}

// Sizes of an experts' product: N may count both halves of a gated one.  The
// kernels round a run's rows up to whole tiles (of at most 256) and look two
// stages (128 rows) past its end in 32 bits.
constexpr int64_t kMaxProductRows = kMaxSlots - 256;
int check_product(int E, int64_t max_rows, int K, int N, int most)
{
    if (E < 1 || E > MOE_MAX_EXPERTS || max_rows < 0 || max_rows > kMaxProductRows || K < 16 ||
        K > MOE_MAX_HIDDEN || (K % 16) != 0 || N < 16 || N > most || (N % 16) != 0)
        return MOE_ERR_SHAPE;
    return MOE_OK;
}

// Rows and eps of the norm (eps >= 0; NaN is none).
int check_norm(int64_t T, int H, float eps)
{
    return T < 0 || T >= kMaxSlots || H < 16 || H > MOE_MAX_HIDDEN || H % 16 != 0 || !(eps >= 0.0f) ? MOE_ERR_SHAPE
                                                                                                  : MOE_OK;
}

// The 8-bit products' grids and lists count tiles of 64 x 128 in 32 bits.
bool fp8_tiles_fit(int E, int64_t max_rows, int cols)
{
    return max_row_tiles(max_rows, E, 64) * code_blocks(cols) < (int64_t(1) << 24) - 1;
}

bool known_act(int act) { return act >= MOE_ACT_NONE && act <= MOE_ACT_SWIGLU; }

}  // namespace

extern "C" {

int64_t moe_row_bytes(int H, int quant)
{
    if (quant == MOE_QUANT_BF16)
        return 2 * static_cast<int64_t>(H);
    if (quant == MOE_QUANT_INT8 || quant == MOE_QUANT_FP8)
        return static_cast<int64_t>(H);
    if (quant == MOE_QUANT_INT4)
        return static_cast<int64_t>(H) / 2;
    return -1;
}

const char *moe_status_string(int status)
{
    switch (status) {
    case MOE_OK: return "MOE_OK";
    case MOE_ERR_NULL: return "MOE_ERR_NULL: a required pointer is NULL";
    case MOE_ERR_SHAPE: return "MOE_ERR_SHAPE: a size argument is out of range";
    case MOE_ERR_ALIGN: return "MOE_ERR_ALIGN: a buffer is not aligned as required";
    case MOE_ERR_WORKSPACE: return "MOE_ERR_WORKSPACE: workspace missing or too small";
    case MOE_ERR_HIP: return "MOE_ERR_HIP: the HIP runtime rejected a launch";
    case MOE_ERR_ALIAS: return "MOE_ERR_ALIAS: an output is the same buffer as an input";
    case MOE_ERR_SCRATCH:
        return "MOE_ERR_SCRATCH: the call needs more than the static scratch buffer holds";
    default: return "unknown moe status";
    }
}

int moe_route_topk(const float *logits, int64_t T, int E, int k, int32_t *topk_idx,
                   float *topk_w, hipStream_t stream)
{
    if (T < 0 || check_ek(E, k) != MOE_OK || too_many_slots(T, k) ||
        !grid_fits(route_topk_blocks(T, E), kRouteThreads))
        return MOE_ERR_SHAPE;
    if (T == 0)
        return MOE_OK;
    if (!logits || !topk_idx || !topk_w)
        return MOE_ERR_NULL;
    if (!aligned(logits, 4) || !aligned(topk_idx, 4) || !aligned(topk_w, 4))
        return MOE_ERR_ALIGN;
    return hip_status(moe::launch_route_topk(logits, T, E, k, topk_idx, topk_w, stream));
}

int moe_dispatch_layout(const int32_t *topk_idx, int64_t T, int E, int k, int R, int capacity,
                        int32_t *expert_counts, int32_t *expert_offsets, int32_t *rank_counts,
                        int32_t *rank_offsets, int32_t *pos, int32_t *row_src, void *workspace,
                        size_t *workspace_bytes, hipStream_t stream)
{
    // one chunk of T tokens
    return moe_dispatch_layout_chunks(topk_idx, T, T, E, k, R, capacity, nullptr, expert_counts,
                                      expert_offsets, rank_counts, rank_offsets, pos, row_src,
                                      workspace, workspace_bytes, stream);
}

int moe_dispatch_layout_chunks(const int32_t *topk_idx, int64_t T, int64_t chunk_tokens, int E,
                               int k, int R, int capacity, const int32_t *chunk_capacity,
                               int32_t *expert_counts, int32_t *expert_offsets,
                               int32_t *rank_counts, int32_t *rank_offsets, int32_t *pos,
                               int32_t *row_src, void *workspace, size_t *workspace_bytes,
                               hipStream_t stream)
{
    if (!workspace_bytes)
        return MOE_ERR_NULL;
    if (T < 0 || check_ek(E, k) != MOE_OK || R < 1 || (E % R) != 0 || too_many_slots(T, k) ||
        chunk_tokens < 0 || (T > 0 && chunk_tokens < 1))
        return MOE_ERR_SHAPE;
    if (chunk_tokens > T)
        chunk_tokens = T;  // one chunk
    if (moe::layout_chunks(T, chunk_tokens) > 65535)  // grid y dimension
        return MOE_ERR_SHAPE;
    const size_t need = moe::layout_workspace_bytes(T, chunk_tokens, E, k);
    if (!workspace) {
        *workspace_bytes = need;
        return MOE_OK;
    }
    if (*workspace_bytes < need)
        return MOE_ERR_WORKSPACE;
    if (!expert_counts || !expert_offsets || !rank_counts || !rank_offsets)
        return MOE_ERR_NULL;
    if (T > 0 && (!topk_idx || !pos || !row_src))
        return MOE_ERR_NULL;
    if (!aligned(expert_counts, 4) || !aligned(expert_offsets, 4) || !aligned(rank_counts, 4) ||
        !aligned(rank_offsets, 4) || !aligned(topk_idx, 4) || !aligned(pos, 4) ||
        !aligned(row_src, 4) || !aligned(chunk_capacity, 4) || !aligned(workspace, 256))
        return MOE_ERR_ALIGN;
    return hip_status(moe::launch_dispatch_layout(topk_idx, T, chunk_tokens, E, k, R,
                                                  chunk_capacity, capacity, expert_counts,
                                                  expert_offsets, rank_counts, rank_offsets, pos,
                                                  row_src, workspace, stream));
}

}  // extern "C"

namespace {

// Sizes of the fused route + layout.  On MOE_OK, chunk_tokens is clamped to
// T (one chunk) and `need` holds the histogram scratch the call takes.
int route_layout_sizes(int64_t T, int64_t &chunk_tokens, int E, int k, int R, size_t &need)
{
    // (the router's grid is checked as for moe_route_topk: a call the fused
    // kernel cannot take runs it over the whole batch)
    if (T < 0 || check_ek(E, k) != MOE_OK || R < 1 || (E % R) != 0 || too_many_slots(T, k) ||
        chunk_tokens < 0 || (T > 0 && chunk_tokens < 1) ||
        !grid_fits(route_topk_blocks(T, E), kRouteThreads))
        return MOE_ERR_SHAPE;
    if (chunk_tokens > T)
        chunk_tokens = T;  // one chunk
    if (moe::layout_chunks(T, chunk_tokens) > 65535)  // grid y dimension
        return MOE_ERR_SHAPE;
    need = moe::route_layout_workspace_bytes(T, chunk_tokens, E, k);
    return MOE_OK;
}

// Array arguments of the fused route + layout.
int route_layout_pointers(int64_t T, const float *logits, const int32_t *chunk_capacity,
                          const int32_t *topk_idx, const float *topk_w,
                          const int32_t *expert_counts, const int32_t *expert_offsets,
                          const int32_t *rank_counts, const int32_t *rank_offsets,
                          const int32_t *pos, const int32_t *row_src)
{
    if (!expert_counts || !expert_offsets || !rank_counts || !rank_offsets)
        return MOE_ERR_NULL;
    if (T > 0 && (!logits || !topk_idx || !topk_w || !pos || !row_src))
        return MOE_ERR_NULL;
    if (!aligned(logits, 4) || !aligned(topk_idx, 4) || !aligned(topk_w, 4) ||
        !aligned(expert_counts, 4) || !aligned(expert_offsets, 4) || !aligned(rank_counts, 4) ||
        !aligned(rank_offsets, 4) || !aligned(pos, 4) || !aligned(row_src, 4) ||
        !aligned(chunk_capacity, 4))
        return MOE_ERR_ALIGN;
    return MOE_OK;
}

}  // namespace

extern "C" {

int moe_route_layout_chunks(const float *logits, int64_t T, int64_t chunk_tokens, int E, int k,
                            int R, int capacity, const int32_t *chunk_capacity, int32_t *topk_idx,
                            float *topk_w, int32_t *expert_counts, int32_t *expert_offsets,
                            int32_t *rank_counts, int32_t *rank_offsets, int32_t *pos,
                            int32_t *row_src, void *workspace, size_t *workspace_bytes,
                            hipStream_t stream)
{
    if (!workspace_bytes)
        return MOE_ERR_NULL;
    size_t need = 0;
    int s = route_layout_sizes(T, chunk_tokens, E, k, R, need);
    if (s != MOE_OK)
        return s;
    if (!workspace) {
        *workspace_bytes = need;
        return MOE_OK;
    }
    if (*workspace_bytes < need)
        return MOE_ERR_WORKSPACE;
    s = route_layout_pointers(T, logits, chunk_capacity, topk_idx, topk_w, expert_counts,
                              expert_offsets, rank_counts, rank_offsets, pos, row_src);
    if (s != MOE_OK)
        return s;
    if (!aligned(workspace, 256))
        return MOE_ERR_ALIGN;
    return hip_status(moe::launch_route_layout(logits, T, chunk_tokens, E, k, R, chunk_capacity,
                                               capacity, topk_idx, topk_w, expert_counts,
                                               expert_offsets, rank_counts, rank_offsets, pos,
                                               row_src, workspace, stream));
}

int moe_route_layout_chunks_noalloc(const float *logits, int64_t T, int64_t chunk_tokens, int E,
                                    int k, int R, int capacity, const int32_t *chunk_capacity,
                                    int32_t *topk_idx, float *topk_w, int32_t *expert_counts,
                                    int32_t *expert_offsets, int32_t *rank_counts,
                                    int32_t *rank_offsets, int32_t *pos, int32_t *row_src,
                                    hipStream_t stream)
{
    size_t need = 0;
    int s = route_layout_sizes(T, chunk_tokens, E, k, R, need);
    if (s != MOE_OK)
        return s;
    s = route_layout_pointers(T, logits, chunk_capacity, topk_idx, topk_w, expert_counts,
                              expert_offsets, rank_counts, rank_offsets, pos, row_src);
    if (s != MOE_OK)
        return s;
    if (need > MOE_NOALLOC_SCRATCH_BYTES)
        return MOE_ERR_SCRATCH;
    void *scratch = nullptr;  // the stream's device's copy of the static buffer
    if (moe::static_scratch(stream, &scratch) != hipSuccess)
        return MOE_ERR_HIP;
    return hip_status(moe::launch_route_layout(logits, T, chunk_tokens, E, k, R, chunk_capacity,
                                               capacity, topk_idx, topk_w, expert_counts,
                                               expert_offsets, rank_counts, rank_offsets, pos,
                                               row_src, scratch, stream));
}

int moe_dispatch_pack(const void *x_bf16, int64_t T, int H, int k, const int32_t *pos,
                      int quant_flags, void *send, float *send_scales, hipStream_t stream)
{
    const int quant = quant_flags & ~MOE_PACK_STREAM;
    const bool stream_stores = (quant_flags & MOE_PACK_STREAM) != 0;
    int s = check_rows(T, H, k, quant);
    if (s != MOE_OK)
        return s;
    if (!grid_fits(T, token_threads(H, quant)))
        return MOE_ERR_SHAPE;
    if (T == 0)
        return MOE_OK;
    if (!x_bf16 || !pos || !send)
        return MOE_ERR_NULL;
    if (!aligned(x_bf16, 16) || !aligned(send, 16) || !aligned(pos, 4))
        return MOE_ERR_ALIGN;
    if ((s = check_scales(send_scales, quant)) != MOE_OK)
        return s;
    return hip_status(moe::launch_dispatch_pack(x_bf16, T, H, k, pos, quant, stream_stores, send,
                                                send_scales, stream));
}

int moe_combine(const void *recv, const float *recv_scales, int quant, const int32_t *pos,
                const float *topk_w, int64_t T, int H, int k, void *out_bf16, hipStream_t stream)
{
    int s = check_rows(T, H, k, quant);
    if (s != MOE_OK)
        return s;
    if (!grid_fits(T, token_threads(H, quant)))
        return MOE_ERR_SHAPE;
    if (T == 0)
        return MOE_OK;
    if (!recv || !pos || !topk_w || !out_bf16)
        return MOE_ERR_NULL;
    if (!aligned(recv, 16) || !aligned(out_bf16, 16) || !aligned(pos, 4) || !aligned(topk_w, 4))
        return MOE_ERR_ALIGN;
    if ((s = check_scales(recv_scales, quant)) != MOE_OK)
        return s;
    return hip_status(
        moe::launch_combine(recv, recv_scales, quant, pos, topk_w, T, H, k, out_bf16, stream));
}

int moe_combine_pack(const void *recv, const float *recv_scales, const int32_t *pos_c,
                     const float *topk_w, int64_t Tc, void *out_bf16, const void *x_bf16,
                     const int32_t *pos_p, int64_t Tp, void *send, float *send_scales, int H,
                     int k, int quant_flags, hipStream_t stream)
{
    const int quant = quant_flags & ~MOE_PACK_STREAM;
    const bool stream_stores = (quant_flags & MOE_PACK_STREAM) != 0;
    int s = check_rows(Tc, H, k, quant);
    if (s == MOE_OK)
        s = check_rows(Tp, H, k, quant);
    if (s != MOE_OK)
        return s;
    if (Tc + Tp >= kMaxSlots || !grid_fits(Tc + Tp, token_threads(H, quant)))
        return MOE_ERR_SHAPE;
    if (Tc > 0) {
        if (!recv || !pos_c || !topk_w || !out_bf16)
            return MOE_ERR_NULL;
        if (!aligned(recv, 16) || !aligned(out_bf16, 16) || !aligned(pos_c, 4) ||
            !aligned(topk_w, 4))
            return MOE_ERR_ALIGN;
        if ((s = check_scales(recv_scales, quant)) != MOE_OK)
            return s;
    }
    if (Tp > 0) {
        if (!x_bf16 || !pos_p || !send)
            return MOE_ERR_NULL;
        if (!aligned(x_bf16, 16) || !aligned(send, 16) || !aligned(pos_p, 4))
            return MOE_ERR_ALIGN;
        if ((s = check_scales(send_scales, quant)) != MOE_OK)
            return s;
    }
    if (Tc > 0 && Tp > 0) {
        // The halves run concurrently: what the pack writes must not meet
        // anything the combine touches, nor the combine's output anything the
        // pack reads.  Row buffers are taken at their largest extent (every
        // slot kept: Tc*k and Tp*k rows).
        const int64_t rb = moe_row_bytes(H, quant);
        const bool q = quant != MOE_QUANT_BF16;
        const Extent send_e{send, Tp * k * rb}, sscale_e{q ? send_scales : nullptr, Tp * k * 4};
        const Extent out_e{out_bf16, Tc * H * 2};
        const Extent comb[] = {{recv, Tc * k * rb}, {q ? recv_scales : nullptr, Tc * k * 4},
                               out_e, {pos_c, Tc * k * 4}, {topk_w, Tc * k * 4}};
        for (const Extent &c : comb)
            if (overlap(send_e, c) || overlap(sscale_e, c))
                return MOE_ERR_ALIAS;
        if (overlap(out_e, {x_bf16, Tp * H * 2}) || overlap(out_e, {pos_p, Tp * k * 4}))
            return MOE_ERR_ALIAS;
    }
    return hip_status(moe::launch_combine_pack(recv, recv_scales, pos_c, topk_w, Tc, out_bf16,
                                               x_bf16, pos_p, Tp, send, send_scales, H, k, quant,
                                               stream_stores, stream));
}

int moe_recv_layout(const int32_t *src_offsets, int E, int R, int64_t max_rows,
                    int32_t *recv_offsets, int32_t *group_offsets, int32_t *group_seg,
                    int32_t *group_pos, int32_t *group_src, hipStream_t stream)
{
    if (check_er(E, R) != MOE_OK || max_rows < 0 || max_rows >= kMaxSlots)
        return MOE_ERR_SHAPE;
    if (!src_offsets || !recv_offsets || !group_offsets || !group_seg)
        return MOE_ERR_NULL;
    if (max_rows > 0 && (!group_pos || !group_src))
        return MOE_ERR_NULL;
    if (!aligned(src_offsets, 4) || !aligned(recv_offsets, 4) || !aligned(group_offsets, 4) ||
        !aligned(group_seg, 4) || !aligned(group_pos, 4) || !aligned(group_src, 4))
        return MOE_ERR_ALIGN;
    return hip_status(moe::launch_recv_layout(src_offsets, E, R, max_rows, recv_offsets,
                                              group_offsets, group_seg, group_pos, group_src,
                                              stream));
}

static int gather_rows(const void *in, const float *in_scales, void *out, float *out_scales,
                       int64_t max_rows, int H, int quant, const int32_t *map, hipStream_t stream)
{
    if (max_rows < 0 || max_rows >= kMaxSlots || check_rows(0, H, 1, quant) != MOE_OK ||
        !grid_fits(max_rows, row_tiling(static_cast<int>(moe_row_bytes(H, quant) / 16)).threads))
        return MOE_ERR_SHAPE;
    if (max_rows == 0)
        return MOE_OK;
    if (!in || !out || !map)
        return MOE_ERR_NULL;
    if (!aligned(in, 16) || !aligned(out, 16) || !aligned(map, 4))
        return MOE_ERR_ALIGN;
    int s = check_scales(in_scales, quant);
    if (s == MOE_OK)
        s = check_scales(out_scales, quant);
    if (s != MOE_OK)
        return s;
    return hip_status(
        moe::launch_gather_rows(in, in_scales, out, out_scales, max_rows, H, quant, map, stream));
}

int moe_recv_regroup(const void *recv, const float *recv_scales, int64_t max_rows, int H,
                     int quant, const int32_t *group_src, void *grouped, float *grouped_scales,
                     hipStream_t stream)
{
    return gather_rows(recv, recv_scales, grouped, grouped_scales, max_rows, H, quant, group_src,
                       stream);
}

int moe_recv_ungroup(const void *grouped, const float *grouped_scales, int64_t max_rows, int H,
                     int quant, const int32_t *group_pos, void *recv, float *recv_scales,
                     hipStream_t stream)
{
    return gather_rows(grouped, grouped_scales, recv, recv_scales, max_rows, H, quant, group_pos,
                       stream);
}

int moe_balance_loss(const float *logits, const int32_t *topk_idx, const uint8_t *token_mask,
                     int64_t T, int64_t seg_tokens, int E, int k, float *loss,
                     int32_t *expert_counts, float *prob_sums, int32_t *seg_live,
                     void *workspace, size_t *workspace_bytes, hipStream_t stream)
{
    if (!workspace_bytes)
        return MOE_ERR_NULL;
    if (check_segments(T, seg_tokens, E, k) != MOE_OK)
        return MOE_ERR_SHAPE;
    const size_t need = moe::balance_workspace_bytes(T, seg_tokens, E);
    if (!workspace) {
        *workspace_bytes = need;
        return MOE_OK;
    }
    if (*workspace_bytes < need)
        return MOE_ERR_WORKSPACE;
    if (!loss || !expert_counts || !prob_sums || !seg_live || (T > 0 && (!logits || !topk_idx)))
        return MOE_ERR_NULL;
    if (!aligned(logits, 4) || !aligned(topk_idx, 4) || !aligned(loss, 4) ||
        !aligned(expert_counts, 4) || !aligned(prob_sums, 4) || !aligned(seg_live, 4) ||
        !aligned(workspace, 256))
        return MOE_ERR_ALIGN;
    return hip_status(moe::launch_balance_loss(logits, topk_idx, token_mask, T, seg_tokens, E, k,
                                               loss, expert_counts, prob_sums, seg_live, workspace,
                                               stream));
}

int moe_route_grad(const float *logits, const int32_t *topk_idx, const float *topk_w,
                   const float *d_topk_w, const uint8_t *token_mask, const float *d_loss,
                   const int32_t *expert_counts, const int32_t *seg_live, int64_t T,
                   int64_t seg_tokens, int E, int k, float *d_logits, hipStream_t stream)
{
    const bool masked_gates = k >= 0 && (k & MOE_ROUTE_MASKED_GATES) != 0;
    if (masked_gates)
        k &= ~MOE_ROUTE_MASKED_GATES;
    if (check_segments(T, seg_tokens, E, k) != MOE_OK ||
        !grid_fits(route_grad_blocks(seg_tokens, E), kRouteThreads))
        return MOE_ERR_SHAPE;
    if (T == 0)
        return MOE_OK;
    if (!d_logits || (!d_topk_w && !d_loss) || (d_topk_w && (!topk_idx || !topk_w)) ||
        (d_loss && (!logits || !expert_counts || !seg_live)))
        return MOE_ERR_NULL;
    if (!aligned(logits, 4) || !aligned(topk_idx, 4) || !aligned(topk_w, 4) ||
        !aligned(d_topk_w, 4) || !aligned(d_loss, 4) || !aligned(expert_counts, 4) ||
        !aligned(seg_live, 4) || !aligned(d_logits, 4))
        return MOE_ERR_ALIGN;
    return hip_status(moe::launch_route_grad(logits, topk_idx, topk_w, d_topk_w, token_mask, d_loss,
                                             expert_counts, seg_live, T, seg_tokens, E, k,
                                             masked_gates, d_logits, stream));
}

int moe_combine_grad(const void *d_out_bf16, const void *recv, const float *recv_scales, int quant,
                     const int32_t *pos, const float *topk_w, int64_t T, int H, int k,
                     void *d_recv, float *d_topk_w, hipStream_t stream)
{
    int s = check_rows(T, H, k, quant);
    if (s != MOE_OK)
        return s;
    if (!grid_fits(T, token_threads(H, MOE_QUANT_BF16)))
        return MOE_ERR_SHAPE;
    if (T == 0)
        return MOE_OK;
    if (!d_out_bf16 || !pos || !topk_w || (!d_recv && !d_topk_w) || (d_topk_w && !recv))
        return MOE_ERR_NULL;
    if (!aligned(d_out_bf16, 16) || !aligned(pos, 4) || !aligned(topk_w, 4) ||
        !aligned(d_recv, 16) || !aligned(d_topk_w, 4))
        return MOE_ERR_ALIGN;
    if (d_topk_w) {
        if (!aligned(recv, 16))
            return MOE_ERR_ALIGN;
        if ((s = check_scales(recv_scales, quant)) != MOE_OK)
            return s;
    }
    if (d_recv && (d_recv == d_out_bf16 || (d_topk_w && d_recv == recv)))
        return MOE_ERR_ALIAS;
    return hip_status(moe::launch_combine_grad(d_out_bf16, recv, recv_scales, quant, pos, topk_w, T,
                                               H, k, d_recv, d_topk_w, stream));
}

int moe_expert_matmul(const void *x, const int32_t *offsets, const void *w, const float *bias,
                      int act, const void *residual, int E, int64_t max_rows, int K, int N,
                      void *out, void *preact, void *workspace, size_t *workspace_bytes,
                      hipStream_t stream)
{
    if (check_product(E, max_rows, K, N, MOE_MAX_HIDDEN) != MOE_OK || !known_act(act) ||
        !product_tiles_fit(max_row_tiles(max_rows, E, 256), act == MOE_ACT_SWIGLU ? 2 * N : N))
        return MOE_ERR_SHAPE;
    const size_t need = moe::forward_parts(act, E, max_rows, K, N).bytes;
    if (!workspace && workspace_bytes) {
        *workspace_bytes = need;
        return MOE_OK;
    }
    if (max_rows == 0)
        return MOE_OK;
    if (workspace && (!workspace_bytes || *workspace_bytes < need))
        return MOE_ERR_WORKSPACE;
    if (!x || !offsets || !w || !out)
        return MOE_ERR_NULL;
    if (!aligned(x, 16) || !aligned(offsets, 4) || !aligned(w, 16) || !aligned(bias, 16) ||
        !aligned(residual, 16) || !aligned(out, 16) || !aligned(preact, 16) ||
        !aligned(workspace, 256))
        return MOE_ERR_ALIGN;
    if (out == x || out == w || out == preact ||
        (preact && (preact == x || preact == w || preact == residual)))
        return MOE_ERR_ALIAS;
    return hip_status(moe::launch_expert_matmul(x, offsets, w, bias, act, residual, E, max_rows, K,
                                                N, out, preact, workspace, stream));
}

int moe_expert_matmul_dx(const void *dy, const int32_t *offsets, const void *w, int act,
                         const void *preact, int E, int64_t max_rows, int K, int N, void *dx,
                         void *workspace, size_t *workspace_bytes, hipStream_t stream)
{
    if (check_product(E, max_rows, K, N, 2 * MOE_MAX_HIDDEN) != MOE_OK || !known_act(act) ||
        !product_tiles_fit(max_row_tiles(max_rows, E, 256), K))
        return MOE_ERR_SHAPE;
    const size_t need = moe::row_parts(E, max_rows, N, K, 128).bytes;
    if (!workspace && workspace_bytes) {
        *workspace_bytes = need;
        return MOE_OK;
    }
    if (max_rows == 0)
        return MOE_OK;
    if (workspace && (!workspace_bytes || *workspace_bytes < need))
        return MOE_ERR_WORKSPACE;
    if (!dy || !offsets || !w || !dx || (act != MOE_ACT_NONE && !preact))
        return MOE_ERR_NULL;
    if (!aligned(dy, 16) || !aligned(offsets, 4) || !aligned(w, 16) || !aligned(preact, 16) ||
        !aligned(dx, 16) || !aligned(workspace, 256))
        return MOE_ERR_ALIGN;
    if (dx == dy || dx == w)
        return MOE_ERR_ALIAS;
    return hip_status(
        moe::launch_expert_matmul_dx(dy, offsets, w, act, preact, E, max_rows, K, N, dx,
                                     workspace, stream));
}

int moe_expert_matmul_dw(const void *dy, const void *x, const int32_t *offsets, int E,
                         int64_t max_rows, int K, int N, int flags, void *dw, float *dbias,
                         void *workspace, size_t *workspace_bytes, hipStream_t stream)
{
    if (check_product(E, max_rows, K, N, 2 * MOE_MAX_HIDDEN) != MOE_OK ||
        (flags != MOE_GRAD_FP32 && flags != MOE_GRAD_BF16 &&
         flags != (MOE_GRAD_FP32 | MOE_GRAD_ACCUMULATE)))
        return MOE_ERR_SHAPE;
    const size_t need = moe::dw_parts(E, max_rows, K, N).bytes;
    if (!workspace && workspace_bytes) {
        *workspace_bytes = need;
        return MOE_OK;
    }
    if (workspace && (!workspace_bytes || *workspace_bytes < need))
        return MOE_ERR_WORKSPACE;
    if (!offsets || !dw || (max_rows > 0 && (!dy || !x)))
        return MOE_ERR_NULL;
    if (!aligned(dy, 16) || !aligned(x, 16) || !aligned(offsets, 4) || !aligned(dw, 16) ||
        !aligned(dbias, 16) || !aligned(workspace, 256))
        return MOE_ERR_ALIGN;
    if (dw == dy || dw == x)
        return MOE_ERR_ALIAS;
    return hip_status(
        moe::launch_expert_matmul_dw(dy, x, offsets, E, max_rows, K, N, flags, dw, dbias, workspace,
                                     stream));
}

int moe_add_norm(const void *x, const void *residual, const float *weight, float eps, int64_t T, int H,
                 void *sum, void *y, int block, void *codes, float *scales, hipStream_t stream)
{
    if (check_norm(T, H, eps) != MOE_OK || (codes && block != MOE_BLOCK_ROW && block != MOE_BLOCK_128))
        return MOE_ERR_SHAPE;
    if (T == 0)
        return MOE_OK;
    if (!x || (!y && !codes) || (codes && !scales))
        return MOE_ERR_NULL;
    if (!aligned(x, 16) || !aligned(residual, 16) || !aligned(weight, 16) || !aligned(sum, 16) || !aligned(y, 16) ||
        !aligned(codes, 16) || (codes && !aligned(scales, 4)))
        return MOE_ERR_ALIGN;
    if (y && y == sum)
        return MOE_ERR_ALIAS;
    if (codes && (codes == x || codes == residual || codes == sum || codes == y))
        return MOE_ERR_ALIAS;
    return hip_status(moe::launch_add_norm(x, residual, weight, eps, T, H, sum, y, block == MOE_BLOCK_128, codes,
                                           scales, stream));
}

int moe_add_norm_grad(const void *d_y, const void *d_sum, const void *sum, const float *weight, float eps, int64_t T,
                      int H, void *d_x, float *d_weight, int accumulate, void *workspace, size_t *workspace_bytes,
                      hipStream_t stream)
{
    if (check_norm(T, H, eps) != MOE_OK || (accumulate != 0 && accumulate != 1))
        return MOE_ERR_SHAPE;
    const size_t need = moe::norm_grad_workspace_bytes(T, H);
    if (!workspace && workspace_bytes) {
        *workspace_bytes = need;
        return MOE_OK;
    }
    if (d_weight && (!workspace_bytes || *workspace_bytes < need) && T > 0)
        return MOE_ERR_WORKSPACE;
    if (T == 0 && (!d_weight || accumulate))
        return MOE_OK;
    if (T > 0 && (!d_y || !sum || !d_x))
        return MOE_ERR_NULL;
    if (!aligned(d_y, 16) || !aligned(d_sum, 16) || !aligned(sum, 16) || !aligned(weight, 16) || !aligned(d_x, 16) ||
        !aligned(d_weight, 16) || !aligned(workspace, 256))
        return MOE_ERR_ALIGN;
    return hip_status(moe::launch_add_norm_grad(d_y, d_sum, sum, weight, eps, T, H, d_x, d_weight, accumulate != 0,
                                                workspace, stream));
}

int moe_quant_rows(const void *x, const int32_t *offsets, int E, int64_t max_rows, int H, int halves, void *codes,
                   float *scales, hipStream_t stream)
{
    if ((halves != 1 && halves != 2) || H < 16 * halves || H > halves * MOE_MAX_HIDDEN || H % (16 * halves) != 0 ||
        max_rows < 0 || max_rows > kMaxProductRows || (offsets && (E < 1 || E > MOE_MAX_EXPERTS)))
        return MOE_ERR_SHAPE;
    if (max_rows == 0)
        return MOE_OK;
    if (!x || !codes || !scales)
        return MOE_ERR_NULL;
    if (!aligned(x, 16) || !aligned(offsets, 4) || !aligned(codes, 16) || !aligned(scales, 4))
        return MOE_ERR_ALIGN;
    if (codes == x)
        return MOE_ERR_ALIAS;
    return hip_status(moe::launch_quant_rows(x, offsets, E, max_rows, H / halves, halves, codes, scales, stream));
}

int moe_quant_weights(const void *w, int E, int N, int K, int halves, void *codes, float *scales, void *codes_t,
                      float *scales_t, hipStream_t stream)
{
    if ((halves != 1 && halves != 2) || check_product(E, 0, K, N, MOE_MAX_HIDDEN) != MOE_OK ||
        !grid_fits(moe::quant_weights_groups(E, N, K, halves), kRouteThreads))
        return MOE_ERR_SHAPE;
    if (!w || !codes || !scales || (codes_t != nullptr) != (scales_t != nullptr))
        return MOE_ERR_NULL;
    if (!aligned(w, 16) || !aligned(codes, 16) || !aligned(scales, 4) || !aligned(codes_t, 16) || !aligned(scales_t, 4))
        return MOE_ERR_ALIGN;
    if (codes == w || codes_t == w || codes_t == codes || scales_t == scales)
        return MOE_ERR_ALIAS;
    return hip_status(moe::launch_quant_weights(w, E, N, K, halves, codes, scales, codes_t, scales_t, stream));
}

int moe_expert_matmul_fp8(const void *x, const float *x_scales, int x_scale_cols, const int32_t *offsets,
                          const void *w, const float *w_scales, const float *bias, int act, const void *residual,
                          int E, int64_t max_rows, int K, int N, void *out, void *codes, float *scales, void *preact,
                          void *workspace, size_t *workspace_bytes, hipStream_t stream)
{
    if (check_product(E, max_rows, K, N, MOE_MAX_HIDDEN) != MOE_OK || !known_act(act) ||
        !fp8_tiles_fit(E, max_rows, act == MOE_ACT_SWIGLU ? 2 * N : N) ||
        (x_scale_cols != 1 && x_scale_cols != code_blocks(K)))
        return MOE_ERR_SHAPE;
    const size_t need = moe::expert_fp8_workspace_bytes(act, E, max_rows, K, N);
    if (!workspace && workspace_bytes) {
        *workspace_bytes = need;
        return MOE_OK;
    }
    if (max_rows == 0)
        return MOE_OK;
    if (workspace && (!workspace_bytes || *workspace_bytes < need))
        return MOE_ERR_WORKSPACE;
    if (!x || !x_scales || !offsets || !w || !w_scales || (!out && !codes) || (codes && !scales))
        return MOE_ERR_NULL;
    if (!aligned(x, 16) || !aligned(x_scales, 4) || !aligned(offsets, 4) || !aligned(w, 16) || !aligned(w_scales, 4) ||
        !aligned(bias, 16) || !aligned(residual, 16) || !aligned(out, 16) || !aligned(codes, 16) ||
        (codes && !aligned(scales, 4)) || !aligned(preact, 16) || !aligned(workspace, 256))
        return MOE_ERR_ALIGN;
    const void *made[] = {out, codes, preact}, *taken[] = {x, w};
    for (const void *m : made)
        for (const void *t : taken)
            if (m && m == t)
                return MOE_ERR_ALIAS;
    if ((out && (out == codes || out == preact)) || (codes && (codes == preact || codes == residual)) ||
        (preact && preact == residual) || (codes && (scales == x_scales || scales == w_scales)))
        return MOE_ERR_ALIAS;
    return hip_status(moe::launch_expert_fp8(x, x_scales, x_scale_cols, offsets, w, w_scales, bias, act, residual, E,
                                             max_rows, K, N, out, codes, scales, preact, workspace, stream));
}

int moe_expert_matmul_fp8_dx(const void *dy, const float *dy_scales, const int32_t *offsets, const void *w_t,
                             const float *w_t_scales, int halves, int act, const void *preact, int E,
                             int64_t max_rows, int K, int N, void *dx, void *codes, float *scales, void *workspace,
                             size_t *workspace_bytes, hipStream_t stream)
{
    if ((halves != 1 && halves != 2) || check_product(E, max_rows, K, N, MOE_MAX_HIDDEN) != MOE_OK ||
        !known_act(act) || !fp8_tiles_fit(E, max_rows, K))
        return MOE_ERR_SHAPE;
    const size_t need = moe::expert_fp8_dx_workspace_bytes(halves, act, E, max_rows, K, N);
    if (!workspace && workspace_bytes) {
        *workspace_bytes = need;
        return MOE_OK;
    }
    if (max_rows == 0)
        return MOE_OK;
    if (workspace && (!workspace_bytes || *workspace_bytes < need))
        return MOE_ERR_WORKSPACE;
    if (!dy || !dy_scales || !offsets || !w_t || !w_t_scales || (!dx && !codes) || (codes && !scales) ||
        (act != MOE_ACT_NONE && !preact))
        return MOE_ERR_NULL;
    if (!aligned(dy, 16) || !aligned(dy_scales, 4) || !aligned(offsets, 4) || !aligned(w_t, 16) ||
        !aligned(w_t_scales, 4) || !aligned(preact, 16) || !aligned(dx, 16) || !aligned(codes, 16) ||
        (codes && !aligned(scales, 4)) || !aligned(workspace, 256))
        return MOE_ERR_ALIGN;
    if ((dx && (dx == dy || dx == w_t || dx == codes)) ||
        (codes && (codes == dy || codes == w_t || (act != MOE_ACT_NONE && codes == preact) || scales == dy_scales ||
                   scales == w_t_scales)))
        return MOE_ERR_ALIAS;
    return hip_status(moe::launch_expert_fp8_dx(dy, dy_scales, offsets, w_t, w_t_scales, halves, act, preact, E,
                                                max_rows, K, N, dx, codes, scales, workspace, stream));
}

}  // extern "C"
