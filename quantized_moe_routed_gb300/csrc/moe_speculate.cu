// moe_speculate.cu -- host side of the C ABI declared in include/moe_speculate.h:
// argument validation and launches.  The computation runs in moe_kv_append.cu,
// moe_kv_attend.cu, moe_kv_attend_tc.cu, moe_kv_move.cu and moe_sample.cu.
#include "moe_layer_host.h"

#include <algorithm>

using moe::aligned;
using moe::check_kv;
using moe::fail;
using moe::kv_params;
using moe::launched;

namespace {

constexpr int kMaxSampleRows = 1 << 27;  // blocks of a launch, 8 a row

// A step of trees: parents for each token, no tree too long.
moe_status_t check_tree(const moe_kv_batch *b, const int32_t *parent)
{
    if (b->max_q > MOE_KV_MAX_TREE)
        return fail(MOE_ERR_UNSUPPORTED_SHAPE, "max_q=%d new tokens are more than a tree's %d", b->max_q, MOE_KV_MAX_TREE);
    if (b->B == 0 || b->N == 0) return MOE_OK;
    if (!parent) return fail(MOE_ERR_INVALID_ARG, "null parent pointer");
    if (!aligned(parent, 4)) return fail(MOE_ERR_MISALIGNED, "parent needs 4-byte alignment");
    return MOE_OK;
}

// Whether two arrays of words share memory.
bool overlap(const void *a, size_t na, const void *b, size_t nb)
{
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return x < y + 4 * nb && y < x + 4 * na;
}

// Whether T words at `out` share memory with one of the T rows of logits (between rows they may lie).
bool in_logits(const moe_sample_desc &d, const void *out)
{
    const uint64_t size = d.bf16 ? 2 : 4, T = static_cast<uint64_t>(d.T), row = size * d.V;
    const uint64_t step = size * std::min(static_cast<uint64_t>(d.stride), uint64_t(1) << 56);  // (past any address)
    const uint64_t a = reinterpret_cast<uintptr_t>(out), b = a + 4 * T, base = reinterpret_cast<uintptr_t>(d.logits_dev);
    const uint64_t r = a < base + row ? 0 : (a - base - row) / step + 1;  // the first row that ends behind a
    return r < T && base + r * step < b;
}

// Whether T words at `out` lie in one of the inputs.
bool in_inputs(const moe_sample_desc &d, const void *out)
{
    const size_t T = static_cast<size_t>(d.T);
    for (const void *in : {static_cast<const void *>(d.u_dev), static_cast<const void *>(d.temperature_dev),
                           static_cast<const void *>(d.top_k_dev), static_cast<const void *>(d.top_p_dev),
                           static_cast<const void *>(d.min_p_dev)})
        if (in && overlap(out, T, in, T)) return true;
    return in_logits(d, out);
}

template <typename F>
moe_status_t on_workspace(void *ws, void *stream, const char *what, F launch)
{
    moe::WsTicket tk;
    const moe_status_t st = moe::ws_claim(ws, static_cast<cudaStream_t>(stream), tk);
    if (st != MOE_OK) return st;
    const cudaError_t e = launch(static_cast<cudaStream_t>(stream));
    moe::ws_release(tk, e == cudaSuccess);
    return launched(e, what);
}

}  // namespace

extern "C" {

moe_status_t moe_kv_append_tree(moe_kv_t kv, const void *q_dev, int64_t q_stride, const void *k_dev, int64_t k_stride,
                                const void *v_dev, int64_t v_stride, void *q_out_dev, const moe_kv_batch *batch,
                                const int32_t *parent_dev, void *ws_dev, void *stream)
{
    moe_status_t st = check_kv(kv, batch, ws_dev);
    if (st != MOE_OK || (st = check_tree(batch, parent_dev)) != MOE_OK) return st;
    moe::AppendParams p;
    if ((st = moe::append_params(kv, q_dev, q_stride, k_dev, k_stride, v_dev, v_stride, q_out_dev, batch, ws_dev, &p)) != MOE_OK)
        return st;
    if (batch->B == 0 || batch->N == 0) return MOE_OK;
    p.parent = parent_dev;
    return on_workspace(ws_dev, stream, "append launch", [&](cudaStream_t cs) { return moe::launch_kv_append(p, cs); });
}

moe_status_t moe_kv_attend_tree(moe_kv_t kv, const void *q_dev, int64_t q_stride, float scale, void *o_dev,
                                const moe_kv_batch *batch, const int32_t *parent_dev, void *ws_dev, void *stream)
{
    moe_status_t st = check_kv(kv, batch, ws_dev);
    if (st != MOE_OK || (st = check_tree(batch, parent_dev)) != MOE_OK) return st;
    moe::AttendParams p;
    int tile_rows = 0;
    if ((st = moe::attend_params(kv, q_dev, q_stride, scale, o_dev, batch, ws_dev, &p, &tile_rows)) != MOE_OK) return st;
    if (batch->B == 0 || batch->N == 0) return MOE_OK;
    p.parent = parent_dev;
    return on_workspace(ws_dev, stream, "attention launch",
                        [&](cudaStream_t cs) { return moe::launch_kv_attend(kv, p, tile_rows, cs); });
}

moe_status_t moe_kv_compact(moe_kv_t kv, const int32_t *keep_dev, const int32_t *n_keep_dev, int max_keep,
                            int32_t *kv_len_out_dev, const moe_kv_batch *batch, void *ws_dev, void *stream)
{
    if (!kv || !batch) return fail(MOE_ERR_INVALID_ARG, "null cache or batch");
    moe_kv_batch b = *batch;
    b.N = b.N == 0 ? 1 : b.N;  // (lengths are written where there are no new tokens too)
    b.max_q = 0;
    const moe_status_t st = check_kv(kv, &b, ws_dev);
    if (st != MOE_OK) return st;
    if (max_keep < 0 || max_keep > MOE_KV_MAX_TREE)
        return fail(MOE_ERR_INVALID_ARG, "max_keep=%d outside [0, %d]", max_keep, MOE_KV_MAX_TREE);
    if (b.B == 0) return MOE_OK;
    if ((!keep_dev && max_keep > 0) || !n_keep_dev || !kv_len_out_dev)
        return fail(MOE_ERR_INVALID_ARG, "null keep/n_keep/kv_len_out pointer");
    if (!aligned(keep_dev, 4) || !aligned(n_keep_dev, 4) || !aligned(kv_len_out_dev, 4))
        return fail(MOE_ERR_MISALIGNED, "int32 arrays need 4-byte alignment");
    const size_t B = static_cast<size_t>(b.B);
    if (overlap(kv_len_out_dev, B, b.kv_len_dev, B) || overlap(kv_len_out_dev, B, b.q_off_dev, B + 1) ||
        overlap(kv_len_out_dev, B, n_keep_dev, B) || overlap(kv_len_out_dev, B, keep_dev, B * max_keep) ||
        overlap(kv_len_out_dev, B, b.pages_dev, B * b.max_pages))
        return fail(MOE_ERR_INVALID_ARG, "kv_len_out lies in one of the inputs");
    moe::CompactParams p{kv_params(kv, &b, ws_dev), keep_dev, n_keep_dev, max_keep, kv_len_out_dev};
    p.c.N = batch->N;
    return on_workspace(ws_dev, stream, "compaction launch", [&](cudaStream_t cs) { return moe::launch_kv_compact(p, cs); });
}

moe_status_t moe_kv_fork(moe_kv_t kv, const int32_t *src_dev, const int32_t *fresh_dev, int C, const int32_t *kv_len_dev,
                         const int32_t *pages_dev, int max_pages, int B, int32_t *kv_len_out_dev, int32_t *pages_out_dev,
                         void *ws_dev, void *stream)
{
    if (!kv) return fail(MOE_ERR_INVALID_ARG, "null cache");
    if (C < 0 || C > MOE_KV_MAX_SEQS) return fail(MOE_ERR_INVALID_ARG, "C=%d outside [0, %d]", C, MOE_KV_MAX_SEQS);
    moe_kv_batch b{};
    b.q_off_dev = kv_len_dev;  // (the checks want one; it is not read)
    b.kv_len_dev = kv_len_dev;
    b.pages_dev = pages_dev;
    b.max_pages = max_pages;
    b.B = B;
    b.N = 1;
    const moe_status_t st = check_kv(kv, &b, ws_dev);
    if (st != MOE_OK) return st;
    if (C == 0) return MOE_OK;
    if (B == 0) return fail(MOE_ERR_INVALID_ARG, "C=%d children of no sequence", C);
    if (!src_dev || !fresh_dev || !kv_len_out_dev || !pages_out_dev)
        return fail(MOE_ERR_INVALID_ARG, "null src/fresh/kv_len_out/pages_out pointer");
    if (!aligned(src_dev, 4) || !aligned(fresh_dev, 4) || !aligned(kv_len_out_dev, 4) || !aligned(pages_out_dev, 4))
        return fail(MOE_ERR_MISALIGNED, "int32 arrays need 4-byte alignment");
    const size_t nc = static_cast<size_t>(C), nb = static_cast<size_t>(B), w = static_cast<size_t>(max_pages);
    const int32_t *outs[2] = {kv_len_out_dev, pages_out_dev};
    const size_t len[2] = {nc, nc * w};
    for (int i = 0; i < 2; ++i)
        if (overlap(outs[i], len[i], src_dev, nc) || overlap(outs[i], len[i], fresh_dev, nc) ||
            overlap(outs[i], len[i], kv_len_dev, nb) || overlap(outs[i], len[i], pages_dev, nb * w))
            return fail(MOE_ERR_INVALID_ARG, "an output lies in one of the inputs");
    if (overlap(kv_len_out_dev, nc, pages_out_dev, nc * w)) return fail(MOE_ERR_INVALID_ARG, "the outputs overlap");
    const moe::ForkParams p{kv_params(kv, &b, ws_dev), src_dev, fresh_dev, C, kv_len_out_dev, pages_out_dev};
    return on_workspace(ws_dev, stream, "fork launch", [&](cudaStream_t cs) { return moe::launch_kv_fork(p, cs); });
}

moe_status_t moe_sample(const moe_sample_desc *desc, void *stream)
{
    if (!desc) return fail(MOE_ERR_INVALID_ARG, "null description");
    const moe_sample_desc &d = *desc;
    if (d.T < 0 || d.T > kMaxSampleRows) return fail(MOE_ERR_INVALID_ARG, "T=%d outside [0, %d]", d.T, kMaxSampleRows);
    if (d.V < 1 || d.V > MOE_SAMPLE_MAX_VOCAB)
        return fail(MOE_ERR_UNSUPPORTED_SHAPE, "V=%d outside [1, %d]", d.V, MOE_SAMPLE_MAX_VOCAB);
    if (d.bf16 != 0 && d.bf16 != 1) return fail(MOE_ERR_INVALID_ARG, "bf16=%d is not 0 or 1", d.bf16);
    if (d.stride < d.V) return fail(MOE_ERR_INVALID_ARG, "stride=%lld < V=%d", static_cast<long long>(d.stride), d.V);
    if (d.T == 0) return MOE_OK;
    if (!d.logits_dev || !d.u_dev || !d.token_dev) return fail(MOE_ERR_INVALID_ARG, "null logits, u or token pointer");
    if (!aligned(d.logits_dev, d.bf16 ? 2 : 4)) return fail(MOE_ERR_MISALIGNED, "logits need their element's alignment");
    for (const void *ptr : {static_cast<const void *>(d.u_dev), static_cast<const void *>(d.temperature_dev),
                            static_cast<const void *>(d.top_k_dev), static_cast<const void *>(d.top_p_dev),
                            static_cast<const void *>(d.min_p_dev), static_cast<const void *>(d.token_dev),
                            static_cast<const void *>(d.prob_dev)})
        if (!aligned(ptr, 4)) return fail(MOE_ERR_MISALIGNED, "settings, u, token and prob need 4-byte alignment");
    if (in_inputs(d, d.token_dev) || (d.prob_dev && in_inputs(d, d.prob_dev)))
        return fail(MOE_ERR_INVALID_ARG, "an output lies in one of the inputs");
    const size_t T = static_cast<size_t>(d.T);
    if (d.prob_dev && overlap(d.token_dev, T, d.prob_dev, T)) return fail(MOE_ERR_INVALID_ARG, "the outputs overlap");
    moe::Device dev;
    const moe_status_t st = moe::query_device(-1, &dev);
    if (st != MOE_OK) return st;
    return launched(moe::launch_sample(d, dev.sms, static_cast<cudaStream_t>(stream)), "sampling launch");
}

}  // extern "C"
