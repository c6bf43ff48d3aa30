// moe_layer_host.h -- what the host sides of the layer operators (moe_layer.cu) and of
// those for speculative decoding (moe_speculate.cu) share: the cache handle, the
// device's attributes, checks of a step's arguments.  Not part of the ABI.
#pragma once
#include "moe_layer.h"
#include "moe_host.h"
#include "moe_internal.h"
#include "moe_layer_internal.h"

#include <cmath>

struct moe_kv {
    moe_kv_desc d;
    int device = 0, num_sms = 0, smem_optin = 0;
    long long timeout_ns = 0;
    CUtensorMap tm_k{};
    size_t off_count = 0, off_part = 0, ws_bytes = 0;
};

namespace moe {

// the kernels count tokens and units of a sequence in 32 bits
constexpr int kMaxSeqPages = 1 << 24;
constexpr int kMaxStepRows = 1 << 30;  // new tokens x query heads of a step

struct Device {
    int ordinal, sms, optin;
};

// The device (-1: the current one), which has to be sm_103 (moe_layer.cu).
moe_status_t query_device(int dev, Device *out);

inline moe_status_t launched(cudaError_t e, const char *what)
{
    return e == cudaSuccess ? MOE_OK : fail(MOE_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

// What is queued goes to the current device: it has to be the cache's.
inline moe_status_t check_device(moe_kv_t kv)
{
    int cur = -1;
    const cudaError_t e = cudaGetDevice(&cur);
    if (e != cudaSuccess) return fail(MOE_ERR_CUDA, "cudaGetDevice: %s", cudaGetErrorString(e));
    if (cur != kv->device)
        return fail(MOE_ERR_INVALID_ARG, "current device %d is not the cache's device %d", cur, kv->device);
    return MOE_OK;
}

inline moe_status_t check_kv(moe_kv_t kv, const moe_kv_batch *b, const void *ws)
{
    if (!kv || !b) return fail(MOE_ERR_INVALID_ARG, "null cache or batch");
    if (b->B < 0 || b->B > MOE_KV_MAX_SEQS)
        return fail(MOE_ERR_INVALID_ARG, "B=%d outside [0, %d]", b->B, MOE_KV_MAX_SEQS);
    if (b->N < 0 || b->N > kMaxStepRows / kv->d.q_heads)
        return fail(MOE_ERR_INVALID_ARG, "N=%d outside [0, %d]", b->N, kMaxStepRows / kv->d.q_heads);
    if (b->max_q < 0 || b->max_q > b->N) return fail(MOE_ERR_INVALID_ARG, "max_q=%d outside [0, N=%d]", b->max_q, b->N);
    if (b->max_pages < 1 || b->max_pages > kMaxSeqPages)
        return fail(MOE_ERR_INVALID_ARG, "max_pages=%d outside [1, %d]", b->max_pages, kMaxSeqPages);
    if (b->B == 0 || b->N == 0) return MOE_OK;
    if (!b->q_off_dev || !b->kv_len_dev || !b->pages_dev || !ws)
        return fail(MOE_ERR_INVALID_ARG, "null q_off/kv_len/pages/workspace pointer");
    if (!aligned(b->q_off_dev, 4) || !aligned(b->kv_len_dev, 4) || !aligned(b->pages_dev, 4) || !aligned(ws, 256))
        return fail(MOE_ERR_MISALIGNED, "int32 arrays need 4-byte, the workspace 256-byte alignment");
    return check_device(kv);
}

inline moe_status_t check_rows(const void *ptr, int64_t stride, int64_t row, const char *name)
{
    if (!ptr) return fail(MOE_ERR_INVALID_ARG, "null %s pointer", name);
    if (stride < row) return fail(MOE_ERR_INVALID_ARG, "%s_stride=%lld < %lld elements of a token", name,
                                  static_cast<long long>(stride), static_cast<long long>(row));
    if (!aligned(ptr, 16) || stride % 8)
        return fail(MOE_ERR_MISALIGNED, "%s needs 16-byte alignment and a stride that is a multiple of 8", name);
    return MOE_OK;
}

inline KvParams kv_params(const moe_kv *kv, const moe_kv_batch *b, void *ws)
{
    KvParams c{};
    const moe_kv_desc &d = kv->d;
    c.tm_k = kv->tm_k;
    c.k = d.k_dev, c.v = d.v_dev, c.ks = d.k_scale_dev, c.vs = d.v_scale_dev, c.rope = d.rope_dev;
    c.n_pages = d.n_pages, c.q_heads = d.q_heads, c.kv_heads = d.kv_heads, c.D = d.head_dim;
    c.rot_dim = d.rot_dim, c.rot_inter = d.rot_interleaved, c.rope_positions = d.rope_positions;
    c.q_off = b->q_off_dev, c.kv_len = b->kv_len_dev, c.pages = b->pages_dev;
    c.max_pages = b->max_pages, c.B = b->B, c.N = b->N, c.max_q = b->max_q;
    c.ctrl = static_cast<uint32_t *>(ws);
    return c;
}

// Query rows of a tile of the attention, from the rows of the sequence with the
// most new tokens: up to 16 the kernel of few rows, whose warps share no rows;
// above, the tensor-memory kernel, whose rows come by 128.
inline int attend_tile_rows(long long rows) { return rows <= 8 ? 8 : (rows <= 16 ? 16 : 128); }

// Check an append's tensors and describe it (after check_kv; nothing where there are no new tokens).
inline moe_status_t append_params(const moe_kv *kv, const void *q_dev, int64_t q_stride, const void *k_dev, int64_t k_stride,
                                  const void *v_dev, int64_t v_stride, void *q_out_dev, const moe_kv_batch *batch,
                                  void *ws_dev, AppendParams *out)
{
    moe_status_t st;
    const moe_kv_desc &d = kv->d;
    if (!q_dev != !q_out_dev) return fail(MOE_ERR_INVALID_ARG, "q and q_out come together");
    if (batch->B == 0 || batch->N == 0) return MOE_OK;
    if (q_dev && (st = check_rows(q_dev, q_stride, static_cast<int64_t>(d.q_heads) * d.head_dim, "q")) != MOE_OK) return st;
    if ((st = check_rows(k_dev, k_stride, static_cast<int64_t>(d.kv_heads) * d.head_dim, "k")) != MOE_OK) return st;
    if ((st = check_rows(v_dev, v_stride, static_cast<int64_t>(d.kv_heads) * d.head_dim, "v")) != MOE_OK) return st;
    if (!aligned(q_out_dev, 16)) return fail(MOE_ERR_MISALIGNED, "q_out needs 16-byte alignment");
    *out = AppendParams{kv_params(kv, batch, ws_dev), static_cast<const uint16_t *>(q_dev),
                        static_cast<const uint16_t *>(k_dev), static_cast<const uint16_t *>(v_dev),
                        q_stride, k_stride, v_stride, static_cast<uint16_t *>(q_out_dev)};
    return MOE_OK;
}

// The same for an attention, and the rows of its tiles.
inline moe_status_t attend_params(const moe_kv *kv, const void *q_dev, int64_t q_stride, float scale, void *o_dev,
                                  const moe_kv_batch *batch, void *ws_dev, AttendParams *out, int *rows)
{
    moe_status_t st;
    if (!std::isfinite(scale)) return fail(MOE_ERR_INVALID_ARG, "the softmax scale is not finite");
    if (batch->B == 0 || batch->N == 0) return MOE_OK;
    if ((st = check_rows(q_dev, q_stride, static_cast<int64_t>(kv->d.q_heads) * kv->d.head_dim, "q")) != MOE_OK) return st;
    if (!o_dev) return fail(MOE_ERR_INVALID_ARG, "null o pointer");
    if (!aligned(o_dev, 16)) return fail(MOE_ERR_MISALIGNED, "o needs 16-byte alignment");
    const long long G = kv->d.q_heads / kv->d.kv_heads;
    const int tile_rows = attend_tile_rows(batch->max_q * G);
    // the kernels count the units of a sequence (pages of all its tiles, and up to 16 more a tile) in 32 bits
    if (batch->N * G / tile_rows + 1 > 0x7FFFFFFFLL / kv->d.kv_heads / (batch->max_pages + 16))
        return fail(MOE_ERR_UNSUPPORTED_SHAPE, "N=%d new tokens over max_pages=%d pages are too many for one step", batch->N,
                    batch->max_pages);
    uint8_t *ws = static_cast<uint8_t *>(ws_dev);
    *out = AttendParams{kv_params(kv, batch, ws_dev), static_cast<const uint16_t *>(q_dev), static_cast<uint16_t *>(o_dev),
                        q_stride, scale * 1.44269504088896341f, reinterpret_cast<uint32_t *>(ws + kv->off_count),
                        reinterpret_cast<float *>(ws + kv->off_part), kv->timeout_ns};
    *rows = tile_rows;
    return MOE_OK;
}

inline cudaError_t launch_kv_attend(const moe_kv *kv, const AttendParams &p, int tile_rows, cudaStream_t st)
{
    return tile_rows <= 16 ? launch_kv_attend_rows(p, tile_rows, kv->num_sms, kv->smem_optin, st)
                           : launch_kv_attend_tc(p, kv->num_sms, st);
}

}  // namespace moe
