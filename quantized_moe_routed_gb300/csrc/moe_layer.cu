// moe_layer.cu -- host side of the C ABI declared in include/moe_layer.h:
// argument validation, the cache handle, its workspace, launches.  The
// computation runs in moe_norm.cu, moe_linear.cu, moe_linear_tc.cu,
// moe_kv_append.cu, moe_kv_attend.cu and moe_kv_attend_tc.cu.
#include "moe_layer.h"
#include "moe_host.h"
#include "moe_internal.h"
#include "moe_layer_internal.h"

#include <cmath>
#include <mutex>
#include <new>

using moe::aligned;
using moe::fail;

struct moe_kv {
    moe_kv_desc d;
    int device = 0, num_sms = 0, smem_optin = 0;
    long long timeout_ns = 0;
    CUtensorMap tm_k{};
    size_t off_count = 0, off_part = 0, ws_bytes = 0;
};

namespace {

constexpr int kMaxNormH = 16384;
constexpr int kMaxLinearK = 1 << 22;  // the kernel counts bytes inside 512 rows in 32 bits
// the kernels count tokens and units of a sequence in 32 bits
constexpr int kMaxSeqPages = 1 << 24;
constexpr int kMaxStepRows = 1 << 30;  // new tokens x query heads of a step

struct Device {
    int ordinal, sms, optin;
};

// The device (-1: the current one), which has to be sm_103.  Attributes do not
// change, so each device is asked once.
moe_status_t query_device(int dev, Device *out)
{
    constexpr int kKnown = 16;
    static std::mutex mu;
    static Device known[kKnown];
    static bool have[kKnown];
    cudaError_t e = cudaSuccess;
    if (dev < 0) e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return fail(MOE_ERR_CUDA, "cudaGetDevice: %s", cudaGetErrorString(e));
    std::lock_guard<std::mutex> lk(mu);
    if (dev < kKnown && have[dev]) {
        *out = known[dev];
        return MOE_OK;
    }
    int major = 0, minor = 0;
    out->ordinal = dev;
    if ((e = cudaDeviceGetAttribute(&out->sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess ||
        (e = cudaDeviceGetAttribute(&out->optin, cudaDevAttrMaxSharedMemoryPerBlockOptin, dev)) != cudaSuccess ||
        (e = cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev)) != cudaSuccess ||
        (e = cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev)) != cudaSuccess)
        return fail(MOE_ERR_CUDA, "device query: %s", cudaGetErrorString(e));
    if (major != 10 || minor != 3)
        return fail(MOE_ERR_UNSUPPORTED_SHAPE, "device %d is sm_%d%d; this library is built for sm_103a only", dev,
                    major, minor);
    if (dev < kKnown) {
        known[dev] = *out;
        have[dev] = true;
    }
    return MOE_OK;
}

moe_status_t launched(cudaError_t e, const char *what)
{
    return e == cudaSuccess ? MOE_OK : fail(MOE_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

// What is queued goes to the current device: it has to be the cache's.
moe_status_t check_device(moe_kv_t kv)
{
    int cur = -1;
    const cudaError_t e = cudaGetDevice(&cur);
    if (e != cudaSuccess) return fail(MOE_ERR_CUDA, "cudaGetDevice: %s", cudaGetErrorString(e));
    if (cur != kv->device)
        return fail(MOE_ERR_INVALID_ARG, "current device %d is not the cache's device %d", cur, kv->device);
    return MOE_OK;
}

moe_status_t check_kv(moe_kv_t kv, const moe_kv_batch *b, const void *ws)
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

moe_status_t check_rows(const void *ptr, int64_t stride, int64_t row, const char *name)
{
    if (!ptr) return fail(MOE_ERR_INVALID_ARG, "null %s pointer", name);
    if (stride < row) return fail(MOE_ERR_INVALID_ARG, "%s_stride=%lld < %lld elements of a token", name,
                                  static_cast<long long>(stride), static_cast<long long>(row));
    if (!aligned(ptr, 16) || stride % 8)
        return fail(MOE_ERR_MISALIGNED, "%s needs 16-byte alignment and a stride that is a multiple of 8", name);
    return MOE_OK;
}

moe::KvParams kv_params(const moe_kv *kv, const moe_kv_batch *b, void *ws)
{
    moe::KvParams c{};
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
int attend_tile_rows(long long rows) { return rows <= 8 ? 8 : (rows <= 16 ? 16 : 128); }

// Whether the tensor-core kernel takes a product: where its loads may go, and where
// the rows and the length give it enough work past what it takes to begin (every
// block reads all of x first).  Measured, it against the others, at K = 4096: 8
// tokens, 64 rows an SM 14.7 / 12.4 us, 96 rows 15.6 / 16.5, 512 rows 41 / 44; 24
// tokens, 64 rows 20.6 / 20.2, 128 rows 21 / 28, 512 rows 47 / 76; 64 tokens, 64
// rows 47 / 55.  At K = 1024: 8 tokens, 128 rows 9.1 / 7.5, 256 rows 10.5 / 10.3;
// 24 tokens, 128 rows 10.4 / 10.7.
bool linear_on_tensor_cores(const moe::LinearParams &p, int sms)
{
    const int rows = p.N / sms;
    return p.K % 256 == 0 && aligned(p.s, 16) && rows >= 64 &&
           static_cast<long long>(rows) * p.K >= (p.T > 16 ? 128 : 320) * 1024;
}

}  // namespace

extern "C" {

moe_status_t moe_norm(const void *x_dev, int x_f32, int64_t x_stride, const void *r_dev, void *r_out_dev,
                      const void *w_dev, float eps, void *y_dev, uint8_t *q_dev, float *q_scale_dev, int T, int H,
                      void *stream)
{
    if (T < 0) return fail(MOE_ERR_INVALID_ARG, "T=%d is negative", T);
    if (H < 8 || H > kMaxNormH || H % 8)
        return fail(MOE_ERR_UNSUPPORTED_SHAPE, "H=%d is not a multiple of 8 up to %d", H, kMaxNormH);
    if (q_dev && H % 128) return fail(MOE_ERR_UNSUPPORTED_SHAPE, "an 8-bit output needs H=%d to be a multiple of 128", H);
    if (x_f32 != 0 && x_f32 != 1) return fail(MOE_ERR_INVALID_ARG, "x_f32=%d is not 0 or 1", x_f32);
    if (!(eps >= 0.f) || !std::isfinite(eps)) return fail(MOE_ERR_INVALID_ARG, "eps is not a non-negative number");
    if (x_stride < H) return fail(MOE_ERR_INVALID_ARG, "x_stride=%lld < H=%d", static_cast<long long>(x_stride), H);
    if (T == 0) return MOE_OK;
    if (!y_dev && !q_dev) return fail(MOE_ERR_INVALID_ARG, "neither a bf16 nor an 8-bit output");
    if (!q_dev != !q_scale_dev) return fail(MOE_ERR_INVALID_ARG, "q and q_scale come together");
    if (!x_dev || !w_dev) return fail(MOE_ERR_INVALID_ARG, "null x or w pointer");
    for (const void *ptr : {x_dev, r_dev, static_cast<const void *>(r_out_dev), w_dev, static_cast<const void *>(y_dev),
                            static_cast<const void *>(q_dev)})
        if (!aligned(ptr, 16)) return fail(MOE_ERR_MISALIGNED, "x, r, r_out, w, y and q need 16-byte alignment");
    if (!aligned(q_scale_dev, 4) || x_stride % (x_f32 ? 4 : 8))
        return fail(MOE_ERR_MISALIGNED, "q_scale needs 4-byte alignment, rows of x 16-byte");
    Device dev;
    const moe_status_t st = query_device(-1, &dev);
    if (st != MOE_OK) return st;
    const moe::NormParams p{x_dev, x_stride, static_cast<const uint16_t *>(r_dev), static_cast<uint16_t *>(r_out_dev),
                            static_cast<const uint16_t *>(w_dev), static_cast<uint16_t *>(y_dev), q_dev, q_scale_dev,
                            eps, T, H, x_f32};
    return launched(moe::launch_norm(p, static_cast<cudaStream_t>(stream)), "norm launch");
}

moe_status_t moe_linear(const uint8_t *q_dev, const uint8_t *s_dev, const float *ts_dev, int N, int K,
                        const void *x_dev, int64_t x_stride, void *y_dev, int y_bf16, int T, void *stream)
{
    if (T < 0) return fail(MOE_ERR_INVALID_ARG, "T=%d is negative", T);
    if (N < 1 || K < 32 || K % 32 || K > kMaxLinearK)
        return fail(MOE_ERR_UNSUPPORTED_SHAPE, "N=%d must be positive and K=%d a multiple of 32 up to %d", N, K, kMaxLinearK);
    if (T > 65535 * moe::kLinearMaxT) return fail(MOE_ERR_INVALID_ARG, "T=%d is more than a launch takes", T);
    if (y_bf16 != 0 && y_bf16 != 1) return fail(MOE_ERR_INVALID_ARG, "y_bf16=%d is not 0 or 1", y_bf16);
    if (x_stride < K) return fail(MOE_ERR_INVALID_ARG, "x_stride=%lld < K=%d", static_cast<long long>(x_stride), K);
    if (T == 0) return MOE_OK;
    if (!q_dev || !s_dev || !ts_dev || !x_dev || !y_dev) return fail(MOE_ERR_INVALID_ARG, "null pointer");
    if (!aligned(q_dev, 16) || !aligned(s_dev, 2) || !aligned(ts_dev, 4) || !aligned(x_dev, 16) || x_stride % 8 ||
        !aligned(y_dev, y_bf16 ? 2 : 4))
        return fail(MOE_ERR_MISALIGNED, "q and rows of x need 16-byte alignment, s 2-byte, ts 4-byte, y its element's");
    Device dev;
    const moe_status_t st = query_device(-1, &dev);
    if (st != MOE_OK) return st;
    const moe::LinearParams p{q_dev, s_dev, ts_dev, static_cast<const uint16_t *>(x_dev), x_stride, y_dev, N, K, T, y_bf16};
    if (!linear_on_tensor_cores(p, dev.sms))
        return launched(moe::launch_linear(p, dev.sms, static_cast<cudaStream_t>(stream)), "linear launch");
    static const long long limit = moe::wait_limit_ns();
    if (!moe::encoder()) return fail(MOE_ERR_CUDA, "cuTensorMapEncodeTiled is not available from the driver");
    const moe::LinearTcPlan plan = moe::linear_tc_plan(p, dev.sms);
    moe::LinearTcParams tp{{}, p, plan.rows, plan.tiles, limit};
    const CUresult r = moe::encode_rows(&tp.tm_q, const_cast<uint8_t *>(q_dev), N, K / 2, 128, plan.rows, 128);
    if (r != CUDA_SUCCESS) return fail(MOE_ERR_CUDA, "tensor-map encoding failed (CUresult %d)", static_cast<int>(r));
    return launched(moe::launch_linear_tc(tp, plan.blocks, static_cast<cudaStream_t>(stream)), "linear launch");
}

moe_status_t moe_kv_create(const moe_kv_desc *desc, moe_kv_t *out)
{
    if (!desc || !out) return fail(MOE_ERR_INVALID_ARG, "null desc or out");
    *out = nullptr;
    const moe_kv_desc &d = *desc;
    if (d.head_dim != 64 && d.head_dim != 128)
        return fail(MOE_ERR_UNSUPPORTED_SHAPE, "head_dim=%d is not 64 or 128", d.head_dim);
    if (d.kv_heads < 1 || d.kv_heads > 1024 || d.q_heads < d.kv_heads || d.q_heads % d.kv_heads || d.q_heads > 65536)
        return fail(MOE_ERR_UNSUPPORTED_SHAPE, "q_heads=%d is not a multiple of kv_heads=%d (1 .. 1024)", d.q_heads,
                    d.kv_heads);
    // the tensor map counts rows of k in 32 bits
    if (d.n_pages < 1 || static_cast<long long>(d.n_pages) * d.kv_heads > (1LL << 30) / MOE_KV_PAGE)
        return fail(MOE_ERR_UNSUPPORTED_SHAPE, "n_pages=%d outside [1, %lld]", d.n_pages,
                    (1LL << 30) / MOE_KV_PAGE / d.kv_heads);
    if (d.rot_dim < 0 || d.rot_dim > d.head_dim || d.rot_dim % 2)
        return fail(MOE_ERR_UNSUPPORTED_SHAPE, "rot_dim=%d is not even and in [0, head_dim=%d]", d.rot_dim, d.head_dim);
    if (d.rot_interleaved != 0 && d.rot_interleaved != 1)
        return fail(MOE_ERR_INVALID_ARG, "rot_interleaved=%d is not 0 or 1", d.rot_interleaved);
    if (!d.k_dev || !d.v_dev || !d.k_scale_dev || !d.v_scale_dev) return fail(MOE_ERR_INVALID_ARG, "null cache pointer");
    if (d.rot_dim > 0 && (!d.rope_dev || d.rope_positions < 1))
        return fail(MOE_ERR_INVALID_ARG, "a rotation needs its table");
    if (!aligned(d.k_dev, 16) || !aligned(d.v_dev, 16) || !aligned(d.k_scale_dev, 4) || !aligned(d.v_scale_dev, 4) ||
        !aligned(d.rope_dev, 8))
        return fail(MOE_ERR_MISALIGNED, "k and v need 16-byte, the table 8-byte, scales 4-byte alignment");
    Device dev;
    const moe_status_t st = query_device(d.device, &dev);
    if (st != MOE_OK) return st;
    if (!moe::encoder()) return fail(MOE_ERR_CUDA, "cuTensorMapEncodeTiled is not available from the driver");
    moe_kv *kv = new (std::nothrow) moe_kv();  // no exception may cross the C ABI
    if (!kv) return fail(MOE_ERR_INVALID_ARG, "out of host memory for the cache handle");
    kv->d = d;
    kv->device = dev.ordinal;
    kv->num_sms = dev.sms;
    kv->smem_optin = dev.optin;
    kv->timeout_ns = moe::wait_limit_ns();
    const uint64_t ph = static_cast<uint64_t>(d.n_pages) * d.kv_heads;
    const CUresult r = moe::encode_rows(&kv->tm_k, d.k_dev, ph * MOE_KV_PAGE, d.head_dim, d.head_dim, MOE_KV_PAGE, d.head_dim);
    if (r != CUDA_SUCCESS) {
        delete kv;
        return fail(MOE_ERR_CUDA, "tensor-map encoding failed (CUresult %d)", static_cast<int>(r));
    }
    kv->off_count = moe::kCtrlBytes;
    kv->off_part = kv->off_count + (static_cast<size_t>(dev.sms) * 4 + 255) / 256 * 256;
    kv->ws_bytes = kv->off_part + static_cast<size_t>(dev.sms) * 2 * moe::attend_part_floats(d.head_dim) * 4;
    *out = kv;
    return MOE_OK;
}

void moe_kv_destroy(moe_kv_t kv) { delete kv; }

size_t moe_kv_workspace_bytes(moe_kv_t kv) { return kv ? kv->ws_bytes : 0; }

moe_status_t moe_kv_workspace_init(moe_kv_t kv, void *ws_dev, size_t bytes, void *stream)
{
    if (!kv) return fail(MOE_ERR_INVALID_ARG, "null cache");
    if (!ws_dev) return fail(MOE_ERR_INVALID_ARG, "null workspace");
    if (!aligned(ws_dev, 256)) return fail(MOE_ERR_MISALIGNED, "workspace must be 256-byte aligned");
    if (bytes < kv->ws_bytes)
        return fail(MOE_ERR_INVALID_ARG, "workspace of %zu bytes < %zu needed", bytes, kv->ws_bytes);
    moe_status_t st = check_device(kv);
    if (st != MOE_OK) return st;
    moe::WsTicket tk;
    st = moe::ws_claim(ws_dev, static_cast<cudaStream_t>(stream), tk);
    if (st != MOE_OK) return st;
    // the partial results behind the counters are written before they are read
    const cudaError_t e = cudaMemsetAsync(ws_dev, 0, kv->off_part, static_cast<cudaStream_t>(stream));
    moe::ws_release(tk, e == cudaSuccess);
    return launched(e, "workspace initialisation");
}

moe_status_t moe_kv_append(moe_kv_t kv, const void *q_dev, int64_t q_stride, const void *k_dev, int64_t k_stride,
                           const void *v_dev, int64_t v_stride, void *q_out_dev, const moe_kv_batch *batch,
                           void *ws_dev, void *stream)
{
    moe_status_t st = check_kv(kv, batch, ws_dev);
    if (st != MOE_OK) return st;
    const moe_kv_desc &d = kv->d;
    if (!q_dev != !q_out_dev) return fail(MOE_ERR_INVALID_ARG, "q and q_out come together");
    if (batch->B == 0 || batch->N == 0) return MOE_OK;
    if (q_dev && (st = check_rows(q_dev, q_stride, static_cast<int64_t>(d.q_heads) * d.head_dim, "q")) != MOE_OK) return st;
    if ((st = check_rows(k_dev, k_stride, static_cast<int64_t>(d.kv_heads) * d.head_dim, "k")) != MOE_OK) return st;
    if ((st = check_rows(v_dev, v_stride, static_cast<int64_t>(d.kv_heads) * d.head_dim, "v")) != MOE_OK) return st;
    if (!aligned(q_out_dev, 16)) return fail(MOE_ERR_MISALIGNED, "q_out needs 16-byte alignment");
    moe::AppendParams p{kv_params(kv, batch, ws_dev), static_cast<const uint16_t *>(q_dev),
                        static_cast<const uint16_t *>(k_dev), static_cast<const uint16_t *>(v_dev),
                        q_stride, k_stride, v_stride, static_cast<uint16_t *>(q_out_dev)};
    moe::WsTicket tk;
    if ((st = moe::ws_claim(ws_dev, static_cast<cudaStream_t>(stream), tk)) != MOE_OK) return st;
    const cudaError_t e = moe::launch_kv_append(p, static_cast<cudaStream_t>(stream));
    moe::ws_release(tk, e == cudaSuccess);
    return launched(e, "append launch");
}

moe_status_t moe_kv_attend(moe_kv_t kv, const void *q_dev, int64_t q_stride, float scale, void *o_dev,
                           const moe_kv_batch *batch, void *ws_dev, void *stream)
{
    moe_status_t st = check_kv(kv, batch, ws_dev);
    if (st != MOE_OK) return st;
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
    moe::AttendParams p{kv_params(kv, batch, ws_dev), static_cast<const uint16_t *>(q_dev), static_cast<uint16_t *>(o_dev),
                        q_stride, scale * 1.44269504088896341f, reinterpret_cast<uint32_t *>(ws + kv->off_count),
                        reinterpret_cast<float *>(ws + kv->off_part), kv->timeout_ns};
    moe::WsTicket tk;
    if ((st = moe::ws_claim(ws_dev, static_cast<cudaStream_t>(stream), tk)) != MOE_OK) return st;
    const cudaError_t e =
        tile_rows <= 16
            ? moe::launch_kv_attend_rows(p, tile_rows, kv->num_sms, kv->smem_optin, static_cast<cudaStream_t>(stream))
            : moe::launch_kv_attend_tc(p, kv->num_sms, static_cast<cudaStream_t>(stream));
    moe::ws_release(tk, e == cudaSuccess);
    return launched(e, "attention launch");
}

moe_status_t moe_kv_check(moe_kv_t kv, void *ws_dev, void *stream)
{
    if (!kv || !ws_dev) return fail(MOE_ERR_INVALID_ARG, "null cache or workspace");
    const moe_status_t st = check_device(kv);
    if (st != MOE_OK) return st;
    cudaStream_t cs = static_cast<cudaStream_t>(stream);
    uint8_t *word_dev = static_cast<uint8_t *>(ws_dev) + 8;
    uint32_t word = 0;
    cudaError_t e = cudaMemcpyAsync(&word, word_dev, 4, cudaMemcpyDeviceToHost, cs);
    if (e == cudaSuccess) e = cudaStreamSynchronize(cs);
    if (e == cudaSuccess && word) e = cudaMemsetAsync(word_dev, 0, 4, cs);
    if (e == cudaSuccess && word) e = cudaStreamSynchronize(cs);
    if (e != cudaSuccess) return fail(MOE_ERR_CUDA, "moe_kv_check: %s", cudaGetErrorString(e));
    if (word & moe::kErrTimeout) return fail(MOE_ERR_TIMEOUT, "a device-side wait timed out");
    if (word & moe::kErrBadIndex)
        return fail(MOE_ERR_BAD_INDEX, "a page id, a position or a sequence's offsets or length are out of range");
    return MOE_OK;
}

}  // extern "C"
