// moe_layer.cu -- host side of the C ABI declared in include/moe_layer.h:
// argument validation, the cache handle, its workspace, launches.  The
// computation runs in moe_norm.cu, moe_linear.cu, moe_linear_tc.cu,
// moe_kv_append.cu, moe_kv_attend.cu and moe_kv_attend_tc.cu.
#include "moe_layer_host.h"

#include <cmath>
#include <mutex>
#include <new>

using moe::aligned;
using moe::check_device;
using moe::check_kv;
using moe::Device;
using moe::fail;
using moe::launched;
using moe::query_device;

namespace moe {

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

}  // namespace moe

namespace {

constexpr int kMaxNormH = 16384;
constexpr int kMaxLinearK = 1 << 22;  // the kernel counts bytes inside 512 rows in 32 bits

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
    moe::AppendParams p;
    if ((st = moe::append_params(kv, q_dev, q_stride, k_dev, k_stride, v_dev, v_stride, q_out_dev, batch, ws_dev, &p)) != MOE_OK)
        return st;
    if (batch->B == 0 || batch->N == 0) return MOE_OK;
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
    moe::AttendParams p;
    int tile_rows = 0;
    if ((st = moe::attend_params(kv, q_dev, q_stride, scale, o_dev, batch, ws_dev, &p, &tile_rows)) != MOE_OK) return st;
    if (batch->B == 0 || batch->N == 0) return MOE_OK;
    moe::WsTicket tk;
    if ((st = moe::ws_claim(ws_dev, static_cast<cudaStream_t>(stream), tk)) != MOE_OK) return st;
    const cudaError_t e = moe::launch_kv_attend(kv, p, tile_rows, static_cast<cudaStream_t>(stream));
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
