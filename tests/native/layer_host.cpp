// The host side of the layer operators (moe_layer.cu) over a runtime that only takes notes:
// a current device that the test sets, and the names of the calls that would queue work.
#include "moe_layer.cu"

#include <cstdarg>
#include <cstdio>
#include <string>

namespace {
int g_device = 0;
std::string g_queued, g_message;
void note(const char *what) { g_queued += std::string(what) + " "; }
}  // namespace

extern "C" {

// ---- what the test sets and reads
void fake_device(int d) { g_device = d; }
const char *fake_queued() { return g_queued.c_str(); }
const char *fake_message() { return g_message.c_str(); }
void fake_clear() { g_queued.clear(); }

// ---- the runtime
cudaError_t cudaGetDevice(int *d)
{
    *d = g_device;
    return cudaSuccess;
}
cudaError_t cudaDeviceGetAttribute(int *v, cudaDeviceAttr a, int)
{
    *v = a == cudaDevAttrMultiProcessorCount                 ? 152
         : a == cudaDevAttrMaxSharedMemoryPerBlockOptin      ? 232448
         : a == cudaDevAttrComputeCapabilityMajor            ? 10
                                                             : 3;
    return cudaSuccess;
}
const char *cudaGetErrorString(cudaError_t) { return "an error"; }
cudaError_t cudaMemsetAsync(void *, int, size_t, cudaStream_t)
{
    note("memset");
    return cudaSuccess;
}
cudaError_t cudaMemcpyAsync(void *, const void *, size_t, cudaMemcpyKind, cudaStream_t)
{
    note("memcpy");
    return cudaSuccess;
}
cudaError_t cudaStreamSynchronize(cudaStream_t) { return cudaSuccess; }

}  // extern "C"

// ---- the rest of the library
namespace moe {

moe_status_t fail(moe_status_t s, const char *fmt, ...)
{
    char buf[512];
    va_list ap;
    va_start(ap, fmt);
    std::vsnprintf(buf, sizeof buf, fmt, ap);
    va_end(ap);
    g_message = buf;
    return s;
}
PFN_cuTensorMapEncodeTiled_v12000 encoder()
{
    return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(&fail);  // (not null; never called)
}
CUresult encode_rows(CUtensorMap *, void *, uint64_t, uint64_t, int, int, int) { return CUDA_SUCCESS; }
long long wait_limit_ns() { return 1; }
moe_status_t ws_claim(const void *, cudaStream_t, WsTicket &)
{
    note("claim");
    return MOE_OK;
}
void ws_release(WsTicket &, bool) {}
LinearTcPlan linear_tc_plan(const LinearParams &, int) { return {128, 1, 1}; }
#define MOE_FAKE_LAUNCH(name, ...)  \
    cudaError_t name(__VA_ARGS__)   \
    {                               \
        note(#name);                \
        return cudaSuccess;         \
    }
MOE_FAKE_LAUNCH(launch_norm, const NormParams &, cudaStream_t)
MOE_FAKE_LAUNCH(launch_linear, const LinearParams &, int, cudaStream_t)
MOE_FAKE_LAUNCH(launch_linear_tc, const LinearTcParams &, int, cudaStream_t)
MOE_FAKE_LAUNCH(launch_kv_append, const AppendParams &, cudaStream_t)
MOE_FAKE_LAUNCH(launch_kv_attend_rows, const AttendParams &, int, int, int, cudaStream_t)
MOE_FAKE_LAUNCH(launch_kv_attend_tc, const AttendParams &, int, cudaStream_t)

}  // namespace moe
