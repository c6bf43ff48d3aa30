// moe_host.h -- host-side helpers the ABI files share (defined in moe_abi.cu):
// error messages, pointer checks, the driver's tensor-map encoder and the
// ownership of workspaces across streams.  Not part of the ABI.
#pragma once
#include "moe_nvfp4.h"

#include <cstddef>
#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

namespace moe {

// Record the calling thread's last-error message (printf format) and return s.
moe_status_t fail(moe_status_t s, const char *fmt, ...);

inline bool aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// cuTensorMapEncodeTiled from the driver, or null where it is not available.
PFN_cuTensorMapEncodeTiled_v12000 encoder();

// Row-major uint8 [rows, cols] with a {box_c, box_r} box, swizzled over 128 or 64
// bytes (0: not).
CUresult encode_rows(CUtensorMap *m, void *base, uint64_t rows, uint64_t cols, int box_c, int box_r, int swizzle);

// Limit of a device-side wait: 1 s, or MOE_WAIT_TIMEOUT_MS.
long long wait_limit_ns();

// One launch on a workspace: ws_claim before it orders the launch after work
// in flight on the workspace from another stream, ws_release after it records
// the event that marks its end.
struct WsUse;
struct WsTicket {
    WsUse *u = nullptr;  // null: not tracked (graph capture)
    cudaStream_t st = nullptr;
};
moe_status_t ws_claim(const void *ws, cudaStream_t st, WsTicket &t);
void ws_release(WsTicket &t, bool launched);

}  // namespace moe
