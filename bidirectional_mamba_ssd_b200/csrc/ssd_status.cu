// The library's own status header, one per device: what calls that were captured
// into a CUDA graph report at its replays. Such a call's workspace lives as long
// as the graph and has no owner who could read it, and the stream that replays it
// need not be the one that it was captured on.
#include "ssd_bidir.h"
#include "ssd_common.cuh"

namespace {

__device__ __align__(256) ssd::DeviceStatus g_captured;

// Its address on the current device. The first lookup on a device loads this module,
// which a thread that is capturing may do in the relaxed mode only.
cudaError_t captured_address(void **out) {
    cudaStreamCaptureMode mode = cudaStreamCaptureModeRelaxed;
    cudaError_t e = cudaThreadExchangeStreamCaptureMode(&mode);
    if (e != cudaSuccess) return e;
    e = cudaGetSymbolAddress(out, g_captured);
    const cudaError_t back = cudaThreadExchangeStreamCaptureMode(&mode);
    return e != cudaSuccess ? e : back;
}

__global__ void init_captured_kernel(ssd::DeviceStatus *st, ssd::DeviceStatus *also) {
    reinterpret_cast<unsigned int *>(st)[threadIdx.x] = 0u;
    __syncthreads();
    if (threadIdx.x == 0) st->also = also;
}

}  // namespace

extern "C" {

int ssd_captured_status(void **header) {
    if (!header) return SSD_ERR_INVALID_ARG;
    return captured_address(header) == cudaSuccess ? SSD_OK : SSD_ERR_CUDA;
}

int ssd_workspace_init_captured(void *workspace, size_t ws_bytes, void *stream) {
    if (!workspace || ws_bytes < ssd::kStatusBytes) return SSD_ERR_WORKSPACE;
    if (reinterpret_cast<uintptr_t>(workspace) & 15) return SSD_ERR_INVALID_ARG;
    void *also = nullptr;
    if (captured_address(&also) != cudaSuccess) return SSD_ERR_CUDA;
    init_captured_kernel<<<1, ssd::kStatusBytes / 4, 0, static_cast<cudaStream_t>(stream)>>>(
        static_cast<ssd::DeviceStatus *>(workspace), static_cast<ssd::DeviceStatus *>(also));
    return cudaGetLastError() == cudaSuccess ? SSD_OK : SSD_ERR_CUDA;
}

}  // extern "C"
