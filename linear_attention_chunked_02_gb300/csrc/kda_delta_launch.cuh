// kda_delta_launch.cuh -- host-side launches of the chunked gated delta rule for one type.
#pragma once

#include <cuda_runtime.h>

#include <mutex>

#include "kda_delta_launch.h"
#include "kda_launch.cuh"

namespace kda {

// Opt-in shared memory, and a check that the kernel launches with the registers that its warp
// groups' shares add up to: with fewer, the groups that take more would wait for ever.
template <typename F>
cudaError_t kernel_ready(F *fn, int bytes, int registers) {
    cudaFuncAttributes a;
    cudaError_t e = cudaFuncGetAttributes(&a, fn);
    if (e == cudaSuccess && a.numRegs < registers) e = cudaErrorInvalidConfiguration;
    return e == cudaSuccess ? cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) : e;
}

// Once per device.
template <typename T, int KW>
cudaError_t chunked_ready(int device) {
    static std::mutex mu;
    static bool done[64] = {false};
    std::lock_guard<std::mutex> lock(mu);
    if (device < 0 || device >= 64) return cudaErrorInvalidDevice;
    if (done[device]) return cudaSuccess;
    cudaError_t e = kernel_ready(kda_delta_prep_kernel<T>, prep_bytes<T>(), PREP_REGISTERS);
    if (e == cudaSuccess)
        e = kernel_ready(kda_delta_scan_kernel<T, KW, false>, scan_bytes<T>(KW == 64 ? 64 : 128), SCAN_REGISTERS);
    if (e == cudaSuccess)
        e = kernel_ready(kda_delta_scan_kernel<T, KW, true>, scan_bytes<T>(KW == 64 ? 64 : 128), SCAN_REGISTERS);
    if (e == cudaSuccess) e = kernel_ready(kda_delta_join_kernel<T>, JOIN_BYTES, 0);
    done[device] = e == cudaSuccess;
    return e;
}

template <typename T, int KW>
cudaError_t launch_widths(const DeltaParams &p, const DeltaMaps &prep, const DeltaMaps &scan, int device, int sms,
                          cudaStream_t s) {
    cudaError_t e = chunked_ready<T, KW>(device);
    if (e != cudaSuccess) return e;
    auto blocks = [&](int64_t n) { return unsigned(n < sms ? n : sms); };     // persistent, one to an SM
    const int64_t walks = int64_t(p.n_units) * p.H;
    const size_t bytes = size_t(scan_bytes<T>(p.K));
    e = launch_pdl(true, kda_delta_prep_kernel<T>, blocks(p.n_tasks), PREP_THREADS, size_t(prep_bytes<T>()), s, prep, p);
    if (e == cudaSuccess && p.seg > 0) {
        e = launch_pdl(true, kda_delta_scan_kernel<T, KW, true>, blocks(2 * walks), SCAN_THREADS, bytes, s, scan, p);
        if (e == cudaSuccess)
            e = launch_pdl(true, kda_delta_join_kernel<T>, unsigned(p.nseq) * unsigned(p.H) * unsigned(p.V / JOIN_COLS),
                           JOIN_THREADS, size_t(JOIN_BYTES), s, p);
    }
    if (e != cudaSuccess) return e;
    return launch_pdl(true, kda_delta_scan_kernel<T, KW, false>, blocks(walks), SCAN_THREADS, bytes, s, scan, p);
}

template <typename T>
cudaError_t launch_chunked(const DeltaParams &p, const DeltaMaps &prep, const DeltaMaps &scan, int device, int sms,
                           cudaStream_t s) {
    return p.K == 128 && p.V == 128 ? launch_widths<T, 128>(p, prep, scan, device, sms, s)
           : p.K <= 64              ? launch_widths<T, 64>(p, prep, scan, device, sms, s)
                                    : launch_widths<T, 0>(p, prep, scan, device, sms, s);
}

}  // namespace kda
