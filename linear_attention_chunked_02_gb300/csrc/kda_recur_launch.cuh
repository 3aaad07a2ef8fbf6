// kda_recur_launch.cuh -- the recurrence's kernels for one type of x and y.
#pragma once

#include <atomic>
#include <type_traits>

#include "kda_recur_launch.h"

namespace kda {

using RecurKernel = void (*)(const RecurParams);

// FN's launch with `smem` bytes of `most` that any of its launches takes; the limit is raised once for every device.
template <RecurKernel FN>
cudaError_t launch_recur(const RecurParams &p, const RecurLaunch &l, unsigned threads, int smem, int most,
                         cudaStream_t stream) {
    static std::atomic<bool> set[64];
    if (l.device < 0 || l.device >= 64) return cudaErrorInvalidDevice;
    if (!set[l.device].load(std::memory_order_relaxed)) {
        cudaError_t e = cudaFuncSetAttribute(FN, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
        if (e == cudaSuccess) e = cudaFuncSetAttribute(FN, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        if (e != cudaSuccess) return e;
        set[l.device].store(true, std::memory_order_relaxed);
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(l.cluster, l.slabs, l.parts);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = size_t(smem);
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = l.cluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = l.cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, FN, p);
}

template <typename T, typename G, int FORM, int VEC, int PIECE>
cudaError_t launch_scan_form(const RecurParams &p, const RecurLaunch &l, cudaStream_t s) {
    constexpr int R = sizeof(T) == 4 ? 8 : 16, W = 7, RING = 2, MIN = sizeof(T) == 4 ? 3 : 2;
    using Shape = ScanShape<T, G, VEC, R, W, RING, PIECE>;
    return launch_recur<kda_gated_scan_kernel<T, G, FORM, VEC, R, W, RING, PIECE, MIN>>(
        p, l, Shape::THREADS, Shape::bytes(int(l.cluster)), Shape::bytes(RECUR_CLUSTER), s);
}
template <typename T, typename G>
cudaError_t launch_scan_g(const RecurParams &p, const RecurLaunch &l, cudaStream_t s) {
    if (!l.staged) return launch_scan_form<T, G, -1, 1, sizeof(T) == 4 ? 4 : 0>(p, l, s);
    switch (p.form) {
        case 0: return launch_scan_form<T, G, 0, 2, 16>(p, l, s);
        case 1: return launch_scan_form<T, G, 1, 2, 16>(p, l, s);
        case 2: return launch_scan_form<T, G, 2, 2, 16>(p, l, s);
        default: return launch_scan_form<T, G, 3, 2, 16>(p, l, s);
    }
}
template <typename T>
cudaError_t launch_scan(const RecurParams &p, const RecurLaunch &l, cudaStream_t s) {
    return l.wide_g || std::is_same_v<T, float> ? launch_scan_g<T, float>(p, l, s) : launch_scan_g<T, T>(p, l, s);
}

template <typename T, typename X, typename S, typename G, int FORM, int VEC, int PIECE>
cudaError_t launch_backward_form(const RecurParams &p, const RecurLaunch &l, cudaStream_t s) {
    constexpr int R = 8, W = 8, RING = 1;
    using Shape = GradShape<T, X, S, VEC, R, W, RING, PIECE>;
    return launch_recur<kda_gated_scan_backward_kernel<T, X, S, G, FORM, VEC, R, W, RING, PIECE, VEC == 1 ? 3 : 2>>(
        p, l, Shape::THREADS, Shape::bytes(int(l.cluster)), Shape::bytes(RECUR_CLUSTER), s);
}
template <typename T, typename X, typename S, typename G>
cudaError_t launch_backward_xs(const RecurParams &p, const RecurLaunch &l, cudaStream_t s) {
    // rows of FP32: four bytes at a time fit any of them
    constexpr int ODD = sizeof(T) == 4 && sizeof(X) == 4 && sizeof(S) == 4 ? 4 : 0, VEC = backward_vec<T, X, S>();
    if (!l.staged) return launch_backward_form<T, X, S, G, -1, 1, ODD>(p, l, s);
    switch (p.form) {
        case 0: return launch_backward_form<T, X, S, G, 0, VEC, 16>(p, l, s);
        case 1: return launch_backward_form<T, X, S, G, 1, VEC, 16>(p, l, s);
        case 2: return launch_backward_form<T, X, S, G, 2, VEC, 16>(p, l, s);
        default: return launch_backward_form<T, X, S, G, 3, VEC, 16>(p, l, s);
    }
}
template <typename T, typename G>
cudaError_t launch_backward_g(const RecurParams &p, const RecurLaunch &l, cudaStream_t s) {
    if (l.x8) return l.g8 ? launch_backward_xs<T, int8_t, int8_t, G>(p, l, s) : launch_backward_xs<T, int8_t, G, G>(p, l, s);
    return l.g8 ? launch_backward_xs<T, T, int8_t, G>(p, l, s) : launch_backward_xs<T, T, G, G>(p, l, s);
}
template <typename T>
cudaError_t launch_backward(const RecurParams &p, const RecurLaunch &l, cudaStream_t s) {
    return l.wide_g || std::is_same_v<T, float> ? launch_backward_g<T, float>(p, l, s) : launch_backward_g<T, T>(p, l, s);
}

}  // namespace kda
