// kda_recur_launch.cuh -- the recurrence's kernels for one type of x and y.
#pragma once

#include <type_traits>

#include "kda_recur_launch.h"

namespace kda {

template <typename... Args>
cudaError_t launch_recur(void (*fn)(Args...), const RecurLaunch &l, unsigned threads, cudaStream_t stream,
                         const Args &...args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(l.slabs, l.parts);
    cfg.blockDim = dim3(threads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, fn, args...);
}

template <typename T, typename G, int VEC>
cudaError_t launch_scan_vec(const RecurParams &p, const RecurLaunch &l, cudaStream_t s) {
    return launch_recur(kda_gated_scan_kernel<T, G, VEC, 8, 8>, l, 256, s, p);
}
template <typename T, typename G>
cudaError_t launch_scan_g(const RecurParams &p, const RecurLaunch &l, cudaStream_t s) {
    return l.vec == 2 ? launch_scan_vec<T, G, 2>(p, l, s) : launch_scan_vec<T, G, 1>(p, l, s);
}
template <typename T>
cudaError_t launch_scan(const RecurParams &p, const RecurLaunch &l, cudaStream_t s) {
    return l.wide_g || std::is_same_v<T, float> ? launch_scan_g<T, float>(p, l, s) : launch_scan_g<T, T>(p, l, s);
}

template <typename T, typename X, typename S, typename G>
cudaError_t launch_backward_vec(const RecurParams &p, const RecurLaunch &l, cudaStream_t s) {
    return l.vec == 2 ? launch_recur(kda_gated_scan_backward_kernel<T, X, S, G, 2, 8, 8>, l, 256, s, p)
                      : launch_recur(kda_gated_scan_backward_kernel<T, X, S, G, 1, 8, 8>, l, 256, s, p);
}
template <typename T, typename G>
cudaError_t launch_backward_g(const RecurParams &p, const RecurLaunch &l, cudaStream_t s) {
    if (l.x8) return l.g8 ? launch_backward_vec<T, int8_t, int8_t, G>(p, l, s) : launch_backward_vec<T, int8_t, G, G>(p, l, s);
    return l.g8 ? launch_backward_vec<T, T, int8_t, G>(p, l, s) : launch_backward_vec<T, T, G, G>(p, l, s);
}
template <typename T>
cudaError_t launch_backward(const RecurParams &p, const RecurLaunch &l, cudaStream_t s) {
    return l.wide_g || std::is_same_v<T, float> ? launch_backward_g<T, float>(p, l, s) : launch_backward_g<T, T>(p, l, s);
}

}  // namespace kda
