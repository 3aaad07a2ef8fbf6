// kda_recur_launch.cuh -- the recurrence's kernels for one type of x and y.
#pragma once

#include <mutex>
#include <type_traits>

#include "kda_recur_launch.h"

namespace kda {

using RecurKernel = void (*)(const RecurParams);

inline void recur_config(cudaLaunchConfig_t &cfg, cudaLaunchAttribute (&attr)[2], unsigned cluster, dim3 grid, unsigned threads,
                         int smem, cudaStream_t stream) {
    cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = size_t(smem);
    cfg.stream = stream;
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
}

// The blocks of FN that run at once on a device by the size of their clusters, looked up once; raises the limits that
// its launches need.
template <RecurKernel FN, typename Shape>
cudaError_t recur_room(int device, RecurRoom &room) {
    static std::mutex mu;
    static RecurRoom known[64];
    if (device < 0 || device >= 64) return cudaErrorInvalidDevice;
    std::lock_guard<std::mutex> lock(mu);
    RecurRoom &k = known[device];
    if (k.blocks[1] == 0) {
        cudaError_t e =
            cudaFuncSetAttribute(FN, cudaFuncAttributeMaxDynamicSharedMemorySize, Shape::bytes(RECUR_CLUSTER));
        if (e == cudaSuccess) e = cudaFuncSetAttribute(FN, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        if (e != cudaSuccess) return e;
        RecurRoom found;
        for (int size = RECUR_CLUSTER; size >= 1; --size) {
            cudaLaunchConfig_t cfg;
            cudaLaunchAttribute attr[2];
            recur_config(cfg, attr, unsigned(size), dim3(unsigned(size)), Shape::THREADS, Shape::bytes(size), nullptr);
            int n = 0;
            if (size > 1) {
                e = cudaOccupancyMaxActiveClusters(&n, FN, &cfg);
                if (e != cudaSuccess) {                    // a size that this device does not take
                    cudaGetLastError();
                    n = 0;
                }
            } else {
                e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, FN, Shape::THREADS, size_t(Shape::bytes(1)));
                if (e != cudaSuccess) return e;
                int sms = 0;
                e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, device);
                if (e != cudaSuccess) return e;
                n = n > 0 ? n * sms : 1;
            }
            found.blocks[size] = n * size;
        }
        k = found;
    }
    room = k;
    return cudaSuccess;
}

// FN over a stream of rows, in the shape that `forward` or gradients take.
template <RecurKernel FN, typename Shape>
cudaError_t launch_recur(RecurParams &p, const RecurLaunch &l, cudaStream_t stream) {
    RecurRoom room;
    cudaError_t e = recur_room<FN, Shape>(l.device, room);
    if (e != cudaSuccess) return e;
    const RecurGrid g = recur_grid(p, room, Shape::COLUMNS, Shape::TILE, l.walk_wide, l.walk_fit);
    cudaLaunchConfig_t cfg;
    cudaLaunchAttribute attr[2];
    recur_config(cfg, attr, g.cluster, dim3(g.cluster * g.clusters), Shape::THREADS, Shape::bytes(int(g.cluster)), stream);
    return cudaLaunchKernelEx(&cfg, FN, p);
}

template <typename T, typename G, int FORM, int VEC, int PIECE>
cudaError_t launch_scan_form(RecurParams &p, const RecurLaunch &l, cudaStream_t s) {
    constexpr int R = sizeof(T) == 4 ? 8 : 16, W = 7, RING = 2, MIN = sizeof(T) == 4 ? 3 : 2;
    using Shape = ScanShape<T, G, VEC, R, W, RING, PIECE>;
    return launch_recur<kda_gated_scan_kernel<T, G, FORM, VEC, R, W, RING, PIECE, MIN>, Shape>(p, l, s);
}
template <typename T, typename G>
cudaError_t launch_scan_g(RecurParams &p, const RecurLaunch &l, cudaStream_t s) {
    if (!l.staged) {
        if constexpr (sizeof(T) == 4) {                     // four bytes at a time fit any row of FP32
            switch (p.form) {
                case 0: return launch_scan_form<T, G, 0, 1, 4>(p, l, s);
                case 1: return launch_scan_form<T, G, 1, 1, 4>(p, l, s);
                case 2: return launch_scan_form<T, G, 2, 1, 4>(p, l, s);
                default: return launch_scan_form<T, G, 3, 1, 4>(p, l, s);
            }
        } else {
            return launch_scan_form<T, G, -1, 1, 0>(p, l, s);
        }
    }
    switch (p.form) {
        case 0: return launch_scan_form<T, G, 0, 2, 16>(p, l, s);
        case 1: return launch_scan_form<T, G, 1, 2, 16>(p, l, s);
        case 2: return launch_scan_form<T, G, 2, 2, 16>(p, l, s);
        default: return launch_scan_form<T, G, 3, 2, 16>(p, l, s);
    }
}
template <typename T>
cudaError_t launch_scan(RecurParams &p, const RecurLaunch &l, cudaStream_t s) {
    return l.wide_g || std::is_same_v<T, float> ? launch_scan_g<T, float>(p, l, s) : launch_scan_g<T, T>(p, l, s);
}

template <typename T, typename X, typename S, typename G, int FORM, int VEC, int PIECE>
cudaError_t launch_backward_form(RecurParams &p, const RecurLaunch &l, cudaStream_t s) {
    constexpr int R = 8, W = 8, RING = sizeof(X) == 1 || sizeof(S) == 1 ? 1 : 2, MIN = VEC == 1 && PIECE != 0 ? 3 : 2;
    using Shape = GradShape<T, X, S, VEC, R, W, RING, PIECE>;
    return launch_recur<kda_gated_scan_backward_kernel<T, X, S, G, FORM, VEC, R, W, RING, PIECE, MIN>, Shape>(p, l, s);
}
template <typename T, typename X, typename S, typename G>
cudaError_t launch_backward_xs(RecurParams &p, const RecurLaunch &l, cudaStream_t s) {
    constexpr int VEC = backward_vec<T, X, S>();
    if (!l.staged) {
        if constexpr (sizeof(T) == 4 && sizeof(X) == 4 && sizeof(S) == 4) {
            switch (p.form) {
                case 0: return launch_backward_form<T, X, S, G, 0, 1, 4>(p, l, s);
                case 1: return launch_backward_form<T, X, S, G, 1, 1, 4>(p, l, s);
                case 2: return launch_backward_form<T, X, S, G, 2, 1, 4>(p, l, s);
                default: return launch_backward_form<T, X, S, G, 3, 1, 4>(p, l, s);
            }
        } else {
            return launch_backward_form<T, X, S, G, -1, 1, 0>(p, l, s);
        }
    }
    switch (p.form) {
        case 0: return launch_backward_form<T, X, S, G, 0, VEC, 16>(p, l, s);
        case 1: return launch_backward_form<T, X, S, G, 1, VEC, 16>(p, l, s);
        case 2: return launch_backward_form<T, X, S, G, 2, VEC, 16>(p, l, s);
        default: return launch_backward_form<T, X, S, G, 3, VEC, 16>(p, l, s);
    }
}
template <typename T, typename G>
cudaError_t launch_backward_g(RecurParams &p, const RecurLaunch &l, cudaStream_t s) {
    if (l.x8) return l.g8 ? launch_backward_xs<T, int8_t, int8_t, G>(p, l, s) : launch_backward_xs<T, int8_t, G, G>(p, l, s);
    return l.g8 ? launch_backward_xs<T, T, int8_t, G>(p, l, s) : launch_backward_xs<T, T, G, G>(p, l, s);
}
template <typename T>
cudaError_t launch_backward(RecurParams &p, const RecurLaunch &l, cudaStream_t s) {
    return l.wide_g || std::is_same_v<T, float> ? launch_backward_g<T, float>(p, l, s) : launch_backward_g<T, T>(p, l, s);
}

}  // namespace kda
