// kda_recur_launch.h -- the recurrence's launches by the type of x and y (kda_recur_inst_*.cu).
#pragma once

#include "kda_recur.cuh"

namespace kda {

// vec: channels to a lane, 1 or 2; wide_g: g and dg in FP32; x8, g8: codes in place of x and g; slabs x parts blocks
struct RecurLaunch {
    int vec;
    bool wide_g, x8, g8;
    unsigned slabs, parts;
};

cudaError_t launch_scan_f32(const RecurParams &p, const RecurLaunch &l, cudaStream_t s);
cudaError_t launch_scan_bf16(const RecurParams &p, const RecurLaunch &l, cudaStream_t s);
cudaError_t launch_scan_f16(const RecurParams &p, const RecurLaunch &l, cudaStream_t s);
cudaError_t launch_scan_backward_f32(const RecurParams &p, const RecurLaunch &l, cudaStream_t s);
cudaError_t launch_scan_backward_bf16(const RecurParams &p, const RecurLaunch &l, cudaStream_t s);
cudaError_t launch_scan_backward_f16(const RecurParams &p, const RecurLaunch &l, cudaStream_t s);

}  // namespace kda
