// kda_recur_launch.h -- the recurrence's launches by the type of x and y (kda_recur_inst_*.cu).
#pragma once

#include "kda_recur.cuh"

namespace kda {

struct RecurLaunch {
    bool staged;                // the inputs' rows are whole, aligned 16-byte pieces
    bool wide_g, x8, g8;        // g and dg in FP32; codes in place of x and g
    int walk_wide;              // forward, staged: channels to a lane of a walking warp, or half as many; 0: no walks
    int walk_fit;               // channels whose vectors fit the addresses of y, the states and the chunk states
    int device;
};

// Blocks of a kernel that run at once, by the size of their clusters (0: none of this size).
struct RecurRoom {
    int blocks[RECUR_CLUSTER + 1] = {0};
};
struct RecurGrid {
    unsigned cluster, clusters;
};
// How the stream is cut for a kernel whose blocks take `columns` channels and `tile` rows at a time (kda_recur.cu).
RecurGrid recur_grid(RecurParams &p, const RecurRoom &room, int columns, int tile, int walk_wide, int walk_fit);

// Channels to a lane of the gradients of staged rows: two, or one where an operand is FP32, whose rows of 64 channels
// would leave room for one block on an SM alone.
template <typename T, typename X, typename S>
constexpr int backward_vec() {
    return sizeof(T) == 4 || sizeof(X) == 4 || sizeof(S) == 4 ? 1 : 2;
}

cudaError_t launch_scan_f32(RecurParams &p, const RecurLaunch &l, cudaStream_t s);
cudaError_t launch_scan_bf16(RecurParams &p, const RecurLaunch &l, cudaStream_t s);
cudaError_t launch_scan_f16(RecurParams &p, const RecurLaunch &l, cudaStream_t s);
cudaError_t launch_scan_backward_f32(RecurParams &p, const RecurLaunch &l, cudaStream_t s);
cudaError_t launch_scan_backward_bf16(RecurParams &p, const RecurLaunch &l, cudaStream_t s);
cudaError_t launch_scan_backward_f16(RecurParams &p, const RecurLaunch &l, cudaStream_t s);

}  // namespace kda
