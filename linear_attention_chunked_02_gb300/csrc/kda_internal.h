// kda_internal.h -- host-side helpers shared by the library's translation units
// (not exported).
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "kda_solve_tril.h"

namespace kda {

inline int elt_size(int32_t dt) { return dt == KDA_F32 ? 4 : 2; }
inline bool dtype_ok(int32_t dt) { return dt == KDA_F32 || dt == KDA_BF16 || dt == KDA_F16; }
inline bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline bool overlaps(const void *a, size_t na, const void *b, size_t nb) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return x < y + nb && y < x + na;
}

// Number of SMs and the address of the error word of a device, looked up once.
struct DeviceInfo {
    int num_sms = 0;
    unsigned *err = nullptr;
};
cudaError_t device_info(int device, DeviceInfo &out);

// cuTensorMapEncodeTiled, looked up once; nullptr if the driver has none.
PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder();

// Upper bound on the number of chunks of length bt that needs no look at cu_seqlens.
int64_t max_chunks(int64_t B, int64_t T, int32_t num_seqs, int bt);

// The host-side argument checks of kda_solve_tril that do not involve the
// workspace: dtypes, shape limits, the packed/dense layout rules, null
// pointers, 16-byte alignment and overlap of A and Ai.  Makes no CUDA call.
kda_status_t validate_solve(const void *A, const void *Ai, const int32_t *cu, int32_t num_seqs, int64_t B,
                            int64_t T, int32_t H, int32_t in_dt, int32_t out_dt);

}  // namespace kda
