// kda_delta_launch.h -- the chunked gated delta rule's launches, one translation unit to a type
// (kda_delta_inst_{f32,bf16,f16}.cu).
#pragma once

#include "kda_delta_scan.cuh"

namespace kda {

cudaError_t launch_chunked_f32(const DeltaParams &, const DeltaMaps &, const DeltaMaps &, int device, int sms, cudaStream_t);
cudaError_t launch_chunked_bf16(const DeltaParams &, const DeltaMaps &, const DeltaMaps &, int device, int sms, cudaStream_t);
cudaError_t launch_chunked_f16(const DeltaParams &, const DeltaMaps &, const DeltaMaps &, int device, int sms, cudaStream_t);

}  // namespace kda
