// kda_vec.cuh -- vectors of consecutive row elements: loads of data that is read
// once, widening to FP32, rounding back, and the values of 8-bit checkpoints.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>
#include <string.h>

namespace kda {

template <int BYTES>
struct RawOf;
template <> struct RawOf<1> { using type = unsigned char; };
template <> struct RawOf<2> { using type = unsigned short; };
template <> struct RawOf<4> { using type = unsigned; };
template <> struct RawOf<8> { using type = uint2; };
template <> struct RawOf<16> { using type = uint4; };
// N elements of S as they lie in memory
template <typename S, int N>
using raw_t = typename RawOf<N * int(sizeof(S))>::type;

template <typename S, int N>
__device__ __forceinline__ raw_t<S, N> load_once(const S *p) {
    return __ldcs(reinterpret_cast<const raw_t<S, N> *>(p));
}
template <typename S, int N>
__device__ __forceinline__ void store_raw(S *p, raw_t<S, N> v) {
    *reinterpret_cast<raw_t<S, N> *>(p) = v;
}

__device__ __forceinline__ float widen_one(float v) { return v; }
__device__ __forceinline__ float widen_one(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float widen_one(__half v) { return __half2float(v); }
__device__ __forceinline__ void narrow_one(float &to, float v) { to = v; }
__device__ __forceinline__ void narrow_one(__nv_bfloat16 &to, float v) { to = __float2bfloat16_rn(v); }
__device__ __forceinline__ void narrow_one(__half &to, float v) { to = __float2half_rn(v); }

template <typename S, int N>
__device__ __forceinline__ void widen(raw_t<S, N> raw, float (&v)[N]) {
    S e[N];
    memcpy(e, &raw, sizeof(raw));
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = widen_one(e[i]);
}
template <typename S, int N>
__device__ __forceinline__ raw_t<S, N> narrow(const float (&v)[N]) {
    S e[N];
#pragma unroll
    for (int i = 0; i < N; ++i) narrow_one(e[i], v[i]);
    raw_t<S, N> raw;
    memcpy(&raw, e, sizeof(raw));
    return raw;
}

// 8-bit checkpoints: blocks of 32 elements of a row share the scale 2^(e - 127), e their exponent byte;
// 255 stands for a block that was not finite, all of whose values are NaN.
constexpr int CKPT_BLOCK = 32, CKPT_BAD = 255;
__device__ __forceinline__ float ckpt_scale(unsigned e) {
    return __uint_as_float(e == 0 ? 0x00400000u : e == CKPT_BAD ? 0x7fffffffu : e << 23);
}

}  // namespace kda
