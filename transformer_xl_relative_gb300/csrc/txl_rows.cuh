// txl_rows.cuh -- loads of fp32 or bf16 rows, expansion of codes and products of rows in shared memory, shared by the kernels of the quantised memory.
#pragma once

#include <cstdint>

namespace txl {

// A load of what an earlier kernel may have written: this grid may start before that one has ended, so that the data
// is not read-only while it runs, as __ldg wants it (that is for u and v alone).  After pdl_wait.
template <typename T>
__device__ __forceinline__ T ld(const T* p) { return *p; }

// Eight channels d0 .. d0+7 of a row; channels at or past D read as 0.  vec: the row starts on a 16-byte boundary.
template <bool F32>
__device__ __forceinline__ void load8(const void* row, int d0, int D, bool vec, float* x)
{
    if (vec && d0 + 8 <= D) {
        if constexpr (F32) {
            const float4* q = reinterpret_cast<const float4*>(static_cast<const float*>(row) + d0);
            const float4 a = ld(q), b = ld(q + 1);
            x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
            x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
        } else {
            const uint4 a = ld(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(row) + d0));
            const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                x[2 * e] = __uint_as_float(w[e] << 16);
                x[2 * e + 1] = __uint_as_float(w[e] & 0xffff0000u);
            }
        }
        return;
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        x[e] = 0.f;
        if (d0 + e < D) {
            if constexpr (F32) x[e] = ld(static_cast<const float*>(row) + d0 + e);
            else x[e] = __uint_as_float(static_cast<uint32_t>(ld(static_cast<const uint16_t*>(row) + d0 + e)) << 16);
        }
    }
}

// lo + step c of eight codes.  A code becomes a float as the low bits of 2^23 + c.
template <int BITS>
__device__ __forceinline__ void expand8(const uint32_t* code, float step, float lo, float* x)
{
    constexpr float kTwo23 = 8388608.f;
    const uint32_t even = BITS == 4 ? code[0] & 0x0f0f0f0fu : 0, odd = BITS == 4 ? (code[0] >> 4) & 0x0f0f0f0fu : 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const uint32_t w = BITS == 4 ? (e & 1 ? odd : even) : code[e >> 2];
        const float c = __uint_as_float(__byte_perm(w, 0x4B000000u, 0x7540 + (BITS == 4 ? e >> 1 : e & 3))) - kTwo23;
        x[e] = fmaf(step, c, lo);
    }
}

__device__ __forceinline__ float4 f4(const float* p) { return *reinterpret_cast<const float4*>(p); }
__device__ __forceinline__ float dot4(float4 a, float4 b, float c)
{
    return fmaf(a.w, b.w, fmaf(a.z, b.z, fmaf(a.y, b.y, fmaf(a.x, b.x, c))));
}
__device__ __forceinline__ void put8(float* dst, const float* x)
{
    reinterpret_cast<float4*>(dst)[0] = make_float4(x[0], x[1], x[2], x[3]);
    reinterpret_cast<float4*>(dst)[1] = make_float4(x[4], x[5], x[6], x[7]);
}

}  // namespace txl
