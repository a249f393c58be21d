// txl_paged.cuh -- addressing of a memory held in pages and the entry of new positions, shared by its kernels.
#pragma once

#include <cstdint>

#include "txl_internal.h"

namespace txl {

// New positions of sequence b that a call brings.
__device__ __forceinline__ int paged_count(const int* counts, int b, int T)
{
    return counts ? min(max(counts[b], 0), T) : T;
}

// The page of slot s of sequence b, or -1 where the sequence has none there.
__device__ __forceinline__ int page_of(const PagedParams& m, int b, int s)
{
    const int i = s / m.page_len;
    if (i >= m.max_pages) return -1;
    const int page = m.table[static_cast<int64_t>(b) * m.max_pages + i];
    return static_cast<unsigned>(page) < static_cast<unsigned>(m.n_pages) ? page : -1;
}

// First element of head h in a page.
__device__ __forceinline__ int64_t page_row0(const PagedParams& m, int page, int h)
{
    return (static_cast<int64_t>(page) * m.H + h) * m.page_len * m.ld;
}

__device__ __forceinline__ void page_error(const PagedParams& m)
{
    if (m.err_flag) atomicCAS(m.err_flag, 0, static_cast<int>(TXL_ERR_PAGE));
}

// Whether slots len .. len + n - 1 of sequence b all have a page (the whole block asks; n > 0).
__device__ __forceinline__ bool paged_room(const PagedParams& m, int b, int len, int n)
{
    bool ok = len >= 0 && static_cast<int64_t>(len) + n <= static_cast<int64_t>(m.max_pages) * m.page_len;
    if (ok)
        for (int i = len / m.page_len + static_cast<int>(threadIdx.x); i <= (len + n - 1) / m.page_len;
             i += static_cast<int>(blockDim.x))
            ok = ok && page_of(m, b, i * m.page_len) >= 0;
    return __syncthreads_and(ok) != 0;
}

// Rows t0 .. t1-1 of sequence b into its slots len + t: keys, values, positions; the weights start at 0.  Every
// slot has its page.  Rows are copied in units of 16 bytes; the channels D .. ld-1 are written as zeros.  A thread keeps its
// unit of a position and goes over the positions, four loaded before the first is stored.
template <typename T>
__device__ __forceinline__ void paged_copy(const PagedPushParams& p, int b, int len, int next, int t0, int t1)
{
    constexpr int kUnit = 16 / sizeof(T), kAtOnce = 4;
    const PagedParams& m = p.m;
    const int units = m.ld / kUnit, per = m.H * units, side = max(1, static_cast<int>(blockDim.x) / per);
    const int first = threadIdx.x / per;                      // of the positions that the block takes side by side
    auto load = [&](const T* src, int c, bool vec) {
        union { uint4 all; T one[kUnit]; } u;
        if (vec && (c + 1) * kUnit <= m.D) {
            u.all = *reinterpret_cast<const uint4*>(src + c * kUnit);
        } else {
            u.all = make_uint4(0, 0, 0, 0);
#pragma unroll
            for (int e = 0; e < kUnit; ++e)
                if (c * kUnit + e < m.D) u.one[e] = src[c * kUnit + e];
        }
        return u.all;
    };
    for (int z = threadIdx.x - first * per; first < side && z < per; z += blockDim.x) {
        const int h = z / units, c = z - h * units;
        const T* k = static_cast<const T*>(p.xk) + b * p.xk_sb + h * p.xk_sh;
        const T* v = static_cast<const T*>(p.xv) + b * p.xv_sb + h * p.xv_sh;
        for (int t = t0 + first; t < t1; t += kAtOnce * side) {
            uint4 w[kAtOnce][2];
#pragma unroll
            for (int i = 0; i < kAtOnce; ++i)
                if (t + i * side < t1) {
                    w[i][0] = load(k + (t + i * side) * p.xk_st, c, p.vec_k);
                    w[i][1] = load(v + (t + i * side) * p.xv_st, c, p.vec_v);
                }
#pragma unroll
            for (int i = 0; i < kAtOnce; ++i)
                if (t + i * side < t1) {
                    const int slot = len + t + i * side;
                    const int64_t at = page_row0(m, page_of(m, b, slot), h) + static_cast<int64_t>(slot % m.page_len) * m.ld + c * kUnit;
                    *reinterpret_cast<uint4*>(static_cast<T*>(m.k) + at) = w[i][0];
                    *reinterpret_cast<uint4*>(static_cast<T*>(m.v) + at) = w[i][1];
                }
        }
    }
    for (int t = t0 + static_cast<int>(threadIdx.x); t < t1; t += blockDim.x) {
        const int slot = len + t;
        const int64_t at = static_cast<int64_t>(page_of(m, b, slot)) * m.page_len + slot % m.page_len;
        m.pos[at] = next + t;
        m.weight[at] = 0.f;
    }
}

}  // namespace txl
