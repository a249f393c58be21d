// txl_qmem_attn.cu -- relative attention of 1 .. 16 queries over a quantised memory and the segment's
// own keys: the generation step over a memory of 4- or 8-bit codes.
//
//     s_ij = scale [ (q_i+u).k'_j + (q_i+v).r[min(M+i-j, C)] ],  out_i = softmax_j(s_ij) v'_j
// with k'_jd = lo + step c_jd for memory keys and the segment's own k, v unquantised.
//
// One block per (query, head, batch entry): the keys in chunks of one per thread, the codes expanded
// in registers, an online softmax over the chunks in fp32.
#include <cuda_bf16.h>

#include "txl_internal.h"
#include "txl_ptx.cuh"

namespace txl {

namespace {

constexpr int kThreads = 128;

__device__ __forceinline__ float ld_elem(const void* p, int64_t i, int f32)
{
    return f32 ? __ldg(static_cast<const float*>(p) + i)
               : __uint_as_float(static_cast<uint32_t>(__ldg(static_cast<const uint16_t*>(p) + i)) << 16);
}

// channel d of a code row
__device__ __forceinline__ float code_at(const uint8_t* row, int d, int bits)
{
    return static_cast<float>(bits == 4 ? (row[d >> 1] >> (4 * (d & 1))) & 15 : row[d]);
}

__global__ void __launch_bounds__(kThreads) qattn_kernel(const __grid_constant__ QattnParams p)
{
    __shared__ float qu[128], qv[128], ps[kThreads], red[kThreads / 32];
    pdl_launch_dependents();
    pdl_wait();
    const int i = blockIdx.x, h = blockIdx.y, b = blockIdx.z, tid = threadIdx.x;
    if (tid < p.D) {
        const float q = ld_elem(p.q, b * p.q_sb + i * p.q_st + h * p.q_sh + tid, p.f32);
        qu[tid] = (q + p.u[h * p.D + tid]) * p.qscale;
        qv[tid] = (q + p.vb[h * p.D + tid]) * p.qscale;
    }
    __syncthreads();
    const int K = p.M + i + 1;                     // keys this query sees
    const int row_bytes = 4 * p.G * p.bits;
    float m = -INFINITY, l = 0.f, o = 0.f;
    for (int j0 = p.lo; j0 < K; j0 += kThreads) {
        const int j = j0 + tid;
        float s = -INFINITY;
        if (j < K) {
            s = 0.f;
            const int64_t rr = static_cast<int64_t>(min(p.M + i - j, p.C)) * p.r_row + h * p.r_head;
            if (j < p.M) {
                const int slot = static_cast<int>((static_cast<int64_t>(p.wp) + j) % p.M);
                const int64_t row = (static_cast<int64_t>(b) * p.H + h) * p.M + slot;
                for (int d = 0; d < p.D; ++d) {
                    const uint16_t* par = p.par + (row * p.G + d / kQGroup) * 4;
                    const float step = __uint_as_float(static_cast<uint32_t>(par[0]) << 16);
                    const float lo = __uint_as_float(static_cast<uint32_t>(par[1]) << 16);
                    s = fmaf(qu[d], fmaf(step, code_at(p.k + row * row_bytes, d, p.bits), lo), s);
                }
            } else {
                for (int d = 0; d < p.D; ++d)
                    s = fmaf(qu[d], ld_elem(p.kcur, b * p.kc_sb + (j - p.M) * p.kc_st + h * p.kc_sh + d, p.f32), s);
            }
            for (int d = 0; d < p.D; ++d) s = fmaf(qv[d], ld_elem(p.r, rr + d, p.f32), s);
        }
        float x = s;
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, off));
        __syncthreads();
        if ((tid & 31) == 0) red[tid >> 5] = x;
        __syncthreads();
        const float mn = fmaxf(fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3])), m);
        ps[tid] = exp2f(s - mn);
        __syncthreads();
        const float w = exp2f(m - mn);
        m = mn;
        l *= w;
        o *= w;
        const int n = min(kThreads, K - j0);
        for (int t = 0; t < n; ++t) {
            const float pr = ps[t];
            l += pr;
            if (tid < p.D) {
                const int jt = j0 + t;
                float v;
                if (jt < p.M) {
                    const int slot = static_cast<int>((static_cast<int64_t>(p.wp) + jt) % p.M);
                    const int64_t row = (static_cast<int64_t>(b) * p.H + h) * p.M + slot;
                    const uint16_t* par = p.par + (row * p.G + tid / kQGroup) * 4;
                    v = fmaf(__uint_as_float(static_cast<uint32_t>(par[2]) << 16), code_at(p.v + row * row_bytes, tid, p.bits),
                             __uint_as_float(static_cast<uint32_t>(par[3]) << 16));
                } else {
                    v = ld_elem(p.vcur, b * p.vc_sb + (jt - p.M) * p.vc_st + h * p.vc_sh + tid, p.f32);
                }
                o = fmaf(pr, v, o);
            }
        }
    }
    if (tid < p.D) {
        const int64_t at = b * p.o_sb + i * p.o_st + h * p.o_sh + tid;
        if (p.f32) static_cast<float*>(p.out)[at] = o / l;
        else static_cast<__nv_bfloat16*>(p.out)[at] = __float2bfloat16_rn(o / l);
    }
}

}  // namespace

cudaError_t launch_qattn(const QattnParams& p, int, cudaStream_t s)
{
    return launch_dependent(qattn_kernel, dim3(p.L, p.H, p.B), dim3(kThreads), 0, s, p);
}

}  // namespace txl
