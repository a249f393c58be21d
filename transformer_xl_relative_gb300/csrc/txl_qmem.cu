// txl_qmem.cu -- the FIFO K/V memory held as 4- or 8-bit codes: quantised as it is written
// (txl_qmem_push) and read back (txl_qmem_read).
//
// A group is 32 consecutive channels of one position and head; n = 2^bits - 1:
//     lo = bf16 floor of min(x),  step = bf16 ceiling of (max(x) - lo) / n,
//     c_d = nearest integer to (x_d - lo) / step (ties to even),  x'_d = lo + step c_d.
// Rounding step up makes n step >= max - lo, so no code is clipped and |x' - x| <= step / 2; a bf16
// minimum is its own floor, so bf16 inputs lose nothing in lo.  lo and step take 16 bits each: 4-bit
// codes cost 5 bits per channel in all.  The definitions are met exactly: fp32 estimates are
// corrected where the exact value could lie on the other side of a border (all comparisons below
// are between exactly represented numbers).
//
// Both kernels are bound by HBM.  Four lanes share a group, eight channels each: 16-byte accesses to
// bf16 rows, and consecutive threads walk the groups of a row, then the positions of one head, which
// are contiguous in the code arrays.
#include <cuda_bf16.h>

#include "txl_internal.h"
#include "txl_ptx.cuh"

namespace txl {

namespace {

constexpr int kQThreads = 256;
constexpr float kTwo64 = 18446744073709551616.f;

__device__ __forceinline__ float bf16_floor(float x)
{
    const uint32_t b = __float_as_uint(x), t = b & 0xffff0000u;
    return __uint_as_float(t + (t != b && (b >> 31) ? 0x10000u : 0u));
}

// x >= 0, not NaN
__device__ __forceinline__ float bf16_ceil_pos(float x)
{
    return __uint_as_float((__float_as_uint(x) + 0xffffu) & 0xffff0000u);
}

// Eight channels d0 .. d0+7 of a row; channels at or past D read as `fill`.
template <bool F32>
__device__ __forceinline__ void load8(const void* row, int d0, int D, bool vec, float fill, float* x)
{
    if (vec && d0 + 8 <= D) {
        if constexpr (F32) {
            const float4* q = reinterpret_cast<const float4*>(static_cast<const float*>(row) + d0);
            const float4 a = __ldg(q), b = __ldg(q + 1);
            x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
            x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
        } else {
            const uint4 a = __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(row) + d0));
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
        x[e] = fill;
        if (d0 + e < D) {
            if constexpr (F32) x[e] = __ldg(static_cast<const float*>(row) + d0 + e);
            else x[e] = __uint_as_float(static_cast<uint32_t>(__ldg(static_cast<const uint16_t*>(row) + d0 + e)) << 16);
        }
    }
}

template <bool F32>
__device__ __forceinline__ void store8(void* row, int d0, int D, bool vec, const float* x)
{
    if (vec && d0 + 8 <= D) {
        if constexpr (F32) {
            float4* q = reinterpret_cast<float4*>(static_cast<float*>(row) + d0);
            q[0] = make_float4(x[0], x[1], x[2], x[3]);
            q[1] = make_float4(x[4], x[5], x[6], x[7]);
        } else {
            *reinterpret_cast<uint4*>(static_cast<uint16_t*>(row) + d0) =
                make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                           pack_bf16x2(x[6], x[7]));
        }
        return;
    }
#pragma unroll
    for (int e = 0; e < 8; ++e)
        if (d0 + e < D) {
            if constexpr (F32) static_cast<float*>(row)[d0 + e] = x[e];
            else static_cast<__nv_bfloat16*>(row)[d0 + e] = __float2bfloat16_rn(x[e]);
        }
}

// One lane's part (eight channels, `live` of them inside D) of quantising a group shared by four
// consecutive lanes.  Returns the codes and the group's step and lo.
template <int BITS>
__device__ __forceinline__ void quantise8(const float* x, int live, uint32_t* code, float& step, float& lo)
{
    constexpr float n = static_cast<float>((1 << BITS) - 1);
    float mn = INFINITY, mx = -INFINITY;
    bool bad = false;
#pragma unroll
    for (int e = 0; e < 8; ++e)
        if (e < live) {
            mn = fminf(mn, x[e]);
            mx = fmaxf(mx, x[e]);
            bad |= !(fabsf(x[e]) < INFINITY);
        }
#pragma unroll
    for (int off = 1; off <= 2; off <<= 1) {
        mn = fminf(mn, __shfl_xor_sync(0xffffffffu, mn, off));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
        bad |= __shfl_xor_sync(0xffffffffu, bad ? 1 : 0, off) != 0;
    }
    lo = bf16_floor(mn);
    // max - lo = span + err exactly
    const float span = mx - lo;
    const float bb = span - mx;
    const float err = (mx - (span - bb)) + (-lo - bb);
    auto below = [&](float s) {                        // s n < max - lo, exactly (s has 8 bits, n at most 8)
        const float p = s * n;
        return p < span || (p == span && err > 0.f);
    };
    step = bf16_ceil_pos(span * (1.f / n));
    const float down = __uint_as_float(__float_as_uint(step) - (step > 0.f ? 0x10000u : 0u));
    if (below(step)) step = __uint_as_float(__float_as_uint(step) + 0x10000u);
    else if (!below(down)) step = down;
    bad |= !(span < INFINITY) || !(lo > -INFINITY);    // (then step = span / n is finite too)
    if (bad) step = lo = __uint_as_float(0x7fc00000u);

    // quotients from the reciprocal (a tiny step scaled up first, so that it has one); within 1e-4 of
    // the exact quotient, so only those near a half need the exact comparison with (c + 1/2) step
    const float sc = step < 1e-30f ? kTwo64 : 1.f;
    const float inv = step > 0.f ? 1.f / (step * sc) : 0.f;
    uint32_t c[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const float d = x[e] - lo;
        const float t = d * sc * inv;
        float r = rintf(t);
        if (fabsf(t - r) > 0.499f && e < live) {
            const float base = floorf(t);
            const float diff = d - (base + 0.5f) * step;           // exact: both sides agree to a factor of 2
            const float b2 = d - x[e];
            const float lost = (x[e] - (d - b2)) + (-lo - b2);     // x - lo = d + lost exactly
            const bool up = diff > 0.f || (diff == 0.f && lost > 0.f);
            const bool tie = diff == 0.f && lost == 0.f;
            r = up ? base + 1.f : base;
            if (tie) r = 2.f * rintf(0.5f * base) == base ? base : base + 1.f;
        }
        c[e] = e < live && !bad ? static_cast<uint32_t>(r) : 0u;
    }
    if constexpr (BITS == 4) {
        code[0] = c[0] | c[1] << 4 | c[2] << 8 | c[3] << 12 | c[4] << 16 | c[5] << 20 | c[6] << 24 | c[7] << 28;
    } else {
        code[0] = c[0] | c[1] << 8 | c[2] << 16 | c[3] << 24;
        code[1] = c[4] | c[5] << 8 | c[6] << 16 | c[7] << 24;
    }
}

// (step, lo) as the bf16 pair a parameter word holds; both are bf16 values already
__device__ __forceinline__ uint32_t par_word(float step, float lo)
{
    return (__float_as_uint(step) >> 16) | (__float_as_uint(lo) & 0xffff0000u);
}

// Byte offset, in the code arrays, of the eight channels from d0 of a row.
template <int BITS, int G>
__device__ __forceinline__ int64_t code_at(int64_t row, int slot, int d0)
{
    constexpr int NC = G * BITS / 4;
    const int byte = d0 * BITS / 8;
    return row * (16 * NC) + ((((byte >> 4) ^ q_swizzle(NC, slot)) << 4) | (byte & 15));
}

struct QPos {
    int64_t row;          // row of the code and parameter arrays
    int slot;
    int t, g, d0;         // position of the segment, group, first channel of the lane
};

// Grid: (ceil(n * G * 4 / kQThreads), H, B); consecutive threads take the lanes of a row's groups,
// then the next position of the same head.
template <int G>
__device__ __forceinline__ bool q_pos(const QmemParams& p, int64_t i, QPos& o)
{
    const int64_t t = i / (4 * G);
    const int rem = static_cast<int>(i - t * (4 * G));
    o.t = static_cast<int>(t);
    o.g = rem >> 2;
    o.d0 = o.g * kQGroup + (rem & 3) * 8;
    int64_t slot = p.slot0 + t;
    if (slot >= p.M) slot -= p.M;
    const bool live = t < p.n;
    if (live && !in_range(slot, 0, p.M, p.chk)) slot = 0;
    o.slot = static_cast<int>(slot);
    o.row = (static_cast<int64_t>(blockIdx.z) * p.H + blockIdx.y) * p.M + slot;
    return live;
}

template <int BITS, int G, bool F32>
__global__ void __launch_bounds__(kQThreads) qmem_push_kernel(const __grid_constant__ QmemParams p)
{
    pdl_launch_dependents();
    pdl_wait();
    QPos o;
    const int64_t i = static_cast<int64_t>(blockIdx.x) * kQThreads + threadIdx.x;
    const bool on = q_pos<G>(p, i, o);                 // the four lanes of a group are on or off together
    constexpr int E = F32 ? 4 : 2;
    float xk[8], xv[8];
    const int live = on ? min(max(p.D - o.d0, 0), 8) : 0;
    const int64_t t = p.t0 + o.t;
    if (on) {
        const char* rk = static_cast<const char*>(p.xk) + (blockIdx.z * p.xk_sb + t * p.xk_st + blockIdx.y * p.xk_sh) * E;
        const char* rv = static_cast<const char*>(p.xv) + (blockIdx.z * p.xv_sb + t * p.xv_st + blockIdx.y * p.xv_sh) * E;
        load8<F32>(rk, o.d0, p.D, p.vec_k, 0.f, xk);
        load8<F32>(rv, o.d0, p.D, p.vec_v, 0.f, xv);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) xk[e] = xv[e] = 0.f;
    }
    uint32_t ck[2], cv[2];
    float ks, kl, vs, vl;
    quantise8<BITS>(xk, live, ck, ks, kl);
    quantise8<BITS>(xv, live, cv, vs, vl);
    if (!on) return;
    const int64_t at = code_at<BITS, G>(o.row, o.slot, o.d0);
    if constexpr (BITS == 4) {
        *reinterpret_cast<uint32_t*>(p.k + at) = ck[0];
        *reinterpret_cast<uint32_t*>(p.v + at) = cv[0];
    } else {
        *reinterpret_cast<uint2*>(p.k + at) = make_uint2(ck[0], ck[1]);
        *reinterpret_cast<uint2*>(p.v + at) = make_uint2(cv[0], cv[1]);
    }
    if ((o.d0 & (kQGroup - 1)) == 0) {
        uint2* par = reinterpret_cast<uint2*>(p.par + o.row * q_par_groups(G) * 4) + o.g;
        *par = make_uint2(par_word(ks, kl), par_word(vs, vl));
        if (G < q_par_groups(G) && o.g == G - 1) par[1] = make_uint2(0, 0);     // the group that fills the row up
    }
}

template <int BITS>
__device__ __forceinline__ void expand8(const uint32_t* code, uint32_t par, float* x)
{
    const float step = __uint_as_float(par << 16), lo = __uint_as_float(par & 0xffff0000u);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const uint32_t c = BITS == 4 ? (code[0] >> (4 * e)) & 15u : (code[e >> 2] >> (8 * (e & 3))) & 255u;
        x[e] = fmaf(step, static_cast<float>(c), lo);
    }
}

template <int BITS, int G, bool F32>
__global__ void __launch_bounds__(kQThreads) qmem_read_kernel(const __grid_constant__ QmemParams p)
{
    pdl_launch_dependents();
    pdl_wait();
    QPos o;
    const int64_t i = static_cast<int64_t>(blockIdx.x) * kQThreads + threadIdx.x;
    if (!q_pos<G>(p, i, o)) return;
    constexpr int E = F32 ? 4 : 2;
    const int64_t at = code_at<BITS, G>(o.row, o.slot, o.d0);
    uint32_t ck[2], cv[2];
    if constexpr (BITS == 4) {
        ck[0] = __ldg(reinterpret_cast<const uint32_t*>(p.k + at));
        cv[0] = __ldg(reinterpret_cast<const uint32_t*>(p.v + at));
    } else {
        const uint2 a = __ldg(reinterpret_cast<const uint2*>(p.k + at)), b = __ldg(reinterpret_cast<const uint2*>(p.v + at));
        ck[0] = a.x; ck[1] = a.y; cv[0] = b.x; cv[1] = b.y;
    }
    const uint2 par = __ldg(reinterpret_cast<const uint2*>(p.par + (o.row * q_par_groups(G) + o.g) * 4));
    float xk[8], xv[8];
    expand8<BITS>(ck, par.x, xk);
    expand8<BITS>(cv, par.y, xv);
    const int64_t t = o.t;
    char* rk = static_cast<char*>(p.xk) + (blockIdx.z * p.xk_sb + t * p.xk_st + blockIdx.y * p.xk_sh) * E;
    char* rv = static_cast<char*>(p.xv) + (blockIdx.z * p.xv_sb + t * p.xv_st + blockIdx.y * p.xv_sh) * E;
    store8<F32>(rk, o.d0, p.D, p.vec_k, xk);
    store8<F32>(rv, o.d0, p.D, p.vec_v, xv);
}

// The operands of the fused attention kernels in fp16, which keeps 11 bits where bf16 keeps 8: K and V
// of the memory and of the segment, and r.  Each takes its range from a power of two, the unit: the
// largest |k| of a (b, h) comes into [1, 2) (its unit multiplies c(q+u)), the largest |v| into
// [2^11, 2^12) (P of the attention goes up to 2^8), and the largest |r| of 64 rows of the head into [1, 2)
// (rows of up to 2^15 times that size have room).  One cluster per (b, h); each CTA takes a share of the rows, first for
// the largest values (a group's end points bound its values, so the parameters suffice for the memory),
// then to write.  Rows are taken four at a time per thread, the loads first.
constexpr int kXThreads = 256;
constexpr int kXRows = 4;

template <int BITS, int G>
__global__ void __launch_bounds__(kXThreads) qmem_expand_kernel(const __grid_constant__ QexpandParams p, int ranks)
{
    __shared__ float red[3][kXThreads / 32];
    __shared__ float rank_max[2];
    pdl_launch_dependents();
    pdl_wait();
    const int tid = threadIdx.x, rank = blockIdx.x, h = blockIdx.y, b = blockIdx.z;
    const int64_t bh = static_cast<int64_t>(b) * p.H + h;
    auto share = [](int64_t n, int64_t part, int64_t parts) { return static_cast<int>(n * part / parts); };
    const int r0 = share(p.n, rank, ranks), r1 = share(p.n, rank + 1, ranks);
    const int s0 = share(p.L, rank, ranks), s1 = share(p.L, rank + 1, ranks);
    auto slot_of = [&](int t) {
        int64_t s = static_cast<int64_t>(p.slot0) + t;
        if (s >= p.M) s -= p.M;
        if (!in_range(s, 0, p.M, p.chk)) s = 0;
        return static_cast<int>(s);
    };
    auto seg = [&](const void* x, int64_t sb, int64_t st, int64_t sh, int t) {
        return static_cast<const uint16_t*>(x) + b * sb + t * st + h * sh;
    };
    constexpr int LPR = 4 * G;                            // lanes of a row, eight channels each
    constexpr int RPP = kXThreads / LPR;                  // rows of a pass
    const int lr = tid / LPR, c = tid % LPR, d0 = 8 * c;
    const bool lane_on = lr < RPP && d0 < p.D;

    float mx[3] = {0.f, 0.f, 0.f};                        // k, v, r; values that are not finite do not count
    auto see = [&](int which, float a) {
        if (a < INFINITY) mx[which] = fmaxf(mx[which], a);
    };
    const int64_t x1 = static_cast<int64_t>(r1) * G;
#pragma unroll 4
    for (int64_t x = static_cast<int64_t>(r0) * G + tid; x < x1; x += kXThreads) {
        const int t = static_cast<int>(x / G), g = static_cast<int>(x - static_cast<int64_t>(t) * G);
        const uint2 w = __ldg(reinterpret_cast<const uint2*>(p.par + ((bh * p.M + slot_of(t)) * q_par_groups(G) + g) * 4));
        const uint32_t kv[2] = {w.x, w.y};
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const float step = __uint_as_float(kv[i] << 16), lo = __uint_as_float(kv[i] & 0xffff0000u);
            see(i, fmaxf(fabsf(lo), fabsf(fmaf(step, static_cast<float>((1 << BITS) - 1), lo))));
        }
    }
    if (lane_on)
#pragma unroll 2
        for (int t = s0 + lr; t < s1; t += RPP) {
            float xk[8], xv[8];
            load8<false>(seg(p.kcur, p.kc_sb, p.kc_st, p.kc_sh, t), d0, p.D, p.vec_k, 0.f, xk);
            load8<false>(seg(p.vcur, p.vc_sb, p.vc_st, p.vc_sh, t), d0, p.D, p.vec_v, 0.f, xv);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                see(0, fabsf(xk[e]));
                see(1, fabsf(xv[e]));
            }
        }
    const int samples = min(p.n_r, 64);                   // the same rows in every CTA of the head
    if (lane_on)
        for (int i = lr; i < samples; i += RPP) {
            const int64_t row = static_cast<int64_t>(share(p.n_r - 1, i, max(samples - 1, 1))) * p.H + h;
            float x[8];
            load8<false>(p.r + row * p.ld_r, d0, p.D, p.vec_r, 0.f, x);
#pragma unroll
            for (int e = 0; e < 8; ++e) see(2, fabsf(x[e]));
        }
    float inv[3];
#pragma unroll
    for (int i = 0; i < 3; ++i) {
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) mx[i] = fmaxf(mx[i], __shfl_xor_sync(0xffffffffu, mx[i], off));
        if ((tid & 31) == 0) red[i][tid >> 5] = mx[i];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 3; ++i) {
#pragma unroll
        for (int w = 0; w < kXThreads / 32; ++w) mx[i] = fmaxf(mx[i], red[i][w]);
        if (tid == 0 && i < 2) rank_max[i] = mx[i];
    }
    if (ranks > 1) {
        __syncthreads();
        cluster_sync_all();
        for (int r = 0; r < ranks; ++r) {
            mx[0] = fmaxf(mx[0], ld_rank(&rank_max[0], r));
            mx[1] = fmaxf(mx[1], ld_rank(&rank_max[1], r));
        }
    }
#pragma unroll
    for (int i = 0; i < 3; ++i) {
        const int ex = min(max(static_cast<int>(__float_as_uint(mx[i]) >> 23) - 127 - (i == 1 ? 11 : 0), -115), 115);
        inv[i] = __uint_as_float(static_cast<uint32_t>(127 - ex) << 23);
        if (rank == 0 && tid == 0) p.units[4 * bh + i] = __uint_as_float(static_cast<uint32_t>(127 + ex) << 23);
    }

    auto put = [&](void* base, int64_t row, const float* x, float f) {
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(base) + row * p.ld + d0) =
            make_uint4(pack_f16x2(x[0] * f, x[1] * f), pack_f16x2(x[2] * f, x[3] * f), pack_f16x2(x[4] * f, x[5] * f),
                       pack_f16x2(x[6] * f, x[7] * f));
    };
    if (lane_on) {
        for (int t0 = r0 + lr; t0 < r1; t0 += kXRows * RPP) {
            uint32_t ck[kXRows][2], cv[kXRows][2];
            uint2 par[kXRows];
#pragma unroll
            for (int k = 0; k < kXRows; ++k) {
                const int t = t0 + k * RPP;
                if (t >= r1) break;
                const int slot = slot_of(t);
                const int64_t row = bh * p.M + slot, at = code_at<BITS, G>(row, slot, d0);
                if constexpr (BITS == 4) {
                    ck[k][0] = __ldg(reinterpret_cast<const uint32_t*>(p.k + at));
                    cv[k][0] = __ldg(reinterpret_cast<const uint32_t*>(p.v + at));
                } else {
                    const uint2 a = __ldg(reinterpret_cast<const uint2*>(p.k + at));
                    const uint2 w = __ldg(reinterpret_cast<const uint2*>(p.v + at));
                    ck[k][0] = a.x; ck[k][1] = a.y; cv[k][0] = w.x; cv[k][1] = w.y;
                }
                par[k] = __ldg(reinterpret_cast<const uint2*>(p.par + (row * q_par_groups(G) + (c >> 2)) * 4));
            }
#pragma unroll
            for (int k = 0; k < kXRows; ++k) {
                const int t = t0 + k * RPP;
                if (t >= r1) break;
                float x[8];
                expand8<BITS>(ck[k], par[k].x, x);
                put(p.k_mem, bh * p.n + t, x, inv[0]);
                expand8<BITS>(cv[k], par[k].y, x);
                put(p.v_mem, bh * p.n + t, x, inv[1]);
            }
        }
#pragma unroll 2
        for (int t = s0 + lr; t < s1; t += RPP) {
            float x[8];
            load8<false>(seg(p.kcur, p.kc_sb, p.kc_st, p.kc_sh, t), d0, p.D, p.vec_k, 0.f, x);
            put(p.k_seg, bh * p.L + t, x, inv[0]);
            load8<false>(seg(p.vcur, p.vc_sb, p.vc_st, p.vc_sh, t), d0, p.D, p.vec_v, 0.f, x);
            put(p.v_seg, bh * p.L + t, x, inv[1]);
            if (p.q_seg) {
                load8<false>(seg(p.q, p.q_sb, p.q_st, p.q_sh, t), d0, p.D, p.vec_q, 0.f, x);
                store8<false>(static_cast<uint16_t*>(p.q_seg) + (bh * p.L + t) * p.ld, d0, p.ld, true, x);
            }
        }
        // this head's rows of r, shared out over the batch entries and ranks
        const int64_t part = static_cast<int64_t>(b) * ranks + rank, parts = static_cast<int64_t>(p.B) * ranks;
        for (int t = share(p.n_r, part, parts) + lr; t < share(p.n_r, part + 1, parts); t += RPP) {
            float x[8];
            const int64_t row = static_cast<int64_t>(t) * p.H + h;
            load8<false>(p.r + row * p.ld_r, d0, p.D, p.vec_r, 0.f, x);
            *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.r16) + row * p.ld + d0) =
                make_uint4(pack_f16x2_sat(x[0] * inv[2], x[1] * inv[2]), pack_f16x2_sat(x[2] * inv[2], x[3] * inv[2]),
                           pack_f16x2_sat(x[4] * inv[2], x[5] * inv[2]), pack_f16x2_sat(x[6] * inv[2], x[7] * inv[2]));
        }
    }
    __syncthreads();
    if (ranks > 1) cluster_sync_all();                    // rank_max stays until every rank has read it
}

template <int BITS, int G>
cudaError_t launch_expand(const QexpandParams& p, int ranks, cudaStream_t s)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(ranks, p.H, p.B);
    cfg.blockDim = dim3(kXThreads);
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = ranks;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, qmem_expand_kernel<BITS, G>, p, ranks);
}

template <int BITS, int G>
cudaError_t launch(const QmemParams& p, bool f32, bool push, cudaStream_t s)
{
    const int64_t units = static_cast<int64_t>(p.n) * G * 4;
    const int64_t blocks = (units + kQThreads - 1) / kQThreads;
    if (blocks > INT32_MAX) return cudaErrorInvalidValue;
    const dim3 grid(static_cast<unsigned>(blocks), p.H, p.B);
    auto* kernel = push ? (f32 ? qmem_push_kernel<BITS, G, true> : qmem_push_kernel<BITS, G, false>)
                        : (f32 ? qmem_read_kernel<BITS, G, true> : qmem_read_kernel<BITS, G, false>);
    return launch_dependent(kernel, grid, dim3(kQThreads), 0, s, p);
}

cudaError_t launch_any(const QmemParams& p, txl_dtype dtype, bool push, cudaStream_t s)
{
    const bool f32 = dtype == TXL_F32;
    switch (p.G * 16 + p.bits) {
    case 1 * 16 + 4: return launch<4, 1>(p, f32, push, s);
    case 2 * 16 + 4: return launch<4, 2>(p, f32, push, s);
    case 3 * 16 + 4: return launch<4, 3>(p, f32, push, s);
    case 4 * 16 + 4: return launch<4, 4>(p, f32, push, s);
    case 1 * 16 + 8: return launch<8, 1>(p, f32, push, s);
    case 2 * 16 + 8: return launch<8, 2>(p, f32, push, s);
    case 3 * 16 + 8: return launch<8, 3>(p, f32, push, s);
    case 4 * 16 + 8: return launch<8, 4>(p, f32, push, s);
    default: return cudaErrorInvalidValue;
    }
}

}  // namespace

cudaError_t launch_qmem_expand(const QexpandParams& p, int sm_count, cudaStream_t s)
{
    // CTAs per (b, h): until eight per SM, while each keeps 128 rows
    int ranks = 1;
    while (ranks < 8 && static_cast<int64_t>(p.B) * p.H * ranks < 8 * sm_count &&
           static_cast<int64_t>(p.n) + p.L > 128 * ranks)
        ranks *= 2;
    switch (p.G * 16 + (p.n > 0 ? p.bits : 4)) {
    case 1 * 16 + 4: return launch_expand<4, 1>(p, ranks, s);
    case 2 * 16 + 4: return launch_expand<4, 2>(p, ranks, s);
    case 3 * 16 + 4: return launch_expand<4, 3>(p, ranks, s);
    case 4 * 16 + 4: return launch_expand<4, 4>(p, ranks, s);
    case 1 * 16 + 8: return launch_expand<8, 1>(p, ranks, s);
    case 2 * 16 + 8: return launch_expand<8, 2>(p, ranks, s);
    case 3 * 16 + 8: return launch_expand<8, 3>(p, ranks, s);
    case 4 * 16 + 8: return launch_expand<8, 4>(p, ranks, s);
    default: return cudaErrorInvalidValue;
    }
}

cudaError_t launch_qmem_push(const QmemParams& p, txl_dtype dtype, cudaStream_t s)
{
    return launch_any(p, dtype, true, s);
}

cudaError_t launch_qmem_read(const QmemParams& p, txl_dtype dtype, cudaStream_t s)
{
    return launch_any(p, dtype, false, s);
}

}  // namespace txl
