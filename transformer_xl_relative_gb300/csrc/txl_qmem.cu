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
// Four lanes share a group, eight channels each: 16-byte accesses to bf16 rows, and consecutive threads walk the
// groups of a row, then the positions of one head, whose rows are contiguous.
//
// What bounds them: push, instructions (98304 rows of 64 bf16 channels to 4 bits: 18.0 us for 33 MB, 500
// instructions per warp at 73% of the issue slots; 4.9 us of HBM); read, HBM and the ramp (131072 rows of 128
// channels from 4 bits: 13.9 us for 88 MB, 6.3 TB/s).  Two units of work per thread in either cost more
// than the addresses they share (push 24 instead of 19.6 us).
#include <algorithm>

#include <cuda_bf16.h>

#include "txl_internal.h"
#include "txl_ptx.cuh"
#include "txl_rows.cuh"

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

__device__ __forceinline__ float min_nan(float a, float b)      // NaN if either is
{
    float r;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float max_nan(float a, float b)
{
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// Of both halves, NaN if either is
__device__ __forceinline__ uint32_t max2_nan(uint32_t a, uint32_t b)
{
    uint32_t r;
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

__device__ __forceinline__ uint32_t min2_nan(uint32_t a, uint32_t b)
{
    uint32_t r;
    asm("min.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// One lane's part (eight channels; ALL: every group is whole, else `live` of them inside D) of quantising
// a group shared by four consecutive lanes.  Returns the codes and the group's step and lo.
//
// Per channel: minimum and maximum (of bf16 inputs in pairs); d = x - lo; y = d / step + 1.5 2^23, whose low bits are
// the rounded quotient c; the remainder e = d - c step, which is exact, and its comparison; and a shift-add into the
// code word, the constant bits of the y subtracted once.  (In all 31 instructions per channel of a lane: the group's
// parameters, which each of its four lanes computes, addresses, conversions and near ties among them.)  Where |e|
// comes to half a step (bf16 inputs: one channel in 300 at 4 bits, exact ties) the channel is decided again, with what
// the subtraction x - lo lost.
template <int BITS, bool ALL, bool F32>
__device__ __forceinline__ void quantise8(const float* xin, int live, uint32_t* code, float& step, float& lo)
{
    constexpr float n = static_cast<float>((1 << BITS) - 1);
    constexpr float kMagic = 12582912.f;                    // 1.5 2^23
    constexpr uint32_t kMagicBits = 0x4B400000u;
    float x[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = xin[e];
    float mx;
    if constexpr (ALL && !F32) {
        uint32_t w[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) w[e] = __byte_perm(__float_as_uint(x[2 * e]), __float_as_uint(x[2 * e + 1]), 0x7632);
        const uint32_t a = max2_nan(max2_nan(w[0], w[1]), max2_nan(w[2], w[3]));
        const uint32_t c = min2_nan(min2_nan(w[0], w[1]), min2_nan(w[2], w[3])) ^ 0x80008000u;
        uint32_t both = max2_nan(__byte_perm(a, c, 0x5410), __byte_perm(a, c, 0x7632));     // (max, -min)
#pragma unroll
        for (int off = 1; off <= 2; off <<= 1) both = max2_nan(both, __shfl_xor_sync(0xffffffffu, both, off));
        mx = __uint_as_float(both << 16);
        lo = -__uint_as_float(both & 0xffff0000u);
    } else {
        float mn = ALL || live > 0 ? x[0] : INFINITY;
        mx = ALL || live > 0 ? x[0] : -INFINITY;
#pragma unroll
        for (int e = 1; e < 8; ++e)
            if (ALL || e < live) {
                mn = min_nan(mn, x[e]);
                mx = max_nan(mx, x[e]);
            }
#pragma unroll
        for (int off = 1; off <= 2; off <<= 1) {
            mn = min_nan(mn, __shfl_xor_sync(0xffffffffu, mn, off));
            mx = max_nan(mx, __shfl_xor_sync(0xffffffffu, mx, off));
        }
        lo = bf16_floor(mn);
    }
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
    // (a NaN or an infinity in the group, or a range that is not finite; otherwise step = span / n is finite too)
    const bool bad = !(span < INFINITY) || !(lo > -INFINITY);
    float st = step, l = lo;
    if (bad || !(step > 0.f)) {                        // every code is 0
        if (bad) step = lo = __uint_as_float(0x7fc00000u);
        code[0] = 0;
        if constexpr (BITS == 8) code[1] = 0;
        return;
    }
    if (step < 1e-30f) {                               // scaled up (exactly), so that its reciprocal is finite
        st *= kTwo64;
        l *= kTwo64;
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] *= kTwo64;
    }
    // inv is off by 2^-23 and d by 2^-24 of themselves, so that d inv (at most 256) is off by less than 2^-14:
    // a code that this rounds to the wrong side lies within that of half a step
    const float inv = rcp_approx(st);
    const float half = 0.5f * st, nearly = half * (1.f - 1.f / 4096.f);
    float y[8];
    uint32_t close = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const float d = x[e] - l;
        y[e] = fmaf(d, inv, kMagic);
        if (fabsf(fmaf(kMagic - y[e], st, d)) >= nearly) close |= 1u << e;
    }
    while (close) {                                        // one channel at a time: few lanes have any
        const uint32_t bit = close & (0u - close);
        close ^= bit;
        float xe = x[0], ye = y[0];
#pragma unroll
        for (int e = 1; e < 8; ++e) {
            xe = bit >> e & 1u ? x[e] : xe;
            ye = bit >> e & 1u ? y[e] : ye;
        }
        const float d = xe - l, b2 = d - xe;
        const float lost = (xe - (d - b2)) + (-l - b2);                    // x - lo = d + lost exactly
        const float rem = fmaf(kMagic - ye, st, d);
        const float over = fabsf(rem) - half;                              // exact: both are near half a step
        const float more = rem > 0.f ? lost : -lost;
        const bool past = over > 0.f || (over == 0.f && more > 0.f);       // |over| > |lost| unless over = 0
        const bool tie = over == 0.f && more == 0.f && (__float_as_uint(ye) & 1u);
        const float move = past || tie ? copysignf(1.f, rem) : 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (bit >> e & 1u) y[e] += move;
    }
    if constexpr (!ALL) {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (e >= live) y[e] = kMagic;
    }
    auto pack = [&](int e0, int count) {               // sum of y's bits, BITS apart, less their constant parts
        uint32_t w = 0, c = 0;
#pragma unroll
        for (int e = count - 1; e >= 0; --e) {
            w = (w << BITS) + __float_as_uint(y[e0 + e]);
            c = (c << BITS) + kMagicBits;
        }
        return w - c;
    };
    if constexpr (BITS == 4) {
        code[0] = pack(0, 8);
    } else {
        code[0] = pack(0, 4);
        code[1] = pack(4, 4);
    }
}

// (step, lo) as the bf16 pair a parameter word holds; both are bf16 values already
__device__ __forceinline__ uint32_t par_word(float step, float lo)
{
    return (__float_as_uint(step) >> 16) | (__float_as_uint(lo) & 0xffff0000u);
}

// Grid: (ceil(n / rows of a block), H, B); the lanes of a row's groups are consecutive, then the next position of
// the same head.  32-bit positions, 64-bit offsets from the head's first row.
template <int G> constexpr int kRowLanes = 4 * G;                      // eight channels each
template <int G> constexpr int kBlockRows = kQThreads / kRowLanes<G>;

struct QPos {
    uint8_t* row;         // of the memory
    int t, g, d0;         // position of the segment, group, first channel of the lane
};

template <int BITS, int G>
__device__ __forceinline__ bool q_pos(const QmemParams& p, QPos& o)
{
    const int lr = threadIdx.x / kRowLanes<G>, c = threadIdx.x % kRowLanes<G>;
    o.t = static_cast<int>(blockIdx.x) * kBlockRows<G> + lr;
    o.g = c >> 2;
    o.d0 = 8 * c;
    const bool live = lr < kBlockRows<G> && o.t < p.n;
    unsigned slot = static_cast<unsigned>(p.slot0) + o.t;              // below 2 M
    if (slot >= static_cast<unsigned>(p.M)) slot -= p.M;
    if (live && !in_range(slot, 0, p.M, p.chk)) slot = 0;
    uint8_t* head = p.rows + (static_cast<int64_t>(blockIdx.z) * p.H + blockIdx.y) * p.M * q_row_bytes(G, BITS);
    o.row = head + static_cast<uint64_t>(slot) * static_cast<unsigned>(q_row_bytes(G, BITS));
    return live;
}

template <int BITS, int G, bool F32>
__global__ void __launch_bounds__(kQThreads, 6) qmem_push_kernel(const __grid_constant__ QmemParams p)
{
    pdl_launch_dependents();
    pdl_wait();
    QPos o;
    const bool on = q_pos<BITS, G>(p, o);              // the four lanes of a group are on or off together
    constexpr int E = F32 ? 4 : 2;
    float xk[8], xv[8];
    const int live = on ? min(max(p.D - o.d0, 0), 8) : 0;
    const int64_t t = p.t0 + o.t;
    if (on) {
        const char* rk = static_cast<const char*>(p.xk) + (blockIdx.z * p.xk_sb + t * p.xk_st + blockIdx.y * p.xk_sh) * E;
        const char* rv = static_cast<const char*>(p.xv) + (blockIdx.z * p.xv_sb + t * p.xv_st + blockIdx.y * p.xv_sh) * E;
        load8<F32>(rk, o.d0, p.D, p.vec_k, xk);
        load8<F32>(rv, o.d0, p.D, p.vec_v, xv);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) xk[e] = xv[e] = 0.f;
    }
    float step[2], lo[2];
#pragma unroll
    for (int w = 0; w < 2; ++w) {
        const float* x = w ? xv : xk;
        uint32_t c[2];
        if (p.D == 32 * G) quantise8<BITS, true, F32>(x, 8, c, step[w], lo[w]);
        else quantise8<BITS, false, F32>(x, live, c, step[w], lo[w]);
        if (on) {
            uint8_t* dst = o.row + w * q_v_offset(G, BITS) + o.d0 * BITS / 8;
            if constexpr (BITS == 4) *reinterpret_cast<uint32_t*>(dst) = c[0];
            else *reinterpret_cast<uint2*>(dst) = make_uint2(c[0], c[1]);
        }
    }
    if (on && (o.d0 & (kQGroup - 1)) == 0) {
        uint2* par = reinterpret_cast<uint2*>(o.row + q_par_offset(G, BITS)) + o.g;
        *par = make_uint2(par_word(step[0], lo[0]), par_word(step[1], lo[1]));
        if (G % 2 && o.g == G - 1) par[1] = make_uint2(0, 0);      // the group that makes their number even
    }
}

// The codes of eight channels from d0 of a row, and their group's parameters.
template <int BITS, int G>
__device__ __forceinline__ uint2 row_unit(const uint8_t* row, int d0, uint32_t* ck, uint32_t* cv)
{
    const uint8_t* k = row + d0 * BITS / 8;
    const uint8_t* v = k + q_v_offset(G, BITS);
    if constexpr (BITS == 4) {
        ck[0] = ld(reinterpret_cast<const uint32_t*>(k));
        cv[0] = ld(reinterpret_cast<const uint32_t*>(v));
    } else {
        const uint2 a = ld(reinterpret_cast<const uint2*>(k)), b = ld(reinterpret_cast<const uint2*>(v));
        ck[0] = a.x; ck[1] = a.y; cv[0] = b.x; cv[1] = b.y;
    }
    return ld(reinterpret_cast<const uint2*>(row + q_par_offset(G, BITS)) + d0 / kQGroup);
}

template <int BITS, int G, bool F32>
__global__ void __launch_bounds__(kQThreads) qmem_read_kernel(const __grid_constant__ QmemParams p)
{
    pdl_launch_dependents();
    pdl_wait();
    QPos o;
    if (!q_pos<BITS, G>(p, o)) return;
    constexpr int E = F32 ? 4 : 2;
    uint32_t ck[2], cv[2];
    const uint2 par = row_unit<BITS, G>(o.row, o.d0, ck, cv);
    float xk[8], xv[8];
    expand8<BITS>(ck, __uint_as_float(par.x << 16), __uint_as_float(par.x & 0xffff0000u), xk);
    expand8<BITS>(cv, __uint_as_float(par.y << 16), __uint_as_float(par.y & 0xffff0000u), xv);
    const int64_t t = o.t;
    char* rk = static_cast<char*>(p.xk) + (blockIdx.z * p.xk_sb + t * p.xk_st + blockIdx.y * p.xk_sh) * E;
    char* rv = static_cast<char*>(p.xv) + (blockIdx.z * p.xv_sb + t * p.xv_st + blockIdx.y * p.xv_sh) * E;
    store8<F32>(rk, o.d0, p.D, p.vec_k, xk);
    store8<F32>(rv, o.d0, p.D, p.vec_v, xv);
}

// Rows that do not start on 16-byte boundaries: a warp per row, a lane per channel of a group, so that the stores of a
// warp are contiguous (by eights, each lane's stores lay 16 bytes apart: 16.5 instead of 12 us on the
// base shape); the loads of kReadRows rows, all groups, come before their stores.
template <int G> constexpr int kReadRows = G <= 2 ? 4 : 2;

template <int BITS, int G, bool F32>
__global__ void __launch_bounds__(kQThreads) qmem_read_rows_kernel(const __grid_constant__ QmemParams p)
{
    constexpr int ROWS = kReadRows<G>;
    pdl_launch_dependents();
    pdl_wait();
    const int lane = threadIdx.x & 31, h = blockIdx.y, b = blockIdx.z;
    const int64_t t0 = (static_cast<int64_t>(blockIdx.x) * (kQThreads / 32) + (threadIdx.x >> 5)) * ROWS;
    const uint8_t* head = p.rows + (static_cast<int64_t>(b) * p.H + h) * p.M * q_row_bytes(G, BITS);
    const int byte = lane * BITS / 8, sh = BITS == 4 ? 4 * (lane & 1) : 0, mask = (1 << BITS) - 1;
    uint2 par[ROWS][G];
    int ck[ROWS][G], cv[ROWS][G];
#pragma unroll
    for (int u = 0; u < ROWS; ++u) {
        int64_t slot = p.slot0 + min(t0 + u, static_cast<int64_t>(p.n - 1));
        if (slot >= p.M) slot -= p.M;
        if (!in_range(slot, 0, p.M, p.chk)) slot = 0;
        const uint8_t* row = head + slot * q_row_bytes(G, BITS);
#pragma unroll
        for (int g = 0; g < G; ++g) {
            par[u][g] = ld(reinterpret_cast<const uint2*>(row + q_par_offset(G, BITS)) + g);
            ck[u][g] = ld(row + 4 * BITS * g + byte);
            cv[u][g] = ld(row + q_v_offset(G, BITS) + 4 * BITS * g + byte);
        }
    }
#pragma unroll
    for (int u = 0; u < ROWS; ++u) {
        const int64_t t = t0 + u;
        if (t >= p.n) break;
        const int64_t ok = b * p.xk_sb + t * p.xk_st + h * p.xk_sh, ov = b * p.xv_sb + t * p.xv_st + h * p.xv_sh;
#pragma unroll
        for (int g = 0; g < G; ++g) {
            const int d = 32 * g + lane;
            if (d >= p.D) break;
            const float k = fmaf(__uint_as_float(par[u][g].x << 16), static_cast<float>((ck[u][g] >> sh) & mask),
                                 __uint_as_float(par[u][g].x & 0xffff0000u));
            const float v = fmaf(__uint_as_float(par[u][g].y << 16), static_cast<float>((cv[u][g] >> sh) & mask),
                                 __uint_as_float(par[u][g].y & 0xffff0000u));
            if constexpr (F32) {
                static_cast<float*>(p.xk)[ok + d] = k;
                static_cast<float*>(p.xv)[ov + d] = v;
            } else {
                static_cast<__nv_bfloat16*>(p.xk)[ok + d] = __float2bfloat16_rn(k);
                static_cast<__nv_bfloat16*>(p.xv)[ov + d] = __float2bfloat16_rn(v);
            }
        }
    }
}

// The operands of the fused attention kernels: K and V of the memory and of the segment, and r, in fp16, which
// keeps 11 bits where bf16 keeps 8, for every (b, h) whose values fp16 has the range for, else in bf16.  In fp16
// each takes its range from a power of two, the unit: the largest |k| of a (b, h) comes into [1, 2) (its unit
// multiplies c(q+u)), the largest |v| into [2^14, 2^15) (P of the attention goes up to 2^8, the sums are fp32), and
// the largest |r| of the head into [1, 2).  What that can lose:
//   * An element of k below 2^-14 of its unit is off by up to 2^-25 of the unit, a score by D max|c(q+u)| max|k|
//     2^-25: 2^-10 where that product is at most 2^15.  No c(q+u) leaves fp16's range then, nor does a
//     score.  The same for r and c(q+v), whose sums, the position terms, are held in fp16.
//   * P is off by up to 2^-25 (of its largest, 1 to 2^8) where it is below 2^-14: of a key whose value is R times
//     another's, by 2^-25 R of that one's.  R is at most 2^12, over all groups of 32 channels that are not zero.
//     (v's own elements are off by 2^-39 of the largest.)
// Ordinary values are far inside (D max|c(q+u)| max|k| around 2^9, R of 2^4); a head with an infinity, a NaN, an element
// far above the rest or nearly empty positions is not, and is computed as txl_rel_attn_fwd would, in bf16.
//
// Two passes: qmem_ranges_kernel takes the ranges of up to kXSplits shares of the rows of a (b, h) (a group's end
// points bound its values, so the parameters suffice for the memory), qmem_expand_kernel writes, one lane per eight
// channels of a row.  (One kernel with a cluster per (b, h), exchanging the maxima through shared memory, took
// 62 us on the large shape: its CTAs waited for one another.)
constexpr int kXSplits = 8;

// A share's ranges, four words: largest |k| and |v| as bf16 halves, rounded up; bounds of |c(q+u)| and |c(q+v)|
// likewise; largest |r| (shares of their own); the smallest over groups that are not zero of a group's largest |v|.
// What is not finite counts as infinite.
struct XRange {
    float k = 0.f, v = 0.f, qu = 0.f, qv = 0.f, v_least = INFINITY;
    __device__ __forceinline__ void join(const uint4& w)
    {
        k = fmaxf(k, __uint_as_float(w.x << 16));
        v = fmaxf(v, __uint_as_float(w.x & 0xffff0000u));
        qu = fmaxf(qu, __uint_as_float(w.y << 16));
        qv = fmaxf(qv, __uint_as_float(w.y & 0xffff0000u));
        v_least = fminf(v_least, __uint_as_float(w.w));
    }
    // whether this (b, h) has the range for fp16 (false for any infinity)
    __device__ __forceinline__ bool fits(int D, float r) const
    {
        return D * qu * k <= 32768.f && D * qv * r <= 32768.f && v < INFINITY && v <= 4096.f * v_least;
    }
};

// First of the n items that fall to share `part` of `parts`.
__device__ __forceinline__ int x_share(int n, int part, int parts)
{
    const unsigned each = static_cast<unsigned>(n) / parts, more = static_cast<unsigned>(n) - each * parts;
    return static_cast<int>(each * part + min(static_cast<unsigned>(part), more));
}

template <int BITS, int G>
__global__ void __launch_bounds__(kQThreads, G == 3 ? 6 : 8) qmem_ranges_kernel(const __grid_constant__ QexpandParams p, int parts)
{
    __shared__ float red[6][kQThreads / 32];
    pdl_launch_dependents();
    pdl_wait();
    const int tid = threadIdx.x, lane = tid & 31, part = blockIdx.x, h = blockIdx.y, b = blockIdx.z;
    const int64_t bh = static_cast<int64_t>(b) * p.H + h;
    if (tid == 0 && part == 0 && bh == 0) p.units[3] = 0.f;      // (set by the expansion where a head is bf16)
    constexpr int LPR = 4 * G;                            // lanes of a row, eight channels each
    constexpr int RPP = kQThreads / LPR;                  // rows of a pass
    const int lr = tid / LPR, d0 = 8 * (tid % LPR);
    const bool lane_on = lr < RPP;                        // the four lanes of a group are on or off together

    float k = 0.f, v = 0.f, q = 0.f, u = 0.f, vb = 0.f, v_least = INFINITY;      // (k: r in blocks of r); NaN stays
    auto group_v = [&](float a) {                         // the largest |v| of a group
        v = max_nan(v, a);
        if (a > 0.f) v_least = fminf(v_least, a);
    };
    if (part < parts) {
        const int64_t x1 = static_cast<int64_t>(x_share(p.n, part + 1, parts)) * G;
#pragma unroll 4
        for (int64_t x = static_cast<int64_t>(x_share(p.n, part, parts)) * G + tid; x < x1; x += kQThreads) {
            const int t = static_cast<int>(x / G), g = static_cast<int>(x - static_cast<int64_t>(t) * G);
            int64_t s = static_cast<int64_t>(p.slot0) + t;
            if (s >= p.M) s -= p.M;
            if (!in_range(s, 0, p.M, p.chk)) s = 0;
            const uint2 w = ld(reinterpret_cast<const uint2*>(p.rows + (bh * p.M + s) * q_row_bytes(G, BITS) +
                                                                  q_par_offset(G, BITS)) + g);
            auto most = [&](uint32_t kv) {
                const float step = __uint_as_float(kv << 16), lo = __uint_as_float(kv & 0xffff0000u);
                return max_nan(fabsf(lo), fabsf(fmaf(step, static_cast<float>((1 << BITS) - 1), lo)));
            };
            k = max_nan(k, most(w.x));
            group_v(most(w.y));
        }
        if (lane_on) {
            const int s0 = x_share(p.L, part, parts) + lr, s1 = x_share(p.L, part + 1, parts);
            auto row = [&](const void* x, int64_t sb, int64_t st, int64_t sh, int64_t t) {
                return static_cast<const uint16_t*>(x) + b * sb + t * st + h * sh;
            };
#pragma unroll 4
            for (int t = s0; t < s1; t += RPP) {
                float x[8];
                load8<false>(row(p.kcur, p.kc_sb, p.kc_st, p.kc_sh, t), d0, p.D, p.vec_k, x);
#pragma unroll
                for (int e = 0; e < 8; ++e) k = max_nan(k, fabsf(x[e]));
            }
#pragma unroll 4
            for (int t = s0; t < s1; t += RPP) {
                float x[8], a = 0.f;
                load8<false>(row(p.vcur, p.vc_sb, p.vc_st, p.vc_sh, t), d0, p.D, p.vec_v, x);
#pragma unroll
                for (int e = 0; e < 8; ++e) a = max_nan(a, fabsf(x[e]));
#pragma unroll
                for (int off = 1; off <= 2; off <<= 1) a = max_nan(a, __shfl_xor_sync(0xfu << (lane & 28), a, off));
                group_v(a);
            }
#pragma unroll 4
            for (int t = s0; t < s1; t += RPP) {
                float x[8];
                load8<false>(row(p.q, p.q_sb, p.q_st, p.q_sh, t), d0, p.D, p.vec_q, x);
#pragma unroll
                for (int e = 0; e < 8; ++e) q = max_nan(q, fabsf(x[e]));
            }
        }
        if (tid < p.D) {
            u = fabsf(__ldg(p.u + h * p.D + tid));
            vb = fabsf(__ldg(p.vb + h * p.D + tid));
        }
    } else if (lane_on) {
        // this entry's share of the head's rows of r
        const int rp = part - parts, r_parts = gridDim.x - parts;
        const int r0 = x_share(p.n_r, b, p.B), n_r = x_share(p.n_r, b + 1, p.B) - r0, s1 = x_share(n_r, rp + 1, r_parts);
#pragma unroll 4
        for (int i = x_share(n_r, rp, r_parts) + lr; i < s1; i += RPP) {
            float x[8];
            load8<false>(p.r + (static_cast<int64_t>(r0 + i) * p.H + h) * p.ld_r, d0, p.D, p.vec_r, x);
#pragma unroll
            for (int e = 0; e < 8; ++e) k = max_nan(k, fabsf(x[e]));
        }
    }
    // over the block (v_least as the maximum of its negative)
    float m[6] = {k, v, q, u, vb, -v_least};
#pragma unroll
    for (int i = 0; i < 6; ++i) {
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) m[i] = max_nan(m[i], __shfl_xor_sync(0xffffffffu, m[i], off));
        if (lane == 0) red[i][tid >> 5] = m[i];
    }
    __syncthreads();
    if (tid >= 32) return;
#pragma unroll
    for (int i = 0; i < 6; ++i) {
        m[i] = red[i][lane & 7];
#pragma unroll
        for (int off = 4; off > 0; off >>= 1) m[i] = max_nan(m[i], __shfl_xor_sync(0xffffffffu, m[i], off));
    }
    if (lane != 0) return;
    uint32_t* out = p.ranges + (bh * kXSplits + (part < parts ? part : part - parts)) * 4;
    auto or_inf = [](float a) { return a < INFINITY ? a : INFINITY; };
    auto pair = [&](float a, float c) {
        return (__float_as_uint(bf16_ceil_pos(or_inf(a))) >> 16) | __float_as_uint(bf16_ceil_pos(or_inf(c)));
    };
    if (part < parts) {
        out[0] = pair(m[0], m[1]);
        out[1] = pair((m[2] + m[3]) * p.qscale, (m[2] + m[4]) * p.qscale);
        out[3] = __float_as_uint(-m[5]);
    } else {
        out[2] = __float_as_uint(or_inf(m[0]));
    }
}

// Grid: x over the lanes of the rows (memory, segment, this entry's share of the head's rows of r), y head, z entry.
template <int BITS, int G>
__global__ void __launch_bounds__(kQThreads, 8) qmem_expand_kernel(const __grid_constant__ QexpandParams p, int parts, int r_parts)
{
    pdl_launch_dependents();
    pdl_wait();
    const int h = blockIdx.y, b = blockIdx.z;
    const int64_t bh = static_cast<int64_t>(b) * p.H + h;
    const int lr = threadIdx.x / kRowLanes<G>, d0 = 8 * (threadIdx.x % kRowLanes<G>);
    int t = static_cast<int>(blockIdx.x) * kBlockRows<G> + lr;
    if (lr >= kBlockRows<G>) t = INT32_MAX;
    uint32_t ck[2], cv[2];
    uint2 par;
    if (t < p.n && d0 < p.D) {                             // requested before the ranges
        unsigned s = static_cast<unsigned>(p.slot0) + t;
        if (s >= static_cast<unsigned>(p.M)) s -= p.M;
        if (!in_range(s, 0, p.M, p.chk)) s = 0;
        const uint8_t* head = p.rows + bh * p.M * q_row_bytes(G, BITS);
        par = row_unit<BITS, G>(head + static_cast<uint64_t>(s) * static_cast<unsigned>(q_row_bytes(G, BITS)), d0, ck, cv);
    }
    // the ranges, by the first warp: this (b, h)'s shares, and the head's rows of r over the shares of every entry
    __shared__ float red[kQThreads / 32], scale_by[4];     // of k, v, r, and of the rows of r16
    __shared__ int in_f16;
    const uint4* ranges = reinterpret_cast<const uint4*>(p.ranges);
    const int lane = threadIdx.x & 31;
    XRange x;
    if (threadIdx.x < parts) x.join(__ldcg(ranges + bh * kXSplits + threadIdx.x));
    float r = 0.f;
#pragma unroll 1
    for (int e = threadIdx.x; e < p.B * r_parts; e += kQThreads)
        r = fmaxf(r, __uint_as_float(__ldcg(p.ranges + ((static_cast<int64_t>(e / r_parts) * p.H + h) * kXSplits + e % r_parts) * 4 + 2)));
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) r = fmaxf(r, __shfl_xor_sync(0xffffffffu, r, off));
    if (lane == 0) red[threadIdx.x >> 5] = r;
    __syncthreads();
    if (threadIdx.x < 32) {
        r = red[lane & 7];
#pragma unroll
        for (int off = 4; off > 0; off >>= 1) {
            r = fmaxf(r, __shfl_xor_sync(0xffffffffu, r, off));
            x.k = fmaxf(x.k, __shfl_xor_sync(0xffffffffu, x.k, off));
            x.v = fmaxf(x.v, __shfl_xor_sync(0xffffffffu, x.v, off));
            x.qu = fmaxf(x.qu, __shfl_xor_sync(0xffffffffu, x.qu, off));
            x.qv = fmaxf(x.qv, __shfl_xor_sync(0xffffffffu, x.qv, off));
            x.v_least = fminf(x.v_least, __shfl_xor_sync(0xffffffffu, x.v_least, off));
        }
        bool f16 = __shfl_sync(0xffffffffu, x.fits(p.D, r) ? 1 : 0, 0);
        if (p.r_alone) {                                   // one copy of r: one type for every entry's share of the head
            bool all = true;
#pragma unroll 1
            for (int e = lane; e < p.B; e += 32) {
                XRange o;
#pragma unroll 1
                for (int y = 0; y < parts; ++y) o.join(__ldcg(ranges + (static_cast<int64_t>(e) * p.H + h) * kXSplits + y));
                all = all && o.fits(p.D, r);
            }
            f16 = __all_sync(0xffffffffu, all);
        }
        if (lane < 3) {
            // bf16 operands stay as they are, but values whose sums could overflow fp32
            const float top = lane == 0 ? x.k : lane == 1 ? x.v : r;
            const int e = static_cast<int>(__float_as_uint(top) >> 23) - 127;      // 128: not finite
            const int fit = min(max(e - (lane == 1 ? 14 : 0), -115), 115);
            const int ex = f16 ? fit : lane == 1 && e > 64 ? 32 : 0;
            scale_by[lane] = __uint_as_float(static_cast<uint32_t>(127 - ex) << 23);
            // (entries in bf16 read r itself where they can)
            if (lane == 2) scale_by[3] = p.r_alone && !f16 ? 1.f : __uint_as_float(static_cast<uint32_t>(127 - fit) << 23);
            if (blockIdx.x == 0) {
                const float unit = __uint_as_float(static_cast<uint32_t>(127 + ex) << 23);
                p.units[4 * bh + lane] = (lane == 0 && !f16) || (lane == 1 && !(x.v < INFINITY)) ? -unit : unit;
            }
        } else if (lane == 3) {
            in_f16 = f16;
            if (blockIdx.x == 0 && !f16) p.units[3] = 1.f;
        }
    }
    __syncthreads();
    const bool f16 = in_f16 != 0;
    if (d0 >= p.D) return;
    const unsigned ld_bytes = 2 * p.ld;
    auto put = [&](void* base, int64_t first_row, int at, const float* a, float f, bool half) {
        char* dst = static_cast<char*>(base) + first_row * ld_bytes + static_cast<uint64_t>(at) * ld_bytes + 2 * d0;
        uint32_t w[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float a0 = a[2 * e] * f, a1 = a[2 * e + 1] * f;
            w[e] = half ? pack_f16x2(a0, a1) : pack_bf16x2(a0, a1);
        }
        *reinterpret_cast<uint4*>(dst) = make_uint4(w[0], w[1], w[2], w[3]);
    };
    float a[8];
    if (t < p.n) {
        // lo + step c in units (a power of two, so scaling the parameters rounds nothing)
        const float ki = scale_by[0], vi = scale_by[1];
        expand8<BITS>(ck, __uint_as_float(par.x << 16) * ki, __uint_as_float(par.x & 0xffff0000u) * ki, a);
        put(p.k_mem, bh * p.n, t, a, 1.f, f16);
        expand8<BITS>(cv, __uint_as_float(par.y << 16) * vi, __uint_as_float(par.y & 0xffff0000u) * vi, a);
        put(p.v_mem, bh * p.n, t, a, 1.f, f16);
        return;
    }
    if (t == INT32_MAX) return;
    t -= p.n;
    auto seg = [&](const void* v, int64_t sb, int64_t st, int64_t sh) {
        return static_cast<const uint16_t*>(v) + b * sb + t * st + h * sh;
    };
    if (t < p.L) {
        load8<false>(seg(p.kcur, p.kc_sb, p.kc_st, p.kc_sh), d0, p.D, p.vec_k, a);
        float c[8];
        load8<false>(seg(p.vcur, p.vc_sb, p.vc_st, p.vc_sh), d0, p.D, p.vec_v, c);
#pragma unroll
        for (int e = 0; e < 8; ++e)                        // (a weight of 0 would not hide them: see AttnTcParams)
            if (!(fabsf(c[e]) < INFINITY)) c[e] = 0.f;
        put(p.k_seg, bh * p.L, t, a, scale_by[0], f16);
        put(p.v_seg, bh * p.L, t, c, scale_by[1], f16);
        if (p.q_seg) {
            load8<false>(seg(p.q, p.q_sb, p.q_st, p.q_sh), d0, p.D, p.vec_q, a);
            store8<false>(static_cast<uint16_t*>(p.q_seg) + (bh * p.L + t) * p.ld, d0, p.ld, true, a);
        }
        return;
    }
    t += x_share(p.n_r, b, p.B) - p.L;
    if (t < x_share(p.n_r, b + 1, p.B)) {
        const int64_t row = static_cast<int64_t>(t) * p.H + h;
        load8<false>(p.r + row * p.ld_r, d0, p.D, p.vec_r, a);
        put(p.r16, row, 0, a, scale_by[3], !p.r_alone || f16);
    }
}

template <int BITS, int G>
cudaError_t launch_expand(const QexpandParams& p, cudaStream_t s)
{
    // shares of about 128 rows
    auto shares = [](int64_t rows) { return static_cast<int>(std::min<int64_t>(kXSplits, std::max<int64_t>(1, (rows + 127) / 128))); };
    const int parts = shares(std::max<int64_t>(p.n / G, p.L)), r_parts = shares(p.n_r / p.B);
    cudaError_t e = launch_dependent(qmem_ranges_kernel<BITS, G>, dim3(parts + r_parts, p.H, p.B), dim3(kQThreads), 0, s, p, parts);
    if (e != cudaSuccess) return e;
    const int64_t rows = static_cast<int64_t>(p.n) + p.L + (p.n_r + p.B - 1) / p.B;
    if (rows > INT32_MAX - kQThreads) return cudaErrorInvalidValue;
    return launch_dependent(qmem_expand_kernel<BITS, G>, dim3((rows - 1) / kBlockRows<G> + 1, p.H, p.B), dim3(kQThreads), 0,
                            s, p, parts, r_parts);
}

template <int BITS, int G>
cudaError_t launch(const QmemParams& p, bool f32, bool push, cudaStream_t s)
{
    if (!push && !(p.vec_k && p.vec_v)) {
        constexpr int rows = kQThreads / 32 * kReadRows<G>;
        return launch_dependent(f32 ? qmem_read_rows_kernel<BITS, G, true> : qmem_read_rows_kernel<BITS, G, false>,
                                dim3((p.n - 1) / rows + 1, p.H, p.B), dim3(kQThreads), 0, s, p);
    }
    const dim3 grid((p.n - 1) / kBlockRows<G> + 1, p.H, p.B);
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

cudaError_t launch_qmem_expand(const QexpandParams& p, cudaStream_t s)
{
    switch (p.G * 16 + (p.n > 0 ? p.bits : 4)) {
    case 1 * 16 + 4: return launch_expand<4, 1>(p, s);
    case 2 * 16 + 4: return launch_expand<4, 2>(p, s);
    case 3 * 16 + 4: return launch_expand<4, 3>(p, s);
    case 4 * 16 + 4: return launch_expand<4, 4>(p, s);
    case 1 * 16 + 8: return launch_expand<8, 1>(p, s);
    case 2 * 16 + 8: return launch_expand<8, 2>(p, s);
    case 3 * 16 + 8: return launch_expand<8, 3>(p, s);
    case 4 * 16 + 8: return launch_expand<8, 4>(p, s);
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
