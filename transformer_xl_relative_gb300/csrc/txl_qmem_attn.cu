// txl_qmem_attn.cu -- relative attention of 1 .. 16 queries over a quantised memory and the segment's
// own keys: the generation step over a memory of 4- or 8-bit codes, in two launches or one.
//
//     s_ij = scale [ (q_i+u).k'_j + (q_i+v).r[min(M+i-j, C)] ],  out_i = softmax_j(s_ij) v'_j
// with k'_jd = lo_jG + step_jG c_jd in group G of 32 channels.  The codes never become k' or v':
//     q.k'_j  = sum_G step_jG (sum_{d in G} q_d c_jd) + lo_jG (sum_{d in G} q_d)
//     out_d   = sum_j (p_j step_jG) c_jd + sum_j p_j lo_jG
// so the inner sums are products with the integer codes, and step and lo act once per key and group.
//
// The work is bound by HBM (a byte of 4-bit codes carries four flops per query); what it must avoid is
// spending instructions per code.  The inner sums run as mma.sync m16n8k16 with the codes as the A
// operand: the bit pattern of a code in the low bits of an fp16 number is the subnormal c 2^-24, which the
// tensor cores multiply exactly, so one AND per pair of codes makes an operand (a nibble at bits 4..7
// is 16 c 2^-24; the 16 goes into q, or into the output).  ldmatrix delivers four codes of a row per
// 16 bits; its transposed form pairs two keys of the same channel for P.V.  At 4 bits a pair of codes
// costs 0.6 instructions for K and for V, where converting to floats took about three.  (tcgen05 would
// want the codes expanded into shared memory first, and 128 rows of queries where there are 1 to 16.)
//
// Precision: q+u is held as two fp16 parts (22 bits) in two columns of the B operand, p step likewise; the
// accumulators are fp32.  Both are scaled by powers of two per row and group of 32 channels, so that a group keeps
// its bits whatever the others hold (one unit for all: a group of values 2^10 times smaller than another was off
// by 5e-5): the largest of q+u into [2^14, 2^15), which leaves 22 bits down to 2^-13 of it (odd channels at 4
// bits; 2^-17 else), the largest p step into [2^8, 2^9) when its unit is set, 22 bits down to 2^-11.  The eight columns of an MMA are four
// slots x (hi, lo).  A slot is a query; with fewer than three queries the other slots take other tiles
// of 16 keys ("streams"), so that the work per key after the first product (scale, softmax, splitting
// p) falls on all 32 lanes whatever L is.  With one query the four k-quarters of a Q.K MMA belong to the
// four streams (each lane holds whole rows of its own two keys, B is block diagonal); with two queries
// B is masked to the tile's own slots.
//
// The position term (q_i+v).r comes from a kernel of its own (qpos_kernel): a product of r's rows with the
// queries of every batch entry, so that each row of r is read once per 64 (entry, query) pairs, written
// by key, E[b][h][i][j - jn], and copied into the stages with the codes.  Keys j < jn are at the clamp
// for every query and take one value per query, far[b][h][i].  (Computed inside the attention kernel
// instead, for the keys of a block between the steps of the one before, the 32 registers of r rows in
// flight and a block barrier per stage cost more than the launch: 66 instead of then 49 us at B8
// H16 D64 M16384.  A CTA that has few such keys computes them itself, before the key loop.)  The attention
// kernel's prologue and first copies run while qpos_kernel does.
//
// One CTA: one batch entry, one head, up to eight queries and a range of keys; eight warps, each with
// its own ring of bulk-copy stages and no block barrier in the key loop (cp.async, 16 bytes per lane, held
// the issuing warp for 2400 to 4000 cycles per stage until its requests were accepted).  The key ranges
// of a head are the ranks of a cluster: each writes its partial results into the shared memory of the
// rank that finishes the row.
//
// Measured (both kernels, B8 H16 D64, one query): 4096 keys of 4 bits 15.8 us (44 MB; 6.5 us of HBM), of 8 bits
// 20.0 us (78 MB), 16384 keys of 4 bits 35.6 us (170 MB, 4.8 TB/s; 6.4 TB/s of what each further key adds).
// The bf16 memory's decode takes 40 us at 4096 keys.  Two CTAs of eight warps fill the registers of an SM; of
// a token's 12 us in the kernel 3 are the prologue (the copies of half the memory are in flight), 2.5 the
// merge.  The loop is latency: every shared-memory access is free of bank conflicts (with the parts of q in the
// same banks it took 1000 instead of 640 cycles per stage for Q.K, and the call 17.0 us).
#include <algorithm>
#include <atomic>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "txl_internal.h"
#include "txl_mma.cuh"
#include "txl_ptx.cuh"
#include "txl_rows.cuh"

namespace txl {

namespace {

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kStages = 2;
constexpr int kMaxRanks = 16;                  // CTAs of a cluster (beyond 8: not portable, but this GPU's)
constexpr int kMaxRows = 8;                    // queries of a CTA
static_assert(kWarps + kDecodeMaxL <= 32 && kMaxRows <= kWarps, "a lane per part of a row, a warp per row");
constexpr float kNoMax = -3e38f;               // running maximum before any key
constexpr float kTwo24 = 16777216.f;
constexpr float kMinUnit = 3.00926553e-36f;    // 2^-118 and 2^126: bounds of the weights' units, so that a weight
constexpr float kMaxUnit = 8.50705917e37f;     // (at most 2^8) over the unit stays finite
constexpr uint32_t kMinUnits = 0x04800480u;    // 2^-118 twice, as below

// Powers of two of two groups in a register, as bf16 halves: the units, and one over them (2^-126 .. 2^126).
__device__ __forceinline__ float unit_of(uint32_t w, int G) { return __uint_as_float(G & 1 ? w & 0xffff0000u : w << 16); }
__device__ __forceinline__ uint32_t one_over(uint32_t w) { return 0x7f007f00u - w; }

// Keys of a stage: 64 where a key's codes are small and the queries few, else 32.
__host__ __device__ constexpr int stage_keys(int bits, int ng, int qt) { return bits * ng <= 8 && qt == 1 ? 64 : 32; }
// Queries whose position terms a stage has room for.
__host__ __device__ constexpr int stage_rows(int qt, bool one) { return one ? 1 : 4 * qt; }
// Floats from one query's position terms to the next: four queries' eight keys lie in different banks.
__host__ __device__ constexpr int e_stride(int bits, int ng, int qt, bool one) { return stage_keys(bits, ng, qt) + (one ? 0 : 8); }
__host__ __device__ constexpr int stage_bytes(int bits, int ng, int qt, bool one)
{
    return stage_keys(bits, ng, qt) * q_row_bytes(ng, bits) + 4 * stage_rows(qt, one) * e_stride(bits, ng, qt, one);
}

struct QSplit {               // how the host divides the work
    int lq;                   // queries of a CTA; blockIdx.x / ranks selects the group of queries
    int ranks;                // CTAs of a cluster: key ranges
    int range;                // keys of a range (a multiple of the stage)
};

__device__ __forceinline__ float ld_bf16(const void* p, int64_t i)
{
    return __uint_as_float(static_cast<uint32_t>(ld(static_cast<const uint16_t*>(p) + i)) << 16);
}

// The rows of r are requested a tile ahead of their use.  The compiler puts plain loads off until then (0.7 us per
// call); a volatile one stays where it is, after the wait for the kernel that may write r.
__device__ __forceinline__ uint4 ld_early(const uint4* p)
{
    uint4 v;
    asm volatile("ld.global.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
    return v;
}

__device__ __forceinline__ void prefetch_l2(const void* p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }

// D += A B: m16n8k16, fp16 operands, fp32 accumulators
__device__ __forceinline__ void mma_f16(float* c, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1)
{
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
                 "{%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// D = A B
__device__ __forceinline__ void mma_f16_first(float* c, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                              uint32_t b1)
{
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
                 "{%8, %9}, {%10, %10, %10, %10};"
                 : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}

// 8 x 8 transpose of 16-bit elements across a warp
__device__ __forceinline__ uint32_t transpose8(uint32_t x)
{
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}


// (hi, lo) fp16 parts of x0 and x1, a word each: hi = x rounded, lo = the rest rounded
__device__ __forceinline__ void split_f16(float x0, float x1, uint32_t& w0, uint32_t& w1)
{
    const uint32_t hi = pack_f16x2(x0, x1);
    const float2 h = __half22float2(*reinterpret_cast<const __half2*>(&hi));
    const uint32_t lo = pack_f16x2(x0 - h.x, x1 - h.y);
    w0 = __byte_perm(hi, lo, 0x5410);
    w1 = __byte_perm(hi, lo, 0x7632);
}


__device__ __forceinline__ void lds128(uint32_t addr, uint32_t* w)
{
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "r"(addr));
}

// Pairs of codes of a register as fp16 numbers; odd = the second pair of a 16-bit half (16 times as large at 4 bits).
// As subnormals, c 2^-24, for bf16 calls: one AND.  The tensor cores align products by the exponents of their operands,
// in which a subnormal's leading zeros count, and drop what lies some 24 bits below, so that sums keep 15 good bits (of
// 4-bit codes; 19 of 8-bit ones).  WIDE, for fp32 calls: c - c0 (8, 128) exactly, by way of 1024 + c, and lo + c0 step in
// place of lo; besides the bits this keeps the sums of codes and of lo from cancelling (those alone left errors of 1e-6 to 1e-5; now 1e-7 to 4e-7).
template <int BITS> constexpr float kCentre = BITS == 4 ? 8.f : 128.f;

__device__ __forceinline__ uint32_t add_f16x2(uint32_t a, uint32_t b)
{
    uint32_t r;
    asm("add.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
template <int BITS, bool WIDE>
__device__ __forceinline__ uint32_t pair_even(uint32_t w)
{
    const uint32_t c = w & (BITS == 4 ? 0x000f000fu : 0x00ff00ffu);
    return WIDE ? add_f16x2(c | 0x64006400u, BITS == 4 ? 0xe408e408u : 0xe480e480u) : c;      // less 1032, 1152
}
template <int BITS, bool WIDE>
__device__ __forceinline__ uint32_t pair_odd(uint32_t w)
{
    const uint32_t c = BITS == 4 ? w & 0x00f000f0u : __byte_perm(w, 0, 0x4341);
    return WIDE ? add_f16x2(c | 0x64006400u, 0xe480e480u) : c;                                // less 1152
}

// A position term from the products with the high and the low part of q+v.  An infinity of r meets a low part of 0 or
// of the other sign: the high part has the answer.
__device__ __forceinline__ float both_parts(float hi, float lo) { return fabsf(hi) < INFINITY ? hi + lo : hi; }

// Rows of r of 16 distances from d0 as the A operand's fragments: this lane's of distances g and g + 8.
template <int NG>
__device__ __forceinline__ void load_r(const QattnParams& p, int h, unsigned d0, uint4 (&a)[2][NG])
{
    const int g = (threadIdx.x & 31) >> 2, c4 = threadIdx.x & 3;
#pragma unroll
    for (int y = 0; y < 2; ++y) {
        int rr = static_cast<int>(min(d0 + g + 8 * y, static_cast<unsigned>(p.C)));
        if (rr >= p.n_rows || !in_range(rr, 0, p.n_rows, p.chk)) rr = 0;  // past the distances of the call
        const uint16_t* src = static_cast<const uint16_t*>(p.r) + rr * p.r_row + h * p.r_head;
#pragma unroll
        for (int G = 0; G < NG; ++G) {
            const int d = 32 * G + 8 * c4;
            if (p.vec_r && d + 8 <= p.D) {
                a[y][G] = ld_early(reinterpret_cast<const uint4*>(src + d));
            } else {
                uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    if (d + e < p.D) w[e >> 1] |= static_cast<uint32_t>(ld(src + d + e)) << (16 * (e & 1));
                a[y][G] = make_uint4(w[0], w[1], w[2], w[3]);
            }
        }
    }
}

// E[b][h][i][x] = (q_i+v).r[min(M+i-j, C)] in log2 units for keys j = jn + x, and far[b][h][i] = (q_i+v).r[C].
// Bound by reading r once: a CTA prepares q+v of up to pos_pairs (entry, query) pairs of a head as two bf16 parts
// (the B operands) and walks over tiles of 128 distances, 16 per warp, whose rows of r (the A operands, read
// from global memory as fragments) are requested one tile ahead.  65537 distances of 16 heads: 26 us, 5.1 TB/s.
// WALK: more tiles than three CTAs per SM; four CTAs per SM (64 registers) then keep more rows in flight (those
// 65537 distances: the whole call 45.2 us, 62.4 with three); with fewer the free choice of registers (75) is
// quicker (token over 4096 keys 15.8 us, 16.6 with 64).
__host__ __device__ constexpr int pos_pairs(int ng) { return ng == 2 ? 64 : 32; }

template <int NG, bool WALK>
__global__ void __launch_bounds__(kThreads, NG > 2 ? 2 : WALK ? 4 : 0) qpos_kernel(const __grid_constant__ QattnParams p)
{
    constexpr int DP = NG * 32, PAIRS = pos_pairs(NG);
    // [2 pair + part][DP], the groups of part 1 swapped in pairs: a load takes both parts, from different banks
    __shared__ __align__(16) uint16_t qvh[2 * PAIRS * DP];
    __shared__ float* e_key[PAIRS];                                   // E of the pair at x = M + i - jn (distance 0)
    __shared__ float* far_at[PAIRS];
    __shared__ int x_zero[PAIRS];                                     // that x
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, c4 = lane & 3;
    const int h = blockIdx.y, pair0 = blockIdx.z * PAIRS, pairs = min(PAIRS, p.B * p.L - pair0);
    // Everything before this kernel is complete when it lets the attention kernel start, which reads the
    // memory and the queries before its own wait.
    pdl_wait();
    pdl_launch_dependents();
    uint4 a[2][NG];
    unsigned d0 = blockIdx.x * 128 + warp * 16;                       // first distance of the warp's tile
    load_r<NG>(p, h, d0, a);
    const int n_ct = (pairs + 3) >> 2;
    float vb[NG];
#pragma unroll
    for (int e = 0; e < NG; ++e) vb[e] = 32 * e + lane < p.D ? __ldg(p.vb + h * p.D + 32 * e + lane) : 0.f;
#pragma unroll 4
    for (int pr = warp; pr < 4 * n_ct; pr += kWarps) {                // a warp per pair
        const int be = (pair0 + pr) / p.L, i = (pair0 + pr) - be * p.L;
        const int64_t at = be * p.q_sb + i * p.q_st + h * p.q_sh;
#pragma unroll
        for (int e = 0; e < NG; ++e) {
            const int d = 32 * e + lane;
            const float c = pr < pairs && d < p.D ? (ld_bf16(p.q, at + d) + vb[e]) * p.qscale : 0.f;
            const __nv_bfloat16 hi = __float2bfloat16_rn(c);
            qvh[2 * pr * DP + d] = __bfloat16_as_ushort(hi);
            qvh[(2 * pr + 1) * DP + (d ^ 32)] = __bfloat16_as_ushort(__float2bfloat16_rn(c - __bfloat162float(hi)));
        }
    }
    if (tid < pairs) {
        const int be = (pair0 + tid) / p.L, i = (pair0 + tid) % p.L;
        const int64_t row = (static_cast<int64_t>(be) * p.H + h) * p.L + i;
        x_zero[tid] = p.M + i - p.jn;
        e_key[tid] = p.E + row * p.e_pitch + x_zero[tid];
        far_at[tid] = p.far + row;
    }
    __syncthreads();
    for (; d0 < static_cast<unsigned>(p.n_dist); d0 += gridDim.x * 128) {
        uint4 next[2][NG];
        load_r<NG>(p, h, d0 + gridDim.x * 128, next);
        for (int ct = 0; ct < n_ct; ++ct) {
            float acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int G = 0; G < NG; ++G) {
                const uint4 bw = *reinterpret_cast<const uint4*>(qvh + (8 * ct + g) * DP + 32 * (G ^ (g & 1)) + 8 * c4);
                mma::mma16816(acc, a[0][G].x, a[1][G].x, a[0][G].y, a[1][G].y, bw.x, bw.y);
                mma::mma16816(acc, a[0][G].z, a[1][G].z, a[0][G].w, a[1][G].w, bw.z, bw.w);
            }
            const int pr = 4 * ct + c4;
            if (pr < pairs) {
                float* e = e_key[pr];
                const int x0 = x_zero[pr];
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                    const int delta = static_cast<int>(d0 + g + 8 * y);
                    const float v = both_parts(acc[2 * y], acc[2 * y + 1]);
                    if (delta <= x0) e[-delta] = v;
                    if (delta == p.C) *far_at[pr] = v;
                }
            }
        }
#pragma unroll
        for (int G = 0; G < NG; ++G) {
            a[0][G] = next[0][G];
            a[1][G] = next[1][G];
        }
    }
}

// The same in fp32 arithmetic: 64 distances (32 of heads above 64) by up to 32 pairs per CTA, rows of both in shared
// memory; a thread takes two pairs, 16 apart, by distances 16 apart.  Bound by the loads from shared memory: 16 pairs
// by 2000 distances of B4 H16 D64 take 11.6 us, half of it the launch (a thread per pair and distance, reading its row of r itself: 125).
template <int NG>
__global__ void __launch_bounds__(kThreads) qpos_f32_kernel(const __grid_constant__ QattnParams p)
{
    constexpr int DP = NG * 32, P = DP + 4, TD = NG == 2 ? 64 : 32, PAIRS = 32, UPR = DP / 8;
    __shared__ __align__(16) float r[TD * P], q[PAIRS * P];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, h = blockIdx.y;
    const int pair0 = blockIdx.z * PAIRS, pairs = min(PAIRS, p.B * p.L - pair0);
    const unsigned d0 = blockIdx.x * static_cast<unsigned>(TD);
    pdl_wait();                                           // as in qpos_kernel
    pdl_launch_dependents();
#pragma unroll
    for (int x = tid; x < TD * UPR; x += kThreads) {
        const int row = x / UPR, d = 8 * (x % UPR);
        int rr = static_cast<int>(min(d0 + row, static_cast<unsigned>(p.C)));
        if (rr >= p.n_rows || !in_range(rr, 0, p.n_rows, p.chk)) rr = 0;      // past the distances of the call
        float v[8];
        load8<true>(static_cast<const float*>(p.r) + rr * p.r_row + h * p.r_head, d, p.D, p.vec_r, v);
        put8(r + row * P + d, v);
    }
    for (int x = tid; x < pairs * DP; x += kThreads) {
        const int pr = x / DP, d = x % DP, be = (pair0 + pr) / p.L, i = (pair0 + pr) - be * p.L;
        const int64_t at = be * p.q_sb + i * p.q_st + h * p.q_sh + d;
        q[pr * P + d] = d < p.D ? (ld(static_cast<const float*>(p.q) + at) + __ldg(p.vb + h * p.D + d)) * p.qscale : 0.f;
    }
    __syncthreads();
    const int qp = (warp & 3) * 4 + (lane >> 3), kq = (warp >> 2) * 8 + (lane & 7);
    if ((warp & 3) * 4 >= pairs) return;                  // none of this warp's pairs
    float s[2][TD / 16] = {};
    const bool both = pairs > 16;
#pragma unroll 4
    for (int d = 0; d < DP; d += 4) {
        const float4 q0 = f4(q + qp * P + d);
#pragma unroll
        for (int x = 0; x < TD / 16; ++x) s[0][x] = dot4(q0, f4(r + (kq + 16 * x) * P + d), s[0][x]);
        if (both) {
            const float4 q1 = f4(q + (qp + 16) * P + d);
#pragma unroll
            for (int x = 0; x < TD / 16; ++x) s[1][x] = dot4(q1, f4(r + (kq + 16 * x) * P + d), s[1][x]);
        }
    }
#pragma unroll
    for (int a = 0; a < 2; ++a) {
        const int pr = qp + 16 * a;
        if (pr >= pairs) break;
        const int be = (pair0 + pr) / p.L, i = (pair0 + pr) - be * p.L;
        const int64_t row = (static_cast<int64_t>(be) * p.H + h) * p.L + i;
#pragma unroll
        for (int x = 0; x < TD / 16; ++x) {
            const int delta = static_cast<int>(d0 + kq + 16 * x), at = p.M + i - delta - p.jn;
            if (at >= 0 && delta < p.n_dist) p.E[row * p.e_pitch + at] = s[a][x];
            if (delta == p.C) p.far[row] = s[a][x];
        }
    }
}

// Position terms of the keys ja <= j < jb for queries i0 .. i0 + Lq - 1 of a CTA that computes them itself, as qpos_kernel
// does, and those at the clamp.
template <int NG>
__device__ __forceinline__ void own_terms(const QattnParams& p, const uint16_t* qvs, float* e_row0, float* far_s, int i0,
                                          int Lq, int ja, int jb, bool clamped)
{
    constexpr int QP = NG * 32 + 8;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, c4 = lane & 3, h = blockIdx.y;
    const int i_end = p.M + i0 + Lq;
    if (!p.f32) {
        auto tile = [&](int d0, bool clamp) {
            uint4 a[2][NG];
            load_r<NG>(p, h, d0, a);
            for (int ct = 0; 4 * ct < Lq; ++ct) {
                float acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int G = 0; G < NG; ++G) {
                    const uint4 bw = *reinterpret_cast<const uint4*>(qvs + (8 * ct + g) * QP + 32 * G + 8 * c4);
                    mma::mma16816(acc, a[0][G].x, a[1][G].x, a[0][G].y, a[1][G].y, bw.x, bw.y);
                    mma::mma16816(acc, a[0][G].z, a[1][G].z, a[0][G].w, a[1][G].w, bw.z, bw.w);
                }
                const int row = 4 * ct + c4;
                if (row >= Lq) continue;
                if (clamp) {
                    if (g == 0) far_s[row] = both_parts(acc[0], acc[1]);
                    continue;
                }
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                    const int j = p.M + i0 + row - (d0 + g + 8 * y);
                    if (j >= ja && j < jb) e_row0[static_cast<int64_t>(row) * p.e_pitch + (j - p.jn)] = both_parts(acc[2 * y], acc[2 * y + 1]);
                }
            }
        };
        for (int d0 = max(0, p.M + i0 + 1 - jb) + 16 * warp; d0 < i_end - ja; d0 += 16 * kWarps) tile(d0, false);
        if (clamped && warp == kWarps - 1) tile(p.C, true);
    } else {
        auto dot = [&](int row, int delta) {
            int rr = min(delta, p.C);
            if (!in_range(rr, 0, p.n_rows, p.chk)) rr = 0;
            const float* r = static_cast<const float*>(p.r) + rr * p.r_row + h * p.r_head;
            float sum = 0.f;
            for (int d = 0; d < p.D; d += 8) {
                float x[8];
                load8<true>(r, d, p.D, p.vec_r, x);
#pragma unroll
                for (int e = 0; e < 8; ++e) sum = fmaf(reinterpret_cast<const float*>(qvs)[row * QP + d + e], x[e], sum);
            }
            return sum;
        };
        const int n = max(0, jb - ja);
        for (int x = tid; x < Lq * n; x += kThreads) {
            const int row = x / n, j = ja + x % n, delta = p.M + i0 + row - j;
            if (delta >= 0) e_row0[static_cast<int64_t>(row) * p.e_pitch + (j - p.jn)] = dot(row, delta);
        }
        if (clamped && tid < Lq) far_s[tid] = dot(tid, p.C);
    }
}

// FUSED: the CTA computes its position terms itself (a variant, because its code costs the others 0.3 us).
template <int BITS, int NG, int QT, bool ONE, bool FUSED, bool WIDE>
__global__ void __launch_bounds__(kThreads, NG == 2 || (BITS == 4 && QT == 1) ? 2 : 1)
qattn_kernel(const __grid_constant__ QattnParams p, const __grid_constant__ QSplit sp)
{
    constexpr int DP = NG * 32;                           // channels, padded
    constexpr int NC = NG * BITS / 4;                     // 16-byte chunks of a code row
    constexpr int CPG = BITS / 4;                         // chunks of a group
    constexpr int KS = stage_keys(BITS, NG, QT);
    constexpr int kEOff = KS * q_row_bytes(NG, BITS);     // of a stage: rows, position terms
    constexpr int kEStride = e_stride(BITS, NG, QT, ONE);
    constexpr int kStageBytes = stage_bytes(BITS, NG, QT, ONE);
    constexpr int SUB = BITS == 4 ? 2 : 1;                // MMAs per register of codes and product
    constexpr int QP = DP + 8;                            // rows of q's parts: the three that a load of ONE reads
                                                          // (both parts, zeros) lie in different banks
    constexpr float kCode = WIDE ? 1.f : kTwo24;           // 1 / what a code of one is
    constexpr float kOdd = BITS == 4 ? 0.0625f : 1.f;     // and of odd channels, besides
    // of a parameter word (step, lo)
    auto lo_of = [](uint32_t w) {
        const float lo = __uint_as_float(w & 0xffff0000u);
        return WIDE ? fmaf(__uint_as_float(w << 16), kCentre<BITS>, lo) : lo;
    };
    constexpr int kOwn = ONE ? 1 : kDecodeMaxL;           // keys of the segment a query can see
    extern __shared__ __align__(128) uint8_t smem[];
    uint8_t* stages = smem;
    float* qu = reinterpret_cast<float*>(smem + kWarps * kStages * kStageBytes);   // [row][DP]: q+u in log2 units
    float* inbox = qu + kMaxRows * DP;                    // [row of this rank][rank][DP + 2]: O, m, l
    // [row][NG] bf16: what the fp16 parts of qu are multiples of, over what a code of one is
    uint16_t* norm = reinterpret_cast<uint16_t*>(inbox + kMaxRanks * (DP + 4));
    float* qsum = reinterpret_cast<float*>(norm + kMaxRows * NG);   // [row][NG]: group sums of qu
    float* own_s = qsum + kMaxRows * NG;                  // [row][kOwn]: scores of the segment's own keys
    float* weights = own_s + kMaxRows * kDecodeMaxL;      // [row][32]: of the parts that make the result
    uint16_t* quh = reinterpret_cast<uint16_t*>(weights + kMaxRows * 32);   // [2 row + part][QP]; rows past Lq are zeros
    uint16_t* qvs = quh + 2 * kMaxRows * QP;              // fused: [2 row + part][QP] of q+v in bf16, or [row][QP] floats
    float* far_s = reinterpret_cast<float*>(qvs + 2 * kMaxRows * QP);       // fused: [row]
    uint64_t* bars = reinterpret_cast<uint64_t*>(far_s + kMaxRows);         // [warp][stage]: copies landed
    int* abort_flag = reinterpret_cast<int*>(bars + kWarps * kStages);

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, c4 = lane & 3;
    const int rank = blockIdx.x % sp.ranks, i0 = blockIdx.x / sp.ranks * sp.lq;
    const int h = blockIdx.y, b = blockIdx.z;
    const int Lq = min(sp.lq, p.L - i0);
    const int64_t bh = static_cast<int64_t>(b) * p.H + h;
    // slots of an MMA's columns: slot = stream * Lp + query
    const int lp_log = ONE ? 0 : Lq >= 3 ? 2 : Lq - 1, Lp = 1 << lp_log;
    const int NS = ONE ? KS / 16 : QT > 1 ? 1 : min(4 >> lp_log, KS / 16);
    if (sp.ranks > 1) cluster_arrive();                   // waited for before the first write to another rank
    if (tid == 0) *abort_flag = 0;
    const WaitCtl wc{abort_flag, p.err_flag, kWaitTimeoutNs};

    if constexpr (FUSED) {
        pdl_wait();
        pdl_launch_dependents();
    }
    // ---- the queries' elements, requested before the copies fill the memory system (raw: the conversion would
    // wait for them).  qpos_kernel started this grid after everything before it had completed; from L2, because
    // this grid has not waited itself.
    uint32_t q_raw[NG];
    const bool my_row = warp < Lq;
#pragma unroll
    for (int e = 0; e < NG; ++e) {
        const int d = 32 * e + lane;
        q_raw[e] = 0;
        if (my_row && d < p.D) {
            const int64_t at = b * p.q_sb + (i0 + warp) * p.q_st + h * p.q_sh + d;
            if (p.f32) q_raw[e] = __ldcg(static_cast<const uint32_t*>(p.q) + at);
            else q_raw[e] = __ldcg(static_cast<const uint16_t*>(p.q) + at);
        }
    }

    // ---- and the lines of the segment's own keys and values (the last rank's work), into L2
    const bool has_own = rank == sp.ranks - 1;
    const int n_own = i0 + Lq;                            // own keys any of these queries sees
    if (has_own && (tid >> 3) < n_own) {
        const int e = p.f32 ? 4 : 2, j = tid >> 3, part = (tid & 3) * 128;     // a row has at most four lines
        const char* src = tid & 4 ? static_cast<const char*>(p.vcur) + (b * p.vc_sb + j * p.vc_st + h * p.vc_sh) * e
                                  : static_cast<const char*>(p.kcur) + (b * p.kc_sb + j * p.kc_st + h * p.kc_sh) * e;
        if (part < p.D * e) prefetch_l2(src + part);
    }

    // ---- this warp's copies: stage n covers keys j_lo + (8 n + warp) KS ..; its rows as they are in memory, one bulk
    // copy, two where the ring wraps.  The position terms follow once qpos_kernel is done; a stage's barrier
    // counts both.
    const int j_lo = static_cast<int>(min(static_cast<int64_t>(p.M), p.lo + static_cast<int64_t>(rank) * sp.range));
    const int j_hi = static_cast<int>(min(static_cast<int64_t>(p.M), static_cast<int64_t>(j_lo) + sp.range));
    const int n_stage = max(0, (j_hi - j_lo - warp * KS + kWarps * KS - 1) / (kWarps * KS));
    const int row_bytes = q_row_bytes(p.G, BITS), v_off = q_v_offset(p.G, BITS), par_off = q_par_offset(p.G, BITS);
    uint8_t* my_stages = stages + warp * kStages * kStageBytes;
    uint64_t* full = bars + warp * kStages;
    auto slot_of = [&](int j) {                           // of a logical key
        const int64_t s = static_cast<int64_t>(p.wp) + j;
        return static_cast<int>(s >= p.M ? s - p.M : s);
    };
    const uint32_t stage_addr = smem_u32(my_stages), full_addr = smem_u32(full);
    const uint8_t* head = p.rows + bh * p.M * row_bytes;
    // keys of the stage from j with position terms of their own, a multiple of four (a stage starts a
    // multiple of four keys from jn, and the rows of E have room)
    auto near_of = [&](int j) { return max(0, min(KS, (min(KS, j_hi - j) + 3) & ~3) - max(0, p.jn - j)); };
    // The whole warp: lane 0 copies rows, lane 1 those past the ring's wrap, lanes 2 .. the queries' position terms.
    // (One lane for all of them took 800 cycles per stage for one query, 1700 for eight.)
    const bool e_lane = lane >= 2 && lane < 2 + Lq;
    const float* e_src = p.E + (bh * p.L + i0 + (e_lane ? lane - 2 : 0)) * p.e_pitch;
    const uint32_t e_dst = kEOff + 4 * kEStride * (e_lane ? lane - 2 : 0);
    auto copy = [&](int n, bool codes, bool terms) {
        const int j = j_lo + (n * kWarps + warp) * KS, near = near_of(j), x0 = max(0, p.jn - j);
        const uint32_t st = stage_addr + (n % kStages) * kStageBytes, bar = full_addr + 8 * (n % kStages);
        const void* src = e_src + (j + x0 - p.jn);
        uint32_t dst = st + e_dst + 4 * x0, bytes = terms && e_lane ? near * 4 : 0;
        if (codes) {
            const int live = min(KS, j_hi - j);
            int slot = slot_of(j);
            if (!in_range(slot, 0, p.M, p.chk)) slot = 0;
            if (lane == 0) mbar_expect_tx_addr(bar, live * row_bytes + near * 4 * Lq);
            const int first = min(live, p.M - slot);
            if (lane < 2) {
                src = head + (lane ? 0 : static_cast<uint64_t>(slot) * row_bytes);
                dst = st + (lane ? first * row_bytes : 0);
                bytes = (lane ? live - first : first) * row_bytes;
            }
            __syncwarp();                                 // the barrier expects what follows
        }
        if (bytes > 0) bulk_load_addr(dst, src, bytes, bar);
    };
    if (lane == 0) {
#pragma unroll
        for (int n = 0; n < kStages; ++n) mbar_init(&full[n], 1);
        fence_mbar_init();
    }
    __syncwarp();
#pragma unroll
    for (int n = 0; n < kStages; ++n)
        if (n < n_stage) copy(n, true, false);

    // ---- queries: warp w prepares row w: (q+u) times scale log2 e in fp32, and with every group scaled by a power of
    // two so that its largest entry lies in [2^14, 2^15) as two fp16 parts, in the order in which the B operands
    // take them (4 bits: d = 0 4 1 5 2 6 3 7 of every eight, odd ones over 16; 8 bits: 0 2 1 3 of every four)
    {
        const int row = warp;
        float a[NG];
#pragma unroll
        for (int e = 0; e < NG; ++e) {
            const int d = 32 * e + lane;
            const float q = __uint_as_float(p.f32 ? q_raw[e] : q_raw[e] << 16);
            a[e] = my_row && d < p.D ? (q + __ldg(p.u + h * p.D + d)) * p.qscale : 0.f;
        }
#pragma unroll
        for (int e = 0; e < NG; ++e) {
            const int d = 32 * e + lane;
            qu[row * DP + d] = a[e];
            float mx = fabsf(a[e]);
#pragma unroll
            for (int off = 16; off > 0; off >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
            const int ex = max(static_cast<int>(__float_as_uint(mx) >> 23) - 127, -100);
            const float up = __uint_as_float(static_cast<uint32_t>(14 - ex + 127) << 23);
            if (lane == 0)
                norm[row * NG + e] = static_cast<uint16_t>(
                    __float_as_uint(__uint_as_float(static_cast<uint32_t>(ex - 14 + 127) << 23) * kCode) >> 16);
            const int at = BITS == 4 ? (d & ~7) + ((d & 3) << 1) + ((d >> 2) & 1) : (d & ~3) + ((d & 1) << 1) + ((d >> 1) & 1);
            uint32_t w, unused;
            split_f16(a[e] * (BITS == 4 && (d & 1) ? up * kOdd : up), 0.f, w, unused);
            quh[2 * row * QP + at] = static_cast<uint16_t>(w);
            quh[(2 * row + 1) * QP + at] = static_cast<uint16_t>(w >> 16);
            float sum = a[e];
#pragma unroll
            for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
            if (lane == 0) qsum[row * NG + e] = sum;
            if constexpr (FUSED) {
                const float q = __uint_as_float(p.f32 ? q_raw[e] : q_raw[e] << 16);
                const float c = my_row && d < p.D ? (q + __ldg(p.vb + h * p.D + d)) * p.qscale : 0.f;
                if (p.f32) {
                    reinterpret_cast<float*>(qvs)[row * QP + d] = c;
                } else {
                    const __nv_bfloat16 hi = __float2bfloat16_rn(c);
                    qvs[2 * row * QP + d] = __bfloat16_as_ushort(hi);
                    qvs[(2 * row + 1) * QP + d] = __bfloat16_as_ushort(__float2bfloat16_rn(c - __bfloat162float(hi)));
                }
            }
        }
    }
    __syncthreads();

    // ---- B operands of Q.K, column g = (slot g/2, part g%2), and per slot c4 the group sums of q.  ONE: the
    // k-quarter of this lane belongs to stream c4, so only columns of slot c4 are not zero there.
    uint32_t bq[QT][NG * 2][2];
    float qs[QT][NG], far_of[QT];
    uint32_t sc[QT][NG / 2];
    const int my_stream = (g >> 1) >> lp_log;             // of the column this lane holds in B operands
    const int one_key = (g + 2 * c4) & 7;
    const uint16_t* one_row = quh + ((g >> 1) == c4 ? (g & 1) : 2) * QP;       // or zeros
#pragma unroll
    for (int t = 0; t < QT; ++t) {
        if constexpr (!ONE) {
            const int il = min(((g >> 1) & (Lp - 1)) + 4 * t, Lq - 1);
            const uint16_t* row = quh + (2 * il + (g & 1)) * QP;
#pragma unroll
            for (int G = 0; G < NG; ++G) {
                if constexpr (BITS == 4) {
                    const uint4 w = *reinterpret_cast<const uint4*>(row + 32 * G + 8 * c4);
                    bq[t][2 * G][0] = w.x; bq[t][2 * G][1] = w.y;
                    bq[t][2 * G + 1][0] = w.z; bq[t][2 * G + 1][1] = w.w;
                } else {
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        const uint2 w = *reinterpret_cast<const uint2*>(row + 32 * G + 16 * x + 4 * c4);
                        bq[t][2 * G + x][0] = w.x; bq[t][2 * G + x][1] = w.y;
                    }
                }
            }
        }
        const int is = min((c4 & (Lp - 1)) + 4 * t, Lq - 1);
#pragma unroll
        for (int G = 0; G < NG; ++G) qs[t][G] = qsum[is * NG + G];
#pragma unroll
        for (int G = 0; G < NG; G += 2) sc[t][G / 2] = *reinterpret_cast<const uint32_t*>(norm + is * NG + G);
    }

    float* e_row0 = p.E + (bh * p.L + i0) * p.e_pitch;
    if constexpr (FUSED) {
        own_terms<NG>(p, qvs, e_row0, far_s, i0, Lq, max(j_lo, p.jn), has_own ? p.M + n_own : j_hi, p.jn > j_lo);
        fence_proxy_async_global();                       // the copies read what was stored
        __syncthreads();
    } else {
        // ---- from here on the position terms are there
        pdl_wait();
        pdl_launch_dependents();
    }
#pragma unroll
    for (int t = 0; t < QT; ++t) {
        const int is = min((c4 & (Lp - 1)) + 4 * t, Lq - 1);
        far_of[t] = p.jn <= j_lo ? 0.f : FUSED ? far_s[is] : __ldcg(p.far + bh * p.L + i0 + is);
    }
#pragma unroll
    for (int n = 0; n < kStages; ++n)
        if (n < n_stage) copy(n, false, true);

    // ---- running state of slot c4: maximum, units rf of the weights by group (O is in units of rf), sums
    float o[QT][NG * 2][4], z[QT][NG], m[QT], l[QT];
    uint32_t rf[QT][NG / 2];
#pragma unroll
    for (int t = 0; t < QT; ++t) {
        m[t] = kNoMax;
        l[t] = 0.f;
#pragma unroll
        for (int G = 0; G < NG / 2; ++G) rf[t][G] = kMinUnits;
#pragma unroll
        for (int G = 0; G < NG; ++G) z[t][G] = 0.f;
#pragma unroll
        for (int x = 0; x < NG * 2; ++x) o[t][x][0] = o[t][x][1] = o[t][x][2] = o[t][x][3] = 0.f;
    }

    int n = 0;
    for (; n < n_stage; ++n) {
        if (!warp_wait(&full[n % kStages], (n / kStages) & 1, wc, 50)) break;      // abandoned: no result is valid
        const int js = j_lo + (n * kWarps + warp) * KS;
        const uint8_t* st = my_stages + (n % kStages) * kStageBytes;
        const uint32_t st_addr = stage_addr + (n % kStages) * kStageBytes;
        const bool whole = js + KS <= j_hi;               // no row past the end
        for (int k0 = 0; k0 < (ONE ? 1 : KS); k0 += 16 * NS) {
            if (js + k0 >= j_hi) break;
            // Q.K: acc[t][G] = for slot c4, two keys of its stream's tile, (hi, lo) parts: keys g and g+8; ONE:
            // keys (g + 2 c4) mod 8 and 8 more, so that eight lanes of a load read rows 0 .. 7 of the eight
            float acc[QT][NG][4];
            if constexpr (QT == 1 && !ONE) {                          // several tiles may add up
#pragma unroll
                for (int G = 0; G < NG; ++G) acc[0][G][0] = acc[0][G][1] = acc[0][G][2] = acc[0][G][3] = 0.f;
            }
            if constexpr (ONE) {
                const uint32_t row0 = st_addr + (16 * min(c4, KS / 16 - 1) + one_key) * row_bytes, row1 = row0 + 8 * row_bytes;
#pragma unroll
                for (int c = 0; c < NC; ++c) {
                    uint32_t wa[4], wb[4];
                    lds128(row0 + 16 * c, wa);
                    lds128(row1 + 16 * c, wb);
                    const uint16_t* bsrc = one_row + c * (128 / BITS);
#pragma unroll
                    for (int w = 0; w < 4; ++w) {
                        uint32_t bb[2 * SUB];
                        if constexpr (BITS == 4) {
                            const uint4 v = *reinterpret_cast<const uint4*>(bsrc + 8 * w);
                            bb[0] = v.x; bb[1] = v.y; bb[2] = v.z; bb[3] = v.w;
                        } else {
                            const uint2 v = *reinterpret_cast<const uint2*>(bsrc + 4 * w);
                            bb[0] = v.x; bb[1] = v.y;
                        }
#pragma unroll
                        for (int s = 0; s < SUB; ++s) {
                            const uint32_t x = wa[w] >> (8 * s), y = wb[w] >> (8 * s);
                            if (c % CPG == 0 && w == 0 && s == 0)
                                mma_f16_first(acc[0][c / CPG], pair_even<BITS, WIDE>(x), pair_even<BITS, WIDE>(y), pair_odd<BITS, WIDE>(x),
                                              pair_odd<BITS, WIDE>(y), bb[2 * s], bb[2 * s + 1]);
                            else
                                mma_f16(acc[0][c / CPG], pair_even<BITS, WIDE>(x), pair_even<BITS, WIDE>(y), pair_odd<BITS, WIDE>(x),
                                        pair_odd<BITS, WIDE>(y), bb[2 * s], bb[2 * s + 1]);
                        }
                    }
                }
            } else {
                for (int T = 0; T < NS; ++T) {
                    const bool on = QT > 1 || my_stream == T;
                    const uint32_t row = st_addr + (k0 + 16 * T + (lane & 15)) * row_bytes + (lane & 16);
#pragma unroll
                    for (int c2 = 0; c2 < NC; c2 += 2) {
                        uint32_t w[4];
                        mma::ldsm_x4(row + 16 * c2, w[0], w[1], w[2], w[3]);
#pragma unroll
                        for (int half = 0; half < 2; ++half) {
                            const int c = c2 + half;
#pragma unroll
                            for (int s = 0; s < SUB; ++s) {
                                const uint32_t x = w[2 * half] >> (8 * s), y = w[2 * half + 1] >> (8 * s);
                                const int ks = c * SUB + s;
#pragma unroll
                                for (int t = 0; t < QT; ++t) {
                                    if (QT > 1 && c % CPG == 0 && s == 0)
                                        mma_f16_first(acc[t][c / CPG], pair_even<BITS, WIDE>(x), pair_even<BITS, WIDE>(y),
                                                      pair_odd<BITS, WIDE>(x), pair_odd<BITS, WIDE>(y), bq[t][ks][0], bq[t][ks][1]);
                                    else
                                        mma_f16(acc[t][c / CPG], pair_even<BITS, WIDE>(x), pair_even<BITS, WIDE>(y), pair_odd<BITS, WIDE>(x),
                                                pair_odd<BITS, WIDE>(y), on ? bq[t][ks][0] : 0u, on ? bq[t][ks][1] : 0u);
                                }
                            }
                        }
                    }
                }
            }
            // scores, weights, and the P operands: two keys per lane
            const int kk = k0 + 16 * (c4 >> lp_log) + (ONE ? one_key : g);     // key of the stage (and kk + 8)
            const bool in_use = (c4 >> lp_log) < NS;              // slots past the streams hold no keys
            uint2 par[2][NG];
            bool live[2] = {true, true};
            const uint8_t* par_row = st + (in_use ? kk : g) * row_bytes + par_off;
#pragma unroll
            for (int x = 0; x < 2; ++x)
#pragma unroll
                for (int G = 0; G < NG; G += 2) {
                    const uint4 w = *reinterpret_cast<const uint4*>(par_row + 8 * x * row_bytes + 8 * G);
                    par[x][G] = make_uint2(w.x, w.y);
                    par[x][G + 1] = make_uint2(w.z, w.w);
                }
            if (!whole || NS << lp_log < 4) {                     // rows past the end hold what was there before
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    live[x] = in_use && js + kk + 8 * x < j_hi;
#pragma unroll
                    for (int G = 0; G < NG; ++G)
                        if (!live[x]) par[x][G] = make_uint2(0, 0);
                }
            }
            const float* e_st = reinterpret_cast<const float*>(st + kEOff) + (in_use ? kk : g);
            const bool near0 = js + kk >= p.jn, near1 = js + kk + 8 >= p.jn;      // terms of their own
            uint32_t bp[QT][NG][2];
#pragma unroll
            for (int t = 0; t < QT; ++t) {
                const int il = ONE ? 0 : min((c4 & (Lp - 1)) + 4 * t, Lq - 1);
                float s[2], pr[2], w[2][NG];
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    float a = (x ? near1 : near0) ? e_st[il * kEStride + 8 * x] : far_of[t], d = 0.f;
#pragma unroll
                    for (int G = 0; G < NG; ++G) {
                        d = fmaf((acc[t][G][2 * x] + acc[t][G][2 * x + 1]) * unit_of(sc[t][G / 2], G),
                                 __uint_as_float(par[x][G].x << 16), d);
                        a = fmaf(lo_of(par[x][G].x), qs[t][G], a);
                    }
                    s[x] = live[x] ? d + a : -INFINITY;
                    pr[x] = ex2_approx(s[x] - m[t]);
                }
                float big = fmaxf(pr[0], pr[1]) * 128.f;
#pragma unroll
                for (int G = 0; G < NG; ++G) {
                    const float f = unit_of(one_over(rf[t][G / 2]), G);
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        w[x][G] = pr[x] * f * __uint_as_float(par[x][G].y << 16);
                        big = fmaxf(big, w[x][G]);
                    }
                }
                if (__any_sync(0xffffffffu, big > 32768.f)) {
                    // a weight grew past 2^8, or its product with a step past 2^15 units: new maximum and units
                    float mx = fmaxf(s[0], s[1]);
#pragma unroll
                    for (int off = 4; off <= 16; off <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
                    const float mn = fmaxf(m[t], mx);
                    const float dl = ex2_approx(m[t] - mn);
#pragma unroll
                    for (int x = 0; x < 2; ++x) pr[x] = ex2_approx(s[x] - mn);
                    m[t] = mn;
                    l[t] *= dl;
#pragma unroll
                    for (int G = 0; G < NG; ++G) {
                        float ref = fmaxf(pr[0] * __uint_as_float(par[0][G].y << 16), pr[1] * __uint_as_float(par[1][G].y << 16));
#pragma unroll
                        for (int off = 4; off <= 16; off <<= 1) ref = fmaxf(ref, __shfl_xor_sync(0xffffffffu, ref, off));
                        const float was = unit_of(rf[t][G / 2], G);
                        ref = fminf(fmaxf(fmaxf(ref * 0.00390625f, was * dl), kMinUnit), kMaxUnit);
                        const uint32_t unit = __float_as_uint(ref) & 0x7f800000u;        // its power of two
                        const float f = __uint_as_float(0x7f000000u - unit), so = dl * was * f;
                        rf[t][G / 2] = __byte_perm(rf[t][G / 2], unit, G & 1 ? 0x7610 : 0x3276);
                        z[t][G] *= dl;
#pragma unroll
                        for (int x = 2 * G; x < 2 * G + 2; ++x) {
                            o[t][x][0] *= so; o[t][x][1] *= so; o[t][x][2] *= so; o[t][x][3] *= so;
                        }
#pragma unroll
                        for (int x = 0; x < 2; ++x) w[x][G] = pr[x] * f * __uint_as_float(par[x][G].y << 16);
                    }
                }
                l[t] += pr[0] + pr[1];
#pragma unroll
                for (int G = 0; G < NG; ++G) {
                    z[t][G] = fmaf(pr[0], lo_of(par[0][G].y), fmaf(pr[1], lo_of(par[1][G].y), z[t][G]));
                    // row = key, columns (2 slot, 2 slot + 1) -> rows = columns of B, pairs of keys
                    uint32_t w0, w1;
                    split_f16(w[0][G], w[1][G], w0, w1);
                    bp[t][G][0] = transpose8(w0);
                    bp[t][G][1] = transpose8(w1);
                }
            }
            // P.V: o[t][mt] = for slot c4, channels of row g and g+8 of the tile, (hi, lo) parts
            auto pv_tile = [&](int T) {
                const bool on = QT > 1 || my_stream == T;
                const int key = ONE ? ((lane + 2 * T) & 7) | (lane & 8) : lane & 15;
                const uint32_t row = st_addr + (k0 + 16 * T + key) * row_bytes + v_off + (lane & 16);
#pragma unroll
                for (int c2 = 0; c2 < NC; c2 += 2) {
                    uint32_t w[4];
                    mma::ldsm_x4_t(row + 16 * c2, w[0], w[1], w[2], w[3]);
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        const int c = c2 + half, G = c / CPG;
#pragma unroll
                        for (int s = 0; s < SUB; ++s) {
                            const uint32_t x = w[2 * half] >> (8 * s), y = w[2 * half + 1] >> (8 * s);
#pragma unroll
                            for (int t = 0; t < QT; ++t)
                                mma_f16(o[t][c * SUB + s], pair_even<BITS, WIDE>(x), pair_odd<BITS, WIDE>(x), pair_even<BITS, WIDE>(y),
                                        pair_odd<BITS, WIDE>(y), on ? bp[t][G][0] : 0u, on ? bp[t][G][1] : 0u);
                        }
                    }
                }
            };
            if constexpr (QT > 1) {
                pv_tile(0);
            } else if constexpr (ONE) {
#pragma unroll
                for (int T = 0; T < KS / 16; ++T) pv_tile(T);
            } else {
                for (int T = 0; T < NS; ++T) pv_tile(T);
            }
        }
        __syncwarp();                                     // every lane has read the stage
        if (n + kStages < n_stage) copy(n + kStages, true, true);
    }
    // ---- scores of the segment's own keys: eight lanes per key hold its row, and the groups of lanes share the
    // queries.  (After the key loop: before it the loads waited behind the copies, 10000 cycles, with the
    // queries of all warps.)
    if (has_own) {
        const int kp_log = ONE ? 0 : 32 - __clz(n_own - 1);          // groups 2^kp_log apart have the same key
        const int group = tid >> 3, j = group & ((1 << kp_log) - 1), row0 = group >> kp_log, row_step = 32 >> kp_log;
        float k[DP / 64][8], e[ONE ? 1 : 4];                         // eight queries at most, and 16 keys
        const int64_t at = b * p.kc_sb + min(j, n_own - 1) * p.kc_st + h * p.kc_sh;
#pragma unroll
        for (int x = 0; x < DP / 64; ++x) {
            const int d = 64 * x + 8 * (lane & 7);
            if (p.f32) load8<true>(static_cast<const float*>(p.kcur) + at, d, p.D, p.vec_k, k[x]);
            else load8<false>(static_cast<const uint16_t*>(p.kcur) + at, d, p.D, p.vec_k, k[x]);
        }
#pragma unroll
        for (int y = 0; y < (ONE ? 1 : 4); ++y) {
            const int row = row0 + y * row_step;
            e[y] = row < Lq && j <= i0 + row ? __ldcg(e_row0 + static_cast<int64_t>(row) * p.e_pitch + (p.M + j - p.jn)) : -INFINITY;
        }
#pragma unroll
        for (int y = 0; y < (ONE ? 1 : 4); ++y) {
            if (y * row_step >= Lq) break;
            const int row = row0 + y * row_step;
            const float* qr = qu + min(row, Lq - 1) * DP + 8 * (lane & 7);
            float s = 0.f;
#pragma unroll
            for (int x = 0; x < DP / 64; ++x)
#pragma unroll
                for (int z8 = 0; z8 < 8; ++z8) s = fmaf(qr[64 * x + z8], k[x][z8], s);
#pragma unroll
            for (int off = 4; off > 0; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
            if ((lane & 7) == 0 && row < Lq && j < n_own) own_s[row * kOwn + j] = s + e[y];
        }
    }
    if (n < n_stage && lane == 0)                         // abandoned: no copy may land after the CTA has gone
        for (int x = n; x < min(n + kStages, n_stage); ++x) {
            int never = 0;
            const WaitCtl dw{&never, nullptr, 100000000ull};
            (void)mbar_wait(&full[x % kStages], (x / kStages) & 1, dw, 51);
        }
    __syncthreads();

    // ---- merge: the streams of a warp, its warps and the segment's own keys, the ranks
    float* part = reinterpret_cast<float*>(stages);       // [warp][query][DP + 2]
#pragma unroll
    for (int t = 0; t < QT; ++t) {
        float lt = l[t], zt[NG], ot[NG * 4];
#pragma unroll
        for (int off = 4; off <= 16; off <<= 1) lt += __shfl_xor_sync(0xffffffffu, lt, off);
#pragma unroll
        for (int G = 0; G < NG; ++G) {
            zt[G] = z[t][G];
#pragma unroll
            for (int off = 4; off <= 16; off <<= 1) zt[G] += __shfl_xor_sync(0xffffffffu, zt[G], off);
        }
#pragma unroll
        for (int x = 0; x < NG * 2; ++x) {
            // (the unit last: times 2^24 it could leave fp32)
            const float unit = unit_of(rf[t][x >> 2], x >> 1);
            ot[2 * x] = fmaf((o[t][x][0] + o[t][x][1]) * kCode, unit, zt[x >> 1]);
            ot[2 * x + 1] = fmaf((o[t][x][2] + o[t][x][3]) * (kCode * kOdd), unit, zt[x >> 1]);
        }
        float mt = m[t];
        for (int off = Lp; off <= 2; off <<= 1) {
            const float mo = __shfl_xor_sync(0xffffffffu, mt, off);
            const float mn = fmaxf(mt, mo);
            const float a = ex2_approx(mt - mn), c = ex2_approx(mo - mn);
            mt = mn;
            lt = lt * a + __shfl_xor_sync(0xffffffffu, lt, off) * c;
#pragma unroll
            for (int x = 0; x < NG * 4; ++x) ot[x] = ot[x] * a + __shfl_xor_sync(0xffffffffu, ot[x], off) * c;
        }
        const int il = c4 + 4 * t;
        if (c4 < Lp && il < Lq) {
            float* dst = part + (warp * sp.lq + il) * (DP + 2);
#pragma unroll
            for (int x = 0; x < NG * 2; ++x) {
                const int d = BITS == 4 ? 32 * (x >> 1) + 4 * g + 2 * (x & 1) : 16 * x + 2 * g;
                dst[d] = ot[2 * x];
                dst[d + 1] = ot[2 * x + 1];
            }
            if (g == 0) {
                dst[DP] = mt;
                dst[DP + 1] = lt;
            }
        }
    }
    if (sp.ranks > 1) cluster_wait();                     // every rank has started
    __syncthreads();
    // Row r is finished by rank r mod ranks, whose inbox takes the ranks' partial results of it.  First a warp per
    // row takes the weights of its parts: lanes 0 .. 7 the warps' partial results, the others own keys.
    if (warp < Lq) {
        const int own = has_own ? min(i0 + warp + 1, kOwn) : 0;
        const float* src = part + (min(lane, kWarps - 1) * sp.lq + warp) * (DP + 2);
        const bool of_warp = lane < kWarps, of_key = lane >= kWarps && lane - kWarps < own;
        const float val = of_warp ? src[DP] : of_key ? own_s[warp * kOwn + lane - kWarps] : kNoMax;
        float mx = val;
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
        const float w = of_warp || of_key ? ex2_approx(val - mx) : 0.f;
        float lt = w * (of_warp ? src[DP + 1] : 1.f);
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) lt += __shfl_xor_sync(0xffffffffu, lt, off);
        weights[warp * 32 + lane] = w;
        if (lane == 0) {
            float* dst = inbox + (warp / sp.ranks * sp.ranks + rank) * (DP + 2) + DP;
            st_rank(dst, warp % sp.ranks, mx);
            st_rank(dst + 1, warp % sp.ranks, lt);
        }
    }
    __syncthreads();
    for (int x = tid; x < Lq * DP; x += kThreads) {
        const int row = x / DP, d = x % DP;
        const int own = has_own && d < p.D ? min(i0 + row + 1, kOwn) : 0;
        // the values of all own keys at once: the type is told apart outside the loop, so that the loads overlap
        uint32_t v[kOwn];
        const int64_t v_at = b * p.vc_sb + h * p.vc_sh + d;
        if (p.f32) {
#pragma unroll
            for (int j = 0; j < kOwn; ++j) v[j] = j < own ? ld(static_cast<const uint32_t*>(p.vcur) + v_at + j * p.vc_st) : 0u;
        } else {
#pragma unroll
            for (int j = 0; j < kOwn; ++j) v[j] = j < own ? ld(static_cast<const uint16_t*>(p.vcur) + v_at + j * p.vc_st) : 0u;
        }
        const float* w = weights + row * 32;
        float ot = 0.f;
#pragma unroll
        for (int k = 0; k < kWarps; ++k) ot = fmaf(part[(k * sp.lq + row) * (DP + 2) + d], w[k], ot);
#pragma unroll
        for (int j = 0; j < kOwn; ++j)
            if (j < own) ot = fmaf(w[kWarps + j], __uint_as_float(p.f32 ? v[j] : v[j] << 16), ot);
        st_rank(inbox + (row / sp.ranks * sp.ranks + rank) * (DP + 2) + d, row % sp.ranks, ot);
    }
    __syncthreads();
    if (sp.ranks > 1) cluster_sync_all();
    const int my_rows = (Lq - rank + sp.ranks - 1) / sp.ranks;
    for (int x = tid; x < my_rows * DP; x += kThreads) {
        const int k = x / DP, d = x % DP, row = rank + k * sp.ranks;
        if (d >= p.D) continue;
        const float* src = inbox + k * sp.ranks * (DP + 2);
        float mx = kNoMax, lt = 0.f, ot = 0.f;
        for (int r = 0; r < sp.ranks; ++r) mx = fmaxf(mx, src[r * (DP + 2) + DP]);
        for (int r = 0; r < sp.ranks; ++r) {
            const float a = ex2_approx(src[r * (DP + 2) + DP] - mx);
            lt += src[r * (DP + 2) + DP + 1] * a;
            ot += src[r * (DP + 2) + d] * a;
        }
        const int64_t at = b * p.o_sb + (i0 + row) * p.o_st + h * p.o_sh + d;
        if (p.f32) static_cast<float*>(p.out)[at] = ot / lt;
        else static_cast<__nv_bfloat16*>(p.out)[at] = __float2bfloat16_rn(ot / lt);
    }
}

cudaError_t launch_qpos(const QattnParams& p, int ng, int sm_count, cudaStream_t s)
{
    const int64_t pairs = static_cast<int64_t>(p.B) * p.L;
    if (p.f32) {
        const int td = ng == 2 ? 64 : 32;
        const dim3 grid((p.n_dist + td - 1) / td, p.H, static_cast<unsigned>((pairs + 31) / 32));
        return launch_dependent(ng == 2 ? qpos_f32_kernel<2> : qpos_f32_kernel<4>, grid, dim3(kThreads), 0, s, p);
    }
    // four CTAs per SM, each walking over its share of the distances (65536 keys of 16 heads, the whole call:
    // 62.4 us with two, 58.3 with three, 56.0 with four, 58.7 with six)
    const int64_t tiles = (static_cast<int64_t>(p.n_dist) + 127) / 128, sets = (pairs + pos_pairs(ng) - 1) / pos_pairs(ng);
    const int64_t per_head = std::max<int64_t>(1, 4 * sm_count / (sets * p.H));
    const dim3 grid(static_cast<unsigned>(std::min(tiles, per_head)), p.H, static_cast<unsigned>(sets));
    auto* kernel = ng > 2 ? qpos_kernel<4, true> : tiles * sets * p.H > 3 * sm_count ? qpos_kernel<2, true> : qpos_kernel<2, false>;
    return launch_dependent(kernel, grid, dim3(kThreads), 0, s, p);
}

template <int BITS, int NG, int QT, bool ONE, bool WIDE>
cudaError_t launch(const QattnParams& p, QSplit sp, int groups, int sm_count, cudaStream_t s)
{
    constexpr int DP = NG * 32;
    constexpr int staged = kWarps * kStages * stage_bytes(BITS, NG, QT, ONE);
    constexpr int bytes = staged + (kMaxRows * (DP + NG / 2 + NG + kDecodeMaxL + 32) + kMaxRanks * (DP + 4)) * 4 +
                          4 * kMaxRows * (DP + 8) * 2 + kMaxRows * 4 + kWarps * kStages * 8 + 16;
    static_assert(staged >= kWarps * stage_rows(QT, ONE) * (DP + 2) * 4, "the warps' partial results fit");
    static_assert(bytes <= 232448, "a CTA's shared memory");
    auto* kernel = qattn_kernel<BITS, NG, QT, ONE, false, WIDE>;
    auto* fused_kernel = qattn_kernel<BITS, NG, QT, ONE, true, WIDE>;
    // once per device: the shared memory, clusters of more than eight, and how many clusters of each size the device
    // holds at a time
    static OncePerDevice once;
    static std::atomic<int> held[64][kMaxRanks + 1];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    e = once([&] {
        for (auto* k : {kernel, fused_kernel}) {
            e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
            if (e == cudaSuccess) e = cudaFuncSetAttribute(k, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
            if (e != cudaSuccess) return e;
        }
        for (int ranks = 1; ranks <= kMaxRanks && e == cudaSuccess; ++ranks) {
            cudaLaunchConfig_t cfg = {};
            cfg.gridDim = dim3(ranks * 64);
            cfg.blockDim = dim3(kThreads);
            cfg.dynamicSmemBytes = bytes;
            cudaLaunchAttribute attr[1];
            attr[0].id = cudaLaunchAttributeClusterDimension;
            attr[0].val.clusterDim.x = ranks;
            attr[0].val.clusterDim.y = 1;
            attr[0].val.clusterDim.z = 1;
            cfg.attrs = attr;
            cfg.numAttrs = 1;
            int n = 0;
            e = cudaOccupancyMaxActiveClusters(&n, kernel, &cfg);
            held[dev & 63][ranks].store(n, std::memory_order_relaxed);
        }
        return e;
    });
    if (e != cudaSuccess) return e;
    // Key ranges: the cluster size whose waves of clusters, each over 1/ranks of the keys, take the least time, while
    // each warp keeps a stage.  A GPC holds a whole number of clusters, so that large ones leave SMs idle: 16 heads of
    // one sequence fit in one wave as clusters of up to 13 (65536 4-bit keys: 48.4 us when chosen), not of 16 (55.6; 8: 57.7).
    constexpr int ks = stage_keys(BITS, NG, QT);
    const int64_t keys = p.M - p.lo, heads = static_cast<int64_t>(p.H) * p.B * groups;
    int64_t waves = 0;
    for (int ranks = 1; ranks <= kMaxRanks; ++ranks) {
        const int n = held[dev & 63][ranks].load(std::memory_order_relaxed);
        if (ranks > 1 && (n == 0 || keys <= static_cast<int64_t>(ranks) * ks * kWarps)) continue;
        const int64_t w = n ? (heads + n - 1) / n : heads;
        if (ranks > 1 && w * sp.ranks >= waves * ranks) continue;
        sp.ranks = ranks;
        waves = w;
    }
    sp.range = static_cast<int>(((keys + sp.ranks - 1) / sp.ranks + ks - 1) / ks * ks);
    if (sp.range == 0) sp.range = ks;
    // Position terms in the kernel itself where a CTA has few: one launch less.  One query of 16 heads, B 1: over 250 keys
    // 8.0 instead of 10.2 us eagerly (the host), 6.2 instead of 6.0 replayed; over 500 keys 8.4 and 7.8, over 1000
    // 11.0 instead of 7.3.  fp32, a dot product per thread: over 250 keys 8.0 instead of 9.6 eagerly, 7.6 instead of
    // 6.4 replayed; over 500 keys 10.4 instead of 9.8.
    const int64_t near = std::min<int64_t>(sp.range, p.M - p.jn) + p.L;
    const bool fused = (p.f32 ? near * sp.lq : near) <= 256;
    if (!fused) {
        e = launch_qpos(p, NG, sm_count, s);
        if (e != cudaSuccess) return e;
    }
    const dim3 grid(sp.ranks * groups, p.H, p.B);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = bytes;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = sp.ranks;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, fused ? fused_kernel : kernel, p, sp);
}

template <int BITS, int NG, bool WIDE>
cudaError_t launch_qt(const QattnParams& p, const QSplit& sp, int groups, int sm_count, cudaStream_t s)
{
    if (sp.lq == 1) return launch<BITS, NG, 1, true, WIDE>(p, sp, groups, sm_count, s);
    return sp.lq <= 4 ? launch<BITS, NG, 1, false, WIDE>(p, sp, groups, sm_count, s)
                      : launch<BITS, NG, 2, false, WIDE>(p, sp, groups, sm_count, s);
}

template <int BITS, int NG>
cudaError_t launch_type(const QattnParams& p, const QSplit& sp, int groups, int sm_count, cudaStream_t s)
{
    return p.f32 ? launch_qt<BITS, NG, true>(p, sp, groups, sm_count, s)
                 : launch_qt<BITS, NG, false>(p, sp, groups, sm_count, s);
}

}  // namespace

cudaError_t launch_qattn(const QattnParams& p, int sm_count, cudaStream_t s)
{
    const int ng = p.G <= 2 ? 2 : 4, bits = p.bits == 8 ? 8 : 4;
    QSplit sp{};
    const int groups = p.L > 8 ? 2 : 1;                   // queries: eight at most per CTA
    sp.lq = (p.L + groups - 1) / groups;
    if (bits == 4) return ng == 2 ? launch_type<4, 2>(p, sp, groups, sm_count, s) : launch_type<4, 4>(p, sp, groups, sm_count, s);
    return ng == 2 ? launch_type<8, 2>(p, sp, groups, sm_count, s) : launch_type<8, 4>(p, sp, groups, sm_count, s);
}

}  // namespace txl
