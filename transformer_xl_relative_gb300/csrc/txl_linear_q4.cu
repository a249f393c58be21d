// txl_linear_q4.cu -- Y = X W for few rows of X, with W held as 4-bit codes: groups of 32, 64 or 128 entries of a
// column share a bf16 step and minimum lo, w = lo + step c (the projections of "TransformerXL 相对位置编码" §3.1).
//
//     y = sum over groups ( step sum_k x_k c_k + lo sum_k x_k ),     c exact in bf16, sums in fp32
//
// 8 rows by 8192 x 8192 (36 MB): 10.9 us, 3.3 TB/s; bound by the ALU that makes operands of the codes (28 instructions for 16 columns by 64 k; 57 % of the
// pipe's cycles over all SMs, 67 % on those that have a block).  4096 x 4096 4.9 us; one row by 1024 x 1024 2.1 us, a launch.
#include <cuda_bf16.h>

#include "txl_mma.cuh"
#include "txl_internal.h"
#include "txl_ptx.cuh"

namespace txl {

namespace {

// A block of codes: 16 columns of W (rows of an mma's A) by 64 k.  Lane (g, t) holds 32 codes: word s (0..3) those of a k16
// step, k = 32 (s / 2) + 8 t + 4 (s % 2) + 0..3, so that a lane's x are two pieces of 16 bytes and a step stays within 32 k.
// Nibble j of a word and nibble j + 4 are a pair of A's register j: column g + 8 (j % 2), k + 2 (j / 2) and the next.
// Blocks of four neighbouring tiles of columns and one block of k follow one another, and so do the parameters of four tiles and a
// group, so that a block of threads reads pieces of up to 2 KB.
constexpr int kQ4K = 64, kQ4N = 16;

__device__ __forceinline__ int64_t code_block(int nt, int kb, int kb_all)        // in 512 bytes
{
    return (static_cast<int64_t>(nt >> 2) * kb_all + kb) * 4 + (nt & 3);
}
__device__ __forceinline__ int64_t par_block(int nt, int group, int groups)      // in 16 words
{
    return (static_cast<int64_t>(nt >> 2) * groups + group) * 4 + (nt & 3);
}
constexpr int kExpandThreads = 256;


__device__ __forceinline__ void copy16(uint32_t dst, const void* src, int bytes)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}

// Eight bf16 of a row of x from channel k on, from any address; 0 at and past k_end.
__device__ __forceinline__ uint4 load_x8(const uint16_t* row, int k, int k_end)
{
    uint32_t e[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) e[i] = k + i < k_end ? row[k + i] : 0u;
    return make_uint4(e[0] | e[1] << 16, e[2] | e[3] << 16, e[4] | e[5] << 16, e[6] | e[7] << 16);
}

// 128 + c as bf16 pairs: a code is the low bits of the mantissa.  One instruction, with both constants in registers.
__device__ __forceinline__ uint32_t code_pair(uint32_t w, int j, uint32_t mask, uint32_t base)
{
    uint32_t x;
    asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(x) : "r"(w >> (4 * j)), "r"(mask), "r"(base));      // (w & mask) | base
    return x;
}

// D = A B without an accumulator to add to.
__device__ __forceinline__ void mma_first(float* c, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1)
{
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
                 "{%8, %9}, {%10, %10, %10, %10};"
                 : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}

// A stage of a warp's ring in shared memory: codes of NT tiles of columns for one block of k, x of 8 MT rows (each lane copies
// and reads its own 16 bytes of both), and the tiles' parameters.
constexpr int kQ4Stages = 4;
template <int MT> constexpr int kQ4MaxWarps = MT == 1 ? 16 : 8;
template <int NT, int MT, int SUB> struct Q4Stage {
    uint4 w[NT][32], x[MT][2][32];
    uint32_t par[SUB][NT][16];
};
template <int NT, int MT, int SUB> constexpr int kQ4Ring = kQ4Stages * static_cast<int>(sizeof(Q4Stage<NT, MT, SUB>));

// A warp's entries of a block's `cols` columns and `rows` rows of Y whose fp32 sums are not finite (they hold NaN) again, one after
// another, as the sum of x times what the codes stand for in double precision: sums of 128 step x and of step x c (beyond fp32 from
// steps of 2.6e36 or x of 2^112 on) may be infinite where Y is not.  A lane takes the four k of a word.
__device__ __noinline__ void entries_again(const LinearQ4Params& p, int row0, int rows, int n0, int cols)
{
    const int lane = threadIdx.x & 31, t = lane >> 2 & 3, s = lane & 3;
    const int kb_all = (p.k + kQ4K - 1) / kQ4K, groups = (p.k + p.group - 1) / p.group;
    __syncwarp();                                              // the entries are the lanes' stores
    for (int i0 = threadIdx.x & ~31; i0 < rows * cols; i0 += blockDim.x)
        for (int i = i0; i < min(i0 + 32, rows * cols); ++i) {
            const int n = n0 + i % cols, nt = n / kQ4N, c = n % kQ4N, row = row0 + i / cols;
            if (n >= p.n) continue;
            __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.y) + row * p.ld_y + n;
            if (!__hisnan(*out)) continue;
            const uint16_t* x = static_cast<const uint16_t*>(p.x) + row * p.ld_x;
            double y = 0.0;
#pragma unroll 1
            for (int kb = lane >> 4; kb < kb_all; kb += 2) {
                const uint32_t w = reinterpret_cast<const uint32_t*>(p.codes + code_block(nt, kb, kb_all) * 32 + (c & 7) * 4 + t)[s];
                const int k = kb * kQ4K + 32 * (s >> 1) + 8 * t + 4 * (s & 1);
                const uint32_t both = p.par[par_block(nt, min(k / p.group, groups - 1), groups) * 16 + c];
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (k + e < p.k) {
                        const uint32_t code = w >> (4 * ((e & 2) + 4 * (e & 1) + (c >> 3))) & 15u;
                        y += static_cast<double>(mma::bf16_lo(x[k + e])) *
                             fma(static_cast<double>(mma::bf16_lo(both)), static_cast<double>(code), static_cast<double>(mma::bf16_hi(both)));
                    }
            }
#pragma unroll
            for (int d = 16; d; d >>= 1) y += __shfl_xor_sync(0xffffffffu, y, d);
            if (lane == 0) *out = __float2bfloat16_rn(static_cast<float>(y));
        }
}

// A block of threads computes 16 NT columns of Y for 8 MT rows: its warps take turns over the blocks of k, three ahead, and
// their sums meet in shared memory.
// The products see 128 + c; what that adds, 128 step sum x, leaves with the minimum: lo - 128 step times sum x, which an mma
// with a matrix of ones gives in the same lanes.  Both cost 2^-24 of 128 step sum |x| (2^-16 of a step for each x).
// VEC: rows of x start on 16-byte boundaries.
template <int NT, int MT, int SUB, bool VEC>
__global__ void __launch_bounds__(32 * kQ4MaxWarps<MT>) linear_q4_kernel(const __grid_constant__ LinearQ4Params p)
{
    using Stage = Q4Stage<NT, MT, SUB>;
    extern __shared__ __align__(16) char smem[];
    constexpr int kOut = 16 * NT * 8 * MT;
    static_assert((kOut + 16 * NT) * 4 <= kQ4Ring<NT, MT, SUB>, "the sums take the rings' place");
    pdl_wait();
    pdl_launch_dependents();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5, g = lane >> 2, t = lane & 3;
    const int kb_all = (p.k + kQ4K - 1) / kQ4K, groups = (p.k + p.group - 1) / p.group;
    const int nt0 = blockIdx.x * NT;
    const int shift = p.group == 128 ? 1 : 0;
    const int row0 = blockIdx.y * 8 * MT, rows = min(8 * MT, p.m - row0);
    Stage* ring = reinterpret_cast<Stage*>(smem) + warp * kQ4Stages;
    const uint16_t* x[MT];
    int live[MT];                                              // bytes of a copy: none for a row that is not there
#pragma unroll
    for (int a = 0; a < MT; ++a) {
        x[a] = static_cast<const uint16_t*>(p.x) + (row0 + min(8 * a + g, rows - 1)) * p.ld_x + 8 * t;
        live[a] = 8 * a + g < rows ? 16 : 0;
    }
    // what a lane copies: its codes of every tile (NT tiles lie in one block of four), its x, and (the first 4 NT SUB lanes) 16
    // bytes of one tile's parameters
    const uint4* codes = p.codes + code_block(nt0, 0, kb_all) * 32 + lane;
    const int par_tile = lane / 4 % NT, par_sub = lane / (4 * NT);
    const uint32_t* par = p.par + par_block(nt0 + par_tile, 0, groups) * 16 + 4 * t;
    const uint32_t at = smem_u32(ring) + 16 * lane, par_at = smem_u32(&ring[0].par[0][0][0]) + 16 * lane;    // (par: [SUB][NT][16])
    auto load = [&](int kb, int stage) {
        const uint32_t dst = at + stage * static_cast<int>(sizeof(Stage));
#pragma unroll
        for (int b = 0; b < NT; ++b) copy16(dst + 512 * b, codes + kb * 128 + 32 * b, 16);
        const int k = kb * kQ4K;
#pragma unroll
        for (int a = 0; a < MT; ++a)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const uint32_t to = dst + 512 * (NT + 2 * a + h);
                if (VEC && k + kQ4K <= p.k) {
                    copy16(to, x[a] + k + 32 * h, live[a]);
                } else if (VEC) {
                    const int bytes = max(0, min(live[a], 2 * (p.k - (k + 32 * h + 8 * t))));
                    copy16(to, bytes ? x[a] + k + 32 * h : x[a] - 8 * t, bytes);
                } else {
                    ring[stage].x[a][h][lane] = load_x8(x[a], k + 32 * h, p.k - 8 * t);
                }
            }
        if (par_sub < SUB)
            copy16(par_at + stage * static_cast<int>(sizeof(Stage)), par + (SUB == 2 ? min(2 * kb + par_sub, groups - 1) : kb >> shift) * 64, 16);
    };
    float tot[NT][MT][4] = {};
    constexpr uint32_t kOnes = 0x3f803f80u;
    uint32_t mask, base;
    asm volatile("mov.u32 %0, 0x000f000f;" : "=r"(mask));
    asm volatile("mov.u32 %0, 0x43004300;" : "=r"(base));
    auto multiply = [&](const Stage& q) {
        uint4 wv[NT], xv[MT][2];
#pragma unroll
        for (int b = 0; b < NT; ++b) wv[b] = q.w[b][lane];
#pragma unroll
        for (int a = 0; a < MT; ++a) xv[a][0] = q.x[a][0][lane], xv[a][1] = q.x[a][1][lane];
#pragma unroll
        for (int s = 0; s < SUB; ++s) {
            float xs[MT][4], c[NT][MT][4];
#pragma unroll
            for (int i = 0; i < 4 / SUB; ++i) {
                const int step = s * (4 / SUB) + i;
                uint32_t b0[MT], b1[MT];
#pragma unroll
                for (int a = 0; a < MT; ++a) {
                    const uint4 v = xv[a][step >> 1];
                    b0[a] = step & 1 ? v.z : v.x;
                    b1[a] = step & 1 ? v.w : v.y;
                    if (i == 0) mma_first(xs[a], kOnes, kOnes, kOnes, kOnes, b0[a], b1[a]);
                    else mma::mma16816(xs[a], kOnes, kOnes, kOnes, kOnes, b0[a], b1[a]);
                }
#pragma unroll
                for (int b = 0; b < NT; ++b) {
                    const uint32_t w = step == 0 ? wv[b].x : step == 1 ? wv[b].y : step == 2 ? wv[b].z : wv[b].w;
                    const uint32_t a0 = code_pair(w, 0, mask, base), a1 = code_pair(w, 1, mask, base),
                                   a2 = code_pair(w, 2, mask, base), a3 = code_pair(w, 3, mask, base);
#pragma unroll
                    for (int a = 0; a < MT; ++a) {
                        if (i == 0) mma_first(c[b][a], a0, a1, a2, a3, b0[a], b1[a]);
                        else mma::mma16816(c[b][a], a0, a1, a2, a3, b0[a], b1[a]);
                    }
                }
            }
#pragma unroll
            for (int b = 0; b < NT; ++b)
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    const uint32_t both = q.par[s][b][g + 8 * r];
                    const float step = mma::bf16_lo(both), lo = fmaf(-128.f, step, mma::bf16_hi(both));
#pragma unroll
                    for (int a = 0; a < MT; ++a)
#pragma unroll
                        for (int e = 0; e < 2; ++e)
                            tot[b][a][2 * r + e] = fmaf(step, c[b][a][2 * r + e], fmaf(lo, xs[a][e], tot[b][a][2 * r + e]));
                }
        }
    };
#pragma unroll
    for (int i = 0; i < kQ4Stages - 1; ++i) {
        if (warp + i * warps < kb_all) load(warp + i * warps, i);
        mma::cp_async_commit();
    }
    int stage = 0;
    // (rolled up, and with room for 16 warps of 16 rows, the compiler interleaves less: 8 rows by 8192 x 8192 11.5 us, 16 rows 15.9)
#pragma unroll 8
    for (int kb = warp; kb < kb_all; kb += warps) {
        asm volatile("cp.async.wait_group %0;" ::"n"(kQ4Stages - 2) : "memory");
        __syncwarp();                                          // the parameters are other lanes' copies
        const int ahead = kb + (kQ4Stages - 1) * warps;
        if (ahead < kb_all) load(ahead, stage == 0 ? kQ4Stages - 1 : stage - 1);
        mma::cp_async_commit();
        multiply(ring[stage]);
        stage = stage + 1 == kQ4Stages ? 0 : stage + 1;
    }
    __syncthreads();                                           // the rings are read: the sums take their place
    float (*red)[16 * NT][8 * MT + 1] = reinterpret_cast<float (*)[16 * NT][8 * MT + 1]>(smem);
#pragma unroll
    for (int b = 0; b < NT; ++b)
#pragma unroll
        for (int a = 0; a < MT; ++a)
#pragma unroll
            for (int e = 0; e < 4; ++e) red[warp][16 * b + g + 8 * (e >> 1)][8 * a + 2 * t + (e & 1)] = tot[b][a][e];
    __syncthreads();
    bool again = false;
    for (int i = threadIdx.x; i < 16 * NT * rows; i += blockDim.x) {
        const int row = i / (16 * NT), col = i % (16 * NT), n = nt0 * kQ4N + col;
        if (n >= p.n) continue;
        float s = 0.f;
#pragma unroll 4
        for (int w = 0; w < warps; ++w) s += red[w][col][row];
        if (!isfinite(s)) again = true, s = __int_as_float(0x7fc00000);        // (marks the entry)
        static_cast<__nv_bfloat16*>(p.y)[(row0 + row) * p.ld_y + n] = __float2bfloat16_rn(s);
    }
    if (__any_sync(0xffffffffu, again)) entries_again(p, row0, rows, nt0 * kQ4N, 16 * NT);
}

// ---------------------------------------------------------------- weights
constexpr int kWThreads = 128, kWK = 128;

// 16 columns by 128 k of W.  lo: the largest bf16 not above the group's minimum; step: the smallest bf16 not below
// (max - lo) / 15; codes: the nearest integers to (w - lo) / step, ties to even; quotients in double precision.
__global__ void __launch_bounds__(kWThreads) q4_quantise_kernel(const __grid_constant__ Q4WeightParams p)
{
    __shared__ float x[kWK][kQ4N + 1];
    __shared__ float step[4][kQ4N], lo[4][kQ4N];
    pdl_wait();
    pdl_launch_dependents();
    const int tid = threadIdx.x, nt = blockIdx.x, k0 = blockIdx.y * kWK;
    const int kb_all = (p.k + kQ4K - 1) / kQ4K, groups = (p.k + p.group - 1) / p.group;
    for (int i = tid; i < kWK * kQ4N; i += kWThreads) {
        const int k = k0 + i / kQ4N, n = nt * kQ4N + i % kQ4N;
        x[i / kQ4N][i % kQ4N] = k < p.k && n < p.n ? __uint_as_float(static_cast<uint32_t>(static_cast<const uint16_t*>(p.w)[k * p.ld_w + n]) << 16) : 0.f;
    }
    __syncthreads();
    const int here = kWK / p.group;
    for (int i = tid; i < here * kQ4N; i += kWThreads) {
        const int gr = i / kQ4N, c = i % kQ4N, first = gr * p.group, n = min(p.group, p.k - k0 - first);
        if (n <= 0) continue;
        float a = x[first][c], z = a;
        bool bad = false;
        for (int k = 0; k < n; ++k) {
            const float v = x[first + k][c];
            bad |= !isfinite(v);
            a = fminf(a, v);
            z = fmaxf(z, v);
        }
        // (bf16 entries: the minimum is a bf16 already)
        const double span = static_cast<double>(z) - a;
        auto up = [](float v) { return __uint_as_float((__float_as_uint(v) + 0xffffu) & 0xffff0000u); };
        float s = up(static_cast<float>(span / 15.0));
        if (static_cast<double>(s) * 15.0 < span) s = __uint_as_float(__float_as_uint(s) + 0x10000u);
        const float less = s > 0.f ? __uint_as_float(__float_as_uint(s) - 0x10000u) : 0.f;
        if (static_cast<double>(less) * 15.0 >= span) s = less;
        if (bad || !isfinite(s)) s = a = __uint_as_float(0x7fc00000u);
        step[gr][c] = s;
        lo[gr][c] = a;
        p.par[par_block(nt, k0 / p.group + gr, groups) * 16 + c] = __float_as_uint(s) >> 16 | (__float_as_uint(a) & 0xffff0000u);
    }
    __syncthreads();
    for (int i = tid; i < kWK / kQ4K * 128; i += kWThreads) {
        const int kb = i / 128, lane = i % 128 / 4, s = i % 4, g = lane >> 2, t = lane & 3;
        if (k0 / kQ4K + kb >= kb_all) continue;
        uint32_t w = 0;
        for (int j = 0; j < 8; ++j) {
            const int c = g + 8 * (j & 1), k = kb * kQ4K + 32 * (s >> 1) + 8 * t + 4 * (s & 1) + (j & 2) + (j >> 2);
            if (k0 + k >= p.k) continue;
            const float a = lo[k / p.group][c], d = step[k / p.group][c];
            if (!(d > 0.f)) continue;
            // the fp32 quotient is within 2^-19 of the exact one: only near a half does it take more bits to round it
            const float q = (x[k][c] - a) / d, half = fabsf(q - floorf(q) - 0.5f);
            w |= static_cast<uint32_t>(half > 0x1p-17f ? rintf(q) : static_cast<float>(rint((static_cast<double>(x[k][c]) - a) / d))) << (4 * j);
        }
        reinterpret_cast<uint32_t*>(p.codes + code_block(nt, k0 / kQ4K + kb, kb_all) * 32 + lane)[s] = w;
    }
}

// 64 columns by 64 k of W from the codes: one fp32 multiply-add, rounded to bf16.  A thread's word holds four k of columns g and
// g + 8; it trades two of the k with the thread of column g ^ 1, so that pairs of columns go into a row of shared memory
// (33 words a row: the rows of a warp in different banks).  4096 x 4096: 12.4 us (43 MB, 3.4 TB/s; single 16-bit stores into shared
// memory took 18.0).
__global__ void __launch_bounds__(kExpandThreads) q4_expand_kernel(const __grid_constant__ Q4WeightParams p)
{
    __shared__ uint32_t x[kQ4K][33];
    pdl_wait();
    pdl_launch_dependents();
    const int tid = threadIdx.x, kb = blockIdx.y, n0 = blockIdx.x * 64;
    const int kb_all = (p.k + kQ4K - 1) / kQ4K, groups = (p.k + p.group - 1) / p.group;
#pragma unroll
    for (int i = tid; i < 4 * 128; i += kExpandThreads) {
        const int nt = n0 / kQ4N + i / 128, lane = i % 128 / 4, s = i % 4, g = lane >> 2, t = lane & 3;
        const uint32_t w = reinterpret_cast<const uint32_t*>(p.codes + code_block(nt, kb, kb_all) * 32 + lane)[s];
        const int k = 32 * (s >> 1) + 8 * t + 4 * (s & 1), gr = min((kb * kQ4K + k) / p.group, groups - 1);
        const uint32_t* q = p.par + par_block(nt, gr, groups) * 16 + g;
        const uint32_t par[2] = {q[0], q[8]};
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            const float step = mma::bf16_lo(par[c]), lo = mma::bf16_hi(par[c]);
            // a code as the low bits of 2^23 + c
            auto value = [&](int j) { return fmaf(step, __uint_as_float((w >> (4 * j) & 15u) | 0x4B000000u) - 8388608.f, lo); };
            const uint32_t front = mma::pack2(value(c), value(4 + c)), back = mma::pack2(value(2 + c), value(6 + c));
            const uint32_t other = __shfl_xor_sync(0xffffffffu, g & 1 ? front : back, 16);
            const uint32_t left = g & 1 ? other : front, right = g & 1 ? back : other;      // columns g & ~1, g | 1
            uint32_t* row = &x[k + 2 * (g & 1)][(i / 128 * kQ4N + (g & 6) + 8 * c) / 2];
            row[0] = __byte_perm(left, right, 0x5410);
            row[33] = __byte_perm(left, right, 0x7632);
        }
    }
    __syncthreads();
    // eight columns a store where rows start on 16-byte boundaries
    const bool vec = (reinterpret_cast<uintptr_t>(p.w) | static_cast<uintptr_t>(2 * p.ld_w)) % 16 == 0;
    for (int i = tid; i < kQ4K * 8; i += kExpandThreads) {
        const int k = kb * kQ4K + i / 8, n = n0 + i % 8 * 8;
        if (k >= p.k || n >= p.n) continue;
        uint16_t* row = static_cast<uint16_t*>(p.w) + static_cast<int64_t>(k) * p.ld_w + n;
        const uint32_t* from = &x[i / 8][i % 8 * 4];
        if (vec && n + 8 <= p.n) *reinterpret_cast<uint4*>(row) = make_uint4(from[0], from[1], from[2], from[3]);
        else
            for (int e = 0; e < min(8, p.n - n); ++e) row[e] = static_cast<uint16_t>(from[e >> 1] >> (16 * (e & 1)));
    }
}

template <int NT, int MT, int SUB, bool VEC>
cudaError_t launch_variant(const LinearQ4Params& p, int warps, cudaStream_t s)
{
    static OncePerDevice once;
    constexpr int most = 226 * 1024 / kQ4Ring<NT, MT, SUB> < kQ4MaxWarps<MT> ? 226 * 1024 / kQ4Ring<NT, MT, SUB> : kQ4MaxWarps<MT>;
    warps = min(warps, most);
    const cudaError_t e = allow_smem(once, most * kQ4Ring<NT, MT, SUB>, linear_q4_kernel<NT, MT, SUB, VEC>);
    if (e != cudaSuccess) return e;
    const dim3 grid((p.n + kQ4N * NT - 1) / (kQ4N * NT), (p.m + 8 * MT - 1) / (8 * MT));
    return launch_dependent(linear_q4_kernel<NT, MT, SUB, VEC>, grid, dim3(32 * warps), warps * kQ4Ring<NT, MT, SUB>, s, p);
}

template <int NT, int MT>
cudaError_t launch_rows(const LinearQ4Params& p, int warps, cudaStream_t s)
{
    if (p.group == 32)
        return p.vec_x ? launch_variant<NT, MT, 2, true>(p, warps, s) : launch_variant<NT, MT, 2, false>(p, warps, s);
    return p.vec_x ? launch_variant<NT, MT, 1, true>(p, warps, s) : launch_variant<NT, MT, 1, false>(p, warps, s);
}

}  // namespace

cudaError_t launch_linear_q4(const LinearQ4Params& p, int sm_count, cudaStream_t s)
{
    // Tiles of columns a block: more share x and its sums, as long as most SMs get a block (us with 1, 2, 4 tiles, when this was
    // measured: n = 8192, k = 8192: 18.3, 14.5, 13.2; n = 4096, k = 1024: 2.44, 2.18, 2.73; n = 1024, k = 1024: 1.79, 1.91, 2.66).
    // Warps: a few blocks of k each (8 and 16 warps: k = 1024 1.79 and 1.89, k = 4096, n = 1024 3.82 and 3.43).  Rows: 8, or 16 at
    // once where there are more than 8 (the same codes serve both).
    // 16 rows, 8 warps: k = n = 8192 25.4, 18.6, 14.7; 4096 8.5, 6.7, 8.5; 64 rows by 4096 x 4096 23.8, 18.5, 16.2.
    const int kb = (p.k + kQ4K - 1) / kQ4K, at_once = p.m <= 8 ? 8 : 16;
    const int64_t blocks = static_cast<int64_t>((p.n + kQ4N - 1) / kQ4N) * ((p.m + at_once - 1) / at_once);
    const int nt = blocks >= 3 * sm_count ? 4 : blocks >= 3 * sm_count / 2 ? 2 : 1, warps = kb >= 48 && p.m <= 8 ? 16 : 8;
    if (p.m <= 8) return nt == 4 ? launch_rows<4, 1>(p, warps, s) : nt == 2 ? launch_rows<2, 1>(p, warps, s) : launch_rows<1, 1>(p, warps, s);
    return nt == 4 ? launch_rows<4, 2>(p, warps, s) : nt == 2 ? launch_rows<2, 2>(p, warps, s) : launch_rows<1, 2>(p, warps, s);
}

cudaError_t launch_q4_quantise(const Q4WeightParams& p, cudaStream_t s)
{
    // (tiles past n fill the last block of four)
    return launch_dependent(q4_quantise_kernel, dim3((p.n + 63) / 64 * 4, (p.k + kWK - 1) / kWK), dim3(kWThreads), 0, s, p);
}

cudaError_t launch_q4_expand(const Q4WeightParams& p, cudaStream_t s)
{
    return launch_dependent(q4_expand_kernel, dim3((p.n + 63) / 64, (p.k + kQ4K - 1) / kQ4K), dim3(kExpandThreads), 0, s, p);
}

}  // namespace txl
