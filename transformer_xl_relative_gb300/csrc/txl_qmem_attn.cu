// txl_qmem_attn.cu -- relative attention of 1 .. 16 queries over a quantised memory and the segment's
// own keys: the generation step over a memory of 4- or 8-bit codes, in one launch.
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
// Precision: q+u is held as two fp16 parts (scaled by a power of two per row; 22 bits) in two columns
// of the B operand, p step likewise; the accumulators are fp32.  The eight columns of an MMA are four
// slots x (hi, lo).  A slot is a query; with fewer than three queries the other slots take other tiles
// of 16 keys ("streams"), so that the work per key after the first product (scale, softmax, splitting
// p) falls on all 32 lanes whatever L is.  With one query the four k-quarters of a Q.K MMA belong to the
// four streams (each lane holds whole rows of its own two keys, B is block diagonal); with two queries
// B is masked to the tile's own slots.
//
// The position term: the keys of a block (one stage of every warp) and the queries meet at consecutive
// distances, so e(i, rho) = (q_i+v).r is a band computed once per block, on the tensor cores too (bf16
// r rows, q+v as two bf16 parts), for up to eight (batch entry, query) rows at once: a CTA covers NB
// batch entries, which share every r row.  The band of the next block is computed between the steps of
// this one, so that its loads of r fly while the codes are multiplied.  Distances at or past the clamp
// share one entry.
//
// One CTA: NB batch entries x one head x a range of keys; 8 / NB warps per entry, each with its own
// ring of bulk-copy stages (cp.async, 16 bytes per lane, held the issuing warp for 2400 to 4000 cycles
// per stage until its requests were accepted).  The key ranges of a head are the ranks of a cluster:
// each writes its partial results into the shared memory of the rank that finishes the row.
#include <algorithm>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "txl_internal.h"
#include "txl_mma.cuh"
#include "txl_ptx.cuh"

namespace txl {

namespace {

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kStages = 2;
constexpr int kMaxRanks = 16;                  // CTAs of a cluster (beyond 8: not portable, but this GPU's)
constexpr int kMaxRows = 8;                    // (batch entry, query) rows of a CTA
constexpr int kBandPad = 40;                   // floats after a row's keys: up to 22 more entries; rows 8 banks apart
constexpr float kNoMax = -3e38f;               // running maximum before any key
constexpr float kTwo24 = 16777216.f;
constexpr float kMinUnit = 3.00926553e-36f;    // 2^-118 and 2^126: bounds of the weights' unit, so that a weight
constexpr float kMaxUnit = 8.50705917e37f;     // (at most 2^8) over the unit stays finite

// Keys of a stage: 64 where a key's codes are small and the queries few, else 32.
__host__ __device__ constexpr int stage_keys(int bits, int ng, int qt) { return bits * ng <= 8 && qt == 1 ? 64 : 32; }
__host__ __device__ constexpr int stage_bytes(int bits, int ng, int qt)
{
    return stage_keys(bits, ng, qt) * (8 * ng * bits + 8 * ng);
}
// Floats of a position band: a row per (batch entry, query), as many keys as a stage of every warp of one
// entry; rows <= 8 / entries * queries, so entries * queries rows of 8 / entries stages.
__host__ __device__ constexpr int band_floats(int bits, int ng, int qt)
{
    return (qt == 1 ? 4 : 8) * kWarps * stage_keys(bits, ng, qt) + kMaxRows * kBandPad;
}

struct QSplit {               // how the host divides the work
    int nb;                   // batch entries of a CTA (1, 2, 4, 8)
    int lq;                   // queries of a CTA; blockIdx.x / ranks selects the group of queries
    int ranks;                // CTAs of a cluster: key ranges
    int range;                // keys of a range (a multiple of the stage)
};

__device__ __forceinline__ float ld_elem(const void* p, int64_t i, int f32)
{
    return f32 ? __ldg(static_cast<const float*>(p) + i)
               : __uint_as_float(static_cast<uint32_t>(__ldg(static_cast<const uint16_t*>(p) + i)) << 16);
}

// D += A B: m16n8k16, fp16 operands, fp32 accumulators
__device__ __forceinline__ void mma_f16(float* c, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1)
{
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
                 "{%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// 8 x 8 transpose of 16-bit elements across a warp
__device__ __forceinline__ uint32_t transpose8(uint32_t x)
{
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

__device__ __forceinline__ void prefetch_l2(const void* p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }

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

// Pairs of codes of a register as fp16 subnormals; odd = the second pair of a 16-bit half (16 times as
// large at 4 bits).  `half` selects the upper byte (4 bits).
template <int BITS>
__device__ __forceinline__ uint32_t pair_even(uint32_t w) { return w & (BITS == 4 ? 0x000f000fu : 0x00ff00ffu); }
template <int BITS>
__device__ __forceinline__ uint32_t pair_odd(uint32_t w) { return BITS == 4 ? w & 0x00f000f0u : (w >> 8) & 0x00ff00ffu; }

template <int BITS, int NG, int QT, bool ONE>
__global__ void __launch_bounds__(kThreads, NG == 2 || (BITS == 4 && QT == 1) ? 2 : 1)
qattn_kernel(const __grid_constant__ QattnParams p, const __grid_constant__ QSplit sp)
{
    constexpr int DP = NG * 32;                           // channels, padded
    constexpr int NC = NG * BITS / 4;                     // 16-byte chunks of a code row
    constexpr int KS = stage_keys(BITS, NG, QT);
    constexpr int kVOff = KS * NC * 16, kParOff = 2 * kVOff;   // of a stage: k rows, v rows, parameters
    constexpr int kStageBytes = stage_bytes(BITS, NG, QT);
    constexpr int kBand = band_floats(BITS, NG, QT);
    constexpr int SUB = BITS == 4 ? 2 : 1;                // MMAs per register of codes and product
    constexpr int kOwn = ONE ? 1 : kDecodeMaxL;           // keys of the segment a query can see
    constexpr int kTileRegs = NG == 2 && QT == 1 ? 2 : 1; // band tiles in flight at a time
    extern __shared__ __align__(128) uint8_t smem[];
    uint8_t* stages = smem;
    float* bands = reinterpret_cast<float*>(smem + kWarps * kStages * kStageBytes);   // two
    float* qu = bands + 2 * kBand;                        // [row][DP]: (q+u) and (q+v) in log2 units
    float* qv = qu + kMaxRows * DP;
    float* inbox = qu;                                    // later [row of this rank][rank][DP + 2]: O, m, l
    float* norm = qu + kMaxRanks * (DP + 4);              // [row]: what the fp16 parts of qu are multiples of
    float* qsum = norm + kMaxRows;                        // [row][NG]: group sums of qu
    float* far = qsum + kMaxRows * NG;                    // [row]: the position term of distances at the clamp
    float* own_s = far + kMaxRows;                        // [row][kDecodeMaxL]: scores of the segment's own keys
    uint16_t* quh = reinterpret_cast<uint16_t*>(own_s + kMaxRows * kDecodeMaxL);   // [2 row + part][DP] fp16 parts of qu
    uint16_t* qvh = quh + (2 * kMaxRows + 1) * DP;        // (a row of zeros between) [2 row + part][DP] bf16 parts of qv
    uint64_t* bars = reinterpret_cast<uint64_t*>(qvh + 2 * kMaxRows * DP);   // [warp][stage]: copies landed
    int* abort_flag = reinterpret_cast<int*>(bars + kWarps * kStages);

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, c4 = lane & 3;
    const int rank = blockIdx.x % sp.ranks, i0 = blockIdx.x / sp.ranks * sp.lq;
    const int h = blockIdx.y, b0 = blockIdx.z * sp.nb;
    const int Lq = min(sp.lq, p.L - i0), rows = sp.nb * Lq;
    const int wpe = kWarps / sp.nb, bs = warp / wpe, sw = warp % wpe;          // this warp's batch entry and part
    const int b = b0 + bs;
    // slots of an MMA's columns: slot = stream * Lp + query
    const int lp_log = ONE ? 0 : Lq >= 3 ? 2 : Lq - 1, Lp = 1 << lp_log;
    const int NS = ONE ? KS / 16 : QT > 1 ? 1 : min(4 >> lp_log, KS / 16);
    pdl_launch_dependents();
    if (tid == 0) *abort_flag = 0;
    const WaitCtl wc{abort_flag, p.err_flag, kWaitTimeoutNs};
    pdl_wait();

    const int j_lo = static_cast<int>(min(static_cast<int64_t>(p.M), p.lo + static_cast<int64_t>(rank) * sp.range));
    const int j_hi = static_cast<int>(min(static_cast<int64_t>(p.M), static_cast<int64_t>(j_lo) + sp.range));

    // ---- requested before the copies below fill the memory system: the queries' elements, the lines of the
    // segment's own keys, values and position rows (into L2), the first rows of r
    const bool has_own = rank == sp.ranks - 1;            // the last rank's work
    const int n_own = i0 + Lq;                            // own keys any of these queries sees
    if (has_own) {
        const int row_of_f32 = p.f32 ? 4 : 2;
        for (int x = tid; x < sp.nb * n_own; x += kThreads) {
            const int be = min(b0 + x / n_own, p.B - 1), j = x % n_own;
            prefetch_l2(static_cast<const char*>(p.kcur) + (be * p.kc_sb + j * p.kc_st + h * p.kc_sh) * row_of_f32);
            prefetch_l2(static_cast<const char*>(p.vcur) + (be * p.vc_sb + j * p.vc_st + h * p.vc_sh) * row_of_f32);
            if (x < n_own)
                prefetch_l2(static_cast<const char*>(p.r) + (min(x, p.C) * p.r_row + h * p.r_head) * row_of_f32);
        }
    }
    const int my_be = b0 + warp / Lq, my_i = i0 + warp % Lq;
    const bool my_row = warp < rows && my_be < p.B;
    float q_raw[NG], u_raw[NG], vb_raw[NG], rc_raw[NG];
    const bool any_far = static_cast<int64_t>(p.M) + i0 + Lq - 1 - j_lo >= p.C;    // then row C exists
#pragma unroll
    for (int e = 0; e < NG; ++e) {
        const int d = 32 * e + lane;
        const bool on = my_row && d < p.D;
        q_raw[e] = on ? ld_elem(p.q, my_be * p.q_sb + my_i * p.q_st + h * p.q_sh + d, p.f32) : 0.f;
        u_raw[e] = on ? __ldg(p.u + h * p.D + d) : 0.f;
        vb_raw[e] = on ? __ldg(p.vb + h * p.D + d) : 0.f;
        rc_raw[e] = on && any_far ? ld_elem(p.r, p.C * p.r_row + h * p.r_head + d, p.f32) : 0.f;
    }

    // ---- position band of block k, keys jb = j_lo + k wpe KS ..: entry rho of row (entry, query i) is distance
    // top - rho, and meets key j at rho = Lq - 1 - i + j - jb; entries up to rho = top - C are at the clamp and
    // are not computed (one value per row serves them all; a band of such entries alone needs no barrier)
    const int block = wpe * KS, pitch = block + kBandPad;
    const int n_block = (j_hi - j_lo + block - 1) / block;
    struct Band { int jb, top, n_rho, first; };           // first: the first tile of 16 entries short of the clamp
    auto band_of = [&](int k) {
        Band x;
        x.jb = j_lo + k * block;
        x.top = p.M + i0 + Lq - 1 - x.jb;
        x.n_rho = k < n_block ? min(block, j_hi - x.jb) + Lq - 1 : 0;
        x.first = max(0, x.top - p.C + 1) >> 4;
        return x;
    };
    auto r_row = [&](const Band& x, int rho) {
        int rr = max(0, min(x.top - rho, p.C));
        if (!in_range(rr, 0, p.n_rows, p.chk)) rr = 0;
        return rr * p.r_row + h * p.r_head;
    };
    uint4 ra[kTileRegs][2][NG];
    auto band_load = [&](const Band& x, int tile) {       // rows of r of kTileRegs tiles
#pragma unroll
        for (int y = 0; y < 2 * kTileRegs; ++y) {
            const uint16_t* src = static_cast<const uint16_t*>(p.r) + r_row(x, tile * 16 + g + 8 * y);
#pragma unroll
            for (int G = 0; G < NG; ++G) {
                const int d = 32 * G + 8 * c4;
                if (p.vec_r && d + 8 <= p.D) {
                    ra[y >> 1][y & 1][G] = __ldg(reinterpret_cast<const uint4*>(src + d));
                } else {
                    uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        if (d + e < p.D) w[e >> 1] |= static_cast<uint32_t>(__ldg(src + d + e)) << (16 * (e & 1));
                    ra[y >> 1][y & 1][G] = make_uint4(w[0], w[1], w[2], w[3]);
                }
            }
        }
    };
    Band cur = band_of(0);
    if (!p.f32 && (cur.first + kTileRegs * warp) * 16 < cur.n_rho) band_load(cur, cur.first + kTileRegs * warp);

    // ---- this warp's copies: stage n covers keys j_lo + (n * wpe + sw) * KS ..; rows as they are in memory,
    // one bulk copy each for the k codes, the v codes and the parameters, two where the ring wraps
    uint8_t* my_stages = stages + warp * kStages * kStageBytes;
    uint64_t* full = bars + warp * kStages;
    const int n_stage = b < p.B ? max(0, (j_hi - j_lo - sw * KS + wpe * KS - 1) / (wpe * KS)) : 0;
    const int nc = p.G * BITS / 4, row_bytes = nc * 16;
    const int64_t head_row = (static_cast<int64_t>(b) * p.H + h) * p.M;
    auto slot_of = [&](int j) {                           // of a logical key
        const int64_t s = static_cast<int64_t>(p.wp) + j;
        return static_cast<int>(s >= p.M ? s - p.M : s);
    };
    auto copy_rows = [&](uint8_t* st, uint64_t* bar, int at, int slot, int count) {
        const int64_t row = head_row + slot;
        bulk_load(st + at * row_bytes, p.k + row * row_bytes, count * row_bytes, bar);
        bulk_load(st + kVOff + at * row_bytes, p.v + row * row_bytes, count * row_bytes, bar);
        bulk_load(st + kParOff + at * 8 * NG, p.par + row * NG * 4, count * 8 * NG, bar);
    };
    auto copy_stage = [&](int n) {                        // one lane
        uint8_t* st = my_stages + (n % kStages) * kStageBytes;
        uint64_t* bar = &full[n % kStages];
        const int j = j_lo + (n * wpe + sw) * KS;
        const int live = min(KS, j_hi - j);
        int slot = slot_of(j);
        if (!in_range(slot, 0, p.M, p.chk)) slot = 0;
        mbar_expect_tx(bar, live * (2 * row_bytes + 8 * NG));
        const int first = min(live, p.M - slot);
        copy_rows(st, bar, 0, slot, first);
        if (first < live) copy_rows(st, bar, first, 0, live - first);
    };
    if (lane == 0) {
#pragma unroll
        for (int n = 0; n < kStages; ++n) mbar_init(&full[n], 1);
        fence_mbar_init();
#pragma unroll
        for (int n = 0; n < kStages; ++n)
            if (n < n_stage) copy_stage(n);
    }

    // ---- queries: warp w prepares row w: (q+u), (q+v) times scale log2 e in fp32; (q+u) scaled by a power
    // of two so that its largest entry lies in [2^11, 2^12) as two fp16 parts, in the order in which the
    // B operands take them (4 bits: d = 0 4 1 5 2 6 3 7 of every eight, odd ones over 16; 8 bits: 0 2 1 3
    // of every four); (q+v) as two bf16 parts.  Rows past the last query are zero.
    {
        const int row = warp;
        float a[NG], mx = 0.f, at_clamp = 0.f;
#pragma unroll
        for (int e = 0; e < NG; ++e) {
            a[e] = (q_raw[e] + u_raw[e]) * p.qscale;
            at_clamp = fmaf((q_raw[e] + vb_raw[e]) * p.qscale, rc_raw[e], at_clamp);
            mx = fmaxf(mx, fabsf(a[e]));
        }
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) {
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
            at_clamp += __shfl_xor_sync(0xffffffffu, at_clamp, off);
        }
        if (lane == 0) far[row] = at_clamp;
        const int ex = max(static_cast<int>(__float_as_uint(mx) >> 23) - 127, -100);
        const float up = __uint_as_float(static_cast<uint32_t>(11 - ex + 127) << 23);
        if (lane == 0) norm[row] = __uint_as_float(static_cast<uint32_t>(ex - 11 + 127) << 23);
#pragma unroll
        for (int e = 0; e < NG; ++e) {
            const int d = 32 * e + lane;
            const float c = (q_raw[e] + vb_raw[e]) * p.qscale;
            qu[row * DP + d] = a[e];
            qv[row * DP + d] = c;
            const int at = BITS == 4 ? (d & ~7) + ((d & 3) << 1) + ((d >> 2) & 1) : (d & ~3) + ((d & 1) << 1) + ((d >> 1) & 1);
            uint32_t w, unused;
            split_f16(a[e] * (BITS == 4 && (d & 1) ? up * 0.0625f : up), 0.f, w, unused);
            quh[2 * row * DP + at] = static_cast<uint16_t>(w);
            quh[(2 * row + 1) * DP + at] = static_cast<uint16_t>(w >> 16);
            if (row == 0) quh[2 * kMaxRows * DP + d] = 0;
            const __nv_bfloat16 hi = __float2bfloat16_rn(c);
            qvh[2 * row * DP + d] = __bfloat16_as_ushort(hi);
            qvh[(2 * row + 1) * DP + d] = __bfloat16_as_ushort(__float2bfloat16_rn(c - __bfloat162float(hi)));
            float sum = a[e];
#pragma unroll
            for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
            if (lane == 0) qsum[row * NG + e] = sum;
        }
    }
    __syncthreads();

    // ---- B operands of Q.K, column g = (slot g/2, part g%2), and per slot c4 the group sums of q.  ONE: the
    // k-quarter of this lane belongs to stream c4, so only columns of slot c4 are not zero there.
    uint32_t bq[QT][NG * 2][2];
    float qs[QT][NG], sc[QT], far_of[QT];
    const int my_stream = (g >> 1) >> lp_log;             // of the column this lane holds in B operands
    const uint16_t* one_row = quh + ((g >> 1) == c4 ? 2 * bs + (g & 1) : 2 * kMaxRows) * DP;
#pragma unroll
    for (int t = 0; t < QT; ++t) {
        if constexpr (!ONE) {
            const int il = min(((g >> 1) & (Lp - 1)) + 4 * t, Lq - 1);
            const uint16_t* row = quh + (2 * (bs * Lq + il) + (g & 1)) * DP;
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
        const int is = bs * Lq + min((c4 & (Lp - 1)) + 4 * t, Lq - 1);
        sc[t] = norm[is] * kTwo24;
        far_of[t] = far[is];
#pragma unroll
        for (int G = 0; G < NG; ++G) qs[t][G] = qsum[is * NG + G];
    }

    // ---- scores of the segment's own keys: eight lanes per (row, key)
    if (has_own) {
        for (int x0 = warp * 4; x0 < rows * n_own; x0 += kWarps * 4) {
            const int x = min(x0 + (lane >> 3), rows * n_own - 1);
            const int row = x / n_own, j = x % n_own, be = b0 + row / Lq, i = i0 + row % Lq;
            const bool on = be < p.B && j <= i;
            int rr = on ? min(i - j, p.C) : 0;
            if (!in_range(rr, 0, p.n_rows, p.chk)) rr = 0;
            float s = 0.f;
#pragma unroll 4
            for (int e = 0; e < DP / 8; ++e) {
                const int d = (lane & 7) + 8 * e;
                if (on && d < p.D) {
                    const float k = ld_elem(p.kcur, be * p.kc_sb + j * p.kc_st + h * p.kc_sh + d, p.f32);
                    const float r = ld_elem(p.r, rr * p.r_row + h * p.r_head + d, p.f32);
                    s = fmaf(qu[row * DP + d], k, fmaf(qv[row * DP + d], r, s));
                }
            }
#pragma unroll
            for (int off = 4; off > 0; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
            if ((lane & 7) == 0) own_s[row * kOwn + j] = on ? s : -INFINITY;
        }
    }

    auto has_tiles = [&](const Band& x) { return x.first * 16 < x.n_rho; };
    const int n_ct = (rows + 3) >> 2;
    auto band_store = [&](const Band& x, int tile, float* band) {
        for (int ct = 0; ct < n_ct; ++ct) {
            uint4 bw[NG];
#pragma unroll
            for (int G = 0; G < NG; ++G) bw[G] = *reinterpret_cast<const uint4*>(qvh + (8 * ct + g) * DP + 32 * G + 8 * c4);
#pragma unroll
            for (int y = 0; y < kTileRegs; ++y) {
                float acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int G = 0; G < NG; ++G) {
                    mma::mma16816(acc, ra[y][0][G].x, ra[y][1][G].x, ra[y][0][G].y, ra[y][1][G].y, bw[G].x, bw[G].y);
                    mma::mma16816(acc, ra[y][0][G].z, ra[y][1][G].z, ra[y][0][G].w, ra[y][1][G].w, bw[G].z, bw[G].w);
                }
                if (4 * ct + c4 < rows && (tile + y) * 16 < x.n_rho) {
                    float* e = band + (4 * ct + c4) * pitch + (tile + y) * 16 + g;
                    e[0] = acc[0] + acc[1];
                    e[8] = acc[2] + acc[3];
                }
            }
        }
    };
    auto band_f32 = [&](const Band& x, float* band) {
        for (int y = tid; y < rows * x.n_rho; y += kThreads) {
            const int row = y / x.n_rho, rho = y % x.n_rho;
            if (rho <= x.top - p.C) continue;
            const float* src = static_cast<const float*>(p.r) + r_row(x, rho);
            float s = 0.f;
            for (int d = 0; d < p.D; ++d) s = fmaf(qv[row * DP + d], __ldg(src + d), s);
            band[row * pitch + rho] = s;
        }
    };
    if (p.f32) {
        band_f32(cur, bands);
    } else {
        for (int t = cur.first + kTileRegs * warp; t * 16 < cur.n_rho; t += kTileRegs * kWarps) {
            if (t != cur.first + kTileRegs * warp) band_load(cur, t);
            band_store(cur, t, bands);
        }
    }
    __syncthreads();
    // the other ranks' partial results may come (waited for before the first is written) where qu and qv are
    // no longer read
    if (sp.ranks > 1 && !p.f32) cluster_arrive();

    // ---- running state of slot c4: maximum, weight unit rf (O is in units of rf), sums
    float o[QT][NG * 2][4], z[QT][NG], m[QT], l[QT], rf[QT];
#pragma unroll
    for (int t = 0; t < QT; ++t) {
        m[t] = kNoMax;
        l[t] = 0.f;
        rf[t] = kMinUnit;
#pragma unroll
        for (int G = 0; G < NG; ++G) z[t][G] = 0.f;
#pragma unroll
        for (int x = 0; x < NG * 2; ++x) o[t][x][0] = o[t][x][1] = o[t][x][2] = o[t][x][3] = 0.f;
    }

    bool ok = true;
    for (int n = 0; n < n_block; ++n) {
        const float* band = bands + (n & 1) * kBand;
        float* next_band = bands + ((n & 1) ^ 1) * kBand;
        const Band next = band_of(n + 1);
        int tile = next.first + kTileRegs * warp;         // this warp's tiles of the next band
        const bool live_stage = n < n_stage && ok && warp_wait(&full[n % kStages], (n / kStages) & 1, wc, 50);
        if (n < n_stage && !live_stage) ok = false;       // a copy that did not come: no result is valid
        bool loaded = !p.f32 && tile * 16 < next.n_rho;
        if (loaded) band_load(next, tile);
        if (live_stage) {
            const int js = j_lo + (n * wpe + sw) * KS;
            const uint8_t* st = my_stages + (n % kStages) * kStageBytes;
            const uint32_t st_addr = smem_u32(st);
            const int slot0 = slot_of(js);
            // permutation of the chunks of the stage's row r: that of its slot, which repeats every eight rows
            // unless the ring wraps within the stage
            const bool wraps = slot0 + KS > p.M;
            auto swap_of = [&](int r) {
                int s = slot0 + r;
                if (wraps && s >= p.M) s -= p.M;
                return q_swizzle(nc, s);
            };
            const int swap_lane = q_swizzle(nc, slot0 + (lane & 15)), swap_key = q_swizzle(nc, slot0 + g);
            const bool whole = js + KS <= j_hi;           // no row past the end
            for (int k0 = 0; k0 < (ONE ? 1 : KS); k0 += 16 * NS) {
                if (js + k0 >= j_hi) break;
                // Q.K: acc[t][G] = for slot c4, keys g and g+8 of its stream's tile, (hi, lo) parts.  ONE: in the
                // place of group G that of group G ^ gx, gx chosen so that the lanes' rows meet in no bank
                float acc[QT][NG][4];
#pragma unroll
                for (int t = 0; t < QT; ++t)
#pragma unroll
                    for (int G = 0; G < NG; ++G) acc[t][G][0] = acc[t][G][1] = acc[t][G][2] = acc[t][G][3] = 0.f;
                constexpr int CPG = BITS / 4;             // chunks of a group
                const int cx = NC == 2 ? c4 & 1 : NC == 4 ? c4 : 2 * c4;       // chunk c ^ cx in the place of chunk c
                const int gx = cx / CPG;
                if constexpr (ONE) {
                    // this lane's rows: keys g and g+8 of tile c4 (of the tiles there are)
                    const int r0 = 16 * min(c4, KS / 16 - 1) + g;
                    const uint32_t row0 = st_addr + r0 * row_bytes, row1 = row0 + 8 * row_bytes;
                    const uint32_t sw0 = wraps ? swap_of(r0) : swap_key, sw1 = wraps ? swap_of(r0 + 8) : swap_key;
#pragma unroll
                    for (int c = 0; c < NC; ++c) {
                        const uint32_t cc = c ^ cx;
                        uint32_t wa[4], wb[4];
                        lds128(row0 + ((cc ^ sw0) << 4), wa);
                        lds128(row1 + ((cc ^ sw1) << 4), wb);
                        const uint16_t* bsrc = one_row + cc * (128 / BITS);
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
                                mma_f16(acc[0][c / CPG], pair_even<BITS>(x), pair_even<BITS>(y), pair_odd<BITS>(x),
                                        pair_odd<BITS>(y), bb[2 * s], bb[2 * s + 1]);
                            }
                        }
                    }
                } else {
                    for (int T = 0; T < NS; ++T) {
                        const bool on = QT > 1 || my_stream == T;
                        const int r = k0 + 16 * T + (lane & 15);
                        const uint32_t row = st_addr + r * row_bytes, swap = wraps ? swap_of(r) : swap_lane;
#pragma unroll
                        for (int c2 = 0; c2 < NC; c2 += 2) {
                            uint32_t w[4];
                            mma::ldsm_x4(row + (((c2 + (lane >> 4)) ^ swap) << 4), w[0], w[1], w[2], w[3]);
#pragma unroll
                            for (int half = 0; half < 2; ++half) {
                                const int c = c2 + half;
#pragma unroll
                                for (int s = 0; s < SUB; ++s) {
                                    const uint32_t x = w[2 * half] >> (8 * s), y = w[2 * half + 1] >> (8 * s);
                                    const int ks = c * SUB + s;
#pragma unroll
                                    for (int t = 0; t < QT; ++t)
                                        mma_f16(acc[t][c / CPG], pair_even<BITS>(x), pair_even<BITS>(y), pair_odd<BITS>(x),
                                                pair_odd<BITS>(y), on ? bq[t][ks][0] : 0u, on ? bq[t][ks][1] : 0u);
                                }
                            }
                        }
                    }
                }
                // scores, weights, and the P operands: two keys per lane
                const int kk = k0 + 16 * (c4 >> lp_log) + g;          // key of the stage (and kk + 8)
                const bool in_use = (c4 >> lp_log) < NS;              // slots past the streams hold no keys
                uint2 par[2][NG];
                float kstep[2][NG];
                bool live[2] = {true, true};
                const uint8_t* par_row = st + kParOff + (in_use ? kk : g) * 8 * NG;
#pragma unroll
                for (int x = 0; x < 2; ++x)
#pragma unroll
                    for (int G = 0; G < NG; ++G) {
                        par[x][G] = *reinterpret_cast<const uint2*>(par_row + 64 * NG * x + 8 * G);
                        kstep[x][G] = __uint_as_float(
                            (ONE ? *reinterpret_cast<const uint32_t*>(par_row + 64 * NG * x + 8 * (G ^ gx)) : par[x][G].x) << 16);
                    }
                if (!whole || NS << lp_log < 4) {                     // rows past the end hold what was there before
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        live[x] = in_use && js + kk + 8 * x < j_hi;
#pragma unroll
                        for (int G = 0; G < NG; ++G)
                            if (!live[x]) {
                                par[x][G] = make_uint2(0, 0);
                                kstep[x][G] = 0.f;
                            }
                    }
                }
                const int rho0 = Lq - 1 + js + kk - cur.jb;           // band entry of key g of query 0
                const int rho_far = cur.top - p.C;                    // entries up to this one are at the clamp
                uint32_t bp[QT][NG][2];
#pragma unroll
                for (int t = 0; t < QT; ++t) {
                    const int il = ONE ? 0 : min((c4 & (Lp - 1)) + 4 * t, Lq - 1);
                    const float* e = band + (bs * Lq + il) * pitch;
                    float s[2], pr[2], w[2][NG];
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        const int rho = rho0 - il + 8 * x;
                        float a = rho > rho_far ? e[rho] : far_of[t], d = 0.f;
#pragma unroll
                        for (int G = 0; G < NG; ++G) {
                            d = fmaf(acc[t][G][2 * x] + acc[t][G][2 * x + 1], kstep[x][G], d);
                            a = fmaf(__uint_as_float(par[x][G].x & 0xffff0000u), qs[t][G], a);
                        }
                        s[x] = live[x] ? fmaf(d, sc[t], a) : -INFINITY;
                        pr[x] = ex2_approx(s[x] - m[t]);
                    }
                    const float f = __uint_as_float(0x7f000000u - __float_as_uint(rf[t]));   // 1 / rf, a power of two
                    float big = fmaxf(pr[0], pr[1]) * 16.f;
#pragma unroll
                    for (int x = 0; x < 2; ++x)
#pragma unroll
                        for (int G = 0; G < NG; ++G) {
                            w[x][G] = pr[x] * f * __uint_as_float(par[x][G].y << 16);
                            big = fmaxf(big, w[x][G]);
                        }
                    if (__any_sync(0xffffffffu, big > 4096.f)) {
                        // a weight grew past 2^8, or its product with a step past 2^12: new maximum and unit
                        float mx = fmaxf(s[0], s[1]);
#pragma unroll
                        for (int off = 4; off <= 16; off <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
                        const float mn = fmaxf(m[t], mx);
                        const float dl = ex2_approx(m[t] - mn);
                        float ref = 0.f;
#pragma unroll
                        for (int x = 0; x < 2; ++x) {
                            pr[x] = ex2_approx(s[x] - mn);
#pragma unroll
                            for (int G = 0; G < NG; ++G) ref = fmaxf(ref, pr[x] * __uint_as_float(par[x][G].y << 16));
                        }
#pragma unroll
                        for (int off = 4; off <= 16; off <<= 1) ref = fmaxf(ref, __shfl_xor_sync(0xffffffffu, ref, off));
                        ref = fminf(fmaxf(fmaxf(ref, rf[t] * dl), kMinUnit), kMaxUnit);
                        const float unit = __uint_as_float(__float_as_uint(ref) & 0x7f800000u);      // its power of two
                        const float f2 = __uint_as_float(0x7f000000u - __float_as_uint(unit));
                        const float so = dl * rf[t] * f2;
                        rf[t] = unit;
                        m[t] = mn;
                        l[t] *= dl;
#pragma unroll
                        for (int G = 0; G < NG; ++G) z[t][G] *= dl;
#pragma unroll
                        for (int x = 0; x < NG * 2; ++x) {
                            o[t][x][0] *= so; o[t][x][1] *= so; o[t][x][2] *= so; o[t][x][3] *= so;
                        }
#pragma unroll
                        for (int x = 0; x < 2; ++x)
#pragma unroll
                            for (int G = 0; G < NG; ++G) w[x][G] = pr[x] * f2 * __uint_as_float(par[x][G].y << 16);
                    }
                    l[t] += pr[0] + pr[1];
#pragma unroll
                    for (int G = 0; G < NG; ++G) {
                        z[t][G] = fmaf(pr[0], __uint_as_float(par[0][G].y & 0xffff0000u),
                                       fmaf(pr[1], __uint_as_float(par[1][G].y & 0xffff0000u), z[t][G]));
                        // row = key, columns (2 slot, 2 slot + 1) -> rows = columns of B, pairs of keys
                        uint32_t w0, w1;
                        split_f16(w[0][G], w[1][G], w0, w1);
                        bp[t][G][0] = transpose8(w0);
                        bp[t][G][1] = transpose8(w1);
                    }
                }
                if (loaded) {                             // the band tiles requested before Q.K; then the next ones
                    band_store(next, tile, next_band);
                    tile += kTileRegs * kWarps;
                    loaded = tile * 16 < next.n_rho;
                    if (loaded) band_load(next, tile);
                }
                // P.V: o[t][mt] = for slot c4, channels of row g and g+8 of the tile, (hi, lo) parts
                auto pv_tile = [&](int T) {
                    const bool on = QT > 1 || my_stream == T;
                    const int r = k0 + 16 * T + (lane & 15);
                    const uint32_t row = st_addr + kVOff + r * row_bytes, swap = wraps ? swap_of(r) : swap_lane;
#pragma unroll
                    for (int c2 = 0; c2 < NC; c2 += 2) {
                        uint32_t w[4];
                        mma::ldsm_x4_t(row + (((c2 + (lane >> 4)) ^ swap) << 4), w[0], w[1], w[2], w[3]);
#pragma unroll
                        for (int half = 0; half < 2; ++half) {
                            const int c = c2 + half, G = c / CPG;
#pragma unroll
                            for (int s = 0; s < SUB; ++s) {
                                const uint32_t x = w[2 * half] >> (8 * s), y = w[2 * half + 1] >> (8 * s);
#pragma unroll
                                for (int t = 0; t < QT; ++t)
                                    mma_f16(o[t][c * SUB + s], pair_even<BITS>(x), pair_odd<BITS>(x), pair_even<BITS>(y),
                                            pair_odd<BITS>(y), on ? bp[t][G][0] : 0u, on ? bp[t][G][1] : 0u);
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
            __syncwarp();                                 // every lane has read the stage
            if (lane == 0 && n + kStages < n_stage) copy_stage(n + kStages);
        }
        while (loaded) {
            band_store(next, tile, next_band);
            tile += kTileRegs * kWarps;
            loaded = tile * 16 < next.n_rho;
            if (loaded) band_load(next, tile);
        }
        if (p.f32) band_f32(next, next_band);
        // the next band is complete, and this one free for the one after it
        if (has_tiles(cur) || has_tiles(next)) __syncthreads();
        cur = next;
    }
    if (!ok && lane == 0)                                 // no copy may land after the CTA has gone
        for (int x = 0; x < n_stage; ++x) {
            int never = 0;
            const WaitCtl dw{&never, nullptr, 100000000ull};
            if (x >= n_stage - kStages) (void)mbar_wait(&full[x % kStages], (x / kStages) & 1, dw, 51);
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
        const float un = rf[t] * kTwo24;
#pragma unroll
        for (int x = 0; x < NG * 2; ++x) {
            ot[2 * x] = fmaf(o[t][x][0] + o[t][x][1], un, zt[x >> 1]);
            ot[2 * x + 1] = fmaf((o[t][x][2] + o[t][x][3]) * (BITS == 4 ? 0.0625f : 1.f), un, zt[x >> 1]);
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
    if (sp.ranks > 1) {
        if (p.f32) cluster_arrive();
        cluster_wait();
    }
    __syncthreads();
    // Row r is finished by rank r mod ranks, whose inbox takes the ranks' partial results of it.
    for (int x = tid; x < rows * DP; x += kThreads) {
        const int row = x / DP, d = x % DP, wb = row / Lq * wpe, il = row % Lq, be = b0 + row / Lq;
        const int own = has_own && be < p.B ? i0 + il + 1 : 0;
        float v[kOwn];
#pragma unroll
        for (int j = 0; j < kOwn; ++j)
            v[j] = j < own && d < p.D ? ld_elem(p.vcur, be * p.vc_sb + j * p.vc_st + h * p.vc_sh + d, p.f32) : 0.f;
        const float* src = part + (wb * sp.lq + il) * (DP + 2);
        const int step = sp.lq * (DP + 2);
        float mx = kNoMax;
        for (int w = 0; w < wpe; ++w) mx = fmaxf(mx, src[w * step + DP]);
        for (int j = 0; j < own; ++j) mx = fmaxf(mx, own_s[row * kOwn + j]);
        float lt = 0.f, ot = 0.f;
        for (int w = 0; w < wpe; ++w) {
            const float a = ex2_approx(src[w * step + DP] - mx);
            lt += src[w * step + DP + 1] * a;
            ot += src[w * step + d] * a;
        }
#pragma unroll
        for (int j = 0; j < kOwn; ++j)
            if (j < own) {
                const float a = ex2_approx(own_s[row * kOwn + j] - mx);
                lt += a;
                ot = fmaf(a, v[j], ot);
            }
        float* dst = inbox + (row / sp.ranks * sp.ranks + rank) * (DP + 2);
        const uint32_t to = row % sp.ranks;
        st_rank(dst + d, to, ot);
        if (d == 0) {
            st_rank(dst + DP, to, mx);
            st_rank(dst + DP + 1, to, lt);
        }
    }
    __syncthreads();
    if (sp.ranks > 1) {
        cluster_arrive();
        cluster_wait();
    }
    const int my_rows = (rows - rank + sp.ranks - 1) / sp.ranks;
    for (int x = tid; x < my_rows * DP; x += kThreads) {
        const int k = x / DP, d = x % DP, row = rank + k * sp.ranks, be = b0 + row / Lq;
        if (d >= p.D || be >= p.B) continue;
        const float* src = inbox + k * sp.ranks * (DP + 2);
        float mx = kNoMax, lt = 0.f, ot = 0.f;
        for (int r = 0; r < sp.ranks; ++r) mx = fmaxf(mx, src[r * (DP + 2) + DP]);
        for (int r = 0; r < sp.ranks; ++r) {
            const float a = ex2_approx(src[r * (DP + 2) + DP] - mx);
            lt += src[r * (DP + 2) + DP + 1] * a;
            ot += src[r * (DP + 2) + d] * a;
        }
        const int64_t at = be * p.o_sb + (i0 + row % Lq) * p.o_st + h * p.o_sh + d;
        if (p.f32) static_cast<float*>(p.out)[at] = ot / lt;
        else static_cast<__nv_bfloat16*>(p.out)[at] = __float2bfloat16_rn(ot / lt);
    }
}

template <int BITS, int NG, int QT, bool ONE>
cudaError_t launch(const QattnParams& p, const QSplit& sp, dim3 grid, cudaStream_t s)
{
    constexpr int DP = NG * 32;
    constexpr int staged = kWarps * kStages * stage_bytes(BITS, NG, QT);
    constexpr int bytes = staged + 2 * band_floats(BITS, NG, QT) * 4 +
                          (kMaxRows * (2 + NG + kDecodeMaxL) + kMaxRanks * (DP + 4)) * 4 +
                          (4 * kMaxRows + 1) * DP * 2 + kWarps * kStages * 8 + 16;
    static_assert(staged >= kWarps * 4 * QT * (DP + 2) * 4, "the warps' partial results fit");
    static_assert(kMaxRanks * (DP + 2) >= 2 * kMaxRows * DP, "the inbox covers qu and qv");
    static_assert(bytes <= 232448, "a CTA's shared memory");
    auto* kernel = qattn_kernel<BITS, NG, QT, ONE>;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess && sp.ranks > 8) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
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
    return cudaLaunchKernelEx(&cfg, kernel, p, sp);
}

template <int BITS, int NG>
cudaError_t launch_qt(const QattnParams& p, const QSplit& sp, dim3 grid, cudaStream_t s)
{
    if (sp.lq == 1) return launch<BITS, NG, 1, true>(p, sp, grid, s);
    return sp.lq <= 4 ? launch<BITS, NG, 1, false>(p, sp, grid, s) : launch<BITS, NG, 2, false>(p, sp, grid, s);
}

}  // namespace

cudaError_t launch_qattn(const QattnParams& p, int sm_count, cudaStream_t s)
{
    const int ng = p.G <= 2 ? 2 : 4, bits = p.bits == 8 ? 8 : 4;
    QSplit sp{};
    const int groups = p.L > 8 ? 2 : 1;                   // queries: eight at most per CTA
    sp.lq = (p.L + groups - 1) / groups;
    const int ks = stage_keys(bits, ng, sp.lq > 4 ? 2 : 1);
    // Batch entries of a CTA: as many as share a position band (eight rows, or the four that a small
    // band holds), but no fewer CTAs than SMs when the keys are split eight ways.
    const int64_t keys = p.M - p.lo;
    sp.nb = 1;
    while (2 * sp.nb * sp.lq <= kMaxRows && sp.nb < p.B) sp.nb *= 2;
    auto blocks = [&](int nb) { return static_cast<int64_t>(p.H) * ((p.B + nb - 1) / nb) * groups; };
    while (sp.nb > 1 && blocks(sp.nb) * 8 < sm_count) sp.nb /= 2;
    // Key ranges: as long as one wave of two CTAs per SM holds them all and each warp keeps two stages; 16
    // ranks only where eight leave SMs idle.
    sp.ranks = 1;
    while (sp.ranks < kMaxRanks && blocks(sp.nb) * sp.ranks <= (sp.ranks < 8 ? sm_count : sm_count - 1) &&
           keys > static_cast<int64_t>(sp.ranks) * 2 * ks * (kWarps / sp.nb))
        sp.ranks *= 2;
    sp.range = static_cast<int>(((keys + sp.ranks - 1) / sp.ranks + ks - 1) / ks * ks);
    if (sp.range == 0) sp.range = ks;
    const dim3 grid(sp.ranks * groups, p.H, (p.B + sp.nb - 1) / sp.nb);
    if (bits == 4) return ng == 2 ? launch_qt<4, 2>(p, sp, grid, s) : launch_qt<4, 4>(p, sp, grid, s);
    return ng == 2 ? launch_qt<8, 2>(p, sp, grid, s) : launch_qt<8, 4>(p, sp, grid, s);
}

}  // namespace txl
