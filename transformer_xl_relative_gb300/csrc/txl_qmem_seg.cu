// txl_qmem_seg.cu -- relative attention of an fp32 segment of more than 16 queries over a quantised memory
// and the segment's own keys, in fp32 arithmetic.
//
//     s_ij = scale [ (q_i+u).k'_j + (q_i+v).r[min(M+i-j, C)] ],  out_i = softmax_j(s_ij) v'_j
//
// One CTA: one batch entry and head, 32 queries, a range of keys in tiles of 64.  The codes of a tile are expanded
// into shared memory as fp32, the tile's 95 rows of r beside them; a thread takes two queries (16 apart) by
// four keys (16 apart), so that five rows of r serve its eight pairs.  Key ranges are the ranks of a cluster, joined
// through shared memory, because 32 queries of few heads fill few SMs.
//
// Bound by shared memory: 13 loads of 16 bytes for 64 multiply-adds of the scores, 6 for 32 of P.V.  (CUDA cores: on the
// tensor cores the codes could be multiplied as they are, as the kernel of few queries does, but q, the weights,
// r and the segment's own keys and values would have to be split.)  B2 H16 D64, 128 queries over 1500 4-bit keys: 150 us,
// 16 TFLOP/s; the general fp32 kernel over the memory read back took three times as long.
#include <algorithm>

#include "txl_internal.h"
#include "txl_ptx.cuh"
#include "txl_rows.cuh"

namespace txl {

namespace {

constexpr int kThreads = 256;
constexpr int kTQ = 32, kTK = 64, kTR = kTQ + kTK - 1;      // queries, keys, rows of r of a tile
constexpr int kMaxRanks = 8;
constexpr int kSPitch = kTK + 4;
constexpr float kNoMax = -3e38f;                            // running maximum before any key

template <int NG>
struct SegSmem {
    static constexpr int DP = 32 * NG, P = DP + 4;          // an odd number of 16 bytes: eight rows, eight bank groups
    float qu[kTQ * P], qv[kTQ * P];                         // (q+u), (q+v) in log2 units
    float k[kTK * P], v[kTK * P], r[kTR * P];
    float s[kTQ * kSPitch];
    float m[kTQ], l[kTQ], alpha[kTQ];
};

template <int NG>
__global__ void __launch_bounds__(kThreads, NG == 2 ? 2 : 1)
qseg_f32_kernel(const __grid_constant__ QattnParams p, int ranks, int tiles_per_rank)
{
    using S = SegSmem<NG>;
    constexpr int P = S::P, UPR = 4 * NG;                   // units of eight channels of a row
    extern __shared__ __align__(16) uint8_t smem_raw[];
    S& sm = *reinterpret_cast<S*>(smem_raw);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int rank = blockIdx.x % ranks, i0 = blockIdx.x / ranks * kTQ, h = blockIdx.y, b = blockIdx.z;
    const int Lq = min(kTQ, p.L - i0);
    const int64_t bh = static_cast<int64_t>(b) * p.H + h;
    pdl_launch_dependents();
    pdl_wait();

    for (int x = tid; x < kTQ * S::DP; x += kThreads) {
        const int ii = x / S::DP, d = x % S::DP;
        float a = 0.f, c = 0.f;
        if (ii < Lq && d < p.D) {
            const float q = ld(static_cast<const float*>(p.q) + b * p.q_sb + (i0 + ii) * p.q_st + h * p.q_sh + d);
            a = (q + __ldg(p.u + h * p.D + d)) * p.qscale;
            c = (q + __ldg(p.vb + h * p.D + d)) * p.qscale;
        }
        sm.qu[ii * P + d] = a;
        sm.qv[ii * P + d] = c;
    }
    if (tid < kTQ) {
        sm.m[tid] = kNoMax;
        sm.l[tid] = 0.f;
    }

    // queries qp, qp + 16; keys kq + 16 x; channels 4 (kq + 16 x) of the output
    const int qp = (warp & 3) * 4 + (lane >> 3), kq = (warp >> 2) * 8 + (lane & 7);
    float o[2][NG / 2][4] = {};
    const int row_bytes = q_row_bytes(p.G, p.bits), v_off = q_v_offset(p.G, p.bits), par_off = q_par_offset(p.G, p.bits);
    const uint8_t* head = p.rows + bh * p.M * row_bytes;
    const int end = p.M + i0 + Lq;                          // keys any of these queries sees
    const int64_t first = p.lo + static_cast<int64_t>(rank) * tiles_per_rank * kTK;
    for (int t = 0; t < tiles_per_rank; ++t) {
        const int64_t j64 = first + static_cast<int64_t>(t) * kTK;
        if (j64 >= end) break;
        const int j0 = static_cast<int>(j64);
        __syncthreads();                                    // the tile before has been used
        for (int x = tid; x < kTK * UPR; x += kThreads) {
            const int kk = x / UPR, d0 = 8 * (x % UPR), j = j0 + kk;
            float a[8] = {}, c[8] = {};
            if (j < p.M) {
                if (d0 < 32 * p.G) {
                    int64_t slot = static_cast<int64_t>(p.wp) + j;
                    if (slot >= p.M) slot -= p.M;
                    if (!in_range(slot, 0, p.M, p.chk)) slot = 0;
                    const uint8_t* row = head + slot * row_bytes;
                    const uint2 par = ld(reinterpret_cast<const uint2*>(row + par_off) + d0 / 32);
                    uint32_t ck[2], cv[2];
                    const uint8_t* at = row + d0 * p.bits / 8;
                    ck[0] = ld(reinterpret_cast<const uint32_t*>(at));
                    cv[0] = ld(reinterpret_cast<const uint32_t*>(at + v_off));
                    const float ks = __uint_as_float(par.x << 16), kl = __uint_as_float(par.x & 0xffff0000u);
                    const float vs = __uint_as_float(par.y << 16), vl = __uint_as_float(par.y & 0xffff0000u);
                    if (p.bits == 4) {
                        expand8<4>(ck, ks, kl, a);
                        expand8<4>(cv, vs, vl, c);
                    } else {
                        ck[1] = ld(reinterpret_cast<const uint32_t*>(at) + 1);
                        cv[1] = ld(reinterpret_cast<const uint32_t*>(at + v_off) + 1);
                        expand8<8>(ck, ks, kl, a);
                        expand8<8>(cv, vs, vl, c);
                    }
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        if (d0 + e >= p.D) a[e] = c[e] = 0.f;
                }
            } else if (j < end) {
                const int tk = j - p.M;
                load8<true>(static_cast<const float*>(p.kcur) + b * p.kc_sb + tk * p.kc_st + h * p.kc_sh, d0, p.D, p.vec_k, a);
                load8<true>(static_cast<const float*>(p.vcur) + b * p.vc_sb + tk * p.vc_st + h * p.vc_sh, d0, p.D, p.vec_v, c);
            }
            put8(sm.k + kk * P + d0, a);
            put8(sm.v + kk * P + d0, c);
        }
        const int delta0 = p.M + i0 - j0 - (kTK - 1);       // distance of row 0
        for (int x = tid; x < kTR * UPR; x += kThreads) {
            const int row = x / UPR, d0 = 8 * (x % UPR);
            int rr = min(max(delta0 + row, 0), p.C);        // (below 0: masked)
            if (rr >= p.n_rows || !in_range(rr, 0, p.n_rows, p.chk)) rr = 0;   // past the call's distances: unused
            float a[8] = {};
            load8<true>(static_cast<const float*>(p.r) + rr * p.r_row + h * p.r_head, d0, p.D, p.vec_r, a);
            put8(sm.r + row * P + d0, a);
        }
        __syncthreads();

        float s[2][4] = {}, e[2][4] = {};                   // summed apart: half the roundings
#pragma unroll 2
        for (int d = 0; d < S::DP; d += 4) {
            float4 qu[2], qv[2], r[5];
#pragma unroll
            for (int a = 0; a < 2; ++a) {
                qu[a] = f4(sm.qu + (qp + 16 * a) * P + d);
                qv[a] = f4(sm.qv + (qp + 16 * a) * P + d);
            }
#pragma unroll
            for (int y = 0; y < 5; ++y) r[y] = f4(sm.r + (qp - kq + 16 * (y - 3) + kTK - 1) * P + d);
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                const float4 k = f4(sm.k + (kq + 16 * x) * P + d);
#pragma unroll
                for (int a = 0; a < 2; ++a) {
                    s[a][x] = dot4(qu[a], k, s[a][x]);
                    e[a][x] = dot4(qv[a], r[a - x + 3], e[a][x]);
                }
            }
        }
#pragma unroll
        for (int a = 0; a < 2; ++a)
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                const int ii = qp + 16 * a, kk = kq + 16 * x;
                sm.s[ii * kSPitch + kk] = j0 + kk <= p.M + i0 + ii && j0 + kk < end ? s[a][x] + e[a][x] : -INFINITY;
            }
        __syncthreads();
#pragma unroll
        for (int y = 0; y < 4; ++y) {                       // a warp: four rows, two keys per lane
            const int ii = 4 * warp + y;
            float* row = sm.s + ii * kSPitch;
            const float x0 = row[lane], x1 = row[lane + 32], before = sm.m[ii];
            float mx = fmaxf(x0, x1);
#pragma unroll
            for (int off = 16; off > 0; off >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
            mx = fmaxf(mx, before);
            const float p0 = ex2_approx(x0 - mx), p1 = ex2_approx(x1 - mx), scale = ex2_approx(before - mx);
            float sum = p0 + p1;
#pragma unroll
            for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
            row[lane] = p0;
            row[lane + 32] = p1;
            __syncwarp();
            if (lane == 0) {
                sm.m[ii] = mx;
                sm.l[ii] = fmaf(sm.l[ii], scale, sum);
                sm.alpha[ii] = scale;
            }
        }
        __syncthreads();
#pragma unroll
        for (int a = 0; a < 2; ++a) {
            const float scale = sm.alpha[qp + 16 * a];
#pragma unroll
            for (int x = 0; x < NG / 2; ++x)
#pragma unroll
                for (int y = 0; y < 4; ++y) o[a][x][y] *= scale;
        }
        float ot[2][NG / 2][4] = {};                        // of this tile: sums of 64 terms, then of tiles
        const bool whole = j0 + kTK - 1 <= p.M + i0;        // no key is masked for any query
#pragma unroll 4
        for (int kk = 0; kk < kTK; kk += 4) {
            float pr[2][4];
#pragma unroll
            for (int a = 0; a < 2; ++a) {
                const float4 w = f4(sm.s + (qp + 16 * a) * kSPitch + kk);
                pr[a][0] = w.x; pr[a][1] = w.y; pr[a][2] = w.z; pr[a][3] = w.w;
            }
#pragma unroll
            for (int y = 0; y < 4; ++y)
#pragma unroll
                for (int x = 0; x < NG / 2; ++x) {
                    const float4 v = f4(sm.v + (kk + y) * P + 4 * (kq + 16 * x));
                    const float vv[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                    for (int a = 0; a < 2; ++a) {
                        // a value that the query does not see may be infinite or NaN
                        const bool seen = whole || j0 + kk + y <= p.M + i0 + qp + 16 * a;
#pragma unroll
                        for (int d = 0; d < 4; ++d) ot[a][x][d] = seen ? fmaf(pr[a][y], vv[d], ot[a][x][d]) : ot[a][x][d];
                    }
                }
        }
#pragma unroll
        for (int a = 0; a < 2; ++a)
#pragma unroll
            for (int x = 0; x < NG / 2; ++x)
#pragma unroll
                for (int d = 0; d < 4; ++d) o[a][x][d] += ot[a][x][d];
    }

    // ---- join the ranks: each leaves its output in its shared memory, row ii is finished by rank ii mod ranks
    __syncthreads();
#pragma unroll
    for (int a = 0; a < 2; ++a)
#pragma unroll
        for (int x = 0; x < NG / 2; ++x)
            *reinterpret_cast<float4*>(sm.k + (qp + 16 * a) * P + 4 * (kq + 16 * x)) =
                make_float4(o[a][x][0], o[a][x][1], o[a][x][2], o[a][x][3]);
    __syncthreads();
    if (ranks > 1) cluster_sync_all();
    const int rows = (Lq - rank + ranks - 1) / ranks;
    for (int x = tid; x < rows * S::DP; x += kThreads) {
        const int ii = rank + x / S::DP * ranks, d = x % S::DP;
        if (d >= p.D) continue;
        float mx = kNoMax, lt = 0.f, ot = 0.f;
        for (int y = 0; y < ranks; ++y) {
            const float my = ranks > 1 ? ld_rank(sm.m + ii, y) : sm.m[ii];
            const float ly = ranks > 1 ? ld_rank(sm.l + ii, y) : sm.l[ii];
            const float oy = ranks > 1 ? ld_rank(sm.k + ii * P + d, y) : sm.k[ii * P + d];
            const float mn = fmaxf(mx, my), w0 = ex2_approx(mx - mn), w1 = ex2_approx(my - mn);
            lt = lt * w0 + ly * w1;
            ot = ot * w0 + oy * w1;
            mx = mn;
        }
        static_cast<float*>(p.out)[b * p.o_sb + (i0 + ii) * p.o_st + h * p.o_sh + d] = ot / lt;
    }
    if (ranks > 1) cluster_sync_all();                      // the others have read this rank's shared memory
}

template <int NG>
cudaError_t launch(const QattnParams& p, int sm_count, cudaStream_t s)
{
    auto* kernel = qseg_f32_kernel<NG>;
    constexpr int bytes = sizeof(SegSmem<NG>);
    static_assert(bytes <= 232448, "a CTA's shared memory");
    static OncePerDevice once;
    const cudaError_t prepared = allow_smem(once, bytes, kernel);
    if (prepared != cudaSuccess) return prepared;
    // key ranges: until every SM has a CTA (with two CTAs each 165 us instead of 150 on the shape above), of a tile at
    // least (two at least: 46 instead of 28 us for 100 queries over 700 keys of 8 heads)
    const int64_t groups = (p.L + kTQ - 1) / kTQ, tiles = (static_cast<int64_t>(p.M) - p.lo + p.L + kTK - 1) / kTK;
    int ranks = 1;
    while (ranks < kMaxRanks && groups * p.H * p.B * ranks < sm_count && tiles >= 2 * ranks) ranks *= 2;
    if (groups * ranks > INT32_MAX) return cudaErrorInvalidValue;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(groups * ranks), p.H, p.B);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = bytes;
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
    return cudaLaunchKernelEx(&cfg, kernel, p, ranks, static_cast<int>((tiles + ranks - 1) / ranks));
}

}  // namespace

cudaError_t launch_qseg_f32(const QattnParams& p, int sm_count, cudaStream_t s)
{
    return p.G <= 2 ? launch<2>(p, sm_count, s) : launch<4>(p, sm_count, s);
}

}  // namespace txl
