// txl_paged_attn.cu -- relative attention of 1 .. 16 new tokens a sequence over a memory held in pages.
//
// Query i of a sequence has position p_i, slot j of its memory position p_j ("跨窗口的相对位置编码" §3; the clamp of
// "TransformerXL 相对位置编码" §2.4), C the last distance with a position term:
//     s_ij = scale [ (q_i+u).k_j + (q_i+v).r_min(p_i - p_j, C) ],  visible iff p_j <= p_i,  out_i = softmax_j(s_ij) V
// and, where asked, weight_j += sum over heads and queries of the softmax.
//
//   paged_prep_kernel    new keys and values enter their pages; position terms E[b][h][i][distance]; what the call works
//                        on (lengths, queries' positions) is fixed in the workspace
//   paged_attn_kernel    the tiles of 16 keys of all (sequence, head) pairs in one line, cut into equal shares: a block
//                        takes a share, and the last block of a pair joins its parts
//   paged_weight_kernel  (accumulate) 2^(score - log-sum-exp) summed over heads and queries, a thread per slot
#include <cuda_bf16.h>

#include "txl_mma.cuh"
#include "txl_paged.cuh"
#include "txl_ptx.cuh"

namespace txl {

namespace {

constexpr int kThreads = 128, kWarps = kThreads / 32;
constexpr int kMinTiles = 8;               // tiles of a share, at least: two a warp
constexpr float kNone = -INFINITY;

template <typename T> __device__ __forceinline__ float to_f(T x);
template <> __device__ __forceinline__ float to_f<float>(float x) { return x; }
template <> __device__ __forceinline__ float to_f<__nv_bfloat16>(__nv_bfloat16 x) { return __bfloat162float(x); }
template <typename T> __device__ __forceinline__ T from_f(float x);
template <> __device__ __forceinline__ float from_f<float>(float x) { return x; }
template <> __device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }

__device__ __forceinline__ uint4 load16(const void* p)
{
    uint4 w;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(w.x), "=r"(w.y), "=r"(w.z), "=r"(w.w) : "l"(p));
    return w;
}

// Keeps the first `live` bf16 of eight.
__device__ __forceinline__ uint4 first_of8(uint4 w, int live)
{
    auto keep = [&](uint32_t x, int e) { return live >= e + 2 ? x : live == e + 1 ? x & 0xffffu : 0u; };
    return make_uint4(keep(w.x, 0), keep(w.y, 2), keep(w.z, 4), keep(w.w, 6));
}

// ---------------------------------------------------------------- fragments of the queries
// A 16 x 16 fragment of mma.m16n8k16 holds eight queries twice: row g the upper 8 bits of (q + bias) * scale, row
// g + 8 the next 8, so that the sum of the two rows' products has 16 bits of the query.  The channels are permuted:
// lane (g, t) holds channels 8 c .. 8 c + 7 of query g for its chunks c = t + 4 j, as the keys' rows are loaded.
template <int NC> struct QFrag { uint32_t hi[NC][4], lo[NC][4]; };

template <int NC>
__device__ __forceinline__ void load_q(QFrag<NC>& f, const __nv_bfloat16* q, const float* bias, bool live, int D, float scale,
                                       int t)
{
#pragma unroll
    for (int j = 0; j < NC; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            float x[2];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const int d = 8 * (t + 4 * j) + 2 * e + k;
                x[k] = live && d < D ? (__bfloat162float(q[d]) + bias[d]) * scale : 0.f;
            }
            f.hi[j][e] = mma::pack2(x[0], x[1]);
            f.lo[j][e] = mma::pack2(x[0] - mma::bf16_lo(f.hi[j][e]), x[1] - mma::bf16_hi(f.hi[j][e]));
        }
}

// Scores of eight queries and the eight rows whose chunks are w: c[0], c[1] rows 2t, 2t+1 for query g.
template <int NC>
__device__ __forceinline__ void score8(const QFrag<NC>& f, const uint4* w, float* s)
{
    float c[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int j = 0; j < NC; ++j) {
        mma::mma16816(c, f.hi[j][0], f.lo[j][0], f.hi[j][1], f.lo[j][1], w[j].x, w[j].y);
        mma::mma16816(c, f.hi[j][2], f.lo[j][2], f.hi[j][3], f.lo[j][3], w[j].z, w[j].w);
    }
    s[0] = c[0] + c[2];
    s[1] = c[1] + c[3];
}

// ---------------------------------------------------------------- preparation
// Blocks 0 .. B-1 take a sequence's new positions, the others position terms: of 8 queries (of all sequences) and a head
// with kPrepRows distances.
constexpr int kPrepRows = 128;

template <typename T>
__device__ __forceinline__ void prep_sequence(const PagedAttnParams& p, int b)
{
    const PagedParams& m = p.n.m;
    const int n = paged_count(p.n.counts, b, p.n.T);
    const int len = m.length[b], next = m.next_pos[b];
    int4 now = make_int4(len, next, n, 0);
    if (p.n.xk && n > 0) {
        if (paged_room(m, b, len, n)) {
            paged_copy<T>(p.n, b, len, next, 0, n);
            now.x = len + n;
        } else {
            if (threadIdx.x == 0) page_error(m);
            now.z = 0;
        }
    } else {
        now.y = next - n;
        if (len < 0 || len > p.cap) {
            if (threadIdx.x == 0) page_error(m);
            now.x = now.z = 0;
        }
    }
    if (threadIdx.x == 0) p.now[b] = now;
    for (int h = threadIdx.x; h < m.H; h += kThreads) p.tickets[b * m.H + h] = 0;
}

template <int NC>
__device__ __forceinline__ void prep_terms_bf16(const PagedAttnParams& p, int h, int f0, int d0)
{
    const PagedParams& m = p.n.m;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
    const int T = p.n.T, f = f0 + g, b = f / T, i = f - b * T;
    const bool live = f < m.B * T;
    QFrag<NC> q;
    const __nv_bfloat16* qr = static_cast<const __nv_bfloat16*>(p.q);
    if (live) qr += b * p.q_sb + i * p.q_st + h * p.q_sh;
    load_q<NC>(q, qr, p.vb + h * m.D, live, m.D, p.qscale, t);
    float* E = p.E + ((static_cast<int64_t>(b) * m.H + h) * T + i) * p.e_pitch;
    const uint16_t* r = static_cast<const uint16_t*>(p.r) + h * p.r_head;
    for (int x0 = d0 + warp * 8; x0 < min(p.n_e, d0 + kPrepRows); x0 += kWarps * 8) {
        const uint16_t* row = r + static_cast<int64_t>(min(x0 + g, p.n_e - 1)) * p.r_row;
        uint4 w[NC];
#pragma unroll
        for (int j = 0; j < NC; ++j) {
            const int c = t + 4 * j;
            if (p.vec_r && 8 * c + 8 <= m.D) {
                w[j] = *reinterpret_cast<const uint4*>(row + 8 * c);
            } else {
                uint32_t x[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) x[e] = 8 * c + e < m.D ? row[8 * c + e] : 0u;
                w[j] = make_uint4(x[0] | x[1] << 16, x[2] | x[3] << 16, x[4] | x[5] << 16, x[6] | x[7] << 16);
            }
        }
        float s[2];
        score8<NC>(q, w, s);
        if (live) *reinterpret_cast<float2*>(E + x0 + 2 * t) = make_float2(s[0], s[1]);
    }
}

// fp32: a thread per distance, the queries' rows from shared memory.
__device__ __forceinline__ void prep_terms_f32(const PagedAttnParams& p, int h, int f0, int d0, float* q)
{
    const PagedParams& m = p.n.m;
    const int T = p.n.T, D = m.D;
    const int n = min(8, m.B * T - f0);
    for (int x = threadIdx.x; x < 8 * D; x += kThreads) {
        const int f = f0 + x / D, d = x % D, b = f / T, i = f - b * T;
        q[x] = x / D < n ? (static_cast<const float*>(p.q)[b * p.q_sb + i * p.q_st + h * p.q_sh + d] + p.vb[h * D + d]) * p.qscale : 0.f;
    }
    __syncthreads();
    const int x = d0 + threadIdx.x;
    if (x < p.n_e) {
        const float* row = static_cast<const float*>(p.r) + h * p.r_head + static_cast<int64_t>(x) * p.r_row;
        float s[8] = {};
        for (int d = 0; d < D; ++d) {
            const float y = row[d];
#pragma unroll
            for (int e = 0; e < 8; ++e) s[e] = fmaf(q[e * D + d], y, s[e]);
        }
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (e < n) {
                const int f = f0 + e, b = f / T, i = f - b * T;
                p.E[((static_cast<int64_t>(b) * m.H + h) * T + i) * p.e_pitch + x] = s[e];
            }
    }
}

template <typename T, int NC>
__global__ void __launch_bounds__(kThreads) paged_prep_kernel(const __grid_constant__ PagedAttnParams p)
{
    __shared__ float qs[sizeof(T) == 4 ? 8 * 128 : 1];
    __shared__ int far;
    pdl_wait();
    pdl_launch_dependents();
    const PagedParams& m = p.n.m;
    if (blockIdx.x < static_cast<unsigned>(m.B)) {
        prep_sequence<T>(p, blockIdx.x);
        return;
    }
    const int x = blockIdx.x - m.B, parts = (p.n_e + kPrepRows - 1) / kPrepRows;
    const int d0 = x % parts * kPrepRows, h = x / parts % m.H, f0 = x / parts / m.H * 8;
    // distances beyond the start of all of these sequences are not met (next_pos changes in the attention's kernel)
    if (threadIdx.x == 0) far = 0;
    __syncthreads();
    const int b0 = f0 / p.n.T, b1 = min(m.B - 1, (f0 + 7) / p.n.T);
    const int b = b0 + static_cast<int>(threadIdx.x);
    if (b <= b1 && paged_count(p.n.counts, b, p.n.T) > 0)
        atomicMax(&far, m.next_pos[b] + (p.n.xk ? p.n.T : 0));
    __syncthreads();
    if (d0 >= far) return;
    if constexpr (sizeof(T) == 4) prep_terms_f32(p, h, f0, d0, qs);
    else prep_terms_bf16<NC>(p, h, f0, d0);
}

// ---------------------------------------------------------------- attention
// What a block knows of the part of a (sequence, head) pair that it works on.
struct Part {
    int b, h, len, first, n;       // slots, position of the first query, queries
    int t0, t1, tiles;             // its tiles, of the pair's
};

// Page of the tiles that a warp will come to: lane x knows that of the warp's x-th tile from `base` on.
struct Pages {
    int base, mine;
    __device__ __forceinline__ void look(const PagedParams& m, const Part& a, int tile, int lane)
    {
        base = tile;
        const int at = tile + kWarps * lane;
        mine = at < a.t1 ? page_of(m, a.b, at * kPageUnit) : -1;
        if (at < a.t1 && mine < 0) page_error(m);
    }
    // page of `tile` (a warp's own, at or after base)
    __device__ __forceinline__ int get(const PagedParams& m, const Part& a, int tile, int lane)
    {
        if (tile - base >= 32 * kWarps) look(m, a, tile, lane);
        return __shfl_sync(0xffffffffu, mine, (tile - base) / kWarps);
    }
};

// Running softmax of one query: maximum, sum, weighted values are kept by the callers.
__device__ __forceinline__ float finite_or_0(float m) { return m == kNone ? 0.f : m; }

// bf16.  A warp's tile is 16 keys: lane (g, t) loads chunks t + 4 j of keys g and g + 8, and chunks g + 8 x of the
// values of keys 2t, 2t+1, 2t+8, 2t+9, all of 16 bytes from global memory: the first are B fragments of the scores' mma as
// they are, the others become those of P.V by pairing the halves of two keys' words.  NV = ceil(D / 64).
template <int NC, int NQ, bool W>
__device__ __forceinline__ void part_bf16(const PagedAttnParams& p, const Part& a, float* buf, float* bml)
{
    constexpr int NV = (NC + 1) / 2;
    const PagedParams& m = p.n.m;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
    const int T = p.n.T;
    QFrag<NC> q[NQ];
    const float* E[NQ];
    float* S[NQ];
    bool live[NQ];
#pragma unroll
    for (int x = 0; x < NQ; ++x) {
        const int i = 8 * x + g;
        live[x] = i < a.n;
        const __nv_bfloat16* qr = static_cast<const __nv_bfloat16*>(p.q);
        if (live[x]) qr += a.b * p.q_sb + i * p.q_st + a.h * p.q_sh;
        load_q<NC>(q[x], qr, p.u + a.h * m.D, live[x], m.D, p.qscale, t);
        const int64_t row = (static_cast<int64_t>(a.b) * m.H + a.h) * T + min(i, T - 1);
        E[x] = p.E + row * p.e_pitch;
        S[x] = W ? p.S + row * p.cap : nullptr;
    }
    float o[NQ][NV][8][4];
    float mx[NQ], sum[NQ];
#pragma unroll
    for (int x = 0; x < NQ; ++x) {
        mx[x] = kNone;
        sum[x] = 0.f;
#pragma unroll
        for (int v = 0; v < NV; ++v)
#pragma unroll
            for (int e = 0; e < 8; ++e) o[x][v][e][0] = o[x][v][e][1] = o[x][v][e][2] = o[x][v][e][3] = 0.f;
    }
    const int chunks = (m.D + 7) / 8, last_live = m.D - 8 * (chunks - 1);       // channels of a row's last chunk

    Pages pages;
    pages.look(m, a, a.t0 + warp, lane);
    uint4 kw[2][NC], vw[4][NV];
    int2 pw[2], pn[2];
    auto row_of = [&](int page, int tile) { return tile * kPageUnit % m.page_len; };
    auto load_k = [&](int page, int tile) {
        const uint16_t* k = static_cast<const uint16_t*>(m.k) + page_row0(m, page, a.h) + static_cast<int64_t>(row_of(page, tile) + g) * m.ld;
#pragma unroll
        for (int y = 0; y < 2; ++y)
#pragma unroll
            for (int j = 0; j < NC; ++j) {
                const int c = t + 4 * j;
                kw[y][j] = c < chunks ? load16(k + y * 8 * m.ld + 8 * c) : make_uint4(0, 0, 0, 0);
            }
    };
    auto load_v = [&](int page, int tile) {
        const uint16_t* v = static_cast<const uint16_t*>(m.v) + page_row0(m, page, a.h) + static_cast<int64_t>(row_of(page, tile) + 2 * t) * m.ld;
#pragma unroll
        for (int y = 0; y < 4; ++y)
#pragma unroll
            for (int x = 0; x < NV; ++x) {
                const int c = g + 8 * x;
                vw[y][x] = c < chunks ? load16(v + ((y & 1) + (y & 2) * 4) * m.ld + 8 * c) : make_uint4(0, 0, 0, 0);
            }
    };
    auto load_pos = [&](int page, int tile, int2* w) {
        const int* at = m.pos + static_cast<int64_t>(page) * m.page_len + row_of(page, tile) + 2 * t;
        w[0] = *reinterpret_cast<const int2*>(at);
        w[1] = *reinterpret_cast<const int2*>(at + 8);
    };
    // position terms of a tile; what its masks leave out is -inf
    float e[NQ][4];
    auto load_e = [&](int tile, const int2* w) {
        const int pos[4] = {w[0].x, w[0].y, w[1].x, w[1].y};
#pragma unroll
        for (int x = 0; x < NQ; ++x)
#pragma unroll
            for (int y = 0; y < 4; ++y) {
                const int slot = tile * kPageUnit + 2 * t + (y & 1) + (y & 2) * 4;
                const int delta = a.first + 8 * x + g - pos[y];
                e[x][y] = kNone;
                if (live[x] && delta >= 0 && slot < a.len) e[x][y] = E[x][min(delta, p.n_e - 1)];
            }
    };
    int page = -1, next = -1;
    int tile = a.t0 + warp;
    if (tile < a.t1) {
        page = pages.get(m, a, tile, lane);
        if (page >= 0) {
            load_pos(page, tile, pw);
            load_k(page, tile);
            load_v(page, tile);
            load_e(tile, pw);
        }
        if (tile + kWarps < a.t1) {
            next = pages.get(m, a, tile + kWarps, lane);
            if (next >= 0) load_pos(next, tile + kWarps, pn);
        }
    }
    for (; tile < a.t1; tile += kWarps) {
        // page, pw's terms e, kw, vw: this tile's; next, pn: the following one's
        const bool more = tile + kWarps < a.t1;
        float s[NQ][4];
        if (page >= 0) {
            if (last_live < 8) {
#pragma unroll
                for (int j = 0; j < NC; ++j)
                    if (t + 4 * j == chunks - 1) {
                        kw[0][j] = first_of8(kw[0][j], last_live);
                        kw[1][j] = first_of8(kw[1][j], last_live);
                    }
            }
#pragma unroll
            for (int x = 0; x < NQ; ++x) {
                score8<NC>(q[x], kw[0], s[x]);
                score8<NC>(q[x], kw[1], s[x] + 2);
#pragma unroll
                for (int y = 0; y < 4; ++y) s[x][y] = e[x][y] == kNone ? kNone : s[x][y] + e[x][y];
            }
        }
        int after = -1;
        if (more) {
            if (next >= 0) {
                load_k(next, tile + kWarps);
                load_e(tile + kWarps, pn);
            }
            if (tile + 2 * kWarps < a.t1) {
                after = pages.get(m, a, tile + 2 * kWarps, lane);
                if (after >= 0) load_pos(after, tile + 2 * kWarps, pn);
            }
        }
        if (page >= 0) {
            // values of slots past the end are anything: they count as 0
            if (tile * kPageUnit + kPageUnit > a.len) {
#pragma unroll
                for (int y = 0; y < 4; ++y)
                    if (tile * kPageUnit + 2 * t + (y & 1) + (y & 2) * 4 >= a.len)
#pragma unroll
                        for (int x = 0; x < NV; ++x) vw[y][x] = make_uint4(0, 0, 0, 0);
            }
#pragma unroll
            for (int x = 0; x < NQ; ++x) {
                if (W && live[x]) {
                    *reinterpret_cast<float2*>(S[x] + tile * kPageUnit + 2 * t) = make_float2(s[x][0], s[x][1]);
                    *reinterpret_cast<float2*>(S[x] + tile * kPageUnit + 8 + 2 * t) = make_float2(s[x][2], s[x][3]);
                }
                float top = fmaxf(fmaxf(s[x][0], s[x][1]), fmaxf(s[x][2], s[x][3]));
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
                if (__any_sync(0xffffffffu, top > mx[x])) {
                    const float now = fmaxf(mx[x], top), f = mma::ex2(mx[x] - finite_or_0(now));
                    mx[x] = now;
                    sum[x] *= f;
#pragma unroll
                    for (int v = 0; v < NV; ++v)
#pragma unroll
                        for (int z = 0; z < 8; ++z)
#pragma unroll
                            for (int y = 0; y < 4; ++y) o[x][v][z][y] *= f;
                }
                const float base = finite_or_0(mx[x]);
                float pr[4];
#pragma unroll
                for (int y = 0; y < 4; ++y) {
                    pr[y] = mma::ex2(s[x][y] - base);
                    sum[x] += pr[y];
                }
                // a weight is held to 16 bits as well: its upper 8 in row g, the next 8 in row g + 8
                const uint32_t h0 = mma::pack2(pr[0], pr[1]), h1 = mma::pack2(pr[2], pr[3]);
                const uint32_t l0 = mma::pack2(pr[0] - mma::bf16_lo(h0), pr[1] - mma::bf16_hi(h0));
                const uint32_t l1 = mma::pack2(pr[2] - mma::bf16_lo(h1), pr[3] - mma::bf16_hi(h1));
#pragma unroll
                for (int v = 0; v < NV; ++v)
#pragma unroll
                    for (int z = 0; z < 8; ++z) {
                        const uint32_t* w0 = reinterpret_cast<const uint32_t*>(&vw[0][v]);
                        const uint32_t* w1 = reinterpret_cast<const uint32_t*>(&vw[1][v]);
                        const uint32_t* w2 = reinterpret_cast<const uint32_t*>(&vw[2][v]);
                        const uint32_t* w3 = reinterpret_cast<const uint32_t*>(&vw[3][v]);
                        const uint32_t pick = z & 1 ? 0x7632 : 0x5410;
                        mma::mma16816(o[x][v][z], h0, l0, h1, l1, __byte_perm(w0[z >> 1], w1[z >> 1], pick),
                                      __byte_perm(w2[z >> 1], w3[z >> 1], pick));
                    }
            }
        }
        if (more && next >= 0) load_v(next, tile + kWarps);
        page = next;
        next = after;
    }
    // the warp's share into shared memory: channels 64 v + 16 t + z and + 8 + z of query g
#pragma unroll
    for (int x = 0; x < NQ; ++x) {
        sum[x] += __shfl_xor_sync(0xffffffffu, sum[x], 1);
        sum[x] += __shfl_xor_sync(0xffffffffu, sum[x], 2);
        if (!live[x]) continue;
        const int i = 8 * x + g;
        if (t == 0) {
            bml[(warp * T + i) * 2] = mx[x];
            bml[(warp * T + i) * 2 + 1] = sum[x];
        }
        float* row = buf + (warp * T + i) * p.Dp;
#pragma unroll
        for (int v = 0; v < NV; ++v)
#pragma unroll
            for (int z = 0; z < 8; ++z)
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                    const int d = 64 * v + 16 * t + 8 * y + z;
                    if (d < p.Dp) row[d] = o[x][v][z][y] + o[x][v][z][y + 2];
                }
    }
}

// fp32, CUDA cores.  Lane (g, t) takes keys g and g + 8 of a tile and channels 4 (t + 4 j) .. + 3; each of the eight g keeps
// maximum and sums of its own, which meet at the end.  NQ queries at a time: their sums stay in registers.
template <int NC, int NQ, bool W>
__device__ __forceinline__ void part_f32(const PagedAttnParams& p, const Part& a, float* buf, float* bml, float* qs)
{
    constexpr int NJ = 2 * NC;             // chunks of four channels of a lane
    const PagedParams& m = p.n.m;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
    const int T = p.n.T, D = m.D;
    for (int i0 = 0; i0 < a.n; i0 += NQ) {
        __syncthreads();
        for (int x = threadIdx.x; x < NQ * p.Dp; x += kThreads) {
            const int i = i0 + x / p.Dp, d = x % p.Dp;
            qs[x] = i < a.n && d < D ? (static_cast<const float*>(p.q)[a.b * p.q_sb + i * p.q_st + a.h * p.q_sh + d] + p.u[a.h * D + d]) * p.qscale : 0.f;
        }
        __syncthreads();
        float o[NQ][NJ][4], mx[NQ], sum[NQ];
#pragma unroll
        for (int x = 0; x < NQ; ++x) {
            mx[x] = kNone;
            sum[x] = 0.f;
#pragma unroll
            for (int j = 0; j < NJ; ++j) o[x][j][0] = o[x][j][1] = o[x][j][2] = o[x][j][3] = 0.f;
        }
        Pages pages;
        pages.look(m, a, a.t0 + warp, lane);
        for (int tile = a.t0 + warp; tile < a.t1; tile += kWarps) {
            const int page = pages.get(m, a, tile, lane);
            if (page < 0) continue;
            const int row = tile * kPageUnit % m.page_len;
#pragma unroll
            for (int y = 0; y < 2; ++y) {
                const int slot = tile * kPageUnit + 8 * y + g;
                const int64_t at = page_row0(m, page, a.h) + static_cast<int64_t>(row + 8 * y + g) * m.ld;
                const int pos = m.pos[static_cast<int64_t>(page) * m.page_len + row + 8 * y + g];
                float4 k[NJ], v[NJ];
#pragma unroll
                for (int j = 0; j < NJ; ++j) {
                    const int d = 4 * (t + 4 * j);
                    k[j] = v[j] = make_float4(0.f, 0.f, 0.f, 0.f);
                    if (slot < a.len && d < D) {
                        k[j] = *reinterpret_cast<const float4*>(static_cast<const float*>(m.k) + at + d);
                        v[j] = *reinterpret_cast<const float4*>(static_cast<const float*>(m.v) + at + d);
                        if (d + 1 >= D) k[j].y = 0.f;          // a row's padding is anything
                        if (d + 2 >= D) k[j].z = 0.f;
                        if (d + 3 >= D) k[j].w = 0.f;
                    }
                }
#pragma unroll
                for (int x = 0; x < NQ; ++x) {
                    const int i = i0 + x;
                    float s = 0.f;
#pragma unroll
                    for (int j = 0; j < NJ; ++j) {
                        const float4 w = *reinterpret_cast<const float4*>(qs + x * p.Dp + 4 * (t + 4 * j));
                        s = fmaf(w.w, k[j].w, fmaf(w.z, k[j].z, fmaf(w.y, k[j].y, fmaf(w.x, k[j].x, s))));
                    }
                    s += __shfl_xor_sync(0xffffffffu, s, 1);
                    s += __shfl_xor_sync(0xffffffffu, s, 2);
                    const int delta = a.first + i - pos;
                    const bool seen = i < a.n && slot < a.len && delta >= 0;
                    const int64_t er = (static_cast<int64_t>(a.b) * m.H + a.h) * T + i;
                    s = seen ? s + p.E[er * p.e_pitch + min(delta, p.n_e - 1)] : kNone;
                    if (W && t == 0 && i < a.n) p.S[er * p.cap + slot] = s;
                    if (seen) {
                        if (!(s <= mx[x])) {
                            const float now = fmaxf(mx[x], s), f = exp2f(mx[x] - finite_or_0(now));
                            mx[x] = now;
                            sum[x] *= f;
#pragma unroll
                            for (int j = 0; j < NJ; ++j) { o[x][j][0] *= f; o[x][j][1] *= f; o[x][j][2] *= f; o[x][j][3] *= f; }
                        }
                        const float pr = exp2f(s - finite_or_0(mx[x]));
                        sum[x] += pr;
#pragma unroll
                        for (int j = 0; j < NJ; ++j) {
                            o[x][j][0] = fmaf(pr, v[j].x, o[x][j][0]);
                            o[x][j][1] = fmaf(pr, v[j].y, o[x][j][1]);
                            o[x][j][2] = fmaf(pr, v[j].z, o[x][j][2]);
                            o[x][j][3] = fmaf(pr, v[j].w, o[x][j][3]);
                        }
                    }
                }
            }
        }
#pragma unroll
        for (int x = 0; x < NQ; ++x) {
            float top = mx[x];
#pragma unroll
            for (int d = 4; d < 32; d <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
            const float f = mx[x] == kNone ? 0.f : exp2f(mx[x] - finite_or_0(top));
            float l = sum[x] * f;
            if (mx[x] == kNone) l = sum[x];                    // (0, or NaN from a score that is not a number)
#pragma unroll
            for (int d = 4; d < 32; d <<= 1) l += __shfl_xor_sync(0xffffffffu, l, d);
#pragma unroll
            for (int j = 0; j < NJ; ++j)
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    float y = mx[x] == kNone ? o[x][j][c] : o[x][j][c] * f;
#pragma unroll
                    for (int d = 4; d < 32; d <<= 1) y += __shfl_xor_sync(0xffffffffu, y, d);
                    if (g == 0 && i0 + x < a.n && 4 * (t + 4 * j) + c < p.Dp)
                        buf[(warp * T + i0 + x) * p.Dp + 4 * (t + 4 * j) + c] = y;
                }
            if (lane == 0 && i0 + x < a.n) {
                bml[(warp * T + i0 + x) * 2] = top;
                bml[(warp * T + i0 + x) * 2 + 1] = l;
            }
        }
    }
}

template <typename T> __device__ __forceinline__ T* out_row(const PagedAttnParams& p, const Part& a, int i)
{
    return static_cast<T*>(p.out) + a.b * p.o_sb + i * p.o_st + a.h * p.o_sh;
}

// One query's row again, key by key on the CUDA cores: its sums are not finite, and a value that is not finite at a key
// that the query does not see must not reach it (0 times infinity).  The whole block calls; tot: 2 + kThreads floats.
template <typename T>
__device__ __noinline__ void row_again(const PagedAttnParams& p, const Part& a, int i, float* tot)
{
    const PagedParams& m = p.n.m;
    const T* q = static_cast<const T*>(p.q) + a.b * p.q_sb + i * p.q_st + a.h * p.q_sh;
    const float* E = p.E + ((static_cast<int64_t>(a.b) * m.H + a.h) * p.n.T + i) * p.e_pitch;
    const int at = a.first + i;
    auto score = [&](int s, int page) {                       // NaN counts as seen
        const int delta = at - m.pos[static_cast<int64_t>(page) * m.page_len + s % m.page_len];
        if (delta < 0) return kNone;
        const T* k = static_cast<const T*>(m.k) + page_row0(m, page, a.h) + static_cast<int64_t>(s % m.page_len) * m.ld;
        float x = 0.f;
        for (int d = 0; d < m.D; ++d) x = fmaf((to_f(q[d]) + p.u[a.h * m.D + d]) * p.qscale, to_f(k[d]), x);
        return x + E[min(delta, p.n_e - 1)];
    };
    float top = kNone;
    for (int s = threadIdx.x; s < a.len; s += kThreads) {
        const int page = page_of(m, a.b, s);
        if (page >= 0) top = fmaxf(top, score(s, page));
    }
    __syncthreads();
    tot[threadIdx.x] = top;
    __syncthreads();
    for (int x = 0; x < kThreads; ++x) top = fmaxf(top, tot[x]);
    top = finite_or_0(top);
    float sum = 0.f, o = 0.f;
    const int d = threadIdx.x;                                // D <= 128: a channel a thread
    for (int s0 = 0; s0 < a.len; s0 += kThreads) {
        const int s = s0 + threadIdx.x;
        const int page = s < a.len ? page_of(m, a.b, s) : -1;
        float x = kNone;
        if (page >= 0) x = score(s, page);
        __syncthreads();
        tot[threadIdx.x] = x;
        __syncthreads();
        for (int y = 0; y < min(kThreads, a.len - s0); ++y) {
            const int from = page_of(m, a.b, s0 + y);
            // (a key that is seen and scores -inf weighs 0 as well; its values count as unseen)
            if (from < 0 || tot[y] == kNone) continue;
            const float w = exp2f(tot[y] - top);
            sum += w;
            if (d < m.D)
                o = fmaf(w, to_f(static_cast<const T*>(m.v)[page_row0(m, from, a.h) + static_cast<int64_t>((s0 + y) % m.page_len) * m.ld + d]), o);
        }
    }
    if (d < m.D) out_row<T>(p, a, i)[d] = from_f<T>(sum == 0.f ? 0.f : o / sum);
}

// The four warps' shares of a part joined: into the output where the part is the whole pair, else into the workspace;
// the last block of a pair joins the parts.  buf: the warps' sums [kWarps][T][Dp]; bml: [kWarps][T][2].
template <typename T, bool W>
__device__ __forceinline__ void join(const PagedAttnParams& p, const Part& a, float* buf, float* bml, int share, int64_t tile0)
{
    __shared__ int last, again;
    const PagedParams& m = p.n.m;
    const int Tq = p.n.T, D = m.D, tid = threadIdx.x;
    if (tid == 0) again = 0;
    __syncthreads();
    const bool whole = a.t0 == 0 && a.t1 == a.tiles;
    const int slot = 2 * static_cast<int>(blockIdx.x) + (a.t0 == 0 ? 1 : 0);
    // (unused rows of buf hold what was there; only queries i < n are touched)
    for (int x = tid; x < a.n * D; x += kThreads) {
        const int i = x / D, d = x - i * D;
        float top = kNone;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) top = fmaxf(top, bml[(w * Tq + i) * 2]);
        const float base = finite_or_0(top);
        float y = 0.f, l = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            const float f = exp2f(bml[(w * Tq + i) * 2] - base);
            y = fmaf(f, buf[(w * Tq + i) * p.Dp + d], y);
            l = fmaf(f, bml[(w * Tq + i) * 2 + 1], l);
        }
        if (whole) {
            const float v = l == 0.f ? 0.f : y / l;
            out_row<T>(p, a, i)[d] = from_f<T>(v);
            if (!isfinite(y) || !isfinite(l)) atomicOr(&again, 1 << i);
            if (W && d == 0) p.lse[(static_cast<int64_t>(a.b) * m.H + a.h) * Tq + i] = base + log2f(l);
        } else {
            p.part[(static_cast<int64_t>(slot) * Tq + i) * p.Dp + d] = y;
            if (d == 0) {
                p.ml[(slot * Tq + i) * 2] = top;
                p.ml[(slot * Tq + i) * 2 + 1] = l;
            }
        }
    }
    if (!whole) {
        // blocks first .. first + n - 1 hold the pair's parts
        const int64_t begin = tile0, end = tile0 + a.tiles;
        const int first = static_cast<int>(begin / share), n = static_cast<int>((end - 1) / share) - first + 1;
        __threadfence();
        __syncthreads();
        if (tid == 0) last = atomicAdd(p.tickets + a.b * m.H + a.h, 1) == n - 1;
        __syncthreads();
        if (last) {
            __threadfence();
            const int warp = tid >> 5, lane = tid & 31;
            auto slot_of = [&](int c) { return 2 * (first + c) + (begin >= static_cast<int64_t>(first + c) * share ? 1 : 0); };
            for (int i = 0; i < a.n; ++i) {
                // every warp takes each fourth part; the maximum of all first
                float top = kNone;
                for (int c = lane; c < n; c += 32) top = fmaxf(top, __ldcg(p.ml + (slot_of(c) * Tq + i) * 2));
#pragma unroll
                for (int d = 16; d; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
                const float base = finite_or_0(top);
                float y[4] = {0.f, 0.f, 0.f, 0.f}, l = 0.f;
                for (int c0 = warp; c0 < n; c0 += 32 * kWarps) {
                    const int mine = c0 + kWarps * lane;
                    float f = 0.f;
                    if (mine < n) {
                        const float2 s = __ldcg(reinterpret_cast<const float2*>(p.ml + (slot_of(mine) * Tq + i) * 2));
                        f = exp2f(s.x - base);
                        l = fmaf(f, s.y, l);
                    }
                    const int here = min(32, (n - c0 + kWarps - 1) / kWarps);
#pragma unroll 4
                    for (int z = 0; z < here; ++z) {
                        const float w = __shfl_sync(0xffffffffu, f, z);
                        const float* src = p.part + (static_cast<int64_t>(slot_of(c0 + kWarps * z)) * Tq + i) * p.Dp;
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            if (32 * k + lane < D) y[k] = fmaf(w, __ldcg(src + 32 * k + lane), y[k]);
                    }
                }
#pragma unroll
                for (int d = 16; d; d >>= 1) l += __shfl_xor_sync(0xffffffffu, l, d);
                __syncthreads();
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    if (32 * k + lane < D) buf[warp * p.Dp + 32 * k + lane] = y[k];
                if (lane == 0) bml[warp] = l;
                __syncthreads();
                const float total = bml[0] + bml[1] + bml[2] + bml[3];
                for (int d = tid; d < D; d += kThreads) {
                    const float v = buf[d] + buf[p.Dp + d] + buf[2 * p.Dp + d] + buf[3 * p.Dp + d];
                    out_row<T>(p, a, i)[d] = from_f<T>(total == 0.f ? 0.f : v / total);
                    if (!isfinite(v) || !isfinite(total)) atomicOr(&again, 1 << i);
                }
                if (W && tid == 0) p.lse[(static_cast<int64_t>(a.b) * m.H + a.h) * Tq + i] = base + log2f(total);
            }
        }
    }
    __syncthreads();
    for (int bits = again; bits; bits &= bits - 1) row_again<T>(p, a, __ffs(bits) - 1, buf);
    __syncthreads();
}

// Blocks of the attention that an SM holds: what the registers of the variants leave room for.
template <typename T, int NC, int NQ> constexpr int kBlocks = sizeof(T) == 4 ? (NQ == 1 ? (NC <= 2 ? 4 : 3) : 2) : NC <= 2 && NQ == 1 ? 4 : NC == 1 ? 3 : 2;

// Shared memory: the pairs' first tiles [B + 1] (64 bits), then the warps' sums.
template <typename T, int NC, int NQ, bool W>
__global__ void __launch_bounds__(kThreads, (kBlocks<T, NC, NQ>)) paged_attn_kernel(const __grid_constant__ PagedAttnParams p)
{
    extern __shared__ __align__(16) int64_t start[];
    __shared__ int64_t scan[kWarps];
    const PagedParams& m = p.n.m;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int n_start = (m.B + 2) & ~1;                        // keeps what follows 16-byte aligned
    float* buf = reinterpret_cast<float*>(start + n_start);
    float* bml = buf + kWarps * p.n.T * p.Dp;
    float* qs = bml + kWarps * p.n.T * 2;
    pdl_wait();
    pdl_launch_dependents();

    // start[b]: tiles of all pairs of the sequences before b
    int64_t done = 0;
    for (int b0 = 0; b0 < m.B; b0 += kThreads) {
        const int b = b0 + tid;
        int64_t x = 0;
        if (b < m.B) {
            const int4 now = p.now[b];
            x = now.z > 0 ? static_cast<int64_t>((now.x + kPageUnit - 1) / kPageUnit) * m.H : 0;
            // this call's positions count from now on (nothing below reads the memory's own numbers)
            if (blockIdx.x == 0 && p.n.xk && now.z > 0) {
                m.length[b] = now.x;
                m.next_pos[b] = now.y + now.z;
            }
        }
        int64_t s = x;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int64_t y = __shfl_up_sync(0xffffffffu, s, d);
            if (lane >= d) s += y;
        }
        if (lane == 31) scan[warp] = s;
        __syncthreads();
        int64_t before = done;
        for (int w = 0; w < warp; ++w) before += scan[w];
        if (b < m.B) start[b] = before + s - x;
        for (int w = 0; w < kWarps; ++w) done += scan[w];
        __syncthreads();
    }
    if (tid == 0) start[m.B] = done;
    __syncthreads();
    const int share = static_cast<int>(max(static_cast<int64_t>(kMinTiles), (done + gridDim.x - 1) / gridDim.x));
    // queries of an empty memory: nothing to see
    for (int b = blockIdx.x; b < m.B; b += gridDim.x) {
        const int4 now = p.now[b];
        if (now.z > 0 && now.x == 0)
            for (int x = tid; x < now.z * m.H * m.D; x += kThreads) {
                const int i = x / (m.H * m.D), h = x / m.D % m.H, d = x % m.D;
                static_cast<T*>(p.out)[b * p.o_sb + i * p.o_st + h * p.o_sh + d] = from_f<T>(0.f);
            }
    }
    int64_t at = static_cast<int64_t>(blockIdx.x) * share;
    const int64_t end = min(done, at + share);
    if (at >= end) return;
    int lo = 0, hi = m.B;                                      // start[lo] <= at < start[hi]
    while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (start[mid] <= at) lo = mid; else hi = mid;
    }
    int b = lo;
    while (at < end) {
        while (start[b + 1] <= at) ++b;
        const int4 now = p.now[b];
        Part a;
        a.b = b;
        a.len = now.x;
        a.first = now.y;
        a.n = now.z;
        a.tiles = (now.x + kPageUnit - 1) / kPageUnit;
        const int64_t x = at - start[b];
        a.h = static_cast<int>(x / a.tiles);
        a.t0 = static_cast<int>(x - static_cast<int64_t>(a.h) * a.tiles);
        a.t1 = static_cast<int>(min(static_cast<int64_t>(a.tiles), a.t0 + (end - at)));
        if constexpr (sizeof(T) == 4) part_f32<NC, NQ, W>(p, a, buf, bml, qs);
        else part_bf16<NC, NQ, W>(p, a, buf, bml);
        join<T, W>(p, a, buf, bml, share, start[b] + static_cast<int64_t>(a.h) * a.tiles);
        at += a.t1 - a.t0;
    }
}

// ---------------------------------------------------------------- attention weights
__global__ void __launch_bounds__(kThreads) paged_weight_kernel(const __grid_constant__ PagedAttnParams p)
{
    pdl_wait();
    pdl_launch_dependents();
    const PagedParams& m = p.n.m;
    const int b = blockIdx.y, s = blockIdx.x * kThreads + threadIdx.x;
    const int4 now = p.now[b];
    if (s >= now.x || now.z == 0) return;
    const int page = page_of(m, b, s);
    if (page < 0) return;
    float sum = 0.f;
    for (int h = 0; h < m.H; ++h) {
        const int64_t row = (static_cast<int64_t>(b) * m.H + h) * p.n.T;
        for (int i = 0; i < now.z; ++i) {
            const float x = p.S[(row + i) * p.cap + s];
            if (x != kNone) sum += exp2f(x - p.lse[row + i]);
        }
    }
    m.weight[static_cast<int64_t>(page) * m.page_len + s % m.page_len] += sum;
}

size_t attn_smem(const PagedAttnParams& p, int f32_queries)
{
    return static_cast<size_t>((p.n.m.B + 2) & ~1) * 8 +
           static_cast<size_t>(kWarps) * p.n.T * (p.Dp + 2) * 4 + static_cast<size_t>(f32_queries) * p.Dp * 4;
}

template <typename T, int NC, int NQ>
cudaError_t launch(const PagedAttnParams& p, int sm_count, cudaStream_t s)
{
    static OncePerDevice once;
    const PagedParams& m = p.n.m;
    const size_t smem = attn_smem(p, sizeof(T) == 4 ? NQ : 0);
    cudaError_t e = allow_smem(once, 120 * 1024, paged_attn_kernel<T, NC, NQ, false>, paged_attn_kernel<T, NC, NQ, true>);
    if (e != cudaSuccess) return e;
    const int64_t terms = static_cast<int64_t>((p.n_e + kPrepRows - 1) / kPrepRows) * m.H * ((static_cast<int64_t>(m.B) * p.n.T + 7) / 8);
    if (terms + m.B > INT32_MAX) return cudaErrorInvalidConfiguration;
    e = launch_dependent(paged_prep_kernel<T, NC>, dim3(static_cast<unsigned>(m.B + terms)), dim3(kThreads), 0, s, p);
    if (e != cudaSuccess) return e;
    const int blocks = min(kBlocks<T, NC, NQ> * sm_count, kPagedMaxCtas);
    if (!p.accumulate) return launch_dependent(paged_attn_kernel<T, NC, NQ, false>, dim3(blocks), dim3(kThreads), smem, s, p);
    e = launch_dependent(paged_attn_kernel<T, NC, NQ, true>, dim3(blocks), dim3(kThreads), smem, s, p);
    if (e != cudaSuccess) return e;
    return launch_dependent(paged_weight_kernel, dim3((p.cap + kThreads - 1) / kThreads, m.B), dim3(kThreads), 0, s, p);
}

template <typename T, int NC>
cudaError_t by_queries(const PagedAttnParams& p, int sm_count, cudaStream_t s)
{
    // bf16: groups of eight queries; fp32: queries whose sums fit the registers
    if constexpr (sizeof(T) == 4) return p.n.T == 1 ? launch<T, NC, 1>(p, sm_count, s) : launch<T, NC, NC <= 2 ? 4 : 2>(p, sm_count, s);
    else return p.n.T <= 8 ? launch<T, NC, 1>(p, sm_count, s) : launch<T, NC, 2>(p, sm_count, s);
}

template <typename T>
cudaError_t by_channels(const PagedAttnParams& p, int sm_count, cudaStream_t s)
{
    switch (p.Dp / 32) {
    case 1: return by_queries<T, 1>(p, sm_count, s);
    case 2: return by_queries<T, 2>(p, sm_count, s);
    case 3: return by_queries<T, 3>(p, sm_count, s);
    default: return by_queries<T, 4>(p, sm_count, s);
    }
}

}  // namespace

cudaError_t launch_paged_attn(const PagedAttnParams& p, txl_dtype dtype, int sm_count, cudaStream_t s)
{
    return dtype == TXL_F32 ? by_channels<float>(p, sm_count, s) : by_channels<__nv_bfloat16>(p, sm_count, s);
}

}  // namespace txl
