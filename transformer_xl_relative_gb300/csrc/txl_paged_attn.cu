// txl_paged_attn.cu -- relative attention of 1 .. 16 new tokens a sequence over a memory held in pages.
//
// Query i of a sequence has position p_i, slot j of its memory position p_j ("跨窗口的相对位置编码" §3; the clamp of
// "TransformerXL 相对位置编码" §2.4), C the last distance with a position term:
//     s_ij = scale [ (q_i+u).k_j + (q_i+v).r_min(p_i - p_j, C) ],  visible iff p_j <= p_i,  out_i = softmax_j(s_ij) V
// and, where asked, weight_j += sum over heads and queries of the softmax.
//
//   paged_prep_kernel    (more than one token, or fp32) new keys and values enter their pages; position terms
//                        E[b][h][i][distance]; what the call works on (lengths, queries' positions) goes to the workspace
//   paged_attn_kernel    the tiles of 16 keys of all (sequence, head) pairs in one line, cut into equal shares: a block
//                        takes a share, and the last block of a pair joins its parts.  One bf16 token a sequence needs no
//                        preparation: each key's row of r is multiplied beside the key, the new key is a part of its own
//   paged_weight_kernel  (accumulate) 2^(score - log-sum-exp) summed over heads and queries
//
// Bound by HBM: K, V and a row of r once a key.  One query over 4096 positions of 8 sequences (H16 D64, 137 MB): 30.5 us, of which
// 21 are the 6.3 TB/s of what further keys add (4096 -> 16384 positions: 403 MB in 64 us) and 9 the schedule (1.5), a part's
// first tile (4.5: positions, then rows) and the join (2.5).  32 ragged sequences with summed weights (232 MB) 46 + 6 us, one
// of 65536 positions with a row of r for each (403 MB) 76, 4 queries 35.8, 16 queries 54, five of d_head 128 over up to 2048
// positions, with summed weights, 25.5.
#include <cuda_bf16.h>

#include "txl_mma.cuh"
#include "txl_paged.cuh"
#include "txl_ptx.cuh"

namespace txl {

namespace {

constexpr int kThreads = 128, kWarps = kThreads / 32;
// A block's work is measured in tiles.  Beginning a pair costs it about as long as kHead tiles take (the chain from the
// table over the first copies to the join), so a pair counts kHead tiles more (32 ragged sequences, kHead 0, 6, 12, 20, 30: 81, 59, 52,
// 50.7, 52 us when this was measured); shares are at least kMinTiles (16: no change), and a pair of up to kWholeTiles goes to one
// block whole (32: no change).
constexpr int kHead = 20, kMinTiles = 8, kWholeTiles = 16;
constexpr float kNone = -INFINITY;

template <typename T> __device__ __forceinline__ float to_f(T x);
template <> __device__ __forceinline__ float to_f<float>(float x) { return x; }
template <> __device__ __forceinline__ float to_f<__nv_bfloat16>(__nv_bfloat16 x) { return __bfloat162float(x); }
template <typename T> __device__ __forceinline__ T from_f(float x);
template <> __device__ __forceinline__ float from_f<float>(float x) { return x; }
template <> __device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }

// Eight bf16 of a row of r from channel d on; channels at and past D are 0.
__device__ __forceinline__ uint4 row_unit(const uint16_t* row, int d, int D, bool vec)
{
    if (vec && d + 8 <= D) return *reinterpret_cast<const uint4*>(row + d);
    uint32_t x[8];
#pragma unroll
    for (int z = 0; z < 8; ++z) x[z] = d + z < D ? row[d + z] : 0u;
    return make_uint4(x[0] | x[1] << 16, x[2] | x[3] << 16, x[4] | x[5] << 16, x[6] | x[7] << 16);
}

// ---------------------------------------------------------------- preparation
// The first B * copies blocks take the sequences' new positions, `share` positions a block, the others position terms: of 8
// queries (of all sequences) and a head with kPrepRows distances.
constexpr int kPrepRows = 128;

template <typename T>
__device__ __forceinline__ void prep_sequence(const PagedAttnParams& p, int b, int part, int share)
{
    const PagedParams& m = p.n.m;
    const int n = paged_count(p.n.counts, b, p.n.T);
    const int len = m.length[b], next = m.next_pos[b];
    int4 now = make_int4(len, next, n, 0);
    if (p.n.xk && n > 0) {
        if (paged_room(m, b, len, n)) {
            const int t0 = part * share, t1 = min(n, t0 + share);
            if (t0 < t1) paged_copy<T>(p.n, b, len, next, t0, t1);
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
    if (threadIdx.x == 0 && part == 0) p.now[b] = now;
}

// bf16: the queries are the 16 rows of the mma's A, row g the upper 8 bits of (q + v) scale and row g + 8 the next 8, so that
// the sum of the two rows' products has 16 bits of the query.  Lane (g, t) loads units t + 4 j of 16 bytes of r's row g as they
// are; the channels' order in A follows.
template <int NC>
__device__ __forceinline__ void prep_terms_bf16(const PagedAttnParams& p, int h, int f0, int d0, const bool* live, uint16_t* qs)
{
    constexpr int kWidth = 32 * NC, kRow = kWidth + 8, kEach = kPrepRows / (8 * kWarps);
    const PagedParams& m = p.n.m;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
    const int T = p.n.T;
    const uint16_t* r = static_cast<const uint16_t*>(p.r) + h * p.r_head;
    uint4 w[kEach][NC];
#pragma unroll
    for (int y = 0; y < kEach; ++y) {
        const uint16_t* row = r + static_cast<int64_t>(min(d0 + (y * kWarps + warp) * 8 + g, p.n_e - 1)) * p.r_row;
#pragma unroll
        for (int j = 0; j < NC; ++j) w[y][j] = row_unit(row, 8 * (t + 4 * j), m.D, p.vec_r);
    }
#pragma unroll
    for (int e = 0; e < 8 * kWidth / kThreads; ++e) {
        const int x = threadIdx.x + e * kThreads, i = x / kWidth, d = x % kWidth, f = f0 + i, b = f / T;
        float y = 0.f;
        if (live[i] && d < m.D)
            y = (__bfloat162float(static_cast<const __nv_bfloat16*>(p.q)[b * p.q_sb + (f - b * T) * p.q_st + h * p.q_sh + d]) + p.vb[h * m.D + d]) * p.qscale;
        const __nv_bfloat16 hi = __float2bfloat16_rn(y);
        qs[i * kRow + d] = __bfloat16_as_ushort(hi);
        qs[(8 + i) * kRow + d] = __bfloat16_as_ushort(__float2bfloat16_rn(y - __bfloat162float(hi)));
    }
    __syncthreads();
    const int f = f0 + g, b = f / T;
    float* E = p.E + ((static_cast<int64_t>(b) * m.H + h) * T + f - b * T) * p.e_pitch;
    float c[kEach][4] = {};
#pragma unroll
    for (int j = 0; j < 2 * NC; ++j) {
        const uint16_t* q = qs + g * kRow + 8 * (t + 4 * (j >> 1)) + 4 * (j & 1);
        const uint2 hi = *reinterpret_cast<const uint2*>(q), lo = *reinterpret_cast<const uint2*>(q + 8 * kRow);
#pragma unroll
        for (int y = 0; y < kEach; ++y) {
            const uint4 u = w[y][j >> 1];
            mma::mma16816(c[y], hi.x, lo.x, hi.y, lo.y, j & 1 ? u.z : u.x, j & 1 ? u.w : u.y);
        }
    }
#pragma unroll
    for (int y = 0; y < kEach; ++y) {
        const int x0 = d0 + (y * kWarps + warp) * 8;
        if (f < m.B * T && x0 < p.n_e) *reinterpret_cast<float2*>(E + x0 + 2 * t) = make_float2(c[y][0] + c[y][2], c[y][1] + c[y][3]);
    }
}

// fp32: a warp takes eight distances at a time; lane (g, t) channels 4 (t + 4 j) .. + 3 of distance g, for eight queries
// whose rows lie in shared memory.
template <int NC>
__device__ __forceinline__ void prep_terms_f32(const PagedAttnParams& p, int h, int f0, int d0, const bool* live, float* q)
{
    constexpr int NJ = 2 * NC, kWidth = 32 * NC;
    const PagedParams& m = p.n.m;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
    const int T = p.n.T, D = m.D, n = min(8, m.B * T - f0);
    for (int x = threadIdx.x; x < 8 * kWidth; x += kThreads) {
        const int e = x / kWidth, d = x % kWidth, f = f0 + e, b = f / T, i = f - b * T;
        q[x] = live[e] && d < D ? (static_cast<const float*>(p.q)[b * p.q_sb + i * p.q_st + h * p.q_sh + d] + p.vb[h * D + d]) * p.qscale : 0.f;
    }
    __syncthreads();
    const float* r = static_cast<const float*>(p.r) + h * p.r_head;
#pragma unroll 1
    for (int x0 = d0 + warp * 8; x0 < min(p.n_e, d0 + kPrepRows); x0 += kWarps * 8) {
        asm volatile("" ::: "memory");                         // (the queries' rows do not fit the registers)
        const int x = x0 + g;
        const float* row = r + static_cast<int64_t>(min(x, p.n_e - 1)) * p.r_row;
        float4 w[NJ];
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
            const int d = 4 * (t + 4 * j);
            if (p.vec_r && d + 4 <= D) w[j] = *reinterpret_cast<const float4*>(row + d);
            else w[j] = make_float4(d < D ? row[d] : 0.f, d + 1 < D ? row[d + 1] : 0.f, d + 2 < D ? row[d + 2] : 0.f, d + 3 < D ? row[d + 3] : 0.f);
        }
        float s[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            s[e] = 0.f;
#pragma unroll
            for (int j = 0; j < NJ; ++j) {
                const float4 y = *reinterpret_cast<const float4*>(q + e * kWidth + 4 * (t + 4 * j));
                s[e] = fmaf(y.w, w[j].w, fmaf(y.z, w[j].z, fmaf(y.y, w[j].y, fmaf(y.x, w[j].x, s[e]))));
            }
            s[e] += __shfl_xor_sync(0xffffffffu, s[e], 1);
            s[e] += __shfl_xor_sync(0xffffffffu, s[e], 2);
        }
        // lane t writes queries t and t + 4
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if ((e & 3) == t && e < n && x < p.n_e) {
                const int f = f0 + e, b = f / T, i = f - b * T;
                p.E[((static_cast<int64_t>(b) * m.H + h) * T + i) * p.e_pitch + x] = s[e];
            }
    }
}

template <typename T, int NC>
__global__ void __launch_bounds__(kThreads) paged_prep_kernel(const __grid_constant__ PagedAttnParams p, int copies, int share)
{
    __shared__ __align__(16) float qs[sizeof(T) == 4 ? 8 * 32 * NC : 8 * (32 * NC + 8)];
    __shared__ int far;
    __shared__ bool live[8];                                   // queries that a sequence has (no others are read)
    pdl_wait();
    pdl_launch_dependents();
    const PagedParams& m = p.n.m;
    if (blockIdx.x < static_cast<unsigned>(m.B * copies)) {
        prep_sequence<T>(p, blockIdx.x / copies, blockIdx.x % copies, share);
        return;
    }
    const int x = blockIdx.x - m.B * copies, parts = (p.n_e + kPrepRows - 1) / kPrepRows;
    const int d0 = x % parts * kPrepRows, h = x / parts % m.H, f0 = x / parts / m.H * 8;
    // distances beyond the start of all of these sequences are not met (next_pos changes in the attention's kernel)
    if (threadIdx.x == 0) far = 0;
    __syncthreads();
    if (threadIdx.x < 8) {
        const int f = f0 + static_cast<int>(threadIdx.x), b = f / p.n.T;
        live[threadIdx.x] = f < m.B * p.n.T && f - b * p.n.T < paged_count(p.n.counts, b, p.n.T);
        if (live[threadIdx.x]) atomicMax(&far, m.next_pos[b] + (p.n.xk ? p.n.T : 0));
    }
    __syncthreads();
    if (d0 >= far) return;
    if constexpr (sizeof(T) == 4) prep_terms_f32<NC>(p, h, f0, d0, live, qs);
    else prep_terms_bf16<NC>(p, h, f0, d0, live, reinterpret_cast<uint16_t*>(qs));
}

// ---------------------------------------------------------------- attention
// a / b where that is an int (64-bit divisions are slow, and most numbers are small).
__device__ __forceinline__ int quotient(int64_t a, int b)
{
    if (static_cast<uint64_t>(a) >> 32 == 0) return static_cast<int>(static_cast<uint32_t>(a) / static_cast<uint32_t>(b));
    return static_cast<int>(a / b);
}

// What a block knows of the part of a (sequence, head) pair that it works on.
struct Part {
    int b, h, len, first, n;       // slots, position of the first query, queries
    int t0, t1, tiles;             // its tiles, of the pair's
    int parts, first_block;        // the pair's parts, and the block of the first
    const int* table;              // the sequence's row of the page table, in shared memory where that holds it
    bool room;                     // the new key has a page (else the sequence is left as it was)
    bool own;                      // the pair has a new key that is not among the slots (k_new, position `first`)
};

// The page of a slot of the part's sequence, or -1.
__device__ __forceinline__ int page_at(const PagedParams& m, const Part& a, int s)
{
    const int i = s / m.page_len;
    if (i >= m.max_pages) return -1;
    const int page = a.table[i];
    return static_cast<unsigned>(page) < static_cast<unsigned>(m.n_pages) ? page : -1;
}

// Where the tiles that a warp will come to lie: lane x knows that of the warp's x-th tile from `base` on (a page's number
// and the row in it take divisions, which are made once in 32 - BACK tiles).  Asked for a tile further on, the lanes look again,
// from BACK tiles of the warp before it on: those stay known.
template <int NW, int BACK> struct Tiles {
    int base, mine;                // first position of the tile in m.pos, or -1 where there is no page
    int64_t mine_kv;               // and its first element of the part's head in m.k and m.v

    __device__ __forceinline__ void look(const PagedParams& m, const Part& a, int tile, int lane)
    {
        base = tile;
        const int at = tile + NW * lane;
        const bool used = at < a.t1 && at * kPageUnit < a.len;
        const int page = used ? page_at(m, a, at * kPageUnit) : -1, row = at * kPageUnit % m.page_len;
        if (used && page < 0) page_error(m);
        mine = page < 0 ? -1 : page * m.page_len + row;
        mine_kv = page < 0 ? -1 : page_row0(m, page, a.h) + static_cast<int64_t>(row) * m.ld;
    }
    // of `tile` (a warp's own; none later than BACK behind it was asked for)
    __device__ __forceinline__ int pos(const PagedParams& m, const Part& a, int tile, int lane)
    {
        if (tile - base >= 32 * NW) look(m, a, tile - BACK * NW, lane);
        return __shfl_sync(0xffffffffu, mine, (tile - base) / NW);
    }
    __device__ __forceinline__ int64_t kv(const PagedParams& m, const Part& a, int tile, int lane)
    {
        if (tile - base >= 32 * NW) look(m, a, tile - BACK * NW, lane);
        return __shfl_sync(0xffffffffu, mine_kv, (tile - base) / NW);
    }
};

// Index of the position term of a query at `at` and a key at pos <= at.
__device__ __forceinline__ int term(const PagedAttnParams& p, int at, int pos)
{
    return static_cast<int>(min(static_cast<unsigned>(at) - static_cast<unsigned>(pos), static_cast<unsigned>(p.n_e - 1)));
}

// The scores of a query of a sequence and head, and the place in them of slot s, which lies at `at` in m.pos.  (All sequences' slots
// are the pool's: a table whose rows could each hold the pool takes no more room for scores than the pool has slots.)
__device__ __forceinline__ float* score_row(const PagedAttnParams& p, int b, int h, int i)
{
    return p.S + (static_cast<int64_t>(h) * p.n.T + i) * p.s_slots + (p.s_pool ? 0 : b * p.cap);
}
__device__ __forceinline__ int score_slot(const PagedAttnParams& p, int s, int at) { return p.s_pool ? at : s; }

__device__ __forceinline__ float finite_or_0(float m) { return m == kNone ? 0.f : m; }

// bf16.  A warp takes every NW-th tile of 16 keys through its own ring of stages in shared memory: asynchronous copies
// of 16 bytes, one or two tiles ahead.  What lies past a sequence's last slot, or past D, arrives as zeros.  Rows are an odd
// number of 16-byte units apart, so that the eight rows of an ldmatrix lie in different banks.
template <int NC> constexpr int kStages = NC == 1 ? 3 : 2;              // (a third stage gains nothing: 16 warps of an SM copy)
template <int NC> constexpr int kPitch = (4 * NC + 1) * 16;               // bytes
template <int NC> constexpr int kStage = 2 * kPageUnit * kPitch<NC>;      // K and V of a tile
template <int NC> constexpr int kWarpBytes = kStages<NC> * kStage<NC>;

__device__ __forceinline__ void copy16(uint32_t dst, const void* src, int bytes)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
// An 8 x 8 matrix of 16-bit elements, two of row lane / 4 in each lane, transposed.
__device__ __forceinline__ uint32_t transpose8(uint32_t x)
{
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
template <int N> __device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// Products: keys are the 16 rows of the mma's A, as ldmatrix brings them, and columns 2 i, 2 i + 1 of its B hold query i
// twice: the upper 8 bits of (q + u) scale, and the next 8.  Lane (g, t) then has both for query 4 x + t and keys g and g + 8,
// and, with the values transposed as A and the weights split likewise as B, the same query's sums of channels g and g + 8 of
// each 16: everything that belongs to a query stays in its lanes.
// ONE (one token): (q + v).r of each key's own distance joins the sums, with r's rows as A (each lane loads units t, t + 4,
// .. of two rows: their channels' order is that of qv).  Otherwise the terms come from E.
template <int NC> struct BFrag { uint32_t w[2 * NC][2]; };

// The part's queries in shared memory as the columns of B want them, by the whole block: row 2 i the upper 8 bits of (q_i + u)
// scale, row 2 i + 1 the next 8; with ONE rows 8 and 9 are for v, and the other rows stay zero.  Rows of kQPitch
// bf16 (in different banks), zeros past D and from query n on.
template <int NC> constexpr int kQPitch = 32 * NC + 8;
template <int NC, int NQ, bool ONE> constexpr int kQRows = ONE ? 16 : 8 * NQ;

// The elements that a thread puts there: loaded before anything that waits, stored later.
template <int NC, int NQ, bool ONE, int NW> struct Queries {
    static constexpr int kWidth = 32 * NC, kRows = ONE ? 2 : 4 * NQ, kEach = (kRows * kWidth + 32 * NW - 1) / (32 * NW);
    float y[kEach];

    __device__ __forceinline__ void load(const PagedAttnParams& p, const Part& a)
    {
        const PagedParams& m = p.n.m;
#pragma unroll
        for (int e = 0; e < kEach; ++e) {
            const int x = threadIdx.x + e * (32 * NW), row = x / kWidth, d = x % kWidth, i = ONE ? 0 : row;
            y[e] = 0.f;
            if (row < kRows && i < a.n && d < m.D)
                y[e] = (__bfloat162float(static_cast<const __nv_bfloat16*>(p.q)[a.b * p.q_sb + i * p.q_st + a.h * p.q_sh + d]) +
                        (ONE && row ? p.vb : p.u)[a.h * m.D + d]) * p.qscale;
        }
    }
    __device__ __forceinline__ void store(uint16_t* qs) const
    {
#pragma unroll
        for (int e = 0; e < kEach; ++e) {
            const int x = threadIdx.x + e * (32 * NW), row = ONE ? x / kWidth * 8 : x / kWidth * 2, d = x % kWidth;
            if (x >= kRows * kWidth) continue;
            const __nv_bfloat16 hi = __float2bfloat16_rn(y[e]);
            qs[row * kQPitch<NC> + d] = __bfloat16_as_ushort(hi);
            qs[(row + 1) * kQPitch<NC> + d] = __bfloat16_as_ushort(__float2bfloat16_rn(y[e] - __bfloat162float(hi)));
        }
    }
};

// ROWS: in the order of the units of r's rows.
template <int NC, bool ROWS>
__device__ __forceinline__ void load_b(BFrag<NC>& f, const uint16_t* row, int t)
{
#pragma unroll
    for (int j = 0; j < 2 * NC; ++j)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int d = ROWS ? 8 * (t + 4 * (j >> 1)) + 4 * (j & 1) + 2 * e : 16 * j + 8 * e + 2 * t;
            f.w[j][e] = *reinterpret_cast<const uint32_t*>(row + d);
        }
}

// ONE: a pair's new key, by one warp: its score, its values as a part of one key, and its row into the page (which the
// sequence may lack: then nothing is written).  Loaded before anything that waits, worked on later.
template <int NC, bool W> struct OwnKey {
    float s;
    uint16_t k[NC], v[NC];
    int page;

    __device__ __forceinline__ void load(const PagedAttnParams& p, const Part& a, int lane)
    {
        const PagedParams& m = p.n.m;
        const __nv_bfloat16* qr = static_cast<const __nv_bfloat16*>(p.q) + a.b * p.q_sb + a.h * p.q_sh;
        const uint16_t* kr = static_cast<const uint16_t*>(p.n.xk) + a.b * p.n.xk_sb + a.h * p.n.xk_sh;
        const uint16_t* vr = static_cast<const uint16_t*>(p.n.xv) + a.b * p.n.xv_sb + a.h * p.n.xv_sh;
        const __nv_bfloat16* r = static_cast<const __nv_bfloat16*>(p.r) + a.h * p.r_head;
        page = page_at(m, a, a.len);
        s = 0.f;
#pragma unroll
        for (int j = 0; j < NC; ++j) {
            const int d = lane + 32 * j;
            k[j] = v[j] = 0;
            if (d < m.D) {
                const float x = __bfloat162float(qr[d]);
                k[j] = kr[d];
                v[j] = vr[d];
                s = fmaf((x + p.u[a.h * m.D + d]) * p.qscale, mma::bf16_lo(k[j]), s);
                s = fmaf((x + p.vb[a.h * m.D + d]) * p.qscale, __bfloat162float(r[d]), s);
            }
        }
    }
    __device__ __forceinline__ void store(const PagedAttnParams& p, const Part& a, int lane, float* values, float* bml)
    {
        const PagedParams& m = p.n.m;
        const int row = a.len % m.page_len;
        const int64_t at = page >= 0 ? page_row0(m, page, a.h) + static_cast<int64_t>(row) * m.ld : 0;
#pragma unroll
        for (int j = 0; j < NC; ++j) {
            const int d = lane + 32 * j;
            if (d < m.D) values[d] = mma::bf16_lo(v[j]);
            if (page >= 0 && d < m.ld) {
                static_cast<uint16_t*>(m.k)[at + d] = k[j];
                static_cast<uint16_t*>(m.v)[at + d] = v[j];
            }
        }
        for (int d = lane + 32 * NC; page >= 0 && d < m.ld; d += 32)
            static_cast<uint16_t*>(m.k)[at + d] = static_cast<uint16_t*>(m.v)[at + d] = 0;
#pragma unroll
        for (int d = 16; d; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
        if (lane) return;
        bml[0] = s;
        bml[1] = s != s ? s : s == kNone ? 0.f : 1.f;
        if (page < 0) {
            page_error(m);
            return;
        }
        if (W) score_row(p, a.b, a.h, 0)[score_slot(p, a.len, page * m.page_len + row)] = s;
        if (a.h == 0) {
            m.pos[static_cast<int64_t>(page) * m.page_len + row] = a.first;
            m.weight[static_cast<int64_t>(page) * m.page_len + row] = 0.f;
        }
    }
};

template <int NC, int NQ, bool ONE, bool W, int NW>
__device__ __forceinline__ void part_bf16(const PagedAttnParams& p, const Part& a, char* ring, float* bml, float* own, uint16_t* qs)
{
    const PagedParams& m = p.n.m;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
    const int T = p.n.T;
    const uint32_t stage0 = smem_u32(ring);

    // a lane's pieces of a tile: a unit of 16 bytes of every kSide-th row of K and of V (a unit wholly past D is never copied, and
    // zero from the start)
    constexpr int kUnits = 4 * NC, kSide = 32 / kUnits, kPieces = kPageUnit / kSide;
    const int units = (m.D + 7) / 8, my_row = lane / kUnits, my_unit = lane % kUnits;
    const bool copies = my_row < kSide && my_unit < units;
    const int bytes = min(16, 2 * (m.D - 8 * my_unit)), from = 2 * (my_row * m.ld + 8 * my_unit), step = 2 * kSide * m.ld;
    const uint32_t into = stage0 + my_row * kPitch<NC> + 16 * my_unit;
    auto copy = [&](int64_t at, int tile, int stage) {
        if (!copies) return;
        const int rows = at < 0 ? 0 : a.len - tile * kPageUnit;            // that hold something
        const int64_t off = 2 * max(at, static_cast<int64_t>(0));
        const char* k = static_cast<const char*>(m.k) + off;
        const char* v = static_cast<const char*>(m.v) + off;
        const uint32_t dst = into + stage * kStage<NC>;
        if (rows >= kPageUnit) {
            k += from;
            v += from;
#pragma unroll
            for (int j = 0; j < kPieces; ++j) {
                copy16(dst + j * kSide * kPitch<NC>, k + j * step, bytes);
                copy16(dst + (kPageUnit + j * kSide) * kPitch<NC>, v + j * step, bytes);
            }
        } else {
#pragma unroll
            for (int j = 0; j < kPieces; ++j) {
                const bool held = my_row + j * kSide < rows;
                copy16(dst + j * kSide * kPitch<NC>, held ? k + from + j * step : k, held ? bytes : 0);
                copy16(dst + (kPageUnit + j * kSide) * kPitch<NC>, held ? v + from + j * step : v, held ? bytes : 0);
            }
        }
    };
    // what hangs on nothing is loaded first, then the pages, then what they lead to
    Queries<NC, NQ, ONE, NW> queries;
    queries.load(p, a);
    OwnKey<NC, W> own_key;
    const bool owner = ONE && a.own && a.t1 == a.tiles && warp == NW - 1;
    if constexpr (ONE)
        if (owner) own_key.load(p, a, lane);
    Tiles<NW, W ? 2 : 0> tiles;                                // (two tiles ahead of the one whose scores are written)
    tiles.look(m, a, a.t0 + warp, lane);
    if (units < kUnits) {
        for (int x = lane; x < kStages<NC> * 2 * kPageUnit * (kUnits - units); x += 32) {
            const int row = x / (kUnits - units), c = units + x % (kUnits - units);
            *reinterpret_cast<uint4*>(ring + row * kPitch<NC> + 16 * c) = make_uint4(0, 0, 0, 0);
        }
    }
    const int first = a.t0 + warp;
    if (!ONE && p.n.xk && a.t1 * kPageUnit > a.len - a.n) pdl_wait();      // new keys are among them
#pragma unroll
    for (int x = 0; x < kStages<NC> - 1; ++x) {
        const int tile = first + x * NW;
        if (tile < a.t1) copy(tiles.kv(m, a, tile, lane), tile, x);
        mma::cp_async_commit();
    }
    // positions of keys g and g + 8, two tiles ahead (a slot that holds nothing is ahead of every query)
    constexpr int kAhead = 0x7fffffff;
    int pos[2];
    auto load_pos = [&](int tile) {
        const int at = tiles.pos(m, a, tile, lane);
#pragma unroll
        for (int y = 0; y < 2; ++y) pos[y] = at >= 0 && tile * kPageUnit + 8 * y + g < a.len ? m.pos[at + 8 * y + g] : kAhead;
    };
    if (first < a.t1) load_pos(first);
    queries.store(qs);
    if (!ONE) pdl_wait();                                      // E is there
    if constexpr (ONE)
        if (owner) own_key.store(p, a, lane, own, bml + 2 * NW);

    // what a tile's position terms come from, one tile ahead: which keys a lane's query sees, E's terms (e) or r's rows (rw)
    float e[NQ][2];
    uint4 rw[2][NC];
    const float* E[NQ];
    bool live[NQ];
#pragma unroll
    for (int x = 0; x < NQ; ++x) {
        live[x] = 4 * x + t < a.n;
        E[x] = ONE ? nullptr : p.E + ((static_cast<int64_t>(a.b) * m.H + a.h) * T + min(4 * x + t, T - 1)) * p.e_pitch;
    }
    const uint16_t* r = static_cast<const uint16_t*>(p.r) + a.h * p.r_head;
    const int r_row = static_cast<int>(p.r_row);
    const bool whole_rows = p.vec_r && m.D == 32 * NC;
    auto load_row = [&](int distance, uint4* w) {
        const uint16_t* row = r + static_cast<int64_t>(distance) * r_row;
        if (whole_rows) {
#pragma unroll
            for (int j = 0; j < NC; ++j) w[j] = *reinterpret_cast<const uint4*>(row + 8 * t + 32 * j);
        } else {
#pragma unroll
            for (int j = 0; j < NC; ++j) w[j] = row_unit(row, 8 * (t + 4 * j), m.D, p.vec_r);
        }
    };
    auto load_terms = [&]() {
#pragma unroll
        for (int x = 0; x < NQ; ++x)
#pragma unroll
            for (int y = 0; y < 2; ++y) {
                const int at = a.first + 4 * x + t;
                const bool seen = live[x] && pos[y] <= at;
                if constexpr (ONE) e[x][y] = seen ? 0.f : kNone;
                else e[x][y] = seen ? E[x][term(p, at, pos[y])] : kNone;
            }
        if constexpr (ONE) {
            load_row(term(p, a.first, min(pos[0], a.first)), rw[0]);
            load_row(term(p, a.first, min(pos[1], a.first)), rw[1]);
        }
    };
    if (first < a.t1) {
        load_terms();
        if (first + NW < a.t1) load_pos(first + NW);
    }
    __syncthreads();

    BFrag<NC> q[NQ], qv;
#pragma unroll
    for (int x = 0; x < NQ; ++x) load_b<NC, false>(q[x], qs + (8 * x + g) * kQPitch<NC>, t);
    float* S = W ? score_row(p, a.b, a.h, t) + g : nullptr;    // (of query t, if there is one)
    if (ONE) load_b<NC, true>(qv, qs + (8 + g) * kQPitch<NC>, t);
    float o[NQ][2 * NC][4];
    float mx[NQ], sum[NQ];
#pragma unroll
    for (int x = 0; x < NQ; ++x) {
        mx[x] = kNone;
        sum[x] = 0.f;
#pragma unroll
        for (int z = 0; z < 2 * NC; ++z) o[x][z][0] = o[x][z][1] = o[x][z][2] = o[x][z][3] = 0.f;
    }
    // ldmatrix addresses in a stage: K as [key][channel], V as [key][channel] transposed
    const uint32_t k_at = stage0 + (lane & 15) * kPitch<NC> + (lane >> 4) * 16;
    const uint32_t v_at = stage0 + (kPageUnit + (lane & 7) + (lane >> 4) * 8) * kPitch<NC> + ((lane >> 3) & 1) * 16;
    int stage = 0, ahead = kStages<NC> - 1;
    for (int tile = first; tile < a.t1; tile += NW) {
        copies_wait<kStages<NC> - 2>();
        __syncwarp();                                          // everyone's pieces are here, and the last stage is read
        if (tile + (kStages<NC> - 1) * NW < a.t1) {
            const int to = tile + (kStages<NC> - 1) * NW;
            copy(tiles.kv(m, a, to, lane), to, ahead);
        }
        mma::cp_async_commit();
        ahead = stage;
        const uint32_t off = stage * kStage<NC>;
        stage = stage + 1 == kStages<NC> ? 0 : stage + 1;

        float c[NQ][4] = {};
#pragma unroll
        for (int j = 0; j < 2 * NC; ++j) {
            uint32_t w[4];
            mma::ldsm_x4(k_at + off + 32 * j, w[0], w[1], w[2], w[3]);
#pragma unroll
            for (int x = 0; x < NQ; ++x) mma::mma16816(c[x], w[0], w[1], w[2], w[3], q[x].w[j][0], q[x].w[j][1]);
        }
        if (ONE) {
#pragma unroll
            for (int j = 0; j < NC; ++j) {
                mma::mma16816(c[0], rw[0][j].x, rw[1][j].x, rw[0][j].y, rw[1][j].y, qv.w[2 * j][0], qv.w[2 * j][1]);
                mma::mma16816(c[0], rw[0][j].z, rw[1][j].z, rw[0][j].w, rw[1][j].w, qv.w[2 * j + 1][0], qv.w[2 * j + 1][1]);
            }
        }
        float s[NQ][2];
#pragma unroll
        for (int x = 0; x < NQ; ++x)
#pragma unroll
            for (int y = 0; y < 2; ++y) s[x][y] = e[x][y] == kNone ? kNone : c[x][2 * y] + c[x][2 * y + 1] + e[x][y];
        if (tile + NW < a.t1) {
            load_terms();
            if (tile + 2 * NW < a.t1) load_pos(tile + 2 * NW);
        }
        // the maximum follows only where a score is far above it: a weight may be up to 2^kSlack
        constexpr float kSlack = 8.f;
        bool grows = false;
#pragma unroll
        for (int x = 0; x < NQ; ++x) grows |= fmaxf(s[x][0], s[x][1]) > mx[x] + kSlack;
        if (__any_sync(0xffffffffu, grows)) {
#pragma unroll
            for (int x = 0; x < NQ; ++x) {
                float top = fmaxf(s[x][0], s[x][1]);
#pragma unroll
                for (int d = 4; d < 32; d <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
                const float now = fmaxf(mx[x], top), f = mma::ex2(mx[x] - finite_or_0(now));
                mx[x] = now;
                sum[x] *= f;
#pragma unroll
                for (int z = 0; z < 2 * NC; ++z)
#pragma unroll
                    for (int y = 0; y < 4; ++y) o[x][z][y] *= f;
            }
        }
        if constexpr (W) {
            const int slot = p.s_pool ? tiles.pos(m, a, tile, lane) : tile * kPageUnit;
#pragma unroll
            for (int x = 0; x < NQ; ++x)
                if (live[x] && slot >= 0) {
                    // (not behind the last slot: that is the new key's)
                    float* to = S + static_cast<int64_t>(4 * x) * p.s_slots + slot;
                    if (tile * kPageUnit + g < a.len) to[0] = s[x][0];
                    if (tile * kPageUnit + 8 + g < a.len) to[8] = s[x][1];
                }
        }
        uint32_t b0[NQ], b1[NQ];
#pragma unroll
        for (int x = 0; x < NQ; ++x) {
            const float base = finite_or_0(mx[x]);
            const float p0 = mma::ex2(s[x][0] - base), p1 = mma::ex2(s[x][1] - base);
            sum[x] += p0 + p1;
            // rows of keys with a query's weight in two columns (its upper 8 bits, the next 8), transposed into the fragment
            const uint32_t hi = mma::pack2(p0, p1);
            const float h0 = mma::bf16_lo(hi), h1 = mma::bf16_hi(hi);
            b0[x] = transpose8(mma::pack2(h0, p0 - h0));
            b1[x] = transpose8(mma::pack2(h1, p1 - h1));
        }
#pragma unroll
        for (int z = 0; z < 2 * NC; ++z) {
            uint32_t w[4];
            mma::ldsm_x4_t(v_at + off + 32 * z, w[0], w[1], w[2], w[3]);
#pragma unroll
            for (int x = 0; x < NQ; ++x) mma::mma16816(o[x][z], w[0], w[1], w[2], w[3], b0[x], b1[x]);
        }
    }
    __syncwarp();                                              // the ring is read: it takes the warp's sums
#pragma unroll
    for (int x = 0; x < NQ; ++x) {
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) sum[x] += __shfl_xor_sync(0xffffffffu, sum[x], d);
        if (!live[x]) continue;
        const int i = 4 * x + t;
        if (g == 0) {
            bml[(warp * T + i) * 2] = mx[x];
            bml[(warp * T + i) * 2 + 1] = sum[x];
        }
        float* row = reinterpret_cast<float*>(ring) + i * (32 * NC) + g;
#pragma unroll
        for (int z = 0; z < 2 * NC; ++z) {
            row[16 * z] = o[x][z][0] + o[x][z][1];
            row[16 * z + 8] = o[x][z][2] + o[x][z][3];
        }
    }
}

// fp32, CUDA cores.  A warp takes its tiles by halves of 8 keys through a ring of its own; lane (g, t) takes key g and channels
// 4 (t + 4 j) .. + 3; each of the eight g keeps maximum and sums of its own, which meet at the end.  NQ queries at a time: their
// sums stay in registers, and their chains of instructions run beside one another.  Rows are 16 floats more than their
// channels apart: two rows' units of four lanes lie in different banks.  A key that a query does not see has weight 0; if its
// value is not finite, row_again computes the row.  Bound by shared memory and the chains of a half (B8 H16 D64 over 2048
// positions: one query 44 us, 4 queries 52, 16 queries 173; with rows loaded into registers one half ahead, query after query, 45,
// 62 and 226).
constexpr int kHalf = kPageUnit / 2;
template <int NC> constexpr int kHalfStages = NC <= 2 ? 3 : 2;
template <int NC> constexpr int kHalfPitch = 32 * NC + 16;                // floats
template <int NC> constexpr int kHalfStage = 2 * kHalf * kHalfPitch<NC>;  // K and V of half a tile
template <int NC, int NQ, bool W, int NW>
__device__ __forceinline__ void part_f32(const PagedAttnParams& p, const Part& a, float* buf, int share, float* bml, float* qs)
{
    constexpr int NJ = 2 * NC;             // chunks of four channels of a lane
    const PagedParams& m = p.n.m;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
    const int T = p.n.T, D = m.D;
    float* ring = buf + NW * share + warp * (kHalfStages<NC> * kHalfStage<NC>);
    // units of 16 bytes that lie past D wholly are never copied
    constexpr int kUnits = 8 * NC, kPieces = kHalf * kUnits / 32;
    for (int x = lane; x < kHalfStages<NC> * 2 * kHalf * kUnits; x += 32)
        if (x % kUnits * 4 >= D) *reinterpret_cast<float4*>(ring + x / kUnits * kHalfPitch<NC> + x % kUnits * 4) = make_float4(0.f, 0.f, 0.f, 0.f);
    pdl_wait();
    for (int i0 = 0; i0 < a.n; i0 += NQ) {
        __syncthreads();
        for (int x = threadIdx.x; x < NQ * p.Dp; x += (32 * NW)) {
            const int i = i0 + x / p.Dp, d = x % p.Dp;
            qs[x] = i < a.n && d < D ? (static_cast<const float*>(p.q)[a.b * p.q_sb + i * p.q_st + a.h * p.q_sh + d] + p.u[a.h * D + d]) * p.qscale : 0.f;
        }
        // u / 2 is the warp's tile, u % 2 its half.  Keys and values are copied two halves ahead, positions loaded two, position
        // terms one.
        Tiles<NW, 0> tiles;
        tiles.look(m, a, a.t0 + warp, lane);
        const int halves = a.t0 + warp < a.t1 ? 2 * ((a.t1 - a.t0 - warp + NW - 1) / NW) : 0;
        constexpr int kAhead = 0x7fffffff;                     // a slot that holds nothing is ahead of every query
        auto tile_of = [&](int u) { return a.t0 + warp + u / 2 * NW; };
        auto copy = [&](int u, int stage) {
            const int64_t at = tiles.kv(m, a, tile_of(u), lane);
            const int rows = at < 0 ? 0 : a.len - tile_of(u) * kPageUnit - u % 2 * kHalf;      // that hold something
            const int64_t off = max(at, static_cast<int64_t>(0));
            const float* k = static_cast<const float*>(m.k) + off;
            const float* v = static_cast<const float*>(m.v) + off;
            float* to = ring + stage * kHalfStage<NC>;
#pragma unroll
            for (int j = 0; j < kPieces; ++j) {
                const int x = lane + 32 * j, row = x / kUnits, d = x % kUnits * 4;
                if (d >= D) continue;
                const bool held = row < rows;
                const int from = held ? (u % 2 * kHalf + row) * m.ld + d : 0, bytes = held ? min(16, 4 * (D - d)) : 0;
                const uint32_t dst = smem_u32(to + row * kHalfPitch<NC> + d);
                copy16(dst, k + from, bytes);
                copy16(dst + kHalf * kHalfPitch<NC> * 4, v + from, bytes);
            }
        };
        int place = 0;                                         // of the half whose positions were loaded last
        auto load_pos = [&](int u) {
            const int at = tiles.pos(m, a, tile_of(u), lane), row = u % 2 * kHalf + g;
            place = at;
            return at >= 0 && tile_of(u) * kPageUnit + row < a.len ? m.pos[at + row] : kAhead;
        };
        const int64_t er = (static_cast<int64_t>(a.b) * m.H + a.h) * T + i0;
        float e[NQ];
        auto load_e = [&](int pos) {
#pragma unroll
            for (int x = 0; x < NQ; ++x)
                e[x] = i0 + x < a.n && pos <= a.first + i0 + x ? p.E[(er + x) * p.e_pitch + term(p, a.first + i0 + x, pos)] : kNone;
        };
#pragma unroll
        for (int u = 0; u < kHalfStages<NC> - 1; ++u) {
            if (u < halves) copy(u, u);
            mma::cp_async_commit();
        }
        int pos = kAhead, place0 = 0;                          // (place0: of the half at work; a tile has two halves)
        if (halves) {
            load_e(load_pos(0));
            pos = load_pos(1);
            place0 = place;
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
        int stage = 0, ahead = kHalfStages<NC> - 1;
        for (int u = 0; u < halves; ++u) {
            copies_wait<kHalfStages<NC> - 2>();
            __syncwarp();                                      // everyone's pieces are here, and the last stage is read
            if (u + kHalfStages<NC> - 1 < halves) copy(u + kHalfStages<NC> - 1, ahead);
            mma::cp_async_commit();
            ahead = stage;
            const float* k = ring + stage * kHalfStage<NC> + g * kHalfPitch<NC> + 4 * t;
            stage = stage + 1 == kHalfStages<NC> ? 0 : stage + 1;
            float s[NQ] = {};
#pragma unroll
            for (int j = 0; j < NJ; ++j) {
                const float4 y = *reinterpret_cast<const float4*>(k + 16 * j);
#pragma unroll
                for (int x = 0; x < NQ; ++x) {
                    const float4 w = *reinterpret_cast<const float4*>(qs + x * p.Dp + 4 * (t + 4 * j));
                    s[x] = fmaf(w.w, y.w, fmaf(w.z, y.z, fmaf(w.y, y.y, fmaf(w.x, y.x, s[x]))));
                }
            }
#pragma unroll
            for (int x = 0; x < NQ; ++x) s[x] += __shfl_xor_sync(0xffffffffu, s[x], 1);
#pragma unroll
            for (int x = 0; x < NQ; ++x) s[x] += __shfl_xor_sync(0xffffffffu, s[x], 2);
#pragma unroll
            for (int x = 0; x < NQ; ++x) s[x] = e[x] == kNone ? kNone : s[x] + e[x];
            if (u + 1 < halves) {
                load_e(pos);
                if (u + 2 < halves) pos = load_pos(u + 2);
            }
            if constexpr (W) {
                const int at = p.s_pool ? place0 : tile_of(u) * kPageUnit, row = u % 2 * kHalf + g;
                if (u % 2) place0 = place;
                if (t == 0 && at >= 0 && tile_of(u) * kPageUnit + row < a.len) {
                    float* S = score_row(p, a.b, a.h, i0) + at + row;
#pragma unroll
                    for (int x = 0; x < NQ; ++x)
                        if (i0 + x < a.n) S[static_cast<int64_t>(x) * p.s_slots] = s[x];
                }
            }
            // the maximum follows only where a score is far above it: a weight may be up to 2^kSlack
            constexpr float kSlack = 8.f;
            bool grows = false;
#pragma unroll
            for (int x = 0; x < NQ; ++x) grows |= s[x] > mx[x] + kSlack;
            if (__any_sync(0xffffffffu, grows)) {
#pragma unroll
                for (int x = 0; x < NQ; ++x) {
                    const float now = fmaxf(mx[x], s[x]), f = exp2f(mx[x] - finite_or_0(now));
                    mx[x] = now;
                    sum[x] *= f;
#pragma unroll
                    for (int j = 0; j < NJ; ++j) { o[x][j][0] *= f; o[x][j][1] *= f; o[x][j][2] *= f; o[x][j][3] *= f; }
                }
            }
#pragma unroll
            for (int x = 0; x < NQ; ++x) {
                s[x] = exp2f(s[x] - finite_or_0(mx[x]));
                sum[x] += s[x];
            }
#pragma unroll
            for (int j = 0; j < NJ; ++j) {
                const float4 y = *reinterpret_cast<const float4*>(k + kHalf * kHalfPitch<NC> + 16 * j);
#pragma unroll
                for (int x = 0; x < NQ; ++x) {
                    o[x][j][0] = fmaf(s[x], y.x, o[x][j][0]);
                    o[x][j][1] = fmaf(s[x], y.y, o[x][j][1]);
                    o[x][j][2] = fmaf(s[x], y.z, o[x][j][2]);
                    o[x][j][3] = fmaf(s[x], y.w, o[x][j][3]);
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
                        buf[warp * share + (i0 + x) * p.Dp + 4 * (t + 4 * j) + c] = y;
                }
            if (lane == 0 && i0 + x < a.n) {
                bml[(warp * T + i0 + x) * 2] = top;
                bml[(warp * T + i0 + x) * 2 + 1] = l;
            }
        }
    }
}

// Adds one to a ticket: what the block wrote before (and a barrier) is seen by the block that finds it the last.
__device__ __forceinline__ int arrive(int* ticket)
{
    int old;
    asm volatile("atom.acq_rel.gpu.global.add.s32 %0, [%1], 1;" : "=r"(old) : "l"(ticket) : "memory");
    return old;
}

template <typename T> __device__ __forceinline__ T* out_row(const PagedAttnParams& p, const Part& a, int i)
{
    return static_cast<T*>(p.out) + a.b * p.o_sb + i * p.o_st + a.h * p.o_sh;
}

// One query's row again, key by key on the CUDA cores: its sums are not finite, and a value that is not finite at a key
// that the query does not see must not reach it (0 times infinity).  A score of -inf comes of the tensor cores as NaN where the
// lower one of the query's two bf16 parts is zero or has the other sign, so the scores and their log-sum-exp, of which the
// weights are made, are written again too.  The whole block calls; tot: a float and a pointer for each of its threads.
template <typename T, int NW>
__device__ __noinline__ void row_again(const PagedAttnParams& p, const Part& a, int i, float* tot)
{
    const PagedParams& m = p.n.m;
    const T* q = static_cast<const T*>(p.q) + a.b * p.q_sb + i * p.q_st + a.h * p.q_sh;
    const int64_t row0 = (static_cast<int64_t>(a.b) * m.H + a.h) * p.n.T + i;
    const int at = a.first + i, keys = a.len + (a.own ? 1 : 0);
    // slot s, or the new key behind the last; null where there is none
    auto row = [&](int s, bool value) -> const T* {
        if (s == a.len)
            return value ? static_cast<const T*>(p.n.xv) + a.b * p.n.xv_sb + a.h * p.n.xv_sh
                         : static_cast<const T*>(p.n.xk) + a.b * p.n.xk_sb + a.h * p.n.xk_sh;
        const int page = page_of(m, a.b, s);
        if (page < 0) return nullptr;
        return static_cast<const T*>(value ? m.v : m.k) + page_row0(m, page, a.h) + static_cast<int64_t>(s % m.page_len) * m.ld;
    };
    auto score = [&](int s) {
        const T* k = s < keys ? row(s, false) : nullptr;
        if (!k) return kNone;
        const int pos = s == a.len ? at : m.pos[static_cast<int64_t>(page_of(m, a.b, s)) * m.page_len + s % m.page_len];
        if (pos > at) return kNone;
        // (E would not do: it comes of two bf16 parts as well)
        const T* r = static_cast<const T*>(p.r) + a.h * p.r_head + term(p, at, pos) * p.r_row;
        float x = 0.f;
        for (int d = 0; d < m.D; ++d) {
            x = fmaf((to_f(q[d]) + p.u[a.h * m.D + d]) * p.qscale, to_f(k[d]), x);
            x = fmaf((to_f(q[d]) + p.vb[a.h * m.D + d]) * p.qscale, to_f(r[d]), x);
        }
        return x;
    };
    float top = kNone;
    bool nan = false;
    for (int s = threadIdx.x; s < keys; s += (32 * NW)) {
        const float x = score(s);
        nan |= x != x;
        top = fmaxf(top, x);
    }
    nan = __syncthreads_or(nan);
    tot[threadIdx.x] = top;
    __syncthreads();
    for (int x = 0; x < (32 * NW); ++x) top = fmaxf(top, tot[x]);
    nan |= top == INFINITY;                                   // (infinity less itself)
    top = finite_or_0(top);
    float sum = nan ? __int_as_float(0x7fc00000) : 0.f, o = sum;
    const int d = threadIdx.x;                                // D <= 128: a channel a thread
    const T** values = reinterpret_cast<const T**>(tot + 32 * NW);
    for (int s0 = 0; s0 < (nan ? 0 : keys); s0 += (32 * NW)) {
        const int s = s0 + threadIdx.x;
        const float x = score(s);
        const int page = p.accumulate && s < keys ? page_of(m, a.b, s) : -1;
        if (page >= 0) score_row(p, a.b, a.h, i)[score_slot(p, s, page * m.page_len + s % m.page_len)] = x;
        __syncthreads();
        // (a key that is seen and scores -inf weighs 0 as well; its values count as unseen)
        tot[threadIdx.x] = x == kNone ? 0.f : exp2f(x - top);
        values[threadIdx.x] = x == kNone ? nullptr : row(s, true);
        __syncthreads();
#pragma unroll 8
        for (int y = 0; y < (32 * NW); ++y) {
            const T* v = values[y];
            const float w = tot[y];
            sum += w;
            if (v && d < m.D) o = fmaf(w, to_f(v[d]), o);
        }
    }
    if (d < m.D) out_row<T>(p, a, i)[d] = from_f<T>(sum == 0.f ? 0.f : o / sum);
    if (p.accumulate && d == 0) p.lse[row0] = top + log2f(sum);
    __syncthreads();
}

// The warps' shares of a part joined: into the output where the part is the whole pair, else into the workspace;
// the last block of a pair joins the parts.  buf: the warps' sums [T][Dp], `pitch` apart, and (a new key's) own[D]; bml:
// their maxima and weights [NW + 1][T][2].  The tickets are zero before and after the call.
template <typename T, bool ONE, bool W, int NW>
__device__ __forceinline__ void join(const PagedAttnParams& p, const Part& a, float* buf, int pitch, const float* own, float* bml)
{
    __shared__ int last, again;
    const PagedParams& m = p.n.m;
    const int Tq = p.n.T, D = m.D, tid = threadIdx.x;
    const bool room = a.room, with_own = ONE && a.own && a.t1 == a.tiles;
    if (tid == 0) again = 0;
    __syncthreads();
    const bool whole = a.t0 == 0 && a.t1 == a.tiles;
    const int slot = 2 * static_cast<int>(blockIdx.x) + (a.t0 == 0 ? 1 : 0);
    // (unused rows of buf hold what was there; only queries i < n are touched)
    for (int x = tid; x < a.n * D; x += (32 * NW)) {
        const int i = x / D, d = x - i * D;
        float top = kNone;
#pragma unroll
        for (int w = 0; w < NW; ++w) top = fmaxf(top, bml[(w * Tq + i) * 2]);
        if (with_own) top = fmaxf(top, bml[2 * NW]);
        const float base = finite_or_0(top);
        float y = 0.f, l = 0.f;
#pragma unroll
        for (int w = 0; w < NW; ++w) {
            const float f = exp2f(bml[(w * Tq + i) * 2] - base);
            y = fmaf(f, buf[w * pitch + i * p.Dp + d], y);
            l = fmaf(f, bml[(w * Tq + i) * 2 + 1], l);
        }
        if (with_own && bml[2 * NW] != kNone) {
            const float f = exp2f(bml[2 * NW] - base);
            y = fmaf(f, own[d], y);
            l = fmaf(f, bml[2 * NW + 1], l);
        }
        if (whole && room) {
            const float v = l == 0.f ? 0.f : y / l;
            out_row<T>(p, a, i)[d] = from_f<T>(v);
            if (!isfinite(y) || !isfinite(l)) atomicOr(&again, 1 << i);
            if (W && d == 0) p.lse[(static_cast<int64_t>(a.b) * m.H + a.h) * Tq + i] = base + log2f(l);
        } else if (!whole) {
            p.part[(static_cast<int64_t>(slot) * Tq + i) * p.Dp + d] = y;
            if (d == 0) {
                p.ml[(slot * Tq + i) * 2] = top;
                p.ml[(slot * Tq + i) * 2 + 1] = l;
            }
        }
    }
    if (!whole) {
        // blocks first_block .. first_block + parts - 1 hold the pair's parts, the first one in its odd slot
        const int n = a.parts;
        __syncthreads();
        if (tid == 0) {
            int* ticket = m.scratch + m.B + 1 + a.b * m.H + a.h;
            last = arrive(ticket) == n - 1;
            if (last) *ticket = 0;
        }
        __syncthreads();
        if (last && room) {
            const int warp = tid >> 5, lane = tid & 31;
            auto slot_of = [&](int c) { return 2 * (a.first_block + c) + (c == 0 ? 1 : 0); };
            // one query: the warps share the parts; more: a warp takes a query
            const int step = a.n == 1 ? NW : 1;
            for (int i = a.n == 1 ? 0 : warp; i < a.n; i += NW) {
                // the maximum of all parts first
                float top = kNone;
                for (int c = lane; c < n; c += 32) top = fmaxf(top, __ldcg(p.ml + (slot_of(c) * Tq + i) * 2));
#pragma unroll
                for (int d = 16; d; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
                const float base = finite_or_0(top);
                float y[4] = {0.f, 0.f, 0.f, 0.f}, l = 0.f;
                for (int c0 = a.n == 1 ? warp : 0; c0 < n; c0 += 32 * step) {
                    const int mine = c0 + step * lane;
                    float f = 0.f;
                    if (mine < n) {
                        const float2 s = __ldcg(reinterpret_cast<const float2*>(p.ml + (slot_of(mine) * Tq + i) * 2));
                        f = exp2f(s.x - base);
                        l = fmaf(f, s.y, l);
                    }
                    const int here = min(32, (n - c0 + step - 1) / step);
#pragma unroll 4
                    for (int z = 0; z < here; ++z) {
                        const float w = __shfl_sync(0xffffffffu, f, z);
                        const float* src = p.part + (static_cast<int64_t>(slot_of(c0 + step * z)) * Tq + i) * p.Dp;
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            if (32 * k + lane < D) y[k] = fmaf(w, __ldcg(src + 32 * k + lane), y[k]);
                    }
                }
#pragma unroll
                for (int d = 16; d; d >>= 1) l += __shfl_xor_sync(0xffffffffu, l, d);
                if (a.n == 1) {
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        if (32 * k + lane < D) buf[warp * p.Dp + 32 * k + lane] = y[k];
                    if (lane == 0) bml[warp] = l;
                    __syncthreads();
                    if (warp) break;
                    l = 0.f;
#pragma unroll
                    for (int w = 0; w < NW; ++w) {
                        l += bml[w];
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            if (32 * k + lane < D) y[k] = w ? y[k] + buf[w * p.Dp + 32 * k + lane] : buf[32 * k + lane];
                    }
                }
                bool finite = isfinite(l);
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    if (32 * k + lane < D) {
                        out_row<T>(p, a, i)[32 * k + lane] = from_f<T>(l == 0.f ? 0.f : y[k] / l);
                        finite = finite && isfinite(y[k]);
                    }
                if (!finite) atomicOr(&again, 1 << i);
                if (W && lane == 0) p.lse[(static_cast<int64_t>(a.b) * m.H + a.h) * Tq + i] = base + log2f(l);
            }
        }
    }
    __syncthreads();
    for (int bits = again; bits; bits &= bits - 1) row_again<T, NW>(p, a, __ffs(bits) - 1, buf);
    __syncthreads();
}

// Warps of a block: four; eight, in one block, for more than eight queries or more than four of d_head above 64 (five drafted tokens
// of d_head 128: 25.5 us, against 28.5 with three blocks of four; 16 queries of d_head 64 53.8 and 56.2; but one query of d_head 96
// over 4096 positions 44.9 and 42.7, of d_head 128 over up to 2048 18.6 and 17.7; of d_head 64 31.9 and, with four blocks, 30.6).
template <typename T, int NC, int NQ> constexpr int kWarpsOf = sizeof(T) == 2 && (NQ > 2 || (NC > 2 && NQ > 1)) ? 8 : 4;
// Blocks of the attention that an SM holds: what registers (bf16: and the rings) of the variants leave room for.
template <typename T, int NC, int NQ>
constexpr int kBlocks = sizeof(T) == 4             ? (NQ > 4 ? 4 - NC : NC == 1 ? 4 : NC == 2 || NQ == 1 ? 3 : 2)
                        : kWarpsOf<T, NC, NQ> == 8 ? 1
                        : NC <= 2                  ? 4
                                                   : 3;

// Floats between the warps' sums in shared memory (bf16: in their rings); row_again takes three a lane.
template <typename T, int NC>
__host__ __device__ __forceinline__ int warp_floats(int queries, int Dp) { return sizeof(T) == 4 ? max(queries * Dp, 96) : kWarpBytes<NC> / 4; }

// Floats of a warp's ring that lie behind all warps' sums (bf16: none, the sums are in the ring).
template <typename T, int NC> constexpr int kOwnRing = sizeof(T) == 4 ? kHalfStages<NC> * kHalfStage<NC> : 0;

// Floats of a new key's values (ONE) and the queries.
template <typename T, int NC, int NQ, bool ONE>
__host__ __device__ __forceinline__ int beside_floats(int Dp)
{
    return sizeof(T) == 4 ? NQ * Dp : (ONE ? Dp : 0) + kQRows<NC, NQ, ONE> * kQPitch<NC> / 2;
}

// Length, position of the first query and queries of sequence b, as the memory stands before the call: with ONE the length
// without the new key, else with the keys that the preparation puts there (its rule; up to 16 of them lie in two pages at
// most).
template <bool ONE>
__device__ __forceinline__ int3 now_of(const PagedAttnParams& p, int b)
{
    const PagedParams& m = p.n.m;
    const int len = m.length[b], next = m.next_pos[b], n = paged_count(p.n.counts, b, ONE ? 1 : p.n.T);
    bool ok = len >= 0 && len <= p.cap;
    if (ONE || !p.n.xk) {
        if (ONE && !ok && n > 0) page_error(m);
        return make_int3(len, p.n.xk ? next : next - n, ok ? n : 0);
    }
    ok = ok && n > 0 && len <= p.cap - n && page_of(m, b, len) >= 0 && page_of(m, b, len + n - 1) >= 0;
    return make_int3(ok ? len + n : len, next, ok ? n : 0);
}

// Shared memory: the warps' rings (fp32: their sums, then their rings); a new key's values; queries; maxima and weights; where the
// sequences' pairs begin [B + 1] (64 bits); the sequences' lengths and first positions [B]; a small page table.
template <typename T, int NC, int NQ, bool ONE, bool W>
__global__ void __launch_bounds__((32 * kWarpsOf<T, NC, NQ>), (kBlocks<T, NC, NQ>)) paged_attn_kernel(const __grid_constant__ PagedAttnParams p)
{
    constexpr int NW = kWarpsOf<T, NC, NQ>;
    extern __shared__ __align__(16) float buf[];
    __shared__ int64_t scan[NW];
    const PagedParams& m = p.n.m;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int pitch = warp_floats<T, NC>(p.n.T, p.Dp);
    float* beside = buf + NW * (pitch + kOwnRing<T, NC>);
    float* bml = beside + beside_floats<T, NC, NQ, ONE>(p.Dp);
    int64_t* start = reinterpret_cast<int64_t*>(bml + ((NW + 1) * p.n.T * 2 + 3) / 4 * 4);
    int2* info = reinterpret_cast<int2*>(start + m.B + 1);
    int* small = reinterpret_cast<int*>(info + m.B);
    if constexpr (ONE) {
        // (the rows of queries that one token does not have)
        uint32_t* rows = reinterpret_cast<uint32_t*>(beside + p.Dp);
        for (int x = tid; x < kQRows<NC, NQ, ONE> * kQPitch<NC> / 2; x += (32 * NW)) rows[x] = 0;
    }
    // (no early launch of the next grid: blocks of the weights' kernel that wait would take the place of later blocks)
    // The preparation began when all before it had ended, and this grid when all of that had begun: what the preparation does not
    // write, which is all but the new positions and the workspace, is read while it still runs (four queries over 4096
    // positions 35.3 us, after a wait for all of it 36.2; fp32 45.4 and 46.9).
    if (ONE) pdl_wait();

    // a small page table comes into shared memory beside the lengths: a part's first look then does not wait for one
    const int entries = p.held;
    for (int x = tid; x < entries; x += (32 * NW))
        asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(small + x)), "l"(m.table + x) : "memory");
    mma::cp_async_commit();
    const int* held = entries ? small : m.table;
    // start[b]: the work of all pairs of the sequences before b (an empty memory counts as a tile)
    int64_t done = 0;
    for (int b0 = 0; b0 < m.B; b0 += (32 * NW)) {
        const int b = b0 + tid;
        int64_t x = 0;
        if (b < m.B) {
            const int3 now = now_of<ONE>(p, b);
            x = now.z > 0 ? static_cast<int64_t>(kHead + max(1, (now.x + kPageUnit - 1) / kPageUnit)) * m.H : 0;
            info[b] = make_int2(now.x, now.y);
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
        for (int w = 0; w < NW; ++w) done += scan[w];
        __syncthreads();
    }
    if (tid == 0) start[m.B] = done;
    // the last block that has read the lengths advances them at its end (the ticket's answer is not waited for before)
    const bool counts = p.n.xk || (ONE && W);
    int ticket = -1;
    if (counts && tid == 32 * NW - 1)
        asm volatile("atom.relaxed.gpu.global.add.s32 %0, [%1], 1;" : "=r"(ticket) : "l"(m.scratch + m.B) : "memory");
    auto advance = [&] {
        if (!ONE) pdl_wait();                                  // (the preparation reads them too, and ends before this grid does)
        if (!counts || warp != NW - 1) return;
        const bool last = ticket == static_cast<int>(gridDim.x) - 1;
        if (!__any_sync(0xffffffffu, last)) return;
        if (last) m.scratch[m.B] = 0;
        for (int b = lane; b < m.B; b += 32) {
            if (!ONE) {
                if (start[b + 1] == start[b]) continue;
                m.length[b] = info[b].x;
                m.next_pos[b] = info[b].y + paged_count(p.n.counts, b, p.n.T);
                continue;
            }
            int4 now = make_int4(info[b].x, info[b].y, start[b + 1] > start[b] ? 1 : 0, 0);
            if (p.n.xk && now.z > 0) {
                if (page_of(m, b, now.x) < 0) {
                    now.z = 0;
                } else {
                    m.length[b] = ++now.x;
                    m.next_pos[b] = now.y + 1;
                }
            }
            if (W) p.now[b] = now;
        }
    };
    copies_wait<0>();
    __syncthreads();
    const int share = max(kMinTiles, quotient(done + gridDim.x - 1, gridDim.x));
    int64_t at = static_cast<int64_t>(blockIdx.x) * share;
    const int64_t end = min(done, at + share);
    if (at >= end) {
        advance();
        return;
    }
    int b = 0, hi = m.B;                                       // start[b] <= at < start[hi]
    while (hi - b > 1) {
        const int mid = (b + hi) / 2;
        if (start[mid] <= at) b = mid; else hi = mid;
    }
    while (at < end) {
        while (start[b + 1] <= at) ++b;
        Part a;
        a.b = b;
        a.len = info[b].x;
        a.first = info[b].y;
        a.n = ONE ? 1 : paged_count(p.n.counts, b, p.n.T);
        a.own = ONE && p.n.xk;
        a.table = held + static_cast<int64_t>(b) * m.max_pages;
        a.room = !a.own || page_at(m, a, a.len) >= 0;
        a.tiles = max(1, (a.len + kPageUnit - 1) / kPageUnit);
        const int size = kHead + a.tiles;
        a.h = quotient(at - start[b], size);
        const int64_t begin = start[b] + static_cast<int64_t>(a.h) * size;
        // the pair's tiles lie at begin + kHead on; a whole pair belongs to the block in whose share it begins
        if (a.tiles <= kWholeTiles) {
            a.t0 = begin >= at ? 0 : a.tiles;
            a.t1 = a.tiles;
            a.parts = 1;
        } else {
            a.t0 = static_cast<int>(max(at - begin - kHead, static_cast<int64_t>(0)));
            a.t1 = static_cast<int>(min(end - begin - kHead, static_cast<int64_t>(a.tiles)));
            a.first_block = quotient(begin + kHead, share);
            a.parts = quotient(begin + size - 1, share) - a.first_block + 1;
        }
        at = min(end, begin + size);
        if (a.t0 >= a.t1) continue;
        if constexpr (sizeof(T) == 4) part_f32<NC, NQ, W, NW>(p, a, buf, pitch, bml, beside);
        else part_bf16<NC, NQ, ONE, W, NW>(p, a, reinterpret_cast<char*>(buf + warp * pitch), bml, beside,
                                       reinterpret_cast<uint16_t*>(beside + (ONE ? p.Dp : 0)));
        join<T, ONE, W, NW>(p, a, buf, pitch, beside, bml);
    }
    advance();
}

// ---------------------------------------------------------------- attention weights
// A block takes 32 V slots of a sequence, a lane V of them; the warps share the heads; the sums meet in a fixed order.
template <int V> constexpr int kWeightWarps = V == 1 ? 16 : 8;

template <int V>
__global__ void __launch_bounds__(32 * kWeightWarps<V>) paged_weight_kernel(const __grid_constant__ PagedAttnParams p)
{
    constexpr int kSlots = 32 * V;
    __shared__ __align__(16) float sums[kWeightWarps<V>][kSlots];
    pdl_wait();
    pdl_launch_dependents();
    const PagedParams& m = p.n.m;
    const int b = blockIdx.y, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int4 now = p.now[b];
    if (now.z == 0) return;
    for (int s0 = blockIdx.x * kSlots; s0 < now.x; s0 += gridDim.x * kSlots) {
        const int s = s0 + V * lane;                           // (a lane's slots lie in one unit of 16, all of them in S)
        float sum[V] = {};
        const int page = s < now.x && p.s_pool ? page_of(m, b, s) : 0;
        if (s < now.x && page >= 0)
            for (int h = warp; h < m.H; h += kWeightWarps<V>) {
                const int64_t row = (static_cast<int64_t>(b) * m.H + h) * p.n.T;
                const float* S = score_row(p, b, h, 0) + score_slot(p, s, page * m.page_len + s % m.page_len);
#pragma unroll 4
                for (int i = 0; i < now.z; ++i) {
                    float y[V];
                    if constexpr (V == 4) *reinterpret_cast<float4*>(y) = *reinterpret_cast<const float4*>(S + static_cast<int64_t>(i) * p.s_slots);
                    else y[0] = S[static_cast<int64_t>(i) * p.s_slots];
                    const float l = p.lse[row + i];
#pragma unroll
                    for (int e = 0; e < V; ++e) sum[e] += y[e] == kNone ? 0.f : exp2f(y[e] - l);
                }
            }
#pragma unroll
        for (int e = 0; e < V; ++e) sums[warp][V * lane + e] = sum[e];
        __syncthreads();
        const int mine = s0 + static_cast<int>(threadIdx.x);
        if (threadIdx.x < kSlots && mine < now.x) {
            const int page = page_of(m, b, mine);
            float w = 0.f;
#pragma unroll
            for (int x = 0; x < kWeightWarps<V>; ++x) w += sums[x][threadIdx.x];
            if (page >= 0) m.weight[static_cast<int64_t>(page) * m.page_len + mine % m.page_len] += w;
        }
        __syncthreads();
    }
}

template <int V>
cudaError_t launch_weights(const PagedAttnParams& p, int sm_count, cudaStream_t s)
{
    const int parts = max(1, min((p.cap + 32 * V - 1) / (32 * V), 16 * sm_count / p.n.m.B));
    return launch_dependent(paged_weight_kernel<V>, dim3(parts, p.n.m.B), dim3(32 * kWeightWarps<V>), 0, s, p);
}

template <typename T, int NC, int NQ, bool ONE>
cudaError_t launch(PagedAttnParams& p, int sm_count, cudaStream_t s)
{
    constexpr int NW = kWarpsOf<T, NC, NQ>;
    static OncePerDevice once;
    const PagedParams& m = p.n.m;
    size_t smem = 4 * (static_cast<size_t>(NW) * (warp_floats<T, NC>(p.n.T, p.Dp) + kOwnRing<T, NC>) +
                       beside_floats<T, NC, NQ, ONE>(p.Dp) + static_cast<size_t>(NW + 1) * 2 * p.n.T + 2) +
                  8 * (2 * static_cast<size_t>(m.B) + 1);
    // all blocks at once: 228 KB of an SM, of which each block takes 1 KB and its few static bytes besides
    auto fit = [&](size_t bytes) { return max(1, min(kBlocks<T, NC, NQ>, static_cast<int>(228 * 1024 / (bytes + 1024 + 128)))); };
    const int per_sm = fit(smem);
    // A page table of up to 8 KB that takes no block's place stands in shared memory: first looks then take 0.1 to 0.4 us less (one
    // query over 64 positions 6.14 against 6.25, five of d_head 128 25.5 and 25.8).
    const int64_t entries = static_cast<int64_t>(m.B) * m.max_pages;
    p.held = entries <= 2048 && smem + 4 * entries <= 224 * 1024 && fit(smem + 4 * entries) == per_sm ? static_cast<int>(entries) : 0;
    smem += 4 * static_cast<size_t>(p.held);
    cudaError_t e = allow_smem(once, 224 * 1024, paged_attn_kernel<T, NC, NQ, ONE, false>, paged_attn_kernel<T, NC, NQ, ONE, true>);
    if (e != cudaSuccess) return e;
    if (!ONE) {
        // a block copies a few hundred units of 16 bytes
        const int units = 2 * m.H * (m.ld * static_cast<int>(sizeof(T)) / 16), share = max(1, 512 / units);
        const int copies = p.n.xk ? (p.n.T + share - 1) / share : 1;
        const int64_t terms = static_cast<int64_t>((p.n_e + kPrepRows - 1) / kPrepRows) * m.H * ((static_cast<int64_t>(m.B) * p.n.T + 7) / 8);
        if (terms + m.B * copies > INT32_MAX) return cudaErrorInvalidConfiguration;
        e = launch_dependent(paged_prep_kernel<T, NC>, dim3(static_cast<unsigned>(m.B * copies + terms)), dim3(kThreads), 0, s, p,
                             copies, share);
        if (e != cudaSuccess) return e;
    }
    const int blocks = min(per_sm * sm_count, kPagedMaxCtas);
    if (!p.accumulate) return launch_dependent(paged_attn_kernel<T, NC, NQ, ONE, false>, dim3(blocks), dim3(32 * NW), smem, s, p);
    e = launch_dependent(paged_attn_kernel<T, NC, NQ, ONE, true>, dim3(blocks), dim3(32 * NW), smem, s, p);
    if (e != cudaSuccess) return e;
    // four slots a lane where that leaves every SM two blocks (32 sequences of up to 4096 slots: 5.6 us a call less), else one (four
    // sequences of up to 2048, 80 rows each: 2.2 us less)
    return static_cast<int64_t>(m.B) * p.cap >= 2 * 128 * sm_count ? launch_weights<4>(p, sm_count, s) : launch_weights<1>(p, sm_count, s);
}

template <typename T, int NC>
cudaError_t by_queries(PagedAttnParams& p, int sm_count, cudaStream_t s)
{
    // fp32: as many queries at a time as the registers hold sums of (d_head 64, 16 queries: 173 us, by fours 226 when loads were
    // into registers; d_head 128, 4 queries: 85 us, by twos 127); bf16: groups of four queries, and one token without preparation (B8 H16 D64 over
    // 4096 positions 38.6 us where two launches took 44.1, one sequence of 65536 with its own distances 84 and 115, when this was
    // measured)
    if constexpr (sizeof(T) == 4) {
        if (p.n.T == 1) return launch<T, NC, 1, false>(p, sm_count, s);
        return p.n.T <= 4 ? launch<T, NC, 4, false>(p, sm_count, s) : launch<T, NC, (NC <= 2 ? 8 : 4), false>(p, sm_count, s);
    } else {
        if (p.n.T == 1) return launch<T, NC, 1, true>(p, sm_count, s);
        if (p.n.T <= 4) return launch<T, NC, 1, false>(p, sm_count, s);
        return p.n.T <= 8 ? launch<T, NC, 2, false>(p, sm_count, s) : launch<T, NC, 4, false>(p, sm_count, s);
    }
}

template <typename T>
cudaError_t by_channels(PagedAttnParams& p, int sm_count, cudaStream_t s)
{
    switch (p.Dp / 32) {
    case 1: return by_queries<T, 1>(p, sm_count, s);
    case 2: return by_queries<T, 2>(p, sm_count, s);
    case 3: return by_queries<T, 3>(p, sm_count, s);
    default: return by_queries<T, 4>(p, sm_count, s);
    }
}

}  // namespace

cudaError_t launch_paged_attn(PagedAttnParams& p, txl_dtype dtype, int sm_count, cudaStream_t s)
{
    return dtype == TXL_F32 ? by_channels<float>(p, sm_count, s) : by_channels<__nv_bfloat16>(p, sm_count, s);
}

}  // namespace txl
