// txl_paged.cu -- a K/V memory held in pages: new positions enter, and the least attended leave.
//
// The memory caches the keys and values that later queries attend to ("Transformer-XL 和相对位置编码" §2.3.1).  Slot s of
// sequence b is row s mod P of page table[b][s / P]; a slot knows its position, so slots may be in any order.
#include <cuda_bf16.h>

#include "txl_paged.cuh"
#include "txl_ptx.cuh"

namespace txl {

namespace {

// ---------------------------------------------------------------- new positions
constexpr int kPushThreads = 256;

// Block (x, b) copies positions [x share, (x + 1) share).  A sequence whose positions do not all have pages is left as
// it was.  The last block of a sequence advances its length: the others have read it by then.
template <typename T>
__global__ void __launch_bounds__(kPushThreads) paged_push_kernel(const __grid_constant__ PagedPushParams p, int share)
{
    pdl_wait();
    pdl_launch_dependents();
    const int b = blockIdx.y, n = paged_count(p.counts, b, p.T);
    const int len = p.m.length[b], next = p.m.next_pos[b];
    if (n == 0) return;
    const bool room = paged_room(p.m, b, len, n);
    const int t0 = static_cast<int>(blockIdx.x) * share, t1 = min(n, t0 + share);
    if (room && t0 < t1) paged_copy<T>(p, b, len, next, t0, t1);
    __syncthreads();
    if (threadIdx.x == 0) {
        bool last = true;
        if (gridDim.x > 1) {
            __threadfence();
            last = atomicAdd(p.m.scratch + b, 1) == static_cast<int>(gridDim.x) - 1;
        }
        if (last) {
            p.m.scratch[b] = 0;
            if (room) {
                p.m.length[b] = len + n;
                p.m.next_pos[b] = next + n;
            } else {
                page_error(p.m);
            }
        }
    }
}

// ---------------------------------------------------------------- eviction
// A slot's rank in the order of leaving: its weight as an integer of the same order (-0 as 0, NaN above all), then
// its position, older ones first.
__device__ __forceinline__ uint64_t leave_key(float w, int pos)
{
    uint32_t k = __float_as_uint(w + 0.f);
    k = w != w ? 0xffffffffu : (k & 0x80000000u) ? ~k : k | 0x80000000u;
    return static_cast<uint64_t>(k) << 32 | static_cast<uint32_t>(pos);
}

constexpr int kEvictThreads = 1024;
constexpr int kDigit = 11, kBins = 1 << kDigit;

// Exclusive sum over the block, and the total (every thread calls; 1024 threads).
__device__ __forceinline__ int block_scan(int x, int* warp_sums, int& total)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int s = x;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, s, d);
        if (lane >= d) s += y;
    }
    __syncthreads();
    if (lane == 31) warp_sums[warp] = s;
    __syncthreads();
    int w = warp_sums[lane];
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, w, d);
        if (lane >= d) w += y;
    }
    total = __shfl_sync(0xffffffffu, w, 31);
    const int before = __shfl_sync(0xffffffffu, w, max(warp - 1, 0));
    return s - x + (warp ? before : 0);
}

// One block per sequence: which slots leave (a selection by digits of the key, from the top), then which survivors
// behind slot `keep` fill which holes in front of it.
__global__ void __launch_bounds__(kEvictThreads) paged_select_kernel(const __grid_constant__ PagedEvictParams p)
{
    __shared__ int bins[kBins];
    __shared__ int sums[32];
    __shared__ int found[2];
    pdl_wait();
    pdl_launch_dependents();
    const PagedParams& m = p.m;
    const int b = blockIdx.x, tid = threadIdx.x;
    const int n = m.length[b], keep = p.keep;
    const bool whole = n > keep ? paged_room(m, b, 0, n) : true;
    if (n <= keep || !whole) {
        if (tid == 0) {
            p.moves[b] = 0;
            if (!whole) page_error(m);
        }
        return;
    }
    const int64_t guard = static_cast<int64_t>(m.next_pos[b]) - p.recent;      // positions from here on stay
    auto row = [&](int s) { return static_cast<int64_t>(page_of(m, b, s)) * m.page_len + s % m.page_len; };

    // the least (n - keep) keys: those whose bits above `shift` are at most `limit`
    int want = n - keep, shift = 64;
    uint64_t limit = 0;
    bool none = false;
    while (shift > 0) {
        const int width = min(kDigit, shift);
        for (int i = tid; i < kBins; i += kEvictThreads) bins[i] = 0;
        __syncthreads();
        for (int s0 = 0; s0 < n; s0 += kEvictThreads) {
            const int s = s0 + tid;
            int bin = -1;
            if (s < n) {
                const int64_t at = row(s);
                const int pos = m.pos[at];
                const uint64_t key = leave_key(m.weight[at], pos);
                if (pos < guard && (shift == 64 || key >> shift == limit))
                    bin = static_cast<int>(key >> (shift - width)) & ((1 << width) - 1);
            }
            // many slots of one weight would queue at one bin: a warp that agrees adds once
            const int first = __shfl_sync(0xffffffffu, bin, 0);
            if (__all_sync(0xffffffffu, bin == first)) {
                if (first >= 0 && (tid & 31) == 0) atomicAdd(bins + first, 32);
            } else if (bin >= 0) {
                atomicAdd(bins + bin, 1);
            }
        }
        __syncthreads();
        constexpr int kPer = kBins / kEvictThreads;
        int mine = 0, total;
#pragma unroll
        for (int i = 0; i < kPer; ++i) mine += bins[tid * kPer + i];
        int below = block_scan(mine, sums, total);
        if (total < want) { want = total; none = total == 0; }      // fewer may leave (positions that are out of order)
        if (none) break;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int c = bins[tid * kPer + i];
            if (below < want && want <= below + c) { found[0] = tid * kPer + i; found[1] = below; }
            below += c;
        }
        __syncthreads();
        const int digit = found[0];
        const bool all = found[1] + bins[digit] == want;            // the whole bin leaves: no need to look closer
        want -= found[1];
        shift -= width;
        limit = (limit << width) | static_cast<uint64_t>(digit);
        __syncthreads();
        if (all) break;
    }
    auto leaves = [&](int s) {
        const int64_t at = row(s);
        const int pos = m.pos[at];
        return !none && pos < guard && leave_key(m.weight[at], pos) >> shift <= limit;
    };
    int holes = 0, movers = 0;
    int* to = p.to + static_cast<int64_t>(b) * p.most;
    int* from = p.from + static_cast<int64_t>(b) * p.most;
    for (int s0 = 0; s0 < n; s0 += kEvictThreads) {
        const int s = s0 + tid;
        bool hole = false, mover = false;
        if (s < n) {
            const bool gone = leaves(s);
            hole = gone && s < keep;
            mover = !gone && s >= keep;
        }
        int total;
        const int rank = block_scan(hole ? 1 : mover ? 0x10000 : 0, sums, total);
        if (hole && holes + (rank & 0xffff) < p.most) to[holes + (rank & 0xffff)] = static_cast<int>(row(s));
        if (mover && movers + (rank >> 16) < p.most) from[movers + (rank >> 16)] = static_cast<int>(row(s));
        holes += total & 0xffff;
        movers += total >> 16;
    }
    if (tid == 0) {
        p.moves[b] = min(holes, movers);
        m.length[b] = keep;
    }
}

constexpr int kMoveThreads = 256;

// A warp moves one position: the rows of all heads, in units of 16 bytes.
__global__ void __launch_bounds__(kMoveThreads) paged_move_kernel(const __grid_constant__ PagedEvictParams p)
{
    pdl_wait();
    pdl_launch_dependents();
    const PagedParams& m = p.m;
    const int b = blockIdx.y, n = p.moves[b], lane = threadIdx.x & 31;
    const int64_t row_bytes = static_cast<int64_t>(m.ld) * p.elem;
    const int units = static_cast<int>(row_bytes / 16), per = m.H * units;
    const int warps = gridDim.x * (kMoveThreads / 32);
    for (int i = blockIdx.x * (kMoveThreads / 32) + (threadIdx.x >> 5); i < n; i += warps) {
        const int dst = p.to[static_cast<int64_t>(b) * p.most + i], src = p.from[static_cast<int64_t>(b) * p.most + i];
        const int64_t d0 = (static_cast<int64_t>(dst / m.page_len) * m.H * m.page_len + dst % m.page_len) * row_bytes;
        const int64_t s0 = (static_cast<int64_t>(src / m.page_len) * m.H * m.page_len + src % m.page_len) * row_bytes;
        for (int x0 = 0; x0 < 2 * per; x0 += 32 * 4) {
            uint4 w[4];
            int64_t at[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int x = x0 + j * 32 + lane, y = x >= per ? x - per : x;
                at[j] = static_cast<int64_t>(y / units) * m.page_len * row_bytes + (y % units) * 16;
                if (x < 2 * per) w[j] = *reinterpret_cast<const uint4*>(static_cast<const char*>(x >= per ? m.v : m.k) + s0 + at[j]);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int x = x0 + j * 32 + lane;
                if (x < 2 * per) *reinterpret_cast<uint4*>(static_cast<char*>(x >= per ? m.v : m.k) + d0 + at[j]) = w[j];
            }
        }
        if (lane == 0) {
            m.pos[dst] = m.pos[src];
            m.weight[dst] = m.weight[src];
        }
    }
}

}  // namespace

cudaError_t launch_paged_push(const PagedPushParams& p, txl_dtype dtype, cudaStream_t s)
{
    // a block copies a few thousand units of 16 bytes
    const int units = 2 * p.m.H * (p.m.ld * (dtype == TXL_F32 ? 4 : 2) / 16);
    const int share = max(1, 2048 / units);
    const dim3 grid((p.T + share - 1) / share, p.m.B);
    if (dtype == TXL_F32) return launch_dependent(paged_push_kernel<float>, grid, dim3(kPushThreads), 0, s, p, share);
    return launch_dependent(paged_push_kernel<__nv_bfloat16>, grid, dim3(kPushThreads), 0, s, p, share);
}

cudaError_t launch_paged_evict(const PagedEvictParams& p, int sm_count, cudaStream_t s)
{
    cudaError_t e = launch_dependent(paged_select_kernel, dim3(p.m.B), dim3(kEvictThreads), 0, s, p);
    if (e != cudaSuccess) return e;
    const int blocks = min(max(1, sm_count * 8 / p.m.B), (p.most + kMoveThreads / 32 - 1) / (kMoveThreads / 32));
    return launch_dependent(paged_move_kernel, dim3(max(1, blocks), p.m.B), dim3(kMoveThreads), 0, s, p);
}

}  // namespace txl
