// txl_paged.cu -- a K/V memory held in pages: new positions enter, and the least attended leave.
//
// The memory caches the keys and values that later queries attend to ("Transformer-XL 和相对位置编码" §2.3.1).  Slot s of
// sequence b is row s mod P of page table[b][s / P]; a slot knows its position, so slots may be in any order.
//
// A push is a copy: 8 prompts of up to 1600 positions (H16 D64, 82 MB in and out) 17.3 us, 4.7 TB/s, bound by the loads that a thread
// has under way.  An eviction of 4 sequences of up to 16384 slots to 4096: selection 15.7 us, a chain of loads (3.4), two
// digits (4.5 and 3.5: histogram, barrier of the cluster, sum, scan) and the lists (3.5); moving 33.7 MB of rows 12.3 us, 5.5 TB/s.
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
constexpr int kEvictHeld = 8192;           // keys of a block that shared memory holds (more are made again each time)
constexpr int kEvictRanks = 8;             // blocks of a sequence, at most
// Slots that are worth a block of the cluster (us with 2048, 4096, 8192: 4 sequences of 16384 30.7, 30.5, 35.8; 8 of 8192 40.8, 42.4, 46.8;
// 8 of 4160 24.2, 23.0, 22.1).
constexpr int kEvictEach = 2048;

// Integers of another block of the cluster.
__device__ __forceinline__ int4 ld_rank4(const int* p, uint32_t rank)
{
    uint32_t a;
    int4 v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
    asm volatile("ld.shared::cluster.v4.s32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
    return v;
}
__device__ __forceinline__ int2 ld_rank2(const int* p, uint32_t rank)
{
    uint32_t a;
    int2 v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
    asm volatile("ld.shared::cluster.v2.s32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a) : "memory");
    return v;
}

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

// A cluster of blocks per sequence, each with a range of its slots: which slots leave (a selection by digits of the key,
// from the top, over the sum of the blocks' histograms), then which survivors behind slot `keep` fill which holes in front.
// Shared memory: the histograms of this digit and the next, the keys.
__global__ void __launch_bounds__(kEvictThreads, 1) paged_select_kernel(const __grid_constant__ PagedEvictParams p, int held)
{
    extern __shared__ __align__(16) uint64_t keys[];
    int* bins = reinterpret_cast<int*>(keys + held);                          // [2][kBins]
    __shared__ int sums[32];
    __shared__ int found[3];
    __shared__ __align__(16) unsigned long long ends[2];                      // least and largest key left
    __shared__ __align__(8) int counts[2];                                    // holes, movers of this block
    pdl_wait();
    pdl_launch_dependents();
    const PagedParams& m = p.m;
    const int b = blockIdx.y, tid = threadIdx.x, ranks = gridDim.x, rank = blockIdx.x;
    const int n = m.length[b], keep = p.keep;
    const bool whole = n > keep ? paged_room(m, b, 0, n) : true;              // (the blocks of a sequence agree)
    if (n <= keep || !whole) {
        if (tid == 0 && rank == 0) {
            p.moves[b] = 0;
            if (!whole) page_error(m);
        }
        return;
    }
    const int64_t guard = static_cast<int64_t>(m.next_pos[b]) - p.recent;      // positions from here on stay
    // this block's slots, an equal number for each thread, in order
    const int per = (n + ranks * kEvictThreads - 1) / (ranks * kEvictThreads);
    const int s0 = rank * kEvictThreads * per, mine = max(0, min(n - s0, kEvictThreads * per));
    constexpr uint64_t kStays = ~uint64_t{0};                                 // (no position is -1)
    auto row = [&](int s) { return page_of(m, b, s) * m.page_len + s % m.page_len; };
    auto make = [&](int i) {
        const int at = row(s0 + i);
        const int pos = m.pos[at];
        return pos < guard ? leave_key(m.weight[at], pos) : kStays;
    };
    for (int i = tid; i < min(mine, held); i += kEvictThreads) keys[i] = make(i);
    for (int i = tid; i < 2 * kBins; i += kEvictThreads) bins[i] = 0;
    if (tid == 0) ends[0] = kStays, ends[1] = 0;
    auto key_of = [&](int i) { return i < held ? keys[i] : make(i); };

    // the least (n - keep) keys: those whose bits above `shift` are at most `limit`
    int want = n - keep, shift = 64, turn = 0, digits = 0;
    uint64_t limit = 0;
    while (shift > 0) {
        const int width = min(kDigit, shift);
        int* own = bins + turn * kBins;
        __syncthreads();
        for (int i0 = 0; i0 < mine; i0 += kEvictThreads) {
            const int i = i0 + tid;
            int bin = -1;
            if (i < mine) {
                const uint64_t key = key_of(i);
                if (key != kStays && (shift == 64 || key >> shift == limit))
                    bin = static_cast<int>(key >> (shift - width)) & ((1 << width) - 1);
            }
            // many slots of one weight would queue at one bin: a warp that agrees adds once
            const int first = __shfl_sync(0xffffffffu, bin, 0);
            if (__all_sync(0xffffffffu, bin == first)) {
                if (first >= 0 && (tid & 31) == 0) atomicAdd(own + first, 32);
            } else if (bin >= 0) {
                atomicAdd(own + bin, 1);
            }
        }
        if (ranks > 1) cluster_sync_all();
        else __syncthreads();
        turn ^= 1;
        // four bins a thread, of all blocks' histograms (loaded together)
        constexpr int kPer = 4;
        static_assert(kBins == kPer * kEvictThreads / 2, "the first half of the threads takes the bins");
        int c[kPer] = {}, sum = 0, total;
        if (tid < kBins / kPer) {
            int4 other[kEvictRanks];
#pragma unroll
            for (int r = 0; r < kEvictRanks; ++r)
                other[r] = r >= ranks ? make_int4(0, 0, 0, 0) : ranks > 1 ? ld_rank4(own + tid * kPer, r) : reinterpret_cast<const int4*>(own)[tid];
#pragma unroll
            for (int r = 0; r < kEvictRanks; ++r) {
                c[0] += other[r].x;
                c[1] += other[r].y;
                c[2] += other[r].z;
                c[3] += other[r].w;
            }
            sum = c[0] + c[1] + c[2] + c[3];
            if (shift != 64) reinterpret_cast<int4*>(bins + turn * kBins)[tid] = make_int4(0, 0, 0, 0);      // (all blocks have read that one)
        }
        int below = block_scan(sum, sums, total);
        if (total < want) want = total;                                       // (positions that are not distinct)
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            if (below < want && want <= below + c[i]) { found[0] = tid * kPer + i; found[1] = below; found[2] = c[i]; }
            below += c[i];
        }
        __syncthreads();
        if (want == 0) break;
        const int digit = found[0];
        const bool all = found[1] + found[2] == want;                         // the whole bin leaves: no need to look closer
        want -= found[1];
        shift -= width;
        limit = (limit << width) | static_cast<uint64_t>(digit);
        if (all) break;
        if (++digits != 2) continue;
        // Two digits that did not do: as a rule many slots of one weight.  The digits that all the keys left share are skipped.
        uint64_t least = kStays, most = 0;
        for (int i = tid; i < mine; i += kEvictThreads) {
            const uint64_t key = key_of(i);
            if (key != kStays && key >> shift == limit) {
                least = min(least, key);
                most = max(most, key);
            }
        }
#pragma unroll
        for (int d = 16; d; d >>= 1) {
            least = min(least, __shfl_xor_sync(0xffffffffu, least, d));
            most = max(most, __shfl_xor_sync(0xffffffffu, most, d));
        }
        if ((tid & 31) == 0) {
            atomicMin(&ends[0], least);
            atomicMax(&ends[1], most);
        }
        if (ranks > 1) cluster_sync_all();
        else __syncthreads();
#pragma unroll
        for (int r = 0; r < kEvictRanks; ++r)
            if (r < ranks) {
                const int4 e = ranks > 1 ? ld_rank4(reinterpret_cast<const int*>(ends), r) : *reinterpret_cast<const int4*>(ends);
                least = min(least, static_cast<uint64_t>(static_cast<uint32_t>(e.y)) << 32 | static_cast<uint32_t>(e.x));
                most = max(most, static_cast<uint64_t>(static_cast<uint32_t>(e.w)) << 32 | static_cast<uint32_t>(e.z));
            }
        if (least < most) {
            shift = 64 - __clzll(least ^ most);
            limit = shift == 64 ? 0 : least >> shift;
        }
    }
    // a thread's slots are neighbours: one sum over the threads each orders its holes and its movers
    auto leaves = [&](int i) {
        const uint64_t key = key_of(i);
        return key != kStays && shift < 64 && key >> shift <= limit;
    };
    int holes = 0, movers = 0;
    for (int i = tid * per; i < min(mine, (tid + 1) * per); ++i) {
        const bool gone = leaves(i);
        holes += gone && s0 + i < keep;
        movers += !gone && s0 + i >= keep;
    }
    int all_holes, all_movers;
    holes = block_scan(holes, sums, all_holes);
    movers = block_scan(movers, sums, all_movers);
    if (tid == 0) {
        counts[0] = all_holes;
        counts[1] = all_movers;
    }
    int total_holes = all_holes, total_movers = all_movers;
    if (ranks > 1) {
        cluster_sync_all();
        const int lane = tid & 31;
        const int2 theirs = lane < ranks ? ld_rank2(counts, lane) : make_int2(0, 0);
        total_holes = total_movers = 0;
#pragma unroll
        for (int r = 0; r < kEvictRanks; ++r) {
            const int h = __shfl_sync(0xffffffffu, theirs.x, r), v = __shfl_sync(0xffffffffu, theirs.y, r);
            if (r < rank) { holes += h; movers += v; }
            total_holes += h;
            total_movers += v;
        }
    }
    int* to = p.to + static_cast<int64_t>(b) * p.most;
    int* from = p.from + static_cast<int64_t>(b) * p.most;
    for (int i = tid * per; i < min(mine, (tid + 1) * per); ++i) {
        const bool gone = leaves(i);
        if (gone && s0 + i < keep) {
            if (holes < p.most) to[holes] = row(s0 + i);
            ++holes;
        } else if (!gone && s0 + i >= keep) {
            if (movers < p.most) from[movers] = row(s0 + i);
            ++movers;
        }
    }
    if (tid == 0 && rank == 0) {
        p.moves[b] = min(p.most, min(total_holes, total_movers));
        m.length[b] = keep;
    }
    if (ranks > 1) cluster_sync_all();                                        // no block leaves while others read its counts
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
    // a block copies about 2048 units of 16 bytes, four positions at once (prompts of d_head 64: 18.3 us, with 4096 units 19.1; d_head 41: 15.3
    // and 18.7)
    const int units = 2 * p.m.H * (p.m.ld * (dtype == TXL_F32 ? 4 : 2) / 16);
    const int share = max(4, 2048 / units);
    const dim3 grid((p.T + share - 1) / share, p.m.B);
    if (dtype == TXL_F32) return launch_dependent(paged_push_kernel<float>, grid, dim3(kPushThreads), 0, s, p, share);
    return launch_dependent(paged_push_kernel<__nv_bfloat16>, grid, dim3(kPushThreads), 0, s, p, share);
}

cudaError_t launch_paged_evict(const PagedEvictParams& p, int sm_count, cudaStream_t s)
{
    static OncePerDevice once;
    const int cap = p.m.max_pages * p.m.page_len;
    int ranks = 1;
    while (ranks < kEvictRanks && cap > ranks * kEvictEach) ranks *= 2;
    const int held = min(kEvictHeld, (cap + ranks * kEvictThreads - 1) / (ranks * kEvictThreads) * kEvictThreads);
    const int most_smem = kEvictHeld * 8 + 2 * kBins * 4, smem = held * 8 + 2 * kBins * 4;
    cudaError_t e = allow_smem(once, most_smem, paged_select_kernel);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(ranks, p.m.B);
    cfg.blockDim = dim3(kEvictThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = ranks;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    e = cudaLaunchKernelEx(&cfg, paged_select_kernel, p, held);
    if (e != cudaSuccess) return e;
    const int blocks = min(max(1, sm_count * 8 / p.m.B), (p.most + kMoveThreads / 32 - 1) / (kMoveThreads / 32));
    return launch_dependent(paged_move_kernel, dim3(max(1, blocks), p.m.B), dim3(kMoveThreads), 0, s, p);
}

}  // namespace txl
