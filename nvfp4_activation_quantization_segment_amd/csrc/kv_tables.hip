// Block tables, row starts, positions and slots of a batch, built on the GPU
// from the requests' lengths; and the blocks of finished requests given back.
// All of it is integers, a few bytes for each row and request: what takes the
// time is the chain of loads that depend on one another, and the launches.
#include "kv_device.h"

namespace nvfp4 {
namespace {

constexpr int kThreads = 1024, kWaves = kThreads / 64;

// Inclusive sum over the workgroup's threads; total: that of all of them.  The
// slots are read by all before the call returns and written by the next one's
// first barrier at the earliest.
__device__ __forceinline__ int64_t group_scan(int64_t x, int64_t* slot, int64_t& total) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
    for (int s = 1; s < 64; s <<= 1) {
        const int64_t other = __shfl_up(x, s);
        x += lane >= s ? other : 0;
    }
    __syncthreads();  // the slots of the scan before are read
    if (lane == 63) slot[wave] = x;
    __syncthreads();
    int64_t before = 0;
    total = 0;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
        const int64_t t = slot[w];
        before += w < wave ? t : 0;
        total += t;
    }
    return x + before;
}

// Blocks that `len` positions take of a table.
__device__ __forceinline__ int32_t blocks_of(int64_t len, int64_t table_blocks) {
    return (int32_t)clamp64(len <= 0 ? 0 : (len + kKvBlock - 1) / kKvBlock, 0, table_blocks);
}

// ---------------------------------------------------------------------------
// Extending.  The requests come first: rows and blocks of each, as running sums,
// by one workgroup (the sums of a few thousand requests are a few rounds of it).
// Then the rows: each finds its request, and the row that starts a block writes
// the table's entry.  A block's number comes from the sums alone, so rows of one
// block need not wait for one another.
// ---------------------------------------------------------------------------
__device__ __forceinline__ void extend_requests(const ExtendArgs& a) {
    __shared__ int64_t slot[kWaves];
    const int64_t had = clamp64(*a.free_count, 0, a.capacity);
    int64_t rows = 0, blocks = 0;  // of the requests before
    if (threadIdx.x == 0) a.row_start[0] = 0;
    for (int64_t b0 = 0; b0 < a.B; b0 += kThreads) {
        const int64_t b = b0 + threadIdx.x;
        const int64_t past = b < a.B ? a.past[b] : 0;
        const int64_t want = b < a.B ? clamp64(a.more[b], 0, INT32_MAX - clamp64(past, 0, INT32_MAX)) : 0;
        int64_t sum_rows, sum_blocks;
        const int64_t end = rows + group_scan(want, slot, sum_rows);
        const int64_t first = clamp64(end - want, 0, a.M), last = clamp64(end, 0, a.M);
        const int64_t len = past + (last - first);
        const int64_t take = blocks_of(len, a.table_blocks) - blocks_of(past, a.table_blocks);
        const int64_t taken = blocks + group_scan(take, slot, sum_blocks) - take;
        if (b < a.B) {
            a.row_start[b + 1] = (int32_t)last;
            a.lens[b] = (int32_t)len;
            a.taken[b] = (int32_t)taken;
        }
        rows += sum_rows;
        blocks += sum_blocks;
    }
    if (threadIdx.x == 0) {
        a.state[0] = (int32_t)had;
        *a.free_left = (int32_t)(had > blocks ? had - blocks : 0);
        *a.missing = (int32_t)(blocks > had ? blocks - had : 0);
    }
}

// The request of a row below row_start[B]: the last that starts at or before it.
// The wave finds its first row's 64 places at a time; its other rows' are mostly
// among the 64 that follow, whose starts its lanes then hold.
__device__ __forceinline__ int64_t request_of(const ExtendArgs& a, int64_t row, int64_t row0) {
    const int lane = threadIdx.x & 63;
    int64_t lo = 0, n = a.B;
    while (n > 1) {
        const int64_t stride = (n + 63) / 64;
        const int64_t at = lane * stride;
        const bool ok = at < n && (lane == 0 || a.row_start[lo + at] <= row0);
        const int64_t skip = (63 - __builtin_clzll(__ballot(ok))) * stride;
        lo += skip;
        n = n - skip < stride ? n - skip : stride;
    }
    // among the 63 after it, by halves
    const int32_t start = a.row_start[lo + lane < a.B ? lo + lane : a.B];
    int at = 0;
#pragma unroll
    for (int s = 32; s > 0; s >>= 1) {
        const int32_t there = __shfl(start, at + s);
        if (lo + at + s < a.B && there <= row) at += s;
    }
    int64_t b = lo + at;
    if (at == 63) {  // beyond them: requests without rows lie between
        int64_t left = a.B - b;
        while (left > 1) {
            const int64_t half = left / 2;
            if (a.row_start[b + half] <= row) {
                b += half;
                left -= half;
            } else {
                left = half;
            }
        }
    }
    return b;
}

__device__ __forceinline__ void extend_rows(const ExtendArgs& a, int64_t row0) {
    const int64_t row = row0 + (threadIdx.x & 63);
    const int32_t used = a.row_start[a.B];
    if (row0 >= used) {
        if (row < a.M) {
            if (a.positions) a.positions[row] = -1;
            if (a.slots) a.slots[row] = -1;
        }
        return;
    }
    const int64_t b = request_of(a, row < used ? row : used - 1, row0);
    if (row >= a.M) return;
    int64_t pos = -1, slot = -1;
    if (row < used) {
        const int64_t first = a.row_start[b], n = a.row_start[b + 1] - first, past = a.lens[b] - n;
        pos = past + row - first;
        const int64_t at = floor_div(pos, kKvBlock);
        if (pos >= 0 && at < a.table_blocks) {
            const int64_t fresh = at - blocks_of(past, a.table_blocks);
            int32_t* entry = a.table + b * a.ld_table + at;
            int32_t page;
            if (fresh < 0) {
                page = *entry;
            } else {
                const int64_t place = (int64_t)a.state[0] - 1 - a.taken[b] - fresh;
                page = place >= 0 ? a.free_blocks[place] : -1;
                if (pos % kKvBlock == 0) *entry = page;
            }
            slot = page < 0 ? -1 : (int64_t)page * kKvBlock + pos % kKvBlock;
        }
    }
    if (a.positions) a.positions[row] = (int32_t)pos;
    if (a.slots) a.slots[row] = slot;
}

__global__ __launch_bounds__(kThreads) void extend_requests_kernel(ExtendArgs a) { extend_requests(a); }

__global__ __launch_bounds__(256) void extend_rows_kernel(ExtendArgs a) {
    const int64_t row0 = ((int64_t)blockIdx.x * 4 + (threadIdx.x >> 6)) * 64;
    if (row0 < a.M) extend_rows(a, row0);
}

__global__ __launch_bounds__(kThreads) void extend_kernel(ExtendArgs a) {
    extend_requests(a);
    __threadfence_block();
    __syncthreads();
    for (int64_t row0 = (threadIdx.x >> 6) * 64; row0 < a.M; row0 += kThreads) extend_rows(a, row0);
}

// ---------------------------------------------------------------------------
// Releasing.  A wave takes a request: its table's entries, 64 at a time.  Their
// places on the stack follow from how many blocks the requests before give back,
// so a first launch counts and a second one moves.
// ---------------------------------------------------------------------------
constexpr int kEach = 4;                 // requests of a wave
constexpr int kOf = kEach * kWaves;      // requests of a workgroup

__device__ __forceinline__ int32_t release_blocks(const ReleaseArgs& a, int64_t b) {
    return b < a.B && a.done[b] != 0 ? blocks_of(a.lens[b], a.table_blocks) : 0;
}

// Blocks that the wave's request gives back, counted, and with move() for each.
template <class Move>
__device__ __forceinline__ int64_t release_request(const ReleaseArgs& a, int64_t b, Move move) {
    const int lane = threadIdx.x & 63;
    const int32_t blocks = release_blocks(a, b);
    int64_t count = 0;
    for (int64_t at = a.keep; at < blocks; at += 64) {
        const int32_t page = at + lane < blocks ? a.table[b * a.ld_table + at + lane] : -1;
        const uint64_t good = __ballot(page >= 0);
        if (page >= 0) move(count + __popcll(good & (((uint64_t)1 << lane) - 1)), page);
        count += __popcll(good);
    }
    return count;
}

__global__ __launch_bounds__(kThreads) void release_count_kernel(ReleaseArgs a) {
    __shared__ int64_t share[kWaves];
    const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    const int64_t b0 = (int64_t)blockIdx.x * kOf + wave * kEach;
    int64_t mine = 0;
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
        const int64_t count = release_request(a, b0 + i, [](int64_t, int32_t) {});
        if (b0 + i < a.B && (threadIdx.x & 63) == 0) a.counts[b0 + i] = (int32_t)count;
        mine += count;
    }
    if ((threadIdx.x & 63) == 0) share[wave] = mine;
    __syncthreads();
    if (threadIdx.x == 0) {
        int64_t all = 0;
        for (int w = 0; w < kWaves; ++w) all += share[w];
        a.totals[blockIdx.x] = all;
        if (blockIdx.x == 0) a.state[0] = *a.free_count;
    }
}

__global__ __launch_bounds__(kThreads) void release_move_kernel(ReleaseArgs a) {
    __shared__ int64_t slot[kWaves];
    const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    // what the workgroups before give back, and all of them
    int64_t before = 0, all = 0;
    for (int64_t i = threadIdx.x; i < gridDim.x; i += kThreads) {
        const int64_t t = a.totals[i];
        before += i < blockIdx.x ? t : 0;
        all += t;
    }
    int64_t sum;
    group_scan(before, slot, sum);
    const int64_t had = clamp64(a.state[0], 0, a.capacity);
    int64_t place = had + sum;
    group_scan(all, slot, sum);
    if (blockIdx.x == 0 && threadIdx.x == 0) *a.free_left = (int32_t)clamp64(had + sum, 0, a.capacity);
    // and the waves before
    const int64_t b0 = (int64_t)blockIdx.x * kOf;
    for (int i = 0; i < wave * kEach; ++i) place += b0 + i < a.B ? a.counts[b0 + i] : 0;
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
        const int64_t b = b0 + wave * kEach + i;
        place += release_request(a, b, [&](int64_t at, int32_t page) {
            if (place + at < a.capacity) a.free_blocks[place + at] = page;
        });
        if (b < a.B && (threadIdx.x & 63) == 0) a.lens_out[b] = a.done[b] != 0 ? 0 : a.lens[b];
    }
}

}  // namespace

// Up to so many rows one workgroup does all of it, in one launch.
constexpr int64_t kOneGroupRows = 4096;

hipError_t launch_kv_extend(const ExtendArgs& a, hipStream_t s) {
    if (a.M <= kOneGroupRows) {
        extend_kernel<<<dim3(1), dim3(kThreads), 0, s>>>(a);
    } else {
        extend_requests_kernel<<<dim3(1), dim3(kThreads), 0, s>>>(a);
        extend_rows_kernel<<<dim3((unsigned)((a.M + 255) / 256)), dim3(256), 0, s>>>(a);
    }
    return hipGetLastError();
}

int64_t kv_release_groups(int64_t B) { return (B + kOf - 1) / kOf; }

hipError_t launch_kv_release(const ReleaseArgs& a, hipStream_t s) {
    const dim3 grid((unsigned)kv_release_groups(a.B)), block(kThreads);
    release_count_kernel<<<grid, block, 0, s>>>(a);
    release_move_kernel<<<grid, block, 0, s>>>(a);
    return hipGetLastError();
}

}  // namespace nvfp4
