// Block tables, row starts, positions and slots of a batch, built on the GPU
// from the requests' lengths; the blocks of finished requests given back; and the
// rows that no request has cleared.
// All of it is integers, a few bytes for each row and request: what takes the
// time is the chain of loads that depend on one another, and the launches.
#include "kv_device.h"

namespace nvfp4 {
namespace {

constexpr int kThreads = 1024, kWaves = kThreads / 64;
template <int V>
struct Int {
    static constexpr int value = V;
};

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

// Inclusive sum, or maximum, over a wave's lanes of what `combine` joins.
template <class Combine>
__device__ __forceinline__ uint32_t wave_scan(uint32_t x, Combine combine) {
    const auto from = [&](auto control, auto rows) {
        return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, decltype(control)::value, decltype(rows)::value, 0xF, false);
    };
    x = combine(x, from(Int<0x111>(), Int<0xF>()));  // 1, 2, 4 and 8 lanes before, within rows of 16
    x = combine(x, from(Int<0x112>(), Int<0xF>()));
    x = combine(x, from(Int<0x114>(), Int<0xF>()));
    x = combine(x, from(Int<0x118>(), Int<0xF>()));
    x = combine(x, from(Int<0x142>(), Int<0xA>()));  // the row before's last, then the half before's
    x = combine(x, from(Int<0x143>(), Int<0xC>()));
    return x;
}
// The same over the workgroup's threads: what comes before each of them, and all.
// 0 joined to anything is that.  The slots are the scan's own.
template <class Combine>
__device__ __forceinline__ uint32_t group_scan32(uint32_t x, uint32_t* slot, uint32_t& all, Combine combine) {
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    const uint32_t mine = wave_scan(x, combine);
    if (lane == 63) slot[wave] = mine;
    const uint32_t up = (uint32_t)__shfl_up((int)mine, 1);
    __syncthreads();
    uint32_t before = 0;
    all = 0;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
        const uint32_t v = slot[w];
        before = w < wave ? combine(before, v) : before;
        all = combine(all, v);
    }
    return lane == 0 ? before : combine(before, up);
}
__device__ __forceinline__ uint32_t add_up(uint32_t x, uint32_t y) { return __builtin_elementwise_add_sat(x, y); }
__device__ __forceinline__ uint32_t larger(uint32_t x, uint32_t y) { return x > y ? x : y; }

// Blocks that `len` positions take of a table.
__device__ __forceinline__ int32_t blocks_of(int64_t len, int64_t table_blocks) {
    return (int32_t)clamp64(len <= 0 ? 0 : (len + kKvBlock - 1) / kKvBlock, 0, table_blocks);
}

// ---------------------------------------------------------------------------
// Extending.  The requests come first: rows and blocks of each, as running sums.
// Then the rows: each finds its request, and the row that starts a block writes
// the table's entry.  A block's number comes from the sums alone, so rows of one
// block need not wait for one another.
//
// Up to 4096 requests, every workgroup takes the sums of all of them by itself,
// into LDS, and then its 4096 rows: one launch.  A request marks its first row,
// and a running maximum over the rows finds each row's request (a search for each
// took 12 us where this takes 8).  What it costs is the chain of loads (past; a
// request's last block; free blocks): 32 tokens 4.2 us in a graph, a million rows
// of 1001 requests 8.2, 12 MB written; 4096 tokens 11 (19 in two launches).  A step
// in place whose rows need several workgroups, of which one writes what the others
// read, and more requests than that take a launch for the sums and one for the rows.
// ---------------------------------------------------------------------------
// Requests b .. b + R - 1 of a thread: what they get, and the sums before them.
template <int R>
struct Asked {
    int32_t past[R];
    int32_t first[R], rows[R];    // rows given
    int32_t taken[R], blocks[R];  // blocks that the requests before take, and they
};
// The requests before a round, and after it all of them.
struct Sums {
    uint32_t rows, blocks;  // rows stop at 2^32 - 1, far above M
};

template <int R>
__device__ __forceinline__ Asked<R> ask(const ExtendArgs& a, int64_t b, Sums& sums, uint32_t (&slot)[2][kWaves]) {
    Asked<R> q;
    const int32_t M = (int32_t)a.M;
    uint32_t want[R], rows = 0, blocks = 0, all;
#pragma unroll
    for (int i = 0; i < R; ++i) {
        q.past[i] = b + i < a.B ? a.past[b + i] : 0;
        const int32_t asked = b + i < a.B ? a.more[b + i] : 0, room = INT32_MAX - (q.past[i] > 0 ? q.past[i] : 0);
        want[i] = asked < 0 ? 0 : asked < room ? asked : room;
        rows = add_up(rows, want[i]);
    }
    uint32_t start = add_up(sums.rows, group_scan32(rows, slot[0], all, add_up));
    sums.rows = add_up(sums.rows, all);
#pragma unroll
    for (int i = 0; i < R; ++i) {
        q.first[i] = start < (uint32_t)M ? (int32_t)start : M;
        q.rows[i] = want[i] < (uint32_t)(M - q.first[i]) ? (int32_t)want[i] : M - q.first[i];
        q.blocks[i] = blocks_of((int64_t)q.past[i] + q.rows[i], a.table_blocks) - blocks_of(q.past[i], a.table_blocks);
        start = add_up(start, want[i]);
        blocks += (uint32_t)q.blocks[i];
    }
    uint32_t taken = sums.blocks + group_scan32(blocks, slot[1], all, add_up);
    sums.blocks += all;
#pragma unroll
    for (int i = 0; i < R; ++i) {
        q.taken[i] = (int32_t)taken;
        taken += (uint32_t)q.blocks[i];
    }
    return q;
}

template <int R>
__device__ __forceinline__ void write_asked(const ExtendArgs& a, int64_t b, const Asked<R>& q) {
#pragma unroll
    for (int i = 0; i < R; ++i)
        if (b + i < a.B) {
            a.row_start[b + i + 1] = q.first[i] + q.rows[i];
            a.lens[b + i] = q.past[i] + q.rows[i];
        }
}
__device__ __forceinline__ void write_stack(const ExtendArgs& a, int64_t had, int64_t blocks) {
    a.row_start[0] = 0;
    *a.free_left = (int32_t)(had > blocks ? had - blocks : 0);
    *a.missing = (int32_t)(blocks > had ? blocks - had : 0);
}

// Position, and slot, of a row of a request; the table's entry where it starts a
// block.  last: the entry of the request's last block, where that has room left.
__device__ __forceinline__ void write_row(const ExtendArgs& a, int64_t row, int64_t b, int64_t past, int64_t first,
                                          int64_t taken, int64_t had, int32_t last) {
    const int64_t pos = past + row - first, at = floor_div(pos, kKvBlock);
    int64_t slot = -1;
    if (pos >= 0 && at < a.table_blocks) {
        const int64_t fresh = at - blocks_of(past, a.table_blocks), place = had - 1 - taken - fresh;
        const int32_t page = fresh < 0 ? last : place >= 0 ? a.free_blocks[place] : -1;
        if (fresh >= 0 && pos % kKvBlock == 0) a.table[b * a.ld_table + at] = page;
        slot = page < 0 ? -1 : (int64_t)page * kKvBlock + pos % kKvBlock;
    }
    if (a.positions) a.positions[row] = (int32_t)pos;
    if (a.slots) a.slots[row] = slot;
}
__device__ __forceinline__ void write_no_row(const ExtendArgs& a, int64_t row) {
    if (a.positions) a.positions[row] = -1;
    if (a.slots) a.slots[row] = -1;
}
// Column of the block that a request's next position falls into, where it has begun.
__device__ __forceinline__ int64_t last_column(const ExtendArgs& a, int64_t past) {
    return past > 0 && past % kKvBlock != 0 && past / kKvBlock < a.table_blocks ? past / kKvBlock : -1;
}

constexpr int kMostEach = 4;  // requests of a thread
constexpr int kRowsEach = 4;
constexpr int kGroupRows = kThreads * kRowsEach;

// What a row needs of its request.
struct __align__(16) Request {
    int32_t shift;    // its position minus the row
    int32_t first;    // first column that is not held
    int32_t top;      // place on the stack of column 0, were it taken like the others
    int32_t last;     // the entry of the block that has room left
};

template <int R>
__global__ __launch_bounds__(kThreads) void extend_kernel(ExtendArgs a) {
    __shared__ uint32_t slot[2][kWaves], rows_slot[kWaves];
    __shared__ Request request[kThreads * R];
    __shared__ __align__(16) uint32_t mark[kGroupRows];  // request + 1 at its first row here
    const int32_t had = (int32_t)clamp64(*a.free_count, 0, a.capacity);
    const int t = threadIdx.x, b0 = R * t;
    const int32_t row0 = (int32_t)(blockIdx.x * kGroupRows), M = (int32_t)a.M;
    *reinterpret_cast<uint4*>(&mark[kRowsEach * t]) = make_uint4(0, 0, 0, 0);
    // the requests' last entries are on their way while the sums are taken
    int32_t entry[R];
#pragma unroll
    for (int i = 0; i < R; ++i) {
        const int64_t column = b0 + i < a.B ? last_column(a, a.past[b0 + i]) : -1;
        entry[i] = column >= 0 ? a.table[(b0 + i) * a.ld_table + column] : -1;
    }
    Sums sums = {0, 0};
    const Asked<R> q = ask<R>(a, b0, sums, slot);
#pragma unroll
    for (int i = 0; i < R; ++i) {
        // a position's shift wraps where past - first leaves 32 bits, and back where the row is added
        const int32_t have = blocks_of(q.past[i], a.table_blocks), first = q.first[i];
        request[b0 + i] = Request{(int32_t)((uint32_t)q.past[i] - (uint32_t)first), have, had - 1 - q.taken[i] + have, entry[i]};
        if (q.rows[i] > 0 && first + q.rows[i] > row0 && first < row0 + kGroupRows)
            mark[first > row0 ? first - row0 : 0] = b0 + i + 1;
    }
    if (blockIdx.x == 0) {
        write_asked<R>(a, b0, q);
        if (t == 0) write_stack(a, had, sums.blocks);
    }
    __syncthreads();
    const uint4 marks = *reinterpret_cast<const uint4*>(&mark[kRowsEach * t]);
    uint32_t of[kRowsEach] = {marks.x, marks.y, marks.z, marks.w};
#pragma unroll
    for (int i = 1; i < kRowsEach; ++i) of[i] = larger(of[i], of[i - 1]);
    uint32_t none;
    const uint32_t before = group_scan32(of[kRowsEach - 1], rows_slot, none, larger);
    const int32_t used = sums.rows < (uint32_t)M ? (int32_t)sums.rows : M;
    int32_t position[kRowsEach];
    int64_t where[kRowsEach];
#pragma unroll
    for (int i = 0; i < kRowsEach; ++i) {
        const int32_t row = row0 + kRowsEach * t + i;
        const uint32_t b = larger(of[i], before);
        position[i] = -1;
        where[i] = -1;
        if (row >= used || b == 0) continue;
        const Request of_row = request[b - 1];
        const int32_t pos = (int32_t)((uint32_t)of_row.shift + (uint32_t)row), at = pos >> 6;
        position[i] = pos;
        if (pos < 0 || at >= a.table_blocks) continue;
        int32_t page = of_row.last;
        if (at >= of_row.first) {
            page = of_row.top - at >= 0 ? a.free_blocks[of_row.top - at] : -1;
            if (pos % kKvBlock == 0) a.table[(b - 1) * a.ld_table + at] = page;
        }
        where[i] = page < 0 ? -1 : (int64_t)page * kKvBlock + pos % kKvBlock;
    }
    const int32_t mine = row0 + kRowsEach * t;
    const bool whole = mine + kRowsEach <= M;
    if (a.positions) {
        if (whole && ((uintptr_t)a.positions & 15) == 0) {
            *reinterpret_cast<int4*>(a.positions + mine) = make_int4(position[0], position[1], position[2], position[3]);
        } else {
#pragma unroll
            for (int i = 0; i < kRowsEach; ++i)
                if (mine + i < M) a.positions[mine + i] = position[i];
        }
    }
    if (a.slots) {
        if (whole && ((uintptr_t)a.slots & 15) == 0) {
            typedef int64_t i64x2 __attribute__((ext_vector_type(2)));
            i64x2* p = reinterpret_cast<i64x2*>(a.slots + mine);
            p[0] = i64x2{where[0], where[1]};
            p[1] = i64x2{where[2], where[3]};
        } else {
#pragma unroll
            for (int i = 0; i < kRowsEach; ++i)
                if (mine + i < M) a.slots[mine + i] = where[i];
        }
    }
}

__global__ __launch_bounds__(kThreads) void extend_requests_kernel(ExtendArgs a) {
    __shared__ uint32_t slot[2][kWaves];
    const int64_t had = clamp64(*a.free_count, 0, a.capacity);
    Sums sums = {0, 0};
    for (int64_t b0 = kMostEach * (int64_t)threadIdx.x; b0 - kMostEach * (int64_t)threadIdx.x < a.B; b0 += kThreads * kMostEach) {
        const Asked<kMostEach> q = ask<kMostEach>(a, b0, sums, slot);
        write_asked<kMostEach>(a, b0, q);
#pragma unroll
        for (int i = 0; i < kMostEach; ++i)
            if (b0 + i < a.B) a.taken[b0 + i] = q.taken[i];
    }
    if (threadIdx.x == 0) {
        a.state[0] = (int32_t)had;
        write_stack(a, had, sums.blocks);
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

__global__ __launch_bounds__(256) void extend_rows_kernel(ExtendArgs a) {
    const int64_t row0 = ((int64_t)blockIdx.x * 4 + (threadIdx.x >> 6)) * 64, row = row0 + (threadIdx.x & 63);
    if (row0 >= a.M) return;
    const int32_t used = a.row_start[a.B];
    if (row0 >= used) {
        if (row < a.M) write_no_row(a, row);
        return;
    }
    const int64_t b = request_of(a, row < used ? row : used - 1, row0);
    if (row >= a.M) return;
    if (row >= used) {
        write_no_row(a, row);
        return;
    }
    const int64_t first = a.row_start[b], past = a.lens[b] - (a.row_start[b + 1] - first), column = last_column(a, past);
    write_row(a, row, b, past, first, a.taken[b], a.state[0], column >= 0 ? a.table[b * a.ld_table + column] : -1);
}

// ---------------------------------------------------------------------------
// Releasing.  A wave takes a few requests: their tables' entries, 64 at a time,
// the first ones of all of them in flight together and kept in registers.  Their
// places on the stack follow from how many blocks the requests before give back:
// one workgroup finds that out in LDS, several of them by a launch that counts
// before the one that moves.  32 requests 4.3 us in a graph, 4099 requests 9.7 (one
// after the other by a wave, tables read twice: 11.4 and 17.5).
// ---------------------------------------------------------------------------
constexpr int kEach = 2;                 // requests of a wave
constexpr int kKept = 4;                 // times 64 entries of each that it keeps
constexpr int kOf = kEach * kWaves;      // requests of a workgroup

struct Released {
    int32_t blocks[kEach];        // entries [keep, blocks) of each
    int32_t page[kEach][kKept];   // this lane's of the first ones, -1 for none
    int32_t lens[kEach];          // what is left of each
    int64_t count[kEach];         // blocks given back
};

__device__ __forceinline__ int32_t entry_of(const ReleaseArgs& a, int64_t b, int64_t at, int32_t blocks) {
    const int32_t page = at < blocks ? a.table[b * a.ld_table + at] : -1;
    return page < 0 ? -1 : page;
}

__device__ __forceinline__ Released take(const ReleaseArgs& a, int64_t b0) {
    const int lane = threadIdx.x & 63;
    Released r;
    int32_t done[kEach];
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
        done[i] = b0 + i < a.B ? a.done[b0 + i] : 0;
        r.lens[i] = b0 + i < a.B ? a.lens[b0 + i] : 0;
    }
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
        r.blocks[i] = done[i] != 0 ? blocks_of(r.lens[i], a.table_blocks) : 0;
        r.lens[i] = done[i] != 0 ? a.done_len : r.lens[i];
#pragma unroll
        for (int k = 0; k < kKept; ++k) r.page[i][k] = entry_of(a, b0 + i, a.keep + 64 * k + lane, r.blocks[i]);
    }
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
        r.count[i] = 0;
#pragma unroll
        for (int k = 0; k < kKept; ++k) r.count[i] += __popcll(__ballot(r.page[i][k] >= 0));
        for (int64_t at = a.keep + 64 * kKept; at < r.blocks[i]; at += 64)
            r.count[i] += __popcll(__ballot(entry_of(a, b0 + i, at + lane, r.blocks[i]) >= 0));
    }
    return r;
}

// Puts them on the stack from `place` on.
__device__ __forceinline__ void give(const ReleaseArgs& a, int64_t b0, const Released& r, int64_t place) {
    const int lane = threadIdx.x & 63;
    const auto put = [&](int32_t page) {
        const uint64_t good = __ballot(page >= 0);
        const int64_t at = place + __popcll(good & (((uint64_t)1 << lane) - 1));
        if (page >= 0 && at < a.capacity) a.free_blocks[at] = page;
        place += __popcll(good);
    };
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
#pragma unroll
        for (int k = 0; k < kKept; ++k) put(r.page[i][k]);
        for (int64_t at = a.keep + 64 * kKept; at < r.blocks[i]; at += 64) put(entry_of(a, b0 + i, at + lane, r.blocks[i]));
        if (b0 + i < a.B && lane == 0) a.lens_out[b0 + i] = r.lens[i];
    }
}

// What the waves before this one give back, and all of them.
__device__ __forceinline__ int64_t waves_before(const Released& r, int64_t* share, int64_t& all) {
    const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    int64_t mine = 0;
#pragma unroll
    for (int i = 0; i < kEach; ++i) mine += r.count[i];
    if ((threadIdx.x & 63) == 0) share[wave] = mine;
    __syncthreads();
    int64_t before = 0;
    all = 0;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
        before += w < wave ? share[w] : 0;
        all += share[w];
    }
    return before;
}

__device__ __forceinline__ int64_t first_request() {
    return (int64_t)blockIdx.x * kOf + __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6)) * kEach;
}

__global__ __launch_bounds__(kThreads) void release_count_kernel(ReleaseArgs a) {
    __shared__ int64_t share[kWaves];
    int64_t all;
    waves_before(take(a, first_request()), share, all);
    if (threadIdx.x == 0) {
        a.totals[blockIdx.x] = all;
        if (blockIdx.x == 0) a.state[0] = *a.free_count;
    }
}

// count: where the stack's size is, a copy of it where several workgroups read it.
__global__ __launch_bounds__(kThreads) void release_move_kernel(ReleaseArgs a, const int32_t* count) {
    __shared__ int64_t share[kWaves], slot[kWaves];
    const int64_t had = clamp64(*count, 0, a.capacity);
    // what the workgroups before give back, and all that are launched
    int64_t before = 0, others = 0;
    if (gridDim.x > 1) {
        for (int64_t i = threadIdx.x; i < gridDim.x; i += kThreads) {
            const int64_t n = a.totals[i];
            before += i < blockIdx.x ? n : 0;
            others += i != blockIdx.x ? n : 0;
        }
        int64_t sum;
        group_scan(before, slot, sum);
        before = sum;
        group_scan(others, slot, sum);
        others = sum;
    }
    const Released r = take(a, first_request());
    int64_t all;
    const int64_t waves = waves_before(r, share, all);
    give(a, first_request(), r, had + before + waves);
    if (blockIdx.x == 0 && threadIdx.x == 0) *a.free_left = (int32_t)clamp64(had + others + all, 0, a.capacity);
}

// ---------------------------------------------------------------------------
// Clearing.  A workgroup takes a row of no sequence at a time, 16 bytes a thread,
// as many whole heads at once as its threads hold.  Nothing to clear: two loads
// and the launch.
// ---------------------------------------------------------------------------
__global__ __launch_bounds__(256) void clear_rest_kernel(HeadsOut out, int64_t M, int32_t pieces, int32_t heads,
                                                         const int32_t* row_start, int64_t B) {
    const RowRange used = row_range(row_start[0], row_start[B], M);
    const int64_t rest = M - (used.last - used.first);
    const int32_t together = 256 / pieces, first = (int32_t)threadIdx.x / pieces, piece = (int32_t)threadIdx.x % pieces;
    if (first >= together) return;
    for (int64_t i = blockIdx.x; i < rest; i += gridDim.x) {
        const int64_t row = i < used.first ? i : i + (used.last - used.first);
        uint16_t* p = out.data + row * out.row + 8 * piece;
        for (int32_t h = first; h < heads; h += together) *reinterpret_cast<u32x4*>(p + h * out.head) = u32x4{0, 0, 0, 0};
    }
}

}  // namespace

hipError_t launch_kv_extend(const ExtendArgs& a, hipStream_t s) {
    const unsigned groups = (unsigned)((a.M + kGroupRows - 1) / kGroupRows);
    const bool in_place = a.lens == a.past || a.free_left == a.free_count;
    if (a.B <= kThreads * kMostEach && (groups == 1 || !in_place)) {
        if (a.B <= kThreads)
            extend_kernel<1><<<dim3(groups), dim3(kThreads), 0, s>>>(a);
        else
            extend_kernel<kMostEach><<<dim3(groups), dim3(kThreads), 0, s>>>(a);
    } else {
        extend_requests_kernel<<<dim3(1), dim3(kThreads), 0, s>>>(a);
        extend_rows_kernel<<<dim3((unsigned)((a.M + 255) / 256)), dim3(256), 0, s>>>(a);
    }
    return hipGetLastError();
}

int64_t kv_release_groups(int64_t B) { return (B + kOf - 1) / kOf; }

hipError_t launch_kv_release(const ReleaseArgs& a, hipStream_t s) {
    const dim3 grid((unsigned)kv_release_groups(a.B)), block(kThreads);
    if (grid.x > 1) release_count_kernel<<<grid, block, 0, s>>>(a);
    release_move_kernel<<<grid, block, 0, s>>>(a, grid.x > 1 ? a.state : a.free_count);
    return hipGetLastError();
}

hipError_t launch_kv_clear_rest(const HeadsOut& out, int64_t M, int32_t heads, int32_t dim, const int32_t* row_start, int64_t B,
                                hipStream_t s) {
    // 8 workgroups for each of 256 CUs, which take several rows where there are more
    clear_rest_kernel<<<dim3((unsigned)clamp64(M, 1, 2048)), dim3(256), 0, s>>>(out, M, dim / 8, heads, row_start, B);
    return hipGetLastError();
}

}  // namespace nvfp4
