// Attention over the paged 8-bit key/value cache:
//   o = sum_j p_j v_j / sum_j p_j,  p_j = exp(scale q.k_j - max),  j < limit(row),
// of all these j, of those in a window and the first ones, or of a prefix that
// many sequences share and of their own keys, joined.
//
// The rows of a tile are the queries of one sequence and one key/value head,
// (token, query head of the group) in that order, 32 to a wave.  Scores are
// formed transposed, S^T = K Q^T, so that a lane holds one query's scores and
// the softmax needs one exchange, between the lane's two halves of the keys.
//
// Keys are multiplied as they lie in the cache, 8-bit codes whose power of two
// the matrix instruction applies.  A query is split into two E4M3 numbers,
//   q 2^-e = hi + lo / 16,  2^e the row's power of two (amax <= 448 2^e),
// each rounded to nearest: bf16's 8 bits are 4 + 4, so the split is exact for
// elements of at least 2^-6 2^e and off by at most 2^-14 2^e below (the largest
// element is above 224 2^e, so by less than 2^-21 of it).  Two 8-bit products at twice the bf16
// rate cost what one bf16 product would, and the keys need no conversion.
//
// Values become bf16 (exact: code times a power of two) and are multiplied with
// probabilities rounded to bf16 (half a step is at most 2^-8 of each p; their
// sum is taken before that rounding).  Two bf16 halves of each p would double
// these products; as it is the outputs' error against 64 bits is 0.0021 to 0.0023
// of their size, where binary32 probabilities and the output's own rounding give
// 0.0016 to 0.0017.  (Through a window and over a prefix the rounded ones are
// summed: where a few keys have the weight the error was 0.0025, and is 0.0023.)
// Scores, maxima, sums and outputs are held in binary32.
#include "kv_device.h"

namespace nvfp4 {
namespace {

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

constexpr int kRows = kNarrowRows;  // rows of a wave
// Probabilities are taken against a reference that need not be the maximum:
// while the sum of a lane's 16 new ones stays below this, the reference stays.
constexpr float kMost = 256.0f;

__device__ __forceinline__ float neg_inf() { return __uint_as_float(0xFF800000u); }
__device__ __forceinline__ float quiet_nan() { return __uint_as_float(0x7FC00000u); }

// What the rows of a launch see of the past.
//   PLAIN   every key below their limit
//   WINDOW  of these, the last `window` positions and the first `sinks`
//   SHARED  rows of all sequences the blocks that they share (a.prefix), or rows
//           their own sequence's keys behind these
enum Mode { PLAIN, WINDOW, SHARED };

struct Tile {
    bool any;
    bool bad;         // a length that the table cannot hold, or that ends inside the shared blocks
    int64_t b;
    int64_t row0;     // first row of the sequence
    int32_t n;        // its new tokens
    int32_t first;    // first tile row, counted in the sequence
    int32_t rows;     // n * group
    int64_t len;
};

template <int MODE>
__device__ __forceinline__ Tile find_tile(const AttentionArgs& a, int64_t unit, int64_t T) {
    Tile t;
    t.any = false;
    const SeqArgs& q = a.seqs;
    if (MODE == SHARED && a.prefix) {
        // one run of rows, from the first sequence's to the last's
        const RowRange r = row_range(q.row_start[0], q.row_start[q.B], q.M);
        const int64_t rows = (r.last - r.first) * a.group;
        if (unit * T >= rows) return t;
        t.any = true;
        t.bad = false;
        t.b = 0;
        t.row0 = r.first;
        t.n = (int32_t)(r.last - r.first);
        t.first = (int32_t)(unit * T);
        t.rows = (int32_t)rows;
        t.len = a.shared * kKvBlock;
        return t;
    }
    const Located at = locate(q, unit, [&](int64_t row, int64_t b) { return tile_first(row, b, a.group, T, q.per_row); });
    t.b = at.b;
    const RowRange r = row_range(at.start, at.end, q.M);
    const int64_t n = r.last - r.first, local = unit - tile_first(r.first, t.b, a.group, T, q.per_row);
    if (local < 0 || local * T >= n * a.group) return t;
    t.any = true;
    t.row0 = r.first;
    t.n = (int32_t)n;
    t.first = (int32_t)(local * T);
    t.rows = (int32_t)(n * a.group);
    t.len = at.len;
    t.bad = kv_length_bad(t.len, q.table_blocks);
    if constexpr (MODE == SHARED) t.bad = t.bad || t.len - t.n < a.shared * kKvBlock;
    return t;
}

// What a lane knows of its row.
struct Row {
    bool valid;
    int64_t token;   // row of q and out
    int32_t head;    // query head
    int32_t limit;   // keys it sees
    int32_t low;     // WINDOW: the first of them that need not be one of the first positions
};

// Keys that token i of the sequence sees.
__device__ __forceinline__ int32_t limit_of(const AttentionArgs& a, const Tile& t, int32_t i) {
    return t.bad ? 0 : kv_limit((int32_t)t.len - t.n + i, (int32_t)t.len, a.causal);
}
// Keys that row rr of the sequence sees, the last row's past it.
__device__ __forceinline__ int32_t limit_of_row(const AttentionArgs& a, const Tile& t, int32_t rr) {
    const int32_t at = rr < t.rows ? rr : t.rows - 1;
    return limit_of(a, t, __builtin_amdgcn_readfirstlane(at / a.group));
}

// WINDOW: the first key inside the window of token i of the sequence, and of row
// rr, the last row's past it.
__device__ __forceinline__ int32_t low_of(const AttentionArgs& a, const Tile& t, int32_t i) {
    return t.bad ? 0 : kv_window_low((int32_t)t.len - t.n + i, a.window);
}
__device__ __forceinline__ int32_t low_of_row(const AttentionArgs& a, const Tile& t, int32_t rr) {
    const int32_t at = rr < t.rows ? rr : t.rows - 1;
    return low_of(a, t, __builtin_amdgcn_readfirstlane(at / a.group));
}

// A window's tile goes over the blocks that some of its rows see, no others: 32
// tokens of 32 query and 8 key/value heads through 4096 of up to 16,384 keys, 240 MB,
// take 49 us (all keys: 118), 4.9 TB/s; prompts of 12,000 rows through 1000 keys
// 207 to 224 us on different cards (all keys: 361); their 3032 tiles go over 15.2
// blocks each on average, for 13.3 full ones' worth of keys.  A path of its own for the blocks at a window's ends, which
// passes over 32 keys that a wave does not see, made these 256 (accumulators copied
// between the paths); tiles that begin at a common block and go round, so as to
// read the same ones at a time, changed nothing.
//
// The blocks that a tile goes over, in order: what it sees of the first ones, and
// then those from the one where `jump` leads.
struct Blocks {
    int32_t count, jump_at, jump;
    __device__ __forceinline__ int32_t operator[](int32_t i) const { return i < jump_at ? i : i + jump; }
};
// Of a tile whose last row sees `seen` keys and whose first row's window starts at low.
template <int MODE>
__device__ __forceinline__ Blocks blocks_of(const AttentionArgs& a, int32_t seen, int32_t low) {
    const int32_t n = (seen + kKvBlock - 1) / kKvBlock;
    if constexpr (MODE == WINDOW) {
        const KvWindowBlocks w = kv_window_blocks(n, low, a.sinks);
        return Blocks{w.count, w.first, w.skipped};
    }
    if constexpr (MODE == SHARED) {
        const int32_t skipped = a.prefix ? 0 : (int32_t)a.shared;
        return Blocks{n > skipped ? n - skipped : 0, 0, skipped};
    }
    return Blocks{n, n, 0};
}

// Whether some row whose window starts at `low` or before does not see all of the
// 64 keys from first_key that are below its limit.
__device__ __forceinline__ bool window_hides(const AttentionArgs& a, int32_t first_key, int32_t low) {
    const int32_t from = first_key > a.sinks ? first_key : a.sinks;
    return from < low && from < first_key + kKvBlock;
}

// Bits of the 64 keys from first_key that a row sees.
__device__ __forceinline__ uint64_t bits_below(int32_t n) { return n <= 0 ? 0 : n >= 64 ? ~(uint64_t)0 : ((uint64_t)1 << n) - 1; }
__device__ __forceinline__ uint64_t window_bits(const AttentionArgs& a, const Row& r, int32_t first_key) {
    return bits_below(r.limit - first_key) & (~bits_below(r.low - first_key) | bits_below(a.sinks - first_key));
}

template <int MODE>
__device__ __forceinline__ Row find_row(const AttentionArgs& a, const Tile& t, int32_t rr, int32_t kv_head) {
    Row r;
    r.valid = rr < t.rows;
    const int32_t at = r.valid ? rr : t.rows - 1;
    const int32_t i = at / a.group;
    r.token = t.row0 + i;
    r.head = kv_head * a.group + (at - i * a.group);
    r.limit = limit_of(a, t, i);
    r.low = MODE == WINDOW ? low_of(a, t, i) : 0;
    return r;
}

// A row of queries as second operands: hi and lo for each 64 dims, and the
// power bytes of the two.
template <int D>
struct Query {
    i32x8 hi[D / 64], lo[D / 64];
    int32_t power_hi, power_lo;
    bool nan;  // an element is not finite
};

// The row's bf16 elements as loaded: this half's 32 dims of each 64.  (Rows past
// the tile's end load its last row's.)
template <int D>
__device__ __forceinline__ void fetch_query(u32x4 (&w)[D / 16], const AttentionArgs& a, const Row& r) {
    const uint16_t* p = a.q.data + r.token * a.q.row + r.head * a.q.head + 32 * ((threadIdx.x & 63) >> 5);
#pragma unroll
    for (int k = 0; k < D / 64; ++k)
#pragma unroll
        for (int j = 0; j < 4; ++j) w[4 * k + j] = *reinterpret_cast<const u32x4*>(p + 64 * k + 8 * j);
}

template <int D>
__device__ __forceinline__ void split_query(Query<D>& f, const u32x4 (&w)[D / 16]) {
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < D / 16; ++j)
        m = pk_max_u16(m, pk_max_u16(pk_max_u16(mag2(w[j].x), mag2(w[j].y)), pk_max_u16(mag2(w[j].z), mag2(w[j].w))));
    m = fold_max(m);
    const uint32_t other = (uint32_t)__shfl_xor((int)m, 32);
    m = m > other ? m : other;
    f.nan = m >= 0x7F80u;
    uint32_t e = f.nan ? 127u : power_for(m);
    e = e < 5u ? 5u : e;  // the low part's power is 2^-4 of it
    f.power_hi = (int32_t)e;
    f.power_lo = (int32_t)(e - 4u);
    const float inv = power_inverse(e);
#pragma unroll
    for (int k = 0; k < D / 64; ++k)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const uint32_t v0 = w[4 * k + j / 2][2 * (j % 2)], v1 = w[4 * k + j / 2][2 * (j % 2) + 1];
            const float x0 = bf16_lo(v0) * inv, x1 = bf16_hi(v0) * inv, x2 = bf16_lo(v1) * inv, x3 = bf16_hi(v1) * inv;
            const uint32_t c = fp8_pack4(x0, x1, x2, x3);
            const auto v01 = __builtin_amdgcn_cvt_pk_f32_fp8((int)c, false);
            const auto v23 = __builtin_amdgcn_cvt_pk_f32_fp8((int)c, true);
            const uint32_t l = fp8_pack4((x0 - v01[0]) * 16.0f, (x1 - v01[1]) * 16.0f, (x2 - v23[0]) * 16.0f,
                                         (x3 - v23[1]) * 16.0f);
            f.hi[k][j] = f.nan ? 0 : (int)c;
            f.lo[k][j] = f.nan ? 0 : (int)l;
        }
}

__device__ __forceinline__ i32x8 pieces(u32x4 a, u32x4 b) {
    return i32x8{(int)a.x, (int)a.y, (int)a.z, (int)a.w, (int)b.x, (int)b.y, (int)b.z, (int)b.w};
}

__device__ __forceinline__ f32x16 mul_scores(i32x8 k, i32x8 q, f32x16 acc, int k_power, int q_power) {
    return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(k, q, acc, 0, 0, 0, k_power, 0, q_power);
}

__device__ __forceinline__ bf16x8 values_bf16(uint32_t a, uint32_t b, float scale) {
    const u32x4 w = u32x4{fp8_to_bf16x2<false>(a, scale), fp8_to_bf16x2<true>(a, scale),
                               fp8_to_bf16x2<false>(b, scale), fp8_to_bf16x2<true>(b, scale)};
    return __builtin_bit_cast(bf16x8, w);
}

// The value of the lane that holds the other half of this lane's row.
__device__ __forceinline__ float other_half(float x) {
    const uint32_t w = __float_as_uint(x);
    const auto r = __builtin_amdgcn_permlane32_swap(w, w, false, false);
    return __uint_as_float((threadIdx.x & 32) ? r[0] : r[1]);
}

// The running softmax of a lane's row.
struct Softmax {
    float m;  // reference, scaled, base 2: some earlier maximum, -inf before the first
    float l;  // sum of this half's p
};

// Probabilities of a tile of 32 keys in bf16, the second operands of two
// k-steps of the products with the values, and their sum.
template <int MODE>
__device__ __forceinline__ float probabilities(const f32x16& s, float scale_log2, float ref, bf16x8 (&p)[2]) {
    float sum[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        uint32_t w[4];
        float part[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float x = __builtin_amdgcn_exp2f(__builtin_fmaf(s[8 * k + 2 * i], scale_log2, -ref));
            const float y = __builtin_amdgcn_exp2f(__builtin_fmaf(s[8 * k + 2 * i + 1], scale_log2, -ref));
            part[i] = x + y;
            w[i] = pack_bf16x2(x, y);
        }
        if constexpr (MODE == PLAIN) {
            sum[k] = (part[0] + part[1]) + (part[2] + part[3]);
        } else {
            // what the products take is what is summed: where a few keys have most
            // of the weight, their roundings then cancel in the quotient (a key
            // alone gives its value exactly).  Two at an instruction
            sum[k] = 0.0f;
#pragma unroll
            for (int i = 0; i < 4; ++i)
                sum[k] = __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2, w[i]),
                                                         __builtin_bit_cast(bf16x2, 0x3F803F80u), sum[k], false);
        }
        p[k] = __builtin_bit_cast(bf16x8, u32x4{w[0], w[1], w[2], w[3]});
    }
    return sum[0] + sum[1];
}

// Accepts the probabilities of a tile, or takes them again against its maximum.
// A maximum for every tile would cost 16 comparisons and an exchange between the
// lanes, on the way from the scores to the exponentials; instead the sum, which
// is there anyway, tells when the reference is too low (more than kMost, or
// infinite, or NaN for the first tile, whose reference is -inf).  p and the sums
// are floating-point numbers: a reference below the maximum costs no precision.
template <int MODE, int NO>
__device__ __forceinline__ void accept(const f32x16& s, float scale_log2, float sum, Softmax& st, f32x16 (&o)[NO],
                                       bf16x8 (&p)[2]) {
    const uint64_t over = __ballot(!(sum <= kMost));
    if (over) {
        // row by row (either half's sum decides for both): the other rows keep
        // their references and get the same p again, so that a row's bytes do
        // not depend on what other rows see
        const bool raise = ((over | over >> 32) >> (threadIdx.x & 31)) & 1;
        float top = s[0];
#pragma unroll
        for (int i = 1; i < 16; ++i) top = fmaxf(top, s[i]);
        top = fmaxf(top, other_half(top)) * scale_log2;
        const float m = raise ? fmaxf(st.m, top) : st.m;
        const float alpha = m == neg_inf() ? 1.0f : __builtin_amdgcn_exp2f(st.m - m);
        st.m = m;
        st.l *= alpha;
#pragma unroll
        for (int d = 0; d < NO; ++d)
#pragma unroll
            for (int i = 0; i < 16; ++i) o[d][i] *= alpha;
        sum = probabilities<MODE>(s, scale_log2, m == neg_inf() ? 0.0f : m, p);  // nothing seen yet: all 0
    }
    st.l += sum;
}

// The power byte of a block's keys; the byte that stands for NaN where the block
// does not exist, so that whoever sees it gets NaN.
__device__ __forceinline__ int key_power(uint32_t loaded, bool good) { return good ? (int)clamp_power(loaded) : 255; }

// Scores of keys past the row's limit become -inf.  left: the limit counted
// from the tile's first key.
__device__ __forceinline__ void mask_scores(f32x16& s, int32_t left) {
    // against constants: 16 keys by name would be 16 registers held in the loop
    const int mine = left - 4 * (int)((threadIdx.x & 63) >> 5);
#pragma unroll
    for (int i = 0; i < 16; ++i)
        if (8 * (i / 4) + i % 4 >= mine) s[i] = neg_inf();
}

// WINDOW: and so do those before its window that are not among the first
// positions.  Bit k: whether the row sees the tile's key k.
__device__ __forceinline__ void mask_window(f32x16& s, uint32_t visible) {
    visible >>= 4 * ((threadIdx.x & 63) >> 5);
#pragma unroll
    for (int i = 0; i < 16; ++i) s[i] = visible & (1u << (8 * (i / 4) + i % 4)) ? s[i] : neg_inf();
}
// Of tile t of the 64 keys from first_key.
template <int MODE>
__device__ __forceinline__ void mask_tile(f32x16& s, const AttentionArgs& a, const Row& r, int32_t first_key, int t) {
    if constexpr (MODE == WINDOW)
        mask_window(s, (uint32_t)(window_bits(a, r, first_key) >> (32 * t)));
    else
        mask_scores(s, r.limit - first_key - 32 * t);
}

// 1 in each byte that is one of E4M3's NaN codes, as bf16 ones for the products,
// and a one for each key that is not masked.
__device__ __forceinline__ uint32_t fp8_nan_bytes(uint32_t w) {
    return (((w & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u) >> 7;
}
__device__ __forceinline__ bf16x8 ones_bf16(uint32_t a, uint32_t b) {
    constexpr uint32_t kOne = 0x3F80u;
    const auto two = [](uint32_t w) { return (w & 1u) * kOne | ((w >> 8) & 1u) * (kOne << 16); };
    return __builtin_bit_cast(bf16x8, u32x4{two(a), two(a >> 16), two(b), two(b >> 16)});
}
__device__ __forceinline__ bf16x8 seen_ones(const f32x16& s, int k) {
    u32x4 w;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        w[i] = (s[8 * k + 2 * i] != neg_inf() ? 0x3F80u : 0u) | (s[8 * k + 2 * i + 1] != neg_inf() ? 0x3F800000u : 0u);
    return __builtin_bit_cast(bf16x8, w);
}

// ---------------------------------------------------------------------------
// Narrow tiles: 32 rows to a workgroup of 4 waves that share out the blocks of
// keys, each with its own softmax, joined at the end through LDS; the keys of
// long sequences are shared out over workgroups too (parts).  For single tokens
// and other short row tiles.  Every lane loads its operands from the cache
// itself, 1 KB of neighbouring bytes a wave and load; keys of the next block
// are in flight while this one's softmax runs, values while its scores are
// formed.  Bound by memory: 32 single tokens of 32 query and 8 key/value heads
// over 1 to 16,384 keys each, 539 MB, take 114 us and 5 for the join, 4.6 TB/s
// of cache read; four over 65,536 keys 102 us, 5.3 TB/s.  With D = 128 all 256
// vector registers are in use and 3 spill (16 bytes of scratch a lane; through a
// window 1, 8 bytes); D = 64 takes up to 186 and spills none.
// ---------------------------------------------------------------------------
constexpr int kNarrowWaves = 4;

template <int D>
struct NarrowShared {
    alignas(16) float o[kNarrowWaves][kRows][D + 4];
    float m[kNarrowWaves][kRows], l[kNarrowWaves][kRows];
};

// Which tile, key/value head and piece of the keys a workgroup takes.
struct Place {
    uint32_t unit;
    int kv_head, part;
};

template <int D, int MODE>
__device__ __forceinline__ void narrow_tile(const AttentionArgs& a, NarrowShared<D>& share, const Place& place) {
    constexpr int kDT = D / 32, kK = D / 64;
    constexpr int kBytes = kKvBlock * D;
    auto& so = share.o;
    auto& sm = share.m;
    auto& sl = share.l;
    const int kv_head = place.kv_head, part = place.part;
    const uint32_t unit = place.unit;
    const Tile t = find_tile<MODE>(a, unit, kRows);
    if (!t.any) return;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    const int c = lane & 31, h = lane >> 5;
    const Row row = find_row<MODE>(a, t, t.first + c, kv_head);
    // keys that the tile's last row sees, and keys that all its rows see: limits
    // do not fall from row to row
    const int seen = __builtin_amdgcn_readlane(row.limit, kRows - 1), all = __builtin_amdgcn_readlane(row.limit, 0);
    const Blocks blocks = blocks_of<MODE>(a, seen, MODE == WINDOW ? __builtin_amdgcn_readlane(row.low, 0) : 0);
    const int low_last = MODE == WINDOW ? __builtin_amdgcn_readlane(row.low, kRows - 1) : 0;
    const BlockRange range = kv_part(blocks.count, part, a.parts);
    const int at0 = range.first + wave;
    u32x4 qw[D / 16];
    fetch_query<D>(qw, a, row);

    // Table entries and powers are loaded like the keys, a block ahead, and are
    // looked at when they are needed: a wait for one of them would be a wait for
    // every load before it.
    const int32_t* table = a.seqs.table + t.b * a.seqs.ld_table;
    const auto entry = [&](int at) { return table[blocks[at < range.last ? at : range.last - 1]]; };
    const auto page_of = [&](int32_t loaded) -> int64_t {
        const int32_t p = __builtin_amdgcn_readfirstlane(loaded);
        return p >= 0 && p < a.cache.blocks ? p : -1;
    };
    u32x4 kf[2][2 * kK];
    uint32_t kp_raw = 127, vp_raw = 127;
    const auto load_keys = [&](int64_t page) {
        const int64_t at = (page < 0 ? 0 : page) * a.cache.heads + kv_head;
        const uint8_t* p = a.cache.k + at * kBytes + (2 * h) * (kKvBlock * 16) + c * 16;
#pragma unroll
        for (int k = 0; k < kK; ++k)
#pragma unroll
            for (int tt = 0; tt < 2; ++tt)
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    kf[tt][2 * k + i] = *reinterpret_cast<const u32x4*>(p + (4 * k + i) * (kKvBlock * 16) + tt * 32 * 16);
        kp_raw = a.cache.k_power[at];
        vp_raw = a.cache.v_power[at];
    };
    int64_t page = -1;
    int32_t next = -1;
    if (at0 < range.last) {
        page = page_of(entry(at0));
        load_keys(page);
        next = entry(at0 + kNarrowWaves);
    }
    // the first keys are on their way while the queries are split
    Query<D> q;
    split_query<D>(q, qw);
    Softmax st = {neg_inf(), 0.0f};
    f32x16 o[kDT];
#pragma unroll
    for (int d = 0; d < kDT; ++d) o[d] = f32x16{};
    for (int at = at0; at < range.last; at += kNarrowWaves) {
        const bool good = page >= 0;
        u32x4 vf[kDT][2];
        {
            const uint8_t* p = a.cache.v + ((good ? page : 0) * a.cache.heads + kv_head) * kBytes + c * 16;
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int d = 0; d < kDT; ++d)
                    vf[d][u] = *reinterpret_cast<const u32x4*>(p + (2 * u + h) * (D * 16) + d * 32 * 16);
        }
        const int kp = key_power(kp_raw, good);
        const float vs = power_value(clamp_power(vp_raw));
        f32x16 s[2] = {f32x16{}, f32x16{}};
#pragma unroll
        for (int k = 0; k < kK; ++k) {
            const i32x8 f0 = pieces(kf[0][2 * k], kf[0][2 * k + 1]), f1 = pieces(kf[1][2 * k], kf[1][2 * k + 1]);
            s[0] = mul_scores(f0, q.hi[k], s[0], kp, q.power_hi);
            s[1] = mul_scores(f1, q.hi[k], s[1], kp, q.power_hi);
            s[0] = mul_scores(f0, q.lo[k], s[0], kp, q.power_lo);
            s[1] = mul_scores(f1, q.lo[k], s[1], kp, q.power_lo);
        }
        if (!good) {
#pragma unroll
            for (int d = 0; d < kDT; ++d)
#pragma unroll
                for (int u = 0; u < 2; ++u) vf[d][u] = u32x4{0, 0, 0, 0};
        }
        page = page_of(next);
        if (at + kNarrowWaves < range.last) {
            load_keys(page);
            next = entry(at + 2 * kNarrowWaves);
        }

        const int first_key = blocks[at] * kKvBlock;
        const bool edge = first_key + kKvBlock > all || (MODE == WINDOW && window_hides(a, first_key, low_last));
        if (edge) {
            mask_tile<MODE>(s[0], a, row, first_key, 0);
            mask_tile<MODE>(s[1], a, row, first_key, 1);
        }
        if (edge) {
            // A masked key has p = 0, but 0 times a NaN value is NaN: NaN codes
            // are taken out and given back to the rows that see their key.
            bool nan = false;
#pragma unroll
            for (int d = 0; d < kDT; ++d)
#pragma unroll
                for (int u = 0; u < 2; ++u)
                    nan |= fp8_any_nan(vf[d][u].x) || fp8_any_nan(vf[d][u].y) || fp8_any_nan(vf[d][u].z) ||
                           fp8_any_nan(vf[d][u].w);
            if (!__any(nan)) {
                // as almost always
            } else if constexpr (MODE != PLAIN) {
                // which keys a row sees, times which are NaN, tells it
#pragma unroll
                for (int d = 0; d < kDT; ++d) {
                    f32x16 hit = f32x16{};
                    asm volatile("" : "+v"(s[0]), "+v"(s[1]));  // taken anew for each, not held in registers
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        u32x4 nans;
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            nans[i] = fp8_nan_bytes(vf[d][u][i]);
                            vf[d][u][i] &= ~(nans[i] * 0xFFu);
                        }
#pragma unroll
                        for (int k = 0; k < 2; ++k)
                            hit = __builtin_amdgcn_mfma_f32_32x32x16_bf16(ones_bf16(nans[2 * k], nans[2 * k + 1]),
                                                                          seen_ones(s[u], k), hit, 0, 0, 0);
                    }
#pragma unroll
                    for (int i = 0; i < 16; ++i) o[d][i] = hit[i] > 0.0f ? quiet_nan() : o[d][i];
                }
            } else {
                int half = h;  // opaque: nothing of this rare path is worth registers in the loop
                asm volatile("" : "+v"(half));
#pragma unroll
                for (int d = 0; d < kDT; ++d) {
                    int lowest = kKvBlock;  // first key of this lane's dim with a NaN
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        uint32_t w[4] = {vf[d][u].x, vf[d][u].y, vf[d][u].z, vf[d][u].w};
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            const uint32_t code = (w[i / 4] >> (8 * (i % 4))) & 0x7Fu;
                            if (code == 0x7Fu) {
                                const int key = 32 * u + 16 * (i / 8) + 8 * (i / 4 % 2) + 4 * half + i % 4;
                                lowest = key < lowest ? key : lowest;
                                w[i / 4] &= ~(0xFFu << (8 * (i % 4)));
                            }
                        }
                        vf[d][u] = u32x4{w[0], w[1], w[2], w[3]};
                    }
                    const int other = __shfl_xor(lowest, 32);
                    lowest = lowest < other ? lowest : other;
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const int key = __shfl(lowest, 8 * (i / 4) + 4 * half + i % 4);
                        if (key < row.limit - first_key && key < kKvBlock) o[d][i] = quiet_nan();
                    }
                }
            }
        }
#pragma unroll
        for (int tt = 0; tt < 2; ++tt) {
            bf16x8 p[2];
            const float sum = probabilities<MODE>(s[tt], a.scale_log2, st.m, p);
            accept<MODE, kDT>(s[tt], a.scale_log2, sum, st, o, p);
#pragma unroll
            for (int k = 0; k < 2; ++k)
#pragma unroll
                for (int d = 0; d < kDT; ++d) {
                    const u32x4 w = vf[d][tt];
                    o[d] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(
                        k ? values_bf16(w.z, w.w, vs) : values_bf16(w.x, w.y, vs), p[k], o[d], 0, 0, 0);
                }
        }
    }

    // join the waves: each row's largest maximum is the common reference
    st.l += __shfl_xor(st.l, 32);
    if (q.nan && row.limit > 0) st.l = quiet_nan();
    if (h == 0) {
        sm[wave][c] = st.m;
        sl[wave][c] = st.l;
    }
#pragma unroll
    for (int d = 0; d < kDT; ++d)
#pragma unroll
        for (int i = 0; i < 4; ++i)
            *reinterpret_cast<float4*>(&so[wave][c][32 * d + 8 * i + 4 * h]) =
                make_float4(o[d][4 * i], o[d][4 * i + 1], o[d][4 * i + 2], o[d][4 * i + 3]);
    __syncthreads();
    constexpr int kEach = D / 8;  // dims of a thread: 8 threads a row
    const int rr = threadIdx.x >> 3, d0 = (threadIdx.x & 7) * kEach;
    const Row mine = find_row<MODE>(a, t, t.first + rr, kv_head);
    if (!mine.valid) return;
    float m = sm[0][rr];
#pragma unroll
    for (int w = 1; w < kNarrowWaves; ++w) m = fmaxf(m, sm[w][rr]);
    const float ref = m == neg_inf() ? 0.0f : m;
    float l = 0.0f, acc[kEach];
#pragma unroll
    for (int i = 0; i < kEach; ++i) acc[i] = 0.0f;
#pragma unroll
    for (int w = 0; w < kNarrowWaves; ++w) {
        const float f = __builtin_amdgcn_exp2f(sm[w][rr] - ref);  // 0 for a wave that saw nothing
        const float lw = sl[w][rr];
        l += lw != lw ? lw : f * lw;
#pragma unroll
        for (int i = 0; i < kEach; ++i) acc[i] += f * so[w][rr][d0 + i];
    }
    const int64_t at = mine.token * a.q_heads + mine.head;
    if (a.all_parts == 1) {
        // no key: 0; a length that the table cannot hold: NaN
        const float inv = t.bad ? quiet_nan() : l == 0.0f ? 0.0f : 1.0f / l;
        uint16_t* p = a.out.data + mine.token * a.out.row + mine.head * a.out.head + d0;
#pragma unroll
        for (int i = 0; i < kEach; i += 8)
            *reinterpret_cast<u32x4*>(p + i) =
                u32x4{pack_bf16x2(acc[i] * inv, acc[i + 1] * inv), pack_bf16x2(acc[i + 2] * inv, acc[i + 3] * inv),
                           pack_bf16x2(acc[i + 4] * inv, acc[i + 5] * inv), pack_bf16x2(acc[i + 6] * inv, acc[i + 7] * inv)};
    } else {
        const int64_t all_rows = a.seqs.M * a.q_heads;
        const int64_t piece = (int64_t)(a.first_part + part) * all_rows + at;
        float* po = a.partial + piece * D + d0;
        float* pm = a.partial + (int64_t)a.all_parts * all_rows * D + piece * 2;
#pragma unroll
        for (int i = 0; i < kEach; i += 4)
            *reinterpret_cast<float4*>(po + i) = make_float4(acc[i], acc[i + 1], acc[i + 2], acc[i + 3]);
        if ((threadIdx.x & 7) == 0) {
            pm[0] = m;
            pm[1] = t.bad ? quiet_nan() : l;
        }
    }
}

// Workgroups go to the 8 XCDs in turn: with a multiple of 8 units, all of a
// long sequence's would go to one of them, were heads and parts not turned
// against each other (32 sequences of 1 to 16,384 keys: 118 us, 124 without).
__device__ __forceinline__ Place narrow_place(uint32_t x, uint32_t y, uint32_t z, uint32_t units) {
    const uint32_t unit = x + (y + z) % units;
    return Place{unit < units ? unit : unit - units, (int)y, (int)z};
}

template <int D, int MODE>
__global__ __launch_bounds__(64 * kNarrowWaves, 2) void attention_narrow_kernel(AttentionArgs a) {
    __shared__ NarrowShared<D> share;
    narrow_tile<D, MODE>(a, share, narrow_place(blockIdx.x, blockIdx.y, blockIdx.z, gridDim.x));
}

// ---------------------------------------------------------------------------
// Wide tiles: 128 rows to a workgroup of 4 waves, 32 rows each, that go over
// the same blocks of keys together.  A block is staged in LDS while the one
// before it is worked on (two buffers, one barrier a block): keys as they are,
// values as bf16, converted once for all four waves.  Both lie in LDS in the
// order the lanes read them, 16 neighbouring bytes each, free of conflicts.
//
// 4096 rows of 56 heads over 37,810 keys: 3.7 to 4.1 ms on different cards, 1080
// to 1195 TFLOP/s, where a library product of 8192^3 in bf16 reaches 1229.  The
// matrix pipes are busy 56% of the cycles, and the card is at its power limit:
// with 10% fewer cycles for the same work its clock fell from 2.05 to 1.9 GHz.
// Wave priorities (raised for the products, or for every other wave) changed
// nothing; one workgroup to a CU instead of two took 5.2 ms.
// ---------------------------------------------------------------------------
constexpr int kWideWaves = 4;
static_assert(kWideRows == kWideWaves * kRows, "32 rows to a wave");

// Which tile and key/value head a workgroup takes.  Workgroups go to the 8 XCDs
// in turn; where the heads divide evenly over them, each XCD takes whole heads,
// so that the tiles in flight at a time read the same keys from its L2.  Tiles
// go from the last to the first: under a causal mask the later ones take
// longer, and the short ones fill the end.
__device__ __forceinline__ Place wide_place(uint32_t x, uint32_t z, uint32_t units, uint32_t heads) {
    if (heads % 8 == 0) {
        const uint32_t at = x / 8, head = at / units;
        return Place{units - 1 - (at - head * units), (int)((x % 8) * (heads / 8) + head), (int)z};
    }
    const uint32_t at = x / heads;
    return Place{units - 1 - at, (int)(x - at * heads), (int)z};
}

// Asks the compiler to lay MATRIX matrix instructions of a stretch of code out
// among VECTOR vector instructions.
template <int MATRIX, int VECTOR>
__device__ __forceinline__ void alternate() {
#pragma unroll
    for (int i = 0; i < MATRIX; ++i) {
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
        __builtin_amdgcn_sched_group_barrier(0x002, VECTOR / MATRIX, 0);
    }
}

template <int D, int MODE>
struct WideShared {
    static constexpr int kPieces = kKvBlock * D / 16;  // 16-byte pieces of a block's keys, and of its values
    static constexpr int kMarks = MODE == PLAIN ? 1 : 2;
    alignas(16) u32x4 k[2][kPieces];
    alignas(16) u32x4 v[2][2 * kPieces];               // [k-step][half][dim] of 8 keys
    // by dim, which keys' values are NaN codes: PLAIN the first of them, else the
    // bits of all, [half of the block][dim]
    int nan_key[2][kMarks * D];
    int nan_any[2];
};

template <int D, int MODE>
__device__ __forceinline__ void wide_tile(const AttentionArgs& a, WideShared<D, MODE>& share, const Place& place) {
    constexpr int kDT = D / 32, kK = D / 64;
    constexpr int kBytes = kKvBlock * D;
    constexpr int kThreads = 64 * kWideWaves;
    constexpr int kEach = WideShared<D, MODE>::kPieces / kThreads;  // pieces of a thread
    constexpr int kMarks = WideShared<D, MODE>::kMarks;
    constexpr int kNoMark = MODE == PLAIN ? kKvBlock : 0;
    auto& sk = share.k;
    auto& sv = share.v;
    auto& nan_key = share.nan_key;
    auto& nan_any = share.nan_any;
    const uint32_t unit = place.unit;
    const int kv_head = place.kv_head;
    const Tile t = find_tile<MODE>(a, unit, kWideRows);
    if (!t.any) return;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    const int c = lane & 31, h = lane >> 5;
    const int row0 = t.first + wave * kRows;
    const Row row = find_row<MODE>(a, t, row0 + c, kv_head);
    // keys that the tile's last row and this wave's last row see, and keys that
    // all rows of the tile and of the wave see
    const int tile_seen = limit_of_row(a, t, t.first + kWideRows - 1), tile_all = limit_of_row(a, t, t.first);
    const int seen = row0 < t.rows ? __builtin_amdgcn_readlane(row.limit, kRows - 1) : 0;
    const int all = __builtin_amdgcn_readlane(row.limit, 0);
    // where the windows of the tile's first and last rows and of this wave's start
    const int tile_low = MODE == WINDOW ? low_of_row(a, t, t.first) : 0;
    const int tile_low_last = MODE == WINDOW ? low_of_row(a, t, t.first + kWideRows - 1) : 0;
    const int low_first = MODE == WINDOW ? __builtin_amdgcn_readlane(row.low, 0) : 0;
    const int low_last = MODE == WINDOW ? __builtin_amdgcn_readlane(row.low, kRows - 1) : 0;
    const int part = place.part;
    const Blocks blocks = blocks_of<MODE>(a, tile_seen, tile_low);
    const BlockRange range = kv_part(blocks.count, part, a.parts);
    const int at0 = range.first, end = range.last;
    // whether some row of the tile does not see all of block i, and whether some row of this wave sees any of it
    const auto edge_of = [&](int i) {
        const int first_key = blocks[i] * kKvBlock;
        return first_key + kKvBlock > tile_all || (MODE == WINDOW && window_hides(a, first_key, tile_low_last));
    };
    const auto sees = [&](int first_key) {
        return first_key < seen && (MODE != WINDOW || first_key + kKvBlock > low_first || first_key < a.sinks);
    };

    u32x4 qw[D / 16];
    fetch_query<D>(qw, a, row);
    for (int i = threadIdx.x; i < 2 * kMarks * D; i += kThreads) nan_key[i / (kMarks * D)][i % (kMarks * D)] = kNoMark;
    if (threadIdx.x < 2) nan_any[threadIdx.x] = 0;

    // table entries and powers are looked at a block after they are asked for,
    // as in the narrow kernel
    const int32_t* table = a.seqs.table + t.b * a.seqs.ld_table;
    const auto entry = [&](int at) { return table[blocks[at < end ? at : end - 1]]; };
    const auto page_of = [&](int32_t loaded) -> int64_t {
        const int32_t p = __builtin_amdgcn_readfirstlane(loaded);
        return p >= 0 && p < a.cache.blocks ? p : -1;
    };
    u32x4 kr[kEach], vr[kEach];
    uint32_t kp_raw = 127, vp_raw = 127;
    const auto fetch = [&](int64_t page) {
        const int64_t at = (page < 0 ? 0 : page) * a.cache.heads + kv_head;
        const u32x4* pk = reinterpret_cast<const u32x4*>(a.cache.k + at * kBytes);
        const u32x4* pv = reinterpret_cast<const u32x4*>(a.cache.v + at * kBytes);
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
            kr[i] = pk[i * kThreads + threadIdx.x];
            vr[i] = pv[i * kThreads + threadIdx.x];
        }
        kp_raw = a.cache.k_power[at];
        vp_raw = a.cache.v_power[at];
    };
    // stages the fetched block; edge: some row of the tile does not see all of
    // it, or it stands in for one that does not exist (!good: then its power may
    // be anything and is not used, so that the rows that do not see it get 0 p)
    const auto stage = [&](int buffer, bool edge, bool good) {
        const float scale = power_value(good ? clamp_power(vp_raw) : 127u);
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
            const int at = i * kThreads + threadIdx.x;
            const int d = at % D, piece = at / D;         // piece 2u + half
            u32x4 w = vr[i];
            if (edge && (fp8_any_nan(w.x) || fp8_any_nan(w.y) || fp8_any_nan(w.z) || fp8_any_nan(w.w))) {
                // as in the narrow kernel: NaN codes are taken out, and given
                // back to the rows that see their key
                if constexpr (MODE != PLAIN) {
                    // dword i holds keys 8i + 4 (piece % 2) .. + 3 of half piece / 2
                    uint32_t mark = 0;
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const uint32_t nans = fp8_nan_bytes(w[j]);
                        w[j] &= ~(nans * 0xFFu);
                        mark |= ((nans | nans >> 7 | nans >> 14 | nans >> 21) & 0xFu) << (8 * j);
                    }
                    atomicOr(&nan_key[buffer][(piece / 2) * D + d], (int)(mark << (4 * (piece % 2))));
                } else {
                    uint32_t x[4] = {w.x, w.y, w.z, w.w};
                    int lowest = kKvBlock;
#pragma unroll
                    for (int j = 0; j < 16; ++j)
                        if (((x[j / 4] >> (8 * (j % 4))) & 0x7Fu) == 0x7Fu) {
                            const int key = 32 * (piece / 2) + 16 * (j / 8) + 8 * (j / 4 % 2) + 4 * (piece % 2) + j % 4;
                            lowest = key < lowest ? key : lowest;
                            x[j / 4] &= ~(0xFFu << (8 * (j % 4)));
                        }
                    w = u32x4{x[0], x[1], x[2], x[3]};
                    atomicMin(&nan_key[buffer][d], lowest);
                }
                nan_any[buffer] = 1;
            }
            sk[buffer][at] = kr[i];
            const int to = (4 * (piece / 2) + piece % 2) * D + d;   // k-step 2u; 2u + 1 is 2 D further on
            sv[buffer][to] = __builtin_bit_cast(u32x4, values_bf16(w.x, w.y, scale));
            sv[buffer][to + 2 * D] = __builtin_bit_cast(u32x4, values_bf16(w.z, w.w, scale));
        }
    };
    __syncthreads();  // the NaN marks are clear
    int32_t next = -1;
    int kp = 127;
    bool edge_now = false, first_good = false;
    if (at0 < end) {
        const int64_t page = page_of(entry(at0));
        fetch(page);
        next = entry(at0 + 1);
        edge_now = page < 0 || edge_of(at0);
        first_good = page >= 0;
    }
    // the first block is on its way while the queries are split
    Query<D> q;
    split_query<D>(q, qw);
    Softmax st = {neg_inf(), 0.0f};
    f32x16 o[kDT];
#pragma unroll
    for (int d = 0; d < kDT; ++d) o[d] = f32x16{};
    if (at0 < end) {
        stage(0, edge_now, first_good);
        kp = key_power(kp_raw, first_good);
    }
    __syncthreads();
    for (int at = at0; at < end; ++at) {
        const int b = (at - at0) & 1, first_key = blocks[at] * kKvBlock;
        const bool more = at + 1 < end;
        const int64_t page = page_of(next);
        if (more) {
            fetch(page);
            next = entry(at + 2);
        }
        if (sees(first_key)) {
            u32x4 kf[2][2 * kK];
#pragma unroll
            for (int k = 0; k < kK; ++k)
#pragma unroll
                for (int tt = 0; tt < 2; ++tt)
#pragma unroll
                    for (int i = 0; i < 2; ++i)
                        kf[tt][2 * k + i] = sk[b][(4 * k + 2 * h + i) * kKvBlock + tt * 32 + c];
            // Two tiles of 32 keys.  The second's scores are multiplied while the
            // first's exponentials are taken, and the first's products with the
            // values while the second's are: matrix and vector instructions of
            // one wave overlap where they alternate.
            const bool edge = first_key + kKvBlock > all || (MODE == WINDOW && window_hides(a, first_key, low_last));
            f32x16 s[2] = {f32x16{}, f32x16{}};
            const auto scores = [&](int tt) {
#pragma unroll
                for (int k = 0; k < kK; ++k) {
                    const i32x8 f = pieces(kf[tt][2 * k], kf[tt][2 * k + 1]);
                    s[tt] = mul_scores(f, q.hi[k], s[tt], kp, q.power_hi);
                    s[tt] = mul_scores(f, q.lo[k], s[tt], kp, q.power_lo);
                }
            };
            // values of a k-step are on their way while the one before is multiplied
            u32x4 vf[2][kDT];
            const auto values = [&](int ks) {
#pragma unroll
                for (int d = 0; d < kDT; ++d) vf[ks & 1][d] = sv[b][(2 * ks + h) * D + 32 * d + c];
            };
            const auto multiply = [&](int ks, bf16x8 p) {
#pragma unroll
                for (int d = 0; d < kDT; ++d)
                    o[d] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, vf[ks & 1][d]), p, o[d], 0, 0,
                                                                  0);
            };
            bf16x8 p0[2], p1[2];
            scores(0);
            values(0);
            __builtin_amdgcn_sched_barrier(0);
            if (edge) mask_tile<MODE>(s[0], a, row, first_key, 0);
            scores(1);
            const float sum0 = probabilities<MODE>(s[0], a.scale_log2, st.m, p0);
            values(1);
            alternate<2 * kK, 56>();
            asm volatile("" : "+v"(s[1]));  // issued here, not after the branch below
            accept<MODE, kDT>(s[0], a.scale_log2, sum0, st, o, p0);
            if (edge) mask_tile<MODE>(s[1], a, row, first_key, 1);
            multiply(0, p0[0]);
            values(2);
            multiply(1, p0[1]);
            const float sum1 = probabilities<MODE>(s[1], a.scale_log2, st.m, p1);
            values(3);
            alternate<2 * kDT, 56>();
            accept<MODE, kDT>(s[1], a.scale_log2, sum1, st, o, p1);
            multiply(2, p1[0]);
            multiply(3, p1[1]);
        }
        if (edge_now && nan_any[b]) {  // the same for all waves
            if (sees(first_key)) {
                int half = h;
                asm volatile("" : "+v"(half));
                const uint64_t visible = MODE == PLAIN ? 0 : window_bits(a, row, first_key);
#pragma unroll
                for (int d = 0; d < kDT; ++d)
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const int at_dim = 32 * d + 8 * (i / 4) + 4 * half + i % 4;
                        const int key = nan_key[b][at_dim];
                        if constexpr (MODE != PLAIN) {
                            const uint32_t hit = ((uint32_t)key & (uint32_t)visible) |
                                                 ((uint32_t)nan_key[b][(kMarks - 1) * D + at_dim] & (uint32_t)(visible >> 32));
                            if (hit) o[d][i] = quiet_nan();
                        } else {
                            if (key < kKvBlock && key < row.limit - first_key) o[d][i] = quiet_nan();
                        }
                    }
            }
            __syncthreads();
            for (int i = threadIdx.x; i < kMarks * D; i += kThreads) nan_key[b][i] = kNoMark;
            if (threadIdx.x == 0) nan_any[b] = 0;
        }
        if (more) {
            const bool good = page >= 0;
            edge_now = !good || edge_of(at + 1);
            stage(1 - b, edge_now, good);
            kp = key_power(kp_raw, good);
        }
        __syncthreads();
    }
    if (!row.valid) return;

    // no key: 0; a length that the table cannot hold, or a query that is not
    // finite: NaN
    float l = st.l + __shfl_xor(st.l, 32);
    if (q.nan && row.limit > 0) l = quiet_nan();
    if (t.bad) l = quiet_nan();
    if (a.all_parts > 1) {
        const int64_t all_rows = a.seqs.M * a.q_heads;
        const int64_t mine = (int64_t)(a.first_part + part) * all_rows + row.token * a.q_heads + row.head;
        float* po = a.partial + mine * D + 4 * h;
#pragma unroll
        for (int d = 0; d < kDT; ++d)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                *reinterpret_cast<float4*>(po + 32 * d + 8 * i) =
                    make_float4(o[d][4 * i], o[d][4 * i + 1], o[d][4 * i + 2], o[d][4 * i + 3]);
        if (h == 0)
            *reinterpret_cast<float2*>(a.partial + (int64_t)a.all_parts * all_rows * D + mine * 2) = make_float2(st.m, l);
        return;
    }
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
    uint16_t* out = a.out.data + row.token * a.out.row + row.head * a.out.head;
#pragma unroll
    for (int d = 0; d < kDT; ++d)
#pragma unroll
        for (int i = 0; i < 4; i += 2) {
            // this half has dims 8 i + 4 h .. + 3 of each i: the halves trade, and
            // each stores 8 dims
            uint32_t x0 = pack_bf16x2(o[d][4 * i] * inv, o[d][4 * i + 1] * inv);
            uint32_t x1 = pack_bf16x2(o[d][4 * i + 2] * inv, o[d][4 * i + 3] * inv);
            uint32_t y0 = pack_bf16x2(o[d][4 * i + 4] * inv, o[d][4 * i + 5] * inv);
            uint32_t y1 = pack_bf16x2(o[d][4 * i + 6] * inv, o[d][4 * i + 7] * inv);
            const auto r0 = __builtin_amdgcn_permlane32_swap(x0, y0, false, false);
            const auto r1 = __builtin_amdgcn_permlane32_swap(x1, y1, false, false);
            *reinterpret_cast<u32x4*>(out + 32 * d + 8 * i + 8 * h) = u32x4{r0[0], r1[0], r0[1], r1[1]};
        }
}

template <int D, int MODE>
__global__ __launch_bounds__(64 * kWideWaves, 2) void attention_wide_kernel(AttentionArgs a) {
    __shared__ WideShared<D, MODE> share;
    wide_tile<D, MODE>(a, share, wide_place(blockIdx.x, blockIdx.z, gridDim.x / a.cache.heads, a.cache.heads));
}

// ---------------------------------------------------------------------------
// A batch over a shared prefix: the first workgroups take tiles of all sequences'
// rows against pieces of the prefix, the others each sequence's rows against its
// own keys, in one launch, so that the loads of the one fill the waits of the
// other.  64 tokens of 32 query and 8 key/value heads, up to 1024 own keys each
// behind 16,384, 103 MB: 40 us and 5 for the join (two launches after one another
// 48 and 11; the prefix alone takes 32, the own keys alone 26); what is left is the
// prefix's blocks, one in flight at a time (1.2 us each with a CU to themselves, of
// which the matrix instructions are 0.41), the pieces' sums (13 of them, 14 MB written
// and read) and the chains of loads at both ends.  500 rows of 32 heads over 32,768: 304 to 335 us, 950 TFLOP/s, the matrix
// pipes busy 39% of the cycles: 432 workgroups for 512 places, and 18 tiles of 128
// rows that hold 17.5.
// Heads of 64 leave room for three workgroups on a CU, which many tiles of few keys
// use: 40 x 2 tokens of 36 and 12 heads behind 12,800 positions 30 us (33.5 with
// two), 30 x 4 of 16 and 16 heads behind 3840 13.7 (17.3).
// ---------------------------------------------------------------------------
template <int D, bool PREFIX_WIDE, bool OWN_WIDE>
__global__ __launch_bounds__(64 * kWideWaves, D == 64 ? 3 : 2) void attention_shared_kernel(AttentionArgs a, SharedGrid g) {
    static_assert(kNarrowWaves == kWideWaves, "one size of workgroup");
    __shared__ union {
        NarrowShared<D> narrow;
        WideShared<D, SHARED> wide;
    } share;
    uint32_t at = blockIdx.y * gridDim.x + blockIdx.x;
    const bool of_prefix = at < g.prefix_groups;
    // one way for both, with these taken by selects
    a.seqs.table = of_prefix ? g.shared : a.seqs.table;
    a.causal = of_prefix ? 0 : a.causal;
    a.parts = of_prefix ? a.first_part : a.parts;
    a.first_part = of_prefix ? 0 : a.first_part;
    a.prefix = of_prefix;
    const uint32_t units = of_prefix ? g.prefix_units : g.own_units, heads = a.cache.heads, each = units * heads;
    at -= of_prefix ? 0 : g.prefix_groups;
    if (!of_prefix && at >= g.own_groups) return;
    const uint32_t z = at / each, x = at - z * each;
    if (of_prefix ? PREFIX_WIDE : OWN_WIDE)
        wide_tile<D, SHARED>(a, share.wide, wide_place(x, z, units, heads));
    else
        narrow_tile<D, SHARED>(a, share.narrow, narrow_place(x % units, x / units, z, units));
}

// Joins the parts of each row; rows that no sequence has are left alone.  WAVES
// waves take a row: each has the maximum and sum of every part in its lanes
// (part s in lane s, at most 64), adds up its share of at most EACH parts, D / 64
// dims a lane, with all their loads in flight at once, and the first adds up
// the waves.  (64 parts of one wave's, eight loads at a time, took 12 us where
// the attention before it takes 25.)
constexpr int kMaxParts = 64;
constexpr int kOwnParts = 16;  // of them the sequences' own, behind a shared prefix

template <int D, int WAVES, int EACH>
__global__ __launch_bounds__(256) void attention_join_kernel(AttentionArgs a) {
    constexpr int kEach = D / 64;
    typedef float Dims __attribute__((ext_vector_type(kEach)));
    __shared__ Dims share[4][64];
    const int64_t all_rows = a.seqs.M * a.q_heads;
    const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6)), lane = threadIdx.x & 63;
    const int64_t at = ((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * (4 / WAVES) + wave / WAVES;
    if (at >= all_rows) return;  // whole workgroups, or with one wave a row: no barrier below
    const int64_t token = at / a.q_heads;
    const int32_t head = (int32_t)(at - token * a.q_heads);
    const int32_t first = a.seqs.row_start[0], last = a.seqs.row_start[a.seqs.B];
    const int mine = lane < a.all_parts ? lane : 0, own = wave % WAVES;
    const float2 ml = *reinterpret_cast<const float2*>(a.partial + a.all_parts * all_rows * D + (mine * all_rows + at) * 2);
    const float* po = a.partial + at * D + lane * kEach;
    Dims v[EACH];
#pragma unroll
    for (int i = 0; i < EACH; ++i) {
        const int s = own + i * WAVES;
        v[i] = *reinterpret_cast<const Dims*>(po + (s < a.all_parts ? s : 0) * all_rows * D);
    }
    if (token < first || token >= last) return;
    float m = lane < a.all_parts ? ml.x : neg_inf();
#pragma unroll
    for (int s = 32; s > 0; s >>= 1) m = fmaxf(m, __shfl_xor(m, s));
    const float w = lane < a.all_parts ? __builtin_amdgcn_exp2f(ml.x - (m == neg_inf() ? 0.0f : m)) : 0.0f;
    float l = lane >= a.all_parts ? 0.0f : ml.y != ml.y ? ml.y : w * ml.y;
#pragma unroll
    for (int s = 32; s > 0; s >>= 1) l += __shfl_xor(l, s);
    Dims acc = {};
#pragma unroll
    for (int i = 0; i < EACH; ++i) {
        const int s = own + i * WAVES;
        const Dims more = __shfl(w, s & 63) * v[i];
        acc += s < a.all_parts ? more : Dims{};
    }
    if constexpr (WAVES > 1) {
        share[wave][lane] = acc;
        __syncthreads();
        if (own != 0) return;
#pragma unroll
        for (int i = 1; i < WAVES; ++i) acc += share[wave + i][lane];
    }
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
    uint16_t* p = a.out.data + token * a.out.row + head * a.out.head + lane * kEach;
    if constexpr (kEach == 2)
        *reinterpret_cast<uint32_t*>(p) = pack_bf16x2(acc[0] * inv, acc[kEach - 1] * inv);
    else
        *p = (uint16_t)pack_bf16x2(acc[0] * inv, 0.0f);
}

}  // namespace

constexpr int64_t kSlots = 512;  // workgroups that are in flight at a time, two on each CU

static AttentionPlan plan_for(int64_t M, int64_t B, int32_t q_heads, int32_t kv_heads, int32_t dim, int64_t max_len,
                              int64_t slots) {
    const int32_t group = q_heads / kv_heads;
    AttentionPlan p;
    const int64_t blocks = clamp64(max_len, 0, (int64_t)1 << 31) / kKvBlock + (max_len % kKvBlock != 0);
    p.wide = attention_wide(M, B, group, kv_heads, blocks);
    const int64_t T = p.wide ? kWideRows : kRows;
    // The keys are cut into pieces until two workgroups for each of 256 CUs are
    // in flight, but not below 8 blocks to a piece of a narrow tile (2 a wave;
    // none below 32 blocks) and 4 of a wide one.  One token of 32 query and 8
    // key/value heads over 16,384 keys: 12.2 us with pieces of 8, 18 of 16, 20 of
    // 32; over 1024 keys 9.9 us in one piece, 10.4 in two.  40 tokens over 2048
    // keys: 16 us with pieces of 4, 20 of 8.
    int64_t tiles = (M * group + T - 1) / T;
    // At most M of the slots have rows, the others are not tiles: one token over
    // 16,384 keys among 255 empty slots 13 us, 117 when they counted.  (Several rows
    // of one slot still count as several: 40 over 65,536 keys take 72 us alone and
    // 274 among 255 empty slots, where the keys are not cut.)
    const int64_t most_seqs = B < M ? B : M;
    tiles = tiles < most_seqs ? most_seqs : tiles;
    int64_t want = slots / (tiles * kv_heads);
    // Many sequences are of many lengths, which the host does not know: pieces
    // half as long even the workgroups out (32 sequences of 1 to 16,384 keys: 123
    // -> 115 us; 32 of 8192: 113 -> 110; 4 of 16,384: 27 -> 30, so few are left).
    if (!p.wide && most_seqs >= 16 && want >= 2 && slots == kSlots) want *= 2;
    const int64_t most = p.wide ? blocks / 4 : blocks >= 32 ? blocks / 8 : 1;
    p.parts = (int32_t)clamp64(want < most ? want : most, 1, kMaxParts);
    p.workspace_bytes = p.parts == 1 ? 0 : (size_t)p.parts * (size_t)(M * q_heads) * (size_t)(dim + 2) * sizeof(float);
    return p;
}

AttentionPlan attention_plan(int64_t M, int64_t B, int32_t q_heads, int32_t kv_heads, int32_t dim, int64_t max_len) {
    return plan_for(M, B, q_heads, kv_heads, dim, max_len, kSlots);
}

// Where no sequence sees many more keys than the others (through a window, or
// behind a prefix), fewer pieces: until one workgroup for each CU.  The last 4096
// of 16,384 keys, 32 and 8 heads, calls from Python after one another: 32 tokens 69
// us in one piece, 84 in four with their join; 8 tokens 35 in four, 36 in eight, 48
// in one.  Behind a prefix they take the CUs' other places (64 tokens, up to 1024
// own keys, in a graph: 45 us in one piece, 57 in four).
static AttentionPlan few_parts_plan(int64_t M, int64_t B, int32_t q_heads, int32_t kv_heads, int32_t dim, int64_t max_len) {
    const bool wide = plan_for(M, B, q_heads, kv_heads, dim, max_len, kSlots).wide;
    return plan_for(M, B, q_heads, kv_heads, dim, max_len, wide ? kSlots : kSlots / 2);
}

// The first positions, the window and a tile's rows, each with what a cut inside a
// block adds: so much of the past can 128 rows see (all of it without a causal mask).
AttentionPlan window_plan(int64_t M, int64_t B, int32_t q_heads, int32_t kv_heads, int32_t dim, int64_t max_len,
                          int32_t causal, int32_t window, int32_t sinks) {
    const int64_t most = (int64_t)sinks + window + causal + kWideRows + 2 * kKvBlock;
    if (causal == 0 || max_len <= most) return attention_plan(M, B, q_heads, kv_heads, dim, max_len);
    return few_parts_plan(M, B, q_heads, kv_heads, dim, most);
}

// The tiles and pieces of a prefix of n blocks for `rows` rows of a key/value
// head: those of the smallest cost, in microseconds, of
//   a workgroup's steps (a block of a wide tile, four of a narrow one, and one
//   more to begin), longer where two workgroups share a CU, and
//   the pieces' sums, written and read once.
// Measured on prefixes of 16 to 512 blocks and 15 shapes of both dims: a step of a
// wide tile 1.2 us alone on a CU and 1.8 with a second one (heads of 64: 0.8 and
// 1.2), of a narrow one 2.1 and 3.3 (0.75 and 1.2).  64 tokens of 32 query and 8
// key/value heads over 16,384 positions: 45 us with 12 or 16 pieces of wide tiles,
// 58 with 32, 75 and more with narrow ones; 21 rows of 16 and 2 heads of 64 over 4032: 9.5
// with 16 pieces of narrow tiles, 12.5 with 15 of wide ones.  More workgroups than
// fit at once lose the keys that tiles share in L2 (500 rows of 32 heads over
// 32,768 positions: 349 in 3 pieces, 379 in 7).  Where the sequences' own keys fill
// the chip for a fourth of the prefix's time or more, it takes fewer places (100
// tokens with 1500 own keys each behind 12,800: 126 us a call in 4 pieces, 153 in
// 16).  Over 21 shapes calls take 5% longer on average than with the best of 15
// numbers of pieces and both tiles, and 16% at most.
static AttentionPlan prefix_plan(int64_t M, int32_t q_heads, int32_t kv_heads, int32_t dim, int64_t n, bool wide_only,
                                 int64_t own_groups, int64_t own_blocks) {
    AttentionPlan best = {wide_only, 0, 0};
    const int64_t rows = M * (q_heads / kv_heads);
    const double piece = (double)(M * q_heads) * (dim + 2) * 8 / 2.4e6;
    const double narrow[2] = {dim == 128 ? 2.1 : 0.75, dim == 128 ? 3.3 : 1.2}, wide[2] = {dim == 128 ? 1.2 : 0.8, dim == 128 ? 1.8 : 1.2};
    // half the bound: the sequences are of many lengths
    const double own = own_groups < kSlots / 2 ? 0.0 : (double)own_groups * (double)own_blocks * narrow[0] / 8;
    double least = 0.0;
    for (int w = wide_only; w <= (rows > kRows ? 1 : 0); ++w) {
        const int64_t T = w ? kWideRows : kRows, at_once = w ? 1 : kNarrowWaves;
        const double* step = w ? wide : narrow;
        const int64_t tiles = (rows + T - 1) / T * kv_heads, pieces = w ? (n + 1) / 2 : (n + 3) / 4;
        const int64_t places = own >= (double)tiles * (double)n * step[0] / (4 * at_once) ? 192 : kSlots;
        const int64_t fit = clamp64(places / tiles, 1, kMaxParts / 2 - 1);
        for (int64_t p = 1; p <= (pieces < fit ? pieces : fit); ++p) {
            const int64_t blocks = (n + p - 1) / p, steps = 1 + (blocks + at_once - 1) / at_once;
            const int64_t rounds = (tiles * p + kSlots - 1) / kSlots;
            const double cost = (double)(steps * rounds) * step[tiles * p > kSlots / 2] + (double)p * piece;
            if (best.parts == 0 || cost < least) {
                least = cost;
                best.wide = w != 0;
                best.parts = (int32_t)p;
            }
        }
    }
    return best;
}

SharedPlan shared_plan(int64_t M, int64_t B, int32_t q_heads, int32_t kv_heads, int32_t dim, int64_t max_len, int64_t shared) {
    SharedPlan p;
    const int64_t common = shared * kKvBlock;
    p.own = few_parts_plan(M, B, q_heads, kv_heads, dim, max_len > common ? max_len - common : 0);
    p.own.parts = p.own.parts < kOwnParts ? p.own.parts : kOwnParts;
    const int64_t group = q_heads / kv_heads, T = p.own.wide ? kWideRows : kRows;
    const int64_t own_groups = tile_first(M, B, group, T, tiles_per_row(M, B, group, T)) * kv_heads * p.own.parts;
    const int64_t own_blocks = max_len > common ? (clamp64(max_len, 0, (int64_t)1 << 31) - common) / kKvBlock + 1 : 0;
    p.prefix = prefix_plan(M, q_heads, kv_heads, dim, shared, p.own.wide, own_groups, own_blocks);
    p.workspace_bytes = (size_t)(p.prefix.parts + p.own.parts) * (size_t)(M * q_heads) * (size_t)(dim + 2) * sizeof(float);
    return p;
}

template <int D, int MODE>
static void attention_tiles(AttentionArgs a, hipStream_t s) {
    const int64_t T = a.wide ? kWideRows : kRows;
    a.seqs.per_row = tiles_per_row(a.seqs.M, a.seqs.B, a.group, T);
    const int64_t units = tile_first(a.seqs.M, a.seqs.B, a.group, T, a.seqs.per_row);
    if (a.wide) {
        // below 2^23, so that the threads of a dimension stay below 2^32: the heads
        // times M group / 128 + B, where B <= M group / 64 and M q_heads <= 2^28
        const dim3 grid((unsigned)(units * a.cache.heads), 1, (unsigned)a.parts);
        attention_wide_kernel<D, MODE><<<grid, dim3(64 * kWideWaves), 0, s>>>(a);
    } else {
        const dim3 grid((unsigned)units, (unsigned)a.cache.heads, (unsigned)a.parts);
        attention_narrow_kernel<D, MODE><<<grid, dim3(64 * kNarrowWaves), 0, s>>>(a);
    }
}

// n workgroups of 256, in two dimensions where their threads would pass 2^32 in one.
static dim3 join_grid(int64_t n) {
    const int64_t row = n < ((int64_t)1 << 20) ? n : (int64_t)1 << 20;
    return dim3((unsigned)row, (unsigned)((n + row - 1) / row));
}

template <int D>
static void attention_join(const AttentionArgs& a, hipStream_t s) {
    const int64_t rows = a.seqs.M * a.q_heads;
    const dim3 four = join_grid((rows + 3) / 4), one = join_grid(rows), threads(256);
    if (a.all_parts > 32)
        attention_join_kernel<D, 4, 16><<<one, threads, 0, s>>>(a);
    else if (a.all_parts > 16)
        attention_join_kernel<D, 4, 8><<<one, threads, 0, s>>>(a);
    else if (a.all_parts > 8)
        attention_join_kernel<D, 4, 4><<<one, threads, 0, s>>>(a);
    else if (a.all_parts > 4)
        attention_join_kernel<D, 1, 8><<<four, threads, 0, s>>>(a);
    else if (a.all_parts > 2)
        attention_join_kernel<D, 1, 4><<<four, threads, 0, s>>>(a);
    else if (a.all_parts > 1)
        attention_join_kernel<D, 1, 2><<<four, threads, 0, s>>>(a);
}

// The join of a batch: where the rows alone fill the chip, a wave takes a row and all
// its parts.  (There are at most 31 of the prefix and 16 own ones; the loads past a
// row's parts take part 0 again.)
template <int D>
static void attention_join_batch(const AttentionArgs& a, hipStream_t s) {
    const int64_t rows = a.seqs.M * a.q_heads;
    if (rows < 1024 || a.all_parts <= 8) return attention_join<D>(a, s);
    const dim3 four = join_grid((rows + 3) / 4), threads(256);
    if (a.all_parts > 32)
        attention_join_kernel<D, 1, 64><<<four, threads, 0, s>>>(a);
    else if (a.all_parts > 16)
        attention_join_kernel<D, 1, 32><<<four, threads, 0, s>>>(a);
    else
        attention_join_kernel<D, 1, 16><<<four, threads, 0, s>>>(a);
}

template <int D>
static void attention_of(const AttentionArgs& a, hipStream_t s) {
    if (a.window > 0)
        attention_tiles<D, WINDOW>(a, s);
    else
        attention_tiles<D, PLAIN>(a, s);
    attention_join<D>(a, s);
}

template <int D>
static void attention_shared_of(const AttentionArgs& a, const SharedPlan& p, const int32_t* shared, hipStream_t s) {
    const int64_t heads = a.cache.heads, rows = a.seqs.M * a.group;
    AttentionArgs own = a;
    own.parts = p.own.parts;
    own.first_part = p.prefix.parts;
    const int64_t T = p.own.wide ? kWideRows : kRows, PT = p.prefix.wide ? kWideRows : kRows;
    own.seqs.per_row = tiles_per_row(a.seqs.M, a.seqs.B, a.group, T);
    // both below 2^30: M q_heads is at most 2^28, tiles are at most 2 a row and
    // head, and the keys are cut only where there are few of them
    SharedGrid g;
    g.shared = shared;
    g.prefix_units = (uint32_t)((rows + PT - 1) / PT);
    g.own_units = (uint32_t)tile_first(a.seqs.M, a.seqs.B, a.group, T, own.seqs.per_row);
    g.prefix_groups = (uint32_t)(g.prefix_units * heads * p.prefix.parts);
    g.own_groups = (uint32_t)(g.own_units * heads * p.own.parts);
    const uint32_t groups = g.prefix_groups + g.own_groups, row = groups < (1u << 20) ? groups : 1u << 20;
    const dim3 grid(row, (groups + row - 1) / row), block(64 * kWideWaves);
    if (p.prefix.wide && p.own.wide)
        attention_shared_kernel<D, true, true><<<grid, block, 0, s>>>(own, g);
    else if (p.prefix.wide)
        attention_shared_kernel<D, true, false><<<grid, block, 0, s>>>(own, g);
    else
        attention_shared_kernel<D, false, false><<<grid, block, 0, s>>>(own, g);
    attention_join_batch<D>(a, s);
}

hipError_t launch_attention(const AttentionArgs& a, hipStream_t s) {
    if (a.cache.dim == 128)
        attention_of<128>(a, s);
    else
        attention_of<64>(a, s);
    return hipGetLastError();
}

hipError_t launch_attention_shared(const AttentionArgs& a, const SharedPlan& p, const int32_t* shared, hipStream_t s) {
    if (a.cache.dim == 128)
        attention_shared_of<128>(a, p, shared, s);
    else
        attention_shared_of<64>(a, p, shared, s);
    return hipGetLastError();
}

}  // namespace nvfp4
