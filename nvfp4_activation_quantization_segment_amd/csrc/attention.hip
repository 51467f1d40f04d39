// Attention over the paged 8-bit key/value cache:
//   o = sum_j p_j v_j / sum_j p_j,  p_j = exp(scale q.k_j - max),  j < limit(row).
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
// 0.0016 to 0.0017.  Scores, maxima, sums and outputs are held in
// binary32.
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

struct Tile {
    bool any;
    bool bad;         // a length that the table cannot hold
    int64_t b;
    int64_t row0;     // first row of the sequence
    int32_t n;        // its new tokens
    int32_t first;    // first tile row, counted in the sequence
    int32_t rows;     // n * group
    int64_t len;
};

__device__ __forceinline__ Tile find_tile(const AttentionArgs& a, int64_t unit, int64_t T) {
    Tile t;
    t.any = false;
    const SeqArgs& q = a.seqs;
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
    return t;
}

// What a lane knows of its row.
struct Row {
    bool valid;
    int64_t token;   // row of q and out
    int32_t head;    // query head
    int32_t limit;   // keys it sees
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

__device__ __forceinline__ Row find_row(const AttentionArgs& a, const Tile& t, int32_t rr, int32_t kv_head) {
    Row r;
    r.valid = rr < t.rows;
    const int32_t at = r.valid ? rr : t.rows - 1;
    const int32_t i = at / a.group;
    r.token = t.row0 + i;
    r.head = kv_head * a.group + (at - i * a.group);
    r.limit = limit_of(a, t, i);
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
        sum[k] = (part[0] + part[1]) + (part[2] + part[3]);
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
template <int NO>
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
        sum = probabilities(s, scale_log2, m == neg_inf() ? 0.0f : m, p);  // nothing seen yet: all 0
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
// vector registers are in use and 2 spill (12 bytes of scratch a lane), with
// 41 scalar ones that go to lanes of a vector register; D = 64 spills 46 scalar
// ones only.
// ---------------------------------------------------------------------------
constexpr int kNarrowWaves = 4;

template <int D>
__global__ __launch_bounds__(64 * kNarrowWaves, 2) void attention_narrow_kernel(AttentionArgs a) {
    constexpr int kDT = D / 32, kK = D / 64;
    constexpr int kBytes = kKvBlock * D;
    constexpr int kLd = D + 4;
    __shared__ __align__(16) float so[kNarrowWaves][kRows][kLd];
    __shared__ float sm[kNarrowWaves][kRows], sl[kNarrowWaves][kRows];
    const int kv_head = blockIdx.y, part = blockIdx.z;
    // Workgroups go to the 8 XCDs in turn: with a multiple of 8 units, all of a
    // long sequence's would go to one of them, were heads and parts not turned
    // against each other (32 sequences of 1 to 16,384 keys: 118 us, 124 without).
    uint32_t unit = blockIdx.x + (blockIdx.y + blockIdx.z) % gridDim.x;
    unit = unit < gridDim.x ? unit : unit - gridDim.x;
    const Tile t = find_tile(a, unit, kRows);
    if (!t.any) return;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    const int c = lane & 31, h = lane >> 5;
    const Row row = find_row(a, t, t.first + c, kv_head);
    // keys that the tile's last row sees, and keys that all its rows see: limits
    // do not fall from row to row
    const int seen = __builtin_amdgcn_readlane(row.limit, kRows - 1), all = __builtin_amdgcn_readlane(row.limit, 0);
    const BlockRange range = kv_part((seen + kKvBlock - 1) / kKvBlock, part, a.parts);
    const int at0 = range.first + wave;
    u32x4 qw[D / 16];
    fetch_query<D>(qw, a, row);

    // Table entries and powers are loaded like the keys, a block ahead, and are
    // looked at when they are needed: a wait for one of them would be a wait for
    // every load before it.
    const int32_t* table = a.seqs.table + t.b * a.seqs.ld_table;
    const auto entry = [&](int at) { return table[at < range.last ? at : range.last - 1]; };
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

        const int first_key = at * kKvBlock;
        const bool edge = first_key + kKvBlock > all;
        if (edge) {
            mask_scores(s[0], row.limit - first_key);
            mask_scores(s[1], row.limit - first_key - 32);
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
            if (__any(nan)) {
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
            const float sum = probabilities(s[tt], a.scale_log2, st.m, p);
            accept<kDT>(s[tt], a.scale_log2, sum, st, o, p);
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
    const Row mine = find_row(a, t, t.first + rr, kv_head);
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
    if (a.parts == 1) {
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
        float* po = a.partial + ((int64_t)part * all_rows + at) * D + d0;
        float* pm = a.partial + (int64_t)a.parts * all_rows * D + ((int64_t)part * all_rows + at) * 2;
#pragma unroll
        for (int i = 0; i < kEach; i += 4)
            *reinterpret_cast<float4*>(po + i) = make_float4(acc[i], acc[i + 1], acc[i + 2], acc[i + 3]);
        if ((threadIdx.x & 7) == 0) {
            pm[0] = m;
            pm[1] = t.bad ? quiet_nan() : l;
        }
    }
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
__device__ __forceinline__ void wide_place(const AttentionArgs& a, int& unit, int& kv_head) {
    const uint32_t heads = a.cache.heads, units = gridDim.x / heads;
    if (heads % 8 == 0) {
        const uint32_t at = blockIdx.x / 8, head = at / units;
        kv_head = (int)((blockIdx.x % 8) * (heads / 8) + head);
        unit = (int)(units - 1 - (at - head * units));
    } else {
        const uint32_t at = blockIdx.x / heads;
        kv_head = (int)(blockIdx.x - at * heads);
        unit = (int)(units - 1 - at);
    }
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

template <int D>
__global__ __launch_bounds__(64 * kWideWaves, 2) void attention_wide_kernel(AttentionArgs a) {
    constexpr int kDT = D / 32, kK = D / 64;
    constexpr int kBytes = kKvBlock * D;
    constexpr int kPieces = kBytes / 16;                  // 16-byte pieces of a block's keys, and of its values
    constexpr int kThreads = 64 * kWideWaves;
    constexpr int kEach = kPieces / kThreads;             // of them a thread's
    __shared__ __align__(16) u32x4 sk[2][kPieces];
    __shared__ __align__(16) u32x4 sv[2][2 * kPieces];    // [k-step][half][dim] of 8 keys
    __shared__ int nan_key[2][D];                         // first key whose value is a NaN code, by dim
    __shared__ int nan_any[2];
    int unit, kv_head;
    wide_place(a, unit, kv_head);
    const Tile t = find_tile(a, unit, kWideRows);
    if (!t.any) return;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    const int c = lane & 31, h = lane >> 5;
    const int row0 = t.first + wave * kRows;
    const Row row = find_row(a, t, row0 + c, kv_head);
    // keys that the tile's last row and this wave's last row see, and keys that
    // all rows of the tile and of the wave see
    const int tile_seen = limit_of_row(a, t, t.first + kWideRows - 1), tile_all = limit_of_row(a, t, t.first);
    const int seen = row0 < t.rows ? __builtin_amdgcn_readlane(row.limit, kRows - 1) : 0;
    const int all = __builtin_amdgcn_readlane(row.limit, 0);
    const int part = blockIdx.z;
    const BlockRange range = kv_part((tile_seen + kKvBlock - 1) / kKvBlock, part, a.parts);
    const int at0 = range.first, end = range.last;

    u32x4 qw[D / 16];
    fetch_query<D>(qw, a, row);
    for (int i = threadIdx.x; i < 2 * D; i += kThreads) nan_key[i / D][i % D] = kKvBlock;
    if (threadIdx.x < 2) nan_any[threadIdx.x] = 0;

    // table entries and powers are looked at a block after they are asked for,
    // as in the narrow kernel
    const int32_t* table = a.seqs.table + t.b * a.seqs.ld_table;
    const auto entry = [&](int at) { return table[at < end ? at : end - 1]; };
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
        edge_now = page < 0 || (at0 + 1) * kKvBlock > tile_all;
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
        const int b = (at - at0) & 1, first_key = at * kKvBlock;
        const bool more = at + 1 < end;
        const int64_t page = page_of(next);
        if (more) {
            fetch(page);
            next = entry(at + 2);
        }
        if (first_key < seen) {
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
            const bool edge = first_key + kKvBlock > all;
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
            if (edge) mask_scores(s[0], row.limit - first_key);
            scores(1);
            const float sum0 = probabilities(s[0], a.scale_log2, st.m, p0);
            values(1);
            alternate<2 * kK, 56>();
            asm volatile("" : "+v"(s[1]));  // issued here, not after the branch below
            accept<kDT>(s[0], a.scale_log2, sum0, st, o, p0);
            if (edge) mask_scores(s[1], row.limit - first_key - 32);
            multiply(0, p0[0]);
            values(2);
            multiply(1, p0[1]);
            const float sum1 = probabilities(s[1], a.scale_log2, st.m, p1);
            values(3);
            alternate<2 * kDT, 56>();
            accept<kDT>(s[1], a.scale_log2, sum1, st, o, p1);
            multiply(2, p1[0]);
            multiply(3, p1[1]);
        }
        if (edge_now && nan_any[b]) {  // the same for all waves
            if (first_key < seen) {
                int half = h;
                asm volatile("" : "+v"(half));
#pragma unroll
                for (int d = 0; d < kDT; ++d)
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const int key = nan_key[b][32 * d + 8 * (i / 4) + 4 * half + i % 4];
                        if (key < kKvBlock && key < row.limit - first_key) o[d][i] = quiet_nan();
                    }
            }
            __syncthreads();
            for (int i = threadIdx.x; i < D; i += kThreads) nan_key[b][i] = kKvBlock;
            if (threadIdx.x == 0) nan_any[b] = 0;
        }
        if (more) {
            const bool good = page >= 0;
            edge_now = !good || first_key + 2 * kKvBlock > tile_all;
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
    if (a.parts > 1) {
        const int64_t all_rows = a.seqs.M * a.q_heads, mine = (int64_t)part * all_rows + row.token * a.q_heads + row.head;
        float* po = a.partial + mine * D + 4 * h;
#pragma unroll
        for (int d = 0; d < kDT; ++d)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                *reinterpret_cast<float4*>(po + 32 * d + 8 * i) =
                    make_float4(o[d][4 * i], o[d][4 * i + 1], o[d][4 * i + 2], o[d][4 * i + 3]);
        if (h == 0)
            *reinterpret_cast<float2*>(a.partial + (int64_t)a.parts * all_rows * D + mine * 2) = make_float2(st.m, l);
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

// Joins the parts of each row; rows that no sequence has are left alone.  WAVES
// waves take a row: each has the maximum and sum of every part in its lanes
// (part s in lane s, at most 64), adds up its share of at most EACH parts, D / 64
// dims a lane, with all their loads in flight at once, and the first adds up
// the waves.  (64 parts of one wave's, eight loads at a time, took 12 us where
// the attention before it takes 25.)
constexpr int kMaxParts = 64;

template <int D, int WAVES, int EACH>
__global__ __launch_bounds__(256) void attention_join_kernel(AttentionArgs a) {
    constexpr int kEach = D / 64;
    typedef float Dims __attribute__((ext_vector_type(kEach)));
    __shared__ Dims share[4][64];
    const int64_t all_rows = a.seqs.M * a.q_heads;
    const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6)), lane = threadIdx.x & 63;
    const int64_t at = (int64_t)blockIdx.x * (4 / WAVES) + wave / WAVES;
    if (at >= all_rows) return;  // with one wave a row only: no barrier below
    const int64_t token = at / a.q_heads;
    const int32_t head = (int32_t)(at - token * a.q_heads);
    const int32_t first = a.seqs.row_start[0], last = a.seqs.row_start[a.seqs.B];
    const int mine = lane < a.parts ? lane : 0, own = wave % WAVES;
    const float2 ml = *reinterpret_cast<const float2*>(a.partial + a.parts * all_rows * D + (mine * all_rows + at) * 2);
    const float* po = a.partial + at * D + lane * kEach;
    Dims v[EACH];
#pragma unroll
    for (int i = 0; i < EACH; ++i) {
        const int s = own + i * WAVES;
        v[i] = *reinterpret_cast<const Dims*>(po + (s < a.parts ? s : 0) * all_rows * D);
    }
    if (token < first || token >= last) return;
    float m = lane < a.parts ? ml.x : neg_inf();
#pragma unroll
    for (int s = 32; s > 0; s >>= 1) m = fmaxf(m, __shfl_xor(m, s));
    const float w = lane < a.parts ? __builtin_amdgcn_exp2f(ml.x - (m == neg_inf() ? 0.0f : m)) : 0.0f;
    float l = lane >= a.parts ? 0.0f : ml.y != ml.y ? ml.y : w * ml.y;
#pragma unroll
    for (int s = 32; s > 0; s >>= 1) l += __shfl_xor(l, s);
    Dims acc = {};
#pragma unroll
    for (int i = 0; i < EACH; ++i) {
        const int s = own + i * WAVES;
        const Dims more = __shfl(w, s & 63) * v[i];
        acc += s < a.parts ? more : Dims{};
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

AttentionPlan attention_plan(int64_t M, int64_t B, int32_t q_heads, int32_t kv_heads, int32_t dim, int64_t max_len) {
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
    int64_t want = 512 / (tiles * kv_heads);
    // Many sequences are of many lengths, which the host does not know: pieces
    // half as long even the workgroups out (32 sequences of 1 to 16,384 keys: 123
    // -> 115 us; 32 of 8192: 113 -> 110; 4 of 16,384: 27 -> 30, so few are left).
    if (!p.wide && most_seqs >= 16 && want >= 2) want *= 2;
    const int64_t most = p.wide ? blocks / 4 : blocks >= 32 ? blocks / 8 : 1;
    p.parts = (int32_t)clamp64(want < most ? want : most, 1, kMaxParts);
    p.workspace_bytes = p.parts == 1 ? 0 : (size_t)p.parts * (size_t)(M * q_heads) * (size_t)(dim + 2) * sizeof(float);
    return p;
}

template <int D>
static void attention_of(const AttentionArgs& args, hipStream_t s) {
    AttentionArgs a = args;
    const int64_t T = a.wide ? kWideRows : kRows;
    a.seqs.per_row = tiles_per_row(a.seqs.M, a.seqs.B, a.group, T);
    const int64_t units = tile_first(a.seqs.M, a.seqs.B, a.group, T, a.seqs.per_row);
    if (a.wide) {
        // below 2^23, so that the threads of a dimension stay below 2^32: the heads
        // times M group / 128 + B, where B <= M group / 64 and M q_heads <= 2^28
        const dim3 grid((unsigned)(units * a.cache.heads), 1, (unsigned)a.parts);
        attention_wide_kernel<D><<<grid, dim3(64 * kWideWaves), 0, s>>>(a);
    } else {
        const dim3 grid((unsigned)units, (unsigned)a.cache.heads, (unsigned)a.parts);
        attention_narrow_kernel<D><<<grid, dim3(64 * kNarrowWaves), 0, s>>>(a);
    }
    const int64_t rows = a.seqs.M * a.q_heads;
    const dim3 four((unsigned)((rows + 3) / 4)), one((unsigned)rows), threads(256);
    if (a.parts > 32)
        attention_join_kernel<D, 4, 16><<<one, threads, 0, s>>>(a);
    else if (a.parts > 16)
        attention_join_kernel<D, 4, 8><<<one, threads, 0, s>>>(a);
    else if (a.parts > 8)
        attention_join_kernel<D, 4, 4><<<one, threads, 0, s>>>(a);
    else if (a.parts > 4)
        attention_join_kernel<D, 1, 8><<<four, threads, 0, s>>>(a);
    else if (a.parts > 2)
        attention_join_kernel<D, 1, 4><<<four, threads, 0, s>>>(a);
    else if (a.parts > 1)
        attention_join_kernel<D, 1, 2><<<four, threads, 0, s>>>(a);
}

hipError_t launch_attention(const AttentionArgs& a, hipStream_t s) {
    if (a.cache.dim == 128)
        attention_of<128>(a, s);
    else
        attention_of<64>(a, s);
    return hipGetLastError();
}

}  // namespace nvfp4
