// Rotary positions with several axes, and the paged 8-bit key/value cache:
// quantised as it is written, and read back.  All three stream their rows once
// and are bound by memory bandwidth.
#include "kv_device.h"
#include "rope_device.h"

namespace nvfp4 {
namespace {

// ---------------------------------------------------------------------------
// Rotation of a pair by (cos, sin): y1 = x1 c - x2 s, y2 = x2 c + x1 s, each
// product and sum a binary32 operation, the result rounded once to bf16.
// ---------------------------------------------------------------------------
__global__ void rope_table_kernel(float2* table, int64_t n, int32_t pairs, double theta) {
    const int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    if (i >= n) return;
    // in binary64: the angle is off by a few 2^-53 of itself, at position 2^24
    // about 2^-27, a fourth of half a step of a result near 1
    const double angle = (double)(i / pairs) * pow(theta, -(double)(i % pairs) / (double)pairs);
    table[i] = make_float2((float)cos(angle), (float)sin(angle));
}

// A workgroup takes a few rows: it looks each row's angles up once, into LDS,
// and then goes over the rows' units of 16 dims (8 rotated pairs, or 16 dims
// that pass through) in the order they lie in, the next unit's loads ahead of
// this one's stores.  Looked up by each thread for its own heads instead, the
// picking of axes and table addresses took more vector time than the rotation
// (340 us for 37,810 rows of 56 heads of 128).  Now 214 us, 5.07 TB/s read and
// written: what a copy reaches (4.93 TB/s over 2 GiB).
struct RopeGeo {
    int64_t M;
    int32_t heads, units;    // 16-dim units per head
    int32_t rows;            // rows of a workgroup
    int32_t du, dh, dr;      // 256 units further on: so many units, heads and rows
};
constexpr int kRopeTurns = 1024;  // angles a workgroup holds

// Rotates the 16 values of a unit: two times 8 dims.
template <bool SPLIT>
__device__ __forceinline__ void rope_unit(uint4& a, uint4& b, const float2 (&t)[8]) {
    uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    if constexpr (SPLIT) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float2 c0 = t[2 * j], c1 = t[2 * j + 1];
            const float p0 = bf16_lo(w[j]), p1 = bf16_hi(w[j]), q0 = bf16_lo(w[4 + j]), q1 = bf16_hi(w[4 + j]);
            w[j] = pack_bf16x2(p0 * c0.x - q0 * c0.y, p1 * c1.x - q1 * c1.y);
            w[4 + j] = pack_bf16x2(q0 * c0.x + p0 * c0.y, q1 * c1.x + p1 * c1.y);
        }
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float p = bf16_lo(w[j]), q = bf16_hi(w[j]);
            w[j] = pack_bf16x2(p * t[j].x - q * t[j].y, q * t[j].x + p * t[j].y);
        }
    }
    a = make_uint4(w[0], w[1], w[2], w[3]);
    b = make_uint4(w[4], w[5], w[6], w[7]);
}

template <bool SPLIT>
__global__ __launch_bounds__(256) void rope_kernel(HeadsIn x, HeadsOut out, RopeArgs r, RopeGeo g) {
    __shared__ __align__(16) float2 turn[kRopeTurns];
    const int64_t row0 = (int64_t)blockIdx.x * g.rows;
    const int rows = (int)(g.M - row0 < g.rows ? g.M - row0 : g.rows);
    const int turning = r.total / 8;
    int u = threadIdx.x % g.units, h = threadIdx.x / g.units % g.heads, in = threadIdx.x / g.units / g.heads;
    // the unit's two times 8 dims, in elements from the head's first
    const auto low = [&](int unit) { return SPLIT && unit < turning ? 8 * unit : 16 * unit; };
    const auto high = [&](int unit) { return SPLIT && unit < turning ? r.total + 8 * unit : 16 * unit + 8; };
    const auto load = [&](uint4& a, uint4& b) {
        const uint16_t* p = x.data + (row0 + in) * x.row + h * x.head;
        a = *reinterpret_cast<const uint4*>(p + low(u));
        b = *reinterpret_cast<const uint4*>(p + high(u));
    };
    uint4 a = make_uint4(0, 0, 0, 0), b = a;
    if (in < rows) load(a, b);  // on its way while the angles are looked up
    const Axes axes = axes_of(r);
    for (int i = threadIdx.x; i < rows * r.total; i += 256) {
        const int j = i / r.total;
        turn[i] = rope_turn(axes, positions_of(r, row0 + j), i - j * r.total);
    }
    __syncthreads();
    while (in < rows) {
        const int u0 = u;
        const float2* t = turn + in * r.total + 8 * u;
        uint16_t* p = out.data + (row0 + in) * out.row + h * out.head;
        uint4 a0 = a, b0 = b;
        u += g.du;
        h += g.dh;
        in += g.dr;
        if (u >= g.units) u -= g.units, ++h;
        if (h >= g.heads) h -= g.heads, ++in;
        if (in < rows) load(a, b);
        if (u0 < turning) {
            float2 c[8];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float4 w = reinterpret_cast<const float4*>(t)[i];
                c[2 * i] = make_float2(w.x, w.y);
                c[2 * i + 1] = make_float2(w.z, w.w);
            }
            rope_unit<SPLIT>(a0, b0, c);
        }
        *reinterpret_cast<uint4*>(p + low(u0)) = a0;
        *reinterpret_cast<uint4*>(p + high(u0)) = b0;
    }
}

// ---------------------------------------------------------------------------
// The cache's writer and reader.  A workgroup takes one block of 64 positions
// of one sequence and several heads.  A thread owns 4 neighbouring positions
// (one dword of a value piece) of 8 dims; a wave owns one or two whole value
// pieces, so that values change places within the wave only.
//   D = 128: 256 threads, wave = (u, h), lane = (e, m) x 16 dim groups
//   D =  64: 128 threads, wave = u, lane = (h, e, m) x 8 dim groups
// A block's power needs all its values, so they stay in registers between the
// maximum and the codes and memory is read once.  37,810 rows of 56 heads of
// 128, keys rotated on three axes: written in 344 us, 4.72 TB/s read and
// written; read back in 350 us, 4.65 TB/s (a copy reaches 4.93).
// ---------------------------------------------------------------------------
template <int D>
struct Owner {
    static constexpr int kGroups = D / 8;     // dim groups
    static constexpr int kThreads = 2 * D;
    static constexpr int kWaves = kThreads / 64;
    int g, t0;      // dims 8g.., positions t0..t0+3
    int piece, em;  // value piece 2u + h and dword 2e + m
    __device__ __forceinline__ Owner() {
        const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
        g = lane % kGroups;
        const int sub = lane / kGroups;
        const int u = D == 128 ? wave >> 1 : wave;
        const int h = D == 128 ? wave & 1 : sub >> 2;
        em = sub & 3;
        piece = 2 * u + h;
        t0 = 32 * u + 16 * (em >> 1) + 8 * (em & 1) + 4 * h;
    }
};

// Where a work unit stands.
struct BlockUnit {
    bool any;       // whether there is anything to do
    bool good;      // whether its cache block exists
    bool bad_len;   // a length that the table cannot hold
    int64_t row0;   // row of the sequence's first new position
    int64_t first;  // first new position
    int64_t len;
    int64_t start;  // position of the block's first slot (negative: before the sequence)
    int64_t page;
};

__device__ __forceinline__ BlockUnit block_unit(const SeqArgs& q, int64_t blocks, int64_t unit) {
    BlockUnit u;
    u.any = false;
    const Located s = locate(q, unit, [&](int64_t row, int64_t b) { return block_first(row, b, q.per_row); });
    const RowRange r = row_range(s.start, s.end, q.M);
    const int64_t n = r.last - r.first, local = unit - block_first(r.first, s.b, q.per_row);
    if (n <= 0 || local < 0) return u;
    u.len = s.len;
    u.first = u.len - n;
    u.row0 = r.first;
    const int64_t at = floor_div(u.first, kKvBlock) + local;
    if (at * kKvBlock >= u.len) return u;
    u.any = true;
    u.start = at * kKvBlock;
    u.bad_len = kv_length_bad(u.len, q.table_blocks);
    u.good = at >= 0 && at < q.table_blocks && !u.bad_len;
    u.page = u.good ? q.table[s.b * q.ld_table + at] : 0;
    if (u.page < 0 || u.page >= blocks) {
        u.good = false;
        u.page = 0;
    }
    return u;
}

__device__ __forceinline__ uint32_t drop_nonfinite(uint32_t m2) {
    return ((m2 & 0x7F80u) == 0x7F80u ? 0u : m2 & 0xFFFFu) | ((m2 & 0x7F800000u) == 0x7F800000u ? 0u : m2 & 0xFFFF0000u);
}

// The largest of both halves over the workgroup, each half for itself.
template <int WAVES>
__device__ __forceinline__ uint32_t group_max(uint32_t m, uint32_t* slot) {
#pragma unroll
    for (int s = 32; s > 0; s >>= 1) m = pk_max_u16(m, (uint32_t)__shfl_xor((int)m, s));
    if ((threadIdx.x & 63) == 0) slot[threadIdx.x >> 6] = m;
    __syncthreads();
    m = slot[0];
#pragma unroll
    for (int w = 1; w < WAVES; ++w) m = pk_max_u16(m, slot[w]);
    return m;
}

// The largest power's byte: that of finite bf16 values above 1.75 * 2^127.
constexpr uint32_t kLargestPower = 247;

// Code of one value: the nearest E4M3 of x / p, or the NaN code for what is not
// finite.  With the largest power, 2^120, codes stop at 240: 256 * 2^120 = 2^128,
// the nearest to values above 1.9375 * 2^127, would not be finite any more.
__device__ __forceinline__ uint32_t encode_any(float x, uint32_t power) {
    const float most = power >= kLargestPower ? 240.0f : 448.0f;
    const float y = fminf(fmaxf(x * power_inverse(power), -most), most);
    const uint32_t bits = __float_as_uint(x) & 0x7F800000u;
    return bits == 0x7F800000u ? 0x7Fu : (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(y, 0.0f, 0, false) & 0xFFu;
}

// Four stored codes moved to a larger power of two.
__device__ __forceinline__ uint32_t shrink4(uint32_t w, float factor) {
    uint32_t r = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t c = (w >> (8 * i)) & 0xFFu;
        const uint32_t n = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(e4m3_value(c) * factor, 0.0f, 0, false) & 0xFFu;
        r |= ((c & 0x7Fu) == 0x7Fu ? c : n) << (8 * i);
    }
    return r;
}

enum { ROPE_NONE = 0, ROPE_PAIRS = 1, ROPE_SPLIT = 2 };

__device__ __forceinline__ float half_of(const uint32_t* w, int i) { return i & 1 ? bf16_hi(w[i >> 1]) : bf16_lo(w[i >> 1]); }

template <int D, int MODE>
__global__ __launch_bounds__(2 * D) void kv_write_kernel(CacheArgs c, SeqArgs q, HeadsIn kx, HeadsIn vx, RopeArgs r,
                                                         int32_t heads_each) {
    using Own = Owner<D>;
    constexpr int kBytes = kKvBlock * D;
    constexpr int kPieceBytes = 16 * D;
    __shared__ uint32_t red[2][Own::kWaves];
    __shared__ uint32_t red2[2][Own::kWaves];
    __shared__ __align__(16) uint32_t stage[kBytes / 4];
    const BlockUnit u = block_unit(q, c.blocks, blockIdx.x);
    if (!u.any) return;
    const Own o;
    // positions of the block that are new: [lo, hi); those before lo are kept
    const int lo = (int)(u.first > u.start ? u.first - u.start : 0);
    const int hi = (int)(u.len - u.start < kKvBlock ? u.len - u.start : kKvBlock);
    const bool full = lo == 0 && hi == kKvBlock;
    if (hi <= 0) return;  // before the sequence
    // this thread's positions' rows; where one is not new, the sequence's first
    // row is loaded in its place and not used
    bool fresh[4];
    int64_t at_row[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        fresh[j] = o.t0 + j >= lo && o.t0 + j < hi;
        at_row[j] = fresh[j] ? u.row0 + (u.start - u.first) + o.t0 + j : u.row0;
    }

    const bool any = fresh[0] || fresh[1] || fresh[2] || fresh[3];

    // this thread's angles, kept over the heads
    constexpr int kTurns = MODE == ROPE_SPLIT ? 8 : 4;
    float cs[4][MODE == ROPE_NONE ? 1 : kTurns], sn[4][MODE == ROPE_NONE ? 1 : kTurns];
    bool turns = false;
    int partner = 0;
    if constexpr (MODE != ROPE_NONE) {
        const int lane = threadIdx.x & 63;
        const Axes axes = axes_of(r);
        int pair0 = 4 * o.g;
        turns = 8 * o.g < 2 * r.total;
        partner = lane;
        if constexpr (MODE == ROPE_SPLIT) {
            const bool upper = 8 * o.g >= r.total;
            pair0 = 8 * o.g - (upper ? r.total : 0);
            if (turns) partner = lane + (upper ? -(r.total / 8) : r.total / 8);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if (!any) break;  // a short write's other threads look nothing up
            const Positions pos = positions_of(r, at_row[j]);
#pragma unroll
            for (int i = 0; i < kTurns; ++i) {
                const float2 t = rope_turn(axes, pos, turns ? pair0 + i : 0);
                cs[j][i] = t.x;
                // y1 = x1 c + x2 (-s): the sign goes with the sine
                sn[j][i] = MODE == ROPE_SPLIT && 8 * o.g < r.total ? -t.y : t.y;
            }
        }
    }

    const int h0 = blockIdx.y * heads_each;
    const int h1 = h0 + heads_each < c.heads ? h0 + heads_each : c.heads;
    for (int h = h0; h < h1; ++h) {
        const int parity = (h - h0) & 1;
        const int64_t at = u.page * c.heads + h;
        uint8_t* const kb = c.k + at * kBytes;
        uint8_t* const vb = c.v + at * kBytes;
        uint32_t kw[4][4], vw[4][4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            uint4 a = make_uint4(0, 0, 0, 0), b = a;
            if (any) {
                a = *reinterpret_cast<const uint4*>(kx.data + at_row[j] * kx.row + h * kx.head + 8 * o.g);
                b = *reinterpret_cast<const uint4*>(vx.data + at_row[j] * vx.row + h * vx.head + 8 * o.g);
            }
            kw[j][0] = a.x, kw[j][1] = a.y, kw[j][2] = a.z, kw[j][3] = a.w;
            vw[j][0] = b.x, vw[j][1] = b.y, vw[j][2] = b.z, vw[j][3] = b.w;
        }
        // the rows are on their way while the block is looked up
        if (!u.good) return;
        // a part of a block: its values' dwords, of which this thread has some
        uint32_t* const vp = reinterpret_cast<uint32_t*>(vb + o.piece * kPieceBytes + 8 * o.g * 16 + 4 * o.em);
        uint32_t was[8] = {};
        if (!full && o.t0 < hi) {
#pragma unroll
            for (int d = 0; d < 8; ++d) was[d] = vp[4 * d];
        }
        uint32_t had_k = 0, had_v = 0;
        if (lo > 0) {
            had_k = clamp_power(c.k_power[at]);
            had_v = clamp_power(c.v_power[at]);
        }
        if constexpr (MODE == ROPE_PAIRS) {
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float x1 = bf16_lo(kw[j][i]), x2 = bf16_hi(kw[j][i]);
                    const uint32_t y = pack_bf16x2(x1 * cs[j][i] - x2 * sn[j][i], x2 * cs[j][i] + x1 * sn[j][i]);
                    kw[j][i] = turns ? y : kw[j][i];
                }
        } else if constexpr (MODE == ROPE_SPLIT) {
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint32_t p = (uint32_t)__shfl((int)kw[j][i], partner);
                    const float y0 = bf16_lo(kw[j][i]) * cs[j][2 * i] + bf16_lo(p) * sn[j][2 * i];
                    const float y1 = bf16_hi(kw[j][i]) * cs[j][2 * i + 1] + bf16_hi(p) * sn[j][2 * i + 1];
                    kw[j][i] = turns ? pack_bf16x2(y0, y1) : kw[j][i];
                }
        }
        if (!full) {
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    kw[j][i] = fresh[j] ? kw[j][i] : 0u;
                    vw[j][i] = fresh[j] ? vw[j][i] : 0u;
                }
        }
        uint32_t mk = 0, mv = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                mk = pk_max_u16(mk, mag2(kw[j][i]));
                mv = pk_max_u16(mv, mag2(vw[j][i]));
            }
        uint32_t top = group_max<Own::kWaves>((fold_max(mk) << 16) | fold_max(mv), red[parity]);
        // a value is not finite, or so large that its block takes the largest power
        const bool odd = (top & 0xFFFFu) > 0x7F60u || (top >> 16) > 0x7F60u;
        if (odd) {
            mk = mv = 0;
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    mk = pk_max_u16(mk, drop_nonfinite(mag2(kw[j][i])));
                    mv = pk_max_u16(mv, drop_nonfinite(mag2(vw[j][i])));
                }
            top = group_max<Own::kWaves>((fold_max(mk) << 16) | fold_max(mv), red2[parity]);
        }
        uint32_t pk = power_for(top >> 16), pv = power_for(top & 0xFFFFu);
        const bool clear = pv >= kLargestPower;
        pk = pk > had_k ? pk : had_k;
        pv = pv > had_v ? pv : had_v;
        const float ik = power_inverse(pk), iv = power_inverse(pv);

        // codes: keys as 8 bytes of each position, values as one dword of 4
        // positions for each dim
        uint32_t kc[4][2], vc[8];
        if (!odd) {
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    kc[j][i] = fp8_pack4(bf16_lo(kw[j][2 * i]) * ik, bf16_hi(kw[j][2 * i]) * ik,
                                         bf16_lo(kw[j][2 * i + 1]) * ik, bf16_hi(kw[j][2 * i + 1]) * ik);
#pragma unroll
            for (int d = 0; d < 8; ++d)
                vc[d] = fp8_pack4(half_of(vw[0], d) * iv, half_of(vw[1], d) * iv, half_of(vw[2], d) * iv,
                                  half_of(vw[3], d) * iv);
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    kc[j][i] = 0;
#pragma unroll
                    for (int x = 0; x < 4; ++x) kc[j][i] |= encode_any(half_of(kw[j], 4 * i + x), pk) << (8 * x);
                }
#pragma unroll
            for (int d = 0; d < 8; ++d) {
                vc[d] = 0;
#pragma unroll
                for (int j = 0; j < 4; ++j) vc[d] |= encode_any(half_of(vw[j], d), pv) << (8 * j);
            }
        }

        if (full) {
            // keys: neighbouring dim groups swap halves, so that each stores
            // whole 16-byte pieces of two positions
            const bool upper = o.g & 1;
            uint32_t got[2][2];
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    got[j][i] = (uint32_t)__shfl_xor((int)(upper ? kc[j][i] : kc[2 + j][i]), 1);
            uint4* kp = reinterpret_cast<uint4*>(kb + (o.g >> 1) * (kKvBlock * 16) + (o.t0 + (upper ? 2 : 0)) * 16);
#pragma unroll
            for (int j = 0; j < 2; ++j)
                kp[j] = upper ? make_uint4(got[j][0], got[j][1], kc[2 + j][0], kc[2 + j][1])
                              : make_uint4(kc[j][0], kc[j][1], got[j][0], got[j][1]);
            // values: through LDS, 16-byte slot s = (piece, dim) at
            // s ^ ((s >> 3) & 7), so that the 64 lanes' dwords fall on all banks
            const int s0 = o.piece * D + 8 * o.g;
#pragma unroll
            for (int d = 0; d < 8; ++d) stage[4 * ((s0 + d) ^ (((s0 + d) >> 3) & 7)) + o.em] = vc[d];
            wave_lds_sync();
            const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int s = wave * 128 + i * 64 + lane;
                reinterpret_cast<uint4*>(vb)[s] = reinterpret_cast<const uint4*>(stage)[s ^ ((s >> 3) & 7)];
            }
            wave_lds_sync();
        } else {
            // part of a block: every dword has one owner, which keeps the bytes
            // that are not new (re-encoded where the power of two grew)
            const float fk = had_k && pk > had_k ? power_value(127u - (pk - had_k < 126u ? pk - had_k : 126u)) : 1.0f;
            const float fv = had_v && pv > had_v ? power_value(127u - (pv - had_v < 126u ? pv - had_v : 126u)) : 1.0f;
            const bool grew_k = had_k && pk > had_k, grew_v = had_v && pv > had_v;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                uint2* p = reinterpret_cast<uint2*>(kb + kv_key_offset(o.t0 + j, 8 * o.g));
                if (fresh[j]) {
                    *p = make_uint2(kc[j][0], kc[j][1]);
                } else if (grew_k && o.t0 + j < lo) {
                    const uint2 w = *p;
                    *p = make_uint2(shrink4(w.x, fk), shrink4(w.y, fk));
                }
            }
            // bytes that stay, and those of them that are positions before lo.
            // Behind the last position an earlier use may have left codes that are
            // not finite with the largest power: they would make 0 p of the rows
            // that do not see them NaN, so with that power they become 0.
            uint32_t keep = 0, old = 0;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if (!fresh[j]) keep |= 0xFFu << (8 * j);
                if (o.t0 + j < lo) old |= 0xFFu << (8 * j);
            }
            const uint32_t stay = clear ? old : keep;
            if (stay != 0xFFFFFFFFu || (grew_v && old)) {
#pragma unroll
                for (int d = 0; d < 8; ++d) {
                    uint32_t w = was[d];
                    if (grew_v) w = (shrink4(w, fv) & old) | (w & ~old);
                    vp[4 * d] = (w & stay) | (vc[d] & ~keep);
                }
            }
        }
        if (threadIdx.x == 0) {
            c.k_power[at] = (uint8_t)pk;
            c.v_power[at] = (uint8_t)pv;
        }
    }
}

// The writer for a few rows a sequence: a lane has 2 dims, a wave takes one new
// position after another (twice: for the maximum and for the codes), and WAVES
// waves share out a block's where there are several.  The same bytes as the
// writer above, from less code and a third of its registers: a call this short
// is a chain of waits, for memory and for instructions.  32 single tokens of 8
// heads, rotated, 4.2 us (8.8 with the writer above), 256 of 56 heads 18 (110).
// Further rows of a sequence cost more than their bytes: single bytes of values
// are stored, and all but a wave's last row are loaded and rotated twice (4 rows
// of 256 sequences and 56 heads 55 to 65 us, 9 at a copy's bandwidth).
template <int D, int MODE, int WAVES>
__global__ __launch_bounds__(64 * WAVES) void kv_append_kernel(CacheArgs c, SeqArgs q, HeadsIn kx, HeadsIn vx, RopeArgs r) {
    constexpr int kBytes = kKvBlock * D;
    __shared__ uint32_t red[2][WAVES];
    const BlockUnit u = block_unit(q, c.blocks, blockIdx.x);
    if (!u.any) return;
    const int lo = (int)(u.first > u.start ? u.first - u.start : 0);
    const int hi = (int)(u.len - u.start < kKvBlock ? u.len - u.start : kKvBlock);
    const int h = blockIdx.y, lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    const bool several = WAVES > 1 && hi - lo > 1;
    if (!several && wave > 0) return;
    const int step = several ? WAVES : 1;  // the others of a single one's waves are done
    const bool mine = 2 * lane < D;
    const int d = mine ? 2 * lane : 0;  // idle lanes load dims 0 and 1 (their keys count as zero) and store nothing
    const int64_t row = u.row0 + (u.start - u.first);
    const Axes axes = axes_of(r);
    // this lane's pair is (d, d + 1), or its two are (d, d + 1) with the dims
    // r.total away, in the other half of the rotated part
    const bool turns = MODE != ROPE_NONE && d < 2 * r.total, upper = MODE == ROPE_SPLIT && d >= r.total;
    const int pair = !turns ? 0 : MODE == ROPE_SPLIT ? d - (upper ? r.total : 0) : d / 2;
    const int partner = MODE == ROPE_SPLIT && turns && mine ? lane + (upper ? -(r.total / 2) : r.total / 2) : lane;
    const auto key_of = [&](int t) -> uint32_t {
        uint32_t w = *reinterpret_cast<const uint32_t*>(kx.data + (row + t) * kx.row + h * kx.head + d);
        if constexpr (MODE == ROPE_PAIRS) {
            const float2 a = rope_turn(axes, positions_of(r, row + t), pair);
            const float x1 = bf16_lo(w), x2 = bf16_hi(w);
            const uint32_t y = pack_bf16x2(x1 * a.x - x2 * a.y, x2 * a.x + x1 * a.y);
            w = turns ? y : w;
        } else if constexpr (MODE == ROPE_SPLIT) {
            const Positions pos = positions_of(r, row + t);
            float2 a = rope_turn(axes, pos, pair), b = rope_turn(axes, pos, turns ? pair + 1 : 0);
            const uint32_t p = (uint32_t)__shfl((int)w, partner);
            a.y = upper ? a.y : -a.y;
            b.y = upper ? b.y : -b.y;
            const uint32_t y = pack_bf16x2(bf16_lo(w) * a.x + bf16_lo(p) * a.y, bf16_hi(w) * b.x + bf16_hi(p) * b.y);
            w = turns ? y : w;
        }
        return mine ? w : 0u;  // (an idle lane's partner is itself: its pair means nothing)
    };
    const auto value_of = [&](int t) -> uint32_t {
        return *reinterpret_cast<const uint32_t*>(vx.data + (row + t) * vx.row + h * vx.head + d);
    };
    uint32_t mk = 0, mv = 0, fk = 0, fv = 0;  // m: magnitudes, f: the finite ones
    const auto look_at = [&](uint32_t kw, uint32_t vw) {
        mk = pk_max_u16(mk, mag2(kw));
        mv = pk_max_u16(mv, mag2(vw));
        fk = pk_max_u16(fk, drop_nonfinite(mag2(kw)));
        fv = pk_max_u16(fv, drop_nonfinite(mag2(vw)));
    };
    // a wave's last position stays in registers: most calls have one.  The others
    // are taken kBatch at a time, their loads in flight together (one sequence of
    // 60 rows and 63 of none, one wave a head: 27 us, 33 one by one; 8 at a time
    // the same)
    constexpr int kBatch = 4;
    uint32_t kw = 0, vw = 0;
    int last = -1, t = lo + wave;
    for (; t + kBatch * step < hi; t += kBatch * step) {
        uint32_t k[kBatch], v[kBatch];
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            v[i] = value_of(t + i * step);
            k[i] = key_of(t + i * step);
        }
#pragma unroll
        for (int i = 0; i < kBatch; ++i) look_at(k[i], v[i]);
    }
    for (; t < hi; t += step) {
        last = t;
        vw = value_of(t);
        kw = key_of(t);
        look_at(kw, vw);
    }
    if (!u.good) return;
    const int64_t at = u.page * c.heads + h;
    uint8_t* const kb = c.k + at * kBytes;
    uint8_t* const vb = c.v + at * kBytes;
    const uint32_t had_k = lo > 0 ? clamp_power(c.k_power[at]) : 0u, had_v = lo > 0 ? clamp_power(c.v_power[at]) : 0u;
    uint32_t any = (fold_max(mk) << 16) | fold_max(mv), top = (fold_max(fk) << 16) | fold_max(fv);
#pragma unroll
    for (int s = 32; s > 0; s >>= 1) {
        any = pk_max_u16(any, (uint32_t)__shfl_xor((int)any, s));
        top = pk_max_u16(top, (uint32_t)__shfl_xor((int)top, s));
    }
    if (several) {
        if (lane == 0) {
            red[0][wave] = any;
            red[1][wave] = top;
        }
        __syncthreads();  // also: all have read the block's powers
#pragma unroll
        for (int w = 0; w < WAVES; ++w) {
            any = pk_max_u16(any, red[0][w]);
            top = pk_max_u16(top, red[1][w]);
        }
    }
    const bool odd = (any & 0xFFFFu) > 0x7F60u || (any >> 16) > 0x7F60u;
    uint32_t pk = power_for(top >> 16), pv = power_for(top & 0xFFFFu);
    const bool clear = pv >= kLargestPower;
    pk = pk > had_k ? pk : had_k;
    pv = pv > had_v ? pv : had_v;
    if (mine && had_k && pk > had_k) {
        const float f = power_value(127u - (pk - had_k < 126u ? pk - had_k : 126u));
        for (int t = wave; t < lo; t += step) {
            uint16_t* p = reinterpret_cast<uint16_t*>(kb + kv_key_offset(t, d));
            *p = (uint16_t)shrink4(*p, f);
        }
    }
    if (mine && had_v && pv > had_v) {
        const float f = power_value(127u - (pv - had_v < 126u ? pv - had_v : 126u));
        for (int t = wave; t < lo; t += step)
            for (int i = 0; i < 2; ++i) {
                uint8_t* p = vb + kv_value_offset(t, d + i, D);
                *p = (uint8_t)shrink4(*p, f);
            }
    }
    // with the largest power, codes behind the last position become 0 (see the other writer)
    if (mine && clear)
        for (int t = hi + wave; t < kKvBlock; t += step)
            for (int i = 0; i < 2; ++i) vb[kv_value_offset(t, d + i, D)] = 0;
    const auto store = [&](int t, uint32_t kw, uint32_t vw) {
        uint32_t kc, vc;
        if (!odd) {
            const float ik = power_inverse(pk), iv = power_inverse(pv);
            kc = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(bf16_lo(kw) * ik, bf16_hi(kw) * ik, 0, false);
            vc = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(bf16_lo(vw) * iv, bf16_hi(vw) * iv, 0, false);
        } else {
            kc = encode_any(bf16_lo(kw), pk) | encode_any(bf16_hi(kw), pk) << 8;
            vc = encode_any(bf16_lo(vw), pv) | encode_any(bf16_hi(vw), pv) << 8;
        }
        if (mine) {
            *reinterpret_cast<uint16_t*>(kb + kv_key_offset(t, d)) = (uint16_t)kc;
            vb[kv_value_offset(t, d, D)] = (uint8_t)vc;
            vb[kv_value_offset(t, d + 1, D)] = (uint8_t)(vc >> 8);
        }
    };
    if (last >= 0) store(last, kw, vw);
    for (t = lo + wave; t + kBatch * step <= last; t += kBatch * step) {
        uint32_t k[kBatch], v[kBatch];
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            v[i] = value_of(t + i * step);
            k[i] = key_of(t + i * step);
        }
#pragma unroll
        for (int i = 0; i < kBatch; ++i) store(t + i * step, k[i], v[i]);
    }
    for (; t < last; t += step) store(t, key_of(t), value_of(t));
    if (threadIdx.x == 0) {
        c.k_power[at] = (uint8_t)pk;
        c.v_power[at] = (uint8_t)pv;
    }
}

// The inverse of the writer: the same ownership, the same rows.
template <int D>
__global__ __launch_bounds__(2 * D) void kv_read_kernel(CacheArgs c, SeqArgs q, HeadsOut kx, HeadsOut vx,
                                                        int32_t heads_each) {
    using Own = Owner<D>;
    constexpr int kBytes = kKvBlock * D;
    __shared__ __align__(16) uint32_t stage[kBytes / 4];
    const BlockUnit u = block_unit(q, c.blocks, blockIdx.x);
    if (!u.any) return;
    const Own o;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int lo = (int)(u.first > u.start ? u.first - u.start : 0);
    const int hi = (int)(u.len - u.start < kKvBlock ? u.len - u.start : kKvBlock);
    const int64_t row = u.row0 + (u.start - u.first);  // of the block's first position
    const bool wrong = !u.good && (u.bad_len || u.start >= 0);
    const uint32_t fill = wrong ? 0x7FC07FC0u : 0u;  // no such block or length: NaN; before the sequence: 0
    const int h0 = blockIdx.y * heads_each;
    const int h1 = h0 + heads_each < c.heads ? h0 + heads_each : c.heads;
    for (int h = h0; h < h1; ++h) {
        if (!u.good) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int t = o.t0 + j;
                if (t < lo || t >= hi) continue;
                const uint4 f = make_uint4(fill, fill, fill, fill);
                *reinterpret_cast<uint4*>(kx.data + (row + t) * kx.row + h * kx.head + 8 * o.g) = f;
                *reinterpret_cast<uint4*>(vx.data + (row + t) * vx.row + h * vx.head + 8 * o.g) = f;
            }
            continue;
        }
        const int64_t at = u.page * c.heads + h;
        const uint8_t* const kb = c.k + at * kBytes;
        const uint8_t* const vb = c.v + at * kBytes;
        const float sk = power_value(clamp_power(c.k_power[at])), sv = power_value(clamp_power(c.v_power[at]));
        // keys: a lane takes whole 16-byte pieces, D / 16 lanes a position
        constexpr int kPieces = D / 16;
        const int piece = threadIdx.x % kPieces, t1 = threadIdx.x / kPieces;  // positions t1 and t1 + 32
        const uint4* const kp = reinterpret_cast<const uint4*>(kb) + piece * kKvBlock + t1;
        const int s1 = wave * 128 + lane;
        const uint4 v0 = reinterpret_cast<const uint4*>(vb)[s1], v1 = reinterpret_cast<const uint4*>(vb)[s1 + 64];
        uint4 k0 = kp[0], k1 = kp[32];
        // all loads are issued here: without this the compiler moves the keys'
        // into the branches below, one wait for memory after the other
        asm volatile("" : "+v"(k0.x), "+v"(k0.y), "+v"(k0.z), "+v"(k0.w), "+v"(k1.x), "+v"(k1.y), "+v"(k1.z), "+v"(k1.w));
        reinterpret_cast<uint4*>(stage)[s1 ^ ((s1 >> 3) & 7)] = v0;
        reinterpret_cast<uint4*>(stage)[(s1 + 64) ^ ((s1 >> 3) & 7)] = v1;
        const auto store_key = [&](int t, uint4 w) {
            if (t < lo || t >= hi) return;
            uint4* p = reinterpret_cast<uint4*>(kx.data + (row + t) * kx.row + h * kx.head + 16 * piece);
            p[0] = make_uint4(fp8_to_bf16x2<false>(w.x, sk), fp8_to_bf16x2<true>(w.x, sk),
                              fp8_to_bf16x2<false>(w.y, sk), fp8_to_bf16x2<true>(w.y, sk));
            p[1] = make_uint4(fp8_to_bf16x2<false>(w.z, sk), fp8_to_bf16x2<true>(w.z, sk),
                              fp8_to_bf16x2<false>(w.w, sk), fp8_to_bf16x2<true>(w.w, sk));
        };
        store_key(t1, k0);
        store_key(t1 + 32, k1);
        wave_lds_sync();
        // values: 4 positions of 8 dims, dword d holding dim d of all four
        const int s0 = o.piece * D + 8 * o.g;
        uint32_t a[8], b[8];  // positions 0, 1 and 2, 3 of each dim
#pragma unroll
        for (int d = 0; d < 8; ++d) {
            const uint32_t w = stage[4 * ((s0 + d) ^ (((s0 + d) >> 3) & 7)) + o.em];
            a[d] = fp8_to_bf16x2<false>(w, sv);
            b[d] = fp8_to_bf16x2<true>(w, sv);
        }
        wave_lds_sync();
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int t = o.t0 + j;
            if (t < lo || t >= hi) continue;
            uint32_t w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t x = j < 2 ? a[2 * i] : b[2 * i], y = j < 2 ? a[2 * i + 1] : b[2 * i + 1];
                w[i] = j & 1 ? (x >> 16) | (y & 0xFFFF0000u) : (x & 0xFFFFu) | (y << 16);
            }
            *reinterpret_cast<uint4*>(vx.data + (row + t) * vx.row + h * vx.head + 8 * o.g) =
                make_uint4(w[0], w[1], w[2], w[3]);
        }
    }
}

// Rows a sequence (on average) up to which the short writer is taken, with one
// wave up to one row and four above.  256 single tokens of 56 heads, when units
// were still counted by sequences: 21 us with one wave (15 now), 48 with four,
// 110 with the long writer.  8 heads, 32 sequences of 4 rows: 5.1 us with four
// waves, 8.9 with the long writer.  One of 60 rows and 63 of one: 10 and 15 us;
// one of 100 and 15 of one (7 on average): 19 and 9.  What the rule costs where
// the rows are one sequence's: 60 rows beside 63 sequences of none take 20 to 27
// us, 10 with the long writer; 1000 rows among 255 empty slots 17 us for 8 heads
// (6 alone, with the long writer), 50 for 56 (12).
constexpr int64_t kAppendRows = 4;

}  // namespace

hipError_t launch_rope_table(float2* table, int64_t rows, int32_t pairs, double theta, hipStream_t s) {
    const int64_t n = rows * pairs;
    rope_table_kernel<<<dim3((unsigned)((n + 255) / 256)), dim3(256), 0, s>>>(table, n, pairs, theta);
    return hipGetLastError();
}

hipError_t launch_rope(const HeadsIn& x, const HeadsOut& out, int64_t M, int32_t heads, int32_t dim, const RopeArgs& r,
                       hipStream_t s) {
    RopeGeo g;
    g.M = M;
    g.heads = heads;
    g.units = dim / 16;
    // one unit a thread at least; 4 rows where that leaves 8 workgroups for
    // each of 256 CUs
    const int64_t per_row = (int64_t)heads * g.units;
    int64_t rows = (256 + per_row - 1) / per_row;
    if (rows < 4 && M >= 4 * 2048) rows = 4;
    g.rows = (int32_t)clamp64(rows, 1, kRopeTurns / r.total);
    g.du = 256 % g.units;
    g.dh = 256 / g.units % heads;
    g.dr = 256 / g.units / heads;
    const dim3 grid((unsigned)((M + g.rows - 1) / g.rows)), block(256);
    if (r.split)
        rope_kernel<true><<<grid, block, 0, s>>>(x, out, r, g);
    else
        rope_kernel<false><<<grid, block, 0, s>>>(x, out, r, g);
    return hipGetLastError();
}

template <int D, int WAVES>
static void kv_append_of(const CacheArgs& c, const SeqArgs& q, const HeadsIn& k, const HeadsIn& v, const RopeArgs& r,
                         hipStream_t s) {
    const dim3 grid((unsigned)block_first(q.M, q.B, q.per_row), (unsigned)c.heads), block(64 * WAVES);
    if (r.axes == 0)
        kv_append_kernel<D, ROPE_NONE, WAVES><<<grid, block, 0, s>>>(c, q, k, v, r);
    else if (r.split)
        kv_append_kernel<D, ROPE_SPLIT, WAVES><<<grid, block, 0, s>>>(c, q, k, v, r);
    else
        kv_append_kernel<D, ROPE_PAIRS, WAVES><<<grid, block, 0, s>>>(c, q, k, v, r);
}

template <int D>
static void kv_write_of(const CacheArgs& c, const SeqArgs& q, const HeadsIn& k, const HeadsIn& v, const RopeArgs& r,
                        hipStream_t s) {
    const int64_t units = block_first(q.M, q.B, q.per_row);
    if (q.M <= q.B) return kv_append_of<D, 1>(c, q, k, v, r, s);
    if (q.M <= kAppendRows * q.B) return kv_append_of<D, 4>(c, q, k, v, r, s);
    const int each = kv_heads_each(units, c.heads, kKvWriteHeads);
    const dim3 grid((unsigned)units, (unsigned)((c.heads + each - 1) / each)), block(2 * D);
    if (r.axes == 0)
        kv_write_kernel<D, ROPE_NONE><<<grid, block, 0, s>>>(c, q, k, v, r, each);
    else if (r.split)
        kv_write_kernel<D, ROPE_SPLIT><<<grid, block, 0, s>>>(c, q, k, v, r, each);
    else
        kv_write_kernel<D, ROPE_PAIRS><<<grid, block, 0, s>>>(c, q, k, v, r, each);
}

hipError_t launch_kv_write(const CacheArgs& c, const SeqArgs& seqs, const HeadsIn& k, const HeadsIn& v, const RopeArgs& r,
                           hipStream_t s) {
    SeqArgs q = seqs;
    q.per_row = blocks_per_row(q.M, q.B);
    if (c.dim == 128)
        kv_write_of<128>(c, q, k, v, r, s);
    else
        kv_write_of<64>(c, q, k, v, r, s);
    return hipGetLastError();
}

hipError_t launch_kv_read(const CacheArgs& c, const SeqArgs& seqs, const HeadsOut& k, const HeadsOut& v, hipStream_t s) {
    SeqArgs q = seqs;
    q.per_row = blocks_per_row(q.M, q.B);
    const int64_t units = block_first(q.M, q.B, q.per_row);
    const int each = kv_heads_each(units, c.heads, kKvReadHeads);
    const dim3 grid((unsigned)units, (unsigned)((c.heads + each - 1) / each));
    if (c.dim == 128)
        kv_read_kernel<128><<<grid, dim3(256), 0, s>>>(c, q, k, v, each);
    else
        kv_read_kernel<64><<<grid, dim3(128), 0, s>>>(c, q, k, v, each);
    return hipGetLastError();
}

}  // namespace nvfp4
