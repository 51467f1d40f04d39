// Norms of query and key heads with the rotary positions in the same pass:
//   n_i = x_i w_i / sqrt(mean_j x_j^2 + eps),  y1 = n1 c - n2 s,  y2 = n2 c + n1 s,
// over each head of the queries and of the keys, in binary32 from the elements
// to the one rounding to bf16.  Every element is read once and written once:
// bound by memory.  37,810 rows of 56 and 56 heads of 128, three axes: 412 us,
// 5.26 TB/s read and written (a copy of 2 GiB reaches 4.9); 32 rows of 32 and 8
// heads 3.4 us in a graph, a chain of positions, angles and sums.
#include "kv_device.h"
#include "rope_device.h"

namespace nvfp4 {
namespace {

constexpr int kThreads = 256;
constexpr int kTurns = 1024;  // angles a workgroup holds

template <int CONTROL>
__device__ __forceinline__ float dpp_move(float x) {
    return __uint_as_float((uint32_t)__builtin_amdgcn_update_dpp(0, (int)__float_as_uint(x), CONTROL, 0xF, 0xF, true));
}

// The sum over the 2^n neighbouring lanes of a head (`lanes` of them), in each.
__device__ __forceinline__ float head_sum(float x, int lanes) {
    if (lanes > 1) x += dpp_move<0xB1>(x);    // lane ^ 1
    if (lanes > 2) x += dpp_move<0x4E>(x);    // lane ^ 2
    if (lanes > 4) x += dpp_move<0x141>(x);   // 7 - lane: the other four, all equal by now
    if (lanes > 8) x += dpp_move<0x140>(x);   // 15 - lane
    if (lanes > 16) x += __shfl_xor(x, 16);
    return x;
}

__device__ __forceinline__ void rotate(float& n1, float& n2, float2 turn) {
    const float y1 = n1 * turn.x - n2 * turn.y, y2 = n2 * turn.x + n1 * turn.y;
    n1 = y1;
    n2 = y2;
}
template <int N>
__device__ __forceinline__ void angles(float2 (&c)[N], const float2* t) {
#pragma unroll
    for (int i = 0; i < N / 2; ++i) {
        const float4 v = reinterpret_cast<const float4*>(t)[i];
        c[2 * i] = make_float2(v.x, v.y);
        c[2 * i + 1] = make_float2(v.z, v.w);
    }
}

template <bool STREAM>
__device__ __forceinline__ void store(uint16_t* p, const float* f) {
    const u32x4 v = {pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7])};
    if constexpr (STREAM)
        __builtin_nontemporal_store(v, reinterpret_cast<u32x4*>(p));
    else
        *reinterpret_cast<u32x4*>(p) = v;
}

// A workgroup takes a few rows of the queries or of the keys; a unit of 16 dims
// of a head, two times 8 of them, is a lane's, and a head's units are
// neighbouring lanes (as many as the next power of two), so that its sum stays in
// the wave.  The first 8 dims of neighbouring lanes lie side by side, and the
// second 8 half a head (or half of what is rotated, or of what is not) further on:
// every load and store of theirs is whole lines.  The angles of the rows are
// looked up once, into LDS, and the next unit's loads are ahead of this one's sum
// and stores.  A lane's dims are the same in every head it takes: its weights stay
// in registers.
template <bool SPLIT, bool STREAM>
__global__ __launch_bounds__(kThreads) void norm_rope_kernel(NormArgs a) {
    __shared__ __align__(16) float2 turn[kTurns];
    const bool keys = blockIdx.x >= a.part[0].groups;
    const NormPart& p = a.part[keys];
    const int64_t row0 = (int64_t)(blockIdx.x - (keys ? a.part[0].groups : 0)) * p.rows;
    const int rows = (int)(a.M - row0 < p.rows ? a.M - row0 : p.rows);
    const int lanes = 1 << a.log_lanes;
    const int u = threadIdx.x & (lanes - 1);
    const bool mine = u < a.units;
    const int total = a.rope.total, turning = total / 8;
    // SPLIT: the first and second elements of 8 pairs, or what is not rotated
    const int after = 2 * total + 8 * (u - turning), rest = 8 * (a.units - turning);
    const int low = SPLIT && u >= turning ? after : 8 * u;
    const int high = !SPLIT ? 8 * (a.units + u) : u < turning ? total + 8 * u : after + rest;
    int at = threadIdx.x >> a.log_lanes;
    int h = at % p.heads, in = at / p.heads;
    const auto load = [&](u32x4& x, u32x4& y) {
        const uint16_t* src = p.x.data + (row0 + in) * p.x.row + h * p.x.head;
        x = *reinterpret_cast<const u32x4*>(src + low);
        y = *reinterpret_cast<const u32x4*>(src + high);
    };
    u32x4 x = {0, 0, 0, 0}, y = x;
    if (mine && in < rows) load(x, y);  // on its way while the angles are looked up
    float w[16];
    if (p.weight && mine) {
        const u32x4 wl = *reinterpret_cast<const u32x4*>(p.weight + low), wh = *reinterpret_cast<const u32x4*>(p.weight + high);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            w[2 * i] = bf16_lo(wl[i]), w[2 * i + 1] = bf16_hi(wl[i]);
            w[8 + 2 * i] = bf16_lo(wh[i]), w[8 + 2 * i + 1] = bf16_hi(wh[i]);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 16; ++i) w[i] = 1.0f;
    }
    if (total > 0) {
        const Axes axes = axes_of(a.rope);
        for (int i = threadIdx.x; i < rows * total; i += kThreads) {
            const int j = i / total;
            turn[i] = rope_turn(axes, positions_of(a.rope, row0 + j), i - j * total);
        }
        __syncthreads();
    }
    while (in < rows) {
        const float2* t = turn + in * total;
        uint16_t* out = p.out.data + (row0 + in) * p.out.row + h * p.out.head;
        float f[16];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[2 * i] = bf16_lo(x[i]), f[2 * i + 1] = bf16_hi(x[i]);
            f[8 + 2 * i] = bf16_lo(y[i]), f[8 + 2 * i + 1] = bf16_hi(y[i]);
        }
        h += p.step_heads;
        in += p.step_rows;
        if (h >= p.heads) h -= p.heads, ++in;
        if (mine && in < rows) load(x, y);
        float part[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int i = 0; i < 16; ++i) part[i & 3] = __builtin_fmaf(f[i], f[i], part[i & 3]);
        const float sum = head_sum((part[0] + part[1]) + (part[2] + part[3]), lanes);
        float r = __builtin_amdgcn_rsqf(__builtin_fmaf(sum, a.inverse_dim, a.eps));
        const bool over = !(sum < __uint_as_float(0x7F800000u));
        if (__any(over)) {
            // Elements that are not finite, or whose squares leave binary32: the
            // squares of elements below 2^128 over 2^70, up to 512 of them, do
            // not.  (An infinite element still gives an infinite sum, and r = 0.)
            const float down = over ? 0x1p-70f : 1.0f;
            float again = 0.0f;
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                f[i] *= down;
                again = __builtin_fmaf(f[i], f[i], again);
            }
            again = head_sum(again, lanes);
            const float q = __builtin_amdgcn_rsqf(__builtin_fmaf(again, a.inverse_dim, a.eps * 0x1p-140f));
            r = over ? q : r;
        }
#pragma unroll
        for (int i = 0; i < 16; ++i) f[i] = f[i] * r * w[i];
        if constexpr (SPLIT) {
            if (u < turning) {
                float2 c[8];
                angles<8>(c, t + 8 * u);
#pragma unroll
                for (int i = 0; i < 8; ++i) rotate(f[i], f[8 + i], c[i]);
            }
        } else {
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                const int pair = 4 * (half * a.units + u);
                if (pair < total) {
                    float2 c[4];
                    angles<4>(c, t + pair);
#pragma unroll
                    for (int i = 0; i < 4; ++i) rotate(f[8 * half + 2 * i], f[8 * half + 2 * i + 1], c[i]);
                }
            }
        }
        if (mine) {
            store<STREAM>(out + low, f);
            store<STREAM>(out + high, f + 8);
        }
    }
}

}  // namespace

hipError_t launch_norm_rope(const NormArgs& args, hipStream_t s) {
    NormArgs a = args;
    a.log_lanes = 0;
    while ((1 << a.log_lanes) < a.units) ++a.log_lanes;
    const int together = kThreads >> a.log_lanes;  // heads that a workgroup takes at a time
    for (NormPart& p : a.part) {
        if (p.heads == 0) continue;
        // a unit a thread at least; 4 rows where that leaves 8 workgroups for each
        // of 256 CUs
        int64_t rows = (together + p.heads - 1) / p.heads;
        if (rows < 4 && a.M >= 4 * 2048) rows = 4;
        const int64_t most = a.rope.total > 0 ? kTurns / a.rope.total : rows;
        p.rows = (int32_t)clamp64(rows, 1, most);
        p.step_heads = together % p.heads;
        p.step_rows = together / p.heads;
        p.groups = (uint32_t)((a.M + p.rows - 1) / p.rows);
    }
    // Outputs that the 256 MB memory-side cache does not hold are streamed past it,
    // others left there for the calls that read them.  (37,810 rows of 112 heads 412
    // us, 422 without; 30,000 of 40, split, 110 and 128; with 16 dims of a lane side
    // by side, so that stores covered halves of lines, streaming them took 446.)
    const int64_t heads = (int64_t)a.part[0].heads + a.part[1].heads;
    const bool stream = a.M * heads * a.units > ((int64_t)256 << 20) / 32;
    const dim3 grid(a.part[0].groups + a.part[1].groups), block(kThreads);
    if (a.rope.split && stream)
        norm_rope_kernel<true, true><<<grid, block, 0, s>>>(a);
    else if (a.rope.split)
        norm_rope_kernel<true, false><<<grid, block, 0, s>>>(a);
    else if (stream)
        norm_rope_kernel<false, true><<<grid, block, 0, s>>>(a);
    else
        norm_rope_kernel<false, false><<<grid, block, 0, s>>>(a);
    return hipGetLastError();
}

}  // namespace nvfp4
