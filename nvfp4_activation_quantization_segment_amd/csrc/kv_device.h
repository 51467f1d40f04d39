// Device helpers shared by the cache and attention kernels.
#pragma once

#include "kv_internal.h"
#include "kv_layout.h"
#include "nvfp4_device.h"

namespace nvfp4 {

// 16 bytes as the compiler keeps them in registers.  (Arrays of HIP's own uint4
// struct, copied between memories, have been left in scratch memory.)
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

// 2^(b - 127) for a power byte 1..254.
__device__ __forceinline__ float power_value(uint32_t b) { return __uint_as_float(b << 23); }
// Its reciprocal, exactly.
__device__ __forceinline__ float power_inverse(uint32_t b) { return __uint_as_float((254u - b) << 23); }

// The byte of the smallest power of two p with amax <= 448 p, of a finite bf16
// magnitude: 448 = 1.75 * 2^8, so p is amax's own power of two over 2^8, or
// over 2^7 where the fraction is above 1.75.  At least 1 (zero blocks), which
// leaves the cache's values exact: a bf16 is a multiple of 2^-133 = 2^-7 p.
__device__ __forceinline__ uint32_t power_for(uint32_t amax16) {
    const int e = (int)(amax16 >> 7) - 8 + ((amax16 & 0x7Fu) > 0x60u ? 1 : 0);
    return (uint32_t)(e < 1 ? 1 : e);
}
__device__ __forceinline__ uint32_t clamp_power(uint32_t b) { return b < 1u ? 1u : b > 254u ? 254u : b; }

__device__ __forceinline__ int64_t uniform64(int64_t v) {
    const uint32_t lo = (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)v);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_readfirstlane((int)(v >> 32));
    return (int64_t)(((uint64_t)hi << 32) | lo);
}

// The sequence whose units start at or before `unit`, with its rows and length.
// base(row, b), the first unit of a sequence whose first row it is, is
// nondecreasing.  All 64 lanes take part.  Below 64 sequences everything comes
// from one pair of loads, so that a short kernel waits for memory once and not
// three times; above, each round looks at 64 places at once.
struct Located {
    int64_t b;
    int64_t start, end;  // row_start[b], row_start[b + 1] as they stand
    int64_t len;
};
template <class Base>
__device__ __forceinline__ Located locate(const SeqArgs& q, int64_t unit, Base base) {
    const int lane = threadIdx.x & 63;
    if (q.B < 64) {
        const int32_t start = q.row_start[lane < q.B ? lane : q.B];
        const int32_t len = q.lens[lane < q.B ? lane : 0];
        const bool ok = lane < q.B && (lane == 0 || base(clamp64(start, 0, q.M), lane) <= unit);
        const int b = 63 - __builtin_clzll(__ballot(ok));
        return Located{b, __builtin_amdgcn_readlane(start, b), __builtin_amdgcn_readlane(start, b + 1),
                       __builtin_amdgcn_readlane(len, b)};
    }
    int64_t lo = 0, n = q.B;
    while (n > 1) {
        const int64_t stride = (n + 63) / 64;
        const int64_t at = lane * stride;
        const bool ok = at < n && (lane == 0 || base(clamp64(q.row_start[lo + at], 0, q.M), lo + at) <= unit);
        const int64_t skip = (63 - __builtin_clzll(__ballot(ok))) * stride;
        lo += skip;
        n = n - skip < stride ? n - skip : stride;
    }
    lo = uniform64(lo);
    return Located{lo, q.row_start[lo], q.row_start[lo + 1], q.lens[lo]};
}

// Orders a wave's own LDS writes before its lanes' reads of one another's.
__device__ __forceinline__ void wave_lds_sync() {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

__device__ __forceinline__ uint32_t fp8_pack4(float a, float b, float c, float d) {
    int w = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
    return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c, d, w, true);
}

// Two E4M3 codes (low or high half of w) times a power of two -> packed bf16.
template <bool HIGH>
__device__ __forceinline__ uint32_t fp8_to_bf16x2(uint32_t w, float scale) {
    const bf16x2 r = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, scale, HIGH);
    return __builtin_bit_cast(uint32_t, r);
}

// Whether any of the four codes is one of E4M3's two NaN codes (0x7F, 0xFF).
__device__ __forceinline__ bool fp8_any_nan(uint32_t w) { return (((w & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u) != 0; }

}  // namespace nvfp4
