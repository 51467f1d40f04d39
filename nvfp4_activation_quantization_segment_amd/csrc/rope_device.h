// Looking up a row's rotary angles, shared by the kernels that rotate.
#pragma once

#include "kv_device.h"

namespace nvfp4 {

// The axes as values of their own: held in an array, picking one by a pair's
// index would put the array into scratch memory.
struct Axes {
    int32_t first1, first2, first3;      // first pairs of axes 1 to 3
    int32_t n0, n1, n2, n3;              // pairs
    int32_t rows0, rows1, rows2, rows3;  // positions covered
    int64_t to1, to2, to3;               // bytes from the first table to the others
    const char* table;
};
__device__ __forceinline__ Axes axes_of(const RopeArgs& r) {
    const auto to = [&](int a) { return (int64_t)((uintptr_t)r.table[a] - (uintptr_t)r.table[0]); };
    return Axes{r.first[1], r.first[2], r.first[3],
                r.first[1], r.first[2] - r.first[1], r.first[3] - r.first[2], r.first[4] - r.first[3],
                r.rows[0],  r.rows[1], r.rows[2], r.rows[3],
                to(1), to(2), to(3), reinterpret_cast<const char*>(r.table[0])};
}
// A row's positions, loaded once for all its pairs.
struct Positions {
    int32_t p0, p1, p2, p3;
};
__device__ __forceinline__ Positions positions_of(const RopeArgs& r, int64_t row) {
    const int32_t* src = r.positions + row * r.ld_positions;
    const int last = r.axes - 1;
    return Positions{src[0], src[last < 1 ? last : 1], src[last < 2 ? last : 2], src[last < 3 ? last : 3]};
}
// (cos, sin) of pair i of the rotated ones: the axis is picked with selects
// (the first pairs of axes not in use are past every i) and one load follows,
// so that a thread's loads are all in flight together.  A position outside its
// table gives NaN (an entry inside is loaded in its place).
__device__ __forceinline__ float2 rope_turn(const Axes x, const Positions pos, int i) {
    const bool a1 = i >= x.first1, a2 = i >= x.first2, a3 = i >= x.first3;
    const int32_t p = a3 ? pos.p3 : a2 ? pos.p2 : a1 ? pos.p1 : pos.p0;
    const int32_t rows = a3 ? x.rows3 : a2 ? x.rows2 : a1 ? x.rows1 : x.rows0;
    const int32_t n = a3 ? x.n3 : a2 ? x.n2 : a1 ? x.n1 : x.n0;
    const int32_t first = a3 ? x.first3 : a2 ? x.first2 : a1 ? x.first1 : 0;
    const int64_t to = a3 ? x.to3 : a2 ? x.to2 : a1 ? x.to1 : 0;
    const bool ok = (uint32_t)p < (uint32_t)rows;
    // a table is below 2^31 bytes: the offset inside it is a 32-bit one
    const uint32_t at = (ok ? (uint32_t)(p * n + (i - first)) : 0u) * (uint32_t)sizeof(float2);
    const float2 t = *reinterpret_cast<const float2*>(x.table + to + at);
    const float nan = __uint_as_float(0x7FC00000u);
    return make_float2(ok ? t.x : nan, ok ? t.y : nan);
}

}  // namespace nvfp4
