// Launch interface of the rotary, cache and attention kernels.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/nvfp4.h"

namespace nvfp4 {

// Records the HIP error for nvfp4_last_hip_error (api.hip).
nvfp4_status report_hip(hipError_t e);

// Heads [rows, heads, dim], unit stride along dim.
struct HeadsIn {
    const uint16_t* data;
    int64_t row, head;
};
struct HeadsOut {
    uint16_t* data;
    int64_t row, head;
};

struct RopeArgs {
    int32_t axes;
    int32_t total;     // rotated pairs of a head
    int32_t first[5];  // first pair of each axis; first[axes..] = total
    int32_t rows[4];
    const float2* table[4];
    const int32_t* positions;
    int64_t ld_positions;
    int32_t split;
};

struct CacheArgs {
    uint8_t* k;
    uint8_t* v;
    uint8_t* k_power;
    uint8_t* v_power;
    int64_t blocks;
    int32_t heads;
    int32_t dim;
};

struct SeqArgs {
    int64_t M;
    int64_t B;
    const int32_t* row_start;
    const int32_t* lens;
    const int32_t* table;
    int64_t ld_table;
    int64_t table_blocks;
    int32_t per_row;   // work units of a row, 0: counted by sequences (kv_layout.h)
};

struct AttentionArgs {
    HeadsIn q;
    HeadsOut out;
    CacheArgs cache;
    SeqArgs seqs;
    int32_t q_heads;
    int32_t group;     // query heads per key/value head
    float scale_log2;  // scale * log2(e)
    int32_t causal;
    int32_t wide;      // 128 rows to a workgroup (else 32)
    int32_t parts;     // pieces the keys of a row tile are cut into
    float* partial;    // parts x (M q_heads) x D, then parts x (M q_heads) x 2
};

hipError_t launch_rope_table(float2* table, int64_t rows, int32_t pairs, double theta, hipStream_t s);
hipError_t launch_rope(const HeadsIn& x, const HeadsOut& out, int64_t M, int32_t heads, int32_t dim, const RopeArgs& r,
                       hipStream_t s);
// r.axes = 0: the keys are not rotated.
hipError_t launch_kv_write(const CacheArgs& c, const SeqArgs& q, const HeadsIn& k, const HeadsIn& v, const RopeArgs& r,
                           hipStream_t s);
hipError_t launch_kv_read(const CacheArgs& c, const SeqArgs& q, const HeadsOut& k, const HeadsOut& v, hipStream_t s);

// How an attention call is cut: from sizes the host knows.
struct AttentionPlan {
    bool wide;
    int32_t parts;
    size_t workspace_bytes;
};
AttentionPlan attention_plan(int64_t M, int64_t B, int32_t q_heads, int32_t kv_heads, int32_t dim, int64_t max_len);
hipError_t launch_attention(const AttentionArgs& a, hipStream_t s);

}  // namespace nvfp4
