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

// One of the two inputs of the norms (queries, keys), and how its rows are
// shared out (set by the launcher).
struct NormPart {
    HeadsIn x;
    HeadsOut out;
    const uint16_t* weight;          // null: ones
    int32_t heads;                   // 0: none
    int32_t rows;                    // rows of a workgroup
    int32_t step_heads, step_rows;   // from one head of a lane to its next
    uint32_t groups;
};
struct NormArgs {
    NormPart part[2];
    RopeArgs rope;       // total = 0: not rotated
    int64_t M;
    int32_t units;       // of 16 dims in a head
    int32_t log_lanes;   // lanes of a head: the next power of two (set by the launcher)
    float inverse_dim, eps;
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

struct ExtendArgs {
    int64_t B, M;
    const int32_t* past;
    const int32_t* more;
    int32_t* table;
    int64_t ld_table, table_blocks;
    const int32_t* free_blocks;
    int64_t capacity;
    const int32_t* free_count;
    int32_t* row_start;
    int32_t* lens;
    int32_t* free_left;
    int32_t* missing;
    int32_t* positions;   // or null
    int64_t* slots;       // or null
    int32_t* state;       // workspace: free blocks before
    int32_t* taken;       // workspace: [B] blocks that the requests before take
};

struct ReleaseArgs {
    int64_t B;
    const int32_t* lens;
    const int32_t* done;
    const int32_t* table;
    int64_t ld_table, table_blocks, keep;
    int32_t done_len;     // what a finished request's length becomes
    int32_t* free_blocks;
    int64_t capacity;
    const int32_t* free_count;
    int32_t* lens_out;
    int32_t* free_left;
    int32_t* state;       // workspace: free blocks before
    int64_t* totals;      // workspace: blocks of each workgroup's requests
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
    int32_t first_part, all_parts;  // the first of them, and how many are joined
    float* partial;    // all_parts x (M q_heads) x D, then all_parts x (M q_heads) x 2
    int32_t window;    // last positions that a row sees, 0: all
    int32_t sinks;     // and first ones
    int64_t shared;    // blocks of the shared prefix
    int32_t prefix;    // the rows are taken against it (else against what is behind it)
};

hipError_t launch_rope_table(float2* table, int64_t rows, int32_t pairs, double theta, hipStream_t s);
hipError_t launch_rope(const HeadsIn& x, const HeadsOut& out, int64_t M, int32_t heads, int32_t dim, const RopeArgs& r,
                       hipStream_t s);
hipError_t launch_norm_rope(const NormArgs& a, hipStream_t s);
// r.axes = 0: the keys are not rotated.
hipError_t launch_kv_write(const CacheArgs& c, const SeqArgs& q, const HeadsIn& k, const HeadsIn& v, const RopeArgs& r,
                           hipStream_t s);
hipError_t launch_kv_read(const CacheArgs& c, const SeqArgs& q, const HeadsOut& k, const HeadsOut& v, hipStream_t s);

hipError_t launch_kv_extend(const ExtendArgs& a, hipStream_t s);
int64_t kv_release_groups(int64_t B);  // workgroups of a release
hipError_t launch_kv_release(const ReleaseArgs& a, hipStream_t s);
hipError_t launch_kv_clear_rest(const HeadsOut& out, int64_t M, int32_t heads, int32_t dim, const int32_t* row_start, int64_t B,
                                hipStream_t s);

// How an attention call is cut: from sizes the host knows.
struct AttentionPlan {
    bool wide;
    int32_t parts;
    size_t workspace_bytes;
};
AttentionPlan attention_plan(int64_t M, int64_t B, int32_t q_heads, int32_t kv_heads, int32_t dim, int64_t max_len);
hipError_t launch_attention(const AttentionArgs& a, hipStream_t s);

// The same through a window.
AttentionPlan window_plan(int64_t M, int64_t B, int32_t q_heads, int32_t kv_heads, int32_t dim, int64_t max_len,
                          int32_t causal, int32_t window, int32_t sinks);

// A call over a shared prefix: its workgroups, tiles of a head and all of them.  (The
// pieces of the prefix are those before the sequences' first one.)
struct SharedGrid {
    const int32_t* shared;  // the prefix's blocks
    uint32_t prefix_units, prefix_groups, own_units, own_groups;
};

// How a call over a shared prefix is cut: all rows against it, and each sequence's
// against its own keys.
struct SharedPlan {
    AttentionPlan prefix, own;
    size_t workspace_bytes;
};
SharedPlan shared_plan(int64_t M, int64_t B, int32_t q_heads, int32_t kv_heads, int32_t dim, int64_t max_len, int64_t shared);
hipError_t launch_attention_shared(const AttentionArgs& a, const SharedPlan& p, const int32_t* shared, hipStream_t s);

}  // namespace nvfp4
