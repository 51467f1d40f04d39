// C ABI of the rotary, norm, cache, table and attention entry points: argument
// validation.
// Every check happens before anything is enqueued.
#include <math.h>
#include <string.h>

#include "kv_internal.h"
#include "kv_layout.h"

using namespace nvfp4;

namespace {

constexpr int64_t kMaxRows = (int64_t)1 << 23;   // rows x threads of a row stay below 2^32
constexpr int64_t kMaxSeqs = (int64_t)1 << 20;
constexpr int32_t kMaxHeads = 65535;             // second dimension of a grid
constexpr int64_t kMaxTableBlocks = INT32_MAX / kKvBlock;

bool aligned(const void* p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) == 0; }

nvfp4_status check_heads(const nvfp4_heads* x, int64_t M, int64_t heads, int64_t dim, bool output) {
    if (!x || !x->data) return NVFP4_ERR_INVALID_ARGUMENT;
    if (x->row_stride < 0 || x->head_stride < 0) return NVFP4_ERR_INVALID_ARGUMENT;
    if (!aligned(x->data, 16) || x->row_stride % 8 != 0 || x->head_stride % 8 != 0) return NVFP4_ERR_ALIGNMENT;
    // the last head's offset stays inside 64 bits, in elements and in bytes
    constexpr int64_t kMost = (int64_t)1 << 38, kReach = (int64_t)1 << 60;
    if (x->row_stride > kMost || x->head_stride > kMost) return NVFP4_ERR_SHAPE;
    if ((M > 1 && x->row_stride > kReach / (M - 1)) || (heads > 1 && x->head_stride > kReach / (heads - 1)))
        return NVFP4_ERR_SHAPE;
    if (output) {
        const bool by_row = (heads == 1 || x->head_stride >= dim) &&
                            (M == 1 || x->row_stride >= (heads - 1) * x->head_stride + dim);
        const bool by_head = (M == 1 || x->row_stride >= dim) &&
                             (heads == 1 || x->head_stride >= (M - 1) * x->row_stride + dim);
        if (!by_row && !by_head) return NVFP4_ERR_INVALID_ARGUMENT;
    }
    return NVFP4_OK;
}

nvfp4_status check_rope(const nvfp4_rope_params* p, int64_t dim, RopeArgs* r) {
    memset(r, 0, sizeof(*r));
    if (!p->positions) return NVFP4_ERR_INVALID_ARGUMENT;
    if (p->axes < 1 || p->axes > NVFP4_ROPE_MAX_AXES) return NVFP4_ERR_SHAPE;
    if (p->ld_positions < p->axes) return NVFP4_ERR_INVALID_ARGUMENT;
    int64_t total = 0;
    for (int a = 0; a < p->axes; ++a) {
        if (!p->table[a]) return NVFP4_ERR_INVALID_ARGUMENT;
        if (p->pairs[a] < 1 || p->pairs[a] > dim / 2 || p->rows[a] < 1 || p->rows[a] > INT32_MAX) return NVFP4_ERR_SHAPE;
        if (p->rows[a] * p->pairs[a] >= (int64_t)1 << 28) return NVFP4_ERR_SHAPE;
        if (!aligned(p->table[a], 8)) return NVFP4_ERR_ALIGNMENT;
        r->first[a] = (int32_t)total;
        r->rows[a] = (int32_t)p->rows[a];
        r->table[a] = reinterpret_cast<const float2*>(p->table[a]);
        total += p->pairs[a];
    }
    if (total % 8 != 0 || total > dim / 2) return NVFP4_ERR_SHAPE;
    if (!aligned(p->positions, 4)) return NVFP4_ERR_ALIGNMENT;
    for (int a = p->axes; a < 5; ++a) r->first[a] = (int32_t)total;
    r->axes = p->axes;
    r->total = (int32_t)total;
    r->positions = p->positions;
    r->ld_positions = p->ld_positions;
    r->split = p->split != 0;
    return NVFP4_OK;
}

nvfp4_status check_cache(const nvfp4_kv_cache* c, CacheArgs* a) {
    if (!c || !c->k || !c->v || !c->k_power || !c->v_power) return NVFP4_ERR_INVALID_ARGUMENT;
    if (c->blocks < 1 || c->heads < 1) return NVFP4_ERR_INVALID_ARGUMENT;
    if ((c->dim != 64 && c->dim != 128) || c->heads > kMaxHeads || c->blocks > INT32_MAX) return NVFP4_ERR_SHAPE;
    if (!aligned(c->k, 16) || !aligned(c->v, 16)) return NVFP4_ERR_ALIGNMENT;
    *a = CacheArgs{c->k, c->v, c->k_power, c->v_power, c->blocks, c->heads, c->dim};
    return NVFP4_OK;
}

nvfp4_status check_sequences(const nvfp4_kv_sequences* s, int64_t M, SeqArgs* a) {
    if (!s || !s->row_start || !s->lens || !s->table || M < 1 || s->count < 1) return NVFP4_ERR_INVALID_ARGUMENT;
    if (s->table_blocks < 1 || s->ld_table < s->table_blocks) return NVFP4_ERR_INVALID_ARGUMENT;
    if (M > kMaxRows || s->count > kMaxSeqs || s->table_blocks > kMaxTableBlocks) return NVFP4_ERR_SHAPE;
    if (!aligned(s->row_start, 4) || !aligned(s->lens, 4) || !aligned(s->table, 4)) return NVFP4_ERR_ALIGNMENT;
    *a = SeqArgs{M, s->count, s->row_start, s->lens, s->table, s->ld_table, s->table_blocks, 0};
    return NVFP4_OK;
}

constexpr size_t kStateBytes = 16;  // what a table call's launches hand on

nvfp4_status check_tables(const nvfp4_kv_tables* t) {
    if (!t || !t->table || !t->free_blocks || t->count < 1 || t->table_blocks < 1 || t->capacity < 1 ||
        t->ld_table < t->table_blocks)
        return NVFP4_ERR_INVALID_ARGUMENT;
    if (t->count > kMaxSeqs || t->table_blocks > kMaxTableBlocks || t->capacity > ((int64_t)1 << 30) ||
        t->ld_table > ((int64_t)1 << 60) / t->count)
        return NVFP4_ERR_SHAPE;
    if (!aligned(t->table, 4) || !aligned(t->free_blocks, 4)) return NVFP4_ERR_ALIGNMENT;
    return NVFP4_OK;
}

bool attention_sizes_ok(int64_t M, int64_t count, int64_t q_heads, int64_t heads, int64_t dim, int64_t max_len) {
    return M >= 1 && M <= kMaxRows && count >= 1 && count <= kMaxSeqs && heads >= 1 && heads <= kMaxHeads &&
           q_heads >= 1 && q_heads % heads == 0 && M * q_heads <= ((int64_t)1 << 28) && (dim == 64 || dim == 128) && max_len >= 0;
}

HeadsIn in(const nvfp4_heads* h) { return HeadsIn{h->data, h->row_stride, h->head_stride}; }
HeadsOut out_of(const nvfp4_heads* h) { return HeadsOut{h->data, h->row_stride, h->head_stride}; }

// The checks that every attention call makes, and what they describe.
nvfp4_status check_attention(const nvfp4_heads* q, int64_t M, int32_t q_heads, const nvfp4_kv_cache* cache,
                             const nvfp4_kv_sequences* seqs, float scale, int32_t causal_block, int64_t max_len,
                             const nvfp4_heads* out, AttentionArgs* a) {
    memset(a, 0, sizeof(*a));
    nvfp4_status st;
    if ((st = check_cache(cache, &a->cache)) != NVFP4_OK) return st;
    if ((st = check_sequences(seqs, M, &a->seqs)) != NVFP4_OK) return st;
    if (q_heads < 1 || causal_block < 0 || max_len < 0) return NVFP4_ERR_INVALID_ARGUMENT;
    const float scale_log2 = scale * 1.44269504088896340736f;
    if (!(scale > 0.0f) || !isfinite(scale_log2)) return NVFP4_ERR_INVALID_ARGUMENT;
    if (!attention_sizes_ok(M, seqs->count, q_heads, cache->heads, cache->dim, max_len)) return NVFP4_ERR_SHAPE;
    if ((st = check_heads(q, M, q_heads, cache->dim, false)) != NVFP4_OK) return st;
    if ((st = check_heads(out, M, q_heads, cache->dim, true)) != NVFP4_OK) return st;
    a->q = in(q);
    a->out = out_of(out);
    a->q_heads = q_heads;
    a->group = q_heads / cache->heads;
    a->scale_log2 = scale_log2;
    a->causal = causal_block;
    return NVFP4_OK;
}

// One launch over the sequences' keys (and the join), cut as planned.
nvfp4_status run_attention(AttentionArgs& a, const AttentionPlan& p, void* workspace, size_t workspace_bytes, void* stream) {
    if (p.workspace_bytes > 0 && (!workspace || workspace_bytes < p.workspace_bytes)) return NVFP4_ERR_INVALID_ARGUMENT;
    if (p.workspace_bytes > 0 && !aligned(workspace, 16)) return NVFP4_ERR_ALIGNMENT;
    a.wide = p.wide;
    a.parts = a.all_parts = p.parts;
    a.partial = (float*)workspace;
    return report_hip(launch_attention(a, (hipStream_t)stream));
}

// to_prefix: a finished request's length becomes that of the kept blocks, else 0.
nvfp4_status run_release(const nvfp4_kv_tables* tables, const int32_t* lens, const int32_t* done, int64_t keep, bool to_prefix,
                         const int32_t* free_count, int32_t* lens_out, int32_t* free_left, void* workspace,
                         size_t workspace_bytes, void* stream) {
    nvfp4_status st;
    if ((st = check_tables(tables)) != NVFP4_OK) return st;
    if (!lens || !done || !free_count || !lens_out || !free_left || keep < 0) return NVFP4_ERR_INVALID_ARGUMENT;
    if (!aligned(lens, 4) || !aligned(done, 4) || !aligned(free_count, 4) || !aligned(lens_out, 4) || !aligned(free_left, 4))
        return NVFP4_ERR_ALIGNMENT;
    const size_t need = nvfp4_kv_release_workspace_bytes(tables->count);
    if (need > 0 && (!workspace || workspace_bytes < need)) return NVFP4_ERR_INVALID_ARGUMENT;
    if (need > 0 && !aligned(workspace, 16)) return NVFP4_ERR_ALIGNMENT;
    ReleaseArgs a;
    a.B = tables->count;
    a.lens = lens;
    a.done = done;
    a.table = tables->table;
    a.ld_table = tables->ld_table;
    a.table_blocks = tables->table_blocks;
    a.keep = keep < tables->table_blocks ? keep : tables->table_blocks;
    a.done_len = to_prefix ? (int32_t)(a.keep * kKvBlock) : 0;
    a.free_blocks = tables->free_blocks;
    a.capacity = tables->capacity;
    a.free_count = free_count;
    a.lens_out = lens_out;
    a.free_left = free_left;
    a.state = (int32_t*)workspace;
    a.totals = (int64_t*)((char*)workspace + kStateBytes);
    return report_hip(launch_kv_release(a, (hipStream_t)stream));
}

}  // namespace

extern "C" {

nvfp4_status nvfp4_rope_table(float* table, int64_t rows, int32_t pairs, double theta, void* stream) {
    if (!table || rows < 1 || pairs < 1 || !(theta > 0.0) || !isfinite(theta)) return NVFP4_ERR_INVALID_ARGUMENT;
    if (rows > (((int64_t)1 << 28) - 1) / pairs) return NVFP4_ERR_SHAPE;
    if (!aligned(table, 8)) return NVFP4_ERR_ALIGNMENT;
    return report_hip(launch_rope_table(reinterpret_cast<float2*>(table), rows, pairs, theta, (hipStream_t)stream));
}

nvfp4_status nvfp4_rope(const nvfp4_heads* x, int64_t M, int32_t heads, int32_t dim, const nvfp4_rope_params* rope,
                        const nvfp4_heads* out, void* stream) {
    if (!rope || M < 1 || heads < 1 || dim < 1) return NVFP4_ERR_INVALID_ARGUMENT;
    if (dim % 16 != 0 || dim > 512 || M > kMaxRows || heads > kMaxHeads) return NVFP4_ERR_SHAPE;
    nvfp4_status st;
    if ((st = check_heads(x, M, heads, dim, false)) != NVFP4_OK) return st;
    if ((st = check_heads(out, M, heads, dim, true)) != NVFP4_OK) return st;
    RopeArgs r;
    if ((st = check_rope(rope, dim, &r)) != NVFP4_OK) return st;
    return report_hip(launch_rope(in(x), out_of(out), M, heads, dim, r, (hipStream_t)stream));
}

nvfp4_status nvfp4_norm_rope(const nvfp4_heads* q, int32_t q_heads, const uint16_t* q_weight, const nvfp4_heads* k,
                             int32_t k_heads, const uint16_t* k_weight, int64_t M, int32_t dim, float eps,
                             const nvfp4_rope_params* rope, const nvfp4_heads* q_out, const nvfp4_heads* k_out,
                             void* stream) {
    if (M < 1 || q_heads < 1 || k_heads < 0 || dim < 1) return NVFP4_ERR_INVALID_ARGUMENT;
    if (!(eps >= 0x1p-126f && eps <= 1.0f)) return NVFP4_ERR_INVALID_ARGUMENT;
    if (dim % 16 != 0 || dim > 512 || M > kMaxRows || q_heads > kMaxHeads || k_heads > kMaxHeads) return NVFP4_ERR_SHAPE;
    if (k_heads == 0 && (k || k_out || k_weight)) return NVFP4_ERR_INVALID_ARGUMENT;
    NormArgs a;
    memset(&a, 0, sizeof(a));
    const nvfp4_heads* xs[2] = {q, k};
    const nvfp4_heads* outs[2] = {q_out, k_out};
    const uint16_t* weights[2] = {q_weight, k_weight};
    const int32_t heads[2] = {q_heads, k_heads};
    nvfp4_status st;
    for (int i = 0; i < 2 && heads[i] > 0; ++i) {
        if ((st = check_heads(xs[i], M, heads[i], dim, false)) != NVFP4_OK) return st;
        if ((st = check_heads(outs[i], M, heads[i], dim, true)) != NVFP4_OK) return st;
        if (!aligned(weights[i], 16)) return NVFP4_ERR_ALIGNMENT;
        a.part[i].x = in(xs[i]);
        a.part[i].out = out_of(outs[i]);
        a.part[i].weight = weights[i];
        a.part[i].heads = heads[i];
    }
    if (rope && (st = check_rope(rope, dim, &a.rope)) != NVFP4_OK) return st;
    a.M = M;
    a.units = dim / 16;
    a.inverse_dim = 1.0f / (float)dim;
    a.eps = eps;
    return report_hip(launch_norm_rope(a, (hipStream_t)stream));
}

nvfp4_status nvfp4_kv_write(const nvfp4_kv_cache* cache, const nvfp4_kv_sequences* seqs, int64_t M,
                            const nvfp4_heads* k, const nvfp4_heads* v, const nvfp4_rope_params* rope, void* stream) {
    CacheArgs c;
    SeqArgs q;
    RopeArgs r;
    memset(&r, 0, sizeof(r));
    nvfp4_status st;
    if ((st = check_cache(cache, &c)) != NVFP4_OK) return st;
    if ((st = check_sequences(seqs, M, &q)) != NVFP4_OK) return st;
    if ((st = check_heads(k, M, c.heads, c.dim, false)) != NVFP4_OK) return st;
    if ((st = check_heads(v, M, c.heads, c.dim, false)) != NVFP4_OK) return st;
    if (rope && (st = check_rope(rope, c.dim, &r)) != NVFP4_OK) return st;
    return report_hip(launch_kv_write(c, q, in(k), in(v), r, (hipStream_t)stream));
}

nvfp4_status nvfp4_kv_read(const nvfp4_kv_cache* cache, const nvfp4_kv_sequences* seqs, int64_t M,
                           const nvfp4_heads* k, const nvfp4_heads* v, void* stream) {
    CacheArgs c;
    SeqArgs q;
    nvfp4_status st;
    if ((st = check_cache(cache, &c)) != NVFP4_OK) return st;
    if ((st = check_sequences(seqs, M, &q)) != NVFP4_OK) return st;
    if ((st = check_heads(k, M, c.heads, c.dim, true)) != NVFP4_OK) return st;
    if ((st = check_heads(v, M, c.heads, c.dim, true)) != NVFP4_OK) return st;
    return report_hip(launch_kv_read(c, q, out_of(k), out_of(v), (hipStream_t)stream));
}

size_t nvfp4_kv_extend_workspace_bytes(int64_t count) {
    return count < 1 || count > kMaxSeqs ? 0 : kStateBytes + (size_t)count * sizeof(int32_t);
}

nvfp4_status nvfp4_kv_extend(const nvfp4_kv_tables* tables, const int32_t* past, const int32_t* more,
                             const int32_t* free_count, int64_t M, int32_t* row_start, int32_t* lens, int32_t* free_left,
                             int32_t* missing, int32_t* positions, int64_t* slots, void* workspace,
                             size_t workspace_bytes, void* stream) {
    nvfp4_status st;
    if ((st = check_tables(tables)) != NVFP4_OK) return st;
    if (!past || !more || !free_count || !row_start || !lens || !free_left || !missing || M < 1)
        return NVFP4_ERR_INVALID_ARGUMENT;
    if (M > kMaxRows) return NVFP4_ERR_SHAPE;
    if (!aligned(past, 4) || !aligned(more, 4) || !aligned(free_count, 4) || !aligned(row_start, 4) || !aligned(lens, 4) ||
        !aligned(free_left, 4) || !aligned(missing, 4) || !aligned(positions, 4) || !aligned(slots, 8))
        return NVFP4_ERR_ALIGNMENT;
    if (!workspace || workspace_bytes < nvfp4_kv_extend_workspace_bytes(tables->count)) return NVFP4_ERR_INVALID_ARGUMENT;
    if (!aligned(workspace, 16)) return NVFP4_ERR_ALIGNMENT;
    ExtendArgs a;
    a.B = tables->count;
    a.M = M;
    a.past = past;
    a.more = more;
    a.table = tables->table;
    a.ld_table = tables->ld_table;
    a.table_blocks = tables->table_blocks;
    a.free_blocks = tables->free_blocks;
    a.capacity = tables->capacity;
    a.free_count = free_count;
    a.row_start = row_start;
    a.lens = lens;
    a.free_left = free_left;
    a.missing = missing;
    a.positions = positions;
    a.slots = slots;
    a.state = (int32_t*)workspace;
    a.taken = (int32_t*)((char*)workspace + kStateBytes);
    return report_hip(launch_kv_extend(a, (hipStream_t)stream));
}

size_t nvfp4_kv_release_workspace_bytes(int64_t count) {
    if (count < 1 || count > kMaxSeqs || kv_release_groups(count) == 1) return 0;
    return kStateBytes + (size_t)kv_release_groups(count) * sizeof(int64_t);
}

nvfp4_status nvfp4_kv_release(const nvfp4_kv_tables* tables, const int32_t* lens, const int32_t* done, int64_t keep,
                              const int32_t* free_count, int32_t* lens_out, int32_t* free_left, void* workspace,
                              size_t workspace_bytes, void* stream) {
    return run_release(tables, lens, done, keep, false, free_count, lens_out, free_left, workspace, workspace_bytes, stream);
}

nvfp4_status nvfp4_kv_release_to_prefix(const nvfp4_kv_tables* tables, const int32_t* lens, const int32_t* done, int64_t keep,
                                        const int32_t* free_count, int32_t* lens_out, int32_t* free_left, void* workspace,
                                        size_t workspace_bytes, void* stream) {
    return run_release(tables, lens, done, keep, true, free_count, lens_out, free_left, workspace, workspace_bytes, stream);
}

nvfp4_status nvfp4_kv_clear_rest(const nvfp4_heads* out, int64_t M, int32_t heads, int32_t dim, const int32_t* row_start,
                                 int64_t count, void* stream) {
    if (M < 1 || heads < 1 || dim < 1 || count < 1 || !row_start) return NVFP4_ERR_INVALID_ARGUMENT;
    if (dim % 16 != 0 || dim > 512 || M > kMaxRows || M * heads > ((int64_t)1 << 28) || count > kMaxSeqs) return NVFP4_ERR_SHAPE;
    const nvfp4_status st = check_heads(out, M, heads, dim, true);
    if (st != NVFP4_OK) return st;
    if (!aligned(row_start, 4)) return NVFP4_ERR_ALIGNMENT;
    return report_hip(launch_kv_clear_rest(out_of(out), M, heads, dim, row_start, count, (hipStream_t)stream));
}

size_t nvfp4_kv_attention_workspace_bytes(int64_t M, int64_t count, int32_t q_heads, int32_t heads, int32_t dim,
                                          int64_t max_len) {
    if (!attention_sizes_ok(M, count, q_heads, heads, dim, max_len)) return 0;
    return attention_plan(M, count, q_heads, heads, dim, max_len).workspace_bytes;
}

nvfp4_status nvfp4_kv_attention(const nvfp4_heads* q, int64_t M, int32_t q_heads, const nvfp4_kv_cache* cache,
                                const nvfp4_kv_sequences* seqs, float scale, int32_t causal_block, int64_t max_len,
                                const nvfp4_heads* out, void* workspace, size_t workspace_bytes, void* stream) {
    AttentionArgs a;
    const nvfp4_status st = check_attention(q, M, q_heads, cache, seqs, scale, causal_block, max_len, out, &a);
    if (st != NVFP4_OK) return st;
    return run_attention(a, attention_plan(M, seqs->count, q_heads, cache->heads, cache->dim, max_len), workspace,
                         workspace_bytes, stream);
}

size_t nvfp4_kv_attention_window_workspace_bytes(int64_t M, int64_t count, int32_t q_heads, int32_t heads, int32_t dim,
                                                 int32_t causal_block, int32_t window, int32_t sinks, int64_t max_len) {
    if (!attention_sizes_ok(M, count, q_heads, heads, dim, max_len) || causal_block < 0 || window < 1 || sinks < 0) return 0;
    return window_plan(M, count, q_heads, heads, dim, max_len, causal_block, window, sinks).workspace_bytes;
}

nvfp4_status nvfp4_kv_attention_window(const nvfp4_heads* q, int64_t M, int32_t q_heads, const nvfp4_kv_cache* cache,
                                       const nvfp4_kv_sequences* seqs, float scale, int32_t causal_block, int32_t window,
                                       int32_t sinks, int64_t max_len, const nvfp4_heads* out, void* workspace,
                                       size_t workspace_bytes, void* stream) {
    AttentionArgs a;
    const nvfp4_status st = check_attention(q, M, q_heads, cache, seqs, scale, causal_block, max_len, out, &a);
    if (st != NVFP4_OK) return st;
    if (window < 1 || sinks < 0) return NVFP4_ERR_INVALID_ARGUMENT;
    a.window = window;
    a.sinks = sinks;
    return run_attention(a, window_plan(M, seqs->count, q_heads, cache->heads, cache->dim, max_len, causal_block, window, sinks),
                         workspace, workspace_bytes, stream);
}

size_t nvfp4_kv_attention_shared_workspace_bytes(int64_t M, int64_t count, int32_t q_heads, int32_t heads, int32_t dim,
                                                 int64_t shared_blocks, int64_t max_len) {
    if (!attention_sizes_ok(M, count, q_heads, heads, dim, max_len) || shared_blocks < 1 || shared_blocks > kMaxTableBlocks)
        return 0;
    return shared_plan(M, count, q_heads, heads, dim, max_len, shared_blocks).workspace_bytes;
}

nvfp4_status nvfp4_kv_attention_shared(const nvfp4_heads* q, int64_t M, int32_t q_heads, const nvfp4_kv_cache* cache,
                                       const nvfp4_kv_sequences* seqs, const int32_t* shared, int64_t shared_blocks,
                                       float scale, int32_t causal_block, int64_t max_len, const nvfp4_heads* out,
                                       void* workspace, size_t workspace_bytes, void* stream) {
    AttentionArgs a;
    const nvfp4_status st = check_attention(q, M, q_heads, cache, seqs, scale, causal_block, max_len, out, &a);
    if (st != NVFP4_OK) return st;
    if (!shared || shared_blocks < 1) return NVFP4_ERR_INVALID_ARGUMENT;
    if (shared_blocks > kMaxTableBlocks) return NVFP4_ERR_SHAPE;
    if (!aligned(shared, 4)) return NVFP4_ERR_ALIGNMENT;
    const SharedPlan p = shared_plan(M, seqs->count, q_heads, cache->heads, cache->dim, max_len, shared_blocks);
    if (!workspace || workspace_bytes < p.workspace_bytes) return NVFP4_ERR_INVALID_ARGUMENT;
    if (!aligned(workspace, 16)) return NVFP4_ERR_ALIGNMENT;
    a.shared = shared_blocks;
    a.all_parts = p.prefix.parts + p.own.parts;
    a.partial = (float*)workspace;
    return report_hip(launch_attention_shared(a, p, shared, (hipStream_t)stream));
}

}  // extern "C"
