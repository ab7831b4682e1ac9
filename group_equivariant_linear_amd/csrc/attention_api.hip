// attention_api.hip -- the C ABI of softmax attention and of its paged cache (declared in
// include/eqlinear.h): plans, argument checks and dispatch.  Checks run before any HIP call.
#include <utility>

#include "api_checks.h"

using namespace eql;

namespace {

constexpr int kMaxHeadNumbers = 128;            // D_k, D_v
constexpr int64_t kMaxTokens = (int64_t)1 << 30;  // positions are ints in the kernels

// Buckets of the distances 0 .. reach on one side: half of them one by one, then bucket
// exact + j, j < m = side - exact, from the least n with n^m >= exact^(m-j) reach^j on.
// Compared by logarithms: over all plans, those of powers that differ are 5e-11 and more
// apart, those of equal ones 6e-17 and less.
void fill_buckets(BucketMap& map, int side, int reach) {
    const int exact = side / 2, m = side - exact;
    const long double le = std::log((long double)exact), lr = std::log((long double)reach);
    for (int b = 0; b <= exact; ++b) map.start[b] = (uint16_t)b;
    for (int n = exact, j = 0; n <= reach; ++n) {
        const long double ln = m * std::log((long double)n);
        while (j + 1 < m && ln >= (m - j - 1) * le + (j + 1) * lr - 1e-13L) map.start[exact + ++j] = (uint16_t)n;
    }
    map.start[side] = (uint16_t)(reach + 1);
}

// Bucket of distance n <= reach on one side: the last that starts there or before.
int bucket_of(const BucketMap& map, int side, int n) {
    int b = side - 1;
    while (map.start[b] > n) --b;
    return b;
}

// A cache tensor [blocks][block_size][kv_heads][D]: extents that stay far from the end of
// the address space, rows that do not overlap if it is written.
bool cache_ok(const eqlinear_pages& c, int64_t blocks, int64_t block_size, int kv_heads, int64_t D, size_t es, bool written,
              uint64_t& bytes) {
    if (!c.ptr || !aligned(c.ptr, es) || c.block_stride < 0 || c.token_stride < 0 || c.head_stride < 0) return false;
    const int64_t big = (int64_t)1 << 40;
    if (c.block_stride > big || c.token_stride > big || c.head_stride > big) return false;
    const double reach = (double)blocks * (double)c.block_stride + (double)block_size * (double)c.token_stride +
                         (double)kv_heads * (double)c.head_stride;
    if (reach > 1e15) return false;
    bytes = (uint64_t)((blocks - 1) * c.block_stride + (block_size - 1) * c.token_stride + (kv_heads - 1) * c.head_stride + D) * es;
    if (!written) return true;
    // every axis steps over what the shorter ones cover
    struct Axis {
        int64_t n, stride;
    } x[3] = {{blocks, c.block_stride}, {block_size, c.token_stride}, {kv_heads, c.head_stride}};
    for (int i = 0; i < 3; ++i)
        for (int j = i + 1; j < 3; ++j)
            if (x[j].stride < x[i].stride) std::swap(x[i], x[j]);
    int64_t covered = D;
    for (const Axis& a : x) {
        if (a.n == 1) continue;
        if (a.stride < covered) return false;
        covered = (a.n - 1) * a.stride + covered;
    }
    return true;
}

// Whether two caches of as many blocks may share a number.  Apart are: address ranges that do
// not meet; with equal block (or block and token) strides, blocks (or tokens' rows) that do not
// meet modulo the stride.
bool caches_apart(const eqlinear_pages& a, const eqlinear_pages& b, int64_t block_size, int kv_heads, int64_t Da, int64_t Db,
                  size_t es, uint64_t na, uint64_t nb) {
    if (!overlaps(a.ptr, na, b.ptr, nb)) return true;
    const int64_t d = (int64_t)((uintptr_t)b.ptr - (uintptr_t)a.ptr);
    auto clear = [&](int64_t stride, int64_t run_a, int64_t run_b) {
        const int64_t step = stride * (int64_t)es;
        if (step <= 0) return false;
        const int64_t at = ((d % step) + step) % step;
        return at >= run_a * (int64_t)es && at + run_b * (int64_t)es <= step;
    };
    if (a.block_stride != b.block_stride) return false;
    const int64_t row_a = (kv_heads - 1) * a.head_stride + Da, row_b = (kv_heads - 1) * b.head_stride + Db;
    if (clear(a.block_stride, (block_size - 1) * a.token_stride + row_a, (block_size - 1) * b.token_stride + row_b)) return true;
    // (a block stride of whole token strides keeps the tokens in step)
    return a.token_stride == b.token_stride && a.token_stride > 0 && a.block_stride % a.token_stride == 0 &&
           clear(a.token_stride, row_a, row_b);
}

Pages pages_of(const eqlinear_pages& c) { return Pages{c.ptr, c.block_stride, c.token_stride, c.head_stride}; }

// (the backward divides lse by it, and all kernels multiply it by log2 e: NaN is refused too)
bool scale_ok(float scale) { return std::fabs(scale) >= 0x1p-100f && std::fabs(scale) <= 0x1p100f; }

bool bias_ok(const eqlinear_plan_s* p, const void* bias) { return !bias || (p->buckets > 0 && aligned(bias, elem_size(p))); }

// Packed or equal lengths of q and of k and v.
bool sequences_ok(const int64_t* offsets, const int64_t* kv_offsets, int64_t batch, int64_t T, int64_t T_kv) {
    return batch_ok(offsets, batch, T) && batch_ok(kv_offsets, batch, T_kv);
}

AttentionArgs attention_args(const eqlinear_plan_s* p, const eqlinear_heads* q, const eqlinear_heads* k,
                             const eqlinear_heads* v, const eqlinear_heads* o, float scale, const void* bias, float* lse,
                             const int64_t* offsets, const int64_t* kv_offsets, int64_t batch, int64_t T, int64_t T_kv) {
    AttentionArgs a{};
    a.causal = p->causal;
    a.scale = scale;
    a.batch = batch, a.T = T, a.T_kv = T_kv;
    a.offsets = offsets, a.kv_offsets = kv_offsets;
    a.heads = p->heads, a.kv_heads = p->kv_heads, a.D_k = p->d_k * p->N, a.D_v = p->d_v * p->N;
    // (no tokens: no tensor, and no kernel reads one)
    if (T > 0) a.q = heads_of(*q), a.o = heads_of(*o);
    if (T_kv > 0) a.k = heads_of(*k), a.v = heads_of(*v);
    a.bias = bias;
    a.buckets = p->buckets, a.reach = p->reach;
    a.lse = lse;
    return a;
}

}  // namespace

extern "C" {

eqlinear_status eqlinear_attention_plan(eqlinear_plan_t* out, int N, int heads, int kv_heads, int d_k, int d_v, int causal,
                                        int buckets, int max_distance, eqlinear_dtype dt) {
    if (!out) return EQL_ERR_INVALID;
    *out = nullptr;
    if (N < 1 || N > 16 || heads < 1 || kv_heads < 1 || heads % kv_heads || d_k < 1 || d_v < 1 || !dtype_ok((int)dt))
        return EQL_ERR_INVALID;
    if ((int64_t)heads * d_k > kMaxWidth / N || (int64_t)heads * d_v > kMaxWidth / N) return EQL_ERR_INVALID;
    const int side = causal ? buckets : buckets / 2;
    if (buckets < 0 || (buckets && (side < 2 || (!causal && buckets % 2) || max_distance <= side / 2))) return EQL_ERR_INVALID;
    if (d_k * N > kMaxHeadNumbers || d_v * N > kMaxHeadNumbers) return EQL_ERR_UNSUPPORTED;
    if (buckets > kMaxBuckets || (buckets && max_distance > kMaxReach)) return EQL_ERR_UNSUPPORTED;
    eqlinear_plan_s* p = new (std::nothrow) eqlinear_plan_s{EQL_KIND_ATTENTION, (int)dt, N, heads * d_k, heads * d_v};
    if (!p) return EQL_ERR_NOMEM;
    p->heads = heads, p->kv_heads = kv_heads;
    p->d_k = d_k, p->d_v = d_v;
    p->causal = causal != 0;
    p->buckets = buckets;
    p->reach = buckets ? max_distance : 0;
    if (buckets) fill_buckets(p->map, side, max_distance);
    *out = p;
    return EQL_OK;
}

int eqlinear_attention_bucket(eqlinear_plan_t p, int64_t distance) {
    if (!p || p->kind != EQL_KIND_ATTENTION || !p->buckets) return -1;
    if (distance < 0 && p->causal) return -1;
    const int side = p->causal ? p->buckets : p->buckets / 2;
    if (distance < 0) return bucket_of(p->map, side, distance > -p->reach ? (int)-distance : p->reach) + side;
    return bucket_of(p->map, side, distance < p->reach ? (int)distance : p->reach);
}

size_t eqlinear_attention_workspace(eqlinear_plan_t p, int64_t T, int64_t T_kv, int64_t batch, int backward) {
    if (!p || p->kind != EQL_KIND_ATTENTION || T < 0 || T_kv < 0 || batch < 0 || T > kMaxTokens || T_kv > kMaxTokens ||
        batch > 0x7fffffff)
        return 0;
    return attention_workspace(p->heads, p->buckets, T, batch, backward != 0);
}

eqlinear_status eqlinear_attention(eqlinear_plan_t p, const eqlinear_heads* q, const eqlinear_heads* k,
                                   const eqlinear_heads* v, float scale, const void* bias, const int64_t* offsets,
                                   const int64_t* kv_offsets, int64_t batch, const eqlinear_heads* o, float* lse, int64_t T,
                                   int64_t T_kv, void* workspace, size_t workspace_bytes, void* stream) {
    if (!p || p->kind != EQL_KIND_ATTENTION || !sequences_ok(offsets, kv_offsets, batch, T, T_kv)) return EQL_ERR_INVALID;
    if (!scale_ok(scale) || !bias_ok(p, bias)) return EQL_ERR_INVALID;
    if (T > kMaxTokens || T_kv > kMaxTokens) return EQL_ERR_UNSUPPORTED;
    if (batch == 0 || T == 0) return EQL_OK;
    const size_t es = elem_size(p);
    const int64_t Dk = (int64_t)p->d_k * p->N, Dv = (int64_t)p->d_v * p->N;
    const size_t need = eqlinear_attention_workspace(p, T, T_kv, batch, 0);
    if (!workspace_ok(workspace, workspace_bytes, need)) return EQL_ERR_INVALID;
    if (!q || !o || (T_kv > 0 && (!k || !v)) || (lse && !aligned(lse, 4))) return EQL_ERR_INVALID;
    Span in[3] = {span_of(*q, T, p->heads, Dk, es)};
    if (T_kv > 0) in[1] = span_of(*k, T_kv, p->kv_heads, Dk, es), in[2] = span_of(*v, T_kv, p->kv_heads, Dv, es);
    const int n = T_kv > 0 ? 3 : 1;
    const Span to[1] = {span_of(*o, T, p->heads, Dv, es)};
    if (!tensors_ok(in, n, to, 1)) return EQL_ERR_INVALID;
    const Range stats{lse, (uint64_t)T * p->heads * 4}, table{bias, (uint64_t)p->heads * p->buckets * es},
        ends{offsets, (uint64_t)(batch + 1) * 8}, kv_ends{kv_offsets, (uint64_t)(batch + 1) * 8};
    if (!disjoint({stats, {workspace, need}}, {table, ends, kv_ends})) return EQL_ERR_INVALID;
    if (!apart(stats.p, stats.n, in, n)) return EQL_ERR_INVALID;
    for (const Range& r : {stats, table, ends, kv_ends})
        if (!apart(r.p, r.n, to, 1)) return EQL_ERR_INVALID;
    if (need && (!apart(workspace, need, in, n) || !apart(workspace, need, to, 1))) return EQL_ERR_INVALID;
    const AttentionArgs a = attention_args(p, q, k, v, o, scale, bias, lse, offsets, kv_offsets, batch, T, T_kv);
    return status_of(launch_attention(p->dtype, a, p->map, (hipStream_t)stream));
}

eqlinear_status eqlinear_attention_backward(eqlinear_plan_t p, const eqlinear_heads* q, const eqlinear_heads* k,
                                            const eqlinear_heads* v, const eqlinear_heads* o, const eqlinear_heads* d_o,
                                            const float* lse, float scale, const void* bias, const int64_t* offsets,
                                            const int64_t* kv_offsets, int64_t batch, const eqlinear_heads* dq,
                                            const eqlinear_heads* dk, const eqlinear_heads* dv, float* d_bias, int64_t T,
                                            int64_t T_kv, void* workspace, size_t workspace_bytes, void* stream) {
    if (!p || p->kind != EQL_KIND_ATTENTION || !sequences_ok(offsets, kv_offsets, batch, T, T_kv)) return EQL_ERR_INVALID;
    if (!scale_ok(scale) || !bias_ok(p, bias) || (d_bias && (!bias || !aligned(d_bias, 4)))) return EQL_ERR_INVALID;
    if (T > kMaxTokens || T_kv > kMaxTokens) return EQL_ERR_UNSUPPORTED;
    if ((batch == 0 || (T == 0 && T_kv == 0)) && !d_bias) return EQL_OK;
    const size_t es = elem_size(p);
    const int64_t Dk = (int64_t)p->d_k * p->N, Dv = (int64_t)p->d_v * p->N;
    const size_t need = eqlinear_attention_workspace(p, T, T_kv, batch, 1);
    if (!workspace_ok(workspace, workspace_bytes, need)) return EQL_ERR_INVALID;
    if ((T > 0 && (!q || !o || !d_o || !lse || !aligned(lse, 4) || !dq)) || (T_kv > 0 && (!k || !v || !dk || !dv)))
        return EQL_ERR_INVALID;
    Span in[5], to[3];
    int n = 0, m = 0;
    if (T > 0) {
        in[n++] = span_of(*q, T, p->heads, Dk, es);
        in[n++] = span_of(*o, T, p->heads, Dv, es);
        in[n++] = span_of(*d_o, T, p->heads, Dv, es);
        to[m++] = span_of(*dq, T, p->heads, Dk, es);
    }
    if (T_kv > 0) {
        in[n++] = span_of(*k, T_kv, p->kv_heads, Dk, es);
        in[n++] = span_of(*v, T_kv, p->kv_heads, Dv, es);
        to[m++] = span_of(*dk, T_kv, p->kv_heads, Dk, es);
        to[m++] = span_of(*dv, T_kv, p->kv_heads, Dv, es);
    }
    if (!tensors_ok(in, n, to, m)) return EQL_ERR_INVALID;
    const uint64_t cells = (uint64_t)p->heads * p->buckets;
    const Range stats{T > 0 ? lse : nullptr, (uint64_t)T * p->heads * 4}, table{bias, cells * es}, grad{d_bias, cells * 4},
        ends{offsets, (uint64_t)(batch + 1) * 8}, kv_ends{kv_offsets, (uint64_t)(batch + 1) * 8};
    if (!disjoint({grad, {workspace, need}}, {stats, table, ends, kv_ends})) return EQL_ERR_INVALID;
    for (const Range& r : {stats, table, grad, ends, kv_ends})
        if (!apart(r.p, r.n, to, m)) return EQL_ERR_INVALID;
    if (!apart(grad.p, grad.n, in, n)) return EQL_ERR_INVALID;
    if (need && (!apart(workspace, need, in, n) || !apart(workspace, need, to, m))) return EQL_ERR_INVALID;
    AttentionArgs a = attention_args(p, q, k, v, o, scale, bias, const_cast<float*>(lse), offsets, kv_offsets, batch, T, T_kv);
    if (T > 0) a.d_o = heads_of(*d_o), a.dq = heads_of(*dq);
    if (T_kv > 0) a.dk = heads_of(*dk), a.dv = heads_of(*dv);
    a.dbias = d_bias;
    return status_of(launch_attention_backward(p->dtype, a, p->map, workspace, (hipStream_t)stream));
}

size_t eqlinear_attention_step_workspace(eqlinear_plan_t p, int64_t batch) {
    if (!p || p->kind != EQL_KIND_ATTENTION || batch < 0 || batch > 0x7fffffff) return 0;
    return attention_step_workspace(p->dtype, p->heads, p->kv_heads, p->d_k * p->N, p->d_v * p->N, batch);
}

eqlinear_status eqlinear_attention_step(eqlinear_plan_t p, const eqlinear_heads* q, const eqlinear_pages* k_cache,
                                        const eqlinear_pages* v_cache, int64_t blocks, int block_size, const int32_t* table,
                                        int64_t max_blocks, const int32_t* lengths, float scale, const void* bias,
                                        const eqlinear_heads* o, float* lse, int64_t batch, void* workspace,
                                        size_t workspace_bytes, void* stream) {
    if (!p || p->kind != EQL_KIND_ATTENTION || batch < 0 || batch > 0x7fffffff) return EQL_ERR_INVALID;
    if (!scale_ok(scale) || !bias_ok(p, bias) || blocks < 0 || block_size < 1 || max_blocks < 0) return EQL_ERR_INVALID;
    if (blocks > 0x7fffffff || max_blocks > kMaxTokens || max_blocks * block_size > kMaxTokens) return EQL_ERR_UNSUPPORTED;
    if (batch == 0) return EQL_OK;
    const size_t es = elem_size(p);
    const int64_t Dk = (int64_t)p->d_k * p->N, Dv = (int64_t)p->d_v * p->N;
    if (!q || !o || !lengths || !aligned(lengths, 4) || (max_blocks > 0 && (!table || !aligned(table, 4))) ||
        (lse && !aligned(lse, 4)))
        return EQL_ERR_INVALID;
    const bool cached = blocks > 0 && max_blocks > 0;
    uint64_t kb = 0, vb = 0;
    if (cached && (!k_cache || !v_cache || !cache_ok(*k_cache, blocks, block_size, p->kv_heads, Dk, es, false, kb) ||
                   !cache_ok(*v_cache, blocks, block_size, p->kv_heads, Dv, es, false, vb)))
        return EQL_ERR_INVALID;
    const size_t need = eqlinear_attention_step_workspace(p, batch);
    if (!workspace_ok(workspace, workspace_bytes, need)) return EQL_ERR_INVALID;
    const Span in[1] = {span_of(*q, batch, p->heads, Dk, es)}, to[1] = {span_of(*o, batch, p->heads, Dv, es)};
    if (!tensors_ok(in, 1, to, 1)) return EQL_ERR_INVALID;
    const Range stats{lse, (uint64_t)batch * p->heads * 4}, cells{bias, (uint64_t)p->heads * p->buckets * es},
        counts{lengths, (uint64_t)batch * 4}, rows{table, (uint64_t)batch * max_blocks * 4},
        keys{cached ? k_cache->ptr : nullptr, kb}, values{cached ? v_cache->ptr : nullptr, vb};
    if (!disjoint({stats, {workspace, need}}, {cells, counts, rows, keys, values})) return EQL_ERR_INVALID;
    for (const Range& r : {stats, cells, counts, rows, keys, values})
        if (r.n && !apart(r.p, r.n, to, 1)) return EQL_ERR_INVALID;
    if (!apart(stats.p, stats.n, in, 1)) return EQL_ERR_INVALID;
    if (need && (!apart(workspace, need, in, 1) || !apart(workspace, need, to, 1))) return EQL_ERR_INVALID;
    StepArgs a{};
    a.q = heads_of(*q), a.o = heads_of(*o);
    if (cached) a.k = pages_of(*k_cache), a.v = pages_of(*v_cache);
    a.table = table, a.lengths = lengths;
    a.batch = batch, a.blocks = blocks;
    a.max_blocks = cached ? (int)max_blocks : 0, a.block_size = block_size;
    a.heads = p->heads, a.kv_heads = p->kv_heads, a.D_k = (int)Dk, a.D_v = (int)Dv;
    a.scale = scale;
    a.bias = bias;
    a.buckets = p->buckets, a.reach = p->reach;
    a.side = p->causal ? p->buckets : p->buckets / 2;
    a.lse = lse;
    return status_of(launch_attention_step(p->dtype, a, p->map, workspace, (hipStream_t)stream));
}

size_t eqlinear_cache_tables_workspace(int64_t batch) {
    return batch < 0 || batch > 0x7fffffff ? 0 : cache_tables_workspace(batch);
}

eqlinear_status eqlinear_cache_tables(const int32_t* lengths, const int32_t* added, const int32_t* free_blocks, int64_t n_free,
                                      const int32_t* cursor, int32_t* table, int64_t max_blocks, int block_size,
                                      int32_t* lengths_out, int32_t* cursor_out, int64_t* slots, int32_t* positions,
                                      int64_t* offsets, int64_t batch, int64_t T, void* workspace, size_t workspace_bytes,
                                      void* stream) {
    if (batch < 1 || batch > 0x7fffffff || T < 0 || n_free < 0 || max_blocks < 0 || block_size < 1) return EQL_ERR_INVALID;
    if (max_blocks > kMaxTokens || max_blocks * block_size > kMaxTokens || T > kMaxTokens || n_free > kMaxTokens)
        return EQL_ERR_UNSUPPORTED;
    if (!lengths || !added || !cursor || !lengths_out || !cursor_out || !offsets || (n_free > 0 && !free_blocks) ||
        (max_blocks > 0 && !table) || (T > 0 && (!slots || !positions)))
        return EQL_ERR_INVALID;
    for (const void* x : {(const void*)lengths, (const void*)added, (const void*)free_blocks, (const void*)cursor,
                          (const void*)table, (const void*)lengths_out, (const void*)cursor_out, (const void*)positions})
        if (!aligned(x, 4)) return EQL_ERR_INVALID;
    if (!aligned(slots, 8) || !aligned(offsets, 8)) return EQL_ERR_INVALID;
    const size_t need = eqlinear_cache_tables_workspace(batch);
    if (!workspace_ok(workspace, workspace_bytes, need)) return EQL_ERR_INVALID;
    const uint64_t nb = (uint64_t)batch * 4, nt = (uint64_t)T;
    const Range n{lengths, nb}, c{cursor, 4};
    if (!disjoint({{table, nb * max_blocks},
                   {lengths_out, nb},
                   {cursor_out, 4},
                   {slots, nt * 8},
                   {positions, nt * 4},
                   {offsets, (uint64_t)(batch + 1) * 8},
                   {workspace, need}},
                  {{added, nb},
                   {free_blocks, (uint64_t)n_free * 4},
                   lengths == lengths_out ? Range{nullptr, 0} : n,
                   cursor == cursor_out ? Range{nullptr, 0} : c}))
        return EQL_ERR_INVALID;
    TablesArgs a{};
    a.lengths = lengths, a.added = added, a.free_blocks = free_blocks, a.cursor = cursor;
    a.table = table;
    a.lengths_out = lengths_out, a.cursor_out = cursor_out;
    a.slots = slots, a.positions = positions, a.offsets = offsets;
    a.batch = batch, a.n_free = n_free, a.T = T;
    a.max_blocks = (int)max_blocks, a.block_size = block_size;
    return status_of(launch_cache_tables(a, workspace, (hipStream_t)stream));
}

eqlinear_status eqlinear_cache_store(eqlinear_plan_t p, const eqlinear_heads* k, const eqlinear_heads* v, const int64_t* slots,
                                     const eqlinear_pages* k_cache, const eqlinear_pages* v_cache, int64_t blocks,
                                     int block_size, int64_t T, void* stream) {
    if (!p || p->kind != EQL_KIND_ATTENTION || T < 0 || blocks < 0 || block_size < 1) return EQL_ERR_INVALID;
    if (T > kMaxTokens || blocks > 0x7fffffff || block_size > kMaxTokens) return EQL_ERR_UNSUPPORTED;
    if (T == 0 || blocks == 0) return EQL_OK;
    const size_t es = elem_size(p);
    const int64_t Dk = (int64_t)p->d_k * p->N, Dv = (int64_t)p->d_v * p->N;
    uint64_t kb = 0, vb = 0;
    if (!k || !v || !slots || !aligned(slots, 8) || !k_cache || !v_cache ||
        !cache_ok(*k_cache, blocks, block_size, p->kv_heads, Dk, es, true, kb) ||
        !cache_ok(*v_cache, blocks, block_size, p->kv_heads, Dv, es, true, vb))
        return EQL_ERR_INVALID;
    const Span in[2] = {span_of(*k, T, p->kv_heads, Dk, es), span_of(*v, T, p->kv_heads, Dv, es)};
    if (!tensors_ok(in, 2, nullptr, 0)) return EQL_ERR_INVALID;
    const Range keys{k_cache->ptr, kb}, values{v_cache->ptr, vb};
    const Range targets{slots, (uint64_t)T * 8};
    if (!disjoint({keys}, {targets}) || !disjoint({values}, {targets}) || !apart(keys.p, kb, in, 2) || !apart(values.p, vb, in, 2) ||
        !caches_apart(*k_cache, *v_cache, block_size, p->kv_heads, Dk, Dv, es, kb, vb))
        return EQL_ERR_INVALID;
    StoreArgs a{};
    a.k = heads_of(*k), a.v = heads_of(*v);
    a.k_cache = pages_of(*k_cache), a.v_cache = pages_of(*v_cache);
    a.slots = slots;
    a.T = T, a.blocks = blocks;
    a.block_size = block_size, a.kv_heads = p->kv_heads, a.D_k = (int)Dk, a.D_v = (int)Dv;
    return status_of(launch_cache_store(p->dtype, a, (hipStream_t)stream));
}

}  // extern "C"
