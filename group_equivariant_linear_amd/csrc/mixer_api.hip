// mixer_api.hip -- the C ABI of the operators between the layers (rotary
// positions, linear attention, group norm; declared in include/eqlinear.h): plans,
// argument checks and dispatch.  Checks run before any HIP call.
#include <cmath>
#include <initializer_list>
#include <new>

#include "eq_plan.h"

using eql::elem_size;
using eql::Heads;
using eql::hip_status;
using eql::kMaxWidth;
using eql::overlaps;

namespace {

constexpr double kTwoPi = 6.283185307179586476925286766559;
constexpr int kMaxHeadNumbers = 128;  // D_k, D_v of linear attention

// A tensor of T rows, each of n_heads runs of `run` elements.
struct Span {
    const void* p;
    int64_t T, ts;
    int n_heads;
    int64_t hs, run;
    size_t es;
    uint64_t bytes() const { return (uint64_t)((T - 1) * ts + (n_heads - 1) * hs + run) * es; }
    // elements of one token's runs when they lie one after the other, else -1
    int64_t row() const { return n_heads == 1 ? run : (hs >= run ? (n_heads - 1) * hs + run : -1); }
};

Span span_of(const eqlinear_heads& h, int64_t T, int n_heads, int64_t run, size_t es) {
    return Span{h.ptr, T, h.token_stride, n_heads, h.head_stride, run, es};
}

bool readable(const Span& s) {
    if (!s.p || (uintptr_t)s.p % s.es != 0 || s.ts < 0 || s.hs < 0) return false;
    // offsets stay far from the end of the address space
    return s.ts <= ((int64_t)1 << 40) && s.hs <= ((int64_t)1 << 40) && s.T <= ((int64_t)1 << 40) &&
           (double)s.T * (double)s.ts + (double)s.n_heads * (double)s.hs < 1e15;
}

// an output: no element twice
bool writable(const Span& s) {
    if (!readable(s)) return false;
    const int64_t row = s.row();
    if (row >= 0 && (s.T == 1 || s.ts >= row)) return true;                       // token after token
    return s.ts >= s.run && (s.n_heads == 1 || s.hs >= (s.T - 1) * s.ts + s.run);  // head after head
}

// Whether two tensors may share an element.  Apart are: address ranges that do not meet; with
// equal token strides, rows (all of a token's runs) that do not meet modulo the stride; and with
// equal head strides besides, runs that do not meet modulo the head stride (heads of q, k and v
// in turn).
bool collide(const Span& a, const Span& b) {
    if (!overlaps(a.p, a.bytes(), b.p, b.bytes())) return false;
    if (a.es != b.es) return true;
    const int64_t es = (int64_t)a.es, d = (int64_t)((uintptr_t)b.p - (uintptr_t)a.p);
    auto rest = [](int64_t x, int64_t m) { return ((x % m) + m) % m; };
    auto clear = [&](int64_t at, int64_t run_a, int64_t run_b, int64_t m) { return at >= run_a * es && at + run_b * es <= m; };
    const int64_t head = (a.n_heads > 1 ? a.hs : b.hs) * es;
    const bool one_head = a.n_heads == 1 && b.n_heads == 1;
    const bool heads_alike = !one_head && head > 0 && (a.n_heads == 1 || b.n_heads == 1 || a.hs == b.hs);
    if (a.T == 1 && b.T == 1) return !heads_alike || !clear(rest(d, head), a.run, b.run, head);
    const int64_t ra = a.row(), rb = b.row();
    if (a.ts != b.ts || ra < 0 || rb < 0 || ra > a.ts || rb > b.ts) return true;
    const int64_t step = a.ts * es, at = rest(d, step);  // byte offset of b's runs in a's rows
    // b's row may meet the row of a that it starts in, and the next one
    const bool this_row = at < ra * es, next_row = at + rb * es > step;
    auto meet = [&](int64_t from) { return !heads_alike || !clear(rest(from, head), a.run, b.run, head); };
    return (this_row && meet(at)) || (next_row && meet(at - step));
}

bool same_place(const Span& a, const Span& b) {
    return a.p == b.p && (a.T == 1 || a.ts == b.ts) && (a.n_heads == 1 || a.hs == b.hs);
}

Heads heads_of(const eqlinear_heads& h) { return Heads{h.ptr, h.token_stride, h.head_stride}; }

bool batch_ok(const int64_t* offsets, int64_t batch, int64_t T) {
    if (T < 0 || batch < 0 || batch > 0x7fffffff || T > ((int64_t)1 << 40)) return false;
    if (offsets) return batch > 0 && ((uintptr_t)offsets & 7u) == 0;
    return batch > 0 ? T % batch == 0 : T == 0;
}

bool workspace_ok(const void* ws, size_t bytes, size_t need) {
    return need == 0 || (ws && ((uintptr_t)ws & 255u) == 0 && bytes >= need);
}

// Flat buffers of a call (null or empty: not given): what it writes shares no byte with
// anything else of it.
struct Range {
    const void* p;
    uint64_t n;
};
bool disjoint(std::initializer_list<Range> written, std::initializer_list<Range> read) {
    auto meet = [](const Range& a, const Range& b) { return a.p && b.p && a.n && b.n && overlaps(a.p, a.n, b.p, b.n); };
    for (auto w = written.begin(); w != written.end(); ++w) {
        for (auto v = written.begin(); v != w; ++v)
            if (meet(*v, *w)) return false;
        for (const Range& r : read)
            if (meet(*w, r)) return false;
    }
    return true;
}

bool aligned(const void* p, size_t a) { return (uintptr_t)p % a == 0; }

eqlinear_status status_of(hipError_t e) { return e == hipErrorNotSupported ? EQL_ERR_UNSUPPORTED : hip_status(e); }

}  // namespace

extern "C" {

eqlinear_status eqlinear_rotary_plan(eqlinear_plan_t* out, int N, int heads, int kv_heads, int d, int rot,
                                     eqlinear_rotary_layout layout, double base, eqlinear_rotary_scaling scaling,
                                     double factor, double context, double turns_slow, double turns_fast,
                                     double magnitude, eqlinear_dtype dt) {
    if (!out) return EQL_ERR_INVALID;
    *out = nullptr;
    if (N < 1 || N > 16 || heads < 1 || kv_heads < 1 || d < 2 || rot < 2 || rot > d || rot % 2 ||
        !eql::dtype_ok((int)dt))
        return EQL_ERR_INVALID;
    if ((int64_t)heads * d > kMaxWidth / N || (int64_t)kv_heads * d > kMaxWidth / N) return EQL_ERR_INVALID;
    if ((int)layout != EQL_ROTARY_HALF && (int)layout != EQL_ROTARY_INTERLEAVED) return EQL_ERR_INVALID;
    if ((int)scaling < EQL_ROTARY_PLAIN || (int)scaling > EQL_ROTARY_BANDED) return EQL_ERR_INVALID;
    if (!(base > 0) || !std::isfinite(base) || !(magnitude > 0) || !std::isfinite(magnitude)) return EQL_ERR_INVALID;
    if (scaling != EQL_ROTARY_PLAIN && (!(factor > 0) || !std::isfinite(factor))) return EQL_ERR_INVALID;
    if (scaling == EQL_ROTARY_BANDED &&
        (!(context > 0) || !std::isfinite(context) || !(turns_slow >= 0) || !(turns_fast > turns_slow) ||
         !std::isfinite(turns_fast)))
        return EQL_ERR_INVALID;
    if (rot / 2 > eql::kMaxRotaryPairs) return EQL_ERR_UNSUPPORTED;
    eqlinear_plan_s* p = new (std::nothrow) eqlinear_plan_s{EQL_KIND_ROTARY, (int)dt, N, heads * d, heads * d};
    if (!p) return EQL_ERR_NOMEM;
    p->heads = heads;
    p->kv_heads = kv_heads;
    p->d_k = p->d_v = d;
    p->rot = rot;
    p->layout = (int)layout;
    const double b = scaling == EQL_ROTARY_RAISED_BASE && rot > 2 ? base * std::pow(factor, rot / (rot - 2.0)) : base;
    for (int j = 0; j < rot / 2; ++j) {
        double f = std::pow(b, -2.0 * j / rot);
        if (scaling == EQL_ROTARY_LINEAR) f /= factor;
        if (scaling == EQL_ROTARY_BANDED) {
            double w = (context * f / kTwoPi - turns_slow) / (turns_fast - turns_slow);
            w = w < 0 ? 0 : (w > 1 ? 1 : w);
            f = f * w + f / factor * (1 - w);
        }
        p->freq.turns[j] = f / kTwoPi;
    }
    p->freq.magnitude = (float)magnitude;
    *out = p;
    return EQL_OK;
}

eqlinear_status eqlinear_rotary(eqlinear_plan_t p, const eqlinear_heads* q, const eqlinear_heads* k,
                                const int32_t* positions, int inverse, const eqlinear_heads* q_out,
                                const eqlinear_heads* k_out, int64_t T, void* stream) {
    if (!p || p->kind != EQL_KIND_ROTARY || T < 0) return EQL_ERR_INVALID;
    if (T == 0) return EQL_OK;
    if (!q || !q_out || !k != !k_out || !positions || !aligned(positions, 4)) return EQL_ERR_INVALID;
    const size_t es = elem_size(p);
    const int64_t D = (int64_t)p->d_k * p->N;
    Span in[2], to[2];
    const int n = k ? 2 : 1;
    in[0] = span_of(*q, T, p->heads, D, es), to[0] = span_of(*q_out, T, p->heads, D, es);
    if (k) in[1] = span_of(*k, T, p->kv_heads, D, es), to[1] = span_of(*k_out, T, p->kv_heads, D, es);
    const Span pos{positions, 1, 0, 1, 0, T, 4};
    for (int i = 0; i < n; ++i) {
        if (!readable(in[i]) || !writable(to[i])) return EQL_ERR_INVALID;
        if (overlaps(to[i].p, to[i].bytes(), pos.p, pos.bytes())) return EQL_ERR_INVALID;
    }
    for (int i = 0; i < n; ++i) {
        if (n == 2 && collide(to[i], in[1 - i])) return EQL_ERR_INVALID;
        if (!same_place(in[i], to[i]) && collide(to[i], in[i])) return EQL_ERR_INVALID;
    }
    if (n == 2 && collide(to[0], to[1])) return EQL_ERR_INVALID;
    eql::RotaryArgs a{};
    a.q = heads_of(*q), a.q_out = heads_of(*q_out);
    if (k) a.k = heads_of(*k), a.k_out = heads_of(*k_out);
    a.positions = positions;
    a.T = T;
    a.q_heads = p->heads, a.k_heads = k ? p->kv_heads : 0;
    a.N = p->N, a.d = p->d_k, a.rot = p->rot, a.layout = p->layout, a.inverse = inverse != 0;
    return status_of(eql::launch_rotary(p->dtype, a, p->freq, (hipStream_t)stream));
}

eqlinear_status eqlinear_mixer_plan(eqlinear_plan_t* out, int N, int heads, int kv_heads, int d_k, int d_v,
                                    eqlinear_dtype dt) {
    if (!out) return EQL_ERR_INVALID;
    *out = nullptr;
    if (N < 1 || N > 16 || heads < 1 || kv_heads < 1 || heads % kv_heads || d_k < 1 || d_v < 1 ||
        !eql::dtype_ok((int)dt))
        return EQL_ERR_INVALID;
    if ((int64_t)heads * d_k > kMaxWidth / N || (int64_t)heads * d_v > kMaxWidth / N) return EQL_ERR_INVALID;
    if (d_k * N > kMaxHeadNumbers || d_v * N > kMaxHeadNumbers) return EQL_ERR_UNSUPPORTED;
    eqlinear_plan_s* p = new (std::nothrow) eqlinear_plan_s{EQL_KIND_MIXER, (int)dt, N, heads * d_k, heads * d_v};
    if (!p) return EQL_ERR_NOMEM;
    p->heads = heads;
    p->kv_heads = kv_heads;
    p->d_k = d_k;
    p->d_v = d_v;
    *out = p;
    return EQL_OK;
}

size_t eqlinear_linear_attention_workspace(eqlinear_plan_t p, int64_t T, int64_t batch, int backward) {
    if (!p || p->kind != EQL_KIND_MIXER || T < 0 || batch < 0 || T > ((int64_t)1 << 40) || batch > 0x7fffffff) return 0;
    return eql::linear_attention_workspace(p->dtype, p->heads, p->kv_heads, p->d_k * p->N, p->d_v * p->N, T, batch,
                                           backward != 0);
}

}  // extern "C"

namespace {

// What the forward, the backward and the step check alike; `n` tensors in, the
// first `n_out` of `to` out.
bool tensors_ok(const Span* in, int n, const Span* to, int n_out) {
    for (int i = 0; i < n; ++i)
        if (!readable(in[i])) return false;
    for (int i = 0; i < n_out; ++i) {
        if (!writable(to[i])) return false;
        for (int j = 0; j < n; ++j)
            if (collide(to[i], in[j])) return false;
        for (int j = 0; j < i; ++j)
            if (collide(to[i], to[j])) return false;
    }
    return true;
}

bool state_ok(const float* in, const float* out, uint64_t bytes) {
    if ((in && !aligned(in, 16)) || (out && !aligned(out, 16))) return false;
    return !in || !out || !overlaps(in, bytes, out, bytes);
}

bool apart(const void* a, uint64_t bytes, const Span* s, int n) {
    for (int i = 0; a && i < n; ++i)
        if (overlaps(a, bytes, s[i].p, s[i].bytes())) return false;
    return true;
}

eql::MixArgs mix_args(const eqlinear_plan_s* p, const eqlinear_heads* q, const eqlinear_heads* k,
                      const eqlinear_heads* v, const float* log_decay, float scale, const int64_t* offsets,
                      int64_t batch, int64_t T) {
    eql::MixArgs a{};
    if (T > 0) a.q = heads_of(*q), a.k = heads_of(*k), a.v = heads_of(*v);
    a.log_decay = log_decay;
    a.scale = scale;
    a.offsets = offsets;
    a.batch = batch;
    a.T = T;
    a.heads = p->heads, a.kv_heads = p->kv_heads, a.D_k = p->d_k * p->N, a.D_v = p->d_v * p->N;
    return a;
}

}  // namespace

extern "C" {

eqlinear_status eqlinear_linear_attention(eqlinear_plan_t p, const eqlinear_heads* q, const eqlinear_heads* k,
                                          const eqlinear_heads* v, const float* log_decay, float scale,
                                          const int64_t* offsets, int64_t batch, const float* state_in,
                                          float* state_out, const eqlinear_heads* o, int64_t T, void* workspace,
                                          size_t workspace_bytes, void* stream) {
    if (!p || p->kind != EQL_KIND_MIXER || !batch_ok(offsets, batch, T)) return EQL_ERR_INVALID;
    if (!std::isfinite(scale) || scale == 0.0f) return EQL_ERR_INVALID;
    if (batch == 0 || (T == 0 && !state_out)) return EQL_OK;
    const size_t es = elem_size(p);
    const int64_t Dk = (int64_t)p->d_k * p->N, Dv = (int64_t)p->d_v * p->N;
    const uint64_t sb = (uint64_t)batch * p->kv_heads * Dk * Dv * 4;
    if (!log_decay || !aligned(log_decay, 4) || !state_ok(state_in, state_out, sb)) return EQL_ERR_INVALID;
    const size_t need = eqlinear_linear_attention_workspace(p, T, batch, 0);
    if (!workspace_ok(workspace, workspace_bytes, need)) return EQL_ERR_INVALID;
    const Range decays{log_decay, (uint64_t)p->kv_heads * 4}, ends{offsets, (uint64_t)(batch + 1) * 8};
    if (!disjoint({{state_out, sb}, {workspace, need}}, {decays, ends, {state_in, sb}})) return EQL_ERR_INVALID;
    eql::MixArgs a = mix_args(p, nullptr, nullptr, nullptr, log_decay, scale, offsets, batch, 0);
    if (T > 0) {
        if (!q || !k || !v || !o) return EQL_ERR_INVALID;
        const Span in[3] = {span_of(*q, T, p->heads, Dk, es), span_of(*k, T, p->kv_heads, Dk, es),
                            span_of(*v, T, p->kv_heads, Dv, es)};
        const Span to[1] = {span_of(*o, T, p->heads, Dv, es)};
        if (!tensors_ok(in, 3, to, 1)) return EQL_ERR_INVALID;
        if (!apart(state_out, sb, in, 3) || !apart(state_out, sb, to, 1) || !apart(state_in, sb, to, 1) ||
            !apart(decays.p, decays.n, to, 1) || !apart(ends.p, ends.n, to, 1))
            return EQL_ERR_INVALID;
        if (need && (!apart(workspace, need, in, 3) || !apart(workspace, need, to, 1))) return EQL_ERR_INVALID;
        a = mix_args(p, q, k, v, log_decay, scale, offsets, batch, T);
        a.o = heads_of(*o);
    }
    a.state_in = state_in;
    a.state_out = state_out;
    return status_of(eql::launch_linear_attention(p->dtype, a, workspace, (hipStream_t)stream));
}

eqlinear_status eqlinear_linear_attention_backward(eqlinear_plan_t p, const eqlinear_heads* q,
                                                   const eqlinear_heads* k, const eqlinear_heads* v,
                                                   const eqlinear_heads* d_o, const float* log_decay, float scale,
                                                   const int64_t* offsets, int64_t batch, const float* state_in,
                                                   const float* d_state_out, const eqlinear_heads* dq,
                                                   const eqlinear_heads* dk, const eqlinear_heads* dv,
                                                   float* d_state_in, int64_t T, void* workspace,
                                                   size_t workspace_bytes, void* stream) {
    if (!p || p->kind != EQL_KIND_MIXER || !batch_ok(offsets, batch, T)) return EQL_ERR_INVALID;
    if (!std::isfinite(scale) || scale == 0.0f) return EQL_ERR_INVALID;
    if (batch == 0 || (T == 0 && !d_state_in)) return EQL_OK;
    const size_t es = elem_size(p);
    const int64_t Dk = (int64_t)p->d_k * p->N, Dv = (int64_t)p->d_v * p->N;
    const uint64_t sb = (uint64_t)batch * p->kv_heads * Dk * Dv * 4;
    if (!log_decay || !aligned(log_decay, 4) || (state_in && !aligned(state_in, 16)) ||
        !state_ok(d_state_out, d_state_in, sb) || (state_in && d_state_in && overlaps(state_in, sb, d_state_in, sb)))
        return EQL_ERR_INVALID;
    const size_t need = eqlinear_linear_attention_workspace(p, T, batch, 1);
    if (!workspace_ok(workspace, workspace_bytes, need)) return EQL_ERR_INVALID;
    const Range decays{log_decay, (uint64_t)p->kv_heads * 4}, ends{offsets, (uint64_t)(batch + 1) * 8};
    if (!disjoint({{d_state_in, sb}, {workspace, need}}, {decays, ends, {state_in, sb}, {d_state_out, sb}}))
        return EQL_ERR_INVALID;
    eql::MixArgs a = mix_args(p, nullptr, nullptr, nullptr, log_decay, scale, offsets, batch, 0);
    if (T > 0) {
        if (!q || !k || !v || !d_o || !dq || !dk || !dv) return EQL_ERR_INVALID;
        const Span in[4] = {span_of(*q, T, p->heads, Dk, es), span_of(*k, T, p->kv_heads, Dk, es),
                            span_of(*v, T, p->kv_heads, Dv, es), span_of(*d_o, T, p->heads, Dv, es)};
        const Span to[3] = {span_of(*dq, T, p->heads, Dk, es), span_of(*dk, T, p->kv_heads, Dk, es),
                            span_of(*dv, T, p->kv_heads, Dv, es)};
        if (!tensors_ok(in, 4, to, 3)) return EQL_ERR_INVALID;
        if (!apart(d_state_in, sb, in, 4) || !apart(d_state_in, sb, to, 3) || !apart(state_in, sb, to, 3) ||
            !apart(d_state_out, sb, to, 3) || !apart(decays.p, decays.n, to, 3) || !apart(ends.p, ends.n, to, 3))
            return EQL_ERR_INVALID;
        if (need && (!apart(workspace, need, in, 4) || !apart(workspace, need, to, 3))) return EQL_ERR_INVALID;
        a = mix_args(p, q, k, v, log_decay, scale, offsets, batch, T);
        a.d_o = heads_of(*d_o);
        a.dq = heads_of(*dq), a.dk = heads_of(*dk), a.dv = heads_of(*dv);
    }
    a.state_in = state_in;
    a.d_state_out = d_state_out;
    a.d_state_in = d_state_in;
    return status_of(eql::launch_linear_attention_backward(p->dtype, a, workspace, (hipStream_t)stream));
}

eqlinear_status eqlinear_linear_attention_step(eqlinear_plan_t p, const eqlinear_heads* q, const eqlinear_heads* k,
                                               const eqlinear_heads* v, const float* log_decay, float scale,
                                               float* state, const eqlinear_heads* o, int64_t batch, void* stream) {
    if (!p || p->kind != EQL_KIND_MIXER || batch < 0 || batch > 0x7fffffff) return EQL_ERR_INVALID;
    if (!std::isfinite(scale) || scale == 0.0f) return EQL_ERR_INVALID;
    if (batch == 0) return EQL_OK;
    if (!q || !k || !v || !o || !state || !aligned(state, 16) || !log_decay || !aligned(log_decay, 4))
        return EQL_ERR_INVALID;
    const size_t es = elem_size(p);
    const int64_t Dk = (int64_t)p->d_k * p->N, Dv = (int64_t)p->d_v * p->N;
    const uint64_t sb = (uint64_t)batch * p->kv_heads * Dk * Dv * 4;
    const Span in[3] = {span_of(*q, batch, p->heads, Dk, es), span_of(*k, batch, p->kv_heads, Dk, es),
                        span_of(*v, batch, p->kv_heads, Dv, es)};
    const Span to[1] = {span_of(*o, batch, p->heads, Dv, es)};
    if (!tensors_ok(in, 3, to, 1) || !apart(state, sb, in, 3) || !apart(state, sb, to, 1)) return EQL_ERR_INVALID;
    const uint64_t db = (uint64_t)p->kv_heads * 4;
    if (!disjoint({{state, sb}}, {{log_decay, db}}) || !apart(log_decay, db, to, 1)) return EQL_ERR_INVALID;
    eql::MixArgs a = mix_args(p, q, k, v, log_decay, scale, nullptr, batch, batch);
    a.o = heads_of(*o);
    a.state_in = a.state_out = state;
    return status_of(eql::launch_linear_attention_step(p->dtype, a, (hipStream_t)stream));
}

eqlinear_status eqlinear_norm_plan(eqlinear_plan_t* out, int N, int C, int groups, eqlinear_act act, double eps,
                                   eqlinear_dtype dt) {
    if (!out) return EQL_ERR_INVALID;
    *out = nullptr;
    if (N < 1 || N > 16 || C < 1 || groups < 1 || C % groups || !eql::dtype_ok((int)dt)) return EQL_ERR_INVALID;
    if ((int64_t)C > kMaxWidth / N || (int)act < EQL_ACT_NONE || (int)act > EQL_ACT_SILU) return EQL_ERR_INVALID;
    if (!(eps >= 0) || !std::isfinite(eps)) return EQL_ERR_INVALID;
    eqlinear_plan_s* p = new (std::nothrow) eqlinear_plan_s{EQL_KIND_NORM, (int)dt, N, C, C};
    if (!p) return EQL_ERR_NOMEM;
    p->groups = groups;
    p->act = (int)act;
    p->eps = (float)eps;
    *out = p;
    return EQL_OK;
}

size_t eqlinear_group_norm_workspace(eqlinear_plan_t p, int64_t T, int64_t batch, int backward) {
    if (!p || p->kind != EQL_KIND_NORM || T < 0 || batch < 0 || T > ((int64_t)1 << 40) || batch > 0x7fffffff) return 0;
    return eql::group_norm_workspace(p->dtype, p->C_in, p->N, p->groups, T, batch, backward != 0);
}

}  // extern "C"

namespace {

eql::NormArgs norm_args(const eqlinear_plan_s* p, const void* x, int64_t ldx, const void* gamma, const void* beta,
                        const int64_t* offsets, int64_t batch, int64_t T) {
    eql::NormArgs a{};
    a.x = x;
    a.ldx = ldx;
    a.gamma = gamma;
    a.beta = beta;
    a.offsets = offsets;
    a.batch = batch;
    a.T = T;
    a.C = p->C_in, a.N = p->N, a.groups = p->groups, a.act = p->act;
    a.eps = p->eps;
    return a;
}

}  // namespace

extern "C" {

eqlinear_status eqlinear_group_norm(eqlinear_plan_t p, const void* x, int64_t x_stride, const void* gamma,
                                    const void* beta, const int64_t* offsets, int64_t batch, void* y,
                                    int64_t y_stride, float* stats, int64_t T, void* workspace,
                                    size_t workspace_bytes, void* stream) {
    if (!p || p->kind != EQL_KIND_NORM || !batch_ok(offsets, batch, T)) return EQL_ERR_INVALID;
    if (batch == 0 || (T == 0 && !stats)) return EQL_OK;
    const size_t es = elem_size(p);
    const int64_t W = (int64_t)p->C_in * p->N;
    if (stats && !aligned(stats, 8)) return EQL_ERR_INVALID;
    const size_t need = eqlinear_group_norm_workspace(p, T, batch, 0);
    if (!workspace_ok(workspace, workspace_bytes, need)) return EQL_ERR_INVALID;
    const uint64_t sb = (uint64_t)batch * p->groups * 8, cb = (uint64_t)p->C_in * es;
    const Range ends{offsets, (uint64_t)(batch + 1) * 8};
    if (!disjoint({{stats, sb}, {workspace, need}}, {{gamma, cb}, {beta, cb}, ends})) return EQL_ERR_INVALID;
    eql::NormArgs a = norm_args(p, x, x_stride, gamma, beta, offsets, batch, T);
    if (T > 0) {
        const Span in{x, T, x_stride, 1, 0, W, es}, to{y, T, y_stride, 1, 0, W, es};
        if (!readable(in) || !writable(to) || (!same_place(in, to) && collide(to, in))) return EQL_ERR_INVALID;
        for (const void* v : {gamma, beta})
            if (v && (!aligned(v, es) || !apart(v, cb, &to, 1))) return EQL_ERR_INVALID;
        if (!apart(stats, sb, &in, 1) || !apart(stats, sb, &to, 1) || !apart(ends.p, ends.n, &to, 1)) return EQL_ERR_INVALID;
        if (need && (!apart(workspace, need, &in, 1) || !apart(workspace, need, &to, 1))) return EQL_ERR_INVALID;
        a.y = y;
        a.ldy = y_stride;
    }
    a.stats = stats;
    return status_of(eql::launch_group_norm(p->dtype, a, workspace, (hipStream_t)stream));
}

eqlinear_status eqlinear_group_norm_backward(eqlinear_plan_t p, const void* dy, int64_t dy_stride, const void* x,
                                             int64_t x_stride, const void* gamma, const void* beta,
                                             const float* stats, const int64_t* offsets, int64_t batch, void* dx,
                                             int64_t dx_stride, float* dgamma, float* dbeta, int64_t T,
                                             void* workspace, size_t workspace_bytes, void* stream) {
    if (!p || p->kind != EQL_KIND_NORM || !batch_ok(offsets, batch, T)) return EQL_ERR_INVALID;
    if ((dgamma && !aligned(dgamma, 16)) || (dbeta && !aligned(dbeta, 16))) return EQL_ERR_INVALID;
    const uint64_t gb = (uint64_t)p->C_in * 4;
    if (dgamma && dbeta && overlaps(dgamma, gb, dbeta, gb)) return EQL_ERR_INVALID;
    if (T == 0 && !dgamma && !dbeta) return EQL_OK;
    const size_t es = elem_size(p);
    const int64_t W = (int64_t)p->C_in * p->N;
    const size_t need = eqlinear_group_norm_workspace(p, T, batch, 1);
    if (!workspace_ok(workspace, workspace_bytes, need)) return EQL_ERR_INVALID;
    const uint64_t sb = (uint64_t)batch * p->groups * 8, cb = (uint64_t)p->C_in * es;
    const Range ends{offsets, (uint64_t)(batch + 1) * 8};
    if (!disjoint({{dgamma, gb}, {dbeta, gb}, {workspace, need}}, {{gamma, cb}, {beta, cb}, {stats, sb}, ends}))
        return EQL_ERR_INVALID;
    eql::NormArgs a = norm_args(p, x, x_stride, gamma, beta, offsets, batch, T);
    if (T > 0) {
        if (!stats || !aligned(stats, 8)) return EQL_ERR_INVALID;
        const Span in[2] = {{x, T, x_stride, 1, 0, W, es}, {dy, T, dy_stride, 1, 0, W, es}};
        const Span to{dx, T, dx_stride, 1, 0, W, es};
        if (!readable(in[0]) || !readable(in[1]) || !writable(to) || collide(to, in[0])) return EQL_ERR_INVALID;
        if (!same_place(in[1], to) && collide(to, in[1])) return EQL_ERR_INVALID;
        for (const void* v : {gamma, beta})
            if (v && (!aligned(v, es) || !apart(v, cb, &to, 1))) return EQL_ERR_INVALID;
        if (!apart(stats, sb, &to, 1) || !apart(ends.p, ends.n, &to, 1)) return EQL_ERR_INVALID;
        for (const float* v : {dgamma, dbeta})
            if (!apart(v, gb, in, 2) || !apart(v, gb, &to, 1)) return EQL_ERR_INVALID;
        if (need && (!apart(workspace, need, in, 2) || !apart(workspace, need, &to, 1))) return EQL_ERR_INVALID;
        a.dy = dy, a.lddy = dy_stride;
        a.dx = dx, a.lddx = dx_stride;
    }
    a.stats = const_cast<float*>(stats);
    a.dgamma = dgamma;
    a.dbeta = dbeta;
    return status_of(eql::launch_group_norm_backward(p->dtype, a, workspace, (hipStream_t)stream));
}

}  // extern "C"
