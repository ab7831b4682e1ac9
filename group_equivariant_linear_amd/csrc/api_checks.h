// api_checks.h -- argument checks shared by the operators' C ABI (mixer_api.hip,
// attention_api.hip; not part of the ABI).
#pragma once

#include <cmath>
#include <initializer_list>
#include <new>

#include "eq_plan.h"

namespace eql {

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

inline Span span_of(const eqlinear_heads& h, int64_t T, int n_heads, int64_t run, size_t es) {
    return Span{h.ptr, T, h.token_stride, n_heads, h.head_stride, run, es};
}

inline bool readable(const Span& s) {
    if (!s.p || (uintptr_t)s.p % s.es != 0 || s.ts < 0 || s.hs < 0) return false;
    // offsets stay far from the end of the address space
    return s.ts <= ((int64_t)1 << 40) && s.hs <= ((int64_t)1 << 40) && s.T <= ((int64_t)1 << 40) &&
           (double)s.T * (double)s.ts + (double)s.n_heads * (double)s.hs < 1e15;
}

// an output: no element twice
inline bool writable(const Span& s) {
    if (!readable(s)) return false;
    const int64_t row = s.row();
    if (row >= 0 && (s.T == 1 || s.ts >= row)) return true;                       // token after token
    return s.ts >= s.run && (s.n_heads == 1 || s.hs >= (s.T - 1) * s.ts + s.run);  // head after head
}

// Whether two tensors may share an element.  Apart are: address ranges that do not meet; with
// equal token strides, rows (all of a token's runs) that do not meet modulo the stride; and with
// equal head strides besides, runs that do not meet modulo the head stride (heads of q, k and v
// in turn).
inline bool collide(const Span& a, const Span& b) {
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

inline bool same_place(const Span& a, const Span& b) {
    return a.p == b.p && (a.T == 1 || a.ts == b.ts) && (a.n_heads == 1 || a.hs == b.hs);
}

inline Heads heads_of(const eqlinear_heads& h) { return Heads{h.ptr, h.token_stride, h.head_stride}; }

inline bool batch_ok(const int64_t* offsets, int64_t batch, int64_t T) {
    if (T < 0 || batch < 0 || batch > 0x7fffffff || T > ((int64_t)1 << 40)) return false;
    if (offsets) return batch > 0 && ((uintptr_t)offsets & 7u) == 0;
    return batch > 0 ? T % batch == 0 : T == 0;
}

inline bool workspace_ok(const void* ws, size_t bytes, size_t need) {
    return need == 0 || (ws && ((uintptr_t)ws & 255u) == 0 && bytes >= need);
}

// Flat buffers of a call (null or empty: not given): what it writes shares no byte with
// anything else of it.
struct Range {
    const void* p;
    uint64_t n;
};
inline bool disjoint(std::initializer_list<Range> written, std::initializer_list<Range> read) {
    auto meet = [](const Range& a, const Range& b) { return a.p && b.p && a.n && b.n && overlaps(a.p, a.n, b.p, b.n); };
    for (auto w = written.begin(); w != written.end(); ++w) {
        for (auto v = written.begin(); v != w; ++v)
            if (meet(*v, *w)) return false;
        for (const Range& r : read)
            if (meet(*w, r)) return false;
    }
    return true;
}

inline bool aligned(const void* p, size_t a) { return (uintptr_t)p % a == 0; }

inline eqlinear_status status_of(hipError_t e) { return e == hipErrorNotSupported ? EQL_ERR_UNSUPPORTED : hip_status(e); }

// What the forward, the backward and the step check alike; `n` tensors in, the
// first `n_out` of `to` out.
inline bool tensors_ok(const Span* in, int n, const Span* to, int n_out) {
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

inline bool apart(const void* a, uint64_t bytes, const Span* s, int n) {
    for (int i = 0; a && i < n; ++i)
        if (overlaps(a, bytes, s[i].p, s[i].bytes())) return false;
    return true;
}

}  // namespace eql
