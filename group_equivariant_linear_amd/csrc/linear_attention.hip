// linear_attention.hip -- causal linear attention with a decay for each head.
//
// Every product of the forward and the backward has one form.  With rows a_t, b_t,
// c_t and a state S (D_a x D_c),
//   out_t = scale (a_t . state),  state = sum over s <= t (t <= s if reversed) of
//           g^|t-s| b_s c_s^T + (decayed initial state)
//   forward:  a = q,   b = k,   c = v                   initial state_in
//   dq:       a = d_o, b = v,   c = k                   initial state_in^T
//   dk:       a = v,   b = d_o, c = q,   reversed       initial d_state_out^T / scale
//   dv:       a = k,   b = q,   c = d_o, reversed       initial d_state_out / scale
// Forward in time the initial state decays before the first token; reversed it does
// not before the last.  d_state_in = g scale (the state of the dv product at token 0).
#include "eq_device.h"
#include "eq_launch.h"

namespace eql {
namespace {

constexpr int kMaxD = 128;

struct Job {
    Heads a, b, c, out;
    int Ha, Hb, Da, Dc;  // heads of a and out, of b and c; numbers per head
    int reverse;
    float scale;
    const float* log_decay;  // min(Ha, Hb) decays
    const float* S0;         // initial and final states [batch][kv][...]: element (i, j)
    float* S1;               // at i sa + j sc
    int sa, sc;
};

__device__ __forceinline__ void sequence(const int64_t* offsets, int64_t batch, int64_t T, int64_t b, int64_t& t0,
                                         int64_t& t1) {
    if (offsets) {
        t0 = offsets[b], t1 = offsets[b + 1];
        t0 = t0 < 0 ? 0 : (t0 > T ? T : t0);
        t1 = t1 < t0 ? t0 : (t1 > T ? T : t1);
    } else {
        const int64_t n = T / batch;
        t0 = b * n, t1 = t0 + n;
    }
}

// One workgroup per (sequence, head of a): token by token, the state in LDS.
template <typename IO>
__global__ __launch_bounds__(256) void recurrent_kernel(Job j, const int64_t* offsets, int64_t batch, int64_t T) {
    extern __shared__ float lds[];
    float* S = lds;                  // [Da][Dc]
    float* va = S + j.Da * j.Dc;     // [Da]
    float* vb = va + kMaxD;          // [Da]
    float* vc = vb + kMaxD;          // [Dc]
    const int64_t b = blockIdx.x / j.Ha;
    const int h = (int)(blockIdx.x % j.Ha), Hkv = j.Ha < j.Hb ? j.Ha : j.Hb;
    const int kv = j.Ha <= j.Hb ? h : h / (j.Ha / j.Hb), rb = j.Hb > j.Ha ? j.Hb / j.Ha : 1;
    const int tid = (int)threadIdx.x, n = j.Da * j.Dc;
    int64_t t0, t1;
    sequence(offsets, batch, T, b, t0, t1);
    const float g = expf(j.log_decay[kv]);
    const int64_t at = (b * Hkv + kv) * n;
    const bool empty = t1 == t0;  // passes its state through as it is
    const float s0 = j.reverse && !empty ? 1.0f / j.scale : 1.0f;
    for (int e = tid; e < n; e += 256)
        S[e] = j.S0 ? s0 * j.S0[at + (int64_t)(e / j.Dc) * j.sa + (int64_t)(e % j.Dc) * j.sc] : 0.0f;
    for (int64_t s = 0; s < t1 - t0; ++s) {
        const int64_t t = j.reverse ? t1 - 1 - s : t0 + s;
        for (int hh = 0; hh < rb; ++hh) {
            const int hb = j.Hb > j.Ha ? h * rb + hh : kv;
            __syncthreads();
            for (int e = tid; e < j.Da; e += 256) {
                va[e] = (float)((const IO*)j.a.p)[t * j.a.ts + h * j.a.hs + e];
                vb[e] = (float)((const IO*)j.b.p)[t * j.b.ts + hb * j.b.hs + e];
            }
            for (int e = tid; e < j.Dc; e += 256) vc[e] = (float)((const IO*)j.c.p)[t * j.c.ts + hb * j.c.hs + e];
            __syncthreads();
            const float gg = hh > 0 || (j.reverse && s == 0) ? 1.0f : g;
            for (int e = tid; e < n; e += 256) S[e] = fmaf(vb[e / j.Dc], vc[e % j.Dc], gg * S[e]);
        }
        __syncthreads();
        for (int c = tid; c < j.Dc; c += 256) {
            float o = 0.0f;
            for (int i = 0; i < j.Da; ++i) o = fmaf(va[i], S[i * j.Dc + c], o);
            ((IO*)const_cast<void*>(j.out.p))[t * j.out.ts + h * j.out.hs + c] = (IO)(o * j.scale);
        }
    }
    __syncthreads();
    if (j.S1 && (j.Ha <= j.Hb || h % (j.Ha / j.Hb) == 0)) {
        const float s1 = j.reverse && !empty ? g * j.scale : 1.0f;
        for (int e = tid; e < n; e += 256)
            j.S1[at + (int64_t)(e / j.Dc) * j.sa + (int64_t)(e % j.Dc) * j.sc] = s1 * S[e];
    }
}

template <typename IO>
hipError_t run(const Job& j, const MixArgs& a, hipStream_t stream) {
    if (a.batch * j.Ha > 0x7fffffff) return hipErrorNotSupported;
    const int lds = (j.Da * j.Dc + 3 * kMaxD) * 4;
    hipLaunchKernelGGL(recurrent_kernel<IO>, dim3((uint32_t)(a.batch * j.Ha)), dim3(256), lds, stream, j, a.offsets,
                       a.batch, a.T);
    return hipGetLastError();
}

Job forward_job(const MixArgs& a) {
    return Job{a.q, a.k, a.v, a.o, a.heads, a.kv_heads, a.D_k, a.D_v, 0, a.scale, a.log_decay,
               a.state_in, a.state_out, a.D_v, 1};
}

template <typename IO>
hipError_t backward(const MixArgs& a, hipStream_t stream) {
    const Job dq{a.d_o, a.v, a.k, a.dq, a.heads, a.kv_heads, a.D_v, a.D_k, 0, a.scale, a.log_decay,
                 a.state_in, nullptr, 1, a.D_v};
    const Job dk{a.v, a.d_o, a.q, a.dk, a.kv_heads, a.heads, a.D_v, a.D_k, 1, a.scale, a.log_decay,
                 a.d_state_out, nullptr, 1, a.D_v};
    const Job dv{a.k, a.q, a.d_o, a.dv, a.kv_heads, a.heads, a.D_k, a.D_v, 1, a.scale, a.log_decay,
                 a.d_state_out, a.d_state_in, a.D_v, 1};
    for (const Job& j : {dq, dk, dv}) {
        const hipError_t e = run<IO>(j, a, stream);
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

}  // namespace

size_t linear_attention_workspace(int, int, int, int, int, int64_t, int64_t, bool) { return 0; }

hipError_t launch_linear_attention(int io, const MixArgs& a, void*, hipStream_t stream) {
    const Job j = forward_job(a);
    return io == kIoF32 ? run<float>(j, a, stream)
                        : (io == kIoBF16 ? run<__bf16>(j, a, stream) : run<_Float16>(j, a, stream));
}

hipError_t launch_linear_attention_backward(int io, const MixArgs& a, void*, hipStream_t stream) {
    return io == kIoF32 ? backward<float>(a, stream)
                        : (io == kIoBF16 ? backward<__bf16>(a, stream) : backward<_Float16>(a, stream));
}

namespace {

// One workgroup per (sequence, kv head): the state in memory, each element read and
// written once, for all query heads that share it.
template <typename IO>
__global__ __launch_bounds__(256) void step_kernel(MixArgs a) {
    __shared__ float vk[kMaxD], vv[kMaxD], vq[kMaxD];
    const int64_t b = blockIdx.x / a.kv_heads;
    const int kv = (int)(blockIdx.x % a.kv_heads), r = a.heads / a.kv_heads, tid = (int)threadIdx.x;
    const float g = expf(a.log_decay[kv]);
    float* S = a.state_out + (int64_t)blockIdx.x * a.D_k * a.D_v;
    for (int e = tid; e < a.D_k; e += 256) vk[e] = (float)((const IO*)a.k.p)[b * a.k.ts + kv * a.k.hs + e];
    for (int e = tid; e < a.D_v; e += 256) vv[e] = (float)((const IO*)a.v.p)[b * a.v.ts + kv * a.v.hs + e];
    __syncthreads();
    for (int e = tid; e < a.D_k * a.D_v; e += 256) S[e] = fmaf(vk[e / a.D_v], vv[e % a.D_v], g * S[e]);
    for (int hh = 0; hh < r; ++hh) {
        const int h = kv * r + hh;
        __syncthreads();
        for (int e = tid; e < a.D_k; e += 256) vq[e] = (float)((const IO*)a.q.p)[b * a.q.ts + h * a.q.hs + e];
        __syncthreads();
        for (int c = tid; c < a.D_v; c += 256) {
            float o = 0.0f;
            for (int i = 0; i < a.D_k; ++i) o = fmaf(vq[i], S[i * a.D_v + c], o);
            ((IO*)const_cast<void*>(a.o.p))[b * a.o.ts + h * a.o.hs + c] = (IO)(o * a.scale);
        }
    }
}

}  // namespace

hipError_t launch_linear_attention_step(int io, const MixArgs& a, hipStream_t stream) {
    if (a.batch * a.kv_heads > 0x7fffffff) return hipErrorNotSupported;
    const dim3 grid((uint32_t)(a.batch * a.kv_heads));
    if (io == kIoF32) hipLaunchKernelGGL(step_kernel<float>, grid, dim3(256), 0, stream, a);
    else if (io == kIoBF16) hipLaunchKernelGGL(step_kernel<__bf16>, grid, dim3(256), 0, stream, a);
    else hipLaunchKernelGGL(step_kernel<_Float16>, grid, dim3(256), 0, stream, a);
    return hipGetLastError();
}

}  // namespace eql
