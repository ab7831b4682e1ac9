// linear_attention.hip -- linear attention: the products of the forward and the
// backward as jobs of the chunk kernels (linear_attention.h, instantiated in
// linear_attention_{bf16,f16,f32}.hip), and the single-token step.
#include "linear_attention.h"

namespace eql {

namespace mix {
extern template hipError_t run<float>(Jobs&, hipStream_t);
extern template hipError_t run<__bf16>(Jobs&, hipStream_t);
extern template hipError_t run<_Float16>(Jobs&, hipStream_t);
}  // namespace mix

namespace {

using namespace mix;

// Segments of long sequences: as many as fill the CUs once (each of the kernel's
// workgroups per CU counted), of at least four chunks; none where the sequences and heads
// alone half fill them.  f16, 32768 tokens, 10 heads of 112: 142 us in 25 segments a head
// (state pass 47, join 11, outputs 104); twice as many took a tenth longer.  Lengths are on
// the device, so the rule goes by their mean: one sequence far longer than the others is one
// workgroup's a head.
struct Split {
    int64_t seg_len = 0, slots = 0;
};
Split split_for(int io, int heads, int D_k, int D_v, int64_t T, int64_t batch, bool ragged) {
    Split s;
    s.slots = batch;
    const int64_t mean = T / batch;
    const int nw = waves_for(D_v > D_k ? D_v : D_k), kb = padded_a(D_v > D_k ? D_v : D_k);
    const int64_t fill = 256 * (int64_t)waves_per_simd(io == kIoF32 ? 4 : 2, kb, nw) * 4 / nw;
    if (2 * batch * heads > fill || mean < 8 * kChunk) return s;
    const int64_t want = fill / (batch * heads);
    int64_t chunks = ((mean + kChunk - 1) / kChunk + want - 1) / want;
    chunks = chunks < 4 ? 4 : chunks;
    s.seg_len = chunks * kChunk;
    s.slots = ragged ? T / s.seg_len + batch : batch * ((mean + s.seg_len - 1) / s.seg_len);
    return s;
}

size_t part_bytes(const Split& s, int Hkv, int Da, int Dc) {
    return s.seg_len ? (size_t)s.slots * Hkv * waves_for(Dc) * 16 * padded_a(Da) * 32 * 4 : 0;
}


Job job(const Heads& x, const Heads& y, const Heads& z, const Heads& out, int Ha, int Hb, int Da, int Dc, int reverse,
        const MixArgs& a, const Split& s, const float* S0, float* S1, int sa, int sc) {
    Job j{};
    j.a = x, j.b = y, j.c = z, j.out = out;
    j.Ha = Ha, j.Hb = Hb, j.Da = Da, j.Dc = Dc;
    j.reverse = reverse;
    j.scale = a.scale;
    j.log_decay = a.log_decay;
    j.S0 = S0, j.S1 = S1;
    j.sa = sa, j.sc = sc;
    j.offsets = a.offsets;
    j.batch = a.batch;
    j.T = a.T;
    j.seg_len = s.seg_len;
    j.slots = s.slots;
    j.mean = a.batch ? a.T / a.batch : 0;
    j.per_seq = s.seg_len ? (uint32_t)((j.mean + s.seg_len - 1) / s.seg_len) : 1;
    return j;
}

hipError_t run_jobs(int io, Jobs& jobs, hipStream_t stream) {
    return io == kIoF32 ? run<float>(jobs, stream)
                        : (io == kIoBF16 ? run<__bf16>(jobs, stream) : run<_Float16>(jobs, stream));
}

}  // namespace

// The backward's parts: of dq and dk (D_v x D_k), then of dv (D_k x D_v).
size_t linear_attention_workspace(int io, int heads, int kv_heads, int D_k, int D_v, int64_t T, int64_t batch,
                                  bool backward) {
    if (T <= 0 || batch <= 0) return 0;
    const Split s = split_for(io, heads, D_k, D_v, T, batch, true);  // packed sequences need the most slots
    const size_t n = part_bytes(s, kv_heads, D_k, D_v);
    return backward ? 2 * part_bytes(s, kv_heads, D_v, D_k) + n : n;
}

hipError_t launch_linear_attention(int io, const MixArgs& a, void* ws, hipStream_t stream) {
    const Split s = split_for(io, a.heads, a.D_k, a.D_v, a.T, a.batch, a.offsets != nullptr);
    Jobs jobs{};
    jobs.count = 1;
    jobs.j[0] = job(a.q, a.k, a.v, a.o, a.heads, a.kv_heads, a.D_k, a.D_v, 0, a, s, a.state_in, a.state_out, a.D_v, 1);
    jobs.j[0].part = static_cast<float*>(ws);
    return run_jobs(io, jobs, stream);
}

// dk and dv first: with shared heads theirs are the longest workgroups.
hipError_t launch_linear_attention_backward(int io, const MixArgs& a, void* ws, hipStream_t stream) {
    const Split s = split_for(io, a.heads, a.D_k, a.D_v, a.T, a.batch, a.offsets != nullptr);
    const size_t n = part_bytes(s, a.kv_heads, a.D_v, a.D_k);
    Job dk = job(a.v, a.d_o, a.q, a.dk, a.kv_heads, a.heads, a.D_v, a.D_k, 1, a, s, a.d_state_out, nullptr, 1, a.D_v);
    Job dv = job(a.k, a.q, a.d_o, a.dv, a.kv_heads, a.heads, a.D_k, a.D_v, 1, a, s, a.d_state_out, a.d_state_in, a.D_v, 1);
    Job dq = job(a.d_o, a.v, a.k, a.dq, a.heads, a.kv_heads, a.D_v, a.D_k, 0, a, s, a.state_in, nullptr, 1, a.D_v);
    dk.part = static_cast<float*>(ws);
    dq.part = reinterpret_cast<float*>(static_cast<char*>(ws) + n);
    dv.part = reinterpret_cast<float*>(static_cast<char*>(ws) + 2 * n);
    Jobs jobs{};
    if (padded_a(a.D_k) == padded_a(a.D_v) && waves_for(a.D_k) == waves_for(a.D_v)) {
        jobs.count = 3;
        jobs.j[0] = dk, jobs.j[1] = dv, jobs.j[2] = dq;
        return run_jobs(io, jobs, stream);
    }
    jobs.count = 2;
    jobs.j[0] = dk, jobs.j[1] = dq;
    const hipError_t e = run_jobs(io, jobs, stream);
    if (e != hipSuccess) return e;
    jobs = Jobs{};
    jobs.count = 1;
    jobs.j[0] = dv;
    return run_jobs(io, jobs, stream);
}

namespace {

// One token.  A workgroup takes one (sequence, kv head): each thread reads, updates
// and writes back four columns (one, where D_v is odd against that) of rows row,
// row + rows, ... of the state, and adds them into the outputs of HB query heads that
// share it; further heads, HB at a time, read the state again.  The state, read and
// written once, is all the traffic that counts; its loads go out U at a time.  512
// sequences, 4 kv heads of 128 x 128 (273 MB): 60.0 us, 4.5 TB/s, a copy's rate; 8
// sequences: 4.8 us of one launch.
template <typename IO, bool VEC, int HB>
__global__ __launch_bounds__(256) void step_kernel(MixArgs a, int cols, uint32_t base) {
    constexpr int U = 4, W = VEC ? 4 : 1;  // columns of a thread
    __shared__ float vk[kMaxD], vq[HB][kMaxD], red[HB][256 * W];
    const uint32_t wg = blockIdx.x + base;
    const int64_t b = wg / (uint32_t)a.kv_heads;
    const int kv = (int)(wg % (uint32_t)a.kv_heads), r = a.heads / a.kv_heads, tid = (int)threadIdx.x;
    const int rows = 256 / cols, row = tid / cols, c = (tid - row * cols) * W;
    const bool on = row < rows;
    using R = std::conditional_t<VEC, f32x4, float>;
    float* S = a.state_out + (int64_t)wg * a.D_k * a.D_v + c;
    const float g = power(a.log_decay[kv] * kLog2e, 1);
    R v{};
    if (on) {
        const IO* p = (const IO*)a.v.p + b * a.v.ts + kv * a.v.hs + c;
        if constexpr (VEC) {
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = (float)p[i];
        } else {
            v = (float)p[0];
        }
    }
    if (tid < a.D_k) vk[tid] = (float)((const IO*)a.k.p)[b * a.k.ts + kv * a.k.hs + tid];
    for (int h0 = 0; h0 < r; h0 += HB) {
        const int nh = r - h0 < HB ? r - h0 : HB;
        const IO* q = (const IO*)a.q.p + b * a.q.ts + (int64_t)(kv * r + h0) * a.q.hs;
        for (int e = tid; e < nh * kMaxD; e += 256) {
            const int h = e / kMaxD, i = e % kMaxD;
            if (i < a.D_k) vq[h][i] = a.scale * (float)q[h * a.q.hs + i];
        }
        __syncthreads();
        R o[HB];
#pragma unroll
        for (int h = 0; h < HB; ++h) o[h] = R{};
        if (on)
            for (int i0 = row; i0 < a.D_k; i0 += U * rows) {
                R s[U];
#pragma unroll
                for (int u = 0; u < U; ++u)
                    if (i0 + u * rows < a.D_k) s[u] = *reinterpret_cast<const R*>(S + (i0 + u * rows) * a.D_v);
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const int i = i0 + u * rows;
                    if (i < a.D_k) {
                        if (h0 == 0) {
                            s[u] = s[u] * g + v * vk[i];
                            *reinterpret_cast<R*>(S + i * a.D_v) = s[u];
                        }
#pragma unroll
                        for (int h = 0; h < HB; ++h)
                            if (h < nh) o[h] += s[u] * vq[h][i];
                    }
                }
            }
#pragma unroll
        for (int h = 0; h < HB; ++h) *reinterpret_cast<R*>(red[h] + tid * W) = o[h];
        __syncthreads();
        IO* out = (IO*)const_cast<void*>(a.o.p) + b * a.o.ts + (int64_t)(kv * r + h0) * a.o.hs;
        for (int e = tid; e < nh * a.D_v; e += 256) {
            const int h = e / a.D_v, i = e - h * a.D_v;
            float w = red[h][i];
            for (int k = 1; k < rows; ++k) w += red[h][k * a.D_v + i];
            out[h * a.o.hs + i] = (IO)w;
        }
        __syncthreads();
    }
}

template <typename IO>
hipError_t step(const MixArgs& a, hipStream_t stream) {
    const int r = a.heads / a.kv_heads;
    const bool vec = a.D_v % 4 == 0;
    const int cols = vec ? a.D_v / 4 : a.D_v;
    in_pieces(a.batch * a.kv_heads, 256, [&](uint32_t base, uint32_t wgs) {
        const dim3 grid(wgs);
        if (!vec) hipLaunchKernelGGL((step_kernel<IO, false, 2>), grid, dim3(256), 0, stream, a, cols, base);
        else if (r == 1) hipLaunchKernelGGL((step_kernel<IO, true, 1>), grid, dim3(256), 0, stream, a, cols, base);
        else if (r == 2) hipLaunchKernelGGL((step_kernel<IO, true, 2>), grid, dim3(256), 0, stream, a, cols, base);
        else hipLaunchKernelGGL((step_kernel<IO, true, 4>), grid, dim3(256), 0, stream, a, cols, base);
    });
    return hipGetLastError();
}

}  // namespace

hipError_t launch_linear_attention_step(int io, const MixArgs& a, hipStream_t stream) {
    if (a.batch * a.kv_heads > 0x7fffffff) return hipErrorNotSupported;
    return io == kIoF32 ? step<float>(a, stream)
                        : (io == kIoBF16 ? step<__bf16>(a, stream) : step<_Float16>(a, stream));
}

}  // namespace eql
