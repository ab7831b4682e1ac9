// group_norm.hip -- group norm with an activation, channels last, and its gradients.
//
// A slab is one sample's part of one group: its tokens x W = (C / groups) N numbers,
// contiguous within a token.  All paths read a token's row in pieces of V numbers (16
// bytes where every row is aligned for them, else single numbers), and every thread
// keeps its columns from token to token, so that gamma, beta and the sums over tokens
// that make dgamma and dbeta stay in registers.  Three paths:
//   token  every token its own sample: a slab is a few lanes' registers;
//   slab   a sample's slab fits the registers of a workgroup: one pass over memory;
//   split  longer samples: blocks of tokens, each block's sums to memory, a join, and
//          a second pass.
// The variance is a mean of squared differences from the mean (in registers), or, over
// blocks, merged from such by mean and squared sum (Chan, Golub, LeVeque 1983).
// The sums run in a fixed order.  Memory is the floor of all three; measured, 96 x 8
// numbers a token in bf16:
//   token  12608 tokens: forward 12.7 us (38.7 MB, 3.0 TB/s), backward 18.0 and 4.2 for the
//          sums of dgamma and dbeta;
//   slab   64 images of 197 tokens: forward 23 us, backward 30 (equal lengths) or 38
//          (unequal ones); bound by GELU's arithmetic and by workgroups of one
//          pass each: all loads first, then all sums, then all stores;
//   split  one map of 32768 tokens (160 x 7, f16): sums 25 us, join 6, outputs 28 (147 MB,
//          5.2 TB/s); x is read twice, the second time partly from the last-level cache.
#include "activation.h"
#include "eq_device.h"
#include "eq_launch.h"

namespace eql {
namespace {

// A norm over its arguments, with what the host derived from them.
struct Norm {
    NormArgs a;
    int W, cols, cpg;      // numbers and pieces of a slab's token; channels per group
    int lps;               // token path: lanes per slab (a power of two)
    int pg, unit;          // token path: groups of a token, padded; workgroups that share a part, or 0
    int rows;              // slab, split paths: tokens that a workgroup covers at once
    int64_t step;          // token path: tokens from one pass to the next; slab path: samples
    int64_t block, slots;  // split path: tokens of a block, blocks
    uint32_t base;         // split path: first workgroup of this launch
    float* part;           // dgamma and dbeta of part of the tokens: [..][2][C]
    float* moments;        // split path: [slots][groups][2]
    float* sums;           // split path, backward: [slots][tiles + groups][2]
    float* joined;         // split path: [batch][groups][2]
};

__device__ __forceinline__ void sample_range(const NormArgs& a, int64_t b, int64_t& t0, int64_t& t1) {
    if (a.offsets) {
        t0 = a.offsets[b], t1 = a.offsets[b + 1];
        t0 = t0 < 0 ? 0 : (t0 > a.T ? a.T : t0);
        t1 = t1 < t0 ? t0 : (t1 > a.T ? a.T : t1);
    } else {
        const int64_t n = a.T / a.batch;
        t0 = b * n, t1 = t0 + n;
    }
}

// A piece of V numbers: 16 bytes, or one number.
template <typename IO, int V>
struct Piece {
    static constexpr bool WIDE = V > 1;
    using R = std::conditional_t<WIDE, u32x4, uint32_t>;
    R r;
    static __device__ __forceinline__ Piece load(const IO* p) {
        if constexpr (WIDE) return Piece{*reinterpret_cast<const u32x4*>(p)};
        else if constexpr (sizeof(IO) == 4) return Piece{*reinterpret_cast<const uint32_t*>(p)};
        else return Piece{(uint32_t)*reinterpret_cast<const uint16_t*>(p)};
    }
    static __device__ __forceinline__ Piece zero() {
        if constexpr (WIDE) return Piece{u32x4{0u, 0u, 0u, 0u}};
        else return Piece{0u};
    }
    // The next get() converts again: without it the compiler keeps the fp32 numbers of
    // one pass for the next, twice the registers of the pieces.
    __device__ __forceinline__ void keep_packed() { asm volatile("" : "+v"(r)); }
    __device__ __forceinline__ void get(float (&v)[V]) const {
        if constexpr (WIDE && sizeof(IO) == 4) {
#pragma unroll
            for (int i = 0; i < V; ++i) v[i] = __uint_as_float(r[i]);
        } else if constexpr (WIDE) {
#pragma unroll
            for (int i = 0; i < V; ++i) v[i] = i & 1 ? Half<IO>::hi(r[i >> 1]) : Half<IO>::lo(r[i >> 1]);
        } else if constexpr (sizeof(IO) == 4) {
            v[0] = __uint_as_float(r);
        } else {
            v[0] = Half<IO>::lo(r);
        }
    }
    static __device__ __forceinline__ void store(IO* p, const float (&v)[V]) {
        if constexpr (WIDE && sizeof(IO) == 4) {
            *reinterpret_cast<f32x4*>(p) = f32x4{v[0], v[1], v[2], v[3]};
        } else if constexpr (WIDE) {
            u32x4 u;
#pragma unroll
            for (int i = 0; i < 4; ++i) u[i] = Half<IO>::pack2(v[2 * i], v[2 * i + 1]);
            *reinterpret_cast<u32x4*>(p) = u;
        } else {
            p[0] = (IO)v[0];
        }
    }
};

// gamma and beta of the numbers e .. e + V - 1 of a token's row: CP of them, V or, where
// N is a multiple of V and a piece lies within a channel, one.
template <typename IO, int CP>
__device__ __forceinline__ void affine(const NormArgs& a, int e, float (&gm)[CP], float (&be)[CP]) {
    int c = e / a.N, n = e - c * a.N;
#pragma unroll
    for (int i = 0; i < CP; ++i) {
        gm[i] = a.gamma ? (float)((const IO*)a.gamma)[c] : 1.0f;
        be[i] = a.beta ? (float)((const IO*)a.beta)[c] : 0.0f;
        if (++n == a.N) n = 0, ++c;
    }
}

template <int ACT, int V>
__device__ __forceinline__ void act_all(float (&v)[V]) {
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = act_value<ACT>(v[i]);
}
template <int V>
__device__ __forceinline__ void act_all(int act, float (&v)[V]) {
    if (act == kActGelu) act_all<kActGelu>(v);
    else if (act == kActSilu) act_all<kActSilu>(v);
}
// d *= act'(z)
template <int V>
__device__ __forceinline__ void slope_all(int act, const float (&z)[V], float (&d)[V]) {
    if (act == kActGelu) {
#pragma unroll
        for (int i = 0; i < V; ++i) d[i] *= act_slope<kActGelu>(z[i]);
    } else if (act == kActSilu) {
#pragma unroll
        for (int i = 0; i < V; ++i) d[i] *= act_slope<kActSilu>(z[i]);
    }
}

// y = act(gamma (x - mean) rstd + beta) of one piece
template <typename IO, int V, int CP>
__device__ __forceinline__ void put_y(const NormArgs& a, IO* to, const Piece<IO, V>& x, float mean, float rstd,
                                      const float (&gm)[CP], const float (&be)[CP]) {
    float v[V];
    x.get(v);
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = fmaf((v[i] - mean) * rstd, gm[i % CP], be[i % CP]);
    act_all(a.act, v);
    Piece<IO, V>::store(to, v);
}

// xh and dz = dy act'(gamma xh + beta) of one piece
template <typename IO, int V, int CP>
__device__ __forceinline__ void get_dz(const NormArgs& a, const Piece<IO, V>& x, const Piece<IO, V>& dy, float mean,
                                       float rstd, const float (&gm)[CP], const float (&be)[CP], float (&xh)[V],
                                       float (&dz)[V]) {
    float z[V];
    x.get(xh);
    dy.get(dz);
#pragma unroll
    for (int i = 0; i < V; ++i) {
        xh[i] = (xh[i] - mean) * rstd;
        z[i] = fmaf(xh[i], gm[i % CP], be[i % CP]);
    }
    slope_all(a.act, z, dz);
}

template <typename IO, int V, int CP>
__device__ __forceinline__ void put_dx(IO* to, const float (&xh)[V], const float (&dz)[V], const float (&gm)[CP],
                                       float m1, float m2, float rstd) {
    float v[V];
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = (fmaf(dz[i], gm[i % CP], -m1) - xh[i] * m2) * rstd;
    Piece<IO, V>::store(to, v);
}

__device__ __forceinline__ float lane_sum(float v, int lanes) {
    for (int o = lanes >> 1; o > 0; o >>= 1) v += __shfl_xor(v, o);
    return v;
}

// Sum over a workgroup of NT threads; red: NT / 64 floats, free again after the call
template <int NT>
__device__ __forceinline__ float block_sum(float v, float* red) {
    v = lane_sum(v, 64);
    if constexpr (NT > 64) {
        if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
        __syncthreads();
        v = red[0];
#pragma unroll
        for (int w = 1; w < NT / 64; ++w) v += red[w];
        __syncthreads();
    }
    return v;
}

// --- token path -----------------------------------------------------------------------
// Slabs are numbered token by token, group by group (pg of them, of which those past the
// last group are nobody's); a wave takes 64 / lps of them at once, a lane K pieces of its
// slab.  Waves step by whole tokens, so a lane keeps its group.  The next token's pieces load
// while the current one's are worked on.
struct Slab {
    int64_t t;
    int g;
    __device__ __forceinline__ Slab(const Norm& s, int64_t slab) : t(slab / s.pg), g((int)(slab - t * s.pg)) {
        if (g >= s.a.groups) t = s.a.T, g = 0;  // no token
    }
};
template <typename IO, int V, int CP, int K>
__global__ __launch_bounds__(256) void token_forward_kernel(Norm s) {
    const NormArgs& a = s.a;
    using P = Piece<IO, V>;
    const int lane = (int)threadIdx.x & 63, sub = lane & (s.lps - 1);
    const int64_t slab = ((int64_t)blockIdx.x * 4 + (threadIdx.x >> 6)) * (64 / s.lps) + lane / s.lps;
    const Slab first(s, slab);
    int64_t t = first.t;
    const int g = first.g, e0 = g * s.W;
    float gm[K][CP], be[K][CP];
    bool in[K];
#pragma unroll
    for (int k = 0; k < K; ++k) {
        in[k] = sub + k * s.lps < s.cols;
        affine<IO>(a, e0 + (in[k] ? (sub + k * s.lps) * V : 0), gm[k], be[k]);
    }
    const float inv = 1.0f / (float)s.W;
    const IO* x = (const IO*)a.x + e0 + sub * V;
    IO* y = (IO*)a.y + e0 + sub * V;
    P now[K];
#pragma unroll
    for (int k = 0; k < K; ++k)
        now[k] = in[k] && t < a.T ? P::load(x + t * a.ldx + k * s.lps * V) : P::zero();
    while (__any(t < a.T)) {  // lanes of a wave may be a token apart
        const int64_t tn = t + s.step;
        P next[K];
#pragma unroll
        for (int k = 0; k < K; ++k)
            next[k] = in[k] && tn < a.T ? P::load(x + tn * a.ldx + k * s.lps * V) : P::zero();
        float sum = 0.0f, sq = 0.0f, v[V];
#pragma unroll
        for (int k = 0; k < K; ++k) {
            now[k].get(v);
#pragma unroll
            for (int i = 0; i < V; ++i) sum += v[i];
        }
        const float mean = lane_sum(sum, s.lps) * inv;
#pragma unroll
        for (int k = 0; k < K; ++k)
            if (in[k]) {
                now[k].get(v);
#pragma unroll
                for (int i = 0; i < V; ++i) sq = fmaf(v[i] - mean, v[i] - mean, sq);
            }
        const float rstd = 1.0f / sqrtf(lane_sum(sq, s.lps) * inv + a.eps);
        if (t < a.T) {
#pragma unroll
            for (int k = 0; k < K; ++k)
                if (in[k]) put_y<IO>(a, y + t * a.ldy + k * s.lps * V, now[k], mean, rstd, gm[k], be[k]);
            if (a.stats && sub == 0) *reinterpret_cast<float2*>(a.stats + 2 * (t * a.groups + g)) = float2{mean, rstd};
        }
#pragma unroll
        for (int k = 0; k < K; ++k) now[k] = next[k];
        t = tn;
    }
}

// The same slabs; the lane's sums of dz xh and dz over its tokens go, through LDS, to
// part as sums per channel.  Where a token takes `unit` whole workgroups, each has channels of
// its own, and unit of them make one part; else every workgroup makes one.
template <typename IO, int V, int CP, int K>
__global__ __launch_bounds__(256) void token_backward_kernel(Norm s) {
    const NormArgs& a = s.a;
    using P = Piece<IO, V>;
    __shared__ float acc[256 * K * CP];  // [slab of the workgroup][its sums, lps K CP]
    const int lane = (int)threadIdx.x & 63, sub = lane & (s.lps - 1), spw = 64 / s.lps;
    const int here = (int)(threadIdx.x >> 6) * spw + lane / s.lps;
    const int64_t base = (int64_t)blockIdx.x * 4 * spw, slab = base + here;
    const Slab first(s, slab);
    int64_t t = first.t;
    const int g = first.g, e0 = g * s.W;
    float gm[K][CP], be[K][CP], dg[K][CP], db[K][CP];
    bool in[K];
#pragma unroll
    for (int k = 0; k < K; ++k) {
        in[k] = sub + k * s.lps < s.cols;
        affine<IO>(a, e0 + (in[k] ? (sub + k * s.lps) * V : 0), gm[k], be[k]);
#pragma unroll
        for (int i = 0; i < CP; ++i) dg[k][i] = db[k][i] = 0.0f;
    }
    const float inv = 1.0f / (float)s.W;
    const IO* x = (const IO*)a.x + e0 + sub * V;
    const IO* dy = (const IO*)a.dy + e0 + sub * V;
    IO* dx = (IO*)a.dx + e0 + sub * V;
    P xn[K], dn[K];
    float2 sn{0.0f, 0.0f};
    auto load = [&](int64_t t) {
        const bool on = t < a.T;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            xn[k] = in[k] && on ? P::load(x + t * a.ldx + k * s.lps * V) : P::zero();
            dn[k] = in[k] && on ? P::load(dy + t * a.lddy + k * s.lps * V) : P::zero();
        }
        if (on) sn = *reinterpret_cast<const float2*>(a.stats + 2 * (t * a.groups + g));
    };
    load(t);
    while (__any(t < a.T)) {
        P xc[K], dc[K];
        const float2 st = sn;
#pragma unroll
        for (int k = 0; k < K; ++k) xc[k] = xn[k], dc[k] = dn[k];
        load(t + s.step);
        float xh[K][V], dz[K][V], s1 = 0.0f, s2 = 0.0f;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            get_dz<IO>(a, xc[k], dc[k], st.x, st.y, gm[k], be[k], xh[k], dz[k]);
            // (a piece past the slab or the last token has dy = 0 and adds nothing)
#pragma unroll
            for (int i = 0; i < V; ++i) {
                dg[k][i % CP] = fmaf(dz[k][i], xh[k][i], dg[k][i % CP]);
                db[k][i % CP] += dz[k][i];
                const float g = dz[k][i] * gm[k][i % CP];
                s1 += g;
                s2 = fmaf(g, xh[k][i], s2);
            }
        }
        const float m1 = lane_sum(s1, s.lps) * inv, m2 = lane_sum(s2, s.lps) * inv;
        if (t < a.T) {
#pragma unroll
            for (int k = 0; k < K; ++k)
                if (in[k]) put_dx<IO>(dx + t * a.lddx + k * s.lps * V, xh[k], dz[k], gm[k], m1, m2, st.y);
        }
        t += s.step;
    }
    if (!s.part) return;
    const int width = s.lps * K * CP, per = a.N * CP / V, g0 = (int)(base % s.pg), slabs = 4 * spw;
    const int64_t row = s.unit ? blockIdx.x / (uint32_t)s.unit : blockIdx.x;
    const int c0 = s.unit ? g0 * s.cpg : 0, c1 = s.unit && g0 + slabs < a.groups ? (g0 + slabs) * s.cpg : a.C;
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        __syncthreads();
#pragma unroll
        for (int k = 0; k < K; ++k)
#pragma unroll
            for (int i = 0; i < CP; ++i)
                acc[here * width + (sub + k * s.lps) * CP + i] = q == 0 ? dg[k][i] : db[k][i];
        __syncthreads();
        for (int c = c0 + (int)threadIdx.x; c < c1; c += 256) {
            const int gc = c / s.cpg, at = (c - gc * s.cpg) * per;
            float v = 0.0f;
            for (int j = (gc - g0 + s.pg) % s.pg; j < slabs; j += s.pg)
                for (int n = 0; n < per; ++n) v += acc[j * width + at + n];
            s.part[(row * 2 + q) * a.C + c] = v;
        }
    }
}

// (n, mean, m2) of two sets together
__device__ __forceinline__ void merge(float& n, float& mean, float& m2, float nb, float mb, float m2b) {
    const float nn = n + nb;
    if (nn == 0.0f) return;
    const float d = mb - mean, f = nb / nn;
    mean = fmaf(d, f, mean);
    m2 = m2 + m2b + d * d * n * f;
    n = nn;
}

// the 64 lanes' sets, in lane 0
__device__ __forceinline__ void merge_wave(float& n, float& mean, float& m2) {
    for (int o = 32; o > 0; o >>= 1) {
        const float nb = __shfl_down(n, o), mb = __shfl_down(mean, o), m2b = __shfl_down(m2, o);
        merge(n, mean, m2, nb, mb, m2b);
    }
}

// --- slab path ------------------------------------------------------------------------
// A workgroup takes one group of samples b, b + step, ...: thread (row, piece) holds
// tokens row, row + rows, ... of its piece, K of them in registers; tokens past those
// (in packed batches, where one sample can be much longer than the mean) are read again
// in each pass.  Past kLong times as many, the sums would be as long as the sample: its
// statistics are merged from short runs, and its gradients' sums carry what their additions lose.
// A sample is one workgroup's whatever its length.
constexpr int kLong = 4;

// sum += v, with the rounding of the addition kept in `lost` for the next one (Kahan 1965)
__device__ __forceinline__ void add_kept(float& sum, float& lost, float v) {
    const float y = v - lost, z = sum + y;
    lost = (z - sum) - y;
    sum = z;
}

// Mean and variance of a sample longer than the registers hold: moments of runs of R tokens
// about `pivot` (a number near the mean), merged per thread, with what the additions lose, per
// wave and over the waves.
template <typename IO, int V, int NT>
__device__ __forceinline__ float2 long_moments(const IO* x, int64_t ld, int64_t n, int row, int rows, bool on, float pivot,
                                               float* red) {
    using P = Piece<IO, V>;
    constexpr int R = 4, WAVES = NT / 64;
    float cn = 0.0f, cmean = 0.0f, cm2 = 0.0f, lmean = 0.0f, lm2 = 0.0f, v[V];
    for (int64_t t0 = on ? row : n; t0 < n; t0 += (int64_t)R * rows) {
        P q[R];
        const int64_t left = (n - t0 + rows - 1) / rows;
        const int m = left < R ? (int)left : R;
#pragma unroll
        for (int u = 0; u < R; ++u) q[u] = u < m ? P::load(x + (t0 + (int64_t)u * rows) * ld) : P::zero();
        float d = 0.0f, d2 = 0.0f;
#pragma unroll
        for (int u = 0; u < R; ++u)
            if (u < m) {
                q[u].get(v);
#pragma unroll
                for (int i = 0; i < V; ++i) d += v[i] - pivot;
            }
        const float nb = (float)(m * V), mb = d / nb;
#pragma unroll
        for (int u = 0; u < R; ++u)
            if (u < m) {
                q[u].keep_packed();
                q[u].get(v);
#pragma unroll
                for (int i = 0; i < V; ++i) d2 = fmaf(v[i] - pivot - mb, v[i] - pivot - mb, d2);
            }
        const float gap = mb - cmean, f = nb / (cn + nb);
        add_kept(cmean, lmean, gap * f);
        add_kept(cm2, lm2, d2 + gap * gap * cn * f);
        cn += nb;
    }
    merge_wave(cn, cmean, cm2);
    const int wave = (int)threadIdx.x >> 6;
    if ((threadIdx.x & 63) == 0) red[wave] = cn, red[WAVES + wave] = cmean, red[2 * WAVES + wave] = cm2;
    __syncthreads();
    cn = red[0], cmean = red[WAVES], cm2 = red[2 * WAVES];
    for (int w = 1; w < WAVES; ++w) merge(cn, cmean, cm2, red[w], red[WAVES + w], red[2 * WAVES + w]);
    __syncthreads();
    return float2{pivot + cmean, cm2 / cn};
}

template <typename IO, int V, int CP, int K, int NT>
__global__ __launch_bounds__(NT) void slab_forward_kernel(Norm s) {
    const NormArgs& a = s.a;
    using P = Piece<IO, V>;
    __shared__ float red[3 * (NT / 64)];
    const int g = (int)(blockIdx.x % (uint32_t)a.groups), tid = (int)threadIdx.x;
    const int row = tid / s.cols, col = tid - row * s.cols;
    const bool on = row < s.rows;
    const int e = g * s.W + (on ? col : 0) * V;
    float gm[CP], be[CP];
    affine<IO>(a, e, gm, be);
    for (int64_t b = blockIdx.x / (uint32_t)a.groups; b < a.batch; b += s.step) {
        int64_t t0, t1;
        sample_range(a, b, t0, t1);
        const int64_t n = t1 - t0;
        const IO* x = (const IO*)a.x + t0 * a.ldx + e;
        IO* y = (IO*)a.y + t0 * a.ldy + e;
        P p[K];
        float v[V], sum = 0.0f, sq = 0.0f;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int64_t t = row + (int64_t)k * s.rows;
            p[k] = on && t < n ? P::load(x + t * a.ldx) : P::zero();
        }
#pragma unroll
        for (int k = 0; k < K; ++k) {
            p[k].get(v);
#pragma unroll
            for (int i = 0; i < V; ++i) sum += v[i];
        }
        if (n > (int64_t)kLong * K * s.rows) [[unlikely]] {
            sum = block_sum<NT>(sum, red) / ((float)(K * s.rows) * (float)s.W);
            const float2 st = long_moments<IO, V, NT>(x, a.ldx, n, row, s.rows, on, sum, red);
            const float mean = st.x, rstd = 1.0f / sqrtf(st.y + a.eps);
            constexpr int U = 4;
            for (int64_t t = on ? row : n; t < n; t += U * s.rows) {
                P q[U];
#pragma unroll
                for (int u = 0; u < U; ++u)
                    q[u] = t + u * s.rows < n ? P::load(x + (t + u * s.rows) * a.ldx) : P::zero();
#pragma unroll
                for (int u = 0; u < U; ++u)
                    if (t + u * s.rows < n) put_y<IO>(a, y + (t + u * s.rows) * a.ldy, q[u], mean, rstd, gm, be);
            }
            if (a.stats && tid == 0)
                *reinterpret_cast<float2*>(a.stats + 2 * (b * a.groups + g)) = float2{mean, rstd};
            continue;
        }
        const int64_t over = on ? row + (int64_t)K * s.rows : n;
        for (int64_t t = over; t < n; t += s.rows) {
            P::load(x + t * a.ldx).get(v);
#pragma unroll
            for (int i = 0; i < V; ++i) sum += v[i];
        }
        const float inv = n ? 1.0f / ((float)n * (float)s.W) : 0.0f;
        const float mean = block_sum<NT>(sum, red) * inv;
#pragma unroll
        for (int k = 0; k < K; ++k)
            if (on && row + (int64_t)k * s.rows < n) {
                p[k].keep_packed();
                p[k].get(v);
#pragma unroll
                for (int i = 0; i < V; ++i) sq = fmaf(v[i] - mean, v[i] - mean, sq);
            }
        for (int64_t t = over; t < n; t += s.rows) {
            P::load(x + t * a.ldx).get(v);
#pragma unroll
            for (int i = 0; i < V; ++i) sq = fmaf(v[i] - mean, v[i] - mean, sq);
        }
        sq = block_sum<NT>(sq, red);
        const float rstd = n ? 1.0f / sqrtf(sq * inv + a.eps) : 0.0f;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int64_t t = row + (int64_t)k * s.rows;
            p[k].keep_packed();
            if (on && t < n) put_y<IO>(a, y + t * a.ldy, p[k], mean, rstd, gm, be);
        }
        for (int64_t t = over; t < n; t += s.rows)
            put_y<IO>(a, y + t * a.ldy, P::load(x + t * a.ldx), mean, rstd, gm, be);
        if (a.stats && tid == 0)
            *reinterpret_cast<float2*>(a.stats + 2 * (b * a.groups + g)) = float2{mean, rstd};
    }
}

// Sums over the rows of a workgroup of each piece's V sums, then over each channel's N
// of them, to out[channel].  acc: NT V floats.
template <int V, int NT>
__device__ __forceinline__ void channel_sums(const float (&v)[V], float* acc, int rows, int cols, int n_channels, int N,
                                             float* out) {
    const int tid = (int)threadIdx.x;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < V; ++i) acc[tid * V + i] = v[i];
    __syncthreads();
    // number e of a row is at [row][e]: pieces of a row lie one after the other
    for (int e = tid; e < cols * V; e += NT) {
        float w = acc[e];
        for (int r = 1; r < rows; ++r) w += acc[r * cols * V + e];
        acc[e] = w;  // row 0: only this thread reads or writes it
    }
    __syncthreads();
    for (int c = tid; c < n_channels; c += NT) {
        float w = acc[c * N];
        for (int n = 1; n < N; ++n) w += acc[c * N + n];
        out[c] = w;
    }
}

template <typename IO, int V, int CP, int K, int NT>
__global__ __launch_bounds__(NT, NT == 1024 ? 4 : 2) void slab_backward_kernel(Norm s) {
    const NormArgs& a = s.a;
    using P = Piece<IO, V>;
    __shared__ float red[NT / 64];
    __shared__ float acc[NT * CP];
    const int g = (int)(blockIdx.x % (uint32_t)a.groups), tid = (int)threadIdx.x;
    const int64_t part = blockIdx.x / (uint32_t)a.groups;
    const int row = tid / s.cols, col = tid - row * s.cols;
    const bool on = row < s.rows;
    const int e = g * s.W + (on ? col : 0) * V;
    float gm[CP], be[CP], dg[CP], db[CP];
    affine<IO>(a, e, gm, be);
#pragma unroll
    for (int i = 0; i < CP; ++i) dg[i] = db[i] = 0.0f;
    for (int64_t b = part; b < a.batch; b += s.step) {
        int64_t t0, t1;
        sample_range(a, b, t0, t1);
        const int64_t n = t1 - t0;
        const IO* x = (const IO*)a.x + t0 * a.ldx + e;
        const IO* dy = (const IO*)a.dy + t0 * a.lddy + e;
        IO* dx = (IO*)a.dx + t0 * a.lddx + e;
        const float2 st = *reinterpret_cast<const float2*>(a.stats + 2 * (b * a.groups + g));
        if (n > (int64_t)kLong * K * s.rows) [[unlikely]] {
            // sums of runs of eight tokens, added with what the additions lose
            float xh[V], dz[V], hg[CP], hb[CP], lg[CP], lb[CP], s1 = 0.0f, s2 = 0.0f;
#pragma unroll
            for (int i = 0; i < CP; ++i) hg[i] = hb[i] = lg[i] = lb[i] = 0.0f;
            for (int64_t t0 = on ? row : n; t0 < n; t0 += 8 * s.rows) {
                float sg[CP], sb[CP];
#pragma unroll
                for (int i = 0; i < CP; ++i) sg[i] = sb[i] = 0.0f;
                for (int64_t t = t0; t < n && t < t0 + 8 * s.rows; t += s.rows) {
                    get_dz<IO>(a, P::load(x + t * a.ldx), P::load(dy + t * a.lddy), st.x, st.y, gm, be, xh, dz);
#pragma unroll
                    for (int i = 0; i < V; ++i) {
                        sg[i % CP] = fmaf(dz[i], xh[i], sg[i % CP]);
                        sb[i % CP] += dz[i];
                    }
                }
#pragma unroll
                for (int i = 0; i < CP; ++i) add_kept(hg[i], lg[i], sg[i]), add_kept(hb[i], lb[i], sb[i]);
            }
#pragma unroll
            for (int i = 0; i < CP; ++i) {
                s1 = fmaf(hb[i], gm[i], s1);
                s2 = fmaf(hg[i], gm[i], s2);
                dg[i] += hg[i];
                db[i] += hb[i];
            }
            const float inv = 1.0f / ((float)n * (float)s.W);
            const float m1 = block_sum<NT>(s1, red) * inv, m2 = block_sum<NT>(s2, red) * inv;
            for (int64_t t = on ? row : n; t < n; t += s.rows) {
                get_dz<IO>(a, P::load(x + t * a.ldx), P::load(dy + t * a.lddy), st.x, st.y, gm, be, xh, dz);
                put_dx<IO>(dx + t * a.lddx, xh, dz, gm, m1, m2, st.y);
            }
            continue;
        }
        P px[K];
        float d[K][V];  // dy, then dz: the slope is the costly part, and taken once
        float xh[V], dz[V], sg[CP], sb[CP];
        {
            P pd[K];
#pragma unroll
            for (int k = 0; k < K; ++k) {
                const int64_t t = row + (int64_t)k * s.rows;
                px[k] = on && t < n ? P::load(x + t * a.ldx) : P::zero();
                pd[k] = on && t < n ? P::load(dy + t * a.lddy) : P::zero();
            }
#pragma unroll
            for (int k = 0; k < K; ++k) pd[k].get(d[k]);
        }
#pragma unroll
        for (int i = 0; i < CP; ++i) sg[i] = sb[i] = 0.0f;
        auto add = [&](const P& xp, const P& dp) {
            get_dz<IO>(a, xp, dp, st.x, st.y, gm, be, xh, dz);
#pragma unroll
            for (int i = 0; i < V; ++i) {
                sg[i % CP] = fmaf(dz[i], xh[i], sg[i % CP]);
                sb[i % CP] += dz[i];
            }
        };
        const int64_t over = on ? row + (int64_t)K * s.rows : n;
#pragma unroll
        for (int k = 0; k < K; ++k) {  // (pieces past the sample have dy = 0 and add nothing)
            __builtin_amdgcn_sched_barrier(0);  // piece by piece: mixed, they take twice the registers
            float z[V];
            px[k].keep_packed();
            px[k].get(xh);
#pragma unroll
            for (int i = 0; i < V; ++i) {
                xh[i] = (xh[i] - st.x) * st.y;
                z[i] = fmaf(xh[i], gm[i % CP], be[i % CP]);
            }
            slope_all(a.act, z, d[k]);
#pragma unroll
            for (int i = 0; i < V; ++i) {
                sg[i % CP] = fmaf(d[k][i], xh[i], sg[i % CP]);
                sb[i % CP] += d[k][i];
            }
        }
        for (int64_t t = over; t < n; t += s.rows) add(P::load(x + t * a.ldx), P::load(dy + t * a.lddy));
        float s1 = 0.0f, s2 = 0.0f;
#pragma unroll
        for (int i = 0; i < CP; ++i) {
            s1 = fmaf(sb[i], gm[i], s1);
            s2 = fmaf(sg[i], gm[i], s2);
            dg[i] += sg[i];
            db[i] += sb[i];
        }
        const float inv = n ? 1.0f / ((float)n * (float)s.W) : 0.0f;
        const float m1 = block_sum<NT>(s1, red) * inv, m2 = block_sum<NT>(s2, red) * inv;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int64_t t = row + (int64_t)k * s.rows;
            px[k].keep_packed();
            __builtin_amdgcn_sched_barrier(0);
            if (on && t < n) {
                px[k].get(xh);
#pragma unroll
                for (int i = 0; i < V; ++i) xh[i] = (xh[i] - st.x) * st.y;
                put_dx<IO>(dx + t * a.lddx, xh, d[k], gm, m1, m2, st.y);
            }
        }
        for (int64_t t = over; t < n; t += s.rows) {
            get_dz<IO>(a, P::load(x + t * a.ldx), P::load(dy + t * a.lddy), st.x, st.y, gm, be, xh, dz);
            put_dx<IO>(dx + t * a.lddx, xh, dz, gm, m1, m2, st.y);
        }
    }
    if (!s.part) return;
    float* to = s.part + part * 2 * a.C + g * s.cpg;
    channel_sums<CP, NT>(dg, acc, s.rows, s.cols, s.cpg, a.N * CP / V, to);
    channel_sums<CP, NT>(db, acc, s.rows, s.cols, s.cpg, a.N * CP / V, to + a.C);
}

// --- split path -----------------------------------------------------------------------
// Sample b owns the blocks from offsets[b] / block + b on (at least as many as it has);
// a workgroup takes one block's part of one group (moments) or of one tile of 256
// pieces of the row, whatever groups they are in (the others).

struct Block {
    int64_t b, t0, t1;
    bool idle;
};

__device__ __forceinline__ Block block_of(const Norm& s, int64_t slot) {
    const NormArgs& a = s.a;
    Block k;
    int64_t first;
    if (!a.offsets) {
        const int64_t n = a.T / a.batch, per = (n + s.block - 1) / s.block;
        k.b = slot / per;
        first = k.b * per;
    } else {
        int64_t lo = 0, hi = a.batch - 1;
        while (lo < hi) {
            const int64_t mid = (lo + hi + 1) / 2;
            int64_t o = a.offsets[mid];
            o = o < 0 ? 0 : (o > a.T ? a.T : o);
            if (o / s.block + mid <= slot) lo = mid;
            else hi = mid - 1;
        }
        k.b = lo;
        int64_t o = a.offsets[lo];
        o = o < 0 ? 0 : (o > a.T ? a.T : o);
        first = o / s.block + lo;
    }
    int64_t q0, q1;
    sample_range(a, k.b, q0, q1);
    k.t0 = q0 + (slot - first) * s.block;
    k.t1 = k.t0 + s.block < q1 ? k.t0 + s.block : q1;
    k.idle = slot < first || k.t0 >= q1;
    return k;
}

// blocks of sample b: the first, and how many
__device__ __forceinline__ void blocks_of(const Norm& s, int64_t b, int64_t& first, int64_t& count, int64_t& n) {
    int64_t t0, t1;
    sample_range(s.a, b, t0, t1);
    n = t1 - t0;
    count = (n + s.block - 1) / s.block;
    first = s.a.offsets ? t0 / s.block + b : b * count;
}

// One workgroup per (block of tokens, group): mean and squared differences.
template <typename IO, int V>
__global__ __launch_bounds__(256) void moments_kernel(Norm s) {
    constexpr int BATCH = 8;  // pieces in flight and averaged at once
    const NormArgs& a = s.a;
    using P = Piece<IO, V>;
    __shared__ float red[3][4];
    const uint32_t wg = blockIdx.x + s.base;
    const int tid = (int)threadIdx.x, g = (int)(wg % (uint32_t)a.groups);
    const int64_t slot = wg / (uint32_t)a.groups;
    const Block k = block_of(s, slot);
    if (k.idle) return;
    const IO* x = (const IO*)a.x + k.t0 * a.ldx + g * s.W;
    // pieces of the block, row by row
    const int total = (int)(k.t1 - k.t0) * s.cols;
    float n = 0.0f, mean = 0.0f, m2 = 0.0f;
    int r = tid / s.cols, c = tid - r * s.cols;
    const int dr = 256 / s.cols, dc = 256 - dr * s.cols;
    for (int i0 = tid; i0 < total; i0 += 256 * BATCH) {
        P p[BATCH];
#pragma unroll
        for (int u = 0; u < BATCH; ++u) {
            p[u] = i0 + 256 * u < total ? P::load(x + r * a.ldx + c * V) : P::zero();
            r += dr;
            c += dc;
            if (c >= s.cols) c -= s.cols, ++r;
        }
        float v[V], sum = 0.0f, sq = 0.0f;
        int left = (total - i0 + 255) / 256;
        left = left < BATCH ? left : BATCH;
#pragma unroll
        for (int u = 0; u < BATCH; ++u) {
            p[u].get(v);
#pragma unroll
            for (int i = 0; i < V; ++i) sum += v[i];
        }
        const float nb = (float)(left * V), mb = sum / nb;
#pragma unroll
        for (int u = 0; u < BATCH; ++u)
            if (u < left) {
                p[u].get(v);
#pragma unroll
                for (int i = 0; i < V; ++i) sq = fmaf(v[i] - mb, v[i] - mb, sq);
            }
        merge(n, mean, m2, nb, mb, sq);
    }
    merge_wave(n, mean, m2);
    const int wave = tid >> 6;
    if ((tid & 63) == 0) red[0][wave] = n, red[1][wave] = mean, red[2][wave] = m2;
    __syncthreads();
    if (tid == 0) {
        for (int w = 1; w < 4; ++w) merge(n, mean, m2, red[0][w], red[1][w], red[2][w]);
        *reinterpret_cast<float2*>(s.moments + 2 * (int64_t)wg) = float2{mean, m2};
    }
}

// One wave per slab: the blocks' moments to mean and 1/sqrt(var + eps).
__global__ __launch_bounds__(64) void join_moments_kernel(Norm s) {
    const NormArgs& a = s.a;
    const uint32_t wg = blockIdx.x + s.base;
    const int64_t b = wg / (uint32_t)a.groups;
    const int g = (int)(wg % (uint32_t)a.groups), lane = (int)threadIdx.x;
    int64_t first, count, tokens;
    blocks_of(s, b, first, count, tokens);
    float n = 0.0f, mean = 0.0f, m2 = 0.0f;
    for (int64_t k = lane; k < count; k += 64) {
        const float2 m = *reinterpret_cast<const float2*>(s.moments + 2 * ((first + k) * a.groups + g));
        const int64_t left = tokens - k * s.block;
        merge(n, mean, m2, (float)(left < s.block ? left : s.block) * (float)s.W, m.x, m.y);
    }
    merge_wave(n, mean, m2);
    if (lane == 0) {
        const float2 r = n > 0.0f ? float2{mean, 1.0f / sqrtf(m2 / n + a.eps)} : float2{0.0f, 0.0f};
        *reinterpret_cast<float2*>(s.joined + 2 * (int64_t)wg) = r;
        if (a.stats) *reinterpret_cast<float2*>(a.stats + 2 * (int64_t)wg) = r;
    }
}

// The largest power of two below n (n > 1), else 0
__device__ __forceinline__ int half_of(int n) { return n > 1 ? 1 << (31 - __builtin_clz(n - 1)) : 0; }

// Tile of columns of the row kernels: 256 pieces from blockIdx.y 256 on; rows of the
// workgroup when a row is narrower than that.
template <typename IO, int V>
struct RowTile {
    int cols, rows, row, e, g;
    bool on;
    __device__ __forceinline__ RowTile(const Norm& s) {
        const int all = s.W / V * s.a.groups, c0 = (int)blockIdx.y * 256;
        cols = all - c0 < 256 ? all - c0 : 256;
        rows = 256 / cols;
        row = (int)threadIdx.x / cols;
        const int c = (int)threadIdx.x - row * cols;
        on = row < rows;
        e = (c0 + (on ? c : 0)) * V;
        g = e / s.W;
    }
};

template <typename IO, int V>
__global__ __launch_bounds__(256) void apply_forward_kernel(Norm s) {
    constexpr int U = 4;
    const NormArgs& a = s.a;
    using P = Piece<IO, V>;
    const Block k = block_of(s, blockIdx.x + s.base);
    if (k.idle) return;
    const RowTile<IO, V> rt(s);
    if (!rt.on) return;
    float gm[V], be[V];
    affine<IO>(a, rt.e, gm, be);
    const float2 st = *reinterpret_cast<const float2*>(s.joined + 2 * (k.b * a.groups + rt.g));
    const IO* x = (const IO*)a.x + rt.e;
    IO* y = (IO*)a.y + rt.e;
    for (int64_t t = k.t0 + rt.row; t < k.t1; t += U * rt.rows) {
        P p[U];
#pragma unroll
        for (int u = 0; u < U; ++u)
            p[u] = t + u * rt.rows < k.t1 ? P::load(x + (t + u * rt.rows) * a.ldx) : P::zero();
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (t + u * rt.rows < k.t1) put_y<IO>(a, y + (t + u * rt.rows) * a.ldy, p[u], st.x, st.y, gm, be);
    }
}

// Sums of gamma dz and gamma dz xh over each block's tokens, per group: sums[slot][tile +
// group] (a tile of columns and a group meet in one run, and the next run is in the next tile or
// the next group).  A workgroup walks the blocks blockIdx.x, blockIdx.x + gridDim.x, ... and
// keeps the sums of dz xh and dz over all of them, per number (a tile may end inside a channel;
// the join adds the N of a channel): part[blockIdx.x], as many as there are workgroups and not
// as there are blocks, of which short samples make one each.
template <typename IO, int V>
__global__ __launch_bounds__(256) void sums_kernel(Norm s) {
    constexpr int U = 4;
    const NormArgs& a = s.a;
    using P = Piece<IO, V>;
    __shared__ float acc[256 * V];
    __shared__ float red[2][256];
    const RowTile<IO, V> rt(s);
    const int tid = (int)threadIdx.x, col = tid - rt.row * rt.cols;
    // this thread's run of pieces: its place in it, and the run's length
    const int c0 = (int)blockIdx.y * 256, from = rt.g * s.cols - c0 > 0 ? rt.g * s.cols - c0 : 0;
    const int end = (rt.g + 1) * s.cols - c0 < rt.cols ? (rt.g + 1) * s.cols - c0 : rt.cols;
    const int pos = col - from, len = end - from, longest = s.cols < rt.cols ? s.cols : rt.cols;
    const int64_t runs = (int64_t)gridDim.y + a.groups;
    float gm[V], be[V], dg[V], db[V], xh[V], dz[V];
    affine<IO>(a, rt.e, gm, be);
#pragma unroll
    for (int i = 0; i < V; ++i) dg[i] = db[i] = 0.0f;
    for (int64_t slot = blockIdx.x; slot < s.slots; slot += gridDim.x) {
        const Block k = block_of(s, slot);
        if (k.idle) continue;
        float s1 = 0.0f, s2 = 0.0f;
        if (rt.on) {
            const float2 st = *reinterpret_cast<const float2*>(a.stats + 2 * (k.b * a.groups + rt.g));
            const IO* x = (const IO*)a.x + rt.e;
            const IO* dy = (const IO*)a.dy + rt.e;
            float sg[V], sb[V];
#pragma unroll
            for (int i = 0; i < V; ++i) sg[i] = sb[i] = 0.0f;
            for (int64_t t = k.t0 + rt.row; t < k.t1; t += U * rt.rows) {
                P px[U], pd[U];
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const bool in = t + u * rt.rows < k.t1;
                    px[u] = in ? P::load(x + (t + u * rt.rows) * a.ldx) : P::zero();
                    pd[u] = in ? P::load(dy + (t + u * rt.rows) * a.lddy) : P::zero();
                }
#pragma unroll
                for (int u = 0; u < U; ++u)
                    if (t + u * rt.rows < k.t1) {
                        get_dz<IO>(a, px[u], pd[u], st.x, st.y, gm, be, xh, dz);
#pragma unroll
                        for (int i = 0; i < V; ++i) {
                            sg[i] = fmaf(dz[i], xh[i], sg[i]);
                            sb[i] += dz[i];
                        }
                    }
            }
#pragma unroll
            for (int i = 0; i < V; ++i) {
                dg[i] += sg[i], db[i] += sb[i];
                s1 = fmaf(sb[i], gm[i], s1);
                s2 = fmaf(sg[i], gm[i], s2);
            }
        }
        // over the rows, then over each run, by halves
        __syncthreads();
        red[0][tid] = s1, red[1][tid] = s2;
        __syncthreads();
        for (int o = half_of(rt.rows); o > 0; o >>= 1) {
            if (rt.row < o && rt.row + o < rt.rows)
                red[0][tid] += red[0][tid + o * rt.cols], red[1][tid] += red[1][tid + o * rt.cols];
            __syncthreads();
        }
        for (int o = half_of(longest); o > 0; o >>= 1) {
            if (rt.row == 0 && pos < o && pos + o < len)
                red[0][tid] += red[0][tid + o], red[1][tid] += red[1][tid + o];
            __syncthreads();
        }
        if (rt.row == 0 && pos == 0)
            *reinterpret_cast<float2*>(s.sums + 2 * (slot * runs + blockIdx.y + rt.g)) = float2{red[0][tid], red[1][tid]};
    }
    const int64_t width = (int64_t)s.W * a.groups;
    float* to = s.part + (int64_t)blockIdx.x * 2 * width + (int64_t)blockIdx.y * 256 * V;
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        __syncthreads();
#pragma unroll
        for (int i = 0; i < V; ++i) acc[tid * V + i] = q == 0 ? dg[i] : db[i];
        __syncthreads();
        for (int e = tid; e < rt.cols * V; e += 256) {
            float w = acc[e];
            for (int r = 1; r < rt.rows; ++r) w += acc[r * rt.cols * V + e];
            to[q * width + e] = w;
        }
    }
}

// One wave per slab: m1 and m2 from its blocks' sums.
__global__ __launch_bounds__(64) void join_sums_kernel(Norm s) {
    const NormArgs& a = s.a;
    const uint32_t wg = blockIdx.x + s.base;
    const int64_t b = wg / (uint32_t)a.groups;
    const int g = (int)(wg % (uint32_t)a.groups);
    int64_t first, count, n;
    blocks_of(s, b, first, count, n);
    const int64_t tiles = ((int64_t)s.cols * a.groups + 255) / 256, runs = tiles + a.groups;
    const int64_t y0 = (int64_t)g * s.cols / 256, ny = ((int64_t)(g + 1) * s.cols - 1) / 256 - y0 + 1;
    float s1 = 0.0f, s2 = 0.0f;
    for (int64_t i = threadIdx.x; i < count * ny; i += 64) {
        const int64_t k = i / ny;
        const float2 v = *reinterpret_cast<const float2*>(s.sums + 2 * ((first + k) * runs + y0 + (i - k * ny) + g));
        s1 += v.x;
        s2 += v.y;
    }
    s1 = lane_sum(s1, 64);
    s2 = lane_sum(s2, 64);
    if (threadIdx.x == 0) {
        const float inv = n ? 1.0f / ((float)n * (float)s.W) : 0.0f;
        *reinterpret_cast<float2*>(s.joined + 2 * (int64_t)wg) = float2{s1 * inv, s2 * inv};
    }
}

template <typename IO, int V>
__global__ __launch_bounds__(256) void apply_backward_kernel(Norm s) {
    constexpr int U = 4;
    const NormArgs& a = s.a;
    using P = Piece<IO, V>;
    const Block k = block_of(s, blockIdx.x + s.base);
    if (k.idle) return;
    const RowTile<IO, V> rt(s);
    if (!rt.on) return;
    float gm[V], be[V], xh[V], dz[V];
    affine<IO>(a, rt.e, gm, be);
    const int64_t slab = k.b * a.groups + rt.g;
    const float2 st = *reinterpret_cast<const float2*>(a.stats + 2 * slab);
    const float2 m = *reinterpret_cast<const float2*>(s.joined + 2 * slab);
    const IO* x = (const IO*)a.x + rt.e;
    const IO* dy = (const IO*)a.dy + rt.e;
    IO* dx = (IO*)a.dx + rt.e;
    for (int64_t t = k.t0 + rt.row; t < k.t1; t += U * rt.rows) {
        P px[U], pd[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const bool in = t + u * rt.rows < k.t1;
            px[u] = in ? P::load(x + (t + u * rt.rows) * a.ldx) : P::zero();
            pd[u] = in ? P::load(dy + (t + u * rt.rows) * a.lddy) : P::zero();
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (t + u * rt.rows < k.t1) {
                get_dz<IO>(a, px[u], pd[u], st.x, st.y, gm, be, xh, dz);
                put_dx<IO>(dx + (t + u * rt.rows) * a.lddx, xh, dz, gm, m.x, m.y, st.y);
            }
    }
}

// dgamma and dbeta: sums over parts [n][2][C per], per numbers of a channel added.  32
// channels per workgroup, 32 threads each; blockIdx.y: 0 dgamma, 1 dbeta.
__global__ __launch_bounds__(1024) void param_sums_kernel(const float* part, int64_t n, int C, int per, float* dgamma,
                                                          float* dbeta) {
    __shared__ float acc[32][33];
    const int lc = (int)threadIdx.x & 31, r = (int)threadIdx.x >> 5, c = (int)blockIdx.x * 32 + lc;
    float* to = blockIdx.y ? dbeta : dgamma;
    if (!to) return;
    const int64_t width = (int64_t)C * per;
    const float* p = part + blockIdx.y * width + (int64_t)c * per;
    float v = 0.0f;
    if (c < C)
        for (int i = 0; i < per; ++i) {
#pragma unroll 8
            for (int64_t k = r; k < n; k += 32) v += p[k * 2 * width + i];
        }
    acc[r][lc] = v;
    for (int o = 16; o > 0; o >>= 1) {
        __syncthreads();
        if (r < o) acc[r][lc] += acc[r + o][lc];
    }
    if (r == 0 && c < C) to[c] = acc[0][lc];
}

__global__ __launch_bounds__(256) void empty_stats_kernel(float* p, int64_t n, uint32_t base) {
    const int64_t i = (int64_t)(blockIdx.x + base) * 256 + threadIdx.x;
    if (i < n) p[i] = 0.0f;
}

// --- host side ------------------------------------------------------------------------

enum Path { kToken, kSlab, kSplit };

// Token path: up to here every workgroup may keep sums of all channels.
constexpr int64_t kStraddleBytes = (int64_t)16 << 20;

struct Choice {
    Path path;
    int V, cols;
    int lps, K, NT, rows;
    int64_t wgs, step;     // token, slab paths
    int64_t parts;         // sums of dgamma and dbeta
    int pg, unit;          // token path
    int64_t block, slots;  // split path
    size_t part, sums, total;  // workspace bytes: of those sums, of the split path's, in all
};

int64_t round_up(int64_t a, int64_t b) { return (a + b - 1) / b * b; }
int gcd(int a, int b) { return b ? gcd(b, a % b) : a; }

// The smallest workgroup of the slab path whose registers hold a sample of `mean`
// tokens, K pieces a thread; false: none.  The backward holds x and dz, half the pieces
// at the largest, and at CP = 1 spreads about 3000 pieces over 1024 threads, which
// compile to under 128 registers: 30 us for 64 images of 197 x 96 x 8 (bf16, GELU) where
// 6 each on 512 threads took 46.  Where a piece crosses channels the sums take registers
// too, and the same step spills: 59 us against 39 at 64 x 300 x 96 x 6; so does K = 4.
bool slab_shape(Choice& c, int64_t mean, bool backward, bool one) {
    const int forward[6][2] = {{2, 64}, {8, 64}, {4, 256}, {8, 256}, {6, 512}, {16, 512}};
    const int wide[6][2] = {{2, 64}, {8, 64}, {4, 256}, {8, 256}, {3, 1024}, {8, 512}};
    const int crossing[6][2] = {{2, 64}, {8, 64}, {4, 256}, {8, 256}, {6, 512}, {8, 512}};
    for (const auto& k : backward ? (one ? wide : crossing) : forward)
        if (c.cols <= k[1] && mean <= (int64_t)k[0] * (k[1] / c.cols)) {
            c.K = k[0];
            c.NT = k[1];
            return true;
        }
    return false;
}

// The path by sizes alone (lengths of packed samples are on the device: their mean
// stands for them).  V: numbers per piece.  T > 0.
Choice choose(int V, int C, int N, int groups, int64_t T, int64_t batch, bool ragged, bool backward) {
    Choice c{};
    const int W = C / groups * N;
    c.V = V;
    c.cols = W / V;
    const int64_t mean = (T + batch - 1) / batch;
    if (!ragged && batch == T && c.cols <= 256) {
        c.path = kToken;
        c.lps = 1;
        while (c.lps < c.cols && c.lps < 64) c.lps *= 2;
        c.K = 1;
        while (c.K * c.lps < c.cols) c.K *= 2;
        // slabs of a workgroup; the workgroups step by whole tokens.  Groups that do not divide
        // into them so that few workgroups are a step are padded: one token of 8191 groups
        // would take 8191 workgroups
        const int per = 4 * (64 / c.lps), cap = backward ? 1024 : 2048;
        c.pg = groups;
        int step = groups / gcd(groups, per);
        if (groups % per && (step > 16 || (int64_t)(cap + step) * C * 8 > kStraddleBytes)) {
            c.pg = (int)round_up(groups, groups > per ? per : (per + 15) / 16);
            step = c.pg / gcd(c.pg, per);
        }
        c.unit = c.pg % per == 0 ? step : 0;
        const int64_t want = (T * c.pg + per - 1) / per;
        c.wgs = round_up(want < cap ? want : cap, step);
        c.step = c.wgs * per / c.pg;
        c.parts = c.unit ? c.wgs / c.unit : c.wgs;
        c.part = backward ? (size_t)c.parts * 2 * C * 4 : 0;
    } else if (slab_shape(c, mean, backward, N % V == 0) && (c.K <= 8 || batch * groups >= 128)) {
        c.path = kSlab;
        c.rows = c.NT / c.cols;
        const int64_t cap = (backward ? 2048 : 8192) / groups;
        c.step = batch < cap ? batch : (cap < 1 ? 1 : cap);
        c.wgs = c.step * groups;
        c.parts = c.step;
        c.part = backward ? (size_t)c.step * 2 * C * 4 : 0;
    } else {
        c.path = kSplit;
        // about two blocks per CU, of at least 16 tokens
        const int64_t b = (T + 511) / 512;
        c.block = b < 16 ? 16 : b;
        c.slots = T / c.block + batch;
        // about four workgroups per CU keep sums of dgamma and dbeta
        const int64_t tiles = ((int64_t)c.cols * groups + 255) / 256, walkers = 1024 / tiles < 1 ? 1 : 1024 / tiles;
        c.parts = c.slots < walkers ? c.slots : walkers;
        c.part = backward ? (size_t)c.parts * 2 * C * N * 4 : 0;
        c.sums = (size_t)c.slots * (backward ? tiles + groups : groups) * 2 * 4;
        c.total = (size_t)batch * groups * 2 * 4;
    }
    c.part = (size_t)round_up((int64_t)c.part, 256);
    c.sums = (size_t)round_up((int64_t)c.sums, 256);
    c.total = c.part + c.sums + (size_t)round_up((int64_t)c.total, 256);
    return c;
}

int full_piece(int io) { return io == kIoF32 ? 4 : 8; }

bool wide_ok(int io, const void* p, int64_t ld, int W) {
    const int V = full_piece(io);
    return W % V == 0 && ld % V == 0 && ((uintptr_t)p & 15u) == 0;
}

Norm norm_of(const NormArgs& a, const Choice& c, void* ws, bool backward) {
    Norm s{};
    s.a = a;
    s.cpg = a.C / a.groups;
    s.W = s.cpg * a.N;
    s.cols = c.cols;
    s.lps = c.lps;
    s.rows = c.rows;
    s.step = c.step;
    s.block = c.block;
    s.slots = !a.offsets && c.path == kSplit ? a.batch * ((a.T / a.batch + c.block - 1) / c.block) : c.slots;
    s.pg = c.pg;
    s.unit = c.unit;
    char* w = static_cast<char*>(ws);
    s.part = reinterpret_cast<float*>(w);
    s.moments = s.sums = reinterpret_cast<float*>(w + c.part);
    s.joined = reinterpret_cast<float*>(w + c.part + c.sums);
    return s;
}

template <typename IO, int V, int CP>
hipError_t forward_v(const NormArgs& a, void* ws, hipStream_t stream) {
    const Choice c = choose(V, a.C, a.N, a.groups, a.T, a.batch, a.offsets != nullptr, false);
    Norm s = norm_of(a, c, ws, false);
    if (c.path == kToken) {
        if (c.wgs > 0x7fffffff) return hipErrorNotSupported;
        const dim3 grid((uint32_t)c.wgs);
        switch (c.K) {
            case 1: hipLaunchKernelGGL((token_forward_kernel<IO, V, CP, 1>), grid, dim3(256), 0, stream, s); break;
            case 2: hipLaunchKernelGGL((token_forward_kernel<IO, V, CP, 2>), grid, dim3(256), 0, stream, s); break;
            default: hipLaunchKernelGGL((token_forward_kernel<IO, V, CP, 4>), grid, dim3(256), 0, stream, s);
        }
    } else if (c.path == kSlab) {
        if (c.wgs > 0x7fffffff) return hipErrorNotSupported;
        const dim3 grid((uint32_t)c.wgs);
#define EQL_SLAB(k, nt)                                                                                       \
    if (c.K == k && c.NT == nt)                                                                                \
        hipLaunchKernelGGL((slab_forward_kernel<IO, V, CP, k, nt>), grid, dim3(nt), 0, stream, s);
        EQL_SLAB(2, 64) EQL_SLAB(8, 64) EQL_SLAB(4, 256) EQL_SLAB(8, 256) EQL_SLAB(6, 512) EQL_SLAB(16, 512)
#undef EQL_SLAB
    } else {
        const int64_t tiles = ((int64_t)c.cols * a.groups + 255) / 256;
        if (s.slots * a.groups > 0x7fffffff || a.batch * a.groups > 0x7fffffff || tiles > 65535 ||
            c.block * (int64_t)c.cols > 0x3fffffff)
            return hipErrorNotSupported;
        in_pieces(s.slots * a.groups, 256, [&](uint32_t base, uint32_t n) {
            s.base = base;
            hipLaunchKernelGGL((moments_kernel<IO, V>), dim3(n), dim3(256), 0, stream, s);
        });
        in_pieces(a.batch * a.groups, 64, [&](uint32_t base, uint32_t n) {
            s.base = base;
            hipLaunchKernelGGL(join_moments_kernel, dim3(n), dim3(64), 0, stream, s);
        });
        in_pieces(s.slots, 256, [&](uint32_t base, uint32_t n) {
            s.base = base;
            hipLaunchKernelGGL((apply_forward_kernel<IO, V>), dim3(n, (uint32_t)tiles), dim3(256), 0, stream, s);
        });
    }
    return hipGetLastError();
}

template <typename IO, int V, int CP>
hipError_t backward_v(const NormArgs& a, void* ws, hipStream_t stream) {
    const Choice c = choose(V, a.C, a.N, a.groups, a.T, a.batch, a.offsets != nullptr, true);
    Norm s = norm_of(a, c, ws, true);
    const bool params = a.dgamma || a.dbeta;
    const dim3 pgrid((uint32_t)((a.C + 31) / 32), 2);
    int64_t parts = c.parts;
    int per = 1;
    if (c.path == kToken) {
        if (!params) s.part = nullptr;
        if (c.wgs > 0x7fffffff) return hipErrorNotSupported;
        const dim3 grid((uint32_t)c.wgs);
        switch (c.K) {
            case 1: hipLaunchKernelGGL((token_backward_kernel<IO, V, CP, 1>), grid, dim3(256), 0, stream, s); break;
            case 2: hipLaunchKernelGGL((token_backward_kernel<IO, V, CP, 2>), grid, dim3(256), 0, stream, s); break;
            default: hipLaunchKernelGGL((token_backward_kernel<IO, V, CP, 4>), grid, dim3(256), 0, stream, s);
        }
    } else if (c.path == kSlab) {
        if (!params) s.part = nullptr;
        if (c.wgs > 0x7fffffff) return hipErrorNotSupported;
        const dim3 grid((uint32_t)c.wgs);
#define EQL_SLAB(k, nt)                                                                                       \
    if (c.K == k && c.NT == nt)                                                                                \
        hipLaunchKernelGGL((slab_backward_kernel<IO, V, CP, k, nt>), grid, dim3(nt), 0, stream, s);
        EQL_SLAB(2, 64) EQL_SLAB(8, 64) EQL_SLAB(4, 256) EQL_SLAB(8, 256)
        if constexpr (CP == 1) { EQL_SLAB(3, 1024) }
        if constexpr (CP > 1) { EQL_SLAB(6, 512) }
        EQL_SLAB(8, 512)
#undef EQL_SLAB
    } else {
        const int64_t tiles = ((int64_t)c.cols * a.groups + 255) / 256;
        if (s.slots > 0x7fffffff || a.batch * a.groups > 0x7fffffff || tiles > 65535) return hipErrorNotSupported;
        const int64_t walkers = s.slots < c.parts ? s.slots : c.parts;
        hipLaunchKernelGGL((sums_kernel<IO, V>), dim3((uint32_t)walkers, (uint32_t)tiles), dim3(256), 0, stream, s);
        in_pieces(a.batch * a.groups, 64, [&](uint32_t base, uint32_t n) {
            s.base = base;
            hipLaunchKernelGGL(join_sums_kernel, dim3(n), dim3(64), 0, stream, s);
        });
        in_pieces(s.slots, 256, [&](uint32_t base, uint32_t n) {
            s.base = base;
            hipLaunchKernelGGL((apply_backward_kernel<IO, V>), dim3(n, (uint32_t)tiles), dim3(256), 0, stream, s);
        });
        parts = walkers;
        per = a.N;
    }
    if (params)
        hipLaunchKernelGGL(param_sums_kernel, pgrid, dim3(1024), 0, stream, s.part, parts, a.C, per, a.dgamma, a.dbeta);
    return hipGetLastError();
}

template <typename IO>
hipError_t forward(int io, const NormArgs& a, void* ws, hipStream_t stream) {
    constexpr int V = 16 / sizeof(IO);
    const int W = a.C / a.groups * a.N;
    if (wide_ok(io, a.x, a.ldx, W) && wide_ok(io, a.y, a.ldy, W))
        return a.N % V == 0 ? forward_v<IO, V, 1>(a, ws, stream) : forward_v<IO, V, V>(a, ws, stream);
    return forward_v<IO, 1, 1>(a, ws, stream);
}

template <typename IO>
hipError_t backward(int io, const NormArgs& a, void* ws, hipStream_t stream) {
    constexpr int V = 16 / sizeof(IO);
    const int W = a.C / a.groups * a.N;
    if (wide_ok(io, a.x, a.ldx, W) && wide_ok(io, a.dy, a.lddy, W) && wide_ok(io, a.dx, a.lddx, W))
        return a.N % V == 0 ? backward_v<IO, V, 1>(a, ws, stream) : backward_v<IO, V, V>(a, ws, stream);
    return backward_v<IO, 1, 1>(a, ws, stream);
}

}  // namespace

size_t group_norm_workspace(int io, int C, int N, int groups, int64_t T, int64_t batch, bool backward) {
    if (T <= 0 || batch <= 0) return 0;
    size_t most = 0;
    const int W = C / groups * N, V = full_piece(io);
    for (int back = 0; back <= (backward ? 1 : 0); ++back)
        for (int ragged = 0; ragged < 2; ++ragged)
            for (int v : {1, V}) {
                if (W % v) continue;
                const Choice c = choose(v, C, N, groups, T, batch, ragged != 0, back != 0);
                const size_t n = back == 0 && c.path != kSplit ? 0 : c.total;
                most = n > most ? n : most;
            }
    return most;
}

hipError_t launch_group_norm(int io, const NormArgs& a, void* ws, hipStream_t stream) {
    if (a.T == 0) {  // empty samples alone
        const int64_t n = a.batch * a.groups * 2;
        if ((n + 255) / 256 > 0x7fffffff) return hipErrorNotSupported;
        in_pieces((n + 255) / 256, 256, [&](uint32_t base, uint32_t wgs) {
            hipLaunchKernelGGL(empty_stats_kernel, dim3(wgs), dim3(256), 0, stream, a.stats, n, base);
        });
        return hipGetLastError();
    }
    return io == kIoF32 ? forward<float>(io, a, ws, stream)
                        : (io == kIoBF16 ? forward<__bf16>(io, a, ws, stream) : forward<_Float16>(io, a, ws, stream));
}

hipError_t launch_group_norm_backward(int io, const NormArgs& a, void* ws, hipStream_t stream) {
    if (a.T == 0) {
        const dim3 grid((uint32_t)((a.C + 31) / 32), 2);
        hipLaunchKernelGGL(param_sums_kernel, grid, dim3(1024), 0, stream, nullptr, 0, a.C, 1, a.dgamma, a.dbeta);
        return hipGetLastError();
    }
    return io == kIoF32 ? backward<float>(io, a, ws, stream)
                        : (io == kIoBF16 ? backward<__bf16>(io, a, ws, stream) : backward<_Float16>(io, a, ws, stream));
}

}  // namespace eql
