// tiles.h -- operands of the matrix cores, tiles in LDS and the loads that fill them, for
// the kernels that contract over tokens (linear_attention.h, attention.h).
#pragma once

#include "cn_fused.h"  // make_rsrc, kOOB
#include "eq_device.h"
#include "eq_launch.h"

namespace eql {
namespace tile {

// --- matrix-core operands of the three types ----------------------------------------
// A fragment holds, in each lane, KF numbers along the contraction: KS over the four
// lane groups kg = lane / 16, at row (column) lane % 16 of the operand; group kg has
// positions KF kg .. KF kg + KF - 1: in a row-major tile one 16-byte piece.

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));

template <typename IO>
struct Op {  // __bf16, _Float16
    using F = typename Half<IO>::x8;
    static constexpr int KS = 32, KF = 8, ES = 2;
    static constexpr bool BF = std::is_same_v<IO, __bf16>;
    // terms in which an fp32 number of the middle of IO's range enters a product: 24 bits of
    // it (bf16) or 21 to 22 (fp16)
    static constexpr int TERMS = BF ? 3 : 2;
    static __device__ __forceinline__ void mma(f32x4& acc, const F& a, const F& b) {
        if constexpr (BF) acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, acc, 0, 0, 0);
        else acc = __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, acc, 0, 0, 0);
    }
    // Two transposed reads: 4 rows x 4 runs of 4 columns from each group of 16 lanes (lane
    // 4r + u points at row r, run u) to lane 4u + v: column v of run u.  lo: rows 8 kg +
    // 0..3 of the contraction, hi: 8 kg + 4..7.
    static __device__ __forceinline__ F column(const char* lo, const char* hi) {
        const s16x4 x = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(lo));
        const s16x4 y = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(hi));
        return __builtin_bit_cast(F, __builtin_shufflevector(x, y, 0, 1, 2, 3, 4, 5, 6, 7));
    }
    static __device__ __forceinline__ float get(const F& f, int e) { return (float)f[e]; }
    // infinities and NaN as 0 (or, rest, all else)
    static __device__ __forceinline__ F finite(F f, bool rest = false) {
#pragma unroll
        for (int e = 0; e < KF; ++e) f[e] = (fabsf((float)f[e]) < __builtin_inff()) != rest ? f[e] : (IO)0.0f;
        return f;
    }
    // v (8 numbers) as N fragments, each what the ones before left, cut off (not rounded: the
    // next term holds the rest exactly).  Three bf16 terms hold all 24 bits; two fp16 terms hold
    // 22 of a number of 2^-3 or more, below that its bits down to 2^-24: hence kColumnLow, kValueLow
    template <int N>
    static __device__ __forceinline__ void split(const float (&v)[8], F (&out)[N]) {
        float r[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) r[e] = v[e];
#pragma unroll
        for (int t = 0; t < N; ++t) {
            u32x4 u;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                float& x = r[2 * q];
                float& y = r[2 * q + 1];
                if constexpr (BF) {
                    u[q] = __builtin_amdgcn_perm(__float_as_uint(y), __float_as_uint(x), 0x07060302u);
                    if (t + 1 < N) {
                        x -= __uint_as_float(__float_as_uint(x) & 0xffff0000u);
                        y -= __uint_as_float(__float_as_uint(y) & 0xffff0000u);
                    }
                } else {
                    u[q] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_pkrtz(x, y));
                    if (t + 1 < N) {
                        x -= Half<IO>::lo(u[q]);
                        y -= Half<IO>::hi(u[q]);
                    }
                }
            }
            out[t] = __builtin_bit_cast(F, u);
        }
    }
    // the largest |number| of N fragments, its 16 bits (kInf or more: an infinity or a NaN)
    static constexpr uint32_t kInf = BF ? 0x7f80 : 0x7c00;
    template <int N>
    static __device__ __forceinline__ uint32_t top(const F (&f)[N]) {
        u16x2 m = {0, 0};
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const u32x4 v = __builtin_bit_cast(u32x4, f[i]);
#pragma unroll
            for (int q = 0; q < 4; ++q) m = __builtin_elementwise_max(m, __builtin_bit_cast(u16x2, v[q] & 0x7fff7fffu));
        }
        return m[0] > m[1] ? m[0] : m[1];
    }
};

template <>
struct Op<float> {
    using F = f32x4;
    static constexpr int KS = 16, KF = 4, ES = 4, TERMS = 1;
    static constexpr bool BF = false;
    static __device__ __forceinline__ void mma(f32x4& acc, const F& a, const F& b) {
#pragma unroll
        for (int e = 0; e < 4; ++e) acc = __builtin_amdgcn_mfma_f32_16x16x4f32(a[e], b[e], acc, 0, 0, 0);
    }
    static __device__ __forceinline__ float get(const F& f, int e) { return f[e]; }
    static __device__ __forceinline__ F finite(F f, bool rest = false) {
#pragma unroll
        for (int e = 0; e < KF; ++e) f[e] = (fabsf(f[e]) < __builtin_inff()) != rest ? f[e] : 0.0f;
        return f;
    }
    template <int N>
    static __device__ __forceinline__ void split(const float (&v)[4], F (&out)[N]) {
        out[0] = F{v[0], v[1], v[2], v[3]};
    }
    // 1 if a fragment holds an infinity or a NaN
    static constexpr uint32_t kInf = 1;
    template <int N>
    static __device__ __forceinline__ uint32_t top(const F (&f)[N]) {
        bool odd = false;
#pragma unroll
        for (int i = 0; i < N; ++i)
#pragma unroll
            for (int e = 0; e < KF; ++e) odd |= !(fabsf(f[i][e]) < __builtin_inff());
        return odd;
    }
};

// One 16-byte piece of a row of any alignment: columns col .. of D, zeros past D.
template <typename IO>
__device__ __forceinline__ u32x4 load_piece(const IO* row, int col, int D) {
    constexpr int E = 16 / (int)sizeof(IO);
    u32x4 v = {0u, 0u, 0u, 0u};
    if constexpr (sizeof(IO) == 2) {
        const uint16_t* p = reinterpret_cast<const uint16_t*>(row);
#pragma unroll
        for (int e = 0; e < E; ++e)
            if (col + e < D) v[e >> 1] |= (uint32_t)p[col + e] << (16 * (e & 1));
    } else {
        const uint32_t* p = reinterpret_cast<const uint32_t*>(row);
#pragma unroll
        for (int e = 0; e < E; ++e)
            if (col + e < D) v[e] = p[col + e];
    }
    return v;
}

// Row-major tiles of P pieces a row: piece p of row r lies at piece p ^ fold(r).  A read
// of fragments along the rows takes the same piece of 16 rows; one along the columns four
// neighbouring pieces of rows r .. r + 3 (16-bit types) or r, r + 4, r + 8, r + 12 (fp32).
// fold() spreads both over the 256 bytes of the LDS banks: the rows of a column read to
// different 64-byte windows (bits 2 and up; rows of 64 and 192 bytes are there already),
// the others to the four pieces of a window.
template <int ES, int P>
__device__ __forceinline__ constexpr int fold(int r) {
    const int near = ES == 2 ? r : r >> 2, far = ES == 2 ? (r >> 2) & 3 : r & 3;
    if (P % 16 == 0) return (near & 3) << 2 | far;
    if (P % 8 == 0) return (ES == 2 ? (r >> 1) & 1 : near & 1) << 2 | far;
    return far;
}
template <int ES, int P>
__device__ __forceinline__ int place(int r, int p) {
    return (r * P + (p ^ fold<ES, P>(r))) * 16;
}

// The power of two that takes a largest number m (finite: of biased exponent e) to
// [2^13, 2^14), out of fp16's reach on either side; held between 2^-115 and 2^64, so that it
// has an inverse and an accumulator times it stays finite where the result fits fp16.
__device__ __forceinline__ float range_scale(float m) {
    int e = 267 - (int)(__float_as_uint(m) >> 23);
    e = e > 191 ? 191 : e;
    return __uint_as_float((uint32_t)e << 23);
}
__device__ __forceinline__ float inverse_of_power(float p) {
    return __uint_as_float(0x7f000000u - __float_as_uint(p));
}

// A barrier that waits for this wave's LDS accesses only.  (__syncthreads() and every LDS
// read after a builtin's load to LDS would also wait for the loads in flight, which are
// the next chunk's: hence this and the loads in assembly, which have no register results.)
__device__ __forceinline__ void lds_barrier() {
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

// 64 pieces of 16 bytes, one from each lane's offset in the resource, to LDS from `to` on.
__device__ __forceinline__ void load_to_lds(const u32x4& rsrc, uint32_t offset, const char* to) {
    // (the low half of a generic LDS address is the address in LDS)
    const uint32_t at = __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)to);
    asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tbuffer_load_dwordx4 %0, %1, 0 offen lds"
                 :
                 : "v"(offset), "s"(rsrc), "s"(at)
                 : "memory");  // (m0 is nobody else's here)
}

// A raw buffer resource as four words; base and size are the same in all lanes.
__device__ __forceinline__ u32x4 resource(const void* base, uint32_t bytes) {
    const uintptr_t p = (uintptr_t)base;
    return u32x4{(uint32_t)__builtin_amdgcn_readfirstlane((uint32_t)p),
                 (uint32_t)__builtin_amdgcn_readfirstlane((uint32_t)(p >> 32) & 0xffffu),
                 (uint32_t)__builtin_amdgcn_readfirstlane(bytes), 0x00020000u};
}

// Loads of 64 rows into a tile of P pieces a row (folded or in order), NP per wave, 64
// pieces each: columns from `col` on, the tile's slots in order.  VEC: rows are whole aligned pieces; they go
// straight to LDS through a buffer resource over the chunk's rows, which reads zeros past
// its last row and (by an offset past any resource) past column D.
template <typename IO, int P, int NP, bool FOLD, bool VEC>
struct Loader {
    static constexpr int ES = (int)sizeof(IO), E = 16 / ES;
    uint32_t off[VEC ? NP : 1];
    static __device__ __forceinline__ void where(int i, int& row, int& piece) {
        const int slot = 64 * i + ((int)threadIdx.x & 63);
        row = slot / P;
        piece = FOLD ? slot % P ^ fold<ES, P>(row) : slot % P;
    }
    // first: the wave's first load; step: from one of its loads to the next
    __device__ __forceinline__ Loader(const Heads& x, int D, int col, int first, int step) {
        if constexpr (VEC) {
#pragma unroll
            for (int k = 0; k < NP; ++k) {
                int row, piece;
                where(first + k * step, row, piece);
                off[k] = col + piece * E < D ? (uint32_t)row * (uint32_t)x.ts * ES + (uint32_t)(col + piece * E) * ES
                                             : kOOB;
            }
        }
    }
    // rows t .. t + n - 1 of head h to the tile at `to`
    __device__ __forceinline__ void run(const Heads& x, int64_t t, int64_t h, int n, int D, int col, int first, int step,
                                        char* to) const {
        const IO* base = (const IO*)x.p + t * x.ts + h * x.hs;
        if constexpr (VEC) {
            const u32x4 rs = resource(base, (uint32_t)(((n - 1) * x.ts + D) * ES));
#pragma unroll
            for (int k = 0; k < NP; ++k) {
                const int i = first + k * step;
                if (i < P) load_to_lds(rs, off[k], to + i * 1024);
            }
        } else {
#pragma unroll
            for (int k = 0; k < NP; ++k) {
                const int i = first + k * step;
                if (i >= P) continue;
                int row, piece;
                where(i, row, piece);
                u32x4 v = {0u, 0u, 0u, 0u};
                if (row < n) v = load_piece<IO>(base + row * x.ts, col + piece * E, D);
                *reinterpret_cast<u32x4*>(to + i * 1024 + ((int)threadIdx.x & 63) * 16) = v;
            }
        }
    }
};

// whole pieces, rows that do not overlap, offsets within a chunk that fit a buffer resource
inline bool vec_ok(const Heads& h, int D, size_t es, size_t piece) {
    return (uintptr_t)h.p % piece == 0 && h.ts * es % piece == 0 && h.hs * es % piece == 0 && D * es % piece == 0 &&
           h.ts >= D && h.ts * es < ((int64_t)1 << 24);
}

}  // namespace tile
}  // namespace eql
