// cache.hip -- the tables of a paged key-value cache, built on the GPU from the requests'
// lengths, and the store of new tokens' keys and values into their slots.
#include "eq_device.h"
#include "eq_launch.h"

namespace eql {

namespace {

constexpr int kScan = 1024;  // requests of one pass of the scan

// Per request, for the tokens' kernel: tokens held before, and the place in the free list of
// its first new block.
struct Request {
    int64_t first;
    int32_t held_tokens, held_blocks;
};

__device__ __forceinline__ int64_t blocks_for(int64_t tokens, const TablesArgs& a) {  // (tokens < 2^31)
    const int64_t n = ((uint32_t)tokens + (uint32_t)a.block_size - 1u) / (uint32_t)a.block_size;
    return n < a.max_blocks ? n : a.max_blocks;
}

// Inclusive scan of v over the workgroup; the sum of all to `all`.
__device__ __forceinline__ int64_t scan(int64_t v, int64_t& all) {
    __shared__ int64_t sums[kScan / 64];
    const int tid = (int)threadIdx.x, lane = tid & 63;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const int64_t w = __shfl_up(v, o);
        if (lane >= o) v += w;
    }
    __syncthreads();
    if (lane == 63) sums[tid >> 6] = v;
    __syncthreads();
    int64_t before = 0;
    all = 0;
    for (int w = 0; w < kScan / 64; ++w) {
        if (w < tid >> 6) before += sums[w];
        all += sums[w];
    }
    return v + before;
}

// New token t: its slot and position, and its request's next block if it is the block's first.
__device__ __forceinline__ void place_token(const TablesArgs& a, const Request* requests, const int64_t* offsets, int64_t t) {
    if (t >= offsets[a.batch]) {
        a.slots[t] = -1;
        a.positions[t] = 0;
        return;
    }
    int lo = 0, hi = (int)a.batch - 1;  // first request whose tokens end after t
    while (lo < hi) {
        const int mid = (int)(((int64_t)lo + hi) / 2);
        if (offsets[mid + 1] > t) hi = mid;
        else lo = mid + 1;
    }
    const Request q = requests[lo];
    const uint32_t pos = (uint32_t)(q.held_tokens + (t - offsets[lo])), at = pos / (uint32_t)a.block_size;
    const uint32_t in = pos - at * (uint32_t)a.block_size;
    int64_t id = -1;
    if (at < (uint32_t)a.max_blocks) {
        int32_t* const entry = a.table + (int64_t)lo * a.max_blocks + at;
        if ((int)at < q.held_blocks) {
            id = *entry;
        } else {
            const int64_t f = q.first + at - q.held_blocks;
            if (f >= 0 && f < a.n_free) id = a.free_blocks[f];
            if (in == 0) *entry = (int32_t)id;
        }
    }
    a.slots[t] = id < 0 ? -1 : id * a.block_size + in;
    a.positions[t] = (int32_t)pos;
}

// One workgroup walks the requests: offsets of their new tokens, lengths, and where in the
// free list their new blocks start.  Few requests and tokens (ALONE) are all its own, in one launch
// instead of two: 8.2 us a call for 10.8 with 64 requests of one token, 10.9 for 12.9 with 2048.  Its
// waves place tokens slower than a launch of their own from about 3000 on (64 requests, in a graph:
// 6.9 us for 8.5 with 2048 tokens, 8.0 for 8.3 with 48 each, 9.2 for 8.5 with 64, 13.5 for 8.6 with
// 128), and 2048 requests' offsets and starts take 48 KB of LDS.
constexpr int kAloneRequests = 2048, kAloneTokens = 2 * kScan;
template <bool ALONE>
__global__ __launch_bounds__(kScan) void requests_kernel(TablesArgs a, Request* ws) {
    __shared__ int64_t start;  // (read by the thread that overwrites it)
    extern __shared__ int64_t mine[];  // ALONE: [batch + 1] offsets, [batch] requests
    int64_t* const offsets = ALONE ? mine : a.offsets;
    Request* const out = ALONE ? reinterpret_cast<Request*>(mine + a.batch + 1) : ws;
    if (threadIdx.x == 0) start = a.cursor[0];
    __syncthreads();
    const int64_t cursor = start;
    int64_t tokens = 0, blocks = 0;
    for (int64_t b0 = 0; b0 < a.batch; b0 += kScan) {
        const int64_t b = b0 + threadIdx.x;
        int64_t n = 0, add = 0;
        if (b < a.batch) {
            n = a.lengths[b] < 0 ? 0 : a.lengths[b];
            add = a.added[b] < 0 ? 0 : a.added[b];
            add = n + add > 0x7fffffff ? 0x7fffffff - n : add;
        }
        int64_t all;
        const int64_t end = scan(add, all) + tokens;
        const int64_t t0 = end - add < a.T ? end - add : a.T, t1 = end < a.T ? end : a.T;  // tokens past T do not exist
        const int64_t held = blocks_for(n, a), fresh = blocks_for(n + t1 - t0, a) - held;
        tokens += all;
        const int64_t last = scan(fresh, all) + blocks;
        if (b < a.batch) {
            if (b == 0) a.offsets[0] = 0;
            if (b == 0 && ALONE) offsets[0] = 0;
            a.offsets[b + 1] = t1;
            if (ALONE) offsets[b + 1] = t1;
            a.lengths_out[b] = (int32_t)(n + t1 - t0);
            out[b] = Request{cursor + last - fresh, (int32_t)n, (int32_t)held};
        }
        blocks += all;
    }
    if (threadIdx.x == 0) a.cursor_out[0] = (int32_t)(cursor + blocks);
    if constexpr (ALONE) {
        __syncthreads();
        for (int64_t t = threadIdx.x; t < a.T; t += kScan) place_token(a, out, offsets, t);
    }
}

__global__ __launch_bounds__(256) void tokens_kernel(TablesArgs a, const Request* requests, uint32_t base) {
    const int64_t t = ((int64_t)blockIdx.x + base) * 256 + threadIdx.x;
    if (t < a.T) place_token(a, requests, a.offsets, t);
}

// W numbers a thread: 16 bytes, or one.  A copy: 104 MB in 24.4 us, 4.3 TB/s.
template <typename R>
__global__ __launch_bounds__(256) void store_kernel(StoreArgs a, int W, int pk, int pv, uint32_t base) {
    const int per = a.kv_heads * (pk + pv);  // pieces of a token
    const int64_t id = ((int64_t)blockIdx.x + base) * 256 + threadIdx.x;
    const int64_t t = id / per;
    if (t >= a.T) return;
    const int64_t slot = a.slots[t];
    if (slot < 0 || slot >= a.blocks * a.block_size) return;
    int at = (int)(id - t * per);
    const bool is_v = at >= a.kv_heads * pk;
    at -= is_v ? a.kv_heads * pk : 0;
    const int p = is_v ? pv : pk, head = at / p, piece = at - head * p;
    const Heads& x = is_v ? a.v : a.k;
    const Pages& y = is_v ? a.v_cache : a.k_cache;
    const int64_t block = slot / a.block_size, in = slot - block * a.block_size;
    const R* from = (const R*)x.p + (t * x.ts + head * x.hs) / W + piece;
    R* to = (R*)const_cast<void*>(y.p) + (block * y.bs + in * y.ts + head * y.hs) / W + piece;
    *to = *from;
}

}  // namespace

size_t cache_tables_workspace(int64_t batch) { return (size_t)batch * sizeof(Request); }

hipError_t launch_cache_tables(const TablesArgs& a, void* ws, hipStream_t stream) {
    Request* const r = static_cast<Request*>(ws);
    if (a.batch <= kAloneRequests && a.T <= kAloneTokens) {
        const size_t lds = (size_t)(a.batch + 1) * 8 + (size_t)a.batch * sizeof(Request);
        hipLaunchKernelGGL((requests_kernel<true>), dim3(1), dim3(kScan), lds, stream, a, r);
        return hipGetLastError();
    }
    hipLaunchKernelGGL((requests_kernel<false>), dim3(1), dim3(kScan), 0, stream, a, r);
    in_pieces((a.T + 255) / 256, 256, [&](uint32_t base, uint32_t wgs) {
        hipLaunchKernelGGL(tokens_kernel, dim3(wgs), dim3(256), 0, stream, a, (const Request*)r, base);
    });
    return hipGetLastError();
}

hipError_t launch_cache_store(int io, const StoreArgs& a, hipStream_t stream) {
    const int es = io == kIoF32 ? 4 : 2, W = 16 / es;
    bool vec = a.D_k % W == 0 && a.D_v % W == 0;
    for (const Heads* x : {&a.k, &a.v}) vec = vec && (uintptr_t)x->p % 16 == 0 && x->ts % W == 0 && x->hs % W == 0;
    for (const Pages* x : {&a.k_cache, &a.v_cache})
        vec = vec && (uintptr_t)x->p % 16 == 0 && x->bs % W == 0 && x->ts % W == 0 && x->hs % W == 0;
    const int w = vec ? W : 1, pk = a.D_k / w, pv = a.D_v / w;
    const int64_t n = a.T * a.kv_heads * (pk + pv);
    in_pieces((n + 255) / 256, 256, [&](uint32_t base, uint32_t wgs) {
        if (vec) hipLaunchKernelGGL((store_kernel<u32x4>), dim3(wgs), dim3(256), 0, stream, a, w, pk, pv, base);
        else if (es == 4) hipLaunchKernelGGL((store_kernel<uint32_t>), dim3(wgs), dim3(256), 0, stream, a, w, pk, pv, base);
        else hipLaunchKernelGGL((store_kernel<uint16_t>), dim3(wgs), dim3(256), 0, stream, a, w, pk, pv, base);
    });
    return hipGetLastError();
}

}  // namespace eql
