// attention.hip -- softmax attention: what a launch takes besides its tensors, the kernels
// by type (attention.h, instantiated in attention_{forward,backward}_{f32,bf16,f16}.hip),
// and the join of the biases' gradients.
#include "attention.h"

namespace eql {

namespace att {
extern template hipError_t forward<float>(AttentionArgs, const BucketMap&, hipStream_t);
extern template hipError_t forward<__bf16>(AttentionArgs, const BucketMap&, hipStream_t);
extern template hipError_t forward<_Float16>(AttentionArgs, const BucketMap&, hipStream_t);
extern template hipError_t backward<float>(AttentionArgs, const BucketMap&, hipStream_t);
extern template hipError_t backward<__bf16>(AttentionArgs, const BucketMap&, hipStream_t);
extern template hipError_t backward<_Float16>(AttentionArgs, const BucketMap&, hipStream_t);
}  // namespace att

namespace {

using namespace att;

// Gradient of one bias: the sums of every slot of its head, in a fixed order.
__global__ __launch_bounds__(256) void reduce_kernel(const float* parts, float* dbias, int64_t n, uint32_t base) {
    __shared__ float sum[256];
    const int tid = (int)threadIdx.x;
    const uint32_t cell = blockIdx.x + base;
    const float* p = parts + (int64_t)cell * n;
    float t = 0.0f;
    for (int64_t i = tid; i < n; i += 256) t += p[i];
    sum[tid] = t;
    for (int w = 128; w > 0; w >>= 1) {
        __syncthreads();
        if (tid < w) sum[tid] += sum[tid + w];
    }
    if (tid == 0) dbias[cell] = sum[0];
}

// (no tokens: no slots, of packed sequences either; nothing launches, and no sums of slots exist)
uint32_t slots_for(const int64_t* offsets, int64_t batch, int64_t T) {
    if (batch <= 0 || T <= 0) return 0;
    return (uint32_t)(offsets ? T / kRows + batch : batch * ((T / batch + kRows - 1) / kRows));
}

// Dealt are sequences of 16 slots and more, packed ones by their mean (their lengths are on the device).
Deal deal_for(const int64_t* offsets, int64_t batch, int64_t T, int heads) {
    const uint32_t slots = slots_for(offsets, batch, T);
    if (slots == 0 || T / batch < 16 * kRows) return Deal{slots, 0, 0};
    if (offsets) return Deal{slots, (uint32_t)heads, 1};
    return Deal{slots / (uint32_t)batch, (uint32_t)(heads * batch), (uint32_t)batch};
}

size_t round_up(size_t n) { return (n + 255) / 256 * 256; }

}  // namespace

// Rows' statistics, marks of steep ones, and the sums of each slot's buckets (packed sequences have the most slots).
size_t attention_workspace(int heads, int buckets, int64_t T, int64_t batch, bool backward) {
    if (!backward || T <= 0) return 0;
    const size_t slots = (size_t)(T / kRows + batch) * heads;
    return 4 * round_up((size_t)T * heads * 4) + round_up(slots * 16) + slots * buckets * 4;
}

hipError_t launch_attention(int io, AttentionArgs a, const BucketMap& map, hipStream_t stream) {
    if (a.T <= 0) return hipSuccess;
    a.slots = slots_for(a.offsets, a.batch, a.T);
    a.deal = deal_for(a.offsets, a.batch, a.T, a.heads);
    if (a.deal.workgroups(a.heads) > 0x7fffffff) return hipErrorNotSupported;
    return io == kIoF32 ? att::forward<float>(a, map, stream)
                        : (io == kIoBF16 ? att::forward<__bf16>(a, map, stream) : att::forward<_Float16>(a, map, stream));
}

hipError_t launch_attention_backward(int io, AttentionArgs a, const BucketMap& map, void* ws, hipStream_t stream) {
    a.slots = slots_for(a.offsets, a.batch, a.T);
    a.rows = static_cast<float*>(ws);
    a.parts = reinterpret_cast<float*>(reinterpret_cast<char*>(a.steep()) + round_up((size_t)a.slots * a.heads * 16));
    a.deal = deal_for(a.offsets, a.batch, a.T, a.heads);
    a.kv_deal = deal_for(a.kv_offsets, a.batch, a.T_kv, a.kv_heads);
    if (a.deal.workgroups(a.heads) > 0x7fffffff || a.kv_deal.workgroups(a.kv_heads) > 0x7fffffff) return hipErrorNotSupported;
    const hipError_t e = io == kIoF32 ? att::backward<float>(a, map, stream)
                         : io == kIoBF16 ? att::backward<__bf16>(a, map, stream)
                                         : att::backward<_Float16>(a, map, stream);
    if (e != hipSuccess) return e;
    if (a.dbias)
        in_pieces((int64_t)a.heads * a.buckets, 256, [&](uint32_t base, uint32_t wgs) {
            hipLaunchKernelGGL(reduce_kernel, dim3(wgs), dim3(256), 0, stream, a.parts, a.dbias, (int64_t)a.slots, base);
        });
    return hipGetLastError();
}

}  // namespace eql
