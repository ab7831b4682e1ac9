// eq_plan.h -- the plan object behind eqlinear_plan_t and the argument checks
// that the files of the C ABI share (not part of the ABI).
#pragma once

#include "../../include/eqlinear.h"
#include "eq_launch.h"

struct eqlinear_plan_s {
    int kind;
    int dtype;
    int N;
    int C_in, C_out;  // rotary and mixer plans: channels of all query heads in and out
    // rotary and mixer plans
    int heads = 0, kv_heads = 0;
    int d_k = 0, d_v = 0;  // channels per head (rotary: both d)
    // rotary plans
    int rot = 0, layout = 0;
    eql::RotaryFreq freq{};
    // norm plans (C_in = C_out = C)
    int groups = 0, act = 0;
    float eps = 0.0f;
};

namespace eql {

inline bool dtype_ok(int dt) { return dt == EQL_F32 || dt == EQL_BF16 || dt == EQL_F16; }

inline size_t elem_size(const eqlinear_plan_s* p) { return p->dtype == EQL_F32 ? 4 : 2; }

inline bool overlaps(const void* a, size_t na, const void* b, size_t nb) {
    const uintptr_t a0 = (uintptr_t)a, b0 = (uintptr_t)b;
    return a0 < b0 + nb && b0 < a0 + na;
}

inline eqlinear_status hip_status(hipError_t e) { return e == hipSuccess ? EQL_OK : EQL_ERR_HIP; }

// Widths are capped so every per-row offset fits an int in the kernels.
constexpr int64_t kMaxWidth = 1 << 20;

}  // namespace eql
