// linear_attention_f32.hip -- chunk kernels of linear attention, f32.
#include "linear_attention.h"

namespace eql {
namespace mix {

template hipError_t run<float>(Jobs&, hipStream_t);

}  // namespace mix
}  // namespace eql
