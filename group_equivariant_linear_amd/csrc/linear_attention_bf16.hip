// linear_attention_bf16.hip -- chunk kernels of linear attention, bf16.
#include "linear_attention.h"

namespace eql {
namespace mix {

template hipError_t run<__bf16>(Jobs&, hipStream_t);

}  // namespace mix
}  // namespace eql
