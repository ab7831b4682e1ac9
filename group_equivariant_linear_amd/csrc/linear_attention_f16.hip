// linear_attention_f16.hip -- chunk kernels of linear attention, f16.
#include "linear_attention.h"

namespace eql {
namespace mix {

template hipError_t run<_Float16>(Jobs&, hipStream_t);

}  // namespace mix
}  // namespace eql
