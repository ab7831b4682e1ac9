// attention_backward_f16.hip -- softmax attention's backward kernels, f16.
#include "attention.h"

namespace eql {
namespace att {

template hipError_t backward<_Float16>(AttentionArgs, const BucketMap&, hipStream_t);

}  // namespace att
}  // namespace eql
