// attention_backward_bf16.hip -- softmax attention's backward kernels, bf16.
#include "attention.h"

namespace eql {
namespace att {

template hipError_t backward<__bf16>(AttentionArgs, const BucketMap&, hipStream_t);

}  // namespace att
}  // namespace eql
