// attention_forward_bf16.hip -- softmax attention's forward kernels, bf16.
#include "attention.h"

namespace eql {
namespace att {

template hipError_t forward<__bf16>(AttentionArgs, const BucketMap&, hipStream_t);

}  // namespace att
}  // namespace eql
