// attention_forward_f16.hip -- softmax attention's forward kernels, f16.
#include "attention.h"

namespace eql {
namespace att {

template hipError_t forward<_Float16>(AttentionArgs, const BucketMap&, hipStream_t);

}  // namespace att
}  // namespace eql
