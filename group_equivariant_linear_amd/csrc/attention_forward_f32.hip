// attention_forward_f32.hip -- softmax attention's forward kernels, f32.
#include "attention.h"

namespace eql {
namespace att {

template hipError_t forward<float>(AttentionArgs, const BucketMap&, hipStream_t);

}  // namespace att
}  // namespace eql
