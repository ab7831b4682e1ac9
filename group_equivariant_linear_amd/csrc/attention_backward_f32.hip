// attention_backward_f32.hip -- softmax attention's backward kernels, f32.
#include "attention.h"

namespace eql {
namespace att {

template hipError_t backward<float>(AttentionArgs, const BucketMap&, hipStream_t);

}  // namespace att
}  // namespace eql
