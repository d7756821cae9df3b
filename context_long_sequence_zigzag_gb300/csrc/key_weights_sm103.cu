// placeholder
#include "internal.h"
namespace cpattn {
bool tc_key_weights_supported(int32_t) { return false; }
cudaError_t launch_tc_key_weights(const AttnArgs&, cudaStream_t) { return cudaErrorInvalidValue; }
}  // namespace cpattn
