#include "s5_delta.cuh"
namespace s5 {
namespace delta {
bool tc_supported(const Args &, s5_dtype, bool) { return false; }
size_t tc_image_bytes(int, int, int) { return 0; }
cudaError_t tc_forward(const Args &, cudaStream_t) { return cudaErrorNotSupported; }
}  // namespace delta
}  // namespace s5
