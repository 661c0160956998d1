// qr_norm_f16.cu -- the norm kernels for fp16 values (qr_norm.cuh).
#include "qr_norm.cuh"

namespace qrk {

template cudaError_t launch_norm_typed<0>(int weight, const NormArgs &a, cudaStream_t s);

}  // namespace qrk
