// mha_packed_simt_f32.cu -- the CUDA-core kernels of packed attention for float (mha_packed_simt.cuh).
#include <atomic>

#include "mha_packed_simt.cuh"

namespace mhapk {

int forward_simt_f32(const Args &a, const mha_packed_params *p, unsigned *error, cudaStream_t st) {
    return forward_any<float>(a, p, error, st);
}
int backward_simt_f32(const Args &a, const mha_packed_params *p, unsigned *error, cudaStream_t st) {
    return backward_any<float>(a, p, error, st);
}

}  // namespace mhapk
