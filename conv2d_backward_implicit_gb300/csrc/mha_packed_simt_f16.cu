// mha_packed_simt_f16.cu -- the CUDA-core kernels of packed attention for __half (mha_packed_simt.cuh).
#include <atomic>

#include "mha_packed_simt.cuh"

namespace mhapk {

int forward_simt_f16(const Args &a, const mha_packed_params *p, unsigned *error, cudaStream_t st) {
    return forward_any<__half>(a, p, error, st);
}
int backward_simt_f16(const Args &a, const mha_packed_params *p, unsigned *error, cudaStream_t st) {
    return backward_any<__half>(a, p, error, st);
}

}  // namespace mhapk
