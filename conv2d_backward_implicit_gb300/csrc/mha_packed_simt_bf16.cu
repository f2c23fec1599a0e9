// mha_packed_simt_bf16.cu -- the CUDA-core kernels of packed attention for __nv_bfloat16 (mha_packed_simt.cuh).
#include <atomic>

#include "mha_packed_simt.cuh"

namespace mhapk {

int forward_simt_bf16(const Args &a, const mha_packed_params *p, unsigned *error, cudaStream_t st) {
    return forward_any<__nv_bfloat16>(a, p, error, st);
}
int backward_simt_bf16(const Args &a, const mha_packed_params *p, unsigned *error, cudaStream_t st) {
    return backward_any<__nv_bfloat16>(a, p, error, st);
}

}  // namespace mhapk
