// norm.cu -- layer norm of token rows (see norm.cuh).
#include "norm.cuh"

namespace moe {

int launch_layernorm(const void *x, int64_t x_stride, int dtype, const float *gamma, const float *beta, float eps, int N,
                     int D, void *y, int64_t y_stride, cudaStream_t s) {
    NormArgs a{};
    a.x = x;
    a.x_stride = x_stride;
    a.gamma = gamma;
    a.beta = beta;
    a.eps = eps;
    a.N = N;
    a.D = D;
    a.out = y;
    a.out_stride = y_stride;
    return launch_norm_mode<NORM_FORWARD>(a, dtype, nullptr, s);
}

}  // namespace moe
