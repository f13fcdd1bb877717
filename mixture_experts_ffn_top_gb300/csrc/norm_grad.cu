// norm_grad.cu -- the gradients of layer norm and RMSNorm (see norm.cuh).
#include "norm.cuh"

namespace moe {

size_t norm_scratch_bytes(int N, int D) { return (size_t)std::min(N, NORM_PARTS) * 2 * D * 4; }

int launch_norm_grad(bool rms, const void *d_y, int64_t d_y_stride, const void *x, int64_t x_stride, int dtype,
                     const float *gamma, float eps, int N, int D, void *d_x, int64_t d_x_stride, float *d_gamma,
                     float *d_beta, void *ws, cudaStream_t s) {
    NormArgs a{};
    a.x = x;
    a.x_stride = x_stride;
    a.dy = d_y;
    a.dy_stride = d_y_stride;
    a.gamma = gamma;
    a.eps = eps;
    a.N = N;
    a.D = D;
    a.out = d_x;
    a.out_stride = d_x_stride;
    a.d_gamma = d_gamma;
    a.d_beta = d_beta;
    void *scratch = ws_ptr<char>(ws, 256);
    return rms ? launch_norm_mode<NORM_RMS_GRAD>(a, dtype, scratch, s) : launch_norm_mode<NORM_GRAD>(a, dtype, scratch, s);
}

}  // namespace moe
