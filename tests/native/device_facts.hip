// Facts about the hardware that the kernels rest on, tried by the tests: the error
// of the router's fp32 sigmoid, and the sums of the 8-bit matrix instruction.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../bitplane_quantized_expert_amd/csrc/pm_fp8.h"
#include "../../bitplane_quantized_expert_amd/csrc/pm_rank.h"

namespace {

// Every fp32 number, `per` of them a thread: out[2 t] the thread's largest error,
// out[2 t + 1] its largest relative error where the sigmoid is kSigmoidSmall or more.
__global__ void sigmoid_errors(double* out, uint32_t per) {
    const uint32_t t = blockIdx.x * blockDim.x + threadIdx.x;
    double error = 0.0, relative = 0.0;
    for (uint32_t i = 0; i < per; ++i) {
        const float l = __uint_as_float(t * per + i);
        if (!(l == l)) continue;
        const double s = 1.0 / (1.0 + exp(-double(l)));
        const double d = fabs(double(pm::sigmoid_rank(l)) - s);
        error = fmax(error, d);
        if (s >= pm::kSigmoidSmall) relative = fmax(relative, d / s);
    }
    out[2 * t] = error;
    out[2 * t + 1] = relative;
}

// d[n][i][j] = sum over k of a[n][i][k] b[n][j][k], 16 x 16 x 128 codes, a wave each.
__global__ void products(const uint8_t* a, const uint8_t* b, float* d) {
    const int lane = threadIdx.x, i = lane & 15, q = lane >> 4;
    const size_t n = blockIdx.x;
    const pm::u32x4* pa = reinterpret_cast<const pm::u32x4*>(a + n * 2048 + i * 128 + q * 32);
    const pm::u32x4* pb = reinterpret_cast<const pm::u32x4*>(b + n * 2048 + i * 128 + q * 32);
    const pm::f32x4 r = pm::mfma_codes(pm::join(pa[0], pa[1]), pm::join(pb[0], pb[1]));
    for (int k = 0; k < 4; ++k) d[n * 256 + (4 * q + k) * 16 + i] = r[k];
}

}  // namespace

// out [2^18][2]
extern "C" int facts_sigmoid(double* out, void* stream) {
    hipLaunchKernelGGL(sigmoid_errors, dim3(1024), dim3(256), 0, hipStream_t(stream), out, 1u << 14);
    return int(hipGetLastError());
}

// a, b [n][16][128] codes, 16-byte aligned; d [n][16][16]
extern "C" int facts_products(int n, const uint8_t* a, const uint8_t* b, float* d, void* stream) {
    if (n < 1) return -1;
    hipLaunchKernelGGL(products, dim3(n), dim3(64), 0, hipStream_t(stream), a, b, d);
    return int(hipGetLastError());
}
