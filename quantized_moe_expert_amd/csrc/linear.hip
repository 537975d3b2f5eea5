// Linear layer: y = act(x W^T + bias) + residual.
#include "backbone.h"

namespace moeq4 {

namespace {

__device__ __forceinline__ float activate(float z, int act) {
    if (act == 1) return z / (1.0f + expf(-z));
    if (act == 2) return 0.5f * z * (1.0f + erff(z * 0.70710678118654752f));
    return z;
}

// One wave per output: products of a row of weights and a row of x.
template <bool INT8>
__global__ __launch_bounds__(256) void linear_row_kernel(LinearArgs a, int64_t outputs) {
    const int lane = threadIdx.x & 63;
    const int64_t o = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
    if (o >= outputs) return;
    const int64_t t = o / a.N;
    const int n = (int)(o % a.N);
    const uint16_t *x = a.x + t * a.ldx;
    float sum = 0.0f;
    if (INT8) {
        const int8_t *w = static_cast<const int8_t *>(a.q) + (int64_t)n * a.K;
        for (int g = 0; g < a.K / 128; ++g) {
            const int k = g * 128 + lane * 2;
            const float p = bf16_to_f32(x[k]) * (float)w[k] + bf16_to_f32(x[k + 1]) * (float)w[k + 1];
            sum += p * f16_to_f32(a.scale[(int64_t)n * (a.K / 128) + g]);
        }
    } else {
        const uint16_t *w = static_cast<const uint16_t *>(a.q) + (int64_t)n * a.K;
        for (int k = lane; k < a.K; k += 64) sum += bf16_to_f32(x[k]) * bf16_to_f32(w[k]);
    }
    sum = seg_sum<64>(sum);
    if (lane == 0) {
        if (a.bias) sum += a.bias[n];
        sum = activate(sum, a.act);
        if (a.residual) sum += bf16_to_f32(a.residual[t * a.ldr + n]);
        if (a.y_f32)
            static_cast<float *>(a.y)[t * a.ldy + n] = sum;
        else
            static_cast<uint16_t *>(a.y)[t * a.ldy + n] = f32_to_bf16_rne(sum);
    }
}

}  // namespace

hipError_t launch_linear(const LinearArgs &a, hipStream_t s) {
    const int64_t outputs = a.T * a.N, blocks = (outputs + 3) / 4;
    if (blocks >= (int64_t)1 << 31) return hipErrorInvalidValue;
    if (a.int8)
        hipLaunchKernelGGL(linear_row_kernel<true>, dim3((unsigned)blocks), dim3(256), 0, s, a, outputs);
    else
        hipLaunchKernelGGL(linear_row_kernel<false>, dim3((unsigned)blocks), dim3(256), 0, s, a, outputs);
    return hipGetLastError();
}

}  // namespace moeq4
