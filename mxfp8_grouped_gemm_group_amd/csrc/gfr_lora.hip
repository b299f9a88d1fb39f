// A dense product with the low-rank adapter of each row's own request.
// include/gfr.h states the operator.
//
//   shrink   inner[t] = scaling[i] (x[t] A[i]^T), FP32
//   dense    the shared product, in FP32
//   expand   out[t] = dense[t] + bias + inner[t] B[i]^T + residual[t]
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "gfr.h"
#include "gfr_device.h"
#include "gfr_layer.h"
#include "gfr_tile.h"

namespace gfr {
namespace {

// The adapter of row t, -1 for none (and for ids out of range, which are flagged).
__device__ __forceinline__ int adapter(const LoraParams &p, int t) {
    const int i = p.ids[t];
    if (i >= -1 && i < p.L) return i;
    if (p.status) atomicOr(p.status, GFR_DEV_BAD_ADAPTER);
    return -1;
}

// A wave per row and rank.
template <bool F16>
__global__ __launch_bounds__(256) void shrink_kernel(LoraParams p) {
    const int lane = threadIdx.x & 63, j = blockIdx.y * 4 + (threadIdx.x >> 6);
    const int t = blockIdx.x;
    if (j >= p.r) return;
    const int i = adapter(p, t);
    if (i < 0) return;
    const uint16_t *x = p.x + static_cast<int64_t>(t) * p.K;
    const uint16_t *a = p.a + (static_cast<int64_t>(i) * p.r + j) * p.K;
    float sum = 0.0f;
    for (int k = lane; k < p.K; k += 64) sum = fmaf(unpack1<F16>(x[k]), unpack1<F16>(a[k]), sum);
    for (int d = 32; d > 0; d >>= 1) sum += __shfl_xor(sum, d);
    if (lane == 0)
        p.inner[static_cast<int64_t>(t) * p.r + j] = sum * (p.scaling ? p.scaling[i] : 1.0f);
}

// A thread per column of a row.
template <bool F16>
__global__ __launch_bounds__(256) void expand_kernel(LoraParams p) {
    const int n = blockIdx.x * 256 + threadIdx.x;
    if (n >= p.N) return;
    for (int t = blockIdx.y; t < p.M; t += gridDim.y) {
        const int64_t at = static_cast<int64_t>(t) * p.N + n;
        float y = p.dense[at];
        const int i = p.ids[t];
        if (i >= 0 && i < p.L) {
            const float *s = p.inner + static_cast<int64_t>(t) * p.r;
            const uint16_t *b = p.b + (static_cast<int64_t>(i) * p.N + n) * p.r;
            float sum = 0.0f;
            for (int j = 0; j < p.r; ++j) sum = fmaf(s[j], unpack1<F16>(b[j]), sum);
            y += sum;
        }
        if (p.residual) y += unpack1<F16>(p.residual[at]);
        if (p.out_f32)
            static_cast<float *>(p.out)[at] = y;
        else
            static_cast<uint16_t *>(p.out)[at] = static_cast<uint16_t>(pack2<F16>(y, 0.0f));
    }
}

template <bool F16>
hipError_t launch_lora_t(const LoraParams &p, hipStream_t stream) {
    hipLaunchKernelGGL((shrink_kernel<F16>), dim3(p.M, (p.r + 3) / 4), dim3(256), 0, stream, p);
    if (hipError_t e = hipGetLastError(); e != hipSuccess) return e;
    LinearParams d{};
    d.x = p.x;
    d.w = p.w;
    d.bias = p.bias;
    d.bias_f32 = p.bias_f32;
    d.out = p.dense;
    d.out_f32 = 1;
    d.f16 = p.f16;
    d.act = GFR_ACT_NONE;
    d.wide = p.N % 8 == 0;
    d.M = p.M;
    d.N = p.N;
    d.K = p.K;
    d.kernel = p.choice.kernel;
    d.split = p.choice.split;
    d.partial = p.partial;
    if (hipError_t e = launch_linear(d, stream); e != hipSuccess) return e;
    hipLaunchKernelGGL((expand_kernel<F16>), dim3((p.N + 255) / 256, p.M < 65535 ? p.M : 65535),
                       dim3(256), 0, stream, p);
    return hipGetLastError();
}

}  // namespace

LoraLayout lora_layout(int64_t M, int64_t N, int64_t K, int64_t r) {
    const auto up = [](size_t n) { return (n + 255) & ~static_cast<size_t>(255); };
    LoraLayout l{};
    l.choice = linear_choice(M, N, K, GFR_ACT_NONE);
    l.dense = up(sizeof(float) * M * r);
    l.partial = l.dense + up(sizeof(float) * M * N);
    l.total = l.partial;
    if (l.choice.split > 1)
        l.total += up(sizeof(float) * l.choice.split * M * ((N + 7) / 8 * 8));
    return l;
}

hipError_t launch_lora(const LoraParams &p, hipStream_t stream) {
    return p.f16 ? launch_lora_t<true>(p, stream) : launch_lora_t<false>(p, stream);
}

}  // namespace gfr
