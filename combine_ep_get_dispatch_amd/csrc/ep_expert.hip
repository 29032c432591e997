// The experts' products with 4-bit weights on gfx950, over the rows that
// dispatch writes:
//   y[r, n] = sum_i x[r, i] * (q[e, n, i] - z[e, i/G, n]) * s[e, i/G, n],
// e the expert of row r, q a 4-bit code, z the group's zero point (8 without
// one) and s its scale; x is bf16, or E4M3 codes with one fp32 scale per 128
// channels.  With SWIGLU the weights hold 2N channels and
//   y[r, n] = silu(gate_n) * up_n,  gate = channels [0, N), up = [N, 2N),
// taken from the fp32 sums and rounded once.
//
// In decode an expert has a few rows and the product is bound by reading its
// weights once.
#include "ep_internal.h"
#include "ep_device.h"

namespace ep {
namespace {

__device__ __forceinline__ float e4m3_value(uint32_t code) {
    return __builtin_amdgcn_cvt_f32_fp8((int)code, 0);
}

// One wave per (expert, channel); lanes over the input channels.
template <bool FP8>
__global__ __launch_bounds__(256) void expert_linear_kernel(
    const void* __restrict__ x, const float* __restrict__ xs, int64_t num_rows,
    const int32_t* __restrict__ offsets, const int32_t* __restrict__ counts, int capacity, int I,
    int N, int G, const uint8_t* __restrict__ wq, const uint16_t* __restrict__ scales,
    const uint8_t* __restrict__ zeros, bool swiglu, uint16_t* __restrict__ y) {
    const int lane = threadIdx.x & 63;
    const int e = blockIdx.y;
    const int n = blockIdx.x * 4 + (threadIdx.x >> 6);
    if (n >= N) return;
    int64_t begin = offsets ? (int64_t)offsets[e] : (int64_t)e * capacity;
    int64_t end = begin + (offsets ? counts[e] : min(counts[e], capacity));
    if (begin < 0) begin = 0;
    if (end > num_rows) end = num_rows;
    const int WN = swiglu ? 2 * N : N;
    const int NG = I / G;
    for (int64_t r = begin; r < end; ++r) {
        float acc[2] = {0.0f, 0.0f};
        for (int h = 0; h < (swiglu ? 2 : 1); ++h) {
            const int c = n + h * N;
            const uint8_t* wr = wq + ((int64_t)e * WN + c) * (I / 2);
            for (int i = lane; i < I; i += 64) {
                const int g = i / G;
                const int64_t sg = ((int64_t)e * NG + g) * WN + c;
                const int q = (wr[i >> 1] >> ((i & 1) * 4)) & 15;
                const float z = zeros ? (float)(zeros[sg] & 15) : 8.0f;
                const float s = __uint_as_float((uint32_t)scales[sg] << 16);
                float v;
                if constexpr (FP8)
                    v = e4m3_value(static_cast<const uint8_t*>(x)[r * I + i]) *
                        xs[r * (I / 128) + i / 128];
                else
                    v = __uint_as_float(
                        (uint32_t) static_cast<const uint16_t*>(x)[r * I + i] << 16);
                acc[h] = __builtin_fmaf(v, ((float)q - z) * s, acc[h]);
            }
        }
#pragma unroll
        for (int m = 32; m >= 1; m >>= 1) {
            acc[0] += __shfl_xor(acc[0], m);
            acc[1] += __shfl_xor(acc[1], m);
        }
        float o = acc[0];
        if (swiglu) o = o / (1.0f + expf(-o)) * acc[1];
        if (lane == 0) y[r * N + n] = (uint16_t)pack_bf16x2(o, 0.0f);
    }
}

}  // namespace

hipError_t launch_expert_linear_w4(const void* x, const float* xs, bool fp8, int64_t num_rows,
                                   const int32_t* offsets, const int32_t* counts, int capacity,
                                   int E, int I, int N, int G, const uint8_t* w,
                                   const uint16_t* scales, const uint8_t* zeros, bool swiglu,
                                   uint16_t* y, hipStream_t s) {
    if (num_rows == 0) return hipSuccess;
    const dim3 grid((unsigned)((N + 3) / 4), (unsigned)E), block(256);
    if (fp8)
        hipLaunchKernelGGL(expert_linear_kernel<true>, grid, block, 0, s, x, xs, num_rows, offsets,
                           counts, capacity, I, N, G, w, scales, zeros, swiglu, y);
    else
        hipLaunchKernelGGL(expert_linear_kernel<false>, grid, block, 0, s, x, xs, num_rows,
                           offsets, counts, capacity, I, N, G, w, scales, zeros, swiglu, y);
    return hipGetLastError();
}

}  // namespace ep
