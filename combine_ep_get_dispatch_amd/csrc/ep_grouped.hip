// The experts' products over ragged runs of rows, and their gradients, on
// gfx950:
//   y[r, n]  = sum_i x[r, i] * w[e, n, i]        e the expert of row r
//   gx[r, i] = sum_n gy[r, n] * w[e, n, i]
//   gw[e, n, i] = sum over e's rows r of gy[r, n] * x[r, i]
// in bf16, or y from E4M3 rows and weights, whose codes' products are summed
// over 128 channels and then scaled, fp32 throughout and rounded once.
//
// First form: a thread per result.
#include "ep_internal.h"
#include "ep_device.h"

namespace ep {
namespace {

struct LinearArgs {
    const void* x;
    const float* xs;
    RowRuns runs;
    int I, N;
    const void* w;
    const float* ws;
    uint16_t* y;
};

__device__ __forceinline__ float bf16(uint16_t v) { return __uint_as_float((uint32_t)v << 16); }

// The expert that holds row r, -1 if none does.
__device__ __forceinline__ int expert_of(const RowRuns& runs, int64_t r) {
    for (int e0 = 0; e0 < runs.E; e0 += 64) {
        const int e = e0 + (threadIdx.x & 63);
        int64_t b = 0, n = 0;
        if (e < runs.E) n = runs.of(e, b);
        const uint64_t hit = __ballot(n > 0 && r >= b && r < b + n);
        if (hit) return e0 + __builtin_ctzll(hit);
    }
    return -1;
}

__device__ __forceinline__ float dot_bf16(const uint16_t* a, const uint16_t* b, int n, int64_t sb) {
    float s = 0.0f;
    for (int i = 0; i < n; ++i) s = __builtin_fmaf(bf16(a[i]), bf16(b[i * sb]), s);
    return s;
}

template <bool FP8, bool SWIGLU>
__device__ __forceinline__ float channel(const LinearArgs& p, int e, int64_t r, int half, int n) {
    const int I = p.I, W = p.N * (SWIGLU ? 2 : 1);
    const int64_t row = ((int64_t)e * W + half * p.N + n) * I;
    if constexpr (!FP8) {
        return dot_bf16(static_cast<const uint16_t*>(p.x) + r * I,
                        static_cast<const uint16_t*>(p.w) + row, I, 1);
    } else {
        const uint8_t* x = static_cast<const uint8_t*>(p.x) + r * I;
        const uint8_t* w = static_cast<const uint8_t*>(p.w) + row;
        const int NB = (p.N + 127) / 128, KB = I / 128;
        const float* ws = p.ws + ((int64_t)(e * (SWIGLU ? 2 : 1) + half) * NB + n / 128) * KB;
        float s = 0.0f;
        for (int k = 0; k < KB; ++k) {
            float t = 0.0f;
            for (int i = k * 128; i < k * 128 + 128; ++i)
                t = __builtin_fmaf(__builtin_amdgcn_cvt_f32_fp8(x[i], 0),
                                   __builtin_amdgcn_cvt_f32_fp8(w[i], 0), t);
            s = __builtin_fmaf(p.xs[r * KB + k] * ws[k], t, s);
        }
        return s;
    }
}

template <bool FP8, bool SWIGLU>
__global__ __launch_bounds__(256) void linear_kernel(const LinearArgs p) {
    const int64_t r = blockIdx.x;
    const int e = expert_of(p.runs, r);
    if (e < 0) return;
    for (int n = threadIdx.x; n < p.N; n += 256) {
        float v = channel<FP8, SWIGLU>(p, e, r, 0, n);
        if constexpr (SWIGLU) v = v / (1.0f + expf(-v)) * channel<FP8, SWIGLU>(p, e, r, 1, n);
        p.y[r * p.N + n] = (uint16_t)pack_bf16x2(v, v);
    }
}

__global__ __launch_bounds__(256) void grad_rows_kernel(const LinearArgs p) {
    const int64_t r = blockIdx.x;
    const int e = expert_of(p.runs, r);
    if (e < 0) return;
    for (int i = threadIdx.x; i < p.I; i += 256) {
        const float v = dot_bf16(static_cast<const uint16_t*>(p.x) + r * p.N,
                                 static_cast<const uint16_t*>(p.w) + (int64_t)e * p.N * p.I + i,
                                 p.N, p.I);
        p.y[r * p.I + i] = (uint16_t)pack_bf16x2(v, v);
    }
}

template <bool F32, bool ADD>
__global__ __launch_bounds__(256) void grad_weight_kernel(const uint16_t* gy, const uint16_t* x,
                                                          RowRuns runs, int I, int N, void* gw) {
    const int e = blockIdx.x / N, n = blockIdx.x % N;
    int64_t b;
    const int64_t rows = runs.of(e, b);
    for (int i = threadIdx.x; i < I; i += 256) {
        float v = 0.0f;
        for (int64_t r = b; r < b + rows; ++r)
            v = __builtin_fmaf(bf16(gy[r * N + n]), bf16(x[r * I + i]), v);
        const int64_t at = (int64_t)blockIdx.x * I + i;
        if constexpr (F32) {
            float* o = static_cast<float*>(gw) + at;
            *o = ADD ? *o + v : v;
        } else {
            static_cast<uint16_t*>(gw)[at] = (uint16_t)pack_bf16x2(v, v);
        }
    }
}

}  // namespace

hipError_t launch_expert_linear(const void* x, const float* xs, const RowRuns& runs, int I, int N,
                                const void* w, const float* ws, bool swiglu, uint16_t* y,
                                hipStream_t s) {
    if (runs.num_rows == 0) return hipSuccess;
    const LinearArgs p = {x, xs, runs, I, N, w, ws, y};
    const dim3 grid((unsigned)runs.num_rows), block(256);
    if (xs) {
        if (swiglu)
            hipLaunchKernelGGL((linear_kernel<true, true>), grid, block, 0, s, p);
        else
            hipLaunchKernelGGL((linear_kernel<true, false>), grid, block, 0, s, p);
    } else {
        if (swiglu)
            hipLaunchKernelGGL((linear_kernel<false, true>), grid, block, 0, s, p);
        else
            hipLaunchKernelGGL((linear_kernel<false, false>), grid, block, 0, s, p);
    }
    return hipGetLastError();
}

hipError_t launch_expert_grad_rows(const uint16_t* gy, const RowRuns& runs, int I, int N,
                                   const uint16_t* w, uint16_t* gx, hipStream_t s) {
    if (runs.num_rows == 0) return hipSuccess;
    const LinearArgs p = {gy, nullptr, runs, I, N, w, nullptr, gx};
    hipLaunchKernelGGL(grad_rows_kernel, dim3((unsigned)runs.num_rows), dim3(256), 0, s, p);
    return hipGetLastError();
}

hipError_t launch_expert_grad_weight(const uint16_t* gy, const uint16_t* x, const RowRuns& runs,
                                     int I, int N, void* gw, bool fp32, bool accumulate,
                                     hipStream_t s) {
    const dim3 grid((unsigned)(runs.E * N)), block(256);
    if (!fp32)
        hipLaunchKernelGGL((grad_weight_kernel<false, false>), grid, block, 0, s, gy, x, runs, I,
                           N, gw);
    else if (accumulate)
        hipLaunchKernelGGL((grad_weight_kernel<true, true>), grid, block, 0, s, gy, x, runs, I, N,
                           gw);
    else
        hipLaunchKernelGGL((grad_weight_kernel<true, false>), grid, block, 0, s, gy, x, runs, I, N,
                           gw);
    return hipGetLastError();
}

}  // namespace ep
