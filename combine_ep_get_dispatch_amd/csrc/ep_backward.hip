// Gradient of combine on gfx950.  With g = d loss / d out and r = dst_row[t,k],
// the forward out[t] = sum_k w[t,k] * y[r] gives
//   grad_y[r]         = w[t,k] * g[t]            (fp32 product, rounded to bf16)
//   grad_weights[t,k] = sum_h g[t,h] * y[r,h]    (fp32)
// and a slot without a row (masked, or outside y) gets grad_weights = 0 and
// writes no row.  (The gradient of dispatch is combine with unit weights; it
// runs combine's kernels, see ep_combine.hip.)
//
// The kernel is HBM-bound: every y row named is read once and every grad_y row
// written once, about 3 flops per 4 bytes, so the design is combine's: 8
// channels per lane, the row loads of a group of slots all in flight before
// the first product, non-temporal loads and stores for rows touched once.  A
// row of g is read once and used for all the token's slots.
#include "ep_internal.h"
#include "ep_device.h"

namespace ep {
namespace {

// Sum over the wave, the same for every lane.  The order is fixed, so equal
// inputs give equal sums.
__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
    for (int m = 32; m >= 1; m >>= 1) v += __shfl_xor(v, m);
    return v;
}

__device__ __forceinline__ void unpack8(float (&f)[8], const uint4& v) {
    f[0] = bf16_lo(v.x);
    f[1] = bf16_hi(v.x);
    f[2] = bf16_lo(v.y);
    f[3] = bf16_hi(v.y);
    f[4] = bf16_lo(v.z);
    f[5] = bf16_hi(v.z);
    f[6] = bf16_lo(v.w);
    f[7] = bf16_hi(v.w);
}

// Slots [k0, k0 + KN) of one token over one 512-channel chunk: load the rows,
// write w * g into the gradient rows and add the chunk's part of <g, y> to dot.
// Either half may be absent (y or gy null).
template <int KN>
__device__ __forceinline__ void backward_slots(float (&dot)[KN], const float (&g)[8],
                                               const uint16_t* __restrict__ y,
                                               uint16_t* __restrict__ gy, int H, int h0, bool act,
                                               int drow, float wl, int k0) {
    uint4 v[KN];
    if (y) {
#pragma unroll
        for (int i = 0; i < KN; ++i) {
            const int d = __builtin_amdgcn_readlane(drow, k0 + i);
            v[i] = make_uint4(0, 0, 0, 0);
            if (d >= 0 && act) v[i] = load_nt(y + (int64_t)d * H + h0);
        }
    }
    if (gy) {
#pragma unroll
        for (int i = 0; i < KN; ++i) {
            const int d = __builtin_amdgcn_readlane(drow, k0 + i);
            const float w = __builtin_bit_cast(
                float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, wl), k0 + i));
            if (d >= 0 && act) {
                uint4 o;
                o.x = pack_bf16x2(w * g[0], w * g[1]);
                o.y = pack_bf16x2(w * g[2], w * g[3]);
                o.z = pack_bf16x2(w * g[4], w * g[5]);
                o.w = pack_bf16x2(w * g[6], w * g[7]);
                store_nt(gy + (int64_t)d * H + h0, o);
            }
        }
    }
    if (y) {
#pragma unroll
        for (int i = 0; i < KN; ++i) {
            float f[8];
            unpack8(f, v[i]);
#pragma unroll
            for (int j = 0; j < 8; ++j) dot[i] = __builtin_fmaf(g[j], f[j], dot[i]);
        }
    }
}

// Workgroup of nw waves per token; wave i takes chunks i, i + nw, ...  Lane k
// holds slot k's row and weight.  The waves' partial dot products of a group
// of KN slots meet in LDS and are added in wave order.
template <int KN>
__global__ __launch_bounds__(kBackwardMaxThreads) void combine_backward_kernel(
    const uint16_t* __restrict__ gout, const uint16_t* __restrict__ y, int64_t nrows,
    const int32_t* __restrict__ dst_row, const float* __restrict__ w, int K, int H,
    uint16_t* __restrict__ gy, float* __restrict__ gw) {
    __shared__ float s_part[kBackwardMaxThreads / 64][KN];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int nw = blockDim.x >> 6;
    const int t = blockIdx.x;
    int drow = -1;
    float wl = 0.0f;
    if (lane < K) {
        drow = dst_row[(int64_t)t * K + lane];
        if (w) wl = w[(int64_t)t * K + lane];
        if (drow >= nrows) drow = -1;   // outside the rows: skipped like a masked slot
    }
    const int nchunk = (H + kCombineChunk - 1) / kCombineChunk;
    for (int k0 = 0; k0 < K; k0 += KN) {
        float dot[KN];
#pragma unroll
        for (int i = 0; i < KN; ++i) dot[i] = 0.0f;
        for (int c = wave; c < nchunk; c += nw) {
            const int h0 = c * kCombineChunk + lane * 8;
            const bool act = h0 < H;
            uint4 gv = make_uint4(0, 0, 0, 0);
            if (act) gv = *reinterpret_cast<const uint4*>(gout + (int64_t)t * H + h0);
            float g[8];
            unpack8(g, gv);
            backward_slots<KN>(dot, g, y, gy, H, h0, act, drow, wl, k0);
        }
        if (gw) {
#pragma unroll
            for (int i = 0; i < KN; ++i) {
                const float s = wave_sum(dot[i]);
                if (lane == i) s_part[wave][i] = s;
            }
            __syncthreads();
            if (threadIdx.x < KN && k0 + (int)threadIdx.x < K) {
                float s = 0.0f;
                for (int i = 0; i < nw; ++i) s += s_part[i][threadIdx.x];
                gw[(int64_t)t * K + k0 + threadIdx.x] = s;
            }
            __syncthreads();
        }
    }
}

}  // namespace

hipError_t launch_combine_backward(const uint16_t* gout, const uint16_t* y, int64_t nrows,
                                   const int32_t* dst_row, const float* w, int T, int K, int H,
                                   uint16_t* gy, float* gw, hipStream_t s) {
    if (T == 0) return hipSuccess;
    const int nchunk = (H + kCombineChunk - 1) / kCombineChunk;
    const int nw = nchunk < kBackwardMaxThreads / 64 ? nchunk : kBackwardMaxThreads / 64;
    const dim3 grid((unsigned)T), block(nw * 64);
#define EP_B_ARGS grid, block, 0, s, gout, y, nrows, dst_row, w, K, H, gy, gw
    switch (K) {
        case 1: hipLaunchKernelGGL(combine_backward_kernel<1>, EP_B_ARGS); break;
        case 2: hipLaunchKernelGGL(combine_backward_kernel<2>, EP_B_ARGS); break;
        case 4: hipLaunchKernelGGL(combine_backward_kernel<4>, EP_B_ARGS); break;
        case 6: hipLaunchKernelGGL(combine_backward_kernel<6>, EP_B_ARGS); break;
        default: hipLaunchKernelGGL(combine_backward_kernel<8>, EP_B_ARGS); break;
    }
#undef EP_B_ARGS
    return hipGetLastError();
}

}  // namespace ep
