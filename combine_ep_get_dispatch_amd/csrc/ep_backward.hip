// Gradient of combine on gfx950.  With g = d loss / d out and r = dst_row[t,k],
// the forward out[t] = sum_k w[t,k] * y[r] gives
//   grad_y[r]         = w[t,k] * g[t]            (fp32 product, rounded to bf16)
//   grad_weights[t,k] = sum_h g[t,h] * y[r,h]    (fp32)
// and a slot without a row (masked, or outside y) gets grad_weights = 0 and
// writes no row.  (The gradient of dispatch is combine with unit weights; it
// runs combine's kernels, see ep_combine.hip.)
//
// What bounds it.  The kernel is HBM-bound: every y row named is read once and
// every grad_y row written once, about 3 flops per 4 bytes, so the design is
// combine's: 8 channels per lane, the row loads of a group of slots all in flight before
// the first product, non-temporal loads and stores for rows touched once.  A
// row of g is read once and used for all the token's slots.
//
// Large batches of many slots run in tiles that read all their rows and then
// write all their gradient rows, so that the HBM turns between the directions
// less often.  On MI355X, tiled against one workgroup per token:
//   4096 tokens x 7168, top-8   170 / 193 us (5.9 TB/s of 6.1 for plain reads)
//   2048 x 7168, top-8           88 /  99      4096 x 7168, top-4   89 /  99
//   8192 x 4096, top-4          102 / 107      4096 x 5120, top-6   93 / 100
//   4096 x 4096, top-10         127 / 139
// but 103.4 / 102.9 at 8192 x 2048 top-8, 45 / 43 at 8192 x 1024 top-6 and
// 262 / 228 at 32768 x 4096 top-2: few channels leave a tile's waves uneven
// rounds, few slots a wave few loads in flight.  A batch that gives the CUs
// one tile each loses too (4096 x 7168, top-4 in 256 tiles: 113 / 99).
// Non-temporal accesses: 193 us, against 204 with write-through and 209 with
// ordinary stores, and 208 with ordinary loads (4096 x 7168, top-8, untiled).
#include "ep_internal.h"
#include "ep_device.h"

namespace ep {
namespace {

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

// A token's slots: lane k holds slot k's row (-1: none) and weight.
struct Slots {
    int row;
    float w;
};
__device__ __forceinline__ Slots load_slots(const int32_t* __restrict__ dst_row,
                                            const float* __restrict__ w, int64_t nrows, int64_t t,
                                            int K) {
    const int lane = threadIdx.x & 63;
    Slots s = {-1, 0.0f};
    if (lane < K) {
        s.row = dst_row[t * K + lane];
        if (w) s.w = w[t * K + lane];
        if (s.row >= nrows) s.row = -1;         // outside the rows: skipped like a masked slot
    }
    return s;
}

// Slots [k0, k0 + KN) over one 512-channel chunk: this lane's part of <g, y>.
template <int KN>
__device__ __forceinline__ void dot_rows(float (&dot)[KN], const float (&g)[8],
                                         const uint16_t* __restrict__ y, const Slots& s, int k0,
                                         int H, int h0, bool act) {
    uint4 v[KN];
#pragma unroll
    for (int i = 0; i < KN; ++i) {
        const int r = __builtin_amdgcn_readlane(s.row, k0 + i);
        v[i] = make_uint4(0, 0, 0, 0);
        if (r >= 0 && act) v[i] = load_nt(y + (int64_t)r * H + h0);
    }
#pragma unroll
    for (int i = 0; i < KN; ++i) {
        float f[8];
        unpack8(f, v[i]);
#pragma unroll
        for (int j = 0; j < 8; ++j) dot[i] = __builtin_fmaf(g[j], f[j], dot[i]);
    }
}

// Slot k's sum over the lanes; 0 for a slot without a row, whatever stands in g.
__device__ __forceinline__ float slot_sum(float dot, const Slots& s, int k) {
    const float v = seg_sum<64>(dot);
    return __builtin_amdgcn_readlane(s.row, k) >= 0 ? v : 0.0f;
}

// ... and w * g into their gradient rows.
template <int KN>
__device__ __forceinline__ void write_rows(const float (&g)[8], uint16_t* __restrict__ gy,
                                           const Slots& s, int k0, int H, int h0, bool act) {
#pragma unroll
    for (int i = 0; i < KN; ++i) {
        const int r = __builtin_amdgcn_readlane(s.row, k0 + i);
        const float w = __builtin_bit_cast(
            float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, s.w), k0 + i));
        if (r >= 0 && act) {
            uint4 o;
            o.x = pack_bf16x2(w * g[0], w * g[1]);
            o.y = pack_bf16x2(w * g[2], w * g[3]);
            o.z = pack_bf16x2(w * g[4], w * g[5]);
            o.w = pack_bf16x2(w * g[6], w * g[7]);
            store_nt(gy + (int64_t)r * H + h0, o);
        }
    }
}

__device__ __forceinline__ void load_grad(float (&g)[8], const uint16_t* __restrict__ gout,
                                          int64_t t, int H, int h0, bool act) {
    uint4 v = make_uint4(0, 0, 0, 0);
    if (act) v = *reinterpret_cast<const uint4*>(gout + t * H + h0);
    unpack8(g, v);
}

// The sums of a token's weight gradients, in both kernels: parts of the chunks
// i, i + kBackwardParts, ..., added up channel by channel in a lane, then over
// the lanes, then over the parts in order.
constexpr int kBackwardParts = kBackwardMaxThreads / 64;
__host__ __device__ __forceinline__ int num_parts(int nchunk) {
    return nchunk < kBackwardParts ? nchunk : kBackwardParts;
}

// Workgroup of nw waves per token, a wave for each part.  The parts of a group
// of KN slots meet in LDS.
template <int KN>
__global__ __launch_bounds__(kBackwardMaxThreads) void combine_backward_kernel(
    const uint16_t* __restrict__ gout, const uint16_t* __restrict__ y, int64_t nrows,
    const int32_t* __restrict__ dst_row, const float* __restrict__ w, int K, int H,
    uint16_t* __restrict__ gy, float* __restrict__ gw) {
    __shared__ float s_part[kBackwardParts][KN];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int nw = blockDim.x >> 6;
    const int64_t t = blockIdx.x;
    const int nchunk = (H + kCombineChunk - 1) / kCombineChunk;
    const Slots s = load_slots(dst_row, w, nrows, t, K);
    for (int k0 = 0; k0 < K; k0 += KN) {
        float dot[KN];
#pragma unroll
        for (int i = 0; i < KN; ++i) dot[i] = 0.0f;
        for (int c = wave; c < nchunk; c += nw) {
            const int h0 = c * kCombineChunk + lane * 8;
            const bool act = h0 < H;
            float g[8];
            load_grad(g, gout, t, H, h0, act);
            if (y) dot_rows<KN>(dot, g, y, s, k0, H, h0, act);
            if (gy) write_rows<KN>(g, gy, s, k0, H, h0, act);
        }
        if (gw) {
#pragma unroll
            for (int i = 0; i < KN; ++i) {
                const float v = slot_sum(dot[i], s, k0 + i);
                if (lane == i) s_part[wave][i] = v;
            }
            __syncthreads();
            if (threadIdx.x < KN && k0 + (int)threadIdx.x < K) {
                float v = 0.0f;
                for (int i = 0; i < nw; ++i) v += s_part[i][threadIdx.x];
                gw[t * K + k0 + threadIdx.x] = v;
            }
            __syncthreads();
        }
    }
}

// Large batches: a workgroup owns a tile of consecutive tokens and first reads
// all their rows (dot products of every (token, part) to LDS), then writes all
// their gradient rows.  g is read again for the second phase, from a cache.
template <int KN>
__global__ __launch_bounds__(kBackwardTileThreads) void combine_backward_tile_kernel(
    const uint16_t* __restrict__ gout, const uint16_t* __restrict__ y, int64_t nrows,
    const int32_t* __restrict__ dst_row, const float* __restrict__ w, int T, int K, int H,
    int tile, uint16_t* __restrict__ gy, float* __restrict__ gw) {
    extern __shared__ EP_LDS_ALIGN float s_dot[];       // [tile * parts][K]
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    constexpr int kWaves = kBackwardTileThreads / 64;
    const int64_t t0 = (int64_t)blockIdx.x * tile;
    const int nt = (int)min((int64_t)tile, T - t0);
    const int nchunk = (H + kCombineChunk - 1) / kCombineChunk;
    const int npart = num_parts(nchunk);
    for (int task = wave; task < nt * npart; task += kWaves) {
        const int tt = task / npart;
        const Slots s = load_slots(dst_row, nullptr, nrows, t0 + tt, K);
        for (int k0 = 0; k0 < K; k0 += KN) {
            float dot[KN];
#pragma unroll
            for (int i = 0; i < KN; ++i) dot[i] = 0.0f;
            for (int c = task - tt * npart; c < nchunk; c += kBackwardParts) {
                const int h0 = c * kCombineChunk + lane * 8;
                const bool act = h0 < H;
                float g[8];
                load_grad(g, gout, t0 + tt, H, h0, act);
                dot_rows<KN>(dot, g, y, s, k0, H, h0, act);
            }
#pragma unroll
            for (int i = 0; i < KN; ++i) {
                const float v = slot_sum(dot[i], s, k0 + i);
                if (lane == i && k0 + i < K) s_dot[task * K + k0 + i] = v;
            }
        }
    }
    __syncthreads();
    for (int task = wave; task < nt * nchunk; task += kWaves) {
        const int tt = task / nchunk;
        const int h0 = (task - tt * nchunk) * kCombineChunk + lane * 8;
        const bool act = h0 < H;
        const Slots s = load_slots(dst_row, w, nrows, t0 + tt, K);
        float g[8];
        load_grad(g, gout, t0 + tt, H, h0, act);
        for (int k0 = 0; k0 < K; k0 += KN) write_rows<KN>(g, gy, s, k0, H, h0, act);
    }
    for (int i = threadIdx.x; i < nt * K; i += kBackwardTileThreads) {
        const int tt = i / K, k = i - tt * K;
        float v = 0.0f;
        for (int c = 0; c < npart; ++c) v += s_dot[(tt * npart + c) * K + k];
        gw[t0 * K + i] = v;
    }
}

template <int KN>
hipError_t launch_backward_k(const uint16_t* gout, const uint16_t* y, int64_t nrows,
                             const int32_t* dst_row, const float* w, int T, int K, int H,
                             uint16_t* gy, float* gw, hipStream_t s) {
    const int nchunk = (H + kCombineChunk - 1) / kCombineChunk;
    // Tiles of as many slots as keep 8 per wave, while the batch still gives
    // every CU of a 256-CU part two tiles, where both gradients are asked for.
    int tile = kBackwardTileSlots / K;
    if (tile > T / kBackwardMinTiles) tile = T / kBackwardMinTiles;
    const int npart = num_parts(nchunk);
    const size_t lds = (size_t)tile * npart * K * sizeof(float);
    if (y && gy && gw && K >= kBackwardTileMinK && H >= kBackwardTileMinH &&
        2 * tile * K >= kBackwardTileSlots) {
        hipLaunchKernelGGL(combine_backward_tile_kernel<KN>,
                           dim3((unsigned)(((int64_t)T + tile - 1) / tile)),
                           dim3(kBackwardTileThreads), lds, s, gout, y, nrows, dst_row, w, T, K, H,
                           tile, gy, gw);
    } else {
        hipLaunchKernelGGL(combine_backward_kernel<KN>, dim3((unsigned)T), dim3(npart * 64), 0, s,
                           gout, y, nrows, dst_row, w, K, H, gy, gw);
    }
    return hipGetLastError();
}

hipError_t launch_slice(const uint16_t* gout, const uint16_t* y, int64_t nrows,
                        const int32_t* dst_row, const float* w, int T, int K, int H, uint16_t* gy,
                        float* gw, hipStream_t s) {
#define EP_B_ARGS gout, y, nrows, dst_row, w, T, K, H, gy, gw, s
    switch (K) {
        case 1: return launch_backward_k<1>(EP_B_ARGS);
        case 2: return launch_backward_k<2>(EP_B_ARGS);
        case 4: return launch_backward_k<4>(EP_B_ARGS);
        case 6: return launch_backward_k<6>(EP_B_ARGS);
        default: return launch_backward_k<8>(EP_B_ARGS);
    }
#undef EP_B_ARGS
}

}  // namespace

hipError_t launch_combine_backward(const uint16_t* gout, const uint16_t* y, int64_t nrows,
                                   const int32_t* dst_row, const float* w, int T, int K, int H,
                                   uint16_t* gy, float* gw, hipStream_t s) {
    const int64_t slice = max_launch_tokens(kBackwardMaxThreads);
    for (int64_t t = 0; t < T; t += slice) {
        const int n = (int)(T - t < slice ? T - t : slice);
        const hipError_t e = launch_slice(gout + t * H, y, nrows, dst_row + t * K,
                                          w ? w + t * K : nullptr, n, K, H, gy,
                                          gw ? gw + t * K : nullptr, s);
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

}  // namespace ep
