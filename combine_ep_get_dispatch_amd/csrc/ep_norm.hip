// Root-mean-square norm of the tokens ahead of the layer, and its gradient, on
// gfx950.  With h = x, or bf16(x + residual):
//   inv = 1 / sqrt(mean over channels of h^2 + eps),   y = h * inv * weight,
// y rounded once, to bf16, or to E4M3 with a scale per 128 channels as dispatch
// writes its rows, or to both.  h is what the next layer's residual reads and
// what the gradient is taken from, so the norm sees it as stored.  With
// n = h * inv and gn = grad_y * weight:
//   grad_h = inv * (gn - n * mean(gn * n)) + grad_residual,
//   grad_weight = sum over tokens of grad_y * n.
//
// A row is read once, kept in registers across its sum, and written once, so both are
// bound by HBM where a row fills its workgroup and fits its registers: 4.9-5.9 TB/s
// of reads and writes forward from 512 channels on, 4.5-6.0 TB/s of the gradient at 1024
// to 16384.  Beside that (in us, floor in brackets, with residuals): narrow rows leave most
// of their workgroup idle, 65536 x 128 forward 26 (11), gradient 80 (11), whose workgroups
// also take their rows one after the other; and the gradient of more than 16384 channels
// keeps row and weight's sums in 412-436 bytes of scratch a lane, 1024 x 32768 190 (44).
#include "ep_internal.h"
#include "ep_device.h"

#include <cfloat>
#include <type_traits>

namespace ep {
namespace {

struct NormArgs {
    const uint16_t* x;
    const uint16_t* res;
    const void* w;
    float eps;
    int H;
    uint16_t* y;
    uint8_t* codes;
    float* scales;
    uint16_t* res_out;
    float* inv;
};

struct NormBackArgs {
    const uint16_t* gy;
    const uint16_t* x;
    const void* w;
    const float* inv;
    const uint16_t* gres;
    int T, H;
    uint16_t* gx;
    float* part;     // [gridDim.x][H]
};

// A weight of bf16 or fp32, eight channels.
template <bool W32>
struct Weight8 {
    uint4 a, b;
};
template <bool W32>
__device__ __forceinline__ Weight8<W32> load_weight(const void* w, int c) {
    Weight8<W32> r;
    if constexpr (W32) {
        r.a = static_cast<const uint4*>(w)[2 * c];
        r.b = static_cast<const uint4*>(w)[2 * c + 1];
    } else {
        r.a = static_cast<const uint4*>(w)[c];
    }
    return r;
}
template <bool W32>
__device__ __forceinline__ void unpack_weight(float (&f)[8], const Weight8<W32>& w) {
    if constexpr (W32) {
        const uint32_t u[8] = {w.a.x, w.a.y, w.a.z, w.a.w, w.b.x, w.b.y, w.b.z, w.b.w};
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = __uint_as_float(u[i]);
    } else {
        unpack8(f, w.a);
    }
}

// Sum over the workgroup, the same in every thread, in an order fixed by its size.
// s holds 16 floats; the caller sees to it that no wave still reads it.
__device__ __forceinline__ float block_sum(float v, float* s) {
    v = seg_sum<64>(v);
    if (blockDim.x == 64) return v;
    if ((threadIdx.x & 63) == 0) s[threadIdx.x >> 6] = v;
    __syncthreads();
    const int waves = blockDim.x >> 6, i = threadIdx.x & 15;
    return seg_sum<16>(i < waves ? s[i] : 0.0f);
}

// Where the mean of the squares (and eps) is at least this, what squares lost below
// 2^-126, up to 2^-150 each, does not count.
constexpr float kLeastMean = 0x1p-80f;

// One row per workgroup; a thread holds chunks of 8 channels tid, tid + blockDim, ...,
// NC of them, so 16 neighbouring lanes hold 128 neighbouring channels, one scale.
template <int NC, bool W32>
__global__ __launch_bounds__(1024) void rms_norm_kernel(const NormArgs p) {
    const int kThreads = blockDim.x;
    __shared__ float part[2][16];
    const int chunks = p.H / 8;
    const int64_t row = blockIdx.x;
    const uint4* x = reinterpret_cast<const uint4*>(p.x + row * p.H);
    uint4 v[NC];
    Weight8<W32> w[NC];
#pragma unroll
    for (int i = 0; i < NC; ++i)
        v[i] = load_nt(x + min((int)threadIdx.x + i * kThreads, chunks - 1));
    if (p.res) {
        const uint4* res = reinterpret_cast<const uint4*>(p.res + row * p.H);
        uint4 r[NC];
#pragma unroll
        for (int i = 0; i < NC; ++i) r[i] = load_nt(res + min((int)threadIdx.x + i * kThreads, chunks - 1));
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            float a[8], b[8];
            unpack8(a, v[i]);
            unpack8(b, r[i]);
#pragma unroll
            for (int j = 0; j < 8; ++j) a[j] += b[j];
            v[i] = pack8(a);
            const int c = threadIdx.x + i * kThreads;
            if (c < chunks) reinterpret_cast<uint4*>(p.res_out + row * p.H)[c] = v[i];
        }
    }
#pragma unroll
    for (int i = 0; i < NC; ++i)
        w[i] = load_weight<W32>(p.w, min((int)threadIdx.x + i * kThreads, chunks - 1));
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < NC; ++i) {
        float a[8], s = 0.0f;
        unpack8(a, v[i]);
#pragma unroll
        for (int j = 0; j < 8; ++j) s = __builtin_fmaf(a[j], a[j], s);
        sum += (int)threadIdx.x + i * kThreads < chunks ? s : 0.0f;
    }
    sum = block_sum(sum, part[0]);
    const float mean = sum / (float)p.H + p.eps;
    float inv = 1.0f / sqrtf(mean), inv_out = inv;
    if (!(mean >= kLeastMean && mean <= FLT_MAX)) {      // the same in every thread
        // Squares that pass fp32's range, or may have lost bits below it: once more, of
        // channels times a power of two.  2^90 h is exact in bf16 and takes h's place
        // (1 / rms itself may pass the range); 2^-72 h might not be.
        const bool up = mean < kLeastMean;
        const float scale = up ? 0x1p90f : 0x1p-72f;
        sum = 0.0f;
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            float a[8], s = 0.0f;
            unpack8(a, v[i]);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                a[j] *= scale;
                s = __builtin_fmaf(a[j], a[j], s);
            }
            if (up) v[i] = pack8(a);
            sum += (int)threadIdx.x + i * kThreads < chunks ? s : 0.0f;
        }
        sum = block_sum(sum, part[1]);
        inv = 1.0f / sqrtf(sum / (float)p.H + p.eps * scale * scale);
        inv_out = inv * scale;
        if (!up) inv = inv_out;
    }
    if (p.inv && threadIdx.x == 0) p.inv[row] = inv_out;
#pragma unroll
    for (int i = 0; i < NC; ++i) {
        const int c = threadIdx.x + i * kThreads;
        if (c >= chunks) break;          // whole groups of 16 lanes where codes are written
        float a[8], f[8];
        unpack8(a, v[i]);
        unpack_weight<W32>(f, w[i]);
#pragma unroll
        for (int j = 0; j < 8; ++j) a[j] = a[j] * inv * f[j];
        if (p.y) reinterpret_cast<uint4*>(p.y + row * p.H)[c] = pack8(a);
        if (p.codes) {
            float scale;
            const uint2 q = quantise8(a, scale);
            reinterpret_cast<uint2*>(p.codes + row * p.H)[c] = q;
            if ((threadIdx.x & 15) == 0) p.scales[row * (p.H / 128) + c / 16] = scale;
        }
    }
}

// Rows blockIdx.x, blockIdx.x + gridDim.x, ...; a thread's channels as above.
// It sums its channels' grad_weight over the workgroup's rows in registers;
// sum_parts_kernel adds the workgroups' sums up in their order.
template <int NC, bool W32>
__global__ __launch_bounds__(1024) void rms_norm_backward_kernel(const NormBackArgs p) {
    const int kThreads = blockDim.x;
    __shared__ float part[2][16];
    const int chunks = p.H / 8;
    float gw[NC][8];
    Weight8<W32> w[NC];
#pragma unroll
    for (int i = 0; i < NC; ++i) {
        w[i] = load_weight<W32>(p.w, min((int)threadIdx.x + i * kThreads, chunks - 1));
#pragma unroll
        for (int j = 0; j < 8; ++j) gw[i][j] = 0.0f;
    }
    const float per = 1.0f / (float)p.H;
    // a row's loads are asked for while the row before it is worked on, where the
    // registers hold both
    constexpr bool kAhead = NC == 1;
    uint4 v[NC], g[NC], r[NC];
    float inv;
    auto load = [&](int64_t row) {
        const uint4* x = reinterpret_cast<const uint4*>(p.x + row * p.H);
        const uint4* gy = reinterpret_cast<const uint4*>(p.gy + row * p.H);
        const uint4* gr = reinterpret_cast<const uint4*>(p.gres + row * p.H);
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            const int c = min((int)threadIdx.x + i * kThreads, chunks - 1);
            v[i] = load_nt(x + c);
            g[i] = load_nt(gy + c);
            if (p.gres) r[i] = load_nt(gr + c);
        }
        inv = p.inv[row];
    };
    if (kAhead) load(blockIdx.x);
    int turn = 0;
    for (int64_t row = blockIdx.x; row < p.T; row += gridDim.x, turn ^= 1) {
        uint4 nb[NC], gn[NC], rb[NC];     // n and grad_y * weight are made of these again
        if (!kAhead) load(row);
        const float inv_row = inv;
        float sum = 0.0f;
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            nb[i] = v[i];
            gn[i] = g[i];
            rb[i] = r[i];
        }
        if (kAhead) load(row + gridDim.x < p.T ? row + gridDim.x : row);
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            float a[8], b[8], f[8], s = 0.0f;
            unpack8(a, nb[i]);
            unpack8(b, gn[i]);
            unpack_weight<W32>(f, w[i]);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float n = a[j] * inv_row;
                gw[i][j] = __builtin_fmaf(b[j], n, gw[i][j]);
                s = __builtin_fmaf(b[j] * f[j], n, s);
            }
            sum += (int)threadIdx.x + i * kThreads < chunks ? s : 0.0f;
        }
        const float mean = block_sum(sum, part[turn]) * per;
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            const int c = threadIdx.x + i * kThreads;
            if (c >= chunks) break;
            float a[8], b[8], f[8], o[8];
            unpack8(a, nb[i]);
            unpack8(b, gn[i]);
            unpack_weight<W32>(f, w[i]);
#pragma unroll
            for (int j = 0; j < 8; ++j)
                o[j] = inv_row * (b[j] * f[j] - a[j] * inv_row * mean);
            if (p.gres) {
                unpack8(f, rb[i]);
#pragma unroll
                for (int j = 0; j < 8; ++j) o[j] += f[j];
            }
            reinterpret_cast<uint4*>(p.gx + row * p.H)[c] = pack8(o);
        }
    }
#pragma unroll
    for (int i = 0; i < NC; ++i) {
        const int c = threadIdx.x + i * kThreads;
        if (c >= chunks) break;
        float4* o = reinterpret_cast<float4*>(p.part + (int64_t)blockIdx.x * p.H + c * 8);
        o[0] = make_float4(gw[i][0], gw[i][1], gw[i][2], gw[i][3]);
        o[1] = make_float4(gw[i][4], gw[i][5], gw[i][6], gw[i][7]);
    }
}

// out[c] = sum over the parts, four channels a thread; 64 threads share a channel's
// parts, each every 64th of them, and add up in a fixed order.
constexpr int kSumThreads = 1024, kSumShare = 64, kSumColumns = kSumThreads / kSumShare;
__global__ __launch_bounds__(kSumThreads) void sum_parts_kernel(const float* part, int parts,
                                                                int H, float* out) {
    __shared__ float4 s[kSumThreads];
    const int col = threadIdx.x % kSumColumns, c = (blockIdx.x * kSumColumns + col) * 4;
    float4 t = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (c < H) {
#pragma unroll 4
        for (int i = threadIdx.x / kSumColumns; i < parts; i += kSumShare) {
            const float4 v = *reinterpret_cast<const float4*>(part + (int64_t)i * H + c);
            t.x += v.x;
            t.y += v.y;
            t.z += v.z;
            t.w += v.w;
        }
    }
    s[threadIdx.x] = t;
    for (int half = kSumThreads / 2; half >= kSumColumns; half /= 2) {
        __syncthreads();
        if ((int)threadIdx.x < half) {
            const float4 v = s[threadIdx.x + half];
            t.x += v.x;
            t.y += v.y;
            t.z += v.z;
            t.w += v.w;
            s[threadIdx.x] = t;
        }
    }
    if ((int)threadIdx.x < kSumColumns && c < H) *reinterpret_cast<float4*>(out + c) = t;
}

// Chunks per thread for rows of `chunks` chunks in workgroups of up to `threads`
// threads, and the threads that this takes.
template <typename F>
void by_width(int chunks, int threads, F&& f) {
    auto run = [&](auto nc) {
        constexpr int NC = decltype(nc)::value;
        f(nc, ((chunks + NC - 1) / NC + 63) / 64 * 64);
    };
    if (chunks <= threads)
        run(std::integral_constant<int, 1>{});
    else if (chunks <= 2 * threads || (chunks <= 2048 && threads < 1024))
        run(std::integral_constant<int, 2>{});
    else
        run(std::integral_constant<int, 4>{});
}

}  // namespace

hipError_t launch_rms_norm(const uint16_t* x, const uint16_t* res, const void* w, bool w32, int T,
                           int H, float eps, uint16_t* y, uint8_t* codes, float* scales,
                           uint16_t* res_out, float* inv, hipStream_t s) {
    by_width(H / 8, kNormThreads, [&](auto nc, int threads) {
        constexpr int NC = decltype(nc)::value;
        const int64_t most = max_launch_tokens(threads);
        for (int64_t t = 0; t < T; t += most) {
            const int64_t at = t * H;
            const NormArgs p = {x + at,
                                res ? res + at : nullptr,
                                w,
                                eps,
                                H,
                                y ? y + at : nullptr,
                                codes ? codes + at : nullptr,
                                codes ? scales + t * (H / 128) : nullptr,
                                res ? res_out + at : nullptr,
                                inv ? inv + t : nullptr};
            const dim3 grid((unsigned)(T - t < most ? T - t : most));
            if (w32)
                hipLaunchKernelGGL((rms_norm_kernel<NC, true>), grid, dim3(threads), 0, s, p);
            else
                hipLaunchKernelGGL((rms_norm_kernel<NC, false>), grid, dim3(threads), 0, s, p);
        }
    });
    return hipGetLastError();
}

hipError_t launch_rms_norm_backward(const uint16_t* gy, const uint16_t* x, const void* w, bool w32,
                                    const float* inv, const uint16_t* gres, int T, int H,
                                    uint16_t* gx, float* gw, float* ws, hipStream_t s) {
    const int parts = norm_parts(T);
    if (T > 0) {
        const NormBackArgs p = {gy, x, w, inv, gres, T, H, gx, ws};
        by_width(H / 8, 1024, [&](auto nc, int threads) {
            constexpr int NC = decltype(nc)::value;
            if (w32)
                hipLaunchKernelGGL((rms_norm_backward_kernel<NC, true>), dim3(parts),
                                   dim3(threads), 0, s, p);
            else
                hipLaunchKernelGGL((rms_norm_backward_kernel<NC, false>), dim3(parts),
                                   dim3(threads), 0, s, p);
        });
    }
    const int per = kSumColumns * 4;
    hipLaunchKernelGGL(sum_parts_kernel, dim3((H + per - 1) / per), dim3(kSumThreads), 0, s, ws,
                       parts, H, gw);
    return hipGetLastError();
}

}  // namespace ep
