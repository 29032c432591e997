// The experts' products with 4-bit weights on gfx950, over the rows that
// dispatch writes:
//   y[r, n] = sum_i x[r, i] * (q[e, n, i] - z[e, i/G, n]) * s[e, i/G, n],
// e the expert of row r, q a 4-bit code, z the group's zero point (8 without
// one) and s its scale; x is bf16, or E4M3 codes with one fp32 scale per 128
// channels.  With SWIGLU the weights hold 2N channels and
//   y[r, n] = silu(gate_n) * up_n,  gate = channels [0, N), up = [N, 2N),
// taken from the fp32 sums and rounded once.
//
// What bounds it.  In decode an expert has a few rows: 2 * rows flops per
// weight of half a byte, so the product is bound by reading the weights once
// from HBM, and everything else has to fit beside that stream.
//
// Codes to matrix operands.  A group's sum splits into
//   sum x (q - z) = sum x q - z sum x,
// so the matrix instructions multiply x with the bare codes, and zero point
// and scale act on a group's fp32 sums, four channels and one row per lane:
//  - E4M3 rows: a byte 0..15 is, read as E4M3, q * 2^-9 exactly (the format's
//    subnormals and its first binade), so a mask and a shift make four
//    operands each.
//  - bf16 rows: 0x4300 | q is the bf16 number 128 + q exactly; the sum takes
//    z + 128 instead of z.
// sum x comes from one more matrix instruction with a row of ones.  The
// products are exact and the sums fp32; the 128 costs five bits of the 24
// before a result that is rounded to 8.
//
// Layout.  Weights are the A operand (16 channels by k), rows the B operand
// (k by 16 rows), so a lane ends with four neighbouring channels of one row.
// A lane loads 16 bytes, 32 codes, of one channel: a wave's load covers 64
// bytes of 16 channels.  Matrix instructions sum over the four lane groups;
// where a group of scales is shorter than the 128 codes that these hold, a
// 4x4 transpose between them (two swaps of half rows, two of rows) first gives
// every instruction 32 neighbouring codes.
//
// A workgroup owns a tile of channels of one expert for a block of its rows;
// its waves take every kWaves-th block of 128 input channels and their sums
// meet in LDS, in wave order.
#include "ep_internal.h"
#include "ep_device.h"

namespace ep {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

struct ExpertArgs {
    const uint8_t* x;
    const float* xs;
    int64_t num_rows;
    const int32_t* offsets;
    const int32_t* counts;
    int capacity;
    int I, N;
    const uint8_t* w;
    const uint16_t* scales;
    const uint8_t* zeros;
    uint16_t* y;
};

// Dword j of lane group g becomes dword g of lane group j.
__device__ __forceinline__ void transpose_groups(i32x4& v) {
    auto a = __builtin_amdgcn_permlane32_swap((unsigned)v[0], (unsigned)v[2], false, false);
    auto b = __builtin_amdgcn_permlane32_swap((unsigned)v[1], (unsigned)v[3], false, false);
    auto c = __builtin_amdgcn_permlane16_swap(a[0], b[0], false, false);
    auto d = __builtin_amdgcn_permlane16_swap(a[1], b[1], false, false);
    v[0] = (int)c[0];
    v[1] = (int)c[1];
    v[2] = (int)d[0];
    v[3] = (int)d[1];
}

// Codes 0..7 of a dword as two dwords of bytes: (0,2,4,6) and (1,3,5,7).
__device__ __forceinline__ void codes_e4m3(int (&o)[2], int v) {
    o[0] = v & 0x0f0f0f0f;
    o[1] = (int)((unsigned)v >> 4) & 0x0f0f0f0f;
}
// ... and as bf16 pairs 128 + q: (0,4) (1,5) (2,6) (3,7).
__device__ __forceinline__ i32x4 codes_bf16(int v) {
    const unsigned u = (unsigned)v;
    i32x4 o;
    o[0] = (int)((u & 0x000f000fu) | 0x43004300u);
    o[1] = (int)(((u >> 4) & 0x000f000fu) | 0x43004300u);
    o[2] = (int)(((u >> 8) & 0x000f000fu) | 0x43004300u);
    o[3] = (int)(((u >> 12) & 0x000f000fu) | 0x43004300u);
    return o;
}
// Eight E4M3 values (two dwords) and eight bf16 values in the same orders.
__device__ __forceinline__ void order_e4m3(int& a, int& b) {
    const int lo = (int)__builtin_amdgcn_perm((unsigned)b, (unsigned)a, 0x06040200u);
    const int hi = (int)__builtin_amdgcn_perm((unsigned)b, (unsigned)a, 0x07050301u);
    a = lo;
    b = hi;
}
__device__ __forceinline__ i32x4 order_bf16(const i32x4& v) {
    i32x4 o;
    o[0] = (int)__builtin_amdgcn_perm((unsigned)v[2], (unsigned)v[0], 0x05040100u);
    o[1] = (int)__builtin_amdgcn_perm((unsigned)v[2], (unsigned)v[0], 0x07060302u);
    o[2] = (int)__builtin_amdgcn_perm((unsigned)v[3], (unsigned)v[1], 0x05040100u);
    o[3] = (int)__builtin_amdgcn_perm((unsigned)v[3], (unsigned)v[1], 0x07060302u);
    return o;
}

__device__ __forceinline__ f32x4 mfma128(const i32x8& a, const i32x8& b, const f32x4& c) {
    // both E4M3; block scales 2^9 for the codes (so that they count as q), 2^0 for the rows
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, c, 0, 0, 0, 127 + 9, 0, 127);
}
__device__ __forceinline__ f32x4 mfma32(const i32x4& a, const i32x4& b, const f32x4& c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a),
                                                   __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}
__device__ __forceinline__ f32x4 mfma32_e4m3(const int (&a)[2], const int (&b)[2],
                                             const f32x4& c) {
    const long la = (long)((uint64_t)(unsigned)a[1] << 32 | (unsigned)a[0]);
    const long lb = (long)((uint64_t)(unsigned)b[1] << 32 | (unsigned)b[0]);
    return __builtin_amdgcn_mfma_f32_16x16x32_fp8_fp8(la, lb, c, 0, 0, 0);
}

// RT row tiles of 16 rows from row r0 of the expert (n rows from `begin`), the
// channel tile at channel n0 (of each half, with SWIGLU).
template <bool FP8, int G, bool ZP, bool SWIGLU, int RT>
__device__ __forceinline__ void expert_tile(const ExpertArgs& p, int e, int n0, int64_t begin,
                                            int n, int r0, f32x4* s_part) {
    constexpr int CT = kExpertTiles;
    constexpr bool kWide = FP8 && G == 128;     // one instruction per 128 codes
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int lg = lane >> 4, lr = lane & 15;
    const int I = p.I, N = p.N;
    const int W = SWIGLU ? 2 * N : N;
    const int NG = I / G;
    const int nblk = (I + 127) / 128;

    // first channel of tile ct, and the channels this lane loads and scales
    const uint8_t* wrow[CT];
    int sch[CT];
#pragma unroll
    for (int ct = 0; ct < CT; ++ct) {
        const int half = SWIGLU ? ct / (CT / 2) : 0;
        const int c0 = n0 + (SWIGLU ? ct % (CT / 2) : ct) * 16;
        // past the last channel: any channel, its sums are not stored
        wrow[ct] = p.w + ((int64_t)e * W + half * N + min(c0 + lr, N - 1)) * (I / 2) + lg * 16;
        sch[ct] = half * N + min(c0 + lg * 4, N - 4);
    }
    const uint16_t* sc = p.scales + (int64_t)e * NG * W;
    const uint8_t* zr = ZP ? p.zeros + (int64_t)e * NG * W : nullptr;
    int64_t xrow[RT];
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) xrow[rt] = begin + min(r0 + rt * 16 + lr, n - 1);

    f32x4 acc[CT][RT];
#pragma unroll
    for (int ct = 0; ct < CT; ++ct)
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) acc[ct][rt] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

    // scale a group's sums (d, and sx of the ones) into acc
    auto apply = [&](int ct, int rt, int g, const f32x4& d, float sx, float xsc) {
        const uint2 sv = *reinterpret_cast<const uint2*>(sc + (int64_t)g * W + sch[ct]);
        float z[4] = {8.0f, 8.0f, 8.0f, 8.0f};
        if constexpr (ZP) {
            const unsigned zv = *reinterpret_cast<const unsigned*>(zr + (int64_t)g * W + sch[ct]);
#pragma unroll
            for (int i = 0; i < 4; ++i) z[i] = (float)((zv >> (8 * i)) & 15u);
        }
        const float s[4] = {bf16_lo(sv.x), bf16_hi(sv.x), bf16_lo(sv.y), bf16_hi(sv.y)};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float t;
            if constexpr (kWide)
                t = __builtin_fmaf(-z[i], sx, d[i]);
            else if constexpr (FP8)
                t = __builtin_fmaf(512.0f, d[i], -z[i] * sx);
            else
                t = __builtin_fmaf(-(z[i] + 128.0f), sx, d[i]);
            acc[ct][rt][i] = __builtin_fmaf(FP8 ? s[i] * xsc : s[i], t, acc[ct][rt][i]);
        }
    };

    for (int b = wave; b < nblk; b += kExpertWaves) {
        const int kb = b * 128;
        i32x4 wv[CT];
        const bool whole = G == 128 || kb + lg * 32 < I;    // the last block may be short
#pragma unroll
        for (int ct = 0; ct < CT; ++ct) {
            wv[ct] = i32x4{0, 0, 0, 0};
            if (whole) wv[ct] = *reinterpret_cast<const i32x4*>(wrow[ct] + b * 64);
        }
        float xsc[RT];
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) xsc[rt] = FP8 ? p.xs[xrow[rt] * (I / 128) + b] : 1.0f;
        const f32x4 zero = {0.0f, 0.0f, 0.0f, 0.0f};

        if constexpr (kWide) {
            i32x8 xv[RT];
            float sx[RT];
            i32x8 ones;
#pragma unroll
            for (int i = 0; i < 8; ++i) ones[i] = 0x38383838;    // 1.0, and 2^-9 undoes the scale
#pragma unroll
            for (int rt = 0; rt < RT; ++rt) {
                const i32x4* xp =
                    reinterpret_cast<const i32x4*>(p.x + xrow[rt] * I + kb + lg * 32);
                const i32x4 a = xp[0], c = xp[1];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    xv[rt][i] = a[i];
                    xv[rt][4 + i] = c[i];
                }
#pragma unroll
                for (int i = 0; i < 8; i += 2) {
                    int u = xv[rt][i], v = xv[rt][i + 1];
                    order_e4m3(u, v);
                    xv[rt][i] = u;
                    xv[rt][i + 1] = v;
                }
                sx[rt] = mfma128(ones, xv[rt], zero)[0] * 0.001953125f;
            }
#pragma unroll
            for (int ct = 0; ct < CT; ++ct) {
                i32x8 a;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    int o[2];
                    codes_e4m3(o, wv[ct][i]);
                    a[2 * i] = o[0];
                    a[2 * i + 1] = o[1];
                }
#pragma unroll
                for (int rt = 0; rt < RT; ++rt)
                    apply(ct, rt, b, mfma128(a, xv[rt], zero), sx[rt], xsc[rt]);
            }
        } else {
            if constexpr (G < 128) {
#pragma unroll
                for (int ct = 0; ct < CT; ++ct) transpose_groups(wv[ct]);
            }
            constexpr int kSteps = G / 32;     // matrix instructions per group of scales
            const i32x4 ones = {0x3f803f80, 0x3f803f80, 0x3f803f80, 0x3f803f80};
            const int ones8[2] = {0x38383838, 0x38383838};
#pragma unroll
            for (int j0 = 0; j0 < 4; j0 += kSteps) {
                if (G < 128 && kb + j0 * 32 >= I) break;
                f32x4 d[CT][RT], sx[RT];
#pragma unroll
                for (int rt = 0; rt < RT; ++rt) {
                    sx[rt] = zero;
#pragma unroll
                    for (int ct = 0; ct < CT; ++ct) d[ct][rt] = zero;
                }
#pragma unroll
                for (int j = j0; j < j0 + kSteps; ++j) {
                    // codes of step j in this lane: 8 from here
                    const int k = kb + (G < 128 ? j * 32 + lg * 8 : lg * 32 + j * 8);
                    if constexpr (FP8) {
                        int xv[RT][2];
#pragma unroll
                        for (int rt = 0; rt < RT; ++rt) {
                            const uint2 v =
                                *reinterpret_cast<const uint2*>(p.x + xrow[rt] * I + k);
                            xv[rt][0] = (int)v.x;
                            xv[rt][1] = (int)v.y;
                            order_e4m3(xv[rt][0], xv[rt][1]);
                            sx[rt] = mfma32_e4m3(ones8, xv[rt], sx[rt]);
                        }
#pragma unroll
                        for (int ct = 0; ct < CT; ++ct) {
                            int a[2];
                            codes_e4m3(a, wv[ct][j]);
#pragma unroll
                            for (int rt = 0; rt < RT; ++rt)
                                d[ct][rt] = mfma32_e4m3(a, xv[rt], d[ct][rt]);
                        }
                    } else {
                        i32x4 xv[RT];
#pragma unroll
                        for (int rt = 0; rt < RT; ++rt) {
                            xv[rt] = order_bf16(*reinterpret_cast<const i32x4*>(
                                p.x + (xrow[rt] * I + k) * 2));
                            sx[rt] = mfma32(ones, xv[rt], sx[rt]);
                        }
#pragma unroll
                        for (int ct = 0; ct < CT; ++ct) {
                            const i32x4 a = codes_bf16(wv[ct][j]);
#pragma unroll
                            for (int rt = 0; rt < RT; ++rt)
                                d[ct][rt] = mfma32(a, xv[rt], d[ct][rt]);
                        }
                    }
                }
                const int g = (kb + j0 * 32) / G;
#pragma unroll
                for (int ct = 0; ct < CT; ++ct)
#pragma unroll
                    for (int rt = 0; rt < RT; ++rt)
                        apply(ct, rt, g, d[ct][rt], sx[rt][0], xsc[rt]);
            }
        }
    }

    // the waves' sums, in wave order; wave i finishes tiles i, i + kExpertWaves, ...
    constexpr int kTiles = CT * RT;
#pragma unroll
    for (int ct = 0; ct < CT; ++ct)
#pragma unroll
        for (int rt = 0; rt < RT; ++rt)
            s_part[(wave * kTiles + ct * RT + rt) * 64 + lane] = acc[ct][rt];
    __syncthreads();
    constexpr int kOut = SWIGLU ? kTiles / 2 : kTiles;
    for (int o = wave; o < kOut; o += kExpertWaves) {
        const int ct = o / RT, rt = o % RT;
        f32x4 a = {0.0f, 0.0f, 0.0f, 0.0f}, u = a;
        for (int v = 0; v < kExpertWaves; ++v) a += s_part[(v * kTiles + o) * 64 + lane];
        if constexpr (SWIGLU) {
            for (int v = 0; v < kExpertWaves; ++v)
                u += s_part[(v * kTiles + kOut + o) * 64 + lane];
#pragma unroll
            for (int i = 0; i < 4; ++i) a[i] = a[i] / (1.0f + expf(-a[i])) * u[i];
        }
        const int row = r0 + rt * 16 + lr, c = n0 + ct * 16 + lg * 4;
        if (row < n && c < N) {
            const uint2 v = make_uint2(pack_bf16x2(a[0], a[1]), pack_bf16x2(a[2], a[3]));
            *reinterpret_cast<uint2*>(p.y + (begin + row) * N + c) = v;
        }
    }
    __syncthreads();
}

template <bool FP8, int G, bool ZP, bool SWIGLU>
__global__ __launch_bounds__(kExpertWaves * 64) void expert_linear_kernel(const ExpertArgs p) {
    __shared__ f32x4 s_part[kExpertWaves * kExpertTiles * kExpertRowTiles * 64];
    const int e = blockIdx.y;
    int64_t begin = p.offsets ? (int64_t)p.offsets[e] : (int64_t)e * p.capacity;
    int64_t end = begin + (p.offsets ? p.counts[e] : min(p.counts[e], p.capacity));
    if (begin < 0) begin = 0;
    if (end > p.num_rows) end = p.num_rows;
    if (end <= begin) return;
    const int n = (int)(end - begin);
    const int n0 = blockIdx.x * (kExpertTiles * 16 / (SWIGLU ? 2 : 1));
    for (int r0 = blockIdx.z * kExpertRowTiles * 16; r0 < n;
         r0 += gridDim.z * kExpertRowTiles * 16) {
        if (n - r0 <= 16)
            expert_tile<FP8, G, ZP, SWIGLU, 1>(p, e, n0, begin, n, r0, s_part);
        else
            expert_tile<FP8, G, ZP, SWIGLU, kExpertRowTiles>(p, e, n0, begin, n, r0, s_part);
    }
}

template <bool FP8, int G>
void launch_g(dim3 grid, hipStream_t s, const ExpertArgs& p, bool swiglu) {
    const dim3 block(kExpertWaves * 64);
    if (p.zeros) {
        if (swiglu)
            hipLaunchKernelGGL((expert_linear_kernel<FP8, G, true, true>), grid, block, 0, s, p);
        else
            hipLaunchKernelGGL((expert_linear_kernel<FP8, G, true, false>), grid, block, 0, s, p);
    } else {
        if (swiglu)
            hipLaunchKernelGGL((expert_linear_kernel<FP8, G, false, true>), grid, block, 0, s, p);
        else
            hipLaunchKernelGGL((expert_linear_kernel<FP8, G, false, false>), grid, block, 0, s, p);
    }
}

template <bool FP8>
void launch_t(int G, dim3 grid, hipStream_t s, const ExpertArgs& p, bool swiglu) {
    switch (G) {
        case 32: launch_g<FP8, 32>(grid, s, p, swiglu); break;
        case 64: launch_g<FP8, 64>(grid, s, p, swiglu); break;
        default: launch_g<FP8, 128>(grid, s, p, swiglu); break;
    }
}

}  // namespace

hipError_t launch_expert_linear_w4(const void* x, const float* xs, bool fp8, int64_t num_rows,
                                   const int32_t* offsets, const int32_t* counts, int capacity,
                                   int E, int I, int N, int G, const uint8_t* w,
                                   const uint16_t* scales, const uint8_t* zeros, bool swiglu,
                                   uint16_t* y, hipStream_t s) {
    if (num_rows == 0) return hipSuccess;
    const ExpertArgs p = {static_cast<const uint8_t*>(x), xs, num_rows, offsets, counts, capacity,
                          I, N, w, scales, zeros, y};
    const int tile = kExpertTiles * 16 / (swiglu ? 2 : 1);
    // row blocks side by side where an expert has many rows on average
    const int64_t avg = offsets ? num_rows / E : capacity;
    int z = (int)((avg + kExpertRowTiles * 16 - 1) / (kExpertRowTiles * 16));
    z = z < 1 ? 1 : z > 8 ? 8 : z;
    const dim3 grid((unsigned)((N + tile - 1) / tile), (unsigned)E, (unsigned)z);
    if (fp8)
        launch_t<true>(G, grid, s, p, swiglu);
    else
        launch_t<false>(G, grid, s, p, swiglu);
    return hipGetLastError();
}

}  // namespace ep
