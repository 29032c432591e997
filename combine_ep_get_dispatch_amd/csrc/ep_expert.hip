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
// sum x comes from one more matrix instruction with a row of ones.  A group's
// sums start from -z sum x (or, where groups are short and have zero points of
// their own, a block's four corrections are one fp32 matrix instruction, which
// took 128 rows over 32 experts, 2048 -> 7168, G = 32 from 92 to 85 us; 72 now).
//
// Precision.  The sums are fp32, the result is rounded once.  bf16 rows: the
// products are exact; the 128 costs five of the sums' 24 bits ahead of a result
// of 8.  E4M3 rows: the E4M3 instructions align the products of eight
// neighbouring channels to the largest and cut them 13 places below its power
// of two, so a code of under 2^-7 of the largest beside it loses its last
// places (an input of eight channels 448, -448 and 2^-j, codes 15, 15 and 1,
// gives 2^-j down to j = 2 and 0 from 3 on).  The rows' own rounding to E4M3 is
// 2^-4 of each value, and on random rows the sums are off by 1e-5 of the
// result's size, a hundredth of its rounding, so that 1.4% of the results are
// the other bf16 neighbour (bf16 rows 0.2%); the bf16 instructions with the
// codes widened would avoid it at bf16 rows' time, 103 against 93 us.
//
// Layout.  Weights are the A operand (16 channels by k), rows the B operand
// (k by 16 rows), so a lane ends with four neighbouring channels of one row.
// A lane loads 16 bytes, 32 codes, of one channel: a wave's load covers 64
// bytes of 16 channels.  Matrix instructions sum over the four lane groups;
// where a group of scales is shorter than the 128 codes that these hold, a
// 4x4 transpose between them (two swaps of half rows, two of rows) first gives
// every instruction 32 neighbouring codes.
//
// A workgroup owns a tile of 64 weight channels of one expert for a block of
// its rows; its four waves take every fourth step along the input channels and
// their sums meet in LDS, in wave order.  Experts of up to 16 rows run with one
// row tile, others with two (16 experts x 4096 -> 2 x 2048, E4M3 rows, one / two
// for all, rows of an expert on average: 4 rows 35 / 37 us, 16 rows 57 / 42, 64
// rows 146 / 106).  Four row tiles do not fit the registers (64 rows: 187 us, 98
// now with two).
//
// What it took on MI355X, 32 experts x 128 rows, 7168 -> 2 x 2048 with SWIGLU,
// E4M3 rows (484 MB): 3670 us with a wave per channel, 111 on matrix
// instructions, 98 with the loads a step ahead and the scales through LDS,
// 91-98 with the two 64-byte halves of a weight line asked for together (5.4
// TB/s in the kernel; reading the weights alone in this pattern took 81).  bf16
// rows, which leave registers for one block at a time (20 to 33 of 256 go to
// scratch where G = 128; a form without took as long): 101-110 us.  One token's
// eight experts, 2048 -> 7168 (60 MB): 17 us, 10 of them the weights.
#include "ep_internal.h"
#include "ep_device.h"

#include <type_traits>

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
    int E, I, N;
    const uint8_t* w;
    const uint16_t* scales;
    const uint8_t* zeros;
    uint16_t* y;
};

// The same value, unknown to the compiler, which would otherwise compute what
// follows from it once, ahead of the loop over tasks, and hold it in registers
// that the loop over blocks needs.
__device__ __forceinline__ int opaque(int v) {
    asm volatile("" : "+v"(v));
    return v;
}

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
// ... and as bf16 pairs 128 + q: (0,4) (1,5) (2,6) (3,7).  one28 = 0x43004300
// in a register, so that mask and constant are one instruction.
__device__ __forceinline__ i32x4 codes_bf16(int v, unsigned one28) {
    const unsigned u = (unsigned)v;
    i32x4 o;
    o[0] = (int)((u & 0x000f000fu) | one28);
    o[1] = (int)(((u >> 4) & 0x000f000fu) | one28);
    o[2] = (int)(((u >> 8) & 0x000f000fu) | one28);
    o[3] = (int)(((u >> 12) & 0x000f000fu) | one28);
    return o;
}
// Eight E4M3 values (two dwords) and eight bf16 values in the same orders.
__device__ __forceinline__ void order_e4m3(int& a, int& b) {
    const int lo = (int)__builtin_amdgcn_perm((unsigned)b, (unsigned)a, 0x06040200u);
    const int hi = (int)__builtin_amdgcn_perm((unsigned)b, (unsigned)a, 0x07050301u);
    a = lo;
    b = hi;
}
// held false: zeros (the byte selector 0x0c).
__device__ __forceinline__ i32x4 order_bf16(const i32x4& v, bool held) {
    const unsigned lo = held ? 0x05040100u : 0x0c0c0c0cu, hi = held ? 0x07060302u : 0x0c0c0c0cu;
    i32x4 o;
    o[0] = (int)__builtin_amdgcn_perm((unsigned)v[2], (unsigned)v[0], lo);
    o[1] = (int)__builtin_amdgcn_perm((unsigned)v[2], (unsigned)v[0], hi);
    o[2] = (int)__builtin_amdgcn_perm((unsigned)v[3], (unsigned)v[1], lo);
    o[3] = (int)__builtin_amdgcn_perm((unsigned)v[3], (unsigned)v[1], hi);
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

// Whether the last block of 128 input channels may be short.  Its missing
// channels are read at places that exist and enter as rows of zeros.
template <bool FP8, int G>
constexpr bool kTail = !FP8 && G < 128;

// What a wave reads for 128 input channels (block b) of its channel and row
// tiles.  All loads of a step's blocks are issued together, one step ahead of
// the arithmetic on it: the wave waits once per step, and while it works on one
// step the next is on its way.
template <bool FP8, int G, bool ZP, int RT, int CT>
struct Block {
    static constexpr int kX = FP8 && G == 128 ? 2 : 4;      // loads per row tile
    using XV = typename std::conditional<FP8 && G != 128, uint2, i32x4>::type;
    i32x4 w[CT];
    XV x[RT][kX];
    float xs[RT];
};

// Bases that are the same for the wave and 32-bit offsets of this lane.
template <int RT, int CT>
struct Lane {
    const uint8_t* w;
    const uint8_t* x;
    const uint8_t* xs;
    uint32_t woff[CT];     // bytes, of the channels that the lane loads
    uint32_t xrow[RT];
    uint32_t I, lg;
};

template <bool FP8, int G, bool ZP, int RT, int CT>
__device__ __forceinline__ void load_weights(Block<FP8, G, ZP, RT, CT>& k,
                                             const Lane<RT, CT>& a, int ct, int b) {
    int at = b * 64;
    // In a short last block the lane groups past it load the row's last codes,
    // which meet zeros.  (Below 128 channels that is ahead of the lane's own
    // place, woff, which holds its 16 lg: a negative step.)
    if (kTail<FP8, G>) at = min(at, (int)(a.I / 2) - 16 - (int)a.lg * 16);
    k.w[ct] = *reinterpret_cast<const i32x4*>(a.w + (a.woff[ct] + (uint32_t)at));
}

template <bool FP8, int G, bool ZP, int RT, int CT>
__device__ __forceinline__ void load_rows(Block<FP8, G, ZP, RT, CT>& k, const Lane<RT, CT>& a,
                                          int b) {
    const uint32_t kb = b * 128, I = a.I;
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
        if constexpr (FP8 && G == 128) {
            const i32x4* xp =
                reinterpret_cast<const i32x4*>(a.x + (a.xrow[rt] * I + kb + a.lg * 32));
            k.x[rt][0] = xp[0];
            k.x[rt][1] = xp[1];
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                // the 8 channels of step j that this lane holds codes of
                uint32_t step = G < 128 ? kb + j * 32 : kb + j * 8;
                if (kTail<FP8, G>) step = min(step, I - 32);
                const uint32_t c = step + a.lg * (G < 128 ? 8 : 32);
                using XV = typename Block<FP8, G, ZP, RT, CT>::XV;
                k.x[rt][j] =
                    *reinterpret_cast<const XV*>(a.x + (a.xrow[rt] * I + c) * (FP8 ? 1 : 2));
            }
        }
        k.xs[rt] = 1.0f;
        if constexpr (FP8)
            k.xs[rt] = *reinterpret_cast<const float*>(a.xs + (a.xrow[rt] * (I / 128) + b) * 4);
    }
}

// What a group's sums start from: -z sum x for each of the lane's channels
// (in units of 2^-9 where the codes count as q * 2^-9; with the 128 that bf16
// codes carry).
template <bool FP8, int G, bool ZP>
__device__ __forceinline__ f32x4 group_start(float sx, unsigned zv) {
    const float unit = FP8 && G != 128 ? 0.001953125f : 1.0f;
    const float more = FP8 ? 0.0f : 128.0f;
    f32x4 c;
    if constexpr (ZP) {
        const unsigned m = zv & 0x0f0f0f0fu;
        const float u = -unit * sx;
#pragma unroll
        for (int i = 0; i < 4; ++i) c[i] = ((float)((m >> (8 * i)) & 255u) + more) * u;
    } else {
        const float u = -unit * (8.0f + more) * sx;
        c = f32x4{u, u, u, u};
    }
    return c;
}

// A group's sums, scaled into acc.
__device__ __forceinline__ void add_group(f32x4& acc, const f32x4& t, uint2 sv, float xs) {
    acc[0] = __builtin_fmaf(bf16_lo(sv.x) * xs, t[0], acc[0]);
    acc[1] = __builtin_fmaf(bf16_hi(sv.x) * xs, t[1], acc[1]);
    acc[2] = __builtin_fmaf(bf16_lo(sv.y) * xs, t[2], acc[2]);
    acc[3] = __builtin_fmaf(bf16_hi(sv.y) * xs, t[3], acc[3]);
}

template <bool FP8, int G, bool ZP, int RT, int CT>
__device__ __forceinline__ void use_block(f32x4 (&acc)[CT][RT],
                                          Block<FP8, G, ZP, RT, CT>& k, int b, int I,
                                          const uint2* s_sc, const unsigned* s_z) {
    const int lg = (threadIdx.x & 63) >> 4, lr = threadIdx.x & 15;
    // the scales and zero points of the lane's channels of tile ct, group i of
    // the block (of a short block: a group that exists, its sums are 0)
    const int last = (kTail<FP8, G> ? min(I - b * 128, 128) : 128) / G - 1;
    auto scale = [&](int ct, int i) { return s_sc[min(i, last) * (CT * 4) + ct * 4 + lg]; };
    auto zero_point = [&](int ct, int i) {
        return ZP && G == 128 ? s_z[i * (CT * 4) + ct * 4 + lg] : 0u;
    };
    // zero points of short groups are taken off at the end of the block
    constexpr bool kLate = ZP && G < 128;
    const f32x4 zero = {0.0f, 0.0f, 0.0f, 0.0f};
    if constexpr (FP8 && G == 128) {
        i32x8 xv[RT], ones;
        float sx[RT];
#pragma unroll
        for (int i = 0; i < 8; ++i) ones[i] = 0x38383838;   // 1.0, taken back 2^-9 below
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) {
#pragma unroll
            for (int i = 0; i < 8; i += 2) {
                int u = k.x[rt][i / 4][i % 4], v = k.x[rt][i / 4][i % 4 + 1];
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
                codes_e4m3(o, k.w[ct][i]);
                a[2 * i] = o[0];
                a[2 * i + 1] = o[1];
            }
#pragma unroll
            for (int rt = 0; rt < RT; ++rt)
                add_group(acc[ct][rt],
                          mfma128(a, xv[rt], group_start<FP8, G, ZP>(sx[rt], zero_point(ct, 0))),
                          scale(ct, 0), k.xs[rt]);
        }
    } else {
        if constexpr (G < 128) {
#pragma unroll
            for (int ct = 0; ct < CT; ++ct) transpose_groups(k.w[ct]);
        }
        constexpr int kSteps = G / 32;     // matrix instructions per group of scales
        const i32x4 ones = {0x3f803f80, 0x3f803f80, 0x3f803f80, 0x3f803f80};
        const int ones8[2] = {0x38383838, 0x38383838};
        const unsigned one28 = opaque(0x43004300);
        float sums[RT][4 / kSteps];
#pragma unroll
        for (int rt = 0; rt < RT; ++rt)
#pragma unroll
            for (int i = 0; i < 4 / kSteps; ++i) sums[rt][i] = 0.0f;
#pragma unroll
        for (int j0 = 0; j0 < 4; j0 += kSteps) {
            f32x4 d[CT][RT];
            if constexpr (FP8) {
                int xv[RT][kSteps][2];
#pragma unroll
                for (int rt = 0; rt < RT; ++rt) {
                    f32x4 sx = zero;
#pragma unroll
                    for (int j = 0; j < kSteps; ++j) {
                        xv[rt][j][0] = (int)k.x[rt][j0 + j].x;
                        xv[rt][j][1] = (int)k.x[rt][j0 + j].y;
                        order_e4m3(xv[rt][j][0], xv[rt][j][1]);
                        sx = mfma32_e4m3(ones8, xv[rt][j], sx);
                    }
                    sums[rt][j0 / kSteps] = sx[0];
#pragma unroll
                    for (int ct = 0; ct < CT; ++ct)
                        d[ct][rt] = kLate ? zero
                                          : group_start<FP8, G, ZP>(sx[0],
                                                                    zero_point(ct, j0 / kSteps));
                }
#pragma unroll
                for (int ct = 0; ct < CT; ++ct)
#pragma unroll
                    for (int j = 0; j < kSteps; ++j) {
                        int a[2];
                        codes_e4m3(a, k.w[ct][j0 + j]);
#pragma unroll
                        for (int rt = 0; rt < RT; ++rt)
                            d[ct][rt] = mfma32_e4m3(a, xv[rt][j], d[ct][rt]);
                    }
            } else {
                i32x4 xv[RT][kSteps];
#pragma unroll
                for (int rt = 0; rt < RT; ++rt) {
                    f32x4 sx = zero;
#pragma unroll
                    for (int j = 0; j < kSteps; ++j) {
                        xv[rt][j] = order_bf16(
                            k.x[rt][j0 + j], !kTail<FP8, G> || b * 128 + (j0 + j) * 32 < I);
                        sx = mfma32(ones, xv[rt][j], sx);
                    }
                    sums[rt][j0 / kSteps] = sx[0];
#pragma unroll
                    for (int ct = 0; ct < CT; ++ct)
                        d[ct][rt] = kLate ? zero
                                          : group_start<FP8, G, ZP>(sx[0],
                                                                    zero_point(ct, j0 / kSteps));
                }
#pragma unroll
                for (int ct = 0; ct < CT; ++ct)
#pragma unroll
                    for (int j = 0; j < kSteps; ++j) {
                        const i32x4 a = codes_bf16(k.w[ct][j0 + j], one28);
#pragma unroll
                        for (int rt = 0; rt < RT; ++rt)
                            d[ct][rt] = mfma32(a, xv[rt][j], d[ct][rt]);
                    }
            }
#pragma unroll
            for (int ct = 0; ct < CT; ++ct)
#pragma unroll
                for (int rt = 0; rt < RT; ++rt)
                    add_group(acc[ct][rt], d[ct][rt], scale(ct, j0 / kSteps),
                              FP8 ? k.xs[rt] * 512.0f : 1.0f);
        }
        if constexpr (kLate) {
            // - sum over the block's groups of (z s) (sum x): one fp32 matrix
            // instruction a tile, lane group g holding group g's factors
            const bool held = lg <= last;
            float bx[RT];
#pragma unroll
            for (int rt = 0; rt < RT; ++rt) {
                bx[rt] = sums[rt][0];
#pragma unroll
                for (int i = 1; i < 4 / kSteps; ++i) bx[rt] = lg == i ? sums[rt][i] : bx[rt];
                if (FP8) bx[rt] *= k.xs[rt];
                bx[rt] = held ? bx[rt] : 0.0f;
            }
#pragma unroll
            for (int ct = 0; ct < CT; ++ct) {
                const int at = (held ? lg * (CT * 4) : 0) * 4 + ct * 16 + lr;
                const float sv = __uint_as_float(
                    (uint32_t)reinterpret_cast<const uint16_t*>(s_sc)[at] << 16);
                const int zv = reinterpret_cast<const uint8_t*>(s_z)[at] & 15;
                const float az = -((float)zv + (FP8 ? 0.0f : 128.0f)) * sv;
#pragma unroll
                for (int rt = 0; rt < RT; ++rt)
                    acc[ct][rt] =
                        __builtin_amdgcn_mfma_f32_16x16x4f32(az, bx[rt], acc[ct][rt], 0, 0, 0);
            }
        }
    }
}

// Rows of expert e: the first one, and how many (0 or less: none).
__device__ __forceinline__ int64_t expert_rows(const ExpertArgs& p, int e, int64_t& begin) {
    begin = p.offsets ? (int64_t)p.offsets[e] : (int64_t)e * p.capacity;
    int64_t end = begin + (p.offsets ? p.counts[e] : min(p.counts[e], p.capacity));
    if (begin < 0) begin = 0;
    if (end > p.num_rows) end = p.num_rows;
    return end - begin;
}

// A workgroup's task: rows [r0, n) (at most RT * 16 of them) of expert e, whose
// rows start at `begin`; its channel tile starts at channel n0 (of each half,
// with SWIGLU).
struct Task {
    int e, n0, n, r0;
    int64_t begin;
};

// The experts come in two classes by their rows: up to 16, which one row tile
// holds, and more, which two take at once.  A class's row blocks of n rows:
template <int RT>
__device__ __forceinline__ int row_blocks(int n) {
    const bool mine = RT == 1 ? n <= 16 : n > 16;
    return mine ? (int)(((unsigned)n + RT * 16 - 1) / (RT * 16)) : 0;
}

// The first kKnown experts, which a workgroup counts once: first row, rows, and
// the class's row blocks of experts 0..i; the others are counted again for
// every task.
constexpr int kKnown = 256;
struct RowBlocks {
    int first[kKnown], rows[kKnown], upto[2][kKnown];
};

// Sums of lanes 0..i, at most 2^30: counts whose runs overlap, all of up to 2^31
// rows, would pass 32 bits.
__device__ __forceinline__ int prefix_sum(int v) {
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int o = __shfl_up(v, d);
        if (lane >= d) v = (int)min((unsigned)v + (unsigned)o, 1u << 30);
    }
    return v;
}

// The task at place `task` of the order: the (row block, channel tile) pairs of
// the class's experts, the row blocks of a tile next to each other (they share
// its weights) and the tiles of an expert next to each other (they share its
// rows, and lines of its scales).  False if there is none.
template <int RT>
__device__ __forceinline__ bool find_task(Task& t, const ExpertArgs& p, const RowBlocks& rbs,
                                          int task, int ntile, int channels) {
    const int lane = threadIdx.x & 63;
    int before = 0;
#pragma unroll 1
    for (int e0 = 0; e0 < p.E; e0 += 64) {
        int first, rows, upto;
        if (e0 < kKnown) {
            first = rbs.first[e0 + lane];
            rows = rbs.rows[e0 + lane];
            upto = rbs.upto[RT - 1][e0 + lane];
        } else {
            int64_t b = 0, m = 0;
            if (e0 + lane < p.E) m = expert_rows(p, e0 + lane, b);
            first = (int)b;
            rows = m > 0 ? (int)m : 0;
            upto = prefix_sum(row_blocks<RT>(rows)) + before;
        }
        const uint64_t hit = __ballot(upto * ntile > task);
        if (hit) {
            const int at = __builtin_ctzll(hit);
            t.e = e0 + at;
            t.n = __builtin_amdgcn_readlane(rows, at);
            t.begin = __builtin_amdgcn_readlane(first, at);
            const int nb = row_blocks<RT>(t.n);
            const unsigned local = task - (__builtin_amdgcn_readlane(upto, at) - nb) * ntile;
            const unsigned tile = nb == 1 ? local : local / (unsigned)nb;
            t.n0 = tile * channels;
            t.r0 = (local - tile * nb) * RT * 16;
            return true;
        }
        before = __builtin_amdgcn_readlane(upto, 63);
    }
    return false;
}

// The scales and zero points of a workgroup's channels for a chunk of input
// channels, [group][channel / 4], and the waves' sums.
template <int G, bool ZP>
struct ExpertLds {
    static constexpr int CT = kExpertTiles;
    static constexpr int kChunk = G == 32 ? 32 : 64;       // blocks of 128 channels
    static constexpr int kEntries = kChunk * (128 / G) * CT * 4;
    uint2 sc[kEntries];
    unsigned z[ZP ? kEntries : 1];
    f32x4 part[kExpertWaves * CT * 2 * 64];
    RowBlocks rbs;
};

// A workgroup's tasks of one class: task, task + stride, ... below end.
template <bool FP8, int G, bool ZP, bool SWIGLU, int RT, int NB>
__device__ __forceinline__ void run_tasks(const ExpertArgs& p, ExpertLds<G, ZP>& lds, int task,
                                          int end, int stride) {
    constexpr int CT = kExpertTiles;
    using Lds = ExpertLds<G, ZP>;
    using Blk = Block<FP8, G, ZP, RT, CT>;
    constexpr int kChannels = CT * 16 / (SWIGLU ? 2 : 1);
    constexpr int kThreads = kExpertWaves * 64;
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int lg = lane >> 4, lr = lane & 15;
    const int I = p.I, N = p.N;
    const int W = SWIGLU ? 2 * N : N;
    const int nblk = (I + 127) / 128;
    const int ntile = (N + kChannels - 1) / kChannels;

    Task t;
    Lane<RT, CT> a;
    a.I = I;
    a.lg = lg;
    const uint16_t* sc;
    const uint8_t* zr;
    auto aim = [&]() {
        const int lg = opaque(lane) >> 4, lr = opaque(lane) & 15;
        a.w = p.w + (int64_t)t.e * W * (I / 2);
        a.x = p.x + (t.begin + t.r0) * I * (FP8 ? 1 : 2);
        a.xs = FP8 ? reinterpret_cast<const uint8_t*>(p.xs + (t.begin + t.r0) * (I / 128))
                   : nullptr;
#pragma unroll
        for (int ct = 0; ct < CT; ++ct) {
            const int half = SWIGLU ? ct / (CT / 2) : 0;
            const int c0 = t.n0 + (SWIGLU ? ct % (CT / 2) : ct) * 16;
            // past the last channel: any channel, its sums are not stored
            a.woff[ct] = (uint32_t)(half * N + min(c0 + lr, N - 1)) * (uint32_t)(I / 2) + lg * 16;
        }
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) a.xrow[rt] = min(rt * 16 + lr, t.n - 1 - t.r0);
        sc = p.scales + (int64_t)t.e * (I / G) * W;
        zr = ZP ? p.zeros + (int64_t)t.e * (I / G) * W : nullptr;
    };

    // Scales of the chunk of blocks from c0, in rounds of kBatch entries a
    // thread: fetched, then kept in LDS.
    constexpr int kBatch = 4, kRound = kBatch * kThreads;
    uint2 bs[kBatch];
    unsigned bz[kBatch];
    auto entries = [&](int c0) {
        return (min((c0 + Lds::kChunk) * 128, I) / G - c0 * (128 / G)) * (CT * 4);
    };
    auto fetch = [&](int c0, int first) {
        const int tid = opaque(threadIdx.x);
#pragma unroll
        for (int q = 0; q < kBatch; ++q) {
            // past the last entry: that one again
            const int i = min(first + q * kThreads + tid, entries(c0) - 1);
            const int u = i % (CT * 4), ct = u / 4;
            const int half = SWIGLU ? ct / (CT / 2) : 0;
            const int ch = t.n0 + (SWIGLU ? ct % (CT / 2) : ct) * 16 + u % 4 * 4;
            const uint32_t at = (uint32_t)(c0 * (128 / G) + i / (CT * 4)) * W + half * N +
                                min(ch, N - 4);
            bs[q] = *reinterpret_cast<const uint2*>(sc + at);
            if constexpr (ZP) bz[q] = *reinterpret_cast<const unsigned*>(zr + at);
        }
    };
    auto keep = [&](int c0, int first) {
        const int tid = opaque(threadIdx.x);
#pragma unroll
        for (int q = 0; q < kBatch; ++q) {
            const int i = first + q * kThreads + tid;
            if (i < entries(c0)) {
                lds.sc[i] = bs[q];
                if constexpr (ZP) lds.z[i] = bz[q];
            }
        }
    };

    // A wave takes steps of NB neighbouring blocks, every kExpertWaves-th step
    // of a chunk; a step's second block past the end is the last one again.
    Blk k0[NB], k1[NB];
    f32x4 acc[CT][RT];
    auto load = [&](Blk (&k)[NB], int c0, int st) {
        const int c1 = min(c0 + Lds::kChunk, nblk);
        // the 64 bytes of a row that neighbouring blocks read share a line
#pragma unroll
        for (int ct = 0; ct < CT; ++ct)
#pragma unroll
            for (int i = 0; i < NB; ++i)
                load_weights<FP8, G, ZP, RT, CT>(k[i], a, ct, min(c0 + st * NB + i, c1 - 1));
#pragma unroll
        for (int i = 0; i < NB; ++i)
            load_rows<FP8, G, ZP, RT, CT>(k[i], a, min(c0 + st * NB + i, c1 - 1));
        __builtin_amdgcn_sched_barrier(0);      // loads stay ahead of the arithmetic
    };
    auto use = [&](Blk (&k)[NB], int c0, int st) {
        const int c1 = min(c0 + Lds::kChunk, nblk);
#pragma unroll
        for (int i = 0; i < NB; ++i) {
            const int b = st * NB + i;          // of the chunk
            if (NB == 1 || c0 + b < c1) {
                const int at = b * (128 / G) * (CT * 4);
                use_block<FP8, G, ZP, RT, CT>(acc, k[i], c0 + b, I, lds.sc + at,
                                              lds.z + (ZP ? at : 0));
            }
        }
        __builtin_amdgcn_sched_barrier(0);
    };
    auto nsteps = [&](int c0) { return (min(Lds::kChunk, nblk - c0) + NB - 1) / NB; };
    // The first loads of a chunk: its scales ahead of the weights, which then
    // travel while the scales are put in place.  They are issued before the last
    // step of the chunk ahead of it (of this task or the last one) is worked on.
    // (Where a step is worked on, the number of loads under way is the same on
    // every path to it, so that it waits for its own alone.)
    int c0 = 0;
    if (task >= end || !find_task<RT>(t, p, lds.rbs, task, ntile, kChannels)) return;
    auto start = [&]() {
        fetch(c0, 0);
        __builtin_amdgcn_sched_barrier(0);
        load(k0, c0, min(wave, nsteps(c0) - 1));
    };
    aim();
    start();
#pragma unroll
    for (int ct = 0; ct < CT; ++ct)
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) acc[ct][rt] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    while (true) {
        const Task done = t;
        const int b0 = c0, nstep = nsteps(b0);
        const bool whole = b0 + Lds::kChunk >= nblk;        // the task's last chunk
        Task then = t;
        bool more = true;
        if (whole) {
            task += stride;
            more = task < end && find_task<RT>(then, p, lds.rbs, task, ntile, kChannels);
        }
        auto next = [&]() {
            t = then;
            c0 = whole ? 0 : b0 + Lds::kChunk;
            aim();
            start();
        };
        keep(b0, 0);
        for (int first = kRound; first < entries(b0); first += kRound) {
            fetch(b0, first);
            keep(b0, first);
        }
        __syncthreads();
        // (a wave without a step has last = wave - kExpertWaves)
        const int last =
            wave + (nstep + kExpertWaves - 1 - wave) / kExpertWaves * kExpertWaves - kExpertWaves;
        int st = wave;
        for (; st + 2 * kExpertWaves <= last; st += 2 * kExpertWaves) {
            load(k1, b0, st + kExpertWaves);
            use(k0, b0, st);
            load(k0, b0, st + 2 * kExpertWaves);
            use(k1, b0, st + kExpertWaves);
        }
        if (st < last) {
            load(k1, b0, st + kExpertWaves);
            use(k0, b0, st);
            if (more) {
                next();
                use(k1, b0, st + kExpertWaves);
            } else {
                use(k1, b0, st + kExpertWaves);
            }
        } else {
            if (st == last) use(k0, b0, st);
            if (more) next();
        }
        if (!whole) {
            __syncthreads();                    // this chunk's scales are done with
            continue;
        }

        // the waves' sums, in wave order; wave i finishes tiles i, i + kExpertWaves, ...
        constexpr int kTiles = CT * RT;
#pragma unroll
        for (int ct = 0; ct < CT; ++ct)
#pragma unroll
            for (int rt = 0; rt < RT; ++rt)
                lds.part[(wave * kTiles + ct * RT + rt) * 64 + lane] = acc[ct][rt];
        __syncthreads();
        constexpr int kOut = SWIGLU ? kTiles / 2 : kTiles;
        for (int o = wave; o < kOut; o += kExpertWaves) {
            const int ct = o / RT, rt = o % RT;
            f32x4 v = {0.0f, 0.0f, 0.0f, 0.0f}, u = v;
            for (int i = 0; i < kExpertWaves; ++i) v += lds.part[(i * kTiles + o) * 64 + lane];
            if constexpr (SWIGLU) {
                for (int i = 0; i < kExpertWaves; ++i)
                    u += lds.part[(i * kTiles + kOut + o) * 64 + lane];
#pragma unroll
                for (int i = 0; i < 4; ++i) v[i] = v[i] / (1.0f + expf(-v[i])) * u[i];
            }
            const int row = rt * 16 + lr, c = done.n0 + ct * 16 + lg * 4;
            if (row < done.n - done.r0 && c < N) {
                const uint2 o2 = make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
                *reinterpret_cast<uint2*>(p.y + (done.begin + done.r0 + row) * N + c) = o2;
            }
        }
        if (!more) break;
#pragma unroll
        for (int ct = 0; ct < CT; ++ct)
#pragma unroll
            for (int rt = 0; rt < RT; ++rt) acc[ct][rt] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    }
}

// Every XCD (workgroups i, i + 8, ...) gets one run of a class's tasks, which
// its workgroups stride over; the second class goes on where the first left
// off.  Experts without rows have no tasks.
template <bool FP8, int G, bool ZP, bool SWIGLU>
__global__ __launch_bounds__(kExpertWaves * 64, kExpertWavesPerSimd) void expert_linear_kernel(
    const ExpertArgs p) {
    __shared__ ExpertLds<G, ZP> lds;
    constexpr int kChannels = kExpertTiles * 16 / (SWIGLU ? 2 : 1);
    const int lane = threadIdx.x & 63;
    const int ntile = (p.N + kChannels - 1) / kChannels;

    // Row blocks of the classes; every wave writes the same numbers, and reads
    // its own.
    int64_t few = 0, many = 0;
#pragma unroll 1
    for (int e0 = 0; e0 < p.E; e0 += 64) {
        int64_t b = 0, m = 0;
        if (e0 + lane < p.E) m = expert_rows(p, e0 + lane, b);
        const int rows = m > 0 ? (int)m : 0;
        const int f = prefix_sum(row_blocks<1>(rows)), g = prefix_sum(row_blocks<2>(rows));
        if (e0 < kKnown) {
            lds.rbs.first[e0 + lane] = (int)b;
            lds.rbs.rows[e0 + lane] = rows;
            lds.rbs.upto[0][e0 + lane] = (int)(few + f);
            lds.rbs.upto[1][e0 + lane] = (int)(many + g);
        }
        few += __builtin_amdgcn_readlane(f, 63);
        many += __builtin_amdgcn_readlane(g, 63);
    }
    // (a y of 2^30 tasks fits no memory: such counts do not belong to these rows)
    if ((few + many) * ntile >= 1 << 30) return;
    const int stride = gridDim.x / kXcds, xcd = blockIdx.x % kXcds;
    int slot = blockIdx.x / kXcds;
    if (few > 0) {
        const int tasks = (int)few * ntile, per = (tasks + kXcds - 1) / kXcds;
        run_tasks<FP8, G, ZP, SWIGLU, 1, few_blocks(FP8)>(p, lds, xcd * per + slot,
                                                          min(tasks, (xcd + 1) * per), stride);
        slot = (slot + stride - per % stride) % stride;
    }
    if (many > 0) {
        const int tasks = (int)many * ntile, per = (tasks + kXcds - 1) / kXcds;
        run_tasks<FP8, G, ZP, SWIGLU, 2, 1>(p, lds, xcd * per + slot,
                                            min(tasks, (xcd + 1) * per), stride);
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
                          E, I, N, w, scales, zeros, y};
    const int tile = kExpertTiles * 16 / (swiglu ? 2 : 1);
    // at most one workgroup per task, and no more than the GPU holds at once
    const int64_t blocks =
        offsets ? E + num_rows / 16 : (int64_t)E * (((int64_t)capacity + 15) / 16);
    const int64_t tasks = blocks * ((N + tile - 1) / tile);
    const int64_t held = kExpertWavesPerSimd * 4 / kExpertWaves * kCus;
    const dim3 grid((unsigned)(((tasks < held ? tasks : held) + kXcds - 1) / kXcds * kXcds));
    if (fp8)
        launch_t<true>(G, grid, s, p, swiglu);
    else
        launch_t<false>(G, grid, s, p, swiglu);
    return hipGetLastError();
}

}  // namespace ep
