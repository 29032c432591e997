// Device-side helpers for the gfx950 kernels: bf16 unpacking, the fp32 ->
// OCP E4M3 and fp32 -> bf16 conversions, and wave-level reductions.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace ep {

typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));
typedef unsigned int u32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

// 16-byte loads and stores with the non-temporal hint, for data that is
// streamed exactly once (rows read once, outputs written once): they do not
// displace reused data from the caches.
__device__ __forceinline__ uint4 load_nt(const void* p) {
    const u32x4 v = __builtin_nontemporal_load(static_cast<const u32x4*>(p));
    return make_uint4(v.x, v.y, v.z, v.w);
}
__device__ __forceinline__ void store_nt(void* p, const uint4& v) {
    const u32x4 w = {v.x, v.y, v.z, v.w};
    __builtin_nontemporal_store(w, static_cast<u32x4*>(p));
}

// 16-byte store with the device-scope cache policy (sc1): the line is
// written through the XCD's L2 instead of staying dirty there.  Used for the
// receive rows, which the next kernel reads from other XCDs: it leaves less
// L2 write-back for the end of the kernel (measured faster than ordinary and
// than non-temporal stores for dispatch's scattered rows).  A store of more
// than 8 bytes needs two wait states on gfx950 before a VALU instruction may
// overwrite its data registers; the compiler inserts them after the stores it
// generates but cannot see into inline asm, so the asm carries its own.
__device__ __forceinline__ void store_wt(void* p, const uint4& v) {
    const u32x4 w = {v.x, v.y, v.z, v.w};
    asm volatile("global_store_dwordx4 %0, %1, off sc1\n\ts_nop 1" : : "v"(p), "v"(w) : "memory");
}

// The same for 8 bytes (no wait states needed after a store of 8 bytes or less).
__device__ __forceinline__ void store_wt8(void* p, const uint2& v) {
    const u32x2 w = {v.x, v.y};
    asm volatile("global_store_dwordx2 %0, %1, off sc1" : : "v"(p), "v"(w) : "memory");
}

// bf16 -> fp32 is exact: the bf16 bits are the top half of the fp32 word.
__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// Two fp32 -> two bf16 (round to nearest even) packed low/high, with gfx950's
// v_cvt_pk_bf16_f32.
__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi) {
    f32x2 v = {lo, hi};
    bf16x2 b = __builtin_convertvector(v, bf16x2);
    return __builtin_bit_cast(uint32_t, b);
}

// Four fp32 -> four OCP E4M3 codes packed into a dword (byte i = value i),
// with gfx950's v_cvt_pk_fp8_f32: round to nearest even.  Inputs of the
// quantiser never exceed 448 * (1 + 2^-23) in magnitude, which rounds to 448,
// so the instruction's out-of-range behaviour is never reached there.
__device__ __forceinline__ uint32_t e4m3x4_hw(float a, float b, float c, float d) {
    int w = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
    w = __builtin_amdgcn_cvt_pk_fp8_f32(c, d, w, true);
    return (uint32_t)w;
}

// Bit-level fp32 -> OCP E4M3, round to nearest even, saturating to +-448,
// sign kept, NaN -> S.1111.111.  Normal results keep the top 3 fp32 mantissa
// bits after rounding the 20 dropped bits to nearest even (a carry moves into
// the exponent); results below 2^-6 are multiples of 2^-9, found by scaling
// by 2^9 (exact) and rounding to an integer.
__device__ __forceinline__ uint32_t e4m3_sw(float v) {
    const uint32_t u = __float_as_uint(v);
    const uint32_t sign = (u >> 24) & 0x80u;
    const uint32_t a = u & 0x7fffffffu;
    if (a > 0x7f800000u) return sign | 0x7fu;           // NaN
    if (a >= 0x43e00000u) return sign | 0x7eu;          // |v| >= 448
    if (a < 0x3c800000u) {                              // |v| < 2^-6
        const float q = __builtin_rintf(__uint_as_float(a) * 512.0f);
        return sign | (uint32_t)q;                      // 0..8 (8 = 2^-6)
    }
    const uint32_t r = (a + 0x7ffffu + ((a >> 20) & 1u)) >> 20;
    uint32_t code = r - ((127u - 7u) << 3);
    if (code > 0x7eu) code = 0x7eu;
    return sign | code;
}

__device__ __forceinline__ uint32_t e4m3x4_sw(float a, float b, float c, float d) {
    return e4m3_sw(a) | (e4m3_sw(b) << 8) | (e4m3_sw(c) << 16) | (e4m3_sw(d) << 24);
}

// Eight neighbouring channels of a bf16 row as fp32, and back (rounded to
// nearest even).
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
__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
    return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                      pack_bf16x2(f[6], f[7]));
}

// What silu(v) = v / (1 + exp(-v)) and its gradient are made of: q = exp(v / 2) and
// r = 1 / (1 + q^2), so that 1 / (1 + exp(-v)) = q * (q r) and 1 - that = r.  In halves
// nothing passes fp32's range where a result does not: exp(-v) would above 88, and its
// reciprocal be lost where silu(v), let alone silu(v) * u, is a normal number; q is 0
// only below v = -174.  (Above 17.5 the sigmoid is 1 to half a step.)
// In half steps of fp32: v_exp_f32 and v_rcp_f32 are off by 2 each, and what v * log2(e)
// / 2 loses to its rounding, which exp would multiply by |v|, is made up for: q is off by
// 3, q^2 / (1 + q^2) by 6 and 4 more, silu(v) * u by 13, under 2^-20.
struct Sigmoid {
    float q, qr, r;
};
__device__ __forceinline__ Sigmoid sigmoid(float v) {
    constexpr float kHigh = 0x1.715476p-1f, kLow = 0x1.4ae0cp-27f;     // log2(e) / 2
    const float c = __builtin_amdgcn_fmed3f(v, -200.0f, 17.5f), y = c * kHigh;
    const float lost = __builtin_fmaf(c, kLow, __builtin_fmaf(c, kHigh, -y));
    const float e = __builtin_amdgcn_exp2f(y);
    const float q = __builtin_fmaf(e, lost * 0.693147181f, e);
    const float r = __builtin_amdgcn_rcpf(__builtin_fmaf(q, q, 1.0f));
    return {q, q * r, r};
}
__device__ __forceinline__ float silu_times(float v, float u) {
    const Sigmoid s = sigmoid(v);
    return v * s.qr * u * s.q;
}

// silu(v) * u of eight channels, where instructions count.  From -8 up the plain form is
// as good: v * log2(e) is off by 1.22 |v| half steps (its rounding and its constant's),
// the rest by 7, together 17.  (32768 x 2048 to E4M3: 61 us, with gates of a deviation of
// 3.5 and more, whose waves take both, 68-73; the above for every element 72; expf and a
// division 83.)
__device__ __forceinline__ void silu_times(const float (&v)[8], const float (&u)[8],
                                           float (&o)[8]) {
    float low = v[0];
#pragma unroll
    for (int i = 1; i < 8; ++i) low = fminf(low, v[i]);
    if (low < -8.0f) {
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] = silu_times(v[i], u[i]);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float e = __builtin_amdgcn_exp2f(v[i] * -1.44269504f);
            o[i] = v[i] * __builtin_amdgcn_rcpf(1.0f + e) * u[i];
        }
    }
}

// Unsigned maximum over the 8 lanes of an aligned group of 8, with three DPP
// moves (no LDS round trip): swap neighbours (quad_perm 1,0,3,2), swap pairs
// (quad_perm 2,3,0,1), then mirror each half row of 8 lanes, which pairs the
// two quads.  A source lane that is inactive reads as 0, which leaves an
// unsigned maximum unchanged.
__device__ __forceinline__ uint32_t group8_max_u32(uint32_t v) {
    v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0xB1, 0xf, 0xf, false));
    v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x4E, 0xf, 0xf, false));
    v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x141, 0xf, 0xf, false));
    return v;
}

// Unsigned maximum over the 16 lanes of a DPP row: the maximum over each
// half row, then a row mirror (lane i reads lane 15 - i) pairs the halves.
__device__ __forceinline__ uint32_t group16_max_u32(uint32_t v) {
    v = group8_max_u32(v);
    v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x140, 0xf, 0xf, false));
    return v;
}

// The E4M3 codes of a lane's eight channels and the scale of the 128 that the 16
// lanes of its DPP row hold, all active, from fp32 values by dispatch's rule:
// a_c = max(max |v|, 1e-4), scale a_c / 448, codes E4M3(v * (448 / a_c)); NaNs
// take no part in the maximum, and an infinite or NaN v gets the code S.1111.111
// with its sign.
__device__ __forceinline__ uint2 quantise8(const float (&v)[8], float& scale) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(v[i]) & 0x7fffffffu);
    m = group16_max_u32(m);
    const bool finite = m < 0x7f800000u;
    if (!finite) {
        m = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint32_t a = __float_as_uint(v[i]) & 0x7fffffffu;
            m = max(m, a > 0x7f800000u ? 0u : a);
        }
        m = group16_max_u32(m);
    }
    const float ac = fmaxf(__uint_as_float(m), 1e-4f), inv = 448.0f / ac;
    scale = ac / 448.0f;
    uint2 q = make_uint2(e4m3x4_hw(v[0] * inv, v[1] * inv, v[2] * inv, v[3] * inv),
                         e4m3x4_hw(v[4] * inv, v[5] * inv, v[6] * inv, v[7] * inv));
    if (!finite) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint32_t b = __float_as_uint(v[i]);
            if ((b & 0x7f800000u) != 0x7f800000u) continue;
            const int sh = 8 * (i & 3);
            uint32_t& w = i < 4 ? q.x : q.y;
            w = (w & ~(0xffu << sh)) | ((b >> 24 & 0x80u) | 0x7fu) << sh;
        }
    }
    return q;
}

// Sum over aligned segments of S lanes (S a power of two, 1..64), every lane
// of a segment receiving its segment's total.  Segments of up to 16 lanes lie
// inside a DPP row and take DPP moves: neighbour and pair swaps, then the
// half-row and row mirrors, which pair the halves; wider segments finish with
// cross-row shuffles.  All 64 lanes must be active.
__device__ __forceinline__ int segment_sum(int v, int S) {
    if (S >= 2) v += __builtin_amdgcn_update_dpp(0, v, 0xB1, 0xf, 0xf, false);
    if (S >= 4) v += __builtin_amdgcn_update_dpp(0, v, 0x4E, 0xf, 0xf, false);
    if (S >= 8) v += __builtin_amdgcn_update_dpp(0, v, 0x141, 0xf, 0xf, false);
    if (S >= 16) v += __builtin_amdgcn_update_dpp(0, v, 0x140, 0xf, 0xf, false);
    if (S >= 32) v += __shfl_xor(v, 16);
    if (S >= 64) v += __shfl_xor(v, 32);
    return v;
}

// Maximum and sum over aligned segments of L lanes, the same for every lane of
// a segment; all lanes active.  Inside a row of 16 lanes a step is one DPP move
// (neighbours, pairs, half rows and rows mirrored), across rows one swap of
// rows or halves, after which both partners stand in one lane.
template <int STEP>
__device__ __forceinline__ void partners(uint32_t& a, uint32_t& b) {
    constexpr int kDpp[4] = {0xB1, 0x4E, 0x141, 0x140};
    if constexpr (STEP < 4) {
        b = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)a, kDpp[STEP], 0xf, 0xf, false);
    } else if constexpr (STEP == 4) {
        const auto r = __builtin_amdgcn_permlane16_swap(a, a, false, false);
        a = r[0];
        b = r[1];
    } else {
        const auto r = __builtin_amdgcn_permlane32_swap(a, a, false, false);
        a = r[0];
        b = r[1];
    }
}
template <int STEP>
__device__ __forceinline__ void partners(float& a, float& b) {
    uint32_t x = __float_as_uint(a), y;
    partners<STEP>(x, y);
    a = __uint_as_float(x);
    b = __uint_as_float(y);
}
template <int STEP>
__device__ __forceinline__ void partners(double& a, double& b) {
    const uint64_t u = __builtin_bit_cast(uint64_t, a);
    uint32_t x0 = (uint32_t)u, x1 = (uint32_t)(u >> 32), y0, y1;
    partners<STEP>(x0, y0);
    partners<STEP>(x1, y1);
    a = __builtin_bit_cast(double, (uint64_t)x1 << 32 | x0);
    b = __builtin_bit_cast(double, (uint64_t)y1 << 32 | y0);
}
__device__ __forceinline__ uint32_t larger(uint32_t a, uint32_t b) { return max(a, b); }
__device__ __forceinline__ float larger(float a, float b) { return fmaxf(a, b); }
__device__ __forceinline__ double larger(double a, double b) { return fmax(a, b); }
template <int L, int STEP = 0, typename V>
__device__ __forceinline__ V seg_max(V v) {
    if constexpr ((1 << STEP) < L) {
        V o;
        partners<STEP>(v, o);
        return seg_max<L, STEP + 1>(larger(v, o));
    }
    return v;
}
template <int L, int STEP = 0, typename V>
__device__ __forceinline__ V seg_sum(V v) {
    if constexpr ((1 << STEP) < L) {
        V o;
        partners<STEP>(v, o);
        return seg_sum<L, STEP + 1>(v + o);
    }
    return v;
}
}  // namespace ep
