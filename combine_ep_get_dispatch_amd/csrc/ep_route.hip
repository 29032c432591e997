// The router on gfx950: from a token's logits over the experts to its K slots
// (topk_idx, topk_weights), and the gradient of the weights with respect to
// the logits.
//
// Mathematics.  s_e = sigmoid(l_e) or softmax over the experts; the order is
// that of choice_e = s_e + bias_e (of l_e itself without a bias: both scores
// grow with the logit).  With groups only the experts of the best groups stay,
// a group's score being the sum of its two largest choices.  The K largest
// remain, equal ones by lowest index, and
//   w_k = scale * s_k   or   scale * s_k / sum over the slots of s.
// An expert whose logit is -inf or NaN is not available.
//
// Precision.  Where a bias or groups decide, choices are compared in fp64: two
// experts whose fp32 scores fall on the same value or swap under its rounding
// would otherwise be picked by the rounding, not by the definition.  Where the
// logits decide they are compared as they are.
//
// Layout.  A token belongs to a segment of L lanes of a wave and a lane holds
// VPL consecutive experts, so that lower lanes hold lower ids: the lowest lane
// among equals, and the first of it, is the lowest id, and the maximum needs no
// index beside it.
//
// What bounds it: not the logits (4.5 MB at 4096 tokens of 256 experts, 1 us)
// but the instructions per token -- about 1000 with a bias and groups, most of
// them the fp64 scores and the K maxima -- and, in a decode batch, their chain:
// 7.0 us per launch at 128 tokens, 2 us of them the launch itself.
#include "ep.h"
#include "ep_internal.h"
#include "ep_device.h"

#include <type_traits>

namespace ep {
namespace {

constexpr float kFltMax = 3.4028234663852886e38f;

// The two largest values of a segment of `lanes` lanes (a power of two, at
// most L), from the two largest of each lane.
template <int L, int STEP = 0>
__device__ __forceinline__ void seg_top2(double& a, double& b, int lanes) {
    if constexpr ((1 << STEP) < L) {
        if ((1 << STEP) < lanes) {
            double c = a, d = b, oa, ob;
            partners<STEP>(c, oa);
            partners<STEP>(d, ob);
            a = larger(c, oa);
            b = larger(fmin(c, oa), larger(d, ob));
            seg_top2<L, STEP + 1>(a, b, lanes);
        }
    }
}

// LDS written by some lanes of a wave is read by others: the wave's LDS
// accesses happen in order, the compiler has to keep them so.
__device__ __forceinline__ void wave_sync() {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

__device__ __forceinline__ float load_logit(const float* p) { return *p; }
__device__ __forceinline__ float load_logit(const uint16_t* p) {
    return __uint_as_float((uint32_t)*p << 16);
}
// -inf where the expert is not available; +inf counts as fp32's largest value.
__device__ __forceinline__ float clean_logit(float v) {
    return v > -INFINITY ? fminf(v, kFltMax) : -INFINITY;
}

// A lane's VPL logits: experts [e0, e0 + VPL), -inf past E.  vec: rows start
// at 16-byte boundaries and E is a multiple of the 16-byte vector.
template <int VPL>
__device__ __forceinline__ void load_row(float (&l)[VPL], const float* row, int e0, int E,
                                         bool vec) {
    if (VPL % 4 == 0 && vec) {
#pragma unroll
        for (int j = 0; j + 3 < VPL; j += 4) {
            float4 v = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
            if (e0 + j < E) v = *reinterpret_cast<const float4*>(row + e0 + j);
            l[j] = v.x;
            l[j + 1] = v.y;
            l[j + 2] = v.z;
            l[j + 3] = v.w;
        }
    } else {
#pragma unroll
        for (int j = 0; j < VPL; ++j) l[j] = e0 + j < E ? row[e0 + j] : -INFINITY;
    }
}
template <int VPL>
__device__ __forceinline__ void load_row(float (&l)[VPL], const uint16_t* row, int e0, int E,
                                         bool vec) {
    if (VPL % 8 == 0 && vec) {
#pragma unroll
        for (int j = 0; j + 7 < VPL; j += 8) {
            uint4 v = make_uint4(0xff80ff80u, 0xff80ff80u, 0xff80ff80u, 0xff80ff80u);
            if (e0 + j < E) v = *reinterpret_cast<const uint4*>(row + e0 + j);
            l[j] = bf16_lo(v.x);
            l[j + 1] = bf16_hi(v.x);
            l[j + 2] = bf16_lo(v.y);
            l[j + 3] = bf16_hi(v.y);
            l[j + 4] = bf16_lo(v.z);
            l[j + 5] = bf16_hi(v.z);
            l[j + 6] = bf16_lo(v.w);
            l[j + 7] = bf16_hi(v.w);
        }
    } else {
#pragma unroll
        for (int j = 0; j < VPL; ++j) l[j] = e0 + j < E ? load_logit(row + e0 + j) : -INFINITY;
    }
}

template <int VPL>
__device__ __forceinline__ void store_row(const float (&o)[VPL], float* row, int e0, int E,
                                          bool vec) {
    if (VPL % 4 == 0 && vec) {
#pragma unroll
        for (int j = 0; j + 3 < VPL; j += 4)
            if (e0 + j < E)
                *reinterpret_cast<float4*>(row + e0 + j) =
                    make_float4(o[j], o[j + 1], o[j + 2], o[j + 3]);
    } else {
#pragma unroll
        for (int j = 0; j < VPL; ++j)
            if (e0 + j < E) row[e0 + j] = o[j];
    }
}
template <int VPL>
__device__ __forceinline__ void store_row(const float (&o)[VPL], uint16_t* row, int e0, int E,
                                          bool vec) {
    if (VPL % 8 == 0 && vec) {
#pragma unroll
        for (int j = 0; j + 7 < VPL; j += 8)
            if (e0 + j < E)
                *reinterpret_cast<uint4*>(row + e0 + j) = make_uint4(
                    pack_bf16x2(o[j], o[j + 1]), pack_bf16x2(o[j + 2], o[j + 3]),
                    pack_bf16x2(o[j + 4], o[j + 5]), pack_bf16x2(o[j + 6], o[j + 7]));
    } else {
#pragma unroll
        for (int j = 0; j < VPL; ++j)
            if (e0 + j < E) row[e0 + j] = (uint16_t)pack_bf16x2(o[j], 0.0f);
    }
}

// v of lane i (within the wave; the same i for every lane where L is 64).
template <int L>
__device__ __forceinline__ double from_lane(double v, int i) {
    if constexpr (L == 64) {
        const uint64_t u = __builtin_bit_cast(uint64_t, v);
        const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)u, i);
        const uint32_t hi = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(u >> 32), i);
        return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
    }
    return __shfl(v, i);
}

// Unsigned keys in the order of the values, above 0 (which is the key of an
// expert that is not available).  Adding 0 makes -0 and +0 the same key.
__device__ __forceinline__ uint32_t order_key(float v) {
    const uint32_t u = __float_as_uint(v + 0.0f);
    return u ^ ((u >> 31) ? 0xffffffffu : 0x80000000u);
}
__device__ __forceinline__ uint64_t order_key(double v) {
    const uint64_t u = (uint64_t)__double_as_longlong(v + 0.0);
    return u ^ ((u >> 63) ? ~0ull : 1ull << 63);
}

__device__ __forceinline__ double sigmoid64(double l) { return 1.0 / (1.0 + exp(-l)); }

// A lane's experts in descending order of their keys, equal ones by id.
template <int VPL, bool FULL>
struct Ranked {
    uint32_t hi[VPL], lo[FULL ? VPL : 1];   // key; lo: its lower half, of 64 bits
    int at[VPL];                            // expert, from the lane's first

    __device__ __forceinline__ bool above(int i, int j) const {
        if constexpr (FULL)
            return ((uint64_t)hi[i] << 32 | lo[i]) > ((uint64_t)hi[j] << 32 | lo[j]);
        return hi[i] > hi[j];
    }
    // Neighbours change places only where the later one is larger, so equal
    // keys keep their order.
    __device__ __forceinline__ void sort() {
#pragma unroll
        for (int n = 0; n < VPL - 1; ++n)
#pragma unroll
            for (int j = VPL - 1; j > n; --j) {
                const bool up = above(j, j - 1);
                swap_if(up, hi[j], hi[j - 1]);
                if constexpr (FULL) swap_if(up, lo[j], lo[j - 1]);
                swap_if(up, at[j], at[j - 1]);
            }
    }
    template <typename V>
    static __device__ __forceinline__ void swap_if(bool c, V& a, V& b) {
        const V x = c ? b : a, y = c ? a : b;
        a = x;
        b = y;
    }
    // The first one leaves; a key of 0 (not available) follows the last.
    __device__ __forceinline__ void pop() {
#pragma unroll
        for (int j = 0; j < VPL - 1; ++j) {
            hi[j] = hi[j + 1];
            if constexpr (FULL) lo[j] = lo[j + 1];
            at[j] = at[j + 1];
        }
        hi[VPL - 1] = 0;
        if constexpr (FULL) lo[VPL - 1] = 0;
    }
};

// FULL: choices in fp64 (a bias or groups); otherwise the logits decide.
// Dynamic LDS, per token of the workgroup: its E logits and its K slots'
// experts, then with groups that do not lie on whole lanes E choices (double),
// NG group scores (double) and NG flags (int).
//
// A lane ranks its own experts once; a slot then takes one maximum over the
// lanes' first ones.  64-bit keys are compared by their upper halves, and by
// the lower ones only where two lanes have the same upper half.
template <typename LT, int VPL, int L, bool FULL>
__global__ __launch_bounds__(kRouteThreads) void route_kernel(
    const LT* __restrict__ logits, const float* __restrict__ bias, int T, int E, int K,
    bool softmax, int NG, int TG, bool normalize, float scale, int64_t* __restrict__ topk_idx,
    float* __restrict__ topk_weights, bool vec) {
    constexpr int kTokens = kRouteThreads / L;
    extern __shared__ EP_LDS_ALIGN unsigned char s_raw[];
    const int lane = threadIdx.x & 63;
    const int sl = lane & (L - 1);
    const int tok = threadIdx.x / L;                 // token of the workgroup
    const int64_t t = (int64_t)blockIdx.x * kTokens + tok;
    const bool live = t < T;
    float* s_logit = reinterpret_cast<float*>(s_raw) + tok * E;
    int* s_idx = reinterpret_cast<int*>(s_raw) + kTokens * E + tok * K;

    const int e0 = sl * VPL;
    float l[VPL];
    if (live) {
        load_row<VPL>(l, logits + t * E, e0, E, vec);
    } else {
#pragma unroll
        for (int j = 0; j < VPL; ++j) l[j] = -INFINITY;
    }
    float bj[VPL];
    if constexpr (FULL) {
#pragma unroll
        for (int j = 0; j < VPL; ++j) bj[j] = bias && e0 + j < E ? bias[e0 + j] : 0.0f;
    }
    float lmax = -INFINITY;
#pragma unroll
    for (int j = 0; j < VPL; ++j) {
        l[j] = clean_logit(l[j]);
        lmax = fmaxf(lmax, l[j]);
        if (e0 + j < E) s_logit[e0 + j] = l[j];
    }
    for (int k = sl; k < K; k += L) s_idx[k] = -1;

    // the softmax over all experts: its maximum and sum
    float m = 0.0f;
    double total = 1.0;
    if (softmax && (FULL || !normalize)) {
        m = fmaxf(seg_max<L>(lmax), -kFltMax);
        if constexpr (FULL) {
            double a = 0.0;
#pragma unroll
            for (int j = 0; j < VPL; ++j) a += exp((double)l[j] - (double)m);
            total = seg_sum<L>(a);
        } else {
            // fp32 terms, each rounded to a multiple of 2^-41: up to 1024 of them,
            // each at most 1, add up in fp64 without rounding, so that a token's
            // total does not depend on how many lanes its batch size gives it
            constexpr float kGrain = 0x1.8p-18f;         // its last place is 2^-41
            double a = 0.0;
#pragma unroll
            for (int j = 0; j < VPL; ++j) a += (double)((expf(l[j] - m) + kGrain) - kGrain);
            total = seg_sum<L>(a);
        }
    }

    Ranked<VPL, FULL> r;
    if constexpr (FULL) {
        double key[VPL];        // what orders the experts; -inf: not available
#pragma unroll
        for (int j = 0; j < VPL; ++j) {
            const double s = softmax ? exp((double)l[j] - (double)m) / total
                                     : sigmoid64((double)l[j]);
            const double c = s + (double)bj[j];
            key[j] = (l[j] > -INFINITY && c > -INFINITY) ? c : -INFINITY;
        }
        if (NG > 1) {
            const int gsz = E / NG;
            const int lanes = gsz / VPL;             // lanes of a group, if whole
            if (gsz % VPL == 0 && (lanes & (lanes - 1)) == 0) {
                double a = -INFINITY, b = -INFINITY;
#pragma unroll
                for (int j = 0; j < VPL; ++j) {
                    b = larger(b, fmin(a, key[j]));
                    a = larger(a, key[j]);
                }
                seg_top2<L>(a, b, lanes);
                const double mine = b > -INFINITY ? a + b : a;
                const int g = e0 / gsz;
                int better = 0;
                for (int i = 0; i < NG; ++i) {
                    const double o = from_lane<L>(mine, (lane - sl) + i * lanes);
                    better += (o > mine || (o == mine && i < g)) ? 1 : 0;
                }
#pragma unroll
                for (int j = 0; j < VPL; ++j) {
                    const bool open = better < TG && key[j] > -INFINITY;
                    const double by = bias ? key[j] : (double)l[j];
                    key[j] = open ? by : -INFINITY;
                }
            } else {
                const size_t head = ((size_t)kTokens * (E + K) * 4 + 15) & ~(size_t)15;
                double* s_ch = reinterpret_cast<double*>(s_raw + head) + tok * (E + 2 * NG);
                double* s_gs = s_ch + E;
                int* s_flag = reinterpret_cast<int*>(s_gs + NG);
#pragma unroll
                for (int j = 0; j < VPL; ++j)
                    if (e0 + j < E) s_ch[e0 + j] = key[j];
                wave_sync();
                for (int g = sl; g < NG; g += L) {
                    double a = -INFINITY, b = -INFINITY;
                    int i = g < gsz ? g : 0;         // lanes start at different banks
                    for (int n = 0; n < gsz; ++n) {
                        const double v = s_ch[g * gsz + i];
                        b = larger(b, fmin(a, v));
                        a = larger(a, v);
                        if (++i == gsz) i = 0;
                    }
                    s_gs[g] = b > -INFINITY ? a + b : a;
                }
                wave_sync();
                for (int g = sl; g < NG; g += L) {
                    const double v = s_gs[g];
                    int better = 0;
                    for (int i = 0; i < NG; ++i) {
                        const double o = s_gs[i];
                        better += (o > v || (o == v && i < g)) ? 1 : 0;
                    }
                    s_flag[g] = better < TG ? 1 : 0;
                }
                wave_sync();
                int g = e0 / gsz, in = e0 - g * gsz;
#pragma unroll
                for (int j = 0; j < VPL; ++j) {
                    // (no expert of a group past the last one is available)
                    const bool open = (s_flag[min(g, NG - 1)] != 0) & (key[j] > -INFINITY);
                    const double by = bias ? key[j] : (double)l[j];
                    key[j] = open ? by : -INFINITY;
                    const bool next = ++in == gsz;
                    in = next ? 0 : in;
                    g += next ? 1 : 0;
                }
            }
        }
#pragma unroll
        for (int j = 0; j < VPL; ++j) {
            const uint64_t u = key[j] > -INFINITY ? order_key(key[j]) : 0;
            r.hi[j] = (uint32_t)(u >> 32);
            r.lo[j] = (uint32_t)u;
            r.at[j] = j;
        }
    } else {
#pragma unroll
        for (int j = 0; j < VPL; ++j) {
            r.hi[j] = l[j] > -INFINITY ? order_key(l[j]) : 0;
            r.at[j] = j;
        }
    }
    r.sort();

    const uint64_t segmask = (L == 64 ? ~0ull : ((1ull << (L & 63)) - 1)) << (lane - sl);
    for (int k = 0; k < K; ++k) {
        const uint32_t top = seg_max<L>(r.hi[0]);
        uint64_t eq = __ballot(r.hi[0] == top && top != 0) & segmask;
        if constexpr (FULL) {
            if (__ballot((eq & (eq - 1)) != 0)) {
                const uint32_t low = seg_max<L>(r.hi[0] == top ? r.lo[0] : 0u);
                eq = __ballot(r.hi[0] == top && r.lo[0] == low && top != 0) & segmask;
            }
        }
        if (eq != 0 && __builtin_ctzll(eq) == (unsigned)lane) {
            s_idx[k] = e0 + r.at[0];
            r.pop();
        }
    }
    wave_sync();

    // slot k of the token: lanes k, k + L, ... of its segment
    if (normalize && softmax) {
        // over the selected experts alone, from their own maximum
        m = -kFltMax;
        for (int k = sl; k < K; k += L)
            if (s_idx[k] >= 0) m = fmaxf(m, s_logit[s_idx[k]]);
        m = seg_max<L>(m);
    }
    double sum = softmax ? total : 1.0;
    if (normalize) {
        sum = 0.0;
        for (int k = sl; k < K; k += L)
            if (s_idx[k] >= 0) {
                const double v = (double)s_logit[s_idx[k]];
                sum += softmax ? exp(v - (double)m) : sigmoid64(v);
            }
        sum = seg_sum<L>(sum);
    }
    for (int k = sl; k < K; k += L) {
        const int e = s_idx[k];
        double w = 0.0;
        if (e >= 0 && sum > 0.0) {
            const double v = (double)s_logit[e];
            w = (softmax ? exp(v - (double)m) : sigmoid64(v)) / sum * (double)scale;
        }
        if (live) {
            topk_idx[t * K + k] = e;
            topk_weights[t * K + k] = (float)w;
        }
    }
}

// Gradient.  With c_k = scale * grad_weights[k] over the token's valid slots:
//   softmax, not normalised:  d_i = p_i (c_i - sum_k c_k p_k), every expert, c_i
//                             the sum of the c of i's slots;
//   softmax, normalised:      d_k = q_k (c_k - sum_j c_j q_j), q the softmax
//                             over the slots;
//   sigmoid, not normalised:  d_k = c_k s_k (1 - s_k);
//   sigmoid, normalised:      d_k = q_k (c_k - sum_j c_j q_j) (1 - s_k),
//                             q_k = s_k / sum_j s_j;
// 0 for every other expert.
//
// Where one expert holds nearly all of the mass, c_k and the sum are nearly the
// same number and their difference is rounding.  The shares add up to 1, so the
// c may all be taken relative to that of the expert with the largest share, a:
//   c_k - sum_j c_j q_j = (c_k - c_a) - sum_j q_j (c_j - c_a).
// The large share then meets an exact 0, and what is left is off by at most
// 2 + 2 / q_a roundings of sum_j q_j |c_k - c_j|.  All in fp64, rounded once to
// the logits' type (to bf16 by way of fp32).
//
// What bounds it: latency at 4096 tokens of 256 experts (6.0 us per launch for
// the dense form, 1.4 of them the bytes; 4.8 for the selected experts'), the
// instructions beyond (23 us at 32768, the floor 11; 21 with sums in fp32).
// Slots of one expert are added up once by the lanes that hold them and meet
// their experts through LDS, in place of a search by every lane (9.7 us).
//
// Dynamic LDS, per token: a value for every expert (double; the lanes' j-th
// experts next to each other, so that their accesses meet no bank twice), then K
// slots' values (double) and experts (int).
template <typename LT, int VPL, int L>
__global__ __launch_bounds__(kRouteThreads) void route_backward_kernel(
    const LT* __restrict__ logits, const int64_t* __restrict__ topk_idx,
    const float* __restrict__ grad_weights, int T, int E, int K, bool softmax, bool normalize,
    float scale, LT* __restrict__ grad_logits, bool vec) {
    constexpr int kTokens = kRouteThreads / L;
    // slot k of a token belongs to lane k % L of its segment
    constexpr int kRounds = L == 8 ? 1 : EP_MAX_TOPK / L;       // (K <= E <= 8 with 8 lanes)
    extern __shared__ EP_LDS_ALIGN unsigned char s_raw[];
    const int sl = threadIdx.x & (L - 1);
    const int tok = threadIdx.x / L;
    const int64_t t = (int64_t)blockIdx.x * kTokens + tok;
    const bool live = t < T;
    double* s_expert = reinterpret_cast<double*>(s_raw) + tok * (VPL * L);
    double* s_slot = reinterpret_cast<double*>(s_raw) + kTokens * (VPL * L) + tok * K;
    int* s_idx =
        reinterpret_cast<int*>(s_raw + (size_t)kTokens * (VPL * L + K) * 8) + tok * K;

    const int e0 = sl * VPL;
    const LT* row = logits + t * E;
    const bool dense = softmax && !normalize;
    float l[VPL];
    if (dense && live) {
        load_row<VPL>(l, row, e0, E, vec);
    } else {
#pragma unroll
        for (int j = 0; j < VPL; ++j) l[j] = -INFINITY;
    }
    int e[kRounds];
    double c[kRounds];
#pragma unroll
    for (int i = 0; i < kRounds; ++i) {
        const int k = sl + i * L;
        const bool held = live && k < K;
        const int64_t e64 = held ? topk_idx[t * K + k] : -1;
        e[i] = e64 >= 0 && e64 < E ? (int)e64 : -1;
        c[i] = e[i] >= 0 ? (double)scale * (double)grad_weights[t * K + k] : 0.0;
        if (k < K) s_idx[k] = e[i];
    }
#pragma unroll
    for (int j = 0; j < VPL; ++j) s_expert[j * L + sl] = 0.0;

    if (!dense) {
        // c becomes the slot's gradient
        float v[kRounds];
        double u[kRounds];
        float m = -kFltMax;
#pragma unroll
        for (int i = 0; i < kRounds; ++i) {
            v[i] = e[i] >= 0 ? clean_logit(load_logit(row + e[i])) : -INFINITY;
            m = fmaxf(m, v[i]);
        }
        double ca = 0.0, total = 1.0, mean = 0.0;
        if (normalize) {
            m = seg_max<L>(m);
            ca = -INFINITY;
#pragma unroll
            for (int i = 0; i < kRounds; ++i) ca = larger(ca, v[i] == m ? c[i] : -INFINITY);
            ca = seg_max<L>(ca);
            ca = ca > -INFINITY ? ca : 0.0;
            total = 0.0;
        }
#pragma unroll
        for (int i = 0; i < kRounds; ++i) {
            u[i] = 0.0;
            if (e[i] >= 0)
                u[i] = softmax ? exp((double)v[i] - (double)m) : sigmoid64((double)v[i]);
            c[i] -= ca;
            if (normalize) {
                total += u[i];
                mean += u[i] * c[i];
            }
        }
        if (normalize) {
            total = seg_sum<L>(total);
            mean = seg_sum<L>(mean);
            mean = total > 0.0 ? mean / total : 0.0;
        }
#pragma unroll
        for (int i = 0; i < kRounds; ++i) {
            double d = total > 0.0 ? u[i] / total * (c[i] - mean) : 0.0;
            if (!softmax && e[i] >= 0) d *= sigmoid64(-(double)v[i]);
            c[i] = e[i] >= 0 ? d : 0.0;
        }
    }
#pragma unroll
    for (int i = 0; i < kRounds; ++i)
        if (sl + i * L < K) s_slot[sl + i * L] = c[i];
    wave_sync();
    // slots of one expert add up in slot order
#pragma unroll
    for (int i = 0; i < kRounds; ++i) {
        if (i * L >= K) break;
        double v = 0.0;
        for (int k = 0; k < K; ++k) v += s_idx[k] == e[i] ? s_slot[k] : 0.0;
        if (e[i] >= 0) s_expert[e[i] % VPL * L + e[i] / VPL] = v;
    }
    wave_sync();
    double o[VPL];
#pragma unroll
    for (int j = 0; j < VPL; ++j) o[j] = s_expert[j * L + sl];
    if (dense) {
        float m = -kFltMax;
#pragma unroll
        for (int j = 0; j < VPL; ++j) {
            l[j] = clean_logit(l[j]);
            m = fmaxf(m, l[j]);
        }
        m = seg_max<L>(m);
        double ca = -INFINITY;
#pragma unroll
        for (int j = 0; j < VPL; ++j) ca = larger(ca, l[j] == m ? o[j] : -INFINITY);
        ca = seg_max<L>(ca);
        ca = ca > -INFINITY ? ca : 0.0;
        double p[VPL], total = 0.0, mean = 0.0;
#pragma unroll
        for (int j = 0; j < VPL; ++j) {
            p[j] = exp((double)l[j] - (double)m);
            o[j] -= ca;
            total += p[j];
            mean += p[j] * o[j];
        }
        total = seg_sum<L>(total);
        const double inv = total > 0.0 ? 1.0 / total : 0.0;
        mean = seg_sum<L>(mean) * inv;
#pragma unroll
        for (int j = 0; j < VPL; ++j) o[j] = p[j] * inv * (o[j] - mean);
    }
    float of[VPL];
#pragma unroll
    for (int j = 0; j < VPL; ++j) of[j] = (float)o[j];
    if (live) store_row<VPL>(of, grad_logits + t * E, e0, E, vec);
}

bool rows_vectorised(const void* p, size_t elem, int E) {
    return (reinterpret_cast<uintptr_t>(p) & 15u) == 0 && (E * elem) % 16 == 0;
}

template <typename LT, int VPL, int L>
hipError_t launch_route_l(const LT* logits, const float* bias, int T, int E, int K, bool softmax,
                          int NG, int TG, bool normalize, float scale, int64_t* topk_idx,
                          float* topk_weights, hipStream_t s) {
    constexpr int kTokens = kRouteThreads / L;
    const dim3 grid((unsigned)((T + kTokens - 1) / kTokens)), block(kRouteThreads);
    const bool vec = rows_vectorised(logits, sizeof(LT), E);
    size_t lds = ((size_t)kTokens * (E + K) * 4 + 15) & ~(size_t)15;
    if (NG > 1) lds += (size_t)kTokens * (E + 2 * NG) * 8;
    if (bias || NG > 1)
        hipLaunchKernelGGL((route_kernel<LT, VPL, L, true>), grid, block, lds, s, logits, bias, T,
                           E, K, softmax, NG, TG, normalize, scale, topk_idx, topk_weights, vec);
    else
        hipLaunchKernelGGL((route_kernel<LT, VPL, L, false>), grid, block, lds, s, logits, bias,
                           T, E, K, softmax, NG, TG, normalize, scale, topk_idx, topk_weights,
                           vec);
    return hipGetLastError();
}

template <typename LT, int VPL, int L>
hipError_t launch_route_backward_l(const LT* logits, const int64_t* topk_idx, const float* gw,
                                   int T, int E, int K, bool softmax, bool normalize, float scale,
                                   LT* grad_logits, hipStream_t s) {
    constexpr int kTokens = kRouteThreads / L;
    const dim3 grid((unsigned)((T + kTokens - 1) / kTokens)), block(kRouteThreads);
    const bool vec = rows_vectorised(logits, sizeof(LT), E) &&
                     rows_vectorised(grad_logits, sizeof(LT), E);
    const size_t lds = (size_t)kTokens * (VPL * L * 8 + K * 12);
    hipLaunchKernelGGL((route_backward_kernel<LT, VPL, L>), grid, block, lds, s, logits, topk_idx,
                       gw, T, E, K, softmax, normalize, scale, grad_logits, vec);
    return hipGetLastError();
}

// Experts per lane and lanes per token: a whole wave for a token while the
// batch is small (short chains) and beyond 256 experts, fewer lanes otherwise
// (less work per token).  On MI355X, us per launch, wave / fewer lanes, K = 6 or 8:
//   tokens               128         2048        4096        16384
//   by logits, fp32
//     64 experts      3.7 / 3.6   3.9 / 3.7   4.7 / 3.8   10.0 / 5.4
//    128              3.9 / 4.4   4.5 / 4.6   5.4 / 4.7   12.2 / 8.1
//    256              4.3 / 4.7   5.0 / 4.8   6.3 / 6.0   14.8 / 13.0
//    512              5.0 / 6.8   6.3 / 7.0   8.6 / 9.7   21.6 / 24.7
//   bias, 8 groups, sigmoid, normalised
//     64              5.3 / 5.7   5.7 / 5.8   7.4 / 6.0   18.0 / 10.0
//    128              5.9 / 7.9   6.5 / 8.2   8.6 / 8.3   21.6 / 17.0
//    256              6.7 / 8.3   7.7 / 8.4  10.6 / 10.9  27.9 / 27.7
//    512              8.7 / 13.0 11.1 / 13.3 17.1 / 19.1  45.7 / 53.4
//   gradient, softmax over all experts
//     64              3.2 / 3.6   3.6 / 3.8   4.2 / 3.8    9.1 / 5.5
//    128              3.3 / 4.1   3.9 / 4.3   4.7 / 4.5   11.1 / 7.7
//    256              3.5 / 4.0   4.2 / 4.5   5.5 / 5.5   14.2 / 12.4
//    512              4.0 / 5.2   5.5 / 6.5   7.7 / 8.6   22.4 / 22.5
#define EP_ROUTE_DISPATCH(FN, LT, ...)                                             \
    do {                                                                           \
        const bool few = T <= kRouteWideTokens;                                    \
        if (E <= 8) return FN<LT, 1, 8>(__VA_ARGS__);                              \
        if (E <= 64)                                                               \
            return few ? FN<LT, 1, 64>(__VA_ARGS__) : FN<LT, 4, 16>(__VA_ARGS__);  \
        if (E <= 128)                                                              \
            return few ? FN<LT, 2, 64>(__VA_ARGS__) : FN<LT, 8, 16>(__VA_ARGS__);  \
        if (E <= 256)                                                              \
            return few ? FN<LT, 4, 64>(__VA_ARGS__) : FN<LT, 8, 32>(__VA_ARGS__);  \
        if (E <= 512) return FN<LT, 8, 64>(__VA_ARGS__);                           \
        return FN<LT, 16, 64>(__VA_ARGS__);                                        \
    } while (0)

template <typename LT>
hipError_t route_any(const void* logits, const float* bias, int T, int E, int K, bool softmax,
                     int NG, int TG, bool normalize, float scale, int64_t* topk_idx,
                     float* topk_weights, hipStream_t s) {
    EP_ROUTE_DISPATCH(launch_route_l, LT, static_cast<const LT*>(logits), bias, T, E, K, softmax,
                      NG, TG, normalize, scale, topk_idx, topk_weights, s);
}

template <typename LT>
hipError_t route_backward_any(const void* logits, const int64_t* topk_idx, const float* gw, int T,
                              int E, int K, bool softmax, bool normalize, float scale,
                              void* grad_logits, hipStream_t s) {
    EP_ROUTE_DISPATCH(launch_route_backward_l, LT, static_cast<const LT*>(logits), topk_idx, gw, T,
                      E, K, softmax, normalize, scale, static_cast<LT*>(grad_logits), s);
}

}  // namespace

hipError_t launch_route(const void* logits, bool bf16, const float* bias, int T, int E, int K,
                        bool softmax, int NG, int TG, bool normalize, float scale,
                        int64_t* topk_idx, float* topk_weights, hipStream_t s) {
    const int64_t slice = max_launch_tokens(64);
    for (int64_t t = 0; t < T; t += slice) {
        const int n = (int)(T - t < slice ? T - t : slice);
        const void* l = static_cast<const char*>(logits) + t * E * (bf16 ? 2 : 4);
        const hipError_t e =
            bf16 ? route_any<uint16_t>(l, bias, n, E, K, softmax, NG, TG, normalize, scale,
                                       topk_idx + t * K, topk_weights + t * K, s)
                 : route_any<float>(l, bias, n, E, K, softmax, NG, TG, normalize, scale,
                                    topk_idx + t * K, topk_weights + t * K, s);
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

hipError_t launch_route_backward(const void* logits, bool bf16, const int64_t* topk_idx,
                                 const float* gw, int T, int E, int K, bool softmax,
                                 bool normalize, float scale, void* grad_logits, hipStream_t s) {
    const int64_t slice = max_launch_tokens(64);
    for (int64_t t = 0; t < T; t += slice) {
        const int n = (int)(T - t < slice ? T - t : slice);
        const int64_t at = t * E * (bf16 ? 2 : 4);
        const void* l = static_cast<const char*>(logits) + at;
        void* g = static_cast<char*>(grad_logits) + at;
        const hipError_t e =
            bf16 ? route_backward_any<uint16_t>(l, topk_idx + t * K, gw + t * K, n, E, K, softmax,
                                                normalize, scale, g, s)
                 : route_backward_any<float>(l, topk_idx + t * K, gw + t * K, n, E, K, softmax,
                                             normalize, scale, g, s);
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

}  // namespace ep
