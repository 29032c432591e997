// The gated activation between an expert's two products, and its gradient, on
// gfx950: of a row's 2N channels (gate, then up)
//   y = silu(gate) * up,   silu(v) = v / (1 + exp(-v)),
// in fp32, rounded once, to bf16 or to E4M3 with a scale per 128 channels as
// dispatch writes its rows; and with s = 1 / (1 + exp(-gate))
//   d gate = grad_y * up * (s + gate * s * (1 - s)),   d up = grad_y * gate * s.
//
// Bound by HBM: every element is read and written once.  A workgroup takes a
// tile of rows; which of them an expert holds is one 64-bit mask, which every
// wave makes for itself from the experts' runs (64 experts a step, one per
// lane), so that holes between runs are neither read nor written.
#include "ep_internal.h"
#include "ep_device.h"

namespace ep {
namespace {

struct GateArgs {
    const uint16_t* a;       // gate_up [rows][2N]
    const uint16_t* gy;      // gradient: [rows][N]
    RowRuns runs;            // counts null: every row
    int64_t rows;
    int N, tile;             // rows of a workgroup, at most 64
    int64_t tile0;           // of the launch's first workgroup
    uint16_t* y;             // bf16 [rows][N]; gradient: [rows][2N]
    uint8_t* codes;
    float* scales;
};

__device__ __forceinline__ uint64_t low_bits(int64_t n) {
    return n >= 64 ? ~0ull : n <= 0 ? 0ull : (1ull << n) - 1;
}

// Bit i: an expert holds row r0 + i.
__device__ __forceinline__ uint64_t held_rows(const RowRuns& runs, int64_t r0) {
    uint64_t m = 0;
    for (int e = threadIdx.x & 63; e < runs.E; e += 64) {
        int64_t b;
        const int64_t n = runs.of(e, b);
        if (n > 0) m |= low_bits(b + n - r0) & ~low_bits(b - r0);
    }
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) m |= (uint64_t)__shfl_xor((unsigned long long)m, d);
    return m;
}

enum { kGateBf16, kGateE4m3, kGateBackward };

template <int KIND>
__global__ __launch_bounds__(kGateThreads) void gate_kernel(const GateArgs p) {
    const int64_t r0 = (p.tile0 + blockIdx.x) * p.tile;
    const int rows = (int)min((int64_t)p.tile, p.rows - r0);
    const uint64_t held = p.runs.counts ? held_rows(p.runs, r0) : ~0ull;
    if ((held & low_bits(rows)) == 0) return;
    const int per = p.N / 8;             // chunks of 8 channels of a row
    // this thread's chunk, and what lies kGateThreads chunks on
    int r = threadIdx.x / per, c = threadIdx.x - r * per;
    const int dr = kGateThreads / per, dc = kGateThreads - dr * per;
    while (r < rows) {
        uint4 g[kGateChunks], u[kGateChunks], d[kGateChunks];
        int row[kGateChunks], at[kGateChunks];
#pragma unroll
        for (int j = 0; j < kGateChunks; ++j) {
            row[j] = r < rows && (held >> r & 1) ? r : -1;
            at[j] = c;
            if (row[j] >= 0) {           // whole groups of 16 lanes where codes are written
                const uint4* a = reinterpret_cast<const uint4*>(p.a + (r0 + r) * 2 * p.N);
                g[j] = load_nt(a + c);
                u[j] = load_nt(a + per + c);
                if constexpr (KIND == kGateBackward)
                    d[j] = load_nt(reinterpret_cast<const uint4*>(p.gy + (r0 + r) * p.N) + c);
            }
            r += dr;
            c += dc;
            if (c >= per) {
                c -= per;
                ++r;
            }
        }
#pragma unroll
        for (int j = 0; j < kGateChunks; ++j) {
            if (row[j] < 0) continue;
            float gf[8], uf[8], o[8];
            unpack8(gf, g[j]);
            unpack8(uf, u[j]);
            if constexpr (KIND == kGateBackward) {
                float df[8], e[8];
                unpack8(df, d[j]);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    // s + g s (1 - s) = s (1 + g r); q last: grad_y * up may pass fp32's
                    // range where the gradient does not
                    const Sigmoid s = sigmoid(gf[i]);
                    const float w = __builtin_fmaf(gf[i] > 17.5f ? 17.5f : gf[i], s.r, 1.0f);
                    o[i] = df[i] * (s.qr * w) * uf[i] * s.q;
                    e[i] = df[i] * s.qr * gf[i] * s.q;
                }
                uint4* out = reinterpret_cast<uint4*>(p.y + (r0 + row[j]) * 2 * p.N);
                store_nt(out + at[j], pack8(o));
                store_nt(out + per + at[j], pack8(e));
            } else {
                silu_times(gf, uf, o);
                if constexpr (KIND == kGateBf16) {
                    reinterpret_cast<uint4*>(p.y + (r0 + row[j]) * p.N)[at[j]] = pack8(o);
                } else {
                    float scale;
                    const uint2 q = quantise8(o, scale);
                    reinterpret_cast<uint2*>(p.codes + (r0 + row[j]) * p.N)[at[j]] = q;
                    if ((at[j] & 15) == 0)
                        p.scales[(r0 + row[j]) * (p.N / 128) + at[j] / 16] = scale;
                }
            }
        }
    }
}

template <int KIND>
hipError_t launch_gate(GateArgs p, hipStream_t s) {
    // tiles of about one round of chunks
    const int64_t want = (int64_t)kGateThreads * kGateChunks * 8 / p.N;
    p.tile = (int)(want < 1 ? 1 : want > 64 ? 64 : want);
    const int64_t tiles = (p.rows + p.tile - 1) / p.tile, most = max_launch_tokens(kGateThreads);
    for (int64_t t = 0; t < tiles; t += most) {
        p.tile0 = t;
        const int64_t n = tiles - t < most ? tiles - t : most;
        hipLaunchKernelGGL(gate_kernel<KIND>, dim3((unsigned)n), dim3(kGateThreads), 0, s, p);
    }
    return hipGetLastError();
}

}  // namespace

hipError_t launch_expert_swiglu(const uint16_t* a, const RowRuns& runs, int N, uint16_t* y,
                                uint8_t* codes, float* scales, hipStream_t s) {
    const GateArgs p = {a, nullptr, runs, runs.num_rows, N, 0, 0, y, codes, scales};
    return codes ? launch_gate<kGateE4m3>(p, s) : launch_gate<kGateBf16>(p, s);
}

hipError_t launch_expert_swiglu_backward(const uint16_t* gy, const uint16_t* a, const RowRuns& runs,
                                         int N, uint16_t* ga, hipStream_t s) {
    const GateArgs p = {a, gy, runs, runs.num_rows, N, 0, 0, ga, nullptr, nullptr};
    return launch_gate<kGateBackward>(p, s);
}

}  // namespace ep
