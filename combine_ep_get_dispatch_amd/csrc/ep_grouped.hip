// The experts' products over ragged runs of rows, and their gradients, on
// gfx950:
//   y[r, n]  = sum_i x[r, i] * w[e, n, i]        e the expert of row r
//   gx[r, i] = sum_n gy[r, n] * w[e, n, i]
//   gw[e, n, i] = sum over e's rows r of gy[r, n] * x[r, i]
// in bf16, or y from E4M3 rows and weights, whose codes' products are summed
// over 128 channels and then scaled, fp32 throughout and rounded once.
#include "ep_internal.h"
#include "ep_device.h"

#include <type_traits>

namespace ep {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

enum Product { kRows, kGradRows, kGradWeight };

struct ProductArgs {
    const uint8_t* a;      // what the results' neighbouring channels come from: w, w or x
    const uint8_t* b;      // what the results' rows come from: x, gy or gy
    const float* as;       // scales (E4M3)
    const float* bs;
    RowRuns runs;
    int K;                 // summed channels (kGradWeight: the experts' rows are summed)
    int M;                 // results' channels: N, I or I
    int B;                 // kGradWeight: results' rows per expert, N
    void* y;
};

// A workgroup's tile: 256 channels by up to 256 rows of results, summed in
// steps of 128 bytes (64 bf16 or 128 E4M3 channels).
constexpr int kTileM = 256;
constexpr int kStepBytes = 128;
constexpr int kWaves = 8;
constexpr int kABytes = kTileM * kStepBytes;
constexpr int kStage = 2 * kABytes;


// 16 (or 4) bytes per lane from a bounded buffer to LDS, lane after lane; what
// lies past the buffer's end arrives as zeros.  Waited for by vmcnt; the
// compiler does not count it.
__device__ __forceinline__ void dma16(uint32_t at, const i32x4& buffer, uint32_t lds) {
    asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tbuffer_load_dwordx4 %0, %1, 0 offen lds"
                 :
                 : "v"(at), "s"(buffer), "s"(lds)
                 : "memory");
}
__device__ __forceinline__ void dma4(uint32_t at, const i32x4& buffer, uint32_t lds) {
    asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tbuffer_load_dword %0, %1, 0 offen lds"
                 :
                 : "v"(at), "s"(buffer), "s"(lds)
                 : "memory");
}
constexpr uint32_t kNowhere = 0x80000000u;   // past every buffer's end

__device__ __forceinline__ i32x4 make_buffer(uint64_t base, int64_t left) {
    const int64_t n = left < 0 ? 0 : left > 0x7fffffff ? 0x7fffffff : left;
    return i32x4{(int)(uint32_t)base, (int)(uint32_t)(base >> 32) & 0xffff, (int)n, 0x00020000};
}

__device__ __forceinline__ uint32_t lds_offset(const void* p) {
    return (uint32_t)(uintptr_t)(const __attribute__((address_space(3))) char*)p;
}

#define EP_WAIT_LDS() asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory")
#define EP_WAIT_DMA() asm volatile("s_waitcnt vmcnt(0)" ::: "memory")

__device__ __forceinline__ void barrier() {
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_sched_barrier(0);
}

// Row blocks of an expert with n rows for the class of row tiles RT: whole
// blocks of 256 rows and what is left over 128 in class 8, up to 128 in class
// 4, up to 64 in class 2.
template <int RT>
__device__ __forceinline__ int row_blocks(int n) {
    const int rest = n & 255;
    if (RT == 8) return (n >> 8) + (rest > 128 ? 1 : 0);
    if (RT == 4) return rest > 64 && rest <= 128 ? 1 : 0;
    return rest > 0 && rest <= 64 ? 1 : 0;
}

constexpr int kKnown = 256;
struct Blocks {
    int first[kKnown], rows[kKnown], upto[3][kKnown];
};
template <int RT>
constexpr int kClass = RT == 8 ? 0 : RT == 4 ? 1 : 2;

__device__ __forceinline__ int prefix_sum(int v) {
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int o = __shfl_up(v, d);
        if (lane >= d) v = (int)min((unsigned)v + (unsigned)o, 1u << 30);
    }
    return v;
}

struct Task {
    int e, m0, r0, n;       // expert, first channel, first row of the run, rows of the run
    int64_t begin;          // first row of the run in the rows' arrays
};

constexpr int kBand = 8;    // channel tiles whose tasks stand next to each other

// (row block, channel tile) of place `local` in bands of kBand channel tiles.
__device__ __forceinline__ void in_bands(unsigned local, unsigned nb, unsigned nt, unsigned& rb,
                                         unsigned& mt) {
    const unsigned band = local / (nb * kBand), rest = local - band * nb * kBand;
    const unsigned width = min((unsigned)kBand, nt - band * kBand);
    rb = rest / width;
    mt = band * kBand + rest - rb * width;
}

template <Product OP, int RT>
__device__ __forceinline__ bool find_task(Task& t, const ProductArgs& p, const Blocks& known,
                                          int task, int end, unsigned nt, int tile) {
    if (task >= end) return false;
    unsigned rb, mt;
    if constexpr (OP == kGradWeight) {
        const unsigned nb = (p.B + 255) / 256, per = nb * nt;
        t.e = (unsigned)task / per;
        in_bands(task - t.e * per, nb, nt, rb, mt);
        const int64_t n = p.runs.of(t.e, t.begin);
        t.n = n > 0 ? (int)n : 0;
        t.e = __builtin_amdgcn_readfirstlane(t.e);
        t.n = __builtin_amdgcn_readfirstlane(t.n);
        t.begin = __builtin_amdgcn_readfirstlane((int)t.begin);
        t.r0 = __builtin_amdgcn_readfirstlane(rb * 256);
        t.m0 = __builtin_amdgcn_readfirstlane(mt * tile);
        return true;
    }
    const int lane = threadIdx.x & 63;
    int before = 0;
#pragma unroll 1
    for (int e0 = 0; e0 < p.runs.E; e0 += 64) {
        int first, rows, upto;
        if (e0 < kKnown) {
            first = known.first[e0 + lane];
            rows = known.rows[e0 + lane];
            upto = known.upto[kClass<RT>][e0 + lane];
        } else {
            int64_t b = 0, m = 0;
            if (e0 + lane < p.runs.E) m = p.runs.of(e0 + lane, b);
            first = (int)b;
            rows = m > 0 ? (int)m : 0;
            upto = prefix_sum(row_blocks<RT>(rows)) + before;
        }
        const uint64_t hit = __ballot(upto * (int)nt > task);
        if (hit) {
            const int at = __builtin_ctzll(hit);
            t.e = e0 + at;
            t.n = __builtin_amdgcn_readlane(rows, at);
            t.begin = __builtin_amdgcn_readlane(first, at);
            const unsigned nb = row_blocks<RT>(t.n);
            const int local = task - (__builtin_amdgcn_readlane(upto, at) - (int)nb) * (int)nt;
            in_bands(local, nb, nt, rb, mt);
            t.r0 = RT == 8 ? rb * 256 : t.n & ~255;
            t.m0 = mt * tile;
            t.r0 = __builtin_amdgcn_readfirstlane(t.r0);
            t.m0 = __builtin_amdgcn_readfirstlane(t.m0);
            return true;
        }
        before = __builtin_amdgcn_readlane(upto, 63);
    }
    return false;
}

template <bool FP8>
struct ProductLds {
    uint8_t stage[2][kStage];
    float scales[2][FP8 ? 256 : 1];
    Blocks known;
};

// 16 rows by 128 bytes as matrix operands, from rows of 128 bytes in LDS.  The
// 16-byte chunk c of row r lies at place c ^ (r / 2 % 8), so that the 16 lanes
// that read a chunk of 16 rows meet 16 different places of 256 bytes.
__device__ __forceinline__ uint32_t row_place(int r, int c) {
    return r * kStepBytes + ((c ^ (r >> 1 & 7)) << 4);
}
// The same from columns: step k's `cols` columns lie in a row of their own, and
// what 16 neighbouring columns take (32 bytes) at place c ^ g(k).
__device__ __forceinline__ int column_turn(int k) { return (k & 3) | (k >> 1 & 4); }

template <Product OP, bool FP8, bool SWIGLU, bool F32, bool ADD, int RT>
__device__ __forceinline__ void run_tasks(const ProductArgs& p, ProductLds<FP8>& lds, int task,
                                          int end, int stride, unsigned nt) {
    constexpr int kTile = SWIGLU ? kTileM / 2 : kTileM;    // result channels
    constexpr bool kAT = OP != kRows;                      // a and b by columns
    constexpr bool kBT = OP == kGradWeight;
    constexpr int kElem = FP8 ? 1 : 2;
    constexpr int kStepK = kStepBytes / kElem;
    constexpr int kRowsB = 2 * RT * 16;
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int group = wave >> 2;
    const int lg = lane >> 4, lr = lane & 15;
    const uint32_t lds0 = __builtin_amdgcn_readfirstlane(lds_offset(&lds.stage[0][0]));
    const uint32_t lds_s = FP8 ? __builtin_amdgcn_readfirstlane(lds_offset(&lds.scales[0][0])) : 0;
    const int64_t a_row = (int64_t)(OP == kRows ? p.K : p.M) * kElem;     // bytes
    const int64_t b_row = (int64_t)(OP == kGradWeight ? p.B : p.K) * kElem;

    // --- what this wave fetches of a step: 1/8 of a's and of b's part ---
    constexpr int kLoadsA = 4;
    constexpr int kLoadsB = RT >= 2 ? RT / 2 : 1;
    uint32_t a_at[kLoadsA], b_at[kLoadsB];
    int a_col, b_col[2];           // by rows: byte of the step, for the last step's end
    (void)a_col;
    (void)b_col;
#pragma unroll
    for (int i = 0; i < kLoadsA; ++i) {
        if constexpr (kAT) {
            const int k = wave * 8 + i * 2 + (lane >> 5), pos = lane & 31;
            const int c = (((pos >> 1) ^ column_turn(k)) << 1) | (pos & 1);
            a_at[i] = (uint32_t)((i * 2 + (lane >> 5)) * a_row) + c * 16;
        } else {
            const int r = i * 8 + (lane >> 3), c = (lane & 7) ^ (r >> 1 & 7);
            a_at[i] = (uint32_t)(r * a_row) + c * 16;
        }
    }
#pragma unroll
    for (int i = 0; i < kLoadsB; ++i) {
        if constexpr (kBT) {
            const int k = wave * 8 + i * 2 + (lane >> 5), pos = lane & 31;
            const int c = (((pos >> 1) ^ column_turn(k)) << 1) | (pos & 1);
            b_at[i] = (uint32_t)((i * 2 + (lane >> 5)) * b_row) + c * 16;
        } else {
            const int r = wave * kLoadsB * 8 + i * 8 + (lane >> 3), c = (lane & 7) ^ (r >> 1 & 7);
            b_at[i] = (uint32_t)((r - wave * kLoadsB * 8) * b_row) + c * 16;
        }
    }

    struct {
        bool live;
        int task, step, steps;
        uint64_t a, b, s;
        int64_t a_left, b_left, s_left;
    } next;
    auto steps_of = [&](const Task& t) {
        return OP == kGradWeight ? (t.n + kStepK - 1) / kStepK : (p.K + kStepK - 1) / kStepK;
    };
    auto aim = [&](const Task& t) {
        next.step = 0;
        next.steps = steps_of(t);
        if constexpr (OP == kRows) {
            const int half = SWIGLU ? wave >> 2 : 0;
            const int c = SWIGLU ? (wave & 3) * 32 : wave * 32;
            const int64_t w0 = ((int64_t)t.e * (SWIGLU ? 2 : 1) + half) * p.M + t.m0 + c;
            next.a = (uint64_t)(p.a + w0 * a_row);
            next.a_left = min((int64_t)32, (int64_t)p.M - t.m0 - c) * a_row;
        } else if constexpr (OP == kGradRows) {
            next.a = (uint64_t)(p.a + (((int64_t)t.e * p.K + wave * 8) * a_row + t.m0 * kElem));
            next.a_left = (int64_t)(p.K - wave * 8) * a_row - t.m0 * kElem;
        } else {
            next.a = (uint64_t)(p.a + ((t.begin + wave * 8) * a_row + t.m0 * kElem));
            next.a_left = (int64_t)(t.n - wave * 8) * a_row - t.m0 * kElem;
        }
        if constexpr (OP == kGradWeight) {
            next.b = (uint64_t)(p.b + ((t.begin + wave * 8) * b_row + t.r0 * kElem));
            next.b_left = (int64_t)(t.n - wave * 8) * b_row - t.r0 * kElem;
        } else {
            const int r = wave * kLoadsB * 8;
            next.b = (uint64_t)(p.b + (t.begin + t.r0 + r) * b_row);
            next.b_left = min((int64_t)kLoadsB * 8, (int64_t)t.n - t.r0 - r) * b_row;
        }
        if constexpr (FP8) {
            const int64_t s_row = (int64_t)(p.K / 128) * 4;
            next.s = (uint64_t)p.bs + (t.begin + t.r0 + wave * 64) * s_row;
            next.s_left = min((int64_t)64, (int64_t)t.n - t.r0 - wave * 64) * s_row;
        }
    };
    // The first task from next.task on that has steps.
    auto seek = [&]() {
        Task t;
        while (true) {
            next.live = find_task<OP, RT>(t, p, lds.known, next.task, end, nt, kTile);
            if (!next.live) return;
            if (OP != kGradWeight || t.n > 0) break;
            next.task += stride;
        }
        aim(t);
    };
    auto issue = [&](int buf) {
        if (!next.live) return;
        const i32x4 ab = make_buffer(next.a, next.a_left), bb = make_buffer(next.b, next.b_left);
        const uint32_t at = lds0 + buf * kStage;
        const bool last = next.step == next.steps - 1;
        // by rows: what of the last step lies past the row's end
        const int over = last ? p.K * kElem - next.step * kStepBytes : kStepBytes;
        if (!kBT && over < kStepBytes) {
#pragma unroll
            for (int i = 0; i < kLoadsA; ++i) {
                if constexpr (kAT) {
                    dma16(a_at[i], ab, at + (wave * kLoadsA + i) * 1024);
                } else {
                    const int r = i * 8 + (lane >> 3), c = ((lane & 7) ^ (r >> 1 & 7)) << 4;
                    dma16(c < over ? a_at[i] : kNowhere, ab, at + (wave * kLoadsA + i) * 1024);
                }
            }
#pragma unroll
            for (int i = 0; i < kLoadsB; ++i) {
                const int r = wave * kLoadsB * 8 + i * 8 + (lane >> 3);
                const int c = ((lane & 7) ^ (r >> 1 & 7)) << 4;
                dma16(c < over ? b_at[i] : kNowhere, bb,
                      at + kABytes + (wave * kLoadsB + i) * 1024);
            }
        } else {
#pragma unroll
            for (int i = 0; i < kLoadsA; ++i)
                dma16(a_at[i], ab, at + (wave * kLoadsA + i) * 1024);
#pragma unroll
            for (int i = 0; i < kLoadsB; ++i)
                dma16(b_at[i], bb, at + kABytes + (wave * kLoadsB + i) * 1024);
        }
        if constexpr (FP8) {
            if (wave < (kRowsB + 63) / 64)
                dma4((uint32_t)(lane * (p.K / 128) * 4), make_buffer(next.s, next.s_left),
                     lds_s + buf * 1024 + wave * 256);
            next.s += 4;
            next.s_left -= 4;
        }
        if (last) {
            next.task += stride;
            seek();
            return;
        }
        ++next.step;
        const int64_t da = kAT ? a_row * kStepK : kStepBytes;
        const int64_t db = kBT ? b_row * kStepK : kStepBytes;
        next.a += da;
        next.a_left -= da;
        next.b += db;
        next.b_left -= db;
    };

    // --- this wave's results: 64 channels (4 tiles) by RT tiles of rows ---
    const int wm = wave & 3;
    const int wr = group;
    f32x4 acc[4][RT];
    i32x4 af[4][2], bf[RT][2];
    float sx[FP8 ? RT : 1];
    auto a_tile = [&](int ct) {      // first of the tile's 16 channels in LDS
        return SWIGLU ? (ct >> 1) * 128 + wm * 32 + (ct & 1) * 16 : wm * 64 + ct * 16;
    };
    const uint32_t a_read = row_place((SWIGLU ? wm * 32 : wm * 64) + lr, lg);
    const uint32_t b_read = row_place(wr * RT * 16 + lr, lg);
    auto by_columns = [&](const uint8_t* s, int col0, int ks) {
        // 16 columns from col0 (a multiple of 16), 32 steps of k
        const int k = lg * 8 + (lr >> 2);
        const uint32_t at =
            k * 512 + (((col0 >> 4) ^ column_turn(k)) << 5) + ((lr & 3) << 3) + ks * 32 * 512;
        typedef __attribute__((address_space(3))) s16x4 L;
        const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((L*)(s + at));
        const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((L*)(s + at + 4 * 512));
        const uint64_t l = __builtin_bit_cast(uint64_t, lo), h = __builtin_bit_cast(uint64_t, hi);
        return i32x4{(int)(uint32_t)l, (int)(uint32_t)(l >> 32), (int)(uint32_t)h,
                     (int)(uint32_t)(h >> 32)};
    };
    auto read = [&](int buf) {
        const uint8_t* s = lds.stage[buf];
#pragma unroll
        for (int ct = 0; ct < 4; ++ct)
#pragma unroll
            for (int ks = 0; ks < 2; ++ks) {
                if constexpr (kAT)
                    af[ct][ks] = by_columns(s, a_tile(ct), ks);
                else
                    af[ct][ks] = *reinterpret_cast<const i32x4*>(
                        s + (a_read ^ ks * 64) +
                        (SWIGLU ? (ct >> 1) * 128 + (ct & 1) * 16 : ct * 16) * kStepBytes);
            }
#pragma unroll
        for (int rt = 0; rt < RT; ++rt)
#pragma unroll
            for (int ks = 0; ks < 2; ++ks) {
                if constexpr (kBT)
                    bf[rt][ks] = by_columns(s + kABytes, (wr * RT + rt) * 16, ks);
                else
                    bf[rt][ks] = *reinterpret_cast<const i32x4*>(
                        s + kABytes + (b_read ^ ks * 64) + rt * 16 * kStepBytes);
            }
        if constexpr (FP8) {
#pragma unroll
            for (int rt = 0; rt < RT; ++rt) sx[rt] = lds.scales[buf][(wr * RT + rt) * 16 + lr];
        }
    };
    auto multiply = [&](const float* as, int step) {
        if constexpr (FP8) {
            const int KB = p.K / 128, NB = (p.M + 127) / 128;
            const float s0 = as[step], s1 = SWIGLU ? as[(int64_t)NB * KB + step] : s0;
            const f32x4 zero = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int rt = 0; rt < RT; ++rt) {
                const float g = sx[rt] * s0, u = sx[rt] * s1;
                i32x8 b;
#pragma unroll
                for (int i = 0; i < 8; ++i) b[i] = bf[rt][i / 4][i % 4];
#pragma unroll
                for (int ct = 0; ct < 4; ++ct) {
                    i32x8 a;
#pragma unroll
                    for (int i = 0; i < 8; ++i) a[i] = af[ct][i / 4][i % 4];
                    const f32x4 t = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                        a, b, zero, 0, 0, 0, 127, 0, 127);
                    const float sc = SWIGLU && ct >= 2 ? u : g;
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        acc[ct][rt][i] = __builtin_fmaf(t[i], sc, acc[ct][rt][i]);
                }
            }
        } else {
#pragma unroll
            for (int ks = 0; ks < 2; ++ks)
#pragma unroll
                for (int rt = 0; rt < RT; ++rt)
#pragma unroll
                    for (int ct = 0; ct < 4; ++ct)
                        acc[ct][rt] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                            __builtin_bit_cast(bf16x8, af[ct][ks]),
                            __builtin_bit_cast(bf16x8, bf[rt][ks]), acc[ct][rt], 0, 0, 0);
        }
    };
    auto store = [&](const Task& t) {
        const int rows = OP == kGradWeight ? p.B : t.n;
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) {
            const int r = t.r0 + (wr * RT + rt) * 16 + lr;
            if (r >= rows) continue;
            const int64_t at =
                (OP == kGradWeight ? (int64_t)t.e * p.B + r : t.begin + r) * p.M + t.m0;
#pragma unroll
            for (int ct = 0; ct < (SWIGLU ? 2 : 4); ++ct) {
                const int c = (SWIGLU ? wm * 32 : wm * 64) + ct * 16 + lg * 4;
                if (t.m0 + c >= p.M) continue;
                f32x4 v = acc[ct][rt];
                if constexpr (SWIGLU) {
                    const f32x4 u = acc[ct + 2][rt];
#pragma unroll
                    for (int i = 0; i < 4; ++i) v[i] = v[i] / (1.0f + expf(-v[i])) * u[i];
                }
                if constexpr (F32) {
                    f32x4* o = reinterpret_cast<f32x4*>(static_cast<float*>(p.y) + at + c);
                    if constexpr (ADD) v += *o;
                    *o = v;
                } else {
                    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.y) + at + c) =
                        make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
                }
            }
        }
    };

    // --- the steps ---
    // Waves 0..3 and 4..7, one of each on a SIMD, take turns: while one half
    // multiplies a step, the other reads its operands.  A step's bytes are asked
    // for as soon as every wave has read the step that lay there before.
    next.task = task;
    seek();
    int buf = 0;
    issue(0);
    EP_WAIT_DMA();
    barrier();
    if (group == 1) {
        issue(1);
        barrier();
    }
    Task t;
    for (; find_task<OP, RT>(t, p, lds.known, task, end, nt, kTile); task += stride) {
        const int steps = steps_of(t);
        const float* as = nullptr;
        if constexpr (FP8) {
            const int KB = p.K / 128, NB = (p.M + 127) / 128;
            const int c = t.m0 + (SWIGLU ? wm * 32 : wm * 64);
            as = p.as + ((int64_t)t.e * (SWIGLU ? 2 : 1) * NB + min(c / 128, NB - 1)) * KB;
        }
#pragma unroll
        for (int ct = 0; ct < 4; ++ct)
#pragma unroll
            for (int rt = 0; rt < RT; ++rt) acc[ct][rt] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 1
        for (int step = 0; step < steps; ++step, buf ^= 1) {
            read(buf);
            if (group == 0)
                issue(buf ^ 1);
            else
                EP_WAIT_DMA();
            EP_WAIT_LDS();
            barrier();
            if (group == 1) issue(buf);
            multiply(as, step);
            if (group == 0) EP_WAIT_DMA();
            barrier();
        }
        if (OP == kGradWeight && ADD && t.n == 0) continue;
        store(t);
    }
    if (group == 0) barrier();
    barrier();
}

template <Product OP, bool FP8, bool SWIGLU, bool F32, bool ADD>
__global__ __launch_bounds__(kWaves * 64, 2) void product_kernel(const ProductArgs p) {
    __shared__ __attribute__((aligned(1024))) ProductLds<FP8> lds;
    const int lane = threadIdx.x & 63;
    constexpr int kTile = SWIGLU ? kTileM / 2 : kTileM;
    const unsigned nt = (p.M + kTile - 1) / kTile;
    const int stride = gridDim.x / kXcds, xcd = blockIdx.x % kXcds;
    int slot = blockIdx.x / kXcds;
    if constexpr (OP == kGradWeight) {
        const int tasks = p.runs.E * ((p.B + 255) / 256) * nt, per = (tasks + kXcds - 1) / kXcds;
        run_tasks<OP, FP8, SWIGLU, F32, ADD, 8>(p, lds, xcd * per + slot,
                                                min(tasks, (xcd + 1) * per), stride, nt);
    } else {
        // Row blocks of the classes; every wave writes the same numbers, and reads
        // its own.
        int64_t sum[3] = {0, 0, 0};
#pragma unroll 1
        for (int e0 = 0; e0 < p.runs.E; e0 += 64) {
            int64_t b = 0, m = 0;
            if (e0 + lane < p.runs.E) m = p.runs.of(e0 + lane, b);
            const int rows = m > 0 ? (int)m : 0;
            const int upto[3] = {prefix_sum(row_blocks<8>(rows)), prefix_sum(row_blocks<4>(rows)),
                                 prefix_sum(row_blocks<2>(rows))};
            if (e0 < kKnown) {
                lds.known.first[e0 + lane] = (int)b;
                lds.known.rows[e0 + lane] = rows;
            }
#pragma unroll
            for (int c = 0; c < 3; ++c) {
                if (e0 < kKnown) lds.known.upto[c][e0 + lane] = (int)(sum[c] + upto[c]);
                sum[c] += __builtin_amdgcn_readlane(upto[c], 63);
            }
        }
        // (a y of 2^30 tasks fits no memory: such counts do not belong to these rows)
        if ((sum[0] + sum[1] + sum[2]) * nt >= 1 << 30) return;
        auto run = [&](auto rt, int c) {
            if (sum[c] == 0) return;
            const int tasks = (int)sum[c] * nt, per = (tasks + kXcds - 1) / kXcds;
            run_tasks<OP, FP8, SWIGLU, F32, ADD, decltype(rt)::value>(
                p, lds, xcd * per + slot, min(tasks, (xcd + 1) * per), stride, nt);
            slot = (slot + stride - per % stride) % stride;
        };
        run(std::integral_constant<int, 8>{}, 0);
        run(std::integral_constant<int, 4>{}, 1);
        run(std::integral_constant<int, 2>{}, 2);
    }
}

template <Product OP, bool FP8, bool SWIGLU, bool F32, bool ADD>
hipError_t launch(const ProductArgs& p, int64_t tasks, hipStream_t s) {
    const unsigned grid = (unsigned)((tasks < kCus ? tasks : kCus) + kXcds - 1) / kXcds * kXcds;
    hipLaunchKernelGGL((product_kernel<OP, FP8, SWIGLU, F32, ADD>), dim3(grid), dim3(kWaves * 64),
                       0, s, p);
    return hipGetLastError();
}

// At most so many row blocks.
int64_t most_blocks(const RowRuns& r) {
    return r.offsets ? r.E + r.num_rows / 256
                     : (int64_t)r.E * (((int64_t)r.capacity + 255) / 256);
}

}  // namespace

hipError_t launch_expert_linear(const void* x, const float* xs, const RowRuns& runs, int I, int N,
                                const void* w, const float* ws, bool swiglu, uint16_t* y,
                                hipStream_t s) {
    if (runs.num_rows == 0) return hipSuccess;
    const ProductArgs p = {static_cast<const uint8_t*>(w), static_cast<const uint8_t*>(x), ws, xs,
                           runs, I, N, 0, y};
    const int tile = swiglu ? kTileM / 2 : kTileM;
    const int64_t tasks = most_blocks(runs) * ((N + tile - 1) / tile);
    if (xs)
        return swiglu ? launch<kRows, true, true, false, false>(p, tasks, s)
                      : launch<kRows, true, false, false, false>(p, tasks, s);
    return swiglu ? launch<kRows, false, true, false, false>(p, tasks, s)
                  : launch<kRows, false, false, false, false>(p, tasks, s);
}

hipError_t launch_expert_grad_rows(const uint16_t* gy, const RowRuns& runs, int I, int N,
                                   const uint16_t* w, uint16_t* gx, hipStream_t s) {
    if (runs.num_rows == 0) return hipSuccess;
    const ProductArgs p = {reinterpret_cast<const uint8_t*>(w),
                           reinterpret_cast<const uint8_t*>(gy),
                           nullptr, nullptr, runs, N, I, 0, gx};
    return launch<kGradRows, false, false, false, false>(
        p, most_blocks(runs) * ((I + kTileM - 1) / kTileM), s);
}

hipError_t launch_expert_grad_weight(const uint16_t* gy, const uint16_t* x, const RowRuns& runs,
                                     int I, int N, void* gw, bool fp32, bool accumulate,
                                     hipStream_t s) {
    const ProductArgs p = {reinterpret_cast<const uint8_t*>(x),
                           reinterpret_cast<const uint8_t*>(gy),
                           nullptr, nullptr, runs, 0, I, N, gw};
    const int64_t tasks =
        (int64_t)runs.E * ((N + 255) / 256) * ((I + kTileM - 1) / kTileM);
    if (!fp32) return launch<kGradWeight, false, false, false, false>(p, tasks, s);
    return accumulate ? launch<kGradWeight, false, false, true, true>(p, tasks, s)
                      : launch<kGradWeight, false, false, true, false>(p, tasks, s);
}

}  // namespace ep
