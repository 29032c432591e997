// The experts' products over ragged runs of rows, and their gradients, on
// gfx950:
//   y[r, n]     = sum_i x[r, i] * w[e, n, i]        e the expert of row r
//   gx[r, i]    = sum_n gy[r, n] * w[e, n, i]
//   gw[e, n, i] = sum over e's rows r of gy[r, n] * x[r, i]
// in bf16, or y from E4M3 rows and weights, whose codes' products are summed
// over 128 channels and then scaled, fp32 throughout and rounded once.
//
// What bounds it.  With n rows an expert, a weight of b bytes takes 2n operations: up to
// about 128 rows (bf16) the weights' way from HBM, beyond that the matrix instructions,
// and for long sums the card's power: while it multiplies without a pause it lowers its
// clock, from 2.4 to 1.9 GHz and less, and a library product of the same size does no
// better than 1.2 times these kernels' rate (65521 x 4096 -> 2048, 8 experts: 852-880 us,
// one library product of as many rows 715 in short runs and 940 in long ones).
//
// Layout.  What gives the results' neighbouring channels (a: weights, or x for gw) is the
// A operand, what gives their rows (b: rows, or gy for gw) the B operand, so that a lane
// ends with four neighbouring channels of one row.  A workgroup owns 256 channels by up to
// 256 rows; both operands' tiles come to LDS by loads that go there directly, in steps of
// 128 bytes of summed channels, bounded by buffer ranges: what lies past a run's last row,
// the last channel or the matrix's end arrives as zeros, and neither a short run nor an odd
// size needs a branch of its own.  (A step by rows that ends inside 128 bytes sends its lanes
// past the range by itself.)  Where the summed index is the slow one (the weights of gx,
// both operands of gw) a step's columns lie in LDS as they came, and the reads that
// transpose make operands of them.  Chunks of 16 or 32 bytes change places with the row
// (row_place, column_turn), so that no read of an operand meets a bank conflict (counted: 0).
//
// Eight waves, four of 64 channels on either half of the rows; a half's row tiles are in
// registers (128 sums a lane).  The halves take turns at reading and multiplying (see
// run_tasks).  Rows per block: whole blocks of 256, what is left in blocks of up to 256, 128
// or 64, so that the last block of an expert costs what its rows need.
//
// What it took on MI355X (65521 x 4096 -> 2048 bf16 / 16384 x 7168 -> 2 x 2048 E4M3):
// 1007 / 1194 us with both halves fetching at once; 1003 / 842 with one half fetching
// and addresses made where they are used (registers had gone to scratch, whose reads waited
// for the loads to LDS); 943 / 749 with b in two parts, which lets each place be asked for
// five phases ahead; 943 / 637 with sums scaled two tiles late; 884 / 605 with four loads an
// address setting (loads between the matrix instructions instead: 1035 / 697); 861 / 576 with
// what is left of the largest blocks in pieces; 852 / 565 with whole lines stored.  Tried
// without gain: 32 x 32 matrix instructions (908), wave priorities, stores that the next
// step does not wait for.  (E4M3, counted: the matrix units busy 41% of the cycles, bf16
// 62; 5.7 other vector instructions a matrix instruction, four of them the scaling; 10%
// more matrix instructions than the rows need, for blocks left part empty.)
//
// Not split: a sum over an expert's rows (gw).  Few tiles of many rows leave most of the
// card idle: 65536 rows, 64 x 64 weights 866 us, 8 x 8192 rows, 512 x 512 123.
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
// Of a step's rows a part of up to 128 is read at a time: class 8 has two parts and
// places for two steps, the others one part and places for three.
constexpr int kBPart = kABytes / 2;
template <int RT>
constexpr int kParts = RT == 8 ? 2 : 1;
template <int RT>
constexpr int kStages = RT == 8 ? 2 : 3;
constexpr int kStageBytes = 3 * (kABytes + kBPart);
// E4M3 rows' scales, four steps' at a time, in a ring of places.
constexpr int kScaleSteps = 4, kScalePlaces = 4;

// 16 bytes per lane from a bounded buffer to LDS, lane after lane, N loads
// one after the other; what lies past the buffer's end arrives as zeros.  A load's
// place i * kLoadBytes counts in both memories, so `at` holds what is missing from
// kShift, which the buffer's base makes up for.  Waited for by vmcnt; the compiler
// does not count it (where it waits for loads of its own it waits for more than it
// knows, never for less).  M0 holds the place in LDS: each block sets it and says so.
constexpr int kLoadBytes = 1024, kShift = 3 * kLoadBytes;
template <int N>
__device__ __forceinline__ void dma16(const uint32_t* at, const i32x4& buffer, uint32_t lds) {
    if constexpr (N == 4)
        asm volatile(
            "s_mov_b32 m0, %5\n\ts_nop 0\n\t"
            "buffer_load_dwordx4 %0, %4, 0 offen lds\n\t"
            "buffer_load_dwordx4 %1, %4, 0 offen offset:%6 lds\n\t"
            "buffer_load_dwordx4 %2, %4, 0 offen offset:%7 lds\n\t"
            "buffer_load_dwordx4 %3, %4, 0 offen offset:%8 lds"
            :
            : "v"(at[0]), "v"(at[1]), "v"(at[2]), "v"(at[3]), "s"(buffer), "s"(lds),
              "n"(kLoadBytes), "n"(2 * kLoadBytes), "n"(3 * kLoadBytes)
            : "memory", "m0");
    else if constexpr (N == 2)
        asm volatile(
            "s_mov_b32 m0, %3\n\ts_nop 0\n\t"
            "buffer_load_dwordx4 %0, %2, 0 offen lds\n\t"
            "buffer_load_dwordx4 %1, %2, 0 offen offset:%4 lds"
            :
            : "v"(at[0]), "v"(at[1]), "s"(buffer), "s"(lds), "n"(kLoadBytes)
            : "memory", "m0");
    else
        asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tbuffer_load_dwordx4 %0, %1, 0 offen lds"
                     :
                     : "v"(at[0]), "s"(buffer), "s"(lds)
                     : "memory", "m0");
}
constexpr uint32_t kNowhere = 0x80000000u;   // past every buffer's end

// `size` bytes (0 or less: none) from `base`, which the loads reach at kShift.
__device__ __forceinline__ i32x4 make_buffer(uint64_t base, int size) {
    base -= kShift;
    return i32x4{__builtin_amdgcn_readfirstlane((int)(uint32_t)base),
                 __builtin_amdgcn_readfirstlane((int)(uint32_t)(base >> 32) & 0xffff),
                 __builtin_amdgcn_readfirstlane(max(0, size) + kShift), 0x00020000};
}

__device__ __forceinline__ uint32_t lds_offset(const void* p) {
    return (uint32_t)(uintptr_t)(const __attribute__((address_space(3))) char*)p;
}

#define EP_WAIT_LDS() asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory")
// Waits until at most N loads to LDS (and stores) are still on their way.
template <int N>
__device__ __forceinline__ void wait_dma() {
    asm volatile("s_waitcnt vmcnt(%0)" : : "n"(N) : "memory");
}

// A barrier that, unlike __syncthreads, does not wait for loads to LDS on their way;
// no access to memory moves across.
__device__ __forceinline__ void barrier() {
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
}

// Row blocks of an expert with n rows, by lists: whole blocks of 256 rows and what is
// left over 128 in list 0, up to 128 in list 1, up to 64 in list 2.
__device__ __forceinline__ int row_blocks(int list, int n) {
    const int rest = n & 255;
    return list == 0   ? (n >> 8) + (rest > 128 ? 1 : 0)
           : list == 1 ? (rest > 64 && rest <= 128 ? 1 : 0)
                       : (rest > 0 && rest <= 64 ? 1 : 0);
}

constexpr int kKnown = 256;
struct Blocks {
    int first[kKnown], rows[kKnown], upto[3][kKnown];
};
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

// Tasks of 256 channels that run as eight times as many of 32: as many as the workgroups
// take in one round, or in two where no expert has more than 32 rows and the waves have
// three steps each or more.  Measured in us, as tasks of 256 / of 32:
//   one round: 7168 -> 2 x 2048, E4M3, one expert x 1 row 51 / 15, x 64 rows 52 / 37,
//   4 experts x 16 rows 52 / 35; 2048 -> 7168, bf16, one expert x 1 row 27 / 13, 2 x 16 rows
//   27 / 23.  Of few steps, 32 tasks x 64 rows: E4M3 128 -> 2 x 4096 (1 step) 8.7 / 6.1, 1024
//   (8 steps) 14.6 / 15.9, 2048 (16) 21.3 / 18.0; bf16 128 -> 8192 (2) 9.0 / 6.1, 1024 18.4 / 12.7.
//   two rounds, 64 tasks x 32 rows: E4M3 512 (4 steps) 10.5 / 12.7, 1024 13.9 / 24.9, 2048 20.6 /
//   27.7, 2560 (20) 24.1 / 25.4, 3584 (28) 30.3 / 28.1, 7168 62 / 55; bf16 512 (8) 12.4 / 17.2, 1024
//   17.6 / 20.1, 1536 (24) 23.2 / 22.7, 2048 28.1 / 25.6.
//   more: 4 experts x 64 rows (512 tasks of 32) 53 / 71, 2 x 64 rows bf16 29 / 34, 4 x 4 rows (896)
//   28 / 40.  One expert of more than 64 rows, in runs of 64, would lose: E4M3, 100 rows
//   53 / 71, 200 rows 53 / 66, 500 rows 53 / 67.
constexpr int kFewTasks = 32, kFewTasksOfFewRows = 64, kStepsOfTwoRounds = 3 * kWaves;

// Channel tiles whose tasks stand next to each other, so that the tasks an XCD has at hand
// share rows as well as channels (65521 x 4096 -> 2048: 4 / 8 / 16 tiles 879 / 859 / 859 us).
constexpr int kBand = 8;

// (row block, channel tile) of place `local` in bands of kBand channel tiles.
__device__ __forceinline__ void in_bands(unsigned local, unsigned nb, unsigned nt, unsigned& rb,
                                         unsigned& mt) {
    const unsigned band = local / (nb * kBand), rest = local - band * nb * kBand;
    const unsigned width = min((unsigned)kBand, nt - band * kBand);
    rb = rest / width;
    mt = band * kBand + rest - rb * width;
}

// Tasks of a list, which a workgroup takes from `first` on, every stride-th below
// `end`, in pieces of a block's rows if the list's blocks are larger than its own.
struct Share {
    int list, first, end, stride, pieces;
};

template <Product OP, int RT>
__device__ __forceinline__ bool find_task(Task& t, const ProductArgs& p, const Blocks& known,
                                          const Share& s, int task, unsigned nt, int tile) {
    if (task >= s.end) return false;
    const int piece = (unsigned)task % (unsigned)s.pieces * (RT * 32);
    task = (unsigned)task / (unsigned)s.pieces;
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
        t.r0 = __builtin_amdgcn_readfirstlane(rb * 256 + piece);
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
            upto = known.upto[s.list][e0 + lane];
        } else {
            int64_t b = 0, m = 0;
            if (e0 + lane < p.runs.E) m = p.runs.of(e0 + lane, b);
            first = (int)b;
            rows = m > 0 ? (int)m : 0;
            upto = prefix_sum(row_blocks(s.list, rows)) + before;
        }
        const uint64_t hit = __ballot(upto * (int)nt > task);
        if (hit) {
            const int at = __builtin_ctzll(hit);
            t.e = e0 + at;
            t.n = __builtin_amdgcn_readlane(rows, at);
            t.begin = __builtin_amdgcn_readlane(first, at);
            const unsigned nb = row_blocks(s.list, t.n);
            const int local = task - (__builtin_amdgcn_readlane(upto, at) - (int)nb) * (int)nt;
            in_bands(local, nb, nt, rb, mt);
            t.r0 = (s.list == 0 ? rb * 256 : t.n & ~255) + piece;
            t.m0 = mt * tile;
            t.r0 = __builtin_amdgcn_readfirstlane(t.r0);
            t.m0 = __builtin_amdgcn_readfirstlane(t.m0);
            return true;
        }
        before = __builtin_amdgcn_readlane(upto, 63);
    }
    return false;
}

constexpr int kRing = 4;    // tasks that a wave's fetching is ahead of its sums, at most

struct ProductLds {
    uint8_t stage[kStageBytes];
    Blocks known;
    int ring[2][kRing][8];
};
// The ring of scales lies behind the places of class 8, or after the rest: 4 KiB a
// place for 256 rows, 2 KiB for 128.
constexpr int kScaleBytes = kScalePlaces * 128 * kScaleSteps * 4;
template <bool FP8>
struct ProductMemory {
    ProductLds lds;
    float scales[FP8 ? kScaleBytes / 4 : 1];
};
static_assert(sizeof(ProductMemory<true>) <= 160 * 1024, "one workgroup's LDS");

// A value that the compiler recomputes from where it is needed rather than hold
// in registers all along.
__device__ __forceinline__ uint32_t opaque(uint32_t v) {
    asm volatile("" : "+v"(v));
    return v;
}

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
__device__ __forceinline__ void run_tasks(const ProductArgs& p, ProductMemory<FP8>& mem,
                                          const Share& share, unsigned nt) {
    ProductLds& lds = mem.lds;
    constexpr int kTile = SWIGLU ? kTileM / 2 : kTileM;    // result channels
    constexpr bool kAT = OP != kRows;                      // a and b by columns
    constexpr bool kBT = OP == kGradWeight;
    constexpr int kElem = FP8 ? 1 : 2;
    constexpr int kStepK = kStepBytes / kElem;
    constexpr int kPart = kParts<RT>, kStage = kStages<RT>;
    constexpr int HT = RT / kPart;                         // row tiles of a part
    constexpr int kBStage = HT * 4096;                     // bytes of a part
    constexpr int kScalePlace = 2 * RT * 16 * kScaleSteps * 4;
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int group = wave >> 2, w4 = wave & 3;
    const int lg = lane >> 4, lr = lane & 15;
    const uint8_t* const stage_a = lds.stage;
    const uint8_t* const stage_b = lds.stage + kStage * kABytes;
    const uint8_t* const stage_s =
        RT == 8 ? lds.stage + kStage * (kABytes + kPart * kBStage)
                : reinterpret_cast<const uint8_t*>(mem.scales);
    const uint32_t lds_a = __builtin_amdgcn_readfirstlane(lds_offset(stage_a));
    const uint32_t lds_b = __builtin_amdgcn_readfirstlane(lds_offset(stage_b));
    const uint32_t lds_s = FP8 ? __builtin_amdgcn_readfirstlane(lds_offset(stage_s)) : 0;
    const uint32_t a_row = (OP == kRows ? p.K : p.M) * kElem;     // bytes
    const uint32_t b_row = (OP == kGradWeight ? p.B : p.K) * kElem;
    const int steps_k = (p.K + kStepK - 1) / kStepK;

    // --- fetching: waves 0..3 a quarter of a's part of a step each, waves 4..7
    // of b's.  A load takes 1 KiB: 8 rows' 128 bytes, 2 steps' 256 or 4 steps' 128
    // columns.
    constexpr int kLoadsA = 8, kLoadsB = HT;      // of b: a part
    struct {
        int task, step, steps;
        uint64_t at, s;
        int left, s_left;       // bytes of the rows, or by columns steps of k
        int col;                // by columns: first byte of the row
    } next;
    int pushed = 0;                               // tasks
    int fetch_to = 0, scale_to = 0;               // places of the step that is fetched next
    auto turn_stage = [](int i) { return i + 1 == kStage ? 0 : i + 1; };
    auto seek = [&]() {
        Task t;
        const bool live = find_task<OP, RT>(t, p, lds.known, share, next.task, nt, kTile);
        next.task += share.stride;
        if (lane == 0) {
            int* q = lds.ring[group][pushed & (kRing - 1)];
            q[0] = live ? t.e : -1;
            q[1] = t.m0;
            q[2] = t.r0;
            q[3] = t.n;
            q[4] = (int)t.begin;
        }
        ++pushed;
        next.step = 0;
        next.steps = 0x7fffffff;                  // after the last task: nothing, for good
        next.left = next.s_left = 0;
        next.col = 0;
        next.at = next.s = (uint64_t)p.a;
        if (!live) return;
        next.steps = OP == kGradWeight ? max(1, (t.n + kStepK - 1) / kStepK) : steps_k;
        if (group == 0) {
            if constexpr (OP == kRows) {
                const int half = SWIGLU ? w4 >> 1 : 0;
                const int c = SWIGLU ? (w4 & 1) * 64 : w4 * 64;
                const int64_t w0 = ((int64_t)t.e * (SWIGLU ? 2 : 1) + half) * p.M + t.m0 + c;
                next.at = (uint64_t)(p.a + w0 * a_row);
                next.left = max(0, min(64, p.M - t.m0 - c)) * (int)a_row;
            } else {
                const int64_t k0 = (OP == kGradRows ? (int64_t)t.e * p.K : t.begin) + w4 * 16;
                next.col = t.m0 * kElem;
                next.at = (uint64_t)(p.a + k0 * a_row + next.col);
                next.left = (OP == kGradRows ? p.K : t.n) - w4 * 16;
            }
        } else if constexpr (kBT) {
            next.col = t.r0 * kElem;
            next.at = (uint64_t)(p.b + (t.begin + w4 * 16) * b_row + next.col);
            next.left = t.n - w4 * 16;
        } else {
            // rows of this wave's share of the first part; those of the second lie 16 HT on
            const int r = t.r0 + (w4 >> 1) * RT * 16 + (w4 & 1) * HT * 8;
            next.at = (uint64_t)(p.b + (t.begin + r) * b_row);
            next.left = (int)min((int64_t)max(0, t.n - r) * b_row, (int64_t)0x7fff0000);
            if constexpr (FP8) {
                const int s_row = p.K / 128 * 4;
                next.s = (uint64_t)p.bs + (t.begin + t.r0 + w4 * 64) * s_row;
                next.s_left = max(0, min(64, t.n - t.r0 - w4 * 64)) * s_row;
            }
        }
    };
    auto advance = [&](bool columns, uint32_t row) {
        if (++next.step == next.steps) {
            seek();
            return;
        }
        next.at += columns ? (int64_t)row * kStepK : kStepBytes;
        next.left -= columns ? kStepK : min(kStepBytes, next.left);
    };
    // The lane's places of a part's loads (a's or of a half of b's), less their kShift.
    uint32_t at[kLoadsA];
    auto chunk = [&](bool columns, int lanes, int i) {
        const uint32_t l = lane;
        if (columns) {
            // 16 places of 32 bytes (256 columns) or 8 for a step of k
            const uint32_t pos = l & ((1u << lanes) - 1), k = (l >> lanes) + i * (64 >> lanes);
            return (((pos >> 1) ^ column_turn(k)) << 5) | (pos & 1) << 4;
        }
        return ((l & 7) ^ ((i * 8 + (l >> 3)) >> 1 & 7)) << 4;
    };
#pragma unroll
    for (int i = 0; i < kLoadsA; ++i) {
        const int shift = kShift - i % 4 * 1024;
        if (group == 0) {
            if constexpr (kAT)
                at[i] = ((lane >> 5) + i * 2) * a_row + chunk(true, 5, i) + shift;
            else
                at[i] = ((lane >> 3) + i * 8) * a_row + chunk(false, 0, i) + shift;
        } else if constexpr (kBT) {
            // 128 of 256 columns: the second wave row's lie 128 columns on
            const uint32_t c = chunk(true, 4, i);
            at[i] = ((lane >> 4) + i * 4) * b_row + c + (kPart == 2 ? c & 128 : 0) + shift;
        } else {
            at[i] = ((lane >> 3) + i * 8) * b_row + chunk(false, 0, i) + shift;
        }
    }
    // Of the last step by rows, what lies past the rows' end.
    auto cut = [&](uint32_t (&v)[kLoadsA]) {
        const int over = p.K * kElem - next.step * kStepBytes;
        const uint32_t l = opaque(lane);
#pragma unroll
        for (int i = 0; i < kLoadsA; ++i) {
            const uint32_t c = ((l & 7) ^ ((i * 8 + (l >> 3)) >> 1 & 7)) << 4;
            v[i] = (int)c < over ? at[i] : kNowhere;
        }
    };
    const bool ragged = !kBT && (p.K * kElem) % kStepBytes != 0;
    auto issue_a = [&]() {
        const i32x4 buffer = make_buffer(
            next.at, kAT ? max(0, min(16, next.left)) * (int)a_row - next.col : next.left);
        const uint32_t to = lds_a + fetch_to * kABytes + w4 * kLoadsA * 1024;
        if (!kAT && ragged && next.step == steps_k - 1) {
            uint32_t v[kLoadsA];
            cut(v);
            dma16<4>(v, buffer, to);
            dma16<4>(v + 4, buffer, to + 4096);
        } else {
            dma16<4>(at, buffer, to);
            dma16<4>(at + 4, buffer, to + 4096);
        }
        fetch_to = turn_stage(fetch_to);
        advance(kAT, a_row);
    };
    auto issue_b = [&](int part) {
        if constexpr (FP8) {
            // ahead of the step's rows, so that these are waited for after them
            if (part == 0 && next.step % kScaleSteps == 0) {
                if (w4 < (2 * RT * 16 + 63) / 64) {
                    const uint32_t v = (uint32_t)(lane * (p.K / 128) * 4) + kShift;
                    dma16<1>(&v, make_buffer(next.s, next.s_left),
                             lds_s + scale_to * kScalePlace + w4 * 1024);
                }
                scale_to = (scale_to + 1) % kScalePlaces;
                next.s += kScaleSteps * 4;
                next.s_left -= kScaleSteps * 4;
            }
        }
        const int more = kBT ? part * 128 : part * HT * 16 * (int)b_row;
        const i32x4 buffer = make_buffer(
            next.at + more,
            kBT ? max(0, min(16, next.left)) * (int)b_row - next.col - more : next.left - more);
        const uint32_t to = lds_b + (fetch_to * kPart + part) * kBStage + w4 * kLoadsB * 1024;
        if (ragged && next.step == steps_k - 1) {
            uint32_t v[kLoadsA];
            cut(v);
            dma16<kLoadsB>(v, buffer, to);
        } else {
            dma16<kLoadsB>(at, buffer, to);
        }
        if (part == kPart - 1) {
            fetch_to = turn_stage(fetch_to);
            advance(kBT, b_row);
        }
    };
    // loads that may be on their way while an older part has to be there (scales not
    // counted: they come every few steps)
    constexpr int kAheadA = kLoadsA, kAheadB = kPart * kLoadsB;

    // --- this wave's results: 64 channels (4 tiles) by RT tiles of rows ---
    const int wm = w4, wr = group;
    f32x4 acc[4][RT];
    i32x4 af[4][2], bf[HT][2];
    float sx[FP8 ? HT : 1];
    // 16 columns of 32 steps of k: lane (lg, lr) holds steps 8 lg .. 8 lg + 7 of
    // column lr
    auto by_columns = [&](const uint8_t* s, int row, uint32_t at, int tile, int ks) {
        typedef __attribute__((address_space(3))) s16x4 L;
        const uint8_t* q = s + (at ^ tile << 5) + ks * 32 * row;
        const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((L*)q);
        const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((L*)(q + 4 * row));
        const uint64_t l = __builtin_bit_cast(uint64_t, lo), h = __builtin_bit_cast(uint64_t, hi);
        return i32x4{(int)(uint32_t)l, (int)(uint32_t)(l >> 32), (int)(uint32_t)h,
                     (int)(uint32_t)(h >> 32)};
    };
    auto lane_columns = [&](int row) {
        const uint32_t l = lane, k = (l >> 4) * 8 + (l >> 2 & 3);
        return k * row + (column_turn(k) << 5) + ((l & 3) << 3);
    };
    auto lane_rows = [&]() {
        return row_place(lr, lg);
    };
    auto read_a = [&](int buf) {
        const uint8_t* s = stage_a + buf * kABytes;
        if constexpr (kAT) {
            const uint32_t at = lane_columns(512);
#pragma unroll
            for (int ct = 0; ct < 4; ++ct)
#pragma unroll
                for (int ks = 0; ks < 2; ++ks)
                    af[ct][ks] = by_columns(s, 512, at, wm * 4 + ct, ks);
        } else {
            const uint32_t at = lane_rows();
            s += (SWIGLU ? wm * 32 : wm * 64) * kStepBytes;
#pragma unroll
            for (int ct = 0; ct < 4; ++ct)
#pragma unroll
                for (int ks = 0; ks < 2; ++ks)
                    af[ct][ks] = *reinterpret_cast<const i32x4*>(
                        s + (at ^ ks * 64) +
                        (SWIGLU ? (ct >> 1) * 128 + (ct & 1) * 16 : ct * 16) * kStepBytes);
        }
    };
    auto read_b = [&](int buf, int part, int scales, int step) {
        const uint8_t* s = stage_b + (buf * kPart + part) * kBStage;
        const uint32_t at = kBT ? lane_columns(256) : lane_rows();
#pragma unroll
        for (int rt = 0; rt < HT; ++rt)
#pragma unroll
            for (int ks = 0; ks < 2; ++ks) {
                if constexpr (kBT)
                    bf[rt][ks] = by_columns(s, 256, at, wr * HT + rt, ks);
                else
                    bf[rt][ks] = *reinterpret_cast<const i32x4*>(
                        s + (at ^ ks * 64) + (wr * HT + rt) * 16 * kStepBytes);
            }
        if constexpr (FP8) {
#pragma unroll
            for (int rt = 0; rt < HT; ++rt)
                sx[rt] = *reinterpret_cast<const float*>(
                    stage_s + scales * kScalePlace +
                    (((wr * RT + part * HT + rt) * 16 + lr) * kScaleSteps + step % kScaleSteps) *
                        4);
        }
    };
    auto multiply = [&](auto part_, float s0, float s1) {
        constexpr int r0 = decltype(part_)::value * HT;
        if constexpr (FP8) {
            const f32x4 zero = {0.0f, 0.0f, 0.0f, 0.0f};
            // a tile's 128 channels are scaled into its sums while the next tiles are
            // multiplied
            constexpr int kLate = 2;
            f32x4 part[kLate + 1];
            float g[HT], u[HT];
#pragma unroll
            for (int rt = 0; rt < HT; ++rt) {
                g[rt] = sx[rt] * s0;
                u[rt] = SWIGLU ? sx[rt] * s1 : g[rt];
            }
#pragma unroll
            for (int i = 0; i < 4 * HT + kLate; ++i) {
                if (i < 4 * HT) {
                    const int rt = i / 4, ct = i % 4;
                    i32x8 a, b;
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        a[j] = af[ct][j / 4][j % 4];
                        b[j] = bf[rt][j / 4][j % 4];
                    }
                    part[i % (kLate + 1)] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                        a, b, zero, 0, 0, 0, 127, 0, 127);
                }
                __builtin_amdgcn_sched_barrier(0);
                if (i >= kLate) {
                    const int rt = (i - kLate) / 4, ct = (i - kLate) % 4;
                    const f32x4 t = part[(i - kLate) % (kLate + 1)];
                    const float sc = SWIGLU && ct >= 2 ? u[rt] : g[rt];
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        acc[ct][r0 + rt][j] = __builtin_fmaf(t[j], sc, acc[ct][r0 + rt][j]);
                }
                __builtin_amdgcn_sched_barrier(0);
            }
        } else {
#pragma unroll
            for (int ks = 0; ks < 2; ++ks)
#pragma unroll
                for (int rt = 0; rt < HT; ++rt)
#pragma unroll
                    for (int ct = 0; ct < 4; ++ct)
                        acc[ct][r0 + rt] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                            __builtin_bit_cast(bf16x8, af[ct][ks]),
                            __builtin_bit_cast(bf16x8, bf[rt][ks]), acc[ct][r0 + rt], 0, 0, 0);
        }
        // done here, not where the sums are next used
#pragma unroll
        for (int rt = 0; rt < HT; ++rt)
#pragma unroll
            for (int ct = 0; ct < 4; ++ct) asm volatile("" : "+v"(acc[ct][r0 + rt]));
    };
    // The largest tiles' results go through LDS, 2 KiB a wave behind the places: 16
    // rows by 128 bytes, of which eight neighbouring lanes then store a whole line
    // (stored as they stand, 8 bytes a lane: 1024 x 1024 weights' gradient 42 us, 34
    // with whole lines; 65521 x 2048 -> 4096 rows' gradient 953, 908).
    constexpr bool kLines = !FP8 && !SWIGLU && RT == 8;
    static_assert(!kLines || kStage * (kABytes + kPart * kBStage) + kWaves * 2048 <= kStageBytes);
    auto store = [&](const Task& t) {
        const int rows = OP == kGradWeight ? p.B : t.n;
        if constexpr (kLines) {
            constexpr int kOut = F32 ? 4 : 2;           // bytes
            constexpr int kTiles = F32 ? 2 : 4;         // 16-channel tiles of a line
            uint8_t* s = lds.stage + kStage * (kABytes + kPart * kBStage) + wave * 2048;
            const uint32_t turn = (lr >> 1 & 7) << 4;
            const uint32_t to = lr * 128 + (F32 ? lg * 16 : lg * 8);
            const int line = lane >> 3;
            const uint32_t from = line * 128 + (((lane & 7) ^ (line >> 1)) << 4);
#pragma unroll
            for (int i = 0; i < RT * 4 / kTiles; ++i) {
                const int rt = i * kTiles / 4, c0 = i * kTiles % 4;
#pragma unroll
                for (int j = 0; j < kTiles; ++j) {
                    const f32x4 v = acc[c0 + j][rt];
                    uint8_t* q = s + ((to + j * 16 * kOut) ^ turn);
                    if constexpr (F32)
                        *reinterpret_cast<f32x4*>(q) = v;
                    else
                        *reinterpret_cast<uint2*>(q) =
                            make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
                }
                const int c = t.m0 + wm * 64 + c0 * 16 + (lane & 7) * (16 / kOut);
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    f32x4 v = *reinterpret_cast<const f32x4*>(s + (from ^ h * 64) + h * 1024);
                    const int r = t.r0 + (wr * RT + rt) * 16 + h * 8 + line;
                    if (r >= rows || c >= p.M) continue;
                    const int64_t row = OP == kGradWeight ? (int64_t)t.e * p.B + r : t.begin + r;
                    f32x4* o = reinterpret_cast<f32x4*>(static_cast<uint8_t*>(p.y) +
                                                        (row * p.M + c) * kOut);
                    if constexpr (ADD) v += *o;
                    *o = v;
                }
            }
            return;
        }
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
                    for (int i = 0; i < 4; ++i) v[i] = silu_times(v[i], u[i]);
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
    // multiplies, the other reads its next operands.  Phases of step t, two for each
    // part of b, the second half's one later: read a and b's first part, multiply
    // (read b's second part, multiply).  What lay in a place is asked for anew once
    // all waves have read it.  In two parts:
    //   a(t + 2)           in the first half's phase 3 of t,  needed six phases later;
    //   b's first (t + 2)  in the second half's phase 3 of t, needed five later;
    //   b's second (t + 1) in the second half's phase 1 of t, needed five later;
    // in one part, whose phases are as long:
    //   a(t + 2) and b(t + 2) in the halves' phase 1 of t, needed four and three later.
    // A wait that the compiler counts.  Loads of its own that it holds for under way here
    // (the narrow form's last ones, which nothing uses) it would wait for inside the steps,
    // and so for the loads to LDS: as the code around it falls, for those of the step before
    // or for those just asked for (8 experts x 100 rows, 7168 -> 2 x 2048, E4M3: 67 and 90 us,
    // 66 with this).
    __builtin_amdgcn_s_waitcnt(0x0f70);            // vmcnt(0)
    next.task = share.first;
    seek();
    if (group == 0) {
        issue_a();
        issue_a();
        wait_dma<kAheadA>();
    } else {
        issue_b(0);
        if (kPart == 2) issue_b(1);
        issue_b(0);
        wait_dma<kAheadB>();
    }
    EP_WAIT_LDS();
    barrier();
    if (group == 1) barrier();
    int place = 0, scales = kScalePlaces - 1;     // of the step at hand
#pragma unroll 1
    for (int taken = 0;; ++taken) {
        const int* q = lds.ring[group][taken & (kRing - 1)];
        Task t;
        t.e = __builtin_amdgcn_readfirstlane(q[0]);
        if (t.e < 0) break;
        t.m0 = __builtin_amdgcn_readfirstlane(q[1]);
        t.r0 = __builtin_amdgcn_readfirstlane(q[2]);
        t.n = __builtin_amdgcn_readfirstlane(q[3]);
        t.begin = __builtin_amdgcn_readfirstlane(q[4]);
        const int steps = OP == kGradWeight ? max(1, (t.n + kStepK - 1) / kStepK) : steps_k;
        typedef const __attribute__((address_space(4))) float* Scalars;
        Scalars as0 = nullptr, as1 = nullptr;
        if constexpr (FP8) {
            const int KB = p.K / 128, NB = (p.M + 127) / 128;
            const int c = t.m0 + (SWIGLU ? wm * 32 : wm * 64);
            as0 = (Scalars)(uint64_t)(p.as + ((int64_t)t.e * (SWIGLU ? 2 : 1) * NB +
                                              min(c / 128, NB - 1)) * KB);
            as1 = as0 + (int64_t)NB * KB;
        }
#pragma unroll
        for (int ct = 0; ct < 4; ++ct)
#pragma unroll
            for (int rt = 0; rt < RT; ++rt) acc[ct][rt] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        float s0 = FP8 ? as0[0] : 0.0f, s1 = FP8 && SWIGLU ? as1[0] : 0.0f;
#pragma unroll 1
        for (int step = 0; step < steps; ++step, place = turn_stage(place)) {
            if (FP8 && step % kScaleSteps == 0) scales = (scales + 1) % kScalePlaces;
            read_a(place);
            read_b(place, 0, scales, step);
            if (group == 1) {
                issue_b(kPart == 2 ? 1 : 0);
                wait_dma<kAheadB>();
            } else if (kPart == 1) {
                issue_a();
            }
            EP_WAIT_LDS();
            barrier();
            const float g = s0, u = s1;
            if (FP8) {      // the next step's (of the last one: that again)
                s0 = as0[min(step + 1, steps - 1)];
                if (SWIGLU) s1 = as1[min(step + 1, steps - 1)];
            }
            multiply(std::integral_constant<int, 0>{}, g, u);
            if constexpr (kPart == 2) {
                barrier();
                read_b(place, 1, scales, step);
                if (group == 0) {
                    issue_a();
                } else {
                    issue_b(0);
                    wait_dma<kAheadB>();
                }
                EP_WAIT_LDS();
                barrier();
                multiply(std::integral_constant<int, 1>{}, g, u);
            }
            if (group == 0) wait_dma<kAheadA>();
            barrier();
        }
        if (OP == kGradWeight && ADD && t.n == 0) continue;
        store(t);
    }
    if (group == 0) barrier();
    wait_dma<0>();
    barrier();
}

// Few tasks of few rows (at most 64 an expert): tiles of 32 channels, whose steps
// the eight waves share, so that eight times as many workgroups read weights.  Wave w
// takes steps w, w + 8, ... from global memory straight into operands, DEPTH of its
// steps ahead (of few rows all of them, where the channels summed are few thousand),
// and the waves' sums meet in LDS, in wave order.
template <bool FP8, bool SWIGLU, int RT>
__device__ __forceinline__ void run_narrow(const ProductArgs& p, ProductMemory<FP8>& mem,
                                           const Task& t) {
    constexpr int kElem = FP8 ? 1 : 2;
    constexpr int CT = 2, DEPTH = RT == 1 ? 7 : RT == 2 ? 5 : 3;
    const int lane = threadIdx.x & 63, lg = lane >> 4, lr = lane & 15;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const uint32_t row = p.K * kElem;
    const int steps = (int)((row + kStepBytes - 1) / kStepBytes);
    const int KB = p.K / 128, NB = (p.M + 127) / 128;

    // a: 16-channel tiles, with SWIGLU one of either half; b: 16-row tiles
    __amdgpu_buffer_rsrc_t ab[SWIGLU ? 2 : 1];
    constexpr int kTile = CT * 16 / (SWIGLU ? 2 : 1);
#pragma unroll
    for (int h = 0; h < (SWIGLU ? 2 : 1); ++h) {
        const int64_t w0 = ((int64_t)t.e * (SWIGLU ? 2 : 1) + h) * p.M + t.m0;
        ab[h] = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(p.a + w0 * row), 0,
                                                  min(kTile, p.M - t.m0) * (int)row, 0x00020000);
    }
    const __amdgpu_buffer_rsrc_t bb = __builtin_amdgcn_make_buffer_rsrc(
        const_cast<uint8_t*>(p.b + t.begin * row), 0, min(RT * 16, t.n) * (int)row, 0x00020000);
    const __amdgpu_buffer_rsrc_t sb = __builtin_amdgcn_make_buffer_rsrc(
        const_cast<float*>(FP8 ? p.bs + t.begin * KB : nullptr), 0,
        FP8 ? min(RT * 16, t.n) * KB * 4 : 0, 0x00020000);
    typedef const __attribute__((address_space(4))) float* Scalars;
    Scalars as0 = nullptr, as1 = nullptr;
    if constexpr (FP8) {
        as0 = (Scalars)(uint64_t)(p.as + ((int64_t)t.e * (SWIGLU ? 2 : 1) * NB + t.m0 / 128) * KB);
        as1 = as0 + (int64_t)NB * KB;
    }
    struct Step {
        i32x4 a[CT][2], b[RT][2];
        float sx[RT], s0, s1;
    };
    auto load = [&](Step& q, int step) {
        // past the last step: nothing, which arrives as zeros
        const uint32_t at = step * kStepBytes;
#pragma unroll
        for (int ks = 0; ks < 2; ++ks) {
            const uint32_t c = at + (ks * 4 + lg) * 16;
            const uint32_t v = c < row ? lr * row + c : kNowhere;
#pragma unroll
            for (int ct = 0; ct < CT; ++ct)
                q.a[ct][ks] = __builtin_bit_cast(
                    i32x4, __builtin_amdgcn_raw_buffer_load_b128(
                               ab[SWIGLU ? ct : 0],
                               v == kNowhere || SWIGLU ? v : v + ct * 16 * row, 0, 0));
#pragma unroll
            for (int rt = 0; rt < RT; ++rt)
                q.b[rt][ks] = __builtin_bit_cast(
                    i32x4, __builtin_amdgcn_raw_buffer_load_b128(
                               bb, v == kNowhere ? v : v + rt * 16 * row, 0, 0));
        }
        if constexpr (FP8) {
#pragma unroll
            for (int rt = 0; rt < RT; ++rt)
                q.sx[rt] = __builtin_bit_cast(
                    float, __builtin_amdgcn_raw_buffer_load_b32(
                               sb, ((rt * 16 + lr) * KB + min(step, KB - 1)) * 4, 0, 0));
            q.s0 = as0[min(step, KB - 1)];
            q.s1 = SWIGLU ? as1[min(step, KB - 1)] : q.s0;
        }
    };
    f32x4 acc[CT][RT];
#pragma unroll
    for (int ct = 0; ct < CT; ++ct)
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) acc[ct][rt] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    auto use = [&](const Step& q) {
#pragma unroll
        for (int rt = 0; rt < RT; ++rt)
#pragma unroll
            for (int ct = 0; ct < CT; ++ct) {
                if constexpr (FP8) {
                    const f32x4 zero = {0.0f, 0.0f, 0.0f, 0.0f};
                    i32x8 a, b;
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        a[j] = q.a[ct][j / 4][j % 4];
                        b[j] = q.b[rt][j / 4][j % 4];
                    }
                    const f32x4 v = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                        a, b, zero, 0, 0, 0, 127, 0, 127);
                    const float sc = q.sx[rt] * (SWIGLU && ct >= 1 ? q.s1 : q.s0);
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        acc[ct][rt][j] = __builtin_fmaf(v[j], sc, acc[ct][rt][j]);
                } else {
#pragma unroll
                    for (int ks = 0; ks < 2; ++ks)
                        acc[ct][rt] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                            __builtin_bit_cast(bf16x8, q.a[ct][ks]),
                            __builtin_bit_cast(bf16x8, q.b[rt][ks]), acc[ct][rt], 0, 0, 0);
                }
            }
    };
    Step q[DEPTH];
#pragma unroll
    for (int i = 0; i < DEPTH; ++i) load(q[i], wave + i * kWaves);
#pragma unroll 1
    for (int step = wave; step < steps; step += DEPTH * kWaves)
#pragma unroll
        for (int i = 0; i < DEPTH; ++i) {
            use(q[i]);           // (past the last step: zeros)
            load(q[i], step + (i + DEPTH) * kWaves);
        }

    f32x4* part = reinterpret_cast<f32x4*>(mem.lds.stage);
    constexpr int kTiles = CT * RT;
    static_assert(kWaves * kTiles * 64 * sizeof(f32x4) <= kStageBytes, "the waves' sums");
    __syncthreads();             // the sums of the task before are done with
#pragma unroll
    for (int ct = 0; ct < CT; ++ct)
#pragma unroll
        for (int rt = 0; rt < RT; ++rt)
            part[(wave * kTiles + ct * RT + rt) * 64 + lane] = acc[ct][rt];
    __syncthreads();
    for (int o = wave; o < (SWIGLU ? kTiles / 2 : kTiles); o += kWaves) {
        const int ct = o / RT, rt = o % RT;
        f32x4 v = {0.0f, 0.0f, 0.0f, 0.0f}, u = v;
        for (int i = 0; i < kWaves; ++i) {
            v += part[(i * kTiles + o) * 64 + lane];
            if constexpr (SWIGLU) u += part[(i * kTiles + kTiles / 2 + o) * 64 + lane];
        }
        if constexpr (SWIGLU) {
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = silu_times(v[i], u[i]);
        }
        const int r = rt * 16 + lr, c = t.m0 + ct * 16 + lg * 4;
        if (r < t.n && c < p.M)
            *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.y) + (t.begin + r) * p.M + c) =
                make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
    }
}

// All tasks of a product.  Every XCD (workgroups i, i + 8, ...) takes one run of each
// list's tasks, so that its workgroups share rows and weights; a workgroup's `slot` among
// them moves on, so that those that have had no task of a round come first in the next.
template <Product OP, bool FP8, bool SWIGLU, bool F32, bool ADD>
__device__ __forceinline__ void run_product(const ProductArgs& p, ProductMemory<FP8>& mem,
                                            int& slot) {
    ProductLds& lds = mem.lds;
    const int lane = threadIdx.x & 63;
    constexpr int kTile = SWIGLU ? kTileM / 2 : kTileM;
    const unsigned nt = (p.M + kTile - 1) / kTile;
    const int stride = gridDim.x / kXcds, xcd = blockIdx.x % kXcds;
    // This XCD's part of a list, [begin, begin + count).
    auto part_of = [&](int64_t blocks, int& begin) {
        const int tasks = (int)(blocks * nt), per = (tasks + kXcds - 1) / kXcds;
        begin = xcd * per;
        return max(0, min(per, tasks - begin));
    };
    // Takes `count` of a list's tasks from `begin` on up, in pieces.
    auto run = [&](auto rt, int list, int begin, int count, int pieces) {
        if (count == 0) return;
        run_tasks<OP, FP8, SWIGLU, F32, ADD, decltype(rt)::value>(
            p, mem,
            Share{list, begin * pieces + slot, (begin + count) * pieces, stride, pieces}, nt);
        slot = (slot + stride - count * pieces % stride) % stride;
    };
    using Rows256 = std::integral_constant<int, 8>;
    using Rows128 = std::integral_constant<int, 4>;
    using Rows64 = std::integral_constant<int, 2>;
    int begin[3] = {0, 0, 0}, count[3] = {0, 0, 0};
    if constexpr (OP == kGradWeight) {
        count[0] = part_of((int64_t)p.runs.E * ((p.B + 255) / 256), begin[0]);
    } else {
        // Row blocks of the lists; every wave writes the same numbers, and reads its
        // own.
        int64_t sum[3] = {0, 0, 0};
        bool few = true;                         // no expert has more than 32 rows
#pragma unroll 1
        for (int e0 = 0; e0 < p.runs.E; e0 += 64) {
            int64_t b = 0, m = 0;
            if (e0 + lane < p.runs.E) m = p.runs.of(e0 + lane, b);
            const int rows = m > 0 ? (int)m : 0;
            few = few && __ballot(rows > 32) == 0;
            if (e0 < kKnown) {
                lds.known.first[e0 + lane] = (int)b;
                lds.known.rows[e0 + lane] = rows;
            }
#pragma unroll
            for (int c = 0; c < 3; ++c) {
                const int upto = prefix_sum(row_blocks(c, rows));
                if (e0 < kKnown) lds.known.upto[c][e0 + lane] = (int)(sum[c] + upto);
                sum[c] += __builtin_amdgcn_readlane(upto, 63);
            }
        }
        // (a y of 2^28 tasks fits no memory: such counts do not belong to these rows)
        if ((sum[0] + sum[1] + sum[2]) * nt >= 1 << 28) return;
        if constexpr (OP == kRows) {
            few = few && p.K * (FP8 ? 1 : 2) > (kStepsOfTwoRounds - 1) * kStepBytes;
            if (sum[0] + sum[1] == 0 && sum[2] * nt <= (few ? kFewTasksOfFewRows : kFewTasks)) {
                constexpr int kNarrow = SWIGLU ? 16 : 32;
                const unsigned tiles = (p.M + kNarrow - 1) / kNarrow;
                const Share all = {2, 0, (int)sum[2] * (int)tiles, 0, 1};
                Task t;
                // neighbouring tiles on neighbouring workgroups: they share the rows
#pragma unroll 1
                for (int i = blockIdx.x; find_task<OP, 2>(t, p, lds.known, all, i, tiles, kNarrow);
                     i += gridDim.x) {
                    if (t.n <= 16)
                        run_narrow<FP8, SWIGLU, 1>(p, mem, t);
                    else if (t.n <= 32)
                        run_narrow<FP8, SWIGLU, 2>(p, mem, t);
                    else
                        run_narrow<FP8, SWIGLU, 4>(p, mem, t);
                }
                return;
            }
        }
#pragma unroll
        for (int c = 0; c < 3; ++c) count[c] = part_of(sum[c], begin[c]);
    }
    // Whole rounds of the largest blocks; what is left of them in pieces, if the
    // workgroups suffice for one more round of those and of the smaller blocks.
    const int whole = count[0] / stride * stride, rest = count[0] - whole;
    const int small = count[1] + count[2];
    int pieces = 1;
    if (rest * 2 + small <= stride) pieces = 2;
    if (OP != kGradWeight && rest * 4 + small <= stride) pieces = 4;
    const bool halve = pieces == 4 && rest * 4 + count[1] * 2 + count[2] <= stride;
    run(Rows256{}, 0, begin[0], pieces == 1 ? count[0] : whole, 1);
#pragma unroll 1
    for (int i = 0; i < (OP == kGradWeight ? 1 : 2); ++i) {
        const int n = i == 0 ? (pieces == 2 ? rest : 0) : halve ? 0 : count[1];
        run(Rows128{}, i, begin[i] + (i == 0 ? whole : 0), n, 2 >> i);
    }
    if constexpr (OP != kGradWeight) {
#pragma unroll 1
        for (int i = 0; i < 3; ++i) {
            const int n = i == 0 ? (pieces == 4 ? rest : 0) : i == 1 ? (halve ? count[1] : 0) : count[2];
            run(Rows64{}, i, begin[i] + (i == 0 ? whole : 0), n, 4 >> i);
        }
    }
}

template <Product OP, bool FP8, bool SWIGLU, bool F32, bool ADD>
__global__ __launch_bounds__(kWaves * 64, 2) void product_kernel(const ProductArgs p) {
    __shared__ __attribute__((aligned(1024))) ProductMemory<FP8> mem;
    int slot = blockIdx.x / kXcds;
    run_product<OP, FP8, SWIGLU, F32, ADD>(p, mem, slot);
}

// Both gradients in one launch: the weights' tasks start on the workgroups that the last
// round of the rows' leaves idle (6001 rows of 40 experts, 1032 -> 1000: 83 us as two
// launches, 77 as one).
template <bool F32, bool ADD>
__global__ __launch_bounds__(kWaves * 64, 2) void gradients_kernel(const ProductArgs rows,
                                                                   const ProductArgs weight) {
    __shared__ __attribute__((aligned(1024))) ProductMemory<false> mem;
    int slot = blockIdx.x / kXcds;
    run_product<kGradRows, false, false, false, false>(rows, mem, slot);
    run_product<kGradWeight, false, false, F32, ADD>(weight, mem, slot);
}

// Workgroups for so many tasks: eight a task, which the narrow form's tiles of 32 channels
// take, and at least four an XCD, for the pieces of its only task (256 rows, 4096 -> 256,
// bf16: 78 us with one an XCD, 49 with four; E4M3 59 / 32).
dim3 workgroups(int64_t tasks) {
    const int64_t want = tasks * 8 < 4 * kXcds ? 4 * kXcds : tasks * 8 < kCus ? tasks * 8 : kCus;
    return dim3((unsigned)(want + kXcds - 1) / kXcds * kXcds);
}

template <Product OP, bool FP8, bool SWIGLU, bool F32, bool ADD>
hipError_t launch(const ProductArgs& p, int64_t tasks, hipStream_t s) {
    hipLaunchKernelGGL((product_kernel<OP, FP8, SWIGLU, F32, ADD>), workgroups(tasks),
                       dim3(kWaves * 64), 0, s, p);
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

hipError_t launch_expert_gradients(const uint16_t* gy, const uint16_t* x, const RowRuns& runs,
                                   int I, int N, const uint16_t* w, uint16_t* gx, void* gw,
                                   bool fp32, bool accumulate, hipStream_t s) {
    const uint8_t* g = reinterpret_cast<const uint8_t*>(gy);
    const ProductArgs rows = {reinterpret_cast<const uint8_t*>(w), g, nullptr, nullptr,
                              runs, N, I, 0, gx};
    const ProductArgs weight = {reinterpret_cast<const uint8_t*>(x), g, nullptr, nullptr,
                                runs, 0, I, N, gw};
    const int64_t tiles = (I + kTileM - 1) / kTileM;
    const int64_t row_tasks = gx ? most_blocks(runs) * tiles : 0;
    const int64_t weight_tasks = gw ? (int64_t)runs.E * ((N + 255) / 256) * tiles : 0;
    if (!gw) {
        if (runs.num_rows == 0) return hipSuccess;
        return launch<kGradRows, false, false, false, false>(rows, row_tasks, s);
    }
    if (!gx || runs.num_rows == 0) {
        if (!fp32) return launch<kGradWeight, false, false, false, false>(weight, weight_tasks, s);
        return accumulate ? launch<kGradWeight, false, false, true, true>(weight, weight_tasks, s)
                          : launch<kGradWeight, false, false, true, false>(weight, weight_tasks, s);
    }
    const dim3 grid = workgroups(row_tasks + weight_tasks), block(kWaves * 64);
    if (!fp32)
        hipLaunchKernelGGL((gradients_kernel<false, false>), grid, block, 0, s, rows, weight);
    else if (accumulate)
        hipLaunchKernelGGL((gradients_kernel<true, true>), grid, block, 0, s, rows, weight);
    else
        hipLaunchKernelGGL((gradients_kernel<true, false>), grid, block, 0, s, rows, weight);
    return hipGetLastError();
}

}  // namespace ep
