// gfx950 kernels of the orthogonalised update and of the shard step that applies it.
//
//   X0 = x / (|x|_F + eps),  X' = a X + (b A + c A^2) X,  A = X X^T
//
// for each of a few (a, b, c): an odd polynomial that moves every singular value
// towards 1.  X is the wide orientation, m <= n, so the inner matrices are m x m.
// All of it is matrix products: A and A^2 are symmetric, of which only the tiles on
// and below the diagonal are computed and written twice, so a pass does
// m^2 n + m^3 + 2 m^2 n operations, or fewer with steps in groups (zsmr_newton_plan.h).
//
// Precision.  The first passes raise small singular values by a factor of several
// hundred, and a rounding of X with them: with operands of one 16-bit rounding the
// result is off by 2e-3 (fp16) or 2e-2 (bf16) of its norm.  So every matrix is held
// as the sum of two fp16 parts, x = hi + lo, together 22 bits, and a product is three
// matrix products of fp16, hi hi + lo hi + hi lo, summed in one fp32 accumulator:
// the accuracy of fp32 operands at a third of the 16-bit matrix rate, where gfx950's
// fp32 matrix instructions run at a sixteenth.  lo lo, 2^-22 of the result, is left
// out.  Powers of two known beforehand keep all parts inside fp16's range
// (zsmr_newton_plan.h).
//
// Layout.  32 columns of a row are 64 bytes of hi and 64 bytes of lo, side by side,
// so a step of 32 k is one 128-byte line a row.  A product loads both parts of a
// tile once for its three uses.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "zsmr_dev.h"
#include "zsmr_mfma.h"
#include "zsmr_newton_launch.h"
#include "zsmr_ops_launch.h"

#pragma clang fp contract(off)

namespace zsmr {
namespace {

constexpr int kThreads = kNsThreads, kWaves = kThreads / 64;

// ---------------------------------------------------------------- split fp16 --
struct Split8 {
    u16x8 hi, lo;
};
__device__ __forceinline__ Split8 split8(f32x8 f) {
    Split8 s;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        s.hi[i] = narrow16<ZSMR_FP16>(f[i]);
        s.lo[i] = narrow16<ZSMR_FP16>(f[i] - widen16<ZSMR_FP16>(s.hi[i]));
    }
    return s;
}
// Element (row, col) of a matrix whose rows are ld 16-bit values apart; col a
// multiple of 8.
__device__ __forceinline__ int64_t split_at(int64_t row, int64_t col, int64_t ld) {
    return row * ld + (col >> 5) * 64 + (col & 31);
}
__device__ __forceinline__ void store_split(uint16_t* p, int64_t at, f32x8 f) {
    const Split8 s = split8(f);
    *reinterpret_cast<u16x8*>(p + at) = s.hi;
    *reinterpret_cast<u16x8*>(p + at + 32) = s.lo;
}
__device__ __forceinline__ f32x8 load_split(const uint16_t* p, int64_t at) {
    const u16x8 hi = *reinterpret_cast<const u16x8*>(p + at), lo = *reinterpret_cast<const u16x8*>(p + at + 32);
    f32x8 f;
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = widen16<ZSMR_FP16>(hi[i]) + widen16<ZSMR_FP16>(lo[i]);
    return f;
}

// ------------------------------------------------------------------ operands --
// Both parts of R rows of an operand and 32 k of it, in LDS.
//  k along rows: R rows of 128 bytes, hi and lo; the 16-byte chunk c of row r sits
//    in slot c ^ (r & 7), so that the 8 rows a read touches at a time lie in
//    different banks.
//  OUTER, k is the row index in memory: 32 rows of R columns, 4 R bytes; the
//    32-byte unit u of row k sits in slot u ^ f(k), f = k's bits 0, 1 and 3: the
//    transposing read of a wave takes a 32-byte unit of 16 rows.
// The loads read through a buffer descriptor whose bound makes rows past the
// operand's end zero; columns are padded with zeros to whole steps.
template <int R, bool OUTER, int WAVES>
struct Operand {
    static constexpr int kBytes = R * 128;
    static constexpr int kLoads = R * 8 / (WAVES * 64);     // of each thread
    static_assert(R * 8 % (WAVES * 64) == 0, "whole loads");
    uint32_t off[kLoads];
    const char* base;
    int64_t left, step;

    __device__ __forceinline__ static int swizzle(int k) { return ((k & 3) | ((k >> 3 & 1) << 2)) << 1; }

    // at: the tile's first row of the product; k0: first k, a multiple of 32; every:
    // steps of 32 k to its next one; thread: of the WAVES
    __device__ __forceinline__ void init(const Mat& m, int64_t at, int64_t k0, int every, int thread) {
        const int64_t row_bytes = m.ld * 2;
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            const int idx = i * (WAVES * 64) + thread;
            if constexpr (OUTER) {
                const int k = idx / (R / 4), chunk = idx % (R / 4) ^ swizzle(k);
                off[i] = at * 4 + chunk * 16 < row_bytes ? (uint32_t)(k * row_bytes + chunk * 16) : 0x80000000u;
            } else {
                const int row = idx / 8, chunk = idx % 8 ^ (row & 7);
                off[i] = at + row < m.rows ? (uint32_t)(row * row_bytes + chunk * 16) : 0x80000000u;
            }
        }
        const char* p = reinterpret_cast<const char*>(m.p);
        if constexpr (OUTER) {
            base = p + k0 * row_bytes + at * 4;
            left = (m.rows - k0) * row_bytes - at * 4;
            step = every * kNsStep * row_bytes;
        } else {
            base = p + at * row_bytes + k0 * 4;
            left = (m.rows - at) * row_bytes - k0 * 4;
            step = every * kNsStep * 4;
        }
    }
    // Start the loads of one step into `to` and move on; `on` false: the same
    // instructions, which read nothing and write zeros.
    __device__ __forceinline__ void load(char* to, bool on) {
        const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64) % WAVES;
        const int bound = !on || left < 0 ? 0 : left > 0x7fffffff ? 0x7fffffff : (int)left;
        const auto rsrc = __builtin_amdgcn_make_buffer_rsrc(const_cast<char*>(base), 0, bound, 0x00027000);
#pragma unroll
        for (int i = 0; i < kLoads; ++i)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc, (lds_ptr)(to + (i * WAVES + wave) * 1024), 16, off[i], 0, 0, 0);
        base += step;
        left -= step;
    }
    // The operand registers of a lane for the 16 rows from `at` of the tile:
    // k = 8 * (lane / 16) + 0..7, of hi (part 0) or lo (1).
    __device__ __forceinline__ static u32x4 read(const char* t, int at, int part) {
        const int lane = threadIdx.x % 64;
        if constexpr (OUTER) {
            const int k = lane / 16 * 8 + lane % 16 / 4;
            const int chunk = (at / 32 * 8 + at % 32 / 8 + part * 4 + lane % 4 / 2) ^ swizzle(k);
            const char* p = t + k * (R * 4) + chunk * 16 + (lane & 1) * 8;
            const u32x2 a = read_transposed(p), b = read_transposed(p + 4 * (R * 4));
            u32x4 r;
            r[0] = a[0];
            r[1] = a[1];
            r[2] = b[0];
            r[3] = b[1];
            return r;
        } else {
            const int row = at + lane % 16;
            return read_lds16(t + row * 128 + ((part * 4 + lane / 16) ^ (row & 7)) * 16);
        }
    }
};

// ------------------------------------------------------------------- product --
// One of the products of a launch: D[p, q] = sum_k P[p, k] Q[q, k] for each matrix of
// the group; a result's row is q.
struct NsSide {
    const uint16_t *p, *q, *old, *old2;     // of the first matrix; old of the result's shape and layout
    uint16_t* dst;
    float mul, old_mul, old2_mul;
};
struct NsProduct {
    NsSide side[2];
    int32_t p_tiles, q_tiles, tiles;    // of 128 x 128, of a product and a matrix
    int32_t first_tile, quarters;   // of the launch; a workgroup takes a quarter of a tile
    int32_t count, steps;           // matrices; steps of 32 k
    int32_t split_steps;            // N_PARTIAL: of a part, which blockIdx.y counts
    float* partial;                 // tiles in quarters of 64 x 64, [part][tile][quarter][q][p]
    int64_t p_rows, p_ld, p_batch;  // rows; 16-bit values from row to row, from matrix to matrix
    int64_t q_rows, q_ld, q_batch;
    int64_t rows, cols, ld, batch;  // of the result and the old matrices
    // N_LAST
    int64_t first;                  // the group's first matrix
    int32_t tall, apply, dtype;     // dtype: of out, or of p16
    void* out;
    int64_t out_stride, out_batch;  // in the matrices' own orientation
    float* master;
    float decay, rate;
};

// Eight results, or fewer, of row r from column c on, in the matrices' own
// orientation.
__device__ __forceinline__ void put_result(const NsProduct& p, int64_t matrix, int64_t r, int64_t c, int n, f32x8 f) {
    if (n <= 0) return;
    if (!p.apply) {
        const int64_t e = matrix * p.out_batch + r * p.out_stride + c;
        if (n >= 8) {
            if (p.dtype == ZSMR_BF16) store8<ZSMR_BF16>(p.out, e, f);
            else if (p.dtype == ZSMR_FP16) store8<ZSMR_FP16>(p.out, e, f);
            else store8<ZSMR_FP32>(p.out, e, f);
        } else {
#pragma unroll
            for (int i = 0; i < 7; ++i)
                if (i < n) {
                    if (p.dtype == ZSMR_BF16) store1<ZSMR_BF16>(p.out, e + i, f[i]);
                    else if (p.dtype == ZSMR_FP16) store1<ZSMR_FP16>(p.out, e + i, f[i]);
                    else store1<ZSMR_FP32>(p.out, e + i, f[i]);
                }
        }
        return;
    }
    // master = decay * master - rate * update, every operation rounded to fp32
    const int64_t e = (matrix * (p.tall ? p.cols : p.rows) + r) * (p.tall ? p.rows : p.cols) + c;
    if (n >= 8) {
        f32x8 w = load8<ZSMR_FP32>(p.master, e);
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] = w[i] * p.decay - p.rate * f[i];
        store8<ZSMR_FP32>(p.master, e, w);
        if (p.dtype == ZSMR_BF16) store8<ZSMR_BF16>(p.out, e, w);
        else store8<ZSMR_FP16>(p.out, e, w);
    } else {
#pragma unroll
        for (int i = 0; i < 7; ++i)
            if (i < n) {
                const float w = p.master[e + i] * p.decay - p.rate * f[i];
                p.master[e + i] = w;
                if (p.dtype == ZSMR_BF16) store1<ZSMR_BF16>(p.out, e + i, w);
                else store1<ZSMR_FP16>(p.out, e + i, w);
            }
    }
}

// The largest r with r (r + 1) / 2 <= i.
__device__ __forceinline__ int triangle_row(int i) {
    int r = (int)((sqrtf(8.f * (float)i + 1.f) - 1.f) * 0.5f);
    while ((int64_t)(r + 1) * (r + 2) / 2 <= i) ++r;
    while ((int64_t)r * (r + 1) / 2 > i) --r;
    return r;
}

// A workgroup's tile of a launch, in tiles of its own size; index: in all tiles of 128
// or their quarters.
struct Unit {
    int side, matrix, tp, tq, index;
};
// Consecutive workgroups go to the eight XCDs in turn; each XCD takes a contiguous
// run of tiles, in groups of 8 rows of tiles, so that the tiles it works on at a time
// share operands in its L2.
template <bool SYMMETRIC>
__device__ __forceinline__ Unit unit_of(const NsProduct& p) {
    const int all = gridDim.x, xcd = blockIdx.x % 8, each = all / 8, rem = all % 8;
    const int at = xcd * each + min(xcd, rem) + (int)blockIdx.x / 8;
    int tile = p.first_tile + (p.quarters ? at / 4 : at);
    Unit u;
    u.index = p.quarters ? p.first_tile * 4 + at : p.first_tile + at;
    u.side = tile >= p.tiles * p.count;
    tile -= u.side * p.tiles * p.count;
    u.matrix = tile / p.tiles;
    tile -= u.matrix * p.tiles;
    constexpr int kGroup = 8;
    if constexpr (SYMMETRIC) {
        // rows tp of tiles, tq <= tp
        const int first = triangle_row(tile) / kGroup * kGroup, height = min(kGroup, p.p_tiles - first);
        tile -= first * (first + 1) / 2;
        if (tile < first * height) {
            u.tp = first + tile % height;
            u.tq = tile / height;
        } else {
            tile -= first * height;
            int column = 0;
            while (tile >= height - column) tile -= height - column++;
            u.tq = first + column;
            u.tp = u.tq + tile;
        }
    } else {
        const int band = tile / (kGroup * p.q_tiles), in_band = tile - band * kGroup * p.q_tiles;
        const int height = min(kGroup, p.p_tiles - band * kGroup);
        u.tp = band * kGroup + in_band % height;
        u.tq = in_band / height;
    }
    if (p.quarters) {
        u.tp = u.tp * 2 + (at & 1);
        u.tq = u.tq * 2 + (at >> 1 & 1);
    }
    return u;
}

// The results' other terms at eight elements: old_mul * old + old2_mul * old2.
struct OldTerms {
    u16x8 h[4];
    __device__ __forceinline__ void load(const NsSide& side, int64_t at) {
        if (side.old) {
            h[0] = *reinterpret_cast<const u16x8*>(side.old + at);
            h[1] = *reinterpret_cast<const u16x8*>(side.old + at + 32);
        }
        if (side.old2) {
            h[2] = *reinterpret_cast<const u16x8*>(side.old2 + at);
            h[3] = *reinterpret_cast<const u16x8*>(side.old2 + at + 32);
        }
    }
    __device__ __forceinline__ f32x8 added(const NsSide& side, f32x8 d) const {
        d *= side.mul;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if (side.old) d[i] = (widen16<ZSMR_FP16>(h[0][i]) + widen16<ZSMR_FP16>(h[1][i])) * side.old_mul + d[i];
            if (side.old2) d[i] = (widen16<ZSMR_FP16>(h[2][i]) + widen16<ZSMR_FP16>(h[3][i])) * side.old2_mul + d[i];
        }
        return d;
    }
};

// A tile of T x T by GROUPS of four waves, each with STAGES of LDS, which take the
// steps in turn and add up their sums in the end.  N_PARTIAL: some of the steps of an
// N_INNER product, whose sums go to memory as they are.
// Bound by the power of the matrix units where the tiles fill the CUs: X' of 4,096 x
// 14,336, wide tiles, takes 1.10 to 1.15 ms on two cards, 1.25 to 1.32 PFLOP/s of fp16 with
// the units busy in 0.77 of the cycles at 1.66 to 1.70 GHz; the inner products of 4,096 run
// at 1.17 to 1.22.  Elsewhere by one round's steps (zsmr_newton_plan.h has what each form
// takes).
constexpr int N_PARTIAL = 100;
template <int KIND, int T, int GROUPS, int STAGES>
__global__ __launch_bounds__(kThreads * GROUPS, T == 64 && STAGES == 2 ? 4 : 2) void ns_product_kernel(NsProduct p) {
#if defined(__HIP_DEVICE_COMPILE__)     // the scheduling hints have no host form
    constexpr bool kPartial = KIND == N_PARTIAL, kSymmetric = KIND == N_INNER || kPartial, kOuter = !kSymmetric;
    constexpr int WP = 2, TP = T / WP / 16, TQ = T / (kWaves / WP) / 16;
    typedef Operand<T, kOuter, kWaves> P;
    typedef Operand<T, false, kWaves> Q;
    constexpr int kStage = P::kBytes + Q::kBytes;
    // The only LDS variable: beside another one the compiler waits for every load
    // that writes LDS before each read of it.
    __shared__ __attribute__((aligned(1024))) char smem[GROUPS * STAGES * kStage];
    static_assert(STAGES * kStage >= T * T * 4, "the results leave through the same LDS");

    const Unit unit = unit_of<kSymmetric>(p);
    const NsSide& side = p.side[unit.side];
    const int matrix = unit.matrix, tp = unit.tp, tq = unit.tq;
    // quarters past the matrix or above the diagonal
    if (T == 64 && ((int64_t)tp * T >= p.cols || (int64_t)tq * T >= p.rows || (kSymmetric && tq > tp))) return;

    const int thread = threadIdx.x % kThreads, group = __builtin_amdgcn_readfirstlane(threadIdx.x / kThreads);
    const int first_step = kPartial ? blockIdx.y * p.split_steps : 0, all_steps = kPartial ? min(p.split_steps, p.steps - first_step) : p.steps;
    // steps of this group, and of all: one past the group's last multiplies zeros
    const int own_steps = (all_steps - group + GROUPS - 1) / GROUPS, steps = (all_steps + GROUPS - 1) / GROUPS;
    char* const lds = smem + group * (STAGES * kStage);
    P op;
    Q oq;
    op.init(Mat{side.p + matrix * p.p_batch, p.p_ld, p.p_rows, p.p_ld}, (int64_t)tp * T, (int64_t)(first_step + group) * kNsStep, GROUPS, thread);
    oq.init(Mat{side.q + matrix * p.q_batch, p.q_ld, p.q_rows, p.q_ld}, (int64_t)tq * T, (int64_t)(first_step + group) * kNsStep, GROUPS, thread);

    const int lane = threadIdx.x % 64, wave = thread / 64, wp = wave % WP, wq = wave / WP;
    f32x4 acc[TP][TQ];
#pragma unroll
    for (int i = 0; i < TP; ++i)
#pragma unroll
        for (int j = 0; j < TQ; ++j) acc[i][j] = 0.f;

    const int64_t p0 = (int64_t)tp * T, q0 = (int64_t)tq * T, padded = p.ld / 2;
    // where a thread has one group of eight results, what is added to them comes early
    constexpr bool kEarly = T * T / 8 == kThreads * GROUPS;
    OldTerms old;
    if (kEarly && !kPartial && q0 + (int)threadIdx.x / (T / 8) < p.rows && p0 + (int)threadIdx.x % (T / 8) * 8 < padded)
        old.load(side, matrix * p.batch + split_at(q0 + threadIdx.x / (T / 8), p0 + threadIdx.x % (T / 8) * 8, p.ld));

    // A step multiplies hi hi while it reads the lo parts, then waits for the next
    // stage and lets this one be filled again, and multiplies lo hi and hi lo while it
    // reads the next stage's hi parts into the other set of registers.
    constexpr int kReads = TP * (kOuter ? 2 : 1) + TQ, kMfma = TP * TQ, kLoads = P::kLoads + Q::kLoads;
    u32x4 ph[2][TP], qh[2][TQ], pl[TP], ql[TQ];
    auto read = [&](u32x4* a, u32x4* b, const char* stage, int part) {
#pragma unroll
        for (int j = 0; j < TQ; ++j) b[j] = Q::read(stage + P::kBytes, (wq * TQ + j) * 16, part);
#pragma unroll
        for (int i = 0; i < TP; ++i) a[i] = P::read(stage, (wp * TP + i) * 16, part);
    };
    auto multiply = [&](const u32x4* a, const u32x4* b) {
#pragma unroll
        for (int i = 0; i < TP; ++i)
#pragma unroll
            for (int j = 0; j < TQ; ++j) acc[i][j] = mfma<ZSMR_FP16>(a[i], b[j], acc[i][j]);
    };
#pragma unroll
    for (int i = 0; i < STAGES; ++i) {
        op.load(lds + i * kStage, i < own_steps);
        oq.load(lds + i * kStage + P::kBytes, i < own_steps);
    }
    ZSMR_WAIT((STAGES - 1) * kLoads);
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    read(ph[0], qh[0], lds, 0);
    auto step = [&](int s, char* cur, const char* next, u32x4* p0, u32x4* q0, u32x4* p1, u32x4* q1) {
        read(pl, ql, cur, 1);
        multiply(p0, q0);
        interleave<kReads, 0, kMfma>();
        ZSMR_WAIT((STAGES - 2) * kLoads);
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
        op.load(cur, s + STAGES < own_steps);
        oq.load(cur + P::kBytes, s + STAGES < own_steps);
        read(p1, q1, next, 0);
        multiply(pl, q0);
        multiply(p0, ql);
        // the reads first: the next step begins with them
        interleave<kReads, 0, kMfma>();
        interleave<0, kLoads, kMfma>();
        asm volatile("" ::: "memory");      // the reads do not move on to the next step
    };
    static_assert(STAGES % 2 == 0, "the sets of registers alternate");
    for (int s = 0; s < steps; s += STAGES) {
#pragma unroll
        for (int i = 0; i < STAGES; ++i) {
            step(s + i, lds + i * kStage, lds + (i + 1) % STAGES * kStage, ph[i % 2], qh[i % 2], ph[1 - i % 2], qh[1 - i % 2]);
            if (s + i + 1 == steps) break;
        }
    }
    ZSMR_WAIT(0);           // no load may still be on its way to this LDS
    __syncthreads();

    if constexpr (GROUPS > 1) {
        f32x4* const from = reinterpret_cast<f32x4*>(smem) + thread;
        if (group > 0) {
#pragma unroll
            for (int i = 0; i < TP; ++i)
#pragma unroll
                for (int j = 0; j < TQ; ++j) from[((group - 1) * TP * TQ + i * TQ + j) * kThreads] = acc[i][j];
        }
        __syncthreads();
        if (group == 0) {
#pragma unroll
            for (int g = 0; g < GROUPS - 1; ++g)
#pragma unroll
                for (int i = 0; i < TP; ++i)
#pragma unroll
                    for (int j = 0; j < TQ; ++j) acc[i][j] += from[(g * TP * TQ + i * TQ + j) * kThreads];
        }
        __syncthreads();
    }
    if constexpr (kPartial) {
        if (group > 0) return;
#pragma unroll
        for (int j = 0; j < TQ; ++j)
#pragma unroll
            for (int i = 0; i < TP; ++i) {
                const int q = (wq * TQ + j) * 16 + lane % 16, c = (wp * TP + i) * 16 + lane / 16 * 4;
                const int64_t quarter = T == 64 ? unit.index : unit.index * (int64_t)4 + q / 64 * 2 + c / 64;
                const int64_t all = (int64_t)p.tiles * p.count * 4;
                *reinterpret_cast<f32x4*>(p.partial + ((blockIdx.y * all + quarter) * 64 + q % 64) * 64 + c % 64) = acc[i][j];
            }
        return;
    }
    // acc[i][j][r] is D at p = 16 i + 4 (lane / 16) + r, q = 16 j + lane % 16 of the
    // wave's part.  Results leave through LDS as [q][p] in fp32, the 16-byte chunk c
    // of row q in slot c ^ f(q): rows are then read along p, columns along q, each
    // with few bank conflicts.
    float* const out = reinterpret_cast<float*>(smem);
    auto at = [&](int q, int c) { return q * T + (c ^ ((q ^ q >> 3) & (T / 4 - 1) & 31)) * 4; };
#pragma unroll
    for (int j = 0; j < TQ; ++j)
#pragma unroll
        for (int i = 0; i < TP; ++i)
            if (group == 0) *reinterpret_cast<f32x4*>(out + at((wq * TQ + j) * 16 + lane % 16, (wp * TP + i) * 4 + lane / 16)) = acc[i][j];
    __syncthreads();
    uint16_t* const dst = side.dst + matrix * p.batch;
    // the other side of a symmetric result, or a tall matrix, is written along q
    const bool turned = kSymmetric ? tp != tq : KIND == N_LAST && p.tall;
    for (int k = threadIdx.x; k < T * T / 8; k += kThreads * GROUPS) {
        const int q = k / (T / 8), c = k % (T / 8);
        if (q0 + q >= p.rows || p0 + c * 8 >= padded) continue;
        const int64_t e = split_at(q0 + q, p0 + c * 8, p.ld);
        if (!kEarly) old.load(side, matrix * p.batch + e);
        f32x4* const lo = reinterpret_cast<f32x4*>(out + at(q, 2 * c));
        f32x4* const hi = reinterpret_cast<f32x4*>(out + at(q, 2 * c + 1));
        f32x8 d;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            d[i] = (*lo)[i];
            d[4 + i] = (*hi)[i];
        }
        d = old.added(side, d);
        if constexpr (KIND != N_LAST) store_split(dst, e, d);
        else if (!p.tall) put_result(p, p.first + matrix, q0 + q, p0 + c * 8, (int)min((int64_t)8, p.cols - p0 - c * 8), d);
        if (turned) {
            f32x4 a, b;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                a[i] = d[i];
                b[i] = d[4 + i];
            }
            *lo = a;
            *hi = b;
        }
    }
    if (!turned) return;
    __syncthreads();
    for (int k = threadIdx.x; k < T * T / 8; k += kThreads * GROUPS) {
        const int row = k / (T / 8), q = k % (T / 8) * 8;
        const int64_t limit = kSymmetric ? p.rows : p.cols;
        if (p0 + row >= limit || q0 + q >= (kSymmetric ? padded : p.rows)) continue;
        f32x8 d;
#pragma unroll
        for (int i = 0; i < 8; ++i) d[i] = out[at(q + i, row / 4) + row % 4];
        if constexpr (KIND == N_LAST) put_result(p, p.first + matrix, p0 + row, q0 + q, (int)min((int64_t)8, p.rows - q0 - q), d);
        else store_split(dst, split_at(p0 + row, q0 + q, p.ld), d);
    }
#endif
}

// What the parts of an N_PARTIAL product add up to, a quarter of a tile a workgroup.
// Reads the parts once: 10 us for 91 tiles of 5 parts, 53 to 55 for 528 of 6 (5.0 TB/s
// with what it writes).
__global__ __launch_bounds__(kThreads) void ns_join_kernel(NsProduct p, int split) {
#if defined(__HIP_DEVICE_COMPILE__)
    constexpr int kPitch = 68;      // rows are read along p and along q
    __shared__ __attribute__((aligned(16))) float out[64 * kPitch];
    const Unit unit = unit_of<true>(p);
    const NsSide& side = p.side[0];
    const int64_t p0 = (int64_t)unit.tp * 64, q0 = (int64_t)unit.tq * 64, padded = p.ld / 2;
    if (p0 >= p.cols || q0 >= p.rows || unit.tq > unit.tp) return;
    uint16_t* const dst = side.dst + unit.matrix * p.batch;
    const int64_t part = (int64_t)p.tiles * p.count * 4 * 64 * 64;
    const float* const from = p.partial + (int64_t)unit.index * 64 * 64;
    f32x8 sum[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) sum[i] = load8<ZSMR_FP32>(from, (i * kThreads + threadIdx.x) * 8);
#pragma unroll 4
    for (int s = 1; s < split; ++s)
#pragma unroll
        for (int i = 0; i < 2; ++i) sum[i] += load8<ZSMR_FP32>(from + s * part, (i * kThreads + threadIdx.x) * 8);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int k = i * kThreads + threadIdx.x, q = k / 8, c = k % 8 * 8;
        const f32x8 d = sum[i] * side.mul;
        if (q0 + q < p.rows && p0 + c < padded) store_split(dst, split_at(q0 + q, p0 + c, p.ld), d);
#pragma unroll
        for (int r = 0; r < 8; ++r) out[q * kPitch + c + r] = d[r];
    }
    if (unit.tp == unit.tq) return;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int k = i * kThreads + threadIdx.x, row = k % 64, q = k / 64 * 8;
        if (p0 + row >= p.rows || q0 + q >= padded) continue;
        f32x8 d;
#pragma unroll
        for (int r = 0; r < 8; ++r) d[r] = out[(q + r) * kPitch + row];
        store_split(dst, split_at(p0 + row, q0 + q, p.ld), d);
    }
#endif
}

// ------------------------------------------------------------ before the products --
// Squares are taken and summed in fp64, as for the gradient norm.
__device__ __forceinline__ void add_squares(f32x8 f, double* s) {
#pragma unroll
    for (int i = 0; i < 8; ++i) *s = __builtin_fma((double)f[i], (double)f[i], *s);
}

// Partial sums of squares of the group's matrices: parts of each.  4,096 x 4,096 bf16 take
// 9 us, 3.6 TB/s.
template <int DT>
__global__ __launch_bounds__(kThreads) void ns_sumsq_kernel(const void* x, int64_t stride, int64_t batch, int64_t rows, int64_t cols,
                                                            int32_t row_threads, double* partial) {
    const int64_t from = blockIdx.y * batch;
    const int each = kThreads / row_threads, t = threadIdx.x % row_threads;
    double s = 0;
    for (int64_t r = (int64_t)blockIdx.x * each + threadIdx.x / row_threads; r < rows; r += (int64_t)gridDim.x * each)
        for (int64_t c = t * 8; c < cols; c += row_threads * 8) {
            const int64_t e = from + r * stride + c;
            if (c + 8 <= cols) {
                add_squares(load8<DT>(x, e), &s);
            } else {
                for (int64_t i = 0; i < cols - c; ++i) {
                    const double f = load1<DT>(x, e + i);
                    s = __builtin_fma(f, f, s);
                }
            }
        }
    s = block_sum<kThreads>(s);
    if (threadIdx.x == 0) partial[blockIdx.y * gridDim.x + blockIdx.x] = s;
}

// The mean gradient over the ranks, the momentum, and the update u before it is
// orthogonalised, with its partial sums of squares.  Rows are summed in rank
// order, in fp32.  Bound by HBM: 28 bytes an element of 8 rows, 5.8 TB/s (283 us for
// 14,336 x 4,096).
struct MomentumArgs {
    StepArgs step;                  // from the group's first matrix on
    int64_t each;                   // elements of a matrix
    int32_t nesterov;
    float beta;
    float* u;
    double* partial;
};
__device__ __forceinline__ float momentum(const StepArgs& s, float beta, int32_t nesterov, float g, float* m) {
    const float sum = s.inv_pow2 ? g * s.inv_nf : g / s.nf, next = beta * *m + sum;
    *m = next;
    return nesterov ? sum + beta * next : next;
}
constexpr int kRows = 8;
template <int DT>
__global__ __launch_bounds__(kThreads) void ns_momentum_kernel(MomentumArgs a) {
    const int64_t from = blockIdx.y * a.each;
    double s = 0;
    for (int64_t i = ((int64_t)blockIdx.x * kThreads + threadIdx.x) * 8; i < a.each; i += (int64_t)gridDim.x * kThreads * 8) {
        const int64_t e = from + i;
        const uint16_t* p = a.step.grads + e;
        if (i + 8 <= a.each) {
            f32x8 g = -0.0f;            // -0 + x is x for every x
            int r = 0;
            for (; r + kRows <= a.step.nrows; r += kRows) {
                u16x8 h[kRows];
#pragma unroll
                for (int k = 0; k < kRows; ++k)
                    h[k] = __builtin_nontemporal_load(reinterpret_cast<const u16x8_any*>(p + (int64_t)(r + k) * a.step.row_stride));
#pragma unroll
                for (int k = 0; k < kRows; ++k)
#pragma unroll
                    for (int j = 0; j < 8; ++j) g[j] += widen16<DT>(h[k][j]);
            }
            for (; r < a.step.nrows; ++r) {
                const u16x8 h = *reinterpret_cast<const u16x8_any*>(p + (int64_t)r * a.step.row_stride);
#pragma unroll
                for (int j = 0; j < 8; ++j) g[j] += widen16<DT>(h[j]);
            }
            f32x8 m = load8<ZSMR_FP32>(a.step.m, e), u;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                float mj = m[j];
                u[j] = momentum(a.step, a.beta, a.nesterov, g[j], &mj);
                m[j] = mj;
            }
            store8<ZSMR_FP32>(a.step.m, e, m);
            store8<ZSMR_FP32>(a.u, e, u);
            add_squares(u, &s);
        } else {
            for (int64_t j = 0; j < a.each - i; ++j) {
                float g = widen16<DT>(p[j]);
                for (int r = 1; r < a.step.nrows; ++r) g += widen16<DT>(p[(int64_t)r * a.step.row_stride + j]);
                const float u = momentum(a.step, a.beta, a.nesterov, g, a.step.m + e + j);
                a.u[e + j] = u;
                s = __builtin_fma((double)u, (double)u, s);
            }
        }
    }
    s = block_sum<kThreads>(s);
    if (threadIdx.x == 0) a.partial[blockIdx.y * gridDim.x + blockIdx.x] = s;
}

// first / (norm + eps) of a matrix; a matrix of zeros stays one with eps 0 too.
__device__ __forceinline__ double inverse_norm(double sum, double eps, double first) {
    const double norm = sqrt(sum) + eps;
    return norm == 0 ? 0 : first / norm;
}
__global__ __launch_bounds__(64) void ns_norm_kernel(const double* partial, int32_t parts, double eps, double first, double* inverse) {
    double s = 0;
    for (int i = threadIdx.x; i < parts; i += 64) s += partial[(int64_t)blockIdx.x * parts + i];
    s = block_sum<64>(s);
    if (threadIdx.x == 0) inverse[blockIdx.x] = inverse_norm(s, eps, first);
}

// X0 in two fp16 parts and in the wide orientation.  A workgroup takes 64 rows and
// 64 columns of it; a tall matrix is turned in LDS.  1,600 x 6,400 of fp32 take 14 us, 5.8
// TB/s; turned, 14,336 x 4,096 105 us, 4.5 TB/s (rows of tiles along n 114, rows of 65 in
// LDS 119).
struct PackArgs {
    const void* x;
    int64_t stride, batch, m, n, np;
    const double* inverse;
    uint16_t* dst;
    int32_t tiles_n, tiles, tall;
};
template <int DT>
__global__ __launch_bounds__(kThreads) void ns_pack_kernel(PackArgs a) {
    // element (row, column) of the wide orientation's tile, in 16-byte chunks of a row
    // that change places: the writes of a column and the reads of two rows use all banks
    __shared__ __attribute__((aligned(16))) float turned[64 * 64];
    auto chunk_at = [&](int row, int chunk) { return row * 64 + (chunk ^ (row >> 3) ^ (row & 1)) * 4; };
    const int64_t matrix = blockIdx.x / a.tiles;
    const int tile = blockIdx.x % a.tiles;
    int tm = tile / a.tiles_n, tn = tile % a.tiles_n;
    if (a.tall) {
        // 8 tiles along n, then the next ones along m: pages of both matrices are used whole
        const int tiles_m = a.tiles / a.tiles_n, band = tile / (8 * tiles_m), width = min(8, a.tiles_n - band * 8), in_band = tile - band * 8 * tiles_m;
        tm = in_band / width;
        tn = band * 8 + in_band % width;
    }
    const int64_t m0 = (int64_t)tm * 64, n0 = (int64_t)tn * 64;
    const int64_t rows = a.tall ? a.n : a.m, cols = a.tall ? a.m : a.n, r0 = a.tall ? n0 : m0, c0 = a.tall ? m0 : n0;
    uint16_t* dst = a.dst + matrix * a.m * a.np * 2;
    f32x8 f[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const int r = k * 32 + threadIdx.x / 8, c = threadIdx.x % 8 * 8;
        f[k] = 0.f;
        if (r0 + r < rows) {
            const int64_t e = matrix * a.batch + (r0 + r) * a.stride + c0 + c;
            if (c0 + c + 8 <= cols) {
                f[k] = load8<DT>(a.x, e);
            } else {
#pragma unroll
                for (int i = 0; i < 7; ++i)
                    if (c0 + c + i < cols) f[k][i] = load1<DT>(a.x, e + i);
            }
        }
    }
    const double inverse = a.inverse[matrix];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const int r = k * 32 + threadIdx.x / 8, c = threadIdx.x % 8 * 8;
#pragma unroll
        for (int i = 0; i < 8; ++i) f[k][i] = (float)((double)f[k][i] * inverse);
        if (!a.tall) {
            if (r0 + r < rows && c0 + c < a.np) store_split(dst, split_at(r0 + r, c0 + c, a.np * 2), f[k]);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) turned[chunk_at(c + i, r / 4) + r % 4] = f[k][i];
        }
    }
    if (!a.tall) return;
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const int r = k * 32 + threadIdx.x / 8, c = threadIdx.x % 8 * 8;
        if (m0 + r >= a.m || n0 + c >= a.np) continue;
        const f32x4 lo = *reinterpret_cast<const f32x4*>(turned + chunk_at(r, c / 4)), hi = *reinterpret_cast<const f32x4*>(turned + chunk_at(r, c / 4 + 1));
        const f32x8 t = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
        store_split(dst, split_at(m0 + r, n0 + c, a.np * 2), t);
    }
}

// ------------------------------------------------------------ small matrices --
// A workgroup takes a whole matrix through every pass.  X is in LDS as two fp16
// parts, and in fp32 in registers: a wave owns up to PARTS blocks of FP x FQ tiles of
// 16 columns and 16 rows, a lane four consecutive columns of a row of each tile.  The
// inner matrix is in LDS once, A and then B.  Rows and columns past the matrix are zeros.
struct SmallArgs {
    NewtonArgs a;
    int64_t first;                  // matrix
};
// The 16-byte chunk c of row r sits in slot c ^ f(r): 8 rows read at one chunk fall
// into different banks, and so do the 32 bytes that a transposing read takes of each of
// 4 rows.  Half of the kernel's LDS cycles are conflicts still; an f of more bits, for 16
// lanes at a time, needs more registers than there are and took a tenth longer.
__device__ __forceinline__ int small_slot(int row, int chunk) { return chunk ^ ((row & 3) << 1 | (row >> 2 & 1)); }
// Where a lane reads its operand registers of 16 rows (or, OUTER, columns) and k =
// 8 (lane / 16) + 0..7 of the hi parts at the matrix's corner; LD: bytes of a row.  The
// lo parts are 64 bytes on or back (the slot's bit 2), 16 rows, 32 k and 32 columns on
// are fixed distances away.
template <int LD, bool OUTER>
__device__ __forceinline__ int small_lane() {
    const int lane = threadIdx.x % 64;
    if constexpr (OUTER) {
        const int row = lane / 16 * 8 + lane % 16 / 4;
        return row * LD + small_slot(row, lane % 4 / 2) * 16 + (lane & 1) * 8;
    } else {
        const int row = lane % 16;
        return row * LD + small_slot(row, lane / 16) * 16;
    }
}
// t: the corner of the 16 rows (columns) and 32 k; at: small_lane(), moved for the lo
// parts and for columns 16..31 of 32.
template <int LD, bool OUTER>
__device__ __forceinline__ u32x4 small_read(const char* t, int at) {
    if constexpr (OUTER) {
        // row + 4 has the other f's bit 0
        const u32x2 a = read_transposed(t + at), b = read_transposed(t + 4 * LD + (at ^ 16));
        u32x4 r;
        r[0] = a[0];
        r[1] = a[1];
        r[2] = b[0];
        r[3] = b[1];
        return r;
    } else {
        return *reinterpret_cast<const u32x4*>(t + at);
    }
}
// Four columns from col on of a row, in both parts.
template <int LD>
__device__ __forceinline__ void small_store(char* t, int row, int col, f32x4 f) {
    u16x4 hi, lo;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        hi[i] = narrow16<ZSMR_FP16>(f[i]);
        lo[i] = narrow16<ZSMR_FP16>(f[i] - widen16<ZSMR_FP16>(hi[i]));
    }
    char* const p = t + row * LD + col / 32 * 128 + (col & 4) * 2;
    const int slot = small_slot(row, col % 32 / 8) * 16;
    *reinterpret_cast<u16x4*>(p + slot) = hi;
    *reinterpret_cast<u16x4*>(p + (slot ^ 64)) = lo;
}

// Up to four elements in memory, `step` apart; those past `count` are zeros.
template <int DT>
__device__ __forceinline__ f32x4 load4(const void* p, int64_t e, int64_t step, int count) {
    f32x4 f = 0.f;
    if (step == 1 && count >= 4) {
        if constexpr (DT == ZSMR_FP32) return *reinterpret_cast<const f32x4_any*>(static_cast<const float*>(p) + e);
        const u16x4 h = *reinterpret_cast<const u16x4_any*>(static_cast<const uint16_t*>(p) + e);
#pragma unroll
        for (int i = 0; i < 4; ++i) f[i] = widen16<DT>(h[i]);
        return f;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (i < count) f[i] = load1<DT>(p, e + i * step);
    return f;
}
template <int DT>
__device__ __forceinline__ void store4(void* p, int64_t e, int64_t step, int count, f32x4 f) {
    if (step == 1 && count >= 4) {
        if constexpr (DT == ZSMR_FP32) {
            *reinterpret_cast<f32x4_any*>(static_cast<float*>(p) + e) = f;
        } else {
            u16x4 h;
#pragma unroll
            for (int i = 0; i < 4; ++i) h[i] = narrow16<DT>(f[i]);
            *reinterpret_cast<u16x4_any*>(static_cast<uint16_t*>(p) + e) = h;
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (i < count) store1<DT>(p, e + i * step, f[i]);
}
// Eight contiguous elements, or (not WHOLE) as many as lie before `end` and repeats of
// the last.  Either way nothing is loaded under a branch, at whose end it would be waited for.
template <int DT, bool WHOLE>
__device__ __forceinline__ f32x8 load_row(const void* p, int64_t e, int64_t end) {
    if constexpr (WHOLE) return load8<DT>(p, e);
    f32x8 f;
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = load1<DT>(p, min(e + i, end - 1));
    return f;
}
// The first `count` of eight contiguous elements.
template <int DT>
__device__ __forceinline__ void store_some(void* p, int64_t e, int count, f32x8 f) {
    if (count >= 8) return store8<DT>(p, e, f);
#pragma unroll
    for (int i = 0; i < 7; ++i)
        if (i < count) store1<DT>(p, e + i, f[i]);
}
template <typename F>
__device__ __forceinline__ void by_dtype(int32_t dtype, F each) {
    if (dtype == ZSMR_BF16) each(std::integral_constant<int, ZSMR_BF16>());
    else if (dtype == ZSMR_FP16) each(std::integral_constant<int, ZSMR_FP16>());
    else each(std::integral_constant<int, ZSMR_FP32>());
}

// A matrix of at most MP x NP.  A product waits for the one before it, so a CU's matrix
// units are busy 0.15 (64 x 64) to 0.29 (128 x 128) of the time; 24 of 64 x 64 take 16.1 us
// where the 18 launches of larger ones took 92.  The plain call reads and writes each register's four
// elements where they lie.  The shard's step (STEP) has nrows + 2 arrays of the matrix's
// shape to read and three to write, so it takes memory in its own order, eight elements of
// a row a thread, and the matrix changes hands in LDS, as fp32 rows a little longer than
// the matrix's: 4 of 128 x 128 with 5 steps take 60.9 us at 4 rows and 64.5 at 16 (61.7
// and 82 where the elements lie), 4 of 64 x 64 17.3 (19.4), while the plain call for 4 of
// 128 x 128 would take 52.0 us for 49.1.
template <int MP, int NP, int WAVES, int FP, int FQ, bool STEP>
__global__ __launch_bounds__(WAVES * 64) void ns_small_kernel(SmallArgs s) {
#if defined(__HIP_DEVICE_COMPILE__)
    __shared__ __attribute__((aligned(1024))) char smem[MP * NP * 4 + MP * MP * 4];
    __shared__ double norm;
    constexpr int kCols = FP * 16, kRows = FQ * 16, PARTS = MP / kRows * (NP / kCols) / WAVES, XLD = NP * 4, ALD = MP * 4;
    static_assert(PARTS * WAVES == MP / kRows * (NP / kCols) && MP / kRows * (MP / kCols) <= WAVES && FP % 2 == 0, "blocks for every wave");
    const NewtonArgs& a = s.a;
    const NsShape& shape = a.shape;
    const int lane = threadIdx.x % 64, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    const int m = (int)shape.m, n = (int)shape.n, mb = (int)shape.mp / kRows, nb = (int)((shape.np + kCols - 1) / kCols);
    char* const xs = smem;
    char* const as = smem + MP * XLD;
    const int64_t matrix = s.first + blockIdx.x;
    const bool tall = shape.tall;

    // Part t of the wave, tile (i, j) of it: columns p from p0 + 16 i on, rows q from q0 + 16 j.
    struct Place {
        int row, col;
    };
    auto place = [&](int id, int i, int j) {
        return Place{id % mb * kRows + j * 16 + lane % 16, id / mb * kCols + i * 16 + lane / 16 * 4};
    };
    auto every = [&](auto each) {
#pragma unroll
        for (int t = 0; t < PARTS; ++t)
#pragma unroll
            for (int i = 0; i < FP; ++i)
#pragma unroll
                for (int j = 0; j < FQ; ++j) each(t, i, j, place(wave + t * WAVES, i, j));
    };
    // How many of a register's elements, from p on along its row, the matrix has.
    auto inside = [&](int t, Place p) { return wave + t * WAVES < mb * nb && p.row < m ? n - p.col : 0; };
    auto element = [&](Place p, int64_t stride, int64_t batch) {
        return matrix * batch + (tall ? p.col * stride + p.row : p.row * stride + p.col);
    };
    constexpr int kChunks = MP * NP / 8 / (WAVES * 64);
    static_assert(kChunks * 8 * WAVES * 64 == MP * NP, "chunks for every thread");
    static_assert(sizeof(smem) >= (MP * (NP + 4) > NP * (MP + 4) ? MP * (NP + 4) : NP * (MP + 4)) * 4, "room for the matrix");
    const int rows = tall ? n : m, cols = tall ? m : n, of_row = (cols + 7) / 8, pitch = (cols + 3) / 4 * 4 + 4;
    const int64_t each = shape.m * shape.n, at = matrix * each;      // of matrices one behind the other
    float* const flat = reinterpret_cast<float*>(smem);
    struct Chunk {
        int row, col, count, at;        // at: in the matrix, and where count is 0, in it too
    };
    auto chunk = [&](int k) {
        const int id = k * (WAVES * 64) + (int)threadIdx.x, row = id / of_row, col = id % of_row * 8;
        return Chunk{row, col, row < rows ? min(8, cols - col) : 0, row < rows ? row * cols + col : 0};
    };
    auto put_flat = [&](Chunk c, f32x8 f) {
        // whole groups of four: the row's end has room for them
        float* const to = flat + c.row * pitch + c.col;
        if (c.count > 0) *reinterpret_cast<f32x4*>(to) = f32x4{f[0], f[1], f[2], f[3]};
        if (c.count > 4) *reinterpret_cast<f32x4*>(to + 4) = f32x4{f[4], f[5], f[6], f[7]};
    };

    f32x4 x[PARTS][FP][FQ];
    double sum = 0;
    if constexpr (STEP) {
        f32x8 w[kChunks], g[kChunks];
        auto load = [&](auto dt, auto whole) {
            constexpr bool kWhole = decltype(whole)::value;
#pragma unroll
            for (int k = 0; k < kChunks; ++k) {
                w[k] = load_row<ZSMR_FP32, kWhole>(a.step.m, at + chunk(k).at, at + each);
                g[k] = -0.0f;               // -0 + x is x for every x
            }
#pragma unroll 2
            for (int r = 0; r < a.step.nrows; ++r) {
                f32x8 h[kChunks];
#pragma unroll
                for (int k = 0; k < kChunks; ++k)
                    h[k] = load_row<decltype(dt)::value, kWhole>(a.step.grads + r * a.step.row_stride, at + chunk(k).at, at + each);
#pragma unroll
                for (int k = 0; k < kChunks; ++k) g[k] += h[k];
            }
        };
        by_dtype(a.grad_dtype, [&](auto dt) {
            if (cols % 8 == 0) load(dt, std::true_type());
            else load(dt, std::false_type());
        });
#pragma unroll
        for (int k = 0; k < kChunks; ++k) {
            const Chunk c = chunk(k);
            f32x8 u;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                float next = w[k][i];
                u[i] = momentum(a.step, a.beta, a.nesterov, g[k][i], &next);
                w[k][i] = next;
                if (i < c.count) sum = __builtin_fma((double)u[i], (double)u[i], sum);
            }
            store_some<ZSMR_FP32>(a.step.m, at + c.at, c.count, w[k]);
            put_flat(c, u);
        }
    } else {
        const int64_t step = tall ? a.x_stride : 1;
        by_dtype(a.x_dtype, [&](auto dt) {
            every([&](int t, int i, int j, Place p) {
                x[t][i][j] = load4<decltype(dt)::value>(a.x, element(p, a.x_stride, a.x_batch), step, inside(t, p));
            });
        });
        every([&](int t, int i, int j, Place) {
#pragma unroll
            for (int r = 0; r < 4; ++r) sum = __builtin_fma((double)x[t][i][j][r], (double)x[t][i][j][r], sum);
        });
    }
    sum = block_sum<WAVES * 64>(sum);
    if (threadIdx.x == 0) norm = inverse_norm(sum, a.eps, a.first);
    __syncthreads();
    const double inverse = norm;
    auto store_x = [&]() {
        every([&](int t, int i, int j, Place p) {
            if (wave + t * WAVES < mb * nb && p.col < (int)shape.np) small_store<XLD>(xs, p.row, p.col, x[t][i][j]);
        });
    };
    every([&](int t, int i, int j, Place p) {
        if constexpr (STEP) {
            const int count = inside(t, p);
            x[t][i][j] = 0.f;
            if (!tall && count > 0) x[t][i][j] = *reinterpret_cast<const f32x4*>(flat + p.row * pitch + p.col);
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                if (tall && r < count) x[t][i][j][r] = flat[(p.col + r) * pitch + p.row];
                if (r >= count) x[t][i][j][r] = 0.f;
            }
        }
#pragma unroll
        for (int r = 0; r < 4; ++r) x[t][i][j][r] = (float)((double)x[t][i][j][r] * inverse);
    });
    if (STEP) __syncthreads();
    store_x();
    __syncthreads();

    // A part of D[p, q] = sum_k P[p, k] Q[q, k], over `steps` of 32 k; OUTER: k is P's
    // row index.  The next step's operands are read while this one's are multiplied.
    // Columns past a block's matrix are read from elsewhere in LDS and not stored.
    f32x4 acc[FP][FQ];
    struct Operands {
        u32x4 ph[FP], pl[FP], qh[FQ], ql[FQ];
    };
    auto product = [&](auto outer, auto p_ld, const char* p, int p0, auto q_ld, const char* q, int q0, int steps) {
        constexpr bool OUTER = decltype(outer)::value;
        constexpr int PLD = decltype(p_ld)::value, QLD = decltype(q_ld)::value;
#pragma unroll
        for (int i = 0; i < FP; ++i)
#pragma unroll
            for (int j = 0; j < FQ; ++j) acc[i][j] = 0.f;
        p += OUTER ? p0 * 4 : p0 * PLD;
        q += q0 * QLD;
        const int pa = small_lane<PLD, OUTER>(), qa = small_lane<QLD, false>();
        auto read = [&](Operands& o, int k) {
            const char* const pk = p + k * (OUTER ? 32 * PLD : 128);
            const char* const qk = q + k * 128;
#pragma unroll
            for (int i = 0; i < FP; ++i) {
                const char* const t = pk + (OUTER ? i / 2 * 128 : i * 16 * PLD);
                const int at = OUTER ? pa ^ (i % 2 * 32) : pa;
                o.ph[i] = small_read<PLD, OUTER>(t, at);
                o.pl[i] = small_read<PLD, OUTER>(t, at ^ 64);
            }
#pragma unroll
            for (int j = 0; j < FQ; ++j) {
                o.qh[j] = small_read<QLD, false>(qk + j * 16 * QLD, qa);
                o.ql[j] = small_read<QLD, false>(qk + j * 16 * QLD, qa ^ 64);
            }
            asm volatile("" ::: "memory");      // the reads stay ahead of what follows
        };
        auto multiply = [&](const u32x4* a, const u32x4* b) {
#pragma unroll
            for (int i = 0; i < FP; ++i)
#pragma unroll
                for (int j = 0; j < FQ; ++j) acc[i][j] = mfma<ZSMR_FP16>(a[i], b[j], acc[i][j]);
        };
        Operands o0, o1;
        read(o0, 0);
        for (int k = 0; k < steps; k += 2) {
            read(o1, min(k + 1, steps - 1));        // always: a branch would make all reads wait at its end
            multiply(o0.ph, o0.qh);
            multiply(o0.pl, o0.qh);
            multiply(o0.ph, o0.ql);
            if (k + 1 == steps) break;
            read(o0, min(k + 2, steps - 1));
            multiply(o1.ph, o1.qh);
            multiply(o1.pl, o1.qh);
            multiply(o1.ph, o1.ql);
        }
    };
    // A wave has one part of the inner matrix: there are no more than waves.
    const bool mine = wave < mb * (((int)shape.mp + kCols - 1) / kCols);
    const int p0 = wave / mb * kCols, q0 = wave % mb * kRows;
    auto store_inner = [&](const f32x4 (&f)[FP][FQ]) {
        if (!mine) return;
#pragma unroll
        for (int i = 0; i < FP; ++i)
#pragma unroll
            for (int j = 0; j < FQ; ++j) {
                const Place p = place(wave, i, j);
                if (p.col < (int)shape.mp) small_store<ALD>(as, p.row, p.col, f[i][j]);
            }
    };
    constexpr std::true_type kRowsOfK;
    constexpr std::false_type kAlongK;
    constexpr std::integral_constant<int, XLD> xld;
    constexpr std::integral_constant<int, ALD> ald;
    const int x_steps = (int)shape.np / 32, a_steps = (int)shape.mp / 32;
    for (int pass = 0; pass < a.steps; ++pass) {
        const NsPass k = a.pass[pass];
        f32x4 inner[FP][FQ];
        // A, then B over it
        if (mine) {
            product(kAlongK, xld, xs, p0, xld, xs, q0, x_steps);
#pragma unroll
            for (int i = 0; i < FP; ++i)
#pragma unroll
                for (int j = 0; j < FQ; ++j) inner[i][j] = acc[i][j] * k.a_mul;
        }
        store_inner(inner);
        __syncthreads();
        if (mine) {
            product(kAlongK, ald, as, p0, ald, as, q0, a_steps);
#pragma unroll
            for (int i = 0; i < FP; ++i)
#pragma unroll
                for (int j = 0; j < FQ; ++j) inner[i][j] = inner[i][j] * k.b_old + acc[i][j] * k.b_mul;
        }
        __syncthreads();
        store_inner(inner);
        __syncthreads();
        // X', which stays in registers until every wave has read X
#pragma unroll
        for (int t = 0; t < PARTS; ++t) {
            const int id = wave + t * WAVES;
            if (id >= mb * nb) continue;
            product(kRowsOfK, xld, xs, id / mb * kCols, ald, as, id % mb * kRows, a_steps);
#pragma unroll
            for (int i = 0; i < FP; ++i)
#pragma unroll
                for (int j = 0; j < FQ; ++j) x[t][i][j] = x[t][i][j] * k.x_old + acc[i][j] * k.x_mul;
        }
        if (pass + 1 == a.steps) break;
        __syncthreads();
        store_x();
        __syncthreads();
    }
    if constexpr (STEP) {
        __syncthreads();
        every([&](int t, int i, int j, Place p) {
            const int count = inside(t, p);
            if (!tall && count > 0) *reinterpret_cast<f32x4*>(flat + p.row * pitch + p.col) = x[t][i][j];
#pragma unroll
            for (int r = 0; r < 4; ++r)
                if (tall && r < count) flat[(p.col + r) * pitch + p.row] = x[t][i][j][r];
        });
        __syncthreads();
        f32x8 w[kChunks];
        auto load = [&](auto whole) {
#pragma unroll
            for (int k = 0; k < kChunks; ++k) w[k] = load_row<ZSMR_FP32, decltype(whole)::value>(a.step.master, at + chunk(k).at, at + each);
        };
        if (cols % 8 == 0) load(std::true_type());
        else load(std::false_type());
#pragma unroll
        for (int k = 0; k < kChunks; ++k) {
            const Chunk c = chunk(k);
            if (c.count <= 0) continue;
            const float* const from = flat + c.row * pitch + c.col;
            f32x8 f = 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (i < c.count) f[i] = from[i];
            const int64_t e = at + c.at;
            f = w[k] * a.decay - a.rate * f;
            store_some<ZSMR_FP32>(a.step.master, e, c.count, f);
            by_dtype(a.param_dtype, [&](auto dt) { store_some<decltype(dt)::value>(a.step.p16, e, c.count, f); });
        }
    } else {
        const int64_t step = tall ? a.out_stride : 1;
        by_dtype(a.out_dtype, [&](auto dt) {
            every([&](int t, int i, int j, Place p) {
                store4<decltype(dt)::value>(a.out, element(p, a.out_stride, a.out_batch), step, inside(t, p), x[t][i][j]);
            });
        });
    }
#endif
}

// ------------------------------------------------------------------ launches --
template <bool STEP>
void small_of(const SmallArgs& s, unsigned count, hipStream_t stream) {
    if (s.a.shape.small == 1) ns_small_kernel<64, 64, 8, 2, 1, STEP><<<count, 512, 0, stream>>>(s);
    else if (s.a.shape.small == 2) ns_small_kernel<64, 256, 8, 4, 2, STEP><<<count, 512, 0, stream>>>(s);
    else ns_small_kernel<128, 128, 8, 4, 2, STEP><<<count, 512, 0, stream>>>(s);
}
hipError_t launch_small(const NewtonArgs& a, hipStream_t stream) {
    SmallArgs s{};
    s.a = a;
    launch_rows(a.shape.count, 512, [&](int64_t first, int64_t count) {
        s.first = first;
        if (a.step.master) small_of<true>(s, (unsigned)count, stream);
        else small_of<false>(s, (unsigned)count, stream);
    });
    return hipGetLastError();
}

struct Space {
    uint16_t* matrix[kNsMatrices];
    double *partial, *inverse;
};
Space space_of(const NsShape& s, void* ws) {
    const NsSpace w = ns_space(s);
    char* p = static_cast<char*>(ws);
    Space r;
    for (int i = 0; i < kNsMatrices; ++i) r.matrix[i] = reinterpret_cast<uint16_t*>(p + w.matrix[i]);
    r.partial = reinterpret_cast<double*>(p + w.partial);
    r.inverse = reinterpret_cast<double*>(p + w.inverse);
    return r;
}

template <int KIND>
void launch_product(NsProduct& p, const NsGrid& grid, hipStream_t stream) {
    p.split_steps = grid.split_steps;
    p.p_tiles = grid.p_tiles;
    p.q_tiles = grid.q_tiles;
    p.tiles = grid.tiles;
    for (int i = 0; i < grid.parts; ++i) {
        const NsPart& part = grid.part[i];
        const dim3 groups((unsigned)ns_groups(part), grid.split);
        p.first_tile = (int32_t)part.first;
        p.quarters = ns_quarters(part.form);
        if (part.form == NS_WIDE) ns_product_kernel<KIND, 128, 1, 2><<<groups, kThreads, 0, stream>>>(p);
        else if (part.form == NS_DEEP) ns_product_kernel<KIND, 128, 2, 2><<<groups, kThreads * 2, 0, stream>>>(p);
        else if (part.form == NS_THIN) ns_product_kernel<KIND, 64, 2, 4><<<groups, kThreads * 2, 0, stream>>>(p);
        else ns_product_kernel<KIND, 64, 2, 2><<<groups, kThreads * 2, 0, stream>>>(p);
    }
}

template <typename F>
void of_dtype(int32_t dtype, F each) {
    if (dtype == ZSMR_BF16) each(std::integral_constant<int, ZSMR_BF16>());
    else if (dtype == ZSMR_FP16) each(std::integral_constant<int, ZSMR_FP16>());
    else each(std::integral_constant<int, ZSMR_FP32>());
}

// From the partial sums on, for `count` matrices from the `first` one on.
void products(const NewtonArgs& a, const NsOp* ops, int n_ops, const Space& w, const void* x, int32_t dtype, int64_t stride, int64_t batch,
              int64_t first, int count, hipStream_t stream) {
    const NsShape& s = a.shape;
    ns_norm_kernel<<<count, 64, 0, stream>>>(w.partial, s.parts, a.eps, a.first, w.inverse);
    PackArgs pack{};
    pack.x = x;
    pack.stride = stride;
    pack.batch = batch;
    pack.m = s.m;
    pack.n = s.n;
    pack.np = s.np;
    pack.inverse = w.inverse;
    pack.dst = w.matrix[M_X0];
    pack.tiles_n = (int32_t)((s.np + 63) / 64);
    pack.tiles = (int32_t)((s.m + 63) / 64) * pack.tiles_n;
    pack.tall = s.tall;
    of_dtype(dtype, [&](auto dt) { ns_pack_kernel<decltype(dt)::value><<<pack.tiles * count, kThreads, 0, stream>>>(pack); });

    NsProduct p{};
    p.count = count;
    p.first = first;
    p.tall = s.tall;
    p.apply = a.step.master != nullptr;
    p.dtype = p.apply ? a.param_dtype : a.out_dtype;
    p.out = p.apply ? a.step.p16 : a.out;
    p.out_stride = a.out_stride;
    p.out_batch = a.out_batch;
    p.master = a.step.master;
    p.decay = a.decay;
    p.rate = a.rate;
    for (int i = 0; i < n_ops;) {
        const NsOp& o = ops[i];
        const int sides = ns_sides(&o);
        for (int k = 0; k < sides; ++k) {
            const NsOp& op = ops[i + k];
            NsSide& side = p.side[k];
            side.p = w.matrix[op.p];
            side.q = w.matrix[op.q];
            side.old = op.old < 0 ? nullptr : w.matrix[op.old];
            side.old2 = op.old2 < 0 ? nullptr : w.matrix[op.old2];
            side.dst = w.matrix[op.dst];
            side.mul = op.mul;
            side.old_mul = op.old_mul;
            side.old2_mul = op.old2_mul;
        }
        i += sides;
        const bool from_x = ns_from_x(o), gram = ns_gram(o);
        p.p_rows = p.q_rows = p.rows = s.m;
        p.p_ld = (from_x ? s.np : s.mp) * 2;
        p.q_ld = (gram ? s.np : s.mp) * 2;
        p.cols = o.kind == N_INNER ? s.m : s.n;
        p.ld = (o.kind == N_INNER ? s.mp : s.np) * 2;
        p.p_batch = s.m * p.p_ld;
        p.q_batch = s.m * p.q_ld;
        p.batch = s.m * p.ld;
        p.steps = (int32_t)ns_steps_of(s, o);
        const NsGrid grid = ns_grid(s, o.kind, (int64_t)sides * count, p.steps, gram);
        if (grid.split > 1) {
            p.partial = reinterpret_cast<float*>(w.matrix[o.p == M_X0 ? M_X1 : M_X0]);
            launch_product<N_PARTIAL>(p, grid, stream);
            p.first_tile = 0;
            p.quarters = 1;
            ns_join_kernel<<<(unsigned)(grid.part[0].count * 4), kThreads, 0, stream>>>(p, grid.split);
        } else if (o.kind == N_INNER) launch_product<N_INNER>(p, grid, stream);
        else if (o.kind == N_UPDATE) launch_product<N_UPDATE>(p, grid, stream);
        else launch_product<N_LAST>(p, grid, stream);
    }
}

}  // namespace

hipError_t launch_orthogonalize(const NewtonArgs& a, const NsOp* ops, int n_ops, void* ws, hipStream_t stream) {
    const NsShape& s = a.shape;
    if (s.small) return launch_small(a, stream);
    const Space w = space_of(s, ws);
    const int64_t rows = s.tall ? s.n : s.m, cols = s.tall ? s.m : s.n;
    int32_t row_threads = 1;
    while (row_threads < kThreads && row_threads * 8 < cols) row_threads *= 2;
    for (int64_t first = 0; first < s.count; first += s.group) {
        const int count = (int)std::min(s.group, s.count - first);
        const char* x = static_cast<const char*>(a.x) + first * a.x_batch * (a.x_dtype == ZSMR_FP32 ? 4 : 2);
        of_dtype(a.x_dtype, [&](auto dt) {
            ns_sumsq_kernel<decltype(dt)::value><<<dim3(s.parts, count), kThreads, 0, stream>>>(x, a.x_stride, a.x_batch, rows, cols,
                                                                                               row_threads, w.partial);
        });
        products(a, ops, n_ops, w, x, a.x_dtype, a.x_stride, a.x_batch, first, count, stream);
    }
    return hipGetLastError();
}

hipError_t launch_muon(const NewtonArgs& a, const NsOp* ops, int n_ops, void* ws, hipStream_t stream) {
    const NsShape& s = a.shape;
    if (s.small) return launch_small(a, stream);
    const Space w = space_of(s, ws);
    const int64_t each = s.m * s.n, cols = s.tall ? s.m : s.n;
    float* const u = reinterpret_cast<float*>(w.matrix[M_X1]);
    for (int64_t first = 0; first < s.count; first += s.group) {
        const int count = (int)std::min(s.group, s.count - first);
        MomentumArgs m{};
        m.step = a.step;
        m.step.grads += first * each;
        m.step.m += first * each;
        m.each = each;
        m.nesterov = a.nesterov;
        m.beta = a.beta;
        m.u = u;
        m.partial = w.partial;
        if (a.grad_dtype == ZSMR_BF16) ns_momentum_kernel<ZSMR_BF16><<<dim3(s.parts, count), kThreads, 0, stream>>>(m);
        else ns_momentum_kernel<ZSMR_FP16><<<dim3(s.parts, count), kThreads, 0, stream>>>(m);
        products(a, ops, n_ops, w, u, ZSMR_FP32, cols, each, first, count, stream);
    }
    return hipGetLastError();
}

}  // namespace zsmr
