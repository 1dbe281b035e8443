// gfx950 kernels of the softmax cross entropy of a large output head.
//
//   s = x w^T,  lse_t = log sum_v exp s[t, v],  loss_t = lse_t - s[t, label_t]
//   G = (exp(s - lse) - onehot) * grad,  dx = scale G w,  dw = scale G^T x
//
// All three products are matrix products on MFMA (16x16x32, 16-bit operands,
// fp32 sums).  The logits never reach memory: the forward epilogue reduces a
// tile to one (maximum, sum of exponentials) pair a token, and the backward
// pass computes them again, a piece of the vocabulary at a time, with an
// epilogue that leaves G in 16 bits as the operand of the other two products.
// So a training step does 8 T V H operations where the mathematics needs 6.
// Measured on MI355X, 8,192 tokens, vocabulary 128,256, width 4,096, bf16: logits
// 1.31-1.36 PFLOP/s, with G's epilogue 1.23-1.28, dx 1.37-1.40, dw 1.28-1.32, where
// the library's products of these shapes reach 1.41 (logits), 1.35 (dx) and 1.10
// (dw).  The matrix units are busy for 63-72% of the cycles at a clock that their
// power holds at 1.6-2.0 GHz.
//
// One main loop serves all products: D[m, n] = sum_k A[m, k] B[n, k] over a
// 256 x BN tile, 64 k a step, by 8 waves.  An operand whose k is contiguous in
// memory and one whose k is the row index both go to LDS as they lie there, by
// loads that write LDS directly; the second kind is transposed on the way to
// the registers by the transposing LDS read, so no operand is ever copied to
// another layout.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "zsmr_dev.h"
#include "zsmr_ops_launch.h"
#include "zsmr_xent_plan.h"

#pragma clang fp contract(off)

namespace zsmr {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) void* lds_ptr;

constexpr int kWaves = 8, kThreads = kWaves * 64;

template <int DT>
__device__ __forceinline__ f32x4 mfma(u32x4 a, u32x4 b, f32x4 c) {
    if constexpr (DT == ZSMR_BF16)
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
}

// ---------------------------------------------------------------- operands --
// A matrix in memory as an operand of a product: `rows` of `cols` elements,
// ld elements apart.  OUTER: k is the row index (rows of the tile are k),
// otherwise k runs along a row.
struct Mat {
    const uint16_t* p;
    int64_t ld, rows, cols;
};

// The transposing LDS read of four 16-bit elements.  __restrict__ tells the
// compiler that no load in flight writes what it reads (the waits of the main
// loop see to that); without it, it waits for all of them before each read.
template <typename = void>
__device__ __forceinline__ u32x2 read_transposed(const char* __restrict__ p) {
    return __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4*)(p)));
}

// A tile of R (rows or columns of the product) x BK, in LDS.
//  k along rows: R rows of 128 bytes; the 16-byte chunk c of row r sits in slot
//    c ^ (r & 7), so that the 8 rows a read touches at a time lie in different
//    banks.
//  k outer: BK rows of R elements; the 32-byte unit u of row k sits in slot
//    u ^ f(k), f = k's bits 0, 1 and 3: the transposing read of a wave takes a
//    32-byte unit of 16 rows, which then fall in all banks evenly.
// The loads that fill it read through a buffer descriptor whose bound makes
// rows past the operand's end zero.
template <int R, bool OUTER>
struct Tile {
    static constexpr int kBytes = R * BK * 2;
    static constexpr int kLoads = R / 64;           // of each thread
    uint32_t off[kLoads];                           // byte offsets of its loads from the tile's corner
    const char* base;                               // the tile's corner at the next step
    int64_t left;                                   // bytes from there to the operand's end
    int64_t step;
    int k_left;                                     // k of the operand still to load

    __device__ __forceinline__ static int swizzle(int k) { return ((k & 3) | ((k >> 3 & 1) << 2)) << 1; }

    // at: the tile's first row (or column) of the product; k0: first k
    __device__ __forceinline__ void init(const Mat& m, int64_t at, int64_t k0) {
        const int lane = threadIdx.x % 64, wave = threadIdx.x / 64;
        if constexpr (OUTER) {
            static_assert(!OUTER || R == 128 || R == 256, "a wave's load is whole rows of k");
#pragma unroll
            for (int i = 0; i < kLoads; ++i) {
                const int k = (wave + kWaves * i) * (512 / R) + lane / (R / 8);
                const int chunk = (lane % (R / 8)) ^ swizzle(k);
                // columns past the end are no part of any result, but their
                // addresses must stay inside the operand
                off[i] = at + chunk * 8 < m.cols ? (uint32_t)(k * m.ld * 2 + chunk * 16) : 0x80000000u;
            }
            base = reinterpret_cast<const char*>(m.p + k0 * m.ld + at);
            left = ((m.rows - k0 - 1) * m.ld + (m.cols - at)) * 2;
            step = BK * m.ld * 2;
            k_left = (int)(m.rows - k0);
        } else {
#pragma unroll
            for (int i = 0; i < kLoads; ++i) {
                const int row = (wave + kWaves * i) * 8 + lane / 8;
                const int chunk = (lane % 8) ^ (row & 7);
                off[i] = at + row < m.rows ? (uint32_t)(row * m.ld * 2 + chunk * 16) : 0x80000000u;
            }
            base = reinterpret_cast<const char*>(m.p + at * m.ld + k0);
            left = ((m.rows - at - 1) * m.ld + (m.cols - k0)) * 2;
            step = BK * 2;
            k_left = (int)(m.cols - k0);
        }
    }
    // Start the loads of one step into `to` (kBytes of LDS) and move on; `on`
    // false: the same instructions, which read nothing and write zeros.
    // AUX: 2 for operands that are read once, past the caches.
    template <int AUX>
    __device__ __forceinline__ void load(char* to, bool on) {
        const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
        const int bound = !on || left < 0 ? 0 : left > 0x7fffffff ? 0x7fffffff : (int)left;
        const auto rsrc = __builtin_amdgcn_make_buffer_rsrc(const_cast<char*>(base), 0, bound, 0x00027000);
        // the last step of rows whose length is no multiple of BK: the next
        // row's values must not come in as k
        const int lane = threadIdx.x % 64;
        const bool past = !OUTER && ((lane % 8) ^ (lane / 8)) * 8 >= k_left;
#pragma unroll
        for (int i = 0; i < kLoads; ++i)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc, (lds_ptr)(to + (wave + kWaves * i) * 1024), 16,
                                                     past ? 0x80000000u : off[i], 0, 0, AUX);
        base += step;
        left -= step;
        k_left -= BK;
    }
    // The operand registers of a lane for the 16 rows (columns) from `at` of the
    // tile and k = 32 * kk + 8 * (lane / 16) + 0..7.
    __device__ __forceinline__ static u32x4 read(const char* t, int at, int kk) {
        const int lane = threadIdx.x % 64;
        if constexpr (OUTER) {
            const int k = kk * 32 + lane / 16 * 8 + (lane % 16) / 4;
            const int chunk = (at / 8 + (lane % 4) / 2) ^ swizzle(k);
            const char* p = t + k * (R * 2) + chunk * 16 + (lane & 1) * 8;
            const u32x2 a = read_transposed(p), b = read_transposed(p + 4 * (R * 2));
            u32x4 r;
            r[0] = a[0];
            r[1] = a[1];
            r[2] = b[0];
            r[3] = b[1];
            return r;
        } else {
            const int row = at + lane % 16;
            const int slot = (kk * 4 + lane / 16) ^ (row & 7);
            return *reinterpret_cast<const u32x4*>(t + row * 128 + slot * 16);
        }
    }
};

// Spread a block's LDS reads and loads evenly among its matrix instructions.
template <int READS, int LOADS, int MFMA>
__device__ __forceinline__ void interleave() {
    constexpr int kOps = READS + LOADS, kEach = kOps < MFMA ? MFMA / kOps : 1;
    constexpr int kRounds = kOps < MFMA ? kOps : MFMA;
#pragma unroll
    for (int i = 0; i < kRounds; ++i) {
        if (i < LOADS) __builtin_amdgcn_sched_group_barrier(0x020, 1, 0);      // vector memory read
        else __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);                // LDS read
        __builtin_amdgcn_sched_group_barrier(0x008, kEach, 0);                 // matrix
    }
}

// vmcnt(n) and lgkmcnt(0)
#define ZSMR_WAIT(n) __builtin_amdgcn_s_waitcnt(((n) & 15) | 0x70 | ((n) >> 4 << 14))

// ------------------------------------------------------------------ product --
struct Product {
    Mat a, b;
    int64_t k;                      // of the product
    int32_t m_tiles, n_tiles, splits, k_split;      // k_split: k of one split, a multiple of BK
    // epilogues
    int64_t v0, vocab, tokens, width;
    const void* labels;
    int32_t id_bytes;
    float2* stats;                  // E_STATS: [part][token]
    float* target;                  // E_STATS: [token]
    const float* lse;               // E_GRAD
    const float* grad;              // E_GRAD: [token] or NULL
    const float* mul;               // {factor of G, factor of the results}, or NULL:
    float g_mul, out_mul;           // these, the latter
    const float* scale;             // times this (NULL: 1)
    uint16_t* g;                    // E_GRAD: [token][ldg]
    int64_t ldg;
    float* sum;                     // E_DX: [split][token][lds], fp32 between pieces
    int64_t lds;
    int32_t sum_in, sum_out;        // E_DX: add what sum holds; leave the result there
    uint16_t* out;                  // E_DX, E_DW
    int64_t ldo;
    int32_t accumulate;             // E_DW
};

__device__ __forceinline__ float out_mul(const Product& p) {
    return p.mul ? p.mul[1] : p.scale ? p.out_mul * *p.scale : p.out_mul;
}
// Exponentials are powers of two of arguments times log2 e, which one fused
// multiply-add moves by the maximum (or by lse): 2^(s log2 e - shift).
constexpr float kLog2e = 1.44269504f, kLn2 = 0.69314718f;
template <typename = void>
__device__ __forceinline__ float exp2_of(float s, float shift) {
    return __builtin_amdgcn_exp2f(__builtin_fmaf(s, kLog2e, -shift));
}
// The shift of a maximum, which is held to +-2.3e38 so that it stays finite: rows
// below that alone (or none at all, -inf) add up to zero and one above it makes the
// sum infinite, where shifts of -+inf would give NaN or pass over it.
template <typename = void>
__device__ __forceinline__ float shift_of(float top) {
    return __builtin_amdgcn_fmed3f(top, -2.3e38f, 2.3e38f) * kLog2e;
}
// Two parts of a softmax: (shift, sum of the powers relative to it).
__device__ __forceinline__ float2 join_parts(float2 a, float2 b) {
    const float top = fmaxf(a.x, b.x);
    return make_float2(top, (a.y == 0.f ? 0.f : a.y * __builtin_amdgcn_exp2f(a.x - top)) +
                                (b.y == 0.f ? 0.f : b.y * __builtin_amdgcn_exp2f(b.x - top)));
}

// Column n of the result, rows m..m+3: 4 consecutive elements for a lane.
template <int DT>
__device__ __forceinline__ void put4(uint16_t* p, int64_t at, int64_t width, f32x4 f, bool add) {
    if (at + 4 <= width) {
        if (add) {
            const u16x4 o = *reinterpret_cast<const u16x4_any*>(p + at);
#pragma unroll
            for (int r = 0; r < 4; ++r) f[r] += widen16<DT>(o[r]);
        }
        u16x4 h;
#pragma unroll
        for (int r = 0; r < 4; ++r) h[r] = narrow16<DT>(f[r]);
        *reinterpret_cast<u16x4_any*>(p + at) = h;
    } else {
#pragma unroll
        for (int r = 0; r < 4; ++r)
            if (at + r < width) p[at + r] = narrow16<DT>(add ? f[r] + widen16<DT>(p[at + r]) : f[r]);
    }
}

// ONCE: no other workgroup reads the same part of A (one tile holds all of n).
template <int DT, int EPI, int BN, int WM, int STAGES, bool ONCE>
__global__ __launch_bounds__(kThreads) void product_kernel(Product p) {
#if defined(__HIP_DEVICE_COMPILE__)     // the scheduling hints have no host form
    constexpr bool A_OUTER = EPI == E_DX || EPI == E_DW, B_OUTER = EPI == E_DW;
    // Weights that are read once go past the caches: 1.05 GB took 160 us on MI355X
    // (16 tokens), through them 177.
    constexpr int kStream = ONCE ? 2 : 0;
    constexpr int WN = kWaves / WM, TM = BM / WM / 16, TN = BN / WN / 16;
    typedef Tile<BM, A_OUTER> TA;
    typedef Tile<BN, B_OUTER> TB;
    constexpr int kLoads = TA::kLoads + TB::kLoads, kStage = TA::kBytes + TB::kBytes;
    __shared__ __attribute__((aligned(1024))) char smem[STAGES * kStage];

    // Consecutive workgroups go to the eight XCDs in turn; each XCD takes a
    // contiguous run of tiles, in groups of 8 in m, so that the tiles it works
    // on at a time share operands in its L2.
    const int tiles = p.m_tiles * p.n_tiles * p.splits;
    const int xcd = blockIdx.x % 8, q = tiles / 8, rem = tiles % 8;
    int tile = xcd * q + min(xcd, rem) + (int)blockIdx.x / 8;
    const int split = tile / (p.m_tiles * p.n_tiles);
    tile -= split * p.m_tiles * p.n_tiles;
    constexpr int kGroup = 8;
    const int group = tile / (kGroup * p.n_tiles), in_group = tile - group * kGroup * p.n_tiles;
    const int height = min(kGroup, p.m_tiles - group * kGroup);
    const int mt = group * kGroup + in_group % height, nt = in_group / height;

    const int64_t k0 = (int64_t)split * p.k_split;
    const int64_t kn = p.k - k0 < p.k_split ? p.k - k0 : p.k_split;
    const int steps = (int)((kn + BK - 1) / BK);

    TA ta;
    TB tb;
    ta.init(p.a, (int64_t)mt * BM, k0);
    tb.init(p.b, (int64_t)nt * BN, k0);

    const int lane = threadIdx.x % 64, wave = threadIdx.x / 64;
    const int wm = wave % WM, wn = wave / WM;
    f32x4 acc[TM][TN];
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j) acc[i][j] = 0.f;

    // STAGES of LDS and two sets of operand registers: the second half's
    // operands of a step (k 32..63) are read while its first half is
    // multiplied, the next step's first half while the second is.  The barrier
    // between the halves is the only one of a step: behind it every wave has the
    // stage's operands in registers, so its LDS is refilled (STAGES steps
    // ahead), and the next step's loads, which had STAGES - 1 steps to arrive,
    // are there.
    constexpr int kReads = TM * (A_OUTER ? 2 : 1) + TN * (B_OUTER ? 2 : 1), kMfma = TM * TN;
    u32x4 a0[TM], b0[TN], a1[TM], b1[TN];
    auto read = [&](u32x4* a, u32x4* b, const char* stage, int kk) {
#pragma unroll
        for (int j = 0; j < TN; ++j) b[j] = TB::read(stage + TA::kBytes, (wn * TN + j) * 16, kk);
#pragma unroll
        for (int i = 0; i < TM; ++i) a[i] = TA::read(stage, (wm * TM + i) * 16, kk);
    };
    auto multiply = [&](const u32x4* a, const u32x4* b) {
#pragma unroll
        for (int i = 0; i < TM; ++i)
#pragma unroll
            for (int j = 0; j < TN; ++j) acc[i][j] = mfma<DT>(a[i], b[j], acc[i][j]);
    };
    if (steps > 0) {
#pragma unroll
        for (int s = 0; s < STAGES; ++s) {
            ta.template load<kStream>(smem + s * kStage, s < steps);
            tb.template load<0>(smem + s * kStage + TA::kBytes, s < steps);
        }
        ZSMR_WAIT((STAGES - 1) * kLoads);       // the first step's
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
        read(a0, b0, smem, 0);
    }
    char* cur = smem;
    for (int s = 0; s < steps; ++s) {
        char* next = cur == smem + (STAGES - 1) * kStage ? smem : cur + kStage;
        read(a1, b1, cur, 1);
        multiply(a0, b0);
        interleave<kReads, 0, kMfma>();
        ZSMR_WAIT((STAGES - 2) * kLoads);
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
        ta.template load<kStream>(cur, s + STAGES < steps);
        tb.template load<0>(cur + TA::kBytes, s + STAGES < steps);
        read(a0, b0, next, 0);
        multiply(a1, b1);
        interleave<kReads, kLoads, kMfma>();
        cur = next;
    }
    ZSMR_WAIT(0);           // no load may still be on its way to this LDS when the workgroup ends

    // acc[i][j][r] is D at m = m0 + 16 i + r, n = n0 + 16 j
    const int64_t m0 = (int64_t)mt * BM + wm * TM * 16 + lane / 16 * 4;
    const int64_t n0 = (int64_t)nt * BN + wn * TN * 16 + lane % 16;
    // The rows that a lane holds as 16 i + r, up to `rows`, belong to the
    // vocabulary; only the last tile's waves have fewer than all.
    const int64_t left = p.vocab - p.v0 - m0;
    const int rows = left > TM * 16 ? TM * 16 : (int)left;
    const bool whole = p.vocab - p.v0 - ((int64_t)mt * BM + wm * TM * 16) >= TM * 16;       // of the wave
    // 16-bit results leave through LDS, as [n][m] where the main loop's tiles
    // were (chunk c of row n in slot c ^ (n % 32)): a lane holds 8 bytes of 16
    // different rows of memory, and stored like that each write is a quarter of
    // a line.  From LDS a wave stores two rows of 512 bytes at a time.  Measured on
    // MI355X, through LDS against stored as they are held, loss and gradients: 129
    // tokens over 50,257 x 768 128 and 135 us, 8,192 tokens 2,494 and 2,498, over
    // 128,256 x 4,096 25.87 and 25.98 ms.
    auto stage = [&](int i, int j, u16x4 h) {
        const int n = (wn * TN + j) * 16 + lane % 16, c = (wm * TM + i) * 2 + lane / 32;
        *reinterpret_cast<u16x4*>(smem + n * (BM * 2) + (c ^ (n & 31)) * 16 + (lane / 16 & 1) * 8) = h;
    };
    // rows: of the tile; cols: from its first on
    auto store_tile = [&](uint16_t* out, int64_t ld, int64_t rows, int64_t cols) {
        __syncthreads();
#pragma unroll 4
        for (int q = threadIdx.x; q < BN * (BM / 8); q += kThreads) {
            const int n = q / (BM / 8), c = q % (BM / 8);
            if (n >= rows || c * 8 >= cols) continue;
            const u16x8 h = *reinterpret_cast<const u16x8*>(smem + n * (BM * 2) + (c ^ (n & 31)) * 16);
            uint16_t* o = out + n * ld + c * 8;
            if (c * 8 + 8 <= cols) {
                *reinterpret_cast<u16x8_any*>(o) = h;
            } else {
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    if (c * 8 + k < cols) o[k] = h[k];
            }
        }
    };
    auto narrow4 = [&](f32x4 f) {
        u16x4 h;
#pragma unroll
        for (int r = 0; r < 4; ++r) h[r] = narrow16<DT>(f[r]);
        return h;
    };
    __syncthreads();        // every wave's last loads are in
    if constexpr (EPI == E_STATS) {
        // the waves' parts, where the main loop's tiles were
        float2* part = reinterpret_cast<float2*>(smem);
#pragma unroll
        for (int j = 0; j < TN; ++j) {
            const int64_t t = n0 + j * 16;
            const int32_t label = t < p.tokens ? token_at(p.labels, p.id_bytes, t, p.vocab) : -1;
            // the label's row among the lane's
            const int64_t far = label - p.v0 - m0;
            const int mine = label >= 0 && far >= 0 && far < rows && (far & 12) == 0 ? (int)far : -1;
            if (__any(mine >= 0)) {
#pragma unroll
                for (int i = 0; i < TM; ++i)
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        if (i * 16 + r == mine) p.target[t] = acc[i][j][r];
            }
            if (!whole) {
#pragma unroll
                for (int i = 0; i < TM; ++i)
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        if (i * 16 + r >= rows) acc[i][j][r] = -INFINITY;
            }
            float top = acc[0][j][0];
#pragma unroll
            for (int i = 0; i < TM; ++i)
#pragma unroll
                for (int r = 0; r < 4; ++r) top = fmaxf(top, acc[i][j][r]);
            // the four lane groups hold other rows of the same column
#pragma unroll
            for (int d = 16; d < 64; d <<= 1) top = fmaxf(top, __shfl_xor(top, d));
            const float shift = shift_of(top);
            float sum = 0.f;
#pragma unroll
            for (int i = 0; i < TM; ++i)
#pragma unroll
                for (int r = 0; r < 4; ++r) sum += exp2_of(acc[i][j][r], shift);
#pragma unroll
            for (int d = 16; d < 64; d <<= 1) sum += __shfl_xor(sum, d);
            if (lane < 16) part[wm * BN + (wn * TN + j) * 16 + lane] = make_float2(sum == 0.f ? -INFINITY : shift, sum);
        }
        __syncthreads();
        const int64_t t = (int64_t)nt * BN + threadIdx.x;
        if (threadIdx.x < BN && t < p.tokens) {
            float2 all = part[threadIdx.x];
#pragma unroll
            for (int i = 1; i < WM; ++i) all = join_parts(all, part[i * BN + threadIdx.x]);
            p.stats[(p.v0 / BM + mt) * p.tokens + t] = all;
        }
    } else if constexpr (EPI == E_GRAD) {
        const float mul = p.mul ? p.mul[0] : p.g_mul;
#pragma unroll
        for (int j = 0; j < TN; ++j) {
            const int64_t t = n0 + j * 16;
            if (t >= p.tokens) continue;
            const int32_t label = token_at(p.labels, p.id_bytes, t, p.vocab);
            const int64_t far = label - p.v0 - m0;
            const int mine = label >= 0 && far >= 0 && far < rows && (far & 12) == 0 ? (int)far : -1;
            const bool none = label < 0;
            const float shift = p.lse[t] * kLog2e, weight = (p.grad ? p.grad[t] : 1.f) * mul;
            const bool has = __any(mine >= 0);
#pragma unroll
            for (int i = 0; i < TM; ++i) {
                f32x4 f;
#pragma unroll
                for (int r = 0; r < 4; ++r) f[r] = exp2_of(acc[i][j][r], shift);
                if (has) {
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        if (i * 16 + r == mine) f[r] -= 1.f;
                }
                u16x4 h = narrow4(f * weight);
                if (none) h = 0;
                if (!whole) {
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        if (i * 16 + r >= rows) h[r] = 0;
                }
                stage(i, j, h);
            }
        }
        // ldg is a multiple of the tile: past the vocabulary there are zeros
        store_tile(p.g + (int64_t)nt * BN * p.ldg + (int64_t)mt * BM, p.ldg, p.tokens - (int64_t)nt * BN, BM);
    } else if (EPI == E_DX && p.sum_out) {
#pragma unroll
        for (int j = 0; j < TN; ++j) {
            const int64_t t = n0 + j * 16;
            if (t >= p.tokens) continue;
            float* s = p.sum + ((int64_t)split * p.tokens + t) * p.lds;
#pragma unroll
            for (int i = 0; i < TM; ++i) {
                const int64_t h = m0 + i * 16;
                if (h >= p.width) continue;
                f32x4 f = acc[i][j];
                if (p.sum_in) f += *reinterpret_cast<const f32x4*>(s + h);
                *reinterpret_cast<f32x4*>(s + h) = f;
            }
        }
    } else {
        // dx's last piece, or dw: rows of the result are columns of the tile
        const float mul = out_mul(p);
        const int64_t rows = EPI == E_DX ? p.tokens : p.vocab - p.v0;
        uint16_t* out = EPI == E_DX ? p.out : p.out + p.v0 * p.ldo;
        const bool add = EPI == E_DW && p.accumulate;
#pragma unroll
        for (int j = 0; j < TN; ++j) {
            const int64_t n = n0 + j * 16;
#pragma unroll
            for (int i = 0; i < TM; ++i) {
                const int64_t h = m0 + i * 16;
                f32x4 f = acc[i][j];
                if (EPI == E_DX && p.sum_in && n < rows && h < p.width)
                    f += *reinterpret_cast<const f32x4*>(p.sum + n * p.lds + h);
                // what is added to has to be added before the one rounding
                if (add) {
                    if (n < rows && h < p.width) put4<DT>(out + n * p.ldo, h, p.width, f * mul, true);
                } else {
                    stage(i, j, narrow4(f * mul));
                }
            }
        }
        const int64_t first = (int64_t)nt * BN, col = (int64_t)mt * BM;
        if (!add) store_tile(out + first * p.ldo + col, p.ldo, rows - first, p.width - col);
    }
#endif
}

// ------------------------------------------------------------ small kernels --
__device__ __forceinline__ void put_summary(double sum, double count, float* summary) {
    summary[0] = count > 0 ? (float)(sum / count) : 0.f;
    summary[1] = count > 0 ? (float)(1.0 / count) : 0.f;
    summary[2] = (float)count;
}

// Join the parts of each token's softmax: `lanes` tokens of a workgroup, its groups
// of lanes share the parts.  A lone workgroup
// has all tokens and leaves the summary too.
constexpr int kStatsThreads = 1024;
__global__ __launch_bounds__(kStatsThreads) void stats_kernel(const float2* stats, const float* target,
                                                              const void* labels, int32_t id_bytes,
                                                              int64_t tokens, int64_t vocab, int32_t parts,
                                                              int32_t lanes, float* loss, float* lse, float* summary) {
    __shared__ float2 part[kStatsThreads];
    const int lane = threadIdx.x % lanes, group = threadIdx.x / lanes, groups = kStatsThreads / lanes;
    const int64_t t = (int64_t)blockIdx.x * lanes + lane;
    float2 s = make_float2(-INFINITY, 0.f);
    if (t < tokens && group < groups) {
        constexpr int kAhead = 16;
        for (int i = group; i < parts; i += groups * kAhead) {
            float2 p[kAhead];
#pragma unroll
            for (int k = 0; k < kAhead; ++k)
                p[k] = i + k * groups < parts ? stats[(int64_t)(i + k * groups) * tokens + t] : make_float2(-INFINITY, 0.f);
#pragma unroll
            for (int k = 0; k < kAhead; ++k) s = join_parts(s, p[k]);
        }
    }
    part[threadIdx.x] = s;
    __syncthreads();
    for (int left = groups; left > 1;) {
        const int half = (left + 1) / 2;
        if (group + half < left) part[threadIdx.x] = s = join_parts(s, part[threadIdx.x + half * lanes]);
        __syncthreads();
        left = half;
    }
    const bool on = group == 0 && t < tokens;
    const bool counts = on && token_at(labels, id_bytes, t, vocab) >= 0;
    float out = 0.f;
    if (on) {
        const float l = kLn2 * (s.x + log2f(s.y));
        if (counts) out = l - target[t];
        lse[t] = l;
        loss[t] = out;
    }
    if (gridDim.x > 1) return;
    const double sum = block_sum<kStatsThreads>(out);
    const int count = __syncthreads_count(counts);
    if (threadIdx.x == 0) put_summary(sum, count, summary);
}

constexpr int kMeanThreads = 1024;
__global__ __launch_bounds__(kMeanThreads) void mean_kernel(const float* loss, const void* labels,
                                                            int32_t id_bytes, int64_t tokens,
                                                            int64_t vocab, float* summary) {
    double sum = 0, count = 0;
    for (int64_t t = threadIdx.x; t < tokens; t += kMeanThreads) {
        sum += loss[t];
        count += token_at(labels, id_bytes, t, vocab) >= 0 ? 1.0 : 0.0;
    }
    sum = block_sum<kMeanThreads>(sum);
    __syncthreads();
    count = block_sum<kMeanThreads>(count);
    if (threadIdx.x == 0) put_summary(sum, count, summary);
}

// What G is multiplied by before it is rounded to 16 bits, a power of two that
// the results are divided by again.  bf16 has fp32's range and needs none.  fp16
// has all its bits down to 2^-14 only, and most probabilities of a large
// vocabulary are below that: there |G| <= max |grad| is moved to [2^14, 2^15),
// just below fp16's largest value.  The maximum is over the tokens that count:
// padding has no gradient, whatever its weight.
constexpr float kFp16Mul = 16384.f;
constexpr int kMulThreads = 1024;
__global__ __launch_bounds__(kMulThreads) void mul_kernel(const float* grad, const void* labels, int32_t id_bytes,
                                                          int64_t tokens, int64_t vocab, const float* scale,
                                                          float* mul) {
    __shared__ float part[kMulThreads / 64];
    float top = 0.f;
    for (int64_t t = threadIdx.x; t < tokens; t += kMulThreads) {
        const float g = fabsf(grad[t]);
        if (g < INFINITY && token_at(labels, id_bytes, t, vocab) >= 0) top = fmaxf(top, g);
    }
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor(top, d));
    if (threadIdx.x % 64 == 0) part[threadIdx.x / 64] = top;
    __syncthreads();
    if (threadIdx.x != 0) return;
    for (int i = 0; i < kMulThreads / 64; ++i) top = fmaxf(top, part[i]);
    // an exponent that neither factor can leave fp32 with
    const int e = top > 0.f ? max(-60, min(60, 14 - ilogbf(top))) : 0;
    mul[0] = ldexpf(1.f, e);
    mul[1] = ldexpf(scale ? *scale : 1.f, -e);
}

// Rows of any length, stride and alignment to rows of a multiple of 8 elements,
// zero-filled: what the products' 16-byte loads need.  With labels, rows of
// tokens that do not count become zeros.
__global__ __launch_bounds__(256) void pack_kernel(const uint16_t* src, int64_t stride, int64_t rows,
                                                   int64_t width, uint16_t* dst, int64_t ld, const void* labels,
                                                   int32_t id_bytes, int64_t vocab) {
    const int64_t vecs = ld / 8, i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const int64_t row = i / vecs, j = (i - row * vecs) * 8;
    if (row >= rows) return;
    u16x8 h = 0;
    if (labels && token_at(labels, id_bytes, row, vocab) < 0) {
    } else if (j + 8 <= width) {
        h = *reinterpret_cast<const u16x8_any*>(src + row * stride + j);
    } else {
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (j + k < width) h[k] = src[row * stride + j + k];
    }
    *reinterpret_cast<u16x8*>(dst + row * ld + j) = h;
}

// dx = rne16(mul * sum over the splits, in order)
template <int DT>
__global__ __launch_bounds__(256) void splits_kernel(Product p) {
    const int64_t vecs = p.lds / 4, i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const int64_t t = i / vecs, h = (i - t * vecs) * 4;
    if (t >= p.tokens) return;
    f32x4 f = 0.f;
    constexpr int kAhead = 8;
    for (int s = 0; s < p.splits; s += kAhead) {
        f32x4 x[kAhead];
#pragma unroll
        for (int k = 0; k < kAhead; ++k)
            if (s + k < p.splits) x[k] = *reinterpret_cast<const f32x4*>(p.sum + ((int64_t)(s + k) * p.tokens + t) * p.lds + h);
#pragma unroll
        for (int k = 0; k < kAhead; ++k)
            if (s + k < p.splits) f += x[k];
    }
    put4<DT>(p.out + t * p.ldo, h, p.width, f * out_mul(p), false);
}

// --------------------------------------------------------------------- host --
struct Space {
    float2* stats;
    float *target, *mul, *sum;
    uint16_t *x, *w, *g;
};
Space space_of(void* ws, int64_t tokens, int64_t vocab, int64_t width, bool backward) {
    const XentSpace at = xent_space(tokens, vocab, width, backward);
    char* const p = static_cast<char*>(ws);
    Space s{};
    s.stats = reinterpret_cast<float2*>(p + at.stats);
    s.target = reinterpret_cast<float*>(p + at.target);
    s.x = reinterpret_cast<uint16_t*>(p + at.x);
    s.w = reinterpret_cast<uint16_t*>(p + at.w);
    s.mul = reinterpret_cast<float*>(p + at.mul);
    s.g = reinterpret_cast<uint16_t*>(p + at.g);
    s.sum = reinterpret_cast<float*>(p + at.sum);
    return s;
}

template <int DT, int EPI>
void launch_product(const Product& p, const ProductShape& shape, hipStream_t stream) {
    const unsigned grid = (unsigned)shape.grid();
    if constexpr (EPI == E_DW) {
        if (shape.tile == 128) product_kernel<DT, EPI, 128, 4, 3, false><<<grid, kThreads, 0, stream>>>(p);
        else product_kernel<DT, EPI, 256, 2, 2, false><<<grid, kThreads, 0, stream>>>(p);
    } else if (shape.tile == 64) {
        if (shape.once) product_kernel<DT, EPI, 64, 8, 2, true><<<grid, kThreads, 0, stream>>>(p);
        else product_kernel<DT, EPI, 64, 8, 4, false><<<grid, kThreads, 0, stream>>>(p);
    } else if (shape.tile == 128) {
        if (shape.once) product_kernel<DT, EPI, 128, 4, 3, true><<<grid, kThreads, 0, stream>>>(p);
        else product_kernel<DT, EPI, 128, 4, 3, false><<<grid, kThreads, 0, stream>>>(p);
    } else if (shape.tile == 192) {
        product_kernel<DT, EPI, 192, 2, 2, false><<<grid, kThreads, 0, stream>>>(p);
    } else {
        product_kernel<DT, EPI, 256, 2, 2, false><<<grid, kThreads, 0, stream>>>(p);
    }
}

bool loads16(const uint16_t* p, int64_t stride, int64_t width) {
    return reinterpret_cast<uintptr_t>(p) % 16 == 0 && stride % 8 == 0 && width % 8 == 0;
}

// The operands of the products over the vocabulary from v0 on.  Operands that
// 16-byte loads cannot read are packed first: x once, w piece by piece.
struct Operands {
    Mat x, w;
};
// counted: dw is asked for.  It adds G's rows times x's, and zero times what is not
// finite is NaN, so tokens that do not count must not bring their x: it is packed
// with zeros there, whatever its alignment.  On MI355X that takes 2 us of the 130
// of 129 tokens over 50,257 x 768, 8 of 2,490 with 8,192 tokens.
void pack_x(const XentArgs& a, const Space& s, bool counted, Operands* o, hipStream_t stream) {
    o->x = Mat{a.x, a.x_stride, a.tokens, a.width};
    if (!a.tokens || (!counted && loads16(a.x, a.x_stride, a.width))) return;
    const int64_t ld = ceil_to(a.width, 8);
    launch_rows(a.tokens, ld / 8, [&](int64_t first, int64_t count) {
        const char* labels = counted ? static_cast<const char*>(a.labels) + first * a.id_bytes : nullptr;
        pack_kernel<<<(unsigned)tiles_of(count * (ld / 8), 256), 256, 0, stream>>>(
            a.x + first * a.x_stride, a.x_stride, count, a.width, s.x + first * ld, ld, labels, a.id_bytes, a.vocab);
    });
    o->x = Mat{s.x, ld, a.tokens, ld};
}
void pack_w(const XentArgs& a, const Space& s, int64_t v0, int64_t rows, Operands* o, hipStream_t stream) {
    const uint16_t* w = a.w + v0 * a.w_stride;
    o->w = Mat{w, a.w_stride, rows, a.width};
    if (loads16(a.w, a.w_stride, a.width)) return;
    const int64_t ld = ceil_to(a.width, 8);
    launch_rows(rows, ld / 8, [&](int64_t first, int64_t count) {
        pack_kernel<<<(unsigned)tiles_of(count * (ld / 8), 256), 256, 0, stream>>>(
            w + first * a.w_stride, a.w_stride, count, a.width, s.w + first * ld, ld, nullptr, 0, 0);
    });
    o->w = Mat{s.w, ld, rows, ld};
}

// A product's sizes; its operands come next.
Product product_of(const XentArgs& a, const ProductShape& shape) {
    Product p{};
    p.k = shape.k;
    p.m_tiles = (int32_t)shape.m_tiles;
    p.n_tiles = (int32_t)shape.n_tiles;
    p.splits = shape.splits;
    p.k_split = (int32_t)shape.k_split;
    p.v0 = shape.v0;
    p.vocab = a.vocab;
    p.tokens = a.tokens;
    p.width = a.width;
    p.labels = a.labels;
    p.id_bytes = a.id_bytes;
    return p;
}
// The operands of the logits.
void set_logits(Product* p, const Operands& o) {
    p->a = o.w;
    p->b = o.x;
    p->a.cols = p->b.cols = p->k;
}

template <int DT>
hipError_t forward(const XentArgs& a, void* ws, hipStream_t stream) {
    const Space s = space_of(ws, a.tokens, a.vocab, a.width, false);
    if (a.tokens) {
        Operands o;
        pack_x(a, s, false, &o, stream);
        forward_products(a.tokens, a.vocab, a.width, !loads16(a.w, a.w_stride, a.width), [&](const ProductShape& shape) {
            pack_w(a, s, shape.v0, shape.rows, &o, stream);
            Product p = product_of(a, shape);
            set_logits(&p, o);
            p.stats = s.stats;
            p.target = s.target;
            launch_product<DT, E_STATS>(p, shape, stream);
        });
        const int32_t parts = (int32_t)tiles_of(a.vocab, BM);
        // up to 256 tokens in one workgroup, which saves the launch of the mean
        const int lanes = a.tokens <= 256 ? (int)ceil_to(a.tokens, 16) : 64;
        const unsigned grid = (unsigned)tiles_of(a.tokens, lanes);
        stats_kernel<<<grid, kStatsThreads, 0, stream>>>(s.stats, s.target, a.labels, a.id_bytes, a.tokens,
                                                         a.vocab, parts, lanes, a.loss, a.lse, a.summary);
        if (grid == 1) return hipGetLastError();
    }
    mean_kernel<<<1, kMeanThreads, 0, stream>>>(a.loss, a.labels, a.id_bytes, a.tokens, a.vocab, a.summary);
    return hipGetLastError();
}

template <int DT>
hipError_t backward(const XentArgs& a, void* ws, hipStream_t stream) {
    const Space s = space_of(ws, a.tokens, a.vocab, a.width, true);
    const bool packed = !loads16(a.w, a.w_stride, a.width);
    const int64_t piece = packed ? packed_piece(a.tokens, a.vocab, a.width) : piece_of(a.tokens, a.vocab, a.width);
    const bool fp16 = DT == ZSMR_FP16, weighted = fp16 && a.grad;
    if (weighted) mul_kernel<<<1, kMulThreads, 0, stream>>>(a.grad, a.labels, a.id_bytes, a.tokens, a.vocab, a.scale, s.mul);
    Operands o;
    pack_x(a, s, a.dw, &o, stream);
    backward_products(a.tokens, a.vocab, a.width, packed, a.dx, a.dw, [&](const ProductShape& shape) {
        Product p = product_of(a, shape);
        p.mul = weighted ? s.mul : nullptr;
        p.g_mul = fp16 ? kFp16Mul : 1.f;
        p.out_mul = fp16 ? 1.f / kFp16Mul : 1.f;
        p.scale = a.scale;
        if (shape.epi == E_GRAD) {
            pack_w(a, s, shape.v0, shape.rows, &o, stream);
            set_logits(&p, o);
            p.lse = a.lse;
            p.grad = a.grad;
            p.g = s.g;
            p.ldg = piece;
            launch_product<DT, E_GRAD>(p, shape, stream);
            return;
        }
        p.b = Mat{s.g, piece, a.tokens, ceil_to(shape.rows, 8)};       // G is zero past the vocabulary
        if (shape.epi == E_DX) {
            p.a = o.w;
            p.sum = s.sum;
            p.lds = ceil_to(a.width, 4);
            p.sum_in = shape.sum_in;
            p.sum_out = shape.sum_out;
            p.out = a.dx;
            p.ldo = a.dx_stride;
            launch_product<DT, E_DX>(p, shape, stream);
            if (shape.splits > 1 && shape.v0 + piece >= a.vocab)
                splits_kernel<DT><<<(unsigned)tiles_of(a.tokens * (p.lds / 4), 256), 256, 0, stream>>>(p);
        } else {
            p.a = o.x;
            p.out = a.dw;
            p.ldo = a.dw_stride;
            p.accumulate = a.accumulate;
            launch_product<DT, E_DW>(p, shape, stream);
        }
    });
    return hipGetLastError();
}

}  // namespace

int64_t xent_bytes(int64_t tokens, int64_t vocab, int64_t width, bool backward) {
    return xent_space(tokens, vocab, width, backward).bytes;
}

hipError_t launch_xent_forward(const XentArgs& a, void* ws, hipStream_t stream) {
    return a.dtype == ZSMR_BF16 ? forward<ZSMR_BF16>(a, ws, stream) : forward<ZSMR_FP16>(a, ws, stream);
}
hipError_t launch_xent_backward(const XentArgs& a, void* ws, hipStream_t stream) {
    return a.dtype == ZSMR_BF16 ? backward<ZSMR_BF16>(a, ws, stream) : backward<ZSMR_FP16>(a, ws, stream);
}

}  // namespace zsmr
