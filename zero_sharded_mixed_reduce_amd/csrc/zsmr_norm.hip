// gfx950 kernels of the global gradient norm, of clipping and of the clipped
// shard step.
//
//   total = sum g^2,  norm = sqrt(total),  coef = min(1, max_norm / (norm + eps))
//
// All of it is bound by HBM.  Squares are taken and summed in fp64: the square
// of an fp32 value is exact there, and neither a large nor a tiny gradient
// leaves the range.  Each workgroup leaves one partial sum and a last small
// launch adds them in order, so the result does not depend on timing.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "zsmr_dev.h"
#include "zsmr_ops_launch.h"

#pragma clang fp contract(off)

namespace zsmr {
namespace {

constexpr int kThreads = 256;
constexpr int kSumsqGrid = 2048;

// The item whose chunks hold chunk b (uniform over the workgroup).
template <typename A>
__device__ __forceinline__ int item_of(const A& a, int b) {
    int lo = 0, hi = a.count - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) / 2;
        if (a.it[mid].chunk0 <= b) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

// A lane reads 16 bytes at a time, so that an instruction covers one contiguous
// KB: past the caches 6.5-6.7 TB/s on MI355X for 498 MB, through them 5.7-6.0.
template <int DT, bool KEEP>
__device__ __forceinline__ double chunk_sumsq(const void* p, int64_t e0, int64_t e1) {
    constexpr int V = kVec<DT>;
    double s0 = 0, s1 = 0;
    const int64_t body = e0 + (e1 - e0) / V * V;
#pragma unroll 4
    for (int64_t e = e0 + threadIdx.x * V; e < body; e += kThreads * V) {
        const Vec<DT> v = load16<DT, KEEP>(p, e);
#pragma unroll
        for (int i = 0; i < V; i += 2) {
            s0 = __builtin_fma((double)v.f[i], (double)v.f[i], s0);
            s1 = __builtin_fma((double)v.f[i + 1], (double)v.f[i + 1], s1);
        }
    }
    const int64_t e = body + threadIdx.x;
    if (e < e1) {
        const double f = load1<DT>(p, e);
        s0 = __builtin_fma(f, f, s0);
    }
    return s0 + s1;
}
template <int DT>
__device__ __forceinline__ double chunk_sumsq(const void* p, int64_t e0, int64_t e1, bool keep) {
    return keep ? chunk_sumsq<DT, true>(p, e0, e1) : chunk_sumsq<DT, false>(p, e0, e1);
}

// The norm reads the list from its start and clipping reads it from its end.
// The last kKeep chunks (118 MB of 16 bits, 236 MB of fp32) go through the caches
// both times, so that clipping finds them in the 256 MB Infinity Cache; the
// others past them, where HBM reads run faster.  Measured on MI355X, 498 MB of
// fp32, norm + flatten: all through the caches 238 us, none 218, 3,000 chunks
// 216, 3,600 212.  A list of more than kNormBatch tensors is several launches of the
// norm, and each keeps its own last chunks: 320 tensors of the same size 234 us,
// 640 of 249M bf16 in all 316, where keeping those of the whole list took 237 and 326.
constexpr int kKeep = 3600;

// A workgroup takes every gridDim.x-th chunk and leaves one sum.
__global__ __launch_bounds__(kThreads) void sumsq_kernel(NormArgs a, double* partial) {
    double s = 0;
    for (int b = blockIdx.x; b < a.chunks; b += gridDim.x) {
        const int k = item_of(a, b);
        const bool keep = b >= a.chunks - kKeep;
        const void* p = a.it[k].p;
        const int64_t e0 = (int64_t)(b - a.it[k].chunk0) * a.chunk, n = a.it[k].n;
        const int64_t e1 = e0 + a.chunk < n ? e0 + a.chunk : n;
        if (a.it[k].dtype == ZSMR_FP32) s += chunk_sumsq<ZSMR_FP32>(p, e0, e1, keep);
        else if (a.it[k].dtype == ZSMR_BF16) s += chunk_sumsq<ZSMR_BF16>(p, e0, e1, keep);
        else s += chunk_sumsq<ZSMR_FP16>(p, e0, e1, keep);
    }
    s = block_sum<kThreads>(s);
    if (threadIdx.x == 0) partial[blockIdx.x] = s;
}

template <int THREADS>
__global__ __launch_bounds__(THREADS) void join_kernel(const double* partial, int64_t n, double* sumsq,
                                                       double max_norm, double eps, float* norm_coef) {
    double s = 0;
#pragma unroll 8
    for (int64_t i = threadIdx.x; i < n; i += THREADS) s += partial[i];
    s = block_sum<THREADS>(s);
    if (threadIdx.x != 0) return;
    if (sumsq) *sumsq = s;
    if (norm_coef) {
        const double norm = sqrt(s), c = max_norm / (norm + eps);
        norm_coef[0] = (float)norm;
        norm_coef[1] = c > 1.0 ? 1.0f : (float)c;       // NaN stays
    }
}

template <int S, bool KEEP>
__device__ __forceinline__ f32x8 clip_load8(const void* p, int64_t e) {
    f32x8 f;
#pragma unroll
    for (int i = 0; i < 8; i += kVec<S>) {
        const Vec<S> v = load16<S, KEEP>(p, e + i);
#pragma unroll
        for (int j = 0; j < kVec<S>; ++j) f[i + j] = v.f[j];
    }
    return f;
}
template <int S, int D, bool KEEP>
__device__ __forceinline__ void chunk_clip(const ClipItem& t, int64_t e0, int64_t e1, float c) {
    const int64_t body = e0 + (e1 - e0) / 8 * 8;
#pragma unroll 4
    for (int64_t e = e0 + threadIdx.x * 8; e < body; e += kThreads * 8) {
        f32x8 f = clip_load8<S, KEEP>(t.src, e);
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] *= c;
        stream8<D>(t.dst, e, f);
    }
    const int64_t e = body + threadIdx.x;
    if (e < e1) store1<D>(t.dst, e, load1<S>(t.src, e) * c);
}
template <int S, int D>
__device__ __forceinline__ void chunk_clip(const ClipItem& t, int64_t e0, int64_t e1, float c, bool keep) {
    if (keep) chunk_clip<S, D, true>(t, e0, e1, c);
    else chunk_clip<S, D, false>(t, e0, e1, c);
}
template <int D>
__device__ __forceinline__ void chunk_zero(const ClipItem& t, int64_t e0, int64_t e1) {
    for (int64_t e = e0 + threadIdx.x; e < e1; e += kThreads) store1<D>(t.dst, e, 0.f);
}

__global__ __launch_bounds__(kThreads) void clip_kernel(ClipArgs a) {
    const float c = a.coef ? *a.coef : 1.0f;
    if (a.in_place && c == 1.0f) return;
    const int b = blockIdx.x;
    const bool keep = a.before + b < kKeep;
    const ClipItem t = a.it[item_of(a, b)];
    const int64_t e0 = ((t.n - 1) / a.chunk - (b - t.chunk0)) * a.chunk;    // from the tensor's end
    const int64_t e1 = e0 + a.chunk < t.n ? e0 + a.chunk : t.n;
    const int s = t.src_dtype, d = t.dst_dtype;
    if (!t.src) {
        chunk_zero<ZSMR_BF16>(t, e0, e1);               // +0 is the same bits in both formats
    } else if (d == ZSMR_FP32) {
        chunk_clip<ZSMR_FP32, ZSMR_FP32>(t, e0, e1, c, keep);  // in place only
    } else if (d == ZSMR_BF16) {
        if (s == ZSMR_FP32) chunk_clip<ZSMR_FP32, ZSMR_BF16>(t, e0, e1, c, keep);
        else if (s == ZSMR_BF16) chunk_clip<ZSMR_BF16, ZSMR_BF16>(t, e0, e1, c, keep);
        else chunk_clip<ZSMR_FP16, ZSMR_BF16>(t, e0, e1, c, keep);
    } else {
        if (s == ZSMR_FP32) chunk_clip<ZSMR_FP32, ZSMR_FP16>(t, e0, e1, c, keep);
        else if (s == ZSMR_BF16) chunk_clip<ZSMR_BF16, ZSMR_FP16>(t, e0, e1, c, keep);
        else chunk_clip<ZSMR_FP16, ZSMR_FP16>(t, e0, e1, c, keep);
    }
}

// ------------------------------------------------------ the clipped step --
__device__ __forceinline__ float mean_of(const StepArgs& a, float sum) {
    if (!a.mean) return sum;
    return a.inv_pow2 ? sum * a.inv_nf : sum / a.nf;
}

// The sum of rows [0, nrows) at one lane's eight elements, in fp32 strictly in
// rank order, kRows loads in flight.
constexpr int kRows = 8;
template <int DT>
__device__ __forceinline__ f32x8 sum_rows(const StepArgs& a, int64_t e) {
    const uint16_t* p = a.grads + e;
    // -0 + x is x for every x, so the sum starts at row 0 with its own bits
    f32x8 g = -0.0f;
    int r = 0;
    for (; r + kRows <= a.nrows; r += kRows) {
        u16x8 h[kRows];
#pragma unroll
        for (int k = 0; k < kRows; ++k)
            h[k] = __builtin_nontemporal_load(reinterpret_cast<const u16x8_any*>(p + (int64_t)(r + k) * a.row_stride));
#pragma unroll
        for (int k = 0; k < kRows; ++k)
#pragma unroll
            for (int i = 0; i < 8; ++i) g[i] += widen16<DT>(h[k][i]);
    }
    for (; r < a.nrows; ++r) {
        const u16x8 h = *reinterpret_cast<const u16x8_any*>(p + (int64_t)r * a.row_stride);
#pragma unroll
        for (int i = 0; i < 8; ++i) g[i] += widen16<DT>(h[i]);
    }
    return g;
}
// The mean and the squares of a lane's eight elements.
__device__ __forceinline__ f32x8 mean_sumsq(const StepArgs& a, f32x8 g, double* s) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        g[i] = mean_of(a, g[i]);
        *s = __builtin_fma((double)g[i], (double)g[i], *s);
    }
    return g;
}
template <int DT>
__device__ __forceinline__ double reduce_some(const StepArgs& a, int64_t e) {
    double s = 0;
    if (e + 8 <= a.n) {
        store8<ZSMR_FP32>(a.g_out, e, mean_sumsq(a, sum_rows<DT>(a, e), &s));
    } else {
        for (int64_t j = e; j < a.n && j < e + 8; ++j) {
            float g = widen16<DT>(a.grads[j]);
            for (int r = 1; r < a.nrows; ++r) g += widen16<DT>(a.grads[(int64_t)r * a.row_stride + j]);
            g = mean_of(a, g);
            a.g_out[j] = g;
            s = __builtin_fma((double)g, (double)g, s);
        }
    }
    return s;
}
template <int DT>
__global__ __launch_bounds__(kThreads) void reduce_sumsq_kernel(StepArgs a, double* partial) {
    const double s = block_sum<kThreads>(reduce_some<DT>(a, (int64_t)blockIdx.x * kTile + threadIdx.x * 8));
    if (threadIdx.x == 0) partial[blockIdx.x] = s;
}

// A small piece in one workgroup, which leaves the whole sum: one launch
// instead of two.
constexpr int kSmall = 1024;
template <int DT>
__global__ __launch_bounds__(kSmall) void reduce_sumsq_small_kernel(StepArgs a, double* sumsq) {
    double s = 0;
    for (int64_t e = threadIdx.x * 8; e < a.n; e += kSmall * 8) s += reduce_some<DT>(a, e);
    s = block_sum<kSmall>(s);
    if (threadIdx.x == 0) *sumsq = s;
}

// Many rows of a large piece.  The g that is written is a thirtieth of the
// bytes, but written as it comes it takes a seventh of the time: HBM loses far
// more to turning between reads and writes than to the writes.  So a wave
// keeps the sums of up to kRing tiles of 512 elements in LDS and stores them
// in short windows that all waves of the chip take at the same time, read from
// the constant-rate clock (100 MHz); no loads are issued in a window until
// kLead before its end.  A ring that fills before its window is stored at once.
// Measured on MI355X, 64 rows of 117,187,500: as they come 2.84-2.93 ms, no
// writes at all 2.35, windows 2.54 (4 us in every 100; 60 us 2.55, 160 us 2.56;
// windows of 8 us the same, 15 us 2.59-2.86; two workgroups a CU with half the
// ring 2.61-2.85).
constexpr int kRing = 18;
constexpr uint32_t kCycle = 10000, kWindow = 400, kLead = 133;      // ticks of 10 ns
__device__ __forceinline__ void wait_clock(uint64_t t) {
    for (int i = 0; i < (1 << 16); ++i) {           // bounded: a wave always goes on
        if (__builtin_amdgcn_s_memrealtime() >= t) break;
        __builtin_amdgcn_s_sleep(1);
    }
}
template <int DT>
__global__ __launch_bounds__(kThreads) void reduce_sumsq_windows_kernel(StepArgs a, double* partial) {
    constexpr int kWaves = kThreads / 64;
    __shared__ f32x4 ring[kWaves][kRing][2][64];    // a lane reads back only its own values
    const int lane = threadIdx.x % 64, wave = threadIdx.x / 64;
    const int64_t tiles = a.n / 512, waves = (int64_t)gridDim.x * kWaves;
    const int64_t me = (int64_t)blockIdx.x * kWaves + wave;
    double s = 0;
    int64_t done = 0, stored = 0;                   // tiles of this wave
    uint64_t taken = ~0ull;                         // the cycle whose window was taken
    auto flush = [&]() {
        for (; stored < done; ++stored) {
            const int64_t e = (me + stored * waves) * 512 + lane * 8;
            const f32x4 lo = ring[wave][stored % kRing][0][lane], hi = ring[wave][stored % kRing][1][lane];
            __builtin_nontemporal_store(lo, reinterpret_cast<f32x4_any*>(a.g_out + e));
            __builtin_nontemporal_store(hi, reinterpret_cast<f32x4_any*>(a.g_out + e + 4));
        }
    };
    for (int64_t tile = me; tile < tiles; tile += waves) {
        const uint16_t* p = a.grads + tile * 512 + lane * 8;
        f32x8 g = -0.0f;
        u16x8 x[kRows], y[kRows];
        // rows past the last are that row again, and are not added
        auto load = [&](u16x8* h, int r) {
#pragma unroll
            for (int k = 0; k < kRows; ++k)
                h[k] = __builtin_nontemporal_load(reinterpret_cast<const u16x8_any*>(
                    p + (int64_t)(r + k < a.nrows ? r + k : a.nrows - 1) * a.row_stride));
        };
        auto add = [&](const u16x8* h, int r) {
#pragma unroll
            for (int k = 0; k < kRows; ++k)
                if (r + kRows <= a.nrows || r + k < a.nrows) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) g[i] += widen16<DT>(h[k][i]);
                }
        };
        load(x, 0);
        for (int r = 0; r < a.nrows; r += 2 * kRows) {
            const uint64_t now = __builtin_amdgcn_s_memrealtime(), cycle = now / kCycle;
            if (now - cycle * kCycle + kWindow >= kCycle && cycle != taken) {
                flush();
                taken = cycle;
                wait_clock((cycle + 1) * kCycle - kLead);
            }
            if (r + kRows < a.nrows) load(y, r + kRows);
            add(x, r);
            if (r + 2 * kRows < a.nrows) load(x, r + 2 * kRows);
            if (r + kRows < a.nrows) add(y, r + kRows);
        }
        g = mean_sumsq(a, g, &s);
        if (done - stored == kRing) flush();
        f32x4 lo, hi;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            lo[i] = g[i];
            hi[i] = g[4 + i];
        }
        ring[wave][done % kRing][0][lane] = lo;
        ring[wave][done % kRing][1][lane] = hi;
        ++done;
    }
    flush();
    if (blockIdx.x == 0 && threadIdx.x * 8 < a.n - tiles * 512)     // the elements past the last tile
        s += reduce_some<DT>(a, tiles * 512 + threadIdx.x * 8);
    s = block_sum<kThreads>(s);
    if (threadIdx.x == 0) partial[blockIdx.x] = s;
}

// Adam with one fp32 rounding per operation, as zero_adam_step has it ("The
// four schemes", Base._adam).
__device__ __forceinline__ void adam(const AdamK& k, float g, float& w, float& m, float& v) {
    m = k.c1 * m + k.c1m * g;
    v = k.c2 * v + (k.c2m * g) * g;
    const float mh = m / k.bc1;
    const float vh = v / k.bc2;
    w = w - (k.lr * mh) / (__builtin_sqrtf(vh) + k.eps);
}

template <int DT>
__global__ __launch_bounds__(kThreads) void clipped_kernel(StepArgs a, const float* coef) {
    const float c = coef ? *coef : 1.0f;
    // two groups of four elements a lane: each instruction of a wave covers
    // one contiguous KB of fp32
    const int64_t t0 = (int64_t)blockIdx.x * kTile + (threadIdx.x / 64) * 512 + (threadIdx.x % 64) * 4;
    if (t0 + 260 <= a.n) {
        f32x4 g[2], w[2], m[2], v[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int64_t e = t0 + j * 256;
            g[j] = __builtin_nontemporal_load(reinterpret_cast<const f32x4_any*>(a.g_in + e));
            w[j] = __builtin_nontemporal_load(reinterpret_cast<const f32x4_any*>(a.master + e));
            m[j] = __builtin_nontemporal_load(reinterpret_cast<const f32x4_any*>(a.m + e));
            v[j] = __builtin_nontemporal_load(reinterpret_cast<const f32x4_any*>(a.v + e));
        }
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int64_t e = t0 + j * 256;
            u16x4 h;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float wi = w[j][i], mi = m[j][i], vi = v[j][i];
                adam(a.k, g[j][i] * c, wi, mi, vi);
                w[j][i] = wi;
                m[j][i] = mi;
                v[j][i] = vi;
                h[i] = narrow16<DT>(wi);
            }
            __builtin_nontemporal_store(w[j], reinterpret_cast<f32x4_any*>(a.master + e));
            __builtin_nontemporal_store(m[j], reinterpret_cast<f32x4_any*>(a.m + e));
            __builtin_nontemporal_store(v[j], reinterpret_cast<f32x4_any*>(a.v + e));
            __builtin_nontemporal_store(h, reinterpret_cast<u16x4_any*>(a.p16 + e));
        }
    } else {
        for (int j = 0; j < 2; ++j)
            for (int i = 0; i < 4; ++i) {
                const int64_t e = t0 + j * 256 + i;
                if (e >= a.n) continue;
                float w = a.master[e], m = a.m[e], v = a.v[e];
                adam(a.k, a.g_in[e] * c, w, m, v);
                a.master[e] = w;
                a.m[e] = m;
                a.v[e] = v;
                a.p16[e] = narrow16<DT>(w);
            }
    }
}

}  // namespace

int sumsq_grid(int64_t chunks) { return (int)std::min<int64_t>(chunks, kSumsqGrid); }

hipError_t launch_sumsq(const NormArgs& a, double* partial, hipStream_t stream) {
    sumsq_kernel<<<sumsq_grid(a.chunks), kThreads, 0, stream>>>(a, partial);
    return hipGetLastError();
}

hipError_t launch_clip(const ClipArgs& a, hipStream_t stream) {
    clip_kernel<<<a.chunks, kThreads, 0, stream>>>(a);
    return hipGetLastError();
}

hipError_t launch_join(const double* partial, int64_t n, double* sumsq, double max_norm,
                       double eps, float* norm_coef, hipStream_t stream) {
    // one wave where it has few sums to add: nothing to wait for between waves
    if (n <= 512) join_kernel<64><<<1, 64, 0, stream>>>(partial, n, sumsq, max_norm, eps, norm_coef);
    else join_kernel<1024><<<1, 1024, 0, stream>>>(partial, n, sumsq, max_norm, eps, norm_coef);
    return hipGetLastError();
}

namespace {
// Windows pay where writes are a small share of a long stream.  Measured on
// MI355X, as it comes against windows, us: 8 rows of 30M 97 / 123; 16 rows of
// 30M 182 / 193, of 100M 664 / 627; 24 rows of 30M 269 / 275; 32 rows of 4.8M
// 58.2 / 58.7, of 9.6M 115 / 109, of 30M 357 / 334; 64 rows of 2.4M 54 / 61, of
// 4.8M 111 / 107, of 30M 684 / 623.
bool windows_pay(int64_t rows, int64_t n) {
    const int64_t read = rows * n;
    return rows >= 32 ? read >= int64_t(1) << 28 : rows >= 16 && read >= int64_t(1) << 30;
}

template <int DT>
hipError_t reduce_launches(const StepArgs& a, double* partial, double* sumsq, hipStream_t stream) {
    // one workgroup: 8 elements a lane, or twice that
    if (a.n <= 2 * kSmall * 8) {
        reduce_sumsq_small_kernel<DT><<<1, kSmall, 0, stream>>>(a, sumsq);
        return hipGetLastError();
    }
    int64_t parts = (a.n + kTile - 1) / kTile;
    int device = 0, cus = 0;
    if (windows_pay(a.nrows, a.n) && hipGetDevice(&device) == hipSuccess &&
        hipDeviceGetAttribute(&cus, hipDeviceAttributeMultiprocessorCount, device) == hipSuccess &&
        a.n / 512 >= (int64_t)cus * (kThreads / 64)) {      // a tile for every wave
        parts = cus;
        reduce_sumsq_windows_kernel<DT><<<cus, kThreads, 0, stream>>>(a, partial);
    } else {
        reduce_sumsq_kernel<DT><<<(unsigned)parts, kThreads, 0, stream>>>(a, partial);
    }
    return launch_join(partial, parts, sumsq, 0, 0, nullptr, stream);
}
}  // namespace

hipError_t launch_reduce_sumsq(int dtype, const StepArgs& a, double* partial, double* sumsq,
                               hipStream_t stream) {
    return dtype == ZSMR_BF16 ? reduce_launches<ZSMR_BF16>(a, partial, sumsq, stream)
                              : reduce_launches<ZSMR_FP16>(a, partial, sumsq, stream);
}

hipError_t launch_clipped(int dtype, const StepArgs& a, const float* coef, hipStream_t stream) {
    const dim3 grid((unsigned)((a.n + kTile - 1) / kTile));
    if (dtype == ZSMR_BF16) clipped_kernel<ZSMR_BF16><<<grid, kThreads, 0, stream>>>(a, coef);
    else clipped_kernel<ZSMR_FP16><<<grid, kThreads, 0, stream>>>(a, coef);
    return hipGetLastError();
}

}  // namespace zsmr
