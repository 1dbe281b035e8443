// gfx950 kernels of the embedding lookup and of its gradient.
//
//   out[t] = rne16(scale * table[id_t]),
//   dtable[v] = rne16([dtable[v] +] scale * sum over id_t = v of dout[t]).
//
// Both are bound by HBM.  The gradient's sum has to give the same bits each
// time, so tokens are sorted by id (a stable radix sort: equal ids stay in
// token order) and each run of equal ids is added up in that order; nothing
// goes through atomics in global memory.  A run may be as long as the batch,
// so it is cut at every 8 to 64 sorted tokens: a run inside one such chunk is
// finished there, the parts of one that crosses chunks are kept in fp32 and
// joined in order.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "zsmr_dev.h"
#include "zsmr_ops_launch.h"

#pragma clang fp contract(off)

namespace zsmr {
namespace {

constexpr int kThreads = 256;

// ----------------------------------------------------------------- lookup --
// One thread, eight elements of one row; a workgroup's threads walk along rows.
template <int DT>
__global__ __launch_bounds__(kThreads) void lookup_kernel(EmbedArgs a, uint32_t vecs) {
    const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    const int64_t t = vecs == 1 ? i : i / vecs;
    if (t >= a.tokens) return;
    const int64_t j = (i - t * vecs) * 8;
    const int32_t id = token_at(a.ids, a.id_bytes, t, a.vocab);
    uint16_t* out = a.dst + t * a.dst_stride;
    const uint16_t* row = a.src + (int64_t)(id < 0 ? 0 : id) * a.src_stride;
    if (j + 8 <= a.width) {
        f32x8 f = 0.f;
        if (id >= 0) {
            f = load8<DT>(row, j);
#pragma unroll
            for (int k = 0; k < 8; ++k) f[k] *= a.scale;
        }
        stream8<DT>(out, j, f);
    } else {
        for (int64_t k = j; k < a.width; ++k) store1<DT>(out, k, id < 0 ? 0.f : load1<DT>(row, k) * a.scale);
    }
}

// ------------------------------------------------------------------- sort --
// One pass of a stable radix sort on 9 bits: a launch that counts each
// workgroup's digits and one in which every workgroup adds up the counts of those
// before it and moves its keys.  Padding is key vocab: last.  Measured on MI355X,
// 16,384 tokens, two passes: 16-20 us; every workgroup counting all keys itself, with
// no launch for it, 23-25.
constexpr int kSortThreads = 1024, kSortWaves = kSortThreads / 64;
constexpr int kDigit = 9, kBins = 1 << kDigit;
struct SortArgs {
    const void* ids;
    int32_t id_bytes;
    int32_t tokens;
    int64_t vocab;
    const uint32_t *key_in, *pos_in;
    uint32_t *key_out, *pos_out;
    uint32_t* counts;               // [workgroup][kBins]
    int32_t part;                   // keys of one workgroup
    int32_t shift;
};
template <bool FIRST>
__device__ __forceinline__ uint32_t sort_key(const SortArgs& a, int64_t i) {
    if constexpr (!FIRST) return a.key_in[i];
    const int32_t id = token_at(a.ids, a.id_bytes, i, a.vocab);
    return id < 0 ? (uint32_t)a.vocab : (uint32_t)id;
}
// The lanes of the wave that hold the same digit; d of a lane that is off does
// not matter.
__device__ __forceinline__ uint64_t same_digit(uint32_t d, bool on) {
    uint64_t same = __ballot(on);
#pragma unroll
    for (int b = 0; b < kDigit; ++b) {
        const uint64_t has = __ballot((d >> b) & 1);
        same &= (d >> b) & 1 ? has : ~has;
    }
    return same;
}
__device__ __forceinline__ int rank_in(uint64_t same) { return __popcll(same & ((1ull << (threadIdx.x % 64)) - 1)); }
// Count a wave's digits: one add if all are the same (a frequent token's keys
// come together after the first pass, and 64 adds to one counter queue up).
__device__ __forceinline__ void count_digits(uint32_t* bins, uint32_t d, bool on) {
    if (!on) return;
    const uint32_t first = __builtin_amdgcn_readfirstlane(d);
    const uint64_t lanes = __ballot(true);
    if (__ballot(d == first) == lanes) {
        if (rank_in(lanes) == 0) atomicAdd(&bins[d], (uint32_t)__popcll(lanes));
    } else {
        atomicAdd(&bins[d], 1u);
    }
}
// cnt[w][d]: the keys of digit d in wave w's part, on return where the first of
// them goes: after those of smaller digits (all: their number), those of other
// workgroups before this one (before) and those of the waves before.
__device__ __forceinline__ void places(uint32_t (*cnt)[kBins], uint32_t all, uint32_t before) {
    __shared__ uint32_t wave_sum[kBins / 64];
    const int tid = threadIdx.x, wave = tid / 64, lane = tid % 64;
    uint32_t upto = all;
    if (tid < kBins) {
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const uint32_t up = __shfl_up(upto, d);
            if (lane >= d) upto += up;
        }
        if (lane == 63) wave_sum[wave] = upto;
    }
    __syncthreads();
    if (tid < kBins) {
        uint32_t at = upto - all + before;
        for (int w = 0; w < wave; ++w) at += wave_sum[w];
#pragma unroll
        for (int w = 0; w < kSortWaves; ++w) {
            const uint32_t c = cnt[w][tid];
            cnt[w][tid] = at;
            at += c;
        }
    }
    __syncthreads();
}
// This lane's key's place; takes it from the wave's row of places.
__device__ __forceinline__ uint32_t take_place(uint32_t* row, uint32_t d, bool on) {
    const uint64_t same = same_digit(d, on);
    const int rank = rank_in(same);
    const uint32_t at = on ? row[d] : 0;
    __builtin_amdgcn_wave_barrier();
    if (on && rank == 0) row[d] = at + __popcll(same);
    __builtin_amdgcn_wave_barrier();
    return at + rank;
}

template <bool FIRST>
__global__ __launch_bounds__(kSortThreads) void count_kernel(SortArgs a) {
    __shared__ uint32_t bins[kBins];
    const int tid = threadIdx.x;
    if (tid < kBins) bins[tid] = 0;
    __syncthreads();
    const int64_t b0 = (int64_t)blockIdx.x * a.part;
    const int64_t b1 = b0 + a.part < a.tokens ? b0 + a.part : a.tokens;
    for (int64_t i = b0 + tid; i < b1; i += kSortThreads) count_digits(bins, (sort_key<FIRST>(a, i) >> a.shift) & (kBins - 1), true);
    __syncthreads();
    if (tid < kBins) a.counts[(int64_t)blockIdx.x * kBins + tid] = bins[tid];
}

template <bool FIRST>
__global__ __launch_bounds__(kSortThreads) void sort_kernel(SortArgs a) {
    __shared__ uint32_t cnt[kSortWaves][kBins];
    const int tid = threadIdx.x, wave = tid / 64, lane = tid % 64;
    for (int i = tid; i < kSortWaves * kBins; i += kSortThreads) (&cnt[0][0])[i] = 0;
    __syncthreads();
    uint32_t all = 0, before = 0;
    if (tid < kBins) {
#pragma unroll 8
        for (unsigned b = 0; b < gridDim.x; ++b) {
            const uint32_t c = a.counts[(int64_t)b * kBins + tid];
            all += c;
            if (b < blockIdx.x) before += c;
        }
    }
    const int64_t b0 = (int64_t)blockIdx.x * a.part;
    const int64_t b1 = b0 + a.part < a.tokens ? b0 + a.part : a.tokens;
    // this workgroup's keys, a contiguous run for each wave
    const int64_t run = (b1 - b0 + kSortThreads - 1) / kSortThreads * 64;
    const int64_t w0 = b0 + wave * run;
    const int64_t w1 = w0 + run < b1 ? w0 + run : b1;
    for (int64_t i0 = w0; i0 < w1; i0 += 64) {
        const bool on = i0 + lane < w1;
        count_digits(cnt[wave], on ? (sort_key<FIRST>(a, i0 + lane) >> a.shift) & (kBins - 1) : 0, on);
    }
    __syncthreads();
    places(cnt, all, before);
    for (int64_t i0 = w0; i0 < w1; i0 += 64) {
        const int64_t i = i0 + lane;
        const bool on = i < w1;
        const uint32_t key = on ? sort_key<FIRST>(a, i) : 0u;
        const uint32_t at = take_place(cnt[wave], (key >> a.shift) & (kBins - 1), on);
        if (on) {
            a.key_out[at] = key;
            a.pos_out[at] = FIRST ? (uint32_t)i : a.pos_in[i];
        }
    }
}

// All passes over a few tokens in one workgroup, between two buffers in LDS.
constexpr int kSmallSort = 4096;
__global__ __launch_bounds__(kSortThreads) void sort_small_kernel(SortArgs a, int bits) {
    __shared__ uint32_t key[2][kSmallSort], cnt[kSortWaves][kBins];
    __shared__ uint16_t pos[2][kSmallSort];
    const int tid = threadIdx.x, wave = tid / 64, lane = tid % 64;
    const int n = a.tokens, run = (n + kSortThreads - 1) / kSortThreads * 64;
    const int w0 = wave * run, w1 = w0 + run < n ? w0 + run : n;
    for (int i = tid; i < n; i += kSortThreads) {
        key[0][i] = sort_key<true>(a, i);
        pos[0][i] = (uint16_t)i;
    }
    int from = 0;
    for (int shift = 0; shift < bits; shift += kDigit, from ^= 1) {
        for (int i = tid; i < kSortWaves * kBins; i += kSortThreads) (&cnt[0][0])[i] = 0;
        __syncthreads();
        for (int i0 = w0; i0 < w1; i0 += 64) {
            const bool on = i0 + lane < w1;
            count_digits(cnt[wave], on ? (key[from][i0 + lane] >> shift) & (kBins - 1) : 0, on);
        }
        __syncthreads();
        uint32_t all = 0;
        if (tid < kBins) {
#pragma unroll
            for (int w = 0; w < kSortWaves; ++w) all += cnt[w][tid];
        }
        places(cnt, all, 0);
        for (int i0 = w0; i0 < w1; i0 += 64) {
            const int i = i0 + lane;
            const bool on = i < w1;
            const uint32_t k = on ? key[from][i] : 0u;
            const uint32_t at = take_place(cnt[wave], (k >> shift) & (kBins - 1), on);
            if (on) {
                key[from ^ 1][at] = k;
                pos[from ^ 1][at] = pos[from][i];
            }
        }
        __syncthreads();
    }
    for (int i = tid; i < n; i += kSortThreads) {
        a.key_out[i] = key[from][i];
        a.pos_out[i] = pos[from][i];
    }
}

// --------------------------------------------------------------- gradient --
constexpr int kCols = 512;          // columns of a wave: eight to a lane
constexpr int kBlockCols = kThreads / 64 * kCols;

template <int DT>
__device__ __forceinline__ void put_row(const EmbedArgs& a, uint32_t v, int64_t j, f32x8 f) {
    uint16_t* row = a.dst + (int64_t)v * a.dst_stride;
#pragma unroll
    for (int k = 0; k < 8; ++k) f[k] *= a.scale;
    if (j + 8 <= a.width) {
        if (a.accumulate) f += load8<DT>(row, j);
        store8<DT>(row, j, f);
    } else {
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (j + k < a.width) store1<DT>(row, j + k, a.accumulate ? load1<DT>(row, j + k) + f[k] : f[k]);
    }
}
__device__ __forceinline__ void put_part(float* p, int64_t j, int64_t width, f32x8 f) {
    if (j + 8 <= width) {
        store8<ZSMR_FP32>(p, j, f);
    } else {
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (j + k < width) p[j + k] = f[k];
    }
}
template <int DT>
__device__ __forceinline__ f32x8 get_row(const void* p, int64_t j, int64_t width) {
    if (j + 8 <= width) {
        if constexpr (DT == ZSMR_FP32) return load8<DT>(p, j);
        f32x8 f;
        const Vec<DT> v = load16<DT, false>(p, j);
#pragma unroll
        for (int k = 0; k < 8; ++k) f[k] = v.f[k];
        return f;
    }
    f32x8 f = 0.f;
#pragma unroll
    for (int k = 0; k < 8; ++k)
        if (j + k < width) f[k] = load1<DT>(p, j + k);
    return f;
}

// Zeros in the rows of absent tokens, kZeroRows to a workgroup.
constexpr int kZeroRows = 16;
__device__ __forceinline__ void zero_rows(const EmbedArgs& a, const uint32_t* key, int64_t v0) {
    __shared__ int present[kZeroRows];
    // 16 lanes a row narrow down its place among the sorted keys 17 ways a step
    const int lane = threadIdx.x % 16, group = threadIdx.x % 64 / 16;
    const uint32_t v = (uint32_t)v0 + threadIdx.x / 16;
    int64_t lo = 0, hi = a.tokens;
    while (lo < hi) {
        const int64_t n = hi - lo, at = lo + n * (lane + 1) / 17;
        const int below = __popc((uint32_t)(__ballot(key[at] < v) >> (group * 16)) & 0xffff);
        const int64_t last = lo + n * below / 17;       // the highest pivot below v
        if (below < 16) hi = lo + n * (below + 1) / 17;
        if (below > 0) lo = last + 1;
    }
    if (lane == 0) present[threadIdx.x / 16] = lo < a.tokens && key[lo] == v;
    __syncthreads();
    for (int r = 0; r < kZeroRows && v0 + r < a.vocab; ++r) {
        if (present[r]) continue;
        uint16_t* row = a.dst + (v0 + r) * a.dst_stride;
        for (int64_t j = threadIdx.x * 8; j < a.width; j += kThreads * 8) {
            if (j + 8 <= a.width) __builtin_nontemporal_store(u16x8(0), reinterpret_cast<u16x8_any*>(row + j));
            else for (int64_t k = j; k < a.width; ++k) row[k] = 0;
        }
    }
}

// The runs of one chunk of sorted tokens in one column block.
// part[chunk][0]: the sum of a run that came from the chunk before; [1]: of one
// that starts here and goes on.
template <int DT>
__device__ __forceinline__ void add_runs(const EmbedArgs& a, const uint32_t* key, const uint32_t* pos,
                                         float* part, int64_t c, int chunk, int64_t j) {
    const int lane = threadIdx.x % 64;
    if (j - lane * 8 >= a.width) return;
    const int64_t i0 = c * chunk;
    const int n = (int)(a.tokens - i0 < chunk ? a.tokens - i0 : chunk);
    const uint32_t none = (uint32_t)a.vocab;
    const uint32_t my_key = lane < n ? key[i0 + lane] : none;
    const uint32_t my_pos = lane < n ? pos[i0 + lane] : 0;
    const uint32_t prev = i0 > 0 ? key[i0 - 1] : none;
    const uint32_t next = i0 + n < a.tokens ? key[i0 + n] : none;
    f32x8 sum = 0.f;
    bool first = true;                              // of the chunk
    constexpr int kAhead = 8;
    for (int b = 0; b < n; b += kAhead) {
        f32x8 f[kAhead];
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            const int i = b + k < n ? b + k : n - 1;
            f[k] = get_row<DT>(a.src + (int64_t)__builtin_amdgcn_readlane(my_pos, i) * a.src_stride, j, a.width);
        }
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            const int i = b + k;
            if (i >= n) break;
            const uint32_t v = __builtin_amdgcn_readlane(my_key, i);
            if (v == none) return;                  // padding is last
            sum += f[k];
            const uint32_t after = i + 1 < n ? __builtin_amdgcn_readlane(my_key, i + 1) : next;
            if (after == v && i + 1 < n) continue;
            const bool came = first && prev == v, goes = after == v;
            if (came) put_part(part + (2 * c) * a.width, j, a.width, sum);
            else if (goes) put_part(part + (2 * c + 1) * a.width, j, a.width, sum);
            else put_row<DT>(a, v, j, sum);
            sum = 0.f;
            first = false;
        }
    }
}

// The first workgroups add up runs, the others write zeros meanwhile.  first: of
// this launch's workgroups.
template <int DT>
__global__ __launch_bounds__(kThreads) void grad_kernel(EmbedArgs a, const uint32_t* key, const uint32_t* pos,
                                                        float* part, int chunk, int64_t chunks, int col_blocks,
                                                        int64_t first) {
    const int64_t b = first + blockIdx.x, runs = chunks * col_blocks;
    if (b < runs) add_runs<DT>(a, key, pos, part, b / col_blocks, chunk, b % col_blocks * kBlockCols + threadIdx.x * 8);
    else zero_rows(a, key, (b - runs) * kZeroRows);
}

// One workgroup for each chunk whose last run starts in it and goes on.
template <int DT>
__global__ __launch_bounds__(kThreads) void join_runs_kernel(EmbedArgs a, const uint32_t* key,
                                                             const float* part, int chunk) {
    const int64_t c = blockIdx.x, last = c * chunk + chunk - 1;
    if (last + 1 >= a.tokens) return;
    const uint32_t v = key[last];
    if (v == (uint32_t)a.vocab || key[last + 1] != v) return;
    if (c > 0 && key[c * chunk - 1] == v) return;         // it started before this chunk
    int64_t lo = last + 1, hi = a.tokens;                 // the run's end
    while (lo < hi) {
        const int64_t mid = (lo + hi) / 2;
        if (key[mid] == v) lo = mid + 1;
        else hi = mid;
    }
    const int64_t end = (lo - 1) / chunk;
    const int64_t j = (int64_t)blockIdx.y * kBlockCols + threadIdx.x * 8;
    if (j >= a.width) return;
    f32x8 sum = get_row<ZSMR_FP32>(part + (2 * c + 1) * a.width, j, a.width);
    constexpr int kAhead = 8;
    for (int64_t k = c + 1; k <= end; k += kAhead) {
        f32x8 f[kAhead];
#pragma unroll
        for (int i = 0; i < kAhead; ++i)
            if (k + i <= end) f[i] = get_row<ZSMR_FP32>(part + 2 * (k + i) * a.width, j, a.width);
#pragma unroll
        for (int i = 0; i < kAhead; ++i)
            if (k + i <= end) sum += f[i];
    }
    put_row<DT>(a, v, j, sum);
}

int64_t up16(int64_t n) { return (n + 15) / 16 * 16; }
int64_t col_blocks_of(int64_t width) { return (width + kBlockCols - 1) / kBlockCols; }
// Sorted tokens of a chunk.  A wave reads a chunk's rows one after another, and
// one wave joins the parts of a frequent token's run, which is about a tenth of
// the tokens in text.  Measured on MI355X, whole gradient: 16,384 tokens of width
// 4,096 240 us in chunks of 64, 237 of 32; 1,302 of width 72 19.6 of 8, 22.7 of 16.
int chunk_of(int64_t tokens) {
    int chunk = 8;
    while (chunk < 64 && (int64_t)chunk * chunk * 32 < tokens) chunk *= 2;
    return chunk;
}

// fp32 elements of the chunks' partial sums
int64_t chunk_sums(int64_t tokens, int64_t width) {
    const int chunk = chunk_of(tokens);
    return (tokens + chunk - 1) / chunk * 2 * width;
}
// Keys of a sorting workgroup: at most kMaxParts workgroups.
constexpr int64_t kMaxParts = 32;
int64_t part_of(int64_t tokens) {
    return std::max<int64_t>(1024, (tokens + kMaxParts * 1024 - 1) / (kMaxParts * 1024) * 1024);
}

template <int DT>
void grad_launches(const EmbedArgs& a, const uint32_t* key, const uint32_t* pos, float* part,
                   hipStream_t stream) {
    const int chunk = chunk_of(a.tokens), cols = (int)col_blocks_of(a.width);
    const int64_t chunks = (a.tokens + chunk - 1) / chunk;
    const int64_t zeros = a.accumulate ? 0 : (a.vocab + kZeroRows - 1) / kZeroRows;
    launch_groups(chunks * cols + zeros, [&](int64_t first, int64_t count) {
        grad_kernel<DT><<<(unsigned)count, kThreads, 0, stream>>>(a, key, pos, part, chunk, chunks, cols, first);
    });
    if (chunks > 1) join_runs_kernel<DT><<<dim3((unsigned)chunks, cols), kThreads, 0, stream>>>(a, key, part, chunk);
}

}  // namespace

hipError_t launch_embed_lookup(const EmbedArgs& a, hipStream_t stream) {
    const int64_t vecs = (a.width + 7) / 8;
    launch_rows(a.tokens, vecs, [&](int64_t first, int64_t count) {
        EmbedArgs part = a;
        part.tokens = count;
        part.ids = static_cast<const char*>(a.ids) + first * a.id_bytes;
        part.dst = a.dst + first * a.dst_stride;
        const unsigned grid = (unsigned)((count * vecs + kThreads - 1) / kThreads);
        if (a.dtype == ZSMR_BF16) lookup_kernel<ZSMR_BF16><<<grid, kThreads, 0, stream>>>(part, (uint32_t)vecs);
        else lookup_kernel<ZSMR_FP16><<<grid, kThreads, 0, stream>>>(part, (uint32_t)vecs);
    });
    return hipGetLastError();
}

int64_t embed_grad_bytes(int64_t, int64_t width, int64_t tokens) {
    return 4 * up16(tokens * 4) + chunk_sums(tokens, width) * 4 + (tokens ? kMaxParts * kBins * 4 : 0);
}

hipError_t launch_embed_grad(const EmbedArgs& a, void* ws, hipStream_t stream) {
    const int64_t each = up16(a.tokens * 4) / 4;
    uint32_t* key[2] = {static_cast<uint32_t*>(ws), static_cast<uint32_t*>(ws) + each};
    uint32_t* pos[2] = {key[1] + each, key[1] + 2 * each};
    float* part = reinterpret_cast<float*>(pos[1] + each);
    int at = 0;
    if (a.tokens) {
        SortArgs s{};
        s.ids = a.ids;
        s.id_bytes = a.id_bytes;
        s.tokens = (int32_t)a.tokens;
        s.vocab = a.vocab;
        s.part = (int32_t)part_of(a.tokens);
        s.counts = reinterpret_cast<uint32_t*>(part + chunk_sums(a.tokens, a.width));
        const unsigned grid = (unsigned)((a.tokens + s.part - 1) / s.part);
        int bits = 1;
        while (a.vocab >> bits) ++bits;                 // the largest key is vocab
        s.key_out = key[0];
        s.pos_out = pos[0];
        if (a.tokens <= kSmallSort) sort_small_kernel<<<1, kSortThreads, 0, stream>>>(s, bits);
        for (int shift = a.tokens <= kSmallSort ? bits : 0; shift < bits; shift += kDigit, at ^= 1) {
            s.shift = shift;
            s.key_in = key[at ^ 1];
            s.pos_in = pos[at ^ 1];
            s.key_out = key[at];
            s.pos_out = pos[at];
            if (shift == 0) {
                count_kernel<true><<<grid, kSortThreads, 0, stream>>>(s);
                sort_kernel<true><<<grid, kSortThreads, 0, stream>>>(s);
            } else {
                count_kernel<false><<<grid, kSortThreads, 0, stream>>>(s);
                sort_kernel<false><<<grid, kSortThreads, 0, stream>>>(s);
            }
        }
        if (a.tokens > kSmallSort) at ^= 1;             // where the last pass wrote
    }
    if (a.dtype == ZSMR_BF16) grad_launches<ZSMR_BF16>(a, key[at], pos[at], part, stream);
    else grad_launches<ZSMR_FP16>(a, key[at], pos[at], part, stream);
    return hipGetLastError();
}

}  // namespace zsmr
