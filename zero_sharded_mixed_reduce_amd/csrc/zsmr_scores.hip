// gfx950 kernels of the scores of logits: log probabilities of given tokens with
// entropy and top alternatives, and their gradient.
//
//   z = scale * s,  lse = log sum_v exp z_v,  logprob = z_id - lse,
//   H = lse - sum_v p_v z_v,  p = exp(z - lse)
//   ds_v = scale * (g ([v = id] - p_v) - h p_v (log p_v + H))
//
// Both are bound by HBM: the forward pass reads the logits once, the gradient reads
// and writes them once.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "zsmr_dev.h"
#include "zsmr_ops_launch.h"
#include "zsmr_scores_launch.h"
#include "zsmr_scores_plan.h"

#pragma clang fp contract(off)

namespace zsmr {
namespace {

constexpr int kWaves = kScoreWaves, kThreads = kWaves * 64;
constexpr float kLog2e = 1.44269504f, kLn2 = 0.69314718f;
constexpr float kFloor = -3.0e38f;

// ---------------------------------------------------------------- statistics --
// A part of a softmax: sums of e = exp(z - ref) and of e * log2 e; ref is finite.
struct Stats {
    float ref, sum, mean;
};
__device__ __forceinline__ float exp_of(float d) { return __builtin_amdgcn_exp2f(d); }
// A part relative to another reference, not below its own by much.
__device__ __forceinline__ Stats moved(Stats a, float ref) {
    // a part without a sum (no logit above -infinity) has any reference
    if (a.sum == 0.f) return Stats{ref, 0.f, 0.f};
    const float d = (a.ref - ref) * kLog2e, f = exp_of(d);
    return Stats{ref, a.sum * f, f == 0.f ? 0.f : f * (a.mean + d * a.sum)};
}
__device__ __forceinline__ Stats join_stats(Stats a, Stats b) {
    const float ref = a.sum == 0.f ? b.ref : b.sum == 0.f ? a.ref : fmaxf(a.ref, b.ref);
    a = moved(a, ref);
    b = moved(b, ref);
    return Stats{ref, a.sum + b.sum, a.mean + b.mean};
}
__device__ __forceinline__ Stats shuffled(Stats a, int d) {
    return Stats{__shfl_xor(a.ref, d), __shfl_xor(a.sum, d), __shfl_xor(a.mean, d)};
}

// ----------------------------------------------------------- top alternatives --
// A key orders logits, ties by the lowest index: the value's bits as an unsigned
// integer in the same order, then the index from the top.  0: no alternative.
__device__ __forceinline__ uint32_t order_of(float x) {
    const uint32_t b = __float_as_uint(x + 0.f);        // -0 is +0
    return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}
__device__ __forceinline__ float value_of(uint32_t o) {
    return __uint_as_float(o ^ (o >> 31 ? 0x80000000u : 0xffffffffu));
}
__device__ __forceinline__ uint64_t key_of(float x, uint32_t index) { return (uint64_t)order_of(x) << 32 | (0xffffffffu - index); }
__device__ __forceinline__ uint64_t shuffled(uint64_t k, int d) {
    return (uint64_t)(uint32_t)__shfl_xor((int)(k >> 32), d) << 32 | (uint32_t)__shfl_xor((int)k, d);
}
__device__ __forceinline__ uint64_t lane_key(uint64_t k, int lane) {
    return (uint64_t)(uint32_t)__shfl((int)(k >> 32), lane) << 32 | (uint32_t)__shfl((int)k, lane);
}
// LDS that the lanes of one wave exchange: its operations are in order, the
// compiler has to keep them so.
__device__ __forceinline__ void wave_order() {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}
// One key a lane, largest first.
__device__ __forceinline__ uint64_t merge_step(uint64_t k, int d, bool larger) {
    const uint64_t o = shuffled(k, d);
    return (k > o) == larger ? k : o;
}
__device__ __forceinline__ uint64_t sort64(uint64_t k) {
    const int lane = threadIdx.x % 64;
#pragma unroll
    for (int n = 2; n <= 64; n *= 2)
#pragma unroll
        for (int d = n / 2; d > 0; d /= 2) k = merge_step(k, d, ((lane & d) == 0) == ((lane & n) == 0));
    return k;
}
// The 64 largest of two sorted lists, sorted.
__device__ __forceinline__ uint64_t merge64(uint64_t a, uint64_t b) {
    const int lane = threadIdx.x % 64;
    b = lane_key(b, 63 - lane);
    uint64_t k = a > b ? a : b;
#pragma unroll
    for (int d = 32; d > 0; d /= 2) k = merge_step(k, d, (lane & d) == 0);
    return k;
}

// ------------------------------------------------------------------- forward --
struct ForwardArgs {
    ScoreArgs a;
    int64_t segment;
    int32_t splits;
    float4* stats;              // [token][split], or NULL: the results themselves
    uint64_t* keys;             // [token][split][top]
};

__device__ __forceinline__ void put_token(const ScoreArgs& a, int64_t t, Stats s) {
    const float log_sum = __builtin_amdgcn_logf(s.sum) * kLn2;
    const bool none = s.sum == 0.f;
    if (a.lse) a.lse[t] = none ? -INFINITY : s.ref + log_sum;
    if (a.entropy) a.entropy[t] = none ? 0.f : log_sum - s.mean / s.sum * kLn2;
    if (a.logprob) {
        const int32_t id = token_at(a.ids, a.id_bytes, t, a.vocab);
        float r = 0.f;
        if (id >= 0) {
            const int64_t e = t * a.stride + id;
            const float x = a.dtype == ZSMR_BF16 ? load1<ZSMR_BF16>(a.logits, e) : a.dtype == ZSMR_FP16 ? load1<ZSMR_FP16>(a.logits, e) : load1<ZSMR_FP32>(a.logits, e);
            r = none ? -INFINITY : x * a.scale - s.ref - log_sum;
        }
        a.logprob[t] = r;
    }
}
__device__ __forceinline__ void put_top(const ScoreArgs& a, int64_t t, Stats s, uint64_t key) {
    const int lane = threadIdx.x % 64;
    if (lane >= a.top) return;
    const int64_t e = t * a.top + lane;
    const float log_sum = __builtin_amdgcn_logf(s.sum) * kLn2;
    const int32_t id = key ? (int32_t)(0xffffffffu - (uint32_t)key) : -1;
    if (a.top_ids) {
        if (a.top_bytes == 8) static_cast<int64_t*>(a.top_ids)[e] = id;
        else static_cast<int32_t*>(a.top_ids)[e] = id;
    }
    if (a.top_logprobs) a.top_logprobs[e] = key ? value_of((uint32_t)(key >> 32)) * a.scale - s.ref - log_sum : -INFINITY;
}

template <int DT, bool TOP>
__global__ __launch_bounds__(kThreads) void scores_kernel(ForwardArgs f) {
    const ScoreArgs& a = f.a;
    const int lane = threadIdx.x % 64, wave = threadIdx.x / 64;
    const int64_t t = blockIdx.x / f.splits;
    const int split = blockIdx.x % f.splits;
    const int64_t first = split * f.segment, end = first + f.segment < a.vocab ? first + f.segment : a.vocab;
    constexpr int kStaged = TOP ? 64 + kScoreBlock : 1;
    __shared__ uint64_t staged[kWaves][kStaged];
    __shared__ uint64_t best[kWaves][64];
    __shared__ Stats part[kWaves];

    Stats s{kFloor, 0.f, 0.f};
    bool begun = false;
    uint64_t keys = 0;
    float above = -INFINITY;            // a logit has to be above it to be among the best
    int count = 0;
    auto flush = [&]() {
        wave_order();
        const uint64_t k = lane < count ? staged[wave][lane] : 0;
        keys = merge64(keys, sort64(k));
        const int rest = count - 64;
        for (int i = lane; i < rest; i += 64) {         // move the rest up, 64 at a time
            const uint64_t m = staged[wave][64 + i];
            wave_order();
            staged[wave][i] = m;
        }
        wave_order();
        count = rest > 0 ? rest : 0;
        const uint64_t last = lane_key(keys, a.top - 1);
        if (last) above = value_of((uint32_t)(last >> 32));
    };
    for (int64_t c0 = first + wave * kScoreBlock; c0 < end; c0 += kWaves * kScoreBlock) {
        const int64_t c = c0 + lane * 8;
        f32x8 x;
        if (c + 8 <= end) {
            x = load8<DT>(a.logits, t * a.stride + c);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = c + i < end ? load1<DT>(a.logits, t * a.stride + c + i) : -INFINITY;
        }
        float top = x[0];
#pragma unroll
        for (int i = 1; i < 8; ++i) top = fmaxf(top, x[i]);
        if constexpr (TOP) {
            if (!begun) {
                // the top-th largest of the lanes' largest is a bound to begin with
                const uint64_t k = sort64(key_of(top == top ? top : -INFINITY, 0));
                const uint32_t o = (uint32_t)(lane_key(k, a.top - 1) >> 32);
                // the next value below it; below +0 that is not -0, which equals it
                if (o > order_of(-INFINITY)) above = value_of(o - (o == 0x80000000u ? 2 : 1));
            }
            if (__any(top > above)) {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const bool in = x[i] > above;
                    const uint64_t mask = __ballot(in);
                    if (in) staged[wave][count + __popcll(mask & ((1ull << lane) - 1))] = key_of(x[i], (uint32_t)(c + i));
                    count += __popcll(mask);
                }
                while (count >= 64) flush();
            }
        }
        begun = true;
        // the reference follows the largest logit only when it is far behind: sums
        // of e up to e^8 lose nothing
        top *= a.scale;
        if (s.sum == 0.f ? top > kFloor : top > s.ref + 8.f) {
            s = moved(s, fminf(top, -kFloor));
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float d = (x[i] * a.scale - s.ref) * kLog2e, e = exp_of(d);
            s.sum += e;
            s.mean += e * fmaxf(d, -200.f);
        }
    }
    if constexpr (TOP) {
        if (count) flush();
        best[wave][lane] = keys;
    }
#pragma unroll
    for (int d = 1; d < 64; d *= 2) s = join_stats(s, shuffled(s, d));
    if (lane == 0) part[wave] = s;
    __syncthreads();
    if (wave) return;
    s = part[0];
#pragma unroll
    for (int i = 1; i < kWaves; ++i) s = join_stats(s, part[i]);
    if constexpr (TOP) {
#pragma unroll
        for (int i = 1; i < kWaves; ++i) keys = merge64(keys, best[i][lane]);
    }
    if (f.stats) {
        if (lane == 0) f.stats[blockIdx.x] = make_float4(s.ref, s.sum, s.mean, 0.f);
        if (TOP && lane < a.top) f.keys[(int64_t)blockIdx.x * a.top + lane] = keys;
    } else {
        if (lane == 0) put_token(a, t, s);
        if (TOP) put_top(a, t, s, keys);
    }
}

// The segments of a row: each wave joins a share of them, then the waves' parts.
constexpr int kJoinWaves = 8;
template <bool TOP>
__global__ __launch_bounds__(kJoinWaves * 64) void scores_join_kernel(ForwardArgs f) {
    __shared__ uint64_t best[kJoinWaves][64];
    __shared__ Stats part[kJoinWaves];
    const int lane = threadIdx.x % 64, wave = threadIdx.x / 64;
    const int64_t t = blockIdx.x;
    Stats s{kFloor, 0.f, 0.f};
    uint64_t keys = 0;
    for (int i = wave; i < f.splits; i += kJoinWaves) {
        const float4 v = f.stats[t * f.splits + i];
        s = join_stats(s, Stats{v.x, v.y, v.z});
        if (TOP) keys = merge64(keys, lane < f.a.top ? f.keys[(t * f.splits + i) * f.a.top + lane] : 0);
    }
    if (lane == 0) part[wave] = s;
    best[wave][lane] = keys;
    __syncthreads();
    if (wave) return;
    for (int i = 1; i < kJoinWaves; ++i) {
        s = join_stats(s, part[i]);
        if (TOP) keys = merge64(keys, best[i][lane]);
    }
    if (lane == 0) put_token(f.a, t, s);
    if (TOP) put_top(f.a, t, s, keys);
}

// ------------------------------------------------------------------ gradient --
constexpr int kGradBlock = 256 * 8;
template <int DT>
__global__ __launch_bounds__(256) void scores_grad_kernel(ScoreArgs a, int64_t first_row, int32_t blocks) {
    const int64_t t = first_row + blockIdx.x / blocks;
    const int64_t c = (int64_t)(blockIdx.x % blocks) * kGradBlock + threadIdx.x * 8;
    if (c >= a.vocab) return;
    const int32_t id = a.ids && a.dlogprob ? token_at(a.ids, a.id_bytes, t, a.vocab) : -1;
    const float g = id >= 0 ? a.dlogprob[t] : 0.f, h = a.dentropy ? a.dentropy[t] : 0.f;
    const float lse = a.lse[t], base = a.dentropy ? g + h * a.entropy[t] : g;
    const bool none = lse < -1e30f;     // a row whose logits are all masked
    auto one = [&](float x, int64_t v) {
        const float logp = x * a.scale - lse, p = exp_of(logp * kLog2e);
        float d = p * (base + h * fmaxf(logp, -200.f));
        d = (v == id ? g : 0.f) - d;
        return none ? 0.f : d * a.scale;
    };
    const int64_t e = t * a.stride + c, o = t * a.dstride + c;
    if (c + 8 <= a.vocab) {
        f32x8 x = load8<DT>(a.logits, e);
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = one(x[i], c + i);
        store8<DT>(a.dlogits, o, x);
    } else {
        for (int64_t i = 0; i < a.vocab - c; ++i) store1<DT>(a.dlogits, o + i, one(load1<DT>(a.logits, e + i), c + i));
    }
}

template <int DT>
void forward(const ForwardArgs& f, int64_t groups, hipStream_t stream) {
    if (f.a.top) scores_kernel<DT, true><<<(unsigned)groups, kThreads, 0, stream>>>(f);
    else scores_kernel<DT, false><<<(unsigned)groups, kThreads, 0, stream>>>(f);
}

}  // namespace

hipError_t launch_logprobs(const ScoreArgs& a, void* ws, hipStream_t stream) {
    const ScoreShape s = score_shape(a.tokens, a.vocab, a.top);
    // with splits there are 1,024 workgroups at most
    launch_groups(a.tokens * s.splits, [&](int64_t first, int64_t count) {
        ForwardArgs f{};
        f.a = a;
        f.segment = s.segment;
        f.splits = s.splits;
        if (s.splits > 1) {
            f.stats = static_cast<float4*>(ws);
            f.keys = reinterpret_cast<uint64_t*>(f.stats + a.tokens * s.splits);
        } else {
            const int64_t bytes = a.dtype == ZSMR_FP32 ? 4 : 2;
            f.a.logits = static_cast<const char*>(a.logits) + first * a.stride * bytes;
            if (a.ids) f.a.ids = static_cast<const char*>(a.ids) + first * a.id_bytes;
            if (a.logprob) f.a.logprob += first;
            if (a.lse) f.a.lse += first;
            if (a.entropy) f.a.entropy += first;
            if (a.top_ids) f.a.top_ids = static_cast<char*>(a.top_ids) + first * a.top * a.top_bytes;
            if (a.top_logprobs) f.a.top_logprobs += first * a.top;
        }
        if (a.dtype == ZSMR_BF16) forward<ZSMR_BF16>(f, count, stream);
        else if (a.dtype == ZSMR_FP16) forward<ZSMR_FP16>(f, count, stream);
        else forward<ZSMR_FP32>(f, count, stream);
        if (s.splits > 1) {
            if (a.top) scores_join_kernel<true><<<(unsigned)a.tokens, kJoinWaves * 64, 0, stream>>>(f);
            else scores_join_kernel<false><<<(unsigned)a.tokens, kJoinWaves * 64, 0, stream>>>(f);
        }
    });
    return hipGetLastError();
}

hipError_t launch_logprobs_grad(const ScoreArgs& a, hipStream_t stream) {
    const int64_t blocks = (a.vocab + kGradBlock - 1) / kGradBlock;
    launch_rows(a.tokens, blocks * 256, [&](int64_t first, int64_t count) {
        const unsigned grid = (unsigned)(count * blocks);
        if (a.dtype == ZSMR_BF16) scores_grad_kernel<ZSMR_BF16><<<grid, 256, 0, stream>>>(a, first, (int32_t)blocks);
        else if (a.dtype == ZSMR_FP16) scores_grad_kernel<ZSMR_FP16><<<grid, 256, 0, stream>>>(a, first, (int32_t)blocks);
        else scores_grad_kernel<ZSMR_FP32><<<grid, 256, 0, stream>>>(a, first, (int32_t)blocks);
    });
    return hipGetLastError();
}

}  // namespace zsmr
