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

constexpr float kLog2e = 1.44269504f, kLn2 = 0.69314718f;
constexpr float kEdge = 2.3e38f * kLog2e;

// ---------------------------------------------------------------- statistics --
// Logits are taken times scale * log2 e, so that e^z is a power of two of one fused
// multiply-add: d = x c - ref.  A part of a softmax is its reference (finite), the sum
// of 2^d and the sum of 2^d d.  A reference follows the largest logit only when a lane's
// eight powers pass 2^10: their sizes cost no accuracy, and no maximum has to be taken.
//
// A reference is the product x c of a logit x, rounded to fp32: for x itself d is that
// rounding and not 0.  References of the streaming pass stay within kNear, where it is a
// 32nd at most; logits far below that add nothing there, logits far above an infinity.
// What is left without a sum, or with a huge one, is a row (or a segment of one) far from
// zero, and a second pass takes its largest logit with the product's other part, `low`:
// d = x c - ref - low.  From 3e9 on the power of that part is infinite or zero.
struct Ref {
    float ref, low;
};
struct Stats {
    float ref, low, sum, mean;
};
constexpr float kNear = 0x1p20f, kTinySum = 0x1p-64f, kHugeSum = 0x1p64f;
__device__ __forceinline__ float power_of(float d) { return __builtin_amdgcn_exp2f(d); }
__device__ __forceinline__ float log2_of(float x) { return __builtin_amdgcn_logf(x); }
__device__ __forceinline__ float fused(float a, float b, float c) { return __builtin_fmaf(a, b, c); }
// FAR: references may have a low part.
template <bool FAR>
__device__ __forceinline__ Stats moved(Stats a, Ref to) {
    // a part without a sum (no logit above -infinity) has any reference
    if (a.sum == 0.f) return Stats{to.ref, to.low, 0.f, 0.f};
    const float d = FAR ? a.ref - to.ref + (a.low - to.low) : a.ref - to.ref, f = power_of(d);
    // an infinite sum, of logits past the range, stays one
    const float sum = FAR && a.sum == INFINITY ? a.sum : a.sum * f;
    return Stats{to.ref, to.low, sum, f == 0.f ? 0.f : f * fused(d, a.sum, a.mean)};
}
template <bool FAR>
__device__ __forceinline__ Stats join_stats(Stats a, Stats b) {
    const bool larger = FAR ? b.ref > a.ref || (b.ref == a.ref && b.low > a.low) : b.ref > a.ref;
    const bool to_b = a.sum == 0.f || (b.sum != 0.f && larger);
    const Ref to{to_b ? b.ref : a.ref, FAR ? to_b ? b.low : a.low : 0.f};
    a = moved<FAR>(a, to);
    b = moved<FAR>(b, to);
    return Stats{to.ref, to.low, a.sum + b.sum, a.mean + b.mean};
}
// Eight logits of a lane.
template <bool FAR>
__device__ __forceinline__ void add_powers(const f32x8& x, float c, Ref to, float* sum, float* mean) {
    float s = 0.f, m = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        float d = fused(x[i], c, -to.ref);
        if (FAR) d -= to.low;
        const float e = power_of(d);
        s += e;
        m = fused(e, fmaxf(d, -200.f), m);      // 0 times -infinity is 0
    }
    *sum = s;
    *mean = m;
}
__device__ __forceinline__ float largest(const f32x8& x) {
    float top = x[0];
#pragma unroll
    for (int i = 1; i < 8; ++i) top = fmaxf(top, x[i]);
    return top;
}
__device__ __forceinline__ float reference(float top, float c) { return __builtin_amdgcn_fmed3f(top * c, -kNear, kNear); }
__device__ __forceinline__ Ref far_reference(float top, float c) {
    const float product = top * c;
    return Ref{__builtin_amdgcn_fmed3f(product, -kEdge, kEdge), fabsf(product) <= kEdge ? fused(top, c, -product) : 0.f};
}
__device__ __forceinline__ void add_logits(Stats& s, const f32x8& x, float c) {
    float sum, mean;
    add_powers<false>(x, c, Ref{s.ref, 0.f}, &sum, &mean);
    if (sum > 1024.f) {
        const float ref = reference(largest(x), c);
        if (ref > s.ref) {
            s = moved<false>(s, Ref{ref, 0.f});
            add_powers<false>(x, c, Ref{ref, 0.f}, &sum, &mean);
        }
    }
    s.sum += sum;
    s.mean += mean;
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
// The value of the lane whose number differs in bits D, by moves between lanes.
template <int D>
__device__ __forceinline__ uint32_t across(uint32_t x) {
#if defined(__HIP_DEVICE_COMPILE__)
    const int lane = threadIdx.x % 64;
    if constexpr (D == 1) return __builtin_amdgcn_update_dpp(x, x, 0xb1, 0xf, 0xf, true);          // quad_perm 1 0 3 2
    if constexpr (D == 2) return __builtin_amdgcn_update_dpp(x, x, 0x4e, 0xf, 0xf, true);          // quad_perm 2 3 0 1
    if constexpr (D == 3) return __builtin_amdgcn_update_dpp(x, x, 0x1b, 0xf, 0xf, true);          // quad_perm 3 2 1 0
    if constexpr (D == 7) return __builtin_amdgcn_update_dpp(x, x, 0x141, 0xf, 0xf, true);         // row_half_mirror
    if constexpr (D == 4) return across<3>(across<7>(x));
    if constexpr (D == 8) return __builtin_amdgcn_update_dpp(x, x, 0x128, 0xf, 0xf, true);         // row_ror 8
    if constexpr (D == 15) return __builtin_amdgcn_update_dpp(x, x, 0x140, 0xf, 0xf, true);        // row_mirror
    if constexpr (D == 16) {
        const auto r = __builtin_amdgcn_permlane16_swap(x, x, false, false);
        return lane & 16 ? r[0] : r[1];
    }
    if constexpr (D == 32) {
        const auto r = __builtin_amdgcn_permlane32_swap(x, x, false, false);
        return lane & 32 ? r[0] : r[1];
    }
    if constexpr (D == 63) return across<32>(across<16>(across<15>(x)));
#endif
    return x;
}
template <int D>
__device__ __forceinline__ uint64_t across(uint64_t k) {
    return (uint64_t)across<D>((uint32_t)(k >> 32)) << 32 | across<D>((uint32_t)k);
}
template <int D>
__device__ __forceinline__ float across(float x) {
    return __uint_as_float(across<D>(__float_as_uint(x)));
}
__device__ __forceinline__ uint64_t lane_key(uint64_t k, int lane) {
    return (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(k >> 32), lane) << 32 | (uint32_t)__builtin_amdgcn_readlane((int)k, lane);
}
// LDS that the lanes of one wave exchange: its operations are in order, the
// compiler has to keep them so.
__device__ __forceinline__ void wave_order() {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}
// One key a lane, largest first: bitonic.
template <int N, int D, typename K>
__device__ __forceinline__ K sort_steps(K k) {
    const int lane = threadIdx.x % 64;
    const K o = across<D>(k);
    k = (k > o) == (((lane & D) == 0) == ((lane & N) == 0)) ? k : o;
    if constexpr (D > 1) return sort_steps<N, D / 2>(k);
    else return k;
}
template <typename K>
__device__ __forceinline__ K sort64(K k) {
    k = sort_steps<2, 1>(k);
    k = sort_steps<4, 2>(k);
    k = sort_steps<8, 4>(k);
    k = sort_steps<16, 8>(k);
    k = sort_steps<32, 16>(k);
    return sort_steps<64, 32>(k);
}
// The 64 largest of two sorted lists, sorted.
__device__ __forceinline__ uint64_t merge64(uint64_t a, uint64_t b) {
    b = across<63>(b);
    return sort_steps<64, 32>(a > b ? a : b);
}
// The largest of a group of `lanes` (a power of two up to 8) lanes.
template <int D = 1>
__device__ __forceinline__ float largest_of(float x, int lanes) {
    if (D < lanes) x = fmaxf(x, across<D>(x));
    if constexpr (D < 4) return largest_of<D * 2>(x, lanes);
    else return x;
}
template <int D>
__device__ __forceinline__ Stats joined(Stats s) {
    s = join_stats<false>(s, Stats{across<D>(s.ref), 0.f, across<D>(s.sum), across<D>(s.mean)});
    if constexpr (D < 32) return joined<D * 2>(s);
    else return s;
}
template <int D = 1>
__device__ __forceinline__ float wave_largest(float x) {
    x = fmaxf(x, across<D>(x));
    if constexpr (D < 32) return wave_largest<D * 2>(x);
    else return x;
}
template <int D = 1>
__device__ __forceinline__ float wave_sum(float x) {
    x += across<D>(x);
    if constexpr (D < 32) return wave_sum<D * 2>(x);
    else return x;
}

// ------------------------------------------------------------------- forward --
struct ForwardArgs {
    ScoreArgs a;
    float c;                    // scale * log2 e
    int64_t segment;
    int32_t splits;
    float4* stats;              // [token][split], or NULL: the results themselves
    uint64_t* keys;             // [token][split][top]
};

__device__ __forceinline__ void put_token(const ForwardArgs& f, int64_t t, Stats s) {
    const ScoreArgs& a = f.a;
    const float log_sum = log2_of(s.sum);
    const bool none = s.sum == 0.f;
    if (a.lse) a.lse[t] = none ? -INFINITY : (s.ref + (s.low + log_sum)) * kLn2;
    if (a.entropy) a.entropy[t] = none ? 0.f : (log_sum - s.mean / s.sum) * kLn2;
    if (a.logprob) {
        const int32_t id = token_at(a.ids, a.id_bytes, t, a.vocab);
        float r = 0.f;
        if (id >= 0) {
            const int64_t e = t * a.stride + id;
            const float x = a.dtype == ZSMR_BF16 ? load1<ZSMR_BF16>(a.logits, e) : a.dtype == ZSMR_FP16 ? load1<ZSMR_FP16>(a.logits, e) : load1<ZSMR_FP32>(a.logits, e);
            r = none ? -INFINITY : (fused(x, f.c, -s.ref) - s.low - log_sum) * kLn2;
        }
        a.logprob[t] = r;
    }
}
__device__ __forceinline__ void put_top(const ForwardArgs& f, int64_t t, Stats s, uint64_t key) {
    const ScoreArgs& a = f.a;
    const int lane = threadIdx.x % 64;
    if (lane >= a.top) return;
    const int64_t e = t * a.top + lane;
    const int32_t id = key ? (int32_t)(0xffffffffu - (uint32_t)key) : -1;
    if (a.top_ids) {
        if (a.top_bytes == 8) static_cast<int64_t*>(a.top_ids)[e] = id;
        else static_cast<int32_t*>(a.top_ids)[e] = id;
    }
    if (a.top_logprobs)
        a.top_logprobs[e] = key && s.sum != 0.f ? (fused(value_of((uint32_t)(key >> 32)), f.c, -s.ref) - s.low - log2_of(s.sum)) * kLn2 : -INFINITY;
}

// A wave's block of 512 logits, eight a lane: 16 bytes a lane and load, which covers a
// contiguous KB.
template <int DT>
struct Block {
    u32x4 raw[DT == ZSMR_FP32 ? 2 : 1];
    __device__ __forceinline__ static int index(int i) {        // of the lane's i-th, in the block
        const int lane = threadIdx.x % 64;
        return DT == ZSMR_FP32 ? i / 4 * 256 + lane * 4 + i % 4 : lane * 8 + i;
    }
    __device__ __forceinline__ void load(const void* p, int64_t e) {
        const int lane = threadIdx.x % 64;
        if constexpr (DT == ZSMR_FP32) {
            const float* q = static_cast<const float*>(p) + e + lane * 4;
            raw[0] = __builtin_bit_cast(u32x4, *reinterpret_cast<const f32x4_any*>(q));
            raw[1] = __builtin_bit_cast(u32x4, *reinterpret_cast<const f32x4_any*>(q + 256));
        } else {
            raw[0] = __builtin_bit_cast(u32x4, *reinterpret_cast<const u16x8_any*>(static_cast<const uint16_t*>(p) + e + lane * 8));
        }
    }
    __device__ __forceinline__ f32x8 values() const {
        f32x8 x;
        if constexpr (DT == ZSMR_FP32) {
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = __uint_as_float(raw[i / 4][i % 4]);
        } else {
            const u16x8 h = __builtin_bit_cast(u16x8, raw[0]);
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = widen16<DT>(h[i]);
        }
        return x;
    }
};

// 8,192 rows of 128,256 bf16: 377 to 413 us, 5.1 to 5.6 TB/s, of which the vector units' work
// on every logit (widen, multiply-add, power, two sums) takes nearly all cycles; 4,096 of fp32
// 360 us, 5.8 TB/s.  1,023 rows of 50,257 fp32 with 5 alternatives 41 us, 5.0 TB/s, where the
// vector work of a logit is more than twice that without them; 16 rows of 128,256 bf16 with
// 20 alternatives 9.6 and 7 for the join, latency.  Rows taken a second time, 8,192 of 128,256:
// 0.85 ms, or 0.59 where all is masked.
template <int DT, bool TOP, int kWaves>
__global__ __launch_bounds__(kWaves * 64, 8) void scores_kernel(ForwardArgs f) {
    const ScoreArgs& a = f.a;
    const int lane = threadIdx.x % 64, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    const int64_t t = blockIdx.x / f.splits;
    const int split = blockIdx.x % f.splits;
    const int64_t first = split * f.segment, end = first + f.segment < a.vocab ? first + f.segment : a.vocab;
    // Top alternatives.  A wave stages the logits above a bound, sorts them into its best
    // when enough have come, and shares the bound that follows with the other waves of
    // the row: what is below the top-th best of any of them is none of the row's.  The
    // order in which bounds arrive decides what is staged in vain, not what is found.
    constexpr int kStaged = TOP ? 64 + kScoreBlock : 1;
    __shared__ uint64_t staged[kWaves][kStaged];
    __shared__ uint32_t shared_bound, counts[kWaves];
    __shared__ uint32_t groups[64];
    __shared__ Stats part[kWaves];

    Stats s{-kNear, 0.f, 0.f, 0.f};
    bool sorted = false;
    uint64_t keys = 0;                  // the wave's best, sorted
    float above = -INFINITY;            // a logit has to be above it to be among the best
    int count = 0;
    const int enough = a.top > 32 ? 64 : a.top > 8 ? 2 * a.top : 16;
    // the value below which a logit is not above one of order o: the next one below it, and
    // below +0 one that is not -0, which equals it
    auto below = [](uint32_t o) { return o - (o == 0x80000000u ? 2 : 1); };
    auto share = [&](uint32_t o) {
        if (lane == 0) atomicMax(&shared_bound, o);
    };
    auto flush = [&]() {
        wave_order();
        uint64_t k = sort64(lane < count ? staged[wave][lane] : 0);
        keys = sorted ? merge64(keys, k) : k;
        sorted = true;
        const int rest = count - 64;
        for (int i = lane; i < rest; i += 64) {         // move the rest up, 64 at a time
            k = staged[wave][64 + i];
            wave_order();
            staged[wave][i] = k;
        }
        wave_order();
        count = rest > 0 ? rest : 0;
        const uint64_t last = lane_key(keys, a.top - 1);
        if (last) {
            // later logits of this wave have larger indices: an equal one is not among the best
            above = fmaxf(above, value_of((uint32_t)(last >> 32)));
            share(below((uint32_t)(last >> 32)));
        }
    };
    auto offer = [&](const f32x8& x, int64_t c0) {
        const float top = largest(x);
        if (!__any(top > above)) return;
        // the row's bound is asked for only where the wave's own is passed
        wave_order();
        above = fmaxf(above, value_of(*(volatile uint32_t*)&shared_bound));
        if (!__any(top > above)) return;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const bool in = x[i] > above;
            const uint64_t mask = __ballot(in);
            if (mask == 0) continue;
            if (in) staged[wave][count + __popcll(mask & ((1ull << lane) - 1))] = key_of(x[i], (uint32_t)(c0 + Block<DT>::index(i)));
            count += __popcll(mask);
        }
        while (count >= enough) flush();
    };
    // whole blocks, the next two on their way
    const int64_t row = t * a.stride, step = kWaves * kScoreBlock;
    int64_t c0 = first + wave * kScoreBlock;
    const bool whole = c0 + kScoreBlock <= end;
    Block<DT> now, next, after;
    float top = -INFINITY;
    if (whole) {
        now.load(a.logits, row + c0);
        if (c0 + step + kScoreBlock <= end) next.load(a.logits, row + c0 + step);
        if (c0 + 2 * step + kScoreBlock <= end) after.load(a.logits, row + c0 + 2 * step);
        top = largest(now.values());
        s.ref = reference(top, f.c);
    }
    if constexpr (TOP) {
        // A bound to begin with: the top-th largest of the largest of 64 groups of logits,
        // taken from the waves' first blocks (from all eight waves, where they have one,
        // groups of 64: for 5 alternatives about 5 of their 4,096 logits are above it, for
        // 20 24).
        const int64_t blocks = (end - first) / kScoreBlock;
        int waves = kWaves;
        while (waves > 1 && waves > blocks) waves /= 2;
        const float group = largest_of(top == top ? top : -INFINITY, waves);
        if (wave < waves && lane % waves == 0) groups[wave * (64 / waves) + lane / waves] = order_of(group);
        if (threadIdx.x == 0) shared_bound = order_of(-INFINITY);
        __syncthreads();
        const uint32_t o = __builtin_amdgcn_readlane(sort64(groups[lane]), a.top - 1);
        if (o > order_of(-INFINITY)) {
            above = value_of(below(o));
            if (wave == 0) share(below(o));
        }
    }
    if (whole)
        for (; c0 + kScoreBlock <= end; c0 += step) {
            const f32x8 x = now.values();
            now = next;
            next = after;
            if (c0 + 3 * step + kScoreBlock <= end) after.load(a.logits, row + c0 + 3 * step);
            if constexpr (TOP) offer(x, c0);
            add_logits(s, x, f.c);
        }
    if (c0 < end) {             // the row's last, shorter one
        f32x8 x;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int64_t c = c0 + Block<DT>::index(i);
            x[i] = c < end ? load1<DT>(a.logits, row + c) : -INFINITY;
        }
        if (!whole) s.ref = reference(largest(x), f.c);
        if constexpr (TOP) offer(x, c0);
        add_logits(s, x, f.c);
    }
    s = joined<1>(s);
    if (lane == 0) part[wave] = s;
    __syncthreads();
    bool tiny = true, huge = false;
#pragma unroll
    for (int i = 0; i < kWaves; ++i) {
        tiny = tiny && part[i].sum < kTinySum;
        huge = huge || part[i].sum > kHugeSum;
    }
    if (tiny || huge) {         // far from zero, or masked: again, from the largest logit
        auto blocks = [&](auto each) {
            for (int64_t c = first + wave * kScoreBlock; c < end; c += step) {
                f32x8 x;
                if (c + kScoreBlock <= end) {
                    now.load(a.logits, row + c);
                    x = now.values();
                } else {
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const int64_t e = c + Block<DT>::index(i);
                        x[i] = e < end ? load1<DT>(a.logits, row + e) : -INFINITY;
                    }
                }
                each(x);
            }
        };
        float top = -INFINITY;
        blocks([&](const f32x8& x) { top = fmaxf(top, largest(x)); });
        top = wave_largest(top);
        __syncthreads();        // every wave has read the sums
        if (lane == 0) part[wave].ref = top;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kWaves; ++i) top = fmaxf(top, part[i].ref);
        const Ref to = far_reference(top, f.c);
        float sum = 0.f, mean = 0.f;
        if (top * f.c >= -kEdge)        // else nothing but masks
            blocks([&](const f32x8& x) {
                float e, m;
                add_powers<true>(x, f.c, to, &e, &m);
                sum += e;
                mean += m;
            });
        sum = wave_sum(sum);
        mean = wave_sum(mean);
        __syncthreads();        // every wave has read the largest
        if (lane == 0) part[wave] = Stats{to.ref, to.low, sum, mean};
        __syncthreads();
    }
    if constexpr (TOP) {
        // what is above the last bound, of the staged and of the best, to the front
        const uint32_t bound = shared_bound;
        wave_order();
        const uint64_t k = lane < count ? staged[wave][lane] : 0;
        wave_order();
        count = 0;
        for (const uint64_t m : {k, keys}) {
            const bool in = (uint32_t)(m >> 32) > bound;
            const uint64_t mask = __ballot(in);
            if (in) staged[wave][count + __popcll(mask & ((1ull << lane) - 1))] = m;
            count += __popcll(mask);
        }
        if (lane == 0) counts[wave] = count;
        __syncthreads();
        if (wave) return;
        // the first wave sorts what all have
        int all = 0;
#pragma unroll
        for (int w = 0; w < kWaves; ++w) all += counts[w];
        for (int at = 0; at < all; at += 64) {
            int w = 0, i = at + lane;
#pragma unroll
            for (int n = 0; n < kWaves - 1; ++n)
                if (w == n && i >= (int)counts[n]) {
                    i -= (int)counts[n];
                    ++w;
                }
            const uint64_t m = sort64(at + lane < all ? staged[w][i] : 0);
            keys = at ? merge64(keys, m) : m;
        }
        if (!all) keys = 0;
    }
    if (wave) return;
    s = part[0];
    // references are one value, or have no low part
#pragma unroll
    for (int i = 1; i < kWaves; ++i) s = join_stats<false>(s, part[i]);
    s.low = part[0].low;
    if (f.stats) {
        if (lane == 0) f.stats[blockIdx.x] = make_float4(s.ref, s.low, s.sum, s.mean);
        if (TOP && lane < a.top) f.keys[(int64_t)blockIdx.x * a.top + lane] = keys;
    } else {
        if (lane == 0) put_token(f, t, s);
        if (TOP) put_top(f, t, s, keys);
    }
}

// The segments of a row: each wave joins a share of them, then pairs of waves.
constexpr int kJoinWaves = 8;
template <bool TOP>
__global__ __launch_bounds__(kJoinWaves * 64) void scores_join_kernel(ForwardArgs f) {
    __shared__ uint64_t best[kJoinWaves][64];
    __shared__ Stats part[kJoinWaves];
    const int lane = threadIdx.x % 64, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    const int64_t t = blockIdx.x;
    Stats s{-kEdge, 0.f, 0.f, 0.f};
    uint64_t keys = 0;
    for (int i = wave; i < f.splits; i += kJoinWaves) {
        const float4 v = f.stats[t * f.splits + i];
        s = join_stats<true>(s, Stats{v.x, v.y, v.z, v.w});
        if (TOP) keys = merge64(keys, lane < f.a.top ? f.keys[(t * f.splits + i) * f.a.top + lane] : 0);
    }
    if (lane == 0) part[wave] = s;
    if (TOP) best[wave][lane] = keys;
#pragma unroll
    for (int n = 1; n < kJoinWaves; n *= 2) {
        __syncthreads();
        if (TOP && wave % (2 * n) == 0) best[wave][lane] = keys = merge64(keys, best[wave + n][lane]);
    }
    if (wave) return;
    s = part[0];
#pragma unroll
    for (int i = 1; i < kJoinWaves; ++i) s = join_stats<true>(s, part[i]);
    if (lane == 0) put_token(f, t, s);
    if (TOP) put_top(f, t, s, keys);
}

// ------------------------------------------------------------------ gradient --
// A workgroup takes kGradBlock elements of a row; what is the row's own is read once.
// 8,192 rows of 128,256 bf16: 680 to 750 us, 5.6 to 6.2 TB/s; 4,096 of fp32 808, 5.2 TB/s.
// ds = g' [v = id] - p (g' + h' (log p + H)) with g' = scale g and h' = scale h, log p in
// the base 2 that the power needs.
//
// log p = scale s - lse has one rounding of its own, but lse, rounded to fp32, is off by up
// to 4.3 * 2^-24 of its size (its constant, reference, sum and product with ln 2), and p
// by as much: at 512 and 4,096 a quarter of what fp16's and bf16's results may be off, at 64
// 1.6e-5.  A row further from zero than that gets the sum again from its largest logit, by
// one workgroup that then writes all of it; at -1e9 lse holds no log p at all.
template <int DT>
constexpr float kFarLse = DT == ZSMR_FP32 ? 64.f : DT == ZSMR_FP16 ? 512.f : 4096.f;
constexpr int kGradThreads = 256, kGradTurns = 4, kGradBlock = kGradThreads * kGradTurns * 8;
struct GradArgs {
    ScoreArgs a;
    float c;                        // scale * log2 e
    int64_t last_row;               // rows go from the last one up: the forward pass read them last
    int32_t blocks;                 // of a row
};
// A whole row by one workgroup: the largest logit, the sum, then the results, which may
// take the logits' place.  8,192 such rows of 128,256 bf16 take 1.58 ms (others 0.69), 16
// of them 31 us (5).
template <int DT, typename F>
__device__ __forceinline__ void far_row(const ScoreArgs& a, float c, int64_t t, int32_t id, float g, F slope_at) {
    __shared__ float part[2][kGradThreads / 64];
    const int64_t row = t * a.stride, to = t * a.dstride;
    auto every = [&](auto each) {
        int64_t v = threadIdx.x * 8;
        for (; v - threadIdx.x * 8 + kGradBlock <= a.vocab; v += kGradBlock) {
            f32x8 x[kGradTurns];
#pragma unroll
            for (int k = 0; k < kGradTurns; ++k) x[k] = load8<DT>(a.logits, row + v + k * kGradThreads * 8);
#pragma unroll
            for (int k = 0; k < kGradTurns; ++k) each(v + k * kGradThreads * 8, 8, x[k]);
        }
        for (; v < a.vocab; v += kGradThreads * 8) {
            const int count = (int)min((int64_t)8, a.vocab - v);
            f32x8 x = -INFINITY;
            if (count == 8) {
                x = load8<DT>(a.logits, row + v);
            } else {
#pragma unroll
                for (int i = 0; i < 7; ++i)
                    if (i < count) x[i] = load1<DT>(a.logits, row + v + i);
            }
            each(v, count, x);
        }
    };
    const int wave = threadIdx.x / 64;
    float top = -INFINITY, sum = 0.f;
    every([&](int64_t, int, const f32x8& x) { top = fmaxf(top, largest(x)); });
    top = wave_largest(top);
    if (threadIdx.x % 64 == 0) part[0][wave] = top;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kGradThreads / 64; ++i) top = fmaxf(top, part[0][i]);
    every([&](int64_t, int, const f32x8& x) {
#pragma unroll
        for (int i = 0; i < 8; ++i) sum += power_of((x[i] - top) * c);
    });
    sum = wave_sum(sum);
    if (threadIdx.x % 64 == 0) part[1][wave] = sum;
    __syncthreads();
    sum = part[1][0];
#pragma unroll
    for (int i = 1; i < kGradThreads / 64; ++i) sum += part[1][i];
    const float log_sum = log2_of(sum);
    every([&](int64_t v, int count, const f32x8& x) {
        f32x8 d;
#pragma unroll
        for (int i = 0; i < 8; ++i) d[i] = slope_at((x[i] - top) * c - log_sum) + (v + i == id ? g : 0.f);
        if (count == 8) {
            store8<DT>(a.dlogits, to + v, d);
        } else {
#pragma unroll
            for (int i = 0; i < 7; ++i)
                if (i < count) store1<DT>(a.dlogits, to + v + i, d[i]);
        }
    });
}
// Six waves a SIMD: with eight the same rows take 0.76 ms, with five 0.77.
template <int DT, bool STREAM>
__global__ __launch_bounds__(kGradThreads, 6) void scores_grad_kernel(GradArgs f) {
    const ScoreArgs& a = f.a;
    const int64_t t = f.last_row - blockIdx.x / f.blocks, c0 = (int64_t)(blockIdx.x % f.blocks) * kGradBlock;
    const int32_t id = a.ids && a.dlogprob ? token_at(a.ids, a.id_bytes, t, a.vocab) : -1;
    const float g = id >= 0 ? a.dlogprob[t] * a.scale : 0.f, h = a.dentropy ? a.dentropy[t] * a.scale : 0.f;
    const float lse = a.lse[t], slope = h * kLn2, base = a.dentropy ? g + h * a.entropy[t] : g;
    const bool none = lse == -INFINITY; // a row whose logits are all masked
    auto slope_at = [&](float d) { return -power_of(d) * fused(slope, fmaxf(d, -200.f), base); };
    if (fabsf(lse) > kFarLse<DT> && fabsf(lse) < INFINITY) {
        // another block of every row: a row's first ones may all be on one XCD
        if (blockIdx.x % f.blocks == t % f.blocks) far_row<DT>(a, f.c, t, id, g, slope_at);
        return;
    }
    auto one = [&](float x) { return slope_at(fused(x, a.scale, -lse) * kLog2e); };
    const int64_t e0 = t * a.stride + c0, o0 = t * a.dstride + c0;
    const int64_t left = a.vocab - c0;
    f32x8 x[kGradTurns];
#pragma unroll
    for (int k = 0; k < kGradTurns; ++k) {
        const int64_t c = (k * kGradThreads + threadIdx.x) * 8;
        if (c + 8 <= left) x[k] = load8<DT>(a.logits, e0 + c);
    }
#pragma unroll
    for (int k = 0; k < kGradTurns; ++k) {
        const int64_t c = (k * kGradThreads + threadIdx.x) * 8;
        if (c >= left) break;
        if (c + 8 <= left) {
#pragma unroll
            for (int i = 0; i < 8; ++i) x[k][i] = none ? 0.f : one(x[k][i]);
            const int64_t at = id - c0 - c;
            if (at >= 0 && at < 8 && !none) {
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (i == at) x[k][i] += g;
            }
            if constexpr (STREAM) stream8<DT>(a.dlogits, o0 + c, x[k]);
            else store8<DT>(a.dlogits, o0 + c, x[k]);
        } else {
            for (int64_t i = c; i < left; ++i) {
                const float d = none ? 0.f : one(load1<DT>(a.logits, e0 + i)) + (c0 + i == id ? g : 0.f);
                store1<DT>(a.dlogits, o0 + i, d);
            }
        }
    }
}

template <int DT, int WAVES>
void forward(const ForwardArgs& f, int64_t groups, hipStream_t stream) {
    if (f.a.top) scores_kernel<DT, true, WAVES><<<(unsigned)groups, WAVES * 64, 0, stream>>>(f);
    else scores_kernel<DT, false, WAVES><<<(unsigned)groups, WAVES * 64, 0, stream>>>(f);
}
template <int DT>
void forward(const ForwardArgs& f, int64_t groups, int waves, hipStream_t stream) {
    if (waves == 2) forward<DT, 2>(f, groups, stream);
    else forward<DT, 8>(f, groups, stream);
}

template <int DT>
void gradient(const GradArgs& f, unsigned grid, bool stream_out, hipStream_t stream) {
    if (stream_out) scores_grad_kernel<DT, true><<<grid, kGradThreads, 0, stream>>>(f);
    else scores_grad_kernel<DT, false><<<grid, kGradThreads, 0, stream>>>(f);
}

}  // namespace

hipError_t launch_logprobs(const ScoreArgs& a, void* ws, hipStream_t stream) {
    const ScoreShape s = score_shape(a.tokens, a.vocab, a.top);
    // with splits there are kScoreSplits workgroups at most, one launch
    score_launches(s, a.tokens, [&](int64_t first, int64_t count) {
        ForwardArgs f{};
        f.a = a;
        f.c = a.scale * kLog2e;
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
        if (a.dtype == ZSMR_BF16) forward<ZSMR_BF16>(f, count, s.waves, stream);
        else if (a.dtype == ZSMR_FP16) forward<ZSMR_FP16>(f, count, s.waves, stream);
        else forward<ZSMR_FP32>(f, count, s.waves, stream);
        if (s.splits > 1) {
            if (a.top) scores_join_kernel<true><<<(unsigned)a.tokens, kJoinWaves * 64, 0, stream>>>(f);
            else scores_join_kernel<false><<<(unsigned)a.tokens, kJoinWaves * 64, 0, stream>>>(f);
        }
    });
    return hipGetLastError();
}

hipError_t launch_logprobs_grad(const ScoreArgs& a, hipStream_t stream) {
    GradArgs f{};
    f.a = a;
    f.c = a.scale * kLog2e;
    f.blocks = (int32_t)((a.vocab + kGradBlock - 1) / kGradBlock);
    // results that the 256 MB Infinity Cache cannot hold beside the logits go past it
    const bool stream_out = a.tokens * a.vocab * (a.dtype == ZSMR_FP32 ? 8 : 4) > (int64_t(200) << 20);
    launch_rows(a.tokens, (int64_t)f.blocks * kGradThreads, [&](int64_t first, int64_t count) {
        const unsigned grid = (unsigned)(count * f.blocks);
        f.last_row = a.tokens - 1 - first;
        if (a.dtype == ZSMR_BF16) gradient<ZSMR_BF16>(f, grid, stream_out, stream);
        else if (a.dtype == ZSMR_FP16) gradient<ZSMR_FP16>(f, grid, stream_out, stream);
        else gradient<ZSMR_FP32>(f, grid, stream_out, stream);
    });
    return hipGetLastError();
}

}  // namespace zsmr
