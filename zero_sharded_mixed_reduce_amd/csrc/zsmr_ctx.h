// The context behind a zsmr_ctx* and the checks and counting that every host
// file of the C ABI shares.  Internal, not part of the public ABI.
#pragma once
#include <cmath>
#include <cstdint>
#include <vector>

#include "zsmr.h"
#include "zsmr_launch.h"

struct zsmr_ctx {
    int64_t numel = 0;
    int32_t world = 0, stage = 0, gdt = 0, pdt = 0, pad = 0;
    std::vector<int64_t> units;        // true unit sizes
    std::vector<int64_t> shard_u;      // S_u (stage 3); {S} stages 1-2; {Psi} DP; P_u (stage 4)
    std::vector<int64_t> unit_pstart;  // padded start Q_u (stage 3); unit start (stage 4); {0} otherwise
    std::vector<int64_t> local_off;    // offset of unit u's piece in its holder's shard
    std::vector<int32_t> owners;       // stage 4: the rank owning each unit
    std::vector<int64_t> own;          // stage 4: elements each rank owns
    int64_t padded = 0, shard_total = 0;
    // counters per rank (elements): all-gathers received; reduce-scatters
    // received = sent at stages 1-3, sent at stage 4; all-reduce
    std::vector<int64_t> rs, ag, ar;
    // ZeRO-3 schedule (live and peak gathered bytes per rank: at stage 4 a
    // rank needs no buffer for its own units)
    std::vector<int64_t> gathers, releases;
    std::vector<char> live;
    int32_t max_live = 1, live_units = 0;
    std::vector<int64_t> live_bytes, peak_live_bytes;
};

namespace zsmr {

// Record a HIP error's text for zsmr_last_hip_error(); returns ZSMR_ERR_HIP.
int32_t hip_fail(hipError_t e);

inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

inline bool dtype_ok(int32_t d) { return d == ZSMR_FP16 || d == ZSMR_BF16; }

inline bool stage3(const zsmr_ctx* c) { return c->stage == ZSMR_ZERO3 || c->stage == ZSMR_ZERO3_OWNER; }

inline int n_pieces(const zsmr_ctx* c) { return stage3(c) ? (int)c->units.size() : 1; }

inline int32_t check_piece(const zsmr_ctx* c, int32_t rank, int32_t unit) {
    if (!c) return ZSMR_ERR_ARG;
    if (rank < 0 || rank >= c->world) return ZSMR_ERR_ARG;
    if (unit < 0 || unit >= n_pieces(c)) return ZSMR_ERR_ARG;
    return ZSMR_OK;
}

inline void piece(const zsmr_ctx* c, int32_t rank, int32_t unit, int64_t* off, int64_t* len, int64_t* loc) {
    int64_t o, l, lo;
    if (c->stage == ZSMR_DP) {
        o = 0;
        l = c->numel;
        lo = 0;
    } else if (c->stage == ZSMR_ZERO3_OWNER) {
        o = c->unit_pstart[unit];
        l = c->owners[unit] == rank ? c->units[unit] : 0;
        lo = c->local_off[unit];
    } else if (c->stage != ZSMR_ZERO3) {
        l = c->shard_u[0];
        o = (int64_t)rank * l;
        lo = 0;
    } else {
        l = c->shard_u[unit];
        o = c->unit_pstart[unit] + (int64_t)rank * l;
        lo = c->local_off[unit];
    }
    if (off) *off = o;
    if (len) *len = l;
    if (loc) *loc = lo;
}

inline bool al(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) % n) == 0; }

inline int32_t check_adam(const zsmr_adam* hp, int32_t t, zsmr::AdamK* k) {
    if (!hp || t < 1) return ZSMR_ERR_ARG;
    const double lr = hp->lr, b1 = hp->beta1, b2 = hp->beta2, eps = hp->eps;
    if (!std::isfinite(lr) || !std::isfinite(b1) || !std::isfinite(b2) || !std::isfinite(eps))
        return ZSMR_ERR_ARG;
    if (lr < 0 || b1 < 0 || b1 >= 1 || b2 < 0 || b2 >= 1 || eps < 0) return ZSMR_ERR_ARG;
    // Each constant is a double expression rounded to fp32 once ("The four
    // schemes", Base._adam uses Python scalars against fp32 arrays).
    k->c1 = (float)b1;
    k->c1m = (float)(1.0 - b1);
    k->c2 = (float)b2;
    k->c2m = (float)(1.0 - b2);
    k->bc1 = (float)(1.0 - std::pow(b1, (double)t));
    k->bc2 = (float)(1.0 - std::pow(b2, (double)t));
    k->lr = (float)lr;
    k->eps = (float)eps;
    return ZSMR_OK;
}

// Counting of one reduce over (rank, unit) of `len` elements: a data-parallel
// replica takes part in one all-reduce of the whole vector; a sharded rank
// receives (N-1) peers' contributions to its piece (and sends as many); at
// stage 4 every other rank sends its contribution to the owner.
inline void count_reduce(zsmr_ctx* c, int32_t rank, int64_t len) {
    const int64_t w = c->world;
    if (c->stage == ZSMR_DP) {
        c->ar[rank] += 2 * (w - 1) * ceil_div(c->numel, w);
    } else if (c->stage == ZSMR_ZERO3_OWNER) {
        for (int32_t q = 0; q < c->world; ++q)
            if (q != rank) c->rs[q] += len;
    } else {
        c->rs[rank] += (w - 1) * len;
    }
}

// Counting of one cast of (rank, unit): at stages 1-2 the all-gather delivers
// the rank's slot to every other rank; DP and stage 3 cast locally.
inline void count_cast(zsmr_ctx* c, int32_t rank, int64_t len) {
    if (c->stage == ZSMR_ZERO1 || c->stage == ZSMR_ZERO2)
        for (int32_t q = 0; q < c->world; ++q)
            if (q != rank) c->ag[q] += len;
}

inline int32_t check_grads(const zsmr_ctx* c, const void* grads, int64_t row_stride,
                           int64_t base, int64_t len) {
    if (!grads || base < 0 || row_stride < 0) return ZSMR_ERR_ARG;
    if (c->world > 1 && row_stride < len) return ZSMR_ERR_ARG;   // rows may not overlap
    if (!al(grads, 2)) return ZSMR_ERR_ALIGN;
    return ZSMR_OK;
}

// N as the divisor of the mean; for N a power of two also 1/N, which the
// kernels multiply by instead (the same bits).
inline void set_mean_divisor(zsmr::StepArgs& a, int32_t world) {
    a.nf = (float)world;
    a.inv_pow2 = world > 0 && (world & (world - 1)) == 0;
    a.inv_nf = a.inv_pow2 ? 1.0f / (float)world : 0.0f;
}

}  // namespace zsmr
