// What the orthogonalised update of zsmr_newton.hip launches for given sizes: the
// matrices of a group, the workspace, the powers of two that keep every matrix in
// fp16's range.  Host arithmetic only, so that it can be checked on any machine.
#pragma once
#include <stdint.h>

#include <algorithm>
#include <cmath>

#include "zsmr_ops.h"

namespace zsmr {

constexpr int kNsStep = 32;             // k of a step
constexpr int kNsThreads = 256;         // of a product's workgroup
constexpr int64_t kNsCus = 256;

inline int64_t ns_ceil(int64_t n, int64_t k) { return (n + k - 1) / k * k; }
inline int64_t ns_tiles(int64_t n, int64_t k) { return (n + k - 1) / k; }

// The wide orientation of a matrix: m <= n.  Rows are padded to whole steps.
struct NsShape {
    int64_t m, n, mp, np;
    bool tall;                          // the wide orientation is the transposed one
    int64_t count, group;               // matrices; of a group, whose launches they share
    int parts;                          // partial sums of squares of a matrix
    bool grouped;                       // steps may be taken in groups
    int small;                          // the form of a matrix that stays in LDS, or 0
};

// A group's matrices have 2^25 elements at most (or are one): enough to fill the
// CUs many times over, while the workspace stays below 1.0 GB for any count (104 x 129
// needs the most an element: 29.8 bytes, with rows padded to 128 and 160).
constexpr int64_t kNsGroupElems = int64_t(1) << 25;

// A matrix that fits a CU's LDS with its inner matrix is one workgroup's: every pass
// without a launch.  Up to 64 x 64 (1), 64 x 256 (2) and 128 x 128 (3).
inline int ns_small(int64_t m, int64_t n) {
    return m <= 64 ? n <= 64 ? 1 : n <= 256 ? 2 : 0 : n <= 128 ? 3 : 0;
}
// single: every step has its own product with X.
inline NsShape ns_shape(int64_t rows, int64_t cols, int64_t count, bool single) {
    NsShape s{};
    s.tall = rows > cols;
    s.m = std::min(rows, cols);
    s.n = std::max(rows, cols);
    s.mp = ns_ceil(s.m, kNsStep);
    s.np = ns_ceil(s.n, kNsStep);
    s.count = count;
    s.small = ns_small(s.m, s.n);
    // from n = 1.2 m on
    s.grouped = !s.small && !single && s.n * 5 >= s.m * 6;
    s.group = std::max<int64_t>(1, std::min({count, kNsGroupElems / (s.m * s.n), int64_t(1) << 14}));
    // a workgroup of the sums takes 2,048 elements at a time
    s.parts = (int)std::min<int64_t>((s.m * s.n + 2047) / 2048, std::max<int64_t>(1, 1024 / s.group));
    return s;
}

// ---- matrices that do not stay in LDS: a list of products ------------------------
// The matrices of the workspace.
enum : int { M_X0, M_X1, M_A, M_B, M_T, M_Q0, M_Q1, kNsMatrices };

// dst = old_mul * old + old2_mul * old2 + mul * (P Q): inner matrices, symmetric (P Q^T
// is the same); X' from X (P Q with P = X, whose rows are k); or the result.
enum : int { N_INNER, N_UPDATE, N_LAST };
struct NsOp {
    int32_t kind, p, q, old, old2, dst; // old, old2: -1 for none
    float mul, old_mul, old2_mul;
    int32_t paired;                     // the next product needs nothing of this one: one launch
};
// How the tiles of 128 x 128 of a product are computed: by four waves, two workgroups
// a CU (NS_WIDE); by eight, one a CU, each four half of the steps (NS_DEEP); in
// quarters of 64 x 64, by eight waves in the same way, with four stages of LDS
// (NS_THIN) or, two workgroups a CU, with two (NS_PAIR).
enum : int { NS_WIDE, NS_DEEP, NS_THIN, NS_PAIR };
inline bool ns_quarters(int form) { return form >= NS_THIN; }
struct NsPart {
    int form;
    int64_t first, count;               // tiles
};
struct NsGrid {
    int32_t p_tiles, q_tiles, tiles;    // of one matrix of one product
    int parts;                          // launches: one, or a second one for the last tiles
    NsPart part[2];
    int32_t split;                      // the steps' parts, whose sums a launch of their own adds up; or 1
    int32_t split_steps;                // of a part; the last one may have fewer
    double us;                          // what it takes
};
inline int64_t ns_groups(const NsPart& p) { return ns_quarters(p.form) ? p.count * 4 : p.count; }
// What a launch takes, in microseconds.  Measured on MI355X, products of m x m, from 10
// to 128 steps: a workgroup with a CU for itself 0.75, 0.58 and 0.21 us a step after
// 7.5, 8 and 5.5 us; under full load (where the power decides) 1.22 us for two wide
// tiles, 0.68 for a deep and 0.26 for a thin one, 0.4 for a pair (0.52
// in each of several rounds).  364 quarters of 50 steps: thin 28.2 us, in pairs 24.6; 78
// of 24: 9.6 and 12.3; 1,456 of 50: in pairs 77.5, 364 wide tiles 68.  Between one round and
// two this is too low: 650 and 676 wide tiles of 50 steps take 106 to 119 us and not 98.5,
// and two products of 91 tiles in one launch, deep, 45 and not 37.
inline double ns_cost(int form, int64_t tiles, int64_t steps) {
    const int64_t groups = ns_quarters(form) ? tiles * 4 : tiles, each = form == NS_WIDE || form == NS_PAIR ? 2 * kNsCus : kNsCus;
    const int64_t full = groups / each, rest = groups % each;
    if (form == NS_WIDE) return 7.5 + steps * (full * 1.22 + (rest > kNsCus ? 1.22 : rest > 0 ? (full ? 0.6 : 0.75) : 0));
    if (form == NS_DEEP) return 8 + steps * (full * 0.68 + (rest > 0 ? full ? 0.62 : 0.58 : 0));
    if (form == NS_PAIR) return 5.5 + steps * (full * 0.52 + (rest > kNsCus ? 0.4 : rest > 0 ? 0.28 : 0));
    return 5.5 + steps * (full + (rest > 0) > 1 ? (full + (rest > 0)) * 0.26 : 0.21);
}
// The form that ends soonest, for whole rounds over the CUs and, if that is sooner,
// another for what is left of the last round.  A symmetric product of 4,096 has 528
// tiles, 16 more than a round: all of them wide 225 us, the 16 in quarters 195.
//
// X X^T of a long X has more steps than tiles.  Its steps may be split: every part's tiles
// go to memory in fp32 (into X's other copy, free at that time), and ns_join_kernel adds
// them up.  1,600 x 6,400: 61 us and 10 to join 5 parts,
// 110 in one; 128 x 8,192: 9 and 7 for 16, 59 in one.
constexpr int kNsMaxSplit = 16;
constexpr int64_t kNsTileBytes = 128 * 128 * 4;
inline double ns_join_cost(int64_t tiles, int split) { return 5.5 + (double)(tiles * kNsTileBytes * split) * 1.7e-7; }
inline NsGrid ns_grid(const NsShape& s, int kind, int64_t products, int64_t steps, bool gram = false) {
    NsGrid g{};
    g.split = 1;
    g.split_steps = (int32_t)steps;
    g.p_tiles = (int32_t)ns_tiles(kind == N_INNER ? s.m : s.n, 128);
    g.q_tiles = (int32_t)ns_tiles(s.m, 128);
    g.tiles = kind == N_INNER ? g.q_tiles * (g.q_tiles + 1) / 2 : g.p_tiles * g.q_tiles;
    const int64_t all = g.tiles * products;
    double least = 0;
    auto best = [&](int64_t first, int64_t count) {
        NsPart p{NS_WIDE, first, count};
        double us = ns_cost(NS_WIDE, count, steps);
        for (int form : {NS_DEEP, NS_THIN, NS_PAIR}) {
            const double t = ns_cost(form, count, steps);
            if (t < us) {
                us = t;
                p.form = form;
            }
        }
        least += us;
        return p;
    };
    g.parts = 1;
    g.part[0] = best(0, all);
    const int64_t whole = all / (2 * kNsCus) * (2 * kNsCus);
    if (whole > 0 && whole < all) {
        const double one = least;
        least = ns_cost(NS_WIDE, whole, steps);
        const NsPart rest = best(whole, all - whole);
        if (least < one) {
            g.parts = 2;
            g.part[0] = NsPart{NS_WIDE, 0, whole};
            g.part[1] = rest;
        } else {
            least = one;
        }
    }
    for (int split = 2; gram && split <= kNsMaxSplit && all * split * kNsTileBytes <= products * s.m * s.np * 4; ++split) {
        const int64_t each = ns_tiles(steps, split);
        if (each < 8 || (split - 1) * each >= steps) continue;
        for (int form : {NS_WIDE, NS_DEEP, NS_THIN, NS_PAIR}) {
            const double us = ns_cost(form, all * split, each) + ns_join_cost(all, split);
            if (us >= least) continue;
            least = us;
            g.parts = 1;
            g.part[0] = NsPart{form, 0, all};
            g.split = split;
            g.split_steps = (int32_t)each;
        }
    }
    g.us = least;
    return g;
}

// The workspace: byte offsets of its parts, and its size.  X is there twice (a
// product cannot write what its other tiles still read); the second copy holds the
// fp32 update before the first product.  Single steps have two inner matrices, steps in
// groups five; the size is that of groups wherever they are allowed, since whether
// they are taken depends on the steps' factors too.
struct NsSpace {
    int64_t matrix[kNsMatrices], partial, inverse, bytes;
};
inline NsSpace ns_space(const NsShape& s) {
    NsSpace w{};
    if (s.small) return w;
    auto take = [&](int64_t bytes) {
        const int64_t at = w.bytes;
        w.bytes += ns_ceil(bytes, 256);
        return at;
    };
    for (int i = 0; i < kNsMatrices; ++i) {
        const bool x = i == M_X0 || i == M_X1, used = x || i == M_A || i == M_Q0 || s.grouped;
        w.matrix[i] = take(used ? s.group * s.m * (x ? s.np : s.mp) * 4 : 0);
    }
    w.partial = take(s.group * s.parts * 8);
    w.inverse = take(s.group * 8);
    return w;
}

// The factors of one pass X' = a X + (b A + c A^2) X, A = X X^T, on matrices that
// are held times powers of two.
struct NsPass {
    float a_mul;                        // A from the sum of X X^T
    float b_old, b_mul;                 // B from A and the sum of A A
    float x_old, x_mul;                 // X' from X and the sum of B X
};

// Singular values of X stay in [0, top]: at first top = 1 (the Frobenius norm is),
// then the largest value of |a s + b s^3 + c s^5|.  No element of a matrix is
// larger than its norm, so a matrix times the largest power of two that keeps its
// bound at 2^15 lies in fp16's range with room for rounding, and the two fp16
// parts of its elements are as far from fp16's smallest values as they can be.
inline double ns_scale(double bound) {
    int e = 0;
    if (!(bound > 0)) return 32768.0;
    std::frexp(bound * 1.001, &e);      // bound < 2^e
    return std::ldexp(1.0, std::min(15, 15 - e));
}
// Bounds of a step on singular values in [0, top].
struct NsBounds {
    double x, b, s;                     // of X', of b A + c A^2, of a + b A + c A^2
};
inline NsBounds ns_bounds(const double* k, double top) {
    const double a = k[0], b = k[1], c = k[2], end = top * top;
    auto odd = [&](double l) { return std::fabs(std::sqrt(l) * (a + l * (b + l * c))); };
    auto even = [&](double l) { return std::fabs(l * (b + l * c)); };
    auto all = [&](double l) { return std::fabs(a + l * (b + l * c)); };
    NsBounds r{odd(end), even(end), std::max(std::fabs(a), all(end))};
    auto inside = [&](double l) { return l > 0 && l < end; };
    // where the derivatives are zero
    if (c != 0) {
        const double l = -b / (2 * c), d = 9 * b * b - 20 * a * c;
        if (inside(l)) {
            r.b = std::max(r.b, even(l));
            r.s = std::max(r.s, all(l));
        }
        if (d >= 0)
            for (int sign = -1; sign <= 1; sign += 2) {
                const double q = (-3 * b + sign * std::sqrt(d)) / (10 * c);
                if (inside(q)) r.x = std::max(r.x, odd(q));
            }
    } else if (b != 0 && inside(-a / (3 * b))) {
        r.x = std::max(r.x, odd(-a / (3 * b)));
    }
    return r;
}

// false: coefficients whose bound leaves the range.  first: the power of two of the
// first X; last: what turns the last sum of a X + B X into the result itself.
inline bool ns_passes(const double (*coef)[3], int steps, NsPass* pass, double* first) {
    double top = 1.0, sx = ns_scale(top);
    *first = sx;
    for (int i = 0; i < steps; ++i) {
        const double a = coef[i][0], b = coef[i][1], c = coef[i][2];
        if (!std::isfinite(a) || !std::isfinite(b) || !std::isfinite(c)) return false;
        const NsBounds to = ns_bounds(coef[i], top);
        if (!(to.x * to.x <= 32768) || !(to.b <= 32768)) return false;
        const double sa = ns_scale(top * top), sb = ns_scale(to.b), next = i + 1 < steps ? ns_scale(to.x * 1.0001) : 1.0;
        pass[i].a_mul = (float)(sa / (sx * sx));
        pass[i].b_old = (float)(b * sb / sa);
        pass[i].b_mul = (float)(c * sb / (sa * sa));
        pass[i].x_old = (float)(a * next / sx);
        pass[i].x_mul = (float)(next / (sb * sx));
        top = to.x * 1.0001;            // roundings may go past it
        sx = next;
    }
    return true;
}

// A group of three steps has 3 + 2 + 2 inner products, the pairs, Gram and X'.
constexpr int kNsMaxOps = 4 * ZSMR_MAX_NS_STEPS + 4;

// Steps in groups.  S = a I + b A + c A^2 of every step is a polynomial of the first A,
// as the A of the next step is: A' = S A S.  So a group of steps forms X X^T once,
// goes on among m x m matrices, all symmetric, and multiplies X once, by Q = S .. S:
// 3 n / m + 4 g - 3 products of m^3 for g steps, where single steps have (3 n / m + 1) g.
// What it costs is accuracy: an error of A grows by S^2 a step.  Small singular values
// are still small at the start, where three steps may be in a group (S^2 twice is 141 for
// the quintic), later two.  Measured in the 2-norm, relative to the result, for 140 x 2,000
// to 1,600 x 6,400: white noise 2.6e-6 to 5.2e-6 in groups, 0.9e-6 to 2.0e-6 step by step,
// 1.3e-6 to 4.2e-6 with the library's fp32 products; singular values of 1/k^3 1.6e-5 to
// 6.4e-5, 1.4e-5 to 5.2e-5, 2.3e-5 to 8.3e-5; near rank one 5.1e-5 to 2.0e-4, 4.6e-5 to
// 1.7e-4, 8.2e-5 to 2.7e-4.  So groups are about as accurate as products of fp32 operands,
// and are taken wherever a call does not ask for its result in fp32.
inline int ns_group_steps(bool grouped, bool at_start, const double (*coef)[3], int left, double top) {
    const int most = std::min(left, !grouped ? 1 : at_start ? 3 : 2);
    const double limit = at_start ? 256 : 16;
    double grown = 1, q = 1, qa = 1;
    int g = 1;
    for (; g < most; ++g) {
        const NsBounds now = ns_bounds(coef[g - 1], top), next = ns_bounds(coef[g], now.x * 1.0001);
        grown *= now.s * now.s;
        q *= now.s;
        qa *= std::fabs(coef[g - 1][0]);
        if (!(grown <= limit) || !(q * next.s + qa * std::fabs(coef[g][0]) <= 32768)) break;
        top = now.x * 1.0001;
    }
    return g;
}

// The products of a call, for coefficients that ns_passes accepts; returns their number.
inline int ns_ops(const double (*coef)[3], int steps, bool grouped, NsOp* ops) {
    double scale[kNsMatrices] = {}, top = 1;
    int n = 0, x = M_X0;
    scale[M_X0] = ns_scale(1);
    auto add = [&](int kind, int p, int q, double k, int old, double k1, int old2, double k2, int dst, double bound) {
        const double to = kind == N_LAST ? 1 : ns_scale(bound);
        NsOp& o = ops[n++];
        o = NsOp{kind, p, q, old, old2, dst, (float)(k * to / (scale[p] * scale[q])), 0, 0, 0};
        if (old >= 0) o.old_mul = (float)(k1 * to / scale[old]);
        if (old2 >= 0) o.old2_mul = (float)(k2 * to / scale[old2]);
        return to;
    };
    for (int i = 0; i < steps;) {
        const int g = ns_group_steps(grouped, i == 0, coef + i, steps - i, top);
        scale[M_A] = add(N_INNER, x, x, 1, -1, 0, -1, 0, M_A, top * top);
        int q = M_Q0;
        double qa = 1, q_top = 1;
        for (int j = 0; j < g; ++j, ++i) {
            const double a = coef[i][0], b = coef[i][1], c = coef[i][2];
            const NsBounds to = ns_bounds(coef[i], top);
            const int now = j ? M_B : M_Q0;
            scale[now] = add(N_INNER, M_A, M_A, c, M_A, b, -1, 0, now, to.b);
            double next_t = 0;
            if (j + 1 < g) {
                next_t = add(N_INNER, M_A, now, 1, M_A, a, -1, 0, M_T, to.x * top);
                ops[n - 1].paired = j > 0;
            }
            q_top *= to.s;
            if (j) {
                const int other = q == M_Q0 ? M_Q1 : M_Q0;
                scale[other] = add(N_INNER, q, M_B, 1, M_B, qa, q, a, other, q_top + std::fabs(qa * a));
                q = other;
            }
            qa *= a;
            if (j + 1 < g) {
                scale[M_T] = next_t;
                scale[M_A] = add(N_INNER, M_T, now, 1, M_T, a, -1, 0, M_A, to.x * to.x);
            }
            top = to.x * 1.0001;
        }
        const int next = x == M_X0 ? M_X1 : M_X0;
        scale[next] = add(i < steps ? N_UPDATE : N_LAST, x, q, 1, x, qa, -1, 0, next, top);
        x = next;
    }
    return n;
}

// Products behind each other that share a launch, and their steps of k.
inline int ns_sides(const NsOp* op) {
    int n = 1;
    while (op[n - 1].paired) ++n;
    return n;
}
inline bool ns_from_x(const NsOp& op) { return op.p == M_X0 || op.p == M_X1; }
inline bool ns_gram(const NsOp& op) { return op.kind == N_INNER && ns_from_x(op); }
inline int64_t ns_steps_of(const NsShape& s, const NsOp& op) { return (ns_gram(op) ? s.np : s.mp) / kNsStep; }
// Groups where they end sooner.  Their products are fewer but one behind the other, so a
// matrix of 767 x 1,003, whose launches all last 9 to 12 us, takes single steps.
inline int ns_choose(const double (*coef)[3], int steps, const NsShape& s, NsOp* ops) {
    auto us = [&](int n) {
        double sum = 0;
        for (int i = 0; i < n; i += ns_sides(ops + i)) sum += ns_grid(s, ops[i].kind, ns_sides(ops + i) * s.group, ns_steps_of(s, ops[i]), ns_gram(ops[i])).us;
        return sum;
    };
    int n = ns_ops(coef, steps, false, ops);
    if (!s.grouped) return n;
    const double single = us(n);
    n = ns_ops(coef, steps, true, ops);
    return us(n) < single ? n : ns_ops(coef, steps, false, ops);
}

}  // namespace zsmr
