// What the orthogonalised update of zsmr_newton.hip launches for given sizes: the
// matrices of a group, the workspace, the powers of two that keep every matrix in
// fp16's range.  Host arithmetic only, so that it can be checked on any machine.
#pragma once
#include <stdint.h>

#include <algorithm>
#include <cmath>

#include "zsmr_ops.h"

namespace zsmr {

constexpr int kNsTile = 128;            // rows and columns of a product's tile
constexpr int kNsStep = 32;             // k of a step
constexpr int kNsThreads = 256;         // of a product's workgroup

inline int64_t ns_ceil(int64_t n, int64_t k) { return (n + k - 1) / k * k; }

// The wide orientation of a matrix: m <= n.  Rows are padded to whole steps.
struct NsShape {
    int64_t m, n, mp, np;
    bool tall;                          // the wide orientation is the transposed one
    int64_t count, group;               // matrices; of a group, whose launches they share
    int parts;                          // partial sums of squares of a matrix
    int64_t m_tiles, n_tiles;
    int small;                          // the form of a matrix that stays in LDS, or 0
};

// A group's matrices have 2^25 elements at most (or are one): enough to fill the
// CUs many times over, while the workspace stays below 600 MB for any count.
constexpr int64_t kNsGroupElems = int64_t(1) << 25;

// A matrix that fits a CU's LDS with its inner matrix is one workgroup's: every pass
// without a launch.  Up to 64 x 64 (1), 64 x 256 (2) and 128 x 128 (3).
inline int ns_small(int64_t m, int64_t n) {
    return m <= 64 ? n <= 64 ? 1 : n <= 256 ? 2 : 0 : n <= 128 ? 3 : 0;
}
inline NsShape ns_shape(int64_t rows, int64_t cols, int64_t count) {
    NsShape s{};
    s.tall = rows > cols;
    s.m = std::min(rows, cols);
    s.n = std::max(rows, cols);
    s.mp = ns_ceil(s.m, kNsStep);
    s.np = ns_ceil(s.n, kNsStep);
    s.count = count;
    s.small = ns_small(s.m, s.n);
    s.group = std::max<int64_t>(1, std::min({count, kNsGroupElems / (s.m * s.n), int64_t(1) << 14}));
    // a workgroup of the sums takes 2,048 elements at a time
    s.parts = (int)std::min<int64_t>((s.m * s.n + 2047) / 2048, std::max<int64_t>(1, 1024 / s.group));
    s.m_tiles = (s.m + kNsTile - 1) / kNsTile;
    s.n_tiles = (s.n + kNsTile - 1) / kNsTile;
    return s;
}

// Workgroups that a product has for one matrix, at most.
inline int64_t ns_largest_grid(const NsShape& s) { return s.m_tiles * std::max(s.n_tiles, (s.m_tiles + 1) / 2); }

// The workspace: byte offsets of its parts, and its size.  X is there twice (a
// product cannot write what its other tiles still read); the second copy holds the
// fp32 update before the first product.
struct NsSpace {
    int64_t x[2], a, b, partial, inverse, bytes;
};
inline NsSpace ns_space(const NsShape& s) {
    NsSpace w{};
    if (s.small) return w;
    auto take = [&](int64_t bytes) {
        const int64_t at = w.bytes;
        w.bytes += ns_ceil(bytes, 256);
        return at;
    };
    w.x[0] = take(s.group * s.m * s.np * 4);
    w.x[1] = take(s.group * s.m * s.np * 4);
    w.a = take(s.group * s.m * s.mp * 4);
    w.b = take(s.group * s.m * s.mp * 4);
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
// false: coefficients whose bound leaves the range.  first: the power of two of the
// first X; last: what turns the last sum of a X + B X into the result itself.
inline bool ns_passes(const double (*coef)[3], int steps, NsPass* pass, double* first) {
    double top = 1.0, sx = ns_scale(top);
    *first = sx;
    for (int i = 0; i < steps; ++i) {
        const double a = coef[i][0], b = coef[i][1], c = coef[i][2];
        if (!std::isfinite(a) || !std::isfinite(b) || !std::isfinite(c)) return false;
        auto odd = [&](double s) { return std::fabs(s * (a + s * s * (b + s * s * c))); };
        auto even = [&](double l) { return std::fabs(l * (b + l * c)); };
        double x_top = odd(top), b_top = even(top * top);
        // where the derivatives are zero
        if (c != 0) {
            const double l = -b / (2 * c);
            if (l > 0 && l < top * top) b_top = std::max(b_top, even(l));
            const double d = 9 * b * b - 20 * a * c;
            if (d >= 0)
                for (int sign = -1; sign <= 1; sign += 2) {
                    const double q = (-3 * b + sign * std::sqrt(d)) / (10 * c);
                    if (q > 0 && q < top * top) x_top = std::max(x_top, odd(std::sqrt(q)));
                }
        } else if (b != 0) {
            const double q = -a / (3 * b);
            if (q > 0 && q < top * top) x_top = std::max(x_top, odd(std::sqrt(q)));
        }
        if (!(x_top * x_top <= 32768) || !(b_top <= 32768)) return false;
        const double sa = ns_scale(top * top), sb = ns_scale(b_top), next = i + 1 < steps ? ns_scale(x_top) : 1.0;
        pass[i].a_mul = (float)(sa / (sx * sx));
        pass[i].b_old = (float)(b * sb / sa);
        pass[i].b_mul = (float)(c * sb / (sa * sa));
        pass[i].x_old = (float)(a * next / sx);
        pass[i].x_mul = (float)(next / (sb * sx));
        top = x_top * 1.0001;           // roundings may go past it
        sx = next;
    }
    return true;
}

}  // namespace zsmr
