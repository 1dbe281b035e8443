// What the softmax cross entropy of zsmr_xent.hip launches for given sizes: the
// vocabulary's pieces, the tiles and splits of every product, the workspace.
// Host arithmetic only, so that it can be checked on any machine.
#pragma once
#include <stdint.h>

#include <algorithm>

#include "zsmr_ops.h"

namespace zsmr {

constexpr int BM = 256, BK = 64;        // rows and k of a product's tile in a step
constexpr int64_t kCus = 256;
// Tiles of one launch: 512 work items each, and a launch has fewer than 2^32.
constexpr int64_t kMaxTiles = int64_t(1) << 22;

// The products: logits reduced to statistics, logits turned into G, and the two
// gradients.
enum : int { E_STATS, E_GRAD, E_DX, E_DW };

inline int64_t ceil_to(int64_t n, int64_t k) { return (n + k - 1) / k * k; }
inline int64_t tiles_of(int64_t n, int64_t k) { return (n + k - 1) / k; }

// Tokens of a tile, and what a step of 64 k takes with so many, in twentieths of a
// microsecond.  Measured on MI355X, logits of 4,096 rows and 16 tiles of tokens,
// bf16, from 8,192 to 16,384 of k: 0.47, 0.71, 1.04 and 1.34 us, the same
// proportions; 1.6 at 256 under the power of 8,192 tokens over 128,256 x 4,096.
constexpr int kWidths = 4, kWidth[kWidths] = {64, 128, 192, 256}, kCost[kWidths] = {11, 18, 25, 32};

// Tokens of a tile, given the tiles on the other side: the width whose rounds
// over the CUs end soonest.  215 tokens over 2,113 x 3,832 with gradients take 134
// us in tiles of 64, in one of 256 230; 8,192 over 50,257 x 768 2.5 ms in tiles of
// 256.
inline int token_tile(int64_t tokens, int64_t others) {
    int best = 0;
    int64_t least = INT64_MAX;
    for (int i = 0; i < kWidths; ++i) {
        const int64_t n = tiles_of(std::max<int64_t>(tokens, 1), kWidth[i]);
        const int64_t ends = tiles_of(n * others, kCus) * kCost[i];
        if (ends < least) {
            least = ends;
            best = kWidth[i];
        }
        if (n == 1) break;                  // wider tiles only pad
    }
    return best;
}

// The vocabulary's pieces: whole tiles, one at least.  G of one takes at most 512
// MB, or 512 bytes a token where a single tile is more than that (from 2^20 tokens
// on), and the tiles of dw over one fill the 256 CUs a whole number of times if it
// has that many.
constexpr int64_t kMaxPiece = int64_t(1) << 21;     // G's rows: byte offsets within a tile fit 31 bits
inline int64_t piece_of(int64_t tokens, int64_t vocab, int64_t width) {
    int64_t tiles = std::max<int64_t>(1, (int64_t(1) << 28) / std::max<int64_t>(tokens, 1) / BM);
    tiles = std::min<int64_t>(tiles, kMaxPiece / BM);
    if (tiles >= tiles_of(vocab, BM)) return ceil_to(vocab, BM);
    const int64_t across = tiles_of(width, BM), rounds = tiles * across / kCus;
    // across > 256: a single tile of rows is more than a round, and no part of one
    if (rounds > 0) tiles = std::max<int64_t>(1, rounds * kCus / across);
    return tiles * BM;
}
// Pieces of weights that have to be packed first: at most 32,768 rows, also where
// G would allow more (268 MB at width 4,096).
inline int64_t packed_piece(int64_t tokens, int64_t vocab, int64_t width) {
    return std::min<int64_t>(piece_of(tokens, vocab, width), 32768);
}
// The dx product: its k splits (none shorter than 512 of k) and the tokens of a
// tile.  Splits fill the CUs once or twice, but each writes and reads T x H sums at
// about 5 TB/s.  8,192 tokens of width 768: 5 splits in tiles of 256; 129 tokens:
// 28 in tiles of 64, 29 us with the sums on MI355X, where 49 in tiles of 192 took
// 36.
struct DxShape {
    int splits, tile;
};
inline DxShape dx_shape(int64_t tokens, int64_t width, int64_t piece) {
    DxShape best{};
    double least = 0;
    for (int i = 0; i < kWidths; ++i) {
        const int64_t n = tiles_of(std::max<int64_t>(tokens, 1), kWidth[i]), tiles = n * tiles_of(width, BM);
        for (int rounds = 1; rounds <= 2; ++rounds) {
            const int64_t splits = std::max<int64_t>(1, std::min(rounds * kCus / tiles, piece / 512));
            double us = (double)tiles_of(tiles * splits, kCus) * kCost[i] / 20 * tiles_of(piece, BK * splits);
            if (splits > 1) us += (double)splits * tokens * width * 8 / 5e6;
            if (!best.tile || us < least) {
                least = us;
                best = DxShape{(int)splits, kWidth[i]};
            }
        }
        if (n == 1) break;
    }
    return best;
}

// Vocabulary rows of a tile of dw: 256, or 128, which take a little over half as
// long, where that ends sooner.  A piece of 27 tiles of 256 across 3 (8,192
// tokens, width 768) fills a third of the CUs once: 184 us on MI355X, in tiles of
// 128 119-124.
inline int dw_tile(int64_t across, int64_t rows) {
    const int64_t wide = tiles_of(across * tiles_of(rows, 256), kCus), narrow = tiles_of(across * tiles_of(rows, 128), kCus);
    return narrow * 11 < wide * 20 ? 128 : 256;
}

// One product of a call, over the vocabulary from v0 on.
struct ProductShape {
    int epi;
    int64_t v0, rows;               // the piece
    int64_t k, k_split;             // k_split: k of one split, a multiple of BK
    int64_t m_tiles, n_tiles;
    int splits;
    int tile;                       // of the n side: tokens, or vocabulary rows of dw
    int stages;                     // of LDS
    bool once;                      // one tile holds all of n: the other operand is read once
    bool sum_in, sum_out;           // dx: add what earlier pieces left; leave the sums for later ones
    int64_t grid() const { return m_tiles * n_tiles * splits; }
};
// Two workgroups share a CU's LDS with two stages of a 64-wide tile each; where
// there is at most one for a CU it takes four, and waits a third as long: 44 tokens
// over 1,892 x 4,008 106 -> 38 us on MI355X.
inline void pick_stages(ProductShape* p) {
    p->once = p->epi != E_DW && p->n_tiles == 1 && (p->tile == 64 ? p->grid() > kCus : p->tile == 128);
    p->stages = p->tile == 64 ? (p->once ? 2 : 4) : p->tile == 128 ? 3 : 2;
}

inline ProductShape logits_shape(int epi, int64_t tokens, int64_t width, int64_t v0, int64_t rows, int tile) {
    ProductShape p{};
    p.epi = epi;
    p.v0 = v0;
    p.rows = rows;
    p.k = ceil_to(width, 8);        // packed rows end in zeros
    p.k_split = ceil_to(p.k, BK);
    p.m_tiles = tiles_of(rows, BM);
    p.n_tiles = tiles_of(tokens, tile);
    p.splits = 1;
    p.tile = tile;
    pick_stages(&p);
    return p;
}

// The products of a forward call, in order: one, but for weights that are packed
// piece by piece, and for more tiles than a launch holds.
template <typename F>
void forward_products(int64_t tokens, int64_t vocab, int64_t width, bool packed, F each) {
    const int64_t most = std::max<int64_t>(1, kMaxTiles / tiles_of(std::max<int64_t>(tokens, 1), kWidth[0])) * BM;
    const int64_t piece = std::min(most, packed ? packed_piece(tokens, vocab, width) : vocab);
    const int tile = token_tile(tokens, tiles_of(std::min(piece, vocab), BM));
    for (int64_t v0 = 0; v0 < vocab; v0 += piece) each(logits_shape(E_STATS, tokens, width, v0, std::min(piece, vocab - v0), tile));
}

// The products of a backward call, in order; dx and dw: which gradients are asked
// for.  Without tokens there is dw alone, of zeros.
template <typename F>
void backward_products(int64_t tokens, int64_t vocab, int64_t width, bool packed, bool dx, bool dw, F each) {
    const int64_t piece = packed ? packed_piece(tokens, vocab, width) : piece_of(tokens, vocab, width);
    const int tile = token_tile(tokens, tiles_of(std::min(piece, vocab), BM));
    const DxShape shape = dx_shape(tokens, width, piece);
    for (int64_t v0 = 0; v0 < vocab; v0 += piece) {
        const int64_t rows = std::min(piece, vocab - v0);
        ProductShape p = logits_shape(E_GRAD, tokens, width, v0, rows, tile);
        if (tokens) each(p);
        p.m_tiles = tiles_of(width, BM);
        if (dx && tokens) {
            p.epi = E_DX;
            p.k = ceil_to(rows, 8);         // G is zero past the vocabulary
            p.tile = shape.tile;
            p.splits = shape.splits;
            p.k_split = ceil_to(tiles_of(p.k, shape.splits), BK);
            p.n_tiles = tiles_of(tokens, shape.tile);
            p.sum_in = v0 > 0;
            p.sum_out = shape.splits > 1 || v0 + piece < vocab;
            pick_stages(&p);
            each(p);
        }
        if (dw) {
            p.epi = E_DW;
            p.k = tokens;
            p.tile = dw_tile(p.m_tiles, rows);
            p.splits = 1;
            p.k_split = ceil_to(p.k, BK);
            p.n_tiles = tiles_of(rows, p.tile);
            p.sum_in = p.sum_out = false;
            pick_stages(&p);
            each(p);
        }
    }
}

// The workspace: byte offsets of its parts, and its size.
struct XentSpace {
    int64_t stats, target, x, w, mul, g, sum, bytes;
};
inline XentSpace xent_space(int64_t tokens, int64_t vocab, int64_t width, bool backward) {
    XentSpace s{};
    auto take = [&](int64_t bytes) {
        const int64_t at = s.bytes;
        s.bytes += ceil_to(bytes, 256);
        return at;
    };
    const int64_t piece = piece_of(tokens, vocab, width), packed = ceil_to(width, 8);
    const int64_t rows = packed_piece(tokens, vocab, width);
    s.stats = take(tiles_of(vocab, BM) * tokens * 8);
    s.target = take(tokens * 4);
    s.x = take(tokens * packed * 2);
    s.w = take(rows * packed * 2);
    if (backward) {
        s.mul = take(8);
        s.g = take(tokens * piece * 2);
        const int splits = std::max(dx_shape(tokens, width, piece).splits, dx_shape(tokens, width, rows).splits);
        s.sum = take(tokens * ceil_to(width, 4) * 4 * splits);
    }
    return s;
}

}  // namespace zsmr
