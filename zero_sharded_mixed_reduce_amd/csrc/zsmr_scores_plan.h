// What the scores of logits (zsmr_scores.hip) launch for given sizes: the segments
// a row is cut into, the workspace.  Host arithmetic only, so that it can be
// checked on any machine.
#pragma once
#include <stdint.h>

#include <algorithm>

#include "zsmr_ops.h"

namespace zsmr {

// A wave reads blocks of 512 elements, 8 a lane; a workgroup has four waves.
constexpr int kScoreBlock = 512, kScoreWaves = 4;

struct ScoreShape {
    int splits;                 // segments of a row, a workgroup each
    int64_t segment;            // elements of a segment, a multiple of kScoreBlock
    int64_t bytes;              // workspace: statistics and best keys of every segment
};
// Rows are cut while there are fewer than four workgroups a CU, into segments of
// two blocks a wave at least.
inline ScoreShape score_shape(int64_t tokens, int64_t vocab, int64_t top) {
    ScoreShape s{};
    const int64_t most = std::max<int64_t>(1, vocab / (2 * kScoreBlock * kScoreWaves));
    const int64_t want = std::max<int64_t>(1, std::min<int64_t>(1024 / std::max<int64_t>(tokens, 1), most));
    s.segment = ((vocab + want - 1) / want + kScoreBlock - 1) / kScoreBlock * kScoreBlock;
    s.splits = (int)((vocab + s.segment - 1) / s.segment);
    if (s.splits > 1) s.bytes = tokens * s.splits * (16 + 8 * top);
    return s;
}

}  // namespace zsmr
