// What the scores of logits (zsmr_scores.hip) launch for given sizes: the segments
// a row is cut into, the workspace.  Host arithmetic only, so that it can be
// checked on any machine.
#pragma once
#include <stdint.h>

#include <algorithm>

#include "zsmr_ops.h"
#include "zsmr_ops_launch.h"

namespace zsmr {

// A wave reads blocks of 512 elements, 8 a lane.
constexpr int kScoreBlock = 512;
// Segments of all rows together, where rows are cut.
constexpr int64_t kScoreSplits = 512;

struct ScoreShape {
    int waves;                  // of a workgroup, 8 or 2
    int splits;                 // segments of a row, a workgroup each
    int64_t segment;            // elements of a segment, a multiple of kScoreBlock
    int64_t bytes;              // workspace: statistics and best keys of every segment
};
// Many short rows: two waves a row.  4,096 rows of 2,000 bf16 on MI355X, 20
// alternatives: 16.2 us, with eight waves 37.6.
// Otherwise eight, and rows of more than 16 blocks a wave are cut while there are fewer
// than two workgroups a CU, into segments of two blocks a wave at least: a wave takes a
// third of a microsecond a block, the launch that joins the segments 5.  129 rows of 50,257
// fp16 in three segments 12 us, whole 8.
inline ScoreShape score_shape(int64_t tokens, int64_t vocab, int64_t top) {
    ScoreShape s{};
    s.waves = vocab < 16 * kScoreBlock && tokens > 256 ? 2 : 8;
    const int64_t most = std::max<int64_t>(1, vocab / (2 * kScoreBlock * s.waves));
    const int64_t want = vocab <= 16 * kScoreBlock * s.waves ? 1 : std::max<int64_t>(1, std::min<int64_t>(kScoreSplits / std::max<int64_t>(tokens, 1), most));
    s.segment = ((vocab + want - 1) / want + kScoreBlock - 1) / kScoreBlock * kScoreBlock;
    s.splits = (int)((vocab + s.segment - 1) / s.segment);
    if (s.splits > 1) s.bytes = tokens * s.splits * (16 + 8 * top);
    return s;
}
// The launches over all segments: each(first, count) workgroups.
template <typename F>
void score_launches(const ScoreShape& s, int64_t tokens, F each) {
    launch_rows(tokens * s.splits, s.waves * 64, each);
}

}  // namespace zsmr
