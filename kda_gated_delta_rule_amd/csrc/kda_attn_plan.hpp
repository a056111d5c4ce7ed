// kda_attn_plan.hpp -- how a decode batch is cut into pieces of keys: the arithmetic that the host (sizes
// of the workspace and the grid) and the kernels share.  Plain C++, so that it can be checked on the CPU at
// the limits of the entry point.
#pragma once

#include <stdint.h>

namespace kda {

constexpr int kStepKeys = 256;  // keys of a workgroup's step: 64 for each of its four waves
// Workgroups that a decode call is cut into: two run on each of 256 compute units, so two rounds.
// With 1536 and 2048, 64 mixed contexts take 193 and 192 us (1024: 199), four long ones 132 and
// 135 us (1024: 124): the evener rounds cost a start and an end each.
constexpr int kPieces = 1024;

// Steps of a table of max_blocks pages (host-checked: at most 2^30 positions, so 2^22 steps).
constexpr int decode_table_steps(int max_blocks, int bt) {
    return static_cast<int>((static_cast<int64_t>(max_blocks) * bt + kStepKeys - 1) / kStepKeys);
}

// About so many pieces per kv head, `per` workgroups each; 0: sequences are not cut.
constexpr int decode_pieces(int N, int64_t per, int table_steps) {
    // Short tables go uncut: one launch, no join (1 x 700 positions on 2 kv heads 7.1 us, cut 8.6;
    // 1 x 2000 on 8: 15.4, cut 9.4; with 32 sequences, a workgroup for each compute unit, 24.9, cut
    // 29.5; longer ones would make a mixed batch wait for the longest).
    if (table_steps <= 4 || (table_steps <= 8 && N * per >= 256)) return 0;
    const int64_t pieces = (kPieces + per - 1) / per, most = static_cast<int64_t>(N) * table_steps;
    return static_cast<int>(pieces < most ? pieces : most);
}

// Steps of a piece, one size for the whole batch of `all` steps.  No sequence has more steps than the
// table, so no piece needs more: its keys then stay within 2^30 where a few pieces share a batch of up
// to 2^30 steps.  (With the bound every sequence is one piece, so there are never more than pieces + N.)
constexpr int decode_piece_steps(int all, int pieces, int table_steps) {
    const int even = (all + pieces - 1) / pieces;
    return even < 1 ? 1 : even < table_steps ? even : table_steps;
}

}  // namespace kda
