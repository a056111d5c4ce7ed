"""The cutting of a decode batch into pieces, compiled for the CPU with overflow checks and run at the
limits of kda_attn_decode: every key of every sequence is in one piece, and there are never more
pieces than the workspace and the grid have room for."""
import os
import subprocess

import pytest

from kda_gated_delta_rule_amd import _build

PROGRAM = r"""
#include <cstdio>
#include <cstdlib>
#include "kda_attn_plan.hpp"
using namespace kda;
// N, max_blocks, block_tokens, workgroups of a piece, then a context length: the first half of the
// batch has it, the others one token
int main(int, char** v) {
    const int N = atoi(v[1]), mb = atoi(v[2]), bt = atoi(v[3]), per = atoi(v[4]), ctx = atoi(v[5]);
    const int table = decode_table_steps(mb, bt), pieces = decode_pieces(N, per, table);
    if (pieces == 0) return puts("uncut"), 0;
    int all = 0;
    for (int n = 0; n < N; ++n) all += ((n < (N + 1) / 2 ? ctx : 1) + kStepKeys - 1) / kStepKeys;
    const int steps = decode_piece_steps(all, pieces, table), keys = steps * kStepKeys;
    if (steps < 1 || keys < kStepKeys || keys > 1 << 30) return printf("keys of a piece: %d\n", keys), 1;
    long long made = 0;
    for (int n = 0; n < N; ++n) {
        const int len = n < (N + 1) / 2 ? ctx : 1, mine = ((len + kStepKeys - 1) / kStepKeys + steps - 1) / steps;
        long long covered = 0;
        for (int p = 0; p < mine; ++p) {
            const int begin = p * keys, end = (len - begin < keys ? len - begin : keys) + begin;
            if (begin >= end) return printf("an empty piece\n"), 1;
            covered += end - begin;
        }
        if (covered != len) return printf("%lld of %d keys\n", covered, len), 1;
        made += mine;
    }
    if (made > static_cast<long long>(pieces) + N) return printf("%lld pieces, room for %d\n", made, pieces + N), 1;
    return printf("%d steps\n", steps), 0;
}
"""


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    d = tmp_path_factory.mktemp("plan")
    (d / "plan.cpp").write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-O1", "-fsanitize=undefined", "-fno-sanitize-recover=all", "-I" + _build.CSRC,
                    str(d / "plan.cpp"), "-o", str(d / "plan")], check=True)
    return lambda *a: subprocess.run([str(d / "plan")] + [str(x) for x in a], capture_output=True, text=True)


FULL = 1 << 30  # positions of the longest table


@pytest.mark.parametrize("N,mb,bt,per,ctx", [
    # full contexts whose even share of the batch's pieces passes 2^31 keys
    (4, FULL // 128, 128, 1024, FULL), (64, FULL // 64, 64, 64, FULL), (256, FULL // 128, 128, 8, FULL),
    (256, FULL // 16, 16, 1024, FULL), (256, FULL // 128, 128, 65535, FULL), (1, FULL // 16, 16, 1, FULL),
    # ordinary ones: long, mixed, empty, just cut
    (64, 250, 64, 8, 16000), (4, 1024, 128, 8, 131072), (3, 300, 64, 2, 0), (1, 17, 64, 2, 1088), (5000, 33, 64, 1, 2112)])
def test_pieces_cover_every_key(plan, N, mb, bt, per, ctx):
    r = plan(N, mb, bt, per, ctx)
    assert r.returncode == 0, r.stdout + r.stderr


def test_short_tables_are_not_cut(plan):
    assert plan(1, 16, 64, 2, 700).stdout.strip() == "uncut"


def test_pieces_are_even_shares(plan):
    """128 pieces of 64 x 63 / 2 steps: 16 a piece."""
    assert plan(64, 250, 64, 8, 16000).stdout.split()[0] == str(-(-(32 * 63 + 32) // 128))
