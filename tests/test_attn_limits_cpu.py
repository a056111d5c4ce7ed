"""Sizes of workspaces at their largest, and limits of the entry points, as include/kda.h states them."""
import os

import pytest

from kda_gated_delta_rule_amd import _build, _lib


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(_build.LIB):
        _build.build(force=True)
    return _lib.load()


def header():
    path = os.path.join(_build.INCLUDE, "kda.h")
    return " ".join(open(path).read().replace("\n *", "\n").split())


def test_most_prefill_workspace(lib):
    """1024 parts of 128 rows, each dv sums, a maximum and a sum of the weights in fp32."""
    size = lib.kda_attn_prefill_workspace_size
    most = 1024 * 128 * (128 + 2) * 4
    assert most == 68157440 and "at most 68,157,440" in header()
    assert size(2, 1 << 20, 1 << 20, 64, 8, 128, 128, 1) == most
    for args in ((1, 5000, 1 << 24, 1, 1, 128, 128, 0), (64, 1 << 24, 1 << 24, 8, 8, 64, 128, 1), (3, 200, 900, 2, 2, 128, 128, 1)):
        assert 0 < size(*args) <= most
    assert size(2, 1 << 20, 1 << 20, 64, 8, 64, 64, 1) == 1024 * 128 * (64 + 2) * 4


@pytest.mark.parametrize("dtype", [0, 1])
def test_no_parts_past_64_sequences(lib, dtype):
    """Longer batches are not shared among workgroups, as the header says: no room for parts."""
    assert lib.kda_attn_prefill_workspace_size(64, 9000, 9000, 4, 2, 128, 128, dtype) > 0
    assert lib.kda_attn_prefill_workspace_size(65, 9000, 9000, 4, 2, 128, 128, dtype) == 0
    assert lib.kda_attn_backward_workspace_size(65, 9000, 9000, 4, 2, 128, 128, dtype) == 9000 * 4 * 8
    assert "more than 64 sequences" in header()


def test_rows_as_wide_as_allowed(lib):
    """2^22 elements between tokens: the copies of 128 rows of them stay within 2^30 bytes in bf16, of 64 in fp32
    within 2^30 too."""
    A = 0x10000
    args = lambda ld: (A, ld, A, 256, A, 256, 1, A, A, 2, 0, 30, 4, 2, 128, 128, 0.1, A, None, None, 0, None)
    assert lib.kda_attn_prefill(*args(1 << 22)) == _lib.KDA_OK
    assert lib.kda_attn_prefill(*args((1 << 22) + 8)) == _lib.KDA_ERR_INVALID_ARG
