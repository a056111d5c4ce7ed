"""Batches that end before their arrays do, which the attention operators take, pass KDA_DEBUG_VALIDATE;
lengths that decrease, do not begin at 0 or pass the arrays do not.  CPU tensors stand in for device
ones: a call that passes the checks is refused for that, last of all."""
import pytest
import torch

from kda_gated_delta_rule_amd import ops


def i32(*x):
    return torch.tensor(x, dtype=torch.int32)


@pytest.fixture(autouse=True)
def on(monkeypatch):
    monkeypatch.setenv("KDA_DEBUG_VALIDATE", "1")


def prompt(cu, cu_k=None):
    z = lambda h: torch.zeros(6, h, 64)
    return dict(q=z(4), k=z(2), v=z(2), cu_seqlens=i32(*cu), cu_seqlens_k=None if cu_k is None else i32(*cu_k))


CU = [((0, 2, 4), "one GPU"), ((0, 0), "one GPU"), ((0, 2, 6), "one GPU"), ((0, 2, 7), "past"), ((1, 2), r"\[0\]"),
      ((0, 4, 2), "decreases")]


@pytest.mark.parametrize("cu,msg", CU)
def test_prompts(cu, msg):
    with pytest.raises(ValueError, match=msg):
        ops.attn_prefill(**prompt(cu))
    with pytest.raises(ValueError, match=msg):
        ops.attn_prefill(**prompt((0,) + (1,) * (len(cu) - 1), cu))
    with pytest.raises(ValueError, match=msg):
        ops.attn_backward(o=torch.zeros(6, 4, 64), do=torch.zeros(6, 4, 64), lse=torch.zeros(6, 4), **prompt(cu))


@pytest.mark.parametrize("cu,msg", CU)
def test_cache_writes(cu, msg):
    f8 = torch.float8_e4m3fn
    N = len(cu) - 1
    z = lambda: torch.zeros(6, 2, 64)
    with pytest.raises(ValueError, match=msg):
        ops.attn_cache_append(z(), z(), i32(*cu), i32(*([0] * N)), torch.zeros(5, 2, 16, 64, dtype=f8),
                              torch.zeros(5, 2, 64, 16, dtype=f8), torch.ones(5, 2), torch.ones(5, 2),
                              torch.arange(N, dtype=torch.int32).reshape(N, 1))
