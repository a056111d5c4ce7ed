"""Prompt attention and its gradients over 64, 65 and more sequences, up to which the work is planned with a
lane for each and past which the sequences go in their order: sequences of several tiles among them, in every
group of 64, with empty ones between and key counts of their own."""
import pytest
import torch

import test_gpu_attn_backward as bwd
import test_gpu_attn_prefill as fwd
from _attn import i32
from _util import announce, need_gpu

import kda_gated_delta_rule_amd as kda

pytestmark = pytest.mark.gpu


def lengths(n):
    """n sequences: mostly short, every seventh empty, some of two to six tiles (129 to 700 tokens), the
    last one long; keys a few or many more than queries for every fifth, none for some."""
    lens_q = [0 if i % 7 == 3 else 1 + i * 37 % 50 for i in range(n)]
    for i, L in ((0, 129), (5, 300), (n // 2, 257), (n - 9, 640), (n - 1, 700)):
        lens_q[i] = L
    lens_k = [L + (200 if i % 2 else 3) if i % 5 == 2 else L for i, L in enumerate(lens_q)]
    lens_k[1], lens_k[n - 2] = 0, lens_q[n - 2] // 2
    return lens_q, lens_k


@pytest.mark.parametrize("n", [63, 64, 65, 128, 130])
@pytest.mark.parametrize("H,Hk,dk,dv,dtype", [(2, 1, 64, 128, torch.bfloat16), (2, 2, 64, 64, torch.float32)])
def test_forward(n, H, Hk, dk, dv, dtype):
    dev = need_gpu()
    announce("prefill, %d sequences %s" % (n, dtype))
    q, k, v, cu_q, cu_k = fwd.case(*lengths(n), H, Hk, dk, dv, dtype, 21, dev)
    lse = torch.full((q.shape[0], H), 7.0, device=dev)
    o = kda.attn_prefill(q.to(dev), k.to(dev), v.to(dev), i32(cu_q, dev), cu_seqlens_k=i32(cu_k, dev), lse=lse)
    fwd.check(q, k, v, cu_q, cu_k, dk ** -0.5, o, lse)


@pytest.mark.parametrize("n", [63, 64, 65, 128, 130])
@pytest.mark.parametrize("H,Hk,dk,dv,dtype", [(2, 1, 128, 64, torch.bfloat16), (2, 1, 64, 64, torch.float32)])
def test_gradients(n, H, Hk, dk, dv, dtype):
    dev = need_gpu()
    announce("backward, %d sequences %s" % (n, dtype))
    x = bwd.case(*lengths(n), H, Hk, dk, dv, dtype, 22)
    bwd.check(*x, dk ** -0.5, bwd.grads(*x, dev))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_an_empty_65th_sequence(dtype):
    """64 sequences, and the same with an empty one behind them: planned, and in their order."""
    dev = need_gpu()
    announce("prefill, 64 sequences and an empty one %s" % dtype)
    lens_q, lens_k = lengths(64)
    q, k, v, cu_q, cu_k = fwd.case(lens_q, lens_k, 2, 1, 64, 64, dtype, 23, dev)
    for more in ([], [0]):
        _, _, _, cq, ck = fwd.case(lens_q + more, lens_k + more, 2, 1, 64, 64, dtype, 23, dev)
        lse = torch.empty(q.shape[:2], device=dev)
        o = kda.attn_prefill(q.to(dev), k.to(dev), v.to(dev), i32(cq, dev), cu_seqlens_k=i32(ck, dev), lse=lse)
        fwd.check(q, k, v, cu_q, cu_k, 0.125, o, lse)
