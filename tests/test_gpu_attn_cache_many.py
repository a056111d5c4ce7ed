"""The 8-bit cache with more sequences than a wave has lanes, and workspaces of exactly the stated size with
guarded bytes behind them."""
import pytest
import torch

import kda_gated_delta_rule_amd as kda
from _attn import cu_of, i32, normal
from _util import announce, need_gpu
from test_gpu_attn_cache import Cache, check_append, check_decode

pytestmark = pytest.mark.gpu


def lengths(n):
    """Contexts of 0, 1 and up to 1200 tokens, in every group of 64."""
    lens = [i * 53 % 90 for i in range(n)]
    for i in (0, 31, n - 66 if n > 66 else 2, n - 1):
        lens[i] = 1200 - i
    lens[n // 2] = 0
    return lens


@pytest.mark.parametrize("n", [64, 65, 130])
@pytest.mark.parametrize("T,dtype", [(1, torch.bfloat16), (3, torch.float32)])
def test_decode(n, T, dtype):
    """A table of more than 1024 positions, so contexts are cut into pieces over all groups of 64."""
    dev = need_gpu()
    announce("decode, %d sequences T=%d %s" % (n, T, dtype))
    lens = lengths(n)
    g = torch.Generator().manual_seed(31)
    cache = Cache(n, 1280, 32, 1, 64, 64, dev, 31)
    assert kda.attn_decode_workspace_size(n, T, 2, 1, 64, dtype, 32, cache.mb) > 0
    k, v = normal(g, sum(lens), 1, 64), normal(g, sum(lens), 1, 64)
    cache.append(k, v, lens, [0] * n)
    q = normal(g, n, T, 2, 64, dtype=dtype)
    check_decode(cache, q, lens, 0.125, kda.attn_decode(q.to(dev), *cache.tensors(), i32(lens, dev)))


@pytest.mark.parametrize("n", [64, 65, 130])
def test_append(n):
    """A prompt for each, then tokens for some: blocks begin and are joined in every group of 64."""
    dev = need_gpu()
    announce("append, %d sequences" % n)
    g = torch.Generator().manual_seed(32)
    cache = Cache(n, 160, 32, 1, 64, 64, dev, 32)
    have = [0] * n
    for step, new in enumerate(([1 + i * 29 % 100 for i in range(n)], [i % 3 for i in range(n)], [1] * n)):
        k, v = normal(g, sum(new), 1, 64) * 1.6 ** step, normal(g, sum(new), 1, 64)
        check_append(cache, k, v, new, have)
        have = [a + b for a, b in zip(have, new)]


def guarded(need, dev):
    """A workspace of `need` bytes and the guard behind it."""
    whole = torch.full((need + 4096,), 0xa5, dtype=torch.uint8, device=dev)
    return whole[:need], whole[need:]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_workspaces_of_the_stated_size(dtype):
    """Given workspaces give what allocated ones give, and nothing is written behind them; a byte less is
    refused."""
    dev = need_gpu()
    announce("attention, guarded workspaces %s" % dtype)
    g = torch.Generator().manual_seed(33)
    lens = [1500, 3, 0, 900]
    T, H, Hk, cu = sum(lens), 4, 1, i32(cu_of(lens), dev)
    q, do = (normal(g, T, H, 64, dtype=dtype).to(dev) for _ in range(2))
    k, v = (normal(g, T, Hk, 64, dtype=dtype).to(dev) for _ in range(2))
    lse = torch.empty(T, H, device=dev)
    o = kda.attn_prefill(q, k, v, cu, lse=lse)
    grads = kda.attn_backward(q, k, v, o, lse, do, cu)
    cache = Cache(2, 5000, 64, Hk, 64, 64, dev, 33)
    ck, cv = normal(g, 4700, Hk, 64), normal(g, 4700, Hk, 64)
    cache.append(ck, cv, [4000, 700], [0, 0])
    qd, ctx = normal(g, 2, 2, H, 64, dtype=dtype).to(dev), i32([4000, 700], dev)
    od = kda.attn_decode(qd, *cache.tensors(), ctx)
    sizes = (kda.attn_prefill_workspace_size(4, T, T, H, Hk, 64, 64, dtype),
             kda.attn_backward_workspace_size(4, T, T, H, Hk, 64, 64, dtype),
             kda.attn_decode_workspace_size(2, 2, H, Hk, 64, dtype, 64, cache.mb))
    calls = (lambda ws: (kda.attn_prefill(q, k, v, cu, workspace=ws),),
             lambda ws: kda.attn_backward(q, k, v, o, lse, do, cu, workspace=ws),
             lambda ws: (kda.attn_decode(qd, *cache.tensors(), ctx, workspace=ws),))
    for need, call, want in zip(sizes, calls, ((o,), grads, (od,))):
        assert need > 0
        ws, guard = guarded(need, dev)
        assert all(torch.equal(a, b) for a, b in zip(call(ws), want))
        assert (guard == 0xa5).all()
        with pytest.raises(kda.KdaError):
            call(ws[:need - 1])
