"""The cache write that clears (kda_attn_cache_append_clear): positions behind the new tokens of every
block written into become zero, and nothing else differs from kda_attn_cache_append, bit for bit."""
import numpy as np
import pytest
import torch

import kda_gated_delta_rule_amd as kda
from _attn import cu_of, i32, normal
from _util import announce, f64, need_gpu
from test_gpu_attn_cache import FP8, Cache, expect

pytestmark = pytest.mark.gpu


def cleared(cache, want, lens, start):
    """The oracle's result with zeros behind the last token of each sequence that got any."""
    kb, vb, ks, vs = (x.copy() for x in want)
    table = cache.table.cpu().numpy()
    for n, L in enumerate(lens):
        end = min(start[n] + L, cache.mb * cache.bt)
        page = table[n, (end - 1) // cache.bt] if L else -1
        if L and 0 <= page < cache.nb and end % cache.bt:
            kb[page, :, end % cache.bt:] = 0
            vb[page, :, :, end % cache.bt:] = 0
    return kb, vb, ks, vs


def check_clear(cache, k, v, lens, start):
    want = cleared(cache, expect(cache, k, v, lens, start, cache.bytes()), lens, start)
    dev = cache.k.device
    kda.attn_cache_append(k.to(dev), v.to(dev), i32(cu_of(lens), dev), i32(start, dev), *cache.tensors(), clear=True)
    for name, a, b in zip(("k", "v", "k_scale", "v_scale"), (cache.k, cache.v, cache.ks, cache.vs), want):
        a = f64(a)
        assert np.array_equal(a, b, equal_nan=True), (name, np.argwhere(~((a == b) | (np.isnan(a) & np.isnan(b))))[:5])


@pytest.mark.parametrize("bt", [16, 32, 64, 128])
@pytest.mark.parametrize("Hk,dk,dv,dtype", [(2, 128, 64, torch.bfloat16), (1, 64, 128, torch.float32)])
def test_positions_behind_the_new_tokens_become_zero(bt, Hk, dk, dv, dtype):
    """Pages full of garbage: blocks begin, end at every place of a word of four, are filled to the end, and
    raise their scale while they are cleared; a sequence without new tokens keeps its page."""
    dev = need_gpu()
    announce("append, clear bt=%d Hk=%d dk=%d dv=%d %s" % (bt, Hk, dk, dv, dtype))
    g = torch.Generator().manual_seed(bt + dk)
    lens = [1, 0, 130, 15, 16, 17, 64]
    cache = Cache(len(lens), 300, bt, Hk, dk, dv, dev)
    have = [0] * len(lens)
    for step, new in enumerate((lens, [1] * 7, [3, 0, 1, 1, 20, 0, 2], [1] * 7)):
        k = (normal(g, sum(new), Hk, dk) * 1.7 ** step).to(dtype)
        v = (normal(g, sum(new), Hk, dv) * 0.9 ** step).to(dtype)
        check_clear(cache, k, v, new, have)
        have = [a + b for a, b in zip(have, new)]


def test_absent_pages_and_the_table_s_end():
    """Nothing is cleared through an absent page, nor behind a block filled to its end."""
    dev = need_gpu()
    announce("append, clear, absent pages")
    g = torch.Generator().manual_seed(3)
    cache = Cache(3, 64, 16, 2, 64, 64, dev)
    cache.table[0, 3] = -1
    cache.ks.fill_(0.125)
    cache.vs.fill_(0.25)
    k, v = normal(g, 130, 2, 64), normal(g, 130, 2, 64)
    check_clear(cache, k[:64], v[:64], [50, 0, 14], [3, 0, 0])
    check_clear(cache, k[:8], v[:8], [0, 8, 0], [0, 56, 0])


def test_a_page_given_back_holds_nothing_of_its_last_sequence():
    """Equal tokens give equal pages, whatever the pages held; decode reads the same from both."""
    dev = need_gpu()
    announce("append, clear, pages used again")
    g = torch.Generator().manual_seed(5)
    k, v = normal(g, 37, 2, 64, dtype=torch.bfloat16), normal(g, 37, 2, 64, dtype=torch.bfloat16)
    q = normal(g, 1, 1, 4, 64, dtype=torch.bfloat16).to(dev)
    got = []
    for garbage in (True, False):
        c = Cache(1, 48, 16, 2, 64, 64, dev, garbage=garbage)
        for a, b in ((0, 20), (20, 37)):
            kda.attn_cache_append(k[a:b].to(dev), v[a:b].to(dev), i32([0, b - a], dev), i32([a], dev), *c.tensors(), clear=True)
        pages = c.table[0].long()
        got.append([c.k.view(torch.uint8)[pages], c.v.view(torch.uint8)[pages], c.ks[pages], c.vs[pages],
                    kda.attn_decode(q, *c.tensors(), i32([37], dev))])
    assert all(torch.equal(a, b) for a, b in zip(*got))
    assert not got[0][0][2, :, 5:].any() and not got[0][1][2, :, :, 5:].any()


def test_in_a_graph():
    """Captured and replayed with other lengths and rows each time, against the same calls made eagerly."""
    dev = need_gpu()
    announce("append, clear, in a graph")
    g = torch.Generator().manual_seed(6)
    a, b = Cache(2, 64, 32, 1, 64, 64, dev, seed=1), Cache(2, 64, 32, 1, 64, 64, dev, seed=1)
    k, v = (torch.zeros(2, 1, 64, dtype=torch.bfloat16, device=dev) for _ in range(2))
    held, cu = i32([0, 32], dev), i32([0, 1, 2], dev)
    step = lambda c: kda.attn_cache_append(k, v, cu, held, *c.tensors(), clear=True)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(a)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(a)
    for rep in range(4):
        for t in (k, v):
            t.copy_((normal(g, 2, 1, 64) * 3.0 ** rep).to(torch.bfloat16).to(dev))
        step(b)
        graph.replay()
        torch.cuda.synchronize()
        for x, y in zip(a.bytes(), b.bytes()):
            assert torch.equal(x.view(torch.uint8), y.view(torch.uint8)), rep
        held += 1
