"""Softmax attention at the ends of the numbers' range: scales of zero and below the smallest normal
number with large scores, and values as large as the header allows."""
import numpy as np
import pytest
import torch

import kda_gated_delta_rule_amd as kda
from _attn import U, cu_of, i32, normal, o_bound
from _util import announce, f64, need_gpu
from oracle import kda_attn as OA
from test_gpu_attn_cache import Cache, check_decode

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("scale", [0.0, 2.0 ** -130, -2.0 ** -127])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_tiny_scales_with_large_products(scale, dtype):
    """Products q.k of up to 2^122 under a scale of zero (equal weights) and of 2^-127 and less (weights
    within 2^-5 of each other): forward and gradients.  A factor of 10^-37 in the scale's place would give
    scores of 60."""
    dev = need_gpu()
    announce("attention, scale %g, large products %s" % (scale, dtype))
    g = torch.Generator().manual_seed(1)
    lens, H = [90, 33], 2
    T, cu = sum(lens), cu_of(lens)
    q, k = (normal(g, T, h, 64) * 2.0 ** 57 for h in (H, 1))
    q, k = q.to(dtype), k.to(dtype)
    v, do = normal(g, T, 1, 64, dtype=dtype), normal(g, T, H, 64, dtype=dtype)
    lse = torch.empty(T, H, device=dev)
    x = [t.to(dev) for t in (q, k, v)]
    o = kda.attn_prefill(*x, i32(cu, dev), lse=lse, scale=scale)
    # scores of at most 2^122 2^-127 = 2^-5 with the same error in the smallest numbers' steps: a scale that is no
    # normal number is off by up to 2^-150 of 2^-130 (2^-20 relative), and log2(e) times it by as much again
    off = 2 * 2.0 ** -5 * 2 * 2.0 ** -20 + 100 * 2.0 ** -24
    if scale == 0:
        off += 2.0 ** 122 * 2.0 ** -149
    ref, ref_lse, o_abs = OA.prefill(f64(q), f64(k), f64(v), cu, cu, scale)
    assert (np.abs(f64(lse) - ref_lse) <= off + 8 * 2.0 ** -24 * 8).all()
    assert (np.abs(f64(o) - ref) <= o_abs * (off + 2 * U[dtype]) * 1.01 + 1e-37).all()
    dv = kda.attn_backward(*x, o, lse, do.to(dev), i32(cu, dev), scale=scale)[2]
    want, mag = OA.backward(f64(q), f64(k), f64(v), f64(do), cu, cu, scale)
    assert (np.abs(f64(dv) - want[2]) <= mag[2] * (2 * off + (200 * 2.0 ** -24) + 2 * U[dtype]) * 1.01 + 1e-37).all()


def late_keys(T, late, d):
    """Keys whose scores with q = (1, 0, ..) are 0 for the first 64 and `late` after them."""
    k = torch.zeros(T, 1, d)
    k[64:, 0, 0] = late
    return k


@pytest.mark.parametrize("T", [1000, 4096])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_values_as_large_as_allowed(T, dtype):
    """|v| up to 2^119 / keys, all of one sign, and scores that pass the running maximum by 2^7.9 without
    moving it: the largest sums that the header allows, in one tile's workgroup and in several parts."""
    dev = need_gpu()
    announce("prefill, values of 2^119 / %d %s" % (T, dtype))
    g = torch.Generator().manual_seed(2)
    q = torch.zeros(T, 2, 64)
    q[:, :, 0] = 1
    k = late_keys(T, 5.4375, 64)  # 8 bits, 7.84 in powers of two
    v = ((1 + torch.rand(T, 1, 64, generator=g)) * 2.0 ** 118 / T)
    q, k, v = (x.to(dtype) for x in (q, k, v))
    assert float(v.abs().max()) * T <= 2.0 ** 119
    o = kda.attn_prefill(q.to(dev), k.to(dev), v.to(dev), i32([0, T], dev), scale=1.0)
    ref, _, o_abs = OA.prefill(f64(q), f64(k), f64(v), [0, T], [0, T], 1.0)
    assert (np.abs(f64(o) - ref) <= o_bound(o_abs, f64(q), f64(k), 1.0, T, dtype)).all()


@pytest.mark.parametrize("L,T", [(1000, 1), (20000, 3)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_cached_values_as_large_as_allowed(L, T, dtype):
    """The same over the 8-bit cache, in one piece and in several: 448 times a block's scale up to
    2^119 / keys."""
    dev = need_gpu()
    announce("decode, values of 2^119 / %d %s" % (L, dtype))
    cache = Cache(1, L, 64, 1, 64, 64, dev)
    g = torch.Generator().manual_seed(3)
    e = int(np.floor(119 - np.log2(448 * L)))
    v = (300 + 148 * torch.rand(L, 1, 64, generator=g)) * 2.0 ** e
    cache.append(late_keys(L, 5.4375, 64), v, [L], [0])
    assert (cache.vs[cache.table[0].long()] == 2.0 ** e).all()
    q = torch.zeros(1, T, 4, 64)
    q[..., 0] = 1
    q = q.to(dtype)
    o = kda.attn_decode(q.to(dev), *cache.tensors(), i32([L], dev), scale=1.0)
    check_decode(cache, q, [L], 1.0, o)
