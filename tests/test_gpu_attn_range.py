"""Softmax attention at the ends of the numbers' range: scales of zero and below the smallest normal
number with large scores, and values as large as the header allows."""
import numpy as np
import pytest
import torch

import kda_gated_delta_rule_amd as kda
from _attn import U, cu_of, i32, normal
from _util import announce, f64, need_gpu
from oracle import kda_attn as OA

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
