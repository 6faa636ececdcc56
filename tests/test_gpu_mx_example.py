"""The expert layer of examples/mxfp4_experts.py: trains, agrees with a plain
fp32 layer on the cast's values, and decodes to the same outputs."""
import importlib.util
import os

import numpy as np
import pytest
import torch

import nvfp4_block_scaled_bf16_amd as nv
from tests import mx_ref

pytestmark = pytest.mark.gpu
PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "mxfp4_experts.py")


@pytest.fixture(scope="module")
def ex():
    spec = importlib.util.spec_from_file_location("mxfp4_experts", PATH)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_trains_and_decodes(ex):
    losses, router, w1, w2, x = ex.train(tokens=300, hidden=160, inner=200, experts=6, topk=2, steps=15, log=lambda s: None)
    assert losses[-1] < 0.7 * losses[0] and all(np.isfinite(losses))
    q1, q2 = ex.cast_weights(w1, columnwise=False), ex.cast_weights(w2, columnwise=False)
    whole = ex.layer(x, router, w1, w2, 2)
    for n in (1, 5, 40):
        y = ex.decode(x[:n], router, q1, q2, 2)
        # the decoded rows' weights multiply before the one rounding (fp32), the
        # trained layer's after a rounding to bf16: 2^-8 of each of its two terms
        scale = whole[:n].abs().amax()
        assert (y - whole[:n]).abs().max() <= 2.0 ** -6 * scale


def test_gradients_of_the_expert_linear(ex):
    # against the formulas in 64 bits, each operand cast along the sum
    rng = np.random.default_rng(1)
    T, K, N, E, R = 50, 96, 70, 4, 120
    off = np.array([0, 30, 30, 85, 120], np.int32)
    idx = rng.integers(0, T, R).astype(np.int32)
    x = torch.from_numpy(rng.standard_normal((T, K))).bfloat16().cuda().requires_grad_()
    w = torch.from_numpy(rng.standard_normal((E, N, K)) / 10).float().cuda().requires_grad_()
    dy = torch.from_numpy(rng.standard_normal((R, N))).bfloat16().cuda()
    y = ex.ExpertLinear.apply(x, w, torch.from_numpy(off).cuda(), torch.from_numpy(idx).cuda())
    y.backward(dy)
    xv, wv, dv = mx_ref.host64(x), mx_ref.host64(w.detach().bfloat16()), mx_ref.host64(dy)
    dx = np.zeros((T, K))
    for e in range(E):
        s, t = off[e], off[e + 1]
        if s == t:
            assert not w.grad[e].any()
            continue
        mx_ref.check_product(y[s:t].detach(), mx_ref.fake(xv)[idx[s:t]], mx_ref.fake(wv[e]))
        mx_ref.check_product(w.grad[e], mx_ref.fake(dv[s:t].T), mx_ref.fake(xv[idx[s:t]].T))
        np.add.at(dx, idx[s:t], mx_ref.fake(dv[s:t]) @ mx_ref.fake(wv[e].T).T)
    # bf16 rows added in fp32, rounded again: at most 2^-7 of the largest sums
    assert np.abs(mx_ref.host64(x.grad) - dx).max() <= 2.0 ** -7 * np.abs(dx).max()


def test_casts_agree_with_the_grouped_layout(ex):
    w = torch.randn(3, 40, 70, device="cuda")
    q = ex.cast_weights(w)
    for e in range(3):
        v = nv.mx_dequantize(q["row_q"][e].contiguous(), q["row_sf"][e].contiguous(), 70)
        assert np.array_equal(mx_ref.host64(v), mx_ref.fake(mx_ref.host64(w[e].bfloat16())))
