"""Edges of the operators of a layer over packed prompts: far tails, sizes at the ends of
their ranges, numbers given in other forms."""
import math

import numpy as np
import pytest
import torch

import oracle

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


@pytest.fixture(scope="module")
def pv():
    import packed_varlen_gb300 as pv
    pv.load_library()
    pv.get_device_status()
    return pv


TAILS = {"silu": np.arange(-99.0, -79.9, 0.5),            # to e^-99
         "gelu_tanh": np.arange(-10.375, -9.0, 0.0625),   # to e^-97
         "gelu": np.arange(-13.75, -11.9, 0.0625)}        # to e^-97


@pytest.mark.parametrize("M", [37, 1300])
@pytest.mark.parametrize("act", sorted(TAILS))
def test_far_tails_of_the_activations(pv, act, M):
    """Results down to bf16's subnormal numbers, where exp of the argument's size has left
    fp32's range.  The exponent is off by 6 roundings (2^-24 each) of at most 99, which
    its power multiplies: 2^-14 of the result holds that, the approximate exp2 and
    quotient, and erfc's argument (2 x^2 2^-23 with x^2 < 95).  The result's
    rounding is 2^-8 of it, or half of the least subnormal number, 2^-134."""
    v = torch.as_tensor(TAILS[act]).to(BF16)
    assert (v.double() == torch.as_tensor(TAILS[act])).all()
    N, K = 2056, 136
    x, w, up = (torch.zeros(n, K, dtype=BF16) for n in (M, N, N))
    x[:, 0], x[:, 1] = v.repeat(M // len(v) + 1)[:M], 1.0
    w[:, 0], up[:, 1] = 1.0, 2.0
    want = oracle.activation(oracle.to_f64(x[:, 0]), act)[:, None]
    assert 0 < -want.max() < 2.0 ** -133
    got = oracle.to_f64(pv.linear_act_bf16(x.cuda(), w.cuda(), act=act))
    loss = (2.0 ** -8 * (1 + 2.0 ** -7) + 2.0 ** -14) * np.abs(want) + 2.0 ** -134 * (1 + 2.0 ** -7)
    assert (np.abs(got - want) <= loss).all()
    got = oracle.to_f64(pv.linear_gated_bf16(x.cuda(), w.cuda(), up.cuda(), act=act))
    assert (np.abs(got - 2 * want) <= 2 * loss).all()
    assert pv.get_device_status() == 0
