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


def _cu(lengths):
    return torch.tensor(np.concatenate([[0], np.cumsum(lengths)]), dtype=torch.int32, device="cuda")


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


def test_most_features(pv):
    """Out features up to the last multiple of 8 below 2^31."""
    N, K = (1 << 31) - 8, 8
    at = torch.tensor([0, 127, 1 << 30, N - 129, N - 128, N - 2, N - 1], device="cuda")
    rows = torch.arange(1, len(at) + 1, device="cuda").to(BF16)
    w = torch.zeros(N, K, dtype=BF16, device="cuda")
    w[at, 3] = rows
    x = torch.zeros(2, K, dtype=BF16, device="cuda")
    x[0, 3], x[1, 3] = 1.0, 2.0
    y = pv.linear_act_bf16(x[:1], w)
    assert torch.equal(y[0, at], rows) and int(y.count_nonzero()) == len(at)
    del y
    y = pv.linear_gated_bf16(x[1:], w, w, act="none")
    assert torch.equal(y[0, at], 4 * rows * rows) and int(y.count_nonzero()) == len(at)
    assert pv.get_device_status() == 0


def test_an_item_of_seconds(pv):
    """One query over 3 2^28 keys, some 4 s of one SM, and behind it items of two tiles, of
    which that one has the first: whoever works on the second tile has nothing to do
    meanwhile.  The keys are alike but for one of the last tile, whose score is 64 above."""
    D, n, more = 64, 3 << 28, 2 * 152 * 256
    kv = torch.zeros(n + 1, 1, D, dtype=BF16, device="cuda")
    kv[n - 3] = 1.0
    kv[n:] = 3.0
    q = torch.full((1 + more, 1, D), 8.0, dtype=BF16, device="cuda")
    out = pv.prompt_attn_fwd(q, kv, kv, _cu([1, more]), _cu([n, 1]), more, n, causal=False)
    assert pv.get_device_status() == 0
    # (the others' weights: 2^30 e^-64 in all at most, of values of zero)
    assert (out[:1] == 1.0).all() and (out[1:] == 3.0).all()


def test_counts_beyond_32_bits_are_refused(pv):
    """Sizes of 2^32 + 8 are not sizes of 8."""
    n = (1 << 32) + 8
    big = torch.zeros(n, 8, dtype=BF16, device="cuda")
    few = torch.zeros(8, 8, dtype=BF16, device="cuda")
    deep = big.view(8, n)
    out = torch.zeros(8, 8, dtype=BF16, device="cuda")
    out[:] = 5.0

    def refused(call, *args, **kw):
        with pytest.raises(pv.PackedAttnError) as e:
            call(*args, **kw)
        assert e.value.status == 2

    refused(pv.linear_bf16, big, few)
    refused(pv.linear_bf16, few, big)
    refused(pv.linear_bf16, deep, deep, out=out)
    refused(pv.linear_act_bf16, big, few)
    refused(pv.linear_act_bf16, few, big)
    refused(pv.linear_act_bf16, deep, deep, out=out)
    refused(pv.linear_gated_bf16, big, few, few)
    refused(pv.linear_gated_bf16, few, big, big)
    refused(pv.linear_gated_bf16, deep, deep, deep, out=out)
    assert (out == 5).all()
    at = torch.zeros(1, n, dtype=torch.int32, device="cuda")
    refused(pv.rope_axes, big.view(n, 1, 8), None, at, [8])
    at = at[:, :1].contiguous()
    refused(pv.rope_axes, big.view(1, n, 8), None, at, [8])
    refused(pv.rope_axes, big.view(-1)[:n].view(1, 1, n), None, at, [8])
    q = big.view(-1)[:(1 << 32) + 64].view(1, 1, -1)
    refused(pv.prompt_attn_fwd, q, q, q, _cu([1]), _cu([1]), 1, 1)
    del big, deep, q
    one = torch.zeros(1, 1, 64, dtype=BF16, device="cuda")
    cu = torch.zeros((1 << 32) + 2, dtype=torch.int32, device="cuda")
    refused(pv.prompt_attn_fwd, one, one, one, cu, cu, 1, 1)
    assert pv.get_device_status() == 0


def test_a_sum_of_seconds(pv):
    """linear_bf16 over K = 3 2^28: a tile of some 3 s."""
    K = 3 << 28
    x, w = (torch.zeros(n, K, dtype=BF16, device="cuda") for n in (2, 8))
    at = torch.tensor([0, 63, 1 << 28, K - 65, K - 1], device="cuda")
    w[:, at] = torch.arange(1, 9, device="cuda").to(BF16)[:, None]
    x[0, at], x[1, at[:2]] = 1.0, 3.0
    y = pv.linear_bf16(x, w)
    assert pv.get_device_status() == 0
    want = torch.arange(1, 9, device="cuda").to(BF16)
    assert torch.equal(y[0], 5 * want) and torch.equal(y[1], 6 * want)
