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


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("power", [80, 104, 112, 120])
def test_small_values(pv, power, causal, D):
    """V near the end of fp32's range.  A product of weight and value, and each sum of them, is
    cut at 2^-149 at the worst; the largest weight is 1 at least, or 2^-24 in causal order, by
    which the sum is divided: 2 n 2^-149 (or 2^-125) beside the relative errors."""
    n, Hq, H = 300, 4, 2
    q, k, v = (torch.randn(n, h, D, generator=torch.Generator().manual_seed(h)).to(BF16)
               for h in (Hq, H, H + 1))
    v = (v[:, :H].float() * 2.0 ** -power).to(BF16)
    out = pv.prompt_attn_fwd(q.cuda(), k.cuda(), v.cuda(), _cu([n]), _cu([n]), n, n, causal=causal)
    want, weight, reach = oracle.prompt_attention(q, k, v, [n], [n], causal, D ** -0.5)
    scores = (D + 4) * 2.0 ** -23 * reach + 2.0 ** -20
    loss = (2.0 ** -8 + 2 * scores) * weight + 2.0 ** -8 * np.abs(want) * (1 + 2.0 ** -7)
    loss = loss + 2 * n * 2.0 ** (-125 if causal else -149) + 2.0 ** -134
    assert (np.abs(oracle.to_f64(out) - want) <= loss).all()
    assert pv.get_device_status() == 0


def test_calls_that_follow_each_other(pv):
    """Calls in a row, each set up beside the one before it, over buffers that the ones before
    write or read (weights among them): the bits of the same calls with a wait after each,
    eager and out of a graph."""
    T, C, H, D = 600, 1024, 8, 128

    def rn(*shape, seed):
        return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(BF16).cuda()

    first = [rn(T, C, seed=i) for i in range(3)] + [rn(C, C, seed=i) / 32 for i in (3, 4)]
    cu, many = _cu([13, 287, 0, 300]), _cu([1, 599])
    pos = torch.arange(2 * T, dtype=torch.int32, device="cuda").view(2, T)
    lens, table = _cu([600])[1:], torch.arange(40, dtype=torch.int32, device="cuda").view(1, 40)
    work = torch.empty(32 << 20, dtype=torch.uint8, device="cuda")
    caches = [torch.zeros(40, 16, 2, D, dtype=BF16, device="cuda") for _ in range(2)]

    def heads(x, n=H, at=0):
        return x.view(T, C // D, D)[:, at:at + n]

    def run(a, b, c, w, u, wait):
        def narrow():                                    # heads of 64, over other boundaries
            pv.prompt_attn_fwd(a.view(T, 16, 64), b.view(T, 16, 64)[:, :4],
                               b.view(T, 16, 64)[:, 4:8], many, many, 599, 599,
                               out=c.view(T, 16, 64))

        calls = [
            lambda: pv.linear_act_bf16(a, w, act="silu", residual=b, out=b),
            lambda: pv.rope_axes(heads(b, 4), heads(b, 4, 4), pos, [64, 64]),
            lambda: pv.kv_cache_write(heads(b, 2), heads(b, 2, 2), *caches, _cu600, table),
            lambda: pv.prompt_attn_fwd(heads(b), heads(a, 2), heads(a, 2, 2), cu, cu, 300, 300,
                                       out=heads(c)),
            lambda: pv.linear_gated_bf16(c, w, u, out=a),
            narrow,
            lambda: pv.linear_act_bf16(c[:13], w, act="gelu", residual=a[:13], out=a[:13]),
            lambda: pv.paged_attn_fwd(heads(a), *caches, _cu600, lens, table, 600, 600,
                                      out=heads(b), workspace=work),
            lambda: pv.linear_act_bf16(b[:20], u, out=w[40:60]),       # weights of the next
            lambda: pv.linear_gated_bf16(a[:5], w, u, act="relu", out=c[7:12]),
            lambda: pv.varlen_attn_fwd(heads(c), heads(b), heads(a), cu, cu, 300, 300,
                                       out=spare),
            lambda: pv.linear_bf16(spare.view(T, C), w, out=b),
            lambda: pv.block_window_attn_fwd(*(x.view(1, T, H, D) for x in (b, c, a)), 24, 1, 0,
                                             out=spare.view(1, T, H, D)),
            lambda: pv.linear_act_bf16(spare.view(T, C)[300:330], u, residual=a[:30], out=a[:30]),
            lambda: a.clamp_(-3, 3),
        ]
        for call in calls * 3:
            call()
            if wait:
                torch.cuda.synchronize()

    _cu600, spare = _cu([600]), torch.zeros(T, H, D, dtype=BF16, device="cuda")

    def fresh():
        torch.cuda.synchronize()
        for t in caches + [spare]:
            t.zero_()
        return [x.clone() for x in first]

    def seen(buffers):
        torch.cuda.synchronize()
        return [t.clone().view(torch.int16) for t in [*buffers, *caches, spare]]

    buffers = fresh()
    run(*buffers, True)
    want = seen(buffers)
    for _ in range(5):
        buffers = fresh()
        torch.cuda.synchronize()
        run(*buffers, False)
        assert all(torch.equal(x, y) for x, y in zip(want, seen(buffers)))
    buffers = fresh()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run(*buffers, False)
    for _ in range(3):
        for x, y in zip(buffers, fresh()):
            x.copy_(y)
        graph.replay()
        assert all(torch.equal(x, y) for x, y in zip(want, seen(buffers)))
    assert pv.get_device_status() == 0
