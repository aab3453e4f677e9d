"""The operators of a layer over packed prompts on the GPU against the fp64 oracle."""
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


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _cu(lengths):
    return _i32(np.concatenate([[0], np.cumsum(lengths)]).tolist())


def _randn(*shape, seed, spread=0.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(*shape, generator=g)
    if spread:
        x = x * torch.exp(spread * torch.randn(*shape[:-1], 1, generator=g))
    return x.to(BF16)


def _bits(x):
    return x.contiguous().view(torch.int16)


def _within(got, want, tolerance):
    got = oracle.to_f64(got)
    assert np.isfinite(got).all()
    excess = np.abs(got - want) - tolerance
    assert excess.size == 0 or excess.max() <= 0, \
        f"{(excess > 0).sum()} of {excess.size} beyond, worst {excess.max():.3e} at " \
        f"{np.unravel_index(excess.argmax(), excess.shape)}"


# ------------------------------------------------------------------ attention

def _attention_tolerance(want, weight, reach, D):
    """fp32 scores, sums and accumulation, weights and output rounded to bf16.
    The weights' rounding (2^-8 of each) moves a result by at most 2^-8 of
    sum w |v|, the output's by 2^-8 of itself.  A score's fp32 sum of D
    products (each exact) is off by at most D 2^-23 of sum |q k| (additions
    that may truncate), the exponent's arithmetic and exp2 by 2^-22 of the
    largest score and of the weight; twice that for numerator and sum."""
    scores = (D + 4) * 2.0 ** -23 * reach + 2.0 ** -20
    return (2.0 ** -8 + 2 * scores) * weight + 2.0 ** -8 * np.abs(want) * (1 + 2.0 ** -7) + 1e-30


def _attend(pv, q, k, v, lq, lk, causal=True, scale=None, extra=3, **kw):
    out = torch.full((q.shape[0] + extra,) + tuple(q.shape[1:]), 5.0, dtype=BF16, device="cuda")
    q = torch.cat([q, q.new_full((extra,) + tuple(q.shape[1:]), math.nan)])
    pv.prompt_attn_fwd(q, k, v, _cu(lq), _cu(lk), max(lq + [0]), max(lk + [0]), causal=causal,
                       scale=scale, out=out, **kw)
    assert pv.get_device_status() == 0
    assert (out[sum(lq):].float() == 5.0).all()
    return out[:sum(lq)]


def _rows_of(lq, per_tile=2, seed=0):
    """Rows of every 128-row tile, and those at the edges."""
    rng, rows, q0 = np.random.default_rng(seed), set(), 0
    for n in lq:
        for t in range(0, n, 128):
            end = min(n, t + 128)
            rows |= {q0 + t, q0 + end - 1}
            rows |= set((q0 + rng.integers(t, end, per_tile)).tolist())
        q0 += n
    return sorted(rows)


def _attention_case(pv, lq, lk, Hq, H, D, causal, scale=None, seed=0, spread=0.3, past=math.nan,
                    sampled=False):
    """Rows past the last sequence hold NaN or infinities."""
    q = _randn(sum(lq), Hq, D, seed=seed)
    k, v = (_randn(sum(lk), H, D, seed=seed + i, spread=spread) for i in (1, 2))
    tail = torch.full((130, H, D), past, dtype=BF16)
    kd, vd = (torch.cat([x, tail]).cuda() for x in (k, v))
    out = _attend(pv, q.cuda(), kd, vd, lq, lk, causal, scale)
    rows = _rows_of(lq) if sampled else None
    want, weight, reach = oracle.prompt_attention(q, k, v, lq, lk, causal,
                                                  D ** -0.5 if scale is None else scale, rows)
    got = out if rows is None else out[torch.as_tensor(rows, device="cuda")]
    _within(got, want, _attention_tolerance(want, weight, reach, D))
    return out


PROMPTS = [
    # query lengths, key lengths (None: the same), Hq, Hkv, D
    ([1], None, 1, 1, 64),
    ([1], None, 8, 2, 128),
    ([1, 2, 3, 1], None, 4, 4, 128),
    ([127, 128, 129], None, 4, 2, 128),
    ([255, 256, 257, 1], None, 6, 3, 64),
    ([511, 513, 40], None, 4, 1, 128),
    ([300, 0, 20], None, 7, 1, 64),
    ([700], None, 2, 2, 128),
    ([384, 640], None, 3, 3, 64),
    ([40, 200, 1], [340, 200, 129], 8, 2, 128),      # behind a prefix
    ([130, 1, 260], [1000, 515, 300], 4, 1, 64),
    ([300, 70, 5, 9], [130, 7, 0, 1], 4, 2, 128),    # fewer keys than queries
    ([600, 3], [257, 2], 2, 1, 64),
]


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("lq,lk,Hq,H,D", PROMPTS)
def test_prompts(pv, lq, lk, Hq, H, D, causal):
    _attention_case(pv, lq, lq if lk is None else lk, Hq, H, D, causal)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("lq,lk", [([3000, 1111, 5], None), ([1500], [4003]), ([2100], [900])])
def test_long_prompts(pv, lq, lk, D):
    _attention_case(pv, lq, lq if lk is None else lk, 4, 2, D, True, sampled=True)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("Hq,H", [(24, 24), (32, 4), (128, 1)])
def test_many_items(pv, Hq, H, D, causal):
    """Several items for every SM, of one to six key tiles, in all orders."""
    lengths = [700, 130, 1, 257, 64, 390, 128, 20, 513, 300]
    _attention_case(pv, lengths, lengths, Hq, H, D, causal, sampled=True)


@pytest.mark.parametrize("D", [64, 128])
def test_rows_that_see_nothing_are_zero(pv, D):
    out = _attention_case(pv, [3, 300, 400, 0], [0, 130, 10, 20], 4, 2, D, True)
    assert (out[:3] == 0).all() and (out[3:173] == 0).all() and (out[303:693] == 0).all()
    assert (out[173:303].float().abs().amax(-1) > 0).all()
    out = _attention_case(pv, [3, 300], [0, 130], 4, 2, D, False)
    assert (out[:3] == 0).all()


@pytest.mark.parametrize("D", [64, 128])
def test_no_keys_in_the_call(pv, D):
    q = _randn(300, 4, D, seed=1).cuda()
    none = torch.empty(0, 2, D, dtype=BF16, device="cuda")
    for causal in (True, False):
        out = _attend(pv, q, none, none, [290, 10], [0, 0], causal)
        assert (out == 0).all()


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("past", [math.inf, -math.inf, math.nan])
def test_rows_past_a_sequence_never_reach_it(pv, past, D):
    """Behind the last sequence, and between two."""
    _attention_case(pv, [130, 77], [200, 77], 4, 2, D, True, past=past)
    lengths = [70, 150, 200]
    q = _randn(sum(lengths), 4, D, seed=3)
    k, v = _randn(sum(lengths), 2, D, seed=4), _randn(sum(lengths), 2, D, seed=5)
    k[70:220] = past
    v[70:220] = past
    out = _attend(pv, q.cuda(), k.cuda(), v.cuda(), lengths, lengths)
    for a, b in ((0, 70), (220, 420)):
        want, weight, reach = oracle.prompt_attention(q[a:b], k[a:b], v[a:b], [b - a], [b - a],
                                                      True, D ** -0.5)
        _within(out[a:b], want, _attention_tolerance(want, weight, reach, D))


@pytest.mark.parametrize("D", [64, 128])
def test_hidden_keys_of_any_bits(pv, D):
    """NaN and infinities in K rows that causal order hides reach nothing."""
    n = 300
    q, k, v = _randn(n, 2, D, seed=1), _randn(n, 1, D, seed=2), _randn(n, 1, D, seed=3)
    for bad in (math.nan, math.inf, -math.inf):
        dirty = k.clone()
        dirty[201:] = bad
        out = _attend(pv, q.cuda(), dirty.cuda(), v.cuda(), [n], [n])[:201]
        want, weight, reach = oracle.prompt_attention(q[:201], k[:201], v[:201], [201], [201], True,
                                                      D ** -0.5)
        _within(out, want, _attention_tolerance(want, weight, reach, D))


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("scale", [0.0, -0.2, 1.5, 1e-4])
def test_scales(pv, scale, D):
    _attention_case(pv, [300, 20, 1], [300, 130, 1], 4, 2, D, True, scale=scale)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("slope", [(0.05, 6.0), (6.0, 0.05)])
def test_growing_and_falling_scores(pv, slope, D):
    n = 1500
    q, v = _randn(n, 2, D, seed=1), _randn(n, 1, D, seed=2)
    k = (_randn(n, 1, D, seed=3).float() * torch.linspace(*slope, n)[:, None, None]).to(BF16)
    out = _attend(pv, q.cuda(), k.cuda(), v.cuda(), [n], [n])
    rows = _rows_of([n], 4)
    want, weight, reach = oracle.prompt_attention(q, k, v, [n], [n], True, D ** -0.5, rows)
    _within(out[torch.as_tensor(rows, device="cuda")], want,
            _attention_tolerance(want, weight, reach, D))


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("reach", [12, 20, 29])
def test_large_scores(pv, reach, causal, D):
    """Exact scores up to 2^reach once scaled, each row's largest one at least 2^(reach - 8)
    above the others, so that its weight is all there is (e^-16 times a few v beside it: below
    2^-18): out is that key's v, but for the rounding of the weight and of the result."""
    lq, lk, Hq, H = [300, 140], [300, 400], 4, 2
    q = torch.zeros(sum(lq), Hq, D, dtype=BF16)
    q[..., 0] = 1.0
    v = _randn(sum(lk), H, D, seed=3)
    rng, k0, q0 = np.random.default_rng(7), 0, 0
    k = torch.zeros(sum(lk), H, D, dtype=BF16)
    for n in lk:
        # multiples of 2^(reach - 8), no two alike among 128 keys; those set apart below are each
        # larger than all before
        size = np.array([rng.permutation(200)[:128] for _ in range(-(-n // 128))]).ravel()[:n]
        k[k0:k0 + n, :, 0] = torch.as_tensor(
            (size[:, None] - 255.0) * 2.0 ** (reach - 8)).to(BF16)
        k[k0 + 5, :, 0] = 2.0 ** (reach - 4)
        k[k0 + n // 2, :, 0] = 2.0 ** (reach - 1)
        k[k0 + n - 9, :, 0] = 2.0 ** reach
        k0 += n
    out = oracle.to_f64(_attend(pv, q.cuda(), k.cuda(), v.cuda(), lq, lk, causal, 1.0))
    k0, seen = 0, 0
    for nq, n in zip(lq, lk):
        for i in range(nq):
            end = n - nq + i + 1 if causal else n
            size = oracle.to_f64(k[k0:k0 + end, 0, 0])
            order = np.sort(size)
            if end > 1 and order[-1] - order[-2] < 2.0 ** (reach - 8):
                continue
            want = oracle.to_f64(v[k0 + int(size.argmax())])[[0, 0, 1, 1]]
            assert (np.abs(out[q0 + i] - want) <= 2.0 ** -7 * 1.01 * np.abs(want) + 2.0 ** -18).all(), \
                (i, end)
            seen += 1
        k0, q0 = k0 + n, q0 + nq
    assert seen > 300


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_a_bad_query_stays_its_own(pv, bad, D):
    """NaN or an infinity in one row of q, beside other heads and tokens of its tile."""
    lq, Hq, H = [70, 300], 6, 2
    q = _randn(sum(lq), Hq, D, seed=1)
    k, v = _randn(sum(lq), H, D, seed=2), _randn(sum(lq), H, D, seed=3)
    rows = [(40, 1), (200, 3), (69, 5)]
    for t, h in rows:
        q[t, h, 7] = bad
    out = oracle.to_f64(_attend(pv, q.cuda(), k.cuda(), v.cuda(), lq, lq))
    for t, h in rows:
        assert not np.isfinite(out[t, h]).any()
        q[t, h] = 0
        out[t, h] = 0
    want, weight, reach = oracle.prompt_attention(q, k, v, lq, lq, True, D ** -0.5)
    for t, h in rows:
        want[t, h] = 0
    _within(torch.as_tensor(out), want, _attention_tolerance(want, weight, reach, D))


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("G", [100, 127])
def test_groups_that_leave_rows_of_a_tile(pv, G, D):
    _attention_case(pv, [1, 5, 140], [1, 300, 140], 2 * G, 2, D, True)


@pytest.mark.parametrize("D", [64, 128])
def test_first_boundary_is_zero(pv, D):
    """Boundaries that start elsewhere: the first sequence is skipped, its rows untouched."""
    lq, at = [40, 3], 29
    q, k, v = (_randn(at + 43, h, D, seed=h + 1) for h in (4, 2, 2))
    out = torch.full(q.shape, 5.0, dtype=BF16, device="cuda")
    cu = _cu(lq) + at
    pv.prompt_attn_fwd(q.cuda(), k.cuda(), v.cuda(), cu, cu, 40, 40, out=out)
    assert pv.get_device_status() == 1 and (out[:69] == 5).all()
    want, weight, reach = oracle.prompt_attention(q[69:], k[69:], v[69:], [3], [3], True, D ** -0.5)
    _within(out[69:], want, _attention_tolerance(want, weight, reach, D))


@pytest.mark.parametrize("D", [64, 128])
def test_slices_of_a_fused_projection(pv, D):
    lengths, Hq, H = [130, 300, 1], 8, 2
    T = sum(lengths)
    fused = _randn(T, Hq + 2 * H + 1, D, seed=6).cuda()      # (a head that is not read)
    q, k, v = fused[:, :Hq], fused[:, Hq:Hq + H], fused[:, Hq + H:Hq + 2 * H]
    cu = _cu(lengths)
    got = pv.prompt_attn_fwd(q, k, v, cu, cu, 300, 300)
    want = pv.prompt_attn_fwd(q.contiguous(), k.contiguous(), v.contiguous(), cu, cu, 300, 300)
    assert pv.get_device_status() == 0
    assert torch.equal(_bits(got), _bits(want))


@pytest.mark.parametrize("D", [64, 128])
def test_bits_do_not_depend_on_the_batch(pv, D):
    lengths, Hq, H = [700, 129, 1, 256, 333], 4, 2
    T, cu = sum(lengths), np.cumsum([0] + lengths)
    q, k, v = (_randn(T, h, D, seed=s).cuda() for s, h in ((1, Hq), (2, H), (3, H)))
    whole = _attend(pv, q, k, v, lengths, lengths)
    assert torch.equal(_bits(whole), _bits(_attend(pv, q, k, v, lengths, lengths)))
    for b, n in enumerate(lengths):
        at = slice(cu[b], cu[b + 1])
        alone = _attend(pv, q[at], k[at], v[at], [n], [n])
        assert torch.equal(_bits(whole[at]), _bits(alone))
    order = [3, 0, 4, 2, 1]
    pick = torch.cat([torch.arange(cu[b], cu[b + 1]) for b in order]).cuda()
    moved = _attend(pv, q[pick], k[pick], v[pick], [lengths[b] for b in order],
                    [lengths[b] for b in order])
    assert torch.equal(_bits(moved), _bits(whole[pick]))


@pytest.mark.parametrize("D", [64, 128])
def test_against_the_operators_beside_it(pv, D):
    """Without causal order and with equal heads: the bits of varlen_attn_fwd.
    With K/V rows repeated for every query head: the bits of grouped heads.
    Single queries over the same rows in a paged cache: the same values."""
    lengths, H = [300, 513, 64], 3
    T = sum(lengths)
    q, k, v = (_randn(T, H, D, seed=s).cuda() for s in (1, 2, 3))
    cu = _cu(lengths)
    plain = pv.varlen_attn_fwd(q, k, v, cu, cu, 513, 513)
    assert torch.equal(_bits(plain), _bits(_attend(pv, q, k, v, lengths, lengths, False)))
    q2 = _randn(T, 2 * H, D, seed=4).cuda()
    for causal in (True, False):
        a = _attend(pv, q2, k, v, lengths, lengths, causal)
        b = _attend(pv, q2, k.repeat_interleave(2, 1), v.repeat_interleave(2, 1), lengths, lengths,
                    causal)
        assert torch.equal(_bits(a), _bits(b))


@pytest.mark.parametrize("D", [64, 128])
def test_attention_refusals_on_the_device(pv, D):
    q, k, v = (_randn(400, h, D, seed=h).cuda() for h in (4, 2, 2))

    def run(cu_q, cu_k, max_q=200, max_k=200):
        out = torch.full_like(q, 5.0)
        pv.prompt_attn_fwd(q, k, v, _i32(cu_q), _i32(cu_k), max_q, max_k, out=out)
        return out

    good = run([0, 100, 200], [0, 100, 200])
    assert pv.get_device_status() == 0
    for cu_q, cu_k, code in [([1, 100, 200], [0, 100, 200], 1), ([0, 100, 401], [0, 100, 200], 1),
                             ([0, 100, 90], [0, 100, 200], 1), ([0, 100, 200], [0, 100, 500], 1),
                             ([0, 100, 200], [-1, 100, 200], 1), ([0, 100, 301], [0, 100, 200], 2),
                             ([0, 100, 200], [0, 100, 305], 2),
                             ([0, -2147483648, 200], [0, 100, 200], 1),
                             ([0, 100, 2147483647], [0, 100, 200], 1)]:
        out = run(cu_q, cu_k)
        assert pv.get_device_status() == code, (cu_q, cu_k)
        first_ok = cu_q[:2] == [0, 100] and cu_k[:2] == [0, 100]
        if first_ok:
            assert torch.equal(_bits(out[:100]), _bits(good[:100]))
        assert (out[200 if not first_ok else 100:].float() == 5.0).all()


def test_attention_binding_refusals(pv):
    q, k = _randn(20, 4, 64, seed=1).cuda(), _randn(20, 2, 64, seed=2).cuda()
    cu = _cu([20])

    def run(**kw):
        a = dict(q=q, k=k, v=k, cu_seqlens_q=cu, cu_seqlens_k=cu, max_q=20, max_k=20)
        a.update(kw)
        return pv.prompt_attn_fwd(**a)

    for kw in [dict(k=k[:10]), dict(q=q[:, :3]), dict(q=q[..., :32]), dict(k=k.transpose(0, 1)),
               dict(q=q.transpose(1, 2)), dict(cu_seqlens_k=_cu([10, 10])), dict(out=q[:10]),
               dict(q=q.cpu()), dict(k=k.cpu()), dict(cu_seqlens_q=cu.cpu()), dict(q=q[0]),
               dict(q=q.float()), dict(v=k.half()), dict(cu_seqlens_q=cu.long()), dict(q=None),
               dict(cu_seqlens_k=None), dict(out=7), dict(k=k[:, :0], v=k[:, :0])]:
        with pytest.raises((TypeError, ValueError)):
            run(**kw)
    for kw in [dict(scale=math.inf), dict(max_q=-1), dict(max_k=1 << 31), dict(max_q=1 << 40),
               dict(q=q[..., :32], k=k[..., :32], v=k[..., :32])]:
        with pytest.raises(pv.PackedAttnError):
            run(**{n: x.contiguous() if isinstance(x, torch.Tensor) else x for n, x in kw.items()})
    assert pv.get_device_status() == 0


@pytest.mark.parametrize("D", [64, 128])
def test_attention_in_graphs_and_on_streams(pv, D):
    """Two captured calls, replayed at once with new lengths and rows."""
    T, Hq, H, B = 900, 4, 2, 3
    q, k, v = (torch.zeros(T, h, D, dtype=BF16, device="cuda") for h in (Hq, H, H))
    cu = _cu([300, 300, 300])
    outs, graphs = [torch.zeros_like(q), torch.zeros_like(q)], []
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for o, s in zip(outs, streams):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            pv.prompt_attn_fwd(q, k, v, cu, cu, T, T, out=o)
        graphs.append(g)
    for step, lengths in enumerate([[300, 300, 300], [1, 0, 899], [257, 400, 30], [0, 0, 0]]):
        cu.copy_(_cu(lengths))
        for x, s in ((q, 0), (k, 1), (v, 2)):
            x.copy_(_randn(*x.shape, seed=10 * step + s).cuda())
        for o in outs:
            o.fill_(5.0)
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        assert pv.get_device_status() == 0
        n = sum(lengths)
        assert torch.equal(_bits(outs[0]), _bits(outs[1])) and (outs[0][n:].float() == 5.0).all()
        if n:
            want, weight, reach = oracle.prompt_attention(q.cpu(), k.cpu(), v.cpu(), lengths,
                                                          lengths, True, D ** -0.5)
            _within(outs[0][:n], want[:n], _attention_tolerance(want, weight, reach, D)[:n])


def test_many_sequences_and_heads(pv):
    rng = np.random.default_rng(5)
    lengths = rng.integers(0, 40, 1024).tolist()
    _attention_case(pv, lengths, lengths, 2, 1, 64, True)
    _attention_case(pv, [40, 3], [40, 3], 256, 2, 128, True)


def test_rows_beyond_32_bit_offsets(pv):
    """More than 2^32 elements of q and of out: the last sequence's rows."""
    Hq, H, D, n, B = 128, 1, 128, 260, 1012
    T = n * B
    assert T * Hq * D > 1 << 32
    q = torch.zeros(T, Hq, D, dtype=BF16, device="cuda")
    k, v = (torch.zeros(T, H, D, dtype=BF16, device="cuda") for _ in range(2))
    ends = [_randn(n, h, D, seed=s).cuda() for s, h in ((1, Hq), (2, H), (3, H))]
    for x, e in zip((q, k, v), ends):
        x[-n:] = e
    cu = _cu([n] * B)
    out = pv.prompt_attn_fwd(q, k, v, cu, cu, n, n)
    assert pv.get_device_status() == 0
    assert torch.equal(_bits(out[-n:]), _bits(_attend(pv, *ends, [n], [n])))
    assert (out[:n] == 0).all() and (out[-2 * n:-n] == 0).all()


# ------------------------------------------------------------------ rope

def _rope_tolerance(want, x, dims, halves):
    """One rounding to bf16; angles to 2^-22 (the fraction of a turn to 2^-53 of it times
    a position below 2^31), sin and cos to 2^-22, two products and a sum in
    fp32 (2^-23 of the pair's size in all): 2^-20 of the pair's size bounds their sum."""
    R = sum(dims)
    xx = oracle.to_f64(x)
    a, b = (xx[..., :R // 2], xx[..., R // 2:R]) if halves else (xx[..., :R:2], xx[..., 1:R:2])
    size = np.hypot(a, b)
    pair = np.zeros_like(xx)
    if halves:
        pair[..., :R // 2] = pair[..., R // 2:R] = size
    else:
        pair[..., :R:2] = pair[..., 1:R:2] = size
    return 2.0 ** -8 * np.abs(want) * (1 + 2.0 ** -7) + 2.0 ** -20 * pair


def _check_rope(got, x, positions, dims, base, halves, shared):
    want = oracle.rope_axes(x, positions, dims, base, halves, shared)
    _within(got, want, _rope_tolerance(want, x, dims, halves))
    R = sum(dims)
    assert torch.equal(_bits(got[..., R:].cpu()), _bits(x[..., R:]))


ROPES = [
    # tokens, Hq, Hkv, D, dims
    (1, 1, 1, 64, [64]),
    (48, 32, 8, 128, [32, 48, 48]),
    (301, 24, 24, 128, [16, 56, 56]),
    (77, 16, 16, 80, [40, 40]),
    (130, 3, 1, 72, [36, 36]),
    (33, 5, 5, 96, [2, 2, 92]),
    (19, 40, 2, 256, [64, 64, 64, 64]),
    (50, 7, 1, 128, [20, 20, 24]),          # half of the head
    (50, 3, 1, 128, [10, 14]),              # vectors of four with halves
    (21, 9, 2, 256, [6, 2]),
    (17, 2, 3, 8, [8]),
    (23, 6, 2, 72, [2, 4, 6, 8, 10, 12, 14, 16]),
    (1000, 1, 0, 64, [22, 42]),
]


@pytest.mark.parametrize("shared", [False, True])
@pytest.mark.parametrize("halves", [False, True])
@pytest.mark.parametrize("T,Hq,H,D,dims", ROPES)
def test_rope_axes(pv, T, Hq, H, D, dims, halves, shared):
    rng = np.random.default_rng(T + D)
    pos = rng.integers(-40, 5000, size=(len(dims), T))
    base = 1e4 if shared else 1e6
    q = _randn(T, Hq, D, seed=1, spread=0.5)
    k = _randn(T, H, D, seed=2, spread=0.5) if H else None
    # into other tensors
    qd, kd = q.cuda(), None if k is None else k.cuda()
    qo = torch.full((T + 2, Hq, D), 5.0, dtype=BF16, device="cuda")
    ko = None if k is None else torch.full((T + 2, H, D), 5.0, dtype=BF16, device="cuda")
    pv.rope_axes(qd, kd, _i32(pos.tolist()), dims, base, halves, shared, q_out=qo[:T],
                 k_out=None if k is None else ko[:T])
    assert pv.get_device_status() == 0
    for o, x, xd in ((qo, q, qd), (ko, k, kd)):
        if x is not None:
            _check_rope(o[:T], x, pos, dims, base, halves, shared)
            assert (o[T:].float() == 5.0).all() and torch.equal(_bits(xd.cpu()), _bits(x))
    # in place, the same bits
    pv.rope_axes(qd, kd, _i32(pos.tolist()), dims, base, halves, shared)
    assert torch.equal(_bits(qd), _bits(qo[:T]))
    assert k is None or torch.equal(_bits(kd), _bits(ko[:T]))


@pytest.mark.parametrize("halves", [False, True])
def test_rope_slices_and_rows_behind_the_batch(pv, halves):
    T, Hq, H, D, dims = 60, 4, 2, 128, [24, 40, 48]
    rng = np.random.default_rng(1)
    pos = rng.integers(0, 300, size=(3, T))
    fused = _randn(T, Hq + 2 * H, D, seed=5)
    fd = fused.cuda()
    pv.rope_axes(fd[:, :Hq], fd[:, Hq:Hq + H], _i32(pos.tolist()), dims, halves=halves,
                 num_tokens=_cu([30, 17])[-1:])
    got = fd.cpu()
    assert torch.equal(_bits(got[47:]), _bits(fused[47:]))
    assert torch.equal(_bits(got[:, Hq + H:]), _bits(fused[:, Hq + H:]))
    _check_rope(got[:47, :Hq + H], fused[:47, :Hq + H], pos[:, :47], dims, 1e4, halves, False)
    for n in (0, -5, 60, 1000):              # no rows, fewer than none, all, more than all
        a, b = fused.cuda(), fused.cuda()
        pv.rope_axes(a[:, :Hq], None, _i32(pos.tolist()), dims, halves=halves, num_tokens=_i32([n]))
        if n >= 60:
            pv.rope_axes(b[:, :Hq], None, _i32(pos.tolist()), dims, halves=halves)
        assert torch.equal(_bits(a), _bits(b))
    assert pv.get_device_status() == 0


@pytest.mark.parametrize("far", [1 << 20, (1 << 31) - 1])
def test_far_positions(pv, far):
    T, dims = 64, [64, 64]
    pos = np.random.default_rng(2).integers(far - 1000, far + 1, size=(2, T))
    pos[0] = -pos[0] - 1
    q = _randn(T, 3, 128, seed=1)
    for shared in (False, True):
        got, _ = pv.rope_axes(q.cuda(), None, _i32(pos.tolist()), dims, 5e5, True, shared)
        _check_rope(got, q, pos, dims, 5e5, True, shared)


def test_rope_bases(pv):
    q = _randn(40, 3, 64, seed=1)
    pos = np.arange(80).reshape(2, 40)
    for base in (0.5, 1.0, 7.0, 1e8):
        got, _ = pv.rope_axes(q.cuda(), None, _i32(pos.tolist()), [24, 40], base)
        _check_rope(got, q, pos, [24, 40], base, False, False)


def test_one_axis_is_the_rope_beside_it(pv):
    lengths, H, D = [30, 100], 4, 128
    q, k = (_randn(130, H, D, seed=s).cuda() for s in (1, 2))
    pos = np.concatenate([np.arange(30) + 7, np.arange(100)])
    a, b = pv.rope_axes(q.clone(), k.clone(), _i32([pos.tolist()]), [D])
    pv.rope_packed(q, k, _cu(lengths), _cu(lengths), _i32([7, 0]))
    for x, y in ((a, q), (b, k)):
        assert (x.float() - y.float()).abs().max() <= 2.0 ** -7 * y.float().abs().max()


def test_rope_of_many_heads(pv):
    q, k = _randn(3, 5000, 64, seed=1), _randn(3, 700, 64, seed=2)
    pos = np.array([[5, -(1 << 31), 9], [(1 << 31) - 1, 0, -1]])
    a, b = pv.rope_axes(q.cuda(), k.cuda(), _i32(pos.tolist()), [40, 24])
    _check_rope(a, q, pos, [40, 24], 1e4, False, False)
    _check_rope(b, k, pos, [40, 24], 1e4, False, False)


def test_rope_many_rows(pv):
    """More rows and heads than the grid takes at once; offsets beyond 32 bits."""
    T, Hq, D = (1 << 32) // (64 * 256) + 37, 64, 256
    q = torch.zeros(T, Hq, D, dtype=BF16, device="cuda")
    x = _randn(50, Hq, D, seed=1)
    q[-50:] = x.cuda()
    pos = torch.zeros(2, T, dtype=torch.int32, device="cuda")
    ends = np.random.default_rng(1).integers(0, 900, size=(2, 50))
    pos[:, -50:] = _i32(ends.tolist())
    pv.rope_axes(q, None, pos, [100, 156])
    _check_rope(q[-50:], x, ends, [100, 156], 1e4, False, False)
    assert (q[:50] == 0).all() and pv.get_device_status() == 0


def test_rope_binding_refusals(pv):
    q, k = _randn(20, 4, 64, seed=1).cuda(), _randn(20, 2, 64, seed=2).cuda()
    pos = torch.zeros(2, 20, dtype=torch.int32, device="cuda")

    def run(**kw):
        a = dict(q=q, k=k, positions=pos, axis_dims=[32, 32])
        a.update(kw)
        return pv.rope_axes(**a)

    before = q.clone()
    for kw in [dict(positions=pos[:1]), dict(positions=pos[:, :10]), dict(positions=pos.T),
               dict(positions=pos.long()), dict(positions=pos.cpu()), dict(k=k[:10]),
               dict(k=k[..., :32]), dict(q=q.float()), dict(q=q.cpu()), dict(q=q.transpose(0, 1)),
               dict(q_out=q[:10]), dict(k_out=q), dict(k=None, k_out=k), dict(q=None),
               dict(axis_dims=None), dict(num_tokens=pos[0]), dict(num_tokens=pos[0, :1].long()),
               dict(num_tokens=pos[0, :1].cpu()), dict(num_tokens=5)]:
        with pytest.raises((TypeError, ValueError)):
            run(**kw)
    for kw in [dict(axis_dims=[33, 31]), dict(axis_dims=[64, 64]), dict(axis_dims=[64, 0]),
               dict(axis_dims=[10, 20]), dict(base=0.0), dict(base=math.nan),
               dict(axis_dims=[1 << 40, 2])]:
        with pytest.raises(pv.PackedAttnError):
            run(**kw)
    with pytest.raises((pv.PackedAttnError, ValueError)):
        run(axis_dims=[])
    assert pv.get_device_status() == 0 and torch.equal(q, before)


# ------------------------------------------------------------------ linear layers

ACTS = ["none", "relu", "silu", "gelu", "gelu_tanh"]
# of any of the activations: |act'| <= 1.13 (gelu and its approximation reach 1.129)
SLOPE = 1.13


def _sums(size, K):
    """What fp32 accumulation of K bf16 products (exact each) loses: an addition that may
    truncate costs 2^-23 of the partial sum, at most K of them."""
    return (K + 1) * 2.0 ** -23 * size


def _act_tolerance(v, size, K, act):
    """Of act(v): the sums' error through the activation, and its own arithmetic in fp32
    (approximate exp2, reciprocal and error function: 2^-18 of the result holds all,
    as the exponents' own rounding, 2^-23 of an argument up to 100, is 2^-16
    only where the result is below 2^-100)."""
    y = np.abs(oracle.activation(v, act))
    return (SLOPE if act != "none" else 1.0) * _sums(size, K) + 2.0 ** -18 * y + 1e-30


def _round(want):
    return 2.0 ** -8 * np.abs(want) * (1 + 2.0 ** -7)


def _check_linear(got, x, w, bias, act, residual):
    K = x.shape[1]
    want, size = oracle.linear_act(x, w, bias, act, residual)
    v, _ = oracle.linear_act(x, w, bias)
    loss = _act_tolerance(v, size, K, act)
    if residual is not None:
        loss = loss + 2.0 ** -23 * (np.abs(want) + np.abs(oracle.to_f64(residual)))
    _within(got, want, loss + _round(np.abs(want) + loss))


def _check_gated(got, x, w, w2, act):
    K = x.shape[1]
    want, gate, gate_size, up, up_size = oracle.linear_gated(x, w, w2, act)
    a, u = np.abs(oracle.activation(gate, act)), np.abs(up)
    da, du = _act_tolerance(gate, gate_size, K, act), _sums(up_size, K)
    loss = a * du + u * da + da * du + 2.0 ** -23 * np.abs(want)
    _within(got, want, loss + _round(np.abs(want) + loss))


def _linear_inputs(M, N, K, seed, bias=True, residual=True):
    x, w = _randn(M, K, seed=seed, spread=0.3), _randn(N, K, seed=seed + 1)
    w = (w.float() / math.sqrt(K)).to(BF16)
    return (x, w, _randn(N, seed=seed + 2) if bias else None,
            _randn(M, N, seed=seed + 3) if residual else None)


def _cuda(*xs):
    return [None if x is None else x.cuda() for x in xs]


SHAPES = [(1, 8, 8), (1, 520, 200), (3, 264, 72), (8, 136, 1032), (13, 1032, 264), (16, 64, 4096),
          (17, 2048, 512), (33, 776, 328), (64, 256, 64), (65, 1288, 136), (100, 72, 2056),
          (128, 512, 128), (129, 264, 520), (200, 1032, 1024), (257, 520, 200), (300, 136, 64),
          (512, 768, 256), (700, 264, 1544)]


@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("act", ACTS)
def test_linear_act(pv, M, N, K, act):
    for bias, residual in ((False, False), (True, True)):
        x, w, b, r = _linear_inputs(M, N, K, M + N + K, bias, residual)
        got = pv.linear_act_bf16(*_cuda(x, w, b), act=act, residual=_cuda(r)[0])
        _check_linear(got, x, w, b, act, r)
    assert pv.get_device_status() == 0


@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("act", ["silu", "gelu", "none"])
def test_linear_gated(pv, M, N, K, act):
    x, w, _, _ = _linear_inputs(M, N, K, M + N + K, False, False)
    w2 = _linear_inputs(1, N, K, 7, False, False)[1]
    both = torch.cat([w, w2]).cuda()
    got = pv.linear_gated_bf16(x.cuda(), both[:N], both[N:], act=act)
    _check_gated(got, x, w, w2, act)
    assert pv.get_device_status() == 0


@pytest.mark.parametrize("act", ACTS)
def test_activations_over_their_range(pv, act):
    """Values from tiny to huge through a product with one: far tails, overflow of the
    exponentials, NaN and infinities."""
    v = torch.cat([torch.linspace(-40, 40, 161), torch.logspace(-30, 30, 61),
                   -torch.logspace(-30, 30, 61), torch.zeros(5)]).to(BF16)
    w = torch.zeros(8, 8, dtype=BF16)
    w[:, 0] = 1.0
    x = torch.zeros(len(v), 8, dtype=BF16)
    x[:, 0] = v
    for M in (len(v), 40):
        got = pv.linear_act_bf16(x[:M].contiguous().cuda(), w.cuda(), act=act)
        want = oracle.activation(oracle.to_f64(v[:M]), act)[:, None].repeat(8, 1)
        # the exponents' rounding: 2^-22 of the argument, relative to the result
        e = np.minimum(np.abs(oracle.to_f64(v[:M])), 100.0)[:, None] ** 2
        _within(got, want, _round(want) + (2.0 ** -18 + 2.0 ** -22 * e) * np.abs(want) + 1.2e-38)
    x[0, 0], x[1, 0], x[2, 0] = math.nan, math.inf, -math.inf
    got = pv.linear_act_bf16(x.cuda(), w[:, :8].cuda(), act=act).float().cpu()
    assert torch.isnan(got[0]).all() and torch.isfinite(got[3:]).all()


def test_linear_strides_and_in_place(pv):
    for M in (5, 40, 300):
        N, K = 264, 136
        x, w, b, r = _linear_inputs(M, N, K, 3)
        wide_x, wide_r, wide_y = (torch.full((M + 1, n + 16), 5.0, dtype=BF16, device="cuda")
                                  for n in (K, N, N))
        wide_x[:M, 8:8 + K], wide_r[:M, 8:8 + N] = x.cuda(), r.cuda()
        wd, bd = _cuda(w, b)
        want = pv.linear_act_bf16(x.cuda(), wd, bd, act="silu", residual=r.cuda())
        pv.linear_act_bf16(wide_x[:M, 8:8 + K], wd, bd, act="silu", residual=wide_r[:M, 8:8 + N],
                           out=wide_y[:M, 8:8 + N])
        assert torch.equal(_bits(wide_y[:M, 8:8 + N]), _bits(want))
        assert (wide_y[:M, :8] == 5).all() and (wide_y[:M, 8 + N:] == 5).all()
        assert (wide_y[M] == 5).all()
        pv.linear_act_bf16(wide_x[:M, 8:8 + K], wd, bd, act="silu", residual=wide_r[:M, 8:8 + N],
                           out=wide_r[:M, 8:8 + N])
        assert torch.equal(_bits(wide_r[:M, 8:8 + N]), _bits(want))
        assert (wide_r[:M, :8] == 5).all() and (wide_r[:M, 8 + N:] == 5).all()
        w2 = _linear_inputs(1, N, K, 9)[1].cuda()
        want = pv.linear_gated_bf16(x.cuda(), wd, w2)
        pv.linear_gated_bf16(wide_x[:M, 8:8 + K], wd, w2, out=wide_y[:M, 8:8 + N])
        assert torch.equal(_bits(wide_y[:M, 8:8 + N]), _bits(want))
        assert (wide_y[:M, :8] == 5).all() and (wide_y[:M, 8 + N:] == 5).all()
    assert pv.get_device_status() == 0


@pytest.mark.parametrize("N,K", [(776, 328), (2056, 1032), (136, 4096)])
def test_linear_rows_do_not_depend_on_the_batch(pv, N, K):
    """Rows packed, alone and at other offsets: the same bits, whatever M; and those of
    linear_bf16 where there is no epilogue."""
    M = 600
    x, w, b, r = _cuda(*_linear_inputs(M, N, K, 11))
    w2 = _linear_inputs(1, N, K, 12)[1].cuda()
    whole = pv.linear_act_bf16(x, w, b, act="gelu", residual=r)
    gated = pv.linear_gated_bf16(x, w, w2)
    assert torch.equal(_bits(pv.linear_act_bf16(x, w, b)), _bits(pv.linear_bf16(x, w, b)))
    for n in (1, 7, 16, 17, 30, 32, 33, 60, 64, 65, 100, 128, 129, 200, 256, 257, 400, 512, 599):
        for at in {0, M - n, (M - n) // 2}:
            rows = slice(at, at + n)
            part = pv.linear_act_bf16(x[rows], w, b, act="gelu", residual=r[rows])
            assert torch.equal(_bits(part), _bits(whole[rows])), (n, at)
            part = pv.linear_gated_bf16(x[rows], w, w2)
            assert torch.equal(_bits(part), _bits(gated[rows])), (n, at)
    assert pv.get_device_status() == 0


def test_linear_of_many_features(pv):
    M, N, K = 3, (1 << 20) + 8, 16
    x, w, b, r = _linear_inputs(M, N, K, 1)
    got = pv.linear_act_bf16(*_cuda(x, w, b), act="relu", residual=r.cuda())
    _check_linear(got, x, w, b, "relu", r)
    _check_gated(pv.linear_gated_bf16(x.cuda(), w.cuda(), w.flip(0).contiguous().cuda()), x, w,
                 w.flip(0), "silu")
    assert pv.get_device_status() == 0


def test_linear_of_no_rows(pv):
    x = torch.zeros(0, 64, dtype=BF16, device="cuda")
    w = torch.ones(16, 64, dtype=BF16, device="cuda")
    assert pv.linear_act_bf16(x, w).shape == (0, 16)
    assert pv.linear_gated_bf16(x, w, w).shape == (0, 16)


def test_linear_guard_band(pv):
    for M in (1, 9, 31, 70, 130, 333):
        N, K = 264, 136
        x, w, b, r = _cuda(*_linear_inputs(M, N, K, 5))
        buf = torch.full((M * N + 512,), 5.0, dtype=BF16, device="cuda")
        for _ in range(2):
            pv.linear_act_bf16(x, w, b, residual=r, act="relu",
                               out=buf[256:256 + M * N].view(M, N))
            assert (buf[:256] == 5).all() and (buf[256 + M * N:] == 5).all()
            pv.linear_gated_bf16(x, w, w, out=buf[256:256 + M * N].view(M, N))
            assert (buf[:256] == 5).all() and (buf[256 + M * N:] == 5).all()
    assert pv.get_device_status() == 0


def test_linear_bad_rows_stay_their_own(pv):
    """NaN and infinities in a row of x, of the residual or of the rows behind it reach no
    other row."""
    for M in (6, 50, 300):
        x, w, b, r = _linear_inputs(M, 264, 136, 6)
        wide = torch.full((M + 300, 136), math.nan, dtype=BF16)
        wide[:M] = x
        want = pv.linear_act_bf16(*_cuda(x, w, b), residual=r.cuda())
        xd, rd = wide.cuda()[:M], r.cuda()
        xd[2], rd[4] = math.inf, math.nan
        got = pv.linear_act_bf16(xd, w.cuda(), b.cuda(), residual=rd)
        keep = [m for m in range(M) if m not in (2, 4)]
        assert torch.equal(_bits(got[keep]), _bits(want[keep]))
        assert torch.isnan(got[4]).all() and not torch.isfinite(got[2]).any()


def test_linear_binding_refusals(pv):
    x, w, b, r = _cuda(*_linear_inputs(20, 64, 32, 1))

    def run(**kw):
        a = dict(x=x, w=w, bias=b, act="silu", residual=r)
        a.update(kw)
        return pv.linear_act_bf16(**a)

    for kw in [dict(w=w[:, :16]), dict(w=w.T), dict(bias=b[:8]), dict(residual=r[:4]),
               dict(residual=r.T.contiguous()), dict(x=x.float()), dict(x=x.cpu()), dict(x=x[0]),
               dict(w=w.cpu()), dict(bias=b.float()), dict(act="tanh"), dict(act=2), dict(act=None),
               dict(out=r[:4]), dict(out=r.float()), dict(x=x.T), dict(residual=r.cpu()),
               dict(out=r.cpu()), dict(x=None), dict(w=None)]:
        with pytest.raises((TypeError, ValueError)):
            run(**kw)
    for kw in [dict(w_up=w[:8]), dict(w_up=w[:, :16]), dict(w_gate=w.float()), dict(x=x[:, :16]),
               dict(act="swish"), dict(out=r[:4])]:
        with pytest.raises((TypeError, ValueError)):
            pv.linear_gated_bf16(**{**dict(x=x, w_gate=w, w_up=w), **kw})
    with pytest.raises(pv.PackedAttnError):        # rows that do not start on 16 bytes
        run(x=torch.zeros(20, 36, dtype=BF16, device="cuda")[:, :32])
    with pytest.raises(pv.PackedAttnError):
        run(x=x[:, :12].contiguous(), w=w[:, :12].contiguous())
    with pytest.raises(pv.PackedAttnError):        # one row that stands for all
        run(x=x[:1].expand(20, 32))
    assert pv.get_device_status() == 0


def test_linear_beyond_32_bit_offsets(pv):
    """More than 2^32 elements of y and of the residual."""
    N, K = 16384, 64
    M = (1 << 32) // N + 5
    x = torch.zeros(M, K, dtype=BF16, device="cuda")
    w = _randn(N, K, seed=1).cuda()
    r = torch.ones(M, N, dtype=BF16, device="cuda")
    ends = _randn(5, K, seed=2).cuda()
    x[-5:] = ends
    y = pv.linear_act_bf16(x, w, act="silu", residual=r)
    want = pv.linear_act_bf16(ends, w, act="silu", residual=r[-5:])
    assert torch.equal(_bits(y[-5:]), _bits(want)) and (y[:1000] == 1).all()
    assert pv.get_device_status() == 0


# ------------------------------------------------------------------ used together

@pytest.mark.parametrize("D", [64, 128])
def test_a_layer(pv, D):
    """One layer over packed prompts, every operator against the oracle on the rows it got;
    then captured, and replayed with other lengths and rows."""
    Hq, H, dims = 4, 2, [D // 4, D // 4, D // 2]
    C, F, T = Hq * D, 3 * Hq * D // 2, 400
    w_qkv, w_o, w_g, w_u, w_d = (
        (_randn(n, m, seed=20 + i).float() / math.sqrt(m)).to(BF16).cuda()
        for i, (n, m) in enumerate([((Hq + 2 * H) * D, C), (C, C), (F, C), (F, C), (C, F)]))
    bias = _randn(C, seed=30).cuda()
    x = torch.zeros(T, C, dtype=BF16, device="cuda")
    cu = _cu([0, 0, 0])
    pos = torch.zeros(3, T, dtype=torch.int32, device="cuda")

    def layer():
        s = {"x": x}
        s["qkv"] = pv.linear_bf16(x, w_qkv).view(T, Hq + 2 * H, D)
        s["q"], s["k"], s["v"] = s["qkv"].split([Hq, H, H], dim=1)
        s["raw"] = s["qkv"].clone()
        pv.rope_axes(s["q"], s["k"], pos, dims, num_tokens=cu[-1:])
        s["a"] = pv.prompt_attn_fwd(s["q"], s["k"], s["v"], cu, cu, T, T)
        s["h"] = pv.linear_act_bf16(s["a"].view(T, C), w_o, bias, residual=x)
        s["f"] = pv.linear_gated_bf16(s["h"], w_g, w_u)
        s["y"] = pv.linear_act_bf16(s["f"], w_d, residual=s["h"])
        return s

    def set_up(lengths, seed):
        cu.copy_(_cu(lengths))
        x.copy_(_randn(T, C, seed=seed).cuda())
        pos.copy_(_i32(np.random.default_rng(seed).integers(0, 60, size=(3, T)).tolist()))

    set_up([150, 1, 130], 1)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        held = layer()
    for seed, lengths in enumerate([[150, 1, 130], [0, 300, 100], [400, 0, 0]]):
        set_up(lengths, seed + 1)
        g.replay()
        torch.cuda.synchronize()
        assert pv.get_device_status() == 0
        n = sum(lengths)
        c = {name: t.cpu() for name, t in held.items()}
        _check_rope(c["q"][:n], c["raw"][:n, :Hq], pos[:, :n].cpu().numpy(), dims, 1e4, False, False)
        _check_rope(c["k"][:n], c["raw"][:n, Hq:Hq + H], pos[:, :n].cpu().numpy(), dims, 1e4, False,
                    False)
        assert torch.equal(_bits(c["qkv"][n:]), _bits(c["raw"][n:]))
        want, weight, reach = oracle.prompt_attention(c["q"], c["k"], c["v"], lengths, lengths, True,
                                                      D ** -0.5)
        _within(c["a"][:n], want[:n], _attention_tolerance(want, weight, reach, D)[:n])
        _check_linear(c["h"], c["a"].view(T, C), w_o.cpu(), bias.cpu(), "none", c["x"])
        _check_gated(c["f"], c["h"], w_g.cpu(), w_u.cpu(), "silu")
        _check_linear(c["y"], c["f"], w_d.cpu(), None, "none", c["h"])
        eager = layer()
        for name in ("q", "k", "a", "h", "f", "y"):
            rows = slice(0, n) if name == "a" else slice(None)
            assert torch.equal(_bits(eager[name][rows]), _bits(held[name][rows])), name


def test_layers_on_two_streams_and_in_two_graphs(pv):
    """Two programs at once over the same weights: eager calls on two streams, then two
    graphs replayed together, each with rows of its own."""
    Hq, H, D, C, T = 8, 2, 128, 1024, 700
    w_q, w_g, w_u, w_d = ((_randn(n, m, seed=40 + i).float() / math.sqrt(m)).to(BF16).cuda()
                          for i, (n, m) in enumerate([((Hq + 2 * H) * D, C), (2048, C), (2048, C),
                                                      (C, 2048)]))
    cu, pos = _cu([500, 13, 187]), torch.arange(2 * T, dtype=torch.int32, device="cuda").view(2, T)

    def layer(x, x1, stream=None):
        kw = dict(stream=stream)
        f = pv.linear_act_bf16(x, w_q, **kw).view(T, Hq + 2 * H, D)
        q, k, v = f.split([Hq, H, H], dim=1)
        pv.rope_axes(q, k, pos, [64, 64], **kw)
        a = pv.prompt_attn_fwd(q, k, v, cu, cu, 500, 500, **kw).view(T, C)
        y = pv.linear_act_bf16(pv.linear_gated_bf16(a, w_g, w_u, **kw), w_d, residual=x, **kw)
        y1 = pv.linear_act_bf16(pv.linear_gated_bf16(x1, w_g, w_u, **kw), w_d, residual=x1, **kw)
        return f, a, y, y1

    xs = [[_randn(n, C, seed=50 + i).cuda() for n in (T, 5)] for i in range(2)]
    want = [[t.clone() for t in layer(*x)] for x in xs]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = [None, None]
    for _ in range(6):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i] = layer(*xs[i])
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        assert all(torch.equal(_bits(x), _bits(y)) for x, y in zip(a, b))
    graphs = []
    for i, s in enumerate(streams):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            got[i] = layer(*xs[i])
        graphs.append(g)
    for t in [*got[0], *got[1]]:
        t.fill_(5.0)
    torch.cuda.synchronize()
    for _ in range(4):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        assert all(torch.equal(_bits(x), _bits(y)) for x, y in zip(a, b))
    assert pv.get_device_status() == 0
