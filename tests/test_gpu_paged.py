"""The paged K/V cache operators on the GPU against the fp64 oracle."""
import math

import numpy as np
import pytest
import torch

import oracle

pytestmark = pytest.mark.gpu

FORMATS = ["bf16", "e4m3"]


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


class Cache:
    """A pool of pages full of other sequences' old rows, and pages of it handed out at random."""

    def __init__(self, held, page, H, D, fmt, seed=0, width=None, spare=3, interleaved=False,
                 old=7.0):
        rng = np.random.default_rng(seed)
        counts = [-(-n // page) for n in held]
        P = sum(counts) + spare
        self.page, self.H, self.D, self.fmt, self.P = page, H, D, fmt, P
        perm = rng.permutation(P)
        self.table = np.full((len(held), width or max(counts + [1])), -1, dtype=np.int64)
        n = 0
        for b, c in enumerate(counts):
            self.table[b, :c] = perm[n:n + c]
            n += c
        dt = torch.bfloat16 if fmt == "bf16" else torch.float8_e4m3fn
        shape = (P, 2, page, H, D) if interleaved else (2, P, page, H, D)
        kv = torch.full(shape, old, device="cuda").to(dt)
        self.k, self.v = (kv[:, 0], kv[:, 1]) if interleaved else (kv[0], kv[1])
        self.ke = self.ve = None
        if fmt == "e4m3":
            byte = 127 if math.isfinite(old) else 255
            self.ke, self.ve = torch.full((2, P, H, page), byte, dtype=torch.uint8, device="cuda")
        self.dev_table = _i32(self.table.tolist())

    def exps(self):
        return dict(k_exp=self.ke, v_exp=self.ve)

    def values(self):
        """What the cache holds, in float64 [P, page, H, D]."""
        out = []
        for x, e in ((self.k, self.ke), (self.v, self.ve)):
            y = x.float().double().cpu().numpy()
            if e is not None:
                y = oracle.dequantise_rows(y, e.cpu().numpy().transpose(0, 2, 1))
            out.append(y)
        return out


def _rows(T, H, D, seed, spread=1.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(T, H, D, generator=g) * torch.exp(spread * torch.randn(T, H, 1, generator=g))
    return x.to(torch.bfloat16)


def _fill(pv, c, lengths, seed, offsets=None, spread=0.3):
    """Writes the first rows of every sequence through the library."""
    T = sum(lengths)
    k, v = _rows(T, c.H, c.D, seed, spread), _rows(T, c.H, c.D, seed + 1, spread)
    pv.kv_cache_write(k.cuda(), v.cuda(), c.k, c.v, _cu(lengths), c.dev_table,
                      pos_offset=None if offsets is None else _i32(offsets), **c.exps())
    return k, v


# ------------------------------------------------------------------ write and read

WRITES = [
    # lengths, offsets, page, H, D
    ([1], None, 16, 1, 64),
    ([1, 1, 1, 1, 1], [0, 15, 16, 31, 100], 16, 8, 128),
    ([37, 0, 64, 1], [5, 3, 0, 77], 16, 2, 64),
    ([300, 17, 129], [0, 250, 31], 32, 3, 128),
    ([1000, 3], [1, 0], 64, 5, 128),
    ([2, 513], [255, 256], 256, 20, 64),
    ([700], [12], 128, 12, 128),
    # one long sequence among many short ones, more sequences than a CTA has threads
    ([1] * 170 + [600] + [0, 1, 2] * 50, list(range(321)), 16, 2, 64),
    ([0] * 300 + [9], [3] * 301, 32, 1, 128),
]


def _write_case(pv, lengths, offsets, page, H, D, fmt, interleaved, strided):
    held = [n + (offsets[b] if offsets else 0) for b, n in enumerate(lengths)]
    c = Cache(held, page, H, D, fmt, seed=page + H, interleaved=interleaved,
              width=max(-(-n // page) for n in held) + 2)
    T, extra = sum(lengths), 3
    k, v = _rows(T + extra, H, D, 1), _rows(T + extra, H, D, 2)
    if strided:
        fused = torch.full((T + extra, 3 * H * D), 9.0, dtype=torch.bfloat16, device="cuda")
        fused[:, H * D:2 * H * D] = k.view(-1, H * D).cuda()
        fused[:, 2 * H * D:] = v.view(-1, H * D).cuda()
        dk, dv = fused[:, H * D:2 * H * D].view(-1, H, D), fused[:, 2 * H * D:].view(-1, H, D)
    else:
        dk, dv = k.cuda(), v.cuda()
    before = [x.view(torch.uint8).clone().cpu() for x in (c.k, c.v)]
    exps_before = [e.clone().cpu() for e in (c.ke, c.ve)] if fmt == "e4m3" else None
    off = None if offsets is None else _i32(offsets)
    got = pv.kv_cache_write(dk, dv, c.k, c.v, _cu(lengths), c.dev_table, pos_offset=off,
                            **c.exps())
    assert got[0] is c.k and got[1] is c.v
    assert pv.get_device_status() == 0
    at = oracle.places(lengths, offsets, c.table, page)
    for i, (x, cache, exp) in enumerate(((k, c.k, c.ke), (v, c.v, c.ve))):
        raw = cache.view(torch.uint8).cpu()
        want = before[i].clone()
        if fmt == "bf16":
            bits = x.view(torch.uint8)
        else:
            y, byte = oracle.quantise_rows(oracle.to_f64(x))
            bits = torch.tensor(y, dtype=torch.float32).to(torch.float8_e4m3fn).view(torch.uint8)
            want_exp = exps_before[i].clone()
        for t, (g, r) in enumerate(at):
            want[g, r] = bits[t].view(H, -1)
            if fmt == "e4m3":
                want_exp[g, :, r] = torch.tensor(byte[t])
        # -0 and 0 are one value: compare 8-bit payloads as values, everything else as bits
        if fmt == "bf16":
            assert torch.equal(raw, want)
        else:
            assert torch.equal(raw.view(torch.float8_e4m3fn).float(),
                               want.view(torch.float8_e4m3fn).float())
            assert torch.equal(exp.cpu(), want_exp)
    # and back
    out = [torch.full((T + extra, H, D), 3.0, dtype=torch.bfloat16, device="cuda")
           for _ in range(2)]
    pv.kv_cache_read(c.k, c.v, _cu(lengths), c.dev_table, T + extra, pos_offset=off,
                     k_out=out[0], v_out=out[1], **c.exps())
    assert pv.get_device_status() == 0
    for x, o in ((k, out[0]), (v, out[1])):
        assert (o[T:].float() == 3.0).all()
        if fmt == "bf16":
            assert torch.equal(o[:T].cpu().view(torch.int16), x[:T].view(torch.int16))
        else:
            y, byte = oracle.quantise_rows(oracle.to_f64(x[:T]))
            assert (oracle.to_f64(o[:T]) == oracle.dequantise_rows(y, byte)).all()


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("lengths,offsets,page,H,D", WRITES)
def test_write_and_read(pv, lengths, offsets, page, H, D, fmt):
    _write_case(pv, lengths, offsets, page, H, D, fmt, False, False)


@pytest.mark.parametrize("fmt", FORMATS)
def test_write_strided_rows_into_interleaved_pages(pv, fmt):
    _write_case(pv, [37, 0, 200, 1], [5, 3, 0, 77], 32, 3, 128, fmt, True, True)


def test_quantised_special_rows(pv):
    """Zeros, borders of the scale, ties, saturation, infinities, NaN, the smallest values."""
    D, rows = 64, []
    base = torch.zeros(D)
    for top in (0.0, 448.0, 450.0, 224.0, 225.0, 1.0, 0.875, 57344.0, 60000.0, 3.38e38, 1e-30,
                9.2e-41, 2.0 ** -92, 2.0 ** -100, math.inf):
        r = base.clone()
        r[3], r[60] = -top, top / 3 if math.isfinite(top) else 5.0
        r[5], r[6] = 1e-3, -17.0 if top > 20 else 0.0
        rows.append(r)
    ties = torch.arange(D).float() * 0.5 + 200.0     # steps of 16 above 128: ties at 8
    rows += [ties, -ties, torch.full((D,), math.nan), torch.full((D,), -0.0)]
    one_nan = torch.randn(D)
    one_nan[63] = math.nan
    rows.append(one_nan)
    x = torch.stack(rows).to(torch.bfloat16)[:, None]          # [T, 1, D]
    T = x.shape[0]
    c = Cache([T], 16, 1, D, "e4m3")
    pv.kv_cache_write(x.cuda(), x.flip(0).contiguous().cuda(), c.k, c.v, _cu([T]), c.dev_table,
                      **c.exps())
    k, v = pv.kv_cache_read(c.k, c.v, _cu([T]), c.dev_table, T, **c.exps())
    assert pv.get_device_status() == 0
    y, byte = oracle.quantise_rows(oracle.to_f64(x))
    want = oracle.dequantise_rows(y, byte)
    np.testing.assert_array_equal(oracle.to_f64(k), want)
    np.testing.assert_array_equal(oracle.to_f64(v), want[::-1])


@pytest.mark.parametrize("fmt", FORMATS)
def test_copy_refusals_on_the_device(pv, fmt):
    """Bad boundaries, offsets, lengths and pages: recorded, that sequence or page left alone."""
    H, D, page = 2, 64, 16
    c = Cache([40, 40], page, H, D, fmt)
    k = _rows(64, H, D, 5).cuda()
    before = c.k.view(torch.uint8).clone()
    for cu, off, code in [([0, 20, 10], [0, 0], 1), ([0, 30, 70], [0, 0], 1), ([3, 5, 6], [0, 0], 1),
                          ([0, 0, 5], [0, -1], 2), ([0, 0, 9], [0, 40], 2),
                          ([0, 0, 1], [0, 2147483647], 2)]:
        pv.kv_cache_write(k, k, c.k, c.v, _i32(cu), c.dev_table, pos_offset=_i32(off), **c.exps())
        assert pv.get_device_status() == code
        pv.kv_cache_read(c.k, c.v, _i32(cu), c.dev_table, 64, pos_offset=_i32(off), **c.exps())
        assert pv.get_device_status() == code
    for bad in (-1, c.P, 2147483647, -2147483648):
        c.k.view(torch.uint8).copy_(before)
        table = c.dev_table.clone()
        table[0, 1] = bad
        pv.kv_cache_write(k, k, c.k, c.v, _cu([40]), table[:1].contiguous(), **c.exps())
        assert pv.get_device_status() == 8
        out, _ = pv.kv_cache_read(c.k, c.v, _cu([40]), table[:1].contiguous(), 64, **c.exps())
        assert pv.get_device_status() == 8
        assert (out[16:32] == 0).all() and (out[40:] == 0).all()
        assert (out[:16] != 0).any() and (out[32:40] != 0).any()
        own = set(c.table[0].tolist()) - {int(c.table[0, 1])}
        for g in set(range(c.P)) - own:
            assert torch.equal(c.k.view(torch.uint8)[g], before[g])


# ------------------------------------------------------------------ attention

def _tolerance(want, weight, reach, D):
    """fp32 scores, sums and accumulation, weights and output rounded to bf16.
    The weights' rounding (2^-8 of each) moves a result by at most 2^-8 of
    sum w |v|, the output's by 2^-8 of itself.  A score's fp32 sum of D
    products (each exact) is off by at most D 2^-23 of sum |q k| (additions
    that may truncate), the exponent's arithmetic and exp2 by 2^-22 of the
    largest score and of the weight; twice that for numerator and sum."""
    scores = (D + 4) * 2.0 ** -23 * reach + 2.0 ** -20
    return (2.0 ** -8 + 2 * scores) * weight + 2.0 ** -8 * np.abs(want) * (1 + 2.0 ** -7) + 1e-30


def _check(got, c, q, lengths, seq_lens, causal, scale, heads=None):
    kc, vc = c.values()
    want, weight, reach = oracle.paged_attention(oracle.to_f64(q), kc, vc, lengths, seq_lens,
                                                 c.table, causal, scale, heads)
    T = sum(lengths)
    got = oracle.to_f64(got)[:T]
    if heads is not None:
        got, want, weight, reach = (x[:, heads] for x in (got, want, weight, reach))
    assert np.isfinite(got).all()
    excess = np.abs(got - want) - _tolerance(want, weight, reach, q.shape[2])
    assert excess.size == 0 or excess.max() <= 0, \
        f"{(excess > 0).sum()} of {excess.size} beyond, worst {excess.max():.3e} at " \
        f"{np.unravel_index(excess.argmax(), excess.shape)}"


def _attend(pv, c, q, lengths, seq_lens, causal, scale=None, extra=2, **kw):
    out = torch.full((sum(lengths) + extra, q.shape[1], q.shape[2]), 5.0, dtype=torch.bfloat16,
                     device="cuda")
    qd = torch.cat([q, q.new_zeros(extra, *q.shape[1:])]).cuda()
    pv.paged_attn_fwd(qd, c.k, c.v, _cu(lengths), _i32(seq_lens), c.dev_table,
                      max(lengths + [0]), max(seq_lens + [0]), causal=causal, scale=scale, out=out,
                      **c.exps(), **kw)
    assert pv.get_device_status() == 0
    assert (out[sum(lengths):].float() == 5.0).all()
    return out


def _attention_case(pv, lengths, seq_lens, Hq, H, D, page, fmt, causal, scale=None, old=7.0,
                    seed=0, spread=0.3, heads=None):
    c = Cache(seq_lens, page, H, D, fmt, seed=seed, old=old)
    _fill(pv, c, seq_lens, seed + 10, spread=spread)
    q = _rows(sum(lengths), Hq, D, seed + 20, 0.0)
    out = _attend(pv, c, q, lengths, seq_lens, causal, scale)
    _check(out, c, q, lengths, seq_lens, causal, 1 / math.sqrt(D) if scale is None else scale,
           heads)
    return out


DECODE = [
    # seq_lens of single-token steps, Hq, Hkv, D, page
    ([1], 1, 1, 64, 16),
    ([1, 15, 16, 17, 2], 8, 8, 128, 16),
    ([127, 128, 129, 1, 300], 8, 2, 128, 16),
    ([64, 65, 1000, 511, 512, 513], 12, 3, 64, 32),
    ([700, 33], 16, 2, 128, 64),
    ([257, 1, 90], 16, 1, 128, 256),
    ([255, 256, 31], 7, 1, 128, 128),
    ([2500, 5], 10, 2, 64, 16),
    ([40, 41], 40, 2, 128, 32),          # 20 query heads to a K/V head
    ([129, 600], 64, 1, 128, 64),
    ([77], 128, 1, 64, 16),
    ([4100, 2049, 1025], 4, 1, 128, 16),
]


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("seq_lens,Hq,H,D,page", DECODE)
def test_single_token_steps(pv, seq_lens, Hq, H, D, page, fmt):
    _attention_case(pv, [1] * len(seq_lens), seq_lens, Hq, H, D, page, fmt, True)


CHUNKS = [
    # lengths, seq_lens, Hq, Hkv, D, page
    ([2, 3, 4, 5, 8], [2, 40, 129, 1000, 9], 8, 2, 128, 16),
    ([16, 17, 33], [16, 300, 33], 4, 4, 64, 32),
    ([128, 129, 127], [128, 129, 500], 2, 2, 128, 16),
    ([255, 256, 257], [300, 256, 800], 1, 1, 64, 64),
    ([64, 65, 63], [64, 65, 200], 8, 2, 128, 128),
    ([37, 200], [37, 1111], 14, 2, 128, 32),       # 7 query heads to a K/V head
    ([50, 1], [513, 77], 15, 5, 64, 16),           # 3
    ([3, 9], [1300, 64], 128, 1, 128, 256),        # 128: one token fills a tile
    ([5, 2], [700, 5], 100, 1, 64, 16),
    ([700], [1500], 4, 1, 128, 64),
    ([1, 300, 1, 1, 0, 40], [900, 300, 1, 250, 30, 41], 8, 2, 128, 16),
    # either side of 32 rows of a K/V head, where another kernel takes over
    ([8, 9, 7, 8, 9], [8, 9, 500, 2000, 2100], 8, 2, 128, 16),
    ([32, 33, 31, 1], [1025, 1024, 1023, 513], 4, 4, 64, 64),
    # either side of one tile of rows, of two and of four
    ([32, 33, 64, 65, 128, 129], [600, 600, 600, 601, 129, 700], 4, 1, 128, 32),
]
# few heads and many keys: a sequence's key tiles are shared out over the SMs
SHARED = [
    ([20], [9000], 8, 2, 128, 16),                   # one tile of rows
    ([300, 40, 1], [7000, 4001, 6500], 4, 1, 128, 64),
    ([150, 33], [3000, 5555], 2, 2, 64, 32),
    ([90], [2500], 14, 2, 128, 128),                 # 7 query heads to a K/V head
    ([500], [450 + 4000], 3, 1, 64, 256),
    ([260, 9], [16, 3000], 16, 1, 128, 16),          # fewer keys than queries beside many
]


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("lengths,seq_lens,Hq,H,D,page", CHUNKS)
def test_chunks(pv, lengths, seq_lens, Hq, H, D, page, fmt, causal):
    _attention_case(pv, lengths, seq_lens, Hq, H, D, page, fmt, causal)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("lengths,seq_lens,Hq,H,D,page", SHARED)
def test_shared_out_keys(pv, lengths, seq_lens, Hq, H, D, page, fmt, causal):
    _attention_case(pv, lengths, seq_lens, Hq, H, D, page, fmt, causal, heads=[0, Hq // 2, Hq - 1])


def test_no_keys_in_the_call(pv):
    for fmt in FORMATS:
        for lq in (1, 100):
            out = _attention_case(pv, [lq, lq], [0, 0], 4, 2, 128, 16, fmt, True)
            assert (out[:2 * lq] == 0).all()


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("D", [64, 128])
def test_rows_that_see_nothing(pv, D, fmt):
    """No keys at all, fewer keys than queries in causal order, no queries: zeros, or nothing."""
    out = _attention_case(pv, [3, 1, 0, 40, 300], [0, 0, 20, 7, 130], 4, 2, D, 16, fmt, True)
    assert (out[:4] == 0).all() and (out[4:4 + 33] == 0).all() and (out[44:44 + 170] == 0).all()
    out = _attention_case(pv, [3, 1, 2], [0, 0, 20], 4, 2, D, 16, fmt, False)
    assert (out[:4] == 0).all()


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("lengths,seq_lens", [([1, 1, 1], [1, 30, 257]), ([40, 7], [70, 7]),
                                              ([300], [333])])
def test_rows_past_a_sequence_never_reach_it(pv, lengths, seq_lens, fmt):
    """NaN and infinities in every place of the pool that no sequence holds."""
    for old in (math.nan, math.inf, -math.inf):
        if fmt == "e4m3" and not math.isnan(old):
            continue
        _attention_case(pv, lengths, seq_lens, 8, 2, 128, 32, fmt, True, old=old)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("scale", [0.0, -0.2, 1.5, 1e-4])
def test_scales(pv, scale, fmt):
    _attention_case(pv, [1, 20, 1], [300, 130, 1], 8, 2, 128, 16, fmt, True, scale=scale)


@pytest.mark.parametrize("fmt", FORMATS)
def test_growing_scores(pv, fmt):
    """Keys that grow along the sequence, so that the running maximum moves at every tile."""
    D, H, n = 128, 1, 1500
    c = Cache([n, n], 16, H, D, fmt)
    k = _rows(2 * n, H, D, 3, 0.0).float()
    k *= torch.linspace(0.05, 6.0, n).repeat(2)[:, None, None]
    v = _rows(2 * n, H, D, 4, 0.0)
    pv.kv_cache_write(k.to(torch.bfloat16).cuda(), v.cuda(), c.k, c.v, _cu([n, n]), c.dev_table,
                      **c.exps())
    q = _rows(301, 4, D, 5, 0.0)
    out = _attend(pv, c, q, [300, 1], [n, n], True)
    _check(out, c, q, [300, 1], [n, n], True, 1 / math.sqrt(D))


def test_rows_of_very_unlike_scale(pv):
    """8-bit rows whose exponents lie far apart: a huge row among tiny ones, values and keys."""
    D, H, n = 128, 2, 400
    c = Cache([n, n], 16, H, D, "e4m3")
    k, v = _rows(2 * n, H, D, 3, 2.0), _rows(2 * n, H, D, 4, 4.0)
    v[5], v[n + 17] = v[5] * 2.0 ** 9, v[n + 17] * 2.0 ** -30
    pv.kv_cache_write(k.cuda(), v.cuda(), c.k, c.v, _cu([n, n]), c.dev_table, **c.exps())
    q = _rows(41, 4, D, 5, 0.0)
    out = _attend(pv, c, q, [1, 40], [n, n], True)
    _check(out, c, q, [1, 40], [n, n], True, 1 / math.sqrt(D))


def test_nan_in_a_visible_row_is_seen(pv):
    for fmt in FORMATS:
        c = Cache([100, 100], 16, 1, 64, fmt)
        k, v = _rows(200, 1, 64, 1), _rows(200, 1, 64, 2)
        k[20, 0, 7] = math.nan
        pv.kv_cache_write(k.cuda(), v.cuda(), c.k, c.v, _cu([100, 100]), c.dev_table, **c.exps())
        q = _rows(60, 2, 64, 3, 0.0)
        out = _attend(pv, c, q, [30, 30], [100, 100], True).float()
        assert torch.isnan(out[:30]).all() and torch.isfinite(out[30:60]).all()
        out = _attend(pv, c, q[:2], [1, 1], [100, 100], True).float()
        assert torch.isnan(out[0]).all() and torch.isfinite(out[1]).all()


@pytest.mark.parametrize("fmt", FORMATS)
def test_independent_of_the_batch(pv, fmt):
    """A sequence alone, in a batch, and in another order: the same bits; twice: the same bits."""
    lengths, seq_lens = [1, 200, 1, 3, 40, 1, 64], [3000, 900, 17, 1200, 40, 600, 5000]
    Hq, H, D, page = 8, 2, 128, 16
    c = Cache(seq_lens, page, H, D, fmt)
    _fill(pv, c, seq_lens, 1)
    q = _rows(sum(lengths), Hq, D, 2, 0.0).cuda()
    cu = np.concatenate([[0], np.cumsum(lengths)])
    ref = pv.paged_attn_fwd(q, c.k, c.v, _cu(lengths), _i32(seq_lens), c.dev_table, 200, 5000,
                            **c.exps())
    again = pv.paged_attn_fwd(q, c.k, c.v, _cu(lengths), _i32(seq_lens), c.dev_table, 200, 5000,
                              **c.exps())
    assert torch.equal(ref.view(torch.int16), again.view(torch.int16))
    for b, (n, m) in enumerate(zip(lengths, seq_lens)):
        one = pv.paged_attn_fwd(q[cu[b]:cu[b + 1]], c.k, c.v, _cu([n]), _i32([m]),
                                c.dev_table[b:b + 1].contiguous(), n, m, **c.exps())
        assert torch.equal(one.view(torch.int16), ref[cu[b]:cu[b + 1]].view(torch.int16)), b
    order = [4, 0, 6, 2, 5, 1, 3]
    qs = torch.cat([q[cu[b]:cu[b + 1]] for b in order])
    got = pv.paged_attn_fwd(qs, c.k, c.v, _cu([lengths[b] for b in order]),
                            _i32([seq_lens[b] for b in order]),
                            c.dev_table[order].contiguous(), 500, 9000, **c.exps())
    want = torch.cat([ref[cu[b]:cu[b + 1]] for b in order])
    assert torch.equal(got.view(torch.int16), want.view(torch.int16))
    assert pv.get_device_status() == 0


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("lq", [1, 2])
def test_same_bits_whatever_the_bounds(pv, lq, fmt):
    """The bounds max_q and max_k, and a large batch, choose among kernels; never a result."""
    Hq, H, D, page = 8, 2, 128, 16
    seq_lens = [1000, 64, 65, 1024, 1, 300, 129, 0]
    lengths = [lq] * len(seq_lens)
    c = Cache(seq_lens, page, H, D, fmt, width=20000 // page)
    _fill(pv, c, seq_lens, 1)
    q = _rows(sum(lengths), Hq, D, 2, 0.0).cuda()

    def attend(max_q, max_k, n=1):
        out = pv.paged_attn_fwd(q.repeat(n, 1, 1), c.k, c.v, _cu(lengths * n), _i32(seq_lens * n),
                                c.dev_table.repeat(n, 1), max_q, max_k, **c.exps())
        assert pv.get_device_status() == 0
        return out

    want = attend(lq, 1024)
    _check(want, c, q.cpu(), lengths, seq_lens, True, 1 / math.sqrt(D))
    for max_q, max_k in ((lq, 5000), (lq, 20000), (3, 1024), (4, 1030), (40, 20000)):
        assert torch.equal(attend(max_q, max_k).view(torch.int16), want.view(torch.int16))
    many = attend(lq, 1024, 40)
    assert torch.equal(many.view(torch.int16), want.repeat(40, 1, 1).view(torch.int16))


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("lengths,seq_lens", [([1], [1000]), ([1], [3000]), ([2, 0, 1], [900, 7, 513]),
                                              ([9], [2000]), ([20, 1], [1024, 700])])
def test_bounds_beyond_the_queries(pv, lengths, seq_lens, fmt):
    """max_q far above the queries that the call has: the same bits, and nothing written beyond
    the workspace that these arguments ask for."""
    Hq, H, D, page = 8, 2, 128, 16
    c = Cache(seq_lens, page, H, D, fmt, width=200)
    _fill(pv, c, seq_lens, 1)
    q = _rows(sum(lengths), Hq, D, 2, 0.0).cuda()
    dtype = torch.bfloat16 if fmt == "bf16" else torch.float8_e4m3fn
    top = max(seq_lens)
    want = pv.paged_attn_fwd(q, c.k, c.v, _cu(lengths), _i32(seq_lens), c.dev_table, max(lengths),
                             top, **c.exps())
    _check(want, c, q.cpu(), lengths, seq_lens, True, 1 / math.sqrt(D))
    for max_q in (4, 5, 8, 9, 100, 5000, 1 << 30):
        if max_q < max(lengths):
            continue
        for max_k in (top, 1024, 3000, 1 << 30):
            if max_k < top:
                continue
            need = pv.paged_attn_workspace_bytes(len(lengths), sum(lengths), max_q, max_k, Hq, H, D,
                                                 dtype)
            ws = torch.full((need + (8 << 20),), 171, dtype=torch.uint8, device="cuda")
            out = pv.paged_attn_fwd(q, c.k, c.v, _cu(lengths), _i32(seq_lens), c.dev_table, max_q,
                                    max_k, workspace=ws[:need], **c.exps())
            assert pv.get_device_status() == 0
            assert torch.equal(out.view(torch.int16), want.view(torch.int16))
            assert (ws[need:] == 171).all()


@pytest.mark.parametrize("D", [64, 128])
def test_rows_widened_ahead_or_in_place(pv, D):
    """Long sequences over an 8-bit cache: their rows as bf16 ahead of the products where
    that takes little memory, else inside the kernel.  The same bits."""
    Hq, H, page = 8, 2, 16
    lengths, seq_lens = [300, 200, 40, 1], [2500, 200, 3000, 77]
    c = Cache(seq_lens, page, H, D, "e4m3")
    _fill(pv, c, seq_lens, 1)
    q = _rows(sum(lengths), Hq, D, 2, 0.0).cuda()
    outs = [pv.paged_attn_fwd(q, c.k, c.v, _cu(lengths), _i32(seq_lens), c.dev_table, 300, max_k,
                              **c.exps()) for max_k in (3000, 1 << 20)]
    assert pv.get_device_status() == 0
    sizes = [pv.paged_attn_workspace_bytes(4, 541, 300, m, Hq, H, D, torch.float8_e4m3fn) -
             pv.paged_attn_workspace_bytes(4, 541, 300, m, Hq, H, D) for m in (3000, 1 << 20)]
    assert sizes[0] > 0 and sizes[1] == 0          # the second call widens nothing ahead
    assert torch.equal(outs[0].view(torch.int16), outs[1].view(torch.int16))
    _check(outs[0], c, q.cpu(), lengths, seq_lens, True, 1 / math.sqrt(D), heads=[0, 5])


@pytest.mark.parametrize("lq", [1, 33])
def test_smallest_values_of_8bit_rows(pv, lq):
    """Rows whose one large element the queries do not see (or that weighs nothing in the
    output dims looked at): what is left are e4m3's subnormals, which must not be lost."""
    D, H, n = 128, 1, 70
    c = Cache([n, n], 16, H, D, "e4m3")
    g = torch.Generator().manual_seed(5)
    k = (torch.randint(-7, 8, (2 * n, H, D), generator=g) * 2.0 ** -9)   # subnormals of a 448 row
    v = (torch.randint(-7, 8, (2 * n, H, D), generator=g) * 2.0 ** -9)
    k[..., 0] = 448.0
    v[..., 0] = 448.0
    q = _rows(lq + 1, 1, D, 3, 0.0)
    q[..., 0] = 0
    k, v = k.to(torch.bfloat16), v.to(torch.bfloat16)
    pv.kv_cache_write(k.cuda(), v.cuda(), c.k, c.v, _cu([n, n]), c.dev_table, **c.exps())
    kc, _ = c.values()
    assert (oracle.cached_rows(kc, c.table[0], n) == oracle.to_f64(k[:n])).all()
    out = _attend(pv, c, q, [lq, 1], [n, n], True, scale=3.0)
    _check(out, c, q, [lq, 1], [n, n], True, 3.0)


@pytest.mark.parametrize("fmt", FORMATS)
def test_strided_queries_and_interleaved_pages(pv, fmt):
    Hq, H, D, page = 6, 2, 128, 32
    lengths, seq_lens = [1, 70, 1, 9], [500, 70, 33, 1000]
    c = Cache(seq_lens, page, H, D, fmt, interleaved=True, width=40)
    _fill(pv, c, seq_lens, 3)
    T = sum(lengths)
    fused = torch.full((T, (Hq + 2 * H) * D), math.nan, dtype=torch.bfloat16, device="cuda")
    q = _rows(T, Hq, D, 9, 0.0)
    fused[:, :Hq * D] = q.view(T, -1).cuda()
    out = pv.paged_attn_fwd(fused[:, :Hq * D].view(T, Hq, D), c.k, c.v, _cu(lengths),
                            _i32(seq_lens), c.dev_table, 70, 1000, **c.exps())
    assert pv.get_device_status() == 0
    _check(out, c, q, lengths, seq_lens, True, 1 / math.sqrt(D))


def test_shared_pages(pv):
    """Two sequences that hold the same pages of a common prefix."""
    Hq, H, D, page = 8, 2, 64, 16
    c = Cache([100, 100], page, H, D, "bf16")
    c.table[1, :4] = c.table[0, :4]
    c.dev_table = _i32(c.table.tolist())
    _fill(pv, c, [64, 0], 1)
    _fill(pv, c, [36, 36], 2, offsets=[64, 64])
    q = _rows(20, Hq, D, 3, 0.0)
    out = _attend(pv, c, q, [1, 19], [100, 100], True)
    _check(out, c, q, [1, 19], [100, 100], True, 1 / math.sqrt(D))


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("lq", [1, 40])
def test_attention_refusals_on_the_device(pv, lq, fmt):
    """Bad lengths and boundaries: recorded, that sequence's rows untouched, the others computed."""
    Hq, H, D, page = 4, 2, 64, 16
    c = Cache([100, 100], page, H, D, fmt)
    _fill(pv, c, [100, 100], 1)
    q = _rows(2 * lq, Hq, D, 2, 0.0)
    want = _attend(pv, c, q, [lq, lq], [100, 100], True, extra=0)
    for cu, lens, mq, mk, code in [
            ([0, lq, 2 * lq], [100, -1], lq, 100, 4), ([0, lq, 2 * lq], [100, 113], lq, 200, 2),
            ([0, lq, 2 * lq], [100, 101], lq, 100, 2), ([0, lq, 2 * lq + 1], [100, 100], lq + 1, 100, 1),
            ([0, lq, lq - 1], [100, 100], lq, 100, 1)]:
        out = torch.full((2 * lq, Hq, D), 5.0, dtype=torch.bfloat16, device="cuda")
        pv.paged_attn_fwd(q.cuda(), c.k, c.v, _i32(cu), _i32(lens), c.dev_table, mq, mk, out=out,
                          **c.exps())
        assert pv.get_device_status() == code
        assert torch.equal(out[:lq], want[:lq]) and (out[lq:].float() == 5.0).all()
    for bad in (-1, c.P, 2147483647, -2147483648):
        table = c.dev_table.clone()
        table[1, 2] = bad
        out = pv.paged_attn_fwd(q.cuda(), c.k, c.v, _cu([lq, lq]), _i32([100, 100]), table, lq, 100,
                                **c.exps())
        assert pv.get_device_status() == 8
        assert torch.equal(out[:lq], want[:lq]) and torch.isfinite(out.float()).all()


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("lq", [1, 10, 30, 200])
def test_overlapping_boundaries_stay_in_the_workspace(pv, lq, fmt):
    """Boundaries that name every token many times over: an error, and nothing written beyond
    the workspace that the arguments ask for."""
    Hq, H, D, page, n = 8, 2, 128, 16, 300
    c = Cache([3000], page, H, D, fmt)
    _fill(pv, c, [3000], 1)
    q = _rows(lq, Hq, D, 2, 0.0).cuda()
    dtype = torch.bfloat16 if fmt == "bf16" else torch.float8_e4m3fn
    cu, lens = _i32([0, lq] * n + [0]), _i32([3000] * 2 * n)
    need = pv.paged_attn_workspace_bytes(2 * n, lq, lq, 3000, Hq, H, D, dtype)
    ws = torch.full((need + (64 << 20),), 171, dtype=torch.uint8, device="cuda")
    pv.paged_attn_fwd(q, c.k, c.v, cu, lens, c.dev_table.repeat(2 * n, 1), lq, 3000,
                      workspace=ws[:need], **c.exps())
    assert pv.get_device_status() == 1
    assert (ws[need:] == 171).all()
    _attention_case(pv, [lq], [3000], Hq, H, D, page, fmt, True)


def test_binding_refusals(pv):
    c = Cache([40], 16, 2, 64, "e4m3")
    x = _rows(4, 2, 64, 1).cuda()
    cu = _cu([4])
    lens = _i32([40])

    def attend(**kw):
        a = dict(q=x, k_cache=c.k, v_cache=c.v, cu_seqlens_q=cu, seq_lens=lens,
                 page_table=c.dev_table, max_q=4, max_k=40, k_exp=c.ke, v_exp=c.ve)
        a.update(kw)
        return pv.paged_attn_fwd(**a)

    for kw in [dict(k_exp=None), dict(k_exp=c.ke.transpose(1, 2)), dict(v_cache=c.v[1:]),
               dict(k_cache=c.k.transpose(1, 2)), dict(q=x[:, :1].expand(4, 3, 64)),
               dict(q=x.transpose(0, 1)), dict(q=x[..., :32]), dict(seq_lens=_i32([1, 2])),
               dict(page_table=c.dev_table[0]), dict(out=x[:2]), dict(out=torch.empty(4, 2, 64)),
               dict(seq_lens=lens.cpu()), dict(page_table=c.dev_table.repeat(2, 1)),
               dict(workspace=torch.empty(64, dtype=torch.uint8))]:
        with pytest.raises(ValueError):
            attend(**kw)
    for kw in [dict(q=x.float()), dict(k_cache=c.k.view(torch.uint8)), dict(seq_lens=lens.long()),
               dict(v_exp=c.ve.float()), dict(cu_seqlens_q=[0, 4]), dict(q=None), dict(out=7),
               dict(cu_seqlens_q=cu.repeat(2)[::2]), dict(v_cache=None), dict(page_table=None),
               dict(q=torch.zeros(4, 2, 64, 2, dtype=torch.bfloat16, device="cuda")[..., 0])]:
        with pytest.raises((TypeError, ValueError)):
            attend(**kw)
    for kw in [dict(scale=math.nan), dict(max_q=-1)]:
        with pytest.raises(pv.PackedAttnError):
            attend(**kw)
    with pytest.raises(ValueError):
        pv.kv_cache_write(x, x[:2], c.k, c.v, cu, c.dev_table, k_exp=c.ke, v_exp=c.ve)
    with pytest.raises(ValueError):
        pv.kv_cache_read(c.k, c.v, cu, c.dev_table, 4, k_exp=c.ke, v_exp=c.ve, k_out=x[:2])
    with pytest.raises(pv.PackedAttnError):       # a page size that is no power of two
        bad = torch.zeros(3, 24, 2, 64, dtype=torch.bfloat16, device="cuda")
        pv.kv_cache_write(x, x, bad, bad, cu, c.dev_table)
    assert pv.get_device_status() == 0


@pytest.mark.parametrize("fmt", FORMATS)
def test_rows_beyond_32_bit_offsets(pv, fmt):
    """A pool of more than 2^32 elements: rows in its last pages."""
    H, D, page = 16, 128, 256
    per_page = page * H * D
    P = (1 << 32) // per_page + 9
    dt = torch.bfloat16 if fmt == "bf16" else torch.float8_e4m3fn
    kc, vc = (torch.empty(P, page, H, D, dtype=dt, device="cuda") for _ in range(2))
    ex = {}
    if fmt == "e4m3":
        ex = dict(k_exp=torch.empty(P, H, page, dtype=torch.uint8, device="cuda"),
                  v_exp=torch.empty(P, H, page, dtype=torch.uint8, device="cuda"))
    table = _i32([[P - 1, 3], [P - 5, P - 2]])
    n = [300, 290]
    k, v = _rows(sum(n), H, D, 1, 0.3), _rows(sum(n), H, D, 2, 0.3)
    pv.kv_cache_write(k.cuda(), v.cuda(), kc, vc, _cu(n), table, **ex)
    rk, rv = pv.kv_cache_read(kc, vc, _cu(n), table, sum(n), **ex)
    if fmt == "bf16":
        assert torch.equal(rk.cpu(), k) and torch.equal(rv.cpu(), v)
    q = _rows(41, H, D, 3, 0.0)
    out = pv.paged_attn_fwd(q.cuda(), kc, vc, _cu([1, 40]), _i32(n), table, 40, 300, **ex)
    assert pv.get_device_status() == 0
    # the same rows in a small pool
    small = Cache(n, page, H, D, fmt)
    pv.kv_cache_write(k.cuda(), v.cuda(), small.k, small.v, _cu(n), small.dev_table,
                      **small.exps())
    want = pv.paged_attn_fwd(q.cuda(), small.k, small.v, _cu([1, 40]), _i32(n), small.dev_table,
                             40, 300, **small.exps())
    assert torch.equal(out, want)
    _check(want, small, q, [1, 40], n, True, 1 / math.sqrt(D), heads=[0, 15])


# ------------------------------------------------------------------ used together

@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("D", [64, 128])
def test_a_serving_run(pv, D, fmt):
    """Prompts taken in chunks beside sequences that answer token by token: rotary
    embedding, write and attention of every step; at the end the cache is read back."""
    Hq, H, page, B = 6, 2, 16, 4
    steps = [[30, 0, 17, 1], [25, 40, 1, 1], [1, 33, 1, 0], [1, 1, 1, 1], [1, 1, 0, 1]]
    total = np.sum(steps, axis=0)
    c = Cache(total.tolist(), page, H, D, fmt, width=12)
    done = np.zeros(B, dtype=np.int64)
    kept = [[] for _ in range(B)]
    for s, lengths in enumerate(steps):
        T = sum(lengths)
        q, k, v = (_rows(T, h, D, 100 * s + i, 0.0).cuda() for i, h in enumerate((Hq, H, H)))
        cu, off = _cu(lengths), _i32(done.tolist())
        pv.rope_packed(k, k.clone(), cu, cu, off)         # a call takes q and k of equal heads
        pv.rope_packed(q, q.clone(), cu, cu, off)
        pv.kv_cache_write(k, v, c.k, c.v, cu, c.dev_table, pos_offset=off, **c.exps())
        lens = (done + np.array(lengths)).tolist()
        out = pv.paged_attn_fwd(q, c.k, c.v, cu, _i32(lens), c.dev_table, max(lengths), max(lens),
                                **c.exps())
        assert pv.get_device_status() == 0
        _check(out, c, q.cpu(), lengths, lens, True, 1 / math.sqrt(D))
        t = 0
        for b, n in enumerate(lengths):
            kept[b].append(k[t:t + n].cpu())
            t += n
        done += np.array(lengths)
    rk, _ = pv.kv_cache_read(c.k, c.v, _cu(total.tolist()), c.dev_table, int(total.sum()),
                             **c.exps())
    want = oracle.to_f64(torch.cat([torch.cat(x) for x in kept]))
    if fmt == "e4m3":
        want = oracle.dequantise_rows(*oracle.quantise_rows(want))
    assert (oracle.to_f64(rk) == want).all()


def test_attention_over_cache_matches_packed_attention(pv):
    """Equal heads, no causal order: the packed kernel on the rows that the cache gives back."""
    H, D, page = 4, 128, 64
    lengths, seq_lens = [300, 5, 64], [300, 700, 129]
    for fmt in FORMATS:
        c = Cache(seq_lens, page, H, D, fmt)
        _fill(pv, c, seq_lens, 1)
        q = _rows(sum(lengths), H, D, 2, 0.0).cuda()
        a = pv.paged_attn_fwd(q, c.k, c.v, _cu(lengths), _i32(seq_lens), c.dev_table, 300, 700,
                              causal=False, **c.exps())
        k, v = pv.kv_cache_read(c.k, c.v, _cu(seq_lens), c.dev_table, sum(seq_lens), **c.exps())
        b = pv.varlen_attn_fwd(q, k, v, _cu(lengths), _cu(seq_lens), 300, 700)
        assert pv.get_device_status() == 0
        _check(a, c, q.cpu(), lengths, seq_lens, False, 1 / math.sqrt(D))
        _check(b, c, q.cpu(), lengths, seq_lens, False, 1 / math.sqrt(D))


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("n,max_k", [(1, 1024), (1, 4096), (5, 1024), (60, 4096), (150, 4096)])
def test_graph_replays_with_new_lengths(pv, n, max_k, fmt):
    """One captured step, replayed as the sequences grow; two graphs with their own workspaces."""
    Hq, H, D, page, B = 8, 2, 128, 16, 3
    lens0 = [850 if max_k == 1024 else 3000, 20, 270]
    c = Cache([x + 4 + n for x in lens0], page, H, D, fmt, width=256)
    _fill(pv, c, lens0, 1)
    lengths = [1, n, 1]
    T = sum(lengths)
    cu, lens, off = _cu(lengths), _i32(lens0), _i32(lens0)
    q = torch.zeros(T, Hq, D, dtype=torch.bfloat16, device="cuda")
    k, v = (torch.zeros(T, H, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    outs = [torch.zeros_like(q), torch.zeros_like(q)]
    side = torch.cuda.Stream()
    graphs = []
    torch.cuda.synchronize()
    for o in outs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            pv.kv_cache_write(k, v, c.k, c.v, cu, c.dev_table, pos_offset=off, **c.exps())
            pv.paged_attn_fwd(q, c.k, c.v, cu, lens, c.dev_table, n, max_k, out=o, **c.exps())
        graphs.append(g)
    for step in range(4):
        now = [x + step for x in lens0]
        after = [x + y for x, y in zip(now, lengths)]
        off.copy_(_i32(now))
        lens.copy_(_i32(after))
        for x, h, s in ((q, Hq, 0), (k, H, 1), (v, H, 2)):
            x.copy_(_rows(T, h, D, 50 * step + s, 0.0).cuda())
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        assert pv.get_device_status() == 0
        _check(outs[0], c, q.cpu(), lengths, after, True, 1 / math.sqrt(D))
        assert torch.equal(outs[0], outs[1])


@pytest.mark.parametrize("fmt", FORMATS)
def test_calls_on_several_streams_at_once(pv, fmt):
    """Calls that overlap, each with the workspace that the binding allocates on its stream."""
    Hq, H, D, page = 8, 2, 128, 16
    seq_lens = [3000, 1500, 40]
    c = Cache(seq_lens, page, H, D, fmt)
    _fill(pv, c, seq_lens, 1)
    lens = [[1, 1, 1], [1, 1, 1], [30, 20, 40], [700, 300, 1]]
    qs = [_rows(sum(n), Hq, D, 10 + i, 0.0).cuda() for i, n in enumerate(lens)]
    args = [(_cu(n), _i32(seq_lens)) for n in lens]
    want = [pv.paged_attn_fwd(q, c.k, c.v, *a, c.dev_table, max(n), 3000, **c.exps())
            for q, a, n in zip(qs, args, lens)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in qs]
    for _ in range(5):
        outs = [torch.zeros_like(q) for q in qs]
        torch.cuda.synchronize()
        for _ in range(4):
            for q, a, n, s, o in zip(qs, args, lens, streams, outs):
                pv.paged_attn_fwd(q, c.k, c.v, *a, c.dev_table, max(n), 3000, out=o, stream=s,
                                  **c.exps())
        torch.cuda.synchronize()
        for o, w in zip(outs, want):
            assert torch.equal(o, w)
    assert pv.get_device_status() == 0


def test_many_sequences(pv):
    """The largest batch, lengths from nothing to a few pages."""
    B, Hq, H, D, page = 1024, 4, 2, 64, 16
    rng = np.random.default_rng(0)
    seq_lens = rng.integers(0, 60, B).tolist()
    lengths = rng.integers(0, 3, B).tolist()
    _attention_case(pv, lengths, seq_lens, Hq, H, D, page, "bf16", True)
    lengths[500], seq_lens[500] = 50, 400
    _attention_case(pv, lengths, seq_lens, Hq, H, D, page, "e4m3", True)
    # and long ones far apart, whose 8-bit rows are widened ahead
    for b, n, keys in ((3, 300, 900), (290, 257, 257), (291, 260, 1500), (1000, 400, 401)):
        lengths[b], seq_lens[b] = n, keys
    _attention_case(pv, lengths, seq_lens, Hq, H, D, page, "e4m3", True, heads=[0, 3])


@pytest.mark.parametrize("fmt", FORMATS)
def test_most_heads(pv, fmt):
    """4096 K/V heads: one token fills a tile of the copies, and a head has one part of the keys."""
    H, D, page = 4096, 128, 16
    _write_case(pv, [1, 2], [0, 15], page, H, D, fmt, False, False)
    _attention_case(pv, [1, 40], [300, 45], H, H, D, page, fmt, True, heads=[0, 1, 2047, 4095])


@pytest.mark.parametrize("fmt", FORMATS)
def test_largest_batch_of_copies(pv, fmt):
    H, D, page, B = 1, 64, 16, 65535
    lengths = np.zeros(B, dtype=np.int64)
    where = [0, 1, 255, 256, 40000, 65534]
    lengths[where] = [3, 1, 20, 1, 2, 5]
    table = np.full((B, 2), -1)
    table[where] = np.arange(12).reshape(6, 2)
    c = Cache([12 * page], page, H, D, fmt)
    k, v = _rows(32, H, D, 1).cuda(), _rows(32, H, D, 2).cuda()
    cu, dev_table = _cu(lengths.tolist()), _i32(table.tolist())
    pv.kv_cache_write(k, v, c.k, c.v, cu, dev_table, **c.exps())
    got = pv.kv_cache_read(c.k, c.v, cu, dev_table, 32, **c.exps())
    assert pv.get_device_status() == 0
    for x, y in zip((k, v), got):
        # what a row holds after it: half a step of e4m3 off, or the same bits
        want, row_max = x.float(), x.float().abs().amax(-1, keepdim=True)
        bound = 0 if fmt == "bf16" else want.abs() / 16 + row_max * 2.0 ** -17
        assert ((y.float() - want).abs() <= bound).all()
    places = oracle.places(lengths[where].tolist(), None, table[where], page)
    kept = torch.ones(c.P, page, dtype=torch.bool)
    for g, r in places:
        kept[g, r] = False
    old = torch.tensor(7.0).to(c.k.dtype).float()
    assert (c.k.float().cpu()[kept] == old).all() and (c.v.float().cpu()[kept] == old).all()


def test_random_sweep(pv):
    rng = np.random.default_rng(77)
    for n in range(40):
        B, H, G = int(rng.integers(1, 7)), int(rng.integers(1, 4)), int(rng.integers(1, 12))
        D, page = int(rng.choice([64, 128])), int(rng.choice([16, 32, 64, 128, 256]))
        top = int(rng.choice([1, 4, 40, 300]))
        lengths = rng.integers(0, top + 1, B).tolist()
        seq_lens = [int(a + rng.integers(0, rng.choice([2, 200, 2500]))) for a in lengths]
        heads = sorted(set(rng.integers(0, H * G, 4).tolist()))
        _attention_case(pv, lengths, seq_lens, H * G, H, D, page, FORMATS[n % 2],
                        bool(rng.random() < 0.7), seed=n, heads=heads)


def test_random_bounds(pv):
    """Random calls whose bounds and buffers are larger than what they hold: the bits of the
    call with the least bounds, rows and workspace beyond theirs untouched."""
    rng = np.random.default_rng(123)
    for n in range(60):
        B, H, G = int(rng.integers(1, 40)), int(rng.choice([1, 2, 3, 8])), int(rng.integers(1, 41))
        D, page, fmt = int(rng.choice([64, 128])), int(rng.choice([16, 64, 256])), FORMATS[n % 2]
        causal = bool(rng.random() < 0.7)
        tops = rng.choice([0, 1, 3, 20, 200], B)
        lengths = [int(rng.integers(0, t + 1)) for t in tops]
        lengths[int(rng.integers(B))] += 1
        seq_lens = [int(a * causal + rng.integers(0, rng.choice([2, 600, 3000]))) for a in lengths]
        if sum(lengths) * H * G > 60000:
            continue
        c = Cache(seq_lens, page, H, D, fmt, seed=n, width=max(seq_lens) // page + 9)
        _fill(pv, c, seq_lens, n)
        T, extra = sum(lengths), int(rng.integers(0, 50))
        q = _rows(T + extra, H * G, D, n + 1, 0.0).cuda()
        cu, lens = _cu(lengths), _i32(seq_lens)
        want = pv.paged_attn_fwd(q[:T], c.k, c.v, cu, lens, c.dev_table, max(lengths),
                                 max(seq_lens), causal=causal, **c.exps())
        dtype = torch.bfloat16 if fmt == "bf16" else torch.float8_e4m3fn
        max_q = max(lengths) + int(rng.choice([0, 1, 7, 40, 3000]))
        max_k = max(seq_lens) + int(rng.choice([0, 1, 500, 1024, 50000]))
        need = pv.paged_attn_workspace_bytes(B, T + extra, max_q, max_k, H * G, H, D, dtype)
        ws = torch.full((need + (4 << 20),), 171, dtype=torch.uint8, device="cuda")
        out = torch.full_like(q, 5.0)
        pv.paged_attn_fwd(q, c.k, c.v, cu, lens, c.dev_table, max_q, max_k, causal=causal, out=out,
                          workspace=ws[:need], **c.exps())
        assert pv.get_device_status() == 0
        what = (n, B, H, G, D, page, lengths, seq_lens, max_q, max_k, extra)
        assert torch.equal(out[:T].view(torch.int16), want.view(torch.int16)), what
        assert (out[T:] == 5.0).all() and (ws[need:] == 171).all(), what


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("B", [31, 32, 33, 700])
def test_work_list_beside_the_first_tiles(pv, B, fmt):
    """The list of work is made where the first K tile lands: batches on both ways of making
    it, every CTA's first tiles right behind it, over and over with the same bits."""
    Hq, H, D, page = 4, 2, 128, 16
    lengths = [33 + b % 7 if b % (B // 30) == 0 else 0 for b in range(B)]
    seq_lens = [n + 3 * (b % 50) if n else 0 for b, n in enumerate(lengths)]
    c = Cache(seq_lens, page, H, D, fmt)
    _fill(pv, c, seq_lens, 1)
    q = _rows(sum(lengths), Hq, D, 2, 0.0).cuda()
    args = (q, c.k, c.v, _cu(lengths), _i32(seq_lens), c.dev_table, 40, max(seq_lens))
    want = pv.paged_attn_fwd(*args, **c.exps())
    _check(want, c, q.cpu(), lengths, seq_lens, True, 1 / math.sqrt(D), heads=[0, 3])
    for _ in range(20):
        assert torch.equal(pv.paged_attn_fwd(*args, **c.exps()).view(torch.int16),
                           want.view(torch.int16))
    assert pv.get_device_status() == 0


@pytest.mark.parametrize("gap", [20, 40, 60, 95])
@pytest.mark.parametrize("n", [40, 700, 3000])
@pytest.mark.parametrize("lq,Hq,D", [(2, 4, 128), (5, 4, 128), (8, 2, 64), (8, 8, 128)])
def test_hidden_rows_of_large_scale(pv, lq, Hq, D, n, gap):
    """8-bit values of later tokens far above those that a token sees: its result is held to the
    values that it sees, as in the other kernels."""
    H = 2
    c = Cache([n, n + 9], 16, H, D, "e4m3")
    k, v = _rows(2 * n + 9, H, D, 3, 0.3), _rows(2 * n + 9, H, D, 4, 0.3).float()
    up = torch.zeros(2 * n + 9)
    for i in range(lq):                    # every new token far above the one before it
        up[n - lq + i] = up[2 * n + 9 - lq + i] = gap * (i + 1) / lq
    v = (v * torch.exp2(up.round() + 4 - gap)[:, None, None]).to(torch.bfloat16)
    pv.kv_cache_write(k.cuda(), v.cuda(), c.k, c.v, _cu([n, n + 9]), c.dev_table, **c.exps())
    q = _rows(2 * lq, Hq, D, 5, 0.0)
    out = _attend(pv, c, q, [lq, lq], [n, n + 9], True)
    _check(out, c, q, [lq, lq], [n, n + 9], True, 1 / math.sqrt(D))


@pytest.mark.parametrize("below,gap", [(115, 60), (115, 95), (40, 40), (40, 36), (60, 20), (110, 107)])
@pytest.mark.parametrize("n", [50, 900, 5000])
@pytest.mark.parametrize("lq,D", [(1, 128), (1, 64), (4, 128)])
def test_weightless_rows_of_large_scale(pv, lq, D, n, below, gap):
    """Keys that weigh 2^-below and hold 8-bit values 2^gap above the others': neither is lost,
    whichever comes first and wherever the parts of the keys end."""
    H, Hq = 1, 2
    g = torch.Generator().manual_seed(9)
    u = (torch.randint(0, 2, (D,), generator=g) * 2 - 1).float()
    for places in ([0], [n // 2, n // 2 + 1], [n - lq - 1], list(range(0, n - lq, 7))):
        c = Cache([n], 16, H, D, "e4m3")
        k, v = _rows(n, H, D, 3, 0.0).float() * 0.25, _rows(n, H, D, 4, 0.3).float()
        k -= (k @ u)[..., None] * u / D
        v *= 2.0 ** (6 - gap)
        k[places], v[places] = -u, v[places] * 2.0 ** gap
        k, v = k.to(torch.bfloat16), v.to(torch.bfloat16)
        pv.kv_cache_write(k.cuda(), v.cuda(), c.k, c.v, _cu([n]), c.dev_table, **c.exps())
        q = u.expand(lq, Hq, D).to(torch.bfloat16).contiguous()
        scale = below * math.log(2) / D
        out = _attend(pv, c, q, [lq], [n], True, scale=scale)
        _check(out, c, q, [lq], [n], True, scale)


@pytest.mark.parametrize("lq,max_k", [(1, 700), (1, 5000), (5, 700), (40, 700), (300, 700),
                                      (300, 1 << 20)])
@pytest.mark.parametrize("D,sign", [(64, 0), (128, 128)])
def test_nan_among_8bit_values(pv, lq, max_k, D, sign):
    """An e4m3 NaN in a cache that something else filled: NaN in every kernel, whether rows are
    widened ahead or in place."""
    Hq, H, page, n = 6, 2, 16, 700
    c = Cache([n, n], page, H, D, "e4m3", width=max(44, n // page))
    _fill(pv, c, [n, n], 1)
    q = _rows(2 * lq, Hq, D, 2, 0.0)

    def attend():
        out = pv.paged_attn_fwd(q.cuda(), c.k, c.v, _cu([lq, lq]), _i32([n, n]), c.dev_table, lq,
                                max_k, causal=False, **c.exps())
        assert pv.get_device_status() == 0
        return out

    want = attend()
    _check(want, c, q, [lq, lq], [n, n], False, 1 / math.sqrt(D), heads=[0, 5])
    spots = [(3, 0, 0), (130, 1, D - 1), (511, 0, 37), (512, 0, 38), (699, 1, 5)]
    for pos, h, d in spots:                # of the first sequence's values
        c.v.view(torch.uint8)[c.table[0, pos // page], pos % page, h, d] = 127 | sign
    hit = torch.zeros(2 * lq, Hq, D, dtype=torch.bool, device="cuda")
    for _, h, d in spots:
        hit[:lq, 3 * h:3 * h + 3, d] = True
    out = attend()
    assert torch.isnan(out[hit]).all() and torch.equal(out[~hit], want[~hit])
    _, rv = pv.kv_cache_read(c.k, c.v, _cu([n, n]), c.dev_table, 2 * n, **c.exps())
    assert torch.isnan(rv).sum() == len(spots) and all(torch.isnan(rv[s]) for s in spots)
    c.k.view(torch.uint8)[c.table[1, 20], 3, 1, 9] = 127 | sign      # a key of the second's
    out = attend()
    assert torch.isnan(out[lq:, 3:]).all() and torch.equal(out[lq:, :3], want[lq:, :3])
    assert torch.equal(out[:lq][~hit[:lq]], want[:lq][~hit[:lq]])


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("Hq,H,D,B", [(64, 8, 128, 330), (32, 32, 64, 701)])
def test_batches_taken_in_turns(pv, Hq, H, D, B, fmt):
    """Bounds that would need more than 2 GB for the whole batch at once: the sequences go in
    turns, to the bits that one turn gives; bad ones in any turn are skipped alone."""
    page = 16
    rng = np.random.default_rng(B)
    lengths, seq_lens = np.ones(B, dtype=int), rng.integers(1, 80, B)
    for b, n, m in [(0, 1, 900), (3, 40, 2500), (100, 3, 2600), (101, 0, 50), (150, 130, 2100),
                    (180, 1, 2000), (181, 9, 9), (200, 300, 2300), (B - 2, 70, 2200), (B - 1, 2, 1500)]:
        lengths[b], seq_lens[b] = n, m
    lengths, seq_lens = lengths.tolist(), np.maximum(seq_lens, lengths).tolist()
    c = Cache(seq_lens, page, H, D, fmt)
    _fill(pv, c, seq_lens, 1)
    T = sum(lengths)
    q = _rows(T, Hq, D, 2, 0.0).cuda()
    cu, top = _cu(lengths), 1 << 20
    dtype = c.k.dtype
    need = pv.paged_attn_workspace_bytes(B, T + 1, 300, top, Hq, H, D, dtype)
    assert need <= 1 << 31
    ws = torch.full(((12 << 30),), 171, dtype=torch.uint8, device="cuda")

    def attend(cu, lens, size):
        out = torch.full((T + 1, Hq, D), 5.0, dtype=torch.bfloat16, device="cuda")
        qd = torch.cat([q, q[:1]])
        pv.paged_attn_fwd(qd, c.k, c.v, cu, lens, c.dev_table, 300, top, out=out,
                          workspace=ws[:size], **c.exps())
        return out

    got = attend(cu, _i32(seq_lens), need)
    assert pv.get_device_status() == 0
    assert (ws[need:need + (64 << 20)] == 171).all()
    one = attend(cu, _i32(seq_lens), ws.numel())
    assert pv.get_device_status() == 0
    assert (ws[need:] != 171).any()                       # all at once took more
    assert torch.equal(got.view(torch.int16), one.view(torch.int16))
    _check(got, c, q.cpu(), lengths, seq_lens, True, 1 / math.sqrt(D), heads=[0, Hq - 1])
    # a bad length in every part of the batch
    where = [1, 99, B // 2, B - 3]
    lens = list(seq_lens)
    for b in where:
        lens[b] = -1
    bad = attend(cu, _i32(lens), need)
    assert pv.get_device_status() == 4
    rows = torch.ones(T + 1, dtype=torch.bool, device="cuda")
    start = np.concatenate([[0], np.cumsum(lengths)])
    for b in where:
        rows[start[b]:start[b + 1]] = False
    assert torch.equal(bad[rows], got[rows]) and (bad[~rows] == 5.0).all()
    # boundaries that do not begin at 0: the first sequence's alone are bad
    late = cu.clone()
    late[0] = 1
    lens = list(seq_lens)
    out = attend(late, _i32(lens), need)
    assert pv.get_device_status() == 1
    assert torch.equal(out[lengths[0]:], got[lengths[0]:])


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("size", [10, 16, 20, 24, 28])
@pytest.mark.parametrize("lq,n,D", [(1, 700, 128), (1, 5000, 64), (4, 3000, 128), (40, 3000, 128),
                                    (150, 400, 64)])
def test_scores_of_any_size(pv, lq, n, D, size, fmt):
    """Keys of equal scores of some 2^size among keys far below them: the mean of their values,
    wherever they lie and however unlike their scale."""
    H, Hq = 1, 2
    g = torch.Generator().manual_seed(size)
    u = (torch.randint(0, 2, (D,), generator=g) * 2 - 1).float()
    c = Cache([n], 16, H, D, fmt)
    # u times signs that repeat in three keys of four sum to less than u u
    k = u * (1 - 2 * (torch.arange(D) % 4 == 3).float()) * 2.0 ** 6
    k = k.expand(n, H, D).clone()
    like = torch.arange(n) % 37 == 5
    like[[n // 2, n // 2 + 1]] = True
    like[n - lq:] = False
    k[like] = u * 2.0 ** 6
    v = _rows(n, H, D, 4, 0.3).float() * torch.exp2(-3.0 * (torch.arange(n) // 37 % 9))[:, None, None]
    k, v = k.to(torch.bfloat16), v.to(torch.bfloat16)
    pv.kv_cache_write(k.cuda(), v.cuda(), c.k, c.v, _cu([n]), c.dev_table, **c.exps())
    q = (u * 2.0 ** (size - 6)).expand(lq, Hq, D).to(torch.bfloat16).contiguous()
    scale = 1.37 / D                       # scores of 1.37 2^size and of half of that
    out = oracle.to_f64(_attend(pv, c, q, [lq], [n], False, scale=scale))[:lq]
    _, vc = c.values()
    rows = oracle.cached_rows(vc, c.table[0], n)[like.numpy()][:, 0]
    want, weight = rows.mean(axis=0), np.abs(rows).mean(axis=0)
    # equal weights, exact up to 2^-21 where they are rounded (f16, bf16: powers of two, or
    # half a step of bf16), fp32 sums, one rounding to bf16
    assert (np.abs(out - want) <= (2.0 ** -8 + 2.0 ** -14) * weight + 2.0 ** -8 * np.abs(want)).all()


def test_turns_with_rows_widened_ahead(pv):
    """Turns over an 8-bit cache whose long sequences' rows are widened ahead in each of them."""
    Hq, H, D, page, B, T = 64, 8, 128, 16, 60, 24000
    rng = np.random.default_rng(8)
    lengths = [int(x) for x in rng.choice([1, 2, 40, 70, 130, 300], B)]
    seq_lens = [n + int(rng.integers(0, 2300)) for n in lengths]
    c = Cache(seq_lens, page, H, D, "e4m3")
    _fill(pv, c, seq_lens, 1)
    n = sum(lengths)
    q = torch.zeros(T, Hq, D, dtype=torch.bfloat16, device="cuda")
    q[:n] = _rows(n, Hq, D, 2, 0.0).cuda()
    args = (q, c.k, c.v, _cu(lengths), _i32(seq_lens), c.dev_table, 300, 2700)
    need = pv.paged_attn_workspace_bytes(B, T, 300, 2700, Hq, H, D, torch.float8_e4m3fn)
    assert need == 1 << 31 and n < T
    ws = torch.full((need + (3 << 30),), 171, dtype=torch.uint8, device="cuda")
    got = pv.paged_attn_fwd(*args, workspace=ws[:need], **c.exps())
    assert (ws[need:] == 171).all()
    one = pv.paged_attn_fwd(*args, workspace=ws, **c.exps())
    assert pv.get_device_status() == 0
    assert torch.equal(got.view(torch.int16), one.view(torch.int16))
    _check(got[:n], c, q[:n].cpu(), lengths, seq_lens, True, 1 / math.sqrt(D), heads=[0, 63])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()                     # and captured
    out = torch.zeros_like(q)
    with torch.cuda.graph(graph):
        pv.paged_attn_fwd(*args, out=out, workspace=ws[:need], **c.exps())
    for _ in range(2):
        out.zero_()
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out.view(torch.int16), got.view(torch.int16))
    assert pv.get_device_status() == 0


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("lq,n", [(1, 1), (1, 300), (1, 3000), (5, 900), (40, 900), (300, 900)])
def test_nan_values_in_a_visible_row(pv, lq, n, fmt):
    """A V row that held a NaN: the queries that see it, and no other sequence's."""
    H, Hq, D = 2, 8, 128
    c = Cache([n + lq, n + lq], 16, H, D, fmt)
    k, v = _rows(2 * (n + lq), H, D, 1), _rows(2 * (n + lq), H, D, 2)
    v[n // 2, 1, 7] = math.nan
    pv.kv_cache_write(k.cuda(), v.cuda(), c.k, c.v, _cu([n + lq, n + lq]), c.dev_table, **c.exps())
    q = _rows(2 * lq, Hq, D, 3, 0.0)
    out = _attend(pv, c, q, [lq, lq], [n + lq, n + lq], True)[:2 * lq]
    dims = slice(None) if fmt == "e4m3" else 7          # an 8-bit row is NaN throughout
    assert torch.isnan(out[:lq, 4:, dims]).all()
    assert torch.isfinite(out[:lq, :4]).all() and torch.isfinite(out[lq:]).all()


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("lq,n,D,size", [(8, 3000, 128, 24), (16, 700, 128, 21), (13, 1500, 64, 28)])
def test_large_scores_of_more_rows(pv, lq, n, D, size, fmt):
    test_scores_of_any_size(pv, lq, n, D, size, fmt)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("n", [60, 1000, 4000])
@pytest.mark.parametrize("lq,Hq", [(4, 2), (7, 4), (16, 2)])
def test_large_scores_beside_ordinary_ones(pv, lq, Hq, n, fmt):
    """Rows of q whose scores are large among rows whose scores are not, over values of unlike
    scale: every row is held to its own bound."""
    H, D = 1, 128
    c = Cache([n], 16, H, D, fmt)
    k, v = _rows(n, H, D, 3, 0.3), _rows(n, H, D, 4, 2.0)
    pv.kv_cache_write(k.cuda(), v.cuda(), c.k, c.v, _cu([n]), c.dev_table, **c.exps())
    q = _rows(lq, Hq, D, 5, 0.0).float()
    q[1::3] *= 2.0 ** 22
    q = q.to(torch.bfloat16)
    out = _attend(pv, c, q, [lq], [n], True)
    _check(out, c, q, [lq], [n], True, 1 / math.sqrt(D))
