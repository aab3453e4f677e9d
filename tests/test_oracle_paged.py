"""The paged-cache oracle pinned against brute force, a library conversion and
the packed oracle; and the binding's refusals, which need no GPU."""
import ctypes
import math

import numpy as np
import pytest
import torch

import oracle


def test_e4m3_round_is_the_nearest_of_all_values():
    grid = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    grid = np.unique(grid[np.isfinite(grid)])
    rng = np.random.default_rng(0)
    y = np.concatenate([grid, (grid[1:] + grid[:-1]) / 2, rng.uniform(-500, 500, 4000),
                        rng.uniform(-0.02, 0.02, 4000)])
    got = oracle.e4m3_round(y)
    assert np.isin(got, grid).all()
    best = np.abs(np.clip(y, -448, 448)[:, None] - grid[None]).min(axis=1)
    assert (np.abs(np.clip(y, -448, 448) - got) == best).all()


def test_e4m3_round_matches_torch():
    x = torch.randn(20000) * torch.exp2(torch.randint(-8, 8, (20000,)).float())
    x = x.clamp(-448, 448)
    want = x.to(torch.float8_e4m3fn).double().numpy()
    assert (oracle.e4m3_round(x.double().numpy()) == want).all()


@pytest.mark.parametrize("top", [448.0, 448.0000001, 1.0, 0.875, 0.8750001, 3e-30, 1e-40, 57344.0,
                                 6e4, 3e38, 0.0, math.inf])
def test_quantise_scale(top):
    y, byte = oracle.quantise_rows(np.array([0.0, -top, top / 3 if math.isfinite(top) else 1.0]))
    e = int(byte) - oracle.paged.E_BIAS
    assert oracle.paged.E_MIN <= e <= oracle.paged.E_MAX
    if oracle.paged.E_MIN < e < oracle.paged.E_MAX:
        assert 224 * 2.0 ** e < top <= 448 * 2.0 ** e
    assert np.abs(y).max() <= 448
    back = oracle.dequantise_rows(y, byte)
    if 1e-28 < top <= 57344:
        assert abs(back[1] + top) <= top * 2.0 ** -4        # half a step of e4m3
        # a stored value is exact in bf16
        assert (torch.tensor(back).to(torch.bfloat16).double().numpy() == back).all()


def test_quantise_nan_row():
    y, byte = oracle.quantise_rows(np.array([[1.0, math.nan], [1.0, 2.0]]))
    assert byte[0] == 255 and byte[1] != 255
    assert np.isnan(oracle.dequantise_rows(y, byte)[0]).all()


@pytest.mark.parametrize("causal", [False, True])
def test_paged_attention_is_packed_attention_of_gathered_rows(causal):
    rng = np.random.default_rng(1)
    lq, lk, page, H, D = [3, 1, 5, 0, 4], [20, 33, 5, 7, 0], 16, 2, 8
    table = np.array([[4, 1, -1], [0, 7, 3], [6, -1, -1], [2, -1, -1], [-1, -1, -1]])
    kc, vc = rng.normal(size=(2, 8, page, H, D))
    q = rng.normal(size=(sum(lq), 2 * H, D))
    out, weight, reach = oracle.paged_attention(q, kc, vc, lq, lk, table, causal, 0.3)
    t = 0
    for b, n in enumerate(lq):
        for i in range(n):
            keys = range(lk[b] - n + i + 1) if causal else range(lk[b])
            for h in range(2 * H):
                num, den = np.zeros(D), 0.0
                for j in keys:
                    g, r = table[b][j // page], j % page
                    w = math.exp(0.3 * float(q[t, h] @ kc[g, r, h // 2]))
                    num, den = num + w * vc[g, r, h // 2], den + w
                want = num / den if den else num
                np.testing.assert_allclose(out[t, h], want, rtol=1e-10, atol=1e-12)
                assert (weight[t, h] >= np.abs(want) - 1e-12).all()
            t += 1


def test_places():
    assert oracle.places([2, 0, 3], [15, 0, 31], [[5, 6, 7], [0, 0, 0], [1, 2, 9]], 16) == \
        [(5, 15), (6, 0), (2, 15), (9, 0), (9, 1)]


# ---- refusals of the C entry points: one broken field each, nothing reaches the device
A, MIS = 0x10000, 0x10008


@pytest.fixture(scope="module")
def lib(lib_path):
    import packed_varlen_gb300 as pv
    return pv.load_library(lib_path)


COPY = dict(k=A, v=A, kc=A, vc=A, ke=A, ve=A, cu=A, off=A, table=A, batch=2, total=10, ks=1024,
            vs=1024, pages=9, page=16, width=4, stride=16 * 1024, H=8, D=128, fmt=1)
COPY_BAD = [(dict(k=None), 1), (dict(vc=None), 1), (dict(ke=None), 1), (dict(ve=None), 1),
            (dict(cu=None), 1), (dict(table=None), 1), (dict(batch=0), 1), (dict(total=-1), 1),
            (dict(pages=0), 1), (dict(width=0), 1), (dict(H=0), 1), (dict(D=0), 1),
            (dict(fmt=2), 1), (dict(fmt=-1), 1), (dict(stride=1024), 1), (dict(page=0), 1),
            (dict(page=8), 2), (dict(page=48), 2), (dict(page=512, stride=1 << 22), 2),
            (dict(D=96), 2), (dict(D=256), 2), (dict(H=5000, stride=1 << 30), 2),
            (dict(stride=1 << 39), 2), (dict(batch=65536), 2), (dict(kc=MIS), 3),
            (dict(k=MIS), 3), (dict(ke=MIS), 3), (dict(cu=A + 2), 3), (dict(off=A + 1), 3),
            (dict(table=A + 2), 3), (dict(stride=16 * 1024 + 8), 3)]


@pytest.mark.parametrize("kw,code", COPY_BAD + [(dict(ks=1023), 1), (dict(vs=8), 1),
                                                (dict(ks=1028), 3), (dict(vs=1030), 3)])
def test_write_host_checks(lib, kw, code):
    a = dict(COPY, **kw)
    assert lib.pa_kv_cache_write(*[a[n] for n in COPY], None) == code


@pytest.mark.parametrize("kw,code", COPY_BAD)
def test_read_host_checks(lib, kw, code):
    a = dict(COPY, **kw)
    order = ["kc", "vc", "ke", "ve", "k", "v"] + [n for n in list(COPY)[6:] if n not in ("ks", "vs")]
    assert lib.pa_kv_cache_read(*[a[n] for n in order], None) == code


ATTN = dict(q=A, kc=A, vc=A, ke=A, ve=A, out=A, cu=A, lens=A, table=A, batch=2, total=10, max_q=8,
            max_k=64, qs=32 * 128, pages=9, page=16, width=4, stride=16 * 1024, Hq=32, H=8, D=128,
            fmt=1, causal=1, scale=0.1, ws=A, wn=1 << 40)


@pytest.mark.parametrize("kw,code", [
    (dict(q=None), 1), (dict(out=None), 1), (dict(kc=None), 1), (dict(ve=None), 1),
    (dict(lens=None), 1), (dict(table=None), 1), (dict(batch=0), 1), (dict(total=-1), 1),
    (dict(max_q=-1), 1), (dict(max_k=-1), 1), (dict(Hq=0), 1), (dict(Hq=30), 1),
    (dict(qs=4095), 1), (dict(scale=math.inf), 1), (dict(scale=math.nan), 1), (dict(fmt=7), 1),
    (dict(D=96), 2), (dict(page=24), 2), (dict(batch=1025), 2), (dict(H=1, Hq=129, qs=1 << 20), 2),
    (dict(total=(1 << 30) + 1), 2), (dict(max_q=(1 << 30) + 1), 2), (dict(max_k=(1 << 31) - 1), 2),
    (dict(q=MIS), 3), (dict(out=MIS), 3), (dict(vc=MIS), 3), (dict(cu=A + 2), 3),
    (dict(lens=A + 2), 3), (dict(qs=32 * 128 + 4), 3), (dict(ws=MIS), 3)])
def test_attention_host_checks(lib, kw, code):
    a = dict(ATTN, **kw)
    assert lib.pa_paged_attn_fwd(*[a[n] for n in ATTN], None) == code


def test_empty_calls_touch_nothing(lib):
    for kw in (dict(total=0), dict(total=0, q=None, out=None), dict(max_q=0)):
        a = dict(ATTN, **kw)
        assert lib.pa_paged_attn_fwd(*[a[n] for n in ATTN], None) == 0
    a = dict(COPY, total=0)
    assert lib.pa_kv_cache_write(*[a[n] for n in COPY], None) == 0


@pytest.mark.parametrize("fmt", [0, 1])
def test_workspace_bytes(lib, fmt):
    f = lib.pa_paged_attn_workspace_bytes
    assert f(0, 1, 1, 1, 8, 8, 128, fmt) == -1 and f(1, 1, 1, 1, 9, 8, 128, fmt) == -1
    assert f(1, -1, 1, 1, 8, 8, 128, fmt) == -1 and f(1, 1, 1, 1, 8, 8, 96, fmt) == -1
    assert f(2000, 1, 1, 1, 8, 8, 128, fmt) == -1 and f(1, 1, 1, 1, 8, 8, 128, 5) == -1
    assert f(1, 1, 1, 1, 129, 1, 128, fmt) == -1 and f(1, 1, 1, 1, 5000, 5000, 128, fmt) == -1
    assert f(1, 1, 1, (1 << 30) + 1, 8, 8, 128, fmt) == -1
    for batch, total, max_q, max_k in [(4, 100, 30, 5000), (4, 3000, 1000, 20000), (1, 7, 7, 90000),
                                       (1024, 100000, 9000, 1 << 20), (1, 1, 1, 1 << 30),
                                       (3, 1 << 20, 1 << 20, 1 << 20)]:
        n = f(batch, total, max_q, max_k, 32, 8, 128, fmt)
        assert 0 < n < 1 << 40
        # a call that is given less is refused
        a = dict(ATTN, batch=batch, total=total, max_q=max_q, max_k=max_k, fmt=fmt, wn=n - 1)
        assert lib.pa_paged_attn_fwd(*[a[k] for k in ATTN], None) == 1
        a = dict(a, ws=None, wn=n)
        assert lib.pa_paged_attn_fwd(*[a[k] for k in ATTN], None) == 1


def test_binding_refuses_host_tensors(lib):
    import packed_varlen_gb300 as pv
    c = torch.zeros(4, 16, 2, 64, dtype=torch.bfloat16)
    cu = torch.tensor([0, 1], dtype=torch.int32)
    t = torch.zeros(1, 4, dtype=torch.int32)
    x = torch.zeros(1, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        pv.kv_cache_write(x, x, c, c, cu, t)
    with pytest.raises(ValueError):
        pv.kv_cache_read(c, c, cu, t, 1)
    with pytest.raises(ValueError):
        pv.paged_attn_fwd(x, c, c, cu, cu[1:], t, 1, 1)
    with pytest.raises(TypeError):
        pv.kv_cache_write(x, x, None, c, cu, t)
    with pytest.raises(pv.PackedAttnError):
        pv.paged_attn_workspace_bytes(0, 1, 1, 1, 8, 8, 128)


@pytest.mark.parametrize("n", [1 << 31, 1 << 32, (1 << 32) + 4, (1 << 40) + 64, -1, -(1 << 32) + 4])
def test_binding_refuses_counts_that_32_bits_cut(lib, n):
    import packed_varlen_gb300 as pv
    c = torch.zeros(4, 16, 2, 64, dtype=torch.bfloat16)
    cu = torch.tensor([0, 1], dtype=torch.int32)
    t = torch.zeros(1, 4, dtype=torch.int32)
    x = torch.zeros(1, 2, 64, dtype=torch.bfloat16)
    for max_q, max_k in ((n, 4), (1, n), (n, n)):
        with pytest.raises(pv.PackedAttnError):
            pv.paged_attn_fwd(x, c, c, cu, cu[1:], t, max_q, max_k)
    with pytest.raises(pv.PackedAttnError):
        pv.kv_cache_read(c, c, cu, t, n)
    for at in range(7):
        sizes = [2, 10, 8, 64, 32, 8, 128]
        sizes[at] = n
        with pytest.raises(pv.PackedAttnError):
            pv.paged_attn_workspace_bytes(*sizes)


def _rows_of_parts(lq, lk, causal, G, Hkv):
    """(shares, items of all heads, rows of a part) of a sequence whose keys are split, else None:
    items of 2 * (128 / G) queries, a lone sequence's shares of at least ten tiles of 128 keys."""
    tokens = 2 * (128 // G)
    items = -(-lq // tokens)
    keys = [max(min(lk, lk - lq + (i + 1) * tokens) if causal else lk, 128) for i in range(items)]
    if items * Hkv >= 6 * 152 or keys[-1] <= 15 * 128:
        return None
    share = max(-(-sum(keys) * Hkv // 152), 1280)
    return -(-sum(keys) * Hkv // share), items * Hkv, min(lq, tokens) * G


def test_workspace_holds_the_parts_of_any_batch(lib):
    """Random batches: the rows that the kernels leave fit what the bounds ask for."""
    rng = np.random.default_rng(3)
    tight = 0.0
    for _ in range(3000):
        B, G = int(rng.integers(1, 12)), int(rng.choice([1, 2, 4, 7, 8, 40, 128]))
        H, D = int(rng.choice([1, 2, 8, 20])), int(rng.choice([64, 128]))
        top = int(rng.choice([3, 40, 200, 900]))
        lq = rng.integers(0, top + 1, B)
        lk = lq + rng.integers(0, int(rng.choice([100, 3000, 40000])), B)
        causal = bool(rng.integers(2))
        few, rows = 32 // G, 0
        for n, m in zip(lq.tolist(), lk.tolist()):
            split = _rows_of_parts(n, m, causal, G, H) if n > few else None
            if split:
                shares, items, part = split
                rows += (shares + min(shares, items)) * part
        bytes_ = lib.pa_paged_attn_workspace_bytes(B, int(lq.sum()), int(lq.max()), int(lk.max()),
                                                   G * H, H, D, 0)
        assert rows * (D * 4 + 8) <= bytes_
        tight = max(tight, rows * (D * 4 + 8) / max(bytes_, 1))
    assert tight > 0.8                     # some batch needs nearly all of it


@pytest.mark.parametrize("fmt", [0, 1])
def test_workspace_is_bounded(lib, fmt):
    """A call asks for no more than 2 GB whatever its bounds, and for little where little can
    be split: two chunks beside single tokens, single tokens over long caches."""
    f = lib.pa_paged_attn_workspace_bytes
    rng = np.random.default_rng(4)
    for _ in range(2000):
        G, B = int(rng.choice([1, 4, 8, 128])), int(2 ** rng.uniform(0, 10))
        H = int(2 ** rng.uniform(0, 12 if G < 128 else 5))
        total, max_q, max_k = (int(2 ** rng.uniform(0, 30)) for _ in range(3))
        assert 0 <= f(B, total, max_q, max_k, G * H, H, 128, fmt) <= 1 << 31
    for args, most in [((128, 8192, 2048, 32768, 32, 8), 2048), ((256, 8192, 2048, 131072, 32, 8), 2048),
                       ((256, 8447, 8192, 131072, 64, 8), 2048), ((24, 860, 500, 4000, 32, 8), 380),
                       ((64, 64, 1, 131072, 32, 8), 250), ((1, 2048, 2048, 16048, 32, 8), 140),
                       ((1, 1, 1, 131072, 32, 8), 5)]:
        assert f(*args, 128, fmt) <= most << 20


def test_workspace_of_smaller_bounds(lib):
    """One workspace, made for the largest bounds, serves every call over a bf16 cache."""
    f = lib.pa_paged_attn_workspace_bytes
    rng = np.random.default_rng(5)
    for _ in range(5000):
        G, H = int(rng.choice([1, 4, 7, 8, 128])), int(rng.choice([1, 2, 8, 20]))
        big = [int(2 ** rng.uniform(0, x)) for x in (10, 17, 13, 20)]
        small = [int(rng.integers(1, x + 1)) if rng.integers(2) else x for x in big]
        assert f(*small, G * H, H, 128, 0) <= f(*big, G * H, H, 128, 0)


@pytest.mark.parametrize("scale", [2.4e38, -2.4e38, 3.4e38])
def test_scale_that_overflows_is_refused(lib, scale):
    """A finite scale whose product with log2(e), which the kernels use, is not."""
    a = dict(ATTN, scale=scale)
    assert lib.pa_paged_attn_fwd(*[a[n] for n in ATTN], None) == 1
