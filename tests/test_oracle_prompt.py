"""The oracle of the operators of a layer over packed prompts, pinned against
brute force and library routines; and the refusals that need no GPU."""
import ctypes
import math

import numpy as np
import pytest
import torch

import oracle


@pytest.mark.parametrize("causal", [False, True])
def test_prompt_attention_against_brute_force(causal):
    rng = np.random.default_rng(0)
    lq, lk, Hq, H, D = [3, 1, 0, 5, 4], [3, 6, 2, 2, 0], 4, 2, 8
    q = rng.normal(size=(sum(lq), Hq, D))
    k, v = rng.normal(size=(2, sum(lk), H, D))
    out, weight, reach = oracle.prompt_attention(q, k, v, lq, lk, causal, 0.4)
    t = k0 = 0
    for n, m in zip(lq, lk):
        for i in range(n):
            keys = [j for j in range(m) if not causal or j <= m - n + i]
            for h in range(Hq):
                num, den = np.zeros(D), 0.0
                for j in keys:
                    w = math.exp(0.4 * float(q[t, h] @ k[k0 + j, h // 2]))
                    num, den = num + w * v[k0 + j, h // 2], den + w
                want = num / den if den else num
                np.testing.assert_allclose(out[t, h], want, rtol=1e-10, atol=1e-12)
                assert (weight[t, h] >= np.abs(want) - 1e-12).all()
                most = max([0.4 * float(np.abs(q[t, h]) @ np.abs(k[k0 + j, h // 2]))
                            for j in keys], default=0.0)
                assert reach[t, h, 0] == pytest.approx(most)
            t += 1
        k0 += m


def test_prompt_attention_against_packed_attention_and_a_library():
    rng = np.random.default_rng(1)
    L, H, D = [5, 9], 2, 16
    q, k, v = rng.normal(size=(3, sum(L), H, D))
    cu = oracle.cu_seqlens_from_lengths(L)
    out, _, _ = oracle.prompt_attention(q, k, v, L, L, False, 0.25)
    np.testing.assert_allclose(out, oracle.varlen_attention(q, k, v, cu, cu, 0.25), atol=1e-12)
    out, _, _ = oracle.prompt_attention(q, k, v, L, L, True, 0.25)
    for a, b in zip(cu[:-1], cu[1:]):
        x = [torch.tensor(t[a:b]).transpose(0, 1) for t in (q, k, v)]
        want = torch.nn.functional.scaled_dot_product_attention(*x, is_causal=True, scale=0.25)
        np.testing.assert_allclose(out[a:b], want.transpose(0, 1).numpy(), atol=1e-12)
    rows, _, _ = oracle.prompt_attention(q, k, v, L, L, True, 0.25, rows=[13, 2, 7])
    np.testing.assert_allclose(rows, out[[13, 2, 7]], atol=1e-12)


def test_rope_axes_of_one_axis_is_rope():
    x = np.random.default_rng(2).normal(size=(6, 3, 16))
    pos = np.array([[0, 3, 1, 9, 200, 4]])
    for shared in (False, True):
        np.testing.assert_allclose(oracle.rope_axes(x, pos, [16], 100.0, shared=shared),
                                   oracle.rope(x, pos[0], 100.0), atol=1e-12)


@pytest.mark.parametrize("halves", [False, True])
@pytest.mark.parametrize("shared", [False, True])
def test_rope_axes_turns_complex_numbers(halves, shared):
    rng = np.random.default_rng(3)
    dims, base, D = [4, 6, 2], 50.0, 20
    x, pos = rng.normal(size=(7, 2, D)), rng.integers(-30, 90, size=(3, 7))
    got = oracle.rope_axes(x, pos, dims, base, halves, shared)
    theta = [base ** (-2 * i / 12) for i in range(6)] if shared else \
        [1.0, base ** (-2 / 4), 1.0, base ** (-2 / 6), base ** (-4 / 6), 1.0]
    axis = [0, 0, 1, 1, 1, 2]
    for i in range(6):
        a, b = (i, i + 6) if halves else (2 * i, 2 * i + 1)
        z = (x[..., a] + 1j * x[..., b]) * np.exp(1j * pos[axis[i]] * theta[i])[:, None]
        np.testing.assert_allclose(got[..., a], z.real, atol=1e-12)
        np.testing.assert_allclose(got[..., b], z.imag, atol=1e-12)
    assert (got[..., 12:] == x[..., 12:]).all()


@pytest.mark.parametrize("name", ["none", "relu", "silu", "gelu", "gelu_tanh"])
def test_activations_match_a_library(name):
    v = torch.linspace(-30, 30, 4001, dtype=torch.float64)
    F = torch.nn.functional
    want = {"none": lambda t: t, "relu": F.relu, "silu": F.silu, "gelu": F.gelu,
            "gelu_tanh": lambda t: F.gelu(t, approximate="tanh")}[name](v)
    np.testing.assert_allclose(oracle.activation(v.numpy(), name), want.numpy(), atol=1e-13)


def test_linear_layers_against_loops():
    rng = np.random.default_rng(4)
    x, w, w2 = rng.normal(size=(3, 5)), rng.normal(size=(4, 5)), rng.normal(size=(4, 5))
    b, r = rng.normal(size=4), rng.normal(size=(3, 4))
    y, size = oracle.linear_act(x, w, b, "relu", r)
    g, _, _, _, _ = oracle.linear_gated(x, w, w2, "relu")
    for m in range(3):
        for n in range(4):
            v = sum(x[m, i] * w[n, i] for i in range(5))
            u = sum(x[m, i] * w2[n, i] for i in range(5))
            assert y[m, n] == pytest.approx(r[m, n] + max(0.0, v + b[n]))
            assert g[m, n] == pytest.approx(max(0.0, v) * u)
            assert size[m, n] == pytest.approx(sum(abs(x[m, i] * w[n, i]) for i in range(5)) +
                                               abs(b[n]))
    np.testing.assert_allclose(oracle.linear_act(x, w, b)[0], oracle.linear(x, w, b))


# ------------------------------------------------------------------ refusals on the host

@pytest.fixture(scope="module")
def lib(lib_path):
    import packed_varlen_gb300 as pv
    return pv.load_library(lib_path)


A, MIS = 0x10000, 0x10008     # never dereferenced: every call is refused before a launch


def _broken(fn, ok, cases):
    """Every call has exactly one broken argument, so nothing reaches the device."""
    for i, value, code in cases:
        args = list(ok)
        args[i] = value
        assert fn(*args) == code, (i, value)


def test_prompt_attention_host_checks(lib):
    ok = [A] * 6 + [2, 10, 10, 8, 8, 4096, 1024, 1024, 32, 8, 128, 1, 0.1, None]
    _broken(lib.pa_prompt_attn_fwd, ok, [
        (0, None, 1), (1, None, 1), (2, None, 1), (3, None, 1), (4, None, 1), (5, None, 1),
        (6, 0, 1), (7, -1, 1), (8, -1, 1), (9, -1, 1), (10, -1, 1), (11, 4088, 1), (12, 1016, 1),
        (13, 0, 1), (14, 0, 1), (14, 30, 1), (15, 0, 1), (15, 5, 1), (18, math.inf, 1),
        (18, math.nan, 1), (18, 3e38, 1), (6, 1025, 2), (7, (1 << 30) + 1, 2),
        (8, (1 << 30) + 1, 2), (11, (1 << 38) + 8, 2), (0, MIS, 3), (1, MIS, 3), (2, MIS, 3),
        (3, MIS, 3), (4, A + 2, 3), (5, A + 1, 3), (11, 4100, 3), (12, 1028, 3), (13, 1025, 3)])
    for D in (32, 96, 256):
        args = list(ok)
        args[11:14], args[16] = [32 * D, 8 * D, 8 * D], D
        assert lib.pa_prompt_attn_fwd(*args) == 2
    # more items than the list's 32 bits are meant for
    args = list(ok)
    args[7], args[11], args[14] = 1 << 30, 128 << 10, 1 << 10
    assert lib.pa_prompt_attn_fwd(*args) == 2
    for i in (7, 9):        # no queries: nothing to do
        args = list(ok)
        args[i] = 0
        if i == 7:
            args[0] = args[3] = None
        assert lib.pa_prompt_attn_fwd(*args) == 0


def _dims(*d):
    arr = (ctypes.c_int32 * len(d))(*d)
    return ctypes.addressof(arr), arr


def test_rope_axes_host_checks(lib):
    at, keep = _dims(32, 48, 48)
    ok = [A] * 4 + [A, None, at, 3, 10, 4096, 1024, 4096, 1024, 32, 8, 128, 0, 1, 1e4, None]
    big = 1 << 39
    _broken(lib.pa_rope_axes, ok, [
        (0, None, 1), (1, None, 1), (2, None, 1), (3, None, 1), (4, None, 1), (6, None, 1),
        (7, 0, 1), (8, -1, 1), (9, 4088, 1), (10, 1016, 1), (11, 8, 1), (12, 8, 1), (13, 0, 1),
        (14, -1, 1), (15, 120, 1), (18, 0.0, 1), (18, -2.0, 1), (18, math.inf, 1),
        (18, math.nan, 1), (7, 9, 2), (15, 264, 2), (15, 132, 2), (9, big, 1), (0, MIS, 3),
        (1, MIS, 3), (2, MIS, 3), (3, MIS, 3), (4, A + 2, 3), (5, A + 2, 3)])
    out = list(ok)
    out[2] = out[3] = A + 4096
    _broken(lib.pa_rope_axes, out, [(9, big, 2), (10, big, 2), (11, big, 2), (12, big, 2),
                                    (9, 4100, 3), (10, 1028, 3), (11, 4100, 3), (12, 1025, 3),
                                    (8, 1 << 30, 2)])
    for dims, code in (((32, 48, 47), 1), ((128, 0), 1), ((64, 66), 1), ((2, 2), 2), ((-8, 8), 1),
                       ((1 << 30, 1 << 30, 1 << 30), 1)):
        args = list(ok)
        args[6], other = _dims(*dims)
        args[7] = len(dims)
        assert lib.pa_rope_axes(*args) == code, dims
    args = [None] * 6 + ok[6:]
    args[8] = 0
    assert lib.pa_rope_axes(*args) == 0
    assert list(keep) == [32, 48, 48]


def test_axis_widths_are_whole_numbers():
    import packed_varlen_gb300 as pv
    with pytest.raises(TypeError):
        pv._host_ints((31.5, 32.5))
    with pytest.raises((ValueError, OverflowError, pv.PackedAttnError)):
        pv._host_ints((1 << 40, 2))


def test_linear_epilogue_host_checks(lib):
    ok = [A, A, A, A, A + 64, 300, 512, 4096, 4096, 512, 512, 3, None]
    big = 1 << 39
    _broken(lib.pa_linear_act_bf16, ok, [
        (0, None, 1), (1, None, 1), (4, None, 1), (5, -1, 1), (6, 0, 1), (7, 0, 1), (8, 4088, 1),
        (9, 504, 1), (10, 504, 1), (11, -1, 1), (11, 5, 1), (8, big, 2), (9, big, 2), (10, big, 2),
        (6, 508, 3), (7, 4092, 3), (8, 4100, 3), (9, 516, 3), (10, 516, 3), (0, MIS, 3),
        (1, MIS, 3), (2, MIS, 3), (3, MIS, 3), (4, MIS, 3)])
    args = list(ok)
    args[3] = args[4]       # in place, but not the same rows
    args[9] = 520
    assert lib.pa_linear_act_bf16(*args) == 1
    args = list(ok)         # sums too long to end within the waits for them
    args[7], args[8] = (1 << 26) + 8, 1 << 27
    assert lib.pa_linear_act_bf16(*args) == 2
    args = list(ok)
    args[0] = args[4] = None
    args[5] = 0
    assert lib.pa_linear_act_bf16(*args) == 0
    ok = [A, A, A, A, 300, 512, 4096, 4096, 512, 2, None]
    _broken(lib.pa_linear_gated_bf16, ok, [
        (0, None, 1), (1, None, 1), (2, None, 1), (3, None, 1), (4, -1, 1), (5, 0, 1), (6, 0, 1),
        (7, 4088, 1), (8, 504, 1), (9, -1, 1), (9, 5, 1), (7, big, 2), (8, big, 2), (5, 508, 3),
        (6, 4092, 3), (7, 4100, 3), (8, 516, 3), (0, MIS, 3), (1, MIS, 3), (2, MIS, 3),
        (3, MIS, 3)])
    args = list(ok)
    args[6], args[7] = (1 << 26) + 8, 1 << 27
    assert lib.pa_linear_gated_bf16(*args) == 2
    args = list(ok)
    args[0] = args[3] = None
    args[4] = 0
    assert lib.pa_linear_gated_bf16(*args) == 0
