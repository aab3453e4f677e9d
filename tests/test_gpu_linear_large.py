"""The linear layers with an epilogue through each of their two kernels (for few rows, and on
CTA pairs).  The one for few rows takes 4096 at most, so the sizes here reach both whatever
rule chooses between them; a call's kernel in a captured graph shows which it took."""
import ctypes
import math

import numpy as np
import pytest
import torch

import oracle
from test_gpu_prompt import (ACTS, BF16, _bits, _check_gated, _check_linear, _cuda, _linear_inputs,
                             _round, _within)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pv():
    import packed_varlen_gb300 as pv
    pv.load_library()
    pv.get_device_status()
    return pv


class _KernelNode(ctypes.Structure):   # CUDA_KERNEL_NODE_PARAMS
    _fields_ = [("func", ctypes.c_void_p), ("dims", ctypes.c_uint * 6), ("smem", ctypes.c_uint),
                ("params", ctypes.c_void_p), ("extra", ctypes.c_void_p), ("kern", ctypes.c_void_p),
                ("ctx", ctypes.c_void_p)]


def _kernels_of(call):
    """Names of the kernels that a call launches."""
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph(keep_graph=True)
    with torch.cuda.graph(graph):
        call()
    cu = ctypes.CDLL("libcuda.so.1")
    raw, count = ctypes.c_void_p(graph.raw_cuda_graph()), ctypes.c_size_t(0)
    assert cu.cuGraphGetNodes(raw, None, ctypes.byref(count)) == 0
    nodes = (ctypes.c_void_p * count.value)()
    assert cu.cuGraphGetNodes(raw, nodes, ctypes.byref(count)) == 0
    names = []
    for node in nodes:
        kind, params, name = ctypes.c_int(-1), _KernelNode(), ctypes.c_char_p()
        assert cu.cuGraphNodeGetType(ctypes.c_void_p(node), ctypes.byref(kind)) == 0
        if kind.value != 0:
            continue
        assert cu.cuGraphKernelNodeGetParams_v2(ctypes.c_void_p(node), ctypes.byref(params)) == 0
        assert cu.cuFuncGetName(ctypes.byref(name), ctypes.c_void_p(params.func)) == 0
        names.append(name.value.decode())
    return names


def _run(call, large):
    """The call's result, by the kernel it has to take."""
    names = _kernels_of(call)
    assert len(names) == 1
    assert ("linear_bf16_kernel" if large else "linear_few_kernel") in names[0], names
    return call()


def _sample(M):
    """Rows of every block of 32, and those at the edges."""
    rng = np.random.default_rng(M)
    rows = {0, M - 1} | {min(M - 1, t + int(rng.integers(32))) for t in range(0, M, 32)}
    rows |= {t + d for t in range(128, M, 128) for d in (-1, 0)}
    return torch.as_tensor(sorted(rows))


# (rows, features, depth): more tiles than CTA pairs in those of 2056 features and more
LARGE = [(4111, 264, 72), (4300, 2056, 136), (4097, 520, 328), (4500, 5128, 200)]
FEW = [(3, 1288, 72), (30, 2056, 136)]


@pytest.mark.parametrize("M,N,K", LARGE + FEW)
@pytest.mark.parametrize("act", ACTS)
def test_linear_act(pv, M, N, K, act):
    at = _sample(M)
    for bias, residual in ((False, False), (True, True), (False, True)):
        x, w, b, r = _linear_inputs(M, N, K, M + N + K, bias, residual)
        xd, wd, bd, rd = _cuda(x, w, b, r)
        got = _run(lambda: pv.linear_act_bf16(xd, wd, bd, act=act, residual=rd), M > 4096)
        _check_linear(got.cpu()[at], x[at], w, b, act, None if r is None else r[at])
        # and in place
        if residual:
            y = rd.clone()
            pv.linear_act_bf16(xd, wd, bd, act=act, residual=y, out=y)
            assert torch.equal(_bits(y), _bits(got))
    assert pv.get_device_status() == 0


@pytest.mark.parametrize("M,N,K", LARGE + FEW)
@pytest.mark.parametrize("act", ACTS)
def test_linear_gated(pv, M, N, K, act):
    at = _sample(M)
    x, w, _, _ = _linear_inputs(M, N, K, M + N + K, False, False)
    w2 = _linear_inputs(1, N, K, 7, False, False)[1]
    xd, wd, w2d = _cuda(x, w, w2)
    got = _run(lambda: pv.linear_gated_bf16(xd, wd, w2d, act=act), M > 4096)
    _check_gated(got.cpu()[at], x[at], w, w2, act)
    assert pv.get_device_status() == 0


@pytest.mark.parametrize("M", [30, 4300])
@pytest.mark.parametrize("act", ["relu", "gelu_tanh"])
def test_strides_guards_and_in_place(pv, M, act):
    """Slices of wider matrices, whose other elements stay what they were."""
    N, K = 2056, 136
    large = M > 4096
    x, w, b, r = _cuda(*_linear_inputs(M, N, K, 3))
    w2 = _linear_inputs(1, N, K, 9)[1].cuda()
    want = _run(lambda: pv.linear_act_bf16(x, w, b, act=act, residual=r), large)
    gated = _run(lambda: pv.linear_gated_bf16(x, w, w2, act=act), large)

    def wide(n):
        return torch.full((M + 2, n + 24), 5.0, dtype=BF16, device="cuda")

    def inside(t, n):
        return t[1:M + 1, 8:8 + n]

    def around(t, n):
        return (t[0] == 5).all() and (t[M + 1] == 5).all() and (t[:, :8] == 5).all() and \
            (t[:, 8 + n:] == 5).all()

    wx, wr, wy = wide(K), wide(N), wide(N)
    inside(wx, K).copy_(x)
    inside(wr, N).copy_(r)
    for out in (wy, wr):           # into another matrix, then in place
        _run(lambda: pv.linear_act_bf16(inside(wx, K), w, b, act=act, residual=r,
                                        out=inside(wy, N)), large)
        pv.linear_act_bf16(inside(wx, K), w, b, act=act, residual=inside(wr, N),
                           out=inside(out, N))
        assert torch.equal(_bits(inside(out, N)), _bits(want)) and around(out, N)
    wy.fill_(5.0)
    pv.linear_gated_bf16(inside(wx, K), w, w2, act=act, out=inside(wy, N))
    assert torch.equal(_bits(inside(wy, N)), _bits(gated)) and around(wy, N)
    assert pv.get_device_status() == 0


@pytest.mark.parametrize("M", [30, 4300])
def test_bad_rows_stay_their_own(pv, M):
    """NaN and infinities in rows of x and of the residual, behind and beside the rows."""
    N, K = 2056, 136
    x, w, b, r = _cuda(*_linear_inputs(M, N, K, 6))
    want = pv.linear_act_bf16(x, w, b, residual=r, act="silu")
    gated = pv.linear_gated_bf16(x, w, w)
    xd = torch.full((M + 300, K + 8), math.nan, dtype=BF16, device="cuda")
    rd = torch.full((M + 300, N + 64), math.nan, dtype=BF16, device="cuda")
    xd[:M, :K], rd[:M, :N] = x, r
    bad_x, bad_r = [2, 17, M - 1], [0, 16, M - 2]
    xd[bad_x, 5], rd[bad_r, 7] = math.inf, math.nan
    got = _run(lambda: pv.linear_act_bf16(xd[:M, :K], w, b, residual=rd[:M, :N], act="silu"),
               M > 4096)
    keep = [m for m in range(M) if m not in bad_x]
    same = _bits(got) == _bits(want)
    same[bad_r, 7] = True
    assert same[keep].all() and torch.isnan(got[bad_r, 7]).all()
    assert not torch.isfinite(got[bad_x]).all()
    got = _run(lambda: pv.linear_gated_bf16(xd[:M, :K], w, w), M > 4096)
    assert torch.equal(_bits(got[keep]), _bits(gated[keep]))
    assert pv.get_device_status() == 0


@pytest.mark.parametrize("M", [289, 4300])    # (the first by either)
@pytest.mark.parametrize("act", ACTS)
def test_activations_over_their_range(pv, act, M):
    """Values from tiny to huge, by a product with one."""
    N, K = 2056, 136
    v = torch.cat([torch.linspace(-40, 40, 161), torch.logspace(-30, 30, 61),
                   -torch.logspace(-30, 30, 61), torch.zeros(6)]).to(BF16)
    x, w = torch.zeros(M, K, dtype=BF16), torch.zeros(N, K, dtype=BF16)
    w[:, 0] = 1.0
    x[:, 0] = v.repeat(M // len(v) + 1)[:M]
    x[7, 0], x[8, 0] = math.nan, math.inf
    xd, wd = x.cuda(), w.cuda()
    got = pv.linear_act_bf16(xd, wd, act=act).cpu()
    assert torch.isnan(got[7]).all() and (got[8].float() == math.inf).all()
    x[7:9, 0], got[7:9] = 0, 0
    want = oracle.activation(oracle.to_f64(x[:, :1]), act)
    # the exponents' rounding: 2^-22 of the argument, relative to the result
    e = np.minimum(np.abs(oracle.to_f64(x[:, :1])), 100.0) ** 2
    _within(got, want, _round(want) + (2.0 ** -18 + 2.0 ** -22 * e) * np.abs(want) + 1.2e-38)
    assert pv.get_device_status() == 0


def test_rows_keep_their_bits_by_either_kernel(pv):
    M, N, K = 4301, 2056, 136
    x, w, b, r = _cuda(*_linear_inputs(M, N, K, 11))
    w2 = _linear_inputs(1, N, K, 12)[1].cuda()
    rows = slice(700, 730)
    for act in ACTS:
        whole = _run(lambda: pv.linear_act_bf16(x, w, b, act=act, residual=r), True)
        part = _run(lambda: pv.linear_act_bf16(x[rows], w, b, act=act, residual=r[rows]), False)
        assert torch.equal(_bits(part), _bits(whole[rows]))
        whole = _run(lambda: pv.linear_gated_bf16(x, w, w2, act=act), True)
        part = _run(lambda: pv.linear_gated_bf16(x[rows], w, w2, act=act), False)
        assert torch.equal(_bits(part), _bits(whole[rows]))
    assert pv.get_device_status() == 0


def test_two_streams(pv):
    """Calls of both kernels at once on two streams, then in two graphs."""
    N, K = 2056, 1032
    w, w2 = (_linear_inputs(1, N, K, s, False, False)[1].cuda() for s in (1, 2))
    xs = [_cuda(*_linear_inputs(m, N, K, 20 + m)) for m in (4300, 4501)]

    def calls(x, b, r):
        return [pv.linear_act_bf16(x, w, b, act="gelu_tanh", residual=r),
                pv.linear_gated_bf16(x, w, w2),
                pv.linear_act_bf16(x[:40], w, b, act="silu", residual=r[:40]),
                pv.linear_gated_bf16(x[:40], w, w2, act="gelu")]

    want = [calls(x, b, r) for x, _, b, r in xs]
    streams, got, graphs = [torch.cuda.Stream(), torch.cuda.Stream()], [None, None], []
    torch.cuda.synchronize()
    for _ in range(5):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                x, _, b, r = xs[i]
                got[i] = calls(x, b, r)
    torch.cuda.synchronize()
    for a, c in zip(want, got):
        assert all(torch.equal(_bits(p), _bits(q)) for p, q in zip(a, c))
    for i, s in enumerate(streams):
        g = torch.cuda.CUDAGraph()
        x, _, b, r = xs[i]
        with torch.cuda.graph(g, stream=s):
            got[i] = calls(x, b, r)
        graphs.append(g)
    for t in got[0] + got[1]:
        t.fill_(5.0)
    torch.cuda.synchronize()
    for _ in range(4):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for a, c in zip(want, got):
        assert all(torch.equal(_bits(p), _bits(q)) for p, q in zip(a, c))
    assert pv.get_device_status() == 0
