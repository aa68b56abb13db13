"""tq_rmsnorm against the formula in 64 bits and against its defined steps."""
from __future__ import annotations

import numpy as np
import pytest

from oracle import BF16, F32, I8
from tests import operator_ref as ref

pytestmark = pytest.mark.gpu
EPS = 1e-5
# widths around the edges of every kernel shape: one wave, workgroups, the widest row
WIDTHS = [16, 48, 64, 256, 272, 1008, 1024, 1040, 2048, 2560, 4096, 4112, 6912, 8192, 8208, 14336, 16384, 16400, 32768, 32784, 65536]


def _torch():
    import torch
    return torch


def _dtype(t):
    torch = _torch()
    return {F32: torch.float32, BF16: torch.bfloat16, I8: torch.int8}[t]


def _typed(a, t):
    """fp32 values of the type, on the host, and the tensor that holds them."""
    v = ref.bf16(a) if t == BF16 else a.astype(np.float32)
    return v, _torch().from_numpy(v).to(_dtype(t)).cuda()


def _inputs(M, K, xt, rt, seed=0):
    rng = np.random.default_rng(1000 * K + M + seed)
    x = rng.standard_normal((M, K)).astype(np.float32) * rng.choice([0.01, 1.0, 30.0], size=(M, 1)).astype(np.float32)
    w = rng.uniform(-1.5, 1.5, K).astype(np.float32)
    res = None if rt is None else rng.standard_normal((M, K)).astype(np.float32)
    return x, res, w


def _guarded(M, K, dtype, fill):
    """An M x K output inside a larger buffer; what is around it must stay."""
    torch = _torch()
    whole = torch.full((64 + M * K + 4096,), fill, dtype=dtype, device="cuda")
    return whole, whole[64:64 + M * K].view(M, K)


def _untouched(whole, n, fill):
    w = whole.float().cpu().numpy()
    assert np.all(w[:64] == fill) and np.all(w[64 + n:] == fill)


def run(M, K, xt, rt, yt, in_place=False, eps=EPS, seed=0, x=None, res=None, w=None):
    from ternary_weight_amd import tq
    torch = _torch()
    if x is None:
        x, res, w = _inputs(M, K, xt, rt, seed)
    x, xd = _typed(x, xt)
    res, rd = (None, None) if rt is None else _typed(res, rt)
    ro = None if rt is None else (rd if in_place else torch.empty_like(rd))
    whole, y = _guarded(M, K, _dtype(yt), 99.0)
    s = torch.full((M,), float("nan"), device="cuda") if yt == I8 else None
    print("norm", M, K, xt, rt, yt, in_place, flush=True)
    tq.rmsnorm(M, K, xt, xd, torch.from_numpy(w).cuda(), eps, yt, y, s, residual_type=F32 if rt is None else rt,
               residual=rd, residual_out=ro)
    torch.cuda.synchronize()
    _untouched(whole, M * K, 99.0)
    return (x, res, w), None if ro is None else ro.float().cpu().numpy(), y.float().cpu().numpy(), \
        None if s is None else s.cpu().numpy()


def check(M, K, xt, rt, yt, **kw):
    (x, res, w), ro, y, s = run(M, K, xt, rt, yt, **kw)
    eps = kw.get("eps", EPS)
    h, n = ref.norm_exact(x, res, w, np.float32(eps))
    hs, ns = ref.norm_steps(x, res, w, eps)
    if rt is not None:
        assert np.array_equal(ro, hs if rt == F32 else ref.bf16(hs))       # one rounding of the sum
        assert np.all(np.abs(ro - h) <= (ref.U24 + (ref.U8 if rt == BF16 else 0)) * 1.001 * np.abs(h))
    if yt == I8:
        q, sc = ref.quant_steps(ns)
        assert np.array_equal(s, sc) and np.array_equal(y.astype(np.int8), q)
        # a code is off by half a step and the roundings of n (8 half steps of fp32) and of the quantiser (3)
        assert np.all(np.abs(y * s[:, None].astype(np.float64) - n) <= s[:, None] * (0.5 + 127 * 16 * ref.U24))
    else:
        # 7 fp32 roundings at most (see the reference's pin), and one of bf16
        tol = 8 * ref.U24 + (ref.U8 if yt == BF16 else 0.0)
        assert np.all(np.abs(y - n) <= 1.001 * tol * np.abs(n))
        assert np.array_equal(y, ns if yt == F32 else ref.bf16(ns))


@pytest.mark.parametrize("K", WIDTHS)
def test_widths(K):
    check(3, K, F32, F32, I8)
    check(2, K, BF16, None, F32)
    check(2, K, BF16, BF16, BF16)


@pytest.mark.parametrize("xt", [F32, BF16])
@pytest.mark.parametrize("rt", [None, F32, BF16])
@pytest.mark.parametrize("yt", [F32, BF16, I8])
def test_types(xt, rt, yt):
    for M, K in ((5, 720), (4, 2560), (2, 20480), (2, 40976)):
        check(M, K, xt, rt, yt)
        if rt is not None:
            check(M, K, xt, rt, yt, in_place=True)


@pytest.mark.parametrize("M", [1, 2, 63, 257, 1500])
def test_token_counts(M):
    check(M, 640, F32, BF16, I8)
    check(M, 1616, BF16, F32, BF16)


def test_many_rows():
    """More rows than one launch has workgroups."""
    from ternary_weight_amd import tq
    torch = _torch()
    M, K = (1 << 20) + 5, 16
    x = torch.randn(M, K, device="cuda", generator=torch.Generator(device="cuda").manual_seed(1))
    w = torch.ones(K, device="cuda")
    q, s = torch.empty(M, K, dtype=torch.int8, device="cuda"), torch.empty(M, device="cuda")
    y = torch.empty_like(x)
    tq.rmsnorm(M, K, F32, x, w, EPS, I8, q, s)
    tq.rmsnorm(M, K, F32, x, w, EPS, F32, y)
    torch.cuda.synchronize()
    _, ns = ref.norm_steps(x.cpu().numpy(), None, np.ones(K, np.float32), EPS)
    rq, rs = ref.quant_steps(ns)
    assert np.array_equal(y.cpu().numpy(), ns)
    assert np.array_equal(q.cpu().numpy(), rq) and np.array_equal(s.cpu().numpy(), rs)


def test_beyond_32_bit_offsets():
    """2^31 elements and more: the last rows equal the same rows by themselves."""
    from ternary_weight_amd import tq
    torch = _torch()
    M, K, n = 32800, 65536, 7
    g = torch.Generator(device="cuda").manual_seed(9)
    x = torch.empty(M, K, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    h = torch.empty(M, K, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    w = torch.rand(K, device="cuda", generator=g)
    tail, htail = x[M - n:].clone(), h[M - n:].clone()
    q, s = torch.empty(M, K, dtype=torch.int8, device="cuda"), torch.empty(M, device="cuda")
    tq.rmsnorm(M, K, BF16, x, w, EPS, I8, q, s, BF16, h, h)
    q2, s2 = torch.empty(n, K, dtype=torch.int8, device="cuda"), torch.empty(n, device="cuda")
    tq.rmsnorm(n, K, BF16, tail, w, EPS, I8, q2, s2, BF16, htail, htail)
    assert torch.equal(q[M - n:], q2) and torch.equal(s[M - n:], s2) and torch.equal(h[M - n:], htail)
    assert torch.equal(x[M - n:], tail) and bool(torch.all(s > 0))


def test_same_codes_as_the_quantiser():
    """int8 straight from the norm = the fp32 norm through tq_act_quant_int8."""
    from ternary_weight_amd import tq
    torch = _torch()
    M, K = 37, 6912
    x = torch.randn(M, K, device="cuda", generator=torch.Generator(device="cuda").manual_seed(2))
    w = torch.rand(K, device="cuda") + 0.5
    q, s, q2, s2, y = (torch.empty(M, K, dtype=torch.int8, device="cuda"), torch.empty(M, device="cuda"),
                       torch.empty(M, K, dtype=torch.int8, device="cuda"), torch.empty(M, device="cuda"),
                       torch.empty_like(x))
    tq.rmsnorm(M, K, F32, x, w, EPS, I8, q, s)
    tq.rmsnorm(M, K, F32, x, w, EPS, F32, y)
    tq.act_quant_int8(M, K, F32, y, q2, s2)
    assert torch.equal(q, q2) and torch.equal(s, s2)


@pytest.mark.parametrize("K", [64, 2560])
def test_zero_rows_and_extreme_values(K):
    rng = np.random.default_rng(3)
    x = rng.standard_normal((6, K)).astype(np.float32)
    x[0] = 0.0                                   # a row of nothing: zeros, scale 0
    x[1] *= np.float32(1e-30)                    # its squares are below fp32: the sum is not
    x[2] *= np.float32(1e15)                     # squares near the top of fp32
    x[3, 1:] = 0.0                               # one element alone
    w = np.ones(K, np.float32)
    check(6, K, F32, None, I8, x=x, w=w)
    check(6, K, F32, None, F32, x=x, w=w)
    _, _, y, s = run(6, K, F32, None, I8, x=x, w=w)
    assert np.all(y[0] == 0) and s[0] == 0.0
    check(1, K, F32, None, F32, x=x[5:], w=w, eps=0.0)


def test_non_finite_values_stay_in_their_row():
    x = np.random.default_rng(4).standard_normal((4, 320)).astype(np.float32)
    clean = x.copy()
    x[1, 7], x[2, 9] = np.nan, np.inf
    w = np.ones(320, np.float32)
    for yt in (F32, BF16, I8):
        _, _, y, _ = run(4, 320, F32, None, yt, x=x, w=w)
        _, _, z, _ = run(4, 320, F32, None, yt, x=clean, w=w)
        assert np.array_equal(y[[0, 3]], z[[0, 3]])
        if yt != I8:
            # NaN everywhere in row 1; 1 / inf = 0 in row 2, and inf * 0 at its infinity
            assert np.all(np.isnan(y[1])) and np.isnan(y[2, 9]) and np.all(np.delete(y[2], 9) == 0.0)


def test_norm_over_its_input():
    """y may be x itself."""
    from ternary_weight_amd import tq
    torch = _torch()
    for K in (512, 5120):
        x = torch.randn(9, K, device="cuda", generator=torch.Generator(device="cuda").manual_seed(5))
        w, y = torch.ones(K, device="cuda"), torch.empty(9, K, device="cuda")
        tq.rmsnorm(9, K, F32, x, w, EPS, F32, y)
        tq.rmsnorm(9, K, F32, x, w, EPS, F32, x)
        assert torch.equal(x, y)


def test_graph_and_streams():
    """Captured and replayed with other inputs between, eager calls beside it
    on another stream."""
    from ternary_weight_amd import tq
    torch = _torch()
    M, K = 33, 2560
    g = torch.Generator(device="cuda").manual_seed(6)
    x, h, w = torch.randn(M, K, device="cuda", generator=g), torch.randn(M, K, device="cuda", generator=g), \
        torch.rand(K, device="cuda", generator=g)
    ho, q, s = torch.empty_like(h), torch.empty(M, K, dtype=torch.int8, device="cuda"), torch.empty(M, device="cuda")
    call = lambda st, out: tq.rmsnorm(M, K, F32, x, w, EPS, I8, out[0], out[1], residual=h, residual_out=out[2],
                                      stream=st)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    call(side, (q, s, ho))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        call(None, (q, s, ho))
    for k in range(3):
        x.copy_(torch.randn(M, K, device="cuda", generator=g))
        q.zero_(), s.zero_(), ho.zero_()
        graph.replay()
        eager = torch.empty_like(q), torch.empty_like(s), torch.empty_like(ho)
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            call(None, eager)
        torch.cuda.synchronize()
        assert torch.equal(q, eager[0]) and torch.equal(s, eager[1]) and torch.equal(ho, eager[2])
