"""tq_moe_dispatch, tq_moe_combine and tq_moe_combine_grad against plain
loops: whole numbers equal, sums within the roundings that they make."""
from __future__ import annotations

import numpy as np
import pytest

from oracle import BF16, F32, I8
from tests import operator_ref as ref

pytestmark = pytest.mark.gpu


def _torch():
    import torch
    return torch


def _dtype(t):
    torch = _torch()
    return {F32: torch.float32, BF16: torch.bfloat16, I8: torch.int8}[t]


def _ids(rng, T, k, E, kind):
    if kind == "uniform":
        return np.stack([rng.permutation(E)[:k] if k <= E else rng.integers(0, E, k) for _ in range(T)]).astype(np.int32)
    if kind == "one":                                     # every pair to the last expert
        return np.full((T, k), E - 1, np.int32)
    if kind == "none":
        return np.full((T, k), -1, np.int32)
    ids = np.minimum(rng.geometric(0.3, size=(T, k)) - 1, E - 1).astype(np.int32)     # skewed, experts named twice
    ids[T - T // 5:] = -1                                 # a padded batch
    ids[rng.random((T, k)) < 0.05] = E + rng.integers(0, 1 << 20)                     # ids past the last expert
    return ids


def _workspace(T, k, E):
    from ternary_weight_amd import tq
    n = tq.moe_dispatch_workspace_size(T, k, E)
    return (_torch().full((n,), 0x55, dtype=_torch().uint8, device="cuda"), n) if n else (None, 0)


def dispatch(ids, E, H=0, xt=F32, x=None, xsc=None, stream=None):
    """The call into guarded outputs; returns the device tensors."""
    from ternary_weight_amd import tq
    torch = _torch()
    T, k = ids.shape
    P = T * k
    idx = torch.full((2 * P + E + 1 + 64,), -77, dtype=torch.int32, device="cuda")
    rows, pairs, offs = idx[16:16 + P].view(T, k), idx[16 + P:16 + 2 * P], idx[16 + 2 * P:17 + 2 * P + E]
    xs = torch.full((P + 2, max(H, 1)), 7, dtype=_dtype(xt), device="cuda") if x is not None else None
    xss = torch.full((P + 2,), -3.0, device="cuda") if xsc is not None else None
    ws, n = _workspace(T, k, E)
    tq.moe_dispatch(T, k, E, torch.from_numpy(ids).cuda(), rows, pairs, offs, H, xt, x, xsc, xs, xss, ws, n, stream)
    torch.cuda.synchronize()
    edge = torch.cat([idx[:16], idx[17 + 2 * P + E:]])
    assert torch.all(edge == -77)
    return rows, pairs, offs, xs, xss


SIZES = [(1, 1, 1), (1, 8, 128), (3, 2, 5), (64, 8, 128), (65, 3, 64), (130, 1, 1000), (511, 4, 2), (1024, 8, 16),
         (1025, 8, 257), (700, 13, 1024), (4099, 5, 60), (9001, 64, 7)]


@pytest.mark.parametrize("kind", ["uniform", "skewed", "one", "none"])
@pytest.mark.parametrize("T,k,E", SIZES)
def test_sort(T, k, E, kind):
    rng = np.random.default_rng(T + 7 * k + E)
    ids = _ids(rng, T, k, E, kind)
    print("sort", T, k, E, kind, flush=True)
    rows, pairs, offs, _, _ = dispatch(ids, E)
    for got, want in zip((rows, pairs, offs), ref.dispatch(ids, E)):
        assert np.array_equal(got.cpu().numpy(), want)


@pytest.mark.parametrize("kind", ["uniform", "skewed", "one"])
@pytest.mark.parametrize("T,k,E", [(128, 8, 1024), (1024, 1, 960), (16, 64, 5), (1025, 1, 961), (300, 4, 1000),
                                   (256, 4, 3), (257, 4, 3), (8193, 1, 2), (66000, 8, 1024), (64, 1, 9), (65, 1, 9),
                                   (256, 1, 40), (257, 1, 40), (64, 8, 128), (513, 1, 7), (640, 8, 64), (5121, 1, 64), (8192, 1, 960)])
def test_sort_at_its_kernels_edges(T, k, E, kind):
    """Pair and expert counts on both sides of each way of sorting."""
    test_sort(T, k, E, kind)


def test_more_tokens_than_waves():
    """Batches that a launch walks in a loop: rows there and back, and the gradient."""
    from ternary_weight_amd import tq
    torch = _torch()
    T, E, H = (1 << 22) + 77, 3, 16
    g = torch.Generator(device="cuda").manual_seed(4)
    ids = torch.randint(-1, E, (T, 1), generator=g, device="cuda", dtype=torch.int32)
    x = torch.randint(-127, 128, (T, H), generator=g, device="cuda", dtype=torch.int8)
    xsc = torch.rand(T, device="cuda", generator=g)
    rows, pairs, offs, xs, xss = dispatch(ids.cpu().numpy(), E, H, I8, x, xsc)
    flat = ids.view(-1).long()
    order = torch.sort(torch.where(flat < 0, E, flat), stable=True).indices
    n = int((flat >= 0).sum())
    assert int(offs[E]) == n and torch.equal(pairs[:n].long(), order[:n]) and torch.all(pairs[n:] == -1)
    assert torch.equal(xs[:n], x[order[:n]]) and torch.equal(xss[:n], xsc[order[:n]]) and torch.all(xs[n:] == 7)
    ys = torch.randn(T, H, device="cuda", generator=g)
    w = torch.rand(T, 1, device="cuda", generator=g)
    y = torch.empty(T, H, device="cuda")
    tq.moe_combine(T, 1, H, T, rows, w, F32, ys, F32, y)
    used = (flat >= 0)[:, None]
    want = torch.where(used, ys[rows.view(-1).clamp_min(0).long()] * w, 0.0)       # one product: exact rounding
    assert torch.equal(y, want)
    d_ys, d_w = torch.full((T, H), 3.0, device="cuda"), torch.empty(T, 1, device="cuda")
    tq.moe_combine_grad(T, 1, H, T, rows, w, F32, y, F32, ys, d_ys, d_w)
    at = rows.view(-1)[flat >= 0].long()
    assert torch.equal(d_ys[at], (y * w)[flat >= 0]) and torch.all(d_ys[n:] == 3.0)
    dots = torch.where(used, (y.double() * ys[rows.view(-1).clamp_min(0).long()].double()).sum(1, keepdim=True), 0.0)
    mag = torch.where(used, (y.double() * ys[rows.view(-1).clamp_min(0).long()].double()).abs().sum(1, keepdim=True), 0.0)
    assert torch.all((d_w.double() - dots).abs() <= 32 * ref.U24 * mag)


def test_beyond_32_bit_offsets():
    """2^31 elements and more in the sorted rows: there, back and the gradient."""
    from ternary_weight_amd import tq
    torch = _torch()
    T, k, E, H = 16400, 2, 5, 65536
    g = torch.Generator(device="cuda").manual_seed(12)
    ids = torch.randint(0, E, (T, k), generator=g, device="cuda", dtype=torch.int32)
    x = torch.randint(-127, 128, (T, H), generator=g, device="cuda", dtype=torch.int8)
    xsc = torch.rand(T, device="cuda", generator=g)
    rows, pairs, offs, xs, xss = dispatch(ids.cpu().numpy(), E, H, I8, x, xsc)
    P = T * k
    for p0 in range(0, P, 4096):
        t = pairs[p0:p0 + 4096].long() // k
        assert torch.equal(xs[p0:p0 + len(t)], x[t]) and torch.equal(xss[p0:p0 + len(t)], xsc[t])
    del x, xs
    # small whole numbers: every product and sum is exact, in bf16 too
    ys = torch.randint(-4, 5, (P, H), generator=g, device="cuda", dtype=torch.int8).to(torch.bfloat16)
    w = torch.randint(1, 4, (T, k), generator=g, device="cuda").float()
    y = torch.empty(T, H, dtype=torch.bfloat16, device="cuda")
    tq.moe_combine(T, k, H, P, rows, w, BF16, ys, BF16, y)
    dy = torch.randint(-3, 4, (T, H), generator=g, device="cuda", dtype=torch.int8).to(torch.bfloat16)
    d_ys, d_w = torch.empty_like(ys), torch.empty(T, k, device="cuda")
    tq.moe_combine_grad(T, k, H, P, rows, w, BF16, dy, BF16, ys, d_ys, d_w)
    for t0 in range(0, T, 1024):
        t = slice(t0, min(t0 + 1024, T))
        r = rows[t].long()
        picked = ys[r.view(-1)].view(-1, k, H).float()
        assert torch.equal(y[t].float(), (picked * w[t, :, None]).sum(1))
        assert torch.equal(d_ys[r.view(-1)].view(-1, k, H).float(), dy[t, None].float() * w[t, :, None])
        assert torch.equal(d_w[t], (picked * dy[t, None].float()).sum(2))


@pytest.mark.parametrize("xt", [F32, BF16, I8])
@pytest.mark.parametrize("T,k,E,H", [(300, 5, 9, 16400), (1, 1, 1, 16), (5, 3, 4, 48), (64, 8, 128, 2048), (200, 2, 9, 4112),
                                     (1500, 8, 33, 272), (7, 4, 6, 65536)])
def test_rows(T, k, E, H, xt):
    torch = _torch()
    rng = np.random.default_rng(T + H)
    ids = _ids(rng, T, k, E, "skewed")
    x = torch.from_numpy(rng.integers(-127, 128, (T, H)).astype(np.float32)).to(_dtype(xt)).cuda()
    xsc = torch.rand(T, device="cuda") if xt == I8 else None
    print("rows", T, k, E, H, xt, flush=True)
    _, _, _, xs, xss = dispatch(ids, E, H, xt, x, xsc)
    _, pairs, offs = ref.dispatch(ids, E)
    want = torch.full_like(xs, 7)
    token = torch.from_numpy(pairs[:offs[E]] // k).long().cuda()
    want[:offs[E]] = x[token]                                       # the rows behind stay as they were
    assert torch.equal(xs, want)
    if xt == I8:
        want = torch.full_like(xss, -3.0)
        want[:offs[E]] = xsc[token]
        assert torch.equal(xss, want)


def test_empty_batch_and_widths():
    ids = np.zeros((0, 4), np.int32)
    _, _, offs, _, _ = dispatch(ids, 9)
    assert torch_equal(offs, np.zeros(10, np.int32))
    # int8 rows of no width still move their scales
    torch = _torch()
    ids = np.array([[1, 0], [0, -1]], np.int32)
    xsc = torch.tensor([0.5, 0.25], device="cuda")
    _, _, _, _, xss = dispatch(ids, 2, 0, I8, torch.empty(2, 1, dtype=torch.int8, device="cuda"), xsc)
    assert xss.cpu().tolist() == [0.5, 0.25, 0.5, -3.0, -3.0, -3.0]


def torch_equal(t, a):
    return np.array_equal(t.cpu().numpy(), a)


def _moe(T, k, E, H, st, yt, kind="skewed", seed=0):
    """Host values and device tensors of one layer's rows."""
    torch = _torch()
    rng = np.random.default_rng(T + 3 * k + H + seed)
    rows, _, offs = ref.dispatch(_ids(rng, T, k, E, kind), E)
    w = rng.standard_normal((T, k)).astype(np.float32)
    cast = lambda a, t: ref.bf16(a) if t == BF16 else a
    ys = cast(rng.standard_normal((T * k, H)).astype(np.float32), st)
    dy = cast(rng.standard_normal((T, H)).astype(np.float32), yt)
    ys[offs[E]:] = np.nan                                 # rows of no pair are never read into a sum
    w[rows < 0] = np.nan                                  # nor the weights of no expert
    dev = lambda a, t: torch.from_numpy(a).to(_dtype(t)).cuda()
    return (rows, w, ys, dy), (torch.from_numpy(rows).cuda(), torch.from_numpy(w).cuda(), dev(ys, st), dev(dy, yt))


MOES = [(1, 1, 1, 16), (1, 8, 16, 2048), (5, 3, 4, 48), (64, 8, 128, 2048), (33, 2, 7, 4112), (9, 13, 20, 272),
        (3, 64, 9, 1040), (2, 4, 6, 65536), (700, 8, 32, 768)]


@pytest.mark.parametrize("st,yt", [(F32, F32), (F32, BF16), (BF16, F32), (BF16, BF16)])
@pytest.mark.parametrize("T,k,E,H", MOES)
def test_combine(T, k, E, H, st, yt):
    from ternary_weight_amd import tq
    torch = _torch()
    (rows, w, ys, _), (rd, wd, yd, _) = _moe(T, k, E, H, st, yt)
    out = torch.full((T + 1, H), 5.0, dtype=_dtype(yt), device="cuda")
    for weights in (w, None):
        print("combine", T, k, E, H, st, yt, flush=True)
        tq.moe_combine(T, k, H, T * k, rd, None if weights is None else wd, st, yd, yt, out)
        torch.cuda.synchronize()
        y, mag = ref.combine(rows, weights, ys)
        # k products and sums of fp32, each off by half a step of at most the magnitudes' sum, and the last rounding
        tol = (k + 1) * ref.U24 * mag + (ref.U8 if yt == BF16 else 0.0) * (np.abs(y) + (k + 1) * ref.U24 * mag)
        got = out.float().cpu().numpy()
        assert np.all(np.abs(got[:T] - y) <= 1.001 * tol) and np.all(got[T] == 5.0)


@pytest.mark.parametrize("dt,st", [(F32, F32), (F32, BF16), (BF16, F32), (BF16, BF16)])
@pytest.mark.parametrize("T,k,E,H", MOES)
def test_combine_grad(T, k, E, H, dt, st):
    from ternary_weight_amd import tq
    torch = _torch()
    (rows, w, ys, dy), (rd, wd, yd, gd) = _moe(T, k, E, H, st, dt)
    R = T * k
    for weights in (w, None):
        d_ys = torch.full((R + 1, H), 5.0, dtype=_dtype(st), device="cuda")
        d_w = torch.full((T * k + 8,), 6.0, device="cuda")
        print("grad", T, k, E, H, dt, st, flush=True)
        tq.moe_combine_grad(T, k, H, R, rd, None if weights is None else wd, dt, gd, st, yd, d_ys, d_w[:T * k].view(T, k))
        torch.cuda.synchronize()
        want, written, want_w, mag = ref.combine_grad(rows, weights, dy, ys)
        got, got_w = d_ys.float().cpu().numpy(), d_w.cpu().numpy()
        assert np.all(got[:R][~written] == 5.0) and np.all(got[R] == 5.0) and np.all(got_w[T * k:] == 6.0)
        tol = (ref.U24 + (ref.U8 if st == BF16 else 0.0)) * np.abs(want[written])
        assert np.all(np.abs(got[:R][written] - want[written]) <= 1.001 * tol)
        # a chain of at most H / 64 products per lane (64 lanes or more share a row), then a tree and a last few sums
        assert np.all(np.abs(got_w[:T * k].reshape(T, k) - want_w) <= (H // 64 + 32) * ref.U24 * mag)
        # either output alone: the same bits
        o_ys, o_w = torch.full_like(d_ys, 5.0), torch.empty(T, k, device="cuda")
        tq.moe_combine_grad(T, k, H, R, rd, None if weights is None else wd, dt, gd, st, None, o_ys, None)
        tq.moe_combine_grad(T, k, H, R, rd, None, dt, gd, st, yd, None, o_w)
        assert torch.equal(o_ys, d_ys) and torch_equal(o_w.view(-1), got_w[:T * k])


def test_gradient_against_differences():
    """<d_w, d> and <d_ys, D> against what the forward call itself changes by
    (it is linear in each), in fp32."""
    from ternary_weight_amd import tq
    torch = _torch()
    T, k, E, H = 24, 4, 9, 256
    (rows, w, ys, dy), (rd, wd, yd, gd) = _moe(T, k, E, H, F32, F32)
    wd, yd = torch.nan_to_num(wd), torch.nan_to_num(yd)
    f = lambda w_, y_: (tq.moe_combine(T, k, H, T * k, rd, w_, F32, y_, F32, out), out.double().clone())[1]
    out, d_ys, d_w = torch.empty(T, H, device="cuda"), torch.zeros_like(yd), torch.empty(T, k, device="cuda")
    tq.moe_combine_grad(T, k, H, T * k, rd, wd, F32, gd, F32, yd, d_ys, d_w)
    g = torch.Generator(device="cuda").manual_seed(3)
    dw, dY = torch.randn(T, k, device="cuda", generator=g), torch.randn(T * k, H, device="cuda", generator=g)
    base = f(wd, yd)
    host = lambda t: t.cpu().numpy()
    mag = lambda w_, y_: ref.combine(rows, host(w_), host(y_))[1]
    _, _, _, dots = ref.combine_grad(rows, host(wd), dy, host(yd))
    for got, want, more, own in (
            (f(wd + dw, yd), d_w.double() * dw.double(), mag(wd + dw, yd),
             np.sum((H // 64 + 32) * ref.U24 * dots * np.abs(host(dw)))),
            (f(wd, yd + dY), d_ys.double() * dY.double(), mag(wd, yd + dY),
             np.sum(ref.U24 * np.abs(host(d_ys) * host(dY))))):
        got = float(torch.sum(gd.double() * (got - base)))
        # both forward results are off by k + 1 half steps of their magnitudes, the sums w + dw and ys + dY by one
        # half step more, and the gradient by its own roundings
        tol = np.sum(np.abs(dy) * (k + 2) * ref.U24 * (mag(wd, yd) + more)) + own
        assert abs(got - float(torch.sum(want))) <= 1.001 * tol


def test_bad_rows_add_nothing():
    """Row numbers outside the array are not followed."""
    from ternary_weight_amd import tq
    torch = _torch()
    rows = torch.tensor([[0, 2 ** 31 - 1], [-2 ** 31, 3], [4, -1]], dtype=torch.int32, device="cuda")
    ys, y = torch.ones(4, 32, device="cuda"), torch.empty(3, 32, device="cuda")
    tq.moe_combine(3, 2, 32, 4, rows, None, F32, ys, F32, y)
    assert torch.equal(y, torch.tensor([[1.0], [1.0], [0.0]], device="cuda").expand(3, 32))
    d_ys, d_w = torch.zeros(4, 32, device="cuda"), torch.empty(3, 2, device="cuda")
    tq.moe_combine_grad(3, 2, 32, 4, rows, None, F32, y, F32, ys, d_ys, d_w)
    assert d_w.cpu().tolist() == [[32.0, 0.0], [0.0, 32.0], [0.0, 0.0]]
    assert torch.equal(d_ys[:, 0].cpu(), torch.tensor([1.0, 0.0, 0.0, 1.0]))
    tq.moe_combine(3, 2, 32, 0, rows, None, F32, None, F32, y)       # no rows at all
    assert torch.all(y == 0)


def test_two_sorts_at_once_and_a_graph():
    """Two streams with a workspace each, and a captured call replayed with
    other ids between eager calls."""
    from ternary_weight_amd import tq
    torch = _torch()
    T, k, E, H = 4096, 8, 64, 64
    rng = np.random.default_rng(8)
    n = tq.moe_dispatch_workspace_size(T, k, E)

    def state():
        ids = torch.from_numpy(_ids(rng, T, k, E, "skewed")).cuda()
        return {"ids": ids, "x": torch.randn(T, H, device="cuda").to(torch.bfloat16),
                "rows": torch.empty(T, k, dtype=torch.int32, device="cuda"),
                "pairs": torch.empty(T * k, dtype=torch.int32, device="cuda"),
                "offs": torch.empty(E + 1, dtype=torch.int32, device="cuda"),
                "xs": torch.zeros(T * k, H, dtype=torch.bfloat16, device="cuda"),
                "ws": torch.empty(n, dtype=torch.uint8, device="cuda")}

    def call(s, stream=None):
        tq.moe_dispatch(T, k, E, s["ids"], s["rows"], s["pairs"], s["offs"], H, BF16, s["x"], None, s["xs"], None,
                        s["ws"], n, stream)

    def check(s):
        rows, pairs, offs = ref.dispatch(s["ids"].cpu().numpy(), E)
        assert torch_equal(s["rows"], rows) and torch_equal(s["pairs"], pairs) and torch_equal(s["offs"], offs)
        token = torch.from_numpy(pairs[:offs[E]] // k).long().cuda()
        assert torch.equal(s["xs"][:offs[E]], s["x"][token])

    a, b = state(), state()
    sa, sb = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        call(a, sa)
        call(b, sb)
    torch.cuda.synchronize()
    check(a), check(b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=sa):
        call(a)
    for _ in range(3):
        a["ids"].copy_(torch.from_numpy(_ids(rng, T, k, E, "skewed")).cuda())
        a["rows"].zero_(), a["xs"].zero_()
        call(b)
        graph.replay()
        torch.cuda.synchronize()
        check(a), check(b)
