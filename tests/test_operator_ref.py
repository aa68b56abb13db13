"""The plain references of the operators, pinned without a GPU: closed forms,
invariants and difference quotients."""
from __future__ import annotations

import numpy as np
import pytest

import oracle
from tests import operator_ref as ref


def test_bf16_rounding():
    import torch
    v = np.random.default_rng(0).standard_normal(4096).astype(np.float32) * 3.0
    v[:4] = [1.0 + 2.0 ** -8, 1.0 + 3 * 2.0 ** -8, -2.0, 0.0]        # two ties: to even
    assert np.array_equal(ref.bf16(v), torch.from_numpy(v).to(torch.bfloat16).float().numpy())


def test_norm_closed_forms():
    # a row of +-c has mean square c^2: the norm is the sign times the weight
    x = np.array([[3.0, -3.0, 3.0, 3.0]], np.float32)
    w = np.array([0.5, 1.0, 2.0, -1.0], np.float32)
    h, n = ref.norm_exact(x, None, w, 0.0)
    assert np.allclose(n, [[0.5, -1.0, 2.0, -1.0]], atol=1e-15) and np.array_equal(h, x)
    # the residual is added before the norm; scaling h scales nothing
    r = np.array([[1.0, 5.0, -1.0, -1.0]], np.float32)
    _, a = ref.norm_exact(x, r, w, 0.0)
    _, b = ref.norm_exact(2 * (x + r), None, w, 0.0)
    assert np.allclose(a, b, rtol=1e-15)


def test_norm_steps_are_near_the_formula():
    rng = np.random.default_rng(1)
    x, r = rng.standard_normal((9, 272)).astype(np.float32), rng.standard_normal((9, 272)).astype(np.float32)
    w = rng.uniform(0.5, 1.5, 272).astype(np.float32)
    _, a = ref.norm_steps(x, r, w, 1e-5)
    # relative roundings of a value: h (1), the mean's (h: 2, itself: 1, + eps: 1, halved by the root), the root,
    # the quotient and the two products: 1 + 2 + 4 = 7 half steps; the sum x + r is exact to one rounding of h
    h, b = ref.norm_exact(x, r, w, np.float32(1e-5))
    assert np.all(np.abs(a - b) <= 8 * ref.U24 * np.abs(b))


def test_quant_steps_are_the_oracles():
    rng = np.random.default_rng(2)
    n = rng.standard_normal((7, 160)).astype(np.float32)
    n[3] = 0.0
    q, s = ref.quant_steps(n)
    oq, os_ = oracle.act_quant_i8(n)
    assert np.array_equal(q, oq) and np.array_equal(s, os_)


@pytest.mark.parametrize("T,k,E", [(1, 1, 1), (5, 3, 4), (40, 8, 16)])
def test_dispatch_invariants(T, k, E):
    rng = np.random.default_rng(T)
    ids = rng.integers(-1, E + 1, size=(T, k)).astype(np.int32)      # some of no expert, on both sides
    rows, pairs, offs = ref.dispatch(ids, E)
    flat = ids.reshape(-1)
    assert offs[0] == 0 and np.array_equal(np.diff(offs), [np.sum(flat == e) for e in range(E)])
    used = pairs[:offs[E]]
    assert np.array_equal(rows.reshape(-1)[used], np.arange(offs[E])) and np.all(pairs[offs[E]:] == -1)
    key = flat[used].astype(np.int64) * (T * k) + used               # by expert, then by pair
    assert np.all(np.diff(key) > 0)
    assert np.array_equal(rows < 0, (ids < 0) | (ids >= E))


def test_combine_gradient_against_differences():
    rng = np.random.default_rng(3)
    T, k, E, H = 4, 3, 5, 16
    ids = rng.integers(-1, E, size=(T, k)).astype(np.int32)
    rows, _, _ = ref.dispatch(ids, E)
    w, ys, dy = rng.standard_normal((T, k)), rng.standard_normal((T * k, H)), rng.standard_normal((T, H))
    d_ys, _, d_w, _ = ref.combine_grad(rows, w, dy, ys)
    loss = lambda w_, ys_: float(np.sum(dy * ref.combine(rows, w_, ys_)[0]))
    base, step = loss(w, ys), 2.0 ** -10
    for t in range(T):
        for j in range(k):
            w1 = w.copy()
            w1[t, j] += step
            assert abs((loss(w1, ys) - base) / step - d_w[t, j]) <= 1e-10     # the loss is linear in each
    for r, i in [(0, 0), (2, 7), (T * k - 1, 15)]:
        y1 = ys.copy()
        y1[r, i] += step
        assert abs((loss(w, y1) - base) / step - d_ys[r, i]) <= 1e-10


def test_dense_matches_integer_sums():
    rng = np.random.default_rng(4)
    xq, wq = rng.integers(-128, 128, (3, 80)).astype(np.int8), rng.integers(-128, 128, (5, 80)).astype(np.int8)
    one = np.ones(3, np.float32), np.ones(5, np.float32)
    want = xq.astype(np.int64) @ wq.astype(np.int64).T
    assert np.array_equal(ref.dense_i8(xq, one[0], wq, one[1]), want.astype(np.float32))
