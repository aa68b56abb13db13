"""A mixture-of-experts layer as a served model runs it, on the library's
calls alone between the router's top-k and the gated activation: RMSNorm with
the residual to int8, the dense router, the tokens sorted by expert, the
experts' ternary products in one launch, the rows back with their weights,
the next norm and the output head.  Every stage against its plain reference
on what the stage before it gave, and the whole run twice for equal bits."""
from __future__ import annotations

import numpy as np
import pytest

import oracle
from oracle import F32, I8, TENSOR
from tests import operator_ref as ref
from tests.gpu_util import pack

pytestmark = pytest.mark.gpu

T, HID, INTER, E, TOP, VOCAB, EPS = 21, 320, 192, 8, 2, 1003, 1e-5


def _weights():
    rng = np.random.default_rng(12)
    trits = lambda n, k: rng.choice(np.array([-1, 0, 1], np.int8), size=(1, n, k), p=[0.3, 0.4, 0.3])
    shapes = [(INTER, HID), (INTER, HID), (HID, INTER)]
    experts = [[(trits(n, k), rng.uniform(0.01, 0.05, 1).astype(np.float32)) for n, k in shapes] for _ in range(E)]
    dense = lambda n, k: (rng.integers(-127, 128, (n, k)).astype(np.int8), rng.uniform(1e-4, 1e-3, n).astype(np.float32))
    norms = [rng.uniform(0.5, 1.5, HID).astype(np.float32) for _ in range(2)]
    return experts, dense(E, HID), dense(VOCAB, HID), norms


def _run(x, h, experts, router, head, norms):
    """One pass; every stage's tensors by name."""
    import torch
    from ternary_weight_amd import tq
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()
    new = lambda *s, dt=torch.float32: torch.empty(*s, dtype=dt, device="cuda")
    o = {"x": dev(x), "h0": dev(h)}
    P = T * TOP
    o["q"], o["s"], o["h"] = new(T, HID, dt=torch.int8), new(T), new(T, HID)
    tq.rmsnorm(T, HID, F32, o["x"], dev(norms[0]), EPS, I8, o["q"], o["s"], residual=o["h0"], residual_out=o["h"])
    o["logits"] = new(T, E)
    tq.gemm_dense_i8(T, E, HID, o["q"], o["s"], dev(router[0]), dev(router[1]), F32, o["logits"])
    top, ids = o["logits"].topk(TOP, dim=1)
    o["ids"], o["w"] = ids.to(torch.int32).contiguous(), torch.softmax(top, 1).contiguous()
    o["ids"][T - 2:] = -1                                          # two padding tokens
    i32 = torch.int32
    o["rows"], o["pairs"], o["offs"] = new(T, TOP, dt=i32), new(P, dt=i32), new(E + 1, dt=i32)
    o["xs"], o["xss"] = torch.zeros(P, HID, dtype=torch.int8, device="cuda"), torch.zeros(P, device="cuda")
    tq.moe_dispatch(T, TOP, E, o["ids"], o["rows"], o["pairs"], o["offs"], HID, I8, o["q"], o["s"], o["xs"], o["xss"])
    offs = o["offs"].cpu().tolist()

    def products(p, x, xs, n):
        """Every expert's p-th matrix, experts with more than 16 rows in pieces."""
        y = torch.zeros(P, n, device="cuda")
        items, tokens = [], []
        for e in range(E):
            for a in range(offs[e], offs[e + 1], 16):
                b = min(a + 16, offs[e + 1])
                items.append((*experts[e][p], x[a:b], xs[a:b], y[a:b], None))
                tokens.append(b - a)
        probs = tq.problems(items)
        ws = torch.empty(tq.gemv_grouped_workspace_size(probs, 16), dtype=torch.uint8, device="cuda")
        tq.gemv_grouped_run(tq.gemv_grouped_prepare_tokens(probs, tokens, I8, ws, ws.numel()))
        return y

    o["gate"], o["up"] = products(0, o["xs"], o["xss"], INTER), products(1, o["xs"], o["xss"], INTER)
    o["act"] = torch.relu(o["gate"]).square() * o["up"]
    o["aq"], o["as"] = new(P, INTER, dt=torch.int8), new(P)
    tq.act_quant_int8(P, INTER, F32, o["act"], o["aq"], o["as"])
    o["down"] = products(2, o["aq"], o["as"], HID)
    o["moe"] = new(T, HID)
    tq.moe_combine(T, TOP, HID, P, o["rows"], o["w"], F32, o["down"], F32, o["moe"])
    o["q2"], o["s2"], o["h2"] = new(T, HID, dt=torch.int8), new(T), o["h"].clone()
    tq.rmsnorm(T, HID, F32, o["moe"], dev(norms[1]), EPS, I8, o["q2"], o["s2"], residual=o["h2"], residual_out=o["h2"])
    o["out"] = new(T, VOCAB)
    tq.gemm_dense_i8(T, VOCAB, HID, o["q2"], o["s2"], dev(head[0]), dev(head[1]), F32, o["out"])
    torch.cuda.synchronize()
    return o


def test_layer():
    import torch
    experts, router, head, norms = _weights()
    packed = [[pack(1, 0, TENSOR, t, s) for t, s in e] for e in experts]
    rng = np.random.default_rng(13)
    x, h = rng.standard_normal((T, HID)).astype(np.float32), 2 * rng.standard_normal((T, HID)).astype(np.float32)
    o = _run(x, h, packed, router, head, norms)
    v = {k: t.cpu().numpy() for k, t in o.items()}

    def norm(x, h, w, q, s, out):
        hs, ns = ref.norm_steps(x, h, w, EPS)
        rq, rs = ref.quant_steps(ns)
        assert np.array_equal(out, hs) and np.array_equal(q, rq) and np.array_equal(s, rs)

    norm(v["x"], v["h0"], norms[0], v["q"], v["s"], v["h"])
    assert np.array_equal(v["logits"], ref.dense_i8(v["q"], v["s"], *router))
    rows, pairs, offs = ref.dispatch(v["ids"], E)
    assert np.array_equal(v["rows"], rows) and np.array_equal(v["pairs"], pairs) and np.array_equal(v["offs"], offs)
    assert offs[E] == (T - 2) * TOP
    used = pairs[:offs[E]] // TOP
    assert np.array_equal(v["xs"][:offs[E]], v["q"][used]) and np.array_equal(v["xss"][:offs[E]], v["s"][used])
    for name, p, src, sc in (("gate", 0, "xs", "xss"), ("up", 1, "xs", "xss"), ("down", 2, "aq", "as")):
        for e in range(E):
            a, b = offs[e], offs[e + 1]
            if a < b:
                y = oracle.gemv_i8(1, 0, TENSOR, *experts[e][p], v[src][a:b], v[sc][a:b])["y32"]
                assert np.array_equal(v[name][a:b], y), (name, e)
    y, mag = ref.combine(rows, v["w"], v["down"])
    assert np.all(np.abs(v["moe"] - y) <= 1.001 * (TOP + 1) * ref.U24 * mag)
    assert np.all(v["moe"][T - 2:] == 0.0)                         # padding: the residual alone goes on
    norm(v["moe"], v["h"], norms[1], v["q2"], v["s2"], v["h2"])
    assert np.array_equal(v["out"], ref.dense_i8(v["q2"], v["s2"], *head))
    again = _run(x, h, packed, router, head, norms)
    for k in o:
        assert torch.equal(o[k], again[k]), k
