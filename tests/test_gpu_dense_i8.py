"""tq_gemm_dense_i8 against exact integer sums: equal bits everywhere."""
from __future__ import annotations

import numpy as np
import pytest

from oracle import BF16, F32
from tests import operator_ref as ref

pytestmark = pytest.mark.gpu


def _torch():
    import torch
    return torch


def _inputs(M, N, K, seed=0, extremes=False):
    rng = np.random.default_rng(M + 31 * N + 977 * K + seed)
    if extremes:
        xq, wq = rng.choice([-128, 127], (M, K)).astype(np.int8), rng.choice([-128, 127], (N, K)).astype(np.int8)
        xq[0], wq[0] = -128, -128
    else:
        xq, wq = rng.integers(-128, 128, (M, K)).astype(np.int8), rng.integers(-128, 128, (N, K)).astype(np.int8)
    xs = rng.uniform(1e-3, 1e-1, M).astype(np.float32)
    ws = rng.uniform(-1e-2, 1e-2, N).astype(np.float32)
    return xq, xs, wq, ws


def run(M, N, K, yt, xq, xs, wq, ws, offset=0):
    """y inside a larger buffer, `offset` elements past an aligned address."""
    from ternary_weight_amd import tq
    torch = _torch()
    dt = torch.float32 if yt == F32 else torch.bfloat16
    whole = torch.full((64 + offset + M * N + 4096,), 99.0, dtype=dt, device="cuda")
    y = whole[64 + offset:64 + offset + M * N].view(M, N)
    d = [torch.from_numpy(a).cuda() for a in (xq, xs, wq, ws)]
    print("dense", M, N, K, yt, offset, flush=True)
    tq.gemm_dense_i8(M, N, K, d[0], d[1], d[2], d[3], yt, y)
    torch.cuda.synchronize()
    w = whole.float().cpu().numpy()
    assert np.all(w[:64 + offset] == 99.0) and np.all(w[64 + offset + M * N:] == 99.0)
    return y.float().cpu().numpy()


def check(M, N, K, yt, offset=0, **kw):
    xq, xs, wq, ws = _inputs(M, N, K, **kw)
    y, want = run(M, N, K, yt, xq, xs, wq, ws, offset), ref.dense_i8(xq, xs, wq, ws)
    assert np.array_equal(y, want if yt == F32 else ref.bf16(want)), (M, N, K, yt)


@pytest.mark.parametrize("M", [1, 2, 3, 4, 5, 7, 8, 9, 13, 15, 16, 17, 24, 31, 32, 33, 48, 63, 64, 65, 100, 127, 128,
                               129, 200, 255, 256, 257, 300, 512, 700])
def test_token_counts(M):
    check(M, 333, 592, F32)
    check(M, 640, 2560, BF16)


@pytest.mark.parametrize("N", [1, 2, 3, 15, 16, 17, 31, 33, 63, 64, 65, 127, 128, 129, 191, 255, 256, 257, 513, 1000, 5003])
def test_output_counts(N):
    for M in (1, 6, 40, 130, 270):
        check(M, N, 320, F32)
    check(3, N, 1040, BF16)
    check(150, N, 1040, BF16)


@pytest.mark.parametrize("K", [16, 32, 48, 64, 80, 112, 128, 144, 192, 240, 256, 272, 496, 512, 528, 1008, 1024, 1040,
                               4096, 6912, 14336, 65536])
def test_depths(K):
    for M, N in ((1, 130), (5, 65), (20, 200), (65, 129), (260, 300)):
        check(M, N, K, F32, extremes=True)


@pytest.mark.parametrize("M,N", [(1, 7), (4, 64), (16, 130), (70, 66), (300, 258)])
def test_unaligned_outputs(M, N):
    for offset in (1, 2, 3):
        check(M, N, 256, F32, offset)
    check(M, N, 256, BF16, 2)


def test_no_depth():
    y = run(3, 5, 0, F32, np.zeros((3, 0), np.int8), np.ones(3, np.float32), np.zeros((5, 0), np.int8),
            np.ones(5, np.float32))
    assert np.all(y == 0.0)


@pytest.mark.parametrize("M,N,K,yt", [(2048, 6912, 2560, F32), (1111, 4096, 4112, BF16), (1, 128256, 2560, F32),
                                      (16, 14336, 4096, F32), (4096, 128, 2048, F32)])
def test_large(M, N, K, yt):
    """Large shapes, sampled rows and columns."""
    from ternary_weight_amd import tq
    torch = _torch()
    g = torch.Generator(device="cuda").manual_seed(M)
    xq = torch.randint(-128, 128, (M, K), generator=g, device="cuda", dtype=torch.int8)
    wq = torch.randint(-128, 128, (N, K), generator=g, device="cuda", dtype=torch.int8)
    xs, ws = torch.rand(M, device="cuda", generator=g), torch.rand(N, device="cuda", generator=g)
    y = torch.empty(M, N, dtype=torch.float32 if yt == F32 else torch.bfloat16, device="cuda")
    tq.gemm_dense_i8(M, N, K, xq, xs, wq, ws, yt, y)
    acc = xq.double() @ wq.double().t()                       # exact below 2^53
    want = acc.float() * (xs[:, None] * ws[None, :])
    assert torch.equal(y, want.to(y.dtype))


# Products of the middle sizes and of the large ones that the wider tiles take, none of whose edges is whole: tokens,
# outputs and columns of every remainder of a tile (Kin mod 256: 16 .. 240, and 0)
EDGES = [(700, 1001, 3312), (300, 4097, 2320), (200, 5002, 4448), (300, 2563, 1856), (257, 7001, 2016), (513, 4097, 896),
         (700, 5002, 304), (2050, 4097, 3584), (1500, 9999, 752), (1025, 9999, 1280), (1500, 7001, 3808), (1025, 9999, 3152),
         (1500, 9999, 1568), (1025, 12001, 4480), (1281, 10001, 1152), (1300, 10002, 1040), (1537, 9001, 1936),
         (257, 2049, 2720), (70, 5002, 704), (130, 1001, 2672), (1023, 9985, 16), (1025, 9987, 176),
         (200, 30001, 960), (385, 9999, 2128), (450, 12001, 1616), (1025, 7001, 1568), (2050, 2563, 496), (70, 7001, 6816),
         (200, 2563, 7280), (450, 1001, 7504), (130, 4097, 3040), (200, 9999, 2576), (257, 7001, 4000), (700, 4097, 1520),
         (257, 30001, 4656), (700, 12001, 672),
         (130, 5002, 928), (385, 9999, 1360), (385, 12001, 2464), (300, 5002, 6480), (161, 5002, 1680),
         (90, 5002, 2464), (300, 2047, 7008), (257, 7001, 4240), (130, 2563, 2112), (200, 12001, 1680),
         (200, 7001, 3792), (90, 4097, 2592), (33, 9999, 5216), (97, 9999, 2352), (90, 5003, 3664),
         (257, 2047, 6960), (130, 2047, 2800), (90, 5002, 3856), (200, 5003, 1344), (450, 2047, 2496),
         (97, 9999, 2480), (300, 5002, 4768), (33, 12001, 4112), (130, 5003, 384), (1025, 12001, 704),
         (1500, 7001, 1344), (1025, 12001, 304), (1025, 9999, 784), (1025, 9999, 1184), (1500, 9999, 160)]


@pytest.mark.parametrize("M,N,K", EDGES)
def test_tiles_with_edges(M, N, K):
    from ternary_weight_amd import tq
    torch = _torch()
    g = torch.Generator(device="cuda").manual_seed(K)
    xq = torch.randint(-128, 128, (M, K), generator=g, device="cuda", dtype=torch.int8)
    wq = torch.randint(-128, 128, (N, K), generator=g, device="cuda", dtype=torch.int8)
    xs, ws = torch.rand(M, device="cuda", generator=g), torch.rand(N, device="cuda", generator=g) - 0.5
    want = (xq.double() @ wq.double().t()).float() * (xs[:, None] * ws[None, :])
    for yt, dt in ((F32, torch.float32), (BF16, torch.bfloat16)):
        whole = torch.full((64 + M * N + 4096,), 99.0, dtype=dt, device="cuda")
        print("edges", M, N, K, yt, flush=True)
        tq.gemm_dense_i8(M, N, K, xq, xs, wq, ws, yt, whole[64:64 + M * N])
        assert torch.equal(whole[64:64 + M * N].view(M, N), want.to(dt))
        assert torch.all(whole[:64] == 99.0) and torch.all(whole[64 + M * N:] == 99.0)


def test_weight_beyond_32_bit_offsets():
    """A weight of more than 4 GiB: its last rows."""
    from ternary_weight_amd import tq
    torch = _torch()
    M, N, K = 3, 70000, 65536
    g = torch.Generator(device="cuda").manual_seed(1)
    wq = torch.zeros(N, K, dtype=torch.int8, device="cuda")
    some = [0, 1, 32767, 32768, 65535, 65536, 69999]
    rows = torch.randint(-128, 128, (len(some), K), generator=g, device="cuda", dtype=torch.int8)
    wq[some] = rows
    xq = torch.randint(-128, 128, (M, K), generator=g, device="cuda", dtype=torch.int8)
    xs, ws, y = torch.ones(M, device="cuda"), torch.ones(N, device="cuda"), torch.empty(M, N, device="cuda")
    tq.gemm_dense_i8(M, N, K, xq, xs, wq, ws, F32, y)
    want = torch.zeros(M, N, device="cuda")
    want[:, some] = (xq.double() @ rows.double().t()).float()
    assert torch.equal(y, want)


def test_output_beyond_32_bit_offsets():
    """An output of more than 4 GiB."""
    from ternary_weight_amd import tq
    torch = _torch()
    M, N, K = 9000, 120001, 16
    g = torch.Generator(device="cuda").manual_seed(2)
    xq = torch.randint(-128, 128, (M, K), generator=g, device="cuda", dtype=torch.int8)
    wq = torch.randint(-128, 128, (N, K), generator=g, device="cuda", dtype=torch.int8)
    xs, ws = torch.rand(M, device="cuda", generator=g), torch.rand(N, device="cuda", generator=g)
    y = torch.empty(M, N, device="cuda")
    tq.gemm_dense_i8(M, N, K, xq, xs, wq, ws, F32, y)
    for m in (0, 4473, 4474, 8947, 8948, M - 1):
        acc = xq[m:m + 1].double() @ wq.double().t()
        assert torch.equal(y[m:m + 1], acc.float() * (xs[m] * ws[None, :]))


def test_graph_and_streams():
    from ternary_weight_amd import tq
    torch = _torch()
    side = torch.cuda.Stream()
    for M, N, K in ((1, 640, 2560), (40, 640, 2560), (300, 1030, 2560)):
        xq, xs, wq, ws = [torch.from_numpy(a).cuda() for a in _inputs(M, N, K)]
        y, z = torch.empty(M, N, device="cuda"), torch.empty(M, N, device="cuda")
        call = lambda out: tq.gemm_dense_i8(M, N, K, xq, xs, wq, ws, F32, out)
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            call(y)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            call(y)
        for k in range(3):
            xq.copy_(torch.from_numpy(_inputs(M, N, K, seed=k + 1)[0]))
            y.zero_()
            graph.replay()
            call(z)
            torch.cuda.synchronize()
            want = ref.dense_i8(xq.cpu().numpy(), xs.cpu().numpy(), wq.cpu().numpy(), ws.cpu().numpy())
            assert np.array_equal(y.cpu().numpy(), want) and torch.equal(y, z)
