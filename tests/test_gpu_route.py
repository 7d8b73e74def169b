"""The router and the grouping of rows on the GPU against their references: selections
and orders exactly, weights within the bound of their arithmetic."""
import numpy as np
import pytest
import torch

import block_scaled_gemm_fp8gemm_amd as F
from oracle import layers as L

from gpu_support import DEV, announce

pytestmark = pytest.mark.gpu

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def _check(logits, k, scoring, renormalize, scale=1.0, sample=None):
    ids, w = F.moe_route(logits, k, scoring, renormalize, scale)
    torch.cuda.synchronize()
    host = logits.double().cpu().numpy()
    rows = slice(None) if sample is None else sample
    want_ids, want_w = L.route_reference(host[rows], k, scoring, renormalize, scale)
    got_ids, got_w = ids.cpu().numpy()[rows], w.cpu().numpy()[rows].astype(np.float64)
    assert np.array_equal(got_ids, want_ids)
    assert np.all(np.abs(got_w - want_w) <= L.route_tolerance(host[rows], want_w, k))
    return ids, w


@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 8, 2), (3, 5, 5), (7, 8, 8), (33, 16, 16),
                                   (5, 17, 4), (65, 32, 1), (9, 60, 4), (130, 64, 8), (4, 65, 6),
                                   (17, 128, 8), (12, 200, 16), (6, 256, 8), (3, 257, 9),
                                   (5, 512, 10), (2, 1000, 16), (2, 1024, 16)])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_route_shapes(T, E, k, dtype):
    g = torch.Generator().manual_seed(T * 1000 + E)
    logits = (2 * torch.randn(T, E, generator=g)).to(DTYPES[dtype]).to(DEV)
    for scoring in ("softmax", "sigmoid"):
        for renormalize in (True, False):
            announce("route", (T, E, k), dtype, scoring, renormalize)
            _check(logits, k, scoring, renormalize, 2.5)


def test_route_many_rows():
    g = torch.Generator().manual_seed(5)
    logits = torch.randn(20001, 48, generator=g).bfloat16().to(DEV)
    announce("route many rows")
    _check(logits, 6, "softmax", True, sample=list(range(0, 20001, 97)) + [20000])


def test_route_ties_take_the_lowest_expert():
    for E, k in ((8, 3), (64, 8), (256, 8), (1024, 16)):
        announce("route ties", (E, k))
        equal = torch.zeros(5, E, device=DEV)
        ids, w = _check(equal, k, "softmax", True)
        assert ids[0].tolist() == list(range(k))
        # few distinct values, and zeros of both signs
        g = torch.Generator().manual_seed(E)
        l = torch.randint(-1, 2, (40, E), generator=g).float()
        l = torch.where(l == 0, torch.where(torch.rand(40, E, generator=g) < 0.5, 0.0, -0.0), l)
        _check(l.to(DEV), k, "sigmoid", True)


@pytest.mark.parametrize("E,k", [(8, 4), (40, 6), (300, 8)])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_route_masks_and_extremes(E, k, dtype):
    dt = DTYPES[dtype]
    low, inf, nan = torch.finfo(dt).min, float("inf"), float("nan")
    g = torch.Generator().manual_seed(E)
    l = torch.randn(12, E, generator=g).to(dt)
    l[0] = -inf                                   # nothing left
    l[1] = nan
    l[2] = -inf
    l[2, E - 1] = 1.0                             # one left
    l[3, 1:] = nan
    l[4] = low                                    # the type's lowest value is a logit
    l[5, : E // 2] = low
    l[6, 2] = inf
    l[7, [1, 4, 6]] = inf
    l[8] = inf
    l[9] = -inf
    l[9, [0, 5]] = low
    l[10] = torch.finfo(dt).max
    l[11] = -200.0                                # every sigmoid underflows fp32
    l[11, 3] = -150.0
    for scoring in ("softmax", "sigmoid"):
        for renormalize in (True, False):
            announce("route masks", (E, k), dtype, scoring, renormalize)
            ids, w = _check(l.to(DEV), k, scoring, renormalize)
            assert bool(torch.isfinite(w).all())
            assert ids[0].tolist() == [-1] * k and not w[0].any()


def test_route_strided_rows_and_given_outputs():
    g = torch.Generator().manual_seed(2)
    wide = torch.randn(10, 100, generator=g).to(DEV)
    ids = torch.full((10, 4), 77, dtype=torch.int32, device=DEV)
    w = torch.full((10, 4), 77.0, device=DEV)
    announce("route strided")
    got = F.moe_route(wide[:, 3:64], 4, ids=ids, weights=w)
    assert got[0] is ids and got[1] is w
    want, want_w = L.route_reference(wide[:, 3:64].double().cpu().numpy(), 4, "softmax", True)
    assert np.array_equal(ids.cpu().numpy(), want)
    odd = torch.randn(7, 33, generator=g).half().to(DEV)[:, 1:]       # rows 2-byte aligned
    _check(odd, 3, "softmax", False)
    _check(wide[4:5, 10:30], 3, "softmax", True)
    empty = F.moe_route(wide[:0], 4)
    assert empty[0].shape == (0, 4)


@pytest.mark.parametrize("n,G", [(1, 1), (1, 1024), (5, 3), (63, 8), (64, 8), (65, 32), (200, 1), (4096, 9), (4097, 9), (65536, 300), (65537, 300),
                                 (1024, 16), (1025, 1024), (5000, 7), (16384, 64), (16385, 64),
                                 (20000, 1024), (70001, 256), (300000, 5)])
@pytest.mark.parametrize("kind", ["uniform", "skewed", "dropped", "none"])
def test_group_rows(n, G, kind):
    g = torch.Generator().manual_seed(n + G)
    ids = torch.randint(0, G, (n,), generator=g)
    if kind == "skewed":
        ids = (torch.rand(n, generator=g) ** 4 * G).long()
    if kind == "dropped":
        bad = torch.rand(n, generator=g) < 0.4
        ids[bad] = torch.tensor([-1, G, 2 ** 31 - 1, -2 ** 31])[
            torch.randint(0, 4, (int(bad.sum()),), generator=g)]
    if kind == "none":
        ids[:] = -5
    announce("group", n, G, kind)
    order, offsets = F.group_rows(ids.to(torch.int32).to(DEV), G)
    key = torch.where((ids >= 0) & (ids < G), ids, G)
    want = torch.sort(key, stable=True).indices
    counts = torch.bincount(key, minlength=G + 1)[:G]
    assert torch.equal(order.cpu().long(), want)
    assert offsets.cpu().tolist() == [0] + torch.cumsum(counts, 0).tolist()
    if n <= 5000:
        ref_order, ref_offsets = L.group_reference(ids.numpy(), G) if G <= 64 else (want, None)
        assert np.array_equal(order.cpu().numpy(), np.asarray(ref_order))


def test_group_rows_of_nothing():
    announce("group nothing")
    order, offsets = F.group_rows(torch.empty(0, dtype=torch.int32, device=DEV), 40)
    assert order.numel() == 0 and offsets.cpu().tolist() == [0] * 41


def test_route_and_group_captured():
    """One graph, replayed under new logits with eager work in between."""
    T, E, k = 300, 64, 8
    logits = torch.empty(T, E, device=DEV)
    ids = torch.empty(T, k, dtype=torch.int32, device=DEV)
    w = torch.empty(T, k, device=DEV)
    order = torch.empty(T * k, dtype=torch.int32, device=DEV)
    offsets = torch.empty(E + 1, dtype=torch.int32, device=DEV)

    def step():
        F.moe_route(logits, k, ids=ids, weights=w)
        F.group_rows(ids, E, order=order, offsets=offsets)

    logits.normal_()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    announce("route + group captured")
    with torch.cuda.graph(graph):
        step()
    for i in range(4):
        logits.copy_(torch.randn(T, E, generator=torch.Generator().manual_seed(i)))
        eager = F.moe_route(logits, k) + F.group_rows(F.moe_route(logits, k)[0], E)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip((ids, w, order, offsets), eager):
            assert torch.equal(a, b)
