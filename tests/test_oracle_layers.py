"""Pins of the serving operators' references: hand-worked values, closed forms, torch's
float64 operations, and planted mistakes that the bounds catch."""
import numpy as np
import pytest
import torch

import oracle as O
from oracle import layers as L
from oracle import quant as Q


def test_route_hand_worked():
    l = [[1.0, 3.0, 3.0, 2.0], [-np.inf, 0.0, -np.inf, np.nan], [-np.inf] * 4,
         [np.inf, 1.0, np.inf, 0.0]]
    ids, w = L.route_reference(l, 2, "softmax", True)
    assert ids.tolist() == [[1, 2], [1, -1], [-1, -1], [0, 2]]
    assert w.tolist() == [[0.5, 0.5], [1.0, 0.0], [0.0, 0.0], [0.5, 0.5]]
    ids, w = L.route_reference([[0.0, np.log(3.0)]], 1, "softmax", False, scale=2.0)
    assert ids.tolist() == [[1]] and w[0, 0] == pytest.approx(1.5)
    _, w = L.route_reference([[0.0, np.log(3.0)]], 2, "sigmoid", False)
    assert w[0].tolist() == pytest.approx([0.75, 0.5])


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [True, False])
def test_route_against_torch(scoring, renormalize):
    l = torch.randn(50, 33, dtype=torch.float64, generator=torch.Generator().manual_seed(1))
    p = torch.softmax(l, 1) if scoring == "softmax" else torch.sigmoid(l)
    top, idx = torch.topk(p, 5, dim=1)
    if renormalize:
        top = top / top.sum(1, keepdim=True)
    ids, w = L.route_reference(l.numpy(), 5, scoring, renormalize)
    assert np.array_equal(ids, idx.numpy())
    np.testing.assert_allclose(w, top.numpy(), rtol=1e-12)


def test_group_hand_worked():
    order, offsets = L.group_reference([2, 0, -1, 2, 7, 0], 3)
    assert order.tolist() == [1, 5, 0, 3, 2, 4] and offsets.tolist() == [0, 2, 2, 4]


def _experts(rng, E, N, K, mode, fmt):
    qs, ss = [], []
    for _ in range(E):
        q, s = Q.quantize((rng.standard_normal((N, K)) * 0.1).astype(np.float32), mode, fmt)
        qs.append(O.pack_fp4(q) if fmt == "e2m1" else q)
        ss.append(s)
    return np.stack(qs), np.stack(ss)


@pytest.mark.parametrize("mode,fmt", [("tensor", "e4m3"), ("rowwise", "e4m3"), ("mx32", "e4m3"),
                                      ("mx32", "e2m1")])
def test_moe_against_the_definition(mode, fmt):
    rng = np.random.default_rng(3)
    E, T, H, I, k = 3, 4, 64, 32, 2
    q13, s13 = _experts(rng, E, 2 * I, H, mode, fmt)
    q2, s2 = _experts(rng, E, H, I, mode, fmt)
    x = rng.standard_normal((T, H))
    ids = np.array([[0, 2], [1, 1], [-1, 5], [2, -3]], np.int32)
    w = rng.random((T, k))
    y, tol = L.moe_reference(x, ids, w, q13, s13, q2, s2, mode, fmt, "silu", "bf16")

    def dq(q, s, e):
        c = O.unpack_fp4(q[e]) if fmt == "e2m1" else q[e]
        v = O.decode(c, fmt)
        if mode == "mx32":
            return v * np.repeat(2.0 ** (s[e].astype(float) - 127), 32, axis=1)
        return v * np.asarray(s[e], np.float64).reshape(-1, 1)

    want = np.zeros((T, H))
    for t in range(T):
        for j in range(k):
            e = ids[t, j]
            if 0 <= e < E:
                g, u = np.split(dq(q13, s13, e) @ x[t], 2)
                want[t] += w[t, j] * (dq(q2, s2, e) @ (g / (1 + np.exp(-g)) * u))
    np.testing.assert_allclose(y, want, rtol=1e-12, atol=1e-13)
    assert not y[2].any()
    # planted mistakes are outside the bound: gate and up swapped, a slot's weight lost
    half = np.concatenate([q13[:, I:], q13[:, :I]], axis=1)
    s_half = s13 if mode == "tensor" else np.concatenate([s13[:, I:], s13[:, :I]], axis=1)
    bad, _ = L.moe_reference(x, ids, w, half, s_half, q2, s2, mode, fmt, "silu", "bf16")
    assert (np.abs(bad - y) > tol)[[0, 1, 3]].any()
    bad, _ = L.moe_reference(x, ids, np.ones_like(w), q13, s13, q2, s2, mode, fmt, "silu", "bf16")
    assert (np.abs(bad - y) > tol)[[0, 1, 3]].any(axis=1).all()


def test_lora_against_the_definition():
    rng = np.random.default_rng(4)
    M, N, K, r, G = 6, 10, 24, 8, 2
    x, base = rng.standard_normal((M, K)), rng.standard_normal((M, N))
    a, b = rng.standard_normal((G, r, K)), rng.standard_normal((G, N, r))
    s = np.array([0.5, 2.0])
    rows = np.array([0, 1, -1, 1, 9, 0])
    y, tol = L.lora_reference(x, base, a, b, rows, s, "none", "bf16")
    for m in range(M):
        d = s[rows[m]] * b[rows[m]] @ (a[rows[m]] @ x[m]) if rows[m] in (0, 1) else 0.0
        np.testing.assert_allclose(y[m], base[m] + d, rtol=1e-12)
    z, _ = L.lora_reference(x, base, a, b, rows, s, "silu", "bf16")
    np.testing.assert_allclose(z, y / (1 + np.exp(-y)), rtol=1e-12)
    bad, _ = L.lora_reference(x, base, a, b, rows, None, "none", "bf16")      # scales lost
    assert (np.abs(bad - y) > tol)[[0, 1, 3, 5]].any(axis=1).all()
    bad, _ = L.lora_reference(x, base, a, b, 1 - rows, s, "none", "bf16")     # wrong adapter
    assert (np.abs(bad - y) > tol)[[0, 1, 3, 5]].any(axis=1).all()
