"""Low-rank adapters beside a projection on the GPU against the float64 reference."""
import numpy as np
import pytest
import torch

import block_scaled_gemm_fp8gemm_amd as F
from oracle import layers as L

from gpu_support import DEV, announce, to_host

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f16": torch.float16}


def _inputs(M, K, N, r, G, dtype, seed, rows=None):
    g = torch.Generator().manual_seed(seed)
    dt = DT[dtype]
    x = torch.randn(M, K, generator=g).to(dt)
    base = torch.randn(M, N, generator=g).to(dt)
    a = (torch.randn(G, r, K, generator=g) / K ** 0.5).to(dt)
    b = (torch.randn(G, N, r, generator=g) * 0.3).to(dt)
    s = torch.rand(G, generator=g) + 0.5
    if rows is None:
        rows = torch.randint(-1, G, (M,), generator=g)
    return x, base, a, b, s, rows.to(torch.int32)


def _padded(t, pad):
    """t on the device with `pad` extra columns (NaN) between its rows."""
    cols = (t.shape[-1] + 7) // 8 * 8 + pad
    buf = torch.full((*t.shape[:-1], cols), float("nan"), dtype=t.dtype, device=DEV)
    buf[..., :t.shape[-1]] = t.to(DEV)
    return buf[..., :t.shape[-1]]


def _check(x, base, a, b, s, rows, act="none", pad=0, out=None, in_place=False):
    M, K = x.shape
    dtype = "bf16" if x.dtype == torch.bfloat16 else "f16"
    announce("lora", dtype, act, (M, K, base.shape[1], a.shape[1], a.shape[0]))
    order, offsets = F.group_rows(rows.to(DEV), a.shape[0])
    based = _padded(base, pad)
    got = F.lora(_padded(x, pad), based, _padded(a, pad), _padded(b, pad), order, offsets,
                 None if s is None else s.to(DEV), act, out=based if in_place else out)
    torch.cuda.synchronize()
    want, tol = L.lora_reference(x.double().numpy(), base.double().numpy(), a.double().numpy(),
                                 b.double().numpy(), rows.numpy(),
                                 None if s is None else s.double().numpy(), act, dtype)
    err = np.abs(to_host(got) - want)
    assert np.all(err <= tol), (float((err - tol).max()), np.argwhere(err > tol)[:3])
    return got


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("M,K,N,r,G", [(1, 64, 64, 8, 1), (1, 256, 100, 16, 4), (2, 8, 1, 8, 2),
                                       (16, 128, 256, 16, 2), (17, 136, 257, 24, 3),
                                       (33, 512, 300, 32, 33), (64, 520, 63, 40, 7),
                                       (100, 96, 513, 64, 5), (130, 72, 72, 72, 130),
                                       (200, 264, 1000, 128, 9), (333, 200, 77, 104, 1)])
def test_shapes(M, K, N, r, G, dtype):
    args = _inputs(M, K, N, r, G, dtype, M + K + N)
    _check(*args)
    _check(*args[:4], None, args[5], pad=8)


@pytest.mark.parametrize("act", ["none", "relu", "gelu", "silu"])
def test_activations(act):
    for dtype in ("bf16", "f16"):
        _check(*_inputs(40, 128, 120, 16, 4, dtype, 3), act)


def test_rows_of_one_adapter_and_of_none():
    for M in (1, 31, 32, 33, 129):
        x, base, a, b, s, _ = _inputs(M, 96, 200, 16, 6, "bf16", M)
        _check(x, base, a, b, s, torch.full((M,), 3, dtype=torch.int32))
        none = torch.full((M,), -1, dtype=torch.int32)
        got = _check(x, base, a, b, s, none)
        assert torch.equal(got.cpu(), base)


def test_long_runs_and_many_adapters():
    rows = torch.arange(1500) // 400
    _check(*_inputs(1500, 128, 192, 32, 4, "bf16", 5, rows))
    rows = torch.randint(0, 1024, (600,), generator=torch.Generator().manual_seed(1))
    _check(*_inputs(600, 64, 72, 8, 1024, "f16", 6, rows))


def test_long_rows():
    _check(*_inputs(3, 4096, 520, 16, 2, "bf16", 7))
    _check(*_inputs(40, 8200, 64, 32, 2, "f16", 8))


def test_in_place_and_canaries():
    x, base, a, b, s, rows = _inputs(45, 128, 100, 16, 4, "bf16", 9)
    want = _check(x, base, a, b, s, rows)
    got = _check(x, base, a, b, s, rows, pad=16, in_place=True)
    assert torch.equal(got, want)
    buf = torch.full((47, 120), 7.0, dtype=torch.bfloat16, device=DEV)
    got = _check(x, base, a, b, s, rows, out=buf[1:46, :100])
    assert torch.equal(got, want)
    assert bool((buf[0] == 7).all()) and bool((buf[46] == 7).all())
    assert bool((buf[:, 100:] == 7).all())


def test_values_beyond_f16_between_the_products():
    """x A^T past f16's largest value and below its smallest, with B bringing it back."""
    x, base, a, b, s, rows = _inputs(20, 256, 64, 16, 2, "f16", 11)
    _check(x * 100, base, (a.float() * 400).half(), (b.float() * 2 ** -14).half(), s, rows)
    _check((x.float() * 2 ** -8).half(), base, (a.float() * 2 ** -8).half(),
           (b.float() * 2000).half(), s, rows)
    zero = torch.zeros_like(x)
    got = _check(zero, base, a, b, s, rows)
    assert torch.equal(got.cpu(), base)


def test_other_adapters_are_not_read():
    """NaN in the adapters that no row names."""
    x, base, a, b, s, rows = _inputs(50, 64, 90, 16, 6, "bf16", 13)
    rows[rows == 2] = 1
    a[2], b[2], s[2] = float("nan"), float("nan"), float("nan")
    _check(x, base, a, b, s, rows)


def test_bad_plans_stay_inside_the_tensors():
    """Entries outside [0, M) and offsets that overlap or leave [0, M]: the host and the
    kernels' own checks keep every access inside, rows named rightly elsewhere are right."""
    M, G = 40, 3
    x, base, a, b, s, rows = _inputs(M, 64, 80, 16, G, "bf16", 15)
    order, offsets = F.group_rows(rows.to(DEV), G)
    args = [_padded(t, 0) for t in (x, base, a, b)]
    buf = torch.full((M + 2, 80), 7.0, dtype=torch.bfloat16, device=DEV)
    for o, f in ((order.clone().fill_(M), offsets), (order.clone().fill_(-1), offsets),
                 (order, torch.tensor([0, 1000, -5, 2 ** 31 - 1], dtype=torch.int32, device=DEV)),
                 (order, torch.tensor([-9, 30, 10, 40], dtype=torch.int32, device=DEV))):
        announce("lora bad plan", f.tolist())
        F.lora(*args, o, f, s.to(DEV), out=buf[1:M + 1])
        torch.cuda.synchronize()
        assert bool((buf[0] == 7).all()) and bool((buf[M + 1] == 7).all())
    bad = order.clone()
    bad[5] = M + 3                                    # one entry lost, the others in place
    buf[1:M + 1] = 7.0
    F.lora(*args, bad, offsets, s.to(DEV), out=buf[1:M + 1])
    good = F.lora(*args, order, offsets, s.to(DEV))
    keep = torch.ones(M, dtype=torch.bool, device=DEV)
    keep[order[5].long()] = False
    assert torch.equal(buf[1:M + 1][keep], good[keep]) and bool((buf[1:M + 1][~keep] == 7).all())


def test_deterministic_empty_and_captured():
    x, base, a, b, s, rows = _inputs(37, 1024, 128, 16, 5, "bf16", 17)
    first = _check(x, base, a, b, s, rows)
    assert torch.equal(first, _check(x, base, a, b, s, rows))
    d = [t.to(DEV) for t in (x, base, a, b)]
    none, zero = F.group_rows(rows[:0].to(DEV), 5)
    assert F.lora(d[0][:0], d[1][:0], d[2], d[3], none, zero).shape == (0, 128)
    order, offsets = F.group_rows(rows.to(DEV), 5)
    out = torch.empty_like(d[1])
    ws = torch.zeros(F.fp8gemm_lora_workspace_size(37, 1024, 16, 5), dtype=torch.uint8, device=DEV)

    def step():
        F.lora(*d, order, offsets, sd, out=out, workspace=ws)

    sd = s.to(DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    announce("lora captured")
    with torch.cuda.graph(graph):
        step()
    for i in range(4):
        g = torch.Generator().manual_seed(i)
        d[0].copy_(torch.randn(37, 1024, generator=g))
        o, f = F.group_rows(torch.randint(-1, 5, (37,), generator=g).to(torch.int32).to(DEV), 5)
        order.copy_(o)
        offsets.copy_(f)
        eager = F.lora(*d, o, f, sd)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, eager)
    assert not ws[:4096].any()


def test_refusals():
    x, base, a, b, s, rows = _inputs(10, 64, 40, 16, 2, "bf16", 19)
    order, offsets = F.group_rows(rows.to(DEV), 2)
    x, base, a, b = (t.to(DEV) for t in (x, base, a, b))
    with pytest.raises(ValueError, match="dtype"):
        F.lora(x, base.half(), a, b, order, offsets)
    with pytest.raises(ValueError, match="shape"):
        F.lora(x, base, a, b[:, :39], order, offsets)
    with pytest.raises(ValueError, match="shape"):
        F.lora(x, base, a, b, order, offsets[:2])
    with pytest.raises(ValueError, match="unit stride"):
        F.lora(x, base, a.transpose(1, 2).contiguous().transpose(1, 2), b, order, offsets)
    with pytest.raises(F.Fp8GemmError, match="NOT_SUPPORTED"):
        F.lora(x, base, a[:, :12], b[:, :, :12], order, offsets)
    with pytest.raises(F.Fp8GemmError, match="MISALIGNED"):
        F.lora(x[:, 4:60], base, a[:, :, 4:60], b, order, offsets)
