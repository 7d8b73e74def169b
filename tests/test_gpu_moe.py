"""The few-token mixture-of-experts layer on the GPU against the float64 reference."""
import numpy as np
import pytest
import torch

import block_scaled_gemm_fp8gemm_amd as F
import oracle as O
from oracle import layers as L
from oracle import quant as Q

from gpu_support import DEV, announce, to_host

pytestmark = pytest.mark.gpu

FORMS = [("tensor", "e4m3"), ("rowwise", "e4m3"), ("mx32", "e4m3"), ("mx32", "e2m1")]
DT = {"bf16": torch.bfloat16, "f16": torch.float16}


def _quantized(rng, E, N, K, mode, fmt, std):
    qs, ss = [], []
    for _ in range(E):
        w = rng.standard_normal((N, K)) * std
        w *= np.exp2(rng.integers(-3, 4, size=(N, 1)))          # rows of different size
        q, s = Q.quantize(w.astype(np.float32), mode, fmt)
        qs.append(O.pack_fp4(q) if fmt == "e2m1" else q)
        ss.append(s)
    return np.stack(qs), np.stack(ss)


def _dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


class Layer:
    """Experts on the host and the device, and one checked call."""

    def __init__(self, H, I, E, mode, fmt, seed=0, std=0.05):
        rng = np.random.default_rng(seed)
        self.H, self.I, self.E, self.mode, self.fmt, self.rng = H, I, E, mode, fmt, rng
        self.q13, self.s13 = _quantized(rng, E, 2 * I, H, mode, fmt, std)
        self.q2, self.s2 = _quantized(rng, E, H, I, mode, fmt, std)
        self.dev = [_dev(v) for v in (self.q13, self.s13, self.q2, self.s2)]

    def inputs(self, T, k, dtype):
        x = torch.from_numpy(self.rng.standard_normal((T, self.H)).astype(np.float32)).to(DT[dtype])
        ids = np.argsort(self.rng.random((T, self.E)), axis=1)[:, :k].astype(np.int32)
        if ids.shape[1] < k:
            ids = np.pad(ids, ((0, 0), (0, k - ids.shape[1])), constant_values=-1)
        return x, ids, self.rng.random((T, k)).astype(np.float32)

    def check(self, x, ids, w, act="silu", out=None, xd=None):
        dtype = "bf16" if x.dtype == torch.bfloat16 else "f16"
        announce("moe", self.mode, self.fmt, dtype, act, (x.shape[0], self.H, self.I, self.E,
                                                          ids.shape[1]))
        got = F.moe_experts(x.to(DEV) if xd is None else xd, _dev(ids), _dev(w), *self.dev,
                            self.mode, self.fmt, act, out=out)
        torch.cuda.synchronize()
        want, tol = L.moe_reference(x.double().numpy(), ids, w, self.q13, self.s13, self.q2,
                                    self.s2, self.mode, self.fmt, act, dtype)
        err = np.abs(to_host(got) - want)
        assert np.all(err <= tol), (float((err - tol).max()), np.argwhere(err > tol)[:3])
        return got


@pytest.mark.parametrize("mode,fmt", FORMS)
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("T,H,I,E,k", [(1, 64, 64, 4, 1), (1, 256, 512, 8, 2), (2, 96, 160, 3, 3),
                                       (5, 512, 96, 8, 2), (16, 320, 288, 4, 2),
                                       (17, 64, 32, 2, 1), (40, 128, 224, 2, 1),
                                       (65, 32, 64, 1, 1), (128, 160, 96, 3, 2),
                                       (9, 544, 1056, 16, 6)])
def test_shapes(mode, fmt, dtype, T, H, I, E, k):
    layer = Layer(H, I, E, mode, fmt, seed=T + H + I)
    layer.check(*layer.inputs(T, k, dtype))


@pytest.mark.parametrize("mode", ["tensor", "rowwise"])
def test_sizes_of_sixteen(mode):
    """H and I that are multiples of 16 and of nothing larger."""
    for H, I in ((16, 16), (48, 80), (272, 528), (1040, 16), (16, 1040)):
        layer = Layer(H, I, 3, mode, "e4m3", seed=H + I)
        layer.check(*layer.inputs(6, 2, "bf16"))


@pytest.mark.parametrize("mode,fmt", FORMS)
def test_long_rows(mode, fmt):
    layer = Layer(2080, 4128, 2, mode, fmt, seed=1, std=0.02)
    layer.check(*layer.inputs(3, 1, "bf16"))
    layer.check(*layer.inputs(20, 2, "f16"))


@pytest.mark.parametrize("act", ["none", "relu", "gelu", "silu"])
def test_activations(act):
    layer = Layer(128, 128, 4, "rowwise", "e4m3", seed=7, std=0.3)
    for dtype in ("bf16", "f16"):
        layer.check(*layer.inputs(10, 2, dtype), act)


def test_ids_that_name_no_expert_and_repeated_ones():
    layer = Layer(160, 192, 5, "mx32", "e4m3", seed=9)
    x, ids, w = layer.inputs(12, 3, "bf16")
    ids[0] = -1                                       # a token without experts
    ids[1] = [5, 2 ** 31 - 1, -2 ** 31]
    ids[2] = [3, 3, 3]                                # one expert in every slot
    ids[3, 1] = -1
    w[4] = 0.0
    got = layer.check(x, ids, w)
    assert not got[0].any() and not got[1].any()
    ids[:] = -1                                       # nobody
    got = layer.check(x, ids, w)
    assert not got.any()


def test_one_expert_takes_every_token():
    layer = Layer(96, 128, 6, "rowwise", "e4m3", seed=11)
    for T in (15, 16, 33, 64, 100, 128):
        x, ids, w = layer.inputs(T, 1, "bf16")
        ids[:] = 4
        layer.check(x, ids, w)


def test_many_experts():
    layer = Layer(64, 32, 1024, "tensor", "e4m3", seed=13)
    x, ids, w = layer.inputs(128, 16, "bf16")
    layer.check(x, ids, w)
    ids[:] = 1023
    layer.check(x[:2], ids[:2, :1], w[:2, :1])


def test_strides_canaries_and_unused_experts():
    """Padded rows of x, out and the weights, experts apart, and a NaN in all that no
    token selects (rows past the tensors, other experts, x's padding)."""
    H, I, E, T, k = 144, 176, 6, 11, 2
    layer = Layer(H, I, E, "rowwise", "e4m3", seed=15)
    x, ids, w = layer.inputs(T, k, "bf16")
    ids[ids == 2] = 0                                 # expert 2 is unused
    ids[ids == 5] = 1
    nan8 = 0x7F

    def spread(q, rows, cols, extra_rows, pitch):
        buf = torch.full((E, rows + extra_rows, pitch), nan8, dtype=torch.uint8, device=DEV)
        buf[:, :rows, :cols] = _dev(q)
        buf[[2, 5]] = nan8
        return buf[:, :rows, :cols]

    q13, q2 = spread(layer.q13, 2 * I, H, 3, 160), spread(layer.q2, H, I, 1, 256)
    s13, s2 = layer.dev[1].clone(), layer.dev[3].clone()
    s13.view(E, -1)[[2, 5]] = float("nan")
    layer.dev = [q13, s13, q2, s2]
    xp = torch.full((T + 1, 192), float("nan"), dtype=torch.bfloat16, device=DEV)
    xp[:T, :H] = x.to(DEV)
    outp = torch.full((T + 2, 152), 7.0, dtype=torch.bfloat16, device=DEV)
    layer.check(x, ids, w, out=outp[1:T + 1, :H], xd=xp[:T, :H])
    assert bool((outp[0] == 7).all()) and bool((outp[T + 1] == 7).all())
    assert bool((outp[:, H:] == 7).all())


def test_mx_scales_over_the_range():
    """Block exponents from the smallest used to large ones in one matrix: bf16 activations
    and f16 ones carried as two bf16 both keep them."""
    H, I, E = 128, 64, 2
    for fmt in ("e4m3", "e2m1"):
        layer = Layer(H, I, E, "mx32", fmt, seed=17)
        layer.s13 = layer.rng.integers(100, 131, size=layer.s13.shape).astype(np.uint8)
        layer.s2 = layer.rng.integers(90, 121, size=layer.s2.shape).astype(np.uint8)
        layer.s13[:, :8] = layer.rng.integers(1, 60, size=layer.s13[:, :8].shape)
        layer.dev[1], layer.dev[3] = _dev(layer.s13), _dev(layer.s2)
        x, ids, w = layer.inputs(4, 1, "bf16")
        layer.check(x, ids, w, "none")
        layer.check((x.float() * 2 ** -6).half(), ids, w * 2.0 ** -12, "relu")


@pytest.mark.parametrize("mode,fmt", FORMS)
@pytest.mark.parametrize("T,H,I,E,k", [(128, 1120, 544, 64, 16), (128, 32, 2080, 100, 16),
                                       (128, 2080, 32, 100, 16), (120, 512, 1024, 56, 8)])
def test_many_tokens_over_many_experts(mode, fmt, T, H, I, E, k):
    """More units than CUs, some with one chunk of K, experts with one column block or more."""
    layer = Layer(H, I, E, mode, fmt, seed=E + k)
    layer.check(*layer.inputs(T, k, "f16" if fmt == "e2m1" else "bf16"))


@pytest.mark.parametrize("fmt", ["e4m3", "e2m1"])
@pytest.mark.parametrize("T", [1, 128])
def test_mx_codes_at_the_ends(fmt, T):
    """Code c is 2^(c - 127), the smallest included, and 255 is NaN: sums of equal powers of
    two, exact in every step."""
    H, I = 128, 64
    one, per = (0x38, 1) if fmt == "e4m3" else (0x22, 2)
    w13 = torch.full((1, 2 * I, H // per), one, dtype=torch.uint8, device=DEV)
    w2 = torch.full((1, H, I // per), one, dtype=torch.uint8, device=DEV)
    ids = torch.zeros((T, 1), dtype=torch.int32, device=DEV)
    weights = torch.ones((T, 1), device=DEV)
    x = torch.full((T, H), 2.0 ** 30, dtype=torch.bfloat16, device=DEV)
    s13 = torch.full((1, 2 * I, H // 32), 120, dtype=torch.uint8, device=DEV)   # g = u = 2^30
    s2 = torch.full((1, H, I // 32), 127, dtype=torch.uint8, device=DEV)
    for code in (0, 1, 2, 254 - 127, 255):
        announce("moe mx code", fmt, T, code)
        s2[0, :16] = code
        out = F.moe_experts(x, ids, weights, w13, s13, w2, s2, "mx32", fmt, "relu").double()
        want = float("nan") if code == 255 else 64 * 2.0 ** 60 * 2.0 ** (code - 127)
        assert torch.equal(out[:, :16].cpu(),
                           torch.full((T, 16), want, dtype=torch.float64)) or (
            code == 255 and bool(out[:, :16].isnan().all()))
        assert bool((out[:, 16:] == 64 * 2.0 ** 60).all())


def test_zero_and_one_tokens_and_determinism():
    layer = Layer(512, 768, 8, "mx32", "e2m1", seed=19)
    x, ids, w = layer.inputs(7, 2, "bf16")
    empty = F.moe_experts(x[:0].to(DEV), _dev(ids[:0]), _dev(w[:0]), *layer.dev, "mx32", "e2m1")
    assert empty.shape == (0, 512)
    first = layer.check(x, ids, w)
    for _ in range(3):
        assert torch.equal(first, layer.check(x, ids, w))
    # a token's row does not depend on the others of the batch
    for t in range(7):
        one = layer.check(x[t:t + 1], ids[t:t + 1], w[t:t + 1])
        alone, together = one[0].float(), first[t].float()
        assert bool(((alone - together).abs() <= 2 ** -7 * together.abs() + 1e-6).all())


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_layer_is_route_then_experts(scoring):
    for T, E, k in ((1, 8, 2), (3, 64, 6), (31, 8, 2), (128, 16, 4), (2, 300, 8)):
        layer = Layer(128, 96, E, "rowwise", "e4m3", seed=21)
        x, _, _ = layer.inputs(T, k, "bf16")
        logits = torch.from_numpy(layer.rng.standard_normal((T, E)).astype(np.float32))
        if T > 2:
            logits[1] = -float("inf")
        announce("moe layer", scoring, (T, E, k))
        out, ids, w = F.moe_layer(x.to(DEV), logits.to(DEV), *layer.dev, k, scoring=scoring,
                                  scale=1.5)
        want_ids, want_w = F.moe_route(logits.to(DEV), k, scoring, scale=1.5)
        assert torch.equal(ids, want_ids) and torch.equal(w, want_w)
        assert torch.equal(out, F.moe_experts(x.to(DEV), ids, w, *layer.dev))
        layer.check(x, ids.cpu().numpy(), w.cpu().numpy())


def test_agrees_with_the_grouped_gemm():
    """The same weights through moe_route, group_rows and two grouped GEMMs, activations
    quantised per row: within what e4m3 activations (half a step of 2^-3, twice) cost."""
    H, I, E, T, k = 256, 512, 4, 50, 2
    layer = Layer(H, I, E, "rowwise", "e4m3", seed=23)
    x, _, _ = layer.inputs(T, k, "bf16")
    logits = torch.from_numpy(layer.rng.standard_normal((T, E)).astype(np.float32)).to(DEV)
    x = x.to(DEV)
    announce("moe against grouped gemm")
    out, ids, w = F.moe_layer(x, logits, *layer.dev, k)
    order, offsets = F.group_rows(ids, E)
    q13, s13, q2, s2 = layer.dev
    qa, sa = F.quantize(x.float()[(order // k).long()].contiguous(), "rowwise")
    gu = F.grouped_gemm(qa, sa, offsets, q13, s13).float()
    h = torch.nn.functional.silu(gu[:, :I]) * gu[:, I:]
    qh, sh = F.quantize(h.contiguous(), "rowwise")
    y = F.grouped_gemm(qh, sh, offsets, q2, s2).float()
    full = torch.zeros(T, H, device=DEV)
    full.index_add_(0, (order // k).long(), y * w.flatten()[order.long()][:, None])
    off = (full - out.float()).norm() / full.norm()
    # each quantisation is off by at most 2^-4 of a value, the gate's and the up row's and h's
    assert float(off) < 3 * 2 ** -4


def test_captured_under_changing_tokens():
    layer = Layer(256, 384, 8, "mx32", "e4m3", seed=25)
    T, k = 6, 2
    x = torch.empty(T, 256, dtype=torch.bfloat16, device=DEV)
    logits = torch.empty(T, 8, device=DEV)
    out = torch.empty(T, 256, dtype=torch.bfloat16, device=DEV)
    ids = torch.empty(T, k, dtype=torch.int32, device=DEV)
    w = torch.empty(T, k, device=DEV)
    ws = torch.zeros(F.fp8gemm_moe_workspace_size(T, 256, 384, 8, k), dtype=torch.uint8, device=DEV)

    def step():
        F.moe_layer(x, logits, *layer.dev, k, "mx32", out=out, ids=ids, weights=w, workspace=ws)

    x.normal_()
    logits.normal_()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    announce("moe captured")
    with torch.cuda.graph(graph):
        step()
    for i in range(4):
        g = torch.Generator().manual_seed(i)
        x.copy_(torch.randn(T, 256, generator=g))
        logits.copy_(torch.randn(T, 8, generator=g))
        eager = F.moe_layer(x, logits, *layer.dev, k, "mx32")
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip((out, ids, w), eager):
            assert torch.equal(a, b)
    assert not ws[:4096].any()                        # the GEMMs' counters are left alone


def test_side_stream_and_shared_workspace():
    """Calls on a side stream, next to split-K GEMMs that use the same cached workspace."""
    layer = Layer(256, 256, 4, "rowwise", "e4m3", seed=27)
    x, ids, w = layer.inputs(5, 2, "bf16")
    want = layer.check(x, ids, w)
    qa = torch.randint(0, 100, (64, 2048), dtype=torch.uint8, device=DEV)
    qb = torch.randint(0, 100, (256, 2048), dtype=torch.uint8, device=DEV)
    one = torch.ones(1, device=DEV)
    base = F.gemm(qa, one, qb, one)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(3):
            c = F.gemm(qa, one, qb, one)
            got = layer.check(x, ids, w)
            assert torch.equal(got, want)
            assert torch.equal(F.gemm(qa, one, qb, one), base) and torch.equal(c, base)
    side.synchronize()


def test_refusals():
    layer = Layer(64, 64, 4, "rowwise", "e4m3")
    x, ids, w = layer.inputs(3, 2, "bf16")
    x, ids, w = x.to(DEV), _dev(ids), _dev(w)
    with pytest.raises(ValueError, match="float16 or bfloat16"):
        F.moe_experts(x.float(), ids, w, *layer.dev)
    with pytest.raises(ValueError, match="shape"):
        F.moe_experts(x[:, :32], ids, w, *layer.dev)
    with pytest.raises(ValueError, match="int32"):
        F.moe_experts(x, ids.long(), w, *layer.dev)
    with pytest.raises(ValueError, match="scales"):
        F.moe_experts(x, ids, w, *layer.dev, mode="tensor")
    with pytest.raises(ValueError, match="logits"):
        F.moe_layer(x, torch.zeros(3, 5, device=DEV), *layer.dev, 2)
    big = torch.zeros(129, 64, dtype=torch.bfloat16, device=DEV)
    with pytest.raises(F.Fp8GemmError, match="NOT_SUPPORTED"):
        F.moe_experts(big, torch.zeros(129, 2, dtype=torch.int32, device=DEV),
                      torch.zeros(129, 2, device=DEV), *layer.dev)
    with pytest.raises(F.Fp8GemmError, match="WORKSPACE"):
        F.moe_experts(x, ids, w, *layer.dev,
                      workspace=torch.zeros(64, dtype=torch.uint8, device=DEV))
