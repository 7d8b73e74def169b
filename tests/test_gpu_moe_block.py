"""The example block on the GPU: every operator's output against the float64 references of its
own inputs, the captured step against the eager one, and both forms of the experts."""
import importlib.util
import os

import numpy as np
import pytest
import torch

from oracle import layers as L

from gpu_support import DEV, announce, to_host

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                    "moe_block.py")


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("moe_block", PATH)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def _rows(block, n, seed):
    gen = torch.Generator(DEV).manual_seed(seed)
    x = torch.randn(n, block.hidden, generator=gen, device=DEV).bfloat16()
    adapter = torch.randint(-1, block.adapters, (n,), generator=gen, device=DEV,
                            dtype=torch.int32)
    return x, adapter


@pytest.mark.parametrize("rows", [1, 19, 128])
def test_decode_step_against_the_references(example, rows):
    block = example.Block(256, 192, 6, 2, 3, 16)
    x, adapter = _rows(block, rows, rows)
    announce("moe_block", rows)
    step = block.decode(x, block.plan(adapter))
    torch.cuda.synchronize()
    xh, base = x.cpu().double().numpy(), step.base.cpu().double().numpy()
    want, tol = L.lora_reference(xh, base, block.lora_a.cpu().double().numpy(),
                                 block.lora_b.cpu().double().numpy(), adapter.cpu().numpy(), None,
                                 "none", "bf16")
    y = step.y.cpu().double().numpy()
    sum_tol = tol + np.abs(xh + want) * 2.0 ** -8 + tol * 2.0 ** -8       # x + lora, rounded
    assert np.all(np.abs(y - (xh + want)) <= sum_tol)
    logits = step.logits.cpu().double().numpy()
    ids, w = L.route_reference(logits, 2, "softmax", True)
    assert np.array_equal(step.ids.cpu().numpy(), ids)
    got_w = step.weights.cpu().double().numpy()
    assert np.all(np.abs(got_w - w) <= L.route_tolerance(logits, w, 2))
    host = [t.cpu().numpy() for t in (*block.w13, *block.w2)]
    want, tol = L.moe_reference(y, ids, got_w, host[0], host[1], host[2], host[3], "rowwise",
                                "e4m3", "silu", "bf16")
    assert np.all(np.abs(to_host(step.experts) - want) <= tol)


def test_graph_follows_its_rows(example):
    block = example.Block(256, 192, 6, 2, 3, 16)
    x, adapter = _rows(block, 24, 7)
    order, offsets = block.plan(adapter)
    graph, step = example.captured(block, x, (order, offsets))
    for seed in (8, 9, 10):
        other, ids = _rows(block, 24, seed)
        plan = block.plan(ids)
        want = block.decode(other, plan).out
        x.copy_(other)
        order.copy_(plan[0])
        offsets.copy_(plan[1])
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(step.out, want)


def test_command(example, capsys):
    """The forms differ by the rounding of activations to e4m3 (3 mantissa bits: at most 2^-4 of
    an element, twice in a row), on the experts' part of the sum alone."""
    _, _, apart = example.main(["--hidden", "512", "--inner", "512", "--requests", "16",
                                "--prompt", "200"])
    assert apart < 2 * 2.0 ** -4
    assert "prompt, 200 rows" in capsys.readouterr().out
