"""C-ABI checks of the serving operators that need no GPU: the library exports every
function of the header and rejects invalid arguments before any HIP call.

Fake device addresses below are never dereferenced: every call either fails validation
or has no work.
"""
import ctypes
import os

import pytest

import block_scaled_gemm_fp8gemm_amd as F

SUCCESS, INVALID, MISALIGNED, NOT_SUPPORTED, WORKSPACE = 0, 1, 2, 3, 4
P = 0x10000
BIG = 1 << 40                        # workspace bytes no check finds too small


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(F.library_path()):
        from block_scaled_gemm_fp8gemm_amd.build import build
        build()
    return F.load_library()


def test_exports_every_declared_symbol(lib):
    names = F.exported_layer_symbols()
    assert set(names) == {
        "fp8gemm_moe_route", "fp8gemm_group_rows_workspace_size", "fp8gemm_group_rows",
        "fp8gemm_moe_workspace_size", "fp8gemm_moe_run", "fp8gemm_moe_layer",
        "fp8gemm_lora_workspace_size", "fp8gemm_lora_run"}
    raw = ctypes.CDLL(F.library_path())
    for n in names:
        assert hasattr(raw, n), n
        assert n in F.__all__ and callable(getattr(F, n))


ROUTE = dict(logits=P, dtype=2, rows=4, ldl=8, experts=8, k=2, scoring=0, renormalize=1, scale=1.0,
             ids=P, weights=P, stream=0)


@pytest.mark.parametrize("change,status", [
    (dict(rows=0, logits=0, ids=0, weights=0), SUCCESS),
    (dict(dtype=3), INVALID), (dict(dtype=-1), INVALID), (dict(rows=-1), INVALID),
    (dict(experts=0), INVALID), (dict(k=0), INVALID), (dict(k=9), INVALID),
    (dict(scoring=2), INVALID), (dict(ldl=7), INVALID), (dict(logits=0), INVALID),
    (dict(ids=0), INVALID), (dict(weights=0), INVALID),
    (dict(experts=1025, ldl=1025), NOT_SUPPORTED), (dict(experts=64, ldl=64, k=17), NOT_SUPPORTED),
    (dict(rows=1 << 31), NOT_SUPPORTED), (dict(logits=P + 2), MISALIGNED),
    (dict(dtype=0, logits=P + 1), MISALIGNED), (dict(ids=P + 2), MISALIGNED),
    (dict(weights=P + 1), MISALIGNED)])
def test_route_arguments(lib, change, status):
    a = {**ROUTE, **change}
    assert lib.fp8gemm_moe_route(*a.values()) == status


GROUP = dict(ids=P, n=100000, groups=8, order=P, offsets=P, workspace=P, bytes=BIG, stream=0)


@pytest.mark.parametrize("change,status", [
    (dict(n=-1), INVALID), (dict(groups=0), INVALID), (dict(offsets=0), INVALID),
    (dict(ids=0), INVALID), (dict(order=0), INVALID), (dict(groups=1025), NOT_SUPPORTED),
    (dict(n=(1 << 31) - 1), NOT_SUPPORTED), (dict(ids=P + 1), MISALIGNED),
    (dict(order=P + 2), MISALIGNED), (dict(offsets=P + 2), MISALIGNED),
    (dict(workspace=0), WORKSPACE), (dict(bytes=64), WORKSPACE),
    (dict(workspace=P + 2), MISALIGNED)])
def test_group_rows_arguments(lib, change, status):
    a = {**GROUP, **change}
    assert lib.fp8gemm_group_rows(*a.values()) == status


def test_workspace_queries(lib):
    assert F.fp8gemm_group_rows_workspace_size(100, 8) == 0
    assert F.fp8gemm_group_rows_workspace_size(100000, 8) > 0
    assert F.fp8gemm_group_rows_workspace_size(0, 8) == 0
    assert F.fp8gemm_group_rows_workspace_size(10, 2000) == 0
    # h in two bf16 and the fp32 rows of every slot
    assert F.fp8gemm_moe_workspace_size(16, 256, 512, 8, 2) >= 32 * (512 + 256) * 4
    assert F.fp8gemm_moe_workspace_size(0, 256, 512, 8, 2) == 0
    assert F.fp8gemm_moe_workspace_size(129, 256, 512, 8, 2) == 0
    assert F.fp8gemm_lora_workspace_size(100, 512, 16, 4) >= 100 * 16 * 4
    assert F.fp8gemm_lora_workspace_size(100, 512, 136, 4) == 0


MOE = dict(T=4, H=256, I=512, experts=8, k=2, x=P, ldx=256, dtype=1, ids=P, weights=P, w13=P,
           ld13=256, stride13=1024 * 256, scale13=P, w2=P, ld2=512, stride2=256 * 512, scale2=P,
           mode=1, format=0, activation=3, out=P, ldo=256, workspace=P, bytes=BIG, stream=0)
MOE_BAD = [
    (dict(T=-1), INVALID), (dict(H=0), INVALID), (dict(I=0), INVALID), (dict(experts=0), INVALID),
    (dict(k=0), INVALID), (dict(dtype=2), INVALID), (dict(mode=3), INVALID),
    (dict(format=5), INVALID), (dict(activation=4), INVALID), (dict(activation=-1), INVALID),
    (dict(x=0), INVALID), (dict(out=0), INVALID), (dict(w13=0), INVALID), (dict(w2=0), INVALID),
    (dict(scale13=0), INVALID), (dict(scale2=0), INVALID), (dict(ids=0), INVALID),
    (dict(weights=0), INVALID), (dict(ldx=248), INVALID), (dict(ldo=248), INVALID),
    (dict(ld13=240), INVALID), (dict(ld2=496), INVALID), (dict(stride13=1023 * 256), INVALID),
    (dict(stride2=255 * 512), INVALID), (dict(stride2=-512), INVALID),
    (dict(T=129), NOT_SUPPORTED), (dict(experts=1025), NOT_SUPPORTED),
    (dict(experts=64, k=17), NOT_SUPPORTED), (dict(format=1), NOT_SUPPORTED),
    (dict(format=2, mode=2), NOT_SUPPORTED), (dict(format=4, mode=1), NOT_SUPPORTED),
    (dict(H=264, ldx=264, ldo=264, ld13=272), NOT_SUPPORTED),
    (dict(I=520, ld2=528), NOT_SUPPORTED), (dict(mode=2, I=528, ld2=528), NOT_SUPPORTED),
    (dict(x=P + 8), MISALIGNED), (dict(out=P + 8), MISALIGNED), (dict(ldx=260), MISALIGNED),
    (dict(ldo=260), MISALIGNED), (dict(w13=P + 8), MISALIGNED), (dict(w2=P + 8), MISALIGNED),
    (dict(ld13=264, stride13=1024 * 264), MISALIGNED), (dict(stride2=256 * 512 + 8), MISALIGNED),
    (dict(scale13=P + 1), MISALIGNED), (dict(ids=P + 2), MISALIGNED),
    (dict(weights=P + 2), MISALIGNED), (dict(workspace=0), WORKSPACE), (dict(bytes=1000), WORKSPACE),
    (dict(workspace=P + 8), MISALIGNED),
    # the fp32 rows of every slot are addressed with 32-bit offsets
    (dict(T=128, k=16, experts=64, H=1 << 20, ldx=1 << 20, ldo=1 << 20, ld13=1 << 20,
          stride13=1 << 30, stride2=1 << 30), NOT_SUPPORTED),
]


@pytest.mark.parametrize("change,status", MOE_BAD + [
    (dict(T=0, x=0, ids=0, weights=0, w13=0, w2=0, out=0, workspace=0), SUCCESS)])
def test_moe_run_arguments(lib, change, status):
    a = {**MOE, **change}
    assert lib.fp8gemm_moe_run(*a.values()) == status


LAYER_KEYS = ["T", "H", "I", "experts", "k", "x", "ldx", "dtype", "logits", "ldl", "logits_dtype",
              "scoring", "renormalize", "scale", "ids", "weights", "w13", "ld13", "stride13",
              "scale13", "w2", "ld2", "stride2", "scale2", "mode", "format", "activation", "out",
              "ldo", "workspace", "bytes", "stream"]
LAYER = {**MOE, "logits": P, "ldl": 1024, "logits_dtype": 2, "scoring": 0, "renormalize": 1,
         "scale": 1.0}


@pytest.mark.parametrize("change,status", MOE_BAD + [
    (dict(T=0, x=0, logits=0, ids=0, weights=0, w13=0, w2=0, out=0, workspace=0), SUCCESS),
    (dict(logits=0), INVALID), (dict(ldl=7), INVALID), (dict(logits_dtype=3), INVALID),
    (dict(scoring=-1), INVALID), (dict(k=9), INVALID), (dict(logits=P + 2), MISALIGNED)])
def test_moe_layer_arguments(lib, change, status):
    a = {**LAYER, **change}
    assert lib.fp8gemm_moe_layer(*[a[n] for n in LAYER_KEYS]) == status


LORA = dict(M=10, N=100, K=256, rank=16, groups=4, x=P, ldx=256, base=P, ldbase=104, dtype=1, a=P,
            lda=256, stride_a=16 * 256, b=P, ldb=16, stride_b=1600, order=P, offsets=P, scales=P,
            activation=0, out=P, ldo=104, workspace=P, bytes=BIG, stream=0)


@pytest.mark.parametrize("change,status", [
    (dict(M=0, x=0, base=0, out=0), SUCCESS), (dict(N=0, base=0, out=0), SUCCESS),
    (dict(M=-1), INVALID), (dict(N=-1), INVALID), (dict(K=0), INVALID), (dict(rank=0), INVALID),
    (dict(groups=0), INVALID), (dict(dtype=2), INVALID), (dict(activation=4), INVALID),
    (dict(x=0), INVALID), (dict(base=0), INVALID), (dict(a=0), INVALID), (dict(b=0), INVALID),
    (dict(order=0), INVALID), (dict(offsets=0), INVALID), (dict(out=0), INVALID),
    (dict(ldx=248), INVALID), (dict(ldbase=96), INVALID), (dict(ldo=96), INVALID),
    (dict(lda=248), INVALID), (dict(ldb=8), INVALID), (dict(stride_a=15 * 256), INVALID),
    (dict(stride_b=1592), INVALID), (dict(stride_b=-16), INVALID),
    (dict(rank=136), NOT_SUPPORTED), (dict(rank=12), NOT_SUPPORTED), (dict(K=252), NOT_SUPPORTED),
    (dict(groups=1025), NOT_SUPPORTED), (dict(M=1 << 31), NOT_SUPPORTED),
    (dict(M=1 << 30, N=1 << 12, ldbase=1 << 12, ldo=1 << 12, stride_b=1 << 16), NOT_SUPPORTED),
    (dict(x=P + 8), MISALIGNED), (dict(base=P + 2), MISALIGNED), (dict(a=P + 8), MISALIGNED),
    (dict(b=P + 8), MISALIGNED), (dict(out=P + 4), MISALIGNED), (dict(order=P + 1), MISALIGNED),
    (dict(scales=P + 2), MISALIGNED), (dict(ldx=260), MISALIGNED), (dict(ldbase=100), MISALIGNED),
    (dict(ldo=100), MISALIGNED), (dict(lda=260, stride_a=16 * 264), MISALIGNED),
    (dict(stride_a=16 * 256 + 4), MISALIGNED), (dict(ldb=20, stride_b=2000), MISALIGNED),
    (dict(workspace=0), WORKSPACE), (dict(bytes=100), WORKSPACE),
    (dict(workspace=P + 8), MISALIGNED)])
def test_lora_arguments(lib, change, status):
    a = {**LORA, **change}
    assert lib.fp8gemm_lora_run(*a.values()) == status


def test_python_layer_refuses_cpu_tensors():
    import torch
    f, i = torch.zeros(4, 64), torch.zeros(4, dtype=torch.int32)
    h = torch.zeros(4, 64, dtype=torch.bfloat16)
    q = torch.zeros(2, 64, 64, dtype=torch.uint8)
    for call in (lambda: F.moe_route(f, 2), lambda: F.group_rows(i, 4),
                 lambda: F.moe_layer(h, f, q, f, q, f, 2),
                 lambda: F.moe_experts(h, i, f, q, f, q, f),
                 lambda: F.lora(h, h, h, h, i, i)):
        with pytest.raises(ValueError, match="CUDA"):
            call()
