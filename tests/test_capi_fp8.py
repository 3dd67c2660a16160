"""The FP8 expert layer's C entry points reject bad arguments on the host before
any HIP call, and the binding rejects wrong tensors before any pointer reaches
the library.  CPU only -- no compute call is made."""
from __future__ import annotations

import pytest
import torch

import q4_swiglu_mlp_amd as Z

A = 0x10000          # a 16-byte aligned fake device address (never dereferenced)
MIS = 0x10004        # 4-byte aligned only
ODD = 0x10002
BIG = 1 << 40
L = Z.lib


def call(fn, order, defaults):
    def f(**kw):
        args = dict(defaults)
        args.update(kw)
        return getattr(L, fn)(*[args[n] for n in order.split()])
    return f


sort = call("zinc_moe_sort", "ids M k E off sr rs ws wsb err stream",
            dict(ids=A, M=4096, k=8, E=64, off=A, sr=A, rs=A, ws=A, wsb=BIG, err=None, stream=None))
gather = call("zinc_moe_gather", "x type M k H sr xs stream", dict(x=A, type=0, M=16, k=8, H=2048, sr=A, xs=A,
                                                                  stream=None))
gather8 = call("zinc_moe_gather_fp8", "x type M k H sr q s stream",
               dict(x=A, type=0, M=16, k=8, H=2048, sr=A, q=A, s=A, stream=None))
combine = call("zinc_moe_combine", "ys type M k H sr p y stream",
               dict(ys=A, type=0, M=16, k=8, H=2048, sr=A, p=A, y=A, stream=None))
back = call("zinc_moe_combine_backward", "dy ys type M k H sr p dys dp stream",
            dict(dy=A, ys=A, type=0, M=16, k=8, H=2048, sr=A, p=A, dys=A, dp=A, stream=None))
quant = call("zinc_fp8_quantize", "x type R C br q s stream", dict(x=A, type=0, R=16, C=256, br=1, q=A, s=A,
                                                                  stream=None))
gemm = call("zinc_gemm_fp8", "a sa w sw M N K out c ws wsb stream",
            dict(a=A, sa=A, w=A, sw=A, M=64, N=256, K=256, out=0, c=A, ws=A, wsb=BIG, stream=None))
group = call("zinc_moe_gemm_fp8", "a sa w sw off E M N K out c ws wsb stream",
             dict(a=A, sa=A, w=A, sw=A, off=A, E=8, M=64, N=256, K=256, out=0, c=A, ws=A, wsb=BIG, stream=None))
experts = call("zinc_moe_fp8_experts", "wg sg wu su wd sd E H I x type M ids p k y ws wsb err stream",
               dict(wg=A, sg=A, wu=A, su=A, wd=A, sd=A, E=64, H=2048, I=768, x=A, type=0, M=16, ids=A, p=A, k=8, y=A,
                    ws=A, wsb=BIG, err=None, stream=None))


def test_sort_argument_errors():
    for n in ("ids", "off", "sr", "rs"):
        assert sort(**{n: None}) == -1
        assert sort(**{n: ODD}) == -3
    assert sort(err=ODD) == -3 and sort(ws=MIS) == -3
    assert sort(M=-1) == -5 and sort(k=0) == -5 and sort(k=1025) == -5 and sort(E=0) == -5 and sort(E=1025) == -5
    assert sort(M=(1 << 24) // 8 + 1) == -5
    assert sort(ws=None) == -1 and sort(wsb=16) == -4
    assert sort(M=0, off=None) == -1
    assert Z.moe_sort_workspace_size(1, 8, 64) == 0
    assert Z.moe_sort_workspace_size(4096, 8, 64) > 0
    assert Z.moe_sort_workspace_size(-1, 8, 64) == 0 and Z.moe_sort_workspace_size(8, 8, 0) == 0


@pytest.mark.parametrize("f,ptrs16,ptrs4", [(gather, ("x", "xs"), ("sr",)), (gather8, ("x", "q"), ("sr", "s")),
                                            (combine, ("ys", "y"), ("sr",)),
                                            (back, ("dy", "ys", "dys"), ("sr", "p", "dp"))])
def test_row_call_argument_errors(f, ptrs16, ptrs4):
    for n in ptrs16 + ptrs4:
        assert f(**{n: None}) == -1
    for n in ptrs16:
        assert f(**{n: MIS}) == -3
    for n in ptrs4:
        assert f(**{n: ODD}) == -3
    assert f(type=3) == -5 and f(type=-1) == -5
    assert f(H=0) == -2 and f(H=2052) == -2 and f(H=65536 + 16) == -2 and f(H=-16) == -2
    assert f(M=-1) == -5 and f(k=0) == -5 and f(M=(1 << 24) // 8 + 1) == -5
    assert f(M=0, **{n: None for n in ptrs16 + ptrs4}) == 0
    if f is combine:
        assert f(p=ODD) == -3
    if f is gather8:
        assert f(H=2056) == -2


def test_quantize_argument_errors():
    for n in ("x", "q", "s"):
        assert quant(**{n: None}) == -1
    assert quant(x=MIS) == -3 and quant(q=MIS) == -3 and quant(s=ODD) == -3
    assert quant(C=8) == -2 and quant(C=0) == -2 and quant(C=65552) == -2
    assert quant(br=64) == -5 and quant(R=-1) == -5 and quant(type=4) == -5
    assert quant(R=0, x=None) == 0


@pytest.mark.parametrize("f", [gemm, group])
def test_gemm_argument_errors(f):
    for n in ("a", "sa", "w", "sw", "c"):
        assert f(**{n: None}) == -1
    for n in ("a", "w", "c"):
        assert f(**{n: MIS}) == -3
    assert f(sa=ODD) == -3 and f(sw=ODD) == -3
    assert f(K=8) == -2 and f(K=0) == -2 and f(K=65552) == -2 and f(N=0) == -2 and f(N=(1 << 20) + 1) == -2
    assert f(M=-1) == -5 and f(M=(1 << 24) + 1) == -5 and f(out=3) == -5
    assert f(M=0) == 0 and f(M=0, a=None, c=None) == 0


def test_grouped_gemm_argument_errors():
    assert group(off=None) == -1 and group(off=ODD) == -3
    assert group(E=0) == -5 and group(E=1025) == -5
    assert Z.moe_gemm_fp8_workspace_size(64, 0, 256, 256) == 0 and Z.gemm_fp8_workspace_size(-1, 256, 256) == 0


def test_experts_argument_errors():
    for n in ("wg", "sg", "wu", "su", "wd", "sd", "x", "ids", "p", "y", "ws"):
        assert experts(**{n: None}) == -1
    for n in ("wg", "wu", "wd", "x", "y", "ws"):
        assert experts(**{n: MIS}) == -3
    for n in ("sg", "su", "sd", "ids", "p", "err"):
        assert experts(**{n: ODD}) == -3
    assert experts(H=2000) == -2 and experts(I=100) == -2 and experts(H=16384 + 128) == -2
    assert experts(k=0) == -5 and experts(k=65) == -5 and experts(E=1025) == -5 and experts(M=-1) == -5
    assert experts(type=3) == -5 and experts(wsb=100) == -4
    assert experts(M=0, ws=None, x=None) == 0
    size = [Z.moe_fp8_workspace_size(m, 8, 64, 2048, 768, torch.float16) for m in (1, 2, 15, 16, 17, 300, 4001, 4096)]
    assert all(a > 0 for a in size) and size == sorted(size)
    assert Z.moe_fp8_workspace_size(16, 65, 64, 2048, 768, torch.float16) == 0


def e4(*shape):
    return torch.zeros(shape, dtype=torch.float8_e4m3fn)


def f4(*shape):
    return torch.zeros(shape)


def i4(*shape):
    return torch.zeros(shape, dtype=torch.int32)


def h2(*shape):
    return torch.zeros(shape, dtype=torch.float16)


CASES = [
    # the call on right tensors (refused for the device), and wrong ones
    (Z.zinc_moe_sort, dict(expert_ids=i4(4, 2), n_experts=8), [
        (dict(expert_ids=i4(8)), "2-D"), (dict(expert_ids=i4(4, 2).long()), "int32"), (dict(n_experts=0), "n_experts"),
        (dict(expert_ids=i4(4, 0)), "top_k"), (dict(offsets=i4(8)), "offsets must have shape"),
        (dict(slot_row=i4(8)), "slot_row must have shape"), (dict(row_slot=i4(4, 2)), "row_slot must have shape"),
        (dict(dev_error=f4(1)), "dev_error"), (dict(expert_ids=i4(2, 4).t()), "contiguous")]),
    (Z.zinc_moe_gather, dict(x=h2(4, 64), slot_row=i4(4, 2)), [
        (dict(x=h2(4, 64).double()), "float16, bfloat16 or float32"), (dict(x=h2(4, 60)), "multiple of 8"),
        (dict(x=h2(64)), "2-D"), (dict(x=h2(64, 4).t()), "contiguous"), (dict(slot_row=i4(5, 2)), "slot_row"),
        (dict(slot_row=i4(4, 2).long()), "int32"), (dict(xs=h2(8, 32)), "xs must have shape"),
        (dict(xs=f4(8, 64)), "xs must be")]),
    (Z.zinc_moe_gather_fp8, dict(x=h2(4, 64), slot_row=i4(4, 2)), [
        (dict(x=h2(4, 56)), "multiple of 16"), (dict(q=h2(8, 64)), "q must be"),
        (dict(scales=f4(8, 2)), "scales must have shape")]),
    (Z.zinc_moe_combine, dict(ys=h2(8, 64), slot_row=i4(4, 2), expert_weights=f4(4, 2)), [
        (dict(ys=h2(7, 64)), "rows"), (dict(expert_weights=h2(4, 2)), "expert_weights must be"),
        (dict(expert_weights=f4(2, 4)), "expert_weights must have shape"), (dict(y=f4(4, 64)), "y must be")]),
    (Z.zinc_moe_gather_backward, dict(dxs=h2(8, 64), slot_row=i4(4, 2)), [(dict(dx=h2(8, 64)), "y must have shape")]),
    (Z.zinc_moe_combine_backward, dict(dy=h2(4, 64), ys=h2(8, 64), slot_row=i4(4, 2), expert_weights=f4(4, 2)), [
        (dict(ys=f4(8, 64)), "ys must be"), (dict(dys=h2(4, 64)), "dys must have shape"),
        (dict(dweights=h2(4, 2)), "dweights must be")]),
    (Z.zinc_fp8_quantize, dict(x=h2(4, 64)), [
        (dict(block_rows=2), "block_rows"), (dict(x=h2(4, 40)), "multiple of 16"), (dict(q=e4(4, 32)), "q must have"),
        (dict(scales=f4(4, 2)), "scales must have"), (dict(x=i4(4, 64)), "float16")]),
    (Z.zinc_gemm_fp8, dict(a=e4(4, 144), a_scales=f4(4, 2), w=e4(130, 144), w_scales=f4(2, 2)), [
        (dict(a=h2(4, 144)), "a must be"), (dict(a_scales=f4(4, 1)), "a_scales must have"),
        (dict(w=e4(130, 128)), "w must have shape"), (dict(w_scales=f4(1, 2)), "scales must have"),
        (dict(a=e4(4, 136), a_scales=f4(4, 2)), "multiple of 16"), (dict(out=h2(4, 129)), "out must have"),
        (dict(out_dtype=torch.float64), "float16, bfloat16 or float32"), (dict(w=e4(1, 130, 144)), "2-D")]),
    (Z.zinc_moe_gemm_fp8, dict(a=e4(4, 144), a_scales=f4(4, 2), w=e4(3, 130, 144), w_scales=f4(3, 2, 2),
                               offsets=i4(4)), [
        (dict(offsets=i4(3)), "offsets must have"), (dict(offsets=i4(4).long()), "int32"), (dict(w=e4(130, 144)), "3-D"),
        (dict(w_scales=f4(2, 2)), "scales must have")]),
    (Z.zinc_moe_fp8_experts, dict(w_gate=e4(2, 256, 128), gate_scales=f4(2, 2, 1), w_up=e4(2, 256, 128),
                                  up_scales=f4(2, 2, 1), w_down=e4(2, 128, 256), down_scales=f4(2, 1, 2),
                                  x=h2(4, 128), expert_ids=i4(4, 2), expert_weights=f4(4, 2)), [
        (dict(x=h2(4, 144)), "multiple of 128"), (dict(w_up=e4(2, 128, 128)), "w_up must have"),
        (dict(w_down=e4(2, 256, 128)), "w_down must have"), (dict(down_scales=f4(2, 2, 1)), "scales must have"),
        (dict(expert_ids=i4(4, 2).long()), "int32"), (dict(expert_ids=i4(4, 3), expert_weights=f4(4, 3)), "top_k"),
        (dict(y=f4(4, 128)), "y must be"), (dict(workspace=torch.zeros(16, dtype=torch.uint8)), "workspace holds")]),
]


@pytest.mark.parametrize("fn,good,wrong", CASES, ids=[c[0].__name__ for c in CASES])
def test_binding_checks(fn, good, wrong):
    with pytest.raises(ValueError, match="GPU"):
        fn(**good)
    for bad, msg in wrong:
        with pytest.raises(ValueError, match=msg):
            fn(**{**good, **bad})


@pytest.mark.parametrize("E", [1, 64, 256, 1024])
@pytest.mark.parametrize("k,H,I", [(1, 256, 128), (8, 2048, 768)])
def test_workspaces_do_not_shrink_with_more_tokens(E, k, H, I):
    """Token by token around each size where the sort is spread otherwise: 4096 slots, one workgroup or more; from
    262144 on every 131072, 512 more slots a workgroup."""
    k = min(k, E)
    slots = [512, 4096, 5120, 131072] + [131072 * i for i in range(2, 129)]
    for sizes in (lambda m: Z.moe_fp8_workspace_size(m, k, E, H, I, torch.bfloat16),
                  lambda m: Z.moe_sort_workspace_size(m, k, E)):
        last = 0
        for m in sorted({s // k + d for s in slots for d in range(-2, 3)}):
            if 0 < m * k <= 1 << 24:
                assert sizes(m) >= last, m
                last = sizes(m)


def test_dense_product_workspace_by_rows():
    """What the header says of it: it rises and falls with M, and 16 MiB are always enough."""
    sizes = {m: Z.gemm_fp8_workspace_size(m, 4096, 4096) for m in (4, 5, 128, 512, 8192)}
    assert sizes[4] == 0 and 0 < sizes[5] < sizes[128] == 12 << 20 and sizes[512] == sizes[8192] == 0
    assert gemm(M=128, N=4096, K=4096, ws=None) == -1 and gemm(M=128, N=4096, K=4096, wsb=sizes[128] - 1) == -4
    for n in (1, 24, 127, 128, 129, 1000, 4096, 11008, 32300, 1 << 20):
        for tiles in range(1, 520):
            assert Z.gemm_fp8_workspace_size(64 * tiles, n, 65536) <= 16 << 20
    # parts of K times tiles of 64 x 128 are at most 380 + tiles / 2, and two parts need fewer than 254 tiles
    assert (380 + 253 / 2) * 64 * 128 * 4 < 16 << 20
    assert all(Z.moe_gemm_fp8_workspace_size(m, 8, 4096, 4096) == 0 for m in (1, 5, 64, 128, 4096))


def test_counts_past_32_bits_are_refused():
    """The C entry points take 32-bit counts: a larger one must not arrive there as its low bits."""
    rows = torch.empty((1 << 32) + 3, 16, dtype=torch.float16, device="meta")
    with pytest.raises(ValueError, match="rows"):
        Z.zinc_fp8_quantize(rows)
    with pytest.raises(ValueError, match="rows"):
        Z.zinc_fp8_quantize(torch.empty(1 << 31, 16, dtype=torch.float16, device="meta"), 128)
    wide = 1 << 32
    assert Z.gemm_fp8_workspace_size(64, 256, 4096) > 0
    for m, n, k in ((64 + wide, 256, 4096), (64, 256 + wide, 4096), (64, 256, 4096 + wide), (64 - wide, 256, 4096)):
        assert Z.gemm_fp8_workspace_size(m, n, k) == 0
    assert Z.moe_sort_workspace_size(4096 + wide, 8, 64) == 0 and Z.moe_sort_workspace_size(4096, 8, 64 + wide) == 0
    assert Z.moe_gemm_fp8_workspace_size(64, 8 + wide, 256, 256) == 0
    assert Z.moe_fp8_workspace_size(16 + wide, 8, 64, 2048, 768, torch.float16) == 0
    assert Z.moe_fp8_workspace_size(16, 8, 64, 2048, 768 + wide, torch.float16) == 0


def test_gather_backward_names_dx():
    for bad in (h2(8, 64), h2(4, 32), f4(4, 64)):
        with pytest.raises(ValueError, match="^dx"):
            Z.zinc_moe_gather_backward(h2(8, 64), i4(4, 2), dx=bad)
