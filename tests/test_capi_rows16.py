"""Refusals of the 16-bit products by expert, SwiGLU and the adapters: by the C entry points before any HIP
call, and by the binding before any pointer reaches the library.  CPU only."""
from __future__ import annotations

import pytest
import torch

import q4_swiglu_mlp_amd as Z

A = 0x10000          # a 16-byte aligned fake device address (never dereferenced)
MIS = 0x10004        # 4-byte aligned only
ODD = 0x10002
BIG = 1 << 40


def call(fn, order, defaults):
    def f(**kw):
        args = dict(defaults)
        args.update(kw)
        return getattr(Z.lib, fn)(*[args[n] for n in order.split()])
    return f


gemm = call("zinc_moe_gemm", "a w type off E M N K out c ws wsb stream",
            dict(a=A, w=A, type=0, off=A, E=8, M=64, N=256, K=256, out=0, c=A, ws=A, wsb=BIG, stream=None))
back = call("zinc_moe_gemm_backward", "dc a w type off E M N K dat da dwt dw ws wsb stream",
            dict(dc=A, a=A, w=A, type=1, off=A, E=8, M=64, N=256, K=256, dat=1, da=A, dwt=2, dw=A, ws=A, wsb=BIG,
                 stream=None))
glu = call("zinc_swiglu", "g u type M C h stream", dict(g=A, u=A, type=0, M=16, C=256, h=A, stream=None))
glu_back = call("zinc_swiglu_backward", "dh g u type M C dg du stream",
                dict(dh=A, g=A, u=A, type=0, M=16, C=256, dg=A, du=A, stream=None))
PLAN = dict(off=A, sr=A, rs=A)
lora = call("zinc_lora", "x type M K a b r E N s off sr rs base y ws wsb stream",
            dict(x=A, type=0, M=16, K=256, a=A, b=A, r=16, E=4, N=512, s=A, base=A, y=A, ws=A, wsb=BIG, stream=None,
                 **PLAN))
lora_back = call("zinc_lora_backward", "dy x type M K a b r E N s off sr rs base dx da db ws wsb stream",
                 dict(dy=A, x=A, type=0, M=16, K=256, a=A, b=A, r=16, E=4, N=512, s=A, base=A, dx=A, da=A, db=A, ws=A,
                      wsb=BIG, stream=None, **PLAN))


def check_pointers(f, needed, optional=(), four=()):
    for n in needed:
        assert f(**{n: None}) == -1, n
    for n in tuple(needed) + tuple(optional):
        assert f(**{n: ODD}) == -3, n
        if n not in four:
            assert f(**{n: MIS}) == -3, n


@pytest.mark.parametrize("f", [gemm, back])
def test_product_argument_errors(f):
    for bad in (0, -8, 12, 65544):
        assert f(N=bad) == -2 and f(K=bad) == -2
    assert f(M=-1) == -5 and f(M=(1 << 24) + 1) == -5 and f(E=0) == -5 and f(E=1025) == -5
    assert f(type=2) == -5 and f(type=3) == -5 and f(type=-1) == -5


def test_product_pointers_and_types():
    check_pointers(gemm, ("a", "w", "off", "c"), four=("off",))
    assert gemm(out=1) == -5 and gemm(type=1, out=0) == -5 and gemm(out=3) == -5
    assert gemm(M=0, a=None, w=None, off=None, c=None) == 0
    check_pointers(back, ("dc", "a", "w", "off"), optional=("da", "dw"), four=("off",))
    assert back(dat=0) == -5 and back(dwt=0) == -5 and back(dwt=3) == -5
    assert back(da=None, dw=None) == -1
    assert back(M=0, dw=None) == 0 and back(M=0, off=None) == -1
    # what a gradient that is not wanted would read may be missing; the next check then speaks
    assert back(da=None, w=None, dat=9, dc=ODD) == -3 and back(dw=None, a=None, dwt=9, dc=ODD) == -3


def test_swiglu_argument_errors():
    check_pointers(glu, ("g", "u", "h"))
    check_pointers(glu_back, ("dh", "g", "u", "dg", "du"))
    for f in (glu, glu_back):
        assert f(C=0) == -2 and f(C=12) == -2 and f(C=65544) == -2 and f(M=-1) == -5 and f(M=(1 << 24) + 1) == -5
        assert f(type=3) == -5 and f(type=-1) == -5
        assert f(M=0, g=None) == 0


def test_adapter_argument_errors():
    plan = ("off", "sr", "rs")
    check_pointers(lora, ("x", "a", "b", "y", "ws") + plan, optional=("base", "s"), four=plan + ("s",))
    check_pointers(lora_back, ("dy", "x", "a", "b", "ws") + plan, optional=("base", "s", "dx", "da", "db"),
                   four=plan + ("s",))
    for f in (lora, lora_back):
        for bad in (0, -8, 12, 65544):
            assert f(N=bad) == -2 and f(K=bad) == -2
        for bad in (0, 4, 12, 264):
            assert f(r=bad) == -2
        assert f(M=-1) == -5 and f(M=(1 << 24) + 1) == -5 and f(E=0) == -5 and f(E=1025) == -5
        assert f(type=2) == -5 and f(type=-1) == -5
        assert f(wsb=16) == -4
    assert lora(M=0, x=None, ws=None) == 0
    assert lora_back(dx=None, da=None, db=None) == -1
    assert lora_back(M=0, da=None, db=None) == 0 and lora_back(M=0, off=None) == -1


def test_workspace_sizes():
    for size in (Z.lora_workspace_size, Z.lora_backward_workspace_size):
        for E, K, N, r in ((1, 4096, 4096, 16), (64, 256, 11008, 8), (1024, 8, 65536, 256)):
            sizes = [size(M, E, K, N, r) for M in (1, 2, 17, 64, 100, 1000, 1025, 5000, 16384, 16385, 100000, 1 << 24)]
            assert sizes == sorted(sizes) and sizes[0] > 0
        assert size(0, 4, 256, 256, 16) == 0 and size(-1, 4, 256, 256, 16) == 0
        assert size(16, 0, 256, 256, 16) == 0 and size(16, 4, 252, 256, 16) == 0 and size(16, 4, 256, 256, 264) == 0
        assert size(1 << 40, 4, 256, 256, 16) == 0
    for size in (Z.moe_gemm_workspace_size, Z.moe_gemm_backward_workspace_size):
        assert size(-1, 4, 256, 256) == 0 and size(16, 0, 256, 256) == 0 and size(16, 4, 12, 256) == 0
        assert size(1 << 40, 4, 256, 256) == 0
    for size in (Z.moe_gemm_workspace_size, Z.moe_gemm_backward_workspace_size):
        for E, N, K in ((1, 8, 800), (1, 4096, 4096), (64, 768, 2048), (1024, 1024, 64), (1, 65536, 65536), (1, 65536, 8)):
            sizes = [size(rows, E, N, K) for rows in (0, 1, 2, 7, 64, 100, 1000, 4096, 10000, 33333, 1 << 20, 1 << 24)]
            assert sizes == sorted(sizes) and sizes[0] == 0 and 0 < sizes[1] and sizes[-1] <= (1 << 26) + (1 << 11)


def test_a_small_workspace_is_refused():
    need = Z.moe_gemm_workspace_size(40, 1, 8, 800)
    with pytest.raises(ValueError, match="workspace holds"):
        Z.zinc_moe_gemm(h(40, 800), h(1, 8, 800), i32(2), workspace=torch.zeros(need - 1, dtype=torch.uint8))
    need = Z.moe_gemm_backward_workspace_size(1685, 2, 8, 8)
    with pytest.raises(ValueError, match="workspace holds"):
        Z.zinc_moe_gemm_backward(h(1685, 8), h(1685, 8), h(2, 8, 8), i32(3),
                                 workspace=torch.zeros(need - 1, dtype=torch.uint8))


# ---------------------------------------------------------------- the binding
H = torch.float16


def h(*shape, dtype=H):
    return torch.zeros(shape, dtype=dtype)


def i32(*shape):
    return torch.zeros(shape, dtype=torch.int32)


def test_right_tensors_on_the_cpu_are_rejected_for_the_device_only():
    for f in (lambda: Z.zinc_moe_gemm(h(4, 16), h(2, 8, 16), i32(3)),
              lambda: Z.zinc_moe_gemm_backward(h(4, 8), h(4, 16), h(2, 8, 16), i32(3)),
              lambda: Z.zinc_swiglu(h(4, 16), h(4, 16)),
              lambda: Z.zinc_swiglu_backward(h(4, 16), h(4, 16), h(4, 16)),
              lambda: Z.zinc_lora(h(4, 16), h(2, 8, 16), h(2, 24, 8), None, i32(3), i32(4, 1), i32(4)),
              lambda: Z.zinc_lora_backward(h(4, 24), h(4, 16), h(2, 8, 16), h(2, 24, 8), None, i32(3), i32(4, 1),
                                           i32(4))):
        with pytest.raises(ValueError, match="GPU"):
            f()


GEMM = dict(a=h(4, 16), w=h(2, 8, 16), offsets=i32(3))
GEMM_BACK = dict(dc=h(4, 8), a=h(4, 16), w=h(2, 8, 16), offsets=i32(3))
GLU = dict(gate=h(4, 16), up=h(4, 16))
LORA = dict(x=h(4, 16), a=h(2, 8, 16), b=h(2, 24, 8), scales=torch.ones(2), offsets=i32(3), slot_row=i32(4, 1),
            row_slot=i32(4))
LORA_BACK = dict(LORA, dy=h(4, 24))


@pytest.mark.parametrize("f,good,bad,msg", [
    (Z.zinc_moe_gemm, GEMM, dict(a=h(4, 16, dtype=torch.float32)), "float16 or bfloat16"),
    (Z.zinc_moe_gemm, GEMM, dict(a=h(4, 12)), "multiple of 8"),
    (Z.zinc_moe_gemm, GEMM, dict(a=h(16, 4).t()), "contiguous"),
    (Z.zinc_moe_gemm, GEMM, dict(a=h(16)), "2-D"),
    (Z.zinc_moe_gemm, GEMM, dict(w=h(2, 8, 16, dtype=torch.bfloat16)), "w must be"),
    (Z.zinc_moe_gemm, GEMM, dict(w=h(2, 8, 24)), "shape"),
    (Z.zinc_moe_gemm, GEMM, dict(w=h(2, 12, 16)), "multiples of 8"),
    (Z.zinc_moe_gemm, GEMM, dict(w=h(8, 16)), "3-D"),
    (Z.zinc_moe_gemm, GEMM, dict(w=h(2, 16, 8).transpose(1, 2)), "contiguous"),
    (Z.zinc_moe_gemm, GEMM, dict(offsets=i32(2)), "offsets"),
    (Z.zinc_moe_gemm, GEMM, dict(offsets=torch.zeros(3, dtype=torch.int64)), "offsets"),
    (Z.zinc_moe_gemm, GEMM, dict(out_dtype=torch.bfloat16), "out_dtype"),
    (Z.zinc_moe_gemm, GEMM, dict(out=h(4, 16)), "out must have shape"),
    (Z.zinc_moe_gemm_backward, GEMM_BACK, dict(dc=h(4, 16)), "w must have shape"),
    (Z.zinc_moe_gemm_backward, GEMM_BACK, dict(a=h(5, 16)), "a must have shape"),
    (Z.zinc_moe_gemm_backward, GEMM_BACK, dict(dw_dtype=torch.bfloat16), "dw_dtype"),
    (Z.zinc_moe_gemm_backward, GEMM_BACK, dict(want_da=False, want_dw=False), "one at least"),
    (Z.zinc_moe_gemm_backward, GEMM_BACK, dict(want_da=False, da=h(4, 16)), "one at least"),
    (Z.zinc_moe_gemm_backward, GEMM_BACK, dict(dw=h(2, 8, 8)), "dw must have shape"),
    (Z.zinc_swiglu, GLU, dict(up=h(4, 24)), "up must have shape"),
    (Z.zinc_swiglu, GLU, dict(up=h(4, 16, dtype=torch.float32)), "up must be"),
    (Z.zinc_swiglu, GLU, dict(gate=h(4, 20)[:, :16]), "contiguous"),
    (Z.zinc_swiglu, GLU, dict(h=h(4, 24)), "h must have shape"),
    (Z.zinc_swiglu_backward, dict(GLU, dh=h(4, 16)), dict(dh=h(3, 16)), "dh must have shape"),
    (Z.zinc_swiglu_backward, dict(GLU, dh=h(4, 16)), dict(dup=h(3, 16)), "dup must have shape"),
    (Z.zinc_lora, LORA, dict(a=h(2, 12, 16)), "rank"),
    (Z.zinc_lora, LORA, dict(a=h(2, 264, 16)), "rank"),
    (Z.zinc_lora, LORA, dict(a=h(2, 8, 24)), "a must have shape"),
    (Z.zinc_lora, LORA, dict(b=h(3, 24, 8)), "b must have shape"),
    (Z.zinc_lora, LORA, dict(b=h(2, 20, 8)), "multiple of 8 rows"),
    (Z.zinc_lora, LORA, dict(scales=torch.ones(3)), "scales"),
    (Z.zinc_lora, LORA, dict(offsets=i32(4)), "offsets"),
    (Z.zinc_lora, LORA, dict(slot_row=i32(4)), "slot_row"),
    (Z.zinc_lora, LORA, dict(row_slot=i32(4, 1)), "row_slot"),
    (Z.zinc_lora, LORA, dict(base=h(4, 16)), "base must have shape"),
    (Z.zinc_lora, LORA, dict(y=h(4, 24, dtype=torch.float32)), "y must be"),
    (Z.zinc_lora, LORA, dict(workspace=torch.zeros(16, dtype=torch.uint8)), "workspace holds"),
    (Z.zinc_lora_backward, LORA_BACK, dict(dy=h(4, 16)), "dy must have shape"),
    (Z.zinc_lora_backward, LORA_BACK, dict(base=h(4, 24)), "base must have shape"),
    (Z.zinc_lora_backward, LORA_BACK, dict(db=h(2, 8, 24)), "db must have shape"),
    (Z.zinc_lora_backward, LORA_BACK, dict(want_da=False, da=h(2, 8, 16)), "one at least"),
])
def test_wrong_tensors_raise_before_any_call(f, good, bad, msg):
    with pytest.raises(ValueError, match=msg):
        f(**dict(good, **bad))
