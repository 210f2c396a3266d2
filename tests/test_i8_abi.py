"""The 8-bit calls' checks of their arguments (no GPU: validation comes first)."""
import ctypes

import pytest
import torch

P = 0x1000  # a non-null pointer value that is never dereferenced


@pytest.fixture(scope="module")
def L():
    import dense_gemm_09_gb300 as dg
    dg.build()
    return dg.lib()


NAN = float("nan")
# the valid calls; each entry of BAD changes some of their arguments
GEMM = dict(M=8, N=8, K=8, A=P, lda=8, sa=P, B=P, ldb=8, sb=P, bias=None, beta=0.0, C=P, ldc=8, ty=0)
QUANT = dict(rows=4, cols=8, X=P, ldx=8, ty=0, Q=P, ldq=8, s=P)
NORM = dict(rows=4, cols=8, X=P, ldx=8, R=P, ldr=8, g=P, gty=0, eps=1e-6, ty=0, H=P, ldh=8, Q=P, ldq=8, s=P)
SWIGLU = dict(rows=4, cols=8, G=P, ldg=8, U=P, ldu=8, ty=0, Q=P, ldq=8, s=P)
DEQUANT = dict(rows=4, cols=8, Q=P, ldq=8, s=P, X=P, ldx=8, ty=0)
CALLS = {"gemm_i8_tn": GEMM, "quantize_i8": QUANT, "rmsnorm_i8": NORM, "swiglu_i8": SWIGLU, "dequantize_i8": DEQUANT}

BAD = [("gemm_i8_tn", d) for d in (
    dict(M=-1), dict(N=-1), dict(K=-1), dict(lda=7), dict(ldb=7), dict(ldc=7), dict(A=None), dict(B=None),
    dict(C=None), dict(sa=None), dict(sb=None), dict(ty=3), dict(ty=-1), dict(M=2**40, N=2**40, lda=8, ldc=2**40))]
BAD += [("quantize_i8", d) for d in (
    dict(rows=-1), dict(cols=-1), dict(ldx=7), dict(ldq=7), dict(X=None), dict(Q=None), dict(s=None), dict(ty=5),
    dict(rows=2**31))]
BAD += [("rmsnorm_i8", d) for d in (
    dict(rows=-1), dict(cols=-1), dict(ldx=7), dict(ldr=7), dict(ldh=7), dict(ldq=7), dict(X=None), dict(g=None),
    dict(Q=None), dict(s=None), dict(ty=5), dict(gty=1), dict(ty=1, gty=2), dict(eps=-1e-6), dict(eps=NAN))]
BAD += [("swiglu_i8", d) for d in (
    dict(rows=-1), dict(ldg=7), dict(ldu=7), dict(ldq=7), dict(G=None), dict(U=None), dict(Q=None), dict(s=None),
    dict(ty=-1))]
BAD += [("dequantize_i8", d) for d in (
    dict(rows=-1), dict(cols=-1), dict(ldq=7), dict(ldx=7), dict(Q=None), dict(s=None), dict(X=None), dict(ty=3))]


@pytest.mark.parametrize("name,change", BAD, ids=["%s-%s" % (n, "-".join(c)) for n, c in BAD])
def test_invalid_arguments(L, name, change):
    assert getattr(L, name)(*dict(CALLS[name], **change).values(), None) == 1


@pytest.mark.parametrize("name", CALLS)
def test_nothing_to_do(L, name):
    for key in ("rows", "cols", "M", "N"):
        if key in CALLS[name]:
            args = {k: (None if v == P else v) for k, v in CALLS[name].items()}
            assert getattr(L, name)(*dict(args, **{key: 0}).values(), None) == 0


@pytest.mark.skipif(torch.cuda.is_available(), reason="only meaningful without a GPU")
@pytest.mark.parametrize("name", CALLS)
def test_no_gpu(L, name):
    assert getattr(L, name)(*CALLS[name].values(), None) == 2


@pytest.mark.skipif(torch.cuda.is_available(), reason="only meaningful without a GPU")
def test_optional_pointers(L):
    # what may be NULL passes validation (and then finds no GPU)
    assert L.gemm_i8_tn(*dict(GEMM, bias=None).values(), None) == 2
    assert L.gemm_i8_tn(*dict(GEMM, K=0, A=None, B=None).values(), None) == 2
    assert L.rmsnorm_i8(*dict(NORM, R=None, ldr=0, H=None, ldh=0).values(), None) == 2


def test_types_are_what_the_header_says(L):
    import dense_gemm_09_gb300 as dg
    assert L.gemm_i8_tn.restype is ctypes.c_int
    assert all(dg.lib().i8_entry[n] for n in CALLS)


def test_binding_checks_tensors_before_the_device(L):
    # CPU tensors reach the checks of the marshalling module, not the library
    import dense_gemm_09_gb300 as dg
    x, q, s = torch.ones((2, 8)), torch.zeros((2, 8), dtype=torch.int8), torch.zeros(2)
    with pytest.raises(ValueError, match="X must be a CUDA tensor"):
        dg.quantize_i8(x, q, s)
    with pytest.raises(ValueError, match="X must be a 2-D tensor"):
        dg.quantize_i8(x[0], q, s)
    with pytest.raises(TypeError, match="X must be a float32, float16 or bfloat16 tensor"):
        dg.quantize_i8(q, q, s)
    with pytest.raises(TypeError, match="X must be a float32"):
        dg.dequantize_i8(q, s, None)
    with pytest.raises(TypeError, match="X must be"):
        dg.rmsnorm_i8([1.0], s, q, s)
    with pytest.raises(TypeError, match="C must be"):
        dg.gemm_i8_tn(q, q, q, s, s)
    with pytest.raises(TypeError):
        dg._calls().quantize_i8(1, x)  # too few arguments


def test_binding_fails_loudly_without_the_marshalling_module(monkeypatch):
    import sys

    import dense_gemm_09_gb300 as dg
    monkeypatch.setattr(dg, "_calls_module", None)
    monkeypatch.setitem(sys.modules, "dense_gemm_09_gb300._i8_calls", None)
    with pytest.raises(RuntimeError, match="not built"):
        dg.quantize_i8(None, None, None)
