"""The checks of arguments of the 8-bit floating-point calls and of the calls on tokens by
expert, in the library and in the binding (no GPU: validation comes first, and stand-ins carry
the attributes that the binding reads)."""
import ctypes

import pytest
import torch

P = 0x1000  # a non-null pointer value that is never dereferenced


@pytest.fixture(scope="module")
def L():
    import dense_gemm_09_gb300 as dg
    dg.build()
    return dg.lib()


def f8(**change):
    import dense_gemm_09_gb300 as dg
    return dg.F8Matrix(**dict(dict(data=P, ld=300, type=0, block=1, scale=P, scale_row=3, scale_blk=1), **change))


def valid():
    """The valid calls: names in order, and a call's own matrices."""
    return {
        "quantize_f8": dict(rows=4, cols=300, X=P, ldx=300, ty=0, transposed=0, Q=f8()),
        "swiglu_f8": dict(rows=4, cols=300, G=P, ldg=300, U=P, ldu=300, ty=0, Q=f8()),
        "dequantize_f8": dict(rows=4, cols=300, Q=f8(), X=P, ldx=300, ty=0),
        "gemm_f8_tn": dict(M=8, N=8, K=300, A=f8(), B=f8(), bias=None, beta=0.0, C=P, ldc=8, ty=0),
        "gemm_f8_tn_experts": dict(M=8, N=8, K=300, E=4, off=P, A=f8(), B=f8(), bs=2400, ss=24, C=P, ldc=8, ty=0),
        "sort_by_expert": dict(tokens=4, top=2, E=8, ids=P, bytes=4, off=P, pos=P),
        "gather_by_expert": dict(tokens=4, top=2, cols=8, X=P, ldx=8, ty=0, pos=P, rows=8, Y=P, ldy=8),
        "gather_by_expert_f8": dict(tokens=4, top=2, cols=300, X=P, ldx=300, ty=0, pos=P, rows=8, Q=f8()),
        "combine_experts": dict(tokens=4, top=2, cols=8, Y=P, ldy=8, rows=8, ty=0, pos=P, w=None, beta=0.0, X=P, ldx=8),
        "combine_experts_grad": dict(tokens=4, top=2, cols=8, dX=P, lddx=8, Y=P, ldy=8, rows=8, ty=0, pos=P, w=P, dY=P, lddy=8, dw=P),
    }


MATRIX = [dict(ld=299), dict(type=2), dict(type=-1), dict(block=0), dict(block=64), dict(scale_row=-1), dict(scale_blk=-1),
          dict(data=None), dict(scale=None)]
WRITTEN = [dict(scale_row=0), dict(scale_blk=0)]
BAD = [("quantize_f8", d) for d in (dict(rows=-1), dict(cols=-1), dict(ldx=299), dict(X=None), dict(ty=3), dict(rows=2 ** 31),
                                    dict(transposed=1, Q=dict(block=128, ld=4)), dict(transposed=1, Q=dict(ld=3)), dict(Q=None))]
BAD += [("swiglu_f8", d) for d in (dict(rows=-1), dict(ldg=299), dict(ldu=299), dict(G=None), dict(U=None), dict(ty=-1), dict(Q=dict(block=128)))]
BAD += [("dequantize_f8", d) for d in (dict(cols=-1), dict(ldx=299), dict(X=None), dict(ty=4))]
BAD += [("gemm_f8_tn", d) for d in (dict(M=-1), dict(N=-1), dict(K=-1), dict(ldc=7), dict(C=None), dict(ty=3), dict(M=2 ** 31),
                                    dict(K=2 ** 31, A=dict(ld=2 ** 31)), dict(M=2 ** 31 - 1, N=2 ** 31 - 1, ldc=2 ** 31),
                                    dict(A=None), dict(B=None))]
BAD += [("gemm_f8_tn_experts", d) for d in (dict(E=0), dict(E=1025), dict(off=None), dict(bs=-1), dict(ss=-1), dict(ldc=7), dict(C=None),
                                            dict(A=dict(block=128)), dict(M=-1), dict(ty=9))]
BAD += [("sort_by_expert", d) for d in (dict(tokens=-1), dict(top=-1), dict(E=0), dict(E=1025), dict(ids=None), dict(bytes=2),
                                        dict(off=None), dict(pos=None), dict(tokens=2 ** 20, top=2 ** 11))]
BAD += [("gather_by_expert", d) for d in (dict(tokens=-1), dict(cols=-1), dict(rows=-1), dict(ldx=7), dict(ldy=7), dict(X=None), dict(Y=None),
                                          dict(pos=None), dict(ty=3), dict(rows=2 ** 31))]
BAD += [("gather_by_expert_f8", d) for d in (dict(ldx=299), dict(X=None), dict(pos=None), dict(Q=dict(block=128)), dict(top=-1))]
BAD += [("combine_experts", d) for d in (dict(tokens=-1), dict(ldx=7), dict(ldy=7), dict(X=None), dict(Y=None), dict(pos=None), dict(ty=3))]
BAD += [("combine_experts_grad", d) for d in (dict(lddx=7), dict(ldy=7), dict(lddy=7), dict(dX=None), dict(Y=None), dict(dY=None), dict(w=None),
                                              dict(dw=None), dict(pos=None), dict(ty=3), dict(lddy=9))]
for name, key in (("quantize_f8", "Q"), ("swiglu_f8", "Q"), ("dequantize_f8", "Q"), ("gemm_f8_tn", "A"), ("gemm_f8_tn", "B"),
                  ("gemm_f8_tn_experts", "A"), ("gemm_f8_tn_experts", "B"), ("gather_by_expert_f8", "Q")):
    written = name in ("quantize_f8", "swiglu_f8", "gather_by_expert_f8")
    BAD += [(name, {key: d}) for d in MATRIX + (WRITTEN if written else [])]


def call(L, name, change):
    args = valid()[name]
    for key, v in change.items():
        args[key] = f8(**v) if isinstance(v, dict) else v
    if name == "combine_experts_grad" and change == dict(lddy=9):  # in place, at another pitch
        args["dY"] = args["Y"]
    vals = [ctypes.byref(v) if isinstance(v, ctypes.Structure) else v for v in args.values()]
    return getattr(L, name)(*vals, None)


@pytest.mark.parametrize("name,change", BAD, ids=["%s-%s" % (n, str(c)) for n, c in BAD])
def test_invalid_arguments(L, name, change):
    assert call(L, name, change) == 1


@pytest.mark.parametrize("name", ["quantize_f8", "swiglu_f8", "dequantize_f8", "gemm_f8_tn", "gemm_f8_tn_experts",
                                                              "gather_by_expert", "gather_by_expert_f8", "combine_experts"])
def test_nothing_to_do(L, name):
    for key in ("rows", "cols", "M", "N", "tokens"):
        if key in valid()[name] and not (name == "combine_experts" and key == "rows"):
            nulls = {k: None for k in ("X", "Y", "G", "U", "C", "pos") if k in valid()[name]}
            mats = {k: dict(data=None, scale=None) for k in ("Q", "A", "B") if k in valid()[name]}
            assert call(L, name, dict(nulls, **mats, **{key: 0})) == 0, key


@pytest.mark.skipif(torch.cuda.is_available(), reason="only meaningful without a GPU")
@pytest.mark.parametrize("name", ["quantize_f8", "swiglu_f8", "dequantize_f8", "gemm_f8_tn", "gemm_f8_tn_experts", "sort_by_expert",
                                  "gather_by_expert", "gather_by_expert_f8", "combine_experts", "combine_experts_grad"])
def test_no_gpu(L, name):
    assert call(L, name, {}) == 2  # valid, and no device to run on


def test_tune_requests_are_checked_and_taken_once(L):
    import dense_gemm_09_gb300 as dg
    for cfg in ((2, 64, 1), (3, 128, 1), (3, 16, 9), (4, 0, 16), (5, 0, 0), (-1, 0, 0)):
        with pytest.raises(dg.DgemmError):
            dg.tune_f8_next(*cfg)
    for cfg in ((0, 0, 1), (1, 0, 1), (2, 128, 1), (2, 256, 1), (3, 16, 8), (4, 0, 4)):
        dg.tune_f8_next(*cfg)
    with pytest.raises((TypeError, ValueError)):
        dg.gemm_f8_tn(None, None, None, None, None)


# ---- the binding

F, I32, I64, E4 = torch.float32, torch.int32, torch.int64, torch.float8_e4m3fn


class Stand:
    """What the binding reads of a CUDA tensor."""
    is_cuda = True

    def __init__(self, shape, dtype, device=0, stride=None):
        self.shape, self.dtype, self._device = tuple(shape), dtype, device
        if stride is None:
            stride, n = [], 1
            for s in reversed(self.shape):
                stride.insert(0, n)
                n *= s
        self._stride = tuple(stride)

    def stride(self):
        return self._stride

    def get_device(self):
        return self._device

    def data_ptr(self):
        return 0x1000


@pytest.fixture
def calls():
    """call(name, *arguments, current=0): the arguments that the entry point got (None if it was not
    reached)."""
    import dense_gemm_09_gb300 as dg
    dg.build()
    m, state = dg._calls(), {"device": 0}
    m.setup(torch.float32, torch.float16, torch.bfloat16, torch.int8, lambda: state["device"], lambda d: 0, dg.DgemmError,
            torch.float8_e4m3fn, torch.float8_e5m2, torch.int32, torch.int64)

    def run(name, *args, current=0):
        got = []

        def entry(*a):
            got.append([(v.contents.block, v.contents.scale_row, v.contents.scale_blk, v.contents.type) if isinstance(v, ctypes.POINTER(dg.F8Matrix))
                        else v for v in a])
            return 0

        fn = ctypes.CFUNCTYPE(ctypes.c_int, *getattr(dg.lib(), name).argtypes)(entry)
        state["device"] = current
        getattr(m, name)(ctypes.cast(fn, ctypes.c_void_p).value, *args)
        return got[0]

    yield run
    dg._calls_module = None
    dg._calls()


def tensors(name, on=lambda key: 0):
    """The call's arguments by name, in order."""
    t = lambda key, shape, dt=F, **kw: (key, Stand(shape, dt, on(key), **kw))
    return dict({
        "quantize_f8": [t("X", (4, 300)), t("Q", (4, 300), E4), t("scale", (4, 3)), ("transposed", False)],
        "swiglu_f8": [t("G", (4, 300)), t("U", (4, 300)), t("Q", (4, 300), E4), t("scale", (4, 3))],
        "dequantize_f8": [t("Q", (4, 300), E4), t("scale", (4, 3)), t("X", (4, 300))],
        "gemm_f8_tn": [t("A", (5, 300), E4), t("B", (200, 300), E4), t("C", (5, 200)), t("scale_a", (5, 3)), t("scale_b", (2, 3)), t("bias", (200,)),
                       ("beta", 0.0)],
        "gemm_f8_tn_experts": [t("A", (5, 300), E4), t("B", (3, 200, 300), E4), t("C", (5, 200)), t("scale_a", (5, 3)), t("scale_b", (3, 2, 3)),
                               t("offsets", (4,), I32)],
        "sort_by_expert": [t("experts", (6, 2), I64), t("offsets", (9,), I32), t("position", (6, 2), I32)],
        "gather_by_expert": [t("X", (6, 40)), t("position", (6, 2), I32), t("Y", (12, 40))],
        "gather_by_expert_f8": [t("X", (6, 40)), t("position", (6, 2), I32), t("Q", (12, 40), E4), t("scale", (12, 1))],
        "combine_experts": [t("Y", (12, 40)), t("position", (6, 2), I32), t("weights", (6, 2)), t("X", (6, 40)), ("beta", 0.0)],
        "combine_experts_grad": [t("dX", (6, 40)), t("Y", (12, 40)), t("position", (6, 2), I32), t("weights", (6, 2)), t("dY", (12, 40)),
                                 t("dweights", (6, 2))],
    }[name])


NAMES = ["quantize_f8", "swiglu_f8", "dequantize_f8", "gemm_f8_tn", "gemm_f8_tn_experts", "sort_by_expert", "gather_by_expert",
         "gather_by_expert_f8", "combine_experts", "combine_experts_grad"]
EACH = [(n, k) for n in NAMES for k, v in tensors(n).items() if isinstance(v, Stand)]


@pytest.mark.parametrize("name", NAMES)
def test_the_call_goes_through(calls, name):
    for device in (0, 3):
        assert calls(name, *tensors(name, lambda key: device).values(), None, current=device)


@pytest.mark.parametrize("name,odd", EACH)
def test_a_tensor_on_another_device_or_the_host(calls, name, odd):
    with pytest.raises(ValueError, match="cuda:"):
        calls(name, *tensors(name, lambda key: int(key == odd)).values(), None)
    args = tensors(name)
    args[odd].is_cuda = False
    with pytest.raises(ValueError, match="CUDA tensor"):
        calls(name, *args.values(), None)


@pytest.mark.parametrize("name", NAMES)
def test_not_the_current_device(calls, name):
    with pytest.raises(ValueError, match="the current device is cuda:0"):
        calls(name, *tensors(name, lambda key: 1).values(), None)


@pytest.mark.parametrize("name,odd", EACH)
def test_a_wrong_type_or_shape(calls, name, odd):
    args = tensors(name)
    args[odd].dtype = torch.float64
    with pytest.raises(TypeError):
        calls(name, *args.values(), None)
    args = tensors(name)
    shape = args[odd].shape
    # (the number of experts and of choices are what the call says)
    if (name, odd) not in (("sort_by_expert", "offsets"), ("gather_by_expert", "position"), ("gather_by_expert_f8", "position")):
        args[odd] = Stand(shape[:-1] + (shape[-1] + 130,), args[odd].dtype)
        with pytest.raises(ValueError):
            calls(name, *args.values(), None)
    args[odd] = Stand((2,) + shape, args[odd].dtype)
    with pytest.raises(ValueError):
        calls(name, *args.values(), None)


def test_blocks_by_the_scales_shape(calls):
    a = tensors("gemm_f8_tn")
    got = calls("gemm_f8_tn", *a.values(), None)
    assert got[3] == (1, 3, 1, 0) and got[4] == (128, 3, 1, 0)
    a["scale_b"] = Stand((200, 3), F, stride=(1, 200))  # K-major
    a["scale_a"] = Stand((1, 3), F, stride=(0, 0))
    assert calls("gemm_f8_tn", *a.values(), None)[3:5] == [(128, 1, 0, 0), (1, 1, 200, 0)]
    a["B"] = Stand((200, 300), torch.float8_e5m2)
    assert calls("gemm_f8_tn", *a.values(), None)[4][3] == 1


def test_layouts_that_are_refused(calls):
    a = tensors("quantize_f8")
    with pytest.raises(ValueError, match="overlapping"):  # scales are written
        calls("quantize_f8", a["X"], a["Q"], Stand((4, 3), F, stride=(0, 1)), False, None)
    with pytest.raises(ValueError, match="a scale for each row"):
        calls("quantize_f8", Stand((300, 200), F), Stand((200, 300), E4), Stand((2, 3), F), True, None)
    with pytest.raises(ValueError, match="unit column stride"):
        calls("quantize_f8", Stand((4, 300), F, stride=(1, 4)), a["Q"], a["scale"], False, None)
    with pytest.raises(ValueError, match="must have a row for each row"):
        calls("swiglu_f8", Stand((200, 300), F), Stand((200, 300), F), Stand((200, 300), E4), Stand((2, 3), F), None)
    a = tensors("sort_by_expert")
    with pytest.raises(ValueError, match="contiguous"):
        calls("sort_by_expert", Stand((6, 2), I32, stride=(4, 1)), a["offsets"], a["position"], None)
    with pytest.raises(ValueError, match="number of experts"):
        calls("sort_by_expert", a["experts"], Stand((1,), I32), a["position"], None)
    a = tensors("gemm_f8_tn_experts")
    a["B"] = Stand((3, 200, 300), E4, stride=(60000, 1, 200))
    with pytest.raises(ValueError, match="unit column stride"):
        calls("gemm_f8_tn_experts", *a.values(), None)
    a["B"] = Stand((3, 200, 300), E4, stride=(60000, 100, 1))
    with pytest.raises(ValueError, match="overlapping"):
        calls("gemm_f8_tn_experts", *a.values(), None)


def test_cpu_tensors(L):
    import dense_gemm_09_gb300 as dg
    with pytest.raises(ValueError, match="X must be a CUDA tensor"):
        dg.quantize_f8(torch.ones(2, 8), torch.zeros(2, 8).to(E4), torch.zeros(2, 1))
    with pytest.raises(TypeError, match="C must be"):
        dg.gemm_f8_tn(*[torch.zeros(2, 8, dtype=torch.int8)] * 5)
