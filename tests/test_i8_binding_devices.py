"""The 8-bit calls refuse tensors of several GPUs, or of another than the current
one, before anything is launched (no GPU: stand-ins carry the attributes that
the binding reads, and the entry point counts its calls)."""
import ctypes

import pytest
import torch


class Stand:
    """What the binding reads of a CUDA tensor."""
    is_cuda = True

    def __init__(self, shape, dtype, device=0):
        self.shape, self.dtype, self._device = tuple(shape), dtype, device

    def stride(self):
        return (self.shape[1], 1) if len(self.shape) == 2 else (1,)

    def get_device(self):
        return self._device

    def data_ptr(self):
        return 0x1000


@pytest.fixture
def calls():
    """call(name, *arguments, current=0): the call through the binding with the
    current device given; returns how often the entry point was reached."""
    import dense_gemm_09_gb300 as dg
    dg.build()
    m, state = dg._calls(), {"device": 0}
    m.setup(torch.float32, torch.float16, torch.bfloat16, torch.int8, lambda: state["device"], lambda d: 0, dg.DgemmError)

    def call(name, *args, current=0):
        reached = []
        entry = ctypes.CFUNCTYPE(ctypes.c_int, *getattr(dg.lib(), name).argtypes)(lambda *a: reached.append(a) or 0)
        state["device"] = current
        getattr(m, name)(ctypes.cast(entry, ctypes.c_void_p).value, *args)
        return len(reached)

    yield call
    dg._calls_module = None
    dg._calls()


def _arguments(name, on):
    """The arguments of a call; on(key): the device of a tensor."""
    f, i = torch.float32, torch.int8
    mat = lambda key, dt, rows=4, cols=8: Stand((rows, cols), dt, on(key))
    vec = lambda key, n: Stand((n,), f, on(key))
    return {"quantize_i8": lambda: (mat("X", f), mat("Q", i), vec("scale", 4), None),
            "rmsnorm_i8": lambda: (mat("X", f), vec("gamma", 8), mat("Q", i), vec("scale", 4), mat("residual", f),
                                   mat("H", f), 1e-6, None),
            "swiglu_i8": lambda: (mat("G", f), mat("U", f), mat("Q", i), vec("scale", 4), None),
            "dequantize_i8": lambda: (mat("Q", i), vec("scale", 4), mat("X", f), None),
            "gemm_i8_tn": lambda: (mat("A", i), mat("B", i, 6), mat("C", f, 4, 6), vec("scale_a", 4), vec("scale_b", 6),
                                   vec("bias", 6), 0.0, None)}[name]()


TENSORS = {"quantize_i8": ("X", "Q", "scale"), "rmsnorm_i8": ("X", "gamma", "Q", "scale", "residual", "H"),
           "swiglu_i8": ("G", "U", "Q", "scale"), "dequantize_i8": ("Q", "scale", "X"),
           "gemm_i8_tn": ("A", "B", "C", "scale_a", "scale_b", "bias")}


@pytest.mark.parametrize("name", TENSORS)
def test_one_device(calls, name):
    for device in (0, 1, 7):
        assert calls(name, *_arguments(name, lambda key: device), current=device) == 1


@pytest.mark.parametrize("name,odd", [(n, t) for n, ts in TENSORS.items() for t in ts])
def test_a_tensor_on_another_device(calls, name, odd):
    for current in (0, 1):
        for here, there in ((0, 1), (1, 0)):
            with pytest.raises(ValueError, match="cuda:"):
                calls(name, *_arguments(name, lambda key: there if key == odd else here), current=current)


@pytest.mark.parametrize("name", TENSORS)
@pytest.mark.parametrize("stream", [None, 0x40])
def test_not_the_current_device(calls, name, stream):
    args = _arguments(name, lambda key: 1)[:-1] + (stream,)
    with pytest.raises(ValueError, match="the tensors are on cuda:1, the current device is cuda:0"):
        calls(name, *args, current=0)
    assert calls(name, *args, current=1) == 1
