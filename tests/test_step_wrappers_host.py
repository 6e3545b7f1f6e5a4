"""What the wrappers of the target's step refuse before they call the library: tensors of another GPU than the engine's, and
sizes that an int of 32 bits does not hold.  On the host alone, with stand-ins for tensors."""
import math

import pytest
import torch


class Tensor:
    """What the wrappers look at of a tensor."""

    def __init__(self, *shape, dtype=torch.float32, gpu=0, pitch=None):
        self.shape, self.dtype, self.device, self.is_cuda = tuple(shape), dtype, torch.device("cuda", gpu), True
        self.pitch = shape[-1] if pitch is None else pitch

    def stride(self, i):
        return 1 if i == len(self.shape) - 1 else self.pitch

    def numel(self):
        return math.prod(self.shape)

    def is_contiguous(self):
        return self.pitch == self.shape[-1]

    def data_ptr(self):
        return 1 << 20


CALLS = ["eagle_mx_quantize", "eagle_mx_unpack", "eagle_mx_linear", "eagle_add_norm", "eagle_sample"]


@pytest.fixture()
def env(monkeypatch):
    """(runtime, engine, calls that reached the library); the engine is on GPU 0."""
    from eagle_feature_level_gb300.build import build
    build()
    from eagle_feature_level_gb300 import runtime as R
    reached = []
    for name in CALLS:
        monkeypatch.setattr(R.B, name, lambda *a, name=name: reached.append(name))

    class Engine:
        ctx, device, ws = None, torch.device("cuda"), Tensor(1, dtype=torch.uint8)
        dims_c = R.B.eagle_dims(64, 4, 4, 16, 64, 64, 1e-5, 1e4)
        dims = dict(vocab=64)

        def stream(self):
            return 0
    return R, Engine(), reached


def matrix(R, eng, rows, cols, fmt="fp8", gpu=0, factor=None):
    data, scale = R.B.eagle_mx_layout(R.MX_FORMATS[fmt], rows, cols)
    u8 = lambda n: Tensor(n, dtype=torch.uint8, gpu=gpu)
    return R.MxTensor(eng, rows, cols, fmt, factor, u8(data), u8(scale))


def elsewhere(R, eng, rows, cols):
    """A matrix of an engine on GPU 1."""
    other = type(eng)()
    other.ws = Tensor(1, dtype=torch.uint8, gpu=1)
    return matrix(R, other, rows, cols, gpu=1)


def test_every_tensor_is_on_the_engines_gpu(env):
    R, eng, reached = env
    a, b = matrix(R, eng, 4, 64), matrix(R, eng, 8, 64)
    far = elsewhere(R, eng, 8, 64)
    i32 = lambda n, gpu=0: Tensor(n, dtype=torch.int32, gpu=gpu)
    t = lambda gpu=0: Tensor(4, 64, gpu=gpu)
    s = R.Sampler(eng, 4, Tensor(4))
    good = [lambda: a.quantize(t()), lambda: a.unpack(t()), lambda: R.mx_linear(a, b, Tensor(4, 8), Tensor(8)),
            lambda: R.add_norm(eng, t(), t(), Tensor(64), t(), t()), lambda: R.add_norm(eng, t(), a),
            lambda: s(t(), i32(4), i32(4), i32(4), t())]
    for call in good:
        call()
    assert reached == ["eagle_mx_quantize", "eagle_mx_unpack", "eagle_mx_linear", "eagle_add_norm", "eagle_add_norm", "eagle_sample"]
    bad = [lambda: matrix(R, eng, 4, 64, gpu=1), lambda: matrix(R, eng, 4, 64, "nv4", 0, Tensor(1, gpu=1)),
           lambda: a.quantize(t(1)), lambda: a.unpack(t(1)),
           lambda: R.mx_linear(a, far, Tensor(4, 8)), lambda: R.mx_linear(a, b, Tensor(4, 8, gpu=1)),
           lambda: R.mx_linear(a, b, Tensor(4, 8), Tensor(8, gpu=1)),
           # all of them on the other GPU, too
           lambda: R.add_norm(eng, t(1), t(1)), lambda: R.add_norm(eng, t(1), t(1), Tensor(64, gpu=1), t(1), t(1)),
           lambda: R.add_norm(eng, t(), t(1)), lambda: R.add_norm(eng, t(), t(), Tensor(64, gpu=1)),
           lambda: R.add_norm(eng, t(), t(), residual=t(1)), lambda: R.add_norm(eng, t(), t(), residual_out=t(1)),
           lambda: R.add_norm(eng, Tensor(8, 64), far),
           lambda: R.Sampler(eng, 4, Tensor(4, gpu=1)), lambda: R.Sampler(eng, 4, top_k=i32(4, 1)),
           lambda: R.Sampler(eng, 4, Tensor(4), rows_used=i32(4, 1)),
           lambda: s(t(1), argmax=i32(4, 1)), lambda: s(t(1), i32(4, 1), i32(4, 1), i32(4, 1), t(1)),
           lambda: s(t(), i32(4, 1), i32(4)), lambda: s(t(), probs=t(1))]
    for call in bad:
        with pytest.raises(ValueError):
            call()
    assert len(reached) == len(good)


def test_a_rounds_filter_is_on_its_engines_gpu(env):
    R, eng, _ = env
    rd = R.Round.__new__(R.Round)
    rd.eng, rd.B, rd.S, rd.temps, rd.t_size = eng, 4, 3, Tensor(4), Tensor(4, dtype=torch.int32)
    rd.set_filter(top_p=Tensor(4))
    assert rd.filter_c.rows_each == 3
    with pytest.raises(ValueError):
        rd.set_filter(top_p=Tensor(4, gpu=1))
    rd.temps, rd.t_size = Tensor(4, gpu=1), Tensor(4, dtype=torch.int32, gpu=1)
    with pytest.raises(ValueError):
        rd.set_filter(top_p=Tensor(4, gpu=1))


def test_sizes_that_an_int_does_not_hold(env):
    """As 32 bits they would look like the right ones."""
    R, eng, reached = env
    big = 1 << 32
    a = matrix(R, eng, 4, 64)
    far = lambda dtype=torch.float32: Tensor(4, 64, dtype=dtype, pitch=big + 64)
    s = R.Sampler(eng, 4)
    for call in (lambda: a.quantize(far()), lambda: a.unpack(far(torch.bfloat16)),
                 lambda: R.mx_linear(a, matrix(R, eng, 64, 64), far()),
                 lambda: R.add_norm(eng, far(), Tensor(4, 64)), lambda: R.add_norm(eng, Tensor(4, 64), far()),
                 lambda: R.add_norm(eng, Tensor(4, 64), Tensor(4, 64), residual=far()),
                 lambda: s(far(), argmax=Tensor(4, dtype=torch.int32)), lambda: s(Tensor(4, 64), probs=far()),
                 lambda: R.add_norm(eng, Tensor(big + 4, 64), Tensor(big + 4, 64)),
                 lambda: R.Sampler(eng, 1, rows_each=big + 4)):
        with pytest.raises(ValueError):
            call()
    assert reached == []
    a.quantize(Tensor(4, 64, pitch=(1 << 31) - 64))
    assert reached == ["eagle_mx_quantize"]
