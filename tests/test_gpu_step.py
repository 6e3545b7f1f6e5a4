"""The target's step around its cache on the GPU: eagle_add_norm, eagle_mx_quantize, eagle_mx_unpack, eagle_mx_linear and
eagle_sample against the oracle (oracle/step.py, fp64), alone and strung together with the cache's calls.

Tolerances, fixed before the first run (u(t) = half a step of type t relative to the value: bf16 2^-8 with the last bit of
fp32 work before it, fp32 2^-24):
* quantisation of given rows: codes and scales are the definition's, bit for bit; behind fp32 arithmetic (SiLU, norms)
  that is off by at most REL = 2^-18 of a value, each block's scale is that of a largest magnitude within REL, and each
  element is a nearest one for that scale to a value within REL (plus the fp32 quotient's 2^-23);
* norms: one fp32 rounding of the sum; the mean of squares sums at most 8 * 4 terms a thread and 10 levels of pairs, 42
  roundings of 2^-24 at most, halved by the root, and five more roundings: below 2^-18 in all;
* products: operands are exact; each of the K additions (and the alignment before it) loses at most 2^-23 of the sum of
  magnitudes so far, a further 8 for split sums, factors and the bias: (K + 8) 2^-23 sum |x w|, then one rounding;
* sampling: a weight is off by at most 2 units of 2^-40, so sums by 2 V: a border of top_p or of the draw may fall on either
  side within that; probabilities by 2^-22 relative."""
import math
import random

import numpy as np
import pytest
import torch

from eagle_feature_level_gb300 import _binding as B
from eagle_feature_level_gb300 import runtime as R
from eagle_feature_level_gb300.runtime import _p
from oracle import step as O
from oracle.sampling import draw_one

pytestmark = pytest.mark.gpu

INVALID_ARG, SHAPE, ALIGN, CAPACITY, NUMERIC = 1, 2, 3, 4, 6
BF16, F32 = torch.bfloat16, torch.float32
U = {BF16: 2.0 ** -8, F32: 2.0 ** -24}
REL = 2.0 ** -18
NAN, INF = float("nan"), float("inf")
_engine = []


def engine():
    if not _engine:
        _engine.append(R.Engine(dict(d=512, n_q_heads=4, n_kv_heads=2, head_dim=64, d_ff=64, vocab=64), max_batch=64,
                                max_rows=8, max_expanded=1, max_children=1, max_tree=2, max_prefix=1024, device="cuda"))
    return _engine[0]


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def normal(seed, *shape, dtype=F32):
    return torch.randn(*shape, generator=gen(seed), device="cuda").to(dtype)


def f64(t):
    return t.detach().double().cpu().numpy()


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def f32(x):
    return torch.tensor(x, dtype=F32, device="cuda")


def pitched(t, more):
    """The same values with rows `more` elements further apart, the gaps NaN."""
    wide = torch.full((t.shape[0], t.shape[1] + more), NAN, dtype=t.dtype, device="cuda")
    wide[:, :t.shape[1]] = t
    return wide[:, :t.shape[1]]


def mx(fmt, rows, cols, g=None):
    t = R.MxTensor(engine(), rows, cols, fmt, None if g is None else f32([g]))
    t.data.fill_(0xa5)
    t.scale.fill_(0xff)                                  # NaN scales where nothing is written
    return t


def codes(t):
    n = t.rows * t.cols // (1 if t.fmt == "fp8" else 2)
    return O.unpack_bytes(t.fmt, t.data[:n].cpu().numpy(), t.scale.cpu().numpy(), t.rows, t.cols)


def factor(t):
    return 1.0 if t.tensor_scale is None else float(t.tensor_scale.reshape(-1)[0])


def held(t):
    c, b = codes(t)
    return O.values(t.fmt, c, b[:, :t.cols // O.BLOCK[t.fmt]], factor(t))


def is_quantized(t, y, rel=0.0):
    code, byte = codes(t)
    n = t.cols // O.BLOCK[t.fmt]
    assert not byte[:, n:].any()
    byte = byte[:, :n]
    want_code, want_byte = O.quantize(t.fmt, y, factor(t))
    if rel == 0.0:
        assert np.array_equal(byte, want_byte)
        assert np.array_equal(code, want_code)
        return
    near = [O.quantize(t.fmt, y * (1 + d), factor(t))[1] for d in (-rel, rel)]
    assert ((byte == near[0]) | (byte == near[1])).all()
    v = O.values(t.fmt, np.zeros_like(code), byte, factor(t))      # shapes
    s = (O.E4M3[byte].astype(np.float32) * np.float32(factor(t))).astype(np.float64) if t.fmt == "nv4" else \
        2.0 ** (byte.astype(float) - 127)
    s = s.repeat(O.BLOCK[t.fmt], 1)
    q = np.where(s > 0, y / np.where(s > 0, s, 1), 0)
    table = O.E4M3 if t.fmt == "fp8" else O.E2M1
    mag, sign = (code & 127, code >> 7) if t.fmt == "fp8" else (code & 7, code >> 3)
    lo, hi = O.nearest_code(table, np.abs(q) * (1 - rel - 2.0 ** -23)), O.nearest_code(table, np.abs(q) * (1 + rel + 2.0 ** -23))
    assert ((mag >= lo) & (mag <= hi)).all()
    assert ((sign == np.signbit(q)) | (mag == 0)).all() and v.shape == code.shape


FORMATS = ["fp8", "fp4", "nv4"]
SHAPES = [(1, 32), (1, 4096), (3, 96), (31, 160), (33, 64), (127, 1056), (129, 256), (260, 288), (700, 32)]


# ---- quantisation ---------------------------------------------------------------

@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("shape", SHAPES)
def test_quantize_and_unpack(fmt, dtype, shape):
    x = normal(1, *shape) * torch.exp(3 * normal(2, shape[0], 1)) * torch.exp(normal(3, 1, shape[1]))
    x[0, :32] = 0
    x[-1, -16:] = x[-1, -16:].sign() * 2.0 ** -20
    x = pitched(x.to(dtype), 8)
    g = float(x.abs().max()) / 2688 if fmt == "nv4" else None
    t = mx(fmt, *shape, g).quantize(x)
    is_quantized(t, f64(x))
    for out in (BF16, F32):
        y = pitched(torch.zeros(shape, dtype=out, device="cuda"), 16)
        t.unpack(y)
        want = held(t)
        assert (np.abs(f64(y) - want) <= U[out] * np.abs(want) + 2.0 ** -24 * np.abs(want)).all()
    assert engine().status() == 0


@pytest.mark.parametrize("fmt", FORMATS)
def test_quantize_borders(fmt):
    """Exact ties, largest magnitudes at the scale's borders, tiny and huge blocks, signed zeros."""
    rows = []
    for e in (-130, -126, -100, -20, -1, 0, 1, 20, 100, 125):
        for m in (1.0, 1.25, 1.5, 1.5 + 2.0 ** -23, 1.75, 1.75 + 2.0 ** -23, 2 - 2.0 ** -23):
            top = m * 2.0 ** e
            r = np.array([top, -top] + [top * k / 48 for k in range(1, 31)])
            rows.append(r)
    for k in range(8):
        rows.append(np.array([6.0, -5.0, 3.5, -3.5, 2.5, 1.75, 1.25, 0.75, 0.25, -0.25, -0.0, 0.0, 5.0, 4.5, 1e-30, -1e-30] * 2) *
                    2.0 ** (k - 4))
    x = torch.tensor(np.array(rows), dtype=F32, device="cuda")
    t = mx(fmt, *x.shape, 2.0 ** 100 if fmt == "nv4" else None).quantize(x)
    is_quantized(t, f64(x))
    if fmt == "nv4":
        for g in (1.0, 0.37, 2.0 ** -90):
            t = mx(fmt, *x.shape, g).quantize(x)
            is_quantized(t, f64(x))
        t = mx(fmt, *x.shape).quantize(x)                # no factor: 1
        is_quantized(t, f64(x))


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("shape", [(1, 32), (5, 11008), (130, 96)])
def test_quantize_gated(fmt, dtype, shape):
    x = (normal(4, shape[0], 2 * shape[1]) * 3).to(dtype)
    x[0, 0], x[0, 1] = -200.0, 200.0                     # SiLU's far ends
    t = mx(fmt, *shape, 0.01 if fmt == "nv4" else None).quantize(pitched(x, 24), swiglu=True)
    y = O.swiglu(f64(x))
    # exp is off by 2 steps (2^-22), 1 + exp, the quotient and the product by one each
    is_quantized(t, y, 2.0 ** -21)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("value", [NAN, INF, -INF])
def test_quantize_reports_non_finite_blocks(fmt, value):
    x = normal(5, 4, 128)
    x[2, 70] = value
    t = mx(fmt, 4, 128, 0.01).quantize(x)
    assert engine().status() == NUMERIC
    y = t.unpack(torch.empty(4, 128, device="cuda"))
    b = O.BLOCK[fmt]
    bad = torch.zeros(4, 128, dtype=torch.bool, device="cuda")
    bad[2, 70 // b * b:70 // b * b + b] = True
    assert torch.equal(torch.isnan(y), bad)
    w = mx(fmt, 40, 128, 0.01).quantize(normal(6, 40, 128))
    out = R.mx_linear(t, w, torch.empty(4, 40, device="cuda"))
    assert torch.isnan(out[2]).all() and torch.isfinite(out[[0, 1, 3]]).all()
    assert engine().status() == 0


# ---- linear layers ----------------------------------------------------------------

def check_linear(fmt, rows, cols, outs, out=BF16, bias=False, seed=0, more=0, g=(0.02, 0.003)):
    a, b = (g if fmt == "nv4" else (None, None))
    x = mx(fmt, rows, cols, a).quantize(normal(seed + 1, rows, cols) * torch.exp(0.5 * normal(seed + 2, 1, cols)))
    w = mx(fmt, outs, cols, b).quantize(normal(seed + 3, outs, cols) * 0.1)
    bs = normal(seed + 4, outs) if bias else None
    ld = (outs + 7) // 8 * 8 + more
    y = torch.full((rows + 1, ld), 77.0, dtype=out, device="cuda")
    R.mx_linear(x, w, y[:rows, :outs], bs)
    xv, wv = (torch.tensor(held(t), device="cuda") for t in (x, w))
    want, size = xv @ wv.t(), xv.abs() @ wv.abs().t()
    if bias:
        want, size = want + bs.double(), size + bs.double().abs()
    err = (y[:rows, :outs].double() - want).abs()
    assert bool((err <= (cols + 8) * 2.0 ** -23 * size + U[out] * want.abs()).all()), float((err / size).max())
    # nothing behind the outputs and the rows
    assert bool((y[rows:] == 77).all()) and bool((y[:, outs:] == 77).all())
    assert engine().status() == 0


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("rows", [1, 2, 15, 16, 17, 31, 64, 65, 100, 128, 129, 191, 192, 193, 250, 320, 500])
def test_linear_rows(fmt, rows):
    check_linear(fmt, rows, 512, 300, seed=rows)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("cols", [32, 64, 96, 128, 160, 224, 256, 288, 384, 992, 2080, 5120, 11008])
def test_linear_inner(fmt, cols):
    check_linear(fmt, 9, cols, 200, F32, seed=cols)
    check_linear(fmt, 200, cols, 130, F32, seed=cols + 1)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("outs", [1, 7, 8, 127, 128, 129, 1000, 20000])
def test_linear_outputs(fmt, outs):
    check_linear(fmt, 5, 1024, outs, BF16, True, seed=outs, more=8)
    check_linear(fmt, 140, 256, outs, F32, True, seed=outs + 1)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("shape", [(1, 4096, 12288), (8, 8192, 1024), (40, 8192, 4096), (777, 1024, 2500), (2000, 512, 3000),
                                   (600, 320, 9000), (4097, 96, 257)])
def test_linear_large(fmt, shape):
    check_linear(fmt, *shape, bias=True)


@pytest.mark.parametrize("fmt", FORMATS)
def test_linear_exact_products(fmt):
    """Whole numbers whose sums fit in fp32: every product and sum is exact, so a wrong scale or element anywhere shows."""
    rows, cols, outs = 150, 640, 190
    r = np.random.default_rng(7)
    def make(n):
        t = mx(fmt, n, cols)
        code = r.integers(0, 16, (n, cols)) if fmt != "fp8" else np.where(r.random((n, cols)) < 0.5, 0x38, 0x40) | \
            (r.integers(0, 2, (n, cols)) << 7)
        blocks = cols // O.BLOCK[fmt]
        byte = r.integers(126, 129, (n, blocks)) if fmt != "nv4" else r.choice([0x30, 0x38, 0x40], (n, blocks))
        data, scale = O.pack_bytes(fmt, code.astype(np.uint8), byte.astype(np.uint8), 0xff if fmt != "nv4" else 0x7f)
        t.data.copy_(torch.tensor(data.reshape(-1)))
        t.scale.copy_(torch.tensor(scale))
        return t
    x, w = make(rows), make(outs)
    y = R.mx_linear(x, w, torch.empty(rows, 192, device="cuda")[:, :outs])
    assert np.array_equal(f64(y), held(x) @ held(w).T)


def test_linear_shared_rows_of_a_buffer():
    """The first rows of a larger buffer, whose other rows hold NaN scales."""
    big = mx("nv4", 300, 256, 0.02)
    x = normal(8, 130, 256)
    part = big.first(130).quantize(x)
    w = mx("nv4", 64, 256, 0.01).quantize(normal(9, 64, 256) * 0.1)
    y = R.mx_linear(part, w, torch.empty(130, 64, device="cuda"))
    want = held(part) @ held(w).T
    assert np.allclose(f64(y), want, atol=1e-4) and np.isfinite(f64(y)).all()


# ---- norms ------------------------------------------------------------------------

def check_norm(rows, cols, dtype, res, out, gain=True, eps=1e-5, seed=0, in_place=False, scale=1.0):
    x = pitched((normal(seed + 1, rows, cols) * scale).to(dtype), 16)
    r = None if res is None else pitched((normal(seed + 2, rows, cols) * 3 * scale).to(res), 8)
    g = 1 + 0.5 * normal(seed + 3, cols) if gain else None
    xs, rs = f64(x), None if r is None else f64(r)
    ro = None if r is None else r if in_place else pitched(torch.zeros_like(r), 24)
    if out in FORMATS:
        y = mx(out, rows, cols, 0.003 if out == "nv4" else None)
    else:
        y = x if in_place and out == dtype else pitched(torch.zeros(rows, cols, dtype=out, device="cuda"), 8)
    R.add_norm(engine(), x, y, g, r, ro, eps)
    h, want = O.add_norm(xs, rs, None if g is None else f64(g), eps)
    if r is not None:
        assert (np.abs(f64(ro) - h) <= (U[res] + 2.0 ** -24) * np.abs(h)).all()
    if out in FORMATS:
        is_quantized(y, want, REL)
    else:
        assert (np.abs(f64(y) - want) <= (U[out] + REL) * np.abs(want) + 1e-40).all()
    assert engine().status() == 0


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("res", [None, BF16, F32])
@pytest.mark.parametrize("out", [BF16, F32] + FORMATS)
def test_norm_types(dtype, res, out):
    check_norm(37, 1056, dtype, res, out)


@pytest.mark.parametrize("shape", [(1, 32), (7, 64), (300, 256), (9, 288), (5, 1024), (3, 4096), (2, 4128), (3, 8192), (2, 11008),
                                   (2, 16416), (1, 32768), (1000, 96)])
@pytest.mark.parametrize("out", [BF16, "fp8", "nv4"])
def test_norm_shapes(shape, out):
    check_norm(*shape, BF16, F32, out, seed=shape[1])


@pytest.mark.parametrize("cols", [8, 24, 40, 1000, 5128])
def test_norm_columns_by_eights(cols):
    check_norm(4, cols, BF16, BF16, BF16)
    check_norm(4, cols, F32, None, F32, gain=False)


def test_norm_in_place_and_extremes():
    check_norm(20, 512, BF16, F32, BF16, in_place=True)
    check_norm(20, 512, F32, BF16, F32, in_place=True)
    check_norm(3, 512, F32, None, F32, eps=0.0, scale=1e-15)
    check_norm(3, 512, F32, F32, F32, scale=1e15)
    x = torch.zeros(2, 64, device="cuda")
    y = R.add_norm(engine(), x, torch.full_like(x, 5.0))
    assert not y.any()                                   # an all-zero row
    x[1, 3] = NAN
    t = mx("fp8", 2, 64)
    R.add_norm(engine(), x, t)
    assert engine().status() == NUMERIC
    y = t.unpack(y)
    assert not y[0].any() and torch.isnan(y[1]).all()


# ---- sampling -----------------------------------------------------------------------

def check_sample(z, t, k=None, p=None, m=None, u=None, each=1, want_probs=True, used=None):
    """z [rows][vocab] (possibly pitched) against the oracle; t, k, p, m: per-request lists or None."""
    n, V = z.shape
    req = n // each
    u = normal(99, n).view(torch.int32) if u is None else u
    token, arg = i32([-7] * n), i32([-7] * n)
    probs = torch.full((n, V), 7.0, device="cuda") if want_probs else None
    s = R.Sampler(engine(), req, None if t is None else f32(t), None if k is None else i32(k), None if p is None else f32(p),
                  None if m is None else f32(m), each, None if used is None else i32(used))
    s(z, u, token, arg, probs)
    zs, us, tok, am = f64(z), u.cpu().numpy().astype(np.int64) & 0xffffffff, token.cpu().numpy(), arg.cpu().numpy()
    ps = f64(probs) if want_probs else None
    at = lambda v, i, d: d if v is None else float(np.float32(v[i // each]))
    for i in range(n):
        if used is not None and i % each >= used[i // each]:
            assert tok[i] == -7 and am[i] == -7 and (ps is None or (ps[i] == 7).all())
            continue
        ti = at(t, i, 1.0)
        w = O.weights(zs[i], ti)
        slack = 2 * V
        assert am[i] == np.flatnonzero(zs[i] == zs[i].max())[0]
        if not ti > 0:
            lo = hi = 1
            order = np.array([am[i]])
        else:
            order, lo, hi = O.kept(zs[i], w, 0 if k is None else k[i // each], at(p, i, 1.0), slack=slack)
        mi = min(at(m, i, 0.0), 1.0)
        ok = False
        for c in range(lo, hi + 1):                      # the cuts that whole weights within the slack allow
            x = np.zeros_like(w)
            x[order[:c]] = w[order[:c]]
            if ti > 0:
                x[x < mi * 2.0 ** 40] = 0
            total = int(x.sum())
            upto = int(x[:tok[i] + 1].sum())
            r = (int(us[i]) * total) >> 32
            near = upto - int(x[tok[i]]) - slack <= r < upto + slack and x[tok[i]] > 0
            if want_probs:
                q = x / total
                # weights of few units may be there or not
                near = near and (np.abs(ps[i] - q) <= 2.0 ** -22 * q + 4.0 / total).all() and ((ps[i] > 0) == (x > 0))[x != 1].all()
            ok = ok or bool(near)
        assert ok, (i, lo, hi, tok[i])
    assert engine().status() == 0
    return token, probs


VOCABS = [1, 2, 7, 33, 1000, 4095, 4096, 4097, 8192, 16385, 32000, 65537, 131072, 262144]


@pytest.mark.parametrize("vocab", VOCABS)
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_sample_vocabularies(vocab, dtype):
    z = (normal(vocab, 4, vocab) * 3).to(dtype)
    check_sample(z, [0.7, 1.0, 0.0, 1.3], [5, 0, 0, 40], [0.9, 0.8, 0.5, 1.0], [0.0, 0.01, 0.0, 0.05])


@pytest.mark.parametrize("case", ["none", "k", "p", "m", "kp", "km", "pm", "kpm"])
@pytest.mark.parametrize("rows", [1, 40, 200])
def test_sample_controls(case, rows):
    r = random.Random(rows)
    z = normal(rows, rows, 3000) * 2.5
    check_sample(z, [r.uniform(0.3, 1.5) for _ in range(rows)],
                 [r.choice([0, 1, 2, 50, 2999, 3000, 9999]) for _ in range(rows)] if "k" in case else None,
                 [r.choice([0.0, -1.0, 1e-6, 0.3, 0.95, 0.9999, 1.0, 2.0]) for _ in range(rows)] if "p" in case else None,
                 [r.choice([0.0, -1.0, 1e-9, 0.05, 0.5, 1.0, 3.0]) for _ in range(rows)] if "m" in case else None)


def test_sample_ties():
    """Equal logits: the lower ids stay; whole rows of one value, more than a list or a bin takes."""
    for V in (64, 5000, 40000):
        z = torch.zeros(3, V, device="cuda")
        check_sample(z, [1.0, 0.5, 2.0], [1, 17, V - 3])
        check_sample(z, [1.0, 0.5, 2.0], None, [0.5, 1e-5, 0.999])
        z[:, 1::2] = 1.0
        z[:, 5] = -3.0
        check_sample(z, [1.0, 0.5, 2.0], [V // 2 + 1, V // 2, 3], [0.7, 1.0, 0.2])
    z = torch.round(normal(3, 6, 20000) * 4) / 4         # a hundred values or so
    check_sample(z, [0.8] * 6, [3000, 1, 700, 0, 0, 0], [1.0, 1.0, 0.6, 0.5, 0.99, 0.9])
    z = normal(4, 4, 30000) * 1e-3                       # all in a hair's breadth of one another
    check_sample(z, [1.0] * 4, [20000, 0, 5, 0], [0.9, 0.5, 1.0, 0.01])
    z = 1000 + normal(5, 4, 30000).to(BF16).float() * 0.01
    check_sample(z, [1.0] * 4, [20000, 0, 5, 0], [0.9, 0.5, 1.0, 0.01])


def test_sample_long_lists():
    """Cuts among more tokens than are sorted at a time, or than a list holds, and behind the bins of weight."""
    z = normal(11, 8, 131072) * 2.5
    check_sample(z, [1.3] * 8, [0, 0, 3000, 3000, 20000, 20000, 130000, 0], [0.97, 0.9999, 1.0, 0.8, 0.9, 1.0, 0.999, 0.6],
                 [0.0, 0.0, 0.0, 0.0, 1e-7, 1e-5, 0.0, 1e-4])
    check_sample((z * 4).to(BF16), [2.5, 2.5, 2.0, 2.0, 3.0, 3.0, 0.1, 2.5], [0, 0, 0, 70000, 70000, 0, 600, 0],
                 [0.9999, 0.99999, 0.9999, 0.9999, 1.0, 0.999999, 0.9, 1.0], [0.0, 1e-9, 0.0, 0.0, 0.0, 0.0, 0.0, 1e-6])


def test_sample_outputs_alone():
    """Each output without the others, and no filter at all."""
    z = normal(12, 5, 9001) * 3
    u = i32([1, -5, 1 << 30, 7, -(1 << 31)])
    s = R.Sampler(engine(), 5, f32([0.8, 0.0, 1.2, 1.0, 0.6]), i32([0, 3, 40, 0, 700]), f32([0.9, 0.9, 0.9, 1.0, 1.0]))
    token, arg, probs = i32([-7] * 5), i32([-7] * 5), torch.full_like(z, 7.0)
    s(z, u, token, arg, probs)
    a, b, c = i32([-7] * 5), i32([-7] * 5), torch.full_like(z, 7.0)
    s(z, u, a)
    s(z, argmax=b)
    s(z, probs=c)
    assert torch.equal(a, token) and torch.equal(b, arg) and torch.equal(c, probs)
    s(z, u, a, probs=c.fill_(7.0))
    assert torch.equal(a, token) and torch.equal(c, probs)
    check_sample(z, None)
    assert engine().status() == 0


def test_sample_masked_and_extreme():
    z = normal(6, 8, 9000) * 3
    z[0, 1:] = -INF                                      # one token left
    z[1, ::2] = -INF
    z[2] = -INF
    z[2, 8999] = -3e38
    z[3] *= 1e30
    z[4, 7], z[4, 8] = 3.3e38, -3.3e38
    z[5] = -0.0
    z[5, 100] = 0.0
    lowest = torch.finfo(F32).min
    z[6, 10:] = lowest
    check_sample(z, [1.0, 0.7, 1.0, 1.0, 2.0, 1.0, 1.0, 1e-3], [0, 60, 2, 5, 0, 3, 50, 0], [0.9, 0.9, 0.5, 1.0, 1.0, 0.9, 0.99, 0.9])
    check_sample(z[1:2], [1e30])
    check_sample(z[7:], [1e-38])
    u = torch.tensor([0, -1, 1, 1 << 30, -(1 << 31), 5, 6, 7], dtype=torch.int32, device="cuda")
    check_sample(z, [1.0] * 8, u=u)


@pytest.mark.parametrize("bad", ["nan", "inf", "none"])
def test_sample_reports_rows_without_a_distribution(bad):
    z = normal(7, 3, 10000)
    if bad == "none":
        z[1] = -INF
    else:
        z[1, 9999] = NAN if bad == "nan" else INF
    token, arg, probs = i32([5] * 3), i32([5] * 3), torch.full_like(z, 3.0)
    R.Sampler(engine(), 3)(z, i32([1, 2, 3]), token, arg, probs)
    assert engine().status() == NUMERIC
    assert int(token[1]) == -1 and int(arg[1]) == -1 and not probs[1].any()
    assert (token[[0, 2]] >= 0).all() and torch.allclose(probs[[0, 2]].sum(-1), torch.ones(2, device="cuda"))


def test_sample_tree_rows_and_pitches():
    used = [5, 0, 1, 3]
    z = normal(8, 20, 1003) * 3
    for b, n in enumerate(used):
        z[b * 5 + n:(b + 1) * 5] = NAN                   # slots behind the trees' sizes
    check_sample(pitched(z, 0), [0.8, 0.9, 0.0, 1.1], [40] * 4, [0.9] * 4, [0.02] * 4, each=5, used=used)
    check_sample(pitched(z, 5), [0.8, 0.9, 0.0, 1.1], None, [0.9] * 4, each=5, used=used, want_probs=False)
    probs = torch.full((20, 1010), 9.0, device="cuda")
    R.Sampler(engine(), 4, rows_each=5, rows_used=i32(used))(z, probs=probs[:, :1003])
    assert (probs[:, 1003:] == 9).all() and torch.allclose(probs[:5, :1003].sum(-1), torch.ones(5, device="cuda"))
    assert engine().status() == 0


def test_sample_draws_follow_the_distribution():
    """One row, many words: every token exactly as often as its weight says (to a word)."""
    z = (normal(9, 1, 50) * 2).expand(4096, 50).contiguous()
    u = torch.arange(4096, device="cuda", dtype=torch.int64).mul(1 << 20).to(torch.int64)
    u = torch.where(u >= 1 << 31, u - (1 << 32), u).int()
    token = i32([0] * 4096)
    R.Sampler(engine(), 4096, top_k=i32([20] * 4096))(z, u, token)
    w = O.distribution(f64(z[0]), 1.0, 20)
    n = np.bincount(token.cpu().numpy(), minlength=50)
    assert (np.abs(n - 4096.0 * w / w.sum()) <= 1.0 + 1e-3).all()


# ---- refusals -------------------------------------------------------------------------

def refused(code, fn, *args):
    with pytest.raises(B.EagleError) as e:
        fn(*args)
    assert e.value.code == code


def test_arguments_checked_before_launch():
    e = engine()
    ws, st = e.ws.data_ptr(), e.stream()
    buf = torch.zeros(1 << 16, device="cuda")
    a = _p(buf)
    before = B.eagle_launch_count(e.ctx)
    X = lambda **kw: B.eagle_mx(*[{**dict(data=a, scale=a + 65536, tensor_scale=None, rows=4, cols=64, format=1), **kw}[f]
                                  for f in ("data", "scale", "tensor_scale", "rows", "cols", "format")])
    Q = lambda m, dtype=0, act=0, x=a + 4096, ld=64, w=ws: B.eagle_mx_quantize(e.ctx, dtype, act, x, ld, m, w, st)
    for fn in (Q, lambda m: B.eagle_mx_unpack(e.ctx, m, 0, a + 4096, 64, ws, st),
               lambda m: B.eagle_mx_linear(e.ctx, m, X(), None, 0, a + 4096, 64, ws, st),
               lambda m: B.eagle_mx_linear(e.ctx, X(), m, None, 0, a + 4096, 64, ws, st)):
        refused(INVALID_ARG, fn, X(format=0))
        refused(INVALID_ARG, fn, X(format=4))
        refused(SHAPE, fn, X(cols=48))
        refused(SHAPE, fn, X(cols=0))
        refused(SHAPE, fn, X(rows=0))
        refused(INVALID_ARG, fn, X(data=None))
        refused(ALIGN, fn, X(scale=a + 4))
        refused(ALIGN, fn, X(format=3, tensor_scale=a + 2))
    refused(INVALID_ARG, Q, X(), 2)
    refused(INVALID_ARG, Q, X(), 0, 2)
    refused(SHAPE, Q, X(), 0, 0, a, 56)
    refused(SHAPE, Q, X(), 0, 1, a + 4096, 64)           # the gate and its partner need 128
    refused(ALIGN, Q, X(), 0, 0, a + 4096, 68)
    refused(ALIGN, Q, X(), 0, 0, a + 4098, 64)
    refused(INVALID_ARG, Q, X(), 0, 0, a, 64)            # x is out
    refused(INVALID_ARG, Q, X(), 0, 0, a + 4096, 64, None)
    refused(INVALID_ARG, lambda: B.eagle_mx_linear(e.ctx, X(), X(format=2), None, 0, a + 4096, 64, ws, st))
    refused(SHAPE, lambda: B.eagle_mx_linear(e.ctx, X(), X(cols=96), None, 0, a + 4096, 64, ws, st))
    refused(SHAPE, lambda: B.eagle_mx_linear(e.ctx, X(), X(rows=72), None, 0, a + 4096, 64, ws, st))
    refused(ALIGN, lambda: B.eagle_mx_linear(e.ctx, X(), X(rows=9), None, 0, a + 4096, 9, ws, st))
    refused(ALIGN, lambda: B.eagle_mx_linear(e.ctx, X(), X(), a + 4, 0, a + 4096, 64, ws, st))
    refused(INVALID_ARG, lambda: B.eagle_mx_linear(e.ctx, X(), X(), None, 0, a, 64, ws, st))
    refused(INVALID_ARG, lambda: B.eagle_mx_linear(e.ctx, X(), X(), None, 3, a + 4096, 64, ws, st))

    def N(code, **kw):
        base = dict(rows=4, cols=64, dtype=0, x=a, ld_x=64, res_dtype=1, residual=a + 4096, ld_res=64, residual_out=a + 8192,
                    ld_res_out=64, gain=a + 16384, eps=1e-5, out_dtype=0, out=a + 32768, ld_out=64, out_mx=None)
        base.update(kw)
        refused(code, B.eagle_add_norm, e.ctx, B.eagle_norm(*base.values()), ws, st)
    N(SHAPE, rows=0)
    N(SHAPE, cols=60)
    N(CAPACITY, cols=32776, ld_x=32776, ld_res=32776, ld_res_out=32776, ld_out=32776)
    N(INVALID_ARG, eps=-1.0)
    N(INVALID_ARG, eps=NAN)
    N(INVALID_ARG, dtype=2)
    N(INVALID_ARG, res_dtype=2)
    N(INVALID_ARG, out_dtype=2)
    N(INVALID_ARG, x=None)
    N(INVALID_ARG, out=None)
    N(ALIGN, x=a + 2)
    N(ALIGN, ld_res=66)
    N(SHAPE, ld_out=56)
    N(INVALID_ARG, residual_out=a + 4096, ld_res_out=68)
    N(INVALID_ARG, out=a, ld_out=72)
    N(INVALID_ARG, out=a, out_dtype=1)
    N(INVALID_ARG, out=a + 8192)
    N(INVALID_ARG, out_mx=B.ref(X()))                    # both outputs
    N(SHAPE, out=None, out_mx=B.ref(X(rows=5)))
    N(SHAPE, out=None, out_mx=B.ref(X(cols=32)))

    F = lambda each=1: B.eagle_filter(None, None, None, None, each, None)
    S = lambda n=2, v=64, dtype=1, z=a, ld=64, f=None, u=a + 4096, token=a + 8192, arg=None, probs=None, lp=64: B.eagle_sample(
        e.ctx, n, v, dtype, z, ld, f or F(), u, token, arg, probs, lp, ws, st)
    for code, kw in [(SHAPE, dict(n=0)), (SHAPE, dict(v=0)), (CAPACITY, dict(v=262145, ld=262145)), (INVALID_ARG, dict(dtype=2)),
                     (INVALID_ARG, dict(z=None)), (SHAPE, dict(ld=63)), (INVALID_ARG, dict(f=F(0))),
                     (INVALID_ARG, dict(token=None)), (INVALID_ARG, dict(u=None)), (INVALID_ARG, dict(u=None, token=None)),
                     (ALIGN, dict(z=a + 4)), (ALIGN, dict(probs=a + 4100)), (SHAPE, dict(probs=a + 16384, lp=63)),
                     (INVALID_ARG, dict(probs=a)), (ALIGN, dict(f=B.eagle_filter(a + 4, None, None, None, 1, None)))]:
        refused(code, lambda: S(**kw))
    with pytest.raises(B.EagleError):
        B.eagle_mx_layout(5, 4, 64)
    assert B.eagle_mx_layout(1, 129, 160) == (129 * 160, 2 * 2 * 512) and B.eagle_mx_layout(3, 1, 32) == (16, 512)
    assert B.eagle_launch_count(e.ctx) == before and e.status() == 0


def test_refuses_extents_that_pass_32_bits():
    e = engine()
    a, ws, st, before = torch.zeros(1 << 16, dtype=torch.uint8, device="cuda").data_ptr(), e.ws.data_ptr(), e.stream(), \
        B.eagle_launch_count(e.ctx)
    most = B.EAGLE_MAX_EXTENT
    for rows, cols in ((most + 1, 32), (1, most + 32), ((1 << 31) - 1, 32), (1, (1 << 31) - 32)):
        m = B.eagle_mx(a, a + 32768, None, rows, cols, B.MX_FP8)
        refused(CAPACITY, B.eagle_mx_quantize, e.ctx, 0, 0, a + 4096, (1 << 31) - 8, m, ws, st)
        refused(CAPACITY, B.eagle_mx_unpack, e.ctx, m, 0, a + 4096, (1 << 31) - 8, ws, st)
        refused(CAPACITY, B.eagle_mx_linear, e.ctx, m, m, None, 0, a + 4096, (1 << 31) - 8, ws, st)
    refused(CAPACITY, B.eagle_add_norm, e.ctx, B.eagle_norm(most + 1, 8, 0, a, 8, 0, None, 0, None, 0, None, 0.0, 0, a + 4096, 8, None), ws, st)
    refused(CAPACITY, B.eagle_sample, e.ctx, most + 1, 1, 0, a, 1, B.eagle_filter(None, None, None, None, 1, None), None, None,
            a + 4096, None, 1, ws, st)
    assert B.eagle_launch_count(e.ctx) == before and e.status() == 0


def test_wrappers_check_their_tensors():
    e = engine()
    t = mx("fp8", 4, 64)
    for x in (torch.zeros(4, 32, device="cuda"), torch.zeros(4, 64), torch.zeros(4, 64, device="cuda", dtype=torch.float16),
              torch.zeros(64, 4, device="cuda").t()):
        with pytest.raises(ValueError):
            t.quantize(x)
    with pytest.raises(ValueError):
        t.first(5)
    with pytest.raises(ValueError):
        R.MxTensor(e, 4, 64, "nv4", torch.zeros(2, device="cuda"))
    x = torch.zeros(4, 64, device="cuda")
    with pytest.raises(ValueError):
        R.add_norm(e, x, torch.zeros_like(x), residual=x.bfloat16(), residual_out=x.clone())
    with pytest.raises(ValueError):
        R.mx_linear(t, t, torch.zeros(4, 4, device="cuda"), torch.zeros(5, device="cuda"))
    with pytest.raises(ValueError):
        R.Sampler(e, 4, temperature=torch.zeros(3, device="cuda"))
    s = R.Sampler(e, 4)
    with pytest.raises(ValueError):
        s(torch.zeros(5, 64, device="cuda"), i32([0] * 5), i32([0] * 5))


def test_wrappers_refuse_host_memory():
    """Tensors of the host among the arguments, or all of them: nothing is launched."""
    e = engine()
    x, t, z = torch.zeros(4, 64), mx("fp8", 4, 64), torch.zeros(4, 64, device="cuda")
    before = B.eagle_launch_count(e.ctx)
    s = R.Sampler(e, 4)
    for call in (lambda: R.add_norm(e, x, torch.zeros_like(x)), lambda: R.add_norm(e, x, t), lambda: R.add_norm(e, z, x),
                 lambda: R.add_norm(e, z, t, torch.ones(64)), lambda: R.mx_linear(t, t, torch.zeros(4, 8)),
                 lambda: R.mx_linear(t, t, torch.zeros(4, 8, device="cuda")[:, :4], torch.zeros(4)), lambda: t.unpack(x),
                 lambda: R.Sampler(e, 4, torch.ones(4)), lambda: R.Sampler(e, 4, torch.ones(4, device="cuda"), top_p=torch.ones(4)),
                 lambda: s(x, torch.zeros(4, dtype=torch.int32), torch.zeros(4, dtype=torch.int32)), lambda: s(z, probs=x),
                 lambda: s(z, torch.zeros(4, dtype=torch.int32), i32([0] * 4)),
                 lambda: R.MxTensor(e, 4, 64, "fp8", data=torch.zeros(256, dtype=torch.uint8)),
                 lambda: R.MxTensor(e, 4, 64, "nv4", torch.ones(1))):
        with pytest.raises(ValueError):
            call()
    assert B.eagle_launch_count(e.ctx) == before


# ---- streams, graphs, runs ---------------------------------------------------------------

def test_other_stream_and_second_engine():
    """Two engines' calls on two streams at once."""
    e2 = R.Engine(engine().dims, max_batch=64, max_rows=8, max_expanded=1, max_children=1, max_tree=2, max_prefix=1024,
                  device="cuda")
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    outs = []
    x0, w0 = normal(1, 70, 2048), normal(2, 5000, 2048) * 0.1
    torch.cuda.synchronize()
    for _ in range(5):
        for s, e in ((a, engine()), (b, e2)):
            with torch.cuda.stream(s):
                x = R.MxTensor(e, 70, 2048, "fp4").quantize(x0)
                w = R.MxTensor(e, 5000, 2048, "fp4").quantize(w0)
                y = R.mx_linear(x, w, torch.empty(70, 5000, device="cuda"))
                z = R.add_norm(e, y, torch.empty_like(y))
                t = torch.empty(70, dtype=torch.int32, device="cuda")
                R.Sampler(e, 70, top_p=torch.full((70,), 0.8, device="cuda"))(z, torch.arange(70, dtype=torch.int32, device="cuda") * 9999991, t)
                outs.append((y, z, t))
    torch.cuda.synchronize()
    for o in outs[1:]:
        assert all(torch.equal(p, q) for p, q in zip(o, outs[0]))
    assert e2.status() == 0 and engine().status() == 0


def test_weights_quantised_directly_before_their_product():
    """A product launched behind the calls that write its operands reads what they wrote, again and again."""
    x = mx("nv4", 3, 4096, 0.01)
    w = mx("nv4", 2000, 4096, 0.01)
    y = torch.empty(3, 2000, device="cuda")
    xs = [normal(i, 3, 4096) for i in range(3)]
    wsrc = [normal(10 + i, 2000, 4096) * 0.1 for i in range(3)]
    wants = []
    for i in range(3):
        x.quantize(xs[i]); w.quantize(wsrc[i])
        torch.cuda.synchronize()
        wants.append(held(x) @ held(w).T)
    for turn in range(12):
        i = turn % 3
        if turn % 2:
            x.quantize(xs[i]); w.quantize(wsrc[i])
        else:
            w.quantize(wsrc[i]); x.quantize(xs[i])
        R.mx_linear(x, w, y)
        got = f64(y)
        assert np.allclose(got, wants[i], atol=4096 * 2.0 ** -20), turn


class Step:
    """One decoder layer and an LM head of a small target over a paged cache: every call of a decoding step."""

    def __init__(self, fmt, seqs, seed=0):
        self.eng = e = engine()
        self.fmt, self.seqs = fmt, seqs
        self.d, self.ff, self.V = 512, 1152, 1000
        Hq, Hkv, dh = 4, 2, 64
        self.qkv_n = (Hq + 2 * Hkv) * dh
        self.cache = R.PagedCache(e, seqs, 16, 40 * seqs, 20)
        self.cache.clear()
        self.rope = R.rope_for(e.dims)
        g = {"nv4": 0.002}.get(fmt)
        W = lambda n, k, s: mx(fmt, n, k, g).quantize(normal(seed + s, n, k) / math.sqrt(k))
        self.wqkv, self.wo = W(self.qkv_n, self.d, 1), W(self.d, Hq * dh, 2)
        self.wgu, self.wd, self.lm = W(2 * self.ff, self.d, 3), W(self.d, self.ff, 4), W(self.V, self.d, 5)
        self.g1, self.g2, self.g3 = (1 + 0.2 * normal(seed + 6 + i, self.d) for i in range(3))
        self.embed = normal(seed + 9, self.V, self.d)
        self.a = 0.003 if fmt == "nv4" else None
        self.sampler = R.Sampler(e, seqs, f32([0.8] * seqs), i32([50] * seqs), f32([0.9] * seqs))

    def buffers(self, n):
        e = lambda *s, dtype=F32: torch.empty(*s, dtype=dtype, device="cuda")
        b = dict(h=e(n, self.d), a=mx(self.fmt, n, self.d, self.a), qkv=e(n, self.qkv_n, dtype=BF16), att=e(n, 4, 64, dtype=BF16),
                 o=mx(self.fmt, n, 256, self.a), x=e(n, self.d, dtype=BF16), m=mx(self.fmt, n, self.d, self.a),
                 gu=e(n, 2 * self.ff, dtype=BF16), s=mx(self.fmt, n, self.ff, self.a), y=e(n, self.d, dtype=BF16),
                 f=mx(self.fmt, n, self.d, self.a), z=e(n, self.V), token=e(self.seqs, dtype=torch.int32), h2=e(n, self.d))
        return b

    def run(self, b, x, start, n_new, last, u):
        """New rows x (fp32 embeddings) of every sequence; tokens from each one's last row."""
        e, c, n = self.eng, self.cache, x.shape[0]
        c.reserve(n_new)
        R.add_norm(e, x, b["a"], self.g1)
        R.mx_linear(b["a"], self.wqkv, b["qkv"])
        q = b["qkv"].view(n, 8, 64)
        c.append(0, start, self.rope, q[:, :4], q[:, 4:6], q[:, 6:])
        c.attend(0, start, q[:, :4], b["att"])
        c.advance()
        b["o"].quantize(b["att"].view(n, 256))
        R.mx_linear(b["o"], self.wo, b["x"])
        R.add_norm(e, b["x"], b["m"], self.g2, residual=x, residual_out=b["h"])
        R.mx_linear(b["m"], self.wgu, b["gu"])
        b["s"].quantize(b["gu"], swiglu=True)
        R.mx_linear(b["s"], self.wd, b["y"])
        R.add_norm(e, b["y"], b["f"], self.g3, residual=b["h"], residual_out=b["h2"])
        R.mx_linear(b["f"], self.lm, b["z"])
        zl = b["z"].index_select(0, last) if n > self.seqs else b["z"]
        self.sampler(zl, u, b["token"])
        return b["token"]


@pytest.mark.parametrize("fmt", FORMATS)
def test_target_step(fmt):
    """A prompt and decoding steps, each call's output against the oracle on that call's own inputs."""
    seqs = 3
    st = Step(fmt, seqs)
    lens = [7, 20, 1]
    start = i32([0, 7, 27, 28])
    last = torch.tensor([6, 26, 27], device="cuda")
    u = i32([123456789, -99999999, 5])
    x = normal(50, 28, st.d)
    for turn in range(3):
        n = x.shape[0]
        b = st.buffers(n)
        xs = f64(x)
        token = st.run(b, x, start, i32(lens), last, u)
        assert engine().status() == 0
        is_quantized(b["a"], O.add_norm(xs, None, f64(st.g1), 1e-5)[1], REL)
        def linear(xq, w, y, dtype):
            a, c = held(xq), held(w)
            want, size = a @ c.T, np.abs(a) @ np.abs(c).T
            assert (np.abs(f64(y) - want) <= (w.cols + 8) * 2.0 ** -23 * size + U[dtype] * np.abs(want)).all()
        linear(b["o"], st.wo, b["x"], BF16)
        is_quantized(b["o"], f64(b["att"]).reshape(n, 256))
        h, y = O.add_norm(f64(b["x"]), xs, f64(st.g2), 1e-5)
        assert (np.abs(f64(b["h"]) - h) <= 2.0 ** -23 * np.abs(h)).all()
        is_quantized(b["m"], y, REL)
        linear(b["m"], st.wgu, b["gu"], BF16)
        is_quantized(b["s"], O.swiglu(f64(b["gu"])), 2.0 ** -21)
        linear(b["s"], st.wd, b["y"], BF16)
        h2, y = O.add_norm(f64(b["y"]), f64(b["h"]), f64(st.g3), 1e-5)
        is_quantized(b["f"], y, REL)
        linear(b["f"], st.lm, b["z"], F32)
        z = f64(b["z"])[last.cpu().numpy()] if n > seqs else f64(b["z"])
        for i in range(seqs):
            w = O.distribution(z[i], float(np.float32(0.8)), 50, float(np.float32(0.9)))
            assert draw_one(w, int(u[i]) & 0xffffffff) == int(token[i])
        # the next step: one token each
        x = st.embed[token.long()]
        lens, start, last = [1] * seqs, i32([0, 1, 2, 3]), torch.arange(3, device="cuda")
    assert st.cache.len.tolist() == [9, 22, 3]


def test_target_step_captured():
    """The decoding step as a CUDA graph: replays on other inputs give what eager calls give; two graphs share the
    workspace."""
    seqs = 4
    runs = []
    for captured in (False, True):
        st = Step("nv4", seqs)
        b = st.buffers(seqs)
        start, ones, last = i32(list(range(seqs + 1))), i32([1] * seqs), torch.arange(seqs, device="cuda")
        u, x = i32([0] * seqs), torch.empty(seqs, st.d, device="cuda")
        words = torch.randint(-(1 << 31), (1 << 31) - 1, (6, seqs), generator=gen(3), device="cuda", dtype=torch.int64).int()
        x.copy_(st.embed[:seqs]); u.copy_(words[0])
        st.run(b, x, start, ones, last, u)
        st.cache.release(i32([0] * seqs))
        st.cache.clear()
        graphs = []
        if captured:
            for _ in range(2):
                g = torch.cuda.CUDAGraph()
                with torch.cuda.graph(g):
                    st.run(b, x, start, ones, last, u)
                graphs.append(g)
            st.cache.clear()
        tokens = []
        x.copy_(st.embed[:seqs])
        for i in range(6):
            u.copy_(words[i])
            if captured:
                graphs[i % 2].replay()
            else:
                st.run(b, x, start, ones, last, u)
            tokens.append(b["token"].clone())
            x.copy_(st.embed[b["token"].long()])
        runs.append((torch.stack(tokens), b["z"].clone(), b["h2"].clone()))
        assert engine().status() == 0
    assert all(torch.equal(p, q) for p, q in zip(*runs))


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("outs", [1, 8, 15, 33, 191, 193, 260, 1000])
def test_linear_many_rows_any_outputs(fmt, outs):
    """Rows as the first operand: 16 outputs a store, 8, and single ones; pitches that are and are not whole sectors."""
    for rows, more, out in ((129, 0, BF16), (300, 8, BF16), (300, 16, F32), (1025, 4, F32)):
        check_linear(fmt, rows, 288, outs, out, True, seed=rows + outs, more=more)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("rows,cols,outs", [(16, 8192, 3840), (9, 8192, 3200), (3, 8192, 2688), (100, 8192, 6400), (128, 16384, 2600),
                                            (77, 12288, 3330), (250, 8192, 1500), (40, 4128, 900)])
def test_linear_inner_dimension_in_parts(fmt, rows, cols, outs):
    """Few tiles and many columns: the inner dimension in up to eight parts, of unlike numbers of stages."""
    check_linear(fmt, rows, cols, outs, F32, True, seed=rows + outs)


@pytest.mark.parametrize("fmt", FORMATS)
def test_linear_many_rows_with_a_non_finite_block(fmt):
    x = normal(21, 700, 512)
    x[431, 100] = INF
    t = mx(fmt, 700, 512, 0.01).quantize(x)
    assert engine().status() == NUMERIC
    w = mx(fmt, 600, 512, 0.01).quantize(normal(22, 600, 512))
    y = R.mx_linear(t, w, torch.empty(700, 600, device="cuda"))
    bad = torch.zeros(700, dtype=torch.bool, device="cuda")
    bad[431] = True
    assert torch.isnan(y[bad]).all() and torch.isfinite(y[~bad]).all()
    assert engine().status() == 0


def test_offsets_beyond_32_bits():
    """Matrices, rows of logits and outputs of more than 2^32 bytes or 2^31 elements: their far ends."""
    rows, cols = 66000, 65536
    x = torch.zeros(rows, cols, dtype=BF16, device="cuda")
    x[-3:] = normal(1, 3, cols, dtype=BF16)
    w = mx("fp8", rows, cols).quantize(x)
    y = w.unpack(x.fill_(5.0))
    code, byte = O.quantize("fp8", f64(normal(1, 3, cols, dtype=BF16)))
    assert np.array_equal(f64(y[-3:]), O.values("fp8", code, byte)) and not y[:-3:997].any()
    a = mx("fp8", 5, cols).quantize(normal(2, 5, cols) * 0.1)
    out = R.mx_linear(a, w, torch.empty(5, rows, device="cuda"))
    av, wv = held(a), O.values("fp8", code, byte)
    assert (np.abs(f64(out[:, -3:]) - av @ wv.T) <= (cols + 8) * 2.0 ** -23 * (np.abs(av) @ np.abs(wv).T)).all()
    assert not out[:, :-3].any()
    del x, y, w, out
    # many rows by many outputs
    a = mx("nv4", 70000, 64, 0.01).quantize(normal(3, 70000, 64))
    b = mx("nv4", 65000, 64, 0.01).quantize(normal(4, 65000, 64))
    y = R.mx_linear(a, b, torch.empty(70000, 65000, dtype=BF16, device="cuda"))
    bv = torch.tensor(held(b), device="cuda")
    for r in (0, 33333, 69999):
        want = torch.tensor(held(a)[r:r + 1], device="cuda") @ bv.t()
        assert torch.allclose(y[r:r + 1].double(), want, rtol=2.0 ** -8, atol=1e-4)
    del y
    n = 70000
    x = torch.zeros(n, 32768, dtype=BF16, device="cuda")
    x[-1] = normal(5, 32768, dtype=BF16)
    y = R.add_norm(engine(), x, torch.empty_like(x))
    want = O.add_norm(f64(x[-1:]), None, None, 1e-5)[1]
    assert (np.abs(f64(y[-1:]) - want) <= (U[BF16] + REL) * np.abs(want)).all() and not y[:-1:999].any()
    del x, y
    n, V = 17000, 131072
    z = torch.zeros(n, V, device="cuda")
    z[-1, V - 2] = 90.0
    token = i32([0] * n)
    probs = torch.empty(n, V, device="cuda")
    R.Sampler(engine(), n, top_k=i32([3] * n))(z, i32([0] * n), token, None, probs)
    assert token[:-1].unique().tolist() == [0] and int(token[-1]) == V - 2
    assert probs[-1, V - 2] == 1 and probs[0, :4].tolist() == pytest.approx([1 / 3, 1 / 3, 1 / 3, 0.0])
    assert engine().status() == 0


def test_two_streams_each_with_its_workspace():
    """Calls of two contexts at once, and graphs of one context in turn, give what each alone gives."""
    engines = [R.Engine(dict(d=512, n_q_heads=4, n_kv_heads=2, head_dim=64, d_ff=64, vocab=64), max_batch=64, max_rows=8,
                        max_expanded=1, max_children=1, max_tree=2, max_prefix=64, device="cuda") for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in engines]

    def job(e, i, seed):
        """A norm into 4 bits, a product and a sampling of its rows, of sizes that differ from seed to seed."""
        rows, outs = [(40, 5000), (7, 20000), (130, 1000), (1, 32000)][seed % 4]
        t, w, z = R.MxTensor(e, rows, 256, "fp4"), R.MxTensor(e, outs, 256, "fp4"), torch.empty(rows, outs, device="cuda")
        x, res, h = normal(seed, rows, 256), normal(seed + 20, rows, 256), torch.empty(rows, 256, device="cuda")
        w.quantize(normal(seed + 50, outs, 256) * 0.2)
        out = i32([-7] * rows), torch.empty(rows, outs, device="cuda")
        u = normal(seed + 99, rows).view(torch.int32)
        s = R.Sampler(e, rows, f32([0.5 + 0.1 * (r % 7) for r in range(rows)]), i32([[0, 40, 700][r % 3] for r in range(rows)]),
                      f32([[0.9, 1.0][r % 2] for r in range(rows)]))

        def run():
            R.add_norm(e, x, t, None, res, h)
            R.mx_linear(t, w, z)
            s(z, u, out[0], None, out[1])
        return run, out

    def results(alone):
        jobs = [[job(e, i, 4 * i + k) for k in range(4)] for i, e in enumerate(engines)]
        torch.cuda.synchronize()
        for _ in range(5):
            for k in range(4):
                for i, st in enumerate(streams):
                    with torch.cuda.stream(st):
                        jobs[i][k][0]()
                    if alone:
                        torch.cuda.synchronize()
        torch.cuda.synchronize()
        assert all(e.status() == 0 for e in engines)
        return [o for js in jobs for _, out in js for o in out], jobs
    expected, _ = results(True)
    together, jobs = results(False)
    assert all(torch.equal(a, b) for a, b in zip(expected, together))
    graphs = []
    for run, out in jobs[0]:
        for o in out:
            o.fill_(-3)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            run()
        graphs.append(g)
    for k in (2, 0, 3, 1, 1, 2, 0, 3):
        graphs[k].replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(expected[:8], [o for _, out in jobs[0] for o in out]))
    assert engines[0].status() == 0


# ---- single weights, words over whole rows, products on every path ------------------------------------

def border(c, most, r):
    """(n, m, u): of n tokens with the largest weight and m behind them of weight w, the word u draws one of the m exactly
    if w >= c."""
    one = 1 << 40
    for _ in range(200000):
        m = r.randint(1, most - 1)
        n = min(max(int(m * c / one * r.uniform(0.3, 3.0)), 1), most - m)
        u = -(-(n << 72) // (n * one + m * c))
        if u < 1 << 32 and u * (n * one + m * (c - 1)) < n << 72:
            return n, m, u
    raise AssertionError(c)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_sample_single_weights(dtype):
    """Weights between the largest and 2^23 of 2^40 are the definition's but within 1/16 of a whole number, where they may be
    one off; below they are off by at most two.  (fp64's value is off by 2^-11 here.  From 2^23 on: the table's entries and the
    fixed point of 46 bits cost 2^-7 each, the exponent's pair of floats and the series less: below 2^-5 in all.  Below 2^23:
    exp2 by 2^-22.7 at most over all exponents that occur, a fused product by 2^-24: 1.75 in all.)"""
    r = random.Random(5)
    rows, V = [], 2000
    for i in range(260):
        t = [1.0, 1.3, 0.5, 0.05, 2.7, 1e-3][i % 6]
        t = float(np.float32(t))
        top = float(torch.tensor([3.0, -7.25, 100.125, 0.0, 0.7109375][i % 5], dtype=dtype))
        far = i % 4 == 3
        y = r.uniform(17.01, 30.0) if far else r.uniform(0.0, 16.9) if i % 2 else math.exp(-r.uniform(0.0, 9.0))
        z = float(torch.tensor(top - y * math.log(2) * t, dtype=dtype))
        w = math.exp((z - top) / t) * 2.0 ** 40
        if z == top or w < 64 or ((w < 2.0 ** 23) != far) or abs(w / 2.0 ** 23 - 1) < 1e-3:
            continue
        slack = 2.0 if far else 1 / 16
        low, high = math.floor(w - slack), math.floor(w + slack)
        for c, above in ((low, True), (high + 1, False)):
            rows.append((t, top, z, above, w) + border(c, V, r))
    assert len(rows) > 300
    z = torch.full((len(rows), V), -INF)
    for i, (_, top, x, _, _, n, m, _) in enumerate(rows):
        z[i, :n], z[i, n:n + m] = top, x
    u = torch.tensor([q[-1] for q in rows], dtype=torch.int64)
    u = torch.where(u >= 1 << 31, u - (1 << 32), u).int().cuda()
    token = i32([-7] * len(rows))
    R.Sampler(engine(), len(rows), f32([q[0] for q in rows]))(z.to(dtype).cuda(), u, token)
    token = token.tolist()
    wrong = [q[:5] for q, k in zip(rows, token) if (k >= q[5]) != q[3]]
    assert not wrong, (len(wrong), len(rows), wrong[:5])
    assert all(0 <= k < q[5] + q[6] for q, k in zip(rows, token))
    assert engine().status() == 0


@pytest.mark.parametrize("vocab", [1, 2, 4097, 8191, 65537, 131072, 262144])
@pytest.mark.parametrize("cut", ["none", "k", "p", "kp", "m"])
def test_sample_words_over_whole_rows(vocab, cut):
    """One flat row under words from the first to the last: every chunk of it is drawn from, and every draw is the
    definition's but for the weights' slack."""
    r = np.random.default_rng(vocab)
    n = 224
    words = np.concatenate(([0, 1, 2, 2 ** 31 - 1, 2 ** 31, 2 ** 31 + 1, 2 ** 32 - 2, 2 ** 32 - 1],
                            (np.arange(160) * 2 ** 32 + 2 ** 31) // 160, r.integers(0, 2 ** 32, 56))).astype(np.int64)
    dtype = F32 if vocab % 2 else BF16
    row = normal(vocab, 1, vocab, dtype=dtype)
    z = row.expand(n, vocab).contiguous()
    k = max(vocab // 2, 1) if "k" in cut else 0
    p = float(np.float32(0.9)) if "p" in cut else 1.0
    m = 2.0 ** -5 if cut == "m" else 0.0
    token = i32([-7] * n)
    u = torch.tensor(np.where(words >= 2 ** 31, words - 2 ** 32, words), dtype=torch.int32, device="cuda")
    R.Sampler(engine(), n, top_k=i32([k] * n), top_p=f32([p] * n), min_p=f32([m] * n))(z, u, token)
    token, w, slack = token.cpu().numpy(), O.weights(f64(row[0]), 1.0), 2 * vocab
    assert (token >= 0).all() and (token < vocab).all()
    order, lo, hi = O.kept(f64(row[0]), w, k, p, slack=slack)
    fits = []
    for c in range(lo, hi + 1):
        x = np.zeros_like(w)
        x[order[:c]] = w[order[:c]]
        x[x < m * 2.0 ** 40] = 0
        cum = np.cumsum(x)
        at = np.array([(int(a) * int(cum[-1])) >> 32 for a in words])
        fits.append(bool(((cum[token] - x[token] - slack <= at) & (at < cum[token] + slack) & (x[token] > 0)).all()))
    assert any(fits)
    assert len(np.unique(token // 4096)) >= vocab // 4096
    assert engine().status() == 0


PATHS = [(140, 1216, 6338), (31, 3840, 8587), (1086, 2304, 3143), (157, 3424, 2226), (153, 3584, 1989), (15, 12096, 5812),
         (1003, 4832, 221), (36, 7904, 3758), (50, 7168, 3009), (41, 9280, 2936), (1391, 11040, 69), (73, 5888, 2445),
         (496, 12320, 175), (40, 10272, 2428), (626, 13536, 127), (70, 7744, 1869), (299, 10976, 6012), (561, 2336, 6163),
         (672, 1728, 924), (1341, 3296, 46), (396, 864, 4931), (727, 832, 1809), (929, 3392, 4352), (1162, 960, 2083)]


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("rows,cols,outs", PATHS)
def test_linear_exact_products_on_every_path(fmt, rows, cols, outs):
    """Whole numbers of at most 16 a product, sums below 2^18: every sum is exact, so one block lost, doubled or under
    another's scale shows.  Shapes for both operand orders, single CTAs and pairs, tiles of 16 to 256 rows (64 and 192: scales
    that start inside a group), and 1 to 8 parts of the inner dimension, the last stage of them part of one."""
    r = gen(rows + cols)
    def make(n):
        t = mx(fmt, n, cols)
        one, two, shift = {"fp8": (0x38, 0x40, 7)}.get(fmt, (2, 4, 3))
        pick = lambda *s: torch.randint(0, 2, s, generator=r, device="cuda", dtype=torch.uint8)
        code = one + (two - one) * pick(n, cols) | pick(n, cols) << shift
        data = code if fmt == "fp8" else code[:, 0::2] | code[:, 1::2] << 4
        blocks = cols // O.BLOCK[fmt]
        low = {"nv4": 0x38}.get(fmt, 127)                # scales 1 and 2
        byte = low + (8 if fmt == "nv4" else 1) * pick(n, blocks)
        scale = torch.full((t.scale.numel(),), 0x7f if fmt == "nv4" else 0xff, dtype=torch.uint8, device="cuda")
        at = torch.tensor(O.scale_layout(n, blocks), device="cuda")
        scale[at.reshape(-1)] = 0
        scale[at[:, :blocks].reshape(-1)] = byte.reshape(-1)
        t.data.copy_(data.reshape(-1))
        t.scale.copy_(scale)
        value = torch.where(code & (two if fmt != "fp8" else 0x40) != 0, 2.0, 1.0) * (1.0 - 2.0 * (code >> shift))
        step = torch.where(byte == low, 1.0, 2.0).repeat_interleave(O.BLOCK[fmt], 1)
        return t, (value * step).double()
    (x, xv), (w, wv) = make(rows), make(outs)
    y = torch.full((rows, (outs + 7) // 8 * 8), 0.5, device="cuda")
    R.mx_linear(x, w, y[:, :outs])
    assert torch.equal(y[:, :outs].double(), xv @ wv.t())
    assert bool((y[:, outs:] == 0.5).all()) and engine().status() == 0


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("rows,cols,outs", [(130, 6528, 3787), (579, 4800, 912), (18, 1344, 3149), (134, 6240, 2149), (1, 1408, 2959),
                                            (67, 2368, 955), (1008, 4416, 267), (842, 8512, 261), (52, 2176, 146), (17, 1600, 130),
                                            (52, 1568, 139), (609, 11360, 259), (1, 1024, 131), (17, 1952, 129), (1, 1600, 131),
                                            (52, 1824, 132), (3, 15488, 3633), (10, 13728, 3692)])
def test_linear_exact_products_in_parts(fmt, rows, cols, outs):
    """The same by 2 to 8 CTAs a tile, a single stage each at the least, with as many clusters as the GPU holds and fewer."""
    test_linear_exact_products_on_every_path(fmt, rows, cols, outs)


def test_quantize_factors_near_the_smallest():
    """NV_FP4 under factors so small that scale * factor passes below the normal numbers, where elements are zeros."""
    r = np.random.default_rng(2)
    x = (r.standard_normal((40, 64)) * 2.0 ** r.integers(-126, -110, (40, 4)).repeat(16, 1)).astype(np.float32)
    x[0] = 2.0 ** -124
    for e in (-110, -117, -120, -124, -126, -127, -130, -140, -149):
        t = mx("nv4", 40, 64, 2.0 ** e).quantize(torch.tensor(x, device="cuda"))
        is_quantized(t, x.astype(np.float64))
        y = t.unpack(torch.empty(40, 64, device="cuda"))
        assert np.array_equal(f64(y), held(t))
    assert engine().status() == 0


@pytest.mark.parametrize("e", [-126, -124, -118, -110, -102, -90, -81, -79, -60, 0, 60, 90, 110])
def test_quantize_next_to_ties_under_any_factor(e):
    """NV_FP4 quotients on a tie and up to two steps beside it, of elements and of scales, whose remainders under small factors
    are below fp32's smallest number; and factors whose multiple of six fp32 does not hold."""
    r = np.random.default_rng(200 + e)
    for turn in range(6):
        g = np.float32((1 + r.random()) * 2.0 ** e)
        ties = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0])
        x = (r.choice(ties, (64, 256)) * float(g)).astype(np.float32)
        x = (x.view(np.int32) + r.integers(-2, 3, x.shape, dtype=np.int32)).view(np.float32)
        x[:, ::16] = np.float32(6) * g                   # the block's largest: its scale is 1
        x *= r.choice(np.float32([-1, 1]), x.shape)
        is_quantized(mx("nv4", 64, 256, g).quantize(torch.tensor(x, device="cuda")), x.astype(np.float64))
        border = (O.E4M3[1:] + O.E4M3[:-1]) / 2
        with np.errstate(over="ignore"):
            x = (r.choice(border, (64, 16)) * 6 * float(g)).astype(np.float32)
        x = np.where(np.isfinite(x), x, np.float32(3e38))
        x = (x.view(np.int32) + r.integers(-2, 3, x.shape, dtype=np.int32)).view(np.float32)
        y = np.zeros((64, 256), np.float32)
        y[:, 3::16] = x
        is_quantized(mx("nv4", 64, 256, g).quantize(torch.tensor(y, device="cuda")), y.astype(np.float64))
    for g in (5e37, 6e37, 3.4e38):                       # 6 g up to infinity, a quotient of 0
        y[0, :16] = 3e38
        is_quantized(mx("nv4", 64, 256, g).quantize(torch.tensor(y, device="cuda")), y.astype(np.float64))
    assert engine().status() == 0


@pytest.mark.parametrize("fmt", ["fp8", "fp4"])
def test_quantize_gated_near_the_largest_exponential(fmt):
    """Gates whose e^(-a) is near fp32's largest number, partners that bring the products back: as near as elsewhere."""
    r = gen(31)
    a = -87.34 - 1.37 * torch.rand(256, 11008, generator=r, device="cuda")
    b = torch.randn(256, 11008, generator=r, device="cuda") * 2.0 ** 120
    x = torch.cat((a, b), 1)
    t = mx(fmt, 256, 11008).quantize(x, swiglu=True)
    is_quantized(t, O.swiglu(f64(x)), 2.0 ** -21)
    assert engine().status() == 0


def test_linear_first_call_is_captured():
    """A context's first products under capture: what a plan asks the runtime for may be asked there."""
    e = R.Engine(engine().dims, max_batch=64, max_rows=8, max_expanded=1, max_children=1, max_tree=2, max_prefix=64, device="cuda")
    for rows, cols, outs in ((17, 1600, 130), (1162, 960, 2083), (31, 3840, 8587)):
        x, w = R.MxTensor(e, rows, cols, "fp8"), R.MxTensor(e, outs, cols, "fp8")
        x.quantize(normal(rows, rows, cols)), w.quantize(normal(outs, outs, cols) * 0.1)
        y, z = (torch.zeros(rows, (outs + 7) // 8 * 8, device="cuda") for _ in range(2))
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            R.mx_linear(x, w, y[:, :outs])
        g.replay()
        R.mx_linear(x, w, z[:, :outs])
        assert torch.equal(y, z) and bool(z[:, :outs].any())
    assert e.status() == 0
    e.close()
