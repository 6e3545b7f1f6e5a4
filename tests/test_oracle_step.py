"""The oracle of the target's step (oracle/step.py) against independent statements of the same rules (no GPU)."""
import numpy as np
import pytest
import torch

from oracle import step as O
from oracle.sampling import draw_one


def test_small_floats_are_the_types_values():
    t = torch.arange(0x7f, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(t, O.E4M3) and list(O.E2M1) == [0, 0.5, 1, 1.5, 2, 3, 4, 6]
    x = np.concatenate((np.linspace(0, 448, 20001), O.E4M3, (O.E4M3[1:] + O.E4M3[:-1]) / 2))
    want = torch.tensor(x).float().to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(O.nearest_code(O.E4M3, x), want)
    ties = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 9.0]
    assert list(O.nearest_code(O.E2M1, ties)) == [0, 2, 2, 4, 4, 6, 6, 7]


@pytest.mark.parametrize("fmt", ["fp8", "fp4", "nv4"])
def test_quantised_values_are_near(fmt):
    rng = np.random.default_rng(3)
    x = rng.standard_normal((37, 96)) * np.exp(rng.standard_normal((37, 1)) * 3)
    x[5] = 0
    g = np.abs(x).max() / 2688
    code, byte = O.quantize(fmt, x, g)
    y = O.values(fmt, code, byte, g)
    top = np.abs(x.reshape(37, -1, O.BLOCK[fmt])).max(-1).repeat(O.BLOCK[fmt], 1)
    # half a step of the element, plus, for nv4, what an 8-bit scale that rounds down cuts off (one part in 16)
    half = {"fp8": 2.0 ** -4, "fp4": 1 / 4, "nv4": 1 / 4}[fmt]
    least = {"fp8": 2.0 ** -9, "fp4": 1 / 6, "nv4": 1 / 6}[fmt]
    bound = np.abs(x) * half + top * least + (top / 16 if fmt == "nv4" else 0) + (g * 6 * 2.0 ** -9 if fmt == "nv4" else 0)
    assert (np.abs(y - x) <= bound).all() and not y[5].any()
    if fmt != "nv4":                                     # no element saturates, and no smaller scale would do
        most = 448.0 if fmt == "fp8" else 6.0
        s = 2.0 ** (byte.astype(float) - 127)
        t = np.abs(x.reshape(37, -1, 32)).max(-1)
        assert (t <= most * s).all() and (t[t > 0] > most * s[t > 0] / 2).all()
    data, scale = O.pack_bytes(fmt, code, byte, 255)
    c2, b2 = O.unpack_bytes(fmt, data, scale, 37, 96)
    n = 96 // O.BLOCK[fmt]
    assert np.array_equal(c2, code) and np.array_equal(b2[:, :n], byte) and not b2[:, n:].any()


def test_scale_layout_is_one_to_one():
    at = O.scale_layout(300, 10)
    assert at.shape == (300, 12) and len(np.unique(at)) == at.size and at.max() < 3 * 3 * 512
    assert at[0, 0] == 0 and at[1, 0] == 16 and at[32, 0] == 4 and at[0, 1] == 1 and at[0, 4] == 512 and at[128, 0] == 1536


def test_distribution_is_the_filters_in_turn():
    rng = np.random.default_rng(4)
    for _ in range(50):
        z = np.round(rng.standard_normal(60) * 2, 1)     # ties
        t, k, p, m = rng.uniform(0.3, 2), int(rng.integers(0, 70)), rng.uniform(0.1, 1.1), rng.uniform(0, 0.3)
        q = np.exp(z / t) / np.exp(z / t).sum()
        alive = sorted(range(60), key=lambda i: (-z[i], i))
        if k > 0:
            alive = alive[:k]
        if p < 1:
            total, s, n = q[alive].sum(), 0.0, 0
            while s < p * total:
                s += q[alive[n]]
                n += 1
            alive = alive[:n]
        alive = [i for i in alive if q[i] >= m * q.max() * (1 - 1e-12)]
        w = O.distribution(z, t, k, p, m)
        assert set(np.flatnonzero(w)) == set(alive)
        assert np.allclose(w / w.sum(), np.where(np.isin(np.arange(60), alive), q, 0) / q[alive].sum(), atol=1e-9)
    w = O.distribution([1.0, 3.0, 3.0], 0.0)
    assert list(w) == [0, 1 << 40, 0] and draw_one(w, 0xffffffff) == 1


def test_nv4_elements_under_the_smallest_normal_scale_are_zeros():
    """d = scale * factor below 2^-126: the elements are zeros, with their signs, whatever the block holds."""
    x = np.full((3, 16), 2.0 ** -124)
    x[:, 1::2] *= -1
    x[1:] *= [[2.0], [16.0]]
    for e in (-127, -130, -149):
        g = 2.0 ** e
        code, byte = O.quantize("nv4", x, g)
        assert byte.all() and np.array_equal(code >> 3, np.signbit(x).astype(int))
        d = (O.E4M3[byte].astype(np.float32) * np.float32(g)).astype(np.float64)[:, 0]
        assert np.array_equal((code & 7).any(1), d >= 2.0 ** -126)
    code, byte = O.quantize("nv4", x[:1], 2.0 ** -127)   # largest / (6 g) = 4 / 3: the scale 1.375, its d 1.375 2^-127
    assert O.E4M3[byte[0, 0]] == 1.375 and not (code & 7).any()
    code, byte = O.quantize("nv4", x[1:2], 2.0 ** -127)  # 8 / 3: the scale 2.75, d 1.375 2^-126, elements 8 / 1.375
    assert O.E4M3[byte[0, 0]] == 2.75 and (O.E2M1[code & 7] == 6.0).all()


def test_draws_are_as_frequent_as_their_weights():
    """Over all 2^32 words a token is drawn as often as its weight says, to one word: counted from where the draw changes."""
    rng = np.random.default_rng(6)
    for t, k, p, m in ((1.0, 0, 1.0, 0.0), (0.7, 5, 1.0, 0.0), (1.4, 0, 0.8, 0.0), (1.0, 0, 1.0, 0.1), (0.9, 12, 0.9, 0.02)):
        w = O.distribution(rng.standard_normal(25) * 2, t, k, p, m)
        total, first, before = int(w.sum()), 0, 0
        for i in np.flatnonzero(w):
            before += int(w[i])
            end = -(-(before << 32) // total)            # the first word whose share reaches the weights up to i
            assert draw_one(w, first) == i and draw_one(w, end - 1) == i
            assert abs((end - first) - 2 ** 32 * int(w[i]) / total) <= 1
            first = end
        assert first == 2 ** 32
    words = rng.integers(0, 2 ** 32, 40000)
    n = np.bincount([draw_one(w, int(u)) for u in words], minlength=25)
    share = w / w.sum()
    assert not n[w == 0].any()
    assert (np.abs(n - 40000 * share) <= 6 * np.sqrt(40000 * share) + 1).all()
