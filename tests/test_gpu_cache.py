"""The target's cache on the GPU: eagle_kv_append, eagle_chunk_attn and eagle_pages_* against the oracle
(oracle/cache.py, fp64), alone and as a serving step uses them.

Tolerances, fixed before the first run (u = 2^-8 is half a bf16 step, relative):
* append: the angle is exact to 2^-23 radians and sincospi to a few fp32 steps, so a rotated element is off by at
  most (|x1| + |x2|) m 2^-21, and by one rounding to its type;
* attention: a probability is rounded once to bf16 (u), its logit is off by delta = (dh + 4) 2^-23 sum|q k| scale plus
  2^-21 for the exponential, which enters the probability and its normalisation; sums over L keys and dh elements add
  (L + dh) 2^-23; all of it weighs the probability-weighted mean of |v|.  The output is rounded once (u).
Cache rows that no request holds are NaN, so that a stray read or write shows."""
import math
import random

import numpy as np
import pytest
import torch

from eagle_feature_level_gb300 import _binding as B
from eagle_feature_level_gb300 import runtime as R
from eagle_feature_level_gb300.runtime import _p
from oracle.cache import OutOfBlocks, Pages, chunk_attention, frequencies, rotate, rows_of

pytestmark = pytest.mark.gpu

INVALID_ARG, SHAPE, ALIGN, CAPACITY = 1, 2, 3, 4
U = 2.0 ** -8
NAN = float("nan")
_engines = {}


def engine(hq, hkv, dh, max_prefix=4096, fresh=False):
    key = (hq, hkv, dh, max_prefix)
    if fresh or key not in _engines:
        d = max(64, hq * dh)
        e = R.Engine(dict(d=d, n_q_heads=hq, n_kv_heads=hkv, head_dim=dh, d_ff=64, vocab=64), max_batch=64, max_rows=8,
                     max_expanded=1, max_children=1, max_tree=2, max_prefix=max_prefix, device="cuda")
        if fresh:
            return e
        _engines[key] = e
    return _engines[key]


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def starts(new, first=0):
    out = [first]
    for n in new:
        out.append(out[-1] + n)
    return out


def f64(t):
    return t.detach().double().cpu().numpy()


class Cache:
    """A cache for requests of lens[b] rows with room for room[b]: contiguous (bs 0) or paged with blocks in random
    order; rows past lens are NaN, blocks past room[b] are not allocated."""

    def __init__(self, lens, room, hkv, dh, bs, seed=0, cap=None):
        g = torch.Generator(device="cuda").manual_seed(seed)
        nb = len(lens)
        self.bs, self.lens = bs, list(lens)
        most = max(max(room), 1)
        self.cap = cap or (most if bs == 0 else -(-most // bs) * bs)
        self.rows = [torch.randn(2, n, hkv, dh, generator=g, device="cuda").to(torch.bfloat16) for n in lens]
        if bs == 0:
            shape, self.table, self.paging = (nb, self.cap, hkv, dh), None, B.eagle_paging()
        else:
            held = [-(-r // bs) for r in room]
            n_blocks = sum(held) + 3
            ids = random.Random(seed).sample(range(n_blocks), sum(held))
            t = [[-1] * (self.cap // bs) for _ in lens]
            for b, h in enumerate(held):
                for c in range(h):
                    t[b][c] = ids.pop()
            self.table, shape = i32(t), (n_blocks, bs, hkv, dh)
            self.paging = B.eagle_paging(_p(self.table), bs, n_blocks)
        self.k = torch.full(shape, NAN, dtype=torch.bfloat16, device="cuda")
        self.v = self.k.clone()
        for b, n in enumerate(lens):
            for c, x in ((self.k, 0), (self.v, 1)):
                c.view(-1, hkv, dh)[self.at(b, 0, n)] = self.rows[b][x]
        self.len = i32(self.lens)

    def at(self, b, lo, hi):
        """Flat rows of positions lo .. hi - 1 of request b."""
        j = torch.arange(lo, hi, device="cuda")
        if self.bs == 0:
            return b * self.cap + j
        return self.table[b].long()[j // self.bs] * self.bs + j % self.bs

    def kv(self, length=None):
        return B.eagle_kv(_p(self.k), _p(self.v), self.cap, _p(self.len if length is None else length), self.paging)


# ---- append -------------------------------------------------------------------

def run_append(eng, c, row_start, n_rows, rope, q, k, v, q_out, pos=None, kv=None):
    dtype = B.DTYPE_F32 if k.dtype == torch.float32 else B.DTYPE_BF16
    len_out = torch.full_like(c.len, -7)
    B.eagle_kv_append(eng.ctx, len(c.lens), B.eagle_rows(_p(row_start), n_rows), rope, dtype, _p(q),
                      0 if q is None else q.stride(0), _p(q_out), 0 if q is None else q_out.stride(0), _p(k),
                      k.stride(0), _p(v), v.stride(0), kv or c.kv(), _p(pos), _p(len_out), eng.ws.data_ptr(),
                      eng.stream())
    return len_out


def is_rotated(got, x, pos, freq, inter, m, u):
    want = rotate(x, pos, freq, inter, m)
    half = len(freq)
    first = np.arange(half) * 2 if inter else np.arange(half)
    second = first + 1 if inter else first + half
    size = np.abs(x)
    size[..., first] = size[..., second] = (np.abs(x[..., first]) + np.abs(x[..., second])) * m
    size[..., 2 * half:] = 0.0
    return np.abs(got - want) <= size * 2.0 ** -21 + u * np.abs(want)


def check_rotated(*args):
    assert is_rotated(*args).all()


APPENDS = [  # heads, dtype, rot, interleaved, scaling, block size, lengths before, new rows
    ((4, 4, 16), torch.bfloat16, 16, False, None, 16, [0, 5, 31], [1, 1, 1]),
    ((4, 2, 64), torch.bfloat16, 64, True, None, 1, [3, 0, 7, 9], [0, 5, 17, 0]),
    ((4, 2, 64), torch.float32, 32, False, "bands", 64, [60, 64, 100], [9, 64, 1]),
    ((8, 2, 128), torch.bfloat16, 128, False, "ramp", 256, [250, 0], [300, 700]),
    ((8, 2, 128), torch.float32, 64, True, "linear", 0, [2, 90, 0, 1], [33, 0, 1, 200]),
    ((6, 2, 32), torch.bfloat16, 2, True, None, 4, [1, 2, 3], [4, 5, 6]),
    ((6, 2, 32), torch.float32, 10, False, None, 8, [7, 8], [1, 9]),
    ((40, 40, 128), torch.bfloat16, 128, False, None, 16, [100] * 8, [1] * 8),
    ((4, 2, 64), torch.bfloat16, 0, False, None, 16, [3, 4], [20, 2]),             # no rotation
]
SC = {"linear": (4.0, 0.0, 0.0, 0), "bands": (8.0, 1.0, 4.0, 8192), "ramp": (16.0, 1.0, 32.0, 4096)}
KIND = {"linear": B.ROPE_LINEAR, "bands": B.ROPE_BANDS, "ramp": B.ROPE_RAMP}


def rope_and_freq(dh, rot, inter, scaling, theta=1e4):
    if rot == 0:
        return None, np.zeros(0), 1.0
    sc = None if scaling is None else B.eagle_rope_scaling(KIND[scaling], *SC[scaling], 0.0)
    r = B.eagle_rope_plan(dh, rot, int(inter), theta, sc)
    return r, frequencies(rot, theta, scaling or "none", *(SC[scaling] if scaling else ())), float(r.mscale)


@pytest.mark.parametrize("heads,dtype,rot,inter,scaling,bs,ctx,new", APPENDS)
@pytest.mark.parametrize("fused", [False, True])
def test_append(heads, dtype, rot, inter, scaling, bs, ctx, new, fused):
    hq, hkv, dh = heads
    eng = engine(*heads)
    rope, freq, m = rope_and_freq(dh, rot, inter, scaling)
    c = Cache(ctx, [a + n for a, n in zip(ctx, new)], hkv, dh, bs, seed=3)
    total, pad = sum(new), 4
    n_rows = total + pad
    g = torch.Generator(device="cuda").manual_seed(5)
    if fused:                              # slices of one projection, q rotated in place
        x = torch.randn(n_rows, hq + 2 * hkv, dh, generator=g, device="cuda").to(dtype)
        q, k, v = x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:]
        q_out = q
    else:
        q, k, v = (torch.randn(n_rows, h, dh, generator=g, device="cuda").to(dtype) for h in (hq, hkv, hkv))
        q_out = torch.full_like(q, NAN)
    first = 2                              # two rows before the first request's, two behind the last's
    rs = i32(starts(new, first))
    q0, k0, v0 = f64(q), f64(k), f64(v)
    before = c.k.clone(), c.v.clone()
    ln = run_append(eng, c, rs, n_rows, rope, q, k, v, q_out)
    torch.cuda.synchronize()
    assert eng.status() == 0
    assert ln.tolist() == [a + n for a, n in zip(ctx, new)]
    u = U if dtype == torch.bfloat16 else 2.0 ** -24
    got = f64(q_out)
    r = first
    for b, n in enumerate(new):
        pos = np.arange(ctx[b], ctx[b] + n)
        check_rotated(got[r:r + n], q0[r:r + n], pos, freq, inter, m, u)
        at = c.at(b, ctx[b], ctx[b] + n)
        check_rotated(f64(c.k.view(-1, hkv, dh)[at]), k0[r:r + n], pos, freq, inter, m, U)
        assert torch.equal(c.v.view(-1, hkv, dh)[at], v[r:r + n].to(torch.bfloat16))
        for now, old in zip((c.k, c.v), before):           # put back, to compare the rest
            now.view(-1, hkv, dh)[at] = old.view(-1, hkv, dh)[at]
        r += n
    for now, old in zip((c.k, c.v), before):               # nothing else of the cache was written
        assert torch.equal(now.view(torch.int16), old.view(torch.int16))
    for rows in (slice(0, first), slice(first + total, None)):
        if fused:
            assert np.array_equal(got[rows], q0[rows])
        else:
            assert np.isnan(got[rows]).all()


def test_append_far_and_given_positions():
    hq, hkv, dh = 8, 2, 128
    eng = engine(hq, hkv, dh)
    rope, freq, m = rope_and_freq(dh, 128, False, None, 5e5)
    pos = [0, 1, 131071, 1 << 20, (1 << 31) - 1, 77, 77]
    c = Cache([0, 4], [5, 6], hkv, dh, 8, seed=1)
    q, k, v = (torch.randn(7, h, dh, device="cuda") for h in (hq, hkv, hkv))
    out = torch.empty_like(q)
    run_append(eng, c, i32([0, 5, 7]), 7, rope, q, k, v, out, pos=i32(pos))
    torch.cuda.synchronize()
    assert eng.status() == 0
    # the oracle's own angle: a position of 2^31 times a frequency of relative error 2^-52 is off by 2^-20
    want = rotate(f64(q), pos, freq, False)
    x = f64(q)
    size = np.concatenate([np.abs(x[..., :64]) + np.abs(x[..., 64:])] * 2, axis=-1)
    slack = 2.0 ** -21 + np.array(pos, dtype=np.float64)[:, None, None] * 2.0 ** -51
    assert (np.abs(f64(out) - want) <= size * slack + 2.0 ** -24 * np.abs(want)).all()


def test_append_keys_alone_and_other_stream():
    hq, hkv, dh = 4, 2, 64
    eng = engine(hq, hkv, dh, fresh=True)
    c = Cache([1, 2], [4, 9], hkv, dh, 4)
    k, v = torch.randn(10, hkv, dh, device="cuda"), torch.randn(10, hkv, dh, device="cuda")
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        ln = run_append(eng, c, i32([0, 3, 10]), 10, None, None, k, v, None)
    s.synchronize()
    assert eng.status() == 0 and ln.tolist() == [4, 9]
    assert torch.equal(c.k.view(-1, hkv, dh)[c.at(1, 2, 9)], k[3:].to(torch.bfloat16))
    eng.close()


@pytest.mark.parametrize("bs", [0, 4])
def test_append_refuses_a_request_whole(bs):
    hq, hkv, dh = 4, 2, 64
    eng = engine(hq, hkv, dh)
    rope, freq, m = rope_and_freq(dh, 64, False, None)
    ctx, new = [2, 3, 6], [3, 20, 2]                       # request 1 has room for 12 rows only
    c = Cache(ctx, [5, 12, 8], hkv, dh, bs, cap=12)
    q, k, v = (torch.randn(25, h, dh, device="cuda").to(torch.bfloat16) for h in (hq, hkv, hkv))
    out = torch.zeros_like(q)
    kb, vb = c.k.clone(), c.v.clone()
    ln = run_append(eng, c, i32(starts(new)), 25, rope, q, k, v, out)
    torch.cuda.synchronize()
    assert eng.status() == CAPACITY
    assert ln.tolist() == [5, 3, 8]
    mine = c.at(1, 0, 12)
    assert torch.equal(c.k.view(-1, hkv, dh)[mine].view(torch.int16), kb.view(-1, hkv, dh)[mine].view(torch.int16))
    assert torch.equal(c.v.view(-1, hkv, dh)[mine].view(torch.int16), vb.view(-1, hkv, dh)[mine].view(torch.int16))
    check_rotated(f64(out[3:23]), f64(q[3:23]), np.arange(3, 23), freq, False, m, U)
    assert torch.equal(c.v.view(-1, hkv, dh)[c.at(2, 6, 8)], v[23:])


def test_append_unallocated_and_bad_starts():
    hq, hkv, dh = 4, 2, 64
    eng = engine(hq, hkv, dh)
    c = Cache([2, 3], [9, 9], hkv, dh, 4)
    c.table[0, 1] = -1
    c.table[1, 1] = 10 ** 6                                # no block of the pool
    k, v = (torch.randn(6, hkv, dh, device="cuda").to(torch.bfloat16) for _ in range(2))
    kb = c.k.clone()
    ln = run_append(eng, c, i32([0, 3, 6]), 6, None, None, k, v, None)
    torch.cuda.synchronize()
    assert eng.status() == CAPACITY and ln.tolist() == [2, 3]
    assert torch.equal(c.k.view(torch.int16), kb.view(torch.int16))
    for rs in ([0, 5, 3], [-1, 2, 7], [4, 2, 9]):
        c = Cache([0, 0], [9, 9], hkv, dh, 4)
        ln = run_append(eng, c, i32(rs), 6, None, None, k, v, None)
        torch.cuda.synchronize()
        assert eng.status() == INVALID_ARG
        good = [0 <= a <= z <= 6 for a, z in zip(rs, rs[1:])]
        assert ln.tolist() == [z - a if g else 0 for a, z, g in zip(rs, rs[1:], good)]


# ---- attention ------------------------------------------------------------------

def attend(eng, c, row_start, q, out, window=0, scale=None, kv=None):
    B.eagle_chunk_attn(eng.ctx, len(c.lens), B.eagle_rows(_p(row_start), q.shape[0]), _p(q), q.stride(0),
                       kv or c.kv(), window, scale or 1.0 / math.sqrt(q.shape[2]), _p(out), out.stride(0),
                       eng.ws.data_ptr(), eng.stream())


def check_attention(got, q, k, v, scale, window):
    want, mean_abs, reach = chunk_attention(q, k, v, scale, window)
    L, dh = k.shape[0], q.shape[2]
    delta = (dh + 4) * 2.0 ** -23 * reach + 2.0 ** -21
    tol = mean_abs * (U + 2 * delta[..., None] + (L + dh) * 2.0 ** -23) + U * np.abs(want) + 1e-30
    err = np.abs(got - want)
    assert np.isfinite(got).all()
    assert (err <= tol).all(), float((err / tol).max())


def attention_case(heads, bs, lens, new, window=0, seed=0, gain=1.0, scale=None, cap=None, eng=None):
    hq, hkv, dh = heads
    eng = eng or engine(*heads)
    c = Cache(lens, lens, hkv, dh, bs, seed=seed, cap=cap)
    first, total = 1, sum(new)
    n_rows = first + total + 3
    g = torch.Generator(device="cuda").manual_seed(seed + 100)
    buf = (gain * torch.randn(n_rows, hq + 2, dh, generator=g, device="cuda")).to(torch.bfloat16)
    q = buf[:, :hq]                                        # a slice: pitch above the row
    obuf = torch.full((n_rows, hq + 1, dh), NAN, dtype=torch.bfloat16, device="cuda")
    out = obuf[:, :hq]
    rs = i32(starts(new, first))
    scale = scale or 1.0 / math.sqrt(dh)
    attend(eng, c, rs, q, out, window, scale)
    torch.cuda.synchronize()
    assert eng.status() == 0
    r = first
    for b, n in enumerate(new):
        check_attention(f64(out[r:r + n]), f64(q[r:r + n]), f64(c.rows[b][0]), f64(c.rows[b][1]), scale, window)
        r += n
    assert torch.isnan(obuf[:first]).all() and torch.isnan(obuf[first + total:]).all()
    assert torch.isnan(obuf[:, hq:]).all()                 # nothing behind a row's heads
    again = torch.full_like(obuf, NAN)
    attend(eng, c, rs, q, again[:, :hq], window, scale)
    torch.cuda.synchronize()
    assert torch.equal(again.view(torch.int16), obuf.view(torch.int16))   # the same bits every time
    return c, q, out


HEADS = [(4, 4, 16), (6, 2, 32), (4, 2, 64), (5, 1, 64), (8, 2, 128), (4, 4, 128), (32, 2, 128), (40, 8, 128)]


@pytest.mark.parametrize("heads", HEADS, ids=lambda h: "x".join(map(str, h)))
@pytest.mark.parametrize("bs", [0, 16])
def test_attention_single_tokens(heads, bs):
    attention_case(heads, bs, [1, 2, 63, 64, 65, 127, 128, 129, 300, 1025], [1] * 10, seed=1)


@pytest.mark.parametrize("heads", HEADS, ids=lambda h: "x".join(map(str, h)))
@pytest.mark.parametrize("bs", [0, 16, 256])
def test_attention_chunks(heads, bs):
    attention_case(heads, bs, [1, 40, 128, 129, 257, 700, 333], [1, 40, 128, 1, 130, 33, 0], seed=2)


@pytest.mark.parametrize("bs", [1, 2, 4, 8, 32, 64, 128])
@pytest.mark.parametrize("heads", [(8, 2, 128), (4, 2, 64)], ids=["dh128", "dh64"])
def test_attention_block_sizes(bs, heads):
    attention_case(heads, bs, [5, 130, 260, 1000], [5, 1, 70, 300], seed=3)


@pytest.mark.parametrize("window", [1, 2, 100, 128, 129, 1000, 10 ** 6, 2 ** 31 - 1])
@pytest.mark.parametrize("heads", [(8, 2, 128), (16, 4, 64)], ids=["dh128", "dh64"])
def test_attention_window(window, heads):
    attention_case(heads, 16, [1, 300, 700, 1500], [1, 300, 1, 520], window=window, seed=4)


def test_attention_long_requests():
    attention_case((64, 8, 128), 64, [4000, 3000], [1, 1], seed=5)
    attention_case((16, 16, 128), 16, [2000], [600], seed=6)
    attention_case((8, 2, 128), 0, [1600, 1600], [1600, 1599], seed=7)


def test_attention_large_scores():
    """Scores far apart (a maximum that keeps moving), and so large that all but one probability vanish."""
    attention_case((8, 2, 128), 16, [700, 1], [200, 1], seed=8, gain=40.0)
    attention_case((4, 2, 64), 0, [500, 300], [1, 300], seed=9, gain=8.0, scale=2.0)


def test_attention_many_requests():
    rng = random.Random(4)
    lens = [rng.choice([1, 3, 50, 128, 200, 513]) for _ in range(64)]
    new = [rng.choice([0, 1, 1, 1, min(n, 17), n]) for n in lens]
    attention_case((8, 2, 128), 16, lens, new, seed=10)
    attention_case((4, 2, 64), 0, lens, new, seed=11)


def test_attention_rising_scores():
    """Keys whose score grows along the sequence: every tile raises the running maximum."""
    hq, hkv, dh = 8, 2, 128
    eng = engine(hq, hkv, dh)
    L, n = 1000, 150
    c = Cache([L], [L], hkv, dh, 16, seed=12)
    ramp = torch.linspace(-3, 3, L, device="cuda")[:, None, None]
    c.rows[0][0] = (torch.ones(L, hkv, dh, device="cuda") * ramp).to(torch.bfloat16)
    c.k.view(-1, hkv, dh)[c.at(0, 0, L)] = c.rows[0][0]
    q = torch.ones(n, hq, dh, device="cuda", dtype=torch.bfloat16) * 2
    q[:, 1::2] *= -1
    out = torch.empty_like(q)
    attend(eng, c, i32([0, n]), q, out)
    torch.cuda.synchronize()
    check_attention(f64(out), f64(q), f64(c.rows[0][0]), f64(c.rows[0][1]), 1 / math.sqrt(dh), 0)


@pytest.mark.parametrize("heads", [(8, 2, 128), (4, 2, 64)], ids=["dh128", "dh64"])
def test_attention_rows_without_keys(heads):
    """A length shorter than the rows: the rows before the first key are zero."""
    hq, hkv, dh = heads
    eng = engine(*heads)
    c = Cache([0, 5, 140], [0, 5, 140], hkv, dh, 16, seed=13)
    q = torch.randn(180, hq, dh, device="cuda").to(torch.bfloat16)
    out = torch.full_like(q, NAN)
    attend(eng, c, i32([0, 3, 20, 180]), q, out)
    torch.cuda.synchronize()
    assert eng.status() == 0
    assert not out[:3].any() and not out[3:15].any() and not out[20:40].any()
    for b, lo, hi in ((1, 3, 20), (2, 20, 180)):
        check_attention(f64(out[lo:hi]), f64(q[lo:hi]), f64(c.rows[b][0]), f64(c.rows[b][1]), 1 / math.sqrt(dh), 0)


@pytest.mark.parametrize("heads", [(8, 2, 128), (4, 2, 64)], ids=["dh128", "dh64"])
@pytest.mark.parametrize("bs", [4, 16])
def test_attention_reports_bad_pages_and_lengths(heads, bs):
    hq, hkv, dh = heads
    eng = engine(*heads)
    lens = [300, 290]
    c = Cache(lens, lens, hkv, dh, bs, seed=14)
    for blk, bad in ((1, -1), (3, 10 ** 7)):
        c.table[1, blk] = bad
        c.rows[1][:, blk * bs:(blk + 1) * bs] = 0          # reads as zeros
    q = torch.randn(41, hq, dh, device="cuda").to(torch.bfloat16)
    out = torch.empty_like(q)
    attend(eng, c, i32([0, 1, 41]), q, out)
    torch.cuda.synchronize()
    assert eng.status() == INVALID_ARG
    for b, lo, hi in ((0, 0, 1), (1, 1, 41)):
        check_attention(f64(out[lo:hi]), f64(q[lo:hi]), f64(c.rows[b][0]), f64(c.rows[b][1]), 1 / math.sqrt(dh), 0)
    # a length beyond the cache is read as the cache
    c = Cache([c.cap, 20], [c.cap, 20], hkv, dh, bs, seed=15)
    attend(eng, c, i32([0, 2, 12]), q[:12], out[:12], kv=c.kv(i32([c.cap + 9, 20])))
    torch.cuda.synchronize()
    assert eng.status() == CAPACITY
    check_attention(f64(out[:2]), f64(q[:2]), f64(c.rows[0][0]), f64(c.rows[0][1]), 1 / math.sqrt(dh), 0)
    # starts out of bounds: that request has no rows
    out.fill_(NAN)
    attend(eng, c, i32([5, 2, 12]), q[:12], out[:12])
    torch.cuda.synchronize()
    assert eng.status() == INVALID_ARG
    assert torch.isnan(out[:2]).all() and torch.isfinite(out[2:12]).all()


def test_attention_two_streams():
    """Two contexts at work at once on one GPU, each on its own stream and workspace."""
    heads = (8, 2, 128)
    engs = [engine(*heads, fresh=True) for _ in range(2)]
    work = []
    for i in range(2):
        c = Cache([900, 400, 77], [900, 400, 77], 2, 128, 16, seed=20 + i)
        q = torch.randn(300, 8, 128, device="cuda").to(torch.bfloat16)
        work.append((c, q, i32([0, 1, 250, 300])))
    alone = []
    for (c, q, rs), e in zip(work, engs):
        o = torch.empty_like(q)
        attend(e, c, rs, q, o)
        torch.cuda.synchronize()
        alone.append(o)
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [[torch.zeros_like(q) for _ in range(8)] for c, q, rs in work]
    torch.cuda.synchronize()
    for j in range(8):
        for i, (c, q, rs) in enumerate(work):
            with torch.cuda.stream(streams[i]):
                attend(engs[i], c, rs, q, outs[i][j])
    torch.cuda.synchronize()
    for i in range(2):
        assert engs[i].status() == 0
        for o in outs[i]:
            assert torch.equal(o, alone[i])
        engs[i].close()


@pytest.mark.parametrize("heads", [(24, 1, 64), (17, 1, 128), (144, 1, 64), (300, 1, 64)],
                         ids=lambda h: "x".join(map(str, h)))
def test_attention_many_heads_a_group(heads):
    """More query heads a kv head than the few-row tile has rows, and than a tensor-core tile has."""
    attention_case(heads, 16, [1, 130, 300], [1, 3, 1], seed=30)
    attention_case(heads, 0, [260, 40], [37, 0], window=50, seed=31)


@pytest.mark.parametrize("heads", [(8, 2, 128), (4, 2, 64)], ids=["dh128", "dh64"])
def test_attention_small_contiguous_caches(heads):
    """Caches shorter than a tile of keys."""
    attention_case(heads, 0, [1], [1], seed=32)
    attention_case(heads, 0, [3, 2], [3, 1], seed=33)
    attention_case(heads, 0, [5, 9, 30], [5, 9, 30], seed=34, cap=30)


@pytest.mark.parametrize("heads", [(8, 2, 128), (4, 4, 64)], ids=["dh128", "dh64"])
def test_attention_short_prompts_between_long_ones(heads):
    """Items of two query tiles and several key tiles beside items of one query tile and one key tile, in turn: one
    softmax group has nothing to do in the latter and may be a segment ahead of the other."""
    G = heads[0] // heads[1]
    T = 128 // G
    lens, new = [], []
    for i in range(32):
        lens += [2 * T + 1 + i, T if T <= 128 else 128]
        new += [2 * T, T - i % 3]
    attention_case(heads, 16, lens, new, seed=50)


@pytest.mark.parametrize("heads,requests", [((40, 8, 128), 12), ((16, 4, 64), 21)], ids=["dh128", "dh64"])
def test_attention_long_decoding_beside_prompts(heads, requests):
    """Enough single tokens over long prefixes that they keep their own phase beside a prompt's tiles."""
    lens = [4000 - 7 * i for i in range(requests)] + [300, 200]
    new = [1] * (requests - 1) + [2, 150, 200]
    attention_case(heads, 16, lens, new, seed=51)
    attention_case(heads, 0, lens, new, window=3500, seed=52)


@pytest.mark.parametrize("heads", [(20, 2, 128), (10, 2, 128), (12, 1, 64), (7, 1, 64)],
                         ids=lambda h: "x".join(map(str, h)))
def test_attention_rows_that_end_inside_a_warp(heads):
    """Groups whose tokens do not fill a tile's 128 rows, and items whose tokens end inside a warp's 32: lanes with and
    without a row read the same accumulator column by column.  Items of one and of two tiles, whole and split."""
    T = 128 // (heads[0] // heads[1])
    lens = [2 * T + 5, T - 1, 2500, 1 + T, 129, 700, 4, 300]
    new = [2 * T + 5, T - 1, T + 3, 1 + T, 2, 333, 4, T // 2 + 1]
    attention_case(heads, 16, lens, new, seed=60)
    attention_case(heads, 0, [3000], [2 * T - 1], seed=61)                    # few items, each split over many CTAs
    attention_case(heads, 16, lens * 4, new * 4, window=150, seed=62)         # many short ones


@pytest.mark.parametrize("heads", [(8, 2, 128), (4, 2, 64)], ids=["dh128", "dh64"])
def test_attention_one_tile_items_over_many_key_tiles(heads):
    """Items of one query tile: the softmax groups share the key tiles, and each reads both groups' accumulators.  Long
    ones back to back on a CTA, of even and odd numbers of key tiles."""
    T = 128 // (heads[0] // heads[1])
    lens = [128 * (2 + i % 7) + i for i in range(60)]
    new = [T - i % 5 for i in range(60)]
    attention_case(heads, 16, lens, new, seed=63)
    attention_case(heads, 0, lens[:5], new[:5], seed=64)


def test_attention_hundreds_of_requests():
    rng = random.Random(5)
    eng = R.Engine(dict(d=256, n_q_heads=4, n_kv_heads=2, head_dim=64, d_ff=64, vocab=64), max_batch=301, max_rows=8,
                   max_expanded=1, max_children=1, max_tree=2, max_prefix=512, device="cuda")
    lens = [rng.choice([1, 2, 20, 130, 257]) for _ in range(301)]
    new = [rng.choice([0, 1, 1, 1, min(n, 3), n]) for n in lens]
    attention_case((4, 2, 64), 16, lens, new, seed=35, eng=eng)
    attention_case((4, 2, 64), 0, lens, [1] * 301, seed=36, eng=eng)
    eng.close()


def test_idle_requests_may_hold_any_length():
    """A padded batch: the length of a request without rows is neither used nor reported."""
    heads = hq, hkv, dh = 8, 2, 128
    eng = engine(*heads)
    for bs in (0, 16):
        c = Cache([6, 0, 40, 0], [12, 12, 41, 12], hkv, dh, bs, seed=37)
        c.len.copy_(i32([6, -9, 40, 10 ** 9]))
        x = torch.randn(4, hq + 2 * hkv, dh, device="cuda").to(torch.bfloat16)
        out = torch.zeros(4, hq, dh, dtype=torch.bfloat16, device="cuda")
        rs = i32([0, 3, 3, 4, 4])
        ln = run_append(eng, c, rs, 4, None, x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:], x[:, :hq])
        attend(eng, c, rs, x[:, :hq], out, kv=c.kv(ln))
        torch.cuda.synchronize()
        assert eng.status() == 0 and ln.tolist() == [9, -9, 41, 10 ** 9]
        for b, lo, hi in ((0, 0, 3), (2, 3, 4)):
            k, v = (np.concatenate([f64(c.rows[b][i]), f64(x[lo:hi, hq + i * hkv:hq + (i + 1) * hkv])]) for i in (0, 1))
            check_attention(f64(out[lo:hi]), f64(x[lo:hi, :hq]), k, v, 1 / math.sqrt(dh), 0)


def test_blocks_beyond_32_bit_offsets():
    """Pools of more than 2^32 elements: append, attention, the copy of a shared tail and compaction at their end."""
    hq, hkv, dh, bs = 8, 2, 128, 256
    eng = engine(hq, hkv, dh)
    n_blocks = (1 << 32) // (bs * hkv * dh) + 20
    c = R.PagedCache.__new__(R.PagedCache)
    zeros, torch.zeros = torch.zeros, lambda *s, **k: torch.empty(*s, **k)     # (the pools need no contents)
    try:
        c.__init__(eng, 2, bs, n_blocks, 4)
    finally:
        torch.zeros = zeros
    c.clear()
    last = n_blocks - 1
    c.table[0, 0], c.ref[last], c.ref[:last - 3] = last, 1, 1                   # the free blocks are last - 3 .. last - 1
    x = torch.randn(300, hq + 2 * hkv, dh, device="cuda").to(torch.bfloat16)
    q, k, v = x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:]
    out = torch.zeros(300, hq, dh, dtype=torch.bfloat16, device="cuda")

    def step(new):
        rs = i32(starts(new))
        c.reserve(i32(new))
        c.append(0, rs, None, q, k, v)
        c.attend(0, rs, q, out)
        c.advance()
        torch.cuda.synchronize()
        assert eng.status() == 0

    def check(row0, n, rows):
        kk, vv = (np.concatenate([f64(t[a:z]) for a, z in rows]) for t in (k, v))
        check_attention(f64(out[row0:row0 + n]), f64(q[row0:row0 + n]), kk, vv, 1 / math.sqrt(dh), 0)

    step([200, 0])
    check(0, 200, [(0, 200)])
    c.fork(i32([0]), i32([1]))
    step([1, 100])                                         # sequence 0 gets a copy of the tail, 1 keeps the block
    assert c.table[:, 0].tolist() == [last - 3, last] and c.table[1, 1] == last - 2
    check(0, 1, [(0, 200), (0, 1)])
    check(1, 100, [(0, 200), (1, 101)])
    c.ref[:last - 3] = 0
    before = [t[i].clone() for t in (c.k[0], c.v[0]) for i in (last - 3, last - 2, last)]
    c.compact()
    torch.cuda.synchronize()
    assert eng.status() == 0
    assert c.table[:, :2].tolist() == [[0, -1], [2, 1]] and c.ref[:4].tolist() == [1, 1, 1, 0]
    for t, w in zip([t[i] for t in (c.k[0], c.v[0]) for i in range(3)], before):
        assert torch.equal(t.view(torch.int16), w.view(torch.int16))


def test_two_graphs_on_one_workspace():
    """Captured calls of different batches share the partials and counters of one workspace, replayed in turn."""
    heads = (8, 2, 128)
    eng = engine(*heads, fresh=True)
    work = []
    for i, (lens, new) in enumerate([([3000, 700], [1, 300]), ([900, 90, 2000, 5], [1, 1, 1, 1]), ([1500], [1500])]):
        c = Cache(lens, lens, 2, 128, 16, seed=40 + i)
        q = torch.randn(sum(new), 8, 128, device="cuda").to(torch.bfloat16)
        rs, o = i32(starts(new)), torch.empty_like(q)
        attend(eng, c, rs, q, o)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        again = torch.zeros_like(o)
        with torch.cuda.graph(g):
            attend(eng, c, rs, q, again)
        work.append((c, q, rs, o, again, g))
    for i in (0, 1, 2, 2, 0, 1, 0, 2, 1):
        work[i][5].replay()
    torch.cuda.synchronize()
    assert eng.status() == 0
    for c, q, rs, o, again, g in work:
        assert torch.equal(o, again)
    eng.close()


# ---- starts that break their bounds ---------------------------------------------------

def random_starts(seed):
    """Starts in order but for a few, some of those out of bounds; more than a warp of requests in half of them."""
    rng = random.Random(seed)
    nb, n = rng.choice([(3, 6), (7, 12), (40, 60), (64, 50)])
    rs = sorted(rng.randint(0, n) for _ in range(nb + 1))
    for _ in range(rng.randint(1, 3)):
        rs[rng.randrange(nb + 1)] = rng.choice([-1, 0, n, n + 1, 10 ** 9, rng.randint(0, n), rng.randint(0, n)])
    return rs, n


STARTS = [([0, 5, 3], 6), ([0, 100, 2, 6], 6), ([0, 4, 2, 6], 6), ([4, 6, 0, 3], 6), ([-1, 2, 6], 6), ([6, 6, 0, 6], 6),
          ([2, 5, 1, 4, 6], 6), ([0, 3, 7, 2, 6], 6), ([0, 2, 4, 6], 6)] + [random_starts(i) for i in range(16)]


@pytest.mark.parametrize("rs,n", STARTS, ids=lambda x: "_".join(map(str, x[:5])) if isinstance(x, list) else str(x))
@pytest.mark.parametrize("bs", [0, 16])
@pytest.mark.parametrize("in_place", [False, True])
def test_rows_and_lengths_agree_whatever_the_starts(rs, n, bs, in_place):
    """A request has the rows of its own two starts, all of them, or none: appended, counted and attended alike."""
    hq, hkv, dh = 4, 2, 64
    eng = engine(hq, hkv, dh)
    rope, freq, m = rope_and_freq(dh, dh, False, None)
    nb, held = len(rs) - 1, rows_of(rs, n)
    ctx = [(7 * b) % 23 for b in range(nb)]
    c = Cache(ctx, [a + n for a in ctx], hkv, dh, bs, seed=nb)
    g = torch.Generator(device="cuda").manual_seed(n)
    q, k, v = (torch.randn(n, h, dh, generator=g, device="cuda").to(torch.bfloat16) for h in (hq, hkv, hkv))
    q0, q_out, out = q.clone(), q if in_place else torch.full_like(q, NAN), torch.full_like(q, NAN)
    before = c.k.clone(), c.v.clone()
    ln = run_append(eng, c, i32(rs), n, rope, q, k, v, q_out)
    torch.cuda.synchronize()
    broken = any(not 0 <= a <= z <= n for a, z in zip(rs, rs[1:]))
    assert eng.status() == (INVALID_ARG if broken else 0)
    assert ln.tolist() == [a + hi - lo for a, (lo, hi) in zip(ctx, held)]
    attend(eng, c, i32(rs), q_out, out, kv=c.kv(ln))
    torch.cuda.synchronize()
    assert eng.status() == (INVALID_ARG if broken else 0)
    owners = np.zeros(n, dtype=int)
    for lo, hi in held:
        owners[lo:hi] += 1
    turned = np.zeros(n, dtype=bool)                       # a row's query turns once, by one of its requests' positions
    for b, (lo, hi) in enumerate(held):
        if lo == hi:
            continue
        pos, at = np.arange(ctx[b], ctx[b] + hi - lo), c.at(b, ctx[b], ctx[b] + hi - lo)
        turned[lo:hi] |= is_rotated(f64(q_out[lo:hi]), f64(q0[lo:hi]), pos, freq, False, m, U).all((1, 2))
        kc, vc = c.k.view(-1, hkv, dh)[at].clone(), c.v.view(-1, hkv, dh)[at].clone()
        check_rotated(f64(kc), f64(k[lo:hi]), pos, freq, False, m, U)
        assert torch.equal(vc, v[lo:hi])
        kk, vv = (np.concatenate([f64(c.rows[b][i]), f64(x)]) for i, x in ((0, kc), (1, vc)))
        if (owners[lo:hi] == 1).all():
            check_attention(f64(out[lo:hi]), f64(q_out[lo:hi]), kk, vv, 1 / math.sqrt(dh), 0)
        for now, old in zip((c.k, c.v), before):           # put back, to compare the rest
            now.view(-1, hkv, dh)[at] = old.view(-1, hkv, dh)[at]
    for now, old in zip((c.k, c.v), before):
        assert torch.equal(now.view(torch.int16), old.view(torch.int16))
    assert (turned == (owners > 0)).all()
    free = torch.tensor(owners == 0, device="cuda")
    assert torch.isnan(out[free]).all() and torch.isfinite(out[~free]).all()
    assert torch.equal(q_out[free], q0[free]) if in_place else torch.isnan(q_out[free]).all()


def test_append_broken_starts_among_many_requests():
    """More requests than two levels of the search for a row's request reach, some prompts among them."""
    hq, hkv, dh, nb, n = 4, 2, 64, 1100, 1500
    eng = R.Engine(dict(d=256, n_q_heads=hq, n_kv_heads=hkv, head_dim=dh, d_ff=64, vocab=64), max_batch=nb, max_rows=8,
                   max_expanded=1, max_children=1, max_tree=2, max_prefix=512, device="cuda")
    rng = random.Random(7)
    for broken in (0, 1, 3, 40):
        rs = sorted(rng.choice([0, 40, 41, 300, 301, 1400, n, rng.randint(0, n), rng.randint(0, n)]) for _ in range(nb + 1))
        for _ in range(broken):
            rs[rng.randrange(nb + 1)] = rng.choice([-5, 0, n, n + 1, rng.randint(0, n), rng.randint(0, n)])
        held = [(lo, hi) if hi - lo <= 512 else (0, 0) for lo, hi in rows_of(rs, n)]     # (no room for more)
        k, v = (torch.randn(n, hkv, dh, device="cuda").to(torch.bfloat16) for _ in range(2))
        kc = torch.full((nb, 512, hkv, dh), NAN, dtype=torch.bfloat16, device="cuda")
        vc = kc.clone()
        want_k, want_v = kc.clone(), vc.clone()
        for b, (lo, hi) in enumerate(held):
            want_k[b, :hi - lo], want_v[b, :hi - lo] = k[lo:hi], v[lo:hi]
        ln = i32([0] * nb)
        out = torch.full_like(ln, -7)
        B.eagle_kv_append(eng.ctx, nb, B.eagle_rows(_p(i32(rs)), n), None, B.DTYPE_BF16, 0, 0, 0, 0, _p(k), k.stride(0),
                          _p(v), v.stride(0), B.eagle_kv(_p(kc), _p(vc), 512, _p(ln)), None, _p(out),
                          eng.ws.data_ptr(), eng.stream())
        torch.cuda.synchronize()
        assert (eng.status() == 0) == (held == list(zip(rs, rs[1:])))
        assert out.tolist() == [hi - lo for lo, hi in held]
        assert torch.equal(kc.view(torch.int16), want_k.view(torch.int16))
        assert torch.equal(vc.view(torch.int16), want_v.view(torch.int16))
    eng.close()


# ---- refusals before any launch ---------------------------------------------------

def test_arguments_checked_before_launch():
    eng = engine(8, 2, 128)
    before = B.eagle_launch_count(eng.ctx)
    x = torch.zeros(1 << 16, dtype=torch.bfloat16, device="cuda")
    a, ws, st = _p(x), eng.ws.data_ptr(), eng.stream()
    i = _p(i32([0, 1]))
    kv = B.eagle_kv(a, a, 64, i)
    rows = B.eagle_rows(i, 4)
    rope = B.eagle_rope_plan(128, 128, 0, 1e4)
    wide = B.eagle_rope_plan(128, 128, 0, 1e4)
    wide.rot_dim = 130

    def append(rows=rows, rope=rope, dtype=0, q=a, ldq=1024, qo=a, ldqo=1024, k=a, ldk=256, v=a, ldv=256, kv=kv,
               pos=None, lo=a, batch=1, ws=ws):
        B.eagle_kv_append(eng.ctx, batch, rows, rope, dtype, q, ldq, qo, ldqo, k, ldk, v, ldv, kv, pos, lo, ws, st)

    def attn(rows=rows, q=a, ldq=1024, kv=kv, w=0, scale=1.0, out=a + 4096, ldo=1024, batch=1, ws=ws):
        B.eagle_chunk_attn(eng.ctx, batch, rows, q, ldq, kv, w, scale, out, ldo, ws, st)

    good = dict(t=a, l=a, r=a, s=a, n=2, per=4, bs=16, nb=8)

    def pages(**k):
        g = dict(good, **k)
        return B.eagle_pages(g["t"], g["l"], g["r"], g["s"], g["n"], g["per"], g["bs"], g["nb"])

    def reserve(pools=None, n_new=a, **k):
        B.eagle_pages_reserve(eng.ctx, pages(**k), pools or B.eagle_pools([a], [a]), n_new, ws, st)

    many = B.eagle_pools([a] * 129, [a] * 129)
    odd = B.eagle_pools([a + 2], [a])
    cases = [
        (lambda: append(batch=0), CAPACITY), (lambda: append(batch=65), CAPACITY),
        (lambda: append(rows=B.eagle_rows(0, 4)), INVALID_ARG), (lambda: append(rows=B.eagle_rows(i, 0)), INVALID_ARG),
        (lambda: append(dtype=2), INVALID_ARG), (lambda: append(rope=wide), SHAPE),
        (lambda: append(ldq=1016), SHAPE), (lambda: append(ldk=260), ALIGN), (lambda: append(ldv=248), SHAPE),
        (lambda: append(q=0), INVALID_ARG), (lambda: append(qo=0), INVALID_ARG),
        (lambda: append(ldq=1032), INVALID_ARG),           # in place at another pitch
        (lambda: append(k=0), INVALID_ARG), (lambda: append(k=a + 8), ALIGN), (lambda: append(lo=i), INVALID_ARG),
        (lambda: append(lo=0), INVALID_ARG), (lambda: append(pos=a + 4), ALIGN), (lambda: append(ws=ws + 16), ALIGN),
        (lambda: append(kv=B.eagle_kv(a, a, 8192, i)), CAPACITY),
        (lambda: append(kv=B.eagle_kv(a, a, 64, i, B.eagle_paging(a, 24, 4))), INVALID_ARG),
        (lambda: attn(batch=65), CAPACITY), (lambda: attn(rows=B.eagle_rows(i, -1)), INVALID_ARG),
        (lambda: attn(q=0), INVALID_ARG), (lambda: attn(ldq=1028), ALIGN), (lambda: attn(ldo=512), SHAPE),
        (lambda: attn(out=a), INVALID_ARG), (lambda: attn(w=-1), INVALID_ARG), (lambda: attn(scale=0.0), INVALID_ARG),
        (lambda: attn(scale=NAN), INVALID_ARG), (lambda: attn(scale=-1.0), INVALID_ARG),
        (lambda: attn(kv=B.eagle_kv(a, 0, 64, i)), INVALID_ARG), (lambda: attn(ws=0), INVALID_ARG),
        (lambda: reserve(n=0), CAPACITY), (lambda: reserve(n=65), CAPACITY), (lambda: reserve(bs=12), INVALID_ARG),
        (lambda: reserve(bs=0), INVALID_ARG), (lambda: reserve(per=0), INVALID_ARG), (lambda: reserve(nb=0), INVALID_ARG),
        (lambda: reserve(per=4096), CAPACITY), (lambda: reserve(t=0), INVALID_ARG), (lambda: reserve(s=a + 4), ALIGN),
        (lambda: reserve(n_new=0), INVALID_ARG), (lambda: reserve(pools=many), CAPACITY),
        (lambda: reserve(pools=odd), ALIGN),
        (lambda: B.eagle_pages_fork(eng.ctx, pages(), 0, a, a, ws, st), INVALID_ARG),
        (lambda: B.eagle_pages_fork(eng.ctx, pages(), 3, a, a, ws, st), CAPACITY),
        (lambda: B.eagle_pages_fork(eng.ctx, pages(), 1, 0, a, ws, st), INVALID_ARG),
        (lambda: B.eagle_pages_release(eng.ctx, pages(), 0, ws, st), INVALID_ARG),
        (lambda: B.eagle_pages_init(eng.ctx, pages(r=0), ws, st), INVALID_ARG),
        (lambda: B.eagle_pages_compact(eng.ctx, pages(), odd, ws, st), ALIGN),
    ]
    for n, (call, code) in enumerate(cases):
        with pytest.raises(B.EagleError) as e:
            call()
        assert e.value.code == code, n
    assert B.eagle_launch_count(eng.ctx) == before
    c = R.PagedCache(eng, 1, 16, 4, 4)
    with pytest.raises(ValueError):
        c.append(0, i32([0, 1]), None, None, torch.zeros(1, 2, 128, device="cuda"),
                 torch.zeros(1, 2, 128, device="cuda", dtype=torch.bfloat16))
    with pytest.raises(ValueError):
        c.attend(0, i32([0, 1]), torch.zeros(1, 8, 128, device="cuda"), torch.zeros(1, 8, 128, device="cuda"))


# ---- pages --------------------------------------------------------------------------

class Twin:
    """A PagedCache and the oracle's pages, compared after every call."""

    def __init__(self, n_seqs, per, bs, n_blocks, layers=2, hkv=4, dh=16, eng=None):
        self.c = R.PagedCache(eng or engine(4, hkv, dh), n_seqs, bs, n_blocks, per, layers)
        self.o = Pages(n_seqs, per, bs, n_blocks)
        self.c.table.fill_(5)
        self.c.len.fill_(3)
        self.c.ref.fill_(7)
        self.c.clear()
        self.pools = []
        for t in self.c.k + self.c.v:
            t.copy_(torch.randn(t.shape, device="cuda"))
            self.pools.append(t.clone())
        self.check()

    def check(self, status=0):
        torch.cuda.synchronize()
        assert self.c.eng.status() == status
        assert self.c.table.tolist() == self.o.table
        assert self.c.ref.tolist() == self.o.ref
        assert self.c.len.tolist() == self.o.len
        for t, w in zip(self.c.k + self.c.v, self.pools):
            assert torch.equal(t, w)

    def reserve(self, n_new):
        self.c.reserve(i32(n_new))
        try:
            for a, z, rows in self.o.reserve(n_new):
                for w in self.pools:
                    w[z, :rows] = w[a, :rows]
            self.check()
            return True
        except OutOfBlocks:
            self.check(CAPACITY)
            return False

    def grow(self, n_new):
        """The rows reserved are appended (their contents are not these tests' concern)."""
        if self.reserve(n_new):
            self.o.len = [a + max(n, 0) for a, n in zip(self.o.len, n_new)]
            self.c.len.copy_(i32(self.o.len))

    def fork(self, src, dst):
        self.c.fork(i32(src), i32(dst))
        self.check(INVALID_ARG if self.o.fork(src, dst) else 0)

    def release(self, keep):
        self.c.release(i32(keep))
        self.o.release(keep)
        self.check()

    def compact(self):
        self.c.compact()
        for a, z in self.o.compact():
            for w in self.pools:
                w[z] = w[a]
        self.check()


@pytest.mark.parametrize("bs,per,n_blocks", [(1, 40, 150), (4, 12, 60), (16, 4, 21), (256, 2, 9)])
def test_pages_random_calls(bs, per, n_blocks):
    rng = random.Random(bs)
    t = Twin(6, per, bs, n_blocks)
    for _ in range(60):
        op = rng.randrange(5)
        if op <= 1:
            t.grow([rng.choice([0, -3, 1, 2, bs, 2 * bs + 1]) for _ in range(6)])
        elif op == 2:
            n = rng.randint(1, 3)
            t.fork([rng.randint(-1, 6) for _ in range(n)], [rng.randint(-1, 6) for _ in range(n)])
        elif op == 3:
            t.release([rng.choice([-1, -1, 0, rng.randint(0, per * bs)]) for _ in range(6)])
        else:
            t.compact()


def test_pages_many_sequences_and_blocks():
    """More sequences than a warp, more blocks than one pass of the plan, odd counts, long runs of new blocks."""
    t = Twin(64, 80, 2, 4999, layers=1, dh=16)
    rng = random.Random(1)
    t.grow([rng.choice([1, 5, 16, 17, 18, 40, 101, 150]) for _ in range(64)])
    t.release([rng.choice([-1, 0, 7]) for _ in range(64)])
    src = [s for s in range(32) if t.o.len[s]]
    t.fork(src, list(range(32, 32 + len(src))))
    t.grow([rng.choice([1, 3, 0]) for _ in range(64)])
    t.release([0] * 32 + [-1] * 32)
    t.compact()
    t.compact()                                            # nothing left to move
    t.release([0] * 64)
    t.compact()
    t.grow([0] * 64)


def test_pages_reserved_ahead_stay():
    t = Twin(2, 8, 4, 12)
    t.reserve([9, 0])                                      # three blocks, no rows yet
    t.reserve([9, 2])                                      # the same three
    t.grow([2, 2])
    t.grow([12, 1])
    t.release([20, 2 ** 31 - 1])                           # no rows beyond: blocks kept, lengths unchanged
    assert not t.reserve([2 ** 31 - 1, 0])                 # past the table's columns
    assert not t.reserve([18, 29])                         # within the columns, out of blocks


def test_pages_block_zero_takes_a_copy():
    """A shared tail copied into block 0 beside sequences that end on a block's end and copy nothing."""
    t = Twin(9, 4, 4, 24)
    t.grow([3, 8, 5, 0, 0, 0, 0, 0, 0])
    t.release([0, -1, -1, -1, -1, -1, -1, -1, -1])
    assert t.o.ref[0] == 0
    t.fork([1, 2, 2, 1, 2], [3, 4, 5, 6, 7])
    assert t.reserve([0, 0, 0, 2, 2, 2, 2, 2, 0])
    assert t.o.table[4][1] == 0 or t.o.table[3][2] == 0
    t.compact()


def test_pages_tables_alone_and_large_copies():
    """No pools: tables only.  And blocks of many copy chunks, copied part by part."""
    t = Twin(3, 4, 8, 12)
    t.c.pools_c = B.eagle_pools()
    t.grow([5, 0, 0])
    t.fork([0, 0], [1, 2])
    t.c.reserve(i32([1, 1, 1]))
    t.o.reserve([1, 1, 1])
    t.check()                                              # pools as they were
    big = Twin(4, 2, 256, 8, layers=3, hkv=8, dh=128, eng=engine(8, 8, 128))
    big.grow([133, 0, 255, 0])
    big.fork([0, 2], [1, 3])
    big.grow([0, 4, 1, 1])
    big.release([0, -1, 0, -1])
    big.compact()


# ---- a serving step ------------------------------------------------------------------

class Model:
    """Random q, k, v rows of a two-layer target, and the oracle's caches of every sequence."""

    def __init__(self, eng, n_seqs, per, bs, n_blocks, seed):
        self.eng, self.c = eng, R.PagedCache(eng, n_seqs, bs, n_blocks, per, 2)
        self.hq, self.hkv, self.dh = eng.dims["n_q_heads"], eng.dims["n_kv_heads"], eng.dims["head_dim"]
        self.rope, self.freq, self.m = rope_and_freq(self.dh, self.dh, False, "bands", 5e5)
        for t in self.c.k + self.c.v:
            t.fill_(NAN)
        self.c.clear()
        self.n_seqs = n_seqs
        self.g = torch.Generator(device="cuda").manual_seed(seed)
        self.hist = [[[np.zeros((0, self.hkv, self.dh))] * 2 for _ in range(2)] for _ in range(n_seqs)]

    def buffers(self, n_rows):
        x = torch.zeros(2, n_rows, self.hq + 2 * self.hkv, self.dh, dtype=torch.bfloat16, device="cuda")
        out = torch.zeros(2, n_rows, self.hq, self.dh, dtype=torch.bfloat16, device="cuda")
        return x, out

    def step(self, x, out, rs, n_new, q_out):
        """The calls of one step (captured or not)."""
        self.c.reserve(n_new)
        for l in range(2):
            q, k, v = x[l, :, :self.hq], x[l, :, self.hq:self.hq + self.hkv], x[l, :, self.hq + self.hkv:]
            self.c.append(l, rs, self.rope, q, k, v, q_out[l])
            self.c.attend(l, rs, q_out[l], out[l])
        self.c.advance()

    def check(self, x, out, q_out, new):
        torch.cuda.synchronize()
        assert self.eng.status() == 0
        r = 0
        for s, n in enumerate(new):
            for l in range(2):
                L = self.hist[s][l][0].shape[0]
                k = f64(x[l, r:r + n, self.hq:self.hq + self.hkv])
                v = f64(x[l, r:r + n, self.hq + self.hkv:])
                pos = np.arange(L, L + n)
                check_rotated(f64(q_out[l, r:r + n]), f64(x[l, r:r + n, :self.hq]), pos, self.freq, False, self.m, U)
                # the cache's own rounded keys go on as the history (each was checked when it was written)
                mine = self.c.table[s].long()[torch.arange(L, L + n, device="cuda") // self.c.bs] * self.c.bs \
                    + torch.arange(L, L + n, device="cuda") % self.c.bs
                kc = f64(self.c.k[l].view(-1, self.hkv, self.dh)[mine])
                check_rotated(kc, k, pos, self.freq, False, self.m, U)
                self.hist[s][l] = [np.concatenate([self.hist[s][l][0], kc]), np.concatenate([self.hist[s][l][1], v])]
                if n:
                    check_attention(f64(out[l, r:r + n]), f64(q_out[l, r:r + n]), *self.hist[s][l],
                                    1 / math.sqrt(self.dh), 0)
            r += n
        assert self.c.len.tolist() == [h[0][0].shape[0] for h in self.hist]

    def fill(self, x):
        x.copy_(torch.randn(x.shape, generator=self.g, device="cuda"))


@pytest.mark.parametrize("heads,bs", [((8, 2, 128), 16), ((4, 2, 64), 8)])
def test_serving_steps(heads, bs):
    """Prompts in chunks, single tokens, forks that diverge, drops and a compaction, each step against the oracle."""
    m = Model(engine(*heads), 5, 400 // bs, bs, 2000 // bs, seed=1)

    def step(new):
        x, out = m.buffers(sum(new) + 2)
        q_out = torch.zeros_like(out)
        m.fill(x)
        m.step(x, out, i32(starts(new)), i32(new), q_out)
        m.check(x, out, q_out, new)

    step([100, 37, 0, 0, 0])                       # a whole prompt and a first chunk
    step([1, 150, 0, 0, 0])                        # a token beside the second chunk
    m.c.fork(i32([0, 1]), i32([2, 3]))
    m.hist[2], m.hist[3] = [list(h) for h in m.hist[0]], [list(h) for h in m.hist[1]]
    step([1, 1, 1, 5, 3])                          # shared tails become private
    step([1, 1, 1, 1, 1])
    m.c.release(i32([-1, 0, 90, -1, 0]))
    m.hist[1] = [[np.zeros((0, m.hkv, m.dh))] * 2 for _ in range(2)]
    m.hist[4] = [[np.zeros((0, m.hkv, m.dh))] * 2 for _ in range(2)]
    m.hist[2] = [[t[:90] for t in h] for h in m.hist[2]]
    m.c.compact()
    live = int((m.c.ref > 0).sum())
    assert int(m.c.table.max()) == live - 1
    step([2, 60, 1, 1, 0])


def test_advance_without_rows_changes_nothing():
    """A step in which nobody has rows, behind calls that changed the lengths: they stay as those calls left them."""
    m = Model(engine(8, 2, 128), 4, 8, 16, 30, seed=5)

    def rows(new):
        x, out = m.buffers(max(sum(new), 1))
        q_out = torch.zeros_like(out)
        m.fill(x)
        m.step(x, out, i32(starts(new)), i32(new), q_out)
        m.check(x, out, q_out, new)

    def idle():
        m.c.reserve(i32([0] * 4))
        m.c.advance()
        torch.cuda.synchronize()
        assert m.eng.status() == 0 and m.c.len.tolist() == [h[0][0].shape[0] for h in m.hist]

    rows([20, 40, 0, 0])
    idle()
    m.c.fork(i32([1]), i32([2]))
    m.hist[2] = [list(h) for h in m.hist[1]]
    idle()
    m.c.release(i32([0, 17, -1, -1]))
    m.hist[0] = [[np.zeros((0, m.hkv, m.dh))] * 2 for _ in range(2)]
    m.hist[1] = [[t[:17] for t in h] for h in m.hist[1]]
    idle()
    rows([3, 1, 0, 5])
    m.c.clear()
    m.hist = [[[np.zeros((0, m.hkv, m.dh))] * 2 for _ in range(2)] for _ in range(4)]
    idle()
    assert int(m.c.ref.sum()) == 0
    rows([2, 0, 1, 0])


def test_serving_step_captured():
    """One captured step, replayed on other rows, lengths and tables."""
    m = Model(engine(8, 2, 128, fresh=True), 4, 32, 16, 90, seed=2)
    x, out = m.buffers(70)
    q_out = torch.zeros_like(out)
    rs, n_new = i32([0] * 5), i32([0] * 4)

    def load(new):
        m.fill(x)
        rs.copy_(i32(starts(new)))
        n_new.copy_(i32(new))

    load([5, 0, 1, 0])
    m.step(x, out, rs, n_new, q_out)
    m.check(x, out, q_out, [5, 0, 1, 0])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        m.step(x, out, rs, n_new, q_out)
    for new in ([1, 60, 1, 1], [1, 1, 1, 1], [0, 0, 0, 0], [33, 1, 30, 6]):
        load(new)
        g.replay()
        m.check(x, out, q_out, new)
    m.eng.close()


@pytest.mark.parametrize("captured", [False, True], ids=["eager", "captured"])
@pytest.mark.parametrize("forks", ["one writes", "both write", "all write"])
def test_a_reserve_that_fails_costs_no_rows(captured, forks):
    """Too few blocks for a step whose calls go on without a look at the status: sequences that share the block they
    would write, or lack one, keep their rows and lengths, the others' rows are appended; with room it all works."""
    heads, bs = (4, 2, 64), 16
    m = Model(engine(*heads, fresh=True), 5, 8, bs, 7, seed=9)
    x, out = m.buffers(80)
    q_out = torch.zeros_like(out)
    rs, n_new = i32([0] * 6), i32([0] * 5)
    graph = None

    def step(new):
        nonlocal graph
        m.fill(x)
        rs.copy_(i32(starts(new)))
        n_new.copy_(i32(new))
        if graph is not None:
            graph.replay()
        else:
            m.step(x, out, rs, n_new, q_out)
        torch.cuda.synchronize()

    step([40, 0, 0, 5, 14])                                # 3, 1 and 1 blocks of 7
    m.check(x, out, q_out, [40, 0, 0, 5, 14])
    m.c.fork(i32([0, 0]), i32([1, 2]))
    m.c.release(i32([-1, 33, 40 if forks == "all write" else 0, -1, -1]))     # a shorter row of the shared tail; a third
    m.hist[1] = [[t[:33] for t in h] for h in m.hist[0]]
    if forks == "all write":
        m.hist[2] = [list(h) for h in m.hist[0]]
    if captured:
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            m.step(x, out, rs, n_new, q_out)
    # two blocks are free: one for a copy, one for sequence 4's third row; sequence 3 wants 100 rows
    new = {"one writes": [0, 1, 0, 27, 3], "both write": [2, 3, 0, 27, 3], "all write": [1, 1, 1, 27, 3]}[forks]
    lens = m.c.len.tolist()
    table, ref = m.c.table.clone(), m.c.ref.clone()
    kept = [[t.view(-1, 2, 64)[rows_at(m.c, s, 0, lens[s])].clone() for t in m.c.k + m.c.v] for s in range(5)]
    new[4] = 40                                            # ... and this one two more blocks: in all more than there are
    step(new)
    assert m.eng.status() == CAPACITY
    assert torch.equal(m.c.table, table) and torch.equal(m.c.ref, ref)
    assert m.c.len.tolist() == lens                        # every one of them shares its block or lacks one
    new[3], new[4] = 3, 40                                 # one that needs nothing: its rows go in
    step(new)
    assert m.eng.status() == CAPACITY
    lens[3] += 3
    assert m.c.len.tolist() == lens
    lo = sum(new[:3])
    for l in range(2):
        k, v = (x[l, lo:lo + 3, 4 + 2 * i:6 + 2 * i] for i in (0, 1))
        at = rows_at(m.c, 3, lens[3] - 3, lens[3])
        check_rotated(f64(m.c.k[l].view(-1, 2, 64)[at]), f64(k), np.arange(lens[3] - 3, lens[3]), m.freq, False, m.m, U)
        assert torch.equal(m.c.v[l].view(-1, 2, 64)[at], v)
        m.hist[3][l] = [np.concatenate([m.hist[3][l][0], f64(m.c.k[l].view(-1, 2, 64)[at])]),
                        np.concatenate([m.hist[3][l][1], f64(v)])]
    for s in range(5):
        for t, w in zip(m.c.k + m.c.v, kept[s]):
            assert torch.equal(t.view(-1, 2, 64)[rows_at(m.c, s, 0, w.shape[0])].view(torch.int16), w.view(torch.int16))
    m.c.release(i32([-1, -1, -1, -1, 0]))                  # room again: the same rows for the forks
    m.hist[4] = [[np.zeros((0, m.hkv, m.dh))] * 2 for _ in range(2)]
    new[3], new[4] = 1, 0
    step(new)
    m.check(x, out, q_out, new)
    m.eng.close()


@pytest.mark.parametrize("heads", [(8, 2, 128), (32, 8, 128), (4, 2, 64)], ids=lambda h: "x".join(map(str, h)))
@pytest.mark.parametrize("call", ["append", "append captured", "compact", "release", "fork"])
def test_verification_directly_behind_a_cache_call(heads, call):
    """The round's verification attention as the very next launch behind a call that writes its prefix, its length or
    its table: the same as after that call has finished."""
    hq, hkv, dh = heads
    nb, S, bs, per = 6, 8, 16, 128
    eng = R.Engine(dict(d=hq * dh, n_q_heads=hq, n_kv_heads=hkv, head_dim=dh, d_ff=64, vocab=64), max_batch=nb + 1,
                   max_rows=8, max_expanded=1, max_children=1, max_tree=S, max_prefix=bs * per, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(90)
    bf = lambda *shape: torch.randn(*shape, generator=g, device="cuda").to(torch.bfloat16)
    q, kt, vt = bf(nb, S, hq, dh), bf(nb, S, hkv, dh), bf(nb, S, hkv, dh)
    anc = torch.tensor([(2 << s) - 1 for s in range(S)], device="cuda").expand(nb, S).contiguous()
    size, other = i32([S] * nb), torch.zeros(nb * S * 64, dtype=torch.int32, device="cuda")
    tree = B.eagle_tree(*[_p(other)] * 5, _p(anc), _p(other), _p(size), S)
    c = R.PagedCache(eng, nb + 1, bs, 2 * nb * per, per)
    for t in (c.k[0], c.v[0]):
        t.copy_(bf(*t.shape))
    rs, n_new = i32([500 * b for b in range(nb + 1)] + [500 * nb]), i32([500] * nb + [0])
    k, v = bf(500 * nb, hkv, dh), bf(500 * nb, hkv, dh)
    outs = [torch.zeros(nb, S, hq, dh, device="cuda") for _ in range(2)]

    def verify(out, kv):
        B.eagle_tree_verify_attn(eng.ctx, nb, _p(q), _p(kt), _p(vt), kv, tree, 1 / math.sqrt(dh), _p(out),
                                 eng.ws.data_ptr(), eng.stream())

    def cache_call():
        if call.startswith("append"):
            c.append(0, rs, None, None, k, v)
        elif call == "compact":
            c.compact()
        elif call == "release":
            B.eagle_pages_release(eng.ctx, c.pages_c, _p(keep), eng.ws.data_ptr(), eng.stream())
        else:
            B.eagle_pages_fork(eng.ctx, c.pages_c, 1, _p(src), _p(dst), eng.ws.data_ptr(), eng.stream())

    keep, src, dst = i32([700] * nb + [-1]), i32([0]), i32([1])
    kv = c._kv_next[0] if call.startswith("append") else c.kv()
    graph = None
    verify(outs[1], c.kv())
    for turn in range(6):
        # 1500 rows each, in blocks behind those of a sequence that goes; the blocks' contents differ from turn to turn
        c.clear()
        c.reserve(i32([0] * nb + [bs * per]))
        c.reserve(i32([1500] * nb + [0]))
        c.len.copy_(i32([1500 - 3 * b for b in range(nb)] + [0]))
        c.release(i32([-1] * nb + [0]))
        c.reserve(n_new)
        for t in (c.k[0], c.v[0]):
            t.copy_(t.roll(turn + 1, 0))
        k.copy_(k.roll(turn + 1, 0))
        c.len_next.copy_(c.len)
        torch.cuda.synchronize()
        if call == "append captured":
            if graph is None:
                graph = torch.cuda.CUDAGraph()
                with torch.cuda.graph(graph):
                    cache_call()
                    verify(outs[0], kv)
            graph.replay()
        else:
            cache_call()
            verify(outs[0], kv)
        torch.cuda.synchronize()
        assert eng.status() == 0
        verify(outs[1], kv)
        torch.cuda.synchronize()
        assert eng.status() == 0 and torch.isfinite(outs[1]).all()
        assert torch.equal(outs[0], outs[1])
    eng.close()


def test_drafting_directly_behind_an_append():
    """A draft step right behind rows appended to the draft's own cache."""
    import eagle_synth as S
    from eagle_feature_level_gb300.workload import dims_of, limits_for
    w = S.variant("13b_x8_eagle2", name="served", d=256, n_q_heads=4, n_kv_heads=4, head_dim=64, d_ff=344, vocab=1000,
                  batch=3, prefix_range=(50, 200), weight_std=0.05, temps=(0.0,))
    eng = R.Engine(dims_of(w), max_prefix=1024, device="cuda", **limits_for(w))
    rd = R.Round(eng, R.plan_for(w.tree, w.top_k, w.depth, w.top_m), w.batch, 1024)
    wc = eng.weights(S.draft_weights(w, 79, device="cuda"))
    g = torch.Generator(device="cuda").manual_seed(91)
    n, lens = 300, [40, 120, 77]
    rd.t_next.copy_(i32([5, 9, 700]))
    rd.f_last.copy_(torch.randn(rd.f_last.shape, generator=g, device="cuda"))
    ln, rs = i32([0] * 3), i32([0, n, 2 * n, 3 * n])
    st, ws = eng.stream(), eng.ws.data_ptr()
    for turn in range(6):
        rd.draft_len.copy_(i32(lens))
        rd.pos0.copy_(i32([a + n for a in lens]))
        ln.copy_(i32(lens))
        for t in (rd.draft_k, rd.draft_v):
            t.copy_(torch.randn(t.shape, generator=g, device="cuda"))
        k, v = (torch.randn(3 * n, 4, 64, generator=g, device="cuda") for _ in range(2))
        B.eagle_tree_expand_rerank(eng.ctx, rd.plan, B.PHASE_ROOT, 0, 3, rd.req_c, None, rd.pool_c, None, ws, st)
        kv = B.eagle_kv(_p(rd.draft_k), _p(rd.draft_v), 1024, _p(ln))
        torch.cuda.synchronize()
        B.eagle_kv_append(eng.ctx, 3, B.eagle_rows(_p(rs), 3 * n), None, B.DTYPE_F32, 0, 0, 0, 0, _p(k), k.stride(0),
                          _p(v), v.stride(0), rd.draft_kv_c, None, _p(ln), ws, st)
        logits = []
        for _ in range(2):
            B.eagle_draft_step(eng.ctx, rd.plan, 0, 3, wc, rd.req_c, kv, rd.pool_c, rd.out_c, rd.children_c,
                               rd.sampling_c, ws, st)
            torch.cuda.synchronize()
            assert eng.status() == 0
            logits.append(rd.logits[:, 0].clone())
        assert ln.tolist() == [a + n for a in lens]
        assert torch.isfinite(logits[1]).all() and torch.equal(logits[0], logits[1])
    eng.close()


def rows_at(c, s, lo, hi):
    """Flat pool rows of positions lo .. hi - 1 of sequence s of a PagedCache."""
    j = torch.arange(lo, hi, device="cuda")
    return c.table[s].long()[j // c.bs] * c.bs + j % c.bs


def test_append_looks_at_counts_where_given():
    """The counts are the caller's to give: without them a shared block is written as it always was."""
    hq, hkv, dh = 4, 2, 64
    eng = engine(hq, hkv, dh)
    c = Cache([6, 3, 0], [12, 12, 12], hkv, dh, 4, seed=80)
    ref = torch.zeros(c.k.shape[0], dtype=torch.int32, device="cuda")
    ref[c.table.flatten().long()] = 1
    k, v = (torch.randn(9, hkv, dh, device="cuda").to(torch.bfloat16) for _ in range(2))
    before = c.k.clone()
    for shared, want in (((2, 0), [9, 6, 0]), ((0, 1), [6, 6, 3]), ((0, 0), [9, 6, 3])):
        c.k.copy_(before)
        counts = ref.clone()
        counts[c.table[shared].long()] = 2                                      # of a sequence, in its column
        paging = B.eagle_paging(_p(c.table), 4, c.k.shape[0], _p(counts))
        ln = run_append(eng, c, i32([0, 3, 6, 9]), 9, None, None, k, v, None,
                        kv=B.eagle_kv(_p(c.k), _p(c.v), c.cap, _p(c.len), paging))
        torch.cuda.synchronize()
        assert eng.status() == (0 if want == [9, 6, 3] else CAPACITY) and ln.tolist() == want
        for b, (n, lo) in enumerate(zip(c.lens, (0, 3, 6))):
            at = c.at(b, n, n + 3)
            expect = k[lo:lo + 3] if want[b] > n else before.view(-1, hkv, dh)[at]
            assert torch.equal(c.k.view(-1, hkv, dh)[at].view(torch.int16), expect.contiguous().view(torch.int16))
    ln = run_append(eng, c, i32([0, 3, 6, 9]), 9, None, None, k, v, None)
    torch.cuda.synchronize()
    assert eng.status() == 0 and ln.tolist() == [9, 6, 3]
    launches = B.eagle_launch_count(eng.ctx)
    with pytest.raises(B.EagleError) as e:
        run_append(eng, c, i32([0, 3, 6, 9]), 9, None, None, k, v, None, kv=B.eagle_kv(
            _p(c.k), _p(c.v), c.cap, _p(c.len), B.eagle_paging(_p(c.table), 4, c.k.shape[0], _p(ref) + 4)))
    assert e.value.code == ALIGN and B.eagle_launch_count(eng.ctx) == launches


def test_commit_writes_no_shared_block():
    """A commit after a fork whose reserve was left out: the forks keep their rows, the third request commits; after
    the reserve all do."""
    import eagle_synth as S
    from eagle_feature_level_gb300.workload import dims_of, limits_for, load_round, standin
    w = S.variant("13b_x8_eagle2", name="served", d=128, n_q_heads=4, n_kv_heads=2, head_dim=64, d_ff=344, vocab=1000,
                  batch=3, prefix_range=(50, 200), weight_std=0.05, temps=(0.0,))
    inp = S.round_inputs(w, 78, device="cuda")
    eng = R.Engine(dims_of(w), max_prefix=512, device="cuda", **limits_for(w))
    rd = R.Round(eng, R.plan_for(w.tree, w.top_k, w.depth, w.top_m), w.batch, inp["kv_cap"])
    load_round(rd, inp)
    rd.run(eng.weights(S.draft_weights(w, 78, device="cuda")), standin(inp))
    torch.cuda.synchronize()
    accepted = rd.accept_len.tolist()
    bs = 64
    m = Model(eng, 3, 512 // bs, bs, 8, seed=4)
    new = [70, 67, 0]                                      # any path fits the blocks they have
    assert rd.path_cap < bs - 6
    x, out = m.buffers(sum(new))
    m.fill(x)
    m.step(x, out, i32(starts(new)), i32(new), torch.zeros_like(out))
    m.c.fork(i32([1]), i32([2]))
    lens = [70, 67, 67]

    def commit():
        kept = [[t.view(-1, 2, 64)[rows_at(m.c, s, 0, lens[s])].clone() for t in m.c.k + m.c.v] for s in range(3)]
        pools = [t.clone() for t in m.c.k + m.c.v]
        B.eagle_commit(eng.ctx, 3, rd.acc_c, rd.tree_c, _p(rd.f_true), [_p(rd.tree_k[0])] * 2, [_p(rd.tree_v[0])] * 2,
                       [_p(t) for t in m.c.k], [_p(t) for t in m.c.v], m.c.cap, _p(m.c.len), rd.out_c, rd.draft_kv_c,
                       rd.commit_c, eng.ws.data_ptr(), eng.stream(), target_paging=m.c.paging)
        torch.cuda.synchronize()
        for s in range(3):
            for t, w in zip(m.c.k + m.c.v, kept[s]):
                assert torch.equal(t.view(-1, 2, 64)[rows_at(m.c, s, 0, lens[s])].view(torch.int16), w.view(torch.int16))
        return pools

    def committed(s):
        path, at = rd.path[s, :accepted[s] + 1].long(), rows_at(m.c, s, lens[s], lens[s] + accepted[s] + 1)
        return all(torch.equal(t.view(-1, 2, 64)[at], tree[s][path]) for t, tree in
                   zip(m.c.k + m.c.v, [rd.tree_k[0]] * 2 + [rd.tree_v[0]] * 2))

    pools = commit()
    assert eng.status() == CAPACITY
    assert rd.prefix_len_out.tolist() == [lens[0] + 1 + accepted[0], 67, 67] and committed(0)
    shared = int(m.c.table[1, 1])
    for t, old in zip(m.c.k + m.c.v, pools):
        assert torch.equal(t[shared].view(torch.int16), old[shared].view(torch.int16))
    m.c.reserve(i32([rd.path_cap] * 3))
    torch.cuda.synchronize()
    commit()
    assert eng.status() == 0
    assert rd.prefix_len_out.tolist() == [n + 1 + a for n, a in zip(lens, accepted)]
    assert all(committed(s) for s in range(3))
    eng.close()


def test_round_on_a_served_cache():
    """The cache the calls filled is what the round's verification attention and commit take: the tree's rows attend
    to it through its table, and the accepted path lands in blocks that reserve handed out."""
    import eagle_synth as S
    from eagle_feature_level_gb300.workload import dims_of, limits_for, load_round, standin
    from oracle.verify import tree_attention
    from tests.gpu_harness import feature_tol, mask_ints
    w = S.variant("13b_x8_eagle2", name="served", d=128, n_q_heads=4, n_kv_heads=2, head_dim=64, d_ff=344, vocab=1000,
                  batch=3, prefix_range=(50, 200), weight_std=0.05, temps=(0.0,))
    inp = S.round_inputs(w, 77, device="cuda")
    eng = R.Engine(dims_of(w), max_prefix=512, device="cuda", **limits_for(w))
    rd = R.Round(eng, R.plan_for(w.tree, w.top_k, w.depth, w.top_m), w.batch, inp["kv_cap"])
    load_round(rd, inp)
    rd.draft_and_tree(eng.weights(S.draft_weights(w, 77, device="cuda")))
    lens = rd.tgt_len.tolist()
    m = Model(eng, 3, 512 // 16, 16, 100, seed=3)
    new = lens
    x, out = m.buffers(sum(new))
    q_out = torch.zeros_like(out)
    m.fill(x)
    m.step(x, out, i32(starts(new)), i32(new), q_out)
    m.check(x, out, q_out, new)
    got = torch.empty_like(rd.attn_out)
    B.eagle_tree_verify_attn(eng.ctx, 3, _p(rd.tree_q), _p(rd.tree_k[0]), _p(rd.tree_v[0]), m.c.kv(1), rd.tree_c,
                             1 / math.sqrt(64), _p(got), eng.ws.data_ptr(), eng.stream())
    torch.cuda.synchronize()
    assert eng.status() == 0
    for b in range(3):
        n = int(rd.t_size[b])
        ref = tree_attention(f64(rd.tree_q[b, :n]), f64(rd.tree_k[0][b, :n]), f64(rd.tree_v[0][b, :n]),
                             *m.hist[b][1], mask_ints(rd.t_anc[b, :n]), 1 / math.sqrt(64))
        assert np.abs(f64(got[b, :n]) - ref).max() <= feature_tol(w)
    rd.verify()
    standin(inp)(rd)
    rd.accept()
    m.c.reserve(i32([rd.path_cap] * 3))                    # room for any accepted path
    kb = [t.clone() for t in m.c.k]
    B.eagle_commit(eng.ctx, 3, rd.acc_c, rd.tree_c, _p(rd.f_true), [_p(rd.tree_k[0])] * 2, [_p(rd.tree_v[0])] * 2,
                   [_p(t) for t in m.c.k], [_p(t) for t in m.c.v], m.c.cap, _p(m.c.len), rd.out_c, rd.draft_kv_c,
                   rd.commit_c, eng.ws.data_ptr(), eng.stream(), target_paging=m.c.paging)
    torch.cuda.synchronize()
    assert eng.status() == 0
    for b in range(3):
        a = int(rd.accept_len[b])
        assert int(rd.prefix_len_out[b]) == lens[b] + 1 + a
        for l in range(2):
            flat, old = m.c.k[l].view(-1, 2, 64), kb[l].view(-1, 2, 64)
            at = lambda lo, hi: m.c.table[b].long()[torch.arange(lo, hi, device="cuda") // 16] * 16 \
                + torch.arange(lo, hi, device="cuda") % 16
            assert torch.equal(flat[at(0, lens[b])], old[at(0, lens[b])])
            path = rd.path[b, :a + 1].long()
            assert torch.equal(flat[at(lens[b], lens[b] + a + 1)], rd.tree_k[0][b][path])
    m.c.len.copy_(rd.prefix_len_out)
    m.c.release(m.c.len)                                   # what the path did not take goes back
    held = [-(-int(n) // 16) for n in m.c.len]
    torch.cuda.synchronize()
    assert int(m.c.ref.sum()) == sum(held)
    eng.close()
