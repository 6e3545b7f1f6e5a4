"""The oracle of the target's cache against independent statements of the same mathematics, and the library's
host-side rotary plan against the oracle (no GPU)."""
import math
import random

import numpy as np
import pytest

from oracle.cache import OutOfBlocks, Pages, chunk_attention, frequencies, rotate
from oracle.layer import rope

SCALED = [("none", 1.0, 0.0, 0.0, 0), ("linear", 4.0, 0.0, 0.0, 0), ("bands", 8.0, 1.0, 4.0, 8192),
          ("ramp", 16.0, 1.0, 32.0, 4096), ("ramp", 1.0, 2.0, 3.0, 1)]


def test_rotate_is_the_layers_rope_and_relative():
    rng = np.random.default_rng(1)
    x = rng.standard_normal((5, 3, 32))
    pos = [0, 1, 17, 4096, 131071]
    got = rotate(x, pos, frequencies(32, 1e4), False)
    for i, p in enumerate(pos):
        assert np.allclose(got[i], rope(x[i], p, 1e4), rtol=0, atol=1e-9)
    # interleaved is the split layout on reordered elements
    order = np.concatenate([np.arange(0, 32, 2), np.arange(1, 32, 2)])
    assert np.allclose(rotate(x, pos, frequencies(32, 1e4), True)[..., order],
                       rotate(x[..., order], pos, frequencies(32, 1e4), False), atol=1e-12)
    # scores depend on the distance alone; elements past the rotating part do not move
    f = frequencies(8, 5e5)
    q, k = rng.standard_normal((2, 1, 1, 16))
    dot = lambda a, b: float((rotate(q, [a], f, True) * rotate(k, [b], f, True)).sum())
    assert dot(9, 4) == pytest.approx(dot(1009, 1004), abs=1e-10)
    assert np.array_equal(rotate(q, [77], f, True)[..., 8:], q[..., 8:])


def test_scaled_frequencies_keep_their_ends():
    f = frequencies(128, 5e5)
    b = frequencies(128, 5e5, "bands", 8.0, 1.0, 4.0, 8192)
    turns = 8192 * f / (2 * math.pi)
    assert np.array_equal(b[turns >= 4], f[turns >= 4]) and np.allclose(b[turns <= 1], f[turns <= 1] / 8)
    assert ((b <= f) & (b >= f / 8 - 1e-18)).all() and (np.diff(b) < 0).all()
    r = frequencies(128, 1e4, "ramp", 16.0, 1.0, 32.0, 4096)
    assert r[0] == 1.0 and r[-1] == pytest.approx(1e4 ** (-126 / 128) / 16)
    assert np.allclose(frequencies(64, 1e4, "linear", 4.0), frequencies(64, 1e4) / 4)


def test_chunk_attention_is_row_by_row_attention():
    rng = np.random.default_rng(2)
    L, n, Hq, Hkv, dh = 23, 9, 4, 2, 8
    q, k, v = rng.standard_normal((n, Hq, dh)), rng.standard_normal((L, Hkv, dh)), rng.standard_normal((L, Hkv, dh))
    for w in (0, 1, 5, 100):
        out, mean_abs, reach = chunk_attention(q, k, v, 0.3, w)
        for i in range(n):
            p = L - n + i
            lo = max(0, p - w + 1) if w else 0
            for h in range(Hq):
                s = 0.3 * k[lo:p + 1, h // 2] @ q[i, h]
                e = np.exp(s - s.max())
                assert np.allclose(out[i, h], e @ v[lo:p + 1, h // 2] / e.sum(), atol=1e-12)
        assert (np.abs(out) <= mean_abs + 1e-12).all() and (reach > 0).all()
    assert not chunk_attention(q, k[:4], v[:4], 0.3)[0][:5].any()      # rows before the first key


def test_pages_keep_every_sequences_rows():
    """Random calls: each sequence reads back exactly what it appended, counts equal the table entries, and two
    sequences never write one row."""
    rng = random.Random(3)
    for bs in (1, 4, 16):
        P = Pages(6, 40 // bs + 2, bs, 7 * (40 // bs + 2))
        store = {}                                     # (block, row) -> value
        want = [[] for _ in range(6)]
        stamp = 0
        for _ in range(400):
            op = rng.randrange(4)
            if op == 0:
                src = rng.sample(range(6), 2)
                dst = rng.sample([s for s in range(6) if s not in src], 2)
                assert P.fork(src, dst) == []
                for s, d in zip(src, dst):
                    want[d] = list(want[s])
            elif op == 1:
                n = [rng.choice([0, 0, 1, 3, bs]) for _ in range(6)]
                before = [list(r) for r in P.table], list(P.ref)
                try:
                    copies = P.reserve(n)
                except OutOfBlocks:
                    assert before == ([list(r) for r in P.table], list(P.ref))
                    continue
                for a, z, rows in copies:
                    for r in range(rows):
                        store[z, r] = store[a, r]
                for s in range(6):
                    for i in range(n[s]):
                        p = P.len[s] + i
                        blk = P.table[s][p // bs]
                        assert P.ref[blk] == 1         # a row is written in a block of one's own
                        store[blk, p % bs] = stamp
                        want[s].append(stamp)
                        stamp += 1
                    P.len[s] += n[s]
            elif op == 2:
                keep = [rng.choice([-1, -1, rng.randint(0, 40)]) for _ in range(6)]
                P.release(keep)
                want = [w if k < 0 else w[:k] for w, k in zip(want, keep)]
            else:
                moved = P.compact()
                held = {z: {r: store[a, r] for r in range(bs) if (a, r) in store} for a, z in moved}
                for z, rows in held.items():
                    store.update({(z, r): x for r, x in rows.items()})
                live = sum(r > 0 for r in P.ref)
                assert all(P.ref[b] > 0 for b in range(live)) and not any(P.ref[live:])
            for s in range(6):
                assert [store[P.table[s][p // bs], p % bs] for p in range(P.len[s])] == want[s]
            flat = [b for row in P.table for b in row if b >= 0]
            assert [flat.count(b) for b in range(P.n_blocks)] == P.ref


def test_pages_last_holder_keeps_its_block():
    P = Pages(3, 4, 8, 8)
    P.reserve([5, 0, 0])
    P.len[0] = 5
    P.fork([0, 0], [1, 2])
    assert P.reserve([1, 1, 1]) == [(0, 1, 5), (0, 2, 5)] and P.ref[:3] == [1, 1, 1]
    assert [row[0] for row in P.table] == [1, 2, 0]
    assert P.fork([0, 0, 1, 9], [1, 1, 2, 2]) == [0, 1, 3]   # 1 is a source, 9 no sequence
    P.release([0, 0, 0])
    assert not any(P.ref)


@pytest.fixture(scope="module")
def binding():
    from eagle_feature_level_gb300.build import build
    build()
    from eagle_feature_level_gb300 import _binding
    return _binding


@pytest.mark.parametrize("kind,factor,low,high,orig", SCALED)
@pytest.mark.parametrize("dh,rot", [(128, 128), (64, 32), (16, 2), (128, 70)])
def test_rope_plan_holds_the_frequencies(binding, dh, rot, kind, factor, low, high, orig):
    code = {"linear": binding.ROPE_LINEAR, "bands": binding.ROPE_BANDS, "ramp": binding.ROPE_RAMP}
    for theta in (1e4, 5e5):
        sc = None if kind == "none" else binding.eagle_rope_scaling(code[kind], factor, low, high, orig, 0.0)
        r = binding.eagle_rope_plan(dh, rot, 1, theta, sc)
        f = frequencies(rot, theta, kind, factor, low, high, orig)
        got = np.array([r.turn[j] / 2.0 ** 64 * 2 * math.pi for j in range(rot // 2)])
        # pow and the few products of each side: some 2^-50 relative, and 2^-64 of a turn
        assert (np.abs(got - f) <= 2.0 ** -48 * f + 2.0 ** -60).all()
        assert (r.rot_dim, r.interleaved) == (rot, 1) and all(r.turn[j] == 0 for j in range(rot // 2, 64))
        want = 1.0 + 0.1 * math.log(factor) if kind == "ramp" else 1.0
        assert r.mscale == pytest.approx(want, rel=2.0 ** -23)
    if kind != "none":
        sc = binding.eagle_rope_scaling(code[kind], factor, low, high, orig, 0.75)
        assert binding.eagle_rope_plan(dh, rot, 0, 1e4, sc).mscale == 0.75


def test_rope_plan_refuses(binding):
    B = binding
    S = B.eagle_rope_scaling
    for args, name in (((129, 2, 0, 1e4), "EAGLE_ERR_SHAPE"), ((64, 0, 0, 1e4), "EAGLE_ERR_SHAPE"),
                       ((64, 66, 0, 1e4), "EAGLE_ERR_SHAPE"), ((64, 7, 0, 1e4), "EAGLE_ERR_SHAPE"),
                       ((64, 64, 0, 1.0), "EAGLE_ERR_INVALID_ARG"), ((64, 64, 0, math.inf), "EAGLE_ERR_INVALID_ARG"),
                       ((64, 64, 0, 1e4, S(0, 2.0, 1, 4, 8, 0)), "EAGLE_ERR_INVALID_ARG"),
                       ((64, 64, 0, 1e4, S(1, 0.5, 0, 0, 0, 0)), "EAGLE_ERR_INVALID_ARG"),
                       ((64, 64, 0, 1e4, S(1, math.nan, 0, 0, 0, 0)), "EAGLE_ERR_INVALID_ARG"),
                       ((64, 64, 0, 1e4, S(1, 2.0, 0, 0, 0, -1.0)), "EAGLE_ERR_INVALID_ARG"),
                       ((64, 64, 0, 1e4, S(2, 2.0, 4, 4, 8, 0)), "EAGLE_ERR_INVALID_ARG"),
                       ((64, 64, 0, 1e4, S(2, 2.0, 1, 4, 0, 0)), "EAGLE_ERR_INVALID_ARG"),
                       ((64, 64, 0, 1e4, S(3, 2.0, 0, 4, 8, 0)), "EAGLE_ERR_INVALID_ARG")):
        with pytest.raises(B.EagleError) as e:
            B.eagle_rope_plan(*args)
        assert e.value.name == name, args


def test_calls_refuse_a_missing_context(binding):
    """Everything else these calls check sits behind a context, which needs the GPU."""
    B = binding
    rows, kv, pages = B.eagle_rows(256, 1), B.eagle_kv(256, 256, 8, 256), B.eagle_pages(256, 256, 256, 256, 1, 1, 1, 1)
    for call in (lambda: B.eagle_kv_append(None, 1, rows, None, 0, 0, 0, 0, 0, 256, 8, 256, 8, kv, None, 512, 256, 0),
                 lambda: B.eagle_chunk_attn(None, 1, rows, 256, 8, kv, 0, 1.0, 512, 8, 256, 0),
                 lambda: B.eagle_pages_init(None, pages, 256, 0),
                 lambda: B.eagle_pages_fork(None, pages, 1, 256, 256, 256, 0),
                 lambda: B.eagle_pages_reserve(None, pages, B.eagle_pools(), 256, 256, 0),
                 lambda: B.eagle_pages_release(None, pages, 256, 256, 0),
                 lambda: B.eagle_pages_compact(None, pages, B.eagle_pools(), 256, 0)):
        with pytest.raises(B.EagleError) as e:
            call()
        assert e.value.name == "EAGLE_ERR_INVALID_ARG"


def test_paged_cache_checks_its_tensors(monkeypatch):
    """What PagedCache refuses before it calls the library: types, counts, shapes, strides, devices."""
    import torch
    from eagle_feature_level_gb300 import _binding as B
    from eagle_feature_level_gb300 import runtime as R
    calls = []
    for name in ("eagle_kv_append", "eagle_chunk_attn", "eagle_pages_fork", "eagle_pages_reserve", "eagle_pages_release"):
        monkeypatch.setattr(B, name, lambda *a, name=name: calls.append(name))
    eng = R.Engine.__new__(R.Engine)
    eng.ctx, eng.device, eng.dims = None, torch.device("cpu"), dict(n_q_heads=4, n_kv_heads=2, head_dim=64)
    eng.ws, eng.stream = torch.empty(0), lambda: 0
    eng.close = lambda: None
    c = R.PagedCache(eng, 3, 16, 8, 4)
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32)
    rs, b = i32(0, 1, 1, 5), torch.bfloat16
    x = torch.zeros(5, 8, 64, dtype=b)
    q, k, v = x[:, :4], x[:, 4:6], x[:, 6:]
    out = torch.zeros(5, 4, 64, dtype=b)
    c.append(0, rs, None, q, k, v, pos=i32(0, 1, 2, 3, 4))
    c.append(0, rs, None, None, k, v)
    c.attend(0, rs, q, out)
    c.fork(i32(0, 1), i32(2, 3))
    c.reserve(i32(0, 1, 2))
    c.release(i32(-1, 1, 2))
    assert len(calls) == 6
    refused = [
        lambda: c.append(0, i32(0, 1, 5), None, q, k, v), lambda: c.append(0, rs.long(), None, q, k, v),
        lambda: c.append(0, rs.repeat(2)[::2], None, q, k, v), lambda: c.append(0, rs.to("meta"), None, q, k, v),
        lambda: c.append(0, rs, None, q[:4], k, v), lambda: c.append(0, rs, None, q, k, v[:4]),
        lambda: c.append(0, rs, None, k, k, v), lambda: c.append(0, rs, None, q, k, v, q_out=out[:3]),
        lambda: c.append(0, rs, None, q.float(), k, v), lambda: c.append(0, rs, None, q.half(), k.half(), v.half()),
        lambda: c.append(0, rs, None, None, k, v, q_out=out), lambda: c.append(0, rs, None, q, k, v, pos=i32(1, 2)),
        lambda: c.append(0, rs, None, q, k, x[:, 1::4]), lambda: c.append(0, rs, None, q, k, v.to("meta")),
        lambda: c.attend(0, rs, q, out[:4]), lambda: c.attend(0, rs, q, out.float()),
        lambda: c.attend(0, rs, q.reshape(5, 2, 128), out), lambda: c.attend(0, rs[:3], q, out),
        lambda: c.fork(i32(0, 1), i32(2)), lambda: c.fork(i32(0).long(), i32(2)), lambda: c.reserve(i32(1, 1)),
        lambda: c.reserve(torch.zeros(3)), lambda: c.release(i32(1, 1, 1, 1)),
    ]
    for i, call in enumerate(refused):
        with pytest.raises(ValueError):
            call()
            raise AssertionError(i)
    assert len(calls) == 6
