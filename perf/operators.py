"""The serving operators around a draft-and-verify round, as measured work: rotary positions with the append of new
rows to a KV cache, attention of a chunk of new rows over that cache, and the life of its pages (fork, reserve with
copy on write, release, compact).

`run` computes each in plain torch (32-bit arithmetic, 64-bit angles) or, with `own` set, through the library's calls.
A case's lengths and block placement come from the case alone (`shape` seeds them), so that `work` knows them; the
values come from the seed.  KV pools hold bf16 values; where only their bits move they are returned as int16.
"""
import math
import random

import torch

own = False

DEV = "cuda"
LAYERS_MOST = 8


# ---- cases ------------------------------------------------------------------

def _append(name, B, heads, new, ctx, bs, f32=False, rot=0, inter=False, scaling="none", theta=1e4, shape=1):
    return dict(name=name, op="append", B=B, hq=heads[0], hkv=heads[1], dh=heads[2], new_lo=new[0], new_hi=new[1],
                ctx_lo=ctx[0], ctx_hi=ctx[1], bs=bs, f32=f32, rot=rot or heads[2], inter=inter, scaling=scaling,
                theta=theta, shape=shape)


def _attend(name, B, heads, new, ctx, bs, window=0, shape=1):
    return dict(name=name, op="attend", B=B, hq=heads[0], hkv=heads[1], dh=heads[2], new_lo=new[0], new_hi=new[1],
                ctx_lo=ctx[0], ctx_hi=ctx[1], bs=bs, window=window, shape=shape)


def _branch(name, parents, children, heads, ctx, new, bs, layers, shape=1):
    return dict(name=name, op="branch", parents=parents, children=children, hkv=heads[1], dh=heads[2], hq=heads[0],
                ctx_lo=ctx[0], ctx_hi=ctx[1], new=new, bs=bs, layers=layers, shape=shape)


def _compact(name, seqs, heads, ctx, blocks, bs, layers, shape=1):
    return dict(name=name, op="compact", seqs=seqs, hkv=heads[1], dh=heads[2], hq=heads[0], ctx_lo=ctx[0],
                ctx_hi=ctx[1], blocks=blocks, bs=bs, layers=layers, shape=shape)


H7, H13, H70 = (32, 32, 128), (40, 40, 128), (64, 8, 128)    # the 7B, 13B and 70B workloads' heads
HEADS = [(4, 4, 16), (4, 2, 64), (8, 2, 128), (12, 4, 32), (16, 4, 64), (20, 4, 128), H7, H13, H70]


def listed():
    return [
        # one new token for each of 8 running requests: what a decoding step appends, latency only
        _append("append tokens", 8, H13, (1, 1), (512, 4096), 16),
        # 16 prompts' chunks in one call, frequencies scaled by wavelength for a long context: bandwidth
        _append("append chunks", 16, H70, (256, 1024), (0, 8192), 64, scaling="bands", theta=5e5),
        # fp32 rows, interleaved pairs, half of the head rotating, far positions of a long contiguous cache
        _append("append fp32 far", 4, (8, 2, 64), (1, 700), (30000, 131072), 0, f32=True, rot=32, inter=True,
                scaling="ramp"),
        # one request's next token over a short prefix: the smallest call, latency only
        _attend("attend token", 1, H7, (1, 1), (1024, 1024), 16),
        # a decoding step of 16 long requests with grouped heads: the cache is read once
        _attend("attend tokens long", 16, H70, (1, 1), (8192, 8192), 16),
        # the last 2048 tokens of a long prompt against everything before them
        _attend("attend chunk long", 1, H70, (2048, 2048), (6144, 6144), 64),
        # ragged chunks of 8 requests, multi-head, decoding and prompt requests mixed
        _attend("attend chunks ragged", 8, H13, (1, 512), (512, 4096), 16),
        # whole prompts of small heads under a sliding window, contiguous cache
        _attend("attend prompts windowed", 6, (16, 4, 64), (700, 4000), (0, 0), 0, window=1000),
        # one request forks into ten branches that each append a few tokens: latency
        _branch("branch one", 1, 10, H7, (1000, 1000), 4, 16, 1),
        # 16 requests into 15 branches each, long pages: the copy on write of the shared tails
        _branch("branch many", 16, 15, H70, (4096, 8191), 60, 256, 4),
        # a small pool after its requests came and went
        _compact("compact small", 8, H13, (512, 4096), 2600, 16, 1),
        # a large pool of several layers: the move of most live pages
        _compact("compact large", 24, H70, (512, 4096), 16384, 16, 6),
    ]


def _logu(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "attend", "branch", "compact"])
    heads = rng.choice(HEADS)
    row = heads[1] * heads[2] * 4                              # bytes of a K and a V row
    bs = rng.choice([0, 1, 2, 4, 8, 16, 32, 64, 128, 256])
    shape = rng.randrange(1 << 30)
    if op == "append":
        B = _logu(rng, 1, 64)
        hi = _logu(rng, 1, max(1, 16384 // B))
        lo = rng.randint(0, hi)
        ctx = _logu(rng, 1, max(64, min(131072, (4 << 30) // (row * B))))
        rot = rng.choice([heads[2], heads[2], heads[2] // 2, 2])
        c = _append("", B, heads, (lo, hi), (ctx // 3, ctx), bs, rng.random() < 0.3, rot, rng.random() < 0.4,
                    rng.choice(["none", "linear", "bands", "ramp"]), rng.choice([1e4, 5e5]), shape)
    elif op == "attend":
        B = _logu(rng, 1, 32)
        hi = _logu(rng, 1, 2048) if rng.random() < 0.7 else 1
        lo = rng.randint(0, hi)
        most = max(64, min(32768, int(6e8 / (B * heads[0] * hi)) - hi, (4 << 30) // (row * B)))
        ctx = _logu(rng, 1, most)
        w = _logu(rng, 1, 4096) if rng.random() < 0.3 else 0
        c = _attend("", B, heads, (lo, hi), (rng.randint(0, ctx), ctx), bs, w, shape)
    elif op == "branch":
        bs = bs or 16
        P, Ch, layers = _logu(rng, 1, 12), _logu(rng, 1, 15), rng.randint(1, 4)
        most = max(32, min(8192, (3 << 30) // (row * layers * P * (1 + Ch))))
        ctx = _logu(rng, 1, most)
        c = _branch("", P, Ch, heads, (ctx // 2, ctx), rng.randint(1, 70), bs, layers, shape)
    else:
        bs = bs or 16
        n, layers = _logu(rng, 2, 64), rng.randint(1, 4)
        most = max(32, min(8192, (1 << 30) // (row * layers * n), 48 * bs * 4096 // (64 * n) + bs))
        ctx = _logu(rng, 16, most)
        need = n * -(-ctx // bs)
        c = _compact("", n, heads, (ctx // 4, ctx), int(need * rng.uniform(1.1, 2.5)) + 2, bs, layers, shape)
    del c["name"]
    return c


# ---- what a case fixes ------------------------------------------------------

def _lens(case):
    """Rows each request has before the call, and the rows that are new."""
    r = random.Random(case["shape"] * 7 + 1)
    ctx = [r.randint(case["ctx_lo"], case["ctx_hi"]) for _ in range(case["B"])]
    new = [r.randint(case["new_lo"], case["new_hi"]) for _ in range(case["B"])]
    if case["new_lo"] < case["new_hi"] and case["B"] > 2:
        new[0], new[-1] = case["new_lo"], case["new_hi"]
    if sum(new) == 0:
        new[-1] = 1
    return ctx, new


def _page_lens(case):
    r = random.Random(case["shape"] * 7 + 2)
    n = case["parents"] if case["op"] == "branch" else case["seqs"]
    return [r.randint(case["ctx_lo"], case["ctx_hi"]) for _ in range(n)]


def _placement(case, need, n_blocks):
    """Block ids of the live pages, in the order the requests hold them."""
    return random.Random(case["shape"] * 7 + 3).sample(range(n_blocks), need)


def _ceil(a, b):
    return -(-a // b)


def _pages_of(case):
    """(lengths, blocks of each, blocks in the pool, table columns) of a page case."""
    bs, lens = case["bs"], _page_lens(case)
    held = [_ceil(n, bs) for n in lens]
    if case["op"] == "branch":
        per = _ceil(max(lens) + case["new"], bs)
        more = case["children"] * sum(_ceil(n + case["new"], bs) - n // bs for n in lens)
        return lens, held, sum(held) + more + 7, per
    return lens, held, max(case["blocks"], sum(held) + 1), max(max(held), 1)


def work(case):
    esz = 4 if case.get("f32") else 2
    if case["op"] == "append":
        ctx, new = _lens(case)
        n, q, kv = sum(new), case["hq"] * case["dh"], case["hkv"] * case["dh"]
        return {"bytes": n * (2 * q * esz + 2 * kv * (esz + 2)), "flops": 3 * n * (case["hq"] + case["hkv"]) * case["rot"]}
    if case["op"] == "attend":
        ctx, new = _lens(case)
        w, dh, pairs, rows = case["window"], case["dh"], 0, 0
        for c, n in zip(ctx, new):
            if n == 0:
                continue
            # row i of the new ones sees the keys 0 .. c + i, at most w of them
            pairs += sum(min(c + i + 1, w) for i in range(n)) if w else n * c + n * (n + 1) // 2
            rows += min(c + n, w + n - 1) if w else c + n
        return {"bytes": 2 * (2 * sum(new) * case["hq"] * dh + 2 * rows * case["hkv"] * dh), "flops": 4 * pairs * case["hq"] * dh}
    lens, held, n_blocks, per = _pages_of(case)
    row = case["hkv"] * case["dh"] * 2 * 2 * case["layers"]    # K and V of every layer
    bs = case["bs"]
    if case["op"] == "branch":
        seqs = case["parents"] * (1 + case["children"])
        copied = sum(n % bs for n in lens) * case["children"]
        return {"bytes": 2 * copied * row + 4 * (2 * seqs * per + 2 * n_blocks + 2 * seqs), "flops": 0}
    need = sum(held)
    moved = sum(1 for b in _placement(case, need, n_blocks) if b >= need)
    return {"bytes": 2 * moved * bs * row + 4 * 2 * (case["seqs"] * per + n_blocks), "flops": 0}


# ---- inputs -----------------------------------------------------------------

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _bf16(g, *shape):
    x = torch.empty(shape, dtype=torch.bfloat16, device=DEV)
    return x.normal_(generator=g)


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def _cache(case, g, lens, layers=0):
    """K and V of a cache that has room for lens[b] rows of request b (blocks beyond them not allocated)."""
    B, bs, hkv, dh = len(lens), case["bs"], case["hkv"], case["dh"]
    if bs == 0:
        cap = max(max(lens), 1)
        k, v = _bf16(g, B, cap, hkv, dh), _bf16(g, B, cap, hkv, dh)
        return dict(k=k, v=v, cap=cap, table=None, n_blocks=0)
    held = [_ceil(n, bs) for n in lens]
    per, n_blocks = max(max(held), 1), sum(held) + 3
    ids = _placement(case, sum(held), n_blocks)
    table = torch.full((B, per), -1, dtype=torch.int32)
    at = 0
    for b, h in enumerate(held):
        table[b, :h] = torch.tensor(ids[at:at + h], dtype=torch.int32)
        at += h
    k, v = _bf16(g, n_blocks, bs, hkv, dh), _bf16(g, n_blocks, bs, hkv, dh)
    return dict(k=k, v=v, cap=per * bs, table=table.to(DEV), n_blocks=n_blocks)


def prepare(case, seed):
    g = _gen(seed)
    s = dict(case=case)
    if case["op"] in ("append", "attend"):
        ctx, new = _lens(case)
        s.update(_cache(case, g, [c + n for c, n in zip(ctx, new)]))
        total = sum(new)
        s["total"], s["nmax"], s["lmax"] = total, max(new), max(c + n for c, n in zip(ctx, new))
        start = [0]
        for n in new:
            start.append(start[-1] + n)
        s["row_start"] = _i32(start)
        n_rows = total + 3                                     # a few rows behind the last request's
        s["n_rows"] = n_rows
        hq, hkv, dh = case["hq"], case["hkv"], case["dh"]
        if case["op"] == "append":
            s["len"] = _i32(ctx)
            s["len_out"] = torch.zeros_like(s["len"])
            # the rows of a fused projection: q, k and v side by side
            qkv = _bf16(g, n_rows, (hq + 2 * hkv) * dh)
            if case["f32"]:
                qkv = torch.empty(qkv.shape, device=DEV).normal_(generator=g)
            s["qkv"] = qkv
            s["q_out"] = torch.zeros(n_rows, hq, dh, dtype=qkv.dtype, device=DEV)
        else:
            s["len"] = _i32([c + n for c, n in zip(ctx, new)])
            s["q"] = _bf16(g, n_rows, hq, dh)
            s["out"] = torch.zeros(n_rows, hq, dh, dtype=torch.bfloat16, device=DEV)
        return s
    bs, layers, hkv, dh = case["bs"], case["layers"], case["hkv"], case["dh"]
    lens, held, n_blocks, per = _pages_of(case)
    s["pools"] = torch.randint(-(1 << 15), 1 << 15, (layers, 2, n_blocks, bs, hkv, dh), dtype=torch.int16, device=DEV,
                               generator=g)
    ids = _placement(case, sum(held), n_blocks)
    n_seqs = case["parents"] * (1 + case["children"]) if case["op"] == "branch" else case["seqs"]
    table = torch.full((n_seqs, per), -1, dtype=torch.int32)
    at = 0
    for b, h in enumerate(held):
        table[b, :h] = torch.tensor(ids[at:at + h], dtype=torch.int32)
        at += h
    ref = torch.zeros(n_blocks, dtype=torch.int32)
    ref[torch.tensor(ids, dtype=torch.int64)] = 1
    s["table"], s["ref"] = table.to(DEV), ref.to(DEV)
    s["len"] = _i32(lens + [0] * (n_seqs - len(lens)))
    s["scratch"] = torch.zeros(2 * n_blocks, dtype=torch.int32, device=DEV)
    s["n_seqs"], s["per"], s["n_blocks"] = n_seqs, per, n_blocks
    if case["op"] == "branch":
        P, Ch = case["parents"], case["children"]
        s["src"] = _i32([p for p in range(P) for _ in range(Ch)])
        s["dst"] = _i32([P + i for i in range(P * Ch)])
        s["n_new"] = _i32([0] * P + [case["new"]] * (P * Ch))
        s["keep"] = _i32([-1] * P + [0] * (P * Ch))
    else:
        s["table0"], s["ref0"] = s["table"].clone(), s["ref"].clone()
    return s


# ---- frequencies ------------------------------------------------------------

# factor, low, high, original length of each kind of scaling
SCALING = {"linear": (4.0, 0.0, 0.0, 0), "bands": (8.0, 1.0, 4.0, 8192), "ramp": (16.0, 1.0, 32.0, 4096)}


def _frequencies(case, dtype=torch.float64):
    """(frequency of each pair in radians a position, the factor on the rotated elements)."""
    rot, theta = case["rot"], case["theta"]
    i = torch.arange(rot // 2, dtype=dtype, device=DEV)
    f = theta ** (-2.0 * i / rot)
    if case["scaling"] == "none":
        return f, 1.0
    factor, low, high, orig = SCALING[case["scaling"]]
    if case["scaling"] == "linear":
        return f / factor, 1.0
    if case["scaling"] == "bands":
        # turns in the original length: at least `high` keep their frequency, at most `low` are slowed by the factor
        t = ((orig * f / (2 * math.pi) - low) / (high - low)).clamp(0.0, 1.0)
        return f * t + f / factor * (1 - t), 1.0
    at = lambda turns: rot * math.log(orig / (2 * math.pi * turns)) / (2 * math.log(theta))
    lo, hi = max(math.floor(at(high)), 0), min(math.ceil(at(low)), rot - 1)
    t = ((i - lo) / max(hi - lo, 1e-3)).clamp(0.0, 1.0)
    return f / factor * t + f * (1 - t), 0.1 * math.log(factor) + 1.0


# ---- plain forms ------------------------------------------------------------

def _request_of(s):
    """(request, index in it, position before it) of each new row."""
    r = torch.arange(s["total"], device=DEV)
    start = s["row_start"].long()
    b = torch.searchsorted(start[1:], r, right=True)
    return b, r - start[b]


def _cache_rows(s, b, pos):
    """Rows of the flat cache that hold positions `pos` of requests `b`."""
    if s["table"] is None:
        return b * s["cap"] + pos
    bs = s["case"]["bs"]
    return s["table"][b, pos // bs].long() * bs + pos % bs


def _plain_append(s):
    c = s["case"]
    hq, hkv, dh, rot, half, n = c["hq"], c["hkv"], c["dh"], c["rot"], c["rot"] // 2, s["total"]
    b, i = _request_of(s)
    pos = s["len"].long()[b] + i
    f, m = _frequencies(c)
    a = pos.double()[:, None] * f
    cos, sin = (a.cos() * m).float()[:, None], (a.sin() * m).float()[:, None]
    x = s["qkv"][:n].float().view(n, hq + 2 * hkv, dh)
    qk, v = x[:, :hq + hkv], x[:, hq + hkv:]
    x1, x2 = (qk[..., 0:rot:2], qk[..., 1:rot:2]) if c["inter"] else (qk[..., :half], qk[..., half:rot])
    y1, y2 = x1 * cos - x2 * sin, x2 * cos + x1 * sin
    y = torch.stack((y1, y2), -1).flatten(-2) if c["inter"] else torch.cat((y1, y2), -1)
    y = torch.cat((y, qk[..., rot:]), -1)
    s["q_out"][:n] = y[:, :hq].to(s["q_out"].dtype)
    at = _cache_rows(s, b, pos)
    s["k"].view(-1, hkv, dh)[at] = y[:, hq:].to(torch.bfloat16)
    s["v"].view(-1, hkv, dh)[at] = v.to(torch.bfloat16)
    s["len_out"].copy_(s["len"] + s["row_start"][1:] - s["row_start"][:-1])


def _plain_attend(s):
    c = s["case"]
    B, hq, hkv, dh, nmax, lmax, w = c["B"], c["hq"], c["hkv"], c["dh"], s["nmax"], s["lmax"], c["window"]
    G = hq // hkv
    start, lens = s["row_start"].long(), s["len"].long()
    n = start[1:] - start[:-1]
    i, j = torch.arange(nmax, device=DEV), torch.arange(lmax, device=DEV)
    q = s["q"][(start[:-1, None] + i).clamp(max=s["n_rows"] - 1)].float()         # [B, nmax, hq, dh]
    q = q.view(B, nmax, hkv, G, dh).permute(0, 2, 3, 1, 4).reshape(B, hkv, G * nmax, dh)
    there = j < lens[:, None]                                                     # [B, lmax]
    rows = torch.where(there, _cache_rows(s, torch.arange(B, device=DEV)[:, None], j.expand(B, -1)), 0)
    k = s["k"].view(-1, hkv, dh)[rows].float().permute(0, 2, 3, 1)
    v = torch.where(there[..., None, None], s["v"].view(-1, hkv, dh)[rows].float(), 0.0).transpose(1, 2)
    at = (lens - n)[:, None] + i                                                  # position of each new row
    sees = (j <= at[..., None]) & there[:, None]
    if w:
        sees &= j > at[..., None] - w
    x = (q @ k).view(B, hkv, G, nmax, lmax).mul_(1.0 / math.sqrt(dh)).masked_fill_(~sees[:, None, None], -math.inf)
    m = x.amax(-1, keepdim=True)
    x = x.sub_(torch.where(m == -math.inf, 0.0, m)).exp_()
    z = x.sum(-1, keepdim=True)
    o = (x.view(B, hkv, G * nmax, lmax) @ v).view(B, hkv, G, nmax, dh) / torch.where(z == 0, 1.0, z)
    b, r = _request_of(s)
    s["out"][:s["total"]] = o.permute(0, 3, 1, 2, 4)[b, r].reshape(-1, hq, dh).to(torch.bfloat16)


def _plain_branch(s):
    c = s["case"]
    bs, per, n_seqs = c["bs"], s["per"], s["n_seqs"]
    table, ref, lens = s["table"], s["ref"], s["len"]
    src, dst = s["src"].long(), s["dst"].long()
    col = torch.arange(per, device=DEV)
    # fork: the destinations hold their sources' blocks too
    held = _ceil_t(lens, bs)
    rows = torch.where(col < held[src, None], table[src], -1)
    table[dst] = rows
    ref.index_add_(0, rows.flatten().clamp(min=0).long(), (rows.flatten() >= 0).int())
    lens[dst] = lens[src]
    # reserve: blocks for the new rows; a shared tail block that would be written becomes the writer's own, the last
    # of its holders keeping it when all of them write
    new, held = s["n_new"], _ceil_t(lens, bs)
    more = torch.where(new > 0, _ceil_t(lens + new, bs) - held, 0)
    tail_col = (lens // bs).clamp(max=per - 1).long()
    seq = torch.arange(n_seqs, device=DEV)
    tail = table[seq, tail_col].long()
    writes = (new > 0) & (lens % bs > 0)
    same = (tail[:, None] == tail) & writes[:, None] & writes
    later = same & (seq > seq[:, None])
    shared = ref[tail.clamp(min=0)]
    own_copy = writes & (shared > 1) & ((same.sum(1) < shared) | later.any(1))
    take = more + own_copy.int()
    first = take.cumsum(0) - take
    free = torch.argsort((ref > 0).int(), stable=True).int()                      # free blocks, lowest first
    old, fresh = tail.clamp(min=0), free[first]
    got = torch.where(own_copy, fresh.long(), old)
    for_new = (col >= held[:, None]) & (col < (held + more)[:, None])
    pick = (first + own_copy.int())[:, None] + col - held[:, None]
    table.copy_(torch.where(for_new, free[pick.clamp(0, s["n_blocks"] - 1).long()], table))
    table[seq, tail_col] = torch.where(own_copy, fresh, table[seq, tail_col])
    ref.index_add_(0, old, -own_copy.int())
    taken = torch.cat((torch.where(for_new, table, -1).flatten(), torch.where(own_copy, fresh, -1))).long()
    ref.index_add_(0, taken.clamp(min=0), (taken >= 0).int())
    kids = dst
    a, z, rows = old[kids], got[kids], (torch.arange(bs, device=DEV) < (lens % bs)[kids, None])[..., None, None]
    s["pools"][:, :, z] = torch.where(rows, s["pools"][:, :, a], s["pools"][:, :, z])
    held_by = dict(table=table.clone(), ref=ref.clone(), len=lens.clone())
    # release: the branches are dropped again
    keep = s["keep"]
    drop = (keep >= 0)[:, None] & (col >= _ceil_t(keep.clamp(min=0), bs)[:, None]) & (table >= 0)
    ref.index_add_(0, table.flatten().clamp(min=0).long(), -drop.flatten().int())
    table.masked_fill_(drop, -1)
    lens.copy_(torch.where(keep >= 0, torch.minimum(lens, keep), lens))
    return held_by


def _ceil_t(a, b):
    return (a + b - 1) // b


def _plain_compact(s):
    table, ref = s["table"], s["ref"]
    table.copy_(s["table0"])
    ref.copy_(s["ref0"])
    live = ref > 0
    used = live.sum()
    ids = torch.arange(s["n_blocks"], device=DEV)
    src = torch.nonzero(live & (ids >= used)).flatten()
    dst = torch.nonzero(~live & (ids < used)).flatten()
    s["pools"][:, :, dst] = s["pools"][:, :, src]
    to = ids.int()
    to[src] = dst.int()
    table.copy_(torch.where(table >= 0, to[table.clamp(min=0).long()], table))
    ref[dst] = ref[src]
    ref[src] = 0


# ---- the library's calls ----------------------------------------------------

_engines = {}


def _engine(case, cap):
    """The program's library context for these heads: capacities rounded up, so that one serves many calls."""
    from eagle_feature_level_gb300 import runtime as R
    most = 1 << max(10, (cap - 1).bit_length())
    key = (case["hq"], case["hkv"], case["dh"], most)
    if key not in _engines:
        dims = dict(d=case["hq"] * case["dh"], n_q_heads=case["hq"], n_kv_heads=case["hkv"], head_dim=case["dh"],
                    d_ff=64, vocab=64)
        _engines[key] = R.Engine(dims, max_batch=256, max_rows=8, max_expanded=1, max_children=1, max_tree=2,
                                 max_prefix=most, device=DEV)
    return _engines[key]


def _bind(s):
    """The structs of the calls over this state's buffers, as a program keeps them beside the buffers."""
    from eagle_feature_level_gb300 import _binding as L
    c = s["case"]
    p = lambda t: t.data_ptr()
    if c["op"] in ("append", "attend"):
        eng = _engine(c, s["cap"])
        rows = L.eagle_rows(p(s["row_start"]), s["n_rows"])
        paging = L.eagle_paging(p(s["table"]), c["bs"], s["n_blocks"]) if c["bs"] else L.eagle_paging()
        kv = L.eagle_kv(p(s["k"]), p(s["v"]), s["cap"], p(s["len"]), paging)
        s["abi"] = dict(eng=eng, rows=rows, kv=kv)
        if c["op"] == "append":
            kind = {"none": None, "linear": L.ROPE_LINEAR, "bands": L.ROPE_BANDS, "ramp": L.ROPE_RAMP}[c["scaling"]]
            sc = None if kind is None else L.eagle_rope_scaling(kind, *SCALING[c["scaling"]], 0.0)
            s["abi"]["rope"] = L.eagle_rope_plan(c["dh"], c["rot"], int(c["inter"]), c["theta"], sc)
            s["abi"]["dtype"] = L.DTYPE_F32 if c["f32"] else L.DTYPE_BF16
            e, ld = s["qkv"].element_size(), s["qkv"].shape[1]
            q, qd, kd = p(s["qkv"]), c["hq"] * c["dh"], c["hkv"] * c["dh"]
            s["abi"]["io"] = (q, ld, p(s["q_out"]), qd, q + qd * e, ld, q + (qd + kd) * e, ld)
        return
    eng = _engine(c, s["per"] * c["bs"])
    pages = L.eagle_pages(p(s["table"]), p(s["len"]), p(s["ref"]), p(s["scratch"]), s["n_seqs"], s["per"], c["bs"],
                          s["n_blocks"])
    pools = L.eagle_pools([p(s["pools"][l, 0]) for l in range(c["layers"])],
                          [p(s["pools"][l, 1]) for l in range(c["layers"])])
    s["abi"] = dict(eng=eng, pages=pages, pools=pools)


def _own(s):
    from eagle_feature_level_gb300 import _binding as L
    if "abi" not in s:
        _bind(s)
    a, c = s["abi"], s["case"]
    eng = a["eng"]
    ws, st = eng.ws.data_ptr(), eng.stream()
    if c["op"] == "append":
        L.eagle_kv_append(eng.ctx, c["B"], a["rows"], a["rope"], a["dtype"], *a["io"], a["kv"], None,
                          s["len_out"].data_ptr(), ws, st)
    elif c["op"] == "attend":
        L.eagle_chunk_attn(eng.ctx, c["B"], a["rows"], s["q"].data_ptr(), c["hq"] * c["dh"], a["kv"], c["window"],
                           1.0 / math.sqrt(c["dh"]), s["out"].data_ptr(), c["hq"] * c["dh"], ws, st)
    elif c["op"] == "branch":
        L.eagle_pages_fork(eng.ctx, a["pages"], s["src"].shape[0], s["src"].data_ptr(), s["dst"].data_ptr(), ws, st)
        L.eagle_pages_reserve(eng.ctx, a["pages"], a["pools"], s["n_new"].data_ptr(), ws, st)
        held = dict(table=s["table"].clone(), ref=s["ref"].clone(), len=s["len"].clone())
        L.eagle_pages_release(eng.ctx, a["pages"], s["keep"].data_ptr(), ws, st)
        return held
    else:
        s["table"].copy_(s["table0"])
        s["ref"].copy_(s["ref0"])
        L.eagle_pages_compact(eng.ctx, a["pages"], a["pools"], ws, st)


def run(s):
    op = s["case"]["op"]
    if own:
        held = _own(s)
    else:
        held = {"append": _plain_append, "attend": _plain_attend, "branch": _plain_branch, "compact": _plain_compact}[op](s)
    if op == "append":
        return dict(q=s["q_out"], k=s["k"], v=s["v"], len=s["len_out"])
    if op == "attend":
        return dict(out=s["out"])
    if op == "branch":
        return dict(held=held, table=s["table"], ref=s["ref"], len=s["len"], pools=s["pools"])
    return dict(table=s["table"], ref=s["ref"], pools=s["pools"])


# ---- the definitions in 64 bits ---------------------------------------------

def _exact_frequencies(case):
    rot, theta, kind = case["rot"], case["theta"], case["scaling"]
    factor, low, high, orig = SCALING.get(kind, (1.0, 0.0, 0.0, 0))
    fs = []
    for i in range(rot // 2):
        f = math.exp(-2.0 * i / rot * math.log(theta))
        wave = 2.0 * math.pi / f
        if kind == "bands":
            if wave > orig / low:
                f = f / factor
            elif wave >= orig / high:
                part = (orig / wave - low) / (high - low)
                f = (1.0 - part) * f / factor + part * f
        elif kind == "ramp":
            # the pair (a real number) whose wave turns `high`, then `low` times in the original length
            ends = [rot / 2.0 * math.log(orig / (2.0 * math.pi * t), theta) for t in (high, low)]
            lo, hi = max(0, math.floor(ends[0])), min(rot - 1, math.ceil(ends[1]))
            slowed = 1.0 if i >= hi and hi > lo else 0.0 if i <= lo else min(1.0, (i - lo) / max(hi - lo, 1e-3))
            f = f * (1.0 - slowed) + f / factor * slowed
        elif kind == "linear":
            f = f / factor
        fs.append(f)
    return torch.tensor(fs, dtype=torch.float64, device=DEV), 1.0 + 0.1 * math.log(factor) if kind == "ramp" else 1.0


def exact(case, seed):
    if case["op"] in ("branch", "compact"):
        return None                                            # whole numbers and moved bits: equality
    s = prepare(case, seed)
    ctx, new = _lens(case)
    hq, hkv, dh, bs = case["hq"], case["hkv"], case["dh"], case["bs"]
    G = hq // hkv
    where = lambda b, lo, hi: (torch.arange(lo, hi, device=DEV) + b * s["cap"] if bs == 0 else
                               s["table"][b].long()[torch.arange(lo, hi, device=DEV) // bs] * bs
                               + torch.arange(lo, hi, device=DEV) % bs)
    if case["op"] == "append":
        rot = case["rot"]
        q = s["q_out"].double()
        k, v = s["k"].double(), s["v"].double()
        f, m = _exact_frequencies(case)
        first, second = (torch.arange(0, rot, 2), torch.arange(1, rot, 2)) if case["inter"] else \
            (torch.arange(rot // 2), torch.arange(rot // 2, rot))
        r = 0
        for b in range(case["B"]):
            n = new[b]
            x = s["qkv"][r:r + n].double().reshape(n, hq + 2 * hkv, dh)
            # each pair as a complex number, times m e^(i position frequency)
            turn = torch.polar(torch.full((), m, dtype=torch.float64, device=DEV).expand(n, rot // 2).contiguous(),
                               torch.arange(ctx[b], ctx[b] + n, device=DEV, dtype=torch.float64)[:, None] * f)
            y = x.clone()
            z = torch.complex(x[..., first], x[..., second]) * turn[:, None]
            y[..., first], y[..., second] = z.real, z.imag
            q[r:r + n] = y[:, :hq]
            at = where(b, ctx[b], ctx[b] + n)
            k.view(-1, hkv, dh)[at] = y[:, hq:hq + hkv]
            v.view(-1, hkv, dh)[at] = x[:, hq + hkv:]
            r += n
        return dict(q=q, k=k, v=v, len=None)
    out = s["out"].double()
    r = 0
    for b in range(case["B"]):
        n, L = new[b], ctx[b] + new[b]
        at = where(b, 0, L)
        pos = torch.arange(ctx[b], L, device=DEV)[:, None]
        j = torch.arange(L, device=DEV)
        hide = (j > pos) | (j <= pos - case["window"]) if case["window"] else j > pos
        for h in range(hkv):
            k = s["k"].view(-1, hkv, dh)[at, h].double()
            v = s["v"].view(-1, hkv, dh)[at, h].double()
            x = torch.einsum("ngd,ld->gnl", s["q"][r:r + n, h * G:(h + 1) * G].double(), k) / math.sqrt(dh)
            x = torch.softmax(x.masked_fill(hide, -math.inf), -1)
            out[r:r + n, h * G:(h + 1) * G] = torch.einsum("gnl,ld->ngd", x, v)
        r += n
    return dict(out=out)
