"""The rest of a target model's step around its KV cache, as measured work: root-mean-square norms with the residual's
addition, linear layers in microscaled 8 and 4 bits with the quantisation of their inputs, and tokens (or whole
distributions for the verified tree) from logits under temperature, top-k, top-p and min-p.

`run` computes each in plain torch or, with `own` set, through the library's calls.  A case's sampling controls come
from the case alone (`shape` seeds them); the values come from the seed.

Microscaled formats, blocks along a row: "fp8" e4m3 in blocks of 32 and "fp4" e2m1 in blocks of 32, each with a power
of two (the smallest that brings the block's largest magnitude within the element type's range); "nv4" e2m1 in blocks
of 16 with an e4m3 scale and one fp32 factor g for the tensor: the scale is rounded from the fp32 quotient largest /
(6 g), the elements from the fp32 quotients x / d with the fp32 product d = scale g.  Two e2m1 share a byte, the first in its low half.  Scales lie in groups of 128 rows x 4 blocks: 32 rows' quadruples 16 bytes apart, the four sets
of 32 rows next to each other.
"""
import math
import random

import torch

own = False

DEV = "cuda"
BF16, F32 = torch.bfloat16, torch.float32


# ---- cases ------------------------------------------------------------------

def _norm(name, rows, cols, res, out, x="bf16"):
    """res, x: "bf16" or "f32" (res "" for none); out: those, or a microscaled format."""
    return dict(name=name, op="norm", rows=rows, cols=cols, x=x, res=res, out=out)


def _linear(name, rows, cols, outs, fmt, out="bf16", gated=False, bias=False, x="bf16"):
    return dict(name=name, op="linear", rows=rows, cols=cols, outs=outs, fmt=fmt, out=out, gated=gated, bias=bias, x=x)


def _sample(name, requests, each, vocab, x, k, p, m, greedy, probs, shape=1):
    """k, p, m: whether requests set top-k, top-p, min-p; greedy: the share of requests at temperature 0."""
    return dict(name=name, op="sample", requests=requests, each=each, vocab=vocab, x=x, k=k, p=p, m=m, greedy=greedy,
                probs=probs, shape=shape)


def listed():
    return [
        # one decoding token of each of 8 requests, hidden size of a 7B target: latency
        _norm("norm tokens", 8, 4096, "bf16", "bf16"),
        # the last norm of a batch of tree rows over an fp32 residual stream, whose sum is the round's feature
        _norm("norm features", 777, 5120, "f32", "f32"),
        # a long prompt's rows on their way into an 8-bit product, hidden size of a 70B target
        _norm("norm prompt 8 bits", 8192, 8192, "bf16", "fp8"),
        # one token through the fused q, k, v projection of a 7B target: latency and the weights' bytes
        _linear("linear token", 1, 4096, 12288, "nv4"),
        # 16 decoding tokens through the LM head of a 70B target
        _linear("linear lm head", 16, 8192, 32000, "nv4", "f32"),
        # the verified trees of 8 requests (27 slots each) through the gate and up projections of a 13B target
        _linear("linear trees", 216, 5120, 27648, "fp8"),
        # an odd number of rows, gated inside the quantisation, through the down projection of a 7B target
        _linear("linear gated rows", 1001, 11008, 4096, "fp4", gated=True),
        # a prompt's rows through the fused projection of a 70B target
        _linear("linear prompt", 4096, 8192, 10240, "nv4"),
        # the first token of one request, with the usual controls: latency
        _sample("sample one", 1, 1, 32000, "f32", True, True, False, 0.0, False),
        # a decoding batch over a large vocabulary, a quarter of it greedy
        _sample("sample batch", 64, 1, 131072, "bf16", False, True, True, 0.25, False),
        # the target's distributions at every slot of 8 verified trees, as acceptance takes them
        _sample("sample trees", 8, 27, 32000, "f32", True, True, True, 0.0, True),
    ]


def _logu(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "linear", "linear", "sample"])
    if op == "norm":
        cols = 32 * _logu(rng, 2, 512)
        rows = _logu(rng, 1, min(32768, (1 << 26) // cols))
        c = _norm("", rows, cols, rng.choice(["bf16", "f32", ""]), rng.choice(["bf16", "f32", "fp8", "fp4", "nv4"]),
                  rng.choice(["bf16", "bf16", "f32"]))
    elif op == "linear":
        cols, outs = 32 * _logu(rng, 2, 896), _logu(rng, 8, 32768)
        most = min(8192, int(4096 * 8192 * 10240 / (cols * outs)), (1 << 27) // cols, (1 << 27) // outs)
        gated = rng.random() < 0.2
        c = _linear("", _logu(rng, 1, max(1, most)), cols, outs, rng.choice(["fp8", "fp4", "nv4"]),
                    "bf16" if gated else rng.choice(["bf16", "bf16", "f32"]), gated, rng.random() < 0.3,
                    rng.choice(["bf16", "bf16", "f32"]))
    else:
        vocab = _logu(rng, 500, 250000)
        each = rng.choice([1, 1, rng.randint(2, 64)])
        rows = _logu(rng, 1, max(1, min(512, (64 * 131072) // vocab)))
        c = _sample("", max(1, rows // each), each, vocab, rng.choice(["bf16", "f32"]), rng.random() < 0.5,
                    rng.random() < 0.6, rng.random() < 0.4, rng.choice([0.0, 0.3]), rng.random() < 0.4,
                    rng.randrange(1 << 30))
    del c["name"]
    return c


BLOCK = {"fp8": 32, "fp4": 32, "nv4": 16}
SIZE = {"bf16": 2, "f32": 4}


def _mx_bytes(fmt, rows, cols):
    return rows * cols // (1 if fmt == "fp8" else 2) + rows * (cols // BLOCK[fmt])


def work(case):
    if case["op"] == "norm":
        n = case["rows"] * case["cols"]
        res = 2 * SIZE[case["res"]] if case["res"] else 0
        return {"bytes": n * (SIZE[case["x"]] + res + SIZE.get(case["out"], 2)) + 4 * case["cols"], "flops": 5 * n}
    if case["op"] == "linear":
        r, k, n = case["rows"], case["cols"], case["outs"]
        return {"bytes": r * k * SIZE[case["x"]] * (2 if case["gated"] else 1) + _mx_bytes(case["fmt"], n, k)
                + r * n * SIZE[case["out"]] + (4 * n if case["bias"] else 0), "flops": 2 * r * k * n}
    rows, v = case["requests"] * case["each"], case["vocab"]
    return {"bytes": rows * (v * SIZE[case["x"]] + (v * 4 if case["probs"] else 0) + 12), "flops": 4 * rows * v}


# ---- microscaled formats in plain torch --------------------------------------

E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _scale_layout(s):
    """Scales [rows, blocks] as bytes in their groups of 128 x 4, zero behind the last row and block."""
    r, c = s.shape
    p = torch.zeros((-r) % 128 + r, (-c) % 4 + c, dtype=torch.uint8, device=DEV)
    p[:r, :c] = s
    return p.view(-1, 4, 32, p.shape[1] // 4, 4).permute(0, 3, 2, 1, 4).contiguous()


def _scale_rows(s, rows, blocks):
    return s.permute(0, 3, 2, 1, 4).reshape(s.shape[0] * 128, -1)[:rows, :blocks]


def _codes4(v):
    """e2m1 of v, ties to the even code, sign in bit 3."""
    a = v.abs()
    c = (a > 0.25).byte() + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0)
    return c + 8 * torch.signbit(v).byte()


def _pow2(n):
    """2^n of whole n in [-127, 127] in 32 bits, by its bits (a power function may be a step off)."""
    return torch.where(n < -126, 1 << 22, (n.int() + 127) << 23).int().view(F32)


def _quantize(fmt, x, g):
    """(elements, scales in their layout) of x (fp32): bytes as the formats hold them."""
    r, k = x.shape
    b = x.view(r, -1, BLOCK[fmt])
    top = b.abs().amax(-1)
    if fmt == "nv4":
        s8 = (top / (6.0 * g)).clamp(max=448.0).to(torch.float8_e4m3fn)
        s = s8.float() * g
        v = torch.where(s[..., None] > 0, b / torch.where(s > 0, s, 1.0)[..., None], b * 0.0)
        byte = s8.view(torch.uint8)
    else:
        m, e = torch.frexp(top / (448.0 if fmt == "fp8" else 6.0))   # the division by 6 cannot cross a power of two
        e = torch.where(m == 0.5, e - 1, e).clamp(min=-127)
        byte = torch.where(top > 0, e + 127, 0).byte()
        v = b * _pow2(127 - byte.int())[..., None]
    v = v.view(r, k)
    if fmt == "fp8":
        return v.to(torch.float8_e4m3fn).view(torch.uint8), _scale_layout(byte)
    c = _codes4(v)
    return c[:, 0::2] | (c[:, 1::2] << 4), _scale_layout(byte)


def _values(fmt, data, scale, g, dtype=F32):
    """The values that elements and scales stand for."""
    if fmt == "fp8":
        v = data.view(torch.float8_e4m3fn).to(dtype)
    else:
        table = torch.tensor(E2M1 + tuple(-x for x in E2M1), dtype=dtype, device=DEV)
        v = table[torch.stack((data & 15, data >> 4), -1).flatten(-2).int()]
    r, k = v.shape
    s = _scale_rows(scale, r, k // BLOCK[fmt])
    if fmt == "nv4":
        s = s.contiguous().view(torch.float8_e4m3fn).to(F32) * g
    else:
        s = _pow2(s.int() - 127)
    return (v.view(r, -1, BLOCK[fmt]) * s.to(dtype)[..., None]).view(r, k)


# ---- inputs -----------------------------------------------------------------

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _normal(g, *shape):
    return torch.empty(shape, device=DEV).normal_(generator=g)


def _rows(g, rows, cols, dtype):
    """Hidden states: normal, channels of unlike sizes, one in 128 of them far larger."""
    size = torch.exp(0.4 * _normal(g, cols))
    size *= torch.where(torch.rand(cols, generator=g, device=DEV) < 1 / 128, 12.0, 1.0)
    return (_normal(g, rows, cols) * size).to({"bf16": BF16, "f32": F32}[dtype])


def _controls(case):
    """Per request: temperature, top-k, top-p, min-p."""
    r = random.Random(case["shape"] * 7 + 1)
    t, k, p, m = [], [], [], []
    for _ in range(case["requests"]):
        t.append(0.0 if r.random() < case["greedy"] else r.uniform(0.5, 1.3))
        k.append(r.choice([1, 5, 20, 50, 50, 400]) if case["k"] and r.random() < 0.8 else 0)
        p.append(r.uniform(0.6, 0.99) if case["p"] and r.random() < 0.8 else 1.0)
        m.append(r.uniform(0.01, 0.2) if case["m"] and r.random() < 0.8 else 0.0)
    return t, k, p, m


def prepare(case, seed):
    g = _gen(seed)
    s = dict(case=case)
    if case["op"] == "norm":
        r, c = case["rows"], case["cols"]
        s["x"] = _rows(g, r, c, case["x"])
        s["res"] = _rows(g, r, c, case["res"]) * 3 if case["res"] else None
        s["gain"] = 1.0 + 0.3 * _normal(g, c)
        s["g"] = torch.full((), 16.0 / (6 * 448), device=DEV)     # as a calibration leaves it: the largest value seen
    elif case["op"] == "linear":
        r, k, n, fmt = case["rows"], case["cols"], case["outs"], case["fmt"]
        s["x"] = _rows(g, r, k * (2 if case["gated"] else 1), case["x"])
        w = _normal(g, n, k) / math.sqrt(k)
        s["gw"] = w.abs().amax() / (6 * 448)
        s["w"], s["ws"] = _quantize(fmt, w, s["gw"])
        s["g"] = (s["x"].abs().amax().float() / (6 * 448)).clone()
        s["bias"] = _normal(g, n) * 0.1 if case["bias"] else None
    else:
        n, v = case["requests"] * case["each"], case["vocab"]
        z = 2.5 * _normal(g, n, v)
        # a few likely tokens a row, from a sharp choice to a dozen of about one size
        at = torch.randint(0, v, (n, 12), generator=g, device=DEV)
        z.scatter_(1, at, 7.0 + 5.0 * _normal(g, n, 12))
        s["z"] = z.to({"bf16": BF16, "f32": F32}[case["x"]])
        s["u"] = torch.randint(-(1 << 31), 1 << 31, (n,), generator=g, device=DEV, dtype=torch.int64).int()
        t, k, p, m = _controls(case)
        s["t"] = torch.tensor(t, dtype=F32, device=DEV)
        s["k"] = torch.tensor(k, dtype=torch.int32, device=DEV)
        s["p"] = torch.tensor(p, dtype=F32, device=DEV)
        s["m"] = torch.tensor(m, dtype=F32, device=DEV)
    return s


# ---- plain forms ------------------------------------------------------------

EPS = 1e-5


def _plain_norm(s):
    c = s["case"]
    h = s["x"].float()
    if s["res"] is not None:
        h = h + s["res"].float()
    y = h / torch.sqrt((h * h).mean(-1, keepdim=True) + EPS) * s["gain"]
    out = {}
    if s["res"] is not None:
        out["sum"] = h.to(s["res"].dtype)
    if c["out"] in BLOCK:
        out["y"] = _values(c["out"], *_quantize(c["out"], y, s["g"]), s["g"]).to(BF16)
    else:
        out["y"] = y.to(BF16 if c["out"] == "bf16" else F32)
    return out


def _plain_linear(s):
    c = s["case"]
    x = s["x"].float()
    if c["gated"]:
        a, b = x[:, :c["cols"]], x[:, c["cols"]:]
        x = a / (1.0 + torch.exp(-a)) * b
    x = _values(c["fmt"], *_quantize(c["fmt"], x, s["g"]), s["g"])
    y = x @ _values(c["fmt"], s["w"], s["ws"], s["gw"]).t()
    if s["bias"] is not None:
        y = y + s["bias"]
    return dict(y=y.to(BF16 if c["out"] == "bf16" else F32))


def _plain_sample(s):
    c = s["case"]
    each, v = c["each"], c["vocab"]
    per = lambda t: t.repeat_interleave(each)[:, None]
    z = s["z"].double()
    t, k, p, m = per(s["t"].double()), per(s["k"].long()), per(s["p"].double()), per(s["m"].double())
    greedy = t <= 0
    top, at = z.max(-1, keepdim=True)
    first = torch.where(z == top, torch.arange(v, device=DEV), v).amin(-1, keepdim=True)
    # whole weights floor(2^40 e^((z - max) / t)); from the largest down, the lower id first among equals
    w = torch.exp((z - top) / torch.where(greedy, 1.0, t)).mul_(2.0 ** 40).floor_().long()
    w = torch.where(greedy, (torch.arange(v, device=DEV) == first).long() << 40, w)
    order = torch.sort(z, dim=-1, descending=True, stable=True).indices
    ws = w.gather(1, order)
    ws = torch.where((torch.arange(v, device=DEV) < k) | (k <= 0), ws, 0)
    cum = ws.cumsum(-1)
    need = torch.ceil(p.clamp(0, 1) * cum[:, -1:].double()).long().clamp(min=1)
    ws = torch.where((cum - ws < need) | (p >= 1), ws, 0)
    ws = torch.where(ws.double() >= m * 2.0 ** 40, ws, 0)
    w = torch.zeros_like(w).scatter_(1, order, ws)
    cum = w.cumsum(-1)
    total = cum[:, -1:]
    # floor(u total / 2^32), u a 32-bit word, in halves that do not overflow
    u = s["u"].long()[:, None] & 0xffffffff
    lo, hi = total & 0xffffffff, total >> 32
    r = u * hi + (((u >> 16) * lo + ((u & 0xffff) * lo >> 16)) >> 16)
    out = dict(token=(cum <= r).sum(-1).int())
    if c["probs"]:
        out["probs"] = (w.double() / total).float()
        out["argmax"] = first[:, 0].int()
    return out


# ---- the library's calls ------------------------------------------------------

_engines = []


def _engine():
    """The program's library context."""
    from eagle_feature_level_gb300 import runtime as R
    if not _engines:
        dims = dict(d=4096, n_q_heads=32, n_kv_heads=32, head_dim=128, d_ff=64, vocab=64)
        _engines.append(R.Engine(dims, max_batch=256, max_rows=8, max_expanded=1, max_children=1, max_tree=2,
                                 max_prefix=1024, device=DEV))
    return _engines[0]


def _bind(s):
    """Output buffers and the structs of the calls over them, as a program keeps them."""
    from eagle_feature_level_gb300 import _binding as L
    c = s["case"]
    p = lambda t: None if t is None else t.data_ptr()
    dtype = {"bf16": L.DTYPE_BF16, "f32": L.DTYPE_F32}
    torch_type = {"bf16": BF16, "f32": F32}
    mx = {"fp8": L.MX_FP8, "fp4": L.MX_FP4, "nv4": L.NV_FP4}

    def tensor(fmt, rows, cols, g):
        data, scale = L.eagle_mx_layout(mx[fmt], rows, cols)
        held = (torch.empty(data, dtype=torch.uint8, device=DEV), torch.empty(scale, dtype=torch.uint8, device=DEV))
        return held, L.eagle_mx(p(held[0]), p(held[1]), p(g), rows, cols, mx[fmt])

    if c["op"] == "norm":
        r, k, quant = c["rows"], c["cols"], c["out"] in BLOCK
        s["y"] = torch.empty(r, k, dtype=torch_type.get(c["out"], BF16), device=DEV)
        s["sum"] = torch.empty_like(s["res"]) if c["res"] else None
        s["held"], s["q"] = tensor(c["out"], r, k, s["g"]) if quant else (None, None)
        s["call"] = L.eagle_norm(r, k, dtype[c["x"]], p(s["x"]), k, dtype.get(c["res"], 0), p(s["res"]), k,
                                 p(s["sum"]), k, p(s["gain"]), EPS, dtype.get(c["out"], 0), None if quant else p(s["y"]), k,
                                 L.ref(s["q"]))
    elif c["op"] == "linear":
        s["y"] = torch.empty(c["rows"], -(-c["outs"] // 8) * 8, dtype=torch_type[c["out"]], device=DEV)
        s["held"], s["q"] = tensor(c["fmt"], c["rows"], c["cols"], s["g"])
        s["wq"] = L.eagle_mx(p(s["w"]), p(s["ws"]), p(s["gw"]), c["outs"], c["cols"], mx[c["fmt"]])
        s["dt"], s["act"] = (dtype[c["x"]], dtype[c["out"]]), L.ACT_SWIGLU if c["gated"] else L.ACT_NONE
    else:
        n, v = c["requests"] * c["each"], c["vocab"]
        s["token"] = torch.empty(n, dtype=torch.int32, device=DEV)
        s["argmax"] = torch.empty_like(s["token"])
        s["probs"] = torch.empty(n, v, device=DEV) if c["probs"] else None
        s["call"] = L.eagle_filter(p(s["t"]), p(s["k"]) if c["k"] else None, p(s["p"]) if c["p"] else None,
                                   p(s["m"]) if c["m"] else None, c["each"], None)
        s["dt"] = dtype[c["x"]]


def _own(s):
    from eagle_feature_level_gb300 import _binding as L
    c, eng = s["case"], _engine()
    if "y" not in s and "token" not in s:
        _bind(s)
    ws, st = eng.ws.data_ptr(), eng.stream()
    if c["op"] == "norm":
        L.eagle_add_norm(eng.ctx, s["call"], ws, st)
        if s["q"] is not None:
            L.eagle_mx_unpack(eng.ctx, s["q"], L.DTYPE_BF16, s["y"].data_ptr(), c["cols"], ws, st)
        return dict(sum=s["sum"], y=s["y"]) if c["res"] else dict(y=s["y"])
    if c["op"] == "linear":
        L.eagle_mx_quantize(eng.ctx, s["dt"][0], s["act"], s["x"].data_ptr(), s["x"].shape[1], s["q"], ws, st)
        L.eagle_mx_linear(eng.ctx, s["q"], s["wq"], None if s["bias"] is None else s["bias"].data_ptr(), s["dt"][1],
                          s["y"].data_ptr(), s["y"].shape[1], ws, st)
        return dict(y=s["y"][:, :c["outs"]])
    L.eagle_sample(eng.ctx, c["requests"] * c["each"], c["vocab"], s["dt"], s["z"].data_ptr(), c["vocab"], s["call"],
                   s["u"].data_ptr(), s["token"].data_ptr(), s["argmax"].data_ptr() if c["probs"] else None,
                   s["probs"].data_ptr() if c["probs"] else None, c["vocab"], ws, st)
    return dict(token=s["token"], probs=s["probs"], argmax=s["argmax"]) if c["probs"] else dict(token=s["token"])


def run(s):
    if own:
        return _own(s)
    return {"norm": _plain_norm, "linear": _plain_linear, "sample": _plain_sample}[s["case"]["op"]](s)


# ---- the definitions in 64 bits ---------------------------------------------

def _two_to(e):
    return ((e.long() + 1023) << 52).view(torch.float64)


def _exponent(v):
    """e of 2^e <= v < 2^(e + 1), v > 0."""
    return torch.frexp(v).exponent - 1


def _exact_rounded(fmt, x, g):
    """x (64 bits) as the format holds it: each block's values to the nearest multiple that its scale allows."""
    r, k = x.shape
    b = x.reshape(r, -1, BLOCK[fmt])
    top = b.abs().max(-1, keepdim=True).values
    if fmt == "nv4":
        # the two quotients and the elements' divisor are 32-bit numbers by definition
        t = torch.clamp((top.float() / (6.0 * g).float()).double(), max=448.0)
        # e4m3: 3 bits behind the leading one down to 2^-6, multiples of 2^-9 below
        grid = _two_to(_exponent(t.clamp(min=2.0 ** -6)) - 3)
        s = (torch.round(t / grid) * grid * g).float().double()
    else:
        lead, whole = (1.75, 8) if fmt == "fp8" else (1.5, 2)    # the largest element is lead 2^whole
        e = _exponent(top.clamp(min=1e-300))
        e = torch.where(top > lead * _two_to(e), e + 1, e) - whole
        s = _two_to(e.clamp(min=-127))
    v = torch.where(s > 0, b / torch.where(s > 0, s, 1.0), 0.0)
    if fmt == "nv4":
        v = torch.where(s > 0, b.float() / torch.where(s > 0, s, 1.0).float(), 0.0).double()
    bits, least, most = (3, -6, 448.0) if fmt == "fp8" else (1, 0, 6.0)
    grid = _two_to(_exponent(v.abs().clamp(min=2.0 ** least)) - bits)
    v = torch.clamp(torch.round(v / grid) * grid, -most, most)
    return (v * s).reshape(r, k)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        h = s["x"].double() + (s["res"].double() if case["res"] else 0.0)
        y = h * torch.rsqrt(torch.sum(h * h, -1, keepdim=True) / case["cols"] + EPS) * s["gain"].double()
        if case["out"] in BLOCK:
            y = _exact_rounded(case["out"], y, s["g"].double())
        return dict(sum=h, y=y) if case["res"] else dict(y=y)
    if case["op"] == "linear":
        x = s["x"].double()
        if case["gated"]:
            k = case["cols"]
            x = x[:, :k] * torch.sigmoid(x[:, :k]) * x[:, k:]
        x = _exact_rounded(case["fmt"], x, s["g"].double())
        # the weights' values, from their bytes
        d, n, k = s["w"].long(), case["outs"], case["cols"]
        if case["fmt"] == "fp8":
            sign, e, f = d >> 7, (d >> 3) & 15, d & 7
            w = torch.where(e > 0, (1 + f.double() / 8) * _two_to(e - 7), f.double() / 512)
        else:
            d = torch.cat(((d & 15)[..., None], (d >> 4)[..., None]), -1).reshape(n, k)
            sign, e, f = d >> 3, (d >> 1) & 3, d & 1
            w = torch.where(e > 0, (1 + f.double() / 2) * _two_to(e - 1), f.double() / 2)
        w = torch.where(sign > 0, -w, w)
        row, blk = torch.arange(n, device=DEV)[:, None], torch.arange(k // BLOCK[case["fmt"]], device=DEV)[None]
        at = ((row // 128 * s["ws"].shape[1] + blk // 4) * 32 + row % 32) * 16 + row % 128 // 32 * 4 + blk % 4
        b = s["ws"].flatten()[at].long()
        if case["fmt"] == "nv4":
            e, f = b >> 3, b & 7
            b = torch.where(e > 0, (1 + f.double() / 8) * _two_to(e - 7), f.double() / 512)
            b = b * s["gw"].double()
        else:
            b = _two_to(b - 127)
        w = (w.reshape(n, -1, BLOCK[case["fmt"]]) * b[..., None]).reshape(n, k)
        y = x @ w.t()
        return dict(y=y if s["bias"] is None else y + s["bias"].double())
    if not case["probs"]:
        return None                                            # tokens alone: equality
    t, k, p, m = _controls(case)
    out = torch.zeros(case["requests"] * case["each"], case["vocab"], dtype=torch.float64, device=DEV)
    for r in range(out.shape[0]):
        i = r // case["each"]
        # the controls are 32-bit numbers
        ti, pi, mi = (torch.tensor(v[i], dtype=F32).item() for v in (t, p, m))
        z = s["z"][r].double()
        if ti <= 0:
            out[r, torch.nonzero(z == z.max())[0]] = 1.0
            continue
        q, order = torch.sort(z, descending=True, stable=True)
        q = torch.softmax(q / ti, 0)
        if k[i] > 0:
            q = q[:k[i]] / q[:k[i]].sum()
        if pi < 1:
            q = q[:int((q.cumsum(0) < pi).sum()) + 1]
        q = q[q >= mi * q[0]]
        out[r, order[:q.shape[0]]] = q / q.sum()
    return dict(token=None, probs=out, argmax=None)
