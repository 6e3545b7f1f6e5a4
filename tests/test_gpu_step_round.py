"""A round whose target distribution is cut by top-k, top-p and min-p (Round.set_filter): eagle_sample's distributions go into
the acceptance walk, and the committed tokens follow the cut distribution (the draft's own, q, stays whole)."""
import numpy as np
import pytest
import torch
from scipy.stats import chisquare

import eagle_synth as S
from eagle_feature_level_gb300 import _binding as B
from eagle_feature_level_gb300 import runtime as R
from eagle_feature_level_gb300.workload import make_round, standin
from oracle import step as O
from oracle import verify as Vf
from oracle.layer import DraftWeights
from oracle.round import run_round
from tests.gpu_harness import GpuGuide, compare_round, round_on

pytestmark = pytest.mark.gpu

V, K, BATCH = 6, 3, 16384


def flat_round(batch, seed):
    """Requests whose root has K drawn children, none expanded: (engine, round, draft distribution)."""
    eng = R.Engine(dict(d=64, n_q_heads=4, n_kv_heads=4, head_dim=16, d_ff=64, vocab=V), max_batch=batch, max_rows=1,
                   max_expanded=1, max_children=K, max_tree=1 + K, max_prefix=1)
    rd = R.Round(eng, B.eagle_plan_static([-1] * K, list(range(K))), batch, kv_cap=1)
    q = np.random.default_rng(seed).dirichlet(np.ones(V)).astype(np.float32)
    rd.t_parent[:, 0], rd.t_parent[:, 1:] = -1, 0
    rd.t_exp.fill_(-1)
    rd.t_exp[:, 0] = 0
    rd.t_size.fill_(1 + K)
    rd.t_child_slot.copy_(torch.arange(1, 1 + K, dtype=torch.int32).expand(batch, 1, K))
    rd.probs.copy_(torch.from_numpy(q).expand(batch, 1, V))
    return eng, rd, q


def draw_children(rd, q, gen):
    d = torch.multinomial(torch.from_numpy(q).expand(rd.B, V), K, replacement=False, generator=gen).int()
    rd.t_token[:, 1:] = d.cuda()
    rd.c_token.copy_(d.view(rd.B, 1, K))


@pytest.mark.parametrize("controls", [dict(top_k=2), dict(top_p=0.6), dict(min_p=0.3), dict(top_k=4, top_p=0.8, min_p=0.05)],
                         ids=["k", "p", "m", "kpm"])
def test_committed_tokens_follow_the_cut_target(controls):
    eng, rd, q = flat_round(BATCH, 5)
    z = torch.tensor(np.random.default_rng(6).standard_normal(V) * 1.2, dtype=torch.float32)
    rd.target_logits.copy_(z.expand(BATCH, 1 + K, V))
    rd.temps.fill_(0.9)
    full = lambda k, t: None if k not in controls else torch.full((BATCH,), controls[k], dtype=t, device="cuda")
    rd.set_filter(full("top_k", torch.int32), full("top_p", torch.float32), full("min_p", torch.float32))
    f32 = lambda k, d: float(np.float32(controls.get(k, d)))
    w = O.distribution(z.numpy(), float(np.float32(0.9)), controls.get("top_k", 0), f32("top_p", 1.0), f32("min_p", 0.0))
    assert 0 < (w == 0).sum() < V - 1
    gen = torch.Generator().manual_seed(11)
    first = np.zeros(V)
    for call in range(12):
        draw_children(rd, q, gen)
        rd.set_sampling(0x5EED, 500 + call)
        rd.accept()
        a, path, fin, tok = (t.cpu().numpy() for t in (rd.accept_len, rd.path, rd.final_token, rd.t_token))
        np.add.at(first, np.where(a >= 1, tok[np.arange(BATCH), path[:, 1].clip(0)], fin), 1)
    assert eng.status() == 0
    eng.close()
    keep = w > 0
    assert not first[~keep].any()
    assert chisquare(first[keep], w[keep] / w.sum() * first.sum()).pvalue > 1e-3, (first / first.sum(), w / w.sum())


def test_a_filter_that_cuts_nothing_changes_nothing():
    eng, rd, q = flat_round(512, 8)
    rd.target_logits.copy_(torch.randn(512, 1 + K, V, generator=torch.Generator().manual_seed(1)))
    rd.temps.copy_(torch.rand(512, generator=torch.Generator().manual_seed(2)) + 0.3)
    rd.temps[::7] = 0.0                                  # greedy requests among them
    rd.t_size[::5] = 2                                   # and trees of two slots, their other children pruned
    rd.t_child_slot[::5, :, 1:] = -1
    draw_children(rd, q, torch.Generator().manual_seed(3))
    rd.set_sampling(1, 2)
    got = []
    for filtered in (False, True):
        rd.set_filter(torch.full((512,), 99, dtype=torch.int32, device="cuda") if filtered else None)
        rd.target_probs.fill_(-3.0)
        rd.target_argmax.fill_(-3)
        rd.accept()
        got.append([t.clone() for t in (rd.accept_len, rd.final_token, rd.last_slot, rd.target_argmax, rd.target_probs)])
    assert eng.status() == 0
    used = torch.arange(1 + K, device="cuda") < rd.t_size[:, None]
    for a, b in zip(got[0][:3], got[1][:3]):
        assert torch.equal(a, b)
    assert torch.equal(got[0][3][used], got[1][3][used])
    assert (got[1][4][~used] == -3).all() and (got[1][3][~used] == -3).all()
    # softmax against whole weights: fp32's exponential and sum, and the 2^-40 that a whole weight drops
    hot = used & (rd.temps > 0)[:, None]
    assert float((got[0][4][hot] - got[1][4][hot]).abs().max()) < 1e-6
    eng.close()


def test_filter_checks_its_tensors():
    eng, rd, _ = flat_round(4, 1)
    with pytest.raises(ValueError):
        rd.set_filter(top_k=torch.zeros(3, dtype=torch.int32, device="cuda"))
    with pytest.raises(ValueError):
        rd.set_filter(top_p=torch.zeros(4, dtype=torch.float64, device="cuda"))
    rd.set_filter(min_p=torch.zeros(4, device="cuda"))
    rd.set_filter()
    assert rd.filter_c is None
    eng.close()


# ---- whole rounds at a real vocabulary -------------------------------------------------------------------

ROUNDS = 3
WORK = S.variant("70b_x16_eagle2", name="filtered_eagle2_gqa", d=256, n_q_heads=8, n_kv_heads=2, head_dim=32, d_ff=688, vocab=32000,
                 batch=4, prefix_len=100, top_k=4, depth=4, top_m=12, weight_std=0.05, temps=(0.7, 0.0, 1.0, 0.9))
TOP_K, TOP_P, MIN_P = [50, 7, 2000, 0], [0.9, 0.5, 0.95, 0.8], [0.0, 0.2, 1e-4, 0.01]


def on_gpu(top_k, top_p, min_p):
    return (torch.tensor(top_k, dtype=torch.int32, device="cuda"), torch.tensor(top_p, dtype=torch.float32, device="cuda"),
            torch.tensor(min_p, dtype=torch.float32, device="cuda"))


class CutGuide(GpuGuide):
    """The oracle follows the GPU's walk where that is its own walk over the GPU's cut distributions (compared with the
    definition's by is_cut)."""

    def accept(self, b, tr, own):
        gpu, size = self.gpu, tr.size
        a = int(gpu["accept_len"][b])
        g = (a, [int(x) for x in gpu["path"][b, :a + 1]], int(gpu["final_token"][b]))
        if self.temps[b] <= 0:
            replay = Vf.accept_greedy(tr, gpu["target_logits"][b, :size].double().numpy())
        else:
            replay = Vf.accept_sampling(tr, gpu["target_probs"][b, :size].double().numpy(), gpu["probs"][b].double().numpy(),
                                        self._st[b].child_tok, b, self.inp["philox_seed"], self.inp["round_id"])
        if (replay[0], list(replay[1]), int(replay[2])) != g:
            self.errors.append(f"b{b} accept: GPU {g} but the oracle's walk is {replay}")
        return g


def is_cut(z, t, k, p, m, probs, argmax):
    """probs and argmax of one row are the definition's from its logits (a border may fall to either side within the weights'
    two units; probabilities by two fp32 roundings and the weights)."""
    z, probs = z.double().numpy(), probs.double().numpy()
    assert argmax == np.flatnonzero(z == z.max())[0]
    w = O.weights(z, t)
    if not t > 0:
        assert np.array_equal(probs, w / w.sum())
        return
    order, lo, hi = O.kept(z, w, k, p, slack=2 * z.size)
    for c in range(lo, hi + 1):
        x = np.zeros_like(w)
        x[order[:c]] = w[order[:c]]
        x[x < m * 2.0 ** 40] = 0
        q = x / x.sum()
        if (np.abs(probs - q) <= 2.0 ** -22 * q + 4.0 / x.sum()).all() and ((probs > 0) == (x > 0))[x != 1].all():
            return
    raise AssertionError((t, k, p, m, lo, hi, int((probs > 0).sum())))


def check_cut_round(rd, gpu, Wd, controls):
    res = run_round(Wd, WORK, gpu["inputs_cpu"], guide=(guide := CutGuide(WORK, gpu)))
    f32 = lambda v: float(np.float32(v))
    for b, r in enumerate(res):
        r["guide"], t, size = guide, f32(gpu["inputs_cpu"]["temps"][b]), r["tree"].size
        for s in range(size):
            is_cut(gpu["target_logits"][b, s], t, controls[0][b], f32(controls[1][b]), f32(controls[2][b]), gpu["target_probs"][b, s],
                   int(gpu["target_argmax"][b, s]))
        r["target_probs"] = gpu["target_probs"][b, :size].double().numpy()
    rep = compare_round(WORK, gpu, res)
    assert rep["ok"], rep["errors"]
    assert rep["reached"] == {b: "commit" for b in range(WORK.batch)}


def host_state(rd, base):
    """Host copy of the round's inputs as the GPU holds them now."""
    inp = dict(base)
    inp.update(prefix_len=[int(x) for x in rd.pos0.cpu()], draft_len=[int(x) for x in rd.draft_len.cpu()], t_next=rd.t_next.cpu(),
               f_last=rd.f_last.cpu(), round_id=rd.round_id)
    for k, t in (("draft_k", rd.draft_k), ("draft_v", rd.draft_v), ("tgt_k", rd.tgt_k[0]), ("tgt_v", rd.tgt_v[0])):
        inp[k] = t.cpu()
    return inp


def cut_round(seed, more=0):
    W = S.draft_weights(WORK, seed, device="cuda")
    inp = dict(S.round_inputs(WORK, seed, device="cuda"))
    for k in ("draft_k", "draft_v", "tgt_k", "tgt_v"):   # room for the rounds' rows
        t = inp[k]
        inp[k] = torch.cat([t, torch.zeros(t.shape[0], more, *t.shape[2:], dtype=t.dtype, device=t.device)], 1)
    inp["kv_cap"] += more
    eng, rd = make_round(WORK, inp)
    rd.set_filter(*on_gpu(TOP_K, TOP_P, MIN_P))
    base = {k: (v.detach().cpu() if torch.is_tensor(v) else v) for k, v in inp.items()}
    return eng, rd, inp, base, eng.weights(W), DraftWeights({k: v.cpu() for k, v in W.items()}, WORK)


def test_cut_rounds_in_a_row_against_the_oracle():
    """Trees of several levels, 32000 tokens, greedy and sampled requests under controls of their own: every distribution is
    the definition's, every walk over them the oracle's, and what is committed that walk's."""
    eng, rd, inp, base, w_c, Wd = cut_round(91, ROUNDS * (WORK.depth + 1))
    accepted = 0
    for r in range(ROUNDS):
        rd.set_sampling(inp["philox_seed"], 7 + r)
        gpu = round_on(eng, rd, w_c, inp, host_state(rd, base))
        check_cut_round(rd, gpu, Wd, (TOP_K, TOP_P, MIN_P))
        accepted += int(rd.accept_len.sum())
        rd.refresh(w_c)
        rd.advance()
    assert eng.status() == 0 and accepted > 0
    eng.close()


def test_cut_round_captured():
    """A round's two graphs with a filter: replays give what the eager round gives, and follow the controls' present values."""
    eng, rd, inp, base, w_c, Wd = cut_round(92)
    filters = [(TOP_K, TOP_P, MIN_P), ([3, 0, 1, 900], [1.0, 0.9, 0.7, 0.99], [0.05, 0.0, 0.0, 1e-3])]
    held = on_gpu(*filters[0])
    rd.set_filter(*held)
    state = [(t, t.clone()) for t in (rd.draft_len, rd.tgt_len, rd.pos0, rd.draft_k, rd.draft_v, rd.tgt_k[0], rd.tgt_v[0])]

    def fresh(controls):
        for t, v in state:
            t.copy_(v)
        for t, v in zip(held, on_gpu(*controls)):
            t.copy_(v)
        for f in ("target_probs", "target_argmax", "accept_len", "path", "final_token", "tok_commit"):
            getattr(rd, f).zero_()
    eager = []
    for controls in filters:
        fresh(controls)
        gpu = round_on(eng, rd, w_c, inp, base)
        check_cut_round(rd, gpu, Wd, controls)
        eager.append(gpu)
    fresh(filters[0])
    pre, post = rd.capture_segments(w_c)
    for i in (0, 1, 1, 0):
        fresh(filters[i])
        pre.replay()
        standin(inp)(rd)
        post.replay()
        torch.cuda.synchronize()
        used = torch.arange(rd.S) < rd.t_size.cpu()[:, None]
        for f in ("target_probs", "target_argmax"):
            assert torch.equal(getattr(rd, f).cpu()[used], eager[i][f][used]), f
        for f in ("accept_len", "path", "final_token", "last_slot", "tok_commit", "t_next_out", "prefix_len_out"):
            assert torch.equal(getattr(rd, f).cpu(), eager[i][f]), f
    assert eng.status() == 0
    eng.close()
