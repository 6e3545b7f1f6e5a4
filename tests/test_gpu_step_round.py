"""A round whose target distribution is cut by top-k, top-p and min-p (Round.set_filter): eagle_sample's distributions go into
the acceptance walk, and the committed tokens follow the cut distribution (the draft's own, q, stays whole)."""
import numpy as np
import pytest
import torch
from scipy.stats import chisquare

from eagle_feature_level_gb300 import _binding as B
from eagle_feature_level_gb300 import runtime as R
from oracle import step as O

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
