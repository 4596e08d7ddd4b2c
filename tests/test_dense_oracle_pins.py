"""Pins of the fp64 oracle of the dense operators: against torch's own fp64 softmax and
autograd, against finite differences, and on hand-made cases."""
import numpy as np
import pytest
import torch

from oracle import dense_oracle as D
from oracle import msa_oracle as O


def _rand(rng, *shape):
    return rng.standard_normal(shape)


@pytest.mark.parametrize("n,m,hq,hkv", [(1, 1, 2, 1), (5, 9, 4, 2), (7, 7, 3, 3), (4, 6, 6, 2)])
def test_dense_matches_the_sparse_oracles_dense_form(n, m, hq, hkv):
    rng = np.random.default_rng(1)
    q, k, v = _rand(rng, n, hq, 8), _rand(rng, m, hkv, 8), _rand(rng, m, hkv, 8)
    got = D.dense_attend(q, k, v, m - n)
    want = O.dense_causal_gqa(q[None], k[None], v[None], m - n)
    want = want[0] if isinstance(want, tuple) else want
    np.testing.assert_allclose(got["out"], np.asarray(want).reshape(n, hq, 8), atol=1e-12)


def test_dense_gradients_match_autograd_and_differences():
    rng = np.random.default_rng(2)
    n, m, hq, hkv, d = 4, 7, 4, 2, 6
    x = {"q": _rand(rng, n, hq, d), "k": _rand(rng, m, hkv, d), "v": _rand(rng, m, hkv, d)}
    g = _rand(rng, n, hq, d)
    r = D.dense_attend(x["q"], x["k"], x["v"], m - n, 0.3, dout=g)
    t = {a: torch.tensor(b, requires_grad=True) for a, b in x.items()}
    kk, vv = (t[a].repeat_interleave(hq // hkv, 1) for a in ("k", "v"))
    s = torch.einsum("ihd,jhd->hij", t["q"], kk) * 0.3
    s = s.masked_fill(~torch.ones(n, m, dtype=torch.bool).tril(m - n), -torch.inf)
    o = torch.einsum("hij,jhd->ihd", s.softmax(-1), vv)
    o.backward(torch.tensor(g))
    np.testing.assert_allclose(r["out"], o.detach().numpy(), atol=1e-13)
    np.testing.assert_allclose(r["lse"], torch.logsumexp(s, -1).detach().numpy().T, atol=1e-13)
    for a in "qkv":
        np.testing.assert_allclose(r["d" + a], t[a].grad.numpy(), atol=1e-12)
        e = _rand(rng, *x[a].shape)
        h = 1e-6
        f = [float((D.dense_attend(**{**{"q": x["q"], "k": x["k"], "v": x["v"]},
                                      a: x[a] + sgn * h * e}, pos0=m - n, scale=0.3)["out"]
                    * g).sum()) for sgn in (1, -1)]
        assert abs((f[0] - f[1]) / (2 * h) - float((r["d" + a] * e).sum())) < 1e-7


def test_tree_chain_equals_causal_and_empty_rows():
    rng = np.random.default_rng(3)
    n, kept, hq, hkv, d = 3, 5, 4, 2, 8
    q, k, v = _rand(rng, n, hq, d), _rand(rng, kept + n, hkv, d), _rand(rng, kept + n, hkv, d)
    chain = np.tril(np.ones((n, n), bool))
    a, b = D.tree_attend(q, k, v, chain, kept), D.dense_attend(q, k, v, kept)
    np.testing.assert_allclose(a["out"], b["out"], atol=1e-14)
    np.testing.assert_allclose(a["lse"], b["lse"], atol=1e-14)
    # nothing cached, nothing seen; an unseen row may hold anything
    v[2] = np.nan
    e = D.tree_attend(q, k, v, np.array([[1, 0, 0], [0, 0, 0], [1, 1, 0]], bool), 0)
    assert (e["out"][1] == 0).all() and np.isneginf(e["lse"][1]).all()
    np.testing.assert_allclose(e["out"][0], np.repeat(v[0], 2, 0))
    assert np.isfinite(e["out"]).all() and np.isfinite(e["out_mag"]).all()


@pytest.mark.parametrize("inter", [False, True])
def test_norm_rope_by_hand_and_by_autograd(inter):
    # one pair, a quarter turn: (a, b) -> (-b, a); a norm of 5 / sqrt(2)
    y = D.norm_rope(np.array([[[3.0, 4.0]]]), [1.0, 1.0], [np.pi / 2], [1], 0.0, inter)
    np.testing.assert_allclose(y[0, 0], np.array([-4.0, 3.0]) * np.sqrt(2) / 5, atol=1e-15)
    rng = np.random.default_rng(4)
    x, w, dy = _rand(rng, 6, 3, 8), _rand(rng, 8), _rand(rng, 6, 3, 8)
    f, pos = np.array([1.0, 0.25, 1e-3]), np.array([0, 1, 5, 100, 10 ** 6, -7])
    dx, dw, mag = D.norm_rope_backward(dy, x, w, f, pos, 1e-5, inter)
    assert (mag >= np.abs(dw)).all()
    for k in range(5):
        ex, ew, h = _rand(rng, 6, 3, 8), _rand(rng, 8), 1e-6
        v = [float((D.norm_rope(x + s * h * ex, w + s * h * ew, f, pos, 1e-5, inter) * dy).sum())
             for s in (1, -1)]
        assert abs((v[0] - v[1]) / (2 * h) - float((dx * ex).sum() + (dw * ew).sum())) < 1e-7
    # rotations keep lengths and undo each other
    r = D.rotate(x, pos, f, inter)
    np.testing.assert_allclose((r ** 2).sum(-1), (x ** 2).sum(-1))
    np.testing.assert_allclose(D.rotate(r, pos, f, inter, back=True), x, atol=1e-12)
