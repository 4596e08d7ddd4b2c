"""A dense layer end to end, as a model runs it: norm and rotation of the projections'
slices, causal attention over the prompt, the cache it leaves behind, a tree of drafted
tokens over that cache; and the layer's training step, gradients down to the projection."""
import numpy as np
import pytest
import torch

from block_sparse_gqa_04_b200 import msa
from oracle import dense_oracle as D
from tests.dense_util import randn

pytestmark = pytest.mark.gpu

HQ, HKV, DIM, EPS = 8, 2, 128, 1e-6


def _weights():
    w = [1 + 0.2 * randn((DIM,), torch.float32, s) for s in (1, 2)]
    f = 1e4 ** (-torch.arange(DIM // 2, dtype=torch.float64, device="cuda") / (DIM // 2))
    return w[0], w[1], f


def _split(qkv):
    q, k, v = qkv.split((HQ * DIM, HKV * DIM, HKV * DIM), -1)
    return tuple(x.unflatten(-1, (-1, DIM)) for x in (q, k, v))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
def test_prompt_then_drafts_over_pages(dtype):
    """The drafted tokens' rows equal the same rows of one causal pass over everything."""
    n, m, b = 200, 6, 2
    qw, kw, f = _weights()
    qw, kw = qw.to(dtype), kw.to(dtype)
    qkv = randn((b, n + m, (HQ + 2 * HKV) * DIM), dtype, 3)
    q, k, v = _split(qkv)
    pos = torch.arange(n + m, device="cuda").expand(b, -1).contiguous()
    qr, kr = msa.qk_norm_rope(q, k, qw, kw, f, pos, eps=EPS)
    v = v.contiguous()
    whole, lse = msa.dense_attend(qr, kr, v, return_lse=True)
    # the prompt alone, then its keys and values into pages
    first = msa.dense_attend(qr[:, :n].contiguous(), kr[:, :n].contiguous(),
                             v[:, :n].contiguous())
    w = -(-(n + m) // 128)
    table = torch.tensor([[2, 0], [3, 1]], dtype=torch.int32, device="cuda")
    pk, pv = (torch.zeros((4, 128, HKV, DIM), dtype=dtype, device="cuda") for _ in range(2))
    for i in range(b):
        for c in range(w):
            rows = slice(128 * c, min(128 * (c + 1), n + m))
            pk[table[i, c], :rows.stop - rows.start] = kr[i, rows]
            pv[table[i, c], :rows.stop - rows.start] = v[i, rows]
    lens = torch.full((b,), n, dtype=torch.int32, device="cuda")
    chain = torch.ones((m, m), dtype=torch.bool, device="cuda").tril()
    out, z = msa.tree_attend(qr[:, n:].contiguous(), pk, pv, chain, lens, return_lse=True,
                             block_table=table, kv_len=n + m)
    # two roundings of the result apart, and of the weights (bf16)
    tol = 1e-5 if dtype == torch.float32 else 4 * 2.0 ** -8
    scale = whole.float().abs().max()
    assert (first.float() - whole[:, :n].float()).abs().max() <= tol * scale
    assert (out.float() - whole[:, n:].float()).abs().max() <= tol * scale
    assert (z - lse[:, n:]).abs().max() <= 1e-5 * lse.abs().max()


def test_training_step_of_packed_documents():
    """Gradients of sum(out * g) with respect to the projection and the norm weights,
    through both backward passes, against fp64 autograd."""
    lens = [70, 1, 131]
    cu = np.cumsum([0] + lens).tolist()
    qw, kw, f = _weights()
    qkv = randn((cu[-1], (HQ + 2 * HKV) * DIM), torch.float32, 5)
    g = randn((cu[-1], HQ, DIM), torch.float32, 6)
    pos = torch.cat([torch.arange(n, device="cuda") for n in lens])
    q, k, v = _split(qkv)
    v = v.contiguous()
    qr, kr = msa.qk_norm_rope(q, k, qw, kw, f, pos, eps=EPS, interleaved=True)
    out, lse = msa.dense_attend_varlen(qr, kr, v, cu, cu, return_lse=True)
    dqr, dkr, dv = msa.dense_backward_varlen(g, qr, kr, v, out, lse, cu, cu)
    dq, dk, dqw, dkw = msa.qk_norm_rope_backward(dqr, dkr, q, k, qw, kw, f, pos, eps=EPS,
                                                 interleaved=True)

    leaves = [x.double().requires_grad_() for x in (qkv, qw, kw)]
    a, b, c = _split(leaves[0])
    turn = torch.polar(torch.ones_like(f), f) ** pos.double()[:, None]

    def heads(x, w):
        y = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w
        z = torch.view_as_complex(y.unflatten(-1, (-1, 2)).contiguous()) * turn[:, None]
        return torch.view_as_real(z).flatten(-2)

    a, b = heads(a, leaves[1]), heads(b, leaves[2])
    o = []
    for i, n in enumerate(lens):
        s = slice(cu[i], cu[i + 1])
        kk, vv = (x[s].repeat_interleave(HQ // HKV, 1) for x in (b, c))
        z = torch.einsum("ihd,jhd->hij", a[s], kk) * DIM ** -0.5
        z = z.masked_fill(~torch.ones(n, n, dtype=torch.bool, device="cuda").tril(), -torch.inf)
        o.append(torch.einsum("hij,jhd->ihd", z.softmax(-1), vv))
    torch.cat(o).backward(g.double())
    got = torch.cat([x.flatten(1) for x in (dq, dk, dv)], 1)
    for name, x, want in (("projection", got, leaves[0].grad), ("q_weight", dqw, leaves[1].grad),
                          ("k_weight", dkw, leaves[2].grad)):
        err = (x.double() - want).norm() / want.norm()
        assert err < 1e-5, (name, float(err))


def test_gradients_against_differences_of_the_kernels_own_outputs():
    """Directional differences of the fp32 forward pass, over all of q, k and v."""
    n = 40
    q, k, v = (randn((1, n, h, 64), torch.float32, s) for h, s in ((4, 1), (2, 2), (2, 3)))
    g = randn((1, n, 4, 64), torch.float32, 4)
    out, lse = msa.dense_attend(q, k, v, return_lse=True)
    grads = msa.dense_backward(g, q, k, v, out, lse)
    h = 2.0 ** -6
    for i, seed in ((0, 7), (1, 8), (2, 9)):
        e = randn((q, k, v)[i].shape, torch.float32, seed)
        side = []
        for sign in (1, -1):
            x = [q, k, v]
            x[i] = x[i] + sign * h * e
            side.append((msa.dense_attend(*x).double() * g.double()).sum())
        slope = float(side[0] - side[1]) / (2 * h)
        want = float((grads[i].double() * e.double()).sum())
        # h^2 / 6 times the third derivative (bounded here by the oracle's own difference
        # below) and the outputs' rounding over 2 h
        ref = []
        for sign in (1, -1):
            x = [t[0].double().cpu().numpy() for t in (q, k, v)]
            x[i] = x[i] + sign * h * e[0].double().cpu().numpy()
            ref.append((D.dense_attend(*x, 0)["out"] * g[0].double().cpu().numpy()).sum())
        exact = (ref[0] - ref[1]) / (2 * h)
        noise = 2.0 ** -20 * float((out.abs() * g.abs()).sum()) / h
        assert abs(slope - exact) <= noise
        assert abs(want - slope) <= abs(want - exact) + noise
        assert abs(want - exact) <= 0.02 * abs(want) + 1e-3 * float((grads[i].abs() * e.abs()).sum())
