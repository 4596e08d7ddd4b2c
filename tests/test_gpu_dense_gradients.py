"""Gradients of dense attention where the tensor-core passes exchange or complete sums:
items of a single key tile, values that are not finite, keys that a call does not hold."""
import numpy as np
import pytest
import torch

from block_sparse_gqa_04_b200 import msa
from oracle import dense_oracle
from tests.dense_util import U, check_sequence, close, np64, randn, weight_error

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


@pytest.mark.parametrize("d,hq,hkv", [(64, 8, 2), (128, 8, 8)])
def test_many_documents_of_one_key_tile(d, hq, hkv):
    """Every item of the dq pass has one key tile: its sums follow one another at the
    shortest distance.  The same bits each time, and sampled documents against the oracle."""
    lens = [1 + (37 * i) % 128 for i in range(600)]
    cu = np.cumsum([0] + lens).tolist()
    q, dout = (randn((cu[-1], hq, d), BF16, 60 + i) for i in range(2))
    k, v = (randn((cu[-1], hkv, d), BF16, 62 + i) for i in range(2))
    out, lse = msa.dense_attend_varlen(q, k, v, cu, cu, return_lse=True)
    want = msa.dense_backward_varlen(dout, q, k, v, out, lse, cu, cu, check_device_status=True)
    for _ in range(20):
        got = msa.dense_backward_varlen(dout, q, k, v, out, lse, cu, cu, check_device_status=True)
        assert all(torch.equal(a, b) for a, b in zip(want, got))
    for i in (0, 1, 38, 299, 599):
        s = slice(cu[i], cu[i + 1])
        check_sequence(q[s], k[s], v[s], out[s], lse[s], 0, dout=dout[s],
                       grads=[x[s] for x in want], name=f"document {i}: ")


@pytest.mark.parametrize("dtype", [BF16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("what", ["q", "lse"])
def test_nan_of_a_row_reaches_the_values_it_sees(what, dtype):
    """Whatever the row's place in its tile: 16 documents of 16 rows, NaN in row i of
    document i.  dv of the keys that it sees is NaN, that of the others as without it."""
    n, docs, hq, hkv, d = 16, 16, 4, 2, 128
    cu = [n * i for i in range(docs + 1)]
    q, dout = (randn((n * docs, hq, d), dtype, 70 + i) for i in range(2))
    k, v = (randn((n * docs, hkv, d), dtype, 72 + i) for i in range(2))
    out, lse = msa.dense_attend_varlen(q, k, v, cu, cu, return_lse=True)
    clean = msa.dense_backward_varlen(dout, q, k, v, out, lse, cu, cu)[2]
    rows = torch.arange(docs, device="cuda") * (n + 1)
    if what == "q":
        q[rows] = float("nan")
        out, lse = msa.dense_attend_varlen(q, k, v, cu, cu, return_lse=True)
        assert lse[rows].isnan().all() and out[rows].isnan().all()
    else:
        lse[rows] = float("nan")
    dv = msa.dense_backward_varlen(dout, q, k, v, out, lse, cu, cu, check_device_status=True)[2]
    row = torch.arange(n, device="cuda")
    sees = row[None] <= row[:, None]                       # key j of document i: j <= i
    dv, clean = dv.view(docs, n, hkv, d), clean.view(docs, n, hkv, d)
    assert dv[sees].isnan().all()
    assert torch.equal(dv[~sees], clean[~sees])


@pytest.mark.parametrize("share", [8e-4, 2e-4, 5e-5, 5e-6, 1e-7])
@pytest.mark.parametrize("d", [64, 128])
def test_keys_elsewhere_that_hold_little_of_a_row(d, share):
    """Out and lse are of one more key, which another rank holds: `share` of every row's
    weight and a value of about 1 / share.  This call's P sums to 1 - share, which fp32 does
    not tell from 1 in the end, and delta is mostly that key's.  The bound is the dk bound
    of dense_util with the other key's part of out in its magnitudes."""
    n, hq, hkv, dt = 96, 4, 2, BF16
    q, dout = (randn((1, n, hq, d), dt, 80 + i).abs() for i in range(2))
    k, v = (randn((1, n, hkv, d), dt, 82 + i) for i in range(2))
    far = 1000 * 2.0 ** -10 / share
    r = dense_oracle.dense_attend(q[0], k[0], v[0], 0, dout=dout[0])
    out64, lse64 = (1 - share) * r["out"] + share * far, r["lse"] - np.log1p(-share)
    out = torch.tensor(out64, device="cuda").to(dt)[None].contiguous()
    lse = torch.tensor(lse64, device="cuda", dtype=torch.float32)[None].contiguous()
    dk = msa.dense_backward(dout, q, k, v, out, lse, check_device_status=True)[1]
    q_, k_, v_, do = (np64(x[0]) for x in (q, k, v, dout))
    want, mag, wide = np.zeros((n, hkv, d)), np.zeros((n, hkv, d)), np.zeros((n, hkv, d))
    for h in range(hq):
        c = h // (hq // hkv)
        s = np.where(np.tril(np.ones((n, n), bool)), q_[:, h] @ k_[:, c].T * d ** -0.5, -np.inf)
        p = np.exp(s - lse64[:, h:h + 1])
        ds = p * (do[:, h] @ v_[:, c].T - (do[:, h] * out64[:, h]).sum(1, keepdims=True))
        size = (1 - share) * r["out_mag"][:, h] + share * far + np.abs(out64[:, h])
        w = p * (np.abs(do[:, h]) * size).sum(1, keepdims=True)
        want[:, c] += d ** -0.5 * ds.T @ q_[:, h]
        mag[:, c] += d ** -0.5 * (np.abs(ds) + w).T @ np.abs(q_[:, h])
        w = w + p * (np.abs(do[:, h]) @ np.abs(v_[:, c]).T)
        wide[:, c] += d ** -0.5 * (np.abs(ds) + w).T @ np.abs(q_[:, h])
    f = weight_error(q[0], k[0])
    close("dk", dk[0], want, U[dt] * (mag + np.abs(want)) + 4 * f * wide, dt)


@pytest.mark.parametrize("n,scale", [(64, None), (128, 4.0), (700, None), (4100, None), (700, 30.0)])
def test_delta_is_completed_where_all_keys_are_here(n, scale):
    """Values around 100: the rounding of out, up to a quarter, takes a tenth of what is left
    of dout . v - delta.  dk does not feel it: dS and the result are off by half a step of
    bf16 at most, 2^-8, and with the signs that they have by less than that in the 2-norm;
    sums of 128 products of 100 in fp32 by 2^-24 x 136 x 100 x 128^0.5 / 128^0.5 = 2^-10."""
    hq, hkv, d = 2, 1, 128
    q, dout = (randn((1, n, hq, d), BF16, 90 + i) for i in range(2))
    k, v = randn((1, n, hkv, d), BF16, 92), randn((1, n, hkv, d), BF16, 93, 8.0) + 100
    how = {} if scale is None else {"softmax_scale": scale * d ** -0.5}
    out, lse = msa.dense_attend(q, k, v, return_lse=True, **how)
    dk = msa.dense_backward(dout, q, k, v, out, lse, **how)[1]
    leaves = [x[0].double().requires_grad_() for x in (q, k, v)]
    s = torch.einsum("ihd,jd->hij", leaves[0], leaves[1][:, 0]) * (scale or 1.0) * d ** -0.5
    s = s.masked_fill(~torch.ones(n, n, dtype=torch.bool, device="cuda").tril(), -torch.inf)
    o = torch.einsum("hij,jd->ihd", s.softmax(-1), leaves[2][:, 0])
    o.backward(dout[0].double())
    err = float((dk[0].double() - leaves[1].grad).norm() / leaves[1].grad.norm())
    # what the rounding of out does to dk where nothing completes delta
    p = s.softmax(-1).detach()
    lost = (dout[0].double() * (out[0].double() - o.detach())).sum(-1).T[..., None] * p
    left = torch.einsum("hij,ihd->jd", lost, q[0].double()) * (scale or 1.0) * d ** -0.5
    lost = float(left.norm() / leaves[1].grad.norm())
    print(f"n {n} scale {scale}: error {err:.2e}, of the rounded out alone {lost:.2e}")
    assert err < 2.0 ** -8 + 2.0 ** -10 and lost > 2 * err
