"""Gradients of dense attention where the tensor-core passes exchange or complete sums:
items of a single key tile, values that are not finite, keys that a call does not hold."""
import numpy as np
import pytest
import torch

from block_sparse_gqa_04_b200 import msa
from tests.dense_util import check_sequence, randn

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
