"""Dense causal attention (msa_dense_attend) and its gradients (msa_dense_backward)
against the fp64 oracle, within the bounds derived in dense_util."""
import numpy as np
import pytest
import torch

from block_sparse_gqa_04_b200 import msa
from oracle import dense_oracle as D_
from tests.dense_util import U, check_grads, check_sequence, randn, weight_error

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


def _inputs(lead_q, lead_k, hq, hkv, d, dtype, seed=0):
    q, dout = (randn(lead_q + (hq, d), dtype, seed + i) for i in (0, 3))
    k, v = (randn(lead_k + (hkv, d), dtype, seed + i) for i in (1, 2))
    return q, k, v, dout


# batch, q_len, kv_len, q_pos0, q heads, kv heads, head_dim
BATCHED = [
    (1, 1, 1, 0, 2, 1, 64),
    (1, 1, 300, 299, 16, 1, 128),
    (2, 127, 127, 0, 4, 2, 64),
    (1, 128, 128, 0, 8, 8, 128),
    (1, 129, 129, 0, 6, 2, 128),
    (3, 65, 200, 100, 4, 4, 64),      # a chunk; keys behind its last row unseen
    (2, 257, 257, 0, 10, 2, 64),      # an odd number of heads per group
    (1, 300, 520, 220, 16, 1, 128),
    (1, 385, 640, 0, 3, 1, 128),      # whole key tiles that no row sees
    (2, 290, 341, 45, 3, 1, 64),      # pairs of tiles that end inside different key groups
    (1, 300, 555, 241, 5, 5, 128),
]


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("b,sq,skv,pos0,hq,hkv,d", BATCHED)
def test_batched(b, sq, skv, pos0, hq, hkv, d, dtype):
    q, k, v, dout = _inputs((b, sq), (b, skv), hq, hkv, d, dtype)
    out, lse = msa.dense_attend(q, k, v, q_pos0=pos0, return_lse=True, check_device_status=True)
    g = msa.dense_backward(dout, q, k, v, out, lse, q_pos0=pos0, check_device_status=True)
    for i in range(b):
        check_sequence(q[i], k[i], v[i], out[i], lse[i], pos0, dout=dout[i],
                       grads=[x[i] for x in g], name=f"sequence {i}: ")


PACKED = {
    "ragged": ([1, 130, 64, 200], [1, 130, 64, 200], 8, 2, 128),
    "last_rows": ([1, 5, 128, 40], [129, 5, 300, 255], 4, 4, 64),
    "empty_ones": ([0, 33, 0, 7, 0], [0, 33, 150, 7, 0], 6, 2, 64),
    "equal": ([96, 96, 96], [96, 96, 96], 16, 1, 128),
    "many": ([3] * 150, [4] * 150, 2, 1, 64),       # more than one launch's records
    "odd_groups": ([200, 131, 300], [233, 131, 411], 6, 2, 128),
    "one": ([260], [260], 12, 4, 128),
}


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("name", list(PACKED))
def test_packed(name, dtype):
    lq, lk, hq, hkv, d = PACKED[name]
    cq, ck = np.cumsum([0] + lq).tolist(), np.cumsum([0] + lk).tolist()
    q, k, v, dout = _inputs((cq[-1],), (ck[-1],), hq, hkv, d, dtype, seed=11)
    out, lse = msa.dense_attend_varlen(q, k, v, cq, ck, return_lse=True, check_device_status=True)
    dq, dk, dv = msa.dense_backward_varlen(dout, q, k, v, out, lse, cq, ck)
    for i in range(len(lq)):
        a, b = slice(cq[i], cq[i + 1]), slice(ck[i], ck[i + 1])
        if lq[i] == 0:
            assert not dk[b].any() and not dv[b].any()
            continue
        check_sequence(q[a], k[b], v[b], out[a], lse[a], lk[i] - lq[i], dout=dout[a],
                       grads=(dq[a], dk[b], dv[b]), name=f"sequence {i}: ")


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128])
def test_large_logits_rise_along_the_keys(d, dtype):
    """Every key tile raises the running maximum, by up to hundreds."""
    q, k, v, dout = _inputs((1, 300), (1, 700), 4, 2, d, dtype, seed=5)
    q = (q.float().abs() + 0.1).to(dtype)
    k = (k.float().abs() * torch.linspace(-1, 1, 700, device="cuda")[None, :, None, None]).to(dtype)
    out, lse = msa.dense_attend(q, k, v, q_pos0=400, softmax_scale=0.5, return_lse=True)
    g = msa.dense_backward(dout, q, k, v, out, lse, q_pos0=400, softmax_scale=0.5)
    check_sequence(q[0], k[0], v[0], out[0], lse[0], 400, 0.5, dout[0], [x[0] for x in g])


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_sequences_do_not_reach_one_another(bad, dtype):
    """NaN or infinity in every row of the neighbours leaves a sequence's results, and
    its gradients, as they are, bit for bit."""
    lens = [50, 77, 61]
    cu = np.cumsum([0] + lens).tolist()
    q, k, v, dout = _inputs((cu[-1],), (cu[-1],), 4, 2, 128, dtype, seed=7)
    clean = msa.dense_attend_varlen(q, k, v, cu, cu, return_lse=True)
    clean += msa.dense_backward_varlen(dout, q, k, v, *clean, cu, cu)
    mid = slice(cu[1], cu[2])
    for x in (q, k, v, dout):
        keep = x[mid].clone()
        x.fill_(bad)
        x[mid] = keep
    dirty = msa.dense_attend_varlen(q, k, v, cu, cu, return_lse=True)
    dirty += msa.dense_backward_varlen(dout, q, k, v, *dirty, cu, cu)
    for a, b in zip(clean, dirty):
        assert torch.equal(a[mid], b[mid])


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
def test_infinite_keys_of_hidden_tokens(dtype):
    """A hidden token's k may hold anything."""
    q, k, v, _ = _inputs((1, 40), (1, 200), 4, 2, 64, dtype, seed=9)
    want = msa.dense_attend(q, k, v, q_pos0=100, return_lse=True)
    k[:, 140:], v[:, 140:] = float("nan"), 3.0
    got = msa.dense_attend(q, k, v, q_pos0=100, return_lse=True)
    assert all(torch.equal(a, b) for a, b in zip(want, got))


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("sq,pos0,skv", [(40, 100, 200), (1, 0, 512), (129, 3, 133), (70, 58, 128)])
def test_tokens_that_no_row_sees_may_hold_anything(sq, pos0, skv, dtype):
    """A cache's rows behind the last query row: not written yet."""
    q, k, v, _ = _inputs((2, sq), (2, skv), 6, 2, 64, dtype, seed=11)
    want = msa.dense_attend(q, k, v, q_pos0=pos0, return_lse=True)
    k[:, pos0 + sq:], v[:, pos0 + sq:] = float("nan"), float("nan")
    got = msa.dense_attend(q, k, v, q_pos0=pos0, return_lse=True)
    assert all(torch.equal(a, b) for a, b in zip(want, got))


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("kv_len", [128, 200, 515])
def test_paged(kv_len, dtype):
    b, sq, hq, hkv, d = 2, 70, 8, 2, 128
    w = -(-kv_len // 128)
    q = randn((b, sq, hq, d), dtype, 1)
    k, v = randn((b, kv_len, hkv, d), dtype, 2), randn((b, kv_len, hkv, d), dtype, 3)
    want = msa.dense_attend(q, k, v, q_pos0=kv_len - sq, return_lse=True)
    # the rows of the last page behind the context hold whatever was there
    pk, pv = (torch.full((2 * w + 3, 128, hkv, d), float("nan"), dtype=dtype, device="cuda")
              for _ in range(2))
    table = torch.randperm(2 * w + 3)[:2 * w].view(2, w).to(torch.int32).cuda()
    for i in range(b):
        for c in range(w):
            n = min(128, kv_len - 128 * c)
            pk[table[i, c], :n] = k[i, 128 * c:128 * c + n]
            pv[table[i, c], :n] = v[i, 128 * c:128 * c + n]
    got = msa.dense_attend(q, pk, pv, q_pos0=kv_len - sq, return_lse=True, block_table=table,
                           kv_len=kv_len, check_device_status=True)
    assert all(torch.equal(x, y) for x, y in zip(want, got))
    table[0, 0] = 2 * w + 3
    with pytest.raises(msa.MsaError, match="MSA_ERR_DEVICE"):
        msa.dense_attend(q, pk, pv, q_pos0=kv_len - sq, block_table=table, kv_len=kv_len,
                         check_device_status=True)


@pytest.mark.parametrize("d,hq,hkv", [(128, 4, 1), (64, 3, 3)])
def test_long_sequence(d, hq, hkv):
    """Many tiles per row: against torch in fp64 on the device, sampled heads whole."""
    n = 2500
    q, k, v, dout = _inputs((1, n), (1, n), hq, hkv, d, BF16, seed=21)
    out, lse = msa.dense_attend(q, k, v, return_lse=True)
    dq, dk, dv = msa.dense_backward(dout, q, k, v, out, lse)
    leaves = [x[0].double().requires_grad_() for x in (q, k, v)]
    kk, vv = (x.repeat_interleave(hq // hkv, 1) for x in leaves[1:])
    s = torch.einsum("ihd,jhd->hij", leaves[0], kk) * d ** -0.5
    s = s.masked_fill(~torch.ones(n, n, dtype=torch.bool, device="cuda").tril(), -torch.inf)
    o = torch.einsum("hij,jhd->ihd", s.softmax(-1), vv)
    o.backward(dout[0].double())
    for name, got, want in (("out", out, o), ("dq", dq, leaves[0].grad), ("dk", dk, leaves[1].grad),
                            ("dv", dv, leaves[2].grad)):
        err = (got[0].double() - want).norm() / want.norm()
        # two or three independent roundings of bf16 (rms 0.42 of half a step each)
        assert err < 2.0 ** -8, (name, float(err))
    assert (lse[0].double() - torch.logsumexp(s, -1).T).abs().max() < 1e-5


def test_same_bits_again_on_other_streams_and_in_used_workspaces():
    lens = [300, 41, 190]
    cu = np.cumsum([0] + lens).tolist()
    q, k, v, dout = _inputs((cu[-1],), (cu[-1],), 8, 2, 128, BF16, seed=13)
    want = msa.dense_attend_varlen(q, k, v, cu, cu, return_lse=True)
    want += msa.dense_backward_varlen(dout, q, k, v, *want, cu, cu)
    torch.cuda.synchronize()
    ws = torch.full((1 << 25,), 0xff, dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(3):
            got = msa.dense_attend_varlen(q, k, v, cu, cu, return_lse=True, workspace=ws)
            got += msa.dense_backward_varlen(dout, q, k, v, *got, cu, cu, workspace=ws)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))


def test_rows_around_the_outputs_are_left_alone():
    for dtype in (BF16, F32):
        q, k, v, _ = _inputs((150,), (150,), 4, 2, 64, dtype, seed=17)
        buf = torch.full((190, 4, 64), 7.0, dtype=dtype, device="cuda")
        msa.dense_attend_varlen(q, k, v, [0, 20, 150], [0, 20, 150], out=buf[20:170])
        assert (buf[:20] == 7).all() and (buf[170:] == 7).all()


def test_captured_and_replayed():
    """A packed training step in a CUDA graph, replayed on new inputs; the prefix sums
    are part of the graph."""
    cu = [0, 100, 133, 400]
    q, k, v, dout = _inputs((400,), (400,), 8, 2, 128, BF16, seed=19)
    msa.dense_attend_varlen(q, k, v, cu, cu)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = msa.dense_attend_varlen(q, k, v, list(cu), cu, return_lse=True)
        got += msa.dense_backward_varlen(dout, q, k, v, *got, cu, cu)
    for seed in (1, 2):
        for x, y in zip((q, k, v, dout), _inputs((400,), (400,), 8, 2, 128, BF16, seed=seed)):
            x.copy_(y)
        g.replay()
        want = msa.dense_attend_varlen(q, k, v, cu, cu, return_lse=True)
        want += msa.dense_backward_varlen(dout, q, k, v, *want, cu, cu)
        assert all(torch.equal(a, b) for a, b in zip(want, got))


def test_nothing_to_do():
    q = torch.empty((2, 0, 4, 64), dtype=BF16, device="cuda")
    k = randn((2, 9, 2, 64), BF16, 0)
    out, lse = msa.dense_attend(q, k, k, return_lse=True)
    assert out.shape == q.shape and lse.shape == (2, 0, 4)
    dq, dk, dv = msa.dense_backward(q, q, k, k, out, lse)
    assert dq.numel() == 0 and not dk.any() and not dv.any()


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
def test_nothing_to_do_reports_no_error(dtype):
    """Whatever the workspace held before."""
    ws = torch.full((1 << 25,), 255, dtype=torch.uint8, device="cuda")
    how = dict(workspace=ws, check_device_status=True)
    q = torch.empty((2, 0, 4, 64), dtype=dtype, device="cuda")
    k = randn((2, 9, 2, 64), dtype, 0)
    out, lse = msa.dense_attend(q, k, k, return_lse=True, **how)
    ws.fill_(255)
    msa.dense_backward(q, q, k, k, out, lse, **how)
    ws.fill_(255)
    out, lse = msa.dense_attend_varlen(q[0], k[0], k[0], [0, 0, 0], [0, 4, 9], return_lse=True, **how)
    ws.fill_(255)
    msa.dense_backward_varlen(q[0], q[0], k[0], k[0], out, lse, [0, 0, 0], [0, 4, 9], **how)
    ws.fill_(255)
    msa.dense_backward_varlen(q[0], q[0], k[0, :0], k[0, :0], out, lse, [0, 0], [0, 0], **how)
    ws.fill_(255)
    msa.tree_attend(q, k, k, torch.ones((0, 0), dtype=torch.bool, device="cuda"),
                    torch.tensor([3, 9], dtype=torch.int32, device="cuda"), **how)


def test_rows_behind_32_bits_of_elements():
    """2100 prompts of 128 rows x 64 heads x 128: q, out and dq hold more than 2^31
    elements.  The last prompt's results equal those of a call on it alone, bit for bit
    (whatever else runs, a prompt's sums have one order)."""
    n, rows, hq, hkv, d = 2100, 128, 64, 4, 128
    total = n * rows
    cu = list(range(0, total + 1, rows))
    q, dout = (torch.zeros((total, hq, d), dtype=BF16, device="cuda") for _ in range(2))
    k, v = (torch.zeros((total, hkv, d), dtype=BF16, device="cuda") for _ in range(2))
    assert q.numel() > 1 << 31
    last = slice(total - rows, total)
    for i, t in enumerate((q, dout, k, v)):
        t[last] = randn((rows,) + t.shape[1:], BF16, 40 + i)
    out, lse = msa.dense_attend_varlen(q, k, v, cu, cu, return_lse=True, check_device_status=True)
    dq, dk, dv = msa.dense_backward_varlen(dout, q, k, v, out, lse, cu, cu)
    one = [x[last].contiguous() for x in (q, k, v, dout)]
    o1, l1 = msa.dense_attend_varlen(*one[:3], [0, rows], [0, rows], return_lse=True)
    g1 = msa.dense_backward_varlen(one[3], *one[:3], o1, l1, [0, rows], [0, rows])
    assert torch.equal(out[last], o1) and torch.equal(lse[last], l1)
    assert torch.equal(dq[last], g1[0])
    # dk and dv may be cut into other splits of the heads: the oracle's bounds
    check_sequence(*one[:3], out[last], lse[last], 0, dout=one[3],
                   grads=(dq[last], dk[last], dv[last]))
    assert not out[:total - rows].any() and not dq[:total - rows].any()


@pytest.mark.parametrize("d", [64, 128])
def test_two_streams_and_two_graphs_at_once(d):
    """Calls that run at the same time, each with its workspace, and two graphs that share
    one and are replayed in turn, give the bits of a call alone."""
    lens = [257, 40, 600]
    cu = np.cumsum([0] + lens).tolist()
    q, k, v, dout = _inputs((cu[-1],), (cu[-1],), 8, 2, d, BF16, seed=31)

    def step(ws=None):
        o = msa.dense_attend_varlen(q, k, v, cu, cu, return_lse=True, workspace=ws)
        return o + msa.dense_backward_varlen(dout, q, k, v, *o, cu, cu, workspace=ws)

    want = step()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    got = []
    for _ in range(4):
        for s in streams:
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):
                got.append(step())
    torch.cuda.synchronize()
    ws = torch.empty(1 << 25, dtype=torch.uint8, device="cuda")
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            got.append(step(ws))
        graphs.append(g)
    for g in graphs * 3:
        g.replay()
    torch.cuda.synchronize()
    for o in got:
        assert all(torch.equal(a, b) for a, b in zip(want, o))


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
def test_gradients_where_hidden_rows_hold_anything(dtype):
    """Keys that no row sees, and every key and value of them, may be NaN: dq does not
    meet them, and their own gradients are zero."""
    q, k, v, dout = _inputs((1, 70), (1, 300), 6, 2, 128, dtype, seed=23)
    o = msa.dense_attend(q, k, v, q_pos0=55, return_lse=True)
    want = msa.dense_backward(dout, q, k, v, *o, q_pos0=55)
    k[:, 125:], v[:, 125:] = float("nan"), float("nan")
    got = msa.dense_backward(dout, q, k, v, *o, q_pos0=55)
    assert torch.equal(got[0], want[0])
    for g, w in zip(got[1:], want[1:]):
        assert torch.equal(g[:, :125], w[:, :125]) and not g[:, 125:].any()


def test_attention_without_lse_and_into_a_given_output():
    q, k, v, _ = _inputs((2, 200), (2, 200), 4, 4, 64, BF16, seed=29)
    want, _ = msa.dense_attend(q, k, v, return_lse=True)
    out = torch.full_like(q, 3.0)
    assert msa.dense_attend(q, k, v, out=out) is out and torch.equal(out, want)


def test_refusals_leave_everything_as_it_was():
    q, k, v, dout = _inputs((1, 20), (1, 30), 4, 2, 64, BF16, seed=37)
    out = torch.full_like(q, 5.0)
    bad = [lambda: msa.dense_attend(q, k, v, q_pos0=11, out=out),        # behind the keys
           lambda: msa.dense_attend(q, k, v, q_pos0=-1, out=out),
           lambda: msa.dense_attend(q, k, v, softmax_scale=-1.0, out=out),
           lambda: msa.dense_attend(q, k, v, workspace=torch.empty(64, dtype=torch.uint8,
                                                                   device="cuda"), out=out),
           lambda: msa.dense_attend(q[..., :32].contiguous(), k[..., :32].contiguous(),
                                    v[..., :32].contiguous()),
           lambda: msa.dense_attend_varlen(q[0], k[0], v[0], [0, 20], [0, 19], out=out[0]),
           lambda: msa.dense_attend_varlen(q[0], k[0], v[0], [0, 30], [0, 30], out=out[0])]
    for call in bad:
        with pytest.raises((msa.MsaError, ValueError)):
            call()
    with pytest.raises(ValueError):
        msa.dense_attend(q, k.cpu(), v)
    with pytest.raises(ValueError):
        msa.dense_attend(q.transpose(1, 2), k, v)
    assert (out == 5).all()


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
def test_gradients_of_keys_in_two_parts(dtype):
    """Out and lse of all keys, dk and dv part by part (the first keys, then the rest, as
    ranks that hold a part of the keys each have them): a part's P does not sum to 1."""
    n, m, hq, hkv, d = 96, 256, 4, 2, 128
    q, k, v, dout = _inputs((1, n), (1, m + n), hq, hkv, d, dtype, seed=43)
    out, lse = msa.dense_attend(q, k, v, q_pos0=m, return_lse=True)
    dq, dk, dv = msa.dense_backward(dout, q, k, v, out, lse, q_pos0=m)
    # behind the first part keys of zeros, whose gradients are not looked at
    a = [x[:, :m].contiguous() for x in (k, v)]
    b = [x[:, m:].contiguous() for x in (k, v)]
    pad = [torch.cat((x, torch.zeros_like(x[:, :n])), 1) for x in a]
    first = msa.dense_backward(dout, q, *pad, out, lse, q_pos0=m)
    rest = msa.dense_backward(dout, q, *b, out, lse)
    r = D_.dense_attend(q[0], k[0], v[0], m, dout=dout[0])
    f, u = weight_error(q[0], k[0]), U[dtype]
    parts = torch.cat((first[1][:, :m], rest[1]), 1), torch.cat((first[2][:, :m], rest[2]), 1)
    # every key's gradient within the bounds of the whole call's (delta, of the rounded out,
    # is not completed for a part: the dk_p term)
    check_grads(dq[0], parts[0][0], parts[1][0], r, f, dtype)
    check_grads(dq[0], dk[0], dv[0], r, f, dtype)
