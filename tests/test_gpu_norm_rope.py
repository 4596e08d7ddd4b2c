"""Norm and rotation of heads (msa_qk_norm_rope) and its gradients against the fp64
oracle.

Bounds, with u half a step of the stored type relative to the value: a result is formed
in fp32 from sums of D squares (D / 2 + 8 steps of 2^-24 at most under the square root
and in the products) and cosines off by less than 2^-21, and rounded once; a rotated
element is the difference of two products of size at most the pair's length.
    |y err| <= u |y| + (D + 32) 2^-24 (|a| + |b|),  a, b the pair before the rotation
    |dx err| <= u |dx| + (D + 32) 2^-23 r max|w g|_row sqrt(D)
(the second term of dx, u mean(t u), is at most max|t| sqrt(D) since mean(u^2) <= 1), and
dw adds n terms of at most that relative error: (D + 32 + 64) 2^-23 dw_mag, its sums being
of at most 64 partial sums in a row in fp32 and in fp64 after that for these sizes.
"""
import numpy as np
import pytest
import torch

from block_sparse_gqa_04_b200 import msa
from oracle import dense_oracle as O
from tests.dense_util import U, np64, randn

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


def _freqs(rotary, theta=1e6):
    half = rotary // 2
    return theta ** (-torch.arange(half, dtype=torch.float64, device="cuda") / max(half, 1))


def _check_out(got, x, w, f, pos, eps, inter):
    d, dt = x.shape[-1], x.dtype
    xs, ws, fs, ps = np64(x), np64(w), np64(f), pos.cpu().numpy()
    want = O.norm_rope(xs, ws, fs, ps, eps, inter)
    y = np.abs(O.norm_rope(xs, ws, [], ps, eps, inter))
    half = len(fs)
    pair = y.copy()
    for i in range(half):
        a, b = (2 * i, 2 * i + 1) if inter else (i, i + half)
        pair[..., a] = pair[..., b] = y[..., a] + y[..., b]
    bound = U[dt] * np.abs(want) + (d + 32) * 2.0 ** -24 * pair + 1e-30
    err = np.abs(np64(got) - want)
    assert (err <= bound).all(), float((err / bound).max())


def _check_grads(dx, dw, dy, x, w, f, pos, eps, inter):
    d, dt = x.shape[-1], x.dtype
    xs, ws, fs, ps, gs = np64(x), np64(w), np64(f), pos.cpu().numpy(), np64(dy)
    want, dw_want, mag = O.norm_rope_backward(gs, xs, ws, fs, ps, eps, inter)
    g = O.rotate(gs, ps, fs, inter, back=True)
    r = 1 / np.sqrt((xs * xs).mean(-1, keepdims=True) + eps)
    # a turned-back element is as exact as its pair is long
    t = np.abs(ws).max() * np.abs(g).max(-1, keepdims=True) * 2 ** 0.5
    bound = U[dt] * np.abs(want) + (d + 32) * 2.0 ** -23 * r * t * d ** 0.5 + 1e-30
    err = np.abs(np64(dx) - want)
    assert (err <= bound).all(), float((err / bound).max())
    # elements of a pair share their error: the row's largest magnitude bounds it
    wb = (d + 96) * 2.0 ** -23 * (mag + mag.max()) + 1e-30
    assert (np.abs(np64(dw) - dw_want) <= wb).all()


# rows, q heads, kv heads, D, rotary, interleaved
CASES = [
    (1, 1, 1, 32, 32, False),
    (5, 64, 4, 128, 128, False),
    (33, 8, 2, 64, 32, True),
    (7, 3, 1, 128, 96, False),
    (7, 3, 1, 128, 96, True),
    (130, 5, 5, 32, 16, False),
    (2, 16, 2, 64, 0, False),
    (1500, 4, 2, 64, 64, False),     # several tokens per block
    (1201, 6, 1, 128, 64, True),
]


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("rows,hq,hkv,d,rot,inter", CASES)
def test_matches_oracle(rows, hq, hkv, d, rot, inter, dtype):
    eps = 1e-5
    # slices of one projection's output
    qkv = randn((rows, (hq + 2 * hkv) * d), dtype, 1, 2.0)
    q = qkv[:, :hq * d].unflatten(1, (hq, d))
    k = qkv[:, hq * d:(hq + hkv) * d].unflatten(1, (hkv, d))
    qw, kw = (1 + 0.3 * randn((d,), F32, s) for s in (2, 3))
    qw, kw = qw.to(dtype), kw.to(dtype)
    f = _freqs(rot)
    pos = torch.randint(-5, 1 << 20, (rows,), device="cuda")
    pos[0] = 0
    qo, ko = msa.qk_norm_rope(q, k, qw, kw, f, pos, eps=eps, interleaved=inter)
    assert qo.is_contiguous() and ko.is_contiguous()
    _check_out(qo, q, qw, f, pos, eps, inter)
    _check_out(ko, k, kw, f, pos, eps, inter)
    dqo, dko = randn((rows, hq, d), dtype, 4), randn((rows, hkv, d), dtype, 5)
    dq, dk, dqw, dkw = msa.qk_norm_rope_backward(dqo, dko, q, k, qw, kw, f, pos, eps=eps,
                                                 interleaved=inter)
    _check_grads(dq, dqw, dqo, q, qw, f, pos, eps, inter)
    _check_grads(dk, dkw, dko, k, kw, f, pos, eps, inter)
    again = msa.qk_norm_rope_backward(dqo, dko, q, k, qw, kw, f, pos, eps=eps, interleaved=inter)
    assert all(torch.equal(a, b) for a, b in zip((dq, dk, dqw, dkw), again))


@pytest.mark.parametrize("shape", [(2, 17), (6,)])
def test_in_place_and_batched_slices(shape):
    """In place in the fused buffer, the value slice untouched; queries alone."""
    hq, hkv, d = 8, 2, 128
    qkv = randn(shape + ((hq + 2 * hkv) * d,), BF16, 1)
    before = qkv.clone()
    q = qkv[..., :hq * d].unflatten(-1, (hq, d))
    k = qkv[..., hq * d:(hq + hkv) * d].unflatten(-1, (hkv, d))
    w, f = torch.ones(d, dtype=BF16, device="cuda"), _freqs(d)
    pos = torch.arange(q.shape[:-2].numel(), device="cuda").view(shape)
    want = msa.qk_norm_rope(q, k, w, w, f, pos)
    alone, none = msa.qk_norm_rope(q, None, w, None, f, pos)
    assert none is None and torch.equal(alone, want[0])
    got = msa.qk_norm_rope(q, k, w, w, f, pos, out=(q, k))
    assert got[0].data_ptr() == q.data_ptr()
    assert torch.equal(q, want[0]) and torch.equal(k, want[1])
    assert torch.equal(qkv[..., (hq + hkv) * d:], before[..., (hq + hkv) * d:])


def test_far_positions_keep_their_angles():
    """Angles of 10^9 radians against fp64: only the fp32 cosine's error is left."""
    d = 64
    q = torch.zeros((4, 1, d), device="cuda")
    q[..., :d // 2] = 1.0   # pairs (1, 0): the result is (cos, sin)
    w = torch.ones(d, device="cuda")
    pos = torch.tensor([1, 10 ** 6 + 1, 10 ** 9 + 7, -10 ** 9], device="cuda")
    f = _freqs(d)
    out, _ = msa.qk_norm_rope(q, None, w, None, f, pos, eps=0.0)
    ang = pos.double()[:, None] * f
    want = torch.cat((ang.cos(), ang.sin()), 1) * 2 ** 0.5
    # the product itself is off by 2^-53 10^9 in both
    assert (out[:, 0].double() - want).abs().max() < 2e-6


def test_rows_of_zeros_and_infinities_stay_in_their_rows():
    q = randn((6, 4, 64), BF16, 1)
    w, f = torch.ones(64, dtype=BF16, device="cuda"), _freqs(64)
    pos = torch.arange(6, device="cuda")
    want, _ = msa.qk_norm_rope(q, None, w, None, f, pos)
    q[1], q[2, 1], q[3, 0] = 0.0, float("inf"), float("nan")
    got, _ = msa.qk_norm_rope(q, None, w, None, f, pos)
    keep = torch.ones((6, 4), dtype=torch.bool, device="cuda")
    keep[1], keep[2, 1], keep[3, 0] = False, False, False
    assert torch.equal(got[keep], want[keep])
    assert not got[1].any() and got[3, 0].isnan().all()


def test_no_rows():
    q = torch.empty((0, 4, 64), dtype=BF16, device="cuda")
    w, f = torch.ones(64, dtype=BF16, device="cuda"), _freqs(64)
    pos = torch.empty(0, dtype=torch.int64, device="cuda")
    qo, ko = msa.qk_norm_rope(q, q, w, w, f, pos)
    assert qo.shape == q.shape
    dq, dk, dqw, dkw = msa.qk_norm_rope_backward(q, q, q, q, w, w, f, pos)
    assert dq.numel() == 0 and not dqw.any() and not dkw.any()


def test_captured_and_replayed():
    q, k = randn((40, 8, 128), BF16, 1), randn((40, 2, 128), BF16, 2)
    w, f = torch.ones(128, dtype=BF16, device="cuda"), _freqs(128)
    pos = torch.arange(40, device="cuda")
    msa.qk_norm_rope(q, k, w, w, f, pos)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = msa.qk_norm_rope(q, k, w, w, f, pos)
        grads = msa.qk_norm_rope_backward(*out, q, k, w, w, f, pos)
    pos += 1000
    q.copy_(randn((40, 8, 128), BF16, 9))
    g.replay()
    want = msa.qk_norm_rope(q, k, w, w, f, pos)
    want += msa.qk_norm_rope_backward(*want, q, k, w, w, f, pos)
    assert all(torch.equal(a, b) for a, b in zip(out + grads, want))


def test_rows_behind_32_bits_of_elements():
    rows, hq, d = 300000, 64, 128
    q = torch.zeros((rows, hq, d), dtype=BF16, device="cuda")
    assert q.numel() > 1 << 31
    q[-5:] = randn((5, hq, d), BF16, 1)
    w, f = torch.ones(d, dtype=BF16, device="cuda"), _freqs(d)
    pos = torch.arange(rows, device="cuda")
    out, _ = msa.qk_norm_rope(q, None, w, None, f, pos)
    want, _ = msa.qk_norm_rope(q[-5:], None, w, None, f, pos[-5:])
    assert torch.equal(out[-5:], want) and not out[:-5].any()
    del out
    g = torch.zeros_like(q)
    g[-5:] = randn((5, hq, d), BF16, 2)
    dq, _, dw, _ = msa.qk_norm_rope_backward(g, None, q, None, w, None, f, pos)
    want, _, dw1, _ = msa.qk_norm_rope_backward(g[-5:], None, q[-5:], None, w, None, f, pos[-5:])
    assert torch.equal(dq[-5:], want) and not dq[:-5].any()
    # the same 320 addends per weight, in another order
    assert (dw - dw1).abs().max() <= 320 * 2.0 ** -23 * dw1.abs().max() + 1e-4


def test_refusals():
    q, k = randn((6, 4, 64), BF16, 1), randn((6, 2, 64), BF16, 2)
    w, f = torch.ones(64, dtype=BF16, device="cuda"), _freqs(64)
    pos = torch.arange(6, device="cuda")
    buf = randn((6, 8, 64), BF16, 3)
    bad = [lambda: msa.qk_norm_rope(q, k, w, None, f, pos),
           lambda: msa.qk_norm_rope(q, k, w, w, f.float(), pos),
           lambda: msa.qk_norm_rope(q, k, w, w, f, pos.int()),
           lambda: msa.qk_norm_rope(q, k, w, w, f, pos[:5]),
           lambda: msa.qk_norm_rope(q, k, w.float(), w, f, pos),
           lambda: msa.qk_norm_rope(q, k[:5], w, w, f, pos),
           lambda: msa.qk_norm_rope(q.transpose(0, 1), k, w, w, f, pos),
           lambda: msa.qk_norm_rope(q, k, w, w, f[:12], pos),                  # rotary 24
           lambda: msa.qk_norm_rope(q, k, w, w, f, pos, eps=-1.0),
           lambda: msa.qk_norm_rope(q, k, w, w, f, pos, out=(buf[:, :4], buf[:, 3:5])),
           lambda: msa.qk_norm_rope(buf[:, :4], k, w, w, f, pos, out=(buf[:, 1:5], k)),
           lambda: msa.qk_norm_rope(q.cpu(), k, w, w, f, pos)]
    for call in bad:
        with pytest.raises((ValueError, msa.MsaError)):
            call()


@pytest.mark.parametrize("rows", [1185, 1215, 5003])
@pytest.mark.parametrize("interleaved", [False, True])
def test_weight_gradients_do_not_depend_on_what_shared_memory_held(rows, interleaved):
    """A block's tokens behind the last row add nothing.  The call before, attention over NaN,
    leaves NaN in the shared memory of every SM."""
    hq, hkv, d = 32, 2, 128
    q, k = randn((rows, hq, d), BF16, 50), randn((rows, hkv, d), BF16, 51)
    gq, gk = randn((rows, hq, d), BF16, 52), randn((rows, hkv, d), BF16, 53)
    w, f = torch.ones(d, dtype=BF16, device="cuda"), _freqs(d)
    pos = torch.arange(rows, device="cuda")
    args = (gq, gk, q, k, w, w, f, pos)
    want = msa.qk_norm_rope_backward(*args, interleaved=interleaved)
    nan = torch.full((8, 1024, 8, 128), float("nan"), device="cuda")
    for _ in range(5):
        msa.dense_attend(nan, nan, nan)
        got = msa.qk_norm_rope_backward(*args, interleaved=interleaved)
        assert all(torch.equal(a, b) for a, b in zip(want, got))
        assert all(x.isfinite().all() for x in got)
