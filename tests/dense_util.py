"""Error bounds of the dense operators against their fp64 oracle.

u is half a step of the stored type (bf16 2^-8, fp32 2^-24, relative to the value) and
f the relative error that fp32 arithmetic leaves on a softmax weight: a score is a sum
of D products of stored values, off by at most (D + 8) 2^-24 A with A = scale max_ij
sum_d |q_d k_d|, it enters as the weight's own score and through the normaliser, sums
over m keys add m 2^-24, and the exponential and logarithm units a few steps more:
    f = 2^-24 (2 (D + 8) A + m + 64).
With the oracle's sums of magnitudes (X_mag and so on) every element then satisfies
    |out err| <= u (out_mag + |out|) + f out_mag      (weights rounded to the type, result too)
    |lse err| <= f + 2^-22 |lse|
    |dv err|  <= u (dv_mag + |dv|) + 2 f dv_mag
    |dq err|  <= u (dq_mag + |dq| + dq_p) + 4 f (dq_mag + dq_f)
since delta is formed from the rounded out (dq_p), dS is rounded once, and dk is like dq.
A result's 2-norm error is held to the library's bars for the type (1e-2 bf16, 1e-5
fp32) as well, which independent roundings stay far below, unless the value itself is the
rest of a cancellation: where a row sees one key, dout . v = delta and dq = dk = 0, and what
is left is the error of the two sums of D products, at most (D + 8) 2^-24 of X_f, and of the
rounded out that delta is formed from, u X_p.  The bar of dq and dk is therefore
    |X err|_2 <= bar |X|_2 + (D + 8) 2^-24 |X_f|_2 + u |X_p|_2.
"""
import numpy as np
import torch

from oracle import dense_oracle as D
from tests.parity_util import rel_fro

U = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
FRO = {torch.bfloat16: 1e-2, torch.float32: 1e-5}


def np64(t):
    return t.detach().double().cpu().numpy()


def weight_error(q, k, scale=None):
    """f for one sequence's q [n, Hq, D], k [m, Hkv, D] (rows that take part)."""
    q, k = np64(q), np64(k)
    n, hq, d = q.shape
    m, hkv, _ = k.shape
    scale = scale or d ** -0.5
    a = max(float((np.abs(q[:, h]) @ np.abs(k[:, h // (hq // hkv)]).T).max()) for h in range(hq))
    return 2.0 ** -24 * (2 * (d + 8) * scale * a + m + 64)


def close(name, got, want, bound, dtype, rest=0.0):
    got = np64(got)
    assert got.shape == want.shape, name
    assert np.isfinite(got).all(), f"{name}: not finite"
    bad = np.abs(got - want) > bound
    assert not bad.any(), (f"{name}: {int(bad.sum())} of {bad.size} values off, worst "
                           f"{float((np.abs(got - want) / bound)[bad].max()):.3g} x its bound, first "
                           f"at {np.argwhere(bad)[0]}")
    if np.linalg.norm(want) > 0 and want.size > 64:
        assert np.linalg.norm(got - want) <= FRO[dtype] * np.linalg.norm(want) + rest, (
            f"{name}: {rel_fro(got, want):.3g}")


def check_forward(out, lse, r, f, dtype, name=""):
    u = U[dtype]
    close(name + "out", out, r["out"], u * (r["out_mag"] + np.abs(r["out"])) + f * r["out_mag"]
          + 1e-30, dtype)
    if lse is not None:
        got, want = np64(lse), r["lse"]
        empty = np.isneginf(want)
        assert np.array_equal(np.isneginf(got), empty), name + "lse of empty rows"
        got, want = got[~empty], want[~empty]
        assert (np.abs(got - want) <= f + 2.0 ** -22 * np.abs(want)).all(), name + "lse"


def check_grads(dq, dk, dv, r, f, dtype, name=""):
    u = U[dtype]
    tiny = 1e-30
    close(name + "dv", dv, r["dv"], u * (r["dv_mag"] + np.abs(r["dv"])) + 2 * f * r["dv_mag"] + tiny,
          dtype)
    for a, got in (("dq", dq), ("dk", dk)):
        close(name + a, got, r[a], u * (r[a + "_mag"] + np.abs(r[a]) + r[a + "_p"])
              + 4 * f * (r[a + "_mag"] + r[a + "_f"]) + tiny, dtype,
              (r[a].shape[-1] + 8) * 2.0 ** -24 * np.linalg.norm(r[a + "_f"])
              + u * np.linalg.norm(r[a + "_p"]))


def randn(shape, dtype, seed, scale=1.0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return (scale * torch.randn(shape, generator=gen, device="cuda")).to(dtype)


def check_sequence(q, k, v, out, lse, pos0, scale=None, dout=None, grads=None, name=""):
    """One sequence's slices against the oracle."""
    r = D.dense_attend(q, k, v, pos0, scale, dout=dout)
    f = weight_error(q, k, scale)
    check_forward(out, lse, r, f, q.dtype, name)
    if grads is not None:
        check_grads(*grads, r, f, q.dtype, name)
