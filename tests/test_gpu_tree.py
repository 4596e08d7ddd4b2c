"""Attention of drafted tokens over a cache (msa_tree_attend) against the fp64 oracle,
within the bounds derived in dense_util."""
import numpy as np
import pytest
import torch

from block_sparse_gqa_04_b200 import msa
from oracle import dense_oracle as D
from tests.dense_util import check_forward, randn, weight_error

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


def _tree_masks(b, n, seed):
    """Random trees: each node below an earlier one, or below the text."""
    rng = np.random.default_rng(seed)
    m = np.zeros((b, n, n), bool)
    for i in range(b):
        for j in range(n):
            p = int(rng.integers(-1, j)) if j else -1
            if p >= 0:
                m[i, j] = m[i, p]
            m[i, j, j] = True
    return m


def _check(q, k, v, mask, lens, out, lse, scale=None):
    """k, v: dense per-sequence views [B, >= len + n, Hkv, D]."""
    n = q.shape[1]
    for i, kept in enumerate(lens):
        m = mask if mask.ndim == 2 else mask[i]
        seen = np.concatenate([np.ones(kept, bool), m.any(0)])
        r = D.tree_attend(q[i], k[i], v[i], m, kept, scale)
        rows = torch.from_numpy(np.flatnonzero(seen)).cuda()
        f = weight_error(q[i], k[i][:kept + n][rows], scale) if len(rows) else 0.0
        check_forward(out[i], lse[i], r, f, q.dtype, f"sequence {i}: ")


# batch, nodes, cached lengths, q heads, kv heads, head_dim
CASES = {
    "token": (3, 1, [0, 1, 300], 16, 2, 128),
    "token_heads_of_their_own": (2, 1, [127, 128], 4, 4, 64),
    "edges": (5, 8, [119, 120, 121, 128, 249], 16, 1, 128),
    "three_per_group": (2, 5, [77, 500], 12, 4, 128),
    "many_rows": (2, 61, [200, 333], 16, 1, 64),
    "all_nodes": (1, 128, [130], 8, 2, 128),
    "only_drafts": (2, 7, [0, 0], 8, 2, 64),
    "long": (1, 4, [6000], 8, 1, 128),
    "five_heads": (1, 30, [260], 5, 1, 64),
    "whole_tile_of_heads": (2, 3, [300, 5], 128, 1, 64),
    "64_heads": (1, 5, [1000], 64, 1, 128),
}


@pytest.mark.parametrize("paged", [False, True], ids=["cache", "pages"])
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("name", list(CASES))
def test_matches_oracle(name, dtype, paged):
    b, n, lens, hq, hkv, d = CASES[name]
    cap = max(lens) + n + 5
    q = randn((b, n, hq, d), dtype, 1)
    k, v = randn((b, cap, hkv, d), dtype, 2), randn((b, cap, hkv, d), dtype, 3)
    for i, kept in enumerate(lens):  # behind a sequence's rows: whatever was there
        k[i, kept + n:], v[i, kept + n:] = float("nan"), float("inf")
    mask = _tree_masks(b, n, 4)
    kv_lens = torch.tensor(lens, dtype=torch.int32, device="cuda")
    kw, kc, vc = {}, k, v
    if paged:
        w = -(-cap // 128)
        perm = torch.randperm(b * w + 2)[:b * w].view(b, w)
        kc, vc = (torch.full((b * w + 2, 128, hkv, d), float("nan"), dtype=dtype, device="cuda")
                  for _ in range(2))
        for i in range(b):
            for c in range(w):
                m = min(128, cap - 128 * c)
                kc[perm[i, c], :m] = k[i, 128 * c:128 * c + m]
                vc[perm[i, c], :m] = v[i, 128 * c:128 * c + m]
        kw = dict(block_table=perm.to(torch.int32).cuda(), kv_len=cap)
    out, lse = msa.tree_attend(q, kc, vc, torch.from_numpy(mask).cuda(), kv_lens, return_lse=True,
                               check_device_status=True, **kw)
    _check(q, k, v, mask, lens, out, lse)


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
def test_masks_that_leave_rows_and_drafts_out(dtype):
    """Rows that see no draft, with and without cached text; drafts that nobody sees and
    that hold NaN; one mask for all sequences; a mask that is no tree."""
    b, n, hq, hkv, d = 3, 9, 8, 2, 128
    lens = [0, 125, 400]
    q = randn((b, n, hq, d), dtype, 5)
    k, v = randn((b, 420, hkv, d), dtype, 6), randn((b, 420, hkv, d), dtype, 7)
    mask = np.random.default_rng(8).random((n, n)) < 0.5
    mask[2] = False
    mask[:, [1, 6]] = False
    for i, kept in enumerate(lens):
        for j in (1, 6):
            k[i, kept + j], v[i, kept + j] = float("inf"), float("nan")
    out, lse = msa.tree_attend(q, k, v, torch.from_numpy(mask).cuda(),
                               torch.tensor(lens, dtype=torch.int32, device="cuda"),
                               return_lse=True)
    _check(q, k, v, mask, lens, out, lse)
    assert not out[0, 2].any() and torch.isneginf(lse[0, 2]).all()


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
def test_rising_logits(dtype):
    q = (randn((1, 6, 8, 128), dtype, 1).float().abs() + 0.1).to(dtype)
    ramp = torch.linspace(-1, 1, 1006, device="cuda")[None, :, None, None]
    k = (randn((1, 1006, 2, 128), dtype, 2).float().abs() * ramp).to(dtype)
    v = randn((1, 1006, 2, 128), dtype, 3)
    mask = np.tril(np.ones((6, 6), bool))
    lens = torch.tensor([1000], dtype=torch.int32, device="cuda")
    out, lse = msa.tree_attend(q, k, v, torch.from_numpy(mask).cuda(), lens, softmax_scale=0.5,
                               return_lse=True)
    _check(q, k, v, mask, [1000], out, lse, 0.5)


def test_many_sequences():
    """More sequences than one warp scans at a time, most of them in one CTA's share."""
    b, hq, hkv, d = 100, 4, 2, 64
    rng = np.random.default_rng(3)
    lens = rng.integers(0, 200, b).tolist()
    q = randn((b, 2, hq, d), BF16, 1)
    k, v = randn((b, 210, hkv, d), BF16, 2), randn((b, 210, hkv, d), BF16, 3)
    mask = np.tril(np.ones((2, 2), bool))
    out, lse = msa.tree_attend(q, k, v, torch.from_numpy(mask).cuda(),
                               torch.tensor(lens, dtype=torch.int32, device="cuda"),
                               return_lse=True)
    _check(q, k, v, mask, lens, out, lse)


def test_lengths_outside_the_cache_are_flagged_and_clamped():
    q = randn((2, 3, 4, 64), BF16, 1)
    k, v = randn((2, 50, 2, 64), BF16, 2), randn((2, 50, 2, 64), BF16, 3)
    mask = torch.tril(torch.ones((3, 3), dtype=torch.bool, device="cuda"))
    bad = torch.tensor([-1, 48], dtype=torch.int32, device="cuda")
    with pytest.raises(msa.MsaError, match="MSA_ERR_DEVICE"):
        msa.tree_attend(q, k, v, mask, bad, check_device_status=True)
    got = msa.tree_attend(q, k, v, mask, bad)
    want = msa.tree_attend(q, k, v, mask, bad.clamp(0, 47), check_device_status=True)
    assert torch.equal(got, want)


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
def test_pages_that_are_read_are_checked_and_no_others(dtype):
    q = randn((2, 2, 4, 64), dtype, 1)
    pk, pv = randn((5, 128, 2, 64), dtype, 2), randn((5, 128, 2, 64), dtype, 3)
    mask = torch.ones((2, 2), dtype=torch.bool, device="cuda").tril()
    lens = torch.tensor([100, 300], dtype=torch.int32, device="cuda")
    table = torch.tensor([[3, 9, -7], [4, 0, 1]], dtype=torch.int32, device="cuda")
    kw = dict(block_table=table, kv_len=384, return_lse=True)
    got = msa.tree_attend(q, pk, pv, mask, lens, check_device_status=True, **kw)
    for i, pages in enumerate(([3], [4, 0, 1])):
        k, v = (x[pages].flatten(0, 1)[None] for x in (pk, pv))
        want = msa.tree_attend(q[i:i + 1], k, v, mask, lens[i:i + 1], return_lse=True)
        r = D.tree_attend(q[i], k[0], v[0], mask.cpu().numpy(), int(lens[i]))
        f = weight_error(q[i], k[0][:int(lens[i]) + 2])
        check_forward(got[0][i], got[1][i], r, f, dtype)
        check_forward(want[0][0], want[1][0], r, f, dtype)
    for bad in (5, -1):
        table[1, 2] = bad
        with pytest.raises(msa.MsaError, match="MSA_ERR_DEVICE"):
            msa.tree_attend(q, pk, pv, mask, lens, check_device_status=True, **kw)
        # a page outside the pool reads as page 0
        table[1, 2] = 0
        want = msa.tree_attend(q, pk, pv, mask, lens, **kw)
        table[1, 2] = bad
        assert all(torch.equal(a, b) for a, b in
                   zip(want, msa.tree_attend(q, pk, pv, mask, lens, **kw)))


def test_captured_and_replayed_with_growing_lengths():
    """One captured call serves every later step: lengths, mask and cache are read when
    it runs.  Two graphs share one workspace."""
    b, n, cap = 3, 4, 900
    q = randn((b, n, 16, 128), BF16, 1)
    k, v = randn((b, cap, 2, 128), BF16, 2), randn((b, cap, 2, 128), BF16, 3)
    lens = torch.tensor([0, 5, 100], dtype=torch.int32, device="cuda")
    mask = torch.tril(torch.ones((n, n), dtype=torch.bool, device="cuda"))
    p = msa.make_problem(b, n, cap, 16, 2, 128, 32)
    import ctypes
    ws = torch.empty(msa.load().msa_tree_workspace_size(ctypes.byref(p)) + 256,
                     dtype=torch.uint8, device="cuda")
    msa.tree_attend(q, k, v, mask, lens)
    torch.cuda.synchronize()
    graphs, outs = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(msa.tree_attend(q, k, v, mask, lens, return_lse=True, workspace=ws))
        graphs.append(g)
    for step in range(3):
        lens += 250
        lens.clamp_(max=cap - n)
        for g, got in zip(graphs, outs):
            g.replay()
            want = msa.tree_attend(q, k, v, mask, lens, return_lse=True)
            assert all(torch.equal(a, b_) for a, b_ in zip(got, want))


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
def test_cache_rows_behind_32_bits_of_elements(dtype):
    """The last sequence's rows lie more than 2^31 elements into the cache."""
    b, cap, hq, hkv, d = 5, 1 << 20, 16, 4, 128
    lens = [3, 0, 50, 1, 700]
    k, v = (torch.empty((b, cap, hkv, d), dtype=dtype, device="cuda") for _ in range(2))
    assert k[:4].numel() >= 1 << 31
    for i, n in enumerate(lens):
        k[i, :n + 2], v[i, :n + 2] = randn((n + 2, hkv, d), dtype, i), randn((n + 2, hkv, d), dtype, 9 + i)
    q = randn((b, 2, hq, d), dtype, 77)
    mask = np.tril(np.ones((2, 2), bool))
    out, lse = msa.tree_attend(q, k, v, torch.from_numpy(mask).cuda(),
                               torch.tensor(lens, dtype=torch.int32, device="cuda"),
                               return_lse=True, check_device_status=True)
    _check(q, k, v, mask, lens, out, lse)


def test_two_streams_at_once():
    q = randn((3, 4, 16, 128), BF16, 1)
    k, v = randn((3, 3000, 2, 128), BF16, 2), randn((3, 3000, 2, 128), BF16, 3)
    mask = torch.ones((4, 4), dtype=torch.bool, device="cuda").tril()
    lens = torch.tensor([2990, 100, 1500], dtype=torch.int32, device="cuda")
    want = msa.tree_attend(q, k, v, mask, lens, return_lse=True)
    torch.cuda.synchronize()
    got = []
    for _ in range(5):
        for s in (torch.cuda.Stream(), torch.cuda.Stream()):
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):
                got.append(msa.tree_attend(q, k, v, mask, lens, return_lse=True))
    torch.cuda.synchronize()
    for o in got:
        assert all(torch.equal(a, b) for a, b in zip(want, o))


def test_nothing_drafted_and_refusals():
    k = randn((2, 50, 2, 64), BF16, 2)
    lens = torch.tensor([1, 2], dtype=torch.int32, device="cuda")
    q = torch.empty((2, 0, 4, 64), dtype=BF16, device="cuda")
    none = torch.empty((0, 0), dtype=torch.bool, device="cuda")
    assert msa.tree_attend(q, k, k, none, lens).shape == q.shape
    q, one = randn((2, 1, 4, 64), BF16, 1), torch.ones((1, 1), dtype=torch.bool, device="cuda")
    for bad in (lambda: msa.tree_attend(q, k, k, one, lens.long()),
                lambda: msa.tree_attend(q, k, k, one.int(), lens),
                lambda: msa.tree_attend(q, k, k, one[0], lens),
                lambda: msa.tree_attend(q, k, k, one, lens.cpu()),
                lambda: msa.tree_attend(q, k, k[:1], one, lens),
                lambda: msa.tree_attend(q, k, k, one, lens, kv_len=50),
                lambda: msa.tree_attend(q, k, k, one, lens, out=q.float()),
                lambda: msa.tree_attend(q.repeat(1, 129, 1, 1), k.repeat(1, 4, 1, 1),
                                        k.repeat(1, 4, 1, 1),
                                        torch.ones((129, 129), dtype=torch.bool, device="cuda"),
                                        lens)):
        with pytest.raises((ValueError, msa.MsaError)):
            bad()
