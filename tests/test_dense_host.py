"""Host-side checks of the dense operators' C ABI: struct layout, workspace sizes and the
refusals, all decided before any launch (no GPU needed; the pointers are never read)."""
import ctypes
import os
import re
import subprocess

import pytest
import torch

from block_sparse_gqa_04_b200 import msa

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 1 << 20
OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3


@pytest.fixture(scope="module")
def lib():
    from block_sparse_gqa_04_b200 import build
    build.build()
    return msa.load()


def _ints(xs):
    return None if xs is None else (ctypes.c_int32 * len(xs))(*xs)


def _problem(**kw):
    a = dict(batch=2, q_len=64, kv_len=256, Hq=8, Hkv=2, D=128, block=32, q_pos0=100)
    a.update({k: v for k, v in kw.items() if k in a})
    p = msa.make_problem(a["batch"], a["q_len"], a["kv_len"], a["Hq"], a["Hkv"], a["D"], a["block"],
                         q_pos0=a["q_pos0"])
    for k, v in kw.items():
        if k not in a:
            setattr(p, k, v)
    return p


def _attend(lib, p, cq=None, ck=None, ptr=FAKE, lse=FAKE, ws=FAKE, ws_bytes=0):
    return lib.msa_dense_attend(ctypes.byref(p), _ints(cq), _ints(ck), ptr, FAKE, FAKE, FAKE, lse,
                                ws, ws_bytes, None)


def _backward(lib, p, cq=None, ck=None, ptr=FAKE, ws=FAKE, ws_bytes=0):
    return lib.msa_dense_backward(ctypes.byref(p), _ints(cq), _ints(ck), *[FAKE] * 7, ptr,
                                  FAKE, ws, ws_bytes, None)


def _tree(lib, p, stride=0, mask=FAKE, lens=FAKE, ws=FAKE, ws_bytes=0):
    return lib.msa_tree_attend(ctypes.byref(p), FAKE, FAKE, FAKE, mask, stride, lens, FAKE, FAKE,
                               ws, ws_bytes, None)


@pytest.mark.parametrize("field,value,code", [
    ("batch", 0, INVALID), ("q_len", -1, INVALID), ("kv_len", 0, INVALID),
    ("num_q_heads", 7, INVALID), ("num_kv_heads", 0, INVALID), ("head_dim", 0, INVALID),
    ("head_dim", 96, UNSUPPORTED), ("head_dim", 32, UNSUPPORTED), ("dtype", 7, INVALID),
    ("qk_dtype", 2, UNSUPPORTED), ("softmax_scale", -1.0, INVALID),
    ("softmax_scale", float("inf"), INVALID), ("softmax_scale", float("nan"), INVALID),
    ("num_pages", -1, INVALID), ("num_pages", 4, INVALID),  # pages without a table
])
def test_problems_that_every_operator_refuses(lib, field, value, code):
    p = _problem()
    setattr(p, field, value)
    assert _attend(lib, p) == code
    assert _backward(lib, p) == code
    assert _tree(lib, p) == code
    for back in (0, 1):
        assert lib.msa_dense_workspace_size(ctypes.byref(p), None, None, back) == 0
    assert lib.msa_tree_workspace_size(ctypes.byref(p)) == 0


def test_positions_behind_the_keys_are_refused(lib):
    assert _attend(lib, _problem(q_pos0=0, q_len=256)) == WORKSPACE   # valid, no workspace given
    p = _problem()
    p.q_pos0 = 193                                                    # 193 + 64 > 256
    assert _attend(lib, p) == INVALID
    p.q_pos0 = -1
    assert _attend(lib, p) == INVALID
    assert _tree(lib, p) == WORKSPACE                                 # ignores q_pos0


@pytest.mark.parametrize("q_pos0", [2**63 - 1, 2**63 - 64, 2**32, 2**31])
def test_positions_behind_every_integer_are_refused(lib, q_pos0):
    """q_pos0 + q_len is not formed: it may pass 64 bits."""
    p = _problem()
    p.q_pos0 = q_pos0
    assert _attend(lib, p) == INVALID
    assert _backward(lib, p) == INVALID
    assert lib.msa_dense_workspace_size(ctypes.byref(p), None, None, 0) == 0


@pytest.mark.parametrize("cq,ck,code", [
    ([0, 3, 9], None, INVALID), (None, [0, 3, 9], INVALID),
    ([1, 3, 9], [0, 3, 9], INVALID), ([0, 3, 9], [1, 3, 9], INVALID),
    ([0, 9, 3], [0, 9, 12], INVALID), ([0, 3, 9], [0, 9, 3], INVALID),
    ([0, 4, 9], [0, 3, 9], INVALID),                                  # more rows than tokens
    ([0, 3, 9], [0, 3, 9], WORKSPACE),
])
def test_prefix_sums(lib, cq, ck, code):
    assert _attend(lib, _problem(), cq, ck) == code
    assert _backward(lib, _problem(), cq, ck) == code
    size = lib.msa_dense_workspace_size(ctypes.byref(_problem()), _ints(cq), _ints(ck), 1)
    assert (size > 0) == (code == WORKSPACE)


def test_longest_sequence(lib):
    """2^23 tokens of a sequence: key tiles times 128 stay below 2^31 and a warp that waits
    for a whole row of key tiles stays within its bounded wait."""
    n = 1 << 23
    for kv_len, code in ((n, WORKSPACE), (n + 1, UNSUPPORTED), (2**31 - 1, UNSUPPORTED)):
        p = _problem(num_pages=9, kv_len=kv_len, q_pos0=0)
        p.block_table = FAKE
        assert _attend(lib, p) == code
        assert _tree(lib, p) == code
        assert (lib.msa_tree_workspace_size(ctypes.byref(p)) > 0) == (code == WORKSPACE)
        assert _backward(lib, _problem(batch=1, kv_len=kv_len, q_pos0=0)) == code
        assert _attend(lib, _problem(), [0, 5, 7], [0, 10, min(kv_len + 10, 2**31 - 1)]) == code


def test_pages(lib):
    p = _problem(num_pages=9)
    p.block_table = FAKE
    assert _attend(lib, p) == WORKSPACE
    assert _backward(lib, p) == UNSUPPORTED       # no gradients of a cache
    assert _attend(lib, p, [0, 1, 2], [0, 1, 2]) == UNSUPPORTED


def test_workspaces_and_pointers(lib):
    p = _problem()
    n = lib.msa_dense_workspace_size(ctypes.byref(p), None, None, 0)
    nb = lib.msa_dense_workspace_size(ctypes.byref(p), None, None, 1)
    assert 0 < n < nb and nb >= 2 * 64 * 8 * 4    # one delta per row and head
    assert _attend(lib, p, ws_bytes=n - 1) == WORKSPACE
    assert _attend(lib, p, ws=FAKE + 16, ws_bytes=n) == INVALID
    assert _attend(lib, p, ws=None, ws_bytes=n) == INVALID
    assert _attend(lib, p, ptr=None, ws_bytes=n) == INVALID
    assert _attend(lib, p, ptr=FAKE + 8, ws_bytes=n) == INVALID
    assert _attend(lib, p, lse=FAKE + 4, ws_bytes=n) == INVALID
    assert _backward(lib, p, ptr=None, ws_bytes=nb) == INVALID
    assert _backward(lib, p, ws_bytes=nb - 1) == WORKSPACE
    # nothing to do: no pointer is looked at
    e = _problem(q_len=0)
    assert _attend(lib, e, ptr=None, ws=None) == OK
    assert _tree(lib, e, mask=None, ws=None) == OK
    assert _backward(lib, _problem(), [0, 0, 0], [0, 0, 0], ptr=None, ws=None) == OK


def test_tree_arguments(lib):
    p = _problem()
    n = lib.msa_tree_workspace_size(ctypes.byref(p))
    assert n > 0
    assert _tree(lib, p, ws_bytes=n - 1) == WORKSPACE
    assert _tree(lib, p, mask=None, ws_bytes=n) == INVALID
    assert _tree(lib, p, lens=None, ws_bytes=n) == INVALID
    assert _tree(lib, p, lens=FAKE + 2, ws_bytes=n) == INVALID
    assert _tree(lib, p, stride=64 * 64 - 1, ws_bytes=n) == INVALID
    assert _tree(lib, p, stride=-1, ws_bytes=n) == INVALID
    assert _tree(lib, _problem(q_len=129)) == UNSUPPORTED
    assert _tree(lib, _problem(q_len=129, kv_len=128)) == INVALID     # more nodes than cache
    assert _tree(lib, _problem(Hq=258)) == UNSUPPORTED                # 129 heads per group


def test_norm_rope_struct_layout_matches_header(tmp_path):
    src = tmp_path / "layout.c"
    names = [n for n, _ in msa.NormRope._fields_]
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "msa.h"\nint main(void){'
                   'printf("%zu", sizeof(msa_norm_rope_t));'
                   + "".join(f'printf(" %zu", offsetof(msa_norm_rope_t, {n}));' for n in names)
                   + "return 0;}\n")
    exe = tmp_path / "layout"
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)],
                   check=True)
    got = subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()
    want = [ctypes.sizeof(msa.NormRope)] + [getattr(msa.NormRope, n).offset for n in names]
    assert [int(x) for x in got] == want


def _norm(**kw):
    a = dict(rows=10, num_q_heads=8, num_kv_heads=2, head_dim=128, rotary_dim=64, interleaved=0,
             dtype=msa.MSA_BF16, eps=1e-6, reserved=0, q_stride=1536, k_stride=1536,
             q_out_stride=1024, k_out_stride=256, dq_stride=1024, dk_stride=256)
    a.update(kw)
    return msa.NormRope(**a)


@pytest.mark.parametrize("kw,code", [
    (dict(rows=-1), INVALID), (dict(num_q_heads=0), INVALID), (dict(num_kv_heads=-1), INVALID),
    (dict(head_dim=96), UNSUPPORTED), (dict(rotary_dim=129), INVALID),
    (dict(rotary_dim=-16), INVALID), (dict(rotary_dim=24), UNSUPPORTED), (dict(dtype=2), INVALID),
    (dict(eps=-1.0), INVALID), (dict(eps=float("nan")), INVALID), (dict(reserved=1), INVALID),
    (dict(rows=1 << 31), UNSUPPORTED), (dict(q_stride=1016), INVALID),
    (dict(q_stride=1028), INVALID), (dict(k_out_stride=128), INVALID),
])
def test_norm_rope_refusals(lib, kw, code):
    p = _norm(**kw)
    args = [FAKE] * 8
    assert lib.msa_qk_norm_rope(ctypes.byref(p), *args, None) == code
    assert lib.msa_qk_norm_rope_backward(ctypes.byref(p), *[FAKE] * 12, FAKE, 0, None) == code
    assert lib.msa_qk_norm_rope(ctypes.byref(_norm()), None, *args[1:], None) == INVALID
    assert lib.msa_qk_norm_rope(ctypes.byref(_norm()), *args[:4], FAKE + 4, *args[5:],
                                None) == INVALID
    assert lib.msa_qk_norm_rope_backward(ctypes.byref(_norm()), *[FAKE] * 12, FAKE, 0,
                                         None) == WORKSPACE
    assert lib.msa_qk_norm_rope(ctypes.byref(_norm(rows=0)), *[None] * 8, None) == OK


def test_python_checks_come_before_the_library():
    q, k = torch.zeros(1, 4, 8, 64), torch.zeros(1, 4, 2, 64)
    for bad in (lambda: msa.dense_attend(q, k, k),                        # not on a GPU
                lambda: msa.dense_attend(q[0], k, k),
                lambda: msa.dense_attend(q.half(), k.half(), k.half()),
                lambda: msa.dense_attend(q.transpose(1, 2), k, k),
                lambda: msa.dense_attend(q, k, k[..., :32]),
                lambda: msa.dense_attend(q, k.bfloat16(), k),
                lambda: msa.tree_attend(q, k, k, torch.ones(4, 4, dtype=torch.bool),
                                        torch.zeros(1, dtype=torch.int64)),
                lambda: msa.tree_attend(q, k, k, torch.ones(4, 3, dtype=torch.bool),
                                        torch.zeros(1, dtype=torch.int32))):
        with pytest.raises(ValueError):
            bad()


def test_an_output_shares_no_memory_with_the_inputs(monkeypatch):
    monkeypatch.setattr(msa, "_one_device", lambda *t: 0)                 # CPU tensors here
    buf = torch.zeros(4, 6, 8, 64)
    q, k, v = buf[0:1], torch.zeros(1, 6, 2, 64), torch.zeros(1, 6, 2, 64)
    msa._given_out(buf[1:2], q, k, v)                                     # next to it
    msa._given_out(torch.zeros_like(q), q, k, v)
    late = buf.view(-1)[64:64 + q.numel()].view(q.shape)                  # a head later
    cache = buf[2:].view(1, -1, 2, 64)
    for out, k_ in ((q, k), (late, k), (buf[3:], cache)):
        with pytest.raises(ValueError, match="overlaps"):
            msa._given_out(out, q, k_, v)


def test_overlap_and_stride_checks_of_norm_rope():
    buf = torch.zeros(6, 1536)
    q, k = buf[:, :1024].unflatten(1, (8, 128)), buf[:, 1024:1280].unflatten(1, (2, 128))
    assert msa._row_stride("q", q, (6,), torch.float32) == 1536
    msa._check_overlap("q_out", q, 1536, (q, 1536), (k, 1536))            # in place; side by side
    with pytest.raises(ValueError):
        msa._check_overlap("q_out", q[1:], 1536, (q[:-1], 1536))          # a row later
    with pytest.raises(ValueError):
        msa._check_overlap("k_out", buf[:, 1000:1256].unflatten(1, (2, 128)), 1536, (q, 1536))
    with pytest.raises(ValueError):
        msa._row_stride("q", q.transpose(1, 2), (6,), torch.float32)
    with pytest.raises(ValueError):
        msa._row_stride("q", torch.zeros(4, 6, 8, 128)[:, :3], (4, 3), torch.float32)


def test_an_output_of_norm_rope_lies_on_its_own_input_only(monkeypatch):
    """As many query as key heads: every tensor of the call has the same shape and strides."""
    calls = []
    monkeypatch.setattr(msa, "_one_device", lambda *t: 0)                 # CPU tensors here
    monkeypatch.setattr(msa, "_run", lambda *a: calls.append(a))
    w, f = torch.ones(128), torch.ones(64, dtype=torch.float64)
    pos = torch.arange(6)
    fused = torch.zeros(6, 3, 8, 128)
    pairs = [[torch.zeros(6, 8, 128) for _ in range(2)], [fused[:, 0], fused[:, 1]]]
    for q, k in pairs:
        new = torch.zeros(6, 8, 128)
        for out in ((k, q), (k, new), (new, q), (new, new), (q, q), (k, k), (k, fused[:, 2])):
            with pytest.raises(ValueError, match="overlaps"):
                msa.qk_norm_rope(q, k, w, w, f, pos, out=out)
        assert not calls
        for out in ((q, k), (q, new), (new, k), (fused[:, 2], new)):
            got = msa.qk_norm_rope(q, k, w, w, f, pos, out=out)
            assert got[0] is out[0] and got[1] is out[1] and calls.pop()


def test_norm_rope_refuses_outputs_on_one_another(lib):
    p = _norm(num_q_heads=8, num_kv_heads=8, k_out_stride=1024, dk_stride=1024)
    q, k, w, new = FAKE, 2 * FAKE, 3 * FAKE, 4 * FAKE
    for qo, ko in ((k, new), (new, q), (new, new), (q, q)):
        assert lib.msa_qk_norm_rope(ctypes.byref(p), q, k, w, w, w, w, qo, ko, None) == INVALID
        g = (ctypes.byref(p), q, k, 5 * FAKE, 6 * FAKE, w, w, w, w, qo, ko, w, w, FAKE, 1 << 30, None)
        assert lib.msa_qk_norm_rope_backward(*g) == INVALID


def test_kernels_that_start_early_promise_nothing_about_scratch():
    """A kernel that waits for its predecessor inside itself must not declare what that one
    writes as read-only for its whole life (const and __restrict__): loads of it could move in
    front of the wait.  The caller's tensors are older than the call."""
    tensors = {"q", "k", "v", "out", "dout", "lse", "mask"}
    src = os.path.join(ROOT, "block_sparse_gqa_04_b200", "csrc")
    found = 0
    kernels = re.compile(r"__global__ void(?: __launch_bounds__\([^)]*\))?\s+(\w+)\((.*?)\) \{\n"
                         r"(.*?)\n\}\n", re.S)
    for name in sorted(os.listdir(src)):
        for kernel, parameters, body in kernels.findall(open(os.path.join(src, name)).read()):
            if "griddep_wait()" not in body:
                continue
            found += 1
            for par in parameters.split(","):
                if "const" in par.split() and "__restrict__" in par:
                    assert par.split()[-1] in tensors, (kernel, par.strip())
    assert found == 7


@pytest.mark.parametrize("kw", [dict(q_pos0=2**64), dict(q_pos0=2**63), dict(q_pos0=-2**64),
                                dict(q_pos0=1.5), dict(softmax_scale=1e-60),
                                dict(softmax_scale=-1e-60)])
def test_numbers_that_do_not_fit_the_call_are_refused(lib, monkeypatch, kw):
    """The C structure would hold another number: 2^64 as 0, a tiny scale as the default."""
    calls = []
    monkeypatch.setattr(msa, "_one_device", lambda *t: 0)                 # CPU tensors here
    monkeypatch.setattr(msa, "_run", lambda *a: calls.append(a))
    q, k = torch.zeros(1, 4, 8, 64), torch.zeros(1, 8, 2, 64)
    lse = torch.zeros(1, 4, 8)
    for call in (lambda: msa.dense_attend(q, k, k, **kw),
                 lambda: msa.dense_backward(q, q, k, k, q, lse, **kw)):
        with pytest.raises((ValueError, TypeError)):
            call()
    if "softmax_scale" in kw:
        with pytest.raises(ValueError):
            msa.dense_attend_varlen(q[0], k[0], k[0], [0, 4], [0, 8], **kw)
        with pytest.raises(ValueError):
            msa.tree_attend(q, k, k, torch.ones(4, 4, dtype=torch.bool),
                            torch.zeros(1, dtype=torch.int32), **kw)
    assert not calls


@pytest.mark.parametrize("cq,ck", [([0, 2**32 + 2, 4], [0, 4, 8]), ([0, 2, 4], [0, 2**32 + 4, 8]),
                                   ([-2**32, 2, 4], [0, 4, 8]), ([0, 2.5, 4], [0, 4, 8])])
def test_prefix_sums_that_do_not_fit_are_refused(lib, monkeypatch, cq, ck):
    calls = []
    monkeypatch.setattr(msa, "_one_device", lambda *t: 0)
    monkeypatch.setattr(msa, "_run", lambda *a: calls.append(a))
    q, k = torch.zeros(4, 8, 64), torch.zeros(8, 2, 64)
    with pytest.raises((ValueError, TypeError)):
        msa.dense_attend_varlen(q, k, k, cq, ck)
    with pytest.raises((ValueError, TypeError)):
        msa.dense_backward_varlen(q, q, k, k, q, torch.zeros(4, 8), cq, ck)
    assert not calls


def test_a_cache_longer_than_32_bits_is_refused():
    """kv_len as the structure would hold it, 100."""
    with pytest.raises(ValueError):
        msa._plan("tree", 1, 4, 2**32 + 100, 8, 2, 64, torch.bfloat16, 0, 0.0, 9)
    with pytest.raises(ValueError):
        msa._plan("forward", 1, 4, 2**32 + 100, 8, 2, 64, torch.bfloat16, 0, 0.0, 9)


def test_a_backward_call_without_rows_needs_the_keys_alone(lib):
    """It sets dk and dv to zero: with no rows the other tensors are not looked at."""
    p = _problem(q_len=0)
    n = lib.msa_dense_workspace_size(ctypes.byref(p), None, None, 1)
    assert n > 0

    def call(k=FAKE, v=FAKE, dk=FAKE, dv=FAKE, ws=FAKE, ws_bytes=0):
        return lib.msa_dense_backward(ctypes.byref(p), None, None, None, None, k, v, None, None,
                                      None, dk, dv, ws, ws_bytes, None)

    assert call() == WORKSPACE and call(ws_bytes=n - 1) == WORKSPACE
    for kw in (dict(k=None), dict(v=None), dict(dk=None), dict(dv=None), dict(ws=None)):
        assert call(ws_bytes=n, **kw) == INVALID
    assert _tree(lib, p, mask=None, lens=None, ws=None) == OK
