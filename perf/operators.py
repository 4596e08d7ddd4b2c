"""Cases of the dense-attention operators: what is run, in plain torch and through the library.

Three families, each named by a case's "op":

  norm_rope / norm_rope_grad   RMS norm of every query and key head and the position rotation
  dense / dense_step           causal attention over whole prompts (grouped heads, packed or
                               batched sequences), and the training step with its gradients
  tree                         attention of a tree of drafted tokens over a KV cache, a single
                               token being the tree of one node

`own` selects what run() calls: False computes the operators from elementary torch operations in
32 bits (angles and long sums in 64), True calls block_sparse_gqa_04_b200.msa.
"""
import math

import torch

own = False

DEVICE = "cuda"
EPS = 1e-6
THETA = 5e6  # rotary base of long-context models

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------
def _norm(op, rows, hq, hkv, dim, rotary, interleaved, dtype, pos0):
    return {"op": op, "rows": rows, "q_heads": hq, "kv_heads": hkv, "dim": dim, "rotary": rotary,
            "interleaved": interleaved, "dtype": dtype, "pos0": pos0}


def _dense(op, lens_q, lens_k, packed, hq, hkv, dim, dtype):
    return {"op": op, "lens_q": ",".join(map(str, lens_q)), "lens_k": ",".join(map(str, lens_k)),
            "packed": packed, "q_heads": hq, "kv_heads": hkv, "dim": dim, "dtype": dtype}


def _tree(batch, nodes, kv_lo, kv_hi, paged, hq, hkv, dim, dtype):
    return {"op": "tree", "batch": batch, "nodes": nodes, "kv_lo": kv_lo, "kv_hi": kv_hi,
            "paged": paged, "q_heads": hq, "kv_heads": hkv, "dim": dim, "dtype": dtype}


def listed():
    named = [
        # one decode step of 32 sequences at 128K: the smallest call, bound by latency
        ("norm_rope_decode", _norm("norm_rope", 32, 64, 4, 128, 128, False, "bf16", 131071)),
        # the queries and keys of a 32K prompt, views of one projection's output
        ("norm_rope_prompt", _norm("norm_rope", 32768, 64, 4, 128, 128, False, "bf16", 0)),
        # their gradients in training: odd rows, half of each head rotated, adjacent pairs
        ("norm_rope_grad", _norm("norm_rope_grad", 8191, 64, 4, 128, 64, True, "bf16", 0)),
        # a training step in full precision at the library's smallest configuration
        ("dense_step_f32", _dense("dense_step", [1024], [1024], False, 8, 2, 64, "f32")),
        # prefill of one 8K prompt
        ("dense_prompt_8k", _dense("dense", [8192], [8192], False, 64, 4, 128, "bf16")),
        # a server's packed prompts, ragged, from a single token on
        ("dense_packed", _dense("dense", [1, 127, 128, 129, 513, 1000, 2047],
                                [1, 127, 128, 129, 513, 1000, 2047], True, 64, 4, 128, "bf16")),
        # chunked prefill: the last 512 tokens of an 8000-token context
        ("dense_chunk", _dense("dense", [512], [8000], False, 64, 4, 128, "bf16")),
        # a training step over two 4K sequences (both branches dense, as in index warm-up)
        ("dense_step_2x4k", _dense("dense_step", [4096, 4096], [4096, 4096], False, 64, 4, 128,
                                   "bf16")),
        # a training step over packed documents with small heads
        ("dense_step_packed", _dense("dense_step", [77, 1024, 2000, 333], [77, 1024, 2000, 333],
                                     True, 16, 2, 64, "bf16")),
        # plain decoding: one token for each of 32 sequences over a paged cache
        ("token_paged", _tree(32, 1, 1999, 6000, True, 64, 4, 128, "bf16")),
        # eight drafted tokens each over 128K contexts: bound by reading the cache
        ("tree_128k", _tree(4, 8, 130000, 131040, False, 64, 4, 128, "bf16")),
        # wide trees over shorter paged contexts
        ("tree_wide", _tree(8, 61, 500, 3000, True, 32, 2, 128, "bf16")),
    ]
    return [dict(c, name=n) for n, c in named]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    heads = [(64, 4, 128), (32, 2, 128), (16, 2, 64), (8, 2, 64), (8, 8, 128), (12, 4, 128)]
    kind = rng.choice(["norm_rope", "norm_rope_grad", "dense", "dense", "dense_step", "dense_step",
                       "tree", "tree"])
    hq, hkv, dim = rng.choice(heads)
    dtype = "f32" if rng.random() < 0.2 else "bf16"
    if kind.startswith("norm_rope"):
        rows = _log(rng, 1, 4000 if dtype == "f32" else 30000)
        return _norm(kind, rows, hq, hkv, dim, rng.choice([dim, dim // 2]), rng.random() < 0.5,
                     dtype, rng.randrange(1 << 20))
    if kind.startswith("dense"):
        total = _log(rng, 64, 1500 if dtype == "f32" else 6000)
        n = rng.randint(1, 6)
        if rng.random() < 0.5:  # packed, ragged
            lens_k = [max(1, int(total * w / 2 / n) + rng.randrange(3)) for w in
                      (rng.uniform(0.1, 1.9) for _ in range(n))]
            lens_q = lens_k if kind == "dense_step" else [rng.randint(max(1, k // 2), k)
                                                          for k in lens_k]
            return _dense(kind, lens_q, lens_k, True, hq, hkv, dim, dtype)
        n = min(n, 3)
        sk = max(2, total // n + rng.randrange(3))
        sq = sk if kind == "dense_step" or rng.random() < 0.5 else rng.randint(1, sk)
        return _dense(kind, [sq] * n, [sk] * n, False, hq, hkv, dim, dtype)
    batch, nodes = _log(rng, 1, 24), rng.choice([1, 1, rng.randint(2, 16), rng.randint(17, 100)])
    top = min(60000 // batch, 4000 if dtype == "f32" else 60000, 600000 // (batch * nodes))
    hi = max(nodes + 2, _log(rng, 40, max(80, top)))
    return _tree(batch, nodes, rng.randint(0, hi), hi, rng.random() < 0.5, hq, hkv, dim, dtype)


def _ints(text):
    return [int(x) for x in text.split(",")]


def _sums(lens):
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    return cu


def _kv_lens(c):
    """Cached tokens of each sequence: spread evenly from kv_lo to kv_hi."""
    lo, hi, b = min(c["kv_lo"], c["kv_hi"]), c["kv_hi"], c["batch"]
    return [hi] if b == 1 else [lo + (hi - lo) * i // (b - 1) for i in range(b)]


def _pairs(nq, nk):
    """Visible (query, key) pairs of a causal sequence whose queries are its last nq tokens."""
    return nq * (nk - nq) + nq * (nq + 1) // 2


def work(case):
    c, e = case, 2 if case["dtype"] == "bf16" else 4
    hq, hkv, d = c["q_heads"], c["kv_heads"], c["dim"]
    if c["op"].startswith("norm_rope"):
        n = c["rows"] * (hq + hkv) * d
        grad = c["op"] == "norm_rope_grad"
        return {"bytes": n * e * (3 if grad else 2) + c["rows"] * 8, "flops": n * (20 if grad else 8)}
    if c["op"].startswith("dense"):
        lq, lk = _ints(c["lens_q"]), _ints(c["lens_k"])
        pairs = sum(_pairs(a, b) for a, b in zip(lq, lk))
        q, kv = sum(lq) * hq * d * e, 2 * sum(lk) * hkv * d * e
        lse = 4 * sum(lq) * hq
        if c["op"] == "dense":
            return {"bytes": 2 * q + kv + lse, "flops": 4 * d * hq * pairs}
        # forward: q, k, v -> out, lse; backward: the same, dout -> dq, dk, dv
        return {"bytes": 4 * q + 2 * kv + lse, "flops": 14 * d * hq * pairs}
    lens, n = _kv_lens(c), c["nodes"]
    keys = sum(lens) + n * c["batch"]
    return {"bytes": 2 * keys * hkv * d * e + 2 * c["batch"] * n * hq * d * e,
            "flops": 4 * d * hq * n * keys}


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------
def _randn(gen, shape, dtype):
    return torch.randn(shape, generator=gen, device=DEVICE, dtype=torch.float32).to(dtype)


def prepare(case, seed):
    c, dt = case, DTYPES[case["dtype"]]
    gen = torch.Generator(device=DEVICE).manual_seed(int(seed))
    hq, hkv, d = c["q_heads"], c["kv_heads"], c["dim"]
    s = {"op": c["op"]}
    if c["op"].startswith("norm_rope"):
        rows = c["rows"]
        # queries and keys as a model has them: slices of one fused projection's output
        qkv = _randn(gen, (rows, (hq + 2 * hkv) * d), dt)
        s["q"] = qkv[:, :hq * d].unflatten(1, (hq, d))
        s["k"] = qkv[:, hq * d:(hq + hkv) * d].unflatten(1, (hkv, d))
        s["qw"] = (1 + 0.2 * _randn(gen, (d,), torch.float32)).to(dt)
        s["kw"] = (1 + 0.2 * _randn(gen, (d,), torch.float32)).to(dt)
        half = c["rotary"] // 2
        s["inv_freq"] = THETA ** (-torch.arange(half, device=DEVICE, dtype=torch.float64) / half)
        s["positions"] = c["pos0"] + torch.arange(rows, device=DEVICE)
        s["interleaved"] = c["interleaved"]
        if c["op"] == "norm_rope_grad":
            s["dq"], s["dk"] = _randn(gen, (rows, hq, d), dt), _randn(gen, (rows, hkv, d), dt)
        return s
    if c["op"].startswith("dense"):
        lq, lk = _ints(c["lens_q"]), _ints(c["lens_k"])
        lead_q, lead_k = ((sum(lq),), (sum(lk),)) if c["packed"] else ((len(lq), lq[0]),
                                                                       (len(lk), lk[0]))
        s["q"] = _randn(gen, lead_q + (hq, d), dt)
        s["k"], s["v"] = (_randn(gen, lead_k + (hkv, d), dt) for _ in range(2))
        if c["packed"]:
            s["cu_q"], s["cu_k"] = _sums(lq), _sums(lk)
        else:
            s["q_pos0"] = lk[0] - lq[0]
        if c["op"] == "dense_step":
            s["dout"] = _randn(gen, lead_q + (hq, d), dt)
        return s
    b, n, lens = c["batch"], c["nodes"], _kv_lens(c)
    cap = max(lens) + n
    s["q"] = _randn(gen, (b, n, hq, d), dt)
    s["kv_lens"] = torch.tensor(lens, device=DEVICE, dtype=torch.int32)
    if c["paged"]:
        width = -(-cap // 128)
        shape = (b * width + 3, 128, hkv, d)
        s["table"] = torch.randperm(b * width + 3, generator=gen, device=DEVICE)[:b * width].view(
            b, width).to(torch.int32)
        s["cap"] = cap
    else:
        shape = (b, cap, hkv, d)
    s["k"], s["v"] = _randn(gen, shape, dt), _randn(gen, shape, dt)
    # random trees: node i hangs below a node before it, or below the cached text (-1)
    parent = (torch.rand((b, n), generator=gen, device=DEVICE)
              * (torch.arange(n, device=DEVICE) + 1)).long() - 1
    step = torch.nn.functional.one_hot(parent + 1, n + 1)[..., 1:].float()
    mask = torch.eye(n, device=DEVICE).expand(b, n, n)
    reach = mask
    while n > 1 and bool((reach := ((reach @ step) > 0).float()).any()):
        mask = torch.maximum(mask, reach)
    s["mask"] = mask > 0
    return s


# ---------------------------------------------------------------------------
# Plain forms
# ---------------------------------------------------------------------------
def _cos_sin(s):
    angle = s["positions"].double()[:, None] * s["inv_freq"]
    return angle.cos().float()[:, None], angle.sin().float()[:, None]


def _rotate(x, cos, sin, interleaved):
    """Turns the first 2 * cos.shape[-1] elements of the last axis by the angles."""
    half = cos.shape[-1]
    head, tail = x[..., :2 * half], x[..., 2 * half:]
    if interleaved:
        a, b = head[..., 0::2], head[..., 1::2]
        turned = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    else:
        a, b = head[..., :half], head[..., half:]
        turned = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    return torch.cat((turned, tail), -1)


def _plain_norm_rope(s):
    cos, sin = _cos_sin(s)

    def one(x, w):
        x32 = x.float()
        unit = x32 * torch.rsqrt((x32 * x32).mean(-1, keepdim=True) + EPS)
        return _rotate(unit * w.float(), cos, sin, s["interleaved"]).to(x.dtype)

    return one(s["q"], s["qw"]), one(s["k"], s["kw"])


def _plain_norm_rope_grad(s):
    cos, sin = _cos_sin(s)

    def one(x, w, g):
        x32 = x.float()
        r = torch.rsqrt((x32 * x32).mean(-1, keepdim=True) + EPS)
        unit = x32 * r
        back = _rotate(g.float(), cos, -sin, s["interleaved"])
        dw = (back * unit).sum((0, 1), dtype=torch.float64).float()
        t = back * w.float()
        return (r * (t - unit * (t * unit).mean(-1, keepdim=True))).to(x.dtype), dw

    dq, dqw = one(s["q"], s["qw"], s["dq"])
    dk, dkw = one(s["k"], s["kw"], s["dk"])
    return dq, dk, dqw, dkw


def _hidden(s):
    """[rows, keys] truth values: the keys that a query row does not see."""
    dev = s["q"].device
    if "cu_q" in s:
        cq, ck = (torch.tensor(s[n], device=dev) for n in ("cu_q", "cu_k"))
        nq, nk = cq.diff(), ck.diff()
        seq = torch.arange(len(nq), device=dev)
        sq, sk = seq.repeat_interleave(nq), seq.repeat_interleave(nk)
        pq = torch.arange(len(sq), device=dev) - cq[sq] + (nk - nq)[sq]
        pk = torch.arange(len(sk), device=dev) - ck[sk]
        return (sq[:, None] != sk) | (pk > pq[:, None])
    pq = s["q_pos0"] + torch.arange(s["q"].shape[1], device=dev)
    return torch.arange(s["k"].shape[1], device=dev) > pq[:, None]


def _grouped(x, hkv):
    """[B, S, H, D] -> [B, Hkv, G * S, D] in 32 bits, the heads of a group one after another."""
    b, n, h, d = x.shape
    return x.float().view(b, n, hkv, h // hkv, d).permute(0, 2, 3, 1, 4).reshape(b, hkv, -1, d)


def _ungrouped(x, n):
    """[B, Hkv, G * S, D] -> [B, S, H, D]."""
    b, hkv, gn, d = x.shape
    return x.view(b, hkv, gn // n, n, d).permute(0, 3, 1, 2, 4).reshape(b, n, -1, d)


def _plain_dense(s, step):
    packed = "cu_q" in s
    q, k, v = (s[n][None] if packed else s[n] for n in ("q", "k", "v"))
    hkv, n, scale = k.shape[2], q.shape[1], q.shape[3] ** -0.5
    qg, kg, vg = _grouped(q, hkv), _grouped(k, hkv), _grouped(v, hkv)
    p = qg @ kg.transpose(-1, -2)
    p *= scale
    p.unflatten(2, (-1, n)).masked_fill_(_hidden(s), -math.inf)
    top = p.amax(-1, keepdim=True)
    p -= top
    p.exp_()
    total = p.sum(-1, keepdim=True)
    p /= total
    og = p @ vg
    out = _ungrouped(og, n).to(q.dtype)
    lse = _ungrouped(top + total.log(), n).squeeze(-1)
    first = (lambda x: x[0]) if packed else (lambda x: x)
    if not step:
        return first(out), first(lse)
    dout = _grouped(s["dout"][None] if packed else s["dout"], hkv)
    dv = p.transpose(-1, -2) @ dout
    dp = dout @ vg.transpose(-1, -2)
    dp -= (dout * og).sum(-1, keepdim=True)
    dp *= p
    dp *= scale
    del p
    dq = _ungrouped(dp @ kg, n).to(q.dtype)
    dk = (dp.transpose(-1, -2) @ qg).transpose(1, 2).to(q.dtype)
    return first(out), first(dq), first(dk), first(dv.transpose(1, 2).to(q.dtype))


def _plain_tree(s):
    q, k, v = s["q"], s["k"], s["v"]
    b, n, hq, d = q.shape
    if "table" in s:
        k, v = (x[s["table"].long()].flatten(1, 2) for x in (k, v))
    hkv, g, cap = k.shape[2], hq // k.shape[2], k.shape[1]
    at = torch.arange(cap, device=q.device)[None] - s["kv_lens"].long()[:, None]   # draft index
    draft = (at >= 0) & (at < n)
    sees = s["mask"].gather(2, at.clamp(0, n - 1)[:, None].expand(b, n, cap)) & draft[:, None]
    sees = (at < 0)[:, None] | sees                                                # [B, n, cap]
    qg = q.float().view(b, n, hkv, g, d).permute(0, 2, 1, 3, 4).reshape(b, hkv, n * g, d)
    p = qg @ k.float().permute(0, 2, 3, 1)
    p *= d ** -0.5
    p.view(b, hkv, n, g, cap).masked_fill_(~sees[:, None, :, None], -math.inf)
    top = p.amax(-1, keepdim=True)
    p -= top
    p.exp_()
    total = p.sum(-1, keepdim=True)
    o = (p @ v.float().transpose(1, 2)) / total

    def back(x):
        return x.view(b, hkv, n, g, -1).permute(0, 2, 1, 3, 4).reshape(b, n, hq, -1)

    return back(o).to(q.dtype), back(top + total.log()).squeeze(-1)


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------
def _own(s):
    from block_sparse_gqa_04_b200 import msa

    if s["op"].startswith("norm_rope"):
        args = (s["q"], s["k"], s["qw"], s["kw"], s["inv_freq"], s["positions"])
        kw = dict(eps=EPS, interleaved=s["interleaved"])
        if s["op"] == "norm_rope":
            return msa.qk_norm_rope(*args, **kw)
        return msa.qk_norm_rope_backward(s["dq"], s["dk"], *args, **kw)
    if s["op"] == "tree":
        paged = dict(block_table=s["table"], kv_len=s["cap"]) if "table" in s else {}
        return msa.tree_attend(s["q"], s["k"], s["v"], s["mask"], s["kv_lens"], return_lse=True,
                               **paged)
    qkv = (s["q"], s["k"], s["v"])
    if "cu_q" in s:
        out, lse = msa.dense_attend_varlen(*qkv, s["cu_q"], s["cu_k"], return_lse=True)
        if s["op"] == "dense":
            return out, lse
        return (out,) + msa.dense_backward_varlen(s["dout"], *qkv, out, lse, s["cu_q"], s["cu_k"])
    out, lse = msa.dense_attend(*qkv, q_pos0=s["q_pos0"], return_lse=True)
    if s["op"] == "dense":
        return out, lse
    return (out,) + msa.dense_backward(s["dout"], *qkv, out, lse, q_pos0=s["q_pos0"])


def run(state):
    if own:
        return _own(state)
    if state["op"] == "norm_rope":
        return _plain_norm_rope(state)
    if state["op"] == "norm_rope_grad":
        return _plain_norm_rope_grad(state)
    if state["op"] == "tree":
        return _plain_tree(state)
    return _plain_dense(state, state["op"] == "dense_step")


# ---------------------------------------------------------------------------
# The definitions in 64 bits, head by head; gradients by differentiation
# ---------------------------------------------------------------------------
def _exact_heads(x, w, s):
    """RMS norm and rotation as products of complex numbers."""
    y = x / ((x ** 2).sum(-1, keepdim=True) / x.shape[-1] + EPS).sqrt() * w
    m = s["inv_freq"].numel()
    turn = torch.polar(torch.ones((), dtype=torch.float64, device=x.device),
                       s["positions"].double().outer(s["inv_freq"]))[:, None]
    if s["interleaved"]:
        z = torch.view_as_complex(y[..., :2 * m].unflatten(-1, (m, 2)).contiguous()) * turn
        z = torch.view_as_real(z).flatten(-2)
    else:
        z = torch.complex(y[..., :m], y[..., m:2 * m]) * turn
        z = torch.cat((z.real, z.imag), -1)
    return torch.cat((z, y[..., 2 * m:]), -1)


def _exact_head(q, k, v, sees):
    """softmax(q k^T / sqrt(D)) v over the keys that each row sees, and its normaliser."""
    z = torch.where(sees, q @ k.T / math.sqrt(q.shape[-1]), -math.inf)
    lse = torch.logsumexp(z, -1)
    return torch.exp(z - lse[:, None]) @ v, lse


def _exact_dense(s, step):
    q, k, v = s["q"], s["k"], s["v"]
    dout = s.get("dout")
    if "cu_q" in s:
        spans = list(zip(s["cu_q"][:-1], s["cu_q"][1:], s["cu_k"][:-1], s["cu_k"][1:]))
    else:
        (b, sq), sk = q.shape[:2], k.shape[1]
        spans = [(i * sq, (i + 1) * sq, i * sk, (i + 1) * sk) for i in range(b)]
    flat = lambda x: None if x is None else x.reshape((-1,) + x.shape[-2:])  # noqa: E731
    qf, kf, vf, gf = flat(q), flat(k), flat(v), flat(dout)
    hq, hkv = qf.shape[1], kf.shape[1]
    new = lambda x: torch.zeros(x.shape, dtype=torch.float64, device=x.device)  # noqa: E731
    out, lse, dq, dk, dv = new(qf), new(qf[..., 0]), new(qf), new(kf), new(vf)
    for q0, q1, k0, k1 in spans:
        nq, nk = q1 - q0, k1 - k0
        sees = torch.ones((nq, nk), dtype=torch.bool, device=q.device).tril(nk - nq)
        for h in range(hq):
            g = h // (hq // hkv)
            leaves = [qf[q0:q1, h].double(), kf[k0:k1, g].double(), vf[k0:k1, g].double()]
            if not step:
                out[q0:q1, h], lse[q0:q1, h] = _exact_head(*leaves, sees)
                continue
            leaves = [x.requires_grad_() for x in leaves]
            o, _ = _exact_head(*leaves, sees)
            a, b_, c_ = torch.autograd.grad(o, leaves, gf[q0:q1, h].double())
            out[q0:q1, h], dq[q0:q1, h] = o.detach(), a
            dk[k0:k1, g] += b_
            dv[k0:k1, g] += c_
    if not step:
        return out.view(q.shape), lse.view(q.shape[:-1])
    return out.view(q.shape), dq.view(q.shape), dk.view(k.shape), dv.view(v.shape)


def _exact_tree(s):
    q, mask = s["q"], s["mask"]
    b, n, hq, d = q.shape
    out = torch.zeros((b, n, hq, d), dtype=torch.float64, device=q.device)
    lse = torch.zeros((b, n, hq), dtype=torch.float64, device=q.device)
    for i, kept in enumerate(s["kv_lens"].tolist()):
        if "table" in s:
            k, v = (s[x][s["table"][i].long()].flatten(0, 1)[:kept + n] for x in ("k", "v"))
        else:
            k, v = s["k"][i, :kept + n], s["v"][i, :kept + n]
        sees = torch.cat((torch.ones((n, kept), dtype=torch.bool, device=q.device), mask[i]), 1)
        for h in range(hq):
            g = h // (hq // k.shape[1])
            out[i, :, h], lse[i, :, h] = _exact_head(q[i, :, h].double(), k[:, g].double(),
                                                     v[:, g].double(), sees)
    return out, lse


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm_rope":
        return tuple(_exact_heads(s[x].double(), s[w].double(), s)
                     for x, w in (("q", "qw"), ("k", "kw")))
    if case["op"] == "norm_rope_grad":
        got = []
        for x, w, g in (("q", "qw", "dq"), ("k", "kw", "dk")):
            leaves = [s[x].double().requires_grad_(), s[w].double().requires_grad_()]
            got.append(torch.autograd.grad(_exact_heads(*leaves, s), leaves, s[g].double()))
        return got[0][0], got[1][0], got[0][1], got[1][1]
    if case["op"] == "tree":
        return _exact_tree(s)
    return _exact_dense(s, case["op"] == "dense_step")
