"""What the operators around the attention cost, case by case.

Three operators: appending keys and values to a paged cache (with the
position rotation), the attention that reads that cache, and the layer norm
with its gate and residual (forward and backward).  Each case is computed
in a plain form (``own`` false: elementary torch operations in 32 bits) or
by the library's kernels (``own`` true).

A case is a dict of plain values.  ``lens`` seeds the sequence lengths, so
that a case's work does not depend on the seed of its values: sequence b
has ``hist_lo`` to ``hist_hi`` cached tokens (uniform, or log-normal with
median 512 clipped to that range) and ``new_lo`` to ``new`` new ones, of
which the last are candidates (``targets``: 0 none, 1 some, 2 all).
"""
from __future__ import annotations

import math
import random

import numpy as np
import torch

own = False

EPS = 1e-6
ROTARY_BASE = 10000.0


# ------------------------------------------------------------------ the cases
def _append(name, lens, batch, hist_lo, hist_hi, new_lo, new, heads, d, page, rot, pairs=False,
            with_q=True, fused=True, targets=0, pad=0, kind="uniform"):
    return dict(name=name, op="append", lens=lens, kind=kind, batch=batch, hist_lo=hist_lo,
                hist_hi=hist_hi, new_lo=new_lo, new=new, targets=targets, heads=heads, d=d, page=page,
                rot=rot, pairs=pairs, with_q=with_q, fused=fused, pad=pad)


def _attn(name, lens, batch, hist_lo, hist_hi, new_lo, new, heads, d, page, targets=0,
          kind="uniform", pad=0):
    return dict(name=name, op="attn", lens=lens, kind=kind, batch=batch, hist_lo=hist_lo,
                hist_hi=hist_hi, new_lo=new_lo, new=new, targets=targets, heads=heads, d=d, page=page,
                pad=pad)


def _norm(name, op, rows, width, gate, residual, scale=1.0, fused=False):
    return dict(name=name, op=op, rows=rows, width=width, gate=gate, residual=residual, scale=scale,
                fused=fused)


def listed():
    return [
        # one decode step of a batch of users: 64 sequences append one token each
        _append("append_step", 1, 64, 0, 2047, 1, 1, heads=4, d=64, page=64, rot=64),
        # filling the cache from 16 whole histories of 4096 tokens, out of the fused projection
        _append("append_histories", 2, 16, 0, 0, 4096, 4096, heads=4, d=64, page=128, rot=64),
        # the smallest attention call: one user, one token, a short history
        _attn("attn_one", 4, 1, 512, 512, 1, 1, heads=4, d=64, page=16),
        # one decode step of a many-user batch with log-normal lengths
        _attn("attn_serving", 5, 512, 0, 8191, 1, 1, heads=2, d=64, page=64, kind="lognormal"),
        # one decode step of four long sequences: few rows, a long axis
        _attn("attn_long", 6, 4, 10239, 20479, 1, 1, heads=4, d=64, page=128),
        # a few candidates per user against cached histories
        _attn("attn_few_candidates", 7, 8, 2048, 8192, 9, 16, heads=4, d=128, page=32, targets=2),
        # ranking: 1024 candidates per user against histories of 2048 to 8192 tokens
        _attn("attn_candidates", 8, 32, 2048, 8192, 1024, 1024, heads=4, d=64, page=64, targets=2),
        # histories that grow by a ragged chunk, causal within the chunk
        _attn("attn_chunk", 9, 16, 0, 4190, 100, 700, heads=4, d=128, page=64),
        # the output stage of one decode step of 64 users
        _norm("norm_gate_step", "norm_fwd", 64, 256, gate=True, residual=False, fused=True),
        # residual and the next layer's norm over a skewed batch (4 heads of 128)
        _norm("norm_residual", "norm_fwd", 37611, 512, gate=False, residual=True, scale=0.5),
        # gradient of the output stage in training: 16 sequences of 4096 tokens, 4 heads of 64
        _norm("norm_gate_bwd", "norm_bwd", 65536, 256, gate=True, residual=False, fused=True),
        # gradient of residual and norm on a small wide batch
        _norm("norm_residual_bwd", "norm_bwd", 4099, 1024, gate=False, residual=True, scale=0.5),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1e-9)))))


def draw(rng: random.Random):
    """One more case over the same ranges, no dearer than the largest listed."""
    most = {}
    for c in listed():
        w = work(c)
        op = c["op"]
        b, f = most.get(op, (0, 0))
        most[op] = (max(b, w["bytes"]), max(f, w["flops"]))
    op = rng.choice(["append", "attn", "attn", "attn", "norm_fwd", "norm_bwd"])
    while True:
        if op == "append":
            c = _append("", rng.randrange(1 << 30), _log(rng, 1, 512), 0, _log(rng, 1, 8192), 1,
                        1 if rng.random() < 0.4 else _log(rng, 1, 4096), heads=rng.choice([1, 2, 3, 4, 8]),
                        d=rng.choice([32, 64, 128]), page=rng.choice([16, 32, 64, 128, 256]), rot=0,
                        pairs=rng.random() < 0.5, with_q=rng.random() < 0.7, fused=rng.random() < 0.5,
                        targets=rng.choice([0, 0, 1, 2]), pad=rng.choice([0, 0, 5, 64]))
            c["rot"] = rng.choice([r for r in (0, 16, 32, 64, 128) if r <= c["d"]])
            c["hist_lo"] = rng.randrange(0, c["hist_hi"] + 1)
            c["new_lo"] = rng.randrange(1, c["new"] + 1)
        elif op == "attn":
            c = _attn("", rng.randrange(1 << 30), _log(rng, 1, 512), 0, _log(rng, 1, 20480), 1,
                      1 if rng.random() < 0.4 else _log(rng, 1, 1024), heads=rng.choice([1, 2, 3, 4, 8]),
                      d=rng.choice([32, 64, 128]), page=rng.choice([16, 32, 64, 128, 256]),
                      targets=rng.choice([0, 1, 2]), kind=rng.choice(["uniform", "uniform", "lognormal"]),
                      pad=rng.choice([0, 0, 5, 64]))
            c["hist_lo"] = rng.randrange(0, c["hist_hi"] + 1)
            c["new_lo"] = rng.randrange(1, c["new"] + 1)
        else:
            c = _norm("", op, _log(rng, 1, 65536), 8 * _log(rng, 1, 1024), gate=rng.random() < 0.5,
                      residual=rng.random() < 0.5, scale=rng.choice([1.0, 0.5, 0.25]),
                      fused=rng.random() < 0.5)
        w = work(c)
        b, f = most[op if op in ("append", "attn") else "norm_bwd"]
        if w["bytes"] <= b and w["flops"] <= f:
            del c["name"]
            return c


def _lengths(case):
    """(cached, new, candidates) tokens of every sequence, as int64 arrays."""
    rng = np.random.default_rng(case["lens"])
    n, lo, hi = case["batch"], case["hist_lo"], case["hist_hi"]
    if case["kind"] == "lognormal":
        hist = np.clip(np.rint(np.exp(math.log(512.0) + rng.standard_normal(n))), lo, hi).astype(np.int64)
    else:
        hist = rng.integers(lo, hi + 1, size=n)
    new = rng.integers(case["new_lo"], case["new"] + 1, size=n)
    if case["targets"] == 0:
        tgt = np.zeros(n, dtype=np.int64)
    elif case["targets"] == 2:
        tgt = new.copy()
    else:
        tgt = rng.integers(0, new + 1)
    return hist, new, tgt


def work(case):
    """The bytes and operations of one pass that no form can do without."""
    if case["op"].startswith("norm"):
        n, w = case["rows"], case["width"]
        if case["op"] == "norm_fwd":
            arrays = 2 + case["gate"] + 2 * case["residual"]  # x, y; u; residual, z
            return dict(bytes=2 * n * w * arrays + 8 * w, flops=n * w * (8 + 2 * case["residual"]))
        # dy, z, dz; u, du; dz_in, dx
        arrays = 3 + 2 * case["gate"] + 2 * case["residual"]
        return dict(bytes=2 * n * w * arrays + 16 * w, flops=n * w * (16 + 4 * case["gate"]))
    hist, new, tgt = _lengths(case)
    row = case["heads"] * case["d"] * 2
    total = int(new.sum())
    if case["op"] == "append":
        arrays = 4 + 2 * case["with_q"]  # k, v read and written; q
        turned = total * case["heads"] * case["rot"] * (1 + case["with_q"])
        return dict(bytes=total * (row * arrays + 4 * case["rot"]) + 8 * case["batch"], flops=3 * turned)
    kv = hist + new
    keep = kv - tgt  # what every candidate sees, besides itself
    plain = new - tgt
    pairs = int((plain * keep - plain * (plain - 1) // 2 + tgt * (keep + 1)).sum())
    pages = int(((kv + case["page"] - 1) // case["page"]).sum())
    return dict(bytes=2 * row * int(kv.sum()) + 2 * row * total + 4 * pages + 8 * case["batch"],
                flops=4 * pairs * case["heads"] * case["d"])


# ------------------------------------------------------------------ the inputs
def _normal(gen, *shape, sigma=1.0, dtype=torch.bfloat16):
    return (torch.randn(*shape, generator=gen, device="cuda", dtype=torch.float32) * sigma).to(dtype)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    s = dict(case=case)
    if case["op"].startswith("norm"):
        n, w = case["rows"], case["width"]
        s["x"] = _normal(gen, n, w)
        s["gamma"] = 1.0 + 0.1 * _normal(gen, w, dtype=torch.float32)
        s["beta"] = 0.1 * _normal(gen, w, dtype=torch.float32)
        if case["gate"]:  # U is one quarter of the layer's first projection
            s["u"] = _normal(gen, n, 4 * w)[:, :w] if case["fused"] else _normal(gen, n, w)
        if case["residual"]:
            s["other"] = _normal(gen, n, w)  # the residual stream, or its gradient so far
        if case["op"] == "norm_bwd":
            s["dy"] = _normal(gen, n, w)
        s["out"] = [torch.empty(n, w, device="cuda", dtype=torch.bfloat16) for _ in range(3)]
        s["sums"] = [torch.empty(w, device="cuda", dtype=torch.float32) for _ in range(2)]
        if own:
            from hstu_jagged_attention_gb300 import binding
            s["binding"] = binding
            s["workspace"] = torch.empty(binding.hstu_norm_bwd_workspace_bytes(w), device="cuda",
                                         dtype=torch.uint8)
        return s

    hist, new, tgt = _lengths(case)
    heads, d, page = case["heads"], case["d"], case["page"]
    sigma = 1.0 if d < 128 else 0.5
    kv = hist + new
    n_pages = (kv + page - 1) // page
    spare = 3
    order = torch.randperm(int(n_pages.sum()) + spare, generator=gen, device="cuda").cpu().numpy()
    table = np.zeros((case["batch"], int(n_pages.max())), dtype=np.int32)
    at = 0
    for b in range(case["batch"]):
        table[b, :n_pages[b]] = order[at:at + n_pages[b]]
        at += int(n_pages[b])
    total = int(new.sum())
    rows = total + case["pad"]  # a padded batch: rows behind the last sequence
    offsets = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    shape = (len(order), page, heads, d)
    s["k_pages"], s["v_pages"] = _normal(gen, *shape, sigma=sigma), _normal(gen, *shape, sigma=sigma)
    s["table"] = torch.from_numpy(table).cuda()
    s["q_offsets"] = torch.from_numpy(offsets).cuda()
    s["kv_lens"] = torch.from_numpy(kv.astype(np.int32)).cuda()
    s["targets"] = torch.from_numpy(tgt.astype(np.int32)).cuda() if case["targets"] else None
    s["hist"], s["new"], s["tgt"], s["total"] = hist.tolist(), new.tolist(), tgt.tolist(), total
    s["out"] = torch.zeros(rows, heads, d, device="cuda", dtype=torch.bfloat16)
    if case["op"] == "append":
        if case["fused"]:  # V, Q and K are quarters of the layer's first projection
            proj = _normal(gen, rows, 4, heads, d, sigma=sigma)
            s["v"], s["q"], s["k"] = proj[:, 1], proj[:, 2], proj[:, 3]
        else:
            s["k"], s["v"], s["q"] = (_normal(gen, rows, heads, d, sigma=sigma) for _ in range(3))
        s["rotary"] = None
        if case["rot"]:
            angle = np.arange(int(kv.max()), dtype=np.float64)[:, None] * \
                ROTARY_BASE ** (-np.arange(0, case["rot"], 2, dtype=np.float64) / case["rot"])
            both = np.concatenate([np.cos(angle), np.sin(angle)], axis=1).astype(np.float32)
            s["rotary"] = torch.from_numpy(both).cuda()
    else:
        s["q"] = _normal(gen, rows, heads, d, sigma=sigma)
        s["alpha"], s["inv_n"] = 1.0 / math.sqrt(d), 1.0 / int(kv.max())
        # slots behind a sequence's end were never written: whatever lies there must not be read
        last = torch.from_numpy(table[np.arange(case["batch"]), n_pages - 1].astype(np.int64)).cuda()
        fill = torch.from_numpy((kv - (n_pages - 1) * page).astype(np.int64)).cuda()
        behind = torch.arange(page, device="cuda")[None, :] >= fill[:, None]
        which, slot = behind.nonzero(as_tuple=True)
        for pages in (s["k_pages"], s["v_pages"]):
            pages[last[which], slot] = float("nan")
    if own:
        from hstu_jagged_attention_gb300 import binding
        s["binding"] = binding
        s["cache"] = binding.hstu_cache_create(s["k_pages"], s["v_pages"])
        s["batch"] = binding.PagedBatch(s["q_offsets"], s["kv_lens"], s["table"], max_q=case["new"],
                                        num_targets=s["targets"])
        if case["op"] == "attn":
            s["workspace"] = torch.zeros(binding.hstu_cache_workspace_bytes(s["cache"]), device="cuda",
                                         dtype=torch.uint8)
    return s


# ------------------------------------------------------------------ one pass
def run(s):
    return (_run_own if own else _run_plain)[s["case"]["op"]](s)


def _own_append(s):
    c = s["case"]
    q, q_out = (s["q"], s["out"]) if c["with_q"] else (None, None)
    s["binding"].hstu_cache_append(s["cache"], s["batch"], s["k"], s["v"], q=q, q_out=q_out,
                                   rotary=s["rotary"], rotary_pairs=c["pairs"])
    return [s["k_pages"], s["v_pages"]] + ([q_out] if c["with_q"] else [])


def _own_attn(s):
    s["binding"].hstu_attn_fwd_cache(s["cache"], s["batch"], s["q"], s["alpha"], s["inv_n"], s["out"],
                                     workspace=s["workspace"])
    return s["out"]


def _own_norm_fwd(s):
    c = s["case"]
    y, z = s["out"][:2]
    if c["residual"]:
        s["binding"].hstu_norm_fwd(s["x"], s["gamma"], s["beta"], EPS, y, u=s.get("u"),
                                   residual=s["other"], scale=c["scale"], z=z)
        return [y, z]
    s["binding"].hstu_norm_fwd(s["x"], s["gamma"], s["beta"], EPS, y, u=s.get("u"))
    return [y]


def _own_norm_bwd(s):
    c = s["case"]
    dz, du, dx = s["out"]
    dgamma, dbeta = s["sums"]
    more = dict(u=s["u"], du=du) if c["gate"] else {}
    if c["residual"]:
        more.update(dz_in=s["other"], dx=dx, scale=c["scale"])
    s["binding"].hstu_norm_bwd(s["dy"], s["x"], s["gamma"], s["beta"], EPS, dz, dgamma, dbeta,
                               workspace=s["workspace"], **more)
    return [dz, dgamma, dbeta] + ([du] if c["gate"] else []) + ([dx] if c["residual"] else [])


def _turn(x, cos, sin, rot, pairs):
    """x (rows, heads, d) with its first ``rot`` channels rotated."""
    x = x.float()
    if not rot:
        return x
    part = x[..., :rot]
    if pairs:
        a, b = part[..., 0::2], part[..., 1::2]
    else:
        a, b = part[..., :rot // 2], part[..., rot // 2:]
    ra, rb = a * cos - b * sin, b * cos + a * sin
    turned = torch.stack([ra, rb], dim=-1).flatten(-2) if pairs else torch.cat([ra, rb], dim=-1)
    return torch.cat([turned, x[..., rot:]], dim=-1)


def _plain_append(s):
    c, n = s["case"], s["total"]
    rows = torch.arange(n, device="cuda")
    seq = torch.searchsorted(s["q_offsets"][1:].long(), rows, right=True)
    new = (s["q_offsets"][1:] - s["q_offsets"][:-1]).long()[seq]
    kv = s["kv_lens"].long()[seq]
    pos = kv - new + rows - s["q_offsets"].long()[seq]
    page = s["table"].long()[seq, pos // c["page"]]
    slot = pos % c["page"]
    cos = sin = None
    if c["rot"]:
        at = pos if s["targets"] is None else torch.minimum(pos, kv - s["targets"].long()[seq])
        table = s["rotary"][at][:, None, :]
        cos, sin = table[..., :c["rot"] // 2], table[..., c["rot"] // 2:]
    s["k_pages"][page, slot] = _turn(s["k"][:n], cos, sin, c["rot"], c["pairs"]).to(torch.bfloat16)
    s["v_pages"][page, slot] = s["v"][:n]
    if not c["with_q"]:
        return [s["k_pages"], s["v_pages"]]
    s["out"][:n] = _turn(s["q"][:n], cos, sin, c["rot"], c["pairs"]).to(torch.bfloat16)
    return [s["k_pages"], s["v_pages"], s["out"]]


def _plain_attn(s):
    # sequences side by side, padded to the group's longest, as many as fit
    c, first, start = s["case"], 0, np.concatenate([[0], np.cumsum(s["new"])]).tolist()
    while first < c["batch"]:
        last, most_new, most_kv = first, 1, 1
        while last < c["batch"]:
            n, kv = max(most_new, s["new"][last]), max(most_kv, s["hist"][last] + s["new"][last])
            if last > first and (last - first + 1) * kv * c["heads"] * max(n, c["d"]) > 1 << 28:
                break
            last, most_new, most_kv = last + 1, n, kv
        some = slice(first, last)
        kv = s["kv_lens"][some].long()[:, None, None]
        begin = s["q_offsets"][first:last].long()[:, None, None]
        new = s["q_offsets"][first + 1:last + 1].long()[:, None, None] - begin
        hist = kv if s["targets"] is None else kv - s["targets"][some].long()[:, None, None]
        j = torch.arange(most_kv, device="cuda")
        i = torch.arange(most_new, device="cuda")[:, None]
        page = s["table"][some].long()[:, j // c["page"]]
        k = s["k_pages"][page, j % c["page"]].float().permute(0, 2, 3, 1)
        v = s["v_pages"][page, j % c["page"]].float().transpose(1, 2)
        v = torch.where((j < kv)[:, :, :, None], v, 0.0)
        row = (begin + i)[:, :, 0].clamp(max=start[-1] - 1)
        q = s["q"][row].float().transpose(1, 2)
        x = torch.matmul(q, k) * s["alpha"]
        x = x * torch.sigmoid(x)
        p = kv - new + i
        keep = (j <= p) & ((j < hist) | (j == p))
        x = torch.where(keep[:, None], x, 0.0)
        out = (torch.matmul(x, v) * s["inv_n"]).transpose(1, 2).to(torch.bfloat16)
        if most_new == 1:
            s["out"][start[first]:start[last]] = out[:, 0]
        else:
            for b in range(first, last):
                s["out"][start[b]:start[b + 1]] = out[b - first, :s["new"][b]]
        first = last
    return s["out"]


def _standard(z):
    mean = z.mean(dim=1, keepdim=True)
    var = ((z - mean) ** 2).mean(dim=1, keepdim=True)
    rstd = torch.rsqrt(var + EPS)
    return (z - mean) * rstd, rstd


def _plain_norm_fwd(s):
    c = s["case"]
    z = s["x"].float()
    if c["residual"]:
        z = s["other"].float() + c["scale"] * z
    y = _standard(z)[0] * s["gamma"] + s["beta"]
    if c["gate"]:
        y = y * s["u"].float()
    return [y.to(torch.bfloat16)] + ([z.to(torch.bfloat16)] if c["residual"] else [])


def _plain_norm_bwd(s):
    c = s["case"]
    xhat, rstd = _standard(s["x"].float())
    dy = s["dy"].float()
    g = dy * s["u"].float() if c["gate"] else dy
    a = g * s["gamma"]
    dz = rstd * (a - a.mean(dim=1, keepdim=True) - xhat * (a * xhat).mean(dim=1, keepdim=True))
    if c["residual"]:
        dz = dz + s["other"].float()
    out = [dz.to(torch.bfloat16), (g * xhat).sum(dim=0), g.sum(dim=0)]
    if c["gate"]:
        out.append((dy * (xhat * s["gamma"] + s["beta"])).to(torch.bfloat16))
    if c["residual"]:
        out.append((c["scale"] * dz).to(torch.bfloat16))
    return out


_run_plain = dict(append=_plain_append, attn=_plain_attn, norm_fwd=_plain_norm_fwd,
                  norm_bwd=_plain_norm_bwd)
_run_own = dict(append=_own_append, attn=_own_attn, norm_fwd=_own_norm_fwd, norm_bwd=_own_norm_bwd)


# ------------------------------------------------------------------ in 64 bits
def exact(case, seed):
    """What run returns, from the definitions in 64 bits."""
    return dict(append=_exact_append, attn=_exact_attn, norm_fwd=_exact_norm_fwd,
                norm_bwd=_exact_norm_bwd)[case["op"]](case, prepare(case, seed))


def _exact_append(c, s):
    # a rotated pair is a complex number times e^(i angle), the table's cos and sin
    k_pages, v_pages, q_out = s["k_pages"].double(), s["v_pages"].double(), s["out"].double()
    table = s["table"].cpu().numpy()
    rot, half, t = c["rot"], c["rot"] // 2, 0
    first = list(range(0, rot, 2)) if c["pairs"] else list(range(half))
    second = list(range(1, rot, 2)) if c["pairs"] else list(range(half, rot))

    def turned(x, at):
        x = x.double().clone()
        if rot:
            tab = s["rotary"][at].double()[:, None, :]
            z = torch.complex(x[..., first], x[..., second]) * torch.complex(tab[..., :half], tab[..., half:])
            x[..., first], x[..., second] = z.real, z.imag
        return x

    for b, (hist, new, tgt) in enumerate(zip(s["hist"], s["new"], s["tgt"])):
        pos = np.arange(hist, hist + new)
        page = torch.from_numpy(table[b, pos // c["page"]].astype(np.int64)).cuda()
        slot = torch.from_numpy(pos % c["page"]).cuda()
        at = torch.from_numpy(np.minimum(pos, hist + new - tgt) if tgt else pos).cuda()
        k_pages[page, slot] = turned(s["k"][t:t + new], at)
        v_pages[page, slot] = s["v"][t:t + new].double()
        q_out[t:t + new] = turned(s["q"][t:t + new], at)
        t += new
    return [k_pages, v_pages] + ([q_out] if c["with_q"] else [])


def _exact_attn(c, s):
    # per sequence: its causal rows over the keys up to each of them, its
    # candidates over the history and, apart, over themselves
    out, t = s["out"].double(), 0
    silu = lambda x: x / (1.0 + torch.exp(-x))
    for b, (hist, new, tgt) in enumerate(zip(s["hist"], s["new"], s["tgt"])):
        kv, page = hist + new, c["page"]
        j = torch.arange(kv, device="cuda")
        where = s["table"][b].long()[j // page]
        k, v = s["k_pages"][where, j % page].double(), s["v_pages"][where, j % page].double()
        q = s["q"][t:t + new].double()
        seen, plain = kv - tgt, new - tgt  # every candidate sees the keys before `seen`
        if plain:
            w = silu(s["alpha"] * torch.einsum("ihd,jhd->hij", q[:plain], k[:seen]))
            w = w * torch.ones(plain, seen, device="cuda", dtype=torch.float64).tril(hist)
            out[t:t + plain] = s["inv_n"] * torch.einsum("hij,jhd->ihd", w, v[:seen])
        if tgt:
            w = silu(s["alpha"] * torch.einsum("ihd,jhd->hij", q[plain:], k[:seen]))
            one = silu(s["alpha"] * (q[plain:] * k[seen:]).sum(dim=-1, keepdim=True))
            out[t + plain:t + new] = s["inv_n"] * (torch.einsum("hij,jhd->ihd", w, v[:seen]) + one * v[seen:])
        t += new
    return out


def _exact_norm(z):
    n = z.shape[1]
    mean = z.sum(dim=1) / n
    dev = z - mean[:, None]
    return dev / torch.sqrt((dev * dev).sum(dim=1) / n + EPS)[:, None], \
        1.0 / torch.sqrt((dev * dev).sum(dim=1) / n + EPS)[:, None]


def _exact_norm_fwd(c, s):
    z = s["x"].double()
    if c["residual"]:
        z = z * c["scale"] + s["other"].double()
    y = _exact_norm(z)[0] * s["gamma"].double() + s["beta"].double()
    if c["gate"]:
        y = y * s["u"].double()
    return [y] + ([z] if c["residual"] else [])


def _exact_norm_bwd(c, s):
    # the projection form: dz is rstd times the part of a orthogonal to the
    # ones and (but for eps) to the standardised row
    n = c["width"]
    h, rstd = _exact_norm(s["x"].double())
    dy, gamma = s["dy"].double(), s["gamma"].double()
    g = dy * s["u"].double() if c["gate"] else dy
    a = g * gamma
    dz = (a - a.sum(dim=1, keepdim=True) / n - h * torch.einsum("ij,ij->i", a, h)[:, None] / n) * rstd
    if c["residual"]:
        dz = dz + s["other"].double()
    out = [dz, torch.einsum("ij,ij->j", g, h), g.sum(dim=0)]
    if c["gate"]:
        out.append(dy * (h * gamma + s["beta"].double()))
    if c["residual"]:
        out.append(dz * c["scale"])
    return out
