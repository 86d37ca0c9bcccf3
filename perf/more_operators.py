"""What the cache held in 4 bits costs, case by case.

Three operators: appending keys and values to a paged cache of 4-bit codes
(rotated by their position, then quantised) and reading the same tokens back;
reading whole histories back; and the attention over such a cache.  Each case
is computed in a plain form (``own`` false: elementary torch operations in 32
bits) or by the library's kernels (``own`` true).

What is held: 16 neighbouring channels of a token's key or value (rounded to
bf16 after the rotation) share a scale s_j = (8 + j % 8) 2^(j / 8 - 23), the
first of j = 0 .. 255 with 7 s_j >= max |x|; a channel is held as the integer
in -7 .. 7 nearest to x / s_j, ties away from zero.  A page is a row of bytes:
for every head its tiles of min(page, 128) tokens, each tile the keys' codes,
the values' codes, the keys' scales and the values' scales, a token's behind
one another.  In a 32-bit word of 8 channels, channel 2 i is bits 4 i .. 4 i +
3 and channel 2 i + 1 bits 16 + 4 i .. 16 + 4 i + 3, in two's complement.

A case is a dict of plain values.  ``lens`` seeds the sequence lengths, so
that a case's work does not depend on the seed of its values: sequence b has
``hist_lo`` to ``hist_hi`` cached tokens (uniform, or log-normal with median
512 clipped to that range) and ``new_lo`` to ``new`` new ones, of which the
last are candidates (``targets``: 0 none, 1 some, 2 all).
"""
from __future__ import annotations

import math
import random

import numpy as np
import torch

own = False

ROTARY_BASE = 10000.0
GROUP = 16


# ------------------------------------------------------------------ the cases
def _case(name, op, lens, batch, hist_lo, hist_hi, new_lo, new, heads, d, page, targets=0, kind="uniform",
          pad=0, rot=0, pairs=False, with_q=False, fused=False):
    return dict(name=name, op=op, lens=lens, kind=kind, batch=batch, hist_lo=hist_lo, hist_hi=hist_hi,
                new_lo=new_lo, new=new, targets=targets, heads=heads, d=d, page=page, pad=pad, rot=rot,
                pairs=pairs, with_q=with_q, fused=fused)


def listed():
    return [
        # one decode step of a batch of users: 64 sequences append one token each
        _case("write_step", "write", 1, 64, 0, 2047, 1, 1, heads=4, d=64, page=64, rot=64, with_q=True,
              fused=True),
        # filling the cache from 16 whole histories of 4096 tokens, out of the fused projection
        _case("write_histories", "write", 2, 16, 0, 0, 4096, 4096, heads=4, d=64, page=128, rot=64,
              with_q=True, fused=True),
        # histories that grow by a ragged chunk whose last tokens are candidates, a padded batch
        _case("write_chunk", "write", 3, 16, 0, 4190, 100, 700, heads=4, d=128, page=32, targets=1, pad=64,
              rot=64, pairs=True),
        # the smallest reading: one user's short history
        _case("read_one", "read", 4, 1, 0, 0, 513, 513, heads=4, d=64, page=16),
        # 32 users' histories leave the cache for the contiguous forward
        _case("read_histories", "read", 5, 32, 0, 0, 2048, 8192, heads=4, d=64, page=64),
        # the smallest attention call: one user, one token, a short history
        _case("attn_one", "attn", 4, 1, 512, 512, 1, 1, heads=4, d=64, page=16),
        # one decode step of a many-user batch with log-normal lengths
        _case("attn_serving", "attn", 5, 512, 0, 8191, 1, 1, heads=2, d=64, page=64, kind="lognormal"),
        # one decode step of four long sequences: few rows, a long axis
        _case("attn_long", "attn", 6, 4, 10239, 20479, 1, 1, heads=4, d=64, page=128),
        # a few candidates per user against cached histories
        _case("attn_few_candidates", "attn", 7, 8, 2048, 8192, 9, 16, heads=4, d=128, page=32, targets=2),
        # ranking: 1024 candidates per user against histories of 2048 to 8192 tokens
        _case("attn_candidates", "attn", 8, 32, 2048, 8192, 1024, 1024, heads=4, d=64, page=64, targets=2),
        # histories that grow by a ragged chunk, causal within the chunk
        _case("attn_chunk", "attn", 9, 16, 0, 4190, 100, 700, heads=4, d=128, page=64),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1e-9)))))


def draw(rng: random.Random):
    """One more case over the same ranges, no dearer than the largest listed."""
    most = {}
    for c in listed():
        w, (b, f) = work(c), most.get(c["op"], (0, 0))
        most[c["op"]] = (max(b, w["bytes"]), max(f, w["flops"]))
    op = rng.choice(["write", "write", "read", "attn", "attn", "attn"])
    while True:
        c = _case("", op, rng.randrange(1 << 30), _log(rng, 1, 512), 0, _log(rng, 1, 20480), 1, 1,
                  heads=rng.choice([1, 2, 3, 4, 8]), d=rng.choice([32, 64, 128]),
                  page=rng.choice([16, 32, 64, 128, 256]), pad=rng.choice([0, 0, 5, 64]))
        c["hist_lo"] = rng.randrange(0, c["hist_hi"] + 1)
        if op == "read":
            c["hist_lo"] = c["hist_hi"] = 0
            c["new"] = _log(rng, 1, 8192)
        elif rng.random() < 0.6:
            c["new"] = _log(rng, 1, 4096 if op == "write" else 1024)
        c["new_lo"] = rng.randrange(1, c["new"] + 1)
        if op != "read":
            c["targets"] = rng.choice([0, 1, 2])
        if op == "attn":
            c["kind"] = rng.choice(["uniform", "uniform", "lognormal"])
        if op == "write":
            c["rot"] = rng.choice([r for r in (0, 16, 32, 64, 128) if r <= c["d"]])
            c["pairs"], c["with_q"], c["fused"] = (rng.random() < p for p in (0.5, 0.7, 0.5))
        w, (b, f) = work(c), most[op]
        if w["bytes"] <= b and w["flops"] <= max(f, w["bytes"]):
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
    hist, new, tgt = _lengths(case)
    row = case["heads"] * case["d"] * 2  # a token's keys, or values, in bf16
    held = row // 4 + row // 2 // GROUP  # and as they are held
    total = int(new.sum())
    if case["op"] == "read":
        return dict(bytes=2 * total * (row + held), flops=2 * total * row // 2)
    if case["op"] == "write":
        # k and v read, held and read back; q
        turned = total * case["heads"] * case["rot"] * (1 + case["with_q"])
        return dict(bytes=total * (2 * (2 * row + held) + 2 * row * case["with_q"] + 4 * case["rot"]),
                    flops=3 * turned + 4 * total * row // 2)
    kv = hist + new
    keep = kv - tgt  # what every candidate sees, besides itself
    plain = new - tgt
    pairs = int((plain * keep - plain * (plain - 1) // 2 + tgt * (keep + 1)).sum())
    pages = int(((kv + case["page"] - 1) // case["page"]).sum())
    return dict(bytes=2 * held * int(kv.sum()) + 2 * row * total + 4 * pages + 8 * case["batch"],
                flops=4 * pairs * case["heads"] * case["d"])


# ------------------------------------------------------------- what is held
def _scales():
    j = torch.arange(256, device="cuda")
    return (8 + j % 8).float() * 2.0 ** (j // 8 - 23).float()


def _parts(pages, case):
    """(keys' codes, values' codes, keys' scales, values' scales) of the pages,
    each a view (pages, heads, tiles, tokens, bytes)."""
    heads, d, page = case["heads"], case["d"], case["page"]
    t = min(page, 128)
    tiles = pages.view(len(pages), heads, page // t, t * d * 9 // 8)
    cut = [0, t * d // 2, t * d, t * d + t * d // GROUP, t * d + 2 * t * d // GROUP]
    return [tiles[..., a:b].unflatten(-1, (t, -1)) for a, b in zip(cut, cut[1:])]


def _quantise(x):
    """Codes (..., d / 2 bytes) and scales (..., d / 16 bytes) of x (..., d)."""
    g = x.unflatten(-1, (-1, GROUP))
    table = _scales()
    j = torch.searchsorted(7 * table, g.abs().amax(dim=-1)).clamp(max=255)
    s = table[j][..., None]
    code = (torch.floor(g.abs() / s + 0.5).clamp(max=7) * torch.sign(g)).to(torch.int16) & 15
    word = code.flatten(-2).unflatten(-1, (-1, 2, 2, 2))  # of 8 channels: two even and two odd ones, twice
    byte = (word[..., 0, :] | word[..., 1, :] << 4).movedim(-1, -2)  # the even channels' two bytes, then the odd ones'
    return byte.flatten(-3).to(torch.uint8), j.to(torch.uint8)


def _values(codes, scales):
    """What codes (..., d / 2 bytes) and scales (..., d / 16 bytes) stand for."""
    byte = codes.to(torch.int16).unflatten(-1, (-1, 2, 2))  # per word: even, odd
    code = torch.stack([byte & 15, byte >> 4], dim=-1)  # (..., words, even | odd, bytes, low | high)
    code = code.movedim(-3, -1).flatten(-4)
    code = (code ^ 8) - 8
    s = _scales()[scales.long()][..., None]
    return (code.float().unflatten(-1, (-1, GROUP)) * s).flatten(-2)


# ------------------------------------------------------------------ the inputs
def _normal(gen, *shape, sigma=1.0):
    return (torch.randn(*shape, generator=gen, device="cuda", dtype=torch.float32) * sigma).to(torch.bfloat16)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    s = dict(case=case)
    hist, new, tgt = _lengths(case)
    heads, d, page = case["heads"], case["d"], case["page"]
    sigma = 1.0 if d < 128 else 0.5
    kv = hist + new
    n_pages = (kv + page - 1) // page
    order = torch.randperm(int(n_pages.sum()) + 3, generator=gen, device="cuda").cpu().numpy()
    table = np.zeros((case["batch"], int(n_pages.max())), dtype=np.int32)
    at = 0
    for b in range(case["batch"]):
        table[b, :n_pages[b]] = order[at:at + n_pages[b]]
        at += int(n_pages[b])
    total = int(new.sum())
    rows = total + case["pad"]  # a padded batch: rows behind the last sequence
    offsets = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    # slots that were never written may hold anything
    s["pages"] = torch.randint(0, 256, (len(order), heads * page * d * 9 // 8), generator=gen, device="cuda",
                               dtype=torch.uint8)
    s["table"] = torch.from_numpy(table).cuda()
    s["q_offsets"] = torch.from_numpy(offsets).cuda()
    s["kv_lens"] = torch.from_numpy(kv.astype(np.int32)).cuda()
    s["targets"] = torch.from_numpy(tgt.astype(np.int32)).cuda() if case["targets"] else None
    s["hist"], s["new"], s["tgt"], s["total"] = hist.tolist(), new.tolist(), tgt.tolist(), total
    # channels differ in size, as they do behind a trained projection
    gain = torch.exp(0.5 * torch.randn(heads, d, generator=gen, device="cuda"))
    if case["op"] == "write":
        if case["fused"]:  # V, Q and K are quarters of the layer's first projection
            proj = _normal(gen, rows, 4, heads, d, sigma=sigma)
            proj[:, 3] *= gain
            s["v"], s["q"], s["k"] = proj[:, 1], proj[:, 2], proj[:, 3]
        else:
            s["k"], s["v"], s["q"] = (_normal(gen, rows, heads, d, sigma=sigma) for _ in range(3))
            s["k"] *= gain
        s["rotary"] = None
        if case["rot"]:
            angle = np.arange(int(kv.max()), dtype=np.float64)[:, None] * \
                ROTARY_BASE ** (-np.arange(0, case["rot"], 2, dtype=np.float64) / case["rot"])
            both = np.concatenate([np.cos(angle), np.sin(angle)], axis=1).astype(np.float32)
            s["rotary"] = torch.from_numpy(both).cuda()
    else:
        t = min(page, 128)
        parts = _parts(s["pages"], case)
        pos = torch.arange(int(n_pages.max()) * page, device="cuda")
        held = pos[None, :] < s["kv_lens"].long()[:, None]
        seq, pos = held.nonzero(as_tuple=True)
        where = s["table"].long()[seq, pos // page]
        piece = max(1, (1 << 25) // (heads * d))
        for a in range(0, len(pos), piece):
            p = pos[a:a + piece]
            w, sub, r = where[a:a + piece], p % page // t, p % t
            for codes, scales, more in ((parts[0], parts[2], gain), (parts[1], parts[3], 1.0)):
                x = (_normal(gen, len(p), heads, d, sigma=sigma) * more).to(torch.bfloat16)
                codes[w, :, sub, r], scales[w, :, sub, r] = _quantise(x.float())
    shape = (rows, heads, d)
    if case["op"] == "attn":
        s["q"] = _normal(gen, *shape, sigma=sigma)
        s["alpha"], s["inv_n"] = 1.0 / math.sqrt(d), 1.0 / int(kv.max())
    if case["op"] == "attn" or case["with_q"]:
        s["out"] = torch.zeros(*shape, device="cuda", dtype=torch.bfloat16)
    if case["op"] != "attn":
        s["k_back"], s["v_back"] = (torch.zeros(*shape, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    if own:
        from hstu_jagged_attention_gb300 import binding
        s["binding"] = binding
        s["cache"] = binding.hstu_cache_create_q4(s["pages"], page, heads, d)
        s["batch"] = binding.PagedBatch(s["q_offsets"], s["kv_lens"], s["table"], max_q=case["new"],
                                        num_targets=s["targets"])
        if case["op"] == "attn":
            s["workspace"] = torch.zeros(binding.hstu_cache_workspace_bytes(s["cache"]), device="cuda",
                                         dtype=torch.uint8)
    return s


# ------------------------------------------------------------------ one pass
def run(s):
    return (_run_own if own else _run_plain)[s["case"]["op"]](s)


def _own_write(s):
    c = s["case"]
    q, q_out = (s["q"], s["out"]) if c["with_q"] else (None, None)
    s["binding"].hstu_cache_append(s["cache"], s["batch"], s["k"], s["v"], q=q, q_out=q_out,
                                   rotary=s["rotary"], rotary_pairs=c["pairs"])
    s["binding"].hstu_cache_read(s["cache"], s["batch"], s["k_back"], s["v_back"])
    return [s["k_back"], s["v_back"]] + ([q_out] if c["with_q"] else [])


def _own_read(s):
    s["binding"].hstu_cache_read(s["cache"], s["batch"], s["k_back"], s["v_back"])
    return [s["k_back"], s["v_back"]]


def _own_attn(s):
    s["binding"].hstu_attn_fwd_cache(s["cache"], s["batch"], s["q"], s["alpha"], s["inv_n"], s["out"],
                                     workspace=s["workspace"])
    return s["out"]


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


def _tokens(s):
    """Of every new token: its sequence, length, position, page, tile and row."""
    c = s["case"]
    t = min(c["page"], 128)
    rows = torch.arange(s["total"], device="cuda")
    seq = torch.searchsorted(s["q_offsets"][1:].long(), rows, right=True)
    new = (s["q_offsets"][1:] - s["q_offsets"][:-1]).long()[seq]
    kv = s["kv_lens"].long()[seq]
    pos = kv - new + rows - s["q_offsets"].long()[seq]
    return seq, kv, pos, s["table"].long()[seq, pos // c["page"]], pos % c["page"] // t, pos % t


def _plain_write(s):
    c, n = s["case"], s["total"]
    seq, kv, pos, page, tile, row = _tokens(s)
    cos = sin = None
    if c["rot"]:
        at = pos if s["targets"] is None else torch.minimum(pos, kv - s["targets"].long()[seq])
        table = s["rotary"][at][:, None, :]
        cos, sin = table[..., :c["rot"] // 2], table[..., c["rot"] // 2:]
    kc, vc, ks, vs = _parts(s["pages"], c)
    k = _turn(s["k"][:n], cos, sin, c["rot"], c["pairs"]).to(torch.bfloat16)
    kc[page, :, tile, row], ks[page, :, tile, row] = _quantise(k.float())
    vc[page, :, tile, row], vs[page, :, tile, row] = _quantise(s["v"][:n].float())
    out = _plain_read(s, (page, tile, row))
    if not c["with_q"]:
        return out
    s["out"][:n] = _turn(s["q"][:n], cos, sin, c["rot"], c["pairs"]).to(torch.bfloat16)
    return out + [s["out"]]


def _plain_read(s, where=None):
    page, tile, row = where or _tokens(s)[3:]
    kc, vc, ks, vs = _parts(s["pages"], s["case"])
    s["k_back"][:s["total"]] = _values(kc[page, :, tile, row], ks[page, :, tile, row]).to(torch.bfloat16)
    s["v_back"][:s["total"]] = _values(vc[page, :, tile, row], vs[page, :, tile, row]).to(torch.bfloat16)
    return [s["k_back"], s["v_back"]]


def _plain_attn(s):
    # sequences side by side, padded to the group's longest, as many as fit
    c, first, start = s["case"], 0, np.concatenate([[0], np.cumsum(s["new"])]).tolist()
    t = min(c["page"], 128)
    kc, vc, ks, vs = _parts(s["pages"], c)
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
        page, tile, slot = s["table"][some].long()[:, j // c["page"]], j % c["page"] // t, j % t
        k = _values(kc[page, :, tile, slot], ks[page, :, tile, slot]).permute(0, 2, 3, 1)
        v = _values(vc[page, :, tile, slot], vs[page, :, tile, slot]).transpose(1, 2)
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


_run_plain = dict(write=_plain_write, read=_plain_read, attn=_plain_attn)
_run_own = dict(write=_own_write, read=_own_read, attn=_own_attn)


# ------------------------------------------------------------------ in 64 bits
def exact(case, seed):
    """What run returns, from the definitions in 64 bits."""
    return dict(write=_exact_write, read=_exact_read, attn=_exact_attn)[case["op"]](case, prepare(case, seed))


def _exact_held(x):
    # the integers below 8 times the least scale that holds them, in 64 bits
    g = x.double().unflatten(-1, (-1, GROUP))
    most = g.abs().amax(dim=-1, keepdim=True) / 7
    e = torch.floor(torch.log2(most.clamp(min=2.0 ** -20)))
    e = torch.where(torch.exp2(e) > most, e - 1, torch.where(torch.exp2(e + 1) <= most, e + 1, e)).clamp(min=-20)
    eighth = torch.exp2(e - 3)
    s = (torch.ceil(most / eighth).clamp(min=8) * eighth).clamp(2.0 ** -20, 1.875 * 2.0 ** 11)
    q = torch.trunc(g / s + torch.where(g < 0, -0.5, 0.5)).clamp(-7, 7)
    return (q * s).flatten(-2)


def _exact_write(c, s):
    # a rotated pair is a complex number times e^(i angle), the table's cos and sin
    rot, half, t = c["rot"], c["rot"] // 2, 0
    first = list(range(0, rot, 2)) if c["pairs"] else list(range(half))
    second = list(range(1, rot, 2)) if c["pairs"] else list(range(half, rot))
    outs = [s["k_back"].double(), s["v_back"].double()] + ([s["out"].double()] if c["with_q"] else [])

    def turned(x, at):
        x = x.double().clone()
        if rot:
            tab = s["rotary"][at].double()[:, None, :]
            z = torch.complex(x[..., first], x[..., second]) * torch.complex(tab[..., :half], tab[..., half:])
            x[..., first], x[..., second] = z.real, z.imag
        return x

    for hist, new, tgt in zip(s["hist"], s["new"], s["tgt"]):
        pos = np.arange(hist, hist + new)
        at = torch.from_numpy(np.minimum(pos, hist + new - tgt) if tgt else pos).cuda()
        outs[0][t:t + new] = _exact_held(turned(s["k"][t:t + new], at).to(torch.bfloat16))
        outs[1][t:t + new] = _exact_held(s["v"][t:t + new])
        if c["with_q"]:
            outs[2][t:t + new] = turned(s["q"][t:t + new], at)
        t += new
    return outs


def _exact_rows(c, s, b, n0, n1):
    """Keys and values of tokens n0 .. n1 - 1 of sequence b, (tokens, heads, d)
    each, from the bytes' places in a page."""
    heads, d, page = c["heads"], c["d"], c["page"]
    t = min(page, 128)
    tile = t * d * 9 // 8
    p = torch.arange(n0, n1, device="cuda")[:, None, None]
    h = torch.arange(heads, device="cuda")[:, None]
    ch = torch.arange(d, device="cuda")
    base = s["table"][b].long()[p // page] * (heads * (page // t) * tile) + (h * (page // t) + p % page // t) * tile
    flat, out = s["pages"].view(-1), []
    for which in (0, 1):
        at = base + which * (t * d // 2) + p % t * (d // 2) + ch // 8 * 4 + ch % 2 * 2 + ch % 8 // 4
        nibble = torch.where(ch % 4 // 2 == 0, flat[at] % 16, flat[at] // 16).double()
        nibble = torch.where(nibble >= 8, nibble - 16, nibble)
        j = flat[base + t * d + which * (t * d // GROUP) + p % t * (d // GROUP) + ch // GROUP].double()
        octave = torch.floor(j / 8)
        out.append(nibble * (1 + (j - 8 * octave) / 8) * torch.exp2(octave - 20))
    return out


def _exact_read(c, s):
    k, v, t = s["k_back"].double(), s["v_back"].double(), 0
    for b, (hist, new) in enumerate(zip(s["hist"], s["new"])):
        k[t:t + new], v[t:t + new] = _exact_rows(c, s, b, hist, hist + new)
        t += new
    return [k, v]


def _exact_attn(c, s):
    # per sequence: its causal rows over the keys up to each of them, its
    # candidates over the history and, apart, over themselves
    out, t = s["out"].double(), 0
    silu = lambda x: x / (1.0 + torch.exp(-x))
    for b, (hist, new, tgt) in enumerate(zip(s["hist"], s["new"], s["tgt"])):
        kv = hist + new
        k, v = _exact_rows(c, s, b, 0, kv)
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
