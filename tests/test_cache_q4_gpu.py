"""The cache of 4-bit codes on the GPU: what the append holds, what the reading
gives back and the attention over it, against the 64-bit forms of
oracle/layer.py, and what a caller may do with them.

What is held is compared bit for bit: it is a rule on bf16 numbers.  Keys that
were rotated first are compared with the rule on the fp32 rotation rounded to
bf16 (two products and a sum, each rounded, as numpy computes them), and with
the 64-bit rotation within the rotation's error, 2^-8 |x| + 2^-22 of the
products' sizes, and half a step of the codes: s / 2, s the scale held.
Tolerance of the attention over what is held: as the bf16 cache's
(tests/test_cache_gpu.py), for the operations are the same.
"""
import numpy as np
import pytest
import torch

from hstu_jagged_attention_gb300 import binding, build, workloads
from oracle import layer
from tests.test_cache import make_batch
from tests.test_cache_gpu import SHAPES, Setup, randn, rotary_table

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()
    binding.hstu_set_wait_timeout_ns(0)
    yield


@pytest.fixture(autouse=True)
def _status():
    binding.hstu_last_status()
    yield
    assert binding.hstu_last_status() == (binding.HSTU_OK, 0)


class Q4(Setup):
    """Setup's batch over a pool of codes: kp and vp are what the pool holds,
    and slots that no sequence holds are any bytes."""

    def __init__(self, *args, seed=0, garbage=0, **kw):
        super().__init__(*args, seed=seed, nan_tail=False, **kw)
        # channels of different sizes; few groups near the scale's ends
        gain = np.exp(0.7 * np.random.default_rng(seed).standard_normal((self.heads, self.d)))
        kp, vp = layer.f64(self.kp) * gain, layer.f64(self.vp)
        kp[:, ::5] *= 2.0 ** -6
        vp[:, ::7, :, 16:] = 0.0
        self.bytes = layer.q4_pack(torch.from_numpy(kp).bfloat16(), torch.from_numpy(vp).bfloat16())
        self.fill_unused(garbage)
        kp, vp = layer.q4_unpack(self.bytes, self.page, self.heads, self.d)
        self.kp, self.vp = torch.from_numpy(kp).bfloat16(), torch.from_numpy(vp).bfloat16()
        self.pages = torch.from_numpy(self.bytes).cuda()
        self.cache = binding.hstu_cache_create_q4(self.pages, self.page, self.heads, self.d)

    def fill_unused(self, garbage):
        kv, table = self.host.keep["kv_lens"], self.host.keep["page_table"]
        used = np.zeros((self.num_pages, self.page), dtype=bool)
        for b, n in enumerate(kv):
            p = np.arange(n)
            used[table[b, p // self.page], p % self.page] = True
        codes, _, scales = layer._q4_places(self.page, self.heads, self.d)
        rng = np.random.default_rng(1000 + garbage)
        for at in (*codes, *scales):
            for page in range(self.num_pages):
                spots = np.unique(at[~used[page]])
                self.bytes[page, spots] = rng.integers(0, 256, len(spots)) if garbage < 2 else 255

    def held(self):
        return layer.q4_unpack(self.pages.cpu().numpy(), self.page, self.heads, self.d)

    def slots(self):
        """(row, page, slot, position, hist) of every new token."""
        a = self.host.keep
        off, kv, table, nt = a["q_offsets"], a["kv_lens"], a["page_table"], a.get("num_targets")
        for b in range(len(kv)):
            n = off[b + 1] - off[b]
            for i in range(n):
                p = kv[b] - n + i
                yield off[b] + i, table[b, p // self.page], p % self.page, p, kv[b] - (0 if nt is None else nt[b])

    def read(self, **kw):
        k, v = (torch.full((self.rows, self.heads, self.d), 7.0, device="cuda", dtype=torch.bfloat16)
                for _ in range(2))
        binding.hstu_cache_read(self.cache, self.batch, k, v, **kw)
        return k, v


GEOMETRY = [(32, 3, 16), (64, 2, 64), (128, 1, 32), (64, 1, 256), (32, 2, 128), (128, 2, 16)]


class Bf16(Setup):
    """Setup's bf16 pools, with what Q4 offers."""
    slots = Q4.slots
    read = Q4.read


# ------------------------------------------------------------------- reading
@pytest.mark.parametrize("kind", [Q4, Bf16])
@pytest.mark.parametrize("d,heads,page", GEOMETRY + [(64, 5, 512)])
@pytest.mark.parametrize("name", SHAPES)
def test_read(name, d, heads, page, kind):
    hist, new, nt = SHAPES[name]
    s = kind(hist, new, page, heads, d, nt, seed=d + page, pad=2)
    k, v = s.read()
    for t, pg, slot, _, _ in s.slots():
        assert torch.equal(k[t].cpu(), s.kp[pg, slot]) and torch.equal(v[t].cpu(), s.vp[pg, slot])
    assert (k[s.total:] == 7).all() and (v[s.total:] == 7).all()


def test_bad_lengths_and_pages_of_a_bf16_cache_are_reported_by_the_reading():
    s = Bf16([100, 40, 70], [2, 20, 1], 16, 2, 64, seed=7)
    good = s.read()
    assert binding.hstu_last_status() == (binding.HSTU_OK, 0)
    for name, at, value, rows in (("kv_lens", 1, -1, slice(2, 22)), ("page_table", (1, 3), -1, slice(10, 22)),
                                  ("page_table", (1, 3), s.num_pages, slice(10, 22))):
        old = s.dev[name][at].clone()
        s.dev[name][at] = value
        k, v = s.read()
        assert binding.hstu_last_status()[0] == binding.HSTU_ERR_INVALID_ARG
        s.dev[name][at] = old
        for x, y in zip((k, v), good):
            left = 7 if name == "kv_lens" else 0  # not written, or read as zeros
            assert (x[rows] == left).all()
            assert torch.equal(x[:rows.start], y[:rows.start]) and torch.equal(x[22:], y[22:])


@pytest.mark.parametrize("q4", [True, False])
def test_read_whole_histories_into_slices(q4):
    kv = [300, 0, 17, 64]
    s = (Q4 if q4 else Setup)([0] * 4, kv, 32, 2, 64, seed=3, pad=3)
    both = torch.full((s.rows, 3, 2, 64), 7.0, device="cuda", dtype=torch.bfloat16)
    binding.hstu_cache_read(s.cache, s.batch, both[:, 0], both[:, 2])
    table, t = s.host.keep["page_table"], 0
    for b, n in enumerate(kv):
        p = np.arange(n)
        at = torch.from_numpy(table[b, p // 32].astype(np.int64)), torch.from_numpy(p % 32)
        assert torch.equal(both[t:t + n, 0].cpu(), s.kp[at]) and torch.equal(both[t:t + n, 2].cpu(), s.vp[at])
        t += n
    assert (both[:, 1] == 7).all() and (both[t:] == 7).all()


# ------------------------------------------------------------------ appending
def rotated_fp32(x, table, at, pairs):
    """x (heads, d) float32, rotated as the append does, rounded to bf16."""
    y, half = x.copy(), table.shape[1] // 2
    i = np.arange(half)
    a, b = (2 * i, 2 * i + 1) if pairs else (i, half + i)
    c, s = table[at, :half], table[at, half:]
    y[:, a], y[:, b] = x[:, a] * c - x[:, b] * s, x[:, b] * c + x[:, a] * s
    return torch.from_numpy(y).bfloat16().float().numpy()


@pytest.mark.parametrize("d,heads,page,rot,pairs", [(64, 2, 16, 64, False), (64, 3, 64, 32, True),
                                                    (32, 1, 32, 16, False), (128, 2, 128, 128, True),
                                                    (128, 1, 16, 96, False), (64, 2, 32, 0, False),
                                                    (64, 1, 256, 48, False), (32, 4, 16, 32, True),
                                                    (128, 3, 32, 80, False), (32, 2, 64, 32, False)])
@pytest.mark.parametrize("name", SHAPES)
def test_append(name, d, heads, page, rot, pairs):
    hist, new, nt = SHAPES[name]
    s = Q4(hist, new, page, heads, d, nt, seed=d + rot, pad=2)
    table = rotary_table(int(s.host.keep["kv_lens"].max()) + 1, rot) if rot else None
    q_out = torch.full((s.rows, heads, d), 7.0, device="cuda", dtype=torch.bfloat16)
    binding.hstu_cache_append(s.cache, s.batch, s.k.cuda(), s.v.cuda(), q=s.q.cuda(), q_out=q_out,
                              rotary=None if table is None else table.cuda(), rotary_pairs=pairs)
    got = s.pages.cpu().numpy()
    held_k, held_v = s.held()
    touched = np.zeros((s.num_pages, page), dtype=bool)
    size = 2.0 * max(layer.f64(s.k).__abs__().max(initial=0), layer.f64(s.q).__abs__().max(initial=0))
    for t, pg, slot, pos, seen in s.slots():
        touched[pg, slot] = True
        k, q = layer.f64(s.k[t]), layer.f64(s.q[t])
        kr = k if table is None else rotated_fp32(s.k[t].float().numpy(), table.numpy(), min(pos, seen), pairs)
        assert np.array_equal(held_k[pg, slot], layer.q4_held(kr)), (t, "keys")
        assert np.array_equal(held_v[pg, slot], layer.q4_held(s.v[t])), (t, "values")
        if table is not None:
            k, q = (layer.rotate(x, min(pos, seen), layer.f64(table), pairs) for x in (k, q))
        step = np.repeat(layer.SCALES[layer.q4_codes(kr)[1]], 16, axis=-1)
        assert np.all(np.abs(held_k[pg, slot] - k) <= step / 2 + 2.0 ** -8 * np.abs(k) + 2.0 ** -22 * size)
        err = np.abs(layer.f64(q_out[t]) - q)
        assert np.all(err <= (2.0 ** -8 * np.abs(q) + 2.0 ** -22 * size if rot else 0.0))
    assert np.all(layer.f64(q_out)[s.total:] == 7.0)
    # every other byte is as it was
    codes, _, scales = layer._q4_places(page, heads, d)
    for at in (*codes, *scales):
        for pg in range(s.num_pages):
            keep = np.unique(at[~touched[pg]])
            assert np.array_equal(got[pg, keep], s.bytes[pg, keep])
    k, v = s.read()
    for t, pg, slot, _, _ in s.slots():
        assert np.array_equal(layer.f64(k[t]), held_k[pg, slot])
        assert np.array_equal(layer.f64(v[t]), held_v[pg, slot])


def test_append_of_every_kind_of_number():
    s = Q4([0, 3], [200, 91], 64, 2, 64, seed=5)
    rng = np.random.default_rng(5)
    x = rng.standard_normal((s.rows, 2, 64)) * np.exp(rng.uniform(-20, 12, size=(s.rows, 2, 1)))
    for _ in range(400):  # ties: (n + 1/2) s beside 7 s in a group
        t, h, g = rng.integers(s.rows), rng.integers(2), 16 * rng.integers(4)
        sc = layer.SCALES[rng.integers(60, 250)]
        x[t, h, g:g + 16] = sc * (rng.integers(-7, 7, size=16) + 0.5)
        x[t, h, g + rng.integers(16)] = 7 * sc
    x[0] = 0.0
    x[1, 0, ::3] = np.nan
    x[2, 1, 5], x[2, 1, 20] = np.inf, -np.inf
    x[3] = np.nan
    x[4] = 3e38
    x[5] = -1e-30
    x[6, :, 1::2] = 5e-7
    x[7] = 7 * 3840.0
    k = torch.from_numpy(x).bfloat16()
    v = -k.flip(0).contiguous()
    with np.errstate(invalid="ignore"):
        ref_k, ref_v = layer.q4_held(k), layer.q4_held(v)
    assert np.any(ref_k == 26880.0) and np.any(ref_v == 2.0 ** -20)
    for positions in (None, rotary_table(300, 64) * 0 + torch.tensor([1.0] * 32 + [0.0] * 32)):
        s.pages.fill_(3)
        args = {} if positions is None else dict(rotary=positions.cuda())
        kk = k if positions is None else k.nan_to_num(nan=1.0, posinf=2.0, neginf=2.0)  # 0 x inf is NaN
        binding.hstu_cache_append(s.cache, s.batch, kk.cuda(), v.cuda(), **args)
        held_k, held_v = s.held()
        for t, pg, slot, _, _ in s.slots():
            assert np.array_equal(held_k[pg, slot], ref_k[t] if positions is None else layer.q4_held(kk[t])), t
            assert np.array_equal(held_v[pg, slot], ref_v[t]), t


def test_append_from_a_fused_projection_and_in_place():
    s = Q4([10, 300, 0], [5, 1, 90], 32, 2, 64, [2, 0, 90], seed=9, pad=4)
    table = rotary_table(512, 64).cuda()
    q_out = torch.zeros(s.rows, 2, 64, device="cuda", dtype=torch.bfloat16)
    binding.hstu_cache_append(s.cache, s.batch, s.k.cuda(), s.v.cuda(), q=s.q.cuda(), q_out=q_out,
                              rotary=table)
    first = s.pages.clone()
    s.pages.copy_(torch.from_numpy(s.bytes))
    proj = torch.stack([s.v, s.q, s.v, s.k], dim=1).cuda()
    q2 = torch.zeros_like(q_out)
    binding.hstu_cache_append(s.cache, s.batch, proj[:, 3], proj[:, 2], q=proj[:, 1], q_out=q2, rotary=table)
    assert torch.equal(q_out, q2) and torch.equal(first, s.pages)
    q3 = s.q.cuda()
    binding.hstu_cache_append(s.cache, s.batch, s.k.cuda(), s.v.cuda(), q=q3, q_out=q3, rotary=table)
    assert torch.equal(q3[:s.total], q_out[:s.total]) and torch.equal(first, s.pages)
    assert torch.equal(q3[s.total:].cpu(), s.q[s.total:])  # a padded batch's rows stay


@pytest.mark.parametrize("d,heads,page,rot,pairs", [(32, 31, 16, 16, False), (64, 7, 256, 48, False),
                                                    (128, 5, 64, 96, True), (64, 13, 32, 0, False)])
def test_more_rows_than_warps(d, heads, page, rot, pairs):
    # warps that take several heads, the last of them fewer
    kv = [1700, 0, 2300, 1, 900]
    s = Q4([0] * 5, kv, page, heads, d, [0, 0, 300, 1, 900], seed=16 + d, pad=5)
    table = rotary_table(2400, rot) if rot else None
    q_out = torch.full((s.rows, heads, d), 7.0, device="cuda", dtype=torch.bfloat16)
    binding.hstu_cache_append(s.cache, s.batch, s.k.cuda(), s.v.cuda(), q=s.q.cuda(), q_out=q_out,
                              rotary=None if table is None else table.cuda(), rotary_pairs=pairs)
    k_back, v_back = s.read()
    at = np.concatenate([np.minimum(np.arange(n), n - t) for n, t in zip(kv, [0, 0, 300, 1, 900])])
    n, half = s.total, rot // 2
    for x, got, held in ((s.q, q_out, lambda y: y), (s.k, k_back, layer.q4_held)):
        x = x[:n].float().numpy()
        y = x.copy()
        if rot:
            c, sn = table.numpy()[at, None, :half], table.numpy()[at, None, half:]
            a, b = (slice(0, rot, 2), slice(1, rot, 2)) if pairs else (slice(0, half), slice(half, rot))
            y[..., a], y[..., b] = x[..., a] * c - x[..., b] * sn, x[..., b] * c + x[..., a] * sn
        assert np.array_equal(layer.f64(got)[:n], held(layer.f64(torch.from_numpy(y).bfloat16())))
    assert np.array_equal(layer.f64(v_back)[:n], layer.q4_held(s.v[:n]))
    assert all((x[n:] == 7).all() for x in (q_out, k_back, v_back))


@pytest.mark.parametrize("pairs", [False, True])
def test_the_rotation_rounds_each_product(pairs):
    # enough values that a fused product would show
    s = Q4([0] * 4, [4000] * 4, 128, 1, 64, seed=15)
    table = rotary_table(4000, 64)
    q_out = torch.zeros(s.rows, 1, 64, device="cuda", dtype=torch.bfloat16)
    binding.hstu_cache_append(s.cache, s.batch, s.k.cuda(), s.v.cuda(), q=s.q.cuda(), q_out=q_out,
                              rotary=table.cuda(), rotary_pairs=pairs)
    k_back, _ = s.read()
    at = np.tile(np.arange(4000), 4)
    c, sn = table.numpy()[at, None, :32], table.numpy()[at, None, 32:]
    a, b = (slice(0, 64, 2), slice(1, 64, 2)) if pairs else (slice(0, 32), slice(32, 64))
    for x, got, held in ((s.q, q_out, lambda y: y), (s.k, k_back, layer.q4_held)):
        x = x.float().numpy()
        y = np.empty_like(x)
        y[..., a], y[..., b] = x[..., a] * c - x[..., b] * sn, x[..., b] * c + x[..., a] * sn
        assert np.array_equal(layer.f64(got), held(layer.f64(torch.from_numpy(y).bfloat16())))


@pytest.mark.parametrize("pairs", [False, True])
def test_queries_rotated_beside_either_cache(pairs):
    # the same queries: fl(fl(x c) -+ fl(y s)) beside a cache of codes, and
    # maybe fl(x c -+ fl(y s)) beside the other: 2^-24 |x c| and two roundings of
    # the sum apart, 2^-22 (|x c| + |y s|) at most, then rounded to bf16 each
    kinds = [kind([0] * 4, [4000] * 4, 128, 1, 64, seed=18) for kind in (Q4, Bf16)]
    table, outs = rotary_table(4000, 64), []
    for s in kinds:
        outs.append(torch.full((s.rows, 1, 64), 7.0, device="cuda", dtype=torch.bfloat16))
        binding.hstu_cache_append(s.cache, s.batch, s.k.cuda(), s.v.cuda(), q=kinds[0].q.cuda(), q_out=outs[-1],
                                  rotary=table.cuda(), rotary_pairs=pairs)
    x, y = (layer.f64(o) for o in outs)
    at = np.tile(np.arange(4000), 4)
    c, sn = layer.f64(table)[at, None, :32], layer.f64(table)[at, None, 32:]
    a, b = (slice(0, 64, 2), slice(1, 64, 2)) if pairs else (slice(0, 32), slice(32, 64))
    q, size = layer.f64(kinds[0].q), np.empty_like(x)
    size[..., a] = np.abs(q[..., a] * c) + np.abs(q[..., b] * sn)
    size[..., b] = np.abs(q[..., b] * c) + np.abs(q[..., a] * sn)
    assert np.all(np.abs(x - y) <= 2.0 ** -22 * size + 2.0 ** -8 * (np.abs(x) + np.abs(y)))


def test_every_sequence_is_checked():
    # more sequences than a CTA of the check has threads, wrong ones among them
    n = 700
    s = Q4([3] * n, [1] * n, 16, 1, 32, seed=8)
    good = s.read()
    binding.hstu_cache_append(s.cache, s.batch, s.k.cuda(), s.v.cuda())
    assert binding.hstu_last_status() == (binding.HSTU_OK, 0)
    for b in (0, 127, 128, 255, 256, 511, 699):
        s.pages.copy_(torch.from_numpy(s.bytes))
        s.dev["kv_lens"][b] = -1
        k, v = s.read()
        assert binding.hstu_last_status()[0] == binding.HSTU_ERR_INVALID_ARG
        assert (k[b] == 7).all() and torch.equal(k[b + 1:], good[0][b + 1:]) and torch.equal(v[:b], good[1][:b])
        binding.hstu_cache_append(s.cache, s.batch, s.k.cuda(), s.v.cuda())
        assert binding.hstu_last_status()[0] == binding.HSTU_ERR_INVALID_ARG
        s.dev["kv_lens"][b] = 4
        held = s.held()[0]
        for t, pg, slot, _, _ in s.slots():
            ref = s.kp[pg, slot] if t == b else layer.q4_held(s.k[t])
            assert np.array_equal(held[pg, slot], layer.f64(ref))


# ------------------------------------------------------------------ attention
@pytest.mark.parametrize("d,heads,page", GEOMETRY)
@pytest.mark.parametrize("name", SHAPES)
@pytest.mark.parametrize("wide", [False, True])
def test_attention_parity(wide, name, d, heads, page):
    # wide: a table for 10,000 tokens, so that few items share the GPU evenly
    # instead of taking a cluster each
    hist, new, nt = SHAPES[name]
    s = Q4(hist, new, page, heads, d, nt, seed=len(name) + d, pad=3, width=10000 // page if wide else 1)
    s.check(s.attend())


def test_many_items():
    # more items than clusters run at once, of one to seven blocks
    rng = np.random.default_rng(50)
    hist, new = rng.integers(0, 850, size=60), rng.integers(0, 4, size=60)
    s = Q4(hist, new, 32, 2, 64, rng.integers(0, new + 1), seed=50)
    s.check(s.attend())


# a table of 2000 pages of 64 asks for 128-row tiles where a bound of more than
# 32 new tokens allows them
@pytest.mark.parametrize("width", [1, 2000])
@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("new,targets,max_q", [(33, 0, None), (47, 47, None), (64, 20, None), (9, 3, 130),
                                               (130, 0, None), (200, 200, None), (257, 9, None)])
def test_several_tiles(d, new, targets, max_q, width):
    s = Q4([0, 140, 300], [new, 1, 17], 64, 2, d, [targets, 0, 17], seed=30 + d, max_q=max_q, width=width)
    s.check(s.attend())


@pytest.mark.parametrize("d,heads,page", GEOMETRY + [(64, 3, 512), (128, 1, 4096)])
@pytest.mark.parametrize("name", SHAPES)
def test_few_rows_on_large_tiles(name, d, heads, page):
    # a bound on the new tokens and a table that ask for 128-row tiles
    hist, new, nt = SHAPES[name]
    s = Q4(hist, new, page, heads, d, nt, seed=20 + d, pad=140, max_q=140, width=200000 // page)
    s.check(s.attend())


@pytest.mark.parametrize("max_q", [1, 4, 16, 32, 33, 500, 2 ** 31 - 1])
def test_max_q_changes_the_tiling_not_the_result(max_q):
    s = Q4([90, 300, 5], [1, 1, 1], 32, 2, 64, seed=1, max_q=max_q)
    s.check(s.attend())


@pytest.mark.parametrize("width", [1, 200])
@pytest.mark.parametrize("new", [1, 5, 8, 9, 40, 130])
def test_long_cache_few_rows(new, width):
    # one sequence and one head over a cluster or the whole GPU: many parts a row
    s = Q4([6000], [new], 64, 1, 64, [new], seed=2, width=width)
    ws = s.workspace()
    a = s.attend(workspace=ws)
    assert not ws[:8192].any(), "the workspace is ready for the next call"
    s.check(a)
    for _ in range(3):  # parts are summed in a fixed order
        assert torch.equal(a, s.attend(workspace=ws))
    assert torch.equal(a, s.attend())  # without a workspace


def test_strided_queries_and_padded_pages():
    s = Q4([100, 20], [4, 20], 16, 2, 64, seed=3)
    wide = torch.randn(s.rows, 4, 2, 64, device="cuda").bfloat16()
    wide[:, 2] = s.q.cuda()
    a = s.attend()
    assert torch.equal(a, s.attend(q=wide[:, 2]))
    n = s.pages.shape[1]
    pool = torch.full((s.num_pages, n + 48), 9, device="cuda", dtype=torch.uint8)
    pool[:, :n] = s.pages
    s.cache = binding.hstu_cache_create_q4(pool[:, :n], 16, 2, 64)
    assert torch.equal(a, s.attend())
    binding.hstu_cache_append(s.cache, s.batch, s.k.cuda(), s.v.cuda())
    other = Q4([100, 20], [4, 20], 16, 2, 64, seed=3)
    binding.hstu_cache_append(other.cache, other.batch, s.k.cuda(), s.v.cuda())
    assert torch.equal(pool[:, :n], other.pages) and (pool[:, n:] == 9).all()
    assert all(torch.equal(x, y) for x, y in zip(s.read(), other.read()))


def test_a_pool_past_32_bits():
    # page numbers whose byte offsets need more than 32 bits
    s = Q4([300, 5], [3, 1], 64, 2, 64, seed=4)
    n = s.pages.shape[1]
    pages = (1 << 32) // n + s.num_pages + 1
    big = torch.empty(pages, n, device="cuda", dtype=torch.uint8)
    move = pages - s.num_pages
    big[move:] = s.pages
    a, kv = s.attend(), s.read()
    s.cache = binding.hstu_cache_create_q4(big, 64, 2, 64)
    s.dev["page_table"].add_(move)
    assert torch.equal(a, s.attend())
    assert all(torch.equal(x, y) for x, y in zip(kv, s.read()))
    k, v = s.k.cuda(), s.v.cuda()
    binding.hstu_cache_append(s.cache, s.batch, k, v)
    small = Q4([300, 5], [3, 1], 64, 2, 64, seed=4)
    binding.hstu_cache_append(small.cache, small.batch, k, v)
    assert torch.equal(big[move:], small.pages)


@pytest.mark.parametrize("new,width", [([1, 2, 1, 40], 1), ([130, 2, 1, 40], 1), ([130, 2, 1, 40], 2000)])
def test_bytes_past_the_end_never_matter(new, width):
    outs = [Q4([100, 63, 0, 30], new, 64, 2, 64, [0, 2, 1, 5], seed=5, garbage=g, width=width).attend()
            for g in range(3)]
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])


def test_a_shared_prefix_is_read_from_shared_pages():
    s = Q4([128, 128, 128], [2, 1, 3], 32, 2, 64, seed=6)
    table = s.host.keep["page_table"]
    table[1, :4] = table[2, :4] = table[0, :4]
    s.dev["page_table"].copy_(torch.from_numpy(table))
    s.check(s.attend())


@pytest.mark.parametrize("new", [[2, 2, 1], [70, 2, 130]])
@pytest.mark.parametrize("page,width", [(16, 1), (16, 600), (16, 8000), (128, 1), (256, 500)])
def test_bad_lengths_and_pages_are_skipped_and_reported(page, width, new):
    s = Q4([100, 340, 70], new, page, 1, 64, seed=7, width=width)
    good, whole = s.attend(), s.read()
    o = np.concatenate([[0], np.cumsum(new)])

    def run(name, at, value, read_meets_it=True):
        t = s.dev[name]
        old = t[at].clone()
        t[at] = value
        out = s.attend()
        status = [binding.hstu_last_status()[0]]
        kv = s.read()
        status.append(binding.hstu_last_status()[0])
        t[at] = old
        bad = binding.HSTU_ERR_INVALID_ARG
        assert status == [bad, bad if read_meets_it else binding.HSTU_OK]
        for x, y in zip((out, *kv), (good, *whole)):
            assert torch.equal(x[:o[1]], y[:o[1]]) and torch.equal(x[o[2]:], y[o[2]:])
        return out, kv

    for name, at, value in (("kv_lens", 1, 1), ("kv_lens", 1, 10 ** 6), ("kv_lens", 1, -5)):
        out, kv = run(name, at, value)
        assert all((x[o[1]:o[2]] == 7).all() for x in (out, *kv))
    bad = s.host.keep["page_table"][1, 0]
    keep = s.pages[bad].clone()
    s.pages[bad] = 0  # the page's keys add nothing: as if it held zeros
    ref = s.attend()
    s.pages[bad] = keep
    for value in (-1, s.num_pages, 2 ** 31 - 1, -2 ** 31):
        out, kv = run("page_table", (1, 0), value, read_meets_it=False)  # the new tokens are elsewhere
        assert torch.equal(out, ref)
    last = (342 - 1) // page
    _, kv = run("page_table", (1, last), -1)
    t = np.arange(o[1], o[2])[340 + np.arange(2) >= last * page]
    assert all((x[t] == 0).all() for x in kv)
    # an append to a bad page, or past the rotation's table, is dropped
    k, v = s.k.cuda(), s.v.cuda()
    old = s.dev["page_table"][1, last].clone()
    for bad_page in (True, False):
        s.pages.copy_(torch.from_numpy(s.bytes))
        if bad_page:
            s.dev["page_table"][1, last] = -3
        binding.hstu_cache_append(s.cache, s.batch, k, v,
                                  rotary=None if bad_page else rotary_table(341, 32).cuda())
        assert binding.hstu_last_status()[0] == binding.HSTU_ERR_INVALID_ARG
        s.dev["page_table"][1, last] = old
        now = s.held()
        for t, pg, slot, pos, _ in s.slots():
            kept = o[1] <= t < o[2] and (pos // page == last if bad_page else pos >= 341)
            assert np.array_equal(now[1][pg, slot], layer.f64(s.vp[pg, slot]) if kept else layer.q4_held(s.v[t]))


@pytest.mark.parametrize("new,width", [(1, 1), (40, 1), (130, 1), (130, 8000)])
def test_rows_before_the_first_sequence_stay(new, width):
    s = Q4([100, 0, 700], [3, new, 1], 16, 2, 64, seed=81, width=width)
    good, kv = s.attend(), s.read()
    s.dev["q_offsets"].add_(4)
    lead = torch.full((4, 2, 64), float("nan"), device="cuda", dtype=torch.bfloat16)
    pad = lambda x: torch.cat([lead, x.cuda(), lead[:1]])
    outs = [torch.full((s.rows + 5, 2, 64), 7.0, device="cuda", dtype=torch.bfloat16) for _ in range(4)]
    s.attend(q=pad(s.q), out=outs[0])
    binding.hstu_cache_read(s.cache, s.batch, *outs[1:3])
    for x, y in zip(outs, (good, *kv)):
        assert torch.equal(x[4:-1], y) and (x[:4] == 7).all() and (x[-1] == 7).all()
    binding.hstu_cache_append(s.cache, s.batch, pad(s.k), pad(s.v), q=pad(s.q), q_out=outs[3])
    assert torch.equal(outs[3][4:-1].cpu(), s.q) and (outs[3][:4] == 7).all() and (outs[3][-1] == 7).all()
    held = s.held()
    for t, pg, slot, _, _ in s.slots():
        assert np.array_equal(held[0][pg, slot], layer.q4_held(s.k[t]))


# table widths (pages of 16) and new tokens that send a call to each of the
# kernels: clusters and shares of 16-row tiles, 128-row tiles
FORMS = [(1, [1, 1, 1]), (600, [1, 1, 1]), (600, [5, 1, 16]), (40, [70, 3, 130]), (8000, [70, 3, 130])]


class Growing:
    """Sequences that grow by ``new`` tokens a step, in a cache of codes."""

    def __init__(self, hist, new, width, steps, heads, d, seed):
        self.hist, self.new, self.steps = np.array(hist), np.array(new), steps
        pages = -(-(self.hist + steps * self.new) // 16)
        rng = np.random.default_rng(seed)
        self.table = np.zeros((len(new), max(int(pages.max()), width)), dtype=np.int32)
        order, at = rng.permutation(int(pages.sum())), 0
        for b, n in enumerate(pages):
            self.table[b, :n] = order[at:at + n]
            at += n
        gen = torch.Generator().manual_seed(seed)
        self.heads, self.d = heads, d
        kp, vp = (randn(gen, at, 16, heads, d, sigma=0.5) for _ in range(2))
        self.pages = torch.from_numpy(layer.q4_pack(kp, vp)).cuda()
        self.off = np.concatenate([[0], np.cumsum(self.new)]).astype(np.int32)
        rows = int(self.off[-1])
        self.qkv = randn(gen, steps, 3, rows, heads, d, sigma=0.5).cuda()
        self.q, self.k, self.v = (torch.zeros(rows, heads, d, device="cuda", dtype=torch.bfloat16)
                                  for _ in range(3))
        self.out, self.k_back, self.v_back = (torch.zeros_like(self.q) for _ in range(3))
        i32 = lambda x: torch.from_numpy(np.asarray(x, dtype=np.int32)).cuda()
        self.kv, self.table_d = i32(self.hist + self.new), i32(self.table)
        self.batch = binding.PagedBatch(i32(self.off), self.kv, self.table_d, int(self.new.max()))
        self.cache = binding.hstu_cache_create_q4(self.pages, 16, heads, d)

    def workspace(self):
        return torch.zeros(binding.hstu_cache_workspace_bytes(self.cache), device="cuda", dtype=torch.uint8)

    def call(self, workspace, stream=None):
        binding.hstu_cache_append(self.cache, self.batch, self.k, self.v, stream=stream)
        binding.hstu_attn_fwd_cache(self.cache, self.batch, self.q, 0.125, 1 / 600, self.out,
                                    workspace=workspace, stream=stream)
        binding.hstu_cache_read(self.cache, self.batch, self.k_back, self.v_back, stream=stream)

    def capture(self, workspace):
        self.kv.copy_(torch.from_numpy((self.hist + self.new).astype(np.int32)))
        keep = self.pages.clone()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            self.call(workspace)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            self.call(workspace)
        self.pages.copy_(keep)
        return graph

    def step(self, i):
        """Step i's inputs, in the arrays that the graph reads."""
        self.kv.copy_(torch.from_numpy((self.hist + (i + 1) * self.new).astype(np.int32)))
        for x, y in zip((self.q, self.k, self.v), self.qkv[i]):
            x.copy_(y)
        self.out.fill_(7.0), self.k_back.fill_(7.0), self.v_back.fill_(7.0)

    def check(self, i):
        kv = self.hist + (i + 1) * self.new
        kp, vp = layer.q4_unpack(self.pages.cpu().numpy(), 16, self.heads, self.d)
        assert np.array_equal(layer.f64(self.k_back), layer.q4_held(self.k))
        assert np.array_equal(layer.f64(self.v_back), layer.q4_held(self.v))
        for b in range(len(self.new)):  # the new keys and values are in their places
            p = np.arange(kv[b] - self.new[b], kv[b])
            rows = slice(int(self.off[b]), int(self.off[b + 1]))
            at = self.table[b, p // 16], p % 16
            assert np.array_equal(kp[at], layer.f64(self.k_back[rows]))
            assert np.array_equal(vp[at], layer.f64(self.v_back[rows]))
        ref, bound = layer.attention(kp, vp, self.q, self.off, kv, self.table, 0.125, 1 / 600)
        assert np.all(np.abs(layer.f64(self.out) - ref) <= 2.0 ** -8 * np.abs(ref) + bound)


@pytest.mark.parametrize("kind", ["q4", "bf16"])
@pytest.mark.parametrize("d,heads,page,batch", [(64, 4, 64, 64), (32, 2, 16, 300), (128, 1, 128, 7)])
def test_readings_between_appends_see_the_last_of_them(d, heads, page, batch, kind):
    # append a token a sequence, read all histories, and again without a pause
    # between any of them: a reading starts while the append before it writes
    # codes and scales beside those that the reading before met
    steps = 48
    first = np.arange(batch) % 5  # tokens of the sequences before the first step
    pages = -(-(int(first.max()) + steps) // page)
    rng = np.random.default_rng(d)
    table = torch.from_numpy(rng.permutation(batch * pages).reshape(batch, pages).astype(np.int32)).cuda()
    if kind == "q4":
        pool = torch.full((batch * pages, binding.hstu_cache_q4_page_bytes(page, heads, d)), 119, device="cuda",
                          dtype=torch.uint8)
        cache = binding.hstu_cache_create_q4(pool, page, heads, d)
    else:
        pool = torch.full((2, batch * pages, page, heads, d), 7.0, device="cuda", dtype=torch.bfloat16)
        cache = binding.hstu_cache_create(pool[0], pool[1])
    i32 = lambda x: torch.from_numpy(np.asarray(x, dtype=np.int32)).cuda()
    gen = torch.Generator().manual_seed(d)
    kv = torch.stack([randn(gen, batch, int(first.max()) + steps, heads, d) for _ in range(2)])
    held = kv if kind == "bf16" else torch.from_numpy(np.stack([layer.q4_held(x) for x in kv])).bfloat16()
    rows_of = lambda x, n: torch.cat([x[:, b, :m] for b, m in enumerate(n)], dim=1)
    calls, seen = [], []
    for i in range(steps):
        n = first + i  # step 0: what stands there before
        new = n if i == 0 else np.ones_like(n)
        off, whole = (i32(np.concatenate([[0], np.cumsum(x)])) for x in (new, n))
        at = lambda x: torch.cat([x[:, b, m - w:m] for b, (m, w) in enumerate(zip(n, new))], dim=1).cuda()
        k, v = at(kv)
        back = torch.full((2, int(n.sum()), heads, d), 7.0, device="cuda", dtype=torch.bfloat16)
        calls.append((binding.PagedBatch(off, i32(n), table, int(new.max())),
                      binding.PagedBatch(whole, i32(n), table, int(n.max())), k, v, back))
        seen.append(rows_of(held, n).cuda())
    for _ in range(3):
        pool.fill_(119 if kind == "q4" else 7.0)
        for *_, back in calls:
            back.fill_(7.0)
        torch.cuda.synchronize()
        for new, whole, k, v, back in calls:
            if len(k):
                binding.hstu_cache_append(cache, new, k, v)
            binding.hstu_cache_read(cache, whole, back[0], back[1])
        torch.cuda.synchronize()
        for i, ref in enumerate(seen):
            assert torch.equal(calls[i][4], ref), i


@pytest.mark.parametrize("kind", ["q4", "bf16"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("width,new", FORMS)
def test_steps_without_a_pause_are_the_steps_one_by_one(width, new, d, kind):
    # append, attend, read back, step after step: each kernel starts while the
    # one before it ends, and finds what that one wrote
    heads, page, steps = 2, 16, 12
    hist, new = np.array([30, 500, 62]), np.array(new)
    of_each = -(-(hist + steps * new) // page)
    pages = int(of_each.sum())
    rng = np.random.default_rng(d)
    order, at = rng.permutation(pages), 0
    table = np.zeros((3, max(int(of_each.max()), width)), dtype=np.int32)
    for b, n in enumerate(of_each):
        table[b, :n] = order[at:at + n]
        at += n
    gen = torch.Generator().manual_seed(d)
    first = torch.stack([randn(gen, pages, page, heads, d, sigma=0.5) for _ in range(2)])
    if kind == "q4":
        first = torch.from_numpy(layer.q4_pack(first[0], first[1])).cuda()
        pool = first.clone()
        cache = binding.hstu_cache_create_q4(pool, page, heads, d)
    else:
        first = first.cuda()
        pool = first.clone()
        cache = binding.hstu_cache_create(pool[0], pool[1])
    i32 = lambda x: torch.from_numpy(np.asarray(x, dtype=np.int32)).cuda()
    off, table = i32(np.concatenate([[0], np.cumsum(new)])), i32(table)
    rows = int(new.sum())
    qkv = randn(gen, steps, 3, rows, heads, d, sigma=0.5).cuda()
    outs = torch.empty(steps, 3, rows, heads, d, device="cuda", dtype=torch.bfloat16)
    ws = torch.zeros(binding.hstu_cache_workspace_bytes(cache), device="cuda", dtype=torch.uint8)
    batches = [binding.PagedBatch(off, i32(hist + (i + 1) * new), table, int(new.max())) for i in range(steps)]

    def run(pause):
        pool.copy_(first)
        outs.fill_(7.0)
        torch.cuda.synchronize()
        for batch, (q, k, v), (out, k_back, v_back) in zip(batches, qkv, outs):
            for call in (lambda: binding.hstu_cache_append(cache, batch, k, v),
                         lambda: binding.hstu_attn_fwd_cache(cache, batch, q, 0.125, 1 / 600, out, workspace=ws),
                         lambda: binding.hstu_cache_read(cache, batch, k_back, v_back)):
                call()
                pause()
        torch.cuda.synchronize()
        return outs.clone(), pool.clone()

    ref, held = run(torch.cuda.synchronize)
    for _ in range(5):
        got, now = run(lambda: None)
        assert torch.equal(got, ref) and torch.equal(now, held)


@pytest.mark.parametrize("own_workspace", [True, False])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("width,new", FORMS)
def test_captured_steps(width, new, d, own_workspace):
    # one captured step (append, attend, read back), replayed while the
    # sequences grow
    g = Growing([30, 500, 62], new, width, 4, 2, d, seed=90 + d)
    ws = g.workspace() if own_workspace else None
    graph = g.capture(ws)
    for i in range(g.steps):
        g.step(i)
        graph.replay()
        torch.cuda.synchronize()
        g.check(i)
    if own_workspace:
        assert not ws[:8192].any(), "the workspace is ready for the next call"


def test_graphs_that_take_turns_share_a_workspace():
    gs = [Growing([30, 500, 62], new, width, 4, 2, 64, seed=95) for width, new in FORMS]
    ws = gs[0].workspace()
    graphs = [g.capture(ws) for g in gs]
    for i in range(4):
        for g in gs:
            g.step(i)
        for graph in graphs:
            graph.replay()
        torch.cuda.synchronize()
        for g in gs:
            g.check(i)


@pytest.mark.parametrize("first,second", [(0, 1), (1, 2), (1, 3), (3, 4), (4, 4)])
def test_two_streams(first, second):
    a, b = (Growing([3000, 90, 700], FORMS[f][1], FORMS[f][0], 1, 2, 64, seed=97 + f) for f in (first, second))
    a.step(0), b.step(0)
    wa, wb = a.workspace(), b.workspace()
    streams = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    a.call(wa), b.call(wb)
    torch.cuda.synchronize()
    a.check(0), b.check(0)
    ra, rb = a.out.clone(), b.out.clone()
    for own in (True, False):
        for _ in range(20):
            a.out.fill_(7.0), b.out.fill_(7.0)
            torch.cuda.synchronize()
            for _ in range(3):
                a.call(wa if own else None, stream=streams[0])
                b.call(wb if own else None, stream=streams[1])
            torch.cuda.synchronize()
            assert torch.equal(a.out, ra) and torch.equal(b.out, rb)


@pytest.mark.parametrize("d,heads,page", [(32, 16, 512), (64, 5, 1024), (128, 12, 512), (64, 2, 4096)])
@pytest.mark.parametrize("name", ["one token", "candidates", "candidate chunks"])
@pytest.mark.parametrize("wide", [False, True])
def test_large_pages_and_many_heads(wide, name, d, heads, page):
    hist, new, nt = SHAPES[name]
    s = Q4(hist, new, page, heads, d, nt, seed=page + d, pad=1, width=-(-10000 // page) if wide else 1)
    s.check(s.attend())


@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("new,width", [(1, 1), (1, 700), (16, 700), (200, 1), (200, 4000)])
@pytest.mark.parametrize("flags", [0, binding.HSTU_DEBUG_UNSIGNALLED_WAIT])
def test_giving_up_at_once_leaves_nothing_behind(flags, new, width, d):
    # a limit that runs out while the first copies are on their way: they land
    # before the kernel ends, and the calls behind it are right
    s = Q4([5000, 40, 1300], [new, 1, 3], 32, 2, d, seed=60 + new, width=width)
    good, ws, q = s.attend(), s.workspace(), s.q.cuda()
    for _ in range(5):
        binding.hstu_set_wait_timeout_ns(1)
        binding.hstu_set_debug_flags(flags)
        try:
            s.attend(q=q, workspace=ws)
        finally:
            binding.hstu_set_debug_flags(0)
            binding.hstu_set_wait_timeout_ns(0)
        after = s.attend(q=q)  # right behind it, with a workspace of its own
        status, site = binding.hstu_last_status()
        assert (status == binding.HSTU_ERR_TIMEOUT) == (site != 0)
        assert status == binding.HSTU_ERR_TIMEOUT or (status == binding.HSTU_OK and not flags)
        assert torch.equal(after, good)
        ws.zero_()
        assert torch.equal(s.attend(q=q, workspace=ws), good)


@pytest.mark.parametrize("new,width", [(1, 1), (1, 400), (70, 1), (70, 4000)])
def test_a_wait_that_runs_out_is_reported(new, width):
    s = Q4([900, 40], [new, 1], 32, 2, 64, seed=40 + new, width=width)
    good, ws = s.attend(), s.workspace()
    torch.cuda.synchronize()
    binding.hstu_set_wait_timeout_ns(20_000_000)
    binding.hstu_set_debug_flags(binding.HSTU_DEBUG_UNSIGNALLED_WAIT)
    try:
        out = s.attend(workspace=ws)
        status, site = binding.hstu_last_status()
    finally:
        binding.hstu_set_debug_flags(0)
        binding.hstu_set_wait_timeout_ns(0)
    assert status == binding.HSTU_ERR_TIMEOUT and site != 0
    assert (out == 7.0).all()
    ws.zero_()
    assert torch.equal(s.attend(workspace=ws), good)


def test_refusals():
    s = Q4([10], [2], 16, 2, 64, seed=13)
    pages = s.pages
    make = lambda p, **kw: binding.hstu_cache_create_q4(p, **{**dict(page_size=16, heads=2, d=64), **kw})
    make(pages)
    for p, kw in ((pages.to(torch.int16), {}), (pages[:, :-16], {}), (pages[0], {}), (pages, dict(heads=3)),
                  (pages.t().contiguous().t(), {}), (pages[:1].expand(3, -1), {})):
        with pytest.raises(ValueError):
            make(p, **kw)
    wide = torch.zeros(s.num_pages, pages.shape[1] + 8, device="cuda", dtype=torch.uint8)
    for p in (wide[:, :-8], torch.zeros(2 * pages.numel(), device="cuda", dtype=torch.uint8)[8:]
              [:pages.numel()].view_as(pages)):
        with pytest.raises(binding.HstuError) as e:
            make(p)
        assert e.value.code == binding.HSTU_ERR_INVALID_ARG
    k, v = s.read()
    call = lambda **kw: binding.hstu_cache_read(**{**dict(cache=s.cache, batch=s.batch, k=k, v=v), **kw})
    for kw in (dict(k=k.float()), dict(v=v[:1]), dict(v=v.cpu()), dict(k=k[:, :1]), dict(k=k.transpose(1, 2)),
               dict(batch=s.host)):
        with pytest.raises(ValueError):
            call(**kw)
    with pytest.raises(binding.HstuError):
        call(k=k[:1].expand(2, 2, 64))
    odd = torch.zeros(2, 132, device="cuda", dtype=torch.bfloat16)
    with pytest.raises(binding.HstuError):
        call(v=odd[:, :128].unflatten(1, (2, 64)))
    q = s.q.cuda()
    for kw in (dict(q=q), dict(q_out=q), dict(rotary=torch.zeros(64, 24, device="cuda"))):
        with pytest.raises(binding.HstuError):
            binding.hstu_cache_append(s.cache, s.batch, s.k.cuda(), s.v.cuda(), **kw)
    with pytest.raises(binding.HstuError):
        binding.hstu_cache_create_q4(torch.zeros(0, pages.shape[1], device="cuda", dtype=torch.uint8), 16, 2, 64)


def test_empty_calls():
    s = Q4([10], [2], 16, 2, 64, seed=14)
    none = torch.empty(0, 2, 64, device="cuda", dtype=torch.bfloat16)
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")
    for batch in (binding.PagedBatch(i32(0), i32(), torch.zeros(0, 3, dtype=torch.int32, device="cuda"), 1),
                  binding.PagedBatch(i32(0, 0), i32(5), torch.zeros(1, 3, dtype=torch.int32, device="cuda"), 4)):
        binding.hstu_attn_fwd_cache(s.cache, batch, none, 1.0, 1.0, none)
        binding.hstu_cache_append(s.cache, batch, none, none)
        binding.hstu_cache_read(s.cache, batch, none, none)
    k, v = torch.full((2, 2, 64), 7.0, device="cuda", dtype=torch.bfloat16), s.v.cuda()
    binding.hstu_cache_read(s.cache, batch, k, v)
    assert (k == 7).all() and torch.equal(v.cpu(), s.v)


@pytest.mark.parametrize("width", [1, 700])
def test_a_bound_of_no_tokens(width):
    s = Q4([40, 7], [2, 1], 16, 2, 64, seed=82, width=width, max_q=0)
    out = s.attend()  # both sequences have more new tokens than the bound
    assert binding.hstu_last_status()[0] == binding.HSTU_ERR_INVALID_ARG
    assert (out == 7.0).all()
    s.dev["q_offsets"].zero_()
    assert (s.attend() == 7.0).all()
    assert binding.hstu_last_status() == (binding.HSTU_OK, 0)


# ------------------------------------------------------------------- together
def test_growing_by_steps_is_the_forward_over_what_is_held():
    # a history cached by one append, then chunks and single tokens, against
    # the contiguous forward of the whole sequence as read back
    w = workloads.custom([150, 40, 333], heads=2, d=64)
    q, k, v = workloads.draw_qkv(w, seed=77)
    plan = [[100, 0, 300], [1, 1, 1], [48, 38, 17], [1, 1, 15]]
    assert np.array_equal(np.sum(plan, axis=0), w.lengths)
    full, num_pages, _ = make_batch(np.zeros(3, dtype=int), w.lengths, 32)
    table = torch.from_numpy(full.keep["page_table"]).cuda()
    pages = torch.full((num_pages, binding.hstu_cache_q4_page_bytes(32, 2, 64)), 255, device="cuda",
                       dtype=torch.uint8)
    cache = binding.hstu_cache_create_q4(pages, 32, 2, 64)
    i32 = lambda x: torch.from_numpy(np.asarray(x, dtype=np.int32)).cuda()
    done = np.zeros(3, dtype=int)
    got = torch.zeros_like(q, device="cuda")
    rot = rotary_table(400, 64).cuda()
    q_rot = torch.zeros_like(got)
    for new in plan:
        rows = np.concatenate([np.arange(w.offsets[b] + done[b], w.offsets[b] + done[b] + new[b])
                               for b in range(3)])
        done += new
        batch = binding.PagedBatch(i32(np.concatenate([[0], np.cumsum(new)])), i32(done), table, max(new))
        at = torch.from_numpy(rows)
        out, turned = (torch.empty(len(rows), 2, 64, device="cuda", dtype=torch.bfloat16) for _ in range(2))
        binding.hstu_cache_append(cache, batch, k[at].cuda(), v[at].cuda(), q=q[at].cuda(), q_out=turned,
                                  rotary=rot)
        binding.hstu_attn_fwd_cache(cache, batch, turned, w.alpha, w.inv_n, out)
        got[at.cuda()], q_rot[at.cuda()] = out, turned
    whole = binding.PagedBatch(i32(w.offsets), i32(w.lengths), table, int(max(w.lengths)))
    k_back, v_back, ref = (torch.zeros_like(got) for _ in range(3))
    binding.hstu_cache_read(cache, whole, k_back, v_back)
    assert np.array_equal(layer.f64(v_back), layer.q4_held(v))
    binding.hstu_attn_fwd(q_rot, k_back, v_back, w.offsets, w.batch, w.heads, w.d, w.max_seqlen, w.alpha,
                          w.inv_n, ref)
    # each is within its bound of the exact value
    kp, vp = layer.q4_unpack(pages.cpu().numpy(), 32, 2, 64)
    ref64, bound = layer.attention(kp, vp, q_rot, w.offsets, w.lengths, full.keep["page_table"], w.alpha, w.inv_n)
    for x in (got, ref):
        assert np.all(np.abs(layer.f64(x) - ref64) <= 2.0 ** -8 * np.abs(ref64) + bound)
