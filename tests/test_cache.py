"""The paged cache without a GPU: slots, shares of work, refusals, and the
64-bit forms against one another."""
import ctypes
import gc

import numpy as np
import pytest

from hstu_jagged_attention_gb300 import binding, build
from oracle import dense, layer

OK, BAD = binding.HSTU_OK, binding.HSTU_ERR_INVALID_ARG


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()


def make_batch(hist, new, page, targets=None, seed=0, max_q=None, spare=2, width=1):
    """A batch of numpy arrays with shuffled pages (a table of at least ``width``
    pages a row): (PagedBatch, num_pages, rows)."""
    rng = np.random.default_rng(seed)
    hist, new = np.asarray(hist), np.asarray(new)
    kv = hist + new
    pages = -(-kv // page)
    order = rng.permutation(int(pages.sum()) + spare)
    table = np.full((len(kv), max(int(pages.max(initial=0)), width)), -7, dtype=np.int32)
    at = 0
    for b, n in enumerate(pages):
        table[b, :n] = order[at:at + n]
        at += n
    off = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    nt = None if targets is None else np.asarray(targets, dtype=np.int32)
    batch = binding.PagedBatch(off, kv.astype(np.int32), table,
                               max_q=int(new.max(initial=0)) if max_q is None else max_q, num_targets=nt)
    return batch, len(order), int(off[-1])


@pytest.mark.parametrize("page", [16, 64, 256])
@pytest.mark.parametrize("seed", range(4))
def test_slots(page, seed):
    rng = np.random.default_rng(seed)
    n = int(rng.integers(1, 30))
    hist = rng.integers(0, 700, size=n)
    new = rng.integers(0, 40, size=n) if seed else np.ones(n, dtype=np.int64)
    nt = [int(rng.integers(0, x + 1)) for x in new]
    batch, num_pages, total = make_batch(hist, new, page, nt, seed)
    rows = total + 5
    slot, pos, ok = binding.hstu_cache_slots(batch, num_pages, page, rows)
    assert ok
    table, t = batch.keep["page_table"], 0
    for b in range(n):
        for i in range(new[b]):
            p = hist[b] + i
            assert slot[t] == table[b, p // page] * page + p % page
            assert pos[t] == min(p, hist[b] + new[b] - nt[b])
            t += 1
    assert np.all(slot[total:] == -1) and np.all(pos[total:] == -1)


def _bad(change, **kw):
    batch, num_pages, rows = make_batch([100, 40, 7], [3, 5, 2], 16, [1, 0, 2], **kw)
    change(batch.keep)
    return binding.hstu_cache_slots(batch, num_pages, 16, rows)


@pytest.mark.parametrize("name,at,value,skipped", [
    ("kv_lens", 1, 4, [1]),          # fewer tokens than new ones
    ("kv_lens", 1, -1, [1]),
    ("kv_lens", 0, 7 * 16 + 1, [0]),  # more tokens than the table holds
    ("num_targets", 0, 4, [0]),      # more candidates than new tokens
    ("num_targets", 2, -1, [2]),
    ("q_offsets", 1, 9, [0, 1]),     # more than max_q, then decreasing
    ("q_offsets", 0, -1, [0]),
    ("q_offsets", 3, 11, [2]),       # past the rows
])
def test_contradictions_are_found(name, at, value, skipped):
    def change(arrays):
        arrays[name][at] = value
    slot, pos, ok = _bad(change)
    assert not ok
    good, _, fine = _bad(lambda arrays: None)
    assert fine
    seq = np.repeat([0, 1, 2], [3, 5, 2])
    for t in range(10):
        if seq[t] in skipped:
            assert slot[t] == -1, t
        else:
            assert slot[t] == good[t], t


@pytest.mark.parametrize("new,name,at,value,skipped", [
    ([3, 5, 2], "q_offsets", 3, 5, range(5, 10)),   # decreasing at the end: rows 5 .. 9 are behind it
    ([3, 5, 2], "q_offsets", 3, -1, range(10)),
    ([3, 0, 2], "kv_lens", 1, -1, ()),              # a sequence without new tokens
    ([3, 0, 2], "kv_lens", 1, 10 ** 6, ()),
    ([3, 5, 0], "num_targets", 2, 1, ()),
    ([3, 5, 0], "q_offsets", 3, 99, ()),            # past the rows, behind the last of them
])
def test_contradictions_without_a_row_are_found(new, name, at, value, skipped):
    batch, num_pages, rows = make_batch([100, 40, 7], new, 16, [0, 0, 0], max_q=5)
    good, _, fine = binding.hstu_cache_slots(batch, num_pages, 16, rows)
    assert fine
    batch.keep[name][at] = value
    slot, _, ok = binding.hstu_cache_slots(batch, num_pages, 16, rows)
    assert not ok
    assert [t for t in range(rows) if slot[t] != good[t]] == list(skipped)


def test_rows_before_the_first_sequence_are_nobodys():
    batch, num_pages, rows = make_batch([100, 0, 40], [3, 2, 1], 16, [0, 2, 0])
    slot, pos, ok = binding.hstu_cache_slots(batch, num_pages, 16, rows)
    batch.keep["q_offsets"] += 4
    slot4, pos4, ok4 = binding.hstu_cache_slots(batch, num_pages, 16, rows + 7)
    assert ok and ok4
    assert np.array_equal(slot4[4:-3], slot) and np.array_equal(pos4[4:-3], pos)
    for x in (slot4, pos4):
        assert np.all(x[:4] == -1) and np.all(x[-3:] == -1)


@pytest.mark.parametrize("value", [-1, 10 ** 6, 2 ** 31 - 1, -2 ** 31])
def test_bad_pages_are_found(value):
    def change(arrays):
        arrays["page_table"][0, 6] = value  # tokens 96 .. of sequence 0: its new ones
    slot, pos, ok = _bad(change)
    assert not ok and np.all(slot[:3] == -1) and np.all(slot[3:] >= 0) and np.all(pos >= 0)


def test_entries_behind_the_last_page_do_not_matter():
    def change(arrays):
        arrays["page_table"][2, 1:] = 2 ** 30
    assert _bad(change)[2]


@pytest.mark.parametrize("seed", range(12))
def test_the_shares_cover_every_block_once(seed):
    rng = np.random.default_rng(50 + seed)
    n = int(rng.integers(1, 12))
    hist = rng.integers(0, 900, size=n)
    new = rng.integers(0, 70, size=n)
    nt = [int(rng.integers(0, x + 1)) if seed % 3 else 0 for x in new]
    tile, keys = [(16, 64), (32, 64), (128, 128)][seed % 3]
    heads, grid = int(rng.integers(1, 5)), int(rng.integers(1, 60))
    min_units = int(rng.integers(1, 6))
    extra = int(rng.integers(0, 4))
    batch, num_pages, rows = make_batch(hist, new, 32, nt, seed)
    segs = binding.hstu_cache_worklist(batch, num_pages, 32, rows, heads, tile, keys, grid, min_units,
                                       extra)
    # every key that a row may see lies in exactly one unit of its (tile, head)
    expect = {}
    for b in range(n):
        kv = hist[b] + new[b]
        for qt in range(-(-new[b] // tile)):
            blocks = set()
            for i in range(qt * tile, min(new[b], qt * tile + tile)):
                p, seen = hist[b] + i, kv - nt[b]
                blocks |= {j // keys for j in range(min(p + 1, seen))} | {p // keys}
            for h in range(heads):
                expect[(b, h, qt)] = len(blocks)
    got, ctas, units = {}, {}, {}
    for cta, b, h, qt, i0, m, c0, parts in segs.tolist():
        assert m >= 1
        got.setdefault((b, h, qt), []).extend(range(i0, i0 + m))
        ctas.setdefault((b, h, qt), set()).add((cta, c0, parts))
        units[cta] = units.get(cta, 0) + m
    assert {k: len(v) for k, v in got.items()} == expect
    for k, v in got.items():
        assert v == list(range(expect[k]))
        assert sorted(c for c, _, _ in ctas[k]) == list(range(min(ctas[k])[1], min(ctas[k])[1] + min(ctas[k])[2]))
    # equal shares of blocks and `extra` units an item, in that order
    total = sum(m + extra for m in expect.values() if m)
    items = -(-batch.max_q // tile) * n * heads
    per = max(-(-total // grid), min_units)
    if items < grid // 16:
        per = max(per, -(-total // (16 * items)))
    want, at = {}, 0
    for qt in range(-(-batch.max_q // tile)):
        for b in range(n):
            for h in range(heads):
                m = expect.get((b, h, qt), 0)
                for i in range(m):
                    want[(at + i) // per] = want.get((at + i) // per, 0) + 1
                at += m + extra if m else 0
    assert units == want
    # a CTA starts at most one shared item that it does not end: its counter is free
    for c in units:
        assert sum(1 for x in segs.tolist() if x[0] == c and x[6] == c and x[7] > 1) <= 1


def test_refusals_on_the_host():
    L, h = binding.lib(), ctypes.c_void_p()
    make = lambda **kw: L.hstu_cache_create(*[kw.get(n, v) for n, v in dict(
        k=16, v=16, num_pages=4, page_size=16, heads=2, d=64, stride=0).items()], ctypes.byref(h))
    assert make(d=96) == binding.HSTU_ERR_UNSUPPORTED
    for kw in (dict(k=0), dict(v=8), dict(num_pages=0), dict(page_size=24), dict(page_size=8),
               dict(page_size=8192), dict(heads=0), dict(stride=16 * 128 - 8), dict(stride=16 * 128 + 4)):
        assert make(**kw) == BAD, kw
    assert L.hstu_cache_destroy(None) == OK
    assert L.hstu_attn_fwd_cache(None, None, None, 0, 1.0, 1.0, None, None, None) == BAD
    assert L.hstu_cache_append(None, None, None, 0, None, 0, None, 0, None, None, None) == BAD
    n = ctypes.c_size_t()
    assert L.hstu_cache_workspace(None, ctypes.byref(n)) == BAD


def test_the_binding_checks_the_batch():
    off, kv, table = (np.zeros(2, np.int32), np.zeros(1, np.int32), np.zeros((1, 3), np.int32))
    binding.PagedBatch(off, kv, table, 1)
    for args in ((off.astype(np.int64), kv, table), (off, np.zeros(2, np.int32), table),
                 (off, kv, table[0]), (off, kv, np.zeros((1, 6), np.int32)[:, ::2])):
        with pytest.raises(ValueError):
            binding.PagedBatch(*args, 1)
    with pytest.raises(ValueError):
        binding.PagedBatch(off, kv, table, 1, num_targets=np.zeros(2, np.int32))


def _norm_call(**kw):
    a = dict(x=16, xs=64, res=None, rs=0, scale=1.0, u=None, us=0, gamma=16, beta=16, eps=1e-6, rows=0,
             width=64, y=16, z=None)
    a.update(kw)
    return binding.lib().hstu_norm_fwd(*a.values(), None)


def test_norm_refusals_on_the_host():
    assert _norm_call() == OK  # no rows: nothing to do
    for kw in (dict(width=0), dict(width=12), dict(width=8200), dict(rows=-1), dict(gamma=None),
               dict(beta=8), dict(eps=-1.0), dict(eps=float("nan")), dict(scale=float("inf")),
               dict(res=16, rs=64), dict(z=16), dict(rows=1, xs=56), dict(rows=1, xs=68),
               dict(rows=1, x=24), dict(rows=1, y=None), dict(rows=1, u=16, us=0),
               dict(rows=1, res=16, rs=60, z=16)):
        assert _norm_call(**kw) == BAD, kw
    n = ctypes.c_size_t()
    for w in (0, 7, 8200):
        assert binding.lib().hstu_norm_bwd_workspace(w, ctypes.byref(n)) == BAD
    a = dict(dy=16, dys=64, z=16, zs=64, u=None, us=0, gamma=16, beta=16, eps=1e-6, dzi=None, dzis=0,
             scale=1.0, rows=1, width=64, dz=16, dx=None, du=None, dus=0, dg=16, db=16, ws=None)
    for kw in (dict(du=16, dus=64), dict(u=16, us=64), dict(dg=None), dict(db=2), dict(dy=None),
               dict(dys=0), dict(zs=60), dict(dz=8), dict(dzi=16, dzis=32), dict(dx=4), dict(ws=8),
               dict(width=65), dict(eps=-0.5)):
        assert binding.lib().hstu_norm_bwd(*{**a, **kw}.values(), None) == BAD, kw


# ------------------------------------------------- the 64-bit forms themselves
def test_attention_over_pages_is_the_dense_definition():
    rng = np.random.default_rng(3)
    lengths, heads, d = [5, 33, 17], 2, 8
    off = np.concatenate([[0], np.cumsum(lengths)]).astype(np.int32)
    q, k, v = (rng.standard_normal((off[-1], heads, d)) for _ in range(3))
    batch, num_pages, rows = make_batch([0, 0, 0], lengths, 16)
    pages = np.full((2, num_pages, 16, heads, d), np.nan)
    kp, vp, qo = layer.append(pages[0], pages[1], k, v, q, off, lengths, batch.keep["page_table"])
    out, _ = layer.attention(kp, vp, qo, off, lengths, batch.keep["page_table"], 0.3, 0.1)
    assert np.allclose(out, dense.hstu_jagged_bruteforce(q, k, v, off, 0.3, 0.1), rtol=0, atol=1e-12)
    nt = [3, 0, 9]
    out, _ = layer.attention(kp, vp, qo, off, lengths, batch.keep["page_table"], 0.3, 0.1, nt)
    ref = dense.hstu_jagged_bruteforce_targets(q, k, v, off, nt, 0.3, 0.1)
    assert np.allclose(out, ref, rtol=0, atol=1e-12)


def test_rotation_keeps_lengths_and_depends_on_the_distance():
    rng = np.random.default_rng(4)
    angle = np.arange(40)[:, None] * 100.0 ** (-np.arange(4) / 4)
    table = np.concatenate([np.cos(angle), np.sin(angle)], axis=1)
    q, k = rng.standard_normal((2, 1, 12))
    for pairs in (False, True):
        r = lambda x, p: layer.rotate(x, p, table, pairs)
        assert np.isclose(np.linalg.norm(r(q, 31)), np.linalg.norm(q))
        assert np.array_equal(r(q, 31)[:, 8:], q[:, 8:])
        assert np.isclose((r(q, 30) * r(k, 21)).sum(), (r(q, 9) * r(k, 0)).sum())


@pytest.mark.parametrize("gate,residual", [(False, False), (True, False), (False, True), (True, True)])
def test_norm_gradient_against_differences(gate, residual):
    rng = np.random.default_rng(5)
    rows, width, eps, scale = 3, 16, 1e-2, 0.5
    a = dict(x=rng.standard_normal((rows, width)), gamma=1 + rng.standard_normal(width),
             beta=rng.standard_normal(width))
    if gate:
        a["u"] = rng.standard_normal((rows, width))
    if residual:
        a["residual"] = rng.standard_normal((rows, width))
    dy, dz_in = rng.standard_normal((2, rows, width))

    def loss(**kw):
        y, z = layer.norm_fwd(**{**a, **kw}, eps=eps, scale=scale)
        return (y * dy).sum() + ((z * dz_in).sum() if residual else 0.0)

    z = layer.norm_fwd(**a, eps=eps, scale=scale)[1]
    g = layer.norm_bwd(dy, z, a["gamma"], a["beta"], eps, a.get("u"), dz_in if residual else None, scale)
    names = dict(x="dx" if residual else "dz", gamma="dgamma", beta="dbeta", u="du", residual="dz")
    for name, value in a.items():
        step, got = 1e-5, g[names[name]]
        for at in np.ndindex(value.shape):
            up, down = value.copy(), value.copy()
            up[at] += step
            down[at] -= step
            diff = (loss(**{name: up}) - loss(**{name: down})) / (2 * step)
            assert abs(diff - got[at]) <= 1e-6 * (1 + abs(diff)), (name, at)


def test_a_cache_of_another_device_is_refused(monkeypatch):
    torch = pytest.importorskip("torch")

    class Pool:  # what the binding asks of a tensor on the second GPU
        shape, is_cuda, dtype = torch.Size((4, 16, 2, 64)), True, torch.bfloat16
        device = torch.device("cuda:1")
        stride = staticmethod(lambda: (16 * 128, 128, 64, 1))
        data_ptr = staticmethod(lambda: 1 << 20)

    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    with pytest.raises(ValueError, match="current device"):
        binding.hstu_cache_create(Pool, Pool)


@pytest.mark.parametrize("max_q", [2 ** 31, 2 ** 32, 2 ** 32 + 1, 2 ** 63])
def test_a_bound_past_32_bits_is_a_bound(max_q):
    batch, num_pages, rows = make_batch([100, 40], [3, 5], 16)
    good = binding.hstu_cache_slots(batch, num_pages, 16, rows)
    large, _, _ = make_batch([100, 40], [3, 5], 16, max_q=max_q)
    got = binding.hstu_cache_slots(large, num_pages, 16, rows)
    assert good[2] and got[2] and np.array_equal(good[0], got[0])


def test_sizes_that_do_not_fit_are_refused():
    batch, num_pages, rows = make_batch([100, 40], [3, 5], 16)
    for n in (2 ** 31, 2 ** 32 + rows):
        with pytest.raises(ValueError):
            batch.struct(n)
    for max_q in (-1, -2 ** 32 + 5):
        with pytest.raises(ValueError):
            make_batch([100, 40], [3, 5], 16, max_q=max_q)


def test_the_stride_of_a_single_row_does_not_matter():
    torch = pytest.importorskip("torch")
    binding._load_torch()
    cpu = torch.device("cpu")
    x = torch.zeros(600, dtype=torch.bfloat16)
    for step in (0, 1, 13, 64, 300):
        row = x.as_strided((1, 2, 32), (step, 32, 1))
        assert binding._row_stride(row, row.shape, cpu, "x") == 64
        flat = x.as_strided((1, 64), (step, 1))
        assert binding._row_stride(flat, flat.shape, cpu, "x") == 64
    rows = x.as_strided((2, 64), (72, 1))
    assert binding._row_stride(rows, rows.shape, cpu, "x") == 72


def test_a_batch_keeps_few_structs():
    batch, _, _ = make_batch([100], [1], 16)
    count = lambda: sum(type(x) is binding._PagedBatch for x in gc.get_objects())
    gc.collect()
    before = count()
    for rows in range(1, 200):
        assert batch.struct(rows) is batch.struct(rows)
    gc.collect()
    assert 0 < count() - before <= 8


@pytest.mark.parametrize("tile", [2 ** 30, 2 ** 31 - 1])
def test_a_tile_of_any_size_holds_all_rows(tile):
    batch, num_pages, rows = make_batch([100, 0, 300], [9, 40, 1], 16)
    args = (batch, num_pages, 16, rows, 2)
    assert np.array_equal(binding.hstu_cache_worklist(*args, tile, 128, 10),
                          binding.hstu_cache_worklist(*args, 64, 128, 10))
