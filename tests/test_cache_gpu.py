"""The paged cache on the GPU: the append and the attention over the cache
against the 64-bit forms of oracle/layer.py, and what a caller may do with
them (strides, streams, captured graphs, padded batches, bad lengths).

Tolerance of the attention: |out - ref| <= 2^-8 |ref| (the rounding to bf16:
half a step, relative to the value) + the bound that layer.attention derives
for what happens before it.  The append: 2^-8 |ref| + 2^-22 of the products'
sizes (three fp32 roundings of 2^-24 and the table's own are exact inputs);
copied values are equal bit for bit.
"""
import numpy as np
import pytest
import torch

from hstu_jagged_attention_gb300 import binding, build, workloads
from oracle import layer
from tests import parity
from tests.test_cache import make_batch

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


def randn(gen, *shape, sigma=1.0):
    return (torch.randn(*shape, generator=gen, dtype=torch.float32) * sigma).bfloat16()


def rotary_table(positions, dim):
    angle = np.arange(positions)[:, None] * 10000.0 ** (-np.arange(0, dim, 2) / dim)
    return torch.from_numpy(np.concatenate([np.cos(angle), np.sin(angle)], axis=1).astype(np.float32))


class Setup:
    """A host batch with its pools, and the same on the device."""

    def __init__(self, hist, new, page, heads, d, targets=None, seed=0, pad=0, max_q=None, nan_tail=True,
                 width=1):
        self.host, self.num_pages, self.total = make_batch(hist, new, page, targets, seed, max_q,
                                                           width=width)
        self.rows, self.heads, self.d, self.page = self.total + pad, heads, d, page
        gen = torch.Generator().manual_seed(seed)
        sigma = 1.0 if d < 128 else 0.5
        self.kp = randn(gen, self.num_pages, page, heads, d, sigma=sigma)
        self.vp = randn(gen, self.num_pages, page, heads, d, sigma=sigma)
        self.q, self.k, self.v = (randn(gen, self.rows, heads, d, sigma=sigma) for _ in range(3))
        keep = self.host.keep
        if nan_tail:  # rows behind a sequence's end, and the pages nobody holds
            kv, table = keep["kv_lens"], keep["page_table"]
            used = np.zeros((self.num_pages, page), dtype=bool)
            for b, n in enumerate(kv):
                p = np.arange(n)
                used[table[b, p // page], p % page] = True
            self.kp[torch.from_numpy(~used)] = float("nan")
            self.vp[torch.from_numpy(~used)] = float("inf")
        self.dev = {n: torch.from_numpy(a).cuda() for n, a in keep.items()}
        self.batch = binding.PagedBatch(self.dev["q_offsets"], self.dev["kv_lens"], self.dev["page_table"],
                                        self.host.max_q, self.dev.get("num_targets"))
        self.kd, self.vd = self.kp.cuda(), self.vp.cuda()
        self.cache = binding.hstu_cache_create(self.kd, self.vd)
        self.alpha, self.inv_n = d ** -0.5, 1.0 / max(int(keep["kv_lens"].max(initial=1)), 1)

    def attend(self, q=None, out=None, workspace=None, **kw):
        q = self.q.cuda() if q is None else q
        out = torch.full((self.rows, self.heads, self.d), 7.0, device="cuda", dtype=torch.bfloat16) \
            if out is None else out
        binding.hstu_attn_fwd_cache(self.cache, self.batch, q, self.alpha, self.inv_n, out,
                                    workspace=workspace, **kw)
        return out

    def oracle(self):
        a = self.host.keep
        return layer.attention(self.kp, self.vp, self.q, a["q_offsets"], a["kv_lens"], a["page_table"],
                               self.alpha, self.inv_n, a.get("num_targets"))

    def workspace(self):
        return torch.zeros(binding.hstu_cache_workspace_bytes(self.cache), device="cuda", dtype=torch.uint8)

    def check(self, out):
        ref, bound = self.oracle()
        got = layer.f64(out)
        held = ~np.isnan(ref)
        assert np.all(np.isfinite(got[held])), "non-finite output"
        err = np.abs(got - ref)[held] / (2.0 ** -8 * np.abs(ref) + bound)[held].clip(1e-300)
        assert err.size == 0 or err.max() <= 1.0, f"worst err/tol {err.max():.3f}"
        assert np.all(got[~held] == 7.0), "a row behind the last sequence was written"
        return err.max() if err.size else 0.0


# name: cached tokens, new tokens, candidates
SHAPES = {
    "one token": ([0, 1, 15, 16, 63, 64, 200, 511], [1] * 8, None),
    "one sequence": ([700], [1], None),
    "few tokens, some without": ([0, 130, 64, 5, 90], [3, 0, 16, 9, 1], None),
    "candidates": ([0, 130, 64, 5, 257], [3, 0, 16, 9, 12], [3, 0, 16, 4, 12]),
    "17 to 32 tokens": ([100, 0, 31, 200], [17, 32, 25, 1], [0, 10, 25, 1]),
    "chunks": ([100, 0, 31, 0, 300], [70, 129, 64, 0, 33], None),
    "candidate chunks": ([100, 0, 31, 128, 300], [70, 129, 64, 1, 140], [70, 100, 0, 1, 140]),
    "nothing": ([4, 0], [0, 0], None),
}


@pytest.mark.parametrize("d,heads,page", [(32, 3, 16), (64, 2, 64), (128, 1, 32), (64, 1, 256),
                                          (32, 2, 128), (128, 2, 16)])
@pytest.mark.parametrize("name", SHAPES)
@pytest.mark.parametrize("wide", [False, True])
def test_attention_parity(wide, name, d, heads, page):
    # wide: a table for 10,000 tokens, so that few items share the GPU evenly
    # instead of taking a cluster each
    hist, new, nt = SHAPES[name]
    s = Setup(hist, new, page, heads, d, nt, seed=len(name) + d, pad=3, width=10000 // page if wide else 1)
    out = s.attend()
    s.check(out)


def test_many_items():
    # more items than clusters run at once, of one to seven blocks
    rng = np.random.default_rng(50)
    hist, new = rng.integers(0, 850, size=60), rng.integers(0, 4, size=60)
    s = Setup(hist, new, 32, 2, 64, rng.integers(0, new + 1), seed=50)
    s.check(s.attend())


@pytest.mark.parametrize("d,heads,page", [(32, 2, 32), (64, 3, 16), (128, 1, 128)])
@pytest.mark.parametrize("name", ["one token", "few tokens, some without", "candidates",
                                  "17 to 32 tokens"])
def test_few_rows_on_large_tiles(name, d, heads, page):
    # a bound on the new tokens that asks for 128-row tiles, with few rows in them
    hist, new, nt = SHAPES[name]
    s = Setup(hist, new, page, heads, d, nt, seed=20 + d, pad=1, max_q=130)
    s.check(s.attend())


@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("new,targets", [(33, 0), (47, 47), (64, 20)])
def test_several_small_tiles(d, new, targets):
    s = Setup([0, 140, 300], [new, 1, 17], 64, 2, d, [targets, 0, 17], seed=30 + d)
    s.check(s.attend())


@pytest.mark.parametrize("max_q", [1, 4, 16, 32, 33, 500, 2 ** 31 - 1])
def test_max_q_changes_the_tiling_not_the_result(max_q):
    s = Setup([90, 300, 5], [1, 1, 1], 32, 2, 64, seed=1, max_q=max_q)
    s.check(s.attend())


@pytest.mark.parametrize("width", [1, 200])
@pytest.mark.parametrize("new", [1, 5, 40, 130])
def test_long_cache_few_rows(new, width):
    # one sequence and one head over a cluster or the whole GPU: many parts a row
    s = Setup([6000], [new], 64, 1, 64, [new], seed=2, width=width)
    ws = s.workspace()
    a = s.attend(workspace=ws)
    assert not ws[:8192].any(), "the workspace is ready for the next call"
    s.check(a)
    for _ in range(3):  # parts are summed in a fixed order
        assert torch.equal(a, s.attend(workspace=ws))
    assert torch.equal(a, s.attend())  # without a workspace


def test_strided_queries_and_interleaved_pools():
    s = Setup([100, 20], [4, 20], 16, 2, 64, seed=3)
    wide = torch.randn(s.rows, 4, 2, 64, device="cuda").bfloat16()
    wide[:, 2] = s.q.cuda()
    a = s.attend()
    assert torch.equal(a, s.attend(q=wide[:, 2]))
    pool = torch.stack([s.kd, s.vd], dim=1).contiguous()  # (pages, K | V, ...)
    s.cache = binding.hstu_cache_create(pool[:, 0], pool[:, 1])
    assert torch.equal(a, s.attend())


def test_a_pool_past_32_bits():
    # page numbers whose byte and element offsets need more than 32 bits
    s = Setup([300, 5], [3, 1], 64, 2, 64, seed=4)
    packed = 64 * 2 * 64
    pages = (1 << 32) // packed + s.num_pages + 1
    big = torch.empty(pages, 64, 2, 64, device="cuda", dtype=torch.bfloat16)
    big_v = torch.empty_like(big)
    move = pages - s.num_pages
    big[move:], big_v[move:] = s.kd, s.vd
    a = s.attend()
    s.cache = binding.hstu_cache_create(big, big_v)
    s.dev["page_table"].add_(move)
    assert torch.equal(a, s.attend())
    # and appended to
    k, v = s.k.cuda(), s.v.cuda()
    binding.hstu_cache_append(s.cache, s.batch, k, v)
    small = Setup([300, 5], [3, 1], 64, 2, 64, seed=4)
    binding.hstu_cache_append(small.cache, small.batch, k, v)
    assert torch.equal(big[move:].nan_to_num(), small.kd.nan_to_num())
    assert torch.equal(big_v[move:].nan_to_num(), small.vd.nan_to_num())


def test_keys_past_the_end_never_matter():
    # the same batch with finite and with non-finite rows behind each end
    a = Setup([100, 63, 0, 30], [1, 2, 1, 40], 64, 2, 64, [0, 2, 1, 5], seed=5, nan_tail=False)
    b = Setup([100, 63, 0, 30], [1, 2, 1, 40], 64, 2, 64, [0, 2, 1, 5], seed=5, nan_tail=True)
    assert torch.equal(a.attend(), b.attend())


def test_a_shared_prefix_is_read_from_shared_pages():
    # three sequences whose first pages are the same
    s = Setup([128, 128, 128], [2, 1, 3], 32, 2, 64, seed=6)
    table = s.host.keep["page_table"]
    table[1, :4] = table[2, :4] = table[0, :4]
    s.dev["page_table"].copy_(torch.from_numpy(table))
    s.check(s.attend())


@pytest.mark.parametrize("width", [1, 600])
def test_bad_lengths_and_pages_are_skipped_and_reported(width):
    s = Setup([100, 40, 70], [2, 2, 1], 16, 1, 64, seed=7, nan_tail=False, width=width)
    good = s.attend()

    def run(name, at, value):
        t = s.dev[name]
        old = t[at].clone()
        t[at] = value
        out = s.attend()
        torch.cuda.synchronize()
        status = binding.hstu_last_status()[0]
        t[at] = old
        return out, status

    for name, at, value in (("kv_lens", 1, 1), ("kv_lens", 1, 10 ** 6), ("kv_lens", 1, -5)):
        out, status = run(name, at, value)
        assert status == binding.HSTU_ERR_INVALID_ARG
        assert torch.equal(out[:2], good[:2]) and torch.equal(out[4:], good[4:]) and (out[2:4] == 7).all()
    for value in (-1, s.num_pages, 2 ** 31 - 1, -2 ** 31):
        out, status = run("page_table", (1, 0), value)
        assert status == binding.HSTU_ERR_INVALID_ARG
        assert torch.equal(out[:2], good[:2]) and torch.equal(out[4:], good[4:])
        # the page's keys add nothing: as if its values were zero
        keep = s.vd.clone()
        s.vd[s.dev["page_table"][1, 0]] = 0
        ref = s.attend()
        s.vd.copy_(keep)
        assert torch.equal(out[2:4], ref[2:4])
    # an append to a bad page, or past the rotation's table, is dropped
    k, v = s.k.cuda(), s.v.cuda()
    before = s.kd.clone(), s.vd.clone()
    old = s.dev["page_table"][2, 4].clone()
    s.dev["page_table"][2, 4] = -3
    binding.hstu_cache_append(s.cache, s.batch, k, v)
    torch.cuda.synchronize()
    assert binding.hstu_last_status()[0] == binding.HSTU_ERR_INVALID_ARG
    assert torch.equal(s.kd[old], before[0][old])
    assert not torch.equal(s.kd, before[0])
    s.dev["page_table"][2, 4] = old
    s.kd.copy_(before[0])
    s.vd.copy_(before[1])
    binding.hstu_cache_append(s.cache, s.batch, k, v, rotary=rotary_table(70, 32).cuda())
    torch.cuda.synchronize()
    assert binding.hstu_last_status()[0] == binding.HSTU_ERR_INVALID_ARG
    assert torch.equal(s.kd[old], before[0][old])  # position 70 is not in the table


@pytest.mark.parametrize("d,heads,page,rot,pairs", [(64, 2, 16, 64, False), (64, 3, 64, 32, True),
                                                    (32, 1, 32, 16, False), (128, 2, 128, 128, True),
                                                    (128, 1, 16, 96, False), (64, 2, 32, 0, False),
                                                    (32, 4, 16, 32, True)])
@pytest.mark.parametrize("name", SHAPES)
def test_append(name, d, heads, page, rot, pairs):
    hist, new, nt = SHAPES[name]
    s = Setup(hist, new, page, heads, d, nt, seed=d + rot, pad=2)
    a = s.host.keep
    table = rotary_table(int(a["kv_lens"].max()) + 1, rot) if rot else None
    q_out = torch.full((s.rows, heads, d), 7.0, device="cuda", dtype=torch.bfloat16)
    binding.hstu_cache_append(s.cache, s.batch, s.k.cuda(), s.v.cuda(), q=s.q.cuda(), q_out=q_out,
                              rotary=None if table is None else table.cuda(), rotary_pairs=pairs)
    kp, vp, qr = layer.append(s.kp, s.vp, s.k, s.v, s.q, a["q_offsets"], a["kv_lens"], a["page_table"],
                              a.get("num_targets"), table, pairs)
    # values, and everything that was not appended, bit for bit
    assert np.array_equal(layer.f64(s.vd), vp, equal_nan=True)
    got_k, got_q = layer.f64(s.kd), layer.f64(q_out)
    old = layer.f64(s.kp)
    same = np.isnan(old) & np.isnan(kp) | (kp == old)
    assert np.array_equal(got_k[same], old[same], equal_nan=True)
    size = 2.0 * max(layer.f64(s.k).__abs__().max(initial=0), layer.f64(s.q).__abs__().max(initial=0))
    for got, ref in ((got_k, kp), (got_q, qr)):
        held = ~np.isnan(ref)
        assert np.all(np.abs(got - ref)[held] <= 2.0 ** -8 * np.abs(ref)[held] + 2.0 ** -22 * size)
        if not rot:
            assert np.array_equal(got[held], ref[held])
    assert np.all(got_q[np.isnan(qr)] == 7.0)


def test_append_from_a_fused_projection_and_in_place():
    s = Setup([10, 300, 0], [5, 1, 90], 32, 2, 64, [2, 0, 90], seed=9, pad=4)
    table = rotary_table(512, 64).cuda()
    q_out = torch.zeros(s.rows, 2, 64, device="cuda", dtype=torch.bfloat16)
    binding.hstu_cache_append(s.cache, s.batch, s.k.cuda(), s.v.cuda(), q=s.q.cuda(), q_out=q_out,
                              rotary=table)
    first = s.kd.clone(), s.vd.clone()
    s.kd.copy_(s.kp)
    s.vd.copy_(s.vp)
    proj = torch.stack([s.v, s.q, s.v, s.k], dim=1).cuda()
    q2 = torch.zeros_like(q_out)
    binding.hstu_cache_append(s.cache, s.batch, proj[:, 3], proj[:, 2], q=proj[:, 1], q_out=q2, rotary=table)
    assert torch.equal(q_out, q2)
    assert torch.equal(s.kd.nan_to_num(), first[0].nan_to_num())
    assert torch.equal(s.vd.nan_to_num(), first[1].nan_to_num())
    q3 = s.q.cuda()
    binding.hstu_cache_append(s.cache, s.batch, s.k.cuda(), s.v.cuda(), q=q3, q_out=q3, rotary=table)
    assert torch.equal(q3[:s.total], q_out[:s.total])
    assert torch.equal(q3[s.total:].cpu(), s.q[s.total:])  # a padded batch's rows stay


def test_two_streams_with_their_own_workspaces():
    a = Setup([4000, 90], [1, 1], 64, 2, 64, seed=10)
    b = Setup([2500, 3000, 7], [20, 3, 1], 32, 2, 64, [20, 0, 0], seed=11)
    ra, rb = a.attend(), b.attend()
    qa, qb = a.q.cuda(), b.q.cuda()
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    wa, wb = a.workspace(), b.workspace()
    oa, ob = [torch.empty_like(ra) for _ in range(20)], [torch.empty_like(rb) for _ in range(20)]
    torch.cuda.synchronize()
    for x, y in zip(oa, ob):
        x.fill_(7.0), y.fill_(7.0)
    torch.cuda.synchronize()
    for x, y in zip(oa, ob):
        a.attend(q=qa, out=x, workspace=wa, stream=s1)
        b.attend(q=qb, out=y, workspace=wb, stream=s2)
    torch.cuda.synchronize()
    assert all(torch.equal(x, ra) for x in oa) and all(torch.equal(y, rb) for y in ob)


@pytest.mark.parametrize("own_workspace", [True, False])
def test_a_captured_step_follows_the_device_arrays(own_workspace):
    # one captured decode step (append, attend), replayed while the sequences
    # grow by a token each: new lengths, new pages, new rows each time
    hist, steps = np.array([30, 500, 62]), 6
    s = Setup(hist, [1, 1, 1], 16, 2, 64, seed=12, nan_tail=False)
    # a table with room for every step
    rng = np.random.default_rng(0)
    pages = -(-(hist + steps) // 16)
    num_pages = int(pages.sum())
    table = np.zeros((3, int(pages.max())), dtype=np.int32)
    order, at = rng.permutation(num_pages), 0
    for b, n in enumerate(pages):
        table[b, :n] = order[at:at + n]
        at += n
    gen = torch.Generator().manual_seed(1)
    kp, vp = randn(gen, num_pages, 16, 2, 64), randn(gen, num_pages, 16, 2, 64)
    q, k, v = (randn(gen, steps, 3, 2, 64) for _ in range(3))
    kd, vd = kp.cuda(), vp.cuda()
    cache = binding.hstu_cache_create(kd, vd)
    kv, off = torch.from_numpy(hist.astype(np.int32) + 1).cuda(), torch.arange(4, dtype=torch.int32).cuda()
    table_d = torch.zeros(3, table.shape[1], dtype=torch.int32).cuda()
    batch = binding.PagedBatch(off, kv, table_d, max_q=1)
    rot = rotary_table(600, 64).cuda()
    qs, ks, vs = (torch.empty(3, 2, 64, device="cuda", dtype=torch.bfloat16) for _ in range(3))
    q_rot, out = torch.empty_like(qs), torch.empty_like(qs)
    ws = torch.zeros(binding.hstu_cache_workspace_bytes(cache), device="cuda", dtype=torch.uint8) \
        if own_workspace else None

    def step():
        binding.hstu_cache_append(cache, batch, ks, vs, q=qs, q_out=q_rot, rotary=rot)
        binding.hstu_attn_fwd_cache(cache, batch, q_rot, 0.125, 1 / 600, out, workspace=ws)

    table_d.copy_(torch.from_numpy(table))
    qs.zero_(), ks.zero_(), vs.zero_()
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    table_d.zero_()
    kd.copy_(kp), vd.copy_(vp)
    ref_k, ref_v = layer.f64(kp), layer.f64(vp)
    for i in range(steps):
        kv.copy_(torch.from_numpy((hist + 1 + i).astype(np.int32)))
        table_d.copy_(torch.from_numpy(table))
        qs.copy_(q[i]), ks.copy_(k[i]), vs.copy_(v[i])
        graph.replay()
        torch.cuda.synchronize()
        args = (np.arange(4), hist + 1 + i, table)
        ref_k, ref_v, ref_q = layer.append(ref_k, ref_v, k[i], v[i], q[i], *args, None, rot.cpu())
        # the rows that the step rounded, as stored
        assert np.allclose(layer.f64(kd), ref_k, rtol=2 ** -8, atol=1e-5)
        ref, bound = layer.attention(kd, vd, q_rot, *args, 0.125, 1 / 600)
        assert np.all(np.abs(layer.f64(out) - ref) <= 2.0 ** -8 * np.abs(ref) + bound)
        ref_k, ref_v = layer.f64(kd), layer.f64(vd)


def test_growing_by_steps_is_the_forward_over_the_whole():
    # a history cached by one append, then chunks and single tokens, against
    # the contiguous forward of the whole sequence
    w = workloads.custom([150, 40, 333], heads=2, d=64)
    q, k, v = workloads.draw_qkv(w, seed=77)
    ref = torch.empty_like(q, device="cuda")
    binding.hstu_attn_fwd(q.cuda(), k.cuda(), v.cuda(), w.offsets, w.batch, w.heads, w.d, w.max_seqlen,
                          w.alpha, w.inv_n, ref)
    plan = [[100, 0, 300], [1, 1, 1], [48, 38, 17], [1, 1, 15]]
    assert np.array_equal(np.sum(plan, axis=0), w.lengths)
    page = 32
    full, num_pages, _ = make_batch(np.zeros(3, dtype=int), w.lengths, page)
    table = torch.from_numpy(full.keep["page_table"]).cuda()
    kp = torch.full((num_pages, page, 2, 64), float("nan"), device="cuda", dtype=torch.bfloat16)
    vp = kp.clone()
    cache = binding.hstu_cache_create(kp, vp)
    done = np.zeros(3, dtype=int)
    got = torch.zeros_like(ref)
    for new in plan:
        rows = np.concatenate([np.arange(w.offsets[b] + done[b], w.offsets[b] + done[b] + new[b])
                               for b in range(3)])
        done += new
        i32 = lambda x: torch.from_numpy(np.asarray(x, dtype=np.int32)).cuda()
        batch = binding.PagedBatch(i32(np.concatenate([[0], np.cumsum(new)])), i32(done), table, max(new))
        at = torch.from_numpy(rows)
        binding.hstu_cache_append(cache, batch, k[at].cuda(), v[at].cuda())
        out = torch.empty(len(rows), 2, 64, device="cuda", dtype=torch.bfloat16)
        binding.hstu_attn_fwd_cache(cache, batch, q[at].cuda(), w.alpha, w.inv_n, out)
        got[at.cuda()] = out
    # each is within its bound of the exact value, so within both of each other
    a = np.array([0, 150, 190, 523])
    ref64, bound = layer.attention(kp, vp, q, a, w.lengths, full.keep["page_table"], w.alpha, w.inv_n)
    for x in (got, ref):
        assert np.all(np.abs(layer.f64(x) - ref64) <= 2.0 ** -8 * np.abs(ref64) + bound)


@pytest.mark.parametrize("new,width", [(1, 1), (1, 400), (70, 1)])
def test_a_wait_that_runs_out_is_reported(new, width):
    # the kernels give up at a barrier nothing signals, write nothing, and
    # leave a device (and, zeroed again, a workspace) that works
    s = Setup([900, 40], [new, 1], 32, 2, 64, seed=40 + new, width=width)
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
    s = Setup([10], [2], 16, 2, 64, seed=13)
    q, out = s.q.cuda(), torch.empty(2, 2, 64, device="cuda", dtype=torch.bfloat16)
    call = lambda **kw: binding.hstu_attn_fwd_cache(**{**dict(
        cache=s.cache, batch=s.batch, q=q, alpha=1.0, inv_n=1.0, out=out), **kw})
    call()
    for kw in (dict(q=q.float()), dict(q=q.cpu()), dict(q=q[:, :1]), dict(q=q.transpose(1, 2)),
               dict(out=torch.empty(2, 4, 64, device="cuda", dtype=torch.bfloat16)[:, ::2]),
               dict(out=out.half()), dict(workspace=torch.zeros(8, device="cuda", dtype=torch.uint8))):
        with pytest.raises(ValueError):
            call(**kw)
    wide = torch.zeros(2, 130, device="cuda", dtype=torch.bfloat16)
    with pytest.raises(binding.HstuError) as e:  # rows 260 bytes apart: not 16-byte aligned
        call(q=wide[:, :128].unflatten(1, (2, 64)))
    assert e.value.code == binding.HSTU_ERR_INVALID_ARG
    with pytest.raises(binding.HstuError):  # broadcast rows
        call(q=q[:1].expand(2, 2, 64))
    with pytest.raises(ValueError):
        binding.hstu_cache_slots(s.batch, s.num_pages, 16, 2)
    k, v = s.k.cuda(), s.v.cuda()
    app = lambda **kw: binding.hstu_cache_append(**{**dict(cache=s.cache, batch=s.batch, k=k, v=v), **kw})
    for kw in (dict(k=k.float()), dict(v=v[:1]), dict(rotary=torch.zeros(64, 64)),
               dict(rotary=torch.zeros(64, 64, device="cuda", dtype=torch.float64))):
        with pytest.raises(ValueError):
            app(**kw)
    for kw in (dict(q=q), dict(q_out=out), dict(rotary=torch.zeros(64, 24, device="cuda")),
               dict(rotary=torch.zeros(64, 80, device="cuda")), dict(rotary=torch.zeros(0, 64, device="cuda"))):
        with pytest.raises(binding.HstuError) as e:
            app(**kw)
        assert e.value.code == binding.HSTU_ERR_INVALID_ARG
    with pytest.raises(ValueError):
        binding.hstu_cache_create(s.kd, s.vd.float())
    with pytest.raises(binding.HstuError):
        binding.hstu_cache_create(s.kd[:, :12].contiguous(), s.vd[:, :12].contiguous())


def test_empty_calls():
    s = Setup([10], [2], 16, 2, 64, seed=14)
    none = torch.empty(0, 2, 64, device="cuda", dtype=torch.bfloat16)
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")
    batch = binding.PagedBatch(i32(0), i32(), torch.zeros(0, 3, dtype=torch.int32, device="cuda"), 1)
    binding.hstu_attn_fwd_cache(s.cache, batch, none, 1.0, 1.0, none)
    binding.hstu_cache_append(s.cache, batch, none, none)
    batch = binding.PagedBatch(i32(0, 0), i32(5), torch.zeros(1, 3, dtype=torch.int32, device="cuda"), 4)
    binding.hstu_attn_fwd_cache(s.cache, batch, none, 1.0, 1.0, none)
    binding.hstu_attn_fwd_cache(s.cache, batch, s.q.cuda(), 1.0, 1.0, s.q.cuda())
    parity.assert_device_ok()


@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("new,width", [(1, 1), (5, 1), (1, 700), (16, 700)])
def test_giving_up_at_once_leaves_nothing_behind(new, width, d):
    # a limit that runs out while the first copies are on their way: they land
    # before the kernel ends, and the calls behind it are right
    s = Setup([5000, 40, 1300], [new, 1, 3], 32, 2, d, seed=60 + new, width=width)
    good, ws, q = s.attend(), s.workspace(), s.q.cuda()
    for _ in range(10):
        binding.hstu_set_wait_timeout_ns(1)
        try:
            s.attend(q=q, workspace=ws)
        finally:
            binding.hstu_set_wait_timeout_ns(0)
        after = s.attend(q=q)  # right behind it, with a workspace of its own
        status, site = binding.hstu_last_status()
        assert (status == binding.HSTU_ERR_TIMEOUT) == (site != 0)
        assert status in (binding.HSTU_OK, binding.HSTU_ERR_TIMEOUT)
        assert torch.equal(after, good)
        ws.zero_()
        assert torch.equal(s.attend(q=q, workspace=ws), good)


@pytest.mark.parametrize("d", [32, 64, 128])
def test_giving_up_at_once_on_large_tiles(d):
    s = Setup([3000, 40, 1300], [200, 1, 130], 32, 2, d, seed=70)
    good, ws, q = s.attend(), s.workspace(), s.q.cuda()
    for flags in (0, binding.HSTU_DEBUG_UNSIGNALLED_WAIT):
        for _ in range(5):
            binding.hstu_set_wait_timeout_ns(1)
            binding.hstu_set_debug_flags(flags)
            try:
                s.attend(q=q, workspace=ws)
            finally:
                binding.hstu_set_debug_flags(0)
                binding.hstu_set_wait_timeout_ns(0)
            after = s.attend(q=q)
            status, site = binding.hstu_last_status()
            assert (status == binding.HSTU_ERR_TIMEOUT) == (site != 0)
            assert status == binding.HSTU_ERR_TIMEOUT or not flags
            assert torch.equal(after, good)
            ws.zero_()
            assert torch.equal(s.attend(q=q, workspace=ws), good)


@pytest.mark.parametrize("name,at,value,kept", [("q_offsets", 3, 5, 5), ("kv_lens", 3, -1, 10),
                                                ("kv_lens", 3, 10 ** 6, 10), ("q_offsets", 5, 99, 10)])
def test_append_reports_contradictions_without_a_row(name, at, value, kept):
    s = Setup([100, 40, 7, 9, 1], [3, 5, 2, 0, 0], 16, 2, 64, seed=80)
    if name == "q_offsets" and at == 3:
        s.dev[name][4:] = value
    s.dev[name][at] = value
    k, v = s.k.cuda(), s.v.cuda()
    binding.hstu_cache_append(s.cache, s.batch, k, v)
    assert binding.hstu_last_status()[0] == binding.HSTU_ERR_INVALID_ARG
    a = s.host.keep
    off, kv, table = a["q_offsets"], a["kv_lens"], a["page_table"]
    for t in range(kept):  # the other sequences' rows are in their places
        b = int(np.searchsorted(off, t, side="right")) - 1
        p = kv[b] - (off[b + 1] - off[b]) + t - off[b]
        assert torch.equal(s.kd[table[b, p // 16], p % 16], k[t])
    assert binding.hstu_last_status() == (binding.HSTU_OK, 0)


@pytest.mark.parametrize("new", [1, 40, 130])
def test_rows_before_the_first_sequence_stay(new):
    s = Setup([100, 0, 700], [3, new, 1], 16, 2, 64, seed=81)
    s.dev["q_offsets"].add_(4)
    lead = torch.full((4, 2, 64), float("nan"), device="cuda", dtype=torch.bfloat16)
    pad = lambda x: torch.cat([lead, x.cuda(), lead[:1]])
    q_out = torch.full((s.rows + 5, 2, 64), 7.0, device="cuda", dtype=torch.bfloat16)
    good = s.kp.clone(), s.vp.clone()
    a = s.host.keep
    for t in range(s.total):
        b = int(np.searchsorted(a["q_offsets"], t, side="right")) - 1
        p = a["kv_lens"][b] - a["q_offsets"][b + 1] + t
        for x, y in zip(good, (s.k, s.v)):
            x[a["page_table"][b, p // 16], p % 16] = y[t]
    binding.hstu_cache_append(s.cache, s.batch, pad(s.k), pad(s.v), q=pad(s.q), q_out=q_out)
    assert torch.equal(s.kd.cpu().nan_to_num(), good[0].nan_to_num())
    assert torch.equal(s.vd.cpu().nan_to_num(), good[1].nan_to_num())
    assert torch.equal(q_out[4:-1].cpu(), s.q) and (q_out[:4] == 7).all() and (q_out[-1] == 7).all()
    out = torch.full_like(q_out, 7.0)
    s.attend(q=pad(s.q), out=out)
    assert (out[:4] == 7).all() and (out[-1] == 7).all()
    s.kp, s.vp = good
    s.check(out[4:-1])


# table widths (pages of 16) and new tokens that send a call to each of the
# kernels: shares of 16-row tiles, 128-row tiles
FORMS = [(600, [1, 1, 1]), (600, [5, 1, 16]), (40, [70, 3, 130])]


class Growing:
    """Sequences that grow by ``new`` tokens a step, with their device arrays."""

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
        self.kp, self.vp = (randn(gen, at, 16, heads, d, sigma=0.5).cuda() for _ in range(2))
        self.off = np.concatenate([[0], np.cumsum(self.new)]).astype(np.int32)
        rows = int(self.off[-1])
        self.qkv = randn(gen, steps, 3, rows, heads, d, sigma=0.5).cuda()
        self.q, self.k, self.v = (torch.zeros(rows, heads, d, device="cuda", dtype=torch.bfloat16)
                                  for _ in range(3))
        self.out = torch.zeros_like(self.q)
        i32 = lambda x: torch.from_numpy(np.asarray(x, dtype=np.int32)).cuda()
        self.kv, self.table_d = i32(self.hist + self.new), i32(self.table)
        self.batch = binding.PagedBatch(i32(self.off), self.kv, self.table_d, int(self.new.max()))
        self.cache = binding.hstu_cache_create(self.kp, self.vp)

    def workspace(self):
        return torch.zeros(binding.hstu_cache_workspace_bytes(self.cache), device="cuda", dtype=torch.uint8)

    def call(self, workspace, stream=None):
        binding.hstu_cache_append(self.cache, self.batch, self.k, self.v, stream=stream)
        binding.hstu_attn_fwd_cache(self.cache, self.batch, self.q, 0.125, 1 / 600, self.out,
                                    workspace=workspace, stream=stream)

    def capture(self, workspace):
        self.kv.copy_(torch.from_numpy((self.hist + self.new).astype(np.int32)))
        keep = self.kp.clone(), self.vp.clone()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            self.call(workspace)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            self.call(workspace)
        self.kp.copy_(keep[0]), self.vp.copy_(keep[1])
        return graph

    def step(self, i):
        """Step i's inputs, in the arrays that the graph reads."""
        self.kv.copy_(torch.from_numpy((self.hist + (i + 1) * self.new).astype(np.int32)))
        for x, y in zip((self.q, self.k, self.v), self.qkv[i]):
            x.copy_(y)
        self.out.fill_(7.0)

    def check(self, i):
        kv = self.hist + (i + 1) * self.new
        for b in range(len(self.new)):  # the new keys and values are in their places
            p = np.arange(kv[b] - self.new[b], kv[b])
            rows = slice(int(self.off[b]), int(self.off[b + 1]))
            at = torch.from_numpy(self.table[b, p // 16].astype(np.int64)), torch.from_numpy(p % 16)
            assert torch.equal(self.kp[at], self.k[rows]) and torch.equal(self.vp[at], self.v[rows])
        ref, bound = layer.attention(self.kp, self.vp, self.q, self.off, kv, self.table, 0.125, 1 / 600)
        assert np.all(np.abs(layer.f64(self.out) - ref) <= 2.0 ** -8 * np.abs(ref) + bound)


@pytest.mark.parametrize("own_workspace", [True, False])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("width,new", FORMS)
def test_captured_steps_with_parts(width, new, d, own_workspace):
    # as the captured step above, in the forms that sum parts of cut items
    g = Growing([30, 500, 62], new, width, 4, 2, d, seed=90 + d)
    ws = g.workspace() if own_workspace else None
    graph = g.capture(ws)
    for i in range(g.steps):
        g.step(i)
        graph.replay()
        torch.cuda.synchronize()
        g.check(i)
    if own_workspace:
        assert ws[8192:].any(), "no item was cut: this is not the form that the test is for"
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


@pytest.mark.parametrize("first,second", [(0, 1), (0, 2), (2, 2)])
def test_two_streams_with_parts(first, second):
    a, b = (Growing([3000, 90, 700], FORMS[f][1], FORMS[f][0], 1, 2, 64, seed=97 + f) for f in (first, second))
    a.step(0), b.step(0)
    wa, wb = a.workspace(), b.workspace()
    streams = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    a.call(wa), b.call(wb)
    torch.cuda.synchronize()
    a.check(0), b.check(0)
    ra, rb = a.out.clone(), b.out.clone()
    assert wa[8192:].any() and wb[8192:].any()
    for own in (True, False):
        for _ in range(20):
            a.out.fill_(7.0), b.out.fill_(7.0)
            torch.cuda.synchronize()
            for _ in range(3):
                a.call(wa if own else None, stream=streams[0])
                b.call(wb if own else None, stream=streams[1])
            torch.cuda.synchronize()
            assert torch.equal(a.out, ra) and torch.equal(b.out, rb)


@pytest.mark.parametrize("page", [512, 1024, 4096])
@pytest.mark.parametrize("d,heads", [(32, 16), (64, 5), (128, 12)])
@pytest.mark.parametrize("name", ["one token", "candidates", "candidate chunks"])
@pytest.mark.parametrize("wide", [False, True])
def test_large_pages_and_many_heads(wide, name, d, heads, page):
    hist, new, nt = SHAPES[name]
    s = Setup(hist, new, page, heads, d, nt, seed=page + d, pad=1, width=-(-10000 // page) if wide else 1)
    s.check(s.attend())
    k, v = s.k.cuda(), s.v.cuda()
    binding.hstu_cache_append(s.cache, s.batch, k, v)
    a = s.host.keep
    kp, vp, _ = layer.append(s.kp, s.vp, s.k, s.v, s.q, a["q_offsets"], a["kv_lens"], a["page_table"])
    assert np.array_equal(layer.f64(s.kd), kp, equal_nan=True)
    assert np.array_equal(layer.f64(s.vd), vp, equal_nan=True)


@pytest.mark.parametrize("new,width", [(1, 1), (1, 700), (16, 700)])
def test_giving_up_before_the_first_block(new, width):
    s = Setup([5000, 40, 1300], [new, 1, 3], 32, 2, 64, seed=61 + new, width=width)
    good, ws, q = s.attend(), s.workspace(), s.q.cuda()
    for _ in range(5):
        binding.hstu_set_wait_timeout_ns(1)
        binding.hstu_set_debug_flags(binding.HSTU_DEBUG_UNSIGNALLED_WAIT)
        try:
            out = s.attend(q=q, workspace=ws)
        finally:
            binding.hstu_set_debug_flags(0)
            binding.hstu_set_wait_timeout_ns(0)
        after = s.attend(q=q)
        status, site = binding.hstu_last_status()
        assert status == binding.HSTU_ERR_TIMEOUT and site != 0
        assert (out == 7.0).all() and torch.equal(after, good)
        ws.zero_()
        assert torch.equal(s.attend(q=q, workspace=ws), good)


@pytest.mark.parametrize("width", [1, 700])
def test_a_bound_of_no_tokens(width):
    s = Setup([40, 7], [2, 1], 16, 2, 64, seed=82, width=width, max_q=0)
    out = s.attend()  # both sequences have more new tokens than the bound
    assert binding.hstu_last_status()[0] == binding.HSTU_ERR_INVALID_ARG
    assert (out == 7.0).all()
    s.dev["q_offsets"].zero_()
    assert (s.attend() == 7.0).all()
    assert binding.hstu_last_status() == (binding.HSTU_OK, 0)
