"""The cache of 4-bit codes without a GPU: the sizes and refusals of its entry
points, and the 64-bit form of what is held."""
import ctypes
import os
import re
import subprocess
import sys

import numpy as np
import pytest

from hstu_jagged_attention_gb300 import binding, build
from oracle import layer
from tests.test_cache import make_batch

OK, BAD = binding.HSTU_OK, binding.HSTU_ERR_INVALID_ARG


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()


@pytest.mark.parametrize("page,heads,d", [(16, 1, 32), (64, 4, 64), (128, 3, 128), (4096, 2, 64)])
def test_page_bytes(page, heads, d):
    assert binding.hstu_cache_q4_page_bytes(page, heads, d) == page * heads * (d // 2 + d // 16) * 2


def test_refusals_on_the_host():
    L, h, n = binding.lib(), ctypes.c_void_p(), ctypes.c_size_t()
    for args, code in (((24, 1, 64), BAD), ((8, 1, 64), BAD), ((8192, 1, 64), BAD), ((16, 0, 64), BAD),
                       ((16, 65537, 64), BAD), ((16, 1, 96), binding.HSTU_ERR_UNSUPPORTED)):
        assert L.hstu_cache_q4_page_bytes(*args, ctypes.byref(n)) == code, args
    assert L.hstu_cache_q4_page_bytes(16, 1, 64, None) == BAD
    make = lambda **kw: L.hstu_cache_create_q4(*[kw.get(n, v) for n, v in dict(
        pages=16, num_pages=4, page_size=16, heads=2, d=64, stride=0).items()], ctypes.byref(h))
    packed = 16 * 2 * 72
    assert make(d=96) == binding.HSTU_ERR_UNSUPPORTED
    for kw in (dict(pages=0), dict(pages=8), dict(num_pages=0), dict(page_size=24), dict(page_size=8),
               dict(page_size=8192), dict(heads=0), dict(stride=packed - 16), dict(stride=packed + 8),
               dict(stride=-packed), dict(stride=1 << 61),
               dict(num_pages=2 ** 31 - 1, stride=1 << 40)):
        assert make(**kw) == BAD and not h, kw
    assert L.hstu_cache_create_q4(16, 4, 16, 2, 64, 0, None) == BAD
    assert L.hstu_cache_read(None, None, None, 0, None, 0, None) == BAD
    for kw in (dict(page_size=24), dict(d=40), dict(heads=0)):
        with pytest.raises(binding.HstuError):
            binding.hstu_cache_q4_page_bytes(**{**dict(page_size=16, heads=1, d=64), **kw})


def test_a_cache_of_another_device_is_refused(monkeypatch):
    torch = pytest.importorskip("torch")

    class Pool:  # what the binding asks of a tensor on the second GPU
        shape, is_cuda, ndim, dtype = torch.Size((4, 16 * 2 * 72)), True, 2, torch.uint8
        device = torch.device("cuda:1")
        stride = staticmethod(lambda: (16 * 2 * 72, 1))
        data_ptr = staticmethod(lambda: 1 << 20)

    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    with pytest.raises(ValueError, match="current device"):
        binding.hstu_cache_create_q4(Pool, 16, 2, 64)
    with pytest.raises(ValueError):
        binding.hstu_cache_create_q4(torch.zeros(4, 16 * 2 * 72, dtype=torch.uint8), 16, 2, 64)


@pytest.mark.parametrize("q4", [False, True])
def test_pages_that_share_memory_are_refused(monkeypatch, q4):
    # a broadcast pool's stride is 0, which the library would take for packed
    # pages, past the end of the one page that there is
    torch = pytest.importorskip("torch")

    class Pool:  # what the binding asks of a device tensor
        shape = torch.Size((4, 16 * 2 * 72) if q4 else (4, 16, 2, 64))
        is_cuda, ndim, dtype, device = True, len(shape), torch.uint8 if q4 else torch.bfloat16, torch.device("cuda:0")
        stride = staticmethod(lambda: (0, 1) if q4 else (0, 128, 64, 1))
        data_ptr = staticmethod(lambda: 1 << 20)

    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    with pytest.raises(ValueError, match="share memory"):
        binding.hstu_cache_create_q4(Pool, 16, 2, 64) if q4 else binding.hstu_cache_create(Pool, Pool)


# ------------------------------------------------- the 64-bit form itself
def bf16(x):
    torch = pytest.importorskip("torch")
    return torch.from_numpy(np.asarray(x, dtype=np.float32)).bfloat16().double().numpy()


def test_the_scales():
    s = layer.SCALES
    assert s[0] == 2.0 ** -20 and s[255] == 3840.0 and np.all(np.diff(s) > 0)
    assert np.allclose(s[8:] / s[:-8], 2.0, rtol=0, atol=0)
    # whatever is held is a bf16 number
    held = (np.arange(-7, 8)[:, None] * s).reshape(-1)
    assert np.array_equal(bf16(held), held)
    # and so is every tie, and every bound on a group's largest value
    ties = ((np.arange(7) + 0.5)[:, None] * s).reshape(-1)
    assert np.array_equal(bf16(ties), ties) and np.array_equal(bf16(7 * s), 7 * s)


def test_what_is_held_is_near():
    rng = np.random.default_rng(0)
    x = bf16(rng.standard_normal((4000, 64)) * np.exp(3 * rng.standard_normal((4000, 1))))
    code, j = layer.q4_codes(x)
    held, s, most = layer.q4_held(x), layer.SCALES[j], np.abs(x.reshape(4000, 4, 16)).max(axis=-1)
    fits = most <= 7 * 3840.0
    assert np.all(np.abs(code) <= 7) and np.all((7 * s >= most)[fits]) and np.all(j[~fits] == 255)
    assert np.all((7 * layer.SCALES[j - 1] < most)[j > 0])
    near = np.abs(held - x).reshape(4000, 4, 16).max(axis=-1) <= s / 2
    assert np.all(near[fits]) and not np.any(near[most > 7.5 * 3840.0])
    assert np.array_equal(layer.q4_held(-x), -held)
    four = (j > 0) & (j < 240)  # the scale times 4 is a scale
    by_group = lambda a: a.reshape(4000, 4, 16)[four]
    assert np.array_equal(by_group(layer.q4_held(x * 4)), by_group(held * 4))


@pytest.mark.parametrize("x,held", [
    ([0.0] * 16, [0.0] * 16),
    ([7.0, 0.5, -0.5, 1.5, -2.5, 0.498046875, 6.5, 3.0] + [0.0] * 8,  # s = 1: ties go away from zero
     [7.0, 1.0, -1.0, 2.0, -3.0, 0.0, 7.0, 3.0] + [0.0] * 8),
    ([7.03125] + [0.0] * 15, [6 * 1.125] + [0.0] * 15),  # past 7: the next scale is 9 / 8
    ([np.nan, 7.0] + [2.0] * 14, [0.0, 7.0] + [2.0] * 14),
    ([np.inf, -np.inf, 7.0] + [26000.0] * 13, [26880.0, -26880.0, 0.0] + [26880.0] * 13),
    ([1e30, -26880.0, 1920.0, 1900.0] + [0.0] * 12, [26880.0, -26880.0, 3840.0, 0.0] + [0.0] * 12),
    ([2.0 ** -21, -2.0 ** -22, 2.0 ** -20] + [0.0] * 13, [2.0 ** -20, 0.0, 2.0 ** -20] + [0.0] * 13),
])
def test_values_worked_by_hand(x, held):
    assert layer.q4_held(np.array(x)).tolist() == held


@pytest.mark.parametrize("page,heads,d", [(16, 2, 32), (256, 1, 64), (128, 3, 128)])
def test_pages_hold_what_was_packed(page, heads, d):
    rng = np.random.default_rng(1)
    k, v = rng.standard_normal((2, 3, page, heads, d))
    pages = layer.q4_pack(k, v)
    assert pages.shape == (3, binding.hstu_cache_q4_page_bytes(page, heads, d))
    ku, vu = layer.q4_unpack(pages, page, heads, d)
    assert np.array_equal(ku, layer.q4_held(k)) and np.array_equal(vu, layer.q4_held(v))
    # by hand: token 5, last head, channels 8 .. 15 are the second word of its codes
    t = min(page, 128)
    tile = (heads - 1) * (page // t) * t * d * 9 // 8
    word = int.from_bytes(pages[1, tile + 5 * d // 2 + 4:tile + 5 * d // 2 + 8].tobytes(), "little")
    s = layer.SCALES[pages[1, tile + t * d + 5 * d // 16]]
    for c in range(8):
        q = word >> (16 * (c % 2) + 4 * (c // 2)) & 15
        assert ku[1, 5, heads - 1, 8 + c] == ((q ^ 8) - 8) * s


def test_zeroed_pages_hold_zeros_and_any_bytes_are_finite():
    assert not np.any(layer.q4_unpack(np.zeros((1, 16 * 72), np.uint8), 16, 1, 64))
    ends = np.full((1, 16 * 72), 255, np.uint8)
    k, v = layer.q4_unpack(ends, 16, 1, 64)
    assert np.all(k == -3840.0) and np.all(np.isfinite(v))


# ----------------------------------------------- the shares, without a GPU
@pytest.mark.parametrize("hist,new", [([], []), ([5, 6], [0, 0]), ([0], [0])])
@pytest.mark.parametrize("grid", [1, 15, 16, 500])
def test_a_batch_without_work_has_no_shares(hist, new, grid):
    # in a process of its own: it ended with a division by zero
    code = (f"import numpy as np\nfrom hstu_jagged_attention_gb300 import binding\n"
            f"from tests.test_cache import make_batch\n"
            f"b, n, rows = make_batch(np.array({hist}, dtype=int), np.array({new}, dtype=int), 16)\n"
            f"assert binding.hstu_cache_worklist(b, n, 16, rows, 2, 16, 128, {grid}).shape == (0, 8)\n")
    assert subprocess.run([sys.executable, "-c", code], cwd=build.ROOT).returncode == 0


@pytest.mark.parametrize("most_parts", [16, 32, 5])
@pytest.mark.parametrize("seed", range(10))
def test_the_shares_cover_every_block_once(seed, most_parts):
    # up to three CTAs an SM, and few items on odd seeds, so that the rule on
    # parts counts
    rng = np.random.default_rng(70 + seed)
    n, heads = (int(rng.integers(1, 3)), int(rng.integers(1, 5))) if seed % 2 else \
        (int(rng.integers(1, 40)), int(rng.integers(1, 9)))
    hist, new = rng.integers(0, 20000, size=n), rng.integers(0 if seed % 4 else 1, 18, size=n)
    nt = [int(rng.integers(0, x + 1)) for x in new]
    grid = int(rng.integers(150, 457)) if seed else 456
    extra = int(rng.integers(0, 3))
    batch, num_pages, rows = make_batch(hist, new, 64, nt, seed)
    segs = binding.hstu_cache_worklist(batch, num_pages, 64, rows, heads, 16, 128, grid, extra=extra,
                                       most_parts=most_parts)
    if most_parts == 16:
        assert np.array_equal(segs, binding.hstu_cache_worklist(batch, num_pages, 64, rows, heads, 16, 128,
                                                                grid, extra=extra))
    tiles = -(-int(new.max()) // 16)
    blocks = {}  # of each item with any, in their order
    for qt in range(tiles):
        for b in range(n):
            last = min(new[b], 16 * qt + 16) - 1
            if 16 * qt <= last:
                p0, p1, seen = hist[b] + 16 * qt, hist[b] + last, hist[b] + new[b] - nt[b]
                m = len({j // 128 for j in range(min(p1 + 1, seen))} | {p // 128 for p in range(p0, p1 + 1)})
                blocks.update({(b, h, qt): m for h in range(heads)})
    total = sum(m + extra for m in blocks.values())
    per, items = max(-(-total // grid), 1), tiles * n * heads
    if 0 < items < grid // most_parts:
        per = max(per, -(-total // (most_parts * items)))
    at, want = 0, []
    for (b, h, qt), m in blocks.items():  # CTA c has units [c per, (c + 1) per)
        c0, c1 = at // per, (at + m - 1) // per
        for c in range(c0, c1 + 1):
            i0, i1 = max(c * per - at, 0), min((c + 1) * per - at, m)
            want.append([c, b, h, qt, i0, i1 - i0, c0, c1 - c0 + 1])
        at += m + extra
    assert sorted(segs.tolist()) == sorted(want)
    assert seed % 2 == 0 or max(x[7] for x in want) > min(most_parts, 16) // 2
    # a CTA starts at most one item that it does not end: its counter is free
    starts = [c for c, *_, c0, parts in want if c == c0 and parts > 1]
    assert len(starts) == len(set(starts))


def test_refusals_of_the_shares():
    b, n, rows = make_batch(np.array([500]), np.array([3]), 16)
    for most_parts in (0, -1):
        with pytest.raises(binding.HstuError) as e:
            binding.hstu_cache_worklist(b, n, 16, rows, 2, 16, 128, 100, most_parts=most_parts)
        assert e.value.code == BAD


# ------------------------------------------- loads of what kernels may write
def test_only_inputs_that_no_kernel_writes_are_loaded_non_coherently():
    # A kernel that starts while the stream's previous one ends sees that one's
    # writes through coherent loads alone; __ldg is for memory that nobody
    # writes while the kernel lives.  No kernel of the library writes rotation
    # and page tables or the norm's weights; the caches' pages, and what is read
    # back, are written by the append and the reading.
    allowed = {"hstu_cache.cu": {"tab", "tab + a.rot / 2"}, "hstu_cache_q4.cu": {"tab", "tab + half"},
               "hstu_norm.cu": {"p + at"}, "hstu_paged.cuh": {"row + p + lane", "row + p + 32 + lane"},
               "hstu_step.cuh": set(), "hstu_q4.cuh": set(), "hstu_fwd_paged.cuh": set()}
    for name, inputs in allowed.items():
        with open(os.path.join(build.CSRC, name)) as f:
            text = re.sub(r"//[^\n]*", "", f.read())
        assert "ld.global.nc" not in text and "__restrict__" not in text, name
        met = set()
        for m in re.finditer(r"__ldg\(", text):
            depth, end = 1, m.end()
            while depth:
                depth += {"(": 1, ")": -1}.get(text[end], 0)
                end += 1
            arg = text[m.end():end - 1]
            met.add(re.sub(r"reinterpret_cast<[^>]*>\((.*?)\)( \+ \w+)?$", r"\1", arg))
        assert met == inputs, (name, met)
