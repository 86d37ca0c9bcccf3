"""The layer norm with its gate and residual on the GPU, forward and backward,
against the 64-bit forms of oracle/layer.py.

Tolerances.  Every stored bf16 is half a step off (2^-8 of the value).  Before
that, with k = 1 + the row's largest |z - mean| / std + |mean| / std (what an
fp32 rounding of a row's values, 2^-24 of their size, is worth in units of its
standard deviation) and sums of at most 8 * 4 terms a lane and 8 joins
(40 roundings): an error of 2^-24 * 48 * k <= 2^-18 k of each normalised value
and, relative, of rstd.  The outputs are products and sums of a few of these:
2^-16 k of their terms' sizes.  dgamma and dbeta also add rows one after the
other: (16 + rows / 64) roundings of 2^-24 of the sum of sizes.
"""
import numpy as np
import pytest
import torch

from hstu_jagged_attention_gb300 import binding, build, workloads
from oracle import layer, reference
from tests import parity

pytestmark = pytest.mark.gpu
EPS = 1e-6


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()
    yield
    parity.assert_device_ok()


def _k(z, eps):
    dev = z - z.mean(axis=1, keepdims=True)
    std = np.sqrt((dev ** 2).mean(axis=1, keepdims=True) + eps)
    return 1 + (np.abs(dev).max(axis=1, keepdims=True) + np.abs(z.mean(axis=1, keepdims=True))) / std


def make(rows, width, gate, residual, seed=0, offset=0.0, device="cuda"):
    gen = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=gen, dtype=torch.float32)
    a = dict(x=(r(rows, width) + offset).bfloat16(), gamma=1 + 0.1 * r(width), beta=0.1 * r(width))
    if gate:
        a["u"] = r(rows, width).bfloat16()
    if residual:
        a["residual"] = r(rows, width).bfloat16()
    return a, r(rows, width).bfloat16(), r(rows, width).bfloat16()


def to_gpu(a):
    return {k: v.cuda() for k, v in a.items()}


def check_fwd(a, y, z, eps, scale):
    ref_y, ref_z = layer.norm_fwd(**a, eps=eps, scale=scale)
    k = _k(ref_z, eps)
    xhat, _ = layer.standard(ref_z, eps)
    u = np.abs(layer.f64(a["u"])) if "u" in a else 1.0
    size = (k * np.abs(layer.f64(a["gamma"])) + np.abs(layer.f64(a["beta"]))) * u
    assert np.all(np.abs(layer.f64(y) - ref_y) <= 2.0 ** -8 * np.abs(ref_y) + 2.0 ** -16 * size)
    if z is not None:
        parts = np.abs(scale * layer.f64(a["x"])) + np.abs(layer.f64(a["residual"]))
        assert np.all(np.abs(layer.f64(z) - ref_z) <= 2.0 ** -8 * np.abs(ref_z) + 2.0 ** -22 * parts)


def run_fwd(a, eps, scale):
    y = torch.empty_like(a["x"])
    z = torch.empty_like(a["x"]) if "residual" in a else None
    binding.hstu_norm_fwd(y=y, z=z, eps=eps, scale=scale, **a)
    return y, z


def run_bwd(dy, z, a, eps, dz_in=None, dx=False, scale=1.0, workspace=None):
    width = z.shape[1]
    o = dict(dz=torch.empty_like(z), dgamma=torch.full((width,), 9.0, device="cuda"),
             dbeta=torch.full((width,), 9.0, device="cuda"))
    if "u" in a:
        o["du"] = torch.empty_like(z)
    if dx:
        o["dx"] = torch.empty_like(z)
    binding.hstu_norm_bwd(dy, z, a["gamma"], a["beta"], eps, u=a.get("u"), dz_in=dz_in, scale=scale,
                          workspace=workspace, **o)
    return o


def check_bwd(o, dy, z, a, eps, dz_in=None, scale=1.0):
    ref = layer.norm_bwd(dy, z, a["gamma"], a["beta"], eps, a.get("u"), dz_in, scale)
    z, dy = layer.f64(z), layer.f64(dy)
    k = _k(z, eps)
    xhat, rstd = layer.standard(z, eps)
    g = dy * layer.f64(a["u"]) if "u" in a else dy
    gm, bt = np.abs(layer.f64(a["gamma"])), np.abs(layer.f64(a["beta"]))
    aa = np.abs(g) * gm
    size = rstd * (aa + aa.mean(axis=1, keepdims=True) * (1 + k * np.abs(xhat))) * k
    size = size + (0 if dz_in is None else np.abs(layer.f64(dz_in)))
    for name, s in (("dz", size), ("dx", abs(scale) * size), ("du", np.abs(dy) * (k * gm + bt))):
        if name in o:
            err = np.abs(layer.f64(o[name]) - ref[name])
            assert np.all(err <= 2.0 ** -8 * np.abs(ref[name]) + 2.0 ** -16 * s), name
    rows = len(z)
    for name, s in (("dgamma", np.abs(g) * k), ("dbeta", np.abs(g))):
        err = np.abs(layer.f64(o[name]) - ref[name])
        tol = 2.0 ** -18 * s.sum(axis=0) + (16 + rows / 64) * 2.0 ** -24 * s.sum(axis=0)
        assert np.all(err <= tol), name


WIDTHS = [8, 40, 64, 72, 128, 256, 264, 512, 520, 1024, 1032, 2048, 2056, 4096, 8192]


@pytest.mark.parametrize("gate,residual", [(False, False), (True, False), (False, True), (True, True)])
@pytest.mark.parametrize("width", WIDTHS)
def test_every_width(width, gate, residual):
    for rows in (1, 7, 133):
        a, dy, dz_in = make(rows, width, gate, residual, seed=width + rows)
        scale = 0.25 if residual else 1.0
        dev = to_gpu(a)
        y, z = run_fwd(dev, EPS, scale)
        check_fwd(a, y, z, EPS, scale)
        z_in = dev["x"] if z is None else z
        o = run_bwd(dy.cuda(), z_in, dev, EPS, dz_in.cuda() if residual else None, residual, scale)
        check_bwd(o, dy, z_in, a, EPS, dz_in if residual else None, scale)


def test_many_rows_and_repeats():
    a, dy, _ = make(70001, 64, True, False, seed=1)
    dev = to_gpu(a)
    y, _ = run_fwd(dev, EPS, 1.0)
    check_fwd(a, y, None, EPS, 1.0)
    ws = torch.full((binding.hstu_norm_bwd_workspace_bytes(64),), 255, device="cuda", dtype=torch.uint8)
    o = run_bwd(dy.cuda(), dev["x"], dev, EPS, workspace=ws)
    check_bwd(o, dy, dev["x"], a, EPS)
    p = run_bwd(dy.cuda(), dev["x"], dev, EPS)  # its own allocation: the same bits
    assert all(torch.equal(o[n], p[n]) for n in o)


@pytest.mark.parametrize("width,rows", [(64, 1024), (64, 1025), (256, 255), (256, 256), (256, 257),
                                        (520, 64), (520, 65), (8192, 16), (8192, 17)])
def test_one_cluster_and_many_ctas(width, rows):
    # on both sides of where one cluster takes the whole gradient
    a, dy, dz_in = make(rows, width, True, True, seed=rows)
    dev = to_gpu(a)
    _, z = run_fwd(dev, EPS, 0.5)
    o = run_bwd(dy.cuda(), z, dev, EPS, dz_in.cuda(), True, 0.5)
    check_bwd(o, dy, z, a, EPS, dz_in, 0.5)


def test_rows_with_a_large_mean_and_with_no_spread():
    a, dy, _ = make(50, 256, True, False, seed=2, offset=30.0)
    a["x"][7] = 3.0   # no spread at all: xhat = 0
    a["x"][8] = 0.0
    dev = to_gpu(a)
    y, _ = run_fwd(dev, 1e-3, 1.0)
    check_fwd(a, y, None, 1e-3, 1.0)
    check_bwd(run_bwd(dy.cuda(), dev["x"], dev, 1e-3), dy, dev["x"], a, 1e-3)


def test_slices_of_a_projection():
    a, dy, dz_in = make(300, 256, True, True, seed=3)
    dev = to_gpu(a)
    y, z = run_fwd(dev, EPS, 0.5)
    o = run_bwd(dy.cuda(), z, dev, EPS, dz_in.cuda(), True, 0.5)
    wide = torch.full((300, 4, 256), 5.0, device="cuda", dtype=torch.bfloat16)
    for i, t in enumerate((dev["x"], dev["u"], dev["residual"], dy.cuda())):
        wide[:, i] = t
    sl = dict(dev, x=wide[:, 0], u=wide[:, 1], residual=wide[:, 2])
    y2, z2 = torch.empty_like(y), torch.empty_like(z)
    binding.hstu_norm_fwd(y=y2, z=z2, eps=EPS, scale=0.5, **sl)
    assert torch.equal(y, y2) and torch.equal(z, z2)
    dproj = torch.full((300, 3, 256), 5.0, device="cuda", dtype=torch.bfloat16)
    dz, dx = torch.empty_like(z), torch.empty_like(z)
    dg, db = torch.empty(256, device="cuda"), torch.empty(256, device="cuda")
    binding.hstu_norm_bwd(wide[:, 3], z, dev["gamma"], dev["beta"], EPS, dz, dg, db, u=wide[:, 1],
                          du=dproj[:, 1], dz_in=dz_in.cuda(), dx=dx, scale=0.5)
    assert torch.equal(dz, o["dz"]) and torch.equal(dx, o["dx"]) and torch.equal(dproj[:, 1], o["du"])
    assert torch.equal(dg, o["dgamma"]) and torch.equal(db, o["dbeta"])
    assert (dproj[:, 0] == 5).all() and (dproj[:, 2] == 5).all()


def test_in_place():
    a, dy, dz_in = make(99, 512, True, True, seed=4)
    dev = to_gpu(a)
    y, z = run_fwd(dev, EPS, 0.5)
    x, r = dev["x"].clone(), dev["residual"].clone()
    binding.hstu_norm_fwd(x, dev["gamma"], dev["beta"], EPS, x, u=dev["u"], residual=r, scale=0.5, z=r)
    assert torch.equal(x, y) and torch.equal(r, z)
    o = run_bwd(dy.cuda(), z, dev, EPS, dz_in.cuda(), True, 0.5)
    g = dy.cuda()
    binding.hstu_norm_bwd(g, z, dev["gamma"], dev["beta"], EPS, g, torch.empty(512, device="cuda"),
                          torch.empty(512, device="cuda"), u=dev["u"], du=torch.empty_like(g),
                          dz_in=dz_in.cuda())
    assert torch.equal(g, o["dz"])


def test_no_rows():
    x = torch.empty(0, 64, device="cuda", dtype=torch.bfloat16)
    g = torch.ones(64, device="cuda")
    binding.hstu_norm_fwd(x, g, g, EPS, x)
    dg, db = torch.full((64,), 3.0, device="cuda"), torch.full((64,), 3.0, device="cuda")
    binding.hstu_norm_bwd(x, x, g, g, EPS, x, dg, db)
    assert not dg.any() and not db.any()


def test_a_nan_row_stays_its_own():
    a, dy, _ = make(64, 128, False, False, seed=5)
    dev = to_gpu(a)
    y, _ = run_fwd(dev, EPS, 1.0)
    dev["x"][9, 3] = float("nan")
    y2, _ = run_fwd(dev, EPS, 1.0)
    keep = torch.arange(64) != 9
    assert torch.equal(y2[keep], y[keep]) and y2[9].isnan().all()


def test_captured():
    a, dy, dz_in = make(200, 256, True, True, seed=6)
    dev = to_gpu(a)
    y, z = run_fwd(dev, EPS, 0.5)
    o = run_bwd(dy.cuda(), z, dev, EPS, dz_in.cuda(), True, 0.5)
    x, g, d = torch.zeros_like(dev["x"]), torch.zeros_like(z), torch.zeros_like(z)
    live = dict(dev, x=x)
    y2, z2 = torch.empty_like(y), torch.empty_like(z)
    p = {n: torch.empty_like(t) for n, t in o.items()}
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        binding.hstu_norm_fwd(y=y2, z=z2, eps=EPS, scale=0.5, **live)
        binding.hstu_norm_bwd(g, z2, dev["gamma"], dev["beta"], EPS, u=dev["u"], dz_in=d, scale=0.5, **p)
    for _ in range(2):
        x.copy_(dev["x"]), g.copy_(dy), d.copy_(dz_in)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y2, y) and torch.equal(z2, z) and all(torch.equal(p[n], o[n]) for n in o)


def test_refusals():
    a, dy, _ = make(4, 64, True, False)
    dev, y = to_gpu(a), torch.empty(4, 64, device="cuda", dtype=torch.bfloat16)
    call = lambda **kw: binding.hstu_norm_fwd(**{**dict(
        x=dev["x"], gamma=dev["gamma"], beta=dev["beta"], eps=EPS, y=y), **kw})
    call()
    for kw in (dict(x=dev["x"].float()), dict(x=a["x"]), dict(gamma=dev["gamma"][:32]), dict(u=dev["u"][:2]),
               dict(gamma=dev["gamma"].double()), dict(y=torch.empty(4, 128, device="cuda",
                                                                      dtype=torch.bfloat16)[:, ::2])):
        with pytest.raises(ValueError):
            call(**kw)
    for kw in (dict(u=dev["u"][:1].expand(4, 64)), dict(eps=-1.0), dict(z=y),
               dict(residual=dev["u"])):
        with pytest.raises(binding.HstuError) as e:
            call(**kw)
        assert e.value.code == binding.HSTU_ERR_INVALID_ARG


def test_matches_the_fused_output_stage():
    # the attention, then Norm (.) U on its bf16 output, against the fused call
    w = workloads.custom([700, 129, 1, 512], heads=4, d=64, inv_n=1.0)
    q, k, v = workloads.draw_qkv(w, seed=670)
    u, g, b = workloads.draw_norm_gate(w, seed=671)
    qd, kd, vd, ud = (t.cuda() for t in (q, k, v, u))
    gd, bd = torch.from_numpy(g).cuda(), torch.from_numpy(b).cuda()
    o, y = torch.empty_like(qd), torch.empty_like(qd)
    args = (w.offsets, w.batch, w.heads, w.d, w.max_seqlen, w.alpha, w.inv_n)
    binding.hstu_attn_fwd(qd, kd, vd, *args, o)
    binding.hstu_norm_fwd(o.flatten(1), gd, bd, EPS, y.flatten(1), u=ud.flatten(1))
    ref = reference.hstu_fwd_norm_gate(q, k, v, u, g, b, EPS, w.offsets, w.alpha, w.inv_n)
    # o is rounded: 2^-8 of it moves xhat by 2^-8 (|x| + mean |x|) rstd at most
    x = np.abs(layer.f64(o).reshape(w.total, -1))
    rstd = layer.standard(layer.f64(o).reshape(w.total, -1), EPS)[1]
    gu = np.abs(g)[None, :] * np.abs(layer.f64(u).reshape(w.total, -1))
    spread = (x + x.mean(axis=1, keepdims=True) + (x ** 2).mean(axis=1, keepdims=True) * rstd * rstd * x) * rstd
    rms = float(np.sqrt(np.mean(ref ** 2)))
    ref = ref.reshape(w.total, -1)
    tol = 2.0 ** -8 * (spread * gu + np.abs(ref)) + 1e-3 * rms
    assert np.all(np.abs(layer.f64(y).reshape(w.total, -1) - ref) <= tol)


@pytest.mark.parametrize("width", [2056, 4096, 4104, 8192])
@pytest.mark.parametrize("rows", [9, 12, 16])
def test_sums_of_one_cluster_with_a_row_a_cta(rows, width):
    # a CTA holds one row at a time and sums dgamma and dbeta where its copies of
    # the rows past the end (zeros) land: no column may be lost, ever
    a, dy, dz_in = make(rows, width, True, True, seed=rows + width)
    dev = to_gpu(a)
    _, z = run_fwd(dev, EPS, 0.5)
    dy_d, in_d = dy.cuda(), dz_in.cuda()
    first = run_bwd(dy_d, z, dev, EPS, in_d, True, 0.5)
    check_bwd(first, dy, z, a, EPS, dz_in, 0.5)
    for _ in range(100):
        o = run_bwd(dy_d, z, dev, EPS, in_d, True, 0.5)
        assert torch.equal(o["dgamma"], first["dgamma"]) and torch.equal(o["dbeta"], first["dbeta"])


@pytest.mark.parametrize("own_workspace", [True, False])
@pytest.mark.parametrize("rows,width", [(1000, 256), (300, 1032)])
def test_captured_in_two_launches(rows, width, own_workspace):
    # more rows than one cluster takes: parts in a workspace, or in an
    # allocation inside the graph, and a second launch that sums them
    a, dy, dz_in = make(rows, width, True, True, seed=8)
    dev = to_gpu(a)
    _, z = run_fwd(dev, EPS, 0.5)
    o = run_bwd(dy.cuda(), z, dev, EPS, dz_in.cuda(), True, 0.5)
    check_bwd(o, dy, z, a, EPS, dz_in, 0.5)
    ws = torch.zeros(binding.hstu_norm_bwd_workspace_bytes(width), device="cuda", dtype=torch.uint8) \
        if own_workspace else None
    g, d = torch.zeros_like(z), torch.zeros_like(z)
    p = {n: torch.zeros_like(t) for n, t in o.items()}
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        binding.hstu_norm_bwd(g, z, dev["gamma"], dev["beta"], EPS, u=dev["u"], dz_in=d, scale=0.5,
                              workspace=ws, **p)
    for _ in range(3):
        g.copy_(dy), d.copy_(dz_in)
        for t in p.values():
            t.fill_(9.0)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p[n], o[n]) for n in o)
    assert ws is None or ws.any(), "the gradient ran in one launch"
