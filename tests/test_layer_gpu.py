"""The operators together, as a layer uses them: serving from the paged cache,
step by step, against the whole sequences at once; and a training step's
gradients against 64-bit autograd of the same layer.

Tolerances.  The layer rounds to bf16 after each operator: normed input,
projection, attention, gated output, and in the gradient dz, dq, dk, dv, du.
Each rounding is at most half a step, 2^-8 of the value, so 2^-8 of an
array's norm; at most eight of them lie between the inputs and any result, and
the layer's maps between them (a layer norm of rows whose standard deviation
is their size, a projection with rows of unit norm, the attention's and the
gate's sums) pass relative errors on with factors of about one: 8 * 2^-8 of
an array's norm.
"""
import numpy as np
import pytest
import torch

from hstu_jagged_attention_gb300 import binding, build, workloads
from tests import parity
from tests.test_cache import make_batch
from tests.test_cache_gpu import rotary_table

pytestmark = pytest.mark.gpu
TOL = 8 * 2.0 ** -8
EPS = 1e-5
HEADS, D = 4, 64
WIDTH = HEADS * D


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()
    binding.hstu_last_status()
    yield
    parity.assert_device_ok()


def close(got, ref):
    got, ref = got.double().cpu(), ref.double().cpu()
    err = float((got - ref).norm() / ref.norm())
    assert err <= TOL, err


class Weights:
    def __init__(self, seed, device="cuda", dtype=torch.bfloat16):
        gen = torch.Generator().manual_seed(seed)
        r = lambda *s: torch.randn(*s, generator=gen)
        self.w_in = (r(WIDTH, 4 * WIDTH) / WIDTH ** 0.5).bfloat16().to(device, dtype)
        self.w_out = (r(WIDTH, WIDTH) / WIDTH ** 0.5).bfloat16().to(device, dtype)
        f = torch.float32 if dtype is torch.bfloat16 else dtype
        self.g1, self.b1, self.g2, self.b2 = ((c + 0.1 * r(WIDTH)).to(device, f) for c in (1, 0, 1, 0))


def project(x, residual, w, scale):
    """(residual stream, U, V, Q, K): residual, norm and the SiLU projection."""
    y, z = torch.empty_like(x), torch.empty_like(x)
    binding.hstu_norm_fwd(x, w.g1, w.b1, EPS, y, residual=residual, scale=scale, z=z)
    p = torch.nn.functional.silu(y @ w.w_in).unflatten(1, (4, HEADS, D))
    return z, p[:, 0].flatten(1), p[:, 1], p[:, 2], p[:, 3]


def gate(attn, u, w):
    y = torch.empty(len(u), WIDTH, device="cuda", dtype=torch.bfloat16)
    binding.hstu_norm_fwd(attn.flatten(1), w.g2, w.b2, EPS, y, u=u)
    return y @ w.w_out


@pytest.mark.parametrize("rotate", [False, True])
def test_serving_by_steps_is_the_whole_at_once(rotate):
    lengths, layers, page = [150, 31, 260], 2, 32
    off = np.concatenate([[0], np.cumsum(lengths)]).astype(np.int32)
    total, inv_n = int(off[-1]), 1.0 / 260
    weights = [Weights(i) for i in range(layers)]
    gen = torch.Generator().manual_seed(9)
    x0 = torch.randn(total, WIDTH, generator=gen).bfloat16().cuda()
    r0 = torch.randn(total, WIDTH, generator=gen).bfloat16().cuda()
    table = rotary_table(300, D).cuda() if rotate else None
    host, num_pages, _ = make_batch([0, 0, 0], lengths, page)
    i32 = lambda a: torch.from_numpy(np.asarray(a, dtype=np.int32)).cuda()
    pages = i32(host.keep["page_table"])
    empty = lambda n: torch.empty(n, HEADS, D, device="cuda", dtype=torch.bfloat16)

    def run(steps):
        """Feed each sequence new[b] tokens a step; the last layer's outputs and residuals."""
        pools = [torch.full((num_pages, 2, page, HEADS, D), float("nan"), device="cuda",
                            dtype=torch.bfloat16) for _ in weights]
        caches = [binding.hstu_cache_create(p[:, 0], p[:, 1]) for p in pools]
        space = torch.zeros(binding.hstu_cache_workspace_bytes(caches[0]), device="cuda", dtype=torch.uint8)
        done = np.zeros(3, dtype=int)
        got_x, got_z = torch.empty_like(x0), torch.empty_like(x0)
        for new in steps:
            rows = torch.from_numpy(np.concatenate(
                [np.arange(off[b] + done[b], off[b] + done[b] + new[b]) for b in range(3)])).cuda()
            done = done + new
            batch = binding.PagedBatch(i32(np.concatenate([[0], np.cumsum(new)])), i32(done), pages,
                                       max_q=int(max(new)))
            x, z = x0[rows], r0[rows]
            for w, cache in zip(weights, caches):
                z, u, v, q, k = project(x, z, w, 0.5)
                out, qr = empty(len(rows)), empty(len(rows))
                binding.hstu_cache_append(cache, batch, k, v, q=q, q_out=qr, rotary=table)
                binding.hstu_attn_fwd_cache(cache, batch, qr, D ** -0.5, inv_n, out, workspace=space)
                x = gate(out, u, w)
            got_x[rows], got_z[rows] = x, z
        assert np.array_equal(done, lengths)
        return got_x, got_z

    whole = run([np.array(lengths)])
    if not rotate:  # the contiguous forward, layer by layer
        x, z = x0, r0
        for w in weights:
            z, u, v, q, k = project(x, z, w, 0.5)
            out = empty(total)
            binding.hstu_attn_fwd(q.contiguous(), k.contiguous(), v.contiguous(), off, 3, HEADS, D, 260,
                                  D ** -0.5, inv_n, out)
            x = gate(out, u, w)
        close(whole[0], x)
        close(whole[1], z)
    by_steps = run([np.array(s) for s in ([100, 0, 200], [1, 1, 1], [1, 1, 1], [40, 20, 50], [7, 8, 7],
                                          [1, 1, 1])])
    close(by_steps[0], whole[0])
    close(by_steps[1], whole[1])


def test_a_training_step_against_autograd():
    lengths = [40, 1, 130, 77]
    off = np.concatenate([[0], np.cumsum(lengths)]).astype(np.int32)
    total, n_max, scale = int(off[-1]), 130, 0.5
    w = Weights(3)
    gen = torch.Generator().manual_seed(4)
    x, res, dy, dz_later = (torch.randn(total, WIDTH, generator=gen).bfloat16() for _ in range(4))
    alpha, inv_n = D ** -0.5, 1.0 / n_max

    # the layer and its gradients on the GPU (the projection's own gradient is a
    # plain product, taken here up to its output)
    z, u, v, q, k = project(x.cuda(), res.cuda(), w, scale)
    u, v, q, k = (t.contiguous() for t in (u, v, q, k))
    o = torch.empty_like(q)
    args = (off, len(lengths), HEADS, D, n_max, alpha, inv_n)
    binding.hstu_attn_fwd(q, k, v, *args, o)
    y = torch.empty(total, WIDTH, device="cuda", dtype=torch.bfloat16)
    binding.hstu_norm_fwd(o.flatten(1), w.g2, w.b2, EPS, y, u=u)
    do, du = torch.empty_like(y), torch.empty_like(y)
    dg2, db2 = torch.empty(WIDTH, device="cuda"), torch.empty(WIDTH, device="cuda")
    binding.hstu_norm_bwd(dy.cuda(), o.flatten(1), w.g2, w.b2, EPS, do, dg2, db2, u=u, du=du)
    dq, dk, dv = (torch.empty_like(q) for _ in range(3))
    binding.hstu_attn_bwd(q, k, v, do.unflatten(1, (HEADS, D)), *args, dq, dk, dv)
    # through the SiLU projection, then the residual and the first norm
    yn = torch.empty_like(y)
    zz = torch.empty_like(y)
    binding.hstu_norm_fwd(x.cuda(), w.g1, w.b1, EPS, yn, residual=res.cuda(), scale=scale, z=zz)
    h = (yn @ w.w_in).float()
    s = torch.sigmoid(h)
    dp = torch.cat([du, dv.flatten(1), dq.flatten(1), dk.flatten(1)], dim=1).float()
    dh = (dp * s * (1 + h * (1 - s))).bfloat16()
    dyn = dh @ w.w_in.T
    dz, dx = torch.empty_like(y), torch.empty_like(y)
    dg1, db1 = torch.empty(WIDTH, device="cuda"), torch.empty(WIDTH, device="cuda")
    binding.hstu_norm_bwd(dyn, zz, w.g1, w.b1, EPS, dz, dg1, db1, dz_in=dz_later.cuda(), dx=dx, scale=scale)

    # the same layer in 64 bits
    w64 = Weights(3, device="cpu", dtype=torch.float64)
    leaves = dict(x=x.double(), res=res.double(), g1=w64.g1, b1=w64.b1, g2=w64.g2, b2=w64.b2)
    for t in leaves.values():
        t.requires_grad_()
    norm = lambda t, g, b: torch.nn.functional.layer_norm(t, (WIDTH,), g, b, EPS)
    z64 = leaves["res"] + scale * leaves["x"]
    p = torch.nn.functional.silu(norm(z64, leaves["g1"], leaves["b1"]) @ w64.w_in).unflatten(1, (4, HEADS, D))
    p.retain_grad()
    u64, v64, q64, k64 = p.unbind(1)
    outs = []
    for b, n in enumerate(lengths):
        rows = slice(int(off[b]), int(off[b + 1]))
        sc = torch.nn.functional.silu(alpha * torch.einsum("ihc,jhc->hij", q64[rows], k64[rows]))
        outs.append(inv_n * torch.einsum("hij,jhc->ihc", sc.tril(), v64[rows]))
    y64 = norm(torch.cat(outs).flatten(1), leaves["g2"], leaves["b2"]) * u64.flatten(1)
    ((y64 * dy.double()).sum() + (z64 * dz_later.double()).sum()).backward()

    close(y, y64.detach())
    for got, i in ((du.unflatten(1, (HEADS, D)), 0), (dv, 1), (dq, 2), (dk, 3)):
        close(got, p.grad[:, i])
    close(dx, leaves["x"].grad)
    close(dz, leaves["res"].grad)
    for got, name in ((dg1, "g1"), (db1, "b1"), (dg2, "g2"), (db2, "b2")):
        close(got, leaves[name].grad)
