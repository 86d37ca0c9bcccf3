"""Bounded device-side waits: a wait that runs out returns instead of hanging.

The kernel's waits are limited by %globaltimer.  The test hook
HSTU_DEBUG_UNSIGNALLED_WAIT makes the MMA warp wait on a barrier that
nothing signals; with a 1 ms limit that wait gives up, and the kernel must
then drain its own copies and MMAs, free TMEM and return, report
HSTU_ERR_TIMEOUT through hstu_last_status, and leave the context usable for
the next (normal) launch.  Nothing here faults or traps the GPU.
"""
import numpy as np
import pytest
import torch

from hstu_jagged_attention_gb300 import binding, build, workloads
from tests import parity

pytestmark = pytest.mark.gpu


def test_wait_limit_gives_timeout_status_and_context_survives():
    build.build()
    w = workloads.custom([700, 300, 5], heads=2, d=64)
    q, k, v = parity.to_device(*workloads.draw_qkv(w, seed=21))
    binding.hstu_last_status()  # clear
    try:
        binding.hstu_set_wait_timeout_ns(1_000_000)
        binding.hstu_set_debug_flags(binding.HSTU_DEBUG_UNSIGNALLED_WAIT)
        out = torch.zeros_like(q)
        plan = binding.hstu_plan_create(w.offsets, w.batch, w.heads, w.d, w.max_seqlen)
        binding.hstu_attn_fwd_plan(plan, q, k, v, w.alpha, w.inv_n, out)
        torch.cuda.synchronize()
        st, site = binding.hstu_last_status()
        assert st == binding.HSTU_ERR_TIMEOUT
        assert site > 0
    finally:
        binding.hstu_set_debug_flags(0)
        binding.hstu_set_wait_timeout_ns(0)
    # the context is still usable and a normal launch is correct
    out = parity.run_plan(w, q, k, v)
    assert binding.hstu_last_status() == (binding.HSTU_OK, 0)
    assert torch.isfinite(out.float()).all()
    binding.hstu_plan_destroy(plan)


def _forward(flags, d, targets=False):
    w = workloads.custom([700, 300, 5, 1024], heads=2, d=d, sigma=1.0 if d < 128 else 0.5)
    q, k, v = parity.to_device(*workloads.draw_qkv(w, seed=31))
    nt = np.array([100, 300, 0, 1], dtype=np.int32) if targets else None
    plan = binding.hstu_plan_create_ex(w.offsets, nt, w.batch, w.heads, w.d, w.max_seqlen, flags)

    def run():
        out = torch.zeros_like(q)
        binding.hstu_attn_fwd_plan(plan, q, k, v, w.alpha, w.inv_n, out)
        return [out]
    return run


def _backward(d, targets=False):
    w = workloads.custom([700, 300, 5, 1024], heads=2, d=d, sigma=1.0 if d < 128 else 0.5)
    q, k, v = parity.to_device(*workloads.draw_qkv(w, seed=32))
    do = torch.randn_like(q.float()).bfloat16()
    nt = np.array([100, 300, 0, 1], dtype=np.int32) if targets else None

    def run():
        g = [torch.zeros_like(q) for _ in range(3)]
        binding.hstu_attn_bwd_ex(q, k, v, do, w.offsets, w.batch, w.heads, w.d, w.max_seqlen, w.alpha,
                                 w.inv_n, *g, num_targets=nt)
        return g
    return run


@pytest.mark.parametrize("name,make", [
    ("forward 32", lambda: _forward(0, 32)), ("forward 64", lambda: _forward(0, 64)),
    ("forward 128", lambda: _forward(0, 128)), ("candidates 64", lambda: _forward(0, 64, True)),
    ("pairs 64", lambda: _forward(binding.HSTU_PLAN_PAIRS, 64)),
    ("pairs 128", lambda: _forward(binding.HSTU_PLAN_PAIRS, 128)),
    ("backward 64", lambda: _backward(64)), ("backward 128", lambda: _backward(128)),
    ("backward candidates 32", lambda: _backward(32, True))])
def test_giving_up_at_once_leaves_nothing_behind(name, make):
    # a limit that runs out while copies and products are on their way: the
    # calls behind it are right (dQ is summed in any order: within its rounding)
    build.build()
    run = make()
    good = run()
    binding.hstu_last_status()
    for _ in range(5):
        binding.hstu_set_wait_timeout_ns(1)
        try:
            run()
        finally:
            binding.hstu_set_wait_timeout_ns(0)
        after = run()
        st, site = binding.hstu_last_status()
        assert st in (binding.HSTU_OK, binding.HSTU_ERR_TIMEOUT) and (st == binding.HSTU_OK) == (site == 0)
        for i, (x, y) in enumerate(zip(after, good)):
            if i == 0 and len(good) == 3:
                # a bf16 step, and 2^-16 of the largest for fp32 sums that cancel
                tol = 2.0 ** -7 * y.float().abs() + 2.0 ** -16 * y.float().abs().max()
                assert ((x.float() - y.float()).abs() <= tol).all()
            else:
                assert torch.equal(x, y)
    assert binding.hstu_last_status() == (binding.HSTU_OK, 0)
