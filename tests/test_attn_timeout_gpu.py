"""The bounded waits of the softmax attention kernels: a test hook makes one role wait on a barrier that nothing
arrives at; the call records BDLA_ERR_TIMEOUT, and the next ordinary call on the same context is right."""
import pytest
import torch

import _attn_ref as ref
from chunked_linear_attention_bounded_gb300 import bdla

pytestmark = pytest.mark.gpu
ROLES = [bdla.STALL_PRODUCER, bdla.STALL_MMA, bdla.STALL_EPILOGUE]


@pytest.mark.parametrize("role", ROLES)
@pytest.mark.parametrize("T", [100, 500])
def test_expired_wait_reports_timeout_and_the_context_stays_usable(role, T):
    g = torch.Generator(device="cuda")
    g.manual_seed(T)
    rn = lambda h: torch.randn((1, T, h, 128), generator=g, device="cuda").bfloat16()
    q, k, v, dO = rn(4), rn(2), rn(2), rn(4)
    want = ref.attn(q, k, v, 0.09, None, dO)
    o, lse = want["o"][0].bfloat16(), want["lse"][0].float()
    ws = bdla.Workspace(1 << 20, "cuda")
    try:
        bdla.set_wait_limit_ns(20_000_000)
        bdla.set_test_stall(bdla.KERNEL_ATTN_FWD, role)
        bdla.attn_fwd(q, k, v, scale=0.09, ws=ws)
        assert ws.read_device_status() == bdla.ERR_TIMEOUT
        bdla.set_test_stall(bdla.KERNEL_ATTN_BWD, role)
        bdla.attn_bwd(q, k, v, o, lse, dO, scale=0.09, ws=ws)
        assert ws.read_device_status() == bdla.ERR_TIMEOUT
    finally:
        bdla.set_test_stall(bdla.KERNEL_ATTN_FWD, bdla.STALL_NONE)
        bdla.set_test_stall(bdla.KERNEL_ATTN_BWD, bdla.STALL_NONE)
        bdla.set_wait_limit_ns(0)
    got_o, got_l = bdla.attn_fwd(q, k, v, scale=0.09, ws=ws)
    ref.check("o", got_o, want["o"])
    ref.check("lse", got_l, want["lse"])
    for n, x in zip(("dq", "dk", "dv"), bdla.attn_bwd(q, k, v, o, lse, dO, scale=0.09, ws=ws)):
        ref.check(n, x, want[n])
    assert ws.read_device_status() == bdla.OK


@pytest.mark.parametrize("role", ROLES)
@pytest.mark.parametrize("page", [32, 24])   # by TMA, and row by row
@pytest.mark.parametrize("n", [60, 700])
def test_expired_wait_over_the_cache(role, page, n):
    g = torch.Generator(device="cuda")
    g.manual_seed(n + page)
    T, width = 20, -(-(n + 20) // page)
    kc, vc = (torch.randn((width, page, 2, 64), generator=g, device="cuda").bfloat16() for _ in range(2))
    q = torch.randn((1, T, 8, 64), generator=g, device="cuda").bfloat16()
    table = torch.arange(width, dtype=torch.int32, device="cuda")[None].contiguous()
    lens = torch.tensor([n], dtype=torch.int32, device="cuda")
    ws = bdla.Workspace(1 << 24, "cuda")
    try:
        bdla.set_wait_limit_ns(20_000_000)
        bdla.set_test_stall(bdla.KERNEL_ATTN_CACHED, role)
        bdla.attn_cached(q, kc, vc, table, lens, ws=ws)
        assert ws.read_device_status() == bdla.ERR_TIMEOUT
    finally:
        bdla.set_test_stall(bdla.KERNEL_ATTN_CACHED, bdla.STALL_NONE)
        bdla.set_wait_limit_ns(0)
    o, lse = bdla.attn_cached(q, kc, vc, table, lens, ws=ws)
    want_o, want_l = ref.cached(q, kc, vc, table, [n], None, 0.125)
    ref.check("o", o, want_o)
    ref.check("lse", lse, want_l)
    assert ws.read_device_status() == bdla.OK
