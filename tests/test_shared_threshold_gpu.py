"""When a call joins what a group shares by itself (bdla_set_share_least).  What is joined is read as the table of the
group's first sequence says, so the others' entries for it may be anything; what is not joined is read as their own say."""
import pytest
import torch

from chunked_linear_attention_bounded_gb300 import bdla
from test_shared_gpu import _batch, _call

pytestmark = pytest.mark.gpu


# sequences, shared pages of 16, new tokens, heads; elements that joining saves; whether it is done
@pytest.mark.parametrize("n,pages,T,Hq,Hk,saved,joined", [
    (256, 4, 1, 32, 8, 33_423_360, False),   # the tensor cores take the group, and run for nothing else
    (256, 8, 1, 32, 8, 66_846_720, True),
    (8, 16, 1, 16, 4, 1_835_008, False),     # 32 rows: warps
    (8, 32, 1, 16, 4, 3_670_016, True),
    (16, 8, 1, 32, 8, 3_932_160, True),      # 64 rows behind a short table: warps
    (2, 60, 17, 32, 8, 1_966_080, False),    # the tensor cores run for the sequences' own positions anyway
    (8, 16, 17, 32, 8, 3_670_016, True)])
def test_what_is_worth_joining(n, pages, T, Hq, Hk, saved, joined):
    assert saved == (n - 1) * pages * 16 * Hk * 128 * 2
    x = _batch([(n, pages)], 0, [5, 70, 33], T, Hq, Hk, 128, 16)
    ws = bdla.Workspace(1 << 28, "cuda")
    for least, once in ((-1, joined), (0, True), (1 << 60, False)):
        bdla.set_share_least(least)
        try:
            want = _call(x, ws)
            assert ws.read_device_status() == bdla.OK
            got = _call({**x, "table": torch.cat((x["table"][:1], x["table"][1:].index_fill(1, torch.arange(pages, device="cuda"), -1)))}, ws)
        finally:
            bdla.set_share_least(-1)
        assert ws.read_device_status() == (bdla.OK if once else bdla.ERR_DEVICE)
        assert all(torch.equal(a, b) for a, b in zip(got, want)) == once
