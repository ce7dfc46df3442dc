"""The smallest and oddest arguments of the softmax layer's calls on a GPU."""
import pytest
import torch

from chunked_linear_attention_bounded_gb300 import bdla

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


@pytest.mark.parametrize("nbytes", [None, 256, 1 << 20])
def test_attn_cached_refuses_no_new_tokens(nbytes):
    q = torch.empty((2, 0, 8, 128), dtype=BF16, device="cuda")
    kc = torch.zeros((4, 16, 2, 128), dtype=BF16, device="cuda")
    table = torch.zeros((2, 2), dtype=torch.int32, device="cuda")
    lens = torch.zeros(2, dtype=torch.int32, device="cuda")
    ws = None if nbytes is None else bdla.Workspace(nbytes, "cuda")
    with pytest.raises(bdla.BdlaError) as e:
        bdla.attn_cached(q, kc, kc, table, lens, ws=ws)
    assert e.value.status == bdla.ERR_SHAPE
