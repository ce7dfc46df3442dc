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


@pytest.mark.parametrize("B", [1, 2])
def test_norm_of_rows_without_tokens(B):
    q, k = torch.empty((B, 0, 4, 64), dtype=BF16, device="cuda"), torch.empty((B, 0, 2, 64), dtype=BF16, device="cuda")
    w = torch.ones(64, device="cuda")
    qn, kn = bdla.qk_norm(q, k, w, w)
    assert qn.shape == q.shape and kn.shape == k.shape
    dq, dk, dwq, dwk = bdla.qk_norm_bwd(q, k, w, w, q, k)
    assert dq.shape == q.shape and dk.shape == k.shape
    assert float(dwq.abs().sum() + dwk.abs().sum()) == 0.0


def test_norm_of_one_token_whatever_its_token_stride_says():
    """A step of one sequence: the strides of its single row and token mean nothing."""
    flat = torch.randn(6 * 64, generator=torch.Generator("cuda").manual_seed(1), device="cuda").to(BF16)
    q, k = torch.as_strided(flat, (1, 1, 4, 64), (3, 5, 64, 1)), torch.as_strided(flat, (1, 1, 2, 64), (7, 1, 64, 1), 256)
    w = torch.linspace(0.5, 1.5, 64, device="cuda")
    got = bdla.qk_norm(q, k, w, w)
    want = bdla.qk_norm(q.clone(memory_format=torch.contiguous_format), k.clone(memory_format=torch.contiguous_format), w, w)
    assert all(torch.equal(x, y) for x, y in zip(got, want))
