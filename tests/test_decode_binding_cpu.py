"""What the decode binding checks of its operands' layouts, on host tensors (no GPU
needed: the device check is taken out)."""
import pytest
import torch

from gemm_decode_q1_amd import decode as D


@pytest.fixture(autouse=True)
def _host(monkeypatch):
    monkeypatch.setattr(D, "_same_device", lambda first, **others: None)


def attn_layout(k_prefix, v_prefix):
    q = torch.zeros(2, 4, 64, dtype=torch.bfloat16)
    return D._check_attn(q, k_prefix, v_prefix, None, None, None, None, None, None, None)


@pytest.mark.parametrize("P", [1, 2])
@pytest.mark.parametrize("which", ["k_prefix", "v_prefix"])
@pytest.mark.parametrize("how", ["transposed", "heads expanded", "all expanded", "every second element"])
def test_prefix_must_be_dense_in_a_row(P, which, how):
    """Whatever the number of prefix tokens, keys and values of a token are dense: the kernel reads them so."""
    dense = torch.zeros(P, 2, 64, dtype=torch.bfloat16)
    odd = {"transposed": torch.zeros(P, 64, 2, dtype=torch.bfloat16).transpose(1, 2),
           "heads expanded": torch.zeros(P, 1, 64, dtype=torch.bfloat16).expand(P, 2, 64),
           "all expanded": torch.zeros(1, 1, 1, dtype=torch.bfloat16).expand(P, 2, 64),
           "every second element": torch.zeros(P, 2, 128, dtype=torch.bfloat16)[..., ::2]}[how]
    assert attn_layout(dense, dense)
    with pytest.raises(ValueError, match=which):
        attn_layout(*((odd, dense) if which == "k_prefix" else (dense, odd)))


def test_one_prefix_token_may_have_any_row_stride():
    """A single row's stride is never used: keys and values may come from differently spaced rows."""
    k, v = (torch.zeros(3, n, 64, dtype=torch.bfloat16)[:1, :2] for n in (2, 5))
    assert attn_layout(k, v)
    with pytest.raises(ValueError, match="row stride"):
        attn_layout(*(torch.zeros(3, n, 64, dtype=torch.bfloat16)[:2, :2] for n in (2, 5)))
