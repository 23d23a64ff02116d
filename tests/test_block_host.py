"""block_fwd, block_bwd and FewLayer without a GPU: what they refuse, and before any device work."""
import pytest
import torch

import sparse_mixture_experts_fp32_b200 as sm

T, D, F, N = 4, 64, 128, 4


def weights(dtype=torch.bfloat16):
    return torch.zeros(N, D), torch.zeros(N, F, D).to(dtype), torch.zeros(N, D, F).to(dtype)


@pytest.fixture
def no_calls(monkeypatch):
    """Every C function of the library raises."""
    class Library:
        def __getattr__(self, name):
            raise AssertionError(f"{name} was called")
    monkeypatch.setattr(sm, "lib", lambda: Library())


def test_gradients_of_a_top2_forward_are_refused(no_calls):
    w_r, w_in, w_out = weights()
    x, dy = torch.zeros(T, D, dtype=torch.bfloat16), torch.zeros(T, D)
    two = torch.zeros(T, 2, dtype=torch.int32)
    fwd = dict(expert=two, gate=two.float(), slot=two, counts=torch.zeros(N, dtype=torch.int32), capacity=T,
               workspace=torch.zeros(1 << 16, dtype=torch.uint8), x=x, sum=x, rstd=torch.ones(T))
    for flags in (None, sm.SWITCH_FLAG_TRAINING):
        if flags is not None:
            fwd["flags"] = flags
        with pytest.raises(ValueError, match="one expert per token"):
            sm.layer_bwd(fwd, x, w_r, w_in, w_out, dy)
        with pytest.raises(ValueError, match="one expert per token"):
            sm.block_bwd(fwd, torch.ones(D), w_r, w_in, w_out, dy)
