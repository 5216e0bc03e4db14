"""AdamW states of trainable parameters, and the version counters that a step raises (no GPU)."""
import copy

import pytest
import torch

import grouped_gemm_histogram_amd as g


@pytest.mark.parametrize("bits", [8, 32])
def test_states_of_parameters_stay_out_of_autograd(bits):
    """The float32 copy of parameters that require gradients is a plain tensor: no graph onto them, and it can be copied."""
    params = [torch.nn.Parameter(torch.randn(3, 50).to(torch.bfloat16)), torch.nn.Parameter(torch.randn(129).to(torch.bfloat16))]
    state = g.adamw_init(params, bits=bits, master=True)
    tensors = [t for t in vars(state).values() if t is not None]
    assert len(tensors) == (5 if bits == 8 else 3)
    assert all(not t.requires_grad and t.grad_fn is None for t in tensors)
    again = copy.deepcopy(state)
    assert torch.equal(again.master, state.master)
    for p, at in zip(params, g.adamw_starts(params)):
        assert torch.equal(state.master[at:at + p.numel()], p.detach().reshape(-1).float())
        assert p.requires_grad and p.is_leaf
