"""Host side of the losses over a vocabulary: what the binding refuses before any device is looked at,
and that the bounds of the GPU tests can fail (CPU)."""

import pytest
import torch

from w8a8_gemm_rl_amd import binding as B


def test_hidden_states_and_head_are_matrices():
    """Contiguous tensors of other ranks, whose second size may well agree with the head's."""
    X, W = torch.zeros((4, 64), dtype=torch.bfloat16), torch.zeros((100, 64), dtype=torch.bfloat16)
    assert B._head_args(X, W) == (4, 100, 64, 64, 64)
    assert B._head_args(torch.zeros((4, 72), dtype=torch.bfloat16)[:, :64], W) == (4, 100, 64, 72, 64)
    for x, w in ((X.view(4, 64, 1), W), (X.new_zeros((4, 64, 64)), W), (X.new_zeros((2, 2, 64)), W), (X[0], W),
                 (X, W.new_zeros((100, 64, 64))), (X, W.view(-1)), (X.new_zeros(()), W)):
        with pytest.raises(ValueError):
            B._head_args(x, w)
