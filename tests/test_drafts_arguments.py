"""CPU checks of what the binding says of arguments that are no tensors."""
import pytest

from log_linear_attention_gb300 import binding

torch = pytest.importorskip("torch")


def test_paths_and_states_that_are_no_tensors():
    binding._torch()
    count = torch.zeros(2, dtype=torch.int32)
    for path in ([[0], [1]], 3, "0"):
        with pytest.raises(TypeError, match="path must be a torch.Tensor"):
            binding._accepted(count, path, 2, -1, count.device)
    for state in ([[0.0] * 4] * 2, 1.0):
        with pytest.raises(TypeError, match="state0 must be a torch.Tensor"):
            binding._gated_state(state, "state0", 2, 4, count.device)
