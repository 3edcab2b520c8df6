"""What the binding keeps between calls, on the CPU."""
from types import SimpleNamespace

import w4a8_ptq_linear_b200 as oq


def test_a_plan_remembers_a_bounded_number_of_workspace_sizes():
    asked = []
    plan = SimpleNamespace(workspace_bytes=lambda T: asked.append(T) or 3 * T + 256)
    for T in range(1, 5000):
        assert oq._layer_bytes(plan, T) == 3 * T + 256
        assert oq._layer_bytes(plan, T) == 3 * T + 256
    assert len(asked) == 4999                      # once for each of the last calls' sizes
    assert len(plan.__dict__["_layer_bytes"]) <= 64
