"""What the differentiable forms ask of the operators beneath them (needs no GPU: those are
replaced by recorders)."""
import pytest
import torch

from stream_compaction_amd import autograd as ops


@pytest.mark.parametrize("trained", [True, False])
@pytest.mark.parametrize("mode", ["grad", "no_grad", "inference"])
def test_states_are_kept_for_a_gradient_alone(monkeypatch, trained, mode):
    # a prompt's pass under no_grad writes no states, though a model's parameters require gradients
    asked = []

    def scan(x, *args, keep_starts=False, **more):
        asked.append(keep_starts)
        out = (torch.empty_like(x), torch.empty(1, 4, 2))
        return out + (torch.empty(8),) if keep_starts else out

    monkeypatch.setattr(ops._ops, "selective_scan", scan)
    x = torch.zeros(1, 3, 4)
    A = torch.nn.Parameter(torch.zeros(4, 2), requires_grad=trained)
    rows = torch.zeros(1, 3, 1, 2)
    where = {"grad": torch.enable_grad, "no_grad": torch.no_grad, "inference": torch.inference_mode}
    with where[mode]():
        y, state = ops.selective_scan(x, x, A, rows, rows)
    kept = trained and mode == "grad"
    assert asked == [kept] and y.requires_grad == kept
