"""The gated scan's oracle against the formulas written out for one token, and its gradients against
differences and against torch's automatic differentiation in 64 bits (needs no GPU)."""
import numpy as np
import pytest
import torch

import gated_ref as ref


def inputs(seed, b=2, l=9, d=3):
    r = np.random.default_rng(seed)
    k = {"x": r.standard_normal((b, l, d)), "forget": r.standard_normal((b, l, d)),
         "rate": r.uniform(0.01, 2.0, d), "input_gate": r.standard_normal((b, l, d)),
         "z": r.standard_normal((b, l, d)), "initial": r.standard_normal((b, d))}
    return k, r.standard_normal((b, l, d)), r.standard_normal((b, d))


def plain(x, forget, rate, input_gate, z, initial, lengths):
    """The definition in torch, float64, differentiable."""
    s = torch.sigmoid(forget)
    if rate is None:
        a, w = s, torch.sigmoid(-forget)
    else:
        a = torch.exp(-rate * s)
        w = torch.sqrt(-torch.expm1(-2 * rate * s))
    v = 1.0 if input_gate is None else torch.sigmoid(input_gate)
    h = torch.zeros_like(x[:, 0]) if initial is None else initial
    ys = []
    for t in range(x.shape[1]):
        on = torch.ones(x.shape[0], 1, dtype=torch.bool) if lengths is None else \
            (t < torch.tensor(lengths))[:, None]
        h = torch.where(on, a[:, t] * h + (w * v * x)[:, t], h)
        y = h if z is None else h * torch.nn.functional.silu(z[:, t])
        ys.append(torch.where(on, y, 0.0))
    return torch.stack(ys, 1), h


@pytest.mark.parametrize("lengths", [None, [9, 4], [0, 9]])
@pytest.mark.parametrize("without", [(), ("rate",), ("input_gate", "z"), ("rate", "input_gate", "z", "initial")])
def test_against_automatic_differentiation(without, lengths):
    k, dy, dfinal = inputs(1)
    for name in without:
        k[name] = None
    got = ref.gated(**k, lengths=None if lengths is None else np.array(lengths), dy=dy, dfinal=dfinal)
    t = {n: None if v is None else torch.tensor(v, requires_grad=True) for n, v in k.items()}
    y, state = plain(t["x"], t["forget"], t["rate"], t["input_gate"], t["z"], t["initial"], lengths)
    torch.autograd.backward([y, state], [torch.tensor(dy), torch.tensor(dfinal)])
    assert np.allclose(got["y"].val, y.detach().numpy(), rtol=1e-12, atol=1e-13)
    assert np.allclose(got["state"].val, state.detach().numpy(), rtol=1e-12, atol=1e-13)
    for name, key in (("x", "dx"), ("forget", "dforget"), ("rate", "drate"), ("z", "dz"),
                      ("input_gate", "dinput_gate"), ("initial", "dstate")):
        if k[name] is not None:
            assert np.allclose(got[key].val, t[name].grad.numpy(), rtol=1e-10, atol=1e-12), key


@pytest.mark.parametrize("rated", [True, False])
def test_against_differences(rated):
    k, dy, dfinal = inputs(2, b=1, l=5, d=2)
    if not rated:
        k["rate"] = None
    got = ref.gated(**k, dy=dy, dfinal=dfinal)
    step = 1e-6

    def loss(changed):
        out = ref.gated(**changed)
        return (out["y"].val * dy).sum() + (out["state"].val * dfinal).sum()

    for name, key in (("x", "dx"), ("forget", "dforget"), ("rate", "drate"), ("z", "dz"),
                      ("input_gate", "dinput_gate"), ("initial", "dstate")):
        if k[name] is None:
            continue
        for i in np.ndindex(k[name].shape):
            up, low = k[name].copy(), k[name].copy()
            up[i] += step
            low[i] -= step
            slope = (loss({**k, name: up}) - loss({**k, name: low})) / (2 * step)
            # the difference's own error: step^2 and the 64-bit rounding over the step
            assert abs(slope - got[key].val[i]) < 1e-8 * (1 + abs(slope)) + 1e-9, (name, i)


def test_rates_of_zero_and_below_hold_the_state():
    k, dy, dfinal = inputs(3)
    k["rate"] = np.array([0.0, -1.0, 0.5])
    k["z"] = None
    got = ref.gated(**k, dy=dy, dfinal=dfinal)
    assert np.array_equal(got["state"].val[:, :2], k["initial"][:, :2])
    assert np.array_equal(got["drate"].val[:2], [0.0, 0.0]) and np.isfinite(got["dforget"].val).all()
    assert (got["dforget"].val[..., :2] == 0).all() and (got["dx"].val[..., :2] == 0).all()


def test_planted_mistakes_are_outside_the_bounds():
    # a token left out, a decay applied twice: far outside what float32 may add
    k, dy, dfinal = inputs(4, l=70)
    good = ref.gated(**k, dy=dy, dfinal=dfinal)
    wrong = {**k, "x": k["x"].copy()}
    wrong["x"][:, 33] = 0
    bad = ref.gated(**wrong, dy=dy, dfinal=dfinal)
    import sequence_ref
    assert sequence_ref.excess(bad["y"].val, good["y"], "f32") > 10
    assert sequence_ref.excess(good["y"].val * (1 + 1e-3), good["y"], "f32") > 10
    assert sequence_ref.excess(good["y"].val, good["y"], "f32") == 0
