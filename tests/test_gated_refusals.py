"""What the gated scan refuses, on the Python side and in the C ABI (needs no GPU)."""
import ctypes

import pytest
import torch

import stream_compaction_amd as sc
from stream_compaction_amd import autograd as ops
from stream_compaction_amd import sequence as seq
from stream_compaction_amd._sequence_abi import GatedArgs, GatedGrads
from test_sequence_refusals import OnGpu, library  # noqa: F401  (a fixture)

OK, EINVAL, ENOTSUP, EALIAS, ESCRATCH = range(5)
S = [0x10000000 * (i + 1) for i in range(24)]


def given(step, **wrong):
    lead = (2,) if step else (2, 8)
    k = {n: OnGpu(*lead, 16) for n in ("x", "forget", "input_gate", "z")}
    k["rate"] = OnGpu(16)
    k.update(wrong)
    return k


@pytest.mark.usefixtures("library")
class TestPython:
    @pytest.mark.parametrize("step", [False, True])
    @pytest.mark.parametrize("name", ["x", "forget", "input_gate", "z", "rate"])
    @pytest.mark.parametrize("shape", [(), (2,), (2, 3), (2, 3, 5), (2, 3, 5, 7)])
    def test_wrong_ranks(self, step, name, shape):
        k = given(step, **{name: OnGpu(*shape)})
        with pytest.raises(ValueError):
            if step:
                seq.gated_scan_step(OnGpu(2, 16), **k)
            else:
                seq.gated_scan(**k)

    @pytest.mark.parametrize("wrong", [
        {"initial_state": OnGpu(2, 15)}, {"initial_state": OnGpu(2, 16, dtype=torch.float16)},
        {"lengths": OnGpu(2)}, {"lengths": OnGpu(3, dtype=torch.int32)},
        {"forget": OnGpu(2, 8, 16, dtype=torch.bfloat16)}, {"forget": OnGpu(2, 8, 16, index=1)},
        {"z": OnGpu(2, 8, 32)[..., ::2]}, {"rate": OnGpu(16, dtype=torch.bfloat16)},
        {"out": OnGpu(2, 8, 15)}, {"final_state": OnGpu(2, 16, dtype=torch.bfloat16)},
        {"scratch": OnGpu(64)}, {"x": torch.zeros(2, 8, 16)}])
    def test_wrong_arguments(self, wrong):
        k = given(False)
        k.update(out=OnGpu(2, 8, 16), final_state=OnGpu(2, 16))
        k.update(wrong)
        with pytest.raises(ValueError):
            seq.gated_scan(**k)

    def test_types(self):
        for ty in (torch.float64, torch.int32):
            x = OnGpu(2, 8, 16, dtype=ty)
            with pytest.raises(NotImplementedError):
                seq.gated_scan(x, x)

    def test_gradients_of_other_shapes(self):
        k = given(False)
        for dy in (OnGpu(), OnGpu(16), OnGpu(2, 8), OnGpu(2, 8, 16, 1)):
            with pytest.raises(ValueError):
                seq.gated_scan_grad(dy, starts=OnGpu(16), **k)
        with pytest.raises(ValueError):
            seq.gated_scan_grad(k["x"], starts=OnGpu(17), **k)
        with pytest.raises(ValueError):
            seq.gated_scan_grad(k["x"], starts=OnGpu(16), dfinal=OnGpu(2, 15), **k)
        with pytest.raises(ValueError):
            seq.gated_scan_step(OnGpu(2, 15), **given(True))
        with pytest.raises(ValueError):
            seq.gated_scan_step(OnGpu(2, 16), new_state=OnGpu(3, 16), **given(True))

    @pytest.mark.parametrize("which", range(3))
    def test_data_of_another_gpu_than_the_stream(self, monkeypatch, which):
        def calls(stream=None):
            x, one = OnGpu(2, 8, 16), OnGpu(2, 16)
            return (lambda: seq.gated_scan(x, x, final_state=one, stream=stream),
                    lambda: seq.gated_scan_grad(x, x, x, OnGpu(16), stream=stream),
                    lambda: seq.gated_scan_step(one, one, one, stream=stream))

        def new(shape, dtype, like, stream):
            return OnGpu(*((shape,) if isinstance(shape, int) else shape), dtype=dtype)
        monkeypatch.setattr(seq, "_new", new)
        with pytest.raises(AssertionError, match="reached the library"):
            calls()[which]()
        monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 1)
        with pytest.raises(ValueError, match="cuda:1"):
            calls()[which]()
        monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0)

        class Other:
            cuda_stream, device_index = 64, 1
        with pytest.raises(ValueError, match="cuda:1"):
            calls(Other())[which]()


def args(**more):
    k = dict(x=S[0], forget=S[1], batch=2, length=200, channels=48,
             x_batch=200 * 48, x_token=48, forget_batch=200 * 48, forget_token=48, dtype=sc.DTYPE_CODES["f32"])
    k.update(more)
    return GatedArgs(**k)


def test_refused_sizes_and_types():
    L = sc.lib()
    for wrong in (dict(batch=-1), dict(batch=1 << 31), dict(length=-1), dict(length=1 << 31),
                  dict(channels=0), dict(channels=(1 << 22) + 1), dict(x=None), dict(forget=None),
                  dict(x=S[0] + 2), dict(rate=S[2] + 1), dict(x_batch=-1),
                  dict(batch=1 << 30, length=1 << 30, channels=16)):
        a = args(**wrong)
        assert L.gated_scan(a, S[10], S[11], None, S[12], 1 << 46, None) == EINVAL, wrong
        if "length" not in wrong:
            assert L.gated_scan_step(a, S[4], S[4], S[10], None) == EINVAL, wrong
    for code in ("f64", "i32"):
        a = args(dtype=sc.DTYPE_CODES[code])
        assert L.gated_scan(a, S[10], None, None, S[12], 1 << 46, None) == ENOTSUP
        assert L.gated_scan_step(a, S[4], S[4], S[10], None) == ENOTSUP
    assert L.gated_scan(None, S[10], None, None, S[12], 1 << 46, None) == EINVAL
    assert L.gated_scan_step(args(batch=1 << 16, channels=1 << 16), S[4], S[4], S[10], None) == EINVAL
    for size in ("starts", "scratch", "grad_scratch"):
        assert getattr(L, f"gated_scan_{size}_bytes")(args(batch=1 << 30, length=1 << 30)) == 0


def test_refused_overlap_and_scratch():
    L = sc.lib()
    a = args(batch=0)
    assert L.gated_scan(a, None, None, None, None, 0, None) == OK
    a = args(rate=S[2], z=S[3], z_batch=200 * 48, z_token=48)
    room = 1 << 46
    assert L.gated_scan(a, S[0], None, None, S[12], room, None) == EALIAS
    assert L.gated_scan(a, S[10], S[10] + 64, None, S[12], room, None) == EALIAS
    assert L.gated_scan(a, S[10], None, S[2], S[12], room, None) == EALIAS
    assert L.gated_scan(a, None, None, None, S[12], room, None) == EINVAL
    long_ = args(length=100000)
    need = L.gated_scan_scratch_bytes(long_)
    if need:
        assert L.gated_scan(long_, S[10], None, None, S[12], need - 1, None) == ESCRATCH
        assert L.gated_scan(long_, S[10], None, None, S[12] + 4, room, None) == EINVAL
        assert L.gated_scan(long_, S[10], None, None, S[10] + 16, room, None) == EALIAS
    g = dict(dy=S[4], dy_stride=(200 * 48, 48), starts=S[5], dx=S[6], dforget=S[7], dz=S[8],
             drate=S[9])
    for wrong in (dict(dz=None), dict(drate=None), dict(dinput_gate=S[11]), dict(dx=None),
                  dict(starts=None), dict(dy=None), dict(dy=S[4] + 2)):
        assert L.gated_scan_grad(a, GatedGrads(**{**g, **wrong}), S[12], room, None) == EINVAL, wrong
    for wrong in (dict(dx=S[0]), dict(dforget=S[6]), dict(drate=S[2]), dict(dinitial=S[5])):
        assert L.gated_scan_grad(a, GatedGrads(**{**g, **wrong}), S[12], room, None) == EALIAS, wrong
    need = L.gated_scan_grad_scratch_bytes(a)
    assert L.gated_scan_grad(a, GatedGrads(**g), S[12], need - 1, None) == ESCRATCH
    assert L.gated_scan_grad(a, None, S[12], room, None) == EINVAL
    # a step's state may be its own successor, not lie across it
    assert L.gated_scan_step(a, S[4], S[4] + 64, S[10], None) == EALIAS
    assert L.gated_scan_step(a, None, S[4], S[10], None) == EINVAL


@pytest.mark.parametrize("mode", ["grad", "no_grad", "inference"])
@pytest.mark.parametrize("trained", [True, False])
def test_states_are_kept_for_a_gradient_alone(monkeypatch, trained, mode):
    asked = []

    def scan(x, *a, keep_starts=False, **more):
        asked.append(keep_starts)
        out = (torch.empty_like(x), torch.empty(1, 4))
        return out + (torch.empty(8),) if keep_starts else out

    monkeypatch.setattr(ops._ops, "gated_scan", scan)
    x = torch.zeros(1, 3, 4)
    rate = torch.nn.Parameter(torch.zeros(4), requires_grad=trained)
    where = {"grad": torch.enable_grad, "no_grad": torch.no_grad, "inference": torch.inference_mode}
    with where[mode]():
        y, state = ops.gated_scan(x, x, rate)
    kept = trained and mode == "grad"
    assert asked == [kept] and y.requires_grad == kept


def test_struct_sizes():
    assert ctypes.sizeof(GatedArgs) == 152 and ctypes.sizeof(GatedGrads) == 88
