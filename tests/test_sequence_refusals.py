"""What the Python side of the sequence operators refuses, with the errors its documentation names:
ValueError for shapes, layouts and devices (needs no GPU: the tensors are stand-ins)."""
import pytest
import torch

from stream_compaction_amd import sequence as seq


class OnGpu(torch.Tensor):
    """A host tensor that says it lies on a GPU; nothing may be launched with it."""

    is_cuda = True
    index = 0

    @staticmethod
    def __new__(cls, *shape, index=0, dtype=torch.float32):
        t = torch.zeros(shape, dtype=dtype).as_subclass(cls)
        t.index = index
        return t

    def get_device(self):
        return self.index


def no_library(*args):
    raise AssertionError("a refused call reached the library")


@pytest.fixture(autouse=True)
def library(monkeypatch):
    class Refuses:
        def __getattr__(self, name):
            return (lambda *a: 64) if name.endswith("_bytes") else no_library
    monkeypatch.setattr(seq, "lib", Refuses)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda i: 0)


def scan_args(step, **wrong):
    lead = (2,) if step else (2, 8)
    k = {"x": OnGpu(*lead, 16), "dt": OnGpu(*lead, 16), "A": OnGpu(16, 4), "B": OnGpu(*lead, 1, 4),
         "C": OnGpu(*lead, 1, 4), "z": OnGpu(*lead, 16)}
    k.update(wrong)
    return k


@pytest.mark.parametrize("step", [False, True])
@pytest.mark.parametrize("name", ["x", "dt", "A", "B", "C", "z"])
@pytest.mark.parametrize("shape", [(), (2,), (2, 3), (2, 3, 5), (2, 3, 5, 7)])
def test_wrong_ranks(step, name, shape):
    # whatever the rank of an argument: the error is about its shape
    k = scan_args(step, **{name: OnGpu(*shape)})
    with pytest.raises(ValueError):
        if step:
            seq.selective_scan_step(OnGpu(2, 16, 4), **k)
        else:
            seq.selective_scan(**k)


@pytest.mark.parametrize("step", [False, True])
@pytest.mark.parametrize("name", ["x", "weight", "bias", "state"])
@pytest.mark.parametrize("shape", [(), (2,), (2, 3), (2, 3, 5), (2, 3, 5, 7)])
def test_wrong_ranks_of_a_convolution(step, name, shape):
    k = {"x": OnGpu(2, 16) if step else OnGpu(2, 8, 16), "weight": OnGpu(16, 4), "bias": OnGpu(16),
         "state": OnGpu(2, 3, 16)}
    k[name] = OnGpu(*shape)
    with pytest.raises(ValueError):
        if step:
            seq.causal_conv_step(k["state"], k["x"], k["weight"], k["bias"])
        else:
            seq.causal_conv(k["x"], k["weight"], k["bias"], k["state"])


def test_gradients_of_other_shapes():
    x, A, rows, w = OnGpu(2, 8, 16), OnGpu(16, 4), OnGpu(2, 8, 1, 4), OnGpu(16, 4)
    for dy in (OnGpu(), OnGpu(16), OnGpu(2, 8), OnGpu(2, 8, 16, 1)):
        with pytest.raises(ValueError):
            seq.selective_scan_grad(dy, x, x, A, rows, rows, OnGpu(16))
        with pytest.raises(ValueError):
            seq.causal_conv_grad(dy, x, w)


def test_rows_of_an_embedding():
    ids = OnGpu(4, 6, dtype=torch.int64)
    for dout in (OnGpu(), OnGpu(8), OnGpu(4, 8), OnGpu(4, 7, 8), OnGpu(4, 12, 8)[:, ::2].transpose(0, 1)):
        with pytest.raises(ValueError):
            seq.embedding_grad(dout, ids, 9)
    # rows of one token in two lie at one stride, every second channel and two batches do not
    with pytest.raises(ValueError):
        seq.embedding_grad(OnGpu(4, 6, 16)[..., ::2], ids, 9)
    with pytest.raises(ValueError):
        seq.embedding_grad(OnGpu(4, 9, 8)[:, :6], ids, 9)
    with pytest.raises(AssertionError, match="reached the library"):
        seq.embedding_grad(OnGpu(4, 12, 8)[:, ::2], ids, 9)
    for table in (OnGpu(), OnGpu(8), OnGpu(4, 8, 2), OnGpu(4, 16)[:, ::2]):
        with pytest.raises(ValueError):
            seq.embedding(table, ids)


def calls(stream=None):
    """One call of every operator on data of GPU 0."""
    x, one = OnGpu(2, 8, 16), OnGpu(2, 16)
    w, A = OnGpu(16, 4), OnGpu(16, 4)
    rows, row, ids = OnGpu(2, 8, 1, 4), OnGpu(2, 1, 4), OnGpu(2, 8, dtype=torch.int64)
    return (lambda: seq.causal_conv(x, w, out=OnGpu(2, 8, 16), final_state=OnGpu(2, 3, 16), stream=stream),
            lambda: seq.causal_conv_grad(x, x, w, stream=stream),
            lambda: seq.causal_conv_step(OnGpu(2, 3, 16), one, w, stream=stream),
            lambda: seq.selective_scan(x, x, A, rows, rows, stream=stream),
            lambda: seq.selective_scan_grad(x, x, x, A, rows, rows, OnGpu(16), stream=stream),
            lambda: seq.selective_scan_step(OnGpu(2, 16, 4), one, one, A, row, row, stream=stream),
            lambda: seq.embedding(w, ids, stream=stream),
            lambda: seq.embedding_grad(x, ids, 9, stream=stream))


@pytest.mark.parametrize("which", range(8))
def test_data_of_another_gpu_than_the_stream(monkeypatch, which):
    # the current stream of GPU 0 may take the work; of GPU 1, or a stream of GPU 1, not
    with pytest.raises(AssertionError, match="reached the library"):
        calls()[which]()
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 1)
    with pytest.raises(ValueError, match="cuda:1"):
        calls()[which]()
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0)

    class Other:
        cuda_stream, device_index = 64, 1

    def new(shape, dtype, like, stream):
        return OnGpu(*((shape,) if isinstance(shape, int) else shape), dtype=dtype)
    monkeypatch.setattr(seq, "_new", new)
    with pytest.raises(ValueError, match="cuda:1"):
        calls(Other())[which]()
