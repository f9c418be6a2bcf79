"""The Python calls refuse tensors of several GPUs, of a GPU that is not the current
one, and workspaces that are not on the call's GPU, before the library sees an address
(no GPU needed: stand-ins report the device)."""
import pytest
import torch

from chunk_wise_weight_gb300 import build, ittt


class On:
    """A tensor as the wrappers see it, on GPU `gpu` (never dereferenced)."""

    def __init__(self, gpu, *shape, dtype=torch.bfloat16):
        self.gpu, self.t = gpu, torch.empty(shape, dtype=dtype, device="meta")
        self.dtype, self.shape, self.is_cuda = dtype, self.t.shape, True
        self.device = torch.device("cuda", gpu)

    def get_device(self):
        return self.gpu

    def data_ptr(self):
        return 1 << 30

    def view(self, n):
        return self

    def __getattr__(self, name):
        return getattr(self.t, name)


class Library:
    def __getattr__(self, name):
        def reached(*args):
            raise AssertionError(f"{name} was reached")
        return reached


@pytest.fixture(autouse=True)
def one_current_gpu(monkeypatch):
    build.build()
    ittt.load()
    monkeypatch.setattr(ittt, "load", lambda: Library())
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda i: 0, raising=False)
    monkeypatch.setattr(ittt, "_like", lambda t, dtype=None: On(t.gpu, *t.shape, dtype=dtype or t.dtype))
    monkeypatch.setattr(torch, "empty_like", lambda t: On(t.gpu, *t.shape, dtype=t.dtype))
    empty = torch.empty
    monkeypatch.setattr(torch, "empty", lambda *s, dtype=None, device=None, **kw: On(device.index, *s, dtype=dtype)
                        if getattr(device, "type", None) == "cuda" else empty(*s, dtype=dtype, device=device, **kw))


def calls(gpus, workspace=None):
    """Each call with its tensors on the GPUs that `gpus` yields."""
    f = torch.float32
    at = lambda *s, **kw: On(next(gpus), *s, **kw)  # noqa: E731
    tok = lambda *b: (at(*b, 1, 64), at(*b, 1, 64), at(*b, 2, 32), at(*b, 2, dtype=f), at(*b, 2, dtype=f))  # noqa: E731
    vec = lambda: at(64, dtype=f)  # noqa: E731
    return {
        "embed": lambda: ittt.embed(at(8, dtype=torch.int32), at(100, 64), out=at(8, 64)),
        "embed_grad": lambda: ittt.embed_grad(at(8, dtype=torch.int64), at(8, 64), 100, grad=at(100, 64, dtype=f),
                                              workspace=workspace),
        "layer_norm": lambda: ittt.layer_norm(at(8, 64), vec(), vec(), out=at(8, 64), mean=at(8, dtype=f)),
        "layer_norm_grad": lambda: ittt.layer_norm_grad(at(8, 64), at(8, 64), vec(), at(8, dtype=f), at(8, dtype=f),
                                                        workspace=workspace),
        "delta_rule": lambda: ittt.delta_rule(*tok(1, 70), state_in=at(1, 2, 32, 64, dtype=f), workspace=workspace),
        "delta_rule_grad": lambda: ittt.delta_rule_grad(*tok(1, 70), at(1, 70, 2, 32), workspace=workspace,
                                                        grad_state_out=at(1, 2, 32, 64, dtype=f)),
        "delta_step": lambda: ittt.delta_step(*tok(3), at(5, 2, 32, 64, dtype=f), slots=at(3, dtype=torch.int32)),
    }


NAMES = list(calls(None))


def forever(*first, then=0):
    yield from first
    while True:
        yield then


@pytest.mark.parametrize("name", NAMES)
@pytest.mark.parametrize("where", [0, 1, 2])
def test_tensors_of_two_gpus(name, where):
    with pytest.raises(ValueError, match="GPU"):
        calls(forever(*[0] * where, 1))[name]()


@pytest.mark.parametrize("name", ["delta_rule", "delta_rule_grad"])
def test_states_of_another_gpu(name):
    n = 5 if name == "delta_rule" else 6
    with pytest.raises(ValueError, match="state.*GPU 1"):
        calls(forever(*[0] * n, 1))[name]()


@pytest.mark.parametrize("name", NAMES)
def test_tensors_of_a_gpu_that_is_not_current(name):
    with pytest.raises(ValueError, match="current"):
        calls(forever(then=1))[name]()


@pytest.mark.parametrize("name", ["embed_grad", "layer_norm_grad", "delta_rule", "delta_rule_grad"])
@pytest.mark.parametrize("workspace", [torch.zeros(1 << 20, dtype=torch.uint8), On(1, 1 << 20, dtype=torch.uint8)])
def test_workspaces_elsewhere(name, workspace):
    with pytest.raises(ValueError, match="workspace"):
        calls(forever(), workspace)[name]()


def test_workspace_with_gaps():
    gaps = On(0, 16, 16, dtype=torch.uint8)
    gaps.t = gaps.t.t()
    with pytest.raises(ValueError, match="workspace"):
        calls(forever(), gaps)["embed_grad"]()


@pytest.mark.parametrize("name", NAMES)
def test_stand_ins_reach_the_library(name):
    """Tensors of the current GPU pass every check up to the call itself."""
    with pytest.raises(AssertionError, match=f"ittt_{name} was reached"):
        calls(forever())[name]()
