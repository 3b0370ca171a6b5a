"""Several devices, without one: tensors that say where they are, and a library that notes the
current device at each launch.  Launches go to the tensors' device whatever the current one is,
and tensors of two devices are refused."""
import types

import pytest
import torch

from linear_recurrence_scan_diagonal_amd import block


class On(torch.Tensor):
    """A tensor (host memory, never touched) that says it is on a device."""
    @staticmethod
    def make(index, shape, dtype=torch.float32):
        t = torch.Tensor._make_subclass(On, torch.zeros(shape).to(dtype))
        t.index = index
        return t

    is_cuda = property(lambda self: True)
    device = property(lambda self: torch.device("cuda", self.index))

    def get_device(self):
        return self.index

    __torch_function__ = torch._C._disabled_torch_function_impl


@pytest.fixture
def world(monkeypatch):
    """Current device 0; .at: the device of each launch."""
    w = types.SimpleNamespace(now=0, at=[])

    class Device:
        def __init__(self, device):
            self.index = device.index

        def __enter__(self):
            self.before, w.now = w.now, self.index

        def __exit__(self, *_):
            w.now = self.before

    class Lib:
        def __getattr__(self, name):
            def call(*_):
                if name.endswith("_bytes"):
                    return 256
                if name.endswith("_rows"):
                    return 1
                w.at.append(w.now)
                return 0
            return call

    def empty_on(*size, device=None, **kw):
        size = size[0] if len(size) == 1 and not isinstance(size[0], int) else size
        return On.make(torch.device(device).index, size, kw.get("dtype") or torch.float32)
    monkeypatch.setattr(block, "load", Lib)
    monkeypatch.setattr(block, "_several", True)
    monkeypatch.setattr(block, "_current", lambda: w.now)
    monkeypatch.setattr(block, "_stream", lambda dev: 0)
    monkeypatch.setattr(torch.cuda, "device", Device)
    monkeypatch.setattr(torch, "empty", empty_on)
    monkeypatch.setattr(torch, "empty_like", lambda t, dtype=None: On.make(t.index, t.shape, dtype or t.dtype))
    monkeypatch.setattr(On, "new_empty", lambda t, size: On.make(t.index, size, t.dtype))
    return w


def calls():
    """{name: (function, {argument: (shape, dtype)}, more arguments)}"""
    f, i = torch.float32, torch.int64
    gdr = dict(q=((64, 2, 1, 8), f), k=((64, 2, 1, 8), f), v=((64, 2, 2, 8), f), log_decay=((64, 2, 2), f),
               beta=((64, 2, 2), f), reset=((64, 2), torch.uint8), workspace=((256,), f))
    kept, state = ((1, 2, 2, 72, 8), f), ((2, 2, 8, 8), f)
    rows = dict(x=((4, 16), f), gamma=((16,), f), residual=((4, 16), f), out_sum=((4, 16), f))
    return {
        "gdr_fwd": dict(gdr, state0=state, checkpoints=kept, out=((64, 2, 2, 8), f)),
        "gdr_bwd": dict(gdr, checkpoints=kept, grad_o=((64, 2, 2, 8), f), grad_state=state),
        "gdr_step": dict(q=((2, 1, 8), f), k=((2, 1, 8), f), v=((2, 2, 8), f), log_decay=((2, 2), f), beta=((2, 2), f),
                         state=state, slots=((2,), torch.int32), out=((2, 2, 8), f)),
        "rmsnorm_fwd": dict(rows, out=((4, 16), f)),
        "rmsnorm_fwd_fp8": dict(rows, out=((4, 16), torch.float8_e4m3fn)),
        "rmsnorm_bwd": dict(s=((4, 16), f), gamma=((16,), f), rstd=((4,), f), grad_y=((4, 16), f), grad_sum=((4, 16), f),
                            out=((4, 16), f), workspace=((256,), f)),
        "logprobs_fwd": dict(logits=((4, 16), f), target=((4,), i)),
        "logprobs_bwd": dict(logits=((4, 16), f), target=((4,), i), lse=((4,), f), entropy=((4,), f), grad_logprob=((4,), f),
                             grad_entropy=((4,), f), out=((4, 16), f)),
    }


NAMES = sorted(calls())


def make(name, where):
    return {k: On.make(where.get(k, where[None]), *v) for k, v in calls()[name].items()}


@pytest.mark.parametrize("name", NAMES)
def test_launches_go_to_the_tensors_device(world, name):
    f = getattr(block, name)
    f(**make(name, {None: 1}))
    f(*list(make(name, {None: 0}).values())[:1], **dict(list(make(name, {None: 0}).items())[1:]))
    assert world.at == [1, 0] and world.now == 0


@pytest.mark.parametrize("name", NAMES)
def test_tensors_of_two_devices_are_refused(world, name):
    for other in calls()[name]:
        for here in (0, 1):
            with pytest.raises((ValueError, TypeError), match="cuda:|device"):
                getattr(block, name)(**make(name, {None: here, other: 1 - here}))
    assert not world.at and world.now == 0


def test_gradients_of_two_devices_are_refused(world):
    for i in range(3):
        a = make("gdr_bwd", {None: 1})
        grads = [On.make(0 if i == j else 1, a[n].shape) for j, n in enumerate("qkv")]
        with pytest.raises(ValueError, match="cuda:"):
            block.gdr_bwd(**a, grad_qkv=grads)
    assert not world.at
