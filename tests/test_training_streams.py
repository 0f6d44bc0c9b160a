"""Where the binding allocates and what it passes on, on a machine without a
GPU: tensors with made-up addresses, a library that only
notes its calls, and streams that are plain names."""
import contextlib
import ctypes

import pytest
import torch

import selective_state_space_ssm_amd as ssm

HERE, THERE = 0x51, 0x52       # handles of the current stream and of the call's


class Fake(torch.Tensor):
    """A tensor on cuda:0 without memory."""
    @staticmethod
    def __new__(cls, shape, dtype=torch.float32, at=0x10000000, made_on=None):
        t = torch.Tensor._make_wrapper_subclass(cls, shape, dtype=dtype, device="cuda:0")
        t.at, t.made_on, t.recorded = at, made_on, []
        return t

    def data_ptr(self):
        return self.at

    def untyped_storage(self):
        return "memory at %#x" % self.at

    def record_stream(self, stream):
        self.recorded.append(stream)

    @classmethod
    def __torch_dispatch__(cls, func, types, args=(), kwargs=None):
        raise NotImplementedError(func)


class Stream:
    """Stands for torch.cuda.Stream and ExternalStream."""
    device = torch.device("cuda:0")

    def __init__(self, handle, device=None):
        self.cuda_stream = handle

    def __eq__(self, other):
        return self.cuda_stream == other.cuda_stream


class Library:
    """Notes the entry points called; the size queries answer 64 bytes."""
    def __init__(self):
        self.calls, self.sizes = [], 0

    def __getattr__(self, name):
        def call(*args):
            if name.endswith("_size"):
                out = args[-1]
                (out._obj if hasattr(out, "_obj") else out).value = 64
                self.sizes += 1
            else:
                self.calls.append((name, args))
            return 0
        return call


@pytest.fixture
def world(monkeypatch):
    """.made: what was allocated; .lib: what was called."""
    class World:
        made, now, lib = [], HERE, Library()

    w = World()
    w.made = []

    @contextlib.contextmanager
    def on_stream(stream):
        w.now, before = stream.cuda_stream, w.now
        yield
        w.now = before

    def empty(*shape, dtype=torch.float32, device=None):
        shape = shape[0] if len(shape) == 1 and not isinstance(shape[0], int) else shape
        t = Fake(tuple(shape), dtype, 0x20000000 + 0x100000 * len(w.made), w.now)
        w.made.append(t)
        return t

    monkeypatch.setattr(ssm, "lib", lambda: w.lib)
    monkeypatch.setattr(ssm, "_current_device", lambda: 0)
    monkeypatch.setattr(ssm, "_current_stream", lambda i: w.now)
    monkeypatch.setattr(torch.cuda, "Stream", Stream)
    monkeypatch.setattr(torch.cuda, "ExternalStream", Stream)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda d=None: Stream(w.now))
    monkeypatch.setattr(torch.cuda, "stream", on_stream)
    monkeypatch.setattr(torch, "empty", empty)
    monkeypatch.setattr(torch, "empty_like", lambda t: empty(t.shape, dtype=t.dtype))
    return w


def _calls():
    x, v, t = Fake((8, 16)), Fake((8,)), Fake((8,), torch.int32)
    grads = ssm.GradList([Fake((40,)), Fake((3, 4), torch.bfloat16)])
    return {
        "ssm_layer_norm_fwd": lambda s: [ssm.ssm_layer_norm_fwd(x, stream=s)],
        "ssm_layer_norm_bwd": lambda s: list(ssm.ssm_layer_norm_bwd(x, x, v, v, stream=s).values()),
        "ssm_token_logp_fwd": lambda s: [ssm.ssm_token_logp_fwd(x, t, stream=s)],
        "ssm_token_logp_bwd": lambda s: [ssm.ssm_token_logp_bwd(x, t, Fake((8, 2)), v, stream=s)],
        "ssm_policy_loss": lambda s: [ssm.ssm_policy_loss(x, t, v, v, stream=s)],
        "ssm_clip_grad_norm": lambda s: [ssm.ssm_clip_grad_norm(grads, 1.0, stream=s)],
    }


CALLS = ["ssm_layer_norm_fwd", "ssm_layer_norm_bwd", "ssm_token_logp_fwd", "ssm_token_logp_bwd", "ssm_policy_loss",
         "ssm_clip_grad_norm"]


@pytest.mark.parametrize("how", ["stream", "handle"])
@pytest.mark.parametrize("name", CALLS)
def test_a_call_allocates_on_the_stream_it_runs_on(name, how, world):
    """Memory freed on the current stream may still be written by work queued
    there, so nothing that the call's own stream uses may come from it."""
    out = _calls()[name](Stream(THERE) if how == "stream" else THERE)
    (called, args), = world.lib.calls
    assert called == name and args[-1] == THERE and world.now == HERE
    assert world.made and all(t.made_on == THERE for t in world.made)
    for t in world.made:       # what the caller receives is used on the current stream too
        assert t.recorded == ([Stream(HERE)] if any(t is o for o in out) else [])


@pytest.mark.parametrize("how", [None, "stream", "handle"])
@pytest.mark.parametrize("name", CALLS)
def test_on_the_current_stream_nothing_is_recorded(name, how, world):
    _calls()[name]({None: None, "stream": Stream(HERE), "handle": HERE}[how])
    (called, args), = world.lib.calls
    assert called == name and args[-1] == HERE
    assert world.made and all(t.made_on == HERE and not t.recorded for t in world.made)


@pytest.mark.parametrize("name", CALLS)
def test_a_stream_of_another_device_is_refused(name, world):
    other = Stream(THERE)
    other.device = torch.device("cuda:1")
    with pytest.raises(ValueError):
        _calls()[name](other)
    assert not world.lib.calls


def _scan_calls():
    x, bc = Fake((2, 8, 16)), Fake((2, 8, 4))
    vec, mat, w = Fake((16,)), Fake((16, 4)), Fake((16, 4))
    desc = ssm.ssm_model_desc(3, 11, 8, 1, 16, 4, 2, 4, 0)
    step = lambda *s: Fake((1, 3) + s)
    layers = ssm.ModelLayers([{f: Fake((4,)) for f in ssm.LAYER_FIELDS}])
    return {
        "conv1d_causal": lambda s: [ssm.conv1d_causal(x, w, stream=s)],
        "ssm_scan_fwd": lambda s: [ssm.ssm_scan_fwd(x, x, mat, bc, bc, stream=s)],
        "ssm_scan_fwd_static": lambda s: [ssm.ssm_scan_fwd_static(x, x, mat, bc, bc, stream=s)],
        "ssm_scan_bwd": lambda s: list(ssm.ssm_scan_bwd(x, x, mat, bc, bc, x, dt_bias=vec, Dskip=vec, z=x, conv_w=w,
                                                        stream=s).values()),
        "ssm_step": lambda s: [ssm.ssm_step(step(16, 4), step(16), step(16), Fake((1, 16, 4)), step(4), step(4),
                                            stream=s)],
        "ssm_model_decode_step": lambda s: [ssm.ssm_model_decode_step(
            desc, Fake((11, 8)), layers, Fake((3,), torch.int32), step(16, 4), step(3, 16), stream=s)],
    }


SCANS = ["conv1d_causal", "ssm_scan_fwd", "ssm_scan_fwd_static", "ssm_scan_bwd", "ssm_step", "ssm_model_decode_step"]


@pytest.mark.parametrize("how", ["stream", "handle"])
@pytest.mark.parametrize("name", SCANS)
def test_a_scan_call_allocates_on_the_stream_it_runs_on(name, how, world):
    out = _scan_calls()[name](Stream(THERE) if how == "stream" else THERE)
    (called, args), = world.lib.calls
    assert called == name and args[-1].value == THERE and world.now == HERE
    assert world.made and all(t.made_on == THERE for t in world.made)
    for t in world.made:
        assert t.recorded == ([Stream(HERE)] if any(t is o for o in out) else [])


@pytest.mark.parametrize("how", [None, "stream", "handle"])
@pytest.mark.parametrize("name", SCANS)
def test_a_scan_call_on_the_current_stream_records_nothing(name, how, world):
    _scan_calls()[name]({None: None, "stream": Stream(HERE), "handle": HERE}[how])
    (called, args), = world.lib.calls
    assert called == name and args[-1].value == HERE
    assert world.made and all(t.made_on == HERE and not t.recorded for t in world.made)


def _addresses(args):
    return [(args[0][i].grad, args[0][i].out) for i in range(args[1])]


@pytest.mark.parametrize("which", ["grad", "out", "in place"])
def test_a_gradient_list_follows_its_tensors(which, world):
    """A tensor whose memory was replaced since the list was built: the call
    takes its present address, not the old one, which may be another tensor's."""
    g = [Fake((40,), at=0x1000), Fake((8,), at=0x2000), Fake((8,), at=0x3000)]
    o = [Fake((40,), at=0x4000), None, Fake((8,), torch.bfloat16, at=0x5000)]
    h = ssm.GradList(g) if which == "in place" else ssm.GradList(g, out=o)
    ssm.ssm_clip_grad_norm(h, 1.0)
    sizes = world.lib.sizes
    ssm.ssm_clip_grad_norm(h, 1.0)
    assert world.lib.sizes == sizes                         # nothing moved: the list is not built again
    (o if which == "out" else g)[2].at = 0x9000
    ssm.ssm_clip_grad_norm(h, 1.0)
    first, second, third = [_addresses(a) for _, a in world.lib.calls]
    assert first == second
    want = {"in place": [(0x1000, 0x1000), (0x2000, 0x2000), (0x9000, 0x9000)],
            "grad": [(0x1000, 0x4000), (0x2000, None), (0x9000, 0x5000)],
            "out": [(0x1000, 0x4000), (0x2000, None), (0x3000, 0x9000)]}[which]
    assert third == want


def test_a_moved_gradient_is_checked_again(world):
    class Strided(Fake):
        def is_contiguous(self):
            return self.at == 0x1000

    g = Strided((40,), at=0x1000)
    h = ssm.GradList([g])
    g.at = 0x2000
    for call in (lambda: ssm.ssm_clip_grad_norm(h, 1.0), lambda: ssm.ssm_clip_grad_norm_workspace_size(h), h.refresh):
        with pytest.raises(ValueError):
            call()
    assert not world.lib.calls
