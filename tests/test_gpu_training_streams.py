"""The training operators on a stream of their own while the current stream
still has work queued, on the GPU: a call's outputs and workspace must not be
memory that such work writes."""
import pytest
import torch

import selective_state_space_ssm_amd as ssm

pytestmark = pytest.mark.gpu

T, V, D = 900, 2048, 384


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(g, *s):
    return torch.randn(*s, generator=g, device="cuda")


def _inputs():
    g = _gen(1)
    x, z = _randn(g, T, D), _randn(g, T, V)
    tgt = torch.randint(0, V, (T,), generator=g, device="cuda", dtype=torch.int32)
    mean, rstd = x.mean(-1), (x.var(-1, unbiased=False) + 1e-5).rsqrt()
    stats = torch.empty(T, 2, device="cuda")
    old = ssm.ssm_token_logp_fwd(z, tgt, stats=stats)
    adv = _randn(g, T)
    out = torch.empty(T, V, device="cuda")
    grads = ssm.GradList([x, z], out=[torch.empty_like(x), out])
    torch.cuda.synchronize()
    return {
        "norm_fwd": lambda s: [ssm.ssm_layer_norm_fwd(x, stream=s)],
        "norm_bwd": lambda s: list(ssm.ssm_layer_norm_bwd(x, x, mean, rstd, stream=s).values()),
        "logp_fwd": lambda s: [ssm.ssm_token_logp_fwd(z, tgt, stream=s)],
        "logp_bwd": lambda s: [ssm.ssm_token_logp_bwd(z, tgt, stats, adv, stream=s)],
        "policy": lambda s: [ssm.ssm_policy_loss(z, tgt, old, adv, stream=s)],
        "clip": lambda s: [ssm.ssm_clip_grad_norm(grads, 1.0, stream=s)],
    }


NAMES = ["norm_fwd", "norm_bwd", "logp_fwd", "logp_bwd", "policy", "clip"]


@pytest.mark.parametrize("how", ["stream", "handle"])
@pytest.mark.parametrize("name", NAMES)
def test_work_queued_on_the_current_stream_keeps_its_memory(name, how):
    """Temporaries of every size that the call may need are written late on the
    current stream and freed at once; the call's results do not change."""
    call = _inputs()[name]
    want = [o.clone() for o in call(None)]
    shapes = [o.shape for o in want]
    s = torch.cuda.Stream()
    a = torch.ones(4096, 4096, device="cuda")
    torch.cuda.synchronize()
    for k in range(3):
        for _ in range(4):
            a = a @ a                          # keeps the current stream busy for milliseconds
        late = [torch.full(sh, float("nan"), device="cuda") for sh in shapes]
        late += [torch.full((n // 4,), float("nan"), device="cuda") for n in (512, 1024, 4096, 1 << 16, 1 << 20, 1 << 22)]
        del late
        got = call(s if how == "stream" else s.cuda_stream)
        s.synchronize()
        torch.cuda.synchronize()
        for o, w in zip(got, want):
            assert torch.equal(o, w), (name, k)


@pytest.mark.parametrize("name", NAMES)
def test_a_stream_forked_in_a_capture(name):
    """A call on a second stream of a captured graph, replayed between eager
    calls."""
    call = _inputs()[name]
    want = [o.clone() for o in call(None)]
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s.wait_stream(torch.cuda.current_stream())
        out = call(s)
        torch.cuda.current_stream().wait_stream(s)
    for k in range(4):
        for o in out:
            o.fill_(7.0)
        graph.replay()
        got = [o.clone() for o in out]
        torch.cuda.synchronize()
        for o, w, e in zip(got, want, call(None)):
            assert torch.equal(o, w) and torch.equal(e, w), k


def test_default_stream_by_its_handle_from_another():
    call = _inputs()["policy"]
    want = call(None)[0].clone()
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        got = call(0)[0]
    torch.cuda.synchronize()
    assert torch.equal(got, want)


@pytest.mark.parametrize("name", ["fwd", "bwd"])
def test_scan_beside_work_queued_on_the_current_stream(name):
    """The same for the scan and its backward, a time split with its workspace."""
    g = _gen(2)
    B, L, D, N = 2, 512, 64, 16
    u, dt, dy = [_randn(g, B, L, D) for _ in range(3)]
    Bm, Cm, A = _randn(g, B, L, N), _randn(g, B, L, N), _randn(g, D, N) * 0.1
    calls = {"fwd": lambda s: [ssm.ssm_scan_fwd(u, dt, A, Bm, Cm, chunk_len=64, stream=s)],
             "bwd": lambda s: list(ssm.ssm_scan_bwd(u, dt, A, Bm, Cm, dy, chunk_len=64, stream=s).values())}
    want = [o.clone() for o in calls[name](None)]
    s = torch.cuda.Stream()
    a = torch.ones(4096, 4096, device="cuda")
    torch.cuda.synchronize()
    for k in range(3):
        for _ in range(4):
            a = a @ a
        late = [torch.full(o.shape, float("nan"), device="cuda") for o in want]
        late += [torch.full((n // 4,), float("nan"), device="cuda") for n in (512, 4096, 1 << 16, 1 << 20, 1 << 22, 1 << 24)]
        del late
        got = calls[name](s)
        torch.cuda.synchronize()
        for o, w in zip(got, want):
            assert torch.equal(o, w), k
