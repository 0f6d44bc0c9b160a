"""GPU parity of the global gradient norm and of clipping against 64 bits.

Bounds: squares and sums are 64-bit, so the norm is off by its own rounding
to float32 (U) and the factor by one more; a clipped value by the factor's,
the product's and the output type's roundings."""
import math

import pytest
import torch

import selective_state_space_ssm_amd as ssm
from bounds import U, half, within

pytestmark = pytest.mark.gpu

F, B = torch.float32, torch.bfloat16


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(g, *s, dtype=F, scale=1.0):
    return (torch.randn(*s, generator=g, device="cuda") * scale).to(dtype)


def _ref(grads, max_norm):
    n = math.sqrt(sum((g.double() ** 2).sum().item() for g in grads))
    return n, min(1.0, max_norm / (n + 1e-6))


def _check(grads, outs, max_norm, got):
    n, c = _ref(grads, max_norm)
    # norm and factor are float32: a norm above its largest value (2 - 2^-23) 2^127
    # rounds to infinity, and below 2^-126 half a step is 2^-150
    n32 = n if n < 2.0 ** 128 * (1 - U / 2) else math.inf
    within(got, torch.tensor([n32, c], dtype=torch.float64, device="cuda"),
           torch.tensor([2 * U * n, 4 * U * c + 2.0 ** -150], dtype=torch.float64, device="cuda"), "norm")
    for g, o in zip(grads, outs):
        if o is not None:
            r = g.double() * c
            within(o, r, 8 * U * r.abs() + half(o.dtype) * r.abs() * (1 + 8 * U) + 2.0 ** -126, "clipped")


@pytest.mark.parametrize("sizes", [[1], [2, 3], [7, 8192, 1], [8191, 8193, 100], [3, 0, 65, 0, 40000],
                                   [131072 * 9 + 5], list(range(1, 96)), [17] * 97, [33] * 168, [65] * 169, [50 + 37 * k for k in range(400)],
                                   [0]])
def test_types_and_sizes(sizes):
    g = _gen(sum(sizes))
    for max_norm in (0.0, 0.3, 1e9, math.inf):
        grads = [_randn(g, n, dtype=(F, B)[k % 2], scale=0.1 + k % 3) for k, n in enumerate(sizes)]
        outs = [torch.empty(n, dtype=(F, F, B, B)[k % 4], device="cuda") for k, n in enumerate(sizes)]
        norm = ssm.ssm_clip_grad_norm(ssm.GradList(grads, out=outs), max_norm)
        _check(grads, outs, max_norm, norm)
        mine = [a.clone() for a in grads]
        again = ssm.ssm_clip_grad_norm(ssm.GradList(mine), max_norm)
        assert torch.equal(again, norm)
        _check(grads, mine, max_norm, again)
        if max_norm >= 1e9:
            for a, b in zip(mine, grads):
                assert torch.equal(a, b)


def test_shapes_slices_and_uncounted_outputs():
    """Gradients of any shape; slices of a flat buffer at any element; an
    output of None leaves its gradient counted and unwritten; the values
    around a slice stay."""
    g = _gen(4)
    flat = _randn(g, 40001, dtype=B)
    into = torch.full((40001,), 5.0, device="cuda")
    cuts = [(1, 1000), (1003, 8192), (9200, 20001), (29202, 7)]
    grads = [flat[a:a + n] for a, n in cuts] + [_randn(g, 3, 5, 7), _randn(g, 4, 4), torch.tensor(2.0, device="cuda")]
    outs = [into[a:a + n] for a, n in cuts] + [torch.empty(3, 5, 7, device="cuda"), None, torch.empty((), device="cuda")]
    keep = grads[5].clone()
    norm = ssm.ssm_clip_grad_norm(ssm.GradList(grads, out=outs), 1.0)
    _check(grads, outs, 1.0, norm)
    assert torch.equal(grads[5], keep)
    left = torch.ones(40001, dtype=torch.bool, device="cuda")
    for a, n in cuts:
        left[a:a + n] = False
    assert (into[left] == 5.0).all()
    mine = flat.clone()
    ssm.ssm_clip_grad_norm(ssm.GradList([mine[a:a + n] for a, n in cuts]), 1e-3)
    assert torch.equal(mine[left], flat[left]) and not torch.equal(mine, flat)


def test_range():
    """Squares far outside float32: 1e30 and 1e-30."""
    for v in (1e30, 1e-30, 3e38):
        g = torch.full((10000,), v, device="cuda")
        out = torch.empty_like(g)
        norm = ssm.ssm_clip_grad_norm(ssm.GradList([g], out=[out]), 2.0)
        _check([g], [out], 2.0, norm)


def test_not_finite():
    g = _gen(5)
    a, b = _randn(g, 9000), _randn(g, 77)
    a[8500] = float("nan")
    outs = [torch.empty_like(a), torch.empty_like(b)]
    norm = ssm.ssm_clip_grad_norm(ssm.GradList([a, b], out=outs), 1.0)
    assert torch.isnan(norm).all() and torch.isnan(outs[0]).all() and torch.isnan(outs[1]).all()
    a[8500] = float("-inf")
    norm = ssm.ssm_clip_grad_norm(ssm.GradList([a, b], out=outs), 1.0)
    assert norm[0] == math.inf and norm[1] == 0.0
    assert torch.isnan(outs[0][8500]) and not outs[1].any()
    for v in (float("-inf"), float("nan")):     # an infinite max_norm only measures
        a[8500] = v
        mine = [a.clone(), b.clone()]
        norm = ssm.ssm_clip_grad_norm(ssm.GradList(mine), math.inf)
        assert torch.equal(norm, torch.tensor([abs(v), 1.0], device="cuda")) or (v != v and torch.isnan(norm[0])
                                                                                and norm[1] == 1.0)
        assert torch.equal(mine[0].view(torch.int32), a.view(torch.int32)) and torch.equal(mine[1], b)


def test_refusals():
    g = torch.ones(64, device="cuda")
    for bad, err in ((lambda: ssm.GradList([g.half()]), TypeError), (lambda: ssm.GradList([g[::2]]), ValueError),
                     (lambda: ssm.GradList([g], out=[g[:32]]), ValueError),
                     (lambda: ssm.GradList([g, torch.ones(3)]), ValueError),
                     (lambda: ssm.GradList([g], out=[g.to(torch.float64)]), TypeError),
                     (lambda: ssm.ssm_clip_grad_norm(ssm.GradList([g, g]), 1.0), ssm.SSMError),
                     (lambda: ssm.ssm_clip_grad_norm(ssm.GradList([g]), float("nan")), ssm.SSMError),
                     (lambda: ssm.ssm_clip_grad_norm(ssm.GradList([g]), 1.0, norm=g[:2].double()), TypeError),
                     (lambda: ssm.ssm_clip_grad_norm(ssm.GradList([g]), 1.0, norm=g[:2]), ssm.SSMError)):
        with pytest.raises(err):
            bad()
    assert torch.equal(g, torch.ones(64, device="cuda"))


def test_captured_call_replays_and_streams():
    g = _gen(6)
    grads = [_randn(g, n, dtype=(F, B)[k % 2]) for k, n in enumerate([5, 100000, 333, 8192, 70001] + [64] * 120)]
    outs = [torch.empty(a.shape, device="cuda") for a in grads]
    h = ssm.GradList(grads, out=outs)
    ssm.ssm_clip_grad_norm(h, 1.0)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        norm = ssm.ssm_clip_grad_norm(h, 1.0)
    for k in range(4):
        for a in grads:
            a.copy_(_randn(g, *a.shape))
        graph.replay()
        got, go = norm.clone(), [o.clone() for o in outs]
        torch.cuda.synchronize()
        eager = ssm.ssm_clip_grad_norm(h, 1.0)
        assert torch.equal(got, eager)
        for a, b in zip(go, outs):
            assert torch.equal(a, b)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    norm2 = ssm.ssm_clip_grad_norm(h, 1.0, stream=s)
    s.synchronize()
    assert torch.equal(norm2, eager)


def test_offsets_past_32_bits():
    n = (1 << 31) + 12345
    g = torch.ones(n, dtype=B, device="cuda")
    norm = ssm.ssm_clip_grad_norm(ssm.GradList([g]), 1.0)
    assert abs(norm[0].item() - math.sqrt(n)) <= 2 * U * math.sqrt(n)
    want = torch.tensor(norm[1].item()).to(B)
    assert (g[:5] == want.cuda()).all() and (g[-70000:] == want.cuda()).all() and (g[n // 2:n // 2 + 9] == want.cuda()).all()


def test_a_kept_list_follows_replaced_memory():
    """Gradients and outputs given new memory by `.data` and `set_` after the
    list was built; the old memory stays as it was."""
    g = _gen(7)
    for in_place in (True, False):
        grads = [_randn(g, n) for n in (100, 9000, 8)]
        outs = None if in_place else [torch.empty(n, dtype=(F, B, F)[k], device="cuda") for k, n in enumerate((100, 9000, 8))]
        h = ssm.GradList(grads, out=outs)
        ssm.ssm_clip_grad_norm(h, 1e9)
        old = grads[1].data
        kept = old.clone()
        grads[1].data = _randn(g, 9000)
        grads[2].set_(_randn(g, 8))
        if outs is not None:
            outs[0].data = torch.full((100,), 9.0, device="cuda")
        before = [t.clone() for t in grads]
        norm = ssm.ssm_clip_grad_norm(h, 0.5)
        _check(before, grads if in_place else outs, 0.5, norm)
        assert torch.equal(old, kept)
