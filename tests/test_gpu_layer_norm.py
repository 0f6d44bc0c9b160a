"""GPU parity of the layer norm and its gradients against the formulas in 64
bits, on sizes around the vector, wavefront and workgroup edges.

Bounds: a value is a sum over the row (each lane's share in order, at most 32
terms, then at most 10 tree levels: under 48 roundings of the row's mean
magnitude) followed by a handful of products, so 64 half-steps of float32 on
the magnitudes the formula adds, plus the rounding to the io type."""
import math

import pytest
import torch

import selective_state_space_ssm_amd as ssm
from bounds import U, half, within

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}
WIDTHS = [1, 2, 3, 7, 8, 14, 31, 64, 100, 127, 128, 257, 384, 500, 513, 768, 1001, 1024, 2047, 2048, 2050, 4096, 5000,
          8192, 12001, 16384]


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(g, *s, dtype=torch.float32, scale=1.0, shift=0.0):
    return (torch.randn(*s, generator=g, device="cuda") * scale + shift).to(dtype)


def _fwd_ref(x, r, w, b, eps):
    s = x.double() + (r.double() if r is not None else 0.0)
    mu = s.mean(-1, keepdim=True)
    rs = 1.0 / torch.sqrt(((s - mu) ** 2).mean(-1, keepdim=True) + eps)
    y = (s - mu) * rs
    if w is not None:
        y = y * w.double()
    if b is not None:
        y = y + b.double()
    return s, mu, rs, y


def _check_fwd(x, r, w, b, eps, y, s, mean, rstd):
    sr, mu, rs, yr = _fwd_ref(x, r, w, b, eps)
    big = sr.abs().amax(-1, keepdim=True)
    wa = w.double().abs() if w is not None else 1.0
    ba = b.double().abs() if b is not None else 0.0
    xh = ((sr - mu) * rs).abs()
    # an error e of the mean moves the variance by e^2 only; that of a small
    # variance under a large mean comes through s - mu itself
    dev = 64 * U * big * rs
    within(y, yr, (dev * (1 + xh * (1 + dev)) + 64 * U * xh) * wa + 4 * U * ba + half(y.dtype) * yr.abs(), "y")
    if s is not None:
        within(s, sr, U * sr.abs() + half(s.dtype) * sr.abs() * (1 + U), "sum")
    if mean is not None:
        within(mean, mu[..., 0], 64 * U * big[..., 0], "mean")
        within(rstd, rs[..., 0], (64 * U + 2 * dev[..., 0] ** 2 + 2 * dev[..., 0]) * rs[..., 0], "rstd")


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("D", WIDTHS)
def test_forward(D, dt):
    g, t = _gen(D), DT[dt]
    for T, res, affine in ((1, False, True), (5, True, True), (131, True, False)):
        x, r = _randn(g, T, D, dtype=t, shift=0.5), _randn(g, T, D, dtype=t) if res else None
        w, b = (_randn(g, D), _randn(g, D)) if affine else (None, None)
        mean, rstd = torch.full((T,), 7.0, device="cuda"), torch.full((T,), 7.0, device="cuda")
        s = torch.empty_like(x) if res else None
        y = ssm.ssm_layer_norm_fwd(x, w, b, residual=r, residual_out=s, mean=mean, rstd=rstd, eps=1e-5)
        _check_fwd(x, r, w, b, 1e-5, y, s, mean, rstd)


def _bwd_ref(x, dy, mean, rstd, w, dr):
    mu, rs = mean.double()[..., None], rstd.double()[..., None]
    xh, d = (x.double() - mu) * rs, dy.double()
    g = d * w.double() if w is not None else d
    dx = rs * (g - g.mean(-1, keepdim=True) - xh * (g * xh).mean(-1, keepdim=True))
    mag = rs * (g.abs() + g.abs().mean(-1, keepdim=True) + xh.abs() * (g * xh).abs().mean(-1, keepdim=True))
    if dr is not None:
        dx, mag = dx + dr.double(), mag + dr.double().abs()
    # the rounding of x - mean, carried through
    loss = (x.double().abs() + mu.abs()) * rs * U * 2
    mag2 = rs * (loss * (g * xh).abs().mean(-1, keepdim=True) + xh.abs() * (g.abs() * loss).mean(-1, keepdim=True))
    dims = tuple(range(x.dim() - 1))
    return dx, 64 * U * mag + mag2, (d * xh).sum(dims), ((d * xh).abs() * 128 * U + d.abs() * loss).sum(dims), \
        d.sum(dims), d.abs().sum(dims) * 128 * U


def _stats(x, eps=1e-5):
    xd = x.double()
    return xd.mean(-1).float(), (xd.var(-1, unbiased=False) + eps).rsqrt().float()


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("D", WIDTHS)
def test_backward(D, dt):
    g, t = _gen(100 + D), DT[dt]
    for T, res, affine in ((1, False, True), (2, True, True), (3, False, True), (6, True, True), (1037, True, True),
                           (40, False, False)):
        x, dy = _randn(g, T, D, dtype=t, shift=0.5), _randn(g, T, D, dtype=t)
        dr = _randn(g, T, D, dtype=t) if res else None
        w = _randn(g, D) if affine else None
        mean, rstd = _stats(x)
        out = ssm.ssm_layer_norm_bwd(x, dy, mean, rstd, weight=w, dresidual=dr)
        dx, bx, dw, bw, db, bb = _bwd_ref(x, dy, mean, rstd, w, dr)
        within(out["dx"], dx, bx + half(t) * (dx.abs() + bx), "dx %d" % T)
        within(out["dweight"], dw, bw, "dweight %d" % T)
        within(out["dbias"], db, bb, "dbias %d" % T)


def test_gradient_against_differences():
    """Directional derivatives of the 64-bit forward against the kernel's
    float32 gradients: central differences with h = 1e-4 are off by
    O(h^2) = 1e-8 of the third derivative, far under 1e-5."""
    g = _gen(3)
    T, D = 9, 77
    x, w, b, dy = _randn(g, T, D), _randn(g, D), _randn(g, D), _randn(g, T, D)
    mean, rstd = _stats(x)
    out = ssm.ssm_layer_norm_bwd(x, dy, mean, rstd, weight=w)
    f = lambda x, w, b: (_fwd_ref(x, None, w, b, 1e-5)[3] * dy.double()).sum()
    p = [x.double(), w.double(), b.double()]
    for i, k in enumerate(("dx", "dweight", "dbias")):
        v = _randn(g, *p[i].shape).double()
        hi, lo = list(p), list(p)
        hi[i], lo[i] = p[i] + 1e-4 * v, p[i] - 1e-4 * v
        num = ((f(*hi) - f(*lo)) / 2e-4).item()
        got = (out[k].double() * v).sum().item()
        scale = (out[k].double() * v).abs().sum().item()
        assert abs(num - got) <= 1e-5 * scale, (k, num, got)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("D,pad", [(384, 384), (384, 1), (33, 7), (2048, 16)])
def test_strided_rows_leave_the_gaps(D, pad, dt):
    """Rows inside a wider buffer: values between rows stay as they were."""
    g, t = _gen(D + pad), DT[dt]
    T = 37
    wide = lambda: _randn(g, T, D + pad, dtype=t)
    X, R, S, Y, DY, DX = [wide() for _ in range(6)]
    before = [a.clone() for a in (S, Y, DX)]
    cut = lambda a: a[:, :D]
    w, b = _randn(g, D), _randn(g, D)
    mean, rstd = torch.empty(T, device="cuda"), torch.empty(T, device="cuda")
    ssm.ssm_layer_norm_fwd(cut(X), w, b, residual=cut(R), residual_out=cut(S), y=cut(Y), mean=mean, rstd=rstd)
    _check_fwd(cut(X), cut(R), w, b, 1e-5, cut(Y), cut(S), mean, rstd)
    out = ssm.ssm_layer_norm_bwd(cut(X), cut(DY), *_stats(cut(X)), weight=w, out={"dx": cut(DX)}, want=())
    dx, bx = _bwd_ref(cut(X), cut(DY), *_stats(cut(X)), w, None)[:2]
    within(out["dx"], dx, bx + half(t) * (dx.abs() + bx), "dx")
    for a, old in zip((S, Y, DX), before):
        assert torch.equal(a[:, D:], old[:, D:])


def test_leading_dimensions_and_refused_layouts():
    g = _gen(8)
    x = _randn(g, 3, 5, 64)
    y = ssm.ssm_layer_norm_fwd(x)
    assert y.shape == x.shape
    _check_fwd(x, None, None, None, 1e-5, y, None, None, None)
    row = _randn(g, 64)
    _check_fwd(row, None, None, None, 1e-5, ssm.ssm_layer_norm_fwd(row), None, None, None)
    for bad in (x.transpose(1, 2), x[:, :4], x[:1].expand(3, 5, 64), x[..., ::2]):
        with pytest.raises(ValueError):
            ssm.ssm_layer_norm_fwd(bad)
    with pytest.raises(TypeError):
        ssm.ssm_layer_norm_fwd(x.half())
    with pytest.raises(TypeError):
        ssm.ssm_layer_norm_fwd(x, residual=x.bfloat16())
    with pytest.raises(ValueError):
        ssm.ssm_layer_norm_fwd(x, torch.ones(63, device="cuda"))
    with pytest.raises(ValueError):
        ssm.ssm_layer_norm_fwd(x, torch.ones(64))
    with pytest.raises(ValueError):
        ssm.ssm_layer_norm_bwd(x, x, x[..., 0].contiguous(), x[..., 0].contiguous(), want=("dz",))
    with pytest.raises(ssm.SSMError):
        ssm.ssm_layer_norm_fwd(x, y=x)
    with pytest.raises(ssm.SSMError):
        ssm.ssm_layer_norm_fwd(x, eps=0.0)


def test_no_rows():
    x = torch.empty(0, 96, device="cuda")
    v = torch.empty(0, device="cuda")
    assert ssm.ssm_layer_norm_fwd(x).shape == (0, 96)
    out = ssm.ssm_layer_norm_bwd(x, x, v, v)
    assert torch.equal(out["dweight"], torch.zeros(96, device="cuda"))
    assert torch.equal(out["dbias"], torch.zeros(96, device="cuda"))


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_in_place_pairs(dt):
    g, t = _gen(5), DT[dt]
    for T, D in ((70, 384), (9, 5001)):
        x, r, dy, dr = [_randn(g, T, D, dtype=t) for _ in range(4)]
        w = _randn(g, D)
        s = torch.empty_like(x)
        y = ssm.ssm_layer_norm_fwd(x, w, residual=r, residual_out=s)
        for over in (0, 1):
            a = [x.clone(), r.clone()]
            y2 = ssm.ssm_layer_norm_fwd(a[0], w, residual=a[1], residual_out=a[over])
            assert torch.equal(y2, y) and torch.equal(a[over], s)
        mean, rstd = _stats(x)
        ref = ssm.ssm_layer_norm_bwd(x, dy, mean, rstd, weight=w, dresidual=dr)
        for over in (0, 1):
            a = [dy.clone(), dr.clone()]
            out = ssm.ssm_layer_norm_bwd(x, a[0], mean, rstd, weight=w, dresidual=a[1], out={"dx": a[over]})
            for k in ref:
                assert torch.equal(out[k], ref[k]), (over, k)


def test_rows_far_from_zero_and_special_rows():
    """A mean a thousand times the deviation; constant rows; rows with an
    infinity or a NaN, which stay their own."""
    g = _gen(6)
    x = _randn(g, 6, 384)
    x[0] += 1000.0
    x[1] = 3.0
    x[2, 17] = float("inf")
    x[3, 5] = float("nan")
    y = ssm.ssm_layer_norm_fwd(x)
    keep = torch.tensor([0, 1, 4, 5], device="cuda")
    _check_fwd(x[keep], None, None, None, 1e-5, y[keep], None, None, None)
    assert torch.isnan(y[2]).all() and torch.isnan(y[3]).all()
    assert torch.equal(y[1], torch.zeros(384, device="cuda"))


@pytest.mark.parametrize("at", [0, 1])
@pytest.mark.parametrize("D,gap", [(2051, 0), (2057, 0), (3001, 2), (4097, 0), (4097, 1), (4106, 1), (5001, 0), (5001, 1),
                                   (8191, 0), (8193, 0), (8201, 0)])
def test_bf16_rows_between_words(D, gap, at):
    """Rows that start on odd values, alone or all of them, in a buffer that
    ends with the last row; dx in a buffer of its own and over dy or dresidual;
    the values beside the rows stay."""
    g, T, st = _gen(D + gap + at), 600, D + gap
    buf = lambda: _randn(g, at + (T - 1) * st + D, dtype=torch.bfloat16, shift=0.25)
    cut = lambda b: b.as_strided((T, D), (st, 1), at)
    X, DY, DR, DX = buf(), buf(), buf(), buf()
    w = _randn(g, D)
    mean, rstd = _stats(cut(X))
    dx, bx, dw, bw, db, bb = _bwd_ref(cut(X), cut(DY), mean, rstd, w, cut(DR))
    first = None
    for into in (DX, DY.clone(), DR.clone()):
        dy = cut(into) if into is not DX and torch.equal(into, DY) else cut(DY)
        dr = cut(into) if into is not DX and torch.equal(into, DR) else cut(DR)
        before = into.clone()
        out = ssm.ssm_layer_norm_bwd(cut(X), dy, mean, rstd, weight=w, dresidual=dr, want=("dweight", "dbias"),
                                     out={"dx": cut(into)})
        within(out["dx"], dx, bx + half(torch.bfloat16) * (dx.abs() + bx), "dx")
        within(out["dweight"], dw, bw, "dweight")
        within(out["dbias"], db, bb, "dbias")
        if first is None:
            first = {k: v.clone() for k, v in out.items()}
        for k, v in out.items():
            assert torch.equal(v, first[k]), k
        cut(before).copy_(out["dx"])
        assert torch.equal(before, into)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("D", [3, 21, 32, 2050])
def test_constant_rows_near_the_largest_value(D, dt):
    """x = mean = 2^121 and rstd 316, whose product float32 does not hold: x - mean
    is exactly 0, so dx = rstd (dy - mean dy) by the sums' roundings alone."""
    g, t = _gen(D), DT[dt]
    T = 3
    x, dy = torch.full((T, D), 2.0 ** 121, dtype=t, device="cuda"), _randn(g, T, D, dtype=t)
    mean, rstd = torch.full((T,), 2.0 ** 121, device="cuda"), torch.full((T,), 1e-5 ** -0.5, device="cuda")
    out = ssm.ssm_layer_norm_bwd(x, dy, mean, rstd)
    d, rs = dy.double(), rstd.double()[:, None]
    dx, mag = rs * (d - d.mean(-1, keepdim=True)), rs * (d.abs() + d.abs().mean(-1, keepdim=True))
    within(out["dx"], dx, 64 * U * mag + half(t) * (dx.abs() + 64 * U * mag), "dx")
    within(out["dweight"], torch.zeros(D, dtype=torch.float64, device="cuda"), 0.0, "dweight")


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_same_bits_twice_and_wanted_gradients_only(dt):
    g, t = _gen(7), DT[dt]
    x, dy, w = _randn(g, 3001, 384, dtype=t), _randn(g, 3001, 384, dtype=t), _randn(g, 384)
    mean, rstd = _stats(x)
    a = ssm.ssm_layer_norm_bwd(x, dy, mean, rstd, weight=w)
    b = ssm.ssm_layer_norm_bwd(x, dy, mean, rstd, weight=w)
    for k in a:
        assert torch.equal(a[k], b[k])
    for k in a:
        one = ssm.ssm_layer_norm_bwd(x, dy, mean, rstd, weight=w, want=(k,))
        assert list(one) == [k] and torch.equal(one[k], a[k])


def test_captured_calls_replay():
    """Forward and backward in one graph, replayed on new inputs between eager
    calls, with the graph's own buffers."""
    g = _gen(9)
    T, D = 1000, 384
    x, r, dy = [_randn(g, T, D) for _ in range(3)]
    w, b = _randn(g, D), _randn(g, D)
    mean, rstd = torch.empty(T, device="cuda"), torch.empty(T, device="cuda")

    def step():
        s = torch.empty_like(x)
        y = ssm.ssm_layer_norm_fwd(x, w, b, residual=r, residual_out=s, mean=mean, rstd=rstd)
        return [y, s] + list(ssm.ssm_layer_norm_bwd(s, dy, mean, rstd, weight=w, dresidual=r).values())

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for k in range(4):
        for a in (x, r, dy):
            a.copy_(_randn(g, T, D))
        graph.replay()
        got = [o.clone() for o in out]
        torch.cuda.synchronize()
        for a, e in zip(got, step()):
            assert torch.equal(a, e), k


def test_another_stream():
    g = _gen(10)
    x = _randn(g, 4096, 384)
    want = ssm.ssm_layer_norm_fwd(x)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for how in (s, s.cuda_stream):
        y = ssm.ssm_layer_norm_fwd(x, stream=how)
        torch.cuda.current_stream().wait_stream(s)
        assert torch.equal(y, want)
    mean, rstd = _stats(x)
    ref = ssm.ssm_layer_norm_bwd(x, x, mean, rstd)
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        out = ssm.ssm_layer_norm_bwd(x, x, mean, rstd)
    s.synchronize()
    for k in ref:
        assert torch.equal(out[k], ref[k])


def test_offsets_past_32_bits():
    """2.3e9 values: the last rows lie past every 32-bit offset."""
    T, D = 140_001, 16384
    x = torch.zeros(T, D, dtype=torch.bfloat16, device="cuda")
    g = _gen(11)
    last = _randn(g, 3, D, dtype=torch.bfloat16)
    x[-3:] = last
    y = ssm.ssm_layer_norm_fwd(x)
    _check_fwd(last, None, None, None, 1e-5, y[-3:], None, None, None)
    assert not y[:-3].any()
    mean, rstd = torch.zeros(T, device="cuda"), torch.ones(T, device="cuda")
    dy = y.zero_()
    dy[-3:] = last.flip(0)
    out = ssm.ssm_layer_norm_bwd(x, dy, mean, rstd, out={"dx": dy})
    dx, bx, dw, bw, db, bb = _bwd_ref(last, last.flip(0), mean[:3], rstd[:3], None, None)
    within(out["dx"][-3:], dx, bx + half(x.dtype) * (dx.abs() + bx), "dx")
    within(out["dweight"], dw, bw, "dweight")
    within(out["dbias"], db, bb, "dbias")


def test_more_rows_than_a_launch_has():
    """A launch has fewer than 2^32 threads: 2^21 workgroups of 16 rows, then
    the rest."""
    T, D = (1 << 23) * 16 + 37, 2
    x = torch.zeros(T, D, device="cuda")
    x[:, 0] = 2.0
    x[-40:] = torch.tensor([1.0, 3.0], device="cuda")
    y = ssm.ssm_layer_norm_fwd(x)
    r = 1.0 / math.sqrt(1.0 + 1e-5)
    assert (y[:-40, 0] - r).abs().max() <= 8 * U and (y[:-40, 1] + r).abs().max() <= 8 * U
    assert (y[-40:, 0] + r).abs().max() <= 8 * U and (y[-40:, 1] - r).abs().max() <= 8 * U


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("D", [5, 384, 2048, 5001])
def test_slices_at_any_element(D, dt):
    """Tensors that start one element past a 16-byte boundary."""
    g, t = _gen(D + 3), DT[dt]
    T = 29

    def off(*s, dtype=torch.float32):
        n = math.prod(s)
        return _randn(g, n + 1, dtype=dtype)[1:].view(*s)

    x, r, dy = off(T, D, dtype=t), off(T, D, dtype=t), off(T, D, dtype=t)
    w, b, mean, rstd = off(D), off(D), off(T), off(T)
    s, y, dx = off(T, D, dtype=t), off(T, D, dtype=t), off(T, D, dtype=t)
    ssm.ssm_layer_norm_fwd(x, w, b, residual=r, residual_out=s, y=y, mean=mean, rstd=rstd)
    _check_fwd(x, r, w, b, 1e-5, y, s, mean, rstd)
    out = ssm.ssm_layer_norm_bwd(x, dy, *_stats(x), weight=w, dresidual=r, out=dict(dx=dx, dweight=off(D), dbias=off(D)))
    rx, bx, dw, bw, db, bb = _bwd_ref(x, dy, *_stats(x), w, r)
    within(out["dx"], rx, bx + half(t) * (rx.abs() + bx), "dx")
    within(out["dweight"], dw, bw, "dweight")
    within(out["dbias"], db, bb, "dbias")


def test_default_stream_by_its_handle():
    x = _randn(_gen(12), 8, 64)
    torch.cuda.synchronize()
    y = ssm.ssm_layer_norm_fwd(x, stream=0)
    torch.cuda.synchronize()
    assert torch.equal(y, ssm.ssm_layer_norm_fwd(x))


def test_with_another_device_current(monkeypatch):
    """The calls make their tensors' device current where it is not (told here
    that it is not), and leave the current one as it was."""
    x = _randn(_gen(13), 40, 384)
    want = ssm.ssm_layer_norm_fwd(x)
    monkeypatch.setattr(ssm, "_current_device", lambda: 63)
    assert torch.equal(ssm.ssm_layer_norm_fwd(x), want)
    out = ssm.ssm_layer_norm_bwd(x, x, *_stats(x))
    z = _randn(_gen(14), 40, 50)
    t = torch.zeros(40, dtype=torch.int32, device="cuda")
    lp = ssm.ssm_token_logp_fwd(z, t)
    loss = ssm.ssm_policy_loss(z, t, lp, lp)
    norm = ssm.ssm_clip_grad_norm(ssm.GradList([out["dx"].clone()]), 1.0)
    monkeypatch.undo()
    assert torch.cuda.current_device() == x.device.index
    assert torch.equal(ssm.ssm_layer_norm_bwd(x, x, *_stats(x))["dx"], out["dx"])
    assert torch.equal(ssm.ssm_policy_loss(z, t, lp, lp), loss)
    assert torch.equal(ssm.ssm_clip_grad_norm(ssm.GradList([out["dx"]]), math.inf)[:1], norm[:1])


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("D", [1, 7, 341, 384, 2050, 8192, 16384])
def test_rows_of_large_values(D, dt):
    """Values up to the documented 1e18 either way, whose squares' sum over a
    wide row float32 does not hold though their mean it does."""
    g, t = _gen(D + 21), DT[dt]
    sign = torch.where(torch.rand(4, D, generator=g, device="cuda") < 0.5, -1.0, 1.0)
    x = (sign * torch.tensor([[1e17], [3e17], [5e17], [0.98e18]], device="cuda")).to(t)
    r = torch.zeros_like(x)
    w, b = _randn(g, D), _randn(g, D)
    mean, rstd = torch.empty(4, device="cuda"), torch.empty(4, device="cuda")
    s = torch.empty_like(x)
    y = ssm.ssm_layer_norm_fwd(x, w, b, residual=r, residual_out=s, mean=mean, rstd=rstd, eps=1e-5)
    _check_fwd(x, r, w, b, 1e-5, y, s, mean, rstd)


@pytest.mark.parametrize("T,D,dt", [(1 << 27, 2, "f32"), (300_001, 4104, "bf16")])
def test_parameter_sums_over_many_rows(T, D, dt):
    """Equal terms, whose float32 sum is off to one side: at most 512 rows are
    added in float32, then at most 16 such sums, then 64 bits: 530 half-steps
    with the term's and the result's own, whatever the number of rows."""
    t = DT[dt]
    c = torch.tensor(1.1, dtype=t).item()
    x, dy = torch.ones(T, D, dtype=t, device="cuda"), torch.full((T, D), c, dtype=t, device="cuda")
    mean, rstd = torch.zeros(T, device="cuda"), torch.ones(T, device="cuda")
    out = ssm.ssm_layer_norm_bwd(x, dy, mean, rstd, want=("dweight", "dbias"))
    ref = torch.full((D,), T * c, dtype=torch.float64, device="cuda")
    within(out["dbias"], ref, 530 * U * ref, "dbias")
    within(out["dweight"], ref, 530 * U * ref, "dweight")
