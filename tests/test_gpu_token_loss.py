"""GPU parity of the token log-probabilities and the policy loss against the
formulas in 64 bits.

Bounds: exp of a float32 difference x is off by about (2 + 1.5 |x|) half-steps
(the product with log2 e and the hardware's 2^x); weighted with the
probabilities the sum is off by (2 + 1.5 E|x|) and a few tens of roundings of
its additions, under 64 + 2 max over the row's mean |x|; `spread` below is
that mean.  Gradients are products of such factors."""
import math

import pytest
import torch

import selective_state_space_ssm_amd as ssm
from bounds import U, half, within

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}
VOCABS = [1, 2, 5, 8, 63, 64, 65, 255, 256, 257, 511, 513, 1000, 1024, 1025, 2048, 2049, 4096, 8191, 8193, 16384,
          16385, 32769, 50001, 65537, 131073]
NEG = float("-inf")


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(g, *s, dtype=torch.float32, scale=1.0):
    return (torch.randn(*s, generator=g, device="cuda") * scale).to(dtype)


def _targets(g, T, V):
    return torch.randint(0, V, (T,), generator=g, device="cuda", dtype=torch.int32)


def _softmax_ref(z, t):
    """m, l, logp, p and the mean |z - m| under p, in 64 bits."""
    z = z.double()
    m = z.amax(-1, keepdim=True)
    e = torch.exp(z - m)
    s = e.sum(-1, keepdim=True)
    logp = (z.gather(-1, t.long()[:, None]) - m - torch.log(s))[:, 0]
    x = torch.where(e > 0, (z - m).abs() * e, 0.0).sum(-1, keepdim=True) / s
    return m[:, 0], torch.log(s)[:, 0], logp, e / s, x[:, 0]


def _onehot(t, V):
    return torch.nn.functional.one_hot(t.long().clamp(0, V - 1), V).double()


def _check_logp(z, t, logp, stats):
    m, l, ref, p, spread = _softmax_ref(z, t)
    e = (64 + 2 * spread) * U
    within(logp, ref, e + U * ref.abs() + U * l.abs(), "logp")
    if stats is not None:
        assert torch.equal(stats[:, 0].double(), m)
        within(stats[:, 1], l, e + 2 * U * l.abs(), "log sum")


def _check_logp_bwd(z, t, d, dz):
    m, l, logp, p, spread = _softmax_ref(z, t)
    h = _onehot(t, z.shape[1])
    ref = d.double()[:, None] * (h - p)
    x = torch.where(p > 0, (z.double() - m[:, None]).abs() + l.abs()[:, None], 0.0)
    # stats are given as float32: half a step of l more
    bound = U * d.double().abs()[:, None] * (p * (16 + 8 * x) + h * 16 * (1 - p + U)) + 2.0 ** -120
    within(dz, ref, bound + half(dz.dtype) * (ref.abs() + bound), "dlogits")


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("V", VOCABS)
def test_logp(V, dt):
    g, t = _gen(V), DT[dt]
    for T in (1, 7, 130 if V < 20000 else 17):
        z = _randn(g, T, V, dtype=t, scale=2.5)
        tgt = _targets(g, T, V)
        stats = torch.empty(T, 2, device="cuda")
        logp = ssm.ssm_token_logp_fwd(z, tgt, stats=stats)
        _check_logp(z, tgt, logp, stats)
        d = _randn(g, T)
        _check_logp_bwd(z, tgt, d, ssm.ssm_token_logp_bwd(z, tgt, stats, d))


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("V", [9, 300, 4096, 40000])
def test_logp_ruled_out_tokens(V, dt):
    """-infinity and the type's lowest value among the logits; rows of one
    value left, of the lowest value only, of -infinity only; a target that is
    ruled out; large offsets."""
    g, t = _gen(V + 1), DT[dt]
    low = torch.finfo(t).min
    z = _randn(g, 8, V, dtype=t)
    tgt = _targets(g, 8, V)
    drop = torch.rand(8, V, generator=g, device="cuda") < 0.5
    drop.scatter_(1, tgt.long()[:, None], False)
    z[0:2] = torch.where(drop[0:2], NEG, z[0:2])
    z[2] = torch.where(drop[2], low, z[2])
    z[3] = NEG
    z[3, tgt[3].long()] = 1.5                      # one value left
    z[4] = low
    z[5] += 1000.0
    z[6] -= 1000.0
    z[7, (tgt[7].long() + 1) % V] = 60.0           # nearly certain of another token
    stats = torch.empty(8, 2, device="cuda")
    logp = ssm.ssm_token_logp_fwd(z, tgt, stats=stats)
    _check_logp(z, tgt, logp, stats)
    d = _randn(g, 8)
    _check_logp_bwd(z, tgt, d, ssm.ssm_token_logp_bwd(z, tgt, stats, d))
    z = z[:3].clone()
    z[0] = NEG
    z[1, tgt[1].long()] = NEG
    z[2, 0] = float("nan")
    logp = ssm.ssm_token_logp_fwd(z, tgt[:3].contiguous())
    assert math.isnan(logp[0]) and logp[1] == NEG and math.isnan(logp[2])


def test_logp_certain_target_keeps_its_gradient():
    """With p = 1 - q, q far below float32's step next to 1, d(1 - p) is q d."""
    z = torch.zeros(1, 2, device="cuda")
    z[0, 0] = 20.0
    t = torch.zeros(1, dtype=torch.int32, device="cuda")
    stats = torch.empty(1, 2, device="cuda")
    ssm.ssm_token_logp_fwd(z, t, stats=stats)
    stats[0, 1] = math.log1p(math.exp(-20.0))       # what 64 bits give
    dz = ssm.ssm_token_logp_bwd(z, t, stats, torch.ones(1, device="cuda"))
    q = math.exp(-20.0) / (1 + math.exp(-20.0))
    assert abs(dz[0, 0].item() - q) <= 64 * U * q and abs(dz[0, 1].item() + q) <= 64 * U * q


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_logp_rows_without_target(dt):
    """Rows without a target are not read: NaN in them stays there."""
    t = DT[dt]
    for V in (100, 5000):
        g = _gen(V)
        z = _randn(g, 9, V, dtype=t)
        tgt = _targets(g, 9, V)
        tgt[3], tgt[8], tgt[5] = -1, -100, V
        z[3] = float("nan")
        z[8] = float("inf")
        z[0] = float("nan")
        d = _randn(g, 9)
        d[0] = 0.0
        keep = torch.tensor([1, 2, 4, 6, 7], device="cuda")
        stats = torch.full((9, 2), 5.0, device="cuda")
        logp = ssm.ssm_token_logp_fwd(z, tgt, stats=stats)
        _check_logp(z[keep], tgt[keep], logp[keep], stats[keep])
        assert logp[3] == 0 and logp[8] == 0 and not stats[3].any() and not stats[8].any()
        assert torch.isnan(logp[5]) and torch.isnan(logp[0])
        dz = ssm.ssm_token_logp_bwd(z, tgt, stats, d)
        _check_logp_bwd(z[keep], tgt[keep], d[keep], dz[keep])
        assert not dz[3].any() and not dz[8].any() and not dz[0].any()
        assert torch.isnan(dz[5]).all()


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("V,pad", [(4096, 64), (50, 3), (1000, 24), (33001, 7)])
def test_strided_and_in_place(V, pad, dt):
    g, t = _gen(V), DT[dt]
    T = 21
    Z, G = _randn(g, T, V + pad, dtype=t), _randn(g, T, V + pad, dtype=t)
    z, dz, gap = Z[:, :V], G[:, :V], G[:, V:].clone()
    tgt, d = _targets(g, T, V), _randn(g, T)
    stats = torch.empty(T, 2, device="cuda")
    logp = ssm.ssm_token_logp_fwd(z, tgt, stats=stats)
    _check_logp(z, tgt, logp, stats)
    ssm.ssm_token_logp_bwd(z, tgt, stats, d, dlogits=dz)
    _check_logp_bwd(z, tgt, d, dz)
    assert torch.equal(G[:, V:], gap)
    adv = _randn(g, T)
    pol = torch.empty_like(G)
    pol.copy_(G)
    loss = ssm.ssm_policy_loss(z, tgt, None, adv, dlogits=pol[:, :V])
    assert torch.equal(pol[:, V:], gap)
    want, wantp = dz.clone(), pol[:, :V].clone()
    a, b = Z.clone(), Z.clone()
    ssm.ssm_token_logp_bwd(a[:, :V], tgt, stats, d, dlogits=a[:, :V])
    loss2 = ssm.ssm_policy_loss(b[:, :V], tgt, None, adv, dlogits=b[:, :V])
    assert torch.equal(a[:, :V], want) and torch.equal(a[:, V:], Z[:, V:])
    assert torch.equal(b[:, :V], wantp) and torch.equal(b[:, V:], Z[:, V:]) and torch.equal(loss, loss2)


# ------------------------------------------------------------------ policy
def _policy_ref(z, tgt, old, adv, ref, w, lo, hi, beta, mean, scale):
    """Loss [4], logp, dlogits and a bound for each, by torch's own
    differentiation of the definition in 64 bits, token by token counted."""
    T, V = z.shape
    keep = tgt >= 0
    if w is not None:
        keep = keep & (w != 0)
    k = torch.nonzero(keep)[:, 0]
    wd = torch.ones(T, dtype=torch.float64, device="cuda") if w is None else w.double()
    zz = z[k].double().requires_grad_()
    t = tgt[k].long()
    logp = torch.log_softmax(zz, -1).gather(1, t[:, None])[:, 0]
    A = adv[k].double()
    r = torch.exp(logp - (logp.detach() if old is None else old[k].double()))
    free, held = r * A, torch.clamp(r, 1 - lo, 1 + hi) * A
    pol = -torch.minimum(free, held)
    gap = ref[k].double() - logp if ref is not None else torch.zeros_like(logp)
    kl = torch.expm1(gap) - gap
    norm = wd[k].sum() if mean else torch.ones((), dtype=torch.float64, device="cuda")
    inv = 0.0 if norm == 0 else 1.0 / norm
    wk = wd[k] * inv
    total = (wk * (pol + beta * kl)).sum()
    parts = torch.stack([total, (wk * pol).sum(), (wk * kl).sum(), (wk * (held < free)).sum()]).detach()
    dz = torch.zeros(T, V, dtype=torch.float64, device="cuda")
    bound = torch.zeros(T, V, dtype=torch.float64, device="cuda")
    lp, bl = (torch.zeros(T, dtype=torch.float64, device="cuda") for _ in range(2))
    lb = torch.zeros(4, dtype=torch.float64, device="cuda")
    if len(k):
        dz[k] = torch.autograd.grad(total, zz)[0] * scale
        m, l, _, p, spread = _softmax_ref(z[k], tgt[k])
        x = torch.where(p > 0, (z[k].double() - m[:, None]).abs() + l.abs()[:, None], 0.0)
        e = (64 + 2 * spread) * U                      # error of logp
        mag = ((r * A).abs() + beta * (torch.exp(gap) + 1)).detach() * wk.abs() * abs(scale)
        bound[k] = mag[:, None] * ((e[:, None] + 8 * U + 8 * U * x) * p + _onehot(tgt[k], V) * (e + 8 * U)[:, None]) + 2.0 ** -120
        lp[k] = logp.detach()
        bl[k] = e + U * (lp[k].abs() + l.abs())
        each = torch.stack([((r * A).abs() + beta * (torch.exp(gap) + 1)), (r * A).abs(), torch.exp(gap) + 1,
                            torch.zeros_like(gap)]).detach()
        lb = (each * (wk.abs() * e)).sum(1)
    return parts, lb + 4 * U * parts.abs() + 2.0 ** -120, lp, bl, dz, bound


def _check_policy(z, tgt, old, adv, ref=None, w=None, lo=0.2, hi=0.25, beta=0.0, mean=True, scale=1.0, **kw):
    T, V = z.shape
    logp = torch.full((T,), 9.0, device="cuda")
    dz = torch.full_like(z, 9.0)
    loss = ssm.ssm_policy_loss(z, tgt, old, adv, ref_logp=ref, weights=w, clip_low=lo, clip_high=hi, kl_beta=beta,
                               reduction=ssm.SSM_REDUCE_MEAN if mean else ssm.SSM_REDUCE_SUM, grad_scale=scale,
                               logp=logp, dlogits=dz, **kw)
    parts, pb, lp, lb, ref_dz, zb = _policy_ref(z, tgt, old, adv, ref, w, lo, hi, beta, mean, scale)
    within(loss, parts, pb, "loss")
    within(logp, lp, lb, "logp")
    within(dz, ref_dz, zb + half(z.dtype) * (ref_dz.abs() + zb), "dlogits")
    # the loss alone: the same bits
    assert torch.equal(ssm.ssm_policy_loss(z, tgt, old, adv, ref_logp=ref, weights=w, clip_low=lo, clip_high=hi,
                                           kl_beta=beta, reduction=0 if mean else 1), loss)
    return loss, dz


def _batch(g, T, V, t, scale=2.0):
    """Logits, targets, and old and reference log-probabilities near the
    present ones, with no ratio within 1e-4 of a bound of 0.8 or 1.25."""
    z = _randn(g, T, V, dtype=t, scale=scale)
    tgt = _targets(g, T, V)
    logp = _softmax_ref(z, tgt)[2]
    gap = _randn(g, T, scale=0.25).double()
    for b in (math.log(0.8), math.log(1.25)):
        gap = torch.where((gap - b).abs() < 1e-4, b + 2e-4, gap)
    return z, tgt, (logp - gap).float(), (logp + _randn(g, T, scale=0.3)).float(), _randn(g, T)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("V", VOCABS)
def test_policy(V, dt):
    g, t = _gen(1000 + V), DT[dt]
    for T in (1, 2, 3, 6, 150 if V < 20000 else 9):
        z, tgt, old, ref, adv = _batch(g, T, V, t)
        _check_policy(z, tgt, old, adv, ref=ref, beta=0.05)
    w = torch.rand(T, generator=g, device="cuda")
    w[::3] = 0.0
    _check_policy(z, tgt, old, adv, w=w, mean=False, scale=8.0)


def test_policy_past_the_persistent_grid():
    """More rows than workgroups hold at once, a third of them left out."""
    g = _gen(77)
    T, V = 9001, 130
    z, tgt, old, ref, adv = _batch(g, T, V, torch.float32)
    tgt[::3] = -1
    z[::3] = float("nan")
    _check_policy(z, tgt, old, adv, ref=ref, beta=0.1)


@pytest.mark.parametrize("V", [40, 3000, 70000])
def test_policy_options(V):
    g = _gen(V)
    T = 12
    z, tgt, old, ref, adv = _batch(g, T, V, torch.float32)
    _check_policy(z, tgt, None, adv)                                  # the present policy
    _check_policy(z, tgt, old, adv, ref=ref, beta=0.0)                # the KL term only reported
    _check_policy(z, tgt, old, adv, lo=1.0, hi=math.inf)              # no bounds
    _check_policy(z, tgt, old, torch.zeros_like(adv), ref=ref, beta=0.3)
    _check_policy(z, tgt, old, adv, scale=0.0)
    w = torch.rand(T, generator=g, device="cuda") + 0.1
    _check_policy(z, tgt, old, adv, ref=ref, w=w, beta=0.2, scale=-2.0)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("V", [60, 4096, 140000])
def test_policy_left_out_tokens(V, dt):
    """Nothing of a left-out token is read: NaN in its logits, scores and
    advantage does not reach the loss, and its gradient is exactly 0."""
    g, t = _gen(V + 5), DT[dt]
    T = 10
    z, tgt, old, ref, adv = _batch(g, T, V, t)
    w = torch.ones(T, device="cuda")
    w[1], tgt[4], w[9], tgt[9] = 0.0, -1, 0.0, V + 3
    for a in (z, old, ref, adv):
        a[1] = a[9] = float("nan")
        a[4] = float("inf")
    w[4] = float("nan")
    _, dz = _check_policy(z, tgt, old, adv, ref=ref, w=w, beta=0.1)
    for i in (1, 4, 9):
        assert not dz[i].any()
    # all of them
    w = torch.zeros(T, device="cuda")
    loss, dz = _check_policy(z, tgt, old, adv, ref=ref, w=w, beta=0.1)
    assert not loss.any() and not dz.any()
    # a target outside the vocabulary spoils the loss and its own row
    tgt[2] = V
    dz = torch.zeros_like(z)
    loss = ssm.ssm_policy_loss(z, tgt, old, adv, weights=torch.where(w == w, 1.0, w) * (torch.arange(T, device="cuda") == 2),
                               dlogits=dz)
    assert torch.isnan(loss[0]) and torch.isnan(dz[2]).all() and not dz[3].any()


@pytest.mark.parametrize("V", [30, 4000, 70001])
def test_policy_ruled_out_logits(V):
    g = _gen(V + 9)
    T = 6
    z, tgt, old, ref, adv = _batch(g, T, V, torch.float32)
    drop = torch.rand(T, V, generator=g, device="cuda") < 0.6
    drop.scatter_(1, tgt.long()[:, None], False)
    z = torch.where(drop, NEG, z)
    z[2] = torch.where(drop[2], torch.finfo(torch.float32).min, z[2])
    z[3] = torch.finfo(torch.float32).min          # nothing left: a uniform row
    old = (_softmax_ref(z, tgt)[2] - 0.1).float()
    _check_policy(z, tgt, old, adv, ref=old + 0.2, beta=0.1)


def test_ratio_exactly_on_a_bound():
    """A one-token vocabulary has logp = 0: with old = 0 the ratio is exactly
    1, and bounds of 0 hold it there without clipping it."""
    z = torch.full((2, 1), 3.0, device="cuda")
    t = torch.zeros(2, dtype=torch.int32, device="cuda")
    zero = torch.zeros(2, device="cuda")
    adv = torch.tensor([1.0, -2.0], device="cuda")
    loss = ssm.ssm_policy_loss(z, t, zero, adv, clip_low=0.0, clip_high=0.0)
    assert loss.tolist() == [0.5, 0.5, 0.0, 0.0]
    loss = ssm.ssm_policy_loss(z, t, zero - 1e-3, adv, clip_low=0.0, clip_high=0.0)
    assert loss[3] == 0.5                           # the positive advantage is clipped
    loss = ssm.ssm_policy_loss(z, t, zero + 1e-3, adv, clip_low=0.0, clip_high=0.0)
    assert loss[3] == 0.5                           # the negative one


def test_policy_gradient_against_differences():
    """Central differences of the 64-bit loss along a direction; h = 1e-4
    leaves O(h^2) = 1e-8 of the third derivative."""
    g = _gen(21)
    z, tgt, old, ref, adv = _batch(g, 11, 50, torch.float32)
    dz = torch.empty_like(z)
    ssm.ssm_policy_loss(z, tgt, old, adv, ref_logp=ref, clip_high=0.25, kl_beta=0.1, dlogits=dz)
    f = lambda q: _policy_ref(q, tgt, old, adv, ref, None, 0.2, 0.25, 0.1, True, 1.0)[0][0].item()
    v = _randn(g, 11, 50).double()
    num = (f(z.double() + 1e-4 * v) - f(z.double() - 1e-4 * v)) / 2e-4
    got, size = (dz.double() * v).sum().item(), (dz.double() * v).abs().sum().item()
    assert abs(num - got) <= 1e-5 * size


def test_no_tokens():
    z = torch.empty(0, 77, device="cuda")
    t, v = torch.empty(0, dtype=torch.int32, device="cuda"), torch.empty(0, device="cuda")
    assert ssm.ssm_token_logp_fwd(z, t).shape == (0,)
    assert ssm.ssm_token_logp_bwd(z, t, torch.empty(0, 2, device="cuda"), v).shape == (0, 77)
    for red in (0, 1):
        assert not ssm.ssm_policy_loss(z, t, v, v, reduction=red, dlogits=z).any()


def test_leading_dimensions_and_refusals():
    g = _gen(31)
    z, tgt, old, ref, adv = _batch(g, 12, 90, torch.float32)
    a = ssm.ssm_policy_loss(z, tgt, old, adv)
    b = ssm.ssm_policy_loss(z.view(3, 4, 90), tgt.view(3, 4), old.view(3, 4), adv.view(3, 4))
    assert torch.equal(a, b)
    lp = ssm.ssm_token_logp_fwd(z.view(3, 4, 90), tgt.view(3, 4))
    assert lp.shape == (3, 4) and torch.equal(lp.view(-1), ssm.ssm_token_logp_fwd(z, tgt))
    with pytest.raises(TypeError):
        ssm.ssm_policy_loss(z, tgt.long(), old, adv)
    with pytest.raises(TypeError):
        ssm.ssm_policy_loss(z.half(), tgt, old, adv)
    with pytest.raises(TypeError):
        ssm.ssm_policy_loss(z, tgt, old, adv, workspace=torch.empty(1 << 16, device="cuda"))
    for bad in (dict(old_logp=old[:5]), dict(advantages=adv.cpu()), dict(loss=torch.empty(3, device="cuda")),
                dict(dlogits=torch.empty(12, 91, device="cuda")), dict(weights=torch.ones(24, device="cuda")[::2])):
        args = dict(old_logp=old, advantages=adv)
        args.update(bad)
        with pytest.raises(ValueError):
            ssm.ssm_policy_loss(z, tgt, **args)
    with pytest.raises(ssm.SSMError):
        ssm.ssm_policy_loss(z, tgt, old, adv, clip_low=2.0)
    with pytest.raises(ssm.SSMError):
        ssm.ssm_policy_loss(z, tgt, old, adv, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))


def test_captured_calls_replay():
    """Scores, loss and gradient in one graph, replayed on new inputs between
    eager calls."""
    g = _gen(41)
    T, V = 300, 4096
    z, tgt, old, ref, adv = _batch(g, T, V, torch.bfloat16)
    w = torch.ones(T, device="cuda")
    dz = torch.empty_like(z)

    def step():
        stats = torch.empty(T, 2, device="cuda")
        logp = ssm.ssm_token_logp_fwd(z, tgt, stats=stats)
        d = ssm.ssm_token_logp_bwd(z, tgt, stats, adv)
        loss = ssm.ssm_policy_loss(z, tgt, old, adv, ref_logp=ref, weights=w, kl_beta=0.1, dlogits=dz)
        return [logp, stats, d, loss, dz]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for k in range(4):
        for a, b in zip((z, tgt, old, ref, adv), _batch(g, T, V, torch.bfloat16)):
            a.copy_(b)
        w.copy_((torch.rand(T, generator=g, device="cuda") < 0.7).float())
        graph.replay()
        got = [o.clone() for o in out]
        torch.cuda.synchronize()
        for a, e in zip(got, step()):
            assert torch.equal(a, e), k


def test_two_streams_at_once():
    """Two calls in flight with a workspace each."""
    g = _gen(51)
    batches = [_batch(g, 2000, 4096, torch.float32) for _ in range(2)]
    want = []
    for z, tgt, old, ref, adv in batches:
        dz = torch.empty_like(z)
        want.append((ssm.ssm_policy_loss(z, tgt, old, adv, dlogits=dz), dz))
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for k in range(3):
        for s, (z, tgt, old, ref, adv) in zip(streams, batches):
            dz = torch.empty_like(z)
            dz.record_stream(s)
            got.append((ssm.ssm_policy_loss(z, tgt, old, adv, dlogits=dz, stream=s), dz))
    torch.cuda.synchronize()
    for i, (loss, dz) in enumerate(got):
        assert torch.equal(loss, want[i % 2][0]) and torch.equal(dz, want[i % 2][1])


def test_offsets_past_32_bits():
    """2.2e9 logits: the last rows lie past every 32-bit offset."""
    T, V = 33_001, 65_537
    z = torch.zeros(T, V, dtype=torch.bfloat16, device="cuda")
    g = _gen(61)
    last, tl, old, ref, adv = _batch(g, 3, V, torch.bfloat16)
    z[-3:] = last
    tgt = torch.full((T,), -1, dtype=torch.int32, device="cuda")
    tgt[-3:] = tl
    full = lambda v: torch.cat([torch.zeros(T - 3, device="cuda"), v])
    stats = torch.empty(T, 2, device="cuda")
    logp = ssm.ssm_token_logp_fwd(z, tgt, stats=stats)
    _check_logp(last, tl, logp[-3:], stats[-3:])
    dz = torch.full_like(z, 1.0)
    ssm.ssm_token_logp_bwd(z, tgt, stats, full(adv), dlogits=dz)
    _check_logp_bwd(last, tl, adv, dz[-3:])
    assert not dz[:-3].any()
    dz.fill_(1.0)
    loss = ssm.ssm_policy_loss(z, tgt, full(old), full(adv), ref_logp=full(ref), clip_high=0.25, kl_beta=0.1, dlogits=dz)
    parts, pb, _, _, ref_dz, zb = _policy_ref(last, tl, old, adv, ref, None, 0.2, 0.25, 0.1, True, 1.0)
    within(loss, parts, pb, "loss")
    within(dz[-3:], ref_dz, zb + half(z.dtype) * (ref_dz.abs() + zb), "dlogits")
    assert not dz[:-3].any()


def test_more_rows_than_a_launch_has():
    """A launch has fewer than 2^32 threads: more than 2^23 rows of four
    logits go in slices."""
    T, V = (1 << 23) + 41, 4
    z = torch.zeros(T, V, device="cuda")
    z[-50:, 1] = 3.0
    tgt = torch.ones(T, dtype=torch.int32, device="cuda")
    stats = torch.empty(T, 2, device="cuda")
    logp = ssm.ssm_token_logp_fwd(z, tgt, stats=stats)
    flat, top = -math.log(4.0), 3.0 - math.log(3.0 + math.exp(3.0))
    assert (logp[:-50] - flat).abs().max() <= 64 * U and (logp[-50:] - top).abs().max() <= 64 * U
    dz = ssm.ssm_token_logp_bwd(z, tgt, stats, torch.ones(T, device="cuda"))
    assert (dz[:-50, 1] - 0.75).abs().max() <= 64 * U and (dz[-50:, 1] - (1 - math.exp(top))).abs().max() <= 64 * U
    dz.zero_()
    loss = ssm.ssm_policy_loss(z, tgt, None, torch.ones(T, device="cuda"), dlogits=dz, reduction=ssm.SSM_REDUCE_SUM)
    assert abs(loss[0].item() + T) <= 2 * U * T
    assert (dz[:-50, 1] + 0.75).abs().max() <= 64 * U and (dz[-50:, 1] + (1 - math.exp(top))).abs().max() <= 64 * U


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("V", [7, 130, 4096, 33001])
def test_slices_at_any_element(V, dt):
    """Tensors that start one element past a 16-byte boundary, and logits and
    gradients whose rows are aligned differently."""
    g, t = _gen(V + 11), DT[dt]
    T = 14
    z0, tgt, old, ref, adv = _batch(g, T, V, t)

    def off(v, k=1):
        return torch.cat([v.new_zeros(k), v.reshape(-1)])[k:].view(v.shape)

    for k in (1, 2, 3):
        z, dz = off(z0, k), off(torch.zeros(T, V, dtype=t, device="cuda"), 1)
        stats = off(torch.empty(T, 2, device="cuda"))
        logp = ssm.ssm_token_logp_fwd(z, off(tgt), stats=stats, logp=off(torch.empty(T, device="cuda")))
        _check_logp(z, tgt, logp, stats)
        ssm.ssm_token_logp_bwd(z, off(tgt), stats, off(adv), dlogits=dz)
        _check_logp_bwd(z, tgt, adv, dz)
        parts, pb, _, _, ref_dz, zb = _policy_ref(z, tgt, old, adv, ref, None, 0.2, 0.25, 0.1, True, 1.0)
        loss = ssm.ssm_policy_loss(z, off(tgt), off(old), off(adv), ref_logp=off(ref), clip_high=0.25, kl_beta=0.1,
                                   dlogits=dz, loss=off(torch.empty(4, device="cuda")))
        within(loss, parts, pb, "loss")
        within(dz, ref_dz, zb + half(t) * (ref_dz.abs() + zb), "dlogits")


@pytest.mark.parametrize("T", [511, 512, 513, 5000])
def test_weights_summed_by_either_launch(T):
    """Few tokens' weights are summed by the loss's own launch, many by one of
    their own."""
    g = _gen(T)
    z, tgt, old, ref, adv = _batch(g, T, 33, torch.float32)
    w = torch.rand(T, generator=g, device="cuda")
    w[::5] = 0.0
    tgt[1::7] = -1
    _check_policy(z, tgt, old, adv, ref=ref, w=w, beta=0.1)
    _check_policy(z, tgt, old, adv, ref=ref, beta=0.1)


def test_two_graphs_with_a_workspace_each():
    """Two captured steps with their own workspaces and outputs, replayed in
    turn and on two streams at once."""
    g = _gen(71)
    batches = [_batch(g, 700, 4096, torch.float32) for _ in range(2)]
    desc = ssm.ssm_policy_desc(700, 4096, 0, 0, 0.2, 0.2, 0.0, 1.0, 0, 0)
    ws = [torch.empty(ssm.ssm_policy_loss_workspace_size(desc), dtype=torch.uint8, device="cuda") for _ in range(2)]
    outs = [(torch.empty(4, device="cuda"), torch.empty(700, 4096, device="cuda")) for _ in range(2)]
    run = lambda i: ssm.ssm_policy_loss(batches[i][0], batches[i][1], batches[i][2], batches[i][4], workspace=ws[i],
                                        loss=outs[i][0], dlogits=outs[i][1])
    want = []
    for i in range(2):
        run(i)
        want.append([o.clone() for o in outs[i]])
    torch.cuda.synchronize()
    graphs = []
    for i in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            run(i)
        graphs.append(graph)
    streams = [torch.cuda.Stream() for _ in range(2)]
    for k in range(4):
        for o in outs:
            o[0].fill_(7.0), o[1].fill_(7.0)
        for i in range(2):
            if k % 2:
                streams[i].wait_stream(torch.cuda.current_stream())
                with torch.cuda.stream(streams[i]):
                    graphs[i].replay()
            else:
                graphs[i].replay()
        torch.cuda.synchronize()
        for i in range(2):
            for a, b in zip(outs[i], want[i]):
                assert torch.equal(a, b), (k, i)
        run(0)


@pytest.mark.parametrize("T,V,dt", [(16384, 4096, "f32"), (16384, 4100, "bf16"), (4096, 50001, "bf16"), (2048, 70001, "f32")])
def test_log_sums_are_off_to_either_side(T, V, dt):
    """The mean signed error of log p over many rows.  With the largest logit as
    the target log p is -log sum, between -8 and -1 here: its rounding to float32
    (half a step 2.4e-7 at most, deviation 1.4e-7) and the row's own roundings
    (deviation under 1e-7) average to 1.8e-7 / sqrt(2048) = 4e-9 over the fewest
    rows; the hardware's 2^x is off by -3.3e-9 on the average (its own rounding,
    measured over 2^24 arguments), which enters log sum as it is.  Four
    deviations and that bias: 2e-8."""
    g, t = _gen(T + V), DT[dt]
    z = _randn(g, T, V, dtype=t, scale=2.5)
    tgt = z.argmax(-1).int()
    ref = torch.cat([_softmax_ref(z[i:i + 512], tgt[i:i + 512])[2] for i in range(0, T, 512)])
    logp = torch.empty(T, device="cuda")
    ssm.ssm_policy_loss(z, tgt, None, logp.new_zeros(T), logp=logp)
    for got in (ssm.ssm_token_logp_fwd(z, tgt), logp):
        assert -8 < ref.min() and ref.max() < 0
        assert abs((got.double() - ref).mean().item()) < 2e-8
