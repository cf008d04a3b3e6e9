"""The gated block on bf16 weights and its gradients against fp64 (needs a B200).

Bars, from the arithmetic: a product of bf16 values is exact in fp32, a tensor
core adds eight or more of them at a time and cuts what does not fit 24 bits,
so a sum of K products is off by at most (K / 8 + 32) * 2^-23 * sum|x w|; a
rounding to bf16 by at most 2^-8 of the value (2^-134 near zero).
"""

import numpy as np
import pytest

import oracle
from oracle import dense

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import sub_bit_sparse_b200 as stq1

HALF, TINY = 2.0 ** -8, 2.0 ** -134


def _bf16(v):
    t = torch.from_numpy(np.ascontiguousarray(v, dtype=np.float32)).to(torch.bfloat16)
    return t.cuda(), t.double().numpy()


def _sum_err(k, mag):
    return (k / 8 + 32) * 2.0 ** -23 * mag


def _guarded(shape, fill=77.0):
    n, pad = int(np.prod(shape)), 64
    whole = torch.full((n + 2 * pad,), fill, dtype=torch.bfloat16, device="cuda")
    return whole[pad:pad + n].view(shape), lambda: bool((whole[:pad] == fill).all()) and bool(
        (whole[pad + n:] == fill).all())


def _within(got, ref, bar, what):
    err = np.abs(got - ref)
    bad = ~(err <= bar)
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} outside; worst {np.nanmax(err / bar):.3g}"


def _check_forward(x, xv, w, wv, act, y=None):
    k, half = xv.shape[1], wv.shape[0] // 2
    ref, s, mag = dense.glu(xv, wv)
    e = _sum_err(k, mag)
    g, u, eg, eu = s[:, :half], s[:, half:], e[:, :half], e[:, half:]
    # SiLU has a slope of at most 1.1
    through = 1.1 * eg * np.abs(u) + (np.abs(oracle.silu(g)) + 1.1 * eg) * eu
    _within(act.double().cpu().numpy(), ref, through + HALF * (np.abs(ref) + through) + TINY, "act")
    if y is not None:
        _within(y.double().cpu().numpy(), s, e + HALF * (np.abs(s) + e) + TINY, "y")


SHAPES = [
    (1, 16, 8), (1, 4096, 7168), (2, 48, 264), (3, 1040, 1032), (5, 512, 40), (8, 256, 512), (9, 144, 136),
    (15, 64, 2048), (16, 1024, 1536), (17, 272, 520), (31, 48, 72), (32, 128, 256), (33, 160, 264), (64, 512, 512),
    (65, 336, 88), (100, 2064, 1032), (128, 128, 64), (129, 272, 1024), (200, 1040, 1032), (256, 512, 256),
    (257, 528, 264), (300, 4096, 640), (513, 1040, 1032), (1000, 2048, 512), (1100, 528, 2056),
    (2600, 1072, 264), (2000, 2704, 72), (4000, 528, 136),
    (1600, 2064, 1544), (2100, 2112, 1160), (700, 4096, 3600),
    # few tokens: outputs for more than one round of CTAs, one or two CTAs per SM, rows longer than what is in flight
    (1, 9488, 72), (8, 9600, 40), (9, 9600, 40), (16, 19200, 24), (1, 20000, 16), (1, 64, 16392), (16, 160, 8200),
]


@pytest.mark.parametrize("t,n,k", SHAPES)
def test_forward(t, n, k):
    rng = np.random.default_rng(t + n + k)
    x, xv = _bf16(rng.standard_normal((t, k)))
    w, wv = _bf16(rng.standard_normal((n, k)) * 1.5 / np.sqrt(k))
    out, clean = _guarded((t, n // 2))
    keep, clean_y = _guarded((t, n))
    act, y = stq1.glu(x, w, save=True, out=out, y=keep)
    assert stq1.status() == 0 and clean() and clean_y()
    _check_forward(x, xv, w, wv, act, y)
    assert torch.equal(stq1.glu(x, w), act)                # keeping y changes nothing


@pytest.mark.parametrize("t,n,k", SHAPES)
def test_backward(t, n, k):
    rng = np.random.default_rng(t + n + k)
    x, xv = _bf16(rng.standard_normal((t, k)))
    w, wv = _bf16(rng.standard_normal((n, k)) * 1.5 / np.sqrt(k))
    d, dv = _bf16(rng.standard_normal((t, n // 2)) * 0.1)
    y, yv = _bf16(xv @ wv.T)
    bx, clean_x = _guarded((t, k))
    bw, clean_w = _guarded((n, k))
    dx, dw = stq1.glu_backward(d, y, x, w, dx=bx, dw=bw)
    assert stq1.status() == 0 and clean_x() and clean_w()
    dy = dense.glu_dy(dv, yv)
    g, u = yv[:, :n // 2], yv[:, n // 2:]
    # dY in fp32: exp, sum, division (2 units), and 1 + g (1 - s) with its cancellation: under 16 units of the terms
    s = 1 / (1 + np.exp(-g))
    e = 16 * 2.0 ** -24 * np.concatenate([np.abs(dv * u) * s * (1 + np.abs(g)), np.abs(dv * g) * s], axis=1)
    e = e + HALF * (np.abs(dy) + e) + TINY
    rx, rw = dense.glu_backward(dv, yv, xv, wv)
    for got, ref, err, mag, kk in (
            (dx, rx, e @ np.abs(wv), np.abs(dy) @ np.abs(wv), n),
            (dw, rw, e.T @ np.abs(xv), np.abs(dy).T @ np.abs(xv), t)):
        bar = err + _sum_err(kk, mag + err)
        _within(got.double().cpu().numpy(), ref, bar + HALF * (np.abs(ref) + bar) + TINY, f"gradient over {kk}")
    only_x, none = stq1.glu_backward(d, y, None, w, need_dw=False)
    assert none is None and torch.equal(only_x, dx)
    none, only_w = stq1.glu_backward(d, y, x, None, need_dx=False)
    assert none is None and torch.equal(only_w, dw)


def test_gradient_against_differences():
    """The gradients of a whole step along random directions, against fp64 central differences of the block."""
    rng = np.random.default_rng(3)
    t, n, k = 40, 64, 96
    x, xv = _bf16(rng.standard_normal((t, k)))
    w, wv = _bf16(rng.standard_normal((n, k)) / np.sqrt(k))
    d, dv = _bf16(rng.standard_normal((t, n // 2)))
    _, y = stq1.glu(x, w, save=True)
    dx, dw = (v.double().cpu().numpy() for v in stq1.glu_backward(d, y, x, w))
    h = 1e-4
    f = lambda a, b: float((dense.glu(a, b)[0] * dv).sum())  # noqa: E731
    for i in range(4):
        vx, vw = rng.standard_normal(xv.shape), rng.standard_normal(wv.shape)
        for v, grad, plus, minus in ((vx, dx, f(xv + h * vx, wv), f(xv - h * vx, wv)),
                                     (vw, dw, f(xv, wv + h * vw), f(xv, wv - h * vw))):
            # each gradient entry carries the bf16 roundings of y, dY and itself: independent ones of 2^-9 of the
            # entries' size on average, so their sum stays within 8 of its standard deviations of 3 * 2^-9 |grad| |v|
            slope = (plus - minus) / (2 * h)
            bar = 8 * 3 * 2.0 ** -9 * np.linalg.norm(grad * v) + 1e-5 * np.abs(grad * v).sum()
            assert abs(slope - (grad * v).sum()) <= bar, (i, slope, (grad * v).sum(), bar)


@pytest.mark.parametrize("t", [4, 40, 300])
def test_empty_rows_and_bad_values_stay_in_their_rows(t):
    rng = np.random.default_rng(t)
    n, k = 272, 520
    xv = rng.standard_normal((t, k))
    xv[0], xv[1, 5], xv[2, 7] = 0.0, np.nan, np.inf
    x, _ = _bf16(xv)
    w, wv = _bf16(rng.standard_normal((n, k)) / np.sqrt(k))
    act, y = stq1.glu(x, w, save=True)
    a, s = act.float().cpu().numpy(), y.float().cpu().numpy()
    assert not a[0].any() and not s[0].any()
    assert np.isnan(s[1]).all() and np.isnan(a[1]).all()
    assert not np.isfinite(s[2]).any()
    assert np.isfinite(a[3:]).all()
    good = x[3:].contiguous()
    assert torch.equal(stq1.glu(good, w), act[3:]) or t > 4    # the kernel may change with the token count
    # a token with a zero gradient adds nothing to dw, whatever its gate
    d, _ = _bf16(rng.standard_normal((t, n // 2)))
    clean = torch.nan_to_num(y, nan=0.0, posinf=100.0, neginf=-100.0)
    xc = torch.nan_to_num(x, nan=0.0, posinf=1.0)
    d[:3] = 0
    dx, dw = stq1.glu_backward(d, clean, xc, w)
    assert not dx[:3].any() and torch.isfinite(dw).all()


def test_far_gates():
    """Gates out to the ends of bf16: the gradients are finite and those of the formula."""
    g = np.array([-3e38, -1e30, -200, -100, -90, -88, -87, -50, 50, 87, 88, 90, 100, 200, 1e30, 3e38], np.float32)
    y, yv = _bf16(np.concatenate([g, np.full(16, 0.5, np.float32)])[None].repeat(16, 0))
    d, dv = _bf16(np.full((16, 16), 2.0 ** -12))
    w, wv = _bf16(np.eye(32))
    dx, _ = stq1.glu_backward(d, y, None, w, need_dw=False)
    ref = dense.glu_dy(dv, yv)
    # s below 2^-126 is lost in fp32: |d u g| * 2^-126 at most, for the gates where that happens
    _within(dx.double().cpu().numpy(), ref, np.abs(ref) * 2.0 ** -7 + 2.0 ** -112, "far gates")


def test_activations_calibrate_the_down_projection():
    """As it is used: the block's rows are the calibration inputs of the down projection's error."""
    rng = np.random.default_rng(8)
    t, n, k, h = 70, 512, 384, 64
    x, _ = _bf16(rng.standard_normal((t, k)))
    w, _ = _bf16(rng.standard_normal((n, k)) / np.sqrt(k))
    act = stq1.glu(x, w)
    diag = stq1.hessian_diag(act)
    a = act.double().cpu().numpy()
    assert np.allclose(diag.cpu().numpy()[0], (a * a).sum(0), rtol=2.0 ** -23)
    down = torch.from_numpy((rng.standard_normal((h, n // 2)) * 0.05).astype(np.float32)).cuda()
    packed = stq1.quantize_gpu(down, diag[0].contiguous(), mode="sherry")
    err = stq1.hessian_error(stq1.FMT_STQ1_0, packed, down[None], act[None], diag).cpu().numpy()[0]
    dhat = oracle.decode(packed.cpu().numpy(), h, n // 2)
    ref = oracle.hessian_error(down.cpu().numpy(), dhat, a)
    assert abs(err[0] - ref) <= 2.0 ** -6 * ref
    # the same layer at 8 bits for the tokens, next to its bf16 form
    q, s = stq1.quantize_i8(act)
    y8 = stq1.i8_matmul(q, s, *stq1.quantize_i8(down)).double().cpu().numpy()
    exact = a @ down.double().cpu().numpy().T
    step = s.double().cpu().numpy()[:, None] * 0.51
    rest = step * np.abs(down.double().cpu().numpy()).sum(1)[None] + (np.abs(a).sum(1)[:, None] + step * n / 2) * (
        np.abs(down.double().cpu().numpy()).max(1) / 127 * 0.51)[None]
    assert np.all(np.abs(y8 - exact) <= rest)


@pytest.mark.parametrize("t", [6, 90, 300])
def test_captured_step_follows_its_inputs(t):
    """Forward and backward captured in one graph, replayed after the inputs changed, give the eager bits."""
    rng = np.random.default_rng(t)
    n, k = 272, 392
    w, _ = _bf16(rng.standard_normal((n, k)) / np.sqrt(k))
    sets = [(_bf16(rng.standard_normal((t, k)))[0], _bf16(rng.standard_normal((t, n // 2)))[0]) for _ in range(2)]

    def step(x, d):
        act, y = stq1.glu(x, w, save=True)
        return (act, y) + stq1.glu_backward(d, y, x, w)

    eager = [step(*s) for s in sets]
    x, d = sets[0][0].clone(), sets[0][1].clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(x, d)
        side.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            got = step(x, d)
    for i in (1, 0):
        x.copy_(sets[i][0])
        d.copy_(sets[i][1])
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, eager[i]))


def test_binding_refuses_what_does_not_fit_together():
    x = torch.zeros((4, 64), dtype=torch.bfloat16, device="cuda")
    w = torch.zeros((32, 64), dtype=torch.bfloat16, device="cuda")
    d, y = x[:, :16].contiguous(), x[:, :32].contiguous()
    for bad in (lambda: stq1.glu(x, w[:, :32].contiguous()), lambda: stq1.glu(x.t(), w),
                lambda: stq1.glu(x, w, out=torch.zeros((4, 32), dtype=torch.bfloat16, device="cuda")),
                lambda: stq1.glu_backward(y, y, x, w), lambda: stq1.glu_backward(d, y, x[:3], w),
                lambda: stq1.glu_backward(d, y, None, w), lambda: stq1.glu_backward(d, y, x, None),
                lambda: stq1.glu_backward(d, y, x, w, need_dx=False, need_dw=False)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(TypeError):
        stq1.glu(x.float(), w)
    with pytest.raises(stq1.Stq1Error):
        stq1.glu(x, w[:24].contiguous())                    # N % 16
    with pytest.raises(stq1.Stq1Error):
        stq1.glu_backward(d, y, x, w, ws=torch.zeros(16, dtype=torch.uint8, device="cuda"))
    assert stq1.status() == 0
