"""Operands and results whose offsets pass 32 bits: more than 2^31 elements (needs a B200).

The inputs make every result exact, so that it is compared bit for bit, part by part.
"""

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import sub_bit_sparse_b200 as stq1


def _gen(seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    return gen


def _int(gen, low, high, shape, dtype):
    """Integers of [low, high], made without a wider copy of the whole."""
    out = torch.empty(shape, dtype=dtype, device="cuda")
    for part in out.split(max(1, (1 << 27) // shape[1])):
        part.copy_(torch.randint(low, high + 1, part.shape, generator=gen, device="cuda", dtype=torch.int8))
    return out


def _parts(n, step):
    return [slice(i, min(i + step, n)) for i in range(0, n, step)]


@pytest.mark.parametrize("t,n", [(70001, 40001), (70001, 40008), (8, 270000001)])
def test_product(t, n):
    gen = _gen(t + n)
    x, w = _int(gen, -128, 127, (t, 16), torch.int8), _int(gen, -128, 127, (n, 16), torch.int8)
    sx, sw = torch.rand(t, generator=gen, device="cuda") + 0.5, torch.rand(n, generator=gen, device="cuda") + 0.5
    y = stq1.i8_matmul(x, sx, w, sw, dtype=torch.bfloat16)
    assert stq1.status() == 0 and y.numel() > 2 ** 31
    for p in _parts(t, 2048):
        for q in _parts(n, 1 << 22):
            ref = (x[p].double() @ w[q].double().T).float().mul_(sx[p, None]).mul_(sw[None, q])
            assert torch.equal(y[p, q], ref.to(torch.bfloat16)), (p, q)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_codes(dtype):
    r, k = 300001, 8192
    src = _int(_gen(1), -127, 127, (r, k), dtype)
    src[:, 0] = 127                                         # inverse scale 1: the codes are the values
    q, s = stq1.quantize_i8(src)
    assert stq1.status() == 0 and bool((s == 1).all())
    for p in _parts(r, 16384):
        assert torch.equal(q[p], src[p].to(torch.int8)), p


def test_gated_block():
    t, n, k = 70001, 32784, 8
    gen = _gen(2)
    x, w = _int(gen, -2, 2, (t, k), torch.bfloat16), _int(gen, -2, 2, (n, k), torch.bfloat16)
    act, y = stq1.glu(x, w, save=True)
    assert stq1.status() == 0 and y.numel() > 2 ** 31
    for p in _parts(t, 4096):
        ref = x[p].float() @ w.float().T                    # integers of at most 32
        assert torch.equal(y[p], ref.to(torch.bfloat16)) and torch.equal(act[p], stq1.swiglu(ref, n)), p


def test_gradients():
    # gates of 0 and 64, where s is 1/2 and 1: dG = d u / 2 and d u, dU = 0 and 64 d, and all sums fit 24 bits
    t, n, k = 70001, 32784, 8
    gen = _gen(3)
    y = _int(gen, -2, 2, (t, n), torch.bfloat16)
    half = n // 2
    y[:, :half] = (y[:, :half] > 0).to(torch.bfloat16) * 64
    d = _int(gen, -1, 1, (t, half), torch.bfloat16)
    x, w = _int(gen, -1, 1, (t, k), torch.bfloat16), _int(gen, -1, 1, (n, k), torch.bfloat16)
    dx, dw = stq1.glu_backward(d, y, x, w)
    assert stq1.status() == 0
    ref = torch.zeros((n, k), dtype=torch.float64, device="cuda")
    for p in _parts(t, 4096):
        g, u, dv = y[p, :half].double(), y[p, half:].double(), d[p].double()
        dy = torch.cat([dv * u * torch.where(g > 0, 1.0, 0.5), dv * g], dim=1)
        assert torch.equal(dx[p], (dy @ w.double()).float().to(torch.bfloat16)), p
        ref += dy.T @ x[p].double()
    assert float(ref.abs().max()) < 2 ** 23
    assert torch.equal(dw, ref.float().to(torch.bfloat16))
