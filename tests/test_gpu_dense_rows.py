"""A token's results do not depend on what the other tokens hold, bit for bit (needs a B200)."""

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import sub_bit_sparse_b200 as stq1

# streaming kernel; few tiles in pieces of K and whole; pairs of CTAs with whole tiles and with halves
SIZES = [(4, 272, 520), (16, 528, 2056), (40, 272, 520), (40, 272, 4104), (300, 272, 136), (640, 4096, 264),
         (1100, 3600, 72)]


def _pair(t, k):
    """bf16 x, the same with zeros, NaN and Inf in some of its rows, and the other rows."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(t + k)
    x = torch.randn((t, k), generator=gen, device="cuda").to(torch.bfloat16)
    bad = x.clone()
    rows = sorted({0, t // 2, t - 1})
    bad[rows[0]], bad[rows[1], 5], bad[rows[2], k - 1] = 0.0, float("nan"), float("inf")
    return gen, x, bad, [i for i in range(t) if i not in rows]


@pytest.mark.parametrize("t,n,k", SIZES)
def test_gated_block(t, n, k):
    gen, x, bad, rest = _pair(t, k)
    w = (torch.randn((n, k), generator=gen, device="cuda") / k ** 0.5).to(torch.bfloat16)
    for a, b in zip(stq1.glu(x, w, save=True), stq1.glu(bad, w, save=True)):
        assert torch.equal(a[rest], b[rest]) and torch.isfinite(b[rest]).all()


@pytest.mark.parametrize("t,n,k", SIZES)
def test_gradient_of_the_inputs(t, n, k):
    gen, y, bad, rest = _pair(t, n)
    w = (torch.randn((n, k), generator=gen, device="cuda") / n ** 0.5).to(torch.bfloat16)
    d = torch.randn((t, n // 2), generator=gen, device="cuda").to(torch.bfloat16)
    a, b = (stq1.glu_backward(d, v, None, w, need_dw=False)[0] for v in (y, bad))
    assert torch.equal(a[rest], b[rest]) and torch.isfinite(b[rest]).all()


@pytest.mark.parametrize("t,n,k", [(t, n // 32 * 32, k // 16 * 16) for t, n, k in SIZES])
def test_layer(t, n, k):
    gen, x, bad, rest = _pair(t, k)
    code = lambda r, c: stq1.quantize_i8(torch.randn((r, c), generator=gen, device="cuda") / c ** 0.5)  # noqa: E731
    gu, dn = code(n, k), code(k, n // 2)
    a, b = (stq1.i8_ffn(v, *gu, *dn) for v in (x, bad))
    assert torch.equal(a[rest], b[rest]) and torch.isfinite(b[rest]).all()
