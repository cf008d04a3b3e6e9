"""Few tokens where a CTA's place is taken by several in turn and its slots are filled again (needs a B200).

The streaming kernel keeps more than one round of CTAs for int8 products of up
to 8 tokens with more than 148 * 128 outputs, and for gated blocks of up to 8
tokens with more than 148 * 32.  With at least 41 steps of 128 bytes (33 where
the codes are made inside) a warp has more steps than its four slots.
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


def _codes(gen, r, k):
    q = torch.randint(-128, 128, (r, k), generator=gen, device="cuda", dtype=torch.int8)
    return q, (torch.rand(r, generator=gen, device="cuda") + 0.5) * 1e-3


def _product(xq, sx, wq, sw):
    """fp64 sums of codes are exact; then the two fp32 products."""
    acc = torch.cat([xq.double() @ part.double().T for part in wq.split(4096)], dim=1).float()
    return (acc * sx[:, None]) * sw[None, :]


@pytest.mark.parametrize("t,n,k", [(1, 18960, 5200), (2, 20001, 5136), (5, 19001, 5248), (8, 30003, 6160),
                                   (8, 18945, 10256)])
def test_product(t, n, k):
    gen = _gen(t + n)
    (xq, sx), (wq, sw) = _codes(gen, t, k), _codes(gen, n, k)
    ref = _product(xq, sx, wq, sw)
    assert torch.equal(stq1.i8_matmul(xq, sx, wq, sw), ref)
    assert torch.equal(stq1.i8_matmul(xq, sx, wq, sw, dtype=torch.bfloat16), ref.to(torch.bfloat16))
    assert stq1.status() == 0


@pytest.mark.parametrize("t,n,k", [(1, 9600, 2632), (3, 9488, 2680), (8, 19200, 4104), (7, 28688, 3080)])
def test_gated_block(t, n, k):
    gen = _gen(t + n)
    x = torch.randn((t, k), generator=gen, device="cuda").to(torch.bfloat16)
    w = (torch.randn((n, k), generator=gen, device="cuda") * (1.5 / k ** 0.5)).to(torch.bfloat16)
    act, y = stq1.glu(x, w, save=True)
    half, xd = n // 2, x.double()
    s = torch.cat([xd @ part.double().T for part in w.split(4096)], dim=1)
    mag = torch.cat([xd.abs() @ part.double().abs().T for part in w.split(4096)], dim=1)
    # a tensor core adds eight or more exact products at a time and cuts what does not fit 24 bits; bf16 rounds by 2^-8
    # of the value at most; SiLU has a slope of at most 1.1
    e = (k / 8 + 32) * 2.0 ** -23 * mag
    g, u, eg, eu = s[:, :half], s[:, half:], e[:, :half], e[:, half:]
    silu = g / (1 + torch.exp(-g))
    through = 1.1 * eg * u.abs() + (silu.abs() + 1.1 * eg) * eu
    ref = silu * u
    assert bool(((y.double() - s).abs() <= e + 2.0 ** -8 * (s.abs() + e) + 2.0 ** -134).all())
    assert bool(((act.double() - ref).abs() <= through + 2.0 ** -8 * (ref.abs() + through) + 2.0 ** -134).all())
    assert torch.equal(stq1.glu(x, w), act) and stq1.status() == 0


@pytest.mark.parametrize("t,n,h", [(1, 8224, 18960), (8, 8256, 18976), (3, 9600, 5200), (8, 19200, 5152)])
def test_layer(t, n, h):
    gen = _gen(t + n)
    x = torch.randn((t, h), generator=gen, device="cuda").to(torch.bfloat16)
    gu, sg = _codes(gen, n, h)
    dn, sd = _codes(gen, h, n // 2)
    sg = sg * (20.0 / h ** 0.5)                             # sums of about unit size
    got = stq1.i8_ffn(x, gu, sg, dn, sd)
    q, s = stq1.quantize_i8(x)
    y = _product(q, s, gu, sg)
    assert 0.05 < float(y.abs().mean()) < 20
    aq, sa = stq1.quantize_i8(stq1.swiglu(y, n))
    assert torch.equal(got, _product(aq, sa, dn, sd)) and stq1.status() == 0
