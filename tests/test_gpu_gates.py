"""The gated activation over the whole range of gates, bit for bit (needs a B200).

stq1_glu and stq1_i8_ffn promise stq1_swiglu's rounding of the fp32 gate and up
sums.  Inputs here make those sums known exactly: a token of the bf16 block has
one or two channels, 1 and 2^-9, so that a sum has at most 17 bits; the 8-bit
layer's sums are integers times scales, which stq1_i8_matmul gives.  Products of
few bits fall on the midpoint between two bf16 values, where only the exact
value decides, far more often than products of random ones.
"""

import numpy as np
import pytest

import oracle
from oracle import dense

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import sub_bit_sparse_b200 as stq1

FAR = [50, 87, 87.5, 88, 88.5, 89, 100, 104, 512, 700, 704, 708, 710, 712, 720, 800, 1000, 1024, 1416, 1424, 2000, 2128,
       2496, 2832, 2848, 4000, 4096, 5000, 1e5, 1e10, 1e30, 3e38]


def _block(seed, t, half, k):
    """bf16 x [t, k] >= 0 and w [2 half, k], and the sums [t, 2 half], exact in fp32."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    rnd = lambda *s: torch.rand(*s, generator=gen, device="cuda", dtype=torch.float64)  # noqa: E731
    # mantissas of eight bits in [1, 2) with a sign; one exponent per row, so that two channels add without loss
    mant = (128 + torch.floor(128 * rnd(2 * half, k))) / 128 * torch.where(rnd(2 * half, k) < 0.5, -1.0, 1.0)
    kind = rnd(half)
    eg = torch.where(kind < 0.4, torch.floor(4 + 10 * rnd(half)),              # 16 to 32768
                     torch.where(kind < 0.8, torch.floor(-8 + 16 * rnd(half)), torch.floor(-60 + 180 * rnd(half))))
    eu = torch.where(rnd(half) < 0.7, torch.floor(-3 + 6 * rnd(half)), torch.floor(-60 + 120 * rnd(half)))
    w = mant * torch.exp2(torch.cat([eg, eu]))[:, None]
    m = len(FAR)
    if half >= 4 * m:                                  # whole rows of far gates, both signs, beside ordinary ones
        far = torch.tensor(FAR, device="cuda", dtype=torch.float64)
        w[0:2 * m:2], w[2 * m:4 * m:2] = far[:, None], -far[:, None]
        w[half:half + 4 * m] = mant[half:half + 4 * m]
        w[half:half + 4 * m:8] = 0.0                   # some with an up sum of zero
    w = w.to(torch.bfloat16)
    a = torch.randint(k, (t,), generator=gen, device="cuda")
    b = (a + 1 + torch.randint(k - 1, (t,), generator=gen, device="cuda")) % k
    two = torch.arange(t, device="cuda") % 3 == 2
    x = torch.zeros((t, k), device="cuda", dtype=torch.bfloat16)
    x[torch.arange(t, device="cuda"), a] = 1.0
    x[torch.arange(t, device="cuda")[two], b[two]] = 2.0 ** -9
    wt = w.double().T.contiguous()
    y = wt[a] + torch.where(two, 2.0 ** -9, 0.0)[:, None] * wt[b]
    assert torch.equal(y.float().double(), y)
    return x, w, y.float()


def _bits(v):
    return v.view(torch.int16)


def _same_bits(got, ref):
    bad = (_bits(got) != _bits(ref)) & ~(torch.isnan(got) & torch.isnan(ref))
    if bad.any():
        at = torch.nonzero(bad)
        i = tuple(at[0].tolist())
        raise AssertionError(f"{len(at)} of {bad.numel()} differ, first at {i}: {got[i].item()} for {ref[i].item()}")


# one token and few, few tiles in several pieces of K and in one, pairs of CTAs with whole and half tiles
@pytest.mark.parametrize("t,n,k", [(1, 4096, 64), (5, 4096, 1024), (9, 4096, 72), (16, 2080, 264), (40, 1024, 4096),
                                   (40, 1024, 2048), (40, 4096, 1024), (100, 4096, 64), (300, 4096, 264),
                                   (640, 4096, 64), (1000, 4112, 136)])
def test_block_activation_is_swiglu_of_the_sums(t, n, k):
    x, w, y = _block(t * 3 + k, t, n // 2, k)
    ref = stq1.swiglu(y, n)
    act, kept = stq1.glu(x, w, save=True)
    _same_bits(act, ref)
    _same_bits(kept, y.to(torch.bfloat16))
    _same_bits(stq1.glu(x, w), ref)
    rows = slice(0, min(t, 64))
    # The oracle's value is fp64 as well: e^-g is off by up to 1 unit of 2^-52, the sum, the division and the product by
    # half a unit each, 2.5 units on each side and so less than 2^-49 between them.  That decides where the exact value
    # is as near to a midpoint (g = 1.5 * 2^-53, u = 131 * 2^-41: g u / 2 is a midpoint and SiLU(g) u is 2^-53 above it).
    yy = y[rows].double().cpu().numpy()
    v = oracle.silu(yy[:, :n // 2]) * yy[:, n // 2:]
    got = _bits(act[rows]).cpu().numpy().view(np.uint16)
    low, high = (oracle.bf16_bits_from_f64(v * (1 + e)) for e in (-2.0 ** -49, 2.0 ** -49))
    assert ((got == low) | (got == high)).all() and (low != high).mean() < 0.02
    assert stq1.status() == 0


def test_block_activation_over_many_values():
    """33 million pairs of sums, a fifth of them with gates between 2^-60 and 2^120."""
    for seed in range(4):
        x, w, y = _block(1000 + seed, 4096, 2048, 64)
        _same_bits(stq1.glu(x, w), stq1.swiglu(y, 4096))
    assert stq1.status() == 0


def _far_layer(rng, n, h):
    """Codes and scales whose sums for one-channel tokens have few bits and gates up to about 6000."""
    gu = np.where(rng.random((n, h)) < 0.5, -1, 1) * rng.integers(16, 128, (n, h))
    half = n // 2
    sg = np.concatenate([2.0 ** rng.integers(3, 6, half), 2.0 ** rng.integers(-7, -4, half)]).astype(np.float32)
    dn, sdn = dense.quantize_i8(rng.standard_normal((h, half)) / np.sqrt(half))
    return gu.astype(np.int8), sg, dn, sdn


@pytest.mark.parametrize("t,n,h", [(1, 4096, 1024), (4, 4096, 256), (9, 4096, 512), (16, 4096, 272), (40, 1024, 2048),
                                   (40, 4096, 1024), (128, 4096, 256), (700, 4096, 144)])
def test_layer_gives_the_bits_of_the_chain_for_far_gates(t, n, h):
    rng = np.random.default_rng(t + n + h)
    lw = _far_layer(rng, n, h)
    xv = np.zeros((t, h), np.float32)
    xv[np.arange(t), rng.integers(0, h, t)] = 1.0
    # the inputs hold what they are for: gates past 710 whose product is on the midpoint of two bf16 values
    xq, sx = dense.quantize_i8(xv)
    y = dense.i8_matmul(xq, sx, lw[0], lw[1]).astype(np.float64)
    g, v = y[:, :n // 2], (y[:, :n // 2] * y[:, n // 2:]).astype(np.float32)
    assert ((g > 712) & ((v.view(np.uint32) & 0xFFFF) == 0x8000)).sum() >= 3
    x = torch.from_numpy(xv).to(torch.bfloat16).cuda()
    dv = [torch.from_numpy(np.ascontiguousarray(a)).cuda() for a in lw]
    got = stq1.i8_ffn(x, *dv)
    q, s = stq1.quantize_i8(x)
    act = stq1.swiglu(stq1.i8_matmul(q, s, dv[0], dv[1]), n)
    chain = stq1.i8_matmul(*stq1.quantize_i8(act), dv[2], dv[3])
    assert torch.isfinite(chain).all() and torch.equal(got, chain)
    assert np.array_equal(got.cpu().numpy(), dense.i8_ffn(xv, *lw))
    assert stq1.status() == 0
