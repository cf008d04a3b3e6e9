"""8-bit integer codes, products and the 8-bit gated layer against the oracle, bit for bit (needs a B200)."""

import os
import subprocess
import sys

import numpy as np
import pytest

import oracle
import workloads
from oracle import dense

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import sub_bit_sparse_b200 as stq1


def _dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def _bf16(v):
    """fp32 array -> (bf16 CUDA tensor, its values as fp32)."""
    t = torch.from_numpy(np.ascontiguousarray(v, dtype=np.float32)).to(torch.bfloat16)
    return t.cuda(), t.float().numpy()


def _same(got, ref):
    """Equal values; NaN where and only where the reference has NaN."""
    got, ref = np.asarray(got), np.asarray(ref)
    assert got.shape == ref.shape and got.dtype == ref.dtype
    bad = ~((got == ref) | (np.isnan(got) & np.isnan(ref)))
    assert not bad.any(), f"{bad.sum()} of {bad.size} differ, first at {np.argwhere(bad)[0]}"


def _guarded(shape, dtype, fill):
    """A tensor inside a larger one whose other elements hold `fill`, and a check that they still do."""
    n, pad = int(np.prod(shape)), 64
    whole = torch.full((n + 2 * pad,), fill, dtype=dtype, device="cuda")
    return whole[pad:pad + n].view(shape), lambda: bool(
        (whole[:pad] == fill).all()) and bool((whole[pad + n:] == fill).all())


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("r,k", [(1, 16), (3, 48), (7, 256), (300, 1024), (2, 1040), (5, 7168), (16, 8192), (3, 8208),
                                 (2, 20000)])
def test_codes_match_the_oracle(r, k, f32):
    rng = np.random.default_rng(r * k)
    v = (rng.standard_normal((r, k)) * 10.0 ** rng.uniform(-6, 6, (r, 1))).astype(np.float32)
    v[0, 0] = -0.0
    if f32:
        t, val = _dev(v), v
    else:
        t, val = _bf16(v)
    out, clean = _guarded((r, k), torch.int8, 77)
    sc, clean_s = _guarded((r,), torch.float32, 77.0)
    q, s = stq1.quantize_i8(t, out=out, scales=sc)
    rq, rs = dense.quantize_i8(val)
    _same(q.cpu().numpy(), rq)
    _same(s.cpu().numpy(), rs)
    assert clean() and clean_s() and stq1.status() == 0


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("k", [64, 2048])
def test_codes_of_zero_tiny_huge_and_non_finite_rows(k, f32):
    v = np.zeros((9, k), dtype=np.float32)
    v[:, 1] = [0, 2.0 ** -126, 2.0 ** -120, 2.0 ** -119, 2.0 ** 127, -np.inf, np.nan, 1, -1]
    v[5, 7], v[7, k - 1], v[8, 5] = 3, np.nan, 0.5
    t, val = (_dev(v), v) if f32 else _bf16(v)
    q, s = stq1.quantize_i8(t)
    rq, rs = dense.quantize_i8(val)
    _same(q.cpu().numpy(), rq)
    _same(s.cpu().numpy(), rs)
    w = _dev(np.ones((3, k), np.int8))
    y = stq1.i8_matmul(q, s, w, torch.ones(3, device="cuda")).cpu().numpy()
    assert np.isnan(y[[5, 6, 7]]).all() and np.isfinite(y[[0, 1, 2, 3, 4, 8]]).all()


def _codes(rng, r, k, low=-127):
    return rng.integers(low, 128, (r, k), dtype=np.int8), (rng.uniform(0.5, 2, r) * 1e-3).astype(np.float32)


SHAPES = [  # T, N, K: every token count where a kernel changes, and its neighbours; ragged N; K tails
    (1, 1, 16), (1, 17, 48), (1, 4096, 7168), (2, 100, 320), (3, 33, 2048), (5, 515, 976), (8, 256, 1024),
    (9, 129, 528), (15, 64, 4096), (16, 1000, 7168), (17, 2053, 2048), (24, 300, 1600), (31, 70, 336), (32, 128, 256),
    (33, 128, 144), (48, 1030, 1024), (64, 255, 640), (65, 257, 640), (77, 2053, 2048), (100, 3, 64), (127, 128, 128),
    (128, 4096, 2048), (129, 130, 112), (200, 1000, 3600), (255, 512, 16), (256, 256, 512), (257, 259, 272),
    (300, 4096, 1024), (512, 777, 1296), (700, 2048, 512), (1000, 1025, 1040), (1500, 4096, 256), (2049, 513, 384),
    (2500, 1001, 272), (2500, 1004, 64), (2561, 2056, 16), (5000, 600, 144), (4100, 4098, 48), (20000, 130, 32),
    # few tokens: outputs for more than one round of CTAs, one or two CTAs per SM, rows longer than what is in flight
    (1, 11008, 144), (2, 9473, 272), (3, 9500, 2064), (8, 18960, 48), (9, 20001, 32), (16, 9473, 80), (12, 25000, 16),
    (1, 200, 32784), (5, 70, 20000), (16, 70, 20000), (2, 20, 131056), (13, 5000, 1040),
]


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("t,n,k", SHAPES)
def test_product_is_bit_exact(t, n, k, bf16):
    rng = np.random.default_rng(t * 7 + n * 3 + k)
    xq, sx = _codes(rng, t, k, low=-128)
    wq, sw = _codes(rng, n, k, low=-128)
    dt = torch.bfloat16 if bf16 else torch.float32
    out, clean = _guarded((t, n), dt, 77.0) if (t * n) % 8 == 0 else (None, lambda: True)
    y = stq1.i8_matmul(_dev(xq), _dev(sx), _dev(wq), _dev(sw), out=out, dtype=dt)
    assert stq1.status() == 0
    ref = dense.i8_matmul(xq, sx, wq, sw)
    if bf16:
        ref = torch.from_numpy(ref).to(torch.bfloat16).float().numpy()
    _same(y.float().cpu().numpy(), ref)
    assert clean()


@pytest.mark.parametrize("t", [1, 40, 300])
def test_largest_sums_do_not_wrap(t):
    # 131056 products of -128 * -128: 2147221504, 262143 below 2^31
    k = 131056
    xq, wq = np.full((t, k), -128, np.int8), np.full((9, k), -128, np.int8)
    wq[1] = 127
    one = np.ones(max(t, 9), np.float32)
    y = stq1.i8_matmul(_dev(xq), _dev(one[:t]), _dev(wq), _dev(one[:9])).cpu().numpy()
    ref = np.full((t, 9), 128.0 * 128 * k, np.float32)
    ref[:, 1] = -128.0 * 127 * k
    _same(y, ref)


@pytest.mark.parametrize("t", [2, 20, 150, 600])
def test_special_scales_reach_only_their_rows_and_channels(t):
    rng = np.random.default_rng(t)
    xq, sx = _codes(rng, t, 256)
    wq, sw = _codes(rng, 70, 256)
    sx[0], sx[1], sw[3], sw[69] = np.inf, np.nan, np.nan, 0.0
    ref = dense.i8_matmul(xq, sx, wq, sw)
    _same(stq1.i8_matmul(_dev(xq), _dev(sx), _dev(wq), _dev(sw)).cpu().numpy(), ref)


def _layer(rng, n, h):
    gu, sgu = dense.quantize_i8(rng.standard_normal((n, h)) / np.sqrt(h))
    dn, sdn = dense.quantize_i8(rng.standard_normal((h, n // 2)) / np.sqrt(n // 2))
    return gu, sgu, dn, sdn


@pytest.mark.parametrize("t,n,h", [(1, 32, 16), (1, 4096, 7168), (2, 96, 272), (3, 2080, 1040), (8, 512, 512),
                                   (9, 160, 128), (16, 1024, 1536), (17, 224, 208), (32, 256, 512), (33, 256, 512),
                                   (65, 544, 336), (128, 1024, 256), (130, 288, 1040), (300, 512, 512),
                                   (520, 1056, 784), (1030, 512, 256), (1, 9600, 64), (2, 9632, 80), (8, 19200, 32),
                                   (9, 9600, 48), (3, 64, 9600), (16, 96, 9600), (7, 32, 20016), (4, 16416, 32)])
def test_layer_gives_the_bits_of_the_chain(t, n, h):
    rng = np.random.default_rng(t + n + h)
    x, xv = _bf16(rng.standard_normal((t, h)) * 2)
    lw = _layer(rng, n, h)
    dv = [_dev(a) for a in lw]
    out, clean = _guarded((t, h), torch.float32, 77.0)
    y = stq1.i8_ffn(x, *dv, out=out)
    assert stq1.status() == 0 and clean()
    # the chain of the library's own calls, and the oracle
    q, s = stq1.quantize_i8(x)
    act = stq1.swiglu(stq1.i8_matmul(q, s, dv[0], dv[1]), n)
    chain = stq1.i8_matmul(*stq1.quantize_i8(act), dv[2], dv[3])
    _same(y.cpu().numpy(), chain.cpu().numpy())
    _same(y.cpu().numpy(), dense.i8_ffn(xv, *lw))


@pytest.mark.parametrize("t", [4, 20, 140, 600])
def test_layer_keeps_a_bad_token_to_its_row(t):
    rng = np.random.default_rng(5)
    v = rng.standard_normal((t, 512))
    v[1, 9], v[2, :] = np.nan, 0.0
    x, xv = _bf16(v)
    lw = _layer(rng, 256, 512)
    y = stq1.i8_ffn(x, *[_dev(a) for a in lw]).cpu().numpy()
    assert np.isnan(y[1]).all() and not y[2].any()
    keep = [i for i in range(t) if i != 1]
    _same(y[keep], dense.i8_ffn(xv[keep], *lw))


@pytest.mark.parametrize("t", [1, 12, 90, 400])
def test_layer_beside_the_routed_experts(t):
    """A layer as it runs: the routed experts in the ternary format plus the expert that every token passes."""
    E, n, h, topk = 6, 512, 512, 3
    rng = np.random.default_rng(t)
    gu = np.concatenate([stq1.quantize_ref(workloads.gaussian_matrix(n, h, 0.05, seed=800 + e)) for e in range(E)])
    dn = np.concatenate([stq1.quantize_ref(workloads.gaussian_matrix(h, n // 2, 0.05, seed=900 + e)) for e in range(E)])
    xb = workloads.activations_bf16(t, h, seed=97)
    ids, wts = workloads.zipf_topk_ids(t, E, topk, seed=98), workloads.softmax_route_weights(t, topk, seed=99)
    x = _dev(xb.astype(np.uint16).view(np.int16)).view(torch.bfloat16)
    lw = _layer(rng, n, h)
    routed = stq1.moe_ffn(_dev(gu), _dev(dn), x, _dev(ids.astype(np.int32)), _dev(wts), n, h, E)
    out = (routed + stq1.i8_ffn(x, *[_dev(a) for a in lw])).cpu().numpy()
    assert stq1.status() == 0
    eg, ed = oracle.packed_size(n, h), oracle.packed_size(h, n // 2)
    ref, scale = oracle.moe_ffn(lambda e: gu[e * eg:(e + 1) * eg], lambda e: dn[e * ed:(e + 1) * ed], xb, ids, wts, n,
                                h, abs_sum=True)
    shared = dense.i8_ffn(workloads.f32_from_bf16_bits(xb), *lw).astype(np.float64)
    # the routed part's own bar, and half a step for the sum
    bar = oracle.tolerance(scale)
    assert np.all(np.abs(out - (ref + shared)) <= bar + 2.0 ** -24 * (np.abs(ref + shared) + bar))


@pytest.mark.parametrize("t", [1, 16, 64, 500])
def test_captured_layer_follows_its_inputs(t):
    """Two graphs of the layer, replayed in turn and after the inputs changed, give the eager bits."""
    n, h = 512, 768
    rng = np.random.default_rng(t)
    dv = [_dev(a) for a in _layer(rng, n, h)]
    xs = [_bf16(rng.standard_normal((t, h)))[0] for _ in range(3)]
    eager = [stq1.i8_ffn(x, *dv) for x in xs]
    static = [xs[0].clone(), xs[1].clone()]
    side = torch.cuda.Stream()
    graphs, outs = [], []
    with torch.cuda.stream(side):
        for x in static:
            stq1.i8_ffn(x, *dv)
            side.synchronize()
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=side):
                outs.append(stq1.i8_ffn(x, *dv))
            graphs.append(g)
    torch.cuda.synchronize()
    for i, want in ((0, (0, None)), (1, (0, 1))):
        graphs[i].replay()
        torch.cuda.synchronize()
        for o, w in zip(outs, want):
            if w is not None:
                assert torch.equal(o, eager[w])
    static[0].copy_(xs[2])
    graphs[0].replay()
    graphs[1].replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], eager[2]) and torch.equal(outs[1], eager[1])


def test_first_call_of_a_process_may_be_captured():
    code = """
import sys; sys.path.insert(0, %r)
import torch, sub_bit_sparse_b200 as stq1
x = torch.randint(-127, 128, (5, 512), dtype=torch.int8, device="cuda")
w = torch.randint(-127, 128, (40, 512), dtype=torch.int8, device="cuda")
sx, sw, y = torch.ones(5, device="cuda"), torch.ones(40, device="cuda"), torch.zeros(5, 40, device="cuda")
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    stq1.i8_matmul(x, sx, w, sw, out=y)
g.replay()
assert torch.equal(y.double(), x.double() @ w.double().T) and stq1.status() == 0
print("OK")
""" % os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    res = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert res.stdout.strip().endswith("OK"), res.stdout + res.stderr


def test_weights_coded_just_before_the_layer():
    """Codes of new weights and the layer that reads them, back to back on one stream, again and again."""
    rng = np.random.default_rng(11)
    n, h = 1024, 1536
    for t in (1, 7, 16, 40):
        x = _bf16(rng.standard_normal((t, h)))[0]
        fw = [torch.randn(n, h, device="cuda") / h ** 0.5 for _ in range(4)]
        fd = [torch.randn(h, n // 2, device="cuda") / (n // 2) ** 0.5 for _ in range(4)]
        want = []
        for a, b in zip(fw, fd):
            gu, dn = stq1.quantize_i8(a), stq1.quantize_i8(b)
            torch.cuda.synchronize()
            want.append(stq1.i8_ffn(x, *gu, *dn))
        gu, dn = stq1.quantize_i8(fw[0]), stq1.quantize_i8(fd[0])
        torch.cuda.synchronize()
        for _ in range(3):
            got = []
            for a, b in zip(fw, fd):
                stq1.quantize_i8(b, out=dn[0], scales=dn[1])
                stq1.quantize_i8(a, out=gu[0], scales=gu[1])
                got.append(stq1.i8_ffn(x, *gu, *dn))
            torch.cuda.synchronize()
            assert all(torch.equal(g, w) for g, w in zip(got, want)), t


def test_two_streams_at_once():
    rng = np.random.default_rng(9)
    dv = [_dev(a) for a in _layer(rng, 1024, 1024)]
    xs = [_bf16(rng.standard_normal((t, 1024)))[0] for t in (1, 7, 40, 300)]
    want = [stq1.i8_ffn(x, *dv) for x in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in xs]
    for _ in range(5):
        got = []
        for s, x in zip(streams, xs):
            with torch.cuda.stream(s):
                got.append(stq1.i8_ffn(x, *dv))
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_binding_refuses_what_does_not_fit_together():
    q, s = torch.zeros((4, 64), dtype=torch.int8, device="cuda"), torch.zeros(4, device="cuda")
    x = torch.zeros((4, 64), dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError):
        stq1.i8_matmul(q, s, q[:, :32].contiguous(), s)          # other K
    with pytest.raises(ValueError):
        stq1.i8_matmul(q, s[:3], q, s)
    with pytest.raises(ValueError):
        stq1.i8_matmul(q.t(), s, q, s)                           # not contiguous
    with pytest.raises(TypeError):
        stq1.i8_matmul(q, s, q, s, dtype=torch.float16)
    with pytest.raises(TypeError):
        stq1.quantize_i8(q)
    with pytest.raises(ValueError):
        stq1.quantize_i8(x, out=torch.zeros((4, 32), dtype=torch.int8, device="cuda"))
    with pytest.raises(stq1.Stq1Error):
        stq1.quantize_i8(x[:, :8].contiguous())                  # K % 16
    with pytest.raises(ValueError):
        stq1.i8_ffn(x, q, s, q, s)                               # down is [H, N/2] = [64, 2]
    with pytest.raises(stq1.Stq1Error):
        stq1.i8_ffn(x, torch.zeros((64, 64), dtype=torch.int8, device="cuda"), torch.zeros(64, device="cuda"),
                    torch.zeros((64, 32), dtype=torch.int8, device="cuda"), torch.zeros(64, device="cuda"),
                    ws=torch.zeros(16, dtype=torch.uint8, device="cuda"))
    assert stq1.status() == 0
