"""Routed experts with one or two (token, expert) pairs in all: one token with top-1 or top-2, two with top-1 (needs a B200).

No expert then has enough pairs for the tensor-core decode kernel.
"""

import numpy as np
import pytest

import oracle
import workloads

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import sub_bit_sparse_b200 as stq1

E, N, H = 5, 1024, 512
IDS = [[[3]], [[0, 4]], [[2, 2]], [[4], [1]], [[1], [1]]]


def _dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def _inputs(ids):
    ids = np.asarray(ids, np.int32)
    t, topk = ids.shape
    gu = np.concatenate([stq1.quantize_ref(workloads.gaussian_matrix(N, H, 0.05, seed=300 + e)) for e in range(E)])
    dn = np.concatenate([stq1.quantize_ref(workloads.gaussian_matrix(H, N // 2, 0.05, seed=400 + e)) for e in range(E)])
    xb = workloads.activations_bf16(t, H, seed=5 + t)
    wts = workloads.softmax_route_weights(t, topk, seed=6)
    x = _dev(xb.astype(np.uint16).view(np.int16)).view(torch.bfloat16)
    return ids, gu, dn, xb, x, wts


@pytest.mark.parametrize("flags", [0, 1])
@pytest.mark.parametrize("ids", IDS)
def test_gateup_and_layer(ids, flags):
    ids, gu, dn, xb, x, wts = _inputs(ids)
    eg, ed = oracle.packed_size(N, H), oracle.packed_size(H, N // 2)
    getg, getd = lambda e: gu[e * eg:(e + 1) * eg], lambda e: dn[e * ed:(e + 1) * ed]  # noqa: E731
    y = stq1.moe_gateup(_dev(gu), x, _dev(ids), _dev(wts), N, H, E, flags=flags).cpu().numpy()
    ref, scale = oracle.moe_gateup(getg, xb, ids, wts, N, H, flags=flags, abs_sum=True)
    assert np.all(np.abs(y.reshape(ref.shape) - ref) <= oracle.tolerance(scale))
    out = stq1.moe_ffn(_dev(gu), _dev(dn), x, _dev(ids), _dev(wts), N, H, E, flags=flags).cpu().numpy()
    ref, scale = oracle.moe_ffn(getg, getd, xb, ids, wts, N, H, flags=flags, abs_sum=True)
    assert np.all(np.abs(out - ref) <= oracle.tolerance(scale))
    assert stq1.status() == 0


@pytest.mark.parametrize("ids", IDS)
def test_local_share_of_the_layer(ids):
    """Both halves of the experts as expert parallelism runs them: their sum is the layer."""
    ids, gu, dn, xb, x, wts = _inputs(ids)
    eg, ed = oracle.packed_size(N, H), oracle.packed_size(H, N // 2)
    out = sum(stq1.moe_ffn_local(_dev(gu[b * eg:e * eg]), _dev(dn[b * ed:e * ed]), x, _dev(ids), _dev(wts), N, H, e - b,
                                 b) for b, e in ((0, 3), (3, E))).cpu().numpy()
    ref, scale = oracle.moe_ffn(lambda e: gu[e * eg:(e + 1) * eg], lambda e: dn[e * ed:(e + 1) * ed], xb, ids, wts, N, H,
                                abs_sum=True)
    assert np.all(np.abs(out - ref) <= oracle.tolerance(scale))
    assert stq1.status() == 0


def test_captured_with_the_8_bit_layer():
    """One token: a routed expert and the layer every token passes, in one graph."""
    ids, gu, dn, xb, x, wts = _inputs([[3]])
    gen = torch.Generator(device="cuda")
    gen.manual_seed(1)
    code = lambda r, c: stq1.quantize_i8(torch.randn((r, c), generator=gen, device="cuda") / c ** 0.5)  # noqa: E731
    a = (_dev(gu), _dev(dn), x, _dev(ids), _dev(wts), N, H, E)
    b = code(N, H) + code(H, N // 2)
    ws = torch.empty(stq1.LIB.stq1_moe_ffn_workspace(1, 1, E, N, H, 0), dtype=torch.uint8, device="cuda")
    step = lambda: stq1.moe_ffn(*a, ws=ws) + stq1.i8_ffn(x, *b)  # noqa: E731
    want = step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
        side.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            got = step()
    for _ in range(2):
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(got, want)
    assert stq1.status() == 0
