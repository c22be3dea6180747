"""The float64 definitions of the scored router, FP8 rows and FP8 products
pinned against something other than themselves (hand-worked cases, torch's
own conversions, autograd), and what the new entry points refuse, without a GPU."""

import ctypes

import numpy as np
import pytest
import torch

from oracle import scored_fp8 as O8
from quantized_rl_fine_b200 import accounting, build, ep, layer, moeq, synth


# ----------------------------------------------------------------------------- definitions

def test_selection_by_hand():
    # four experts in two groups; the bias moves expert 3 ahead, its gate stays its score
    logits = np.array([[2.0, 0.0, 1.0, -1.0]])
    s = 1 / (1 + np.exp(-logits[0]))
    idx, g = O8.route_scored(logits, 2, score="sigmoid", renorm=False, bias=np.array([0, 0, 0, 1.0]))
    assert idx.tolist() == [[3, 0]] and np.allclose(g, [[s[3], s[0]]])
    # one group kept: by the maximum group 0 (2.0), by the two largest keys too (s0 + s1 > s2 + s3)
    idx, g = O8.route_scored(logits, 2, score="sigmoid", groups=2, topk_groups=1, group_top=2, scale=3.0)
    assert idx.tolist() == [[0, 1]] and np.allclose(g, [3 * s[:2] / s[:2].sum()])
    # ties: the lower id, and the lower group
    idx, _ = O8.route_scored(np.zeros((1, 6)), 3, groups=3, topk_groups=2)
    assert idx.tolist() == [[0, 1, 2]]
    # masked experts come last with gate 0
    idx, g = O8.route_scored(np.array([[-np.inf, 1.0, np.nan, 0.0]]), 3)
    assert idx.tolist() == [[1, 3, 0]] and g[0, 2] == 0 and np.isclose(g.sum(), 1)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
def test_router_gradient_matches_autograd(score, renorm):
    g = torch.Generator().manual_seed(4)
    x = torch.randn((7, 9), generator=g, dtype=torch.float64, requires_grad=True)
    dg = torch.randn((7, 3), generator=g, dtype=torch.float64)
    idx, gates = O8.route_scored(x.detach().numpy(), 3, score=score, renorm=renorm, scale=2.0)
    s = torch.sigmoid(x) if score == "sigmoid" else torch.softmax(x, 1)
    w = s.gather(1, torch.from_numpy(idx).long())
    if renorm:
        w = w / w.sum(1, keepdim=True)
    assert np.allclose(gates, 2.0 * w.detach().numpy(), rtol=1e-12)
    (want,) = torch.autograd.grad((2.0 * w * dg).sum(), x)
    got = O8.route_scored_bwd(dg.numpy(), x.detach().numpy(), idx, score, renorm, 2.0)
    assert np.allclose(got, want.numpy(), rtol=1e-10, atol=1e-14)


def test_e4m3_table_and_rounding_match_torch():
    codes = np.arange(256, dtype=np.uint8)
    want = torch.from_numpy(codes).view(torch.float8_e4m3fn).float().numpy()
    have = O8.e4m3_values()
    assert np.array_equal(np.isnan(have), np.isnan(want))
    assert np.array_equal(have[~np.isnan(have)], want[~np.isnan(want)])
    x = torch.randn(50000, generator=torch.Generator().manual_seed(0)) * 2.0 ** torch.randint(-14, 8, (50000,))
    mid = torch.from_numpy((have[:126] + have[1:127]) / 2).float()          # every halfway point
    x = torch.cat([x, mid, -mid]).clamp(-448, 448)
    assert np.array_equal(O8.e4m3_nearest(x.numpy()), x.to(torch.float8_e4m3fn).view(torch.uint8).numpy())


def test_block_exponents_by_hand():
    v = np.zeros((6, 128))
    v[1, 3], v[2, 3], v[3, 3], v[4, 3], v[5, 3] = 448.0, 448.0001, 1.0, 2.0 ** -133, np.inf
    assert O8.block_exponents(v, 128)[:, 0].tolist() == [0, 0, 1, -8, -126, 0]


def test_swiglu_backward_matches_autograd():
    g = torch.Generator().manual_seed(2)
    gu = torch.randn((5, 8), generator=g, dtype=torch.float64, requires_grad=True)
    dh = torch.randn((5, 4), generator=g, dtype=torch.float64)
    (want,) = torch.autograd.grad((torch.nn.functional.silu(gu[:, :4]) * gu[:, 4:] * dh).sum(), gu)
    assert np.allclose(O8.swiglu_bwd(dh.numpy(), gu.detach().numpy()), want.numpy(), rtol=1e-12)


def test_fp8_weight_encoder():
    w = torch.randn((2, 144, 272), generator=torch.Generator().manual_seed(1)) * 0.02
    w[1, 128:, 256:] = 0
    q, s = synth.quantize_fp8(w)
    assert q.shape == w.shape and s.shape == (2, 2, 3) and s[1, 1, 2] == 1.0
    v = O8.weight_values(q.view(torch.uint8).numpy(), s.numpy())
    block = np.repeat(np.repeat(s.numpy(), 128, 1)[:, :144], 128, 2)[:, :, :272]
    # half a step of e4m3 (2^-4 relative, 2^-10 of the scale below its normals), and one FP32 division
    assert np.all(np.abs(v - w.numpy()) <= (2.0 ** -4 + 2.0 ** -23) * np.abs(w.numpy()) + 2.0 ** -10 * block)


def test_accounting_of_fp8():
    assert accounting.fp8_bytes_per_param() == 1 + 1 / 4096
    assert accounting.saved_gu_bytes_per_row(2048, False) == 8192
    assert accounting.saved_gu_bytes_per_row(2048, True) == 4096 + 128


# ----------------------------------------------------------------------------- refusals of the C ABI

@pytest.fixture(scope="module")
def L():
    build.build()
    return moeq.lib()


P = 0x10000


def _router(**kw):
    a = dict(score=1, groups=1, topk_groups=1, group_top=1, renorm=1, scale=1.0)
    a.update(kw)
    return moeq.RouterC(a["score"], a["groups"], a["topk_groups"], a["group_top"], a["renorm"], a["scale"])


def _scored(L, T=64, E=8, k=2, d=256, C=8, x=None, logits=P, bias=None, ws=None, wsb=None, router=None, **kw):
    r = _router(**kw) if router is None else router
    return L.moe_route_scored(logits, bias, x, T, E, k, d, ctypes.byref(r), C, P, P, P, P, P, P, P, P, P, P,
                              ws, ctypes.byref(wsb) if wsb is not None else None, None)


def test_route_scored_refusals(L):
    wsb = ctypes.c_size_t(7)
    assert _scored(L, wsb=wsb) == 0 and wsb.value == 0
    assert _scored(L, wsb=wsb, T=4096, E=384, k=8) == 0 and wsb.value == 64 * 384 * 4
    assert _scored(L, T=4096, E=384, k=8) == 4                         # needs a workspace
    for kw in (dict(T=0), dict(E=0), dict(E=1025), dict(k=0), dict(k=9), dict(k=33, E=64), dict(C=0),
               dict(score=0), dict(score=3), dict(groups=0), dict(groups=3), dict(groups=33, E=66),
               dict(groups=4, topk_groups=5), dict(groups=4, topk_groups=0), dict(group_top=0),
               dict(group_top=3), dict(groups=4, topk_groups=1, k=3), dict(renorm=2),
               dict(scale=float("nan")), dict(scale=float("inf"))):
        assert _scored(L, wsb=wsb, **kw) == 1, kw
    assert _scored(L, T=1 << 31, wsb=wsb) == 3 and _scored(L, T=1 << 30, k=2, wsb=wsb) == 3
    assert _scored(L, logits=P + 4) == 2 and _scored(L, bias=P + 4) == 2
    assert _scored(L, logits=None) == 1 and _scored(L, x=P, d=12) == 1 and _scored(L, x=P + 2) == 2
    r = None
    assert L.moe_route_scored(P, None, None, 64, 8, 2, 0, r, 8, P, P, P, P, P, P, P, P, P, P, None, None, None) == 1


def test_router_gradient_refusals(L):
    def call(dg=P, lg=P, idx=P, T=4, E=8, k=2, out=P, g=None, **kw):
        return L.moe_route_scored_bwd(dg, g, lg, idx, T, E, k, ctypes.byref(_router(**kw)), out, None)
    for kw in (dict(dg=None), dict(lg=None), dict(idx=None), dict(out=None), dict(T=0), dict(E=1025), dict(k=9),
               dict(k=0), dict(score=5), dict(renorm=-1), dict(scale=float("inf"))):
        assert call(**kw) == 1, kw
    assert call(dg=P + 4) == 2 and call(out=P + 8) == 2 and call(g=P + 4) == 2 and call(T=1 << 31) == 3

    def comb(dy=P, rows=0x900000, inv=P, g=P, T=4, k=2, D=64, dr=0xA00000, dg=P):
        return L.moe_combine_bwd(dy, rows, inv, g, T, k, D, dr, dg, None)
    for kw in (dict(dy=None), dict(rows=None), dict(inv=None), dict(dr=None), dict(dg=None), dict(T=0), dict(k=0),
               dict(k=33), dict(D=4), dict(D=12), dict(dr=0x900000), dict(dr=0x900000 + 16), dict(dy=0xA00010)):
        assert comb(**kw) == 1, kw
    assert comb(dy=P + 8) == 2 and comb(g=P + 8) == 2 and comb(T=1 << 31) == 3


def test_fp8_refusals(L):
    q = lambda x=P, T=4, K=64, inv=None, k=1, o=P, s=P: L.moe_quantize_fp8_rows(x, T, K, inv, k, o, s, None)  # noqa: E731
    assert q(x=None) == 1 and q(o=None) == 1 and q(s=None) == 1 and q(T=0) == 1 and q(K=0) == 1
    assert q(k=2) == 1 and q(inv=P, k=33) == 1 and q(K=24) == 3 and q(T=1 << 31) == 3 and q(K=1 << 31) == 3
    assert q(x=P + 8) == 2 and q(inv=P + 4, k=2) == 2
    dq = lambda a=P, s=P, M=4, K=64, fmt=1, o=P: L.moe_dequantize_fp8_rows(a, s, M, K, fmt, o, None)  # noqa: E731
    assert dq(a=None) == 1 and dq(fmt=0) == 1 and dq(fmt=3) == 1 and dq(K=8) == 3 and dq(o=P + 8) == 2 and dq(M=0) == 1

    def gemm(bwd=False, a=P, s=P, M=64, E=4, N=256, K=512, wq=P, ws=P, g=None, epi=0, out=P, os=None, sv=None, ss=None):
        w = moeq.Fp8WeightC(wq, ws, E, N, K)
        gr = g if g is not None else moeq.GroupsC(P, P, P, P, P, E)
        if bwd:
            return L.moe_grouped_fp8_gemm_bwd_dx(a, s, M, ctypes.byref(w), ctypes.byref(gr), epi, sv, ss, out, os, None)
        return L.moe_grouped_fp8_gemm_fwd(a, s, M, ctypes.byref(w), ctypes.byref(gr), epi, out, os, sv, ss, None)
    for bwd in (False, True):
        for kw in (dict(a=None), dict(s=None), dict(M=0), dict(M=1 << 31), dict(E=0), dict(E=1025), dict(wq=None), dict(ws=None),
                   dict(out=None), dict(g=moeq.GroupsC(P, P, P, P, P, 5)), dict(g=moeq.GroupsC(None, P, P, P, P, 4)),
                   dict(epi=3), dict(epi=1 if bwd else 2), dict(os=P), dict(sv=P, ss=P)):
            assert gemm(bwd, **kw) == 1, (bwd, kw)
        assert gemm(bwd, K=520) == 3 and gemm(bwd, N=200) == 3
        assert gemm(bwd, a=P + 8) == 2 and gemm(bwd, s=P + 4) == 2 and gemm(bwd, wq=P + 1) == 2 and gemm(bwd, out=P + 2) == 2
    assert gemm(epi=1) == 1 and gemm(epi=1, os=P, sv=P) == 1 and gemm(epi=1, os=P, ss=P) == 1     # parts of the outputs missing
    assert gemm(epi=1, os=P, N=384) == 3 and gemm(epi=1, os=P + 4) == 2 and gemm(epi=1, os=P, sv=P + 8, ss=P) == 2
    assert gemm(True, epi=2, os=P) == 1 and gemm(True, epi=2, sv=P, ss=P) == 1
    assert gemm(True, epi=2, os=P, sv=P, ss=P, K=528) == 3 and gemm(True, epi=2, os=P, sv=P, ss=P + 4) == 2


def test_fp8_products_refuse_sizes_past_their_32_bit_indices(L):
    """Up to a tile past the last row or feature, and 2K in the SwiGLU backward, is indexed with 32 bits."""
    def gemm(bwd, M, N, K, epi=0):
        w, gr = moeq.Fp8WeightC(P, P, 1, N, K), moeq.GroupsC(P, P, P, P, P, 1)
        f = L.moe_grouped_fp8_gemm_bwd_dx if bwd else L.moe_grouped_fp8_gemm_fwd
        if bwd:
            return f(P, P, M, ctypes.byref(w), ctypes.byref(gr), epi, P if epi else None, P if epi else None, P, P if epi else None, None)
        return f(P, P, M, ctypes.byref(w), ctypes.byref(gr), epi, P, P if epi else None, None, None, None)
    top = 1 << 30
    for M in ((1 << 31) - 1, (1 << 31) - 128, (1 << 31) - 511):
        for bwd in (False, True):
            assert gemm(bwd, M, 16, 16) == 3
    for n in (top, 2 * top - 256):
        for bwd, epi in ((False, 0), (True, 0), (False, 1)):
            assert gemm(bwd, 64, n, 16, epi) == 3
        for bwd, epi in ((False, 0), (True, 0), (True, 2)):
            assert gemm(bwd, 64, 16, n, epi) == 3


def test_bindings_refuse_on_the_host():
    lg = torch.zeros((4, 8))
    spec = moeq.RouterSpec()
    with pytest.raises(ValueError):
        moeq.moe_route_scored(lg, None, 2, 8, spec)                     # CPU tensor
    with pytest.raises(ValueError):
        moeq.moe_route_scored(lg[0], None, 2, 8, spec)
    with pytest.raises(ValueError):
        moeq.RouterSpec(score="tanh").c()
    with pytest.raises(ValueError):
        moeq.moe_quantize_fp8_rows(torch.zeros((4, 32), dtype=torch.bfloat16))
    with pytest.raises(ValueError):
        moeq.moe_dequantize_fp8_rows(moeq.Fp8Rows(lg, lg))
    w = moeq.Fp8WeightT(torch.zeros((2, 16, 16), dtype=torch.float8_e4m3fn), torch.ones((2, 1, 1)))
    with pytest.raises(ValueError):
        moeq.moe_grouped_fp8_gemm_fwd(moeq.Fp8Rows(torch.zeros((4, 16), dtype=torch.float8_e4m3fn), torch.ones((1, 4))), w, None)
    with pytest.raises(ValueError):
        layer.route(lg, None, 2, 8, None, bias=torch.zeros(8))
    with pytest.raises(ValueError):
        layer.forward(lg, lg, w, w, 2, 8, adapter=torch.zeros(1))
    four = synth.QWeightT("int4", torch.zeros((2, 64, 32), dtype=torch.uint8), torch.ones((2, 2, 64), dtype=torch.bfloat16))
    for pair in ((w, four), (four, w)):                                 # one layer, one format
        with pytest.raises(ValueError, match="both"):
            layer.forward(lg, lg, *pair, 2, 8)
        with pytest.raises(ValueError, match="both"):
            layer.backward(dict(routing=None), lg, *pair)
        with pytest.raises(ValueError, match="both"):
            ep.expert_compute(lg, lg, *pair, 8)


def test_streams_and_devices_of_a_step(monkeypatch):
    """Without a GPU: a stream of another device than the tensors' is refused, and a step enters the tensors'
    device and the given stream before its first call."""
    class Stream:
        def __init__(self, index):
            self.device = torch.device("cuda", index)
    with pytest.raises(ValueError, match="stream"):
        moeq._on(torch.device("cuda", 0), Stream(1))
    with pytest.raises(ValueError, match="CUDA"):
        moeq._on(torch.device("cpu"), None)

    class Entered(Exception):
        pass
    seen = []

    def on(device, stream):
        seen.append((device, stream))
        raise Entered
    monkeypatch.setattr(moeq, "_on", on)
    lg = torch.zeros((4, 8))
    fp8 = moeq.Fp8WeightT(torch.zeros((2, 16, 16), dtype=torch.float8_e4m3fn), torch.ones((2, 1, 1)))
    four = synth.QWeightT("int4", torch.zeros((2, 64, 32), dtype=torch.uint8), torch.ones((2, 2, 64), dtype=torch.bfloat16))
    s = Stream(0)
    state = dict(routing=None, saved_gu=lg)
    for w in (fp8, four):
        for call in (lambda: layer.forward(lg, lg, w, w, 2, 8, stream=s), lambda: layer.backward(state, lg, w, w, stream=s)):
            with pytest.raises(Entered):
                call()
    for call in (lambda: layer.route(lg, lg, 2, 8, stream=s), lambda: layer.route(lg, lg, 2, 8, moeq.RouterSpec(), stream=s),
                 lambda: layer.up_projection(lg, lg, four, 2, 8, stream=s)):
        with pytest.raises(Entered):
            call()
    assert seen == [(lg.device, s)] * 7
    with pytest.raises(Entered):
        ep.expert_compute(lg, lg, fp8, fp8, 8)
    assert seen[-1] == (lg.device, None)
