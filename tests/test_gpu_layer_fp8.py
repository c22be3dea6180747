"""The new operators as they are used together: the MoE layer with a scored
router, on FP8 experts and on the 4-bit base, forward and backward, and the
expert-parallel phases with FP8 experts.

Every stage is compared with its float64 definition applied to the stage's
own inputs, so each has the tolerance of its operator (derived in
test_gpu_fp8.py and test_gpu_router.py) and nothing accumulates between them.
"""

import numpy as np
import pytest
import torch

from oracle import scored_fp8 as O8
from quantized_rl_fine_b200 import ep, layer, moeq, synth
from quantized_rl_fine_b200.configs import MoEConfig

from _common import f64
from test_gpu_fp8 import _check_quantized, _codes

pytestmark = pytest.mark.gpu

DEV = "cuda"
U = 2.0 ** -24


def _values(rows):
    if rows.scales.dtype == torch.uint8:
        return O8.rows_values(_codes(rows.q), 2.0 ** (rows.scales.cpu().numpy().astype(np.float64).T - 127), 32)
    return O8.rows_values(_codes(rows.q), f64(rows.scales).T, 128)


def _fp8_layer(E, d, f, T, seed):
    g = torch.Generator().manual_seed(seed)
    w = [moeq.Fp8WeightT(*synth.quantize_fp8(0.05 * torch.randn((E, n, k), generator=g))).to(DEV)
         for n, k in ((2 * f, d), (d, f))]
    x = torch.randn((T, d), generator=g).to(torch.bfloat16).to(DEV)
    dy = torch.randn((T, d), generator=g).to(torch.bfloat16).to(DEV)
    return g, x, dy, w[0], w[1]


def _wv(w):
    return O8.weight_values(_codes(w.q), f64(w.scales))


@pytest.mark.parametrize("E,k,d,f,T,score,renorm,pair", [(8, 2, 256, 128, 100, "sigmoid", True, "0"),
                                                        (5, 3, 272, 256, 37, "softmax", False, "0"),
                                                        (4, 2, 256, 128, 900, "sigmoid", True, "1"),
                                                        (16, 4, 128, 128, 1, "sigmoid", True, "0")])
def test_fp8_layer_step(E, k, d, f, T, score, renorm, pair, monkeypatch):
    monkeypatch.setenv("MOEQ_F8FORM", pair)
    g, x, dy, wg, wd = _fp8_layer(E, d, f, T, E + T)
    logits = torch.randn((T, E), generator=g).to(DEV)
    bias = (0.1 * torch.randn(E, generator=g)).to(DEV)
    spec = moeq.RouterSpec(score=score, renorm=renorm, scale=1.5)
    st = layer.forward(x, logits, wg, wd, k, 8, train=True, router=spec, bias=bias)
    bw = layer.backward(st, dy, wg, wd)
    assert moeq.moe_get_device_error() == 0
    r, M = st["routing"], T * k
    off = r.expert_offsets.cpu().numpy()
    inv, tok = r.inv_perm.cpu().numpy(), r.perm_token.cpu().numpy()
    topk, gates = O8.route_scored(f64(logits), k, score=score, renorm=renorm, scale=1.5, bias=f64(bias))
    assert np.array_equal(r.topk_idx.cpu().numpy(), topk)
    codes, e = O8.quantize_rows(f64(x)[tok])
    assert np.array_equal(_codes(st["a"].q), codes)
    gu, mag = O8.fp8_gemm(_values(st["a"]), _wv(wg), off)
    dl = (d + 8) * 2 * U * mag
    _check_quantized(st["saved_gu"], gu, dl, 32, M, 2 * f)
    h = O8.swiglu(gu)
    dh = 1.1 * (np.abs(gu[:, f:]) + dl[:, f:]) * dl[:, :f] + (np.abs(gu[:, :f]) + 1.1 * dl[:, :f]) * dl[:, f:]
    _check_quantized(st["h"], h, dh + 2.0 ** -18 * np.abs(h), 128, M, f)
    y, mag = O8.fp8_gemm(_values(st["h"]), _wv(wd), off)
    lim = (f + 8) * 2 * U * mag
    assert np.all(np.abs(f64(st["y_perm"]) - y) <= 2.0 ** -8 * (np.abs(y) + lim) + lim)
    # backward
    yp = f64(st["y_perm"])
    want_rows, want_g = O8.combine_bwd(f64(dy), yp, inv, f64(r.gates), k)
    magg = np.stack([(np.abs(f64(dy)) * np.abs(yp[inv.reshape(T, k)[:, j]])).sum(1) for j in range(k)], 1)
    assert np.all(np.abs(f64(bw["d_gates"]) - want_g) <= (d + 16) * U * magg)
    assert np.all(np.abs(f64(bw["dy_perm"]) - want_rows) <= 2.0 ** -8 * np.abs(want_rows))
    dl_want = O8.route_scored_bwd(f64(bw["d_gates"]), f64(logits), topk, score, renorm, 1.5)
    s = O8.scored_scores(f64(logits), score)
    w = np.take_along_axis(s, topk.astype(np.int64), 1)
    dw = np.abs(1.5 * f64(bw["d_gates"]))
    S = w.sum(1, keepdims=True)
    n = (dw + (dw * w).sum(1, keepdims=True) / S) / S if renorm else dw
    full = np.zeros((T, E))
    np.put_along_axis(full, topk.astype(np.int64), n, 1)
    lim = s * full + (s * (full * s).sum(1, keepdims=True) if score == "softmax" else 0)
    assert np.all(np.abs(f64(bw["d_logits"]) - dl_want) <= 256 * U * lim + 2.0 ** -120)
    dq, e = O8.quantize_rows(f64(bw["dy_perm"]))
    dhv, mag = O8.fp8_gemm(O8.rows_values(dq, 2.0 ** e.astype(np.float64), 128), _wv(wd), off, True)
    dd = (d + 8) * 2 * U * mag
    ck = _values(st["saved_gu"])
    want = O8.swiglu_bwd(dhv, ck)
    size = np.concatenate([np.abs(ck[:, f:]) * (1 + np.abs(ck[:, :f])), np.abs(ck[:, :f])], 1)
    lim = size * np.tile(dd, 2) + 2.0 ** -18 * size * np.tile(np.abs(dhv) + dd, 2)
    _check_quantized(bw["dgu"], want, lim + 2.0 ** -8 * (np.abs(want) + lim), 128, M, 2 * f)
    dx, mag = O8.fp8_gemm(_values(bw["dgu"]), _wv(wg), off, True)
    lim = (2 * f + 8) * 2 * U * mag
    assert np.all(np.abs(f64(bw["dx_perm"]) - dx) <= 2.0 ** -8 * (np.abs(dx) + lim) + lim)
    dxt = f64(bw["dx_perm"])[inv].reshape(T, k, d)
    assert np.all(np.abs(f64(bw["dx"]) - dxt.sum(1)) <= 2.0 ** -8 * np.abs(dxt.sum(1)) + k * U * 2 * np.abs(dxt).sum(1))


def test_fp8_layer_without_training_keeps_nothing():
    _, x, dy, wg, wd = _fp8_layer(4, 128, 128, 20, 1)
    logits = torch.randn((20, 4), generator=torch.Generator().manual_seed(1)).to(DEV)
    a = layer.forward(x, logits, wg, wd, 2, 8)
    b = layer.forward(x, logits, wg, wd, 2, 8, train=True)
    assert a["saved_gu"] is None and torch.equal(a["y"], b["y"])
    assert b["saved_gu"].nbytes() == 20 * 2 * (256 + 8)
    with pytest.raises(ValueError):
        layer.backward(a, dy, wg, wd)
    bw = layer.backward(b, dy, wg, wd)                       # gates are constants without a router
    assert bw["d_gates"] is None and bw["d_logits"] is None
    same = moeq.moe_unpermute_combine(dy, b["routing"], b["routing"].gates, 20, mode=1)
    assert torch.equal(bw["dy_perm"], same)


@pytest.mark.parametrize("fmt", ["int4", "mxfp4"])
def test_scored_router_on_the_4_bit_layer(fmt):
    """The router's calls in front of and behind the 4-bit products: same rows, same products, and its gradients."""
    cfg = MoEConfig("t", E=8, k=2, d=256, f=128, T=70, fmt=fmt, swiglu=True, logits="normal", adapter=True, train=True, seed=5)
    wl = synth.make_workload(cfg, "cpu")
    w_gu, w_d = wl["w_gu"].to(DEV), wl["w_d"].to(DEV)
    x, lg, dy, R = (wl[n].to(DEV) for n in ("x", "logits", "dy", "adapter"))
    plain = layer.forward(x, lg, w_gu, w_d, 2, 8, adapter=R, train=True)
    st = layer.forward(x, lg, w_gu, w_d, 2, 8, adapter=R, train=True, router=moeq.RouterSpec())
    # softmax scores renormalised over the selection are the softmax over the selected logits
    assert torch.equal(st["routing"].perm_token, plain["routing"].perm_token)
    assert torch.equal(st["y_perm"], plain["y_perm"])
    g0, g1 = f64(plain["routing"].gates), f64(st["routing"].gates)
    assert np.all(np.abs(g0 - g1) <= 96 * U * g0)
    bw = layer.backward(st, dy, w_gu, w_d, adapter=R)
    ref = layer.backward(plain, dy, w_gu, w_d, adapter=R)
    assert ref["d_logits"] is None and bw["d_adapter"].shape == ref["d_adapter"].shape
    inv = st["routing"].inv_perm.cpu().numpy()
    yp = f64(st["y_perm"])
    _, want = O8.combine_bwd(f64(dy), yp, inv, g1, 2)
    mag = np.stack([(np.abs(f64(dy)) * np.abs(yp[inv.reshape(70, 2)[:, j]])).sum(1) for j in range(2)], 1)
    assert np.all(np.abs(f64(bw["d_gates"]) - want) <= (256 + 16) * U * mag)
    assert np.abs(f64(bw["d_logits"]).sum(1)).max() <= 256 * U * np.abs(f64(bw["d_gates"])).sum(1).max()


def test_expert_parallel_phases_with_fp8_experts():
    """Two ranks' phases one after the other on one GPU, exchanged by copies: the layer's own result, bit for bit."""
    E, k, d, f, T, W = 8, 2, 256, 128, 48, 2
    g, x, _, wg, wd = _fp8_layer(E, d, f, T * W, 11)
    logits = torch.randn((T * W, E), generator=g).to(DEV)
    spec, bias = moeq.RouterSpec(score="sigmoid", groups=2, topk_groups=2, group_top=2), (0.1 * torch.randn(E, generator=g)).to(DEV)
    want = layer.forward(x, logits, wg, wd, k, 8, router=spec, bias=bias)["y"]
    dsp = [ep.route(x[s * T:(s + 1) * T], logits[s * T:(s + 1) * T], k, 8, W, spec, bias) for s in range(W)]
    n = E // W
    back = [[None] * W for _ in range(W)]
    for rank in range(W):
        counts = torch.stack([s.counts[rank * n:(rank + 1) * n] for s in dsp])
        rows = torch.cat([torch.split(s.routing.x_perm, s.send)[rank] for s in dsp])
        loc = [moeq.Fp8WeightT(w.q[rank * n:(rank + 1) * n].contiguous(), w.scales[rank * n:(rank + 1) * n].contiguous()) for w in (wg, wd)]
        out = ep.expert_compute(rows, counts.contiguous(), loc[0], loc[1], 8)
        for s, piece in enumerate(torch.split(out, [dsp[s].send[rank] for s in range(W)])):
            back[s][rank] = piece
    got = torch.cat([ep.combine(dsp[s], torch.cat(back[s]), T) for s in range(W)])
    assert moeq.moe_get_device_error() == 0
    assert torch.equal(got, want)


def _pool_stream(t):
    """The stream whose memory pool holds the tensor."""
    p = t.data_ptr()
    for seg in torch.cuda.memory_snapshot():
        if seg["address"] <= p < seg["address"] + seg["total_size"]:
            return seg["stream"]
    raise AssertionError("not in a pool")


@pytest.mark.parametrize("kind", ["fp8", "int4", "int4_adapter", "up"])
def test_a_step_on_another_stream_lives_in_that_streams_memory(kind):
    """Whatever a step on a given stream writes comes from that stream's pool: memory of the current stream's
    pool may still be in use there. And the results are those of the current stream."""
    E, k, d, f, T = 4, 2, 128, 128, 50
    if kind == "fp8":
        g, x, dy, wg, wd = _fp8_layer(E, d, f, T, 3)
        lg, R = torch.randn((T, E), generator=g).to(DEV), None
    else:
        cfg = MoEConfig("t", E=E, k=k, d=d, f=f, T=T, fmt="int4", swiglu=True, logits="normal", adapter=True, train=True, seed=6)
        wl = synth.make_workload(cfg, "cpu")
        wg, wd = wl["w_gu"].to(DEV), wl["w_d"].to(DEV)
        x, lg, dy, R = (wl[n].to(DEV) for n in ("x", "logits", "dy", "adapter"))
        R = R if kind == "int4_adapter" else None

    def step(stream=None):
        if kind == "up":
            st = layer.up_projection(x, lg, wg, k, 8, stream=stream)
            return dict(out=st["out"], a=st["a"], perm=st["routing"].perm_token)
        st = layer.forward(x, lg, wg, wd, k, 8, adapter=R, train=True, stream=stream, router=moeq.RouterSpec())
        bw = layer.backward(st, dy, wg, wd, adapter=R, stream=stream)
        outs = {n: t for n, t in {**st, **bw}.items() if isinstance(t, torch.Tensor) and n not in ("x", "logits", "a", "a_rows")}
        return dict(outs, perm=st["routing"].perm_token)
    want = {n: t.clone() for n, t in step().items()}
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = step(side)
    side.synchronize()
    assert moeq.moe_get_device_error() == 0
    for n, t in want.items():
        assert torch.equal(got[n], t), n
        assert _pool_stream(got[n]) == side.cuda_stream, n


@pytest.mark.parametrize("kind", ["fp8", "int4"])
def test_a_captured_step_replays_on_new_inputs(kind):
    """Forward and backward of a layer with a scored router in one graph: replayed on other inputs it gives the bits
    of the calls themselves, with a second graph of the same layer and eager steps in between."""
    E, k, d, f, T = 8, 2, 128, 128, 1100
    g, x0, dy0, wg, wd = _fp8_layer(E, d, f, T, 21)
    if kind == "int4":
        cfg = MoEConfig("t", E=E, k=k, d=d, f=f, T=T, fmt="int4", swiglu=True, logits="normal", adapter=False, train=True, seed=7)
        wl = synth.make_workload(cfg, "cpu")
        wg, wd = wl["w_gu"].to(DEV), wl["w_d"].to(DEV)
    spec, bias = moeq.RouterSpec(score="sigmoid", groups=4, topk_groups=2, group_top=2), (0.1 * torch.randn(E, generator=g)).to(DEV)
    sets = [(x0, torch.randn((T, E), generator=g).to(DEV), dy0)]
    sets.append(tuple(torch.randn(t.shape, generator=g).to(t.dtype).to(DEV) for t in sets[0]))

    def step(x, lg, dy):
        st = layer.forward(x, lg, wg, wd, k, 8, train=True, router=spec, bias=bias)
        bw = layer.backward(st, dy, wg, wd)
        return st["y"], st["routing"].gates, bw["dx"], bw["d_logits"], bw["d_gates"]
    want = [[t.clone() for t in step(*s)] for s in sets]
    graphs = []
    for _ in range(2):
        ins = [t.clone() for t in sets[0]]
        graph = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph):
            outs = step(*ins)
        graphs.append((graph, ins, outs))
    for i, (a, b) in ((0, (1, 0)), (1, (0, 1))):
        for (graph, ins, _), s in zip(graphs, (a, b)):
            for t, v in zip(ins, sets[s]):
                t.copy_(v)
            graph.replay()
        assert all(torch.equal(p, q) for p, q in zip(step(*sets[i]), want[i]))
        for (_, _, outs), s in zip(graphs, (a, b)):
            assert all(torch.equal(p, q) for p, q in zip(outs, want[s]))
    assert moeq.moe_get_device_error() == 0
