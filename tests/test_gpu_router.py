"""moe_route_scored, moe_route_scored_bwd and moe_combine_bwd against their
float64 definitions.

Tolerances. Gates: a score is an exponential and a division in FP32 (expf:
2 ulp, division and the sum of at most 1024 positive terms in warp order: 40
rounding steps at most), so 64 * 2^-24 relative. d_gates: D products summed in
FP32, every rounding at most 2^-24 of the sum of magnitudes: (D + 16) * 2^-24 *
sum |dy * row| bounds any order. d_rows: one BF16 rounding, 2^-8 relative.
d_logits: built from numbers c_i s_i / S with the relative error of the
scores, 64 * 2^-24 each; the subtraction makes that an error relative to the
magnitudes |dw| + sum |dw| s / S, as derived beside the check.
"""

import numpy as np
import pytest
import torch

from oracle import scored_fp8 as O8
import oracle as O
from quantized_rl_fine_b200 import moeq

from _common import f64

pytestmark = pytest.mark.gpu

DEV = "cuda"
U = 2.0 ** -24


def _spec(**kw):
    return moeq.RouterSpec(**kw)


def _check(logits, k, spec, bias=None, x=None, chunk=8, r=None):
    if r is None:
        r = moeq.moe_route_scored(logits.to(DEV), None if x is None else x.to(DEV), k, chunk, spec,
                                  bias=None if bias is None else bias.to(DEV))
    kw = dict(score=spec.score, groups=spec.groups, topk_groups=spec.topk_groups,
              group_top=spec.group_top, renorm=spec.renorm, scale=spec.scale)
    topk, gates = O8.route_scored(logits.numpy(), k, bias=None if bias is None else bias.numpy(), **kw)
    E = logits.shape[1]
    assert np.array_equal(r.topk_idx.cpu().numpy(), topk)
    # 64 rounding steps on every factor of a gate; below 2^-126 absolute
    assert np.all(np.abs(f64(r.gates) - gates) <= 64 * U * np.abs(gates) + 2.0 ** -126)
    g = O.group_by_expert(topk, E, chunk)
    A, nch = int(r.num_active.item()), int(r.num_chunks.item())
    assert np.array_equal(r.expert_offsets.cpu().numpy(), g.offsets)
    assert A == g.num_active and nch == g.num_chunks
    assert np.array_equal(r.active.cpu().numpy()[:A], g.active)
    assert np.array_equal(r.chunk_offsets.cpu().numpy()[:nch + 1], g.chunk_offsets)
    assert np.array_equal(r.perm_token.cpu().numpy(), g.perm_token)
    assert np.array_equal(r.inv_perm.cpu().numpy(), g.inv_perm)
    if x is not None:
        xp = r.x_perm.cpu().view(torch.int16).numpy()
        assert np.array_equal(xp, x.view(torch.int16).numpy()[g.perm_token])
    return r, topk


CASES = [
    # T, E, k, spec, bias
    (1, 1, 1, dict(score="softmax"), False),
    (1, 384, 8, dict(score="sigmoid", groups=8, topk_groups=4, group_top=2, scale=2.5), True),
    (37, 5, 3, dict(score="softmax", renorm=False), False),
    (64, 8, 2, dict(score="sigmoid", renorm=False, scale=0.5), True),
    (130, 384, 8, dict(score="softmax", groups=8, topk_groups=3, group_top=1), False),
    (100, 160, 6, dict(score="softmax", groups=8, topk_groups=3, group_top=1, renorm=False), False),
    (257, 64, 32, dict(score="sigmoid", groups=2, topk_groups=1, group_top=2), False),
    (33, 96, 4, dict(score="sigmoid", groups=32, topk_groups=2, group_top=2), True),
    (90, 21, 3, dict(score="softmax", groups=7, topk_groups=1, group_top=2), True),
    (40, 12, 12, dict(score="sigmoid", groups=3, topk_groups=3, group_top=2), True),
    (1500, 256, 8, dict(score="sigmoid", groups=8, topk_groups=4, group_top=2, scale=2.5), True),
    (1100, 48, 4, dict(score="softmax", groups=6, topk_groups=2, group_top=1), True),
    (65, 1024, 8, dict(score="sigmoid", groups=16, topk_groups=4, group_top=2), True),
    (50, 1000, 5, dict(score="softmax", renorm=False), True),
]


@pytest.mark.parametrize("T,E,k,kw,with_bias", CASES)
def test_route_scored_against_definition(T, E, k, kw, with_bias):
    g = torch.Generator().manual_seed(T * 31 + E)
    logits = torch.randn((T, E), generator=g)
    bias = 0.1 * torch.randn(E, generator=g) if with_bias else None
    x = torch.randn((T, 24), generator=g).to(torch.bfloat16)
    _check(logits, k, _spec(**kw), bias, x)


@pytest.mark.parametrize("T,E,k,kw,with_bias", CASES[1:])
def test_exact_ties_go_to_the_lower_id(T, E, k, kw, with_bias):
    """Few distinct logits and biases: most selections and groups are decided by ties."""
    g = torch.Generator().manual_seed(T + 7 * E)
    logits = torch.randint(-1, 2, (T, E), generator=g).float()
    bias = torch.randint(0, 2, (E,), generator=g).float() if with_bias else None
    _check(logits, k, _spec(**kw), bias)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("groups,topk_groups,group_top", [(1, 1, 1), (4, 2, 1), (4, 2, 2)])
@pytest.mark.parametrize("with_bias", [False, True])
def test_masked_experts(score, groups, topk_groups, group_top, with_bias):
    T, E, k = 70, 24, 6
    g = torch.Generator().manual_seed(5)
    logits = torch.randn((T, E), generator=g)
    logits[0] = -float("inf")                                # nothing left
    logits[1, 1:] = -float("inf")                            # one expert left
    logits[2] = float("nan")
    logits[3, ::2] = float("nan")
    logits[4, :20] = -float("inf")                           # fewer than k left in one group
    logits[5] = torch.finfo(torch.float32).min               # the type's lowest value is a number
    logits[6, 3:] = torch.finfo(torch.float32).min
    logits[7, 5] = float("inf")
    logits[8] = -200.0                                       # sigmoid underflows in FP32
    logits[9, :] = 60.0                                      # sigmoid saturates
    logits[9, 7] = 90.0
    logits[10:40][torch.rand((30, E), generator=g) < 0.6] = -float("inf")
    bias = 0.1 * torch.randn(E, generator=g) if with_bias else None
    if with_bias:
        bias[2], bias[9] = -float("inf"), float("nan")
    spec = _spec(score=score, groups=groups, topk_groups=topk_groups, group_top=group_top)
    r, topk = _check(logits, k, spec, bias)
    assert all(len(set(row)) == k for row in r.topk_idx.cpu().tolist())
    d = moeq.moe_route_scored_bwd(torch.ones((T, k), device=DEV), logits.to(DEV), r, spec)
    assert torch.isfinite(d).all()
    assert not d.cpu()[0].any() and not d.cpu()[2].any()


def test_keys_that_differ_below_single_precision():
    """Scores closer than FP32 resolves: the order is the one of the 64-bit keys."""
    E, k = 64, 8
    g = torch.Generator().manual_seed(3)
    bias = torch.zeros(E)
    # logits one FP32 step apart around 12: their sigmoids differ by 1e-11
    base = torch.full((E,), 12.0)
    step = torch.nextafter(base, torch.full((E,), 100.0)) - base
    logits = torch.stack([base + step * torch.randperm(E, generator=g).float() for _ in range(40)])
    for spec in (_spec(score="sigmoid"), _spec(score="softmax"),
                 _spec(score="sigmoid", groups=8, topk_groups=4, group_top=2)):
        _check(logits, k, spec, bias)
        _check(logits, k, spec, None)
    # bias and score that cancel: keys near 0 from numbers near 0.5
    bias = -torch.sigmoid(torch.linspace(-1, 1, E))
    logits = torch.linspace(-1, 1, E).repeat(20, 1) + 1e-6 * torch.randn((20, E), generator=g)
    _check(logits, k, _spec(score="sigmoid"), bias)


@pytest.mark.parametrize("T,E,k,score,renorm,scale", [
    (1, 1, 1, "softmax", False, 1.0), (1, 384, 8, "sigmoid", True, 2.5),
    (131, 64, 4, "softmax", False, 1.0), (77, 21, 5, "softmax", True, 1.5),
    (300, 1000, 32, "sigmoid", False, 2.5), (64, 100, 2, "sigmoid", True, 1.0)])
def test_router_gradient(T, E, k, score, renorm, scale):
    g = torch.Generator().manual_seed(T + E)
    logits = 2 * torch.randn((T, E), generator=g)
    dg = torch.randn((T, k), generator=g)
    spec = _spec(score=score, renorm=renorm, scale=scale)
    r = moeq.moe_route_scored(logits.to(DEV), None, k, 8, spec)
    out = torch.full((T, E), float("nan"), device=DEV)
    got = f64(moeq.moe_route_scored_bwd(dg.to(DEV), logits.to(DEV), r, spec, out=out))
    topk = r.topk_idx.cpu().numpy()
    want = O8.route_scored_bwd(dg.numpy(), logits.numpy(), topk, score, renorm, scale)
    # Magnitudes of what is subtracted: with n = |dw_j| + sum |dw| s / S (over S for
    # renorm) an error of 64 U of every s moves ds by at most 128 U * n, and the
    # result by s * (that + the 64 U of s itself on |ds|), the softmax term likewise.
    s = O8.scored_scores(logits.numpy(), score)
    w = np.take_along_axis(s, topk.astype(np.int64), 1)
    dw = np.abs(scale * dg.numpy().astype(np.float64))
    if renorm:
        S = w.sum(1, keepdims=True)
        n = (dw + (dw * w).sum(1, keepdims=True) / S) / S
    else:
        n = dw
    full = np.zeros((T, E))
    np.put_along_axis(full, topk.astype(np.int64), n, 1)
    lim = s * full
    if score == "softmax":
        lim = lim + s * (full * s).sum(1, keepdims=True)
    assert np.all(np.abs(got - want) <= 256 * U * lim + 2.0 ** -120)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
def test_router_gradient_against_differences(score, renorm):
    """The definition's own gates, moved by small steps of the logits, in float64."""
    T, E, k, h = 6, 12, 3, 1e-5
    g = torch.Generator().manual_seed(9)
    logits = torch.randn((T, E), generator=g)
    dg = torch.randn((T, k), generator=g)
    spec = _spec(score=score, renorm=renorm, scale=1.5)
    r = moeq.moe_route_scored(logits.to(DEV), None, k, 8, spec)
    got = f64(moeq.moe_route_scored_bwd(dg.to(DEV), logits.to(DEV), r, spec))
    idx = r.topk_idx.cpu().numpy().astype(np.int64)

    def loss(x):
        s = O8.scored_scores(x, score)
        w = np.take_along_axis(s, idx, 1)
        if renorm:
            w = w / w.sum(1, keepdims=True)
        return (1.5 * w * dg.numpy().astype(np.float64)).sum(1)

    x = f64(logits)
    num = np.zeros((T, E))
    for e in range(E):
        d = np.zeros((1, E))
        d[0, e] = h
        num[:, e] = (loss(x + d) - loss(x - d)) / (2 * h)
    # second-order differences of functions with derivatives of order one: h^2, and FP32 results
    assert np.abs(got - num).max() <= 10 * h * h + 256 * U * np.abs(dg.numpy()).sum(1).max() * 1.5


@pytest.mark.parametrize("T,E,k,D,with_gates", [(1, 4, 1, 8, True), (5, 8, 3, 72, True),
                                                (131, 64, 4, 2048, True), (33, 40, 32, 264, True),
                                                (64, 12, 9, 4104, False), (20, 32, 16, 7168, True)])
def test_combine_bwd(T, E, k, D, with_gates):
    g = torch.Generator().manual_seed(T + D)
    logits = torch.randn((T, E), generator=g)
    dy = torch.randn((T, D), generator=g).to(torch.bfloat16)
    rows = torch.randn((T * k, D), generator=g).to(torch.bfloat16)
    r = moeq.moe_route_scored(logits.to(DEV), None, k, 8, _spec())
    if not with_gates:
        r.gates = None
    out = torch.full((T * k, D), float("nan"), dtype=torch.bfloat16, device=DEV)
    d_rows, d_gates = moeq.moe_combine_bwd(dy.to(DEV), rows.to(DEV), r, out=out)
    inv = r.inv_perm.cpu().numpy()
    gates = None if r.gates is None else f64(r.gates)
    wr, wg = O8.combine_bwd(f64(dy), f64(rows), inv, gates, k)
    mag = np.stack([[np.abs(f64(dy[t]) * f64(rows[int(inv[t * k + j])])).sum() for j in range(k)]
                    for t in range(T)])
    assert np.all(np.abs(f64(d_gates) - wg) <= (D + 16) * U * mag)
    assert np.all(np.abs(f64(d_rows) - wr) <= 2.0 ** -8 * np.abs(wr))
    # the same bits as the existing scatter
    assert torch.equal(d_rows, moeq.moe_unpermute_combine(dy.to(DEV), r, r.gates, T, mode=1))
    again = moeq.moe_combine_bwd(dy.to(DEV), rows.to(DEV), r)
    assert torch.equal(again[0], d_rows) and torch.equal(again[1], d_gates)


def test_router_chain_captured_and_on_another_stream():
    """Forward, combine backward and router backward captured into a graph and replayed with
    new inputs, and the same calls on a stream of their own."""
    T, E, k, D = 1200, 64, 4, 64
    spec = _spec(score="sigmoid", groups=4, topk_groups=2, group_top=2)
    g = torch.Generator().manual_seed(1)
    sets = [(torch.randn((T, E), generator=g).to(DEV), torch.randn((T, D), generator=g).to(torch.bfloat16).to(DEV),
             torch.randn((T * k, D), generator=g).to(torch.bfloat16).to(DEV)) for _ in range(2)]
    bias = (0.1 * torch.randn(E, generator=g)).to(DEV)

    def chain(lg, dy, rows, stream=None):
        r = moeq.moe_route_scored(lg, None, k, 8, spec, bias=bias, stream=stream)
        d_rows, d_gates = moeq.moe_combine_bwd(dy, rows, r, stream=stream)
        return r.topk_idx, r.gates, d_rows, d_gates, moeq.moe_route_scored_bwd(d_gates, lg, r, spec, stream=stream)

    want = [[t.clone() for t in chain(*s)] for s in sets]
    lg, dy, rows = (t.clone() for t in sets[0])
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        outs = chain(lg, dy, rows)
    for s, w in zip(sets[::-1], want[::-1]):
        for dst, src in zip((lg, dy, rows), s):
            dst.copy_(src)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, w))
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = chain(*sets[1], stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want[1]))


@pytest.mark.parametrize("E,groups", [(1024, 32), (992, 31), (62, 31), (64, 32), (1000, 8), (513, 27)])
@pytest.mark.parametrize("T", [1, 29, 40, 1100])
def test_many_groups(E, groups, T):
    """Group scratch from a few bytes to more than a block holds for 32 warps; both table paths and the one-launch one."""
    g = torch.Generator().manual_seed(E + T)
    logits = torch.randn((T, E), generator=g)
    bias = 0.1 * torch.randn(E, generator=g)
    for gt, b in ((1, None), (2, bias)):
        _check(logits, 4, _spec(score="sigmoid", groups=groups, topk_groups=5, group_top=gt), b)


@pytest.mark.parametrize("T", [1025, 1056, 1057, 1089, 4736, 4737, 9001])
@pytest.mark.parametrize("E,groups", [(64, 1), (384, 8)])
def test_many_tokens(T, E, groups):
    """One and two blocks per histogram of 64 tokens, blocks without tokens among them."""
    g = torch.Generator().manual_seed(E + T)
    logits = torch.randn((T, E), generator=g)
    _check(logits, 6, _spec(score="sigmoid", groups=groups, topk_groups=max(1, groups // 2)), 0.1 * torch.randn(E, generator=g))


@pytest.mark.parametrize("score,spread", [("sigmoid", 2e-5), ("sigmoid", 2e-6), ("softmax", 2e-4), ("softmax", 2e-5)])
@pytest.mark.parametrize("groups,group_top", [(1, 1), (8, 1), (8, 2)])
def test_keys_within_the_errors_of_single_precision(score, spread, groups, group_top):
    """Keys so close that single precision settles some selections, a few need 64 bits for their candidates and others for all."""
    T, E = 1500, 256
    g = torch.Generator().manual_seed(int(spread * 1e7) + groups + group_top)
    logits = 0.5 + spread * torch.randn((T, E), generator=g)
    bias = (0.25 if score == "sigmoid" else 1 / 256) * spread * torch.randn(E, generator=g)
    bias[::2] *= 40.0                                   # and gaps between some of them
    _check(logits, 8, _spec(score=score, groups=groups, topk_groups=max(1, groups // 2), group_top=group_top), bias)


def test_infinite_and_huge_biases():
    T, E, k = 40, 48, 5
    g = torch.Generator().manual_seed(12)
    logits = torch.randn((T, E), generator=g)
    bias = 0.1 * torch.randn(E, generator=g)
    bias[3] = float("inf")
    for kw in (dict(), dict(groups=4, topk_groups=2, group_top=2)):
        _check(logits, k, _spec(score="sigmoid", **kw), bias)
        _check(logits, k, _spec(score="softmax", **kw), bias * 1e30)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
def test_experts_masked_by_the_bias_get_no_gradient(score, renorm):
    """A bias of -inf leaves fewer than k experts: the slots filled up have gate 0, and neither they nor
    their scores enter the gradient."""
    T, E, k = 30, 6, 4
    g = torch.Generator().manual_seed(2)
    logits = torch.randn((T, E), generator=g)
    bias = torch.tensor([0.0, -float("inf"), 0.1, -float("inf"), -float("inf"), -0.2])
    dg = torch.randn((T, k), generator=g)
    spec = _spec(score=score, renorm=renorm)
    r, topk = _check(logits, k, spec, bias)
    assert np.all(f64(r.gates)[:, 3] == 0) and np.all(f64(r.gates)[:, :3] > 0)
    got = f64(moeq.moe_route_scored_bwd(dg.to(DEV), logits.to(DEV), r, spec))
    want = O8.route_scored_bwd(dg.numpy(), logits.numpy(), topk, score, renorm, 1.0, gates=f64(r.gates))
    # scores at most 1, the sum of three of them at least 1e-3 here: 256 U of |dg| / 1e-3
    assert np.abs(got - want).max() <= 256 * U * np.abs(dg.numpy()).sum(1).max() * (1e3 if renorm else 1)
    r.gates = None                                     # without the gates the scores count
    assert not np.allclose(f64(moeq.moe_route_scored_bwd(dg.to(DEV), logits.to(DEV), r, spec)), want, rtol=1e-3)


def test_combine_bwd_skips_slots_that_are_no_rows():
    T, E, k, D = 6, 8, 2, 64
    g = torch.Generator().manual_seed(4)
    r = moeq.moe_route_scored(torch.randn((T, E), generator=g).to(DEV), None, k, 8, _spec())
    dy = torch.randn((T, D), generator=g).to(torch.bfloat16).to(DEV)
    rows = torch.randn((T * k, D), generator=g).to(torch.bfloat16).to(DEV)
    want, wg = moeq.moe_combine_bwd(dy, rows, r)
    lost = r.inv_perm[5].item(), r.inv_perm[8].item()
    r.inv_perm = r.inv_perm.clone()
    r.inv_perm[5], r.inv_perm[8] = -1, T * k
    out = torch.full((T * k, D), 7.0, dtype=torch.bfloat16, device=DEV)
    got, gg = moeq.moe_combine_bwd(dy, rows, r, out=out)
    keep = [p for p in range(T * k) if p not in lost]
    assert torch.equal(got[keep], want[keep]) and bool((got[list(lost)] == 7.0).all())
    wg = wg.clone().view(-1)
    wg[5] = wg[8] = 0
    assert torch.equal(gg.view(-1), wg)


def test_calls_from_several_host_threads():
    """Different sizes at once, each thread on a stream of its own."""
    import threading
    jobs = [(20, 384, 8), (3000, 256, 8), (700, 1024, 32), (1, 64, 4)]
    g = torch.Generator().manual_seed(8)
    data = [(torch.randn((T, E), generator=g).to(DEV), (0.1 * torch.randn(E, generator=g)).to(DEV),
             _spec(score="sigmoid", groups=gr, topk_groups=2, group_top=2)) for T, E, gr in jobs]
    want = [moeq.moe_route_scored(lg, None, 4, 8, sp, bias=b) for lg, b, sp in data]
    torch.cuda.synchronize()
    bad = []

    def work(i):
        s = torch.cuda.Stream()
        for _ in range(20):
            r = moeq.moe_route_scored(data[i][0], None, 4, 8, data[i][2], bias=data[i][1], stream=s)
            s.synchronize()
            if not (torch.equal(r.topk_idx, want[i].topk_idx) and torch.equal(r.inv_perm, want[i].inv_perm)):
                bad.append(i)
    ts = [threading.Thread(target=work, args=(i,)) for i in range(len(jobs))]
    for t in ts:
        t.start()
    for t in ts:
        t.join()
    assert not bad


def test_refusals_of_wrong_tensors():
    lg = torch.zeros((4, 8), device=DEV)
    spec = _spec()
    bad = [dict(logits=lg.half()), dict(logits=lg.t()), dict(logits=lg[:, ::2]), dict(bias=torch.zeros(7, device=DEV)),
           dict(bias=torch.zeros(8)), dict(x=torch.zeros((4, 16), device=DEV)), dict(x=torch.zeros((3, 16), device=DEV, dtype=torch.bfloat16))]
    for kw in bad:
        a = dict(logits=lg, x=None, bias=None)
        a.update(kw)
        with pytest.raises(ValueError):
            moeq.moe_route_scored(a["logits"], a["x"], 2, 8, spec, bias=a["bias"])
    with pytest.raises(moeq.MoeError):
        moeq.moe_route_scored(lg, None, 9, 8, spec)
    r = moeq.moe_route_scored(lg, None, 2, 8, spec)
    with pytest.raises(ValueError):
        moeq.moe_route_scored(torch.zeros((5, 8), device=DEV), None, 2, 8, spec, out=r)
    with pytest.raises(ValueError):
        moeq.moe_route_scored_bwd(torch.zeros((4, 3), device=DEV), lg, r, spec)
    rows = torch.zeros((8, 16), dtype=torch.bfloat16, device=DEV)
    with pytest.raises(moeq.MoeError):
        moeq.moe_combine_bwd(rows[:4], rows, r, out=rows)              # in place
    with pytest.raises(ValueError):
        moeq.moe_combine_bwd(rows[:3], rows, r)


# ----------------------------------------------------------------------------- k = 32 with a bias

def test_the_first_expert_left_out_of_32_is_compared_too():
    """31 experts far ahead by their bias; the 32nd place lies between logits 12 and the next float, whose
    sigmoids are equal in single precision and differ by 7e-12 in 64 bits: the larger one, of the higher id, wins."""
    E, k = 40, 32
    logits = torch.linspace(-3, 3, E).repeat(5, 1)
    logits[:, 31] = 12.0
    logits[:, 32] = torch.nextafter(torch.tensor(12.0), torch.tensor(13.0))
    bias = torch.full((E,), -1.0)
    bias[:31], bias[31:33] = 2.0, 0.0
    r, topk = _check(logits, k, _spec(score="sigmoid"), bias)
    assert np.all(topk[:, 31] == 32)


@pytest.mark.parametrize("E,groups", [(33, 1), (40, 1), (64, 1), (65, 1), (384, 1), (384, 8), (1024, 4)])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("k", [31, 32])
def test_near_ties_around_the_last_of_32_places(E, groups, score, k):
    """Some experts ahead by a clear margin (none to 31), all others within a few floats of one another: the
    last places are decided in 64 bits, with the candidates filling the warp's 32 lanes or more."""
    T = 64
    g = torch.Generator().manual_seed(E + k + groups)
    step = 2.0 ** -23 if score == "softmax" else 2.0 ** -20
    base = 1.0 if score == "softmax" else 12.0
    logits = base + step * torch.stack([torch.randperm(E, generator=g) for _ in range(T)]).float()
    bias = torch.zeros(E)
    for i, e in enumerate(torch.randperm(E, generator=g)[:31].tolist()):
        bias[e] = 2.0 + 0.01 * i
    spec = _spec(score=score, groups=groups, topk_groups=groups)
    _check(logits, k, spec, bias)
    bias[bias > 2.2] = 0.0                             # 20 ahead
    _check(logits, k, spec, bias)


@pytest.mark.parametrize("chunk", [1, 7, 8, 1 << 20, (1 << 31) - 8, (1 << 31) - 1])
@pytest.mark.parametrize("T", [20, 200, 1500])
def test_chunks_of_any_size(T, chunk):
    """The chunk table for chunk sizes up to the type's largest, on each path to the tables."""
    g = torch.Generator().manual_seed(T)
    logits = torch.randn((T, 24), generator=g)
    _check(logits, 3, _spec(), chunk=chunk)
    r = moeq.moe_route_permute(logits.to(DEV), None, 3, chunk)
    s = moeq.moe_route_scored(logits.to(DEV), None, 3, chunk, _spec())
    n = int(r.num_chunks.item())
    assert n == s.num_chunks.item() and torch.equal(r.chunk_offsets[:n + 1], s.chunk_offsets[:n + 1])
    counts = (r.expert_offsets[1:] - r.expert_offsets[:-1]).view(1, 24).contiguous()
    rows = torch.zeros((3 * T, 8), dtype=torch.bfloat16, device=DEV)
    _, local = moeq.moe_ep_regroup(counts, rows, 0, chunk)
    assert local.num_chunks.item() == n and torch.equal(local.chunk_offsets[:n + 1], r.chunk_offsets[:n + 1])


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("scale", [1.0, 2.5])
def test_gradient_of_experts_masked_by_the_bias(score, renorm, scale):
    """An expert that only its key masks stays in the softmax's denominator, as in the forward: with plain softmax
    gates its logit gets -s_e sum_j ds_j s_j like every expert that is not selected, and 0 otherwise. An expert
    masked by its logit gets 0. Against the formula and against differences of the forward's own gates."""
    T, E, k, h = 40, 9, 4, 2.0 ** -7
    g = torch.Generator().manual_seed(3)
    logits = (512 * torch.randn((T, E), generator=g)).round() / 1024          # logits +- h are exact
    logits[:, 8] = -float("inf")
    bias = torch.tensor([0.0, -float("inf"), 0.3, float("nan"), -float("inf"), -0.3, 0.6, 0.1, 0.2])
    dg = torch.randn((T, k), generator=g)
    by_key, open_ = [1, 3, 4], [0, 2, 5, 6, 7]
    spec = _spec(score=score, renorm=renorm, scale=scale)

    def gates(lg):
        r = moeq.moe_route_scored(lg.to(DEV), None, k, 8, spec, bias=bias.to(DEV))
        return r, f64(r.gates)
    r, w = gates(logits)
    idx = r.topk_idx.cpu().numpy()
    assert set(idx.ravel().tolist()) <= set(open_)
    got = f64(moeq.moe_route_scored_bwd(dg.to(DEV), logits.to(DEV), r, spec))
    d = dg.numpy().astype(np.float64)
    s = O8.scored_scores(logits.numpy(), score)
    sel = np.take_along_axis(s, idx.astype(np.int64), 1)
    if score == "softmax" and not renorm:
        want = -s[:, by_key] * (scale * d * sel).sum(1, keepdims=True)
        assert np.all(np.abs(got[:, by_key] - want) <= 256 * U * s[:, by_key] * (scale * np.abs(d) * sel).sum(1, keepdims=True))
        assert np.abs(got[:, by_key]).max() > 0.05
    else:
        assert not got[:, by_key].any()
    assert not got[:, 8].any()
    # Differences: gates have third derivatives below 6 scale (scores above 0.2 here), so h^2 scale; each gate is
    # off by 64 U, twice over 2 h.
    lim = (h * h + 64 * U / h) * scale * np.abs(d).sum(1)
    for e in range(8):
        step = torch.zeros(E)
        step[e] = h
        up, down = gates(logits + step), gates(logits - step)
        same = (up[0].topk_idx.cpu().numpy() == idx).all(1) & (down[0].topk_idx.cpu().numpy() == idx).all(1)
        assert same.sum() > T / 2                                             # (the selection itself moves in few)
        num = ((up[1] - down[1]) * d).sum(1) / (2 * h)
        assert np.all(np.abs(num - got[:, e])[same] <= lim[same] + 256 * U * scale * np.abs(d).sum(1)[same])


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("spread", [10.0, 30.0, 60.0])
@pytest.mark.parametrize("groups,with_bias", [(1, False), (1, True), (8, False), (8, True)])
def test_gates_of_scores_far_apart(score, renorm, spread, groups, with_bias):
    """Logits over hundreds: differences with a rounding of their own, and tokens whose bias or groups leave only
    experts with scores near and below single precision's smallest number."""
    T, E, k = 200, 64, 8
    g = torch.Generator().manual_seed(int(spread) + groups)
    logits = spread * torch.randn((T, E), generator=g)
    logits[:40] -= 40 + logits[:40].amax(1, keepdim=True)                     # sigmoids of -40 and below
    bias = 2 * torch.randn(E, generator=g) if with_bias else None
    _check(logits, k, _spec(score=score, renorm=renorm, groups=groups, topk_groups=max(1, groups // 4), scale=1.5), bias)


def test_gates_of_scores_that_are_zero():
    """A logit of +inf that the bias keeps out of the selection takes the whole softmax: the gates are 0."""
    logits = torch.randn((20, 16), generator=torch.Generator().manual_seed(1))
    logits[:, 3] = float("inf")
    logits[10:, 3] = 3.0e38
    bias = torch.zeros(16)
    bias[3] = -10.0
    for renorm in (False, True):
        r, topk = _check(logits, 4, _spec(renorm=renorm), bias)
        assert not np.any(topk == 3) and not r.gates.any()
