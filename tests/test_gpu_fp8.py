"""FP8 rows, the grouped FP8 products and the 8-bit checkpoint against their
float64 definitions.

Tolerances. The quantizer rounds once and is compared bit for bit. A product
of R terms accumulates in FP32: every addition is off by at most 2^-23 of the
sum of magnitudes (2^-24 rounded, 2^-23 if the tensor core truncates), the block
scales add three roundings, so |acc - exact| <= delta = (R + 8) * 2^-23 * sum |a w|.
BF16 outputs add 2^-8 relative. A quantized output is the nearest e4m3 value,
half a step: 2^-4 relative or half a subnormal step, 2^-10 of its scale (which is at most 2 amax / 448);
the value quantized is off by delta carried through the epilogue. silu(g) u moves by at most
1.1 |u| dg + |silu g| du, and its own FP32 evaluation by 2^-18 relative (fast exponential: 2 + |g| ulp,
|g| < 100 where the result is not 0).
"""

import numpy as np
import pytest
import torch

from oracle import scored_fp8 as O8
from quantized_rl_fine_b200 import moeq

from _common import f64

pytestmark = pytest.mark.gpu

DEV = "cuda"
U = 2.0 ** -24


def _routing(counts, k=1, seed=0):
    """Tables of a layer whose experts have `counts` rows: T*k = sum(counts) rows in a random stable permutation."""
    counts = np.asarray(counts)
    E, M = len(counts), int(counts.sum())
    T = M // k
    off = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    perm = np.random.RandomState(seed).permutation(M).astype(np.int32)       # slot -> row
    tok = np.empty(M, np.int32)
    tok[perm] = np.arange(M) // k
    act = np.flatnonzero(counts).astype(np.int32)
    active = np.full(E, -7, np.int32)                                        # the tail is not read
    active[: len(act)] = act
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(DEV)       # noqa: E731
    z = torch.zeros(E + 1, dtype=torch.int32, device=DEV)
    return moeq.Routing(topk_idx=None, gates=None, expert_offsets=dev(off), active=dev(active),
                        num_active=torch.tensor([len(act)], dtype=torch.int32, device=DEV), chunk_offsets=z,
                        num_chunks=z[:1], perm_token=dev(tok), inv_perm=dev(perm), x_perm=None, E=E, k=k), off


def _codes(t):
    return t.cpu().view(torch.uint8).numpy()


def _fp8(codes):
    return torch.from_numpy(codes).to(DEV).view(torch.float8_e4m3fn)


def _rows(g, M, K):
    """Random e4m3 rows with arbitrary fp32 scales."""
    codes = torch.randint(0, 256, (M, K), generator=g).to(torch.uint8)
    codes[(codes & 0x7F) == 0x7F] = 0x12
    s = 2.0 ** torch.randint(-4, 3, (-(-K // 128), M), generator=g).float() * (1 + torch.rand((-(-K // 128), M), generator=g))
    return moeq.Fp8Rows(_fp8(codes.numpy()), s.to(DEV)), O8.rows_values(codes.numpy(), f64(s).T, 128)


def _weight(g, E, N, K):
    codes = torch.randint(0, 256, (E, N, K), generator=g).to(torch.uint8)
    codes[(codes & 0x7F) == 0x7F] = 0x83
    s = 1e-3 * (0.5 + torch.rand((E, -(-N // 128), -(-K // 128)), generator=g))
    return moeq.Fp8WeightT(_fp8(codes.numpy()), s.to(DEV)), O8.weight_values(codes.numpy(), f64(s))


# ----------------------------------------------------------------------------- rows

@pytest.mark.parametrize("T,K,k", [(1, 16, 1), (3, 128, 2), (5, 144, 3), (37, 1040, 4), (64, 4096, 8), (9, 7168, 32)])
def test_quantize_rows_bit_exact(T, K, k):
    g = torch.Generator().manual_seed(T + K)
    x = torch.randn((T, K), generator=g) * torch.exp2(torch.randint(-20, 20, (T, 1), generator=g).float())
    x[0, : K // 2] = 0                                            # a block of zeros, or half of one
    x = x.to(torch.bfloat16)
    r, _ = _routing([T * k], k, seed=K)
    got = moeq.moe_quantize_fp8_rows(x.to(DEV), r)
    codes, e = O8.quantize_rows(f64(x)[r.perm_token.cpu().numpy()])
    assert np.array_equal(_codes(got.q), codes)
    assert np.array_equal(f64(got.scales), 2.0 ** e.T.astype(np.float64))
    plain = moeq.moe_quantize_fp8_rows(x.to(DEV))
    codes, e = O8.quantize_rows(f64(x))
    assert np.array_equal(_codes(plain.q), codes)
    assert np.array_equal(f64(plain.scales), 2.0 ** e.T.astype(np.float64))
    assert np.array_equal(f64(moeq.moe_dequantize_fp8_rows(plain)), O8.rows_values(codes, 2.0 ** e.astype(np.float64), 128))


def test_quantize_every_bf16_value():
    """Blocks whose largest magnitude is each positive BF16 value (the first two exponents subnormal), next to halves,
    NaN and infinities."""
    bits = np.arange(0, 0x7F80, dtype=np.uint16)
    amax = torch.from_numpy(bits.view(np.int16)).view(torch.bfloat16)
    x = torch.zeros((len(bits), 128), dtype=torch.bfloat16)
    frac = torch.tensor([1.0, -1.0, 0.5, 0.75, 0.3, -0.07, 0.011, 0.0013, 1e-4, -1e-5, 0.9961, 0.34375])
    x[:, : len(frac)] = (amax.float()[:, None] * frac).to(torch.bfloat16)
    x[::3, 100], x[::3, 101], x[::3, 102] = float("inf"), -float("inf"), float("nan")
    got = moeq.moe_quantize_fp8_rows(x.to(DEV))
    codes, e = O8.quantize_rows(f64(x))
    have = _codes(got.q)
    nan = (codes & 0x7F) == 0x7F
    assert np.array_equal((have & 0x7F) == 0x7F, nan)             # the sign of a NaN is not specified
    assert np.array_equal(have[~nan], codes[~nan])
    assert np.array_equal(f64(got.scales), 2.0 ** e.T.astype(np.float64))


def test_dequantize_every_code_and_scale():
    codes = np.tile(np.arange(256, dtype=np.uint8), (256, 1))
    X = np.tile(np.arange(256, dtype=np.uint8), (8, 1))             # [256 / 32 groups][row m = X]
    rows = moeq.Fp8Rows(_fp8(codes), torch.from_numpy(X).to(DEV))
    got = f64(moeq.moe_dequantize_fp8_rows(rows))
    with np.errstate(invalid="ignore"):
        s = np.where(np.arange(256) == 255, np.nan, 2.0 ** (np.arange(256.0) - 127))
        want = O8.e4m3_values()[None, :] * s[:, None]
    want = torch.from_numpy(want).to(torch.float32).to(torch.bfloat16)   # exact but for overflow and subnormals
    assert np.array_equal(np.isnan(got), np.isnan(f64(want)))
    ok = ~np.isnan(got)
    assert np.array_equal(got[ok], f64(want)[ok])


def test_out_of_range_slots_are_skipped():
    T, K, k = 4, 32, 2
    x = torch.randn((T, K)).to(torch.bfloat16).to(DEV)
    r, _ = _routing([T * k], k)
    r.inv_perm = r.inv_perm.clone()
    r.inv_perm[3], r.inv_perm[6] = -1, T * k
    lost = sorted(set(range(T * k)) - set(r.inv_perm.cpu().tolist()))
    out = moeq.Fp8Rows(torch.zeros((T * k, K), dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn),
                       torch.full((1, T * k), 7.0, device=DEV))
    moeq.moe_quantize_fp8_rows(x, r, out=out)
    assert not _codes(out.q)[lost].any() and np.all(f64(out.scales)[0, lost] == 7.0)


# ----------------------------------------------------------------------------- products

COUNTS = {
    "one_row": [1],
    "empty_ends": [0, 5, 0, 130, 0],
    "tile_edges": [128, 127, 129, 1, 256, 0, 257],
    "ragged": [3, 0, 61, 200, 17, 1, 90, 40],
    "many": [int(v) for v in np.random.RandomState(4).randint(0, 40, 70)],
}
SHAPES = [(16, 16), (128, 256), (272, 144), (1040, 400), (640, 1392)]


@pytest.fixture(params=["0", "1", "2", "3"], ids=["single", "pair", "few", "some"])
def ctas(request, monkeypatch):
    """Tiles of 128 rows, CTA pairs on 256 (above 512 rows an expert), tiles of 32 (up to 16) and of 64 (up to 40)."""
    monkeypatch.setenv("MOEQ_F8FORM", request.param)
    return request.param


@pytest.mark.parametrize("name", sorted(COUNTS))
@pytest.mark.parametrize("K,N", SHAPES)
@pytest.mark.parametrize("bwd", [False, True])
def test_product(name, K, N, bwd, ctas):
    g = torch.Generator().manual_seed(K + N)
    counts = COUNTS[name]
    r, off = _routing(counts)
    M, E = int(off[-1]), len(counts)
    R = N if bwd else K
    a, av = _rows(g, M, R)
    w, wv = _weight(g, E, N, K)
    got = (moeq.moe_grouped_fp8_gemm_bwd_dx if bwd else moeq.moe_grouped_fp8_gemm_fwd)(a, w, r)
    assert moeq.moe_get_device_error() == 0
    want, mag = O8.fp8_gemm(av, wv, off, bwd)
    lim = (R + 8) * 2 * U * mag
    assert np.all(np.abs(f64(got) - want) <= 2.0 ** -8 * (np.abs(want) + lim) + lim)


def _check_quantized(rows, want, delta, block, M, width):
    """rows: e4m3 blocks of numbers within delta of `want`."""
    e8 = rows.scales.dtype == torch.uint8
    s = 2.0 ** (rows.scales.cpu().numpy().astype(np.float64).T - 127) if e8 else f64(rows.scales).T
    got = O8.rows_values(_codes(rows.q), s, block)
    n = width // block
    amax = np.abs(want).reshape(M, n, block).max(2)
    dmax = delta.reshape(M, n, block).max(2)
    assert np.all(s * 448 >= amax - dmax)                           # large enough, and no larger than needed
    assert np.all((s * 224 <= amax + dmax) | (s == 2.0 ** -126) | ((amax <= dmax) & (s == 1.0)))
    full = np.repeat(s, block, 1)
    lim = 2.0 ** -4 * (np.abs(want) + delta) + 2.0 ** -10 * full + delta
    assert np.all(np.abs(got - want) <= lim)


@pytest.mark.parametrize("name", sorted(COUNTS))
@pytest.mark.parametrize("K,f,save", [(16, 128, True), (400, 128, False), (272, 384, True), (1024, 256, True)])
def test_swiglu_product_and_checkpoint(name, K, f, save, ctas):
    g = torch.Generator().manual_seed(K + f)
    counts = COUNTS[name]
    r, off = _routing(counts)
    M, E, N = int(off[-1]), len(counts), 2 * f
    a, av = _rows(g, M, K)
    w, wv = _weight(g, E, N, K)
    w.scales *= 0.02                                                # gate values of order one and ten
    wv = wv * (f64(w.scales)[:, :1, :1] * 0 + 0.02)
    h, saved = moeq.moe_grouped_fp8_gemm_fwd(a, w, r, moeq.EPI_SWIGLU, save_gu=save)
    assert moeq.moe_get_device_error() == 0
    gu, mag = O8.fp8_gemm(av, wv, off)
    # (the scales times 0.02 round once more)
    d = (K + 10) * 2 * U * mag
    want = O8.swiglu(gu)
    gg, uu = gu[:, :f], gu[:, f:]
    dh = 1.1 * (np.abs(uu) + d[:, f:]) * d[:, :f] + (np.abs(O8.swiglu(np.concatenate([gg, np.ones_like(gg)], 1))) + 1.1 * d[:, :f]) * d[:, f:]
    _check_quantized(h, want, dh + 2.0 ** -18 * np.abs(want), 128, M, f)
    if save:
        _check_quantized(saved, gu, d, 32, M, N)
    else:
        assert saved is None
    h2, _ = moeq.moe_grouped_fp8_gemm_fwd(a, w, r, moeq.EPI_SWIGLU)      # the checkpoint changes nothing
    assert np.array_equal(_codes(h2.q), _codes(h.q)) and torch.equal(h2.scales, h.scales)


@pytest.mark.parametrize("name", sorted(COUNTS))
@pytest.mark.parametrize("N,f", [(16, 128), (400, 384), (1040, 256)])
def test_swiglu_backward_from_checkpoint(name, N, f, ctas):
    g = torch.Generator().manual_seed(N + f)
    counts = COUNTS[name]
    r, off = _routing(counts)
    M, E = int(off[-1]), len(counts)
    dv, dval = _rows(g, M, N)
    w, wv = _weight(g, E, N, f)
    codes, e = O8.quantize_rows(f64(3 * torch.randn((M, 2 * f), generator=g)), 32)
    ck = moeq.Fp8Rows(_fp8(codes), torch.from_numpy(np.ascontiguousarray((e.T + 127).astype(np.uint8))).to(DEV))
    gu = O8.rows_values(codes, 2.0 ** e.astype(np.float64), 32)
    got = moeq.moe_grouped_fp8_gemm_bwd_dx(dv, w, r, moeq.EPI_SWIGLU_BWD, saved=ck)
    assert moeq.moe_get_device_error() == 0
    dh, mag = O8.fp8_gemm(dval, wv, off, True)
    want = O8.swiglu_bwd(dh, gu)
    # linear in dh: the factor's magnitude times delta, its FP32 evaluation (2^-18 of the
    # magnitudes |u| (1 + |g|)), and the BF16 rounding of dg and du
    d = (N + 8) * 2 * U * mag
    gg, uu = np.abs(gu[:, :f]), np.abs(gu[:, f:])
    size = np.concatenate([uu * (1 + gg), gg], 1)
    lim = size * np.tile(d, 2) + 2.0 ** -18 * size * np.tile(np.abs(dh) + d, 2)
    _check_quantized(got, want, lim + 2.0 ** -8 * (np.abs(want) + lim), 128, M, 2 * f)


def test_rows_do_not_depend_on_the_batch(ctas):
    """A row's bits are the same alone and among others (plain and SwiGLU)."""
    g = torch.Generator().manual_seed(2)
    K, f = 400, 128
    a, _ = _rows(g, 300, K)
    w, _ = _weight(g, 1, 2 * f, K)
    big, _ = _routing([300])
    one, _ = _routing([1])
    y = moeq.moe_grouped_fp8_gemm_fwd(a, w, big)
    h, s = moeq.moe_grouped_fp8_gemm_fwd(a, w, big, moeq.EPI_SWIGLU, save_gu=True)
    for m in (0, 131, 299):
        am = moeq.Fp8Rows(a.q[m:m + 1].clone(), a.scales[:, m:m + 1].clone())
        assert torch.equal(moeq.moe_grouped_fp8_gemm_fwd(am, w, one)[0], y[m])
        hm, sm = moeq.moe_grouped_fp8_gemm_fwd(am, w, one, moeq.EPI_SWIGLU, save_gu=True)
        assert np.array_equal(_codes(hm.q)[0], _codes(h.q)[m]) and torch.equal(sm.scales[:, 0], s.scales[:, m])


def test_nothing_past_the_rows_is_written_and_nan_stays_in_its_row():
    """Outputs sit in the middle of larger buffers; a NaN in one row does not reach another."""
    g = torch.Generator().manual_seed(8)
    K, N, M = 144, 272, 70
    r, off = _routing([30, 0, 40])
    a, av = _rows(g, M, K)
    w, wv = _weight(g, 3, N, K)
    codes = _codes(a.q).copy()
    codes[33, 7] = 0x7F
    a.q = _fp8(codes)
    buf = torch.full((M + 16, N), 7.0, dtype=torch.bfloat16, device=DEV)
    wc = moeq.Fp8WeightC(w.q.data_ptr(), w.scales.data_ptr(), 3, N, K)
    import ctypes
    gc = r.groups()
    st = moeq.lib().moe_grouped_fp8_gemm_fwd(a.q.data_ptr(), a.scales.data_ptr(), M, ctypes.byref(wc), ctypes.byref(gc), 0,
                                             buf[8].data_ptr(), None, None, None, torch.cuda.current_stream().cuda_stream)
    assert st == 0 and moeq.moe_get_device_error() == 0
    got = f64(buf)
    assert np.all(got[:8] == 7.0) and np.all(got[M + 8:] == 7.0)
    assert np.all(np.isnan(got[8 + 33]))
    want, mag = O8.fp8_gemm(np.nan_to_num(av), wv, off)
    rest = [m for m in range(M) if m != 33]
    lim = (K + 8) * 2 * U * mag + 2.0 ** -8 * np.abs(want) * (1 + 2.0 ** -8)
    assert np.all(np.abs(got[8:M + 8] - want)[rest] <= lim[rest])


def test_tables_that_do_not_fit_the_rows_are_an_error_and_launch_no_tile(ctas):
    g = torch.Generator().manual_seed(8)
    a, _ = _rows(g, 40, 128)
    w, _ = _weight(g, 2, 128, 128)
    for off in ([0, 10, 39], [0, 50, 40], [1, 20, 40]):
        r, _ = _routing([20, 20])
        r.expert_offsets = torch.tensor(off, dtype=torch.int32, device=DEV)
        moeq.moe_grouped_fp8_gemm_fwd(a, w, r)
        assert moeq.moe_get_device_error() == moeq.DEVERR_BAD_OFFSETS
    r, _ = _routing([20, 20])
    r.active = torch.tensor([0, 2], dtype=torch.int32, device=DEV)
    moeq.moe_grouped_fp8_gemm_fwd(a, w, r)
    assert moeq.moe_get_device_error() == moeq.DEVERR_BAD_OFFSETS


def test_offsets_past_32_bits():
    """More than 2^31 output elements and input bytes: the last rows are where they belong."""
    K, N, M = 16400, 16, 132000                                     # M * K > 2^31
    x = torch.zeros((M, K), dtype=torch.bfloat16, device=DEV)
    g = torch.Generator().manual_seed(3)
    tail = torch.randn((5, K), generator=g).to(torch.bfloat16)
    x[-5:] = tail.to(DEV)
    rows = moeq.moe_quantize_fp8_rows(x)
    codes, e = O8.quantize_rows(f64(tail))
    assert np.array_equal(_codes(rows.q[-5:]), codes)
    assert np.array_equal(f64(rows.scales[:, -5:]).T, 2.0 ** e.astype(np.float64))
    r, _ = _routing([M])
    w, wv = _weight(g, 1, N, K)
    y = moeq.moe_grouped_fp8_gemm_fwd(rows, w, r)
    want, mag = O8.fp8_gemm(O8.rows_values(codes, 2.0 ** e.astype(np.float64), 128), wv, [0, 5])
    lim = (K + 8) * 2 * U * mag
    assert np.all(np.abs(f64(y[-5:]) - want) <= 2.0 ** -8 * (np.abs(want) + lim) + lim)
    del x
    # the transposed use: 132000 rows of 16 through [16][16400] give M * 16400 outputs
    d, dv = _rows(g, 5, N)
    big = moeq.Fp8Rows(torch.zeros((M, N), dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn),
                       torch.ones((1, M), device=DEV))
    big.q[-5:] = d.q
    big.scales[:, -5:] = d.scales
    z = moeq.moe_grouped_fp8_gemm_bwd_dx(big, w, r)
    want, mag = O8.fp8_gemm(dv, wv, [0, 5], True)
    lim = (N + 8) * 2 * U * mag
    assert np.all(np.abs(f64(z[-5:]) - want) <= 2.0 ** -8 * (np.abs(want) + lim) + lim)
    assert not z[:100].any()


def test_captured_replayed_and_two_streams_at_once(ctas):
    g = torch.Generator().manual_seed(6)
    K, f, M = 256, 128, 200
    r, off = _routing([90, 0, 110])
    w, _ = _weight(g, 3, 2 * f, K)
    wd, _ = _weight(g, 3, K, f)
    xs = [torch.randn((M, K), generator=g).to(torch.bfloat16).to(DEV) for _ in range(2)]

    def chain(x, stream=None):
        a = moeq.moe_quantize_fp8_rows(x, r, stream=stream)
        h, saved = moeq.moe_grouped_fp8_gemm_fwd(a, w, r, moeq.EPI_SWIGLU, save_gu=True, stream=stream)
        y = moeq.moe_grouped_fp8_gemm_fwd(h, wd, r, stream=stream)
        d = moeq.moe_quantize_fp8_rows(y, stream=stream)
        dgu = moeq.moe_grouped_fp8_gemm_bwd_dx(d, wd, r, moeq.EPI_SWIGLU_BWD, saved=saved, stream=stream)
        return y, moeq.moe_grouped_fp8_gemm_bwd_dx(dgu, w, r, stream=stream)

    want = [[t.clone() for t in chain(x)] for x in xs]
    x = xs[0].clone()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        outs = chain(x)
    for i in (1, 0):
        x.copy_(xs[i])
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want[i]))
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [chain(xs[i], stream=streams[i]) for i in range(2)]
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(a, b) for a, b in zip(got[i], want[i]))
    assert moeq.moe_get_device_error() == 0


def test_all_forms_give_the_same_bits(monkeypatch):
    g = torch.Generator().manual_seed(9)
    K, f = 640, 256
    r, off = _routing([300, 0, 5, 513])
    M = int(off[-1])
    a, _ = _rows(g, M, K)
    w, _ = _weight(g, 4, 2 * f, K)
    res = []
    for p in "0123":
        monkeypatch.setenv("MOEQ_F8FORM", p)
        h, s = moeq.moe_grouped_fp8_gemm_fwd(a, w, r, moeq.EPI_SWIGLU, save_gu=True)
        res.append((moeq.moe_grouped_fp8_gemm_fwd(a, w, r), h.q.view(torch.uint8), h.scales, s.q.view(torch.uint8), s.scales))
    assert all(torch.equal(x, y) for z in res[1:] for x, y in zip(res[0], z))


@pytest.mark.parametrize("M", [64, 65, 160, 161, 256, 257, 2048, 2049])
def test_the_form_chosen_by_the_mean_rows_changes_no_bit(M, monkeypatch):
    """Four experts: 16, 40, 64 and 512 mean rows and one more, most of them in one expert."""
    g = torch.Generator().manual_seed(M)
    K, N = 272, 400
    r, off = _routing([1, M - 34, 0, 33])
    a, _ = _rows(g, M, K)
    d, _ = _rows(g, M, N)
    w, _ = _weight(g, 4, N, K)
    monkeypatch.delenv("MOEQ_F8FORM", raising=False)
    got = (moeq.moe_grouped_fp8_gemm_fwd(a, w, r), moeq.moe_grouped_fp8_gemm_bwd_dx(d, w, r))
    monkeypatch.setenv("MOEQ_F8FORM", "0")
    want = (moeq.moe_grouped_fp8_gemm_fwd(a, w, r), moeq.moe_grouped_fp8_gemm_bwd_dx(d, w, r))
    assert all(torch.equal(x, y) for x, y in zip(got, want))
    assert moeq.moe_get_device_error() == 0


def test_infinities_and_nan_in_the_epilogues(ctas):
    """An accumulator that overflows or is NaN makes NaN where it enters, and the rest of its block is
    quantized as if it were not there."""
    f, K, M = 128, 128, 3
    r, off = _routing([M])
    codes = np.zeros((M, K), np.uint8)
    codes[:, 0] = 0x38                                            # 1.0
    a = moeq.Fp8Rows(_fp8(codes), torch.ones((1, M), device=DEV))
    wc = np.full((1, 2 * f, K), 0x38, np.uint8)
    ws = torch.full((1, 2, 1), 1.0, device=DEV)
    # row 1 overflows through its scale, row 2 is NaN in one code
    a.scales[0, 1] = 3.0e38
    codes[2, 5] = 0x7F
    a.q = _fp8(codes)
    wc[0, 7, 0] = 0x7E                                            # gate feature 7 of row 1: 448 * 3e38
    w = moeq.Fp8WeightT(_fp8(wc), ws)
    h, s = moeq.moe_grouped_fp8_gemm_fwd(a, w, r, moeq.EPI_SWIGLU, save_gu=True)
    hv, sv = f64(moeq.moe_dequantize_fp8_rows(h)), f64(moeq.moe_dequantize_fp8_rows(s))
    assert moeq.moe_get_device_error() == 0
    assert np.isfinite(hv[0]).all() and np.isfinite(sv[0]).all() and np.all(sv[0, :7] == 1.0) and sv[0, 7] == 448.0
    assert np.isnan(sv[2]).all() and np.isnan(hv[2]).all()
    # row 1: gate 7 overflowed; its neighbours are 3e38 to half a step; h = silu(3e38) * 3e38 overflows everywhere
    assert np.isnan(sv[1, 7]) and np.all(np.abs(np.delete(sv[1], 7) / 3.0e38 - 1) <= 2.0 ** -4) and np.isnan(hv[1]).all()
    # backward: dh finite, a checkpoint with NaN and infinite-like scales in single groups
    d = moeq.Fp8Rows(_fp8(np.full((M, 128), 0x38, np.uint8)), torch.ones((1, M), device=DEV))
    wd = moeq.Fp8WeightT(_fp8(np.full((1, 128, f), 0x38, np.uint8)), torch.ones((1, 1, 1), device=DEV))
    ck = np.full((M, 2 * f), 0x38, np.uint8)
    ck[1, 3] = 0x7F
    X = np.full((8, M), 127, np.uint8)
    X[5, 2] = 254                                                 # u of features 32..63 of row 2: 2^127
    got = moeq.moe_grouped_fp8_gemm_bwd_dx(d, wd, r, moeq.EPI_SWIGLU_BWD, saved=moeq.Fp8Rows(_fp8(ck), torch.from_numpy(X).to(DEV)))
    v = f64(moeq.moe_dequantize_fp8_rows(got))
    sg = 1 / (1 + np.exp(-1.0))
    dg, du = 128 * sg * (2 - sg), 128 * sg
    near = lambda x, y: np.all(np.abs(x / y - 1) <= 2.0 ** -4 + 2.0 ** -7)       # noqa: E731  e4m3 and BF16
    assert near(v[0, :f], dg) and near(v[0, f:], du)
    assert np.isnan(v[1, 3]) and np.isnan(v[1, f + 3]) and near(np.delete(v[1, :f], 3), dg) and near(np.delete(v[1, f:], 3), du)
    assert np.isnan(v[2, 32:64]).all() and near(v[2, :32], dg) and near(v[2, 64:f], dg) and near(v[2, f:], du)


def test_waits_that_run_out_are_reported_and_the_next_call_is_clean(ctas):
    """With a budget of 200 cycles a wait of tens of microseconds runs out: the checkpoint warp waits that long
    for its next tile (56 reduction blocks), and there are more tiles than CTAs."""
    f, R, counts = 256, 7168, [9000, 11000]
    g = torch.Generator(device=DEV).manual_seed(7)
    r, off = _routing(counts)
    M = int(off[-1])
    codes = lambda *n: (torch.randint(0, 0x70, n, generator=g, device=DEV, dtype=torch.int16).to(torch.uint8)     # noqa: E731
                        .view(torch.float8_e4m3fn))
    a = moeq.Fp8Rows(codes(M, R), torch.ones((R // 128, M), device=DEV))
    w = moeq.Fp8WeightT(codes(2, R, f), torch.full((2, R // 128, 2), 1e-3, device=DEV))
    ck = moeq.Fp8Rows(codes(M, 2 * f), torch.full((2 * f // 32, M), 120, dtype=torch.uint8, device=DEV))

    def run():
        d = moeq.moe_grouped_fp8_gemm_bwd_dx(a, w, r, moeq.EPI_SWIGLU_BWD, saved=ck)
        return d.q.view(torch.uint8), d.scales
    want = [t.clone() for t in run()]
    assert moeq.moe_get_device_error() == moeq.DEVERR_NONE
    try:
        moeq.moe_test_set_wait_budget(200)
        run()
        code = moeq.moe_get_device_error()
    finally:
        moeq.moe_test_set_wait_budget(0)
    assert code == moeq.DEVERR_WAIT_TIMEOUT
    assert all(torch.equal(x, y) for x, y in zip(run(), want)) and moeq.moe_get_device_error() == moeq.DEVERR_NONE


def test_pairs_of_experts_of_many_rows():
    """More than 512 rows an expert: the pair kernel by the library's own choice, ragged ends of its 256-row tiles."""
    g = torch.Generator().manual_seed(3)
    counts = [700, 512, 769, 513]
    K, N = 272, 400
    r, off = _routing(counts)
    a, av = _rows(g, int(off[-1]), K)
    w, wv = _weight(g, 4, N, K)
    want, mag = O8.fp8_gemm(av, wv, off)
    lim = (K + 8) * 2 * U * mag
    assert np.all(np.abs(f64(moeq.moe_grouped_fp8_gemm_fwd(a, w, r)) - want) <= 2.0 ** -8 * (np.abs(want) + lim) + lim)
    assert moeq.moe_get_device_error() == 0


def test_refusals_of_wrong_rows_and_weights():
    g = torch.Generator().manual_seed(1)
    r, _ = _routing([4, 4])
    a, _ = _rows(g, 8, 128)
    w, _ = _weight(g, 2, 256, 128)
    F = moeq.Fp8Rows
    for bad in (F(a.q[:, :112], a.scales), F(a.q.view(torch.uint8), a.scales), F(a.q, a.scales.double()), F(a.q, a.scales[:, :7]),
                F(a.q[:, ::2], a.scales), F(a.q[0], a.scales)):
        with pytest.raises(ValueError):
            moeq.moe_grouped_fp8_gemm_fwd(bad, w, r)
    with pytest.raises(ValueError):
        moeq.moe_grouped_fp8_gemm_fwd(a, moeq.Fp8WeightT(w.q, w.scales.transpose(1, 2)), r)
    with pytest.raises(ValueError):
        moeq.moe_grouped_fp8_gemm_fwd(a, moeq.Fp8WeightT(w.q[:1].contiguous(), w.scales[:1].contiguous()), r)     # tables of two experts
    with pytest.raises(ValueError):
        moeq.moe_grouped_fp8_gemm_fwd(a, w, r, save_gu=True)
    with pytest.raises(moeq.MoeError):
        moeq.moe_grouped_fp8_gemm_fwd(a, w, r, moeq.EPI_SWIGLU_BWD)
    d, _ = _rows(g, 8, 256)
    with pytest.raises(ValueError):
        moeq.moe_grouped_fp8_gemm_bwd_dx(d, w, r, moeq.EPI_SWIGLU_BWD)
    with pytest.raises(ValueError):
        moeq.moe_grouped_fp8_gemm_bwd_dx(d, w, r, saved=a)
    with pytest.raises(ValueError):
        moeq.moe_quantize_fp8_rows(torch.zeros((4, 32), device=DEV))
    with pytest.raises(moeq.MoeError):
        moeq.moe_quantize_fp8_rows(torch.zeros((4, 24), dtype=torch.bfloat16, device=DEV))
    with pytest.raises(ValueError):
        moeq.moe_quantize_fp8_rows(torch.zeros((5, 32), dtype=torch.bfloat16, device=DEV), r)


@pytest.mark.parametrize("epi", ["none", "glu", "bwd", "glu_bwd"])
@pytest.mark.parametrize("form", ["0", "1", "2", "3"])
def test_products_stopped_anywhere_leave_the_next_call_clean(form, epi, monkeypatch):
    """Budgets from about a microsecond up, so that different roles give up at different points (in a pair, in either
    CTA): a product that reports no timeout has all its bits, and the next one with the default budget has them too."""
    monkeypatch.setenv("MOEQ_F8FORM", form)
    g = torch.Generator(device=DEV).manual_seed(11)
    K, N = (7168, 512) if epi in ("none", "glu") else (512, 7168)
    # (more than one tile for a CTA or pair: the checkpoint warp then waits for most of a tile's 56 blocks)
    counts = [9000, 11000] if epi == "glu_bwd" else [3000, 4100]
    r, off = _routing(counts)
    M = int(off[-1])
    codes = lambda *n: (torch.randint(0, 0x70, n, generator=g, device=DEV, dtype=torch.int16).to(torch.uint8)     # noqa: E731
                        .view(torch.float8_e4m3fn))
    a = moeq.Fp8Rows(codes(M, 7168), torch.ones((56, M), device=DEV))
    w = moeq.Fp8WeightT(codes(2, N, K), torch.full((2, -(-N // 128), -(-K // 128)), 1e-3, device=DEV))
    ck = moeq.Fp8Rows(codes(M, 2 * K), torch.full((2 * K // 32, M), 120, dtype=torch.uint8, device=DEV)) if epi == "glu_bwd" else None

    def run():
        if epi == "none":
            return [moeq.moe_grouped_fp8_gemm_fwd(a, w, r)]
        if epi == "glu":
            h, s = moeq.moe_grouped_fp8_gemm_fwd(a, w, r, moeq.EPI_SWIGLU, save_gu=True)
            return [h.q.view(torch.uint8), h.scales, s.q.view(torch.uint8), s.scales]
        if epi == "bwd":
            return [moeq.moe_grouped_fp8_gemm_bwd_dx(a, w, r)]
        d = moeq.moe_grouped_fp8_gemm_bwd_dx(a, w, r, moeq.EPI_SWIGLU_BWD, saved=ck)
        return [d.q.view(torch.uint8), d.scales]
    want = [t.clone() for t in run()]
    assert moeq.moe_get_device_error() == moeq.DEVERR_NONE
    for budget in (1, 3000, 6000, 12000, 25000, 50000, 200000):
        try:
            moeq.moe_test_set_wait_budget(budget)
            got = run()
            code = moeq.moe_get_device_error()
        finally:
            moeq.moe_test_set_wait_budget(0)
        assert code in (moeq.DEVERR_NONE, moeq.DEVERR_WAIT_TIMEOUT)
        if code == moeq.DEVERR_NONE:
            assert all(torch.equal(x, y) for x, y in zip(got, want)), budget
        again = run()
        assert moeq.moe_get_device_error() == moeq.DEVERR_NONE
        assert all(torch.equal(x, y) for x, y in zip(again, want)), budget


@pytest.mark.parametrize("blocks", [1, 2, 3, 4, 5, 9])
def test_pairs_leave_no_arrival_behind(blocks, monkeypatch):
    """Pairs of fewer, as many and more reduction blocks than stages, each followed at once by products of the other
    forms on the same SMs, whose barriers lie where a late arrival of the pair would go."""
    g = torch.Generator().manual_seed(blocks)
    K, N = 128 * blocks, 512
    r, _ = _routing([700, 0, 900])
    a, _ = _rows(g, 1600, K)
    w, _ = _weight(g, 3, N, K)
    monkeypatch.setenv("MOEQ_F8FORM", "0")
    want = moeq.moe_grouped_fp8_gemm_fwd(a, w, r).clone()
    got = []
    for i in range(60):
        for form in ("1", "1", "023"[i % 3]):
            monkeypatch.setenv("MOEQ_F8FORM", form)
            got.append(moeq.moe_grouped_fp8_gemm_fwd(a, w, r))
    assert all(torch.equal(y, want) for y in got)
    assert moeq.moe_get_device_error() == 0


# ----------------------------------------------------------------------------- any FP32 scale

def _bf16_round(v):
    """float64 to the nearest BF16 value (ties to even, subnormals, overflow), as float64."""
    with np.errstate(over="ignore", invalid="ignore"):
        _, e = np.frexp(v)
        step = np.ldexp(1.0, np.maximum(e - 8, -133))
        r = np.rint(v / step) * step
        return np.where(np.abs(r) > (2.0 - 2.0 ** -7) * 2.0 ** 127, np.copysign(np.inf, r), r)


def test_dequantize_rounds_once_for_any_scale():
    """q * scale has up to 28 significant bits (exact in float64). Scales are random, and such that some code's
    product lies at a halfway point between BF16 values or next to it, also among subnormals and near the largest."""
    g = np.random.RandomState(11)
    vals = O8.e4m3_values()
    pos = vals[(vals > 0)]
    tie = (1 + (2 * g.randint(0, 128, 6000) + 1) / 256.0) * 2.0 ** g.randint(-140, 127, 6000)
    near = (tie / g.choice(pos, 6000)).astype(np.float32)
    s = np.concatenate([[1.6541667], near, np.nextafter(near, np.float32(np.inf)), np.nextafter(near, np.float32(0)),
                        2.0 ** g.uniform(-149, 127.9, 6000), 2.0 ** np.arange(-126, 127)]).astype(np.float32)
    M = len(s)
    codes = np.tile(np.arange(256, dtype=np.uint8), (M, 1))
    sc = np.stack([s, -s])                                  # the negative half of the codes with a negative scale
    got = f64(moeq.moe_dequantize_fp8_rows(moeq.Fp8Rows(_fp8(codes), torch.from_numpy(sc).to(DEV))))
    want = vals[None, :] * np.repeat(sc.T.astype(np.float64), 128, 1)
    nan = np.isnan(want)
    assert np.array_equal(np.isnan(got), nan)
    assert np.array_equal(got[~nan], _bf16_round(want)[~nan])


def test_calls_from_several_host_threads_at_once():
    """Routing of several sizes and FP8 products of all four tile forms, each thread on a stream of its own: every
    output of every iteration, and an error in a thread is an error of the test."""
    from concurrent.futures import ThreadPoolExecutor
    g = torch.Generator().manual_seed(8)
    jobs = []
    for T, E, groups in ((20, 384, 8), (3000, 256, 8), (700, 1024, 32), (1, 64, 4)):
        lg, b = torch.randn((T, E), generator=g).to(DEV), (0.1 * torch.randn(E, generator=g)).to(DEV)
        sp = moeq.RouterSpec(score="sigmoid", groups=groups, topk_groups=2, group_top=2)
        dg = torch.randn((T, 4), generator=g).to(DEV)

        def route(stream, lg=lg, b=b, sp=sp, dg=dg):
            r = moeq.moe_route_scored(lg, None, 4, 8, sp, bias=b, stream=stream)
            n = int(r.num_active.item())
            return (r.topk_idx, r.gates, r.expert_offsets, r.active[:n], r.num_active, r.num_chunks, r.perm_token, r.inv_perm,
                    moeq.moe_route_scored_bwd(dg, lg, r, sp, stream=stream))
        jobs.append(route)
    K, f = 272, 128
    w, wd = _weight(g, 2, 2 * f, K)[0], _weight(g, 2, K, f)[0]
    for counts in ([9, 20], [30, 40], [100, 200], [700, 600]):              # 32, 64 and 128 rows a tile, pairs
        r, off = _routing(counts)
        x = torch.randn((int(off[-1]), K), generator=g).to(torch.bfloat16).to(DEV)

        def product(stream, r=r, x=x):
            a = moeq.moe_quantize_fp8_rows(x, r, stream=stream)
            h, s = moeq.moe_grouped_fp8_gemm_fwd(a, w, r, moeq.EPI_SWIGLU, save_gu=True, stream=stream)
            y = moeq.moe_grouped_fp8_gemm_fwd(h, wd, r, stream=stream)
            d = moeq.moe_grouped_fp8_gemm_bwd_dx(moeq.moe_quantize_fp8_rows(y, stream=stream), wd, r, moeq.EPI_SWIGLU_BWD,
                                                 saved=s, stream=stream)
            return (h.q.view(torch.uint8), h.scales, s.q.view(torch.uint8), s.scales, y, d.q.view(torch.uint8), d.scales)
        jobs.append(product)
    want = [[t.clone() for t in job(None)] for job in jobs]
    torch.cuda.synchronize()

    def work(i):
        done = 0
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            for _ in range(20):
                got = jobs[i](s)
                s.synchronize()
                for n, (a, b) in enumerate(zip(got, want[i])):
                    assert torch.equal(a, b), (i, n)
                done += 1
        return done
    with ThreadPoolExecutor(len(jobs)) as pool:
        assert [t.result() for t in [pool.submit(work, i) for i in range(len(jobs))]] == [20] * len(jobs)
    assert moeq.moe_get_device_error() == 0
