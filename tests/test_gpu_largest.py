"""The router and the FP8 rows at the largest counts that their entry points
take: 2^31 - 1 tokens or rows of the smallest width (up to 112 GB of tensors)."""

import pytest
import torch

from oracle import scored_fp8 as O8
from quantized_rl_fine_b200 import moeq

from _common import f64

pytestmark = pytest.mark.gpu

DEV = "cuda"
N = (1 << 31) - 1


@pytest.fixture(autouse=True)
def room():
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 130e9:
        pytest.skip("needs 130 GB of free memory")
    yield
    torch.cuda.empty_cache()


def test_router_of_the_most_tokens():
    spec = moeq.RouterSpec(score="sigmoid", renorm=False, scale=2.0)
    lg = torch.zeros((N, 1), device=DEV)
    lg[-3:, 0] = torch.tensor([1.0, -2.0, 0.5])
    r = moeq.moe_route_scored(lg, None, 1, 8, spec)
    assert r.expert_offsets.tolist() == [0, N] and r.num_active.item() == 1
    assert r.perm_token[-3:].tolist() == [N - 3, N - 2, N - 1] and r.inv_perm[-3:].tolist() == [N - 3, N - 2, N - 1]
    assert not r.topk_idx[-3:].any() and bool((r.gates[:5] == 1.0).all())
    s = torch.sigmoid(lg[-3:].double())
    assert bool(((r.gates[-3:] - 2 * s).abs() <= 2 * 64 * 2.0 ** -24 * s).all())
    dg = torch.ones((N, 1), device=DEV)
    d = moeq.moe_route_scored_bwd(dg, lg, r, spec)
    want = 2 * s * (1 - s)
    assert bool((d[:5] == 0.5).all()) and bool(((d[-3:] - want).abs() <= 2.0 ** -23 * want).all())


def test_fp8_rows_of_the_most_rows():
    K = 16
    x = torch.zeros((N, K), dtype=torch.bfloat16, device=DEV)
    tail = torch.randn((3, K), generator=torch.Generator().manual_seed(1)).to(torch.bfloat16)
    x[-3:] = tail.to(DEV)
    rows = moeq.moe_quantize_fp8_rows(x)
    codes, e = O8.quantize_rows(f64(tail))
    assert (rows.q[-3:].view(torch.uint8).cpu().numpy() == codes).all()
    assert (f64(rows.scales[0, -3:]) == 2.0 ** e[:, 0]).all() and bool((rows.scales[0, :1000] == 1.0).all())
    del x
    y = moeq.moe_dequantize_fp8_rows(rows)
    assert (f64(y[-3:]) == O8.rows_values(codes, 2.0 ** e, 128)).all() and not y[:1000].any()
