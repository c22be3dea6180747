"""One MoE layer step through the C ABI: the orchestration of the calls only.

forward : route_permute -> fwd GEMM (gate/up, SwiGLU [, adapter]) -> fwd GEMM
          (down) -> combine
backward: scatter (gate-scaled dy) -> bwd_dx down (SwiGLU backward) ->
          bwd_dx gate/up [+ adapter backward] -> combine (unpermute-sum)
up-projection only: route_permute -> fwd GEMM (no epilogue)

With the adapter the permuted token rows are never written: routing returns
the permutation only and the adapter kernels read row p as x[perm_token[p]]
(plain loads, at no extra cost). Without it the routing call writes x_perm
and the gate/up GEMM reads it through its tensor map; gather=True makes the
GEMM gather the rows itself instead (same bits; at 341 rows per expert on
B200 its gathering producer is about 2.2x slower than the tensor-map copy,
because each stage is handed over only once its row copies have landed).

router=RouterSpec(...) routes by scores (moe_route_scored, with an optional
selection bias) and makes backward return the gradients of the gates and of
the logits as well. With FP8 expert weights (Fp8WeightT) the products run in
FP8: the token rows are quantized once and written in expert order, gate/up
writes h as FP8 rows and gate|up as an 8-bit checkpoint, and the backward
reads that checkpoint; no BF16 gate|up is kept.

A step runs on the tensors' device and on `stream`, or on that device's
current stream; what it allocates belongs to the stream it runs on.
"""

from __future__ import annotations

import torch

from . import moeq as M
from .synth import QWeightT


def route(logits: torch.Tensor, x: torch.Tensor | None, k: int, chunk_size: int,
          router: M.RouterSpec | None = None, bias: torch.Tensor | None = None, stream=None) -> M.Routing:
    """Softmax over the selected logits, or the scored routing when a router is given."""
    if router is None and bias is not None:
        raise ValueError("a selection bias needs a router (RouterSpec)")
    with M._on(logits.device, stream):
        if router is not None:
            return M.moe_route_scored(logits, x, k, chunk_size, router, bias=bias)
        return M.moe_route_permute(logits, x, k, chunk_size)


def check_weights(w_gu: QWeightT | M.Fp8WeightT, w_d: QWeightT | M.Fp8WeightT):
    if isinstance(w_gu, M.Fp8WeightT) != isinstance(w_d, M.Fp8WeightT):
        raise ValueError("w_gu and w_d: both 4-bit or both FP8 (the rows between them have one format)")


def forward(x: torch.Tensor, logits: torch.Tensor, w_gu: QWeightT | M.Fp8WeightT,
            w_d: QWeightT | M.Fp8WeightT, k: int, chunk_size: int, adapter: torch.Tensor | None = None,
            train: bool = False, stream=None, gather: bool | None = None,
            router: M.RouterSpec | None = None, bias: torch.Tensor | None = None) -> dict:
    T = x.shape[0]
    check_weights(w_gu, w_d)
    fp8 = isinstance(w_gu, M.Fp8WeightT)
    if fp8 and (adapter is not None or gather):
        raise ValueError("FP8 experts take neither an adapter nor gather (their rows are written quantized)")
    scored = dict(router=router, logits=logits if router is not None else None)
    with M._on(x.device, stream):
        if fp8:
            r = route(logits, None, k, chunk_size, router, bias)
            a = M.moe_quantize_fp8_rows(x, r)
            h, saved = M.moe_grouped_fp8_gemm_fwd(a, w_gu, r, M.EPI_SWIGLU, save_gu=train)
            y_perm = M.moe_grouped_fp8_gemm_fwd(h, w_d, r)
            y = M.moe_unpermute_combine(y_perm, r, r.gates, T, mode=0)
            return dict(routing=r, x=x, a=a, a_rows=None, h=h, saved_gu=saved, y_perm=y_perm, y=y, **scored)
        if gather is None:
            gather = adapter is not None
        r = route(logits, None if gather else x, k, chunk_size, router, bias)
        a, a_rows = (x, r.perm_token) if gather else (r.x_perm, None)
        h, saved = M.moe_grouped_qgemm_fwd(a, w_gu, r, M.EPI_SWIGLU, adapter=adapter,
                                           save_gu=train, a_rows=a_rows)
        y_perm = M.moe_grouped_qgemm_fwd(h, w_d, r, M.EPI_NONE)
        y = M.moe_unpermute_combine(y_perm, r, r.gates, T, mode=0)
        return dict(routing=r, x=x, a=a, a_rows=a_rows, h=h, saved_gu=saved, y_perm=y_perm, y=y, **scored)


def backward(state: dict, dy: torch.Tensor, w_gu: QWeightT | M.Fp8WeightT, w_d: QWeightT | M.Fp8WeightT,
             adapter: torch.Tensor | None = None, stream=None) -> dict:
    """Gradients of the step; with a router also d_gates [T, k] and d_logits [T, E]."""
    r: M.Routing = state["routing"]
    T = dy.shape[0]
    check_weights(w_gu, w_d)
    fp8 = isinstance(w_gu, M.Fp8WeightT)
    if fp8 and adapter is not None:
        raise ValueError("FP8 experts take no adapter")
    if fp8 and state["saved_gu"] is None:
        raise ValueError("backward needs a forward with train=True")
    with M._on(dy.device, stream):
        d_gates = d_logits = None
        if state.get("router") is not None:
            dy_perm, d_gates = M.moe_combine_bwd(dy, state["y_perm"], r)
            d_logits = M.moe_route_scored_bwd(d_gates, state["logits"], r, state["router"])
        else:
            dy_perm = M.moe_unpermute_combine(dy, r, r.gates, T, mode=1)
        if fp8:
            d = M.moe_quantize_fp8_rows(dy_perm)
            dgu = M.moe_grouped_fp8_gemm_bwd_dx(d, w_d, r, M.EPI_SWIGLU_BWD, saved=state["saved_gu"])
            dx_perm = M.moe_grouped_fp8_gemm_bwd_dx(dgu, w_gu, r)
            dx = M.moe_unpermute_combine(dx_perm, r, None, T, mode=0)
            return dict(dy_perm=dy_perm, dgu=dgu, dx_perm=dx_perm, dx=dx, d_adapter=None, d_gates=d_gates,
                        d_logits=d_logits)
        dgu = M.moe_grouped_qgemm_bwd_dx(dy_perm, w_d, r, M.EPI_SWIGLU_BWD, saved_gu=state["saved_gu"])
        if adapter is not None:
            dx_perm, d_adapter = M.moe_grouped_qgemm_bwd_dx(dgu, w_gu, r, M.EPI_NONE, adapter=adapter,
                                                            a=state["a"], a_rows=state["a_rows"])
        else:
            dx_perm = M.moe_grouped_qgemm_bwd_dx(dgu, w_gu, r, M.EPI_NONE)
            d_adapter = None
        dx = M.moe_unpermute_combine(dx_perm, r, None, T, mode=0)
        return dict(dy_perm=dy_perm, dgu=dgu, dx_perm=dx_perm, dx=dx, d_adapter=d_adapter, d_gates=d_gates,
                    d_logits=d_logits)


def up_projection(x: torch.Tensor, logits: torch.Tensor, w_up: QWeightT, k: int, chunk_size: int,
                  stream=None, gather: bool = False) -> dict:
    with M._on(x.device, stream):
        r = M.moe_route_permute(logits, None if gather else x, k, chunk_size)
        a, a_rows = (x, r.perm_token) if gather else (r.x_perm, None)
        out = M.moe_grouped_qgemm_fwd(a, w_up, r, M.EPI_NONE, a_rows=a_rows)
        return dict(routing=r, a=a, a_rows=a_rows, out=out)
