"""Cases of the MoE layer's router, its gradient, and the FP8 expert products.

Five operators, each in a plain torch form (`own` false) and as the calls a
user makes of quantized_rl_fine_b200.moeq (`own` true):

  route        moe_route_scored: scores, bias, expert groups, top-k, gates and
               the group tables of the grouped products
  router_grad  moe_combine_bwd and moe_route_scored_bwd: from dy to the
               gradient of the per-slot rows, of the gates and of the logits
  experts      moe_quantize_fp8_rows and moe_grouped_fp8_gemm_fwd: BF16 token
               rows to FP8 rows in expert order, times the FP8 expert weights
  glu          the same with the SwiGLU epilogue: FP8 rows out, and the gate|up
               activations kept as an 8-bit checkpoint
  grad         moe_grouped_fp8_gemm_bwd_dx: activation gradients through the
               same weights, plain or with the SwiGLU backward from the checkpoint

Formats. FP8 rows: e4m3 with one power-of-two scale per 128 elements, the
smallest 2^e >= 2^-126 with amax <= 448 * 2^e (1 for a block of zeros). FP8 weights: e4m3
with one fp32 scale per 128 x 128 block. Checkpoint: e4m3 with one E8M0 scale
2^(X-127) per 32 elements, chosen by the same rule. e4m3 times a power of two
is a BF16 number, so what is held in 8 bits is returned as BF16 values.
"""

import math

import torch

own = False

DEV = "cuda"


# --------------------------------------------------------------------------
# Cases
# --------------------------------------------------------------------------

def _route(T, E, k, score, groups=1, topk_groups=1, group_top=1, bias=False, renorm=True,
           scale=1.0, spread=1.0):
    return dict(op="route", T=T, E=E, k=k, score=score, groups=groups, topk_groups=topk_groups,
                group_top=group_top, bias=bias, renorm=renorm, scale=scale, spread=spread)


def _router_grad(T, E, k, D, score, renorm, scale=1.0):
    return dict(op="router_grad", T=T, E=E, k=k, D=D, score=score, renorm=renorm, scale=scale)


def _product(op, T, k, E, K, N, spread=1.0, **kw):
    return dict(op=op, T=T, k=k, E=E, K=K, N=N, spread=spread, **kw)


def listed():
    return [
        # One decoded token through the router of a 384-expert layer.
        dict(_route(1, 384, 8, "sigmoid", 8, 4, 2, bias=True, scale=2.5), name="route_token"),
        # A training micro-batch with balance bias and group-limited selection.
        dict(_route(4096, 256, 8, "sigmoid", 8, 4, 2, bias=True, scale=2.5), name="route_batch"),
        # The longest prompt batch of the 384-expert layer, plain softmax scores.
        dict(_route(16384, 384, 8, "softmax", renorm=False), name="route_prompt"),
        # Router gradient of the training step (T = 4096 rows of 7168).
        dict(_router_grad(4096, 384, 8, 7168, "sigmoid", True, 2.5), name="router_grad_train"),
        # Small fine-tuning batch: softmax scores without renormalisation, odd token count.
        dict(_router_grad(131, 64, 4, 2048, "softmax", False), name="router_grad_small"),
        # Decode: one token, eight experts out of the 48 a rank holds; weight stream only.
        dict(_product("experts", 1, 8, 48, 7168, 4096), name="experts_token"),
        # Ragged everything: experts of a few rows, sizes that end inside a block.
        dict(_product("experts", 509, 3, 21, 1040, 1392, spread=1.5), name="experts_ragged"),
        # Down projection of a long prompt batch.
        dict(_product("experts", 8192, 8, 48, 2048, 7168), name="experts_prompt"),
        # Decode batch through gate/up and SwiGLU, nothing saved.
        dict(_product("glu", 16, 8, 48, 7168, 4096, save=False), name="glu_decode"),
        # Training step: gate/up, SwiGLU and the 8-bit checkpoint.
        dict(_product("glu", 4096, 8, 48, 7168, 4096, save=True), name="glu_train"),
        # Its backward: dy through the down projection and the SwiGLU from the checkpoint.
        dict(_product("grad", 4096, 8, 48, 2048, 7168, glu=True), name="grad_glu_train"),
        # Activation gradient of a gate/up projection, mid-sized experts.
        dict(_product("grad", 1000, 4, 64, 2048, 2048, glu=False), name="grad_batch"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["route", "router_grad", "experts", "glu", "grad"])
    if op == "route":
        per = rng.choice([4, 5, 8, 16, 32, 48])
        groups = rng.choice([1, 2, 4, 8])
        E = per * groups
        tg = rng.randint(1, groups)
        k = rng.randint(1, min(8, per * tg))
        score = rng.choice(["softmax", "sigmoid"])
        return _route(_log(rng, 1, 16384), E, k, score, groups, tg, rng.choice([1, 2]),
                      rng.random() < 0.6, rng.random() < 0.6, rng.choice([1.0, 1.5, 2.5]),
                      rng.choice([0.5, 1.0, 2.0]))
    if op == "router_grad":
        E = rng.choice([8, 21, 64, 100, 256, 384])
        k = rng.randint(1, min(8, E))
        # one renormalised gate is constant: its gradient is rounding noise around zero
        return _router_grad(_log(rng, 1, 4096), E, k, 8 * _log(rng, 8, 896),
                            rng.choice(["softmax", "sigmoid"]), k > 1 and rng.random() < 0.6,
                            rng.choice([1.0, 2.5]))
    E = rng.randint(3, 48)
    k = rng.randint(1, min(8, E))
    T = _log(rng, 1, 4096)
    spread = rng.choice([0.0, 1.0, 1.5])
    if op == "experts":
        return _product(op, T, k, E, 16 * _log(rng, 8, 256), 16 * _log(rng, 8, 256), spread)
    if op == "glu":
        return _product(op, T, k, E, 16 * _log(rng, 8, 256), 256 * _log(rng, 1, 16), spread,
                        save=rng.random() < 0.5)
    glu = rng.random() < 0.5
    K = 128 * _log(rng, 1, 16) if glu else 16 * _log(rng, 8, 256)
    return _product(op, T, k, E, K, 16 * _log(rng, 8, 256), spread, glu=glu)


def work(case):
    T, k, E = case["T"], case["k"], case["E"]
    M = T * k
    if case["op"] == "route":
        return {"bytes": 4 * T * E + 16 * M + 8 * E, "flops": 8 * T * E}
    if case["op"] == "router_grad":
        D = case["D"]
        logits = 4 * T * E if case["score"] == "softmax" else 4 * M
        return {"bytes": 2 * T * D + 4 * M * D + 16 * M + logits + 4 * T * E, "flops": 3 * M * D}
    K, N = case["K"], case["N"]
    # experts that get rows at all: at most one per row
    wb = min(E, M) * N * K
    if case["op"] == "experts":
        b = 2 * T * K + wb + 2 * M * N + 4 * M
    elif case["op"] == "glu":
        b = 2 * T * K + wb + M * N // 2 + 4 * M + (M * N + M * N // 32 if case["save"] else 0)
    else:
        b = 2 * M * N + wb + (4 * M * K + M * K // 16 if case["glu"] else 2 * M * K)
    return {"bytes": b, "flops": 2 * M * N * K}


# --------------------------------------------------------------------------
# Inputs
# --------------------------------------------------------------------------

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(1000003 * (seed + 1))
    return g


def _tables(topk, E, chunk=8):
    """Group tables of a selection [T, k], as the routing writes them."""
    T, k = topk.shape
    flat = topk.reshape(-1)
    order = torch.sort(flat, stable=True).indices
    counts = torch.bincount(flat, minlength=E)
    offsets = torch.zeros(E + 1, dtype=torch.int64, device=DEV)
    offsets[1:] = counts.cumsum(0)
    inv = torch.empty_like(flat)
    inv[order] = torch.arange(T * k, device=DEV)
    act = torch.nonzero(counts).reshape(-1)
    active = torch.zeros(E, dtype=torch.int64, device=DEV)
    active[: act.numel()] = act
    n = act.numel()
    nch = -(-n // chunk)
    chunks = torch.clamp(torch.arange(E + 1, device=DEV) * chunk, max=n)
    i32 = lambda t: t.to(torch.int32).contiguous()  # noqa: E731
    return dict(topk=i32(topk), offsets=i32(offsets), active=i32(active),
                num_active=torch.tensor([n], dtype=torch.int32, device=DEV), chunks=i32(chunks),
                num_chunks=torch.tensor([nch], dtype=torch.int32, device=DEV),
                perm_token=i32(order // k), inv_perm=i32(inv), most=int(counts.max()), n_active=n)


def _weights(g, E, N, K):
    """Expert weights N(0, 0.02) in e4m3 with one fp32 scale amax / 448 per 128 x 128 block."""
    nb, kb = -(-N // 128), -(-K // 128)
    wq = torch.empty((E, N, K), dtype=torch.float8_e4m3fn, device=DEV)
    ws = torch.empty((E, nb, kb), dtype=torch.float32, device=DEV)
    for e0 in range(0, E, 8):
        n = min(8, E - e0)
        w = torch.zeros((n, nb * 128, kb * 128), device=DEV)
        w[:, :N, :K] = torch.randn((n, N, K), generator=g, device=DEV) * 0.02
        w = w.view(n, nb, 128, kb, 128)
        s = w.abs().amax((2, 4)) / 448.0
        q = (w / s[:, :, None, :, None]).view(n, nb * 128, kb * 128)[:, :N, :K]
        wq[e0:e0 + n] = q.to(torch.float8_e4m3fn)
        ws[e0:e0 + n] = s
    return wq, ws


def prepare(case, seed):
    g = _gen(seed)
    T, k, E = case["T"], case["k"], case["E"]
    rnd = lambda *s: torch.randn(s, generator=g, device=DEV)  # noqa: E731
    st = dict(case)
    if case["op"] == "route":
        st["logits"] = rnd(T, E) * case["spread"]
        st["bias_t"] = rnd(E) * 0.1 if case["bias"] else None
        return st
    if case["op"] == "router_grad":
        st["logits"] = rnd(T, E)
        topk = st["logits"].topk(k, dim=1).indices
        st["tables"] = _tables(topk, E)
        s = _scores(st["logits"], case["score"]).gather(1, topk)
        w = case["scale"] * (s / s.sum(1, keepdim=True) if case["renorm"] else s)
        st["gates"] = w.float().contiguous()
        st["dy"] = rnd(T, case["D"]).to(torch.bfloat16)
        st["rows"] = (0.1 * rnd(T * k, case["D"])).to(torch.bfloat16)
        return st
    K, N = case["K"], case["N"]
    # popularity of the experts: none, or a normal spread of their logits
    lg = rnd(T, E) + case["spread"] * 0.3 * rnd(E)
    st["tables"] = _tables(lg.topk(k, dim=1).indices, E)
    st["wq"], st["ws"] = _weights(g, E, N, K)
    if case["op"] in ("experts", "glu"):
        st["x"] = rnd(T, K).to(torch.bfloat16)
    else:
        st["dout"] = rnd(T * k, N).to(torch.bfloat16)
        if case["glu"]:
            gu = rnd(T * k, 2 * K).to(torch.bfloat16).float()
            e = _block_exp(gu, 32)
            st["ck_q"] = _to_e4m3(gu, e, 32)
            st["ck_s"] = (e + 127).to(torch.uint8).t().contiguous()
    return st


# --------------------------------------------------------------------------
# Plain form
# --------------------------------------------------------------------------

def _scores(logits, score):
    """Scores in 64 bits: selections compare scores that may lie next to each other."""
    x = logits.double()
    if score == "sigmoid":
        return 1.0 / (1.0 + torch.exp(-x))
    z = torch.exp(x - x.amax(1, keepdim=True))
    return z / z.sum(1, keepdim=True)


def _block_exp(v, block):
    """Exponent e of each block's scale 2^e: the smallest with amax <= 448 * 2^e."""
    M, K = v.shape
    nb = -(-K // block)
    p = torch.zeros((M, nb * block), device=v.device)
    p[:, :K] = v
    amax = p.view(M, nb, block).abs().amax(2)
    m, ex = torch.frexp(amax)                       # amax = m * 2^ex, m in [0.5, 1); 448 = 0.875 * 2^9
    e = torch.where(m <= 0.875, ex - 9, ex - 8)
    return torch.where(amax == 0, torch.zeros_like(e), e.clamp(min=-126))


def _spread(s, K, block):
    return s.repeat_interleave(block, dim=1)[:, :K]


def _to_e4m3(v, e, block):
    return torch.ldexp(v, -_spread(e, v.shape[1], block)).to(torch.float8_e4m3fn)


def _quantized(v, block):
    """The values that v's e4m3 blocks stand for, in fp32."""
    v = v.float()
    e = _block_exp(v, block)
    return torch.ldexp(_to_e4m3(v, e, block).float(), _spread(e, v.shape[1], block))


def _weight_values(st):
    """The weights of the experts that have rows, in fp32."""
    N, K = st["N"], st["K"]
    act = st["tables"]["active"][: st["tables"]["n_active"]].long()
    s = st["ws"][act].repeat_interleave(128, dim=1)[:, :N].repeat_interleave(128, dim=2)[:, :, :K]
    return st["wq"].view(torch.uint8)[act].view(torch.float8_e4m3fn).float() * s


def _per_expert(a, w, st):
    """Rows a [M, R] times their expert's w [active, R, F]: experts padded to the longest one."""
    tb, n, most = st["tables"], st["tables"]["n_active"], st["tables"]["most"]
    p = torch.arange(a.shape[0], device=a.device)
    first = tb["offsets"].long()[tb["active"][:n].long()]
    i = torch.searchsorted(first, p, right=True) - 1
    slot = i * most + p - first[i]
    pad = torch.zeros((n * most, a.shape[1]), device=a.device)
    pad[slot] = a
    return torch.bmm(pad.view(n, most, -1), w).view(n * most, -1)[slot]


def _route_plain(st):
    T, E, k, G = st["T"], st["E"], st["k"], st["groups"]
    s = _scores(st["logits"], st["score"])
    key = s if st["bias_t"] is None else s + st["bias_t"].double()
    if G > 1:
        by = key.view(T, G, E // G)
        best = torch.sort(by, dim=2, descending=True).values[:, :, : st["group_top"]].sum(2)
        kept = torch.sort(best, dim=1, descending=True, stable=True).indices[:, : st["topk_groups"]]
        open_ = torch.zeros((T, G), dtype=torch.bool, device=DEV).scatter_(1, kept, True)
        key = torch.where(open_[:, :, None].expand(T, G, E // G).reshape(T, E), key, -math.inf)
    topk = torch.sort(key, dim=1, descending=True, stable=True).indices[:, :k]
    w = s.gather(1, topk)
    if st["renorm"]:
        w = w / w.sum(1, keepdim=True)
    flat = topk.reshape(-1)
    order = torch.sort(flat, stable=True).indices
    inv = torch.empty_like(flat)
    inv[order] = torch.arange(T * k, device=DEV)
    offsets = torch.zeros(E + 1, dtype=torch.int32, device=DEV)
    counts = torch.zeros(E, dtype=torch.int32, device=DEV).scatter_add_(
        0, flat, torch.ones_like(flat, dtype=torch.int32))
    offsets[1:] = counts.cumsum(0)
    return dict(topk=topk.int(), gates=(st["scale"] * w).float(), offsets=offsets,
                perm_token=(order // k).int(), inv_perm=inv.int(),
                num_active=(counts > 0).sum().int().reshape(1))


def _router_grad_plain(st):
    T, k, D = st["T"], st["k"], st["D"]
    tb = st["tables"]
    inv = tb["inv_perm"].long()
    dy = st["dy"].float()
    by_slot = st["rows"][inv].float().view(T, k, D)
    d_gates = (by_slot * dy[:, None, :]).sum(2)
    d_rows = torch.empty((T * k, D), dtype=torch.bfloat16, device=DEV)
    d_rows[inv] = (st["gates"][:, :, None] * dy[:, None, :]).reshape(T * k, D).to(torch.bfloat16)
    p = _scores(st["logits"], st["score"])
    idx = tb["topk"].long()
    s, dw = p.gather(1, idx), d_gates.double() * st["scale"]
    if st["renorm"]:
        total = s.sum(1, keepdim=True)
        ds = (dw - (dw * s).sum(1, keepdim=True) / total) / total
    else:
        ds = dw
    d_s = torch.zeros_like(p).scatter_(1, idx, ds)
    if st["score"] == "sigmoid":
        d_logits = d_s * p * (1.0 - p)
    else:
        d_logits = p * (d_s - (d_s * p).sum(1, keepdim=True))
    return dict(d_rows=d_rows, d_gates=d_gates, d_logits=d_logits.float())


def _plain(st):
    op = st["op"]
    if op == "route":
        return _route_plain(st)
    if op == "router_grad":
        return _router_grad_plain(st)
    w = _weight_values(st)
    if op == "experts":
        a = _quantized(st["x"], 128)[st["tables"]["perm_token"].long()]
        return _per_expert(a, w.transpose(1, 2), st).to(torch.bfloat16)
    if op == "glu":
        a = _quantized(st["x"], 128)[st["tables"]["perm_token"].long()]
        gu = _per_expert(a, w.transpose(1, 2), st)
        f = st["N"] // 2
        h = gu[:, :f] / (1.0 + torch.exp(-gu[:, :f])) * gu[:, f:]
        out = dict(h=_quantized(h, 128).to(torch.bfloat16))
        if st["save"]:
            out["saved"] = _quantized(gu, 32).to(torch.bfloat16)
        return out
    d = _per_expert(_quantized(st["dout"], 128), w, st)
    if not st["glu"]:
        return d.to(torch.bfloat16)
    K = st["K"]
    e = st["ck_s"].t().int() - 127
    gu = torch.ldexp(st["ck_q"].float(), _spread(e, 2 * K, 32))
    g, u = gu[:, :K], gu[:, K:]
    s = 1.0 / (1.0 + torch.exp(-g))
    # dg and du are BF16 tensors that are then quantized
    dgu = torch.cat([d * u * s * (1.0 + g * (1.0 - s)), d * g * s], 1).to(torch.bfloat16)
    return _quantized(dgu, 128).to(torch.bfloat16)


# --------------------------------------------------------------------------
# The framework's calls
# --------------------------------------------------------------------------

def _routing(M, st, gates=None):
    tb = st["tables"]
    return M.Routing(topk_idx=tb["topk"], gates=gates, expert_offsets=tb["offsets"],
                     active=tb["active"], num_active=tb["num_active"], chunk_offsets=tb["chunks"],
                     num_chunks=tb["num_chunks"], perm_token=tb["perm_token"],
                     inv_perm=tb["inv_perm"], x_perm=None, E=st["E"], k=st["k"])


def _own(st):
    from quantized_rl_fine_b200 import moeq as M
    op = st["op"]
    if op == "route":
        spec = M.RouterSpec(score=st["score"], groups=st["groups"], topk_groups=st["topk_groups"],
                            group_top=st["group_top"], renorm=st["renorm"], scale=st["scale"])
        r = M.moe_route_scored(st["logits"], None, st["k"], 8, spec, bias=st["bias_t"])
        return dict(topk=r.topk_idx, gates=r.gates, offsets=r.expert_offsets,
                    perm_token=r.perm_token, inv_perm=r.inv_perm, num_active=r.num_active)
    if op == "router_grad":
        spec = M.RouterSpec(score=st["score"], renorm=st["renorm"], scale=st["scale"])
        r = _routing(M, st, st["gates"])
        d_rows, d_gates = M.moe_combine_bwd(st["dy"], st["rows"], r)
        d_logits = M.moe_route_scored_bwd(d_gates, st["logits"], r, spec)
        return dict(d_rows=d_rows, d_gates=d_gates, d_logits=d_logits)
    r = _routing(M, st)
    w = M.Fp8WeightT(st["wq"], st["ws"])
    if op == "experts":
        a = M.moe_quantize_fp8_rows(st["x"], r)
        return M.moe_grouped_fp8_gemm_fwd(a, w, r)
    if op == "glu":
        a = M.moe_quantize_fp8_rows(st["x"], r)
        h, saved = M.moe_grouped_fp8_gemm_fwd(a, w, r, M.EPI_SWIGLU, save_gu=st["save"])
        out = dict(h=M.moe_dequantize_fp8_rows(h))
        if st["save"]:
            out["saved"] = M.moe_dequantize_fp8_rows(saved)
        return out
    d = M.moe_quantize_fp8_rows(st["dout"])
    if not st["glu"]:
        return M.moe_grouped_fp8_gemm_bwd_dx(d, w, r)
    ck = M.Fp8Rows(st["ck_q"], st["ck_s"])
    return M.moe_dequantize_fp8_rows(M.moe_grouped_fp8_gemm_bwd_dx(d, w, r, M.EPI_SWIGLU_BWD, saved=ck))


def run(state):
    return _own(state) if own else _plain(state)


# --------------------------------------------------------------------------
# The definitions in 64 bits
# --------------------------------------------------------------------------

def _exact_blocks(v, block):
    """Values of v's e4m3 blocks from the definition: round to 4 significant bits, no finer than 2^-9 of the scale."""
    out = torch.empty_like(v)
    for c in range(0, v.shape[1], block):
        b = v[:, c:c + block]
        amax = b.abs().amax(1, keepdim=True)
        e = torch.ceil(torch.log2(torch.where(amax == 0, torch.full_like(amax, 448.0), amax) / 448.0))
        e = torch.where(amax > 448.0 * torch.exp2(e), e + 1, e)
        e = torch.where(amax <= 448.0 * torch.exp2(e - 1), e - 1, e)
        e = torch.where(amax == 0, torch.zeros_like(e), e.clamp(min=-126.0))
        y = b / torch.exp2(e)
        step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
        out[:, c:c + block] = torch.round(y / step) * step * torch.exp2(e)
    return out


def _exact_product(a, st, transposed):
    tb, K, N = st["tables"], st["K"], st["N"]
    off = tb["offsets"].tolist()
    out = torch.empty((a.shape[0], K if transposed else N), dtype=torch.float64, device=a.device)
    for e in range(st["E"]):
        lo, hi = off[e], off[e + 1]
        if hi > lo:
            s = torch.kron(st["ws"][e].double(), torch.ones((128, 128), dtype=torch.float64, device=DEV))
            w = st["wq"][e].double() * s[:N, :K]
            out[lo:hi] = a[lo:hi] @ (w if transposed else w.t())
    return out


def _exact_route(st):
    T, E, k, G = st["T"], st["E"], st["k"], st["groups"]
    x = st["logits"].double()
    s = torch.sigmoid(x) if st["score"] == "sigmoid" else torch.softmax(x, 1)
    key = s.clone()
    if st["bias_t"] is not None:
        key += st["bias_t"].double()
    n = E // G
    rank = torch.stack([key[:, g * n:(g + 1) * n].topk(min(st["group_top"], n), 1).values.sum(1)
                        for g in range(G)], 1)
    cut = rank.topk(st["topk_groups"], 1).values[:, -1:]
    for g in range(G):
        key[:, g * n:(g + 1) * n].masked_fill_(rank[:, g:g + 1] < cut, -math.inf)
    idx = key.topk(k, 1).indices
    w = s.gather(1, idx)
    if st["renorm"]:
        w = w / w.sum(1, keepdim=True)
    return dict(topk=None, gates=st["scale"] * w, offsets=None, perm_token=None, inv_perm=None,
                num_active=None)


def _exact_router_grad(st):
    T, k = st["T"], st["k"]
    inv, idx = st["tables"]["inv_perm"].long().view(T, k), st["tables"]["topk"].long()
    dy, rows = st["dy"].double(), st["rows"].double()
    d_gates = torch.stack([(rows[inv[:, j]] * dy).sum(1) for j in range(k)], 1)
    d_rows = torch.empty_like(rows)
    for j in range(k):
        d_rows[inv[:, j]] = st["gates"][:, j:j + 1].double() * dy
    with torch.enable_grad():
        x = st["logits"].double().requires_grad_()
        s = torch.sigmoid(x) if st["score"] == "sigmoid" else torch.softmax(x, 1)
        w = s.gather(1, idx)
        if st["renorm"]:
            w = w / w.sum(1, keepdim=True)
        (d_logits,) = torch.autograd.grad((st["scale"] * w * d_gates).sum(), x)
    return dict(d_rows=d_rows, d_gates=d_gates, d_logits=d_logits)


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "route":
        return _exact_route(st)
    if op == "router_grad":
        return _exact_router_grad(st)
    if op in ("experts", "glu"):
        a = _exact_blocks(st["x"].double(), 128)[st["tables"]["perm_token"].long()]
        y = _exact_product(a, st, False)
        if op == "experts":
            return y
        f = case["N"] // 2
        out = dict(h=_exact_blocks(torch.nn.functional.silu(y[:, :f]) * y[:, f:], 128))
        if case["save"]:
            out["saved"] = _exact_blocks(y, 32)
        return out
    d = _exact_product(_exact_blocks(st["dout"].double(), 128), st, True)
    if not case["glu"]:
        return d
    K = case["K"]
    s = torch.exp2(st["ck_s"].double().t() - 127.0).contiguous()
    gu = st["ck_q"].double() * torch.kron(s, torch.ones((1, 32), dtype=torch.float64, device=DEV))
    with torch.enable_grad():
        g, u = gu[:, :K].clone().requires_grad_(), gu[:, K:].clone().requires_grad_()
        dg, du = torch.autograd.grad((torch.nn.functional.silu(g) * u * d).sum(), (g, u))
    # dg and du are held in BF16 before they are quantized
    return _exact_blocks(torch.cat([dg, du], 1).to(torch.bfloat16).double(), 128)
