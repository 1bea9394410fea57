"""Measured cases of the INT8 feed-forward operators: the gated front and the
routed expert layer (a mixture of experts), both on 8-bit integer weights with a
scale for each output channel and activations quantised to 8 bits with a scale
for each token.

  glu   s = max |x| / 127, q = rne(x / s)                     (each token)
        g, u = (q W13^T) s ws  for rows 0..I-1 and I..2I-1;  y = act(g) * u
  moe   ids, gw = the topk largest router logits of each token (ties to the
        lower expert) and their softmax, over the selected ones or over all
        experts; or ids and gw as given, where an id outside the experts
        contributes nothing
        h = glu of the token with each of its experts, quantised again;
        y = sum_j gw[j] * (hq W2^T) hs ws2

The hidden values between the two products are 16-bit, as they are between two
dense layers.  ``own`` false: plain torch in 32 bits, rounded once at the end.
``own`` true: the calls a user makes of skinny_gemm_qlin_amd.
"""
import math

import torch

own = False

_ql = None


def _lib():
    global _ql
    if _ql is None:
        import skinny_gemm_qlin_amd as ql
        _ql = ql
    return _ql


def _glu(name, m, i, k, dtype, **more):
    c = {"name": name, "op": "glu", "m": m, "i": i, "k": k, "dtype": dtype, "pad": 0, "act": "silu"}
    c.update(more)
    return c


def _moe(name, m, e, topk, h, i, dtype, **more):
    c = {"name": name, "op": "moe", "m": m, "e": e, "topk": topk, "k": h, "i": i, "dtype": dtype, "pad": 0,
         "act": "silu", "route": "selected", "given": False}
    c.update(more)
    return c


def listed():
    return [
        # one token through a small front: launch and call latency
        _glu("glu-1-small", 1, 512, 1024, "bf16"),
        # one token through a decode layer's front
        _glu("glu-1-decode", 1, 14336, 4096, "bf16"),
        # a ragged decode batch, odd width, long rows, padded pitches, gelu
        _glu("glu-5-odd", 5, 2051, 14336, "bf16", pad=32, act="gelu"),
        # a full decode batch, fp16
        _glu("glu-16-decode", 16, 8704, 5120, "fp16"),
        # a prompt of odd length
        _glu("glu-509-prompt", 509, 4096, 7168, "bf16"),
        # a long prompt
        _glu("glu-2048-prompt", 2048, 14336, 4096, "bf16"),
        # one token through a layer of a few small experts: latency
        _moe("moe-1-small", 1, 8, 2, 1024, 512, "bf16"),
        # one token through the expert layer this repository's benchmark uses
        _moe("moe-1-decode", 1, 64, 6, 7168, 2048, "bf16"),
        # a decode batch through the same layer
        _moe("moe-8-decode", 8, 64, 6, 7168, 2048, "fp16"),
        # a padded batch over many narrow experts: routing given, some tokens have none
        _moe("moe-13-given", 13, 128, 8, 2064, 752, "bf16", pad=32, given=True, act="gelu"),
        # a large decode batch over the narrow experts, weights of the softmax over all experts
        _moe("moe-64-decode", 64, 128, 8, 2048, 768, "bf16", route="all"),
        # a prompt through the expert layer of the benchmark
        _moe("moe-1000-prompt", 1000, 64, 6, 7168, 2048, "bf16"),
    ]


_MOST_FLOPS = 6.0 * 1000 * 6 * 7168 * 2048
_MOST_BYTES = 3.0 * 64 * 7168 * 2048


def draw(rng):
    def spread(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    def m_of(hi):
        return spread(1, 16) if rng.random() < 0.5 else spread(17, hi)

    c = {"op": rng.choice(["glu", "moe"]), "dtype": rng.choice(["bf16", "fp16"]), "pad": rng.choice([0, 0, 32]),
         "act": rng.choice(["silu", "silu", "gelu"])}
    if c["op"] == "glu":
        c.update(m=m_of(4096), i=spread(128, 16384), k=spread(32, 1024) * 16)
        while 4.0 * c["m"] * c["i"] * c["k"] > _MOST_FLOPS and c["m"] > 1:
            c["m"] = c["m"] * 3 // 4
        return c
    c.update(m=m_of(1024), e=spread(4, 128), k=spread(32, 448) * 16, i=spread(16, 256) * 16,
             route=rng.choice(["selected", "all"]), given=rng.random() < 0.3)
    c["topk"] = rng.randint(1, min(8, c["e"]))
    while 3.0 * c["e"] * c["k"] * c["i"] > _MOST_BYTES:
        c["i"] = max(16, c["i"] * 3 // 4 // 16 * 16)
    while 6.0 * c["m"] * c["topk"] * c["k"] * c["i"] > _MOST_FLOPS and c["m"] > 1:
        c["m"] = c["m"] * 3 // 4
    return c


_DT = {"bf16": torch.bfloat16, "fp16": torch.float16}


def _codes(shape, cols, pad, gen):
    """int8 weight codes in rows of `cols`, `pad` more bytes from row to row."""
    w = torch.randint(-127, 128, (*shape, cols + pad), dtype=torch.int8, device="cuda", generator=gen)
    return w[..., :cols]


def _scales(shape, cols, gen):
    """Channel scales that put the weights' standard deviation near 1 / sqrt(cols)."""
    s = torch.empty(shape, dtype=torch.float32, device="cuda").uniform_(0.5, 1.5, generator=gen)
    return s / (73.0 * math.sqrt(cols))


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    dt, m, k, i, pad = _DT[case["dtype"]], case["m"], case["k"], case["i"], case["pad"]
    # normalised activations: near one, tokens of different size
    x = torch.empty((m, (k + 7) // 8 * 8 + pad), dtype=torch.float32, device="cuda").normal_(0.0, 1.0, generator=gen)
    x *= torch.empty((m, 1), dtype=torch.float32, device="cuda").uniform_(0.5, 2.0, generator=gen)
    st = {"case": dict(case), "x": x.to(dt)[:, :k]}
    if case["op"] == "glu":
        st["w13"] = _codes((2 * i,), k, pad // 16 * 16, gen)
        st["s13"] = _scales((2 * i,), k, gen)
        st["y"] = torch.empty((m, i), dtype=dt, device="cuda")
        st["xq"] = torch.empty((m, k), dtype=torch.int8, device="cuda")
        st["xs"] = torch.empty((m,), dtype=torch.float32, device="cuda")
        return st
    e, topk = case["e"], case["topk"]
    st["w13"], st["s13"] = _codes((e, 2 * i), k, 0, gen), _scales((e, 2 * i), k, gen)
    st["w2"], st["s2"] = _codes((e, k), i, 0, gen), _scales((e, k), i, gen)
    logits = torch.empty((m, e), dtype=torch.float32, device="cuda").normal_(0.0, 1.5, generator=gen)
    st["y"] = torch.empty((m, k), dtype=dt, device="cuda")
    st["logits"] = None if case["given"] else logits
    if case["given"]:
        # a router of the user's own; every fourth token is padding, and so is the odd slot
        order = torch.argsort(logits, dim=1, descending=True)[:, :topk].to(torch.int32)
        drop = torch.rand((m, topk), device="cuda", generator=gen) < 0.05
        drop |= (torch.arange(m, device="cuda") % 4 == 3)[:, None]
        st["ids"] = torch.where(drop, torch.full_like(order, -1), order).contiguous()
        st["gw"] = torch.rand((m, topk), dtype=torch.float32, device="cuda", generator=gen) / topk
    else:
        st["ids"] = torch.empty((m, topk), dtype=torch.int32, device="cuda")
        st["gw"] = torch.empty((m, topk), dtype=torch.float32, device="cuda")
    st["workspace"] = None
    if own:  # kept from call to call, as a serving loop keeps it
        need = _lib().qlin_moe_ffn_i8_workspace_bytes(m, k, i, topk, e)
        st["workspace"] = torch.empty((need,), dtype=torch.uint8, device="cuda")
    return st


def _act(g, act):
    if act == "silu":
        return g / (1.0 + torch.exp(-g))
    return 0.5 * g * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (g + 0.044715 * g * g * g)))


def _quant(x):
    """32-bit values -> whole-number codes and the scale of each row."""
    s = x.abs().amax(dim=1, keepdim=True) / 127.0
    return torch.where(s > 0, torch.round(x / s).clamp(-127.0, 127.0), torch.zeros_like(x)), s


def _front(q, s, w13, s13, i, act):
    gu = (q @ w13.float().t()) * s * s13
    return _act(gu[:, :i], act) * gu[:, i:]


def _run_plain(st):
    c = st["case"]
    dt, i = _DT[c["dtype"]], c["i"]
    q, s = _quant(st["x"].float())
    if c["op"] == "glu":
        return _front(q, s, st["w13"], st["s13"], i, c["act"]).to(dt)
    ids, gw = st["ids"], st["gw"]
    if st["logits"] is not None:
        top, order = torch.sort(st["logits"], dim=1, descending=True, stable=True)
        ids, top = order[:, :c["topk"]], top[:, :c["topk"]]
        each = torch.exp(top - top[:, :1])
        gw = each / (torch.exp(st["logits"] - top[:, :1]) if c["route"] == "all" else each).sum(dim=1, keepdim=True)
        ids = ids.to(torch.int32)
    y = torch.zeros((c["m"], c["k"]), dtype=torch.float32, device="cuda")
    for e in torch.unique(ids).tolist():
        if not 0 <= e < c["e"]:
            continue
        t, j = torch.where(ids == e)
        h = _front(q[t], s[t], st["w13"][e], st["s13"][e], i, c["act"]).to(dt).float()
        hq, hs = _quant(h)
        y.index_add_(0, t, gw[t, j, None] * ((hq @ st["w2"][e].float().t()) * hs * st["s2"][e]))
    y = y.to(dt)
    return y if st["logits"] is None else (y, ids, gw)


def _run_own(st):
    ql, c = _lib(), st["case"]
    act = ql.QLIN_ACT_SILU if c["act"] == "silu" else ql.QLIN_ACT_GELU_TANH
    if c["op"] == "glu":
        return ql.qlin_glu_i8(st["x"], st["w13"], st["s13"], act=act, xq=st["xq"], xs=st["xs"], y=st["y"])[0]
    route = ql.QLIN_ROUTE_ALL if c["route"] == "all" else ql.QLIN_ROUTE_SELECTED
    y, ids, gw = ql.qlin_moe_ffn_i8(st["x"], st["w13"], st["s13"], st["w2"], st["s2"], logits=st["logits"],
                                    topk=c["topk"], route=route, act=act, ids=st["ids"], gw=st["gw"], y=st["y"],
                                    workspace=st["workspace"])
    return y if st["logits"] is None else (y, ids, gw)


def run(state):
    return _run_own(state) if own else _run_plain(state)


def work(case):
    m, k, i = case["m"], case["k"], case["i"]
    if case["op"] == "glu":
        return {"bytes": 2.0 * i * (k + 4) + 2.0 * m * (k + i), "flops": 4.0 * m * i * k}
    e, topk = case["e"], case["topk"]
    tokens = m - m // 4 if case["given"] else m
    live = e * (1.0 - (1.0 - topk / e) ** tokens)  # experts that a token of the batch goes to, on average
    return {"bytes": live * (3.0 * k * i + 8.0 * i + 4.0 * k) + 4.0 * m * k + (0 if case["given"] else 4.0 * m * e)
            + 8.0 * m * topk, "flops": 6.0 * tokens * topk * k * i}


def _exact_codes(x):
    """Codes and scale of each row of 16-bit values: the scale and the quotient are 32-bit numbers, as defined."""
    s = (x.abs().max(dim=1).values / 127.0).float().double()
    quotient = (x / torch.where(s > 0, s, torch.ones_like(s))[:, None]).float().double()
    return torch.clamp(torch.round(quotient), min=-127, max=127), s


def _exact_act(g, act):
    if act == "silu":
        return g * torch.sigmoid(g)
    # 0.5 (1 + tanh(z)) = sigmoid(2 z)
    return g * torch.sigmoid(math.sqrt(8.0 / math.pi) * (g + 0.044715 * g ** 3))


def _exact_front(q, s, w13, s13, act):
    """In 64 bits, a block of columns at a time."""
    i, out = w13.shape[0] // 2, []
    for a in range(0, i, 4096):
        b = min(i, a + 4096)
        gate = torch.mm(q, w13[a:b].double().t().contiguous()) * s13[a:b].double() * s[:, None]
        up = torch.mm(q, w13[i + a:i + b].double().t().contiguous()) * s13[i + a:i + b].double() * s[:, None]
        out.append(_exact_act(gate, act) * up)
    return torch.cat(out, dim=1)


def exact(case, seed):
    st = prepare(case, seed)
    dt = _DT[case["dtype"]]
    q, s = _exact_codes(st["x"].double())
    if case["op"] == "glu":
        return _exact_front(q, s, st["w13"], st["s13"], case["act"])
    m, topk = case["m"], case["topk"]
    ids, gw = st["ids"], st["gw"].double()
    if st["logits"] is not None:
        lg = st["logits"].double()
        at = torch.arange(case["e"], device="cuda")
        # place of each expert: how many are ahead of it
        ahead = (lg[:, None, :] > lg[:, :, None]) | ((lg[:, None, :] == lg[:, :, None]) & (at[None, :] < at[:, None]))
        place = ahead.sum(dim=2)
        ids = torch.stack([(place == j).int().argmax(dim=1) for j in range(topk)], dim=1)
        share = torch.softmax(lg, dim=1)
        gw = torch.gather(share, 1, ids)
        if case["route"] != "all":
            gw = gw / gw.sum(dim=1, keepdim=True)
        ids = ids.to(torch.int32)
    per_slot = torch.zeros((m, topk, case["k"]), dtype=torch.float64, device="cuda")
    for e in range(case["e"]):
        t, j = torch.nonzero(ids == e, as_tuple=True)
        if len(t) == 0:
            continue
        h = _exact_front(q[t], s[t], st["w13"][e], st["s13"][e], case["act"])
        hq, hs = _exact_codes(h.to(dt).double())
        per_slot[t, j] = torch.mm(hq, st["w2"][e].double().t().contiguous()) * st["s2"][e].double() * hs[:, None]
    y = (per_slot * gw[:, :, None]).sum(dim=1)
    return y if st["logits"] is None else (y, ids, gw)
