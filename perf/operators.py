"""Measured cases of the 4-bit weight operators: the linear layer (forward and
input gradient) and the gated feed-forward front (forward and backward).

A weight matrix W[n, k] = ws[n, k // G] * (code[n, k] - wz[n, k // G]) is held as
two 4-bit codes a byte (element 2i in the low nibble of byte i), 16-bit scales
and optional 8-bit zero points per group of G elements of a row; without zero
points the zero is 8.  The operators:

  gemv      y  = x W^T (+ bias)
  gemv_bwd  dx = dy W
  glu       g, u = x W[:I]^T, x W[I:]^T;  y = act(g) * u   (gu = [g, u] if kept)
  glu_bwd   dgu = [dy * u * act'(g), dy * act(g)];  dx = dgu W,
            with g, u read back from gu or recomputed from x

``own`` false: plain torch in 32 bits, rounded once at the end.  ``own`` true:
the calls a user makes of skinny_gemm_qlin_amd.
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


def _case(name, op, m, n, k, group, dtype, zeros, **more):
    """n: rows of W (gemv) or the width I of the gated block (W has 2 I rows)."""
    c = {"name": name, "op": op, "m": m, "n": n, "k": k, "group": group, "dtype": dtype, "zeros": zeros,
         "pad": 0, "bias": False, "act": "silu", "keep": False}
    c.update(more)
    return c


def listed():
    return [
        # one token through a small projection: launch and call latency
        _case("gemv-1-small", "gemv", 1, 1024, 1024, 128, "bf16", False),
        # one token through the decode layer this repository's benchmark uses
        _case("gemv-1-decode", "gemv", 1, 17408, 5120, 128, "bf16", True),
        # a full decode batch through the same layer, finer groups, fp16
        _case("gemv-16-decode", "gemv", 16, 17408, 5120, 64, "fp16", True),
        # a ragged decode batch, odd row count, long rows, padded pitches, bias
        _case("gemv-5-odd", "gemv", 5, 4099, 14336, 32, "bf16", False, pad=32, bias=True),
        # a prompt of odd length
        _case("gemv-509-prompt", "gemv", 509, 4096, 7168, 128, "bf16", True),
        # input gradient of a handful of tokens
        _case("gemv_bwd-7", "gemv_bwd", 7, 5120, 5120, 64, "fp16", False),
        # input gradient of a training batch
        _case("gemv_bwd-2048", "gemv_bwd", 2048, 17408, 5120, 128, "bf16", True),
        # one token through a gated feed-forward front
        _case("glu-1-decode", "glu", 1, 14336, 4096, 128, "bf16", True),
        # a short prompt, odd width, fine groups, gelu
        _case("glu-48-odd", "glu", 48, 2051, 7168, 32, "fp16", False, act="gelu", pad=32),
        # a training batch that keeps gate and up for its backward pass
        _case("glu-2048-train", "glu", 2048, 14336, 4096, 128, "bf16", True, keep=True),
        # backward of a short batch that kept nothing: gate and up recomputed
        _case("glu_bwd-33-recompute", "glu_bwd", 33, 2048, 7168, 64, "fp16", True, act="gelu"),
        # backward of the training batch from the kept gate and up
        _case("glu_bwd-2048-train", "glu_bwd", 2048, 14336, 4096, 128, "bf16", True, keep=True),
    ]


_MOST_FLOPS = 2.0 * 2048 * 28672 * 4096


def draw(rng):
    op = rng.choice(["gemv", "gemv", "gemv_bwd", "glu", "glu", "glu_bwd"])
    dtype = rng.choice(["bf16", "fp16"])
    group = rng.choice([32, 64, 128, 128])
    keep = op in ("glu", "glu_bwd") and rng.random() < 0.5

    def spread(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    k = max(1, spread(512, 16384) // group) * group
    n = spread(256, 20480)
    if op in ("glu", "glu_bwd"):
        n = max(128, n * 3 // 4)
    m = spread(1, 16) if rng.random() < 0.5 else spread(17, 4096)
    rows = 2 * n if op in ("glu", "glu_bwd") else n
    times = 2 if op == "glu_bwd" and not keep else 1
    while 2.0 * times * m * rows * k > _MOST_FLOPS and m > 1:
        m = m * 3 // 4
    return {"op": op, "m": m, "n": n, "k": k, "group": group, "dtype": dtype, "zeros": rng.random() < 0.6,
            "pad": rng.choice([0, 0, 32]), "bias": op == "gemv" and rng.random() < 0.3,
            "act": rng.choice(["silu", "silu", "gelu"]), "keep": keep}


_DT = {"bf16": torch.bfloat16, "fp16": torch.float16}


def _rows(case):
    return 2 * case["n"] if case["op"] in ("glu", "glu_bwd") else case["n"]


def _pitched(rows, cols, pad, dtype, gen, std, align=8):
    """Normal values [rows, cols] in a buffer whose row pitch is a multiple of `align` plus `pad`."""
    pitch = (cols + align - 1) // align * align + pad
    buf = torch.empty((rows, pitch), dtype=dtype, device="cuda")
    buf.normal_(0.0, std, generator=gen)
    return buf[:, :cols]


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    dt, m, n, k, group, op = _DT[case["dtype"]], case["m"], case["n"], case["k"], case["group"], case["op"]
    rows = _rows(case)
    # 4-bit codes are close to uniform in a quantised matrix; scales put the
    # weights' standard deviation near 1 / sqrt(K), zero points lie around 8
    w = torch.randint(0, 256, (rows, k // 2 + case["pad"]), dtype=torch.uint8, device="cuda", generator=gen)
    ws = torch.empty((rows, k // group), dtype=torch.float32, device="cuda")
    ws.uniform_(0.5, 1.5, generator=gen)
    st = {"case": dict(case), "w": w[:, :k // 2], "ws": (ws * (0.22 / math.sqrt(k))).to(dt), "wz": None,
          "bias": None, "out": None, "x": None, "dy": None, "gu": None}
    if case["zeros"]:
        st["wz"] = torch.randint(5, 12, (rows, k // group), dtype=torch.uint8, device="cuda", generator=gen)
    if case["bias"]:
        st["bias"] = torch.empty((rows,), dtype=dt, device="cuda").normal_(0.0, 0.1, generator=gen)
    if op in ("gemv", "glu") or (op == "glu_bwd" and not case["keep"]):
        st["x"] = _pitched(m, k, case["pad"], dt, gen, 1.0)
    if op in ("gemv_bwd", "glu_bwd"):
        st["dy"] = _pitched(m, n, case["pad"], dt, gen, 0.1)
    if op == "glu_bwd" and case["keep"]:
        st["gu"] = _pitched(m, rows, 0, dt, gen, 1.5)
    # the buffers that a serving loop or a trainer keeps from call to call
    if op in ("gemv", "glu"):
        st["out"] = torch.empty((m, n), dtype=dt, device="cuda")
        if case["keep"]:
            st["gu"] = torch.empty((m, (rows + 7) // 8 * 8), dtype=dt, device="cuda")[:, :rows]
    else:
        st["out"] = torch.empty((m, k), dtype=dt, device="cuda")
        if op == "glu_bwd":
            st["dgu"] = torch.empty((m, (rows + 7) // 8 * 8), dtype=dt, device="cuda")[:, :rows]
    return st


def _dense(st):
    """The dequantised matrix in 32 bits."""
    c = st["case"]
    group = c["group"]
    codes = torch.stack((st["w"] & 15, st["w"] >> 4), dim=-1).reshape(st["w"].shape[0], c["k"]).float()
    zero = 8.0 if st["wz"] is None else st["wz"].float().repeat_interleave(group, dim=1)
    return (codes - zero) * st["ws"].float().repeat_interleave(group, dim=1)


def _act(g, act):
    if act == "silu":
        return g / (1.0 + torch.exp(-g))
    return 0.5 * g * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (g + 0.044715 * g * g * g)))


def _act_grad(g, act):
    if act == "silu":
        s = 1.0 / (1.0 + torch.exp(-g))
        return s * (1.0 + g * (1.0 - s))
    c = math.sqrt(2.0 / math.pi)
    t = torch.tanh(c * (g + 0.044715 * g * g * g))
    return 0.5 * (1.0 + t) + 0.5 * g * (1.0 - t * t) * c * (1.0 + 3.0 * 0.044715 * g * g)


def _run_plain(st):
    c = st["case"]
    dt, n, op = _DT[c["dtype"]], c["n"], c["op"]
    w = _dense(st)
    if op == "gemv":
        y = st["x"].float() @ w.t()
        if st["bias"] is not None:
            y = y + st["bias"].float()
        return y.to(dt)
    if op == "gemv_bwd":
        return (st["dy"].float() @ w).to(dt)
    if op == "glu":
        gu = st["x"].float() @ w.t()
        y = (_act(gu[:, :n], c["act"]) * gu[:, n:]).to(dt)
        return (y, gu.to(dt)) if c["keep"] else y
    gu = st["gu"].float() if c["keep"] else st["x"].float() @ w.t()
    dy, g, u = st["dy"].float(), gu[:, :n], gu[:, n:]
    dgu = torch.cat((dy * u * _act_grad(g, c["act"]), dy * _act(g, c["act"])), dim=1)
    return (dgu @ w).to(dt), dgu.to(dt)


def _run_own(st):
    ql, c = _lib(), st["case"]
    op = c["op"]
    if op == "gemv":
        return ql.qlin_gemv_w4(st["x"], st["w"], st["ws"], st["wz"], bias=st["bias"], y=st["out"])
    if op == "gemv_bwd":
        return ql.qlin_gemv_w4_bwd(st["dy"], st["w"], st["ws"], st["wz"], dx=st["out"])
    act = ql.QLIN_ACT_SILU if c["act"] == "silu" else ql.QLIN_ACT_GELU_TANH
    if op == "glu":
        y = ql.qlin_glu_w4(st["x"], st["w"], st["ws"], st["wz"], act=act, y=st["out"], gu=st["gu"])
        return (y, st["gu"]) if c["keep"] else y
    return ql.qlin_glu_w4_bwd(st["dy"], st["w"], st["ws"], st["wz"], act=act, x=st["x"], gu=st["gu"],
                              dgu=st["dgu"], dx=st["out"])


def run(state):
    return _run_own(state) if own else _run_plain(state)


def work(case):
    m, n, k, group, op = case["m"], case["n"], case["k"], case["group"], case["op"]
    rows = _rows(case)
    weights = rows * (k / 2 + k / group * (3 if case["zeros"] else 2))
    product = 2.0 * m * rows * k
    if op == "gemv":
        return {"bytes": weights + 2.0 * m * (k + n) + (2 * n if case["bias"] else 0), "flops": product}
    if op == "gemv_bwd":
        return {"bytes": weights + 2.0 * m * (k + n), "flops": product}
    if op == "glu":
        return {"bytes": weights + 2.0 * m * (k + n + (rows if case["keep"] else 0)), "flops": product}
    read = rows if case["keep"] else k  # gu, or x
    return {"bytes": weights + 2.0 * m * (n + read + rows + k), "flops": product * (1 if case["keep"] else 2)}


def _exact_products(x, st, forward):
    """x W^T (forward) or x W in 64 bits, group by group: the codes minus their
    zero are whole numbers, the scale of a group multiplies its sum (forward)
    or the rows' values ahead of it (input gradient)."""
    c = st["case"]
    group, groups = c["group"], c["k"] // c["group"]
    rows = st["w"].shape[0]
    parts = []
    total = torch.zeros((x.shape[0], rows), dtype=torch.float64, device="cuda") if forward else None
    for j in range(groups):
        b = st["w"][:, j * group // 2:(j + 1) * group // 2].to(torch.int64)
        q = torch.empty((rows, group), dtype=torch.float64, device="cuda")
        q[:, 0::2] = (b % 16).double()
        q[:, 1::2] = torch.div(b, 16, rounding_mode="floor").double()
        q -= 8.0 if st["wz"] is None else st["wz"][:, j:j + 1].double()
        s = st["ws"][:, j].double()
        if forward:
            total += torch.mm(x[:, j * group:(j + 1) * group].contiguous(), q.t().contiguous()) * s
        else:
            parts.append(torch.mm(x * s, q))
    return total if forward else torch.cat(parts, dim=1)


def _exact_act(g, act):
    """act(g) and its derivative in 64 bits."""
    if act == "silu":
        s = torch.sigmoid(g)
        return g * s, s + g * s * torch.sigmoid(-g)
    # 0.5 (1 + tanh(z)) = sigmoid(2 z)
    c = math.sqrt(8.0 / math.pi)
    p = torch.sigmoid(c * (g + 0.044715 * g ** 3))
    q = torch.sigmoid(-c * (g + 0.044715 * g ** 3))
    return g * p, p + g * p * q * c * (1.0 + 0.134145 * g ** 2)


def exact(case, seed):
    st = prepare(case, seed)
    n, op = case["n"], case["op"]
    if op == "gemv":
        y = _exact_products(st["x"].double(), st, True)
        return y if st["bias"] is None else y + st["bias"].double()
    if op == "gemv_bwd":
        return _exact_products(st["dy"].double(), st, False)
    gu = st["gu"].double() if op == "glu_bwd" and case["keep"] else _exact_products(st["x"].double(), st, True)
    a, da = _exact_act(gu[:, :n], case["act"])
    if op == "glu":
        y = a * gu[:, n:]
        return (y, gu) if case["keep"] else y
    dy = st["dy"].double()
    dgu = torch.cat((dy * gu[:, n:] * da, dy * a), dim=1)
    return _exact_products(dgu, st, False), dgu
