"""The INT8 feed-forward operators where they can go wrong: values that are not finite, masks that leave nothing,
slots without an expert, views, memory past 32 bits, tokens of every batch size."""
import numpy as np
import pytest
import torch

from gpu_util import lib, need_gpu
from i8ffn_util import DT, check, cuda, f64, gen_codes, gen_layer, gen_logits, gen_scales, gen_x
from oracle import i8ffn
from skinny_gemm_qlin_amd._lib import QlinError

pytestmark = pytest.mark.gpu

SIZES = (1, 5, 16, 20, 140)  # codes made by every workgroup; by a kernel ahead; more than 16 tokens; two tiles


@pytest.fixture(scope="module")
def ql():
    need_gpu()
    return lib()


def bits(t):
    return t.contiguous().view(torch.int16)


@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("M", SIZES)
def test_a_row_that_is_not_finite_stays_alone(ql, M, dt):
    """Its scale, codes and outputs are NaN, 0 and NaN; every other row's bits are those of the call without it."""
    I, K = 72, 1040
    x, w, s = gen_x(M, K, dt, 1).cuda(), gen_codes((2 * I, K), 2).cuda(), gen_scales((2 * I,), K, 3).cuda()
    layer = [t.cuda() for t in gen_layer(6, K, 64, 4)]
    lg = gen_logits(M, 6, 5).cuda()
    want, wq, wsc = ql.qlin_glu_i8(x, w, s)
    moe = ql.qlin_moe_ffn_i8(x, *layer, logits=lg, topk=3)[0]
    for at, v in ((K - 1, float("inf")), (0, float("nan")), (K // 2, float("-inf"))):
        r = M // 2
        z = x.clone()
        z[r, at] = v
        y, xq, xs = ql.qlin_glu_i8(z, w, s)
        m = ql.qlin_moe_ffn_i8(z, *layer, logits=lg, topk=3)[0]
        rest = [i for i in range(M) if i != r]
        assert torch.isnan(xs[r]) and (xq[r] == 0).all() and torch.isnan(y[r]).all() and torch.isnan(m[r]).all()
        assert torch.equal(bits(y[rest]), bits(want[rest])) and torch.equal(xq[rest], wq[rest])
        assert torch.equal(xs[rest], wsc[rest]) and torch.equal(bits(m[rest]), bits(moe[rest]))


@pytest.mark.parametrize("M", SIZES)
def test_rows_of_zeros(ql, M):
    """Scale and codes 0, outputs 0, also where the scales are not finite only on the way to other rows."""
    I, K = 40, 528
    x, w, s = gen_x(M, K, "bf16", 1).cuda(), gen_codes((2 * I, K), 2).cuda(), gen_scales((2 * I,), K, 3).cuda()
    x[M // 2] = -0.0
    y, xq, xs = ql.qlin_glu_i8(x, w, s)
    assert xs[M // 2] == 0 and (xq[M // 2] == 0).all() and (y[M // 2] == 0).all()
    layer = [t.cuda() for t in gen_layer(5, K, 48, 4)]
    y = ql.qlin_moe_ffn_i8(x, *layer, logits=gen_logits(M, 5, 6).cuda(), topk=2)[0]
    assert (y[M // 2] == 0).all()


@pytest.mark.parametrize("dt,scale", [("bf16", 2.0 ** -131), ("bf16", 2.0 ** -105), ("bf16", 2.0 ** -95), ("bf16", 2.0 ** 120),
                                      ("fp16", 2.0 ** -23), ("fp16", 2.0 ** -14), ("fp16", 2.0 ** 12)])
@pytest.mark.parametrize("M", SIZES)
def test_codes_over_the_whole_exponent_range(ql, M, dt, scale):
    """Subnormal rows and scales, and the largest: codes and scales of the definition, bit for bit."""
    K = 1040
    x = (gen_x(M, K, dt, 7).double() * scale).to(DT[dt])
    assert torch.isfinite(x).all()
    _, xq, xs = ql.qlin_glu_i8(x.cuda(), gen_codes((4, K), 1).cuda(), gen_scales((4,), K, 2).cuda())
    q, s = i8ffn.quantise(f64(x))
    assert np.array_equal(f64(xq), q) and np.array_equal(f64(xs), s)


def masked_logits(M, E):
    """Rows of every kind in turn, and what each of them is."""
    rng = np.random.default_rng(M)
    lg = (rng.standard_normal((M, E)) * 2).astype(np.float32)
    low, inf = np.finfo(np.float32).min, np.inf
    for t in range(M):
        k = t % 9
        if k == 1:
            lg[t] = -inf
        elif k == 2:
            lg[t] = np.nan
        elif k == 3:
            lg[t, 1:] = -inf                     # one left
        elif k == 4:
            lg[t, :E - 2] = low                  # masked by the type's lowest value: selectable, weight 0
        elif k == 5:
            lg[t] = np.round(lg[t])              # ties
        elif k == 6:
            lg[t, [0, E - 1]] = inf              # two infinities: half each
        elif k == 7:
            lg[t] = np.where(rng.random(E) < 0.5, 0.0, -0.0)
        elif k == 8:
            lg[t, ::2] = np.nan
            lg[t, 1] = -1e30
    return torch.from_numpy(lg)


@pytest.mark.parametrize("mode", [0, 1])
@pytest.mark.parametrize("E", [6, 64, 70, 300])
@pytest.mark.parametrize("M", [1, 9, 16, 40, 140])
def test_masks(ql, M, E, mode):
    H, I, topk = 48, 32, 4
    for first in (range(9) if M == 1 else (0,)):
        lg = masked_logits(9, E)[first:first + 1] if M == 1 else masked_logits(M, E)
        x, (w13, s13, w2, s2) = gen_x(M, H, "bf16", M), gen_layer(E, H, I, E)
        y, ids, gw = ql.qlin_moe_ffn_i8(x.cuda(), w13.cuda(), s13.cuda(), w2.cuda(), s2.cuda(), logits=lg.cuda(), topk=topk,
                                        route=mode)
        want_ids, want = i8ffn.route(lg.numpy(), topk, mode)
        assert np.array_equal(ids.cpu().numpy(), want_ids)
        assert np.allclose(f64(gw), want, rtol=2.0 ** -18, atol=1e-30)  # as check_routing: differences below 16, or 0 and inf
        y64, tol = i8ffn.layer(f64(x), want_ids, f64(gw), w13.numpy(), s13.numpy(), w2.numpy(), s2.numpy(), 0, "bf16")
        check(y, y64, tol, f"masks {M} x {E}")
        for t in np.nonzero((want_ids < 0).all(axis=1))[0]:
            assert (y[t] == 0).all() and (gw[t] == 0).all()


@pytest.mark.parametrize("M", SIZES)
def test_slots_without_an_expert(ql, M):
    """Ids of every kind outside the experts, their weights not finite; the same expert twice; tokens without any."""
    E, topk, H, I = 7, 5, 144, 48
    rng = np.random.default_rng(M)
    ids = rng.integers(0, E, (M, topk)).astype(np.int32)
    gw = rng.standard_normal((M, topk)).astype(np.float32)
    out = np.array([-1, E, np.iinfo(np.int32).min, np.iinfo(np.int32).max, 1 << 20, -E], dtype=np.int32)
    hole = rng.random((M, topk)) < 0.5
    hole[M // 2] = True
    ids[hole] = rng.choice(out, hole.sum())
    gw[hole] = rng.choice(np.array([np.nan, np.inf, -np.inf, 1.0], dtype=np.float32), hole.sum())
    x, layer = gen_x(M, H, "bf16", M), gen_layer(E, H, I, 3)
    y, i, g = ql.qlin_moe_ffn_i8(x.cuda(), *[t.cuda() for t in layer], ids=torch.from_numpy(ids).cuda(),
                                 gw=torch.from_numpy(gw).cuda())
    assert np.array_equal(i.cpu().numpy(), ids) and np.array_equal(g.cpu().numpy(), gw, equal_nan=True)
    w13, s13, w2, s2 = (t.numpy() for t in layer)
    want, tol = i8ffn.layer(f64(x), ids, np.where(hole, 0, gw), w13, s13, w2, s2, 0, "bf16")
    check(y, want, tol, f"holes {M}")
    assert (y[M // 2] == 0).all()


@pytest.mark.parametrize("M", SIZES)
def test_weights_of_the_caller_that_are_not_finite(ql, M):
    """They reach their token and no other."""
    E, topk, H, I = 4, 2, 80, 48
    x, layer = gen_x(M, H, "fp16", 1).cuda(), [t.cuda() for t in gen_layer(E, H, I, 3)]
    rng = np.random.default_rng(1)
    ids = torch.from_numpy(rng.integers(0, E, (M, topk)).astype(np.int32)).cuda()
    gw = torch.from_numpy(rng.standard_normal((M, topk)).astype(np.float32)).cuda()
    want = ql.qlin_moe_ffn_i8(x, *layer, ids=ids, gw=gw)[0]
    bad = gw.clone()
    bad[M // 2, 1] = float("nan")
    y = ql.qlin_moe_ffn_i8(x, *layer, ids=ids, gw=bad)[0]
    rest = [i for i in range(M) if i != M // 2]
    assert torch.isnan(y[M // 2]).all() and torch.equal(bits(y[rest]), bits(want[rest]))


@pytest.mark.parametrize("M", SIZES)
def test_hidden_rows_beyond_the_range_of_fp16(ql, M):
    """A hidden value that rounds to an infinity makes its token's row NaN, and only that."""
    E, H, I = 3, 64, 32
    w13, s13, w2, s2 = (t.cuda() for t in gen_layer(E, H, I, 3))
    x = gen_x(M, H, "fp16", 2).clamp(-4, 4).cuda()
    ids = torch.full((M, 1), 2, dtype=torch.int32, device="cuda")
    gw = torch.ones((M, 1), device="cuda")
    want = ql.qlin_moe_ffn_i8(x, w13, s13, w2, s2, ids=ids, gw=gw)[0]
    big = x.clone()
    big[M // 2] *= 4000.0
    y = ql.qlin_moe_ffn_i8(big, w13, s13, w2, s2, ids=ids, gw=gw)[0]
    h = ql.qlin_glu_i8(big, w13[2], s13[2])[0]
    assert torch.isinf(h[M // 2]).any()
    rest = [i for i in range(M) if i != M // 2]
    assert torch.isnan(y[M // 2]).all() and torch.equal(bits(y[rest]), bits(want[rest]))


def test_a_token_does_not_see_its_batch_in_the_front(ql):
    """One token alone, a few, a tile, and rows enough for the largest tiles: the same bits."""
    M, I, K = 1100, 6800, 128
    x, w, s = gen_x(M, K, "bf16", 1).cuda(), gen_codes((2 * I, K), 2).cuda(), gen_scales((2 * I,), K, 3).cuda()
    full, q, sc = ql.qlin_glu_i8(x, w, s)
    rows = np.r_[0:40, 500:530, 1060:1100]
    want, _, tol = i8ffn.front(f64(q)[rows], f64(sc)[rows], w.cpu().numpy(), s.cpu().numpy(), 0, "bf16")
    check(full[rows], want, tol, "large tiles")
    for m in (1, 2, 4, 5, 8, 9, 16, 17, 64, 65, 300, 1024):
        first = M - m
        y = ql.qlin_glu_i8(x[first:], w, s)[0]
        assert torch.equal(bits(y), bits(full[first:])), m


@pytest.mark.parametrize("dt", ["bf16", "fp16"])
def test_a_token_does_not_see_its_batch_in_the_layer(ql, dt):
    M, E, topk, H, I = 260, 4, 3, 528, 208
    x, layer = gen_x(M, H, dt, 1).cuda(), [t.cuda() for t in gen_layer(E, H, I, 2)]
    lg = gen_logits(M, E, 3).cuda()
    full = ql.qlin_moe_ffn_i8(x, *layer, logits=lg, topk=topk)
    for m in (1, 2, 4, 5, 8, 9, 16, 17, 40, 70, 200):
        got = ql.qlin_moe_ffn_i8(x[M - m:], *layer, logits=lg[M - m:], topk=topk)
        assert torch.equal(bits(got[0]), bits(full[0][M - m:])), m
        assert torch.equal(got[1], full[1][M - m:]) and torch.equal(got[2], full[2][M - m:]), m


@pytest.mark.parametrize("M", SIZES)
def test_views_and_what_lies_beside_them(ql, M):
    """Row pitches of every operand; columns and rows behind the outputs stay as they were, junk beside the inputs is
    not read into them."""
    I, K, E, topk = 41, 176, 5, 2
    x, w, s = gen_x(M, K, "bf16", 1), gen_codes((2 * I, K), 2), gen_scales((2 * I,), K, 3)
    want, wq, wsc = ql.qlin_glu_i8(x.cuda(), w.cuda(), s.cuda())

    def view(t, pad, rows=2):
        buf = torch.empty((t.shape[0] + rows, t.shape[1] + pad), dtype=t.dtype, device="cuda")
        buf.fill_(float("nan") if t.dtype.is_floating_point else 77)
        buf[:t.shape[0], :t.shape[1]] = t.cuda()
        return buf, buf[:t.shape[0], :t.shape[1]]

    _, xv = view(x, 24)
    _, wv = view(w, 32)
    yb, yv = view(torch.zeros_like(want), 3)
    qb, qv = view(torch.zeros_like(wq), 48)
    sb = torch.full((M + 4,), -5.0, device="cuda")
    ql.qlin_glu_i8(xv, wv, s.cuda(), xq=qv, xs=sb[:M], y=yv)
    assert torch.equal(bits(yv), bits(want)) and torch.equal(qv, wq) and torch.equal(sb[:M], wsc)
    assert torch.isnan(yb[M:]).all() and torch.isnan(yb[:, I:]).all() and (sb[M:] == -5).all()
    assert (qb[M:] == 77).all() and (qb[:, K:] == 77).all()

    w13, s13, w2, s2 = gen_layer(E, K, 48, 4)
    lg = gen_logits(M, E, 5)
    want, wi, wg = ql.qlin_moe_ffn_i8(x.cuda(), w13.cuda(), s13.cuda(), w2.cuda(), s2.cuda(), logits=lg.cuda(), topk=topk)
    p13, p2 = (torch.full((*t.shape[:2], t.shape[2] + 80), 99, dtype=torch.int8, device="cuda") for t in (w13, w2))
    p13[..., :K], p2[..., :48] = w13.cuda(), w2.cuda()
    _, lv = view(lg, 3)
    yb, yv = view(torch.zeros_like(want), 5)
    need = ql.qlin_moe_ffn_i8_workspace_bytes(M, K, 48, topk, E)
    work = torch.full((need + 64,), 255, dtype=torch.uint8, device="cuda")
    ids, gw = torch.full((M + 1, topk), 99, dtype=torch.int32, device="cuda"), torch.full((M + 1, topk), 9.0, device="cuda")
    ql.qlin_moe_ffn_i8(xv, p13[..., :K], s13.cuda(), p2[..., :48], s2.cuda(), logits=lv, topk=topk, ids=ids[:M], gw=gw[:M],
                       y=yv, workspace=work[:need])
    assert torch.equal(bits(yv), bits(want)) and torch.equal(ids[:M], wi) and torch.equal(gw[:M], wg)
    assert torch.isnan(yb[M:]).all() and torch.isnan(yb[:, K:]).all() and (work[need:] == 255).all()
    assert (ids[M:] == 99).all() and (gw[M:] == 9).all()


def _codes_on_device(shape, seed):
    """Int8 codes of more than 4 GiB, made in parts."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    w = torch.empty(shape, dtype=torch.int8, device="cuda")
    for part in w.view(-1).split(1 << 30):
        part.random_(-128, 128, generator=g)
    return w


def test_weights_past_4_gib(ql):
    """A dense front of 8 GiB and experts of 5 GiB each way: the last rows are those of a copy of their own."""
    I, K = 1 << 20, 4096
    w, s = _codes_on_device((2 * I, K), 1), torch.rand((2 * I,), device="cuda") * 1e-3
    pick = torch.tensor([0, 1, I // 2, I - 300, I - 2, I - 1], device="cuda")
    rows = torch.cat([pick, pick + I])
    for M in (1, 6, 17):
        x = gen_x(M, K, "bf16", M).cuda()
        y = ql.qlin_glu_i8(x, w, s)[0]
        assert torch.equal(bits(y[:, pick]), bits(ql.qlin_glu_i8(x, w[rows].contiguous(), s[rows].contiguous())[0]))
    del w, s, y
    torch.cuda.empty_cache()
    E, H, I = 300, 4096, 2048
    w13, w2 = _codes_on_device((E, 2 * I, H), 2), _codes_on_device((E, H, 2 * I), 3)[..., :I]
    s13, s2 = torch.rand((E, 2 * I), device="cuda") * 1e-4, torch.rand((E, H), device="cuda") * 1e-4
    for M in (1, 6, 20):
        x = gen_x(M, H, "bf16", M).cuda()
        ids = torch.tensor([[0, 299, 255, 256]], dtype=torch.int32, device="cuda").repeat(M, 1)
        gw = torch.rand((M, 4), device="cuda")
        y = ql.qlin_moe_ffn_i8(x, w13, s13, w2, s2, ids=ids, gw=gw)[0]
        some = [0, 299, 255, 256]
        few = [w13[some].contiguous(), s13[some].contiguous(), w2[some].contiguous(), s2[some].contiguous()]
        own = torch.arange(4, dtype=torch.int32, device="cuda").repeat(M, 1)
        assert torch.equal(bits(y), bits(ql.qlin_moe_ffn_i8(x, *few, ids=own, gw=gw)[0])), M


def test_activations_past_4_gib(ql):
    """16384 tokens whose rows, codes, logits and outputs lie more than 2^18 elements apart."""
    M, I, K, far = 16384, 20, 32, (1 << 18) + 16
    x, w, s = gen_x(M, K, "bf16", 1).cuda(), gen_codes((2 * I, K), 2).cuda(), gen_scales((2 * I,), K, 3).cuda()
    want, wq, wsc = ql.qlin_glu_i8(x, w, s)
    xf = torch.empty((M, far), dtype=x.dtype, device="cuda")[:, :K]
    xf.copy_(x)
    yf = torch.empty((M, far), dtype=x.dtype, device="cuda")[:, :I]
    qf = torch.empty((M, far), dtype=torch.int8, device="cuda")[:, :K]
    _, _, xs = ql.qlin_glu_i8(xf, w, s, xq=qf, y=yf)
    assert torch.equal(bits(yf), bits(want)) and torch.equal(qf, wq) and torch.equal(xs, wsc)
    E, topk = 3, 2
    layer = [t.cuda() for t in gen_layer(E, K, 16, 4)]
    lg = gen_logits(M, E, 5).cuda()
    lf = torch.empty((M, far), device="cuda")[:, :E]
    lf.copy_(lg)
    want = ql.qlin_moe_ffn_i8(x, *layer, logits=lg, topk=topk)
    yf = yf.as_strided((M, K), (far, 1))
    got = ql.qlin_moe_ffn_i8(xf, *layer, logits=lf, topk=topk, y=yf)
    assert torch.equal(bits(got[0]), bits(want[0])) and torch.equal(got[1], want[1]) and torch.equal(got[2], want[2])


BAD = {"x type": lambda a: a.update(x=a["x"].float()), "x rows": lambda a: a.update(x=a["x"].t().contiguous().t()),
       "x width": lambda a: a.update(x=a["x"][:, :32].contiguous()),
       "w13 type": lambda a: a.update(w13=a["w13"].float()), "w13 odd": lambda a: a.update(w13=a["w13"][:, :-1]),
       "w13 host": lambda a: a.update(w13=a["w13"].cpu()), "s13 type": lambda a: a.update(s13=a["s13"].half()),
       "s13 length": lambda a: a.update(s13=a["s13"][..., :-1].contiguous())}
GLU_BAD = {"xq type": lambda a: a.update(xq=torch.empty((3, 64), device="cuda")),
           "xs shape": lambda a: a.update(xs=torch.empty((4,), device="cuda")),
           "y type": lambda a: a.update(y=torch.empty((3, 8), device="cuda")),
           "y shape": lambda a: a.update(y=torch.empty((3, 9), dtype=torch.bfloat16, device="cuda")), **BAD}
MOE_BAD = {"w2 type": lambda a: a.update(w2=a["w2"].view(torch.uint8)), "w2 shape": lambda a: a.update(w2=a["w2"][:, :-1]),
           "w2 experts": lambda a: a.update(w2=a["w2"][:1]), "w2 gaps": lambda a: a.update(w2=torch.cat([a["w2"]] * 2, 1)[:, :64]),
           "s2 shape": lambda a: a.update(s2=a["s2"][:, :-1].contiguous()),
           "logits type": lambda a: a.update(logits=a["logits"].half()),
           "logits shape": lambda a: a.update(logits=a["logits"][:, :1]),
           "topk missing": lambda a: a.update(topk=None), "ids missing": lambda a: a.update(logits=None, topk=None),
           "ids type": lambda a: a.update(ids=torch.zeros((3, 1), dtype=torch.int64, device="cuda")),
           "gw shape": lambda a: a.update(gw=torch.zeros((3, 2), device="cuda")),
           "y shape": lambda a: a.update(y=torch.empty((3, 32), dtype=torch.bfloat16, device="cuda")),
           "workspace host": lambda a: a.update(workspace=torch.empty((1 << 20,), dtype=torch.uint8)), **BAD}


def _glu_args():
    return dict(x=gen_x(3, 64, "bf16", 1).cuda(), w13=gen_codes((16, 64), 2).cuda(), s13=gen_scales((16,), 64, 3).cuda())


def _moe_args():
    w13, s13, w2, s2 = (t.cuda() for t in gen_layer(2, 64, 16, 1))
    return dict(x=gen_x(3, 64, "bf16", 1).cuda(), w13=w13, s13=s13, w2=w2, s2=s2, logits=gen_logits(3, 2, 2).cuda(), topk=1)


@pytest.mark.parametrize("call", ["glu", "moe"])
def test_refusals_of_the_binding(ql, call):
    """Each names the operand; the arguments without the change are taken."""
    fn, args, bad = ((ql.qlin_glu_i8, _glu_args, GLU_BAD) if call == "glu" else (ql.qlin_moe_ffn_i8, _moe_args, MOE_BAD))
    fn(**args())
    for name, change in bad.items():
        a = args()
        change(a)
        word = name.split()[0]
        if name == "x width":
            word = "w13|K="
        if name == "w13 odd":
            word = "w13|s13"
        with pytest.raises((TypeError, ValueError), match=word):
            fn(**a)


def test_refusals_of_the_library(ql):
    for a in (dict(act=2), dict(act=-1)):
        with pytest.raises(QlinError):
            ql.qlin_glu_i8(**_glu_args(), **a)
    for a in (dict(topk=3), dict(topk=0), dict(route=2), dict(act=2),
              dict(workspace=torch.empty((16,), dtype=torch.uint8, device="cuda"))):
        with pytest.raises(QlinError):
            ql.qlin_moe_ffn_i8(**{**_moe_args(), **a})
    a = _glu_args()
    with pytest.raises(QlinError):
        ql.qlin_glu_i8(a["x"][:0], a["w13"], a["s13"])
    with pytest.raises(QlinError):
        ql.qlin_glu_i8(a["x"][:, :40].contiguous(), a["w13"][:, :40].contiguous(), a["s13"])
    with pytest.raises(QlinError):
        ql.qlin_glu_i8(a["x"][:1].expand(3, -1), a["w13"], a["s13"])
