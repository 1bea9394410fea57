"""Inputs and checks of the INT8 feed-forward tests."""
import numpy as np
import torch

from oracle import i8ffn

DT = {"bf16": torch.bfloat16, "fp16": torch.float16}


def f64(t):
    return t.detach().double().cpu().numpy()


def gen_x(M, K, dt, seed, pad=0):
    """[M, K] view of a buffer whose row pitch is a multiple of 8 plus pad; tokens of different size."""
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((M, (K + 7) // 8 * 8 + pad)) * rng.uniform(0.2, 3.0, (M, 1))
    return torch.from_numpy(x).to(DT[dt])[:, :K]


def gen_codes(shape, seed, pad=0):
    """int8 codes, -128 among them, in rows with pad more bytes (a multiple of 16)."""
    rng = np.random.default_rng(seed)
    w = rng.integers(-128, 128, (*shape[:-1], shape[-1] + pad), dtype=np.int8)
    return torch.from_numpy(w)[..., :shape[-1]]


def gen_scales(shape, K, seed):
    rng = np.random.default_rng(seed)
    return torch.from_numpy((rng.uniform(0.3, 1.7, shape) / (73 * K ** 0.5)).astype(np.float32))


def gen_logits(M, E, seed, pad=0):
    rng = np.random.default_rng(seed)
    return torch.from_numpy((rng.standard_normal((M, E + pad)) * 2).astype(np.float32))[:, :E]


def gen_layer(E, H, I, seed, pad=0):
    return (gen_codes((E, 2 * I, H), seed, pad), gen_scales((E, 2 * I), H, seed + 1),
            gen_codes((E, H, I), seed + 2, pad), gen_scales((E, H), I, seed + 3))


def cuda(t):
    """The tensor on the GPU with the strides that it has here."""
    base = torch.empty_strided(t.shape, t.stride(), dtype=t.dtype, device="cuda")
    base.copy_(t)
    return base


def check(got, want, tol, what):
    got = f64(got)
    assert got.shape == want.shape, (what, got.shape, want.shape)
    assert np.isfinite(got).all(), f"{what}: not finite"
    off = np.abs(got - want)
    bad = off > tol
    assert not bad.any(), (f"{what}: {bad.sum()} of {bad.size} outside, first {np.argwhere(bad)[:4].tolist()}, "
                           f"worst {np.max(off / tol):.3g} times the bound")


def check_glu(ql, M, I, K, dt, kind=0, seed=0, pad=0, one_scale=False):
    x, w = gen_x(M, K, dt, seed, pad), gen_codes((2 * I, K), seed + 1, pad // 16 * 16)
    s = gen_scales((1,) if one_scale else (2 * I,), K, seed + 2)
    y, xq, xs = ql.qlin_glu_i8(cuda(x), cuda(w), s.cuda(), act=kind)
    torch.cuda.synchronize()
    q, sc = i8ffn.quantise(f64(x))
    assert np.array_equal(f64(xq), q) and np.array_equal(f64(xs), sc), "codes or scales"
    want, _, tol = i8ffn.front(q, sc, w.numpy(), np.broadcast_to(s.numpy(), (2 * I,)), kind, dt)
    assert y.dtype == DT[dt]
    check(y, want, tol, f"glu {M} x {I} x {K} {dt}")


def check_routing(ids, gw, logits, topk, mode):
    want_ids, want = i8ffn.route(logits.numpy(), topk, mode)
    assert np.array_equal(ids.cpu().numpy(), want_ids), "ids"
    # differences below 16 here: an error of 2^-24 times that in the exponent, two units of exp, the sum and quotient
    assert np.allclose(f64(gw), want, rtol=2.0 ** -18, atol=1e-30), "weights"


def check_moe(ql, M, E, topk, H, I, dt, kind=0, mode=0, seed=0, pad=0, given=False):
    x, (w13, s13, w2, s2) = gen_x(M, H, dt, seed, pad), gen_layer(E, H, I, seed + 1, pad // 16 * 16)
    logits = gen_logits(M, E, seed + 5, 3)
    dev = [cuda(x), cuda(w13), s13.cuda(), cuda(w2), s2.cuda()]
    if given:
        rng = np.random.default_rng(seed)
        ids = rng.integers(-1, E + 1, (M, topk)).astype(np.int32)  # the same expert twice, and none
        ids[M // 2] = -1
        gw = rng.standard_normal((M, topk)).astype(np.float32)
        y, i, g = ql.qlin_moe_ffn_i8(*dev, ids=torch.from_numpy(ids).cuda(), gw=torch.from_numpy(gw).cuda(), act=kind)
        torch.cuda.synchronize()
        assert np.array_equal(i.cpu().numpy(), ids) and np.array_equal(g.cpu().numpy(), gw)
    else:
        y, i, g = ql.qlin_moe_ffn_i8(*dev, logits=cuda(logits), topk=topk, route=mode, act=kind)
        torch.cuda.synchronize()
        check_routing(i, g, logits, topk, mode)
    want, tol = i8ffn.layer(f64(x), i.cpu().numpy(), g.cpu().numpy(), w13.numpy(), s13.numpy(), w2.numpy(), s2.numpy(),
                            kind, dt)
    assert y.dtype == DT[dt]
    check(y, want, tol, f"moe {M} x {E} top {topk} {H} x {I} {dt}")
    if given:
        assert (y[M // 2] == 0).all()
