"""Inputs and device helpers of the 4-bit weight tests."""
import numpy as np
import torch

DT = {"bf16": torch.bfloat16, "fp16": torch.float16}


def gen_w4(N, K, group, dtype, zeros, seed, exact_scales=False):
    """Codes uniform over 0..15 (packed), scales, zero points 0..15 or None.
    exact_scales: powers of two, so every weight is exact in the 16-bit type."""
    rng = np.random.default_rng(seed)
    w = rng.integers(0, 256, size=(N, K // 2), dtype=np.uint8)
    shape = (N, K // group)
    s = 2.0 ** rng.integers(-6, -2, size=shape) if exact_scales else rng.uniform(0.02, 0.1, size=shape)
    s = s * np.where(rng.random(shape) < 0.1, -1.0, 1.0)
    ws = torch.from_numpy(s.astype(np.float32)).to(DT[dtype])
    wz = rng.integers(0, 16, size=shape, dtype=np.uint8) if zeros else None
    return w, ws, wz


def gen_x(M, K, dtype, seed, scale=1.0):
    rng = np.random.default_rng(seed + 1000)
    return torch.from_numpy((rng.standard_normal((M, K)) * scale).astype(np.float32)).to(DT[dtype])


def f64(t):
    return t.float().cpu().numpy().astype(np.float64)


def pitched(t, pad, fill=float("nan"), multiple=8):
    """Device view of `t` inside rows padded to a multiple of `multiple` plus `pad`; the padding holds `fill`."""
    rows, cols = t.shape
    pitch = (cols + multiple - 1) // multiple * multiple + pad
    buf = torch.full((rows, pitch), fill if t.is_floating_point() else 0xA5, dtype=t.dtype, device="cuda")
    buf[:, :cols] = t.cuda()
    return buf[:, :cols]


def dev_w(w, ws, wz, pad=0):
    wt = torch.from_numpy(w)
    wd = pitched(wt, pad, multiple=16) if pad else wt.cuda()
    return wd, ws.cuda(), None if wz is None else torch.from_numpy(wz).cuda()


def out_view(M, C, dtype, pad):
    """An output view with `pad` guard columns and one guard row, all holding a marker."""
    buf = torch.full((M + 1, C + pad), 77.0, dtype=DT[dtype], device="cuda")
    return buf[:M, :C], buf


def guards_intact(buf, M, C):
    b = buf.float().cpu()
    assert bool((b[M:] == 77.0).all()) and bool((b[:, C:] == 77.0).all()), "wrote outside the output"


def close(got, want, tol, what):
    g = f64(got)
    assert g.shape == want.shape
    bad = ~(np.abs(g - want) <= tol)
    if bad.any():
        i = np.unravel_index(np.argmax(np.where(bad, np.abs(g - want) / tol, 0)), g.shape)
        raise AssertionError(f"{what}: {int(bad.sum())} of {g.size} off; at {i}: got {g[i]}, exact {want[i]}, "
                             f"allowed {tol[i]}")
