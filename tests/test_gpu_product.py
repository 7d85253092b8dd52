"""The expert products in 16 bits on the GPU, against their 64-bit definitions.

Tolerances.  U = 2^-24 is half a step of fp32.  A sum of n products is off by at
most (n + 4) U times the sum of the products' magnitudes (n additions in any
order; the products of 16-bit numbers are exact in fp32).  A value rounded to the
rows' type is off by half a step of it, relative to its value, and half a
subnormal step.  Activations and their slopes are off by at most 32 U (1 + |z|):
exp of an argument rounded at |z| U and a few roundings of values up to 1 + |z|.
These are carried through the formulas with absolute values in 64 bits.  Sums of
small whole numbers are exact, and so are the tests on them.  Every case prints
what it runs first.
"""
import sys

import numpy as np
import pytest

import oracle.product_oracle as po
from any_precision_bitplane_amd import binding as B

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
DEV = "cuda:0"
DTYPES = ["f16", "bf16"]
ACTS = {"none": B.PW_ACT_NONE, "silu": B.PW_ACT_SILU, "gelu": B.PW_ACT_GELU}


def say(msg):
    print(msg, flush=True)
    sys.stdout.flush()


@pytest.fixture(scope="module")
def torch():
    import torch as _t
    if not _t.cuda.is_available():
        pytest.fail("GPU tests need a GPU")
    B.load()
    return _t


def dtype_of(torch, name):
    return {"f16": torch.float16, "bf16": torch.bfloat16}[name]


def half_step(torch, name):
    f = torch.finfo(dtype_of(torch, name))
    return f.eps / 2, f.smallest_normal * f.eps / 2


def f64(t):
    return t.detach().cpu().float().double().numpy()


def rand(torch, seed, shape, name, std=1.0, pad=0):
    g = torch.Generator().manual_seed(seed)
    a = torch.randn((*shape[:-1], shape[-1] + pad), generator=g) * std
    return a.to(dtype_of(torch, name)).to(DEV)[..., :shape[-1]]


def whole(torch, seed, shape, name, n, pad=0):
    """-1, 0 and 1, so rare that sums of n products of two such numbers stay below 256 and a bf16 holds them."""
    g = torch.Generator().manual_seed(seed)
    p = min(1.0, (256.0 / max(n, 1)) ** 0.5)
    full = (*shape[:-1], shape[-1] + pad)
    a = torch.randint(0, 2, full, generator=g) * 2 - 1
    a = a * (torch.rand(full, generator=g) < p)
    return a.to(dtype_of(torch, name)).to(DEV)[..., :shape[-1]]


def near(got, ref, allowed, what):
    err = np.abs(got - ref)
    assert np.all(np.isfinite(got)), what
    worst = float(np.max(err / np.maximum(allowed, 1e-300))) if err.size else 0.0
    say(f"  {what}: max abs {float(err.max()) if err.size else 0.0:.3e}, {worst:.2f} of what is allowed")
    assert not err.size or (err - allowed).max() <= 0, (what, worst)


def starts(seed, S, E, empty=True, behind=0):
    """Offsets of E experts over S rows, `behind` of them of no expert; some experts without rows."""
    rng = np.random.default_rng(seed)
    share = rng.random(E) ** 2
    if empty and E > 2:
        share[rng.permutation(E)[:max(1, E // 4)]] = 0
    n = S - behind
    counts = np.floor(share / share.sum() * n).astype(np.int64)
    counts[int(np.argmax(share))] += n - counts.sum()
    return np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)


def on_gpu(torch, off):
    return None if off is None else torch.tensor(off, dtype=torch.int32, device=DEV)


def scratch(torch, n):
    return torch.full((n,), 0x7F, dtype=torch.uint8, device=DEV)


def experts(off, E, S):
    return 1 if off is None else E


# One expert or several; rows for the forms for few and for many; every size around a tile's.
SIZES = [  # E, S, N, K, offsets
    (1, 1, 8, 8, False), (1, 3, 264, 72, False), (1, 17, 48, 264, True), (1, 40, 1032, 136, False),
    (1, 49, 264, 64, False), (1, 100, 520, 200, False), (1, 129, 256, 320, True), (1, 513, 776, 72, False),
    (5, 4, 64, 64, True), (60, 16, 96, 544, True), (60, 300, 136, 128, True), (8, 500, 264, 72, True),
    (7, 630, 504, 136, True), (2, 600, 328, 2696, True), (1, 4100, 4104, 2568, False), (1, 1355, 496, 48, True), (3, 3100, 136, 264, True), (3, 1000, 248, 1000, True), (256, 700, 40, 56, True), (2, 1537, 1024, 136, True),
]
IDS = [f"E{e}-S{s}-N{n}-K{k}" for e, s, n, k, _ in SIZES]


@pytest.mark.parametrize("name", DTYPES)
@pytest.mark.parametrize("E,S,N,K,ragged", SIZES, ids=IDS)
def test_product_of_whole_numbers(torch, E, S, N, K, ragged, name):
    say(f"product {name} E={E} S={S} N={N} K={K}")
    off = starts(S, S, E, behind=S // 5 if ragged else 0) if ragged else None
    n = S if off is None else int(off[-1])
    x, w = whole(torch, 1, (S, K), name, K, pad=8), whole(torch, 2, (E, N, K), name, K)
    x[n:] = float("nan")                              # rows of no expert
    y = torch.full((S, N + 16), 7.0, dtype=x.dtype, device=DEV)
    B.pw_moe_product(E, S, N, K, x, w, y[:, :N], scratch(torch, B.pw_moe_product_workspace_bytes(E, S, N, K)),
                     offsets=on_gpu(torch, off))
    torch.cuda.synchronize()
    ref = po.product(f64(x), f64(w), off)[1]
    assert np.abs(ref[:n]).max(initial=0) <= 256
    assert np.array_equal(f64(y[:n, :N]), ref[:n])
    assert bool((y[n:] == 7.0).all()) and bool((y[:, N:] == 7.0).all())


@pytest.mark.parametrize("name", DTYPES)
@pytest.mark.parametrize("E,S,N,K,ragged", SIZES, ids=IDS)
def test_product_backward_of_whole_numbers(torch, E, S, N, K, ragged, name):
    say(f"product backward {name} E={E} S={S} N={N} K={K}")
    off = starts(S + 1, S, E, behind=S // 5 if ragged else 0) if ragged else None
    n = S if off is None else int(off[-1])
    most = max(S, N)
    dy, x, w = (whole(torch, 3, (S, N), name, most, pad=24), whole(torch, 4, (S, K), name, most, pad=8),
                whole(torch, 5, (E, N, K), name, most))
    dy[n:], x[n:] = float("nan"), float("nan")
    dx = torch.full((S, K), 7.0, dtype=x.dtype, device=DEV)
    dw, db = torch.full_like(w, 7.0), torch.full((E, N), 7.0, dtype=x.dtype, device=DEV)
    ws = scratch(torch, B.pw_moe_product_backward_workspace_bytes(E, S, N, K))
    B.pw_moe_product_backward(E, S, N, K, dy, x, w, ws, offsets=on_gpu(torch, off), dx=dx, dw=dw, dbias=db)
    torch.cuda.synchronize()
    rx, rw, rb, _ = po.product_backward(f64(dy)[:n], f64(x)[:n], f64(w), off)
    assert max(np.abs(a).max(initial=0) for a in (rx, rw, rb)) <= 256
    assert np.array_equal(f64(dx[:n]), rx) and bool((dx[n:] == 7.0).all())
    assert np.array_equal(f64(dw), rw)
    assert np.array_equal(f64(db), rb)


@pytest.mark.parametrize("act", ["none", "silu", "gelu"])
@pytest.mark.parametrize("name", DTYPES)
@pytest.mark.parametrize("E,S,N,K", [(1, 5, 136, 264), (9, 70, 264, 136), (3, 800, 520, 200), (1, 300, 264, 64)])
def test_product_epilogue(torch, E, S, N, K, name, act):
    say(f"product epilogue {name} {act} E={E} S={S} N={N} K={K}")
    off = starts(S, S, E, behind=S // 7) if E > 1 else None
    n = S if off is None else int(off[-1])
    x, w = rand(torch, 1, (S, K), name, pad=8), rand(torch, 2, (E, N, K), name, 2 * K ** -0.5)
    bias, res = rand(torch, 3, (E, N), name), rand(torch, 4, (S, N), name, pad=16)
    y, pre = torch.full((S, N), 7.0, dtype=x.dtype, device=DEV), torch.full((S, N + 8), 7.0, dtype=x.dtype, device=DEV)
    ws = scratch(torch, B.pw_moe_product_workspace_bytes(E, S, N, K))
    B.pw_moe_product(E, S, N, K, x, w, y, ws, offsets=on_gpu(torch, off), bias=bias, act=ACTS[act], residual=res,
                     pre=pre[:, :N])
    over = res.clone()
    B.pw_moe_product(E, S, N, K, x, w, over, ws, offsets=on_gpu(torch, off), bias=bias, act=ACTS[act], residual=over)
    torch.cuda.synchronize()
    z, ry = po.product(f64(x), f64(w), off, f64(bias), act, f64(res))
    mags = po.product(np.abs(f64(x)), np.abs(f64(w)), off, np.abs(f64(bias)))[0][:n]
    rel, ab = half_step(torch, name)
    z, ry, dz = z[:n], ry[:n], (K + 5) * U * mags
    near(f64(pre[:n, :N]), z, dz + rel * (np.abs(z) + dz) + ab, "pre")
    da = dz if act == "none" else 1.13 * dz + 32 * U * (1 + np.abs(z))
    dy = da + 2 * U * (np.abs(ry) + np.abs(f64(res))[:n])
    near(f64(y[:n]), ry, dy + rel * (np.abs(ry) + dy) + ab, "y")
    assert torch.equal(over[:n], y[:n]) and torch.equal(over[n:], res[n:])
    assert bool((y[n:] == 7.0).all()) and bool((pre[n:] == 7.0).all()) and bool((pre[:, N:] == 7.0).all())


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("name", DTYPES)
@pytest.mark.parametrize("E,S,N,K", [(1, 5, 136, 264), (9, 300, 264, 136), (3, 800, 520, 200)])
def test_product_backward_through_the_activation(torch, E, S, N, K, name, act):
    say(f"product backward {name} {act} E={E} S={S} N={N} K={K}")
    off = starts(S, S, E, behind=S // 7) if E > 1 else None
    n = S if off is None else int(off[-1])
    dy, x, w = rand(torch, 1, (S, N), name), rand(torch, 2, (S, K), name), rand(torch, 3, (E, N, K), name, K ** -0.5)
    pre = rand(torch, 4, (S, N), name, 2.0, pad=8)
    dx, dw, db = torch.full_like(x, 7.0), torch.full_like(w, 7.0), torch.full((E, N), 7.0, dtype=x.dtype, device=DEV)
    ws = scratch(torch, B.pw_moe_product_backward_workspace_bytes(E, S, N, K))
    B.pw_moe_product_backward(E, S, N, K, dy, x, w, ws, offsets=on_gpu(torch, off), act=ACTS[act], pre=pre, dx=dx, dw=dw,
                              dbias=db)
    only = [torch.full_like(t, 7.0) for t in (dx, dw, db)]
    call = dict(offsets=on_gpu(torch, off), act=ACTS[act], pre=pre)
    B.pw_moe_product_backward(E, S, N, K, dy, None, w, ws, dx=only[0], **call)
    B.pw_moe_product_backward(E, S, N, K, dy, x, None, ws, dw=only[1], **call)
    B.pw_moe_product_backward(E, S, N, K, dy, None, None, ws, dbias=only[2], **call)
    torch.cuda.synchronize()
    assert torch.equal(only[0], dx) and torch.equal(only[1], dw) and torch.equal(only[2], db)
    D, X, W, Z = f64(dy)[:n], f64(x)[:n], f64(w), f64(pre)[:n]
    rx, rw, rb, dz = po.product_backward(D, X, W, off, act, Z)
    rel, ab = half_step(torch, name)
    ez = np.abs(D) * 32 * U * (1 + np.abs(Z)) + 2 * U * np.abs(dz)       # of dz, and of dz as the products take it
    eb = ez
    ez = ez + rel * (np.abs(dz) + ez) + ab
    mx, mw, _, _ = po.product_backward(np.abs(dz), np.abs(X), np.abs(W), off)
    mb = po.product_backward(np.abs(dz), np.abs(X), np.abs(W), off)[2]
    ex, ew, _, _ = po.product_backward(ez, np.abs(X), np.abs(W), off)
    eb = po.product_backward(eb, np.abs(X), np.abs(W), off)[2]
    for got, ref, e, what in [(f64(dx[:n]), rx, ex + (N + 4) * U * (mx + ex), "dx"),
                              (f64(dw), rw, ew + (S + 4) * U * (mw + ew), "dw"),
                              (f64(db), rb, eb + (S + 4) * U * (mb + eb), "dbias")]:
        near(got, ref, e + rel * (np.abs(ref) + e) + ab, what)
    assert bool((dx[n:] == 7.0).all())


FFN = [  # E, S, H, I, ragged
    (1, 1, 64, 32, False), (1, 1, 2048, 352, False), (1, 20, 96, 160, True), (60, 16, 256, 96, True),
    (8, 32, 256, 512, True), (8, 200, 96, 160, True), (5, 400, 160, 288, True), (1, 130, 128, 128, False),
    (3, 900, 256, 416, True), (2, 700, 2624, 288, True), (2, 500, 160, 2720, True), (256, 300, 32, 32, True),
]
FFN_IDS = [f"E{e}-S{s}-H{h}-I{i}" for e, s, h, i, _ in FFN]


def ffn_inputs(torch, E, S, H, I, name, ragged):
    off = starts(S, S, E, behind=S // 6) if ragged else None
    n = S if off is None else int(off[-1])
    x = rand(torch, 1, (S, H), name, pad=8)
    x[n:] = float("nan")
    return (off, n, x, rand(torch, 2, (E, 2 * I, H), name, 1.5 * H ** -0.5), rand(torch, 3, (E, H, I), name, I ** -0.5))


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("name", DTYPES)
@pytest.mark.parametrize("E,S,H,I,ragged", FFN, ids=FFN_IDS)
def test_ffn(torch, E, S, H, I, ragged, name, act):
    say(f"ffn {name} {act} E={E} S={S} H={H} I={I}")
    off, n, x, wg, wd = ffn_inputs(torch, E, S, H, I, name, ragged)
    shp = B.shape(H, I, E, min(2, E))
    y = torch.full((S, H + 8), 7.0, dtype=x.dtype, device=DEV)
    z = torch.full((S, 2 * I + 16), 7.0, dtype=x.dtype, device=DEV)
    ws = scratch(torch, B.pw_moe_ffn_workspace_bytes(shp, S))
    call = dict(offsets=on_gpu(torch, off), act=ACTS[act])
    B.pw_moe_ffn(shp, S, x, wg, wd, y[:, :H], ws, z=z[:, :2 * I], **call)
    bare = torch.full((S, H), 7.0, dtype=x.dtype, device=DEV)
    B.pw_moe_ffn(shp, S, x, wg, wd, bare, ws, **call)
    code = torch.full((S, 2 * I), 1, dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn)
    G = -(-I // 128)
    scale = torch.full((S, 2 * G), -1.0, device=DEV)
    eight = torch.full((S, H), 7.0, dtype=x.dtype, device=DEV)
    B.pw_moe_ffn(shp, S, x, wg, wd, eight, ws, z=code, z_scale=scale, **call)
    torch.cuda.synchronize()
    assert torch.equal(bare, y[:, :H])                # the checkpoint changes nothing
    X, WG, WD = f64(x)[:n], f64(wg), f64(wd)
    rz, rh, ry = po.ffn(X, WG, WD, off, act)
    rel, ab = half_step(torch, name)
    ez = (H + 4) * U * po.product(np.abs(X), np.abs(WG), off)[0]
    near(f64(z[:n, :2 * I]), rz, ez + rel * (np.abs(rz) + ez) + ab, "z")
    g, u, eg, eu = rz[:, :I], rz[:, I:], ez[:, :I], ez[:, I:]
    s = np.abs(po.act(g, act))
    es = 1.13 * eg + 32 * U * (1 + np.abs(g))
    eh = es * (np.abs(u) + eu) + s * eu + 2 * U * np.abs(rh)
    eh = eh + rel * (np.abs(rh) + eh) + ab
    ey = po.product(eh, np.abs(WD), off)[0] + (I + 4) * U * po.product(np.abs(rh) + eh, np.abs(WD), off)[0]
    allowed = ey + rel * (np.abs(ry) + ey) + ab
    near(f64(y[:n, :H]), ry, allowed, "y")
    near(f64(eight[:n]), ry, allowed, "y beside the 8-bit checkpoint")
    rs = po.scales(rz)
    wide_e = np.maximum(po.scales(ez), 0)             # the largest error of a group's values over 448
    near(f64(scale[:n]), rs, wide_e + 4 * U * rs, "scales")
    got = f64(code[:n].float()) * po.spread_scales(f64(scale[:n]), I)
    step = po.spread_scales(f64(scale[:n]), I)
    near(got, rz, ez + (np.abs(rz) + ez) * 2.0 ** -4 * (1 + 1e-3) + step * 2.0 ** -10 * 1.01, "8-bit z")
    for t, keep in [(y, 7.0), (z, 7.0), (eight, 7.0), (scale, -1.0)]:
        assert bool((t[n:] == keep).all())
    assert bool((code.view(torch.uint8)[n:] == 1).all())
    assert bool((y[:, H:] == 7.0).all()) and bool((z[:, 2 * I:] == 7.0).all())


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("eight", [False, True], ids=["z16", "z8"])
@pytest.mark.parametrize("name", DTYPES)
@pytest.mark.parametrize("E,S,H,I,ragged", FFN, ids=FFN_IDS)
def test_ffn_backward(torch, E, S, H, I, ragged, name, eight, act):
    say(f"ffn backward {name} {act} {'z8' if eight else 'z16'} E={E} S={S} H={H} I={I}")
    off, n, x, wg, wd = ffn_inputs(torch, E, S, H, I, name, ragged)
    shp = B.shape(H, I, E, 1)
    dy = rand(torch, 4, (S, H), name, pad=16)
    z = rand(torch, 5, (S, 2 * I), name, 2.0, pad=32)
    dy[n:], z[n:] = float("nan"), float("nan")
    scale = None
    Z = f64(z)[:n]
    if eight:
        G = -(-I // 128)
        code = (torch.randn((S, 2 * I), generator=torch.Generator().manual_seed(6)) * 150).clamp(-448, 448)
        z = code.to(torch.float8_e4m3fn).to(DEV)
        scale = (0.01 + 0.01 * torch.rand((S, 2 * G), generator=torch.Generator().manual_seed(7))).to(DEV)
        scale[n:] = float("nan")
        Z = f64(z.float())[:n] * po.spread_scales(f64(scale), I)[:n]
    dx, dg, dd = torch.full((S, H + 8), 7.0, dtype=x.dtype, device=DEV), torch.full_like(wg, 7.0), torch.full_like(wd, 7.0)
    ws = scratch(torch, B.pw_moe_ffn_backward_workspace_bytes(shp, S))
    call = dict(offsets=on_gpu(torch, off), act=ACTS[act], z_scale=scale)
    B.pw_moe_ffn_backward(shp, S, dy, x, wg, wd, z, ws, dx=dx[:, :H], dw_gate_up=dg, dw_down=dd, **call)
    only = [torch.full((S, H), 7.0, dtype=x.dtype, device=DEV), torch.full_like(wg, 7.0), torch.full_like(wd, 7.0)]
    B.pw_moe_ffn_backward(shp, S, dy, None, wg, wd, z, ws, dx=only[0], **call)
    B.pw_moe_ffn_backward(shp, S, dy, x, None, wd, z, ws, dw_gate_up=only[1], **call)
    B.pw_moe_ffn_backward(shp, S, dy, None, None, wd, z, ws, dw_down=only[2], **call)
    torch.cuda.synchronize()
    assert torch.equal(only[0], dx[:, :H]) and torch.equal(only[1], dg) and torch.equal(only[2], dd)
    D, X, WG, WD = f64(dy)[:n], f64(x)[:n], f64(wg), f64(wd)
    rx, rg, rd, dh = po.ffn_backward(D, X, WG, WD, Z, off, act)
    rel, ab = half_step(torch, name)
    g, u = Z[:, :I], Z[:, I:]
    s, sl = po.act(g, act), po.slope(g, act)
    eg = 32 * U * (1 + np.abs(g)) + 4 * U * np.abs(g)                    # of act and slope, the scale's rounding in it
    h0 = np.zeros((n, I))
    edh = (H + 4) * U * po.product_backward(np.abs(D), np.abs(h0), np.abs(WD), off)[0]
    d1, d2, h = dh * u * sl, dh * s, s * u
    e1 = edh * np.abs(u * sl) + (np.abs(dh) + edh) * (np.abs(u) * eg * (1 + 2 * U) + 6 * U * np.abs(u * sl))
    e2 = edh * np.abs(s) + (np.abs(dh) + edh) * (eg + 4 * U * np.abs(s))
    eh = eg * np.abs(u) * (1 + 2 * U) + 6 * U * np.abs(h)
    dz, ez = np.concatenate([d1, d2], 1), np.concatenate([e1, e2], 1)
    ez = ez + rel * (np.abs(dz) + ez) + ab
    eh = eh + rel * (np.abs(h) + eh) + ab
    ax, ag = po.product_backward(np.abs(dz) + ez, np.abs(X), np.abs(WG), off)[:2]
    ex, e_g = po.product_backward(ez, np.abs(X), np.abs(WG), off)[:2]
    ad = po.product_backward(np.abs(D), np.abs(h) + eh, np.abs(WD), off)[1]
    ed = po.product_backward(np.abs(D), eh, np.abs(WD), off)[1]
    for got, ref, e, what in [(f64(dx[:n, :H]), rx, ex + (2 * I + 4) * U * ax, "dx"),
                              (f64(dg), rg, e_g + (S + 4) * U * ag, "dw_gate_up"),
                              (f64(dd), rd, ed + (S + 4) * U * ad, "dw_down")]:
        near(got, ref, e + rel * (np.abs(ref) + e) + ab, what)
    assert bool((dx[n:] == 7.0).all()) and bool((dx[:, H:] == 7.0).all())


def test_no_rows_at_all(torch):
    say("S = 0")
    E, N, K, H, I = 3, 40, 24, 64, 96
    x, dy = torch.empty((0, K), dtype=torch.float16, device=DEV), torch.empty((0, N), dtype=torch.float16, device=DEV)
    w = rand(torch, 1, (E, N, K), "f16")
    dw, db = torch.full_like(w, 7.0), torch.full((E, N), 7.0, dtype=w.dtype, device=DEV)
    off = torch.zeros(E + 1, dtype=torch.int32, device=DEV)
    ws = scratch(torch, B.pw_moe_product_backward_workspace_bytes(E, 0, N, K))
    B.pw_moe_product_backward(E, 0, N, K, dy, x, w, ws, offsets=off, dw=dw, dbias=db)
    shp = B.shape(H, I, E, 1)
    e, wg, wd = torch.empty((0, H), dtype=w.dtype, device=DEV), rand(torch, 2, (E, 2 * I, H), "f16"), rand(torch, 3, (E, H, I), "f16")
    dg, dd = torch.full_like(wg, 7.0), torch.full_like(wd, 7.0)
    z = torch.empty((0, 2 * I), dtype=w.dtype, device=DEV)
    ws = scratch(torch, B.pw_moe_ffn_backward_workspace_bytes(shp, 0))
    B.pw_moe_ffn_backward(shp, 0, e, e, wg, wd, z, ws, offsets=off, dw_gate_up=dg, dw_down=dd)
    B.pw_moe_ffn(shp, 0, e, wg, wd, e, ws, offsets=off)
    # rows, but none of an expert's: nothing but zero gradients is written
    S = 40
    x, dy = rand(torch, 4, (S, K), "f16") * float("nan"), rand(torch, 5, (S, N), "f16") * float("nan")
    dx, dw2, db2 = torch.full_like(x, 7.0), torch.full_like(w, 7.0), torch.full_like(db, 7.0)
    ws = scratch(torch, B.pw_moe_product_backward_workspace_bytes(E, S, N, K))
    B.pw_moe_product_backward(E, S, N, K, dy, x, w, ws, offsets=off, dx=dx, dw=dw2, dbias=db2)
    y = torch.full_like(dy, 7.0)
    B.pw_moe_product(E, S, N, K, x, w, y, ws, offsets=off)
    torch.cuda.synchronize()
    for t in (dw, db, dg, dd, dw2, db2):
        assert not bool(t.any())
    assert bool((dx == 7.0).all()) and bool((y == 7.0).all())


@pytest.mark.parametrize("S", [9, 300])
def test_broadcast_and_far_rows(torch, S):
    say(f"rows at stride 0 and 2^21 elements apart, S={S}")
    N, K = 72, 136
    w = whole(torch, 1, (1, N, K), "f16", K)
    one = whole(torch, 2, (1, K), "f16", K)
    y, dw = torch.empty((S, N), dtype=w.dtype, device=DEV), torch.empty_like(w)
    ws = scratch(torch, B.pw_moe_product_backward_workspace_bytes(1, S, N, K))
    B.pw_moe_product(1, S, N, K, one.expand(S, K), w, y, ws)
    dy = (torch.arange(N, device=DEV) % 3 - 1).to(w.dtype).expand(S, N)
    B.pw_moe_product_backward(1, S, N, K, dy, one.expand(S, K), w, ws, dw=dw)
    ref = f64(one) @ f64(w)[0].T
    assert np.array_equal(f64(y), np.repeat(ref, S, 0))
    assert np.array_equal(f64(dw)[0], S * np.outer(f64(dy)[0], f64(one)[0]))
    far = torch.zeros((S * 5, 1 << 21), dtype=torch.float16, device=DEV)      # past 2^32 bytes from row 1024 on
    x = far[:, 8:8 + K]
    x.copy_(whole(torch, 3, (5 * S, K), "f16", K))
    wide = torch.zeros((5 * S, N), dtype=w.dtype, device=DEV)
    off = np.array([0, 2 * S + 1, 5 * S - 1], dtype=np.int32)
    w2 = whole(torch, 4, (2, N, K), "f16", K)
    ws = scratch(torch, B.pw_moe_product_workspace_bytes(2, 5 * S, N, K))
    B.pw_moe_product(2, 5 * S, N, K, x, w2, wide, ws, offsets=on_gpu(torch, off))
    torch.cuda.synchronize()
    assert np.array_equal(f64(wide)[:-1], po.product(f64(x), f64(w2), off)[0][:-1])
    assert not bool(wide[-1].any()) and not bool(far[:, :8].any()) and not bool(far[:, 8 + K:8 + 2 * K].any())


@pytest.mark.parametrize("S,eight", [(3, False), (40, True)])
def test_matrices_past_32_bits(torch, S, eight):
    H, I = 32768, 32736
    say(f"gate and up of {4 * I * H} bytes, S={S}")
    shp = B.shape(H, I, 1, 1)
    g = torch.Generator(device=DEV)
    g.manual_seed(3)
    wg = torch.empty((1, 2 * I, H), dtype=torch.float16, device=DEV).normal_(0, H ** -0.5, generator=g)
    wd = torch.empty((1, H, I), dtype=torch.float16, device=DEV).normal_(0, I ** -0.5, generator=g)
    x = rand(torch, 1, (S, H), "f16")
    z = torch.empty((S, 2 * I), dtype=torch.uint8 if eight else x.dtype, device=DEV)
    z = z.view(torch.float8_e4m3fn) if eight else z
    G = -(-I // 128)
    scale = torch.empty((S, 2 * G), device=DEV) if eight else None
    y = torch.empty((S, H), dtype=x.dtype, device=DEV)
    B.pw_moe_ffn(shp, S, x, wg, wd, y, scratch(torch, B.pw_moe_ffn_workspace_bytes(shp, S)), z=z, z_scale=scale)
    torch.cuda.synchronize()
    rz = torch.cat([x.double() @ w.double().T for w in wg[0].split(8192)], dim=1)
    mz = torch.cat([x.double().abs() @ w.double().abs().T for w in wg[0].split(8192)], dim=1)
    h = rz[:, :I] / (1 + torch.exp(-rz[:, :I])) * rz[:, I:]
    ry = torch.cat([h @ w.double().T for w in wd[0].split(8192)], dim=1)
    my = torch.cat([h.abs() @ w.double().abs().T for w in wd[0].split(8192)], dim=1)
    ez = (H + 4) * U * mz
    if eight:
        at = torch.arange(I, device=DEV) // 128
        s = scale.double()[:, torch.cat([at, G + at])]
        assert bool((((z.float().double() * s) - rz).abs() <= ez + rz.abs() * 2.0 ** -4 * 1.01 + s * 2.0 ** -10 * 1.01).all())
    else:
        assert bool(((z.double() - rz).abs() <= ez + rz.abs() * 2.0 ** -11 * 1.01 + 2.0 ** -25).all())
    # h is off by its rounding and by what gate and up are off, times at most 1.13 |up| and |gate|
    eh = h.abs() * 2.0 ** -11 * 1.01 + 2.0 ** -25 + ez[:, :I] * 1.13 * rz[:, I:].abs() * 1.01 + ez[:, I:] * rz[:, :I].abs() * 1.01 + 64 * U
    ey = torch.cat([eh @ w.double().abs().T for w in wd[0].split(8192)], dim=1) + (I + 4) * U * my * 1.01
    assert bool(((y.double() - ry).abs() <= ey + (ry.abs() + ey) * 2.0 ** -11 + 2.0 ** -25).all())


def test_not_a_number_stays_where_it_is(torch):
    say("NaN and infinity in one row, in one group of the 8-bit checkpoint")
    E, S, H, I = 2, 300, 64, 288
    shp = B.shape(H, I, E, 1)
    off = np.array([0, 140, 300], dtype=np.int32)
    x, wg, wd = rand(torch, 1, (S, H), "bf16"), rand(torch, 2, (E, 2 * I, H), "bf16", 0.1), rand(torch, 3, (E, H, I), "bf16", 0.1)
    clean = [torch.empty((S, H), dtype=x.dtype, device=DEV), torch.empty((S, 2 * I), dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn),
             torch.empty((S, 6), device=DEV)]
    got = [torch.empty_like(t) for t in clean]
    ws = scratch(torch, B.pw_moe_ffn_workspace_bytes(shp, S))
    run = lambda o: B.pw_moe_ffn(shp, S, x, wg, wd, o[0], ws, offsets=on_gpu(torch, off), z=o[1], z_scale=o[2])
    run(clean)
    x[139, 5] = float("nan")
    wg[1, 130, 7] = float("inf")                     # gate's second group of every row of the second expert
    run(got)
    torch.cuda.synchronize()
    assert torch.equal(got[0][:139], clean[0][:139]) and bool(got[0][139].isnan().all())
    assert torch.equal(got[1].view(torch.uint8)[:139], clean[1].view(torch.uint8)[:139])
    assert bool(got[2][139].isnan().all()) and bool((got[1].view(torch.uint8)[139] == 0x7F).all())
    assert bool(got[2][140:, 1].isnan().all()) and bool((got[1].view(torch.uint8)[140:, 128:256] == 0x7F).all())
    keep = [0, 2, 3, 4, 5]
    assert torch.equal(got[2][140:, keep], clean[2][140:, keep])
    assert torch.equal(got[1].view(torch.uint8)[140:, 256:], clean[1].view(torch.uint8)[140:, 256:])


def training_calls(torch, seed, S, E, H, I, name="bf16"):
    """A forward and a backward call on buffers of their own, and what they write."""
    shp = B.shape(H, I, E, 1)
    off = on_gpu(torch, starts(seed, S, E, behind=S // 9))
    x, dy = rand(torch, seed, (S, H), name), rand(torch, seed + 1, (S, H), name)
    wg, wd = rand(torch, seed + 2, (E, 2 * I, H), name, H ** -0.5), rand(torch, seed + 3, (E, H, I), name, I ** -0.5)
    z = torch.zeros((S, 2 * I), dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn)
    scale = torch.zeros((S, 2 * -(-I // 128)), device=DEV)
    out = [torch.zeros_like(x), z, scale, torch.zeros_like(x), torch.zeros_like(wg), torch.zeros_like(wd)]
    ws = [scratch(torch, B.pw_moe_ffn_workspace_bytes(shp, S)), scratch(torch, B.pw_moe_ffn_backward_workspace_bytes(shp, S))]

    def run(stream=None):
        B.pw_moe_ffn(shp, S, x, wg, wd, out[0], ws[0], offsets=off, z=z, z_scale=scale, stream=stream)
        B.pw_moe_ffn_backward(shp, S, dy, x, wg, wd, z, ws[1], offsets=off, z_scale=scale, dx=out[3], dw_gate_up=out[4],
                              dw_down=out[5], stream=stream)
    return run, out, x


def bits(torch, out):
    return [t.clone().view(torch.uint8) for t in out]


def test_two_streams_and_two_graphs(torch):
    say("two streams at once, then two graphs replayed in turn with eager work between")
    sizes = [(1200, 4, 256, 352), (300, 9, 128, 2720)]
    calls = [training_calls(torch, 10 * i + 1, *s) for i, s in enumerate(sizes)]
    for run, _, _ in calls:
        run()
    torch.cuda.synchronize()
    want = [bits(torch, out) for _, out, _ in calls]
    for _, out, _ in calls:
        for t in out:
            t.view(torch.uint8).zero_()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(3):
        for (run, _, _), s in zip(calls, streams):
            run(stream=s)
    torch.cuda.synchronize()
    for (_, out, _), w in zip(calls, want):
        assert all(torch.equal(a, b) for a, b in zip(bits(torch, out), w))
    graphs = []
    for run, _, _ in calls:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            run()
        graphs.append(g)
    inputs = [x.clone() for _, _, x in calls]
    for turn in range(3):
        for (run, out, x), x0, w in zip(calls, inputs, want):
            x.copy_(x0 * (1 + turn))
            run()                                       # eager, for the same inputs
        torch.cuda.synchronize()
        eager = [bits(torch, out) for _, out, _ in calls]
        for _, out, _ in calls:
            for t in out:
                t.view(torch.uint8).fill_(0x55)
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        for (_, out, _), w, off in zip(calls, eager, sizes):
            n = off[0] - off[0] // 9
            now = bits(torch, out)
            assert all(torch.equal(a[:n], b[:n]) for a, b in zip(now[:4], w[:4]))
            assert all(torch.equal(a, b) for a, b in zip(now[4:], w[4:]))


def test_chain_from_the_router_and_back(torch):
    """Router, sort, block, weighted return, and the gradients back to x, the matrices and the router, against automatic
    differentiation in 64 bits with the router's choice held.

    On every path at most four values are rounded to fp16 between input and result (h, the rows, y; or drows, dz, the
    sorted gradient, dx), each by at most half a step, 2^-11, of itself.  A rounding's error passes at most two matrices
    after it, and a matrix of n x m random numbers stretches no vector more than (sqrt n + sqrt m) / sqrt n <= 2.3 times
    as much as it does a random one, so in the 2-norm a result is off by less than 4 * 2.3^2 < 24 half steps of its size.
    """
    T, H, I, E, k = 200, 96, 128, 6, 2
    say(f"chain T={T} H={H} I={I} E={E} k={k}")
    shp = B.shape(H, I, E, k)
    S = T * k
    x, rw = rand(torch, 1, (T, H), "f16"), rand(torch, 2, (E, H), "f16", H ** -0.5)
    wg, wd = rand(torch, 3, (E, 2 * I, H), "f16", H ** -0.5), rand(torch, 4, (E, H, I), "f16", I ** -0.5)
    dy = rand(torch, 5, (T, H), "f16")
    i32, f16 = dict(dtype=torch.int32, device=DEV), dict(dtype=torch.float16, device=DEV)
    ids, w = torch.empty((T, k), **i32), torch.empty((T, k), device=DEV)
    ws = scratch(torch, max(B.pw_workspace_bytes(shp, T), B.pw_moe_permute_workspace_bytes(shp, T),
                            B.pw_moe_ffn_backward_workspace_bytes(shp, S), B.pw_router_backward_workspace_bytes(shp, T)))
    B.pw_router_topk(shp, T, x, rw, ids, w, workspace=ws)
    xs, off, inv = torch.empty((S, H), **f16), torch.empty(E + 1, **i32), torch.empty(S, **i32)
    B.pw_moe_permute(shp, T, x, ids, xs, off, inv, None, ws)
    rows, y, z = torch.empty((S, H), **f16), torch.empty((T, H), **f16), torch.empty((S, 2 * I), **f16)
    B.pw_moe_ffn(shp, S, xs, wg, wd, rows, ws, offsets=off, z=z)
    B.pw_moe_unpermute(shp, T, rows, inv, w, y)
    drows, dw = torch.empty((S, H), **f16), torch.empty((T, k), device=DEV)
    B.pw_moe_unpermute_backward(shp, T, dy, rows, inv, w, drows, dw)
    dxs, dwg, dwd = torch.empty((S, H), **f16), torch.empty_like(wg), torch.empty_like(wd)
    B.pw_moe_ffn_backward(shp, S, drows, xs, wg, wd, z, ws, offsets=off, dx=dxs, dw_gate_up=dwg, dw_down=dwd)
    dx, drw = torch.empty((T, H), **f16), torch.empty((E, H), device=DEV)
    B.pw_moe_permute_backward(shp, T, dxs, inv, dx)
    B.pw_router_backward(shp, T, x, rw, ids, w, dw, dx, drw, ws, dx_add=dx)
    torch.cuda.synchronize()
    X, RW, WG, WD = (t.cpu().double().requires_grad_() for t in (x, rw, wg, wd))
    at = ids.cpu().long()
    weight = torch.softmax((X @ RW.T).gather(1, at), dim=1)
    out = torch.zeros((T, H), dtype=torch.float64)
    for e in range(E):
        zz = X @ WG[e].T
        o = (torch.nn.functional.silu(zz[:, :I]) * zz[:, I:]) @ WD[e].T
        out = out + o * (weight * (at == e)).sum(1, keepdim=True)
    out.backward(dy.cpu().double())
    for got, ref, what in [(y, out.detach(), "y"), (dx, X.grad, "dx"), (dwg, WG.grad, "dw_gate_up"), (dwd, WD.grad, "dw_down"),
                           (drw, RW.grad, "drouter_w")]:
        off_by = float((got.cpu().double() - ref).norm() / ref.norm())
        say(f"  {what}: {off_by * 2 ** 11:.2f} half steps")
        assert off_by < 24 * 2.0 ** -11, what


def test_binding_refusals_on_the_gpu(torch):
    x, w = rand(torch, 1, (8, 64), "f16"), rand(torch, 2, (1, 64, 64), "f16")
    y, ws = torch.empty_like(x), scratch(torch, 1 << 16)
    bad = B.PW_ERR_INVALID_ARG
    call = lambda **k: B.pw_moe_product(1, 8, 64, 64, **{**dict(x=x, w=w, y=y, workspace=ws), **k}, check=False)
    assert call() == B.PW_OK
    assert call(x=x.float()) == bad and call(w=w.bfloat16()) == bad and call(y=y.t()) == bad and call(x=x[:7]) == bad
    assert call(w=w[:, :63]) == bad and call(bias=x[0, :32]) == bad and call(offsets=torch.zeros(2, device=DEV)) == bad
    assert call(workspace=None) == bad and call(residual=x[:, ::2]) == bad
    assert call(stream=torch.cuda.Stream()) == B.PW_OK
    assert B.pw_moe_product(1, 8, 64, 64, x.float(), w.float(), y.float(), ws, check=False) == bad
    shp = B.shape(64, 64, 1, 1)
    wg, z = rand(torch, 3, (1, 128, 64), "f16"), torch.empty((8, 128), dtype=torch.float8_e4m3fn, device=DEV)
    f = lambda **k: B.pw_moe_ffn(shp, 8, **{**dict(x=x, w_gate_up=wg, w_down=w, y=y, workspace=ws), **k}, check=False)
    assert f() == B.PW_OK and f(z=z) == bad and f(z=z, z_scale=torch.empty((8, 1), device=DEV)) == bad
    assert f(z=z, z_scale=torch.empty((8, 2), device=DEV)) == B.PW_OK
    assert f(w_gate_up=w) == bad and f(z=z[:, :64], z_scale=torch.empty((8, 2), device=DEV)) == bad
    torch.cuda.synchronize()
