"""The operators around the layer on the GPU, against their 64-bit definitions.

Tolerances.  U = 2^-24 is half a step of fp32.  Every result is computed in fp32
and rounded once, so it may be off by half a step of its type relative to its
value (plus half a subnormal step), and by U times the length of the longest
chain of additions times the sum of the addends' magnitudes.  Chains: a row's
sums add at most 32 values a lane, then 6 levels of a wave and 15 waves, so 64
covers them with the few factors' roundings; the others are stated where used.
Copies and whole numbers are equal.  Every case prints what it runs first.
"""
import sys

import numpy as np
import pytest

import oracle.ops_oracle as oo
import oracle.pagedweight_oracle as orc
from any_precision_bitplane_amd import binding as B
from any_precision_bitplane_amd import synth
from any_precision_bitplane_amd.device import DeviceLayer

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
ROW = 64
EPS = 1e-5
DEV = "cuda:0"
DTYPES = ["f32", "f16", "bf16"]


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
    return {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn}[name]


def half_step(torch, name):
    """(relative, absolute) half steps of a row type."""
    f = torch.finfo(dtype_of(torch, name))
    return f.eps / 2, f.smallest_normal * f.eps / 2


def f64(t):
    return t.detach().cpu().to(__import__("torch").float32).double().numpy()


def rand(torch, seed, shape, name, std=1.0, pad=0):
    g = torch.Generator().manual_seed(seed)
    a = torch.randn((*shape[:-1], shape[-1] + pad), generator=g) * std
    return a.to(dtype_of(torch, name)).to(DEV)[..., :shape[-1]]


def near(got, ref, allowed, what):
    err = np.abs(got - ref)
    assert np.all(np.isfinite(got)), what
    over = err - allowed
    worst = float(np.max(err / np.maximum(allowed, 1e-300))) if err.size else 0.0
    say(f"  {what}: max abs {float(err.max()) if err.size else 0.0:.3e}, {worst:.2f} of what is allowed")
    assert not err.size or over.max() <= 0, (what, worst)


# ----- norm -----------------------------------------------------------------

NORM_SIZES = [(1, 8), (37, 40), (2050, 128), (19, 136), (1500, 256), (3, 64), (5, 520), (1, 2048),
              (2, 4104), (7, 8192), (2, 16384), (1, 32768),
              (1025, 64), (1030, 520), (1027, 1000), (1026, 2080), (1025, 4096), (1025, 8200), (1025, 16392),
              (1025, 24576)]


@pytest.mark.parametrize("name", DTYPES)
@pytest.mark.parametrize("T,H", NORM_SIZES, ids=[f"{t}x{h}" for t, h in NORM_SIZES])
def test_rmsnorm(torch, T, H, name):
    say(f"rmsnorm {name} T={T} H={H}")
    x, res = rand(torch, 1, (T, H), name, pad=8), rand(torch, 2, (T, H), name, 4.0)
    g = rand(torch, 3, (1, H), name)[0]
    out, y = torch.full_like(res, 7.0), torch.full((T, H + 16), 7.0, dtype=res.dtype, device=DEV)
    B.pw_rmsnorm(T, H, x, g, EPS, y[:, :H], residual=res, residual_out=out)
    plain = torch.full_like(res, 7.0)
    B.pw_rmsnorm(T, H, x, g, EPS, plain)
    torch.cuda.synchronize()
    rel, ab = half_step(torch, name)
    assert torch.equal(out, (x.float() + res.float()).to(res.dtype))
    assert bool((y[:, H:] == 7.0).all())
    for got, ref, what in [(y[:, :H], oo.rmsnorm(f64(x), f64(g), EPS, f64(res))[1], "y"),
                           (plain, oo.rmsnorm(f64(x), f64(g), EPS)[1], "y without a residual")]:
        near(f64(got), ref, np.abs(ref) * (rel + ROW * U) + ab, what)


@pytest.mark.parametrize("name", DTYPES)
@pytest.mark.parametrize("T,H,group", [(1, 64, 0), (1, 64, 128), (70, 40, 128), (70, 40, 0), (2049, 128, 128),
                                       (9, 128, 0), (1026, 256, 128),
                                       (33, 232, 0), (3, 136, 128), (5, 2048, 128), (4, 2080, 0),
                                       (2, 32768, 0), (1, 32768, 128), (1030, 520, 128), (1025, 4096, 0),
                                       (1025, 8200, 128), (1025, 16384, 0)])
def test_rmsnorm_e4m3(torch, T, H, group, name):
    say(f"rmsnorm e4m3 {name} T={T} H={H} group={group}")
    x, res = rand(torch, 1, (T, H), name), rand(torch, 2, (T, H), name, 4.0, pad=8)
    g = rand(torch, 3, (1, H), name)[0]
    x[0, :min(H, 128)] = 0
    res[0, :min(H, 128)] = 0                       # a group of zeros (a whole row of them where H <= 128)
    groups = -(-H // 128) if group else 1
    out = torch.empty_like(x)
    y = torch.empty((T, H), dtype=torch.float8_e4m3fn, device=DEV)
    scale = torch.full((T, groups), -1.0, device=DEV)
    B.pw_rmsnorm(T, H, x, g, EPS, y, residual=res, residual_out=out, scale=scale, group=group)
    torch.cuda.synchronize()
    assert torch.equal(out, (x.float() + res.float()).to(x.dtype))
    ref = oo.rmsnorm(f64(x), f64(g), EPS, f64(res))[1]
    rs = oo.e4m3_scales(ref, group)
    near(f64(scale), rs, rs * (ROW + 2) * U, "scale")
    wide = np.repeat(f64(scale), group if group else H, axis=1)[:, :H]
    # half a step of e4m3 (2^-4 of the value, 2^-10 of the scale below its normal numbers), and the fp32 work before it
    code = np.maximum(np.abs(ref) * 2.0 ** -4, wide * 2.0 ** -10)
    near(f64(y) * wide, ref, code + (np.abs(ref) + wide) * 2 * ROW * U, "code * scale")
    assert np.max(np.abs(f64(y))) == (448.0 if ref.any() else 0.0)


def test_rmsnorm_in_place_and_special_rows(torch):
    say("rmsnorm: sum and output in place, rows with NaN, infinity, zeros, largest and smallest values")
    T, H = 6, 512
    x, res = rand(torch, 1, (T, H), "f16"), rand(torch, 2, (T, H), "f16")
    g = rand(torch, 3, (1, H), "f16")[0]
    out, y = torch.empty_like(x), torch.empty_like(x)
    B.pw_rmsnorm(T, H, x, g, EPS, y, residual=res, residual_out=out)
    x2, res2 = x.clone(), res.clone()
    B.pw_rmsnorm(T, H, x2, g, EPS, x2, residual=res2, residual_out=res2)      # y over x, r over residual
    x3 = x.clone()
    B.pw_rmsnorm(T, H, x3, g, EPS, y3 := torch.empty_like(x), residual=res, residual_out=x3)   # r over x
    assert torch.equal(x2, y) and torch.equal(res2, out) and torch.equal(x3, out) and torch.equal(y3, y)

    x[0, 5], x[1, 7], x[2], x[3], x[4] = float("nan"), float("inf"), 0.0, 65504.0, 2.0 ** -24
    codes = torch.zeros((T, H), dtype=torch.float8_e4m3fn, device=DEV)
    scale = torch.empty((T, 4), device=DEV)
    B.pw_rmsnorm(T, H, x, g, EPS, y)
    B.pw_rmsnorm(T, H, x, g, EPS, codes, scale=scale, group=128)
    torch.cuda.synchronize()
    assert bool(y[0].isnan().all())
    assert bool(y[1, 7].isnan()) and bool((y[1, 8:] == 0).all())
    assert bool((y[2] == 0).all()) and bool((scale[2] == 2.0 ** -100).all()) and bool((codes[2].float() == 0).all())
    assert bool(scale[0].isnan().all()) and bool(codes[0].float().isnan().all())
    assert bool(scale[1, 0].isnan()) and bool(codes[1, :128].float().isnan().all())
    assert bool((scale[1, 1:] == 2.0 ** -100).all()) and bool((codes[1, 128:].float() == 0).all())
    for t in (3, 4, 5):
        ref = oo.rmsnorm(f64(x[t:t + 1]), f64(g), EPS)[1]
        near(f64(y[t:t + 1]), ref, np.abs(ref) * (2.0 ** -11 + ROW * U) + 2.0 ** -25, f"row {t}")


@pytest.mark.parametrize("H", [40, 136, 520, 1160, 4104, 8200, 16392])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_rmsnorm_e4m3_weight_that_is_not_finite(torch, H, value):
    say(f"rmsnorm e4m3 H={H}: weight[3] = {value} shows in its own group only")
    T, groups = 5, -(-H // 128)
    x, g = rand(torch, 1, (T, H), "bf16"), rand(torch, 2, (1, H), "bf16")[0]
    good = [torch.zeros((T, H), dtype=torch.float8_e4m3fn, device=DEV), torch.zeros((T, groups), device=DEV)]
    bad = [torch.zeros_like(good[0]), torch.zeros_like(good[1])]
    B.pw_rmsnorm(T, H, x, g, EPS, good[0], scale=good[1], group=128)
    g[3] = value
    B.pw_rmsnorm(T, H, x, g, EPS, bad[0], scale=bad[1], group=128)
    torch.cuda.synchronize()
    assert bool(bad[1][:, 0].isnan().all()) and bool(bad[0][:, :128].float().isnan().all())
    assert torch.equal(bad[1][:, 1:], good[1][:, 1:])
    assert torch.equal(bad[0][:, 128:].view(torch.uint8), good[0][:, 128:].view(torch.uint8))


GRAD_SIZES = [(1, 8), (6007, 40), (9000, 128), (4500, 200), (2050, 256), (3, 64), (2, 32768),
              (5, 8200), (700, 4096), (2500, 520), (1025, 2080), (513, 8192), (514, 16384),
              (515, 24576), (3000, 512)]


@pytest.mark.parametrize("name", DTYPES)
@pytest.mark.parametrize("T,H", GRAD_SIZES, ids=[f"{t}x{h}" for t, h in GRAD_SIZES])
def test_rmsnorm_backward(torch, T, H, name):
    say(f"rmsnorm_backward {name} T={T} H={H}")
    dy, r = rand(torch, 1, (T, H), name, 0.1, pad=8), rand(torch, 2, (T, H), name, 3.0)
    g, dres = rand(torch, 3, (1, H), name)[0], rand(torch, 4, (T, H), name, 0.1, pad=16)
    ws = torch.full((B.pw_rmsnorm_backward_workspace_bytes(T, H),), 255, dtype=torch.uint8, device=DEV)
    dx, dg = torch.empty_like(r), torch.full((H,), 7.0, device=DEV)
    B.pw_rmsnorm_backward(T, H, dy, r, g, EPS, dx, dg, ws, dresidual=dres)
    alone = torch.empty_like(r)
    B.pw_rmsnorm_backward(T, H, dy, r, g, EPS, alone)
    over = [dy.clone(), r.clone(), dres.clone()]
    B.pw_rmsnorm_backward(T, H, over[0], r, g, EPS, over[0], dresidual=dres)
    B.pw_rmsnorm_backward(T, H, dy, over[1], g, EPS, over[1], dresidual=dres)
    B.pw_rmsnorm_backward(T, H, dy, r, g, EPS, over[2], dresidual=over[2])
    torch.cuda.synchronize()
    assert all(torch.equal(o, dx) for o in over)
    d, rr, gg, a = f64(dy), f64(r), f64(g), f64(dres)
    rel, ab = half_step(torch, name)
    s = 1 / np.sqrt(np.mean(rr * rr, axis=1, keepdims=True) + EPS)
    mag = np.abs(s * gg * d) + np.abs(rr) * s ** 3 * np.sum(np.abs(gg * d * rr), axis=1, keepdims=True) / H
    for got, add, what in [(dx, a, "dx"), (alone, np.zeros_like(a), "dx without the stream's gradient")]:
        ref, dgr = oo.rmsnorm_backward(d, rr, gg, EPS, add)
        near(f64(got), ref, np.abs(ref) * rel + ab + 2 * ROW * U * (mag + np.abs(add)), what)
    # a lane adds at most ceil(T / 256) rows, a block 32 lanes' shares, then 512 blocks: 8 a thread and six levels
    chain = -(-T // 256) + 32 + 8 + 6 + ROW
    near(f64(dg), dgr, chain * U * np.sum(np.abs(d * rr * s), axis=0), "dweight")


def test_rmsnorm_backward_against_differences(torch):
    say("rmsnorm_backward: central differences of the fp32 forward")
    T, H, h = 3, 64, 2.0 ** -7
    r, dy, g = rand(torch, 1, (T, H), "f32"), rand(torch, 2, (T, H), "f32"), rand(torch, 3, (1, H), "f32")[0]
    ws = torch.empty(B.pw_rmsnorm_backward_workspace_bytes(T, H), dtype=torch.uint8, device=DEV)
    dx, dg = torch.empty_like(r), torch.empty(H, device=DEV)
    B.pw_rmsnorm_backward(T, H, dy, r, g, EPS, dx, dg, ws)

    def loss(a, b):
        y = torch.empty_like(a)
        B.pw_rmsnorm(T, H, a, b, EPS, y)
        return float((y.double() * dy.double()).sum())

    # |y| <= ~4, so a difference carries 2 * 192 * 4 * 64 U / (2 h) ~ 0.4 at the very worst and about 1e-4 as roundings
    # fall; the second-order term of the difference is h^2 |y'''| / 6 ~ 1e-5 times |dy|
    for t, c in [(0, 0), (1, 17), (2, 63)]:
        up, down = r.clone(), r.clone()
        up[t, c] += h
        down[t, c] -= h
        assert abs((loss(up, g) - loss(down, g)) / (2 * h) - float(dx[t, c])) < 5e-3
        up, down = g.clone(), g.clone()
        up[c] += h
        down[c] -= h
        assert abs((loss(r, up) - loss(r, down)) / (2 * h) - float(dg[c])) < 5e-3


def test_rmsnorm_backward_of_no_rows(torch):
    say("rmsnorm_backward: T = 0 clears dweight")
    e = torch.empty((0, 64), device=DEV)
    dg = torch.full((64,), 7.0, device=DEV)
    B.pw_rmsnorm_backward(0, 64, e, e, torch.ones(64, device=DEV), EPS, e, dg)
    torch.cuda.synchronize()
    assert bool((dg == 0).all())


# ----- sorting ----------------------------------------------------------------

# name, T, H, E, k, share of dropped slots; up to 6144 slots one launch, above two, from about half a million three
SORT_CASES = [("one", 1, 32, 1, 1, 0.0), ("decode", 4, 2048, 60, 4, 0.0), ("odd", 7, 96, 5, 3, 0.3),
              ("all_dropped", 9, 64, 8, 2, 1.0), ("E256_k64", 5, 64, 256, 64, 0.1), ("E256_k256", 2, 32, 256, 256, 0.0),
              ("more_experts_than_tokens", 3, 64, 200, 2, 0.0), ("edge_4096", 1024, 96, 60, 4, 0.1),
              ("edge_6144", 1536, 96, 60, 4, 0.1), ("above_6144", 1537, 320, 60, 4, 0.1),
              ("above_4096", 1025, 96, 60, 4, 0.1), ("one_expert", 5000, 64, 1, 1, 0.0),
              ("large", 4099, 160, 8, 2, 0.05),
              ("E256_k8", 1500, 64, 256, 8, 0.2), ("E256_k256_large", 40, 32, 256, 256, 0.1),
              ("all_dropped_large", 5001, 32, 9, 1, 1.0), ("k7", 3001, 64, 33, 7, 0.5),
              ("scanned", 140003, 32, 60, 4, 0.1), ("scanned_k64", 9001, 32, 256, 64, 0.1)]


def draw_ids(seed, T, E, k, dropped):
    rng = np.random.default_rng(seed)
    ids = np.stack([rng.permutation(E)[:k] for _ in range(T)]).astype(np.int32)
    lost = rng.random((T, k)) < dropped
    ids[lost] = rng.choice(np.array([-1, E, 2 ** 31 - 1, -2 ** 31], np.int64), size=int(lost.sum())).astype(np.int32)
    return ids


def plan(ids, E):
    """(offsets, inv, perm) of the oracle's sort, quickly: the definition is pinned on small inputs."""
    flat = ids.reshape(-1).astype(np.int64)
    kept = (flat >= 0) & (flat < E)
    perm = np.nonzero(kept)[0][np.argsort(flat[kept], kind="stable")]
    inv = np.full(flat.shape, -1, np.int64)
    inv[perm] = np.arange(len(perm))
    return np.concatenate([[0], np.cumsum(np.bincount(flat[kept], minlength=E))]), inv, perm


def run_permute(torch, x, ids, E, scale=None, stream=None, ws=None, perm=True, xs_pad=0):
    T, H = x.shape
    k = ids.shape[1]
    S = T * k
    shp = B.shape(H, 32, E, k)
    raw = torch.full((S, H + xs_pad), 3, dtype=torch.uint8 if x.element_size() == 1 else x.dtype, device=DEV)
    xs = raw.view(x.dtype)[:, :H]
    offsets = torch.full((E + 1,), -9, dtype=torch.int32, device=DEV)
    inv, pm = (torch.full((S,), -9, dtype=torch.int32, device=DEV) for _ in range(2))
    xsc = torch.full((S, scale.shape[1]), 3.0, device=DEV) if scale is not None else None
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    if ws is None:
        ws = torch.full((B.pw_moe_permute_workspace_bytes(shp, T),), 255, dtype=torch.uint8, device=DEV)
    idd = torch.from_numpy(ids).to(DEV)
    B.pw_moe_permute(shp, T, x, idd, xs, offsets, inv, pm if perm else None, ws, x_scale=scale, xs_scale=xsc,
                     status=status, stream=stream)
    torch.cuda.synchronize()
    return xs, offsets, inv, pm, xsc, int(status.item()), raw


@pytest.mark.parametrize("name,T,H,E,k,dropped", SORT_CASES, ids=[c[0] for c in SORT_CASES])
def test_permute(torch, name, T, H, E, k, dropped):
    ids = draw_ids(11, T, E, k, dropped)
    offsets, inv, perm = plan(ids, E)
    n = len(perm)
    if T * k <= 600:
        o = oo.sort_slots(ids, E)
        assert all(np.array_equal(a, b) for a, b in zip(o, (offsets, inv, perm)))
    for dt in DTYPES + ["e4m3"]:
        say(f"permute {name} {dt} T={T} H={H} E={E} k={k}: {n} of {T * k} slots kept")
        x = rand(torch, 5, (T, H), dt, pad=16)
        scale = torch.rand((T, 3), device=DEV) if dt == "e4m3" else None
        xs, off, iv, pm, xsc, status, raw = run_permute(torch, x, ids, E, scale, xs_pad=16)
        assert np.array_equal(off.cpu().numpy(), offsets)
        assert np.array_equal(iv.cpu().numpy(), inv)
        assert np.array_equal(pm[:n].cpu().numpy(), perm) and bool((pm[n:] == -9).all())
        assert status == (B.PW_DEV_BAD_EXPERT_ID if n < T * k else 0)
        bits = lambda t: t.contiguous().view(torch.uint8)
        tok = torch.from_numpy(perm // k).to(DEV)
        assert torch.equal(bits(xs[:n]), bits(x).reshape(T, -1)[tok].reshape(bits(xs[:n]).shape))
        assert bool((raw[n:] == 3).all()) and bool((raw[:, H:] == 3).all())       # left as they were
        if scale is not None:
            assert torch.equal(xsc[:n], scale[tok]) and bool((xsc[n:] == 3.0).all())
    if dropped == 0.0:
        assert run_permute(torch, x, ids, E, scale, perm=False)[3].eq(-9).all()


@pytest.mark.parametrize("T,H", [(30001, 1024), (140001, 512), (120001, 256), (230001, 128)])
def test_permute_of_large_outputs(torch, T, H):
    """Wide and narrow rows, with and without the scan launch, at hundreds of MiB."""
    E, k = 60, 4
    say(f"permute T={T} H={H} k={k}: {T * k * H * 2 >> 20} MiB of copies")
    ids = draw_ids(5, T // 100, E, k, 0.1)
    ids = np.tile(ids, (101, 1))[:T].copy()
    offsets, inv, perm = plan(ids, E)
    x = rand(torch, 5, (T, H), "f16")
    xs, off, iv, pm, _, _, raw = run_permute(torch, x, ids, E)
    n = len(perm)
    assert np.array_equal(off.cpu().numpy(), offsets) and np.array_equal(iv.cpu().numpy(), inv)
    assert np.array_equal(pm[:n].cpu().numpy(), perm)
    assert torch.equal(xs[:n], x[torch.from_numpy(perm // k).to(DEV)]) and bool((raw[n:] == 3).all())


def test_permute_same_expert_twice(torch):
    say("permute: tokens that list an expert more than once")
    for T in (50, 3000):
        ids = np.random.default_rng(1).integers(0, 3, size=(T, 4)).astype(np.int32)
        offsets, inv, perm = plan(ids, 4)
        x = rand(torch, 5, (T, 64), "f16")
        xs, off, iv, pm, _, status, _ = run_permute(torch, x, ids, 4)
        assert status == 0 and np.array_equal(off.cpu().numpy(), offsets) and np.array_equal(iv.cpu().numpy(), inv)
        assert np.array_equal(pm.cpu().numpy(), perm)
        assert torch.equal(xs, x[torch.from_numpy(perm // 4).to(DEV)])


def test_permute_of_no_tokens(torch):
    say("permute: T = 0 clears the offsets")
    shp = B.shape(64, 32, 8, 2)
    e, i = torch.empty((0, 64), device=DEV), torch.empty(0, dtype=torch.int32, device=DEV)
    off = torch.full((9,), 5, dtype=torch.int32, device=DEV)
    B.pw_moe_permute(shp, 0, e, i, e, off, i, i, torch.empty(8192, dtype=torch.uint8, device=DEV))
    B.pw_moe_unpermute(shp, 0, e, i, None, e)
    torch.cuda.synchronize()
    assert bool((off == 0).all())


@pytest.mark.parametrize("dt", DTYPES)
@pytest.mark.parametrize("name,T,H,E,k,dropped", SORT_CASES, ids=[c[0] for c in SORT_CASES])
def test_unpermute_and_gradients(torch, name, T, H, E, k, dropped, dt):
    say(f"unpermute {name} {dt} T={T} H={H} E={E} k={k}")
    ids = draw_ids(11, T, E, k, dropped)
    _, inv, perm = plan(ids, E)
    S, n = T * k, len(perm)
    shp = B.shape(H, 32, E, k)
    iv = torch.from_numpy(inv.astype(np.int32)).to(DEV)
    rows, dy = rand(torch, 5, (S, H), dt, pad=16), rand(torch, 6, (T, H), dt, 0.1, pad=8)
    rows[n:] = float("nan")                          # rows without a slot are never read
    w = rand(torch, 7, (T, k), "f32")
    y, dx = (torch.full((T, H + 8), 7.0, dtype=dy.dtype, device=DEV) for _ in range(2))
    drows, dw = torch.full((S, H + 8), 7.0, dtype=dy.dtype, device=DEV), torch.full((T, k), 7.0, device=DEV)
    B.pw_moe_unpermute(shp, T, rows, iv, w, y[:, :H])
    B.pw_moe_permute_backward(shp, T, rows, iv, dx[:, :H])
    B.pw_moe_unpermute_backward(shp, T, dy, rows, iv, w, drows[:, :H], dw)
    ones, only = torch.full_like(y, 7.0), torch.full_like(drows, 7.0)
    B.pw_moe_unpermute(shp, T, rows, iv, None, ones[:, :H])
    B.pw_moe_unpermute_backward(shp, T, dy, None, iv, w, only[:, :H])
    place = rows.clone()
    dw2 = torch.empty_like(dw)
    B.pw_moe_unpermute_backward(shp, T, dy, place, iv, w, place, dw2)             # drows over rows
    torch.cuda.synchronize()
    assert torch.equal(ones, dx) and torch.equal(only, drows) and torch.equal(place[:n], drows[:n, :H])
    assert torch.equal(dw2, dw)
    assert bool((y[:, H:] == 7).all()) and bool((drows[n:] == 7).all()) and bool((drows[:, H:] == 7).all())
    rel, ab = half_step(torch, dt)
    R, W, D = f64(rows), f64(w), f64(dy)
    R[n:] = 0.0
    got = R[np.where(inv >= 0, inv, S - 1)].reshape(T, k, H) * (inv >= 0).reshape(T, k, 1)
    for out, weights, what in [(y, W, "y"), (dx, np.ones_like(W), "dx")]:
        ref = np.sum(got * weights[:, :, None], axis=1)
        mag = np.sum(np.abs(got * weights[:, :, None]), axis=1)
        if S * H <= 20000:
            np.testing.assert_allclose(ref, oo.unpermute(R, inv, weights, T, k), rtol=0, atol=1e-12)
        near(f64(out[:, :H]), ref, np.abs(ref) * rel + ab + (k + 1) * U * mag, what)
    tok, kept = perm // k, (inv >= 0).reshape(T, k)
    ref = W.reshape(-1)[perm][:, None] * D[tok]
    near(f64(drows[:n, :H]), ref, np.abs(ref) * (rel + U) + ab, "drows")
    refdw = np.sum(got * D[:, None, :], axis=2)
    mag = np.sum(np.abs(got * D[:, None, :]), axis=2)
    near(f64(dw), refdw, (8 * (-(-H // 512)) + 8) * U * mag, "dw")                # a lane's chunks, then 6 levels
    assert np.all(f64(dw)[~kept] == 0)


def test_unpermute_long_rows_and_bad_places(torch):
    say("unpermute: H = 8192, entries of inv outside the rows are dropped slots")
    T, H, k = 6, 8192, 3
    shp = B.shape(H, 32, 8, k)
    inv = np.arange(T * k, dtype=np.int32)
    inv[[2, 5, 9]] = [-5, T * k, 2 ** 31 - 1]
    iv = torch.from_numpy(inv).to(DEV)
    rows, w, dy = rand(torch, 5, (T * k, H), "bf16"), rand(torch, 7, (T, k), "f32"), rand(torch, 6, (T, H), "bf16")
    y, dw = torch.empty((T, H), dtype=torch.bfloat16, device=DEV), torch.empty((T, k), device=DEV)
    drows = torch.full_like(rows, 7.0)
    B.pw_moe_unpermute(shp, T, rows, iv, w, y)
    B.pw_moe_unpermute_backward(shp, T, dy, rows, iv, w, drows, dw)
    torch.cuda.synchronize()
    ok = inv.copy()
    ok[(inv < 0) | (inv >= T * k)] = -1
    R, W, D = f64(rows), f64(w), f64(dy)
    ref, mag = oo.unpermute(R, ok, W, T, k), oo.unpermute(np.abs(R), ok, np.abs(W), T, k)
    near(f64(y), ref, np.abs(ref) * 2.0 ** -8 + (k + 1) * U * mag, "y")
    dr, rdw = oo.unpermute_backward(D, R, ok, W, T, k)
    assert bool((drows[[2, 5, 9]] == 7).all())
    keep = np.setdiff1d(np.arange(T * k), [2, 5, 9])
    near(f64(drows)[keep], dr[keep], np.abs(dr[keep]) * (2.0 ** -8 + U), "drows")
    near(f64(dw), rdw, 256 * U * oo.unpermute_backward(np.abs(D), np.abs(R), ok, W, T, k)[1], "dw")


def test_rows_past_32_bits(torch):
    """Element offsets past 2^31 and byte offsets past 2^32."""
    T, H, E, k = 150001, 8192, 8, 2
    say(f"permute and back: {T * k} rows of {H} bf16, {T * k * H * 2 / 2 ** 30:.1f} GiB")
    shp = B.shape(H, 32, E, k)
    g = torch.Generator(device=DEV).manual_seed(1)
    x = torch.randn((T, H), generator=g, device=DEV, dtype=torch.bfloat16)
    ids = torch.rand((T, E), generator=g, device=DEV).topk(k, dim=1).indices.int().contiguous()
    xs = torch.empty((T * k, H), dtype=torch.bfloat16, device=DEV)
    off, inv = torch.empty(E + 1, dtype=torch.int32, device=DEV), torch.empty(T * k, dtype=torch.int32, device=DEV)
    ws = torch.empty(B.pw_moe_permute_workspace_bytes(shp, T), dtype=torch.uint8, device=DEV)
    B.pw_moe_permute(shp, T, x, ids, xs, off, inv, None, ws)
    order = torch.argsort(ids.reshape(-1).long(), stable=True)
    for s in range(0, T * k, 50000):
        assert torch.equal(xs[s:s + 50000], x[order[s:s + 50000] // k])
    y = torch.empty_like(x)
    B.pw_moe_unpermute(shp, T, xs, inv, torch.full((T, k), 0.5, device=DEV), y)     # 0.5 x + 0.5 x
    assert torch.equal(y, x)
    dw = torch.empty((T, k), device=DEV)
    B.pw_moe_unpermute_backward(shp, T, x, xs, inv, torch.full((T, k), 2.0, device=DEV), xs, dw)
    for s in range(0, T * k, 50000):
        assert torch.equal(xs[s:s + 50000], (2 * x[order[s:s + 50000] // k].float()).bfloat16())
    out = torch.empty_like(x)
    B.pw_rmsnorm(T, H, x, torch.ones(H, dtype=torch.bfloat16, device=DEV), EPS, y, residual=y, residual_out=out)
    tail = x[-3:]
    assert torch.equal(out[-3:], (tail.float() * 2).bfloat16())
    ref = oo.rmsnorm(f64(tail), np.ones(H), EPS, f64(tail))[1]
    near(f64(y[-3:]), ref, np.abs(ref) * (2.0 ** -8 + ROW * U), "last rows' norm")
    square = np.repeat(np.sum(f64(tail) ** 2, axis=1, keepdims=True), k, axis=1)
    near(f64(dw[-3:]), square, (H // 64 + 8) * U * square, "last dw")


def test_more_rows_than_a_grid_has_blocks(torch):
    """Launches end at 2^20 blocks; the blocks then walk the remaining rows."""
    T, H = 34_000_001, 8
    say(f"norm and its gradient: {T} rows of {H}")
    g = torch.Generator(device=DEV).manual_seed(1)
    x = torch.randn((T, H), generator=g, device=DEV, dtype=torch.float16)
    w, y = torch.ones(H, dtype=torch.float16, device=DEV), torch.empty_like(x)
    B.pw_rmsnorm(T, H, x, w, EPS, y)
    ref = x.float() * torch.rsqrt(x.float().square().mean(dim=1, keepdim=True) + EPS)
    # two fp32 computations, each within ROW half steps, and one rounding to fp16 on this side
    assert bool(((y.float() - ref).abs() <= ref.abs() * (2.0 ** -11 + 2 * ROW * U) + 2.0 ** -25).all())
    del x, y, ref
    T, H, E = 67_200_003, 32, 8
    say(f"permute and back: {T} rows of {H}")
    shp = B.shape(H, 32, E, 1)
    x = torch.randint(0, 255, (T, H), generator=g, device=DEV, dtype=torch.uint8).half()
    ids = torch.randint(-1, E, (T, 1), generator=g, device=DEV, dtype=torch.int32)
    off, inv = torch.empty(E + 1, dtype=torch.int32, device=DEV), torch.empty(T, dtype=torch.int32, device=DEV)
    ws = torch.empty(B.pw_moe_permute_workspace_bytes(shp, T), dtype=torch.uint8, device=DEV)
    xs = torch.zeros_like(x)
    B.pw_moe_permute(shp, T, x, ids, xs, off, inv, None, ws)
    order = torch.argsort(torch.where(ids.reshape(-1) < 0, E, ids.reshape(-1)).to(torch.uint8), stable=True)
    n = int(off[E])
    assert n == int((ids >= 0).sum())
    assert torch.equal(inv[order[:n]], torch.arange(n, dtype=torch.int32, device=DEV))
    assert bool((inv[order[n:]] == -1).all())
    for s in range(0, n, 1 << 23):
        e = min(n, s + (1 << 23))
        assert torch.equal(xs[s:e], x[order[s:e]])
    y = torch.empty_like(x)
    B.pw_moe_unpermute(shp, T, xs, inv, None, y)
    kept = ids >= 0
    assert torch.equal(y, torch.where(kept, x, torch.zeros_like(x)))
    dw = torch.empty((T, 1), device=DEV)
    B.pw_moe_unpermute_backward(shp, T, x, xs, inv, None, xs, dw)      # whole numbers up to 32 * 254^2: exact in fp32
    torch.cuda.synchronize()
    assert torch.equal(dw, torch.where(kept, x.float().square().sum(dim=1, keepdim=True), 0.0))


def test_nan_in_masked_places(torch):
    """Padding holds anything: what a dropped slot or a padded token carries is never read into a result."""
    nan = float("nan")
    for T in (40, 900):
        H, E, k = 160, 12, 3
        say(f"NaN in the weights, gradients and rows of dropped slots and padded tokens, T={T}")
        shp = B.shape(H, 32, E, k)
        ids = draw_ids(3, T, E, k, 0.3)
        ids[T // 2:] = -1                                # the second half of the batch is padding
        idd = torch.from_numpy(ids).to(DEV)
        lost = idd < 0
        lost |= idd >= E
        w, dw = torch.softmax(rand(torch, 4, (T, k), "f32"), dim=1).contiguous(), rand(torch, 5, (T, k), "f32")
        x, add, wr = rand(torch, 1, (T, H), "f16"), rand(torch, 2, (T, H), "f16"), rand(torch, 3, (E, H), "f16")
        inv = torch.from_numpy(plan(ids, E)[1].astype(np.int32)).to(DEV)
        rows = rand(torch, 6, (T * k, H), "f16")
        ws = torch.empty(B.pw_router_backward_workspace_bytes(shp, T), dtype=torch.uint8, device=DEV)
        got = []
        for value in (0.0, nan):
            w2, dw2, x2 = w.masked_fill(lost, value), dw.masked_fill(lost, value), x.clone()
            x2[T // 2:] = value
            rows2 = rows.clone()
            rows2[int((~lost).sum()):] = value
            dx, dwr, y = torch.empty_like(x), torch.empty((E, H), device=DEV), torch.empty_like(x)
            drows, dws = torch.zeros_like(rows), torch.empty((T, k), device=DEV)
            B.pw_router_backward(shp, T, x2, wr, idd, w2, dw2, dx, dwr, ws, dx_add=add)
            B.pw_moe_unpermute(shp, T, rows2, inv, w2, y)
            B.pw_moe_unpermute_backward(shp, T, x2, rows2, inv, w2, drows, dws)
            torch.cuda.synchronize()
            got.append((dx, dwr, y, drows, dws))
        assert all(torch.equal(a, b) and bool(a.isfinite().all()) for a, b in zip(*got))


def test_broadcast_and_wide_inputs(torch):
    say("rows that are one row repeated (stride 0), and rows of a much wider matrix")
    T, H, E, k = 70, 64, 8, 2
    shp = B.shape(H, 32, E, k)
    one, wide = rand(torch, 1, (1, H), "f16"), rand(torch, 2, (T, 40 * H), "f16")[:, 8 * H:9 * H]
    ids = draw_ids(4, T, E, k, 0.0)
    g = rand(torch, 3, (1, H), "f16")[0]
    for x in (one.expand(T, H), wide):
        y, yc = (torch.empty((T, H), dtype=torch.float16, device=DEV) for _ in range(2))
        B.pw_rmsnorm(T, H, x, g, EPS, y, residual=x, residual_out=torch.empty_like(y))
        B.pw_rmsnorm(T, H, x.contiguous(), g, EPS, yc, residual=x.contiguous(), residual_out=torch.empty_like(y))
        assert torch.equal(y, yc)
        xs, _, inv, perm, _, _, _ = run_permute(torch, x, ids, E)
        assert torch.equal(xs, x.contiguous()[perm.long() // k])
        big = torch.zeros((T * k, 3 * H), dtype=torch.float16, device=DEV)
        w, dw, dw2 = rand(torch, 7, (T, k), "f32"), torch.empty((T, k), device=DEV), torch.empty((T, k), device=DEV)
        B.pw_moe_unpermute_backward(shp, T, x, xs, inv, w, big[:, H:2 * H], dw)
        plain = torch.empty_like(xs)
        B.pw_moe_unpermute_backward(shp, T, x.contiguous(), xs, inv, w, plain, dw2)
        torch.cuda.synchronize()
        assert torch.equal(big[:, H:2 * H], plain) and torch.equal(dw, dw2)
        assert bool((big[:, :H] == 0).all()) and bool((big[:, 2 * H:] == 0).all())


# ----- the router's gradient --------------------------------------------------

ROUTER_CASES = [("one", 1, 32, 1, 1, 0.0), ("decode", 4, 2048, 60, 4, 0.0), ("odd", 7, 96, 5, 3, 0.3),
                ("E256_k64", 6, 160, 256, 64, 0.1), ("qwen", 257, 2048, 60, 4, 0.05), 
                ("mixtral", 1100, 4096, 8, 2, 0.0), ("E256_k8", 1500, 288, 256, 8, 0.2),
                ("all_dropped", 33, 64, 8, 2, 1.0), ("large", 5001, 544, 33, 6, 0.1)]


@pytest.mark.parametrize("name,T,H,E,k,dropped", ROUTER_CASES, ids=[c[0] for c in ROUTER_CASES])
def test_router_backward(torch, name, T, H, E, k, dropped):
    say(f"router_backward {name} T={T} H={H} E={E} k={k}")
    ids = draw_ids(12, T, E, k, dropped)
    if name == "large":
        ids[::3, 1] = ids[::3, 0]                       # the same expert twice in a token
    shp = B.shape(H, 32, E, k)
    x, wr = rand(torch, 1, (T, H), "f16"), rand(torch, 2, (E, H), "f16", H ** -0.5)
    add = rand(torch, 3, (T, H), "f16", 0.1)
    w = torch.softmax(rand(torch, 4, (T, k), "f32"), dim=1).contiguous()
    dw = rand(torch, 5, (T, k), "f32")
    idd = torch.from_numpy(ids).to(DEV)
    ws = torch.full((B.pw_router_backward_workspace_bytes(shp, T),), 255, dtype=torch.uint8, device=DEV)
    dx, dwr = torch.full_like(x, 7.0), torch.full((E, H), 7.0, device=DEV)
    B.pw_router_backward(shp, T, x, wr, idd, w, dw, dx, dwr, ws, dx_add=add)
    alone, dwr2 = torch.full_like(x, 7.0), torch.empty_like(dwr)
    B.pw_router_backward(shp, T, x, wr, idd, w, dw, alone, dwr2, ws)
    over = add.clone()
    B.pw_router_backward(shp, T, x, wr, idd, w, dw, over, dwr2, ws, dx_add=over)
    torch.cuda.synchronize()
    assert torch.equal(dwr, dwr2) and torch.equal(over, dx)
    X, Wr, A, W, D = f64(x), f64(wr), f64(add), f64(w), f64(dw)
    kept = (ids >= 0) & (ids < E)
    dense, amag = np.zeros((T, E + 1)), np.zeros((T, E + 1))
    mean = np.sum(W * D * kept, axis=1, keepdims=True)
    dl = np.where(kept, W * (D - mean), 0.0)
    dm = np.where(kept, W * (np.abs(D) + np.sum(np.abs(W * D) * kept, axis=1, keepdims=True)), 0.0)
    for j in range(k):
        at = np.where(kept[:, j], ids[:, j], E)
        np.add.at(dense, (np.arange(T), at), dl[:, j])
        np.add.at(amag, (np.arange(T), at), dm[:, j])
    dense, amag = dense[:, :E], amag[:, :E]
    refx, refw = dense @ Wr, dense.T @ X
    if T * k * H < 100000:
        ox, ow = oo.router_backward(X, Wr, ids, W, D)
        np.testing.assert_allclose(refx, ox, rtol=0, atol=1e-11)
        np.testing.assert_allclose(refw, ow, rtol=0, atol=1e-11)
    magx, magw = amag @ np.abs(Wr), amag.T @ np.abs(X)
    for got, plus, what in [(dx, A, "dx"), (alone, 0 * A, "dx with nothing to add to")]:
        ref = refx + plus
        near(f64(got), ref, np.abs(ref) * 2.0 ** -11 + 2.0 ** -25 + (2 * k + 8) * U * (magx + np.abs(plus)), what)
    # at most 512 listed rows in turn, at most 64 sums of those; k + 8 roundings of dl
    near(f64(dwr), refw, (min(T, 512) + 64 + 2 * k + 8) * U * magw, "drouter_w")


def test_router_backward_of_no_tokens(torch):
    say("router_backward: T = 0 clears drouter_w")
    shp = B.shape(64, 32, 8, 2)
    e, i, f = (torch.empty(0, dtype=d, device=DEV) for d in (torch.float16, torch.int32, torch.float32))
    out = torch.full((8, 64), 5.0, device=DEV)
    B.pw_router_backward(shp, 0, e, torch.zeros(8, 64, dtype=torch.float16, device=DEV), i, f, f, e, out,
                         torch.empty(8192, dtype=torch.uint8, device=DEV))
    torch.cuda.synchronize()
    assert bool((out == 0).all())


# ----- together -----------------------------------------------------------------

@pytest.mark.parametrize("wl,T", [("tiny", 16), ("tiny", 256), ("tiny", 257), ("qwen_decode", 4), ("qwen_decode", 1)])
def test_forward_block(torch, wl, T):
    say(f"forward_block {wl} T={T}: equal to norm, router and layer called apart")
    check_block(torch, synth.make_layer(synth.WORKLOADS[wl].with_T(T)))


@pytest.mark.parametrize("H,T", [(32, 3), (64, 5), (96, 2), (288, 9), (1056, 4), (8192, 2), (8224, 2)])
def test_forward_block_sizes(torch, H, T):
    say(f"forward_block H={H} T={T}: narrow and long rows, one launch up to H = 8192 and two above")
    check_block(torch, synth.make_layer(synth.Workload("block", H=H, I=64, E=5, k=2, T=T, seed=77)))


def check_block(torch, L):
    dev = DeviceLayer(L, device=DEV)
    w = L.wl
    x, res0 = rand(torch, 1, (w.T, w.H), "f16"), rand(torch, 2, (w.T, w.H), "f16", 2.0)
    g = rand(torch, 3, (1, w.H), "f16")[0]
    wr = torch.from_numpy(synth.draw_router_weights(5, w.E, w.H)).to(DEV)
    stats = [(torch.zeros(w.E, dtype=torch.int32, device=DEV), torch.zeros(w.E, device=DEV)) for _ in range(2)]
    res, xn, y = res0.clone(), torch.empty_like(x), torch.empty_like(x)
    B.pw_rmsnorm(w.T, w.H, x, g, EPS, xn, residual=res, residual_out=res)
    B.pw_moe_forward_routed(dev.shape, w.T, xn, wr, dev.blocks[0], dev.q, y, *stats[0], dev.ws)
    res2, y2 = res0.clone(), torch.empty_like(x)
    B.pw_moe_forward_block(dev.shape, w.T, x, res2, g, EPS, wr, dev.blocks[0], dev.q, y2, *stats[1], dev.ws)
    x3, res3 = x.clone(), res0.clone()
    B.pw_moe_forward_block(dev.shape, w.T, x3, res3, g, EPS, wr, dev.blocks[0], dev.q, x3, None, None, dev.ws)
    torch.cuda.synchronize()
    assert torch.equal(res, res2) and torch.equal(y, y2) and torch.equal(stats[0][0], stats[1][0])
    assert torch.equal(x3, y) and torch.equal(res3, res) and dev.status() == 0
    assert float(y.float().abs().max()) > 0


def test_forward_block_in_a_graph(torch):
    say("forward_block captured and replayed: the residual stream goes on, as in eager calls")
    L = synth.make_layer(synth.WORKLOADS["tiny"])
    dev, w = DeviceLayer(L, device=DEV), L.wl
    x, res0 = rand(torch, 1, (w.T, w.H), "f16"), rand(torch, 2, (w.T, w.H), "f16")
    g = rand(torch, 3, (1, w.H), "f16")[0]
    wr = torch.from_numpy(synth.draw_router_weights(5, w.E, w.H)).to(DEV)
    res, y = res0.clone(), torch.empty_like(x)
    call = lambda r, o: B.pw_moe_forward_block(dev.shape, w.T, x, r, g, EPS, wr, dev.blocks[0], dev.q, o, None, None,
                                               dev.ws)
    call(res, y)
    torch.cuda.synchronize()
    res.copy_(res0)
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        call(res, y)
    eager, ye = res0.clone(), torch.empty_like(x)
    for n in range(4):
        gr.replay()
        torch.cuda.synchronize()
        call(eager, ye)
        torch.cuda.synchronize()
        assert torch.equal(res, eager) and torch.equal(y, ye), n


def experts(torch, L, e, rows):
    """fp64 SwiGLU of expert e with its dequantized weights."""
    gu, dn = (torch.from_numpy(orc.fp16_bits_to_f64(orc.dequant_block(L.planes[e][m], L.luts[e][m],
                                                                      int(L.q[e][m])))).to(DEV) for m in (0, 1))
    a = rows.double() @ gu.t().contiguous()
    I = L.wl.I
    return (torch.nn.functional.silu(a[:, :I]) * a[:, I:]) @ dn.t().contiguous()


def test_sorted_products_equal_the_layer(torch):
    """Norm, router, sort, each expert's products on its own rows, back with the
    weights: the fused layer's output on the same routing."""
    say("permute -> own expert products -> unpermute against pw_moe_forward")
    L = synth.make_layer(synth.WORKLOADS["tiny"])
    w = L.wl
    dev = DeviceLayer(L, device=DEV)
    x, res = rand(torch, 1, (w.T, w.H), "f16"), rand(torch, 2, (w.T, w.H), "f16")
    xn, y = torch.empty_like(x), torch.empty_like(x)
    B.pw_rmsnorm(w.T, w.H, x, torch.ones(w.H, dtype=torch.float16, device=DEV), EPS, xn, residual=res, residual_out=res)
    wr = torch.from_numpy(synth.draw_router_weights(5, w.E, w.H)).to(DEV)
    ids, wt = torch.empty((w.T, w.k), dtype=torch.int32, device=DEV), torch.empty((w.T, w.k), device=DEV)
    B.pw_router_topk(dev.shape, w.T, xn, wr, ids, wt, None, None, dev.ws)
    B.pw_moe_forward(dev.shape, w.T, xn, ids, wt, dev.blocks[0], dev.q, y, dev.ws)
    xs, off, inv, _, _, status, _ = run_permute(torch, xn, ids.cpu().numpy(), w.E)
    rows = torch.zeros((w.T * w.k, w.H), dtype=torch.float32, device=DEV)
    ends = off.tolist()
    for e in range(w.E):
        if ends[e + 1] > ends[e]:
            rows[ends[e]:ends[e + 1]] = experts(torch, L, e, xs[ends[e]:ends[e + 1]]).float()
    mine = torch.empty((w.T, w.H), device=DEV)
    B.pw_moe_unpermute(dev.shape, w.T, rows, inv, wt, mine)
    torch.cuda.synchronize()
    assert status == 0
    rel = float((mine.double() - y.double()).norm() / y.double().norm())
    say(f"  rel_l2 {rel:.2e}")
    assert rel <= 1e-3                                  # the layer's own tolerance against the 64-bit oracle


def test_gradients_through_the_chain(torch):
    """residual + x -> norm -> router weights -> sort -> a linear map per expert ->
    back with the weights, and the gradient of all of it, in fp32 and fp16 where
    the library has only that; against torch's automatic gradient in 64 bits."""
    T, H, E, k = 37, 128, 6, 2
    say(f"gradient of the whole chain, T={T} H={H} E={E} k={k}")
    shp = B.shape(H, 32, E, k)
    x, res, g = rand(torch, 1, (T, H), "f16"), rand(torch, 2, (T, H), "f16"), rand(torch, 3, (1, H), "f16")[0]
    wr, M = rand(torch, 4, (E, H), "f16", H ** -0.5), rand(torch, 5, (E, H, H), "f16", H ** -0.5)
    dy, dout = rand(torch, 6, (T, H), "f16"), rand(torch, 7, (T, H), "f16")
    new = lambda *s, d=torch.float16: torch.empty(s, dtype=d, device=DEV)
    r, xn, xs, off, inv = new(T, H), new(T, H), new(T * k, H), new(E + 1, d=torch.int32), new(T * k, d=torch.int32)
    ids, w = new(T, k, d=torch.int32), new(T, k, d=torch.float32)
    ws = torch.empty(max(B.pw_workspace_bytes(shp, T), B.pw_router_backward_workspace_bytes(shp, T),
                         B.pw_moe_permute_workspace_bytes(shp, T), B.pw_rmsnorm_backward_workspace_bytes(T, H)),
                     dtype=torch.uint8, device=DEV)
    B.pw_rmsnorm(T, H, x, g, EPS, xn, residual=res, residual_out=r)
    B.pw_router_topk(shp, T, xn, wr, ids, w, workspace=ws)
    B.pw_moe_permute(shp, T, xn, ids, xs, off, inv, None, ws)
    ends = off.tolist()
    rows, y = new(T * k, H), new(T, H)
    for e in range(E):
        rows[ends[e]:ends[e + 1]] = (xs[ends[e]:ends[e + 1]].double() @ M[e].double()).half()
    B.pw_moe_unpermute(shp, T, rows, inv, w, y)
    drows, dw, dxs, dxn, dr = new(T * k, H), new(T, k, d=torch.float32), new(T * k, H), new(T, H), new(T, H)
    dwr, dg = new(E, H, d=torch.float32), new(H, d=torch.float32)
    B.pw_moe_unpermute_backward(shp, T, dy, rows, inv, w, drows, dw)
    for e in range(E):
        dxs[ends[e]:ends[e + 1]] = (drows[ends[e]:ends[e + 1]].double() @ M[e].double().t().contiguous()).half()
    B.pw_moe_permute_backward(shp, T, dxs, inv, dxn)
    B.pw_router_backward(shp, T, xn, wr, ids, w, dw, dxn, dwr, ws, dx_add=dxn)
    B.pw_rmsnorm_backward(T, H, dxn, r, g, EPS, dr, dg, ws, dresidual=dout)
    torch.cuda.synchronize()

    leaf = lambda t: t.detach().double().cpu().requires_grad_()
    X, G, W = leaf(x), leaf(g), leaf(wr)
    R = X + res.double().cpu()
    N = R / torch.sqrt((R * R).mean(1, keepdim=True) + EPS) * G
    sel = ids.long().cpu()
    p = torch.softmax(torch.gather(N @ W.t(), 1, sel), dim=1)
    out = sum(p[:, j:j + 1] * torch.stack([N[t] @ M[sel[t, j]].double().cpu() for t in range(T)]) for j in range(k))
    ((out * dy.double().cpu()).sum() + (R * dout.double().cpu()).sum()).backward()
    # five fp16 roundings (2^-11) lie between a leaf and its gradient, each at most once per addend
    for got, ref, what in [(y, out.detach(), "y"), (dr, X.grad, "dx"), (dg, G.grad, "dweight"),
                           (dwr, W.grad, "drouter_w")]:
        rel = float((got.double().cpu() - ref).norm() / ref.norm())
        say(f"  {what}: rel_l2 {rel:.2e}")
        assert rel <= 5 * 2.0 ** -11, what


# ----- streams, graphs, refusals -------------------------------------------------

def all_ops(torch, seed, T=1500, H=256, E=8, k=4):
    """Buffers of one use of every operator, and the calls on them."""
    shp = B.shape(H, 32, E, k)
    S = T * k
    new = lambda *s, d=torch.float16: torch.zeros(s, dtype=d, device=DEV)
    b = {"x": rand(torch, seed, (T, H), "f16"), "res": rand(torch, seed + 1, (T, H), "f16"),
         "g": rand(torch, seed + 2, (1, H), "f16")[0], "wr": rand(torch, seed + 3, (E, H), "f16", H ** -0.5),
         "ids": torch.from_numpy(draw_ids(seed, T, E, k, 0.1)).to(DEV), "w": rand(torch, seed + 4, (T, k), "f32"),
         "r": new(T, H), "y": new(T, H), "codes": new(T, H, d=torch.uint8).view(torch.float8_e4m3fn),
         "scale": new(T, 2, d=torch.float32), "xs": new(S, H),
         "xs8": new(S, H, d=torch.uint8).view(torch.float8_e4m3fn),
         "sc": new(S, 2, d=torch.float32), "off": new(E + 1, d=torch.int32), "inv": new(S, d=torch.int32),
         "back": new(T, H), "drows": new(S, H), "dw": new(T, k, d=torch.float32), "dx": new(T, H), "dx2": new(T, H),
         "dwr": new(E, H, d=torch.float32), "dr": new(T, H), "dg": new(H, d=torch.float32)}
    ws = {"p": torch.empty(B.pw_moe_permute_workspace_bytes(shp, T), dtype=torch.uint8, device=DEV),
          "r": torch.empty(B.pw_router_backward_workspace_bytes(shp, T), dtype=torch.uint8, device=DEV),
          "n": torch.empty(B.pw_rmsnorm_backward_workspace_bytes(T, H), dtype=torch.uint8, device=DEV)}

    def calls(stream=None):
        B.pw_rmsnorm(T, H, b["x"], b["g"], EPS, b["y"], residual=b["res"], residual_out=b["r"], stream=stream)
        B.pw_rmsnorm(T, H, b["x"], b["g"], EPS, b["codes"], residual=b["res"], scale=b["scale"], group=128,
                     stream=stream)
        B.pw_moe_permute(shp, T, b["codes"], b["ids"], b["xs8"], b["off"], b["inv"], None, ws["p"], x_scale=b["scale"],
                         xs_scale=b["sc"], stream=stream)
        B.pw_moe_permute(shp, T, b["y"], b["ids"], b["xs"], b["off"], b["inv"], None, ws["p"], stream=stream)
        B.pw_moe_unpermute(shp, T, b["xs"], b["inv"], b["w"], b["back"], stream=stream)
        B.pw_moe_unpermute_backward(shp, T, b["back"], b["xs"], b["inv"], b["w"], b["drows"], b["dw"], stream=stream)
        B.pw_moe_permute_backward(shp, T, b["drows"], b["inv"], b["dx"], stream=stream)
        B.pw_router_backward(shp, T, b["y"], b["wr"], b["ids"], b["w"], b["dw"], b["dx2"], b["dwr"], ws["r"],
                             dx_add=b["dx"], stream=stream)
        B.pw_rmsnorm_backward(T, H, b["dx2"], b["r"], b["g"], EPS, b["dr"], b["dg"], ws["n"], dresidual=b["dx"],
                              stream=stream)

    outs = ["r", "y", "codes", "scale", "xs8", "sc", "xs", "off", "inv", "back", "drows", "dw", "dx", "dx2",
            "dwr", "dr", "dg"]
    return b, calls, outs


def snapshot(torch, b, outs):
    torch.cuda.synchronize()
    return [b[o].contiguous().view(torch.uint8).clone() for o in outs]


def test_two_streams_at_once(torch):
    say("every operator on two streams at once, each with its own workspaces, equal to calls alone")
    sets = [all_ops(torch, s) for s in (100, 200)]
    want = []
    for b, calls, outs in sets:
        calls()
        want.append(snapshot(torch, b, outs))
    for b, _, outs in sets:
        for o in outs:
            b[o].view(torch.uint8).zero_()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    for _ in range(3):
        for (b, calls, outs), st in zip(sets, streams):
            calls(st)
    for (b, _, outs), w in zip(sets, want):
        assert all(torch.equal(a, c) for a, c in zip(snapshot(torch, b, outs), w))


def test_captured_graphs(torch):
    say("two captured graphs with their own workspaces, replayed in turn with changed inputs and eager calls between")
    sets = [all_ops(torch, s) for s in (300, 400)]
    graphs = []
    for b, calls, outs in sets:
        calls()
        torch.cuda.synchronize()
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            calls()
        graphs.append(gr)
    eager = all_ops(torch, 500)
    for n in range(4):
        for b, _, _ in sets:
            b["x"].mul_(-0.5 if n % 2 else 2.0)
            b["ids"].copy_(b["ids"].roll(n + 1, dims=0))
        torch.cuda.synchronize()
        for gr in graphs:
            gr.replay()
        eager[1]()
        got = [snapshot(torch, b, outs) for b, _, outs in sets]
        for (b, calls, outs), g in zip(sets, got):
            # rows without a slot keep what an earlier replay left there; everything else is written again
            calls()
            again = snapshot(torch, b, outs)
            for o, a, c in zip(outs, g, again):
                assert torch.equal(a, c), (n, o)


def test_binding_refusals(torch):
    say("binding: wrong types, shapes, strides and streams are refused before any launch")
    T, H, E, k = 4, 64, 8, 2
    shp = B.shape(H, 32, E, k)
    h = lambda *s: torch.zeros(s, dtype=torch.float16, device=DEV)
    f = lambda *s: torch.zeros(s, device=DEV)
    i = lambda *s: torch.zeros(s, dtype=torch.int32, device=DEV)
    ws = torch.zeros(1 << 20, dtype=torch.uint8, device=DEV)
    x, g, xs = h(T, H), h(H), h(T * k, H)
    bad = [
        lambda: B.pw_rmsnorm(T, H, None, g, EPS, x),
        lambda: B.pw_rmsnorm(T, H, x, None, EPS, x),
        lambda: B.pw_rmsnorm(T, H, x, g, EPS, None),
        lambda: B.pw_moe_unpermute(shp, T, xs, None, None, x),
        lambda: B.pw_rmsnorm(T, H, x, f(H), EPS, x),                              # weight of another type
        lambda: B.pw_rmsnorm(T, H, x, g, EPS, f(T, H)),                           # output of another type
        lambda: B.pw_rmsnorm(T, H, h(H, T).t(), g, EPS, x),                       # columns apart
        lambda: B.pw_rmsnorm(T + 1, H, x, g, EPS, x),                             # too few rows
        lambda: B.pw_rmsnorm(T, H, x[:, :32], g, EPS, x),                         # too few columns
        lambda: B.pw_rmsnorm(T, H, x, g, EPS, x, residual=f(T, H)),
        lambda: B.pw_rmsnorm(T, H, x, g, EPS, ws[:T * H].view(torch.float8_e4m3fn).view(T, H), scale=f(T - 1, 1)),
        lambda: B.pw_rmsnorm(T, H, x, g, EPS, x.double()),
        lambda: B.pw_rmsnorm(T, H, x, g, EPS, h(1, H).expand(T, H)),              # rows that overlap
        lambda: B.pw_rmsnorm(T, H, x, g.cpu(), EPS, x),
        lambda: B.pw_rmsnorm_backward(T, H, x, x, g, EPS, h(T, H), f(H)),         # no workspace
        lambda: B.pw_rmsnorm_backward(T, H, x, x, g, EPS, h(T, H), f(H // 2), ws),
        lambda: B.pw_moe_permute(shp, T, x, i(T, k).long(), xs, i(E + 1), i(T * k), None, ws),
        lambda: B.pw_moe_permute(shp, T, x, i(T, k), h(T, H), i(E + 1), i(T * k), None, ws),
        lambda: B.pw_moe_permute(shp, T, x, i(T, k), xs, i(E), i(T * k), None, ws),
        lambda: B.pw_moe_permute(shp, T, x, i(T, 2 * k)[:, ::2], xs, i(E + 1), i(T * k), None, ws),
        lambda: B.pw_moe_permute(shp, T, x, i(T, k), xs, i(E + 1), i(T * k), None, ws, x_scale=f(T, 2)),
        lambda: B.pw_moe_unpermute(shp, T, xs, i(T * k), h(T, k), x),
        lambda: B.pw_moe_unpermute_backward(shp, T, x, None, i(T * k), f(T, k), xs, f(T, k)),
        lambda: B.pw_router_backward(shp, T, f(T, H), h(E, H), i(T, k), f(T, k), f(T, k), x, f(E, H), ws),
        lambda: B.pw_router_backward(shp, T, h(T, 2 * H)[:, :H], h(E, H), i(T, k), f(T, k), f(T, k), x, f(E, H), ws),
    ]
    for n, call in enumerate(bad):
        with pytest.raises(B.PwError) as e:
            call()
        assert e.value.status == B.PW_ERR_INVALID_ARG, n
    with pytest.raises(B.PwError) as e:
        B.pw_rmsnorm(T, H, h(T * H + 1)[1:].view(T, H), g, EPS, x)
    assert e.value.status == B.PW_ERR_ALIGNMENT
    with pytest.raises(B.PwError) as e:
        B.pw_rmsnorm_backward(T, H, x, x, g, EPS, h(T, H), f(H), ws[:256])
    assert e.value.status == B.PW_ERR_WORKSPACE


# ----- the 8-bit codes ----------------------------------------------------------

@pytest.mark.parametrize("name", DTYPES)
@pytest.mark.parametrize("T,H,group", [(2000, 40, 0), (3000, 520, 128), (1000, 4096, 128), (500, 4096, 0),
                                       (100, 8200, 128), (60, 16392, 0)])
def test_rmsnorm_e4m3_codes_are_nearest(torch, T, H, group, name):
    """A code is the e4m3 number nearest to the fp32 quotient y / scale, to the bit: fp32 rows store the y that is
    divided as it is, and 16-bit rows are widened without a change."""
    say(f"rmsnorm e4m3 codes {name} T={T} H={H} group={group}")
    x, res, g = rand(torch, 1, (T, H), name), rand(torch, 2, (T, H), name, 4.0), rand(torch, 3, (1, H), name)[0]
    wide = torch.empty((T, H), device=DEV)
    B.pw_rmsnorm(T, H, x.float(), g.float(), EPS, wide, residual=res.float(), residual_out=torch.empty_like(wide))
    y = torch.empty((T, H), dtype=torch.float8_e4m3fn, device=DEV)
    scale = torch.empty((T, -(-H // 128) if group else 1), device=DEV)
    B.pw_rmsnorm(T, H, x, g, EPS, y, residual=res, scale=scale, group=group)
    torch.cuda.synchronize()
    pieces = wide.cpu().split(group or H, dim=1)
    want = torch.stack([p.abs().amax(dim=1) / 448.0 for p in pieces], dim=1)
    assert torch.equal(scale.cpu(), want)
    codes = torch.cat([(p / want[:, i:i + 1]).clamp(-448, 448).to(torch.float8_e4m3fn)
                       for i, p in enumerate(pieces)], dim=1)
    off = int((y.cpu().float() != codes.float()).sum())
    say(f"  {off} of {T * H} codes differ")
    assert off == 0


# ----- the router's gradient by the form of its tiles ----------------------------

def router_chain(T, H, E, k):
    """Most fp32 additions in turn behind one element of drouter_w: a wave's part of a list of up to 2048 slots (its
    block's four waves share the rows of 512 columns up to 8192 slots; above, 2 or 4 of them take other columns where H
    is over 512 or 1024), the lists of a stretch, the parts, the stretches.  Stretches: at least 1024 slots and 4 E
    tokens, as many as make 4096 blocks; a list's length is bounded by the slots too."""
    waves = 1 if T * k <= 8192 or H <= 512 else 2 if H <= 1024 else 4
    tiles = E * -(-H // (512 * waves))
    least = max(1024, 4 * E * k)
    stretch = max(least, -(-T * k // (-(-4096 // tiles))) + 255)
    parts = 4 // waves * (1 if H >= 512 else 64)
    return min(T * k, 512 * waves) + -(-stretch // 2048) + parts + -(-T * k // least) + 2 * k + 8


def draw_skewed(seed, T, E, k, hot, share):
    """Distinct experts a token, with expert `hot` in the first slot of `share` of the tokens."""
    ids = draw_ids(seed, T, E, k, 0.0)
    rng = np.random.default_rng(seed)
    at = (rng.random(T) < share) & ~(ids == hot).any(axis=1)
    ids[at, 0] = hot
    return ids


# below and above 8192 slots; H over 1024 with whole tiles of 2048 columns, with a last tile of 32, and with waves past
# H; full lists (every slot the same expert, twice a token); nearly all tokens at one expert; several stretches
ROUTER_TILES = [("below", 4096, 1056, 8, 2), ("above", 4097, 4096, 8, 2), ("waves_past_H", 2100, 1056, 60, 4),
                ("last_tile_32", 2100, 2080, 60, 4), ("full_lists", 5000, 2080, 2, 2), ("skewed", 4099, 2048, 60, 4),
                ("E256", 3000, 1056, 256, 8), ("two_columns", 4200, 1024, 9, 2), ("E1", 8200, 1056, 1, 1)]


@pytest.mark.parametrize("name,T,H,E,k", ROUTER_TILES, ids=[c[0] for c in ROUTER_TILES])
def test_router_backward_tiles(torch, name, T, H, E, k):
    chain = router_chain(T, H, E, k)
    say(f"router_backward tiles {name} T={T} H={H} E={E} k={k}, chain {chain}")
    ids = draw_skewed(13, T, E, k, 7, 0.95) if name == "skewed" else draw_ids(13, T, E, k, 0.05)
    if name == "full_lists":
        ids[:] = 0
    shp = B.shape(H, 32, E, k)
    x, wr = rand(torch, 1, (T, H), "f16"), rand(torch, 2, (E, H), "f16", H ** -0.5)
    add = rand(torch, 3, (T, H), "f16", 0.1)
    # one expert for all of a token's slots: weights that do not sum to one, or the gradients would cancel
    part = 0.5 if E == 1 or name == "full_lists" else 1.0
    w = (torch.softmax(rand(torch, 4, (T, k), "f32"), dim=1) * part).contiguous()
    dw = rand(torch, 5, (T, k), "f32")
    idd = torch.from_numpy(ids).to(DEV)
    ws = torch.full((B.pw_router_backward_workspace_bytes(shp, T),), 255, dtype=torch.uint8, device=DEV)
    dx, dwr, again = torch.full_like(x, 7.0), torch.full((E, H), 7.0, device=DEV), torch.empty((E, H), device=DEV)
    B.pw_router_backward(shp, T, x, wr, idd, w, dw, dx, dwr, ws, dx_add=add)
    B.pw_router_backward(shp, T, x, wr, idd, w, dw, torch.empty_like(x), again, ws)
    torch.cuda.synchronize()
    assert torch.equal(dwr, again)
    X, Wr, A, W, D = f64(x), f64(wr), f64(add), f64(w), f64(dw)
    kept = (ids >= 0) & (ids < E)
    dl = np.where(kept, W * (D - np.sum(W * D * kept, axis=1, keepdims=True)), 0.0)
    dm = np.where(kept, W * (np.abs(D) + np.sum(np.abs(W * D) * kept, axis=1, keepdims=True)), 0.0)
    dense, mag = np.zeros((T, E + 1)), np.zeros((T, E + 1))
    for j in range(k):
        np.add.at(dense, (np.arange(T), np.where(kept[:, j], ids[:, j], E)), dl[:, j])
        np.add.at(mag, (np.arange(T), np.where(kept[:, j], ids[:, j], E)), dm[:, j])
    dense, mag = dense[:, :E], mag[:, :E]
    ref = dense @ Wr + A
    near(f64(dx), ref, np.abs(ref) * 2.0 ** -11 + 2.0 ** -25 + (2 * k + 8) * U * (mag @ np.abs(Wr) + np.abs(A)), "dx")
    near(f64(dwr), dense.T @ X, chain * U * (mag.T @ np.abs(X)), "drouter_w")

    # whole numbers: dl = w (dw - sum w dw) with w = part / k and dw a multiple of (k / part)^2 is one too, at most
    # 4 k / part, and every partial sum stays below 2^24, so fp32 adds without a rounding and no row may be missing
    whole = lambda seed, shape, most: torch.randint(-most, most + 1, shape,
                                                    generator=torch.Generator().manual_seed(seed))
    x, w = whole(1, (T, H), 3).half().to(DEV), torch.full((T, k), part / k, device=DEV)
    dw = (whole(2, (T, k), 2) * int(k / part) ** 2).float().to(DEV)
    B.pw_router_backward(shp, T, x, wr, idd, w, dw, dx, dwr, ws)
    torch.cuda.synchronize()
    D = f64(dw) * kept
    dl = np.where(kept, (D - np.sum(D, axis=1, keepdims=True) * part / k) * part / k, 0.0)
    dense = np.zeros((T, E + 1))
    for j in range(k):
        np.add.at(dense, (np.arange(T), np.where(kept[:, j], ids[:, j], E)), dl[:, j])
    assert np.max(np.sum(np.abs(dl), axis=1)) * T * 3 < 2 ** 24 and dl.any()
    assert np.array_equal(f64(dwr), dense[:, :E].T @ f64(x))


@pytest.mark.parametrize("T,H", [(4_200_003, 512), (67_200_003, 32)])
def test_router_backward_of_more_tokens_than_a_grid_takes(torch, T, H):
    """The launch's dx blocks end at 2^20, each four tokens (H = 512) or 64 (H = 32); they then walk the rest.  Whole
    numbers: w = 1/2 and dw a multiple of 4 give a whole dl of at most 2, and the partial sums, walks of at most 2^27
    steps of up to 6 in both directions, stay far below 2^24 (the last line checks), so every sum is exact."""
    E, k = 4, 2
    say(f"router_backward T={T} H={H}: {T * H * 2 / 2 ** 30:.1f} GiB a matrix")
    shp = B.shape(H, 32, E, k)
    g = torch.Generator(device=DEV).manual_seed(1)
    x = torch.empty((T, H), dtype=torch.float16, device=DEV)
    step = (1 << 27) // H
    for s in range(0, T, step):
        x[s:s + step] = torch.randint(-3, 4, x[s:s + step].shape, generator=g, device=DEV, dtype=torch.int8).half()
    wr = torch.randint(-8, 9, (E, H), generator=g, device=DEV).half()
    first = torch.randint(0, E, (T, 1), generator=g, device=DEV, dtype=torch.int32)
    ids = torch.cat([first, (first + 1) % E], dim=1).contiguous()
    w = torch.full((T, k), 0.5, device=DEV)
    dw = 4.0 * torch.randint(-1, 2, (T, k), generator=g, device=DEV).float()
    dx, dwr = torch.full_like(x, 7.0), torch.empty((E, H), device=DEV)
    ws = torch.empty(B.pw_router_backward_workspace_bytes(shp, T), dtype=torch.uint8, device=DEV)
    B.pw_router_backward(shp, T, x, wr, ids, w, dw, dx, dwr, ws)
    torch.cuda.synchronize()
    ref, reach = torch.zeros((E, H), dtype=torch.float64, device=DEV), 0.0
    for s in range(0, T, step):
        D = dw[s:s + step].double()
        dl = 0.5 * (D - 0.5 * D.sum(1, keepdim=True))
        dense = torch.zeros((D.shape[0], E), dtype=torch.float64, device=DEV)
        dense.scatter_add_(1, ids[s:s + step].long(), dl)
        assert torch.equal(dx[s:s + step].double(), dense @ wr.double()), s
        ref += dense.t() @ x[s:s + step].double()
        reach = max(reach, float(ref.abs().max()))
    assert torch.equal(dwr.double(), ref)
    say(f"  largest partial sum seen {reach:.0f}")
    assert reach < 2 ** 22


# ----- loops that only the largest calls turn twice --------------------------------

@pytest.mark.parametrize("T,H,out", [(2_097_160, 520, "same"), (2_097_160, 520, "e4m3"), (1_048_581, 1032, "same"),
                                     (1_048_581, 1032, "e4m3")])
def test_rmsnorm_walks_long_rows(torch, T, H, out):
    """More than 2^20 blocks of rows that take several waves, two (H = 520, two rows a block) or four."""
    say(f"rmsnorm {out} T={T} H={H}")
    g = torch.Generator(device=DEV).manual_seed(1)
    x = torch.empty((T, H), dtype=torch.float16, device=DEV).normal_(generator=g)
    x *= torch.rand((T, 1), generator=g, device=DEV).half() + 0.25       # rows of different size
    w = torch.randn(H, generator=g, device=DEV).half()
    y = torch.empty((T, H), dtype=torch.float8_e4m3fn if out == "e4m3" else torch.float16, device=DEV)
    scale = torch.empty((T, 1), device=DEV) if out == "e4m3" else None
    B.pw_rmsnorm(T, H, x, w, EPS, y, scale=scale)
    torch.cuda.synchronize()
    for s in range(0, T, 1 << 17):
        X = x[s:s + (1 << 17)].double()
        ref = X / (X.square().mean(1, keepdim=True) + EPS).sqrt() * w.double()
        got = y[s:s + (1 << 17)].float().double()
        if out == "same":
            ok = (got - ref).abs() <= ref.abs() * (2.0 ** -11 + ROW * U) + 2.0 ** -25
        else:
            sc = scale[s:s + (1 << 17)].double()
            want = ref.abs().amax(1, keepdim=True) / 448
            assert bool(((sc - want).abs() <= want * (ROW + 2) * U).all()), s
            ok = (got * sc - ref).abs() <= torch.maximum(ref.abs() * 2.0 ** -4, sc * 2.0 ** -10) + \
                (ref.abs() + sc) * 2 * ROW * U
        assert bool(ok.all()), s


@pytest.mark.parametrize("T,H,k,dt", [(5, 8192, 3, "f32"), (300, 4128, 4, "f16"), (1100, 2080, 5, "f16")])
def test_permute_of_few_long_rows(torch, T, H, k, dt):
    """One launch, rows longer than its threads take at a time: 16 KB (up to 256 tokens), 8 KB (1024), 4 KB."""
    say(f"permute {dt} T={T} H={H} k={k}: {H * (4 if dt == 'f32' else 2)} bytes a row")
    E = 9
    ids = draw_ids(6, T, E, k, 0.1)
    offsets, inv, perm = plan(ids, E)
    x = rand(torch, 5, (T, H), dt)
    xs, off, iv, _, _, _, raw = run_permute(torch, x, ids, E)
    n = len(perm)
    assert np.array_equal(off.cpu().numpy(), offsets) and np.array_equal(iv.cpu().numpy(), inv)
    assert torch.equal(xs[:n], x[torch.from_numpy(perm // k).to(DEV)]) and bool((raw[n:] == 3).all())


# ----- the norm's range -----------------------------------------------------------

@pytest.mark.parametrize("eps", [0.0, 2.0 ** -99, 1e-5, 1e30])
@pytest.mark.parametrize("name", ["f32", "bf16"])
@pytest.mark.parametrize("H", [40, 128, 520, 4096, 16392, 32768])
def test_rmsnorm_range(torch, H, name, eps):
    """Rows at both ends of the stated range: every value +-2^56, and a mean square of 2^-100 (any, down to subnormal
    values, where eps is at least that); a lone 2^56 among zeros and among values 2^-100 of it."""
    say(f"rmsnorm and its gradient {name} H={H} eps={eps}: the ends of the range")
    g64 = torch.Generator().manual_seed(1)
    signs = (torch.randint(0, 2, (8, H), generator=g64) * 2 - 1).double()
    part = 0.25 + 0.75 * torch.rand((8, H), generator=g64, dtype=torch.float64)
    power = torch.tensor([56, 56, 56, 30, 0, -49, -50, -50 if eps == 0 else -126], dtype=torch.float64)
    a = signs * part * torch.exp2(power)[:, None]
    a[0] = signs[0] * 2.0 ** 56
    a[1, 1:], a[1, 0] = 0.0, 2.0 ** 56
    a[2, 1:] *= 2.0 ** -100
    a[6] = signs[6] * 2.0 ** -50                                  # a mean square of 2^-100 exactly
    if eps == 0:
        a[7] = signs[7] * 2.0 ** -49
    x = a.to(dtype_of(torch, name)).to(DEV)
    g = rand(torch, 3, (1, H), name)[0]
    rel, ab = half_step(torch, name)
    y, codes = torch.empty_like(x), torch.empty((8, H), dtype=torch.float8_e4m3fn, device=DEV)
    scale = torch.empty((8, 1), device=DEV)
    B.pw_rmsnorm(8, H, x, g, eps, y)
    B.pw_rmsnorm(8, H, x, g, eps, codes, scale=scale)
    dy = rand(torch, 5, (8, H), name)
    dx, dg = torch.empty_like(x), torch.empty(H, device=DEV)
    ws = torch.empty(B.pw_rmsnorm_backward_workspace_bytes(8, H), dtype=torch.uint8, device=DEV)
    B.pw_rmsnorm_backward(8, H, dy, x, g, eps, dx, dg, ws)
    torch.cuda.synchronize()
    X, G, D = f64(x), f64(g), f64(dy)
    ref = oo.rmsnorm(X, G, eps)[1]
    # r / rms below fp32's normal numbers has half a subnormal step of its own, which the weight multiplies
    near(f64(y), ref, np.abs(ref) * (rel + ROW * U) + ab + 2.0 ** -149 * (1 + np.abs(G)), "y")
    rs = oo.e4m3_scales(ref, 0)
    near(f64(scale), rs, rs * (ROW + 2) * U, "scale")
    wide = np.repeat(f64(scale), H, axis=1)
    code = np.maximum(np.abs(ref) * 2.0 ** -4, wide * 2.0 ** -10)
    near(f64(codes) * wide, ref, code + (np.abs(ref) + wide) * 2 * ROW * U, "code * scale")
    s = 1 / np.sqrt(np.mean(X * X, axis=1, keepdims=True) + eps)
    mag = np.abs(s * G * D) + np.abs(X * s) * s * s * np.sum(np.abs(G * D * X), axis=1, keepdims=True) / H
    ref, dgr = oo.rmsnorm_backward(D, X, G, eps)
    near(f64(dx), ref, np.abs(ref) * rel + ab + 2 * ROW * U * mag + 2.0 ** -148, "dx")
    near(f64(dg), dgr, (1 + 32 + 8 + 6 + ROW) * U * np.sum(np.abs(D * X * s), axis=0) + 2.0 ** -145, "dweight")


def test_rmsnorm_past_its_range(torch):
    """Finite values whose squares' sum is past fp32 give zeros, as stated, and no other row is touched."""
    say("rmsnorm: rows past the range give zeros")
    for H in (40, 520, 4096):
        x = rand(torch, 1, (3, H), "bf16")
        one = x[0:1].clone()
        x[1, 0] = 2.0 ** 70
        y, alone, g = torch.empty_like(x), torch.empty_like(one), rand(torch, 3, (1, H), "bf16")[0]
        B.pw_rmsnorm(3, H, x, g, EPS, y)
        B.pw_rmsnorm(1, H, one, g, EPS, alone)
        torch.cuda.synchronize()
        assert bool((y[1] == 0).all()) and torch.equal(y[0:1], alone) and bool((y[2] != 0).any())


# ----- the fused call's routing statistics ------------------------------------------

@pytest.mark.parametrize("wl,T", [("tiny", 16), ("tiny", 256), ("tiny", 257), ("qwen_decode", 4)])
def test_forward_block_statistics(torch, wl, T):
    say(f"forward_block {wl} T={T}: counts and masses of two calls in a row, against the router's own ids and weights")
    L = synth.make_layer(synth.WORKLOADS[wl].with_T(T))
    dev, w = DeviceLayer(L, device=DEV), L.wl
    x, res = rand(torch, 1, (T, w.H), "f16"), rand(torch, 2, (T, w.H), "f16", 2.0)
    g = rand(torch, 3, (1, w.H), "f16")[0]
    wr = torch.from_numpy(synth.draw_router_weights(5, w.E, w.H)).to(DEV)
    count, mass = torch.zeros(w.E, dtype=torch.int32, device=DEV), torch.zeros(w.E, device=DEV)
    counted, weighed = np.zeros(w.E, np.int64), np.zeros(w.E)
    y, xn, ref = torch.empty_like(x), torch.empty_like(x), res.clone()
    ids, wt = torch.empty((T, w.k), dtype=torch.int32, device=DEV), torch.empty((T, w.k), device=DEV)
    for _ in range(2):
        B.pw_rmsnorm(T, w.H, x, g, EPS, xn, residual=ref, residual_out=ref)
        B.pw_router_topk(dev.shape, T, xn, wr, ids, wt, None, None, dev.ws)
        torch.cuda.synchronize()
        np.add.at(counted, ids.cpu().numpy().reshape(-1), 1)
        np.add.at(weighed, ids.cpu().numpy().reshape(-1), f64(wt).reshape(-1))
        B.pw_moe_forward_block(dev.shape, T, x, res, g, EPS, wr, dev.blocks[0], dev.q, y, count, mass, dev.ws)
        torch.cuda.synchronize()
    assert torch.equal(res, ref) and np.array_equal(count.cpu().numpy(), counted)
    near(f64(mass), weighed, counted * U * weighed, "mass")       # an fp32 sum of that many weights, in any order


def test_router_gradient_of_slots_masked_after_the_router(torch):
    """An expert's capacity: slots lose their expert after the router, the others keep their weights.  The sort and the
    way back take the masked ids, the router's gradient the router's own, with the dw that the way back writes."""
    T, H, E, k = 50, 96, 6, 3
    say(f"router_backward after masking, T={T} H={H} E={E} k={k}")
    shp = B.shape(H, 32, E, k)
    x, wr = rand(torch, 1, (T, H), "f16"), rand(torch, 2, (E, H), "f16", H ** -0.5)
    dy, rows = rand(torch, 3, (T, H), "f32"), rand(torch, 4, (T * k, H), "f32")
    ids, w = torch.empty((T, k), dtype=torch.int32, device=DEV), torch.empty((T, k), device=DEV)
    ws = torch.empty(max(B.pw_workspace_bytes(shp, T), B.pw_router_backward_workspace_bytes(shp, T)),
                     dtype=torch.uint8, device=DEV)
    B.pw_router_topk(shp, T, x, wr, ids, w, workspace=ws)
    kept = np.random.default_rng(1).random((T, k)) < 0.7
    masked = np.where(kept, ids.cpu().numpy(), -1).astype(np.int32)
    _, inv, perm = plan(masked, E)
    iv = torch.from_numpy(inv.astype(np.int32)).to(DEV)
    drows, dw = torch.zeros_like(rows), torch.empty((T, k), device=DEV)
    B.pw_moe_unpermute_backward(shp, T, dy, rows, iv, w, drows, dw)
    dx, dwr = torch.empty_like(x), torch.empty((E, H), device=DEV)
    B.pw_router_backward(shp, T, x, wr, ids, w, dw, dx, dwr, ws)
    torch.cuda.synchronize()
    leaf = lambda t: t.detach().double().cpu().requires_grad_()
    X, W = leaf(x), leaf(wr)
    p = torch.softmax(torch.gather(X @ W.t(), 1, ids.long().cpu()), dim=1)
    mine = torch.from_numpy(f64(rows)[np.where(inv >= 0, inv, 0)] * (inv >= 0)[:, None]).reshape(T, k, H)
    ((p[:, :, None] * mine).sum(1) * dy.double().cpu()).sum().backward()
    # w carries the router's fp32 logits (H + 8 roundings of sums of |x wr|, times the softmax's slope of at most one)
    D = np.abs(f64(dy))[:, None, :] * np.abs(mine.numpy())
    big = np.max(np.sum(D, axis=2))
    logits = np.max(np.abs(f64(x)) @ np.abs(f64(wr)).T)
    slack = 4 * k * big * ((H + 8) * logits + 16) * U
    ref = X.grad.numpy()
    near(f64(dx), ref, np.abs(ref) * 2.0 ** -11 + 2.0 ** -25 + slack * np.max(np.abs(f64(wr))), "dx")
    near(f64(dwr), W.grad.numpy(), slack * np.sum(np.abs(f64(x)), axis=0), "drouter_w")


def test_forward_block_on_another_stream(torch):
    say("forward_block on two streams at once, each with its own workspace, equal to calls alone")
    L = synth.make_layer(synth.WORKLOADS["tiny"])
    dev, w = DeviceLayer(L, device=DEV), L.wl
    g, wr = rand(torch, 3, (1, w.H), "f16")[0], torch.from_numpy(synth.draw_router_weights(5, w.E, w.H)).to(DEV)
    sets, want = [], []
    for n in range(2):
        ws = torch.empty_like(dev.ws)
        B.pw_workspace_init(ws)
        sets.append((rand(torch, 10 + n, (w.T, w.H), "f16"), rand(torch, 20 + n, (w.T, w.H), "f16"), ws))
    call = lambda x, res, y, ws, st: B.pw_moe_forward_block(dev.shape, w.T, x, res, g, EPS, wr, dev.blocks[0], dev.q, y,
                                                            None, None, ws, stream=st)
    for x, res, ws in sets:
        r, y = res.clone(), torch.empty_like(x)
        for _ in range(3):
            call(x, r, y, ws, None)
        want.append((r, y))
    torch.cuda.synchronize()
    out = [(res.clone(), torch.empty_like(x)) for x, res, _ in sets]
    streams = [torch.cuda.Stream() for _ in sets]
    torch.cuda.synchronize()
    for _ in range(3):
        for (x, _, ws), (r, y), st in zip(sets, out, streams):
            call(x, r, y, ws, st)
    torch.cuda.synchronize()
    for (r, y), (rw, yw) in zip(out, want):
        assert torch.equal(r, rw) and torch.equal(y, yw)
