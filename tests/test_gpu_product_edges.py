"""The expert products in 16 bits at the edges of what their calls take, on the GPU.

Tolerances count roundings: U = 2^-24 is half a step of fp32, a stored value is
off by half a step of its type relative to itself and half a subnormal step.
Every case prints what it runs first.
"""
import math

import numpy as np
import pytest

from any_precision_bitplane_amd import binding as B
from test_gpu_product import DEV, DTYPES, U, dtype_of, f64, half_step, near, rand, say, scratch, torch, whole  # noqa: F401

pytestmark = pytest.mark.gpu


def gelu64(z):
    """GELU, its slope, and by how much fp32 may be off from either, at z < -2.

    exp(-z^2 / 2): three roundings of the exponent (z^2, the constant log2 e, their product), each z^2 / 2 times as
    large in the result, and the function 1 ulp (2 U).  Phi is that times t P(t), t = 1 / (1 + 0.3 |z|) off by 4 U and
    P by at most 2 times as much of it, P's fit 3 U, its coefficients' roundings and seven steps of magnitudes up to
    1.85 times its value 2 and 14 U, the two products 2 U: with exp's 2 below 44 U.  Its product with z is one rounding
    more; the slope's other part has four (with z and 1 / sqrt(2 pi)), and the sum one.
    """
    phi = np.vectorize(lambda v: math.erfc(-v / math.sqrt(2)) / 2, otypes=[np.float64])(z)
    bell = z * np.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    of_phi = phi * (1.5 * z * z + 44) * U
    return z * phi, phi + bell, np.abs(z) * of_phi, of_phi + np.abs(bell) * (1.5 * z * z + 8) * U + np.abs(phi + bell) * U


@pytest.mark.parametrize("S", [9, 300])
@pytest.mark.parametrize("name", DTYPES)
def test_gelu_far_below_zero(torch, name, S):  # noqa: F811
    """z from -12.5 on, where z Phi(z) is some 1e-35: off by so much relative to itself, as bf16 holds it."""
    say(f"GELU of -12.5 .. -3, {name}, S={S}")
    t, I = dtype_of(torch, name), 64
    z = torch.linspace(-12.5, -3, S * I).reshape(S, I).to(t).to(DEV)
    act, slope, ea, es = gelu64(f64(z))
    rel, ab = half_step(torch, name)
    ok = lambda got, ref, e, what: near(f64(got), ref, e + rel * (np.abs(ref) + e) + ab, what)
    eye = torch.eye(I, dtype=t, device=DEV)

    # the product with the unit matrix
    y = torch.empty((S, I), dtype=t, device=DEV)
    B.pw_moe_product(1, S, I, I, z, eye, y, scratch(torch, B.pw_moe_product_workspace_bytes(1, S, I, I)), act=B.PW_ACT_GELU)
    ok(y, act, ea, "act")
    one, dx = torch.ones_like(z), torch.empty_like(z)
    ws = scratch(torch, B.pw_moe_product_backward_workspace_bytes(1, S, I, I))
    B.pw_moe_product_backward(1, S, I, I, one, None, eye, ws, act=B.PW_ACT_GELU, pre=z, dx=dx)
    ok(dx, slope, es, "slope")

    # the block with gate = z, up = 1 and h taken as it is
    H, shp = 2 * I, B.shape(2 * I, I, 1, 1)
    x = torch.cat([z, one], dim=1)
    w_gate_up = torch.eye(H, dtype=t, device=DEV)
    w_down = torch.cat([eye, 0 * eye])
    y, kept = torch.empty((S, H), dtype=t, device=DEV), torch.empty((S, 2 * I), dtype=t, device=DEV)
    B.pw_moe_ffn(shp, S, x, w_gate_up, w_down, y, scratch(torch, B.pw_moe_ffn_workspace_bytes(shp, S)), act=B.PW_ACT_GELU,
                 z=kept)
    assert torch.equal(kept, x) and not bool(y[:, I:].any())
    ok(y[:, :I], act, ea, "h")
    dx = torch.empty_like(x)
    B.pw_moe_ffn_backward(shp, S, torch.cat([one, one], dim=1), None, w_gate_up, w_down, kept,
                          scratch(torch, B.pw_moe_ffn_backward_workspace_bytes(shp, S)), act=B.PW_ACT_GELU, dx=dx)
    ok(dx[:, :I], slope, es, "dgate")
    ok(dx[:, I:], act, ea, "dup")


@pytest.mark.parametrize("act", [B.PW_ACT_SILU, B.PW_ACT_GELU], ids=["silu", "gelu"])
def test_gradient_of_no_rows_with_an_activation(torch, act):  # noqa: F811
    say("product backward of no rows, the sum's buffer there or not")
    E, N, K = 3, 64, 72
    none = torch.empty((0, N), dtype=torch.float16, device=DEV), torch.empty((0, K), dtype=torch.float16, device=DEV)
    w, pre = rand(torch, 1, (E, N, K), "f16"), rand(torch, 2, (40, N), "f16")
    off = torch.zeros(E + 1, dtype=torch.int32, device=DEV)
    ws = scratch(torch, B.pw_moe_product_backward_workspace_bytes(E, 0, N, K))
    for kept in (None, pre):
        dx, dw, db = torch.full((8, K), 7.0, device=DEV).half(), torch.full_like(w, 7.0), torch.full((E, N), 7.0, dtype=w.dtype, device=DEV)
        B.pw_moe_product_backward(E, 0, N, K, *none, w, ws, offsets=off, act=act, pre=kept, dx=dx, dw=dw, dbias=db)
        B.pw_moe_product_backward(E, 0, N, K, *none, w, None, offsets=off, act=act, pre=kept, dx=dx)
        torch.cuda.synchronize()
        assert not bool(dw.any()) and not bool(db.any()) and bool((dx == 7.0).all())


def test_long_matrices_of_many_experts(torch):  # noqa: F811
    """A row for every expert, and more blocks of 16 columns than one launch has threads for."""
    E = S = 256
    N, K = 1 << 20, 8
    say(f"product E={E} S={S} N={N} K={K}")
    g = torch.Generator(device=DEV)
    g.manual_seed(1)
    w = torch.randint(-3, 4, (E, N, K), dtype=torch.int8, generator=g, device=DEV).half()
    x = torch.randint(-3, 4, (S, K), dtype=torch.int8, generator=g, device=DEV).half()
    y = torch.full((S, N), 7.0, dtype=x.dtype, device=DEV)
    off = torch.arange(E + 1, dtype=torch.int32, device=DEV)
    B.pw_moe_product(E, S, N, K, x, w, y, scratch(torch, B.pw_moe_product_workspace_bytes(E, S, N, K)), offsets=off)
    for e in range(E):     # whole numbers below 256: exact
        assert torch.equal(y[e], (w[e].float() * x[e].float()).sum(1).half()), e


@pytest.mark.parametrize("N,K", [(1 << 22, 8), (8, 1 << 22)])
def test_a_row_of_the_largest_size(torch, N, K):  # noqa: F811
    say(f"one row, N={N} K={K}")
    x, w = whole(torch, 1, (1, K), "f16", 1 << 22), whole(torch, 2, (1, N, K), "f16", 1 << 22)
    dy = whole(torch, 3, (1, N), "f16", 1 << 22)
    y, dx, dw = torch.empty_like(dy), torch.empty_like(x), torch.empty_like(w)
    db = torch.empty_like(dy)
    B.pw_moe_product(1, 1, N, K, x, w, y, scratch(torch, B.pw_moe_product_workspace_bytes(1, 1, N, K)))
    B.pw_moe_product_backward(1, 1, N, K, dy, x, w, scratch(torch, B.pw_moe_product_backward_workspace_bytes(1, 1, N, K)), dx=dx,
                              dw=dw, dbias=db)
    assert np.array_equal(f64(y), f64(x) @ f64(w)[0].T) and np.array_equal(f64(dx), f64(dy) @ f64(w)[0])
    assert np.array_equal(f64(dw)[0], f64(dy).T * f64(x)) and torch.equal(db, dy)


def test_offsets_past_the_rows_count_as_the_nearer_end(torch):  # noqa: F811
    E, S, N, K, I = 4, 300, 264, 136, 160
    say(f"offsets below 0 and past S, E={E} S={S}")
    off = torch.tensor([-7, 40, 40, 131, 1 << 30], dtype=torch.int32, device=DEV)
    same = torch.tensor([0, 40, 40, 131, S], dtype=torch.int32, device=DEV)
    x, w, dy = rand(torch, 1, (S, K), "f16"), rand(torch, 2, (E, N, K), "f16"), rand(torch, 3, (S, N), "f16")
    ws = scratch(torch, B.pw_moe_product_backward_workspace_bytes(E, S, N, K))
    shp = B.shape(K - 8, I, E, 1)
    wg, wd, xs = rand(torch, 4, (E, 2 * I, K - 8), "f16", 0.1), rand(torch, 5, (E, K - 8, I), "f16", 0.1), x[:, :K - 8].contiguous()
    wf = scratch(torch, B.pw_moe_ffn_backward_workspace_bytes(shp, S))
    got = []
    for o in (same, off):
        t = [torch.full(s, float("nan"), dtype=x.dtype, device=DEV) for s in
             [(S, N), (S, K), (E, N, K), (E, N), (S, K - 8), (S, 2 * I), (S, K - 8), (E, 2 * I, K - 8), (E, K - 8, I)]]
        B.pw_moe_product(E, S, N, K, x, w, t[0], ws, offsets=o)
        B.pw_moe_product_backward(E, S, N, K, dy, x, w, ws, offsets=o, dx=t[1], dw=t[2], dbias=t[3])
        B.pw_moe_ffn(shp, S, xs, wg, wd, t[4], wf, offsets=o, z=t[5])
        B.pw_moe_ffn_backward(shp, S, xs, xs, wg, wd, t[5], wf, offsets=o, dx=t[6], dw_gate_up=t[7], dw_down=t[8])
        got.append(t)
    torch.cuda.synchronize()
    assert all(torch.equal(a.view(torch.int16), b.view(torch.int16)) for a, b in zip(*got))
    # all of every output is written (a number of the inputs' size could be any fill but NaN), zero for no rows
    assert not bool(got[0][2][1].any()) and not any(bool(t.isnan().any()) for t in got[0])


@pytest.mark.parametrize("S", [3, 200])
def test_overflow_between_two_products(torch, S):  # noqa: F811
    """act(gate) up past the largest fp16 is an infinity, in its row alone; bf16 holds it, and so does the checkpoint."""
    H, I = 64, 32
    say(f"h of 90000 in a row of S={S}")
    shp = B.shape(H, I, 1, 1)
    for name in DTYPES:
        t = dtype_of(torch, name)
        x = torch.zeros((S, H), dtype=t, device=DEV)
        x[:, 0] = 1
        x[S - 2, 0] = 300
        wg, wd = torch.zeros((1, 2 * I, H), dtype=t, device=DEV), torch.full((1, H, I), 2.0 ** -10, dtype=t, device=DEV)
        wg[:, :, 0] = 1
        y, z = torch.empty((S, H), dtype=t, device=DEV), torch.empty((S, 2 * I), dtype=t, device=DEV)
        B.pw_moe_ffn(shp, S, x, wg, wd, y, scratch(torch, B.pw_moe_ffn_workspace_bytes(shp, S)), z=z)
        one = 1 / (1 + math.exp(-1))
        want = np.full((S, H), one * I / 1024)
        want[S - 2] = math.inf if name == "f16" else 90000 * I / 1024
        rel = half_step(torch, name)[0]
        got = f64(y)
        far = np.isinf(want)
        assert np.array_equal(np.isinf(got), far) and bool((z[S - 2] == 300).all())
        # h and y are rounded, sums of equal values are exact but for fp32's rounding, SiLU is off by at most 64 U of itself
        near(got[~far], want[~far], (2 * rel + rel * rel + (64 + I) * U) * want[~far] * (1 + rel), name)
