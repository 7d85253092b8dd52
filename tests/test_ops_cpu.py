"""The operators around the layer refuse bad arguments on the host, before any
launch: C entry points by made-up pointers, the binding by tensors that are not
on a GPU.  No GPU needed."""
import ctypes
import os
import subprocess

import pytest

from any_precision_bitplane_amd import binding as B

P = 1 << 20     # a made-up aligned address: every call below ends before it is used
HUGE = 1 << 60


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(B.LIB_PATH):
        pytest.fail("libpagedweight.so is not built (python -m any_precision_bitplane_amd.build)")
    return B.load()


def test_rmsnorm_refusals(lib):
    def call(T=4, H=64, dt=B.PW_F16, x=P, xs=64, res=P, rs=64, out=P, os_=64, w=P, eps=1e-5, ydt=B.PW_F16, y=P, ys=64,
             scale=None, group=0):
        return lib.pw_rmsnorm(T, H, dt, x, xs, res, rs, out, os_, w, eps, ydt, y, ys, scale, group, None)

    inv, shape, align = B.PW_ERR_INVALID_ARG, B.PW_ERR_UNSUPPORTED_SHAPE, B.PW_ERR_ALIGNMENT
    assert call(T=0) == B.PW_OK and call(T=0, x=None, y=None) == B.PW_OK
    assert call(T=-1) == inv and call(H=0) == inv and call(H=-8) == inv
    assert call(H=60) == shape and call(H=32776) == shape
    assert call(dt=7) == inv and call(dt=B.PW_E4M3) == inv and call(ydt=B.PW_BF16) == inv
    assert call(eps=-1e-5) == inv and call(eps=float("nan")) == inv and call(eps=float("inf")) == inv
    assert call(x=None) == inv and call(w=None) == inv and call(y=None) == inv
    assert call(res=None) == inv                         # a sum to store, nothing to add
    assert call(xs=-64) == inv and call(ys=56) == inv and call(os_=56) == inv
    assert call(x=P + 2) == align and call(w=P + 8) == align and call(y=P + 4) == align and call(res=P + 8) == align
    assert call(xs=65) == align and call(rs=68) == align
    assert call(scale=P) == inv and call(group=128) == inv
    e = dict(ydt=B.PW_E4M3, scale=P)
    assert call(**{**e, "scale": None}) == inv and call(**e, group=64) == inv
    assert call(**{**e, "scale": P + 2}) == align and call(**e, ys=68) == align


def test_rmsnorm_backward_refusals(lib):
    def call(T=4, H=64, dt=B.PW_BF16, dy=P, dys=64, r=P, rs=64, w=P, eps=1e-5, res=None, ress=0, dx=P, dxs=64, dw=P,
             ws=P, n=HUGE):
        return lib.pw_rmsnorm_backward(T, H, dt, dy, dys, r, rs, w, eps, res, ress, dx, dxs, dw, ws, n, None)

    inv, align = B.PW_ERR_INVALID_ARG, B.PW_ERR_ALIGNMENT
    assert call(T=0, dw=None) == B.PW_OK
    assert call(T=-1) == inv and call(H=0) == inv and call(dt=B.PW_E4M3) == inv and call(eps=-1.0) == inv
    assert call(H=12) == B.PW_ERR_UNSUPPORTED_SHAPE
    assert call(dy=None) == inv and call(r=None) == inv and call(w=None) == inv and call(dx=None) == inv
    assert call(ws=None) == inv and call(dxs=32) == inv and call(rs=-8) == inv
    assert call(dw=P + 4) == align and call(ws=P + 16) == align and call(dy=P + 2) == align
    assert call(res=P, ress=65) == align
    need = B.pw_rmsnorm_backward_workspace_bytes(4, 64)
    assert need > 0 and call(n=need - 1) == B.PW_ERR_WORKSPACE
    assert B.pw_rmsnorm_backward_workspace_bytes(4, 12) == 0 and B.pw_rmsnorm_backward_workspace_bytes(-1, 64) == 0


@pytest.fixture
def shp():
    return B.shape(256, 512, 8, 2)


def test_permute_refusals(lib, shp):
    def call(shape=shp, T=4, dt=B.PW_F16, x=P, xst=256, xsc=None, groups=0, ids=P, xs=P, xss=256, xssc=None, off=P,
             inv=P, perm=P, status=None, ws=P, n=HUGE):
        return lib.pw_moe_permute(ctypes.byref(shape), T, dt, x, xst, xsc, groups, ids, xs, xss, xssc, off, inv, perm,
                                  status, ws, n, None)

    bad, align = B.PW_ERR_INVALID_ARG, B.PW_ERR_ALIGNMENT
    assert call(T=-1) == bad and call(dt=9) == bad and call(shape=B.shape(256, 512, 8, 9)) == B.PW_ERR_UNSUPPORTED_SHAPE
    assert call(shape=B.shape(250, 512, 8, 2)) == B.PW_ERR_UNSUPPORTED_SHAPE
    for name in ("x", "ids", "xs", "off", "inv", "ws"):
        assert call(**{name: None}) == bad, name
    assert call(T=0, off=None) == bad
    assert call(groups=2) == bad and call(xsc=P, groups=2) == bad and call(groups=-1) == bad and call(xsc=P) == bad
    assert call(xss=128) == bad and call(xst=-256) == bad
    assert call(dt=B.PW_E4M3, xss=264) == align          # 8-bit rows: 264 bytes apart
    for name in ("x", "ids", "xs", "off", "inv", "perm", "status", "ws"):
        assert call(**{name: P + 2}) == align, name
    need = B.pw_moe_permute_workspace_bytes(shp, 4)
    assert need > 0 and call(n=need - 1) == B.PW_ERR_WORKSPACE
    assert B.pw_moe_permute_workspace_bytes(B.shape(250, 512, 8, 2), 4) == 0


def test_unpermute_refusals(lib, shp):
    def back(T=4, dt=B.PW_F16, rows=P, rs=256, inv=P, w=P, y=P, ys=256, shape=shp):
        return lib.pw_moe_unpermute(ctypes.byref(shape), T, dt, rows, rs, inv, w, y, ys, None)

    bad, align = B.PW_ERR_INVALID_ARG, B.PW_ERR_ALIGNMENT
    assert back(T=0) == B.PW_OK and back(T=-1) == bad and back(dt=B.PW_E4M3) == bad
    assert back(rows=None) == bad and back(inv=None) == bad and back(y=None) == bad and back(ys=8) == bad
    assert back(rows=P + 2) == align and back(inv=P + 1) == align and back(w=P + 2) == align and back(ys=260) == align
    assert back(shape=B.shape(256, 512, 300, 2)) == B.PW_ERR_UNSUPPORTED_SHAPE
    f = lib.pw_moe_permute_backward
    s = ctypes.byref(shp)
    assert f(s, 0, B.PW_F16, P, 256, P, P, 256, None) == B.PW_OK
    assert f(s, 4, B.PW_E4M3, P, 256, P, P, 256, None) == bad and f(s, 4, B.PW_F16, P, 256, None, P, 256, None) == bad
    assert f(s, 4, B.PW_F16, P, 256, P, P + 8, 256, None) == align

    def grad(T=4, dt=B.PW_F16, dy=P, dys=256, rows=P, rs=256, inv=P, w=P, drows=P, ds=256, dw=P):
        return lib.pw_moe_unpermute_backward(s, T, dt, dy, dys, rows, rs, inv, w, drows, ds, dw, None)

    assert grad(T=0) == B.PW_OK and grad(T=-1) == bad and grad(dt=5) == bad
    assert grad(dy=None) == bad and grad(rows=None) == bad and grad(drows=None) == bad and grad(inv=None) == bad
    assert grad(ds=128) == bad and grad(dw=P + 2) == align and grad(rows=P + 4) == align and grad(dys=257) == align


def test_router_backward_refusals(lib, shp):
    def call(shape=shp, T=4, x=P, wr=P, ids=P, w=P, dw=P, add=None, dx=P, out=P, ws=P, n=HUGE):
        return lib.pw_router_backward(ctypes.byref(shape), T, x, wr, ids, w, dw, add, dx, out, ws, n, None)

    assert call(T=-1) == B.PW_ERR_INVALID_ARG
    for name in ("x", "wr", "ids", "w", "dw", "dx", "out", "ws"):
        assert call(**{name: None}) == B.PW_ERR_INVALID_ARG, name
    for name in ("x", "wr", "ids", "w", "dw", "add", "dx", "out", "ws"):
        assert call(**{name: P + 2}) == B.PW_ERR_ALIGNMENT, name
    assert call(shape=B.shape(256, 512, 128, 65)) == B.PW_ERR_UNSUPPORTED_SHAPE
    need = B.pw_router_backward_workspace_bytes(shp, 4)
    assert need > 0 and call(n=need - 1) == B.PW_ERR_WORKSPACE


def test_workspaces_serve_smaller_calls(lib):
    """A workspace for T_max tokens is enough for every smaller call."""
    for H, E, k in [(32, 1, 1), (256, 8, 2), (2048, 60, 4), (4096, 8, 2), (8192, 256, 8)]:
        s = B.shape(H, 32, E, k)
        last = (0, 0, 0)
        for T in list(range(0, 3000, 7)) + [4095, 4096, 16383, 16384, 16385, 32768, 100000, 1 << 20]:
            now = (B.pw_router_backward_workspace_bytes(s, T), B.pw_moe_permute_workspace_bytes(s, T),
                   B.pw_rmsnorm_backward_workspace_bytes(T, H))
            assert all(a <= b for a, b in zip(last, now)), (H, E, k, T)
            last = now


def test_forward_block_refusals(lib, shp):
    def call(shape=shp, T=4, x=P, res=P, g=P, eps=1e-5, wr=P, bl=P, q=P, y=P, cnt=None, mass=None, ws=P, n=HUGE,
             opts=None):
        return lib.pw_moe_forward_block(ctypes.byref(shape), T, x, res, g, eps, wr, bl, q, y, cnt, mass, ws, n,
                                        ctypes.byref(opts) if opts is not None else None, None)

    assert call(T=0) == B.PW_OK and call(T=-1) == B.PW_ERR_INVALID_ARG and call(eps=-1.0) == B.PW_ERR_INVALID_ARG
    for name in ("x", "res", "g", "wr", "bl", "q", "y", "ws"):
        assert call(**{name: None}) == B.PW_ERR_INVALID_ARG, name
    for name in ("x", "res", "g", "wr", "bl", "y", "cnt", "mass", "ws"):
        assert call(**{name: P + 2}) == B.PW_ERR_ALIGNMENT, name
    assert call(n=256) == B.PW_ERR_WORKSPACE
    assert call(opts=B.make_options(path=9)) == B.PW_ERR_INVALID_ARG
    assert call(opts=B.make_options(event_mode=9)) == B.PW_ERR_INVALID_ARG
    assert call(shape=B.shape(256, 512, 128, 65)) == B.PW_ERR_UNSUPPORTED_SHAPE
    assert call(shape=B.shape(32800, 32, 8, 2)) == B.PW_ERR_UNSUPPORTED_SHAPE


def test_binding_refuses_host_tensors(lib, shp):
    import torch
    x = torch.zeros(4, 256, dtype=torch.float16)
    i = torch.zeros(8, dtype=torch.int32)
    f = torch.zeros(8)
    ws = torch.zeros(1 << 16, dtype=torch.uint8)
    calls = [
        lambda check: B.pw_rmsnorm(4, 256, x, x[0], 1e-5, x, check=check),
        lambda check: B.pw_rmsnorm_backward(4, 256, x, x, x[0], 1e-5, x, check=check),
        lambda check: B.pw_moe_permute(shp, 4, x, i, x, i, i, i, ws, check=check),
        lambda check: B.pw_moe_permute_backward(shp, 4, x, i, x, check=check),
        lambda check: B.pw_moe_unpermute(shp, 4, x, i, f, x, check=check),
        lambda check: B.pw_moe_unpermute_backward(shp, 4, x, x, i, f, x, f, check=check),
        lambda check: B.pw_router_backward(shp, 4, x, x, i, f, f, x, f, ws, check=check),
    ]
    for call in calls:
        assert call(False) == B.PW_ERR_INVALID_ARG
        with pytest.raises(B.PwError, match="GPU") as e:
            call(True)
        assert e.value.status == B.PW_ERR_INVALID_ARG


def block_args(torch, shp, T=4, where=lambda t: t):
    """Arguments of pw_moe_forward_block by name, as zeros on the host; `where` puts each somewhere."""
    h = lambda *n: where(torch.zeros(n, dtype=torch.float16))
    H, E = shp.hidden, shp.num_experts
    return {"x": h(T, H), "residual": h(T, H), "norm_w": h(H), "eps": 1e-5, "router_w": h(E, H),
            "blocks": where(torch.zeros((E, 2, 2), dtype=torch.int64)),
            "q": where(torch.zeros((E, 2), dtype=torch.uint8)), "y": h(T, H), "stat_count": where(torch.zeros(E, dtype=torch.int32)), "stat_mass": where(torch.zeros(E)),
            "workspace": where(torch.zeros(B.pw_workspace_bytes(shp, T), dtype=torch.uint8))}


class Elsewhere:
    """A host tensor that says it is on GPU `index`: enough for the binding's checks, never launched on."""

    def __init__(self, t, index):
        self.t, self.index = t, index

    def get_device(self):
        return self.index

    def __getattr__(self, name):
        return getattr(self.t, name)


def test_forward_block_binding_refuses_host_tensors(lib, shp):
    import torch
    args = block_args(torch, shp)
    assert B.pw_moe_forward_block(shp, 4, **args, check=False) == B.PW_ERR_INVALID_ARG
    with pytest.raises(B.PwError, match="GPU"):
        B.pw_moe_forward_block(shp, 4, **args)


def test_forward_block_binding_checks_and_device(lib, shp, monkeypatch):
    """Every tensor's device, type and size are checked before the call, which goes to the tensors' GPU and a stream
    of it, whichever GPU is current."""
    import contextlib

    import torch
    B._load_ops()
    calls, entered = [], []

    @contextlib.contextmanager
    def device(d):
        entered.append(d)
        yield

    class Lib:
        @staticmethod
        def pw_moe_forward_block(*a):
            calls.append(a)
            return B.PW_OK

    monkeypatch.setattr(B, "_lib", Lib)
    monkeypatch.setattr(B, "_current_device", lambda: 0)
    monkeypatch.setattr(B, "_current_stream", lambda dev: 1000 + dev)
    monkeypatch.setattr(torch.cuda, "device", device)
    with monkeypatch.context() as m:
        m.setattr(B, "_lib", lib)
        good = block_args(torch, shp, where=lambda t: Elsewhere(t, 1))
    call = lambda **kw: B.pw_moe_forward_block(shp, 4, **{**good, **kw}, check=False)
    assert call() == B.PW_OK and entered == [1] and calls[-1][-1] == 1001
    assert call(blocks=1 << 20, q=1 << 21, stat_count=None, stat_mass=None) == B.PW_OK     # raw tables, no statistics
    assert calls[-1][7] == 1 << 20 and calls[-1][8] == 1 << 21
    assert call(stat_count=Elsewhere(good["stat_count"].t.view(torch.uint32), 1)) == B.PW_OK
    n = len(calls)
    for name, arg in good.items():
        if name == "eps":
            continue
        t = arg.t
        assert call(**{name: Elsewhere(t, 0)}) == B.PW_ERR_INVALID_ARG, name                # another GPU
        assert call(**{name: t}) == B.PW_ERR_INVALID_ARG, name                              # the host
        wide = torch.zeros((*t.shape, 2), dtype=t.dtype)[..., 0]
        assert call(**{name: Elsewhere(wide, 1)}) == B.PW_ERR_INVALID_ARG, name             # elements apart
        if name == "workspace":
            continue                                                                        # the library's own check
        assert call(**{name: Elsewhere(t.reshape(-1)[:-1], 1)}) == B.PW_ERR_INVALID_ARG, name
        if name not in ("blocks", "q"):
            assert call(**{name: Elsewhere(t.double(), 1)}) == B.PW_ERR_INVALID_ARG, name
    for name in ("x", "residual", "norm_w", "router_w", "y"):
        assert call(**{name: Elsewhere(good[name].t.bfloat16(), 1)}) == B.PW_ERR_INVALID_ARG, name
    assert call(x=None) == B.PW_ERR_INVALID_ARG and len(calls) == n


def test_router_gradient_workspace_is_what_its_plan_uses(tmp_path):
    """For up to 2^20 tokens: enough for every smaller call, and at most about twice what the largest uses."""
    from any_precision_bitplane_amd import build
    exe = str(tmp_path / "plan_test")
    subprocess.run([build.hipcc(), "-x", "hip", "--offload-host-only", "-O1", "-std=c++17", "-I", build.CSRC,
                    os.path.join(build.ROOT, "tests", "cpp", "router_grad_plan_test.cpp"), "-o", exe], check=True)
    r = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stdout


def test_router_gradient_workspace_of_large_calls(lib):
    """What 4096 blocks' shares take, whatever the number of tokens."""
    size = lambda H, E, k, T: B.pw_router_backward_workspace_bytes(B.shape(H, 32, E, k), T) >> 20
    assert size(8192, 256, 8, 1 << 20) <= 34 and size(7168, 256, 8, 1 << 18) <= 34
    assert size(4096, 8, 2, 1 << 20) <= 34 and size(2048, 60, 4, 32768) <= 34


def test_permute_binding_takes_unsigned_status(lib, shp, monkeypatch):
    """The status word is a device uint32: torch.uint32 and int32 are both passed on, other types refused."""
    import torch
    B._load_ops()
    calls = []

    class Lib:
        @staticmethod
        def pw_moe_permute(*a):
            calls.append(a)
            return B.PW_OK

    monkeypatch.setattr(B, "_lib", Lib)
    monkeypatch.setattr(B, "_current_device", lambda: 0)
    monkeypatch.setattr(B, "_current_stream", lambda dev: 0)
    on = lambda *n, d=torch.int32: Elsewhere(torch.zeros(n, dtype=d), 0)
    x, xs = on(4, 256, d=torch.float16), on(8, 256, d=torch.float16)
    call = lambda st: B.pw_moe_permute(shp, 4, x, on(4, 2), xs, on(9), on(8), None, on(64), status=st, check=False)
    for dtype in (torch.int32, torch.uint32):
        status = on(1, d=dtype)
        assert call(status) == B.PW_OK and calls[-1][14] == status.t.data_ptr()
    assert call(None) == B.PW_OK and calls[-1][14] is None
    assert call(on(1, d=torch.int64)) == B.PW_ERR_INVALID_ARG and len(calls) == 3
