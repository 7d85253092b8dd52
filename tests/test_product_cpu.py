"""The expert products refuse bad arguments on the host, before any launch: C
entry points by made-up pointers, the binding by tensors that are not on a GPU.
No GPU needed."""
import ctypes
import os
import subprocess

import pytest

from any_precision_bitplane_amd import binding as B
from any_precision_bitplane_amd import build

P = 1 << 20     # a made-up aligned address: every call below ends before it is used
HUGE = 1 << 60
BAD, SHAPE, ALIGN = B.PW_ERR_INVALID_ARG, B.PW_ERR_UNSUPPORTED_SHAPE, B.PW_ERR_ALIGNMENT


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(B.LIB_PATH):
        pytest.fail("libpagedweight.so is not built (python -m any_precision_bitplane_amd.build)")
    return B.load()


def test_product_refusals(lib):
    def call(E=3, S=4, N=64, K=72, dt=B.PW_F16, x=P, xs=72, off=P, w=P, bias=None, act=0, res=None, rs=64, pre=None, ps=64,
             y=P, ys=64, ws=P, n=HUGE):
        return lib.pw_moe_product(E, S, N, K, dt, x, xs, off, w, bias, act, res, rs, pre, ps, y, ys, ws, n, None)

    assert call(S=0) == B.PW_OK and call(S=0, x=None, y=None, w=None) == B.PW_OK
    assert call(E=0) == BAD and call(S=-1) == BAD and call(N=0) == BAD and call(K=-8) == BAD
    assert call(E=257) == SHAPE and call(N=60) == SHAPE and call(K=68) == SHAPE
    assert call(N=1 << 23) == SHAPE and call(K=1 << 23) == SHAPE and call(N=1 << 16, K=1 << 15) == SHAPE
    assert call(xs=1 << 22) == SHAPE and call(ys=1 << 22) == SHAPE
    assert call(dt=B.PW_F32) == BAD and call(dt=B.PW_E4M3) == BAD and call(dt=9) == BAD
    assert call(act=3) == BAD and call(act=-1) == BAD
    assert call(off=None) == BAD and call(off=P + 2) == ALIGN
    for name in ("x", "w", "y", "ws"):
        assert call(**{name: None}) == BAD, name
    assert call(xs=-72) == BAD and call(ys=56) == BAD and call(pre=P, ps=56) == BAD
    assert call(x=P + 8) == ALIGN and call(w=P + 8) == ALIGN and call(bias=P + 8) == ALIGN and call(y=P + 8) == ALIGN
    assert call(xs=76) == ALIGN and call(res=P, rs=65) == ALIGN and call(pre=P + 2) == ALIGN and call(ws=P + 16) == ALIGN
    need = B.pw_moe_product_workspace_bytes(3, 4, 64, 72)
    assert need > 0 and call(n=need - 1) == B.PW_ERR_WORKSPACE
    assert B.pw_moe_product_workspace_bytes(3, 4, 60, 72) == 0 and B.pw_moe_product_workspace_bytes(0, 4, 64, 72) == 0


def test_product_backward_refusals(lib):
    def call(E=3, S=4, N=64, K=72, dt=B.PW_BF16, dy=P, dys=64, x=P, xs=72, off=P, w=P, act=0, pre=None, ps=64, dx=P,
             dxs=72, dw=P, db=P, ws=P, n=HUGE):
        return lib.pw_moe_product_backward(E, S, N, K, dt, dy, dys, x, xs, off, w, act, pre, ps, dx, dxs, dw, db, ws, n,
                                           None)

    assert call(S=0, dw=None, db=None) == B.PW_OK
    assert call(S=-1) == BAD and call(N=4) == SHAPE and call(dt=B.PW_F32) == BAD and call(off=None) == BAD
    assert call(act=1) == BAD and call(pre=P) == BAD            # the slope needs the sum, and nothing else does
    assert call(dy=None) == BAD and call(w=None) == BAD and call(x=None) == BAD and call(ws=None) == BAD
    assert call(dxs=64) == BAD and call(dxs=76) == ALIGN and call(dys=1 << 22) == SHAPE
    assert call(dw=P + 4) == ALIGN and call(db=P + 2) == ALIGN and call(act=2, pre=P + 8) == ALIGN
    need = B.pw_moe_product_backward_workspace_bytes(3, 4, 64, 72)
    assert need >= 4 * 64 * 2 and call(n=need - 1) == B.PW_ERR_WORKSPACE
    assert B.pw_moe_product_backward_workspace_bytes(3, -4, 64, 72) == 0


def test_gradient_of_no_rows_with_an_activation(lib):
    """pre is needed where there are rows; without rows it may be there (a buffer for the largest step) or not."""
    def call(act, pre, S=0):
        return lib.pw_moe_product_backward(3, S, 64, 72, B.PW_BF16, P, 64, P, 72, P, P, act, pre, 64, P, 72, None, None, P,
                                           HUGE, None)

    for act in (B.PW_ACT_SILU, B.PW_ACT_GELU):
        assert call(act, None) == B.PW_OK and call(act, P) == B.PW_OK and call(act, None, 4) == BAD
    assert call(B.PW_ACT_NONE, None) == B.PW_OK and call(B.PW_ACT_NONE, P) == BAD


def test_strides_of_single_rows(lib):
    """One row of the largest size is no shape to refuse (the null matrix behind it is), two rows that far apart are."""
    def call(S, N, K, xs, ys):
        return lib.pw_moe_product(1, S, N, K, B.PW_F16, P, xs, None, P, None, 0, None, 0, None, 0, None if S == 1 else P, ys, P,
                                  HUGE, None)

    far = 1 << 22
    assert call(1, far, 64, 64, far) == BAD and call(1, 64, far, far, 64) == BAD
    assert call(1, 64, 64, far + 8, 64) == SHAPE and call(2, 64, 64, far, 64) == SHAPE and call(2, far, 64, 64, far) == SHAPE


def test_rows_that_tiles_cannot_count(lib):
    """Rounded up to whole tiles of 256, the rows have to be a 32-bit number."""
    most = (1 << 31) - 256
    for size in (B.pw_moe_product_workspace_bytes, B.pw_moe_product_backward_workspace_bytes):
        assert size(1, most, 8, 8) > 0
        assert all(size(1, S, 8, 8) == 0 for S in (most + 1, (1 << 31) - 1))
    for S in (most + 1, (1 << 31) - 1):
        assert lib.pw_moe_product(1, S, 8, 8, B.PW_F16, P, 8, None, P, None, 0, None, 0, None, 0, P, 8, P, HUGE, None) == SHAPE
        assert lib.pw_moe_product_backward(1, S, 8, 8, B.PW_F16, P, 8, P, 8, None, P, 0, None, 0, P, 8, P, P, P, HUGE,
                                           None) == SHAPE


def test_ffn_refusals(lib):
    shp = B.shape(64, 96, 3, 2)

    def call(shape=shp, S=4, dt=B.PW_F16, x=P, xs=64, off=P, wg=P, wd=P, act=1, zt=B.PW_F16, z=None, zs=192, sc=None, y=P,
             ys=64, ws=P, n=HUGE):
        return lib.pw_moe_ffn(ctypes.byref(shape), S, dt, x, xs, off, wg, wd, act, zt, z, zs, sc, y, ys, ws, n, None)

    assert call(S=0) == B.PW_OK and call(S=-1) == BAD
    assert call(shape=B.shape(60, 96, 3, 2)) == SHAPE and call(shape=B.shape(64, 96, 300, 2)) == SHAPE
    assert call(shape=B.shape(32, 1 << 22, 3, 2)) == SHAPE and call(shape=B.shape(1 << 23, 32, 3, 2)) == SHAPE
    assert B.pw_moe_ffn_backward_workspace_bytes(B.shape(32, 1 << 22, 3, 2), 4) == 0
    assert call(dt=B.PW_F32) == BAD and call(act=0) == BAD and call(act=3) == BAD and call(off=None) == BAD
    for name in ("x", "wg", "wd", "y", "ws"):
        assert call(**{name: None}) == BAD, name
    assert call(sc=P) == BAD and call(z=P, sc=P) == BAD and call(z=P, zt=B.PW_BF16) == BAD
    assert call(z=P, zt=B.PW_E4M3) == BAD and call(z=P, zt=B.PW_E4M3, sc=P + 2) == ALIGN
    assert call(z=P, zs=184) == BAD and call(z=P, zt=B.PW_E4M3, sc=P, zs=200) == ALIGN and call(z=P + 4) == ALIGN
    assert call(xs=68) == ALIGN and call(ys=32) == BAD and call(wd=P + 2) == ALIGN and call(ws=P + 8) == ALIGN
    need = B.pw_moe_ffn_workspace_bytes(shp, 4)
    assert need >= 4 * 96 * 2 and call(n=need - 1) == B.PW_ERR_WORKSPACE
    assert B.pw_moe_ffn_workspace_bytes(B.shape(60, 96, 3, 2), 4) == 0


def test_ffn_of_no_rows_with_a_checkpoint(lib):
    """Of codes without rows the address is null; the scales' buffer may be one for the largest step."""
    shp = B.shape(64, 96, 3, 2)
    call = lambda S, z: lib.pw_moe_ffn(ctypes.byref(shp), S, B.PW_F16, P, 64, P, P, P, B.PW_ACT_SILU, B.PW_E4M3, z, 192, P, P, 64,
                                       None, 0, None)
    assert call(0, None) == B.PW_OK and call(0, P) == B.PW_OK and call(4, None) == BAD


def test_ffn_backward_refusals(lib):
    shp = B.shape(64, 96, 3, 2)

    def call(shape=shp, S=4, dt=B.PW_F16, dy=P, dys=64, x=P, xs=64, off=P, wg=P, wd=P, act=1, zt=B.PW_F16, z=P, zs=192,
             sc=None, dx=P, dxs=64, dg=P, dd=P, ws=P, n=HUGE):
        return lib.pw_moe_ffn_backward(ctypes.byref(shape), S, dt, dy, dys, x, xs, off, wg, wd, act, zt, z, zs, sc, dx, dxs,
                                       dg, dd, ws, n, None)

    assert call(S=0, dg=None, dd=None) == B.PW_OK and call(S=-1) == BAD
    assert call(dt=B.PW_E4M3) == BAD and call(act=0) == BAD and call(off=None) == BAD
    for name in ("dy", "x", "wg", "wd", "z", "ws"):
        assert call(**{name: None}) == BAD, name
    assert call(zt=B.PW_E4M3) == BAD and call(sc=P) == BAD and call(zt=B.PW_BF16) == BAD
    assert call(zs=190) == ALIGN and call(zt=B.PW_E4M3, sc=P, zs=200) == ALIGN
    assert call(dxs=60) == BAD and call(dg=P + 2) == ALIGN and call(dd=P + 8) == ALIGN and call(dys=68) == ALIGN
    need = B.pw_moe_ffn_backward_workspace_bytes(shp, 4)
    assert need >= 4 * 3 * 96 * 2 and call(n=need - 1) == B.PW_ERR_WORKSPACE


def test_workspaces_grow_with_rows(lib):
    shp = B.shape(2048, 1408, 60, 4)
    for size in (lambda S: B.pw_moe_ffn_workspace_bytes(shp, S), lambda S: B.pw_moe_ffn_backward_workspace_bytes(shp, S),
                 lambda S: B.pw_moe_product_workspace_bytes(8, S, 4096, 2048),
                 lambda S: B.pw_moe_product_backward_workspace_bytes(8, S, 4096, 2048)):
        sizes = [size(S) for S in list(range(0, 700)) + [1000, 4095, 4096, 100000, 1 << 24]]
        assert all(a <= b for a, b in zip(sizes, sizes[1:])) and all(s % 256 == 0 and s > 0 for s in sizes)


@pytest.mark.parametrize("fuse", ["off", "fast"])
def test_parts_of_a_cut_tile_are_the_same_however_the_compiler_fuses(tmp_path, fuse):
    """The products and the launch that joins their parts work the number out apart: it has ties, and no rounding may break them."""
    exe = str(tmp_path / "parts_test")
    subprocess.run([build.hipcc(), "-x", "hip", "--offload-host-only", "-O2", "-mfma", f"-ffp-contract={fuse}", "-std=c++17",
                    "-I", build.CSRC, os.path.join(build.ROOT, "tests", "cpp", "product_parts_test.cpp"), "-o", exe], check=True)
    r = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stdout


def test_copies_to_lds_compile_without_a_warning(tmp_path):
    """Inline assembly that changes a register behind the compiler's back is warned of, and is no behaviour to build on."""
    src = tmp_path / "copy.hip"
    src.write_text("""#include "pw_product.h"
__global__ void copy(const char* p, char* q) {
  __shared__ char lds[2048];
  pw::copy16<1024>(pw::copy_rsrc(p), pw::lds_at(lds), threadIdx.x * 16, 64);
  pw::step_barrier<0>();
  q[threadIdx.x] = lds[1024 + threadIdx.x];
}
""")
    r = subprocess.run([build.hipcc(), *build.COMMON, "-Werror", "-I", build.CSRC, "-x", "hip", "--cuda-device-only", "-S",
                        str(src), "-o", str(tmp_path / "copy.s")], capture_output=True, text=True)
    assert r.returncode == 0 and "warning" not in r.stderr, r.stderr
    text = (tmp_path / "copy.s").read_text()
    assert "offen lds" in text and "m0" in text


def test_binding_refuses_tensors_that_are_on_no_gpu():
    import torch
    x, w = torch.zeros((4, 64), dtype=torch.float16), torch.zeros((1, 64, 64), dtype=torch.float16)
    ws = torch.zeros(1 << 16, dtype=torch.uint8)
    with pytest.raises(B.PwError):
        B.pw_moe_product(1, 4, 64, 64, x, w, x, ws)
    with pytest.raises(B.PwError):
        B.pw_moe_product_backward(1, 4, 64, 64, x, x, w, ws, dx=x)
    assert B.pw_moe_ffn(B.shape(64, 64, 1, 1), 4, None, w, w, x, ws, check=False) == BAD
    assert B.pw_moe_ffn_backward(B.shape(64, 64, 1, 1), 4, x, x, w, w, x, ws, check=False) == BAD
