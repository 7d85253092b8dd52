"""Every form of the expert products in 16 bits: tiles of 32 to 256 rows, whole and cut along the reduction, and the
three tiles of the weights' gradients, on experts of unequal rows.

The first tests ask the host's rules (csrc/pw_internal.h) which form each size takes, on the CPU, so that a changed rule
fails here instead of leaving a form untested; the others run the sizes on the GPU, by the bodies and tolerances of
test_gpu_product.py.
"""
import os
import subprocess

import pytest

import test_gpu_product as tp
from any_precision_bitplane_amd import build
from test_gpu_product import DTYPES, torch  # noqa: F401

ACT, GATE, BACK, GATE_BACK = range(4)

PRODUCTS = {   # (E, S, N, K, ragged): form of the product, of dx, of dw
    (3, 1500, 2760, 136, True): ("256 whole", "32 cut", "128x128 1"),
    (2, 700, 5000, 2600, True): ("256 cut", "32 cut", "256x256 1"),
    (1, 2600, 2296, 2888, False): ("256 cut", "256 whole", "128x128 1"),
    (1, 100, 16600, 1000, False): ("128 whole", "32 cut", "256x128 1"),
    (3, 330, 3304, 1496, True): ("128 cut", "32 cut", "128x128 1"),
    (5, 450, 2504, 136, True): ("128 whole", "32 cut", "128x128 1"),
    (6, 270, 2048, 2056, True): ("64 cut", "64 cut", "256x128 1"),
    (6, 270, 9600, 440, True): ("64 whole", "32 cut", "256x128 1"),
    (3, 1500, 136, 2760, True): ("32 cut", "256 whole", "128x128 1"),
    (5, 450, 136, 2504, True): ("32 cut", "128 whole", "128x128 1"),
    (6, 270, 136, 2200, True): ("few", "64 whole", "128x128 1"),
    (3, 1500, 2312, 2568, True): ("128 cut", "256 cut", "256x256 1"),
    (9, 700, 2312, 904, True): ("128 whole", "32 cut", "256x128 1"),
    (3, 330, 1496, 3304, True): ("32 cut", "128 cut", "128x128 1"),
    (1, 2048, 2040, 1848, False): ("128 cut", "128 cut", "128x128 2"),
    (5, 100, 136, 2200, True): ("few", "32 whole", "128x128 1"),
    (4, 128, 16600, 512, True): ("32 whole", "32 cut", "256x128 1"),
}
FFN = {   # (E, S, H, I, ragged): gate and up, the same with 8-bit copies, down; back to gate and up, back to x; dw_down, dw_gate_up
    (3, 1500, 96, 1408, True): ("256 whole", "256 whole", "32 cut", "32 whole", "32 cut", "128x128 1", "128x128 1"),
    (3, 1500, 96, 2720, True): ("256 whole", "256 whole", "32 cut", "256 whole", "32 cut", "128x128 1", "128x128 1"),
    (3, 1500, 2720, 96, True): ("32 cut", "32 cut", "256 whole", "32 cut", "256 whole", "128x128 1", "128x128 1"),
    (5, 450, 96, 2560, True): ("128 whole", "128 whole", "32 cut", "128 whole", "32 cut", "128x128 1", "128x128 1"),
    (6, 270, 96, 2080, True): ("few", "64 whole", "few", "64 whole", "32 cut", "128x128 1", "128x128 1"),
    (6, 270, 416, 5152, True): ("64 whole", "64 whole", "few", "64 whole", "32 cut", "128x128 1", "256x128 1"),
    (6, 270, 2080, 2080, True): ("64 cut", "64 cut", "64 cut", "64 cut", "64 cut", "256x128 1", "256x128 1"),
    (1, 2600, 2880, 1120, False): ("256 cut", "256 cut", "256 whole", "32 whole", "256 whole", "128x128 2", "128x128 1"),
    (3, 330, 1504, 3296, True): ("128 cut", "128 cut", "32 cut", "128 cut", "32 cut", "128x128 1", "256x128 1"),
    (2, 700, 2592, 2720, True): ("256 cut", "256 cut", "32 cut", "32 cut", "32 cut", "128x128 1", "256x256 1"),
    (2, 700, 2592, 5024, True): ("256 whole", "256 whole", "32 cut", "256 cut", "32 cut", "256x256 1", "256x256 1"),
}


def offsets(S, E, ragged, seed, behind):
    return tp.starts(seed, S, E, behind=behind) if ragged else None


def line(kind, z8, E, S, N, K, off):
    rows = "" if off is None else " ".join(str(int(b - a)) for a, b in zip(off, off[1:]))
    return f"product {kind} {z8} {E} {S} {N} {K} {int(off is not None)} {rows}"


@pytest.fixture(scope="module")
def forms(tmp_path_factory):
    exe = str(tmp_path_factory.mktemp("forms") / "forms")
    subprocess.run([build.hipcc(), "-x", "hip", "--offload-host-only", "-O1", "-std=c++17", "-I", build.CSRC,
                    os.path.join(build.ROOT, "tests", "cpp", "product_forms.cpp"), "-o", exe], check=True)

    def ask(lines):
        r = subprocess.run([exe], input="\n".join(lines) + "\n", capture_output=True, text=True, timeout=60, check=True)
        return tuple(r.stdout.splitlines())
    return ask


def forms_of_product(ask, E, S, N, K, ragged):
    """By the offsets of the tests of whole numbers, and with those of the epilogue's test the product's again."""
    there, back = offsets(S, E, ragged, S, S // 5), offsets(S, E, ragged, S + 1, S // 5)
    got = ask([line(ACT, 0, E, S, N, K, there), line(BACK, 0, E, S, K, N, back), f"outer {E} {S} {N} {K}"])
    epilogue = offsets(S, E, E > 1, S, S // 7)
    return got, ask([line(ACT, 0, E, S, N, K, epilogue)])[0]


def forms_of_ffn(ask, E, S, H, I, ragged):
    off = offsets(S, E, ragged, S, S // 6)
    return ask([line(GATE, 0, E, S, I, H, off), line(GATE, 1, E, S, I, H, off), line(ACT, 0, E, S, H, I, off),
                line(GATE_BACK, 0, E, S, I, H, off), line(BACK, 0, E, S, H, 2 * I, off), f"outer {E} {S} {H} {I}",
                f"outer {E} {S} {2 * I} {H}"])


def test_sizes_take_the_forms_they_stand_for(forms):
    for size, want in PRODUCTS.items():
        got, epilogue = forms_of_product(forms, *size)
        assert got == want and (epilogue == want[0]), (size, got, epilogue)
    for size, want in FFN.items():
        assert forms_of_ffn(forms, *size) == want, (size, forms_of_ffn(forms, *size))


def test_every_form_has_a_size_of_experts_with_unequal_rows():
    every = {f"{rows} {cut}" for rows in (32, 64, 128, 256) for cut in ("whole", "cut")}
    products = {s: f for s, f in PRODUCTS.items() if s[4]}
    ffn = {s: f for s, f in FFN.items() if s[4]}
    assert every <= {f[0] for f in products.values()} and every <= {f[1] for f in products.values()}
    tiled = every - {"32 whole", "32 cut"}   # of those the sizes of test_gpu_product.py are many
    for call in (0, 1, 3):
        assert tiled <= {f[call] for f in ffn.values()}, call
    # tiles of the weights' gradients in both directions, more rows of them than go through the columns together
    for form in ("256x256 1", "256x128 1"):
        assert any(f[2] == form and s[2] > 8 * 256 and s[3] > 3 * 256 for s, f in products.items()), form


def label(size):
    return "E{}-S{}-{}x{}".format(*size)


sized = pytest.mark.parametrize("size", PRODUCTS, ids=label)


@pytest.mark.gpu
@sized
@pytest.mark.parametrize("name", DTYPES)
def test_product_of_whole_numbers(torch, size, name):  # noqa: F811
    tp.test_product_of_whole_numbers(torch, *size, name)


@pytest.mark.gpu
@sized
@pytest.mark.parametrize("name", DTYPES)
def test_product_backward_of_whole_numbers(torch, size, name):  # noqa: F811
    tp.test_product_backward_of_whole_numbers(torch, *size, name)


@pytest.mark.gpu
@sized
@pytest.mark.parametrize("name,act", [("f16", "gelu"), ("bf16", "silu")])
def test_product_epilogue(torch, size, name, act):  # noqa: F811
    """Bias, activation, residual and kept sum behind whole tiles and behind joined parts."""
    tp.test_product_epilogue(torch, *size[:4], name, act)


@pytest.mark.gpu
@pytest.mark.parametrize("size", [(9, 700, 2312, 904), (3, 1500, 136, 2760), (6, 270, 2048, 2056)], ids=label)
@pytest.mark.parametrize("name,act", [("f16", "gelu"), ("bf16", "silu")])
def test_product_backward_through_the_activation(torch, size, name, act):  # noqa: F811
    tp.test_product_backward_through_the_activation(torch, *size, name, act)


@pytest.mark.gpu
@pytest.mark.parametrize("size", FFN, ids=label)
@pytest.mark.parametrize("name,act", [("f16", "gelu"), ("bf16", "silu")])
def test_ffn(torch, size, name, act):  # noqa: F811
    tp.test_ffn(torch, *size, name, act)


@pytest.mark.gpu
@pytest.mark.parametrize("size", FFN, ids=label)
@pytest.mark.parametrize("name,act,eight", [("f16", "silu", False), ("bf16", "gelu", True)])
def test_ffn_backward(torch, size, name, act, eight):  # noqa: F811
    tp.test_ffn_backward(torch, *size, name, eight, act)
