"""Rows that are not 16-byte aligned: no read outside the caller's matrix (on the CPU), and
the block norms' values on matrices whose rows lie less than 16 bytes apart (on a GB300)."""

import os
import subprocess

import pytest

import ops64

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_reads_stay_inside_the_matrix(tmp_path):
    exe = os.path.join(str(tmp_path), "granules_check")
    subprocess.run(["g++", "-std=c++17", "-O1", "-I",
                    os.path.join(ROOT, "tiled_fp16_gemm_gb300", "csrc"),
                    os.path.join(ROOT, "tests", "granules_check.cpp"), "-o", exe], check=True)
    r = subprocess.run([exe], capture_output=True, text=True)
    assert r.returncode == 0 and r.stdout.strip() == "OK", r.stdout


@pytest.mark.gpu
@pytest.mark.parametrize("cols", [1, 2, 3, 5, 7])
@pytest.mark.parametrize("dtype,stream", [("float16", "float16"), ("bfloat16", "float32"),
                                          ("float32", "float32")])
@pytest.mark.parametrize("gates", [1, 12])
def test_narrow_rows_behind_an_offset(cols, dtype, stream, gates):
    torch = pytest.importorskip("torch")
    from tiled_fp16_gemm_gb300 import build
    build.build()
    import tiled_fp16_gemm_gb300 as tg
    rows, dtype, stream = 12, getattr(torch, dtype), getattr(torch, stream)
    g = torch.Generator(device="cuda").manual_seed(cols)

    def mat(r, kind, offset):
        whole = torch.full((offset + r * cols + 8,), float("nan"), device="cuda", dtype=kind)
        view = whole[offset:offset + r * cols].view(r, cols)
        return view.copy_(torch.randn(r, cols, generator=g, device="cuda"))

    for offset in (1, 2, 3):
        x, r = mat(rows, dtype, offset), mat(rows, stream, offset)
        kept = dict(residual=r, post_weight=1 + 0.2 * torch.randn(cols, device="cuda"),
                    gate=mat(gates, dtype, offset), scale=0.7,
                    pre_weight=1 + 0.2 * torch.randn(cols, device="cuda"), eps=1e-5)
        dy, dh = mat(rows, stream, offset), mat(rows, dtype, offset)
        ref = ops64.Norm(x, **kept)
        ref.check(*tg.norm_residual(x, **kept), f"{cols} {offset}")
        ref.check_grads(tg.norm_residual_backward(dy, dh, x, **kept), dy, dh, f"{cols} {offset}")
