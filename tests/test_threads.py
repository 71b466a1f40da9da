"""Calls from several host threads on one stream: each is right, as if made alone.

An operator of more than one launch hands its intermediate results from one to the next in
the stream's workspace, so no other call's launch may come between them.
"""

import os
import subprocess
import threading

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_a_call_holds_its_workspace(tmp_path):
    from tiled_fp16_gemm_gb300 import build
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(build._nvcc())))
    exe = os.path.join(str(tmp_path), "workspace_check")
    subprocess.run(["g++", "-std=c++17", "-O1", "-pthread", "-I", build.CSRC, "-I", build.INCLUDE,
                    "-I", os.path.join(cuda, "include"),
                    os.path.join(ROOT, "tests", "workspace_check.cpp"), "-o", exe], check=True)
    r = subprocess.run([exe], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == "OK", r.stdout


@pytest.fixture(scope="module")
def tg():
    from tiled_fp16_gemm_gb300 import build
    build.build()
    import tiled_fp16_gemm_gb300 as t
    return t


def in_threads(calls, reps):
    """Each of ``calls`` ``reps`` times in a thread of its own; raises what one raised."""
    start, errors = threading.Barrier(len(calls)), []

    def run(call):
        try:
            start.wait()
            for i in range(reps):
                call(i)
        except Exception as e:  # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=run, args=(c,)) for c in calls]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    if errors:
        raise errors[0]


@pytest.mark.gpu
@pytest.mark.parametrize("M,N,K,reps", [(40, 4096, 4096, 1000), (100, 2048, 2048, 1000), (4096, 512, 2048, 200)])
def test_products_of_two_threads(tg, M, N, K, reps):
    import torch
    stream = torch.cuda.Stream()
    g = torch.Generator(device="cuda").manual_seed(M)
    bq = torch.randint(0, 256, (N, K // 2), generator=g, device="cuda", dtype=torch.uint8)
    scale = torch.full((K // 64, N), 0.01, device="cuda", dtype=torch.half)
    calls, results, wanted = [], [], []
    for _ in range(2):
        a = torch.randn(M, K, generator=g, device="cuda").half()
        wanted.append(tg.gemm_w4(a, bq, scale, N, 64))
        out = torch.zeros(min(reps, 300), M, N, device="cuda", dtype=torch.half)
        results.append(out)
        # (a stream is given: this way through the binding lets other threads run)
        calls.append(lambda i, a=a, out=out: tg.gemm_w4(a, bq, scale, N, 64, out=out[i % len(out)],
                                                        stream=stream))
    torch.cuda.synchronize()
    in_threads(calls, reps)
    torch.cuda.synchronize()
    tg.sync_status()
    for out, want in zip(results, wanted):
        assert torch.equal(out, want.expand_as(out))


@pytest.mark.gpu
def test_gradients_of_two_threads(tg):
    import torch
    stream = torch.cuda.Stream()
    g = torch.Generator(device="cuda").manual_seed(7)
    mat = lambda: torch.randn(64, 512, generator=g, device="cuda")  # noqa: E731
    w = 1 + 0.1 * torch.randn(512, generator=g, device="cuda")
    calls, got, wanted = [], [], []
    for _ in range(2):
        x, r, dy, dh = mat(), mat(), mat(), mat()
        kept = dict(post_weight=w, pre_weight=w)
        wanted.append(tg.norm_residual_backward(dy, dh, x, r, **kept))
        mine = []
        got.append(mine)
        calls.append(lambda i, t=(dy, dh, x, r), kept=kept, mine=mine: mine.append(
            tg.norm_residual_backward(*t, **kept, stream=stream)))
    torch.cuda.synchronize()
    in_threads(calls, 1000)
    torch.cuda.synchronize()
    tg.sync_status()
    for mine, want in zip(got, wanted):
        assert len(mine) == 1000
        for grads in mine:
            for a, b in zip(grads, want):
                assert (a is None) == (b is None) and (a is None or torch.equal(a, b))


@pytest.mark.gpu
@pytest.mark.parametrize("M,N,K,mx", [(200, 512, 1032, False), (40, 512, 1032, False), (200, 512, 1024, True),
                                      (40, 512, 1024, True)])
def test_staged_products_of_two_threads(tg, M, N, K, mx):
    """Rows of A off 16 bytes go through the stream's staging buffer; MXFP4 weights for many
    rows of A through its decoded weights."""
    import torch
    stream = torch.cuda.Stream()
    g = torch.Generator(device="cuda").manual_seed(M + K)
    calls, results, wanted = [], [], []
    for _ in range(2):
        a = torch.randn(M, K + 1, generator=g, device="cuda").half()[:, :K]
        if mx:
            bq = torch.randint(0, 256, (N, K // 2), generator=g, device="cuda", dtype=torch.uint8)
            scale = torch.full((K // 32, N), 120, device="cuda", dtype=torch.uint8)
            call = lambda a=a, bq=bq, scale=scale, **kw: tg.gemm_mxfp4(a, bq, scale, N, **kw)  # noqa: E731
        else:
            b = torch.randn(K, N, generator=g, device="cuda").half()
            call = lambda a=a, b=b, **kw: tg.gemm(a, b, **kw)  # noqa: E731
        wanted.append(call())
        out = torch.zeros(300, M, N, device="cuda", dtype=torch.half)
        results.append(out)
        calls.append(lambda i, call=call, out=out: call(out=out[i % 300], stream=stream))
    torch.cuda.synchronize()
    in_threads(calls, 600)
    torch.cuda.synchronize()
    tg.sync_status()
    for out, want in zip(results, wanted):
        assert torch.equal(out, want.expand_as(out))


PER_THREAD = 2  # cudaStreamPerThread: one handle, a stream for each thread


@pytest.mark.gpu
@pytest.mark.parametrize("M,N,K", [(16, 512, 8192), (40, 512, 1031), (2048, 2048, 1024)])
def test_products_on_the_threads_own_streams(tg, M, N, K):
    """Streams of two threads overlap, though their handle is the same: each has buffers of its
    own (partial sums of k-pieces, staged operands)."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(M + K)
    calls, results, wanted = [], [], []
    for _ in range(2):
        a = torch.randn(M, K, generator=g, device="cuda").half()
        b = torch.randn(K, N, generator=g, device="cuda").half()
        wanted.append(tg.gemm(a, b))
        out = torch.zeros(50, M, N, device="cuda", dtype=torch.half)
        results.append(out)

        def call(i, a=a, b=b, out=out):
            st = tg.tg_gemm_f16(a.data_ptr(), b.data_ptr(), out[i % 50].data_ptr(), M, N, K, K, N, N, 0, PER_THREAD)
            assert st == tg.TG_OK

        calls.append(call)
    torch.cuda.synchronize()
    in_threads(calls, 500)
    torch.cuda.synchronize()
    tg.sync_status()
    for out, want in zip(results, wanted):
        assert torch.equal(out, want.expand_as(out))


@pytest.mark.gpu
def test_host_products_on_the_threads_own_streams(tg):
    import numpy as np
    import torch
    M, N, K = 64, 1500, 512
    calls, results, wanted = [], [], []
    for seed in range(2):
        r = np.random.RandomState(seed)
        a, b = (r.uniform(-1, 1, s).astype(np.float16) for s in ((M, K), (K, N)))
        wanted.append(tg.gemm(torch.from_numpy(a).cuda(), torch.from_numpy(b).cuda()).cpu().numpy())
        out = np.zeros((20, M, N), np.float16)
        results.append(out)

        def call(i, a=a, b=b, out=out):
            c = out[i % 20]
            st = tg.tg_gemm_f16_host(a.ctypes.data, b.ctypes.data, c.ctypes.data, M, N, K, K, N, N, 0, PER_THREAD)
            assert st == tg.TG_OK

        calls.append(call)
    in_threads(calls, 100)
    torch.cuda.synchronize()
    tg.sync_status()
    for out, want in zip(results, wanted):
        assert all(np.array_equal(c, want) for c in out)
