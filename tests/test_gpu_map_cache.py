"""The maps of one call keep one another in the map cache, at whatever addresses, on a GB300."""

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu


def test_a_repeated_call_encodes_no_map():
    from tiled_fp16_gemm_gb300 import build
    build.build()
    import tiled_fp16_gemm_gb300 as tg
    M, N, K = 300, 504, 400
    a = torch.ones(M, K, device="cuda", dtype=torch.half)
    room = torch.zeros(3000 * 64 + K * N, device="cuda", dtype=torch.half)
    c = torch.empty(M, N, device="cuda", dtype=torch.half)
    s = torch.cuda.current_stream().cuda_stream
    again = 0
    for i in range(3000):
        b = room[64 * i:]

        def call():
            assert tg.tg_gemm_f16(a.data_ptr(), b.data_ptr(), c.data_ptr(), M, N, K, K, N, N, 0, s) == tg.TG_OK

        call()
        _, before = tg.tg_debug_map_cache_stats()
        call()
        _, after = tg.tg_debug_map_cache_stats()
        again += after - before
    tg.sync_status()
    assert again == 0
