"""Windows of any size through the C call itself (the Python layer shortens
them first): one that covers everything is no window, also for sequences with
more new tokens than the cache holds."""
import ctypes

import pytest
import torch

import tests.pagedref as ref
from tests.test_gpu_paged import BF16, E4M3, batch_of, filled, gen, on_gpu, sz

pytestmark = pytest.mark.gpu

LARGE = [1 << 20, (1 << 30) - 1, 1 << 30, (1 << 30) + 1, (1 << 31) - 64, (1 << 31) - 2, (1 << 31) - 1]


@pytest.mark.parametrize("dtype", [BF16, E4M3])
@pytest.mark.parametrize("lens,new,G", [([5, 0, 90], [16, 3, 2], 1), ([5, 40, 0], [60, 70, 20], 2), ([300], [301], 4)],
                         ids=["few", "many", "one"])
def test_windows_that_hide_nothing(dtype, lens, new, G):
    H, D, P = 2, 128, 16
    table, kv, starts, T, pages = ref.layout(lens, new, P, seed=3, gap=1)
    data, scales = filled(dtype, pages, H, P, D, 9)
    cache = on_gpu(dtype, data, scales)
    batch = batch_of(table, kv, starts, T, max_new=max(new), max_kv=max(lens))
    q = torch.randn(T, H * G, D, generator=gen(2)).to(torch.bfloat16)
    on = q.cuda()
    ws = sz().attention_workspace(cache, batch, H * G)
    from fp8_kv_cache_sz_amd import _native
    want, want_l, tol, tol_l = ref.attention(q, data, scales, table, kv, starts, P, D ** -0.5, 0)
    none = torch.ones(T, dtype=torch.bool)
    none[int(starts[0]):int(starts[-1])] = False
    want[none], want_l[none], tol[none], tol_l[none] = 3.0, 3.0, 0.0, 0.0
    for window in [0] + LARGE:
        print("window", window, flush=True)
        out = torch.full((T, H * G, D), 3.0, dtype=torch.bfloat16, device="cuda")
        lse = torch.full((T, H * G), 3.0, dtype=torch.float32, device="cuda")
        rc = _native.lib.sz_paged_attention(cache._ref, batch._ref(P), on.data_ptr(), H * G, H * G * D, D,
                                            ctypes.c_float(D ** -0.5), window, out.data_ptr(), lse.data_ptr(),
                                            ws.data_ptr(), ws.nbytes, cache.status.data_ptr(),
                                            torch.cuda.current_stream().cuda_stream)
        assert rc == 0
        cache.raise_status()
        assert not ref.close(out, want, tol), window
        assert not ref.close(lse, want_l, tol_l), window
