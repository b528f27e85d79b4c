"""Scored attention of more rows than the scores' grid can have: refused before anything is launched."""
import ctypes

import pytest

pytestmark = pytest.mark.gpu


def test_more_rows_than_a_grid():
    import torch
    import dense_linear_projection_gb300 as dlp
    heads, sequences, dim, page = 1 << 26, 32, 16, 16
    desc = dlp.KvDesc(1, 0, 0, 16, sequences, page, heads, heads, dim, dlp.PROJ_BF16)
    h = dlp.proj_kv_create(desc, None)
    try:
        # Memory that no kernel would have room in: it is never reached.
        some = torch.full((64,), 7.0, device="cuda")
        p = ctypes.c_void_p(some.data_ptr())
        out = torch.full((64,), 3.0, device="cuda", dtype=torch.bfloat16)
        L = dlp.lib()
        status = L.proj_kv_attend_scored(h, sequences, p, heads * dim, p, p, None, None, p, 1, p, 0, 1.0, p, p, page, p,
                                         ctypes.c_void_p(out.data_ptr()), heads * dim, None, None)
        assert status == dlp.PROJ_ERR_UNSUPPORTED
        torch.cuda.synchronize()
        assert bool((some == 7.0).all()) and bool((out == 3.0).all())
        assert dlp.proj_kv_device_status(h) == dlp.PROJ_OK
    finally:
        dlp.proj_kv_destroy(h)
