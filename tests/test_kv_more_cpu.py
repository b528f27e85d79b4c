"""The paged cache's further operators, host side, without a GPU: refusals before any device call."""
import ctypes

import dense_linear_projection_gb300 as dlp


def test_null_handles():
    L, bad = dlp.lib(), dlp.PROJ_ERR_INVALID_ARG
    n = ctypes.c_size_t(7)
    none = lambda k: [None] * k  # noqa: E731
    assert L.proj_kv_shared_workspace(None, 1, 1, ctypes.byref(n)) == bad and n.value == 0
    assert L.proj_kv_scored_workspace(None, 1, 1, None) == bad
    assert L.proj_kv_scored_workspace(None, 1, 1, ctypes.byref(n)) == bad
    assert L.proj_kv_append_normed(None, 1, None, 0, None, None, 0, None, None, 0, 1e-6, None, None, None, 1, 1, None, None, 0, 0, 0,
                                   *none(5), 0, None) == bad
    assert L.proj_kv_attend_shared(None, 1, None, 0, *none(5), 1, 1, None, 1, None, 1.0, None, None, 0, None, None) == bad
    assert L.proj_kv_attend_scored(None, 1, None, 0, *none(5), 1, None, 0, 1.0, None, None, 16, None, None, 0, None, None) == bad
    assert L.proj_kv_evict(None, 1, None, 1, None, None, 16, None, 1, 1, 0, *none(6)) == bad
