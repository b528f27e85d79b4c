"""The decode-step operators' host side, without a GPU: sizes, refusals before any device call."""
import ctypes

import pytest

import dense_linear_projection_gb300 as dlp


def test_packed_bytes():
    # 64-row tiles and 64-wide blocks of half-byte codes, bf16 scales, half-byte zero points.
    assert dlp.proj_q4_packed_bytes(64, 64, 64) == 64 * 32 + 64 * 2
    assert dlp.proj_q4_packed_bytes(64, 128, 128, True) == 64 * 64 + 64 * 2 + 32
    assert dlp.proj_q4_packed_bytes(65, 32, 32) == 2 * (64 * 32 + 2 * 64 * 2)  # padded to whole tiles and blocks
    assert dlp.proj_q4_packed_bytes(0, 64, 64) == dlp.proj_q4_packed_bytes(64, 0, 64) == 0
    for args, status in [((64, 64, 16), dlp.PROJ_ERR_UNSUPPORTED), ((64, 100, 64), dlp.PROJ_ERR_INVALID_ARG),
                         ((-1, 64, 64), dlp.PROJ_ERR_INVALID_ARG)]:
        with pytest.raises(dlp.ProjError) as e:
            dlp.proj_q4_packed_bytes(*args)
        assert e.value.status == status


@pytest.mark.parametrize("change,status", [
    (dict(kv_dtype=dlp.PROJ_F32), dlp.PROJ_ERR_UNSUPPORTED),
    (dict(head_dim=40), dlp.PROJ_ERR_UNSUPPORTED),
    (dict(head_dim=512), dlp.PROJ_ERR_UNSUPPORTED),
    (dict(q_heads=9), dlp.PROJ_ERR_INVALID_ARG),
    (dict(page_size=0), dlp.PROJ_ERR_INVALID_ARG),
    (dict(kv_heads=0), dlp.PROJ_ERR_INVALID_ARG),
    (dict(max_sequences=-1), dlp.PROJ_ERR_INVALID_ARG),
    (dict(token_stride=132), dlp.PROJ_ERR_MISALIGNED),
])
def test_cache_geometry_refusals(change, status):
    good = dict(num_pages=4, page_stride=16 * 128, token_stride=128, head_stride=64, max_sequences=2, page_size=16,
                q_heads=8, kv_heads=2, head_dim=64, kv_dtype=dlp.PROJ_BF16)
    with pytest.raises(dlp.ProjError) as e:
        dlp.proj_kv_create(dlp.KvDesc(**{**good, **change}))
    assert e.value.status == status


def test_projection_refusals():
    for args, status in [((2097121, 64, 64, 64), dlp.PROJ_ERR_UNSUPPORTED), ((1, 64, 64, 16), dlp.PROJ_ERR_UNSUPPORTED),
                         ((1, 64, 65, 64), dlp.PROJ_ERR_INVALID_ARG), ((1, -1, 64, 64), dlp.PROJ_ERR_INVALID_ARG)]:
        with pytest.raises(dlp.ProjError) as e:
            dlp.proj_q4_create(*args)
        assert e.value.status == status


def test_null_handles():
    L = dlp.lib()
    assert L.proj_q4_run(None, 1, None, None, None, None, None) == dlp.PROJ_ERR_INVALID_ARG
    assert L.proj_q4_pack(None, None, None, None, None, None) == dlp.PROJ_ERR_INVALID_ARG
    assert L.proj_kv_create(None, None, None) == dlp.PROJ_ERR_INVALID_ARG
    assert dlp.proj_kv_device_status(None) == dlp.PROJ_ERR_INVALID_ARG
    assert L.proj_q4_destroy(None) == L.proj_kv_destroy(None) == dlp.PROJ_OK
    h = ctypes.c_void_p(1)
    assert L.proj_kv_create(ctypes.byref(h), None, None) == dlp.PROJ_ERR_INVALID_ARG and h.value is None


def test_rope_table():
    import math
    t = dlp.rope_table(5, 4, base=100.0, device="cpu")
    assert tuple(t.shape) == (5, 4)
    for p in range(5):
        for j, rate in enumerate((1.0, 0.1)):
            assert abs(t[p, j].item() - math.cos(p * rate)) < 1e-7
            assert abs(t[p, 2 + j].item() - math.sin(p * rate)) < 1e-7


def test_cluster_arrivals_are_ordered():
    # A CTA of a cluster may leave once every other has arrived: an arrival without release does not
    # order the reads of another CTA's shared memory that come before it, so no kernel has one.
    import os
    import re
    csrc = os.path.join(os.path.dirname(dlp.__file__), "csrc")
    arrivals = []
    for name in sorted(os.listdir(csrc)):
        with open(os.path.join(csrc, name), encoding="utf-8") as f:
            arrivals += [(name, m) for m in re.findall(r"barrier\.cluster\.arrive[.\w]*", f.read())]
    assert arrivals and all(m.endswith((".release", ".arrive", ".aligned")) and "relaxed" not in m for _, m in arrivals), arrivals


def test_no_loads_past_the_coherent_path():
    # The kernels may be resident while the kernel before them still writes their inputs (programmatic
    # launches): a load that takes memory for unchanging over the kernel's life is not theirs to use.
    import os
    import re
    csrc = os.path.join(os.path.dirname(dlp.__file__), "csrc")
    for name in sorted(os.listdir(csrc)):
        with open(os.path.join(csrc, name), encoding="utf-8") as f:
            assert not re.search(r"__ldg\(|ld\.global\.nc|__ldlu", f.read()), name
