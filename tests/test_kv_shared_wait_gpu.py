"""Attention behind a shared prefix when a bounded wait runs out (PROJ_FAULT=wait<n>, read once per process:
in a handle's first such call every block waits at its n-th tile for a barrier that nobody arrives on).  The
kernel gives up by itself, with its copies and products landed: the call returns, the status tells once,
the rows that were not computed are NaN, and the handle's next call is right."""
import json
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CHILD = r"""
import json, sys, torch
sys.path.insert(0, "tests")
import dense_linear_projection_gb300 as dlp
import kv_util as ku
from test_kv_shared_gpu import case, shared64

result = []
for prefix_len, lens, heads, kv_heads, dim, page, dtype in json.loads(sys.argv[1]):
    kv, q, prefix, table, n, scales = case(prefix_len, lens, heads, kv_heads, dim, page, dtype=dtype)
    ref = shared64(q, kv.k_cache, kv.v_cache, prefix, prefix_len, table, lens, page, dim ** -0.5, *scales)
    r = {}
    out, lse = kv.attend_shared(q, prefix, prefix_len, table, n, return_lse=True)
    r["gave_up"] = [kv.status(), kv.status()]
    for _ in range(2):  # the next ones: right, in the same memory
        out, lse = kv.attend_shared(q, prefix, prefix_len, table, n, return_lse=True)
        r["after"] = kv.status()
        ku.check_attention(out, lse, ref)
    result.append(r)
print("RESULT " + json.dumps(result))
"""

CASES = [(prefix_len, lens, 8, 2, dim, page, dtype)
         for prefix_len, lens in ((1, [0, 3]), (1000, [5, 0, 130]), (40000, [9] * 20))
         for dim in (64, 128, 256) for page, dtype in ((16, "bf16"), (3, "bf16"), (16, "e4m3"), (17, "e4m3"))]


# An earlier call's results in the memory that the workspace comes from: other values, as plausible.
STALE = r"""
import json, sys, torch
sys.path.insert(0, "tests")
import dense_linear_projection_gb300 as dlp
import kv_util as ku
from test_kv_shared_gpu import case, shared64

result = []
for prefix_len, lens, heads, kv_heads, dim, page, dtype in json.loads(sys.argv[1]):
    kv, q, prefix, table, n, scales = case(prefix_len, lens, heads, kv_heads, dim, page, dtype=dtype)
    before, _, lim, lim_lse = shared64(q, kv.k_cache, kv.v_cache, prefix, prefix_len, table, lens, page, dim ** -0.5, *scales)
    kv.attend_shared(-q, prefix, prefix_len, table, n)   # gives up
    kv.attend_shared(-q, prefix, prefix_len, table, n)
    assert kv.status() == dlp.PROJ_ERR_DEVICE_TIMEOUT
    late = dlp.PagedKV(kv.k_cache, kv.v_cache, heads, len(lens), k_scale=scales[0], v_scale=scales[1])
    out, lse = late.attend_shared(q, prefix, prefix_len, table, n, return_lse=True)  # gives up
    assert late.status() == dlp.PROJ_ERR_DEVICE_TIMEOUT
    good, good_lse = late.attend_shared(q, prefix, prefix_len, table, n, return_lse=True)
    assert late.status() == dlp.PROJ_OK
    # Each row is the right one, bit for bit, or NaN.
    nan = out.isnan().all(-1)
    assert torch.equal(nan, out.isnan().any(-1)) and torch.equal(nan, lse.isnan())
    assert torch.equal(out[~nan], good[~nan]) and torch.equal(lse[~nan], good_lse[~nan]) and not good.isnan().any()
    result.append(int(nan.sum()) / nan.numel())
print("RESULT " + json.dumps(result))
"""


def child(cases, fault, code=CHILD):
    import dense_linear_projection_gb300 as dlp
    dlp.build()
    env = {k: v for k, v in os.environ.items() if k != "PROJ_FAULT"}
    if fault:
        env["PROJ_FAULT"] = fault
    r = subprocess.run([sys.executable, "-c", code, json.dumps(cases)], cwd=ROOT, env=env, capture_output=True, text=True, timeout=300)
    lines = [x for x in r.stdout.splitlines() if x.startswith("RESULT ")]
    assert r.returncode == 0 and lines, r.stdout + r.stderr
    return json.loads(lines[-1][7:])


@pytest.mark.parametrize("place", [0, 1, 4])
def test_gives_up_and_goes_on(place):
    # Blocks with fewer tiles are done as ever; a prefix of one token or of 1000 has one tile a block.
    import dense_linear_projection_gb300 as dlp
    for case, r in zip(CASES, child(CASES, f"wait{place}")):
        gives_up = place == 0 or case[0] == 40000
        assert r == {"gave_up": [dlp.PROJ_ERR_DEVICE_TIMEOUT if gives_up else dlp.PROJ_OK, dlp.PROJ_OK], "after": dlp.PROJ_OK}, case


@pytest.mark.parametrize("place", [0, 2])
def test_rows_that_were_not_computed_are_nan(place):
    # At the first tile every row lacks something, and so does every row whose tiles are shared by blocks
    # of more; five row tiles a key head, of 313 or 625 tiles each.
    cases = [(40000, [9] * 160, 8, 2, dim, page, dtype) for dim in (64, 128, 256) for page, dtype in ((16, "bf16"), (3, "bf16"), (16, "e4m3"))]
    assert child(cases, f"wait{place}", STALE) == [1.0] * len(cases)
    if place == 0:
        assert child([CASES[i] for i in range(0, len(CASES), 3)], "wait0", STALE) == [1.0] * -(-len(CASES) // 3)


def test_nothing_is_injected_without_the_variable():
    import dense_linear_projection_gb300 as dlp
    for case, r in zip(CASES[:4], child(CASES[:4], "")):
        assert r == {"gave_up": [dlp.PROJ_OK, dlp.PROJ_OK], "after": dlp.PROJ_OK}, case


def test_what_else_was_found_is_told_after_the_wait():
    import dense_linear_projection_gb300 as dlp
    code = CHILD[:CHILD.index("result = []")] + r"""
kv, q, prefix, table, n, _ = case(1000, [20, 20], 8, 2, 64, 16)
table[0, 1] = -1
kv.attend_shared(q, prefix, 1000, table, n)
print("RESULT " + json.dumps([kv.status() for _ in range(3)]))
"""
    assert child([], "wait0", code) == [dlp.PROJ_ERR_DEVICE_TIMEOUT, dlp.PROJ_ERR_INVALID_ARG, dlp.PROJ_OK]
