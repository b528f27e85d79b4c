"""Host-side fault injection (PROJ_FAULT, read once per process) at the paged cache's further entry
points: each failure becomes its status, nothing leaks, and the context stays usable.  The failure is
made on the host, before anything reaches the device."""
import json
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CHILD = r"""
import hashlib, json, torch
import dense_linear_projection_gb300 as dlp
bf16, dev = torch.bfloat16, "cuda"
torch.manual_seed(5)
k, v = (torch.randn((24, 16, 2, 64), device=dev).to(bf16) for _ in "kv")
rows = torch.randn((2, 8, 64), device=dev).to(bf16)
ints = torch.tensor([20, 5], dtype=torch.int32, device=dev)
table = torch.arange(4, dtype=torch.int32, device=dev).view(2, 2)
prefix = torch.arange(4, 16, dtype=torch.int32, device=dev)
to = torch.arange(16, 18, dtype=torch.int32, device=dev).view(2, 1)
w = torch.ones(64, device=dev)
digest = {}


def status(name, f):
    try:
        r = f()
        r = r if isinstance(r, tuple) else (r,)
        torch.cuda.synchronize()
        digest[name] = hashlib.sha256(b"".join(t.cpu().contiguous().view(torch.uint8).numpy().tobytes() for t in r)).hexdigest()
        return 0
    except dlp.ProjError as e:
        return e.status


def scenario():
    out = {}
    kv = []
    out["create"] = status("create", lambda: (kv.append(dlp.PagedKV(k, v, 4, 2)), ints)[1])
    if kv:
        scores = torch.arange(128, device=dev).float().view(2, 2, 32) / 7
        out["append"] = status("append", lambda: kv[0].append(rows[:, :4], rows[:, 4:6], rows[:, 6:], ints, table, q_norm=w, k_norm=w))
        out["shared"] = status("shared", lambda: kv[0].attend_shared(rows[:, :4], prefix, 180, table, ints))
        out["scored"] = status("scored", lambda: kv[0].attend_scored(rows[:, :4], table, ints, scores))
        out["evict"] = status("evict", lambda: kv[0].evict(table, ints, scores, to, 10, 2))
        out["status"] = kv[0].status()
        kv[0].close()
    torch.cuda.synchronize()
    return out


first = scenario()
torch.cuda.empty_cache()
free = torch.cuda.mem_get_info()[0]
for _ in range(3):
    assert scenario() == first
torch.cuda.empty_cache()
first["leak"] = max(0, free - torch.cuda.mem_get_info()[0])
first["alive"] = (torch.ones(10, device=dev) * 2).sum().item() == 20.0
first["digest"] = digest
print("RESULT " + json.dumps(first))
"""


def child(fault):
    import dense_linear_projection_gb300 as dlp
    dlp.build()
    env = {k: v for k, v in os.environ.items() if k != "PROJ_FAULT"}
    if fault:
        env["PROJ_FAULT"] = fault
    r = subprocess.run([sys.executable, "-c", CHILD], cwd=ROOT, env=env, capture_output=True, text=True, timeout=300)
    lines = [x for x in r.stdout.splitlines() if x.startswith("RESULT ")]
    assert r.returncode == 0 and lines, r.stdout + r.stderr
    got = json.loads(lines[-1][7:])
    assert got.pop("alive") and got.pop("leak") == 0
    return got, got.pop("digest")


def test_faults():
    import dense_linear_projection_gb300 as dlp
    calls = ("append", "shared", "scored", "evict")
    good, digest = child("")
    assert set(good.values()) == {dlp.PROJ_OK}
    got, _ = child("launch")
    assert {k: got[k] for k in calls} == {k: dlp.PROJ_ERR_CUDA for k in calls} and got["create"] == got["status"] == dlp.PROJ_OK
    got, _ = child("alloc")
    assert got == {"create": dlp.PROJ_ERR_OUT_OF_MEMORY}
    got, _ = child("device")  # every handle is another device's
    assert {k: got[k] for k in calls} == {k: dlp.PROJ_ERR_INVALID_ARG for k in calls} and got["create"] == dlp.PROJ_OK
    # Without tensor maps the prefix comes by plain copies: the same bits.
    got, other = child("encode")
    assert got == good and other == digest
