"""Calls on a stream of the caller's choice: what they allocate belongs to that stream.

A buffer is given back on the current stream while work that writes it is still waiting there.  A call on
another stream must not be handed its memory: the late write would land in the call's result."""
import pytest

pytestmark = pytest.mark.gpu


def check(call, like, as_handle):
    """``call(stream)`` -> tensors, next to late writes to buffers of the shapes and types of ``like``."""
    import torch
    side = torch.cuda.Stream()
    want = [x.clone() for x in call(None)]
    torch.cuda.synchronize()
    torch.cuda._sleep(50_000_000)
    for shape, dtype in like:
        late = [torch.empty(shape, dtype=dtype, device="cuda") for _ in range(3)]
        for x in late:
            x.fill_(3)
        del late, x
    got = call(side.cuda_stream if as_handle else side)
    side.synchronize()
    torch.cuda.synchronize()
    for x, y in zip(got, want):
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))
    # The default stream, by its handle: the current one here.
    for x, y in zip(call(0), want):
        torch.cuda.synchronize()
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))


@pytest.mark.parametrize("as_handle", [False, True])
def test_projections(as_handle):
    import torch
    import dense_linear_projection_gb300 as dlp
    M, N, K = 16, 4096, 1024
    X = torch.randn((M, K), device="cuda").to(torch.bfloat16)
    codes = torch.randint(0, 256, (N, K // 2), device="cuda", dtype=torch.uint8)
    scales = torch.rand((N, K // 64), device="cuda").to(torch.bfloat16)
    q4 = dlp.Q4Projection(M, N, K, 64)
    packed = q4.pack(codes, scales)
    check(lambda s: [q4(X, packed, stream=s)], [((M, N), torch.bfloat16)], as_handle)
    check(lambda s: [q4.pack(codes, scales, stream=s)], [(packed.shape, torch.uint8)], as_handle)
    W = torch.randn((N, K), device="cuda").to(torch.bfloat16)
    proj = dlp.Projection(M, N, K)
    P = proj.pack(W)
    check(lambda s: [proj(X, P, packed=True, stream=s)], [((M, N), torch.bfloat16)], as_handle)
    check(lambda s: [proj.pack(W, stream=s)], [(P.shape, torch.bfloat16)], as_handle)


@pytest.mark.parametrize("as_handle", [False, True])
def test_paged_cache(as_handle):
    import torch
    import dense_linear_projection_gb300 as dlp
    B, H, hk, D, page = 40, 16, 4, 128, 16
    bf16 = torch.bfloat16
    k_cache, v_cache = (torch.randn((B * 4, page, hk, D), device="cuda").to(bf16) for _ in "kv")
    kv = dlp.PagedKV(k_cache, v_cache, H, B)
    table = torch.randperm(B * 4, device="cuda").to(torch.int32).view(B, 4)
    rows = torch.randn((B, H + 2 * hk, D), device="cuda").to(bf16)
    pos = torch.arange(B, device="cuda").to(torch.int32)
    lens, rope = pos + 1, dlp.rope_table(64, D)
    check(lambda s: [kv.append(rows[:, :H], rows[:, H:H + hk], rows[:, H + hk:], pos, table, rope=rope, stream=s)],
          [((B, H, D), bf16)], as_handle)
    q = rows[:, :H].contiguous()
    check(lambda s: kv.attend(q, table, lens, return_lse=True, stream=s), [((B, H, D), bf16), ((B, H), torch.float32)], as_handle)


def test_projection_status_waits_for_the_current_stream():
    import torch
    import dense_linear_projection_gb300 as dlp
    X, W = (torch.randn(s, device="cuda").to(torch.bfloat16) for s in ((16, 1024), (2048, 1024)))
    proj = dlp.Projection(16, 2048, 1024)
    torch.cuda.synchronize()
    done = torch.cuda.Event()
    with torch.cuda.stream(torch.cuda.Stream()):
        torch.cuda._sleep(100_000_000)
        proj(X, W)
        done.record()
        assert proj.status() == dlp.PROJ_OK and done.query()
