"""The 4-bit projection against its definition in 64 bits.

Bound of |Y − exact|: the products of bf16 X with the integers q − z are exact in fp32; every
fp32 sum (inside a tensor-core step, between steps, over groups and over split parts) rounds or
truncates by at most 2⁻²² of the absolute sum S = Σ_k |x|·s·|q − z| so far, and there are at most
K/16 steps, K/32 groups and 64 joins: (K/16 + K/32 + 64)·2⁻²²·S, S with the bias.  A bf16 output
has to lie between the rounded ends of that interval (kv_util.beyond)."""
import math

import pytest

from kv_util import beyond

pytestmark = pytest.mark.gpu


def stored(N, K, group, zeros, seed, device="cuda"):
    import torch
    g = torch.Generator(device=device)
    g.manual_seed(seed)
    codes = torch.randint(0, 256, (N, K // 2), generator=g, device=device, dtype=torch.uint8)
    scales = ((torch.rand((N, K // group), generator=g, device=device) - 0.3) * 0.02).to(torch.bfloat16)
    z = torch.randint(0, 16, (N, K // group), generator=g, device=device, dtype=torch.uint8) if zeros else None
    return codes, scales, z


def dequantised(codes, scales, z, group):
    """[N, K] in 64 bits."""
    import torch
    N, K = codes.shape[0], codes.shape[1] * 2
    q = torch.empty((N, K), dtype=torch.float64, device=codes.device)
    q[:, 0::2] = (codes & 15).double()
    q[:, 1::2] = (codes >> 4).double()
    zero = z.double().repeat_interleave(group, 1) if z is not None else 8.0
    return (q - zero) * scales.double().repeat_interleave(group, 1)


def check(Y, X, W, bias, what=""):
    import torch
    K = X.shape[1]
    ref = X.double() @ W.t()
    S = X.double().abs() @ W.abs().t()
    if bias is not None:
        ref = ref + bias.double()
        S = S + bias.double().abs()
    lim = (K / 16 + K / 32 + 64) * 2.0 ** -22 * S
    assert torch.isfinite(Y).all(), what
    over = beyond(Y, ref, lim)
    assert (over <= 0).all(), f"{what}: {int((over > 0).sum())} of {Y.numel()} beyond the bound, by up to {over.max().item():.3e}"


def run(M, N, K, group, zeros, bias, f32, seed=1, max_tokens=None):
    import torch
    import dense_linear_projection_gb300 as dlp
    codes, scales, z = stored(N, K, group, zeros, seed)
    X = torch.randn((M, K), device="cuda").to(torch.bfloat16)
    b = torch.randn(N, device="cuda").to(torch.bfloat16) if bias else None
    proj = dlp.Q4Projection(max_tokens or M, N, K, group, has_zeros=zeros,
                            y_dtype=dlp.PROJ_F32 if f32 else dlp.PROJ_BF16, has_bias=bias)
    P = proj.pack(codes, scales, z)
    return proj, P, X, b, dequantised(codes, scales, z, group)


@pytest.mark.parametrize("M,N,K,group,zeros,bias,f32", [
    (1, 1, 32, 32, False, False, True),
    (1, 64, 64, 64, True, False, False),
    (2, 17, 96, 32, True, True, True),       # K ends inside a block of 64, N inside a tile
    (7, 65, 128, 128, False, True, False),
    (8, 63, 256, 64, True, False, True),
    (9, 1000, 4128, 32, False, True, False),
    (16, 2048, 1024, 128, True, False, True),
    (17, 130, 8192, 64, True, True, False),
    (31, 4099, 1056, 32, True, False, True),
    (32, 512, 2048, 128, False, False, False),
    (33, 200, 640, 128, True, True, True),   # a second pass over the weights
    (100, 333, 512, 64, True, True, False),
    (1, 2048, 8192, 128, False, False, True),
    (4, 28672, 1024, 128, True, False, False),
    (1, 20000, 64, 32, True, False, True),   # many rows, one block of K
    (3, 16, 65536, 64, True, False, True),   # few rows, long K
])
def test_against_64_bits(M, N, K, group, zeros, bias, f32):
    import torch
    proj, P, X, b, W = run(M, N, K, group, zeros, bias, f32)
    Y = proj(X, P, b)
    check(Y, X, W, b, f"M={M} N={N} K={K} group={group}")
    assert torch.equal(proj(X, P, b), Y)  # bit for bit


def test_every_token_count_up_to_two_passes():
    # One handle for all of them, and nothing of one run left for the next.
    proj, P, X, b, W = run(66, 208, 1184, 32, True, True, True)
    for M in list(range(1, 35)) + [63, 64, 65, 66]:
        check(proj(X[:M].contiguous(), P, b), X[:M], W, b, f"M={M}")


def test_exact_small_integers():
    # Scale 1, integer X: every sum is an integer below 2²⁴ and comes out exactly.
    import torch
    import dense_linear_projection_gb300 as dlp
    M, N, K = 5, 77, 512
    codes, _, z = stored(N, K, 64, True, 3)
    scales = torch.ones((N, K // 64), device="cuda", dtype=torch.bfloat16)
    X = torch.randint(-8, 9, (M, K), device="cuda").to(torch.bfloat16)
    proj = dlp.Q4Projection(M, N, K, 64, has_zeros=True, y_dtype=dlp.PROJ_F32)
    Y = proj(X, proj.pack(codes, scales, z))
    assert torch.equal(Y.double(), X.double() @ dequantised(codes, scales, z, 64).t())


def test_each_weight_position():
    # One-hot rows of X pick single weights: every code, scale and zero lies where it belongs.
    import torch
    import dense_linear_projection_gb300 as dlp
    N, K = 80, 96
    codes, scales, z = stored(N, K, 32, True, 5)
    proj = dlp.Q4Projection(K, N, K, 32, has_zeros=True, y_dtype=dlp.PROJ_F32)
    Y = proj(torch.eye(K, device="cuda").to(torch.bfloat16), proj.pack(codes, scales, z))
    assert torch.equal(Y.double(), dequantised(codes, scales, z, 32).t())


def test_empty_sums_and_empty_shapes():
    import torch
    import dense_linear_projection_gb300 as dlp
    b = torch.randn(50, device="cuda").to(torch.bfloat16)
    proj = dlp.Q4Projection(3, 50, 0, 64, has_bias=True, y_dtype=dlp.PROJ_F32)
    X = torch.empty((3, 0), device="cuda", dtype=torch.bfloat16)
    P = proj.pack(torch.empty((50, 0), device="cuda", dtype=torch.uint8),
                  torch.empty((50, 0), device="cuda", dtype=torch.bfloat16))
    assert torch.equal(proj(X, P, b), b.float().expand(3, 50))
    proj = dlp.Q4Projection(3, 50, 0, 64)
    assert (proj(X, P) == 0).all()
    proj, P, X, b, _ = run(4, 32, 64, 32, False, False, False)
    assert proj(X[:0], P).shape == (0, 32)


def test_code_offsets_past_31_bits():
    # 2.1 GB of codes: the last rows' offsets do not fit 31 bits.
    import torch
    import dense_linear_projection_gb300 as dlp
    N, K = 131072 + 40, 32768
    codes, scales, _ = stored(N, K, 128, False, 9)
    proj = dlp.Q4Projection(2, N, K, 128, y_dtype=dlp.PROJ_F32)
    P = proj.pack(codes, scales)
    X = torch.randn((2, K), device="cuda").to(torch.bfloat16)
    Y = proj(X, P)
    for rows in (slice(0, 200), slice(N - 300, N)):
        check(Y[:, rows], X, dequantised(codes[rows], scales[rows], None, 128), None, str(rows))


def test_streams_and_graphs():
    import torch
    proj, P, X, b, W = run(6, 520, 2048, 128, True, True, True)
    ref = proj(X, P, b)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        Y = proj(X * 1, P, b)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(Y, ref)
    g, out = torch.cuda.CUDAGraph(), torch.empty_like(ref)
    X2 = X.clone()
    with torch.cuda.graph(g):
        proj(X2, P, b, out=out)
    X2.copy_(X.flip(0))
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, ref.flip(0))


def test_infinities_and_nan_stay_in_their_rows():
    import torch
    proj, P, X, b, W = run(9, 100, 256, 64, True, False, False)
    X[3, 17] = math.inf
    X[5, 200] = math.nan
    Y = proj(X, P)
    ref = X.double() @ W.t()
    fine = [m for m in range(9) if m not in (3, 5)]
    check(Y[fine], X[fine], W, None)
    assert Y[5].isnan().all()
    # ∞·w: of w's sign, NaN where w is 0.
    assert torch.equal(Y[3].isnan(), ref[3].isnan()) and torch.equal(Y[3] == math.inf, ref[3] == math.inf)


@pytest.mark.parametrize("sizes", [(1e-30,), (1e-20,), (1e5,), (1e12,), (1e25,), (1.0, 1e30), (1e-30, 1.0), (1e-25, 1e25)], ids=str)
@pytest.mark.parametrize("M", [1, 6, 16, 32])
def test_activations_of_any_size(M, sizes):
    # Every size of activation that fp32 sums can hold, and sizes that change along K or between tokens.
    import torch
    proj, P, X, _, W = run(M, 70, 512, 64, True, False, True, seed=11)
    size = torch.tensor(sizes, device="cuda", dtype=torch.float64)
    for at in (torch.arange(512, device="cuda") // 64 % len(sizes), torch.arange(512, device="cuda") // 5 % len(sizes)):
        x = (X.double() * size[at][None]).to(torch.bfloat16)
        check(proj(x, P), x, W, None, f"{sizes} along K")
    x = (X.double() * size[torch.arange(M, device="cuda") % len(sizes)][:, None]).to(torch.bfloat16)
    check(proj(x, P), x, W, None, f"{sizes} between tokens")


def test_refusals():
    import torch
    import dense_linear_projection_gb300 as dlp
    proj, P, X, b, _ = run(4, 64, 256, 64, True, True, False)
    codes, scales, z = stored(64, 256, 64, True, 1)
    invalid = dlp.PROJ_ERR_INVALID_ARG
    for what, status in [
        (lambda: proj(torch.cat([X, X]), P, b), invalid),                     # more than max_tokens
        (lambda: proj(X, P), invalid),                                        # bias missing
        (lambda: proj(X.float(), P, b), invalid),
        (lambda: proj(X[:, :128], P, b), invalid),
        (lambda: proj(X, P, b, out=torch.empty((4, 64), device="cuda")), invalid),
        (lambda: proj.pack(codes, scales), invalid),                          # zeros missing
        (lambda: proj.pack(codes[:32], scales, z), invalid),
        (lambda: dlp.Q4Projection(4, 64, 256, 48), dlp.PROJ_ERR_UNSUPPORTED),
        (lambda: dlp.Q4Projection(4, 64, 200, 64), invalid),
        (lambda: dlp.Q4Projection(-1, 64, 256, 64), invalid),
        (lambda: dlp.Q4Projection(4, 64, 256, 64, y_dtype=dlp.PROJ_E4M3), invalid),
        (lambda: dlp.proj_q4_run(proj.handle, 4, X.data_ptr() + 2, P, b, X), dlp.PROJ_ERR_MISALIGNED),
        (lambda: dlp.proj_q4_run(proj.handle, 4, None, P, b, X), invalid),
        (lambda: dlp.proj_q4_run(None, 4, X, P, b, X), invalid),
    ]:
        with pytest.raises(dlp.ProjError) as e:
            what()
        assert e.value.status == status


@pytest.mark.parametrize("M,N,K,group", [(1, 2048, 8192, 128), (8, 130, 8192, 64), (16, 4100, 8192, 64),
                                         (16, 500, 4096, 128), (31, 12300, 4128, 32), (32, 6000, 2048, 128), (64, 1000, 2048, 64)])
def test_clusters_that_leave_and_start_back_to_back(M, N, K, group):
    # Shared K ranges: a cluster's sums are read by its other CTAs while the next launch's CTAs wait
    # for the places that it leaves.  Integers below 2²⁴ come out exactly whenever all are read in time.
    import torch
    import dense_linear_projection_gb300 as dlp
    codes, _, z = stored(N, K, group, True, 21)
    scales = torch.ones((N, K // group), device="cuda", dtype=torch.bfloat16)
    proj = dlp.Q4Projection(M, N, K, group, has_zeros=True, y_dtype=dlp.PROJ_F32)
    P = proj.pack(codes, scales, z)
    X = torch.randint(-3, 4, (4, M, K), device="cuda").to(torch.bfloat16)
    out = torch.empty((24, M, N), device="cuda")
    for i in range(24):
        proj(X[i % 4], P, out=out[i])
    W = dequantised(codes, scales, z, group)
    for i in range(4):
        ref = (X[i].double() @ W.t()).float()
        for j in range(i, 24, 4):
            assert torch.equal(out[j], ref), (i, j)


@pytest.mark.parametrize("powers", [(100, -100), (-100, 100), (120, -60), (-120, 118), (126, -100)], ids=str)
@pytest.mark.parametrize("M", [1, 16, 32])
def test_scales_of_any_size(M, powers):
    # Scales and activations far from 1 whose products are not.
    import torch
    import dense_linear_projection_gb300 as dlp
    N, K, group = 70, 512, 64
    codes, _, z = stored(N, K, group, True, 13)
    scales = (torch.rand((N, K // group), device="cuda").double().add(0.25) * 2.0 ** powers[0]).to(torch.bfloat16)
    proj = dlp.Q4Projection(M, N, K, group, has_zeros=True, y_dtype=dlp.PROJ_F32)
    X = (torch.randn((M, K), device="cuda").double() * 2.0 ** powers[1]).to(torch.bfloat16)
    check(proj(X, proj.pack(codes, scales, z)), X, dequantised(codes, scales, z, group), None, str(powers))
