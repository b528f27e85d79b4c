"""A NaN in a head that is otherwise zero or tiny: the whole head's norm is NaN, as for heads of any size."""
import math

import pytest

import kv_util as ku
from test_kv_norm_gpu import normed64

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("eps", [0.0, 1e-30, 1e-6, 1.0])
@pytest.mark.parametrize("dim,rot", [(128, 128), (64, 20), (64, 0)])
@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
def test_nan_among_small_elements(dim, rot, eps, dtype):
    import torch
    import dense_linear_projection_gb300 as dlp
    tokens, heads, kv_heads, page = 8, 4, 2, 16
    g = torch.Generator()
    g.manual_seed(dim + rot)
    x = torch.randn((tokens, heads + 2 * kv_heads, dim), generator=g)
    x[1], x[2], x[4], x[5] = 0, x[2] * 2.0 ** -100, x[4] * 2.0 ** -126, x[5] * 2.0 ** 100
    for t in (1, 2, 4, 5):
        x[t, ::2, 3 + t] = math.nan  # (every other head stays finite)
    x = x.cuda().to(torch.bfloat16)
    q, k, v = x[:, :heads], x[:, heads:heads + kv_heads], x[:, heads + kv_heads:]
    w = (1 + 0.3 * torch.randn(dim, generator=g)).cuda()
    pos = torch.arange(tokens, dtype=torch.int32, device="cuda")
    rope = dlp.rope_table(tokens, rot) if rot else None
    k_cache, v_cache = ku.make_cache(1, page, kv_heads, dim, dtype)
    kv = dlp.PagedKV(k_cache, v_cache, heads, 1)
    got = kv.append(q, k, v, pos, torch.zeros((1, 1), dtype=torch.int32, device="cuda"), seq_ids=torch.zeros_like(pos), rope=rope,
                    q_norm=w, k_norm=w, eps=eps)
    assert kv.status() == dlp.PROJ_OK
    for have, rows in ((got, q), (k_cache[0, :tokens], k)):
        want, _ = normed64(rows, w, eps, rope, False)
        assert torch.equal(have.float().isnan(), want.isnan())
        # Heads without a NaN, and those that are one: nothing between.
        of_head = want.isnan().sum(-1)
        assert bool(((of_head == 0) | (of_head == dim)).all()) and bool((of_head == dim).any())
