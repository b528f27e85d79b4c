"""Attention that adds each token's weight to its score.

The bound of a weight: a logit is off by δ (kv_util.attention64's), so the weight and its sum by a
factor within 2δ, two exponentials 2⁻²⁰, the sum over n tokens (n/16 + 64)·2⁻²², its reciprocal
and product 2⁻²²; a score is the sum over the heads of a key head, in fp32: 2⁻²² of it more."""
import math

import pytest

import kv_util as ku

pytestmark = pytest.mark.gpu


def weights64(q, k_cache, table, lens, page_size, scale, window=0, k_scale=None, keep=None):
    """(Σ of weights, bound) [sequences, kv_heads, tokens of the table] in 64 bits."""
    import torch
    B, H, D = q.shape
    hk = k_cache.shape[2]
    out = torch.zeros((B, hk, table.shape[1] * page_size), dtype=torch.float64, device="cuda")
    lim = torch.zeros_like(out)
    for b, n in enumerate(lens):
        low = max(0, n - window) if window else 0
        if n <= low:
            continue
        k = ku.tokens_of(k_cache, table, b, low, n, page_size)
        if k_scale is not None:
            k = k * k_scale.double()[:, None]
        k = k.repeat_interleave(H // hk, 1)
        s = torch.einsum("hd,thd->ht", q[b].double(), k) * scale
        a = torch.einsum("hd,thd->ht", q[b].double().abs(), k.abs()).amax(1) * abs(scale)
        if keep is not None:
            s = torch.where(keep(b, torch.arange(low, n, device="cuda"))[None], s, -math.inf)
        p = torch.softmax(s, 1).nan_to_num(0.0)
        delta = (D / 16 + 8) * 2.0 ** -22 * a
        rel = 2 * delta + 2.0 ** -19 + ((n - low) / 16 + 66) * 2.0 ** -22
        out[b, :, low:n] = p.view(hk, H // hk, -1).sum(1)
        lim[b, :, low:n] = (p * rel[:, None]).view(hk, H // hk, -1).sum(1)
    return out, lim


def run(lens, heads, kv_heads, dim, page, window=0, dtype="bf16", layout="tokens_first", scale=None, in_place=False, extra=0, seed=0,
        size=1.0):
    import torch
    import dense_linear_projection_gb300 as dlp
    pages = sum(-(-n // page) for n in lens) + 2
    k_cache, v_cache = ku.make_cache(pages, page, kv_heads, dim, dtype, layout, seed)
    table = ku.make_table(lens, page, pages, seed)
    g = torch.Generator()
    g.manual_seed(seed)
    q = (torch.randn((len(lens), heads, dim), generator=g) * size).cuda().to(torch.bfloat16)
    scales = [torch.rand(kv_heads, generator=g).cuda() + 0.2 for _ in "kv"] if dtype == "e4m3" else [None, None]
    tokens = table.shape[1] * page
    scores = torch.rand((len(lens), kv_heads, tokens + extra), generator=g).cuda()
    before = scores.clone()
    kv = dlp.PagedKV(k_cache, v_cache, heads, len(lens), k_scale=scales[0], v_scale=scales[1])
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    s = dim ** -0.5 if scale is None else scale
    to = None if in_place else torch.full_like(scores, math.nan)
    out, got, lse = kv.attend_scored(q, table, n, scores, scale=scale, window=window, scores_out=to, return_lse=True)
    assert kv.status() == dlp.PROJ_OK and got is (scores if in_place else to)
    plain, plain_lse = kv.attend(q, table, n, scale=scale, window=window, return_lse=True)
    assert torch.equal(out, plain) and torch.equal(lse, plain_lse)  # the same kernel's own results
    ku.check_attention(out, lse, ku.attention64(q, k_cache, v_cache, table, lens, page, s, window, *scales))
    want, lim = weights64(q, k_cache, table, lens, page, s, window, scales[0])
    more = torch.zeros((len(lens), kv_heads, extra), device="cuda", dtype=torch.float64)
    want, lim = before.double() + torch.cat([want, more], 2), torch.cat([lim, more], 2)
    over = ku.beyond(got, want, lim + 2.0 ** -22 * (want - before))
    assert (over <= 0).all(), f"{int((over > 0).sum())} of {over.numel()}, by up to {over.max().item():.3e}"
    if not in_place:
        assert torch.equal(scores, before)


@pytest.mark.parametrize("lens", [[1], [0], [2, 0, 1], [15, 16, 17], [127, 128, 129], [1000, 0, 3, 4097]])
@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("in_place", [False, True])
def test_lengths(lens, dtype, in_place):
    run(lens, 8, 2, 128, 16, dtype=dtype, in_place=in_place)


@pytest.mark.parametrize("heads,kv_heads", [(1, 1), (8, 8), (2, 1), (6, 2), (14, 2), (16, 2), (32, 2), (20, 1), (96, 2), (64, 8), (71, 1),
                                            (40, 40), (51, 3)])
@pytest.mark.parametrize("dtype,dim", [("bf16", 128), ("e4m3", 128), ("bf16", 64), ("bf16", 256)])
def test_head_groups(heads, kv_heads, dtype, dim):
    run([300, 77], heads, kv_heads, dim, 16, dtype=dtype)


@pytest.mark.parametrize("dim", [16, 48, 80, 144])
@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
def test_head_dims(dim, dtype):
    run([200, 0, 31], 8, 2, dim, 16, dtype=dtype)


@pytest.mark.parametrize("page", [1, 3, 17, 100])
@pytest.mark.parametrize("layout", ["tokens_first", "heads_first", "together"])
def test_pages_and_layouts(page, layout):
    run([250, 31, 99], 8, 4, 64, page, layout=layout, extra=7)


@pytest.mark.parametrize("window", [1, 15, 100, 5000])
@pytest.mark.parametrize("in_place", [False, True])
def test_windows(window, in_place):
    run([1000, 16, 0, 101], 8, 2, 64, 16, window, in_place=in_place, extra=3)


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("lens,heads,kv_heads,dim", [([30000], 8, 1, 128), ([100, 40000, 3], 4, 1, 64), ([9000, 17000], 16, 1, 128)])
def test_rows_of_many_parts(lens, heads, kv_heads, dim, dtype):
    run(lens, heads, kv_heads, dim, 64, dtype=dtype)


@pytest.mark.parametrize("scale", [0.0, -0.1, 3.0])
def test_scales(scale):
    run([300, 7], 8, 2, 64, 16, scale=scale)
    run([300, 7], 8, 2, 64, 16, scale=scale, size=20.0)


def test_bad_pages_have_no_weight():
    import torch
    import dense_linear_projection_gb300 as dlp
    page, lens = 16, [70, 40, 32]
    k_cache, v_cache = ku.make_cache(20, page, 2, 64)
    table = ku.make_table(lens, page, 20)
    table[0, 1], table[2, :2] = 20, -1  # the last sequence has no page at all
    q = torch.randn((3, 8, 64), device="cuda").to(torch.bfloat16)
    kv = dlp.PagedKV(k_cache, v_cache, 8, 3)
    scores = torch.zeros((3, 2, table.shape[1] * page), device="cuda")
    kv.attend_scored(q, table, torch.tensor(lens, dtype=torch.int32, device="cuda"), scores)
    assert kv.status() == dlp.PROJ_ERR_INVALID_ARG and kv.status() == dlp.PROJ_OK
    good = table.clamp(0, 19)
    want, lim = weights64(q, k_cache, good, lens, page, 64 ** -0.5, keep=lambda b, t: torch.ones_like(t, dtype=torch.bool) if b == 1
                          else torch.zeros_like(t, dtype=torch.bool) if b == 2 else (t < 16) | (t >= 32))
    assert (ku.beyond(scores, want, lim + 2.0 ** -22 * want) <= 0).all()


def test_nan_and_infinity():
    # A key of NaN spoils its own key head's scores of that sequence, and nothing else.
    import torch
    import dense_linear_projection_gb300 as dlp
    k_cache, v_cache = ku.make_cache(12, 16, 2, 64)
    table = torch.arange(12, dtype=torch.int32, device="cuda").view(2, 6)
    k_cache[0, 3, 1, 5] = math.nan
    k_cache[5, 15] = math.nan  # past both sequences' ends
    q = torch.randn((2, 8, 64), device="cuda").to(torch.bfloat16)
    kv = dlp.PagedKV(k_cache, v_cache, 8, 2)
    scores = torch.zeros((2, 2, 96), device="cuda")
    kv.attend_scored(q, table, torch.tensor([90, 60], dtype=torch.int32, device="cuda"), scores)
    assert scores[0, 1, :90].isnan().all() and not scores[0, 0].isnan().any() and not scores[1].isnan().any()
    assert (scores[0, :, 90:] == 0).all() and (scores[1, :, 60:] == 0).all()


def test_sums_over_steps_in_a_graph():
    # Steps of a decode loop: the scores' sum over the tokens is the heads of a key head for each step.
    import torch
    import dense_linear_projection_gb300 as dlp
    k_cache, v_cache = ku.make_cache(40, 16, 2, 128)
    table = torch.randperm(40).to(torch.int32).view(2, 20).cuda()
    kv = dlp.PagedKV(k_cache, v_cache, 8, 2)
    q = torch.randn((2, 8, 128), device="cuda").to(torch.bfloat16)
    lens, scores = torch.tensor([100, 7], dtype=torch.int32, device="cuda"), torch.zeros((2, 2, 320), device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        kv.attend_scored(q, table, lens, scores)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, _ = kv.attend_scored(q, table, lens, scores)
    for step in range(5):
        lens += 31
        q.normal_()
        graph.replay()
        eager = scores.clone()
        again, _ = kv.attend_scored(q, table, lens, eager)
        assert torch.equal(out, again)
    total = scores.double().sum(2)
    assert ((total - 4 * 6).abs() <= 24 * 2.0 ** -14).all(), total  # 2⁻²⁰·(320/16 + …) of each step's weights
    assert kv.status() == dlp.PROJ_OK


def test_refusals():
    import torch
    import dense_linear_projection_gb300 as dlp
    k_cache, v_cache = ku.make_cache(8, 16, 2, 64)
    kv = dlp.PagedKV(k_cache, v_cache, 4, 2)
    q = torch.randn((2, 4, 64), device="cuda").to(torch.bfloat16)
    table, lens = torch.arange(4, dtype=torch.int32, device="cuda").view(2, 2), torch.full((2,), 20, dtype=torch.int32, device="cuda")
    scores = torch.zeros((2, 2, 40), device="cuda")
    flat = torch.zeros(400, device="cuda")
    good = dict(q=q, page_table=table, seq_lens=lens, scores=scores)
    for change in (dict(scores=scores[:, :, :31].contiguous()), dict(scores=scores[:, :, :36]), dict(scores=scores.bfloat16()),
                   dict(scores=scores.cpu()), dict(scores=None), dict(scores_out=scores[:1]), dict(scores_out=torch.zeros((2, 2, 41), device="cuda")),
                   dict(scores=flat[:160].view(2, 2, 40), scores_out=flat[8:168].view(2, 2, 40)), dict(window=-1), dict(scale=math.inf),
                   dict(scale="x"), dict(q=q[:1]), dict(q=q.float()), dict(seq_lens=lens.long()), dict(page_table=table.cpu()),
                   dict(out=q[:1]), dict(q=torch.cat([q, q]), page_table=torch.cat([table, table]), seq_lens=torch.cat([lens, lens]),
                                         scores=torch.zeros((4, 2, 40), device="cuda"))):
        with pytest.raises((dlp.ProjError, TypeError)) as e:
            kv.attend_scored(**{**good, **change})
        assert not isinstance(e.value, dlp.ProjError) or e.value.status == dlp.PROJ_ERR_INVALID_ARG, change
    assert (scores == 0).all()
    out, got = kv.attend_scored(q[:0], table[:0], lens[:0], scores[:0])
    assert out.shape == (0, 4, 64)
    # A page table of no pages: empty sequences.
    out, got = kv.attend_scored(q, table[:, :0], lens * 0, torch.ones((2, 2, 3), device="cuda"))
    assert (out == 0).all() and (got == 1).all() and kv.status() == dlp.PROJ_OK
    kv.close()
    with pytest.raises(dlp.ProjError):
        kv.attend_scored(**good)
