"""Eviction by score: which tokens stay is exact (whole numbers and copies), so every result has to be equal."""
import math

import pytest

import kv_util as ku

pytestmark = pytest.mark.gpu


def chosen(scores, n, keep, recent):
    """Places kept, from a plain list of scores: the definition, token by token."""
    if n <= keep:
        return list(range(n))
    key = [math.inf if s != s else s for s in scores[:n]]
    nan = [s != s for s in scores[:n]]
    order = sorted(range(n - recent), key=lambda i: (not nan[i], -key[i], i))
    return sorted(order[:keep - recent]) + list(range(n - recent, n))


def run(lens, kv_heads, dim, page, keep, recent, dtype="bf16", layout="tokens_first", scores=None, extra_to=0, seed=0, extra_scores=0,
        stream=None):
    import torch
    import dense_linear_projection_gb300 as dlp
    B = len(lens)
    need = sum(-(-n // page) for n in lens)
    to_width = -(-keep // page) + extra_to
    pages = need + B * to_width + 3
    k_cache, v_cache = ku.make_cache(pages, page, kv_heads, dim, dtype, layout, seed)
    g = torch.Generator()
    g.manual_seed(seed)
    free = torch.randperm(pages, generator=g).to(torch.int32)
    width = max(-(-n // page) for n in lens) + 1 if lens else 1
    table = torch.full((B, width), 2 ** 31 - 1, dtype=torch.int32)  # what is not used is not read
    at = 0
    for i, n in enumerate(lens):
        m = -(-n // page)
        table[i, :m] = free[at:at + m]
        at += m
    to = free[at:at + B * to_width].view(B, to_width).cuda()
    table, n_dev = table.cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda")
    if scores is None:
        scores = torch.randn((B, kv_heads, width * page + extra_scores), generator=g).exp()
    scores = scores.cuda()
    want_k, want_v = k_cache.clone(), v_cache.clone()
    raw = lambda c: c.view(torch.uint8) if dtype == "e4m3" else c  # noqa: E731
    want_kept = torch.full((B, kv_heads, keep), -1, dtype=torch.int32)
    want_scores = torch.zeros((B, kv_heads, to_width * page))
    for b, n in enumerate(lens):
        for h in range(kv_heads):
            stay = torch.tensor(chosen(scores[b, h].tolist(), n, keep, recent), dtype=torch.long)
            m = len(stay)
            if not m:
                continue
            want_kept[b, h, :m] = stay.to(torch.int32)
            want_scores[b, h, :m] = scores[b, h].cpu()[stay]
            i, s = torch.arange(m, device="cuda"), stay.cuda()
            for want, old in ((want_k, k_cache), (want_v, v_cache)):
                raw(want)[to[b].long()[i // page], i % page, h] = raw(old)[table[b].long()[s // page], s % page, h]
    kv = dlp.PagedKV(k_cache, v_cache, kv_heads, 1)
    given = scores.clone(), table.clone(), n_dev.clone()
    got_lens, got_scores, kept = kv.evict(table, n_dev, scores, to, keep, recent, stream=stream)
    torch.cuda.synchronize()
    assert kv.status(stream) == dlp.PROJ_OK
    assert got_lens.tolist() == [min(n, keep) for n in lens] and got_lens.dtype == torch.int32
    assert torch.equal(kept.cpu(), want_kept)
    assert torch.equal(got_scores.cpu().view(torch.int32), want_scores.view(torch.int32))
    bits = lambda c: c.contiguous().view(torch.uint8 if dtype == "e4m3" else torch.int16)  # noqa: E731
    assert torch.equal(bits(k_cache), bits(want_k)) and torch.equal(bits(v_cache), bits(want_v))
    assert torch.equal(scores.view(torch.int32), given[0].view(torch.int32))
    assert torch.equal(table, given[1]) and torch.equal(n_dev, given[2])


@pytest.mark.parametrize("lens", [[1], [0], [2, 0, 1], [15, 16, 17, 18], [1000, 0, 3, 1025, 999]])
@pytest.mark.parametrize("keep,recent", [(1, 0), (1, 1), (16, 3), (16, 16), (17, 0), (1000, 100)])
def test_lengths_and_budgets(lens, keep, recent):
    run(lens, 2, 64, 16, keep, recent)


@pytest.mark.parametrize("n", [1023, 4096, 4097, 8192, 8193, 20000, 70001, 140001])
@pytest.mark.parametrize("part", [0.01, 0.5, 0.999])
def test_long_rows(n, part):
    run([n, n // 3], 2, 16, 64, max(2, int(n * part)), 1)


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("dim", [16, 48, 64, 80, 128, 256])
def test_head_dims(dim, dtype):
    run([100, 33], 3, dim, 16, 20, 5, dtype)


@pytest.mark.parametrize("page", [1, 3, 16, 100])
@pytest.mark.parametrize("layout", ["tokens_first", "heads_first", "together"])
def test_pages_and_layouts(page, layout):
    run([50, 301, 0], 4, 32, page, 37, 9, layout=layout, extra_to=2, extra_scores=5)


@pytest.mark.parametrize("kind", ["zeros", "two", "negative", "signs", "special", "close", "falling", "wide"])
@pytest.mark.parametrize("n,keep,recent", [(60, 21, 4), (9000, 4444, 17), (30001, 29999, 1)])
def test_scores(kind, n, keep, recent):
    import torch
    g = torch.Generator()
    g.manual_seed(3)
    shape = (1, 2, -(-n // 16) * 16 + 16)
    x = torch.randn(shape, generator=g)
    if kind == "zeros":  # equal: the earliest stay
        x = torch.zeros(shape)
    elif kind == "two":
        x = (x > 0.3).float()
    elif kind == "negative":
        x = -x.abs()
    elif kind == "signs":  # both zeros are one number
        x = torch.where(x > 0, 0.0, -0.0)
    elif kind == "special":
        x[..., ::7], x[..., 1::11], x[..., 2::13], x[..., 3::17] = math.inf, -math.inf, math.nan, -math.nan
    elif kind == "close":  # neighbouring floats
        x = (torch.full(shape, 1.0).view(torch.int32) + torch.randint(0, 40, shape, generator=g, dtype=torch.int32)).view(torch.float32)
    elif kind == "falling":
        x = torch.arange(shape[2], 0, -1).float().expand(shape).contiguous()
    elif kind == "wide":  # every exponent
        x = torch.ldexp(x, torch.randint(-140, 120, shape, generator=g))
    run([n], 2, 16, 16, keep, recent, scores=x)


def test_keep_nothing():
    run([50, 0, 3], 2, 64, 16, 0, 0)
    run([50, 0, 3], 2, 64, 16, 0, 0, extra_to=1)


def test_many_rows():
    run([40 + i for i in range(70)], 16, 16, 8, 33, 7)


def test_offsets_past_31_bits():
    # Old and new pages more than 2^31 elements apart.
    import torch
    import dense_linear_projection_gb300 as dlp
    stride, hk, dim = 1 << 26, 2, 64
    base = [torch.zeros(stride * 43 + 16 * hk * dim, dtype=torch.bfloat16, device="cuda") for _ in "kv"]
    k_cache, v_cache = (x.as_strided((44, 16, hk, dim), (stride, hk * dim, dim, 1)) for x in base)
    ints = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    for c in (k_cache, v_cache):
        c[43], c[2] = torch.randn((16, hk, dim), device="cuda"), torch.randn((16, hk, dim), device="cuda")
    kv = dlp.PagedKV(k_cache, v_cache, 2, 1)
    scores = torch.arange(32, device="cuda").float().expand(1, hk, 32).contiguous()
    lens, _, kept = kv.evict(ints(43, 2)[None], ints(32), scores, ints(40)[None], 16)
    assert kv.status() == dlp.PROJ_OK and lens.tolist() == [16] and kept[0, 1].tolist() == list(range(16, 32))
    assert torch.equal(k_cache[40], k_cache[2]) and torch.equal(v_cache[40], v_cache[2])


def test_bad_pages_and_lengths():
    import torch
    import dense_linear_projection_gb300 as dlp
    ints = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    for table, lens, to, status in ((ints(0, 9), ints(32), ints(3, 4), "bad"), (ints(0, -1), ints(32), ints(3, 4), "bad"),
                                    (ints(0, 1), ints(32), ints(3, 9), "bad"), (ints(0, 1), ints(33), ints(3, 4), "bad"),
                                    (ints(0, 1), ints(-1), ints(3, 4), "bad"), (ints(0, 1), ints(32), ints(3, 4), "good"),
                                    (ints(0, -1), ints(16), ints(3, -1), "good")):
        k_cache, v_cache = ku.make_cache(5, 16, 1, 64)
        before = k_cache.clone()
        kv = dlp.PagedKV(k_cache, v_cache, 1, 1)
        scores = torch.ones((1, 1, 32), device="cuda")
        new_lens, new_scores, kept = kv.evict(table[None], lens, scores, to[None], 20, 4)
        assert kv.status() == (dlp.PROJ_OK if status == "good" else dlp.PROJ_ERR_INVALID_ARG)
        assert kv.status() == dlp.PROJ_OK
        n = min(max(lens.item(), 0), 32)
        want = chosen([1.0] * 32, n, 20, 4)
        assert new_lens.item() == len(want) and kept[0, 0].tolist() == want + [-1] * (20 - len(want))
        after = before.clone()
        for i, s in enumerate(want):
            p0, p1 = table[s // 16].item(), to[i // 16].item()
            if 0 <= p0 < 5 and 0 <= p1 < 5:
                after[p1, i % 16] = before[p0, s % 16]
        assert torch.equal(k_cache, after)


def test_on_a_stream_and_in_a_graph():
    import torch
    import dense_linear_projection_gb300 as dlp
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    run([100, 3000], 2, 64, 16, 50, 7, stream=side)
    k_cache, v_cache = ku.make_cache(40, 16, 2, 64)
    kv = dlp.PagedKV(k_cache, v_cache, 2, 2)
    table = torch.randperm(40).to(torch.int32).cuda()
    old, to = table[:20].view(2, 10).contiguous(), table[20:26].view(2, 3).contiguous()
    lens, scores = torch.tensor([100, 30], dtype=torch.int32, device="cuda"), torch.rand((2, 2, 160), device="cuda")
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        kv.evict(old, lens, scores, to, 40, 8)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        results = kv.evict(old, lens, scores, to, 40, 8)
    for n0, n1 in ((160, 41), (7, 0), (40, 99)):
        scores.uniform_()
        lens.copy_(torch.tensor([n0, n1], dtype=torch.int32))
        graph.replay()
        again = kv.evict(old, lens, scores, to, 40, 8)
        assert all(torch.equal(a, b) for a, b in zip(results, again))
        for b, n in enumerate((n0, n1)):
            for h in range(2):
                assert [x for x in results[2][b, h].tolist() if x >= 0] == chosen(scores[b, h].tolist(), n, 40, 8)
    assert kv.status() == dlp.PROJ_OK


def test_empty_batch_and_refusals():
    import torch
    import dense_linear_projection_gb300 as dlp
    k_cache, v_cache = ku.make_cache(8, 16, 2, 64)
    kv = dlp.PagedKV(k_cache, v_cache, 4, 2)
    table = torch.arange(4, dtype=torch.int32, device="cuda").view(2, 2)
    to = torch.arange(4, 6, dtype=torch.int32, device="cuda").view(2, 1)
    lens, scores = torch.full((2,), 20, dtype=torch.int32, device="cuda"), torch.rand((2, 2, 32), device="cuda")
    good = dict(page_table=table, seq_lens=lens, scores=scores, to_table=to, keep=16, recent=3)
    for change in (dict(keep=17), dict(keep=-1), dict(recent=17), dict(recent=-1), dict(scores=scores[:, :, :31]), dict(scores=scores[:, :1]),
                   dict(scores=scores.double()), dict(scores=scores.cpu()), dict(scores=None), dict(to_table=to[:1]), dict(to_table=to.long()),
                   dict(page_table=table.t()), dict(page_table=table.cpu()), dict(seq_lens=lens[:1]), dict(seq_lens=lens.long()),
                   dict(scores=scores.transpose(0, 1)), dict(keep=2.5)):
        with pytest.raises((dlp.ProjError, TypeError)) as e:
            kv.evict(**{**good, **change})
        assert not isinstance(e.value, dlp.ProjError) or e.value.status == dlp.PROJ_ERR_INVALID_ARG, change
    lens_out, scores_out, kept = kv.evict(table[:0], lens[:0], scores[:0], to[:0], 16)
    assert lens_out.shape == (0,) and scores_out.shape == (0, 2, 16) and kept.shape == (0, 2, 16)
    kv.evict(**good)
    assert kv.status() == dlp.PROJ_OK
    kv.close()
    with pytest.raises(dlp.ProjError):
        kv.evict(**good)
