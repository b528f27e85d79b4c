"""Attention of a batch that shares a prefix.

The bound: kv_util.attention64's for the own tokens, with the weights' parts as fp32 holds them;
for the prefix a logit is a sum of dim products in dim/16 steps of the tensor core, δ = (dim/16 + 8)·2⁻²²·A;
a weight is off by a factor within 2δ and the exponentials' 2⁻²⁰; sums over n tokens take 3·n/16 steps of
2⁻²³ and a few dozen joins: (n/8 + 64)·2⁻²²."""
import math

import pytest

import kv_util as ku

pytestmark = pytest.mark.gpu


def shared64(q, k_cache, v_cache, prefix, prefix_len, table, lens, page, scale, k_scale=None, v_scale=None, keep=None):
    """(out, lse, bound of out, bound of lse) in 64 bits."""
    import torch
    B, H, D = q.shape
    hk = k_cache.shape[2]
    G = H // hk
    out = torch.zeros((B, H, D), dtype=torch.float64, device="cuda")
    lse = torch.full((B, H), -math.inf, dtype=torch.float64, device="cuda")
    lim, lim_lse = torch.zeros_like(out), torch.zeros_like(lse)
    one = torch.ones(hk, dtype=torch.float64, device="cuda")
    ks, vs = (one if s is None else s.double() for s in (k_scale, v_scale))
    k0, v0 = (ku.tokens_of(c, prefix[None], 0, 0, prefix_len, page) * s[:, None] for c, s in ((k_cache, ks), (v_cache, vs)))
    if keep is not None:
        sel = keep(torch.arange(prefix_len, device="cuda"))
        k0, v0 = k0[sel], v0[sel]
    for b, n in enumerate(lens):
        k1, v1 = (ku.tokens_of(c, table, b, 0, n, page) * s[:, None] for c, s in ((k_cache, ks), (v_cache, vs)))
        for j in range(hk):
            k, v = torch.cat([k0[:, j], k1[:, j]]), torch.cat([v0[:, j], v1[:, j]])
            if not k.shape[0]:
                continue
            rows = slice(j * G, (j + 1) * G)
            x = q[b, rows].double()
            s = (x @ k.t()) * scale
            a = (x.abs() @ k.abs().t()).amax(1) * abs(scale)
            p = torch.softmax(s, 1)
            out[b, rows], lse[b, rows] = p @ v, torch.logsumexp(s, 1)
            rel = 2 * (D / 16 + 8) * 2.0 ** -22 * a + 2.0 ** -20 + (k.shape[0] / 8 + 64) * 2.0 ** -22
            lim[b, rows] = (p @ v.abs()) * rel[:, None]
            lim_lse[b, rows] = rel + 2.0 ** -22 * lse[b, rows].abs()
    return out, lse, lim + 1e-38, lim_lse


def case(prefix_len, lens, heads, kv_heads, dim, page, dtype="bf16", layout="tokens_first", seed=0, size=1.0):
    import torch
    import dense_linear_projection_gb300 as dlp
    need = -(-prefix_len // page)
    pages = sum(-(-n // page) for n in lens) + need + 2
    k_cache, v_cache = ku.make_cache(pages, page, kv_heads, dim, dtype, layout, seed)
    both = ku.make_table([prefix_len, *lens], page, pages, seed, unused=2 ** 31 - 1)
    prefix, table = both[0, :need + 1].contiguous(), both[1:, :max([-(-n // page) for n in lens], default=0) + 1].contiguous()
    g = torch.Generator()
    g.manual_seed(seed)
    q = (torch.randn((len(lens), heads, dim), generator=g) * size).cuda().to(torch.bfloat16)
    scales = [torch.rand(kv_heads, generator=g).cuda() + 0.2 for _ in "kv"] if dtype == "e4m3" else [None, None]
    kv = dlp.PagedKV(k_cache, v_cache, heads, len(lens), k_scale=scales[0], v_scale=scales[1])
    return kv, q, prefix, table, torch.tensor(lens, dtype=torch.int32, device="cuda"), scales


def run(prefix_len, lens, heads, kv_heads, dim, page, scale=None, **more):
    import dense_linear_projection_gb300 as dlp
    kv, q, prefix, table, n, scales = case(prefix_len, lens, heads, kv_heads, dim, page, **more)
    out, lse = kv.attend_shared(q, prefix, prefix_len, table, n, scale=scale, return_lse=True)
    assert kv.status() == dlp.PROJ_OK
    ref = shared64(q, kv.k_cache, kv.v_cache, prefix, prefix_len, table, lens, page, dim ** -0.5 if scale is None else scale, *scales)
    ku.check_attention(out, lse, ref, f"{prefix_len} {lens[:4]}")
    return out, lse


@pytest.mark.parametrize("prefix_len", [1, 2, 127, 128, 129, 1000, 5000])
@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
def test_prefix_lengths(prefix_len, dtype):
    run(prefix_len, [5, 0, 130], 8, 2, 128, 16, dtype=dtype)


@pytest.mark.parametrize("lens", [[0], [1], [0, 0, 0], [15, 16, 17], [1000, 0, 3, 2000]])
@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
def test_own_lengths(lens, dtype):
    run(300, lens, 8, 2, 64, 16, dtype=dtype)


@pytest.mark.parametrize("heads,kv_heads", [(1, 1), (8, 8), (6, 2), (14, 2), (64, 8), (71, 1), (96, 2), (40, 40)])
@pytest.mark.parametrize("batch", [1, 3, 33])
def test_rows(heads, kv_heads, batch):
    # Row tiles of 128 that end inside a group of heads or with a few rows.
    run(700, [(7 * b) % 40 for b in range(batch)], heads, kv_heads, 64, 16)


@pytest.mark.parametrize("dim", [16, 32, 48, 64, 80, 112, 128, 144, 192, 240, 256])
@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
def test_head_dims(dim, dtype):
    run(333, [20, 0, 7], 8, 2, dim, 16, dtype=dtype)


@pytest.mark.parametrize("page", [1, 3, 16, 17, 64, 100, 300])
@pytest.mark.parametrize("layout", ["tokens_first", "heads_first", "together"])
def test_pages_and_layouts(page, layout):
    run(410, [50, 3], 8, 4, 64, page, layout=layout)


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_long_prefixes_and_many_rows(dim, dtype):
    run(20000, [9] * 40, 32, 2, dim, 64, dtype=dtype)     # five row tiles a key head
    run(1500, [3] * 150, 64, 8, dim, 64, dtype=dtype)      # more units than CTAs: whole units and shared ones
    run(30000, [1], 4, 1, dim, 64, dtype=dtype)            # one unit over every CTA


@pytest.mark.parametrize("scale", [0.0, -0.1, 3.0])
def test_scales(scale):
    run(500, [30, 7], 8, 2, 64, 16, scale=scale)
    run(500, [30, 7], 8, 2, 128, 16, scale=scale, size=20.0)


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_growing_logits(dim):
    # Keys that grow along the prefix: the running maximum moves past its slack again and again, over
    # sequences of one CTA and of several.
    import torch
    import dense_linear_projection_gb300 as dlp
    for prefix_len, batch in ((2000, 3), (24000, 40)):
        kv, q, prefix, table, n, _ = case(prefix_len, [5] * batch, 8, 1, dim, 16)
        q[:] = torch.rand_like(q.float()).add_(0.5).to(torch.bfloat16)
        at = torch.arange(prefix_len, device="cuda")
        grow = (torch.linspace(0.01, 12, prefix_len, device="cuda")[:, None, None] * (1 + 0.05 * torch.randn((prefix_len, 1, dim), device="cuda")))
        kv.k_cache[prefix.long()[at // 16], at % 16] = grow.to(torch.bfloat16)
        out, lse = kv.attend_shared(q, prefix, prefix_len, table, n, return_lse=True)
        ku.check_attention(out, lse, shared64(q, kv.k_cache, kv.v_cache, prefix, prefix_len, table, [5] * batch, 16, dim ** -0.5))
        assert kv.status() == dlp.PROJ_OK


@pytest.mark.parametrize("nats", [3, 12, 24, 60])
@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
def test_small_weights_count(dtype, nats):
    # One token of value 0 that has nearly all the weight, wherever it is: the others are the output.
    import torch
    # (Among the own tokens, in 8 bits, weights are held to 2^-52 of the largest: up to 24 nats below.)
    for where in (0, 1000, 3999) + ((-1,) if nats <= 24 else ()):
        kv, q, prefix, table, n, scales = case(4000, [40], 4, 1, 128, 16, dtype=dtype)
        for s in scales:
            if s is not None:
                s.fill_(1.0)
        q[:] = 0
        q[..., 0] = 1
        zero = torch.zeros((), dtype=torch.uint8, device="cuda")
        raw = lambda c: c.view(torch.uint8) if dtype == "e4m3" else c  # noqa: E731
        t = kv.k_cache.dtype
        big = torch.tensor(float(nats), device="cuda").to(t)
        raw(kv.k_cache)[..., 0] = raw(torch.zeros((), device="cuda").to(t)) if dtype == "e4m3" else 0
        page, place = (prefix[where // 16], where % 16) if where >= 0 else (table[0, 0], 0)
        raw(kv.k_cache)[page.item(), place, 0, 0] = big.view(torch.uint8) if dtype == "e4m3" else big
        raw(kv.v_cache)[page.item(), place, 0] = zero if dtype == "e4m3" else 0
        out, lse = kv.attend_shared(q, prefix, 4000, table, n, scale=1.0, return_lse=True)
        ku.check_attention(out, lse, shared64(q, kv.k_cache, kv.v_cache, prefix, 4000, table, [40], 16, 1.0, *scales), f"{where}")


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
def test_weights_are_held_as_fp32(dtype):
    # Two prefix tokens of nearly equal weight and opposite values: what 16 bits of a weight lose would show.
    import torch
    kv, q, prefix, table, n, scales = case(2, [0] * 64, 8, 1, 128, 16, dtype=dtype)
    for s in scales:
        if s is not None:
            s.fill_(1.0)
    v = kv.v_cache.float()
    v[prefix[0].item(), 1] = -v[prefix[0].item(), 0]
    kv.v_cache.copy_(v)
    out, lse = kv.attend_shared(q, prefix, 2, table, n, scale=1e-4, return_lse=True)
    ku.check_attention(out, lse, shared64(q, kv.k_cache, kv.v_cache, prefix, 2, table, [0] * 64, 16, 1e-4, *scales))


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_infinite_values(dim):
    import torch
    kv, q, prefix, table, n, _ = case(900, [20, 0], 8, 2, dim, 16)
    v = kv.v_cache
    v[prefix[0].item(), 0, 0, 1], v[prefix[3].item(), 5, 0, 2] = math.inf, -math.inf
    v[prefix[0].item(), 1, 1, 3], v[prefix[20].item(), 1, 1, 3] = math.inf, -math.inf
    v[prefix[2].item(), 1, 1, 4] = math.nan
    v[table[0, 0].item(), 1, 1, 5] = math.inf
    out = kv.attend_shared(q, prefix, 900, table, n)
    assert (out[:, :4, 1] == math.inf).all() and (out[:, :4, 2] == -math.inf).all()
    assert out[:, 4:, 3:5].isnan().all() and (out[0, 4:, 5] == math.inf).all()
    spoilt = torch.zeros_like(out, dtype=torch.bool)
    spoilt[:, :4, 1:3], spoilt[:, 4:, 3:5], spoilt[0, 4:, 5] = True, True, True
    assert torch.isfinite(out[~spoilt]).all()


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
def test_nothing_outside_the_prefix_is_used(dtype):
    # NaN in every place that is not a token's: past the prefix's end, in unused pages.
    import torch
    import dense_linear_projection_gb300 as dlp
    kv, q, prefix, table, n, scales = case(405, [37, 0], 8, 2, 64, 16, dtype=dtype)
    ref = shared64(q, kv.k_cache, kv.v_cache, prefix, 405, table, [37, 0], 16, 64 ** -0.5, *scales)
    used = torch.zeros(kv.k_cache.shape[:2], dtype=torch.bool, device="cuda")
    for row, m in ((prefix, 405), (table[0], 37)):
        t = torch.arange(m, device="cuda")
        used[row.long()[t // 16], t % 16] = True
    for c in (kv.k_cache, kv.v_cache):
        x = c.float()
        x[~used] = math.nan
        c.copy_(x)
    out, lse = kv.attend_shared(q, prefix, 405, table, n, return_lse=True)
    ku.check_attention(out, lse, ref)
    assert kv.status() == dlp.PROJ_OK


def test_bad_pages_are_reported_and_left_out():
    import torch
    import dense_linear_projection_gb300 as dlp
    kv, q, prefix, table, n, _ = case(700, [20, 0], 8, 2, 64, 16)
    good = prefix.clone()
    prefix[3], prefix[20] = -1, kv.k_cache.shape[0]
    out, lse = kv.attend_shared(q, prefix, 700, table, n, return_lse=True)
    assert kv.status() == dlp.PROJ_ERR_INVALID_ARG and kv.status() == dlp.PROJ_OK
    ref = shared64(q, kv.k_cache, kv.v_cache, good, 700, table, [20, 0], 16, 0.125, keep=lambda t: (t // 16 != 3) & (t // 16 != 20))
    ku.check_attention(out, lse, ref)
    prefix[:] = -1  # no token of the prefix is left: the own ones, or nothing
    out, lse = kv.attend_shared(q, prefix, 700, table, n, return_lse=True)
    assert kv.status() == dlp.PROJ_ERR_INVALID_ARG
    plain, plain_lse = kv.attend(q, table, n, return_lse=True)
    assert (out[1] == 0).all() and (lse[1] == -math.inf).all()
    ku.check_attention(out, lse, shared64(q, kv.k_cache, kv.v_cache, good, 700, table, [20, 0], 16, 0.125, keep=lambda t: t < 0))


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("size", [1.0, 30.0])
def test_beginnings_on_bad_pages(dtype, size):
    # No token in the first tiles of a CTA's stretch, and logits far below and above 0 in the others.
    import torch
    import dense_linear_projection_gb300 as dlp
    for prefix_len, batch in ((2000, 5), (30000, 40)):
        kv, q, prefix, table, n, scales = case(prefix_len, [3] * batch, 8, 1, 128, 16, dtype=dtype, size=size)
        good = prefix.clone()
        prefix[:20] = -1
        prefix[60:70] = 2 ** 30
        out, lse = kv.attend_shared(q, prefix, prefix_len, table, n, return_lse=True)
        assert kv.status() == dlp.PROJ_ERR_INVALID_ARG
        ref = shared64(q, kv.k_cache, kv.v_cache, good, prefix_len, table, [3] * batch, 16, 128 ** -0.5, *scales,
                       keep=lambda t: (t // 16 >= 20) & ((t // 16 < 60) | (t // 16 >= 70)))
        ku.check_attention(out, lse, ref)


@pytest.mark.parametrize("shift", [-300.0, 300.0])
def test_logits_far_from_zero(shift):
    # Every logit shifted by one element that all queries and keys share: far beyond what 2^x holds.
    kv, q, prefix, table, n, _ = case(5000, [40, 0, 7], 8, 2, 64, 16)
    q[..., 0] = 16
    kv.k_cache[..., 0] = shift / 2
    kv.k_cache[prefix[100].item(), 3, :, 0] = 0
    for scale in (0.125, 1.0):
        out, lse = kv.attend_shared(q, prefix, 5000, table, n, scale=scale, return_lse=True)
        ku.check_attention(out, lse, shared64(q, kv.k_cache, kv.v_cache, prefix, 5000, table, [40, 0, 7], 16, scale))


def test_many_stretches_a_block():
    # More than 63 stretches of row tiles a thread block, of which those of a growing prefix are done again.
    import torch
    import dense_linear_projection_gb300 as dlp
    B, hk, D, page, prefix_len = 39500, 32, 16, 16, 200
    k_cache, v_cache = ku.make_cache(20, page, hk, D)
    prefix = torch.randperm(20).to(torch.int32).cuda()
    at = torch.arange(prefix_len, device="cuda")
    k_cache[prefix.long()[at[128:] // page], at[128:] % page, ::3] *= 60  # past the first tile, every third key head
    q = torch.randn((B, hk, D), device="cuda").to(torch.bfloat16)
    kv = dlp.PagedKV(k_cache, v_cache, hk, B)
    n, table = torch.zeros(B, dtype=torch.int32, device="cuda"), torch.zeros((B, 0), dtype=torch.int32, device="cuda")
    out, lse = kv.attend_shared(q, prefix, prefix_len, table, n, return_lse=True)
    assert kv.status() == dlp.PROJ_OK
    k, v = (ku.tokens_of(c, prefix[None], 0, 0, prefix_len, page) for c in (k_cache, v_cache))
    for j in range(hk):
        x = q[:, j].double()
        s = x @ k[:, j].t() / 4
        a = (x.abs() @ k[:, j].abs().t()).amax(1) / 4
        p = torch.softmax(s, 1)
        rel = 2 * (D / 16 + 8) * 2.0 ** -22 * a + 2.0 ** -20 + (prefix_len / 8 + 64) * 2.0 ** -22
        over = ku.beyond(out[:, j], p @ v[:, j], (p @ v[:, j].abs()) * rel[:, None] + 1e-38)
        assert (over <= 0).all(), (j, over.max().item())
        want = torch.logsumexp(s, 1)
        assert ((lse[:, j].double() - want).abs() <= rel + 2.0 ** -22 * want.abs()).all(), j


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
def test_a_million_tokens(dtype):
    run(1000003, [0, 70], 4, 1, 64, 16, dtype=dtype)


def test_strided_queries_and_outputs():
    import torch
    kv, q, prefix, table, n, _ = case(600, [20, 0, 9], 8, 2, 64, 16)
    want = kv.attend_shared(q, prefix, 600, table, n)
    rows = torch.zeros((3, 20, 64), dtype=torch.bfloat16, device="cuda")
    rows[:, 3:11] = q
    to = torch.full((3, 24, 64), 5.0, dtype=torch.bfloat16, device="cuda")
    got = kv.attend_shared(rows[:, 3:11], prefix, 600, table, n, out=to[:, 8:16])
    assert got.data_ptr() == to[:, 8:16].data_ptr() and torch.equal(to[:, 8:16], want)
    assert (to[:, :8] == 5).all() and (to[:, 16:] == 5).all()


def test_cache_offsets_past_31_bits():
    import torch
    import dense_linear_projection_gb300 as dlp
    stride, hk, dim = 1 << 26, 2, 64
    base = [torch.zeros(stride * 43 + 16 * hk * dim, dtype=torch.bfloat16, device="cuda") for _ in "kv"]
    k_cache, v_cache = (x.as_strided((44, 16, hk, dim), (stride, hk * dim, dim, 1)) for x in base)
    for c in (k_cache, v_cache):
        c[43], c[2] = torch.randn((16, hk, dim), device="cuda"), torch.randn((16, hk, dim), device="cuda")
    kv = dlp.PagedKV(k_cache, v_cache, 8, 1)
    q = torch.randn((1, 8, dim), device="cuda").to(torch.bfloat16)
    ints = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    out, lse = kv.attend_shared(q, ints(43, 2), 29, ints(2)[None], ints(0), return_lse=True)
    ku.check_attention(out, lse, shared64(q, k_cache, v_cache, ints(43, 2), 29, ints(2)[None], [0], 16, 0.125))


def test_reruns_graphs_and_other_work():
    # The same bits every time: eagerly, replayed, beside work on another stream, and with another
    # prefix length or batch in between.
    import torch
    import dense_linear_projection_gb300 as dlp
    kv, q, prefix, table, n, _ = case(9000, [50, 0, 777, 13] * 8, 32, 4, 128, 16)
    want, want_lse = kv.attend_shared(q, prefix, 9000, table, n, return_lse=True)
    side = torch.cuda.Stream()
    a = torch.randn((4096, 4096), device="cuda", dtype=torch.bfloat16)
    with torch.cuda.stream(side):
        for _ in range(30):
            a @ a
    for _ in range(20):
        out, lse = kv.attend_shared(q, prefix, 9000, table, n, return_lse=True)
        kv.attend_shared(q[:3], prefix, 100, table[:3], n[:3])
        assert torch.equal(out, want) and torch.equal(lse, want_lse)
    torch.cuda.synchronize()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, lse = kv.attend_shared(q, prefix, 9000, table, n, return_lse=True)
    for _ in range(3):
        out.zero_()
        graph.replay()
        assert torch.equal(out, want) and torch.equal(lse, want_lse)
    assert kv.status() == dlp.PROJ_OK
    n[:4] = torch.tensor([0, 9, 776, 1], dtype=torch.int32)  # (the second has no page of its own: left out, and told)
    graph.replay()
    again, _ = kv.attend_shared(q, prefix, 9000, table, n, return_lse=True)
    assert torch.equal(out, again)
    with torch.cuda.stream(side):
        third = kv.attend_shared(q, prefix, 9000, table, n)
    side.synchronize()
    assert torch.equal(third, again) and kv.status() == dlp.PROJ_ERR_INVALID_ARG


def test_no_prefix_is_attend():
    import torch
    kv, q, prefix, table, n, _ = case(0, [50, 0, 777], 8, 2, 128, 16)
    out, lse = kv.attend_shared(q, prefix, 0, table, n, return_lse=True)
    want, want_lse = kv.attend(q, table, n, return_lse=True)
    assert torch.equal(out, want) and torch.equal(lse, want_lse)


def test_refusals():
    import torch
    import dense_linear_projection_gb300 as dlp
    kv, q, prefix, table, n, _ = case(100, [20, 7], 8, 2, 64, 16)
    good = dict(q=q, prefix_pages=prefix, prefix_len=100, page_table=table, seq_lens=n)
    for change in (dict(prefix_len=-1), dict(prefix_len=prefix.numel() * 16 + 1), dict(prefix_pages=prefix.long()), dict(prefix_pages=prefix.cpu()),
                   dict(prefix_pages=prefix[None]), dict(prefix_pages=prefix[::2]), dict(prefix_pages=None), dict(prefix_len=3.5),
                   dict(scale=math.nan), dict(q=q[:1]), dict(seq_lens=n.long()), dict(page_table=table[:1]), dict(out=q[:1]),
                   dict(q=torch.cat([q, q]), page_table=torch.cat([table, table]), seq_lens=torch.cat([n, n]))):
        with pytest.raises((dlp.ProjError, TypeError)) as e:
            kv.attend_shared(**{**good, **change})
        assert not isinstance(e.value, dlp.ProjError) or e.value.status == dlp.PROJ_ERR_INVALID_ARG, change
    assert kv.attend_shared(q[:0], prefix, 100, table[:0], n[:0]).shape == (0, 8, 64)
    # No pages of their own.
    out, lse = kv.attend_shared(q, prefix, 100, table[:, :0], n * 0, return_lse=True)
    ku.check_attention(out, lse, shared64(q, kv.k_cache, kv.v_cache, prefix, 100, table, [0, 0], 16, 0.125))
    assert kv.status() == dlp.PROJ_OK
    kv.close()
    with pytest.raises(dlp.ProjError):
        kv.attend_shared(**good)
