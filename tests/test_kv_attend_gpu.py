"""Attention of one new token of each sequence over the paged cache, against 64 bits (the bounds
are derived in kv_util.attention64)."""
import math

import pytest

import kv_util as ku

pytestmark = pytest.mark.gpu


def case(lens, heads, kv_heads, dim, page, dtype="bf16", layout="tokens_first", seed=0, unused=0):
    import torch
    import dense_linear_projection_gb300 as dlp
    pages = sum(-(-n // page) for n in lens) + 3
    k, v = ku.make_cache(pages, page, kv_heads, dim, dtype, layout, seed)
    table = ku.make_table(lens, page, pages, seed, unused=unused)
    g = torch.Generator(device="cuda")
    g.manual_seed(seed + 1)
    q = torch.randn((len(lens), heads, dim), generator=g, device="cuda").to(torch.bfloat16)
    scales = [torch.rand(kv_heads, generator=g, device="cuda") + 0.5 for _ in "kv"] if dtype == "e4m3" else [None, None]
    kv = dlp.PagedKV(k, v, heads, max_sequences=len(lens), k_scale=scales[0], v_scale=scales[1])
    return kv, q, table, torch.tensor(lens, dtype=torch.int32, device="cuda")


def run(lens, heads, kv_heads, dim, page, window=0, scale=None, **more):
    import torch
    kv, q, table, lens_dev = case(lens, heads, kv_heads, dim, page, **more)
    out, lse = kv.attend(q, table, lens_dev, scale=scale, window=window, return_lse=True)
    ref = ku.attention64(q, kv.k_cache, kv.v_cache, table, lens, page, scale or dim ** -0.5, window, kv.k_scale, kv.v_scale)
    what = f"lens={lens[:8]} heads={heads}/{kv_heads} dim={dim} page={page} window={window} {more}"
    ku.check_attention(out, lse, ref, what)
    again, lse2 = kv.attend(q, table, lens_dev, scale=scale, window=window, return_lse=True)
    assert torch.equal(again, out) and torch.equal(lse2, lse), what
    import dense_linear_projection_gb300 as dlp
    assert kv.status() == dlp.PROJ_OK


@pytest.mark.parametrize("lens", [[1], [0], [2, 0, 1], [15, 16, 17], [63, 64, 65], [127, 128, 129], [1000, 0, 3, 4097],
                                  [37] * 33, [20000], [1, 9000, 1, 1]], ids=str)
@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
def test_lengths(lens, dtype):
    run(lens, 16, 4, 128, 16, dtype=dtype)


@pytest.mark.parametrize("heads,kv_heads", [(1, 1), (8, 8), (2, 1), (6, 2), (14, 2), (16, 2), (32, 2), (20, 1), (96, 2), (64, 8), (40, 40)])
@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
def test_head_groups(heads, kv_heads, dtype):
    run([300, 5, 77], heads, kv_heads, 64, 16, dtype=dtype)


@pytest.mark.parametrize("heads,kv_heads", [(32, 2), (24, 2), (4, 4), (18, 6), (16, 1)])
@pytest.mark.parametrize("dtype,dim", [("e4m3", 128), ("e4m3", 96), ("bf16", 64), ("bf16", 128)])
def test_pairs_of_key_heads(heads, kv_heads, dtype, dim):
    # Short rows of memory are taken two key heads at a time, where those are even.
    run([700, 1, 0, 130], heads, kv_heads, dim, 16, dtype=dtype)
    run([2500], heads, kv_heads, dim, 16, dtype=dtype, window=900)


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
def test_nan_and_infinity_stay_with_their_heads(dtype):
    # A NaN in one sequence's keys of one head makes that head's outputs and sums NaN, no others.
    import torch
    lens, page = [900, 40], 16
    kv, q, table, lens_dev = case(lens, 8, 4, 64, page, dtype=dtype)
    ref = ku.attention64(q, kv.k_cache, kv.v_cache, table, lens, page, 64 ** -0.5, 0, kv.k_scale, kv.v_scale)
    raw = kv.k_cache.view(torch.uint8) if dtype == "e4m3" else kv.k_cache
    raw[table[0, 20].long(), 3, 2, 5] = 0x7F if dtype == "e4m3" else math.nan
    out, lse = kv.attend(q, table, lens_dev, return_lse=True)
    hit = torch.zeros((2, 8), dtype=torch.bool, device="cuda")
    hit[0, 4:6] = True  # two query heads to a key head
    assert torch.equal(out.isnan().all(2), hit) and torch.equal(out.isnan().any(2), hit) and torch.equal(lse.isnan(), hit)
    out, lse = out.masked_fill(hit[..., None], 0), lse.masked_fill(hit, 0)
    want, want_lse, lim, lim_lse = ref
    ku.check_attention(out, lse, (want.masked_fill(hit[..., None], 0), want_lse.masked_fill(hit, 0), lim, lim_lse), "others")


@pytest.mark.parametrize("dim", [16, 32, 48, 64, 80, 96, 128, 144, 192, 256])
@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
def test_head_dims(dim, dtype):
    run([200, 33], 8, 2, dim, 16, dtype=dtype)


@pytest.mark.parametrize("page", [1, 2, 3, 7, 16, 17, 64, 100, 300])
@pytest.mark.parametrize("layout", ["tokens_first", "heads_first", "together"])
def test_pages_and_layouts(page, layout):
    run([301, 2, 64], 8, 2, 64, page, layout=layout)
    run([301, 2, 64], 8, 2, 64, page, layout=layout, dtype="e4m3")


@pytest.mark.parametrize("window", [1, 15, 16, 100, 300, 5000])
def test_windows(window):
    run([301, 0, 16, 2000, 1], 8, 4, 128, 16, window=window)
    run([301, 0, 16, 2000, 1], 8, 4, 128, 16, window=window, dtype="e4m3")


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("lens,heads,kv_heads,dim", [([30000], 8, 1, 128), ([100, 40000, 3], 4, 1, 64), ([9000, 17000], 16, 1, 128), ([15000], 8, 1, 256)])
def test_rows_of_many_parts(lens, heads, kv_heads, dim, dtype):
    # One key head: a row is shared by up to every CTA of the launch, and its parts are joined in groups.
    run(lens, heads, kv_heads, dim, 16, dtype=dtype)


def test_scales():
    for scale in (1.0, -0.2, 1e-6, 0.0):
        import torch
        kv, q, table, lens = case([70, 9], 8, 2, 64, 16)
        out, lse = kv.attend(q, table, lens, scale=scale, return_lse=True)
        ref = ku.attention64(q, kv.k_cache, kv.v_cache, table, [70, 9], 16, scale)
        ku.check_attention(out, lse, ref, f"scale={scale}")


def test_wide_logits():
    # Logits hundreds apart: one token takes all the weight, wherever it is.
    import torch
    kv, q, table, lens = case([500] * 4, 8, 2, 64, 16)
    q *= 40
    out, lse = kv.attend(q, table, lens, return_lse=True)
    ku.check_attention(out, lse, ku.attention64(q, kv.k_cache, kv.v_cache, table, [500] * 4, 16, 64 ** -0.5), "wide")


def test_extreme_queries_over_8_bits():
    # Queries of any bf16 size: the 8-bit path must not lose or overflow them.
    import torch
    kv, q, table, lens = case([100] * 2, 4, 2, 64, 16, dtype="e4m3")
    for size in (1e30, 1e-30):
        x = (q.float() * size).to(torch.bfloat16)
        out, lse = kv.attend(x, table, lens, scale=0.125 / size, return_lse=True)
        ref = ku.attention64(x, kv.k_cache, kv.v_cache, table, [100] * 2, 16, 0.125 / size, 0, kv.k_scale, kv.v_scale)
        ku.check_attention(out, lse, ref, f"size={size}")


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("window", [0, 20])
def test_nothing_outside_the_sequences_is_used(dtype, window):
    # Every place no sequence sees holds NaN, and the table's unused entries are no pages at all.
    import torch
    import dense_linear_projection_gb300 as dlp
    lens, page, dim = [45, 0, 130, 1], 16, 64
    kv, q, table, lens_dev = case(lens, 8, 2, dim, page, dtype=dtype, unused=-7)
    ref = ku.attention64(q, kv.k_cache, kv.v_cache, table, lens, page, dim ** -0.5, window, kv.k_scale, kv.v_scale)
    seen = torch.zeros(kv.k_cache.shape[:2], dtype=torch.bool, device="cuda")
    for b, n in enumerate(lens):
        t = torch.arange(max(0, n - window) if window else 0, n, device="cuda")
        seen[table[b].long()[t // page], t % page] = True
        if window:  # pages wholly before the window are not read either
            table[b, :max(0, n - window) // page] = 1 << 30
    for c in (kv.k_cache, kv.v_cache):
        raw = c.view(torch.uint8) if dtype == "e4m3" else c
        raw[~seen] = 0x7F if dtype == "e4m3" else math.nan
    out, lse = kv.attend(q, table, lens_dev, window=window, return_lse=True)
    ku.check_attention(out, lse, ref, "poisoned")
    assert kv.status() == dlp.PROJ_OK


def test_strided_queries_and_outputs():
    # Queries inside the rows of a query, key and value projection, outputs inside wider rows.
    import torch
    kv, q, table, lens = case([90, 33, 4], 8, 2, 64, 16)
    rows = torch.randn((3, 12, 64), device="cuda").to(torch.bfloat16)
    rows[:, :8] = q
    wide = torch.full((3, 11, 64), 7.0, device="cuda", dtype=torch.bfloat16)
    out = kv.attend(rows[:, :8], table, lens, out=wide[:, :8])
    assert torch.equal(out, kv.attend(q, table, lens)) and (wide[:, 8:] == 7).all()


def test_cache_offsets_past_31_bits():
    # Pages far apart: element offsets above 2³¹ in each array.
    import torch
    import dense_linear_projection_gb300 as dlp
    lens, page, hk, dim = [700], 16, 2, 64
    stride = 1 << 26
    base = [torch.empty(stride * 43 + page * hk * dim, dtype=torch.bfloat16, device="cuda") for _ in "kv"]
    k, v = (x.as_strided((44, page, hk, dim), (stride, hk * dim, dim, 1)) for x in base)
    for x in (k, v):
        x.copy_(torch.randn(x.shape, device="cuda"))
    table = torch.randperm(44).to(torch.int32)[None].cuda()
    q = torch.randn((1, 8, dim), device="cuda").to(torch.bfloat16)
    kv = dlp.PagedKV(k, v, 8, 1)
    out, lse = kv.attend(q, table, torch.tensor(lens, dtype=torch.int32, device="cuda"), return_lse=True)
    ku.check_attention(out, lse, ku.attention64(q, k, v, table, lens, page, dim ** -0.5), "far pages")


def test_streams_graphs_and_shrinking_lengths():
    # A captured call follows the lengths and tables that the buffers hold at replay.
    import torch
    lens = [800, 40, 1500, 0]
    kv, q, table, lens_dev = case(lens, 16, 2, 128, 16)
    ref = kv.attend(q, table, lens_dev)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = kv.attend(q, table, lens_dev)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(other, ref)
    g, out = torch.cuda.CUDAGraph(), torch.empty_like(ref)
    with torch.cuda.graph(g):
        kv.attend(q, table, lens_dev, out=out)
    for now in ([800, 40, 1500, 0], [1, 0, 1499, 5], [0, 0, 0, 0], [799, 39, 3, 0]):
        now[3] = min(now[3], 0)  # the last sequence has no pages of its own
        lens_dev.copy_(torch.tensor(now, dtype=torch.int32))
        g.replay()
        torch.cuda.synchronize()
        ku.check_attention(out, None, ku.attention64(q, kv.k_cache, kv.v_cache, table, now, 16, 128 ** -0.5), str(now))


def test_bad_pages_and_lengths_are_reported_and_left_out():
    import torch
    import dense_linear_projection_gb300 as dlp
    lens, page = [100, 64], 16
    kv, q, table, lens_dev = case(lens, 8, 2, 64, page)
    good = table.clone()
    table[0, 2], table[1, 0] = kv.k_cache.shape[0], -1
    out, lse = kv.attend(q, table, lens_dev, return_lse=True)
    assert kv.status() == dlp.PROJ_ERR_INVALID_ARG and kv.status() == dlp.PROJ_OK
    keep = lambda b, t: (t // page != 2) if b == 0 else (t // page != 0)  # noqa: E731
    ref = ku.attention64(q, kv.k_cache, kv.v_cache, good, lens, page, 64 ** -0.5, keep=keep)
    ku.check_attention(out, lse, ref, "bad pages")
    # A sequence whose every page is bad is an empty row.
    table.fill_(-1)
    out, lse = kv.attend(q, table, lens_dev, return_lse=True)
    assert (out == 0).all() and (lse == -math.inf).all() and kv.status() == dlp.PROJ_ERR_INVALID_ARG
    # Lengths past the table (cut to it) and below zero (an empty row).
    full = good.shape[1] * page
    pages = torch.randperm(kv.k_cache.shape[0], device="cuda").to(torch.int32)[:good.shape[1]]
    both = pages.expand(2, -1).contiguous()
    out, lse = kv.attend(q, both, torch.tensor([full + 9, -3], dtype=torch.int32, device="cuda"), return_lse=True)
    assert kv.status() == dlp.PROJ_ERR_INVALID_ARG
    ku.check_attention(out, lse, ku.attention64(q, kv.k_cache, kv.v_cache, both, [full, 0], page, 64 ** -0.5), "bad lengths")


def test_empty_batch_and_empty_table():
    import torch
    kv, q, table, lens = case([5, 5], 8, 2, 64, 16)
    assert kv.attend(q[:0], table[:0], lens[:0]).shape == (0, 8, 64)
    out, lse = kv.attend(q, torch.empty((2, 0), dtype=torch.int32, device="cuda"), torch.zeros_like(lens), return_lse=True)
    assert (out == 0).all() and (lse == -math.inf).all()


def test_refusals():
    import torch
    import dense_linear_projection_gb300 as dlp
    kv, q, table, lens = case([50, 20], 8, 2, 64, 16)
    k, v = kv.k_cache, kv.v_cache
    invalid, unsupported, misaligned = dlp.PROJ_ERR_INVALID_ARG, dlp.PROJ_ERR_UNSUPPORTED, dlp.PROJ_ERR_MISALIGNED
    for what, status in [
        (lambda: kv.attend(torch.cat([q, q]), torch.cat([table, table]), torch.cat([lens, lens])), invalid),
        (lambda: kv.attend(q.float(), table, lens), invalid),
        (lambda: kv.attend(q[:, :4], table, lens), invalid),
        (lambda: kv.attend(q, table.long(), lens), invalid),
        (lambda: kv.attend(q, table[:1], lens), invalid),
        (lambda: kv.attend(q, table, lens[:1]), invalid),
        (lambda: kv.attend(q, table, lens, window=-1), invalid),
        (lambda: kv.attend(q, table, lens, scale=math.nan), invalid),
        (lambda: dlp.PagedKV(k, v, 7, 2), invalid),                                  # heads not a multiple
        (lambda: dlp.PagedKV(k, v[:1], 8, 2), invalid),
        (lambda: dlp.PagedKV(k.float(), v.float(), 8, 2), unsupported),
        (lambda: dlp.PagedKV(k[..., :40], v[..., :40], 8, 2), unsupported),
        (lambda: dlp.PagedKV(*ku.make_cache(4, 16, 1, 272), 1, 2), unsupported),
        (lambda: dlp.PagedKV(k, v, 8, 2, k_scale=torch.ones(2, device="cuda")), invalid),
        (lambda: dlp.proj_kv_attend(kv.handle, 2, q.data_ptr() + 2, 512, k, v, None, None, table, table.shape[1], lens, 0,
                                    1.0, q, 512, None), misaligned),
        (lambda: dlp.proj_kv_attend(kv.handle, 2, q, 512, None, v, None, None, table, table.shape[1], lens, 0, 1.0, q,
                                    512, None), invalid),
        (lambda: dlp.proj_kv_attend(kv.handle, 2, q, 512, k, v, None, None, table, (1 << 31) // 16, lens, 0, 1.0, q, 512,
                                    None), invalid),                             # more tokens than 32 bits count
        (lambda: dlp.proj_kv_attend(None, 2, q, 512, k, v, None, None, table, table.shape[1], lens, 0, 1.0, q, 512,
                                    None), invalid),
    ]:
        with pytest.raises(dlp.ProjError) as e:
            what()
        assert e.value.status == status


@pytest.mark.parametrize("nats", [3, 8, 12, 15, 17.5, 20, 24])
@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
def test_small_weights_count(dtype, nats):
    # One token takes the largest weight and has the value 0; all others lie e^-nats below it and are all of
    # the output.  The bound holds each weight to 2⁻¹⁶ of itself (e4m3: down to 2⁻³⁶ = e^-24.9 of the largest).
    import torch
    for lens, at, heads, kv_heads, dim in (([4000, 40], 0, 8, 2, 64), ([4000, 33], 3999, 16, 1, 128), ([9000], 100, 4, 1, 256)):
        kv, q, table, lens_dev = case(lens, heads, kv_heads, dim, 16, dtype=dtype)
        q.zero_()
        q[..., 3] = 1
        raw = lambda c: c.view(torch.uint8) if dtype == "e4m3" else c  # noqa: E731
        raw(kv.k_cache).zero_()
        key = torch.zeros((kv_heads, dim), device="cuda")
        key[:, 3] = 16
        for b, n in enumerate(lens):
            page, place = table[b, min(at, n - 1) // 16].long(), min(at, n - 1) % 16
            raw(kv.k_cache)[page, place] = raw(key.to(kv.k_cache.dtype))
            raw(kv.v_cache)[page, place] = 0
        if kv.k_scale is not None:
            kv.k_scale.fill_(1.0)
        out, lse = kv.attend(q, table, lens_dev, scale=nats / 16, return_lse=True)
        ref = ku.attention64(q, kv.k_cache, kv.v_cache, table, lens, 16, nats / 16, 0, kv.k_scale, kv.v_scale)
        ku.check_attention(out, lse, ref, f"{nats} nats, {lens}")


@pytest.mark.parametrize("power", [10, 16, 22])
@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
def test_queries_of_unequal_elements(dtype, power):
    # One element of each query is 2^power, against keys that are 0 there: the others make the logits.
    import torch
    lens = [300, 20]
    for dim in (64, 128, 256):
        kv, q, table, lens_dev = case(lens, 8, 2, dim, 16, dtype=dtype)
        q[..., 5] = 2.0 ** power
        raw = kv.k_cache.view(torch.uint8) if dtype == "e4m3" else kv.k_cache
        raw[..., 5] = 0
        out, lse = kv.attend(q, table, lens_dev, return_lse=True)
        ref = ku.attention64(q, kv.k_cache, kv.v_cache, table, lens, 16, dim ** -0.5, 0, kv.k_scale, kv.v_scale)
        ku.check_attention(out, lse, ref, f"2^{power}, {dim}")


def test_queries_at_the_ends_of_bf16_over_8_bits():
    # The largest and the smallest bf16 queries, subnormal ones among them.
    import torch
    kv, q, table, lens = case([100] * 2, 4, 2, 64, 16, dtype="e4m3")
    for size, scale in ((2.0 ** 125, 2.0 ** -126), (2.0 ** -124, 2.0 ** 121), (2.0 ** -130, 2.0 ** 122)):
        x = (q.float() * size).to(torch.bfloat16)
        out, lse = kv.attend(x, table, lens, scale=scale, return_lse=True)
        ref = ku.attention64(x, kv.k_cache, kv.v_cache, table, [100] * 2, 16, scale, 0, kv.k_scale, kv.v_scale)
        ku.check_attention(out, lse, ref, f"size={size}")


@pytest.mark.parametrize("lens", [[1, 17], [900, 40], [20000], [130] * 40], ids=lambda x: f"{len(x)}x{x[0]}")
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_infinite_values(lens, dim):
    # An infinite value makes its element of its heads infinite, two of both signs or a NaN make it NaN.
    import torch
    kv, q, table, lens_dev = case(lens, 8, 4, dim, 16)
    ref = ku.attention64(q, kv.k_cache, kv.v_cache, table, lens, 16, dim ** -0.5)
    last = lens[0] - 1
    kv.v_cache[table[0, last // 16].long(), last % 16, 2, 5:9] = torch.tensor([math.inf, -math.inf, math.nan, math.inf], device="cuda").to(torch.bfloat16)
    kv.v_cache[table[0, 0].long(), 0, 2, 8] = -math.inf
    out, lse = kv.attend(q, table, lens_dev, return_lse=True)
    got = out[0, 4:6, 5:9].clone()
    assert (got[:, 0] == math.inf).all() and (got[:, 1] == -math.inf).all() and got[:, 2].isnan().all()
    assert got[:, 3].isnan().all() if lens[0] > 1 else (got[:, 3] == -math.inf).all()
    out[0, 4:6, 5:9] = ref[0][0, 4:6, 5:9].to(torch.bfloat16)
    ku.check_attention(out, lse, ref, "the others")


def test_infinite_keys():
    # A logit of -inf has no weight; one of +inf makes its heads' outputs NaN, as in the definition.
    import torch
    lens, dim = [700, 30], 64
    kv, q, table, lens_dev = case(lens, 8, 4, dim, 16)
    q[0, 4:6, 7] = 1
    ref = ku.attention64(q, kv.k_cache, kv.v_cache, table, lens, 16, dim ** -0.5, keep=lambda b, t: (t != 650) | (b != 0))
    whole = ku.attention64(q, kv.k_cache, kv.v_cache, table, lens, 16, dim ** -0.5)
    page = table[0, 650 // 16].long()
    kv.k_cache[page, 650 % 16, 2, 7] = -math.inf
    out, lse = kv.attend(q, table, lens_dev, return_lse=True)
    mixed = [w.clone() for w in whole]
    for m, r in zip(mixed, ref):
        m[0, 4:6] = r[0, 4:6]
    ku.check_attention(out, lse, mixed, "-inf")
    kv.k_cache[page, 650 % 16, 2, 7] = math.inf
    out, lse = kv.attend(q, table, lens_dev, return_lse=True)
    assert out[0, 4:6].isnan().all() and lse[0, 4:6].isnan().all()
    out[0, 4:6], lse[0, 4:6] = whole[0][0, 4:6].to(torch.bfloat16), whole[1][0, 4:6].float()
    ku.check_attention(out, lse, whole, "+inf")


@pytest.mark.parametrize("B,n,heads,kv_heads", [(3, 5000, 64, 8), (33, 9600, 8, 1), (4, 30000, 16, 1)])
def test_reruns_beside_other_work(B, n, heads, kv_heads):
    # Bit-identical whichever CTA joins a row: copies on another stream change the order of arrival, the
    # second half's values are the first's with the other sign (what is left of the sums is their rounding),
    # and the last token's logit is the largest, so that a later part has the maximum.
    import torch
    kv, q, table, lens = case([n] * B, heads, kv_heads, 128, 16)
    t, half = torch.arange(n, device="cuda"), n // 2
    for b in range(B):
        pages = table[b].long()[t // 16]
        k, v = kv.k_cache[pages, t % 16], kv.v_cache[pages, t % 16]
        k[half:2 * half], v[half:2 * half] = k[:half], -v[:half]
        k[..., 0] = k[-1] = 0
        k[-1, :, 0] = 30
        v[-1] = v[half - 1] = 0
        kv.k_cache[pages, t % 16], kv.v_cache[pages, t % 16] = k, v
    q[..., 0] = 2
    first, lse0 = kv.attend(q, table, lens, return_lse=True)
    side, a = torch.cuda.Stream(), torch.empty(1 << 28, device="cuda", dtype=torch.uint8)
    c = torch.empty_like(a)
    differ = torch.zeros((), dtype=torch.int64, device="cuda")
    for i in range(400):
        with torch.cuda.stream(side):
            c[:1 << (20 + i % 9)].copy_(a[:1 << (20 + i % 9)])
        out, lse = kv.attend(q, table, lens, return_lse=True)
        differ += (out != first).any() | (lse != lse0).any()
    assert differ.item() == 0


def test_truth_values_that_have_none():
    # What an argument's own test raises comes out, before anything is launched.
    import torch

    class Neither:
        def __bool__(self):
            raise ValueError("neither")

    kv, q, table, lens = case([5, 5], 8, 2, 64, 16)
    out = torch.full_like(q, 7.0)
    with pytest.raises(ValueError, match="neither"):
        kv.attend(q, table, lens, out=out, return_lse=Neither())
    with pytest.raises(ValueError, match="neither"):
        kv.append(q, q[:, :2], q[:, 2:4], lens, table, interleaved=Neither(), q_out=out)
    assert (out == 7).all()


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
def test_weights_are_held_as_fp32(dtype):
    # Two tokens of nearly equal weight and opposite values: the output is their weights' difference.
    # Logits are at most 2⁻³ and exact but for the scale (2⁻²³ of them); the exponential's 2⁻²¹, the weights'
    # parts 2⁻²³, three 16-token products and a sum 2⁻²² each and the division 2⁻²³ stay below 2⁻¹⁹ of Σ w|v|,
    # which is 1.  (With 16 bits a weight: 2⁻¹⁷.)
    import torch
    lens, heads, kv_heads, dim = [2] * 16, 64, 8, 64
    kv, q, table, lens_dev = case(lens, heads, kv_heads, dim, 16, dtype=dtype)
    raw = lambda c: c.view(torch.uint8) if dtype == "e4m3" else c  # noqa: E731
    raw(kv.k_cache).zero_()
    plus, minus = (raw(torch.full((), x, device="cuda").to(kv.k_cache.dtype)) for x in (1.0, -1.0))
    step = 2.0 ** -6 if dtype == "e4m3" else 2.0 ** -11
    if dtype == "e4m3":
        kv.k_scale.fill_(2.0 ** -5)
        kv.v_scale.fill_(1.0)
    for b in range(16):
        page = table[b, 0].long()
        keys = torch.zeros((kv_heads, dim), device="cuda")
        keys[:, 0] = (torch.arange(kv_heads, device="cuda") + 1 + b % 8) * step
        raw(kv.k_cache)[page, 0] = raw(keys.to(kv.k_cache.dtype))
        raw(kv.v_cache)[page, 0], raw(kv.v_cache)[page, 1] = plus, minus
    q.zero_()
    q[..., 0] = (1 + torch.arange(heads, device="cuda") / 64)[None]
    out = kv.attend(q, table, lens_dev, scale=1.0)
    want, _, _, _ = ku.attention64(q, kv.k_cache, kv.v_cache, table, lens, 16, 1.0, 0, kv.k_scale, kv.v_scale)
    over = ku.beyond(out, want, 2.0 ** -19)
    assert (over <= 0).all(), f"{int((over > 0).sum())} of {out.numel()} beyond the bound, by up to {over.max().item():.3e}"
