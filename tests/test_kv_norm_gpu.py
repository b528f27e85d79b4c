"""Append with the norm of each head before the rotation, and rotary rows of their own.

Against 64 bits.  In units u = 2⁻²⁴ of the value: the sum of squares has 16 products and additions
in a lane and at most 5 across lanes, 21 u, which its root halves; the division by head_dim, the
addition of eps, the root and the reciprocal round once each (their errors enter by a half or by one):
15 u at most; three products with the element 3 u; scaled heads two more.  So a normed element is within
20 u, and a rotated one, two products and a sum more, within 23 u of |a·cos| + |b·sin|: below 2⁻¹⁹ of it.
The division by an 8-bit cache's scale is one more u.  Then one rounding to the type written."""
import math

import pytest

import kv_util as ku

pytestmark = pytest.mark.gpu


def normed64(x, weight, eps, rope_rows, interleaved):
    """(y, absolute terms) [tokens, heads, dim] in 64 bits; weight or rope_rows may be None."""
    import torch
    x = x.double()
    if weight is not None:
        x = x * weight.double() / torch.sqrt(x.square().mean(-1, keepdim=True) + eps)
    y, terms = x.clone(), x.abs()
    if rope_rows is not None:
        rot = rope_rows.shape[1]
        cos, sin = rope_rows.double()[:, None].split(rot // 2, -1)
        first, second = (slice(0, rot, 2), slice(1, rot, 2)) if interleaved else (slice(0, rot // 2), slice(rot // 2, rot))
        a, b = x[..., first], x[..., second]
        y[..., first], y[..., second] = a * cos - b * sin, b * cos + a * sin
        terms[..., first] = (a * cos).abs() + (b * sin).abs()
        terms[..., second] = (b * cos).abs() + (a * sin).abs()
    return y, terms


def run(tokens, heads, kv_heads, dim, page, rot, interleaved=False, dtype="bf16", layout="tokens_first", weights="bf16",
        norms="qk", rows=True, eps=1e-6, in_place=False, size=1.0, q_given=True, rows_of=None, seed=0):
    import torch
    import dense_linear_projection_gb300 as dlp
    g = torch.Generator()
    g.manual_seed(seed)
    sequences = 3
    per = -(-tokens // sequences) + 5
    spots = torch.randperm(sequences * per, generator=g)[:tokens]
    seq, pos = (spots // per).to(torch.int32), (spots % per).to(torch.int32)
    if tokens > 2:
        pos[::3] = -1 - pos[::3]  # padding
    width = -(-per // page) + 1
    pages = sequences * width + 2
    k_cache, v_cache = ku.make_cache(pages, page, kv_heads, dim, dtype, layout, seed)
    table = torch.randperm(pages, generator=g)[:sequences * width].to(torch.int32).view(sequences, width)
    rope = dlp.rope_table(per + 700, rot) if rot else None
    rope_rows = torch.randint(0, per + 700, (tokens,), generator=g, dtype=torch.int32).cuda() if rot and rows else None
    scales = [torch.rand(kv_heads, generator=g).cuda() * 0.2 + 0.01 for _ in "kv"] if dtype == "e4m3" else [None, None]
    kind = torch.float32 if weights == "f32" else torch.bfloat16
    wq, wk = ((1 + 0.3 * torch.randn(dim, generator=g)).cuda().to(kind) if c in norms else None for c in "qk")
    kv = dlp.PagedKV(k_cache, v_cache, heads, 1, k_scale=scales[0], v_scale=scales[1])
    x = (torch.randn((tokens, heads + 2 * kv_heads, dim), generator=g) * size).cuda().to(torch.bfloat16)
    if rows_of is not None:
        rows_of(x)
    original = x.clone()
    q, k, v = x[:, :heads], x[:, heads:heads + kv_heads], x[:, heads + kv_heads:]
    before_k, before_v = k_cache.clone(), v_cache.clone()
    live = (pos >= 0).cuda()
    at = pos.cuda()[live].long()
    to, place = table.cuda()[seq.cuda()[live].long(), at // page].long(), at % page
    turn = rope[(rope_rows if rope_rows is not None else pos.cuda())[live].long()] if rot else None
    got = kv.append(q if q_given else None, k, v, pos.cuda(), table.cuda(), seq_ids=seq.cuda(), rope=rope, interleaved=interleaved,
                    q_out=q if in_place else None, q_norm=wq, k_norm=wk, eps=eps, rope_rows=rope_rows)
    assert kv.status() == dlp.PROJ_OK

    def check(have, ref, terms, what):
        # What is not finite in 64 bits has to be the same; the rest is within the bound.
        ref = ref.to(torch.float64)
        odd = ~torch.isfinite(ref)
        assert torch.equal(have.double()[odd].nan_to_num(7.0, 8.0, 9.0), ref[odd].nan_to_num(7.0, 8.0, 9.0)), what
        over = ku.beyond(have[~odd].float() if have.dtype == torch.float8_e4m3fn else have[~odd], ref[~odd], terms[~odd] * 2.0 ** -19 + 1e-40) \
            if have.dtype != torch.float8_e4m3fn else beyond8(have[~odd], ref[~odd], terms[~odd] * 2.0 ** -19)
        assert (over <= 0).all(), f"{what}: {int((over > 0).sum())} of {over.numel()}, by up to {over.max().item():.3e}"

    def beyond8(have, ref, lim):
        # Clamped, and in 32 bits first: the e4m3 values are some 2⁻⁴ apart.
        low, high = ((e.clamp(-448, 448).float().to(torch.float8_e4m3fn)).double() for e in (ref - lim - 1e-12, ref + lim + 1e-12))
        return torch.maximum(low - have.double(), have.double() - high)

    want_k, terms_k = normed64(original[:, heads:heads + kv_heads][live], wk, eps, turn, interleaved)
    want_v = original[:, heads + kv_heads:][live].double()
    if dtype == "e4m3":
        want_k, terms_k = want_k / scales[0].double()[:, None], terms_k / scales[0].double()[:, None]
        want_v = want_v / scales[1].double()[:, None]
    raw = lambda c: c.view(torch.uint8) if dtype == "e4m3" else c  # noqa: E731
    check(raw(k_cache)[to, place].view(k_cache.dtype), want_k, terms_k, "keys")
    check(raw(v_cache)[to, place].view(v_cache.dtype), want_v, want_v.abs(), "values")
    if q_given:
        assert got is q if in_place else got is not None
        check(got[live], *normed64(original[:, :heads][live], wq, eps, turn, interleaved), "queries")
        if in_place:
            assert torch.equal(got[~live], original[:, :heads][~live])
    # Nothing else is written.
    raw(k_cache)[to, place], raw(v_cache)[to, place] = raw(before_k)[to, place], raw(before_v)[to, place]
    bits = lambda c: c.contiguous().view(torch.uint8 if dtype == "e4m3" else torch.int16)  # noqa: E731
    assert torch.equal(bits(k_cache), bits(before_k)) and torch.equal(bits(v_cache), bits(before_v))
    assert torch.equal(x[:, heads:], original[:, heads:])


@pytest.mark.parametrize("tokens", [1, 2, 7, 300, 2111])
@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
def test_token_counts(tokens, dtype):
    run(tokens, 16, 4, 128, 16, 128, dtype=dtype)


@pytest.mark.parametrize("dim,rot", [(16, 16), (64, 64), (64, 32), (128, 64), (80, 80), (96, 48), (256, 256), (64, 0), (128, 2),
                                     (64, 20), (112, 110), (256, 250), (240, 16), (48, 32)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_dims_and_rotary_parts(dim, rot, interleaved):
    run(40, 6, 2, dim, 16, rot, interleaved)
    run(40, 6, 2, dim, 16, rot, interleaved, dtype="e4m3", weights="f32")


@pytest.mark.parametrize("norms", ["q", "k", "", "qk"])
@pytest.mark.parametrize("rows", [False, True])
def test_either_norm_and_rows(norms, rows):
    if norms or rows:
        run(50, 8, 2, 64, 16, 64, norms=norms, rows=rows)
        run(50, 8, 2, 64, 16, 64, norms=norms, rows=rows, in_place=True, weights="f32")
    run(20, 8, 2, 64, 16, 64, norms=norms.replace("q", ""), rows=rows, q_given=False)


@pytest.mark.parametrize("page", [1, 3, 64])
@pytest.mark.parametrize("layout", ["tokens_first", "heads_first", "together"])
def test_pages_and_layouts(page, layout):
    run(50, 8, 8, 64, page, 64, layout=layout)


def test_head_counts():
    for heads, kv_heads in ((1, 1), (7, 1), (71, 1), (64, 8), (48, 48)):
        run(9, heads, kv_heads, 128, 16, 128)


@pytest.mark.parametrize("power", [-133, -126, -100, -63, -40, -20, 0, 30, 60, 64, 100, 120])
@pytest.mark.parametrize("eps", [0.0, 1e-30, 1e-6, 1.0])
def test_sizes_of_heads(power, eps):
    # Squares below and above fp32's range, heads with one large element, heads of zeros.
    def rows_of(x):
        x[1::4] = 0
        x[2::4, :, 1:] = x[2::4, :, 1:] * 2.0 ** -12
    run(30, 4, 2, 128, 16, 128, size=2.0 ** power, eps=eps, rows_of=rows_of)
    run(30, 4, 2, 64, 16, 20, size=2.0 ** power, eps=eps, weights="f32", rows_of=rows_of)


def test_infinity_and_nan_stay_with_their_heads():
    def rows_of(x):
        x[1, :2, 3], x[2, 1, 60], x[4, 4, 5] = math.inf, math.nan, -math.inf
    run(30, 4, 2, 64, 16, 0, rows_of=rows_of)


def test_equal_to_append_without_norms():
    # Rows that are the positions, no norm: the same bits as without them.
    import torch
    import dense_linear_projection_gb300 as dlp
    x = torch.randn((40, 12, 128), device="cuda").to(torch.bfloat16)
    pos = torch.arange(40, dtype=torch.int32, device="cuda")
    table = torch.arange(4, dtype=torch.int32, device="cuda")[None]
    seq = torch.zeros(40, dtype=torch.int32, device="cuda")
    rope = dlp.rope_table(64, 128)
    results = []
    for rows in (None, pos):
        k_cache, v_cache = ku.make_cache(4, 16, 2, 128)
        kv = dlp.PagedKV(k_cache, v_cache, 8, 1)
        q = kv.append(x[:, :8], x[:, 8:10], x[:, 10:], pos, table, seq_ids=seq, rope=rope, rope_rows=rows)
        results.append((q, k_cache, v_cache))
    assert all(torch.equal(a, b) for a, b in zip(*results))


def test_bad_rows_are_reported_and_skipped():
    import torch
    import dense_linear_projection_gb300 as dlp
    k_cache, v_cache = ku.make_cache(4, 16, 2, 64)
    before = k_cache.clone(), v_cache.clone()
    kv = dlp.PagedKV(k_cache, v_cache, 2, 1)
    k, v = (torch.randn((1, 2, 64), device="cuda").to(torch.bfloat16) for _ in "kv")
    ints = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    rope, table, zero, w = dlp.rope_table(20, 64), ints(0, 9, -1)[None], ints(0), torch.ones(64, device="cuda")
    for pos, seq, row in ((3, 0, 20), (3, 0, -1), (48, 0, 1), (3, 1, 1), (3, -1, 1), (17, 0, 1), (40, 0, 1)):
        kv.append(None, k, v, ints(pos), table, seq_ids=ints(seq), rope=rope, k_norm=w, rope_rows=ints(row))
        assert kv.status() == dlp.PROJ_ERR_INVALID_ARG, (pos, seq, row)
        assert kv.status() == dlp.PROJ_OK
    assert torch.equal(k_cache, before[0]) and torch.equal(v_cache, before[1])
    # A position past the rope table is fine where the row is not.
    kv.append(None, k, v, ints(30), ints(0, 1)[None], seq_ids=zero, rope=rope, rope_rows=ints(19))
    assert kv.status() == dlp.PROJ_OK and torch.equal(v_cache[1, 14], v[0])


def test_refusals():
    import torch
    import dense_linear_projection_gb300 as dlp
    k_cache, v_cache = ku.make_cache(4, 16, 2, 64)
    kv = dlp.PagedKV(k_cache, v_cache, 4, 1)
    x = torch.randn((3, 8, 64), device="cuda").to(torch.bfloat16)
    pos = torch.arange(3, dtype=torch.int32, device="cuda")
    table = torch.arange(4, dtype=torch.int32, device="cuda").view(1, 4)
    seq, w, rope = torch.zeros_like(pos), torch.ones(64, device="cuda"), dlp.rope_table(20, 64)
    good = dict(seq_ids=seq, rope=rope, q_norm=w, k_norm=w, rope_rows=pos)

    def refused(q=x[:, :4], **change):
        with pytest.raises((dlp.ProjError, TypeError)) as e:
            kv.append(q, x[:, 4:6], x[:, 6:], pos, table, **{**good, **change})
        return e.value.status if isinstance(e.value, dlp.ProjError) else dlp.PROJ_ERR_INVALID_ARG

    bad = dlp.PROJ_ERR_INVALID_ARG
    for change in (dict(q_norm=w[:32]), dict(q_norm=w.bfloat16()), dict(k_norm=w.half(), q_norm=w.half()), dict(k_norm=w.cpu()),
                   dict(k_norm=torch.ones(128, device="cuda")[::2]), dict(q_norm=3), dict(eps=-1e-6), dict(eps=math.nan),
                   dict(eps=math.inf), dict(eps="x"), dict(rope_rows=pos[:2]), dict(rope_rows=pos.long()), dict(rope=None),
                   dict(rope_rows=pos.cpu()), dict(q=None)):
        assert refused(**change) == bad, change
    kv.append(x[:, :4], x[:, 4:6], x[:, 6:], pos, table, **good)
    assert kv.status() == dlp.PROJ_OK
    kv.close()
    assert refused() == bad
