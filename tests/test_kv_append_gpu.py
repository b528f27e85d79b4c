"""Append to the paged cache with the rotary position.

The rotation is defined with separate fp32 products and sums and one rounding to the type
written, so it has to equal the same elementary torch operations bit for bit; against 64 bits it
is the rounding of a number within 2⁻²² of the absolute terms."""
import pytest

import kv_util as ku

pytestmark = pytest.mark.gpu


def rotated(x, rope_rows, interleaved, f64=False):
    """[tokens, heads, dim] at rope_rows [tokens, rot], in fp32 (or 64 bits)."""
    import torch
    x = x.double() if f64 else x.float()
    if rope_rows is None:
        return x
    rot = rope_rows.shape[1]
    r = (rope_rows.double() if f64 else rope_rows)[:, None]
    cos, sin = r[..., :rot // 2], r[..., rot // 2:]
    y = x.clone()
    a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if interleaved else (x[..., :rot // 2], x[..., rot // 2:rot])
    u, w = a * cos - b * sin, b * cos + a * sin
    if interleaved:
        y[..., 0:rot:2], y[..., 1:rot:2] = u, w
    else:
        y[..., :rot // 2], y[..., rot // 2:rot] = u, w
    return y


def quantised(x, scale):
    import torch
    return (x / scale[:, None]).clamp(-448, 448).to(torch.float8_e4m3fn)


def run(tokens, heads, kv_heads, dim, page, rot, interleaved=False, dtype="bf16", layout="tokens_first", in_place=False,
        sequences=3, pad=True, seed=0):
    import torch
    import dense_linear_projection_gb300 as dlp
    g = torch.Generator()
    g.manual_seed(seed)
    # Distinct (sequence, position) places, in any order, some tokens padding.
    per = -(-tokens // sequences) + 5
    spots = torch.randperm(sequences * per, generator=g)[:tokens]
    seq, pos = (spots // per).to(torch.int32), (spots % per).to(torch.int32)
    if pad and tokens > 2:
        pos[::3] = -1 - pos[::3]
    width = -(-per // page) + 1
    pages = sequences * width + 2
    k_cache, v_cache = ku.make_cache(pages, page, kv_heads, dim, dtype, layout, seed)
    table = torch.randperm(pages, generator=g)[:sequences * width].to(torch.int32).view(sequences, width)
    rope = dlp.rope_table(per + 3, rot) if rot else None
    scales = [torch.rand(kv_heads, generator=g).cuda() * 0.2 + 0.01 for _ in "kv"] if dtype == "e4m3" else [None, None]
    kv = dlp.PagedKV(k_cache, v_cache, heads, 1, k_scale=scales[0], v_scale=scales[1])
    rows = (torch.randn((tokens, heads + 2 * kv_heads, dim), generator=g) * 3).cuda().to(torch.bfloat16)
    original = rows.clone()
    q, k, v = rows[:, :heads], rows[:, heads:heads + kv_heads], rows[:, heads + kv_heads:]
    want_k, want_v = k_cache.clone(), v_cache.clone()
    live = pos >= 0
    at = pos[live].long()
    to, place = table[seq[live].long(), at // page].long().cuda(), (at % page).cuda()
    rope_rows = rope[at.cuda()] if rot else None
    lk, lv = original[:, heads:heads + kv_heads][live.cuda()], original[:, heads + kv_heads:][live.cuda()]
    kr = rotated(lk, rope_rows, interleaved)
    if dtype == "e4m3":
        ku.put(want_k, to, place, quantised(kr, scales[0]))
        ku.put(want_v, to, place, quantised(lv.float(), scales[1]))
    else:
        ku.put(want_k, to, place, kr.to(torch.bfloat16))
        ku.put(want_v, to, place, lv)
    q_out = q if in_place else torch.full((tokens, heads, dim), 9.0, dtype=torch.bfloat16, device="cuda")
    got = kv.append(q, k, v, pos.cuda(), table.cuda(), seq_ids=seq.cuda(), rope=rope, interleaved=interleaved, q_out=q_out)
    assert got is q_out
    bits = lambda x: x.contiguous().view(torch.uint8 if dtype == "e4m3" else torch.int16)  # noqa: E731
    assert torch.equal(bits(k_cache), bits(want_k)) and torch.equal(bits(v_cache), bits(want_v))
    lq = original[:, :heads][live.cuda()]
    assert torch.equal(got[live.cuda()], rotated(lq, rope_rows, interleaved).to(torch.bfloat16))
    exact = rotated(lq, rope_rows, interleaved, f64=True)
    lim = 2.0 ** -22 * 2 * lq.abs().amax().double()
    assert (ku.beyond(got[live.cuda()], exact, lim) <= 0).all()
    # Padding rows: nothing written.
    assert torch.equal(got[~live.cuda()], original[:, :heads][~live.cuda()] if in_place
                       else torch.full_like(got[~live.cuda()], 9.0))
    assert torch.equal(rows[:, heads:], original[:, heads:])
    assert kv.status() == dlp.PROJ_OK


@pytest.mark.parametrize("tokens", [1, 2, 7, 64, 300, 2111])
@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
def test_token_counts(tokens, dtype):
    run(tokens, 16, 4, 128, 16, 128, dtype=dtype)


@pytest.mark.parametrize("dim,rot", [(16, 16), (64, 64), (64, 32), (128, 64), (80, 80), (96, 48), (256, 256), (64, 0), (128, 2),
                                     (64, 20), (112, 110), (256, 250)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_dims_and_rotary_parts(dim, rot, interleaved):
    run(40, 6, 2, dim, 16, rot, interleaved)
    run(40, 6, 2, dim, 16, rot, interleaved, dtype="e4m3")


@pytest.mark.parametrize("page", [1, 3, 16, 64])
@pytest.mark.parametrize("layout", ["tokens_first", "heads_first", "together"])
def test_pages_and_layouts(page, layout):
    run(50, 8, 8, 64, page, 64, layout=layout)


@pytest.mark.parametrize("rot,interleaved", [(128, False), (128, True), (64, False), (20, False)])
def test_in_place(rot, interleaved):
    run(100, 8, 2, 128, 16, rot, interleaved, in_place=True)


def test_head_counts():
    for heads, kv_heads in ((1, 1), (7, 1), (71, 1), (64, 8), (48, 48)):
        run(9, heads, kv_heads, 64, 16, 64)


def test_one_token_of_each_sequence_and_keys_only():
    # seq_ids left out: token i belongs to sequence i; q left out: keys and values alone.
    import torch
    import dense_linear_projection_gb300 as dlp
    k_cache, v_cache = ku.make_cache(20, 16, 2, 64)
    table = torch.randperm(20).to(torch.int32)[:10].view(5, 2).cuda()
    pos = torch.tensor([0, 15, 16, 31, 7], dtype=torch.int32, device="cuda")
    k, v = (torch.randn((5, 2, 64), device="cuda").to(torch.bfloat16) for _ in "kv")
    kv = dlp.PagedKV(k_cache, v_cache, 4, 5)
    assert kv.append(None, k, v, pos, table) is None
    rows = table.long()[torch.arange(5, device="cuda"), pos.long() // 16]
    assert torch.equal(k_cache[rows, pos.long() % 16], k) and torch.equal(v_cache[rows, pos.long() % 16], v)


def test_8_bit_range():
    # Beyond ±448 units a value is clamped; infinities too, a NaN stays one; ties go to even.
    import math
    import torch
    import dense_linear_projection_gb300 as dlp
    k_cache, v_cache = ku.make_cache(1, 16, 1, 16, "e4m3")
    x = torch.tensor([[[1e6, -1e6, math.inf, -math.inf, math.nan, 448, 464, 500, 0.0, -0.0, 2.0 ** -9, 2.0 ** -10, 1.0625, 1.1875, 17, 19]]],
                     device="cuda").to(torch.bfloat16)
    kv = dlp.PagedKV(k_cache, v_cache, 1, 1)
    zero = torch.zeros(1, dtype=torch.int32, device="cuda")
    kv.append(None, x, -x, zero, zero[None])
    for cache, y in ((k_cache, x), (v_cache, -x)):
        want = y[0, 0].float().clamp(-448, 448).to(torch.float8_e4m3fn)
        got = cache[0, 0, 0].float()
        assert torch.equal(got.isnan(), want.float().isnan())
        assert torch.equal(got.nan_to_num(0), want.float().nan_to_num(0))


def test_offsets_past_31_bits():
    import torch
    import dense_linear_projection_gb300 as dlp
    stride, hk, dim = 1 << 26, 2, 64
    base = [torch.empty(stride * 43 + 16 * hk * dim, dtype=torch.bfloat16, device="cuda") for _ in "kv"]
    k_cache, v_cache = (x.as_strided((44, 16, hk, dim), (stride, hk * dim, dim, 1)) for x in base)
    k, v = (torch.randn((44, hk, dim), device="cuda").to(torch.bfloat16) for _ in "kv")
    kv = dlp.PagedKV(k_cache, v_cache, 2, 1)
    table = torch.randperm(44).to(torch.int32)[None].cuda()
    pos = (torch.arange(44, device="cuda") * 16 + 3).to(torch.int32)
    kv.append(None, k, v, pos, table, seq_ids=torch.zeros(44, dtype=torch.int32, device="cuda"))
    assert torch.equal(k_cache[table[0].long(), 3], k) and torch.equal(v_cache[table[0].long(), 3], v)


def test_bad_places_are_reported_and_skipped():
    import torch
    import dense_linear_projection_gb300 as dlp
    k_cache, v_cache = ku.make_cache(8, 16, 2, 64)
    before = k_cache.clone(), v_cache.clone()
    kv = dlp.PagedKV(k_cache, v_cache, 2, 1)
    k, v = (torch.randn((1, 2, 64), device="cuda").to(torch.bfloat16) for _ in "kv")
    rope = dlp.rope_table(20, 64)
    ints = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    table = ints(0, 8, -1)[None]
    for pos, seq in ((48, 0), (25, 0), (3, 1), (3, -1), (17, 0), (35, 0)):
        rope_now = rope if pos == 25 else None  # 25 is past this rope table
        kv.append(None, k, v, ints(pos), table, seq_ids=ints(seq), rope=rope_now)
        assert kv.status() == dlp.PROJ_ERR_INVALID_ARG, (pos, seq)
        assert kv.status() == dlp.PROJ_OK
    assert torch.equal(k_cache, before[0]) and torch.equal(v_cache, before[1])
    kv.append(None, k, v, ints(3), table, seq_ids=ints(0), rope=rope)
    assert kv.status() == dlp.PROJ_OK and torch.equal(v_cache[0, 3], v[0])


def test_append_then_attend_on_a_stream_and_in_a_graph():
    # The new token's own key and value are seen by the attention of the same step.
    import torch
    import dense_linear_projection_gb300 as dlp
    B, H, hk, D, page = 3, 8, 2, 64, 16
    k_cache, v_cache = ku.make_cache(30, page, hk, D)
    table = torch.randperm(30).to(torch.int32)[:24].view(3, 8).cuda()
    kv = dlp.PagedKV(k_cache, v_cache, H, B)
    rope = dlp.rope_table(128, D)
    rows = torch.randn((B, H + 2 * hk, D), device="cuda").to(torch.bfloat16)
    pos = torch.tensor([0, 40, 100], dtype=torch.int32, device="cuda")
    lens = pos + 1

    def step():
        q = kv.append(rows[:, :H], rows[:, H:H + hk], rows[:, H + hk:], pos, table, rope=rope)
        return q, kv.attend(q, table, lens)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        q, out = step()
    torch.cuda.current_stream().wait_stream(side)
    ref = ku.attention64(q, k_cache, v_cache, table, [1, 41, 101], page, D ** -0.5)
    ku.check_attention(out, None, ref, "stream")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        q, out = step()
    rows.copy_(torch.randn(rows.shape, device="cuda"))
    pos += 1
    lens += 1
    g.replay()
    torch.cuda.synchronize()
    ref = ku.attention64(q, k_cache, v_cache, table, [2, 42, 102], page, D ** -0.5)
    ku.check_attention(out, None, ref, "graph")


def test_refusals():
    import torch
    import dense_linear_projection_gb300 as dlp
    k_cache, v_cache = ku.make_cache(8, 16, 2, 64)
    kv = dlp.PagedKV(k_cache, v_cache, 4, 1)
    q = torch.zeros((2, 4, 64), device="cuda", dtype=torch.bfloat16)
    k, v = (torch.zeros((2, 2, 64), device="cuda", dtype=torch.bfloat16) for _ in "kv")
    pos, table = torch.zeros(2, dtype=torch.int32, device="cuda"), torch.zeros((2, 3), dtype=torch.int32, device="cuda")
    f32 = torch.zeros((9, 64), device="cuda")
    invalid = dlp.PROJ_ERR_INVALID_ARG
    for what, status in [
        (lambda: kv.append(q, k, v[:1], pos, table), invalid),
        (lambda: kv.append(q[:1], k, v, pos, table), invalid),
        (lambda: kv.append(q, k.float(), v, pos, table), invalid),
        (lambda: kv.append(q, k, v, pos.long(), table), invalid),
        (lambda: kv.append(q, k, v, pos[:1], table), invalid),
        (lambda: kv.append(q, k, v, pos, table, rope=f32.double()), invalid),
        (lambda: kv.append(q, k, v, pos, table, rope=torch.zeros((9, 66), device="cuda")), invalid),  # wider than a head
        (lambda: kv.append(q, k, v, pos, table, rope=torch.zeros((9, 63), device="cuda")), invalid),
        (lambda: kv.append(q, k, v, pos, table, seq_ids=pos[:1]), invalid),
        (lambda: kv.append(None, k, v, pos, table, q_out=q), invalid),
        (lambda: dlp.proj_kv_append(kv.handle, 2, None, 0, k.data_ptr() + 2, v, 128, pos, None, table, 2, 3, None, 0, 0, False,
                                    None, None, k_cache, v_cache, None, 0), dlp.PROJ_ERR_MISALIGNED),
        (lambda: dlp.proj_kv_append(kv.handle, 2, None, 0, k, v, 128, None, None, table, 2, 3, None, 0, 0, False,
                                    None, None, k_cache, v_cache, None, 0), invalid),
    ]:
        with pytest.raises(dlp.ProjError) as e:
            what()
        assert e.value.status == status


def test_status_follows_the_stream():
    # status() waits for the stream that the calls run on, the current one by default.
    import torch
    import dense_linear_projection_gb300 as dlp
    k_cache, v_cache = ku.make_cache(8, 16, 2, 64)
    kv = dlp.PagedKV(k_cache, v_cache, 2, 1)
    k, v = (torch.zeros((1, 2, 64), device="cuda").to(torch.bfloat16) for _ in "kv")
    pos, table = torch.full((1,), 99, dtype=torch.int32, device="cuda"), torch.zeros((1, 2), dtype=torch.int32, device="cuda")
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        for _ in range(2):
            torch.cuda._sleep(100_000_000)
            kv.append(None, k, v, pos, table)
            assert kv.status() == dlp.PROJ_ERR_INVALID_ARG
            assert kv.status() == dlp.PROJ_OK
    torch.cuda._sleep(100_000_000)
    kv.append(None, k, v, pos, table, stream=side)
    assert kv.status(side) == dlp.PROJ_ERR_INVALID_ARG and kv.status(side.cuda_stream) == dlp.PROJ_OK
