"""The normed append where its numbers are the append's: the same bits.

The rotation is products and sums of fp32 numbers, each rounded by itself, and one rounding to the
type written; PyTorch's elementwise operations on fp32 tensors are the same ones."""
import pytest

import kv_util as ku

pytestmark = pytest.mark.gpu


def rows(shape, seed):
    import torch
    g = torch.Generator()
    g.manual_seed(seed)
    return torch.randn(shape, generator=g).cuda().to(torch.bfloat16)


def turned32(x, rope_rows, interleaved):
    """The rotation in fp32, operation by operation."""
    import torch
    rot = rope_rows.shape[1]
    cos, sin = rope_rows[:, None].split(rot // 2, -1)
    first, second = (slice(0, rot, 2), slice(1, rot, 2)) if interleaved else (slice(0, rot // 2), slice(rot // 2, rot))
    y = x.float()
    a, b = y[..., first].clone(), y[..., second].clone()
    y[..., first], y[..., second] = torch.sub(torch.mul(a, cos), torch.mul(b, sin)), torch.add(torch.mul(b, cos), torch.mul(a, sin))
    return y


@pytest.mark.parametrize("dim,rot", [(128, 128), (128, 64), (64, 20), (256, 256), (80, 80), (48, 2)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation(dim, rot, interleaved):
    # Rows that are the positions, and no norm: the append, and the formula's own roundings.
    import torch
    import dense_linear_projection_gb300 as dlp
    tokens, page = 700, 16
    x = rows((tokens, 12, dim), dim + rot)
    pos = torch.arange(tokens, dtype=torch.int32, device="cuda")
    table = torch.arange(-(-tokens // page), dtype=torch.int32, device="cuda")[None]
    seq, rope = torch.zeros_like(pos), dlp.rope_table(tokens, rot)
    want = turned32(x[:, :10], rope, interleaved).to(torch.bfloat16)
    for given in (None, pos):
        k_cache, v_cache = ku.make_cache(table.shape[1], page, 2, dim)
        kv = dlp.PagedKV(k_cache, v_cache, 8, 1)
        q = kv.append(x[:, :8], x[:, 8:10], x[:, 10:], pos, table, seq_ids=seq, rope=rope, interleaved=interleaved, rope_rows=given)
        assert kv.status() == dlp.PROJ_OK
        assert torch.equal(q, want[:, :8]), given
        assert torch.equal(k_cache.flatten(0, 1)[:tokens], want[:, 8:]) and torch.equal(v_cache.flatten(0, 1)[:tokens], x[:, 10:])


@pytest.mark.parametrize("dim,rot", [(128, 16), (128, 20), (64, 64), (48, 2)])
def test_8_bits(dim, rot):
    # Every bf16 value as an element of a value head and of a key head, at scales whose quotients come
    # to the middle between two e4m3 numbers: x / scale, rounded once in fp32 and once to e4m3, whichever
    # of the calls stores it.
    import torch
    import dense_linear_projection_gb300 as dlp
    page, scales = 16, torch.tensor([2.06, 0.3, 1 / 3, 1.0, 0.0117, 3.0, 2.0 ** -101, 2.0 ** 101], device="cuda")
    heads = scales.shape[0]
    tokens = -(-65536 // dim)
    every = torch.arange(-32768, 32768, dtype=torch.int32, device="cuda").to(torch.int16).view(torch.bfloat16)
    every = torch.cat([every, every[:tokens * dim - 65536]]).view(tokens, 1, dim).expand(tokens, heads, dim)
    q = rows((tokens, heads, dim), 3)
    x = torch.cat([q, every, every], 1)
    pos = torch.arange(tokens, dtype=torch.int32, device="cuda")
    table = torch.arange(-(-tokens // page), dtype=torch.int32, device="cuda")[None]
    seq, rope, w = torch.zeros_like(pos), dlp.rope_table(tokens, rot), torch.ones(dim, device="cuda")
    divided = torch.div(every.float(), scales[:, None]).clamp(-448, 448)
    finite = torch.isfinite(every)
    first = None
    for more in (dict(), dict(rope_rows=pos), dict(q_norm=w), dict(q_norm=w, rope_rows=pos), dict(k_norm=w)):
        k_cache, v_cache = (c.view(torch.uint8).fill_(0x7f).view(c.dtype) for c in ku.make_cache(table.shape[1], page, heads, dim, "e4m3"))
        kv = dlp.PagedKV(k_cache, v_cache, heads, 1, k_scale=scales, v_scale=scales)
        kv.append(x[:, :heads], x[:, heads:2 * heads], x[:, 2 * heads:], pos, table, seq_ids=seq, rope=rope, **more)
        assert kv.status() == dlp.PROJ_OK
        got = [c.view(torch.uint8).flatten(0, 1)[:tokens].clone() for c in (k_cache, v_cache)]
        first = first or got
        assert torch.equal(got[1], first[1]), more
        assert torch.equal(got[0], first[0]) or "k_norm" in more, more
        assert torch.equal(got[1][finite], divided.to(torch.float8_e4m3fn).view(torch.uint8)[finite]), more
