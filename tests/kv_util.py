"""Caches, page tables and 64-bit references of the paged key-value tests."""
import math


def make_cache(pages, page_size, kv_heads, dim, dtype="bf16", layout="tokens_first", seed=0, poison=False):
    """k_cache, v_cache [pages, page_size, kv_heads, dim]; layout: which strides.  ``poison``: NaN
    everywhere, for tests that fill only the places in use."""
    import torch
    t = torch.float8_e4m3fn if dtype == "e4m3" else torch.bfloat16
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def values(shape):
        x = torch.randn(shape, generator=g, device="cuda")
        return (x * math.nan if poison else x).to(t)

    if layout == "tokens_first":
        return [values((pages, page_size, kv_heads, dim)) for _ in "kv"]
    if layout == "heads_first":
        return [values((pages, kv_heads, page_size, dim)).transpose(1, 2) for _ in "kv"]
    assert layout == "together"  # keys and values of a token next to each other
    both = values((pages, page_size, 2, kv_heads, dim))
    return [both[:, :, 0], both[:, :, 1]]


def make_table(lens, page_size, pages, seed=0, extra=1, unused=0):
    """int32 [B, width]: distinct pages in a shuffled order, ``unused`` past each length."""
    import torch
    g = torch.Generator()
    g.manual_seed(seed)
    need = [-(-n // page_size) for n in lens]
    assert sum(need) <= pages
    free = torch.randperm(pages, generator=g).to(torch.int32)
    table = torch.full((len(lens), max(need, default=0) + extra), unused, dtype=torch.int32)
    at = 0
    for i, n in enumerate(need):
        table[i, :n] = free[at:at + n]
        at += n
    return table.cuda()


def tokens_of(cache, table, b, low, high, page_size):
    """[high − low, kv_heads, dim] in 64 bits."""
    import torch
    t = torch.arange(low, high, device="cuda")
    pages = table[b].long()[t // page_size]
    raw = cache.view(torch.uint8) if cache.dtype == torch.float8_e4m3fn else cache
    x = raw[pages, t % page_size]
    return (x.view(torch.float8_e4m3fn) if cache.dtype == torch.float8_e4m3fn else x).double()


def put(cache, pages, places, rows):
    """cache[pages, places] = rows, for 8-bit caches too."""
    import torch
    if cache.dtype == torch.float8_e4m3fn:
        cache.view(torch.uint8)[pages, places] = rows.view(torch.uint8)
    else:
        cache[pages, places] = rows


def attention64(q, k_cache, v_cache, table, lens, page_size, scale, window=0, k_scale=None, v_scale=None, keep=None):
    """(out, lse, bound of out, bound of lse) in 64 bits.

    The bounds: a logit is a sum of dim products in fp32 (dim/16 steps and a few roundings, 2⁻²²
    each of its absolute terms A): δ = (dim/16 + 8)·2⁻²²·A.  Each weight e^(logit − top) then is off
    by a factor within 2δ, the exponential's own 2⁻²⁰, and its split into two 8-bit-mantissa parts,
    2⁻¹⁶; sums over n tokens add (n/16 + 64)·2⁻²².  The rounding to bf16 is not part of the bound: see
    beyond()."""
    import torch
    B, H, D = q.shape
    hk = k_cache.shape[2]
    G = H // hk
    out = torch.zeros((B, H, D), dtype=torch.float64, device="cuda")
    lse = torch.full((B, H), -math.inf, dtype=torch.float64, device="cuda")
    lim, lim_lse = torch.zeros_like(out), torch.zeros_like(lse)
    for b, n in enumerate(lens):
        low = max(0, n - window) if window else 0
        if n <= low:
            continue
        k, v = (tokens_of(c, table, b, low, n, page_size) for c in (k_cache, v_cache))
        if k_scale is not None:
            k, v = k * k_scale.double()[:, None], v * v_scale.double()[:, None]
        if keep is not None:
            sel = keep(b, torch.arange(low, n, device="cuda"))
            if not bool(sel.any()):
                continue
            k, v = k[sel], v[sel]
        k, v = k.repeat_interleave(G, 1), v.repeat_interleave(G, 1)
        x = q[b].double()
        s = torch.einsum("hd,thd->ht", x, k) * scale
        a = torch.einsum("hd,thd->ht", x.abs(), k.abs()).amax(1) * abs(scale)
        p = torch.softmax(s, 1)
        out[b] = torch.einsum("ht,thd->hd", p, v)
        lse[b] = torch.logsumexp(s, 1)
        delta = (D / 16 + 8) * 2.0 ** -22 * a
        rel = 2 * delta + 2.0 ** -20 + 2.0 ** -16 + ((n - low) / 16 + 64) * 2.0 ** -22
        lim[b] = torch.einsum("ht,thd->hd", p, v.abs()) * rel[:, None]
        lim_lse[b] = rel + 2.0 ** -22 * lse[b].abs()
    return out, lse, lim + 1e-38, lim_lse


def beyond(got, ref, lim):
    """How far each value of ``got`` lies outside what rounding a number within ``lim`` of ``ref`` to
    its type can give (rounding is monotonic: between the rounded ends of that interval); <= 0: inside."""
    import torch
    low, high = ((ref - lim).to(got.dtype).double(), (ref + lim).to(got.dtype).double())
    return torch.maximum(low - got.double(), got.double() - high)


def check_attention(got, lse, ref, what=""):
    import torch
    out, want, lim, lim_lse = ref
    assert torch.isfinite(got).all(), what
    over = beyond(got, out, lim)
    assert (over <= 0).all(), f"{what}: {int((over > 0).sum())} of {got.numel()} beyond the bound, by up to {over.max().item():.3e}"
    if lse is not None:
        empty = want == -math.inf
        assert torch.equal(lse == -math.inf, empty), what
        off = (lse.double() - want).abs()[~empty] - lim_lse[~empty]
        assert (off <= 0).all(), f"{what}: lse beyond its bound by {off.max().item():.3e}"
