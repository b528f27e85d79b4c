"""Cases and plain forms of the paged cache's further operators:

* ``norm``: the append of new tokens with a root-mean-square norm of every head's queries and keys
  before the rotary position, which is read at a row of its own (a token of a cache that was evicted
  from stands at another place than its position);
* ``shared``: attention of one new token of each sequence where the whole batch shares a long prefix;
* ``scored``: attention that adds each cached token's weight, over the heads of its key head, to a score;
* ``evict``: the tokens of the highest scores, and the last ones, of each sequence and key head, copied
  to other pages.

``run`` computes a case in its plain form (elementary torch operations in 32 bits), or, where
``own`` is true, with the library's kernels.  ``exact`` gives the same outputs in 64 bits.
"""
import math

import torch

own = False

BF16, F32, E4M3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
EPS = 1e-6


# ---------------------------------------------------------------- cases
def listed():
    return [
        # One token of one sequence: latency.
        dict(name="norm_one_token", op="norm", tokens=1, sequences=1, max_len=2048, heads=32, kv_heads=8, dim=128,
             rot=128, interleaved=False, page=16, heads_first=False, kv="bf16", weights="bf16", shift=0),
        # A large decode batch into an 8-bit cache, at scattered places, after an eviction.
        dict(name="norm_batch256_8bit", op="norm", tokens=256, sequences=256, max_len=1024, heads=64, kv_heads=8,
             dim=128, rot=64, interleaved=True, page=64, heads_first=True, kv="e4m3", weights="f32", shift=700),
        # The prompts of three sequences, an odd number of tokens.
        dict(name="norm_prompts", op="norm", tokens=8191, sequences=3, max_len=0, heads=32, kv_heads=32, dim=128,
             rot=128, interleaved=False, page=16, heads_first=False, kv="bf16", weights="bf16", shift=0),
        # A few answers to one short instruction.
        dict(name="shared_few", op="shared", batch=4, prefix=1000, max_len=37, ragged=False, heads=32, kv_heads=8,
             dim=128, page=16, heads_first=False, kv="bf16"),
        # A serving batch behind one system prompt, unequal texts of their own, one of them empty.
        dict(name="shared_batch64", op="shared", batch=64, prefix=8192, max_len=1024, ragged=True, heads=64, kv_heads=8,
             dim=128, page=32, heads_first=True, kv="bf16"),
        # Many samples about one long document: the products with the prefix count most.
        dict(name="shared_batch128_long", op="shared", batch=128, prefix=32768, max_len=256, ragged=True, heads=64,
             kv_heads=8, dim=128, page=64, heads_first=False, kv="bf16"),
        # Narrow heads with a key head each, an odd batch and prefix, 8 bits.
        dict(name="shared_narrow_8bit", op="shared", batch=31, prefix=12345, max_len=500, ragged=True, heads=32,
             kv_heads=32, dim=64, page=16, heads_first=False, kv="e4m3"),
        # A few cached tokens of one sequence.
        dict(name="scored_short", op="scored", batch=1, max_len=301, ragged=False, heads=32, kv_heads=8, dim=128,
             page=16, heads_first=False, window=0, kv="bf16"),
        # A serving batch of unequal lengths.
        dict(name="scored_batch64_ragged", op="scored", batch=64, max_len=8192, ragged=True, heads=64, kv_heads=8,
             dim=128, page=32, heads_first=True, window=0, kv="bf16"),
        # One token over its budget: the step of a short conversation.
        dict(name="evict_one_short", op="evict", batch=1, max_len=1040, ragged=False, kv_heads=8, dim=128, keep=1024,
             recent=128, page=16, heads_first=False, kv="bf16"),
        # A batch of prompts brought down to a budget; the short ones are copied whole.
        dict(name="evict_batch32", op="evict", batch=32, max_len=8192, ragged=True, kv_heads=8, dim=128, keep=2048,
             recent=256, page=32, heads_first=True, kv="bf16"),
        # One long document in 8 bits, an odd budget.
        dict(name="evict_one_long_8bit", op="evict", batch=1, max_len=131071, ragged=False, kv_heads=8, dim=128,
             keep=32001, recent=1000, page=64, heads_first=False, kv="e4m3"),
    ]


def _log(rng, low, high):
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


#: No drawn case of an operator moves more bytes or computes more than this (the largest listed one of its kind).
MOST_BYTES = {"norm": 406e6, "shared": 206e6, "scored": 1096e6, "evict": 472e6}
MOST_FLOPS = 1.37e11


def draw(rng):
    while True:
        op = rng.choice(("norm", "shared", "scored", "evict"))
        dim = rng.choice((64, 128, 128))
        kv_heads = rng.choice((1, 2, 4, 8, 8, 16, 32))
        heads = kv_heads * rng.choice([g for g in (1, 2, 4, 7, 8, 16) if g * kv_heads <= 64])
        case = dict(op=op, kv_heads=kv_heads, dim=dim, page=rng.choice((16, 32, 64)), heads_first=rng.random() < 0.5,
                    kv=rng.choice(("bf16", "bf16", "e4m3")))
        if op != "evict":
            case["heads"] = heads
        if op == "norm":
            tokens = _log(rng, 1, 8192)
            case.update(tokens=tokens, rot=rng.choice((dim, dim, dim // 2)), interleaved=rng.random() < 0.5,
                        weights=rng.choice(("bf16", "f32")), shift=rng.choice((0, rng.randint(1, 2000))))
            if tokens <= 256 and rng.random() < 0.7:
                case.update(sequences=tokens, max_len=_log(rng, 32, 1024))
            else:
                case.update(sequences=min(tokens, rng.randint(1, 5)), max_len=0)
        elif op == "evict":
            most = _log(rng, 20, 131072)
            keep = rng.randint(max(1, most // 8), most)
            case.update(batch=_log(rng, 1, 64), max_len=most, ragged=rng.random() < 0.7, keep=keep,
                        recent=rng.randint(0, keep // 2))
        else:
            case.update(batch=_log(rng, 1, 128), max_len=_log(rng, 20, 131072 if op == "scored" else 1024),
                        ragged=rng.random() < 0.7)
            if op == "shared":
                case.update(prefix=_log(rng, 64, 32768))
            else:
                case.update(window=rng.choice((0, 0, _log(rng, 16, 4096))))
        if "batch" in case and case["batch"] * case["max_len"] * kv_heads * dim > 64 * 8192 * 8 * 128:
            continue  # the plain form pads every sequence to the longest
        cost = work(case)
        if cost["bytes"] <= MOST_BYTES[op] and cost["flops"] <= MOST_FLOPS:
            return case


def lengths(case):
    """Cached tokens of each sequence (its own ones in a ``shared`` case); a ragged batch has an empty one."""
    n, most = case["batch"], case["max_len"]
    if not case["ragged"] or n == 1:
        return [most] * n
    return [most if i == 0 else 0 if i == 1 else 1 + (most - 1) * ((29 * i + 17) % 97) // 96 for i in range(n)]


def places(case):
    """(sequence, place) of each token of a ``norm`` case."""
    t, s = case["tokens"], case["sequences"]
    if t == s and case["max_len"]:
        return list(range(t)), [(case["max_len"] - 1) * ((61 * i + 96) % 97) // 96 for i in range(t)]
    first = [-(-t * i // s) for i in range(s + 1)]
    seq = [i for i in range(s) for _ in range(first[i], first[i + 1])]
    return seq, [13 * i + at - first[i] for at, i in enumerate(seq)]


def _pages(n, case):
    return -(-n // case["page"])


def work(case):
    hk, d, e = case["kv_heads"], case["dim"], 1 if case["kv"] == "e4m3" else 2
    if case["op"] == "norm":
        t, h = case["tokens"], case["heads"]
        size = t * (h + 2 * hk) * d * 2 + t * h * d * 2 + t * 2 * hk * d * e + t * (case["rot"] * 4 + 16)
        size += 2 * d * (4 if case["weights"] == "f32" else 2)
        return {"bytes": float(size), "flops": t * (h + hk) * (3.0 * case["rot"] + 4.0 * d)}
    lens = lengths(case)
    if case["op"] == "evict":
        kept, wide = sum(min(x, case["keep"]) for x in lens), _pages(case["keep"], case) * case["page"]
        size = kept * hk * d * e * 4 + sum(lens) * hk * 4 + case["batch"] * hk * (wide + case["keep"]) * 4
        return {"bytes": float(size), "flops": float(sum(lens) * hk)}
    h, batch = case["heads"], case["batch"]
    if case["op"] == "shared":
        size = (case["prefix"] + sum(lens)) * hk * d * 2 * e + batch * h * (d * 4 + 4)
        size += (_pages(case["prefix"], case) + sum(_pages(x, case) for x in lens) + batch) * 4
        return {"bytes": float(size), "flops": 4.0 * (batch * case["prefix"] + sum(lens)) * h * d}
    seen = [min(x, case["window"]) if case["window"] else x for x in lens]
    wide = max(1, _pages(max(lens), case)) * case["page"]
    size = sum(seen) * hk * d * 2 * e + batch * h * (d * 4 + 4) + sum(_pages(x, case) for x in seen) * 4
    return {"bytes": float(size + batch * hk * wide * 8), "flops": (4.0 * d + 1) * sum(seen) * h}


# ---------------------------------------------------------------- inputs
def _randn(gen, shape, scale=1.0, dtype=BF16):
    return torch.randn(shape, generator=gen, device="cuda", dtype=F32).mul_(scale).to(dtype)


def _cache(gen, case, pages):
    """Keys and values [pages, page, kv_heads, dim] (a view where heads come first in memory)."""
    page, hk, d = case["page"], case["kv_heads"], case["dim"]
    shape = (pages, hk, page, d) if case["heads_first"] else (pages, page, hk, d)
    out = []
    for _ in "kv":
        x = torch.empty(shape, device="cuda", dtype=E4M3 if case["kv"] == "e4m3" else BF16)
        for at in range(0, pages, 4096):  # a part at a time: the normals are four bytes each
            part = x[at:at + 4096]
            part.copy_(_randn(gen, part.shape, 1.0, F32))
        out.append(x.transpose(1, 2) if case["heads_first"] else x)
    scales = (None, None)
    if case["kv"] == "e4m3":
        scales = [torch.rand(hk, generator=gen, device="cuda") * 0.5 + 0.25 for _ in "kv"]
    return out[0], out[1], scales[0], scales[1]


def _table(free, lens, width, case):
    """A page table [sequences, width] of pages from the list ``free``, and how many it takes."""
    table, used = torch.zeros((len(lens), width), dtype=torch.int32, device="cuda"), 0
    for i, n in enumerate(lens):
        need = _pages(n, case)
        table[i, :need] = free[used:used + need]
        used += need
    return table, used


def _inputs(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed) * 1000003 + 29)
    s, hk, d, page = {"case": case}, case["kv_heads"], case["dim"], case["page"]
    permuted = lambda n: torch.randperm(n, generator=gen, device="cuda").to(torch.int32)  # noqa: E731
    if case["op"] == "norm":
        h = case["heads"]
        seq, at = places(case)
        width = max(at) // page + 1
        # The rows of a query, key and value projection; its heads are not of one size.
        rows = torch.randn((case["tokens"], h + 2 * hk, d), generator=gen, device="cuda")
        rows *= torch.rand((case["tokens"], h + 2 * hk, 1), generator=gen, device="cuda") * 3 + 0.1
        rows = rows.to(BF16)
        s["q"], s["k"], s["v"] = rows[:, :h], rows[:, h:h + hk], rows[:, h + hk:]
        kind = F32 if case["weights"] == "f32" else BF16
        s["q_norm"], s["k_norm"] = ((1 + 0.2 * torch.randn(d, generator=gen, device="cuda")).to(kind) for _ in "qk")
        s["seq"] = torch.tensor(seq, dtype=torch.int32, device="cuda")
        s["pos"] = torch.tensor(at, dtype=torch.int32, device="cuda")
        # The rotary row of each token: its position, ``shift`` or fewer evicted tokens past its place.
        s["rows"] = s["pos"] + (torch.arange(case["tokens"], dtype=torch.int32, device="cuda") * 7919) % (case["shift"] + 1)
        angle = torch.arange(width * page + case["shift"], dtype=torch.float64, device="cuda")[:, None]
        half = case["rot"] // 2
        angle = angle * (10000.0 ** (-torch.arange(half, dtype=torch.float64, device="cuda") / half))[None, :]
        s["rope"] = torch.cat([angle.cos(), angle.sin()], 1).to(F32)
        pages = case["sequences"] * width
        s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"] = _cache(gen, case, pages)
        s["table"] = permuted(pages).view(case["sequences"], width)
        return s
    lens = lengths(case)
    s["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    width = max(1, _pages(max(lens), case))
    pages = sum(_pages(x, case) for x in lens) + 8
    more = _pages(case["prefix"], case) if case["op"] == "shared" else 0
    if case["op"] == "evict":
        to_width = _pages(case["keep"], case)
        more = case["batch"] * to_width
    s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"] = _cache(gen, case, pages + more)
    free = permuted(pages + more)
    s["table"], used = _table(free, lens, width, case)
    if case["op"] != "evict":
        s["q"] = _randn(gen, (case["batch"], case["heads"], d))
    if case["op"] == "shared":
        s["prefix"] = free[used:used + more].clone()
        return s
    if case["op"] == "evict":
        s["to"] = free[used:used + more].view(case["batch"], to_width).clone()
    # Scores as sums of softmax weights are: a few large ones, most small.
    scores = torch.randn((case["batch"], hk, width * page), generator=gen, device="cuda").mul_(2).exp_()
    s["scores"] = scores * (torch.arange(width * page, device="cuda")[None, None, :] < s["lens"][:, None, None])
    if case["op"] == "scored":
        s["scores_out"] = torch.empty_like(s["scores"])
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    if own:
        import dense_linear_projection_gb300 as dlp
        s["kv"] = dlp.PagedKV(s["k_cache"], s["v_cache"], case.get("heads", case["kv_heads"]),
                              max_sequences=s["table"].shape[0], k_scale=s["k_scale"], v_scale=s["v_scale"])
    return s


# ---------------------------------------------------------------- one pass
def run(state):
    s, case = state, state["case"]
    if own:
        kv = s["kv"]
        if case["op"] == "norm":
            q = kv.append(s["q"], s["k"], s["v"], s["pos"], s["table"], seq_ids=s["seq"], rope=s["rope"],
                          interleaved=case["interleaved"], q_norm=s["q_norm"], k_norm=s["k_norm"], eps=EPS,
                          rope_rows=s["rows"])
            return {"q": q, "k": s["k_cache"], "v": s["v_cache"]}
        if case["op"] == "shared":
            out, lse = kv.attend_shared(s["q"], s["prefix"], case["prefix"], s["table"], s["lens"], return_lse=True)
            return {"out": out, "lse": lse}
        if case["op"] == "scored":
            out, scores, lse = kv.attend_scored(s["q"], s["table"], s["lens"], s["scores"], window=case["window"],
                                                scores_out=s["scores_out"], return_lse=True)
            return {"out": out, "scores": scores, "lse": lse}
        lens, scores, kept = kv.evict(s["table"], s["lens"], s["scores"], s["to"], case["keep"], recent=case["recent"])
        return {"lens": lens, "scores": scores, "kept": kept, "k": s["k_cache"], "v": s["v_cache"]}
    return {"norm": _plain_norm, "shared": _plain_shared, "scored": _plain_scored, "evict": _plain_evict}[case["op"]](s, case)


def _put(cache, pages, at, rows, e4m3):
    if e4m3:  # bytes: an indexed write of 8-bit floating values is not there for every layout
        cache.view(torch.uint8)[pages, at] = rows.view(torch.uint8)
    else:
        cache[pages, at] = rows


def _plain_norm(s, case):
    rot, page, e4m3 = case["rot"], case["page"], case["kv"] == "e4m3"
    pos = s["pos"].long()
    cos, sin = s["rope"][s["rows"].long()].unsqueeze(1).split(rot // 2, -1)

    def turned(x, weight):
        x = x.to(F32)
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS) * weight.to(F32)
        x, rest = x[..., :rot], x[..., rot:]
        a, b = (x[..., 0::2], x[..., 1::2]) if case["interleaved"] else (x[..., :rot // 2], x[..., rot // 2:])
        u, v = a * cos - b * sin, b * cos + a * sin
        x = torch.stack([u, v], -1).flatten(-2) if case["interleaved"] else torch.cat([u, v], -1)
        return torch.cat([x, rest], -1)

    q, k, v = turned(s["q"], s["q_norm"]), turned(s["k"], s["k_norm"]), s["v"].to(F32)
    if e4m3:
        k = (k / s["k_scale"][:, None]).clamp(-448, 448)
        v = (v / s["v_scale"][:, None]).clamp(-448, 448)
    to, at = s["table"][s["seq"].long(), pos // page].long(), pos % page
    _put(s["k_cache"], to, at, k.to(E4M3 if e4m3 else BF16), e4m3)
    _put(s["v_cache"], to, at, v.to(E4M3 if e4m3 else BF16), e4m3)
    return {"q": q.to(BF16), "k": s["k_cache"], "v": s["v_cache"]}


def _gathered(cache, scale, table):
    """[tables, kv_heads, tokens, dim] in 32 bits: the tokens of every row of a page table."""
    if scale is not None:
        x = cache.view(torch.uint8)[table].view(E4M3).to(F32) * scale[:, None]
    else:
        x = cache[table].to(F32)
    return x.flatten(1, 2).transpose(1, 2)


def _softmax_parts(logits):
    top = logits.amax(-1, keepdim=True).clamp(min=-1e30)
    p = torch.exp(logits - top)
    return top, p, p.sum(-1, keepdim=True)


def _own_logits(s, case, low):
    """Logits [batch, kv_heads, group, tokens] of each sequence's own tokens, and which count."""
    b, h, hk, d = case["batch"], case["heads"], case["kv_heads"], case["dim"]
    table = s["table"].long()
    at = torch.arange(table.shape[1] * case["page"], device="cuda")[None, :]
    seen = ((at < s["lens"][:, None]) & (at >= low))[:, None, None, :]
    q = s["q"].to(F32).view(b, hk, h // hk, d)
    logits = q @ _gathered(s["k_cache"], s["k_scale"], table).transpose(2, 3)
    v = torch.where(seen.transpose(2, 3), _gathered(s["v_cache"], s["v_scale"], table), 0.0)
    return torch.where(seen, logits * (1.0 / math.sqrt(d)), -math.inf), v


def _plain_shared(s, case):
    b, h, hk, d = case["batch"], case["heads"], case["kv_heads"], case["dim"]
    own_logits, own_v = _own_logits(s, case, 0)
    k, v = (_gathered(c, x, s["prefix"].long()[None])[0, :, :case["prefix"]]
            for c, x in ((s["k_cache"], s["k_scale"]), (s["v_cache"], s["v_scale"])))
    # All sequences' queries of a key head against the prefix at once: [kv_heads, batch · group, tokens].
    q = s["q"].to(F32).view(b, hk, h // hk, d).transpose(0, 1).reshape(hk, -1, d)
    m0, p0, l0 = _softmax_parts((q @ k.transpose(1, 2)) * (1.0 / math.sqrt(d)))
    o0 = p0 @ v
    m0, l0, o0 = (x.view(hk, b, h // hk, -1).transpose(0, 1) for x in (m0, l0, o0))
    m1, p1, l1 = _softmax_parts(own_logits)
    o1 = p1 @ own_v
    m = torch.maximum(m0, m1)
    w0, w1 = torch.exp(m0 - m), torch.exp(m1 - m)
    total = l0 * w0 + l1 * w1
    out = (o0 * w0 + o1 * w1) / total
    return {"out": out.reshape(b, h, d).to(BF16), "lse": (m + total.log()).reshape(b, h)}


def _plain_scored(s, case):
    b, h, d = case["batch"], case["heads"], case["dim"]
    low = (s["lens"][:, None] - case["window"]).clamp(min=0) if case["window"] else 0
    logits, v = _own_logits(s, case, low)
    top, p, total = _softmax_parts(logits)
    p = p / torch.where(total > 0, total, 1.0)
    torch.add(s["scores"], p.sum(2), out=s["scores_out"])
    lse = torch.where(s["lens"][:, None] > 0, (top + total.log()).view(b, h), -math.inf)
    return {"out": (p @ v).reshape(b, h, d).to(BF16), "scores": s["scores_out"], "lse": lse}


def _plain_evict(s, case):
    page, keep, recent, b, hk = case["page"], case["keep"], case["recent"], case["batch"], case["kv_heads"]
    wide = s["to"].shape[1] * page
    at = torch.arange(s["scores"].shape[2], device="cuda")
    n = s["lens"].long()[:, None, None]
    # The last ones before all others, what is past the end after them; equal scores by their place.
    key = torch.where(at >= n - recent, math.inf, s["scores"])
    key = torch.where(at < n, key, -math.inf)
    order = torch.sort(key, dim=-1, descending=True, stable=True).indices
    if order.shape[2] < keep:
        order = torch.cat([order, order.new_full((b, hk, keep - order.shape[2]), at.shape[0])], 2)
    order = order[..., :keep]
    kept = torch.sort(torch.where(order < n, order, 1 << 40), dim=-1).values
    there = kept < n
    kept = torch.where(there, kept, -1)
    scores = torch.zeros((b, hk, wide), dtype=F32, device="cuda")
    scores[..., :keep] = torch.where(there, s["scores"].gather(2, kept.clamp(min=0).clamp(max=at.shape[0] - 1)), 0.0)
    who, head, to = torch.nonzero(there, as_tuple=True)
    token = kept[who, head, to]
    source, target = s["table"].long()[who, token // page], s["to"].long()[who, to // page]
    for cache in (s["k_cache"], s["v_cache"]):
        raw = cache.view(torch.uint8) if case["kv"] == "e4m3" else cache
        raw[target, to % page, head] = raw[source, token % page, head]
    return {"lens": s["lens"].clamp(max=keep), "scores": scores, "kept": kept.to(torch.int32), "k": s["k_cache"],
            "v": s["v_cache"]}


# ---------------------------------------------------------------- the definition, in 64 bits
def exact(case, seed):
    s = _inputs(case, seed)
    f64 = torch.float64
    hk, d, page = case["kv_heads"], case["dim"], case["page"]
    one = torch.ones(hk, dtype=f64, device="cuda")
    ks, vs = (x.to(f64) if x is not None else one for x in (s["k_scale"], s["v_scale"]))

    if case["op"] == "norm":
        half = case["rot"] // 2
        index = torch.arange(half, device="cuda")
        first, second = (2 * index, 2 * index + 1) if case["interleaved"] else (index, index + half)
        turn = torch.complex(s["rope"][:, :half].to(f64), s["rope"][:, half:].to(f64))[s["rows"].long()][:, None, :]

        def turned(x, weight):
            x = x.to(f64)
            x = x * weight.to(f64) * (x.square().sum(-1, keepdim=True) / d + EPS) ** -0.5
            y = torch.complex(x[..., first], x[..., second]) * turn
            x[..., first], x[..., second] = y.real, y.imag
            return x

        k_cache, v_cache = s["k_cache"].to(f64), s["v_cache"].to(f64)
        k, v = turned(s["k"], s["k_norm"]), s["v"].to(f64)
        if case["kv"] == "e4m3":
            k = torch.minimum(torch.maximum(k / ks[:, None], k.new_tensor(-448.0)), k.new_tensor(448.0))
            v = torch.minimum(torch.maximum(v / vs[:, None], v.new_tensor(-448.0)), v.new_tensor(448.0))
        seq, pos = places(case)
        table = s["table"].cpu()
        to = torch.tensor([int(table[i, p // page]) for i, p in zip(seq, pos)], device="cuda")
        at = torch.tensor([p % page for p in pos], device="cuda")
        k_cache[to, at], v_cache[to, at] = k, v
        return {"q": turned(s["q"], s["q_norm"]), "k": k_cache, "v": v_cache}

    def tokens(cache, scales, pages, where, j):
        raw = cache.view(torch.uint8) if case["kv"] == "e4m3" else cache
        return raw[:, :, j][pages.long()[where // page], where % page].view(cache.dtype).to(f64) * scales[j]

    if case["op"] == "evict":
        k_cache, v_cache = s["k_cache"].to(f64), s["v_cache"].to(f64)
        k_new, v_new = k_cache.clone(), v_cache.clone()
        keep, recent = case["keep"], case["recent"]
        scores = torch.zeros((case["batch"], hk, s["to"].shape[1] * page), dtype=f64, device="cuda")
        kept = torch.full((case["batch"], hk, keep), -1, dtype=torch.int32, device="cuda")
        lens = lengths(case)
        for i, n in enumerate(lens):
            if n == 0:
                continue
            for j in range(hk):
                if n <= keep:
                    chosen = torch.arange(n, device="cuda")
                else:
                    old = s["scores"][i, j, :n - recent]
                    want = keep - recent
                    # All above the last one taken, and the first of those that equal it.
                    border = torch.topk(old, want).values[-1] if want else old.new_tensor(math.inf)
                    above, equal = old > border, old == border
                    fill = equal & (equal.cumsum(0) <= want - above.sum())
                    chosen = torch.cat([torch.nonzero(above | fill)[:, 0], torch.arange(n - recent, n, device="cuda")])
                m = chosen.shape[0]
                at = torch.arange(m, device="cuda")
                kept[i, j, :m] = chosen.to(torch.int32)
                scores[i, j, :m] = s["scores"][i, j, chosen].to(f64)
                source, target = s["table"][i].long()[chosen // page], s["to"][i].long()[at // page]
                k_new[target, at % page, j] = k_cache[source, chosen % page, j]
                v_new[target, at % page, j] = v_cache[source, chosen % page, j]
        return {"lens": torch.tensor([min(n, keep) for n in lens], dtype=torch.int32, device="cuda"), "scores": scores,
                "kept": kept, "k": k_new, "v": v_new}

    h, batch = case["heads"], case["batch"]
    group = h // hk
    out = torch.zeros((batch, h, d), dtype=f64, device="cuda")
    lse = torch.full((batch, h), -math.inf, dtype=f64, device="cuda")
    scores = s["scores"].to(f64) if case["op"] == "scored" else None
    for j in range(hk):  # one key head at a time
        mine = slice(j * group, (j + 1) * group)
        if case["op"] == "shared":
            where = torch.arange(case["prefix"], device="cuda")
            k0, v0 = tokens(s["k_cache"], ks, s["prefix"], where, j), tokens(s["v_cache"], vs, s["prefix"], where, j)
            t0 = torch.einsum("bgd,td->bgt", s["q"][:, mine].to(f64), k0) / math.sqrt(d)
            z0 = torch.logsumexp(t0, -1)
            o0 = torch.einsum("bgt,td->bgd", torch.exp(t0 - z0[..., None]), v0)
        for i, n in enumerate(lengths(case)):
            low = max(0, n - case["window"]) if case.get("window") else 0
            if n == 0:
                if case["op"] == "shared":
                    out[i, mine], lse[i, mine] = o0[i], z0[i]
                continue
            where = torch.arange(low, n, device="cuda")
            t = (s["q"][i, mine].to(f64) @ tokens(s["k_cache"], ks, s["table"][i], where, j).t()) / math.sqrt(d)
            v = tokens(s["v_cache"], vs, s["table"][i], where, j)
            z = torch.logsumexp(t, 1)
            if case["op"] == "shared":
                both = torch.logaddexp(z0[i], z)
                lse[i, mine] = both
                out[i, mine] = torch.exp(z0[i] - both)[:, None] * o0[i] + torch.exp(t - both[:, None]) @ v
            else:
                p = torch.exp(t - z[:, None])
                lse[i, mine], out[i, mine] = z, p @ v
                scores[i, j, low:n] += p.sum(0)
    return {"out": out, "lse": lse} if case["op"] == "shared" else {"out": out, "scores": scores, "lse": lse}
