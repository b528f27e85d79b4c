"""Cases and plain forms of the decode-step operators that stand between a model's projections:

* ``q4``: a projection whose weights are 4-bit codes with group scales,
  ``Y[m,n] = Σ_k X[m,k]·s[n,g(k)]·(q[n,k] − z[n,g(k)]) (+ bias[n])``;
* ``append``: the rotary position applied to the queries and keys of new tokens, and the keys and
  values written to their places in a paged cache;
* ``attend``: attention of one new token of each sequence over that cache.

``run`` computes a case in its plain form (elementary torch operations in 32 bits), or, where
``own`` is true, with the library's kernels.  ``exact`` gives the same outputs in 64 bits.
"""
import math

import torch

own = False

BF16, F32, E4M3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn


# ---------------------------------------------------------------- cases
def listed():
    return [
        # One token against the narrowest decode weight, symmetric codes, fp32 out: a call of a few
        # microseconds, where latency counts.
        dict(name="q4_one_token_narrow", op="q4", m=1, n=2048, k=8192, group=128, zeros=False, bias=False, out="f32"),
        # One token against the FFN up weight: the largest weight stream of a decode step.
        dict(name="q4_one_token_ffn", op="q4", m=1, n=28672, k=8192, group=128, zeros=True, bias=False, out="bf16"),
        # A decode batch of 16 against the square weight with a bias.
        dict(name="q4_batch16_bias", op="q4", m=16, n=8192, k=8192, group=64, zeros=True, bias=True, out="bf16"),
        # An odd batch, the finest groups, and neither N nor K a multiple of a tile.
        dict(name="q4_batch31_ragged", op="q4", m=31, n=12300, k=4128, group=32, zeros=False, bias=True, out="bf16"),
        # One new token of one sequence.
        dict(name="append_one_token", op="append", tokens=1, sequences=1, max_len=2048, heads=32, kv_heads=8, dim=128,
             rot=128, interleaved=False, page=16, heads_first=False, kv="bf16"),
        # A large decode batch into an 8-bit cache: one token of each sequence, at scattered places.
        dict(name="append_batch256_8bit", op="append", tokens=256, sequences=256, max_len=1024, heads=64, kv_heads=8,
             dim=128, rot=64, interleaved=True, page=64, heads_first=True, kv="e4m3"),
        # Prompts of three sequences together, every query head with a key head of its own (the
        # 12288-wide query, key and value projection), an odd number of tokens.
        dict(name="append_prompts", op="append", tokens=8191, sequences=3, max_len=0, heads=32, kv_heads=32, dim=128,
             rot=128, interleaved=False, page=16, heads_first=False, kv="bf16"),
        # The start of an answer: a few cached tokens of one sequence.
        dict(name="attend_short", op="attend", batch=1, max_len=37, ragged=False, heads=32, kv_heads=8, dim=128,
             page=16, heads_first=False, window=0, kv="bf16"),
        # One sequence with a long context: the work has to be split over its length.
        dict(name="attend_one_long", op="attend", batch=1, max_len=131071, ragged=False, heads=64, kv_heads=8, dim=128,
             page=16, heads_first=False, window=0, kv="bf16"),
        # A serving batch of unequal lengths, one of them empty.
        dict(name="attend_batch64_ragged", op="attend", batch=64, max_len=8192, ragged=True, heads=64, kv_heads=8,
             dim=128, page=32, heads_first=True, window=0, kv="bf16"),
        # Every query head with a key head of its own, narrow heads, a sliding window.
        dict(name="attend_window_narrow", op="attend", batch=24, max_len=4000, ragged=True, heads=32, kv_heads=32,
             dim=64, page=64, heads_first=False, window=1000, kv="bf16"),
        # A batch of long contexts in an 8-bit cache.
        dict(name="attend_batch16_8bit", op="attend", batch=16, max_len=32768, ragged=True, heads=64, kv_heads=8,
             dim=128, page=64, heads_first=False, window=0, kv="e4m3"),
    ]


def _log(rng, low, high):
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


#: No drawn case of an operator moves more bytes than this (the largest listed one of its kind).
MOST_BYTES = {"q4": 123e6, "append": 410e6, "attend": 1100e6}


def draw(rng):
    while True:
        op = rng.choice(("q4", "append", "attend"))
        if op == "q4":
            group = rng.choice((32, 64, 128))
            case = dict(op=op, m=_log(rng, 1, 32), n=_log(rng, 500, 28672), k=group * _log(rng, 1024 // group, 8192 // group),
                        group=group, zeros=rng.random() < 0.5, bias=rng.random() < 0.5, out=rng.choice(("bf16", "bf16", "f32")))
        else:
            dim = rng.choice((64, 128, 128))
            kv_heads = rng.choice((1, 2, 4, 8, 8, 16, 32))
            heads = kv_heads * rng.choice([g for g in (1, 2, 4, 7, 8, 16) if g * kv_heads <= 64])
            both = dict(heads=heads, kv_heads=kv_heads, dim=dim, page=rng.choice((16, 32, 64)),
                        heads_first=rng.random() < 0.5, kv=rng.choice(("bf16", "bf16", "e4m3")))
            if op == "append":
                tokens = _log(rng, 1, 8192)
                rot = {"rot": rng.choice((dim, dim, dim // 2)), "interleaved": rng.random() < 0.5}
                if tokens <= 256 and rng.random() < 0.7:
                    case = dict(op=op, tokens=tokens, sequences=tokens, max_len=_log(rng, 32, 1024), **both, **rot)
                else:
                    case = dict(op=op, tokens=tokens, sequences=min(tokens, rng.randint(1, 5)), max_len=0, **both, **rot)
            else:
                case = dict(op=op, batch=_log(rng, 1, 128), max_len=_log(rng, 20, 131072), ragged=rng.random() < 0.7,
                            window=rng.choice((0, 0, _log(rng, 16, 4096))), **both)
                # The plain form pads every sequence to the longest.
                if case["batch"] * case["max_len"] * kv_heads * dim > 64 * 8192 * 8 * 128:
                    continue
        if work(case)["bytes"] <= MOST_BYTES[op]:
            return case


def lengths(case):
    """Cached tokens of each sequence of an ``attend`` case; a ragged batch has an empty one."""
    n, most = case["batch"], case["max_len"]
    if not case["ragged"] or n == 1:
        return [most] * n
    return [most if i == 0 else 0 if i == 1 else 1 + (most - 1) * ((29 * i + 17) % 97) // 96 for i in range(n)]


def places(case):
    """(sequence, position) of each token of an ``append`` case."""
    t, s = case["tokens"], case["sequences"]
    if t == s and case["max_len"]:
        return list(range(t)), [(case["max_len"] - 1) * ((61 * i + 96) % 97) // 96 for i in range(t)]
    first = [-(-t * i // s) for i in range(s + 1)]
    seq = [i for i in range(s) for _ in range(first[i], first[i + 1])]
    return seq, [13 * i + at - first[i] for at, i in enumerate(seq)]


def work(case):
    if case["op"] == "q4":
        m, n, k = case["m"], case["n"], case["k"]
        groups = n * (k // case["group"])
        size = n * k / 2 + groups * (2.5 if case["zeros"] else 2) + m * k * 2 + m * n * (4 if case["out"] == "f32" else 2)
        return {"bytes": size + (2 * n if case["bias"] else 0), "flops": 2.0 * m * n * k}
    h, hk, d, e = case["heads"], case["kv_heads"], case["dim"], 1 if case["kv"] == "e4m3" else 2
    if case["op"] == "append":
        t = case["tokens"]
        size = t * (h + 2 * hk) * d * 2 + t * h * d * 2 + t * 2 * hk * d * e + t * (case["rot"] * 4 + 12)
        return {"bytes": float(size), "flops": 3.0 * t * (h + hk) * case["rot"]}
    seen = [min(x, case["window"]) if case["window"] else x for x in lengths(case)]
    size = sum(seen) * hk * d * 2 * e + case["batch"] * h * (d * 4 + 4) + sum(-(-x // case["page"]) for x in seen) * 4
    return {"bytes": float(size), "flops": 4.0 * sum(seen) * h * d}


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


def _inputs(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed) * 1000003 + 17)
    s = {"case": case}
    if case["op"] == "q4":
        m, n, k, groups = case["m"], case["n"], case["k"], case["k"] // case["group"]
        s["x"] = _randn(gen, (m, k))
        # Codes of weights that are about normal, two to a byte: the even k in the low four bits.
        codes = torch.empty((n, k // 2), device="cuda", dtype=torch.uint8)
        for at in range(0, n, 4096):
            q = torch.randn((min(4096, n - at), k), generator=gen, device="cuda").mul_(2.7).add_(7.5).round_().clamp_(0, 15)
            q = q.to(torch.uint8)
            codes[at:at + 4096] = q[:, 0::2] | (q[:, 1::2] << 4)
        s["codes"] = codes
        s["scales"] = ((torch.rand((n, groups), generator=gen, device="cuda") + 0.5) / (2.7 * math.sqrt(k))).to(BF16)
        s["zeros"] = torch.randint(5, 11, (n, groups), generator=gen, device="cuda", dtype=torch.uint8) if case["zeros"] else None
        s["bias"] = _randn(gen, (n,), 0.02) if case["bias"] else None
        return s
    h, hk, d, page = case["heads"], case["kv_heads"], case["dim"], case["page"]
    if case["op"] == "append":
        seq, pos = places(case)
        width = max(pos) // page + 1
        pages = case["sequences"] * width
        # The rows of a query, key and value projection: queries, then keys, then values.
        rows = _randn(gen, (case["tokens"], h + 2 * hk, d))
        s["q"], s["k"], s["v"] = rows[:, :h], rows[:, h:h + hk], rows[:, h + hk:]
        s["seq"] = torch.tensor(seq, dtype=torch.int32, device="cuda")
        s["pos"] = torch.tensor(pos, dtype=torch.int32, device="cuda")
        # cos, then sin, of position · 10000^(−2i / rot) for each position.
        at = torch.arange(width * page, dtype=torch.float64, device="cuda")[:, None]
        half = case["rot"] // 2
        angle = at * (10000.0 ** (-torch.arange(half, dtype=torch.float64, device="cuda") / half))[None, :]
        s["rope"] = torch.cat([angle.cos(), angle.sin()], 1).to(F32)
    else:
        lens = lengths(case)
        width = max(1, -(-max(lens) // page))
        pages = sum(-(-x // page) for x in lens) + 8
        s["q"] = _randn(gen, (case["batch"], h, d))
        s["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"] = _cache(gen, case, pages)
    free = torch.randperm(pages, generator=gen, device="cuda").to(torch.int32)
    if case["op"] == "append":
        s["table"] = free.view(case["sequences"], width)
    else:
        table, used = torch.zeros((case["batch"], width), dtype=torch.int32, device="cuda"), 0
        for i, x in enumerate(lens):
            need = -(-x // page)
            table[i, :need] = free[used:used + need]
            used += need
        s["table"] = table
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    if own:
        import dense_linear_projection_gb300 as dlp
        if case["op"] == "q4":
            s["proj"] = dlp.Q4Projection(case["m"], case["n"], case["k"], case["group"], has_zeros=case["zeros"],
                                         y_dtype=dlp.PROJ_F32 if case["out"] == "f32" else dlp.PROJ_BF16,
                                         has_bias=case["bias"])
            s["packed"] = s["proj"].pack(s["codes"], s["scales"], s["zeros"])
        else:
            s["kv"] = dlp.PagedKV(s["k_cache"], s["v_cache"], case["heads"], max_sequences=s["table"].shape[0],
                                  k_scale=s["k_scale"], v_scale=s["v_scale"])
    return s


# ---------------------------------------------------------------- one pass
def run(state):
    s, case = state, state["case"]
    if own:
        if case["op"] == "q4":
            return s["proj"](s["x"], s["packed"], s["bias"])
        if case["op"] == "append":
            q = s["kv"].append(s["q"], s["k"], s["v"], s["pos"], s["table"], seq_ids=s["seq"], rope=s["rope"],
                               interleaved=case["interleaved"])
            return {"q": q, "k": s["k_cache"], "v": s["v_cache"]}
        out, lse = s["kv"].attend(s["q"], s["table"], s["lens"], window=case["window"], return_lse=True)
        return {"out": out, "lse": lse}
    return {"q4": _plain_q4, "append": _plain_append, "attend": _plain_attend}[case["op"]](s, case)


def _plain_q4(s, case):
    n, k, group = case["n"], case["k"], case["group"]
    q = torch.stack([s["codes"] & 15, s["codes"] >> 4], 2).view(n, k // group, group).to(F32)
    z = s["zeros"].to(F32)[:, :, None] if case["zeros"] else 8.0
    w = ((q - z) * s["scales"].to(F32)[:, :, None]).view(n, k)
    y = s["x"].to(F32) @ w.t()
    if case["bias"]:
        y = y + s["bias"].to(F32)
    return y if case["out"] == "f32" else y.to(BF16)


def _rotate(x, cos, sin, rot, interleaved):
    x, rest = x[..., :rot], x[..., rot:]
    a, b = (x[..., 0::2], x[..., 1::2]) if interleaved else (x[..., :rot // 2], x[..., rot // 2:])
    u, v = a * cos - b * sin, b * cos + a * sin
    x = torch.stack([u, v], -1).flatten(-2) if interleaved else torch.cat([u, v], -1)
    return torch.cat([x, rest], -1)


def _plain_append(s, case):
    rot, page = case["rot"], case["page"]
    pos = s["pos"].long()
    cos, sin = s["rope"][pos].unsqueeze(1).split(rot // 2, -1)
    q = _rotate(s["q"].to(F32), cos, sin, rot, case["interleaved"])
    k, v = _rotate(s["k"].to(F32), cos, sin, rot, case["interleaved"]), s["v"].to(F32)
    if case["kv"] == "e4m3":
        k = (k / s["k_scale"][:, None]).clamp(-448, 448)
        v = (v / s["v_scale"][:, None]).clamp(-448, 448)
    to, at = s["table"][s["seq"].long(), pos // page].long(), pos % page
    if case["kv"] == "e4m3":  # bytes: an indexed write of 8-bit floating values is not there for every layout
        s["k_cache"].view(torch.uint8)[to, at] = k.to(E4M3).view(torch.uint8)
        s["v_cache"].view(torch.uint8)[to, at] = v.to(E4M3).view(torch.uint8)
    else:
        s["k_cache"][to, at], s["v_cache"][to, at] = k.to(BF16), v.to(BF16)
    return {"q": q.to(BF16), "k": s["k_cache"], "v": s["v_cache"]}


def _plain_attend(s, case):
    b, h, hk, d = case["batch"], case["heads"], case["kv_heads"], case["dim"]
    table, lens = s["table"].long(), s["lens"].long()

    def gathered(cache, scale):  # [batch, kv_heads, tokens, dim], every sequence padded to the longest
        if case["kv"] == "e4m3":
            x = cache.view(torch.uint8)[table].view(E4M3).to(F32) * scale[:, None]
        else:
            x = cache[table].to(F32)
        return x.reshape(b, -1, hk, d).transpose(1, 2)

    at = torch.arange(table.shape[1] * case["page"], device="cuda")[None, :]
    seen = at < lens[:, None]
    if case["window"]:
        seen = seen & (at >= lens[:, None] - case["window"])
    seen = seen[:, None, None, :]
    logits = s["q"].to(F32).view(b, hk, h // hk, d) @ gathered(s["k_cache"], s["k_scale"]).transpose(2, 3)
    logits = torch.where(seen, logits * (1.0 / math.sqrt(d)), -math.inf)
    top = logits.amax(-1, keepdim=True).clamp(min=-1e30)
    p = torch.exp(logits - top)
    total = p.sum(-1, keepdim=True)
    v = torch.where(seen.transpose(2, 3), gathered(s["v_cache"], s["v_scale"]), 0.0)
    out = (p @ v) / torch.where(total > 0, total, 1.0)
    lse = (top + total.log()).view(b, h)
    return {"out": out.reshape(b, h, d).to(BF16), "lse": torch.where(s["lens"][:, None] > 0, lse, -math.inf)}


# ---------------------------------------------------------------- the definition, in 64 bits
def exact(case, seed):
    s = _inputs(case, seed)
    f64 = torch.float64
    if case["op"] == "q4":
        # Σ_g s[n,g]·(Σ_k x·q − z·Σ_k x), some rows of the weights at a time.
        m, k, group = case["m"], case["k"], case["group"]
        x = s["x"].to(f64).view(m, k // group, group)
        parts = []
        for at in range(0, case["n"], 2048):
            c = s["codes"][at:at + 2048]
            q = torch.empty((c.shape[0], k), dtype=f64, device="cuda")
            q[:, 0::2], q[:, 1::2] = torch.remainder(c, 16).to(f64), torch.div(c, 16, rounding_mode="floor").to(f64)
            by_group = torch.einsum("mgi,ngi->gmn", x, q.view(-1, k // group, group))
            z = s["zeros"][at:at + 2048].to(f64) if case["zeros"] else torch.full((c.shape[0], k // group), 8.0, dtype=f64, device="cuda")
            by_group -= x.sum(2).t()[:, :, None] * z.t()[:, None, :]
            parts.append((by_group * s["scales"][at:at + 2048].to(f64).t()[:, None, :]).sum(0))
        y = torch.cat(parts, 1)
        return y + s["bias"].to(f64) if case["bias"] else y
    d, page = case["dim"], case["page"]
    if case["op"] == "append":
        half, style = case["rot"] // 2, case["interleaved"]
        index = torch.arange(half, device="cuda")
        first, second = (2 * index, 2 * index + 1) if style else (index, index + half)
        turn = torch.complex(s["rope"][:, :half].to(f64), s["rope"][:, half:].to(f64))[s["pos"].long()][:, None, :]

        def turned(x):
            x = x.to(f64)
            y = torch.complex(x[..., first], x[..., second]) * turn
            x[..., first], x[..., second] = y.real, y.imag
            return x

        k_cache, v_cache = s["k_cache"].to(f64), s["v_cache"].to(f64)
        k, v = turned(s["k"]), s["v"].to(f64)
        if case["kv"] == "e4m3":
            k = torch.minimum(torch.maximum(k / s["k_scale"].to(f64)[:, None], k.new_tensor(-448.0)), k.new_tensor(448.0))
            v = torch.minimum(torch.maximum(v / s["v_scale"].to(f64)[:, None], v.new_tensor(-448.0)), v.new_tensor(448.0))
        seq, pos = places(case)
        table = s["table"].cpu()
        to = torch.tensor([int(table[i, p // page]) for i, p in zip(seq, pos)], device="cuda")
        at = torch.tensor([p % page for p in pos], device="cuda")
        k_cache[to, at], v_cache[to, at] = k, v
        return {"q": turned(s["q"]), "k": k_cache, "v": v_cache}
    h, hk = case["heads"], case["kv_heads"]
    out = torch.zeros((case["batch"], h, d), dtype=f64, device="cuda")
    lse = torch.full((case["batch"], h), -math.inf, dtype=f64, device="cuda")
    ks = s["k_scale"].to(f64) if s["k_scale"] is not None else torch.ones(hk, dtype=f64, device="cuda")
    vs = s["v_scale"].to(f64) if s["v_scale"] is not None else torch.ones(hk, dtype=f64, device="cuda")
    for i, n in enumerate(lengths(case)):
        low = max(0, n - case["window"]) if case["window"] else 0
        if n == 0:
            continue
        tokens = torch.arange(low, n, device="cuda")
        pages, at = s["table"][i].long()[tokens // page], tokens % page
        for j in range(hk):  # one key head at a time
            own_heads = slice(j * (h // hk), (j + 1) * (h // hk))
            k = s["k_cache"][:, :, j].to(f64)[pages, at] * ks[j]
            t = (s["q"][i, own_heads].to(f64) @ k.t()) / math.sqrt(d)
            lse[i, own_heads] = torch.logsumexp(t, 1)
            v = s["v_cache"][:, :, j].to(f64)[pages, at] * vs[j]
            out[i, own_heads] = torch.softmax(t, 1) @ v
    return {"out": out, "lse": lse}
