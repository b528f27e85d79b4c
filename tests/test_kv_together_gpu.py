"""The paged cache's further operators together, as a server would use them: a batch behind a common
prefix, normed appends, attention over prefix and own tokens, scores, evictions to fresh pages, and on
with rotary rows that are no places any more; and two captured graphs of one handle.

The reference keeps every token in 64 bits and rounds keys to bf16 as the cache does, but from 64-bit
values: where one lies next to a rounding boundary the two differ by a unit in the last place, 2⁻⁷ of a
key's element in one of 2⁻²⁰/2⁻⁸ cases.  In a logit of dim elements that is far below 2⁻⁸ of its terms' root
sum of squares, so outputs, rounded to bf16 (2⁻⁹ of each), agree to 1e-2 in norm with room to spare."""
import pytest

import kv_util as ku

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("captured", [False, True])
@pytest.mark.parametrize("dim,page", [(64, 16), (128, 8), (64, 5)])
def test_serving_loop(captured, dim, page):
    import torch
    import dense_linear_projection_gb300 as dlp
    B, H, hk, P, keep, recent, steps = 3, 8, 2, 70, 24, 6, 60
    G, eps, bf16 = H // hk, 1e-6, torch.bfloat16
    g = torch.Generator(device="cuda")
    g.manual_seed(dim + page)
    randn = lambda *s: torch.randn(s, generator=g, device="cuda").to(bf16)  # noqa: E731
    room = -(-(keep + steps) // page)
    prefix_pages = -(-P // page)
    k_cache, v_cache = ku.make_cache(prefix_pages + 2 * B * room, page, hk, dim)
    free = torch.randperm(prefix_pages + 2 * B * room, generator=g, device="cuda").to(torch.int32)
    prefix, halves = free[:prefix_pages].contiguous(), free[prefix_pages:].view(2, B, room)
    table, spare = halves[0].contiguous(), halves[1].contiguous()
    kv = dlp.PagedKV(k_cache, v_cache, H, B)
    rope = dlp.rope_table(P + steps + 1, dim)
    wq, wk = (1 + 0.2 * torch.randn(dim, generator=g, device="cuda") for _ in "qk")

    def normed(x, w, row):
        x = x.double()
        x = x * w.double() / torch.sqrt(x.square().mean(-1, keepdim=True) + eps)
        cos, sin = rope[row].double().split(dim // 2)
        a, b = x[..., :dim // 2], x[..., dim // 2:]
        return torch.cat([a * cos - b * sin, b * cos + a * sin], -1)

    # The prefix: one sequence of its own table.
    rows = randn(P, H + 2 * hk, dim)
    at = torch.arange(P, dtype=torch.int32, device="cuda")
    kv.append(None, rows[:, H:H + hk], rows[:, H + hk:], at, prefix[None], seq_ids=torch.zeros_like(at), rope=rope, k_norm=wk, eps=eps)
    prefix_k = torch.stack([normed(rows[t, H:H + hk], wk, t) for t in range(P)]).to(bf16).double()
    prefix_v = rows[:, H + hk:].double()
    own_k = [[[] for _ in range(hk)] for _ in range(B)]  # of each sequence and key head, in the order of their places
    own_v = [[[] for _ in range(hk)] for _ in range(B)]

    x = randn(B, H + 2 * hk, dim)
    places, text = torch.zeros(B, dtype=torch.int32, device="cuda"), torch.full((B,), P, dtype=torch.int32, device="cuda")
    scores = torch.zeros((B, hk, room * page), device="cuda")
    lens = places + 1

    def step():
        q = kv.append(x[:, :H], x[:, H:H + hk], x[:, H + hk:], places, table, rope=rope, q_norm=wq, k_norm=wk, eps=eps, rope_rows=text)
        out = kv.attend_shared(q, prefix, P, table, lens)
        kv.attend_scored(q, table, lens, scores)
        return out

    graph, out = None, None
    if captured:
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            step()
        torch.cuda.current_stream().wait_stream(side)
        scores.zero_()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = step()
    want_scores = [[[] for _ in range(hk)] for _ in range(B)]
    evictions = 0
    for t in range(steps):
        if t:
            x.copy_(randn(B, H + 2 * hk, dim))
        if captured:
            graph.replay()
        else:
            out = step()
        for b in range(B):
            q64 = normed(x[b, :H], wq, P + t).to(bf16).double()
            k64 = normed(x[b, H:H + hk], wk, P + t).to(bf16).double()
            for j in range(hk):
                own_k[b][j].append(k64[j])
                own_v[b][j].append(x[b, H + hk + j].double())
                want_scores[b][j].append(0.0)
                k, v = torch.stack(own_k[b][j]), torch.stack(own_v[b][j])
                s = q64[j * G:(j + 1) * G] @ torch.cat([prefix_k[:, j], k]).t() / dim ** 0.5
                ref = torch.softmax(s, 1) @ torch.cat([prefix_v[:, j], v])
                assert (out[b, j * G:(j + 1) * G].double() - ref).norm() <= 1e-2 * ref.norm(), (t, b, j)
                w = torch.softmax(s[:, P:], 1).sum(0)
                want_scores[b][j] = [a + c for a, c in zip(want_scores[b][j], w.tolist())]
                have = scores[b, j, :len(want_scores[b][j])].double()
                assert (have - torch.tensor(want_scores[b][j], dtype=torch.float64, device="cuda")).abs().max() <= 1e-2 * (t + 1), (t, b, j)
        places += 1
        text += 1
        lens += 1
        if t in (27, 41, 55):  # past the budget: down to it, into the spare pages, and on
            n = (lens - 1).contiguous()
            new_lens, new_scores, kept = kv.evict(table, n, scores, spare, keep, recent=recent)
            assert new_lens.tolist() == [min(v, keep) for v in n.tolist()]
            for b in range(B):
                for j in range(hk):
                    stay = [i for i in kept[b, j].tolist() if i >= 0]
                    old = scores[b, j, :n[b]].tolist()
                    order = sorted(range(n[b].item() - recent), key=lambda i: (-old[i], i))[:keep - recent]
                    assert stay == sorted(order) + list(range(n[b].item() - recent, n[b].item()))
                    for of in (own_k, own_v, want_scores):
                        of[b][j] = [of[b][j][i] for i in stay]
            scores.copy_(new_scores)
            taken = table.clone()
            table.copy_(spare)
            spare.copy_(taken)
            places.copy_(new_lens)
            lens.copy_(new_lens + 1)
            evictions += 1
    assert evictions == 3 and kv.status() == dlp.PROJ_OK


def test_two_graphs_of_one_handle():
    # Each capture has a workspace of its own: replays in any order give what eager calls give.
    import torch
    import dense_linear_projection_gb300 as dlp
    H, hk, D, page = 16, 2, 128, 16
    k_cache, v_cache = ku.make_cache(400, page, hk, D)
    kv = dlp.PagedKV(k_cache, v_cache, H, 9)
    free = torch.randperm(400).to(torch.int32).cuda()
    prefix = free[:200].contiguous()
    inputs = []
    for batch, prefix_len, width in ((9, 3000, 10), (2, 130, 40)):
        inputs.append((torch.randn((batch, H, D), device="cuda").to(torch.bfloat16), prefix_len, free[200:200 + batch * width].view(batch, width).contiguous(),
                       torch.arange(batch, dtype=torch.int32, device="cuda") * 17 + 1, torch.zeros((batch, hk, width * page), device="cuda")))

    def call(q, prefix_len, table, lens, scores):
        return (kv.attend_shared(q, prefix, prefix_len, table, lens),
                *kv.attend_scored(q, table, lens, scores, scores_out=torch.empty_like(scores)))

    want = [call(*x) for x in inputs]
    torch.cuda.synchronize()
    graphs, outs = [], []
    for x in inputs:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(call(*x))
        graphs.append(graph)
    for which in (0, 1, 1, 0, 0, 1, 0, 1, 1, 0):
        for o in outs[which]:
            o.zero_()
        graphs[which].replay()
        assert all(torch.equal(a, b) for a, b in zip(outs[which], want[which]))
    assert kv.status() == dlp.PROJ_OK


def test_two_handles_on_two_streams():
    import torch
    import dense_linear_projection_gb300 as dlp
    H, hk, D, page = 8, 2, 64, 16
    sides = [torch.cuda.Stream() for _ in range(2)]
    work = []
    for k, side in enumerate(sides):
        k_cache, v_cache = ku.make_cache(300, page, hk, D, seed=k)
        kv = dlp.PagedKV(k_cache, v_cache, H, 20)
        q = torch.randn((20, H, D), device="cuda").to(torch.bfloat16)
        table = torch.randperm(100).to(torch.int32).cuda().view(20, 5)
        lens = torch.arange(20, dtype=torch.int32, device="cuda") * 4
        prefix = torch.arange(100, 300, dtype=torch.int32, device="cuda")
        scores = torch.rand((20, hk, 80), device="cuda")
        work.append((kv, q, prefix, table, lens, scores))

    def call(kv, q, prefix, table, lens, scores):
        return (kv.attend_shared(q, prefix, 3001, table, lens), *kv.attend_scored(q, table, lens, scores, scores_out=torch.empty_like(scores)))

    want = [call(*w) for w in work]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(20):
        for k, side in enumerate(sides):
            with torch.cuda.stream(side):
                got[k].append(call(*work[k]))
    torch.cuda.synchronize()
    for k in range(2):
        for results in got[k]:
            assert all(torch.equal(a, b) for a, b in zip(results, want[k]))
        assert work[k][0].status() == dlp.PROJ_OK


def test_tensors_of_a_given_stream():
    # ``stream=`` as for the other calls: results come from that stream's memory and are complete on it.
    import torch
    import dense_linear_projection_gb300 as dlp
    k_cache, v_cache = ku.make_cache(40, 16, 2, 64)
    kv = dlp.PagedKV(k_cache, v_cache, 8, 2)
    q = torch.randn((2, 8, 64), device="cuda").to(torch.bfloat16)
    table, prefix = torch.arange(10, dtype=torch.int32, device="cuda").view(2, 5), torch.arange(10, 30, dtype=torch.int32, device="cuda")
    to = torch.arange(30, 34, dtype=torch.int32, device="cuda").view(2, 2)
    lens, scores = torch.tensor([70, 3], dtype=torch.int32, device="cuda"), torch.rand((2, 2, 80), device="cuda")
    want = (kv.attend_shared(q, prefix, 300, table, lens), *kv.attend_scored(q, table, lens, scores, scores_out=torch.empty_like(scores)),
            *kv.evict(table, lens, scores, to, 20, 3))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for stream in (side, side.cuda_stream):
        scores_out = torch.empty_like(scores)
        side.wait_stream(torch.cuda.current_stream())
        got = (kv.attend_shared(q, prefix, 300, table, lens, stream=stream),
               *kv.attend_scored(q, table, lens, scores, scores_out=scores_out, stream=stream),
               *kv.evict(table, lens, scores, to, 20, 3, stream=stream))
        side.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert kv.status() == dlp.PROJ_OK
