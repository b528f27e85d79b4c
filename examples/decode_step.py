"""The attention block of a decode step, on one GPU, from the library's own operators:

    x ── 4-bit q·k·v projection ── rotary + append to the paged cache ── attention ── 4-bit output projection ── y

A batch of sequences of unequal lengths is given a prompt each, then decodes a few tokens; the
decode step is captured in a CUDA graph once and replayed, with only lengths and positions
changing.  The weights are random; ``reference`` computes the same block in plain 64-bit torch.

    python examples/decode_step.py [--batch 8] [--steps 4] [--cache e4m3]
"""
import argparse
import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import torch  # noqa: E402

import dense_linear_projection_gb300 as dlp  # noqa: E402


def quantise(W, group):
    """[N, K] fp32 weights as 4-bit codes, bf16 scales and zero points, by each group's range."""
    N, K = W.shape
    g = W.view(N, K // group, group)
    low, high = g.amin(2), g.amax(2)
    scales = ((high - low) / 15).clamp(min=1e-8).to(torch.bfloat16)
    zeros = (-low / scales.float()).round().clamp(0, 15)
    q = (g / scales.float()[..., None] + zeros[..., None]).round().clamp(0, 15).to(torch.uint8).view(N, K)
    return (q[:, 0::2] | (q[:, 1::2] << 4)).contiguous(), scales, zeros.to(torch.uint8)


def dequantise(codes, scales, zeros, group):
    """The weights that the codes stand for, [N, K] in 64 bits."""
    q = torch.stack([codes & 15, codes >> 4], 2).flatten(1).double()
    return (q - zeros.double().repeat_interleave(group, 1)) * scales.double().repeat_interleave(group, 1)


class AttentionBlock:
    """One layer's attention with 4-bit projections and a paged cache."""

    def __init__(self, width=1024, heads=8, kv_heads=2, dim=128, group=64, max_batch=16, pages=256, page=16,
                 max_positions=2048, cache="bf16", seed=0):
        gen = torch.Generator(device="cuda")
        gen.manual_seed(seed)
        self.heads, self.kv_heads, self.dim, self.group, self.page = heads, kv_heads, dim, group, page
        self.qkv_out = (heads + 2 * kv_heads) * dim
        self.stored = {}
        for name, (n, k) in {"qkv": (self.qkv_out, width), "out": (width, heads * dim)}.items():
            self.stored[name] = quantise(torch.randn((n, k), generator=gen, device="cuda") / k ** 0.5, group)
        self.tokens = max(max_batch, 256)  # of one projection call: prompts go in one after another
        self.qkv = dlp.Q4Projection(self.tokens, self.qkv_out, width, group, has_zeros=True)
        self.out = dlp.Q4Projection(self.tokens, width, heads * dim, group, has_zeros=True)
        self.w_qkv, self.w_out = self.qkv.pack(*self.stored["qkv"]), self.out.pack(*self.stored["out"])
        self.rope = dlp.rope_table(max_positions, dim)
        dtype = torch.float8_e4m3fn if cache == "e4m3" else torch.bfloat16
        k_cache, v_cache = (torch.zeros((pages, page, kv_heads, dim), device="cuda").to(dtype) for _ in "kv")
        scales = [torch.full((kv_heads,), 1 / 32, device="cuda") for _ in "kv"] if cache == "e4m3" else [None, None]
        self.kv = dlp.PagedKV(k_cache, v_cache, heads, max_batch, k_scale=scales[0], v_scale=scales[1])

    def _project_and_append(self, x, positions, table, seq_ids=None):
        rows = self.qkv(x, self.w_qkv).view(x.shape[0], self.heads + 2 * self.kv_heads, self.dim)
        q, k, v = rows.split([self.heads, self.kv_heads, self.kv_heads], 1)  # views: read in place
        return self.kv.append(q, k, v, positions, table, seq_ids=seq_ids, rope=self.rope, q_out=q)

    def prompt(self, x, positions, table, seq_ids):
        """Fill the cache from the tokens of some prompts (their own outputs are not computed here)."""
        for at in range(0, x.shape[0], self.tokens):
            part = slice(at, at + self.tokens)
            self._project_and_append(x[part].contiguous(), positions[part].contiguous(), table, seq_ids[part].contiguous())

    def step(self, x, positions, table, lengths):
        """One new token of each sequence: x [batch, width] -> [batch, width]."""
        q = self._project_and_append(x, positions, table)
        o = self.kv.attend(q, table, lengths)
        return self.out(o.view(x.shape[0], -1), self.w_out)


def reference(block, history, b, cache):
    """The block's output for the last token of sequence b, in 64 bits, from all its inputs.  The
    roundings that the block's data formats make (bf16 rows, the cache's type) are made here too."""
    bf16 = lambda t: t.to(torch.bfloat16).double()  # noqa: E731
    w_qkv, w_out = (dequantise(*block.stored[n], block.group) for n in ("qkv", "out"))
    x = torch.cat([h[b] for h in history]).double()
    rows = bf16(x @ w_qkv.t()).view(-1, block.heads + 2 * block.kv_heads, block.dim)
    half = block.dim // 2
    table = block.rope[:x.shape[0]].double()[:, None]
    cos, sin = table[..., :half], table[..., half:]
    turn = lambda t: torch.cat([t[..., :half] * cos - t[..., half:] * sin, t[..., half:] * cos + t[..., :half] * sin], -1)  # noqa: E731
    q, k, v = rows.split([block.heads, block.kv_heads, block.kv_heads], 1)
    q, k = bf16(turn(q)[-1]), turn(k)
    if cache == "e4m3":
        k, v = ((t.float() * 32).clamp(-448, 448).to(torch.float8_e4m3fn).double() / 32 for t in (k, v))
    else:
        k, v = bf16(k), bf16(v)
    k, v = (t.repeat_interleave(block.heads // block.kv_heads, 1) for t in (k, v))
    p = torch.softmax(torch.einsum("hd,thd->ht", q, k) / block.dim ** 0.5, 1)
    return bf16(torch.einsum("ht,thd->hd", p, v)).reshape(1, -1) @ w_out.t()


def main(argv=None):
    parser = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    parser.add_argument("--batch", type=int, default=8)
    parser.add_argument("--steps", type=int, default=4)
    parser.add_argument("--cache", choices=("bf16", "e4m3"), default="bf16")
    args = parser.parse_args(argv)
    width, batch = 1024, args.batch
    block = AttentionBlock(width, max_batch=batch, pages=batch * 16, cache=args.cache)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(1)
    randn = lambda n: torch.randn((n, width), generator=gen, device="cuda").to(torch.bfloat16)  # noqa: E731
    table = torch.randperm(batch * 16, generator=gen, device="cuda").to(torch.int32).view(batch, 16)

    # Prompts of unequal lengths (the first is empty), all tokens in one list.
    prompts = [(37 * b) % 150 for b in range(batch)]
    history = [[randn(n) for n in prompts]]
    seq_ids = torch.cat([torch.full((n,), b, dtype=torch.int32) for b, n in enumerate(prompts)]).cuda()
    positions = torch.cat([torch.arange(n, dtype=torch.int32) for n in prompts]).cuda()
    block.prompt(torch.cat(history[0]), positions, table, seq_ids)

    # One decode step in a graph; its inputs are buffers that change between replays.
    x, pos = randn(batch), torch.tensor(prompts, dtype=torch.int32, device="cuda")
    lengths = pos + 1
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        block.step(x, pos, table, lengths)  # once outside the graph, with the same effect on the cache
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = block.step(x, pos, table, lengths)

    worst = 0.0
    for step in range(args.steps):
        if step:
            x.copy_(randn(batch))
            pos += 1
            lengths += 1
        history.append([x[b:b + 1].clone() for b in range(batch)])
        graph.replay()
        torch.cuda.synchronize()
        for b in range(batch):
            ref = reference(block, history, b, args.cache)
            worst = max(worst, ((y[b:b + 1].double() - ref).norm() / ref.norm()).item())
    status = block.kv.status()
    if status != dlp.PROJ_OK:
        raise RuntimeError(dlp.proj_status_string(status))
    print(f"{args.steps} steps of {batch} sequences, {args.cache} cache: largest relative error {worst:.2e}")
    return worst


if __name__ == "__main__":
    main()
