"""A decoder of int4 linears end to end: the layer operators as a serving program calls them.

    python -m examples.decoder [--layers 4] [--prompts 700,2000,33] [--steps 32] [--system 0]

A batch of prompts goes through the layers in one pass (w4_attn_prefill), then every sequence gets one
token a step (w4_attn_decode), the step recorded once as a HIP graph and replayed. Weights are random
(RTN-packed), and hidden states stand in for embeddings: a step's input is the last step's output.

One layer, with the residual stream h in fp32:
    y, h = residual_norm(previous block's output, h)     w4_residual_norm
    qkv  = y Wqkv^T                                      w4_gemv / w4_gemm
    q    = rope(qkv), k and v into the paged cache       w4_rope_append
    a    = attention over the cache                      w4_attn_prefill / w4_attn_decode
    y, h = residual_norm(a Wo^T, h)                      w4_residual_norm
    out  = (silu(y Wgate^T) * y Wup^T) Wdown^T           w4_gemv_glu, w4_gemv / w4_gemm

With --system N the prompts follow one system prompt of N tokens. Its keys and values are made once and
shared: the tables of every pass, the recorded step's too, are made on the GPU from the pool's free
pages (w4_batch_tables), and attention reads the shared keys once for all sequences (w4_attn_shared).
"""
import argparse
from dataclasses import dataclass

import torch

import int4_weight_only_amd as w4
import workloads


@dataclass
class Shape:
    """Sizes of a layer (the defaults: the 7B-class decoder of the workloads)."""
    layers: int = 4
    hidden: int = workloads.HIDDEN
    heads: int = 28
    kv_heads: int = workloads.KV_DIM // 128
    head_dim: int = 128
    inter: int = workloads.INTER
    group_size: int = 128
    page_size: int = 64
    window: int = 0
    sinks: int = 0
    rope_base: float = 1e6


class Cache:
    """Pages for `lens[b]` positions of each sequence b, one table for all layers."""

    def __init__(self, shape, lens, device):
        pages = [-(-n // shape.page_size) for n in lens]
        total, cols = sum(pages), max(pages)
        table = torch.zeros(len(lens), cols, dtype=torch.int32)
        order = torch.randperm(total, generator=torch.Generator().manual_seed(1)).to(torch.int32)
        at = 0
        for b, n in enumerate(pages):
            table[b, :n] = order[at:at + n]
            at += n
        self.table = table.to(device)
        self.kv_len = torch.zeros(len(lens), dtype=torch.int32, device=device)
        size = (shape.layers, total, shape.page_size, shape.kv_heads, shape.head_dim)
        self.k = torch.empty(size, dtype=torch.bfloat16, device=device)
        self.v = torch.empty(size, dtype=torch.bfloat16, device=device)

    def layer(self, i):
        return self.k[i], self.v[i], self.table, self.kv_len


class SharedCache:
    """A pool of `pages` pages for `n` sequences that may share the system prompt, whose keys are those
    of one sequence more, the last. Which pages a sequence has is known on the GPU alone."""

    def __init__(self, shape, n, pages, most, device):
        def ints(*size):
            return torch.zeros(size, dtype=torch.int32, device=device)

        self.shape, self.n = shape, n
        self.table = ints(n + 1, -(-most // shape.page_size))
        self.kv_len, self.spans = ints(n + 1), ints(n + 1, 2)
        self.ring = torch.arange(pages, dtype=torch.int32, device=device)
        self.state = ints(3)
        self.state[1] = pages
        self.missing = ints(1)
        self.prefix_of = torch.full((n + 1,), -1, dtype=torch.int32, device=device)
        self.prefix_len = ints(1)
        size = (shape.layers, pages, shape.page_size, shape.kv_heads, shape.head_dim)
        self.k = torch.empty(size, dtype=torch.bfloat16, device=device)
        self.v = torch.empty(size, dtype=torch.bfloat16, device=device)

    def layer(self, i):
        return self.k[i], self.v[i], self.table, self.kv_len

    def advance(self, n_new, T):
        """Pages for n_new[b] tokens of each sequence, T in all (-1: the sequence ends and its pages
        are free again); returns where each sequence's rows begin. Where the pool runs dry, keys of the
        pass have no place, and it cannot be made again: its lengths are changed in place. See check."""
        starts = w4.w4_batch_tables(self.kv_len, n_new, self.spans, self.table, self.shape.page_size,
                                    self.ring, self.state, T, in_place=True)[0]
        self.missing += self.state[2:]
        return starts

    def check(self):
        """Raises if any pass so far, replayed ones among them, ran out of pages. Waits for the GPU."""
        if self.missing.item() > 0:
            raise RuntimeError(f"the pool of {self.ring.shape[0]} pages is too small: results are wrong")

    def share(self, b):
        """Sequence b begins after the system prompt."""
        P = self.kv_len[self.n]
        self.prefix_len[0] = P
        self.prefix_of[b] = 0
        self.kv_len[b] = P
        self.spans[b] = P // self.shape.page_size  # (a page that it shares in part is not its own)

    def attention(self, i, q, q_start):
        s = self.shape
        return w4.w4_attn_shared(q, *self.layer(i), self.prefix_of, self.table[self.n:],
                                 self.prefix_len, q_start=q_start, window=s.window, sinks=s.sinks)


class Decoder:
    def __init__(self, shape, device="cuda", seed=0):
        self.shape = s = shape
        g = torch.Generator(device=device).manual_seed(seed)

        def linear(d_out, d_in):
            w = torch.randn(d_out, d_in, generator=g, device=device) * d_in ** -0.5
            return *w4.w4_pack(w, s.group_size, w4.W4_SYM), None, d_in, s.group_size

        def norm():
            return (1 + 0.1 * torch.randn(s.hidden, generator=g, device=device)).bfloat16()

        self.layers = [dict(
            norm_in=norm(), norm_mlp=norm(),
            qkv=linear((s.heads + 2 * s.kv_heads) * s.head_dim, s.hidden),
            o=linear(s.hidden, s.heads * s.head_dim),
            gate_up=linear(2 * s.inter, s.hidden),
            down=linear(s.hidden, s.inter)) for _ in range(s.layers)]
        self.norm_out = norm()
        self.inv_freq = w4.w4_rope_frequencies(s.head_dim, base=s.rope_base)[0].to(device)

    def fused_gate(self, T):
        """Does w4_gemv_glu serve T tokens?"""
        s = self.shape
        k_pad = w4.packed_layout(2 * s.inter, s.hidden, s.group_size)[0]
        return T <= 4 and s.group_size in (128, 256) and T * k_pad <= 32768

    def forward(self, h, cache, q_start=None):
        """h fp32 [T][hidden], overwritten by the residual stream: the T newest tokens of the
        sequences (cache.kv_len counts them already), one per sequence if q_start is None. Returns
        the normalized output, bf16 [T][hidden]."""
        s = self.shape
        out = None
        for i, layer in enumerate(self.layers):
            y, h = w4.w4_residual_norm(out, h, layer["norm_in"],
                                       residual_out=None if out is None else h)
            qkv = w4.w4_linear(y, *layer["qkv"])
            q = w4.w4_rope_append(qkv, s.heads, *cache.layer(i), self.inv_freq, q_start)
            if isinstance(cache, SharedCache):
                a = cache.attention(i, q, q_start)
            elif q_start is None:
                a = w4.w4_attn_decode(q, *cache.layer(i), window=s.window, sinks=s.sinks)
            else:
                a = w4.w4_attn_prefill(q, *cache.layer(i), q_start, window=s.window,
                                       sinks=s.sinks)
            y, h = w4.w4_residual_norm(w4.w4_linear(a, *layer["o"]), h, layer["norm_mlp"],
                                       residual_out=h)
            if self.fused_gate(y.shape[0]):
                z = w4.w4_gemv_glu(y, *layer["gate_up"])
            else:
                gate, up = w4.w4_linear(y, *layer["gate_up"]).chunk(2, dim=1)
                z = torch.nn.functional.silu(gate) * up
            out = w4.w4_linear(z, *layer["down"])
        return w4.w4_residual_norm(out, h, self.norm_out, residual_out=h)[0]

    def prompts(self, x, lens, cache):
        """A pass over prompts of `lens` tokens, x [sum(lens)][hidden] one after the other."""
        ends = torch.tensor([0] + list(lens)).cumsum(0).to(torch.int32).to(x.device)
        cache.kv_len += ends[1:] - ends[:-1]
        return self.forward(x.float().clone(), cache, ends)

    def shared_pass(self, x, n_new, cache):
        """A pass over n_new[b] tokens (int32 [n + 1], on the GPU) of each sequence of a SharedCache, x
        [sum of n_new][hidden] one after the other."""
        return self.forward(x.float().clone(), cache, cache.advance(n_new, x.shape[0]))

    def step(self, x, cache):
        """One token of each sequence, x [n_seqs][hidden]."""
        cache.kv_len += 1
        return self.forward(x.float().clone(), cache)


def main(argv=None):
    p = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    p.add_argument("--layers", type=int, default=4)
    p.add_argument("--prompts", default="700,2000,33", help="tokens of each prompt")
    p.add_argument("--steps", type=int, default=32, help="tokens generated per sequence")
    p.add_argument("--window", type=int, default=0, help="attention window (0: none)")
    p.add_argument("--system", type=int, default=0, help="tokens of a shared system prompt")
    args = p.parse_args(argv)
    lens = [int(n) for n in args.prompts.split(",")]
    if min(lens) < 1 or args.steps < 1 or len(lens) > w4.GEMV_MAX_M:
        p.error("prompts need a token each, --steps one, and the batch at most "
                f"{w4.GEMV_MAX_M} sequences")
    model = Decoder(Shape(layers=args.layers, window=args.window))
    # (+ 4: the steps that warm up and record the graph)
    ends = [n + args.steps + 4 for n in lens]
    x = torch.randn(sum(lens), model.shape.hidden, device="cuda").bfloat16()
    begin, mid, end = (torch.cuda.Event(enable_timing=True) for _ in range(3))
    if args.system > 0:
        size = model.shape.page_size
        pages = sum(-(-(args.system % size + n) // size) for n in ends) + -(-args.system // size)
        cache = SharedCache(model.shape, len(lens), pages, args.system + max(ends), "cuda")

        def tokens(*counts):
            return torch.tensor(counts, dtype=torch.int32, device="cuda")

        model.shared_pass(torch.randn(args.system, model.shape.hidden, device="cuda").bfloat16(),
                          tokens(*[0] * len(lens), args.system), cache)
        for b in range(len(lens)):
            cache.share(b)
        one_each = tokens(*[1] * len(lens), 0)

        def prompts():
            return model.shared_pass(x, tokens(*lens, 0), cache)

        def step(token):
            return model.shared_pass(token, one_each, cache)
    else:
        cache = Cache(model.shape, ends, "cuda")

        def prompts():
            return model.prompts(x, lens, cache)

        def step(token):
            return model.step(token, cache)

        prompts()  # the first pass loads the kernels
        cache.kv_len.zero_()
    begin.record()
    y = prompts()
    mid.record()
    torch.cuda.synchronize()
    print(f"{sum(lens)} prompt tokens in {begin.elapsed_time(mid):.3f} ms", flush=True)

    token = y[torch.tensor(lens).cumsum(0).to(y.device) - 1].clone()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        side.wait_stream(torch.cuda.default_stream())
        token.copy_(step(token))
        side.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            token.copy_(step(token))
    torch.cuda.default_stream().wait_stream(side)
    graph.replay()
    begin.record()
    for _ in range(args.steps):
        graph.replay()
    end.record()
    torch.cuda.synchronize()
    if args.system > 0:
        cache.check()
    ms = begin.elapsed_time(end) / args.steps
    print(f"{len(lens)} sequences, {args.steps} steps, {ms:.3f} ms a step "
          f"({len(lens) * 1e3 / ms:.0f} tokens/s through {args.layers} layers)", flush=True)
    assert torch.isfinite(token.float()).all()


if __name__ == "__main__":
    main()
