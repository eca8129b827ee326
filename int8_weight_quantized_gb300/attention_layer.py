"""One attention layer of a transformer, from the library's operators: a prompt, then tokens one
by one.

    python -m int8_weight_quantized_gb300.attention_layer --tokens 2048 --steps 16 --cache int8

Prompt: INT8 QKV projection, norm and rotation into the paged cache, attention over the prompt,
INT8 output projection with the residual.  Each further token: the same with 4-bit projections
and attention over the cache.  Random weights and activations; prints the time of each part and
how far the last token's attention over the cache is from the same token's over the whole
sequence at once.
"""
import argparse

import torch

import int8_weight_quantized_gb300 as ck


class AttentionLayer:
    """y = x + O(attention(rope(norm(Q, K)), V)), [Q K V] = P x, with INT8 projections for prompts
    and 4-bit ones for single tokens, over a paged cache."""

    def __init__(self, hidden, q_heads, kv_heads, head_dim, max_tokens, batch=1, page_size=32, cache_dtype=torch.bfloat16,
                 window=0, sinks=0, seed=0, device="cuda"):
        g = torch.Generator(device=device)
        g.manual_seed(seed)
        self.q_heads, self.kv_heads, self.head_dim, self.hidden = q_heads, kv_heads, head_dim, hidden
        self.window, self.sinks, self.page_size = window, sinks, page_size
        width = (q_heads + 2 * kv_heads) * head_dim

        def weight(n, k):
            return torch.randn((n, k), generator=g, device=device) * k ** -0.5

        self.projections = {}
        for name, (n, k) in (("qkv", (width, hidden)), ("out", (hidden, q_heads * head_dim))):
            W = weight(n, k)
            w_scale = W.abs().amax(1) / 127
            w8 = (W / w_scale[:, None]).round().clamp(-127, 127).to(torch.int8)
            self.projections[name] = (w8, w_scale, *ck.ck_int4_prepare_weight(W))
        self.q_weight = (1 + 0.1 * torch.randn(head_dim, generator=g, device=device)).to(torch.bfloat16)
        self.k_weight = (1 + 0.1 * torch.randn(head_dim, generator=g, device=device)).to(torch.bfloat16)
        self.table = ck.rope_table(max_tokens, head_dim, device=device)
        blocks = -(-max_tokens // page_size)
        self.cache = ck.KVCache.empty(batch * blocks, page_size, kv_heads, head_dim, dtype=cache_dtype, device=device)
        # pages of the sequences mixed, as a serving loop's allocator leaves them
        self.block_table = torch.randperm(batch * blocks, generator=g, device=device).to(torch.int32).view(batch, blocks)

    def slots(self, sequence, positions):
        """Cache slots of positions of sequences (int64 tensors of one shape)."""
        page = self.block_table[sequence, positions // self.page_size].long()
        return page * self.page_size + positions % self.page_size

    def rotate(self, qkv, sequence, positions, return_k):
        return ck.ck_qk_norm_rope(qkv, positions.to(torch.int32), self.table, self.q_heads, self.kv_heads,
                                  q_weight=self.q_weight, k_weight=self.k_weight, cache=self.cache,
                                  slots=self.slots(sequence, positions), return_k=return_k)

    def prompt(self, x, lengths):
        """x [tokens, hidden] bf16, the prompts of `lengths` one after the other -> y [tokens, hidden]."""
        w8, w_scale, _, _ = self.projections["qkv"]
        qkv = ck.ck_int8_linear(x, w8, w_scale)
        n = torch.tensor(lengths, device=x.device)
        cu = torch.cat([n.new_zeros(1), n.cumsum(0)])
        sequence = torch.repeat_interleave(torch.arange(len(lengths), device=x.device), n)
        positions = torch.arange(x.shape[0], device=x.device) - cu[sequence]
        q, k = self.rotate(qkv, sequence, positions, True)
        v = qkv.view(x.shape[0], -1, self.head_dim)[:, self.q_heads + self.kv_heads:]
        a = ck.ck_attention(q, k, v, cu.to(torch.int32), window=self.window, sinks=self.sinks)
        w8, w_scale, _, _ = self.projections["out"]
        return ck.ck_int8_linear(a.view(x.shape[0], -1), w8, w_scale, residual=x)

    def step(self, x, lengths):
        """x [batch, hidden] bf16, one new token of each sequence; lengths [batch] (int64) cached
        tokens before it -> (y [batch, hidden], the attention's output)."""
        _, _, w4, scale = self.projections["qkv"]
        qkv = ck.ck_int4_linear(x, w4, scale)
        q, _ = self.rotate(qkv, torch.arange(x.shape[0], device=x.device), lengths, False)
        a = ck.ck_paged_attention(q, self.cache, self.block_table, (lengths + 1).to(torch.int32), window=self.window,
                                  sinks=self.sinks)
        _, _, w4, scale = self.projections["out"]
        return ck.ck_int4_linear(a.view(x.shape[0], -1), w4, scale, residual=x), a


def run(tokens, steps, cache_dtype=torch.bfloat16, window=0, sinks=0, hidden=2048, q_heads=16, kv_heads=4, head_dim=128,
        seed=0):
    """A prompt and `steps` tokens; returns (prompt ms, ms a step, relative difference of the last
    step's attention from the same over the whole sequence at once)."""
    layer = AttentionLayer(hidden, q_heads, kv_heads, head_dim, tokens + steps, cache_dtype=cache_dtype, window=window,
                           sinks=sinks, seed=seed)
    g = torch.Generator(device="cuda")
    g.manual_seed(seed + 1)
    x = torch.randn((tokens + steps, hidden), generator=g, device="cuda").to(torch.bfloat16)
    lengths = [torch.full((1,), tokens + i, device="cuda") for i in range(steps)]
    layer.prompt(x[:tokens], [tokens])  # warm-up
    ev = [torch.cuda.Event(enable_timing=True) for _ in range(3)]
    ev[0].record()
    layer.prompt(x[:tokens], [tokens])
    ev[1].record()
    for i in range(steps):
        _, a = layer.step(x[tokens + i:tokens + i + 1], lengths[i])
    ev[2].record()
    torch.cuda.synchronize()
    # the last token again: its keys and those of the steps from the 4-bit projection as well
    w8, w_scale, w4, scale = layer.projections["qkv"]
    qkv = torch.cat([ck.ck_int8_linear(x[:tokens], w8, w_scale)] +
                    [ck.ck_int4_linear(x[tokens + i:tokens + i + 1], w4, scale) for i in range(steps)])
    positions = torch.arange(tokens + steps, device="cuda", dtype=torch.int32)
    q, k = ck.ck_qk_norm_rope(qkv, positions, layer.table, q_heads, kv_heads, q_weight=layer.q_weight,
                              k_weight=layer.k_weight)
    v = qkv.view(tokens + steps, -1, head_dim)[:, q_heads + kv_heads:]
    cu = torch.tensor([0, tokens + steps], device="cuda", dtype=torch.int32)
    whole = ck.ck_attention(q, k, v, cu, window=window, sinks=sinks)[-1].float()
    off = ((a[0].float() - whole).norm() / whole.norm()).item()
    return ev[0].elapsed_time(ev[1]), ev[1].elapsed_time(ev[2]) / steps, off


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--tokens", type=int, default=2048)
    ap.add_argument("--steps", type=int, default=16)
    ap.add_argument("--cache", choices=["bf16", "int8"], default="bf16")
    ap.add_argument("--window", type=int, default=0)
    ap.add_argument("--sinks", type=int, default=0)
    args = ap.parse_args(argv)
    if args.tokens < 1 or args.steps < 1:
        ap.error("--tokens and --steps must be at least 1")
    dtype = torch.int8 if args.cache == "int8" else torch.bfloat16
    prompt_ms, step_ms, off = run(args.tokens, args.steps, dtype, args.window, args.sinks)
    print("prompt of %d tokens %.3f ms, %.3f ms a token after it; the last token's attention over the %s cache is "
          "%.2g off that over the whole sequence" % (args.tokens, prompt_ms, step_ms, args.cache, off))


if __name__ == "__main__":
    main()
