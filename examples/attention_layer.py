"""One attention layer from the library's operators: a prompt, then single tokens over its cache.

    python examples/attention_layer.py [--tokens 2000] [--steps 8]

Every product is linear_forward, the queries' and keys' norms and rotation with the stores to the cache are one
qk_rope_forward, and attention_forward reads the cache.  The descriptors, the cache and the workspaces are made once;
a step of single tokens is captured into a HIP graph.  The last rows of the prompt, fed again as single tokens, have to
give what they gave within the prompt.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import convolution_conv2d_forward_amd as cc  # noqa: E402


class AttentionLayer:
    """x + out(attention(rope(qkv(x)))), then y + down(act(up(y))): weights of one layer, and a cache for `batch`
    sequences of up to `max_len` tokens."""

    def __init__(self, width, heads_q, heads_kv, head_dim, hidden, batch, max_len, dtype="bf16", softcap=0.0, window=0,
                 seed=0):
        t = {"bf16": torch.bfloat16, "f32": torch.float32}[dtype]
        gen = torch.Generator(device="cuda").manual_seed(seed)
        rand = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
        self.t, self.batch, self.max_len = t, batch, max_len
        self.heads_q, self.heads_kv, self.head_dim = heads_q, heads_kv, head_dim
        n_qkv, n_out = (heads_q + 2 * heads_kv) * head_dim, heads_q * head_dim
        sizes = {"qkv": (n_qkv, width), "out": (width, n_out), "up": (hidden, width), "down": (width, hidden)}
        self.w = {n: (rand(*s) * s[1] ** -0.5).to(t) for n, s in sizes.items()}
        self.b = {n: 0.1 * rand(s[0]) for n, s in sizes.items()}
        self.gamma = 1 + 0.1 * rand(2, head_dim)
        lin = lambda n, **kw: cc.linear_desc_create(cc.make_linear_params(  # noqa: E731
            sizes[n][1], sizes[n][0], has_bias=True, dtype=dtype, **kw))
        self.linear = {"qkv": lin("qkv"), "out": lin("out", has_residual=True), "up": lin("up", act="gelu_tanh"),
                       "down": lin("down", has_residual=True)}
        self.rope = cc.qk_rope_desc_create(cc.make_qk_rope_params(heads_q, heads_kv, head_dim, has_norm=True,
                                                                  dtype=dtype))
        # Keys and values of sequence b, token i: row b * max_len + i.
        self.k, self.v = (torch.zeros((batch * max_len, heads_kv, head_dim), dtype=t, device="cuda") for _ in "kv")
        cache = self.k.view(batch, max_len, heads_kv, head_dim)
        self.attention, self.params = {}, dict(causal=True, softcap=softcap, window=window, dtype=dtype,
                                               k_strides=cache.stride()[:3], v_strides=cache.stride()[:3])

    def _attention(self, q_len):
        """Descriptor and workspace for `q_len` new tokens of each sequence."""
        if q_len not in self.attention:
            s = (q_len * self.heads_q * self.head_dim, self.heads_q * self.head_dim, self.head_dim)
            d = cc.attention_desc_create(cc.make_attention_params(self.heads_q, self.heads_kv, self.head_dim,
                                                                  q_strides=s, out_strides=s, **self.params))
            n = cc.attention_workspace_bytes(d, self.batch, q_len, self.max_len)
            self.attention[q_len] = d, torch.empty(max(n, 1), dtype=torch.uint8, device="cuda")
        return self.attention[q_len]

    def __call__(self, x, positions, slots, kv_lens):
        """x [batch * q_len, width]: the last q_len tokens of each sequence, whose lengths with them are kv_lens;
        positions and slots (cache rows) of each token."""
        rows = x.shape[0]
        new = lambda n: torch.empty((rows, n), dtype=self.t, device="cuda")  # noqa: E731
        q_len, n_out = rows // self.batch, self.heads_q * self.head_dim
        qkv, q, o, y, h, z = (new(n) for n in (self.w["qkv"].shape[0], n_out, n_out, x.shape[1],
                                               self.w["up"].shape[0], x.shape[1]))
        cc.linear_forward(self.linear["qkv"], x, self.w["qkv"], self.b["qkv"], None, qkv)
        cc.qk_rope_forward(self.rope, qkv, self.gamma[0], self.gamma[1], positions, slots,
                           q.view(rows, self.heads_q, self.head_dim), self.k, self.v)
        desc, workspace = self._attention(q_len)
        heads = lambda a: a.view(self.batch, q_len, self.heads_q, self.head_dim)  # noqa: E731
        cache = lambda a: a.view(self.batch, self.max_len, self.heads_kv, self.head_dim)  # noqa: E731
        cc.attention_forward(desc, heads(q), cache(self.k), cache(self.v), heads(o), kv_lens=kv_lens,
                             workspace=workspace)
        cc.linear_forward(self.linear["out"], o, self.w["out"], self.b["out"], x, y)
        cc.linear_forward(self.linear["up"], y, self.w["up"], self.b["up"], None, h)
        cc.linear_forward(self.linear["down"], h, self.w["down"], self.b["down"], y, z)
        return z


def run(tokens=2000, steps=8, batch=2, width=1024, heads_q=8, heads_kv=2, head_dim=128, hidden=4096, dtype="bf16",
        softcap=50.0):
    """Prompt of `tokens` tokens, then its last `steps` tokens again one by one through a captured step.  Returns the
    prompt's outputs of those tokens, the single steps' outputs, and the times in us."""
    layer = AttentionLayer(width, heads_q, heads_kv, head_dim, hidden, batch, tokens + 16, dtype, softcap)
    gen = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn((batch, tokens, width), generator=gen, device="cuda").to(layer.t)
    ints = lambda v: v.to(torch.int32).contiguous()  # noqa: E731
    at = torch.arange(tokens, device="cuda")
    first = torch.arange(batch, device="cuda")[:, None] * layer.max_len
    prompt = lambda: layer(x.view(-1, width), ints(at.repeat(batch)), ints((first + at).view(-1)),  # noqa: E731
                           torch.full((batch,), tokens, dtype=torch.int32, device="cuda"))
    whole = prompt().view(batch, tokens, width)
    events = [torch.cuda.Event(enable_timing=True) for _ in range(4)]
    events[0].record()
    prompt()
    events[1].record()

    token = torch.empty((batch, width), dtype=layer.t, device="cuda")
    pos, slot, lens = (torch.full((batch,), v, dtype=torch.int32, device="cuda") for v in (0, -1, 0))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        # Makes the descriptor, the workspace and the allocator's buffers; slots of -1 store nothing.
        layer(token.zero_(), pos, slot, lens)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = layer(token, pos, slot, lens)
    single = []
    events[2].record()
    for i in range(tokens - steps, tokens):
        token.copy_(x[:, i])
        pos.fill_(i)
        slot.copy_(first.view(-1) + i)
        lens.fill_(i + 1)
        graph.replay()
        single.append(out.clone())
    events[3].record()
    torch.cuda.synchronize()
    return (whole[:, tokens - steps:], torch.stack(single, 1), events[0].elapsed_time(events[1]) * 1e3,
            events[2].elapsed_time(events[3]) * 1e3 / steps)


def main():
    p = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    p.add_argument("--tokens", type=int, default=2000)
    p.add_argument("--steps", type=int, default=8)
    a = p.parse_args()
    want, got, prompt_us, token_us = run(a.tokens, a.steps)
    off = float((got.float() - want.float()).abs().max())
    print(f"prompt of 2 x {a.tokens} tokens: {prompt_us:.0f} us; a step of single tokens: {token_us:.0f} us; "
          f"the steps differ from the prompt by at most {off:.3g} (largest output {float(want.abs().max()):.3g})")


if __name__ == "__main__":
    main()
