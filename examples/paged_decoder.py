"""A decoder over a paged cache: prompts in chunks of any size, then single tokens of all sequences at once.

    python examples/paged_decoder.py [--steps 16] [--cache e4m3]

Every layer is block_norm_forward, linear_forward, qk_rope_forward, kv_cache_store (an E4M3 cache; rows of the
computations' type go to their pages by qk_rope_forward itself), paged_attention_forward, and the products and
block_norm_forward that follow.  The prompts' chunks are ragged batches, some sequences with many tokens, some with one;
the steps of single tokens are one captured HIP graph.  The steps' last tokens, computed again by attention_forward over
rows that kv_cache_load brings back, have to give what the steps gave.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import convolution_conv2d_forward_amd as cc  # noqa: E402


def _ints(v):
    return torch.as_tensor(v, dtype=torch.int32, device="cuda").contiguous()


class PagedDecoder:
    """Layers of x + post(out(attention(rope(qkv(pre(x)))))), then x + post(down(act(up(pre(x))))), and their pages."""

    def __init__(self, layers, width, heads_q, heads_kv, head_dim, hidden, n_pages, page_size, dtype="bf16",
                 cache="e4m3", window=0, sinks=0, softcap=0.0, seed=0):
        t = {"bf16": torch.bfloat16, "f32": torch.float32}[dtype]
        gen = torch.Generator(device="cuda").manual_seed(seed)
        rand = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
        self.t, self.heads_q, self.heads_kv, self.head_dim = t, heads_q, heads_kv, head_dim
        self.params = dict(window=window, softcap=softcap, dtype=dtype)
        self.quantised = cache == "e4m3"
        sizes = {"qkv": ((heads_q + 2 * heads_kv) * head_dim, width), "out": (width, heads_q * head_dim),
                 "up": (hidden, width), "down": (width, hidden)}
        cache_type = torch.float8_e4m3fn if self.quantised else t
        pages = (n_pages, page_size, heads_kv, head_dim)
        self.layers = []
        for _ in range(layers):
            w = {n: (rand(*s) * s[1] ** -0.5).to(t) for n, s in sizes.items()}
            gamma = {n: 1 + 0.1 * rand(width) for n in ("post1", "pre1", "post2", "pre2")}
            w["head"] = 1 + 0.1 * rand(2, head_dim)
            # Zero bytes are zeros of every type; a cache needs no clearing to be right, only to be finite when read.
            got = [torch.zeros(pages, dtype=torch.uint8 if self.quantised else t, device="cuda").view(cache_type)
                   for _ in "kv"]
            got += [torch.full(pages[:3], 127, dtype=torch.uint8, device="cuda") if self.quantised else None for _ in "kv"]
            self.layers.append((w, gamma, got))
        self.linear = {n: cc.linear_desc_create(cc.make_linear_params(
            s[1], s[0], dtype=dtype, act="gelu_tanh" if n == "up" else "none")) for n, s in sizes.items()}
        norm = lambda **kw: cc.block_norm_desc_create(cc.make_block_norm_params(  # noqa: E731
            width, pre_norm="rms", dtype=dtype, **kw))
        self.first, self.block = norm(residual_scale=0.0), norm(post_norm="rms")
        self.rope = cc.qk_rope_desc_create(cc.make_qk_rope_params(heads_q, heads_kv, head_dim, has_norm=True,
                                                                  dtype=dtype))
        self.cache = cc.kv_cache_desc_create(cc.make_kv_cache_params(heads_kv, head_dim, page_size, dtype=dtype,
                                                                     cache_dtype=cache))
        self.attention = cc.paged_attention_desc_create(cc.make_paged_attention_params(
            heads_q, heads_kv, head_dim, page_size, window=window, sinks=sinks, softcap=softcap, dtype=dtype,
            cache_dtype=cache))
        self.workspaces = {}

    def workspace(self, *sizes):
        """Kept for each size of a batch: a captured step's has to outlive it."""
        if sizes not in self.workspaces:
            n = cc.paged_attention_workspace_bytes(self.attention, *sizes)
            self.workspaces[sizes] = torch.empty(max(n, 1), dtype=torch.uint8, device="cuda")
        return self.workspaces[sizes]

    def _read_pages(self, q, offsets, kv_lens, table, got, o):
        cc.paged_attention_forward(self.attention, q, offsets, kv_lens, table, *got, o,
                                   workspace=self.workspace(q.shape[0], *table.shape))

    def _read_rows(self, kv_len):
        """Attention by way of contiguous rows, for the same number of tokens of each sequence."""
        def read(q, offsets, kv_lens, table, got, o):
            batch, row = table.shape[0], (self.heads_kv, self.head_dim)
            k, v = (torch.zeros((batch, kv_len) + row, dtype=self.t, device="cuda") for _ in "kv")
            cc.kv_cache_load(self.cache, table, kv_lens, *got, k, v)
            q, out = (a.view(batch, -1, self.heads_q, self.head_dim) for a in (q, o))
            d = cc.attention_desc_create(cc.make_attention_params(
                self.heads_q, self.heads_kv, self.head_dim, causal=True, q_strides=q.stride()[:3],
                k_strides=k.stride()[:3], v_strides=v.stride()[:3], out_strides=out.stride()[:3], **self.params))
            n = cc.attention_workspace_bytes(d, batch, q.shape[1], kv_len)
            cc.attention_forward(d, q, k, v, out, kv_lens=kv_lens,
                                 workspace=torch.empty(max(n, 1), dtype=torch.uint8, device="cuda"))
        return read

    def __call__(self, x, positions, slots, offsets, kv_lens, table, kv_len=None):
        """x [tokens, width]: rows offsets[b] .. offsets[b + 1] - 1 are the last tokens of sequence b, which has
        kv_lens[b] with them; positions and cache slots of each row.  With kv_len, nothing is stored, and attention
        reads rows brought back from the pages."""
        rows = x.shape[0]
        new = lambda n: torch.empty((rows, n), dtype=self.t, device="cuda")  # noqa: E731
        heads = lambda n: torch.empty((rows, n, self.head_dim), dtype=self.t, device="cuda")  # noqa: E731
        attend = self._read_rows(kv_len) if kv_len else self._read_pages
        there = torch.arange(rows, dtype=torch.int32, device="cuda")
        stream, n = torch.empty_like(x), torch.empty_like(x)
        cc.block_norm_forward(self.first, x, x, None, None, None, self.layers[0][1]["pre1"], None, stream, n)
        for i, (w, gamma, got) in enumerate(self.layers):
            following = self.layers[(i + 1) % len(self.layers)][1]["pre1"]
            qkv, q, o, y = new(w["qkv"].shape[0]), heads(self.heads_q), heads(self.heads_q), torch.empty_like(x)
            cc.linear_forward(self.linear["qkv"], n, w["qkv"], None, None, qkv)
            direct = not self.quantised and not kv_len
            k, v = (a.view(-1, self.heads_kv, self.head_dim) for a in got[:2]) if direct else (
                heads(self.heads_kv), heads(self.heads_kv))
            cc.qk_rope_forward(self.rope, qkv, w["head"][0], w["head"][1], positions, slots if direct else there, q, k, v)
            if self.quantised and not kv_len:
                cc.kv_cache_store(self.cache, k, v, slots, *got)
            attend(q, offsets, kv_lens, table, got, o)
            cc.linear_forward(self.linear["out"], o.view(rows, -1), w["out"], None, None, y)
            cc.block_norm_forward(self.block, y, stream, None, gamma["post1"], None, gamma["pre2"], None, stream, n)
            h = new(w["up"].shape[0])
            cc.linear_forward(self.linear["up"], n, w["up"], None, None, h)
            cc.linear_forward(self.linear["down"], h, w["down"], None, None, y)
            cc.block_norm_forward(self.block, y, stream, None, gamma["post2"], None, following, None, stream, n)
        return stream


def run(lens=(700, 90, 1, 333), chunk=256, steps=6, page_size=16, layers=2, width=512, heads_q=8, heads_kv=2,
        head_dim=64, hidden=1024, dtype="bf16", cache="e4m3", softcap=30.0, window=0, sinks=0):
    """Prompts of `lens` tokens in chunks, then `steps` tokens of each sequence by a captured step.  Returns those
    steps' outputs, the same tokens' by rows brought back from the pages (None with first tokens kept, which
    attention_forward does not do), and the us of a step."""
    batch, top = len(lens), max(lens) + steps
    max_pages = -(-top // page_size)
    n_pages = batch * max_pages + 1
    m = PagedDecoder(layers, width, heads_q, heads_kv, head_dim, hidden, n_pages, page_size, dtype, cache, window, sinks,
                     softcap)
    gen = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn((batch, top, width), generator=gen, device="cuda").to(m.t)
    order = torch.randperm(n_pages, generator=torch.Generator().manual_seed(2))[:batch * max_pages]
    table = order.view(batch, max_pages)
    slot = lambda b, i: int(table[b, i // page_size]) * page_size + i % page_size  # noqa: E731
    pages = _ints(table)

    done = [0] * batch
    while any(d < n for d, n in zip(done, lens)):
        new = [min(chunk, n - d) for d, n in zip(done, lens)]
        at = [[d + j for j in range(c)] for d, c in zip(done, new)]
        rows = torch.cat([x[b, a] for b, a in enumerate(at) if a])
        done = [d + c for d, c in zip(done, new)]
        m(rows, _ints(sum(at, [])), _ints([slot(b, i) for b, a in enumerate(at) for i in a]),
          _ints([0] + torch.tensor(new).cumsum(0).tolist()), _ints(done), pages)

    token = torch.zeros((batch, width), dtype=m.t, device="cuda")
    pos, slots, kv_lens = _ints([0] * batch), _ints([-1] * batch), _ints([0] * batch)
    offsets = _ints(range(batch + 1))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        m(token, pos, slots, offsets, kv_lens, pages)   # makes the workspace; slots of -1 store nothing
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = m(token, pos, slots, offsets, kv_lens, pages)
    events = [torch.cuda.Event(enable_timing=True) for _ in range(2)]
    single = []
    events[0].record()
    for i in range(steps):
        for b in range(batch):
            token[b] = x[b, lens[b] + i]
        pos.copy_(_ints([n + i for n in lens]))
        slots.copy_(_ints([slot(b, n + i) for b, n in enumerate(lens)]))
        kv_lens.copy_(_ints([n + i + 1 for n in lens]))
        graph.replay()
        single.append(out.clone())
    events[1].record()
    torch.cuda.synchronize()
    got, again = torch.stack(single, 1), None
    if not sinks:
        rows = torch.cat([x[b, n:n + steps] for b, n in enumerate(lens)])
        again = m(rows, _ints([n + i for n in lens for i in range(steps)]), None, None,
                  _ints([n + steps for n in lens]), pages, kv_len=top).view(batch, steps, width)
    return got, again, events[0].elapsed_time(events[1]) * 1e3 / steps


def main():
    p = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    p.add_argument("--steps", type=int, default=16)
    p.add_argument("--cache", default="e4m3", choices=("e4m3", "bf16"))
    a = p.parse_args()
    got, again, us = run(steps=a.steps, cache=a.cache)
    off = float((got.float() - again.float()).abs().max())
    print(f"a step of {got.shape[0]} single tokens: {us:.0f} us; by rows brought back from the pages the outputs differ "
          f"by at most {off:.3g} (largest {float(again.abs().max()):.3g})")


if __name__ == "__main__":
    main()
