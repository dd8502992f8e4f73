"""One decoder layer's attention with everything it needs between its quantized
linears: a prompt is run through, branches of it are sampled in parallel, and
the cache is kept tidy.

    python examples/decoder_attention.py [--hidden 4096] [--prompt 700] [--steps 40]

Every step is what a serving loop does for each layer:

    quantize_act -> linear (QKV) -> kv_append -> attn_prefill / attn_decode
                 -> quantize_act -> linear (O)

with the page bookkeeping around it once per step: kv_reserve before new tokens
are stored, kv_fork when a sequence is continued in several ways, kv_trim as the
window moves on, kv_free when a sequence ends, kv_compact when the cache has
holes.  The weights are random; the outputs are checked for what holds whatever
they are: branches of one prompt that are fed the same tokens give the same
outputs, also after the cache has been compacted.  (Bit for bit at these sizes,
where every tile of the attention's work has a workgroup of its own; in a fuller
batch a sequence's sums may be split at other tokens than its twin's.)
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import w4a4_block_scaled_amd as w4  # noqa: E402

FORMAT = "mxfp4"


class Linear:
    """A packed W4A4 linear with random weights."""

    def __init__(self, n, k, gen, device):
        self.n, self.k = n, k
        self.c = torch.exp2(torch.randint(-1, 2, (k,), generator=gen)).float().to(device)
        self.blob = torch.empty(0)
        weight = (torch.randn(n, k, generator=gen) * k ** -0.5).to(torch.bfloat16).to(device)
        codes, scales, _ = w4.quantize_act((weight.float() / self.c).to(torch.bfloat16), None, FORMAT)
        self.blob = w4.pack_weight(codes, scales, None, torch.ones(n, device=device), FORMAT)

    def __call__(self, x):
        codes, scales, t = w4.quantize_act(x, self.c, FORMAT)
        return w4.linear(codes, scales, t, self.blob, FORMAT, self.n, self.k)


class Attention:
    """QKV linear, cache, attention and O linear of one layer."""

    def __init__(self, hidden, q_heads, kv_heads, pages, page, cache_type, gen, device):
        self.dim = hidden // q_heads
        self.q_heads, self.kv_heads = q_heads, kv_heads
        self.qkv = Linear((q_heads + 2 * kv_heads) * self.dim, hidden, gen, device)
        self.o = Linear(hidden, hidden, gen, device)
        shape = (2, pages, page, kv_heads, self.dim)
        self.cache = torch.zeros(shape, dtype=torch.bfloat16, device=device).to(cache_type)
        self.scales = {}
        if cache_type == torch.float8_e4m3fn:
            self.scales = {"k_scale": torch.full((kv_heads,), 0.02, device=device),
                           "v_scale": torch.full((kv_heads,), 0.02, device=device)}

    def __call__(self, x, tables, lens, cu=None, **mask):
        rows = self.qkv(x).view(len(x), -1, self.dim)
        q, k, v = rows.split([self.q_heads, self.kv_heads, self.kv_heads], dim=1)
        w4.kv_append(k, v, *self.cache, tables, lens, cu_seqlens=cu, **self.scales)
        if cu is None:
            y = w4.attn_decode(q, *self.cache, tables, lens, **mask, **self.scales)
        else:
            y = w4.attn_prefill(q, cu, *self.cache, tables, lens, **mask, **self.scales)
        return self.o(y.view(len(x), -1))


def run(hidden=1024, q_heads=8, kv_heads=2, prompt=300, steps=24, branches=3, page=16, window=128, sinks=4,
        cache_type=torch.bfloat16, device="cuda", say=print):
    gen = torch.Generator().manual_seed(1)
    seqs = 2 + branches                                  # two prompts, and the branches of the first
    per_seq = -(-(prompt + steps) // page) + 1
    pages = 2 * per_seq + branches * (steps // page + 3) + 4
    layer = Attention(hidden, q_heads, kv_heads, pages, page, cache_type, gen, device)
    tables = torch.full((seqs, per_seq), -1, dtype=torch.int32, device=device)
    lens = torch.zeros(seqs, dtype=torch.int32, device=device)
    refs = torch.zeros(pages, dtype=torch.int32, device=device)
    lacking = torch.zeros(1, dtype=torch.int32, device=device)

    def ids(*v):
        return torch.tensor(v, dtype=torch.int32, device=device)

    def data(n):
        return torch.randn(n, hidden, generator=gen).to(torch.bfloat16).to(device)

    # both prompts in one ragged call; the other rows have no tokens
    half = prompt // 2
    counts = [prompt, half] + [0] * branches
    cu = torch.tensor([0, *torch.tensor(counts).cumsum(0).tolist()], dtype=torch.int32, device=device)
    lens[:2] = ids(prompt, half)
    w4.kv_reserve(tables, lens, refs, page, lacking=lacking)
    y = layer(data(prompt + half), tables, lens, cu, window=window, sinks=sinks)
    assert lacking.item() == 0 and torch.isfinite(y).all()
    say(f"prompts of {prompt} and {half} tokens: {int((refs > 0).sum())} of {pages} pages in use")

    # the first prompt is continued in several ways: the branches share its whole pages
    children = torch.arange(2, seqs, dtype=torch.int32, device=device)
    w4.kv_fork(layer.cache, tables, lens, refs, torch.zeros_like(children), children, lacking=lacking)
    say(f"{branches} branches: {int((refs > 0).sum())} pages in use, {int((refs > 1).sum())} of them shared")

    compacted = steps // 2
    for step in range(steps):
        lens += 1
        w4.kv_reserve(tables, lens, refs, page, lacking=lacking)
        x = data(2)
        x = torch.cat([x, x[:1].expand(branches, -1)]).contiguous()        # the branches get the first one's token
        y = layer(x, tables, lens, window=window, sinks=sinks)
        assert torch.isfinite(y[0]).all()
        assert torch.equal(y[2:], y[:1].expand(branches, -1)), f"step {step}: branches fed alike differ"
        w4.kv_trim(tables, lens, refs, page, window, sinks)
        if step == compacted:
            w4.kv_free(tables, lens, refs, ids(1))                         # the second prompt has ended
            before = int((refs > 0).sum())
            w4.kv_compact(layer.cache, tables, refs)
            assert int((refs[:before] > 0).sum()) == before
            say(f"step {step}: second prompt ended, {before} pages in use, moved to the front")
    assert lacking.item() == 0
    w4.kv_free(tables, lens, refs)
    assert int(refs.abs().sum()) == 0
    say(f"{steps} steps of {seqs} sequences, all pages free again")


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--hidden", type=int, default=4096)
    ap.add_argument("--prompt", type=int, default=700)
    ap.add_argument("--steps", type=int, default=40)
    ap.add_argument("--e4m3", action="store_true", help="an 8-bit cache")
    a = ap.parse_args()
    run(a.hidden, a.hidden // 128, max(a.hidden // 512, 1), a.prompt, a.steps,
        cache_type=torch.float8_e4m3fn if a.e4m3 else torch.bfloat16)
