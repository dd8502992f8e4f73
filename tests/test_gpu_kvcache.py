"""The paged cache's own operators against the oracle: storing new tokens, and
the page bookkeeping (reserve, copy, fork, free, trim, compact) on states made
at random, with shared pages, holes, missing entries and too few pages."""
import numpy as np
import pytest
import torch

import w4a4_block_scaled_amd as w4
from gpu_common import device, say
from kv_common import TYPES, as_f64, ints, on_device, table_of, values
from oracle import attention as A
from test_gpu_attn_decode import ORDERS

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------ append --

@pytest.mark.parametrize("kind,high,order", [("bf16", "bf16", "page token head"), ("fp16", "fp16", "page head token"),
                                             ("fp8", "bf16", "page token head"), ("fp8", "fp16", "head page token")])
@pytest.mark.parametrize("past,new,page,dim", [([0, 5, 100], [1, 1, 1], 16, 128), ([0, 33, 7, 0], [70, 0, 9, 1], 11, 64),
                                               ([3], [1300], 16, 64), ([1, 0], [40, 2], 1, 256)])
def test_append_matches_the_oracle(kind, high, order, past, new, page, dim):
    say(f"[append] {kind} from {high}, {order}, past {past} new {new} page {page} dim {dim}")
    dev, kv = device(), 3
    rng, gen = np.random.default_rng(dim), torch.Generator().manual_seed(dim)
    lens = [a + b for a, b in zip(past, new)]
    pages = sum(-(-n // page) for n in lens) + 2
    tables = table_of(lens, page, pages, max(-(-n // page) for n in lens) + 1, rng)
    cu = np.concatenate([[0], np.cumsum(new)])
    rows = values((int(cu[-1]), 4 + 2 * kv, dim), high, gen) * 30
    caches = [values((pages, page, kv, dim), kind, gen) for _ in range(2)]
    scales = [torch.rand(kv, generator=gen) * 0.2 + 0.05 if kind == "fp8" else None for _ in range(2)]
    wide = rows.to(dev)
    parts = wide[:, 4:4 + kv], wide[:, 4 + kv:]
    got = [on_device(c.view(torch.uint8), ORDERS[order], dev).view(c.dtype) if kind == "fp8" else
           on_device(c, ORDERS[order], dev) for c in caches]
    every = all(n == 1 for n in new)
    for cu_arg in ([ints(cu, dev), None] if every else [ints(cu, dev)]):
        w4.kv_append(*parts, *got, ints(tables, dev), ints(lens, dev), cu_seqlens=cu_arg,
                     k_scale=None if scales[0] is None else scales[0].to(dev),
                     v_scale=None if scales[1] is None else scales[1].to(dev))
        for i in range(2):
            want = as_f64(caches[i])
            A.append(want, as_f64(rows[:, 4 + i * kv:4 + (i + 1) * kv]), tables, lens, cu,
                     None if scales[i] is None else scales[i].numpy())
            assert np.array_equal(as_f64(got[i]), want), f"{'KV'[i]}"


def test_append_e4m3_every_rounding():
    """All finite FP16 values through a scale of 1 and one that is no power of
    two: nearest E4M3 value, ties to even, saturation, signed zeros; NaN stays."""
    say("[append] every FP16 value")
    dev = device()
    bits = torch.arange(65536, dtype=torch.int32).to(torch.int16)
    x = bits.view(torch.float16).reshape(512, 2, 64)
    k = torch.zeros(32, 16, 2, 64, dtype=torch.float8_e4m3fn, device=dev)
    v = torch.zeros_like(k)
    scale = torch.tensor([1.0, 0.37])
    table = ints([np.arange(32)], dev)
    w4.kv_append(x.to(dev), x.to(dev), k, v, table, ints([512], dev), cu_seqlens=ints([0, 512], dev),
                 k_scale=scale.to(dev))
    f = x.float()
    for got, s in ((k, scale[:, None]), (v, torch.ones(2, 1))):
        quotient = (f / s)
        want = A.e4m3_value(quotient.double().numpy())
        g = as_f64(got).reshape(512, 2, 64)
        assert np.array_equal(g, want, equal_nan=True)
        zero = want == 0
        assert np.array_equal(np.signbit(g[zero]), np.signbit(quotient.numpy()[zero]))


def test_append_skips_rows_without_a_place():
    """Negative positions, missing pages and lengths beyond the table are left
    out; everything else in the cache stays as it was."""
    say("[append] rows without a place")
    dev = device()
    gen = torch.Generator().manual_seed(1)
    k = values((6, 16, 2, 64), "bf16", gen)
    v = values((6, 16, 2, 64), "bf16", gen)
    new = values((5, 2, 64), "bf16", gen)
    tables = np.array([[0, 1], [2, -1], [6, 3], [4, 5], [-2 ** 31, 1]], np.int32)
    lens = np.array([0, 20, 3, 2 ** 31 - 1, 2])
    kd, vd = k.to(dev), v.to(dev)
    w4.kv_append(new.to(dev), new.to(dev), kd, vd, ints(tables, dev), ints(lens, dev))
    assert torch.equal(kd.cpu(), k) and torch.equal(vd.cpu(), v)
    lens = np.array([17, 16, 33, 32, 18])
    w4.kv_append(new.to(dev), new.to(dev), kd, vd, ints(tables, dev), ints(lens, dev))
    want = as_f64(k)
    A.append(want, as_f64(new), tables, lens, np.arange(6))
    assert np.array_equal(as_f64(kd), want)


# ------------------------------------------------------------------- pages --

def random_state(seed, seqs, width, page, pages, fill=0.7):
    """Sequences of random lengths, some sharing their first pages."""
    rng = np.random.default_rng(seed)
    tables = np.full((seqs, width), -1, np.int32)
    lens, refs = np.zeros(seqs, np.int32), np.zeros(pages, np.int32)
    free = list(rng.permutation(pages)[:int(pages * fill)])
    for s in range(seqs):
        n = int(rng.integers(0, width * page + 1))
        held = -(-n // page)
        shared = 0
        if s and rng.random() < 0.4:
            p = int(rng.integers(0, s))
            shared = min(int(lens[p]) // page, held)
            tables[s, :shared] = tables[p, :shared]
        if held - shared > len(free):
            held = shared + len(free)
            n = min(n, held * page)
        for j in range(shared, held):
            tables[s, j] = free.pop()
        lens[s] = n
        np.add.at(refs, tables[s, :held], 1)
    return tables, lens, refs, rng


class State:
    """The same state on the device and in the oracle."""

    def __init__(self, seed, seqs, width, page, pages, layers=2, heads=2, dim=64, **more):
        tables, lens, refs, self.rng = random_state(seed, seqs, width, page, pages, **more)
        dev = device()
        data = torch.randn(layers, 2, pages, page, heads, dim, generator=torch.Generator().manual_seed(seed)).to(torch.bfloat16)
        self.pool = data.to(dev)
        self.tables, self.lens, self.refs = (ints(x, dev) for x in (tables, lens, refs))
        self.o = A.Pages(tables, lens, refs, page, as_f64(data).reshape(layers, 2, pages, -1))
        self.lacking = ints([99], dev)
        self.page, self.dev = page, dev

    def same(self, lacking=None):
        torch.cuda.synchronize()
        for name in ("tables", "lens", "refs"):
            got, want = getattr(self, name).cpu().numpy(), getattr(self.o, name)
            assert np.array_equal(got, want), f"{name}: {np.argwhere(got != want)[:4].tolist()}"
        got = as_f64(self.pool)
        assert np.array_equal(got.reshape(self.o.data.shape), self.o.data), "pages"
        if lacking is not None:
            assert self.lacking.item() == lacking


@pytest.mark.parametrize("seed,seqs,width,page,pages", [(1, 5, 7, 16, 60), (2, 1, 3, 1, 10), (3, 40, 9, 8, 400),
                                                        (4, 1500, 3, 4, 4000), (5, 7, 300, 2, 1500)])
def test_reserve(seed, seqs, width, page, pages):
    say(f"[reserve] {seqs} sequences, {width} x {page}, {pages} pages")
    st = State(seed, seqs, width, page, pages, layers=1)
    for _ in range(3):
        grow = st.rng.integers(0, 3 * page + 1, seqs)
        st.o.lens = np.minimum(st.o.lens + grow, width * page).astype(np.int32)
        st.lens.copy_(ints(st.o.lens, st.dev))
        st.o.reserve()
        w4.kv_reserve(st.tables, st.lens, st.refs, page, lacking=st.lacking)
        st.same(st.o.lacking)


def test_reserve_too_few_pages_and_lengths_beyond_the_table():
    say("[reserve] too few pages")
    st = State(6, 6, 5, 16, 12, layers=1)
    st.o.lens[:] = [80, 80, 3, 200, -4, 80]
    st.lens.copy_(ints(st.o.lens, st.dev))
    st.o.reserve()
    assert st.o.lacking > 0
    w4.kv_reserve(st.tables, st.lens, st.refs, 16, lacking=st.lacking)
    st.same(st.o.lacking)


def test_reserve_after_trim_keeps_the_gap():
    """Entries that were let go before the window are not filled again."""
    say("[reserve] after trim")
    st = State(7, 4, 12, 8, 60, layers=1)
    for step in range(4):
        st.o.trim(range(4), 20, 3)
        w4.kv_trim(st.tables, st.lens, st.refs, 8, 20, 3)
        st.same()
        st.o.lens = np.minimum(st.o.lens + 9, 96).astype(np.int32)
        st.lens.copy_(ints(st.o.lens, st.dev))
        st.o.reserve()
        w4.kv_reserve(st.tables, st.lens, st.refs, 8, lacking=st.lacking)
        st.same(st.o.lacking)


@pytest.mark.parametrize("seed,seqs,width,page,pages,n", [(11, 6, 5, 16, 80, 3), (12, 30, 8, 5, 400, 20),
                                                          (13, 3, 4, 1, 30, 1), (14, 2600, 2, 8, 6000, 1200)])
def test_fork(seed, seqs, width, page, pages, n):
    say(f"[fork] {n} of {seqs} sequences, {width} x {page}, {pages} pages")
    st = State(seed, seqs, width, page, pages, fill=0.5)
    ids = st.rng.permutation(seqs)
    children, rest = ids[:n], ids[n:]
    parents = st.rng.choice(rest, n)
    st.o.free(children)
    w4.kv_free(st.tables, st.lens, st.refs, ints(children, st.dev))
    st.same()
    st.o.fork(parents, children)
    w4.kv_fork(st.pool, st.tables, st.lens, st.refs, ints(parents, st.dev), ints(children, st.dev), lacking=st.lacking)
    st.same(st.o.lacking)


def test_fork_too_few_pages_and_invalid_pairs():
    say("[fork] too few pages, invalid pairs")
    st = State(15, 8, 4, 16, 30, fill=0.5)
    st.o.lens[:2] = [20, 40]
    st.lens.copy_(ints(st.o.lens, st.dev))
    st.o.reserve()
    w4.kv_reserve(st.tables, st.lens, st.refs, 16)
    keep = np.flatnonzero(st.o.refs == 0)[2:]      # two pages are free
    st.o.refs[keep] = 1
    st.refs[ints(keep, st.dev).long()] = 1
    children = [4, 5, 6, 7]
    st.o.free(children)
    w4.kv_free(st.tables, st.lens, st.refs, ints(children, st.dev))
    free = np.flatnonzero(st.o.refs == 0)[2:]
    st.o.refs[free] = 1
    st.refs[ints(free, st.dev).long()] = 1
    parents = [0, 1, 0, 1, 8, 0, 2]
    children = [4, 5, 6, 7, 3, -1, 2]
    st.o.fork(parents, children)
    assert st.o.lacking == 2
    w4.kv_fork(st.pool, st.tables, st.lens, st.refs, ints(parents, st.dev), ints(children, st.dev), lacking=st.lacking)
    st.same(st.o.lacking)


def test_free_listed_twice_and_outside():
    say("[free]")
    st = State(16, 9, 6, 8, 90, layers=1)
    ids = [3, 5, 3, -1, 9, 5, 0]
    st.o.free([3, 5, 0])
    w4.kv_free(st.tables, st.lens, st.refs, ints(ids, st.dev))
    st.same()
    st.o.free(range(9))
    w4.kv_free(st.tables, st.lens, st.refs)
    st.same()
    assert st.refs.abs().sum().item() == 0


@pytest.mark.parametrize("window,sinks", [(1, 0), (8, 0), (9, 4), (50, 17), (1000, 2), (1, 2 ** 31 - 1), (2 ** 31 - 1, 0)])
def test_trim(window, sinks):
    say(f"[trim] window {window} sinks {sinks}")
    st = State(17, 12, 10, 8, 200, layers=1)
    st.o.trim([1, 4, 7], window, sinks)
    w4.kv_trim(st.tables, st.lens, st.refs, 8, window, sinks, seqs=ints([1, 4, 7, 4, 99], st.dev))
    st.same()
    st.o.trim(range(12), window, sinks)
    w4.kv_trim(st.tables, st.lens, st.refs, 8, window, sinks)
    st.same()


@pytest.mark.parametrize("seed,seqs,width,page,pages", [(21, 6, 5, 16, 70), (22, 50, 6, 3, 900), (23, 2, 2, 1, 3),
                                                        (24, 700, 5, 2, 20000)])
def test_compact(seed, seqs, width, page, pages):
    say(f"[compact] {seqs} sequences, {width} x {page}, {pages} pages")
    st = State(seed, seqs, width, page, pages)
    gone = st.rng.permutation(seqs)[: seqs // 3]
    st.o.free(gone)
    w4.kv_free(st.tables, st.lens, st.refs, ints(gone, st.dev))
    for _ in range(2):              # the second time there is nothing to move
        want = st.o.compact()
        remap = w4.kv_compact(st.pool, st.tables, st.refs)
        st.same()
        assert np.array_equal(remap.cpu().numpy(), want)
    live = int((st.o.refs != 0).sum())
    assert np.all(st.o.refs[:live] > 0)


def test_compact_all_free_all_used_and_stray_entries():
    say("[compact] edges")
    st = State(25, 3, 4, 8, 20)
    st.o.free(range(3))
    w4.kv_free(st.tables, st.lens, st.refs)
    st.tables[0, 1] = 7             # a free page
    st.tables[1, 2] = 20            # outside
    st.tables[2, 0] = -5
    st.o.tables[0, 1], st.o.tables[1, 2], st.o.tables[2, 0] = 7, 20, -5
    want = st.o.compact()
    remap = w4.kv_compact(st.pool, st.tables, st.refs)
    st.same()
    assert np.array_equal(remap.cpu().numpy(), want) and torch.all(remap == -1)
    st.refs.fill_(1)
    st.o.refs[:] = 1
    st.o.compact()
    remap = w4.kv_compact(st.pool, st.tables, st.refs)
    st.same()
    assert torch.equal(remap.cpu(), torch.arange(20, dtype=torch.int32))


@pytest.mark.parametrize("shape,layers", [((40, 16, 2, 64), 3), ((40, 7, 3, 64), 1), ((33, 1, 1, 64), 150)])
def test_copy_pages(shape, layers):
    """Lists of caches of any dense order; pairs outside are skipped.  150
    layers take more than one launch."""
    say(f"[copy] {layers} x {shape}")
    dev = device()
    gen = torch.Generator().manual_seed(1)
    caches = [values(shape, "bf16", gen) for _ in range(layers)]
    got = [on_device(c, (0, 2, 1), dev) for c in caches]
    order = np.random.default_rng(2).permutation(shape[0])
    src, dst = [*order[:9], -1, 3, 2 ** 31 - 1], [*order[9:18], 4, shape[0], 0]
    w4.kv_copy_pages(got, ints(src, dev), ints(dst, dev))
    for c, g in zip(caches, got):
        want = c.clone()
        want[order[9:18]] = c[order[:9]]
        assert torch.equal(g.cpu(), want)


def test_copy_pages_odd_bytes_and_large_offsets():
    say("[copy] E4M3 pages, a pool past 4 GiB")
    dev = device()
    pool = torch.empty(2, 70000, 8, 4, 128, dtype=torch.float8_e4m3fn, device=dev).view(torch.uint8)   # 573 MB
    src, dst = [1, 69990], [69999, 2]
    pool[:, src[0]], pool[:, src[1]] = 5, 9
    w4.kv_copy_pages(pool.view(torch.float8_e4m3fn), ints(src, dev), ints(dst, dev))
    assert torch.all(pool[:, 69999] == 5) and torch.all(pool[:, 2] == 9)
    del pool
    pool = torch.empty(70000, 64, 8, 64, dtype=torch.bfloat16, device=dev)      # 4.6 GB
    pool[69998] = 3.0
    pool[0] = 4.0
    w4.kv_copy_pages([pool], ints([69998, 0], dev), ints([5, 69999], dev))
    assert torch.all(pool[5] == 3) and torch.all(pool[69999] == 4)


# -------------------------------------------------------------------- graph --

def test_a_decoding_step_in_a_graph():
    """reserve, append and attention of a step captured once and replayed, the
    lengths counted up by the graph: every replay equals the eager calls."""
    say("[graph] a decoding step")
    dev = device()
    kv, group, dim, page, seqs = 2, 4, 128, 16, 5
    gen = torch.Generator().manual_seed(3)
    start = [0, 15, 30, 100, 47]

    def fresh():
        pages = 80
        return {"k": torch.zeros(pages, page, kv, dim, dtype=torch.bfloat16, device=dev),
                "v": torch.zeros(pages, page, kv, dim, dtype=torch.bfloat16, device=dev),
                "tables": torch.full((seqs, 12), -1, dtype=torch.int32, device=dev), "lens": ints(start, dev),
                "refs": torch.zeros(pages, dtype=torch.int32, device=dev)}

    rows = values((8, seqs, (group + 2) * kv, dim), "bf16", gen).to(dev)

    def step(s, x, out, ws):
        s["lens"] += 1
        w4.kv_reserve(s["tables"], s["lens"], s["refs"], page)
        q, k, v = x.split([group * kv, kv, kv], dim=1)
        w4.kv_append(k, v, s["k"], s["v"], s["tables"], s["lens"])
        return w4.attn_decode(q, s["k"], s["v"], s["tables"], s["lens"], window=64, sinks=4, out=out, workspace=ws)

    eager = fresh()
    out = torch.empty(seqs, group * kv, dim, dtype=torch.bfloat16, device=dev)
    wants = [step(eager, rows[i], torch.empty_like(out), None).clone() for i in range(8)]
    s, x = fresh(), rows[0].clone()
    ws = torch.empty(16 << 20, dtype=torch.uint8, device=dev)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(fresh(), x, out, ws)                      # warm-up
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(s, x, out, ws)
    for name, t in fresh().items():
        s[name].copy_(t)
    for i in range(8):
        x.copy_(rows[i])
        out.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, wants[i]), f"replay {i}"
        if i % 3 == 0:
            step(fresh(), rows[i], torch.empty_like(out), None)      # other work between the replays
    for name in s:
        assert torch.equal(s[name], eager[name]), name
