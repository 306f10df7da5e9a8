"""The pages of a cache on the GPU against the plain pool (kv8_reference.Pool):
tables, lengths, counts, statuses and bytes are equal after every call."""
import numpy as np
import pytest
import torch

import kv8_reference as ref
from sparse_long_context_03_b200 import dsa

pytestmark = pytest.mark.gpu
DEV = "cuda"


def i32(x):
    return torch.tensor(np.asarray(x, np.int32), device=DEV)


class Both:
    """A plain pool and one on the GPU, called alike and compared after each call."""

    def __init__(self, P, slots, max_pages, shapes, seed):
        rng = np.random.default_rng(seed)
        self.bufs = [rng.integers(0, 256, (P,) + s).astype(np.uint8) for s in shapes]
        self.pool = ref.Pool(P, slots, max_pages, [b.copy() for b in self.bufs])
        self.g = [torch.from_numpy(b).to(DEV) for b in self.bufs]
        self.state = [i32(x) for x in (self.pool.table, self.pool.lens, self.pool.refs)]

    def same(self, status=None, want=None):
        torch.cuda.synchronize()
        for name, a, b in zip(("table", "lens", "refs"), self.state, (self.pool.table, self.pool.lens, self.pool.refs)):
            assert np.array_equal(a.cpu().numpy(), b), name
        if status is not None:
            assert np.array_equal(status.cpu().numpy(), want), "status"
        for i, (a, b) in enumerate(zip(self.g, self.pool.bufs)):
            assert np.array_equal(a.cpu().numpy(), b), f"buffer {i}"

    def extend(self, slots, lens):
        st = torch.full((len(slots),), 99, dtype=torch.int32, device=DEV)
        dsa.pages_extend(i32(slots), i32(lens), *self.state, st)
        self.same(st, want := self.pool.extend(slots, lens))
        return want

    def fork(self, parents, children):
        st = torch.full((len(parents),), 99, dtype=torch.int32, device=DEV)
        dsa.pages_fork(self.g, i32(parents), i32(children), *self.state, st)
        self.same(st, want := self.pool.fork(parents, children))
        return want

    def free(self, slots):
        dsa.pages_free(i32(slots), *self.state)
        self.pool.free(slots)
        self.same()

    def compact(self, in_place=True):
        P = len(self.pool.refs)
        pmap, used = torch.empty(P, dtype=torch.int32, device=DEV), i32([0])
        ws = torch.empty(dsa.pages_compact_workspace_size(P), dtype=torch.uint8, device=DEV)
        kw = {}
        if not in_place:
            before = [t.clone() for t in self.state]
            kw = dict(block_table_out=torch.full_like(self.state[0], 55), refcount_out=torch.full_like(self.state[2], 55))
        dsa.pages_compact(self.g, *self.state, pmap, used, ws, **kw)
        if kw:
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(before, self.state))
            self.state = [kw["block_table_out"], self.state[1], kw["refcount_out"]]
        m, n = self.pool.compact()
        self.same()
        assert np.array_equal(pmap.cpu().numpy(), m) and int(used) == n


# page sizes of 16-byte units and of 8, 4, 2 and 1 byte units, larger and smaller than a piece
SHAPES = [(64, 40), (24,), (4, 3), (6,), (13,), (16,), (5, 4096)]


@pytest.mark.parametrize("P", [37, 700])
@pytest.mark.parametrize("seed", [0, 1, 2])
def test_random_calls(P, seed):
    rng = np.random.default_rng(seed * 100 + P)
    slots, max_pages = 12, 9
    b = Both(P, slots, max_pages, SHAPES, seed)
    for _ in range(60):
        op = rng.integers(5)
        n = int(rng.integers(1, 9))
        s = rng.integers(-1, slots + 1, n)      # out of range and the same one twice among them
        if op <= 1:
            at = np.clip(s, 0, slots - 1)
            b.extend(s, b.pool.lens[at] + rng.integers(-3, 200, n))
        elif op == 2:
            b.fork(rng.integers(0, slots, n), s)
        elif op == 3:
            b.free(s[:3])
        else:
            b.compact(in_place=bool(rng.integers(2)))


def test_statuses():
    b = Both(4, 6, 3, [(16,)], 1)
    assert list(b.extend([0, 1, 0, 6, -1, 2], [100, 0, 128, 5, 5, 193])) == [0, 0, 2, 2, 2, 2]
    # two pages left: the second entry is refused, then every one that needs a page
    assert list(b.extend([2, 3, 4, 0, 5], [64, 128, 64, 128, 0])) == [0, 1, 1, 0, 0]
    assert list(b.extend([0], [127])) == [2]                       # never shorter
    assert list(b.fork([0, 2, 0, 3], [1, 2, 9, 3])) == [0, 2, 2, 0]  # slot 2 is not empty, 9 is none, 3 is empty itself
    assert list(b.extend([4], [33])) == [0]
    assert list(b.fork([4, 0, 4], [3, 5, 3])) == [1, 0, 2]           # no page for a partly filled last one


def test_fork_shares_and_frees_in_any_order():
    b = Both(300, 40, 20, SHAPES[:3], 2)
    b.extend([0, 1, 2], [1000, 64, 130])
    b.fork([0] * 10 + [1] * 5 + [2] * 5, np.arange(10, 30))
    b.fork([12, 29], [30, 31])                 # forks of forks
    b.extend(np.arange(10, 30), b.pool.lens[10:30] + 70)
    b.free([0, 0, 1, 2, 2, 0])                 # the same slot several times
    b.free(np.arange(10, 32))
    assert b.pool.refs.sum() == 0


@pytest.mark.parametrize("P", [16384, 16385, 200001])
def test_large_pools(P):
    # over the size from which several CTAs share the counts; the free pages at
    # the far end, and a pool with none left
    rng = np.random.default_rng(P)
    slots, max_pages = 1024, 256
    b = Both(P, slots, max_pages, [(16,)], 3)
    b.pool.refs[:] = rng.random(P) < 0.7
    b.pool.refs[: P // 2] = 1
    b.pool.refs[-1] = 0
    b.state[2].copy_(i32(b.pool.refs))
    n_free = int((b.pool.refs == 0).sum())
    want = rng.integers(0, 64 * max(n_free // 1000, 2), slots)
    b.extend(rng.permutation(slots), want)
    b.extend(rng.permutation(slots), np.minimum(b.pool.lens.max() + 700, 64 * max_pages) + np.zeros(slots, int))
    b.fork(rng.integers(0, 10, 20), rng.integers(0, slots, 20))
    b.free(rng.permutation(slots)[:1000])
    b.compact()


def test_extend_grants_every_last_page():
    b = Both(20000, 2, 20000, [(16,)], 4)
    assert list(b.extend([1], [64 * 20000])) == [0]
    assert list(b.extend([0], [1])) == [1]
    b.free([1])
    assert list(b.extend([0], [64 * 20000 - 1])) == [0]


def test_counts_below_zero_are_never_granted():
    b = Both(50, 3, 60, [(16,)], 5)
    b.pool.refs[[0, 3, 49]] = -1
    b.state[2].copy_(i32(b.pool.refs))
    assert list(b.extend([0], [64 * 48])) == [1]
    assert list(b.extend([0], [64 * 47])) == [0]
    b.free([0])
    assert list(b.pool.refs[[0, 3, 49]]) == [-1, -1, -1]


@pytest.mark.parametrize("P", [40, 5000])
def test_compact_of_empty_full_and_packed_pools(P):
    b = Both(P, 4, P, [(64,), (3,)], 6)
    b.compact()
    b.extend([0], [64 * P])
    b.compact()
    b.free([0])
    b.extend([1, 2, 3], [64 * (P // 4), 1, 64 * (P // 2)])
    b.compact(in_place=False)
    b.free([1])
    b.compact()
    b.compact()


@pytest.mark.parametrize("n", [1, 500])
def test_copy(n):
    rng = np.random.default_rng(n)
    P = 1200
    bufs = [rng.integers(0, 256, (P,) + s).astype(np.uint8) for s in SHAPES]
    both = rng.permutation(P)
    src, dst = both[:n].copy(), both[n:2 * n].copy()
    if n > 10:
        src[3] = src[4]              # one page to two places
        dst[5], src[6], dst[7] = P, -1, -9   # skipped
        dst[8] = src[8]
    g = [torch.from_numpy(b).to(DEV) for b in bufs]
    g.append(torch.arange(P * 6, device=DEV, dtype=torch.float32).view(P, 6))
    want = [t.cpu().numpy().copy() for t in g]
    for s, d in zip(src, dst):
        if 0 <= s < P and 0 <= d < P:
            for w in want:
                w[d] = w[s]
    dsa.pages_copy(g, i32(src), i32(dst))
    torch.cuda.synchronize()
    for a, b in zip(g, want):
        assert np.array_equal(a.cpu().numpy(), b)


def test_copy_of_buffers_off_their_alignment():
    # a buffer that starts 4 bytes past a 16-byte boundary moves in smaller units
    P = 30
    base = torch.randint(0, 256, (P * 48 + 4,), dtype=torch.uint8, device=DEV)
    t = base[4:].view(P, 48)
    want = t.cpu().numpy().copy()
    want[[7, 9]] = want[[1, 2]]
    dsa.pages_copy([t], i32([1, 2]), i32([7, 9]))
    torch.cuda.synchronize()
    assert np.array_equal(t.cpu().numpy(), want)


def test_copy_behind_four_gigabytes():
    P, size = 70000, 65536
    t = torch.zeros(P, size, dtype=torch.uint8, device=DEV)
    t[P - 1] = 7
    t[65537, ::2] = 9
    dsa.pages_copy([t], i32([P - 1, 65537]), i32([3, P - 2]))
    torch.cuda.synchronize()
    assert bool((t[3] == 7).all()) and bool((t[P - 2] == t[65537]).all())


def test_captured_calls_replay():
    b = Both(400, 10, 30, [(64, 8)], 7)
    slots, to, st = i32([0, 1, 2]), i32([0, 0, 0]), i32([9, 9, 9])
    par, chi, st2 = i32([0, 1]), i32([5, 6]), i32([9, 9])
    dsa.pages_free(chi, *b.state)      # every kernel has run once before the capture
    dsa.pages_extend(slots, to, *b.state, st)
    dsa.pages_fork(b.g, par, chi, *b.state, st2)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        dsa.pages_free(chi, *b.state)
        dsa.pages_extend(slots, to, *b.state, st)
        dsa.pages_fork(b.g, par, chi, *b.state, st2)
    lens = np.zeros(3, int)
    rng = np.random.default_rng(0)
    for _ in range(12):
        lens = lens + rng.integers(0, 150, 3)
        to.copy_(i32(lens))
        g.replay()
        b.pool.free([5, 6])
        w1 = b.pool.extend([0, 1, 2], lens)
        w2 = b.pool.fork([0, 1], [5, 6])
        b.same(st, w1)
        assert np.array_equal(st2.cpu().numpy(), w2)


def test_lengths_given_as_the_pool_s_own_tensor_and_calls_on_a_stream():
    b = Both(100, 6, 20, [(32,)], 8)
    b.extend([0, 1, 4], [100, 700, 1])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    slots, st = i32([1, 0, 2]), i32([9, 9, 9])
    lens = b.pool.lens.copy()
    # seq_lens[0..2] as the new lengths of slots 1, 0 and 2: 100 < 700 is refused, 700 > 100 is not
    dsa.pages_extend(slots, b.state[1][:3], *b.state, st, stream=side)
    dsa.pages_free(i32([4]), *b.state, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    want = b.pool.extend([1, 0, 2], lens[:3])
    b.pool.free([4])
    b.same(st, want)
    assert list(want) == [2, 0, 0]


def test_cache_object_takes_slots_out_of_range_as_empty():
    c = dsa.KV8Cache(20, 3, 4, 2, 64, scale_block=16)
    good = i32([0, 2])
    assert not c.extend(good, i32([70, 5])).any()
    kv = torch.randn(3, 2, 64, device=DEV).to(torch.bfloat16)
    slots = i32([0, 7, -2])
    c.append(kv, kv, slots=slots)
    before = c.k.clone()
    c.append(kv[1:], kv[1:], slots=slots[1:])     # nothing has a place
    q = torch.randn(3, 4, 64, device=DEV).to(torch.bfloat16)
    idx = i32([[69, -1], [0, 1], [0, 1]])
    out = torch.full_like(q, 3.0)
    c.prefill(q, idx, i32([0, 1, 2, 3]), out, slots=slots)
    torch.cuda.synchronize()
    assert torch.equal(before, c.k) and not out[1:].any() and bool(out[0].any())
    with pytest.raises(ValueError):
        c.decode(q, None, None, None, 70, 2, None, out, slots=slots)   # holds no indexer keys


def test_a_serving_run_of_them_together():
    """Prompts appended and attended, a sequence forked, single tokens appended
    to all and decoded, one freed, the pool compacted: the forked sequence
    decodes like its parent, and compacting changes no bit of a decode."""
    from sparse_long_context_03_b200 import inputs
    cfg = inputs.config(3)
    Hq, Hkv, D, HI, dI, k = cfg.Hq, cfg.Hkv, cfg.D, cfg.HI, cfg.dI, 256
    gen = torch.Generator(device=DEV)
    gen.manual_seed(5)
    c = dsa.KV8Cache(200, 6, 30, Hkv, D, dI=dI, scale_block=32)

    def tokens(n):
        kv = torch.randn(n, 2 * Hkv * D, generator=gen, device=DEV).to(torch.bfloat16)
        k8, ks = inputs.quantize_e4m3_per_token(torch.randn(n, dI, generator=gen, device=DEV))
        return kv[:, :Hkv * D].unflatten(1, (Hkv, D)), kv[:, Hkv * D:].unflatten(1, (Hkv, D)), k8, ks

    # prompts in slots 0, 2 and 3, packed
    slots, new = i32([0, 2, 3]), [700, 64, 333]
    assert not c.extend(slots, i32(new)).any()
    cu = i32(np.concatenate([[0], np.cumsum(new)]))
    n = sum(new)
    K, V, k8, ks = tokens(n)
    c.append(K, V, cu, k8, ks, slots=slots)
    plan = dsa.PrefillPlan(n, HI, dI, Hq, Hkv, D, k)
    q8, sq = inputs.quantize_e4m3_per_token(torch.randn(n, HI, dI, generator=gen, device=DEV))
    w = torch.rand(n, HI, generator=gen, device=DEV)
    Q = torch.randn(n, Hq, D, generator=gen, device=DEV).to(torch.bfloat16)
    O16, idx = torch.empty_like(Q), torch.empty(n, k, dtype=torch.int32, device=DEV)
    dsa.prefill_forward_packed(plan, cu, q8, sq, w, k8, ks, Q, K.contiguous(), V.contiguous(), O16, idx_out=idx)
    O8 = torch.empty_like(Q)
    c.prefill(Q, idx, cu, O8, slots=slots)
    # the cache holds K and V with a relative error of 2^-4 per value: the
    # outputs agree as far as random errors of that size average out
    a, b = O8.double(), O16.double()
    assert ((a - b).norm() / b.norm()).item() < 0.06
    # fork slot 0 to 4 and 5; one new token each, the same for all of them
    assert not c.fork(i32([0, 0]), i32([4, 5])).any()
    assert c.refcount.max().item() == 3
    ws = torch.empty(dsa.decode_kv8_workspace_size(4, 1024, k), dtype=torch.uint8, device=DEV)
    live = i32([0, 4, 5, 3])
    for step in range(70):     # over a page's border
        assert not c.extend(live, c.seq_lens[live.long()] + 1).any()
        K, V, k8, ks = (t[:1].expand(4, *t.shape[1:]).contiguous() for t in tokens(1))
        c.append(K, V, None, k8, ks, slots=live)
    q = torch.randn(1, Hq, D, generator=gen, device=DEV).to(torch.bfloat16).expand(4, Hq, D).contiguous()
    q8, sq = inputs.quantize_e4m3_per_token(torch.randn(1, HI, dI, generator=gen, device=DEV).expand(4, HI, dI))
    w = torch.rand(1, HI, generator=gen, device=DEV).expand(4, HI).contiguous()
    outs, sets = [], []
    for _ in range(2):
        out, sel = torch.empty(4, Hq, D, dtype=torch.bfloat16, device=DEV), torch.empty(4, k, dtype=torch.int32, device=DEV)
        c.decode(q, q8, sq, w, 1024, k, ws, out, idx_out=sel, slots=live)
        torch.cuda.synchronize()
        assert torch.equal(out[0], out[1]) and torch.equal(out[0], out[2])
        assert torch.equal(sel[0], sel[1]) and not torch.equal(sel[0], sel[3])
        outs.append(out)
        sets.append(sel)
        c.free(i32([2]))
        page_map, used = c.compact()
        assert int(used) == int((c.refcount > 0).sum()) and not c.refcount[int(used):].any()
    assert torch.equal(outs[0], outs[1]) and torch.equal(sets[0], sets[1])
    c.free(i32([0, 3, 4, 5]))
    assert not c.refcount.any() and bool((c.block_table == -1).all())


@pytest.mark.parametrize("how", ["one stream", "two streams", "a graph", "a graph of two streams"])
def test_calls_that_follow_each_other_see_what_came_before(how):
    """Calls begin while the ones before them end: rounds of every call, each
    on what the last one wrote, give the bits that they give one at a time;
    between them lie copies, fills and kernels that are not the library's."""
    S, Hq, Hkv, D, k, rounds = 24, 16, 2, 128, 96, 12
    gen = torch.Generator(device=DEV)
    gen.manual_seed(11)
    kv = torch.randn(rounds, 2, S * 40, Hkv, D, generator=gen, device=DEV).to(torch.bfloat16)
    qs = torch.randn(rounds, S, Hq, D, generator=gen, device=DEV).to(torch.bfloat16)
    order = torch.stack([torch.randperm(S, generator=gen, device=DEV) for _ in range(rounds)]).to(torch.int32)
    cu = i32(np.arange(S + 1) * 40)
    plus = i32([40] * S)
    picks = torch.arange(k, dtype=torch.int32, device=DEV)

    def run(between, outs, sync, c):
        for t in (c.k, c.v, c.seq_lens, c.refcount):
            t.zero_()
        c.exp.fill_(87)
        c.block_table.fill_(-1)
        for r in range(rounds):
            all_slots = order[r]
            half = all_slots[:S // 2]
            calls = [lambda: c.extend(all_slots, c.seq_lens[all_slots.long()] + plus),
                     lambda: c.append(kv[r, 0], kv[r, 1], cu, slots=all_slots),
                     lambda: dsa.sparse_gqa_decode_attention_kv8(
                         qs[r], c.k, c.v, c.exp, c.block_table, c.seq_lens,
                         (c.seq_lens[:, None] - k + picks).clamp(min=0).to(torch.int32), k, 0.05, outs[r]),
                     lambda: dsa.sparse_gqa_decode_attention_kv8(
                         outs[r], c.k, c.v, c.exp, c.block_table, c.seq_lens, picks.repeat(S, 1), k, 0.05, outs[r + 1]),
                     lambda: c.free(half),
                     lambda: c.fork(all_slots[S // 2:], half),
                     lambda: c.free(all_slots[:3]),
                     lambda: c.compact()]
            for i, call in enumerate(calls):
                between(i + r)
                call()
                if sync:
                    torch.cuda.synchronize()
        if torch.cuda.current_stream() == side:
            between(3)

    def cache():
        return dsa.KV8Cache(S * 8 + 20, S, 12, Hkv, D)

    def outputs():
        return torch.zeros(rounds + 1, S, Hq, D, dtype=torch.bfloat16, device=DEV)

    small, other = torch.ones(64, device=DEV), torch.zeros(64, device=DEV)
    main, side = torch.cuda.Stream(), torch.cuda.Stream()
    want_c, want = cache(), outputs()
    run(lambda i: None, want, True, want_c)
    c, outs = cache(), outputs()

    def between(i):
        # a copy, a fill, a kernel, nothing; with two streams the next call is
        # on the other one, behind an event
        if i % 4 == 0:
            other.copy_(small)
        elif i % 4 == 1:
            other.zero_()
        elif i % 4 == 2:
            other.add_(small)
        if "two streams" in how:
            here = torch.cuda.current_stream()
            there = side if here == main else main
            there.wait_stream(here)
            torch.cuda.set_stream(there)

    torch.cuda.synchronize()
    before = torch.cuda.current_stream()
    if "graph" in how:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=main):
            run(between, outs, False, c)
        for _ in range(3):
            outs.zero_()
            g.replay()
    else:
        torch.cuda.set_stream(main)
        try:
            for _ in range(3):
                run(between, outs, False, c)
        finally:
            torch.cuda.set_stream(before)
    torch.cuda.synchronize()
    assert torch.equal(outs.view(torch.int16), want.view(torch.int16)) and bool(want.any())
    for a, b in ((c.k, want_c.k), (c.v, want_c.v), (c.exp, want_c.exp), (c.block_table, want_c.block_table),
                 (c.seq_lens, want_c.seq_lens), (c.refcount, want_c.refcount)):
        assert torch.equal(a, b)
    assert int(c.seq_lens.max()) > 40
