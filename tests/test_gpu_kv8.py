"""The 8-bit KV cache on the GPU against plain 64-bit implementations
(kv8_reference.py, which derives the bounds): appending is exact, attention is
within its bounds."""
import numpy as np
import pytest
import torch

import kv8_reference as ref
from sparse_long_context_03_b200 import dsa, inputs

pytestmark = pytest.mark.gpu
DEV = "cuda"


def dev(x, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(x))
    return (t if dtype is None else t.to(dtype)).to(DEV)


def deal(lens, rng, spare=2, max_pages=None):
    """Block table of randomly dealt pages; (table, number of pages)."""
    need = [-(-max(int(n), 0) // 64) for n in lens]
    P = sum(need) + spare
    perm, at = rng.permutation(P), 0
    table = np.full((len(lens), max_pages or max(max(need, default=1), 1)), -1, np.int32)
    for b, n in enumerate(need):
        table[b, :n] = perm[at:at + n]
        at += n
    return table, P


def random_cache(P, Hkv, D, block, rng, lo=120, hi=134):
    data = [rng.integers(0, 127, (P, 64, Hkv, D)).astype(np.uint8) |
            (rng.integers(0, 2, (P, 64, Hkv, D)).astype(np.uint8) << 7) for _ in range(2)]
    exp = rng.integers(lo, hi + 1, (P, 64 // block, Hkv, 2)).astype(np.uint8)
    return data[0], data[1], exp


def bf16(x):
    """float64 values of x rounded to bf16, and the tensor."""
    t = torch.from_numpy(np.ascontiguousarray(x)).to(torch.bfloat16)
    return t.double().numpy(), t.to(DEV)


# ---------------------------------------------------------------------------
# append
# ---------------------------------------------------------------------------

def run_append(x, cu, lens, table, cache, keys=None, wide=0, single=False):
    """x: (K, V) bf16 tensors [n, Hkv, D] on the GPU."""
    g = [dev(c) for c in cache]
    if wide:
        # rows as parts of wider ones, the surroundings NaN
        x = [torch.cat([torch.full((t.shape[0], wide, t.shape[2]), float("nan"), dtype=t.dtype, device=DEV), t], 1)
             [:, wide:] for t in x]
    kw = {}
    if keys is not None:
        kw = dict(k8=dev(keys[0]), k_scale=dev(keys[1]), k8_cache=dev(keys[2]), k_scale_cache=dev(keys[3]))
    dsa.kv8_append(x[0], x[1], *g, dev(table), dev(lens, torch.int32),
                   cu_seqlens=None if single else dev(cu, torch.int32), **kw)
    torch.cuda.synchronize()
    got = [t.cpu().numpy() for t in g]
    return got + ([kw["k8_cache"].cpu().numpy(), kw["k_scale_cache"].cpu().numpy()] if keys is not None else [])


@pytest.mark.parametrize("block", [16, 32, 64])
@pytest.mark.parametrize("Hkv,D", [(4, 128), (3, 64), (1, 128)])
@pytest.mark.parametrize("old,new", [
    ([0], [1]), ([0, 0], [64, 65]), ([5, 63, 64, 15, 16, 0, 100], [1, 2, 130, 0, 17, 300, 64]),
    ([0, 200, 0], [0, 0, 0]),
])
def test_append_is_exact(block, Hkv, D, old, new):
    rng = np.random.default_rng(block * 1000 + Hkv * 10 + len(old) + D)
    old, new = np.array(old), np.array(new)
    lens, cu = old + new, np.concatenate([[0], np.cumsum(new)])
    table, P = deal(lens, rng)
    kc, vc, exp = random_cache(P, Hkv, D, block, rng, 100, 140)
    n = int(cu[-1])
    # magnitudes from far below to far above the old tokens': some blocks' scales grow
    K, Kt = bf16(rng.standard_normal((n, Hkv, D)) * 2.0 ** rng.integers(-30, 30, (n, 1, 1)))
    V, Vt = bf16(rng.standard_normal((n, Hkv, D)) * 2.0 ** rng.integers(-30, 30, (n, Hkv, 1)))
    want = [kc.copy(), vc.copy(), exp.copy()]
    ref.append(K, V, *want, table, lens, cu)
    dI = 64
    keys = [rng.integers(0, 256, (n, dI)).astype(np.uint8), rng.random(n).astype(np.float32),
            rng.integers(0, 256, (P, 64, dI)).astype(np.uint8), rng.random((P, 64)).astype(np.float32)]
    wk, ws = keys[2].copy(), keys[3].copy()
    for b in range(len(lens)):
        for i in range(new[b]):
            pos = old[b] + i
            wk[table[b, pos // 64], pos % 64] = keys[0][cu[b] + i]
            ws[table[b, pos // 64], pos % 64] = keys[1][cu[b] + i]
    got = run_append((Kt, Vt), cu, lens, table, (kc, vc, exp), keys, wide=2)
    for name, a, b in zip(("k", "v", "exp", "k8", "k_scale"), got, want + [wk, ws]):
        assert np.array_equal(a, b), f"{name}: {(a != b).sum()} of {a.size} differ"


@pytest.mark.parametrize("D", [64, 128])
def test_append_token_by_token(D):
    # 150 single tokens of growing and falling size, three sequences; the same
    # as the plain implementation after every one of them
    rng = np.random.default_rng(7)
    Hkv, block, n = 2, 16, 150
    start = np.array([0, 3, 61])
    table, P = deal(start + n, rng)
    cache = [c.copy() for c in random_cache(P, Hkv, D, block, rng, 87, 120)]
    g = [dev(c) for c in cache]
    bt = dev(table)
    for i in range(n):
        lens = start + i + 1
        K, Kt = bf16(rng.standard_normal((3, Hkv, D)) * 2.0 ** rng.integers(-50, 45))
        V, Vt = bf16(rng.standard_normal((3, Hkv, D)) * 2.0 ** rng.integers(-3, 3))
        ref.append(K, V, *cache, table, lens, np.arange(4))
        dsa.kv8_append(Kt, Vt, *g, bt, dev(lens, torch.int32))
    for a, b in zip(g, cache):
        assert np.array_equal(a.cpu().numpy(), b)


def test_append_extremes():
    # zeros, the smallest and largest bf16 values, values at the saturation
    # border and at the border between two scales
    rng = np.random.default_rng(8)
    vals = np.array([0.0, -0.0, 2.0 ** -133, 2.0 ** -126, 1e-20, 448 * 2.0 ** 40, 449 * 2.0 ** 40, 3.3e38, 1.75, 1.7578125,
                     -1.75, 448.0, 450.0, 1.0])
    Hkv, D, block = 2, 64, 16
    n = len(vals)
    x = np.zeros((n, Hkv, D))
    x[:, 0] = vals[:, None]
    x[:, 1, ::3] = vals[:, None]
    K, Kt = bf16(x)
    lens, cu = np.full(n, 17), np.arange(n + 1)      # one token each, all in blocks of their own
    table, P = deal(lens, rng)
    cache = random_cache(P, Hkv, D, block, rng)
    want = [c.copy() for c in cache]
    ref.append(K, K, *want, table, lens, cu)
    got = run_append((Kt, Kt), cu, lens, table, cache)
    for a, b in zip(got, want):
        assert np.array_equal(a, b)


def test_append_drops_what_has_no_place():
    # pages outside the pool, positions below zero and past the table, NaN rows
    # behind the last sequence: nothing of them is written
    rng = np.random.default_rng(9)
    Hkv, D, block = 2, 128, 32
    lens = np.array([40, 130, 3, 70, -5, 500])
    new = np.array([40, 100, 5, 70, 2, 450])
    cu = np.concatenate([[0], np.cumsum(new)])
    table, P = deal([40, 130, 0, 70, 0, 128], rng)
    table = np.concatenate([table[:, :2], np.full((6, 1), -1, np.int32)], 1)[:, :2].copy()
    table[3, 0] = P + 7
    table[1, 1] = -3
    n = int(cu[-1])
    x = rng.standard_normal((n + 9, Hkv, D))
    x[n:] = np.nan
    K, Kt = bf16(x)
    cache = random_cache(P, Hkv, D, block, rng)
    want = [c.copy() for c in cache]
    ref.append(K[:n], K[:n], *want, table, lens, cu)
    got = run_append((Kt, Kt), cu, lens, table, cache)
    for a, b in zip(got, want):
        assert np.array_equal(a, b)


def test_append_many_sequences():
    # more sequences than one round of the search over them covers, many of them empty
    rng = np.random.default_rng(10)
    Hkv, D, block = 1, 64, 16
    new = rng.integers(0, 4, 1500) * (rng.random(1500) < 0.5)
    old = rng.integers(0, 40, 1500)
    lens, cu = old + new, np.concatenate([[0], np.cumsum(new)])
    table, P = deal(lens, rng)
    cache = random_cache(P, Hkv, D, block, rng)
    K, Kt = bf16(rng.standard_normal((int(cu[-1]), Hkv, D)) * 50)
    want = [c.copy() for c in cache]
    ref.append(K, K, *want, table, lens, cu)
    got = run_append((Kt, Kt), cu, lens, table, cache)
    for a, b in zip(got, want):
        assert np.array_equal(a, b)


# ---------------------------------------------------------------------------
# attention
# ---------------------------------------------------------------------------

def pick_rows(seen, k, rng):
    """Ascending distinct positions, -1 behind them."""
    idx = np.full((len(seen), k), -1, np.int32)
    for r, n in enumerate(seen):
        m = min(k, max(int(n), 0))
        idx[r, :m] = np.sort(rng.permutation(int(n))[:m]) if m else []
    return idx


def check(out, lse, want, what=""):
    o, l, to, tl = want
    out, lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
    assert np.array_equal(np.isfinite(lse), np.isfinite(l)), what
    fin = np.isfinite(l)
    assert np.all(np.abs(lse[fin] - l[fin]) <= tl[fin]), f"{what}: lse off by {np.max(np.abs(lse[fin] - l[fin]) / tl[fin])} bounds"
    bad = np.abs(out - o) > to
    assert not bad.any(), f"{what}: {bad.sum()} outputs off, worst {np.nanmax(np.abs(out - o) / np.maximum(to, 1e-300))} bounds"


def decode(q, cache, table, lens, idx, sm):
    B, Hq, D = q.shape
    out = torch.full((B, Hq, D), float("nan"), dtype=torch.bfloat16, device=DEV)
    lse = torch.full((B, Hq), float("nan"), device=DEV)
    dsa.sparse_gqa_decode_attention_kv8(q, *cache, table, lens, idx, idx.shape[1], sm, out, lse)
    torch.cuda.synchronize()
    return out, lse


@pytest.mark.parametrize("Hq,Hkv,D,block", [(32, 4, 128, 64), (8, 2, 64, 16), (3, 3, 128, 32), (7, 1, 64, 64),
                                            (40, 8, 128, 16)])
@pytest.mark.parametrize("lens,k", [([1], 1), ([1, 63, 64, 65, 300, 1000, 0], 64), ([700], 700), ([2500, 31], 2048),
                                    ([90] * 40, 33)])
def test_decode_attention(Hq, Hkv, D, block, lens, k):
    rng = np.random.default_rng(Hq + D + k)
    table, P = deal(lens, rng)
    kc, vc, exp = random_cache(P, Hkv, D, block, rng, 118, 128)
    q, qt = bf16(rng.standard_normal((len(lens), Hq, D)))
    idx = pick_rows(lens, k, rng)
    sm = 0.02 / np.sqrt(D)
    out, lse = decode(qt, [dev(c) for c in (kc, vc, exp)], dev(table), dev(np.array(lens), torch.int32), dev(idx), sm)
    pos = np.array(lens) - 1
    check(out, lse, ref.attention(q, kc, vc, exp, table, idx, np.arange(len(lens)), pos, float(np.float32(sm))))


@pytest.mark.parametrize("sm,qscale", [(0.3, 1.0), (1e-3, 2.0 ** -100), (-0.01, 1.0), (0.0, 1.0), (1e-3, 2.0 ** 100)])
def test_decode_attention_sharp_flat_and_scaled_queries(sm, qscale):
    # weights from one key's to all equal; queries whose size fp16 could not hold
    rng = np.random.default_rng(12)
    lens, Hq, Hkv, D, block, k = [1200, 5, 400], 16, 2, 128, 16, 512
    table, P = deal(lens, rng)
    kc, vc, exp = random_cache(P, Hkv, D, block, rng, 112, 120)
    q, qt = bf16(rng.standard_normal((3, Hq, D)) * qscale * 2.0 ** rng.integers(-12, 12, (3, 1, D)))
    sm = sm / qscale if abs(qscale) < 2.0 ** 90 and qscale >= 2.0 ** -100 and qscale != 1.0 else sm / qscale
    idx = pick_rows(lens, k, rng)
    out, lse = decode(qt, [dev(c) for c in (kc, vc, exp)], dev(table), dev(np.array(lens), torch.int32), dev(idx), sm)
    check(out, lse, ref.attention(q, kc, vc, exp, table, idx, np.arange(3), np.array(lens) - 1, float(np.float32(sm))))


def test_decode_attention_scales_over_their_whole_range():
    # V's scales from 2^-40 to 2^40 side by side: a key of a tiny scale counts in
    # the sum of the weights, one of a huge scale decides the output
    rng = np.random.default_rng(13)
    lens, Hq, Hkv, D, block, k = [900, 64, 2000], 8, 2, 64, 16, 1024
    table, P = deal(lens, rng)
    kc, vc, exp = random_cache(P, Hkv, D, block, rng, 87, 167)
    exp[..., 0] = rng.integers(116, 122, exp.shape[:-1])
    q, qt = bf16(rng.standard_normal((3, Hq, D)))
    idx = pick_rows(lens, k, rng)
    sm = 0.02
    out, lse = decode(qt, [dev(c) for c in (kc, vc, exp)], dev(table), dev(np.array(lens), torch.int32), dev(idx), sm)
    check(out, lse, ref.attention(q, kc, vc, exp, table, idx, np.arange(3), np.array(lens) - 1, float(np.float32(sm))))


def test_nothing_of_unselected_rows_reaches_the_output():
    # NaN bytes and scale bytes of 255 everywhere but in the selected tokens'
    # rows and blocks, wrong pages and entries among the indices
    rng = np.random.default_rng(14)
    lens, Hq, Hkv, D, block, k = [500, 200, 77, 64, 300], 16, 4, 128, 16, 96
    table, P = deal(lens, rng)
    kc, vc, exp = random_cache(P, Hkv, D, block, rng, 118, 126)
    idx = pick_rows(lens, k, rng)
    idx[0, 5] = 500          # past the end
    idx[0, 6] = -7
    idx[1, :] = -1           # nothing selected
    idx[3, 0] = 2 ** 31 - 1
    table[2, 0] = P + 3      # a page outside the pool
    table[4, :] = -1         # no pages at all
    keep = np.zeros((P, 64), bool)
    for r in range(5):
        for e in idx[r]:
            if 0 <= e < lens[r] and 0 <= table[r, e // 64] < P:
                keep[table[r, e // 64], e % 64] = True
    kc[~keep] = 0x7F
    vc[~keep] = 0xFF
    exp[~keep.reshape(P, 64 // block, block).any(-1)] = 255
    q, qt = bf16(rng.standard_normal((5, Hq, D)))
    sm = 0.01
    out, lse = decode(qt, [dev(c) for c in (kc, vc, exp)], dev(table), dev(np.array(lens), torch.int32), dev(idx), sm)
    want = ref.attention(q, kc, vc, exp, table, idx, np.arange(5), np.array(lens) - 1, float(np.float32(sm)))
    check(out, lse, want)
    assert torch.all(out[1] == 0) and torch.all(out[4] == 0)
    assert torch.all(torch.isneginf(lse[1])) and torch.all(torch.isneginf(lse[4]))


def prefill(Q, cache, table, lens, idx, cu, r0, n, sm):
    Hq, D = Q.shape[1:]
    O = torch.full((n, Hq, D), 7.0, dtype=torch.bfloat16, device=DEV)
    lse = torch.full((n, Hq), 7.0, device=DEV)
    dsa.sparse_gqa_prefill_kv8(Q[r0:r0 + n], *cache, table, lens, idx[r0:r0 + n], cu, r0, n, idx.shape[1], sm, O, lse)
    torch.cuda.synchronize()
    return O, lse


@pytest.mark.parametrize("Hq,Hkv,D,block,k", [(32, 4, 128, 64, 48), (8, 2, 64, 16, 300), (5, 5, 64, 32, 1)])
@pytest.mark.parametrize("old,new", [([0], [1]), ([0, 10, 500, 64], [70, 0, 9, 64]), ([0, 0], [0, 3])])
def test_prefill_attention(Hq, Hkv, D, block, k, old, new):
    rng = np.random.default_rng(k + len(old))
    old, new = np.array(old), np.array(new)
    lens, cu = old + new, np.concatenate([[0], np.cumsum(new)])
    table, P = deal(lens, rng)
    kc, vc, exp = random_cache(P, Hkv, D, block, rng, 118, 126)
    n, tail = int(cu[-1]), 3
    seq = np.repeat(np.arange(len(new)), new)
    pos = old[seq] + np.arange(n) - cu[seq]
    idx = np.concatenate([pick_rows(pos + 1, k, rng), np.zeros((tail, k), np.int32)])
    q, qt = bf16(rng.standard_normal((n + tail, Hq, D)))
    sm = 0.01
    cache, bt = [dev(c) for c in (kc, vc, exp)], dev(table)
    args = (bt, dev(lens, torch.int32), dev(idx), dev(cu, torch.int32))
    O, lse = prefill(qt, cache, *args, 0, n + tail, sm)
    want = ref.attention(q[:n], kc, vc, exp, table, idx[:n], seq, pos, float(np.float32(sm)))
    check(O[:n], lse[:n], want)
    assert torch.all(O[n:] == 7) and torch.all(lse[n:] == 7)   # rows behind the last sequence
    # the same rows in two calls
    m = n // 2
    if m:
        for r0, c in ((0, m), (m, n - m)):
            O2, l2 = prefill(qt, cache, *args, r0, c, sm)
            check(O2, l2, [w[r0:r0 + c] for w in want], "chunk")


def test_prefill_agrees_with_the_bf16_kernel():
    # a cache whose values bf16 holds exactly: both kernels see the same K and V
    rng = np.random.default_rng(15)
    L, Hq, Hkv, D, k = 700, 32, 4, 128, 128
    table, P = deal([L], rng)
    kc, vc, exp = random_cache(P, Hkv, D, 32, rng, 119, 125)
    pos = np.arange(L)
    K, V = ((ref.e4m3_values(c[table[0, pos // 64], pos % 64]) *
             2.0 ** (exp[table[0, pos // 64], pos % 64 // 32, :, i].astype(float) - 127)[..., None])
            for i, c in enumerate((kc, vc)))
    idx = dev(pick_rows(pos + 1, k, rng))
    q, qt = bf16(rng.standard_normal((L, Hq, D)))
    sm = 0.02
    O, lse = prefill(qt, [dev(c) for c in (kc, vc, exp)], dev(table), dev(np.array([L]), torch.int32), idx,
                     dev(np.array([0, L]), torch.int32), 0, L, sm)
    O2, l2 = torch.empty_like(O), torch.empty_like(lse)
    dsa.sparse_gqa_prefill(qt, bf16(K)[1], bf16(V)[1], idx, 0, L, k, sm, O2, l2)
    # both round weights (bf16 2^-8, fp16 2^-11) against values up to 448 * 2^-2,
    # and their outputs (bf16 2^-8 each)
    vmax = float(np.abs(V).max())
    assert (O.double() - O2.double()).abs().max() <= (2.0 ** -8 + 2.0 ** -11 + 2 * 2.0 ** -8) * vmax
    assert (lse - l2).abs().max() <= 1e-3


def test_rows_behind_four_gigabytes():
    # a cache whose offsets pass 32 bits, in bytes of K and in the table
    Hq, Hkv, D, block, k = 8, 4, 128, 64, 64
    P = 2 ** 32 // (64 * Hkv * D) + 1000
    rng = np.random.default_rng(16)
    pages = np.array([P - 1, 3, P - 700, 2 ** 32 // (64 * Hkv * D)], np.int32)
    kc, vc, exp = random_cache(4, Hkv, D, block, rng, 118, 126)
    gk = torch.zeros(P, 64, Hkv, D, dtype=torch.uint8, device=DEV)
    gv = torch.zeros_like(gk)
    ge = torch.full((P, 1, Hkv, 2), 127, dtype=torch.uint8, device=DEV)
    at = torch.from_numpy(pages).long().to(DEV)
    # appended there, then read there
    lens, cu = np.array([250]), np.array([0, 250])
    K, Kt = bf16(rng.standard_normal((250, Hkv, D)))
    V, Vt = bf16(rng.standard_normal((250, Hkv, D)))
    dsa.kv8_append(Kt, Vt, gk, gv, ge, dev(pages[None]), dev(lens, torch.int32), cu_seqlens=dev(cu, torch.int32))
    kc[:], vc[:], exp[:] = 0, 0, 127
    ref.append(K, V, kc, vc, exp, np.arange(4)[None], lens, cu)
    for a, b in ((gk, kc), (gv, vc), (ge, exp)):
        assert np.array_equal(a[at].cpu().numpy(), b)
    idx = pick_rows(lens, k, rng)
    q, qt = bf16(rng.standard_normal((1, Hq, D)))
    out, lse = decode(qt, [gk, gv, ge], dev(pages[None]), dev(lens, torch.int32), dev(idx), 0.1)
    check(out, lse, ref.attention(q, kc, vc, exp, np.arange(4)[None], idx, [0], lens - 1, float(np.float32(0.1))))


def test_decode_attention_repeats_bit_for_bit_and_replays():
    cfg = inputs.config(3)
    rng = np.random.default_rng(17)
    lens = [5000, 1, 2047, 2049, 70000, 64]
    table, P = deal(lens, rng)
    kc, vc, exp = random_cache(P, cfg.Hkv, cfg.D, 64, rng, 112, 118)
    cache = [dev(c) for c in (kc, vc, exp)]
    bt, ln = dev(table), dev(np.array(lens), torch.int32)
    idx = dev(pick_rows(lens, cfg.k, rng))
    q = [bf16(rng.standard_normal((6, cfg.Hq, cfg.D)))[1] for _ in range(2)]
    first = [decode(x, cache, bt, ln, idx, cfg.sm_scale) for x in q]
    # two captured graphs, replayed in turn and against an eager call on another stream
    outs, graphs = [], []
    for x in q:
        o, l = torch.empty_like(first[0][0]), torch.empty_like(first[0][1])
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            dsa.sparse_gqa_decode_attention_kv8(x, *cache, bt, ln, idx, cfg.k, cfg.sm_scale, o, l)
        outs.append((o, l))
        graphs.append(g)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    eager = torch.empty_like(first[0][0])
    for _ in range(3):
        for g in graphs:
            g.replay()
        dsa.sparse_gqa_decode_attention_kv8(q[0], *cache, bt, ln, idx, cfg.k, cfg.sm_scale, eager, stream=side)
    torch.cuda.synchronize()
    for a, b in zip(outs, first):
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    assert torch.equal(eager, first[0][0])


def test_decode_chain_is_its_stages():
    cfg = inputs.config(3)
    lens = [1, 64, 2048, 2049, 5000, 30000]
    d = inputs.decode_inputs(cfg, seq_lens=lens, seed=21, device=DEV)
    P, B = d["num_pages"], len(lens)
    rng = np.random.default_rng(18)
    cache = [dev(c) for c in random_cache(P, cfg.Hkv, cfg.D, 32, rng, 112, 118)]
    ws = torch.empty(dsa.decode_kv8_workspace_size(B, d["max_seq_len"], cfg.k), dtype=torch.uint8, device=DEV)
    out = torch.empty(B, cfg.Hq, cfg.D, dtype=torch.bfloat16, device=DEV)
    idx = torch.empty(B, cfg.k, dtype=torch.int32, device=DEV)
    args = (d["q"], d["q8"], d["sq"], d["w"], d["k8_cache"], d["sk_cache"], *cache, d["block_table"], d["seq_lens"],
            d["max_seq_len"], cfg.k, cfg.sm_scale, ws)
    dsa.sparse_gqa_decode_kv8(*args, out, idx_out=idx)
    # the set is the bf16 chain's, the output the attention stage's
    ws2 = torch.empty(dsa.decode_workspace_size(B, d["max_seq_len"], cfg.Hq, cfg.Hkv, cfg.D, cfg.k), dtype=torch.uint8,
                      device=DEV)
    o2, i2 = torch.empty_like(out), torch.empty_like(idx)
    dsa.sparse_gqa_decode(d["q"], d["q8"], d["sq"], d["w"], d["k8_cache"], d["sk_cache"], d["k_cache"], d["v_cache"],
                          d["block_table"], d["seq_lens"], d["max_seq_len"], cfg.k, cfg.sm_scale, ws2, o2, idx_out=i2)
    o3, _ = decode(d["q"], cache, d["block_table"], d["seq_lens"], idx, cfg.sm_scale)
    torch.cuda.synchronize()
    assert torch.equal(idx, i2) and torch.equal(out, o3)
    out2 = torch.empty_like(out)
    dsa.sparse_gqa_decode_kv8(*args, out2)     # its own index rows in the workspace
    torch.cuda.synchronize()
    assert torch.equal(out, out2)


def test_decode_chain_with_empty_sequences():
    cfg = inputs.config(3)
    rng = np.random.default_rng(19)
    d = inputs.decode_inputs(cfg, seq_lens=[300, 1, 2100], seed=22, device=DEV)
    cache = [dev(c) for c in random_cache(d["num_pages"], cfg.Hkv, cfg.D, 64, rng, 112, 118)]
    for lens, most in (([300, 0, 2100], d["max_seq_len"]), ([0, 0, 0], d["max_seq_len"]), ([0, 0, 0], 0)):
        ws = torch.empty(dsa.decode_kv8_workspace_size(3, most, cfg.k), dtype=torch.uint8, device=DEV)
        out = torch.full((3, cfg.Hq, cfg.D), 7.0, dtype=torch.bfloat16, device=DEV)
        idx = torch.full((3, cfg.k), 7, dtype=torch.int32, device=DEV)
        ln = dev(np.array(lens), torch.int32)
        dsa.sparse_gqa_decode_kv8(d["q"], d["q8"], d["sq"], d["w"], d["k8_cache"], d["sk_cache"], *cache,
                                  d["block_table"], ln, most, cfg.k, cfg.sm_scale, ws, out, idx_out=idx)
        want, _ = decode(d["q"], cache, d["block_table"], ln, idx, cfg.sm_scale)
        torch.cuda.synchronize()
        assert torch.equal(out, want)
        for b, n in enumerate(lens):
            assert int((idx[b] >= 0).sum()) == min(n, cfg.k)
            assert n or not out[b].any()


@pytest.mark.parametrize("Hq,Hkv,D,k,B,n", [(8, 4, 128, 5000, 2, 21000), (8, 1, 64, 64, 3000, 90),
                                            (16, 16, 128, 40, 300, 70)])
def test_decode_attention_large_budgets_and_batches(Hq, Hkv, D, k, B, n):
    rng = np.random.default_rng(B)
    lens = rng.integers(n // 2, n, B)
    table, P = deal(lens, rng)
    kc, vc, exp = random_cache(P, Hkv, D, 32, rng, 118, 124)
    q, qt = bf16(rng.standard_normal((B, Hq, D)))
    idx = pick_rows(lens, k, rng)
    out, lse = decode(qt, [dev(c) for c in (kc, vc, exp)], dev(table), dev(lens, torch.int32), dev(idx), 0.01)
    rows = np.unique(rng.integers(0, B, 40))
    want = ref.attention(q[rows], kc, vc, exp, table, idx[rows], rows, lens[rows] - 1, float(np.float32(0.01)))
    at = torch.from_numpy(rows).to(DEV)
    check(out[at], lse[at], want)


@pytest.mark.parametrize("Hq,Hkv,D", [(4, 2, 64), (6, 3, 128), (32, 4, 128), (8, 8, 64), (5, 5, 128)])
def test_prefill_of_many_rows(Hq, Hkv, D):
    # enough rows for one warp to a pair, more entries than a block of the
    # lookup, and among them blocks and rows that select nothing, entries out
    # of range and pages outside the pool
    rng = np.random.default_rng(Hkv)
    old, new, k, block = 2600, 1000, 2100, 32
    lens, cu = np.array([old + new]), np.array([0, new])
    table, P = deal(lens, rng)
    table[0, 7] = P + 1
    kc, vc, exp = random_cache(P, Hkv, D, block, rng, 118, 124)
    spare = np.setdiff1d(np.arange(P), table[0])
    kc[spare], vc[spare], exp[spare] = 0x7F, 0x7F, 255       # pages that nobody selects
    pos = old + np.arange(new)
    idx = pick_rows(pos + 1, k, rng)
    idx[::7, ::5] = -1
    idx[1::7, :1024] = 2 ** 31 - 1                            # a block of nothing, then a block of something
    idx[2::7, 1024:] = -3
    idx[3::50] = -1
    idx[4::50] = 7 * 64 + 5                                   # the page that is none
    q, qt = bf16(rng.standard_normal((new, Hq, D)))
    O, lse = prefill(qt, [dev(c) for c in (kc, vc, exp)], dev(table), dev(lens, torch.int32), dev(idx),
                     dev(cu, torch.int32), 0, new, 0.01)
    rows = np.unique(np.concatenate([np.arange(8), [53, 54, 999], rng.integers(0, new, 12)]))
    want = ref.attention(q[rows], kc, vc, exp, table, idx[rows], np.zeros(len(rows), int), pos[rows],
                         float(np.float32(0.01)))
    at = torch.from_numpy(rows).to(DEV)
    check(O[at], lse[at], want)
    assert not O[3::50].any() and not O[4::50].any()
    assert bool(torch.isfinite(O).all())
    O2, l2 = prefill(qt, [dev(c) for c in (kc, vc, exp)], dev(table), dev(lens, torch.int32), dev(idx),
                     dev(cu, torch.int32), 0, new, 0.01)
    assert torch.equal(O, O2) and torch.equal(lse, l2)


@pytest.mark.parametrize("k", [1, 40, 130, 1030])
@pytest.mark.parametrize("B", [3, 4, 12, 13, 24, 25, 37, 38, 111, 112, 230])
def test_every_way_to_split_a_pair(B, k):
    """Batches on both sides of each change of the split, budgets of less than
    a step to more steps than a pair has warps; some sequences shorter than
    that, some empty."""
    rng = np.random.default_rng(B * k)
    Hq, Hkv, D, block = 12, 4, 64, 32
    lens = rng.integers(1, 1100, B)
    lens[rng.integers(0, B)] = 0
    table, P = deal(lens, rng)
    kc, vc, exp = random_cache(P, Hkv, D, block, rng, 118, 128)
    q, qt = bf16(rng.standard_normal((B, Hq, D)))
    idx = pick_rows(lens, k, rng)
    idx[0, rng.integers(0, k)] = -1
    sm = 0.02 / np.sqrt(D)
    out, lse = decode(qt, [dev(c) for c in (kc, vc, exp)], dev(table), dev(lens, torch.int32), dev(idx), sm)
    check(out, lse, ref.attention(q, kc, vc, exp, table, idx, np.arange(B), lens - 1, float(np.float32(sm))))


def test_prefill_of_many_sequences():
    # more sequences than one round of the search covers, most of them empty
    rng = np.random.default_rng(20)
    Hq, Hkv, D, block, k = 4, 2, 64, 16, 24
    new = rng.integers(0, 3, 1300) * (rng.random(1300) < 0.3)
    old = rng.integers(0, 100, 1300)
    lens, cu = old + new, np.concatenate([[0], np.cumsum(new)])
    table, P = deal(lens, rng)
    kc, vc, exp = random_cache(P, Hkv, D, block, rng, 118, 126)
    n = int(cu[-1])
    seq = np.repeat(np.arange(len(new)), new)
    pos = old[seq] + np.arange(n) - cu[seq]
    idx = pick_rows(pos + 1, k, rng)
    q, qt = bf16(rng.standard_normal((n, Hq, D)))
    O, lse = prefill(qt, [dev(c) for c in (kc, vc, exp)], dev(table), dev(lens, torch.int32), dev(idx),
                     dev(cu, torch.int32), 0, n, 0.02)
    check(O, lse, ref.attention(q, kc, vc, exp, table, idx, seq, pos, float(np.float32(0.02))))


def test_two_calls_at_once_and_a_repeated_entry():
    rng = np.random.default_rng(21)
    lens, Hq, Hkv, D, block, k = [3000, 700], 16, 4, 128, 64, 512
    table, P = deal(lens, rng)
    kc, vc, exp = random_cache(P, Hkv, D, block, rng, 118, 124)
    idx = pick_rows(lens, k, rng)
    idx[1, 100:200] = idx[1, 7]      # one key a hundred times: counted as often
    q, qt = bf16(rng.standard_normal((2, Hq, D)))
    cache, bt, ln, ix = [dev(c) for c in (kc, vc, exp)], dev(table), dev(np.array(lens), torch.int32), dev(idx)
    streams = [torch.cuda.Stream() for _ in range(4)]
    outs = [(torch.empty(2, Hq, D, dtype=torch.bfloat16, device=DEV), torch.empty(2, Hq, device=DEV)) for _ in streams]
    for s, (o, l) in zip(streams, outs):
        s.wait_stream(torch.cuda.current_stream())
        for _ in range(20):
            dsa.sparse_gqa_decode_attention_kv8(qt, *cache, bt, ln, ix, k, 0.01, o, l, stream=s)
    torch.cuda.synchronize()
    want = ref.attention(q, kc, vc, exp, table, idx, np.arange(2), np.array(lens) - 1, float(np.float32(0.01)))
    for o, l in outs:
        check(o, l, want)
        assert torch.equal(o, outs[0][0]) and torch.equal(l, outs[0][1])


def test_refusals_of_the_binding():
    kc = torch.zeros(3, 64, 2, 64, dtype=torch.uint8, device=DEV)
    exp = torch.full((3, 2, 2, 2), 127, dtype=torch.uint8, device=DEV)
    bt, ln = torch.zeros(2, 3, dtype=torch.int32, device=DEV), torch.ones(2, dtype=torch.int32, device=DEV)
    q = torch.zeros(2, 4, 64, dtype=torch.bfloat16, device=DEV)
    idx = torch.zeros(2, 8, dtype=torch.int32, device=DEV)

    def attend(**kw):
        a = dict(q=q, k=kc, v=kc, exp=exp, bt=bt, ln=ln, idx=idx, out=torch.empty_like(q))
        a.update(kw)
        dsa.sparse_gqa_decode_attention_kv8(a["q"], a["k"], a["v"], a["exp"], a["bt"], a["ln"], a["idx"], 8, 0.1,
                                            a["out"])

    attend()
    for kw in (dict(v=kc[:2]), dict(exp=exp[:, :1, :, :1]), dict(idx=idx[:, :7]), dict(bt=bt[:1]), dict(ln=ln.cpu()),
               dict(q=q[:, :, ::2]), dict(out=q[:1]), dict(exp=torch.cat([exp, exp, exp], 1)), dict(bt=bt[:, ::2])):
        with pytest.raises(ValueError):
            attend(**kw)
    for kw in (dict(q=q.half()), dict(k=kc.to(torch.int8)), dict(idx=idx.long()), dict(ln=ln.float())):
        with pytest.raises(TypeError):
            attend(**kw)
    kv = torch.zeros(2, 2, 64, dtype=torch.bfloat16, device=DEV)
    with pytest.raises(ValueError):
        dsa.kv8_append(kv[:1], kv[:1], kc, kc, exp, bt, ln)                      # one token for two sequences
    with pytest.raises(ValueError):
        dsa.kv8_append(kv.transpose(1, 2).contiguous().transpose(1, 2), kv, kc, kc, exp, bt, ln)
    with pytest.raises(ValueError):
        dsa.kv8_append(kv, kv, kc, kc, exp, bt, ln, k_scale=torch.ones(2, device=DEV))
    with pytest.raises(dsa.DSAError):
        dsa.kv8_append(kv.new_zeros(2, 132)[:, 4:].unflatten(1, (2, 64)), kv, kc, kc, exp, bt, ln)  # rows off 16 bytes
    torch.cuda.synchronize()
