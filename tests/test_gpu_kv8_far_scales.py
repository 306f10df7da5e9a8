"""Attention over the 8-bit cache where V's block scales lie far apart: each
dim of the output is held to the weighted mean of that dim's own values, also
where the keys of the largest scales hold zeros in it."""
import numpy as np
import pytest
import torch

import kv8_reference as ref
from sparse_long_context_03_b200 import dsa

pytestmark = pytest.mark.gpu
DEV = "cuda"


def dev(x, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(x))
    return (t if dtype is None else t.to(dtype)).to(DEV)


def exact(q, kc, vc, exp, table, idx, seq, pos, sm):
    """(out, lse, tol_out, tol_lse) in 64 bits.

    Bounds: d, an exponent's error, as in kv8_reference.attention, and the sums'
    there.  A weight is rounded to fp16, 2^-11 of itself, but for one below
    fp16's normal range beside a V scale no more than 2^4 below that of the
    key that set the reference: that one is off by 2^-25 on a scale on which
    the reference's key has 2^7, so with softmax weights of sum 1 by at most
    2^-32 * 2^4 = 2^-28.  The output is rounded to bf16 (2^-8)."""
    n, Hq, D = q.shape
    Hkv, block = kc.shape[2], 64 // exp.shape[1]
    out, lse = np.zeros((n, Hq, D)), np.full((n, Hq), -np.inf)
    tol_o, tol_l = np.zeros((n, Hq, D)), np.zeros((n, Hq))
    for r in range(n):
        e = idx[r][: max(min(idx.shape[1], pos[r] + 1), 0)]
        e = e[(e >= 0) & (e <= pos[r])]
        if not len(e):
            continue
        page, s = table[seq[r]][e // 64], e % 64
        sc = 2.0 ** (exp[page, s // block].astype(np.float64) - 127)
        kk, vv = ref.e4m3_values(kc[page, s]), ref.e4m3_values(vc[page, s])
        for h in range(Hq):
            g = h // (Hq // Hkv)
            x = (kk[:, g] @ q[r, h]) * sc[:, g, 0] * sm
            mag = (np.abs(kk[:, g]) @ np.abs(q[r, h])) * sc[:, g, 0] * abs(sm)
            p = np.exp(x - x.max())
            L = p.sum()
            V = vv[:, g] * sc[:, g, 1:2]
            out[r, h], lse[r, h] = p @ V / L, x.max() + np.log(L)
            ev = np.abs(np.log2(sc[:, g, 1])).max()
            d = 2.0 ** -19 * mag.max() + np.log(2) * (2.0 ** -22 * (np.abs(x).max() * 1.45 + ev + 40) + 2.0 ** -21)
            sums = (len(e) / 16 + 64) * 2.0 ** -23
            tol_o[r, h] = 2.0 ** -8 * np.abs(out[r, h]) + 1.01 * (2 * d + 2.0 ** -11 + 2 * sums) * (p @ np.abs(V) / L) \
                + len(e) * 2.0 ** -28 * np.abs(V).max(0)
            tol_l[r, h] = d + sums + 2.0 ** -22 * (abs(lse[r, h]) + 60)
    return out, lse, tol_o, tol_l


def check(out, lse, want):
    o, l, to, tl = want
    out, lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
    assert np.array_equal(np.isfinite(lse), np.isfinite(l))
    fin = np.isfinite(l)
    assert np.all(np.abs(lse[fin] - l[fin]) <= tl[fin])
    bad = ~(np.abs(out - o) <= to)
    assert not bad.any(), f"{bad.sum()} of {bad.size} outputs off, worst {np.max(np.abs(out - o)[bad] / np.maximum(to, 1e-300)[bad])} bounds"


def test_a_zero_of_a_large_scale_beside_a_one():
    # two keys of equal score: 0 at 2^40 and 1 at 2^0
    kc = np.zeros((2, 64, 1, 64), np.uint8)
    vc = np.zeros_like(kc)
    exp = np.full((2, 1, 1, 2), 127, np.uint8)
    exp[0, ..., 1] = 167
    vc[1, 0] = 0x38                                   # 1.0
    q = torch.ones(1, 1, 64, dtype=torch.bfloat16, device=DEV)
    out = torch.empty_like(q)
    dsa.sparse_gqa_decode_attention_kv8(q, dev(kc), dev(vc), dev(exp), dev(np.array([[0, 1]], np.int32)),
                                        dev(np.array([65], np.int32)), dev(np.array([[0, 64]], np.int32)), 2, 0.1, out)
    assert torch.all(out == 0.5)


@pytest.mark.parametrize("d", [5, 20, 29, 32, 36, 47, 60, 80])
@pytest.mark.parametrize("D,B,k", [(64, 2, 33), (128, 2, 700), (128, 40, 96), (64, 450, 40), (128, 600, 1100)])
def test_one_outlier_s_block_among_ordinary_ones(D, B, k, d):
    # one block of a scale 2^d above the others', all its V in one dim; the
    # other dims are means of the ordinary blocks
    rng = np.random.default_rng(d * 1000 + B)
    Hq, Hkv, block, L = 8, 4, 32, max(2 * k, 64)
    P = -(-L // 64)
    kc = rng.integers(0, 127, (P, 64, Hkv, D)).astype(np.uint8) | (rng.integers(0, 2, (P, 64, Hkv, D)).astype(np.uint8) << 7)
    vc = rng.integers(32, 127, (P, 64, Hkv, D)).astype(np.uint8)
    exp = np.empty((P, 64 // block, Hkv, 2), np.uint8)
    exp[..., 0] = 118
    base = int(rng.integers(87, 168 - d))
    exp[..., 1] = base
    exp[0, 0, :, 1] = base + d
    vc[0, :block, :, 1:] = 0
    table = np.tile(rng.permutation(P).astype(np.int32)[None], (B, 1))
    kc[table[0]], vc[table[0]], exp[table[0]] = kc.copy(), vc.copy(), exp.copy()
    idx = np.stack([np.sort(np.concatenate([[r % block], block + rng.permutation(L - block)[: k - 1]])) for r in range(B)])
    lens, q = np.full(B, L), torch.randn(B, Hq, D).to(torch.bfloat16)
    out, lse = torch.empty(B, Hq, D, dtype=torch.bfloat16, device=DEV), torch.empty(B, Hq, device=DEV)
    sm = 0.05 / np.sqrt(D)
    dsa.sparse_gqa_decode_attention_kv8(q.to(DEV), dev(kc), dev(vc), dev(exp), dev(table), dev(lens, torch.int32),
                                        dev(idx, torch.int32), k, sm, out, lse)
    rows = np.unique(rng.integers(0, B, 12))
    want = exact(q.double().numpy()[rows], kc, vc, exp, table, idx[rows], rows, lens[rows] - 1, float(np.float32(sm)))
    check(out[torch.from_numpy(rows).to(DEV)], lse[torch.from_numpy(rows).to(DEV)], want)


@pytest.mark.parametrize("sm", [0.0, 1.0, 30.0])
@pytest.mark.parametrize("Hq,Hkv,D,block,n,k", [(7, 1, 64, 16, 3, 200), (32, 4, 128, 32, 30, 300), (8, 8, 128, 64, 1, 64),
                                                (16, 4, 64, 16, 500, 700), (10, 5, 128, 16, 600, 130)])
def test_prefill_over_the_whole_range_of_scales(Hq, Hkv, D, block, n, k, sm):
    # scales from 2^-40 to 2^40 side by side; in each block three dims of four
    # are zero, so that every dim has its own largest scale; flat and sharp
    # weights; entries that select nothing among them
    rng = np.random.default_rng(n + k)
    L = n + 1000
    P = -(-L // 64)
    kc = rng.integers(0, 127, (P, 64, Hkv, D)).astype(np.uint8) | (rng.integers(0, 2, (P, 64, Hkv, D)).astype(np.uint8) << 7)
    vc = rng.integers(1, 127, (P, 64, Hkv, D)).astype(np.uint8) | (rng.integers(0, 2, (P, 64, Hkv, D)).astype(np.uint8) << 7)
    per = 64 // block
    exp = rng.integers(87, 168, (P, per, Hkv, 2)).astype(np.uint8)
    exp[..., 0] = rng.integers(116, 120, exp.shape[:-1])
    vc[np.repeat(rng.random((P, per, Hkv, D)) < 0.75, block, axis=1)] = 0
    table = rng.permutation(P).astype(np.int32)[None]
    pos = L - n + np.arange(n)
    idx = np.stack([np.sort(rng.permutation(int(p) + 1)[:k]) for p in pos])
    idx[::3, ::7] = -1
    q = torch.randn(n, Hq, D).to(torch.bfloat16)
    O, lse = torch.empty(n, Hq, D, dtype=torch.bfloat16, device=DEV), torch.empty(n, Hq, device=DEV)
    sm = sm / np.sqrt(D)
    dsa.sparse_gqa_prefill_kv8(q.to(DEV), dev(kc), dev(vc), dev(exp), dev(table), dev(np.array([L]), torch.int32),
                               dev(idx, torch.int32), dev(np.array([0, n]), torch.int32), 0, n, k, sm, O, lse)
    rows = np.unique(np.concatenate([[0], rng.integers(0, n, 12)]))
    want = exact(q.double().numpy()[rows], kc, vc, exp, table, idx[rows], np.zeros(len(rows), int), pos[rows],
                 float(np.float32(sm)))
    check(O[torch.from_numpy(rows).to(DEV)], lse[torch.from_numpy(rows).to(DEV)], want)
