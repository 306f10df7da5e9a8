"""Appending to the 8-bit cache where a sequence is shorter than its new
tokens: those at negative positions are dropped, the others have their places."""
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


@pytest.mark.parametrize("block", [16, 32, 64])
@pytest.mark.parametrize("Hkv,D", [(2, 128), (3, 64)])
def test_only_tokens_at_negative_positions_are_dropped(block, Hkv, D):
    rng = np.random.default_rng(block + D)
    lens = np.array([3, 40, 0, -5, 130, 64, 17, 100, -2 ** 31, 1])
    new = np.array([5, 100, 7, 3, 131, 200, 17, 30, 9, 64])
    cu = np.concatenate([[0], np.cumsum(new)])
    P = 3 * len(lens)
    table = rng.permutation(P).astype(np.int32).reshape(-1, 3)
    n = int(cu[-1])
    kc, vc = (rng.integers(0, 127, (P, 64, Hkv, D)).astype(np.uint8) for _ in range(2))
    exp = rng.integers(100, 140, (P, 64 // block, Hkv, 2)).astype(np.uint8)
    K, V = (torch.from_numpy(rng.standard_normal((n, Hkv, D)) * 2.0 ** rng.integers(-9, 9, (n, 1, 1))).to(torch.bfloat16)
            for _ in range(2))
    k8, ks = rng.integers(0, 256, (n, 32)).astype(np.uint8), rng.random(n).astype(np.float32)
    k8c, ksc = rng.integers(0, 256, (P, 64, 32)).astype(np.uint8), rng.random((P, 64)).astype(np.float32)
    want = [kc.copy(), vc.copy(), exp.copy(), k8c.copy(), ksc.copy()]
    ref.append(K.double().numpy(), V.double().numpy(), *want[:3], table, lens, cu)
    written = 0
    for b in range(len(lens)):
        for i in range(new[b]):
            pos = int(lens[b]) - int(new[b]) + i
            if pos >= 0:
                want[3][table[b, pos // 64], pos % 64] = k8[cu[b] + i]
                want[4][table[b, pos // 64], pos % 64] = ks[cu[b] + i]
                written += 1
    assert written == 3 + 40 + 130 + 64 + 17 + 30 + 1
    g = [dev(x) for x in (kc, vc, exp, k8c, ksc)]
    dsa.kv8_append(K.to(DEV), V.to(DEV), *g[:3], dev(table), dev(lens, torch.int32), cu_seqlens=dev(cu, torch.int32),
                   k8=dev(k8), k_scale=dev(ks), k8_cache=g[3], k_scale_cache=g[4])
    for name, a, b in zip(("k", "v", "exp", "k8", "k_scale"), g, want):
        assert np.array_equal(a.cpu().numpy(), b), name
