"""The 8-bit KV cache's and the pages' argument checks, and the plain
implementations' own pins.  Nothing here needs a GPU or launches anything."""
import ctypes

import numpy as np
import pytest
import torch

import kv8_reference as ref
from sparse_long_context_03_b200 import build, dsa

OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3
B = 0x1000  # never dereferenced


@pytest.fixture(scope="module")
def lib():
    build.build()
    return dsa.lib()


def test_e4m3_rounding_is_torch_s():
    # every half-way point and its neighbours, both signs: torch rounds to nearest even
    v = ref.e4m3_values(np.arange(127))
    mid = (v[:-1] + v[1:]) / 2
    x = np.concatenate([v, mid, np.nextafter(mid, 0), np.nextafter(mid, 1e9)])
    x = np.concatenate([x, -x]).astype(np.float32).astype(np.float64)
    want = torch.from_numpy(x).float().to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(ref.e4m3_round(x), want)


def test_block_exponents():
    assert ref.block_exponent(448.0) == 127 and ref.block_exponent(np.nextafter(448.0, 500)) == 128
    assert ref.block_exponent(0.0) == 87 and ref.block_exponent(1e30) == 167


def test_a_fallen_scale_rounds_only_what_becomes_subnormal():
    # bytes written at one scale and moved to a larger one are those written at
    # the larger one, for every value that is normal there
    rng = np.random.default_rng(0)
    x = rng.uniform(-448, 448, 20000) * 2.0 ** rng.integers(-8, 1, 20000)
    for d in range(1, 9):
        moved = ref.e4m3_round(ref.e4m3_values(ref.e4m3_round(x)) * 2.0 ** -d)
        at_once = ref.e4m3_round(x * 2.0 ** -d)
        normal = np.abs(x) * 2.0 ** -d >= 2.0 ** -6
        assert normal.any() and np.array_equal(moved[normal], at_once[normal])


def append_args(**kw):
    a = dict(K=B, ld_k=512, V=B, ld_v=512, k8=None, ks=None, cu=B, nseq=2, n=5, lens=B, table=B, max_pages=4,
             num_pages=9, Hkv=4, D=128, dI=0, block=64, kc=B, vc=B, exp=B, k8c=None, ksc=None)
    a.update(kw)
    return list(a.values()) + [None]


@pytest.mark.parametrize("kw,want", [
    (dict(nseq=-1), INVALID), (dict(n=-1), INVALID), (dict(max_pages=0), INVALID), (dict(num_pages=0), INVALID),
    (dict(Hkv=0), INVALID), (dict(cu=None), INVALID), (dict(D=96), UNSUPPORTED), (dict(block=8), UNSUPPORTED),
    (dict(block=48), UNSUPPORTED), (dict(num_pages=1 << 25), UNSUPPORTED), (dict(Hkv=1025), UNSUPPORTED),
    (dict(k8=B), INVALID), (dict(k8=B, ks=B, k8c=B, ksc=B, dI=48), UNSUPPORTED), (dict(K=None), INVALID),
    (dict(V=None), INVALID), (dict(lens=None), INVALID), (dict(table=None), INVALID), (dict(exp=None), INVALID),
    (dict(ld_k=511), INVALID), (dict(ld_v=516), INVALID), (dict(K=B + 8), INVALID), (dict(kc=B + 8), INVALID),
    (dict(k8=B + 8, ks=B, k8c=B, ksc=B, dI=64), INVALID), (dict(exp=B + 1), INVALID),
    (dict(max_pages=1 << 25), UNSUPPORTED), (dict(nseq=2 ** 29), UNSUPPORTED), (dict(n=0), OK), (dict(nseq=0, n=0), OK),
])
def test_append_refusals(lib, kw, want):
    assert lib.dsa_kv8_append(*append_args(**kw)) == want


@pytest.mark.parametrize("kw,want", [
    (dict(n=-1), INVALID), (dict(k=0), INVALID), (dict(Hq=30), UNSUPPORTED), (dict(Hq=36), UNSUPPORTED),
    (dict(D=96), UNSUPPORTED), (dict(block=128), UNSUPPORTED), (dict(num_pages=1 << 25), UNSUPPORTED),
    (dict(q=None), INVALID), (dict(idx=None), INVALID), (dict(out=None), INVALID), (dict(out=B + 8), INVALID),
    (dict(q=B + 2), INVALID), (dict(exp=B + 1), INVALID), (dict(kc=B + 16), INVALID), (dict(vc=B + 16), INVALID), (dict(max_pages=0), INVALID),
    (dict(n=2 ** 29), UNSUPPORTED), (dict(k=2 ** 30 + 1), UNSUPPORTED), (dict(n=0), OK),
])
@pytest.mark.parametrize("prefill", [False, True])
def test_attention_refusals(lib, kw, want, prefill):
    a = dict(q=B, kc=B, vc=B, exp=B, block=64, table=B, max_pages=4, num_pages=9, lens=B, idx=B, n=3, Hq=32, Hkv=4,
             D=128, k=64, sm=0.1, out=B)
    a.update(kw)
    v = list(a.values())
    if prefill:
        v[10:10] = [B, 2, 0]   # cu_seqlens, nseq, row_begin
        assert lib.dsa_sparse_gqa_prefill_kv8(*v, None, None) == want
    else:
        assert lib.dsa_sparse_gqa_decode_attention_kv8(*v, None, None) == want


def test_prefill_refuses_bad_sequences(lib):
    head = [B, B, B, B, 64, B, 4, 9, B, B]
    tail = [4, 32, 4, 128, 64, 0.1, B, None, None]
    f = lib.dsa_sparse_gqa_prefill_kv8
    assert f(*head, None, 2, 0, *tail) == INVALID
    assert f(*head, B, 0, 0, *tail) == INVALID
    assert f(*head, B, 2, -1, *tail) == INVALID
    assert f(*head, B, 2, 2 ** 31 - 2, *tail) == INVALID


def test_decode_chain_refusals(lib):
    need = lib.dsa_decode_kv8_workspace_size(3, 200, 64)
    assert need > 0 and lib.dsa_decode_kv8_workspace_size(3, 200, 0) == 0

    def call(q8=B, max_len=200, HI=32, k=64, ws=B, ws_bytes=need, block=64):
        return lib.dsa_sparse_gqa_decode_kv8(B, q8, B, B, B, B, B, B, B, block, B, 4, 9, B, max_len, 3, 32, 4, 128, HI,
                                             64, k, 0.1, ws, ws_bytes, B, None, None)

    assert call(max_len=257) == INVALID        # longer than the block table
    assert call(HI=12) == UNSUPPORTED
    assert call(block=65) == UNSUPPORTED
    assert call(k=0) == INVALID
    assert call(q8=B + 4) == INVALID
    assert call(ws=None) == WORKSPACE and call(ws_bytes=need - 1) == WORKSPACE and call(ws=B + 4) == WORKSPACE


def bufs(ptrs=(B, B), sizes=(128, 6)):
    return (ctypes.c_void_p * len(ptrs))(*ptrs), (ctypes.c_size_t * len(sizes))(*sizes), len(ptrs)


@pytest.mark.parametrize("kw,want", [
    (dict(n=-1), INVALID), (dict(n=1025), UNSUPPORTED), (dict(n_slots=0), INVALID), (dict(max_pages=0), INVALID),
    (dict(num_pages=0), INVALID), (dict(num_pages=1 << 25), UNSUPPORTED), (dict(slots=None), INVALID),
    (dict(table=None), INVALID), (dict(lens=None), INVALID), (dict(refs=None), INVALID), (dict(n=0), OK),
])
def test_pool_refusals(lib, kw, want):
    a = dict(slots=B, other=B, n=3, table=B, n_slots=5, max_pages=4, lens=B, refs=B, num_pages=9)
    a.update(kw)
    v = list(a.values())
    assert lib.dsa_pages_extend(*v, B, None) == want
    assert lib.dsa_pages_fork(*bufs(), v[1], v[0], *v[2:], B, None) == want
    assert lib.dsa_pages_free(v[0], *v[2:], None) == want


def test_page_buffer_refusals(lib):
    f = lib.dsa_pages_copy
    assert f(*bufs(), None, B, 2, 9, None) == INVALID
    assert f(*bufs(), B, B, -1, 9, None) == INVALID
    assert f(*bufs((B, None)), B, B, 2, 9, None) == INVALID
    assert f(*bufs((B, B), (0, 4)), B, B, 2, 9, None) == INVALID
    assert f(*bufs((B, B), ((1 << 24) + 1, 4)), B, B, 2, 9, None) == UNSUPPORTED
    assert f(*bufs([B] * 9, [4] * 9), B, B, 2, 9, None) == UNSUPPORTED
    assert f(None, None, 1, B, B, 2, 9, None) == INVALID
    assert f(*bufs(), B, B, 0, 9, None) == OK
    g = lib.dsa_pages_compact
    need = lib.dsa_pages_compact_workspace_size(9)
    assert need >= 16 and lib.dsa_pages_compact_workspace_size(0) == 0

    def compact(table=B, ws=B, size=need, used=B):
        return g(*bufs(), table, B, 5, 4, B, B, B, 9, B, used, ws, size, None)

    assert compact(table=None) == INVALID and compact(used=None) == INVALID
    assert compact(ws=None) == WORKSPACE and compact(size=need - 1) == WORKSPACE and compact(ws=B + 8) == WORKSPACE


def test_binding_refuses_tensors_of_the_host_and_wrong_shapes():
    kc = torch.zeros(3, 64, 2, 64, dtype=torch.uint8)
    exp = torch.zeros(3, 1, 2, 2, dtype=torch.uint8)
    i32 = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError):
        dsa.kv8_append(torch.zeros(2, 2, 64, dtype=torch.bfloat16), torch.zeros(2, 2, 64, dtype=torch.bfloat16), kc,
                       kc, exp, torch.zeros(2, 1, dtype=torch.int32), i32)
    with pytest.raises(ValueError):
        dsa.pages_copy([kc], i32, i32)
    with pytest.raises(ValueError):
        dsa.pages_copy([], i32, i32)
    with pytest.raises(ValueError):
        dsa.pages_free(i32, torch.zeros(2, 1, dtype=torch.int32), i32, i32)
    with pytest.raises(ValueError):
        dsa.KV8Cache(4, 2, 2, 2, 64, scale_block=8, device="cpu")


def test_plain_pool_keeps_its_counts():
    # the plain pool itself: after any run of calls each page's count is the number of rows that hold it
    rng = np.random.default_rng(3)
    pool = ref.Pool(40, 8, 6)
    for _ in range(200):
        op = rng.integers(4)
        s = rng.integers(0, 8, 3)
        if op == 0:
            pool.extend(s, pool.lens[s] + rng.integers(0, 100, 3))
        elif op == 1:
            pool.fork(s, rng.integers(0, 8, 3))
        elif op == 2:
            pool.free(s[:1])
        else:
            pool.compact()
        held = np.bincount(pool.table[pool.table >= 0], minlength=40)
        assert np.array_equal(held, pool.refs)
        last = [pool.table[i, pool.lens[i] // 64] for i in range(8) if pool.lens[i] % 64]
        assert all(pool.refs[p] == 1 for p in last)   # partly filled pages belong to one sequence
