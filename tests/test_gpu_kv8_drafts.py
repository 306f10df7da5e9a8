"""Several query tokens of one cached sequence: their keys are selected by the
decode chain with a batch row per token, and attended by the packed form."""
import numpy as np
import pytest
import torch

import kv8_reference as ref
from sparse_long_context_03_b200 import dsa, inputs

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("lens,new", [([5000], [5]), ([2047, 70, 9000], [8, 1, 3])])
def test_rows_of_a_repeated_table_select_for_packed_query_rows(lens, new):
    cfg = inputs.config(3)
    rng = np.random.default_rng(len(lens))
    d = inputs.decode_inputs(cfg, seq_lens=lens, seed=31, device=DEV)
    P, n = d["num_pages"], sum(new)
    kc, vc = (rng.integers(0, 127, (P, 64, cfg.Hkv, cfg.D)).astype(np.uint8) for _ in range(2))
    exp = rng.integers(112, 119, (P, 2, cfg.Hkv, 2)).astype(np.uint8)
    cache = [torch.from_numpy(x).to(DEV) for x in (kc, vc, exp)]
    cu = np.concatenate([[0], np.cumsum(new)])
    seq = np.repeat(np.arange(len(lens)), new)
    pos = np.array(lens)[seq] - np.array(new)[seq] + np.arange(n) - cu[seq]
    gen = torch.Generator(device=DEV)
    gen.manual_seed(32)
    q = torch.randn(n, cfg.Hq, cfg.D, generator=gen, device=DEV).to(torch.bfloat16)
    q8, sq = inputs.quantize_e4m3_per_token(torch.randn(n, cfg.HI, cfg.dI, generator=gen, device=DEV))
    w = torch.rand(n, cfg.HI, generator=gen, device=DEV)
    table = d["block_table"][torch.from_numpy(seq).to(DEV)].contiguous()
    seen = torch.from_numpy(pos + 1).to(torch.int32).to(DEV)
    most = d["max_seq_len"]

    def chain(r0, r1):
        ws = torch.empty(dsa.decode_kv8_workspace_size(r1 - r0, most, cfg.k), dtype=torch.uint8, device=DEV)
        out, idx = torch.empty_like(q[r0:r1]), torch.empty(r1 - r0, cfg.k, dtype=torch.int32, device=DEV)
        dsa.sparse_gqa_decode_kv8(q[r0:r1], q8[r0:r1], sq[r0:r1], w[r0:r1], d["k8_cache"], d["sk_cache"], *cache,
                                  table[r0:r1], seen[r0:r1], most, cfg.k, cfg.sm_scale, ws, out, idx_out=idx)
        return out, idx

    out, idx = chain(0, n)
    O, lse = torch.empty_like(q), torch.empty(n, cfg.Hq, device=DEV)
    dsa.sparse_gqa_prefill_kv8(q, *cache, d["block_table"], torch.tensor(lens, dtype=torch.int32, device=DEV), idx,
                               torch.from_numpy(cu).to(torch.int32).to(DEV), 0, n, cfg.k, cfg.sm_scale, O, lse)
    picks = idx.cpu().numpy()
    for r in range(n):
        assert torch.equal(chain(r, r + 1)[1][0], idx[r])
        sel = picks[r][picks[r] >= 0]
        assert len(np.unique(sel)) == len(sel) == min(cfg.k, pos[r] + 1) and sel.max() <= pos[r]
    want = ref.attention(q.double().cpu().numpy(), kc, vc, exp, d["block_table"].cpu().numpy(), picks, seq, pos,
                         float(np.float32(cfg.sm_scale)))
    for o in (out, O):
        assert not (np.abs(o.double().cpu().numpy() - want[0]) > want[2]).any()
    assert np.all(np.abs(lse.double().cpu().numpy() - want[1]) <= want[3])
