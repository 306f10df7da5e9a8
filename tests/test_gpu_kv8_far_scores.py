"""Attention over the 8-bit cache with finite scores of extreme size."""
import numpy as np
import pytest
import torch

from sparse_long_context_03_b200 import dsa

pytestmark = pytest.mark.gpu
DEV = "cuda"


def attend(q, k_bytes, v_bytes, exp_k, rows):
    """One sequence of 64 * pages tokens seen whole by `rows` query rows q
    [Hq, D]; k_bytes, v_bytes [tokens, Hkv, D]."""
    n, Hkv, D = k_bytes.shape
    P = n // 64
    kc, vc = (torch.from_numpy(x).view(P, 64, Hkv, D).to(DEV) for x in (k_bytes, v_bytes))
    exp = torch.full((P, 1, Hkv, 2), 127, dtype=torch.uint8, device=DEV)
    exp[..., 0] = exp_k
    q = q.expand(rows, *q.shape[-2:]).contiguous().to(DEV)
    idx = torch.arange(n, dtype=torch.int32, device=DEV).expand(rows, n).contiguous()
    table = torch.arange(P, dtype=torch.int32, device=DEV).expand(rows, P).contiguous()
    lens = torch.full((rows,), n, dtype=torch.int32, device=DEV)
    out, lse = torch.empty_like(q), torch.empty(rows, q.shape[1], device=DEV)
    dsa.sparse_gqa_decode_attention_kv8(q, kc, vc, exp, table, lens, idx, n, 0.125, out, lse)
    return out.double().cpu(), lse.double().cpu()


@pytest.mark.parametrize("rows", [1, 40, 600])
def test_rows_whose_scores_all_lie_far_below_zero(rows):
    # every score is -2^(105 + 6 - 3) = -2^108; the output is the mean of V
    k = np.full((128, 4, 64), 0xB8, np.uint8)             # -1
    v = np.where(np.arange(128)[:, None, None] < 64, 0x40, 0x38).astype(np.uint8) + np.zeros_like(k)   # 2, then 1
    out, lse = attend(torch.full((8, 64), 2.0 ** 105, dtype=torch.bfloat16), k, v, 127, rows)
    assert torch.all(out == 1.5)
    # ln 128 vanishes beside 2^108; log2 e, its product with the scale, the
    # score, the reference and the way back to nats round, 2^-24 each, and ln 2
    assert torch.all((lse / -2.0 ** 108 - 1).abs() <= 8 * 2.0 ** -24)


@pytest.mark.parametrize("rows", [1, 40, 600])
def test_scores_of_zero_beside_those_that_overflow(rows):
    # q is 2^110 in one dim; K there is 0, or -1 at a scale of 2^40: scores of 0
    # and of -2^147, which fp32 does not hold and whose weight is 0
    k = np.zeros((128, 4, 64), np.uint8)
    k[::2, :, 0] = 0xB8
    v = np.where(np.arange(128)[:, None, None] % 4 == 1, 0x40, 0x38).astype(np.uint8) + np.zeros_like(k)
    v[::2] = 0x7E                                         # 448, where the weight is 0
    q = torch.zeros(8, 64, dtype=torch.bfloat16)
    q[:, 0] = 2.0 ** 110
    out, lse = attend(q, k, v, 167, rows)
    assert torch.all(out == 1.5)
    # ln 64 by way of log2: its result and ln 2 round, and the approximation's last bits
    assert torch.all((lse - np.log(64)).abs() <= 2.0 ** -20)
