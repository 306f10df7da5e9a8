"""Granting pages to entries that together want more than 31 bits hold."""
import pytest
import torch

from sparse_long_context_03_b200 import dsa

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("P", [3000, 5000])
def test_sums_of_wanted_pages_beyond_31_bits(P):
    # 1022 entries that want 2^21 + 2^13 pages each, between two that want few:
    # the first is served, the last comes after them and is refused as they are
    n, most = 1025, 2 ** 21 + 2 ** 13
    table = torch.full((n, most), -1, dtype=torch.int32, device=DEV)
    lens = torch.zeros(n, dtype=torch.int32, device=DEV)
    refs = torch.zeros(P, dtype=torch.int32, device=DEV)
    refs[1] = 1
    for order in (torch.arange(1024), torch.arange(1024, 0, -1)):
        slots = order.to(torch.int32).to(DEV)
        to = torch.full((1024,), 64 * most, dtype=torch.int32, device=DEV)
        to[0], to[-1] = 130, 1
        status = torch.full((1024,), 9, dtype=torch.int32, device=DEV)
        dsa.pages_extend(slots, to, table, lens, refs, status)
        assert status.tolist() == [0] + [1] * 1023
        s = int(slots[0])
        assert int(lens[s]) == 130 and int(lens.sum()) == 130
        free = [0, 2, 3]
        assert table[s, :4].tolist() == free + [-1] and int((table >= 0).sum()) == 3
        assert refs[:5].tolist() == [1, 1, 1, 1, 0] and int(refs.sum()) == 4
        dsa.pages_free(slots[:1], table, lens, refs)
    assert int(refs.sum()) == 1 and not bool((table >= 0).any())
