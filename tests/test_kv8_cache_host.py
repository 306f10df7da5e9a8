"""KV8Cache's own refusals.  Nothing here needs a GPU or launches anything."""
import pytest
import torch

from sparse_long_context_03_b200 import dsa


def test_a_cache_of_indexer_keys_takes_no_tokens_without_them():
    # the page's earlier keys would stay, and a later decode would select by them
    c = dsa.KV8Cache(4, 2, 2, 2, 64, dI=32, device="cpu")
    kv = torch.zeros(2, 2, 64, dtype=torch.bfloat16)
    for kw in (dict(), dict(k_scale=torch.ones(2))):
        with pytest.raises(ValueError, match="indexer keys"):
            c.append(kv, kv, **kw)
    with pytest.raises(ValueError, match="go together|CUDA"):
        c.append(kv, kv, k8=torch.zeros(2, 32, dtype=torch.uint8))
    # a cache without them takes none
    with pytest.raises(ValueError, match="indexer keys"):
        dsa.KV8Cache(4, 2, 2, 2, 64, device="cpu").append(kv, kv, k8=torch.zeros(2, 32, dtype=torch.uint8),
                                                          k_scale=torch.ones(2))
