"""AttentionMixer's buffers, on the CPU: nothing is launched."""
from __future__ import annotations

import pytest

import quantized_moe_expert_amd as m

FAKE = 0x10000


def mixer(hq, hkv, max_tokens, max_seqs, d=64, page=16, cols=64):
    cache = m.KVCache(hkv, d, page, cols, cols * max_seqs, FAKE, FAKE, FAKE, FAKE)
    w_in = m.LinearWeights(256, (hq + 2 * hkv) * d, m.LINEAR_BF16, FAKE, None, None)
    w_out = m.LinearWeights(hq * d, 256, m.LINEAR_BF16, FAKE, None, None)
    return m.AttentionMixer(w_in, w_out, hq, cache, max_tokens, max_seqs, device="cpu"), cache


@pytest.mark.parametrize("hq,hkv", [(1, 1), (3, 1), (5, 1), (6, 2), (7, 1), (9, 1), (11, 1), (12, 4), (15, 1), (16, 1), (17, 1),
                                    (18, 1), (20, 1), (31, 1), (40, 2), (128, 1)])
@pytest.mark.parametrize("max_tokens,max_seqs", [(1, 1), (2, 2), (3, 4), (16, 5), (17, 17), (64, 20), (300, 6), (9, 40)])
def test_workspace_fits_every_batch(hq, hkv, max_tokens, max_seqs):
    """Also where the query heads of a head of the cache do not divide 16."""
    lay, cache = mixer(hq, hkv, max_tokens, max_seqs)
    for n in range(1, max_seqs + 1):
        for t in range(1, max_tokens + 1):
            assert m.attention_workspace_size(t, n, hq, cache) <= lay.ws.numel(), (t, n)


def test_a_cache_needs_kv_cache_struct():
    """A KVCache of the caller's own has no number of sequences and no device."""
    from quantized_moe_expert_amd import _backbone
    cache = m.KVCache(2, 64, 16, 4, 8, FAKE, FAKE, FAKE, FAKE)
    with pytest.raises(ValueError, match="kv_cache_struct"):
        _backbone._cached(cache, None, 0)
