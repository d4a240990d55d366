"""Pins of the single-token serving oracle: attention against brute force and
its invariants, eviction against a direct reading of the rule, sampling
against the distributions that its filters define."""
import ctypes

import numpy as np
import pytest

from oracle import serving as S
from speculative_decoding_block_gb300 import binding


def test_attention_is_a_softmax_mean_and_joins_by_lse():
    rng = np.random.default_rng(0)
    q, k, v = rng.normal(size=(6, 8)), rng.normal(size=(13, 2, 8)), rng.normal(size=(13, 2, 8))
    out, lse, w = S.decode_attention(q, k, v)
    for hq in range(6):
        s = np.array([q[hq] @ k[i, hq // 3] for i in range(13)]) / np.sqrt(8)
        assert np.allclose(out[hq], sum(np.exp(s[i]) * v[i, hq // 3] for i in range(13)) / np.exp(s).sum())
    assert np.allclose(w.sum(1), 3.0)
    # two parts of the cache, joined by their lse, give the whole
    a, la, _ = S.decode_attention(q, k[:5], v[:5])
    b, lb, _ = S.decode_attention(q, k[5:], v[5:])
    z = np.logaddexp(la, lb)
    assert np.allclose(z, lse)
    assert np.allclose(a * np.exp(la - z)[:, None] + b * np.exp(lb - z)[:, None], out)


def test_attention_window_and_empty_set():
    rng = np.random.default_rng(1)
    q, k, v = rng.normal(size=(2, 4)), rng.normal(size=(9, 1, 4)), rng.normal(size=(9, 1, 4))
    out, lse, w = S.decode_attention(q, k[:8], v[:8], k[8], v[8], window=3)
    ref, rl, _ = S.decode_attention(q, k[6:], v[6:])
    assert np.allclose(out, ref) and np.allclose(lse, rl) and not w[:, :6].any()
    out, lse, w = S.decode_attention(q, k[:0], v[:0])
    assert not out.any() and np.isneginf(lse).all() and w.shape == (1, 0)
    out, _, _ = S.decode_attention(q, k[:0], v[:0], k[0], v[0])
    assert np.allclose(out, v[0])


def test_eviction_rule_on_a_hand_built_row():
    score = [9.0, 1.0, 5.0, np.nan, 5.0, 0.0, 7.0, 5.0, 2.0, 0.0]
    assert S.evict_rows(score, 10, 6, sinks=1, recent=2).tolist() == [0, 2, 4, 6, 8, 9]  # two of the three fives
    assert S.evict_rows(score, 10, 10).tolist() == list(range(10))
    assert S.evict_rows(score, 4, 6).tolist() == [0, 1, 2, 3]
    assert S.evict_rows(score, 10, 3, sinks=1, recent=2).tolist() == [0, 8, 9]
    assert S.evict_rows([np.nan, -1.0, np.nan], 3, 2).tolist() == [0, 1]  # NaN below every number


def test_filters_are_prefixes_of_the_falling_order():
    x = np.log([0.4, 0.1, 0.3, 0.15, 0.05])
    assert np.nonzero(S.filtered(x, 1.0, top_k=2))[0].tolist() == [0, 2]
    assert np.nonzero(S.filtered(x, 1.0, top_p=0.71))[0].tolist() == [0, 2, 3]
    assert np.nonzero(S.filtered(x, 1.0, min_p=0.3))[0].tolist() == [0, 2, 3]
    assert np.nonzero(S.filtered(x, 1.0, top_k=3, top_p=0.5))[0].tolist() == [0, 2]  # mass of the three: 0.85
    assert np.nonzero(S.filtered(np.zeros(4), 1.0, top_p=0.5))[0].tolist() == [0, 1]  # equals: lowest ids
    assert np.nonzero(S.filtered(x, 1.0, top_p=0.0))[0].tolist() == [0]


def test_samples_follow_the_filtered_distribution():
    rng = np.random.default_rng(3)
    x = rng.normal(size=40) * 2
    w = S.filtered(x, 0.8, top_k=12, top_p=0.95, min_p=0.01)
    p = w / w.sum()
    n = 4000
    toks = np.array([S.sample_logits(x, (i + 0.5) / n, 0.8, 12, 0.95, 0.01)[0] for i in range(n)])
    # evenly spaced uniforms: each token's count is within one of its share
    counts = np.bincount(toks, minlength=40)
    assert np.abs(counts - p * n).max() <= 1.0 + 1e-9


def test_sampling_edge_rows():
    assert S.sample_logits([np.nan, -np.inf], 0.5) == (-1, -np.inf, np.inf)
    assert S.sample_logits([1.0, 3.0, 3.0], 0.9, T=0.0)[:2] == (1, 0.0)
    tok, lp, _ = S.sample_logits([np.inf, 0.0, np.inf], 0.75)
    assert tok == 2 and np.isclose(lp, np.log(0.5))


@pytest.mark.parametrize("call", [
    lambda L: L.vsd_kv_pools(None, None, None),
    lambda L: L.vsd_decode_attention(None, None, 0, 1, None, None, None, None, 0, None, None, None, None),
    lambda L: L.vsd_kv_evict(None, 1, None, None, None, 16, 0, 0, None, None),
    lambda L: L.vsd_sample_logits(None, 1, 8, 8, None, None, None, None, None, None, None, None),
])
def test_null_arguments_are_refused_without_a_gpu(call):
    L = binding.lib()
    assert call(L) == binding.VSD_ERR_ARG
    assert b"NULL" in L.vsd_last_error()


def test_sampling_sizes_are_refused_without_a_gpu():
    """Sizes are checked before anything touches a device (the pointers are never read)."""
    L = binding.lib()
    p = ctypes.c_void_p(4096)

    def call(rows, vocab, ld):
        return L.vsd_sample_logits(p, rows, vocab, ld, None, None, None, None, p, p, None, None)

    assert call(-1, 8, 8) == binding.VSD_ERR_ARG
    assert call(1, 0, 8) == binding.VSD_ERR_ARG
    assert call(1, 8, 7) == binding.VSD_ERR_ARG
    assert call(1, (1 << 18) + 1, 1 << 20) == binding.VSD_ERR_UNSUPPORTED
    assert call(0, 8, 8) == binding.VSD_OK


def test_tensors_of_another_device_are_refused():
    class Fake:
        def __init__(self, device):
            self.device = device

        def get_device(self):
            return self.device

    binding._on_device(0, q=Fake(0), lse=None)
    with pytest.raises(ValueError, match="out is on device 1"):
        binding._on_device(0, q=Fake(0), out=Fake(1))
    with pytest.raises(ValueError, match="u is on device -1"):  # a host tensor
        binding._on_device(0, u=Fake(-1))
