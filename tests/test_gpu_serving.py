"""GPU parity of the single-token serving operators (decode attention, cache
eviction, token sampling) against the float64 oracle, at the sizes and masks
where they can go wrong, and a run of them together."""
import ctypes

import numpy as np
import pytest
import torch

from oracle import serving as S
from tests.gpu_helpers import gpu, require_gpu
from workload import gen

pytestmark = gpu

_models = {}


def tiny_model(B, layers, n_q, n_kv, hd, max_positions=8192):
    """A model object of this head layout; its weights are never used."""
    key = (layers, n_q, n_kv, hd, max_positions)
    if key not in _models:
        H, F, V = 64, 64, 64
        mats = [(n_q * hd, H), (n_kv * hd, H), (n_kv * hd, H), (H, n_q * hd), (F, H), (F, H), (H, F)]
        w = [torch.zeros(s, dtype=torch.bfloat16, device="cuda") for s in mats]
        cfg = B.ModelConfig(layers, H, n_q, n_kv, hd, F, V, 1e4, 1e-6, 1, 0, 0, max_positions)
        embed = torch.zeros((V, H), dtype=torch.bfloat16, device="cuda")
        _models[key] = B.vsd_model_create(cfg, embed, [B.weight_entry("bf16", x) for x in w] * layers)
        torch.cuda.synchronize()
    return _models[key]


def bf16(shape, std, *tag):
    return gen.normal_bf16(shape, std, *tag).cuda()


def f64(t):
    return t.detach().double().cpu().numpy()


class Cache:
    """A cache over shuffled pages, every row of its pools set to `fill`, then the requests' rows to random values."""

    def __init__(self, B, layers, n_q, n_kv, hd, lens, max_tokens, fill=float("nan"), tag="c", spare=3):
        self.B, self.layers, self.n_q, self.n_kv, self.hd = B, layers, n_q, n_kv, hd
        self.lens, self.max_tokens = list(lens), max_tokens
        n = len(lens)
        self.model = tiny_model(B, layers, n_q, n_kv, hd)
        ppr = -(-max_tokens // 16)
        self.kv = B.vsd_kv_create(self.model, n, max_tokens, 16, n * ppr + spare)
        table = gen._rng("pt", tag).permutation(self.kv.num_pages)[: n * ppr].astype(np.int32)
        self.table = table.reshape(n, ppr)
        B.vsd_kv_set_page_table(self.kv, torch.tensor(table, device="cuda"))
        self.k_pool, self.v_pool = B.vsd_kv_pools(self.kv)
        assert self.k_pool.shape == (layers, self.kv.num_pages, n_kv, 16, hd)
        self.k_pool.fill_(fill)
        self.v_pool.fill_(fill)
        self.k, self.v = [], []
        for b, L in enumerate(self.lens):
            L = max(L, 0)
            k = bf16((layers, L, n_kv, hd), 1.0, tag, "k", b)
            v = bf16((layers, L, n_kv, hd), 1.0, tag, "v", b)
            if L:
                B.vsd_kv_write(self.kv, b, 0, k, v)
            self.k.append(k)
            self.v.append(v)
        self.seq = torch.tensor(self.lens, dtype=torch.int32, device="cuda")

    def rows(self, b, n):
        k = torch.empty((self.layers, n, self.n_kv, self.hd), dtype=torch.bfloat16, device="cuda")
        v = torch.empty_like(k)
        if n:
            self.B.vsd_kv_read(self.kv, b, 0, k, v)
        return k, v


def attention_tolerance(q, k, v, ref, n):
    """Bound of |out - ref| per element.

    The scores are float32 sums of hd exact products: off by at most (hd + 4) 2^-24 sum|q_i k_i| scale, which is a relative
    error of p (and of its normaliser).  p enters the product with 16 bits (2^-16), exponentials and the n-term sums add
    2^-20 + n 2^-24; the output is rounded once to f16 (2^-11, or half a subnormal step, 2^-25)."""
    hd = q.shape[-1]
    g = q.shape[0] // k.shape[1]
    mag = max(float((np.abs(k[:, h]) @ np.abs(q[h * g:(h + 1) * g]).T).max()) for h in range(k.shape[1])) / np.sqrt(hd)
    eps = (hd + 4) * 2.0 ** -24 * mag + 2.0 ** -16 + 2.0 ** -20 + n * 2.0 ** -24
    return 2.0 ** -11 * np.abs(ref) + 2.0 ** -25 + 2 * eps * np.abs(v).max(), eps


def check_attention(c, layer, append, window, use_score, use_lse=True, stream=None):
    B, n_b = c.B, len(c.lens)
    q = bf16((n_b, c.n_q, c.hd), 2.0, "q", layer)
    kn = bf16((n_b, c.n_kv, c.hd), 1.0, "kn", layer) if append else None
    vn = bf16((n_b, c.n_kv, c.hd), 1.0, "vn", layer) if append else None
    out = torch.full((n_b, c.n_q * c.hd), float("nan"), dtype=torch.float16, device="cuda")
    lse = torch.full((n_b, c.n_q), float("nan"), device="cuda") if use_lse else None
    score = torch.rand((n_b, c.n_kv, c.max_tokens), device="cuda", generator=torch.Generator("cuda").manual_seed(5)) if use_score else None
    before = score.clone() if use_score else None
    kp, vp = c.k_pool.clone(), c.v_pool.clone()
    B.vsd_decode_attention(c.model, c.kv, layer, n_b, c.seq, q, kn, vn, out, window=window, score=score, lse=lse)
    torch.cuda.synchronize()
    assert B.vsd_get_device_status(c.kv) == 0
    want = before.double().cpu().numpy() if use_score else None
    for b, L in enumerate(c.lens):
        got = f64(out[b]).reshape(c.n_q, c.hd)
        if L < 0:
            assert not got.any()
            if use_lse:
                assert torch.isneginf(lse[b]).all()
            continue
        k, v = f64(c.k[b][layer]), f64(c.v[b][layer])
        ref, rl, w = S.decode_attention(f64(q[b]), k, v, f64(kn[b]) if append else None, f64(vn[b]) if append else None, window)
        n = L + (1 if append else 0)
        if n == 0:
            assert not got.any() and (not use_lse or torch.isneginf(lse[b]).all())
            continue
        ka = np.concatenate([k, f64(kn[b])[None]]) if append else k
        va = np.concatenate([v, f64(vn[b])[None]]) if append else v
        tol, eps = attention_tolerance(f64(q[b]), ka, va, ref, n)
        assert (np.abs(got - ref) <= tol).all(), (b, L, np.abs(got - ref).max(), tol.min())
        if use_lse:
            assert (np.abs(f64(lse[b]) - rl) <= eps + 2.0 ** -22 * np.maximum(1.0, np.abs(rl))).all(), (b, L)
        if use_score:
            lo = max(0, n - window) if window else 0
            if append:
                want[b, :, L] = 0.0
            want[b, :, lo:n] += w[:, lo:]
            err = np.abs(f64(score[b]) - want[b])
            assert (err[:, :n] <= 2 * eps * w + 2.0 ** -22 * (want[b, :, :n] + 1e-30)).all(), (b, L, err.max())
            # entries of rows that were not attended to keep their bits
            assert torch.equal(score[b, :, n:], before[b, :, n:]) and torch.equal(score[b, :, :lo], before[b, :, :lo])
        if append:  # the new row joined the cache; nothing else changed
            p, r = c.table[b, L // 16], L % 16
            kp[layer, p, :, r] = kn[b]
            vp[layer, p, :, r] = vn[b]
    assert torch.equal(c.k_pool.view(torch.int16), kp.view(torch.int16))
    assert torch.equal(c.v_pool.view(torch.int16), vp.view(torch.int16))
    return out, lse, score


HEADS = [(4, 2, 64), (14, 2, 64), (8, 2, 128), (7, 1, 128), (3, 3, 64)]


# the most rows that a cache has room for decides how a call's work is dealt out: a CTA per pair, or even shares and a join
ROOMS = [1008, 8000]


@pytest.mark.parametrize("room", ROOMS)
@pytest.mark.parametrize("append", [True, False])
@pytest.mark.parametrize("heads", HEADS)
def test_decode_attention_matches_oracle_over_lengths(heads, append, room):
    """Lengths around pages and tiles, an empty request and an idle slot; rows behind the lengths hold NaN."""
    B = require_gpu()
    lens = [0, 1, 15, 16, 17, 31, 32, 33, 63, 65, 127, 130, -1, 500, 1007]
    c = Cache(B, 2, *heads, lens, room, tag=f"len{heads}{append}")
    check_attention(c, 1, append, 0, True)


@pytest.mark.parametrize("window", [1, 5, 16, 33, 100, 5000, 4000])
@pytest.mark.parametrize("heads", [(14, 2, 64), (8, 2, 128)])
def test_decode_attention_window(heads, window):
    B = require_gpu()
    lens = [0, 4, 16, 31, 48, 100, 101, 999] + ([7990, 4100] if window == 4000 else [])
    c = Cache(B, 1, *heads, lens, 8000 if window == 4000 else 1000, tag=f"win{heads}{window == 4000}")
    # infinities in every row that the window leaves out
    for b, L in enumerate(lens):
        for i in range(0, max(0, L + 1 - window)):
            c.k_pool[0, c.table[b, i // 16], :, i % 16] = float("inf")
            c.v_pool[0, c.table[b, i // 16], :, i % 16] = float("-inf")
    check_attention(c, 0, True, window, True)


@pytest.mark.parametrize("score,lse", [(False, True), (True, False), (False, False)])
def test_decode_attention_optional_outputs(score, lse):
    B = require_gpu()
    c = Cache(B, 1, 14, 2, 64, [300, 77], 400, tag="opt")
    check_attention(c, 0, True, 0, score, lse)


@pytest.mark.parametrize("heads,L", [((14, 2, 64), 8001), ((4, 1, 128), 6143), ((4, 4, 64), 7)])
def test_decode_attention_one_request(heads, L):
    """Few (request, KV head) pairs: the cache's length is what the work is split over."""
    B = require_gpu()
    c = Cache(B, 1, *heads, [L], 8100, tag=f"one{heads}")
    check_attention(c, 0, True, 0, True)


@pytest.mark.parametrize("room", [100, 2000])
@pytest.mark.parametrize("n_b", [40, 76, 200])
def test_decode_attention_many_requests(n_b, room):
    B = require_gpu()
    lens = [int(x) for x in gen._rng("many", n_b).integers(0, 90, n_b)]
    c = Cache(B, 1, 14, 2, 64, lens, room, tag="many")
    check_attention(c, 0, True, 0, True)


def test_decode_attention_of_a_very_long_context():
    """One KV head's 100,001 rows over every warp of the grid: over a thousand records to join."""
    B = require_gpu()
    L, n_q, n_kv, hd = 100_001, 7, 1, 64
    model = tiny_model(B, 1, n_q, n_kv, hd, 131072)
    kv = B.vsd_kv_create(model, 1, 100_100)
    kp, vp = B.vsd_kv_pools(kv)
    g = torch.Generator("cuda").manual_seed(1)
    kp.normal_(generator=g)
    vp.normal_(generator=g)
    k = kp[0].permute(1, 0, 2, 3).reshape(n_kv, -1, hd)[:, :L].transpose(0, 1)
    v = vp[0].permute(1, 0, 2, 3).reshape(n_kv, -1, hd)[:, :L].transpose(0, 1)
    q, kn, vn = bf16((1, n_q, hd), 2.0, "lq"), bf16((1, n_kv, hd), 1.0, "lk"), bf16((1, n_kv, hd), 1.0, "lv")
    ref, rl, w = S.decode_attention(f64(q[0]), f64(k), f64(v), f64(kn[0]), f64(vn[0]))
    seq = torch.tensor([L], dtype=torch.int32, device="cuda")
    out = torch.empty((1, n_q * hd), dtype=torch.float16, device="cuda")
    lse = torch.empty((1, n_q), device="cuda")
    score = torch.zeros((1, n_kv, 100_100), device="cuda")
    B.vsd_decode_attention(model, kv, 0, 1, seq, q, kn, vn, out, score=score, lse=lse)
    torch.cuda.synchronize()
    assert B.vsd_get_device_status(kv) == 0
    tol, eps = attention_tolerance(f64(q[0]), f64(k), f64(v), ref, L + 1)
    assert (np.abs(f64(out[0]).reshape(n_q, hd) - ref) <= tol).all()
    assert np.abs(f64(lse[0]) - rl).max() <= eps + 2.0 ** -22 * np.abs(rl).max()
    assert (np.abs(f64(score[0])[:, : L + 1] - w) <= (2 * eps + 2.0 ** -22) * w + 1e-30).all()


def test_decode_attention_offsets_beyond_32_bits():
    """Pages whose offsets in the pool pass 2^31 elements."""
    B = require_gpu()
    layers, n_q, n_kv, hd, T = 2, 8, 8, 128, 65536
    model = tiny_model(B, layers, n_q, n_kv, hd, 131072)
    kv = B.vsd_kv_create(model, 17, T)
    kp, vp = B.vsd_kv_pools(kv)
    assert kp.numel() > 2 ** 31
    L = 200
    k, v = bf16((layers, L, n_kv, hd), 1.0, "bk"), bf16((layers, L, n_kv, hd), 1.0, "bv")
    b = 16
    for i in range(-(-L // 16)):  # identity page table: the last slot's pages
        page = b * kv.pages_per_req + i
        n = min(16, L - 16 * i)
        kp[:, page, :, :n] = k[:, 16 * i: 16 * i + n].transpose(1, 2)
        vp[:, page, :, :n] = v[:, 16 * i: 16 * i + n].transpose(1, 2)
    seq = torch.tensor([-1] * b + [L], dtype=torch.int32, device="cuda")
    q = bf16((17, n_q, hd), 2.0, "bq")
    kn, vn = bf16((17, n_kv, hd), 1.0, "bkn"), bf16((17, n_kv, hd), 1.0, "bvn")
    out = torch.empty((17, n_q * hd), dtype=torch.float16, device="cuda")
    B.vsd_decode_attention(model, kv, 1, 17, seq, q, kn, vn, out)
    ref, _, _ = S.decode_attention(f64(q[b]), f64(k[1]), f64(v[1]), f64(kn[b]), f64(vn[b]))
    tol, _ = attention_tolerance(f64(q[b]), f64(k[1]), f64(v[1]), ref, L + 1)
    assert (np.abs(f64(out[b]).reshape(n_q, hd) - ref) <= tol).all()
    assert torch.equal(kp[1, b * kv.pages_per_req + L // 16, :, L % 16], kn[b])
    # eviction at the same offsets
    score = torch.rand((layers, 17, n_kv, T), device="cuda", generator=torch.Generator("cuda").manual_seed(2))
    host = score[:, b].cpu().numpy()
    new = torch.empty_like(seq)
    B.vsd_kv_evict(kv, 17, seq, new, score, 64, sinks=2, recent=10)
    torch.cuda.synchronize()
    assert B.vsd_get_device_status(kv) == 0
    assert new.tolist() == [-1] * b + [64]
    for l in range(layers):
        for h in (0, n_kv - 1):
            rows = S.evict_rows(host[l, h], L, 64, 2, 10)
            got = kp[l, b * kv.pages_per_req: b * kv.pages_per_req + 4, h].reshape(-1, hd)
            assert torch.equal(got, k[l, torch.tensor(rows, device="cuda"), h])


@pytest.mark.parametrize("room", [112, 8000])
def test_decode_attention_rejects_bad_requests_and_spares_the_others(room):
    B = require_gpu()
    c = Cache(B, 1, 14, 2, 64, [100, 50, 40, 60], room, fill=0.0, tag="bad")
    table = c.table.copy()
    table[1, 2] = c.kv.num_pages       # a page of request 1's rows [32, 48)
    table[2, 40 // 16 + 1] = -5        # not among request 2's rows [0, 41)
    B.vsd_kv_set_page_table(c.kv, torch.tensor(table.reshape(-1), device="cuda"))
    assert B.vsd_get_device_status(c.kv) == B.VSD_DEV_BAD_PAGE
    seq = torch.tensor([room, 50, 40, 60], dtype=torch.int32, device="cuda")  # request 0: no room for its new row
    q, kn, vn = bf16((4, 14, 64), 2.0, "rq"), bf16((4, 2, 64), 1.0, "rk"), bf16((4, 2, 64), 1.0, "rv")
    out = torch.full((4, 14 * 64), float("nan"), dtype=torch.float16, device="cuda")
    lse = torch.full((4, 14), float("nan"), device="cuda")
    score = torch.ones((4, 2, room), device="cuda")
    kp = c.k_pool.clone()
    B.vsd_decode_attention(c.model, c.kv, 0, 4, seq, q, kn, vn, out, score=score, lse=lse)
    torch.cuda.synchronize()
    assert B.vsd_get_device_status(c.kv) == B.VSD_DEV_BAD_PAGE | B.VSD_DEV_BAD_SEQLEN
    assert not out[:2].any() and torch.isneginf(lse[:2]).all() and (score[:2] == 1).all()
    for b, L in ((2, 40), (3, 60)):
        ref, _, _ = S.decode_attention(f64(q[b]), f64(c.k[b][0]), f64(c.v[b][0]), f64(kn[b]), f64(vn[b]))
        tol, _ = attention_tolerance(f64(q[b]), f64(c.k[b][0]), f64(c.v[b][0]), ref, L + 1)
        assert (np.abs(f64(out[b]).reshape(14, 64) - ref) <= tol).all()
        kp[0, c.table[b, L // 16], :, L % 16] = kn[b]
    assert torch.equal(c.k_pool, kp)


@pytest.mark.parametrize("append", [True, False])
@pytest.mark.parametrize("room", [112, 8000])
def test_decode_attention_rejects_lengths_at_the_type_s_ends(room, append):
    """2^31 - 1 rows and one more do not wrap around to a valid length."""
    B = require_gpu()
    c = Cache(B, 1, 14, 2, 64, [0, 0, 40], room, fill=0.0, tag="ends")
    seq = torch.tensor([2 ** 31 - 1, -2 ** 31, 40], dtype=torch.int32, device="cuda")
    q, kn, vn = bf16((3, 14, 64), 2.0, "eq"), bf16((3, 2, 64), 1.0, "ek"), bf16((3, 2, 64), 1.0, "ev")
    out = torch.full((3, 14 * 64), float("nan"), dtype=torch.float16, device="cuda")
    lse = torch.full((3, 14), float("nan"), device="cuda")
    score = torch.ones((3, 2, room), device="cuda")
    kp = c.k_pool.clone()
    B.vsd_decode_attention(c.model, c.kv, 0, 3, seq, q, kn if append else None, vn if append else None, out, score=score, lse=lse)
    torch.cuda.synchronize()
    assert B.vsd_get_device_status(c.kv) == B.VSD_DEV_BAD_SEQLEN
    assert not out[:2].any() and torch.isneginf(lse[:2]).all() and (score[:2] == 1).all()
    assert torch.isfinite(lse[2]).all()
    if append:
        kp[0, c.table[2, 40 // 16], :, 40 % 16] = kn[2]
    assert torch.equal(c.k_pool, kp)


def test_first_calls_of_a_cache_can_be_captured():
    """A new cache's first calls, without and with scores, inside a capture."""
    B = require_gpu()
    c = Cache(B, 1, 4, 2, 64, [30], 64, fill=0.0, tag="first")
    q, kn, vn = bf16((1, 4, 64), 2.0, "fq"), bf16((1, 2, 64), 1.0, "fk"), bf16((1, 2, 64), 1.0, "fv")
    out, again = (torch.zeros((1, 256), dtype=torch.float16, device="cuda") for _ in range(2))
    score = torch.zeros((1, 2, 64), device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        B.vsd_decode_attention(c.model, c.kv, 0, 1, c.seq, q, kn, vn, out)
        B.vsd_decode_attention(c.model, c.kv, 0, 1, c.seq, q, kn, vn, again, score=score)
    graph.replay()
    torch.cuda.synchronize()
    assert out.any() and torch.equal(out, again) and not score[:, :, 31:].any()
    # 4 query heads' weights over 31 rows: each KV head's two sum to 2, of 62 terms within 2^-16 (of the weights' own bound)
    assert (score.sum(-1) - 2).abs().max() < 2 * (2 ** -16 + 62 * 2 ** -24)


@pytest.mark.parametrize("room", [1600, 8000])
def test_decode_attention_graph_replay_streams_and_repeat(room):
    """Captured and replayed, on another stream: the same bits."""
    B = require_gpu()
    c = Cache(B, 1, 14, 2, 64, [700, 90, 1500], room, tag="graph")
    n_b = 3
    q, kn, vn = bf16((n_b, 14, 64), 2.0, "gq"), bf16((n_b, 2, 64), 1.0, "gk"), bf16((n_b, 2, 64), 1.0, "gv")

    def call(stream=None):
        out = torch.empty((n_b, 14 * 64), dtype=torch.float16, device="cuda")
        score = torch.zeros((n_b, 2, room), device="cuda")
        B.vsd_decode_attention(c.model, c.kv, 0, n_b, c.seq, q, kn, vn, out, score=score, stream=stream)
        return out, score

    first = call()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        second = call()
    side.synchronize()
    out, score = torch.empty_like(first[0]), torch.zeros_like(first[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        B.vsd_decode_attention(c.model, c.kv, 0, n_b, c.seq, q, kn, vn, out, score=score)
    score.zero_()
    graph.replay()
    torch.cuda.synchronize()
    for o, s in (second, (out, score)):
        assert torch.equal(o, first[0]) and torch.equal(s, first[1])
    graph.replay()  # a second token's worth: the weights add up
    torch.cuda.synchronize()
    assert torch.equal(out, first[0])
    new = torch.zeros_like(score, dtype=torch.bool)
    for b, L in enumerate(c.lens):
        new[b, :, L] = True
    assert torch.equal(score[~new], (first[1] * 2)[~new]) and torch.equal(score[new], first[1][new])


# ------------------------------------------------------------------ eviction
def check_eviction(c, score, budget, sinks, recent, in_place=False, use_kept=True):
    B, n_b = c.B, len(c.lens)
    host = score.cpu().numpy().copy() if score is not None else None
    old = [c.rows(b, max(L, 0)) for b, L in enumerate(c.lens)]
    kp, vp = c.k_pool.clone(), c.v_pool.clone()
    seq = c.seq.clone()
    new = seq if in_place else torch.full_like(seq, 77)
    kept = torch.full((c.layers, n_b, c.n_kv, budget), 99, dtype=torch.int32, device="cuda") if use_kept else None
    B.vsd_kv_evict(c.kv, n_b, seq, new, score, budget, sinks=sinks, recent=recent, kept=kept)
    torch.cuda.synchronize()
    assert B.vsd_get_device_status(c.kv) == 0
    assert new.tolist() == [min(L, budget) for L in c.lens]
    if not in_place:
        assert seq.tolist() == c.lens
    want = None if host is None else torch.tensor(host, device="cuda")
    for b, L in enumerate(c.lens):
        for l in range(c.layers):
            for h in range(c.n_kv):
                if L < 0:
                    rows = np.zeros(0, np.int64)
                else:
                    rows = S.evict_rows(host[l, b, h] if host is not None else np.zeros(max(L, 1)), L, budget, sinks, recent)
                n = len(rows)
                if use_kept:
                    assert kept[l, b, h].tolist() == rows.tolist() + [-1] * (budget - n), (l, b, h)
                r = torch.tensor(rows, device="cuda", dtype=torch.long)
                for pool, rowset in ((kp, old[b][0]), (vp, old[b][1])):
                    pages = torch.tensor(c.table[b][np.arange(n) // 16], device="cuda", dtype=torch.long)
                    pool[l, pages, h, torch.arange(n, device="cuda") % 16] = rowset[l, r, h]
                if want is not None and L > budget:
                    want[l, b, h, :n] = torch.tensor(host[l, b, h][rows], device="cuda")
    bits = lambda t: t.view(torch.int16 if t.dtype == torch.bfloat16 else torch.int32)  # noqa: E731
    assert torch.equal(bits(c.k_pool), bits(kp)) and torch.equal(bits(c.v_pool), bits(vp))
    if want is not None:
        assert torch.equal(bits(score), bits(want))


def scores_for(c, kind, seed=0):
    g = torch.Generator("cuda").manual_seed(seed)
    s = torch.rand((c.layers, len(c.lens), c.n_kv, c.max_tokens), device="cuda", generator=g)
    if kind == "ties":
        s = (s * 4).floor()
    elif kind == "equal":
        s.fill_(0.25)
    elif kind == "odd":  # NaN, infinities and both zeros
        x = torch.randint(0, 7, s.shape, device="cuda", generator=g)
        for i, v in enumerate((float("nan"), float("inf"), -float("inf"), 0.0, -0.0)):
            s[x == i] = v
    elif kind == "subnormal":
        s = s * 1e-44
    return s


@pytest.mark.parametrize("kind", ["random", "ties", "equal", "odd", "subnormal"])
@pytest.mark.parametrize("heads", [(14, 2, 64), (8, 2, 128), (3, 3, 64)])
def test_eviction_matches_oracle(heads, kind):
    B = require_gpu()
    c = Cache(B, 2, *heads, [0, 1, 63, 64, 65, 100, 257, -1, 600, 1000], 1000, tag=f"ev{heads}")
    check_eviction(c, scores_for(c, kind), 64, 3, 17)


@pytest.mark.parametrize("budget,sinks,recent", [(1, 0, 0), (1, 1, 0), (1, 0, 1), (256, 0, 0), (257, 0, 256), (511, 255, 0),
                                                 (300, 100, 200), (999, 4, 4), (1000, 0, 0)])
def test_eviction_budgets(budget, sinks, recent):
    B = require_gpu()
    c = Cache(B, 1, 4, 2, 64, [1000, 300, 512], 1000, tag="evb")
    check_eviction(c, scores_for(c, "ties", budget), budget, sinks, recent)


def test_eviction_in_place_lengths_without_kept_or_scores():
    B = require_gpu()
    c = Cache(B, 2, 4, 2, 64, [200, 30, -1, 90], 256, tag="evp")
    check_eviction(c, scores_for(c, "random"), 50, 1, 5, in_place=True, use_kept=False)
    c = Cache(B, 2, 4, 2, 64, [200, 30, -1, 90], 256, tag="evq")
    check_eviction(c, None, 50, 20, 30, in_place=True)


@pytest.mark.parametrize("L", [8001, 20000])
def test_eviction_of_a_long_request(L):
    B = require_gpu()
    model_layers = 1
    c = Cache.__new__(Cache)
    c.B, c.layers, c.n_q, c.n_kv, c.hd, c.lens, c.max_tokens = B, model_layers, 4, 1, 64, [L], L + 5
    c.model = tiny_model(B, 1, 4, 1, 64, 131072)
    c.kv = B.vsd_kv_create(c.model, 1, L + 5)
    c.table = np.arange(c.kv.num_pages).reshape(1, -1)
    c.k_pool, c.v_pool = B.vsd_kv_pools(c.kv)
    g = torch.Generator("cuda").manual_seed(L)
    c.k_pool.normal_(generator=g)
    c.v_pool.normal_(generator=g)
    c.seq = torch.tensor([L], dtype=torch.int32, device="cuda")
    check_eviction(c, scores_for(c, "ties"), L // 3, 4, 100)


def filled_cache(B, layers, n_q, n_kv, hd, lens, room):
    """A cache over shuffled pages whose pools hold random values everywhere."""
    c = Cache.__new__(Cache)
    c.B, c.layers, c.n_q, c.n_kv, c.hd, c.lens, c.max_tokens = B, layers, n_q, n_kv, hd, list(lens), room
    c.model = tiny_model(B, layers, n_q, n_kv, hd, 131072)
    ppr = -(-room // 16)
    c.kv = B.vsd_kv_create(c.model, len(lens), room, 16, len(lens) * ppr + 2)
    c.table = gen._rng("fill", room).permutation(c.kv.num_pages)[: len(lens) * ppr].astype(np.int32).reshape(len(lens), ppr)
    B.vsd_kv_set_page_table(c.kv, torch.tensor(c.table.reshape(-1), device="cuda"))
    c.k_pool, c.v_pool = B.vsd_kv_pools(c.kv)
    g = torch.Generator("cuda").manual_seed(room)
    c.k_pool.normal_(generator=g)
    c.v_pool.normal_(generator=g)
    c.seq = torch.tensor(c.lens, dtype=torch.int32, device="cuda")
    return c


@pytest.mark.parametrize("kind", ["random", "ties", "equal", "odd"])
@pytest.mark.parametrize("heads,lens,room,budget", [
    ((4, 2, 128), [9000, 4097, 5003, -1, 8999, 33], 9000, 4097),     # clusters of CTAs, budgets past one list of them
    ((4, 2, 64), [9000, 4097, 5003, 0], 9000, 8998),
    ((4, 1, 128), [20011], 20011, 700),
    ((4, 4, 64), [33001] + [700] * 19, 33001, 640),                  # a CTA a head, its scores too many for shared memory
    ((8, 8, 64), [1100, 640, 601, 599] * 5, 1100, 600),              # more heads than SMs
    ((8, 8, 128), [8300, 9000, 77] + [300] * 17, 9000, 256),         # the same, scores not kept
])
def test_eviction_forms(kind, heads, lens, room, budget):
    """Few, long requests split over clusters; heads for every SM; scores that fit in shared memory and not."""
    B = require_gpu()
    c = filled_cache(B, 1, *heads, lens, room)
    check_eviction(c, scores_for(c, kind), budget, 4, 60)


@pytest.mark.parametrize("kind", ["random", "ties", "odd"])
@pytest.mark.parametrize("hd,budget", [(64, 200), (128, 100), (128, 1), (64, 17)])
def test_eviction_of_many_short_requests(kind, hd, budget):
    B = require_gpu()
    c = filled_cache(B, 2, 4, 4, hd, [300, 101, 200, 99, 0, -1, 257, 18, 2, 33] * 6, 300)
    check_eviction(c, scores_for(c, kind), budget, budget // 8, budget // 3)


def test_eviction_rejects_bad_requests_and_spares_the_others():
    B = require_gpu()
    c = Cache(B, 1, 4, 2, 64, [100, 100, 100], 128, fill=0.0, tag="evbad")
    table = c.table.copy()
    table[1, 6] = -1  # a page of request 1's rows
    B.vsd_kv_set_page_table(c.kv, torch.tensor(table.reshape(-1), device="cuda"))
    assert B.vsd_get_device_status(c.kv) == B.VSD_DEV_BAD_PAGE
    seq = torch.tensor([129, 100, 100], dtype=torch.int32, device="cuda")
    for in_place in (False, True):
        score = scores_for(c, "random")
        before, kp = score.clone(), c.k_pool.clone()
        s = seq.clone()
        new = s if in_place else torch.zeros_like(seq)
        kept = torch.zeros((1, 3, 2, 40), dtype=torch.int32, device="cuda")
        B.vsd_kv_evict(c.kv, 3, s, new, score, 40, kept=kept)
        torch.cuda.synchronize()
        assert B.vsd_get_device_status(c.kv) == B.VSD_DEV_BAD_PAGE | B.VSD_DEV_BAD_SEQLEN
        assert new.tolist() == [129, 100, 40]
        assert (kept[:, :2] == -1).all() and (kept[:, 2] >= 0).all()
        assert torch.equal(score[:, :2], before[:, :2])
        good = torch.tensor(c.table[2], device="cuda", dtype=torch.long)
        kp[:, good] = c.k_pool[:, good]
        assert torch.equal(c.k_pool, kp)


# ------------------------------------------------------------------ sampling
def run_sample(B, x, u, T=None, k=None, p=None, m=None, logprob=True):
    rows = x.shape[0]
    dev = lambda a, t: None if a is None else torch.tensor(np.broadcast_to(np.asarray(a), (rows,)).copy(), dtype=t, device="cuda")  # noqa: E731
    tok = torch.full((rows,), -9, dtype=torch.int32, device="cuda")
    lp = torch.full((rows,), float("nan"), device="cuda") if logprob else None
    B.vsd_sample_logits(x, dev(u, torch.float32), tok, temperature=dev(T, torch.float32), top_k=dev(k, torch.int32),
                        top_p=dev(p, torch.float32), min_p=dev(m, torch.float32), logprob=lp)
    torch.cuda.synchronize()
    return tok.cpu().numpy(), None if lp is None else lp.double().cpu().numpy()


def check_sample(B, x, u, T=None, k=None, p=None, m=None):
    """Token ids equal the oracle's; where u lies within 2^-30 of a boundary of the cumulative mass (more than the weights'
    rounding can move it) the neighbour counts too.  logprob: float32 rounding of a value with a 2^-30 error."""
    rows = x.shape[0]
    tok, lp = run_sample(B, x, u, T, k, p, m)
    h = x.double().cpu().numpy()
    at = lambda a, r, d: d if a is None else float(np.float32(np.broadcast_to(np.asarray(a), (rows,))[r]))  # noqa: E731
    for r in range(rows):
        t, l, margin = S.sample_logits(h[r], at(u, r, 0.5), at(T, r, 1.0), int(at(k, r, 0)), at(p, r, 1.0), at(m, r, 0.0))
        if margin > 2.0 ** -30:
            assert tok[r] == t, (r, tok[r], t, margin)
            assert lp[r] == l or abs(lp[r] - l) <= 2.0 ** -23 * max(1.0, abs(l)), (r, lp[r], l)
    return tok


def logits(rows, vocab, seed, std=2.0):
    g = torch.Generator("cuda").manual_seed(seed)
    x = std * torch.randn((rows, vocab), device="cuda", generator=g)
    hot = torch.randint(0, vocab, (rows, min(20, vocab)), device="cuda", generator=g)
    return x.scatter_add(1, hot, 8 * torch.rand(hot.shape, device="cuda", generator=g))


def uniforms(rows, seed):
    return np.random.default_rng(seed).uniform(1e-6, 1 - 1e-6, rows).astype(np.float32)


@pytest.mark.parametrize("vocab", [1, 2, 31, 33, 513, 4096, 32000, 50257, 151936, 262144])
@pytest.mark.parametrize("setting", ["plain", "k", "p", "m", "all"])
def test_sampling_matches_oracle(vocab, setting):
    B = require_gpu()
    rows = 9 if vocab < 60000 else 4
    a = {"plain": {}, "k": dict(k=[1, 2, 50, 7, 400, 3, 0, -4, 10 ** 6][:rows]),
         "p": dict(p=[0.9, 0.0, 0.5, 0.99, 1.0, 0.3, 0.95, 0.999, 2.0][:rows]),
         "m": dict(m=[0.05, 1.0, 0.0, 0.3, 2.0, 0.001, -1.0, 0.1, 0.9][:rows]),
         "all": dict(k=[40, 3, 0, 100, 1, 5, 50, 20, 1000][:rows], p=[0.9, 0.5, 0.8, 1.0, 0.1, 0.99, 0.7, 0.95, 0.9][:rows],
                     m=[0.02, 0.0, 0.1, 0.05, 0.5, 0.0, 0.01, 0.3, 0.001][:rows])}[setting]
    check_sample(B, logits(rows, vocab, vocab), uniforms(rows, vocab), T=[0.7, 1.0, 1.5, 0.2, 0.0, 0.9, 3.0, 0.5, 1.0][:rows], **a)


@pytest.mark.parametrize("levels", [1, 2, 5])
def test_sampling_ties_go_to_the_lowest_ids(levels):
    B = require_gpu()
    g = torch.Generator("cuda").manual_seed(levels)
    x = torch.randint(0, levels, (12, 3001), device="cuda", generator=g).float()
    x[3:6] *= -0.0 if levels == 1 else 1.0
    x[6:] = torch.where(torch.rand((6, 3001), device="cuda", generator=g) < 0.5, -0.0, 0.0) if levels == 1 else x[6:]
    for a in (dict(k=7), dict(p=0.33), dict(k=900, p=0.5, m=0.01), dict(m=1.0), {}):
        check_sample(B, x, uniforms(12, levels), T=0.8, **a)


def test_sampling_masked_infinite_and_nan_logits():
    B = require_gpu()
    inf = float("inf")
    x = logits(8, 777, 3)
    x[0] = -inf                         # nothing to sample
    x[1] = float("nan")
    x[2, 1:] = -inf                     # one token
    x[3, ::2] = -inf
    x[4, 5] = inf
    x[5, [3, 700]] = inf                # two tokens share the mass
    x[6, ::3] = float("nan")
    x[7] = -3.0e38                      # the lowest values a mask may use, but for two
    x[7, [10, 20]] = 1.0
    for a in ({}, dict(k=5), dict(p=0.9), dict(m=0.1), dict(k=30, p=0.8, m=0.01)):
        tok = check_sample(B, x, uniforms(8, 1), T=0.9, **a)
        assert tok[0] == tok[1] == -1 and tok[2] == 0 and tok[4] == 5 and tok[5] in (3, 700)
    tok, lp = run_sample(B, x, 0.5, T=[0.0, -1.0, float("nan"), 0.0, 0.0, 0.0, 0.0, 0.0])
    h = x.double().cpu().numpy()
    for r in range(8):
        assert tok[r] == S.sample_logits(h[r], 0.5, 0.0)[0]
    assert lp[0] == -inf and lp[2] == 0.0


def test_sampling_extreme_temperatures_and_uniforms():
    B = require_gpu()
    x = logits(6, 1000, 8)
    tiny, huge = float(np.float32(1e-38)), float(np.float32(3e38))
    tok = check_sample(B, x, 0.37, T=[tiny, 1e-5, 0.01, 100.0, huge, float("inf")])
    assert tok[0] == int(x[0].argmax())
    # uniforms at and outside the ends of (0, 1)
    tok, _ = run_sample(B, x, [0.0, -1.0, float("nan"), 1.0, 7.0, 0.5], T=1.0)
    w = S.filtered(x[3].double().cpu().numpy(), 1.0)
    assert tok[:3].tolist() == [0, 0, 0] and (tok[3:5] >= np.nonzero(w > 2.0 ** -43)[0].max() - 5).all()


def test_sampling_row_stride_alignment_and_rows_behind():
    """Rows inside a wider array, starting anywhere, and rows=0; what lies behind the rows stays out."""
    B = require_gpu()
    for off, vocab in ((0, 1001), (1, 1002), (3, 998), (5, 4093)):
        wide = torch.full((7, vocab + 37), float("inf"), device="cuda")
        x = wide[:, off: off + vocab]
        x.copy_(logits(7, vocab, off))
        for a in ({}, dict(k=20, p=0.9)):
            check_sample(B, x, uniforms(7, off), T=0.8, **a)
    tok = torch.full((3,), 5, dtype=torch.int32, device="cuda")
    B.vsd_sample_logits(torch.zeros((0, 10), device="cuda"), torch.zeros(0, device="cuda"), tok)
    assert tok.tolist() == [5, 5, 5]


def test_sampling_follows_the_distribution_and_repeats_in_a_graph():
    """Evenly spaced uniforms over one row: each token's count is its share, within one; a replayed graph gives the same."""
    B = require_gpu()
    n, vocab = 2000, 700
    x = logits(1, vocab, 4).expand(n, vocab).contiguous()
    u = torch.tensor((np.arange(n) + 0.5) / n, dtype=torch.float32, device="cuda")
    tok = torch.empty(n, dtype=torch.int32, device="cuda")
    p = torch.full((n,), 0.9, device="cuda")
    B.vsd_sample_logits(x, u, tok, top_p=p)
    w = S.filtered(x[0].double().cpu().numpy(), 1.0, top_p=float(np.float32(0.9)))
    counts = np.bincount(tok.cpu().numpy(), minlength=vocab)
    assert np.abs(counts - w / w.sum() * n).max() <= 1.0 + 1e-3
    first = tok.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        B.vsd_sample_logits(x, u, tok, top_p=p)
    tok.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(tok, first)


@pytest.mark.parametrize("tie", [1, 3])
@pytest.mark.parametrize("extra", [dict(), dict(p=0.8), dict(m=0.02), dict(p=0.95, m=0.001)])
def test_sampling_candidates_of_every_number(extra, tie):
    """Lists of candidates around the sizes at which they are dealt out otherwise; alone and in threes of equal logits."""
    B = require_gpu()
    k = [1, 2, 31, 32, 33, 64, 65, 128, 129, 255, 256, 257, 300, 1023, 1024, 1025]
    rows, vocab = len(k), 5003
    ids = torch.randperm(vocab, device="cuda", generator=torch.Generator("cuda").manual_seed(2))
    x = torch.empty(vocab, device="cuda")
    x[ids] = -0.05 * torch.div(torch.arange(vocab, device="cuda"), tie, rounding_mode="floor").float()
    for seed, T in ((1, 1.0), (2, 7.0)):
        check_sample(B, x.expand(rows, vocab).contiguous(), uniforms(rows, seed), T=T, k=k, **extra)


@pytest.mark.parametrize("rows", [1, 40])
@pytest.mark.parametrize("filters", [dict(), dict(k=7), dict(p=1 - 2.0 ** -24)])
def test_log_probability_of_a_token_alone_or_nearly(rows, filters):
    """A token alone has a logarithm of exactly 0; one that a little mass stands beside keeps its digits.

    The rest, exp(-gap / T), has a relative error of 2^-31 and a rounding of half a step of 2^-44 against a largest weight of
    1/2 to 1 (2^-44 relative to that); then four float32 roundings of 2^-24."""
    B = require_gpu()
    vocab, inf = 5000, float("inf")
    g = torch.Generator("cuda").manual_seed(11)
    x = torch.randn((rows, vocab), device="cuda", generator=g)
    for T in (0.37, 1.0, 1.7):
        for one in (dict(k=1), dict(m=1.0), dict(k=1, p=0.5, m=0.1), dict(p=1e-6)):
            tok, lp = run_sample(B, x, 0.7, T=T, **one)
            assert (tok == x.argmax(1).cpu().numpy()).all() and (lp == 0).all(), (T, one)
        y = torch.full((rows, vocab), -inf, device="cuda")
        y[:, 4321] = 2.5
        tok, lp = run_sample(B, y, 0.7, T=T, **filters)
        assert (tok == 4321).all() and (lp == 0).all()
        for gap in (0.5, 3.0, 9.0, 15.0):
            y[:, 17] = 2.5 - gap
            tok, lp = run_sample(B, y, 1 - 2.0 ** -24, T=T, **filters)  # the higher id, whatever its share
            rest = np.exp(-gap / np.float64(np.float32(T)))
            want = -np.log1p(rest if "p" not in filters or 1 / (1 + rest) < np.float32(filters["p"]) else 0.0)
            assert (tok == 4321).all()
            assert np.abs(lp - want).max() <= abs(want) * (2.0 ** -31 + 2.0 ** -43 / rest + 4 * 2.0 ** -24), (T, gap)


@pytest.mark.parametrize("vocab", [1, 3, 511, 513, 4099, 32000, 151936])
def test_sampling_rows_without_filters(vocab):
    """Enough rows for the streamed form: temperatures of every size, greedy rows among them, flat and peaked logits."""
    B = require_gpu()
    rows = 24
    x = logits(rows, vocab, vocab + 1, std=0.3)
    x[::3] = logits(rows // 3, vocab, vocab + 2, std=6.0)
    T = [0.7, 1.0, 1.5, 0.05, 0.0, 0.3, 3.0, 100.0] * 3
    check_sample(B, x, uniforms(rows, vocab), T=T)
    check_sample(B, x, uniforms(rows, vocab + 5))


def test_sampling_rows_without_filters_odd_values():
    """Masked, infinite, NaN and huge logits, extreme temperatures and unaligned rows in the streamed form."""
    B = require_gpu()
    rows, vocab, inf = 32, 5003, float("inf")
    wide = torch.full((rows, vocab + 2), inf, device="cuda")
    x = wide[:, 1: vocab + 1]
    x.copy_(logits(rows, vocab, 9))
    x[0] = -inf
    x[1] = float("nan")
    x[2, 1:] = -inf
    x[3, ::2] = -inf
    x[4, 5] = inf
    x[5, [3, 4000]] = inf
    x[6, ::3] = float("nan")
    x[7] = -3.0e38
    x[7, [10, 4020]] = 1.0
    x[8] *= 1e6                       # x / T beyond the first rounding's range: the shifted form
    x[9] = 3.0e38
    x[9, 77] = 3.1e38
    x[10] -= 1e5
    x[11, 600:] = -inf                # whole tiles of nothing
    x[12, :4999] = float("nan")
    for T in (0.9, 0.01, 50.0):
        tok = check_sample(B, x, uniforms(rows, 4), T=T)
        assert tok[0] == tok[1] == -1 and tok[2] == 0 and tok[4] == 5 and tok[5] in (3, 4000) and tok[9] == 77
    tiny, huge = float(np.float32(1e-38)), float(np.float32(3e38))
    check_sample(B, x, 0.37, T=[tiny, 1e-5, 1e-3, huge, float("inf"), huge, 0.0, -1.0] * 4)
    tok, lp = run_sample(B, x, 0.5, T=0.0)
    h = x.double().cpu().numpy()
    for r in range(rows):
        assert tok[r] == S.sample_logits(h[r], 0.5, 0.0)[0]
        assert lp[r] == (-inf if tok[r] < 0 else 0.0)
    tok, _ = run_sample(B, x[13:], [0.0, -1.0, float("nan"), 1.0, 7.0] + [0.5] * 14, T=1.0)
    assert tok[:3].tolist() == [0, 0, 0] and (tok >= 0).all()


@pytest.mark.parametrize("rows", [1, 5, 40])
def test_sampling_many_kept_tokens(rows):
    """Kept sets too large to gather: their border alone is, or, among many equals and beyond the bins, nothing."""
    B = require_gpu()
    x = logits(rows, 50257, 31, std=1.0)
    for a in (dict(k=2000), dict(k=20000), dict(p=0.98), dict(p=0.999), dict(k=20000, p=0.9), dict(k=3000, p=0.5, m=0.001)):
        check_sample(B, x, uniforms(rows, 7), T=1.3, **a)
    # coarse logits: thousands of equals at the border
    for step in (0.5, 2.0):
        y = (x / step).round() * step
        for a in (dict(k=3000), dict(k=40000), dict(p=0.9), dict(k=9000, p=0.7), dict(p=0.3, m=0.01), dict(k=1), dict(p=0.0)):
            check_sample(B, y, uniforms(rows, 8), T=1.1, **a)
    # a few tokens far above all others: the k-th lies behind the last bin
    z = x.clone()
    z[:, [5, 40000]] += 500.0
    for a in (dict(k=1), dict(k=2), dict(k=3), dict(k=50), dict(k=60000), dict(p=0.9), dict(k=50, p=0.99)):
        check_sample(B, z, uniforms(rows, 9), T=[0.2, 30.0, 300.0, 1.0, 80.0][0:1] * rows if rows != 5 else [0.2, 30.0, 300.0, 1.0, 80.0], **a)


def test_calls_of_two_caches_at_once_and_a_shared_workspace():
    """Two caches' calls on two streams; a captured call replayed after other calls have used the cache's workspace."""
    B = require_gpu()
    rooms = [8000, 900]
    caches = [Cache(B, 1, 14, 2, 64, [700, 90, 650], room, tag=f"two{room}") for room in rooms]
    q, kn, vn = bf16((3, 14, 64), 2.0, "tq"), bf16((3, 2, 64), 1.0, "tk"), bf16((3, 2, 64), 1.0, "tv")

    def call(c, out, score, n=3):
        B.vsd_decode_attention(c.model, c.kv, 0, n, c.seq, q, kn, vn, out, score=score)

    outs = [(torch.empty((3, 14 * 64), dtype=torch.float16, device="cuda"), torch.zeros((3, 2, room), device="cuda")) for room in rooms]
    for c, (o, s) in zip(caches, outs):
        call(c, o, s)
    torch.cuda.synchronize()
    want = [(o.clone(), s.clone()) for o, s in outs]
    side = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(20):
        for c, (o, s), st in zip(caches, outs, side):
            with torch.cuda.stream(st):
                s.zero_()
                call(c, o, s)
    torch.cuda.synchronize()
    for (o, s), (wo, ws) in zip(outs, want):
        assert torch.equal(o, wo) and torch.equal(s, ws)
    graphs = []
    for c, (o, s) in zip(caches, outs):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call(c, o, s)
        graphs.append(g)
    for c, g, (o, s), (wo, ws) in zip(caches, graphs, outs, want):
        other = torch.empty_like(o)
        call(c, other, None, 1)  # another shape through the same workspace
        s.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, wo) and torch.equal(s, ws) and torch.equal(other[0], wo[0])
    assert all(B.vsd_get_device_status(c.kv) == 0 for c in caches)


def test_decode_attention_follows_a_verify_step():
    """A verify step, a decode call and a verify step again on one cache share its workspace: the steps' results are those of
    a cache on which no decode call was made."""
    B = require_gpu()
    from speculative_decoding_block_gb300.target import build_target
    from tests.gpu_helpers import StepIO
    from workload import TINY
    model = build_target(TINY, gen.master_weights(TINY, seed=5), max_positions=4096)[0]
    k, v = (bf16((TINY.layers, 300, TINY.n_kv, TINY.head_dim), 0.6, "vs", i) for i in range(2))
    q, kn, vn = bf16((2, TINY.n_q, 64), 1.0, "vq"), bf16((2, TINY.n_kv, 64), 1.0, "vk"), bf16((2, TINY.n_kv, 64), 1.0, "vv")
    results = []
    for decode in (False, True):
        kv = B.vsd_kv_create(model, 2, 2000)
        for b in range(2):
            B.vsd_kv_write(kv, b, 0, k, v)
        io = StepIO(2, [300, 250], [5, 6], [list(range(16)), list(range(16, 32))])
        got = []
        for step in range(3):
            if decode:
                out = torch.empty((2, TINY.n_q * 64), dtype=torch.float16, device="cuda")
                B.vsd_decode_attention(model, kv, 1, 2, io.seq, q, kn, vn, out, score=torch.zeros((2, TINY.n_kv, 2000), device="cuda"))
            B.vsd_verify_step(model, kv, 2, io.seq, io.pending, io.drafts, io.acc, io.out)
            torch.cuda.synchronize()
            got += [io.seq.tolist(), io.pending.tolist(), io.acc.tolist(), io.out.tolist()]
        assert B.vsd_get_device_status(kv) == 0
        results.append(got)
    assert results[0] == results[1]


def test_eviction_refuses_a_room_beyond_its_bitmap():
    B = require_gpu()
    room, n_b = 950_000, 80  # more requests than half the SMs: a CTA each
    kv = B.vsd_kv_create(tiny_model(B, 1, 1, 1, 64, 1_000_000), n_b, room, 16, 64)
    seq = torch.full((n_b,), 10, dtype=torch.int32, device="cuda")
    score = torch.zeros((1, n_b, 1, room), device="cuda")
    new = torch.zeros_like(seq)
    with pytest.raises(B.VsdError) as e:
        B.vsd_kv_evict(kv, n_b, seq, new, score, 4)
    assert e.value.status == B.VSD_ERR_UNSUPPORTED
    # one request of that room is split over a cluster
    B.vsd_kv_set_page_table(kv, torch.zeros(n_b * (room // 16), dtype=torch.int32, device="cuda"))
    B.vsd_kv_evict(kv, 1, seq, new, score, 4)
    torch.cuda.synchronize()
    assert new[0] == 4 and not new[1:].any() and B.vsd_get_device_status(kv) == 0


def test_eviction_with_a_budget_of_the_whole_type():
    """The list of kept rows is filled to its end, past where a 32-bit index of the loop would wrap."""
    B = require_gpu()
    budget = 2 ** 31 - 1
    if torch.cuda.mem_get_info()[0] < 16 * 2 ** 30:
        pytest.skip("16 GB of free memory")
    c = Cache(B, 1, 1, 1, 64, [20], 64, fill=0.0, tag="max")
    kept, new = torch.zeros((1, 1, 1, budget), dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    B.vsd_kv_evict(c.kv, 1, c.seq, new, torch.zeros((1, 1, 1, 64), device="cuda"), budget, kept=kept)
    torch.cuda.synchronize()
    assert new.tolist() == [20] and kept[0, 0, 0, :20].tolist() == list(range(20))
    assert int(kept[0, 0, 0, 20:].max()) == -1 and int(kept[0, 0, 0, 20:].min()) == -1


# ------------------------------------------------------------------ arguments
def test_arguments_are_refused():
    B = require_gpu()
    c = Cache(B, 2, 4, 2, 64, [20, 30], 64, fill=0.0, tag="arg")
    other = tiny_model(B, 1, 4, 2, 64)
    q, kn = bf16((2, 4, 64), 1.0, "aq"), bf16((2, 2, 64), 1.0, "ak")
    out = torch.zeros((2, 256), dtype=torch.float16, device="cuda")
    score = torch.zeros((2, 2, 2, 64), device="cuda")
    new = torch.zeros(2, dtype=torch.int32, device="cuda")

    def attend(model=c.model, layer=0, batch=2, q=q, k=kn, v=kn, out=out, **a):
        B.vsd_decode_attention(model, c.kv, layer, batch, c.seq, q, k, v, out, **a)

    for bad in (dict(model=other), dict(layer=2), dict(layer=-1), dict(batch=0), dict(window=-1), dict(k=None), dict(v=None)):
        with pytest.raises(B.VsdError) as e:
            attend(**bad)
        assert e.value.status == B.VSD_ERR_ARG, bad
    with pytest.raises(B.VsdError, match="aligned"):
        attend(q=torch.empty(2 * 256 + 1, dtype=torch.bfloat16, device="cuda")[1:])
    both = bf16((2, 4, 64), 1.0, "ab")
    with pytest.raises(B.VsdError, match="overlap"):
        attend(q=both, out=both.view(torch.float16))
    with pytest.raises(B.VsdError, match="overlap"):
        attend(k=both.view(-1)[256:].view(2, 2, 64), out=both.view(torch.float16))
    with pytest.raises(TypeError, match="CUDA"):
        attend(out=out.cpu())
    with pytest.raises(ValueError):
        attend(batch=3)  # q, out and lengths hold two requests
    with pytest.raises(ValueError):
        attend(score=score[0, :1])
    with pytest.raises(TypeError):
        attend(out=out.float())
    with pytest.raises(ValueError):
        attend(q=q.transpose(0, 1))

    def evict(seq=c.seq, new=new, score=score, budget=16, **a):
        B.vsd_kv_evict(c.kv, 2, seq, new, score, budget, **a)

    for bad in (dict(budget=0), dict(sinks=-1), dict(recent=-1), dict(sinks=9, recent=8), dict(score=None),
                dict(sinks=2 ** 31 - 1, recent=2 ** 31 - 1)):
        with pytest.raises(B.VsdError) as e:
            evict(**bad)
        assert e.value.status == B.VSD_ERR_ARG, bad
    long = torch.zeros(3, dtype=torch.int32, device="cuda")
    with pytest.raises(B.VsdError, match="apart"):
        evict(seq=long[:2], new=long[1:])
    with pytest.raises(ValueError):
        evict(kept=torch.zeros(5, dtype=torch.int32, device="cuda"))

    x, u, tok = torch.zeros((2, 8), device="cuda"), torch.zeros(2, device="cuda"), torch.zeros(2, dtype=torch.int32, device="cuda")
    with pytest.raises(TypeError):
        B.vsd_sample_logits(x.half(), u, tok)
    with pytest.raises(ValueError):
        B.vsd_sample_logits(x.t(), u.new_zeros(8), tok.new_zeros(8))
    with pytest.raises(ValueError):
        B.vsd_sample_logits(x, u[:1], tok)
    with pytest.raises(B.VsdError) as e:
        B.vsd_sample_logits(torch.zeros((1, 2 ** 18 + 1), device="cuda"), u, tok)
    assert e.value.status == B.VSD_ERR_UNSUPPORTED
    torch.cuda.synchronize()
    assert B.vsd_get_device_status(c.kv) == 0


# ------------------------------------------------------------------ together
def test_a_run_of_tokens_with_eviction_and_sampling():
    """Two layers, three requests, tokens one by one: attention adds weights and rows, the cache is cut whenever a request
    passes 48 rows, the attention's output makes the logits, the sampled token picks the next inputs.  The oracle follows with
    the library's own tokens, rows and kept sets; every attention output is compared."""
    B = require_gpu()
    layers, n_q, n_kv, hd, budget = 2, 4, 2, 64, 40
    c = Cache(B, layers, n_q, n_kv, hd, [44, 3, 0], 64, tag="run")
    n_b = 3
    vocab = 97
    emb_q, emb_k, emb_v = (bf16((vocab, layers, h, hd), s, "emb", i) for i, (h, s) in enumerate(((n_q, 2.0), (n_kv, 1.0), (n_kv, 1.0))))
    head = torch.randn((n_q * hd, vocab), device="cuda", generator=torch.Generator("cuda").manual_seed(9))
    seq, tok = c.seq.clone(), torch.tensor([1, 2, 3], dtype=torch.int32, device="cuda")
    score = torch.zeros((layers, n_b, n_kv, 64), device="cuda")
    out = torch.empty((n_b, n_q * hd), dtype=torch.float16, device="cuda")
    kept = torch.empty((layers, n_b, n_kv, budget), dtype=torch.int32, device="cuda")
    # the oracle's rows: per request, layer, head
    K = [[[f64(c.k[b][l, :, h]) for h in range(n_kv)] for l in range(layers)] for b in range(n_b)]
    V = [[[f64(c.v[b][l, :, h]) for h in range(n_kv)] for l in range(layers)] for b in range(n_b)]
    cuts = 0
    for step in range(20):
        q, kn, vn = emb_q[tok.long()], emb_k[tok.long()], emb_v[tok.long()]
        lens = seq.tolist()
        for l in range(layers):
            B.vsd_decode_attention(c.model, c.kv, l, n_b, seq, q[:, l].contiguous(), kn[:, l].contiguous(), vn[:, l].contiguous(),
                                   out, score=score[l])
            for b in range(n_b):
                for h in range(n_kv):
                    K[b][l][h] = np.concatenate([K[b][l][h], f64(kn[b, l, h])[None]])
                    V[b][l][h] = np.concatenate([V[b][l][h], f64(vn[b, l, h])[None]])
                k, v = np.stack(K[b][l], 1), np.stack(V[b][l], 1)
                assert k.shape[0] == lens[b] + 1
                ref, _, _ = S.decode_attention(f64(q[b, l]), k, v)
                tol, _ = attention_tolerance(f64(q[b, l]), k, v, ref, k.shape[0])
                assert (np.abs(f64(out[b]).reshape(n_q, hd) - ref) <= tol).all(), (step, l, b)
        seq += 1
        if int(seq.max()) >= 48:
            cuts += 1
            host, lens = score.cpu().numpy().copy(), seq.tolist()
            B.vsd_kv_evict(c.kv, n_b, seq, seq, score, budget, sinks=2, recent=8, kept=kept)
            for b in range(n_b):
                for l in range(layers):
                    for h in range(n_kv):
                        rows = S.evict_rows(host[l, b, h], lens[b], budget, 2, 8)
                        assert kept[l, b, h, : len(rows)].tolist() == rows.tolist()
                        K[b][l][h], V[b][l][h] = K[b][l][h][rows], V[b][l][h][rows]
        x = out.float() @ head
        u = uniforms(n_b, step)
        want = [S.sample_logits(r, float(uu), float(np.float32(0.8)), 20, float(np.float32(0.9))) for r, uu in zip(x.double().cpu().numpy(), u)]
        B.vsd_sample_logits(x, torch.tensor(u, device="cuda"), tok, temperature=torch.full((n_b,), 0.8, device="cuda"),
                            top_k=torch.full((n_b,), 20, dtype=torch.int32, device="cuda"), top_p=torch.full((n_b,), 0.9, device="cuda"))
        assert all(t == w[0] or w[2] < 2.0 ** -30 for t, w in zip(tok.tolist(), want))
    assert cuts >= 2 and B.vsd_get_device_status(c.kv) == 0


def test_sampling_next_to_the_verify_step():
    """The verify step's own logits, sampled at a temperature: the token of the first row is the one that the stochastic step's
    rule gives for the same uniform when its draft is refused and nothing is excluded (the bonus row's rule)."""
    B = require_gpu()
    from oracle.sampling import sample_row
    x = logits(17, 4096, 21)
    u = uniforms(17, 21)
    tok, _ = run_sample(B, x, u, T=0.7)
    for r in range(17):
        t, margin = sample_row(x[r].double().cpu().numpy(), float(np.float32(0.7)), float(u[r]))
        assert tok[r] == t or margin < 2.0 ** -30


def test_pools_are_the_caches_memory():
    B = require_gpu()
    c = Cache(B, 2, 4, 2, 64, [20], 32, fill=0.0, tag="pool")
    k, v = c.rows(0, 20)
    assert torch.equal(k, c.k[0]) and torch.equal(v, c.v[0])
    c.k_pool[1, c.table[0, 1], 0, 3] = 2.5  # row 19 of layer 1, KV head 0
    k, _ = c.rows(0, 20)
    assert (k[1, 19, 0] == 2.5).all() and torch.equal(k[1, 19, 1], c.k[0][1, 19, 1])
    p = ctypes.c_void_p()
    assert B.lib().vsd_kv_pools(c.kv.handle, ctypes.byref(p), None) == B.VSD_ERR_ARG
