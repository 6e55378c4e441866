"""Paged KV cache on the GPU: the write with rotation and 8-bit rounding, the
attention over selected rows of the cache and the index upkeep from its pages,
against plain float64 statements of the same."""
import math

import numpy as np
import pytest
import torch

import oracle as O
from hierarchical_latent_key_gemm_b200 import lsa, pipeline

pytestmark = pytest.mark.gpu

BF, F32, E4 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
HALF_STEP = {BF: 2.0 ** -8, F32: 2.0 ** -24}     # a rounding's largest relative error


@pytest.fixture(autouse=True)
def _clean():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    assert lsa.lsa_check() == lsa.LSA_OK
    yield
    torch.cuda.synchronize()


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _values(cache, which):
    """The pool's values [n_pages, hkv, page, d] in float64 numpy."""
    pool, scale = getattr(cache, which), getattr(cache, which + "_scale")
    x = pool.double()
    return (x if scale is None else x * scale.double()[:, :, None, None]).cpu().numpy()


def _shuffled_cache(batch, tokens, hkv, d, page, dtype, seed, spare=2):
    """A cache whose pages are handed out in random order, garbage (NaN too) in every slot."""
    g = _gen(seed)
    per = -(-tokens // page)
    c = lsa.make_kv_cache(batch, per * page, hkv, d, page, dtype, n_pages=batch * per + spare)
    c.page_table.copy_(torch.randperm(batch * per + spare, generator=g, device="cuda")[:batch * per].view(batch, per))
    raw = torch.randint(0, 256, c.K.shape + (c.K.element_size(),), generator=g, device="cuda").to(torch.uint8)
    c.K.view(torch.uint8).copy_(raw.view(c.K.view(torch.uint8).shape))
    c.V.view(torch.uint8).copy_(raw.flip(0).view(c.K.view(torch.uint8).shape))
    return c


def _inv_freq(rot, base=10000.0):
    return base ** (-torch.arange(rot // 2, dtype=torch.float64, device="cuda") / max(1, rot // 2)) if rot else None


def _new_tokens(lens, hkv, hq, d, io, seed, pad=0, loud=()):
    g = _gen(seed)
    n = sum(lens) + pad
    mk = lambda h: (torch.randn(n, h, d, generator=g, device="cuda")
                    * torch.exp(0.5 * torch.randn(h, d, generator=g, device="cuda"))).to(io)
    K, V, Q = mk(hkv), mk(hkv), mk(hq) if hq else None
    for t, f in loud:
        K[t] *= f
        V[t] *= f
    cu = torch.tensor([0] + list(np.cumsum(lens)), dtype=torch.int64, device="cuda")
    return K, V, Q, cu


def _check_write(cache, before, K, V, Q, K_out, Q_out, cu, pos0, rot, interleaved):
    """Everything a write leaves behind against the float64 statement of it."""
    io, page = K.dtype, cache.page
    f64 = lambda t: t.double().cpu().numpy()
    f = np.zeros(0) if rot == 0 else _inv_freq(rot).cpu().numpy()
    cu, pos0 = cu.tolist(), pos0.tolist()
    pos = np.concatenate([pos0[b] + np.arange(cu[b + 1] - cu[b]) for b in range(cache.batch)])
    n = cu[-1]
    # a turned component: cos, sin and two products and a sum in fp32, each within 2^-23 of |x| + |y| <= 2 amax
    slack = lambda x: 2.0 ** -21 * 2 * np.abs(x).max(-1, keepdims=True) if rot else 0.0
    for raw, out in ((Q, Q_out), (K, K_out)):
        if raw is None or out is None:
            continue
        x = f64(raw)[:n]
        want = O.rotate(x, pos, f, interleaved)
        assert np.all(np.abs(f64(out)[:n] - want) <= HALF_STEP[io] * np.abs(want) + slack(x))
    k = O.rotate(f64(K)[:n], pos, f, interleaved)
    v = f64(V)[:n]
    table = cache.page_table.cpu().numpy()
    touched = set()
    for name, new, raw, lim in (("K", k, f64(K), O.LIM_K), ("V", v, f64(V), O.LIM_V)):
        got, held = _values(cache, name), before[name]
        sl = slack(f64(K)[:n]) if name == "K" and rot else np.zeros((n, cache.hkv, 1))
        for b in range(cache.batch):
            t = cu[b]
            while t < cu[b + 1]:
                p = pos0[b] + t - cu[b]
                first, pid = p % page, int(table[b, p // page])
                m = min(page - first, cu[b + 1] - t)
                touched.add(pid)
                for h in range(cache.hkv):
                    if cache.scaled:
                        s, want = O.write_page(held[pid, h], before[name + "_scale"][pid, h], first,
                                               raw[t:t + m, h], new[t:t + m, h], lim)
                        assert float(getattr(cache, name + "_scale")[pid, h]) == s
                        assert np.array_equal(got[pid, h, :first], want[:first], equal_nan=True)
                        w = want[first:first + m]
                        g = got[pid, h, first:first + m]
                        if name == "V":
                            assert np.array_equal(g, O.round_e4m3(w / s) * s, equal_nan=True)
                        else:
                            ok = np.maximum(2.0 ** -4 * np.abs(w), 2.0 ** -10 * s) + sl[t:t + m, h]
                            assert np.all(np.isnan(w) == np.isnan(g))
                            assert np.all((np.abs(g - w) <= ok) | np.isnan(w))
                        # slots behind the last token keep their codes
                        code = lambda pools: pools.view(torch.uint8)[pid, h, first + m:]
                        assert torch.equal(code(getattr(cache, name)), code(before[name + "_codes"]))
                    else:
                        assert np.array_equal(got[pid, h, :first], held[pid, h, :first], equal_nan=True)
                        assert np.array_equal(got[pid, h, first + m:], held[pid, h, first + m:], equal_nan=True)
                        w, g = new[t:t + m, h], got[pid, h, first:first + m]
                        assert np.all(np.abs(g - w) <= 2.0 ** -8 * np.abs(w) + sl[t:t + m, h])
                t += m
    for name in "KV":
        for pid in range(cache.K.shape[0]):
            if pid not in touched:
                assert torch.equal(getattr(cache, name)[pid].view(torch.uint8),
                                   before[name + "_codes"][pid].view(torch.uint8))
                if cache.scaled:
                    assert np.array_equal(getattr(cache, name + "_scale")[pid].cpu().numpy(),
                                          before[name + "_scale"][pid])


def _snapshot(cache):
    s = {}
    for name in "KV":
        s[name] = _values(cache, name)
        s[name + "_codes"] = getattr(cache, name).clone()
        if cache.scaled:
            s[name + "_scale"] = getattr(cache, name + "_scale").cpu().numpy().copy()
    return s


WRITES = [
    # lens, first positions, hkv, hq, d, page, pages, io, rot, interleaved
    ([1], [0], 1, 0, 64, 16, E4, BF, 0, False),
    ([1, 1, 1, 1], [10_000_003, 10_000_063, 9_999_999, 10_000_064], 1, 16, 128, 64, E4, BF, 128, False),
    ([17], [0], 2, 2, 64, 16, E4, F32, 64, True),
    ([33, 0, 5, 1], [15, 16, 31, 200], 3, 6, 128, 32, E4, BF, 48, False),
    ([40, 3], [127, 1], 4, 4, 64, 128, E4, F32, 16, False),
    ([300, 2, 0, 131], [5, 0, 0, 66], 2, 10, 128, 64, E4, BF, 128, True),
    ([50, 7], [9, 100], 2, 4, 128, 16, BF, BF, 128, False),
    ([50, 7], [9, 100], 2, 4, 64, 16, BF, F32, 32, True),
    ([9], [3], 40, 48, 64, 16, E4, BF, 64, False),
    ([1] * 70, list(range(70)), 2, 2, 64, 32, E4, BF, 64, False),
]


@pytest.mark.parametrize("lens,pos0,hkv,hq,d,page,dtype,io,rot,inter", WRITES)
def test_write_matches_the_float64_statement(lens, pos0, hkv, hq, d, page, dtype, io, rot, inter):
    B = len(lens)
    # the table covers far positions; only the pages from the first position on exist
    last = max(p + n for p, n in zip(pos0, lens))
    near = _shuffled_cache(B, page * (max((p % page + n + page - 1) // page for p, n in zip(pos0, lens)) + 1), hkv, d,
                           page, dtype, 1)
    table = torch.full((B, last // page + 2), -1, dtype=torch.int32, device="cuda")
    for b in range(B):
        k = pos0[b] // page
        w = min(near.page_table.shape[1], table.shape[1] - k)
        table[b, k:k + w] = near.page_table[b, :w]
    cache = lsa.KVCache(near.K, near.V, table, near.K_scale, near.V_scale)
    pos = torch.tensor(pos0, dtype=torch.int64, device="cuda")
    for step, f in ((0, 1.0), (1, 300.0), (2, 0.01)):
        # three writes in a row: the second one's values are larger, so a part-filled page changes its scale
        K, V, Q, cu = _new_tokens(lens, hkv, hq, d, io, 10 + step, pad=3, loud=[(i, f) for i in range(sum(lens))])
        before = _snapshot(cache)
        if step == 0 and cache.scaled:
            for name in "KV":        # what a page held before has no codes that are NaN
                p = getattr(cache, name).view(torch.uint8)
                p.copy_(torch.where((p & 0x7f) == 0x7f, p & 0x80, p))
            before = _snapshot(cache)
        K_out = torch.full_like(K, 7.0)
        Q_out = torch.full_like(Q, 7.0) if hq else None
        lsa.lsa_cache_write(cache, K, V, cu, pos, Q=Q, inv_freq=_inv_freq(rot), interleaved=inter, K_out=K_out,
                            Q_out=Q_out)
        assert lsa.lsa_check() == lsa.LSA_OK
        _check_write(cache, before, K, V, Q, K_out, Q_out, cu, pos, rot, inter)
        n = sum(lens)
        assert torch.all(K_out[n:] == 7.0) and (not hq or torch.all(Q_out[n:] == 7.0))


def test_write_in_place_and_without_outputs_leaves_the_same_pages():
    lens, pos0 = [37, 5], [11, 60]
    K, V, Q, cu = _new_tokens(lens, 2, 4, 128, BF, 3)
    pos, f = torch.tensor(pos0, device="cuda"), _inv_freq(128)
    pools = []
    for mode in range(3):
        c = _shuffled_cache(2, 128, 2, 128, 32, E4, 5)
        k, q = K.clone(), Q.clone()
        if mode == 0:
            q, k = lsa.lsa_cache_write(c, k, V, cu, pos, Q=q, inv_freq=f, want_K=True)
        elif mode == 1:
            lsa.lsa_cache_write(c, k, V, cu, pos, Q=q, inv_freq=f, K_out=k, Q_out=q)
        else:
            assert lsa.lsa_cache_write(c, k, V, cu, pos, inv_freq=f) == (None, None)
            k, q = pools[0][0], pools[0][1]
        pools.append((k, q, c.K.view(torch.uint8), c.V.view(torch.uint8), c.K_scale, c.V_scale))
    for p in pools[1:]:
        assert all(torch.equal(x, y) for x, y in zip(p, pools[0]))


def test_write_values_that_are_not_finite_or_too_large():
    c = lsa.make_kv_cache(1, 32, 1, 64, page=16)
    K, V, _, cu = _new_tokens([20], 1, 0, 64, F32, 4)
    V[3, 0, 5], V[3, 0, 6], V[4, 0, 7], V[17, 0, 0] = math.inf, -math.inf, math.nan, 3e38
    K[2, 0, 1] = math.nan
    before = _snapshot(c)
    lsa.lsa_cache_write(c, K, V, cu, torch.zeros(1, dtype=torch.int64, device="cuda"))
    assert lsa.lsa_check() == lsa.LSA_OK
    got = _values(c, "V")[0, 0]
    assert np.isnan(got[3, 5]) and np.isnan(got[3, 6]) and np.isnan(got[4, 7]) and np.isnan(got).sum() == 3
    assert np.isnan(_values(c, "K")[0, 0]).sum() == 1
    assert c.V_scale[0, 0] <= 1 and c.V_scale[1, 0] == 2.0 ** 64        # only the finite ones count; clamped
    assert _values(c, "V")[1, 0, 1, 0] == 448 * 2.0 ** 64               # saturates
    _check_write(c, before, K, V, None, None, None, cu, torch.zeros(1, dtype=torch.int64), 0, False)


def test_write_latches_bad_pages_and_offsets():
    f = _inv_freq(64)
    K, V, Q, cu = _new_tokens([20, 20], 2, 2, 64, BF, 6)
    pos = torch.tensor([0, 0], device="cuda")
    for what in ("page id", "page id past the pool", "past the table", "negative position", "cu falls", "cu too long"):
        c = _shuffled_cache(2, 32, 2, 64, 16, E4, 7)
        ref = _shuffled_cache(2, 32, 2, 64, 16, E4, 7)
        lsa.lsa_cache_write(ref, K, V, cu, pos, Q=Q, inv_freq=f)
        assert lsa.lsa_check() == lsa.LSA_OK
        untouched = _snapshot(c)["K_codes"].view(torch.uint8)
        p, q, bad = pos.clone(), cu.clone(), None
        if what == "page id":
            bad, c.page_table[1, 1] = (1, 1), -1
        elif what == "page id past the pool":
            bad, c.page_table[0, 0] = (0, 0), c.K.shape[0]
        elif what == "past the table":
            p[1] = 16
        elif what == "negative position":
            p[1] = -1
        elif what == "cu falls":
            q[1] = 45
        else:
            q[2] = 41
        lsa.lsa_cache_write(c, K, V, q, p, Q=Q, inv_freq=f)
        assert lsa.lsa_check() == lsa.LSA_ERR_DEVICE
        assert lsa.lsa_check() == lsa.LSA_OK
        now = c.K.view(torch.uint8)
        if what.startswith("cu"):
            assert torch.equal(now, untouched)
        elif bad:        # the other pages are as they should be
            for b in range(2):
                for j in range(2):
                    pid = int(ref.page_table[b, j])
                    want = untouched[pid] if (b, j) == bad else ref.K.view(torch.uint8)[pid]
                    assert torch.equal(now[pid], want)


def test_write_refuses_what_it_cannot_take():
    c = lsa.make_kv_cache(1, 32, 1, 64, page=16)
    K, V, Q, cu = _new_tokens([4], 1, 1, 64, BF, 6)
    pos = torch.zeros(1, dtype=torch.int64, device="cuda")
    with pytest.raises(ValueError, match="contiguous"):
        lsa.lsa_cache_write(c, K, torch.cat([V, V], 2)[..., ::2], cu, pos)
    flat = torch.zeros(4 * 64 + 8, dtype=BF, device="cuda")
    with pytest.raises(lsa.LsaError):           # not on a 16-byte boundary
        lsa.lsa_cache_write(c, flat[1:257].view(4, 1, 64), V, cu, pos)
    with pytest.raises(ValueError, match="the cache on"):
        lsa.lsa_cache_write(c, K.cpu(), V.cpu(), cu, pos)
    # no token at all
    lsa.lsa_cache_write(c, K[:0], V[:0], cu * 0, pos)
    assert lsa.lsa_check() == lsa.LSA_OK


# ------------------------------------------------------------------ attention
def _filled(batch, tokens, hkv, d, page, dtype, seed, spread=0):
    """A cache full of values; `spread`: page scales up to 2^spread apart, the values' sizes unchanged for K and
    following the scale for V."""
    c = _shuffled_cache(batch, tokens, hkv, d, page, dtype, seed)
    g = _gen(seed + 1)
    for name in "KV":
        x = torch.randn(c.K.shape, generator=g, device="cuda")
        pool, scale = getattr(c, name), getattr(c, name + "_scale")
        if scale is None:
            pool.copy_(x.to(dtype))
            continue
        e = torch.randint(-spread, spread + 1, scale.shape, generator=g, device="cuda").float()
        s = torch.exp2(e - 6)
        scale.copy_(s)
        y = x / (s[:, :, None, None] if name == "K" and spread <= 6 else 2.0 ** -6)
        pool.copy_(y.clamp(-440, 440).to(dtype))
    return c


def _selection(g, batch, nq, hkv, max_sel, tokens, lengths):
    """Rows of `lengths` distinct ascending tokens, entries behind them garbage."""
    n = batch * nq * hkv
    idx = np.full((n, max_sel), 2 ** 31 - 1, dtype=np.int64)
    idx[:, 1::2] = -12345
    cnt = np.array([lengths[i % len(lengths)] for i in range(n)])
    for i in range(n):
        idx[i, :cnt[i]] = np.sort(g.choice(tokens, size=cnt[i], replace=False))
    to = lambda a, *s: torch.tensor(a, dtype=torch.int32, device="cuda").view(*s)
    return to(idx, batch, nq, hkv, max_sel), to(cnt, batch, nq, hkv)


def _check_attn(cache, Q, idx, cnt, Oo, lse):
    """Against float64 softmax attention over the cache's values, row by row."""
    B, nq, hq, d = Q.shape
    G = hq // cache.hkv
    vals = {n: _values(cache, n) for n in "KV"}
    table = cache.page_table.cpu().numpy()
    q, o, z = Q.double().cpu().numpy(), Oo.double().cpu().numpy(), lse.cpu().numpy()
    idx, cnt = idx.cpu().numpy(), cnt.cpu().numpy()
    worst = 0.0
    for b in range(B):
        for i in range(nq):
            for h in range(cache.hkv):
                n = cnt[b, i, h]
                hs = slice(h * G, (h + 1) * G)
                if n == 0:
                    assert np.all(o[b, i, hs] == 0) and np.all(z[b, i, hs] == -np.inf)
                    continue
                t = idx[b, i, h, :n]
                k, v = (vals[x][table[b, t // cache.page], h, t % cache.page] for x in "KV")
                s = q[b, i, hs] @ k.T / math.sqrt(d)
                m = s.max(1, keepdims=True)
                p = np.exp(s - m)
                want = p @ v / p.sum(1, keepdims=True)
                wz = (m + np.log(p.sum(1, keepdims=True)))[:, 0]
                # a score: d products summed in fp32 (each within 2^-24 of the sum of magnitudes), the scale and the
                # base-2 exponent; a weight is off by that much relative, the sums by 2^-24 an addition
                ds = 2.0 ** -24 * (d + 8) * (np.abs(q[b, i, hs]) @ np.abs(k).T).max(1) / math.sqrt(d) + 2.0 ** -21
                spread = (p @ np.abs(v)) / p.sum(1, keepdims=True)       # what the weights' errors act on
                # weights rounded to 11 bits where they meet the tensor cores, to 2^-25 of the largest at least
                w11 = 2.0 ** -11 if Q.dtype == BF else 0.0
                tol = spread * (2 * ds[:, None] + 2.0 ** -23 * n + w11)
                if Q.dtype == BF:
                    tol = tol + 2.0 ** -25 * n * np.abs(v).max(0) / p.sum(1, keepdims=True)
                tol = tol + HALF_STEP[Q.dtype] * np.abs(want) + 1e-30
                err = np.abs(o[b, i, hs] - want)
                assert np.all(err <= tol), (b, i, h, n, float((err / tol).max()))
                worst = max(worst, float((err / tol).max()))
                assert np.all(np.abs(z[b, i, hs] - wz) <= ds + 2.0 ** -23 * (n + np.abs(wz)))
    return worst


ATTN = [
    # batch, nq, hq, hkv, d, page, pages, io, max_sel, tokens, lengths
    (1, 1, 1, 1, 64, 16, E4, BF, 1, 1, [1]),
    (1, 1, 16, 1, 128, 64, E4, BF, 900, 5000, [900]),
    (2, 3, 8, 2, 128, 32, E4, BF, 333, 700, [0, 1, 15, 16, 17, 333]),
    (2, 3, 8, 2, 64, 16, E4, BF, 333, 700, [333, 0, 31, 32, 33, 2]),
    (2, 2, 12, 4, 128, 128, BF, BF, 150, 300, [150, 0, 7, 64]),
    (2, 2, 12, 4, 64, 16, BF, BF, 150, 300, [150, 0, 7, 64]),
    (1, 2, 5, 1, 128, 64, E4, BF, 65, 129, [65, 64]),
    (1, 3, 40, 2, 128, 64, E4, BF, 100, 200, [100, 3, 0]),
    (1, 2, 64, 1, 64, 32, BF, BF, 100, 200, [100, 99]),
    (2, 3, 6, 2, 128, 32, E4, F32, 200, 400, [200, 0, 1, 33]),
    (1, 2, 10, 1, 64, 16, BF, F32, 77, 100, [77, 76]),
    (1, 70, 8, 4, 64, 64, E4, BF, 48, 500, [48, 0, 47, 1]),
    (3, 1, 16, 4, 128, 64, E4, BF, 3001, 4000, [3001, 2999, 0]),
    (3, 400, 4, 1, 64, 64, E4, BF, 40, 500, [40, 0, 39, 1, 17]),
]


@pytest.mark.parametrize("batch,nq,hq,hkv,d,page,dtype,io,max_sel,tokens,lengths", ATTN)
def test_attention_matches_float64(batch, nq, hq, hkv, d, page, dtype, io, max_sel, tokens, lengths):
    c = _filled(batch, tokens, hkv, d, page, dtype, 20)
    Q = torch.randn(batch, nq, hq, d, generator=_gen(21), device="cuda").to(io)
    idx, cnt = _selection(np.random.RandomState(22), batch, nq, hkv, max_sel, tokens, lengths)
    Oo, lse = lsa.lsa_cache_attn(c, Q, idx, cnt)
    assert lsa.lsa_check() == lsa.LSA_OK
    print("worst error over its bound: %.3f" % _check_attn(c, Q, idx, cnt, Oo, lse))
    again, none = lsa.lsa_cache_attn(c, Q, idx, cnt, want_lse=False)
    assert none is None and torch.equal(again, Oo)


@pytest.mark.parametrize("io", [BF, F32])
@pytest.mark.parametrize("spread", [6, 30])
def test_attention_with_scales_far_apart(io, spread):
    """V scales 2^(2 spread) apart within a row (K's follow their values up to 2^6, scores beyond that are decided by
    the largest page)."""
    c = _filled(1, 600, 2, 128, 32, E4, 30, spread=spread)
    if spread > 6:
        c.K_scale.fill_(2.0 ** -6)
    Q = torch.randn(1, 2, 8, 128, generator=_gen(31), device="cuda").to(io)
    idx, cnt = _selection(np.random.RandomState(32), 1, 2, 2, 300, 600, [300, 17])
    Oo, lse = lsa.lsa_cache_attn(c, Q, idx, cnt)
    _check_attn(c, Q, idx, cnt, Oo, lse)


@pytest.mark.parametrize("io", [BF, F32])
def test_attention_with_large_scores_and_queries(io):
    """Scores of thousands (one key takes all the weight) and queries near the type's ends."""
    c = _filled(1, 100, 1, 64, 16, E4, 33)
    idx, cnt = _selection(np.random.RandomState(34), 1, 3, 1, 60, 100, [60, 59, 1])
    Q = torch.randn(1, 3, 4, 64, generator=_gen(35), device="cuda")
    Q[:, 0] *= 1e3
    Q[:, 1] *= 1e-30
    Q[:, 2, 1:] = 0
    Q = Q.to(io)
    Oo, lse = lsa.lsa_cache_attn(c, Q, idx, cnt)
    _check_attn(c, Q, idx, cnt, Oo, lse)
    # near the largest number: the largest score takes all the weight
    Q.zero_()
    Q[:, :, :, 3] = 1e37
    Oo, lse = lsa.lsa_cache_attn(c, Q, idx, cnt)
    k, v = _values(c, "K"), _values(c, "V")
    table, rows = c.page_table[0].cpu().numpy(), idx[0, :, 0].cpu().numpy()
    for i, n in enumerate(cnt[0, :, 0].tolist()):
        t = rows[i, :n]
        s = k[table[t // 16], 0, t % 16, 3]
        top = v[table[t // 16], 0, t % 16][s == s.max()].mean(0)     # 8-bit keys tie
        assert np.all(np.abs(Oo[0, i].double().cpu().numpy() - top) <= 2.0 ** -7 * np.abs(top) + 2.0 ** -20)
        assert torch.isfinite(lse[0, i]).all()


@pytest.mark.parametrize("io", [BF, F32])
def test_attention_any_order_repeats_and_what_is_not_selected(io):
    """A token may stand in a row twice (it counts twice), in any order; NaN in slots that no row selects, and in
    entries of the table that no row reaches, are not read."""
    c = _filled(1, 200, 1, 64, 16, E4, 40)
    row = torch.tensor([7, 150, 7, 3, 3, 3, 199, 0], dtype=torch.int32, device="cuda")
    idx = row.view(1, 1, 1, -1).expand(1, 2, 1, -1).contiguous()
    cnt = torch.tensor([8, 3], dtype=torch.int32, device="cuda").view(1, 2, 1)
    keep = torch.zeros(200, dtype=torch.bool)
    keep[row.long().cpu()] = True
    for t in range(200):
        if not keep[t]:
            pid = int(c.page_table[0, t // 16])
            c.K.view(torch.uint8)[pid, :, t % 16] = 0x7f
            c.V.view(torch.uint8)[pid, :, t % 16] = 0xff
    c.page_table[0, 5] = -7
    Q = torch.randn(1, 2, 4, 64, generator=_gen(41), device="cuda").to(io)
    Oo, lse = lsa.lsa_cache_attn(c, Q, idx, cnt)
    assert lsa.lsa_check() == lsa.LSA_OK
    _check_attn(c, Q, idx, cnt, Oo, lse)
    # a selected NaN reaches its heads, and no other row
    c.K.view(torch.uint8)[int(c.page_table[0, 0]), 0, 0] = 0x7f
    Oo, lse = lsa.lsa_cache_attn(c, Q, idx, cnt)
    assert torch.isnan(Oo[0, 0]).all() and torch.isnan(lse[0, 0]).all()
    assert torch.isfinite(Oo[0, 1].float()).all() and torch.isfinite(lse[0, 1]).all()


@pytest.mark.parametrize("io", [BF, F32])
def test_attention_skips_and_latches_bad_tokens(io):
    c = _filled(2, 64, 1, 64, 16, E4, 50)
    Q = torch.randn(2, 1, 4, 64, generator=_gen(51), device="cuda").to(io)
    good = torch.tensor([1, 5, 20, 40], dtype=torch.int32, device="cuda")
    idx = good.view(1, 1, 1, 4).expand(2, 1, 1, 4).contiguous()
    cnt = torch.full((2, 1, 1), 4, dtype=torch.int32, device="cuda")
    ref, rl = lsa.lsa_cache_attn(c, Q, idx, cnt)
    for bad in (-1, 64, 2 ** 31 - 1, -2 ** 31):
        i2 = torch.cat([idx[..., :2], torch.full_like(idx[..., :1], bad), idx[..., 2:]], -1).contiguous()
        Oo, lse = lsa.lsa_cache_attn(c, Q, i2, cnt + 1)
        assert lsa.lsa_check() == lsa.LSA_ERR_DEVICE
        _check_attn(c, Q, idx, cnt, Oo, lse)
    c.page_table[1, 1] = c.K.shape[0]
    Oo, lse = lsa.lsa_cache_attn(c, Q, idx, cnt)
    assert lsa.lsa_check() == lsa.LSA_ERR_DEVICE
    assert torch.equal(Oo[0], ref[0])
    # a count out of range is clamped and latched; all tokens bad gives the empty row
    lsa.lsa_cache_attn(c, Q, idx, cnt * 2)
    assert lsa.lsa_check() == lsa.LSA_ERR_DEVICE
    Oo, lse = lsa.lsa_cache_attn(c, Q, idx * 0 - 1, cnt)
    assert lsa.lsa_check() == lsa.LSA_ERR_DEVICE
    assert torch.all(Oo == 0) and torch.all(lse == -math.inf)


def test_attention_refuses_what_it_cannot_take():
    c = _filled(1, 64, 1, 64, 16, E4, 50)
    idx = torch.zeros(1, 1, 1, 4, dtype=torch.int32, device="cuda")
    cnt = torch.zeros(1, 1, 1, dtype=torch.int32, device="cuda")
    with pytest.raises(lsa.LsaError):           # more than 64 heads share a row
        lsa.lsa_cache_attn(c, torch.zeros(1, 1, 65, 64, dtype=BF, device="cuda"), idx, cnt)
    flat = torch.zeros(68, dtype=BF, device="cuda")
    with pytest.raises(lsa.LsaError):           # not on a 16-byte boundary
        lsa.lsa_cache_attn(c, flat[1:65].view(1, 1, 1, 64), idx, cnt)
    with pytest.raises(ValueError, match="contiguous"):
        lsa.lsa_cache_attn(c, torch.zeros(1, 1, 2, 128, dtype=BF, device="cuda")[..., ::2], idx, cnt)
    pool = torch.zeros(4 * 16 * 64 + 32, dtype=E4, device="cuda")[8:-24].view(4, 1, 16, 64)
    odd = lsa.KVCache(pool, pool.clone(), c.page_table, c.K_scale[:4].contiguous(), c.V_scale[:4].contiguous())
    with pytest.raises(lsa.LsaError):           # pools not on a 16-byte boundary
        lsa.lsa_cache_attn(odd, torch.zeros(1, 1, 4, 64, dtype=BF, device="cuda"), idx, cnt)
    none = torch.zeros(1, 0, 4, 64, dtype=BF, device="cuda")
    Oo, lse = lsa.lsa_cache_attn(c, none, idx[:, :0], cnt[:, :0])
    assert Oo.shape == none.shape and lse.shape == (1, 0, 4)


def test_offsets_past_32_bits():
    """Pools of more than 2^31 elements: pages at both ends are written and read."""
    page, hkv, d = 128, 8, 128
    n_pages = 2 ** 31 // (page * hkv * d) + 64
    K = torch.empty(n_pages, hkv, page, d, dtype=E4, device="cuda")
    V = torch.empty(n_pages, hkv, page, d, dtype=E4, device="cuda")
    assert K.numel() > 2 ** 31
    s = torch.ones(n_pages, hkv, device="cuda")
    table = torch.tensor([[0, n_pages - 1, n_pages - 2, 5]], dtype=torch.int32, device="cuda")
    big = lsa.KVCache(K, V, table, s, s.clone())
    small = lsa.make_kv_cache(1, 512, hkv, d, page)
    Kn, Vn, Qn, cu = _new_tokens([500], hkv, 16, d, BF, 60)
    pos = torch.zeros(1, dtype=torch.int64, device="cuda")
    for c in (big, small):
        q, _ = lsa.lsa_cache_write(c, Kn, Vn, cu, pos, Q=Qn, inv_freq=_inv_freq(128))
    for i, pid in enumerate(table[0].tolist()):
        m = min(page, 500 - i * page)
        assert torch.equal(K[pid, :, :m].view(torch.uint8), small.K[i, :, :m].view(torch.uint8))
        assert torch.equal(V[pid, :, :m].view(torch.uint8), small.V[i, :, :m].view(torch.uint8))
    idx, cnt = _selection(np.random.RandomState(61), 1, 4, hkv, 300, 500, [300])
    Q = q[-4:].reshape(1, 4, 16, d).contiguous()
    a, b = lsa.lsa_cache_attn(big, Q, idx, cnt), lsa.lsa_cache_attn(small, Q, idx, cnt)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    assert lsa.lsa_check() == lsa.LSA_OK


def test_two_streams_and_two_replayed_graphs():
    """Two caches served on two streams at once, eagerly and from captured graphs whose inputs change between
    replays, give the bits of calls made one after another."""
    sets = []
    for k in range(2):
        K, V, Q, cu = _new_tokens([9, 30], 2, 8, 128, BF, 70 + k)
        sets.append(dict(cache=_filled(2, 128, 2, 128, 32, E4, 72 + k), K=K, V=V, Q=Q, cu=cu, f=_inv_freq(128),
                         pos=torch.tensor([40, 64], device="cuda"), q=torch.empty_like(Q),
                         O=torch.empty(2, 5, 8, 128, dtype=BF, device="cuda"),
                         lse=torch.empty(2, 5, 8, device="cuda")))
        sets[k]["idx"], sets[k]["cnt"] = _selection(np.random.RandomState(k), 2, 5, 2, 60, 90, [60, 5, 0])

    def step(s):
        lsa.lsa_cache_write(s["cache"], s["K"], s["V"], s["cu"], s["pos"], Q=s["Q"], inv_freq=s["f"], Q_out=s["q"])
        lsa.lsa_cache_attn(s["cache"], s["q"][:10].view(2, 5, 8, 128), s["idx"], s["cnt"], O=s["O"], lse=s["lse"])

    def state(s):
        c = s["cache"]
        return [t.clone() for t in (s["O"], s["lse"], s["q"], c.K.view(torch.uint8), c.V.view(torch.uint8), c.K_scale,
                                    c.V_scale)]

    start = [state(s) for s in sets]

    def reset():
        for s, st in zip(sets, start):
            c = s["cache"]
            for t, v in zip((c.K.view(torch.uint8), c.V.view(torch.uint8), c.K_scale, c.V_scale), st[3:]):
                t.copy_(v)

    want = []
    for s in sets:
        step(s)
        want.append(state(s))
    reset()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    for s, st in zip(sets, streams):
        with torch.cuda.stream(st):
            step(s)
    torch.cuda.synchronize()
    for s, w in zip(sets, want):
        assert all(torch.equal(a, b) for a, b in zip(state(s), w))
    graphs = []
    for s, st in zip(sets, streams):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=st):
            step(s)
        graphs.append(g)
    saved = [s["K"].clone() for s in sets]
    for s in sets:       # other inputs in the same buffers, then the first ones again
        s["K"].mul_(-2)
    for round_ in range(2):
        reset()
        torch.cuda.synchronize()
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
        torch.cuda.synchronize()
        for k, s in enumerate(sets):
            same = all(torch.equal(a, b) for a, b in zip(state(s), want[k]))
            assert same == (round_ == 1)
            s["K"].copy_(saved[k])
        torch.cuda.synchronize()
    assert lsa.lsa_check() == lsa.LSA_OK
    del graphs


# ------------------------------------------------------ the calls as they are used together
def _served(dtype, seed=80, n0=2000, steps=40, hkv=2, hq=8, d=64):
    """A prompt and decode tokens, and a cache they have been written into."""
    lens = [n0, n0]
    K, V, Q, _ = _new_tokens([2 * (n0 + steps)], hkv, hq, d, BF, seed)
    B = 2
    K, V, Q = (t.view(B, n0 + steps, -1, d) for t in (K, V, Q))
    cache = _shuffled_cache(B, n0 + steps, hkv, d, 32, dtype, seed + 1)
    return K, V, Q, cache


@pytest.mark.parametrize("dtype", [E4, BF])
def test_prompt_then_decode_from_the_cache(dtype):
    """Write the prompt, build the index of its rotated keys, then decode: write, index, select, attend.  The index
    and the selections equal, bit for bit, those kept up from dense keys that hold the cache's values; the attention
    is checked against float64 at every step."""
    n0, steps, hkv, hq, d, pool, sink, window, topk = 2000, 40, 2, 8, 64, 4, 8, 64, 256
    K, V, Q, cache = _served(dtype)
    B, f = 2, _inv_freq(d)
    dev = K.device
    cu = torch.tensor([0, n0, 2 * n0], dtype=torch.int64, device=dev)
    flat = lambda t, a, b: t[:, a:b].reshape(-1, t.shape[2], d).contiguous()
    _, k_rot = lsa.lsa_cache_write(cache, flat(K, 0, n0), flat(V, 0, n0), cu, torch.zeros(B, dtype=torch.int64,
                                   device=dev), Q=flat(Q, 0, n0), inv_freq=f, want_K=True)
    ld = n0 + steps
    W = torch.linalg.qr(torch.randn(d, d, generator=_gen(90), device=dev))[0][:, :32].contiguous()
    dense = torch.zeros(B, ld, hkv, d, device=dev)

    def from_cache(a, b):
        """The cache's keys of tokens [a, b) as fp32 [B, b - a, hkv, d]."""
        t = torch.arange(a, b, device=dev)
        pid = cache.page_table[:, t // cache.page].long()
        x = cache.K.view(torch.uint8 if cache.scaled else BF)[pid, :, t % cache.page]
        if not cache.scaled:
            return x.float()
        return x.view(E4).float() * cache.K_scale[pid][..., None]

    dense[:, :n0] = k_rot.view(B, n0, hkv, d).float()
    mk = lambda dt: lsa.make_build_params(B, n0, ld, hkv, d, 32, pool, dt, (8, 64), 3, 0, sink, steps)
    mine = lsa.lsa_build_index(mk(lsa.LSA_BF16), dense.to(BF), W)
    ref = lsa.lsa_build_index(mk(lsa.LSA_F32), dense, W)      # the same keys; fp32, so that it can hold 8-bit values
    sp = lsa.make_select_params(hq, 16, topk, sink, window)
    one = torch.arange(B + 1, dtype=torch.int64, device=dev)
    for i in range(n0, n0 + steps):
        pos = torch.full((B,), i, dtype=torch.int64, device=dev)
        q, _ = lsa.lsa_cache_write(cache, flat(K, i, i + 1), flat(V, i, i + 1), one, pos, Q=flat(Q, i, i + 1),
                                   inv_freq=f)
        lsa.lsa_append_cached(mine, cache, 1)
        if (i + 1) % pool == 0:
            dense[:, i + 1 - pool:i + 1] = from_cache(i + 1 - pool, i + 1)
        lsa.lsa_append(ref, dense, 1)
        q = q.view(B, 1, hq, d)
        idx, cnt = lsa.lsa_select(mine, sp, q, q_pos0=i)
        ridx, rcnt = lsa.lsa_select(ref, sp, q.float(), q_pos0=i)
        assert torch.equal(idx, ridx) and torch.equal(cnt, rcnt)
        Oo, lse = lsa.lsa_cache_attn(cache, q, idx, cnt)
        if i % 8 == 0 or i > n0 + steps - 3:
            _check_attn(cache, q, idx, cnt, Oo, lse)
    assert torch.equal(mine.get(lsa.LSA_GET_LATENT), ref.get(lsa.LSA_GET_LATENT))
    assert torch.equal(mine.get(lsa.LSA_GET_LEAF_OF_BLOCK), ref.get(lsa.LSA_GET_LEAF_OF_BLOCK))
    assert lsa.lsa_check(mine) == lsa.lsa_check(ref) == lsa.lsa_check() == lsa.LSA_OK
    mine.free()
    ref.free()


def test_append_cached_latches_missing_pages():
    K, V, Q, cache = _served(BF, n0=64, steps=16)
    k = K[:, :64].contiguous()
    bp = lsa.make_build_params(2, 64, 80, 2, 64, 16, 4, lsa.LSA_BF16, (4,), 2, 0, 0, 16)
    ix = lsa.lsa_build_index(bp, torch.cat([k, K[:, 64:]], 1).contiguous(), torch.eye(64, device="cuda")[:, :16]
                             .contiguous())
    cache.page_table[1, 2] = -1
    lsa.lsa_append_cached(ix, cache, 4)
    assert lsa.lsa_check(ix) == lsa.LSA_ERR_DEVICE
    with pytest.raises(lsa.LsaError):           # past the append capacity
        lsa.lsa_append_cached(ix, cache, 13)
    ix.free()


def test_decode_steps_replayed_from_a_graph_match_plain_calls():
    """pipeline.CachedDecodeStep against the same calls made one by one on a second index and cache: the same bits at
    every step."""
    n0, steps, hkv, hq, d, pool, sink, window, topk = 1000, 12, 2, 8, 64, 4, 8, 64, 128
    dev, f = "cuda", _inv_freq(d)
    K, V, Q, _ = _served(E4, n0=n0, steps=steps)
    sides = []
    for _ in range(2):
        cache = _shuffled_cache(2, n0 + steps, hkv, d, 32, E4, 5)
        flat = lambda t, a, b: t[:, a:b].reshape(-1, t.shape[2], d).contiguous()
        cu = torch.tensor([0, n0, 2 * n0], dtype=torch.int64, device=dev)
        _, k = lsa.lsa_cache_write(cache, flat(K, 0, n0), flat(V, 0, n0), cu, torch.zeros(2, dtype=torch.int64,
                                   device=dev), inv_freq=f, want_K=True)
        dense = torch.zeros(2, n0 + steps, hkv, d, dtype=BF, device=dev)
        dense[:, :n0] = k.view(2, n0, hkv, d)
        bp = lsa.make_build_params(2, n0, n0 + steps, hkv, d, 32, pool, lsa.LSA_BF16, (8, 32), 3, 0, sink, steps)
        ix = lsa.lsa_build_index(bp, dense, torch.eye(d, device=dev)[:, :32].contiguous())
        sides.append((ix, cache))
    sp = lsa.make_select_params(hq, 16, topk, sink, window)
    max_sel = topk + sink + window
    step = pipeline.CachedDecodeStep(sides[0][0], sp, sides[0][1], hq, max_sel, inv_freq=f)
    one = torch.arange(3, dtype=torch.int64, device=dev)
    for i in range(n0, n0 + steps):
        k, v, q = flat(K, i, i + 1), flat(V, i, i + 1), flat(Q, i, i + 1)
        got = [t.clone() for t in step.step(k, v, q, i)]
        ix, cache = sides[1]
        qr, _ = lsa.lsa_cache_write(cache, k, v, one, torch.full((2,), i, dtype=torch.int64, device=dev), Q=q,
                                    inv_freq=f)
        lsa.lsa_append_cached(ix, cache, 1)
        idx, cnt = lsa.lsa_select(ix, sp, qr.view(2, 1, hq, d), q_pos0=i)
        want = lsa.lsa_cache_attn(cache, qr.view(2, 1, hq, d), idx, cnt)
        assert torch.equal(step.idx, idx) and torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert lsa.lsa_check(sides[0][0]) == lsa.lsa_check() == lsa.LSA_OK
    for ix, _ in sides:
        ix.free()


@pytest.mark.parametrize("page,d,io,dtype,rot,inter", [
    (16, 64, BF, E4, 64, False), (16, 128, F32, BF, 48, True), (32, 128, BF, BF, 80, True), (64, 64, F32, E4, 16, True),
    (64, 128, BF, E4, 128, False), (128, 64, BF, E4, 32, True), (128, 128, F32, E4, 96, False),
    (128, 128, BF, BF, 0, False), (32, 64, F32, BF, 64, False)])
def test_write_of_long_chunks(page, d, io, dtype, rot, inter):
    """Chunks of many pages (the kernel for whole pages), starting inside a page whose scale then grows, several KV
    heads per CTA, query heads that do not fill a group, one sequence without a token."""
    lens, pos0 = [2 * page + 2 ** 21 // page ** 2, 0, 3 * page + 5, 1], [page - 3, 7, 2 * page, 5 * page - 1]
    cache = _shuffled_cache(4, max(lens) + max(pos0) + page, 3, d, page, dtype, 11)
    if cache.scaled:
        for name in "KV":
            p = getattr(cache, name).view(torch.uint8)
            p.copy_(torch.where((p & 0x7f) == 0x7f, p & 0x80, p))
            getattr(cache, name + "_scale").fill_(2.0 ** -12)
    before = _snapshot(cache)
    K, V, Q, cu = _new_tokens(lens, 3, 15, d, io, 12, pad=2)
    pos = torch.tensor(pos0, dtype=torch.int64, device="cuda")
    K_out, Q_out = torch.zeros_like(K), torch.zeros_like(Q)
    lsa.lsa_cache_write(cache, K, V, cu, pos, Q=Q, inv_freq=_inv_freq(rot), interleaved=inter, K_out=K_out, Q_out=Q_out)
    assert lsa.lsa_check() == lsa.LSA_OK
    _check_write(cache, before, K, V, Q, K_out, Q_out, cu, pos, rot, inter)
    assert torch.all(K_out[sum(lens):] == 0) and torch.all(Q_out[sum(lens):] == 0)
    # the same into other pages, in place and without queries
    twin = _shuffled_cache(4, max(lens) + max(pos0) + page, 3, d, page, dtype, 11)
    for a, b in (("K", before["K_codes"]), ("V", before["V_codes"])):
        getattr(twin, a).view(torch.uint8).copy_(b.view(torch.uint8))
        if twin.scaled:
            getattr(twin, a + "_scale").fill_(2.0 ** -12)
    k = K.clone()
    lsa.lsa_cache_write(twin, k, V, cu, pos, inv_freq=_inv_freq(rot), interleaved=inter, K_out=k)
    n = sum(lens)
    assert torch.equal(k[:n], K_out[:n])
    assert torch.equal(twin.K.view(torch.uint8), cache.K.view(torch.uint8))
    assert torch.equal(twin.V.view(torch.uint8), cache.V.view(torch.uint8))


@pytest.mark.parametrize("io,dtype,d,G", [(BF, E4, 128, 8), (BF, BF, 64, 16), (F32, E4, 64, 3), (BF, E4, 64, 1)])
def test_many_short_rows_take_whole_row_warps(io, dtype, d, G):
    """Enough short rows that every warp takes whole ones, an odd number of them; against the same rows a few at a
    time, which CTAs share."""
    nq, hkv = 2501, 3
    c = _filled(1, 400, hkv, d, 32, dtype, 95)
    Q = torch.randn(1, nq, hkv * G, d, generator=_gen(96), device="cuda").to(io)
    idx, cnt = _selection(np.random.RandomState(97), 1, nq, hkv, 50, 400, [50, 0, 1, 17, 33])
    Oo, lse = lsa.lsa_cache_attn(c, Q, idx, cnt)
    assert lsa.lsa_check() == lsa.LSA_OK
    pick = torch.cat([torch.arange(0, 20), torch.arange(1230, 1240), torch.arange(nq - 20, nq)]).cuda()
    few = [t[:, pick].contiguous() for t in (Q, idx, cnt, Oo, lse)]
    _check_attn(c, *few)
    o2, l2 = lsa.lsa_cache_attn(c, *few[:3])
    # the same sums in another order: fp32 roundings of some 50 terms, then the output's
    tol = {BF: 2.0 ** -7, F32: 2.0 ** -16}[io]
    assert torch.all((o2.float() - few[3].float()).abs() <= tol * few[3].float().abs() + 2.0 ** -12)
    assert torch.equal(torch.isinf(l2), torch.isinf(few[4]))


def test_a_long_row_over_a_cluster():
    """One row of 100,003 tokens shared by a cluster of CTAs."""
    c = _filled(1, 131_072, 1, 128, 128, E4, 98)
    for G, io in ((1, BF), (16, BF), (4, F32)):
        Q = torch.randn(1, 1, G, 128, generator=_gen(99), device="cuda").to(io)
        idx, cnt = _selection(np.random.RandomState(98), 1, 1, 1, 100_003, 131_072, [100_003])
        Oo, lse = lsa.lsa_cache_attn(c, Q, idx, cnt)
        assert lsa.lsa_check() == lsa.LSA_OK
        _check_attn(c, Q, idx, cnt, Oo, lse)


def test_calls_on_a_stream_of_their_own():
    """Rotated keys without queries, on a stream given to the calls, with the current stream left alone."""
    K, V, Q, cu = _new_tokens([33, 7], 2, 8, 64, BF, 130)
    pos = torch.zeros(2, dtype=torch.int64, device="cuda")
    f = _inv_freq(64)
    c, ref = (_shuffled_cache(2, 64, 2, 64, 16, E4, 131) for _ in range(2))
    _, want = lsa.lsa_cache_write(ref, K, V, cu, pos, inv_freq=f, want_K=True)
    idx, cnt = _selection(np.random.RandomState(132), 2, 1, 2, 7, 7, [7, 3])
    q = Q[:2].reshape(2, 1, 8, 64).contiguous()
    wO, wl = lsa.lsa_cache_attn(ref, q, idx, cnt)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):               # outputs of the side stream's own
        got, O, lse = torch.empty_like(K), torch.empty_like(q), torch.empty_like(wl)
    none, k = lsa.lsa_cache_write(c, K, V, cu, pos, inv_freq=f, K_out=got, stream=side)
    lsa.lsa_cache_attn(c, q, idx, cnt, O=O, lse=lse, stream=side)
    torch.cuda.synchronize()
    assert none is None and k is got and torch.equal(got, want)
    assert torch.equal(O, wO) and torch.equal(lse, wl)
    assert torch.equal(c.K.view(torch.uint8), ref.K.view(torch.uint8)) and torch.equal(c.K_scale, ref.K_scale)
    assert lsa.lsa_check() == lsa.LSA_OK


@pytest.mark.parametrize("dtype", [E4, BF])
def test_write_again_from_an_earlier_position(dtype):
    """Tokens taken back and written once more leave the pages as they were; shorter ones leave what is behind them."""
    K, V, _, cu = _new_tokens([90], 2, 2, 64, BF, 140)
    f = _inv_freq(64)
    c = _shuffled_cache(1, 96, 2, 64, 32, dtype, 141)
    at = lambda t: torch.tensor([t], device="cuda")
    lsa.lsa_cache_write(c, K, V, cu, at(0), inv_freq=f)
    before = [t.clone().view(torch.uint8) for t in (c.K, c.V)]
    for t, m in ((41, 49), (41, 5), (32, 58), (0, 90), (89, 1)):
        lsa.lsa_cache_write(c, K[t:t + m].contiguous(), V[t:t + m].contiguous(), at(0).repeat(2) + at(0).new_tensor([0, m]),
                            at(t), inv_freq=f)
        assert all(torch.equal(a, b.view(torch.uint8)) for a, b in zip(before, (c.K, c.V))), (t, m)
    assert lsa.lsa_check() == lsa.LSA_OK


@pytest.mark.parametrize("batch,most,page,dtype", [(3001, 3, 16, E4), (1025, 40, 16, E4), (2500, 2, 64, BF), (65535, 1, 16, E4)])
def test_many_sequences(batch, most, page, dtype):
    """More sequences than a CTA looks over: the pages of calls for a few hundred of them each."""
    g = np.random.RandomState(batch)
    lens = g.randint(0, most + 1, batch) if most < 40 else g.randint(10, most, batch)
    n, pad = int(lens.sum()), 5
    K, V, Q, cu = _new_tokens(list(lens), 1, 2, 64, BF, 150, pad=pad)
    cu += 2                                     # padding on both sides
    pos = torch.tensor(g.randint(0, 2 * page, batch), device="cuda")
    f = _inv_freq(64)
    c, ref = (lsa.make_kv_cache(batch, 5 * page, 1, 64, page, dtype=dtype) for _ in range(2))
    q, k = torch.full_like(Q, 7), torch.full_like(K, 7)
    lsa.lsa_cache_write(c, K, V, cu, pos, Q=Q, inv_freq=f, K_out=k, Q_out=q)
    qr, kr = torch.full_like(Q, 7), torch.full_like(K, 7)
    for b0 in range(0, batch, 1000):
        b1 = min(batch, b0 + 1000)
        part = lsa.KVCache(ref.K, ref.V, ref.page_table[b0:b1], ref.K_scale, ref.V_scale)
        lsa.lsa_cache_write(part, K, V, cu[b0:b1 + 1], pos[b0:b1], Q=Q, inv_freq=f, K_out=kr, Q_out=qr)
    assert lsa.lsa_check() == lsa.LSA_OK
    assert torch.equal(q, qr) and torch.equal(k, kr)
    assert torch.all(q[:2] == 7) and torch.all(q[2 + n:] == 7)
    for name in ("K", "V", "K_scale", "V_scale"):
        a, b = getattr(c, name), getattr(ref, name)
        if a is not None:
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8)), name
    bad = cu.clone()                            # a fall somewhere, and an end past the rows
    bad[batch // 2] = n + 2 + pad
    lsa.lsa_cache_write(c, K, V, bad, pos, Q=Q, inv_freq=f, K_out=k, Q_out=q)
    assert lsa.lsa_check() == lsa.LSA_ERR_DEVICE
    bad = cu.clone()
    bad[-1] = n + pad + 1
    lsa.lsa_cache_write(c, K, V, bad, pos, Q=Q, inv_freq=f, K_out=k, Q_out=q)
    assert lsa.lsa_check() == lsa.LSA_ERR_DEVICE
    assert lsa.lsa_check() == lsa.LSA_OK


@pytest.mark.parametrize("lens,page,hkv,hq,d,io,dtype,rot,inter", [
    ([300, 11, 700], 64, 8, 0, 128, BF, E4, 128, False),
    ([10 + i % 11 for i in range(40)], 128, 4, 16, 128, F32, E4, 96, True),
    ([900, 30, 500], 64, 3, 15, 64, BF, BF, 64, False),
    ([19] * 60, 16, 2, 8, 128, F32, BF, 128, False),
    ([12, 9] * 75, 32, 4, 8, 64, BF, E4, 32, True)])
def test_write_by_pages_that_stay_part_empty(lens, page, hkv, hq, d, io, dtype, rot, inter):
    """Enough rows for the kernel that reads them once, few of them in a page, from inside a page on; none of the
    queries, or more of them than side by side."""
    pos0 = [(7 * i + 3) % (2 * page) for i in range(len(lens))]
    cache = _shuffled_cache(len(lens), max(lens) + 3 * page, hkv, d, page, dtype, 160)
    if cache.scaled:
        for name in "KV":
            p = getattr(cache, name).view(torch.uint8)
            p.copy_(torch.where((p & 0x7f) == 0x7f, p & 0x80, p))
            getattr(cache, name + "_scale").fill_(2.0 ** -11)
    before = _snapshot(cache)
    K, V, Q, cu = _new_tokens(lens, hkv, hq, d, io, 161, pad=3)
    pos = torch.tensor(pos0, dtype=torch.int64, device="cuda")
    K_out, Q_out = torch.zeros_like(K), torch.zeros_like(Q) if hq else None
    lsa.lsa_cache_write(cache, K, V, cu, pos, Q=Q, inv_freq=_inv_freq(rot), interleaved=inter, K_out=K_out, Q_out=Q_out)
    assert lsa.lsa_check() == lsa.LSA_OK
    _check_write(cache, before, K, V, Q, K_out, Q_out, cu, pos, rot, inter)
    assert torch.all(K_out[sum(lens):] == 0) and (Q is None or torch.all(Q_out[sum(lens):] == 0))


@pytest.mark.parametrize("nq,G,d", [(3, 8, 64), (2, 16, 128), (1, 5, 64), (2501, 4, 64)])
def test_weights_carry_more_bits_than_the_output(nq, G, d):
    """Two tokens whose values are 1 and -1: O is the difference of two weights that are nearly equal, so that its own
    rounding is small and a weight's would show.  Scores are single products, exact but for the exponent's roundings:
    2^-22 for each of two additions at up to 2^4, the exponential's 2^-22 and the weight's two halves of 11 bits
    (2^-22) are off by less than 2^-20 of a weight together."""
    c = lsa.make_kv_cache(1, 16, 1, d, page=16)
    c.K[0, 0, 0, 0], c.K[0, 0, 1, 0] = 1.0, 1.125
    c.V[0, 0, 0], c.V[0, 0, 1] = 1.0, -1.0
    Q = torch.randn(1, nq, G, d, generator=_gen(170), device="cuda")
    Q[..., 0] = torch.exp2(-5 + 3 * torch.rand(1, nq, G, generator=_gen(171), device="cuda"))
    Q = Q.to(BF)
    idx = torch.tensor([0, 1], dtype=torch.int32, device="cuda").expand(1, nq, 1, 2).contiguous()
    Oo, _ = lsa.lsa_cache_attn(c, Q, idx, torch.full((1, nq, 1), 2, dtype=torch.int32, device="cuda"))
    assert lsa.lsa_check() == lsa.LSA_OK
    want = torch.tanh(-0.125 * Q[..., :1].double() / math.sqrt(d) / 2)
    assert torch.all((Oo.double() - want).abs() <= HALF_STEP[BF] * want.abs() + 2.0 ** -20)


def test_acc_of_long_rows_is_rounded_not_cut_off():
    """Values 1 in a row's first half, -1 in its second, under weights that are no short numbers: acc climbs to half of
    the weights' sum and back, and what every addition cuts off is left over (2.3e-5 where the tensor cores add).
    Scores are single products.  Bounds: a weight 2^-20 as in the test above; acc over the S = 1,563 steps of a warp,
    rounded to nearest once a step, by 2^-24 of half the sum at most, each way alike: six standard deviations of S such
    roundings; the products of a step cut off four times by 2^-23 of them."""
    n, nq, d = 200_000, 300, 64
    c = lsa.make_kv_cache(1, n, 1, d, page=128)
    g = _gen(172)
    c.K[:, 0, :, 0] = (1 + torch.randint(0, 8, (c.K.shape[0], 128), generator=g, device="cuda") / 8.0).to(E4)
    t = torch.arange(c.K.shape[0] * 128, device="cuda").view(-1, 128)
    c.V[:, 0] = torch.where(t < n // 2, 1.0, -1.0)[..., None].to(E4)
    Q = torch.zeros(1, nq, 2, d, device="cuda")
    Q[..., 0] = 0.5 + torch.rand(1, nq, 2, generator=g, device="cuda")
    Q = Q.to(BF)
    idx = torch.arange(n, dtype=torch.int32, device="cuda").expand(1, nq, 1, n).contiguous()
    cnt = torch.full((1, nq, 1), n, dtype=torch.int32, device="cuda")
    Oo, _ = lsa.lsa_cache_attn(c, Q, idx, cnt)
    assert lsa.lsa_check() == lsa.LSA_OK
    w = torch.exp(Q[0, :, :, :1].double() * c.K[:, 0, :, 0].double().flatten()[:n] / math.sqrt(d))
    v = c.V[:, 0, :, 0].double().flatten()[:n]
    want = (w @ v / w.sum(-1))[None, ..., None]
    S = -(-n // (4 * 32))
    tol = 2.0 ** -20 + 6 * math.sqrt(S / 3) * 2.0 ** -25 + 2.0 ** -21
    assert torch.all((Oo.double() - want).abs() <= HALF_STEP[BF] * want.abs() + tol)


@pytest.mark.parametrize("io", [BF, F32])
@pytest.mark.parametrize("nq", [1, 2, 2501])
def test_scores_that_are_all_nan_give_nan(io, nq):
    """A head whose every score is NaN (a NaN among its queries, or among the only key of its row) is no empty row, in
    a row of its own warp, of a CTA or of a cluster."""
    c = _filled(1, 2048, 1, 128, 64, E4, 180)
    Q = torch.randn(1, nq, 4, 128, generator=_gen(181), device="cuda").to(io)
    n = 2048 if nq < 100 else 40
    idx = torch.arange(n, dtype=torch.int32, device="cuda").expand(1, nq, 1, n).contiguous()
    cnt = torch.full((1, nq, 1), n, dtype=torch.int32, device="cuda")
    Q[0, nq - 1, 2, 77] = math.nan
    Oo, lse = lsa.lsa_cache_attn(c, Q, idx, cnt)
    assert torch.isnan(Oo[0, nq - 1, 2]).all() and torch.isnan(lse[0, nq - 1, 2])
    assert torch.isnan(Oo).sum() == 128 and torch.isnan(lse).sum() == 1
    Q[0, nq - 1, 2, 77] = 0
    # one token, its key NaN
    c.K.view(torch.uint8)[int(c.page_table[0, 0]), 0, 5, 9] = 0x7f
    idx[0, nq - 1, 0, 0], cnt[0, nq - 1] = 5, 1
    if nq > 1:
        cnt[0, :nq - 1] = 5                     # without token 5
    Oo, lse = lsa.lsa_cache_attn(c, Q, idx, cnt)
    assert torch.isnan(Oo[0, nq - 1]).all() and torch.isnan(lse[0, nq - 1]).all()
    assert torch.isfinite(Oo[0, :nq - 1].float()).all() and torch.isfinite(lse[0, :nq - 1]).all()
    # the empty row stays what it is
    cnt[0, nq - 1] = 0
    Oo, lse = lsa.lsa_cache_attn(c, Q, idx, cnt)
    assert torch.all(Oo[0, nq - 1] == 0) and torch.all(lse[0, nq - 1] == -math.inf)
    # a run of tokens that one CTA of a cluster takes
    c.K.view(torch.uint8)[c.page_table[0, :2].long()] = 0x7f
    idx[0, :, 0] = torch.arange(n, dtype=torch.int32, device="cuda")
    cnt.fill_(n)
    Oo, lse = lsa.lsa_cache_attn(c, Q, idx, cnt)
    assert torch.isnan(Oo).all() and torch.isnan(lse).all()
    assert lsa.lsa_check() == lsa.LSA_OK


def test_a_bad_count_is_latched_whichever_warp_has_its_row():
    nq, n = 2501, 50
    c = _filled(1, 400, 1, 64, 32, E4, 190)
    Q = torch.randn(1, nq, 4, 64, generator=_gen(191), device="cuda").to(BF)
    idx, cnt = _selection(np.random.RandomState(192), 1, nq, 1, n, 400, [n, 0, 17])
    want = lsa.lsa_cache_attn(c, Q, idx, cnt)
    assert lsa.lsa_check() == lsa.LSA_OK
    for row in (0, 1, 2, 3, 1230, nq - 1):
        for bad in (-1, n + 1, -2 ** 31, 2 ** 31 - 1):
            k, x = cnt.clone(), idx.clone()
            k[0, row], x[0, row] = bad, idx[0, 0]
            Oo, lse = lsa.lsa_cache_attn(c, Q, x, k)
            assert lsa.lsa_check() == lsa.LSA_ERR_DEVICE, (row, bad)
            keep = torch.arange(nq, device="cuda") != row
            assert torch.equal(Oo[0, keep], want[0][0, keep]) and torch.equal(lse[0, keep], want[1][0, keep])
            if bad < 0:                         # clamped
                assert torch.all(Oo[0, row] == 0) and torch.all(lse[0, row] == -math.inf)
    assert lsa.lsa_check() == lsa.LSA_OK


def test_write_whose_shared_memory_just_fits_the_default():
    """127 tokens x 96 turned components and 48 lists a CTA: 49,152 bytes next to what the kernel holds by itself."""
    hkv, hq, d, page, B = 32, 128, 128, 128, 127
    K, V, Q, cu = _new_tokens([1] * B, hkv, hq, d, BF, 200)
    pos = torch.arange(B, device="cuda")
    c, ref = (lsa.make_kv_cache(B, page, hkv, d, page) for _ in range(2))
    q, k = lsa.lsa_cache_write(c, K, V, cu, pos, Q=Q, inv_freq=_inv_freq(96), want_K=True)
    for b in range(0, B, 40):
        e = min(B, b + 40)
        part = lsa.KVCache(ref.K, ref.V, ref.page_table[b:e], ref.K_scale, ref.V_scale)
        qr, kr = lsa.lsa_cache_write(part, K[b:e], V[b:e], cu[:e - b + 1], pos[b:e], Q=Q[b:e], inv_freq=_inv_freq(96),
                                     want_K=True)
        assert torch.equal(q[b:e], qr) and torch.equal(k[b:e], kr)
    for name in ("K", "V", "K_scale", "V_scale"):
        assert torch.equal(getattr(c, name).view(torch.uint8), getattr(ref, name).view(torch.uint8))
    assert lsa.lsa_check() == lsa.LSA_OK


def test_writes_from_two_host_threads():
    """Calls of different sizes from two threads at once: what one asks of the driver does not reach the other's."""
    import threading
    sets = []
    for k, (rot, tokens) in enumerate(((128, 128), (112, 128))):
        lens = [1] * tokens
        K, V, Q, cu = _new_tokens(lens, 2, 4, 128, BF, 210 + k)
        sets.append((lsa.make_kv_cache(tokens, 128, 2, 128, 128), K, V, cu, torch.zeros(tokens, dtype=torch.int64,
                     device="cuda"), Q, _inv_freq(rot), torch.empty_like(Q), torch.cuda.Stream()))
    torch.cuda.synchronize()
    failed = []

    def work(c, K, V, cu, pos, Q, f, Q_out, stream):
        try:
            for _ in range(2000):
                lsa.lsa_cache_write(c, K, V, cu, pos, Q=Q, inv_freq=f, Q_out=Q_out, stream=stream)
        except Exception as e:      # noqa: BLE001
            failed.append(e)

    threads = [threading.Thread(target=work, args=s) for s in sets]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not failed and lsa.lsa_check() == lsa.LSA_OK


def test_appends_from_two_host_threads():
    """Indexes of different widths kept up from two caches by two threads at once."""
    import threading
    n0, steps, jobs, failed = 256, 600, [], []
    for k, (d, r, pool, per) in enumerate(((128, 128, 1, 1), (128, 16, 1, 1), (64, 64, 1, 200))):
        cache = _filled(1, n0 + steps, 1, d, 32, BF, 260 + k)
        dense = torch.randn(1, n0 + steps, 1, d, generator=_gen(261), device="cuda").to(BF)
        W = torch.linalg.qr(torch.randn(d, d, generator=_gen(262), device="cuda"))[0][:, :r].contiguous()
        bp = lsa.make_build_params(1, n0, n0 + steps, 1, d, r, pool, lsa.LSA_BF16, (8,), 2, 0, 0, steps)
        jobs.append((lsa.lsa_build_index(bp, dense, W), cache, per, torch.cuda.Stream()))
    torch.cuda.synchronize()

    def work(ix, cache, per, stream):
        try:
            for _ in range(steps // per):
                lsa.lsa_append_cached(ix, cache, per, stream=stream)
        except Exception as e:      # noqa: BLE001
            failed.append(e)

    threads = [threading.Thread(target=work, args=j) for j in jobs]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    for ix, *_ in jobs:
        assert lsa.lsa_check(ix) in (lsa.LSA_OK, lsa.LSA_ERR_CAPACITY)     # 8 leaves may fill up
        ix.free()
    assert not failed


@pytest.mark.parametrize("io", [BF, F32])
@pytest.mark.parametrize("d,G", [(64, 4), (128, 16)])
@pytest.mark.parametrize("low,high", [(-4, 1), (-10, 0), (-12, 12), (-20, 20), (-50, 50), (-64, 64)])
def test_values_on_pages_of_far_smaller_scales(io, d, G, low, high):
    """Components that only pages of small scales fill, next to pages of large ones whose codes are zero there: each
    component of O is a sum of its own, to the accuracy of the others."""
    page, pages, n = 16, 40, 640
    c = _filled(1, n, 1, d, page, E4, 220)
    lo = torch.rand(pages, generator=_gen(221), device="cuda") < 0.5
    lo[0], lo[1] = True, False
    pid = c.page_table[0].long()
    V = torch.randn(pages, page, d, generator=_gen(222), device="cuda").clamp(-3, 3) * 100
    V[~lo, :, :d // 2] = 0
    V[2] = 0                                    # a page of zeros
    c.V.view(torch.uint8)[pid] = V.to(E4).view(torch.uint8)[:, None]
    c.V_scale[pid, 0] = torch.exp2(torch.where(lo, float(low), float(high)))
    c.V_scale[pid[2], 0] = 2.0 ** -64
    Q = torch.randn(1, 8, G, d, generator=_gen(223), device="cuda").to(io)
    g = np.random.RandomState(224)
    idx, cnt = _selection(g, 1, 8, 1, n, n, [n, 300, 33, 2, 100, 64, 17, 500])
    for i in range(1, 8, 2):                    # in any order
        m = int(cnt[0, i])
        idx[0, i, 0, :m] = idx[0, i, 0, torch.tensor(g.permutation(m), device="cuda")]
    idx[0, 3, 0, :2] = torch.tensor([16, 3])    # one token of each
    Oo, lse = lsa.lsa_cache_attn(c, Q, idx, cnt)
    assert lsa.lsa_check() == lsa.LSA_OK
    k, v = _values(c, "K"), _values(c, "V")
    table, q = c.page_table[0].cpu().numpy(), Q.double().cpu().numpy()
    for i in range(8):
        t = idx[0, i, 0, :int(cnt[0, i])].cpu().numpy()
        kk, vv = k[table[t // page], 0, t % page], v[table[t // page], 0, t % page]
        s = q[0, i] @ kk.T / math.sqrt(d)
        p = np.exp(s - s.max(1, keepdims=True))
        z = np.log(p.sum(1)) + s.max(1)
        p /= p.sum(1, keepdims=True)
        # scores as in _check_attn; weights in 22 bits, or to 2^-28 of the largest; sums of n terms; a weight times its
        # scale is nothing below 2^-125, where the largest is 2^7 at least
        ds = 2.0 ** -24 * (d + 8) * (np.abs(q[0, i]) @ np.abs(kk).T).max(1, keepdims=True) / math.sqrt(d) + 2.0 ** -20
        some = (np.abs(vv) * p.max(1)[:, None, None]).sum(1)
        tol = (p @ np.abs(vv)) * (2 * ds + 2.0 ** -23 * len(t)) + 2.0 ** -28 * some
        sc = c.V_scale[:, 0].double().cpu().numpy()[table[t // page]]
        tol = tol + 2.0 ** -132 * (p * sc).max(1, keepdims=True) * (np.abs(vv) / sc[:, None]).sum(0)
        want = p @ vv
        tol = tol + HALF_STEP[io] * np.abs(want)
        err = np.abs(Oo[0, i].double().cpu().numpy() - want)
        assert np.all(err <= tol), (i, len(t), float((err / np.maximum(tol, 1e-300)).max()))
        assert np.all(np.abs(lse[0, i].cpu().numpy() - z) <= ds[:, 0] + 2.0 ** -23 * (len(t) + np.abs(z)))


@pytest.mark.parametrize("io", [BF, F32])
def test_large_queries_on_keys_of_large_pages_that_are_zero(io):
    """Queries of 2^90 on a page with the largest scale: where the products are zero the scores are, too."""
    c = lsa.make_kv_cache(1, 32, 1, 64, page=16)
    c.K[:, :, 3, 0] = 1.0
    c.K[1, 0, :, 1] = 2.0
    c.K_scale[0], c.K_scale[1] = 2.0 ** 64, 2.0 ** -64
    c.V.copy_(torch.randn(c.V.shape, generator=_gen(230), device="cuda").to(E4))
    Q = torch.zeros(1, 1, 2, 64, device="cuda")
    Q[..., 1] = 2.0 ** 66                       # scores of 0 on page 0, of 2^66 2^-64 2 / 8 = 1 on page 1
    Q[0, 0, 1, 5] = 2.0 ** 90                   # no key has this component
    Q = Q.to(io)
    idx = torch.tensor([[[[1, 3, 17, 19, 30]]]], dtype=torch.int32, device="cuda")
    cnt = torch.full((1, 1, 1), 5, dtype=torch.int32, device="cuda")
    Oo, lse = lsa.lsa_cache_attn(c, Q, idx, cnt)
    _check_attn(c, Q[:, :, :1].contiguous(), idx, cnt, Oo[:, :, :1], lse[:, :, :1])
    assert torch.isfinite(Oo.float()).all() and torch.isfinite(lse).all()


@pytest.mark.parametrize("tokens", [2, 200])
def test_a_sequence_without_a_token_has_no_position(tokens):
    """Idle sequences marked by a position of -1, whether units are tokens or page slots."""
    K, V, _, cu = _new_tokens([tokens], 2, 2, 64, BF, 240)
    c, ref = (lsa.make_kv_cache(3, 256, 2, 64, page=16) for _ in range(2))
    cu = torch.tensor([0, 0, tokens, tokens], dtype=torch.int64, device="cuda")
    for pos, to in (([-1, 5, -1], c), ([0, 5, 0], ref)):
        lsa.lsa_cache_write(to, K, V, cu, torch.tensor(pos, device="cuda"), inv_freq=_inv_freq(64))
        assert lsa.lsa_check() == lsa.LSA_OK
    for name in ("K", "V", "K_scale", "V_scale"):
        assert torch.equal(getattr(c, name).view(torch.uint8), getattr(ref, name).view(torch.uint8))


@pytest.mark.parametrize("io,dtype,d", [(BF, E4, 128), (F32, E4, 64), (BF, BF, 64), (F32, BF, 128)])
@pytest.mark.parametrize("rows", [1, 60, 1000])
def test_every_step_of_a_long_row_reaches_the_output(io, dtype, d, rows):
    """Token j's value is 1 in component (j // 16) % d only, and every score is 0: a component counts the tokens of its
    tiles, of which there are 50 at most, and a tile of 16 tokens left out, taken twice or taken for another is 2 % of
    some component, whose bound is 0.4 %."""
    n = {1: 16 * d * 49, 60: 16 * d * 3, 1000: 8 * d}[rows] + 5
    c = lsa.make_kv_cache(1, n, 1, d, 64, dtype=dtype)
    t = torch.arange(n, device="cuda")
    raw = torch.zeros(n, d, device="cuda")
    raw[t, t // 16 % d] = 1.0
    pages = torch.zeros(c.V.shape[0] * 64, d, device="cuda")
    pages[:n] = raw
    c.V.copy_(pages.view(-1, 1, 64, d).to(dtype))
    Q = torch.randn(1, rows, 3, d, generator=_gen(250), device="cuda").to(io)
    idx = t.int().expand(1, rows, 1, n).contiguous()
    cnt = torch.full((1, rows, 1), n, dtype=torch.int32, device="cuda")
    Oo, lse = lsa.lsa_cache_attn(c, Q, idx, cnt)
    assert lsa.lsa_check() == lsa.LSA_OK
    want = raw.double().sum(0) / n
    # equal weights and small whole numbers: exact sums, one quotient and its rounding
    assert torch.all((Oo.double() - want).abs() <= (HALF_STEP[io] + 2.0 ** -22) * want)
    assert torch.all((lse.double() - math.log(n)).abs() <= 2.0 ** -20)


def test_forms_first_used_inside_a_capture():
    """In a process of its own: one call of the library outside a capture, then writes and attentions of other types and
    sizes, used for the first time while they are captured."""
    import os
    import subprocess
    import sys
    src = """
import torch
from hierarchical_latent_key_gemm_b200 import lsa
assert lsa.lsa_check() == lsa.LSA_OK
def forms():
    for dtype, io, d, n in ((torch.float8_e4m3fn, torch.bfloat16, 128, 1), (torch.float8_e4m3fn, torch.bfloat16, 128, 700),
                            (torch.bfloat16, torch.float32, 64, 130), (torch.float8_e4m3fn, torch.float32, 128, 70)):
        c = lsa.make_kv_cache(2, 1024, 2, d, 128, dtype=dtype)
        g = torch.Generator(device="cuda").manual_seed(d + n)
        K, V, Q = (torch.randn(2 * n, h, d, generator=g, device="cuda").to(io) for h in (2, 2, 8))
        f = 10000.0 ** (-torch.arange(d // 2, dtype=torch.float64, device="cuda") / (d // 2))
        cu = torch.tensor([0, n, 2 * n], device="cuda")
        idx = torch.arange(n, dtype=torch.int32, device="cuda").expand(2, 1, 2, n).contiguous()
        s = dict(c=c, K=K, V=V, Q=Q, f=f, cu=cu, pos=cu[:2] * 0, idx=idx, cnt=torch.full((2, 1, 2), n, dtype=torch.int32,
                 device="cuda"), q=torch.zeros_like(Q), k=torch.zeros_like(K),
                 O=torch.zeros(2, 1, 8, d, dtype=io, device="cuda"), lse=torch.zeros(2, 1, 8, device="cuda"))
        yield s
def call(s):
    lsa.lsa_cache_write(s["c"], s["K"], s["V"], s["cu"], s["pos"], Q=s["Q"], inv_freq=s["f"], Q_out=s["q"], K_out=s["k"])
    lsa.lsa_cache_attn(s["c"], s["q"][:2].view(2, 1, 8, -1), s["idx"], s["cnt"], O=s["O"], lse=s["lse"])
a, b = list(forms()), list(forms())
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    for s in a:
        call(s)
graph.replay()
for s in b:
    call(s)
torch.cuda.synchronize()
for x, y in zip(a, b):
    for name in ("q", "k", "O", "lse"):
        assert torch.equal(x[name], y[name]), name
    assert torch.equal(x["c"].K.view(torch.uint8), y["c"].K.view(torch.uint8))
assert lsa.lsa_check() == lsa.LSA_OK
del graph
print("same")
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    out = subprocess.run([sys.executable, "-c", src], cwd=root, capture_output=True, text=True, timeout=300)
    assert out.returncode == 0 and out.stdout.strip() == "same", out.stderr[-2000:]
