"""Paged KV cache without a GPU: the oracle's 8-bit rounding, the C struct, and
the refusals of the calls (every check comes before any CUDA work)."""
import ctypes as C
import os
import subprocess
import tempfile

import numpy as np
import pytest
import torch

import oracle as O
from hierarchical_latent_key_gemm_b200 import lsa

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BF, E4 = torch.bfloat16, torch.float8_e4m3fn


def test_oracle_rounding_is_the_8_bit_float():
    # every code is its own rounding; halfway points go to the even mantissa
    codes = torch.arange(256, dtype=torch.uint8).view(E4).double().numpy()
    fin = codes[np.isfinite(codes)]
    assert np.array_equal(O.round_e4m3(fin), fin)
    pos = np.unique(fin[fin >= 0])
    mid = (pos[:-1] + pos[1:]) / 2
    got = O.round_e4m3(mid)
    assert np.all((got == pos[:-1]) | (got == pos[1:]))
    even = torch.tensor(got).to(E4).view(torch.uint8).numpy() % 2
    assert np.all(even == 0)
    assert O.round_e4m3(1e9) == 448 and O.round_e4m3(-449) == -448
    assert np.isnan(O.round_e4m3(np.inf)) and np.isnan(O.round_e4m3(np.nan))
    assert O.page_scale([0.0], 448) == 2.0 ** -64 and O.page_scale([448.0], 448) == 1
    assert O.page_scale([448.1, np.inf, np.nan], 448) == 2 and O.page_scale([316.0], 316) == 1
    assert O.page_scale([3e38], 448) == 2.0 ** 64


def test_oracle_rotation_is_a_turn():
    x = np.random.RandomState(0).randn(3, 2, 8)
    for inter in (False, True):
        y = O.rotate(x, [0, 1, 7], [0.5, 0.25], inter)
        assert np.array_equal(y[0], x[0]) and np.array_equal(y[..., 4:], x[..., 4:])
        assert np.allclose((y ** 2).sum(-1), (x ** 2).sum(-1))
        a, b = (2, 3) if inter else (1, 3)
        z = (x[2, :, a] + 1j * x[2, :, b]) * np.exp(1j * 7 * 0.25)
        assert np.allclose(y[2, :, a], z.real) and np.allclose(y[2, :, b], z.imag)


def test_cache_struct_layout_matches_c_header():
    fields = [f[0] for f in lsa.KVCacheDesc._fields_]
    src = ('#include <stddef.h>\n#include <stdio.h>\n#include "lsa.h"\nint main(void) {\n'
           'printf("%zu", sizeof(lsa_kv_cache));\n'
           + "".join(f'printf(" %zu", offsetof(lsa_kv_cache, {f}));\n' for f in fields)
           + 'printf(" %d", (int)LSA_E4M3);\nreturn 0;\n}\n')
    with tempfile.TemporaryDirectory() as td:
        c, exe = os.path.join(td, "t.c"), os.path.join(td, "t")
        open(c, "w").write(src)
        subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), c, "-o", exe], check=True)
        out = subprocess.run([exe], capture_output=True, text=True, check=True).stdout.split()
    want = [C.sizeof(lsa.KVCacheDesc)] + [getattr(lsa.KVCacheDesc, f).offset for f in fields] + [lsa.LSA_E4M3]
    assert [int(x) for x in out] == want


def _pools(n_pages=4, hkv=2, page=16, d=64, dtype=E4):
    return torch.zeros(n_pages, hkv, page, d).to(dtype), torch.zeros(n_pages, hkv, page, d).to(dtype)


def test_cache_refuses_tensors_that_do_not_fit():
    K, V = _pools()
    s, tab = torch.ones(4, 2), torch.zeros(1, 3, dtype=torch.int32)
    cases = [
        (dict(V=V[:3]), "V must have shape"),
        (dict(V=V.to(BF)), "V must be"),
        (dict(K=K.float(), V=V.float()), "pages must be"),
        (dict(K_scale=None), "need K_scale"),
        (dict(V_scale=torch.ones(4, 3)), "V_scale must have shape"),
        (dict(K=K.to(BF), V=V.to(BF)), "no scales"),
        (dict(K=_pools(page=24)[0], V=_pools(page=24)[0]), "pages hold"),
        (dict(K=_pools(d=96)[0], V=_pools(d=96)[0]), "pages hold"),
        (dict(page_table=tab[0]), "page_table"),
        (dict(), "CUDA device"),
    ]
    for over, msg in cases:
        a = dict(K=K, V=V, page_table=tab, K_scale=s, V_scale=s)
        a.update(over)
        with pytest.raises(ValueError, match=msg):
            lsa.KVCache(**a)


def _host_cache(hkv=2, d=64, batch=1):
    """A cache description over no memory: the calls must refuse before they use it."""
    c = lsa.KVCache.__new__(lsa.KVCache)
    c.index, c.batch, c.hkv, c.page, c.d, c.scaled = -1, batch, hkv, 16, d, True
    c.desc = lsa.KVCacheDesc(4, batch, 3, 16, hkv, d, lsa.LSA_E4M3)
    c.ref = C.byref(c.desc)
    return c


def test_cache_write_checks_before_the_call():
    K = torch.zeros(5, 2, 64, dtype=BF)
    Q = torch.zeros(5, 4, 64, dtype=BF)
    cu, pos0 = torch.zeros(2, dtype=torch.int64), torch.zeros(1, dtype=torch.int64)
    f = torch.ones(32, dtype=torch.float64)
    cases = [
        (dict(K=K[0]), "K must have shape"),
        (dict(K=K[:, :1]), "K must have shape"),
        (dict(V=K[:4]), "V must have shape"),
        (dict(V=K.float()), "V must be"),
        (dict(Q=Q[:4]), "Q must have shape"),
        (dict(Q=Q[0]), "Q must have shape"),
        (dict(Q=Q.float()), "Q must be"),
        (dict(Q=None, Q_out=Q), "Q_out without Q"),
        (dict(Q_out=Q[:, :2]), "Q_out must have shape"),
        (dict(K_out=K[:4]), "K_out must have shape"),
        (dict(cu=cu[:1]), "cu must have shape"),
        (dict(cu=cu.int()), "cu must be"),
        (dict(pos0=cu), "pos0 must have shape"),
        (dict(pos0=pos0.int()), "pos0 must be"),
        (dict(inv_freq=f[:7]), "multiple of 16"),
        (dict(inv_freq=torch.ones(40, dtype=torch.float64)), "multiple of 16"),
        (dict(inv_freq=f.view(32, 1)), "inv_freq must have shape"),
        (dict(inv_freq=f.float()), "inv_freq must be"),
        (dict(K=K.half(), V=K.half(), Q=Q.half()), "unsupported dtype"),
        (dict(V=torch.cat([K, K], 2)[..., ::2]), "V must be contiguous"),
    ]
    for over, msg in cases:
        a = dict(K=K, V=K, cu=cu, pos0=pos0, Q=Q, inv_freq=f)
        a.update(over)
        with pytest.raises(ValueError, match=msg):
            lsa.lsa_cache_write(_host_cache(), **a, stream=0)
    c = _host_cache()
    c.index = 0
    with pytest.raises(ValueError, match="K is on cpu, the cache on CUDA device 0"):
        lsa.lsa_cache_write(c, K, K, cu, pos0, stream=0)
    # well-formed, but the cache's own tensors are missing: the library refuses it
    with pytest.raises(lsa.LsaError):
        lsa.lsa_cache_write(_host_cache(), K, K, cu, pos0, stream=0)


def test_cache_attn_checks_before_the_call():
    Q = torch.zeros(1, 3, 4, 64, dtype=BF)
    idx, cnt = torch.zeros(1, 3, 2, 9, dtype=torch.int32), torch.zeros(1, 3, 2, dtype=torch.int32)
    cases = [
        (dict(Q=Q[0]), "Q must be"),
        (dict(Q=torch.zeros(2, 3, 4, 64, dtype=BF)), "Q must have shape"),
        (dict(Q=torch.zeros(1, 3, 4, 128, dtype=BF)), "Q must have shape"),
        (dict(idx=idx[:, :2]), "idx must have shape"),
        (dict(idx=idx[0]), r"idx \[batch, nq, hkv, max_sel\]"),
        (dict(idx=idx.long()), "idx must be"),
        (dict(cnt=cnt[..., None]), "cnt must have shape"),
        (dict(cnt=cnt.long()), "cnt must be"),
        (dict(O=Q.float()), "O must be"),
        (dict(O=Q[:, :2]), "O must have shape"),
        (dict(lse=torch.zeros(1, 3, 2)), "lse must have shape"),
        (dict(lse=torch.zeros(1, 3, 4, dtype=torch.float64)), "lse must be"),
        (dict(Q=Q.half()), "unsupported dtype"),
        (dict(cnt=torch.zeros(1, 3, 4, dtype=torch.int32)[..., ::2]), "cnt must be contiguous"),
    ]
    for over, msg in cases:
        a = dict(Q=Q, idx=idx, cnt=cnt)
        a.update(over)
        with pytest.raises(ValueError, match=msg):
            lsa.lsa_cache_attn(_host_cache(), **a, stream=0)
    with pytest.raises(lsa.LsaError):
        lsa.lsa_cache_attn(_host_cache(), Q, idx, cnt, stream=0)


def test_append_cached_checks_before_the_call():
    bp = lsa.make_build_params(1, 64, 64, 2, 64, 16, 1, lsa.LSA_BF16, (2, 4), 1, 0, 0, 0)
    ix = lsa.Index(C.c_void_p(None), bp)
    for kw in (dict(hkv=1), dict(d=128), dict(batch=2)):
        with pytest.raises(ValueError, match="the cache holds"):
            lsa.lsa_append_cached(ix, _host_cache(**kw), 1)
    with pytest.raises(lsa.LsaError):
        lsa.lsa_append_cached(ix, _host_cache(), 1, stream=0)  # a handle that is not a live index


def test_c_calls_refuse_null_and_bad_caches():
    L = lsa.lib()
    d = _host_cache().desc
    one = C.c_void_p(256)
    inv = lsa.LSA_ERR_INVALID_ARG
    assert L.lsa_cache_attn(None, one, one, one, 1, 4, lsa.LSA_BF16, 9, one, None, None) == inv
    assert L.lsa_cache_write(None, one, one, None, 1, one, one, 0, lsa.LSA_BF16, None, 0, 0, None, None, None) == inv
    assert L.lsa_append_cached(None, C.byref(d), 1, None) == inv
    for k, v in dict(page=24, d=96, hkv=0, batch=0, n_pages=0, ld_pages=0, dtype=lsa.LSA_F32).items():
        bad = lsa.KVCacheDesc.from_buffer_copy(d)
        setattr(bad, k, v)
        assert L.lsa_cache_attn(C.byref(bad), one, one, one, 1, 4, lsa.LSA_BF16, 9, one, None, None) == inv
        assert L.lsa_cache_write(C.byref(bad), one, one, None, 1, one, one, 0, lsa.LSA_BF16, None, 0, 0, None, None,
                                 None) == inv


def test_a_failed_question_to_the_driver_is_asked_again():
    """csrc/ask_once.cuh: answers are kept, zero among them; a failure is not."""
    src = ('#include "ask_once.cuh"\n#include <cstdio>\nint main() {\n'
           '    std::atomic<int> known{0};\n    int asked = 0, answers[] = {-1, -1, 0, 7};\n'
           '    auto ask = [&] { return answers[asked++]; };\n'
           '    for (int i = 0; i < 5; ++i) printf("%d ", lsa::ask_once(known, ask));\n'
           '    printf("%d ", asked);\n    known = 0;\n'
           '    for (int i = 0; i < 2; ++i) printf("%d ", lsa::ask_once(known, ask));\n'
           '    printf("%d\\n", asked);\n    return 0;\n}\n')
    with tempfile.TemporaryDirectory() as td:
        c, exe = os.path.join(td, "t.cpp"), os.path.join(td, "t")
        open(c, "w").write(src)
        subprocess.run(["g++", "-std=c++17", "-I", os.path.join(ROOT, "hierarchical_latent_key_gemm_b200", "csrc"), c,
                        "-o", exe], check=True)
        out = subprocess.run([exe], capture_output=True, text=True, check=True).stdout.split()
    assert out == ["0"] * 5 + ["3"] + ["7", "7"] + ["4"]
