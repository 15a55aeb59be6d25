"""Host-side checks of the cache entries: refusals, and the index rules of the kernels
compiled for the host from their header.  No call here launches GPU work."""
import ctypes
import os
import subprocess

import numpy as np
import pytest
import torch

import attention_forward_fa2_gb300 as fa
from attention_forward_fa2_gb300 import build as fabuild

A = 0x10000      # never-dereferenced addresses
MIS = 0x10008
BAD, UNS, ALI = fa.FA_ERR_INVALID_ARG, fa.FA_ERR_UNSUPPORTED, fa.FA_ERR_ALIGN


@pytest.fixture(scope="module")
def L():
    fabuild.build()
    return fa.lib()


APPEND = dict(k=A, v=A, k_stride=256, v_stride=256, q=A, q_stride=512, q_out=A + 4096, cos=A, sin=A, max_pos=100, rot=64,
              inter=0, k8=A, v8=A, ks=A, vs=A, table=A, lens=A, cu=None, B=2, total=6, max_new=3, H=4, Hk=2, d=128,
              page=16, num_pages=8, width=4, stream=None)
ATTEND = dict(q=A, k8=A, v8=A, ks=A, vs=A, table=A, lens=A, cu=None, o=A, lse=A, B=2, total_q=6, max_q=3, max_k=60, H=4,
              Hk=2, d=128, page=16, num_pages=8, width=4, scale=0.1, causal=1, window=0, sinks=0, ws=A, ws_bytes=1 << 30,
              stream=None)


@pytest.mark.parametrize("kw,code", [
    (dict(B=-1), BAD), (dict(total=5), BAD), (dict(max_new=-1), BAD), (dict(page=24), BAD), (dict(page=256), BAD),
    (dict(rot=24), BAD), (dict(rot=144), BAD), (dict(rot=-16), BAD), (dict(d=96, rot=32), UNS), (dict(k=0), BAD),
    (dict(v8=0), BAD), (dict(ks=0), BAD), (dict(table=0), BAD), (dict(lens=0), BAD), (dict(cos=0), BAD),
    (dict(q_out=None), BAD), (dict(q=None), BAD), (dict(k_stride=248), BAD), (dict(v_stride=0), BAD),
    (dict(q_stride=504), BAD), (dict(q_stride=1024, q_out=A), BAD), (dict(k_stride=260), ALI), (dict(k=MIS), ALI),
    (dict(k8=MIS), ALI), (dict(cos=MIS), ALI), (dict(ks=A + 2), ALI), (dict(cu=A + 1), ALI), (dict(H=70000), BAD),
    (dict(num_pages=-1), BAD), (dict(width=-1), BAD),
])
def test_append_refusals(L, kw, code):
    assert fa.fa_kvcache_append(*dict(APPEND, **kw).values()) == code


@pytest.mark.parametrize("kw", [dict(B=0, total=0), dict(total=0, max_new=0), dict(total=0, cu=A)])
def test_empty_append(L, kw):
    assert fa.fa_kvcache_append(*dict(APPEND, **kw).values()) == fa.FA_OK


@pytest.mark.parametrize("kw,code", [
    (dict(B=-1), BAD), (dict(total_q=7), BAD), (dict(max_k=-1), BAD), (dict(page=8), BAD), (dict(H=3), BAD),
    (dict(Hk=0), BAD), (dict(d=32), UNS), (dict(scale=0.0), BAD), (dict(scale=float("inf")), BAD),
    (dict(window=-1), BAD), (dict(sinks=-1), BAD), (dict(window=8, causal=0), BAD), (dict(q=0), BAD),
    (dict(k8=0), BAD), (dict(vs=0), BAD), (dict(table=0), BAD), (dict(lens=0), BAD), (dict(q=MIS), ALI),
    (dict(v8=MIS), ALI), (dict(ws=MIS), ALI), (dict(lse=A + 2), ALI), (dict(table=A + 2), ALI),
    (dict(num_pages=1 << 28), BAD), (dict(max_k=0x7fffffff, B=1, total_q=3), BAD),
    (dict(max_q=0x7fffffff, B=1, total_q=0x7fffffff, H=1, Hk=1), BAD),
])
def test_attention_refusals(L, kw, code):
    assert fa.fa_fwd_kvcache(*dict(ATTEND, **kw).values()) == code


@pytest.mark.parametrize("kw", [dict(B=0, total_q=0), dict(max_q=0, total_q=0), dict(H=0, Hk=0), dict(cu=A, total_q=0)])
def test_empty_attention(L, kw):
    assert fa.fa_fwd_kvcache(*dict(ATTEND, **kw).values()) == fa.FA_OK


def test_wrappers_refuse_cpu_tensors(L):
    with pytest.raises(ValueError, match="CUDA"):
        fa.KvCache.empty(2, 16, 1, 64, device="cpu")


HARNESS = """
#define FA_HD static inline
#include "fa_kvcache.h"
extern "C" int page_ok(int id, int n) { return fa::kv_page_ok(id, n); }
extern "C" int fits(long long o, long long r, long long n, long long m, long long t, long long w, long long p, long long x) {
  return fa::kv_append_fits(o, r, n, m, t, w, p, x);
}
extern "C" int scale_exp(unsigned bits) { return fa::kv_scale_exp(bits); }
extern "C" int range(int p0, int p1, int w, int s, int* tiles) {
  fa::KvRange r = fa::kv_range(p0, p1, w, s);
  for (int j = 0; j < r.steps; ++j) tiles[j] = j < r.ns ? j : j + r.gap;
  return r.steps;
}
extern "C" int needed(int p0, int p1, int w, int s, int a, int n) {
  return fa::kv_needed(fa::kv_range(p0, p1, w, s), a, n);
}
"""


@pytest.fixture(scope="module")
def rules(tmp_path_factory):
    d = tmp_path_factory.mktemp("rules")
    (d / "r.cpp").write_text(HARNESS)
    subprocess.run(["g++", "-std=c++17", "-shared", "-fPIC", "-O1", "-I", fabuild.CSRC, "-o", str(d / "r.so"), str(d / "r.cpp")],
                   check=True)
    lib = ctypes.CDLL(str(d / "r.so"))
    lib.fits.argtypes = [ctypes.c_longlong] * 8
    return lib


def test_pages_outside_the_cache_are_refused(rules):
    for n in (0, 1, 7):
        for i in (-2 ** 31, -1, 0, n - 1, n, 2 ** 31 - 1):
            assert bool(rules.page_ok(i, n)) == (0 <= i < n)


def test_lengths_that_do_not_fit_are_refused(rules):
    ok = dict(old=10, row0=4, n=3, max_new=5, total=7, width=1, page=16, max_pos=13)
    assert rules.fits(*ok.values())
    for kw in (dict(old=-1), dict(row0=-1), dict(n=-1), dict(n=6, total=99), dict(total=6), dict(old=14, max_pos=-1),
               dict(max_pos=12), dict(old=2 ** 31 - 1, width=2 ** 20), dict(row0=2 ** 31 - 1)):
        assert not rules.fits(*dict(ok, **kw).values()), kw
    assert rules.fits(*dict(ok, old=13, max_pos=-1).values())


def test_scale_is_the_smallest_power_of_two(rules):
    rng = np.random.default_rng(0)
    x = np.concatenate([np.exp2(rng.uniform(-70, 127, 4000)).astype(np.float32),
                        np.float32([448, 224, 449, 447.99997, 448.00003, 0, 1e-45, 3.4028235e38]),
                        (448 * np.exp2(np.arange(-64., 110))).astype(np.float32)])
    for v in x:
        e = rules.scale_exp(int(np.float32(v).view(np.uint32)))
        assert e >= -64 and float(v) <= 448 * 2.0 ** e
        assert e == -64 or float(v) > 448 * 2.0 ** (e - 1)


def test_tiles_walked_are_those_in_sight(rules):
    rng = np.random.default_rng(1)
    out = (ctypes.c_int * 4096)()
    for _ in range(400):
        n = int(rng.integers(1, 3000))
        q = int(rng.integers(1, 40))
        window = int(rng.choice([0, 1, 5, 127, 128, 129, int(rng.integers(1, 3000))]))
        sinks = int(rng.choice([0, 1, 4, 128, 200])) if window else 0
        p0, p1 = n - q, n - 1
        j = np.arange(n)
        seen = np.zeros(n, bool)
        for p in range(p0, p1 + 1):
            seen |= (j <= p) & ((p - j < window) | (j < sinks) if window else True)
        steps = rules.range(p0, p1, window, sinks, out)
        tiles = list(out[:steps])
        assert tiles == sorted(set(tiles))
        want = sorted(set((np.flatnonzero(seen) // 128).tolist()))
        assert set(want) <= set(tiles) and len(tiles) <= len(want) + 0
        for a in range(0, n, 16):
            assert bool(rules.needed(p0, p1, window, sinks, a, 16)) == bool(seen[a:a + 16].any())
    assert rules.range(-5, -1, 0, 0, out) == 0


def test_page_slots_cover_every_new_token_once():
    """The append's items (page of the sequence, slots [s0, s1)) over all lengths near page borders."""
    for page in (16, 32, 64, 128):
        for old in list(range(0, 3 * page, 7)) + [page - 1, page, page + 1]:
            for n in (1, 2, page - 1, page, page + 1, 3 * page + 5):
                touch = (page - 1 + n + page - 1) // page
                seen = []
                for g in range(touch):
                    pg = old // page + g
                    s0, s1 = max(old - pg * page, 0), min(old + n - pg * page, page)
                    seen += [pg * page + s for s in range(s0, s1)]
                assert seen == list(range(old, old + n))
