"""Host-side checks of the window entries: argument refusals, workspace sizes and
the rule that names the query blocks of a key block and the key tiles of a query
tile.  No call here launches GPU work."""
import os
import subprocess

import numpy as np
import pytest
import torch

import attention_forward_fa2_gb300 as fa
from attention_forward_fa2_gb300 import build as fabuild

A = 0x10000      # never-dereferenced addresses
MIS = 0x10008


@pytest.fixture(scope="module")
def L():
    fabuild.build()
    return fa.lib()


FWD = dict(q=A, k=A, v=A, o=A, lse=A, B=1, Nq=64, Nk=64, H=4, Hk=2, d=128, scale=0.1, window=16, sinks=2, cu_q=None,
           cu_k=None, total_q=0, total_k=0, stream=None)
BWD = dict(q=A, k=A, v=A, o=A, dout=A, lse=A, dq=A, dk=A, dv=A, B=1, Nq=64, Nk=64, H=4, Hk=2, d=128, scale=0.1,
           window=16, sinks=2, cu_q=None, cu_k=None, total_q=0, total_k=0, ws=A, ws_bytes=1 << 30, stream=None)

REFUSED = [
    (dict(window=0), fa.FA_ERR_INVALID_ARG), (dict(window=-5), fa.FA_ERR_INVALID_ARG),
    (dict(sinks=-1), fa.FA_ERR_INVALID_ARG), (dict(d=96), fa.FA_ERR_UNSUPPORTED),
    (dict(scale=0.0), fa.FA_ERR_INVALID_ARG), (dict(scale=float("nan")), fa.FA_ERR_INVALID_ARG),
    (dict(B=-1), fa.FA_ERR_INVALID_ARG), (dict(Hk=3), fa.FA_ERR_INVALID_ARG), (dict(Hk=0), fa.FA_ERR_INVALID_ARG),
    (dict(cu_q=A), fa.FA_ERR_INVALID_ARG), (dict(cu_q=A, cu_k=A, total_q=-1), fa.FA_ERR_INVALID_ARG),
    (dict(cu_q=A + 2, cu_k=A, total_q=9, total_k=9), fa.FA_ERR_ALIGN), (dict(q=0), fa.FA_ERR_INVALID_ARG),
    (dict(v=MIS), fa.FA_ERR_ALIGN), (dict(lse=A + 2), fa.FA_ERR_ALIGN), (dict(Nk=0), fa.FA_ERR_INVALID_ARG),
    (dict(H=70000, Hk=70000), fa.FA_ERR_INVALID_ARG), (dict(B=40000, Nq=65536), fa.FA_ERR_INVALID_ARG),
    (dict(H=1, Hk=1, Nq=0x7fffffff), fa.FA_ERR_INVALID_ARG), (dict(Nk=0x7fffffff), fa.FA_ERR_INVALID_ARG),
]


@pytest.mark.parametrize("kw,code", REFUSED)
def test_refusals(L, kw, code):
    assert fa.fa_fwd_window(*dict(FWD, **kw).values()) == code
    assert fa.fa_bwd_window(*dict(BWD, **kw).values()) == code


def test_backward_workspace(L):
    def need(B, Nq, Nk, H, Hk, d, window, sinks):
        blocks, kb, skb = -(-Nq // 128), -(-Nk // 128), -(-min(sinks, Nk) // 128)
        chunk = max(4, (min(window, max(Nk, 1)) + 126) // 128 + 1)
        chunks = -(-blocks // chunk)
        units, steps = B * Hk * (skb * chunks + kb - skb), H // Hk * min(blocks, chunk)
        # Parts of a unit: the fewest steps on the busiest of 152 SMs.
        split = min([(-(-units * n // 152) * (-(-steps // n) + 1) + (n > 1) * (2 + units * n // 64), n)
                     for n in range(1, min(8, steps) + 1)] or [(0, 1)])[1]
        rows = chunks * skb + (kb - skb if split > 1 else 0)
        listed = 4 * (units * split + 1) if units * split <= 16384 else 0
        return B * H * blocks * 128 * (d + 2) * 4 + split * B * Hk * rows * 128 * 2 * d * 4 + listed
    for case in ((2, 100, 300, 4, 2, 64, 50, 0), (1, 5000, 5000, 4, 1, 128, 256, 4), (1, 5000, 5000, 4, 1, 128, 256, 300),
                 (3, 0, 40, 2, 2, 64, 9, 4), (1, 700, 700, 2, 2, 128, 10 ** 9, 10 ** 9), (8, 2000, 2000, 8, 8, 64, 100, 1)):
        assert fa.bwd_window_workspace_bytes(*case) == need(*case), case
    n = need(1, 64, 64, 4, 2, 128, 16, 2)
    assert fa.fa_bwd_window(*dict(BWD, ws_bytes=n - 1).values()) == fa.FA_ERR_INVALID_ARG
    assert fa.fa_bwd_window(*dict(BWD, ws=0, ws_bytes=n).values()) == fa.FA_ERR_INVALID_ARG
    assert fa.fa_bwd_window(*dict(BWD, ws=MIS).values()) == fa.FA_ERR_ALIGN
    with pytest.raises(fa.FaError):
        fa.bwd_window_workspace_bytes(1, 64, 64, 4, 2, 128, 0, 2)


def test_empty_calls_are_noops(L):
    for kw in (dict(B=0), dict(H=0, Hk=0), dict(Nq=0)):
        assert fa.fa_fwd_window(*dict(FWD, **kw).values()) == fa.FA_OK
    for kw in (dict(B=0), dict(Nq=0, Nk=0), dict(cu_q=A, cu_k=A, total_q=0, total_k=0)):
        assert fa.fa_bwd_window(*dict(BWD, **kw).values()) == fa.FA_OK


def test_wrapper_refuses_cpu_tensors(L):
    q = torch.zeros(1, 8, 1, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        fa.forward_window(q, q, q, 4)


HARNESS = r"""
#define __host__
#define __device__
#define __forceinline__ inline
#include <algorithm>
using std::min;
static const int kBwdBK = 128, kBwdBQ = 128;
%s
struct WinSteps { int s, a, e; };
%s
extern "C" void query_blocks(int kb, int len_q, int len_k, int window, int sink, int* out) {
  win_query_blocks(kb, len_q, len_k, window, sink != 0, out[0], out[1]);
}
extern "C" int sees(int lo, int hi, int nsk, int ns, int gap, int j) {
  return win_sees(win_steps(lo, hi, nsk, ns, gap), j);
}
extern "C" int last(int lo, int hi, int nsk, int ns, int gap, int j0, int j1) {
  return win_last(win_steps(lo, hi, nsk, ns, gap), j0, j1);
}
"""


def _function(path, name):
    src = open(os.path.join(fabuild.CSRC, path)).read()
    at = src.index(name)
    at = src.rindex("__host__", 0, at)
    return src[at:src.index("\n}\n", at) + 3]


def test_blocks_walked_are_those_that_hold_a_visible_pair(tmp_path):
    """The index rules of the kernels, compiled for the host from their source, against the mask."""
    import ctypes
    code = HARNESS % (_function("fa_win_bwd_kernel.cuh", "win_query_blocks("), "".join(
        _function("fa_win_kernel.cuh", name) for name in ("WinSteps win_steps(", "bool win_sees(")))
    (tmp_path / "w.cpp").write_text(code)
    so = str(tmp_path / "w.so")
    subprocess.run(["g++", "-shared", "-fPIC", "-O1", "-o", so, str(tmp_path / "w.cpp")], check=True)
    lib = ctypes.CDLL(so)
    out = (ctypes.c_int * 2)()
    rng = np.random.default_rng(5)
    for _ in range(300):
        n_k = int(rng.integers(1, 1500))
        n_q = int(rng.integers(1, 1500))
        window = int(rng.integers(1, 700))
        sinks = int(rng.choice([0, 1, 4, 130, 300]))
        window, sinks = min(window, n_k), min(sinks, n_k)
        p = np.arange(n_q)[:, None] + n_k - n_q
        j = np.arange(n_k)[None]
        mask = (j <= p) & ((p - j < window) | (j < sinks))
        for kb in range(-(-n_k // 128)):
            cols = mask[:, kb * 128:kb * 128 + 128]
            rows = np.flatnonzero(cols.any(1))
            sink = kb * 128 < sinks
            lib.query_blocks(kb, n_q, n_k, window, int(sink), out)
            got = set(range(out[0], out[0] + out[1]))
            assert all(0 <= b < -(-n_q // 128) for b in got)
            assert set((rows // 128).tolist()) <= got
            if len(rows) and not sink:  # tight: no block without a visible pair but at the ends
                assert len(got) <= len(set((rows // 128).tolist())) + 1
        # Forward: the steps of a unit of two query tiles, and which of them each takes part in.
        nsk = -(-sinks // 128)
        for u in range(-(-n_q // 256)):
            tiles = []
            for t in (2 * u, 2 * u + 1):
                r = np.arange(t * 128, min(n_q, t * 128 + 128)) + n_k - n_q
                if len(r) and r[-1] >= 0:
                    tiles.append((t, max(0, int(r[0]) - window + 1) // 128, int(r[-1]) // 128))
            if not tiles:
                continue
            first, end = min(t[1] for t in tiles), max(t[2] for t in tiles)
            ns = min(nsk, first)
            gap = first - ns
            steps = ns + end - first + 1
            for t, lo, hi in tiles:
                on = []
                for j in range(steps):
                    kt = j if j < ns else j + gap
                    any_seen = bool(mask[t * 128:t * 128 + 128, kt * 128:kt * 128 + 128].any())
                    assert bool(lib.sees(lo, hi, nsk, ns, gap, j)) == any_seen
                    on.append(any_seen)
                covered = [j if j < ns else j + gap for j in range(steps) if on[j]]
                want = [kt for kt in range(-(-n_k // 128)) if mask[t * 128:t * 128 + 128, kt * 128:kt * 128 + 128].any()]
                assert covered == want
                for j0 in range(0, steps, 3):
                    for j1 in (j0 + 1, steps):
                        got = [j for j in range(j0, j1) if on[j]]
                        assert lib.last(lo, hi, nsk, ns, gap, j0, j1) == (got[-1] if got else -1)
