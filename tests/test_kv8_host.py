"""The 8-bit cache and the per-head norm with rotation on a machine without a
GPU: what the entry points refuse, the kernels' index arithmetic (compiled as
plain C++) and the frequency plan."""
import ctypes
import os
import subprocess
from fractions import Fraction

import numpy as np
import pytest

from conftest import ROOT

CSRC = os.path.join(ROOT, "attention_forward_tk_gb300", "csrc")
A = [(i + 1) << 40 for i in range(16)]  # never-dereferenced addresses far apart
OK, INVALID, UNSUPPORTED = 0, -1, -2


# ------------------------------------------------------------------ refusals


def norm(tk_lib, **kw):
    a = dict(q=A[0], qs=(4096, 64, 256), k=A[1], ks=(4096, 64, 256), qw=A[2], kw=A[3], f32=0,
             turns=A[4], pos=A[5], oq=A[6], ok=A[7], B=2, H=4, Hk=2, N=16, D=64, rot=64, inter=0,
             eps=1e-6)
    a.update(kw)
    return tk_lib.tk_attn_qk_norm_rope_check_args(*a.values())


def test_norm_rope_arguments(tk_lib):
    assert norm(tk_lib) == OK
    assert norm(tk_lib, turns=0, rot=0) == OK and norm(tk_lib, pos=0) == OK
    for kw in (dict(q=0), dict(k=0), dict(qw=0), dict(kw=0), dict(turns=0), dict(oq=0),
               dict(ok=0), dict(B=0), dict(H=0), dict(Hk=-1), dict(N=0), dict(rot=-8),
               dict(rot=72), dict(eps=-1.0), dict(eps=float("nan")), dict(oq=A[0]),
               dict(ok=A[6]), dict(oq=A[1] - 64), dict(ok=A[4])):
        assert norm(tk_lib, **kw) == INVALID, kw
    for kw in (dict(D=96), dict(rot=12), dict(q=A[0] + 8), dict(ok=A[7] + 4), dict(turns=A[4] + 4),
               dict(pos=A[5] + 2), dict(qs=(4096, 64, 252)), dict(ks=(-4096, 64, 256)),
               dict(qw=A[2] + 1), dict(f32=1, qw=A[2] + 2)):
        assert norm(tk_lib, **kw) == UNSUPPORTED, kw


def bwd(tk_lib, **kw):
    need = tk_lib.tk_attn_qk_norm_rope_bwd_workspace_bytes(64)
    a = dict(q=A[0], qs=(4096, 64, 256), k=A[1], ks=(4096, 64, 256), qw=A[2], kw=A[3], f32=0,
             turns=A[4], pos=A[5], gq=A[6], gqs=(4096, 1024, 64), gk=A[7], gks=(2048, 1024, 64),
             dq=A[8], dqs=(4096, 64, 256), dk=A[9], dks=(4096, 64, 256), dqw=A[10], dkw=A[11],
             B=2, H=4, Hk=2, N=16, D=64, rot=64, inter=0, eps=1e-6, ws=A[12], wsb=need)
    a.update(kw)
    return tk_lib.tk_attn_qk_norm_rope_bwd_check_args(*a.values())


def test_norm_rope_bwd_arguments(tk_lib):
    assert tk_lib.tk_attn_qk_norm_rope_bwd_workspace_bytes(96) == 0
    need = tk_lib.tk_attn_qk_norm_rope_bwd_workspace_bytes(64)
    assert bwd(tk_lib) == OK
    fused = (16 * 512, 64, 512)  # [B, N, (4 + 2 + 2) * 64]
    assert bwd(tk_lib, dqs=fused, dk=A[8] + 2 * 256, dks=fused) == OK
    for kw in (dict(gq=0), dict(dq=0), dict(dqw=0), dict(ws=0), dict(wsb=need - 1),
               dict(dq=A[0]), dict(dqw=A[12] + 16), dict(dk=A[6]),
               dict(dqs=(4096, 0, 256)),             # one element written twice
               dict(dqs=(4096, 64, 192)),            # heads run into the next token
               dict(dqs=fused, dk=A[8], dks=fused),  # the same heads
               dict(dqs=fused, dk=A[8] + 2 * 192, dks=fused),
               dict(dqs=fused, dk=A[8] + 2 * 448, dks=fused)):
        assert bwd(tk_lib, **kw) == INVALID, kw
    for kw in (dict(gq=A[6] + 2), dict(dqs=(4096, 64, 250)), dict(dqw=A[10] + 2)):
        assert bwd(tk_lib, **kw) == UNSUPPORTED, kw
    # one token a sequence: the batch stride is the period
    one = dict(N=1, qs=(512, 64, 0), ks=(512, 64, 0), gqs=(256, 64, 0), gks=(128, 64, 0))
    assert bwd(tk_lib, dqs=(512, 64, 0), dk=A[8] + 512, dks=(512, 64, 0), **one) == OK
    assert bwd(tk_lib, dqs=(512, 64, 0), dk=A[8] + 384, dks=(512, 64, 0), **one) == INVALID


GEOM = dict(num_pages=10, page=32, max_pages=4, stride=4)


def write(tk_lib, **kw):
    a = dict(k=A[0], ks=(4096, 64, 128), v=A[1], vs=(4096, 64, 128), kc=A[2], vc=A[3], ke=A[4],
             ve=A[5], table=A[6], start=A[7], counts=0, B=2, H=2, N=16, D=64, **GEOM)
    a.update(kw)
    return tk_lib.tk_attn_kv8_write_check_args(*a.values())


def read(tk_lib, **kw):
    a = dict(kc=A[2], vc=A[3], ke=A[4], ve=A[5], table=A[6], lengths=A[7], k=A[0], v=A[1], B=2,
             H=2, N=16, D=64, **GEOM)
    a.update(kw)
    return tk_lib.tk_attn_kv8_read_check_args(*a.values())


def attend(tk_lib, **kw):
    a = dict(q=A[0], kc=A[2], vc=A[3], ke=A[4], ve=A[5], table=A[6], lengths=A[7], counts=0,
             o=A[8], lse=A[9], B=2, H=4, Hkv=2, Nq=3, D=64, num_pages=10, page=32, max_pages=4,
             stride=4, scale=0.125, causal=1, ws=A[10], wsb=1 << 20)
    a.update(kw)
    return tk_lib.tk_attn_fwd_kv8_check_args(*a.values())


def test_kv8_arguments(tk_lib):
    for f in (write, read, attend):
        assert f(tk_lib) == OK and f(tk_lib, stride=9) == OK
        for kw in (dict(kc=0), dict(vc=0), dict(ke=0), dict(ve=0), dict(table=0), dict(B=0),
                   dict(num_pages=0), dict(max_pages=0), dict(stride=3)):
            assert f(tk_lib, **kw) == INVALID, (f, kw)
        for kw in (dict(D=96), dict(page=48), dict(page=8), dict(page=256), dict(kc=A[2] + 8),
                   dict(table=A[6] + 2), dict(max_pages=1 << 27, stride=1 << 27)):
            assert f(tk_lib, **kw) == UNSUPPORTED, (f, kw)
    for kw in (dict(k=0), dict(start=0), dict(N=0), dict(H=0), dict(kc=A[3]), dict(ke=A[2] + 64),
               dict(k=A[2]), dict(table=A[4] + 16), dict(counts=A[5])):
        assert write(tk_lib, **kw) == INVALID, kw
    for kw in (dict(k=A[0] + 8), dict(vs=(4096, 64, 4)), dict(start=A[7] + 1), dict(B=70000)):
        assert write(tk_lib, **kw) == UNSUPPORTED, kw
    for kw in (dict(lengths=0), dict(v=0), dict(k=A[1] + 64), dict(v=A[2]), dict(N=-1)):
        assert read(tk_lib, **kw) == INVALID, kw
    for kw in (dict(q=0), dict(o=0), dict(lse=0), dict(lengths=0), dict(ws=0), dict(Hkv=3),
               dict(Nq=0), dict(scale=0.0), dict(scale=float("inf")), dict(o=A[0]),
               dict(lse=A[8] + 256), dict(ws=A[3] - 64), dict(o=A[2] + 64)):
        assert attend(tk_lib, **kw) == INVALID, kw
    for kw in (dict(q=A[0] + 8), dict(lse=A[9] + 4), dict(ws=A[10] + 8), dict(lengths=A[7] + 2)):
        assert attend(tk_lib, **kw) == UNSUPPORTED, kw


def test_kv8_without_a_gpu_reports_arch(tk_lib):
    import torch
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    assert tk_lib.tk_attn_kv8_read(A[2], A[3], A[4], A[5], A[6], A[7], A[0], A[1], 2, 2, 16, 64,
                                   10, 32, 4, 4, 0) == tk_lib.TK_ATTN_ERR_ARCH
    assert tk_lib.tk_attn_fwd_kv8_workspace_bytes(2, 4, 2, 3, 64) == 0


def test_binding_raises_when_missing(tk_lib, monkeypatch):
    monkeypatch.setattr(tk_lib, "_binding", None)
    monkeypatch.setattr(tk_lib, "BINDING_PATH", "/nonexistent/_tk_torch.so")
    with pytest.raises(tk_lib.TkAttnError):
        tk_lib.binding()


def test_helpers_refuse_cpu_tensors_and_wrong_shapes(tk_lib):
    import torch
    from attention_forward_tk_gb300.build import build_binding
    build_binding()
    import attention_forward_tk_gb300 as tk
    x = torch.zeros((1, 2, 3, 64), dtype=torch.bfloat16)
    w = torch.ones(64, dtype=torch.bfloat16)
    turns = tk.rope_turns(64, device="cpu")
    with pytest.raises(ValueError):
        tk.qk_norm_rope_forward(x, x, w, w, turns)
    cache = tk.kv8_cache(4, 2, 16, 64, device="cpu")
    table = torch.zeros((1, 2), dtype=torch.int32)
    n = torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError):
        tk.kv8_write(cache, x, x, table, n)
    with pytest.raises(ValueError):
        tk.kv8_read(cache, table, n, n=3)
    with pytest.raises(ValueError):
        tk.attention_forward_kv8(x, cache, table, n)
    with pytest.raises(ValueError):
        tk.rope_turns(12)
    with pytest.raises(ValueError):
        tk.rope_turns(16, inv_freq=[1.0] * 7)


# ------------------------------------------------------------------ index arithmetic

HARNESS = r"""
#include "tk_kv8.h"
using namespace tkattn;
extern "C" {
int rows_of(int max_pages, int page, int start, int count, int N, int *bad) {
  Kv8Geom g{100, 2, page, 64, max_pages, max_pages};
  bool b = false;
  const int n = kv8_write_rows(g, start, count, N, &b);
  *bad = b;
  return n;
}
int length_of(int max_pages, int page, int len, int *bad) {
  Kv8Geom g{100, 2, page, 64, max_pages, max_pages};
  bool b = false;
  const int n = kv8_length(g, len, &b);
  *bad = b;
  return n;
}
int span_of(int N, int page) { return kv8_span(N, page); }
int exponent_of(unsigned bits) { return kv8_exponent(bits); }
long long row_offset(int num_pages, int Hkv, int page, int D, int id, int h, int row) {
  Kv8Geom g{num_pages, Hkv, page, D, 1, 1};
  return kv8_page_ok(g, id) ? kv8_row_offset(g, id, h, row) : -1;
}
}
"""


@pytest.fixture(scope="module")
def index(tmp_path_factory):
    d = tmp_path_factory.mktemp("kv8")
    src = d / "index.cpp"
    src.write_text(HARNESS)
    subprocess.run(["g++", "-O1", "-std=c++17", "-shared", "-fPIC", "-fsanitize=undefined",
                    "-fno-sanitize-recover=undefined", "-I", CSRC, "-o", str(d / "index.so"),
                    str(src)], check=True)
    lib = ctypes.CDLL(str(d / "index.so"))
    lib.row_offset.restype = ctypes.c_longlong
    return lib


@pytest.mark.parametrize("page", [16, 32, 64, 128])
def test_a_write_covers_its_rows_once_inside_the_table(index, page):
    rng = np.random.default_rng(page)
    bad = ctypes.c_int()
    for _ in range(2000):
        mp, N = int(rng.integers(1, 9)), int(rng.integers(1, 300))
        cap = mp * page
        start = int(rng.integers(-20, cap + 40))
        count = int(rng.integers(-3, N + 4))
        n = index.rows_of(mp, page, start, count, N, ctypes.byref(bad))
        c = min(max(count, 0), N)
        want = 0 if c == 0 or start < 0 or start >= cap else min(c, cap - start)
        assert n == want
        assert bool(bad.value) == (count < 0 or count > N or (c > 0 and (
            start < 0 or start + c > cap)))
        covered = []
        for x in range(index.span_of(N, page)):  # the kernel's blocks
            if n == 0:
                break
            first = (start // page + x) * page
            if first >= start + n:
                continue
            assert 0 <= first // page < mp
            covered += range(max(start, first), min(start + n, first + page))
        assert covered == list(range(start, start + n))


def test_lengths_and_rows_stay_inside(index):
    bad = ctypes.c_int()
    for mp, page, n, want in ((4, 16, 64, 64), (4, 16, 65, 64), (4, 16, -1, 0), (4, 16, 0, 0),
                              (1 << 24, 64, (1 << 30) - 1, (1 << 30) - 1),
                              (1 << 24, 64, 2 ** 31 - 1, 1 << 30)):
        assert index.length_of(mp, page, n, ctypes.byref(bad)) == want
        assert bool(bad.value) == (want != n)
    # offsets past 32 bits, and ids that are never followed
    assert index.row_offset(1 << 20, 64, 128, 128, (1 << 20) - 1, 63, 127) == \
        (1 << 20) * 64 * 128 * 128 - 128
    for pid in (-1, 7, 2 ** 31 - 1, -2 ** 31):
        assert index.row_offset(7, 2, 16, 64, pid, 0, 0) == -1
    # the largest write position arithmetic stays in 32 bits
    assert index.rows_of((1 << 25) - 1, 64, (1 << 31) - 200, 1 << 20, 1 << 20,
                         ctypes.byref(bad)) == ((1 << 25) - 1) * 64 - ((1 << 31) - 200)


def test_exponents_of_every_bf16_magnitude(index):
    for bits in list(range(0, 0x7F80, 7)) + [0x7F7F, 0x43E0, 0x43E1, 0x43DF, 1, 0x80, 0x7F]:
        m = Fraction(float(np.array([bits << 16], dtype=np.uint32).view(np.float32)[0]))
        e = index.exponent_of(bits)
        assert -117 <= e <= 119
        assert e == 119 or 448 * Fraction(2) ** e >= m
        assert e == -117 or 448 * Fraction(2) ** (e - 1) < m


def test_rope_turns_are_the_frequencies_in_turns():
    import attention_forward_tk_gb300 as tk
    pi = Fraction(3141592653589793238462643383279502884197169399375105820974944, 10 ** 60)
    for rot, base in ((8, 10000.0), (64, 500000.0), (128, 1e6)):
        t = tk.rope_turns(rot, base, device="cpu").tolist()
        for j, x in enumerate(t):
            want = Fraction(base ** (-2.0 * j / rot)) / (2 * pi)
            got = Fraction(x % (1 << 64), 1 << 64)
            assert abs(got - want % 1) <= Fraction(1, 1 << 65)
    # negative, large and scaled frequencies
    t = tk.rope_turns(8, inv_freq=[-0.5, 7.0, 0.0, 1e-12], device="cpu").tolist()
    for x, f in zip(t, (-0.5, 7.0, 0.0, 1e-12)):
        d = (Fraction(x, 1 << 64) - Fraction(f) / (2 * pi)) % 1
        assert min(d, 1 - d) <= Fraction(1, 1 << 65)
