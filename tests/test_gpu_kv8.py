"""The 8-bit paged cache and attention over it (GPU) against the float64 oracle.

Writing and reading back are exact: codes, exponents and bf16 values are
compared bit for bit.

Bounds of the attention, before any run.  A score is off by `off` (the oracle's:
fp32 sums of D products, and how the kernels hold the queries), so a weight by 2 off relative (its own and the sum's); a weight is rounded to fp16
(half a step 2^-11) and the special-function units' 2^x and the fp32 sums add
less than 2^-16; O is rounded to bf16 (half a step 2^-8):
  |dO| <= 2^-8 |O| + (2^-11 + 2^-16 + 2 off) sum p|v|,
  |dLSE| <= off + 2^-20 (1 + |LSE|)."""
import numpy as np
import pytest
import torch

import attention_forward_tk_gb300 as tk
from oracle import kv8 as ref

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)


def f64(t):
    return t.detach().float().cpu().double().numpy()


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def codes(t):
    return t.view(torch.uint8).cpu().numpy()


def same_codes(got, want):
    """Equal codes, any NaN code for a NaN."""
    nan = (want & 0x7F) == 0x7F
    return np.array_equal(np.where(nan, 0x7F, want), np.where((got & 0x7F) == 0x7F, 0x7F, got))


def make(lengths, H, page, D, seed, spare=3, stale=None, spread=1.0, table_pad=0):
    """A filled cache on the device and the same on the host, pages scattered;
    `stale` fills every code first (what unwritten rows hold)."""
    g = torch.Generator().manual_seed(seed)
    need = [-(-n // page) for n in lengths]
    P = sum(need) + spare
    order = torch.randperm(P, generator=g).tolist()
    width = max(max(need), 1)
    table = torch.full((len(lengths), width + table_pad), -5, dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = torch.tensor(order[at:at + n], dtype=torch.int32)
        at += n
    cache = tk.kv8_cache(P, H, page, D, device=DEV)
    for t in cache[:2]:
        t.view(torch.uint8).fill_(0 if stale is None else stale)
    table = table.to(DEV)[:, :width]
    N = max(max(lengths), 1)
    kv = [(torch.randn((len(lengths), H, N, D), generator=g) * spread).to(torch.bfloat16).to(DEV)
          for _ in range(2)]
    tk.kv8_write(cache, *kv, table, i32([0] * len(lengths)), i32(lengths))
    return cache, table


def host(cache):
    return [codes(cache.k), codes(cache.v), cache.k_exp.cpu().numpy(), cache.v_exp.cpu().numpy()]


# ------------------------------------------------------------------ write and read


@pytest.mark.parametrize("page,D", [(16, 64), (32, 128), (64, 64), (128, 128)])
def test_writes_in_pieces_and_reads_back(tk_lib, page, D):
    B, H = 4, 3
    g = torch.Generator().manual_seed(page)
    width = 5
    P = B * width + 2
    perm = torch.randperm(P, generator=g)[:B * width].reshape(B, width)
    table = i32(perm.tolist())
    cache = tk.kv8_cache(P, H, page, D, device=DEV)
    for t in cache[:2]:
        t.view(torch.uint8).copy_(torch.randint(0, 256, t.shape, generator=g).to(torch.uint8))
    h = host(cache)
    tb = table.cpu().numpy()
    start = np.array([0, 0, 0, 0])
    # pieces of uneven lengths, magnitudes that grow and fall, single tokens, none
    for step, (N, gain) in enumerate(((page + 5, 1.0), (1, 300.0), (7, 0.01), (1, 1.0), (2 * page, 5.0),
                                      (1, 2.0 ** 40), (1, 2.0 ** -60))):
        counts = np.array([N, max(N - 3, 0), N // 2, 0 if step % 2 else N])
        x = [(torch.randn((B, N, H, D), generator=g) * gain).to(torch.bfloat16).to(DEV).transpose(1, 2)
             for _ in range(2)]
        tk.kv8_write(cache, *x, table, i32(start.tolist()), i32(counts.tolist()))
        for c, e, y in ((h[0], h[2], x[0]), (h[1], h[3], x[1])):
            ref.write(c, e, f64(y), tb, start, counts)
        start = start + counts
        got = host(cache)
        for a, b in zip(got, h):
            assert same_codes(a, b) if a.dtype == np.uint8 else np.array_equal(a, b)
    assert tk.last_device_error() == 0
    n = int(start.max()) + 3
    out = [torch.full((B, H, n, D), 7.0, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    tk.kv8_read(cache, table, i32(start.tolist()), out_k=out[0], out_v=out[1])
    for o, c, e in ((out[0], h[0], h[2]), (out[1], h[1], h[3])):
        o = f64(o)
        for b in range(B):
            m = int(start[b])
            assert np.array_equal(o[b, :, :m], ref.read(c, e, tb, b, m))
            assert (o[b, :, m:] == 7.0).all()
    # n shorter than the sequences, allocated by the call
    k, v = tk.kv8_read(cache, table, i32(start.tolist()), n=5)
    assert torch.equal(k, out[0][:, :, :5]) and torch.equal(v, out[1][:, :, :5])


def test_every_magnitude_and_what_is_not_finite(tk_lib):
    D = 64
    bits = torch.arange(0, 65536, dtype=torch.int32)
    x = bits.to(torch.int16).view(torch.bfloat16).reshape(1, 1, 1024, D).to(DEV)
    cache = tk.kv8_cache(64, 1, 16, D, device=DEV)
    table = i32([list(range(64))])
    tk.kv8_write(cache, x, x, table, i32([0]))
    h = [np.zeros((64, 1, 16, D), np.uint8), np.zeros((64, 1), np.int8)]
    ref.write(*h, f64(x), table.cpu().numpy(), [0], None)
    assert same_codes(codes(cache.k), h[0]) and same_codes(codes(cache.v), h[0])
    assert np.array_equal(cache.k_exp.cpu().numpy(), h[1])
    k, _ = tk.kv8_read(cache, table, i32([1024]), n=1024)
    want = ref.read(*h, table.cpu().numpy(), 0, 1024)
    assert np.array_equal(f64(k)[0], want, equal_nan=True)


def test_bad_indices_are_skipped_and_reported(tk_lib):
    page, D, H = 16, 64, 2
    cache = tk.kv8_cache(6, H, page, D, device=DEV)
    for t in cache[:2]:
        t.view(torch.uint8).fill_(0x11)
    before = host(cache)
    x = torch.ones((4, H, 20, D), dtype=torch.bfloat16, device=DEV)
    table = i32([[6, -1], [2 ** 31 - 1, -2 ** 31], [0, 1], [2, 3]])

    def write(start, counts):
        tk.kv8_write(cache, x, x, table, i32(start), i32(counts))
        return tk.last_device_error()

    assert write([0, 0, 0, 0], [20, 20, 0, 0]) == tk_lib.TK_ATTN_ERR_BAD_INDEX
    assert write([0, 0, -1, 32], [0, 0, 4, 1]) == tk_lib.TK_ATTN_ERR_BAD_INDEX
    assert write([0, 0, 0, 2 ** 31 - 1], [0, 0, -7, 20]) == tk_lib.TK_ATTN_ERR_BAD_INDEX
    for a, b in zip(host(cache), before):
        assert np.array_equal(a, b)
    # rows past the table are dropped, the others written
    assert write([0, 0, 30, 0], [0, 0, 20, 0]) == tk_lib.TK_ATTN_ERR_BAD_INDEX
    c = codes(cache.k)
    assert (c[1, :, :14] == 0x11).all() or (c[1, :, 14:] == 0x7E).all()
    assert f64(tk.kv8_read(cache, table, i32([0, 0, 32, 0]), n=32)[0])[2, :, 30:].min() == 1.0
    assert tk.last_device_error() == 0
    out = [torch.full((4, H, 40, D), 7.0, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    tk.kv8_read(cache, table, i32([40, 20, -3, 0]), out_k=out[0], out_v=out[1])
    assert tk.last_device_error() == tk_lib.TK_ATTN_ERR_BAD_INDEX
    assert (out[0] == 7.0).all() and (out[1] == 7.0).all()
    # attention: positions of a bad page count as masked, lengths are clamped
    q = torch.randn((4, 2, 1, D), device=DEV).to(torch.bfloat16)
    o, lse = tk.attention_forward_kv8(q, cache, table, i32([20, 0, 100, -4]))
    assert tk.last_device_error() == tk_lib.TK_ATTN_ERR_BAD_INDEX
    for b in (0, 1, 3):
        assert (o[b] == 0).all() and (lse[b] == -float("inf")).all()
    o2, lse2 = tk.attention_forward_kv8(q, cache, table, i32([0, 0, 32, 0]))
    assert torch.equal(o2[2], o[2]) and torch.equal(lse2[2], lse[2])
    assert tk.last_device_error() == 0


# ------------------------------------------------------------------ attention


def check(q, cache, table, lengths, counts, causal, scale, o, lse, untouched=None):
    ck, cv, ke, ve = host(cache)
    tb = table.cpu().numpy()
    B, H, Nq, D = q.shape
    G = H // cache.k.shape[1]
    Q, O, L = f64(q), f64(o), f64(lse)
    for b in range(B):
        n, m = lengths[b], Nq if counts is None else counts[b]
        k, v = ref.read(ck, ke, tb, b, n), ref.read(cv, ve, tb, b, n)
        see = [max(0, n - (m - 1 - i)) if causal else n for i in range(m)]
        for h in range(H):
            wo, wl, mag, off = ref.attention(Q[b, h, :m], k[h // G], v[h // G], see, scale)
            tol = 2.0 ** -8 * np.abs(wo) + (2.0 ** -11 + 2.0 ** -16 + 2 * off[:, None]) * mag
            err = np.abs(O[b, h, :m] - wo)
            assert (err <= tol + 1e-30).all(), (b, h, (err - tol).max())
            fin = np.isfinite(wl)
            assert np.array_equal(L[b, h, :m][~fin], wl[~fin])
            le = np.abs(L[b, h, :m][fin] - wl[fin])
            assert (le <= off[fin] + 2.0 ** -20 * (1 + np.abs(wl[fin]))).all(), (b, h, le.max())
        if untouched is not None:
            assert (O[b, :, m:] == untouched).all() and (L[b, :, m:] == untouched).all()


CASES = [
    # lengths, Hkv, G, Nq, counts, page, D, causal
    ([1], 1, 1, 1, None, 16, 64, True),
    ([0, 1, 17, 64], 2, 4, 1, None, 16, 128, True),
    ([1000], 8, 4, 1, None, 16, 128, True),
    ([300, 5, 129, 640], 3, 5, 1, None, 64, 128, True),
    ([777, 2000], 1, 16, 1, None, 128, 64, True),
    ([777, 2000], 1, 16, 1, None, 32, 128, False),
    ([513, 40], 2, 32, 1, None, 32, 128, True),     # more rows than one 16-row tile
    ([5, 300, 64], 2, 4, 4, None, 16, 64, True),    # 16 rows, one sequence barely longer
    ([3, 0, 2], 1, 2, 5, None, 16, 128, True),      # rows that see nothing
    ([200, 333, 90], 2, 3, 7, [7, 0, 3], 32, 128, True),
    ([200, 333, 90], 2, 3, 7, [2, 7, 0], 32, 64, False),
    ([260, 700], 2, 4, 130, None, 64, 128, True),   # chunks
    ([260, 700], 4, 1, 200, [200, 129], 16, 64, True),
    ([1100], 1, 8, 300, None, 128, 128, True),
    ([500, 129], 2, 2, 257, [120, 129], 32, 128, False),
    ([100], 2, 1, 300, None, 16, 64, False),        # more queries than positions
    ([100], 2, 1, 300, None, 16, 128, True),
    ([900, 300, 20] * 30, 1, 2, 1, None, 16, 64, True),
    ([33] * 300, 1, 2, 1, None, 16, 64, True),      # more sequences than a scan's width
    ([700] * 3, 2, 7, 40, None, 64, 128, True),
    ([700] * 2, 1, 96, 3, None, 64, 64, True),
    # between one tile of rows and the tensor core's: three to eight tiles of eight
    ([600, 77, 0], 2, 8, 3, None, 16, 64, True),
    ([600, 77, 1], 2, 6, 4, [4, 0, 1], 32, 128, True),
    ([2000, 300], 2, 8, 5, None, 32, 64, True),
    ([2000, 300], 1, 4, 8, [8, 5], 64, 128, False),
    ([900, 130], 2, 7, 9, None, 16, 64, True),
    ([900, 130], 1, 10, 5, None, 128, 128, True),
    # runs that hold many short sequences, of every kernel
    ([33, 300, 1] * 70, 2, 5, 12, None, 128, 64, True),
    ([33, 300, 1] * 70, 2, 10, 6, None, 16, 128, True),
    ([33, 300, 7] * 60, 2, 10, 14, None, 32, 128, True),
    ([33, 300, 1] * 90, 2, 8, 5, None, 32, 64, True),
    # more sequences than the tensor-core kernel has threads; sequences of many units
    ([40, 3] * 350, 1, 6, 5, None, 16, 128, True),
    ([40, 3] * 350, 1, 9, 5, None, 16, 64, False),
    ([700, 1300], 1, 4, 600, [600, 577], 128, 64, True),
    ([700, 10, 1300], 1, 3, 900, [600, 0, 900], 64, 128, True),
    # many rows of few partials each
    ([300, 900, 64, 1] * 16, 8, 4, 1, None, 64, 128, True),
    ([300, 900, 0, 65] * 12, 3, 9, 2, [2, 1, 1, 0] * 12, 16, 128, True),
    # calls without a query or without a position
    ([100, 50], 2, 4, 2, [0, 0], 16, 128, True),
    ([100, 50], 2, 4, 90, [0, 0], 64, 64, True),
    ([0, 0], 1, 32, 3, None, 32, 64, False),
    ([0, 0], 2, 4, 300, None, 32, 128, True),
]


@pytest.mark.parametrize("case", range(len(CASES)))
def test_attention(tk_lib, case):
    lengths, Hkv, G, Nq, counts, page, D, causal = CASES[case]
    cache, table = make(lengths, Hkv, page, D, seed=100 + case, stale=0x7F, table_pad=case % 3)
    g = torch.Generator().manual_seed(case)
    q = (torch.randn((len(lengths), Hkv * G, Nq, D), generator=g) * 2).to(torch.bfloat16).to(DEV)
    o = torch.full_like(q, 7.0)
    lse = torch.full(q.shape[:3], 7.0, device=DEV)
    scale = D ** -0.5
    tk.attention_forward_kv8(q, cache, table, i32(lengths),
                             None if counts is None else i32(counts), causal, out=o, lse=lse)
    assert tk.last_device_error() == 0
    check(q, cache, table, lengths, counts, causal, scale, o, lse, 7.0)
    o2, lse2 = torch.full_like(o, 7.0), torch.full_like(lse, 7.0)
    tk.attention_forward_kv8(q, cache, table, i32(lengths),
                             None if counts is None else i32(counts), causal, out=o2, lse=lse2)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("Nq,G,D", [(1, 4, 128), (2, 8, 128), (5, 8, 64), (7, 9, 64),
                                    (90, 3, 64), (90, 3, 128)])
def test_bad_pages_among_good_ones(tk_lib, Nq, G, D):
    """The positions of a page out of range are masked, wherever it lies."""
    page, H, lengths = 32, 2, [700, 333, 32]
    cache, table = make(lengths, H, page, D, seed=5)
    good = table.clone()
    bad = {0: [0, 7, 20, 21], 1: [9, 10], 2: [0]}  # (the whole of the last sequence)
    for b, slots in bad.items():
        for i, x in enumerate(slots):
            table[b, x] = (-1, cache.k.shape[0], 2 ** 31 - 1, -2 ** 31)[(b + i) % 4]
    q = torch.randn((3, H * G, Nq, D), generator=torch.Generator().manual_seed(2))
    q = q.to(torch.bfloat16).to(DEV)
    o, lse = tk.attention_forward_kv8(q, cache, table, i32(lengths))
    assert tk.last_device_error() == tk_lib.TK_ATTN_ERR_BAD_INDEX
    ck, cv, ke, ve = host(cache)
    tb = good.cpu().numpy()
    for b, n in enumerate(lengths):
        k, v = ref.read(ck, ke, tb, b, n), ref.read(cv, ve, tb, b, n)
        on = np.array([t // page not in bad[b] for t in range(n)])
        # the first positions that each row sees, counted among the good ones
        see = [int(on[:max(0, n - (Nq - 1 - i))].sum()) for i in range(Nq)]
        for h in range(H * G):
            wo, wl, mag, off = ref.attention(f64(q)[b, h], k[h // G][on], v[h // G][on], see,
                                             D ** -0.5)
            tol = 2.0 ** -8 * np.abs(wo) + (2.0 ** -11 + 2.0 ** -16 + 2 * off[:, None]) * mag
            assert (np.abs(f64(o)[b, h] - wo) <= tol + 1e-30).all()
            fin = np.isfinite(wl)
            got = f64(lse)[b, h]
            assert np.array_equal(got[~fin], wl[~fin])
            assert (np.abs(got[fin] - wl[fin]) <=
                    off[fin] + 2.0 ** -20 * (1 + np.abs(wl[fin]))).all()


@pytest.mark.parametrize("Nq,G", [(1, 4), (3, 4), (40, 4)])
def test_pages_of_very_different_magnitude(tk_lib, Nq, G):
    """Exponents from -40 to 20 in one sequence; scores that one key decides."""
    page, D, H, n = 16, 128, 2, 200
    g = torch.Generator().manual_seed(3)
    cache = tk.kv8_cache(20, H, page, D, device=DEV)
    table = i32([list(range(20))])
    gain = 2.0 ** torch.randint(-30, 6, (n // page + 1,), generator=g).repeat_interleave(page)[:n]
    k = torch.randn((1, H, n, D), generator=g) * gain[:, None].clamp(2.0 ** -20, 1.0)
    vg = 2.0 ** torch.randint(-9, 9, (n // page + 1,), generator=g).repeat_interleave(page)[:n]
    v = torch.randn((1, H, n, D), generator=g) * vg[:, None]
    tk.kv8_write(cache, k.to(torch.bfloat16).to(DEV), v.to(torch.bfloat16).to(DEV), table, i32([0]))
    q = (torch.randn((1, H * G, Nq, D), generator=g) * 4).to(torch.bfloat16).to(DEV)
    o, lse = tk.attention_forward_kv8(q, cache, table, i32([n]))
    check(q, cache, table, [n], None, True, D ** -0.5, o, lse)


@pytest.mark.parametrize("Nq,G", [(1, 2), (4, 3), (5, 5), (60, 4), (300, 1)])
@pytest.mark.parametrize("which", ["k", "v"])
def test_nan_in_masked_positions_has_no_effect(tk_lib, Nq, G, which):
    """Rows behind the length, and later positions of the same call, may hold
    NaN codes: rows that do not see them are as without, the others NaN."""
    page, D, H, n = 32, 128, 2, 333
    cache, table = make([n], H, page, D, seed=9)
    q = torch.randn((1, H * G, Nq, D), generator=torch.Generator().manual_seed(2))
    q = q.to(torch.bfloat16).to(DEV)
    o, lse = tk.attention_forward_kv8(q, cache, table, i32([n]))
    # behind the length
    t = getattr(cache, which).view(torch.uint8)
    last = int(table[0, n // page])
    t[last, :, n % page:] = 0xFF
    o1, lse1 = tk.attention_forward_kv8(q, cache, table, i32([n]))
    assert torch.equal(o, o1) and torch.equal(lse, lse1)
    # the last position but one, one value of it: seen by the last two queries
    p = n - 2
    t[int(table[0, p // page]), :, p % page, 5] = 0x7F
    o2, lse2 = tk.attention_forward_kv8(q, cache, table, i32([n]))
    blind = max(Nq - 2, 0)
    assert torch.equal(o[:, :, :blind], o2[:, :, :blind])
    assert torch.equal(lse[:, :, :blind], lse2[:, :, :blind])
    if which == "k":
        assert torch.isnan(o2[:, :, blind:]).all() and torch.isnan(lse2[:, :, blind:]).all()
    else:
        assert torch.isnan(o2[:, :, blind:, 5]).all()
        assert torch.equal(o[..., :5], o2[..., :5]) and torch.equal(o[..., 6:], o2[..., 6:])
        assert torch.equal(lse, lse2)


def test_far_positions_and_shared_pages(tk_lib):
    """A table that repeats its pages: 600,000 positions of which each page holds
    the same 64, so O is the mean over one page's softmax and the sum grows by
    the repeats; byte offsets past 32 bits in a cache of 4.3 GB."""
    page, D, H, n = 64, 128, 1, 600000
    P = (1 << 32) // (page * D) + 3
    cache = tk.kv8_cache(P, H, page, D, device=DEV)
    k = torch.randn((1, H, page, D), generator=torch.Generator().manual_seed(4)).to(torch.bfloat16)
    v = torch.randn((1, H, page, D), generator=torch.Generator().manual_seed(5)).to(torch.bfloat16)
    one = i32([[P - 1]])
    tk.kv8_write(cache, k.to(DEV), v.to(DEV), one, i32([0]))
    q = torch.randn((1, 4, 1, D), generator=torch.Generator().manual_seed(6)).to(torch.bfloat16)
    table = torch.full((1, n // page), P - 1, dtype=torch.int32, device=DEV)
    small = tk.kv8_cache(1, H, page, D, device=DEV)
    for x, y in zip(small, cache):
        x.view(torch.uint8)[0] = y.view(torch.uint8)[P - 1]
    # one query of 4 heads, and 20 of 4 (the tensor core's tiles), all positions visible
    for Nq in (1, 20):
        qn = q.expand(1, 4, Nq, D).contiguous().to(DEV)
        o, lse = tk.attention_forward_kv8(qn, cache, table, i32([n]), causal=False)
        check(qn, small, i32([[0]]), [page], None, False, D ** -0.5,
              o, lse - float(np.log(n // page)))
    kk, vv = tk.kv8_read(cache, one, i32([page]), n=page)
    ks, vs = tk.kv8_read(small, i32([[0]]), i32([page]), n=page)
    assert torch.equal(kk, ks) and torch.equal(vv, vs)


def test_streams_capture_and_workspaces(tk_lib):
    lengths = [700, 64, 1500]
    cache, table = make(lengths, 2, 32, 128, seed=1)
    n = i32(lengths)
    q = torch.randn((3, 8, 1, 128), device=DEV).to(torch.bfloat16)
    want = tk.attention_forward_kv8(q, cache, table, n)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for s in (side, side.cuda_stream, 0):
        got = tk.attention_forward_kv8(q, cache, table, n, stream=s)
        torch.cuda.synchronize()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    # a decode step captured once, replayed while the cache grows
    new_k = torch.randn((3, 2, 1, 128), device=DEV).to(torch.bfloat16)
    new_v = torch.randn((3, 2, 1, 128), device=DEV).to(torch.bfloat16)
    wide = torch.full((3, 50), 0, dtype=torch.int32, device=DEV)
    wide[:, :table.shape[1]] = table
    wide[0, 21] = wide[1, 2] = wide[2, 46] = 0
    P = cache.k.shape[0]
    used = set(int(x) for b, l in enumerate(lengths) for x in table[b, :-(-l // 32)])
    free = [x for x in range(P) if x not in used]
    wide[1, 2] = free[0]  # sequence 1 (64 positions) starts a new page
    start = n.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        tk.kv8_write(cache, new_k, new_v, wide, start)
        start.add_(1)
        got = tk.attention_forward_kv8(q, cache, wide, start)
    for step in range(3):
        new_k.copy_(torch.randn(new_k.shape, device=DEV))
        graph.replay()
        torch.cuda.synchronize()
        now = [x + step + 1 for x in lengths]
        assert start.tolist() == now
        check(q, cache, wide, now, None, True, 128 ** -0.5, *got)
    assert tk.last_device_error() == 0


def test_a_cache_without_heads_is_refused(tk_lib):
    cache = tk.kv8_cache(2, 0, 16, 64, device=DEV)
    q = torch.zeros((1, 4, 1, 64), dtype=torch.bfloat16, device=DEV)
    table, n = i32([[0, 1]]), i32([1])
    with pytest.raises(ValueError):
        tk.attention_forward_kv8(q, cache, table, n)
    with pytest.raises(tk.TkAttnError):
        tk.kv8_write(cache, q[:, :0], q[:, :0], table, n)
    with pytest.raises(tk.TkAttnError):
        tk.kv8_read(cache, table, n, n=4)


def test_refusals(tk_lib):
    cache, table = make([40], 2, 16, 64, seed=1)
    n = i32([40])
    q = torch.zeros((1, 4, 1, 64), dtype=torch.bfloat16, device=DEV)
    x = torch.zeros((1, 2, 1, 64), dtype=torch.bfloat16, device=DEV)
    for f in (lambda: tk.attention_forward_kv8(q[:, :3].contiguous(), cache, table, n),
              lambda: tk.attention_forward_kv8(q.half(), cache, table, n),
              lambda: tk.attention_forward_kv8(q, cache, table.long(), n),
              lambda: tk.attention_forward_kv8(q, cache, table, n.long()),
              lambda: tk.attention_forward_kv8(q, cache, table, n.cpu()),
              lambda: tk.attention_forward_kv8(q, cache, table, n, out=q.float()),
              lambda: tk.attention_forward_kv8(q, cache._replace(k=cache.k.view(torch.uint8)),
                                               table, n),
              lambda: tk.kv8_write(cache, x, x[:, :1], table, n),
              lambda: tk.kv8_write(cache, x, x, table, i32([1, 2])),
              lambda: tk.kv8_read(cache, table, n)):
        with pytest.raises(ValueError):
            f()
    with pytest.raises(tk.TkAttnError):
        tk.attention_forward_kv8(q, cache, table, n, scale=-1.0)
    with pytest.raises(tk.TkAttnError):
        tk.attention_forward_kv8(q, cache, table, n, out=q)
    with pytest.raises(tk.TkAttnError):
        tk.attention_forward_kv8(q, cache, table, n,
                                 workspace=torch.empty(64, dtype=torch.uint8, device=DEV))


# ------------------------------------------------------------------ together


@pytest.mark.parametrize("D,page", [(64, 16), (128, 64)])
def test_a_decoders_steps_together(tk_lib, D, page):
    """Norm and rotation, the cache's write and the attention over it, as a
    decoder runs them: a prompt in two chunks, then single tokens; every step's attention
    against the oracle on what the cache then holds, and the cache against the
    rotated keys."""
    B, H, Hk = 2, 6, 2
    prompt = [150, 90]
    g = torch.Generator().manual_seed(D)
    cache = tk.kv8_cache(2 * 5 * (128 // page) + 1, Hk, page, D, device=DEV)
    width = 5 * (128 // page)
    table = torch.randperm(2 * width, generator=g).reshape(2, width).to(torch.int32).to(DEV)
    qw, kw = ((1 + 0.1 * torch.randn(D, generator=g)).to(torch.bfloat16).to(DEV) for _ in range(2))
    turns = tk.rope_turns(D)
    start = [0, 0]
    keys = [[], []]
    for N in (100, 60, 1, 1, 1):
        counts = [min(N, p - s) if N > 1 else 1 for p, s in zip(prompt, start)]
        counts = [max(c, 0) for c in counts]
        x = torch.randn((B, N, H + 2 * Hk, D), generator=g).to(torch.bfloat16).to(DEV)
        pos = i32(start)[:, None] + torch.arange(N, dtype=torch.int32, device=DEV)
        q, k = tk.qk_norm_rope(x[:, :, :H].transpose(1, 2), x[:, :, H:H + Hk].transpose(1, 2), qw,
                               kw, turns, pos)
        tk.kv8_write(cache, k, x[:, :, H + Hk:].transpose(1, 2), table, i32(start), i32(counts))
        start = [s + c for s, c in zip(start, counts)]
        for b in range(B):
            keys[b].append(k[b, :, :counts[b]])
        o = torch.zeros_like(q)
        lse = torch.zeros(q.shape[:3], device=DEV)
        tk.attention_forward_kv8(q, cache, table, i32(start), i32(counts), out=o, lse=lse)
        check(q, cache, table, start, counts, True, D ** -0.5, o, lse, 0.0)
    kk, _ = tk.kv8_read(cache, table, i32(start), n=max(start))
    for b in range(B):
        want = f64(torch.cat(keys[b], 1))
        # half an E4M3 step (2^-4), twice where an exponent grew; below 2^-6 of the
        # grid's unit the step is absolute: 2^-10 of 448ths of the page's largest, twice
        got = f64(kk[b, :, :start[b]])
        assert (np.abs(got - want) <= 2.0 ** -3 * np.abs(want) + 2.0 ** -16 * np.abs(want).max()).all()
    assert tk.last_device_error() == 0
