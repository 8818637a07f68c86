"""Per-head norm with rotation and its gradients (GPU) against the float64
oracle.

Bounds, before any run: an output is one rounding to bf16 (half a step, 2^-8 of
the value) of an fp32 value; the fp32 value is off by its pair's magnitude
times the errors of sine and cosine (angle held to 2^-25 of a half turn, the
functions to 2^-22) and of a D-term mean and a reciprocal square root, together
below 2^-18 of the row's largest n o w."""
import numpy as np
import pytest
import torch

import attention_forward_tk_gb300 as tk
from oracle import norm_rope as ref

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)


def f64(t):
    return t.detach().float().cpu().double().numpy()


def freqs(rot, base=10000.0):
    return base ** (-2.0 * np.arange(rot // 2) / rot)


def fused(B, N, H, Hk, D, seed, spread=1.0):
    """Query and key heads as views of one token-major projection."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((B, N, H + 2 * Hk, D), generator=g) * spread
    x = x.to(torch.bfloat16).to(DEV)
    return x[:, :, :H].transpose(1, 2), x[:, :, H:H + Hk].transpose(1, 2)


def weights(D, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    return [(1 + 0.3 * torch.randn(D, generator=g)).to(dtype).to(DEV) for _ in range(2)]


def check_out(y, x, w, pos, freq, eps, inter):
    want = ref.norm_rope(f64(x), f64(w), pos, freq, eps, inter)
    y = f64(y)
    nw = f64(x) / np.sqrt((f64(x) ** 2).mean(-1, keepdims=True) + eps) * f64(w)
    tol = 2.0 ** -8 * np.abs(want) + 2.0 ** -18 * np.abs(nw).max(-1, keepdims=True)
    assert (np.abs(y - want) <= tol + 1e-30).all(), np.abs(y - want).max()


CASES = [
    # B, N, H, Hk, D, rot, interleaved, weight type, positions
    (1, 1, 1, 1, 64, 64, False, torch.bfloat16, "none"),
    (1, 1, 1, 1, 128, 128, True, torch.float32, "far"),
    (3, 7, 5, 1, 128, 128, False, torch.bfloat16, "far"),
    (2, 33, 4, 2, 64, 32, True, torch.bfloat16, "random"),
    (2, 129, 32, 8, 128, 64, False, torch.float32, "random"),
    (1, 515, 3, 3, 64, 8, False, torch.bfloat16, "none"),
    (2, 50, 17, 9, 128, 0, False, torch.bfloat16, "none"),
    (1, 1000, 16, 4, 128, 16, True, torch.bfloat16, "random"),
    (70, 1, 32, 8, 128, 128, False, torch.bfloat16, "random"),
]


def positions(kind, B, N, seed):
    if kind == "none":
        return None, np.tile(np.arange(N), (B, 1))
    g = np.random.default_rng(seed)
    hi = 2 ** 31 - 1 if kind == "far" else 5000
    p = g.integers(-hi, hi, (B, N))
    if kind == "far":
        p.flat[0] = 2 ** 31 - 1
        p.flat[-1] = -2 ** 31
    return torch.tensor(p, dtype=torch.int32, device=DEV), p


def plan_freq(rot, kind):
    # at far positions the oracle's own float64 angle (position * frequency) is
    # good to 2^31 * 2^-53 radians
    return freqs(rot)


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c)))
def test_forward_and_gradients(tk_lib, case):
    B, N, H, Hk, D, rot, inter, wt, kind = case
    q, k = fused(B, N, H, Hk, D, seed=N + H)
    qw, kw = weights(D, wt, seed=D)
    turns = tk.rope_turns(rot) if rot else None
    pt, pos = positions(kind, B, N, seed=B)
    freq, eps = plan_freq(rot, kind), 1e-6
    y = tk.qk_norm_rope_forward(q, k, qw, kw, turns, pt, eps, inter)
    for out, x, w in ((y[0], q, qw), (y[1], k, kw)):
        assert out.is_contiguous()
        check_out(out, x, w, pos, freq, eps, inter)
    g = torch.Generator().manual_seed(5)
    dy = [torch.randn(t.shape, generator=g).to(torch.bfloat16).to(DEV) for t in (q, k)]
    # into one fused gradient, its value heads untouched
    fg = torch.full((B, N, H + 2 * Hk, D), 7.0, dtype=torch.bfloat16, device=DEV)
    gq, gk = fg[:, :, :H].transpose(1, 2), fg[:, :, H:H + Hk].transpose(1, 2)
    dq, dk, dqw, dkw = tk.qk_norm_rope_backward(q, k, qw, kw, turns, *dy, pt, eps, inter, dq=gq,
                                                dk=gk)
    assert (fg[:, :, H + Hk:] == 7.0).all()
    for dx, dw, x, w, d in ((dq, dqw, q, qw, dy[0]), (dk, dkw, k, kw, dy[1])):
        x, w, d = f64(x), f64(w), f64(d)
        wx, ww, mag = ref.norm_rope_bwd(x, w, d, pos, freq, eps, inter)
        r = 1 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
        # the fp32 value: r (g w - n mean(g w n)), a D-term mean among it
        gw = np.abs(d).max(-1, keepdims=True) * np.abs(w).max() * 1.5
        n = np.abs(x * r).max(-1, keepdims=True)
        tol = 2.0 ** -8 * np.abs(wx) + 2.0 ** -17 * r * gw * (1 + n)
        assert (np.abs(f64(dx) - wx) <= tol).all(), np.abs(f64(dx) - wx).max()
        # sums in fp32 over a tree of runs: 2^-24 a level, angles to 2^-22
        assert (np.abs(f64(dw) - ww) <= 2.0 ** -17 * mag + 1e-30).all()
    again = tk.qk_norm_rope_backward(q, k, qw, kw, turns, *dy, pt, eps, inter)
    for a, b in zip(again, (dq, dk, dqw, dkw)):
        assert torch.equal(a, b)
    assert tk.last_device_error() == 0


def test_extremes(tk_lib):
    # rows of zeros (eps alone under the root), tiny and huge rows, one NaN row
    x = torch.randn((1, 1, 6, 128), generator=torch.Generator().manual_seed(1))
    x[0, 0, 0] = 0
    x[0, 0, 1] *= 2.0 ** -60
    x[0, 0, 2] *= 2.0 ** 60
    x[0, 0, 4, 5] = float("nan")
    x = x.to(torch.bfloat16).to(DEV)
    qw, kw = weights(128, torch.float32, 3)
    y, _ = tk.qk_norm_rope_forward(x, x, qw, kw, tk.rope_turns(128))
    assert torch.isnan(y[0, 0, 4]).all()
    keep = [0, 1, 2, 3, 5]
    pos = np.array([keep])
    check_out(y[:, :, keep], x[:, :, keep], qw, pos, freqs(128), 1e-6, False)


def test_autograd_against_differences(tk_lib):
    """The function's gradients against central differences of the float64
    forward along random directions, and bf16 weights' gradients in bf16."""
    B, N, H, Hk, D, rot = 2, 9, 3, 1, 64, 32
    q, k = (t.contiguous().requires_grad_() for t in fused(B, N, H, Hk, D, 4))
    qw, kw = (w.requires_grad_() for w in weights(D, torch.bfloat16, 9))
    turns = tk.rope_turns(rot)
    oq, ok = tk.qk_norm_rope(q, k, qw, kw, turns)
    g = torch.Generator().manual_seed(8)
    dq, dk = (torch.randn(t.shape, generator=g).to(torch.bfloat16).to(DEV) for t in (oq, ok))
    torch.autograd.backward((oq, ok), (dq, dk))
    assert qw.grad.dtype == torch.bfloat16
    pos = np.tile(np.arange(N), (B, 1))
    rng = np.random.default_rng(0)

    def loss(x, w, d):
        return float((ref.norm_rope(x, w, pos, freqs(rot), 1e-6, False) * d).sum())

    for x, w, d in ((q, qw, dq), (k, kw, dk)):
        X, W, Dy = f64(x), f64(w), f64(d)
        for arr, grad, other in ((X, f64(x.grad), 0), (W, f64(w.grad), 1)):
            u = rng.standard_normal(arr.shape)
            h = 1e-5
            lo, hi = (loss(X, W + s * h * u, Dy) if other else loss(X + s * h * u, W, Dy)
                      for s in (-1, 1))
            want = (hi - lo) / (2 * h)
            # each gradient element is off by at most 2^-8 of itself plus the fp32 part
            tol = 2.0 ** -8 * float(np.abs(grad * u).sum()) + 1e-3
            assert abs(float((grad * u).sum()) - want) <= tol


def test_streams_capture_and_refusals(tk_lib):
    B, N, H, Hk, D = 2, 40, 4, 2, 128
    q, k = fused(B, N, H, Hk, D, 6)
    qw, kw = weights(D, torch.bfloat16, 2)
    turns = tk.rope_turns(D)
    dy = [torch.randn(t.shape, device=DEV).to(torch.bfloat16) for t in (q, k)]
    want = tk.qk_norm_rope_forward(q, k, qw, kw, turns)
    wantb = tk.qk_norm_rope_backward(q, k, qw, kw, turns, *dy)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for s in (side, side.cuda_stream):
        got = tk.qk_norm_rope_forward(q, k, qw, kw, turns, stream=s)
        gotb = tk.qk_norm_rope_backward(q, k, qw, kw, turns, *dy, stream=s)
        side.synchronize()
        for a, b in zip((*got, *gotb), (*want, *wantb)):
            assert torch.equal(a, b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = tk.qk_norm_rope_forward(q, k, qw, kw, turns)
        gotb = tk.qk_norm_rope_backward(q, k, qw, kw, turns, *dy)
    for t in (*got, *gotb):
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip((*got, *gotb), (*want, *wantb)):
        assert torch.equal(a, b)
    # in place and wrong types, devices and layouts
    flat = torch.randn((1, 2, 3, D), device=DEV).to(torch.bfloat16)
    with pytest.raises(tk.TkAttnError):
        tk.qk_norm_rope_forward(flat, flat, qw, kw, turns, out_q=flat)
    for bad in (dict(q=q.float()), dict(q=q[..., ::2]), dict(k=k[:, :, :-1]), dict(qw=qw[:64]),
                dict(qw=qw.half()), dict(turns=turns.int()),
                dict(positions=torch.zeros((B, N), dtype=torch.int64, device=DEV)),
                dict(positions=torch.zeros((B, N), dtype=torch.int32))):
        a = dict(q=q, k=k, qw=qw, kw=kw, turns=turns, positions=None)
        a.update(bad)
        with pytest.raises(ValueError):
            tk.qk_norm_rope_forward(a["q"], a["k"], a["qw"], a["kw"], a["turns"], a["positions"])


def test_a_training_step_captured(tk_lib):
    """Forward and backward in one graph, replayed on new inputs."""
    B, N, H, Hk, D = 2, 33, 4, 2, 64
    x = torch.randn((B, N, H + Hk, D), device=DEV).to(torch.bfloat16)
    qw, kw = weights(D, torch.float32, 2)
    turns = tk.rope_turns(D)
    dy = [torch.randn(s, device=DEV).to(torch.bfloat16) for s in ((B, H, N, D), (B, Hk, N, D))]

    def step():
        leaf = x.detach().requires_grad_()
        ws = [w.detach().requires_grad_() for w in (qw, kw)]
        q, k = tk.qk_norm_rope(leaf[:, :, :H].transpose(1, 2), leaf[:, :, H:].transpose(1, 2), *ws,
                               turns)
        return (q, k, *torch.autograd.grad((q, k), (leaf, *ws), dy))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for seed in (1, 2):
        x.copy_(torch.randn(x.shape, generator=torch.Generator().manual_seed(seed)))
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, step()):
            assert torch.equal(a, b)


def test_broadcast_gradients(tk_lib):
    """A gradient expanded over heads and tokens is read where it lies."""
    B, N, H, Hk, D = 2, 17, 3, 2, 64
    q, k = fused(B, N, H, Hk, D, 3)
    qw, kw = weights(D, torch.float32, 5)
    turns = tk.rope_turns(D)
    one = torch.randn((B, 1, 1, D), device=DEV).to(torch.bfloat16)
    dy = [one.expand(t.shape) for t in (q, k)]
    got = tk.qk_norm_rope_backward(q, k, qw, kw, turns, *dy)
    want = tk.qk_norm_rope_backward(q, k, qw, kw, turns, *(t.contiguous() for t in dy))
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_gradients_at_odd_addresses(tk_lib):
    """Gradients that autograd hands on as views no 16-byte load could read."""
    q, k = (t.contiguous().requires_grad_() for t in fused(1, 5, 2, 1, 64, 6))
    qw, kw = (w.requires_grad_() for w in weights(64, torch.float32, 7))
    y = tk.qk_norm_rope(q, k, qw, kw, tk.rope_turns(64))
    odd = torch.zeros(1, dtype=torch.bfloat16, device=DEV)
    flat = torch.cat([odd, *(t.flatten() for t in y)])
    dy = torch.randn(flat.shape, device=DEV).to(torch.bfloat16)
    got = torch.autograd.grad(flat, (q, k, qw, kw), dy)
    n = y[0].numel()
    want = tk.qk_norm_rope_backward(q.detach(), k.detach(), qw.detach(), kw.detach(),
                                    tk.rope_turns(64), dy[1:1 + n].clone().view_as(y[0]),
                                    dy[1 + n:].clone().view_as(y[1]))
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_flags_that_are_neither(tk_lib):
    q, k = fused(1, 5, 2, 1, 64, 6)
    qw, kw = weights(64, torch.float32, 7)
    with pytest.raises(RuntimeError):
        tk.qk_norm_rope_forward(q, k, qw, kw, None, interleaved=torch.zeros(2))
