"""The serving and training operators around attention, as cases that can be timed and checked.

Three operators that belong together in a decoder whose cache is held in 8 bits:

  norm_rope   the RMS norm of each head's query and key with the position rotation in the same
              pass, and its gradients
  kv_write,   quantising keys and values into a paged cache as they are written (E4M3 payload, one
  kv_read     power-of-two scale for each page and head), and reading the cache back
  attend      attention over that cache: decode, several query rows a sequence, prefill chunks

``run`` computes a case either in plain torch operations (``own`` false) or through the calls a
user of this package makes (``own`` true).  ``exact`` gives the same outputs from the operators'
definitions in 64 bits.

The cache's format.  A page holds ``page`` consecutive positions of one sequence for every
key/value head: payload [pages, heads, page, D] in E4M3, exponents [pages, heads] in int8; the
value held is payload * 2^exponent.  A page's exponent is the least e >= -117 with
448 * 2^e >= the largest finite magnitude written to it (at most 119), and never falls while rows
already in the page stay: if a later write needs a larger one, the rows already there are rounded
again onto the new grid.
"""
import math

import torch

own = False

E4M3 = torch.float8_e4m3fn
EXP_MIN, EXP_MAX = -117, 119


def listed():
    return [
        # one token for each of 8 sequences: the smallest call of a serving loop
        dict(name="norm_rope decode b8", op="norm_rope", B=8, N=1, H=32, Hkv=8, D=128, rot=128,
             interleaved=False, far=16384, backward=False),
        # a prompt's projection, 4 x 4096 tokens, query and key heads inside one fused projection
        dict(name="norm_rope prompt 4x4096", op="norm_rope", B=4, N=4096, H=32, Hkv=8, D=128,
             rot=128, interleaved=False, far=0, backward=False),
        # a training step at 16 x 1024 tokens, half of each head rotated: forward and gradients
        dict(name="norm_rope train 16x1024", op="norm_rope", B=16, N=1024, H=16, Hkv=16, D=64,
             rot=32, interleaved=True, far=0, backward=True),
        # the decode loop's append: one token for each of 64 sequences at ragged positions
        dict(name="kv_write append b64", op="kv_write", B=64, N=1, Hkv=8, D=128, page=64,
             longest=1024, ragged=True),
        # prompts of up to 4096 tokens written at once, behind what the cache already holds
        dict(name="kv_write prompts 8x4096", op="kv_write", B=8, N=4096, Hkv=8, D=128, page=64,
             longest=8192, ragged=True),
        # one short sequence handed back in bf16 (a prefix given to the dense attention calls)
        dict(name="kv_read 1x1000", op="kv_read", B=1, Hkv=8, D=64, page=16, longest=1000,
             ragged=False),
        # eight long sequences read back
        dict(name="kv_read 8x16384", op="kv_read", B=8, Hkv=8, D=128, page=64, longest=16384,
             ragged=True),
        # one sequence, one query: latency
        dict(name="attend decode 1x1000", op="attend", B=1, N=1, H=32, Hkv=8, D=128, page=16,
             longest=1000, ragged=False),
        # 8 sequences of 16K keys, every query head with its own keys
        dict(name="attend decode 8x16384 mha", op="attend", B=8, N=1, H=32, Hkv=32, D=128, page=64,
             longest=16384, ragged=False),
        # a serving batch of ragged lengths, four query heads for each key head
        dict(name="attend decode 32x32768 gqa", op="attend", B=32, N=1, H=32, Hkv=8, D=128,
             page=64, longest=32768, ragged=True),
        # a few drafted tokens checked at once for each of 16 sequences
        dict(name="attend drafts 16x5", op="attend", B=16, N=5, H=16, Hkv=2, D=64, page=32,
             longest=16384, ragged=True),
        # a prompt's chunk of 2048 behind 14336 positions that the cache holds
        dict(name="attend chunk 2048x16384", op="attend", B=1, N=2048, H=32, Hkv=8, D=128, page=64,
             longest=16384, ragged=False),
    ]


def _spread(rng, lo, hi):
    """A whole number between lo and hi, even over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    most = {c["op"]: [work(d) for d in listed() if d["op"] == c["op"]] for c in listed()}
    op = rng.choice(["norm_rope", "kv_write", "kv_read", "attend", "attend"])
    while True:
        D = rng.choice([64, 128])
        Hkv = rng.choice([1, 2, 3, 4, 8, 16, 32])
        page = rng.choice([16, 32, 64, 128])
        if op == "norm_rope":
            c = dict(op=op, B=_spread(rng, 1, 64), N=_spread(rng, 1, 16384),
                     H=Hkv * rng.choice([1, 2, 4, 5, 8]), Hkv=Hkv, D=D,
                     rot=rng.choice([D, D, D // 2, D // 4]), interleaved=rng.random() < 0.4,
                     far=rng.choice([0, 1, 1000, 131072, 1 << 20]), backward=rng.random() < 0.5)
        elif op == "kv_write":
            c = dict(op=op, B=_spread(rng, 1, 64), N=_spread(rng, 1, 8192), Hkv=Hkv, D=D, page=page,
                     longest=_spread(rng, 256, 16384), ragged=rng.random() < 0.7)
            c["N"] = min(c["N"], c["longest"])
        elif op == "kv_read":
            c = dict(op=op, B=_spread(rng, 1, 32), Hkv=Hkv, D=D, page=page,
                     longest=_spread(rng, 16, 65536), ragged=rng.random() < 0.7)
        else:
            kind = rng.choice(["decode", "decode", "drafts", "chunk"])
            n = {"decode": 1, "drafts": rng.randint(2, 16), "chunk": _spread(rng, 17, 4096)}[kind]
            c = dict(op=op, B=_spread(rng, 1, 64), N=n, H=Hkv * rng.choice([1, 2, 4, 5, 8, 16]),
                     Hkv=Hkv, D=D, page=page, longest=_spread(rng, max(n, 64), 65536),
                     ragged=rng.random() < 0.7)
        w = work(c)
        if c["op"] != "norm_rope" and c["B"] * c["longest"] * c["Hkv"] * c["D"] > 1.3e9:
            continue
        # scores of the plain form, which holds them whole
        if op == "attend" and c["B"] * c["H"] * c["N"] * c["longest"] > 1.2e9:
            continue
        if all(w[k] <= max(x[k] for x in most[op]) for k in ("bytes", "flops")):
            return c


# ------------------------------------------------------------------ inputs


def _lengths(case, new):
    """(keys held, query rows) of each sequence: deterministic, so that a case has one amount of
    work; ragged lengths are spread evenly down from the longest, in a scattered order."""
    B, longest = case["B"], case["longest"]
    held, rows = [], []
    for b in range(B):
        f = ((b * 7 + 3) % B + 1) / B if case["ragged"] else 1.0
        n = max(1, int(new * f)) if new > 1 and case["op"] == "kv_write" else new
        held.append(max(n, int(round(longest * f)) if f < 1 else longest))
        rows.append(n)
    return held, rows


def _pages_of(held, page):
    return [-(-n // page) for n in held]


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _keys(shape, g, outlier):
    """bf16 rows as projections give them: near normal, with a few channels far larger."""
    x = torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)
    gain = torch.ones(shape[-1], device="cuda")
    gain[:: shape[-1] // 4] = outlier
    return (x * gain).to(torch.bfloat16)


def _cache(case, held, g, fill):
    """A cache with room for `held` positions of each sequence, its pages scattered: payloads and
    exponents of what `fill` positions of each hold."""
    Hkv, D, page = case["Hkv"], case["D"], case["page"]
    need = _pages_of(held, page)
    total = sum(need) + 7
    order = torch.randperm(total, generator=g, device="cuda").to(torch.int32)
    table = torch.zeros((len(held), max(need)), dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    out = []
    for outlier in (6.0, 2.0):  # keys, values
        x = torch.empty((total, Hkv, page, D), dtype=E4M3, device="cuda")
        e = torch.empty((total, Hkv), dtype=torch.int8, device="cuda")
        step = max(1, (1 << 26) // (Hkv * page * D))
        for i in range(0, total, step):
            y = _keys((min(step, total - i), Hkv, page, D), g, outlier).float()
            m = y.abs().amax((2, 3))
            x[i:i + step], e[i:i + step] = _to_grid(y, _exponent(m))
        out += [x, e]
    k, ke, v, ve = out
    return dict(k=k, v=v, k_exp=ke, v_exp=ve, table=table)


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    s = dict(case=case)
    if op == "norm_rope":
        B, N, H, Hkv, D, rot = (case[x] for x in ("B", "N", "H", "Hkv", "D", "rot"))
        # one fused projection: [tokens, (queries, keys, values) heads, D], as a linear layer gives it
        x = torch.randn((B, N, H + 2 * Hkv, D), generator=g, device="cuda") * 1.7
        x = x.to(torch.bfloat16)
        s["q"] = x[:, :, :H].transpose(1, 2)
        s["k"] = x[:, :, H:H + Hkv].transpose(1, 2)
        s["qw"] = (1 + 0.2 * torch.randn(D, generator=g, device="cuda")).to(torch.bfloat16)
        s["kw"] = (1 + 0.2 * torch.randn(D, generator=g, device="cuda")).to(torch.bfloat16)
        start = torch.randint(0, case["far"] + 1, (B, 1), generator=g, device="cuda")
        s["pos"] = (start + torch.arange(N, device="cuda")).to(torch.int32).contiguous()
        freq = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
        s["freq"] = freq.cuda()
        # each frequency in turns a position, as a 64-bit fraction of one turn (the package's plan)
        turns = [int(f / (2 * math.pi) * 2.0 ** 64) & ((1 << 64) - 1) for f in freq.tolist()]
        turns = [t - (1 << 64) if t >= 1 << 63 else t for t in turns]
        s["turns"] = torch.tensor(turns, dtype=torch.int64, device="cuda")
        if case["backward"]:
            s["dq"] = torch.randn((B, H, N, D), generator=g, device="cuda").to(torch.bfloat16)
            s["dk"] = torch.randn((B, Hkv, N, D), generator=g, device="cuda").to(torch.bfloat16)
        return s
    new = case.get("N", 0)
    held, rows = _lengths(case, new)
    s.update(_cache(case, held, g, held))
    s["held"] = torch.tensor(held, dtype=torch.int32, device="cuda")
    s["rows"] = torch.tensor(rows, dtype=torch.int32, device="cuda")
    B, Hkv, D = case["B"], case["Hkv"], case["D"]
    if op == "kv_write":
        s["start"] = s["held"] - s["rows"]
        # token-major, as the projection gives values; keys come head-major from the rotation
        s["new_k"] = _keys((B, Hkv, new, D), g, 6.0)
        s["new_v"] = _keys((B, new, Hkv, D), g, 2.0).transpose(1, 2)
    elif op == "kv_read":
        s["out_k"] = torch.zeros((B, Hkv, max(held), D), dtype=torch.bfloat16, device="cuda")
        s["out_v"] = torch.zeros_like(s["out_k"])
    else:
        s["q"] = (torch.randn((B, case["H"], new, D), generator=g, device="cuda") * 1.5).to(
            torch.bfloat16)
    return s


# ------------------------------------------------------------------ the plain forms


def _exponent(m):
    """The least e in [-117, 119] with 448 * 2^e >= m (m >= 0, finite)."""
    f, x = torch.frexp(m)  # m = f * 2^x, 0.5 <= f < 1; 448 = 0.875 * 2^9
    e = x - 9 + (f > 0.875).to(x.dtype)
    e = torch.where(m == 0, torch.full_like(e, EXP_MIN), e)
    return e.clamp(EXP_MIN, EXP_MAX).to(torch.int8)


def _grid(e):
    """2^e in fp32, from the exponent bits."""
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def _to_grid(y, e):
    """y [pages, heads, rows, D] (fp32) rounded onto its pages' grids: (payload, exponents)."""
    s = _grid(-e)[..., None, None]
    y = torch.where(y.isinf(), torch.full_like(y, math.nan), y)
    return (y * s).clamp(-448, 448).to(E4M3), e


def _norm_rope(x, w, cos, sin, case):
    x = x.float()
    n = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6)
    return _turn(n * w.float(), cos, sin, case)


def _turn(y, cos, sin, case):
    rot = case["rot"]
    r, rest = y[..., :rot], y[..., rot:]
    if case["interleaved"]:
        a, b = r[..., 0::2], r[..., 1::2]
        r = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    else:
        a, b = r[..., :rot // 2], r[..., rot // 2:]
        r = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    return torch.cat((r, rest), -1)


def _norm_rope_grad(x, w, g, cos, sin, case):
    x, w = x.float(), w.float()
    g = _turn(g.float(), cos, -sin, case)  # the rotation's transpose
    r = torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6)
    n = x * r
    gn = g * w
    dx = r * (gn - n * (gn * n).mean(-1, keepdim=True))
    return dx.to(torch.bfloat16), (g * n).sum((0, 1, 2))


def _run_norm_rope(s, case):
    angle = s["pos"].double()[:, None, :, None] * s["freq"]
    cos, sin = angle.cos().float(), angle.sin().float()
    out = dict(q=_norm_rope(s["q"], s["qw"], cos, sin, case).to(torch.bfloat16),
               k=_norm_rope(s["k"], s["kw"], cos, sin, case).to(torch.bfloat16))
    if case["backward"]:
        out["dq"], out["dqw"] = _norm_rope_grad(s["q"], s["qw"], s["dq"], cos, sin, case)
        out["dk"], out["dkw"] = _norm_rope_grad(s["k"], s["kw"], s["dk"], cos, sin, case)
    return out


def _write_one(payload, exps, new, s, case):
    page, N = case["page"], case["N"]
    start, rows, table = s["start"].long(), s["rows"].long(), s["table"].long()
    # the pages a write can touch, at their places in the sequences
    span = (N + page - 2) // page + 1
    at = start[:, None] // page + torch.arange(span, device=start.device)  # [B, span]
    live = at * page < (start + rows)[:, None]
    b, j = live.nonzero(as_tuple=True)
    ids = table[b, at[b, j]]
    pos = at[b, j][:, None] * page + torch.arange(page, device=start.device)  # [pages, page]
    i = pos - start[b][:, None]
    fresh = (i >= 0) & (i < rows[b][:, None])
    old = i < 0
    y = new[b[:, None], :, i.clamp(0, N - 1)].permute(0, 2, 1, 3).float()  # [pages, heads, page, D]
    size = torch.where(y.isfinite(), y.abs(), torch.zeros_like(y))
    size = torch.where(fresh[:, None, :, None], size, torch.zeros_like(size)).amax((2, 3))
    e = _exponent(size)
    kept = exps[ids]
    e = torch.where(old.any(1)[:, None], torch.maximum(e, kept), e)
    held = payload.view(torch.uint8)[ids].view(E4M3)
    again, _ = _to_grid(held.float() * _grid(kept)[..., None, None], e)
    again = torch.where((e == kept)[..., None, None], held.view(torch.uint8), again.view(torch.uint8))
    put, _ = _to_grid(y, e)
    mix = torch.where(fresh[:, None, :, None], put.view(torch.uint8),
                      torch.where(old[:, None, :, None], again, held.view(torch.uint8)))
    payload.view(torch.uint8)[ids] = mix
    exps[ids] = e


def _gather(payload, exps, s, longest):
    """[B, heads, longest (whole pages), D] fp32 of every sequence's pages."""
    table = s["table"].long()
    page = payload.shape[2]
    table = table[:, :-(-longest // page)]
    y = payload.view(torch.uint8)[table].view(E4M3).float() * _grid(exps[table])[..., None, None]  # [B, pages, heads, page, D]
    return y.permute(0, 2, 1, 3, 4).flatten(2, 3)


def _run_attend(s, case):
    B, N, H, Hkv, D = (case[x] for x in ("B", "N", "H", "Hkv", "D"))
    k = _gather(s["k"], s["k_exp"], s, case["longest"])
    L = k.shape[2]
    q = s["q"].float().reshape(B, Hkv, H // Hkv * N, D)
    p = (q @ k.transpose(2, 3)) / math.sqrt(D)
    del k
    p = p.view(B, Hkv, H // Hkv, N, L)
    last = s["held"].long()[:, None] - s["rows"].long()[:, None] + torch.arange(N, device="cuda")
    seen = torch.arange(L, device="cuda") <= last[..., None]  # [B, N, L]
    p.masked_fill_(~seen[:, None, None], -math.inf)
    m = p.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    p = p.sub_(m).exp_()
    z = p.sum(-1, keepdim=True)
    v = _gather(s["v"], s["v_exp"], s, case["longest"])
    v = torch.where((torch.arange(L, device="cuda") < s["held"][:, None])[:, None, :, None], v,
                    torch.zeros_like(v))
    o = (p.view(B, Hkv, -1, L) @ v).view(B, H, N, D) / z.view(B, H, N, 1)
    lse = (m + z.log()).view(B, H, N)
    return dict(o=o.to(torch.bfloat16), lse=lse)


def run(s):
    case = s["case"]
    op = case["op"]
    if own:
        return _own(s, case, op)
    if op == "norm_rope":
        return _run_norm_rope(s, case)
    if op == "kv_write":
        _write_one(s["k"], s["k_exp"], s["new_k"], s, case)
        _write_one(s["v"], s["v_exp"], s["new_v"], s, case)
        return dict(k=s["k"], v=s["v"], k_exp=s["k_exp"], v_exp=s["v_exp"])
    if op == "kv_read":
        n = s["out_k"].shape[2]
        keep = (torch.arange(n, device="cuda") < s["held"][:, None])[:, None, :, None]
        for name in ("k", "v"):
            y = _gather(s[name], s[name + "_exp"], s, n)[:, :, :n].to(torch.bfloat16)
            s["out_" + name].copy_(torch.where(keep, y, s["out_" + name]))
        return dict(k=s["out_k"], v=s["out_v"])
    return _run_attend(s, case)


# ------------------------------------------------------------------ a user's calls


def _own(s, case, op):
    import attention_forward_tk_gb300 as tk
    if op == "norm_rope":
        q, k = tk.qk_norm_rope_forward(s["q"], s["k"], s["qw"], s["kw"], s["turns"],
                                       positions=s["pos"], interleaved=case["interleaved"])
        out = dict(q=q, k=k)
        if case["backward"]:
            out["dq"], out["dk"], out["dqw"], out["dkw"] = tk.qk_norm_rope_backward(
                s["q"], s["k"], s["qw"], s["kw"], s["turns"], s["dq"], s["dk"],
                positions=s["pos"], interleaved=case["interleaved"])
        return out
    cache = tk.Kv8Cache(s["k"], s["v"], s["k_exp"], s["v_exp"])
    if op == "kv_write":
        tk.kv8_write(cache, s["new_k"], s["new_v"], s["table"], s["start"], counts=s["rows"])
        return dict(k=s["k"], v=s["v"], k_exp=s["k_exp"], v_exp=s["v_exp"])
    if op == "kv_read":
        tk.kv8_read(cache, s["table"], s["held"], out_k=s["out_k"], out_v=s["out_v"])
        return dict(k=s["out_k"], v=s["out_v"])
    o, lse = tk.attention_forward_kv8(s["q"], cache, s["table"], s["held"], causal=True)
    return dict(o=o, lse=lse)


# ------------------------------------------------------------------ work and exact values


def work(case):
    op = case["op"]
    if op == "norm_rope":
        n = case["B"] * case["N"] * (case["H"] + case["Hkv"]) * case["D"]
        # x in, y out; and with gradients dy in, dx out (x once)
        return dict(bytes=n * (8 if case["backward"] else 4),
                    flops=n * (24 if case["backward"] else 8))
    Hkv, D = case["Hkv"], case["D"]
    held, rows = _lengths(case, case.get("N", 0))
    if op == "kv_write":
        n = 2 * sum(rows) * Hkv * D
        return dict(bytes=3 * n, flops=3 * n)
    if op == "kv_read":
        n = 2 * sum(held) * Hkv * D
        return dict(bytes=3 * n, flops=n)
    B, N, H = case["B"], case["N"], case["H"]
    pairs = sum(N * n - N * (N - 1) // 2 for n in held) * H
    return dict(bytes=2 * sum(held) * Hkv * D + 4 * B * N * H * D + 4 * B * N * H,
                flops=4 * pairs * D)


def _two(e):
    """2^e in float64 for whole e, from the exponent bits."""
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)


def exact(case, seed):
    op = case["op"]
    w = work(case)
    if w["flops"] > 1e12:
        return None
    s = prepare(case, seed)
    if op == "norm_rope":
        return _exact_norm_rope(s, case)
    if op == "kv_write":
        return _exact_write(s, case)
    held = s["held"].tolist()
    page = case["page"]
    rows = []
    for b, n in enumerate(held):
        ids = s["table"][b, :-(-n // page)].long()
        rows.append([(s[x].view(torch.uint8)[ids].view(E4M3).double() *
                      _two(s[x + "_exp"][ids])[..., None, None])
                     .transpose(0, 1).reshape(case["Hkv"], -1, case["D"])[:, :n] for x in "kv"])
    if op == "kv_read":
        out = dict(k=s["out_k"].double(), v=s["out_v"].double())
        for b, n in enumerate(held):
            out["k"][b, :, :n], out["v"][b, :, :n] = rows[b]
        return out
    N, G = case["N"], case["H"] // case["Hkv"]
    o = torch.empty(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.empty(s["q"].shape[:3], dtype=torch.float64, device="cuda")
    for b, n in enumerate(held):
        for h in range(case["H"]):
            k, v = rows[b][0][h // G], rows[b][1][h // G]
            t = s["q"][b, h].double() @ k.T * case["D"] ** -0.5
            i = torch.arange(n - N, n, device="cuda")
            t[torch.arange(n, device="cuda")[None] > i[:, None]] = -math.inf
            lse[b, h] = torch.logsumexp(t, -1)
            o[b, h] = (t - lse[b, h][:, None]).exp() @ v
    return dict(o=o, lse=lse)


def _exact_norm_rope(s, case):
    rot, D = case["rot"], case["D"]
    half = rot // 2
    i = torch.arange(half, device="cuda")
    first, second = (2 * i, 2 * i + 1) if case["interleaved"] else (i, half + i)
    turn = torch.exp(1j * s["pos"].double()[:, None, :, None] * s["freq"])
    out = {}
    for name in "qk":
        x = s[name].double().detach().requires_grad_()
        w = s[name + "w"].double().requires_grad_()
        y = x / (x.pow(2).sum(-1, keepdim=True) / D + 1e-6).sqrt() * w
        z = torch.complex(y[..., first], y[..., second]) * turn
        r = y.clone()
        r[..., first] = z.real
        r[..., second] = z.imag
        out[name] = r.detach()
        if case["backward"]:
            out["d" + name], out["d" + name + "w"] = torch.autograd.grad(
                r, (x, w), s["d" + name].double())
    return out


def _exact_write(s, case):
    page = case["page"]
    start, rows = s["start"].tolist(), s["rows"].tolist()
    out = {x: s[x].double() for x in "kv"}
    exps = {x: s[x + "_exp"].clone() for x in "kv"}
    if sum(-(-r // page) + 1 for r in rows) > 4000:
        return None
    # E4M3's values and the borders between neighbours; a value on a border goes to the even code
    codes = torch.arange(127, dtype=torch.uint8, device="cuda").view(E4M3).double()
    border = (codes[1:] + codes[:-1]) / 2

    def near(y):
        a = y.abs()
        lo, hi = torch.bucketize(a, border), torch.bucketize(a, border, right=True)
        at = torch.where(lo == hi, lo, torch.where(lo % 2 == 0, lo, hi))
        return codes[at] * y.sign()

    for b in range(case["B"]):
        for j in range(start[b] // page, -(-(start[b] + rows[b]) // page)):
            at = int(s["table"][b, j])
            lo, hi = max(start[b], j * page), min(start[b] + rows[b], (j + 1) * page)
            for x in "kv":
                new = s["new_" + x][b, :, lo - start[b]:hi - start[b]].double()
                m = new.abs().amax((1, 2)).clamp_min(2.0 ** -200)
                e = torch.ceil(torch.log2(m / 448)).clamp(EXP_MIN, EXP_MAX)
                # log2 next to a power of two may round across it
                e = torch.where(448 * _two(e - 1) >= m, e - 1, e)
                e = torch.where(448 * _two(e) < m, e + 1, e).clamp(EXP_MIN, EXP_MAX)
                was = exps[x][at].double()
                if lo > j * page:
                    e = torch.maximum(e, was)
                    shift = _two(was - e)[:, None, None]
                    out[x][at, :, :lo - j * page] = near(out[x][at, :, :lo - j * page] * shift)
                out[x][at, :, lo - j * page:hi - j * page] = near(new * _two(-e)[:, None, None])
                exps[x][at] = e.to(torch.int8)
    return dict(k=out["k"], v=out["v"], k_exp=exps["k"], v_exp=exps["v"])
