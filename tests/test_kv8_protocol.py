"""Barrier protocol of the tensor-core kernel over the 8-bit paged cache, checked
on the CPU with the simulator of the other kernels' protocols: every role ends, no
barrier is ever two phases ahead of a waiter, and what one role hands another
through shared memory is read before it is written again.

A run is a list of segments (n0, n1): the key-tile steps that each of the two
tiles of queries takes part in.  With `pair` both tiles hold the same rows and a step
is two key tiles, one for each.
"""
import pytest
from test_pipeline_protocols import Sim


def chunk_roles(sim, segs, pair=False, KS=3, VS=2, drop=()):
    """tk_kv8_chunk_kernel.  Converter warps are two roles (of four), so that
    one may run ahead of the other; a tile's four softmax warps are one."""
    conv = ("a", "b")
    for t in range(2):
        for b in ("q_full", "s_full", "p_full", "o_full", "v_free", "fin_full0", "fin_full1"):
            sim.bar(f"{b}{t}")
        sim.bar(f"o_free{t}", len(conv)), sim.bar(f"v_ready{t}", len(conv))
    for s in range(4):
        sim.bar(f"seg_full{s}"), sim.bar(f"seg_empty{s}", 5 + len(conv))
        sim.bar(f"k_full{s}"), sim.bar(f"k_empty{s}")
        sim.bar(f"v_full{s}"), sim.bar(f"v_empty{s}", len(conv))
    sim.bar("conv_bar", len(conv))
    readers = ["softmax0", "softmax1", "mma", "load_k", "load_v", *conv]

    def tiles(n0, n1):  # of keys
        return 2 * max(n0, n1) if pair else max(n0, n1)

    def joins(t, n0, n1, j):  # tile t reads key tile j of the segment
        return j % 2 == t if pair else j < (n0, n1)[t]

    def poster():
        for x in range(len(segs) + 1):  # the last says that the run is over
            if x >= 4:
                yield ("wait", f"seg_empty{x % 4}", x // 4 - 1)
            for r in readers:
                yield ("write", f"seg{x % 4}:{r}", x)
            yield ("arrive", f"seg_full{x % 4}")

    def segment(me, x):
        yield ("wait", f"seg_full{x % 4}", x // 4)
        yield ("read", f"seg{x % 4}:{me}", x)
        yield ("arrive", f"seg_empty{x % 4}")

    def loader(me, v):
        ring, name = (VS, "v") if v else (KS, "k")
        idx = 0
        for x, (n0, n1) in enumerate(segs):
            yield from segment(me, x)
            for j in range(tiles(n0, n1)):
                if idx >= ring and "empty" not in drop:
                    yield ("wait", f"{name}_empty{idx % ring}", idx // ring - 1)
                if v:
                    for c in conv:
                        yield ("write", f"v_exp8:{idx % 8}:{c}", idx)
                else:
                    for t in range(2):
                        if joins(t, n0, n1, j):
                            yield ("write", f"k_scale:{idx % 8}:{t}", idx)
                yield ("commit", f"{name}_full{idx % ring}", "tma_" + name)
                idx += 1
        yield from segment(me, len(segs))

    def softmax(t):
        step0 = phase = part = 0
        for x, (n0, n1) in enumerate(segs):
            yield from segment(f"softmax{t}", x)
            n_t = (n0, n1)[t]
            if n_t:
                yield ("arrive", f"q_full{t}")
                for j in range(n_t):
                    yield ("wait", f"s_full{t}", phase)
                    phase += 1
                    idx = 2 * (step0 + j) + t if pair else step0 + j
                    yield ("read", f"k_scale:{idx % 8}:{t}", idx)
                    if "v_ready" not in drop:
                        yield ("wait", f"v_ready{idx % 2}", idx // 2)
                    yield ("read", f"v_exp:{idx % 2}:{t}", idx)
                    if j == n_t - 1:
                        for c in conv:
                            yield ("write", f"fin:{part % 2}:{t}:{c}", part)
                    yield ("arrive", f"p_full{t}")
                    if j == n_t - 1:
                        yield ("arrive", f"fin_full{part % 2}{t}", part // 2)
                part += 1
            step0 += max(n0, n1)
        yield from segment(f"softmax{t}", len(segs))

    def converter(me):
        idx, part, pend = 0, [0, 0], None
        first = me == conv[0]
        for x in range(len(segs) + 1):
            yield from segment(me, x)
            have = x < len(segs)
            n0, n1 = segs[x] if have else (0, 0)
            n = tiles(n0, n1)
            for j in range(n + 1):
                if pend is not None and (j == 1 or not have):
                    if "conv_bar" not in drop:
                        yield ("wait", "conv_bar", x - 1)
                    for c in conv:  # NaN positions that the other warps noted
                        yield ("read", f"nan:{(x - 1) % 8}:{c}>{me}", x - 1)
                    for t in range(2):
                        if pend[t] == 0:
                            continue
                        pc = part[t]
                        part[t] += 1
                        yield ("wait", f"fin_full{pc % 2}{t}", pc // 2)
                        yield ("wait", f"o_full{t}", pc)
                        yield ("read", f"fin:{pc % 2}:{t}:{me}", pc)
                        yield ("read", f"o:{t}:{me}", pc)
                        yield ("arrive", f"o_free{t}", pc)
                    pend = None
                if j == n:
                    break
                yield ("wait", f"v_full{idx % VS}", idx // VS)
                if idx >= 2 and "v_free" not in drop:
                    yield ("wait", f"v_free{idx % 2}", idx // 2 - 1)
                yield ("read", f"v_exp8:{idx % 8}:{me}", idx)
                for t in range(2):
                    if joins(t, n0, n1, j):
                        yield ("write", f"v16:{idx % 2}:{me}:{t}", idx)
                        if first:
                            yield ("write", f"v_exp:{idx % 2}:{t}", idx)
                yield ("arrive", f"v_ready{idx % 2}", idx // 2)
                yield ("arrive", f"v_empty{idx % VS}", idx // VS)
                idx += 1
            if have:
                for c in conv:
                    yield ("write", f"nan:{x % 8}:{me}>{c}", x)
                yield ("arrive", "conv_bar", x)
                pend = (n0, n1)

    def mma():
        phase, parts, k = [0, 0], [0, 0], 0
        step0 = 0
        for x, (n0, n1) in enumerate(segs):
            yield from segment("mma", x)
            n = max(n0, n1)
            for j in range(n + 1):
                k_ready = False
                for t in range(2):
                    n_t = (n0, n1)[t]
                    pv, s = 1 <= j <= n_t, j < n_t
                    if pv:
                        if j == 1 and parts[t] and "o_free" not in drop:
                            yield ("wait", f"o_free{t}", parts[t] - 1)
                        yield ("wait", f"p_full{t}", phase[t])
                        phase[t] += 1
                    if s:
                        if j == 0:
                            yield ("wait", f"q_full{t}", parts[t])
                        if not k_ready:
                            yield ("wait", f"k_full{k % KS}", k // KS)
                            k_ready = True
                    if pv:
                        idx = 2 * (step0 + j - 1) + t if pair else step0 + j - 1
                        yield ("check", f"v_ready{idx % 2}", idx // 2)
                        for c in conv:
                            yield ("read", f"v16:{idx % 2}:{c}:{t}", idx)
                    if s:
                        yield ("check", f"k_full{k % KS}", k // KS)
                        yield ("commit", f"s_full{t}")
                    if pair:
                        if pv:
                            yield ("commit", f"v_free{t}")
                        if s:
                            yield ("commit", f"k_empty{k % KS}")
                            k_ready = False
                            k += 1
                    if pv and j == 1:  # (the tile's first product overwrites O)
                        for c in conv:
                            yield ("write", f"o:{t}:{c}", parts[t])
                    if pv and j == n_t:
                        yield ("commit", f"o_full{t}")
                        parts[t] += 1
                if not pair:
                    if j < n:
                        yield ("commit", f"k_empty{k % KS}")
                        k += 1
                    if j >= 1:
                        yield ("commit", f"v_free{(step0 + j - 1) % 2}")
            step0 += n
        yield from segment("mma", len(segs))

    roles = {"poster": poster(), "load_k": loader("load_k", False),
             "load_v": loader("load_v", True), "softmax0": softmax(0), "softmax1": softmax(1),
             "mma": mma(), **{c: converter(c) for c in conv}}
    return {name: by_parity(role) for name, role in roles.items()}


def by_parity(role):
    """A wait sees a phase's parity: the phase before it has to be over already, or
    the one before that would pass for it."""
    for op in role:
        if op[0] == "wait" and op[2] > 0:
            yield ("check", op[1], op[2] - 1)
        yield op


RUNS = [
    [],
    [(1, 1)],
    [(1, 2)] * 6,
    [(1, 1)] * 12,
    [(4, 5), (1, 2), (0, 3), (5, 5), (2, 0)],   # a run's ends, and a unit without a second tile
    [(0, 1)] * 5 + [(1, 1)] * 5 + [(3, 0)] * 3,
    [(1, 0), (0, 2), (9, 9), (0, 1), (0, 1), (0, 1), (2, 3)],
    [(17, 18)],
]


@pytest.mark.parametrize("segs", RUNS, ids=lambda s: "-".join(f"{a}.{b}" for a, b in s) or "none")
@pytest.mark.parametrize("KS,VS", [(3, 2), (4, 4)], ids=["d128", "d64"])
def test_chunk_protocol(segs, KS, VS):
    for seed in range(60):
        sim = Sim(seed)
        sim.run(chunk_roles(sim, segs, False, KS, VS))


@pytest.mark.parametrize("steps", [[1], [1] * 9, [2, 1, 5], [7, 1, 1, 3], [12]],
                         ids=lambda s: "-".join(map(str, s)))
def test_chunk_protocol_with_both_tiles_on_the_same_rows(steps):
    for seed in range(60):
        sim = Sim(seed)
        sim.run(chunk_roles(sim, [(n, n) for n in steps], True, 4, 4))


@pytest.mark.parametrize("drop", ["o_free", "v_free", "v_ready", "empty", "conv_bar"])
@pytest.mark.parametrize("pair", [False, True], ids=["two", "same"])
def test_chunk_model_sees_a_missing_wait(drop, pair):
    segs = [(3, 3), (1, 1), (2, 2), (1, 1), (1, 1), (4, 4), (1, 1)] if pair else \
        [(3, 4), (1, 2), (2, 3), (1, 1), (1, 2), (4, 4), (1, 1)]
    failures = 0
    for seed in range(300):
        sim = Sim(seed)
        try:
            sim.run(chunk_roles(sim, segs, pair, drop=(drop,)))
        except AssertionError as e:
            assert "deadlock" not in str(e), str(e)
            failures += 1
    assert failures > 0
