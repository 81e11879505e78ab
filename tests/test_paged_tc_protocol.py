"""CPU checks of the barrier protocol of paged_tc_kernel over 8-bit pages (csrc/paged_tc.cu), whose
converting warps stand between the loads and the products: the roles are written out from the source and run
under many random schedules (see barrier_model), also with a wait that gives up in a converting warp.
"""
import os
import random
import re
from collections import defaultdict

import pytest

import barrier_model as bm

SOURCE = os.path.join(os.path.dirname(os.path.abspath(__file__)), "..", "exact_tiled_softmax_gb300", "csrc", "paged_tc.cu")
CONVERTERS, KEEP_BLOCKS = 2, 4  # warps that convert (the kernel: 4), blocks whose masks are kept


def kernel(segments, NS=3, NR=3, keep_blocks=KEEP_BLOCKS, gives_up=None, stops=True):
    """segments: (blocks, whether half B has rows) of each.  gives_up: number of the wait of converting warp 0
    that runs out; stops: whether the warp ends there.  (need, roles, log); the log holds the masks that the
    softmax found not to be its block's, and what warp 0 did behind the wait that gave up."""
    need = defaultdict(lambda: 1)
    for e in (0, 1):
        need[f"SEGE{e}"] = 5 + CONVERTERS  # loads, products, a warp of Q, both halves' softmax
    need["Q"] = 2
    for s in range(NS):
        need[f"KVF{s}"] = CONVERTERS
    for s in range(NR):
        need[f"RE{s}"] = CONVERTERS
    ring, keep, log = [None, None], {}, {"masks": [], "behind": [], "timeout": False}
    N = len(segments)

    def take(seg):
        e = seg & 1
        yield ("wait", f"SEGF{e}", seg >> 1)
        t = ring[e]
        yield ("arrive", f"SEGE{e}")
        return t

    def walker():  # gives the segments out, and copies its half of the rows of Q
        for seg in range(N + 1):
            e = seg & 1
            if seg >= 2:
                yield ("wait", f"SEGE{e}", (seg >> 1) - 1)
            ring[e] = segments[seg] if seg < N else (0, False)
            yield ("arrive", f"SEGF{e}")
            if seg == N:
                return
            if seg > 0:
                yield ("wait", "QFREE", seg - 1)
            yield ("arrive", "Q")

    def rows_of_q():
        for seg in range(N + 1):
            n, _ = yield from take(seg)
            if n == 0:
                return
            if seg > 0:
                yield ("wait", "QFREE", seg - 1)
            yield ("arrive", "Q")

    def loads():
        fill = 0
        for seg in range(N + 1):
            n, _ = yield from take(seg)
            if n == 0:
                break
            for _ in range(2 * n):
                if fill >= NR:
                    yield ("wait", f"RE{fill % NR}", fill // NR - 1)
                yield ("tma", f"RF{fill % NR}")
                fill += 1
        for u in range(min(NR, fill)):
            i = fill - 1 - u
            yield ("wait", f"RF{i % NR}", i // NR)

    def converter(w):
        def run():
            fill, waits, seg = 0, 0, 0

            def out():
                nonlocal waits
                waits += 1
                return w == 0 and gives_up is not None and waits - 1 == gives_up

            ok = True
            while True:
                if out():
                    ok = False
                    break
                ok = True
                n, _ = yield from take(seg)
                if n == 0:
                    break
                for u in range(2 * n):
                    if out():
                        ok = False
                        break
                    yield ("wait", f"RF{fill % NR}", fill // NR)
                    if out():
                        ok = False
                        break
                    if fill >= NS:
                        yield ("wait", f"KVE{fill % NS}", fill // NS - 1)
                    if u % 2 == 0:
                        keep[fill // 2 % keep_blocks] = fill // 2
                    yield ("arrive", f"RE{fill % NR}")
                    yield ("arrive", f"KVF{fill % NS}")
                    fill += 1
                if not ok and stops:
                    break
                if not ok:
                    log["behind"].append(seg)
                seg += 1
            if not ok:
                log["timeout"] = True

        return run()

    def products():
        fill, p = 0, [0, 0]
        for seg in range(N + 1):
            n, two = yield from take(seg)
            if n == 0:
                break
            yield ("wait", "Q", seg)
            prev = -1
            for u in range(n):
                ks, kph, vs, vph = fill % NS, fill // NS, (fill + 1) % NS, (fill + 1) // NS
                fill += 2
                yield ("wait", f"KVF{ks}", kph)
                yield ("mma", "S_A")
                yield ("commit", "S0")
                if u > 0:
                    if two:
                        yield ("wait", "P1", p[1])
                        p[1] += 1
                        yield ("mma", "PV_B")
                    yield ("commit", f"KVE{prev}")
                if two:
                    yield ("mma", "S_B")
                yield ("commit", "S1") if two else ("mma", "none")
                if u == n - 1:
                    yield ("commit", "QFREE")
                yield ("commit", f"KVE{ks}")
                yield ("wait", f"KVF{vs}", vph)
                yield ("wait", "P0", p[0])
                p[0] += 1
                yield ("mma", "PV_A")
                prev = vs
            if two:
                yield ("wait", "P1", p[1])
                p[1] += 1
                yield ("mma", "PV_B")
            yield ("commit", f"KVE{prev}")
            for X in (0, 1):
                if seg > 0:
                    yield ("wait", f"OREAD{X}", seg - 1)
                yield ("commit", f"O{X}")
        yield ("commit", "DRAIN")
        yield ("wait", "DRAIN", 0)

    def softmax(X):
        block, cnt = 0, 0
        for seg in range(N + 1):
            n, two = yield from take(seg)
            if n == 0:
                return
            for u in range(n if X == 0 or two else 0):
                yield ("wait", f"S{X}", cnt)
                yield ("arrive", f"late{X}.{cnt}")  # any other role may run before the masks are read
                if keep.get((block + u) % keep_blocks) != block + u:
                    log["masks"].append((X, block + u))
                cnt += 1
                yield ("arrive", f"P{X}")
            block += n
            yield ("wait", f"O{X}", seg)
            yield ("arrive", f"OREAD{X}")

    roles = {"walker": walker(), "rows": rows_of_q(), "loads": loads(), "products": products(), "A": softmax(0), "B": softmax(1)}
    for w in range(CONVERTERS):
        roles[f"converter{w}"] = converter(w)
    return need, roles, log


def _run(segments, seed, skip_waits=(), **kw):
    need, roles, log = kernel(segments, **kw)
    try:
        bm.Sim(need, seed, skip_waits).run(roles)
    except bm.ProtocolError as e:
        return str(e), log
    return None, log


def _segments(rnd):
    return [(rnd.choice((1, 1, 2, 3, 5)), rnd.random() < 0.6) for _ in range(rnd.randint(0, 6))]


@pytest.mark.parametrize("ring", [3, 6])  # slots of either ring: 128 columns, 64
def test_protocol_holds(ring):
    rnd = random.Random(ring)
    for seed in range(400):
        failure, log = _run(_segments(rnd), seed, NS=ring, NR=ring)
        assert failure is None and not log["masks"] and not log["timeout"]


@pytest.mark.parametrize("ring", [3, 6])
def test_masks_of_fewer_blocks_would_be_written_over(ring):
    rnd = random.Random(ring)
    blocks = 1 if ring == 3 else 3
    assert any(_run([(9, True), (4, False)], seed, NS=ring, NR=ring, keep_blocks=blocks)[1]["masks"] for seed in range(400))


@pytest.mark.parametrize("drop,segments", [("KVE0", [(3, True)] * 4), ("RE0", [(3, True)] * 4), ("QFREE", [(3, True)] * 4),
                                           ("SEGE0", [(1, False)] * 6)])
def test_model_catches_a_missing_wait(drop, segments):
    assert any(_run(segments, seed, {drop})[0] for seed in range(400))


def test_a_wait_that_gives_up_ends_its_warp():
    """Nothing is touched behind it, and the time-out is reported."""
    for at in range(12):
        _, log = _run([(2, True), (1, True), (2, False)], at, gives_up=at)
        assert log["timeout"] and log["behind"] == []


def test_a_warp_that_went_on_would_lose_the_time_out():
    """With its wait given up and the next segment taken all the same, the warp's fills are those of another
    block, and its last wait says that all is well."""
    lost = 0
    for at in range(1, 12):
        _, log = _run([(2, True), (1, True), (2, False)], at, gives_up=at, stops=False)
        lost += bool(log["behind"]) and not log["timeout"]
    assert lost


def _loops(text):
    """The bodies of the loops over segments."""
    for m in re.finditer(r"for \(int seg = 0;[^{;]*take\(seg, t, ok\)[^{;]*; \+\+seg\) \{", text):
        depth, i = 1, m.end()
        while depth:
            depth += {"{": 1, "}": -1}.get(text[i], 0)
            i += 1
        yield text[m.end():i - 1]


def test_every_role_of_the_source_ends_where_a_wait_gave_up():
    """A loop over segments whose inner loop breaks on a wait is left behind that loop."""
    with open(SOURCE) as f:
        loops = list(_loops(f.read()))
    assert len(loops) == 5  # converters, loads, products, rows of Q, softmax
    inner = 0
    for body in loops:
        m = list(re.finditer(r"\n( *)for \([^\n]*\) \{\n", body))
        for head in m:
            end = body.index("\n" + head.group(1) + "}", head.end())
            waits = re.search(r"if \(!\(ok = wait_all[^\n]*break;", body[head.end():end])
            if waits is None:
                continue
            nested = any(o.start() < head.start() and body.index("\n" + o.group(1) + "}", o.end()) > end for o in m if o is not head)
            if nested:  # left with its outer loop, whose condition asks for ok
                continue
            inner += 1
            assert re.search(r"if \(!ok\) break;", body[end:]), body[head.start():head.start() + 80]
    assert inner >= 4
