"""Host models of the attention kernels over a 4-bit cache (no GPU): the shares
with their weights, and the tile kernel's roles where they differ from those
over a 16-bit one.

There, four warps widen keys and values into the ring that TMA fills otherwise
(a slot is full when all four have arrived), the producer brings queries alone,
and the softmax warps, which prepare the queries' rows, say that they are there
for the products; the relay waits for that and not for the copy.  Keys of an
fp16 cache are two tiles.
"""
import pytest

from test_fwd_protocol_model import SLOTS, MBar
from test_paged_protocol_model import (BATCHES, CTAS, WALKS, Tile, run_roles, softmax,
                                       test_partition as check_partition)

TILE4 = dict(unit=128, key1=3, key2=4, overhead=1536, single=False, min_share=1024)
# six warps a CTA (8 rows) and four (16 rows), blocks of 32 keys
DECODE4 = [dict(unit=32 * w, key1=1, key2=1, overhead=512, single=True, min_share=192) for w in (6, 4)]


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("batch,heads,W", BATCHES)
@pytest.mark.parametrize("cost,ctas", [(TILE4, CTAS), (DECODE4[0], 2 * CTAS), (DECODE4[1], 2 * CTAS), (TILE4, 7)])
def test_partition_by_the_weights_of_a_4_bit_cache(batch, heads, W, causal, cost, ctas):
    check_partition(batch, heads, W, causal, cost, ctas)


class Tile4(Tile):
    def __init__(self, walk, fail_p, seed, keys, early=False):
        super().__init__(walk, fail_p, seed, early)
        self.keys = keys  # tiles of keys of a block
        self.kvfull = [MBar(4) for _ in range(SLOTS)]
        self.qready = [MBar(), MBar()]


def producer4(c):
    q_it = [0, 0]
    for *nb, _, _ in c.walk:
        for t in range(2):
            if nb[t] == 0:
                continue
            if not c.wait(c.qempty[t], (q_it[t] & 1) ^ 1):
                return
            c.qfull[t].arrive()
            q_it[t] += 1


def widen(c):
    it = 0
    for *nb, _, _ in c.walk:
        for _ in range((c.keys + 1) * max(nb)):
            if not c.wait(c.kvempty[it % SLOTS], ((it // SLOTS) & 1) ^ 1):
                return
            c.kvfull[it % SLOTS].arrive()
            it += 1


def relay4(c):
    it, q_it, aborted = 0, [0, 0], False

    def ready(n):
        nonlocal it, aborted
        for _ in range(n):
            if not aborted:
                aborted = not c.wait(c.kvfull[it % SLOTS], (it // SLOTS) & 1)
            it += 1

    for *nb, _, _ in c.walk:
        if max(nb) == 0:
            continue
        for t in range(2):
            if nb[t] == 0:
                continue
            if not aborted:
                aborted = not c.wait(c.qready[t], q_it[t] & 1)
            q_it[t] += 1
        ready(c.keys)
        aborted = c.kv.go(aborted)
        for j in range(max(nb)):
            ready(1 + (c.keys if j + 1 < max(nb) else 0))
            aborted = c.kv.go(aborted)


def issuer4(c):
    it, aborted = 0, False

    def take(n):
        nonlocal it
        it += n
        return [i % SLOTS for i in range(it - n, it)]

    def free(slots):
        for s in slots:
            c.kvempty[s].arrive()

    for *nb, _, _ in c.walk:
        if max(nb) == 0:
            continue
        aborted = c.kv.go(aborted)
        k = take(c.keys)
        if not aborted:
            for t in range(2):
                if nb[t] > 0:
                    c.sfull[t].arrive()
                    if nb[t] == 1:
                        c.qempty[t].arrive()
            free(k)
        for j in range(max(nb)):
            aborted = c.kv.go(aborted)
            v = take(1)
            k = take(c.keys) if j + 1 < max(nb) else []
            for t in range(2):
                if j >= nb[t]:
                    continue
                aborted = c.p[t].go(aborted)
                if aborted:
                    continue
                if j == nb[t] - 1:
                    c.ofull[t].arrive()
                if j + 1 < nb[t]:
                    c.sfull[t].arrive()
                    if j + 1 == nb[t] - 1:
                        c.qempty[t].arrive()
            if not aborted:
                free(v + k)


def softmax4(c, t):
    s_it = q_it = 0
    aborted = False
    for *nb, nothing, _ in c.walk:
        if nothing:
            continue
        if nb[t] == 0:
            with c.lock:
                c.written += 1
            continue
        if not aborted:
            aborted = not c.wait(c.qfull[t], q_it & 1)
        if not aborted:
            c.qready[t].arrive()
        if aborted and c.early:
            return
        for _ in range(nb[t]):
            if not aborted:
                aborted = not c.wait(c.sfull[t], s_it & 1)
            s_it += 1
            aborted = c.p[t].go(aborted)
        if not aborted:
            aborted = not c.wait(c.ofull[t], q_it & 1)
        q_it += 1
        if not aborted:
            with c.lock:
                c.written += 1


ROLES = [(producer4, ()), (relay4, ()), (issuer4, ()), (softmax4, (0,)), (softmax4, (1,))] + [(widen, ())] * 4


@pytest.mark.parametrize("keys", [1, 2])
@pytest.mark.parametrize("n", range(len(WALKS)))
def test_clean_walk_writes_every_tile(n, keys):
    c = Tile4(WALKS[n], 0.0, n, keys)
    hangs, alive = run_roles(c, ROLES)
    assert not hangs and alive == 0 and not c.abort
    assert c.written == 2 * sum(not p[2] for p in c.walk)


@pytest.mark.parametrize("keys", [1, 2])
@pytest.mark.parametrize("seed", range(16))
def test_wait_failures_never_hang(seed, keys):
    c = Tile4(WALKS[seed % len(WALKS)], [0.003, 0.02, 0.1, 0.3][seed % 4], seed, keys)
    hangs, alive = run_roles(c, ROLES)
    assert not hangs and alive == 0, hangs


def test_model_catches_a_softmax_that_leaves_before_its_queries():
    walk = max(WALKS, key=lambda w: sum(sum(p[:2]) for p in w))
    assert any(any(run_roles(Tile4(walk, 0.3, 100 + s, 1, early=True), ROLES)) for s in range(6))


def test_model_catches_queries_that_nobody_prepares():
    c = Tile4(WALKS[0], 0.0, 1, 1)
    roles = [r for r in ROLES if r[0] is not softmax4] + [(softmax, (0,)), (softmax, (1,))]
    hangs, alive = run_roles(c, roles)
    assert hangs or alive or c.abort
