"""Host models of the paged attention kernels (no GPU): how a batch is cut into
shares, and how their roles wind down when a bounded wait runs out.

The partition is restated here (items laid end to end by cost, equal shares, a
key block to the share its first key falls in) and checked for what the kernels
rely on: every key block of every item in one piece, parts numbered in the order
of the CTAs, each item's rows seen to once.  Its pieces then drive the models.

The tile kernel's issuer meets the relay warp and the softmax warpgroups at
named barriers, which have no time limit; after an abort every role walks the
pieces to the end with waits and work skipped, so each barrier generation pairs
up.  Its roles decide for themselves which pieces to skip (a share that ends in
an item's overhead, rows without a key, a tile that sees none of a piece's
keys).  The decoding kernel's warps leave a piece together, at a block barrier,
and the CTAs of a cluster meet twice at its end whether they gave up or not.
"""
import random
import threading

import pytest

from test_fwd_protocol_model import CTA, HANG_S, SLOTS, Hang, MBar

CTAS = 152
TILE = dict(unit=128, key1=3, key2=4, overhead=1024, single=False, min_share=1024)
DECODE = dict(unit=64, key1=1, key2=1, overhead=128, single=True, min_share=128)


# ------------------------------------------------------------ the partition ---

def items_of(seq, W, causal, cost):
    """(keys, second half has rows, cost) of the items of one key/value head."""
    qlen, klen = seq
    if cost["single"]:
        return [(klen, False, klen + cost["overhead"])] if qlen else []
    out = []
    for i in range(-(-qlen // W)):
        keys = max(min((i + 1) * W, qlen) + klen - qlen, 0) if causal else klen
        two = i * W + W // 2 < qlen
        out.append((keys, two, keys * cost["key2" if two else "key1"] + cost["overhead"]))
    return out


def line_cost(seq, W, causal, cost, q):
    """Cost of the first q items in closed form, as the kernels sum it."""
    qlen, klen = seq
    if q == 0:
        return 0
    if cost["single"]:
        return cost["overhead"] + klen * cost["key1"]
    koff, keys = klen - qlen, 0
    if not causal:
        keys = (q - 1) * klen
    else:
        i0 = 0 if koff + W > 0 else -koff // W
        n = q - 1 - i0
        if n > 0:
            keys = n * ((i0 + 1) * W + koff) + n * (n - 1) // 2 * W
    last, two, _ = items_of(seq, W, causal, cost)[q - 1]
    return q * cost["overhead"] + keys * cost["key2"] + last * cost["key2" if two else "key1"]


def pieces(batch, heads, W, causal, cost, ctas=CTAS):
    """Per CTA its pieces: (sequence, head, item, keys, two, u0, u1, whole,
    nothing, part, parts) in the order it walks them."""
    line = [(b, h, i, *it) for b, s in enumerate(batch) for h in range(heads)
            for i, it in enumerate(items_of(s, W, causal, cost))]
    total = sum(it[-1] for it in line)
    share = max(-(-total // ctas), cost["min_share"])
    out = [[] for _ in range(ctas)]
    at = 0
    for b, h, i, keys, two, c in line:
        unit = cost["unit"] * cost["key2" if two else "key1"]
        nb = -(-keys // cost["unit"])
        blocks = lambda x: min(-(-x // unit), nb)  # noqa: E731
        first, last = at // share, (at + c - 1) // share
        for cta in range(first, last + 1):
            x0 = max(cta * share - at, 0)
            x1 = min((cta + 1) * share - at, c)
            u0, u1 = blocks(x0), blocks(x1)
            parts = (at % share + (nb - 1) * unit) // share + 1 if nb else 1
            out[cta].append((b, h, i, keys, two, u0, u1, x0 == 0 and u1 == nb,
                             u0 == u1 and (nb > 0 or x0 > 0), -(-x0 // share), parts))
        at += c
    return out


BATCHES = [
    ([(17, 17), (1, 90), (128, 128), (129, 300), (0, 5), (5, 400), (63, 64), (200, 777)], 2, 64),
    ([(150, 40), (30, 0), (200, 199)], 2, 64), ([(20, 3500)], 1, 128), ([(40, 16000)], 1, 256),
    ([(33, 2000)], 1, 128),
    ([(700, 16000), (3, 1)], 3, 256), ([(18, 20)] * 60, 1, 256), ([(1, 1)] * 400, 1, 2),
    ([(300, 3000)] * 3, 8, 128), ([(4096, 16384)], 8, 128), ([(1, 0)] * 9 + [(1, 70000)], 2, 1)]


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("batch,heads,W", BATCHES)
@pytest.mark.parametrize("cost,ctas", [(TILE, CTAS), (DECODE, 2 * CTAS), (TILE, 7)])
def test_partition(batch, heads, W, causal, cost, ctas):
    got = pieces(batch, heads, W, causal, cost, ctas)
    seen = {}
    for cta, walk in enumerate(got):
        split = [p for p in walk if not p[7] and not p[8]]
        # a CTA has room for two parts: one it continues (first), one it begins (last)
        assert len(split) <= 2 and sum(p[9] == 0 for p in split) <= 1
        assert sum(p[9] > 0 for p in split) <= 1
        for p in walk:
            seen.setdefault(p[:3], []).append((cta, p))
    for b, s in enumerate(batch):
        its = items_of(s, W, causal, cost)
        for q in range(len(its) + 1):
            assert line_cost(s, W, causal, cost, q) == sum(it[2] for it in its[:q])
        for h in range(heads):
            for i, (keys, _, _) in enumerate(its):
                nb = -(-keys // cost["unit"])
                at = 0
                live = [(c, p) for c, p in seen[b, h, i] if not p[8]]
                for n, (cta, p) in enumerate(live):
                    assert p[5] == at and p[6] >= at
                    at = p[6]
                    # the join finds part n in CTA (first + n), and as many as there are
                    assert p[9] == n and cta == live[0][0] + n and p[10] == len(live)
                    assert p[7] == (len(live) == 1)
                assert at == nb and live


def test_partition_reaches_every_form_of_the_join():
    """2, 3 to 4, 5 to 8, 9 to 16 and more parts occur among the batches."""
    parts = {p[10] for batch, heads, W in BATCHES for walk in pieces(batch, heads, W, True, TILE)
             for p in walk if not p[7] and not p[8]}
    for lo, hi in ((2, 2), (3, 4), (5, 8), (9, 16), (17, CTAS)):
        assert any(lo <= n <= hi for n in parts), (lo, hi, sorted(parts))


# ---------------------------------------------------------- the tile kernel ---

def tile_blocks(p, batch, W, causal):
    """Key blocks of the piece that tile 0 and tile 1 see."""
    qlen, klen = batch[p[0]]
    keys, two, u0, u1 = p[3], p[4], p[5], p[6]
    k0 = -(-keys // 128)
    if two and causal:
        k0 = max((2 * p[2] + 1) * (W // 2) + klen - qlen, 0) + 127 >> 7
    return max(min(u1, k0) - u0, 0), (u1 - u0 if two else 0)


class Tile(CTA):
    def __init__(self, walk, fail_p, seed, early=False):
        super().__init__(fail_p, seed, early)
        self.walk = walk  # (blocks of tile 0, of tile 1, nothing, whole)
        self.written, self.described = 0, 0


def producer(c):
    kv_it, q_it = 0, [0, 0]
    for *nb, _, _ in c.walk:
        if max(nb) == 0:
            continue
        for t in range(2):
            if nb[t] == 0:
                continue
            if not c.wait(c.qempty[t], (q_it[t] & 1) ^ 1):
                return
            c.qfull[t].arrive()
            q_it[t] += 1
        for _ in range(2 * max(nb)):
            slot = kv_it % SLOTS
            if not c.wait(c.kvempty[slot], ((kv_it // SLOTS) & 1) ^ 1):
                return
            c.kvfull[slot].arrive()
            kv_it += 1


def relay(c):
    kv_it, q_it, aborted = 0, [0, 0], False

    def kv_ready():
        nonlocal kv_it, aborted
        slot, par = kv_it % SLOTS, (kv_it // SLOTS) & 1
        kv_it += 1
        if not aborted:
            aborted = not c.wait(c.kvfull[slot], par)

    for *nb, nothing, whole in c.walk:
        if not nothing and not whole:
            c.described += 1
        if max(nb) == 0:
            continue
        for t in range(2):
            if nb[t] == 0:
                continue
            par = q_it[t] & 1
            q_it[t] += 1
            if not aborted:
                aborted = not c.wait(c.qfull[t], par)
        kv_ready()
        aborted = c.kv.go(aborted)
        for j in range(max(nb)):
            kv_ready()
            if j + 1 < max(nb):
                kv_ready()
            aborted = c.kv.go(aborted)


def issuer(c):
    kv_it, aborted = 0, False
    for *nb, _, _ in c.walk:
        if max(nb) == 0:
            continue
        aborted = c.kv.go(aborted)
        kslot = kv_it % SLOTS
        kv_it += 1
        if not aborted:
            for t in range(2):
                if nb[t] > 0:
                    c.sfull[t].arrive()
                    if nb[t] == 1:
                        c.qempty[t].arrive()
            c.kvempty[kslot].arrive()
        for j in range(max(nb)):
            aborted = c.kv.go(aborted)
            vslot = kv_it % SLOTS
            kv_it += 1
            have_next = j + 1 < max(nb)
            if have_next:
                kslot = kv_it % SLOTS
                kv_it += 1
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
                c.kvempty[vslot].arrive()
                if have_next:
                    c.kvempty[kslot].arrive()


def softmax(c, t):
    s_it = o_it = 0
    aborted = False
    for *nb, nothing, _ in c.walk:
        if nothing:
            continue
        if nb[t] == 0:
            with c.lock:
                c.written += 1
            continue
        for _ in range(nb[t]):
            par = s_it & 1
            s_it += 1
            if not aborted:
                aborted = not c.wait(c.sfull[t], par)
            if aborted and c.early:
                return
            aborted = c.p[t].go(aborted)
        par = o_it & 1
        o_it += 1
        if not aborted:
            aborted = not c.wait(c.ofull[t], par)
        if not aborted:
            with c.lock:
                c.written += 1


def run_roles(c, roles):
    hangs = []

    def wrap(f, *a):
        try:
            f(c, *a)
        except Hang as e:
            hangs.append(str(e))

    threads = [threading.Thread(target=wrap, args=(f,) + a, daemon=True) for f, a in roles]
    for th in threads:
        th.start()
    for th in threads:
        th.join(4 * HANG_S)
    return hangs, sum(th.is_alive() for th in threads)


TILE_ROLES = [(producer, ()), (relay, ()), (issuer, ()), (softmax, (0,)), (softmax, (1,))]


def walks():
    """The most varied walks of a few batches: short ones of many pieces, parts
    of items, pieces without a key, tiles that end early."""
    out = []
    for batch, heads, W in BATCHES[:7]:
        for causal in (True, False):
            cut = pieces(batch, heads, W, causal, TILE, 7 if len(batch) > 2 else CTAS)
            for walk in cut:
                w = [(*tile_blocks(p, batch, W, causal), p[8], p[7]) for p in walk]
                if w and sum(max(p[:2]) for p in w) <= 40:
                    out.append(w)
    out.sort(key=lambda w: -len({(min(p[0], 2), min(p[1], 2), p[2], p[3]) for p in w}))
    return out[:16]


WALKS = walks()


def test_walks_hold_every_kind_of_piece():
    kinds = {(p[0] > 0, p[1] > 0, p[2], p[3]) for w in WALKS for p in w}
    assert {(True, True, False, True), (True, False, False, True), (True, True, False, False),
            (False, False, False, True), (False, False, True, False)} <= kinds
    assert any(0 < p[0] < p[1] for w in WALKS for p in w)


@pytest.mark.parametrize("n", range(len(WALKS)))
def test_tile_kernel_clean_walk_writes_every_tile(n):
    c = Tile(WALKS[n], 0.0, n)
    hangs, alive = run_roles(c, TILE_ROLES)
    assert not hangs and alive == 0 and not c.abort
    assert c.written == 2 * sum(not p[2] for p in c.walk)
    assert c.described == sum(not p[2] and not p[3] for p in c.walk)


@pytest.mark.parametrize("seed", range(24))
def test_tile_kernel_wait_failures_never_hang(seed):
    c = Tile(WALKS[seed % len(WALKS)], [0.005, 0.02, 0.1, 0.3][seed % 4], seed)
    hangs, alive = run_roles(c, TILE_ROLES)
    assert not hangs and alive == 0, hangs


def test_model_catches_tile_softmax_that_leaves_early():
    walk = max(WALKS, key=lambda w: sum(sum(p[:2]) for p in w))
    assert any(any(run_roles(Tile(walk, 0.3, 100 + s, early=True), TILE_ROLES)) for s in range(6))


# ------------------------------------------------------ the decoding kernel ---

class Barrier:
    """Barrier of n threads returning the OR of their predicates."""

    def __init__(self, name, n):
        self.name, self.n = name, n
        self.cv = threading.Condition()
        self.count, self.acc, self.gen, self.res = 0, False, 0, {}

    def go(self, pred=False):
        with self.cv:
            g = self.gen
            self.acc |= pred
            self.count += 1
            if self.count == self.n:
                self.res[g], self.count, self.acc = self.acc, 0, False
                self.gen += 1
                self.cv.notify_all()
            elif not self.cv.wait_for(lambda: self.gen > g, timeout=HANG_S):
                raise Hang(f"{self.name} generation {g}")
            return self.res[g]


WARPS, RING = 4, 3


class Decode:
    """A cluster of CTAs (one without CLUSTER): their warps' pieces, rings and
    barriers; copies land unless the model lets a wait fail."""

    def __init__(self, walk, ctas, rows, fail_p, seed, skip_cluster_sync=False):
        self.walk, self.ctas, self.rows = walk, ctas, rows
        self.cluster = Barrier("cluster", ctas * WARPS)
        self.block = [Barrier(f"block {i}", WARPS) for i in range(ctas)]
        self.abort = [False] * ctas
        self.skip = skip_cluster_sync
        self.lock = threading.Lock()
        self.rng = random.Random(seed)
        self.fail_p = fail_p
        self.done = [0] * ctas
        self.drained = 0

    def fails(self, cta):
        with self.lock:
            if self.abort[cta]:
                return True
            if self.rng.random() < self.fail_p:
                self.abort[cta] = True
                return True
        return False


def decode_warp(c, cta, warp):
    clustered = c.ctas > 1
    ring = [MBar() for _ in range(RING)]
    stream = [n for piece in c.walk[cta] for n in range(piece[warp])]
    issued = it = 0

    def issue():
        nonlocal issued
        if issued < len(stream):
            ring[issued % RING].arrive()  # the copy lands
            issued += 1

    for _ in range(RING):
        issue()
    given_up = False
    for piece in c.walk[cta]:
        aborted = False
        for _ in range(piece[warp]):
            if c.fails(cta):
                aborted = True
                break
            assert ring[it % RING].done((it // RING) & 1)
            it += 1
            issue()
        given_up = c.block[cta].go(aborted)
        if given_up:
            break
        for n in range(-(-c.rows // 4)):
            if n > 0:
                c.block[cta].go()
            c.block[cta].go()
        if warp == 0:
            c.done[cta] += 1
    if clustered and not (given_up and c.skip):
        c.cluster.go()
        c.cluster.go()
    with c.lock:
        c.drained += issued - it
    for k in range(it, issued):
        assert ring[k % RING].done((k // RING) & 1)


def decode_walk(ctas, seed):
    g = random.Random(seed)
    if ctas > 1:  # one piece each, some without blocks
        return [[[g.randrange(0, 9) for _ in range(WARPS)]] for _ in range(ctas)]
    return [[[g.randrange(0, 7) for _ in range(WARPS)] for _ in range(5)]]


@pytest.mark.parametrize("ctas", [1, 2, 8])
@pytest.mark.parametrize("seed", range(8))
def test_decoding_kernel_wait_failures_never_hang(ctas, seed):
    fail_p = [0.0, 0.02, 0.1, 0.4][seed % 4]
    c = Decode(decode_walk(ctas, seed), ctas, 1 + seed * 2, fail_p, seed)
    hangs, alive = run_roles(c, [(decode_warp, (i, w)) for i in range(ctas) for w in range(WARPS)])
    assert not hangs and alive == 0, hangs
    if fail_p == 0.0:
        assert all(c.done[i] == len(c.walk[i]) for i in range(ctas)) and c.drained == 0


def test_model_catches_a_cta_that_leaves_its_cluster():
    walk = [[[4] * WARPS] for _ in range(2)]
    found = False
    for seed in range(6):
        c = Decode(walk, 2, 4, 0.1, seed, skip_cluster_sync=True)
        hangs, alive = run_roles(c, [(decode_warp, (i, w)) for i in range(2) for w in range(WARPS)])
        found = found or bool(hangs) or alive > 0
    assert found
