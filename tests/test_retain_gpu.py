"""Accumulated attention weights and eviction: CUDA path vs the oracle.

Weights.  A term exp(s - lse) is off by the score's error d_j, the rounding of
lse log2(e) and of the difference (each 2^-24 of its size, at most L = max |lse| +
max |s|), and the exponential's 2^-22; n terms are summed in fp32 (n 2^-24), and the
sum is added to the weight (2^-24 of it).  d_j: over 16 bits, d exact products
summed, d 2^-24 M with M = scale max sum |q| |k|; over 4 bits 48 2^-24 M with
M = scale max sum |q| (|m| + 15 s) (test_kv4_gpu.py).  So
|w - ref| <= (d_j + 2 L 2^-24 + 2^-21 + n 2^-24) new + 2^-24 ref.

Eviction moves bytes: everything is equal.
"""
import numpy as np
import pytest
import torch

import oracle
import test_paged_gpu as paged
from helpers import to64
from test_kv4_gpu import exact4, largest, pack4, parts4
from test_paged_gpu import CHUNKS, DECODE, DRAFTS, cuda_i32, widen

pytestmark = pytest.mark.gpu


def make(lens, Hq, Hkv, d, page, dtype, bits, causal, seed, **kw):
    """A batch, its lse from the oracle, and weights to begin with (poison where
    no position of a sequence lies)."""
    x = paged.make(lens, Hq, Hkv, d, page, dtype, seed=seed, **kw)
    dt = x["q"].dtype
    if bits == 4:
        x["k"] = pack4(x["k"])
    x["exact"] = exact4(x["k"], dt) if bits == 4 else x["k"].double()
    v = torch.where(torch.isnan(x["v"]), x["v"].new_zeros(()), x["v"])
    _, L, _, x["big"] = oracle.attention_paged(to64(x["q"]), to64(x["exact"]), to64(v), x["table"].cpu().numpy(),
                                              x["cu"].cpu().numpy(), x["kv"].cpu().numpy(), causal, d ** -0.5)
    x["lse"] = torch.tensor(L, dtype=torch.float32).cuda()
    g = torch.Generator().manual_seed(seed + 1)
    w = torch.rand(x["k"].shape[:3], generator=g).cuda() * 4
    x["weights"] = w.masked_fill(torch.isnan(x["exact"]).any(-1), float("nan"))
    x["bits"] = bits
    return x


def call(attn, x, causal, weights=None, **kw):
    w = x["weights"].clone() if weights is None else weights
    attn.kv_weights(x["q"], x["k"], x["table"], x["cu"], x["kv"], x["lse"], w, x["max_q"], causal=causal, **kw)
    return w


def check(x, got, causal):
    dt, d = x["q"].dtype, x["q"].shape[2]
    cu, kv = x["cu"].cpu().numpy(), x["kv"].cpu().numpy()
    ref, new = oracle.weights_paged(to64(x["q"]), to64(x["exact"]), to64(x["lse"]), to64(x["weights"]),
                                    x["table"].cpu().numpy(), cu, kv, causal, d ** -0.5)
    if x["bits"] == 4:
        s, m, _ = parts4(x["k"], dt)
        err = 48 * 2.0 ** -24 * largest(x, causal, d ** -0.5, m.abs() + 15 * s)
    else:
        err = d * 2.0 ** -24 * largest(x, causal, d ** -0.5, x["exact"].abs())
    lse = to64(x["lse"])[:, :int(cu[-1])]
    L = np.max(np.abs(lse), where=np.isfinite(lse), initial=0.0) + x["big"]
    n = x["max_q"] * (x["q"].shape[0] // x["k"].shape[1])
    tol = (err + 2 * L * 2.0 ** -24 + 2.0 ** -21 + n * 2.0 ** -24) * new + 2.0 ** -24 * np.abs(ref)
    got = to64(got)
    outside = np.isnan(ref)  # no position of a sequence: left as it was
    assert np.array_equal(np.isnan(got), outside)
    assert (np.abs(got - ref) <= tol)[~outside].all(), float(np.max((np.abs(got - ref) - tol)[~outside]))


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("bits", [4, 16])
@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("fp16", 64), ("bf16", 96)])
@pytest.mark.parametrize("lens,Hq,Hkv,page", [
    (DECODE, 4, 1, 16), (DECODE * 5, 2, 2, 64), (DRAFTS, 10, 2, 32), (DRAFTS, 3, 1, 256), (CHUNKS, 4, 2, 16),
    (CHUNKS, 7, 1, 128), ([(1, 5)], 1, 1, 16), ([(32, 3000)], 8, 2, 64), ([(2, 600), (9, 50)], 128, 1, 16),
    ([(1, 1)] * 400, 1, 1, 16), ([(18, 20)] * 40, 1, 1, 16), ([(1, 2000), (0, 50)], 24, 8, 32)])
def test_weights(attn_lib, causal, bits, dtype, d, lens, Hq, Hkv, page):
    x = make(lens, Hq, Hkv, d, page, dtype, bits, causal, seed=d + page + len(lens), pad=2)
    got = call(attn_lib, x, causal)
    assert attn_lib.poll_status() == (0, 0)
    check(x, got, causal)
    again = call(attn_lib, widen(x), causal)  # a longer table, run again: the same bits
    assert torch.equal(again.view(torch.int32), got.view(torch.int32))


@pytest.mark.parametrize("bits", [4, 16])
@pytest.mark.parametrize("lens", [[(4, 0), (3, 2), (1, 7)], [(150, 40), (30, 0), (200, 199)]])
def test_weights_of_rows_without_a_key(attn_lib, bits, lens):
    """Rows before the first key have lse -inf and add nothing."""
    x = make(lens, 4, 2, 64, 16, "bf16", bits, True, seed=5)
    got = call(attn_lib, x, True)
    assert attn_lib.poll_status() == (0, 0)
    check(x, got, True)


@pytest.mark.parametrize("bits", [4, 16])
@pytest.mark.parametrize("lens", [DECODE, CHUNKS])
def test_weights_sum_to_the_rows(attn_lib, bits, lens):
    """What a call adds over all positions is 1 for each row and head that sees a key."""
    x = make(lens, 4, 2, 128, 16, "fp16", bits, True, seed=9)
    zero = torch.zeros_like(x["weights"])
    call(attn_lib, x, True, weights=zero)
    rows = sum(1 for n, k in lens for i in range(n) if i + k - n >= 0)
    assert abs(zero.double().sum().item() - 4 * rows) <= 2.0 ** -15 * 4 * rows


def test_weights_of_nan_and_infinite_rows(attn_lib):
    """A NaN query, or a NaN lse, makes the weights of the keys it sees NaN, and no
    others; an lse of +inf adds 0."""
    lens = [(3, 90), (1, 40), (2, 70)]
    x = make(lens, 2, 1, 64, 16, "bf16", 16, True, seed=15)
    clean = call(attn_lib, x, True)
    q = x["q"].clone()
    q[1, 1] = float("nan")  # sequence 0, its second row: keys 0 .. 88
    got = call(attn_lib, dict(x, q=q), True)
    lse = x["lse"].clone()
    lse[0, 3] = float("nan")  # sequence 1: all 40 keys
    got2 = call(attn_lib, dict(x, lse=lse), True)
    table = x["table"].tolist()
    for w, b, seen in ((got, 0, 89), (got2, 1, 40)):
        hit = torch.zeros(w.shape[0], 16, dtype=torch.bool, device="cuda")
        for j in range(seen):
            hit[table[b][j // 16], j % 16] = True
        assert torch.isnan(w[:, 0][hit]).all()
        assert torch.equal(w[:, 0][~hit].view(torch.int32), clean[:, 0][~hit].view(torch.int32))
    lse = torch.full_like(x["lse"], float("inf"))
    w = call(attn_lib, dict(x, lse=lse), True)
    for b, (n, k) in enumerate(lens):
        for j in range(k):
            at = table[b][j // 16], 0, j % 16
            assert w[at] == (x["weights"][at] if j < k - n else 0.0)


@pytest.mark.parametrize("bits", [4, 16])
@pytest.mark.parametrize("lens", [[(1, 50), (1, 40), (1, 30)], [(50, 50), (1, 40), (20, 30)]])
def test_weights_report_bad_pages_lengths_and_offsets(attn_lib, bits, lens):
    x = make(lens, 4, 2, 64, 16, "bf16", bits, True, seed=13)
    good = call(attn_lib, x, True)
    cu, table = x["cu"].tolist(), x["table"].tolist()
    cases = []
    for page in (-1, 1 << 30, x["k"].shape[0]):
        t = x["table"].clone()
        t[1, 1] = page
        cases.append(dict(x, table=t))
    for n in (x["table"].shape[1] * 16 + 1, -3):
        kv = x["kv"].clone()
        kv[1] = n
        cases.append(dict(x, kv=kv, table=x["table"].clamp(max=x["k"].shape[0] - 1)))
    for i, c in enumerate(cases):
        w = call(attn_lib, c, True)
        st, detail = attn_lib.poll_status()
        if i == 3:  # the padding of the table is no page of the sequence
            assert st == 1
            continue
        assert st == 1 and detail >> 16 == 1, (i, st, hex(detail))
        for b in (0, 2):
            for j in range(lens[b][1]):
                at = table[b][j // 16], slice(None), j % 16
                assert torch.equal(w[at], good[at]), (i, b, j)
    for bad in (cu[:2] + [cu[1] - 1] + cu[3:], cu[:-1] + [cu[-1] + 9], [1] + cu[1:]):
        call(attn_lib, dict(x, cu=cuda_i32(bad)), True)
        assert attn_lib.poll_status()[0] == 1
    assert torch.equal(call(attn_lib, x, True).view(torch.int32), good.view(torch.int32))
    assert attn_lib.poll_status() == (0, 0)


# ---------------------------------------------------------------- eviction ---

def cache(lens, Hkv, d, page, bits, seed, weights="tails", extra=2):
    g = torch.Generator().manual_seed(seed)
    need = [-(-n // page) for n in lens]
    n_pages = sum(need) + extra
    order = torch.randperm(n_pages, generator=g).tolist()
    width = max(1, max(need)) + 1
    table, at = np.full((len(lens), width), -1), 0
    for b, m in enumerate(need):
        table[b, :m] = order[at:at + m]
        at += m
    shape = (n_pages, Hkv, page, d // 8 * 5 if bits == 4 else d)
    dtype = torch.uint8 if bits == 4 else torch.int16
    k, v = (torch.randint(0, 256 if bits == 4 else 30000, shape, generator=g).to(dtype) for _ in range(2))
    w = torch.rand(shape[:3], generator=g)
    if weights == "tails":
        w = (w ** 8 * 4096).round() / 1024
    elif weights == "few":  # a handful of values
        w = (w * 5).floor()
    elif weights == "equal":
        w = torch.full(shape[:3], 0.25)
    elif weights == "wild":
        pick = torch.randint(0, 9, shape[:3], generator=g)
        for i, value in enumerate([float("nan"), float("inf"), float("-inf"), -0.0, 0.0, -1.5, 1e-42]):
            w = torch.where(pick == i, torch.tensor(value), w)
    if bits == 16:
        k, v = k.view(torch.bfloat16), v.view(torch.bfloat16)
    return dict(k=k.cuda(), v=v.cuda(), w=w.cuda(), table=cuda_i32(table), kv=cuda_i32(lens))


def raw(t):
    return t.view(torch.uint8 if t.dtype == torch.uint8 else {2: torch.int16, 4: torch.int32}[t.element_size()])


def evict(attn, x, budget, sinks, recent, **kw):
    y = {n: t.clone() for n, t in x.items()}
    kept, lens = attn.evict_kv(y["k"], y["v"], y["w"], y["table"], y["kv"], budget, sinks=sinks, recent=recent, **kw)
    return y, kept, lens


def check_evict(x, y, kept, lens, budget, sinks, recent):
    pages = [raw(x[n]).cpu().numpy() for n in ("k", "v", "w")]
    out, want, new = oracle.evict_paged(pages, x["w"].cpu().numpy(), x["table"].cpu().numpy(),
                                        x["kv"].cpu().numpy(), budget, sinks, recent)
    assert np.array_equal(kept.cpu().numpy(), want)
    assert np.array_equal(lens.cpu().numpy(), new)
    for n, o in zip(("k", "v", "w"), out):
        assert np.array_equal(raw(y[n]).cpu().numpy(), o), n
    assert torch.equal(y["kv"], x["kv"]) and torch.equal(y["table"], x["table"])


SHAPES = [([100], 1, 16, 40, 0, 0), ([0, 1, 39, 40, 41, 300], 2, 16, 40, 4, 8), ([700, 5, 650], 3, 64, 64, 0, 64),
          ([700, 699], 2, 32, 600, 17, 33), ([5000], 1, 256, 1000, 4, 200), ([333] * 30, 5, 16, 100, 3, 20),
          ([90] * 400, 1, 32, 17, 1, 1), ([2049, 2048, 1], 2, 128, 1, 0, 0), ([64, 65], 1, 64, 64, 64, 0),
          ([1000, 40], 2, 16, 500, 250, 250), ([3000] * 9, 4, 64, 2999, 0, 0)]


@pytest.mark.parametrize("bits,d", [(16, 128), (16, 64), (16, 96), (16, 192), (16, 256), (4, 128), (4, 64), (4, 96)])
@pytest.mark.parametrize("weights", ["tails", "wild"])
@pytest.mark.parametrize("lens,Hkv,page,budget,sinks,recent", SHAPES)
def test_evict(attn_lib, bits, d, weights, lens, Hkv, page, budget, sinks, recent):
    x = cache(lens, Hkv, d, page, bits, seed=d + len(lens), weights=weights)
    y, kept, new = evict(attn_lib, x, budget, sinks, recent)
    assert attn_lib.poll_status() == (0, 0)
    check_evict(x, y, kept, new, budget, sinks, recent)


@pytest.mark.parametrize("weights", ["few", "equal", "tails"])
@pytest.mark.parametrize("lens,Hkv", [([70000], 1), ([9000, 33000], 2), ([1500] * 100, 2)])
@pytest.mark.parametrize("share", [0.1, 0.5, 0.99])
def test_evict_long_and_many(attn_lib, weights, lens, Hkv, share):
    x = cache(lens, Hkv, 64, 64, 4, seed=len(lens), weights=weights)
    budget = int(max(lens) * share)
    y, kept, new = evict(attn_lib, x, budget, 4, budget // 4)
    assert attn_lib.poll_status() == (0, 0)
    check_evict(x, y, kept, new, budget, 4, budget // 4)


@pytest.mark.parametrize("seed", range(24))
def test_random_eviction(attn_lib, seed):
    g = np.random.default_rng(seed)
    bits = int(g.choice([4, 16]))
    d = int(g.choice([64, 96, 128]))
    lens = [int(g.integers(0, int(g.choice([30, 400, 3000])))) for _ in range(int(g.choice([1, 3, 20])))]
    budget = int(g.integers(1, max(lens) + 5))
    sinks = int(g.integers(0, budget + 1)) if g.random() < 0.5 else 0
    recent = int(g.integers(0, budget - sinks + 1)) if g.random() < 0.7 else 0
    x = cache(lens, int(g.choice([1, 2, 5])), d, int(g.choice([16, 32, 64, 128, 256])), bits, seed=seed,
              weights=str(g.choice(["tails", "few", "wild"])))
    y, kept, new = evict(attn_lib, x, budget, sinks, recent)
    assert attn_lib.poll_status() == (0, 0)
    check_evict(x, y, kept, new, budget, sinks, recent)


def test_eviction_reports_bad_pages_and_lengths(attn_lib):
    """A page outside the cache and lengths out of range: reported; the other
    sequences are cut as ever, and nothing outside the pages is touched."""
    x = cache([200, 210, 220], 2, 64, 16, 16, seed=3)
    good = evict(attn_lib, x, 100, 4, 10)
    assert attn_lib.poll_status() == (0, 0)
    cases = []
    for page in (-1, 1 << 30, x["k"].shape[0]):
        t = x["table"].clone()
        t[1, 3] = page
        cases.append((dict(x, table=t), 1))
    for n in (-5, x["table"].shape[1] * 16 + 1):
        kv = x["kv"].clone()
        kv[1] = n
        cases.append((dict(x, kv=kv, table=x["table"].clamp(min=0)), 1))
    for c, bad in cases:
        y, kept, new = evict(attn_lib, c, 100, 4, 10)
        st, detail = attn_lib.poll_status()
        assert st == 1 and detail >> 16 == bad
        for b in (0, 2):
            assert torch.equal(kept[b], good[1][b]) and new[b] == 100
            at = c["table"][b, :7].long()
            if c["kv"][1] <= 220:  # (a length past the table's pages reaches other sequences' pages)
                assert torch.equal(raw(y["k"])[at], raw(good[0]["k"])[at])


def test_captured_eviction_replays(attn_lib):
    """A graph of weights and eviction, replayed on new contents of the same
    tensors on a side stream."""
    xs = [cache([300, 500, 90], 2, 64, 16, 4, seed=s) for s in (21, 22)]
    kvs = [cuda_i32([300, 500, 90]), cuda_i32([290, 120, 90])]
    hold = {n: t.clone() for n, t in xs[0].items()}
    kept = torch.empty(3, 2, 128, dtype=torch.int32, device="cuda")
    lens = torch.empty(3, dtype=torch.int32, device="cuda")
    attn_lib.evict_kv(*(hold[n] for n in ("k", "v", "w", "table", "kv")), 128, 4, 30, kept=kept, new_lens=lens)
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=side):
        attn_lib.evict_kv(*(hold[n] for n in ("k", "v", "w", "table", "kv")), 128, 4, 30, kept=kept, new_lens=lens)
    for i in (0, 1, 1, 0):
        x = dict(xs[i], kv=kvs[i])
        for n in hold:
            hold[n].copy_(x[n])
        graph.replay()
        y = {n: t.clone() for n, t in hold.items()}
        check_evict(x, y, kept, lens, 128, 4, 30)
    assert attn_lib.poll_status() == (0, 0)


@pytest.mark.parametrize("bits", [4, 16])
def test_serving_run_with_eviction(attn_lib, bits):
    """As a server uses them together: prompts, then single tokens; every step
    appends, attends and adds up the weights, and a cache that has grown past its
    budget is cut.  Outputs stay the attention over what the cache holds, and
    what the cache holds is the oracle's choice."""
    Hq, Hkv, d, page, dt = 6, 2, 64, 16, torch.bfloat16
    budget, sinks, recent = 48, 2, 12
    rope = attn_lib.rope_table(d)
    table = cuda_i32(np.random.default_rng(0).permutation(24).reshape(2, 12))
    row = 40 if bits == 4 else d
    kp, vp = (torch.zeros(24, Hkv, page, row, dtype=torch.uint8 if bits == 4 else dt, device="cuda")
              for _ in range(2))
    w = torch.full((24, Hkv, page), 9e9, device="cuda")  # what pages held before does not count
    append, fwd = (attn_lib.append_kv4, attn_lib.fwd_paged4) if bits == 4 else (attn_lib.append_kv,
                                                                               attn_lib.fwd_paged)
    values = (lambda t: to64(exact4(t, dt))) if bits == 4 else to64
    kv, seen = np.array([0, 0]), np.array([0, 0])
    for step, new in enumerate([(70, 20), (10, 0), (1, 33), (1, 1), (1, 1), (4, 1), (1, 1)]):
        total = sum(new)
        g = torch.Generator().manual_seed(step)
        q, k, v = (torch.randn((h, total, d), generator=g).to(dt).cuda() for h in (Hq, Hkv, Hkv))
        kv, seen = kv + new, seen + new
        pos = torch.cat([torch.arange(a - n, a) for a, n in zip(seen, new)]).int().cuda()[None]  # in the text
        cu, lens = cuda_i32([0, new[0], total]), cuda_i32(kv)
        q = append(k, v, kp, vp, table, cu, lens, table=rope, positions=pos, q=q)
        o, lse = fwd(q, kp, vp, table, cu, lens, max(new), causal=True)
        before = w.clone()
        attn_lib.kv_weights(q, kp, table, cu, lens, lse, w, max(new), causal=True)
        x = dict(q=q, k=kp, exact=torch.tensor(values(kp)), lse=lse, weights=before, table=table, cu=cu, kv=lens,
                 bits=bits, max_q=max(new))
        O, L, A, x["big"] = oracle.attention_paged(to64(q), values(kp), values(vp), table.cpu().numpy(),
                                                   cu.cpu().numpy(), kv, True, d ** -0.5)
        assert np.max(np.abs(to64(o) - O)) <= 2.0 ** -6 * np.max(np.abs(A))
        x["lse"] = lse
        check(x, w, True)
        held = dict(k=kp.clone(), v=vp.clone(), w=w.clone(), table=table, kv=lens)
        kept, new_lens = attn_lib.evict_kv(kp, vp, w, table, lens, budget, sinks=sinks, recent=recent)
        check_evict(held, dict(k=kp, v=vp, w=w, table=table, kv=lens), kept, new_lens, budget, sinks, recent)
        kv = new_lens.cpu().numpy()
        assert attn_lib.poll_status() == (0, 0)
    assert kv.tolist() == [48, 48]


def test_weights_and_eviction_on_two_streams(attn_lib):
    xs = [make([(1, 900)] * 30, 4, 2, 64, 16, "bf16", 16, True, seed=3), make([(40, 700)] * 4, 4, 2, 64, 16, "bf16", 4,
                                                                              True, seed=4)]
    want = [call(attn_lib, x, True) for x in xs]
    cs = [cache([2000, 1500], 2, 64, 16, 16, seed=5), cache([700] * 20, 2, 64, 16, 4, seed=6)]
    cut = [evict(attn_lib, c, 400, 4, 30) for c in cs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in xs]
    got = []
    for _ in range(6):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got.append((i, call(attn_lib, xs[i], True), evict(attn_lib, cs[i], 400, 4, 30)))
    torch.cuda.synchronize()
    for i, w, (y, kept, lens) in got:
        assert torch.equal(w.view(torch.int32), want[i].view(torch.int32))
        assert torch.equal(kept, cut[i][1]) and torch.equal(lens, cut[i][2])
        assert all(torch.equal(raw(y[n]), raw(cut[i][0][n])) for n in ("k", "v", "w"))
    assert attn_lib.poll_status() == (0, 0)


@pytest.mark.parametrize("bits", [4, 16])
def test_caches_past_two_to_the_31(attn_lib, bits):
    """Pages at both ends of a cache of more than 2^31 bytes (4 bits) or elements."""
    Hkv, d, page = 2, 128, 64
    n_pages = 460_000 if bits == 4 else 147_000
    small = cache([500], Hkv, d, page, bits, seed=8, extra=0)
    k, v = (torch.empty((n_pages,) + tuple(small["k"].shape[1:]), dtype=small["k"].dtype, device="cuda")
            for _ in range(2))
    assert k.numel() > 2 ** 31
    w = torch.empty((n_pages, Hkv, page), device="cuda")
    far = torch.tensor([n_pages - 1, 0, n_pages - 2, 7, n_pages // 2, n_pages - 9, 1, n_pages - 70][:8], device="cuda")
    for big, t in ((k, small["k"]), (v, small["v"]), (w, small["w"])):
        big[far] = t
    table = torch.where(small["table"] >= 0, far[small["table"].clamp(min=0).long()].int(), small["table"])
    kept, lens = attn_lib.evict_kv(k, v, w, table, small["kv"], 200, sinks=3, recent=20)
    y = dict(small, k=k[far], v=v[far], w=w[far])
    assert attn_lib.poll_status() == (0, 0)
    check_evict(small, y, kept, lens, 200, 3, 20)
    if bits == 4:
        k[far] = pack4(torch.randn(8, Hkv, page, d).bfloat16()).cuda()
    q = torch.randn(4, 1, d, device="cuda").bfloat16()
    lse = torch.full((4, 1), 5.0, device="cuda")
    if bits == 16:
        k[far] = torch.randn(8, Hkv, page, d, device="cuda").bfloat16()
    one = [t.clone() for t in (k[far], w[far])]
    args = cuda_i32([0, 1]), small["kv"], lse
    attn_lib.kv_weights(q, k, table, *args, w, 1)
    attn_lib.kv_weights(q, one[0], small["table"], *args, one[1], 1)
    assert torch.equal(w[far], one[1])
    assert attn_lib.poll_status() == (0, 0)


def test_binding_refuses_wrong_tensors(attn_lib):
    x = make([(1, 5), (2, 40)], 4, 2, 64, 16, "bf16", 16, True, seed=71)
    w = x["weights"]
    good = [x["q"], x["k"], x["table"], x["cu"], x["kv"], x["lse"], w, 2]
    bad = [(0, x["q"].half(), ValueError), (0, x["q"].float(), TypeError), (0, x["q"].cpu(), ValueError),
           (0, x["q"][:3], ValueError), (0, None, TypeError), (1, x["k"].transpose(1, 2), ValueError),
           (1, x["k"].half(), ValueError), (1, pack4(x["k"])[..., :32], ValueError), (2, x["table"].long(), ValueError),
           (3, x["cu"][:2], ValueError), (4, x["kv"][None], ValueError), (5, x["lse"].half(), ValueError),
           (5, x["lse"][:, :2], ValueError), (5, x["lse"].t(), ValueError), (6, w.half(), ValueError),
           (6, w[1:], ValueError), (6, w.transpose(1, 2), ValueError), (6, w.cpu(), ValueError), (6, None, TypeError),
           (7, 0, ValueError), (7, 4, ValueError)]
    for i, value, error in bad:
        with pytest.raises(error):
            attn_lib.kv_weights(*(good[:i] + [value] + good[i + 1:]))
    with pytest.raises(attn_lib.AttnError):
        attn_lib.kv_weights(*good, scale=-1.0)
    c = cache([60, 70], 2, 64, 16, 16, seed=1)
    good2 = [c["k"], c["v"], c["w"], c["table"], c["kv"], 50]
    bad = [(0, c["k"].float(), TypeError), (0, c["k"][1:], ValueError), (0, c["k"].cpu(), ValueError),
           (0, c["v"].half(), ValueError), (1, c["v"].transpose(0, 1), ValueError), (1, None, TypeError),
           (2, c["w"].double(), ValueError), (2, c["w"][..., :8], ValueError), (3, c["table"].long(), ValueError),
           (3, c["table"][:1], ValueError), (4, c["kv"].cpu(), ValueError), (5, 0, ValueError), (5, "x", ValueError),
           (5, 1 << 40, ValueError)]
    for i, value, error in bad:
        with pytest.raises(error):
            attn_lib.evict_kv(*(good2[:i] + [value] + good2[i + 1:]))
    for kw in (dict(sinks=-1), dict(recent=-1), dict(sinks=30, recent=21), dict(kept=c["kv"]),
               dict(kept=torch.empty(2, 2, 50, device="cuda")), dict(new_lens=c["kv"].long()),
               dict(new_lens=c["table"])):
        with pytest.raises(ValueError):
            attn_lib.evict_kv(*good2, **kw)
    for args, kw in ((good2, dict(new_lens=c["kv"])), ([c["k"], c["k"]] + good2[2:], {})):
        with pytest.raises(attn_lib.AttnError):
            attn_lib.evict_kv(*args, **kw)
    odd = torch.zeros(10, 2, 16, 80, dtype=torch.bfloat16, device="cuda")  # d = 80
    with pytest.raises(attn_lib.AttnError) as e:
        attn_lib.evict_kv(odd, odd.clone(), torch.zeros(10, 2, 16, device="cuda"), *good2[3:])
    assert e.value.status == 2
    assert attn_lib.poll_status() == (0, 0)
    attn_lib.kv_weights(*good)
    attn_lib.evict_kv(*good2)
    assert attn_lib.poll_status() == (0, 0)
