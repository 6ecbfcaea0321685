"""Attention over a paged cache: CUDA path vs the fp64 oracle.

Tolerances, from the arithmetic.  The probabilities are rounded to 16 bits
before the product with V (half a step u each, at most u * A with A = sum_j
P_ij |v_j|) and the output once more (u |O|).  In fp32: a score is a sum of d
exact products (d 2^-24 of its size, carried into P by the exponential), the
sums over n keys lose at most n 2^-24, and the exponential and the joins a few
2^-22.  So |O - O_ref| <= (u + e) A + u |O| and |LSE - LSE_ref| <= e + 2^-23
|LSE| with e = 2^-20 + n 2^-24 + d 2^-24 max |S|, u = finfo.eps / 2.
"""
import numpy as np
import pytest
import torch

import oracle
from helpers import to64

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp16": torch.float16}


def cuda_i32(a):
    return torch.tensor(np.asarray(a), dtype=torch.int32, device="cuda")


def make(lens, Hq, Hkv, d, page, dtype, seed=0, pad=0, amp=1.0):
    """A batch with (new, keys) per sequence; every cache row outside the
    sequences, and every table entry past their lengths, is poison."""
    dt = DT[dtype]
    g = torch.Generator().manual_seed(seed)
    new, keys = [n for n, _ in lens], [k for _, k in lens]
    cu = np.concatenate([[0], np.cumsum(new)])
    width = max(1, -(-max(keys) // page)) + 1
    need = [-(-k // page) for k in keys]
    n_pages = sum(need) + 2
    order = torch.randperm(n_pages, generator=g).numpy()
    table = np.full((len(lens), width), 0x7FFFFFFF, np.int64)
    kp = torch.full((n_pages, Hkv, page, d), float("nan"), dtype=dt)
    vp = torch.full((n_pages, Hkv, page, d), float("nan"), dtype=dt)
    at = 0
    for b, (m, k) in enumerate(zip(need, keys)):
        table[b, :m] = order[at:at + m]
        at += m
        for j in range(m):
            n = min(page, k - j * page)
            kp[table[b, j], :, :n] = torch.randn((Hkv, n, d), generator=g).to(dt)
            vp[table[b, j], :, :n] = torch.randn((Hkv, n, d), generator=g).to(dt)
    q = (amp * torch.randn((Hq, int(cu[-1]) + pad, d), generator=g)).to(dt)
    if pad:
        q[:, int(cu[-1]):] = float("nan")
    return dict(q=q.cuda(), k=kp.cuda(), v=vp.cuda(), table=cuda_i32(table), cu=cuda_i32(cu),
                kv=cuda_i32(keys), max_q=max(max(new), 1))


def widen(x, keys=5000):
    """The same batch with a block table that reaches further (poison past the
    lengths): decoding then runs in equal shares, not in clusters."""
    t = x["table"]
    more = -(-keys // x["k"].shape[2]) - t.shape[1]
    if more <= 0:
        return x
    return dict(x, table=torch.cat([t, t.new_full((t.shape[0], more), 0x7FFFFFFF)], 1))


def run(attn, x, causal, **kw):
    return attn.fwd_paged(x["q"], x["k"], x["v"], x["table"], x["cu"], x["kv"], x["max_q"],
                          causal=causal, **kw)


def workspace_bytes(attn, x):
    return attn.fwd_paged_workspace_bytes(len(x["kv"]), x["max_q"],
                                          x["table"].shape[1] * x["k"].shape[2], x["q"].shape[0],
                                          x["k"].shape[1], x["q"].shape[2])


def check(x, o, lse, causal, scale=None):
    d = x["q"].shape[2]
    scale = d ** -0.5 if scale is None else scale
    cu, kv = x["cu"].cpu().numpy(), x["kv"].cpu().numpy()
    O, L, A, big = oracle.attention_paged(to64(x["q"]), to64(x["k"]), to64(x["v"]),
                                          x["table"].cpu().numpy(), cu, kv, causal, scale)
    live = slice(0, int(cu[-1]))
    u = torch.finfo(x["q"].dtype).eps / 2
    e = 2.0 ** -20 + int(kv.max()) * 2.0 ** -24 + d * 2.0 ** -24 * big
    got, ref = to64(o)[:, live], O[:, live]
    tiny = torch.finfo(x["q"].dtype).smallest_normal * u
    tol = (u + e) * A[:, live] + u * np.abs(ref) + tiny
    assert np.isfinite(got).all()
    assert (np.abs(got - ref) <= tol).all(), float(np.max(np.abs(got - ref) - tol))
    gl, rl = to64(lse)[:, live], L[:, live]
    empty = np.isneginf(rl)
    assert np.array_equal(np.isneginf(gl), empty)
    assert (np.abs(gl[~empty] - rl[~empty]) <= e + 2.0 ** -23 * np.abs(rl[~empty])).all()


DECODE = [(1, 1), (1, 15), (1, 16), (1, 17), (0, 40), (1, 64), (1, 65), (1, 300), (1, 129)]
DRAFTS = [(3, 3), (1, 200), (0, 9), (2, 2), (3, 131), (2, 64)]
CHUNKS = [(17, 17), (1, 90), (128, 128), (129, 300), (0, 5), (5, 400), (63, 64), (200, 777)]


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("fp16", 64), ("bf16", 96)])
@pytest.mark.parametrize("lens,Hq,Hkv,page", [
    (DECODE, 4, 1, 16), (DECODE, 2, 2, 64), (DRAFTS, 10, 2, 32), (DRAFTS, 3, 1, 256),
    ([(1, 5)], 1, 1, 16), ([(1, 2000)], 16, 1, 128)])
def test_few_rows(attn_lib, causal, dtype, d, lens, Hq, Hkv, page):
    x = make(lens, Hq, Hkv, d, page, dtype, seed=d + page, pad=2)
    o, lse = run(attn_lib, x, causal)
    assert attn_lib.poll_status() == (0, 0)
    check(x, o, lse, causal)


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("fp16", 64), ("bf16", 96)])
@pytest.mark.parametrize("copies,Hq,Hkv", [(1, 16, 4), (4, 8, 2), (8, 4, 2), (16, 2, 2), (30, 1, 1)])
def test_clusters_of_every_size(attn_lib, dtype, d, copies, Hq, Hkv):
    """Small batches with 8, 4, 2 and 1 CTAs an item, and one past them."""
    x = make(DECODE * copies, Hq, Hkv, d, 32, dtype, seed=copies, pad=1)
    assert workspace_bytes(attn_lib, x) == 0
    o, lse = run(attn_lib, x, True)
    assert attn_lib.poll_status() == (0, 0)
    check(x, o, lse, True)


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("fp16", 64), ("bf16", 96)])
@pytest.mark.parametrize("lens,Hq,Hkv,page", [
    (DECODE * 5, 4, 1, 16), (DECODE * 3, 8, 4, 64), (DRAFTS * 4, 10, 2, 32), ([(1, 5000)], 16, 1, 256),
    ([(2, 4700), (1, 4097)], 4, 2, 16), ([(1, 1)] * 400, 1, 1, 16), ([(1, 64)] * 37, 2, 1, 64),
    ([(16, 900)] * 38, 1, 1, 32)])
def test_few_rows_in_equal_shares(attn_lib, causal, dtype, d, lens, Hq, Hkv, page):
    """Batches past the sizes that run in clusters: pieces of items, items of
    one CTA, items spread over many, CTAs without work."""
    x = widen(make(lens, Hq, Hkv, d, page, dtype, seed=d + page + len(lens), pad=1))
    assert workspace_bytes(attn_lib, x) > 0
    o, lse = run(attn_lib, x, causal)
    assert attn_lib.poll_status() == (0, 0)
    check(x, o, lse, causal)


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("fp16", 64), ("bf16", 96)])
@pytest.mark.parametrize("lens,Hq,Hkv,page", [
    (CHUNKS, 4, 2, 16), (CHUNKS, 2, 2, 64), (CHUNKS, 3, 1, 32), (CHUNKS, 7, 1, 128),
    ([(33, 1000)], 8, 1, 256), ([(1, 100), (1, 900)], 34, 1, 64), ([(9, 50), (2, 600)], 128, 1, 16),
    ([(700, 700)], 1, 1, 64), ([(257, 1500)], 2, 1, 16), ([(18, 20)] * 40, 1, 1, 16)])
def test_chunks(attn_lib, causal, dtype, d, lens, Hq, Hkv, page):
    x = make(lens, Hq, Hkv, d, page, dtype, seed=d + page + len(lens), pad=3)
    o, lse = run(attn_lib, x, causal)
    assert attn_lib.poll_status() == (0, 0)
    check(x, o, lse, causal)


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("lens,Hq,Hkv", [([(4, 0), (3, 2), (1, 7)], 4, 2),
                                         ([(150, 40), (30, 0), (200, 199)], 4, 2)])
def test_rows_without_a_key(attn_lib, causal, lens, Hq, Hkv):
    """Fewer keys than new tokens: causal rows before the first key, and all
    rows of a sequence with an empty cache, give O = 0, LSE = -inf."""
    x = make(lens, Hq, Hkv, 64, 16, "bf16", seed=5)
    o, lse = run(attn_lib, x, causal)
    assert attn_lib.poll_status() == (0, 0)
    check(x, o, lse, causal)


@pytest.mark.parametrize("max_q,n_seq,reach", [(1, 2, 16), (1, 50, 5000), (30, 2, 16)])
def test_no_new_tokens_at_all(attn_lib, max_q, n_seq, reach):
    x = widen(make([(0, 5), (0, 0)] * (n_seq // 2), 4, 2, 64, 16, "bf16", seed=6, pad=30), reach)
    o = torch.full_like(x["q"], 5.0)
    lse = torch.full(x["q"].shape[:2], 5.0, device="cuda")
    run(attn_lib, dict(x, max_q=max_q), True, out=o, lse=lse)
    assert attn_lib.poll_status() == (0, 0)
    assert (o == 5.0).all() and (lse == 5.0).all()


@pytest.mark.parametrize("lens,reach", [(DECODE, 16), (DECODE * 5, 5000), (CHUNKS, 16)])
def test_padding_rows_are_left_alone_and_runs_repeat(attn_lib, lens, reach):
    x = widen(make(lens, 4, 2, 128, 16, "bf16", seed=8, pad=5), reach)
    live = int(x["cu"][-1])
    outs = []
    ws = torch.full((max(workspace_bytes(attn_lib, x), 256),), 0xFF,
                    dtype=torch.uint8, device="cuda")
    for fill in (3.0, -2.0):
        o = torch.full_like(x["q"], fill)
        lse = torch.full(x["q"].shape[:2], fill, device="cuda")
        run(attn_lib, x, True, out=o, lse=lse, workspace=ws)
        assert (o[:, live:] == fill).all() and (lse[:, live:] == fill).all()
        outs.append((o[:, :live].clone(), lse[:, :live].clone()))
    assert attn_lib.poll_status() == (0, 0)
    assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1])


@pytest.mark.parametrize("lens", [[(1, 700), (1, 64)], [(1, 700), (1, 64)] * 12,
                                  [(40, 700), (1, 64)]])
@pytest.mark.parametrize("amp,scale", [(30.0, None), (1.0, 1e-4)])
@pytest.mark.parametrize("reach", [16, 5000])
def test_large_and_small_logits(attn_lib, lens, amp, scale, reach):
    x = widen(make(lens, 4, 2, 128, 32, "fp16", seed=11, amp=amp), reach)
    o, lse = run(attn_lib, x, True, scale=scale)
    assert attn_lib.poll_status() == (0, 0)
    check(x, o, lse, True, scale)


@pytest.mark.parametrize("lens", [[(1, 50), (1, 40), (1, 30)], [(1, 50), (1, 40), (1, 30)] * 8,
                                  [(50, 50), (1, 40), (20, 30)]])
@pytest.mark.parametrize("reach", [16, 5000])
def test_bad_pages_lengths_and_offsets_are_reported(attn_lib, lens, reach):
    """Out-of-range page numbers, lengths past the table and offsets past the
    tensors: the call reports them and the other sequences keep their values."""
    x = widen(make(lens, 4, 2, 64, 16, "bf16", seed=13), reach)
    good, _ = run(attn_lib, x, True)
    assert attn_lib.poll_status() == (0, 0)
    cu = x["cu"].tolist()
    cases = []
    for page in (-1, 1 << 30, x["k"].shape[0]):
        t = x["table"].clone()
        t[1, 1] = page
        cases.append(dict(x, table=t))
    kv = x["kv"].clone()
    kv[1] = x["table"].shape[1] * 16 + 1
    cases.append(dict(x, kv=kv))
    kv = x["kv"].clone()
    kv[1] = -3
    cases.append(dict(x, kv=kv))
    for i, c in enumerate(cases):
        o, _ = run(attn_lib, c, True)
        st, detail = attn_lib.poll_status()
        assert st == 1 and detail >> 16 == 1, (i, st, hex(detail))
        for b in [j for j in range(len(lens)) if j != 1]:
            assert torch.isfinite(o[:, cu[b]:cu[b + 1]]).all()
            err = (o - good)[:, cu[b]:cu[b + 1]].float().abs().max()
            assert err <= 2 ** -5 * good.float().abs().max(), (i, b)
    for bad in (cu[:2] + [cu[1] - 1] + cu[3:], cu[:-1] + [cu[-1] + 9], [1] + cu[1:]):
        run(attn_lib, dict(x, cu=cuda_i32(bad)), True)
        assert attn_lib.poll_status()[0] == 1
    o, _ = run(attn_lib, x, True)
    assert attn_lib.poll_status() == (0, 0) and torch.equal(o, good)


def test_many_sequences(attn_lib):
    """More sequences than the CTA has threads, most of them without tokens."""
    g = np.random.default_rng(3)
    lens = [(int(g.integers(0, 2)), int(g.integers(1, 40))) for _ in range(1500)]
    x = make(lens, 2, 1, 64, 16, "fp16", seed=17)
    o, lse = run(attn_lib, x, True)
    assert attn_lib.poll_status() == (0, 0)
    check(x, o, lse, True)


@pytest.mark.parametrize("chunk", [1, 50])
def test_captured_call_replays_with_new_lengths(attn_lib, chunk):
    """A graph of append + attention replays on new lengths, pages and tokens
    written into the same tensors, on a side stream."""
    Hq, Hkv, d, page, dt = 4, 2, 64, 16, torch.bfloat16
    table = attn_lib.rope_table(d)
    x = make([(chunk, chunk + 30), (1, 9)], Hq, Hkv, d, page, "bf16", seed=19)
    y = make([(1, chunk + 29), (chunk, 2 * chunk + 3)], Hq, Hkv, d, page, "bf16", seed=23)
    n = max(x["k"].shape[0], y["k"].shape[0])
    wide = max(x["table"].shape[1], y["table"].shape[1])
    pad = lambda t, size: torch.cat([t, t.new_zeros(size - t.shape[0], *t.shape[1:])])  # noqa: E731
    for s in (x, y):
        s["k"], s["v"] = pad(s["k"], n), pad(s["v"], n)
        s["table"] = torch.cat([s["table"], s["table"].new_zeros(2, wide - s["table"].shape[1])], 1)
        s["new"] = torch.randn(2, Hkv, s["q"].shape[1], d, device="cuda").to(dt)
    hold = {k: v.clone() if torch.is_tensor(v) else v for k, v in x.items()}
    ws = torch.empty(attn_lib.fwd_paged_workspace_bytes(2, chunk, 4096, Hq, Hkv, d), dtype=torch.uint8,
                     device="cuda")

    def step(s):
        q = attn_lib.append_kv(s["new"][0], s["new"][1], s["k"], s["v"], s["table"], s["cu"],
                               s["kv"], table=table, q=s["q"])
        return attn_lib.fwd_paged(q, s["k"], s["v"], s["table"], s["cu"], s["kv"], chunk,
                                  causal=True, workspace=ws)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(hold)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        o, lse = step(hold)
    for s in (x, y, x):
        for key in ("q", "k", "v", "table", "cu", "kv", "new"):
            hold[key].copy_(s[key])
        graph.replay()
        got = o.clone(), lse.clone()
        want = step({k: v.clone() if torch.is_tensor(v) else v for k, v in s.items()})
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert attn_lib.poll_status() == (0, 0)


@pytest.mark.parametrize("axes", [1, 3])
def test_serving_run(attn_lib, axes):
    """As a server uses them together: two prompts in chunks, then single
    tokens, each step appending turned keys and attending over the cache; every
    output row is the full causal attention of its sequence."""
    Hq, Hkv, d, page, dt = 6, 2, 64, 16, torch.bfloat16
    steps = [(70, 20), (50, 0), (1, 33), (1, 1), (1, 1), (4, 1)]  # new tokens of the two sequences
    half = d // 2
    axis = (np.arange(half) * axes // half)
    inv = 10000.0 ** (-np.arange(half) / half)
    rope = attn_lib.rope_table(d, axes=axis.tolist())
    table = np.random.default_rng(0).permutation(24).reshape(2, 12)
    kp = torch.full((24, Hkv, page, d), float("nan"), dtype=dt, device="cuda")
    vp = torch.full_like(kp, float("nan"))
    full = [np.zeros((n, 0, d)) for n in (Hkv, Hkv) * 2]  # k0, v0, k1, v1 as cached
    kv = [0, 0]
    g = torch.Generator().manual_seed(29)
    for new in steps:
        total = sum(new)
        q, k, v = (torch.randn((h, total, d), generator=g).to(dt).cuda() for h in (Hq, Hkv, Hkv))
        kv = [a + n for a, n in zip(kv, new)]
        pos = torch.randint(0, 4000, (axes, total), generator=g).to(torch.int32).cuda()
        cu = cuda_i32([0, new[0], total])
        q2 = attn_lib.append_kv(k, v, kp, vp, cuda_i32(table), cu, cuda_i32(kv), table=rope,
                                positions=pos, q=q)
        ref_q, ref_k = attn_lib.rope(q, k, pos, rope)
        assert torch.equal(q2, ref_q)
        o, lse = attn_lib.fwd_paged(q2, kp, vp, cuda_i32(table), cu, cuda_i32(kv), max(new),
                                    causal=True)
        assert attn_lib.poll_status() == (0, 0)
        turned = oracle.rotary(to64(q), pos.cpu().numpy(), inv, axis, False)
        assert np.max(np.abs(to64(q2) - turned)) <= 2 ** -8 * np.abs(turned).max() + 1e-5
        for b in range(2):
            rows = slice(0, new[0]) if b == 0 else slice(new[0], total)
            full[2 * b] = np.concatenate([full[2 * b], to64(ref_k)[:, rows]], 1)
            full[2 * b + 1] = np.concatenate([full[2 * b + 1], to64(v)[:, rows]], 1)
            assert np.array_equal(
                oracle.paged_rows(to64(kp), table[b], kv[b]), full[2 * b])
        x = dict(q=q2, k=kp, v=vp, table=cuda_i32(table), cu=cu, kv=cuda_i32(kv))
        check(x, o, lse, True)


def test_max_q_below_a_length_is_reported(attn_lib):
    for lens, max_q in (([(1, 9), (3, 50), (2, 60)], 2), ([(40, 90), (60, 60), (3, 5)], 50)):
        x = make(lens, 4, 2, 64, 16, "bf16", seed=14)
        good, _ = run(attn_lib, x, True)
        assert attn_lib.poll_status() == (0, 0)
        o = torch.full_like(good, 9.0)
        run(attn_lib, dict(x, max_q=max_q), True, out=o)
        st, detail = attn_lib.poll_status()
        assert st == 1 and detail >> 16 == 1
        cu = x["cu"].tolist()
        assert (o[:, cu[1] + max_q:cu[2]] == 9.0).all()
        for b in (0, 2):
            err = (o - good)[:, cu[b]:cu[b + 1]].float().abs().max()
            assert err <= 2 ** -5 * good.float().abs().max()


@pytest.mark.parametrize("chunk", [1, 3, 40])
def test_pages_past_two_to_the_31_elements(attn_lib, chunk):
    """A cache of 2.4e9 elements: pages at both ends, two sequences that share
    their first pages; the append writes there and the attention reads it."""
    Hq, Hkv, d, page, dt = 4, 2, 128, 64, torch.float16
    n_pages = 147_000
    kp = torch.empty(n_pages, Hkv, page, d, dtype=dt, device="cuda")
    vp = torch.empty_like(kp)
    assert kp.numel() > 2 ** 31
    table = cuda_i32([[n_pages - 1, 3, n_pages - 2], [n_pages - 1, 3, n_pages - 7]])
    kv = [150 + chunk, 170]
    g = torch.Generator("cuda").manual_seed(41)
    for t in (kp, vp):
        for i in set(table.flatten().tolist()):
            t[i].normal_(generator=g)
    n = chunk + 1
    q, k, v = (torch.randn(h, n, d, generator=g, device="cuda").to(dt) for h in (Hq, Hkv, Hkv))
    cu = cuda_i32([0, chunk, n])
    small = lambda t: t[table.flatten().long()].clone()  # noqa: E731
    kref, vref = small(kp), small(vp)
    tref = np.arange(6).reshape(2, 3)
    attn_lib.append_kv(k, v, kp, vp, table, cu, cuda_i32(kv))
    kref = oracle.append_paged(to64(k), to64(kref), tref, cu.tolist(), kv)
    vref = oracle.append_paged(to64(v), to64(vref), tref, cu.tolist(), kv)
    o, lse = attn_lib.fwd_paged(q, kp, vp, table, cu, cuda_i32(kv), chunk, causal=True)
    assert attn_lib.poll_status() == (0, 0)
    assert np.array_equal(to64(small(kp)), kref) and np.array_equal(to64(small(vp)), vref)
    y = dict(q=q, k=torch.tensor(kref), v=torch.tensor(vref), table=torch.tensor(tref), cu=cu,
             kv=cuda_i32(kv))
    check(y, o, lse, True)


def test_two_graphs_share_a_workspace(attn_lib):
    """Captured calls of different shapes (decoding, chunks) over one workspace,
    replayed in turn, give what they give with workspaces of their own."""
    xs = [widen(make(DECODE * 5, 4, 2, 64, 16, "bf16", seed=43)), make(CHUNKS, 4, 2, 64, 16, "bf16", seed=47),
          make([(1, 6000), (2, 900)], 8, 1, 64, 16, "bf16", seed=53)]
    ws = torch.empty(max(workspace_bytes(attn_lib, x) for x in xs), dtype=torch.uint8, device="cuda")
    want = [run(attn_lib, x, True) for x in xs]
    side = torch.cuda.Stream()
    graphs, outs = [], []
    for x in xs:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1], stream=side):
            outs.append(run(attn_lib, x, True, workspace=ws))
    for i in (0, 1, 2, 1, 0, 2, 2, 0):
        outs[i][0].fill_(7.0)
        graphs[i].replay()
        assert torch.equal(outs[i][0], want[i][0]) and torch.equal(outs[i][1], want[i][1])
    assert attn_lib.poll_status() == (0, 0)


def test_calls_on_two_streams(attn_lib):
    """Calls that overlap on two streams, each with its own workspace."""
    xs = [widen(make(DECODE * 20, 4, 2, 128, 16, "bf16", seed=59)),
          make([(200, 900), (128, 2000)], 4, 2, 128, 16, "bf16", seed=61)]
    want = [run(attn_lib, x, True) for x in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in xs]
    got = [[], []]
    for _ in range(10):
        for x, st, g in zip(xs, streams, got):
            with torch.cuda.stream(st):
                g.append(run(attn_lib, x, True))
    torch.cuda.synchronize()
    assert attn_lib.poll_status() == (0, 0)
    for g, w in zip(got, want):
        assert all(torch.equal(o, w[0]) and torch.equal(l, w[1]) for o, l in g)


@pytest.mark.parametrize("lens,reach", [([(1, 60), (1, 300)], 16), ([(1, 60), (1, 300)] * 6, 5000),
                                        ([(40, 60), (1, 300)], 16)])
def test_inputs_written_just_before_the_call(attn_lib, lens, reach):
    """The kernels may start before the work ahead of them in the stream has
    finished; what that work writes (copies from the host, a kernel's output)
    is what they read, and what they overwrite has been read."""
    Hq, Hkv, d, page = 4, 2, 64, 16
    xs = [widen(make(lens, Hq, Hkv, d, page, "bf16", seed=s), reach) for s in (73, 79)]
    table = attn_lib.rope_table(d)
    hold = {k: v.clone() if torch.is_tensor(v) else v for k, v in xs[0].items()}
    pinned = [{k: x[k].cpu().pin_memory() for k in ("cu", "kv", "table")} for x in xs]
    new = [torch.randn(2, Hkv, x["q"].shape[1], d, device="cuda").bfloat16() for x in xs]
    big = torch.randn(64 << 20, device="cuda")

    def step(x, q, kv):
        q = attn_lib.append_kv(kv[0], kv[1], x["k"], x["v"], x["table"], x["cu"], x["kv"],
                               table=table, q=q)
        return attn_lib.fwd_paged(q, x["k"], x["v"], x["table"], x["cu"], x["kv"], x["max_q"],
                                  causal=True)

    want = [step({k: v.clone() if torch.is_tensor(v) else v for k, v in x.items()}, x["q"], n)
            for x, n in zip(xs, new)]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = []
    with torch.cuda.stream(side):
        for i in (0, 1) * 8:
            big.mul_(1.0)  # keeps the stream busy
            for key in ("cu", "kv", "table"):
                hold[key].copy_(pinned[i][key], non_blocking=True)
            hold["k"].copy_(xs[i]["k"])
            hold["v"].copy_(xs[i]["v"])
            q = xs[i]["q"] * 2.0 * 0.5  # a kernel's output
            o, lse = step(hold, q, new[i])
            got.append((i, o * 1.0, lse * 1.0))
            o.fill_(float("nan"))  # the memory goes back for the next step's outputs
            del o, lse, q
    torch.cuda.synchronize()
    assert attn_lib.poll_status() == (0, 0)
    for i, o, lse in got:
        assert torch.equal(o, want[i][0]) and torch.equal(lse, want[i][1])


def test_timeouts_wind_down(attn_lib):
    """Waits that run out report ATTN_ERR_TIMEOUT and the next call is right."""
    x = make([(1, 3000)] * 40, 16, 8, 128, 64, "bf16", seed=31)
    y = make([(300, 3000)] * 3, 16, 8, 128, 64, "bf16", seed=37)
    z = make([(1, 3000)] * 4, 16, 8, 128, 64, "bf16", seed=67)
    assert workspace_bytes(attn_lib, x) > 0 and workspace_bytes(attn_lib, z) == 0
    for s in (x, y, z):
        run(attn_lib, s, True)
        assert attn_lib.poll_status() == (0, 0)
        want, _ = run(attn_lib, s, True)
        attn_lib.set_wait_limit_us(1)
        try:
            for _ in range(3):
                run(attn_lib, s, True)
            st, _ = attn_lib.poll_status()
        finally:
            attn_lib.set_wait_limit_us(0)
        assert st in (0, 4)
        got, _ = run(attn_lib, s, True)
        assert attn_lib.poll_status() == (0, 0) and torch.equal(got, want)


def test_binding_refuses_wrong_tensors(attn_lib):
    """What the Python entry checks before the C ABI: types, shapes, devices,
    strides.  Nothing is launched; the same arguments put right then work."""
    x = make([(1, 5), (2, 40)], 4, 2, 64, 16, "bf16", seed=71)
    good = [x["q"], x["k"], x["v"], x["table"], x["cu"], x["kv"], 2]
    half, cpu = x["q"].half(), x["q"].cpu()
    wide = torch.zeros(4, 3, 128, dtype=torch.bfloat16, device="cuda")
    bad = [(0, half, ValueError), (0, x["q"].float(), TypeError), (0, cpu, ValueError),
           (0, wide, ValueError), (0, x["q"][:3], ValueError), (0, x["q"][0], ValueError),
           (0, wide[..., ::2], ValueError), (0, None, TypeError), (0, 3, TypeError),
           (1, x["k"][1:], ValueError), (1, x["k"].transpose(1, 2), ValueError),
           (3, x["table"].long(), ValueError), (3, x["table"][:1], ValueError),
           (3, x["table"].cpu(), ValueError), (4, x["cu"][:2], ValueError),
           (5, x["kv"].long(), ValueError), (5, x["kv"][None], ValueError),
           (6, 0, ValueError), (6, 4, ValueError), (6, 1 << 40, ValueError), (6, "two", ValueError)]
    for i, value, error in bad:
        with pytest.raises(error):
            attn_lib.fwd_paged(*(good[:i] + [value] + good[i + 1:]))
    o, lse = torch.empty_like(x["q"]), torch.empty(4, 3, device="cuda")
    for kw, error in ((dict(out=half), ValueError), (dict(out=o.cpu()), ValueError),
                      (dict(out=wide[..., :64]), ValueError), (dict(lse=lse.half()), ValueError),
                      (dict(lse=lse.t()), ValueError), (dict(workspace=lse), ValueError),
                      (dict(scale="x"), TypeError), (dict(out=1), TypeError)):
        with pytest.raises(error):
            attn_lib.fwd_paged(*good, **kw)
    with pytest.raises(attn_lib.AttnError) as e:
        attn_lib.fwd_paged(*good, scale=-1.0)
    assert e.value.status == 1

    table = attn_lib.rope_table(64)
    k = torch.zeros(2, 3, 64, dtype=torch.bfloat16, device="cuda")
    pos = torch.zeros(1, 3, dtype=torch.int32, device="cuda")
    cache = [x["k"], x["v"], x["table"], x["cu"], x["kv"]]
    for args, kw in (((k, k.half()), {}), ((k[:1], k[:1]), {}), ((k, k[:, :2]), {}),
                     ((k.float(), k.float()), {}), ((wide[:2, :, ::2], k), {}),
                     ((k, k), dict(positions=pos)), ((k, k), dict(table=table.int())),
                     ((k, k), dict(table=table[:1])), ((k, k), dict(table=attn_lib.rope_table(128))),
                     ((k, k), dict(table=table, positions=pos.long())),
                     ((k, k), dict(table=table, positions=pos[:, :2])),
                     ((k, k), dict(q=x["q"][:3])), ((k, k), dict(q=half)), ((k, k), dict(out_q=x["q"])),
                     ((k, k), dict(q=x["q"], out_q=x["q"].transpose(0, 1).contiguous().transpose(0, 1)))):
        with pytest.raises((ValueError, TypeError)):
            attn_lib.append_kv(*args, *cache, **kw)
    q4 = torch.zeros(2, 4, 3, 64, dtype=torch.bfloat16, device="cuda")
    for args, kw in (((q4, q4[:1], pos), {}), ((q4, q4.half(), pos), {}), ((q4[0, 0], None, pos), {}),
                     ((q4, None, pos[:, :2]), {}), ((q4, None, pos[0]), {}),
                     ((q4, None, pos[:, None].expand(1, 3, 3)), {}), ((q4, None, pos.long()), {}),
                     ((q4[..., ::2], None, pos), {}), ((q4[:, :0], None, pos), {}),
                     ((q4, None, pos), dict(out_k=q4)), ((q4, None, pos), dict(out_q=q4[:1])),
                     ((q4, None, pos), dict(out_q=q4[:, :1].expand(2, 4, 3, 64)))):
        with pytest.raises((ValueError, TypeError)):
            attn_lib.rope(*args, table, **kw)
    assert attn_lib.poll_status() == (0, 0)
    attn_lib.fwd_paged(*good)
    attn_lib.append_kv(k, k, *cache, table=table, positions=pos, q=x["q"])
    attn_lib.rope(q4, q4[:, :2], pos, table)
    assert attn_lib.poll_status() == (0, 0)


@pytest.mark.parametrize("seed", range(48))
def test_random_paged_case(attn_lib, seed):
    """Seeded draws of everything at once: head layout, head dim, dtype, page
    size, masking, lengths (empty sequences, fewer keys than tokens), a table
    that reaches further, padding rows, a scale of its own."""
    g = np.random.default_rng(1000 + seed)
    Hkv = int(g.choice([1, 2, 3, 5]))
    G = int(g.choice([1, 2, 3, 4, 7, 8, 16, 40]))
    d, page = int(g.choice([64, 96, 128])), int(g.choice([16, 32, 64, 128, 256]))
    n = int(g.choice([1, 2, 5, 30, 140]))
    kind = g.choice(["single", "few", "chunks"])
    lens = []
    for _ in range(n):
        new = {"single": 1, "few": int(g.integers(0, 4)),
               "chunks": int(g.integers(0, 300 if n < 10 else 12))}[kind]
        if g.random() < 0.1:
            new = 0
        lens.append((new, int(g.integers(0, 900 if n < 50 else 90))))
    if all(m == 0 for m, _ in lens):
        lens[0] = (1, lens[0][1])
    x = make(lens, Hkv * G, Hkv, d, page, str(g.choice(["bf16", "fp16"])), seed=seed,
             pad=int(g.integers(0, 4)))
    if g.random() < 0.5:
        x = widen(x)
    causal, scale = bool(g.random() < 0.7), float(g.choice([d ** -0.5, 0.02, 0.3]))
    o, lse = run(attn_lib, x, causal, scale=scale)
    assert attn_lib.poll_status() == (0, 0)
    check(x, o, lse, causal, scale)


# (batch, reach of the table): decoding in clusters; in equal shares, items whole
# and split; one item over many CTAs; chunks whole and in 2 to 7 parts; chunks
# in more than 8 and more than 16 parts
NAN_BATCHES = [(DECODE, 16, 4, 1), (DECODE * 5, 5000, 4, 1), ([(1, 5000), (4, 70)], 16, 4, 1),
               ([(16, 900)] * 38, 5000, 1, 1), (CHUNKS, 16, 4, 2), ([(700, 3000), (1, 50)], 16, 2, 1),
               ([(20, 3500)], 16, 2, 1), ([(40, 16000)], 16, 2, 1)]


def _live_rows(lens, causal):
    """Packed rows that see a key, by sequence."""
    at, rows = 0, []
    for n, k in lens:
        rows.append([at + i for i in range(n) if (i + k - n >= 0 if causal else k > 0)])
        at += n
    return rows


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("fp16", 64), ("bf16", 96)])
@pytest.mark.parametrize("lens,reach,Hq,Hkv", NAN_BATCHES)
def test_nan_and_infinite_queries_give_nan(attn_lib, causal, dtype, d, lens, reach, Hq, Hkv):
    """A query with a NaN or an infinity has a NaN score at every key it sees
    (inf x +-k sums to NaN): its row is NaN in O and LSE however the batch is
    cut, and every other row keeps its bits."""
    x = widen(make(lens, Hq, Hkv, d, 16, dtype, seed=83, pad=2), reach)
    clean_o, clean_lse = run(attn_lib, x, causal)
    check(x, clean_o, clean_lse, causal)
    rows = [r[len(r) // 2] for r in _live_rows(lens, causal) if r]
    hit = torch.zeros(x["q"].shape[:2], dtype=torch.bool, device="cuda")
    q = x["q"].clone()
    for i, r in enumerate(rows):
        h = i % Hq
        hit[h, r] = True
        if i % 2:
            q[h, r] = float("nan")
        else:  # both infinities: some product of each sign, inf - inf
            q[h, r, 0], q[h, r, 1] = float("inf"), float("inf")
            q[h, r, 2:] = float("-inf")
    o, lse = run(attn_lib, dict(x, q=q), causal)
    assert attn_lib.poll_status() == (0, 0)
    live = int(x["cu"][-1])
    assert torch.isnan(o[hit]).all() and torch.isnan(lse[hit]).all()
    keep = ~hit[:, :live]
    assert torch.equal(o[:, :live][keep], clean_o[:, :live][keep])
    assert torch.equal(lse[:, :live][keep], clean_lse[:, :live][keep])


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("fp16", 64), ("bf16", 96)])
@pytest.mark.parametrize("lens,reach,Hq,Hkv", NAN_BATCHES)
def test_nan_key_reaches_the_rows_that_see_it(attn_lib, dtype, d, lens, reach, Hq, Hkv):
    """A NaN in the last key of each sequence: its last row (causal) is NaN,
    every row before keeps its bits."""
    x = widen(make(lens, Hq, Hkv, d, 16, dtype, seed=89), reach)
    clean_o, clean_lse = run(attn_lib, x, True)
    k, table = x["k"].clone(), x["table"].tolist()
    hit = torch.zeros(x["q"].shape[1], dtype=torch.bool, device="cuda")
    at = 0
    for b, (n, keys) in enumerate(lens):
        if n and keys:
            k[table[b][(keys - 1) // 16], :, (keys - 1) % 16, 5] = float("nan")
            hit[at + n - 1] = True
        at += n
    o, lse = run(attn_lib, dict(x, k=k), True)
    assert attn_lib.poll_status() == (0, 0)
    assert torch.isnan(o[:, hit]).all() and torch.isnan(lse[:, hit]).all()
    assert torch.equal(o[:, ~hit], clean_o[:, ~hit]) and torch.equal(lse[:, ~hit], clean_lse[:, ~hit])


def parts_of(attn, x, causal):
    """O, LSE and the numbers of parts of the items that the call split, read
    from the descriptions at the head of its workspace (per CTA and slot: parts
    in all, 0 where the slot is empty)."""
    ws = torch.zeros(workspace_bytes(attn, x), dtype=torch.uint8, device="cuda")
    o, lse = run(attn, x, causal, workspace=ws)
    few = x["max_q"] * (x["q"].shape[0] // x["k"].shape[1]) <= 16
    ctas = 2 * 160 if few else 160
    desc = ws[:ctas * 64].view(torch.int32).view(ctas, 2, 2, 4)
    return o, lse, set(desc[:, :, 0, 0].flatten().tolist()) - {0}


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("fp16", 64), ("bf16", 96)])
@pytest.mark.parametrize("lens,Hq,Hkv,parts", [
    ([(17, 600)], 1, 1, (2, 4)), ([(33, 2000)], 2, 1, (5, 8)), ([(200, 1900)], 1, 1, (5, 8)),
    ([(20, 3500)], 2, 1, (9, 16)), ([(64, 3900)], 7, 1, (9, 16)), ([(130, 3000), (1, 40)], 2, 2, (9, 16)),
    ([(40, 16000)], 2, 1, (17, 160)), ([(250, 9000)], 1, 1, (17, 160)),
    ([(64, 12000), (5, 9000), (0, 3)], 4, 2, (17, 160)), ([(300, 130)] * 9, 1, 1, None)])
def test_chunks_in_many_parts(attn_lib, causal, dtype, d, lens, Hq, Hkv, parts):
    """The join of tiles at every number of parts it has a form for, the last
    parts seen by none of a causal item's first rows."""
    x = make(lens, Hq, Hkv, d, 32, dtype, seed=101 + d, pad=2)
    o, lse, got = parts_of(attn_lib, x, causal)
    assert attn_lib.poll_status() == (0, 0)
    if parts is not None:
        assert any(parts[0] <= n <= parts[1] for n in got), got
    check(x, o, lse, causal)


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("fp16", 64), ("bf16", 96)])
@pytest.mark.parametrize("lens,Hq,Hkv,parts", [
    ([(1, 4600)] * 38, 4, 4, (2, 4)), ([(2, 4500)] * 10, 8, 4, (5, 16)),
    ([(1, 9000), (1, 70)], 8, 1, (17, 320))])
def test_few_rows_in_many_parts(attn_lib, dtype, d, lens, Hq, Hkv, parts):
    """The join of decoding items at every number of parts it has a form for."""
    x = widen(make(lens, Hq, Hkv, d, 64, dtype, seed=103 + d, pad=1))
    o, lse, got = parts_of(attn_lib, x, True)
    assert attn_lib.poll_status() == (0, 0)
    assert any(parts[0] <= n <= parts[1] for n in got), got
    check(x, o, lse, True)
