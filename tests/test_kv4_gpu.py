"""The paged cache in 4 bits: append, reading back, and attention over it, CUDA
path vs the fp64 oracle.

Attention: the cases are those of the 16-bit cache (test_paged_gpu.py), keys and
values the exact m + c s.  With u = finfo.eps / 2, a value is rounded to u (|v|), or c s
is, to u (c s): together with P's rounding at most u of A = sum P (|v| + max(|v|, c s)).
A score's error d_j:
* few rows: a group's product with c sums 32 exact products, and s and m are applied
  in fp32: at most 48 2^-24 M with M = scale max sum |q| (|m| + 15 s);
* chunks: 2 d exact products and 12 more are summed in fp32, and of m + 8 s and the
  sum of q two terms of 11 bits are taken each: (2 d + 16) 2^-24 M + 2^-20 M with
  M = scale max sum |q| (|m + 8 s| + 8 s).
With e = 2^-20 + n 2^-24 + d_j for the exponential and the sums as there,
|LSE - LSE_ref| <= e + 2^-23 |LSE| and, P_ij being off by d_j and by the row's
l, |O - O_ref| <= (u + 2 e) (1 + u) A + u |O|.  P may exceed 1 by 2^8, which scales its
rounding and l alike.

Append: the scale and the minimum have to be those of the definition, and a code
c lies within 1/2 + 2^-19 of (x - m) / s, the difference and the quotient (at
most 15.1) being rounded once each in fp32 (2^-24 of their size).
"""
import numpy as np
import pytest
import torch

import oracle
import test_paged_gpu as paged
from helpers import to64
from test_paged_gpu import CHUNKS, DECODE, DRAFTS, DT, cuda_i32, widen

pytestmark = pytest.mark.gpu


def pack4(x):
    """Rows of the 4-bit cache for 16-bit values x [..., d]; rows with a NaN
    become poison (all bits set: NaN scales and minima)."""
    g = x.float().unflatten(-1, (-1, 32))
    low = g.amin(-1, keepdim=True)
    scale = ((g.amax(-1, keepdim=True) - low) / 15).to(x.dtype)
    code = ((g - low) / torch.where(scale > 0, scale.float(), float("inf"))).round().clamp(0, 15)
    code = code.nan_to_num(0.0).to(torch.uint8).flatten(-2)
    par = torch.cat([scale, low.to(x.dtype)], -1).flatten(-2).contiguous().view(torch.uint8)
    rows = torch.cat([code[..., ::2] | code[..., 1::2] << 4, par], -1)
    return rows.masked_fill(torch.isnan(x).any(-1, keepdim=True), 0xFF).contiguous()


def parts4(rows, dtype):
    """s, m and codes by channel, in 64 bits."""
    d = rows.shape[-1] // 5 * 8
    par = rows[..., d // 2:].contiguous().view(dtype).double().unflatten(-1, (-1, 2))
    code = torch.stack([rows[..., :d // 2] & 15, rows[..., :d // 2] >> 4], -1).flatten(-2)
    return par[..., 0].repeat_interleave(32, -1), par[..., 1].repeat_interleave(32, -1), code.double()


def exact4(rows, dtype):
    """What rows stand for (exact in 64 bits but for far exponents, which these
    tests do not have)."""
    s, m, c = parts4(rows, dtype)
    return m + c * s


def unpack4(rows, dtype):
    return exact4(rows, dtype).to(dtype)


def largest(x, causal, scale, weight):
    """scale max sum |q| weight over the rows and keys of every sequence; weight
    like the pages."""
    q, w = np.abs(to64(x["q"])), weight.cpu().numpy()
    cu, kv, table = x["cu"].tolist(), x["kv"].tolist(), x["table"].cpu().numpy()
    group, top = q.shape[0] // w.shape[1], 0.0
    for b, n in enumerate(kv):
        rows = q[:, cu[b]:cu[b + 1]]
        if n == 0 or rows.shape[1] == 0:
            continue
        k = oracle.paged_rows(w, table[b], n)
        for h in range(w.shape[1]):
            r = rows[h * group:(h + 1) * group].reshape(-1, q.shape[2])
            got = (r[np.isfinite(r).all(1)] @ k[h].T) * scale
            top = max(top, float(got.max(initial=0.0)))
    return top


def check4(x, o, lse, causal, scale=None):
    dt, d = x["q"].dtype, x["q"].shape[2]
    scale = d ** -0.5 if scale is None else scale
    cu, kv = x["cu"].cpu().numpy(), x["kv"].cpu().numpy()
    k, v = exact4(x["k4"], dt), exact4(x["v4"], dt)
    args = x["table"].cpu().numpy(), cu, kv, causal, scale
    O, L, _, _ = oracle.attention_paged(to64(x["q"]), k.cpu().numpy(), to64(v), *args)
    s, m, c = parts4(x["v4"], dt)
    A = oracle.attention_paged(to64(x["q"]), k.cpu().numpy(), to64(v.abs() + torch.maximum(v.abs(), c * s)),
                               *args)[0]
    s, m, _ = parts4(x["k4"], dt)
    few = x["max_q"] * (x["q"].shape[0] // k.shape[1]) <= 16
    err = (48 * 2.0 ** -24 if few else (2 * d + 16) * 2.0 ** -24 + 2.0 ** -20) * \
        largest(x, causal, scale, m.abs() + 15 * s if few else (m + 8 * s).abs() + 8 * s)
    live = slice(0, int(cu[-1]))
    u = torch.finfo(dt).eps / 2
    e = 2.0 ** -20 + int(kv.max()) * 2.0 ** -24 + err
    got, ref = to64(o)[:, live], O[:, live]
    tol = (u + 2 * e) * (1 + u) * A[:, live] + u * np.abs(ref) + torch.finfo(dt).smallest_normal * u
    assert np.isfinite(got).all()
    assert (np.abs(got - ref) <= tol).all(), float(np.max(np.abs(got - ref) - tol))
    gl, rl = to64(lse)[:, live], L[:, live]
    empty = np.isneginf(rl)
    assert np.array_equal(np.isneginf(gl), empty)
    assert (np.abs(gl[~empty] - rl[~empty]) <= e + 2.0 ** -23 * np.abs(rl[~empty])).all()


@pytest.fixture
def four(monkeypatch, attn_lib):
    """The 16-bit cache's tests over a 4-bit one: batches get packed pages."""
    make = paged.make

    def make4(*a, **kw):
        x = make(*a, **kw)
        return dict(x, k4=pack4(x["k"]), v4=pack4(x["v"]))

    def run4(attn, x, causal, **kw):
        return attn.fwd_paged4(x["q"], x["k4"], x["v4"], x["table"], x["cu"], x["kv"], x["max_q"],
                               causal=causal, **kw)

    monkeypatch.setattr(paged, "make", make4)
    monkeypatch.setattr(paged, "run", run4)
    monkeypatch.setattr(paged, "check", check4)
    return attn_lib


def again(name):
    """A test of the 16-bit cache, run over the 4-bit one."""
    f = getattr(paged, name)
    names = [n for n in f.__code__.co_varnames[:f.__code__.co_argcount] if n != "attn_lib"]
    src = f"def test(four{''.join(', ' + n for n in names)}):\n    f(four{''.join(', ' + n for n in names)})"
    scope = {"f": f}
    exec(src, scope)
    for mark in getattr(f, "pytestmark", []):
        if mark.name == "parametrize":
            scope["test"] = pytest.mark.parametrize(*mark.args, **mark.kwargs)(scope["test"])
    scope["test"].__doc__ = f.__doc__
    return scope["test"]


test_few_rows = again("test_few_rows")
test_clusters_of_every_size = again("test_clusters_of_every_size")
test_few_rows_in_equal_shares = again("test_few_rows_in_equal_shares")
test_chunks = again("test_chunks")
test_rows_without_a_key = again("test_rows_without_a_key")
test_no_new_tokens_at_all = again("test_no_new_tokens_at_all")
test_padding_rows_are_left_alone_and_runs_repeat = again(
    "test_padding_rows_are_left_alone_and_runs_repeat")
test_large_and_small_logits = again("test_large_and_small_logits")
test_bad_pages_lengths_and_offsets_are_reported = again(
    "test_bad_pages_lengths_and_offsets_are_reported")
test_many_sequences = again("test_many_sequences")
test_max_q_below_a_length_is_reported = again("test_max_q_below_a_length_is_reported")
test_two_graphs_share_a_workspace = again("test_two_graphs_share_a_workspace")
test_calls_on_two_streams = again("test_calls_on_two_streams")
test_random_paged_case = again("test_random_paged_case")
test_nan_and_infinite_queries_give_nan = again("test_nan_and_infinite_queries_give_nan")
test_chunks_in_many_parts = again("test_chunks_in_many_parts")
test_few_rows_in_many_parts = again("test_few_rows_in_many_parts")
test_timeouts_wind_down = again("test_timeouts_wind_down")


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("fp16", 64), ("bf16", 96)])
@pytest.mark.parametrize("lens,reach,Hq,Hkv", paged.NAN_BATCHES)
def test_nan_key_reaches_the_rows_that_see_it(four, dtype, d, lens, reach, Hq, Hkv):
    """A group that stands for NaN in the last key of each sequence: its last row
    (causal) is NaN, every row before keeps its bits."""
    x = widen(paged.make(lens, Hq, Hkv, d, 16, dtype, seed=89), reach)
    clean_o, clean_lse = paged.run(four, x, True)
    k, table = x["k4"].clone(), x["table"].tolist()
    hit = torch.zeros(x["q"].shape[1], dtype=torch.bool, device="cuda")
    at = 0
    for b, (n, keys) in enumerate(lens):
        if n and keys:
            # 0xFFFF is a NaN in both types (0x7F7F in fp16 alone)
            k[table[b][(keys - 1) // 16], :, (keys - 1) % 16, d // 2:d // 2 + 4] = 0xFF
            hit[at + n - 1] = True
        at += n
    o, lse = paged.run(four, dict(x, k4=k), True)
    assert four.poll_status() == (0, 0)
    assert torch.isnan(o[:, hit]).all() and torch.isnan(lse[:, hit]).all()
    assert torch.equal(o[:, ~hit], clean_o[:, ~hit]) and torch.equal(lse[:, ~hit], clean_lse[:, ~hit])


# ------------------------------------------------------------------ append ---

def batch(lens, page, seed, n_extra=2):
    """cu, kv and a table of shuffled pages."""
    g = np.random.default_rng(seed)
    cu = np.concatenate([[0], np.cumsum([n for n, _ in lens])])
    need = [-(-k // page) for _, k in lens]
    order = g.permutation(sum(need) + n_extra)
    table = np.full((len(lens), max(need) + 1), -1)
    at = 0
    for b, m in enumerate(need):
        table[b, :m] = order[at:at + m]
        at += m
    return cu, [k for _, k in lens], table, len(order)


def normal(shape, dt, seed):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(dt).cuda()


def check_codes(rows, x, bf16):
    """rows against 16-bit values x: scale and minimum as defined, nearest codes."""
    rows, x = rows.cpu().numpy(), to64(x)
    d = x.shape[-1]
    want = oracle.quantize4(x, bf16)
    assert np.array_equal(rows[..., d // 2:], want[..., d // 2:])
    par = np.ascontiguousarray(rows[..., d // 2:]).view("<u2")
    code = np.stack([rows[..., :d // 2] & 15, rows[..., :d // 2] >> 4], -1).reshape(x.shape)
    s = np.repeat(oracle.from16(np.ascontiguousarray(par[..., ::2]), bf16), 32, -1)
    m = np.repeat(oracle.from16(np.ascontiguousarray(par[..., 1::2]), bf16), 32, -1)
    fine = np.isfinite(s)
    with np.errstate(all="ignore"):
        at = np.where(s > 0, (x - m) / s, 0.0)
    near = np.abs(code - at) <= 0.5 + 2.0 ** -19
    assert (near | (code == 15) & (at > 15) | ~fine).all()


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("fp16", 64), ("bf16", 96), ("fp16", 96), ("bf16", 64),
                                     ("fp16", 128)])
@pytest.mark.parametrize("rot,inter,axes", [("none", False, 1), ("whole", False, 1), ("half", True, 2),
                                            ("half", False, 3), (16, False, 1), (48, False, 1)])
@pytest.mark.parametrize("lens,Hq,Hkv,page", [
    ([(1, 1), (1, 33), (0, 9), (1, 64)], 4, 2, 16), ([(37, 37), (5, 100), (64, 64), (1, 300)], 3, 3, 64),
    ([(200, 260)], 40, 5, 128), ([(1, 20)] * 70, 0, 1, 32)])
def test_append_quantizes_what_the_16_bit_append_stores(attn_lib, dtype, d, rot, inter, axes, lens, Hq, Hkv,
                                                       page):
    dt, bf16 = DT[dtype], dtype == "bf16"
    cu, kv, table, n_pages = batch(lens, page, d + len(lens))
    total = int(cu[-1])
    qkv = normal((total + 3, Hq + 2 * Hkv, d), dt, d)  # views of one projection, three rows of padding
    q, k, v = (t.transpose(0, 1) for t in qkv.split([Hq, Hkv, Hkv], 1))
    kw = dict(q=q if Hq else None, interleaved=inter)
    if rot != "none":
        rot = {"whole": d, "half": d // 2}.get(rot, rot)
        kw["table"] = attn_lib.rope_table(rot, axes=[p % axes for p in range(rot // 2)])
        if axes > 1:
            kw["positions"] = torch.randint(0, 5000, (axes, total + 3), dtype=torch.int32, device="cuda")
    args = cuda_i32(table), cuda_i32(cu), cuda_i32(kv)
    k16, v16 = (torch.zeros(n_pages, Hkv, page, d, dtype=dt, device="cuda") for _ in range(2))
    q16 = attn_lib.append_kv(k, v, k16, v16, *args, **kw)
    k4, v4 = (torch.full((n_pages, Hkv, page, d // 8 * 5), 0xA5, dtype=torch.uint8, device="cuda")
              for _ in range(2))
    q4 = attn_lib.append_kv4(k, v, k4, v4, *args, **kw)
    assert attn_lib.poll_status() == (0, 0)
    assert q4 is None if Hq == 0 else torch.equal(q4[:, :total], q16[:, :total])
    fresh = torch.zeros(n_pages, page, dtype=torch.bool, device="cuda")
    for b, (n, keys) in enumerate(lens):
        for p in range(keys - n, keys):
            fresh[table[b, p // page], p % page] = True
    for rows, x in ((k4, k16), (v4, v16)):
        rows, x = rows.transpose(1, 2), x.transpose(1, 2)
        assert (rows[~fresh] == 0xA5).all()
        check_codes(rows[fresh], x[fresh], bf16)
    # and back: the new tokens, then the whole cache
    ok, ov = (torch.full((Hkv, total + 3, d), 7.0, dtype=dt, device="cuda") for _ in range(2))
    attn_lib.read_kv4(k4, v4, *args, total + 3, dtype=dt, out_k=ok, out_v=ov)
    assert attn_lib.poll_status() == (0, 0)
    for got, rows in ((ok, k4), (ov, v4)):
        assert (got[:, total:] == 7.0).all()
        want = unpack4(rows, dt)
        for b, (n, keys) in enumerate(lens):
            p = torch.arange(keys - n, keys)
            at = torch.tensor(table[b])[p // page].cuda(), p.cuda() % page
            assert torch.equal(got[:, cu[b]:cu[b + 1]], want[at[0], :, at[1]].transpose(0, 1))


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_append_of_special_groups(attn_lib, dtype):
    """One value, zeros, both signs of zero, the type's largest and least
    numbers, an infinity, a NaN, a range past fp32: by the definition."""
    dt, bf16, d = DT[dtype], dtype == "bf16", 64
    big, tiny = torch.finfo(dt).max, torch.finfo(dt).smallest_normal
    g = torch.Generator().manual_seed(3)
    base = torch.randn(14, 32, generator=g)
    rows = [torch.full((32,), 3.25), torch.zeros(32), torch.zeros(32) * -1, base[0] * tiny, base[1] * big / 8,
            torch.linspace(-1, 1, 32) * (big / 2 if bf16 else big), base[2] * tiny / 8,
            torch.where(torch.arange(32) == 7, float("inf"), base[3]),
            torch.where(torch.arange(32) == 31, float("-inf"), base[4]),
            torch.where(torch.arange(32) == 0, float("nan"), base[5]),
            torch.linspace(-1, 1, 32) * big, base[6] + 300.0,
            torch.where(torch.arange(32) == 5, big, 0.0), torch.where(torch.arange(32) == 5, -big, 0.0)]
    n = len(rows)
    x = torch.stack([torch.cat([r, base[i % 14]]) for i, r in enumerate(rows)]).to(dt)
    x[1, 0] = -0.0
    k = x[None].cuda()
    k4, v4 = (torch.zeros(1, 1, 16, d // 8 * 5, dtype=torch.uint8, device="cuda") for _ in range(2))
    args = cuda_i32([[0]]), cuda_i32([0, n]), cuda_i32([n])
    attn_lib.append_kv4(k, k, k4, v4, *args)
    ok, ov = attn_lib.read_kv4(k4, v4, *args, n, dtype=dt)
    assert attn_lib.poll_status() == (0, 0)
    assert torch.equal(k4, v4) and torch.equal(ok.view(torch.int16), ov.view(torch.int16))
    rows4 = k4[0, 0, :n].cpu().numpy()
    want = oracle.quantize4(to64(x), bf16)
    par, wpar = (np.ascontiguousarray(r[:, d // 2:]).view("<u2") for r in (rows4, want))
    same = (par == wpar) | ((par & 0x7FFF) + (wpar & 0x7FFF) == 0)  # -0 for 0
    assert same.all()
    fine = np.isfinite(oracle.from16(wpar[:, ::2], bf16)).repeat(32, 1)
    got = to64(ok)[0]
    assert np.isnan(got[~fine]).all() and np.isfinite(got[fine]).all()
    # within half a step, and the two roundings of s and of the value
    s = oracle.from16(wpar[:, ::2], bf16).repeat(32, 1)
    u = torch.finfo(dt).eps / 2
    ref = to64(x)
    span = np.where(fine, 15 * s, 0)
    least = torch.finfo(dt).smallest_normal * torch.finfo(dt).eps  # a step of the subnormal numbers
    tol = s / 2 + span * 2 * u + 15 * least + np.abs(ref) * u + span * u
    assert (np.abs(got - ref)[fine] <= tol[fine] * (1 + 2 ** -10)).all()
    # three with an infinity or a NaN; in bf16 also base[1], whose product with the
    # largest number passes fp32 and is infinite, and the range of twice that number
    assert (~fine).any(1).sum() == (5 if bf16 else 3)


def test_append_reports_bad_pages_and_lengths(attn_lib):
    """As the 16-bit append: reported, nothing written for those rows."""
    dt, Hkv, page, d = torch.bfloat16, 1, 16, 64
    k, v = normal((Hkv, 3, d), dt, 3), normal((Hkv, 3, d), dt, 4)
    kp, vp = (torch.full((4, Hkv, page, 40), 0x11, dtype=torch.uint8, device="cuda") for _ in range(2))
    cu = cuda_i32([0, 1, 2, 3])
    for lens, table, bad in [([1, 33, 5], [[0, 1], [2, 3], [3, 3]], 1),
                             ([1, 17, 5], [[0, 1], [2, 4], [3, 3]], 1),
                             ([1, 2, 0], [[0, 1], [2, 3], [3, 3]], 2),
                             ([1, 2, 5], [[0, 1], [2, 3], [-1, 3]], 2)]:
        k1, v1 = kp.clone(), vp.clone()
        args = k1, v1, cuda_i32(table), cu, cuda_i32(lens)
        attn_lib.append_kv4(k, v, *args)
        st, detail = attn_lib.poll_status()
        assert st == 1 and detail >> 16 == bad, (st, hex(detail))
        for rows, x in ((k1, k), (v1, v)):
            want = kp.clone()
            for b in range(3):
                if b != bad:
                    want[table[b][(lens[b] - 1) // page], :, (lens[b] - 1) % page] = pack4(x[:, b])
            assert torch.equal(rows, want)
        ok, ov = torch.full_like(k, 9.0), torch.full_like(k, 9.0)
        attn_lib.read_kv4(*args, 3, dtype=dt, out_k=ok, out_v=ov)
        st, detail = attn_lib.poll_status()
        assert st == 1 and detail >> 16 == bad
        for got, x in ((ok, k), (ov, v)):
            assert (got[:, bad] == 9.0).all()
            for b in {0, 1, 2} - {bad}:
                assert torch.equal(got[:, b], unpack4(pack4(x[:, b]), dt))
    for c, n in (([0, 1, 2, 9], [9, 9, 9]), ([0, 2, 1, 3], [9, 9, 9]), ([0, 1, 1, 3], [9, 33, 9])):
        attn_lib.append_kv4(k, v, kp.clone(), vp.clone(), cuda_i32([[0, 1], [2, 3], [3, 3]]), cuda_i32(c),
                            cuda_i32(n))
        assert attn_lib.poll_status()[0] == 1
        attn_lib.read_kv4(kp, vp, cuda_i32([[0, 1], [2, 3], [3, 3]]), cuda_i32(c), cuda_i32(n), 3)
        assert attn_lib.poll_status()[0] == 1


# ------------------------------------------------------------ used together ---

@pytest.mark.parametrize("d", [64, 96, 128])
def test_serving_run(attn_lib, d):
    """Two prompts in chunks, then single tokens and drafts: each step appends
    turned keys in 4 bits and attends over the cache; the cache holds what was
    appended, and every output row is attention over what it stands for."""
    Hq, Hkv, page, dt = 6, 2, 16, torch.bfloat16
    steps = [(70, 20), (50, 0), (1, 33), (1, 1), (1, 1), (4, 1)]  # new tokens of the two sequences
    rope = attn_lib.rope_table(d)
    table = np.random.default_rng(0).permutation(24).reshape(2, 12)
    kp, vp = (torch.full((24, Hkv, page, d // 8 * 5), 0xFF, dtype=torch.uint8, device="cuda") for _ in range(2))
    full = [[], []]  # what was stored, by sequence
    kv = [0, 0]
    for i, new in enumerate(steps):
        total = sum(new)
        q, k, v = (normal((h, total, d), dt, 10 * i + h) for h in (Hq, Hkv, Hkv + 100))
        v = v[:Hkv].contiguous()
        kv = [a + n for a, n in zip(kv, new)]
        cu = cuda_i32([0, new[0], total])
        args = cuda_i32(table), cu, cuda_i32(kv)
        q2 = attn_lib.append_kv4(k, v, kp, vp, *args, table=rope, q=q)
        pos = torch.cat([torch.arange(a - n, a) for a, n in zip(kv, new)]).int().cuda()[None]
        ref_q, ref_k = attn_lib.rope(q, k, pos, rope)
        assert torch.equal(q2, ref_q)
        o, lse = attn_lib.fwd_paged4(q2, kp, vp, *args, max(new), causal=True)
        whole = cuda_i32([0, kv[0], sum(kv)])
        ck, cv = attn_lib.read_kv4(kp, vp, cuda_i32(table), whole, cuda_i32(kv), sum(kv), dtype=dt)
        assert attn_lib.poll_status() == (0, 0)
        for b in range(2):
            rows = slice(0, new[0]) if b == 0 else slice(new[0], total)
            full[b].append((unpack4(pack4(ref_k[:, rows]), dt), unpack4(pack4(v[:, rows]), dt)))
            at = slice(0, kv[0]) if b == 0 else slice(kv[0], sum(kv))
            assert torch.equal(ck[:, at], torch.cat([f[0] for f in full[b]], 1))
            assert torch.equal(cv[:, at], torch.cat([f[1] for f in full[b]], 1))
        x = dict(q=q2, k4=kp, v4=vp, table=args[0], cu=cu, kv=args[2], max_q=max(new))
        check4(x, o, lse, True)


@pytest.mark.parametrize("chunk", [1, 50])
def test_captured_step_replays_with_new_lengths(attn_lib, chunk):
    """A graph of append + attention + reading back replays on new lengths, pages
    and tokens written into the same tensors, on a side stream."""
    Hq, Hkv, d, page, dt = 4, 2, 64, 16, torch.bfloat16
    rope = attn_lib.rope_table(d)
    kp, vp = (torch.zeros(20, Hkv, page, 40, dtype=torch.uint8, device="cuda") for _ in range(2))
    batches = []
    for i, lens in enumerate([[(chunk, chunk + 30), (1, 9)], [(1, chunk + 29), (chunk, chunk + 40)]]):
        cu, kv, table, _ = batch(lens, page, i)
        table = np.pad(table, ((0, 0), (0, 10 - table.shape[1])))
        new = [normal((h, chunk + 1, d), dt, 7 * i + h) for h in (Hq, Hkv, Hkv)]
        batches.append([*new, cuda_i32(table), cuda_i32(cu), cuda_i32(kv)])
    hold = [t.clone() for t in batches[0]]
    pages = kp.random_(0, 112).clone(), vp.random_(0, 112).clone()  # any bytes but NaN
    ws = torch.empty(max(1, attn_lib.fwd_paged_workspace_bytes(2, chunk, 160, Hq, Hkv, d)), dtype=torch.uint8,
                     device="cuda")

    def step(s, k4, v4):
        q = attn_lib.append_kv4(s[1], s[2], k4, v4, *s[3:], table=rope, q=s[0])
        o, lse = attn_lib.fwd_paged4(q, k4, v4, *s[3:], chunk, causal=True, workspace=ws)
        return (q, o, lse, *attn_lib.read_kv4(k4, v4, *s[3:], chunk + 1, dtype=dt))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(hold, kp, vp)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        out = step(hold, kp, vp)
    for s in (batches[0], batches[1], batches[0]):
        for h, t in zip(hold, s):
            h.copy_(t)
        kp.copy_(pages[0])
        vp.copy_(pages[1])
        graph.replay()
        got = [t.clone() for t in out]
        want = step(s, pages[0].clone(), pages[1].clone())
        # by their bits: some of the cache's random scales are so large that scores are NaN
        assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(got, want))
    assert attn_lib.poll_status() == (0, 0)


@pytest.mark.parametrize("chunk", [1, 40])
def test_pages_past_two_to_the_31_bytes(attn_lib, chunk):
    """A cache of 4.7e9 bytes a tensor: pages at both ends."""
    Hq, Hkv, d, page, dt = 4, 2, 128, 64, torch.float16
    n_pages = 460_000
    kp, vp = (torch.empty(n_pages, Hkv, page, 80, dtype=torch.uint8, device="cuda") for _ in range(2))
    table = [[n_pages - 1, 3, n_pages - 2]]
    n = 150
    q, k, v = (normal((h, n, d), dt, h) for h in (Hq, Hkv, Hkv + 1))
    v = v[:Hkv].contiguous()
    args = cuda_i32(table), cuda_i32([0, n]), cuda_i32([n])
    attn_lib.append_kv4(k, v, kp, vp, *args)
    ck, cv = attn_lib.read_kv4(kp, vp, *args, n, dtype=dt)
    assert torch.equal(ck, unpack4(pack4(k), dt)) and torch.equal(cv, unpack4(pack4(v), dt))
    q = q[:, :chunk].contiguous()
    o, lse = attn_lib.fwd_paged4(q, kp, vp, args[0], cuda_i32([0, chunk]), args[2], chunk, causal=True)
    assert attn_lib.poll_status() == (0, 0)
    at = torch.tensor(table[0]).cuda()
    x = dict(q=q, k4=kp[at], v4=vp[at], table=cuda_i32([[0, 1, 2]]), cu=cuda_i32([0, chunk]), kv=args[2],
             max_q=chunk)
    check4(x, o, lse, True)


def test_binding_refuses_wrong_tensors(attn_lib):
    """What the Python entry checks; the same arguments put right then work."""
    dt, Hkv, page, d = torch.bfloat16, 2, 16, 64
    kp, vp = (torch.zeros(4, Hkv, page, 40, dtype=torch.uint8, device="cuda") for _ in range(2))
    k, q = normal((Hkv, 3, d), dt, 1), normal((4, 3, d), dt, 2)
    rest = cuda_i32([[0, 1]]), cuda_i32([0, 3]), cuda_i32([20])
    wrong = [kp.float(), kp.bfloat16(), kp.cpu(), kp[..., :32], kp[..., :32].contiguous(), kp[:3], kp[0],
             kp.transpose(1, 2), kp.view(torch.int8), None, 3]
    for w in wrong:
        for pages in ((w, vp), (kp, w)):
            for call in (lambda: attn_lib.append_kv4(k, k, *pages, *rest),
                         lambda: attn_lib.fwd_paged4(q, *pages, *rest, 3),
                         lambda: attn_lib.read_kv4(*pages, *rest, 3)):
                with pytest.raises((ValueError, TypeError)):
                    call()
    with pytest.raises(ValueError):  # a 4-bit cache is none of 16 bits, nor the other way round
        attn_lib.append_kv(k, k, kp, vp, *rest)
    with pytest.raises(ValueError):
        attn_lib.fwd_paged(q, kp, vp, *rest, 3)
    for kw in (dict(dtype=torch.float32), dict(dtype="bf16"), dict(out_k=k.half()), dict(out_k=k[:1]),
               dict(out_v=k.transpose(0, 1).contiguous().transpose(0, 1)), dict(out_v=k.cpu()), dict(total=0),
               dict(total="x")):
        with pytest.raises((ValueError, TypeError)):
            attn_lib.read_kv4(kp, vp, *rest, **dict(dict(total=3), **kw))
    same = torch.empty_like(k)
    with pytest.raises(attn_lib.AttnError):
        attn_lib.read_kv4(kp, vp, *rest, 3, out_k=same, out_v=same)
    wide = [torch.zeros(4, Hkv, page, 120, dtype=torch.uint8, device="cuda") for _ in range(2)]
    with pytest.raises(attn_lib.AttnError) as e:  # d = 192
        attn_lib.read_kv4(*wide, *rest, 3)
    assert e.value.status == 2
    assert attn_lib.poll_status() == (0, 0)
    attn_lib.append_kv4(k, k, kp, vp, *rest)
    attn_lib.fwd_paged4(q, kp, vp, *rest, 3)
    attn_lib.read_kv4(kp, vp, *rest, 3)
    assert attn_lib.poll_status() == (0, 0)


@pytest.mark.parametrize("lens,reach", [([(1, 700), (2, 64)], 16), ([(1, 700), (1, 64)] * 12, 5000),
                                        ([(40, 700), (33, 64)], 16), ([(20, 3500)], 16)])
@pytest.mark.parametrize("k_amp,q_amp", [(2.0 ** 40, 2.0 ** -40), (2.0 ** -60, 2.0 ** 60), (2.0 ** -70, 2.0 ** -40),
                                         (2.0 ** 17, 2.0 ** -17)])
def test_far_exponents_of_bf16(four, lens, reach, k_amp, q_amp):
    """Keys and queries outside fp16's range in a bf16 cache: by themselves far
    too large or small, their scores ordinary (or all but 0)."""
    x = widen(paged.make(lens, 4, 2, 128, 32, "bf16", seed=107), reach)
    x["k4"] = pack4(x["k"] * k_amp)
    x["q"] = x["q"] * q_amp
    o, lse = paged.run(four, x, True)
    assert four.poll_status() == (0, 0)
    check4(x, o, lse, True)


@pytest.mark.parametrize("lens,reach", [([(1, 700)], 16), ([(40, 700)], 16)])
def test_a_large_key_among_others(four, lens, reach):
    """One key a thousand times the others: its neighbours keep their precision."""
    x = widen(paged.make(lens, 4, 2, 128, 32, "bf16", seed=109), reach)
    k, table = x["k"].clone(), x["table"].tolist()
    k[table[0][300 // 32], :, 300 % 32] *= 1000.0
    x["k4"] = pack4(k)
    o, lse = paged.run(four, x, True)
    assert four.poll_status() == (0, 0)
    check4(x, o, lse, True)
