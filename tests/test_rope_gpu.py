"""Rotary positions and the paged append: CUDA path vs the fp64 oracle.

Tolerance per element, from the arithmetic: the output rounding is half a step
(u = finfo.eps / 2 of the value; below the normal range half the smallest
step); before it, |a| + |b| times the error of cosine, sine and the two
products in fp32: sincospi within 2 ulp of 1 (1.2e-7), its argument rounded to
24 bits of half a turn (2^-25 turns, 1.9e-7 rad), two products and a sum
(3 * 2^-24): 5e-7 in all.
"""
import numpy as np
import pytest
import torch

import oracle
from helpers import to64

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp16": torch.float16}


def _freq(rot, axes):
    half = rot // 2
    return 10000.0 ** (-np.arange(half) / half), np.arange(half) * axes // half


def _table(attn, rot, axes):
    return attn.rope_table(rot, axes=_freq(rot, axes)[1].tolist())


def _close(got, ref, x, dtype):
    """got vs ref, x the input rows (their channel pairs bound |a| + |b|)."""
    u = torch.finfo(dtype).eps / 2
    pre = 5e-7 * 2 * np.max(np.abs(to64(x)), axis=-1, keepdims=True)
    tol = u * np.abs(ref) + (1 + u) * pre + torch.finfo(dtype).smallest_normal * u
    err = np.abs(to64(got) - ref)
    assert (err <= tol).all(), float(np.max(err - tol))


def _normal(shape, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(shape, generator=g).to(dtype).cuda()


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("B,Hq,Hkv,N,d,rot,axes", [
    (1, 1, 1, 1, 64, 64, 1), (2, 4, 2, 37, 96, 96, 3), (3, 5, 1, 129, 128, 64, 2),
    (1, 7, 7, 300, 192, 16, 4), (2, 2, 1, 65, 256, 256, 8), (1, 16, 4, 1030, 128, 48, 3)])
def test_rope_and_its_backward(attn_lib, dtype, interleaved, B, Hq, Hkv, N, d, rot, axes):
    dt = DT[dtype]
    q, k = _normal((B, Hq, N, d), dt, 1), _normal((B, Hkv, N, d), dt, 2)
    g = np.random.default_rng(N)
    pos = g.integers(-1000, 100000, (axes, B, N))
    inv, axis = _freq(rot, axes)
    table = _table(attn_lib, rot, axes)
    p = torch.tensor(pos, dtype=torch.int32, device="cuda")
    for inverse, fn in ((False, attn_lib.rope), (True, attn_lib.rope_bwd)):
        yq, yk = fn(q, k, p, table, interleaved=interleaved)
        for x, y in ((q, yq), (k, yk)):
            ref = np.stack([oracle.rotary(to64(x[b]), pos[:, b], inv, axis, interleaved, inverse)
                            for b in range(B)])
            _close(y, ref, x, dt)
    assert attn_lib.poll_status() == (0, 0)


def test_rope_views_broadcast_positions_and_in_place(attn_lib):
    """q and k sliced out of a fused projection [B, N, heads, d], one set of
    positions for the batch, k left out, and outputs over the inputs."""
    B, N, H, Hkv, d = 2, 50, 4, 2, 64
    dt = torch.bfloat16
    qkv = _normal((B, N, H + 2 * Hkv, d), dt, 3)
    keep = qkv.clone()
    q, k = qkv[:, :, :H].transpose(1, 2), qkv[:, :, H:H + Hkv].transpose(1, 2)
    table = _table(attn_lib, d, 1)
    pos = torch.arange(N, dtype=torch.int32, device="cuda")[None]
    yq, yk = attn_lib.rope(q, k, pos, table)
    assert yq.is_contiguous() and yk.is_contiguous() and torch.equal(qkv, keep)
    a, b = attn_lib.rope(q.contiguous(), k.contiguous(),
                         pos[:, None].expand(1, B, N).contiguous(), table)
    assert torch.equal(a, yq) and torch.equal(b, yk)
    assert torch.equal(attn_lib.rope(q, None, pos, table)[0], yq)
    packed = attn_lib.rope(q[1], k[1], pos, table)
    assert torch.equal(packed[0], yq[1]) and torch.equal(packed[1], yk[1])
    attn_lib.rope(q, k, pos, table, out_q=q, out_k=k)
    assert torch.equal(q, yq) and torch.equal(k, yk)
    assert torch.equal(qkv[:, :, H + Hkv:], keep[:, :, H + Hkv:])


def test_rope_holds_at_far_positions(attn_lib):
    """Positions up to 2^31 - 1 and below zero: the angle is exact modulo a turn."""
    pos = np.array([[0, 1, -1, 2 ** 20, 2 ** 24 + 1, 2 ** 31 - 1, -2 ** 31]])
    q = _normal((1, pos.shape[1], 128), torch.float16, 4)
    inv, axis = _freq(128, 1)
    y, _ = attn_lib.rope(q, None, torch.tensor(pos, dtype=torch.int32, device="cuda"),
                         _table(attn_lib, 128, 1))
    # the fp64 angle itself is off by 2^-53 of up to 2^31 radians: 2^-21 there
    near = [i for i in range(pos.shape[1]) if abs(int(pos[0, i])) < 2 ** 25]
    ref = oracle.rotary(to64(q), pos, inv, axis, False)
    _close(y[:, near], ref[:, near], q[:, near], torch.float16)
    err = np.abs(to64(y) - ref)
    assert err.max() <= 2 ** -11 * np.abs(ref).max() + 2 ** -20 * 2 * np.abs(to64(q)).max()


def test_rope_of_many_rows(attn_lib):
    """More blocks of rows than a grid's second dimension holds, elements past
    2^31 bytes; the first, last and some middle rows against the oracle."""
    N, d, H = 600_000, 256, 4
    q = torch.empty(1, H, N, d, dtype=torch.bfloat16, device="cuda")
    q.normal_(generator=torch.Generator("cuda").manual_seed(3))
    pos = torch.arange(N, dtype=torch.int32, device="cuda")[None]
    inv, axis = _freq(d, 1)
    y, _ = attn_lib.rope(q, None, pos, _table(attn_lib, d, 1))
    at = torch.tensor([0, 1, 524_287, 524_288, 524_300, N - 2, N - 1], device="cuda")
    for h in (0, H - 1):
        ref = oracle.rotary(to64(q[0, h, at]), at.cpu().numpy()[None], inv, axis, False)
        _close(y[0, h, at], ref, q[0, h, at], torch.bfloat16)


def test_rope_gradient_by_differences(attn_lib):
    """<dy, rope(x + e) - rope(x - e)> against <rope_bwd(dy), 2 e>: the map is
    linear, so large steps are exact up to the fp16 roundings (2^-11 each)."""
    table = _table(attn_lib, 64, 2)
    pos = torch.tensor([[3, 50], [9, 4]], dtype=torch.int32, device="cuda")
    x, dy = _normal((1, 2, 64), torch.float16, 5), _normal((1, 2, 64), torch.float16, 6)
    dx = to64(attn_lib.rope_bwd(dy, None, pos, table)[0])
    w = to64(dy)
    for n, c in [(0, 0), (0, 40), (1, 31), (1, 32), (1, 63)]:
        e = torch.zeros_like(x)
        e[0, n, c] = 4.0
        up, dn = (to64(attn_lib.rope(x + s * e, None, pos, table)[0]) for s in (1, -1))
        size = np.sum(np.abs(w) * (np.abs(up) + np.abs(dn)))
        step = abs(to64(x)[0, n, c]) + 4.0  # rounding of x +- e
        assert abs(np.sum(w * (up - dn)) - 8.0 * dx[0, n, c]) <= \
            2 ** -11 * (size + 8 * abs(dx[0, n, c]) + 4 * step * np.abs(w).max())


def _cache(n_pages, Hkv, page, d, dt, seed):
    return _normal((n_pages, Hkv, page, d), dt, seed), _normal((n_pages, Hkv, page, d), dt, seed + 1)


@pytest.mark.parametrize("dtype,d,rot", [("bf16", 128, 128), ("fp16", 64, 32), ("bf16", 96, 96),
                                         ("fp16", 256, 64), ("bf16", 192, None)])
@pytest.mark.parametrize("page", [16, 64, 256])
@pytest.mark.parametrize("with_q,given", [(True, False), (False, True), (True, True)])
def test_append(attn_lib, dtype, d, rot, page, with_q, given):
    """Ragged sequences (one empty, one new, one that fills its pages), views
    of a projection, padding rows behind the last sequence."""
    dt = DT[dtype]
    Hq, Hkv, axes = 4, 2, 2
    new, keys = [1, 0, 5, 40, 16], [33, 7, 5, 256, 16]
    total = sum(new) + 3
    cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    width = -(-max(keys) // page)
    g = np.random.default_rng(page + d)
    n_pages = width * len(keys) + 2
    table = g.permutation(n_pages)[:width * len(keys)].reshape(-1, width).astype(np.int32)
    dead = table.copy()
    for b, n in enumerate(keys):
        dead[b, -(-n // page):] = -5  # entries past the length are not read
    kp, vp = _cache(n_pages, Hkv, page, d, dt, 7)
    qkv = _normal((total, Hq + 2 * Hkv, d), dt, 9)
    q, k, v = (t.transpose(0, 1) for t in qkv.split([Hq, Hkv, Hkv], 1))
    pos = g.integers(0, 5000, (axes, total)) if given and rot else None
    place = np.zeros((1, total), np.int64)
    for b, n in enumerate(new):
        place[0, cu[b]:cu[b + 1]] = np.arange(keys[b] - n, keys[b])
    cuda = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    kw = {}
    if rot:
        inv, axis = _freq(rot, axes)
        kw = dict(table=_table(attn_lib, rot, axes), interleaved=given,
                  positions=None if pos is None else cuda(pos))
        turn = lambda x: oracle.rotary(  # noqa: E731
            to64(x), np.repeat(place, axes, 0) if pos is None else pos, inv, axis, given)
    else:
        turn = to64
    if with_q:
        kw["q"] = q
        kw["out_q"] = torch.full((Hq, total, d), 7.0, dtype=dt, device="cuda")
    k0, v0 = kp.clone(), vp.clone()
    out = attn_lib.append_kv(k, v, kp, vp, cuda(dead), cuda(cu), cuda(keys), **kw)
    assert attn_lib.poll_status() == (0, 0)
    live = slice(0, int(cu[-1]))
    if with_q:
        _close(out[:, live], turn(q)[:, live], q[:, live], dt)
        assert (out[:, live.stop:] == 7.0).all()
    else:
        assert out is None
    kref = oracle.append_paged(turn(k), to64(k0), table, cu, np.array(keys))
    vref = oracle.append_paged(to64(v), to64(v0), table, cu, np.array(keys))
    assert np.array_equal(to64(vp), vref)
    touched = np.any(kref != to64(k0), axis=-1)
    assert torch.equal(kp[torch.tensor(~touched).cuda()], k0[torch.tensor(~touched).cuda()])
    _close(kp, kref, torch.full_like(kp, float(k.abs().max())), dt)


def test_append_reports_bad_pages_and_lengths(attn_lib):
    """A page number outside the cache, a length past the table and a negative
    place: reported, nothing written for those rows, the others written."""
    dt, Hkv, page, d = torch.bfloat16, 1, 16, 64
    kp, vp = _cache(4, Hkv, page, d, dt, 1)
    k, v = _normal((Hkv, 3, d), dt, 3), _normal((Hkv, 3, d), dt, 4)
    cuda = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    cu = cuda([0, 1, 2, 3])
    for lens, table, bad in [([1, 33, 5], [[0, 1], [2, 3], [3, 3]], 1),
                             ([1, 17, 5], [[0, 1], [2, 4], [3, 3]], 1),
                             ([1, 2, 0], [[0, 1], [2, 3], [3, 3]], 2),
                             ([1, 2, 5], [[0, 1], [2, 3], [-1, 3]], 2)]:
        k1, v1 = kp.clone(), vp.clone()
        attn_lib.append_kv(k, v, k1, v1, cuda(table), cu, cuda(lens))
        st, detail = attn_lib.poll_status()
        assert st == 1 and detail >> 16 == bad, (st, hex(detail))
        want_k, want_v = kp.clone(), vp.clone()
        for b in range(3):
            if b != bad:
                at = lens[b] - 1
                want_k[table[b][at // page], :, at % page] = k[:, b]
                want_v[table[b][at // page], :, at % page] = v[:, b]
        assert torch.equal(k1, want_k) and torch.equal(v1, want_v)


def test_append_reports_lengths_and_offsets_out_of_range(attn_lib):
    """Offsets that run past the tokens, fall, or do not begin at 0, and a
    length past the table of a sequence without new tokens: reported."""
    dt, Hkv, page, d = torch.bfloat16, 1, 16, 64
    kp, vp = _cache(6, Hkv, page, d, dt, 1)
    k, v = _normal((Hkv, 3, d), dt, 3), _normal((Hkv, 3, d), dt, 4)
    cuda = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    table = cuda([[0, 1], [2, 3], [4, 5]])
    good = ([0, 1, 2, 3], [30, 30, 30])
    for cu, lens, bad in [([0, 1, 2, 9], [30, 30, 30], 2), ([0, 2, 1, 3], [30, 30, 30], 1),
                          ([0, 1, 1, 3], [30, 33, 30], 1), ([0, 1, 1, 3], [30, -1, 30], 1),
                          ([0, 3, 3, 3], [30, 30, 40], 2), ([0, 5, 3, 3], [30, 30, 30], None),
                          ([-1, 1, 2, 3], [30, 30, 30], 0)]:
        for c, n, want in ((cu, lens, 1), (good[0], good[1], 0)):
            attn_lib.append_kv(k, v, kp.clone(), vp.clone(), table, cuda(c), cuda(n))
            st, detail = attn_lib.poll_status()
            assert st == want, (c, n, st, hex(detail))
            assert not want or bad is None or detail >> 16 == bad, (c, n, hex(detail))
    # more sequences than tokens
    many = 4000
    cu, lens = [0] + [3] * many, [30] * many
    table = cuda([[0, 1]] * many)
    attn_lib.append_kv(k, v, kp.clone(), vp.clone(), table, cuda(cu), cuda(lens))
    assert attn_lib.poll_status() == (0, 0)
    lens[3777] = 33
    attn_lib.append_kv(k, v, kp.clone(), vp.clone(), table, cuda(cu), cuda(lens))
    st, detail = attn_lib.poll_status()
    assert st == 1 and detail >> 16 == 3777


def test_outputs_over_inputs(attn_lib):
    """Outputs at the address of their input: the same layout works, whatever
    the strides of dimensions of size 1; another one is refused and leaves the
    input alone."""
    d, dt = 64, torch.bfloat16
    table = _table(attn_lib, d, 1)
    for heads, n in ((4, 30), (4, 1), (1, 30)):
        pos = torch.arange(n, dtype=torch.int32, device="cuda")[None]
        rows = _normal((n, heads, d), dt, heads + n)  # by token
        q, flat = rows.transpose(0, 1), rows.view(heads, n, d)
        keep, want = rows.clone(), attn_lib.rope(q.contiguous(), None, pos, table)[0]
        kp, vp = _cache(2, 1, 64, d, dt, 1)
        kv = _normal((1, n, d), dt, 3)
        cuda = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
        batch = kp, vp, cuda([[0]]), cuda([0, n]), cuda([n])
        if heads > 1 and n > 1:
            for call in (lambda: attn_lib.rope(q, None, pos, table, out_q=flat),
                         lambda: attn_lib.append_kv(kv, kv, *batch, table=table, q=q, out_q=flat)):
                with pytest.raises(attn_lib.AttnError) as e:
                    call()
                assert e.value.status == 1 and torch.equal(rows, keep)
        else:
            attn_lib.rope(q, None, pos, table, out_q=flat)
            assert torch.equal(flat, want)
            rows.copy_(keep)
            attn_lib.append_kv(kv, kv, *batch, table=table, q=q, out_q=flat)
            assert torch.equal(flat, want)
            rows.copy_(keep)
        attn_lib.rope(q, None, pos, table, out_q=q)
        assert torch.equal(q, want)
        full = keep.transpose(0, 1).contiguous()
        attn_lib.append_kv(kv, kv, *batch, table=table, q=full, out_q=full)
        assert torch.equal(full, want)
        with pytest.raises(attn_lib.AttnError):
            attn_lib.append_kv(full, full, *(t.expand(2, heads, 64, d).contiguous() for t in batch[:2]),
                               *batch[2:], table=table, q=want, out_q=full)
    assert attn_lib.poll_status() == (0, 0)
