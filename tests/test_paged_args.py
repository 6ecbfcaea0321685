"""Argument checks of rotary positions and the paged cache: refused on the
host before anything is launched (CPU)."""
import ctypes
import math

import numpy as np
import pytest
import torch

import exact_attention_75_gb300 as attn

P, BAD = ctypes.c_void_p(0x10000), ctypes.c_void_p(0x10008)
INVALID, UNSUPPORTED = 1, 2


@pytest.fixture(scope="module")
def L():
    from exact_attention_75_gb300 import build
    build.build()
    return attn.lib()


def _strides(n, value=64):
    return (ctypes.c_int64 * n)(*[value] * n)


ROPE = dict(q=P, k=P, oq=P, ok=P, strides=_strides(12), pos=P, pos_batches=1, axes=1, table=P,
            rot=64, inter=0, inverse=0, B=2, Hq=4, Hkv=2, N=8, d=64, dtype=1, stream=None)


@pytest.mark.parametrize("change,want", [
    (dict(q=BAD), INVALID), (dict(oq=None), INVALID), (dict(k=None), INVALID),
    (dict(ok=None), INVALID), (dict(k=None, ok=None), INVALID), (dict(Hkv=0), INVALID),
    (dict(table=None), INVALID), (dict(table=BAD), INVALID), (dict(pos=None), INVALID), (dict(pos_batches=3), INVALID),
    (dict(rot=0), INVALID), (dict(rot=24), INVALID), (dict(rot=80), INVALID),
    (dict(axes=0), INVALID), (dict(axes=9), INVALID), (dict(strides=_strides(12, 63)), INVALID),
    (dict(strides=_strides(12, -64)), INVALID), (dict(strides=None), INVALID),
    (dict(B=0), INVALID), (dict(N=0), INVALID), (dict(d=80), UNSUPPORTED),
    (dict(dtype=2), INVALID), (dict(inter=2), INVALID), (dict(inverse=-1), INVALID),
    (dict(B=70000, pos_batches=1), INVALID)])
def test_rope_refusals(L, change, want):
    assert L.attn_rope(*dict(ROPE, **change).values()) == want


APPEND = dict(k=P, v=P, q=P, oq=P, strides=_strides(6), kp=P, vp=P, table=P, cu=P, kv=P, pos=None,
              axes=1, rtable=P, rot=64, inter=0, n_seq=2, total=9, n_pages=8, page=16, max_pages=4,
              Hq=4, Hkv=2, d=64, dtype=0, stream=None)


@pytest.mark.parametrize("change,want", [
    (dict(k=BAD), INVALID), (dict(v=None), INVALID), (dict(q=None), INVALID),
    (dict(oq=None), INVALID), (dict(Hq=0), INVALID), (dict(Hq=3), INVALID),
    (dict(kp=None), INVALID), (dict(vp=BAD), INVALID), (dict(cu=None), INVALID),
    (dict(kv=None), INVALID), (dict(table=None), INVALID), (dict(page=48), UNSUPPORTED),
    (dict(page=8), UNSUPPORTED), (dict(d=72), UNSUPPORTED), (dict(rot=128), INVALID),
    (dict(rtable=None, pos=P), INVALID), (dict(n_seq=0), INVALID), (dict(total=0), INVALID),
    (dict(n_pages=0), INVALID), (dict(max_pages=0), INVALID), (dict(Hkv=0), INVALID),
    (dict(max_pages=1 << 26), INVALID), (dict(rtable=BAD), INVALID), (dict(n_pages=1 << 30), INVALID),
    (dict(strides=_strides(6, 12)), INVALID), (dict(inter=3), INVALID)])
def test_append_refusals(L, change, want):
    assert L.attn_append_kv(*dict(APPEND, **change).values()) == want


# the refusals above once more with operands that lie apart, so that each is due
# to its own change alone
P1, P2, P3, P4 = (ctypes.c_void_p(x << 20) for x in (2, 3, 4, 5))
ROPE_APART = dict(ROPE, k=P1, oq=P2, ok=P3)
APPEND_APART = dict(APPEND, v=P1, q=P2, oq=P3, kp=P4, vp=ctypes.c_void_p(6 << 20))


@pytest.mark.parametrize("change,want", test_rope_refusals.pytestmark[0].args[1])
def test_rope_refusals_of_operands_apart(L, change, want):
    assert L.attn_rope(*dict(ROPE_APART, **change).values()) == want


@pytest.mark.parametrize("change,want", test_append_refusals.pytestmark[0].args[1])
def test_append_refusals_of_operands_apart(L, change, want):
    assert L.attn_append_kv(*dict(APPEND_APART, **change).values()) == want


def _i64(*s):
    return (ctypes.c_int64 * len(s))(*s)


# q, k views of a projection [B, N, heads, d]; contiguous outputs
ROPE_VIEWS = _i64(8 * 512, 64, 512, 4 * 8 * 64, 8 * 64, 64, 8 * 512, 64, 512, 2 * 8 * 64, 8 * 64, 64)


@pytest.mark.parametrize("change", [
    dict(oq=P, strides=ROPE_VIEWS), dict(ok=P1, strides=ROPE_VIEWS), dict(oq=P1), dict(ok=P),
    dict(ok=P2), dict(oq=P, strides=_i64(64, 64, 64, 64, 64, 128, 64, 64, 64, 64, 64, 64)),
    dict(oq=P, B=1, pos_batches=1, strides=_i64(0, 64, 512, 0, 128, 512, 0, 64, 64, 0, 64, 64)),
    dict(ok=P1, N=1, strides=_i64(64, 64, 0, 64, 64, 0, 128, 64, 0, 256, 64, 64))])
def test_rope_refuses_outputs_over_inputs_of_another_layout(L, change):
    assert L.attn_rope(*dict(ROPE_APART, **change).values()) == INVALID


@pytest.mark.parametrize("change", [
    dict(oq=P2), dict(oq=P2, strides=_i64(64, 512, 64, 512, 64, 512)),  # rows by token, by head
    dict(oq=P2, Hq=2, strides=_i64(576, 64, 576, 64, 640, 64)),
    dict(oq=P2, total=1, strides=_i64(64, 0, 64, 0, 128, 0)),
    dict(oq=P), dict(oq=P1), dict(oq=P4), dict(oq=ctypes.c_void_p(6 << 20))])
def test_append_refuses_turned_queries_over_inputs(L, change):
    assert L.attn_append_kv(*dict(APPEND_APART, **change).values()) == INVALID


PAGED = dict(q=P, kp=P, vp=P, o=P, lse=P, table=P, cu=P, kv=P, ws=P, ws_bytes=1 << 40, n_seq=2,
             max_q=4, total=9, n_pages=8, page=16, max_pages=4, Hq=4, Hkv=2, d=64, causal=1,
             scale=0.1, dtype=1, stream=None)


@pytest.mark.parametrize("change,want", [
    (dict(q=BAD), INVALID), (dict(o=None), INVALID), (dict(lse=None), INVALID),
    (dict(kp=BAD), INVALID), (dict(ws=BAD, max_q=9), INVALID), (dict(ws=None, max_q=9), INVALID),
    (dict(ws_bytes=256, max_q=9), INVALID), (dict(max_q=0), INVALID), (dict(max_q=10), INVALID),
    (dict(Hq=5), INVALID), (dict(Hq=258), UNSUPPORTED), (dict(d=192), UNSUPPORTED),
    (dict(d=80), UNSUPPORTED), (dict(page=512), UNSUPPORTED), (dict(causal=2), INVALID),
    (dict(scale=0.0), INVALID), (dict(scale=math.inf), INVALID), (dict(scale=math.nan), INVALID),
    (dict(dtype=5), INVALID), (dict(n_seq=0), INVALID)])
def test_paged_refusals(L, change, want):
    assert L.attn_fwd_paged(*dict(PAGED, **change).values()) == want


def test_workspace_sizes(L):
    assert attn.fwd_paged_workspace_bytes(64, 1, 65536, 16, 4, 128) > 0
    assert attn.fwd_paged_workspace_bytes(1, 40, 64, 16, 4, 128) > 0
    assert attn.fwd_paged_workspace_bytes(1, 1, 64, 16, 4, 128) == 0  # small: none needed
    for bad in ((0, 40, 64, 16, 4, 128), (1, 0, 64, 16, 4, 128), (1, 40, 0, 16, 4, 128),
                (1, 40, 1 << 40, 16, 4, 128), (1, 40, 64, 16, 5, 128), (1, 40, 64, 16, 4, 192),
                (1, 40, 64, 0, 1, 64)):
        assert attn.fwd_paged_workspace_bytes(*bad) == 0


def test_workspace_of_sizes_the_call_refuses(L):
    assert attn.fwd_paged_workspace_bytes(1, 40, 64, 128, 1, 64) > 0
    assert attn.fwd_paged_workspace_bytes(1, 40, 64, 129, 1, 64) == 0
    assert attn.fwd_paged_workspace_bytes(1, 1, 64, 258, 2, 64) == 0


def test_rope_table_is_the_angle_per_position():
    t = attn.rope_table(32, theta=500.0, axes=[0] * 4 + [1] * 6 + [2] * 6, device="cpu")
    assert t.shape == (2, 16) and t.dtype == torch.int64
    want = 500.0 ** (-np.arange(16) / 16) / (2 * math.pi)
    assert np.allclose(t[0].numpy() / 2.0 ** 64, want, rtol=1e-15)
    assert t[1].tolist() == [0] * 4 + [1] * 6 + [2] * 6
    # whole turns drop out, a negative frequency is the opposite turn
    t = attn.rope_table(16, inv_freq=[2 * math.pi * x for x in (0.75, -0.25, 5.25, 0, 1, 2, 3, 4)],
                        device="cpu")
    assert np.allclose(t[0].numpy() / 2.0 ** 64, [-0.25, -0.25, 0.25, 0, 0, 0, 0, 0], atol=1e-15)
    for kw in (dict(rot=24), dict(rot=0), dict(rot=32, axes=[0] * 15), dict(rot=16, axes=[8] * 8),
               dict(rot=16, axes=[-1] * 8), dict(rot=16, inv_freq=[math.nan] * 8)):
        with pytest.raises(ValueError):
            attn.rope_table(device="cpu", **kw)


def test_binding_refuses_cpu_tensors():
    t = attn.rope_table(64, device="cpu")
    q = torch.zeros(2, 5, 64, dtype=torch.bfloat16)
    pages = torch.zeros(3, 2, 16, 64, dtype=torch.bfloat16)
    i = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    with pytest.raises(ValueError):
        attn.rope(q, q, i(1, 5), t)
    with pytest.raises(ValueError):
        attn.append_kv(q, q, pages, pages, i(1, 2), i(2), i(1))
    with pytest.raises(ValueError):
        attn.fwd_paged(q, pages, pages, i(1, 2), i(2), i(1), 1)


@pytest.mark.parametrize("n_seq,Hkv,keys,clusters", [
    (1, 4, 2048, True), (1, 4, 4096, False), (4, 4, 4096, False), (6, 4, 4096, True),
    (9, 4, 4096, True), (9, 4, 8192, False), (10, 4, 1024, True), (10, 4, 2048, True),
    (14, 4, 2048, True), (20, 4, 1024, True), (75, 4, 1024, True), (75, 4, 2048, False)])
def test_decoding_batches_in_clusters(L, n_seq, Hkv, keys, clusters):
    """Clusters (which need no workspace) where they measured faster: few keys
    a CTA, and a short reach where they leave CTAs idle."""
    assert (attn.fwd_paged_workspace_bytes(n_seq, 1, keys, 4 * Hkv, Hkv, 128) == 0) == clusters
