"""Calls over a 4-bit cache, and eviction, whose inputs the stream has only just
written: every kernel here may start before the work ahead of it has finished, and reads
lengths, pages, tokens, weights and caches that this work writes.  Bits are compared with
those of calls on idle streams."""
import pytest
import torch

import test_paged_gpu as paged
import test_retain_gpu as retain
from test_kv4_gpu import normal, pack4
from test_paged_gpu import widen

pytestmark = pytest.mark.gpu

HQ, HKV, D, PAGE = 4, 2, 64, 16


def rotate(x):
    """The rows of x as a kernel's output just before the call."""
    return x * 2.0 * 0.5


def bits(t):
    return t.contiguous().view(torch.uint8)


def alternate(attn, xs, written, step):
    """step(x) -> tensors, on each of xs by itself; then 16 times in a row on one set of
    tensors that get xs[0]'s and xs[1]'s contents (of the names in `written`) by copies,
    those from the host among them, right before."""
    want = []
    for x in xs:
        torch.cuda.synchronize()
        want.append([t.clone() for t in step({k: v.clone() if torch.is_tensor(v) else v for k, v in x.items()})])
    torch.cuda.synchronize()
    assert attn.poll_status() == (0, 0)
    hold = {k: v.clone() if torch.is_tensor(v) else v for k, v in xs[0].items()}
    host = [{k: x[k].cpu().pin_memory() for k in ("cu", "kv", "table")} for x in xs]
    big = torch.randn(64 << 20, device="cuda")
    side, got = torch.cuda.Stream(), []
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for i in (0, 1) * 8:
            big.mul_(1.0)  # keeps the stream busy
            for k in ("cu", "kv", "table"):
                hold[k].copy_(host[i][k], non_blocking=True)
            for k in written:
                hold[k].copy_(xs[i][k])
            out = step(hold)
            got.append((i, [t.clone() for t in out]))
            for t in out:  # the memory goes back for the next call's outputs
                if all(t is not v for v in hold.values()):
                    t.zero_()
            del out
    torch.cuda.synchronize()
    assert attn.poll_status() == (0, 0)
    for i, out in got:
        assert all(torch.equal(bits(a), bits(b)) for a, b in zip(out, want[i]))


BATCHES = [([(1, 60), (1, 300)], 16), ([(1, 60), (1, 300)] * 6, 5000), ([(40, 60), (1, 300)], 16)]


def batches(lens, reach, n_bits=4):
    xs = []
    for s in (73, 79):
        # a second batch of the same sizes and other lengths
        x = widen(paged.make([(n, k - 7 * (s == 79)) for n, k in lens], HQ, HKV, D, PAGE, "bf16", seed=s), reach)
        if n_bits == 4:
            x["k"], x["v"] = pack4(x["k"]), pack4(x["v"])
        total = x["q"].shape[1]
        x["nk"], x["nv"] = normal((HKV, total, D), torch.bfloat16, s), normal((HKV, total, D), torch.bfloat16, s + 1)
        xs.append(x)
    pages, width = max(x["k"].shape[0] for x in xs), max(x["table"].shape[1] for x in xs)
    for x in xs:  # one size of tensors
        for n in ("k", "v"):
            x[n] = torch.cat([x[n], x[n][:1].expand(pages - x[n].shape[0], *x[n].shape[1:])])
        t = x["table"]
        x["table"] = torch.cat([t, t.new_full((t.shape[0], width - t.shape[1]), 0x7FFFFFFF)], 1)
    return xs


@pytest.mark.parametrize("lens,reach", BATCHES)
def test_append_read_and_attention(attn_lib, lens, reach):
    table = attn_lib.rope_table(D)

    def step(x):
        args = x["table"], x["cu"], x["kv"]
        q = attn_lib.append_kv4(rotate(x["nk"]), rotate(x["nv"]), x["k"], x["v"], *args, table=table, q=rotate(x["q"]))
        o, lse = attn_lib.fwd_paged4(q, x["k"], x["v"], *args, x["max_q"], causal=True)
        k, v = attn_lib.read_kv4(x["k"], x["v"], *args, q.shape[1], dtype=torch.bfloat16)
        return q, o, lse, k, v, x["k"], x["v"]

    alternate(attn_lib, batches(lens, reach), ("k", "v", "nk", "nv", "q"), step)


@pytest.mark.parametrize("lens,reach", BATCHES)
@pytest.mark.parametrize("call", ["attention", "read"])
def test_pages_written_just_before(attn_lib, lens, reach, call):
    """The cache itself comes from copies right before the call."""

    def step(x):
        args = x["k"], x["v"], x["table"], x["cu"], x["kv"]
        if call == "read":
            return attn_lib.read_kv4(*args, x["q"].shape[1], dtype=torch.bfloat16)
        return attn_lib.fwd_paged4(x["q"], *args, x["max_q"], causal=True)

    alternate(attn_lib, batches(lens, reach), ("q", "v", "k"), step)


@pytest.mark.parametrize("n_bits", [4, 16])
@pytest.mark.parametrize("lens,reach", BATCHES)
def test_weights(attn_lib, n_bits, lens, reach):
    xs = []
    for x in batches(lens, reach, n_bits):
        call = attn_lib.fwd_paged4 if n_bits == 4 else attn_lib.fwd_paged
        _, x["lse"] = call(x["q"], x["k"], x["v"], x["table"], x["cu"], x["kv"], x["max_q"], causal=True)
        x["w"] = torch.rand(x["k"].shape[:3], generator=torch.Generator().manual_seed(5)).cuda()
        xs.append(x)

    def step(x):
        return [attn_lib.kv_weights(rotate(x["q"]), x["k"], x["table"], x["cu"], x["kv"], x["lse"] * 1.0, x["w"],
                                    x["max_q"], causal=True)]

    alternate(attn_lib, xs, ("k", "lse", "q", "w"), step)


@pytest.mark.parametrize("n_bits", [4, 16])
@pytest.mark.parametrize("lens", [[300, 500, 90], [400, 120, 333] * 30])
def test_eviction(attn_lib, n_bits, lens):
    """Eviction, and what runs right behind it on what it has moved."""
    xs = []
    for s in (21, 22):
        x = retain.cache(lens, HKV, D, PAGE, n_bits, seed=s)
        x["kv"] = x["kv"] - 5 * (s - 21)
        x["cu"] = torch.zeros(1, dtype=torch.int32, device="cuda")  # not of the call
        xs.append(x)

    def step(x):
        kept, lens = attn_lib.evict_kv(x["k"], x["v"], x["w"], x["table"], x["kv"], 128, sinks=4, recent=30)
        out = [kept, lens, x["k"], x["v"], x["w"]]
        if n_bits == 4:
            cu = torch.cat([lens.new_zeros(1), lens.cumsum(0, dtype=torch.int32)])
            room = 128 * len(lens)
            ks = [torch.zeros(HKV, room, D, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
            out += attn_lib.read_kv4(x["k"], x["v"], x["table"], cu, lens, room, out_k=ks[0], out_v=ks[1])
        return out

    alternate(attn_lib, xs, ("v", "k", "w"), step)


@pytest.mark.parametrize("lens,reach", BATCHES)
def test_captured_step_with_weights_and_eviction(attn_lib, lens, reach):
    """Append, attention, weights and eviction in one graph, replayed on other lengths,
    pages and tokens: the bits of the calls by themselves."""
    rope = attn_lib.rope_table(D)
    xs = batches(lens, reach)
    for i, x in enumerate(xs):
        x["w"] = torch.rand(x["k"].shape[:3], generator=torch.Generator().manual_seed(i)).cuda()
    keys = xs[0]["table"].shape[1] * PAGE
    room = attn_lib.fwd_paged_workspace_bytes(len(lens), xs[0]["max_q"], keys, HQ, HKV, D)
    ws = torch.empty(max(1, room), dtype=torch.uint8, device="cuda")

    def step(x):
        args = x["table"], x["cu"], x["kv"]
        q = attn_lib.append_kv4(x["nk"], x["nv"], x["k"], x["v"], *args, table=rope, q=x["q"])
        o, lse = attn_lib.fwd_paged4(q, x["k"], x["v"], *args, x["max_q"], causal=True, workspace=ws)
        attn_lib.kv_weights(q, x["k"], *args, lse, x["w"], x["max_q"], causal=True)
        kept, new = attn_lib.evict_kv(x["k"], x["v"], x["w"], x["table"], x["kv"], 48, sinks=2, recent=8)
        return q, o, lse, kept, new, x["k"], x["v"], x["w"]

    copy = lambda x: {k: v.clone() if torch.is_tensor(v) else v for k, v in x.items()}  # noqa: E731
    want = [[t.clone() for t in step(copy(x))] for x in xs]
    hold, side, graph = copy(xs[0]), torch.cuda.Stream(), torch.cuda.CUDAGraph()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=side):
        out = step(hold)
    for i in (0, 1, 1, 0):
        for n, t in xs[i].items():
            if torch.is_tensor(t):
                hold[n].copy_(t)
        graph.replay()
        assert all(torch.equal(bits(a), bits(b)) for a, b in zip(out, want[i]))
    assert want[0][4].max() == 48
    assert attn_lib.poll_status() == (0, 0)
