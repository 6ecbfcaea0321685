"""Workloads of a smaller paged key/value cache: keys and values held in 4
bits (append, read back, attention over them), and eviction by accumulated
attention weight (the weights, and the move of the rows that stay).

Each workload makes its inputs from a seed and computes either the plain form
(elementary torch operations in 32 bits) or, with ``own`` set, the calls a
program makes of this framework.

Shared layouts:

* packed tokens  [H, total, d], sequence b owning rows cu_seqlens[b]..cu_seqlens[b+1];
* 16-bit cache   [n_pages, Hkv, page, d], the page of position p of sequence b
  being block_table[b, p // page];
* 4-bit cache    uint8 [n_pages, Hkv, page, 5 d / 8]: a row is d/2 bytes of codes
  (channel 2i in the low half of byte i), then for each 32 channels the scale s
  and the minimum m in the cache's 16-bit type; a code c stands for m + c s;
* kv_lens[b]     keys of sequence b, its new tokens (the last ones) included;
* weights        float32 [n_pages, Hkv, page], a position's accumulated weight;
* rope table     int64 [2, rot/2]: row 0 the angle of each channel pair per
  position, in units of 2^-64 turns; row 1 the position axis of the pair.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
GROUP = 32  # channels that share a scale and a minimum


# ------------------------------------------------------------------- cases ---

def listed():
    return [
        # one decoding step of a batch into the 4-bit cache: latency of the append
        dict(name="append4 decode s64", op="append4", dtype="bf16", seqs=64, chunks=0, new_max=1,
             kv_max=2048, heads=16, kv_heads=4, dim=128, rot=128, axes=1, interleaved=False,
             page=64, lens=1),
        # prompts of several requests, ragged, 16-token pages, position axes of an image prompt
        dict(name="append4 prompts s12 d64", op="append4", dtype="fp16", seqs=12, chunks=12, new_max=2048,
             kv_max=4096, heads=16, kv_heads=16, dim=64, rot=64, axes=3, interleaved=False,
             page=16, lens=2),
        # one long prompt whole
        dict(name="append4 prompt n16384", op="append4", dtype="bf16", seqs=1, chunks=1, new_max=16384,
             kv_max=16384, heads=16, kv_heads=8, dim=128, rot=128, axes=1, interleaved=False,
             page=64, lens=3),
        # one user's decoding step, a short cache: latency
        dict(name="paged4 decode s1 kv1000", op="paged4", dtype="bf16", seqs=1, chunks=0, new_max=1,
             kv_max=1000, heads=16, kv_heads=4, dim=128, page=16, causal=True, lens=4),
        # a serving batch's decoding step, ragged caches
        dict(name="paged4 decode s64 kv8192", op="paged4", dtype="bf16", seqs=64, chunks=0, new_max=1,
             kv_max=8192, heads=16, kv_heads=4, dim=128, page=64, causal=True, lens=5),
        # few users with very long caches, draft tokens
        dict(name="paged4 drafts s3 kv65536", op="paged4", dtype="fp16", seqs=3, chunks=3, new_max=4,
             kv_max=65536, heads=16, kv_heads=4, dim=64, page=128, causal=True, lens=6),
        # chunked prefill together with decoding requests
        dict(name="paged4 mixed s16 q509 kv4096", op="paged4", dtype="bf16", seqs=16, chunks=4, new_max=509,
             kv_max=4096, heads=16, kv_heads=4, dim=128, page=16, causal=True, lens=7),
        # the last chunk of a long prompt
        dict(name="paged4 prefill q4096 kv16384", op="paged4", dtype="bf16", seqs=1, chunks=1, new_max=4096,
             kv_max=16384, heads=16, kv_heads=8, dim=128, page=64, causal=True, lens=9),
        # weights after a decoding step of a batch
        dict(name="weights decode s64 kv8192", op="weights", dtype="bf16", seqs=64, chunks=0, new_max=1,
             kv_max=8192, heads=16, kv_heads=4, dim=128, page=64, causal=True, bits=16, lens=10),
        # weights that the last tokens of long prompts give the cache, held in 4 bits
        dict(name="weights window s4 q32 kv16384", op="weights", dtype="fp16", seqs=4, chunks=4, new_max=32,
             kv_max=16384, heads=16, kv_heads=8, dim=128, page=32, causal=True, bits=4, lens=11),
        # a batch whose caches are halved
        dict(name="evict s16 kv8192", op="evict", dtype="bf16", seqs=16, chunks=0, new_max=1,
             kv_max=8192, heads=16, kv_heads=4, dim=128, page=64, bits=16, budget=4096, sinks=4,
             recent=256, lens=12),
        # one very long cache in 4 bits, cut to a quarter
        dict(name="evict s1 kv65536 4 bits", op="evict", dtype="fp16", seqs=1, chunks=0, new_max=1,
             kv_max=65536, heads=16, kv_heads=8, dim=64, page=128, bits=4, budget=16384, sinks=16,
             recent=1024, lens=13),
    ]


def _log(rng, lo, hi):
    """A whole number spread over the logarithm of [lo, hi]."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _heads(rng):
    kv = rng.choice([1, 2, 4, 8])
    return kv * rng.choice([1, 2, 3, 4, 7, 8] if kv < 4 else [1, 2, 4]), kv


def draw(rng):
    op = rng.choice(["append4", "append4", "paged4", "paged4", "paged4", "weights", "weights", "evict", "evict"])
    heads, kv = _heads(rng)
    dim = rng.choice([64, 96, 128])
    c = dict(op=op, dtype=rng.choice(["bf16", "fp16"]), heads=heads, kv_heads=kv, dim=dim,
             page=rng.choice([16, 32, 64, 128, 256]), lens=rng.randrange(1, 1 << 20))
    if op == "append4":
        seqs = _log(rng, 1, 128)
        new = rng.choice([1, _log(rng, 2, max(2, 8192 // seqs))])
        return dict(c, seqs=seqs, chunks=0 if new == 1 else rng.randint(1, seqs), new_max=new,
                    kv_max=new + _log(rng, 1, max(1, 65536 // seqs)), rot=rng.choice([dim, dim, dim // 2]),
                    axes=rng.choice([1, 2, 3]), interleaved=rng.random() < 0.4)
    if op == "evict":
        seqs = _log(rng, 1, 64)
        kv_max = _log(rng, 24, min(65536, 98304 // seqs))
        budget = max(8, int(kv_max * rng.uniform(0.1, 0.9)))
        return dict(c, seqs=seqs, chunks=0, new_max=1, kv_max=kv_max, bits=rng.choice([4, 16]),
                    budget=budget, sinks=rng.choice([0, 4, budget // 8]),
                    recent=rng.choice([0, 1, budget // 4, budget // 2]))
    kind = rng.choice(["decode", "decode", "drafts", "chunk"])
    if kind == "chunk":
        seqs = _log(rng, 1, 8)
        new = _log(rng, 17, (2048 if op == "paged4" else 256) // seqs)
        kv_max = new + _log(rng, 1, 16384 // seqs)
    else:
        seqs = _log(rng, 1, 128)
        new = 1 if kind == "decode" else rng.randint(2, 16)
        kv_max = new + _log(rng, 1, min(65536, 262144 // seqs))
    c = dict(c, seqs=seqs, chunks=0 if new == 1 else rng.randint(1, seqs), new_max=new, kv_max=kv_max,
             causal=rng.random() < 0.8)
    return c if op == "paged4" else dict(c, bits=rng.choice([4, 16]))


def _lengths(case):
    """(new tokens, keys) of every sequence, from the case alone."""
    rng = random.Random(case["lens"])
    got = []
    for i in range(case["seqs"]):
        new = 1
        if i < case["chunks"]:
            new = case["new_max"] if i == 0 else rng.randint((case["new_max"] + 1) // 2, case["new_max"])
        keys = case["kv_max"] if i == 0 else rng.randint(max(new, case["kv_max"] // 4), case["kv_max"])
        got.append((new, keys))
    rng.shuffle(got)
    return got


# ------------------------------------------------------------------ inputs ---

def _frequencies(case, dev):
    """Angle per position of each channel pair (radians, 64 bits) and its axis."""
    half = case["rot"] // 2
    inv = 10000.0 ** (-torch.arange(half, dtype=torch.float64, device=dev) / half)
    axis = torch.arange(half, device=dev) * case["axes"] // half
    table = torch.stack([(inv / (2 * math.pi) * 2.0 ** 64).to(torch.int64), axis.to(torch.int64)])
    return inv, axis, table


def _positions(case, n, gen, dev):
    """[axes, n] int32: image and video tokens walk a grid."""
    base = int(torch.randint(0, 64, (1,), generator=gen))
    i = torch.arange(n, device=dev)
    grid = [i // 576, i // 24 % 24, i % 24] if case["axes"] == 3 else [i // 24, i % 24]
    return (torch.stack(grid) + base).to(torch.int32)


def _normal(shape, case, dev, seed, offsets=False):
    """Normal values; with offsets each channel has a mean and a width of its
    own, as keys and values have."""
    g = torch.Generator(device=dev).manual_seed(seed)
    x = torch.randn(shape, generator=g, device=dev, dtype=torch.float32)
    if offsets:
        d = shape[-1]
        x = x * torch.rand(d, generator=g, device=dev).add_(0.5) + torch.randn(d, generator=g, device=dev) / 2
    return x.to(DTYPES[case["dtype"]])


def _paging(case, gen, dev):
    """cu_seqlens, kv_lens, a block table of shuffled pages, and their number."""
    lens = _lengths(case)
    page = case["page"]
    cu = torch.tensor([0] + [n for n, _ in lens]).cumsum(0).to(torch.int32)
    need = [-(-k // page) for _, k in lens]
    n_pages = sum(need) + 3
    order = torch.randperm(n_pages, generator=gen)
    table = torch.zeros(len(lens), max(need), dtype=torch.int32)
    at = 0
    for b, m in enumerate(need):
        table[b, :m] = order[at:at + m]
        at += m
    kv = torch.tensor([k for _, k in lens], dtype=torch.int32)
    return cu.to(dev), kv.to(dev), table.to(dev), n_pages


def _pages(case, n_pages, dev, seed):
    shape = (n_pages, case["kv_heads"], case["page"], case["dim"])
    x = _normal(shape, case, dev, seed, offsets=True)
    return _pack(x) if case.get("bits", 4) == 4 else x


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator().manual_seed(seed)
    s = dict(case=case)
    H, Hkv, d = case["heads"], case["kv_heads"], case["dim"]
    s["cu"], s["kv"], s["blocks"], n_pages = _paging(case, gen, dev)
    s["total"] = total = sum(n for n, _ in _lengths(case))
    s["k_pages"] = _pages(case, n_pages, dev, seed + 2)
    if case["op"] != "weights":
        s["v_pages"] = _pages(case, n_pages, dev, seed + 3)
    if case["op"] == "append4":  # views of one projection [total, heads, d]
        qkv = _normal((total, H + 2 * Hkv, d), case, dev, seed, offsets=True)
        s["q"], s["k"], s["v"] = (t.transpose(0, 1) for t in qkv.split([H, Hkv, Hkv], 1))
        s["pos"] = None if case["axes"] == 1 else _positions(case, total, gen, dev)
        s["inv"], s["axis"], s["table"] = _frequencies(case, dev)
        return s
    if case["op"] in ("weights", "evict"):
        # long tails, and many positions of the same small weight
        g = torch.Generator(device=dev).manual_seed(seed + 4)
        w = torch.rand((n_pages, Hkv, case["page"]), generator=g, device=dev) ** 8 * 64
        s["weights"] = (w * 1024).round() / 1024
    if case["op"] != "evict":
        s["q"] = _normal((H, total, d), case, dev, seed)
    if case["op"] == "weights":
        x = _scores(s)
        m = x.amax(-1)
        s["lse"] = _packed(s, m + (x - m[..., None]).exp().sum(-1).log()).contiguous()
    return s


# ------------------------------------------------------------- plain forms ---

def _pack(x):
    """Rows of the 4-bit cache for 16-bit values x [..., d]."""
    g = x.float().unflatten(-1, (-1, GROUP))
    low = g.amin(-1, keepdim=True)
    scale = ((g.amax(-1, keepdim=True) - low) / 15).to(x.dtype)
    code = ((g - low) / torch.where(scale > 0, scale.float(), math.inf)).round().clamp(max=15)
    code = code.to(torch.uint8).flatten(-2)
    both = torch.cat([scale, low.to(x.dtype)], -1).flatten(-2).contiguous()
    return torch.cat([code[..., ::2] | code[..., 1::2] << 4, both.view(torch.uint8)], -1)


def _unpack(rows, dtype, d):
    """fp32 values that rows of the 4-bit cache stand for."""
    both = rows[..., d // 2:].contiguous().view(dtype).float().unflatten(-1, (-1, 1, 2))
    code = torch.stack([rows[..., :d // 2] & 15, rows[..., :d // 2] >> 4], -1).flatten(-2)
    return (code.float().unflatten(-1, (-1, GROUP)) * both[..., 0] + both[..., 1]).flatten(-2)


def _values(s, name):
    """fp32 [S, Hkv, nk, d] of every sequence's rows."""
    c = s["case"]
    j = torch.arange(c["kv_max"], device=s["kv"].device)
    rows = s[name][s["blocks"].long()[:, j // c["page"]], :, j % c["page"]].transpose(1, 2)
    return _unpack(rows, DTYPES[c["dtype"]], c["dim"]) if c.get("bits", 4) == 4 else rows.float()


def _turn(x, pos, s):
    """x [..., n, d] turned by positions pos [axes, ..., n] (fp32 values, angles
    in 64 bits)."""
    c = s["case"]
    rot, half = c["rot"], c["rot"] // 2
    at = pos.double().movedim(0, -1)[..., s["axis"]] * s["inv"]  # [..., n, half]
    cos, sin = at.cos().float(), at.sin().float()
    x = x.float()
    a, b = (x[..., :rot:2], x[..., 1:rot:2]) if c["interleaved"] else (x[..., :half], x[..., half:rot])
    u, v = a * cos - b * sin, b * cos + a * sin
    turned = torch.stack([u, v], -1).flatten(-2) if c["interleaved"] else torch.cat([u, v], -1)
    return torch.cat([turned, x[..., rot:]], -1)


def _slots(s):
    """(page, row in the page, position) of every new token."""
    cu, kv = s["cu"].long(), s["kv"].long()
    t = torch.arange(s["total"], device=cu.device)
    b = torch.searchsorted(cu, t, right=True) - 1
    p = t - cu[b + 1] + kv[b]
    page = s["case"]["page"]
    return s["blocks"].long()[b, p // page], p % page, p


def _plain_append(s):
    page, row, p = _slots(s)
    pos = p[None] if s["pos"] is None else s["pos"]
    dt, d = s["k"].dtype, s["case"]["dim"]
    s["k_pages"][page, :, row] = _pack(_turn(s["k"], pos[:, None], s).to(dt)).transpose(0, 1)
    s["v_pages"][page, :, row] = _pack(s["v"]).transpose(0, 1)
    k, v = (_unpack(s[n][page, :, row], dt, d).to(dt).transpose(0, 1).contiguous()
            for n in ("k_pages", "v_pages"))
    return dict(q=_turn(s["q"], pos[:, None], s).to(dt), k=k, v=v)


def _seen(s):
    """[S, nq, nk]: which keys a sequence's new token sees."""
    c = s["case"]
    cu, kv = s["cu"].long(), s["kv"].long()
    i = torch.arange(c["new_max"], device=cu.device)
    j = torch.arange(c["kv_max"], device=cu.device)
    last = kv[:, None] - 1
    last = last - (cu[1:] - cu[:-1])[:, None] + 1 + i if c["causal"] else last.expand(-1, c["new_max"])
    return j <= torch.minimum(last, kv[:, None] - 1)[..., None]


def _rows(s):
    """Rows [S, nq] of the packed tokens, and which of them are tokens."""
    cu = s["cu"].long()
    i = torch.arange(s["case"]["new_max"], device=cu.device)
    return (cu[:-1, None] + i).clamp(max=s["total"] - 1), i < (cu[1:] - cu[:-1])[:, None]


def _scores(s):
    """fp32 [S, Hkv, G, nq, nk] scores, -inf where a token does not see the key."""
    c = s["case"]
    H, Hkv, d, nq = c["heads"], c["kv_heads"], c["dim"], c["new_max"]
    S = len(s["kv"])
    q = s["q"].float()[:, _rows(s)[0]].view(Hkv, H // Hkv, S, nq, d).permute(2, 0, 1, 3, 4).reshape(S, Hkv, -1, d)
    x = (q @ _values(s, "k_pages").transpose(2, 3)).view(S, Hkv, H // Hkv, nq, -1) / math.sqrt(d)
    return x.masked_fill(~_seen(s)[:, None, None], -math.inf)


def _packed(s, x):
    """[S, Hkv, G, nq] -> packed [H, total]."""
    return x.permute(0, 3, 1, 2)[_rows(s)[1]].view(s["total"], -1).t()


def _plain_paged(s):
    c = s["case"]
    H, Hkv, d, nq, nk = c["heads"], c["kv_heads"], c["dim"], c["new_max"], c["kv_max"]
    x = _scores(s)
    m = x.amax(-1, keepdim=True)
    x = (x - m).exp()
    l = x.sum(-1, keepdim=True)
    o = (x.view(len(s["kv"]), Hkv, -1, nk) @ _values(s, "v_pages")).view(-1, Hkv, H // Hkv, nq, d) / l
    o = o.permute(0, 3, 1, 2, 4)[_rows(s)[1]].view(s["total"], H, d).transpose(0, 1)
    return o.to(s["q"].dtype).contiguous(), _packed(s, (m + l.log())[..., 0]).contiguous()


def _plain_weights(s):
    c = s["case"]
    rows, live = _rows(s)
    H, Hkv = c["heads"], c["kv_heads"]
    S = len(s["kv"])
    lse = s["lse"][:, rows].view(Hkv, H // Hkv, S, c["new_max"]).permute(2, 0, 1, 3)
    p = (_scores(s) - lse[..., None]).exp().masked_fill(~live[:, None, None, :, None], 0)
    p = p.sum((2, 3))  # [S, Hkv, nk]
    j = torch.arange(c["kv_max"], device=p.device)
    b, at = (j < s["kv"][:, None]).nonzero(as_tuple=True)
    page, row = s["blocks"].long()[b, at // c["page"]], at % c["page"]
    older = at < (s["kv"] - (s["cu"][1:] - s["cu"][:-1])).long()[b]
    s["weights"][page, :, row] = s["weights"][page, :, row] * older[:, None] + p[b, :, at]
    return s["weights"]


def _plain_evict(s):
    c = s["case"]
    Hkv, page, budget = c["kv_heads"], c["page"], c["budget"]
    kv, blocks = s["kv"].long()[:, None], s["blocks"].long()
    j = torch.arange(c["kv_max"], device=kv.device)
    w = s["weights"][blocks[:, j // page], :, j % page].transpose(1, 2)  # [S, Hkv, nk]
    rank = torch.where((j < c["sinks"]) | (j >= kv - c["recent"]), math.inf, 0.0)
    rank = torch.where(j < kv, rank, -1.0)[:, None] + w * (j < kv)[:, None]
    order = rank.sort(dim=-1, descending=True, stable=True).indices[..., :budget]
    n = torch.minimum(kv, torch.tensor(budget, device=kv.device))
    i = torch.arange(order.shape[-1], device=kv.device)
    kept = order.masked_fill((i >= n)[:, None], c["kv_max"]).sort(dim=-1).values
    out = torch.full((len(kv), Hkv, budget), -1, dtype=torch.int32, device=kv.device)
    b, h, i = (i < n)[:, None].expand_as(kept).nonzero(as_tuple=True)
    at = kept[b, h, i]
    out[b, h, i] = at.to(torch.int32)
    for t in (s["k_pages"], s["v_pages"], s["weights"]):
        t[blocks[b, i // page], h, i % page] = t[blocks[b, at // page], h, at % page]
    return dict(kept=out, lens=n[:, 0].to(torch.int32), k=s["k_pages"], v=s["v_pages"], weights=s["weights"])


def run(s):
    c = s["case"]
    if own:
        import exact_attention_75_gb300 as attn
        if c["op"] == "append4":
            q = attn.append_kv4(s["k"], s["v"], s["k_pages"], s["v_pages"], s["blocks"], s["cu"], s["kv"],
                                table=s["table"], positions=s["pos"], interleaved=c["interleaved"], q=s["q"])
            k, v = attn.read_kv4(s["k_pages"], s["v_pages"], s["blocks"], s["cu"], s["kv"], s["total"],
                                 dtype=s["k"].dtype)
            return dict(q=q, k=k, v=v)
        if c["op"] == "paged4":
            return attn.fwd_paged4(s["q"], s["k_pages"], s["v_pages"], s["blocks"], s["cu"], s["kv"],
                                   c["new_max"], causal=c["causal"])
        if c["op"] == "weights":
            return attn.kv_weights(s["q"], s["k_pages"], s["blocks"], s["cu"], s["kv"], s["lse"], s["weights"],
                                   c["new_max"], causal=c["causal"])
        kept, lens = attn.evict_kv(s["k_pages"], s["v_pages"], s["weights"], s["blocks"], s["kv"], c["budget"],
                                   sinks=c["sinks"], recent=c["recent"])
        return dict(kept=kept, lens=lens, k=s["k_pages"], v=s["v_pages"], weights=s["weights"])
    return {"append4": _plain_append, "paged4": _plain_paged, "weights": _plain_weights,
            "evict": _plain_evict}[c["op"]](s)


def work(case):
    H, Hkv, d = case["heads"], case["kv_heads"], case["dim"]
    lens = _lengths(case)
    n, keys = sum(a for a, _ in lens), sum(k for _, k in lens)
    pages = sum(-(-k // case["page"]) for _, k in lens)
    row = 5 * d // 8 if case.get("bits", 4) == 4 else 2 * d
    if case["op"] == "append4":
        touched = sum((k - 1) // case["page"] - (k - a) // case["page"] + 1 for a, k in lens)
        pos = 0 if case["axes"] == 1 else 4 * case["axes"]
        # tokens read, queries, rows of the cache and what they stand for written
        return dict(bytes=n * (H * d * 4 + Hkv * (8 * d + 2 * row) + pos) + 4 * (touched + 2 * len(lens)),
                    flops=n * (H + Hkv) * case["rot"] * 3 + n * Hkv * d * 12)
    if case["op"] == "evict":
        kept = sum(min(k, case["budget"]) if k > case["budget"] else 0 for _, k in lens)
        cut = sum(k for _, k in lens if k > case["budget"])
        return dict(bytes=Hkv * (kept * (4 * row + 8) + 4 * cut + 4 * case["budget"] * len(lens)) + 4 * pages,
                    flops=Hkv * cut)
    pairs = sum(a * (k - a) + a * (a + 1) // 2 if case["causal"] else a * k for a, k in lens)
    if case["op"] == "weights":
        return dict(bytes=n * H * (2 * d + 4) + keys * Hkv * (row + 8) + 4 * (pages + 2 * len(lens)),
                    flops=2 * d * H * pairs)
    return dict(bytes=n * H * (4 * d + 4) + 2 * keys * Hkv * row + 4 * (pages + 2 * len(lens)),
                flops=4 * d * H * pairs)


# ---------------------------------------------------- by definition, 64 bits ---

def _rotation(case, pos):
    """[n, d] values of cos and sin by channel, from the definition: channel
    pair p turns by pos[axis of p] * 10000^(-2p/rot)."""
    half, d = case["rot"] // 2, case["dim"]
    cos = torch.ones(pos.shape[-1], d, dtype=torch.float64, device=pos.device)
    sin = torch.zeros_like(cos)
    for p in range(half):
        angle = pos[p * case["axes"] // half].double() / 10000.0 ** (2.0 * p / case["rot"])
        for ch, sign in ((2 * p, -1), (2 * p + 1, 1)) if case["interleaved"] else ((p, -1), (p + half, 1)):
            cos[:, ch] = angle.cos()
            sin[:, ch] = sign * angle.sin()
    return cos, sin


def _exact_turn(case, x, pos):
    cos, sin = _rotation(case, pos)
    half, rot = case["rot"] // 2, case["rot"]
    at = torch.arange(case["dim"], device=x.device)
    if case["interleaved"]:
        at[:rot] = at[:rot] ^ 1
    else:
        at[:rot] = (at[:rot] + half) % rot
    return x.double() * cos + sin * x.double()[..., at]


def _exact_kept(x):
    """What 16-bit values x stand for after 4 bits."""
    out = torch.empty(x.shape, dtype=torch.float64, device=x.device)
    for c in range(0, x.shape[-1], GROUP):
        g = x[..., c:c + GROUP].double()
        m = g.min(-1, keepdim=True).values
        step = ((g.max(-1, keepdim=True).values - m) / 15).to(x.dtype).double()
        n = torch.where(step > 0, (g - m) / step, 0).round().clamp(max=15)
        out[..., c:c + GROUP] = m + n * step
    return out


def _exact_rows(case, pages):
    """[slots, d] values of one head's rows [slots, bytes or d]."""
    if case.get("bits", 4) == 16:
        return pages.double()
    d = case["dim"]
    ch = torch.arange(d, device=pages.device)
    code = pages.int()[:, ch // 2] >> ch % 2 * 4 & 15
    par = pages[:, d // 2:].contiguous().view(DTYPES[case["dtype"]]).double()
    return par[:, ch // GROUP * 2 + 1] + code * par[:, ch // GROUP * 2]


def _exact_evict(case, s):
    budget, page = case["budget"], case["page"]
    kv = s["kv"].tolist()
    kept = torch.full((len(kv), case["kv_heads"], budget), -1, dtype=torch.int32)
    k, v, w = s["k_pages"], s["v_pages"], s["weights"]
    old = [t.clone() for t in (k, v, w)]
    for b, n in enumerate(kv):
        slot = s["blocks"][b].long().repeat_interleave(page)[:n], torch.arange(n, device=w.device) % page
        for h in range(case["kv_heads"]):
            keep = list(range(n))
            if n > budget:
                mid = range(case["sinks"], n - case["recent"])
                score = w[slot[0], h, slot[1]].tolist()
                best = sorted(mid, key=lambda j: (-score[j], j))[:budget - case["sinks"] - case["recent"]]
                keep = sorted([*range(case["sinks"]), *best, *range(n - case["recent"], n)])
            kept[b, h, :len(keep)] = torch.tensor(keep, dtype=torch.int32)
            at = torch.tensor(keep, device=w.device)
            for t, o in zip((k, v, w), old):
                t[slot[0][:len(keep)], h, slot[1][:len(keep)]] = o[slot[0][at], h, slot[1][at]]
    out = dict(kept=kept, lens=torch.tensor([min(n, budget) for n in kv], dtype=torch.int32))
    whole = case["bits"] == 4
    return dict(out, k=k if whole else k.double(), v=v if whole else v.double(), weights=w.double())


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "evict":
        return _exact_evict(case, s)
    cu, kv, page = s["cu"].tolist(), s["kv"].tolist(), case["page"]
    if case["op"] == "append4":
        seq = [torch.arange(kv[b] - cu[b + 1] + cu[b], kv[b], device=s["cu"].device) for b in range(len(kv))]
        pos = torch.cat(seq)[None] if s["pos"] is None else s["pos"]
        dt = s["k"].dtype
        return dict(q=_exact_turn(case, s["q"], pos), k=_exact_kept(_exact_turn(case, s["k"], pos).to(dt)),
                    v=_exact_kept(s["v"]))
    H, total = case["heads"], s["total"]
    group = H // case["kv_heads"]
    o = torch.empty(H, total, case["dim"], dtype=torch.float64, device=s["q"].device)
    lse = torch.empty(H, total, dtype=torch.float64, device=s["q"].device)
    weights = s["weights"].double() if case["op"] == "weights" else None
    for b in range(len(kv)):
        a, e = cu[b], cu[b + 1]
        pages = s["blocks"][b, :-(-kv[b] // page)].long()
        at = torch.arange(kv[b], device=pages.device)
        at = pages[at // page], at % page
        for h in range(H):
            k = _exact_rows(case, s["k_pages"][pages, h // group].flatten(0, 1)[:kv[b]])
            x = s["q"][h, a:e].double() @ k.t() * case["dim"] ** -0.5
            if case["causal"]:
                x += torch.full_like(x, -math.inf).triu(kv[b] - (e - a) + 1)
            if weights is not None:
                got = torch.exp(x - s["lse"][h, a:e].double()[:, None]).sum(0)
                if h % group == 0:
                    weights[at[0][kv[b] - (e - a):], h // group, at[1][kv[b] - (e - a):]] = 0
                weights[at[0], h // group, at[1]] += got
                continue
            v = _exact_rows(case, s["v_pages"][pages, h // group].flatten(0, 1)[:kv[b]])
            lse[h, a:e] = torch.logsumexp(x, -1)
            o[h, a:e] = torch.softmax(x, -1) @ v
    return weights if weights is not None else (o, lse)
