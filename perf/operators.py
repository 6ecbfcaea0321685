"""Workloads of the serving and position operators: rotary positions (forward
and backward), appending to a paged key/value cache, and attention of new
tokens over such a cache.

Each workload makes its inputs from a seed and computes either the plain form
(elementary torch operations in 32 or 64 bits) or, with ``own`` set, the call
a program makes of this framework.

Shared layouts:

* packed tokens  [H, total, d], sequence b owning rows cu_seqlens[b]..cu_seqlens[b+1];
* paged cache    [n_pages, Hkv, page, d], the page of position p of sequence b
  being block_table[b, p // page];
* kv_lens[b]     keys of sequence b, its new tokens (the last ones) included;
* rope table     int64 [2, rot/2]: row 0 the angle of each channel pair per
  position, in units of 2^-64 turns; row 1 the position axis of the pair.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


# ------------------------------------------------------------------- cases ---

def listed():
    return [
        # training step of a text model: q and k of a fused projection, 8192 tokens
        dict(name="rope train b2 n8192 d128", op="rope", dtype="bf16", batch=2, heads=16, kv_heads=16,
             tokens=8192, dim=128, rot=128, axes=1, interleaved=False, fused=True, far=0),
        # its backward pass on a video model: time, height and width axes, grouped heads
        dict(name="rope bwd b2 n8192 3 axes", op="rope_bwd", dtype="bf16", batch=2, heads=16, kv_heads=4,
             tokens=8192, dim=128, rot=128, axes=3, interleaved=False, fused=False, far=0),
        # one image of an odd token count, partial rotation, pairs of neighbours
        dict(name="rope image n577 d64", op="rope", dtype="fp16", batch=1, heads=16, kv_heads=16,
             tokens=577, dim=64, rot=32, axes=2, interleaved=True, fused=True, far=0),
        # one decoding step of a batch: latency of the append
        dict(name="append decode s64", op="append", dtype="bf16", seqs=64, chunks=0, new_max=1,
             kv_max=8192, heads=16, kv_heads=4, dim=128, rot=128, axes=1, interleaved=False,
             page=64, far=0, lens=1),
        # prompts of several requests, ragged, 16-token pages, position axes of an image prompt
        dict(name="append prompts s12 d64", op="append", dtype="fp16", seqs=12, chunks=12, new_max=2048,
             kv_max=4096, heads=16, kv_heads=16, dim=64, rot=64, axes=3, interleaved=False,
             page=16, far=0, lens=2),
        # one long prompt whole
        dict(name="append prompt n16384", op="append", dtype="bf16", seqs=1, chunks=1, new_max=16384,
             kv_max=16384, heads=16, kv_heads=8, dim=128, rot=128, axes=1, interleaved=False,
             page=64, far=0, lens=3),
        # one user's decoding step, a short cache: latency
        dict(name="paged decode s1 kv1000", op="paged", dtype="bf16", seqs=1, chunks=0, new_max=1,
             kv_max=1000, heads=16, kv_heads=4, dim=128, page=16, causal=True, lens=4),
        # a serving batch's decoding step, ragged caches
        dict(name="paged decode s64 kv8192", op="paged", dtype="bf16", seqs=64, chunks=0, new_max=1,
             kv_max=8192, heads=16, kv_heads=4, dim=128, page=64, causal=True, lens=5),
        # few users with very long caches, draft tokens
        dict(name="paged drafts s3 kv65536", op="paged", dtype="fp16", seqs=3, chunks=3, new_max=4,
             kv_max=65536, heads=16, kv_heads=4, dim=64, page=128, causal=True, lens=6),
        # chunked prefill together with decoding requests
        dict(name="paged mixed s16 q512 kv4096", op="paged", dtype="bf16", seqs=16, chunks=4, new_max=509,
             kv_max=4096, heads=16, kv_heads=4, dim=128, page=16, causal=True, lens=7),
        # a chunk of a few hundred tokens against a long cache
        dict(name="paged chunk s2 q256 kv16384", op="paged", dtype="bf16", seqs=2, chunks=2, new_max=256,
             kv_max=16384, heads=16, kv_heads=16, dim=96, page=32, causal=True, lens=8),
        # the last chunk of a long prompt
        dict(name="paged prefill q4096 kv16384", op="paged", dtype="bf16", seqs=1, chunks=1, new_max=4096,
             kv_max=16384, heads=16, kv_heads=8, dim=128, page=64, causal=True, lens=9),
    ]


def _log(rng, lo, hi):
    """A whole number spread over the logarithm of [lo, hi]."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _heads(rng):
    kv = rng.choice([1, 2, 4, 8])
    return kv * rng.choice([1, 2, 3, 4, 7, 8] if kv < 4 else [1, 2, 4]), kv


def draw(rng):
    op = rng.choice(["rope", "rope_bwd", "append", "append", "paged", "paged", "paged", "paged"])
    heads, kv = _heads(rng)
    dtype = rng.choice(["bf16", "fp16"])
    dim = rng.choice([64, 96, 128])
    rot = rng.choice([dim, dim, dim // 2])
    lens = rng.randrange(1, 1 << 20)
    page = rng.choice([16, 32, 64, 128, 256])
    turn = dict(rot=rot, axes=rng.choice([1, 2, 3]), interleaved=rng.random() < 0.4,
                far=rng.choice([0, 0, 100000, 1 << 20]))
    if op in ("rope", "rope_bwd"):
        tokens = _log(rng, 1, 16384)
        batch = max(1, min(4, 16384 // tokens))
        return dict(op=op, dtype=dtype, batch=rng.randint(1, batch), heads=heads, kv_heads=kv,
                    tokens=tokens, dim=dim, fused=rng.random() < 0.5, **turn)
    if op == "append":
        seqs = _log(rng, 1, 128)
        new = rng.choice([1, _log(rng, 2, max(2, 8192 // seqs))])
        return dict(op=op, dtype=dtype, seqs=seqs, chunks=0 if new == 1 else rng.randint(1, seqs),
                    new_max=new, kv_max=new + _log(rng, 1, max(1, 65536 // seqs)), heads=heads,
                    kv_heads=kv, dim=dim, page=page, lens=lens, **turn)
    kind = rng.choice(["decode", "decode", "drafts", "chunk"])
    if kind == "chunk":
        seqs = _log(rng, 1, 8)
        new = _log(rng, 17, 2048 // seqs)
        kv_max = new + _log(rng, 1, 16384 // seqs)
    else:
        seqs = _log(rng, 1, 128)
        new = 1 if kind == "decode" else rng.randint(2, 16)
        kv_max = new + _log(rng, 1, min(65536, 262144 // seqs))
    return dict(op=op, dtype=dtype, seqs=seqs, chunks=0 if new == 1 else rng.randint(1, seqs),
                new_max=new, kv_max=kv_max, heads=heads, kv_heads=kv, dim=dim, page=page,
                causal=rng.random() < 0.8, lens=lens)


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
    """Angle per position of each channel pair (radians, 64 bits) and its axis:
    with several axes the first pairs turn with time, the next with height,
    the last with width."""
    half = case["rot"] // 2
    inv = 10000.0 ** (-torch.arange(half, dtype=torch.float64, device=dev) / half)
    axis = torch.arange(half, device=dev) * case["axes"] // half
    table = torch.stack([(inv / (2 * math.pi) * 2.0 ** 64).to(torch.int64), axis.to(torch.int64)])
    return inv, axis, table


def _positions(case, n, gen, dev):
    """[axes, n] int32: text counts up; image and video tokens walk a grid."""
    base = int(torch.randint(0, 64, (1,), generator=gen)) + case["far"]
    i = torch.arange(n, device=dev)
    if case["axes"] == 1:
        return (i + base).to(torch.int32)[None]
    grid = [i // 576, i // 24 % 24, i % 24] if case["axes"] == 3 else [i // 24, i % 24]
    return (torch.stack(grid) + base).to(torch.int32)


def _normal(shape, case, dev, seed):
    g = torch.Generator(device=dev).manual_seed(seed)
    return torch.randn(shape, generator=g, device=dev, dtype=torch.float32).to(DTYPES[case["dtype"]])


def _paging(case, gen, dev):
    """cu_seqlens, kv_lens, a block table of shuffled pages, and their number."""
    lens = _lengths(case)
    page = case["page"]
    cu = torch.tensor([0] + [n for n, _ in lens]).cumsum(0).to(torch.int32)
    need = [-(-k // page) for _, k in lens]
    width = max(need)
    n_pages = sum(need) + 3
    order = torch.randperm(n_pages, generator=gen)
    table = torch.zeros(len(lens), width, dtype=torch.int32)
    at = 0
    for b, m in enumerate(need):
        table[b, :m] = order[at:at + m]
        at += m
    kv = torch.tensor([k for _, k in lens], dtype=torch.int32)
    return cu.to(dev), kv.to(dev), table.to(dev), n_pages


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator().manual_seed(seed)
    s = dict(case=case)
    H, Hkv, d = case["heads"], case["kv_heads"], case["dim"]
    if case["op"] in ("rope", "rope_bwd"):
        B, N = case["batch"], case["tokens"]
        if case["fused"]:  # views of one projection [B, N, heads, d]
            qkv = _normal((B, N, H + 2 * Hkv, d), case, dev, seed)
            s["q"], s["k"] = qkv[:, :, :H].transpose(1, 2), qkv[:, :, H:H + Hkv].transpose(1, 2)
        else:
            s["q"], s["k"] = _normal((B, H, N, d), case, dev, seed), _normal((B, Hkv, N, d), case, dev, seed + 1)
        s["pos"] = torch.stack([_positions(case, N, gen, dev) for _ in range(B)], 1).contiguous()
        s["inv"], s["axis"], s["table"] = _frequencies(case, dev)
        return s
    s["cu"], s["kv"], s["blocks"], n_pages = _paging(case, gen, dev)
    total = sum(n for n, _ in _lengths(case))
    s["k_pages"] = _normal((n_pages, Hkv, case["page"], d), case, dev, seed + 2)
    s["v_pages"] = _normal((n_pages, Hkv, case["page"], d), case, dev, seed + 3)
    if case["op"] == "append":  # views of one projection [total, heads, d]
        qkv = _normal((total, H + 2 * Hkv, d), case, dev, seed)
        s["q"], s["k"], s["v"] = (t.transpose(0, 1) for t in qkv.split([H, Hkv, Hkv], 1))
        s["pos"] = None if case["axes"] == 1 else _positions(case, total, gen, dev)
        s["inv"], s["axis"], s["table"] = _frequencies(case, dev)
        return s
    s["q"] = _normal((H, total, d), case, dev, seed)
    return s


# ------------------------------------------------------------- plain forms ---

def _turn(x, pos, s, back):
    """x [..., n, d] turned by positions pos [axes, ..., n] (fp32 values, angles
    in 64 bits), or turned back."""
    c = s["case"]
    rot, half = c["rot"], c["rot"] // 2
    at = pos.double().movedim(0, -1)[..., s["axis"]] * s["inv"]  # [..., n, half]
    cos, sin = at.cos().float(), (-at.sin() if back else at.sin()).float()
    x = x.float()
    a, b = (x[..., :rot:2], x[..., 1:rot:2]) if c["interleaved"] else (x[..., :half], x[..., half:rot])
    u, v = a * cos - b * sin, b * cos + a * sin
    turned = torch.stack([u, v], -1).flatten(-2) if c["interleaved"] else torch.cat([u, v], -1)
    return torch.cat([turned, x[..., rot:]], -1)


def _slots(s):
    """(page, row in the page, position) of every new token."""
    cu, kv = s["cu"].long(), s["kv"].long()
    t = torch.arange(s["q"].shape[1], device=cu.device)
    b = torch.searchsorted(cu, t, right=True) - 1
    p = t - cu[b + 1] + kv[b]
    page = s["case"]["page"]
    return s["blocks"].long()[b, p // page], p % page, p


def _plain_append(s):
    page, row, p = _slots(s)
    pos = p[None] if s["pos"] is None else s["pos"]
    dt = s["k"].dtype
    s["k_pages"][page, :, row] = _turn(s["k"], pos[:, None], s, False).to(dt).transpose(0, 1)
    s["v_pages"][page, :, row] = s["v"].transpose(0, 1)
    return dict(q=_turn(s["q"], pos[:, None], s, False).to(dt), k=s["k_pages"], v=s["v_pages"])


def _plain_paged(s):
    c = s["case"]
    H, Hkv, d = c["heads"], c["kv_heads"], c["dim"]
    cu, kv = s["cu"].long(), s["kv"].long()
    S, total = len(kv), s["q"].shape[1]
    nq, nk = c["new_max"], c["kv_max"]
    i = torch.arange(nq, device=cu.device)
    j = torch.arange(nk, device=cu.device)
    new = cu[1:] - cu[:-1]
    rows = (cu[:-1, None] + i).clamp(max=total - 1)  # [S, nq]
    q = s["q"].float()[:, rows].view(Hkv, H // Hkv, S, nq, d).permute(2, 0, 1, 3, 4).reshape(S, Hkv, -1, d)
    at = s["blocks"].long()[:, j // c["page"]]  # [S, nk]
    k = s["k_pages"][at, :, j % c["page"]].float().transpose(1, 2)  # [S, Hkv, nk, d]
    v = s["v_pages"][at, :, j % c["page"]].float().transpose(1, 2)
    last = kv[:, None] - 1
    last = last - new[:, None] + 1 + i if c["causal"] else last.expand(S, nq)
    seen = j <= torch.minimum(last, kv[:, None] - 1)[..., None]  # [S, nq, nk]
    x = (q @ k.transpose(2, 3)).view(S, Hkv, H // Hkv, nq, nk) / math.sqrt(d)
    x = x.masked_fill(~seen[:, None, None], -math.inf)
    m = x.amax(-1, keepdim=True)
    x = (x - m).exp()
    l = x.sum(-1, keepdim=True)
    o = (x.view(S, Hkv, -1, nk) @ v).view(S, Hkv, H // Hkv, nq, d) / l
    lse = (m + l.log())[..., 0]
    live = i < new[:, None]  # [S, nq]; in packed order
    o = o.permute(0, 3, 1, 2, 4)[live].view(total, H, d).transpose(0, 1)
    lse = lse.permute(0, 3, 1, 2)[live].view(total, H).t()
    return o.to(s["q"].dtype).contiguous(), lse.contiguous()


def run(s):
    c = s["case"]
    if own:
        import exact_attention_75_gb300 as attn
        if c["op"] == "rope":
            return attn.rope(s["q"], s["k"], s["pos"], s["table"], interleaved=c["interleaved"])
        if c["op"] == "rope_bwd":
            return attn.rope_bwd(s["q"], s["k"], s["pos"], s["table"], interleaved=c["interleaved"])
        if c["op"] == "append":
            q = attn.append_kv(s["k"], s["v"], s["k_pages"], s["v_pages"], s["blocks"], s["cu"], s["kv"],
                               table=s["table"], positions=s["pos"], interleaved=c["interleaved"], q=s["q"])
            return dict(q=q, k=s["k_pages"], v=s["v_pages"])
        return attn.fwd_paged(s["q"], s["k_pages"], s["v_pages"], s["blocks"], s["cu"], s["kv"],
                              c["new_max"], causal=c["causal"])
    if c["op"] in ("rope", "rope_bwd"):
        back = c["op"] == "rope_bwd"
        return tuple(_turn(s[n], s["pos"][:, :, None], s, back).to(s[n].dtype) for n in ("q", "k"))
    return _plain_append(s) if c["op"] == "append" else _plain_paged(s)


def work(case):
    H, Hkv, d = case["heads"], case["kv_heads"], case["dim"]
    if case["op"] in ("rope", "rope_bwd"):
        n = case["batch"] * case["tokens"]
        return dict(bytes=n * ((H + Hkv) * d * 4 + 4 * case["axes"]), flops=n * (H + Hkv) * case["rot"] * 3)
    lens = _lengths(case)
    n = sum(a for a, _ in lens)
    pages = sum(-(-k // case["page"]) for _, k in lens)
    if case["op"] == "append":
        touched = sum((k - 1) // case["page"] - (k - a) // case["page"] + 1 for a, k in lens)
        pos = 0 if case["axes"] == 1 else 4 * case["axes"]
        return dict(bytes=n * ((H + 2 * Hkv) * d * 4 + pos) + 4 * (touched + 2 * len(lens)),
                    flops=n * (H + Hkv) * case["rot"] * 3)
    pairs = sum(a * (k - a) + a * (a + 1) // 2 if case["causal"] else a * k for a, k in lens)
    keys = sum(k for _, k in lens)
    return dict(bytes=n * H * (4 * d + 4) + 4 * keys * Hkv * d + 4 * (pages + 2 * len(lens)),
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


def _partner(case, x):
    half, rot = case["rot"] // 2, case["rot"]
    at = torch.arange(case["dim"], device=x.device)
    if case["interleaved"]:
        at[:rot] = at[:rot] ^ 1
    else:
        at[:rot] = (at[:rot] + half) % rot
    return x[..., at]


def _exact_turn(case, x, pos, sign=1.0):
    cos, sin = _rotation(case, pos)
    x = x.double()
    return x * cos + sign * sin * _partner(case, x)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] in ("rope", "rope_bwd"):
        sign = -1.0 if case["op"] == "rope_bwd" else 1.0
        return tuple(torch.stack([_exact_turn(case, s[n][b], s["pos"][:, b], sign)
                                  for b in range(case["batch"])]) for n in ("q", "k"))
    cu, kv, page = s["cu"].tolist(), s["kv"].tolist(), case["page"]
    if case["op"] == "append":
        seq = [torch.arange(kv[b] - cu[b + 1] + cu[b], kv[b], device=s["cu"].device) for b in range(len(kv))]
        slot = torch.cat([s["blocks"][b, p // page] * page + p % page for b, p in enumerate(seq)])
        pos = torch.cat(seq)[None] if s["pos"] is None else s["pos"]
        out = dict(q=_exact_turn(case, s["q"], pos))
        for n, rows in (("k", _exact_turn(case, s["k"], pos)), ("v", s["v"].double())):
            flat = s[n + "_pages"].double().transpose(0, 1).flatten(1, 2)  # [Hkv, slots, d]
            flat[:, slot.long()] = rows
            out[n] = flat.unflatten(1, (-1, page)).transpose(0, 1).contiguous()
        return out
    group = case["heads"] // case["kv_heads"]
    o = torch.empty(s["q"].shape, dtype=torch.float64, device=s["q"].device)
    lse = torch.empty(s["q"].shape[:2], dtype=torch.float64, device=s["q"].device)
    for b in range(len(kv)):
        a, e = cu[b], cu[b + 1]
        pages = s["blocks"][b, :-(-kv[b] // page)].long()
        for h in range(case["heads"]):
            k, v = (s[n][pages, h // group].flatten(0, 1)[:kv[b]].double() for n in ("k_pages", "v_pages"))
            x = s["q"][h, a:e].double() @ k.t() * case["dim"] ** -0.5
            if case["causal"]:
                x += torch.full_like(x, -math.inf).triu(kv[b] - (e - a) + 1)
            lse[h, a:e] = torch.logsumexp(x, -1)
            o[h, a:e] = torch.softmax(x, -1) @ v
    return o, lse
