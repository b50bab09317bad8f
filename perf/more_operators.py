"""Cases of serving from a paged cache, for measurement.

Four families of calls, each in a plain form (elementary torch operations) and through the
package's own entry points (`own`):

  append   kv_cache_append_paged: QK-Norm and RoPE (scaled for long contexts where asked) of a ragged
           batch of new tokens, written into the pages that each sequence's table names
  attn     kv_attn_paged: attention of those tokens, one or many a sequence, over the pages
  beam     beam_select: the best continuations over beams and vocabulary
  reorder  kv_cache_reorder_paged: page tables and partly filled pages follow the selected beams

A pool holds pages of `page` slots: K [pages, KV heads, page, Dk] and V [pages, KV heads, page, Dv].
Slot s of a sequence lies in page table[sequence, s // page] at row s % page.  A batch lists its new
tokens one sequence after another (token_start [B + 1]); lengths [B] count a sequence's slots with
the new tokens, which are its last ones.
"""
import math

import numpy as np
import torch

own = False

F32, F64, BF16 = torch.float32, torch.float64, torch.bfloat16
DTYPES = {"f32": F32, "bf16": BF16}

# The geometry that the repository's workloads use: 16/8 heads of 128, vocabulary 151936, 28 layers;
# 32 heads of K 192 / V 128 with 64 interleaved rotary dims for the expanded MLA layer; xdRoPE
# sections of 16 with base 1.11588e7 for the image-span layer.
THETA, XD_BASE, LAYERS = 1.0e6, 1.11588e7, 28


def _batch(name, op, singles, chunks, clo, chi, lo, hi, idle, page, Hq, Hkv, Dk, Dv, ctx):
    """`singles` sequences of one new token, `chunks` of clo..chi new ones, `idle` of none, after lo..hi older ones."""
    return dict(name=name, op=op, singles=singles, chunks=chunks, clo=clo, chi=chi, lo=lo, hi=hi, idle=idle, page=page,
                Hq=Hq, Hkv=Hkv, Dk=Dk, Dv=Dv, ctx=ctx)


def _append(batch, in_dtype, cache, rope, norm, fused, scaled, start):
    return dict(batch, in_dtype=in_dtype, cache=cache, rope=rope, norm=norm, fused=fused, scaled=scaled, start=start)


def _attn(batch, cache, out):
    return dict(batch, cache=cache, out=out)


def _beam(name, B, K, V, n, dtype, first, done, pad):
    return dict(name=name, op="beam", B=B, K=K, V=V, n=n, dtype=dtype, first=first, done=done, pad=pad)


def _reorder(name, B, K, extra, layers, page, lo, hi, Hkv, Dk, Dv, cache, ctx):
    return dict(name=name, op="reorder", B=B, K=K, extra=extra, layers=layers, page=page, lo=lo, hi=hi, Hkv=Hkv, Dk=Dk,
                Dv=Dv, cache=cache, ctx=ctx)


def listed():
    return [
        # a decode step of a serving batch: one new token in each of 64 sequences (latency)
        _append(_batch("append_step_64", "append", 64, 0, 0, 0, 100, 1000, 0, 16, 16, 8, 128, 128, 1),
                "f32", "bf16", "1d", True, False, False, 0),
        # ragged prompt chunks of 24 sequences straight from a fused projection, positions scaled for a long context
        _append(_batch("append_chunks_24", "append", 6, 18, 64, 1024, 0, 700, 1, 64, 16, 8, 128, 128, 2),
                "bf16", "bf16", "1d", True, True, True, 60000),
        # one sequence, one layer, a short context: the smallest attention call
        _attn(_batch("attn_step_1", "attn", 1, 0, 0, 0, 767, 767, 0, 16, 16, 8, 128, 128, 3), "bf16", "f32"),
        # batched serving: 64 sequences with ragged contexts of 1k to 32k tokens
        _attn(_batch("attn_step_64", "attn", 64, 0, 0, 0, 1024, 32767, 0, 64, 16, 8, 128, 128, 4), "bf16", "bf16"),
        # a chunk of a long prompt: 2048 new tokens behind 30000
        _attn(_batch("attn_chunk_2048", "attn", 0, 1, 2048, 2048, 29987, 29987, 0, 128, 32, 8, 128, 128, 5), "bf16", "bf16"),
        # a step that mixes decoding sequences with odd prompt chunks and idle rows
        _attn(_batch("attn_mixed_64", "attn", 56, 6, 33, 301, 500, 4000, 2, 16, 16, 8, 128, 128, 6), "bf16", "bf16"),
        # short draft blocks over the expanded MLA layer, results in 32 bits
        _attn(_batch("attn_mla_16", "attn", 8, 8, 2, 9, 1500, 4096, 0, 32, 32, 32, 192, 128, 7), "bf16", "f32"),
        # a small fp32 model, odd chunks
        _attn(_batch("attn_f32_7", "attn", 3, 4, 5, 37, 0, 700, 1, 16, 12, 4, 64, 64, 8), "f32", "f32"),
        # the second step of one sequence's beam search
        _beam("beam_4", 1, 4, 151936, 8, "f32", False, 0, 0),
        # a batch of beam searches over bf16 logits of a padded table, some beams done
        _beam("beam_32x8", 32, 8, 151643, 8, "bf16", False, 40, 293),
        # one sequence's four beams, every layer
        _reorder("reorder_4", 1, 4, 2, LAYERS, 16, 700, 700, 8, 128, 128, "bf16", 9),
        # 32 sequences of eight beams, every layer
        _reorder("reorder_32x8", 32, 8, 4, LAYERS, 16, 300, 2000, 8, 128, 128, "bf16", 10),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "attn", "attn", "attn", "beam", "reorder"])
    Dk, Dv = rng.choice([(64, 64), (128, 128), (128, 128), (192, 128)])
    if op == "beam":
        B, K, V = _log_int(rng, 1, 64), _log_int(rng, 1, 16), _log_int(rng, 1000, 151936)
        B = max(1, min(B, 256 * 151936 // (K * V)))
        n = min(32, rng.choice([K, K, 2 * K, 1]))
        c = _beam("", B, K, V, n, rng.choice(["f32", "bf16"]), rng.random() < 0.3, rng.choice([0, 0, 20]), rng.choice([0, 5, 64]))
    elif op == "reorder":
        K = rng.choice([2, 3, 4, 5, 8, 16])
        B, layers = _log_int(rng, 1, 32), _log_int(rng, 1, LAYERS)
        page = rng.choice([16, 32, 64])
        Hkv = rng.choice([1, 2, 4, 8])
        B = max(1, min(B, 32 * 8 * LAYERS * 16 * 8 * 256 // (K * layers * page * Hkv * (Dk + Dv))))
        lo = _log_int(rng, 1, 2000)
        c = _reorder("", B, K, rng.randrange(K), layers, page, lo, lo + rng.choice([0, 100, 1000]), Hkv, Dk, Dv,
                     rng.choice(["bf16", "bf16", "f32"]), rng.randrange(1 << 20))
    else:
        cache = rng.choice(["bf16", "bf16", "bf16", "f32"])
        Hkv = rng.choice([1, 2, 4, 8])
        G = rng.choice([1, 2, 3, 4, 7, 8])
        page = rng.choice([16, 32, 64, 128, 256])
        singles = rng.choice([0, _log_int(rng, 1, 64)])
        chunks = rng.choice([0, _log_int(rng, 1, 12)]) if singles else _log_int(rng, 1, 12)
        chi = _log_int(rng, 2, 2048 if op == "append" else 600)
        clo = max(1, int(chi * rng.choice([1.0, 0.5, 0.05])))
        hi = _log_int(rng, 1, 2000 if op == "append" else 32000)
        lo = int(hi * rng.choice([1.0, 0.5, 0.0]))
        if op == "append":
            chunks = max(1 - min(1, singles), min(chunks, 10000 // chi))
        else:                                        # scores of the padded batch, and the rows that it gathers
            T = chi if chunks else 1
            most = 120_000_000 if cache == "f32" else 1_000_000_000
            n = max(1, min(most // (Hkv * G * T * (hi + T)), 6_500_000 // ((hi + T) * Hkv)))
            singles, chunks = min(singles, max(0, n - chunks)), min(chunks, n)
        if singles + chunks == 0:
            singles = 1
        b = _batch("", op, singles, chunks, clo, chi, lo, hi, rng.choice([0, 0, 1]), page, Hkv * G, Hkv, Dk, Dv, rng.randrange(1 << 20))
        if op == "append":
            c = _append(b, rng.choice(["f32", "bf16"]), cache, rng.choice(["none", "1d", "sections", "2d", "interleaved64"]),
                        rng.random() < 0.7, rng.random() < 0.5, rng.random() < 0.5, rng.choice([0, 0, 40000, 1000000]))
        else:
            c = _attn(b, cache, "f32" if cache == "f32" else rng.choice(["f32", "bf16", "bf16"]))
    del c["name"]
    return c


# ---------------------------------------------------------------------------------
# what a program has in hand
# ---------------------------------------------------------------------------------
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _randn(g, *shape):
    return torch.randn(shape, device="cuda", generator=g)


def _lengths(case):
    """New tokens and slots (with them) of each sequence."""
    r = np.random.RandomState(case["ctx"])
    new = np.concatenate([np.ones(case["singles"], np.int64), r.randint(case["clo"], case["chi"] + 1, case["chunks"]),
                          np.zeros(case["idle"], np.int64)])
    old = r.randint(case["lo"], case["hi"] + 1, len(new))
    if case["idle"]:
        old[-1] = 0                                                       # a padding row
    order = r.permutation(len(new))
    return new[order], (old + new)[order]


def _pages(case, g, lengths, spare=0):
    """A shuffled page table and the number of pages."""
    need = np.maximum(1, -(-lengths // case["page"]))
    first = np.concatenate([[0], np.cumsum(need)])
    total = int(first[-1]) + spare
    shuffled = torch.randperm(total, device="cuda", generator=g, dtype=torch.int32)
    at = np.minimum(first[:-1, None] + np.arange(need.max()), first[1:, None] - 1)
    return shuffled[torch.from_numpy(at).cuda()].contiguous(), total


def _rope_layout(case):
    """Pairs of the rotary embedding: input dims (a_j, b_j), output dims (c_j, d_j), position axis and
    inverse frequency (64 bits) of pair j; the dims outside the pairs pass through."""
    D, kind = case["Dk"], case["rope"]
    j = np.arange(D // 2)
    if kind == "none":
        e = np.zeros(0, np.int64)
        a, b, c, d, axis, inv = e, e, e, e, e, np.zeros(0)
    elif kind == "1d":
        a, b, c, d, axis, inv = j, j + D // 2, j, j + D // 2, 0 * j, THETA ** (-2.0 * j / D)
    elif kind == "sections":
        a, b, c, d, axis, inv = j, j + D // 2, j, j + D // 2, j // (D // 8), XD_BASE ** (-2.0 * j / D)
    elif kind == "2d":
        h, q = j // (D // 4), j % (D // 4)
        a = h * (D // 2) + q
        b, c, d, axis, inv = a + D // 4, a, a + D // 4, h, THETA ** (-2.0 * q / (D // 2))
    else:                                            # the last 64 dims, interleaved pairs on input, halves on output
        r, off = np.arange(32), D - 64
        a, b, c, d, axis, inv = off + 2 * r, off + 2 * r + 1, off + r, off + 32 + r, 0 * r, THETA ** (-2.0 * r / 64)
    if case["scaled"]:
        # frequencies that turn less than LOW times in the ORIG first positions are divided by FACTOR,
        # those that turn more than HIGH times stay, the ones between are interpolated
        keep = np.clip((ORIG * inv / (2 * math.pi) - LOW) / (HIGH - LOW), 0.0, 1.0)
        inv = inv * (keep + (1 - keep) / FACTOR)
    return a, b, c, d, axis, inv


FACTOR, ORIG, LOW, HIGH, MAGNITUDE = 8.0, 8192, 1.0, 4.0, 1.2079441541679836   # 0.1 ln 8 + 1


def _n_axes(case):
    return {"none": 1, "1d": 1, "sections": 4, "2d": 2, "interleaved64": 1}[case["rope"]]


def _prepare_append(case, s, g):
    Hq, Hkv, Dk, Dv = (case[k] for k in ("Hq", "Hkv", "Dk", "Dv"))
    T, dt = int(s["start_host"][-1]), DTYPES[case["in_dtype"]]
    q = _randn(g, T, Hq, Dk).to(dt)
    k = (_randn(g, T, Hkv, Dk) * torch.exp(0.3 * _randn(g, Hkv, Dk))).to(dt)
    v = _randn(g, T, Hkv, Dv).to(dt)
    if case["fused"]:                                # one row a token: q, k, v of all heads
        row = torch.cat([x.flatten(1) for x in (q, k, v)], 1)
        q, k, v = (x.unflatten(1, (-1, D)) for x, D in
                   zip(row.split([Hq * Dk, Hkv * Dk, Hkv * Dv], 1), (Dk, Dk, Dv)))
    s["q"], s["k"], s["v"] = q, k, v
    s["qw"] = 1 + 0.1 * _randn(g, Dk) if case["norm"] else None
    s["kw"] = 1 + 0.1 * _randn(g, Dk) if case["norm"] else None
    seq = torch.repeat_interleave(torch.arange(len(s["lengths_host"]), device="cuda"), s["new"])
    s["seq"] = seq
    s["slot"] = torch.arange(T, device="cuda") - s["start"].long()[seq] + (s["lengths"].long() - s["new"])[seq]
    pos = case["start"] + s["slot"].to(torch.int32)[:, None]
    s["pos"] = (pos - torch.arange(_n_axes(case), device="cuda", dtype=torch.int32) * (case["start"] // 5)).contiguous()
    cd = DTYPES[case["cache"]]
    s["kc"] = torch.zeros((s["pages"], Hkv, case["page"], Dk), dtype=cd, device="cuda")
    s["vc"] = torch.zeros((s["pages"], Hkv, case["page"], Dv), dtype=cd, device="cuda")
    s["q_out"] = torch.empty((T, Hq, Dk), dtype=cd, device="cuda")


def _prepare_attn(case, s, g):
    Hq, Hkv, Dk, Dv = (case[k] for k in ("Hq", "Hkv", "Dk", "Dv"))
    cd = DTYPES[case["cache"]]
    s["kc"] = torch.empty((s["pages"], Hkv, case["page"], Dk), dtype=cd, device="cuda")
    s["vc"] = torch.empty((s["pages"], Hkv, case["page"], Dv), dtype=cd, device="cuda")
    for x in (s["kc"], s["vc"]):
        for part in x.split(max(1, (1 << 28) // x[0].numel())):
            part.copy_(_randn(g, *part.shape))
    T = int(s["start_host"][-1])
    s["q"] = (1.5 * _randn(g, T, Hq, Dk)).to(cd)
    s["out"] = torch.empty((T, Hq, Dv), dtype=DTYPES[case["out"]], device="cuda")


def _prepare_beam(case, s, g):
    B, K, V = (case[k] for k in ("B", "K", "V"))
    z = _randn(g, B * K, V + case["pad"]) * 1.7
    near = torch.randint(0, V, (B * K, 40), device="cuda", generator=g)      # a few likely tokens a beam
    z.scatter_add_(1, near, 12.0 * torch.rand((B * K, 40), device="cuda", generator=g))
    z[:, :3] = -math.inf                                                      # tokens that may not follow
    s["logits"] = z.to(DTYPES[case["dtype"]])[:, :V].unflatten(0, (B, K))
    s["scores"] = -30.0 * torch.rand((B, K), device="cuda", generator=g)
    if case["first"]:
        s["scores"][:, 1:] = -math.inf
    s["done"] = (100 * torch.rand((B, K), device="cuda", generator=g) < case["done"]).to(torch.int32)
    s["beam"] = torch.empty((B, case["n"]), dtype=torch.int32, device="cuda")
    s["token"] = torch.empty((B, case["n"]), dtype=torch.int32, device="cuda")
    s["score"] = torch.empty((B, case["n"]), device="cuda")


END = 1000 - 7                                       # the end token's id


def _beam_lengths(case):
    r = np.random.RandomState(case["ctx"])
    return r.randint(case["lo"], case["hi"] + 1, case["B"]).astype(np.int64)


def _prepare_reorder(case, s, g):
    B, K, page, layers = (case[k] for k in ("B", "K", "page", "layers"))
    per_group = _beam_lengths(case)
    s["lengths_host"] = np.repeat(per_group[:, None], K, 1).astype(np.int32)
    s["lengths"] = torch.from_numpy(s["lengths_host"]).cuda()
    need = -(-per_group // page)
    wide = int(need.max()) + 2
    # beams share a few pages of context; each has its last, partly filled page and a spare one
    shared, tails = 64, B * K
    total = shared + 2 * tails
    names = torch.randperm(total, device="cuda", generator=g, dtype=torch.int32)
    r = np.random.RandomState(case["ctx"] + 1)
    table = r.randint(0, shared, (B, 1, wide)).repeat(K, 1)
    for b in range(B):
        table[b, :, need[b] - 1] = shared + b * K + np.arange(K)
    s["table"] = names[torch.from_numpy(table).cuda()].contiguous()
    s["spare"] = names[shared + tails + torch.arange(tails, device="cuda")].view(B, K).contiguous()
    # K - extra beams survive, `extra` of them (or one, several times) carry on as two
    keep = torch.rand((B, K), device="cuda", generator=g).argsort(1)[:, : K - case["extra"]]
    again = torch.randint(0, K - case["extra"], (B, case["extra"]), device="cuda", generator=g)
    parent = torch.cat([keep, keep.gather(1, again)], 1)
    mix = torch.rand((B, K), device="cuda", generator=g).argsort(1)
    s["parent"] = parent.gather(1, mix).to(torch.int32)
    cd = DTYPES[case["cache"]]
    s["kc"] = torch.empty((layers, total, case["Hkv"], page, case["Dk"]), dtype=cd, device="cuda")
    s["vc"] = torch.empty((layers, total, case["Hkv"], page, case["Dv"]), dtype=cd, device="cuda")
    for x in (s["kc"], s["vc"]):
        for part in x:
            part.copy_(_randn(g, *part.shape))
    s["table_out"] = torch.zeros_like(s["table"])
    s["lengths_out"] = torch.empty_like(s["lengths"])
    s["spare_out"] = torch.empty_like(s["spare"])


def prepare(case, seed):
    g = _gen(seed)
    s = {"case": dict(case)}
    if case["op"] in ("append", "attn"):
        new, lengths = _lengths(case)
        s["lengths_host"] = lengths.astype(np.int32)
        s["start_host"] = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        s["new"], s["lengths"] = torch.from_numpy(new).cuda(), torch.from_numpy(s["lengths_host"]).cuda()
        s["start"] = torch.from_numpy(s["start_host"]).cuda()
        s["table"], s["pages"] = _pages(case, g, lengths)
    {"append": _prepare_append, "attn": _prepare_attn, "beam": _prepare_beam, "reorder": _prepare_reorder}[case["op"]](case, s, g)
    return s


# ---------------------------------------------------------------------------------
# the plain form
# ---------------------------------------------------------------------------------
def _rms(x, w, eps=1e-6):
    return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + eps) * w


def _rotate(x, case, pos):
    a, b, c, d, axis, inv = _rope_layout(case)
    if len(a) == 0:
        return x
    a, b, c, d, axis = (torch.from_numpy(t).cuda() for t in (a, b, c, d, axis))
    size = MAGNITUDE if case["scaled"] else 1.0
    ang = pos[..., axis].to(F64) * torch.from_numpy(inv).cuda()               # far positions need 64 bits
    cos, sin = (size * ang.cos()).float()[:, None], (size * ang.sin()).float()[:, None]
    y = x.clone()
    y[..., c] = x[..., a] * cos - x[..., b] * sin
    y[..., d] = x[..., b] * cos + x[..., a] * sin
    return y


def _plain_append(s):
    case, pos = s["case"], s["pos"]
    q, k = s["q"].float(), s["k"].float()
    if s["qw"] is not None:
        q, k = _rms(q, s["qw"]), _rms(k, s["kw"])
    s["q_out"].copy_(_rotate(q, case, pos))
    k = _rotate(k, case, pos)
    page = s["table"][s["seq"], s["slot"] // case["page"]].long()
    row = s["slot"] % case["page"]
    s["kc"][page, :, row] = k.to(s["kc"].dtype)
    s["vc"][page, :, row] = s["v"].to(s["vc"].dtype)
    return {"q": s["q_out"], "k": s["kc"], "v": s["vc"]}


def _gathered(s, pool):
    """[B, KV heads, slots, D] float32 rows of every sequence's pages."""
    x = pool[s["table"].long()]                                               # [B, pages, Hkv, page, D]
    return x.transpose(1, 2).flatten(2, 3).float()


def _plain_attn(s):
    case = s["case"]
    Hq, Hkv, Dk, Dv = (case[k] for k in ("Hq", "Hkv", "Dk", "Dv"))
    G, B, T = Hq // Hkv, len(s["lengths_host"]), int(np.diff(s["start_host"]).max())
    step = torch.arange(T, device="cuda")
    here = step < s["new"][:, None]                                           # [B, T] tokens that exist
    at = (s["start"].long()[:-1, None] + step).clamp_max(s["q"].shape[0] - 1)
    q = s["q"][at].float().view(B, T, Hkv, G, Dk).permute(0, 2, 1, 3, 4).reshape(B, Hkv, T * G, Dk)
    x = (q @ _gathered(s, s["kc"]).transpose(-1, -2)).mul_(Dk ** -0.5)        # [B, Hkv, T*G, W]
    seen = (s["lengths"].long() - s["new"])[:, None] + step                   # the last visible slot of a row
    slots = torch.arange(x.shape[-1], device="cuda")
    x.masked_fill_(slots > seen.repeat_interleave(G, 1)[:, None, :, None], -math.inf)
    x.sub_(x.amax(-1, keepdim=True).clamp_min(-1e30)).exp_()
    total = x.sum(-1, keepdim=True)
    v = _gathered(s, s["vc"]).masked_fill_((slots >= s["lengths"][:, None])[:, None, :, None], 0.0)
    o = (x @ v) / torch.where(total > 0, total, 1.0)                          # rows that see nothing: zeros
    s["out"].copy_(o.view(B, Hkv, T, G, Dv).permute(0, 2, 1, 3, 4).reshape(B, T, Hq, Dv)[here])
    return s["out"]


def _plain_beam(s):
    case = s["case"]
    B, K, V, n = (case[k] for k in ("B", "K", "V", "n"))
    z = s["logits"].double()
    m = z.amax(-1, keepdim=True)
    e = torch.exp(z - m).sum(-1, keepdim=True)                                # 64 bits: beams that are nearly even
    ids = s["logits"].sort(dim=-1, descending=True, stable=True).indices[..., :n]
    total = s["scores"].double()[..., None] + (z.gather(-1, ids) - m - e.log())
    width = ids.shape[-1]
    done = s["done"].bool()[..., None]
    only = torch.arange(width, device="cuda") == 0                            # a beam that is done stays as it is
    total = torch.where(done, torch.where(only, s["scores"].double()[..., None], -math.inf), total)
    ids = torch.where(done, END, ids)
    flat, order = total.flatten(1).sort(dim=-1, descending=True, stable=True)
    flat, order = flat[:, :n], order[:, :n]
    none = flat == -math.inf
    s["beam"][:, : flat.shape[1]] = torch.where(none, -1, order // width).to(torch.int32)
    s["token"][:, : flat.shape[1]] = torch.where(none, -1, ids.flatten(1).gather(1, order)).to(torch.int32)
    s["score"][:, : flat.shape[1]] = flat.float()
    return {"beam": s["beam"], "token": s["token"], "score": s["score"]}


def _plain_reorder(s):
    case = s["case"]
    B, K, page = case["B"], case["K"], case["page"]
    p = s["parent"].long()
    length = s["lengths"].gather(1, p)
    s["lengths_out"].copy_(length)
    wide = torch.arange(s["table"].shape[2], device="cuda")
    used = -(-length // page)
    rows = s["table"].gather(1, p[..., None].expand(-1, -1, len(wide)))
    last = lambda t, n: t.gather(2, (n.long() - 1).clamp_min(0)[..., None])[..., 0]  # noqa: E731
    partly = length % page != 0
    tail = last(rows, used)
    earlier = torch.arange(K, device="cuda")[:, None] > torch.arange(K, device="cuda")
    # a partly filled page stays with the first beam that carries on from it; the others copy it
    copy = partly & ((tail[:, :, None] == tail[:, None]) & partly[:, None] & earlier).any(2)
    own_partly = s["lengths"] % page != 0
    own_tail = last(s["table"], -(-s["lengths"] // page))
    kept = ((own_tail[:, :, None] == tail[:, None]) & partly[:, None]).any(2)
    twice = ((own_tail[:, :, None] == own_tail[:, None]) & own_partly[:, None] & earlier).any(2)
    free = own_partly & ~kept & ~twice
    # freed pages, in order, become the spares of the beams that used theirs, in order
    place = (~free).to(torch.int32).sort(dim=1, stable=True).indices
    freed = torch.where(torch.arange(K, device="cuda") < free.sum(1, keepdim=True), own_tail.gather(1, place), -1)
    nth = (copy.long().cumsum(1) - 1).clamp_min(0)
    s["spare_out"].copy_(torch.where(copy, freed.gather(1, nth), s["spare"]))
    at_tail = wide == (used - 1)[..., None]
    rows = torch.where(copy[..., None] & at_tail, s["spare"][..., None], rows)
    s["table_out"].copy_(torch.where(wide < used[..., None], rows, s["table_out"]))
    b, k = copy.nonzero(as_tuple=True)
    fill = (length[b, k] % page).long()
    sel = torch.arange(page, device="cuda") < fill[:, None]
    i, r = sel.nonzero(as_tuple=True)
    src, dst = tail[b, k].long()[i], s["spare"][b, k].long()[i]
    for pool in (s["kc"], s["vc"]):
        pool[:, dst, :, r] = pool[:, src, :, r]
    return {"table": s["table_out"], "lengths": s["lengths_out"], "spare": s["spare_out"], "k": s["kc"], "v": s["vc"]}


# ---------------------------------------------------------------------------------
# the package's calls
# ---------------------------------------------------------------------------------
def _own_batch(K, s):
    return (K.PagedKVCache(s["kc"], s["vc"]),
            K.PagedBatch(s["table"], s["lengths"], s["start"], s["lengths_host"], s["start_host"]))


def _own_append(s):
    import kv_cache_gqa_gb300 as K
    if "call" not in s:                                                       # descriptors that a program keeps
        case = s["case"]
        cache, batch = _own_batch(K, s)
        kind, D = case["rope"], case["Dk"]
        if kind == "sections":
            rope = K.Rope("sections", XD_BASE, (D // 8,) * 4)
        elif kind == "interleaved64":
            rope = K.Rope("interleaved", THETA, rot_offset=D - 64, rot_dim=64)
        else:
            rope = K.Rope(kind, THETA)
        scale = K.RopeScale(FACTOR, ORIG, LOW, HIGH, MAGNITUDE) if case["scaled"] else None
        s["call"] = K.prepare_append_paged(s["q"], s["k"], s["v"], s["pos"], cache, batch, s["q_out"], rope,
                                           rope_scale=scale, q_norm_w=s["qw"], k_norm_w=s["kw"])
    s["call"]()
    return {"q": s["q_out"], "k": s["kc"], "v": s["vc"]}


def _own_attn(s):
    import kv_cache_gqa_gb300 as K
    if "call" not in s:
        case = s["case"]
        cache, batch = _own_batch(K, s)
        need = K.workspace_bytes("attn_paged", n_kv_heads=case["Hkv"], n_q_heads=case["Hq"], head_dim=case["Dv"])
        s["ws"] = torch.zeros(need, dtype=torch.uint8, device="cuda")
        s["call"] = K.prepare_attn_paged(s["q"], cache, batch, s["out"], s["ws"])
    s["call"]()
    return s["out"]


def _own_beam(s):
    import kv_cache_gqa_gb300 as K
    if "call" not in s:
        case = s["case"]
        need = K.workspace_bytes("beam_select", B=case["B"], vocab=case["V"], block=case["K"])
        s["ws"] = torch.zeros(need, dtype=torch.uint8, device="cuda")
        s["call"] = K.prepare_beam_select(s["logits"], s["scores"], s["beam"], s["token"], s["score"], s["ws"],
                                          finished=s["done"], end_id=END)
    s["call"]()
    return {"beam": s["beam"], "token": s["token"], "score": s["score"]}


def _own_reorder(s):
    import kv_cache_gqa_gb300 as K
    if "call" not in s:
        s["call"] = K.prepare_reorder_paged(K.PagedKVCache(s["kc"], s["vc"]), s["parent"], s["table"], s["lengths"],
                                            s["lengths_host"], s["spare"], s["table_out"], s["lengths_out"],
                                            s["spare_out"])
    s["call"]()
    return {"table": s["table_out"], "lengths": s["lengths_out"], "spare": s["spare_out"], "k": s["kc"], "v": s["vc"]}


def run(state):
    op = state["case"]["op"]
    if own:
        return {"append": _own_append, "attn": _own_attn, "beam": _own_beam, "reorder": _own_reorder}[op](state)
    return {"append": _plain_append, "attn": _plain_attn, "beam": _plain_beam, "reorder": _plain_reorder}[op](state)


# ---------------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------------
def work(case):
    if case["op"] == "beam":
        B, K, V, n = (case[k] for k in ("B", "K", "V", "n"))
        return {"bytes": B * K * V * (2 if case["dtype"] == "bf16" else 4) + B * (8 * K + 12 * n), "flops": 4 * B * K * V}
    es = 2 if case["cache"] == "bf16" else 4
    if case["op"] == "reorder":
        lengths = _beam_lengths(case)
        row = case["layers"] * case["Hkv"] * (case["Dk"] + case["Dv"]) * es
        return {"bytes": int((lengths % case["page"]).sum()) * case["extra"] * row * 2 +
                int((-(-lengths // case["page"])).sum()) * case["K"] * 8, "flops": 0}
    new, lengths = _lengths(case)
    Hq, Hkv, Dk, Dv = (case[k] for k in ("Hq", "Hkv", "Dk", "Dv"))
    T = int(new.sum())
    if case["op"] == "append":
        ins = 2 if case["in_dtype"] == "bf16" else 4
        return {"bytes": T * (Hq * Dk + Hkv * (Dk + Dv)) * (ins + es), "flops": T * 8 * (Hq + Hkv) * Dk}
    old = lengths - new
    pairs = int((new * old + new * (new + 1) // 2).sum())                     # keys that the new tokens see
    keys = int(lengths[new > 0].sum())
    return {"bytes": keys * Hkv * (Dk + Dv) * es + T * Hq * (Dk * es + Dv * (2 if case["out"] == "bf16" else 4)),
            "flops": 2 * pairs * Hq * (Dk + Dv)}


# ---------------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------------
def _exact_append(case, s):
    a, b, c, d, axis, inv = _rope_layout(case)
    size = MAGNITUDE if case["scaled"] else 1.0
    got = []
    for x, w in ((s["q"], s["qw"]), (s["k"], s["kw"])):
        x = x.to(F64)
        if w is not None:
            x = x / torch.sqrt(torch.mean(x * x, -1, keepdim=True) + 1e-6) * w.to(F64)
        z = x.clone()
        for j in range(len(a)):
            t = s["pos"][:, None, int(axis[j])].to(F64) * float(inv[j])
            z[..., int(c[j])] = size * (x[..., int(a[j])] * torch.cos(t) - x[..., int(b[j])] * torch.sin(t))
            z[..., int(d[j])] = size * (x[..., int(b[j])] * torch.cos(t) + x[..., int(a[j])] * torch.sin(t))
        got.append(z)
    pools = [torch.zeros(s[n].shape, dtype=F64, device="cuda") for n in ("kc", "vc")]
    for i in range(len(s["lengths_host"])):
        lo, hi = int(s["start_host"][i]), int(s["start_host"][i + 1])
        slot = torch.arange(hi - lo, device="cuda") + int(s["lengths_host"][i]) - (hi - lo)
        at = s["table"][i, slot // case["page"]].long()
        pools[0][at, :, slot % case["page"]] = got[1][lo:hi]
        pools[1][at, :, slot % case["page"]] = s["v"][lo:hi].to(F64)
    return {"q": got[0], "k": pools[0], "v": pools[1]}


def _exact_attn(case, s):
    Hq, Hkv, Dk, Dv = (case[k] for k in ("Hq", "Hkv", "Dk", "Dv"))
    out = torch.zeros(s["out"].shape, dtype=F64, device="cuda")
    for i in range(len(s["lengths_host"])):
        lo, hi, L = int(s["start_host"][i]), int(s["start_host"][i + 1]), int(s["lengths_host"][i])
        slot = torch.arange(L, device="cuda")
        at, row = s["table"][i, slot // case["page"]].long(), slot % case["page"]
        for g in range(Hkv):
            k, v = s["kc"][at, g, row].to(F64), s["vc"][at, g, row].to(F64)
            heads = slice(g * (Hq // Hkv), (g + 1) * (Hq // Hkv))
            for t in range(lo, hi, 512):
                u = min(hi, t + 512)
                x = torch.einsum("thd,kd->thk", s["q"][t:u, heads].to(F64), k) / math.sqrt(Dk)
                sees = slot[None] <= (L - hi + torch.arange(t, u, device="cuda"))[:, None]
                out[t:u, heads] = torch.softmax(x.masked_fill(~sees[:, None], -math.inf), -1) @ v
    return out


def _exact_beam(case, s):
    lp = s["scores"].to(F64)[..., None] + torch.log_softmax(s["logits"].to(F64), -1)
    for b, k in s["done"].nonzero().tolist():
        lp[b, k] = -math.inf
        lp[b, k, END] = s["scores"][b, k].to(F64)
    return {"beam": None, "token": None, "score": lp.flatten(1).topk(case["n"], -1).values}


def _exact_reorder(case, s):
    pools = [s[n].to(F64) for n in ("kc", "vc")]
    before = [s[n].clone() for n in ("kc", "vc")]
    parent, table, spare = (s[n].tolist() for n in ("parent", "table", "spare"))
    for b in range(case["B"]):
        L = int(s["lengths_host"][b, 0])
        fill, last, seen = L % case["page"], (L - 1) // case["page"], set()
        for k in range(case["K"]):
            p = parent[b][k]
            if fill and p in seen:
                for pool, old in zip(pools, before):
                    pool[:, spare[b][k], :, :fill] = old[:, table[b][p][last], :, :fill].to(F64)
            seen.add(p)
    return {"table": None, "lengths": None, "spare": None, "k": pools[0], "v": pools[1]}


def exact(case, seed):
    s = prepare(case, seed)
    return {"append": _exact_append, "attn": _exact_attn, "beam": _exact_beam, "reorder": _exact_reorder}[case["op"]](case, s)
