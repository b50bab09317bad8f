"""Cases of the 4-bit cache and of the vocabulary scoring, for measurement.

Three families of calls, each in a plain form (elementary torch operations) and through the
package's own entry points (`own`):

  append     kv_cache_append_q4, the appended rows read back with kv_cache_expand_q4
  decode     kv_attn_decode_q4: one token, or a block of T tokens, per sequence
  logprobs   lmhead_logprobs: log probability of given tokens, entropy, top alternatives

The 4-bit cache.  A row (one slot of one KV head) of D values is cut into D/64 groups of 64.  A
group has a scale and a midpoint, both bf16, and 64 codes u in 0..15; it stands for the values
scale * (u - 8) + mid.  A row's codes are D/8 little-endian 32-bit words, 8 codes each, lowest code
in the lowest 4 bits; word w holds dims 64 * (w % G) + 8 * (w // G) + 0..7, G = D/64 groups.
"""
import math

import numpy as np
import torch

own = False

GROUP = 64
F32, F64 = torch.float32, torch.float64
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}

# The geometry that the repository's workloads use: 16/8 heads of 128, hidden 1024, vocabulary
# 151936, 28 layers; 32 heads of K 192 / V 128 with 64 interleaved rotary dims for the expanded
# MLA layer; xdRoPE sections of 16 with base 1.11588e7 for the image-span layer.
THETA, XD_BASE = 1.0e6, 1.11588e7


def _append(name, N, T, Hq, Hkv, Dk, Dv, in_dtype, q_dtype, rope, norm, start=0):
    return dict(name=name, op="append", N=N, T=T, Hq=Hq, Hkv=Hkv, Dk=Dk, Dv=Dv, in_dtype=in_dtype,
                q_dtype=q_dtype, rope=rope, norm=norm, start=start)


def _decode(name, B, T, Hq, Hkv, Dk, Dv, lo, hi, q_dtype, idle=0, ctx=0):
    return dict(name=name, op="decode", B=B, T=T, Hq=Hq, Hkv=Hkv, Dk=Dk, Dv=Dv, lo=lo, hi=hi, q_dtype=q_dtype,
                idle=idle, ctx=ctx)


def _logprobs(name, B, H, V, h_dtype, w_dtype, norm, top):
    return dict(name=name, op="logprobs", B=B, H=H, V=V, h_dtype=h_dtype, w_dtype=w_dtype, norm=norm, top=top)


def listed():
    return [
        # one new token in each of 28 layer caches, as a decode step appends it (latency)
        _append("append_token_28", 28, 1, 16, 8, 128, 128, "f32", "bf16", "1d", True, 512),
        # a 512-token prompt in each of 28 layer caches
        _append("append_prompt_28x512", 28, 512, 16, 8, 128, 128, "bf16", "bf16", "1d", True),
        # an odd-length prompt of the expanded MLA layer (K 192, V 128, rotary sub-range), 8 layers
        _append("append_mla_8x333", 8, 333, 32, 32, 192, 128, "f32", "f32", "interleaved64", False, 7),
        # one sequence, one layer, a short context: the smallest decode call
        _decode("decode_1x768", 1, 1, 16, 8, 128, 128, 768, 768, "bf16"),
        # batched serving: 64 sequences with ragged contexts of 1k to 32k tokens
        _decode("decode_serving_64", 64, 1, 16, 8, 128, 128, 1024, 32768, "bf16", 0, 1),
        # two long documents, four query heads per KV head, contexts that end inside a tile
        _decode("decode_long_2", 2, 1, 32, 8, 128, 128, 100001, 131071, "f32", 0, 2),
        # the expanded MLA layer, 16 sequences
        _decode("decode_mla_16x4096", 16, 1, 32, 32, 192, 128, 4096, 4096, "bf16"),
        # a 16-token draft block per sequence, some padding sequences in the batch
        _decode("decode_block_64x16", 64, 16, 16, 8, 128, 128, 1900, 2048, "bf16", 3, 3),
        # every decode step of one sequence: the sampled token's log probability and 5 alternatives
        _logprobs("logprobs_1", 1, 1024, 151936, "f32", "bf16", True, 5),
        # the same for a serving batch
        _logprobs("logprobs_64", 64, 1024, 151936, "f32", "bf16", True, 8),
        # scoring a prompt of 1999 tokens whose hidden states are already normalised
        _logprobs("logprobs_prompt_1999", 1999, 1024, 151936, "bf16", "bf16", False, 1),
        # a small fp32 model's table, odd sizes
        _logprobs("logprobs_f32_5", 5, 520, 4099, "f32", "f32", True, 3),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "decode", "logprobs"])
    if op == "append":
        Dk, Dv = rng.choice([(64, 64), (128, 128), (128, 128), (192, 128)])
        Hkv = rng.choice([1, 2, 4, 8, 16])
        N = _log_int(rng, 1, 28)
        T = _log_int(rng, 1, 512)
        c = _append("", N, T, Hkv * rng.choice([1, 2, 3, 4]), Hkv, Dk, Dv, rng.choice(["f32", "bf16"]),
                    rng.choice(["f32", "bf16"]), rng.choice(["none", "1d", "sections", "2d", "interleaved64"]),
                    rng.random() < 0.7, rng.choice([0, 0, 5, 512, 40000]))
    elif op == "decode":
        Dk, Dv = rng.choice([(64, 64), (128, 128), (128, 128), (192, 128)])
        Hkv = rng.choice([1, 2, 4, 8, 16])
        B = _log_int(rng, 1, 64)
        T = rng.choice([1, 1, 1, 1, 2, 5, 16])
        hi = min(_log_int(rng, 1, 100000), max(1, 4000000 // (B * Hkv)))
        lo = max(1, int(hi * rng.choice([1.0, 0.5, 0.05])))
        c = _decode("", B, T, Hkv * rng.choice([1, 2, 4, 8]), Hkv, Dk, Dv, lo, hi, rng.choice(["f32", "bf16"]),
                    rng.choice([0, 0, 1]), rng.randrange(1 << 20))
    else:
        H = rng.choice([64, 200, 512, 520, 1024, 2048])
        V = _log_int(rng, 1000, 151936)
        w = rng.choice(["bf16", "bf16", "bf16", "f32"])
        B = _log_int(rng, 1, 1999 if w == "bf16" and H % 64 == 0 else 16)
        B = max(1, min(B, int(1999 * 1024 * 151936 / (H * V))))
        c = _logprobs("", B, H, V, rng.choice(["f32", "bf16"]), w, rng.random() < 0.5, rng.choice([0, 1, 5, 8, 20]))
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


def _rope_layout(case):
    """Pairs of the rotary embedding: input dims (a_j, b_j), output dims (c_j, d_j), position axis and
    inverse frequency (64 bits) of pair j; the dims outside the pairs pass through."""
    D, kind = case["Dk"], case["rope"]
    j = np.arange(D // 2)
    if kind == "none":
        e = np.zeros(0, np.int64)
        return e, e, e, e, e, np.zeros(0)
    if kind == "1d":
        return j, j + D // 2, j, j + D // 2, 0 * j, THETA ** (-2.0 * j / D)
    if kind == "sections":
        return j, j + D // 2, j, j + D // 2, j // (D // 8), XD_BASE ** (-2.0 * j / D)
    if kind == "2d":
        h, q = j // (D // 4), j % (D // 4)
        a = h * (D // 2) + q
        return a, a + D // 4, a, a + D // 4, h, THETA ** (-2.0 * q / (D // 2))
    # the last 64 dims, pairs interleaved on input and split in halves on output
    r, off = np.arange(32), D - 64
    return off + 2 * r, off + 2 * r + 1, off + r, off + 32 + r, 0 * r, THETA ** (-2.0 * r / 64)


def _n_axes(case):
    return {"none": 1, "1d": 1, "sections": 4, "2d": 2, "interleaved64": 1}[case["rope"]]


def _bf16_down(x):
    """The largest bf16 not above x, and _bf16_up the smallest not below it (finite x)."""
    i = x.view(torch.int32)
    i = torch.where((i < 0) & ((i & 0xFFFF) != 0), i + 0x10000, i) & -65536
    return i.view(F32)


def _bf16_up(x):
    return -_bf16_down(-x)


def _quantise(x):
    """x [.., D] float32: codes u [.., D/64, 64], scale and mid [.., D/64] (bf16 values in float32)."""
    g = x.reshape(*x.shape[:-1], -1, GROUP)
    lo, hi = g.amin(-1), g.amax(-1)
    scale = _bf16_up((hi - lo) / torch.full_like(hi, 15.0))                # quotients, not products with an
    mid = (lo + 8.0 * scale).bfloat16().float()                            # inverse: bf16 inputs meet exact ties
    u = torch.round((g - mid[..., None]) / scale[..., None]).clamp(-8, 7) + 8
    return u, scale, mid


def _pack(u):
    """Codes [.., G, 64] to bytes [.., 32 G] in the cache's word order."""
    w = u.to(torch.uint8).unflatten(-1, (8, 8)).transpose(-3, -2)          # [.., 8, G, 8]
    return (w[..., 0::2] | (w[..., 1::2] << 4)).flatten(-3).contiguous()


def _empty_q4(N, Hkv, W, D):
    codes = torch.zeros((N, Hkv, W, D // 2), dtype=torch.uint8, device="cuda")
    return codes, torch.zeros((N, Hkv, W, D // GROUP, 2), dtype=torch.bfloat16, device="cuda")


def _filled_q4(g, N, Hkv, W, D, spread):
    """A cache of normal values whose channels differ in width."""
    codes, par = _empty_q4(N, Hkv, W, D)
    width = torch.exp(spread * _randn(g, Hkv, 1, D))
    for n in range(N):
        u, scale, mid = _quantise(_randn(g, Hkv, W, D) * width)
        codes[n] = _pack(u)
        par[n] = torch.stack([scale, mid], -1).bfloat16()
    return codes, par


def _lengths(case):
    r = np.random.RandomState(case["ctx"])
    L = r.randint(case["lo"], case["hi"] + 1, case["B"]).astype(np.int32)
    L[-1] = case["hi"]
    L[: min(case["idle"], case["B"] - 1)] = 0                              # padding sequences
    return L


def prepare(case, seed):
    g = _gen(seed)
    s = {"case": dict(case)}
    if case["op"] == "append":
        N, T, Hq, Hkv, Dk, Dv = (case[k] for k in ("N", "T", "Hq", "Hkv", "Dk", "Dv"))
        W = (T + 8 + 3) // 4 * 4
        dt = DTYPES[case["in_dtype"]]
        s["q"] = _randn(g, N, T, Hq, Dk).to(dt)
        s["k"] = (_randn(g, N, T, Hkv, Dk) * torch.exp(0.3 * _randn(g, Hkv, Dk))).to(dt)
        s["v"] = _randn(g, N, T, Hkv, Dv).to(dt)
        s["qw"] = 1 + 0.1 * _randn(g, N, Dk) if case["norm"] else None
        s["kw"] = 1 + 0.1 * _randn(g, N, Dk) if case["norm"] else None
        pos = case["start"] + torch.arange(T, device="cuda", dtype=torch.int32)[:, None]
        pos = pos - torch.arange(_n_axes(case), device="cuda", dtype=torch.int32) * (case["start"] // 5)
        s["pos"] = pos.expand(N, T, _n_axes(case)).contiguous()
        s["slot_host"] = np.tile(np.arange(3, 3 + T, dtype=np.int32), (N, 1))
        s["slot"] = torch.from_numpy(s["slot_host"]).cuda()
        s["kc"], s["kp"] = _empty_q4(N, Hkv, W, Dk)
        s["vc"], s["vp"] = _empty_q4(N, Hkv, W, Dv)
        s["q_out"] = torch.empty((N, T, Hq, Dk), dtype=DTYPES[case["q_dtype"]], device="cuda")
        s["k_val"] = torch.empty((N, Hkv, T, Dk), dtype=torch.bfloat16, device="cuda")
        s["v_val"] = torch.empty((N, Hkv, T, Dv), dtype=torch.bfloat16, device="cuda")
    elif case["op"] == "decode":
        B, T, Hq, Hkv, Dk, Dv = (case[k] for k in ("B", "T", "Hq", "Hkv", "Dk", "Dv"))
        s["lengths_host"] = _lengths(case)
        s["lengths"] = torch.from_numpy(s["lengths_host"]).cuda()
        W = (int(s["lengths_host"].max()) + 3) // 4 * 4
        s["kc"], s["kp"] = _filled_q4(g, B, Hkv, W, Dk, 0.3)
        s["vc"], s["vp"] = _filled_q4(g, B, Hkv, W, Dv, 0.0)
        s["q"] = (1.5 * _randn(g, B, T, Hq, Dk)).to(DTYPES[case["q_dtype"]])
        s["out"] = torch.empty((B, T, Hq, Dv), dtype=F32, device="cuda")
    else:
        B, H, V, k = (case[x] for x in ("B", "H", "V", "top"))
        s["W"] = (0.02 * _randn(g, V, H)).to(DTYPES[case["w_dtype"]])
        # hidden states that point towards a few tokens each, as a trained model's do
        near = torch.randint(0, V, (B, 24), device="cuda", generator=g)
        pull = torch.rand((B, 24), device="cuda", generator=g) * 24.0 * 1024 / H
        h = _randn(g, B, H) + torch.einsum("bj,bjh->bh", pull, s["W"][near].float())
        s["h"] = h.to(DTYPES[case["h_dtype"]])
        s["nw"] = 1 + 0.1 * _randn(g, H) if case["norm"] else None
        some = torch.randint(0, V, (B,), device="cuda", generator=g)
        pick = torch.rand((B,), device="cuda", generator=g) < 0.75
        s["targets"] = torch.where(pick, near[torch.arange(B, device="cuda"), pull.argmax(1)], some).to(torch.int32)
        s["logprob"] = torch.empty((B,), device="cuda")
        s["entropy"] = torch.empty((B,), device="cuda")
        s["ids"] = torch.empty((B, k), dtype=torch.int32, device="cuda")
        s["top"] = torch.empty((B, k), device="cuda")
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
    ang = pos[..., axis].to(F64) * torch.from_numpy(inv).cuda()            # far positions need 64 bits
    cos, sin = ang.cos().float()[:, :, None], ang.sin().float()[:, :, None]
    y = x.clone()
    y[..., c] = x[..., a] * cos - x[..., b] * sin
    y[..., d] = x[..., b] * cos + x[..., a] * sin
    return y


def _values(codes, par):
    """The float32 values of packed rows."""
    G = par.shape[-2]
    w = codes.unflatten(-1, (8, G, 4))
    u = torch.stack([w & 15, w >> 4], -1).flatten(-2).transpose(-3, -2).flatten(-2)   # [.., G, 64]
    par = par.float()
    return ((u.float() - 8.0) * par[..., 0:1] + par[..., 1:2]).flatten(-2)


def _plain_append(s):
    case, pos = s["case"], s["pos"]
    q, k, v = s["q"].float(), s["k"].float(), s["v"].float()
    if s["qw"] is not None:
        q, k = _rms(q, s["qw"][:, None, None]), _rms(k, s["kw"][:, None, None])
    s["q_out"].copy_(_rotate(q, case, pos))
    k = _rotate(k, case, pos)
    n = torch.arange(case["N"], device="cuda")[:, None, None]
    head = torch.arange(case["Hkv"], device="cuda")[None, :, None]
    slot = s["slot"].long()[:, None, :]
    for x, c, p, out in ((k, "kc", "kp", "k_val"), (v, "vc", "vp", "v_val")):
        u, scale, mid = _quantise(x.transpose(1, 2))
        s[c][n, head, slot] = _pack(u)
        s[p][n, head, slot] = torch.stack([scale, mid], -1).bfloat16()
        s[out].copy_(_values(s[c][n, head, slot], s[p][n, head, slot]))
    return {"q": s["q_out"], "k": s["k_val"], "v": s["v_val"]}


def _plain_decode(s):
    case = s["case"]
    B, T, Hq, Hkv, Dk, Dv = (case[k] for k in ("B", "T", "Hq", "Hkv", "Dk", "Dv"))
    G, W = Hq // Hkv, s["kc"].shape[2]
    q = s["q"].float().view(B, T, Hkv, G, Dk).permute(0, 2, 1, 3, 4).reshape(B, Hkv, T * G, Dk)
    x = q @ _values(s["kc"], s["kp"]).transpose(-1, -2) * Dk ** -0.5        # [B, Hkv, T*G, W]
    seen = s["lengths"].long()[:, None] - T + torch.arange(T, device="cuda")   # the last visible slot of a row
    hide = torch.arange(W, device="cuda") > seen.repeat_interleave(G, 1)[:, None, :, None]
    x = x.masked_fill(hide, -math.inf)
    p = torch.exp(x - x.amax(-1, keepdim=True).clamp_min(-1e30))
    total = p.sum(-1, keepdim=True)
    o = (p @ _values(s["vc"], s["vp"])) / torch.where(total > 0, total, 1.0)   # rows that see nothing: zeros
    s["out"].copy_(o.view(B, Hkv, T, G, Dv).permute(0, 2, 1, 3, 4).reshape(B, T, Hq, Dv))
    return s["out"]


def _plain_logprobs(s):
    case, k = s["case"], s["case"]["top"]
    h = s["h"].float()
    if s["nw"] is not None:
        h = _rms(h, s["nw"])
    z = h @ s["W"].float().T
    m = z.amax(-1, keepdim=True)
    e = torch.exp(z - m)
    total = e.sum(-1)
    lse = m[:, 0] + total.log()
    s["entropy"].copy_(total.log() - (e * (z - m)).sum(-1) / total)
    rows = torch.arange(case["B"], device="cuda")

    def again(ids):                                                        # logits of a few ids, 64 bits
        return (s["W"][ids].to(F64) * h.to(F64)[:, None]).sum(-1)

    s["logprob"].copy_(again(s["targets"].long()[:, None])[:, 0] - lse)
    if k:
        ids = z.topk(k + 8, -1).indices.sort(-1).values                    # neighbours change places in 32 bits
        fine = again(ids)
        order = fine.sort(dim=-1, descending=True, stable=True).indices[:, :k]
        s["ids"].copy_(ids[rows[:, None], order])
        s["top"].copy_(fine[rows[:, None], order] - lse[:, None])
    return {"logprob": s["logprob"], "entropy": s["entropy"], "ids": s["ids"], "top": s["top"]}


# ---------------------------------------------------------------------------------
# the package's calls
# ---------------------------------------------------------------------------------
def _own_rope(K, case):
    kind, D = case["rope"], case["Dk"]
    if kind == "sections":
        return K.Rope("sections", XD_BASE, (D // 8,) * 4)
    if kind == "interleaved64":
        return K.Rope("interleaved", THETA, rot_offset=D - 64, rot_dim=64)
    return K.Rope(kind, THETA)


def _own_append(s):
    import kv_cache_gqa_gb300 as K
    if "calls" not in s:                                                   # descriptors that a program keeps
        case = s["case"]
        cache = K.KVCacheQ4(s["kc"], s["vc"], s["kp"], s["vp"])
        s["calls"] = (
            K.prepare_append_q4(s["q"], s["k"], s["v"], s["pos"], s["slot"], s["slot_host"], cache, s["q_out"],
                                _own_rope(K, case), q_norm_w=s["qw"], k_norm_w=s["kw"],
                                norm_inst_stride=case["Dk"] if case["norm"] else 0),
            K.prepare_expand_q4(cache, s["slot"], s["slot_host"], K.KVCache(s["k_val"], s["v_val"])))
    s["calls"][0]()
    s["calls"][1]()
    return {"q": s["q_out"], "k": s["k_val"], "v": s["v_val"]}


def _own_decode(s):
    import kv_cache_gqa_gb300 as K
    if "call" not in s:
        case = s["case"]
        cache = K.KVCacheQ4(s["kc"], s["vc"], s["kp"], s["vp"])
        need = K.workspace_bytes("decode_q4", B=case["B"], n_kv_heads=case["Hkv"], n_q_heads=case["Hq"],
                                 max_len=s["kc"].shape[2], head_dim=case["Dv"], block=case["T"])
        s["ws"] = torch.zeros(need, dtype=torch.uint8, device="cuda")
        s["call"] = K.prepare_decode_q4(s["q"], cache, s["lengths"], s["lengths_host"], s["out"], s["ws"])
    s["call"]()
    return s["out"]


def _own_logprobs(s):
    import kv_cache_gqa_gb300 as K
    if "call" not in s:
        case = s["case"]
        need = K.workspace_bytes("lmhead_logprobs", B=case["B"], hidden=case["H"], vocab=case["V"], block=case["top"])
        s["ws"] = torch.zeros(need, dtype=torch.uint8, device="cuda")
        s["call"] = K.prepare_lmhead_logprobs(
            s["h"], s["W"], s["ws"], targets=s["targets"], out_logprob=s["logprob"], out_entropy=s["entropy"],
            top_ids=s["ids"], top_logprobs=s["top"], norm_w=s["nw"])
    s["call"]()
    return {"logprob": s["logprob"], "entropy": s["entropy"], "ids": s["ids"], "top": s["top"]}


def run(state):
    op = state["case"]["op"]
    if own:
        return {"append": _own_append, "decode": _own_decode, "logprobs": _own_logprobs}[op](state)
    return {"append": _plain_append, "decode": _plain_decode, "logprobs": _plain_logprobs}[op](state)


# ---------------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------------
def _row_bytes(D):
    return D // 2 + D // GROUP * 4


def work(case):
    if case["op"] == "append":
        N, T, Hq, Hkv, Dk, Dv = (case[k] for k in ("N", "T", "Hq", "Hkv", "Dk", "Dv"))
        es = 2 if case["in_dtype"] == "bf16" else 4
        qs = 2 if case["q_dtype"] == "bf16" else 4
        token = Hq * Dk * (es + qs) + Hkv * ((Dk + Dv) * (es + 2) + _row_bytes(Dk) + _row_bytes(Dv))
        return {"bytes": N * T * token, "flops": N * T * (8 * (Hq + Hkv) * Dk + 6 * Hkv * (Dk + Dv))}
    if case["op"] == "decode":
        B, T, Hq, Hkv, Dk, Dv = (case[k] for k in ("B", "T", "Hq", "Hkv", "Dk", "Dv"))
        keys = int(_lengths(case).astype(np.int64).sum())
        qs = 2 if case["q_dtype"] == "bf16" else 4
        return {"bytes": keys * Hkv * (_row_bytes(Dk) + _row_bytes(Dv)) + B * T * Hq * (Dk * qs + Dv * 4),
                "flops": 2 * keys * T * Hq * (Dk + Dv)}
    B, H, V = case["B"], case["H"], case["V"]
    return {"bytes": V * H * (2 if case["w_dtype"] == "bf16" else 4) + B * H * (2 if case["h_dtype"] == "bf16" else 4) +
            B * (12 + 8 * case["top"]), "flops": 2 * B * V * H}


# ---------------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------------
def _round_bf16(x, how):
    """float64 values to bf16 precision: how is torch.floor, torch.ceil or torch.round (half to even)."""
    power = (x.view(torch.int64) & 0x7FF0000000000000).view(F64)           # 2^e with 2^e <= |x| < 2^(e+1)
    return torch.where(x == 0, x, how(x / power * 128.0) * power / 128.0)


def _exact_q4(x):
    """The values that a row x [.., D] of float64 stands for once it is held in 4 bits."""
    g = x.unflatten(-1, (-1, GROUP))
    lo, hi = torch.aminmax(g, dim=-1, keepdim=True)
    step = _round_bf16((hi - lo) / 15.0, torch.ceil)
    mid = _round_bf16(lo + 8.0 * step, torch.round)
    return (step * ((g - mid) / step).round().clamp(-8, 7) + mid).flatten(-2)


def _exact_unpacked(codes, par):
    """[.., D] float64 values of packed rows, word by word."""
    words = codes.contiguous().view(torch.int32).to(torch.int64)           # [.., D/8]
    G = par.shape[-2]
    D = G * GROUP
    x = torch.empty((*words.shape[:-1], D), dtype=F64, device="cuda")
    for w in range(D // 8):
        g, first = w % G, 64 * (w % G) + 8 * (w // G)
        for i in range(8):
            u = (words[..., w] >> (4 * i)) & 15
            x[..., first + i] = par[..., g, 0].to(F64) * (u - 8) + par[..., g, 1].to(F64)
    return x


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "append":
        a, b, c, d, axis, inv = _rope_layout(case)
        got = []
        for x, w in ((s["q"], s["qw"]), (s["k"], s["kw"])):
            x = x.to(F64)
            if w is not None:
                x = x / torch.sqrt(torch.mean(x * x, -1, keepdim=True) + 1e-6) * w.to(F64)[:, None, None, :]
            z = x.clone()
            for j in range(len(a)):
                t = s["pos"][:, :, None, int(axis[j])].to(F64) * float(inv[j])
                z[..., int(c[j])] = x[..., int(a[j])] * torch.cos(t) - x[..., int(b[j])] * torch.sin(t)
                z[..., int(d[j])] = x[..., int(b[j])] * torch.cos(t) + x[..., int(a[j])] * torch.sin(t)
            got.append(z)
        return {"q": got[0], "k": _exact_q4(got[1].transpose(1, 2)), "v": _exact_q4(s["v"].to(F64).transpose(1, 2))}
    if case["op"] == "decode":
        B, T, Hq, Hkv, Dk, Dv = (case[k] for k in ("B", "T", "Hq", "Hkv", "Dk", "Dv"))
        out = torch.zeros((B, T, Hq, Dv), dtype=F64, device="cuda")
        for b in range(B):
            L = int(s["lengths_host"][b])
            if L == 0:
                continue
            for g in range(Hkv):
                k = _exact_unpacked(s["kc"][b, g, :L], s["kp"][b, g, :L])
                v = _exact_unpacked(s["vc"][b, g, :L], s["vp"][b, g, :L])
                for t in range(T):
                    n = L - T + t + 1
                    if n > 0:
                        heads = slice(g * (Hq // Hkv), (g + 1) * (Hq // Hkv))
                        p = torch.softmax(s["q"][b, t, heads].to(F64) @ k[:n].T / math.sqrt(Dk), -1)
                        out[b, t, heads] = p @ v[:n]
        return out
    B, k = case["B"], case["top"]
    out = {"logprob": torch.empty(B, dtype=F64, device="cuda"), "entropy": torch.empty(B, dtype=F64, device="cuda"),
           "ids": None, "top": torch.empty((B, k), dtype=F64, device="cuda")}
    table = s["W"].to(F64)
    for i in range(0, B, 256):
        h = s["h"][i:i + 256].to(F64)
        if s["nw"] is not None:
            h = h / torch.sqrt(torch.mean(h * h, -1, keepdim=True) + 1e-6) * s["nw"].to(F64)
        lp = torch.log_softmax(h @ table.T, -1)
        out["logprob"][i:i + 256] = lp.gather(1, s["targets"][i:i + 256].long()[:, None])[:, 0]
        out["entropy"][i:i + 256] = -(lp.exp() * lp).sum(-1)
        out["top"][i:i + 256] = lp.topk(k, -1).values
    return out
