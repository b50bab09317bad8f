"""The paged cache on a GPU: append, attention and the two together against the fp64 definitions.

Tolerances.  Attention: a weight reaches V rounded to half a step of its type, 2^-8 of itself in bf16 and 2^-16 in two
bf16 parts (exact for an fp32 cache), so a row is off by that times the sum of weight * |value| (`size`), by 1e-5 of `size` for
the float32 scores, exponentials and sums (the contract's 1e-5), and by half a step of the output.  Append: half a step of the stored
type, and 1e-6 of the row's root mean square for the float32 steps before it (norm, angle, two products: about 8
roundings of 2^-24, cancelled at worst)."""
import numpy as np
import pytest

import oracle as O
import workloads as WL
from helpers import dev, host
from oracle import paged_oracle as P

pytestmark = pytest.mark.gpu

HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}


@pytest.fixture(scope="module")
def K():
    from kv_cache_gqa_gb300 import build
    build.build_library(verbose=False)
    import kv_cache_gqa_gb300 as K
    yield K
    import torch
    torch.cuda.synchronize()
    assert K.wait_timeouts() == 0


def dtype(name):
    import torch
    return {"f32": torch.float32, "bf16": torch.bfloat16}[name]


def values(r, shape, name):
    """Numbers that a tensor of this type holds."""
    x = r.standard_normal(shape).astype(np.float32)
    return WL.bf16_bits_to_f32(WL.f32_to_bf16_bits(x)) if name == "bf16" else x


class Case:
    """A batch over a pool whose unused rows, and pages of no sequence, hold NaN."""

    def __init__(self, K, seed, new, lengths, page, Hq, Hkv, Dk, Dv, cache="bf16", wide=None):
        r = np.random.default_rng(seed)
        self.r, self.new, self.lengths = r, np.asarray(new), np.asarray(lengths, np.int32)
        self.start = np.concatenate([[0], np.cumsum(self.new)]).astype(np.int32)
        self.page, self.Hq, self.Hkv, self.Dk, self.Dv, self.cache = page, Hq, Hkv, Dk, Dv, cache
        need = [max(0, -(-int(L) // page)) for L in self.lengths]
        self.n_pages = sum(need) + 3
        ids = r.permutation(self.n_pages).astype(np.int32)
        self.table = np.full((len(need), wide or max(need + [1])), -7, np.int32)      # what is not needed names no page
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = ids[at:at + n]
            at += n
        self.pool_k = np.full((self.n_pages, Hkv, page, Dk), np.nan, np.float32)
        self.pool_v = np.full((self.n_pages, Hkv, page, Dv), np.nan, np.float32)

    def fill(self):
        for b, L in enumerate(self.lengths):
            for s0 in range(0, max(0, int(L)), self.page):
                n = min(self.page, int(L) - s0)
                p = self.table[b, s0 // self.page]
                self.pool_k[p, :, :n] = values(self.r, (self.Hkv, n, self.Dk), self.cache)
                self.pool_v[p, :, :n] = values(self.r, (self.Hkv, n, self.Dv), self.cache)
        return self

    def on_gpu(self, K):
        cache = K.PagedKVCache(dev(self.pool_k, dtype(self.cache)), dev(self.pool_v, dtype(self.cache)))
        return cache, K.PagedBatch(dev(self.table), dev(self.lengths), dev(self.start), self.lengths, self.start, self.table)

    def workspace(self, K):
        import torch
        return torch.zeros(K.paged_workspace_bytes(self.Hkv, self.Hq, self.Dv), dtype=torch.uint8, device="cuda")


def check_attention(got, q, c, out, scale=None, rows=None):
    o, size = P.paged_attention(q, c.pool_k.astype(np.float64), c.pool_v.astype(np.float64), c.table, c.lengths, c.start, scale)
    weight = 0.0 if c.cache == "f32" else (2.0 ** -8 if out == "bf16" else 2.0 ** -16)
    tol = size * (weight + 1e-5) + np.abs(o) * HALF[out] * (1 + weight)
    err = np.abs(got - o)
    assert not np.isnan(got).any()
    worst = np.max(err / np.maximum(tol, 1e-30))
    assert (err <= tol).all(), f"worst error {worst:.2f} of the tolerance"


def attend(K, c, out="f32", scale=0.0, q=None, ws=None):
    import torch
    q = values(c.r, (int(c.start[-1]), c.Hq, c.Dk), c.cache) * np.float32(2) if q is None else q
    cache, batch = c.on_gpu(K)
    o = torch.full((int(c.start[-1]) + 2, c.Hq, c.Dv), 7.0, dtype=dtype(out), device="cuda")   # rows behind the last token stay
    ws = c.workspace(K) if ws is None else ws
    K.kv_attn_paged(dev(q, dtype(c.cache)), cache, batch, o[:-2], ws, scale=scale)
    torch.cuda.synchronize()
    assert (o[-2:] == 7).all()
    assert not ws[:K.paged_workspace_zero_bytes()].any()
    return q, host(o[:-2])


SHAPES = [  # new tokens, lengths, page, Hq, Hkv, Dk, Dv
    ([1], [1], 16, 1, 1, 128, 128),
    ([1], [300], 16, 16, 8, 128, 128),
    ([1, 1, 1], [17, 0, 64], 32, 8, 2, 64, 64),                     # a padding row with length 0: zeros
    ([1, 0, 1, 1], [129, 40, 128, 127], 64, 4, 4, 128, 128),        # a sequence without new tokens
    ([1, 1], [257, 511], 256, 7, 1, 192, 128),
    ([8, 3], [8, 100], 16, 2, 1, 128, 128),                         # from the first token on
    ([16, 1, 5], [333, 50, 5], 16, 16, 8, 128, 128),
    ([33, 64, 65], [70, 64, 200], 32, 6, 2, 64, 64),
    ([130], [300], 128, 3, 1, 128, 128),
    ([5], [3], 16, 4, 2, 128, 128),                                 # the first two tokens see nothing
    ([70], [40], 16, 4, 2, 128, 128),                               # nor do the first thirty
    ([129, 2, 1], [400, 400, 400], 16, 16, 4, 192, 128),
    ([2], [40], 16, 64, 1, 64, 64),                                 # many heads a KV head
    ([9], [140], 16, 40, 2, 128, 128),
]


@pytest.mark.parametrize("cache", ["bf16", "f32"])
@pytest.mark.parametrize("i", range(len(SHAPES)))
def test_attention(K, i, cache):
    c = Case(K, i, *SHAPES[i], cache=cache).fill()
    for out in ("f32", "bf16"):
        q, got = attend(K, c, out)
        check_attention(got, q, c, out)


@pytest.mark.parametrize("cache", ["bf16", "f32"])
def test_attention_of_a_long_context_in_many_runs(K, cache):
    """Units that many CTAs share, and CTAs that hold several units."""
    c = Case(K, 5, [1, 1, 2, 20], [5000, 3, 2777, 1500], 16, 4, 2, 128, 128, cache=cache).fill()
    q, got = attend(K, c)
    check_attention(got, q, c, "f32")


def test_attention_of_many_short_sequences(K):
    """More sequences than a CTA has threads, with idle ones among them."""
    n = 700
    r = np.random.default_rng(0)
    new = r.integers(0, 2, n)
    c = Case(K, 6, new, r.integers(0, 40, n) * (r.random(n) < 0.9), 16, 2, 1, 64, 64).fill()
    q, got = attend(K, c, "bf16")
    check_attention(got, q, c, "bf16")


def test_attention_scale_and_growing_scores(K):
    """A scale of the caller's, and scores that grow along the keys, so that the reference maximum moves often."""
    c = Case(K, 7, [1, 40], [600, 500], 16, 4, 2, 128, 128).fill()
    q = values(c.r, (41, 4, 128), "bf16")
    for b in range(2):
        for s in range(int(c.lengths[b])):
            p, row = c.table[b, s // 16], s % 16
            u = q[c.start[b], ::2] / np.linalg.norm(q[c.start[b], ::2], axis=1, keepdims=True)
            c.pool_k[p, :, row] = WL.bf16_bits_to_f32(WL.f32_to_bf16_bits((u * (0.02 * s)).astype(np.float32)))
    for out in ("f32", "bf16"):
        _, got = attend(K, c, out, scale=0.3, q=q)
        check_attention(got, q, c, out, scale=0.3)


def test_pages_apart_and_bad_pages(K):
    """A layer of a pool whose layers alternate; and a page id outside the pool gives NaN where it is seen, nothing else."""
    import torch
    c = Case(K, 8, [1, 4, 40], [40, 70, 90], 16, 4, 2, 128, 128).fill()
    cache, _ = c.on_gpu(K)
    wide = [torch.full((c.n_pages, 3) + tuple(t.shape[1:]), float("nan"), dtype=t.dtype, device="cuda") for t in (cache.k, cache.v)]
    for w, t in zip(wide, (cache.k, cache.v)):
        w[:, 1] = t
    layer = K.PagedKVCache(wide[0][:, 1], wide[1][:, 1])
    q = values(c.r, (45, 4, 128), "bf16")
    for table, bad in ((c.table, False), (np.where(np.arange(len(c.table[0])) == 1, c.n_pages, c.table), True)):
        o = torch.empty((45, 4, 128), device="cuda")
        batch = K.PagedBatch(dev(table.astype(np.int32)), dev(c.lengths), dev(c.start), c.lengths, c.start)
        K.kv_attn_paged(dev(q, torch.bfloat16), layer, batch, o, c.workspace(K))
        torch.cuda.synchronize()
        if not bad:
            check_attention(host(o), q, c, "f32")
        else:
            assert np.isnan(host(o)).all()                            # every token here sees slots 16..31


def test_device_lengths_below_the_mirror(K):
    """A captured step: the mirror holds the largest lengths, the device the present ones; replays follow the device."""
    import torch
    c = Case(K, 9, [1, 1, 20], [500, 90, 300], 16, 4, 2, 128, 128).fill()
    cache, batch = c.on_gpu(K)
    q = values(c.r, (22, 4, 128), "bf16")
    qd, o, ws = dev(q, torch.bfloat16), torch.empty((22, 4, 128), device="cuda"), c.workspace(K)
    K.kv_attn_paged(qd, cache, batch, o, ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        K.kv_attn_paged(qd, cache, batch, o, ws)
    for lens in ([500, 90, 300], [33, 1, 25], [2, 80, 20], [499, 0, 10]):
        batch.lengths.copy_(dev(np.asarray(lens, np.int32)))
        g.replay()
        torch.cuda.synchronize()
        c.lengths = np.asarray(lens, np.int32)
        check_attention(host(o), q, c, "f32")


def test_one_workspace_for_calls_of_every_shape(K):
    """One after another, on one workspace: results as on a fresh one."""
    import torch
    ws = torch.zeros(K.paged_workspace_bytes(1, 64, 128), dtype=torch.uint8, device="cuda")
    for i in (12, 1, 6, 8, 2):
        c = Case(K, 20 + i, *SHAPES[i]).fill()
        q, got = attend(K, c, ws=ws)
        check_attention(got, q, c, "f32")


def test_another_stream(K):
    import torch
    c = Case(K, 10, [1, 30], [700, 300], 32, 4, 2, 128, 128).fill()
    cache, batch = c.on_gpu(K)
    q = values(c.r, (31, 4, 128), "bf16")
    qd, o, ws = dev(q, torch.bfloat16), torch.empty((31, 4, 128), device="cuda"), c.workspace(K)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    K.kv_attn_paged(qd, cache, batch, o, ws, stream=s)
    s.synchronize()
    check_attention(host(o), q, c, "f32")


# ---------------------------------------------------------------------------------
def stored(got, want, name, what):
    want = np.asarray(want, np.float64)
    rms = np.sqrt(np.mean(want * want, -1, keepdims=True))
    step = np.abs(want) * HALF[name] if name == "f32" else \
        np.ldexp(0.5, np.floor(np.log2(np.maximum(np.abs(want), 1e-300))).astype(int) - 7)
    tol = step * (1 + 1e-6) + 1e-6 * rms
    assert (np.abs(got - want) <= tol).all(), f"{what}: {np.max(np.abs(got - want) / tol):.2f} of the tolerance"


ROPES = [("none", {}, 1), ("1d", {}, 1), ("sections", dict(sections=True), 4), ("2d", {}, 2), ("interleaved", dict(tail=64), 1),
         ("1d", dict(tail=20), 1)]


def append_case(K, seed, new, lengths, page, Hq, Hkv, Dk, Dv, cache, in_dtype, rope_i, norm, after, scale, fused, with_q=True, start_pos=0):
    import torch
    c = Case(K, seed, new, lengths, page, Hq, Hkv, Dk, Dv, cache=cache)
    T = int(c.start[-1])
    kind, opt, axes = ROPES[rope_i]
    secs = (Dk // 8,) * 4 if "sections" in opt else ()
    off = dict(rot_offset=Dk - opt["tail"], rot_dim=opt["tail"]) if "tail" in opt else {}
    q, k, v = (values(c.r, (T, h, d), in_dtype) for h, d in ((Hq, Dk), (Hkv, Dk), (Hkv, Dv)))
    qw, kw = ((1 + 0.1 * c.r.standard_normal(Dk)).astype(np.float32) for _ in range(2)) if norm else (None, None)
    pos = (start_pos + c.r.integers(0, 3000, (T, axes))).astype(np.int32)
    cache_t, batch = c.on_gpu(K)
    if fused:
        row = dev(np.concatenate([x.reshape(T, -1) for x in (q, k, v)], 1), dtype(in_dtype))
        qd, kd, vd = (t.unflatten(1, (h, d)) for t, h, d in
                      zip(row.split([Hq * Dk, Hkv * Dk, Hkv * Dv], 1), (Hq, Hkv, Hkv), (Dk, Dk, Dv)))
    else:
        qd, kd, vd = (dev(x, dtype(in_dtype)) for x in (q, k, v))
    qo = torch.full((T + 1, Hq, Dk), 7.0, dtype=dtype(cache), device="cuda")
    K.kv_cache_append_paged(qd if with_q else None, kd, vd, dev(pos), cache_t, batch, qo[:-1] if with_q else None,
                            K.Rope(kind, 1e6, secs, **off), rope_scale=K.RopeScale(*scale) if scale else None,
                            q_norm_w=None if qw is None else dev(qw), k_norm_w=None if kw is None else dev(kw),
                            norm_after_rope=after)
    torch.cuda.synchronize()
    ref = O.Rope(kind, 1e6, secs or None, **({} if not off else dict(rot_offset=off["rot_offset"], rot_dim=off["rot_dim"])))
    qx, kx = P.qk_step(q, pos, qw, 1e-6, ref, scale, after), P.qk_step(k, pos, kw, 1e-6, ref, scale, after)
    if with_q:
        stored(host(qo[:-1]), qx, cache, "q")
    assert (qo[-1] == 7).all()
    wk, wv = np.full(c.pool_k.shape, np.nan), np.full(c.pool_v.shape, np.nan)
    P.paged_append(kx, v, wk, wv, c.table, c.lengths, c.start, "f32")
    gk, gv = host(cache_t.k), host(cache_t.v)
    for got, want, what in ((gk, wk, "k"), (gv, wv, "v")):
        assert (np.isnan(got) == np.isnan(want)).all(), f"{what}: rows written are not those of the new tokens"
    for b in range(len(c.new)):
        for i in range(int(c.new[b])):
            slot, t = int(c.lengths[b] - c.new[b]) + i, int(c.start[b]) + i
            p, row = c.table[b, slot // page], slot % page
            stored(gk[p, :, row], kx[t], cache, "k")
            stored(gv[p, :, row], v[t], cache, "v")
    return c


@pytest.mark.parametrize("cache,in_dtype", [("bf16", "f32"), ("bf16", "bf16"), ("f32", "f32"), ("f32", "bf16")])
@pytest.mark.parametrize("rope_i", range(len(ROPES)))
def test_append(K, rope_i, cache, in_dtype):
    norm, after, scale = rope_i % 2 == 0, rope_i == 4, (4.0, 2048, 1.0, 4.0, 1.3) if rope_i in (1, 3, 4) else None
    append_case(K, rope_i, [1, 0, 7, 20], [33, 5, 7, 61], 16, 6, 3, 128, 128, cache, in_dtype, rope_i, norm, after, scale,
                fused=in_dtype == "bf16", start_pos=0 if rope_i else 100000)


@pytest.mark.parametrize("shape", [(16, 8, 64, 64), (4, 4, 192, 128), (5, 1, 256, 192), (3, 3, 64, 256)])
def test_append_head_dims(K, shape):
    append_case(K, 3, [3, 1], [40, 64], 32, *shape, "bf16", "f32", 1, True, False, None, False)


def test_append_far_positions_and_all_frequencies_divided(K):
    append_case(K, 4, [5], [9], 16, 4, 2, 128, 128, "f32", "f32", 1, True, False, (8.0, 0.0, 0.0, 0.0, 1.0), False, start_pos=3_000_000)


def test_append_without_queries(K):
    append_case(K, 5, [2, 3], [18, 3], 16, 4, 2, 128, 128, "bf16", "bf16", 1, True, False, None, False, with_q=False)


def test_append_of_thousands_of_tokens(K):
    """A token a warp: more tokens than four CTAs an SM, in uneven sequences, the last CTA not full."""
    new = [1, 2900, 0, 1999, 1]
    append_case(K, 6, new, [40, 3000, 5, 1999, 1], 128, 2, 1, 64, 64, "bf16", "bf16", 1, True, False, None, True)


def test_append_drops_what_has_no_page(K):
    """A page id outside the pool, and a device length below the new tokens: those rows are dropped, nothing else is touched."""
    import torch
    c = Case(K, 11, [3, 2], [18, 20], 16, 2, 2, 64, 64)
    c.table[0, 1] = 1000                                            # slots 16, 17 of the first sequence
    cache, _ = c.on_gpu(K)
    lens = np.array([18, 1], np.int32)                              # the second one's first token has slot -1
    batch = K.PagedBatch(dev(c.table), dev(lens), dev(c.start), c.lengths, c.start)
    k = torch.ones((5, 2, 64), device="cuda")
    K.kv_cache_append_paged(None, k, k, None, cache, batch, None, K.Rope("none"))
    torch.cuda.synchronize()
    got = host(cache.k)
    want = np.full(got.shape, np.nan)
    want[c.table[0, 0], :, 15] = 1
    want[c.table[1, 0], :, 0] = 1
    assert np.array_equal(got, want, equal_nan=True)


def test_a_prompt_in_chunks_then_tokens(K):
    """Append and attention together as a server calls them: ragged chunks, then single tokens, pages growing, one
    sequence joining late; every step's outputs against the definition over everything appended so far."""
    import torch
    r = np.random.default_rng(12)
    Hq, Hkv, D, page, W = 8, 2, 128, 16, 12
    n_pages = 40
    ids = r.permutation(n_pages).astype(np.int32)
    table = np.stack([ids[:W], ids[W:2 * W], ids[2 * W:3 * W]])
    cache = K.PagedKVCache.zeros(n_pages, Hkv, page, D)
    ws = torch.zeros(K.paged_workspace_bytes(Hkv, Hq, D), dtype=torch.uint8, device="cuda")
    w = [(1 + 0.1 * r.standard_normal(D)).astype(np.float32) for _ in range(2)]
    scale = (4.0, 64.0, 1.0, 4.0, 1.1)
    lengths = np.zeros(3, np.int32)
    pk, pv = np.zeros((n_pages, Hkv, page, D)), np.zeros((n_pages, Hkv, page, D))
    for new in ([40, 17, 0], [30, 1, 0], [1, 1, 70], [1, 1, 1], [1, 1, 1], [5, 0, 1]):
        new = np.array(new)
        lengths = (lengths + new).astype(np.int32)
        start = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        T = int(start[-1])
        q, k, v = (values(r, (T, h, D), "bf16") for h in (Hq, Hkv, Hkv))
        pos = np.concatenate([np.arange(L - n, L) for L, n in zip(lengths, new)]).astype(np.int32)[:, None]
        batch = K.PagedBatch(dev(table), dev(lengths), dev(start), lengths, start, table)
        qo = torch.empty((T, Hq, D), dtype=torch.bfloat16, device="cuda")
        K.kv_cache_append_paged(dev(q, torch.bfloat16), dev(k, torch.bfloat16), dev(v, torch.bfloat16), dev(pos), cache, batch,
                                qo, K.Rope("1d", 1e4), rope_scale=K.RopeScale(*scale), q_norm_w=dev(w[0]), k_norm_w=dev(w[1]))
        o = torch.empty((T, Hq, D), device="cuda")
        K.kv_attn_paged(qo, cache, batch, o, ws)
        torch.cuda.synchronize()
        kx = P.qk_step(k, pos, w[1], 1e-6, O.Rope("1d", 1e4), scale, False)
        P.paged_append(kx, v, pk, pv, table, lengths, start, "bf16")
        got = host(cache.k)
        step = np.ldexp(1.0, np.floor(np.log2(np.maximum(np.abs(pk), 1e-30))).astype(int) - 7)
        assert (np.abs(got - pk) <= step).all() and np.array_equal(host(cache.v), pv)    # a tie may fall either way
        ref, size = P.paged_attention(host(qo), got, pv, table, lengths, start)
        assert (np.abs(host(o) - ref) <= size * (2.0 ** -16 + 1e-5) + 1e-30).all()


def test_refusals_of_the_binding(K):
    import torch
    c = Case(K, 13, [1, 4], [20, 30], 16, 4, 2, 64, 64).fill()
    cache, batch = c.on_gpu(K)
    q, o, ws = torch.zeros((5, 4, 64), dtype=torch.bfloat16, device="cuda"), torch.zeros((5, 4, 64), device="cuda"), c.workspace(K)
    bad = [(q[:4], o), (q.float(), o), (q, o[:4]), (q.cpu(), o), (q.transpose(0, 1), o), (q, o.half()), (q[..., :32], o)]
    for qq, oo in bad:
        with pytest.raises(K.KvaError):
            K.kv_attn_paged(qq, cache, batch, oo, ws)
    with pytest.raises(K.KvaError):
        K.kv_attn_paged(q, cache, batch, o, ws[:100])
    for name, t in (("table", batch.table.long()), ("lengths", batch.lengths[:1]), ("token_start", batch.token_start[:2]),
                    ("table_host", c.table[:1]), ("lengths_host", c.lengths[:1])):
        args = dict(table=batch.table, lengths=batch.lengths, token_start=batch.token_start, lengths_host=c.lengths,
                    token_start_host=c.start, table_host=c.table)
        args[name] = t
        with pytest.raises(K.KvaError):
            K.kv_attn_paged(q, cache, K.PagedBatch(**args), o, ws)
    k = torch.zeros((5, 2, 64), device="cuda")
    pos = torch.zeros((5, 1), dtype=torch.int32, device="cuda")
    for args in ((None, k[:, :, ::2], k, pos), (None, k, k.double(), pos), (None, k, k, pos.long()), (None, k, k, pos[:4]),
                 (q, k, k, pos), (None, k.transpose(1, 2).contiguous().transpose(1, 2), k, pos), (None, k, k[:1].expand(5, 2, 64), pos)):
        with pytest.raises(K.KvaError):
            K.kv_cache_append_paged(*args, cache, batch, q, K.Rope("1d"))
    with pytest.raises(K.KvaError):
        K.PagedKVCache(cache.k[:, :, ::2], cache.v[:, :, ::2]).struct
    with pytest.raises(K.KvaError):
        K.PagedKVCache(cache.k, cache.v.float()).struct
