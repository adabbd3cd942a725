"""The serving operators over the paged cache (mpk_rope_table, mpk_kv_append,
mpk_prefix_attention, mpk_verify_drafts) against float64 forms, and what they
refuse."""
import ctypes
import math

import numpy as np
import pytest
import torch

import serving_ref as ref
from task_graph_runtime_gb300 import mpk

gpu = pytest.mark.gpu


# ------------------------------------------------------- refusals (no GPU)
FAKE = 1 << 20     # never followed: every call below is refused first


def _append(lib, shape=None, tok=None, kv=None, layer=0, q=FAKE, qs=256,
            k=FAKE, ks=128, v=FAKE, vs=128, qn=None, kn=None, eps=1e-6,
            rope=None, qo=FAKE, qos=256):
    ref_ = lambda x: ctypes.byref(x) if x is not None else None
    return lib.mpk_kv_append(ref_(shape), ref_(tok), ref_(kv), layer, q, qs,
                             k, ks, v, vs, qn, kn, eps, ref_(rope), qo, qos,
                             None, None)


def _parts(**kw):
    shape = mpk.AttnShape(4, 2, 64, 16, 8)
    tok = mpk.TokenBatch(2, 4, None, 2)
    kv = mpk._KVCache(FAKE, FAKE, FAKE, FAKE, 5)
    for k, v in kw.items():
        o = {"s": shape, "t": tok, "k": kv}[k[0]]
        setattr(o, k[2:], v)
    return dict(shape=shape, tok=tok, kv=kv)


INVALID, UNSUPPORTED = mpk.MPK_ERR_INVALID_ARG, mpk.MPK_ERR_UNSUPPORTED
BAD_PARTS = [
    (dict(s_n_q_heads=0), INVALID), (dict(s_n_q_heads=3), INVALID),
    (dict(s_n_kv_heads=0), INVALID), (dict(s_page_size=0), INVALID),
    (dict(s_max_pages_per_seq=0), INVALID), (dict(s_head_dim=96), UNSUPPORTED),
    (dict(s_page_size=1 << 20, s_max_pages_per_seq=1 << 20), UNSUPPORTED),
    (dict(s_page_size=1 << 20, s_max_pages_per_seq=1025), UNSUPPORTED),
    (dict(s_page_size=1 << 20, k_num_pages=2048), UNSUPPORTED),
    (dict(t_batch=0), INVALID), (dict(t_n_tokens=-1), INVALID),
    (dict(t_tokens_per_seq=3), INVALID), (dict(t_tokens_per_seq=-1), INVALID),
    (dict(t_batch=(1 << 20) + 1, t_tokens_per_seq=0), UNSUPPORTED),
    (dict(t_q_start=FAKE + 2), INVALID),
    (dict(k_k_pool=None), INVALID), (dict(k_v_pool=FAKE + 8), INVALID),
    (dict(k_page_table=None), INVALID), (dict(k_seq_lens=FAKE + 1), INVALID),
    (dict(k_num_pages=0), INVALID)]


@pytest.mark.parametrize("change,status", BAD_PARTS)
def test_append_and_attend_refuse_bad_shapes(mpk_lib, change, status):
    p = _parts(**change)
    assert _append(mpk_lib, **p) == status
    assert mpk_lib.mpk_prefix_attention(
        ctypes.byref(p["shape"]), ctypes.byref(p["tok"]), None,
        ctypes.byref(p["kv"]), 0, FAKE, 256, 0.0, FAKE + 4096, 256, None,
        FAKE, 1 << 40, None, None) == status


def test_append_refuses_bad_arguments(mpk_lib):
    ok = _parts()
    assert _append(mpk_lib) == INVALID
    for kw in (dict(layer=-1), dict(k=None), dict(v=FAKE + 8),
               dict(ks=120), dict(vs=132), dict(qs=252), dict(q=None),
               dict(qo=FAKE + 4), dict(qos=128), dict(qn=FAKE + 2),
               dict(kn=FAKE + 8), dict(eps=-1.0), dict(eps=math.nan),
               dict(rope=mpk._Rope(None, 8, 64, 0)),
               dict(rope=mpk._Rope(FAKE + 4, 8, 64, 0)),
               dict(rope=mpk._Rope(FAKE, 0, 64, 0)),
               dict(rope=mpk._Rope(FAKE, 8, -16, 0))):
        assert _append(mpk_lib, **ok, **kw) == INVALID, kw
    for rot in (24, 80):
        assert _append(mpk_lib, **ok, rope=mpk._Rope(FAKE, 8, rot, 0)) == \
            UNSUPPORTED
    # nothing to do is no error, whatever the tensors
    none = _parts(t_n_tokens=0, t_tokens_per_seq=0)
    assert _append(mpk_lib, **none, k=None, v=None, qo=None) == mpk.MPK_OK


def test_attend_refuses_bad_arguments(mpk_lib):
    p = _parts()
    r = [ctypes.byref(p[k]) for k in ("shape", "tok", "kv")]
    need = mpk_lib.mpk_prefix_attention_workspace(r[0], r[1], 1)
    assert need > 0
    good = dict(groups=mpk.PrefixGroups(1, FAKE, FAKE), layer=0, q=FAKE,
                qs=256, scale=0.0, out=FAKE + 4096, os=256, lse=None, ws=FAKE,
                n=need)

    def call(**kw):
        a = dict(good, **kw)
        return mpk_lib.mpk_prefix_attention(
            r[0], r[1], ctypes.byref(a["groups"]) if a["groups"] else None,
            r[2], a["layer"], a["q"], a["qs"], a["scale"], a["out"], a["os"],
            a["lse"], a["ws"], a["n"], None, None)
    for kw in (dict(layer=-1), dict(q=None), dict(q=FAKE + 8), dict(qs=248),
               dict(out=FAKE), dict(out=None), dict(os=260), dict(lse=2),
               dict(scale=math.inf), dict(scale=math.nan), dict(ws=None),
               dict(ws=FAKE + 16), dict(n=need - 1),
               dict(groups=mpk.PrefixGroups(0, FAKE, FAKE)),
               dict(groups=mpk.PrefixGroups(3, FAKE, FAKE)),
               dict(groups=mpk.PrefixGroups(1, None, FAKE)),
               dict(groups=mpk.PrefixGroups(1, FAKE, FAKE + 2))):
        assert call(**kw) == INVALID, kw
    assert mpk_lib.mpk_prefix_attention_workspace(r[0], r[1], 3) == 0
    assert mpk_lib.mpk_prefix_attention_workspace(None, r[1], 0) == 0


def test_rope_table_refuses_bad_arguments(mpk_lib):
    def call(first=0, n=4, out=FAKE, **kw):
        a = dict(rotary_dim=64, theta=1e4, scaling=0, factor=1.0, low=1.0,
                 high=4.0, old_ctx=8192.0, attn_factor=1.0)
        a.update(kw)
        return mpk_lib.mpk_rope_table(ctypes.byref(mpk.RopeScaling(**a)),
                                      first, n, out, None)
    for kw in (dict(out=None), dict(out=FAKE + 2), dict(first=-1), dict(n=-1),
               dict(rotary_dim=0), dict(rotary_dim=63), dict(theta=0.0),
               dict(scaling=4), dict(scaling=-1),
               dict(scaling=1, factor=0.0), dict(scaling=2, low=0.0),
               dict(scaling=2, low=4.0), dict(scaling=3, old_ctx=0.0),
               dict(scaling=3, theta=1.0)):
        assert call(**kw) == INVALID, kw
    assert call(n=0) == mpk.MPK_OK


def test_verify_refuses_bad_arguments(mpk_lib):
    tok = mpk.TokenBatch(2, 6, None, 3)
    need = mpk_lib.mpk_verify_drafts_workspace(ctypes.byref(tok), 100)
    assert need > 0
    base = dict(vocab=100, max_out=3, tokens=FAKE, logits=FAKE,
                logits_stride=100, draft=None, draft_stride=0,
                draft_is_logits=0, temperature=None, uniform=FAKE, noise=FAKE,
                noise_stride=100, n_accepted=FAKE, out_tokens=FAKE,
                logprobs=None, next_tokens=None, seq_lens=None,
                seq_lens_out=None)

    def call(t=tok, ws=FAKE, n=need, **kw):
        a = mpk.VerifyArgs(**dict(base, **kw))
        return mpk_lib.mpk_verify_drafts(ctypes.byref(t), ctypes.byref(a), ws,
                                         n, None, None)
    for kw in (dict(vocab=0), dict(max_out=0), dict(max_out=2),
               dict(tokens=None), dict(logits=None), dict(logits=FAKE + 2),
               dict(logits_stride=99), dict(draft=FAKE, draft_stride=99),
               dict(uniform=None), dict(noise=None), dict(noise_stride=99),
               dict(n_accepted=None), dict(out_tokens=None),
               dict(logprobs=FAKE + 1), dict(seq_lens=FAKE + 2),
               dict(ws=None), dict(ws=FAKE + 8), dict(n=need - 1)):
        assert call(**kw) == INVALID, kw
    assert call(max_out=129) == UNSUPPORTED
    big = mpk.TokenBatch(2, 65536, FAKE, 0)
    assert call(t=big) == UNSUPPORTED
    assert mpk_lib.mpk_verify_drafts_workspace(ctypes.byref(big), 100) == 0


def test_binding_refuses_before_it_calls():
    """What the GPU wrappers' tests refuse, with tensors of the CPU."""
    nat = mpk._native()
    shape, tok = mpk.AttnShape(4, 2, 64, 16, 4), mpk.TokenBatch(2, 2, None, 1)
    kv = mpk._KVCache()
    at = ctypes.addressof
    p = nat.paged(at(shape), at(tok), at(kv), None, None, 3, 0)
    x = torch.zeros(2, 128, dtype=torch.bfloat16)
    rest = (None, None, None, None, 1e-6, 0)
    assert "k must be bfloat16 [2, 128] on cuda:0" in nat.append(
        p, 0, None, x, x, *rest)
    assert "k must be a torch tensor" == nat.append(p, 0, None, [1], x, *rest)
    assert nat.append(p, 3, None, x, x, *rest) == "layer 3 of 3"
    assert "q must be bfloat16 [2, 256]" in nat.attend(
        p, 0, x, x, None, 0.0, 0, 0, 0)
    j = nat.judge(2, 3, 10, 4, None, 0, 0, 0)
    f = torch.zeros(3, 10)
    assert "multiple of the batch" in nat.verify(
        j, f, f, f, f, f, f, None, None, False, *[None] * 5, 0)
    assert "q_start must be a contiguous Int tensor of 3" in nat.verify(
        j, f, f, f, f, f, f, f, None, False, *[None] * 5, 0)
    for call in (nat.append, nat.attend, nat.verify, nat.paged, nat.judge):
        with pytest.raises(TypeError, match="arguments"):
            call(p)
    with pytest.raises(ValueError):              # another call's plan
        nat.verify(p, f, f, f, f, f, f, None, None, False, *[None] * 5, 0)
    with pytest.raises(TypeError):
        nat.append(p, "0", None, x, x, *rest)


def test_wrappers_refuse_tensors_of_the_cpu():
    k = torch.zeros(1, 2, 2, 16, 64, dtype=torch.bfloat16)
    kv = mpk.KVCache(k, k, torch.zeros(1, 2, dtype=torch.int32),
                     torch.zeros(1, dtype=torch.int32))
    with pytest.raises(mpk.MpkError, match="CUDA"):
        mpk.PagedBatch(kv, 4, 1)
    with pytest.raises(mpk.MpkError, match="CUDA"):
        mpk.DraftVerifier(1, 1, 10, 1, device="cpu")
    with pytest.raises(mpk.MpkError, match="CUDA"):
        mpk.Rope(torch.zeros(4, 8, 2), 16)
    with pytest.raises(mpk.MpkError, match="CUDA"):
        mpk.mpk_rope_table(16, 4, 1e4, device="cpu")


# ------------------------------------------------------------------ inputs
class Case:
    """A ragged batch over a paged cache on the GPU, with float64 copies."""

    def __init__(self, seed, n, ctx, hq=4, hkv=2, d=64, page=16, layers=2,
                 layer=1, groups=None, pad=0, spare=3, stale=None, wide=0):
        g = np.random.Generator(np.random.PCG64(seed))
        self.n, self.ctx, self.page, self.layer = n, ctx, page, layer
        self.hq, self.hkv, self.d = hq, hkv, d
        self.starts = np.concatenate([[0], np.cumsum(n)]).astype(int)
        self.T = int(self.starts[-1])
        B = len(n)
        cut, pre = groups if groups else ([0, B], [0])
        self.prefix = [pre[i] for i in range(len(pre))
                       for _ in range(cut[i], cut[i + 1])]
        self.first = [cut[i] for i in range(len(pre))
                      for _ in range(cut[i], cut[i + 1])]
        need = [-(-(c + m) // page) for c, m in zip(ctx, n)]
        cols = max(max(need), 1) + 1 + wide
        pages, rows = 0, []
        for b in range(B):
            share = self.prefix[b] // page if b != self.first[b] else 0
            own = max(need[b] - share, 0)
            rows.append((rows[self.first[b]][:share] if share else []) +
                        list(range(pages, pages + own)))
            pages += own
        ids = g.permutation(pages + spare)
        self.table = np.full((B, cols), -1, np.int32)
        for b, r in enumerate(rows):
            self.table[b, :len(r)] = ids[r]
        self.num_pages = pages + spare
        bf = lambda *s: torch.from_numpy(
            g.standard_normal(s, dtype=np.float32)).bfloat16()
        shape = (layers, self.num_pages, hkv, page, d)
        k, v = bf(*shape), bf(*shape)
        if stale is not None:
            # every slot that no live token owns
            live = np.zeros((self.num_pages, page), bool)
            for b in range(B):
                t = np.arange(ctx[b] + n[b])
                live[self.table[b, t // page], t % page] = True
            dead = torch.from_numpy(~live)[None, :, None, :, None]
            k.masked_fill_(dead, stale)
            v.masked_fill_(dead, stale)
        self.k, self.v = k.cuda(), v.cuda()
        self.q = bf(self.T + pad, hq * d).cuda()
        self.kv = mpk.KVCache(self.k, self.v,
                              torch.from_numpy(self.table).cuda(),
                              ref.as_dev(ctx, torch.int32))
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")
        kw = {}
        if groups:
            kw = dict(group_start=ref.as_dev(cut, torch.int32),
                      prefix_len=ref.as_dev(pre, torch.int32))
        self.plan = mpk.PagedBatch(
            self.kv, hq, self.T + pad,
            q_start=ref.as_dev(self.starts, torch.int32), status=self.status,
            **kw)
        self.g = g

    def attend(self, **kw):
        out = torch.full_like(self.q, 7.0)
        lse = torch.full((self.q.shape[0], self.hq), 7.0, device="cuda")
        self.plan.attend(self.layer, self.q, out, lse, **kw)
        torch.cuda.synchronize()
        return out, lse

    def check(self, out, lse, scale=None):
        q = ref.f64(self.q)[:self.T].reshape(self.T, self.hq, self.d)
        o, l, tol, ltol = ref.attend(
            q, ref.f64(self.k)[self.layer], ref.f64(self.v)[self.layer],
            self.table, self.page, self.ctx, self.starts, self.prefix,
            self.first, scale if scale else 1 / math.sqrt(self.d))
        got = ref.f64(out)[:self.T].reshape(o.shape)
        assert np.array_equal(np.isfinite(got), np.isfinite(o))
        fin = np.isfinite(o)
        over = (np.abs(got - o) - tol)[fin]
        assert over.size == 0 or over.max() <= 0, over.max()
        gl = ref.f64(lse)[:self.T]
        same = (gl == l) | (np.isnan(gl) & np.isnan(l))
        with np.errstate(invalid="ignore"):
            assert (same | (np.abs(gl - l) <= ltol)).all()
        # rows behind the last sequence are left as they were
        assert (out[self.T:] == 7.0).all() and (lse[self.T:] == 7.0).all()


# --------------------------------------------------------------- attention
ATTEND = {
    # one token against 0, 1 and many cached ones
    "single": dict(n=[1, 1, 1], ctx=[0, 1, 200]),
    "block_edges": dict(n=[1] * 6, ctx=[62, 63, 64, 127, 128, 129]),
    # drafts, an empty sequence in the middle, one at each end
    "ragged": dict(n=[0, 3, 1, 0, 8, 0], ctx=[5, 0, 70, 9, 61, 0], pad=3),
    "wide_group": dict(n=[2, 1], ctx=[30, 100], hq=16, hkv=1, d=128),
    "odd_group": dict(n=[1, 5], ctx=[3, 80], hq=6, hkv=2, d=32),
    "many_heads": dict(n=[1, 2], ctx=[40, 10], hq=8, hkv=8, d=128),
    # pages that end inside a tile, one-token pages
    "page7": dict(n=[3, 1], ctx=[100, 65], page=7),
    "page1": dict(n=[2], ctx=[70], page=1),
    "page100": dict(n=[2, 1], ctx=[250, 99], page=100),
    # a prompt chunk: more rows than a tile, causal inside
    "prompt": dict(n=[70, 1, 33], ctx=[0, 4, 100], d=128),
    "prefix": dict(n=[1, 1, 2, 1], ctx=[150, 129, 200, 128],
                   groups=([0, 4], [128])),
    "prefix_odd": dict(n=[1, 3, 1], ctx=[77, 90, 133], page=24,
                       groups=([0, 3], [77])),
    # groups of one, an empty prefix, a prefix and nothing else cached
    "groups": dict(n=[1, 2, 0, 1, 4], ctx=[64, 64, 80, 9, 31],
                   groups=([0, 2, 3, 4, 5], [64, 17, 0, 31])),
    "prefix_rows": dict(n=[1] * 40, ctx=[65 + i for i in range(40)], hq=8,
                        hkv=2, d=128, groups=([0, 40], [65])),
    "many": dict(n=[1] * 150, ctx=[3 * i for i in range(150)], d=32,
                 groups=([0, 50, 150], [0, 147])),
}

# Groups with more rows than a sequence.  A page table that could hold long
# prefixes (WIDE columns more) gives groups of more than 64 rows a kernel of
# their own.
WIDE = 100_000
PREFIX = {
    "one_block": dict(n=[1] * 20, ctx=[100] * 20, d=128, hq=8,
                      groups=([0, 20], [100])),
    "two_slots": dict(n=[1] * 50, ctx=[130] * 50, d=128, hq=8,
                      groups=([0, 50], [128])),
    "tiles": dict(n=[2] * 90, ctx=[300] * 90, d=128, hq=8,
                  groups=([0, 90], [257])),
    "d64": dict(n=[1] * 40, ctx=[270] * 40, d=64, hq=16, hkv=2, page=8,
                groups=([0, 40], [270])),
    "page24": dict(n=[1, 4] * 10, ctx=[205] * 20, d=64, page=24,
                   groups=([0, 20], [201])),
    "page128": dict(n=[3] * 12, ctx=[1000] * 12, d=128, page=128,
                    groups=([0, 12], [999])),
    "page64_long": dict(n=[1] * 16, ctx=[5000] * 16, d=128, page=64, hq=8,
                        hkv=2, groups=([0, 16], [4999])),
    "page100": dict(n=[1] * 16, ctx=[205] * 16, d=64, page=100, hq=8,
                    groups=([0, 16], [201])),
    "d32": dict(n=[1] * 16, ctx=[205] * 16, d=32, hq=8,
                groups=([0, 16], [201])),
    "several": dict(n=[1, 5, 0] * 20, ctx=[300 + i for i in range(60)], d=64,
                    hq=12, hkv=4, groups=([0, 7, 8, 33, 60],
                                          [300, 0, 1, 129]), pad=5),
}


@gpu
@pytest.mark.parametrize("wide", [0, WIDE])
@pytest.mark.parametrize("name", sorted(PREFIX))
def test_attend_prefix_launches(name, wide):
    c = Case(41, wide=wide, **PREFIX[name])
    out, lse = c.attend()
    assert c.status.item() == 0
    c.check(out, lse)
    again, la = c.attend()
    assert torch.equal(out, again) and torch.equal(lse, la)


@gpu
@pytest.mark.parametrize("name", ["tiles", "d64", "page100"])
@pytest.mark.parametrize("stale", [math.nan, -math.inf])
@pytest.mark.parametrize("wide", [0, WIDE])
def test_attend_prefix_launches_stale_slots(name, stale, wide):
    c = Case(42, stale=stale, wide=wide, **PREFIX[name])
    out, lse = c.attend()
    c.check(out, lse)
    assert torch.isfinite(out[:c.T].float()).all()


@gpu
@pytest.mark.parametrize("scale", [2.0, -0.3])
@pytest.mark.parametrize("wide", [0, WIDE])
@pytest.mark.parametrize("name", ["page64_long", "two_slots"])
def test_attend_prefix_launches_scale(scale, wide, name):
    # large scores: the running maximum grows often; a negative scale
    c = Case(43, wide=wide, **PREFIX[name])
    out, lse = c.attend(scale=scale)
    c.check(out, lse, scale)


@gpu
@pytest.mark.parametrize("wide", [0, WIDE])
def test_attend_prefix_launches_growing_maximum(wide):
    # keys that grow along the prefix: every block raises the maximum
    c = Case(44, wide=wide, **PREFIX["tiles"])
    t = torch.arange(300, device="cuda").float().div(40)
    for b in [0]:
        row = torch.from_numpy(c.table[b].astype(np.int64)).cuda()
        pg, sl = row[torch.arange(300).cuda() // 16], torch.arange(300) % 16
        k = c.k[c.layer, pg, :, sl].float() * t[:, None, None]
        c.k[c.layer, pg, :, sl] = k.bfloat16()
    out, lse = c.attend()
    c.check(out, lse)


@gpu
@pytest.mark.parametrize("wide", [0, WIDE])
def test_attend_prefix_launches_missing_page(wide):
    c = Case(45, n=[1] * 40, ctx=[200] * 40, d=128, hq=8, wide=wide,
             groups=([0, 20, 40], [128, 128]))
    want, _ = c.attend()
    c.kv.page_table[0, 3] = -1
    out, _ = c.attend()
    assert c.status.item() == mpk.MPK_ERR_KV_PAGE
    assert torch.equal(out[20:], want[20:])


@gpu
@pytest.mark.parametrize("name", sorted(ATTEND))
def test_attend(name):
    c = Case(11, **ATTEND[name])
    out, lse = c.attend()
    assert c.status.item() == 0
    c.check(out, lse)


@gpu
@pytest.mark.parametrize("seed", range(6))
def test_attend_random(seed):
    g = np.random.Generator(np.random.PCG64(seed))
    B = int(g.integers(1, 30))
    G = int(g.integers(1, min(B, 4) + 1))
    cut = [0] + sorted(g.choice(np.arange(1, B), G - 1, replace=False).tolist()
                       ) + [B]
    pre = [int(g.integers(0, 300)) for _ in range(G)]
    of = [k for k in range(G) for _ in range(cut[k], cut[k + 1])]
    hkv = int(g.choice([1, 2, 4]))
    c = Case(100 + seed, n=[int(x) for x in g.integers(0, 6, B)],
             ctx=[pre[k] + int(g.integers(0, 200)) for k in of],
             hq=hkv * int(g.choice([1, 2, 3, 4, 8])), hkv=hkv,
             d=int(g.choice([32, 64, 128])), page=int(g.integers(1, 70)),
             groups=(cut, pre), pad=int(g.integers(0, 3)))
    if c.T == 0:
        pytest.skip("no rows drawn")
    out, lse = c.attend()
    assert c.status.item() == 0
    c.check(out, lse)


@gpu
@pytest.mark.parametrize("stale", [math.nan, math.inf, -math.inf, 3e38])
@pytest.mark.parametrize("groups", [None, ([0, 3], [70])])
def test_attend_stale_slots_do_not_reach_a_row(stale, groups):
    c = Case(5, n=[1, 3, 1], ctx=[70, 80, 129], page=48, stale=stale,
             groups=groups)
    out, lse = c.attend()
    c.check(out, lse)
    assert torch.isfinite(out[:c.T].float()).all()


@gpu
@pytest.mark.parametrize("page", [15, 16, 17, 20, 30, 47, 63, 94])
@pytest.mark.parametrize("d", [32, 64, 128])
def test_attend_pages_that_end_inside_eight_keys(page, d):
    # keys come eight at a time but where a page ends between them; contexts
    # at and around the pages' ends, a prefix that ends there too
    ctx = [3 * page + i for i in (-2, -1, 0, 1, 7, 8)]
    c = Case(21, n=[1, 2, 1, 3, 1, 9], ctx=ctx, page=page, d=d, hq=8, hkv=2,
             groups=([0, 3, 6], [3 * page - 2, 2 * page + 5]), stale=math.nan)
    out, lse = c.attend()
    assert c.status.item() == 0
    c.check(out, lse)
    assert torch.isfinite(out[:c.T].float()).all()


@gpu
@pytest.mark.parametrize("bad", [-1, 1 << 20])
@pytest.mark.parametrize("col", [0, 1, 2])
def test_attend_reports_a_bad_page_inside_eight_keys(bad, col):
    c = Case(22, n=[1, 1], ctx=[50, 50], page=21)
    c.kv.page_table[1, col] = bad
    out, lse = c.attend()
    assert c.status.item() == mpk.MPK_ERR_KV_PAGE
    want, wl = Case(22, n=[1, 1], ctx=[50, 50], page=21).attend()
    assert torch.equal(out[0], want[0]) and torch.equal(lse[0], wl[0])


@gpu
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("n", [4, 40])
def test_attend_values_of_later_tokens_do_not_reach_earlier_rows(bad, n):
    # V of the second to last new token: only it and the last one see it
    c = Case(6, n=[n], ctx=[50], d=128)
    t = 50 + n - 2
    page, slot = c.table[0, t // c.page], t % c.page
    c.v[c.layer, page, :, slot, 5] = bad
    out, lse = c.attend()
    o = out.float().view(c.T, c.hq, c.d)
    assert torch.isfinite(o[:n - 2]).all()
    assert not torch.isfinite(o[n - 2:, :, 5]).any()
    clean = torch.ones(c.d, dtype=torch.bool)
    clean[5] = False
    assert torch.isfinite(o[:, :, clean]).all()
    if bad != bad:
        assert torch.isnan(o[n - 2:, :, 5]).all()
    else:
        assert (o[n - 2:, :, 5] == bad).all()
    c.v[c.layer, page, :, slot, 5] = 0.5
    again, _ = c.attend()
    assert torch.equal(out[:n - 2], again[:n - 2])


@gpu
def test_attend_keys_that_are_not_finite():
    # a NaN key makes the rows that see it NaN, and no others
    c = Case(7, n=[3, 1], ctx=[20, 30])
    c.k[c.layer, c.table[0, 22 // 16], 0, 22 % 16, 1] = math.nan
    out, lse = c.attend()
    o = out.float().view(c.T, c.hq, c.d)
    assert torch.isfinite(o[:2]).all() and torch.isfinite(o[3]).all()
    assert torch.isnan(o[2, :2]).all() and torch.isnan(lse[2, :2]).all()
    assert torch.isfinite(o[2, 2:]).all()


@gpu
@pytest.mark.parametrize("scale", [1.0, 0.01, -0.2])
def test_attend_scale(scale):
    c = Case(8, n=[2, 1], ctx=[90, 10], groups=([0, 2], [10]))
    out, lse = c.attend(scale=scale)
    c.check(out, lse, scale)


@gpu
def test_attend_rounds_no_large_score_away():
    # scores of some hundreds: the softmax is one-hot or nearly so
    c = Case(9, n=[1, 4], ctx=[200, 64], d=128)
    c.q *= 40
    out, lse = c.attend()
    c.check(out, lse)


@gpu
def test_attend_strided_rows_and_three_dimensions():
    c = Case(10, n=[2, 1], ctx=[33, 66], hq=4, hkv=2, d=64)
    want, wl = c.attend()
    big = torch.zeros(c.T, 4 * 64 + 40, dtype=torch.bfloat16, device="cuda")
    big[:, 8:8 + 256] = c.q
    out = torch.full((c.T, 300 * 8), 7.0, dtype=torch.bfloat16, device="cuda")
    c.plan.attend(c.layer, big[:, 8:264], out[:, 16:272])
    assert torch.equal(out[:, 16:272], want)
    assert (out[:, :16] == 7).all() and (out[:, 272:] == 7).all()
    o3 = torch.empty(c.T, 4, 64, dtype=torch.bfloat16, device="cuda")
    c.plan.attend(c.layer, c.q.view(c.T, 4, 64), o3)
    assert torch.equal(o3.view(c.T, -1), want)


@gpu
def test_attend_same_bits_every_time():
    c = Case(12, n=[1] * 20, ctx=[400 + 7 * i for i in range(20)],
             groups=([0, 20], [390]), d=128, hq=8)
    a, la = c.attend()
    for _ in range(5):
        b, lb = c.attend()
        assert torch.equal(a, b) and torch.equal(la, lb)


@gpu
def test_attend_reports_missing_pages():
    c = Case(13, n=[1, 1, 1], ctx=[40, 40, 40])
    want, wl = c.attend()
    c.kv.page_table[1, 1] = -1
    out, lse = c.attend()
    assert c.status.item() == mpk.MPK_ERR_KV_PAGE
    for b in (0, 2):
        assert torch.equal(out[b], want[b])
    c.status.zero_()
    c.kv.page_table[1, 1] = c.num_pages       # past the pool
    c.attend()
    assert c.status.item() == mpk.MPK_ERR_KV_PAGE
    c.status.zero_()
    c.kv.page_table[1, 1] = int(c.table[1, 1])
    c.kv.seq_lens[2] = 10 ** 6                # past the table's columns
    out, lse = c.attend()
    assert c.status.item() == mpk.MPK_ERR_KV_PAGE
    assert torch.equal(out[:2], want[:2])
    c.status.zero_()
    c.kv.seq_lens[2] = -5
    c.attend()
    assert c.status.item() == mpk.MPK_ERR_KV_PAGE


@gpu
def test_attend_reports_a_sequence_shorter_than_its_prefix():
    c = Case(14, n=[1, 1, 1], ctx=[100, 100, 30],
             groups=([0, 2, 3], [64, 10]))
    want, _ = c.attend()
    assert c.status.item() == 0
    c.kv.seq_lens[1] = 63
    out, _ = c.attend()
    assert c.status.item() == mpk.MPK_ERR_INVALID_ARG
    assert torch.equal(out[2], want[2])


@gpu
@pytest.mark.parametrize("cut", [[1, 3], [0, 2], [2, 2]])
def test_attend_reports_sequences_outside_the_groups(cut):
    c = Case(18, n=[1, 2, 1], ctx=[70, 70, 70], groups=([0, 3], [64]))
    c.plan._keep[1].copy_(ref.as_dev(cut, torch.int32))
    c.attend()
    assert c.status.item() == mpk.MPK_ERR_INVALID_ARG


@gpu
@pytest.mark.parametrize("starts", [[0, 9, 0, 9, 0], [5, 4, 3, 2, 1],
                                    [-3, 2, 99, 1 << 30, 7]])
def test_attend_stays_inside_its_memory_with_bad_starts(starts):
    # results are unspecified; nothing outside the arguments is touched
    c = Case(15, n=[2, 2, 2, 3], ctx=[64] * 4, groups=([0, 4], [64]))
    c.plan._keep[0].copy_(ref.as_dev(starts, torch.int32))
    k, v = c.k.clone(), c.v.clone()
    c.attend()
    assert torch.equal(c.k, k) and torch.equal(c.v, v)


@gpu
def test_attend_on_another_stream_and_in_a_graph():
    c = Case(16, n=[1, 4, 2], ctx=[64, 100, 300], groups=([0, 3], [64]))
    want, wl = c.attend()
    s = torch.cuda.Stream()
    out, lse = torch.zeros_like(want), torch.zeros_like(wl)
    s.wait_stream(torch.cuda.current_stream())
    c.plan.attend(c.layer, c.q, out, lse, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(out, want) and torch.equal(lse, wl)
    g = torch.cuda.CUDAGraph()
    out.zero_()
    with torch.cuda.graph(g):
        c.plan.attend(c.layer, c.q, out, lse)
    # the replay reads the lengths that the arrays hold then
    c.kv.seq_lens.sub_(ref.as_dev([0, 7, 100], torch.int32))
    g.replay()
    torch.cuda.synchronize()
    c.ctx = [64, 93, 200]
    c.check(out, lse)


@gpu
def test_plan_keeps_the_tensors_it_was_given():
    c = Case(19, n=[1, 2], ctx=[33, 20])
    want, wl = c.attend()
    c.kv.seq_lens = torch.full((2,), 10 ** 6, dtype=torch.int32,
                               device="cuda")
    c.kv.page_table = torch.full_like(c.kv.page_table, -1)
    out, lse = c.attend()
    assert torch.equal(out, want) and torch.equal(lse, wl)


@gpu
def test_attend_wrapper_refusals():
    c = Case(17, n=[1], ctx=[4])
    out = torch.empty_like(c.q)
    for bad in (c.q.float(), c.q[:, :-8], c.q.t(), c.q.cpu()):
        with pytest.raises(mpk.MpkError):
            c.plan.attend(0, bad, out)
        with pytest.raises(mpk.MpkError):
            c.plan.attend(0, c.q, bad)
    with pytest.raises(mpk.MpkError):
        c.plan.attend(2, c.q, out)
    with pytest.raises(mpk.MpkError):
        c.plan.attend(0, c.q, out, lse=torch.empty(1, device="cuda"))
    with pytest.raises(mpk.MpkError):
        c.plan.attend(0, c.q, c.q)
    with pytest.raises(mpk.MpkError):
        mpk.PagedBatch(c.kv, 4, 1, group_start=c.kv.seq_lens)
    with pytest.raises(mpk.MpkError):
        mpk.PagedBatch(mpk.KVCache(c.k.float(), c.v, c.kv.page_table,
                                   c.kv.seq_lens), 4, 1)


@gpu
def test_wrapper_refusals_name_the_argument():
    c = Case(20, n=[1, 1], ctx=[4, 9], d=64, hq=4, hkv=2)
    W = c.hq * c.d
    q, k = c.q.clone(), torch.zeros(2, 128, dtype=torch.bfloat16,
                                    device="cuda")
    w = torch.ones(64, dtype=torch.bfloat16, device="cuda")
    args = (0, q, k, k)

    def refused(what, **kw):
        with pytest.raises(mpk.MpkError, match=what):
            c.plan.append(*[kw.pop(n, x) for n, x in zip(
                ("layer", "q", "k", "v"), args)], **kw)
    refused("layer 2", layer=2)
    refused("layer -1", layer=-1)
    for bad in (k.float(), k[:1], k[:, :120], k.cpu(), k.t(), [1.0], None,
                k.view(2, 4, 32), k.repeat(1, 2)[:, ::2], k.to_sparse()):
        refused("k must", k=bad)
        refused("v must", v=bad)
    refused("q must", q=q[:, 8:], q_out=q)
    refused("q_out must", q_out=q.float())
    refused("q_out without q", q=None, q_out=q)
    for bad in (w[:63], w.float(), w.cpu(), w.repeat(2)[::2], 1):
        refused("q_norm must", q_norm=bad)
        refused("k_norm must", k_norm=bad)
    with pytest.raises(TypeError):
        c.plan.append(0, q, k, k, eps="much")
    with pytest.raises(TypeError):
        c.plan.append("0", q, k, k)
    with pytest.raises(AttributeError):
        c.plan.append(0, q, k, k, stream=1.5)
    # heads apart, rows longer than they need be, a stream by name
    c.k.zero_()
    c.v.zero_()
    x = torch.randn(3, 3 * W).bfloat16().cuda()
    k3, v2 = x[:, :128].view(3, 2, 64), x[:, 200:328]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    c.plan.append(0, None, k3, v2, stream=s)
    s.synchronize()
    c.plan.append(1, None, k3, v2, stream=s.cuda_stream)
    s.synchronize()
    assert torch.equal(c.k[0], c.k[1]) and torch.equal(c.v[0], c.v[1])
    assert c.k[0].any() and c.v[0].any()


@gpu
def test_verify_wrapper_refusals_name_the_argument():
    f, i = torch.float32, torch.int32
    z = lambda *s, t=f: torch.zeros(*s, dtype=t, device="cuda")
    v = mpk.DraftVerifier(2, 5, 40, 3)
    good = dict(tokens=z(5, t=i), logits=z(5, 40), uniform=z(5),
                noise=z(2, 40) + 1, n_accepted=z(2, t=i),
                out_tokens=z(2, 3, t=i), q_start=torch.tensor(
                    [0, 3, 5], dtype=i, device="cuda"))
    v.verify(**good)

    def refused(what, **kw):
        with pytest.raises(mpk.MpkError, match=what):
            v.verify(**{**good, **kw})
    refused("n_tokens must be a multiple", q_start=None)
    for name, t in good.items():
        refused(name, **{name: t.cpu()})
        refused(name, **{name: t[:-1]})
        refused(name, **{name: t.double()})
    for name in ("logits", "noise", "draft"):
        refused(name, **{name: z(5, 41)})
        refused(name, **{name: z(5, 80)[:, ::2]})
    for name in ("temperature", "logprobs"):
        refused(name, **{name: z(1)})
    for name in ("next_tokens", "seq_lens", "seq_lens_out"):
        refused(name, **{name: z(2)})
    for name in ("tokens", "uniform", "n_accepted", "out_tokens"):
        refused("INVALID_ARG", **{name: None})      # the C call's own check
    refused("logits must be a torch tensor", logits=None)


# ------------------------------------------------------------------ append
APPEND = {
    "one": dict(n=[1], ctx=[0]),
    "ragged": dict(n=[0, 3, 1, 0, 9], ctx=[5, 0, 70, 9, 61], pad=2),
    "norm": dict(n=[1, 2, 5], ctx=[130, 15, 16], norm=True, d=128, hq=8),
    "interleaved": dict(n=[2, 7], ctx=[3, 40], inter=True),
    "partial": dict(n=[4, 1], ctx=[12, 31], rot=32, d=128),
    "partial_inter": dict(n=[4, 1], ctx=[12, 31], rot=16, inter=True),
    "d32": dict(n=[3, 3], ctx=[0, 20], d=32, hq=6, norm=True),
    "no_rope": dict(n=[3, 1], ctx=[2, 2], rot=0, norm=True),
    "page5": dict(n=[11, 1], ctx=[2, 9], page=5),
    "prompt": dict(n=[300, 150], ctx=[0, 37], d=128, hq=8, norm=True),
    "no_q": dict(n=[2, 3], ctx=[8, 8], q=False, norm=True),
}


def _append_case(seed, n, ctx, norm=False, inter=False, rot=None, q=True,
                 pad=0, layer=1, **kw):
    c = Case(seed, n=n, ctx=ctx, pad=pad, layer=layer, **kw)
    rot = c.d if rot is None else rot
    bf = lambda *s: torch.from_numpy(c.g.standard_normal(
        s, dtype=np.float32)).bfloat16().cuda()
    W = (c.hq + 2 * c.hkv) * c.d
    qkv = bf(c.T + pad, W)
    rope = mpk.Rope(mpk.mpk_rope_table(rot, max(ctx) + max(n), 1e4), rot,
                    inter) if rot else None
    qn = (1 + 0.1 * bf(c.d).float()).bfloat16() if norm else None
    kn = (1 + 0.1 * bf(c.d).float()).bfloat16() if norm else None
    k0, v0 = c.k.clone(), c.v.clone()
    qo = torch.full((c.T + pad, c.hq * c.d), 7.0, dtype=torch.bfloat16,
                    device="cuda") if q else None
    a, b = c.hq * c.d, (c.hq + c.hkv) * c.d
    c.plan.append(layer, qkv[:, :a] if q else None, qkv[:, a:b], qkv[:, b:],
                  rope, q_out=qo, q_norm=qn, k_norm=kn, eps=1e-5)
    torch.cuda.synchronize()
    return c, qkv, rot, qn, kn, k0, v0, qo


@gpu
@pytest.mark.parametrize("name", sorted(APPEND))
def test_append(name):
    kw = APPEND[name]
    c, qkv, rot, qn, kn, k0, v0, qo = _append_case(21, **kw)
    assert c.status.item() == 0
    inter, norm = kw.get("inter", False), kw.get("norm", False)
    x = ref.f64(qkv)[:c.T].reshape(c.T, c.hq + 2 * c.hkv, c.d)
    pos = np.array([c.ctx[b] + i for b in range(len(c.n))
                    for i in range(c.n[b])], float)
    q, k, v = (x[:, :c.hq], x[:, c.hq:c.hq + c.hkv], x[:, c.hq + c.hkv:])

    def want(h, w):
        if norm:
            h = ref.rms(h, ref.f64(w), 1e-5)
        y, mag = ref.rotate(h, pos, ref.inv_freq(rot, 1e4) if rot else
                            np.zeros(0), rot, inter)
        # the norm's own rounding reaches a rotated value through both
        # members of its pair; fp32 sums and products besides
        fp = 16 * ref.F32 * mag
        return y, (ref.BF * mag * 1.01 if norm else 0) + fp + \
            ref.BF * np.abs(y) * 1.01
    k1, v1 = k0.clone(), v0.clone()
    yk, tk = want(k, kn)
    got_k = ref.f64(c.k)
    for b in range(len(c.n)):
        for i in range(c.n[b]):
            t, p = c.starts[b] + i, c.ctx[b] + i
            pg, sl = int(c.table[b, p // c.page]), p % c.page
            assert (np.abs(got_k[1, pg, :, sl] - yk[t]) <= tk[t]).all()
            k1[1, pg, :, sl] = c.k[1, pg, :, sl]
            v1[1, pg, :, sl] = qkv[t, (c.hq + c.hkv) * c.d:].view(c.hkv, c.d)
    # v bit for bit, and nothing else in either pool has changed
    assert torch.equal(c.v, v1) and torch.equal(c.k, k1)
    if qo is not None:
        yq, tq = want(q, qn)
        got = ref.f64(qo)[:c.T].reshape(yq.shape)
        assert (np.abs(got - yq) <= tq).all()
        assert (qo[c.T:] == 7).all()


@gpu
def test_append_values_keep_their_bits():
    # payloads of NaNs, infinities, signed zeros; q and k too when nothing is
    # done to them
    c, qkv, *_ = _append_case(22, n=[4], ctx=[3], rot=0)
    bits = torch.arange(qkv.numel(), device="cuda").remainder(65536).to(
        torch.int32).to(torch.int16)
    raw = bits.view(torch.bfloat16).view_as(qkv)
    a, b = c.hq * c.d, (c.hq + c.hkv) * c.d
    qo = torch.empty_like(raw[:, :a])
    c.plan.append(0, raw[:, :a], raw[:, a:b], raw[:, b:], q_out=qo)
    i16 = lambda t: t.contiguous().view(torch.int16)
    assert torch.equal(i16(qo), i16(raw[:, :a]))
    t = np.arange(3, 7)
    pg, sl = c.table[0, t // 16].tolist(), (t % 16).tolist()
    assert torch.equal(i16(c.k[0, pg, :, sl].flatten(1)), i16(raw[:, a:b]))
    assert torch.equal(i16(c.v[0, pg, :, sl].flatten(1)), i16(raw[:, b:]))


@gpu
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("d", [32, 64, 128])
def test_append_rotation_rounds_each_operation(inter, d):
    # products and the sum of a pair are fp32 operations of their own, as in
    # the decode step: the result is the same to the last bit
    c, qkv, rot, qn, kn, k0, v0, qo = _append_case(25, n=[40, 7], ctx=[9, 200],
                                                   inter=inter, d=d)
    pos = np.array([9 + i for i in range(40)] + [200 + i for i in range(7)])
    table = mpk.mpk_rope_table(d, 240, 1e4).cpu().numpy()[pos]
    x = qkv[:, :c.hq * d].float().cpu().numpy().reshape(-1, c.hq, d)
    cs, sn = table[:, None, :, 0], table[:, None, :, 1]
    a, b = (x[..., 0::2], x[..., 1::2]) if inter else (x[..., :d // 2],
                                                       x[..., d // 2:])
    lo, hi = a * cs - b * sn, b * cs + a * sn       # numpy: no fusing
    y = (np.stack([lo, hi], -1).reshape(x.shape) if inter else
         np.concatenate([lo, hi], -1))
    want = torch.from_numpy(y).bfloat16().reshape(-1, c.hq * d)
    assert torch.equal(qo.cpu(), want)


@gpu
def test_append_in_place_and_separate_tensors():
    c, qkv, rot, qn, kn, k0, v0, qo = _append_case(23, n=[2, 5], ctx=[6, 1],
                                                   norm=True)
    k1 = c.k.clone()
    a, b = c.hq * c.d, (c.hq + c.hkv) * c.d
    q, k, v = (qkv[:, :a].contiguous(), qkv[:, a:b].contiguous(),
               qkv[:, b:].contiguous())
    c.k.copy_(k0)
    rope = mpk.Rope(mpk.mpk_rope_table(64, 11, 1e4), 64)
    c.plan.append(1, q, k, v, rope, q_out=q, q_norm=qn, k_norm=kn, eps=1e-5)
    assert torch.equal(q, qo) and torch.equal(c.k, k1)


@gpu
def test_append_reports_errors_and_skips_the_token():
    c, qkv, *_ = _append_case(24, n=[1, 1, 1], ctx=[4, 20, 4])
    a, b = c.hq * c.d, (c.hq + c.hkv) * c.d
    args = (qkv[:, :a], qkv[:, a:b], qkv[:, b:])
    short = mpk.Rope(mpk.mpk_rope_table(64, 20, 1e4), 64)
    qo = torch.full((3, a), 7.0, dtype=torch.bfloat16, device="cuda")
    k0 = c.k.clone()
    c.plan.append(0, *args, short, q_out=qo)       # position 20 of 20
    assert c.status.item() == mpk.MPK_ERR_INVALID_ARG
    assert (qo[1] == 7).all() and not (qo[0] == 7).all()
    assert torch.equal(c.k[0, c.table[1, 1]], k0[0, c.table[1, 1]])
    for bad in (-1, c.num_pages):
        c.status.zero_()
        c.kv.page_table[1, 1] = bad
        c.k.zero_()
        k0 = c.k.clone()
        c.plan.append(1, *args)
        assert c.status.item() == mpk.MPK_ERR_KV_PAGE
        diff = (c.k != k0).flatten(2).any(-1)
        assert not diff[0].any() and diff[1].sum() == 2
    c.status.zero_()
    c.kv.page_table[1, 1] = int(c.table[1, 1])
    for bad in (-1, 10 ** 9):
        c.kv.seq_lens[0] = bad
        c.status.zero_()
        c.plan.append(1, *args)
        assert c.status.item() == mpk.MPK_ERR_KV_PAGE


@gpu
@pytest.mark.parametrize("kind", ["plain", "linear", "bands", "ramp"])
@pytest.mark.parametrize("theta", [1e4, 5e5])
def test_rope_table(kind, theta):
    first, n, rot = 1_000_000, 33, 128
    kw = dict(factor=8.0, low=1.0, high=4.0 if kind == "bands" else 32.0,
              old_ctx=8192.0)
    t = mpk.mpk_rope_table(rot, n, theta, first, dict(
        plain=0, linear=1, bands=2, ramp=3)[kind], attn_factor=1.25, **kw)
    f = ref.inv_freq(rot, theta, kind, kw["factor"], kw["low"], kw["high"],
                     kw["old_ctx"])
    ang = (first + np.arange(n))[:, None] * f
    want = np.stack([np.cos(ang), np.sin(ang)], -1) * 1.25
    # a frequency to a few 2^-53, times a million, plus one rounding of 1.25
    assert np.abs(ref.f64(t) - want).max() <= 8 * 2.0 ** -53 * 1.1e6 + \
        1.25 * ref.F32


# ------------------------------------------------------------------ verify
def _verify_case(seed, rows, vocab, kind, temp, near=0.7, pad=0, extra=0):
    g = np.random.Generator(np.random.PCG64(seed))
    starts = np.concatenate([[0], np.cumsum(rows)]).astype(int)
    T, B = int(starts[-1]), len(rows)
    logits = (2 * g.standard_normal((T, vocab))).astype(np.float32)
    dl = (logits + near * g.standard_normal((T, vocab))).astype(np.float32)
    temp = np.broadcast_to(np.float32(temp), (B,)).copy()
    draft = dl
    if kind == "probs":
        t = np.repeat(np.where(temp > 0, temp, 1), rows)[:, None]
        e = np.exp((dl.astype(float) - dl.max(-1, keepdims=True)) / t)
        draft = (e / e.sum(-1, keepdims=True)).astype(np.float32)
    tokens = g.integers(0, vocab, T).astype(np.int32)
    for b in range(B):
        for r in range(starts[b], starts[b + 1] - 1):
            tokens[r + 1] = np.argmax(dl[r]) if temp[b] <= 0 else np.argmax(
                dl[r] / temp[b] - np.log(g.exponential(size=vocab)))
    return dict(starts=starts, T=T, B=B, vocab=vocab, kind=kind, temp=temp,
                logits=logits, draft=None if kind == "none" else draft,
                tokens=tokens, pad=pad,
                uniform=g.random(T, dtype=np.float32),
                noise=g.exponential(size=(B, vocab)).astype(np.float32),
                max_out=max(int(max(rows)), 1) + extra,
                lens=g.integers(0, 99, B).astype(np.int32))


def _verify_run(c, temperature=True, **kw):
    f, i = torch.float32, torch.int32
    T, B, mo = c["T"] + c["pad"], c["B"], c["max_out"]

    def rows(x, dt):
        t = ref.as_dev(x, dt)
        return torch.cat([t, torch.zeros((c["pad"],) + t.shape[1:], dtype=dt,
                                         device="cuda")])
    o = dict(acc=torch.full((B,), 99, dtype=i, device="cuda"),
             out=torch.full((B, mo), 99, dtype=i, device="cuda"),
             lp=torch.full((B, mo), 99.0, device="cuda"),
             nxt=torch.full((B,), 99, dtype=i, device="cuda"),
             lens=ref.as_dev(c["lens"], i))
    st = torch.zeros(1, dtype=i, device="cuda")
    v = mpk.DraftVerifier(B, T, c["vocab"], mo, status=st)
    v.verify(rows(c["tokens"], i), rows(c["logits"], f), rows(c["uniform"], f),
             ref.as_dev(c["noise"], f), o["acc"], o["out"],
             q_start=ref.as_dev(c["starts"], i),
             draft=None if c["draft"] is None else rows(c["draft"], f),
             draft_is_logits=c["kind"] == "logits",
             temperature=ref.as_dev(c["temp"], f) if temperature else None,
             logprobs=o["lp"], next_tokens=o["nxt"], seq_lens=o["lens"],
             seq_lens_out=o["lens"], **kw)
    torch.cuda.synchronize()
    assert st.item() == 0
    return {k: x.cpu().numpy() for k, x in o.items()}


def _verify_check(c, o):
    draft = c["draft"]
    acc, out, lp = ref.verify(
        c["logits"].astype(float), c["tokens"], c["starts"],
        c["uniform"].astype(float), c["noise"].astype(float),
        c["temp"].astype(float), draft if draft is None else
        draft.astype(float), c["kind"], c["vocab"], c["max_out"])
    assert np.array_equal(o["acc"], acc)
    assert np.array_equal(o["out"], out)
    # (x - m) / T in 64 bits, log of a sum whose terms are good to 2^-19
    # (an fp32 exponent of at most 64, ex2 to 2^-22), one rounding
    same = o["lp"] == lp
    assert (same | (np.abs(o["lp"] - lp) <=
                    2.0 ** -18 + 2.0 ** -24 * np.abs(lp))).all()
    n = np.diff(c["starts"])
    assert np.array_equal(o["lens"], c["lens"] + np.where(n > 0, acc + 1, 0))
    assert np.array_equal(o["nxt"], [out[b, acc[b]] for b in range(c["B"])])
    return acc


VERIFY = {
    "b1": dict(rows=[5], vocab=1000),
    "no_drafts": dict(rows=[1, 1, 1], vocab=333),
    "ragged": dict(rows=[3, 0, 1, 9, 0, 4], vocab=2049, pad=3, extra=2),
    "odd_vocab": dict(rows=[4] * 7, vocab=50257),
    "wide": dict(rows=[6, 2, 3], vocab=151936),
    "tiny_vocab": dict(rows=[3, 4], vocab=2),
    "one_word": dict(rows=[3], vocab=1),
    "many": dict(rows=[3] * 90, vocab=515),
    "long_draft": dict(rows=[128], vocab=700, near=0.05),
}


@gpu
@pytest.mark.parametrize("kind", ["none", "probs", "logits"])
@pytest.mark.parametrize("name", sorted(VERIFY))
def test_verify(name, kind):
    c = _verify_case(31, kind=kind, temp=0.8, **VERIFY[name])
    _verify_check(c, _verify_run(c))


@gpu
@pytest.mark.parametrize("kind", ["none", "probs", "logits"])
def test_verify_temperatures(kind):
    c = _verify_case(32, [4] * 8, 5003, kind,
                     np.array([0, 1, 0.3, -1, 2.5, 0.05, 0, 1]), near=0.2)
    acc = _verify_check(c, _verify_run(c))
    assert acc.min() < 3 <= acc.max()
    c["temp"][:] = 1
    _verify_check(c, _verify_run(c, temperature=False))


@gpu
@pytest.mark.parametrize("kind", ["none", "probs", "logits"])
@pytest.mark.parametrize("temp", [0.0, 1.0])
def test_verify_masked_logits(kind, temp):
    c = _verify_case(33, [3] * 6, 1003, kind, temp, near=0.2)
    lg = c["logits"]
    lg[:, 500:] = -np.inf                       # a grammar's mask
    lg[::4, :400] = -np.inf
    lg[::5, 7] = np.nan
    lg[2] = -np.finfo(np.float32).max           # all at the lowest value
    lg[5] = -np.inf                             # nothing left
    lg[7, 30] = np.inf
    lg[10, [40, 60]] = np.inf
    lg[12] = np.nan
    _verify_check(c, _verify_run(c))


@gpu
@pytest.mark.parametrize("kind", ["none", "probs", "logits"])
def test_verify_extreme_temperatures(kind):
    c = _verify_case(39, [3] * 5, 1003, kind, 1.0, near=0.2)
    c["logits"][:, 500:] = -np.inf
    c["temp"][:] = [np.inf, 3e38, 1e-39, 1e-45, np.nan]
    o = _verify_run(c)
    c["temp"][:] = [1e30, 1e30, 1e-30, 1e-30, 0]
    _verify_check(c, o)


@gpu
@pytest.mark.parametrize("kind", ["none", "probs", "logits"])
def test_verify_noise_below_the_normal_numbers(kind):
    c = _verify_case(40, [1, 2, 1], 5003, kind, 1.0, near=0.2)
    c["uniform"][:] = 1                         # (nearly) nothing accepted
    c["noise"][:, 17] = 1e-39                   # e^-60 / 1e-39 is less
    c["noise"][:, 900] = 1e-30                  # than e^-9 / 1e-30
    c["logits"][:, 17] = -60
    c["logits"][:, 900] = 0
    if c["draft"] is not None:
        c["draft"][:, [17, 900]] = 0 if kind == "probs" else -99
    c["tokens"][:] = 5
    o = _verify_run(c)
    _verify_check(c, o)
    assert o["nxt"].tolist() == [900] * 3


@gpu
def test_verify_ties_take_the_lowest_index():
    c = _verify_case(34, [1, 1], 4099, "none", np.array([0.0, 1.0]))
    c["logits"][:] = 0.5
    c["noise"][:] = 2.0
    c["noise"][1, [3001, 77, 4098]] = 0.25
    o = _verify_run(c)
    assert o["out"][:, 0].tolist() == [0, 77]
    c["logits"][0, [4000, 2222]] = 3.0
    assert _verify_run(c)["out"][0, 0] == 2222


@gpu
@pytest.mark.parametrize("kind", ["none", "probs", "logits"])
def test_verify_drafts_that_end_early(kind):
    c = _verify_case(35, [5, 5, 5], 600, kind, 1.0, near=0.01)
    c["uniform"][:] = 0                         # accept whatever is judged
    c["tokens"][[2, 9, 11]] = [-1, 600, -7]
    o = _verify_run(c)
    _verify_check(c, o)
    assert o["acc"].tolist() == [1, 3, 0]


@gpu
def test_verify_equal_distributions_always_accept():
    c = _verify_case(36, [4] * 5, 900, "logits", 0.9)
    c["draft"] = c["logits"].copy()
    o = _verify_run(c)
    assert (o["acc"] == 3).all()


@gpu
def test_verify_samples_follow_the_target():
    # 4000 one-draft sequences over 8 words: emitted first tokens are
    # distributed as p, not as q.  A count of N p has standard deviation
    # sqrt(N p (1 - p)) <= sqrt(N) / 2 = 32; 5 of them allowed.
    N, V = 4000, 8
    g = np.random.Generator(np.random.PCG64(5))
    p = np.array([.3, .2, .15, .1, .1, .08, .05, .02])
    q = p[::-1].copy()
    c = dict(starts=2 * np.arange(N + 1), T=2 * N, B=N, vocab=V, kind="probs",
             temp=np.ones(N, np.float32), pad=0, max_out=2,
             logits=np.tile(np.log(p).astype(np.float32), (2 * N, 1)),
             draft=np.tile(q.astype(np.float32), (2 * N, 1)),
             tokens=np.zeros(2 * N, np.int32),
             uniform=g.random(2 * N, dtype=np.float32),
             noise=g.exponential(size=(N, V)).astype(np.float32),
             lens=np.zeros(N, np.int32))
    c["tokens"][1::2] = g.choice(V, N, p=q)
    o = _verify_run(c)
    cnt = np.bincount(o["out"][:, 0], minlength=V)
    assert (np.abs(cnt - N * p) <= 5 * np.sqrt(N * p * (1 - p))).all()
    assert 0 < o["acc"].sum() < N


@gpu
def test_verify_row_count_past_max_out_is_reported():
    c = _verify_case(37, [4, 2], 100, "none", 1.0)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    i, f = torch.int32, torch.float32
    v = mpk.DraftVerifier(2, 6, 100, 3, status=st)
    acc = torch.zeros(2, dtype=i, device="cuda")
    out = torch.zeros(2, 3, dtype=i, device="cuda")
    v.verify(ref.as_dev(c["tokens"], i), ref.as_dev(c["logits"], f),
             ref.as_dev(c["uniform"], f), ref.as_dev(c["noise"], f), acc, out,
             q_start=ref.as_dev(c["starts"], i))
    assert st.item() == mpk.MPK_ERR_INVALID_ARG
    assert (out < 100).all()


@gpu
def test_verify_strided_and_in_a_graph():
    c = _verify_case(38, [3, 3], 1001, "probs", 0.7)
    want = _verify_run(c)
    i, f = torch.int32, torch.float32
    wide = torch.zeros(6, 1300, device="cuda")
    wide[:, 5:1006] = ref.as_dev(c["logits"], f)
    dr = torch.zeros(6, 1100, device="cuda")
    dr[:, :1001] = ref.as_dev(c["draft"], f)
    v = mpk.DraftVerifier(2, 6, 1001, 3)
    acc = torch.zeros(2, dtype=i, device="cuda")
    out = torch.zeros(2, 3, dtype=i, device="cuda")
    args = (ref.as_dev(c["tokens"], i), wide[:, 5:1006],
            ref.as_dev(c["uniform"], f), ref.as_dev(c["noise"], f), acc, out)
    kw = dict(draft=dr[:, :1001], temperature=ref.as_dev(c["temp"], f))
    v.verify(*args, **kw)               # uniform rows: 3 a sequence
    assert np.array_equal(out.cpu().numpy(), want["out"])
    out.zero_()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        v.verify(*args, **kw)
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    assert np.array_equal(out.cpu().numpy(), want["out"])
    assert np.array_equal(acc.cpu().numpy(), want["acc"])


# ------------------------------------------------------ one after another
@gpu
@pytest.mark.parametrize("d,hq,hkv", [(64, 4, 2), (128, 8, 2)])
def test_append_then_attend_equals_one_token_at_a_time(d, hq, hkv):
    """A prompt chunk, then drafts, against the same tokens fed singly."""
    g = torch.Generator().manual_seed(3)
    T, page = 37, 16
    W = (hq + 2 * hkv) * d
    x = torch.randn(2, T, W, generator=g).bfloat16().cuda()
    rope = mpk.Rope(mpk.mpk_rope_table(d, 64, 1e4), d)

    def fresh(n):
        z = lambda: torch.zeros(1, 8, hkv, page, d, dtype=torch.bfloat16,
                                device="cuda")
        kv = mpk.KVCache(z(), z(), torch.arange(8, dtype=torch.int32).view(
            2, 4).cuda(), torch.zeros(2, dtype=torch.int32, device="cuda"))
        return kv

    def feed(kv, sizes):
        outs, at = [], 0
        for m in sizes:
            rows = x[:, at:at + m].reshape(2 * m, W)
            p = mpk.PagedBatch(kv, hq, 2 * m)
            q = torch.empty(2 * m, hq * d, dtype=torch.bfloat16,
                            device="cuda")
            o = torch.empty_like(q)
            p.append(0, rows[:, :hq * d], rows[:, hq * d:(hq + hkv) * d],
                     rows[:, (hq + hkv) * d:], rope, q_out=q)
            p.attend(0, q, o)
            kv.seq_lens += m
            outs.append(o.view(2, m, -1))
            at += m
        return torch.cat(outs, 1), kv
    a, ka = feed(fresh(T), [1] * T)
    b, kb = feed(fresh(T), [29, 5, 1, 2])
    assert torch.equal(ka.k_pool, kb.k_pool)
    assert torch.equal(ka.v_pool, kb.v_pool)
    # the same products in another grouping: both are within their bound of
    # the exact value, which is at most (2 * 2^-8 + small) of max |v| off
    lim = 2 * (2 * 2.0 ** -8 + 2.0 ** -10) * x[..., -hkv * d:].abs().max()
    assert (a.float() - b.float()).abs().max() <= lim
