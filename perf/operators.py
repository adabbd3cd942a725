"""The serving operators over the paged KV cache, as measurable cases.

Three operators that one step of drafted (speculative) decoding makes of a
batch whose sequences share prompts:

  append   norm and rotate the new tokens' queries and keys, and append keys
           and values to the paged cache;
  attend   attention of the new tokens over the paged cache, where a group of
           sequences shares a prefix that is read once for all of them;
  verify   accept or reject the drafted tokens against the model's logits with
           given random numbers, and sample the token that follows.

``own`` selects what ``run`` does: False, the operators written out in
elementary torch operations; True, the calls of task_graph_runtime_gb300.
"""
import math
import random

import torch

own = False

DEV = "cuda"


# ------------------------------------------------------------------- cases
def listed():
    return [
        # one decode step of the 8B-shaped model at batch 16: a token a
        # sequence, per-head norms of q and k
        _append("append b16 one token", batch=16, lo=1, hi=1, hq=32, hkv=8,
                d=128, page=64, ctx_lo=128, ctx_hi=4096, rot=128, inter=False,
                norm=True, theta=1e6, lens=1),
        # drafted tokens of 64 sequences of the 1B shape, ragged,
        # interleaved pairs
        _append("append b64 drafts", batch=64, lo=1, hi=8, hq=32, hkv=8, d=64,
                page=16, ctx_lo=1, ctx_hi=2048, rot=64, inter=True, norm=False,
                theta=1e4, lens=2),
        # one long prompt chunk far into a long context
        _append("append prompt 8192", batch=1, lo=8192, hi=8192, hq=32, hkv=8,
                d=128, page=64, ctx_lo=98304, ctx_hi=98304, rot=128,
                inter=False, norm=True, theta=1e6, lens=3),
        # ragged prompts of many requests, half of each head rotated, pages
        # of an odd size
        _append("append ragged prompts", batch=23, lo=1, hi=4001, hq=32,
                hkv=8, d=128, page=24, ctx_lo=0, ctx_hi=700, rot=64,
                inter=False, norm=False, theta=1e4, lens=4),
        # the toy shape: all latency
        _attend("attend b4 tiny", groups=1, batch=4, lo=1, hi=1, hq=4, hkv=2,
                d=64, page=16, pre_lo=128, pre_hi=128, own_lo=1, own_hi=40,
                lens=5),
        # batch 16 of the 8B shape: a system prompt and own text of each
        _attend("attend b16", groups=1, batch=16, lo=1, hi=1, hq=32, hkv=8,
                d=128, page=64, pre_lo=2048, pre_hi=2048, own_lo=1,
                own_hi=2048, lens=6),
        # drafts of 64 sequences of the 1B shape, four prompts shared by some
        # of them each
        _attend("attend b64 drafts", groups=4, batch=64, lo=1, hi=6, hq=32,
                hkv=8, d=64, page=16, pre_lo=333, pre_hi=4099, own_lo=1,
                own_hi=700, lens=7),
        # many samples of one long prompt: the prefix is a dense product
        _attend("attend b256 long prefix", groups=1, batch=256, lo=1, hi=1,
                hq=32, hkv=8, d=128, page=64, pre_lo=16384, pre_hi=16384,
                own_lo=1, own_hi=512, lens=8),
        # one sequence, four drafts, the 1B shape's vocabulary
        _verify("verify b1", batch=1, lo=4, hi=4, vocab=32000, draft="probs",
                temp_lo=0.8, temp_hi=0.8, lens=9),
        # batch 16 with up to eight drafts, the drafting model's logits, a
        # temperature each (some greedy)
        _verify("verify b16 logits", batch=16, lo=0, hi=8, vocab=151936,
                draft="logits", temp_lo=0.0, temp_hi=1.3, lens=10),
        # drafts looked up in the prompt (no distribution), odd vocabulary
        _verify("verify b33 lookup", batch=33, lo=1, hi=3, vocab=50257,
                draft="none", temp_lo=0.6, temp_hi=1.0, lens=11),
        # the largest: 64 sequences of five drafts
        _verify("verify b64", batch=64, lo=5, hi=5, vocab=151936,
                draft="probs", temp_lo=0.7, temp_hi=1.1, lens=12),
    ]


def _append(name=None, **kw):
    c = dict(op="append", **kw)
    return dict(c, name=name) if name else c


def _attend(name=None, **kw):
    c = dict(op="attend", **kw)
    return dict(c, name=name) if name else c


def _verify(name=None, **kw):
    c = dict(op="verify", **kw)
    return dict(c, name=name) if name else c


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(
        math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["append", "attend", "attend", "verify"])
    lens = rng.randrange(1 << 30)
    if kind == "verify":
        vocab = _log_int(rng, 1000, 151936)
        hi = rng.randint(0, 8)
        batch = max(1, min(_log_int(rng, 1, 64),
                           int(64 * 6 * 151936 / (vocab * (hi + 1)))))
        greedy = rng.random() < 0.2
        return _verify(batch=batch, lo=rng.randint(0, hi), hi=hi, vocab=vocab,
                       draft=rng.choice(["none", "probs", "logits"]),
                       temp_lo=0.0 if greedy else 0.6, temp_hi=1.3, lens=lens)
    d = rng.choice([32, 64, 128, 128])
    hkv = rng.choice([1, 2, 4, 8])
    hq = hkv * rng.choice([1, 2, 4, 4, 8])
    page = rng.choice([16, 64, 64, rng.randint(5, 100)])
    if kind == "append":
        hi = _log_int(rng, 1, 8192)
        batch = _log_int(rng, 1, max(1, min(256, 16384 // hi)))
        return _append(batch=batch, lo=rng.randint(max(1, hi // 4), hi), hi=hi,
                       hq=hq, hkv=hkv, d=d, page=page, ctx_lo=0,
                       ctx_hi=_log_int(rng, 1, 4096),
                       rot=rng.choice([d, d, d // 2]),
                       inter=rng.random() < 0.5, norm=rng.random() < 0.5,
                       theta=rng.choice([1e4, 1e6]), lens=lens)
    batch = _log_int(rng, 1, 256)
    groups = rng.randint(1, min(batch, 4))
    hi = rng.randint(1, 6) if batch <= 64 else 1
    pre = _log_int(rng, 16, 16384)
    return _attend(groups=groups, batch=batch, lo=rng.randint(1, hi), hi=hi,
                   hq=hq, hkv=hkv, d=d, page=page,
                   pre_lo=rng.randint(max(1, pre // 4), pre), pre_hi=pre,
                   own_lo=1, own_hi=_log_int(rng, 1, 512), lens=lens)


# ------------------------------------------------- lengths, from the case
def _lengths(case):
    """New tokens of each sequence, its length before them, the group bounds
    and the groups' prefix lengths: whole numbers from the case alone."""
    r = random.Random(case["lens"])
    n = [r.randint(case["lo"], case["hi"]) for _ in range(case["batch"])]
    if case["op"] == "append":
        ctx = [r.randint(case["ctx_lo"], case["ctx_hi"]) for _ in n]
        return n, ctx, [0, len(n)], [0]
    if case["op"] == "verify":
        return [x + 1 for x in n], [0] * len(n), None, None
    G, B = case["groups"], case["batch"]
    cut = [0] + sorted(r.sample(range(1, B), G - 1)) + [B]
    pre = [r.randint(case["pre_lo"], case["pre_hi"]) for _ in range(G)]
    of = [g for g in range(G) for _ in range(cut[g], cut[g + 1])]
    # own keys of a sequence: those before the new tokens
    ctx = [pre[g] + r.randint(case["own_lo"], case["own_hi"]) - 1 for g in of]
    return n, ctx, cut, pre


def _starts(n):
    out = [0]
    for x in n:
        out.append(out[-1] + x)
    return out


def _tables(case, n, ctx, cut, pre):
    """Page tables (the whole pages of a prefix are shared by its group) and
    the number of pages; ids in a permuted order."""
    P = case["page"]
    rows, free = [], 0
    for g in range(len(pre)):
        share = pre[g] // P
        base = list(range(free, free + share))
        free += share
        for b in range(cut[g], cut[g + 1]):
            need = -(-(ctx[b] + n[b]) // P)
            mine = base[:need] + list(range(free, free + max(0, need - share)))
            free += max(0, need - share)
            rows.append(mine)
    ids = list(range(free))
    random.Random(case["lens"] + 1).shuffle(ids)
    width = max(len(x) for x in rows)
    return [[ids[p] for p in x] + [-1] * (width - len(x)) for x in rows], free


# ------------------------------------------------------------------ inputs
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _randn(g, *shape, std=1.0):
    return torch.empty(shape, device=DEV).normal_(0.0, std, generator=g).to(
        torch.bfloat16)


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def prepare(case, seed):
    g = _gen(seed)
    n, ctx, cut, pre = _lengths(case)
    start = _starts(n)
    T = start[-1]
    s = dict(case=case, T=T, B=len(n), q_start=_i32(start), most=max(n))
    if case["op"] == "verify":
        V, B = case["vocab"], len(n)
        # the model's logits, and a drafting model's that nearly agree
        logits = torch.empty(T, V, device=DEV).normal_(0.0, 2.0, generator=g)
        draft = logits + torch.empty(T, V, device=DEV).normal_(
            0.0, 0.7, generator=g)
        t = torch.empty(B, device=DEV).uniform_(
            case["temp_lo"], case["temp_hi"], generator=g)
        if case["temp_lo"] == 0.0:
            t[::3] = 0.0
        seq = torch.repeat_interleave(
            torch.arange(B, device=DEV), _i32(n).long())
        tt = torch.where(t > 0, t, torch.ones_like(t))[seq][:, None]
        probs = torch.softmax(draft / tt, -1)
        noise = torch.empty(T, V, device=DEV).exponential_(generator=g)
        pick = torch.argmax(probs / noise, -1)          # drafted after row i
        del noise
        pick = torch.where(t[seq] > 0, pick, torch.argmax(logits + 0.2 * (
            draft - logits), -1))
        tokens = torch.randint(0, V, (T,), device=DEV, generator=g)
        tokens[1:] = torch.where(seq[1:] == seq[:-1], pick[:-1], tokens[1:])
        s.update(logits=logits, tokens=tokens.int(), temp=t,
                 draft=None if case["draft"] == "none" else
                 probs if case["draft"] == "probs" else draft,
                 uniform=torch.rand(T, device=DEV, generator=g),
                 noise=torch.empty(B, V, device=DEV).exponential_(generator=g),
                 seq_lens=torch.randint(0, 4096, (B,), device=DEV,
                                        generator=g).int())
        return s
    table, pages = _tables(case, n, ctx, cut, pre)
    hq, hkv, d, P = case["hq"], case["hkv"], case["d"], case["page"]
    s.update(k_pool=_randn(g, 1, pages, hkv, P, d),
             v_pool=_randn(g, 1, pages, hkv, P, d), page_table=_i32(table),
             seq_lens=_i32(ctx), hi=max(c + m for c, m in zip(ctx, n)))
    if case["op"] == "append":
        # the rows of a fused q, k, v projection
        s["qkv"] = _randn(g, T, (hq + 2 * hkv) * d)
        if case["norm"]:
            s["q_norm"] = (1 + 0.02 * _randn(g, d).float()).bfloat16()
            s["k_norm"] = (1 + 0.02 * _randn(g, d).float()).bfloat16()
        # the rotation's table, made once for a model: cos and sin of
        # position * theta^(-2i/rot), angles in 64 bits
        half = case["rot"] // 2
        inv = case["theta"] ** (-2.0 * torch.arange(
            half, dtype=torch.float64, device=DEV) / case["rot"])
        ang = torch.arange(s["hi"], dtype=torch.float64,
                           device=DEV)[:, None] * inv
        s["table"] = torch.stack([torch.cos(ang), torch.sin(ang)], -1).float()
        s["q_out"] = torch.empty(T, hq * d, dtype=torch.bfloat16, device=DEV)
        return s
    of = [g_ for g_ in range(len(pre)) for _ in range(cut[g_], cut[g_ + 1])]
    s.update(q=_randn(g, T, hq * d), group_start=_i32(cut),
             prefix_len=_i32(pre), pre=max(pre),
             own=max(c + m - pre[k] for c, m, k in zip(ctx, n, of)),
             rows=max(start[cut[k + 1]] - start[cut[k]]
                      for k in range(len(pre))),
             out=torch.empty(T, hq * d, dtype=torch.bfloat16, device=DEV),
             lse=torch.empty(T, hq, device=DEV))
    return s


# ------------------------------------------------------------- plain forms
def _of_token(s):
    """Sequence and place in it of each of the T token rows."""
    row = torch.arange(s["T"], device=DEV)
    seq = torch.bucketize(row, s["q_start"][1:].long(), right=True)
    return row, seq, row - s["q_start"].long()[seq]


def _norm(x, w):
    return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6) * w.float()


def _rotate(x, cs, rot, inter):
    c, sn, r = cs[..., 0][:, None], cs[..., 1][:, None], x[..., :rot]
    if inter:
        a, b = r[..., 0::2], r[..., 1::2]
        y = torch.stack([a * c - b * sn, b * c + a * sn], -1).flatten(-2)
    else:
        a, b = r[..., :rot // 2], r[..., rot // 2:]
        y = torch.cat([a * c - b * sn, b * c + a * sn], -1)
    return torch.cat([y, x[..., rot:]], -1)


def _plain_append(s):
    c = s["case"]
    hq, hkv, d, P = c["hq"], c["hkv"], c["d"], c["page"]
    _, seq, place = _of_token(s)
    pos = s["seq_lens"].long()[seq] + place
    x = s["qkv"].float().view(s["T"], hq + 2 * hkv, d)
    q, k, v = x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:]
    if c["norm"]:
        q, k = _norm(q, s["q_norm"]), _norm(k, s["k_norm"])
    cs = s["table"][pos]
    s["q_out"].copy_(_rotate(q, cs, c["rot"], c["inter"]).flatten(1))
    page = s["page_table"].long()[seq, pos // P]
    s["k_pool"][0, page, :, pos % P] = _rotate(
        k, cs, c["rot"], c["inter"]).bfloat16()
    s["v_pool"][0, page, :, pos % P] = v.bfloat16()
    return s["q_out"], s["k_pool"], s["v_pool"]


def _keys(s, pool, rows, at):
    """Tokens `at` of the sequences `rows` ([n] each way), in 32 bits:
    [n, tokens, Hkv, d].  Places past a sequence's pages read page 0."""
    P = s["case"]["page"]
    slot = (at // P).clamp(max=s["page_table"].shape[1] - 1)
    page = torch.gather(s["page_table"].long()[rows], 1, slot).clamp(min=0)
    return pool[0, page, :, at % P].float()


def _part(q, k, v, see):
    """Un-normalised attention of q [n, R, Hkv, G, d] over k, v [n, L, Hkv, d]
    where see [n, R, L]: maximum, sum and weighted values."""
    n, R, H, G, d = q.shape
    sc = torch.matmul(q.permute(0, 2, 1, 3, 4).reshape(n, H, R * G, d),
                      k.permute(0, 2, 3, 1)).view(n, H, R, G, -1)
    sc = sc * (1.0 / math.sqrt(d))
    sc = sc.masked_fill(~see[:, None, :, None], -math.inf)
    m = sc.amax(-1, keepdim=True)
    p = torch.exp(sc - m.clamp(min=-3e38))
    o = torch.matmul(p.view(n, H, R * G, -1), v.permute(0, 2, 1, 3))
    return (m[..., 0].permute(0, 2, 1, 3), p.sum(-1).permute(0, 2, 1, 3),
            o.view(n, H, R, G, d).permute(0, 2, 1, 3, 4))


def _plain_attend(s):
    c = s["case"]
    hq, hkv, d = c["hq"], c["hkv"], c["d"]
    G, B, T = c["groups"], s["B"], s["T"]
    _, seq, place = _of_token(s)
    pos = s["seq_lens"].long()[seq] + place
    cut, pre = s["group_start"].long(), s["prefix_len"].long()
    grp = torch.bucketize(seq, cut[1:], right=True)
    in_grp = torch.arange(T, device=DEV) - s["q_start"].long()[cut][grp]
    q = s["q"].float().view(T, hkv, hq // hkv, d)

    # the prefix, once for the tokens of a group
    def pad(rows, most, at, x):
        y = torch.zeros((rows, most) + x.shape[1:], dtype=x.dtype, device=DEV)
        y[at] = x
        return y
    at = torch.arange(s["pre"], device=DEV)
    see = ((at < pre[:, None])[:, None] &
           (at <= pad(G, s["rows"], (grp, in_grp), pos)[..., None]))
    keys = at.expand(G, -1)
    a = _part(pad(G, s["rows"], (grp, in_grp), q),
              _keys(s, s["k_pool"], cut[:-1], keys),
              _keys(s, s["v_pool"], cut[:-1], keys).masked_fill(
                  ~(at < pre[:, None])[..., None, None], 0.0), see)
    a = [x[grp, in_grp] for x in a]
    # a sequence's own keys
    gs = torch.bucketize(torch.arange(B, device=DEV), cut[1:], right=True)
    keys = pre[gs][:, None] + torch.arange(s["own"], device=DEV)
    end = s["seq_lens"].long() + (s["q_start"][1:] - s["q_start"][:-1])
    see = keys[:, None] <= pad(B, s["most"], (seq, place), pos)[..., None]
    own_ = _part(pad(B, s["most"], (seq, place), q),
                 _keys(s, s["k_pool"], torch.arange(B, device=DEV), keys),
                 _keys(s, s["v_pool"], torch.arange(B, device=DEV),
                       keys).masked_fill(
                     ~(keys < end[:, None])[..., None, None], 0.0), see)
    b = [x[seq, place] for x in own_]
    m = torch.maximum(a[0], b[0])
    wa, wb = torch.exp(a[0] - m), torch.exp(b[0] - m)
    l = a[1] * wa + b[1] * wb
    o = (a[2] * wa[..., None] + b[2] * wb[..., None]) / l[..., None]
    s["out"].copy_(o.reshape(T, hq * d))
    s["lse"].copy_((m + torch.log(l)).reshape(T, hq))
    return s["out"], s["lse"]


def _plain_verify(s):
    # in 64 bits: whole numbers come out, and two candidates may lie close
    c, T, B = s["case"], s["T"], s["B"]
    row, seq, place = _of_token(s)
    start = s["q_start"].long()
    drafts = (start[1:] - start[:-1] - 1)                      # per sequence
    t = s["temp"].double()[seq][:, None]
    lg = s["logits"].double()
    greedy = (t <= 0)
    x = lg / torch.where(greedy, torch.ones_like(t), t)
    logp = x - torch.logsumexp(x, -1, keepdim=True)
    best = torch.argmax(lg, -1)
    nxt = s["tokens"].long()[(row + 1).clamp(max=T - 1)]       # drafted token
    p_d = torch.exp(logp.gather(1, nxt[:, None])[:, 0])
    if s["draft"] is None:
        q_d = torch.ones_like(p_d)
    else:
        q = s["draft"].double()
        if c["draft"] == "logits":
            q = torch.softmax(q / torch.where(greedy, torch.ones_like(t), t),
                              -1)
        q_d = q.gather(1, nxt[:, None])[:, 0]
    ok = torch.where(greedy[:, 0], nxt == best,
                     s["uniform"].double() * q_d < p_d)
    ok &= place < drafts[seq]
    # accepted: the drafts before the first one refused
    bad = torch.where(ok, s["most"], place)
    n_acc = torch.full((B,), s["most"], dtype=torch.int64,
                       device=DEV).scatter_reduce(0, seq, bad, "amin")
    at = start[:-1] + n_acc
    p = torch.exp(logp[at])
    rest = p
    if s["draft"] is not None:
        rest = (p - q[at]).clamp(min=0.0)
    else:
        rest = p.scatter(1, nxt[at][:, None], 0.0)
    rest = torch.where(rest.amax(-1, keepdim=True) > 0, rest, p)
    w = torch.where((n_acc < drafts)[:, None], rest, p)
    tok = torch.argmax(w / s["noise"].double(), -1)
    tok = torch.where(s["temp"] <= 0, best[at], tok)
    # the emitted tokens and their log probabilities
    col = torch.arange(s["most"], device=DEV)
    src = (start[:-1][:, None] + col).clamp(max=T - 1)
    out = torch.where(col < n_acc[:, None], nxt[src], -1)
    out = torch.where(col == n_acc[:, None], tok[:, None], out)
    lp = torch.where(greedy, torch.zeros_like(logp), logp)[
        src, out.clamp(min=0)]
    lp = torch.where(out >= 0, lp, torch.zeros_like(lp)).float()
    lens = s["seq_lens"] + n_acc.int() + 1
    return n_acc.int(), out.int(), lp, lens


# ------------------------------------------------------------ the framework
def _own_append(s):
    from task_graph_runtime_gb300 import mpk
    c = s["case"]
    if "plan" not in s:   # what a serving program keeps beside its cache
        s["plan"] = mpk.PagedBatch(
            mpk.KVCache(s["k_pool"], s["v_pool"], s["page_table"],
                        s["seq_lens"]), c["hq"], s["T"], q_start=s["q_start"])
        s["rope"] = mpk.Rope(s["table"], c["rot"], c["inter"])
    hq, hkv, d, x = c["hq"], c["hkv"], c["d"], s["qkv"]
    s["plan"].append(0, x[:, :hq * d], x[:, hq * d:(hq + hkv) * d],
                     x[:, (hq + hkv) * d:], s["rope"], q_out=s["q_out"],
                     q_norm=s.get("q_norm"), k_norm=s.get("k_norm"), eps=1e-6)
    return s["q_out"], s["k_pool"], s["v_pool"]


def _own_attend(s):
    from task_graph_runtime_gb300 import mpk
    if "plan" not in s:
        s["plan"] = mpk.PagedBatch(
            mpk.KVCache(s["k_pool"], s["v_pool"], s["page_table"],
                        s["seq_lens"]), s["case"]["hq"], s["T"],
            q_start=s["q_start"], group_start=s["group_start"],
            prefix_len=s["prefix_len"])
    s["plan"].attend(0, s["q"], s["out"], lse=s["lse"])
    return s["out"], s["lse"]


def _own_verify(s):
    from task_graph_runtime_gb300 import mpk
    if "plan" not in s:
        s["plan"] = mpk.DraftVerifier(s["B"], s["T"], s["case"]["vocab"],
                                      s["most"], device=DEV)
        s["outs"] = (torch.empty(s["B"], dtype=torch.int32, device=DEV),
                     torch.empty(s["B"], s["most"], dtype=torch.int32,
                                 device=DEV),
                     torch.empty(s["B"], s["most"], device=DEV),
                     torch.empty(s["B"], dtype=torch.int32, device=DEV))
    acc, out, lp, lens = s["outs"]
    s["plan"].verify(s["tokens"], s["logits"], s["uniform"], s["noise"],
                     acc, out, q_start=s["q_start"], draft=s["draft"],
                     draft_is_logits=s["case"]["draft"] == "logits",
                     temperature=s["temp"], logprobs=lp,
                     seq_lens=s["seq_lens"], seq_lens_out=lens)
    return acc, out, lp, lens


def run(s):
    op = s["case"]["op"]
    if own:
        return {"append": _own_append, "attend": _own_attend,
                "verify": _own_verify}[op](s)
    return {"append": _plain_append, "attend": _plain_attend,
            "verify": _plain_verify}[op](s)


# -------------------------------------------------------------------- work
def work(case):
    n, ctx, cut, pre = _lengths(case)
    T, B = sum(n), len(n)
    if case["op"] == "verify":
        V = case["vocab"]
        rows = T + B + (0 if case["draft"] == "none" else
                        B if case["draft"] == "probs" else T - B)
        return {"bytes": 4.0 * (rows * V + 2 * T + 4 * B + 2 * B * max(n)),
                "flops": 4.0 * rows * V}
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    if case["op"] == "append":
        return {"bytes": 2.0 * 2 * T * (hq + 2 * hkv) * d +
                4.0 * T * case["rot"],
                "flops": 3.0 * T * (hq + hkv) * case["rot"]}
    keys = sum(pre)
    seen = 0
    for g in range(len(pre)):
        for b in range(cut[g], cut[g + 1]):
            keys += ctx[b] + n[b] - pre[g]
            seen += n[b] * ctx[b] + n[b] * (n[b] + 1) // 2
    return {"bytes": 2.0 * 2 * keys * hkv * d + 2.0 * 2 * T * hq * d +
            4.0 * T * hq, "flops": 4.0 * seen * hq * d}


# -------------------------------------------- the definition, in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    n, ctx, cut, pre = _lengths(case)
    start = _starts(n)
    if case["op"] == "append":
        return _exact_append(case, s, n, ctx, start)
    if case["op"] == "attend":
        return _exact_attend(case, s, n, ctx, start, cut, pre)
    return _exact_verify(case, s, n, start)


def _exact_append(case, s, n, ctx, start):
    hq, hkv, d, P, rot = (case[k] for k in ("hq", "hkv", "d", "page", "rot"))
    x = s["qkv"].double().view(-1, hq + 2 * hkv, d)
    if case["norm"]:
        rms = (x.pow(2).sum(-1, keepdim=True) / d + 1e-6).sqrt()
        x = torch.cat([x[:, :hq] / rms[:, :hq] * s["q_norm"].double(),
                       x[:, hq:hq + hkv] / rms[:, hq:hq + hkv] *
                       s["k_norm"].double(), x[:, hq + hkv:]], 1)
    pos = torch.tensor([ctx[b] + i for b in range(len(n))
                        for i in range(n[b])], device=DEV)
    # pairs as complex numbers, turned by e^(i angle)
    i = torch.arange(rot // 2, device=DEV, dtype=torch.float64)
    ang = pos[:, None].double() * torch.exp(
        -2.0 * i / rot * math.log(case["theta"]))
    turn = torch.polar(torch.ones_like(ang), ang)[:, None]
    lo = torch.arange(rot // 2, device=DEV) * (2 if case["inter"] else 1)
    hi = lo + (1 if case["inter"] else rot // 2)
    z = torch.complex(x[:, :hq + hkv, lo], x[:, :hq + hkv, hi]) * turn
    y = x.clone()
    y[:, :hq + hkv, lo], y[:, :hq + hkv, hi] = z.real, z.imag
    kp, vp = s["k_pool"].double(), s["v_pool"].double()
    table = s["page_table"].tolist()
    flat = torch.tensor([table[b][(ctx[b] + j) // P] for b in range(len(n))
                         for j in range(n[b])], device=DEV)
    kp[0, flat, :, pos % P] = y[:, hq:hq + hkv]
    vp[0, flat, :, pos % P] = y[:, hq + hkv:]
    return y[:, :hq].reshape(-1, hq * d), kp, vp


def _exact_attend(case, s, n, ctx, start, cut, pre):
    hq, hkv, d, P = (case[k] for k in ("hq", "hkv", "d", "page"))
    table = s["page_table"].tolist()
    q = s["q"].double().view(-1, hkv, hq // hkv, d)
    out = torch.empty(q.shape, dtype=torch.float64, device=DEV)
    lse = torch.empty(q.shape[:-1], dtype=torch.float64, device=DEV)

    def load(pool, b, lo, hi):
        t = torch.arange(lo, hi)
        pages = torch.tensor(table[b])[t // P].to(DEV)
        return pool[0, pages, :, (t % P).to(DEV)].double()
    for g in range(len(pre)):
        kp = load(s["k_pool"], cut[g], 0, pre[g])
        vp = load(s["v_pool"], cut[g], 0, pre[g])
        for b in range(cut[g], cut[g + 1]):
            end = ctx[b] + n[b]
            k = torch.cat([kp, load(s["k_pool"], b, pre[g], end)])
            v = torch.cat([vp, load(s["v_pool"], b, pre[g], end)])
            for i in range(n[b]):
                t, m = start[b] + i, ctx[b] + i + 1
                sc = torch.einsum("hgd,lhd->hgl", q[t], k[:m]) / math.sqrt(d)
                lse[t] = torch.logsumexp(sc, -1)
                out[t] = torch.einsum("hgl,lhd->hgd", torch.exp(
                    sc - lse[t][..., None]), v[:m])
    return out.reshape(-1, hq * d), lse.reshape(-1, hq)


def _exact_verify(case, s, n, start):
    B, most = len(n), max(n)
    acc = torch.zeros(B, dtype=torch.int32)
    out = torch.full((B, most), -1, dtype=torch.int32)
    lp = torch.zeros(B, most, dtype=torch.float64)
    tok, temp = s["tokens"].tolist(), s["temp"].tolist()
    u = s["uniform"].double().tolist()
    for b in range(B):
        a, T = 0, temp[b]
        while True:
            r = start[b] + a
            row = s["logits"][r].double()
            last = a == n[b] - 1
            d = None if last else tok[r + 1]
            if T <= 0:
                e = int(torch.argmax(row))
                if last or d != e:
                    out[b, a] = e
                    break
                out[b, a], a = d, a + 1
                continue
            p = torch.softmax(row / T, -1)
            w = p
            if not last:
                if case["draft"] == "none":
                    q = torch.zeros_like(p)
                    q[d] = 1.0
                elif case["draft"] == "probs":
                    q = s["draft"][r].double()
                else:
                    q = torch.softmax(s["draft"][r].double() / T, -1)
                if u[r] * float(q[d]) < float(p[d]):
                    out[b, a], lp[b, a], a = d, float(torch.log(p[d])), a + 1
                    continue
                w = torch.clamp(p - q, min=0.0)
                if case["draft"] == "none":
                    w = p * (1.0 - q)
                if float(w.max()) <= 0:
                    w = p
            e = int(torch.argmax(w / s["noise"][b].double()))
            out[b, a], lp[b, a] = e, float(torch.log(p[e]))
            break
        acc[b] = a
    lens = s["seq_lens"].cpu() + acc + 1
    return acc, out, lp, lens
