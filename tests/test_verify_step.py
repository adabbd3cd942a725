"""mpk_verify_step: one step of drafted decoding of a whole model through the
graph's kernel-per-operator form, against the oracle's decode step fed the
same tokens one at a time, and against mpk_decode_step."""
import ctypes

import numpy as np
import pytest
import torch

import serving_ref as ref
from oracle import numerics as nx
from task_graph_runtime_gb300 import mpk, synth

from gpu_util import dev_kv, dev_weights, within_bound

gpu = pytest.mark.gpu

SHAPES = {
    "tiny": synth.TINY,
    "qk_norm": synth.ModelShape(2, 256, 8, 2, 128, 512, 1500, 1e-6, 1e6, True),
    "d32": synth.ModelShape(3, 128, 4, 4, 32, 256, 700),
}


def _setup(shape, ctx, page, seed, rows, wide=0):
    """Weights, cache of len(ctx) sequences with room for more tokens, and a
    graph of `rows` rows."""
    wl = synth.Workload("t", shape, len(ctx), tuple(ctx), page, 12)
    W = synth.model_weights(shape, seed)
    kv = synth.kv_inputs(wl, seed)
    g = mpk.Graph(shape, rows, page_size=page,
                  max_pages_per_seq=wl.max_pages_per_seq)
    Wd = dev_weights(W, shape)
    g.bind(Wd)
    return wl, W, kv, g, Wd


def _buffers(rows, B, V, mo, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    i = dict(dtype=torch.int32, device="cuda")
    return dict(lg=torch.full((rows, V), 7.0, device="cuda"),
                u=torch.rand(rows, device="cuda", generator=gen),
                e=torch.empty(B, V, device="cuda").exponential_(generator=gen),
                acc=torch.full((B,), 99, **i), out=torch.full((B, mo), 99, **i),
                lp=torch.zeros(B, mo, device="cuda"),
                nxt=torch.full((B,), 99, **i))


def _oracle_rows(shape, W, kv, tokens, starts):
    """The oracle's logits after each row's token."""
    n = np.diff(starts)
    k, v, lens = kv.k_pool.copy(), kv.v_pool.copy(), kv.seq_lens.copy()
    rows = {}
    for i in range(int(n.max())):
        live = [b for b in range(len(n)) if i < n[b]]
        sl = lens[live].copy()
        r = nx.decode_step(shape, W, tokens[[starts[b] + i for b in live]], k,
                           v, kv.page_table[live], sl)
        lens[live] = sl
        for j, b in enumerate(live):
            rows[starts[b] + i] = r["logits"][j]
    return rows, k, v


CASES = {
    "even": dict(shape="tiny", ctx=(37, 52), n=[4, 4]),
    "one_row_each": dict(shape="tiny", ctx=(0, 5, 16, 130), n=[1, 1, 1, 1]),
    "ragged": dict(shape="qk_norm", ctx=(9, 31, 64), n=[3, 0, 5], rows=9),
    "groups": dict(shape="qk_norm", ctx=(40, 33, 70, 12), n=[2, 1, 3, 2],
                   groups=([0, 2, 4], [33, 12])),
    "sixteen": dict(shape="d32", ctx=(21,) * 4, n=[4] * 4,
                    groups=([0, 4], [21]), page=8),
}


@gpu
@pytest.mark.parametrize("name", sorted(CASES))
def test_rows_match_the_oracle_fed_singly(name):
    c = CASES[name]
    shape = SHAPES[c["shape"]]
    starts = np.concatenate([[0], np.cumsum(c["n"])]).astype(int)
    rows = c.get("rows", int(starts[-1]))
    B = len(c["n"])
    wl, W, kv, g, Wd = _setup(shape, c["ctx"], c.get("page", 16), 5, rows)
    kw = {}
    if "groups" in c:
        cut, pre = c["groups"]
        # the groups' prefixes are the first sequence's
        P = wl.page_size
        for k in range(len(pre)):
            for b in range(cut[k] + 1, cut[k + 1]):
                for t in range(pre[k]):
                    for pool in (kv.k_pool, kv.v_pool):
                        pool[:, kv.page_table[b, t // P], :, t % P] = pool[
                            :, kv.page_table[cut[k], t // P], :, t % P]
        kw = dict(group_start=ref.as_dev(cut, torch.int32),
                  prefix_len=ref.as_dev(pre, torch.int32))
    rng = np.random.Generator(np.random.PCG64(9))
    tokens = rng.integers(0, shape.vocab, rows).astype(np.int32)
    want, ko, vo = _oracle_rows(shape, W, kv, tokens, starts)
    kvd = dev_kv(kv)
    mo = max(c["n"])
    b = _buffers(rows, B, shape.vocab, mo, 3)
    temp = ref.as_dev(np.linspace(0, 1.2, B), torch.float32)
    g.verify_step(ref.as_dev(tokens, torch.int32), kvd, b["lg"], b["u"],
                  b["e"], b["acc"], b["out"],
                  q_start=ref.as_dev(starts, torch.int32), temperature=temp,
                  logprobs=b["lp"], next_tokens=b["nxt"], **kw)
    torch.cuda.synchronize()
    assert g.status() == mpk.MPK_OK
    got = b["lg"].cpu().numpy()
    for r, w in want.items():
        ok, err, lim = within_bound(got[r], w)
        assert ok, f"row {r}: {err} > {lim}"
    # the judgement is that of these logits, exactly
    acc, out, lp = ref.verify(got.astype(float), tokens, starts,
                              b["u"].cpu().double().numpy(),
                              b["e"].cpu().double().numpy(),
                              temp.cpu().double().numpy(), None, "none",
                              shape.vocab, mo)
    assert np.array_equal(b["acc"].cpu().numpy(), acc)
    assert np.array_equal(b["out"].cpu().numpy(), out)
    n = np.array(c["n"])
    assert np.array_equal(kvd.seq_lens.cpu().numpy(),
                          kv.seq_lens + np.where(n > 0, acc + 1, 0))
    # the first layer's new keys come from the same products: they differ
    # from the oracle's by the rounding of a few values
    P = wl.page_size
    for s in range(B):
        for i in range(c["n"][s]):
            t = int(kv.seq_lens[s]) + i
            pg = kv.page_table[s, t // P]
            a = nx.bf16_to_f32(ko[0, pg, :, t % P])
            d = kvd.k_pool[0, int(pg), :, t % P].float().cpu().numpy()
            assert within_bound(d, a)[0]
    g.close()


@gpu
def test_one_row_a_sequence_is_the_decode_step():
    shape = SHAPES["qk_norm"]
    wl, W, kv, g, Wd = _setup(shape, (20, 3, 47, 64), 16, 6, 4)
    tokens = ref.as_dev(synth.tokens(wl, 6), torch.int32)
    kva, kvb = dev_kv(kv), dev_kv(kv)
    lg = torch.empty(4, shape.vocab, device="cuda")
    nt = torch.empty(4, dtype=torch.int32, device="cuda")
    g.set_mode(mpk.MODE_KPO)
    g.decode_step(tokens, kva, lg, nt)
    b = _buffers(4, 4, shape.vocab, 1, 1)
    g.verify_step(tokens, kvb, b["lg"], b["u"], b["e"], b["acc"], b["out"],
                  temperature=torch.zeros(4, device="cuda"))
    torch.cuda.synchronize()
    assert g.status() == mpk.MPK_OK
    ok, err, lim = within_bound(b["lg"].cpu().numpy(), lg.cpu().numpy())
    assert ok, (err, lim)
    assert torch.equal(kva.seq_lens, kvb.seq_lens)
    # the first layer sees the same input: its keys and values are the same
    # bit for bit
    assert torch.equal(kva.k_pool[0], kvb.k_pool[0])
    assert torch.equal(kva.v_pool[0], kvb.v_pool[0])
    assert torch.equal(b["out"][:, 0], b["lg"].argmax(-1).int())
    g.close()


@gpu
def test_greedy_drafts_follow_greedy_decoding():
    """Right drafts are accepted, wrong ones replaced: the tokens of a loop
    are those of one-token steps."""
    shape = SHAPES["tiny"]
    wl, W, kv, g4, Wd = _setup(shape, (30, 17), 16, 8, 8)
    g1 = mpk.Graph(shape, 2, page_size=16,
                   max_pages_per_seq=wl.max_pages_per_seq)
    g1.bind(Wd)
    lg = torch.empty(2, shape.vocab, device="cuda")

    def greedy(first):
        tok = t = ref.as_dev(first, torch.int32)
        kva, seqs, gaps = dev_kv(kv), [tok.cpu().numpy()], []
        for _ in range(10):
            nt = torch.empty(2, dtype=torch.int32, device="cuda")
            g1.decode_step(t, kva, lg, nt)
            top = lg.topk(2, -1).values
            gaps.append(float((top[:, 0] - top[:, 1]).min()))
            t = nt
            seqs.append(nt.cpu().numpy())
        return np.stack(seqs, 1), min(gaps)         # [2, 11]
    # the first start whose ten tokens have no near tie (as the decode
    # step's own tests: below 1e-2 either token is right)
    seqs = next(s for s, gap in (greedy([k, 1023 - k]) for k in range(500))
                if gap > 1e-2)
    kvb = dev_kv(kv)
    at = np.zeros(2, int)
    done = [[], []]
    zero = torch.zeros(2, device="cuda")
    for step in range(3):
        rows = np.zeros((2, 4), np.int32)
        for s in range(2):
            d = seqs[s, at[s]:at[s] + 4].copy()
            if step == 1:
                d[2] = (d[2] + 1) % shape.vocab     # a wrong second draft
            rows[s] = d
        b = _buffers(8, 2, shape.vocab, 4, step)
        g4.verify_step(ref.as_dev(rows.reshape(-1), torch.int32), kvb,
                       b["lg"], b["u"], b["e"], b["acc"], b["out"],
                       temperature=zero)
        torch.cuda.synchronize()
        acc, out = b["acc"].cpu().numpy(), b["out"].cpu().numpy()
        assert acc.tolist() == ([1, 1] if step == 1 else [3, 3])
        for s in range(2):
            done[s] += out[s, :acc[s] + 1].tolist()
        at += acc + 1
    for s in range(2):
        assert done[s] == seqs[s, 1:1 + len(done[s])].tolist()
    assert kvb.seq_lens.tolist() == (kv.seq_lens + at).tolist()
    g1.close()
    g4.close()


@gpu
def test_captured_and_replayed():
    shape = SHAPES["tiny"]
    wl, W, kv, g, Wd = _setup(shape, (30, 17), 16, 8, 4)
    tok = ref.as_dev([1, 2, 3, 4], torch.int32)
    kvd = dev_kv(kv)
    b = _buffers(4, 2, shape.vocab, 2, 0)
    args = (tok, kvd, b["lg"], b["u"], b["e"], b["acc"], b["out"])
    g.verify_step(*args, advance=False)
    torch.cuda.synchronize()
    want = [b[k].clone() for k in ("lg", "acc", "out")]
    cg = torch.cuda.CUDAGraph()
    with torch.cuda.graph(cg):
        g.verify_step(*args, advance=False)
    for k in ("lg", "acc", "out"):
        b[k].zero_()
    cg.replay()
    torch.cuda.synchronize()
    assert g.status() == mpk.MPK_OK
    assert all(torch.equal(x, b[k]) for x, k in zip(want,
                                                     ("lg", "acc", "out")))
    assert kvd.seq_lens.tolist() == kv.seq_lens.tolist()
    g.close()


@gpu
def test_unmapped_page_is_reported_and_reset():
    shape = SHAPES["tiny"]
    wl, W, kv, g, Wd = _setup(shape, (30, 17), 16, 8, 2)
    kvd = dev_kv(kv)
    tok = ref.as_dev([1, 2], torch.int32)
    b = _buffers(2, 2, shape.vocab, 1, 0)
    args = (tok, kvd, b["lg"], b["u"], b["e"], b["acc"], b["out"])
    g.verify_step(*args, advance=False)
    good = b["lg"].clone()
    kvd.page_table[0, 1] = -1
    g.verify_step(*args, advance=False)
    assert g.status() == mpk.MPK_ERR_KV_PAGE
    kvd.page_table[0, 1] = int(kv.page_table[0, 1])
    g.reset()
    assert g.status() == mpk.MPK_OK
    g.verify_step(*args, advance=False)
    assert g.status() == mpk.MPK_OK and torch.equal(good, b["lg"])
    g.close()


@gpu
def test_wrapper_refusals():
    shape = SHAPES["tiny"]
    wl, W, kv, g, Wd = _setup(shape, (30, 17), 16, 8, 4)
    kvd = dev_kv(kv)
    tok = ref.as_dev([1, 2, 3, 4], torch.int32)
    b = _buffers(4, 2, shape.vocab, 2, 0)
    good = dict(tokens=tok, kv=kvd, logits=b["lg"], uniform=b["u"],
                noise=b["e"], n_accepted=b["acc"], out_tokens=b["out"])
    three = mpk.KVCache(kvd.k_pool, kvd.v_pool,
                        kvd.page_table[[0, 1, 1]].contiguous(),
                        torch.zeros(3, dtype=torch.int32, device="cuda"))
    for bad in (dict(tokens=tok[:3]), dict(tokens=tok.long()),
                dict(kv=three), dict(logits=b["lg"][:3]),
                dict(noise=b["e"][:, :-1]), dict(out_tokens=b["acc"]),
                dict(out_tokens=b["out"][:, :1]), dict(uniform=b["u"].cpu()),
                dict(prefix_len=b["acc"]),
                dict(kv=mpk.KVCache(kvd.k_pool[:1], kvd.v_pool[:1],
                                    kvd.page_table, kvd.seq_lens)),
                dict(kv=mpk.KVCache(kvd.k_pool, kvd.v_pool,
                                    kvd.page_table[:, :-1], kvd.seq_lens))):
        with pytest.raises(mpk.MpkError) as e:
            g.verify_step(**dict(good, **bad))
        assert e.value.status == mpk.MPK_ERR_INVALID_ARG, bad
    g.verify_step(**good)
    torch.cuda.synchronize()
    assert g.status() == mpk.MPK_OK
    g.close()


# ------------------------------------------------------- refusals (no GPU)
def test_refusals_without_a_device(mpk_lib):
    FAKE = 1 << 20
    g = mpk.Graph(synth.TINY, 4, num_workers=8, page_size=16,
                  max_pages_per_seq=4)
    tok = mpk.TokenBatch(2, 4, None, 2)
    kv = mpk._KVCache(FAKE, FAKE, FAKE, FAKE, 5)
    a = mpk.VerifyArgs(tokens=FAKE)

    def call(h=g.handle, t=tok, v=a, lg=FAKE):
        return mpk_lib.mpk_verify_step(
            h, ctypes.byref(t) if t else None, None, ctypes.byref(kv),
            ctypes.byref(v) if v else None, lg, FAKE, 1 << 40, None)
    assert call(h=None) == mpk.MPK_ERR_INVALID_ARG
    assert call(v=None) == mpk.MPK_ERR_INVALID_ARG
    assert call(lg=None) == mpk.MPK_ERR_INVALID_ARG
    assert call(v=mpk.VerifyArgs()) == mpk.MPK_ERR_INVALID_ARG
    assert call() == mpk.MPK_ERR_NOT_BOUND
    ws = mpk_lib.mpk_verify_step_workspace
    assert ws(g.handle, ctypes.byref(tok), 0) > 0
    assert ws(g.handle, ctypes.byref(mpk.TokenBatch(2, 6, None, 3)), 0) == 0
    assert ws(g.handle, ctypes.byref(tok), 3) == 0
    assert ws(None, ctypes.byref(tok), 0) == 0
    chain = mpk.Graph(synth.CHAIN, 1, num_workers=8)
    assert ws(chain.handle, ctypes.byref(mpk.TokenBatch(1, 1, None, 1)),
              0) == 0
    chain.close()
    g.close()
