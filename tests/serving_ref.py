"""Plain float64 forms of the serving operators (numpy), written from their
definitions, with the error bounds their tests use.

A rounding to bf16 is off by at most 2^-8 of the value, one to fp32 by 2^-24.
"""
import numpy as np
import torch

BF, F32 = 2.0 ** -8, 2.0 ** -24


def f64(t):
    return t.detach().cpu().double().numpy()


def gather(pool, row, page_size, lo, hi):
    """Tokens lo..hi-1 of a sequence from one layer's pool [pages, Hkv, P, d]
    (float64): [hi - lo, Hkv, d]."""
    t = np.arange(lo, hi)
    pages = np.asarray(row)[t // page_size]
    assert (pages >= 0).all()
    return pool[pages, :, t % page_size]


def inv_freq(rot, theta, scaling="plain", factor=1.0, low=1.0, high=4.0,
             old=8192.0):
    i = np.arange(rot // 2, dtype=np.float64)
    f = theta ** (-2.0 * i / rot)
    if scaling == "linear":
        return f / factor
    if scaling == "bands":
        out = []
        for x in f:
            wave = 2 * np.pi / x
            if wave > old / low:
                out.append(x / factor)
            elif wave < old / high:
                out.append(x)
            else:
                m = (old / wave - low) / (high - low)
                out.append((1 - m) * x / factor + m * x)
        return np.array(out)
    if scaling == "ramp":
        def dim(turns):
            return rot * np.log(old / (turns * 2 * np.pi)) / (2 * np.log(theta))
        a, b = max(np.floor(dim(high)), 0), min(np.ceil(dim(low)), rot - 1)
        if a == b:
            b += 0.001
        ramp = np.clip((i - a) / (b - a), 0, 1)
        return f / factor * ramp + f * (1 - ramp)
    return f


def rotate(x, pos, inv, rot, inter, attn=1.0):
    """x [..., heads, d] at positions pos [...]: value and the sum of the
    magnitudes that a rotated value is formed from."""
    c = np.cos(pos[..., None] * inv)[..., None, :] * attn
    s = np.sin(pos[..., None] * inv)[..., None, :] * attn
    a_at = np.arange(rot // 2) * (2 if inter else 1)
    b_at = a_at + (1 if inter else rot // 2)
    y, mag = x.copy(), np.abs(x)
    a, b = x[..., a_at], x[..., b_at]
    y[..., a_at], y[..., b_at] = a * c - b * s, b * c + a * s
    mag[..., a_at] = np.abs(a * c) + np.abs(b * s)
    mag[..., b_at] = np.abs(b * c) + np.abs(a * s)
    return y, mag


def rms(x, w, eps):
    r = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    return x * r * w


def attend(q, kpool, vpool, table, page_size, seq_lens, starts, prefix, first,
           scale):
    """q [T, Hq, d]; kpool, vpool one layer, float64; prefix[b], first[b]: the
    sequence's prefix length and the one whose row holds it.  Returns out,
    lse, the outputs' error bound and the log sums' bound."""
    T, Hq, d = q.shape
    Hkv = kpool.shape[1]
    grp = Hq // Hkv
    out, lse = np.zeros_like(q), np.full((T, Hq), -np.inf)
    tol, ltol = np.zeros_like(q), np.zeros((T, Hq))
    for b in range(len(starts) - 1):
        n = starts[b + 1] - starts[b]
        end = seq_lens[b] + n
        if n == 0:
            continue
        k, v = (np.concatenate([
            gather(p, table[first[b]], page_size, 0, prefix[b]),
            gather(p, table[b], page_size, prefix[b], end)])
            for p in (kpool, vpool))
        for i in range(n):
            t, m = starts[b] + i, seq_lens[b] + i + 1
            for h in range(Hq):
                kk, vv = k[:m, h // grp], v[:m, h // grp]
                s = kk @ q[t, h] * scale
                top = s.max()
                with np.errstate(invalid="ignore", over="ignore"):
                    e = np.exp(s - top)
                    L = e.sum()
                    p = e / L
                    out[t, h] = p @ vv
                    # a score's fp32 error: a dot of d products, the scale
                    # and the exponent's rounding (times log2 e on the way)
                    mags = np.abs(kk) @ np.abs(q[t, h]) * abs(scale)
                    err = ((d + 8) * mags.max() + 4 * np.abs(s).max()) * F32
                    # ex2 to 2^-22, weights rounded to bf16 once, sums of m
                    rel = BF + 2 * err + 2.0 ** -20 + 2 * m * F32
                    tol[t, h] = BF * np.abs(out[t, h]) + rel * 1.01 * (
                        p @ np.abs(vv)) + 1e-30
                lse[t, h] = top + np.log(L)
                ltol[t, h] = (err + 2.0 ** -21 + m * F32 +
                              4 * F32 * (abs(top) + abs(lse[t, h])))
    return out, lse, tol, ltol


def verify(logits, tokens, starts, uniform, noise, temp, draft, kind, vocab,
           max_out):
    """One sequence after the other, one draft after the other."""
    B = len(starts) - 1
    acc = np.zeros(B, np.int64)
    out = np.full((B, max_out), -1, np.int64)
    lp = np.zeros((B, max_out))

    def soft(x, T):
        x = np.where(np.isnan(x), -np.inf, x)
        if x.max() == -np.inf:
            return np.zeros_like(x)
        if x.max() == np.inf:
            return (x == np.inf) / (x == np.inf).sum()
        e = np.exp((x - x.max()) / T)
        return e / e.sum()

    def race(w, e):
        if not (w > 0).any():
            return -1
        with np.errstate(divide="ignore", invalid="ignore"):
            s = np.where(w > 0, w / e, -1.0)
        return int(np.argmax(s))

    for b in range(B):
        n, T = starts[b + 1] - starts[b], temp[b]
        for i in range(n):
            r = starts[b] + i
            row = np.where(np.isnan(logits[r]), -np.inf, logits[r])
            d = tokens[r + 1] if i < n - 1 else -1
            have = 0 <= d < vocab
            if T <= 0:
                best = -1 if row.max() == -np.inf else int(np.argmax(row))
                if have and d == best:
                    out[b, i] = d
                    acc[b] += 1
                    continue
                out[b, i] = best
                break
            p = soft(logits[r], T)
            q = None
            if have:
                if kind == "none":
                    q = np.zeros(vocab)
                    q[d] = 1.0
                elif kind == "probs":
                    q = draft[r]
                else:
                    q = soft(draft[r], T)
                if uniform[r] * q[d] < p[d]:
                    out[b, i], lp[b, i] = d, np.log(p[d])
                    acc[b] += 1
                    continue
            w = p
            if have:
                w = np.maximum(p - q, 0.0)
                if kind == "none":
                    w = np.where(np.arange(vocab) == d, 0.0, p)
                if not (w > 0).any():
                    w = p
            t = race(w, noise[b])
            out[b, i] = t
            lp[b, i] = np.log(p[t]) if t >= 0 else 0.0
            break
    return acc, out, lp


def as_dev(x, dtype):
    return torch.as_tensor(np.asarray(x)).to(dtype).cuda()
