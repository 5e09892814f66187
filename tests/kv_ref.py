"""Plain numpy restatement of the history-cache calls (include/mpzch.h), one request, run or row
at a time.  Whole numbers and binary32 results are exact; attention is computed in 64 bits."""
import numpy as np

BADLEN, NOBLOCK, BADBLOCK = 32, 64, 128
TOP = 2**31 - 1


def tables(cached, new, bs, free, free_count, table, n_slots):
    """(table, cu_new, seq_len, slots, free_count_out, status)"""
    B, width = table.shape
    table = table.copy()
    count = min(max(int(free_count), 0), len(free))
    cu, seq = np.zeros(B + 1, np.int64), np.zeros(B, np.int64)
    slots = np.full(n_slots, -1, np.int64)
    upto = given = end = status = 0
    for b in range(B):
        c, w = int(cached[b]), int(new[b])
        start, end = end, end + max(w, 0)
        cu[b + 1] = min(end, TOP)
        old, every = -(-c // bs), -(-(c + w) // bs)
        bad = c < 0 or w < 0 or every > width or end > n_slots
        need = 0 if bad else every - old
        upto += need
        short = need > 0 and upto > count
        status |= (BADLEN if bad else 0) | (NOBLOCK if short else 0)
        seq[b] = max(c, 0) if bad or short else c + w
        if bad or short:
            continue
        if need:
            for j in range(need):
                table[b, old + j] = free[count - 1 - (upto - need + j)]
            given = upto
        pos = c + np.arange(w)
        slots[start:end] = table[b, pos // bs].astype(np.int64) * bs + pos % bs
    return table, cu.astype(np.int32), seq.astype(np.int32), slots, count - given, status


def codes(x, s):
    """clamp(rne(x / s)) in binary32; 0 where s is 0, infinite or NaN."""
    if not (s > 0 and np.isfinite(s)):
        return np.zeros(x.shape, np.int8)
    q = (x.astype(np.float32) / np.float32(s)).astype(np.float32)
    return np.clip(np.rint(q), -127, 127).astype(np.int8)


def append(x, slots, cache, scale):
    """x: float32 [n, H, D]; updates cache [blocks, H, bs, D] and scale in place; status bits."""
    blocks, H, bs, _ = cache.shape
    status, i, n = 0, 0, len(slots)
    with np.errstate(all="ignore"):
        while i < n:
            slot, j = int(slots[i]), i + 1
            if slot < 0 or slot // bs >= blocks:
                status |= BADBLOCK if slot >= 0 else 0
                i = j
                continue
            while j < n and int(slots[j]) == slot + j - i and int(slots[j]) % bs:
                j += 1
            blk, o = slot // bs, slot % bs
            for h in range(H):
                run = x[i:j, h]
                own = np.float32(np.abs(run).max()) / np.float32(127)  # max carries NaN on
                before = scale[blk, h] if o else np.float32(0)
                s = np.maximum(own, before)  # carries NaN on
                if o and s != before and not (np.isnan(s) and np.isnan(before)):
                    held = cache[blk, h, :o].astype(np.float32) * before
                    cache[blk, h, :o] = codes(held, s)
                cache[blk, h, o:o + j - i] = codes(run, s)
                scale[blk, h] = s
            i = j
    return status


def attend(q, kc, vc, ks, vs, table, cu, seq, softmax_scale, causal, window):
    """(out, lse, size) in 64 bits, q as float64 [n, Hq, D].  Rows of no request are NaN.  Block ids
    outside the cache hide their keys.  size: what attend_bound needs, (spread, reach, codes):
    the sum of the weights times |v| for each output; the largest softmax_scale * sum |q||k| over
    the keys that a row sees; the sum of |value code| over them times the largest value scale."""
    n, Hq, D = q.shape
    blocks, H, bs, _ = kc.shape
    G = Hq // H
    out, spread = np.full(q.shape, np.nan), np.zeros(q.shape)
    codes = np.zeros(q.shape)
    lse, reach = np.full((n, Hq), np.nan), np.zeros((n, Hq))
    for b in range(len(seq)):
        s = min(max(int(cu[b]), 0), n)
        e = min(max(int(cu[b + 1]), s), n)
        L, w = min(max(int(seq[b]), 0), table.shape[1] * bs), e - s
        if w == 0:
            continue
        ids = table[b, :-(-L // bs)].astype(np.int64)
        there = np.repeat((ids >= 0) & (ids < blocks), bs)[:L]
        ids = np.clip(ids, 0, blocks - 1)
        key = np.arange(L)[None, :]
        pos = (L - w + np.arange(w))[:, None]
        sees = np.broadcast_to(there[None, :], (w, L)).copy()
        if causal:
            sees &= key <= pos
        if window:
            sees &= key > pos - window
        for h in range(H):
            with np.errstate(all="ignore"):
                k = (kc[ids, h].astype(np.float64) * ks[ids, h].astype(np.float64)[:, None, None])
                v = (vc[ids, h].astype(np.float64) * vs[ids, h].astype(np.float64)[:, None, None])
                k, v = k.reshape(-1, D)[:L], v.reshape(-1, D)[:L]
                top = np.abs(vs[ids, h][np.isfinite(vs[ids, h])]).max(initial=0.0)
                many = sees.astype(np.float64) @ np.abs(
                    vc[ids, h].astype(np.float64).reshape(-1, D)[:L]) * float(top)
                for g in range(G):
                    codes[s:e, h * G + g] = many
                    x = q[s:e, h * G + g]
                    z = np.where(sees, softmax_scale * (x @ k.T), -np.inf)
                    far = np.where(sees, abs(softmax_scale) * (np.abs(x) @ np.abs(k).T), 0)
                    reach[s:e, h * G + g] = far.max(1, initial=0.0)
                    m = z.max(1, initial=-np.inf, keepdims=True)
                    p = np.where(sees, np.exp(z - np.where(np.isinf(m), 0, m)), 0)
                    total = p.sum(1, keepdims=True)
                    p = np.divide(p, total, out=np.zeros_like(p), where=total != 0)
                    vz = np.where(np.any(sees, 0)[:, None], v, 0)  # no NaN from hidden blocks
                    out[s:e, h * G + g] = np.where(total != 0, _weighted(p, vz, sees), 0)
                    spread[s:e, h * G + g] = _weighted(p, np.abs(vz), sees)
                    lse[s:e, h * G + g] = np.where(total[:, 0] != 0,
                                                   m[:, 0] + np.log(total[:, 0]), -np.inf)
    return out, lse, (spread, reach, codes)


def _weighted(p, v, sees):
    if np.isfinite(v).all():
        return p @ v
    return np.stack([p[i][sees[i]] @ v[sees[i]] for i in range(len(p))])


def attend_bound(out, size, keys, D, kind):
    """Largest |difference| that the kernels' roundings allow, element by element.

    Weights p_j carry: the score, a dot product of D terms accumulated in fp32 (each add within
    2^-23 of the running sum of |q||k|) and three fp32 factors, (D + 8) 2^-23 reach absolute, plus
    the rounding of a score of up to `reach` itself, 2^-23 reach; the exponential, 2^-21; and the
    rounding to fp16, eps/2 = 2^-11, or to two fp16 parts, 2^-22 (float32 and float16 outputs).
    A weight is kept as p 2^7 scale/vref with vref at most twice the largest scale; where that is
    subnormal in fp16 its rounding is 2^-25 absolute, so an output gets at most 2^-25 2^-7 vref
    sum |code| <= 2^-31 codes (the denominator is at least 1: the largest weight has p >= 1).
    fp16 query parts: exact for 16-bit types, 2^-22 for float32 (inside the D + 8 above).  The
    numerator and the denominator are fp32 sums; with chains of c additions each is c 2^-23 off.
    The quotient doubles what both share.  Then the output is rounded to its type."""
    spread, reach, codes = size
    chain = keys / (16 if kind == "fp32" else 4) + 32
    weight = 2.0**-11 if kind == "bf16" else 2.0**-22
    off = 2 * ((D + 10) * 2.0**-23 * reach[..., None] + 2.0**-21 + chain * 2.0**-23) + weight
    half = {"bf16": 2.0**-8, "fp16": 2.0**-11, "fp32": 2.0**-24}[kind]
    tiny = {"bf16": 0.0, "fp16": 2.0**-25, "fp32": 0.0}[kind]
    return (spread * off + codes * 2.0**-31) * (1 + half) + np.abs(out) * half + tiny + 1e-37


def lse_bound(size, keys, D, kind):
    """The score's error, the sum's relative error, and fp32 roundings of a result of up to
    reach + log(keys)."""
    reach = size[1]
    chain = keys / (16 if kind == "fp32" else 4) + 32
    return ((D + 10) * 2.0**-23 * reach + 2.0**-21 + chain * 2.0**-23
            + 2.0**-22 * (reach + np.log(max(keys, 1)) + 1))
