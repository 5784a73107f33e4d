"""Plain 64-bit restatements of the KV-cache operators, on the CPU, for the
tests: written from the definitions in the header, sharing no code with the
library."""
import numpy as np
import torch


def quantize_row(x):
    """x fp16 [..., D] (numpy) -> codes uint8, scale fp16, zero int, as the
    header defines them (IEEE fp32 divisions, rounding half to even)."""
    x32 = x.astype(np.float32)
    bad = ~np.isfinite(x32).all(-1)
    x32 = np.where(bad[..., None], np.float32(0), x32)
    lo = np.minimum(x32.min(-1), np.float32(0))
    hi = np.maximum(x32.max(-1), np.float32(0))
    s16 = ((hi - lo) / np.float32(15)).astype(np.float16)
    s = s16.astype(np.float32)
    div = np.where(s > 0, s, np.float32(1))
    z = np.clip(np.rint(-lo / div), 0, 15).astype(np.int64)
    q = np.clip(np.rint(x32 / div[..., None]).astype(np.int64) + z[..., None], 0, 15)
    z = np.where(s > 0, z, 0)
    q = np.where((s > 0)[..., None], q, 0)
    s16 = np.where(bad, np.float16(np.nan), s16)
    return q.astype(np.uint8), s16, z


def pack(codes, s16, z):
    """-> code bytes [..., D/2] and meta uint32 [...]."""
    by = (codes[..., 0::2] | codes[..., 1::2] << 4).astype(np.uint8)
    return by, s16.view(np.uint16).astype(np.uint32) | z.astype(np.uint32) << 16


def values(codes, meta):
    """fp64 values of code bytes [..., D/2] and meta int32 [...] (torch, any device)."""
    q = torch.stack((codes & 15, codes >> 4), -1).flatten(-2).double()
    s = (meta & 0xFFFF).to(torch.int16).view(torch.float16).double()
    return (q - (meta >> 16 & 15).double()[..., None]) * s[..., None]


def rotate(x, table, pos, rotary):
    """x fp16 [T, H, D] -> rotated, every product and sum rounded to fp32, then
    fp16 (numpy)."""
    half = rotary // 2
    c, s = table[pos][:, None, :half], table[pos][:, None, half:]
    a, b = x[..., :half].astype(np.float32), x[..., half:rotary].astype(np.float32)
    out = x.copy()
    out[..., :half] = (a * c - b * s).astype(np.float16)
    out[..., half:rotary] = (b * c + a * s).astype(np.float16)
    return out


def attention(q, codes, meta, table, kv_lens, cu_q, scale, causal, bad_pages=()):
    """fp64 outputs [T, Hq, D], lse [T, Hq] and the tolerance of every output;
    rows outside every request are NaN.

    Tolerance of one output o = sum p v / sum p, with A = sum p |v| / sum p:
      * p times the value's scale is rounded once to fp16: 2^-11 of each term
        (2^-11 A), or, where the scaled weight p s / max s is below fp16's
        smallest normal 2^-14, an absolute 2^-25 max s per term, times |code - z|
        <= 15;
      * the denominator sums p as rounded where the value's scale is at least an
        eighth of the largest: 2^-11 |o| for its terms of normal weights, and
        2^-25 * 8 |o| / sum p for each of a smaller one;
      * the result is rounded once to fp16: 2^-11 |o| (2^-25 below 2^-14);
      * the score's products are exact; their fp32 sum over D channels, the
        scale factors, the subtraction of the maximum and the exponential leave a
        relative error in p of at most e = (D + 16) 2^-24 max_t sum |q k| scale +
        2^-20, which moves numerator and denominator by e A and e |o|;
      * the remaining fp32 sums over n terms (in tiles of 16 and a few parts)
        by (n / 16 + 64) 2^-24 A at most;
      * the sum of p s (code - z) is taken as sum p s code - sum p s z, each of
        non-negative terms and at most 15 B, B = sum p s / sum p: where code = z
        carries nearly all the weight, A is far below B.  A tensor-core step
        adds 16 products to the running sum: aligning them to the largest one's
        exponent drops at most 2^-17 of the largest p s, in units of a code (24 bits
        below a product of up to 2^4 codes, with a factor 2^2 for the
        unnormalized high nibbles and one 2^1 for the addends), and the sum is
        cut to 24 bits, 2^-23 of up to 15 B; n / 16 + 1 steps, two sums:
        2 (2^-17 + (n / 16 + 1) 15 2^-23) B."""
    T, Hq, D = q.shape
    H, page = codes.shape[2], codes.shape[3]
    g = Hq // H
    out = torch.full((T, Hq, D), float("nan"), dtype=torch.float64)
    lse = torch.full((T, Hq), float("nan"), dtype=torch.float64)
    tol = torch.zeros((T, Hq, D), dtype=torch.float64)
    for b in range(len(kv_lens)):
        n, first, last = int(kv_lens[b]), int(cu_q[b]), int(cu_q[b + 1])
        m = last - first
        used = -(-n // page)
        ids = [int(table[b, j]) for j in range(used)]
        ok = torch.tensor([0 <= i < codes.shape[0] for i in ids for _ in range(page)], dtype=torch.bool)[:n]
        pick = torch.tensor([i if 0 <= i < codes.shape[0] else 0 for i in ids], dtype=torch.long)
        kv = values(codes[pick], meta[pick])                       # [used, 2, H, page, D]
        kv = kv.permute(1, 2, 0, 3, 4).reshape(2, H, used * page, D)[:, :, :n]
        s_v = (meta[pick, 1] & 0xFFFF).to(torch.int16).view(torch.float16).double()
        s_v = s_v.permute(1, 0, 2).reshape(H, used * page)[:, :n]
        for i in range(m):
            see = (n - m + i + 1 if causal else n)
            see = max(0, min(n, see))
            for h in range(Hq):
                keep = ok[:see]
                k, v, sv = kv[0, h // g, :see][keep], kv[1, h // g, :see][keep], s_v[h // g, :see][keep]
                if k.shape[0] == 0:
                    out[first + i, h], lse[first + i, h] = 0, -float("inf")
                    continue
                x = q[first + i, h].double()
                sc = (k @ x) * scale
                p = torch.exp(sc - sc.max())
                w = p / p.sum()
                o = w @ v
                out[first + i, h] = o
                lse[first + i, h] = torch.logsumexp(sc, 0)
                A = w @ v.abs()
                big = sv.max() if sv.numel() else torch.zeros(())
                small = (p * sv < 2.0 ** -14 * big).sum()
                e = (D + 16) * 2.0 ** -24 * float(((k.abs() @ x.abs()) * abs(scale)).max()) + 2.0 ** -20
                tol[first + i, h] = (2.0 ** -11 * (A + 2 * o.abs()) + 2.0 ** -25
                                     + small * 2.0 ** -25 * (15 * big + 8 * o.abs()) / p.sum()
                                     + e * (A + o.abs()) + (see / 16 + 64) * 2.0 ** -24 * A
                                     + 2 * (2.0 ** -17 + (see / 16 + 1) * 15 * 2.0 ** -23) * (w @ sv))
    return out, lse, tol
