"""Plain restatements of the 8-bit operators for the tests, from the header's
definitions, sharing no code with the library."""
import numpy as np
import torch

BLOCK = 16


def quantize_rows(x):
    """x [M, K] (numpy, fp16 or fp32) -> int8 codes and fp32 scales, IEEE fp32 quotients, rounding half to even."""
    x = x.astype(np.float32)
    bad = ~np.isfinite(x).all(1)
    s = (np.where(bad[:, None], np.float32(0), np.abs(x)).max(1, initial=0) / np.float32(127)).astype(np.float32)
    div = np.where(s > 0, s, np.float32(1))[:, None]
    q = np.where((s > 0)[:, None] & ~bad[:, None], np.clip(np.rint(np.where(bad[:, None], 0, x) / div), -127, 127), 0)
    return q.astype(np.int8), np.where(bad, np.float32(np.nan), s)


def turned(x, w, eps, table, pos, rotary):
    """x fp16 [T, H, D] -> fp64 heads, normalized by w (or None) and rotated, and the sum of the magnitudes of what
    each output adds up."""
    x = x.double()
    if w is not None:
        x = x / (x.square().mean(-1, keepdim=True) + eps).sqrt() * w.double()
    out, mag = x.clone(), x.abs()
    if rotary:
        half = rotary // 2
        c, s = table.double()[pos.long()][:, None, :half], table.double()[pos.long()][:, None, half:]
        a, b = x[..., :half], x[..., half:rotary]
        out[..., :half], out[..., half:rotary] = a * c - b * s, b * c + a * s
        mag[..., :half], mag[..., half:rotary] = (a * c).abs() + (b * s).abs(), (b * c).abs() + (a * s).abs()
    return out, mag


def append(codes, scales, slots, k, v):
    """Writes k, v fp16 [T, H, D] (numpy; as they go into the cache) into copies of codes uint8 [pages, 2, H, page, D]
    and scales fp32 [pages, 2, H, page / 16], block by block."""
    codes, scales = codes.copy(), scales.copy()
    page = codes.shape[3]
    blocks = {}
    for t, slot in enumerate(slots):
        if slot >= 0:
            blocks.setdefault(int(slot) // BLOCK, []).append((t, int(slot) % BLOCK))
    f32 = np.float32
    for block, tokens in blocks.items():
        at, sub = block * BLOCK // page, block * BLOCK % page // BLOCK
        rows = slice(sub * BLOCK, sub * BLOCK + BLOCK)
        for kind, x in ((0, k), (1, v)):
            for h in range(codes.shape[2]):
                new = np.stack([x[t, h] for t, _ in tokens]).astype(f32)
                before = f32(0) if any(r == 0 for _, r in tokens) else scales[at, kind, h, sub]
                if not np.isfinite(new).all() or np.isnan(before):
                    s = f32(np.nan)
                else:
                    s = max(before, np.abs(new).max() / f32(127))
                if s > before and not any(r == 0 for _, r in tokens):
                    old = codes[at, kind, h, rows].astype(f32) - f32(128)
                    codes[at, kind, h, rows] = np.clip(np.rint(old * (before / s)), -127, 127) + 128
                q = np.clip(np.rint(new / s), -127, 127) if s > 0 else np.zeros_like(new)
                for (_, r), row in zip(tokens, q):
                    codes[at, kind, h, sub * BLOCK + r] = row + 128
                scales[at, kind, h, sub] = s
    return codes, scales


def values(codes, scales):
    """fp64 values of codes [..., page, D] and scales [..., page / 16] (torch)."""
    return (codes.double() - 128) * scales.double().repeat_interleave(BLOCK, -1)[..., None]


def attention(q, codes, scales, table, kv_lens, cu_q, scale, causal):
    """fp64 outputs [T, Hq, D], lse [T, Hq] and the tolerance of every output; rows outside every request are NaN.

    Tolerance of one output o = sum p v / sum p, with A = sum p |v| / sum p, W the row's largest weight p s_v and S its
    largest scale of a value:
      * a weight is rounded once to fp16, 2^-11 of it, or below 2^-21 W by at most 2^-32 W, times |code - 128| <= 128;
      * the denominator sums p as rounded where the value's scale is at least S / 8: 2^-11 |o| for normal weights and
        2^-32 W 8 / S |o| for each smaller one;
      * the result is rounded once to fp16: 2^-11 |o|, and 2^-25 below its normal numbers;
      * the score's products are exact; their fp32 sum over D channels, the scale factors, the sum with the logarithm
        of the value's scale, the subtraction of the reference and the exponential leave a relative error in p of at
        most e = (D + 16) 2^-24 max_t sum |q k| scale + 2^-24 max |score| + 2^-20, which moves numerator and
        denominator by e A and e |o|;
      * fp32 sums over n terms, in steps of 16 that may cut instead of round: (n / 16 + 64) 2^-23 A."""
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
        kv = values(codes[pick], scales[pick]).permute(1, 2, 0, 3, 4).reshape(2, H, used * page, D)[:, :, :n]
        s_v = scales[pick, 1].double().repeat_interleave(BLOCK, -1).permute(1, 0, 2).reshape(H, used * page)[:, :n]
        for i in range(m):
            see = max(0, min(n, n - m + i + 1 if causal else n))
            for h in range(Hq):
                keep = ok[:see]
                k, v, sv = kv[0, h // g, :see][keep], kv[1, h // g, :see][keep], s_v[h // g, :see][keep]
                if k.shape[0] == 0:
                    out[first + i, h], lse[first + i, h] = 0, -float("inf")
                    continue
                x = q[first + i, h].double()
                sc = (k @ x) * scale
                p = torch.exp(sc - sc.max())
                total = p.sum()
                o = (p / total) @ v
                out[first + i, h], lse[first + i, h] = o, torch.logsumexp(sc, 0)
                A, W, S = (p / total) @ v.abs(), float((p * sv).max()), max(float(sv.max()), 1e-300)
                small = int((p * sv < 2.0 ** -21 * W).sum())
                e = (D + 16) * 2.0 ** -24 * float(((k.abs() @ x.abs()) * abs(scale)).max()) \
                    + 2.0 ** -24 * float(sc.abs().max()) + 2.0 ** -20
                tol[first + i, h] = (2.0 ** -11 * (A + 2 * o.abs()) + 2.0 ** -25
                                     + small * 2.0 ** -32 * W * (128 + 8 * o.abs() / S) / total
                                     + e * (A + o.abs()) + (see / 16 + 64) * 2.0 ** -23 * A)
    return out, lse, tol
