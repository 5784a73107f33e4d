"""Attention over the 4-bit cache in 64 bits on the tensors' own device, one
request and key head at a time, for contexts too long for plain loops, with the
tolerance of every output: from the definition in the header, sharing no code
with the library."""
import torch

from tests import kv4_ref


def attention(q, cache, table, lens, cu, scale, causal=True):
    """out [T, Hq, D], lse [T, Hq] and their tolerances, in 64 bits; rows outside
    every request are NaN.  Tokens of pages that do not exist are not seen.

    With p the probabilities, s a value's scale, o = sum p v, A = sum p |v|,
    B = sum p s and W = max p s over the n tokens that a row sees:
      * a weight p s is rounded once to fp16, relative to the row's largest so
        far, which is kept between 2^7 and 2^15: 2^-11 A for normal results, and
        2^-25 2^-7 W each for subnormal ones, times |code - z| <= 15;
      * the denominator may be the sum of p as those roundings leave it: 2^-11 |o|,
        and for subnormal weights, taken into account where s is at least a 32nd of
        the largest, 2^-27 |o| each;
      * the result is rounded once to fp16: 2^-11 |o|, 2^-25 below 2^-14;
      * a score is scale s_k (sum q code - z sum q): fp32 sums over D channels of
        terms of at most 15 |q| and products of a few factors, off by at most
        (D + 16) 2^-24 (2 * 15 s_k sum |q|) scale, and tensor-core steps that cut each
        of 17 addends to 24 bits below the largest product's nominal exponent: half
        of the D / 16 steps take normal numbers, products of up to 15 |q|, and half
        unnormalized ones, whose nominal exponent is 2^6 steps of a code:
        17 D / 32 (15 2^-23 + 2^-18) s_k max |q| scale.  The subtraction of the maximum
        and the exponential add 2^-22 of the score's size and 2^-20.  That relative
        error e of p moves numerator and denominator by e A and e |o|;
      * the remaining fp32 sums, of n / 16 steps and a few parts, lose
        (n / 16 + 64) 2^-24 A, and where sum p s code - sum p s z is formed
        2 (2^-17 + (n / 16 + 1) 15 2^-23) B (as kv4_ref derives).
    lse is off by e, by (n / 16 + 64) 2^-24 for its sum, and by 2^-22 of itself."""
    T, Hq, D = q.shape
    pages, _, H, page, _ = cache.codes.shape
    g = Hq // H
    out, tol = (torch.full((T, Hq, D), float("nan"), dtype=torch.float64, device=q.device) for _ in range(2))
    lse, lse_tol = (torch.full((T, Hq), float("nan"), dtype=torch.float64, device=q.device) for _ in range(2))
    cu = cu.tolist()
    for b, n in enumerate(lens.tolist()):
        first, m = cu[b], cu[b + 1] - cu[b]
        if m == 0:
            continue
        row = table[b, :-(-n // page)].long().to(q.device)
        there = ((row >= 0) & (row < pages)).repeat_interleave(page)[:n]
        row = row.clamp(0, pages - 1)
        at = torch.arange(n, device=q.device)
        last = n - m + torch.arange(m, device=q.device) if causal else torch.full((m,), n - 1, device=q.device)
        see = (at[None, :] <= last[:, None]) & there[None, :]                    # [m, n]
        for h in range(H):
            k, v = (kv4_ref.values(cache.codes[row, i, h].reshape(-1, D // 2)[:n], cache.meta[row, i, h].reshape(-1)[:n])
                    for i in (0, 1))
            s_k, s_v = ((cache.meta[row, i, h].reshape(-1)[:n] & 0xFFFF).to(torch.int16).view(torch.float16).double()
                        for i in (0, 1))
            # rows that nobody sees may hold anything
            seen = see.any(0)
            k, v, s_k, s_v = k[seen], v[seen], s_k[seen], s_v[seen]
            x = q[first:first + m, h * g:(h + 1) * g].double()                   # [m, g, D]
            a = torch.einsum("igd,td->igt", x, k) * scale
            a = a.masked_fill(~see[:, None, seen], -torch.inf)
            some = see[:, seen].any(1)
            to = slice(h * g, (h + 1) * g)
            if not some.all():
                out[first:first + m, to][~some], lse[first:first + m, to][~some] = 0, -torch.inf
                tol[first:first + m, to][~some] = lse_tol[first:first + m, to][~some] = 0
            if not some.any():
                continue
            a, x = a[some], x[some]
            big = a.amax(-1, keepdim=True)
            p = torch.exp(a - big)
            total = p.sum(-1, keepdim=True)
            p /= total
            o, A = torch.einsum("igt,td->igd", p, v), torch.einsum("igt,td->igd", p, v.abs())
            B, W = (p * s_v).sum(-1), (p * s_v).amax(-1)
            count = see[some][:, seen].sum(1).double()[:, None]
            mass = x.abs()
            top_k = torch.where(see[some][:, seen], s_k, 0).amax(1)[:, None]
            e = abs(scale) * top_k * (15 * (D + 16) * 2.0 ** -23 * mass.sum(-1)
                                      + 17 * D / 32 * (15 * 2.0 ** -23 + 2.0 ** -18) * mass.amax(-1)) \
                + 2.0 ** -22 * torch.where(a > -torch.inf, a.abs(), 0).amax(-1) + 2.0 ** -20
            steps = count / 16 + 64
            out_tol = (2.0 ** -11 * (A + 2 * o.abs()) + 2.0 ** -25
                       + (count * 15 * 2.0 ** -32 * W)[..., None] + count[..., None] * 2.0 ** -27 * o.abs()
                       + e[..., None] * (A + o.abs()) + steps[..., None] * 2.0 ** -24 * A
                       + (2 * (2.0 ** -17 + (count / 16 + 1) * 15 * 2.0 ** -23) * B)[..., None])
            big = (big + total.log())[..., 0]
            for whole, part in ((out, o), (tol, out_tol), (lse, big), (lse_tol, e + steps * 2.0 ** -24 + 2.0 ** -22 * big.abs())):
                whole[first:first + m, to][some] = part
    return out, lse, tol, lse_tol


def off_by(got, want, tol):
    """The largest error in units of its tolerance (NaN or infinite errors count as infinite)."""
    want, tol = want.to(got.device), tol.to(got.device)
    off = (got.double() - want).abs() / tol.clamp(min=1e-300)
    off = torch.where(got.double() == want, 0.0, off)
    return float(torch.nan_to_num(off, nan=float("inf")).max()) if off.numel() else 0.0
