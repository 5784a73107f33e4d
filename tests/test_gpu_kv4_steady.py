"""The attention kernels in their steady state, against 64 bits: calls with more
units than the GPU has blocks (prompts: tile after tile in one block, buffers
and barriers reused, several segments and cut ones) or warps (decode: rings
that wrap, several segments a warp), references that move on the way, and what
pages may hold.  GPU only."""
import pytest

torch = pytest.importorskip("torch")

import mixed_precision_quantized_act_b200 as mx  # noqa: E402
from mixed_precision_quantized_act_b200 import _lib  # noqa: E402
from tests import kv4_exact  # noqa: E402

pytestmark = pytest.mark.gpu
BLOCKS = 148  # of one launch


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    mx.load()
    return torch.device("cuda:0")


class _Case:
    """A cache of random codes; rows behind a request's last token have NaN
    scales, table entries behind its pages are out of range."""

    def __init__(self, dev, kv, qs, Hq, H, D, page, seed, wide=False, ramp=None, tail=0):
        g = torch.Generator(device=dev).manual_seed(seed)
        rand = lambda *s: torch.rand(s, generator=g, device=dev)  # noqa: E731
        used = [-(-n // page) for n in kv]
        pages = sum(used) + 2
        self.codes = torch.randint(0, 256, (pages, 2, H, page, D // 2), generator=g, device=dev, dtype=torch.uint8)
        s = rand(pages, 2, H, page) * 0.3 + 0.05
        if wide:  # value scales of all sizes, some zero
            s[:, 1] = torch.exp2(rand(pages, H, page) * 36 - 24)
            s[:, 1][rand(pages, H, page) < 0.1] = 0
        z = torch.randint(0, 16, (pages, 2, H, page), generator=g, device=dev, dtype=torch.int32)
        order = torch.randperm(pages, generator=g, device=dev).to(torch.int32)
        self.table = torch.full((len(kv), max(used) + 1), 2 ** 31 - 1, dtype=torch.int32, device=dev)
        free = torch.ones((pages, page), dtype=torch.bool, device=dev)
        at = 0
        for b, n in enumerate(kv):
            ids = order[at:at + used[b]]
            self.table[b, :used[b]] = ids
            t = torch.arange(used[b] * page, device=dev).view(-1, page)
            free[ids.long()] = t >= n
            if ramp:  # key scales grow along the context
                lo, hi = ramp
                s[ids.long(), 0] = (lo * (hi / lo) ** (t.float() / max(1, n)))[:, None, :].expand(-1, H, -1)
            at += used[b]
        meta = (s.half().view(torch.int16).to(torch.int32) & 0xFFFF) | z << 16
        self.meta = torch.where(free[:, None, None, :], torch.tensor(0x0FFF7E00, dtype=torch.int32, device=dev), meta)
        i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=dev)  # noqa: E731
        self.cu, self.lens = i32([sum(qs[:i]) for i in range(len(qs) + 1)]), i32(kv)
        self.q = torch.randn((sum(qs) + tail, Hq, D), generator=g, device=dev).half()
        self.max_q, self.H, self.kv, self.qs = max(qs), H, kv, qs

    def cache(self):
        return mx.KV4Cache(self.codes, self.meta)

    def prompt_units(self):
        """(pair of 128-row tiles, key head, 128 tokens) at most."""
        g = self.q.shape[1] // self.H
        return sum(-(-n * g // 256) * -(-max(1, k) // 128) for k, n in zip(self.kv, self.qs)) * self.H

    def decode_units(self):
        """(request, key head, 32 tokens)."""
        return sum(-(-max(1, k) // 32) for k, n in zip(self.kv, self.qs) if n) * self.H

    def check(self, causal=True, scale=None, poisoned=None):
        cache, D, n = self.cache(), self.q.shape[2], int(self.cu[-1])
        scale = D ** -0.5 if scale is None else scale
        out = torch.full_like(self.q, 77.0)
        lse = torch.full(self.q.shape[:2], 77.0, device=self.q.device)
        ws = mx.kv4_attention_workspace(len(self.kv), self.max_q, self.q.shape[1], cache, self.table.shape[1])
        args = (self.q, cache, self.table, self.lens, self.cu, self.max_q)
        mx.kv4_attention_into(*args, out, ws, scale, causal, lse)
        want, want_lse, tol, lse_tol = kv4_exact.attention(self.q, cache, self.table, self.lens, self.cu, scale, causal)
        keep = torch.ones(self.q.shape[:2], dtype=torch.bool, device=self.q.device) if poisoned is None else ~poisoned
        keep[n:] = False
        off = (kv4_exact.off_by(out[keep], want[keep], tol[keep]),
               kv4_exact.off_by(lse[keep], want_lse[keep], lse_tol[keep]))
        assert max(off) <= 1, off
        assert (out[n:] == 77).all() and (lse[n:] == 77).all()
        if poisoned is not None:
            assert out[:n][poisoned[:n]].isnan().all()
        again = torch.full_like(out, 77.0)
        mx.kv4_attention_into(*args, again, ws, scale, causal)
        assert torch.equal(again.view(torch.int16), out.view(torch.int16))
        assert not ws[:4096].any()
        return out


# ------------------------------------------------------------------ prompts

LONG_PROMPTS = [
    # kv, qs, Hq, H, page
    ([3333], [515], 8, 4, 64),              # pairs of tiles, many tiles a block, every block cuts segments
    ([2100, 1, 900], [300, 1, 257], 8, 8, 16),
    ([1500] * 12, [40] * 12, 6, 2, 128),      # one tile of 120 rows each
    ([260] * 90, [130] * 90, 2, 2, 32),     # short segments, several in one block
    ([1024, 1024], [1024, 1024], 8, 4, 256),
    ([20000], [17], 8, 8, 64),              # few rows, a context cut between nearly all blocks
]


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("kv,qs,Hq,H,page", LONG_PROMPTS, ids=str)
@pytest.mark.parametrize("causal", [True, False])
def test_prompts_of_many_tiles(dev, D, kv, qs, Hq, H, page, causal):
    case = _Case(dev, kv, qs, Hq, H, D, page, seed=D + len(kv), tail=2)
    assert case.prompt_units() > BLOCKS
    case.check(causal)
    mx.sync_status()


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("kv,qs,Hq,H,page", LONG_PROMPTS[:4], ids=str)
@pytest.mark.parametrize("how", ["values", "keys", "both", "steep", "negative"])
def test_prompts_whose_references_move(dev, D, kv, qs, Hq, H, page, how):
    """Scores that grow along the context and value scales of all sizes: the
    reference is passed late, in either half of a tile, and O rescaled."""
    ramp = None if how == "values" else (0.01, 2.0)
    scale = {"steep": 3.0 * D ** -0.5, "negative": -0.5}.get(how)
    case = _Case(dev, kv, qs, Hq, H, D, page, seed=D + sum(qs), wide=how in ("values", "both"), ramp=ramp)
    case.check(scale=scale)
    case.check(causal=False, scale=scale)
    mx.sync_status()


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("scale", [1e-4, 3.0, -0.5, 0.0])
def test_prompts_with_other_scales(dev, D, scale):
    _Case(dev, [333, 90], [100, 90], 4, 2, D, 64, seed=9).check(scale=scale)
    mx.sync_status()


@pytest.mark.parametrize("D", [64, 128])
def test_prompts_nan_rows_poison_only_who_sees_them(dev, D):
    for where in (1050, 1090, 1299):  # in either half of a tile, and the last token
        for kind in (0, 1):
            case = _Case(dev, [1300], [250], 4, 2, D, 64, seed=4)
            case.meta[case.table[0, where // 64].long(), kind, 1, where % 64] = 0x7FFF
            poisoned = torch.zeros((250, 4), dtype=torch.bool, device=dev)
            poisoned[max(0, where - 1050):, 2:] = True
            cache, clean = case.cache(), case.meta.clone()
            out = mx.kv4_attention(case.q, cache, case.table, case.lens, case.cu, 250)
            assert out[poisoned].isnan().all() and out[~poisoned].isfinite().all()
            case.meta[case.table[0, where // 64].long(), kind, 1, where % 64] = 0  # a row of zeros for the reference
            want, _, tol, _ = kv4_exact.attention(case.q, case.cache(), case.table, case.lens, case.cu, D ** -0.5)
            assert kv4_exact.off_by(out[~poisoned], want[~poisoned], tol[~poisoned]) <= 1
            case.meta = clean
    mx.sync_status()


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("causal", [True, False])
def test_prompts_report_pages_and_lengths_out_of_range(dev, D, causal):
    kv, qs, page = [1500, 700], [300, 200], 64

    def bounds():
        with pytest.raises(_lib.MixLLMError) as e:
            mx.sync_status()
        assert e.value.status == _lib.ERR_BOUNDS

    for wrong in (-1, -2 ** 31, 2 ** 31 - 1):
        for entry in (0, 3, -(-kv[0] // page) - 1):
            case = _Case(dev, kv, qs, 8, 4, D, page, seed=5)
            case.table[0, entry] = wrong
            case.check(causal)
            bounds()
    case = _Case(dev, kv, qs, 8, 4, D, page, seed=6, tail=1)
    want, _, tol, _ = kv4_exact.attention(case.q, case.cache(), case.table, case.lens, case.cu, D ** -0.5, causal)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=dev)  # noqa: E731
    for lens, cu in ((i32([1500, case.table.shape[1] * page + 1]), case.cu), (i32([1500, -1]), case.cu),
                     (case.lens, i32([0, 300, 2000])), (case.lens, i32([0, 300, 0])), (case.lens, i32([0, 300, 2 ** 31 - 1]))):
        out = torch.full_like(case.q, 77.0)
        ws = mx.kv4_attention_workspace(2, 300, 8, case.cache(), case.table.shape[1])
        mx.kv4_attention_into(case.q, case.cache(), case.table, lens, cu, 300, out, ws, causal=causal)
        bounds()
        assert kv4_exact.off_by(out[:300], want[:300], tol[:300]) <= 1 and (out[300:] == 77).all()


@pytest.mark.parametrize("D", [64, 128])
def test_prompts_take_strided_tensors(dev, D):
    case = _Case(dev, [1300, 60], [200, 33], 4, 2, D, 64, seed=7)
    T, Hq = case.q.shape[:2]
    wide = torch.zeros((T, Hq + 2, D), dtype=torch.float16, device=dev)
    wide[:, 1:1 + Hq] = case.q
    out = torch.full((T, Hq + 3, D), 77.0, dtype=torch.float16, device=dev)
    big = torch.full((2, case.table.shape[1] + 5), -1, dtype=torch.int32, device=dev)
    big[:, :case.table.shape[1]] = case.table
    ws = mx.kv4_attention_workspace(2, 200, Hq, case.cache(), case.table.shape[1])
    mx.kv4_attention_into(wide[:, 1:1 + Hq], case.cache(), big[:, :case.table.shape[1]], case.lens, case.cu, 200,
                          out[:, 2:2 + Hq], ws)
    want = case.check()
    mx.sync_status()
    assert torch.equal(out[:, 2:2 + Hq], want)
    assert (out[:, :2] == 77).all() and (out[:, 2 + Hq:] == 77).all()


# ------------------------------------------------------------------ few queries

LONG_DECODES = [
    # kv, queries of each, Hq, H, page
    ([5000, 9000, 16000, 1, 0, 12000], 1, 8, 8, 64),
    ([80000, 3], 1, 16, 4, 128),
    ([30000, 28000, 5, 22000], 3, 16, 4, 16),           # 12 rows: two 8-row tiles
    ([300 + 37 * i % 900 for i in range(200)], 1, 4, 4, 32),   # more requests than one warp's scan
    ([2000 + i for i in range(150)], 2, 8, 2, 64),
]


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("kv,n,Hq,H,page", LONG_DECODES, ids=lambda v: str(v)[:30])
@pytest.mark.parametrize("how", ["plain", "values", "keys", "both"])
def test_decodes_whose_rings_wrap(dev, D, kv, n, Hq, H, page, how):
    case = _Case(dev, kv, [n] * len(kv), Hq, H, D, page, seed=D + len(kv), tail=1, wide=how in ("values", "both"),
                 ramp=(0.01, 2.0) if how in ("keys", "both") else None)
    warps, stages = 8 if D * (1 if n * Hq // H <= 8 else 2) > 128 else 16, 3 if D == 128 else 4
    assert case.decode_units() > BLOCKS * warps * stages  # more units a warp than its ring has stages
    case.check()
    if n > 1:
        case.check(causal=False)
    mx.sync_status()
