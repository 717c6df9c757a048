"""Paged cache on the GPU: rotary positions, appended rows and attention over
pages against plain 64-bit evaluations, through the public binding.

Tolerances come from the roundings of each path.  A rounding to nearest is off
by at most finfo.eps / 2 relative (bf16 2^-8, fp32 2^-24).

rope: the cosine and sine are rounded once (2^-24 each), the rotation takes two
FP32 roundings, so |error| <= 2^-22 mscale (|x_a| + |x_b|) covers them; then one
rounding to the type.
attention, FP32: a score sums D products in FP32, |error| <= (D + 2) 2^-24 scale
sum |q||k|, which shifts a weight by that relative amount; the sums over n keys
add n 2^-24 and exp2f, rescaling and merging a few 2^-22.
attention, BF16: weights enter the product with V rounded to bf16 (2^-8 each),
against sum p |v|; the output is rounded once more; scores and sums as above."""
import math

import numpy as np
import pytest
import torch

import block_attention_b200 as ba

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}
HALF_STEP = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}


def gen(seed):
    return torch.Generator().manual_seed(seed)


def randn(g, *shape, dt):
    return torch.randn(*shape, generator=g).to(DT[dt])


# --------------------------------------------------------------------- rope

def turned(x, pos, freq, m, inter, sign=1.0):
    """float64 rotation of x [rows, H, D] and the sum |x_a| + |x_b| behind each value."""
    x = x.double()
    h = freq.numel()
    y, mag = x.clone(), x.abs() / 2 ** 40
    a, b = (slice(0, 2 * h, 2), slice(1, 2 * h, 2)) if inter else (slice(0, h), slice(h, 2 * h))
    ang = sign * pos.double()[:, None] * freq
    c, s = m * torch.cos(ang)[:, None], m * torch.sin(ang)[:, None]
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., b] * c + x[..., a] * s
    mag[..., a] = mag[..., b] = abs(m) * (x[..., a].abs() + x[..., b].abs())
    return y, mag


def check_turned(got, ref, mag, dt):
    err = (got.cpu().double() - ref).abs()
    tol = 2.0 ** -22 * mag + (HALF_STEP[dt] * ref.abs() if dt == "bf16" else 0)
    assert (err <= tol + 1e-30).all(), float((err - tol).max())


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("rows,H,D,rot", [(1, 1, 128, 128), (33, 5, 128, 64), (7, 3, 64, 64),
                                          (300, 2, 80, 34), (5, 40, 96, 2), (4, 2, 64, 0)])
def test_rope(dt, inter, rows, H, D, rot):
    g = gen(rows + rot)
    x = randn(g, rows, H, D, dt=dt)
    pos = torch.randint(-1000, 1000000, (rows,), generator=g, dtype=torch.int32)
    freq, m = (ba.rope_freqs(rot, 1e6, scaling="yarn", factor=8, original_ctx=16384)
               if rot >= 2 else (None, 1.0))
    ref, mag = turned(x, pos, torch.zeros(0).double() if freq is None else freq.cpu(), m, inter)
    out = ba.rope(x.cuda(), pos.cuda(), freq, layout=int(inter), mscale=m)
    check_turned(out, ref, mag, dt)
    # strided views of one buffer, in place, next to rows that must stay
    buf = randn(g, rows, H + 2, D + 16, dt=dt).cuda()
    before = buf.clone()
    view = buf[:, 1:H + 1, 8:D + 8]
    view.copy_(x)
    ba.rope(view, pos.cuda(), freq, layout=int(inter), mscale=m, out=view)
    assert torch.equal(view, out)
    view.copy_(before[:, 1:H + 1, 8:D + 8])
    assert torch.equal(buf, before)


@pytest.mark.parametrize("inter", [False, True])
def test_rope_inverse_is_the_gradient(inter):
    rows, H, D, rot = 9, 3, 64, 48
    g = gen(5)
    x, dy = randn(g, rows, H, D, dt="f32"), randn(g, rows, H, D, dt="f32")
    pos = torch.arange(rows, dtype=torch.int32) * 1001
    freq, _ = ba.rope_freqs(rot, 1e4)
    kw = dict(layout=int(inter), mscale=1.25)
    back = ba.rope(dy.cuda(), pos.cuda(), freq, inverse=True, **kw)
    # the formula's gradient
    ref, mag = turned(dy, pos, freq.cpu(), 1.25, inter, sign=-1.0)
    check_turned(back, ref, mag, "f32")
    # differences: the call is linear, so <dy, rope(x + h e) - rope(x)> = h <back, e>
    e = randn(g, rows, H, D, dt="f32")
    y0 = ba.rope(x.cuda(), pos.cuda(), freq, **kw).cpu().double()
    y1 = ba.rope((x + e).cuda(), pos.cuda(), freq, **kw).cpu().double()
    lhs, rhs = (dy.double() * (y1 - y0)).sum(), (back.cpu().double() * ((x + e) - x).double()).sum()
    bound = 2.0 ** -20 * (dy.double().norm() * (x.double().norm() + e.double().norm()))
    assert abs(lhs - rhs) <= bound


def test_rope_zero_rows_and_infinities():
    freq, _ = ba.rope_freqs(64, 1e6)
    assert ba.rope(torch.empty(0, 4, 64, device="cuda"),
                   torch.empty(0, dtype=torch.int32, device="cuda"), freq).shape == (0, 4, 64)
    x = torch.ones(2, 1, 64, device="cuda")
    x[0, 0, 3] = math.inf
    y = ba.rope(x, torch.tensor([5, 5], dtype=torch.int32, device="cuda"), freq)
    assert torch.isfinite(y[1]).all() and (~torch.isfinite(y[0])).sum() == 2


# ------------------------------------------------------------------- append

def pool(g, pages, Hkv, ps, D, dt):
    return randn(g, pages, Hkv, ps, D, dt=dt)


def deal(g, pages, B, width):
    """A table of distinct random pages."""
    return torch.randperm(pages, generator=g)[:B * width].view(B, width).to(torch.int32)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("D,rot,ps", [(128, 128, 16), (64, 32, 7), (40, 20, 32), (128, 0, 1)])
def test_append_ragged(dt, inter, D, rot, ps):
    g = gen(D + ps)
    lens, counts = [0, 3, 30, 15, 9, 0], [5, 0, 1, 40, 2, 7]
    B, Hq, Hkv, rows = len(lens), 4, 2, sum(counts) + 3  # three rows behind the last sequence
    width = -(-(max(a + b for a, b in zip(lens, counts))) // ps)
    pages = B * width + 4
    qkv = randn(g, rows, Hq + 2 * Hkv, D, dt=dt)
    kp, vp = pool(g, pages, Hkv, ps, D, dt), pool(g, pages, Hkv, ps, D, dt)
    table = deal(g, pages, B, width)
    starts = torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32)
    freq, m = ba.rope_freqs(rot, 1e6) if rot else (None, 1.0)
    q_out = torch.full((rows, Hq, D), 7.0, dtype=DT[dt])
    dev = [t.cuda() for t in (qkv, kp, vp, table, torch.tensor(lens, dtype=torch.int32), starts,
                              q_out)]
    dq, dk, dv = dev[0].split([Hq, Hkv, Hkv], 1)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    ba.paged_append(dk, dv, dev[1], dev[2], dev[3], dev[4], row_starts=dev[5], inv_freq=freq,
                    layout=int(inter), mscale=m, q=dq, q_out=dev[6], advance=True, err=err)
    f = torch.zeros(0).double() if freq is None else freq.cpu()
    ek, ev, eq = kp.double(), vp.double(), q_out.double()
    mk, mq = torch.zeros_like(ek), torch.zeros_like(eq)
    for b in range(B):
        for j in range(counts[b]):
            r, p = int(starts[b]) + j, lens[b] + j
            t = torch.tensor([p])
            page, slot = int(table[b, p // ps]), p % ps
            y, mag = turned(qkv[r:r + 1, Hq:Hq + Hkv], t, f, m, inter)
            ek[page, :, slot], mk[page, :, slot] = y[0], mag[0]
            ev[page, :, slot] = qkv[r, Hq + Hkv:].double()
            y, mag = turned(qkv[r:r + 1, :Hq], t, f, m, inter)
            eq[r], mq[r] = y[0], mag[0]
    assert torch.equal(dev[2].cpu().double(), ev)  # V is copied; the other slots are untouched
    untouched = mk == 0
    assert torch.equal(dev[1].cpu().double()[untouched], ek[untouched])
    check_turned(dev[1], ek, mk, dt)
    check_turned(dev[6], eq, mq, dt)
    assert torch.equal(dev[6][sum(counts):].cpu(), q_out[sum(counts):])
    assert dev[4].tolist() == [a + b for a, b in zip(lens, counts)] and err.item() == 0


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_append_commits_a_round_in_all_layers(dt):
    """n_emit rows of each block into every layer's pools, as kv_commit does on a dense cache."""
    g = gen(3)
    L, B, blk, Hkv, D, ps, cap = 3, 4, 8, 2, 64, 16, 64
    lens = torch.tensor([0, 15, 16, 40], dtype=torch.int32)
    n_emit = torch.tensor([8, 1, 0, 5], dtype=torch.int32)
    kb, vb = randn(g, L, B, blk, Hkv, D, dt=dt).cuda(), randn(g, L, B, blk, Hkv, D, dt=dt).cuda()
    table = deal(g, 20, B, cap // ps)
    kp = torch.zeros(L, 20, Hkv, ps, D, dtype=DT[dt], device="cuda")
    vp = torch.zeros_like(kp)
    kc = torch.zeros(L, B, Hkv, cap, D, dtype=DT[dt], device="cuda")
    vc = torch.zeros_like(kc)
    l1, l2 = lens.cuda(), lens.cuda()
    ba.kv_commit(kc, vc, kb, vb, l1, n_emit.cuda())
    ba.paged_append(kb, vb, kp, vp, table.cuda(), l2, n_rows=n_emit.cuda(), advance=True)
    assert torch.equal(l1, l2)
    for p, c in ((kp, kc), (vp, vc)):
        flat = p[:, table.cuda().long()]  # [L, B, pages, Hkv, ps, D]
        assert torch.equal(flat.permute(0, 1, 3, 2, 4, 5).reshape(c.shape), c)


def test_append_refused_rows_are_skipped_and_reported():
    """Device-side refusals: a page outside the pool, a position outside the
    table, a count outside the block; the other sequences are written."""
    Hkv, D, ps, blk = 1, 64, 16, 4
    k = torch.ones(4, blk, Hkv, D, device="cuda")
    table = torch.tensor([[0, 9], [1, 1], [2, -1], [3, 3]], dtype=torch.int32).cuda()
    lens = torch.tensor([14, 30, 16, 0], dtype=torch.int32).cuda()
    kp = torch.zeros(4, Hkv, ps, D, device="cuda")
    vp = torch.zeros_like(kp)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    ba.paged_append(k, k, kp, vp, table, lens, advance=True, err=err)
    assert err.item() in (-1, -4)
    assert lens.tolist() == [14, 30, 16, 4]
    used = kp[:, 0, :, 0].bool()
    assert used[0].nonzero().flatten().tolist() == [14, 15]  # the rows before the bad page
    assert used[1].nonzero().flatten().tolist() == [14, 15]
    assert not used[2].any() and used[3].nonzero().flatten().tolist() == [0, 1, 2, 3]
    err.zero_()
    n = torch.tensor([5, 0, 0, -1], dtype=torch.int32).cuda()
    ba.paged_append(k, k, kp.zero_(), vp, table, lens, n_rows=n, advance=True, err=err)
    assert err.item() == -4 and lens.tolist() == [14, 30, 16, 4] and not kp.any()


def test_append_refuses_starts_past_the_rows_and_lengths_past_32_bits():
    """Starts beyond the rows given, and lengths beyond 2^31 - 1, neither write
    nor advance."""
    dev = dict(dtype=torch.int32, device="cuda")

    def run(starts, lens, ps, cols):
        k = torch.ones(6, 1, 4, device="cuda")
        pool = torch.zeros(2, 3, 1, ps, 4, device="cuda")
        err = torch.zeros(1, **dev)
        ctx = torch.tensor(lens, **dev)
        table = torch.arange(3, **dev)[:, None].expand(3, cols).contiguous()
        ba.paged_append(k, k, pool[0], pool[1], table, ctx, row_starts=torch.tensor(starts, **dev),
                        advance=True, err=err)
        return ctx.tolist(), err.item(), [int(n) // 4 for n in pool[0].sum((1, 2, 3))]

    assert run([0, 2, 4, 6], [1, 2, 3], 16, 1) == ([3, 4, 5], 0, [2, 2, 2])
    # the last sequence's end is not there
    assert run([0, 2, 4, 9], [1, 2, 3], 16, 1) == ([3, 4, 3], -4, [2, 2, 0])
    lens, err, slots = run([0, 4, 2, 6], [1, 2, 3], 16, 1)  # a negative count
    assert lens[1] == 2 and slots[1] == 0
    top = 2 ** 31 - 1
    got = run([0, 2, 4, 6], [top - 1, 0, top - 2], 1 << 16, 1 << 15)
    assert got == ([top - 1, 2, top], -4, [0, 2, 2])


# ---------------------------------------------------------------- attention

class Attn:
    """Inputs of one call, with everything that no key may come from set to NaN."""

    def __init__(self, dt, D, Hq, Hkv, blk, in_cache, causal, ps, lens, P=0, seed=0, max_ctx=None):
        g = gen(seed + 17 * len(lens) + blk)
        self.__dict__.update(dt=dt, D=D, Hq=Hq, Hkv=Hkv, blk=blk, in_cache=in_cache,
                             causal=causal, ps=ps, lens=lens, P=P)
        B = len(lens)
        width = max(1, -(-max(lens + [P]) // ps)) + 1
        pages = B * width + 2
        self.table = deal(g, pages, B, width)
        self.k, self.v = pool(g, pages, Hkv, ps, D, dt), pool(g, pages, Hkv, ps, D, dt)
        used = torch.zeros(pages, ps, dtype=torch.bool)
        for b in range(B):
            for key in range(lens[b]):
                used[self.page(b, key)] = True
        if P:
            for key in range(P):
                used[int(self.table[0, key // ps]), key % ps] = True
        for t in (self.k, self.v):
            t.masked_fill_(~used[:, None, :, None], math.nan)
        # entries that no key needs lie outside the pool
        for b in range(B):
            for j in range(width):
                lo, hi = j * ps, (j + 1) * ps
                if lo >= max(lens[b], P if b == 0 else 0) or (self.shares(b) and b and hi <= P):
                    self.table[b, j] = -5 if j % 2 else pages + 100
        self.q = randn(g, B, blk, Hq, D, dt=dt)
        self.kb = self.vb = None
        if not in_cache:
            self.kb, self.vb = randn(g, B, blk, Hkv, D, dt=dt), randn(g, B, blk, Hkv, D, dt=dt)
        self.max_ctx = max(lens + [P]) if max_ctx is None else max_ctx

    def shares(self, b):
        return self.P > 0 and self.lens[b] - (self.blk if self.in_cache else 0) >= self.P

    def page(self, b, key):
        row = 0 if self.shares(b) and key < self.P else b
        return int(self.table[row, key // self.ps]), key % self.ps

    def run(self, **kw):
        d = lambda t: None if t is None else t.cuda()
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        out = torch.full(self.q.shape, 3.0, dtype=self.q.dtype, device="cuda")
        ba.paged_block_attn(d(self.q), d(self.kb), d(self.vb), d(self.k), d(self.v),
                            d(self.table), torch.tensor(self.lens, dtype=torch.int32).cuda(),
                            ba.CAUSAL_VERIFY if self.causal else ba.BIDIR_BLOCK, out=out,
                            shared_prefix=self.P, max_ctx=self.max_ctx, err=err, **kw)
        return out.cpu(), err.item()

    def reference(self, b):
        """float64 output of sequence b, and its tolerance."""
        n, blk, G = self.lens[b], self.blk, self.Hq // self.Hkv
        at = [self.page(b, key) for key in range(n)]
        pg, sl = [a for a, _ in at], [s for _, s in at]
        k, v = self.k[pg, :, sl].double(), self.v[pg, :, sl].double()  # [n, Hkv, D]
        if n == 0:
            k, v = k.reshape(0, self.Hkv, self.D), v.reshape(0, self.Hkv, self.D)
        if not self.in_cache:
            k, v = torch.cat([k, self.kb[b].double()]), torch.cat([v, self.vb[b].double()])
        total = k.shape[0]
        out, tol = (torch.zeros(blk, self.Hq, self.D, dtype=torch.float64) for _ in range(2))
        scale, u24 = self.D ** -0.5, 2.0 ** -24
        for h in range(self.Hq):
            kh, vh, qh = k[:, h // G], v[:, h // G], self.q[b, :, h].double()
            for i in range(blk):
                lim = total - blk + i + 1 if self.causal else total
                if lim <= 0:
                    continue
                z = scale * (kh[:lim] @ qh[i])
                p = torch.softmax(z, 0)
                out[i, h] = p @ vh[:lim]
                a = p @ vh[:lim].abs()
                ds = (self.D + 2) * u24 * scale * (kh[:lim].abs() @ qh[i].abs()).max()
                tol[i, h] = a * (2 * ds + (lim + 64) * u24)
                if self.dt == "bf16":
                    tol[i, h] += a * HALF_STEP["bf16"] + out[i, h].abs() * HALF_STEP["bf16"]
        return out, tol

    def check(self, **kw):
        got, err = self.run(**kw)
        assert err == 0
        for b in range(len(self.lens)):
            ref, tol = self.reference(b)
            e = (got[b].double() - ref).abs()
            assert (e <= tol * 1.01 + 1e-30).all(), (b, float((e / (tol + 1e-30)).max()))
        return got


CASES = [
    # D, Hq, Hkv, blk, in_cache, causal, ps, lens, P
    (128, 4, 1, 32, False, False, 64, [300], 0),
    (128, 4, 1, 32, False, True, 16, [0, 1, 127, 128, 129, 700], 0),
    (64, 8, 4, 16, False, True, 32, [64, 0, 513], 0),
    (64, 2, 2, 5, False, False, 128, [1, 255, 256, 257], 0),
    (128, 8, 2, 1, True, True, 16, [1, 2, 0, 130, 1000], 0),
    (128, 8, 2, 7, True, True, 32, [7, 3, 0, 1, 135, 128], 0),
    (64, 4, 4, 32, True, True, 64, [31, 32, 33, 160, 5], 0),
    (128, 4, 4, 9, True, False, 256, [0, 4, 600], 0),
    (128, 16, 2, 16, False, True, 16, [333, 90], 0),
    (128, 4, 1, 32, False, True, 64, [400, 256, 300, 255, 0], 256),
    (128, 4, 2, 1, True, True, 16, [301 + i for i in range(70)] + [0, 5], 300),
    (64, 4, 1, 8, False, False, 32, [200, 200, 777, 40], 200),
    (128, 6, 2, 3, True, True, 128, [103, 102, 104, 500, 1], 100),
    (64, 2, 1, 1, False, True, 256, [1000, 1001], 1000),
]


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_attention(dt, case):
    D, Hq, Hkv, blk, in_cache, causal, ps, lens, P = CASES[case]
    Attn(dt, D, Hq, Hkv, blk, in_cache, causal, ps, lens, P, seed=case).check()


@pytest.mark.parametrize("P", [0, 40])
def test_attention_more_sequences_than_a_cta_has_threads(P):
    """The schedule of the first 384 sequences and of the others, summed in two steps."""
    lens = [(37 * i) % 150 for i in range(801)]
    Attn("bf16", 64, 2, 1, 1, True, True, 32, lens, P, seed=31).check()


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_attention_long_and_loose_bound(dt):
    """Several splits of one sequence, with a length bound far above the lengths."""
    a = Attn(dt, 128, 8, 2, 4, False, True, 64, [5000, 17], 0, seed=9)
    got = a.check()
    a.table = torch.cat([a.table, torch.full((2, 800), -1, dtype=torch.int32)], 1)
    a.max_ctx = 50000
    a.check()
    assert got.isfinite().all()


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("in_cache", [False, True])
@pytest.mark.parametrize("bad", [math.nan, math.inf])
def test_attention_non_finite_rows_reach_only_the_rows_that_see_them(dt, in_cache, bad):
    a = Attn(dt, 64, 4, 2, 8, in_cache, True, 16, [40, 130], 0, seed=4)
    clean, _ = a.run()
    # the block's row 5 of sequence 1, kv-head 0: V element 3
    if in_cache:
        page, slot = a.page(1, 130 - 8 + 5)
        a.v[page, 0, slot, 3] = bad
    else:
        a.vb[1, 5, 0, 3] = bad
    got, err = a.run()
    assert err == 0
    sees = torch.zeros(got.shape, dtype=torch.bool)
    sees[1, 5:, 0:2, 3] = True  # the two query heads of kv-head 0
    assert torch.equal(got[~sees], clean[~sees])
    if math.isnan(bad):
        assert got[sees].isnan().all()
    else:
        assert (got[sees] == math.inf).all()
    # the same for K: whole rows, from the first that sees it
    if in_cache:
        a.v[page, 0, slot, 3] = 0.0
        a.k[page, 0, slot, 3] = bad
    else:
        a.vb[1, 5, 0, 3] = 0.0
        a.kb[1, 5, 0, 3] = math.nan
    got, _ = a.run()
    assert got[0].isfinite().all() and got[1, :5].isfinite().all()
    assert got[1, :, 2:].isfinite().all()
    if not in_cache or math.isnan(bad):
        assert got[1, 5:, :2].isnan().all()


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_attention_scores_all_minus_infinity_is_nan(dt):
    a = Attn(dt, 64, 2, 1, 2, False, False, 16, [5], 0)
    a.q.fill_(1.0)
    a.k[:, :, :, 0] = -math.inf
    a.kb[..., 0] = -math.inf
    got, _ = a.run()
    assert got.isnan().all()


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_attention_refused_sequences_keep_their_rows(dt):
    a = Attn(dt, 64, 2, 1, 4, False, True, 16, [100, 50, 300], 0, seed=2)
    clean, _ = a.run()
    a.table[1, 2] = a.k.shape[0]
    got, err = a.run()
    assert err == -1 and (got[1] == 3.0).all()
    assert torch.equal(got[0], clean[0]) and torch.equal(got[2], clean[2])
    a.table[1, 2] = -1
    a.lens[2] = a.max_ctx + 1  # past the bound
    got, err = a.run()
    assert err != 0 and (got[1:] == 3.0).all() and torch.equal(got[0], clean[0])
    a.lens[2] = -1
    got, err = a.run()
    assert (got[1:] == 3.0).all() and torch.equal(got[0], clean[0])


def test_attention_refused_prefix_page_keeps_only_its_sequences():
    a = Attn("bf16", 64, 2, 1, 4, False, True, 16, [100, 150, 20], 64, seed=2)
    clean, _ = a.run()
    a.table[0, 1] = -1
    got, err = a.run()
    assert err == -1 and (got[:2] == 3.0).all()
    assert torch.equal(got[2], clean[2])  # shorter than the prefix: its own pages


def test_attention_f32_rows_are_invariant():
    """FP32: a causal row of a block has the bits of a one-token call at its position."""
    g = gen(8)
    Hq, Hkv, D, ps, n, blk = 4, 2, 64, 16, 70, 8
    table = deal(g, 12, 1, 10).cuda()
    kp, vp = pool(g, 12, Hkv, ps, D, "f32").cuda(), pool(g, 12, Hkv, ps, D, "f32").cuda()
    q, kb, vb = (randn(g, 1, blk, h, D, dt="f32").cuda() for h in (Hq, Hkv, Hkv))
    lens = torch.tensor([n], dtype=torch.int32).cuda()
    block = ba.paged_block_attn(q, kb, vb, kp, vp, table, lens, ba.CAUSAL_VERIFY)
    for i in range(blk):
        one = ba.paged_block_attn(q[:, i:i + 1].contiguous(), kb[:, i:i + 1].contiguous(),
                                  vb[:, i:i + 1].contiguous(), kp, vp, table, lens,
                                  ba.CAUSAL_VERIFY)
        assert torch.equal(one[0, 0], block[0, i])
        ba.paged_append(kb[:, i:i + 1], vb[:, i:i + 1], kp, vp, table, lens, advance=True)
    # and with the rows in the pages
    again = ba.paged_block_attn(q, None, None, kp, vp, table, lens, ba.CAUSAL_VERIFY)
    assert torch.equal(again, block)


# ------------------------------------------------- streams, graphs, together

def test_attention_captured_with_changing_lengths_and_two_streams():
    a = Attn("bf16", 128, 8, 2, 8, False, True, 32, [300, 64, 1], 0, seed=6)
    d = [None if t is None else t.cuda() for t in (a.q, a.kb, a.vb, a.k, a.v, a.table)]
    lens = torch.tensor(a.lens, dtype=torch.int32).cuda()
    out = torch.empty_like(d[0])
    call = lambda **kw: ba.paged_block_attn(*d, lens, ba.CAUSAL_VERIFY, max_ctx=300, **kw)
    eager = call()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(out=out)
    big = Attn("bf16", 128, 8, 2, 8, False, True, 32, [900] * 9, 400, seed=7)
    big.check()  # outgrows the default workspace
    graph.replay()
    assert torch.equal(out, eager)
    lens.copy_(torch.tensor([17, 64, 0], dtype=torch.int32))
    graph.replay()
    assert torch.equal(out, call())
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [call(stream=s) for s in streams for _ in range(3)]
    torch.cuda.synchronize()
    assert all(torch.equal(o, out) for o in got)


def test_graphs_replayed_at_once_share_no_scratch():
    """Captured without a workspace of their own: two graphs of append (with its
    ticket) and split attention, replayed on two streams together."""
    sets = []
    for seed in (21, 22):
        a = Attn("bf16", 128, 8, 2, 8, False, True, 32, [2000, 1500, 700], 0, seed=seed)
        d = [None if t is None else t.cuda() for t in (a.q, a.kb, a.vb, a.k, a.v, a.table)]
        lens = torch.tensor(a.lens, dtype=torch.int32).cuda()
        count, none = lens.clone(), torch.zeros_like(lens)
        out = torch.empty_like(d[0])
        ref = ba.paged_block_attn(*d, lens, ba.CAUSAL_VERIFY, max_ctx=a.max_ctx)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            for _ in range(4):
                # no rows are taken, so the pools and the lengths stay
                ba.paged_append(d[1], d[2], d[3], d[4], d[5], count, n_rows=none, advance=True)
                ba.paged_block_attn(*d, lens, ba.CAUSAL_VERIFY, max_ctx=a.max_ctx, out=out)
        sets.append((graph, out, ref, d, lens, count, none, torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(25):
        for s in sets:
            s[1].zero_()
        torch.cuda.synchronize()
        for s in sets:
            with torch.cuda.stream(s[-1]):
                s[0].replay()
        torch.cuda.synchronize()
        for _, out, ref, _, lens, count, _, _ in sets:
            assert torch.equal(out, ref) and torch.equal(count, lens)


def test_append_then_attention_matches_the_dense_cache():
    """A prefill in two ragged pieces, a decoding step and a round's verify view
    over pages, against the same keys in a dense cache."""
    g = gen(12)
    B, Hq, Hkv, D, ps, cap = 3, 8, 2, 128, 16, 160
    freq, m = ba.rope_freqs(D, 1e6)
    table = deal(g, 40, B, cap // ps).cuda()
    kp = torch.zeros(40, Hkv, ps, D, dtype=torch.bfloat16, device="cuda")
    vp = torch.zeros_like(kp)
    lens = torch.zeros(B, dtype=torch.int32, device="cuda")
    kc = torch.zeros(B, Hkv, cap, D, dtype=torch.bfloat16, device="cuda")
    vc = torch.zeros_like(kc)
    for counts in ([50, 1, 64], [3, 70, 0], [1, 1, 1]):
        rows = sum(counts)
        qkv = randn(g, rows, Hq + 2 * Hkv, D, dt="bf16").cuda()
        starts = torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32).cuda()
        q, k, v = qkv.split([Hq, Hkv, Hkv], 1)
        pos = torch.cat([int(n) + torch.arange(c) for n, c in zip(lens.tolist(), counts)])
        k_rot = ba.rope(k, pos.to(torch.int32).cuda(), freq, mscale=m)
        at = 0
        for b, c in enumerate(counts):
            n = int(lens[b])
            kc[b, :, n:n + c] = k_rot[at:at + c].transpose(0, 1)
            vc[b, :, n:n + c] = v[at:at + c].transpose(0, 1)
            at += c
        q_rot = ba.paged_append(k, v, kp, vp, table, lens, row_starts=starts, inv_freq=freq,
                                mscale=m, q=q, advance=True)
    assert lens.tolist() == [54, 72, 65]
    # decoding step: the last row of each sequence is in the cache
    one = ba.paged_block_attn(q_rot.view(B, 1, Hq, D), None, None, kp, vp, table, lens,
                              ba.CAUSAL_VERIFY)
    last = [(kc[b:b + 1, :, int(lens[b]) - 1], vc[b:b + 1, :, int(lens[b]) - 1]) for b in range(B)]
    dense = ba.block_attn(q_rot.view(B, 1, Hq, D), torch.stack([k for k, _ in last]),
                          torch.stack([v for _, v in last]), kc, vc, lens - 1, ba.CAUSAL_VERIFY)
    ref = dense.float()
    # two bf16 results of the same formula: each within 2^-8 of sum p|v| and of itself
    tol = 4 * 2.0 ** -8 * vc.float().abs().max()
    assert (one.float() - ref).abs().max() <= tol
    blk = 16
    qb, kb, vb = (randn(g, B, blk, h, D, dt="bf16").cuda() for h in (Hq, Hkv, Hkv))
    got = ba.paged_block_attn(qb, kb, vb, kp, vp, table, lens, ba.CAUSAL_VERIFY)
    ref = ba.block_attn(qb, kb, vb, kc, vc, lens, ba.CAUSAL_VERIFY)
    assert (got.float() - ref.float()).abs().max() <= tol
