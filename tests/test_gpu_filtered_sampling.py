"""Filtered sampling on the GPU against a plain 64-bit evaluation.

Indices have to be equal: weights are summed exactly on the device (fixed
point), and the inputs are random, so that no draw lies within the rounding of
a border.  A log-probability is a 64-bit value rounded to float (2^-24
relative) plus what the fixed point loses, below vocab 2^-44 / mass."""
import math

import numpy as np
import pytest
import torch

import block_attention_b200 as ba

pytestmark = pytest.mark.gpu


def plain(x, u, T=1.0, k=0, p=1.0, mp=0.0):
    """(index, logprob, kept set) of one row, float64."""
    x = np.where(np.isnan(x), -np.inf, x.astype(np.float64))
    T, u, p, mp = (float(np.float32(t)) for t in (T, u, p, mp))
    M = x.max()
    if M == -np.inf:
        return 0, math.nan, np.zeros(0, np.int64)
    if T == 0:
        return int(np.argmax(x)), 0.0, np.array([int(np.argmax(x))])
    with np.errstate(invalid="ignore"):
        w = np.exp(np.where(x == M, 0.0, (x - M) / T))
    order = np.lexsort((np.arange(x.size), -x))
    order = order[x[order] > -np.inf]
    if k > 0:
        order = order[:k]
    if p < 1:
        c = np.cumsum(w[order])
        order = order[:max(1, int((c < p * c[-1]).sum()) + 1)]
    if mp > 0:
        order = order[w[order] >= min(mp, 1.0)]
    kept = np.sort(order)
    c = np.cumsum(w[kept])
    i = int((c <= min(max(u, 0.0), 1.0) * c[-1]).sum())
    if i >= kept.size:
        i = int(np.nonzero(w[kept] > 0)[0][-1])
    j = int(kept[i])
    return j, (0.0 if x[j] == M else (x[j] - M) / T) - math.log(c[-1]), kept


def compare(x, u, **kw):
    """x float32 [rows, vocab] CPU tensor or bf16; parameters as lists or None."""
    rows = x.shape[0]
    dev = {n: torch.tensor(v, dtype=torch.int32 if n == "top_k" else torch.float32).cuda()
           for n, v in kw.items() if v is not None}
    lp = torch.empty(rows, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = ba.vocab_sample_filtered(x.cuda(), torch.tensor(u, dtype=torch.float32).cuda(),
                                   logprob=lp, err=err, **dev).cpu().numpy()
    assert err.item() == 0
    xf, lp = x.float().numpy(), lp.cpu().numpy()
    pick = lambda n, r, d: d if kw.get(n) is None else kw[n][r]
    for r in range(rows):
        j, l, _ = plain(xf[r], u[r], pick("temperature", r, 1.0), pick("top_k", r, 0),
                        pick("top_p", r, 1.0), pick("min_p", r, 0.0))
        assert got[r] == j, (r, got[r], j)
        if math.isnan(l):
            assert math.isnan(lp[r])
        else:
            assert abs(lp[r] - l) <= 2.0 ** -23 * abs(l) + 1e-7, (r, lp[r], l)


def uniforms(g, rows):
    return ((g.integers(0, 1 << 23, rows) + 0.5) * 2.0 ** -23).tolist()


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("vocab", [1, 2, 7, 100, 2048, 2049, 5000, 8192, 151936])
def test_every_filter(dt, vocab):
    g = np.random.default_rng(vocab)
    rows = 24
    x = torch.from_numpy((2.5 * g.standard_normal((rows, vocab))).astype(np.float32)).to(dt)
    u = uniforms(g, rows)
    T = (0.3 + 1.2 * g.random(rows)).tolist()
    k = g.integers(1, 300, rows).tolist()
    p = (0.05 + 0.94 * g.random(rows)).tolist()
    mp = (0.2 * g.random(rows)).tolist()
    compare(x, u)
    compare(x, u, temperature=T)
    compare(x, u, top_k=k)
    compare(x, u, top_p=p, temperature=T)
    compare(x, u, min_p=mp)
    compare(x, u, temperature=T, top_k=k, top_p=p, min_p=mp)
    big = [min(5 * i * i + 1, vocab + 3) for i in range(rows)]  # past the list, past the row
    compare(x, u, top_k=big, top_p=p)
    compare(x, u, top_k=[vocab // 2 + 1] * rows, min_p=mp)


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
def test_ties(dt):
    """Rows of few distinct values: cuts fall inside runs of thousands of equal logits."""
    g = np.random.default_rng(1)
    vocab, rows = 20000, 16
    x = torch.from_numpy(g.integers(0, 3, (rows, vocab)).astype(np.float32)).to(dt)
    x[0] = 1.5
    x[1, ::2], x[1, 1::2] = 0.0, -0.0  # equal as numbers
    u = uniforms(g, rows)
    for kw in (dict(top_k=[3000] * rows), dict(top_p=[0.5] * rows), dict(top_k=[7] * rows),
               dict(top_k=[9001] * rows, top_p=[0.77] * rows),
               dict(top_k=[12000] * rows, top_p=[0.3] * rows, min_p=[0.2] * rows),
               dict(min_p=[1.0] * rows), dict(top_p=[1e-6] * rows), dict(top_k=[1] * rows)):
        compare(x, u, **kw)


def test_extreme_rows():
    vocab = 6000
    g = np.random.default_rng(2)
    base = g.standard_normal(vocab).astype(np.float32)
    rows = []
    lowest = np.finfo(np.float32).min
    a = base.copy(); a[10:] = lowest; rows.append(a)          # masks of the lowest value
    a = base.copy(); a[:5990] = -np.inf; rows.append(a)       # and of -inf
    a = base.copy(); a[::3] = np.nan; rows.append(a)
    a = np.full(vocab, np.nan, np.float32); rows.append(a)
    a = np.full(vocab, -np.inf, np.float32); rows.append(a)
    a = base.copy(); a[[5, 4000]] = np.inf; rows.append(a)
    a = np.full(vocab, lowest, np.float32); rows.append(a)
    a = base * 1e30; rows.append(a.astype(np.float32))
    a = base * 1e-30; rows.append(a.astype(np.float32))
    a = np.full(vocab, -np.inf, np.float32); a[777] = -3; rows.append(a)
    x = torch.from_numpy(np.stack(rows))
    n = len(rows)
    for u in (0.25, 0.0, 1.0, 0.9999999):
        compare(x, [u] * n)
        compare(x, [u] * n, top_p=[0.6] * n, temperature=[0.7] * n)
        compare(x, [u] * n, top_k=[40] * n, min_p=[0.01] * n)
        compare(x, [u] * n, temperature=[0.0] * n)
        compare(x, [u] * n, temperature=[1e-6] * n, top_p=[0.9] * n)
        compare(x, [u] * n, top_k=[3000] * n, top_p=[0.9] * n)


def test_strided_unaligned_rows_and_scalars():
    g = np.random.default_rng(3)
    full = torch.from_numpy(g.standard_normal((9, 5003)).astype(np.float32)).cuda()
    x = full[:, 1:4998]
    u = torch.tensor(uniforms(g, 9), dtype=torch.float32).cuda()
    got = ba.vocab_sample_filtered(x, u, temperature=0.8, top_k=50, top_p=0.9, min_p=0.02)
    for r in range(9):
        assert got[r].item() == plain(x[r].cpu().numpy(), u[r].item(), 0.8, 50, 0.9, 0.02)[0]


def test_vocabulary_read_from_memory_more_than_once():
    """A row too long for the cluster's shared memory."""
    g = np.random.default_rng(4)
    vocab = 400003
    x = torch.from_numpy(g.standard_normal((2, vocab)).astype(np.float32))
    compare(x, uniforms(g, 2))
    compare(x, uniforms(g, 2), top_p=[0.9, 0.001])
    compare(x, uniforms(g, 2), top_k=[5000, 50], top_p=[0.9, 0.5])


def test_bad_temperature_leaves_its_row():
    x = torch.randn(4, 3000, device="cuda")
    u = torch.full((4,), 0.5, device="cuda")
    idx = torch.full((4,), -9, dtype=torch.int32, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    T = torch.tensor([1.0, -1.0, math.nan, math.inf], device="cuda")
    ba.vocab_sample_filtered(x, u, temperature=T, idx=idx, err=err)
    assert err.item() == -1 and idx[1:].tolist() == [-9] * 3 and idx[0].item() >= 0


def test_draws_follow_the_kept_distribution():
    """Uniforms on a fine grid give every kept token its share, exactly."""
    g = np.random.default_rng(5)
    vocab, n = 500, 4096
    row = g.standard_normal(vocab).astype(np.float32) * 2
    u = (np.arange(n) + 0.5) / n
    x = torch.from_numpy(row).expand(n, vocab).contiguous().cuda()
    got = ba.vocab_sample_filtered(x, torch.from_numpy(u.astype(np.float32)).cuda(), top_k=20,
                                   top_p=0.9).cpu().numpy()
    _, _, kept = plain(row, 0.5, 1.0, 20, 0.9)
    w = np.exp(row[kept].astype(np.float64))
    share = w / w.sum()
    counts = np.array([(got == j).sum() for j in kept])
    assert counts.sum() == n and (np.abs(counts - n * share) <= 1.0 + 1e-6).all()
    assert (np.diff(got) >= 0).all()  # the draw grows with u, in vocabulary order


def test_captured_graph_follows_new_uniforms():
    x = torch.randn(3, 9000, device="cuda")
    u = torch.rand(3, device="cuda")
    p = torch.full((3,), 0.95, device="cuda")
    idx = torch.empty(3, dtype=torch.int32, device="cuda")
    ba.vocab_sample_filtered(x, u, top_p=p, idx=idx)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ba.vocab_sample_filtered(x, u, top_p=p, idx=idx)
    for _ in range(3):
        u.copy_(torch.rand(3, device="cuda"))
        x.copy_(torch.randn(3, 9000, device="cuda"))
        graph.replay()
        assert torch.equal(idx, ba.vocab_sample_filtered(x, u, top_p=p))
