"""Workloads of the paged-cache and filtered-sampling operators.

Each case is one call a serving loop makes: rotating queries and keys
(``rope``), writing keys and values into a paged cache (``append``), the
decoding block's attention over the pages (``attn``), the same for a batch
that shares its first keys (``prefix``), and drawing tokens from filtered
logits (``sample``).

``run`` computes a case with elementary torch operations, or, with ``own``
set, with the framework's kernels; ``exact`` evaluates the definition in 64
bits, written separately."""
import math
import random

import torch

own = False

DEV = "cuda"
_DT = {"bf16": torch.bfloat16, "f32": torch.float32}
_ES = {"bf16": 2, "f32": 4}


# ------------------------------------------------------------------ cases
#
# A ragged batch is given by its size, the range of its lengths and a number
# that picks them ("mix").

def listed():
    return [
        # one decoding block's queries, one layer of the 8B shape: the smallest call
        {"name": "rope_block", "op": "rope", "dtype": "bf16", "rows": 32, "heads": 32, "D": 128,
         "rot": 128, "layout": "half", "scaling": "none", "pos0": 8192, "inverse": False},
        # queries of a long prefill, part of each head, interleaved pairs, far positions with
        # interpolated frequencies
        {"name": "rope_prefill", "op": "rope", "dtype": "f32", "rows": 8190, "heads": 32, "D": 128,
         "rot": 64, "layout": "interleaved", "scaling": "yarn", "pos0": 120000, "inverse": False},
        # one token for each of 64 sequences: q, k and v of a fused projection
        {"name": "append_decode", "op": "append", "dtype": "bf16", "B": 64, "lo": 0, "hi": 4096,
         "new_lo": 1, "new_hi": 1, "mix": 1, "Hq": 32, "Hkv": 8, "D": 128, "ps": 16, "rot": 128,
         "layout": "half"},
        # ragged prefill of eight prompts behind cached prefixes that end inside a page
        {"name": "append_prefill", "op": "append", "dtype": "bf16", "B": 8, "lo": 0, "hi": 1000,
         "new_lo": 1, "new_hi": 4097, "mix": 2, "Hq": 32, "Hkv": 8, "D": 128, "ps": 64, "rot": 128,
         "layout": "half"},
        # one sequence, diffusion view, 8B layer at 8192 keys: latency counts
        {"name": "attn_block", "op": "attn", "dtype": "bf16", "B": 1, "lo": 8192, "hi": 8192,
         "mix": 0, "blk": 32, "in_cache": False, "mode": "bidir", "Hq": 32, "Hkv": 8, "D": 128,
         "ps": 64, "prefix": 0},
        # verify view of a ragged batch, 1k to 32k keys, small pages
        {"name": "attn_ragged", "op": "attn", "dtype": "bf16", "B": 16, "lo": 1024, "hi": 32767,
         "mix": 3, "blk": 32, "in_cache": False, "mode": "causal", "Hq": 32, "Hkv": 8, "D": 128,
         "ps": 16, "prefix": 0},
        # plain decoding, one token a sequence, already appended
        {"name": "attn_decode", "op": "attn", "dtype": "bf16", "B": 64, "lo": 1, "hi": 8192,
         "mix": 4, "blk": 1, "in_cache": True, "mode": "causal", "Hq": 32, "Hkv": 8, "D": 128,
         "ps": 32, "prefix": 0},
        # the FP32 path at the 1.7B layer
        {"name": "attn_f32", "op": "attn", "dtype": "f32", "B": 2, "lo": 700, "hi": 2048, "mix": 5,
         "blk": 32, "in_cache": False, "mode": "bidir", "Hq": 16, "Hkv": 8, "D": 128, "ps": 16,
         "prefix": 0},
        # 16 requests behind one 8192-key prompt, verify view
        {"name": "prefix_block", "op": "attn", "dtype": "bf16", "B": 16, "lo": 32, "hi": 1024,
         "mix": 6, "blk": 32, "in_cache": False, "mode": "causal", "Hq": 32, "Hkv": 8, "D": 128,
         "ps": 64, "prefix": 8192},
        # 128 requests behind one 16k-key prompt, one token each
        {"name": "prefix_decode", "op": "attn", "dtype": "bf16", "B": 128, "lo": 1, "hi": 512,
         "mix": 7, "blk": 1, "in_cache": True, "mode": "causal", "Hq": 32, "Hkv": 8, "D": 128,
         "ps": 64, "prefix": 16384},
        # one row of the 8B vocabulary
        {"name": "sample_row", "op": "sample", "dtype": "bf16", "rows": 1, "vocab": 151936,
         "filters": "kp"},
        # a batch whose requests ask for different filters
        {"name": "sample_batch", "op": "sample", "dtype": "f32", "rows": 256, "vocab": 151936,
         "filters": "mixed"},
    ]


def _lens(c):
    """Keys of each sequence before the call (common keys included)."""
    r = random.Random(c["mix"])
    return [c.get("prefix", 0) + r.randint(c["lo"], c["hi"]) for _ in range(c["B"])]


def _counts(c):
    """Rows that each sequence appends."""
    r = random.Random(1000 + c["mix"])
    return [r.randint(c["new_lo"], c["new_hi"]) for _ in range(c["B"])]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "append", "attn", "attn", "prefix", "sample"])
    dt = rng.choice(["bf16", "bf16", "f32"])
    D = rng.choice([64, 128, 128])
    mix = rng.randrange(1 << 20)
    if op == "rope":
        heads = rng.randint(1, 40)
        rot = rng.choice([D, D // 2, 2 * rng.randint(2, D // 2)])
        return {"op": "rope", "dtype": dt, "rows": _log(rng, 1, 8190 * 16 // heads),
                "heads": heads, "D": D, "rot": rot, "layout": rng.choice(["half", "interleaved"]),
                "scaling": rng.choice(["none", "linear", "ntk", "bands", "yarn"]),
                "pos0": _log(rng, 1, 1000000), "inverse": rng.random() < 0.3}
    Hkv = rng.choice([1, 2, 4, 8])
    G = rng.choice([1, 2, 4, 4, 8])
    ps = rng.choice([16, 32, 64, 128, 256])
    if op == "append":
        B = _log(rng, 1, 64)
        return {"op": "append", "dtype": dt, "B": B, "lo": 0, "hi": rng.randint(0, 1500),
                "new_lo": rng.choice([0, 1]), "new_hi": _log(rng, 1, 8192 // B), "mix": mix,
                "Hq": Hkv * min(G, 4), "Hkv": Hkv, "D": D, "ps": ps,
                "rot": rng.choice([D, D // 2]), "layout": rng.choice(["half", "interleaved"])}
    if op == "sample":
        return {"op": "sample", "dtype": dt, "rows": _log(rng, 1, 256),
                "vocab": _log(rng, 8, 151936),
                "filters": rng.choice(["mixed", "kp", "k", "p", "m", "none"])}
    blk = max(1, min(rng.choice([1, 2, 5, 8, 16, 31, 32]), 128 // G))
    in_cache = rng.random() < 0.5
    prefix = 0
    if op == "prefix":
        dt = "bf16"
        B = _log(rng, 2, 128 if blk == 1 else 16)
        prefix = _log(rng, 100, 16384 if blk == 1 else 8192)
        hi = 512
    elif dt == "f32":
        B, hi = _log(rng, 1, 2), 2048
    else:
        B, hi = _log(rng, 1, 64), 8192
    lo = blk if in_cache else 0
    return {"op": "attn", "dtype": dt, "B": B, "lo": lo, "hi": max(lo, _log(rng, 1, hi)),
            "mix": mix, "blk": blk, "in_cache": in_cache, "mode": rng.choice(["bidir", "causal"]),
            "Hq": Hkv * G, "Hkv": Hkv, "D": D, "ps": ps, "prefix": prefix}


# ----------------------------------------------------------------- inputs

def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _randn(g, *shape, dt=torch.float32):
    out = torch.empty(*shape, dtype=dt, device=DEV)
    flat = out.view(-1)
    for i in range(0, flat.numel(), 1 << 26):  # pools of a few GB: no fp32 copy of the whole
        n = min(1 << 26, flat.numel() - i)
        flat[i:i + n] = torch.randn(n, generator=g, device=DEV)
    return out


def _freqs(rot, scaling, theta=1e6):
    """Angles per position, float64 [rot / 2], and the factor on the rotated values."""
    i = torch.arange(rot // 2, dtype=torch.float64)
    f = theta ** (-2.0 * i / rot)
    m = 1.0
    s, base = 8.0, 16384.0  # stretch of the context, length it was trained at
    if scaling == "linear":
        f = f / s
    elif scaling == "ntk":
        f = (theta * s ** (rot / (rot - 2))) ** (-2.0 * i / rot)
    elif scaling == "bands":
        turns = base * f / (2 * math.pi)  # turns over the trained length
        t = ((turns - 1.0) / (4.0 - 1.0)).clamp(0, 1)
        f = (1 - t) * f / s + t * f
    elif scaling == "yarn":
        dim = lambda turns: rot * math.log(base / (2 * math.pi * turns)) / (2 * math.log(theta))
        lo, hi = max(math.floor(dim(32.0)), 0), min(math.ceil(dim(1.0)), rot - 1)
        t = ((i - lo) / max(hi - lo, 1e-3)).clamp(0, 1)
        f = (1 - t) * f + t * f / s
        m = 0.1 * math.log(s) + 1.0
    return f.to(DEV), m


def _pages(g, lens, ps):
    """A pool just large enough, with its pages dealt out at random."""
    need = [max(1, -(-n // ps)) for n in lens]
    pages = sum(need)
    perm = torch.randperm(pages, generator=g, device=DEV).to(torch.int32)
    table = torch.zeros(len(lens), max(need), dtype=torch.int32, device=DEV)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = perm[at:at + n]
        at += n
    return table, pages


def prepare(case, seed):
    g = _gen(seed)
    c = dict(case)
    s = {"case": c}
    dt = _DT[c["dtype"]]
    if c["op"] == "rope":
        s["x"] = _randn(g, c["rows"], c["heads"], c["D"], dt=dt)
        s["pos"] = (c["pos0"] + torch.arange(c["rows"], device=DEV)).to(torch.int32)
        s["freq"], s["m"] = _freqs(c["rot"], c["scaling"])
        s["out"] = torch.empty_like(s["x"])
    elif c["op"] == "append":
        lens, counts, D = _lens(c), _counts(c), c["D"]
        rows, H = sum(counts), c["Hq"] + 2 * c["Hkv"]
        qkv = _randn(g, rows, H, D, dt=dt)  # a fused projection's output: strided views of it
        s["q"], s["k"], s["v"] = qkv.split([c["Hq"], c["Hkv"], c["Hkv"]], dim=1)
        s["table"], pages = _pages(g, [a + b for a, b in zip(lens, counts)], c["ps"])
        s["k_pages"] = _randn(g, pages, c["Hkv"], c["ps"], D, dt=dt)
        s["v_pages"] = _randn(g, pages, c["Hkv"], c["ps"], D, dt=dt)
        s["ctx"] = torch.tensor(lens, dtype=torch.int32, device=DEV)
        s["starts"] = torch.tensor([sum(counts[:b]) for b in range(len(counts) + 1)],
                                   dtype=torch.int32, device=DEV)
        s["freq"], s["m"] = _freqs(c["rot"], "none")
        s["q_out"] = torch.empty(rows, c["Hq"], D, dtype=dt, device=DEV)
    elif c["op"] == "attn":
        lens, blk, D, ps, P = _lens(c), c["blk"], c["D"], c["ps"], c["prefix"]
        B = len(lens)
        s["lens"] = lens
        if P:
            # pages of the common keys first (the page that the prefix ends in is shared by
            # row 0 only: the others read its first keys through row 0's entry)
            shared = P // ps
            own_lens = [n - shared * ps for n in lens]
            tail, pages = _pages(g, own_lens, ps)
            head = torch.arange(pages, pages + shared, device=DEV, dtype=torch.int32)
            head = head[torch.randperm(shared, generator=g, device=DEV)]
            s["table"] = torch.cat([head.expand(B, shared), tail], 1).contiguous()
            pages += shared
        else:
            s["table"], pages = _pages(g, lens, ps)
        s["k_pages"] = _randn(g, pages, c["Hkv"], ps, D, dt=dt)
        s["v_pages"] = _randn(g, pages, c["Hkv"], ps, D, dt=dt)
        s["ctx"] = torch.tensor(lens, dtype=torch.int32, device=DEV)
        s["q"] = _randn(g, B, blk, c["Hq"], D, dt=dt)
        s["kb"] = s["vb"] = None
        if not c["in_cache"]:
            s["kb"] = _randn(g, B, blk, c["Hkv"], D, dt=dt)
            s["vb"] = _randn(g, B, blk, c["Hkv"], D, dt=dt)
        s["out"] = torch.empty_like(s["q"])
        if own:
            import block_attention_b200 as ba
            s["ws"] = ba.Workspace(DEV)
    else:
        rows, V = c["rows"], c["vocab"]
        x = _randn(g, rows, V)
        x.mul_(2.5)
        # a few likely tokens stand out, as in a language model's rows
        at = torch.randint(V, (rows, 8), generator=g, device=DEV)
        x.scatter_add_(1, at, 4 + 8 * torch.rand(rows, 8, generator=g, device=DEV))
        s["x"] = x.to(dt)
        f32 = dict(dtype=torch.float32, device=DEV)
        s["u"] = (torch.randint(1 << 23, (rows,), generator=g, device=DEV).float() + 0.5) * 2 ** -23
        r = torch.rand(rows, 4, generator=g, device=DEV)
        s["T"] = 0.6 + 0.6 * r[:, 0]
        f = c["filters"]
        pick = torch.randint(2, (rows, 3), generator=g, device=DEV) if f == "mixed" else \
            torch.tensor([[k in f and f != "none" for k in "kpm"]], device=DEV).expand(rows, 3)
        s["k"] = torch.where(pick[:, 0] > 0, (1 + 200 * r[:, 1]).to(torch.int32),
                             torch.zeros(rows, dtype=torch.int32, device=DEV))
        s["p"] = torch.where(pick[:, 1] > 0, 0.7 + 0.29 * r[:, 2], torch.ones(rows, **f32))
        s["mp"] = torch.where(pick[:, 2] > 0, 0.1 * r[:, 3], torch.zeros(rows, **f32))
        s["idx"] = torch.empty(rows, dtype=torch.int32, device=DEV)
        s["lp"] = torch.empty(rows, **f32)
    return s


# -------------------------------------------------------------- plain forms

def _rotate(x, pos, freq, m, layout, inverse=False):
    """x [rows, heads, D] -> float32, the first 2 len(freq) values of each head rotated."""
    rot = 2 * freq.numel()
    a = pos.double()[:, None] * freq  # far positions: the angle in 64 bits
    cos, sin = (m * a.cos()).float()[:, None], (m * a.sin()).float()[:, None]
    if inverse:
        sin = -sin
    y = x.float().clone()
    h = x[..., :rot].float()
    if layout == "half":
        h1, h2 = h[..., :rot // 2], h[..., rot // 2:]
        y[..., :rot // 2] = h1 * cos - h2 * sin
        y[..., rot // 2:rot] = h2 * cos + h1 * sin
    else:
        h1, h2 = h[..., 0::2], h[..., 1::2]
        y[..., 0:rot:2] = h1 * cos - h2 * sin
        y[..., 1:rot:2] = h2 * cos + h1 * sin
    return y


def _plain_append(s, c):
    rows = s["k"].shape[0]
    r = torch.arange(rows, device=DEV)
    b = torch.searchsorted(s["starts"].long(), r, right=True) - 1
    pos = s["ctx"].long()[b] + r - s["starts"].long()[b]
    page = s["table"].long()[b, pos // c["ps"]]
    slot = pos % c["ps"]
    s["q_out"].copy_(_rotate(s["q"], pos, s["freq"], s["m"], c["layout"]))
    s["k_pages"][page, :, slot] = _rotate(s["k"], pos, s["freq"], s["m"], c["layout"]).to(
        s["k_pages"].dtype)
    s["v_pages"][page, :, slot] = s["v"]
    return s["q_out"], s["k_pages"], s["v_pages"]


def _plain_attn(s, c):
    blk, Hkv, D, ps, P = c["blk"], c["Hkv"], c["D"], c["ps"], c["prefix"]
    G = c["Hq"] // Hkv
    for b, n in enumerate(s["lens"]):
        need = -(-n // ps)
        ids = s["table"][b, :need].long()

        def keys(pool, block):
            k = pool[ids].permute(1, 0, 2, 3).reshape(Hkv, need * ps, D)[:, :n].float()
            if P and b:
                ids0 = s["table"][0, :-(-P // ps)].long()
                k0 = pool[ids0].permute(1, 0, 2, 3).reshape(Hkv, -1, D)[:, :P].float()
                k = torch.cat([k0, k[:, P:]], 1)
            if block is not None:
                k = torch.cat([k, block[b].permute(1, 0, 2).float()], 1)
            return k

        k, v = keys(s["k_pages"], s["kb"]), keys(s["v_pages"], s["vb"])
        q = s["q"][b].view(blk, Hkv, G, D).permute(1, 0, 2, 3).reshape(Hkv, blk * G, D).float()
        z = (q @ k.transpose(1, 2)) * D ** -0.5
        total = k.shape[1]
        if c["mode"] == "causal":
            lim = total - blk + 1 + torch.arange(blk, device=DEV).repeat_interleave(G)
            z = z.masked_fill(torch.arange(total, device=DEV) >= lim[:, None], -math.inf)
        z = (z - z.amax(-1, keepdim=True)).exp()
        o = (z @ v) / z.sum(-1, keepdim=True)
        s["out"][b] = o.view(Hkv, blk, G, D).permute(1, 0, 2, 3).reshape(blk, c["Hq"], D)
    return s["out"]


def _plain_sample(s, c):
    V = c["vocab"]
    x, order = s["x"].float().sort(dim=1, descending=True, stable=True)  # ties: lowest index first
    # weights and their sums in 64 bits: a draw next to a border depends on them
    w = ((x.double() - x[:, :1].double()) / s["T"].double()[:, None]).exp()
    k = torch.where((s["k"] <= 0) | (s["k"] > V), torch.full_like(s["k"], V), s["k"])
    rank = torch.arange(V, device=DEV)
    w = torch.where(rank < k[:, None], w, torch.zeros_like(w))
    cum = w.cumsum(1)
    before = cum - w
    p = s["p"].double()[:, None]
    keep = (w > 0) & ((before < p * cum[:, -1:]) | (p >= 1)) & (w >= s["mp"].double()[:, None])
    w = torch.where(keep, w, torch.zeros_like(w))
    by_index = torch.zeros_like(w).scatter_(1, order, w)
    cum = by_index.cumsum(1)
    total = cum[:, -1:]
    hit = (cum > s["u"].double()[:, None] * total) & (by_index > 0)
    idx = hit.to(torch.uint8).argmax(1)
    s["idx"].copy_(idx)
    s["lp"].copy_((by_index.gather(1, idx[:, None]) / total).log()[:, 0])
    return s["idx"], s["lp"]


# --------------------------------------------------------------------- run

def run(state):
    s, c = state, state["case"]
    if own:
        import block_attention_b200 as ba
        layout = ba.ROPE_HALF if c.get("layout") == "half" else ba.ROPE_INTERLEAVED
        if c["op"] == "rope":
            return ba.rope(s["x"], s["pos"], s["freq"], layout=layout, mscale=s["m"],
                           inverse=c["inverse"], out=s["out"])
        if c["op"] == "append":
            ba.paged_append(s["k"], s["v"], s["k_pages"], s["v_pages"], s["table"], s["ctx"],
                            row_starts=s["starts"], inv_freq=s["freq"], layout=layout,
                            mscale=s["m"], q=s["q"], q_out=s["q_out"])
            return s["q_out"], s["k_pages"], s["v_pages"]
        if c["op"] == "attn":
            mode = ba.CAUSAL_VERIFY if c["mode"] == "causal" else ba.BIDIR_BLOCK
            return ba.paged_block_attn(s["q"], s["kb"], s["vb"], s["k_pages"], s["v_pages"],
                                       s["table"], s["ctx"], mode, shared_prefix=c["prefix"],
                                       max_ctx=max(s["lens"]), out=s["out"], workspace=s["ws"])
        ba.vocab_sample_filtered(s["x"], s["u"], temperature=s["T"], top_k=s["k"], top_p=s["p"],
                                 min_p=s["mp"], idx=s["idx"], logprob=s["lp"])
        return s["idx"], s["lp"]
    if c["op"] == "rope":
        s["out"].copy_(_rotate(s["x"], s["pos"], s["freq"], s["m"], c["layout"], c["inverse"]))
        return s["out"]
    if c["op"] == "append":
        return _plain_append(s, c)
    if c["op"] == "attn":
        return _plain_attn(s, c)
    return _plain_sample(s, c)


def work(case):
    c = case
    if c["op"] == "rope":
        n = c["rows"] * c["heads"] * c["D"]
        return {"bytes": 2 * n * _ES[c["dtype"]] + 4 * c["rows"],
                "flops": 3 * c["rows"] * c["heads"] * c["rot"]}
    if c["op"] == "append":
        rows = sum(_counts(c))
        n = rows * (c["Hq"] + 2 * c["Hkv"]) * c["D"]
        return {"bytes": 2 * n * _ES[c["dtype"]], "flops": 3 * rows * (c["Hq"] + c["Hkv"]) * c["rot"]}
    if c["op"] == "attn":
        es, blk, D, P = _ES[c["dtype"]], c["blk"], c["D"], c["prefix"]
        extra = 0 if c["in_cache"] else blk
        lens, B = _lens(c), c["B"]
        keys = sum(n - P + extra for n in lens) + P  # the common keys are read once
        seen = 0  # (row, key) pairs a head takes in
        for n in lens:
            total = n + extra
            seen += blk * total - (blk * (blk - 1) // 2 if c["mode"] == "causal" else 0)
        return {"bytes": 2 * keys * c["Hkv"] * D * es + 2 * B * blk * c["Hq"] * D * es,
                "flops": 4 * seen * c["Hq"] * D}
    n = c["rows"] * c["vocab"]
    return {"bytes": n * _ES[c["dtype"]] + c["rows"] * 28, "flops": 6 * n}


# ------------------------------------------------------------------- exact

def _exact_turn(x, pos, freq, m, layout, sign):
    """Rotation as a product of complex numbers, 64 bits."""
    h = freq.numel()
    out = x.double().clone()
    part = out[..., :2 * h]
    z = torch.complex(part[..., :h], part[..., h:]) if layout == "half" else \
        torch.complex(part[..., 0::2].contiguous(), part[..., 1::2].contiguous())
    ang = sign * pos.double()[:, None] * freq
    z = z * torch.polar(torch.full_like(ang, m), ang)[:, None]
    if layout == "half":
        out[..., :2 * h] = torch.cat([z.real, z.imag], -1)
    else:
        out[..., :2 * h] = torch.view_as_real(z).flatten(-2)
    return out


def exact(case, seed):
    c = dict(case)
    s = prepare(case, seed)
    if c["op"] == "rope":
        return _exact_turn(s["x"], s["pos"], s["freq"], s["m"], c["layout"],
                           -1.0 if c["inverse"] else 1.0)
    if c["op"] == "append":
        kp, vp = s["k_pages"].double(), s["v_pages"].double()
        q_out = torch.empty(s["q"].shape, dtype=torch.float64, device=DEV)
        row, ps, table = 0, c["ps"], s["table"].tolist()
        for b, (n, cnt) in enumerate(zip(_lens(c), _counts(c))):
            pos = torch.arange(n, n + cnt, device=DEV)
            sl = slice(row, row + cnt)
            q_out[sl] = _exact_turn(s["q"][sl], pos, s["freq"], s["m"], c["layout"], 1.0)
            k = _exact_turn(s["k"][sl], pos, s["freq"], s["m"], c["layout"], 1.0)
            at = n
            while at < n + cnt:  # page by page
                end = min(n + cnt, (at // ps + 1) * ps)
                page, lo = table[b][at // ps], at % ps
                kp[page, :, lo:lo + end - at] = k[at - n:end - n].transpose(0, 1)
                vp[page, :, lo:lo + end - at] = s["v"][row + at - n:row + end - n].double() \
                    .transpose(0, 1)
                at = end
            row += cnt
        return q_out, kp, vp
    if c["op"] == "attn":
        B, blk, Hq, Hkv, D, ps, P = (c["B"], c["blk"], c["Hq"], c["Hkv"], c["D"], c["ps"],
                                     c["prefix"])
        out = torch.empty(B, blk, Hq, D, dtype=torch.float64, device=DEV)
        for b, n in enumerate(s["lens"]):
            at = torch.arange(n, device=DEV)
            src = torch.where(at < P, torch.zeros_like(at), torch.full_like(at, b))
            page, slot = s["table"].long()[src, at // ps], at % ps
            for g in range(Hkv):
                k, v = s["k_pages"][page, g, slot].double(), s["v_pages"][page, g, slot].double()
                if s["kb"] is not None:
                    k = torch.cat([k, s["kb"][b, :, g].double()])
                    v = torch.cat([v, s["vb"][b, :, g].double()])
                q = s["q"][b, :, g * (Hq // Hkv):(g + 1) * (Hq // Hkv)].double()
                z = torch.einsum("ihd,kd->ihk", q, k) / math.sqrt(D)
                if c["mode"] == "causal":
                    for i in range(blk):
                        z[i, :, k.shape[0] - blk + i + 1:] = -math.inf
                out[b, :, g * (Hq // Hkv):(g + 1) * (Hq // Hkv)] = \
                    torch.einsum("ihk,kd->ihd", torch.softmax(z, -1), v)
        return out
    idx, lp = [], []
    for r in range(c["rows"]):
        x = s["x"][r].double()
        T, u = s["T"][r].double(), s["u"][r].double()
        k, p, mp = int(s["k"][r]), float(s["p"][r]), float(s["mp"][r])
        w = torch.exp((x - x.max()) / T)
        order = torch.argsort(x, descending=True, stable=True)
        if 0 < k < c["vocab"]:
            order = order[:k]
        ws = w[order]
        if p < 1:
            mass = torch.cumsum(ws, 0)
            order = order[:int((mass < p * mass[-1]).sum()) + 1]
        kept = order[w[order] >= mp].sort().values
        mass = torch.cumsum(w[kept], 0)
        i = kept[min(int((mass <= u * mass[-1]).sum()), kept.numel() - 1)]
        idx.append(i)
        lp.append((x[i] - x.max()) / T - torch.log(mass[-1]))
    return torch.stack(idx).to(torch.int32), torch.stack(lp)
