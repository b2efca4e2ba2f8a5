"""Measured cases of the serving operators: prompt attention over packed sequences, the paged 8-bit
key/value cache (writing tokens, managing pages) and the attention of single tokens over it.

``run`` computes an operator on the state that ``prepare`` made: in its plain form, with elementary
torch operations in 32 bits, or, where ``own`` is true, through the package's entry points.

Formulas.  For query row i with allowed keys j, S_ij = scale <Q_i, K_j>:
  softmax (alpha = 1)     p_ij = exp(S_ij - tau_i),          tau_i = log sum_j exp(S_ij);
  1.5-entmax (alpha 1.5)  p_ij = max(0, (S_ij - tau_i)/2)^2, tau_i with sum_j p_ij = 1;
  O_i = sum_j p_ij V_j.
Query head h reads key/value head h // (H / H_kv).  A cached key or value is its e4m3 number times the
power-of-two scale of its (layer, page, head) block; a page holds 64 tokens.
"""
import random

import torch

own = False

D = 64       # head size
PAGE = 64    # tokens of a page
E4M3_MAX = 448.0
MIN_EXP = -100  # smallest block scale: 2^-100


# ---------------------------------------------------------------------------------------------- cases

def listed():
    return [
        # a batch of short chat turns, packed: encoder-sized heads, lengths as in the padded workload of the
        # same shape (64 to 512), fp32 output
        dict(name="prompt softmax: short turns", op="prompt", alpha=1.0, lens=_pick(3, 32, 64, 512), H=12, Hkv=12, f32=True),
        # long documents beside each other, four query heads to a key/value head
        dict(name="prompt softmax: documents", op="prompt", alpha=1.0, lens="8192,4097,2999", H=16, Hkv=4, f32=False),
        # the framework's own weighting over mixed lengths, one token among them
        dict(name="prompt entmax: mixed", op="prompt", alpha=1.5, lens="4096,2500,1000,513,64,1", H=12, Hkv=12, f32=False),
        # one user's next token: latency
        dict(name="token softmax: one user", op="attn", alpha=1.0, n=1, lo=2049, hi=2049, pick=1, H=32, Hkv=8, f32=False),
        # a full serving batch, ragged contexts
        dict(name="token softmax: batch", op="attn", alpha=1.0, n=64, lo=700, hi=16384, pick=2, H=32, Hkv=8, f32=False),
        # one user with a long context, plain heads
        dict(name="token entmax: one user", op="attn", alpha=1.5, n=1, lo=16384, hi=16384, pick=3, H=12, Hkv=12, f32=True),
        # a serving batch of the framework's own weighting, three query heads to a key/value head
        dict(name="token entmax: batch", op="attn", alpha=1.5, n=48, lo=500, hi=16000, pick=4, H=12, Hkv=4, f32=False),
        # one new token for each running sequence
        dict(name="append: one token each", op="append", n=64, lo=1, hi=8000, new_lo=1, new_hi=1, pick=5, Hkv=8),
        # the keys and values of a batch of prompts
        dict(name="append: prompts", op="append", n=24, lo=0, hi=900, new_lo=100, new_hi=4096, pick=6, Hkv=8),
        # room for the next token of a running batch, after the last drafts were dropped
        dict(name="pages: next token", op="resize", n=128, lo=1, hi=4000, new=5, pick=7, layers=2, Hkv=4),
        # beams: sixteen sequences forked four times each, every fork about to write a token of its own
        dict(name="pages: beams", op="beams", n=16, width=4, lo=60, hi=3000, pick=8, layers=12, Hkv=12),
        # a fragmented pool packed to its front
        dict(name="pages: compact", op="compact", pages=2500, share=0.6, pick=9, layers=12, Hkv=8),
    ]


def draw(rng):
    op = rng.choice(["prompt", "prompt", "attn", "attn", "append", "resize", "beams", "compact"])
    pick = rng.randrange(1 << 30)
    hkv = rng.choice([1, 2, 3, 4, 8, 12])
    if op == "prompt":
        n = _log(rng, 1, 24)
        most = max(1, min(8192, int(8192 / n ** 0.5)))
        lens = _pick(pick, n, 1, _log(rng, 16, max(16, most)))
        heads = hkv * rng.choice([1, 2, 4] if hkv <= 4 else [1])
        return dict(op=op, alpha=rng.choice([1.0, 1.5]), lens=lens, H=heads, Hkv=hkv, f32=rng.random() < 0.3)
    if op == "attn":
        n = _log(rng, 1, 64)
        hi = _log(rng, 1, 16384)
        heads = hkv * rng.choice([1, 2, 3, 4, 5, 8] if hkv <= 4 else [1, 2, 4])
        if heads > 32:
            heads = hkv
        hi = min(hi, 4_000_000 // (n * hkv))
        return dict(op=op, alpha=rng.choice([1.0, 1.5]), n=n, lo=rng.randint(1, hi), hi=hi, pick=pick, H=heads, Hkv=hkv, f32=rng.random() < 0.3)
    if op == "append":
        lo = _log(rng, 1, 1400)
        return dict(op=op, n=_log(rng, 1, 24), lo=0, hi=_log(rng, 1, 2000), new_lo=lo, new_hi=rng.randint(lo, 2 * lo), pick=pick, Hkv=min(hkv, 8))
    if op == "resize":
        return dict(op=op, n=_log(rng, 1, 128), lo=1, hi=_log(rng, 1, 4000), new=_log(rng, 1, 300), pick=pick, layers=rng.randint(1, 4), Hkv=min(hkv, 4))
    if op == "beams":
        return dict(op=op, n=_log(rng, 1, 16), width=rng.randint(1, 4), lo=1, hi=_log(rng, 1, 3000), pick=pick, layers=rng.randint(1, 12), Hkv=hkv)
    return dict(op=op, pages=_log(rng, 20, 2500), share=round(rng.uniform(0.2, 0.95), 3), pick=pick, layers=rng.randint(1, 12), Hkv=min(hkv, 8))


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def _pick(seed, n, lo, hi):
    r = random.Random(seed)
    return ",".join(str(r.randint(lo, hi)) for _ in range(n))


def _lens(case):
    r = random.Random(case["pick"])
    return [r.randint(case["lo"], case["hi"]) for _ in range(case["n"])]


def _new(case):
    r = random.Random(case["pick"] + 1)
    return [r.randint(case["new_lo"], case["new_hi"]) for _ in range(case["n"])]


def _pages(tokens):
    return (tokens + PAGE - 1) // PAGE


def work(case):
    op = case["op"]
    if op == "prompt":
        lens = [int(x) for x in case["lens"].split(",")]
        pairs = case["H"] * sum(n * (n + 1) // 2 for n in lens)
        rows = sum(lens)
        # Q, K, V in bf16, O, tau; products S and P V.  The weights of 1.5-entmax are zero for most keys: what cannot be done
        # without is S (2 D a pair) and the products of the support, a small share
        return {"bytes": rows * D * (2 * case["H"] + 4 * case["Hkv"] + (4 if case["f32"] else 2) * case["H"]) + 4 * rows * case["H"],
                "flops": pairs * D * (4 if case["alpha"] == 1.0 else 2)}
    if op == "attn":
        tokens = sum(_lens(case))
        # every key once; every value once for softmax, a small share for 1.5-entmax
        return {"bytes": tokens * case["Hkv"] * D * (2 if case["alpha"] == 1.0 else 1) + case["n"] * case["H"] * (D * (2 + (4 if case["f32"] else 2)) + 4),
                "flops": tokens * case["H"] * D * (4 if case["alpha"] == 1.0 else 2)}
    if op == "append":
        new = sum(_new(case))
        return {"bytes": new * case["Hkv"] * D * 2 * (2 + 1), "flops": new * case["Hkv"] * D * 2 * 3}
    page = case["layers"] * case["Hkv"] * (2 * PAGE * D + 8)  # bytes of a page's blocks and scales
    if op == "resize":
        total = sum(_pages(n + case["new"]) for n in _lens(case))
        return {"bytes": 4 * (2 * total + 6 * case["n"]), "flops": 0}
    if op == "beams":
        lens = _lens(case)
        copied = sum(case["width"] for n in lens if n % PAGE)
        return {"bytes": 2 * copied * page + 4 * sum(_pages(n) for n in lens) * (1 + case["width"]) * 2, "flops": 0}
    used = _used(case)
    low = sum(1 for p in used if p >= len(used))
    return {"bytes": 2 * low * page + 4 * 3 * case["pages"], "flops": 0}


def _used(case):
    r = random.Random(case["pick"])
    used = [p for p in range(case["pages"]) if r.random() < case["share"]]
    return used or [case["pages"] - 1]


# --------------------------------------------------------------------------------------------- inputs

def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)
    op = case["op"]

    def normal(*shape):
        return torch.randn(shape, generator=g, device=dev)

    def ints(v):
        return torch.tensor(v, dtype=torch.int32, device=dev)

    if op == "prompt":
        lens = [int(x) for x in case["lens"].split(",")]
        T, H, Hkv = sum(lens), case["H"], case["Hkv"]
        # Q, K and V side by side, as a fused projection writes them
        qkv = normal(T, H + 2 * Hkv, D).to(torch.bfloat16)
        cu = torch.zeros(len(lens) + 1, dtype=torch.int64)
        cu[1:] = torch.tensor(lens).cumsum(0)
        return dict(op=op, Q=qkv[:, :H], K=qkv[:, H:H + Hkv], V=qkv[:, H + Hkv:], cu=cu.to(dev, torch.int32), max_len=max(lens),
                    scale=D ** -0.5, alpha=case["alpha"], dtype=torch.float32 if case["f32"] else torch.bfloat16)

    if op == "compact":
        used = _used(case)
        lens, have = [], len(used)
        while have:  # sequences of at most 40 pages
            lens.append(min(have, 40) * PAGE)
            have -= min(have, 40)
        n_pages, spread = case["pages"], used
    else:
        lens = _lens(case)
        if op == "append":
            lens = [a + b for a, b in zip(lens, _new(case))]
        spread = None
        spare = {"attn": 3, "append": 3, "resize": case["n"] * (_pages(case.get("new", 0)) + 1), "beams": case["n"] * case.get("width", 0) * 2 + 4}[op]
        n_pages = sum(_pages(n) for n in lens) + spare
    layers = case.get("layers", 2)
    slots = len(lens) * (1 + case.get("width", 0))
    max_pages = _pages(max(lens) + case.get("new", 1)) + 1
    shape = (layers, n_pages, case["Hkv"])
    r = random.Random(seed)
    if spread is None:
        spread = list(range(n_pages))
    r.shuffle(spread)
    table, refs, at = [[-1] * max_pages for _ in range(slots)], [0] * n_pages, 0
    for s, n in enumerate(lens):
        for k in range(_pages(n)):
            table[s][k] = spread[at]
            refs[spread[at]] = 1
            at += 1
    # blocks as the cache holds them: the largest of a block's 4096 numbers lies near the format's end, and the
    # values behind them have a deviation near one
    pools, scales = [], []
    for _ in range(2):
        pool = torch.empty(shape + (PAGE, D), dtype=torch.float8_e4m3fn, device=dev)
        for k in range(layers):
            size = 58 + 40 * torch.rand(shape[1:] + (1, 1), generator=g, device=dev)
            pool[k] = (normal(*shape[1:], PAGE, D) * size).clamp_(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
        pools.append(pool)
        scales.append(torch.exp2(torch.randint(-7, -5, shape, generator=g, device=dev).float()))
    st = dict(op=op, K=pools[0], V=pools[1], k_scale=scales[0], v_scale=scales[1], refs=ints(refs), table=ints(table),
              lens=ints(lens + [0] * (slots - len(lens))), layer=layers - 1)
    order = list(range(len(lens)))
    r.shuffle(order)
    st["seqs"] = ints(order)
    if op == "attn":
        st.update(Q=normal(len(lens), case["H"], D).to(torch.bfloat16), scale=D ** -0.5, alpha=case["alpha"], max_len=max(lens),
                  dtype=torch.float32 if case["f32"] else torch.bfloat16)
    elif op == "append":
        new = [_new(case)[s] for s in order]
        cu = torch.zeros(len(new) + 1, dtype=torch.int64)
        cu[1:] = torch.tensor(new).cumsum(0)
        kv = normal(int(cu[-1]), 2 * case["Hkv"], D).to(torch.bfloat16)  # one projection writes both
        st.update(newK=kv[:, :case["Hkv"]], newV=kv[:, case["Hkv"]:], cu=cu.to(dev, torch.int32), most=max(new))
    elif op == "resize":
        st.update(base=ints([lens[s] for s in order]), grown=ints([lens[s] + case["new"] for s in order]))
    elif op == "beams":
        w = case["width"]
        st.update(src=ints([s for s in order for _ in range(w)]), dst=ints([len(lens) + k for k in range(w * len(lens))]),
                  none=ints([0] * (w * len(lens))), grown=ints([lens[s] + 1 for s in order for _ in range(w)]))
    elif op == "compact":
        st.update(refs0=st["refs"].clone(), table0=st["table"].clone())
    return st


# ------------------------------------------------------------------------------------------ plain forms

def _weights(S, alpha):
    """S [..., keys] in fp32, -inf where masked, overwritten: (weights, tau)."""
    m = S.amax(-1, keepdim=True)
    S -= torch.where(m.isinf(), 0.0, m)
    if alpha == 1.0:
        P = S.exp_()
        l = P.sum(-1, keepdim=True)
        return P.div_(l), (m + l.log()).squeeze(-1)
    # Newton's method on sum max(0, x - t)^2 = 4 from t = max - 2: convex and decreasing, so t rises to the root
    t = torch.full_like(m, -2.0)
    for _ in range(16):
        d = (S - t).clamp_(min=0)
        s1 = d.sum(-1, keepdim=True)
        t += (d.square_().sum(-1, keepdim=True) - 4) / (2 * s1)
    return S.sub_(t).clamp_(min=0).mul_(0.5).square_(), (m + t).squeeze(-1)


def _plain_prompt(st):
    Q, K, V, cu = st["Q"], st["K"], st["V"], st["cu"].long()
    T, H, Hkv = Q.shape[0], Q.shape[1], K.shape[1]
    L, n = st["max_len"], cu.numel() - 1
    lens = cu[1:] - cu[:-1]
    pos = torch.arange(L, device=Q.device)
    live = pos[None] < lens[:, None]
    at = (cu[:-1, None] + pos[None]).clamp_(max=T - 1)
    q = Q.float()[at].permute(0, 2, 1, 3).reshape(n, Hkv, (H // Hkv) * L, D)
    k = K.float()[at].permute(0, 2, 3, 1)
    v = torch.where(live[:, :, None, None], V.float()[at], 0.0).permute(0, 2, 1, 3)
    S = (q @ k).mul_(st["scale"]).view(n, Hkv, H // Hkv, L, L)
    S.masked_fill_(~((pos[:, None] >= pos[None])[None] & live[:, None])[:, None, None], float("-inf"))
    P, tau = _weights(S, st["alpha"])
    O = (P.view(n, Hkv, -1, L) @ v).view(n, H, L, D).permute(0, 2, 1, 3)
    return O[live].to(st["dtype"]), tau.reshape(n, H, L).permute(1, 0, 2)[:, live]


def _gather(pool, scale, layer, pages):
    """Tokens of the listed pages [n, p] in fp32: [n, H_kv, p * 64, 64]."""
    n, p = pages.shape
    x = pool[layer].view(torch.uint8)[pages].view(torch.float8_e4m3fn).float() * scale[layer][pages][..., None, None]
    return x.permute(0, 2, 1, 3, 4).reshape(n, x.shape[2], p * PAGE, D)


def _plain_attn(st):
    seqs = st["seqs"].long()
    lens = st["lens"][seqs].long()
    n, H = st["Q"].shape[:2]
    pages = st["table"][seqs].long()[:, :_pages(st["max_len"])].clamp_(min=0)
    live = (torch.arange(pages.shape[1] * PAGE, device=pages.device)[None] < lens[:, None])[:, None, :]
    k = _gather(st["K"], st["k_scale"], st["layer"], pages)
    q = st["Q"].float().view(n, k.shape[1], -1, D)
    S = (q @ k.transpose(2, 3)).mul_(st["scale"])
    del k
    S.masked_fill_(~live[:, None], float("-inf"))
    P, tau = _weights(S, st["alpha"])
    v = _gather(st["V"], st["v_scale"], st["layer"], pages).masked_fill_(~live[..., None], 0.0)
    return (P @ v).view(n, H, D).to(st["dtype"]), tau.reshape(n, H)


def _block_scale(amax):
    """Smallest power of two s with amax / s <= 448, at least 2^-100."""
    m, e = torch.frexp(amax)  # amax = m 2^e, m in [0.5, 1); 448 = 0.875 * 2^9
    e = torch.where(m > 0.875, e - 8, e - 9)
    return torch.ldexp(torch.ones_like(amax), torch.where(amax > 0, e, MIN_EXP).clamp(min=MIN_EXP))


def _plain_append(st):
    seqs, cu, most = st["seqs"].long(), st["cu"].long(), st["most"]
    end = st["lens"][seqs].long()
    start = end - (cu[1:] - cu[:-1])
    n, dev = seqs.numel(), seqs.device
    first = start // PAGE
    p = _pages(most) + 1                                         # pages that an entry touches, at most
    which = first[:, None] + torch.arange(p, device=dev)         # [n, p] page of the sequence
    touched = which * PAGE < end[:, None]
    entry, k = touched.nonzero(as_tuple=True)
    page = st["table"][seqs].long()[entry, which[entry, k]]      # [m] page of the pool
    pos = which[entry, k][:, None] * PAGE + torch.arange(PAGE, device=dev)
    is_new = (pos >= start[entry][:, None]) & (pos < end[entry][:, None])
    is_kept = pos < start[entry][:, None]
    tok = (cu[entry][:, None] + pos - start[entry][:, None]).clamp_(0, st["newK"].shape[0] - 1)
    for pool, scale, x in ((st["K"], st["k_scale"], st["newK"]), (st["V"], st["v_scale"], st["newV"])):
        new = x.float()[tok].permute(0, 2, 1, 3)                  # [m, H_kv, 64, 64]
        bytes_ = pool[st["layer"]].view(torch.uint8)
        old8 = bytes_[page]
        old_scale = scale[st["layer"]][page]                      # [m, H_kv]
        amax = new.abs().masked_fill(~is_new[:, None, :, None], 0.0).amax((2, 3))
        s = torch.maximum(_block_scale(amax), torch.where(is_kept.any(1)[:, None], old_scale, 0.0))[..., None, None]
        kept = old8.view(torch.float8_e4m3fn).float() * old_scale[..., None, None]
        q8 = (torch.where(is_new[:, None, :, None], new, kept) / s).to(torch.float8_e4m3fn).view(torch.uint8)
        bytes_[page] = torch.where((is_new | is_kept)[:, None, :, None], q8, old8)
        scale[st["layer"]][page] = s[..., 0, 0]
    return st["K"], st["V"], st["k_scale"], st["v_scale"]


def _plain_resize(st, seqs, new):
    seqs, new, table, refs = seqs.long(), new.long(), st["table"], st["refs"]
    old = st["lens"][seqs].long()
    have, want = _pages(old), _pages(new)
    rows = table[seqs].long()
    k = torch.arange(rows.shape[1], device=seqs.device)
    # release what lies behind the new end
    drop = (k >= want[:, None]) & (k < have[:, None])
    refs.index_add_(0, rows.clamp(min=0).view(-1), -drop.view(-1).int())
    rows = torch.where(drop, -1, rows)
    # a page that is written on and shared is copied, but for the last of the list where all its holders grow
    last = torch.where(have > 0, rows.gather(1, (have - 1).clamp(min=0)[:, None])[:, 0], -1)
    writes = (new > old) & (old % PAGE != 0)
    shared = writes & (refs[last.clamp(min=0)] > 1)
    same = (last[:, None] == last[None]) & shared[:, None] & shared[None]
    i = torch.arange(seqs.numel(), device=seqs.device)
    keeps = shared & (same.sum(1) == refs[last.clamp(min=0)]) & ~(same & (i[None] > i[:, None])).any(1)
    copies = shared & ~keeps
    refs.index_add_(0, last.clamp(min=0), -copies.int())
    # the lowest free pages, in the order of the list
    before = refs + torch.zeros_like(refs).index_add_(0, last.clamp(min=0), copies.int())
    free = torch.argsort((before > 0).int(), stable=True)
    need = copies.long() + (want - have).clamp(min=0)
    base = need.cumsum(0) - need
    fresh = free[base.clamp(max=free.numel() - 1)]
    c = copies.nonzero()[:, 0]
    if c.numel():
        for name in ("K", "V", "k_scale", "v_scale"):
            x = st[name].view(torch.uint8) if name in ("K", "V") else st[name]
            x[:, fresh[c]] = x[:, last[c]]
    rows = torch.where(copies[:, None] & (k == have[:, None] - 1), fresh[:, None], rows)
    add = (k >= have[:, None]) & (k < want[:, None])
    rows = torch.where(add, free[(base[:, None] + copies[:, None].long() + k - have[:, None]).clamp(0, free.numel() - 1)], rows)
    taken = add | (copies[:, None] & (k == have[:, None] - 1))
    refs.index_add_(0, rows.clamp(min=0).view(-1), taken.view(-1).int())
    table[seqs] = rows.int()
    st["lens"][seqs] = new.int()
    return (need.sum() - (before == 0).sum()).clamp(min=0).int().view(1)


def _plain_fork(st):
    src, dst = st["src"].long(), st["dst"].long()
    rows = st["table"][src]
    held = torch.arange(rows.shape[1], device=src.device) < _pages(st["lens"][src].long())[:, None]
    st["refs"].index_add_(0, rows.clamp(min=0).long().view(-1), held.view(-1).int())
    st["table"][dst] = torch.where(held, rows, -1)
    st["lens"][dst] = st["lens"][src]


def _plain_compact(st):
    refs, n = st["refs"], st["refs"].numel()
    used = refs > 0
    count = used.sum()
    p = torch.arange(n, device=refs.device)
    src, dst = (used & (p >= count)).nonzero()[:, 0], (~used & (p < count)).nonzero()[:, 0]
    for name in ("K", "V", "k_scale", "v_scale"):
        x = st[name].view(torch.uint8) if name in ("K", "V") else st[name]
        x[:, dst] = x[:, src]
    to = p.clone()
    to[src] = dst
    refs[dst] = refs[src]
    refs[src] = 0
    table = st["table"]
    table.copy_(torch.where(table >= 0, to[table.clamp(min=0).long()], -1))
    return count.int().view(1)


def _plain(st):
    op = st["op"]
    if op == "prompt":
        return _plain_prompt(st)
    if op == "attn":
        return _plain_attn(st)
    if op == "append":
        return _plain_append(st)
    if op == "resize":
        _plain_resize(st, st["seqs"], st["base"])
        short = _plain_resize(st, st["seqs"], st["grown"])
        return st["table"], st["refs"], st["lens"], short
    if op == "beams":
        _plain_resize(st, st["dst"], st["none"])
        _plain_fork(st)
        short = _plain_resize(st, st["dst"], st["grown"])
        return st["table"], st["refs"], st["lens"], short, st["K"], st["V"], st["k_scale"], st["v_scale"]
    st["table"].copy_(st["table0"])
    st["refs"].copy_(st["refs0"])
    count = _plain_compact(st)
    return st["table"], st["refs"], count, st["K"], st["V"], st["k_scale"], st["v_scale"]


# ---------------------------------------------------------------------------------- the package's calls

def _own(st):
    import entmax_tcgen05_tma_b200 as E

    op = st["op"]
    if op == "prompt":
        return E.entmax_attn_prompt(st["Q"], st["K"], st["V"], st["cu"], st["max_len"], scale=st["scale"], alpha=st["alpha"], out_dtype=st["dtype"])
    c = st.get("cache")
    if c is None:  # the handle that a user's program makes once for its pool
        c = st["cache"] = E.EntmaxCache(st["K"], st["V"], st["k_scale"], st["v_scale"], st["refs"], st["table"], st["lens"])
    if op == "attn":
        return E.entmax_cache_attn(c, st["layer"], st["Q"], st["seqs"], st["max_len"], scale=st["scale"], alpha=st["alpha"], out_dtype=st["dtype"])
    if op == "append":
        E.entmax_cache_append(c, st["layer"], st["newK"], st["newV"], st["seqs"], st["cu"])
        return st["K"], st["V"], st["k_scale"], st["v_scale"]
    if op == "resize":
        E.entmax_cache_resize(c, st["seqs"], st["base"])
        short = E.entmax_cache_resize(c, st["seqs"], st["grown"])
        return st["table"], st["refs"], st["lens"], short
    if op == "beams":
        E.entmax_cache_resize(c, st["dst"], st["none"])
        E.entmax_cache_fork(c, st["src"], st["dst"])
        short = E.entmax_cache_resize(c, st["dst"], st["grown"])
        return st["table"], st["refs"], st["lens"], short, st["K"], st["V"], st["k_scale"], st["v_scale"]
    st["table"].copy_(st["table0"])
    st["refs"].copy_(st["refs0"])
    count = E.entmax_cache_compact(c)
    return st["table"], st["refs"], count, st["K"], st["V"], st["k_scale"], st["v_scale"]


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------------------------------ in 64 bits

def _exact_rows(S, alpha):
    """Weights and tau of rows of scores in fp64 (-inf where masked; at least one key a row)."""
    if alpha == 1.0:
        tau = torch.logsumexp(S, -1)
        return torch.exp(S - tau[..., None]), tau
    # the sorted closed form: on the k largest scores z the root of sum (z - t)^2 = 4 is mean - sqrt(4/k - variance);
    # the support is the largest k with root < z_k.  Scores two or more below the maximum never belong to it.
    m = S.amax(-1, keepdim=True)
    X = (S - m).clamp(min=-2.0)
    z = X.sort(-1, descending=True).values
    k = torch.arange(1, z.shape[-1] + 1, device=z.device, dtype=torch.float64)
    mean = z.cumsum(-1) / k
    var = (z * z).cumsum(-1) / k - mean * mean
    root = mean - (4.0 / k - var).clamp(min=0).sqrt()
    ok = (4.0 / k - var >= 0) & (root < z)
    size = (ok * k).amax(-1, keepdim=True).long() - 1
    t = root.gather(-1, size)
    return ((X - t).clamp(min=0) / 2) ** 2, (m + t).squeeze(-1)


def _exact_e4m3(x):
    """x in fp64 to the nearest e4m3 number, ties to even, from the format: 4 significant bits, least exponent -6."""
    e = torch.frexp(x).exponent - 1
    step = torch.ldexp(torch.ones_like(x), e.clamp(min=-6) - 3)
    return torch.round(x / step) * step


def exact(case, seed):
    op = case["op"]
    if op in ("resize", "beams", "compact"):
        return None  # pages and counts: nothing is computed
    st = prepare(case, seed)
    if op == "prompt":
        Q, K, V = st["Q"], st["K"], st["V"]
        T, H, G = Q.shape[0], Q.shape[1], Q.shape[1] // K.shape[1]
        O = torch.empty(T, H, D, dtype=torch.float64, device=Q.device)
        tau = torch.empty(H, T, dtype=torch.float64, device=Q.device)
        at = 0
        for n in (int(x) for x in case["lens"].split(",")):
            later = torch.ones(n, n, dtype=torch.bool, device=Q.device).triu(1)
            for h in range(H):
                S = st["scale"] * (Q[at:at + n, h].double() @ K[at:at + n, h // G].double().T)
                P, tau[h, at:at + n] = _exact_rows(S.masked_fill_(later, float("-inf")), case["alpha"])
                O[at:at + n, h] = P @ V[at:at + n, h // G].double()
            at += n
        return O, tau
    if op == "attn":
        n, H = st["Q"].shape[:2]
        O = torch.empty(n, H, D, dtype=torch.float64, device=st["Q"].device)
        tau = torch.empty(n, H, dtype=torch.float64, device=st["Q"].device)
        for i, s in enumerate(st["seqs"].tolist()):
            N = int(st["lens"][s])
            pages = st["table"][s, :_pages(N)].long()
            G = H // st["K"].shape[2]
            for g in range(st["K"].shape[2]):
                k, v = ((x[st["layer"], :, g].view(torch.uint8).index_select(0, pages).view(torch.float8_e4m3fn).double()
                         * f[st["layer"], :, g].index_select(0, pages).double()[:, None, None]).reshape(-1, D)[:N]
                        for x, f in ((st["K"], st["k_scale"]), (st["V"], st["v_scale"])))
                P, tau[i, g * G:(g + 1) * G] = _exact_rows(st["scale"] * (st["Q"][i, g * G:(g + 1) * G].double() @ k.T), case["alpha"])
                O[i, g * G:(g + 1) * G] = P @ v
        return O, tau
    cu, layer = st["cu"].tolist(), st["layer"]
    out = []
    for pool, scale, x in (("K", "k_scale", "newK"), ("V", "v_scale", "newV")):
        num, f = st[pool].double(), st[scale].double()
        for i, s in enumerate(st["seqs"].tolist()):
            end = int(st["lens"][s])
            start = end - (cu[i + 1] - cu[i])
            for k in range(start // PAGE, _pages(end)):
                page = int(st["table"][s, k])
                a, b = max(start, k * PAGE), min(end, (k + 1) * PAGE)
                new = st[x][cu[i] + a - start:cu[i] + b - start].double()                     # [tokens, heads, 64]
                top = new.abs().amax((0, 2))
                need = torch.exp2(torch.ceil(torch.log2(top / E4M3_MAX))).clamp(min=2.0 ** MIN_EXP)
                was = f[layer, page].clone()
                f[layer, page] = torch.maximum(need, was) if a > k * PAGE else need
                by = f[layer, page][:, None, None]
                kept = a - k * PAGE
                num[layer, page, :, :kept] = _exact_e4m3(num[layer, page, :, :kept] * (was[:, None, None] / by))
                num[layer, page, :, kept:kept + b - a] = _exact_e4m3(new.permute(1, 0, 2) / by)
        out.append((num, f))
    return out[0][0], out[1][0], out[0][1], out[1][1]
