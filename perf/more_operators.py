"""A serving step's and a training step's operators around paged attention: what is measured of them.

  slots   a step's bookkeeping from its request lengths: page tables extended from the free pages, the new tokens'
          positions and cache slots, the sequences' offsets and lengths
  norm    queries and keys normed for each head (root mean square) and rotated in the same pass: forward, backward with
          the weights' gradients, and on the way into a paged cache
  chunk   attention of a ragged batch's new tokens over the paged cache, causal: prompts, parts of prompts, drafts
  window  the same where a token sees the last keys of a sliding window and a few first keys (sinks)

``run`` computes them in plain torch operations (``own`` false) or calls the framework (``own`` true);
``exact`` computes them from their definitions in float64.
"""
import math
import random

import torch

own = False

DEV = "cuda"


# ------------------------------------------------------------------------------------------ cases

def _slots(name, B, page, new_lo, new_hi, ctx_lo, ctx_hi, pad, lens_seed=1):
    return {"name": name, "op": "slots", "B": B, "page": page, "new_lo": new_lo, "new_hi": new_hi, "ctx_lo": ctx_lo,
            "ctx_hi": ctx_hi, "pad": pad, "lens_seed": lens_seed}


def _norm(name, way, B, H, Hkv, N, d, dtype, axes, interleaved, rot=None, far=0, page=16, pad=0):
    return {"name": name, "op": "norm", "way": way, "B": B, "H": H, "Hkv": Hkv, "N": N, "d": d, "dtype": dtype,
            "axes": axes, "interleaved": interleaved, "rot": d if rot is None else rot, "far": far, "page": page,
            "pad": pad}


def _chunk(name, B, H, Hkv, d, page, new_lo, new_hi, ctx_lo, ctx_hi, window=0, sinks=0, lens_seed=1):
    return {"name": name, "op": "window" if window else "chunk", "B": B, "H": H, "Hkv": Hkv, "d": d, "page": page,
            "new_lo": new_lo, "new_hi": new_hi, "ctx_lo": ctx_lo, "ctx_hi": ctx_hi, "window": window, "sinks": sinks,
            "lens_seed": lens_seed}


def listed():
    return [
        # a generation step of a large batch: a token each, a new page here and there, unused places at the end
        _slots("slots decode batch", 237, 16, 1, 1, 1, 32768, 19),
        # a step that admits prompts of all lengths beside running sequences
        _slots("slots prompts", 61, 16, 1, 8192, 0, 8192, 0),
        # one short clip of video patches in fp32: three position axes, an odd number of tokens
        _norm("norm small clip fp32", "forward", 1, 16, 4, 333, 64, "fp32", 3, False),
        # a training step's q and k, text positions far into a long document
        _norm("norm train bf16", "forward", 2, 32, 8, 8192, 128, "bf16", 1, False, far=900_000),
        # the same step's backward, with the gradients of both norms' weights
        _norm("norm train backward", "backward", 2, 32, 8, 8192, 128, "bf16", 1, False, far=900_000),
        # a decode batch's new tokens into the cache, with unused places at the end, part of each head rotated
        _norm("norm append decode batch", "append", 1, 32, 8, 237, 64, "bf16", 1, False, rot=32, far=30_000, pad=19),
        # a short question behind a context: latency counts
        _chunk("chunk one question", 1, 32, 8, 128, 16, 23, 23, 1000, 1000),
        # a serving step that mixes running sequences (a token each) with pieces of prompts
        _chunk("chunk mixed batch", 37, 32, 4, 64, 16, 1, 512, 0, 8192),
        # drafted tokens of a batch verified over long contexts: bound by the cache's bytes
        _chunk("chunk drafts", 24, 32, 8, 128, 16, 3, 7, 4096, 32768),
        # a long prompt from its first token on: bound by the matrix products
        _chunk("chunk long prompt", 1, 32, 8, 128, 64, 8191, 8191, 0, 0),
        # a piece of a long prompt through a sliding-window layer
        _chunk("window prompt", 1, 32, 8, 64, 32, 2048, 2048, 16384, 16384, window=1024, sinks=4),
        # single tokens through a sliding-window layer
        _chunk("window single tokens", 48, 32, 8, 128, 16, 1, 1, 100, 16384, window=4096, sinks=4),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["slots", "norm", "chunk", "chunk", "window"])
    if op == "slots":
        B = _log(rng, 1, 1024)
        hi = _log(rng, 1, max(1, min(8192, 200_000 // B)))
        c = _slots("", B, rng.choice([1, 16, 32, 64, 24]), rng.choice([0, 1, hi]), hi, 0, _log(rng, 1, 32768),
                   rng.randint(0, 64), lens_seed=rng.randint(1, 1 << 30))
        del c["name"]
        return c
    d = rng.choice([64, 128])
    Hkv = rng.choice([1, 2, 4, 8])
    H = Hkv * rng.choice([1, 2, 3, 4, 8])
    # no drawn case costs more than the largest listed one of its operator: the sizes drawn last are cut to that
    if op == "norm":
        way = rng.choice(["forward", "backward", "append"])
        B = 1 if way == "append" else rng.randint(1, 4)
        dtype = "bf16" if way == "append" else rng.choice(["bf16", "bf16", "fp32"])
        most = 2 * 40 * 8192 * 128 * (2 if dtype == "bf16" else 1) // (2 * B * (H + 2 * Hkv) * d)
        N = _log(rng, 1, min(8192, most))
        c = _norm("", way, B, H, Hkv, N, d, dtype, rng.choice([1, 1, 3]), rng.random() < 0.4,
                  rot=rng.choice([d, d, 32]), far=rng.choice([0, 100_000]), page=rng.choice([16, 32, 64, 24]),
                  pad=rng.randint(0, N // 8) if way == "append" else 0)
    else:
        B = _log(rng, 1, 64)
        new_hi = _log(rng, 1, 2048)
        ctx_hi = _log(rng, 16, 32768)
        # padded scores of the plain form, and the keys of all sequences
        new_hi = max(1, min(new_hi, (8192 * 8192 * 32) // (B * H * (ctx_hi + new_hi))))
        ctx_hi = max(1, min(ctx_hi, 24 * 32768 * 8 * 128 // (B * Hkv * d)))
        window = 0 if op == "chunk" else _log(rng, 1, 8192)
        c = _chunk("", B, H, Hkv, d, rng.choice([16, 32, 64, 24, 128]), rng.choice([1, new_hi]), new_hi,
                   rng.choice([0, ctx_hi // 2, ctx_hi]), ctx_hi, window=window,
                   sinks=rng.choice([0, 1, 4, 64, 130]) if window else 0, lens_seed=rng.randint(1, 1 << 30))
    del c["name"]
    return c


def _lengths(case):
    """(tokens in the cache before the step, new tokens) of the case's sequences: spread over their logarithm, the
    longest and the shortest of both among them."""
    rng = random.Random(case["lens_seed"])

    def spread(lo, hi):
        lens = [min(hi, max(lo, _log(rng, max(lo, 1), max(hi, 1)))) for _ in range(case["B"])]
        lens[0] = hi
        if case["B"] > 1:
            lens[rng.randrange(1, case["B"])] = lo
        return lens

    return spread(case["ctx_lo"], case["ctx_hi"]), spread(case["new_lo"], case["new_hi"])


# ------------------------------------------------------------------------------------------ inputs

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _randn(shape, g, dtype=torch.bfloat16, mult=1.0):
    return (torch.randn(shape, generator=g, device=DEV) * mult).to(dtype)


def _int32(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


def _rotation(case):
    """Frequencies (radians a position, float64) and the axis of each pair: thirds (or halves) of the pairs in turn."""
    n = case["rot"] // 2
    freqs = torch.tensor([10000.0 ** (-i / n) for i in range(n)], dtype=torch.float64, device=DEV)
    return freqs, _int32([i * case["axes"] // n for i in range(n)])


def _positions(case, shape, g):
    """int32 positions [axes, *shape]: consecutive on the first axis, rows and columns of a picture on the others."""
    N = shape[-1]
    t = torch.arange(N, device=DEV, dtype=torch.int32)
    start = torch.randint(0, case["far"] + 64, shape[:-1] + (1,), generator=g, device=DEV, dtype=torch.int32)
    side = max(1, math.isqrt(N))
    every = [t.expand(shape) + start, (t // side).expand(shape) + start // 7, (t % side).expand(shape) + start // 9]
    return torch.stack(every[: case["axes"]]).contiguous()


def _tables(lens, page, g, width, spare):
    """Pages of sequences of `lens` tokens out of a shuffled pool with `spare` more: (table [B, width], the pages left,
    how many the pool has).  Entries past a sequence's pages are 0."""
    need = [-(-n // page) for n in lens]
    total = max(1, sum(need) + spare)
    order = torch.randperm(total, generator=g, device=DEV).to(torch.int32)
    starts = [0]
    for n in need:
        starts.append(starts[-1] + n)
    at = torch.tensor(starts[:-1], device=DEV)[:, None] + torch.arange(width, device=DEV)[None, :]
    used = torch.arange(width, device=DEV)[None, :] < torch.tensor(need, device=DEV)[:, None]
    table = torch.where(used, order[at.clamp(max=total - 1)], 0).to(torch.int32)
    return table.contiguous(), order[starts[-1]:].contiguous(), total


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    s = {"op": op, "case": case}
    if op == "slots":
        ctx, new = _lengths(case)
        page = case["page"]
        ctx = [max(0, c - int(torch.randint(0, 3, (1,), generator=torch.Generator().manual_seed(seed)))) for c in ctx]
        extra = sum(-(-(c + n) // page) - -(-c // page) for c, n in zip(ctx, new))
        width = max(1, max(-(-(c + n) // page) for c, n in zip(ctx, new)))
        s["table"], free, _ = _tables(ctx, page, g, width, extra + 7)
        s["free"], s["count"] = free, _int32([free.numel()])
        s["ctx"], s["new"] = _int32(ctx), _int32(new)
        s["T"] = sum(new) + case["pad"]
        return s
    H, Hkv, d = case["H"], case["Hkv"], case["d"]
    if op == "norm":
        dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
        B, N = case["B"], case["N"]
        s["wq"], s["wk"] = (1 + _randn((d,), g, torch.float32, 0.2)).to(dt), (1 + _randn((d,), g, torch.float32, 0.2)).to(dt)
        s["freqs"], s["axes"] = _rotation(case)
        if case["way"] == "append":
            qkv = _randn((N, H + 2 * Hkv, d), g, mult=2.0)  # one projection's output
            s["q"], s["k"], s["v"] = qkv[:, :H], qkv[:, H:H + Hkv], qkv[:, H + Hkv:]
            page = case["page"]
            pages = -(-N // page) + 3
            s["kc"], s["vc"] = _randn((pages, Hkv, page, d), g), _randn((pages, Hkv, page, d), g)
            s["n"] = N - case["pad"]  # the places behind the last token are unused
            slots = torch.randperm(pages * page, generator=g, device=DEV)[:N]
            slots[s["n"]:] = -1
            s["slots"] = slots.contiguous()
            s["pos"] = _positions(case, (N,), g)
            return s
        # heads of a projection's output [B, N, heads, d]; their sizes differ from token to token
        size = torch.exp(torch.randn((B, N, 1, 1), generator=g, device=DEV))
        s["q"] = (torch.randn((B, N, H, d), generator=g, device=DEV) * size).to(dt).transpose(1, 2)
        s["k"] = (torch.randn((B, N, Hkv, d), generator=g, device=DEV) * size).to(dt).transpose(1, 2)
        s["pos"] = _positions(case, (B, N), g)
        if case["way"] == "backward":  # gradients as the attention's backward leaves them
            s["dq"], s["dk"] = _randn((B, H, N, d), g, dt), _randn((B, Hkv, N, d), g, dt)
        return s
    ctx, new = _lengths(case)
    lens = [c + n for c, n in zip(ctx, new)]
    width = max(1, max(-(-n // case["page"]) for n in lens))
    s["table"], _, pages = _tables(lens, case["page"], g, width, 0)
    s["lens"] = _int32(lens)
    s["cu"] = _int32([sum(new[:b]) for b in range(len(new) + 1)])
    s["new_hi"] = max(new)
    s["q"] = _randn((sum(new), H, d), g, mult=1.5)
    s["kc"], s["vc"] = _randn((pages, Hkv, case["page"], d), g), _randn((pages, Hkv, case["page"], d), g)
    return s


# ------------------------------------------------------------------------------------------ one pass

EPS = 1e-6


def _plain_slots(s):
    page, T, table = s["case"]["page"], s["T"], s["table"]
    ctx, new = s["ctx"].long(), s["new"].long()
    ends = new.cumsum(0)
    cu = torch.cat((ends.new_zeros(1), ends))
    t = torch.arange(T, device=DEV)
    used = t < ends[-1]
    b = torch.searchsorted(ends, t, right=True).clamp(max=ends.numel() - 1)
    pos = torch.where(used, ctx[b] + t - cu[b], 0)
    held = (ctx + page - 1) // page
    take = (ctx + new + page - 1) // page - held  # new pages of each sequence, dealt from the top of the free ones
    before = take.cumsum(0) - take
    at = torch.arange(table.shape[1], device=DEV)
    fresh = (at >= held[:, None]) & (at < (held + take)[:, None])
    order = s["count"].long() - 1 - (before[:, None] + at - held[:, None])
    table.copy_(torch.where(fresh, s["free"][order.clamp(0, s["free"].numel() - 1)], table))
    slots = torch.where(used, table[b, (pos // page).clamp(max=table.shape[1] - 1)].long() * page + pos % page, -1)
    return (cu.int(), pos.int(), slots, (ctx + new).int(), s["count"] - take.sum().int(), table)


def _rotate(f, cos, sin, rot, interleaved):
    """Rotates the first `rot` elements of f's last axis, in fp32."""
    if interleaved:
        a, b = f[..., 0:rot:2], f[..., 1:rot:2]
        turned = torch.stack((a * cos - b * sin, a * sin + b * cos), -1).flatten(-2)
    else:
        a, b = f[..., : rot // 2], f[..., rot // 2: rot]
        turned = torch.cat((a * cos - b * sin, a * sin + b * cos), -1)
    return torch.cat((turned, f[..., rot:]), -1)


def _angles(s):
    """cos and sin [..., rot / 2] in fp32 of angles formed in float64 (fp32 would lose far positions)."""
    phi = s["pos"][s["axes"].long()].double().movedim(0, -1) * s["freqs"]
    return phi.cos().float(), phi.sin().float()


def _unit(x):
    """x in fp32 over its root mean square, and what it was multiplied by."""
    f = x.float()
    r = torch.rsqrt((f * f).mean(-1, keepdim=True) + EPS)
    return f * r, r


def _plain_norm(s):
    c = s["case"]
    cos, sin = (x[:, None] for x in _angles(s))
    turn = (c["rot"], c["interleaved"])
    if c["way"] == "backward":
        out, grads = [], []
        for dy, x, w in ((s["dq"], s["q"], s["wq"]), (s["dk"], s["k"], s["wk"])):
            g = _rotate(dy.float(), cos, -sin, *turn)
            u, r = _unit(x)
            wg = g * w.float()
            out.append((r * (wg - u * (wg * u).mean(-1, keepdim=True))).to(x.dtype).contiguous())
            grads.append((g * u).sum((0, 1, 2), dtype=torch.float64).float())
        return (*out, *grads)
    q, k = (_rotate(_unit(s[n])[0] * s["w" + n].float(), cos, sin, *turn).to(s[n].dtype).contiguous() for n in "qk")
    if c["way"] == "forward":
        return q, k
    n = s["n"]
    at, row = s["slots"][:n] // c["page"], s["slots"][:n] % c["page"]
    s["kc"][at, :, row] = k[:n]
    s["vc"][at, :, row] = s["v"][:n]
    return q, s["kc"], s["vc"]


def _gather(cache, table):
    """[B, pages] -> fp32 [B, Hkv, pages * page, d]: the rows a table names, in order."""
    return cache[table.long()].permute(0, 2, 1, 3, 4).flatten(2, 3).float()


def _plain_chunk(s):
    """Attention of all sequences at once, padded to the longest; the padding's rows are left out at the end."""
    c = s["case"]
    B, H, Hkv, d = c["B"], c["H"], c["Hkv"], c["d"]
    G, M = H // Hkv, s["new_hi"]
    cu, lens = s["cu"].long(), s["lens"].long()
    new = cu[1:] - cu[:-1]
    i = torch.arange(M, device=DEV)
    real = i < new[:, None]  # [B, M]
    q = s["q"][(cu[:-1, None] + i).clamp(max=s["q"].shape[0] - 1)].float()  # [B, M, H, d]
    q = q.view(B, M, Hkv, G, d).permute(0, 2, 3, 1, 4).reshape(B, Hkv, G * M, d)
    k, v = _gather(s["kc"], s["table"]), _gather(s["vc"], s["table"])
    N = k.shape[2]
    sc = torch.matmul(q, k.transpose(2, 3)).view(B, Hkv, G, M, N).mul_(1.0 / math.sqrt(d))
    at = torch.arange(N, device=DEV)
    last = ((lens - new)[:, None] + i)[..., None]  # the token's own position: the last key it sees
    seen = (at <= last) & (at < lens[:, None, None]) & real[..., None]
    if c["window"]:
        seen &= (at > last - c["window"]) | (at < c["sinks"])
    sc.masked_fill_(~seen[:, None, None], -math.inf)
    top = sc.amax(-1, keepdim=True)
    some = top > -math.inf
    p = sc.sub_(torch.where(some, top, 0.0)).exp_()
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(B, Hkv, G * M, N), v).view(B, Hkv, G, M, d) / torch.where(some, total, 1.0)
    lse = torch.where(some, top + total.log(), -math.inf)
    o, lse = (x.permute(0, 3, 1, 2, 4).reshape(B, M, H, -1)[real] for x in (o, lse))
    return o.to(s["q"].dtype), lse[..., 0].contiguous()


def _own(s):
    import attention_forward_05_gb300 as fa

    c = s["case"]
    if s["op"] == "slots":
        return (*fa.fa_paged_slots(s["ctx"], s["new"], s["table"], s["free"], s["count"], c["page"], s["T"]), s["table"])
    if s["op"] == "norm":
        how = {"axes": s["axes"], "interleaved": c["interleaved"], "eps": EPS}
        if c["way"] == "forward":
            return fa.fa_norm_rope(s["q"], s["k"], s["wq"], s["wk"], s["pos"], s["freqs"], **how)
        if c["way"] == "backward":
            return fa.fa_norm_rope_bwd(s["dq"], s["dk"], s["q"], s["k"], s["wq"], s["wk"], s["pos"], s["freqs"], **how)
        q = fa.fa_paged_append(s["k"], s["v"], s["kc"], s["vc"], s["slots"], q=s["q"], positions=s["pos"],
                               freqs=s["freqs"], q_weight=s["wq"], k_weight=s["wk"], **how)
        return q, s["kc"], s["vc"]
    return fa.fa_fwd_paged(s["q"], s["kc"], s["vc"], s["table"], s["cu"], s["lens"], window=c["window"],
                           sinks=c["sinks"], with_lse=True)


def run(state):
    if own:
        return _own(state)
    if state["op"] == "slots":
        return _plain_slots(state)
    return _plain_norm(state) if state["op"] == "norm" else _plain_chunk(state)


# ------------------------------------------------------------------------------------------ what it takes

def _spans(case):
    """For each sequence (first key that a token of the chunk sees in its window, keys, pairs of token and key)."""
    out = []
    w, s = case["window"], case["sinks"]
    for c, n in zip(*_lengths(case)):
        if not w:
            out.append((0, c + n, n * c + n * (n + 1) // 2))
            continue
        first = max(0, c - w + 1)
        pairs = sum(min(p + 1, w) + min(s, max(0, p + 1 - w)) for p in range(c, c + n))
        out.append((first, c + n - first + min(s, first), pairs))
    return out


def work(case):
    if case["op"] == "slots":
        ctx, new = _lengths(case)
        pages = sum(-(-(c + n) // case["page"]) - -(-c // case["page"]) for c, n in zip(ctx, new))
        return {"bytes": 16 * case["B"] + 12 * (sum(new) + case["pad"]) + 8 * pages + 12, "flops": 0}
    H, Hkv, d = case["H"], case["Hkv"], case["d"]
    if case["op"] == "norm":
        n = case["B"] * case["N"]
        e = 2 if case["dtype"] == "bf16" else 4
        pos = 4 * case["axes"] * n
        if case["way"] == "append":
            stored = n - case["pad"]
            return {"bytes": 4 * d * (n * H + 2 * stored * Hkv) + 8 * n + pos, "flops": 8 * d * (n * H + stored * Hkv)}
        if case["way"] == "backward":
            return {"bytes": 3 * n * (H + Hkv) * d * e + pos + 8 * d, "flops": 16 * n * (H + Hkv) * d}
        return {"bytes": 2 * n * (H + Hkv) * d * e + pos, "flops": 8 * n * (H + Hkv) * d}
    spans, T = _spans(case), sum(_lengths(case)[1])
    keys, pairs = sum(s[1] for s in spans), sum(s[2] for s in spans)
    return {"bytes": 4 * keys * Hkv * d + 4 * T * H * d + 4 * T * H + 8 * case["B"] + 4 * keys // case["page"],
            "flops": 4 * H * d * pairs}


# ------------------------------------------------------------------------------------------ in 64 bits

def _exact_turn(x, pos, s, c):
    """x [..., heads, d] (float64) and pos [axes, ...] (one entry a row of heads): each pair as a complex number, turned."""
    n = c["rot"] // 2
    which = s["axes"].long()
    phi = torch.stack([pos[which[i]].double() * s["freqs"][i] for i in range(n)], -1)[..., None, :]
    turn = torch.polar(torch.ones_like(phi), phi)
    if c["interleaved"]:
        pairs = x[..., : 2 * n].unflatten(-1, (n, 2))
    else:
        pairs = x[..., : 2 * n].unflatten(-1, (2, n)).transpose(-1, -2)
    y = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turn)
    y = y.flatten(-2) if c["interleaved"] else y.transpose(-1, -2).flatten(-2)
    return torch.cat((y, x[..., 2 * n:]), -1)


def _exact_norm_turn(x, w, pos, s, c):
    """x [..., heads, d] in float64."""
    return _exact_turn(x / torch.sqrt(x.square().sum(-1, keepdim=True) / c["d"] + EPS) * w, pos, s, c)


def _exact_norm(c, s):
    if c["way"] == "append":
        q, k = (_exact_norm_turn(s[n].double(), s["w" + n].double(), s["pos"], s, c) for n in "qk")
        kc, vc = s["kc"].double(), s["vc"].double()
        flat_k = kc.permute(0, 2, 1, 3).reshape(-1, c["Hkv"], c["d"])
        flat_v = vc.permute(0, 2, 1, 3).reshape(-1, c["Hkv"], c["d"])
        put = s["slots"][: s["n"]]
        flat_k[put], flat_v[put] = k[: s["n"]], s["v"][: s["n"]].double()
        back = [f.view(kc.shape[0], c["page"], c["Hkv"], c["d"]).permute(0, 2, 1, 3).contiguous()
                for f in (flat_k, flat_v)]
        return q, back[0], back[1]
    outs, grads = [], []
    for n in "qk":
        x = s[n].transpose(1, 2).double().requires_grad_(c["way"] == "backward")
        w = s["w" + n].double().requires_grad_(c["way"] == "backward")
        y = _exact_norm_turn(x, w, s["pos"], s, c)
        if c["way"] == "backward":  # the definition's own derivative
            dx, dw = torch.autograd.grad(y, (x, w), s["d" + n].transpose(1, 2).double())
            outs.append(dx.transpose(1, 2).contiguous())
            grads.append(dw)
        else:
            outs.append(y.transpose(1, 2).contiguous())
    return (*outs, *grads)


def _exact_slots(c, s):
    """One sequence at a time."""
    page, T = c["page"], s["T"]
    table, free, top = s["table"].tolist(), s["free"].tolist(), s["count"].item()
    cu, pos, slots, lens = [0], [], [], []
    for b, (held, n) in enumerate(zip(s["ctx"].tolist(), s["new"].tolist())):
        for p in range(held, held + n):
            if p % page == 0:
                top -= 1
                table[b][p // page] = free[top]
            pos.append(p)
            slots.append(table[b][p // page] * page + p % page)
        cu.append(cu[-1] + n)
        lens.append(held + n)
    pad = T - len(pos)
    return (_int32(cu), _int32(pos + [0] * pad), torch.tensor(slots + [-1] * pad, device=DEV), _int32(lens),
            _int32([top]), _int32(table))


def exact(case, seed):
    s = prepare(case, seed)
    c = case
    if c["op"] == "slots":
        return _exact_slots(c, s)
    if c["op"] == "norm":
        return _exact_norm(c, s)
    ctx, new = _lengths(c)
    G, page = c["H"] // c["Hkv"], c["page"]
    o = torch.zeros(sum(new), c["H"], c["d"], dtype=torch.float64, device=DEV)
    lse = torch.full((sum(new), c["H"]), -math.inf, dtype=torch.float64, device=DEV)
    first = 0
    for b, (held, n) in enumerate(zip(ctx, new)):
        if n == 0:
            continue
        at = torch.arange(held + n, device=DEV)
        rows = s["table"][b].long()[at // page], at % page
        p = torch.arange(held, held + n, device=DEV)[:, None]
        hidden = at > p
        if c["window"]:
            hidden |= (at <= p - c["window"]) & (at >= c["sinks"])
        for h in range(c["Hkv"]):
            k, v = (x[rows[0], h, rows[1]].double() for x in (s["kc"], s["vc"]))
            for g in range(h * G, (h + 1) * G):
                t = (s["q"][first:first + n, g].double() @ k.T / math.sqrt(c["d"])).masked_fill(hidden, -math.inf)
                total = torch.logsumexp(t, -1)
                o[first:first + n, g] = torch.exp(t - total[:, None]) @ v
                lse[first:first + n, g] = total
        first += n
    return o, lse
