"""The position, cache and paged-decode operators: what is measured of them.

Four operators that a training or serving program runs around attention:

  rope    rotary positions with one or several axes on q and k (forward, and backward on their gradients)
  append  keys and values of new tokens into a paged cache, keys (and queries) rotated on the way
  decode  one query per head for every sequence of a ragged batch, over the paged cache
  prefix  the same when all sequences begin with one shared prefix

``run`` computes them in plain torch operations (``own`` false) or calls the framework (``own`` true);
``exact`` computes them from their definitions in float64.
"""
import math
import random

import torch

own = False

DEV = "cuda"


# ------------------------------------------------------------------------------------------ cases

def _rope(name, B, H, Hkv, N, d, dtype, axes, interleaved, backward, rot=None, far=0):
    return {"name": name, "op": "rope", "B": B, "H": H, "Hkv": Hkv, "N": N, "d": d, "rot": rot or d, "dtype": dtype,
            "axes": axes, "interleaved": interleaved, "backward": backward, "far": far}


def _append(name, T, pad, H, Hkv, d, page, axes, interleaved, rot=None, far=0):
    return {"name": name, "op": "append", "T": T, "pad": pad, "H": H, "Hkv": Hkv, "d": d, "rot": rot or d,
            "page": page, "axes": axes, "interleaved": interleaved, "far": far}


def _decode(name, B, H, Hkv, d, page, longest, shortest, lens_seed=1):
    return {"name": name, "op": "decode", "B": B, "H": H, "Hkv": Hkv, "d": d, "page": page, "longest": longest,
            "shortest": shortest, "lens_seed": lens_seed}


def _prefix(name, B, H, Hkv, d, page, prefix, longest, shortest, lens_seed=1):
    return {"name": name, "op": "prefix", "B": B, "H": H, "Hkv": Hkv, "d": d, "page": page, "prefix": prefix,
            "longest": longest, "shortest": shortest, "lens_seed": lens_seed}


def listed():
    return [
        # one short clip of video patches in fp32: three position axes, an odd number of tokens
        _rope("rope small clip fp32", 1, 16, 4, 333, 64, "fp32", 3, False, False),
        # the multi-head prefill workload's q and k, text positions far into a long document
        _rope("rope train bf16", 4, 16, 16, 4096, 64, "bf16", 1, False, False, far=900_000),
        # gradients of q and k for long image sequences, grouped heads, adjacent pairs
        _rope("rope image backward", 2, 16, 4, 8192, 128, "bf16", 3, True, True),
        # one sequence generating one token
        _append("append one token", 1, 0, 32, 8, 128, 16, 1, False, far=30_000),
        # a decode batch with unused places at its end, part of each head rotated
        _append("append decode batch", 237, 19, 32, 8, 64, 16, 1, False, rot=32, far=30_000),
        # a long prompt with images, cut from one projection's output
        _append("append long prompt", 8191, 0, 32, 8, 128, 64, 3, True),
        # one user, a short context: latency counts
        _decode("decode one short", 1, 32, 8, 128, 16, 777, 777),
        # a serving batch: a few long contexts, many short ones, one empty
        _decode("decode ragged batch", 61, 32, 4, 128, 16, 32768, 0),
        # the split-KV decode workload's batch and length with grouped heads
        _decode("decode full batch", 32, 32, 8, 64, 64, 32768, 32768),
        # a handful of continuations of one question
        _prefix("prefix few", 5, 16, 2, 64, 16, 1000, 100, 0),
        # a batch on one system prompt
        _prefix("prefix batch", 32, 32, 8, 64, 64, 8192, 300, 1),
        # many short answers on one long document: bound by the matrix products
        _prefix("prefix large", 256, 32, 8, 128, 16, 16384, 600, 1),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "append", "decode", "prefix"])
    d = rng.choice([64, 128])
    Hkv = rng.choice([1, 2, 4, 8])
    H = Hkv * rng.choice([1, 2, 3, 4, 8])
    # no drawn case costs more than the largest listed one of its operator: the last size drawn is cut to that
    if op == "rope":
        B, dtype = rng.randint(1, 4), rng.choice(["bf16", "bf16", "fp32"])
        most = 2 * 20 * 8192 * 128 * (2 if dtype == "bf16" else 1) // (2 * B * (H + Hkv) * d)
        c = _rope("", B, H, Hkv, _log(rng, 16, min(8192, most)), d, dtype, rng.choice([1, 2, 3]),
                  rng.random() < 0.4, rng.random() < 0.5, rot=rng.choice([d, d, 32]), far=rng.choice([0, 100_000]))
    elif op == "append":
        T = _log(rng, 1, min(8191, 8191 * 48 * 128 // ((H + 2 * Hkv) * d)))
        c = _append("", T, rng.randint(0, T // 8), H, Hkv, d, rng.choice([16, 32, 64, 24]), rng.choice([1, 1, 3]),
                    rng.random() < 0.4, rot=rng.choice([d, d, 32]), far=rng.choice([0, 100_000]))
    elif op == "decode":
        B = _log(rng, 1, 96)
        longest = _log(rng, 64, min(32768, 32 * 32768 * 8 * 64 // (B * Hkv * d)))
        c = _decode("", B, H, Hkv, d, rng.choice([16, 32, 64, 24, 128]), longest,
                    rng.choice([0, 1, longest // 2, longest]), lens_seed=rng.randint(1, 1 << 30))
    else:
        B = _log(rng, 2, 256)
        longest = _log(rng, 16, 600)
        prefix = _log(rng, 200, min(16384, 256 * 16384 * 32 * 128 // (B * H * d)))
        c = _prefix("", B, H, Hkv, d, rng.choice([16, 32, 64, 24]), prefix, longest,
                    rng.choice([0, 1, longest // 2]), lens_seed=rng.randint(1, 1 << 30))
    del c["name"]
    return c


def _lengths(case):
    """Own lengths of the case's sequences: spread over their logarithm, the longest and the shortest among them."""
    rng = random.Random(case["lens_seed"])
    lo, hi = case["shortest"], case["longest"]
    lens = [min(hi, max(lo, _log(rng, max(lo, 1), hi))) for _ in range(case["B"])]
    lens[0] = hi
    if case["B"] > 1:
        lens[-1] = lo
    return lens


# ------------------------------------------------------------------------------------------ inputs

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _randn(shape, g, dtype=torch.bfloat16, mult=1.0):
    return (torch.randn(shape, generator=g, device=DEV) * mult).to(dtype)


def _rotation(case):
    """Frequencies (radians a position, float64) and the axis of each pair: thirds (or halves) of the pairs in turn."""
    n = case["rot"] // 2
    freqs = torch.tensor([10000.0 ** (-i / n) for i in range(n)], dtype=torch.float64, device=DEV)
    axes = torch.tensor([i * case["axes"] // n for i in range(n)], dtype=torch.int32, device=DEV)
    return freqs, axes


def _positions(case, shape, g):
    """int32 positions [axes, *shape]: consecutive on the first axis, rows and columns of a picture on the others."""
    N = shape[-1]
    t = torch.arange(N, device=DEV, dtype=torch.int32)
    start = torch.randint(0, case["far"] + 64, shape[:-1] + (1,), generator=g, device=DEV, dtype=torch.int32)
    side = max(1, math.isqrt(N))
    every = [t.expand(shape) + start, (t // side).expand(shape) + start // 7, (t % side).expand(shape) + start // 9]
    return torch.stack(every[: case["axes"]]).contiguous()


def _tables(case, lens, g, extra=0):
    """A page table [B, most pages a sequence has] over shuffled pages, the pages of `extra` shared tokens, and how many
    pages the cache has."""
    page = case["page"]
    need = [-(-n // page) for n in lens]
    shared = -(-extra // page)
    total = sum(need) + shared
    order = torch.randperm(max(total, 1), generator=g, device=DEV).to(torch.int32)
    width = max(1, max(need))
    starts = [0]
    for n in need:
        starts.append(starts[-1] + n)
    at = torch.tensor(starts[:-1], device=DEV)[:, None] + torch.arange(width, device=DEV)[None, :]
    count = torch.tensor(need, device=DEV)[:, None]
    used = torch.arange(width, device=DEV)[None, :] < count
    table = torch.where(used, order[at.clamp(max=max(total, 1) - 1)], 0).to(torch.int32)
    return table.contiguous(), order[sum(need):sum(need) + shared].contiguous(), max(total, 1)


def prepare(case, seed):
    g = _gen(seed)
    op, H, Hkv, d = case["op"], case["H"], case["Hkv"], case["d"]
    s = {"op": op, "case": case}
    if op == "rope":
        dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
        B, N = case["B"], case["N"]
        if case["backward"]:  # gradients as the attention's backward leaves them
            s["q"], s["k"] = _randn((B, H, N, d), g, dt), _randn((B, Hkv, N, d), g, dt)
        else:  # heads of a projection's output [B, N, heads, d]
            s["q"] = _randn((B, N, H, d), g, dt).transpose(1, 2)
            s["k"] = _randn((B, N, Hkv, d), g, dt).transpose(1, 2)
        s["freqs"], s["axes"] = _rotation(case)
        s["pos"] = _positions(case, (B, N), g)
    elif op == "append":
        T, page = case["T"], case["page"]
        qkv = _randn((T, H + 2 * Hkv, d), g)  # one projection's output
        s["q"], s["k"], s["v"] = qkv[:, :H], qkv[:, H:H + Hkv], qkv[:, H + Hkv:]
        pages = -(-T // page) + 3
        s["kc"], s["vc"] = _randn((pages, Hkv, page, d), g), _randn((pages, Hkv, page, d), g)
        s["n"] = T - case["pad"]  # the places behind the last token are unused
        slots = torch.randperm(pages * page, generator=g, device=DEV)[:T]
        if T > 300:  # a prompt: whole pages in turn
            at = torch.arange(T, device=DEV)
            slots = torch.randperm(pages, generator=g, device=DEV)[at // page] * page + at % page
        slots[s["n"]:] = -1
        s["slots"] = slots.contiguous()
        s["freqs"], s["axes"] = _rotation(case)
        s["pos"] = _positions(case, (T,), g)
    else:
        lens = _lengths(case)
        table, shared, pages = _tables(case, lens, g, case.get("prefix", 0))
        s["table"], s["shared"] = table, shared
        s["lens"] = torch.tensor(lens, dtype=torch.int32, device=DEV)
        s["q"] = _randn((case["B"], H, d), g, mult=1.5)
        s["kc"], s["vc"] = _randn((pages, Hkv, case["page"], d), g), _randn((pages, Hkv, case["page"], d), g)
    return s


# ------------------------------------------------------------------------------------------ one pass

def _rotate(x, cos, sin, rot, interleaved):
    """Rotates the first `rot` elements of x's last axis in fp32 and rounds once to x's type."""
    f = x.float()
    if interleaved:
        a, b = f[..., 0:rot:2], f[..., 1:rot:2]
        turned = torch.stack((a * cos - b * sin, a * sin + b * cos), -1).flatten(-2)
    else:
        a, b = f[..., : rot // 2], f[..., rot // 2: rot]
        turned = torch.cat((a * cos - b * sin, a * sin + b * cos), -1)
    return torch.cat((turned, f[..., rot:]), -1).to(x.dtype)


def _angles(s):
    """cos and sin [..., rot / 2] in fp32 of angles formed in float64 (fp32 would lose far positions)."""
    phi = s["pos"][s["axes"].long()].double().movedim(0, -1) * s["freqs"]
    return phi.cos().float(), phi.sin().float()


def _gather(cache, table, page):
    """[B, pages] -> fp32 [B, Hkv, pages * page, d]: the rows a table names, in order."""
    x = cache[table.long()]  # [B, pages, Hkv, page, d]
    return x.permute(0, 2, 1, 3, 4).flatten(2, 3).float()


def _attend(q, k, v, seen):
    """softmax(q k^T / sqrt(d)) v and its log-sum-exp; q [B,H,d] bf16, k/v fp32 [B,Hkv,N,d], seen [B,N] truth values."""
    B, H, d = q.shape
    Hkv = k.shape[1]
    sc = torch.matmul(q.float().view(B, Hkv, H // Hkv, d), k.transpose(2, 3)) * (1.0 / math.sqrt(d))
    sc = sc.masked_fill(~seen[:, None, None, :], -math.inf)
    top = sc.amax(-1, keepdim=True)
    some = top > -math.inf
    p = torch.exp(sc - torch.where(some, top, 0.0))
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p, v) / torch.where(some, total, 1.0)
    lse = torch.where(some, top + total.log(), -math.inf)
    return o.reshape(B, H, d).to(q.dtype), lse.reshape(B, H)


def _plain(s):
    c = s["case"]
    if s["op"] == "rope":
        cos, sin = _angles(s)
        if c["backward"]:
            sin = -sin
        cos, sin = cos[:, None], sin[:, None]
        return (_rotate(s["q"], cos, sin, c["rot"], c["interleaved"]).contiguous(),
                _rotate(s["k"], cos, sin, c["rot"], c["interleaved"]).contiguous())
    if s["op"] == "append":
        cos, sin = _angles(s)
        cos, sin = cos[:, None], sin[:, None]
        n = s["n"]
        at, row = s["slots"][:n] // c["page"], s["slots"][:n] % c["page"]
        s["kc"][at, :, row] = _rotate(s["k"], cos, sin, c["rot"], c["interleaved"])[:n]
        s["vc"][at, :, row] = s["v"][:n]
        return _rotate(s["q"], cos, sin, c["rot"], c["interleaved"]), s["kc"], s["vc"]
    table, lens, first = s["table"], s["lens"], 0
    if s["op"] == "prefix":
        table = torch.cat((s["shared"].expand(c["B"], -1), table), 1)
        first = s["shared"].numel() * c["page"]
    at = torch.arange(table.shape[1] * c["page"], device=DEV)
    seen = (at >= first) & (at - first < lens[:, None])
    if s["op"] == "prefix":
        seen = seen | (at < c["prefix"])
    return _attend(s["q"], _gather(s["kc"], table, c["page"]), _gather(s["vc"], table, c["page"]), seen)


def _own(s):
    import attention_forward_05_gb300 as fa

    c = s["case"]
    if s["op"] == "rope":
        call = fa.fa_rope_bwd if c["backward"] else fa.fa_rope
        return call(s["q"], s["k"], s["pos"], s["freqs"], axes=s["axes"], interleaved=c["interleaved"])
    if s["op"] == "append":
        q = fa.fa_paged_append(s["k"], s["v"], s["kc"], s["vc"], s["slots"], q=s["q"], positions=s["pos"],
                               freqs=s["freqs"], axes=s["axes"], interleaved=c["interleaved"])
        return q, s["kc"], s["vc"]
    if s["op"] == "decode":
        return fa.fa_decode_paged(s["q"], s["kc"], s["vc"], s["table"], s["lens"], with_lse=True)
    return fa.fa_decode_paged_prefix(s["q"], s["kc"], s["vc"], s["shared"], c["prefix"], s["table"], s["lens"],
                                     with_lse=True)


def run(state):
    if own:
        return _own(state)
    return _plain(state)


# ------------------------------------------------------------------------------------------ what it takes

def work(case):
    H, Hkv, d = case["H"], case["Hkv"], case["d"]
    if case["op"] == "rope":
        n = case["B"] * case["N"]
        e = 2 if case["dtype"] == "bf16" else 4
        return {"bytes": 2 * n * (H + Hkv) * d * e + 4 * case["axes"] * n, "flops": 3 * n * (H + Hkv) * case["rot"]}
    if case["op"] == "append":
        T, n = case["T"], case["T"] - case["pad"]
        return {"bytes": 4 * d * (T * H + 2 * n * Hkv) + (8 + 4 * case["axes"]) * T,
                "flops": 3 * case["rot"] * (T * H + n * Hkv)}
    lens = _lengths(case)
    own_keys, P = sum(lens), case.get("prefix", 0)
    small = 4 * case["B"] * H * d + 4 * case["B"] * H + 4 * case["B"] + 4 * (own_keys + P) // case["page"]
    return {"bytes": 4 * (own_keys + P) * Hkv * d + small, "flops": 4 * H * d * (own_keys + case["B"] * P)}


# ------------------------------------------------------------------------------------------ in 64 bits

def _exact_turn(x, pos, s, c, sign):
    """x [..., heads, d] and pos [axes, ...] (one entry a row of heads): each pair as a complex number, turned."""
    z = x.double()
    n = c["rot"] // 2
    which = s["axes"].long()
    phi = sign * torch.stack([pos[which[i]].double() * s["freqs"][i] for i in range(n)], -1)[..., None, :]
    turn = torch.polar(torch.ones_like(phi), phi)
    out = z.clone()
    if c["interleaved"]:
        first, second = torch.arange(0, 2 * n, 2, device=DEV), torch.arange(1, 2 * n, 2, device=DEV)
    else:
        first, second = torch.arange(n, device=DEV), torch.arange(n, 2 * n, device=DEV)
    w = torch.complex(z[..., first], z[..., second]) * turn
    out[..., first], out[..., second] = w.real, w.imag
    return out


def exact(case, seed):
    s = prepare(case, seed)
    c = case
    if c["op"] == "rope":
        sign = -1.0 if c["backward"] else 1.0
        return tuple(_exact_turn(x.transpose(1, 2), s["pos"], s, c, sign).transpose(1, 2).contiguous()
                     for x in (s["q"], s["k"]))
    if c["op"] == "append":
        kc, vc = s["kc"].double(), s["vc"].double()
        k = _exact_turn(s["k"], s["pos"], s, c, 1.0)
        flat_k = kc.permute(0, 2, 1, 3).reshape(-1, c["Hkv"], c["d"])
        flat_v = vc.permute(0, 2, 1, 3).reshape(-1, c["Hkv"], c["d"])
        put = s["slots"][: s["n"]]
        flat_k[put], flat_v[put] = k[: s["n"]], s["v"][: s["n"]].double()
        back = [f.view(kc.shape[0], c["page"], c["Hkv"], c["d"]).permute(0, 2, 1, 3).contiguous()
                for f in (flat_k, flat_v)]
        return _exact_turn(s["q"], s["pos"], s, c, 1.0), back[0], back[1]
    lens, G = _lengths(c), c["H"] // c["Hkv"]
    o = torch.zeros(c["B"], c["H"], c["d"], dtype=torch.float64, device=DEV)
    lse = torch.full((c["B"], c["H"]), -math.inf, dtype=torch.float64, device=DEV)

    def rows(cache, pages, n):  # the first n rows of some pages: [Hkv, n, d]
        return cache[pages.long()].transpose(0, 1).flatten(1, 2)[:, :n].double()

    P = c.get("prefix", 0)
    shared = [rows(x, s["shared"], P) for x in (s["kc"], s["vc"])]
    for b, n in enumerate(lens):
        if n + P == 0:
            continue
        pages = s["table"][b, : -(-n // c["page"])]
        k, v = (torch.cat((p, rows(x, pages, n)), 1) for p, x in zip(shared, (s["kc"], s["vc"])))
        t = torch.einsum("hgd,hnd->hgn", s["q"][b].double().view(c["Hkv"], G, c["d"]), k) / math.sqrt(c["d"])
        total = torch.logsumexp(t, -1)
        o[b] = torch.einsum("hgn,hnd->hgd", torch.exp(t - total[..., None]), v).reshape(c["H"], c["d"])
        lse[b] = total.reshape(-1)
    return o, lse
