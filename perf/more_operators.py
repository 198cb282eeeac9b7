"""More operators of a target pass and of what follows its verification, in plain form and as the library's calls.

  rope     rotary positions of new tokens' queries: pairs (i, i + rot/2) or (2i, 2i + 1) of a part of each head,
           turned by position times frequency, the frequencies scaled for long contexts;
  kv       the new tokens' keys rotated and written, with their values, into a paged cache (bf16, or e4m3 bytes
           with a power-of-two scale per token and head), their queries rotated in the same call; after
           verification the accepted path's keys again (`path`);
  put      new tokens of a latent cache: one vector of C elements a token that all heads share, and R rotary
           elements, rotated on the way;
  latent   the new tokens' attention over a latent cache: keys are a position's C + R elements, values its C;
           every head's query comes with its key projection multiplied in;
  logp     after verification, of each emitted token: its log probability and rank under the target's row, the
           row's entropy and its most likely tokens.

A case is one pass of one of them.  Sequence lengths are ragged: the longest is `L`, the shortest about L / 2.
"""
import math
import random

import torch

own = False

E4M3_MAX = 448.0
ORIGINAL = 8192  # context that scaled frequencies were made for
BASE = 10000.0


# ------------------------------------------------------------------ cases

def _rope(name, B, N, H, D, rot, first, inter, scaling, far, dtype):
    return {"name": name, "kind": "rope", "B": B, "N": N, "H": H, "D": D, "rot": rot, "first": first,
            "interleaved": inter, "scaling": scaling, "far": far, "dtype": dtype}


def _kv(name, B, N, Hq, Hkv, D, rot, inter, scaling, page, L, cache, path=0):
    return {"name": name, "kind": "kv", "B": B, "N": N, "Hq": Hq, "Hkv": Hkv, "D": D, "rot": rot,
            "interleaved": inter, "scaling": scaling, "page": page, "L": L, "cache": cache, "path": path}


def _put(name, B, N, C, page, L, scaling, path=0):
    return {"name": name, "kind": "put", "B": B, "N": N, "C": C, "page": page, "L": L, "interleaved": True,
            "scaling": scaling, "path": path}


def _latent(name, B, N, H, C, page, L, tree=0):
    return {"name": name, "kind": "latent", "B": B, "N": N, "H": H, "C": C, "page": page, "L": L, "tree": tree}


def _logp(name, B, M, V, dtype, top, T, nodes=0):
    return {"name": name, "kind": "logp", "B": B, "M": M, "V": V, "dtype": dtype, "top": top, "T": T, "nodes": nodes}


R = 64  # rotary elements of a latent cache's row


def listed():
    return [
        # queries of one verification step, k + 1 = 6 new tokens of 64 sequences: latency
        _rope("rope_step", 64, 6, 32, 128, 128, 0, False, "plain", 8200, "bf16"),
        # queries of eight prompts, half of each head turned, fp32 as a projection leaves them
        _rope("rope_prompt", 8, 4099, 16, 128, 64, 64, True, "turns", 4099, "f32"),
        # the same step's keys into an e4m3 cache with its queries, far along a scaled context
        _kv("kv_step", 64, 6, 32, 8, 128, 128, False, "turns", 64, 8200, "e4m3"),
        # eight prompts' keys, values and queries, a bf16 cache
        _kv("kv_prompt", 8, 4099, 32, 8, 128, 128, False, "linear", 16, 4099, "bf16"),
        # after verification: the accepted path's nodes of 85-node trees into a latent cache
        _put("put_path", 16, 85, 512, 64, 2100, "plain", path=4),
        # the prompts of sixteen sequences into a latent cache
        _put("put_prompt", 16, 6001, 512, 64, 6001, "index"),
        # one token of one sequence over a latent cache: the smallest call, all latency
        _latent("latent_token", 1, 1, 16, 512, 64, 2049),
        # k = 5 chain verification for 64 sequences
        _latent("latent_chain", 64, 6, 32, 512, 64, 8200),
        # 85-node trees (branching 4, depth 3) for 16 sequences
        _latent("latent_tree", 16, 85, 16, 512, 64, 7001, tree=1),
        # one emitted token of one sequence, five alternatives: latency
        _logp("logp_token", 1, 1, 32000, "f32", 5, 1.0),
        # the emitted tokens of a verification step, twenty alternatives each
        _logp("logp_step", 64, 6, 151936, "bf16", 20, 0.7),
        # the accepted paths of 16 trees of 85 nodes, log probabilities alone
        _logp("logp_tree", 16, 4, 32000, "f32", 0, 1.0, nodes=85),
    ]


HEADS = ((32, 8, 128), (32, 4, 64), (24, 8, 128), (12, 12, 64), (28, 4, 128), (8, 1, 128), (16, 2, 64))
SCALINGS = ("plain", "linear", "turns", "index")


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(("rope", "kv", "kv", "put", "latent", "latent", "latent", "logp", "logp"))
    Hq, Hkv, D = rng.choice(HEADS)
    page = rng.choice((16, 32, 64, 128))
    scaling, inter = rng.choice(SCALINGS), rng.random() < 0.5
    if kind == "rope":
        rot = rng.choice((16, 32, 64, D))
        first = rng.choice((0, D - rot))
        B = _log(rng, 1, 128)
        N = _log(rng, 1, max(1, 8 * 4099 * 16 // (B * Hq * D // 128 + 1)))
        c = _rope("", B, N, Hq, D, rot, first, inter, scaling, N + _log(rng, 1, 200000), rng.choice(("bf16", "f32")))
    elif kind == "kv":
        rot = rng.choice((16, 32, 64, D))
        cache = rng.choice(("bf16", "e4m3"))
        B = _log(rng, 1, 128)
        # an e4m3 cache's exponents are whole numbers: few enough rows that none lies at a border
        room = 16000 // Hkv if cache == "e4m3" else 8 * 4099 * 8 * 128 // (Hkv * D)
        N = _log(rng, 1, max(1, room // B))
        path = rng.choice((0, 0, min(N, 4) if N <= 128 else 0))
        c = _kv("", B, N, Hq, Hkv, D, rot, inter, scaling, page, N + _log(rng, 1, 4000), cache, path)
    elif kind == "put":
        B, C = _log(rng, 1, 128), rng.choice((128, 256, 512))
        N = _log(rng, 1, max(1, 16 * 6001 // B))
        c = _put("", B, N, C, page, N + _log(rng, 1, 4000), scaling, rng.choice((0, 0, min(N, 4) if N <= 128 else 0)))
        c["interleaved"] = inter
    elif kind == "latent":
        H, C, tree = rng.choice((8, 16, 20, 32, 64, 128)), rng.choice((128, 256, 512, 512)), rng.choice((0, 0, 1))
        B = _log(rng, 1, 16 if tree else 128)
        N = _log(rng, 9, 128) if tree else rng.randrange(1, 9)
        most = 64 * 6 * 32 * 8200 // (B * N * H)  # scores of the larger listed case
        L = _log(rng, N + 1, max(N + 2, min(140000, most, 64 * 8200 // B)))
        c = _latent("", B, N, H, C, page, L, tree)
    else:
        V = rng.choice((32000, 128256, 151936, _log(rng, 100, 160000)))
        dtype = rng.choice(("bf16", "f32"))
        nodes = rng.choice((0, 0, 0, 21, 85))
        B = _log(rng, 1, max(1, min(128, 64 * 151936 // (V * (nodes or 6) * (2 if dtype == "f32" else 1)) * 6)))
        c = _logp("", B, 4 if nodes else rng.randrange(1, 7), V, dtype, rng.choice((0, 1, 5, 20, 32)),
                  rng.choice((1.0, 0.7, 1.3)), nodes)
    del c["name"]
    return c


# ------------------------------------------------------------------ inputs

def _lens(case):
    """The sequences' lengths: a fixed ragged pattern, the first the longest."""
    L = case["L"]
    return [max(case["N"], L - int(0.5 * L * ((b * 2654435761) % 4294967296) / 4294967296))
            for b in range(case["B"])]


def _generator(seed):
    g = torch.Generator("cuda")
    g.manual_seed(seed)
    return g


def _normal(g, *shape, dtype=torch.bfloat16):
    return torch.randn(shape, generator=g, device="cuda", dtype=dtype)


def _scaling(case):
    """What a user sets for the frequencies: (factor, low, high)."""
    return {"plain": (1.0, 0.0, 0.0), "linear": (4.0, 0.0, 0.0), "turns": (8.0, 1.0, 4.0),
            "index": (16.0, 1.0, 32.0)}[case["scaling"]]


def _angles(case, rot):
    """The pairs' angles a position, in 64 bits."""
    i = torch.arange(rot // 2, dtype=torch.float64)
    f = BASE ** (-2.0 * i / rot)
    factor, low, high = _scaling(case)
    if case["scaling"] == "linear":
        f = f / factor
    elif case["scaling"] == "turns":  # by how often a pair turns within the original context
        w = ((ORIGINAL * f / (2 * math.pi) - low) / (high - low)).clamp(0, 1)
        f = f * (w + (1 - w) / factor)
    elif case["scaling"] == "index":  # between the pairs that turn `high` and `low` times there
        at = [rot * math.log(ORIGINAL / (t * 2 * math.pi)) / (2 * math.log(BASE)) for t in (high, low)]
        a, b = max(0, math.floor(at[0])), min(rot - 1, math.ceil(at[1]))
        w = 1 - ((i - a) / max(b - a, 1e-3)).clamp(0, 1)
        f = f * (w + (1 - w) / factor)
    return f


def _table(rs, pages, width, ids):
    """[B, width] page ids (-1 where a sequence has none), handed out in a random order."""
    t = torch.full((len(pages), width), -1, dtype=torch.int32)
    ids = list(ids)
    rs.shuffle(ids)
    for b, n in enumerate(pages):
        t[b, :n] = torch.tensor([ids.pop() for _ in range(n)], dtype=torch.int32)
    return t.cuda()


def _trees(rs, case):
    """[B, N, N] masks and [B, N] depths: the full tree of branching 4 where N is its size, else grown at random."""
    B, N = case["B"], case["N"]
    mask, depth = torch.zeros((B, N, N), dtype=torch.uint8), torch.zeros((B, N), dtype=torch.int32)
    for b in range(B):
        if b and N == 85:
            mask[b], depth[b] = mask[0], depth[0]
            continue
        for n in range(N):
            if n:
                p = (n - 1) // 4 if N == 85 else rs.randrange(max(0, n - 12), n)
                mask[b, n], depth[b, n] = mask[b, p], depth[b, p] + 1
            mask[b, n, n] = 1
    return mask.cuda(), depth.cuda()


def _paths(rs, B, N, M):
    """[B, M]: the root, then deeper and deeper nodes, and -1 past the accepted depth."""
    rows = torch.full((B, M), -1, dtype=torch.int32)
    for b in range(B):
        keep = sorted(rs.sample(range(1, N), min(N - 1, rs.randrange(0, M)))) if N > 1 else []
        rows[b, :1 + len(keep)] = torch.tensor([0] + keep, dtype=torch.int32)
    return rows.cuda()


def _prepare_logp(case, rs, g, s):
    B, M, V, nodes = case["B"], case["M"], case["V"], case["nodes"]
    rows = nodes or M
    ranks = -1.1 * torch.log(torch.arange(1, V + 1, device="cuda", dtype=torch.float32))
    logits = torch.empty((B, rows, V), device="cuda", dtype=torch.bfloat16 if case["dtype"] == "bf16" else torch.float32)
    tokens = torch.empty((B, rows), device="cuda", dtype=torch.int32)
    for b in range(B):  # -1.1 log(rank) of a random order, and noise; a token drawn from each row
        perm = torch.rand((V,), generator=g, device="cuda").argsort()
        x = (ranks[perm] + 1.5 * _normal(g, rows, V, dtype=torch.float32)).to(logits.dtype)
        logits[b] = x
        noise = -torch.log(-torch.log(torch.rand((rows, V), generator=g, device="cuda").clamp(1e-30, 1 - 1e-7)))
        tokens[b] = (x.float() / case["T"] + noise).argmax(-1).int()
    s["logits"], s["rows"] = logits, None
    if nodes:
        s["rows"] = _paths(rs, B, nodes, M)
        picked = tokens.gather(1, s["rows"].clamp(min=0).long())
        tokens = torch.where(s["rows"] >= 0, picked, picked.new_full((), -1))
    else:  # emitted tokens, then -1
        last = torch.tensor([rs.randrange(1, M + 1) for _ in range(B)], device="cuda")
        tokens = torch.where(torch.arange(M, device="cuda") < last[:, None], tokens, tokens.new_full((), -1))
    s["tokens"] = tokens.int().contiguous()


def prepare(case, seed):
    rs, g = random.Random(seed), _generator(seed)
    kind = case["kind"]
    s = {"case": case}
    if kind == "logp":
        _prepare_logp(case, rs, g, s)
    elif kind == "rope":
        dtype = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
        s["x"] = _normal(g, case["B"], case["N"], case["H"], case["D"], dtype=dtype)
        start = torch.tensor([rs.randrange(0, case["far"] - case["N"] + 1) for _ in range(case["B"])])
        s["pos"] = (start[:, None] + torch.arange(case["N"])).int().cuda()
        s["angles"] = _angles(case, case["rot"]).cuda()
    else:
        B, N, page = case["B"], case["N"], case["page"]
        lens = _lens(case)
        pages = [-(-n // page) for n in lens]
        total = sum(pages) + 3  # a pool holds pages of others too
        s["lens"] = torch.tensor(lens, dtype=torch.int32).cuda()
        s["table"] = _table(rs, pages, max(pages), range(total))
        s["starts"] = s["lens"] - N
        if kind != "latent":
            s["rows"] = _paths(rs, B, N, case["path"]) if case["path"] else None
            _, depth = _trees(rs, case) if case["path"] else (None, torch.arange(N, device="cuda").int())
            s["pos"] = (s["starts"][:, None] + depth).int().contiguous()  # a node's position index: the root's + its depth
            s["angles"] = _angles(case, R if kind == "put" else case["rot"]).cuda()
        if kind == "kv":
            Hkv, D = case["Hkv"], case["D"]
            s["pool"] = {"k_exp": None, "v_exp": None}
            for w in "kv":
                s["pool"][w] = _normal(g, total, Hkv, page, D)
                if case["cache"] == "e4m3":
                    s["pool"][w] = s["pool"][w].to(torch.float8_e4m3fn)
                    s["pool"][w + "_exp"] = torch.zeros((total, Hkv, page), device="cuda", dtype=torch.int8)
                s[w] = _normal(g, B, N, Hkv, D)
            s["q"] = None if case["path"] else _normal(g, B, N, case["Hq"], D)
        else:
            s["pool"] = _normal(g, total, page, case["C"] + R)
            if kind == "put":
                s["c"], s["r"] = _normal(g, B, N, case["C"]), _normal(g, B, N, R)
            else:
                s["q"] = _normal(g, B, N, case["H"], case["C"] + R)
                s["mask"] = _trees(rs, case)[0] if case["tree"] else None
                s["scale"] = 1.0 / math.sqrt(128 + R)  # of the head the latent stands for
    if own:
        import speculative_decoding_verification_top_gb300 as sv
        if "angles" in s:
            factor, low, high = _scaling(case)
            s["freqs"] = sv.rope_freqs(2 * s["angles"].numel(), BASE, case["scaling"], factor, ORIGINAL, low, high,
                                       device="cuda")
        if kind == "kv":
            s["cache"] = sv.KVCache(s["pool"]["k"], s["pool"]["v"], s["pool"]["k_exp"], s["pool"]["v_exp"])
        elif kind in ("put", "latent"):
            s["cache"] = sv.LatentCache(s["pool"], R)
        if kind == "latent":
            s["workspace"] = sv.new_workspace(
                sv.spec_latent_workspace_size(case["B"], case["N"], case["H"], case["C"]), "cuda")
        elif kind == "logp":
            s["workspace"] = sv.new_workspace(sv.spec_verify_logprobs_workspace_size(), "cuda")
    return s


# ------------------------------------------------------------------ plain forms

def _power(e):
    """2 ** e in fp32, exactly."""
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def _quantise(x):
    """x [..., D] fp32 -> e4m3 values and, per row, the smallest exponent e with max |x| <= 448 * 2 ** e."""
    m, e = torch.frexp(x.abs().amax(-1))
    e = torch.where(m > 0, e - 9 + (m > E4M3_MAX / 512).int(), torch.zeros_like(e)).clamp(-120, 120)
    return (x * _power(-e)[..., None]).to(torch.float8_e4m3fn), e.to(torch.int8)


def _turn(x, pos, angles, interleaved):
    """x [B, N, H, rot] fp32 turned to its positions; the angles in 64 bits, as far positions need."""
    a = pos[:, :, None, None].double() * angles
    c, s = torch.cos(a).float(), torch.sin(a).float()
    if interleaved:
        u, v = x[..., 0::2], x[..., 1::2]
        return torch.stack((u * c - v * s, v * c + u * s), -1).flatten(-2)
    u, v = x.chunk(2, -1)
    return torch.cat((u * c - v * s, v * c + u * s), -1)


def _plain_rope(s):
    c = s["case"]
    a, b = c["first"], c["first"] + c["rot"]
    out = s["x"].clone()
    out[..., a:b] = _turn(s["x"][..., a:b].float(), s["pos"], s["angles"], c["interleaved"]).to(out.dtype)
    return out


def _places(s, count):
    """Page and slot of `count` positions from each sequence's start."""
    at = s["starts"][:, None].long() + torch.arange(count, device="cuda")
    page = s["case"]["page"]
    return s["table"].long().gather(1, at // page), at % page


def _picked(s, x):
    """The tokens of x [B, N, ...] that are written, flat, with their pages and slots."""
    rows = s["rows"]
    p, o = _places(s, x.shape[1] if rows is None else rows.shape[1])
    if rows is None:
        return x.flatten(0, 1), p.flatten(), o.flatten()
    some = rows >= 0
    b = torch.arange(len(rows), device="cuda")[:, None].expand_as(rows)
    return x[b[some], rows[some].long()], p[some], o[some]


def _plain_kv(s):
    c, pool = s["case"], s["pool"]
    rot = c["rot"]

    def turned(x):
        return torch.cat((_turn(x[..., :rot].float(), s["pos"], s["angles"], c["interleaved"]), x[..., rot:].float()), -1)

    for w, x in (("k", turned(s["k"])), ("v", s["v"].float())):
        x, p, o = _picked(s, x)
        if pool["k_exp"] is None:
            pool[w][p, :, o] = x.to(torch.bfloat16)
        else:
            x, e = _quantise(x)
            pool[w].view(torch.uint8)[p, :, o] = x.view(torch.uint8)
            pool[w + "_exp"][p, :, o] = e
    return {"q": None if s["q"] is None else turned(s["q"]).to(s["q"].dtype), **pool}


def _plain_put(s):
    r = _turn(s["r"].float()[:, :, None], s["pos"], s["angles"], s["case"]["interleaved"])[:, :, 0]
    x, p, o = _picked(s, torch.cat((s["c"], r.to(torch.bfloat16)), -1))
    s["pool"][p, o] = x
    return s["pool"]


def _plain_latent(s):
    c = s["case"]
    B, N, H, C = c["B"], c["N"], c["H"], c["C"]
    K = s["pool"][s["table"].clamp(min=0).long()].float().flatten(1, 2)  # [B, pages * page, C + R]
    j = torch.arange(K.shape[1], device="cuda")
    lens = s["lens"].long()[:, None]
    here = j < lens
    K = K * here[:, :, None]
    at = j - (lens - N)                                                  # which new token a position holds
    if s["mask"] is None:
        among = torch.arange(N, device="cuda")[:, None] >= at[:, None, :]
    else:
        among = s["mask"].gather(2, at.clamp(0, N - 1)[:, None, :].expand(B, N, K.shape[1])) != 0
    seen = here[:, None, :] & ((at < 0)[:, None, :] | among)             # [B, N, positions]
    q = s["q"].float().flatten(1, 2) * s["scale"]
    scores = (q @ K.transpose(1, 2)).view(B, N, H, -1).masked_fill(~seen[:, :, None, :], -math.inf)
    m = scores.amax(-1, keepdim=True)
    w = torch.exp(scores - torch.where(m == -math.inf, torch.zeros_like(m), m))
    total = w.sum(-1, keepdim=True)
    out = (w.view(B, N * H, -1) @ K[..., :C]).view(B, N, H, C)
    return (out / torch.where(total > 0, total, torch.ones_like(total))).to(s["q"].dtype)


def _plain_logp(s):
    c = s["case"]
    logits, tokens = s["logits"], s["tokens"]
    if s["rows"] is not None:
        logits = logits.gather(1, s["rows"].clamp(min=0).long()[:, :, None].expand(-1, -1, c["V"]))
    raw, some = logits.float(), tokens >= 0
    x = raw / c["T"]
    x = x - x.amax(-1, keepdim=True)
    e = torch.exp(x)
    total = e.sum(-1, keepdim=True)
    log_total = torch.log(total)
    at = tokens.clamp(min=0).long()[..., None]
    entropy = log_total[..., 0] - (e * x).sum(-1) / total[..., 0]
    mine = raw.gather(2, at)
    before = torch.arange(c["V"], device="cuda") < at
    rank = ((raw > mine) | ((raw == mine) & before)).sum(-1).int()
    out = {"logprob": torch.where(some, (x.gather(2, at) - log_total)[..., 0], torch.zeros_like(entropy)),
           "entropy": torch.where(some, entropy, torch.zeros_like(entropy)),
           "rank": torch.where(some, rank, rank.new_full((), -1))}
    if c["top"]:
        order = torch.sort(raw, dim=-1, descending=True, stable=True)[1][..., :c["top"]]
        top = x.gather(2, order) - log_total
        out["ids"] = torch.where(some[..., None], order.int(), rank.new_full((), -1))
        out["top"] = torch.where(some[..., None], top, torch.zeros_like(top))
    return out


def run(s):
    c = s["case"]
    kind = c["kind"]
    if not own:
        return {"rope": _plain_rope, "kv": _plain_kv, "put": _plain_put, "latent": _plain_latent,
                "logp": _plain_logp}[kind](s)
    import speculative_decoding_verification_top_gb300 as sv
    if kind == "rope":
        return sv.rope(s["x"], s["freqs"], s["pos"], first=c["first"], interleaved=c["interleaved"])
    if kind == "kv":
        q = sv.kv_append_rope(s["cache"], s["table"], s["starts"], s["k"], s["v"], s["freqs"], q=s["q"], rows=s["rows"],
                              pos=s["pos"], interleaved=c["interleaved"])
        return {"q": q, **s["pool"]}
    if kind == "put":
        sv.latent_append(s["cache"], s["table"], s["starts"], s["c"], s["r"], s["freqs"], rows=s["rows"], pos=s["pos"],
                         interleaved=c["interleaved"])
        return s["pool"]
    if kind == "latent":
        return sv.latent_attn(s["q"], s["cache"], s["table"], s["lens"], s["scale"], mask=s["mask"],
                              workspace=s["workspace"])
    r = sv.logprobs(s["logits"], s["tokens"], rows=s["rows"], temperature=c["T"], top=c["top"],
                    workspace=s["workspace"])
    return {"logprob": r.logprob, "entropy": r.entropy, "rank": r.rank,
            **({"ids": r.top_ids, "top": r.top_logprobs} if c["top"] else {})}


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    kind, B = case["kind"], case["B"]
    if kind == "rope":
        n = B * case["N"] * case["H"]
        size = 2 if case["dtype"] == "bf16" else 4
        return {"bytes": 2 * n * case["D"] * size + 4 * B * case["N"], "flops": 3 * n * case["rot"]}
    if kind == "logp":
        rows = B * (1 + (case["M"] - 1) / 2)  # emitted tokens, on average
        size = 2 if case["dtype"] == "bf16" else 4
        return {"bytes": rows * case["V"] * size + B * case["M"] * (16 + 8 * case["top"]), "flops": 5 * rows * case["V"]}
    N = case["N"]
    written = B * (min(case["path"], 1 + (case["path"] - 1) / 2) if case.get("path") else N)
    if kind == "kv":
        Hkv, D = case["Hkv"], case["D"]
        row = Hkv * (D + 1 if case["cache"] == "e4m3" else 2 * D)
        q = 0 if case["path"] else 4 * B * N * case["Hq"] * D
        return {"bytes": 2 * written * (2 * Hkv * D + row) + q,
                "flops": 3 * case["rot"] * (written * Hkv + (0 if case["path"] else B * N * case["Hq"]))}
    C = case["C"]
    if kind == "put":
        return {"bytes": 4 * written * (C + R), "flops": 3 * written * R}
    H, total = case["H"], sum(_lens(case))
    return {"bytes": 2 * total * (C + R) + 2 * B * N * H * (2 * C + R) + (B * N * N if case["tree"] else 0),
            "flops": 2 * N * H * total * (2 * C + R)}


# ------------------------------------------------------------------ the definitions in 64 bits

def _turned64(x, pos, angles, interleaved):
    """x [n, H, rot] at pos [n]: as complex numbers times e^(i angle)."""
    half = x.shape[-1] // 2
    x = x.double()
    z = torch.complex(x[..., 0::2], x[..., 1::2]) if interleaved else torch.complex(x[..., :half], x[..., half:])
    a = (pos.double()[:, None] * angles)[:, None, :]
    z = z * torch.polar(torch.ones_like(a), a)
    out = torch.empty_like(x)
    if interleaved:
        out[..., 0::2], out[..., 1::2] = z.real, z.imag
    else:
        out[..., :half], out[..., half:] = z.real, z.imag
    return out


def _exact_rope(s):
    c = s["case"]
    out = s["x"].double()
    for b in range(c["B"]):
        part = out[b, :, :, c["first"]:c["first"] + c["rot"]]
        part.copy_(_turned64(part.clone(), s["pos"][b], s["angles"], c["interleaved"]))
    return out


def _entries(s):
    """Per sequence: its tokens that are written, and the pages and slots they go to."""
    c = s["case"]
    for b in range(c["B"]):
        rows = list(range(c["N"])) if s["rows"] is None else s["rows"][b].tolist()
        put = [(t, r) for t, r in enumerate(rows) if r >= 0]
        at = torch.tensor([t for t, _ in put], device="cuda") + int(s["starts"][b])
        yield b, torch.tensor([r for _, r in put], device="cuda"), s["table"][b][at // c["page"]].long(), at % c["page"]


def _exact_kv(s):
    c, pool = s["case"], s["pool"]
    out = {w: pool[w].double() for w in ("k", "v")}
    rot = c["rot"]

    def turned(x, pos):
        x = x.double()
        return torch.cat((_turned64(x[..., :rot], pos, s["angles"], c["interleaved"]), x[..., rot:]), -1)

    for b, r, page, slot in _entries(s):
        for w in ("k", "v"):
            x = turned(s["k"][b, r], s["pos"][b, r]) if w == "k" else s["v"][b, r].double()
            if pool["k_exp"] is not None:
                most = x.abs().amax(-1, keepdim=True)
                e = torch.floor(torch.log2(most / E4M3_MAX)) - 1
                for _ in range(2):
                    e = e + (most > E4M3_MAX * torch.exp2(e)).double()
                y = x / torch.exp2(e)
                grid = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
                x = torch.round(y / grid) * grid  # halves to even, as the format rounds
            out[w][page, :, slot] = x
    q = None if s["q"] is None else torch.stack([turned(s["q"][b], s["pos"][b]) for b in range(c["B"])])
    return {"q": q, "k_exp": None, "v_exp": None, **out}


def _exact_put(s):
    out, C = s["pool"].double(), s["case"]["C"]
    for b, r, page, slot in _entries(s):
        out[page, slot, :C] = s["c"][b, r].double()
        out[page, slot, C:] = _turned64(s["r"][b, r][:, None], s["pos"][b, r], s["angles"], s["case"]["interleaved"])[:, 0]
    return out


def _exact_latent(s):
    c, out = s["case"], []
    N, C = c["N"], c["C"]
    for b in range(c["B"]):
        n = int(s["lens"][b])
        j = torch.arange(n, device="cuda")
        K = s["pool"][s["table"][b][j // c["page"]].long(), j % c["page"]].double()
        seen = torch.ones((N, n), dtype=torch.bool, device="cuda")
        seen[:, -N:] = torch.ones((N, N), device="cuda").tril() > 0 if s["mask"] is None else s["mask"][b] > 0
        a = torch.einsum("nhd,ld->nhl", s["q"][b].double(), K) * s["scale"]
        out.append(torch.softmax(a.masked_fill(~seen[:, None], -math.inf), -1) @ K[:, :C])
    return torch.stack(out)


def _exact_logp(s):
    c = s["case"]
    B, M, V, k = c["B"], c["M"], c["V"], c["top"]
    out = {"logprob": torch.zeros((B, M), dtype=torch.float64), "entropy": torch.zeros((B, M), dtype=torch.float64),
           "rank": torch.full((B, M), -1, dtype=torch.int32)}
    if k:
        out |= {"ids": torch.full((B, M, k), -1, dtype=torch.int32), "top": torch.zeros((B, M, k), dtype=torch.float64)}
    for b in range(B):
        for t in range(M):
            token = int(s["tokens"][b, t])
            if token < 0:
                continue
            x = s["logits"][b, t if s["rows"] is None else int(s["rows"][b, t])].double()
            p = torch.log_softmax(x / c["T"], -1)
            out["logprob"][b, t] = p[token]
            out["entropy"][b, t] = -(p.exp() * p).sum()
            out["rank"][b, t] = (x > x[token]).sum() + (x[:token] == x[token]).sum()
            if k:
                least = x.topk(k)[0][-1]  # everything down to it, the earlier of equals first
                at = torch.nonzero(x >= least)[:, 0]
                at = at[torch.argsort(x[at], descending=True, stable=True)][:k]
                out["ids"][b, t], out["top"][b, t] = at.int(), p[at]
    return out


def exact(case, seed):
    s = prepare(case, seed)
    return {"rope": _exact_rope, "kv": _exact_kv, "put": _exact_put, "latent": _exact_latent,
            "logp": _exact_logp}[case["kind"]](s)
