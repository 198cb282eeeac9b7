"""The operators of the target pass that tree verification needs, in plain form and as the library's calls.

A verification step scores k + 1 chain positions, or the N nodes of a candidate tree, for every sequence in one
target pass.  Around the logits that pass needs

  append  the new tokens' keys and values written into a paged cache, in bf16 or as e4m3 bytes with a
          power-of-two scale per token and head; after verification the accepted path's nodes only (`rows`);
  read    cached positions back as bf16 rows;
  attn    the new tokens' attention over their sequence's cache: the context, and among the new tokens the
          chain before each one or its tree ancestors, with a tanh cap on the scores, a bias per head that is
          linear in the distance, and a window;
  shared  the same where every sequence of the batch continues one long prefix held once.

A case is one pass of one of them.  Sequence lengths are ragged: the longest is `L`, the shortest about
`L * (1 - spread)`.
"""
import math
import random

import torch

own = False

E4M3_MAX = 448.0


# ------------------------------------------------------------------ cases

def _attn(name, B, N, Hq, Hkv, D, page, L, cache, tree=0, cap=0.0, window=0, slopes=False, shared=0, spread=0.5):
    kind = "shared" if shared else "attn"
    return {"name": name, "kind": kind, "B": B, "N": N, "Hq": Hq, "Hkv": Hkv, "D": D, "page": page, "L": L,
            "cache": cache, "tree": tree, "cap": cap, "window": window, "slopes": slopes, "shared": shared,
            "spread": spread}


def _append(name, B, N, Hkv, D, page, L, cache, path=0):
    return {"name": name, "kind": "append", "B": B, "N": N, "Hkv": Hkv, "D": D, "page": page, "L": L,
            "cache": cache, "path": path, "spread": 0.5}


def _read(name, B, M, Hkv, D, page, L, cache):
    return {"name": name, "kind": "read", "B": B, "M": M, "Hkv": Hkv, "D": D, "page": page, "L": L,
            "cache": cache, "spread": 0.0}


def listed():
    return [
        # one verification step's k + 1 = 6 new tokens of 64 sequences: latency
        _append("append_step", 64, 6, 8, 128, 64, 4100, "e4m3"),
        # the prompts of eight sequences, an odd number of tokens each
        _append("append_prompt", 8, 4099, 8, 128, 16, 4099, "e4m3"),
        # after verification: the accepted path's nodes of 85-node trees (depth 3), at most 4 of each tree's 85
        _append("append_path", 16, 85, 8, 128, 64, 2100, "bf16", path=4),
        # sixteen sequences' caches back as bf16, to move them to another machine or layer form
        _read("read_batch", 16, 6001, 8, 128, 64, 6001, "e4m3"),
        # one short sequence's cache
        _read("read_one", 1, 777, 4, 64, 16, 777, "bf16"),
        # a single token of a single sequence: the smallest call, all latency
        _attn("attn_token", 1, 1, 32, 8, 128, 64, 2049, "bf16"),
        # k = 5 chain verification for 64 sequences over an e4m3 cache
        _attn("attn_chain_e4m3", 64, 6, 32, 8, 128, 64, 8200, "e4m3"),
        # k = 3 chain verification for 128 sequences, capped scores, 64-wide heads in groups of eight
        _attn("attn_chain_cap", 128, 4, 32, 4, 64, 16, 5003, "bf16", cap=30.0),
        # 85-node trees (branching 4, depth 3) for 16 sequences, distance bias
        _attn("attn_tree", 16, 85, 32, 8, 128, 64, 7001, "bf16", tree=1, slopes=True),
        # k = 4 chain of one sequence with a long context: the work is split along the cache
        _attn("attn_long", 1, 5, 32, 8, 128, 128, 131077, "e4m3", spread=0.0),
        # k = 5 chains of 64 sequences that continue one prompt of 16001 tokens
        _attn("shared_chain", 64, 6, 32, 8, 128, 64, 700, "e4m3", shared=16001),
        # 85-node trees of 16 sequences under one prompt
        _attn("shared_tree", 16, 85, 32, 8, 128, 32, 401, "bf16", tree=1, shared=8190),
    ]


HEADS = ((32, 8, 128), (32, 4, 64), (24, 8, 128), (12, 12, 64), (28, 4, 128), (8, 1, 128), (16, 2, 64))


def _log(rng, lo, hi):
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    v = max(lo, min(hi, v))
    return v + 1 if v == 3 << 10 else v


def draw(rng):
    kind = rng.choice(("append", "read", "attn", "attn", "attn", "shared", "shared"))
    Hq, Hkv, D = rng.choice(HEADS)
    page = rng.choice((16, 32, 64, 128))
    cache = rng.choice(("bf16", "e4m3"))
    room = 16 * 7001 * 8 * 128  # cached elements of the larger listed cases
    if kind == "append":
        B = _log(rng, 1, 128)
        N = _log(rng, 1, max(2, min(8000, room // 4 // (B * Hkv * D))))
        path = rng.choice((0, 0, min(N, 4)))
        c = _append("", B, N, Hkv, D, page, N + _log(rng, 1, 2000), cache, path)
    elif kind == "read":
        B = _log(rng, 1, 64)
        M = _log(rng, 1, max(2, min(16000, room // (B * Hkv * D))))
        c = _read("", B, M, Hkv, D, page, M + rng.randrange(0, 50), cache)
    else:
        tree = rng.choice((0, 0, 1))
        B = _log(rng, 1, 16 if tree else 128)
        N = _log(rng, 9, 128) if tree else rng.randrange(1, 9)
        most = max(N + 2, min(140000, room // (B * Hkv * D)))
        if tree:
            most = max(N + 2, min(most, 16 * 85 * 32 * 7001 // (B * N * Hq)))
        L = _log(rng, N + 1, most)
        shared = 0
        if kind == "shared":
            L = _log(rng, N + 1, max(N + 2, min(most, 2000)))
            shared = _log(rng, 100, max(101, min(17000, 64 * 6 * 32 * 16001 // (B * N * Hq))))
        c = _attn("", B, N, Hq, Hkv, D, page, L, cache, tree=tree, cap=rng.choice((0.0, 0.0, 20.0, 50.0)),
                  window=rng.choice((0, 0, 0, _log(rng, 100, 4000))), slopes=rng.random() < 0.3, shared=shared)
    del c["name"]
    return c


# ------------------------------------------------------------------ inputs

def _lens(case):
    """The sequences' lengths: a fixed ragged pattern, the first the longest."""
    L, least = case["L"], case.get("N", case.get("M", 1))
    return [max(least, L - int(case["spread"] * L * ((b * 2654435761) % 4294967296) / 4294967296))
            for b in range(case["B"])]


def _generator(seed):
    g = torch.Generator("cuda")
    g.manual_seed(seed)
    return g


def _normal(g, *shape):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16)


def _pool(g, n, case):
    """A cache of n pages: keys and values as a pass leaves them, drawn page by page."""
    Hkv, page, D = case["Hkv"], case["page"], case["D"]
    out = []
    for what in ("k", "v"):
        if case["cache"] == "bf16":
            out.append((_normal(g, n, Hkv, page, D), None))
            continue
        x = torch.empty((n, Hkv, page, D), device="cuda", dtype=torch.float8_e4m3fn)
        e = torch.empty((n, Hkv, page), device="cuda", dtype=torch.int8)
        step = max(1, (1 << 26) // (Hkv * page * D))
        for i in range(0, n, step):
            x[i:i + step], e[i:i + step] = _quantise(_normal(g, min(step, n - i), Hkv, page, D).float())
        out.append((x, e))
    return {"k": out[0][0], "v": out[1][0], "k_exp": out[0][1], "v_exp": out[1][1]}


def _table(rs, pages, width, ids):
    """[B, width] page ids (-1 where a sequence has none), handed out in a random order."""
    t = torch.full((len(pages), width), -1, dtype=torch.int32)
    ids = list(ids)
    rs.shuffle(ids)
    for b, n in enumerate(pages):
        t[b, :n] = torch.tensor([ids.pop() for _ in range(n)], dtype=torch.int32)
    return t.cuda()


def _trees(rs, case):
    """Parents of each sequence's tree: the full tree of branching 4 where N is its size, else grown at random."""
    N, B = case["N"], case["B"]
    if N == 85:
        return [[-1] + [(n - 1) // 4 for n in range(1, N)]] * B
    return [[-1] + [rs.randrange(max(0, n - 12), n) for n in range(1, N)] for _ in range(B)]


def prepare(case, seed):
    rs, g = random.Random(seed), _generator(seed)
    B, page, Hkv, D = case["B"], case["page"], case["Hkv"], case["D"]
    lens = _lens(case)
    pages = [-(-n // page) for n in lens]
    width = max(pages)
    s = {"case": case, "lens": torch.tensor(lens, dtype=torch.int32).cuda()}
    shared = case.get("shared", 0)
    sp = -(-shared // page)
    total = sum(pages) + sp + 3  # a pool holds pages of others too
    s["table"] = _table(rs, pages + ([sp] if sp else []), max(width, sp), range(total))
    if sp:
        s["shared_table"] = s["table"][B, :sp].contiguous()
        s["table"] = s["table"][:B, :width].contiguous()
    s["pool"] = _pool(g, total, case)
    if case["kind"] == "append":
        N = case["N"]
        s["k"], s["v"] = _normal(g, B, N, Hkv, D), _normal(g, B, N, Hkv, D)
        s["starts"] = torch.tensor([n - N for n in lens], dtype=torch.int32).cuda()
        s["rows"] = None
        if case["path"]:  # the root, then deeper and deeper nodes, and -1 past the accepted depth
            rows = torch.full((B, case["path"]), -1, dtype=torch.int32)
            for b in range(B):
                keep = sorted(rs.sample(range(1, N), min(N - 1, rs.randrange(0, case["path"])))) if N > 1 else []
                rows[b, :1 + len(keep)] = torch.tensor([0] + keep, dtype=torch.int32)
            s["rows"] = rows.cuda()
    elif case["kind"] == "read":
        s["starts"] = torch.tensor([n - case["M"] for n in lens], dtype=torch.int32).cuda()
    else:
        N, Hq = case["N"], case["Hq"]
        s["q"] = _normal(g, B, N, Hq, D)
        s["mask"] = s["pos"] = s["slopes"] = None
        if case["tree"]:
            m = torch.zeros((B, N, N), dtype=torch.uint8)
            p = torch.zeros((B, N), dtype=torch.int32)
            for b, parents in enumerate(_trees(rs, case)):
                if b and parents is last:
                    m[b], p[b] = m[b - 1], p[b - 1]
                else:
                    for n in range(N):
                        if n:
                            m[b, n], p[b, n] = m[b, parents[n]], p[b, parents[n]] + 1
                        m[b, n, n] = 1
                last = parents
            s["mask"] = m.cuda()
            s["pos"] = (p.cuda() + (s["lens"] - N + shared)[:, None]).int().contiguous()
        if case["slopes"]:
            s["slopes"] = torch.pow(2.0, -8.0 * torch.arange(1, Hq + 1, dtype=torch.float32) / Hq).cuda()
        s["scale"] = 1.0 / math.sqrt(D)
    if own:
        import speculative_decoding_verification_top_gb300 as sv
        s["cache"] = sv.KVCache(s["pool"]["k"], s["pool"]["v"], s["pool"]["k_exp"], s["pool"]["v_exp"])
        if case["kind"] in ("attn", "shared"):
            s["workspace"] = sv.new_workspace(
                sv.spec_attn_workspace_size(B, case["N"], case["Hq"], Hkv, D), "cuda")
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


def _values(pool, what, index=None):
    """The fp32 values of a pool's pages, all or those of `index`."""
    x, e = pool[what], pool[what + "_exp"]
    if index is not None:
        x = x.view(torch.uint8)[index].view(x.dtype) if e is not None else x[index]
        e = None if e is None else e[index]
    x = x.float()
    return x if e is None else x * _power(e)[..., None]


def _places(s, count):
    """Page and slot of `count` positions from each sequence's start."""
    at = s["starts"][:, None].long() + torch.arange(count, device="cuda")
    page = s["case"]["page"]
    return s["table"].long().gather(1, at // page), at % page


def _plain_append(s):
    k, v, pool, rows = s["k"], s["v"], s["pool"], s["rows"]
    p, o = _places(s, k.shape[1] if rows is None else rows.shape[1])
    if rows is not None:
        at = rows.clamp(min=0).long()[:, :, None, None].expand(-1, -1, k.shape[2], k.shape[3])
        k, v, some = k.gather(1, at), v.gather(1, at), rows >= 0
        p, o, k, v = p[some], o[some], k[some], v[some]
    for what, x in (("k", k), ("v", v)):
        if pool["k_exp"] is None:
            pool[what][p, :, o] = x
        else:
            x, e = _quantise(x.float())
            pool[what].view(torch.uint8)[p, :, o] = x.view(torch.uint8)
            pool[what + "_exp"][p, :, o] = e
    return pool


def _plain_read(s):
    p, o = _places(s, s["case"]["M"])
    out = []
    for what in ("k", "v"):
        x, e = s["pool"][what], s["pool"][what + "_exp"]
        x = x[p, :, o].float() if e is None else x.view(torch.uint8)[p, :, o].view(x.dtype).float()
        out.append((x if e is None else x * _power(e[p, :, o])[..., None]).to(torch.bfloat16))
    return out


def _heads(pool, what, table):
    """[..., pages] page ids -> [..., Hkv, pages * page, D] fp32."""
    x = _values(pool, what, table.clamp(min=0).long()).transpose(-4, -3)
    return x.reshape(*x.shape[:-3], -1, x.shape[-1])


def _plain_attention(s):
    c = s["case"]
    B, N, Hq, Hkv, D, Ls = c["B"], c["N"], c["Hq"], c["Hkv"], c["D"], c["shared"]
    G = Hq // Hkv
    q = s["q"].float().view(B, N, Hkv, G, D).permute(0, 2, 1, 3, 4).reshape(B, Hkv, N * G, D) * s["scale"]
    K, V = _heads(s["pool"], "k", s["table"]), _heads(s["pool"], "v", s["table"])
    Lp = K.shape[2]
    j = torch.arange(Lp, device="cuda")
    lens = s["lens"].long()[:, None]
    here = j < lens                                          # [B, Lp]
    V = V * here[:, None, :, None]
    node = j - (lens - N)                                    # which new token a position holds
    isnode = here & (node >= 0)
    at = node.clamp(0, N - 1)
    pos = Ls + lens - N + torch.arange(N, device="cuda") if s["pos"] is None else s["pos"].long()
    jpos = torch.where(isnode, pos.gather(1, at), Ls + j.expand(B, Lp))
    if s["mask"] is None:
        among = torch.arange(N, device="cuda")[:, None] >= at[:, None, :]
    else:
        among = s["mask"].gather(2, at[:, None, :].expand(B, N, Lp)) != 0
    seen = torch.where(isnode[:, None, :], among, here[:, None, :])  # [B, N, Lp]
    scores = q @ K.transpose(2, 3)
    if Ls:
        Ks, Vs = _heads(s["pool"], "k", s["shared_table"])[:, :Ls], _heads(s["pool"], "v", s["shared_table"])[:, :Ls]
        first = (q.transpose(0, 1).reshape(Hkv, B * N * G, D) @ Ks.transpose(1, 2)).view(Hkv, B, N * G, Ls)
        scores = torch.cat((first.transpose(0, 1), scores), 3)
        jpos = torch.cat((torch.arange(Ls, device="cuda").expand(B, Ls), jpos), 1)
        seen = torch.cat((torch.ones((B, N, Ls), dtype=torch.bool, device="cuda"), seen), 2)
    if c["cap"]:
        scores = c["cap"] * torch.tanh(scores / c["cap"])
    scores = scores.view(B, Hkv, N, G, -1)
    far = pos[:, :, None] - jpos[:, None, :]                 # [B, N, all]
    if s["slopes"] is not None:
        scores = scores - s["slopes"].view(1, Hkv, 1, G, 1) * far[:, None, :, None, :].float()
    if c["window"]:
        seen = seen & (far < c["window"])
    scores = scores.masked_fill(~seen[:, None, :, None, :], -math.inf)
    m = scores.amax(-1, keepdim=True)
    w = torch.exp(scores - torch.where(m == -math.inf, torch.zeros_like(m), m))
    total = w.sum(-1, keepdim=True)
    w = w.view(B, Hkv, N * G, -1)
    out = w[..., Ls:] @ V
    if Ls:
        first = w[..., :Ls].transpose(0, 1).reshape(Hkv, B * N * G, Ls) @ Vs
        out = out + first.view(Hkv, B, N * G, D).transpose(0, 1)
    out = out.view(B, Hkv, N, G, D) / torch.where(total > 0, total, torch.ones_like(total))
    return out.permute(0, 2, 1, 3, 4).reshape(B, N, Hq, D).to(s["q"].dtype)


def run(s):
    kind = s["case"]["kind"]
    if not own:
        return {"append": _plain_append, "read": _plain_read}.get(kind, _plain_attention)(s)
    import speculative_decoding_verification_top_gb300 as sv
    if kind == "append":
        sv.kv_append(s["cache"], s["table"], s["starts"], s["k"], s["v"], rows=s["rows"])
        return s["pool"]
    if kind == "read":
        return sv.kv_read(s["cache"], s["table"], s["starts"], s["case"]["M"])
    c = s["case"]
    more = dict(mask=s["mask"], pos=s["pos"], slopes=s["slopes"], scale=s["scale"], cap=c["cap"],
                window=c["window"], workspace=s["workspace"])
    if kind == "attn":
        return sv.attn_tree(s["q"], s["cache"], s["table"], s["lens"], **more)
    return sv.attn_shared(s["q"], s["cache"], s["shared_table"], c["shared"], s["table"], s["lens"], **more)


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    B, Hkv, D = case["B"], case["Hkv"], case["D"]
    row = Hkv * (D + 1 if case["cache"] == "e4m3" else 2 * D)  # one position's keys or values in the cache
    new = Hkv * D * 2
    if case["kind"] == "append":
        n = B * (min(case["path"], 1 + (case["path"] - 1) / 2) if case["path"] else case["N"])
        return {"bytes": 2 * n * (new + row), "flops": 0}
    if case["kind"] == "read":
        return {"bytes": 2 * B * case["M"] * (new + row), "flops": 0}
    N, Hq, Ls, w = case["N"], case["Hq"], case["shared"], case["window"]
    lens = _lens(case)
    held = [min(n, w + N) if w else n for n in lens]
    first = [min(Ls, max(0, w - n)) if w else Ls for n in lens]
    bytes_ = 2 * row * (sum(held) + max(first)) + 2 * 2 * B * N * Hq * D + (B * N * N if case["tree"] else 0)
    return {"bytes": bytes_, "flops": 4 * D * Hq * N * (sum(held) + sum(first))}


# ------------------------------------------------------------------ the definitions in 64 bits

def _two64(e):
    """2 ** e in 64 bits, exactly."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _row64(pool, what, page, slot):
    """The values of positions (page, slot): [n, Hkv, D] in 64 bits."""
    x, e = pool[what], pool[what + "_exp"]
    if e is None:
        return x[page, :, slot].double()
    return x.view(torch.uint8)[page, :, slot].view(x.dtype).double() * _two64(e[page, :, slot])[..., None]


def _where64(table, page, positions):
    return table[positions // page].long(), positions % page


def _exact_append(s):
    c, pool = s["case"], s["pool"]
    out = {w: pool[w].double() for w in ("k", "v")}
    for b in range(c["B"]):
        rows = list(range(c["N"])) if s["rows"] is None else s["rows"][b].tolist()
        put = [(t, r) for t, r in enumerate(rows) if r >= 0]
        t = torch.tensor([p[0] for p in put], device="cuda") + int(s["starts"][b])
        r = torch.tensor([p[1] for p in put], device="cuda")
        page, slot = _where64(s["table"][b], c["page"], t)
        for w in ("k", "v"):
            x = s[w][b, r].double()
            if pool["k_exp"] is not None:
                most = x.abs().amax(-1, keepdim=True)
                e = torch.frexp(most)[1] - 9
                e = e + (most > E4M3_MAX * _two64(e)).int()
                y = x / _two64(e)
                grid = _two64(torch.frexp(y.abs().clamp(min=2.0 ** -6))[1] - 4)
                x = torch.round(y / grid) * grid  # halves to even, as the format rounds
            out[w][page, :, slot] = x
    return {"k": out["k"], "v": out["v"], "k_exp": None, "v_exp": None}


def _exact_read(s):
    c = s["case"]
    got = {"k": [], "v": []}
    for b in range(c["B"]):
        t = int(s["starts"][b]) + torch.arange(c["M"], device="cuda")
        page, slot = _where64(s["table"][b], c["page"], t)
        for w in got:
            got[w].append(_row64(s["pool"], w, page, slot))
    return [torch.stack(got["k"]), torch.stack(got["v"])]


def _exact_attention(s):
    c = s["case"]
    N, Hq, Hkv, Ls = c["N"], c["Hq"], c["Hkv"], c["shared"]
    G, out = Hq // Hkv, []
    if Ls:
        page, slot = _where64(s["shared_table"], c["page"], torch.arange(Ls, device="cuda"))
        prefix = [_row64(s["pool"], w, page, slot) for w in ("k", "v")]
    for b in range(c["B"]):
        n = int(s["lens"][b])
        page, slot = _where64(s["table"][b], c["page"], torch.arange(n, device="cuda"))
        K, V = (_row64(s["pool"], w, page, slot) for w in ("k", "v"))
        if Ls:
            K, V = torch.cat((prefix[0], K)), torch.cat((prefix[1], V))
        where = torch.arange(Ls + n, device="cuda")
        mine = where[-N:].clone() if s["pos"] is None else s["pos"][b].long()
        seen = torch.ones((N, Ls + n), dtype=torch.bool, device="cuda")
        seen[:, -N:] = torch.ones((N, N), device="cuda").tril() > 0 if s["mask"] is None else s["mask"][b] > 0
        where[-N:] = mine
        far = (mine[:, None] - where[None, :]).double()
        if c["window"]:
            seen &= far < c["window"]
        rows = []
        for h in range(Hq):
            a = s["q"][b, :, h].double() @ K[:, h // G].T * s["scale"]
            if c["cap"]:
                a = c["cap"] * torch.tanh(a / c["cap"])
            if s["slopes"] is not None:
                a = a - s["slopes"][h].double() * far
            a = a.masked_fill(~seen, -math.inf)
            rows.append(torch.softmax(a, -1) @ V[:, h // G])
        out.append(torch.stack(rows, 1))
    return torch.stack(out)


def exact(case, seed):
    s = prepare(case, seed)
    return {"append": _exact_append, "read": _exact_read}.get(case["kind"], _exact_attention)(s)
