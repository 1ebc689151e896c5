"""What is measured of attention over packed sequences, its gradient, and attention of drafted tokens
over a paged cache.

`listed()` names the measured cases and `draw()` gives more of the same ranges.  `run()` is one
pass: in elementary torch operations, or, where `own` is set, through this package's entry points.
`exact()` is the operator's definition in 64 bits.
"""
import math

import torch

own = False

DEV = "cuda"


def listed():
    return [
        # six short prompts of a small model (1 to 48 tokens): launch latency counts
        dict(name="packed small d64", op="packed", R=6, lo=1, hi=48, plo=0, phi=0, Hq=8, Hk=2, d=64, causal=True, fused=True),
        # a server's batch of prompts, 20 to 2000 tokens
        dict(name="packed prompts", op="packed", R=24, lo=20, hi=2000, plo=0, phi=0, Hq=32, Hk=8, d=128, causal=True, fused=True),
        # the next 512 tokens or so of four prompts whose first 4000 to 30000 are in the cache
        dict(name="packed chunks", op="packed", R=4, lo=300, hi=512, plo=4001, phi=30011, Hq=32, Hk=8, d=128, causal=True, fused=False),
        # clips of different lengths seen in both directions, as many key heads as query heads
        dict(name="packed clips d64", op="packed", R=7, lo=500, hi=6143, plo=0, phi=0, Hq=16, Hk=16, d=64, causal=False, fused=False),
        # few long documents: the matrix products are the time
        dict(name="packed long", op="packed", R=4, lo=3001, hi=16384, plo=0, phi=0, Hq=32, Hk=8, d=128, causal=True, fused=True),
        # training on five short texts of a small model: latency
        dict(name="packed bwd small d64", op="packed_bwd", R=5, lo=1, hi=200, plo=0, phi=0, Hq=4, Hk=4, d=64, causal=True, fused=False),
        # training on packed texts, six query heads to a key head
        dict(name="packed bwd texts", op="packed_bwd", R=24, lo=10, hi=2501, plo=0, phi=0, Hq=24, Hk=4, d=128, causal=True, fused=True),
        # training on long documents
        dict(name="packed bwd long", op="packed_bwd", R=3, lo=2000, hi=16384, plo=0, phi=0, Hq=16, Hk=8, d=128, causal=True, fused=False),
        # eight drafted tokens for each of four requests of a small model: latency
        dict(name="tree small d64", op="tree", R=4, T=8, lo=9, hi=600, Hq=8, Hk=2, d=64, page=16, breadth=2, token_major=True),
        # one new token for each of 128 requests, pages of 16
        dict(name="tree one token", op="tree", R=128, T=1, lo=1, hi=4099, Hq=32, Hk=8, d=128, page=16, breadth=1, token_major=True),
        # trees of 24 drafted tokens for 48 requests
        dict(name="tree batch", op="tree", R=48, T=24, lo=1000, hi=9001, Hq=32, Hk=8, d=128, page=64, breadth=3, token_major=False),
        # trees of 60 drafted tokens at the end of two very long documents
        dict(name="tree long", op="tree", R=2, T=60, lo=90000, hi=131000, Hq=16, Hk=8, d=128, page=128, breadth=4, token_major=False),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["packed", "packed", "packed_bwd", "tree"])
    d = rng.choice([64, 128, 128])
    Hk = rng.choice([1, 2, 4, 8])
    G = rng.choice([1, 2, 3, 4, 7, 8])
    if op == "tree":
        R = _log(rng, 1, 128)
        T = rng.choice([1, 1, _log(rng, 2, 64)])
        hi = _log(rng, T, max(T, min(131000, (1 << 21) // (R * Hk), (1 << 27) // (R * T * Hk * G))))
        return dict(op=op, R=R, T=T, lo=rng.choice([T, max(T, hi // 2)]), hi=hi, Hq=Hk * G, Hk=Hk, d=d,
                    page=rng.choice([16, 32, 64, 128, 256]), breadth=rng.choice([1, 2, 4]), token_major=rng.random() < 0.5)
    R = _log(rng, 1, 48)
    causal = rng.random() < 0.75
    most = 5.5e9 if op == "packed" else 2.2e9  # pairs of a query and a key over all heads
    hi = _log(rng, 1, 12000)
    phi = _log(rng, 1, 30000) if op == "packed" and rng.random() < 0.3 else 0
    low = rng.choice([0, 0, 0.5])
    while True:
        case = dict(op=op, R=R, lo=int(hi * low), hi=hi, plo=phi // 3, phi=phi, Hq=Hk * G, Hk=Hk, d=d, causal=causal)
        ql, kl = _lens(case)
        if sum(a * b for a, b in zip(ql, kl)) * Hk * G <= most and sum(kl) * Hk <= 1 << 20 and sum(ql) * Hk * (G + 1) <= 1 << 20:
            break
        hi, phi, R = max(1, hi * 3 // 4), phi * 3 // 4, max(1, R * 9 // 10)
    case["fused"] = phi == 0 and rng.random() < 0.5
    return case


def _lens(case):
    """Queries and keys of the sequences: queries from `lo` to `hi`, short ones more often; before them, `plo` to `phi` keys
    that are there already."""
    R, lo, hi, plo, phi = (case[x] for x in ("R", "lo", "hi", "plo", "phi"))
    lo = min(lo, hi)
    at = [i / (R - 1) if R > 1 else 1.0 for i in range(R)]
    q = [lo + int((hi - lo) * x * x) for x in at]
    past = [plo + int((phi - plo) * (1 - x)) for x in at]
    return q, [a + b for a, b in zip(q, past)]


def _tree_lens(case):
    """Keys of the requests, the drafted tokens among them, spread evenly."""
    R, T, lo, hi = (case[x] for x in ("R", "T", "lo", "hi"))
    lo = max(T, min(lo, hi))
    return [lo + ((hi - lo) * i) // max(1, R - 1) if R > 1 else hi for i in range(R)]


def _parents(case):
    """The drafted token that each one follows (-1: the last token before them): a tree of even breadth."""
    return [(t - 1) // case["breadth"] if t else -1 for t in range(case["T"])]


def _seen(case):
    """[T][T] truth values: the drafted tokens that each one sees, itself and those that it follows."""
    T, parents = case["T"], _parents(case)
    rows = []
    for t in range(T):
        row = list(rows[parents[t]]) if parents[t] >= 0 else [False] * T
        row[t] = True
        rows.append(row)
    return rows


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device=DEV, dtype=torch.float32).to(torch.bfloat16)


def _starts(lens):
    return torch.tensor([0] + lens, dtype=torch.int64).cumsum(0).to(torch.int32).to(DEV)


def prepare(case, seed):
    g = torch.Generator(DEV).manual_seed(seed)
    s = dict(case)
    d, Hq, Hk, R = case["d"], case["Hq"], case["Hk"], case["R"]
    order = torch.randperm(R, generator=torch.Generator().manual_seed(seed)).tolist()
    s["scale"] = 1.0 / math.sqrt(d)
    if case["op"] == "tree":
        T, page = case["T"], case["page"]
        lens = [_tree_lens(case)[i] for i in order]
        s["host_lens"], s["lens"] = lens, torch.tensor(lens, dtype=torch.int32, device=DEV)
        need = [(n + page - 1) // page for n in lens]
        # the pages of all requests in the order in which a cache in use would have given them out
        total = sum(need)
        ids = torch.randperm(total, generator=g, device=DEV).to(torch.int32)
        s["table"] = torch.zeros((R, max(need)), dtype=torch.int32, device=DEV)
        first = 0
        for r, n in enumerate(need):
            s["table"][r, :n] = ids[first:first + n]
            first += n
        if case["token_major"]:
            s["kc"], s["vc"] = (_randn(g, total, page, Hk, d).transpose(1, 2) for _ in range(2))
        else:
            s["kc"], s["vc"] = (_randn(g, total, Hk, page, d) for _ in range(2))
        s["q"] = _randn(g, R, T, Hq, d).transpose(1, 2)
        seen = torch.tensor(_seen(case), dtype=torch.bool)
        s["seen"] = seen.to(DEV).expand(R, T, T).contiguous()
        # the same as the rows of bits that the entry point takes, made once a tree is drafted
        words = (T + 31) // 32
        bits = torch.zeros((T, words * 32), dtype=torch.int64)
        bits[:, :T] = seen.long()
        bits = (bits.view(T, words, 32) << torch.arange(32)).sum(-1)
        s["bits"] = torch.where(bits >= 1 << 31, bits - (1 << 32), bits).to(torch.int32).to(DEV).expand(R, T, words).contiguous()
        s["out"] = torch.empty((R, T, Hq, d), dtype=torch.bfloat16, device=DEV).transpose(1, 2)
        s["lse"] = torch.empty((R, Hq, T), dtype=torch.float32, device=DEV)
        return s
    ql, kl = _lens(case)
    ql, kl = [ql[i] for i in order], [kl[i] for i in order]
    s["ql"], s["kl"] = ql, kl
    s["q_starts"] = _starts(ql)
    s["k_starts"] = None if ql == kl else _starts(kl)
    Nq, Nk = sum(ql), sum(kl)
    if case["fused"]:  # views of the projection's output [tokens, (Hq + 2 Hk) d]
        qkv = _randn(g, Nq, Hq + 2 * Hk, d)
        s["q"], s["k"], s["v"] = (x.transpose(0, 1) for x in qkv.split([Hq, Hk, Hk], 1))
    else:
        s["q"] = _randn(g, Nq, Hq, d).transpose(0, 1)
        s["k"], s["v"] = (_randn(g, Nk, Hk, d).transpose(0, 1) for _ in range(2))
    # outputs are token-major, as the next projection reads them
    s["out"] = torch.empty((Nq, Hq, d), dtype=torch.bfloat16, device=DEV).transpose(0, 1)
    s["lse"] = torch.empty((Hq, Nq), dtype=torch.float32, device=DEV)
    if case["op"] == "packed_bwd":
        s["do"] = _randn(g, Nq, Hq, d).transpose(0, 1)
        s["o"], s["lse"] = _packed(s)  # the forward's, which a training step keeps
        s["dk"], s["dv"] = (torch.empty((Nk, Hk, d), dtype=torch.bfloat16, device=DEV).transpose(0, 1) for _ in range(2))
    return s


# ------------------------------------------------------------------ plain forms
def _pieces(s):
    """(queries, keys, first key of the sequence, its keys, visible) of blocks of queries whose scores fit memory; visible is
    None where all are."""
    q0 = k0 = 0
    for nq, nk in zip(s["ql"], s["kl"]):
        step = max(1, (1 << 30) // max(1, s["Hq"] * nk))
        for a in range(0, nq, step):
            b = min(nq, a + step)
            seen = None
            if s["causal"]:
                at = torch.arange(a, b, device=DEV) + (nk - nq)
                seen = torch.arange(nk, device=DEV) <= at[:, None]
            yield slice(q0 + a, q0 + b), slice(k0, k0 + nk), seen
        q0 += nq
        k0 += nk


def _packed(s):
    Hq, Hk = s["Hq"], s["Hk"]
    G, d = Hq // Hk, s["d"]
    out, lse = torch.empty_like(s["q"], memory_format=torch.contiguous_format), torch.empty(s["q"].shape[:2], device=DEV)
    for qs, ks, seen in _pieces(s):
        q = s["q"][:, qs].float().reshape(Hk, -1, d)
        x = torch.matmul(q, s["k"][:, ks].float().transpose(1, 2)).mul_(s["scale"]).view(Hq, -1, ks.stop - ks.start)
        if seen is not None:
            x.masked_fill_(~seen, -math.inf)
        m = x.amax(-1, keepdim=True)
        x.sub_(m).exp_()
        l = x.sum(-1, keepdim=True)
        o = torch.matmul(x.view(Hk, -1, x.shape[-1]), s["v"][:, ks].float()).view(Hq, -1, d)
        out[:, qs] = (o / l).to(torch.bfloat16)
        lse[:, qs] = (m + torch.log(l)).squeeze(-1)
    return out, lse


def _packed_bwd(s):
    Hq, Hk = s["Hq"], s["Hk"]
    d = s["d"]
    dq = torch.empty_like(s["q"], memory_format=torch.contiguous_format)
    dk, dv = (torch.zeros(s["k"].shape, device=DEV) for _ in range(2))
    for qs, ks, seen in _pieces(s):
        nk = ks.stop - ks.start
        q, do = (s[x][:, qs].float().reshape(Hk, -1, d) for x in ("q", "do"))
        k, v = s["k"][:, ks].float(), s["v"][:, ks].float()
        p = torch.matmul(q, k.transpose(1, 2)).mul_(s["scale"]).view(Hq, -1, nk)
        p.sub_(s["lse"][:, qs, None]).exp_()
        if seen is not None:
            p.masked_fill_(~seen, 0)
        p = p.view(Hk, -1, nk)
        dv[:, ks] += torch.matmul(p.transpose(1, 2), do)
        delta = (do * s["o"][:, qs].float().reshape(Hk, -1, d)).sum(-1, keepdim=True)
        ds = torch.matmul(do, v.transpose(1, 2)).sub_(delta).mul_(p).mul_(s["scale"])
        del p
        dq[:, qs] = torch.matmul(ds, k).view(Hq, -1, d).to(torch.bfloat16)
        dk[:, ks] += torch.matmul(ds.transpose(1, 2), q)
        del ds
    return dq, dk.to(torch.bfloat16), dv.to(torch.bfloat16)


def _tree(s):
    R, Hq, T, d = s["q"].shape
    Hk, page = s["Hk"], s["page"]
    G = Hq // Hk
    C = s["table"].shape[1] * page
    k, v = (s[x][s["table"]].permute(0, 2, 1, 3, 4).reshape(R, Hk, C, d).float() for x in ("kc", "vc"))
    q = s["q"].float().reshape(R, Hk, G * T, d)
    x = torch.matmul(q, k.transpose(2, 3)).mul_(s["scale"]).view(R, Hk, G, T, C)
    at = torch.arange(C, device=DEV) - (s["lens"] - T).view(R, 1)  # which drafted token a key is; negative: before them
    drafted = torch.gather(s["seen"], 2, at.clamp(0, T - 1).view(R, 1, C).expand(R, T, C))
    seen = (at < 0).view(R, 1, C) | (drafted & (at < T).view(R, 1, C))
    x.masked_fill_(~seen.view(R, 1, 1, T, C), -math.inf)
    m = x.amax(-1, keepdim=True)
    x.sub_(m).exp_()
    l = x.sum(-1, keepdim=True)
    o = torch.matmul(x.view(R, Hk, G * T, C), v).view(R, Hk, G, T, d) / l
    return o.view(R, Hq, T, d).to(torch.bfloat16), (m + torch.log(l)).view(R, Hq, T)


def run(s):
    if own:
        import exact_long_sequence_gb300 as ela

        if s["op"] == "packed":
            return ela.attn_fwd_packed(s["q"], s["k"], s["v"], s["q_starts"], s["k_starts"], causal=s["causal"], out=s["out"],
                                       lse=s["lse"])
        if s["op"] == "packed_bwd":
            return ela.attn_bwd_packed(s["q"], s["k"], s["v"], s["o"], s["lse"], s["do"], s["q_starts"], s["k_starts"],
                                       causal=s["causal"], dq=s["out"], dk=s["dk"], dv=s["dv"])
        return ela.attn_fwd_tree(s["q"], s["kc"], s["vc"], s["table"], s["lens"], s["bits"], out=s["out"], lse=s["lse"])
    return {"packed": _packed, "packed_bwd": _packed_bwd, "tree": _tree}[s["op"]](s)


def work(case):
    d, Hq, Hk = case["d"], case["Hq"], case["Hk"]
    if case["op"] == "tree":
        R, T = case["R"], case["T"]
        lens = _tree_lens(case)
        seen = sum(map(sum, _seen(case)))
        rows = R * Hq * T
        pages = sum((n + case["page"] - 1) // case["page"] for n in lens)
        return {"bytes": 2 * 2 * d * Hk * sum(lens) + rows * (2 * 2 * d + 4) + 4 * (pages + R + R * T * ((T + 31) // 32)),
                "flops": 4 * d * Hq * sum(T * (n - T) + seen for n in lens)}
    ql, kl = _lens(case)
    pairs = 0
    for nq, nk in zip(ql, kl):
        pairs += nq * nk - (nq * (nq - 1) // 2 if case["causal"] else 0)
    Nq, Nk = sum(ql), sum(kl)
    x = 2 if case["op"] == "packed" else 4  # q and o; in the gradient q, o, do and dq (and k, v, dk, dv)
    return {"bytes": 2 * x * d * (Nq * Hq) + x * 2 * d * Nk * Hk + 4 * Nq * Hq + 8 * (case["R"] + 1),
            "flops": (4 if case["op"] == "packed" else 10) * d * Hq * pairs}


# ------------------------------------------------------------------ the definitions in 64 bits
def _rows(s, h, i):
    """Query head h of sequence i: where its queries and keys lie, and the number of keys that each query sees."""
    q0, k0, nq, nk = sum(s["ql"][:i]), sum(s["kl"][:i]), s["ql"][i], s["kl"][i]
    t = torch.arange(nq, device=DEV)
    return q0, k0, nq, nk, (t + 1 + nk - nq if s["causal"] else torch.full_like(t, nk))


def exact(case, seed):
    w = work(case)
    if w["flops"] > 8e12:
        return None
    s = prepare(case, seed)
    wide = lambda x: x.to(torch.float64)  # noqa: E731
    d, Hq, Hk = case["d"], case["Hq"], case["Hk"]
    G = Hq // Hk
    f64 = dict(dtype=torch.float64, device=DEV)
    if case["op"] == "tree":
        T, page = case["T"], case["page"]
        out, lse = torch.zeros(s["q"].shape, **f64), torch.zeros(s["lse"].shape, **f64)
        parents = _parents(case)
        for r, n in enumerate(s["host_lens"]):
            ids = s["table"][r, : (n + page - 1) // page].long()
            k, v = (wide(s[x][ids]).transpose(0, 1).flatten(1, 2)[:, :n] for x in ("kc", "vc"))
            hidden = torch.zeros((T, n), dtype=torch.bool, device=DEV)
            for t in range(T):
                path, at = set(), t
                while at >= 0:
                    path.add(at)
                    at = parents[at]
                for j in set(range(T)) - path:
                    hidden[t, n - T + j] = True
            for h in range(Hq):
                z = (wide(s["q"][r, h]) @ k[h // G].T) / math.sqrt(d)
                z[hidden] = -math.inf
                lse[r, h] = torch.logsumexp(z, -1)
                out[r, h] = torch.softmax(z, -1) @ v[h // G]
        return out, lse
    step = 2048
    if case["op"] == "packed":
        out, lse = torch.zeros(s["q"].shape, **f64), torch.zeros(s["q"].shape[:2], **f64)
    else:
        dq, dk, dv = (torch.zeros(s[x].shape, **f64) for x in ("q", "k", "v"))
    for i in range(case["R"]):
        for h in range(Hq):
            q0, k0, nq, nk, sees = _rows(s, h, i)
            for a in range(0, nq, step):
                rows = slice(q0 + a, q0 + min(nq, a + step))
                most = min(nk, int(sees[a: a + step].max()))
                keys = slice(k0, k0 + most)
                k, v = wide(s["k"][h // G, keys]), wide(s["v"][h // G, keys])
                q = wide(s["q"][h, rows])
                z = q @ k.T / math.sqrt(d)
                z[torch.arange(most, device=DEV) >= sees[a: a + step, None]] = -math.inf
                if case["op"] == "packed":
                    lse[h, rows] = torch.logsumexp(z, -1)
                    out[h, rows] = torch.softmax(z, -1) @ v
                    continue
                p = torch.exp(z - wide(s["lse"][h, rows])[:, None])
                g = wide(s["do"][h, rows])
                dv[h // G, keys] += p.T @ g
                ds = p * (g @ v.T - (g * wide(s["o"][h, rows])).sum(-1, keepdim=True)) / math.sqrt(d)
                dq[h, rows] = ds @ k
                dk[h // G, keys] += ds.T @ q
    return (out, lse) if case["op"] == "packed" else (dq, dk, dv)
