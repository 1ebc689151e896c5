"""What is measured of the operators around the attention kernels: making queries and keys ready
for attention (normalisation of each head and rotary positions in one pass), the gradient of that
step, and attention of a batch of requests that share a long prefix.

`listed()` names the measured cases and `draw()` gives more of the same ranges.  `run()` is one
pass: in elementary torch operations, or, where `own` is set, through this package's entry points.
`exact()` is the operator's definition in 64 bits.
"""
import math

import torch

own = False

DEV = "cuda"
EPS = 1e-6


def listed():
    return [
        # one new token for each of 64 requests, far into their sequences: the smallest call of a decoding step
        dict(name="ready decode 64", op="ready", B=64, N=1, Hq=32, Hk=8, d=128, rot=128, axes="128", inter=False, fused=True,
             norm=True, far=1000000),
        # a prompt of 4096 tokens of a small model, neighbouring pairs rotated
        dict(name="ready 4096 d64", op="ready", B=1, N=4096, Hq=8, Hk=8, d=64, rot=64, axes="64", inter=True, fused=False,
             norm=True, far=0),
        # four video clips, three position axes (time, height, width), a fused projection's output
        dict(name="ready video", op="ready", B=4, N=8192, Hq=32, Hk=8, d=128, rot=128, axes="32,48,48", inter=False, fused=True,
             norm=True, far=0),
        # training on a short sequence: launch latency counts
        dict(name="ready bwd 256 d64", op="ready_bwd", B=1, N=256, Hq=1, Hk=1, d=64, rot=64, axes="64", inter=False, fused=False,
             norm=True, far=0),
        # training on one long sequence with as many key heads as query heads
        dict(name="ready bwd 16384", op="ready_bwd", B=1, N=16384, Hq=16, Hk=16, d=128, rot=128, axes="128", inter=False,
             fused=False, norm=True, far=0),
        # training on video clips
        dict(name="ready bwd video", op="ready_bwd", B=4, N=8192, Hq=32, Hk=8, d=128, rot=128, axes="32,48,48", inter=False,
             fused=True, norm=True, far=0),
        # eight short requests after a system prompt of 1000 tokens: latency
        dict(name="prefix small", op="prefix", R=8, T=1, Hq=32, Hk=8, d=128, P=1000, C=64, lo=1, token_major=False),
        # drafted tokens checked four at a time, odd lengths, one key head for each query head
        dict(name="prefix drafts d64", op="prefix", R=3, T=4, Hq=8, Hk=8, d=64, P=4097, C=300, lo=4, token_major=True),
        # 64 requests on a document of 16384 tokens, up to 1024 tokens of their own
        dict(name="prefix 64 x 16384", op="prefix", R=64, T=1, Hq=32, Hk=8, d=128, P=16384, C=1024, lo=16, token_major=False),
        # four requests on a very long document: reading the prefix is all the time
        dict(name="prefix 4 x 131071", op="prefix", R=4, T=1, Hq=64, Hk=8, d=128, P=131071, C=128, lo=1, token_major=True),
        # many requests, a single key head for all query heads
        dict(name="prefix one key head", op="prefix", R=128, T=1, Hq=16, Hk=1, d=128, P=8192, C=256, lo=0, token_major=False),
        # many requests on a long document: the matrix products are the time
        dict(name="prefix 256 x 65536", op="prefix", R=256, T=1, Hq=32, Hk=8, d=128, P=65536, C=512, lo=1, token_major=False),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["ready", "ready_bwd", "prefix", "prefix"])
    d = rng.choice([64, 128, 128])
    Hk = rng.choice([1, 2, 4, 8])
    G = rng.choice([1, 2, 4, 8])
    if op != "prefix":
        N = _log(rng, 1, min(20000, 32768 * 40 // (Hk * (G + 1))))
        B = _log(rng, 1, max(1, min(64, 32768 * 40 // (N * Hk * (G + 1)))))
        rot = rng.choice([d, d, d // 2])
        pairs = rot // 2
        A = rng.choice([1, 1, 2, 3])
        cuts = sorted(rng.sample(range(1, pairs), A - 1))
        axes = [2 * (b - a) for a, b in zip([0] + cuts, cuts + [pairs])]
        return dict(op=op, B=B, N=N, Hq=Hk * G, Hk=Hk, d=d, rot=rot, axes=",".join(map(str, axes)), inter=rng.random() < 0.4,
                    fused=rng.random() < 0.5, norm=rng.random() < 0.8, far=rng.choice([0, 0, 100000]))
    T = rng.choice([1, 1, 1, 2, 5])
    R = _log(rng, 1, 256)
    most = 256 * 32 * 65536 // 2
    P = _log(rng, 1, max(1, min(131072, most // (R * T * Hk * G))))
    C = max(T, _log(rng, 1, max(1, min(4096, 256 * 1024 * 8 // (R * Hk), most // (R * T * Hk * G)))))
    return dict(op=op, R=R, T=T, Hq=Hk * G, Hk=Hk, d=d, P=P, C=C, lo=rng.choice([0, T, T]), token_major=rng.random() < 0.5)


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device=DEV, dtype=torch.float32).to(torch.bfloat16)


def _lens(case):
    """Own lengths of the requests, spread evenly from `lo` to the caches' capacity."""
    R, lo, C = case["R"], case["lo"], case["C"]
    return [lo + ((C - lo) * i) // max(1, R - 1) if R > 1 else C for i in range(R)]


def prepare(case, seed):
    g = torch.Generator(DEV).manual_seed(seed)
    s = dict(case)
    d = case["d"]
    if case["op"] == "prefix":
        R, T, Hq, Hk, P, C = (case[x] for x in ("R", "T", "Hq", "Hk", "P", "C"))
        s["q"] = _randn(g, R, Hq, T, d)
        s["kp"], s["vp"] = _randn(g, Hk, P, d), _randn(g, Hk, P, d)
        if case["token_major"]:
            s["ko"], s["vo"] = (_randn(g, R, C, Hk, d).transpose(1, 2) for _ in range(2))
        else:
            s["ko"], s["vo"] = (_randn(g, R, Hk, C, d) for _ in range(2))
        order = torch.randperm(R, generator=g, device=DEV)
        s["lens"] = torch.tensor(_lens(case), dtype=torch.int32, device=DEV)[order].contiguous()
        # the buffers a decoding loop keeps
        s["out"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty((R, Hq, T), dtype=torch.float32, device=DEV)
        return s
    B, N, Hq, Hk = case["B"], case["N"], case["Hq"], case["Hk"]
    if case["fused"]:  # views of the projection's output [B, N, (Hq + 2 Hk) d]
        qkv = _randn(g, B, N, Hq + 2 * Hk, d)
        s["q"], s["k"] = qkv[:, :, :Hq].transpose(1, 2), qkv[:, :, Hq:Hq + Hk].transpose(1, 2)
    else:
        s["q"], s["k"] = _randn(g, B, N, Hq, d).transpose(1, 2), _randn(g, B, N, Hk, d).transpose(1, 2)
    s["sections"] = tuple(int(x) // 2 for x in case["axes"].split(","))
    A = len(s["sections"])
    start = torch.randint(0, case["far"] + 1, (B, 1), generator=g, device=DEV)
    t = start + torch.arange(N, device=DEV)
    # one axis: the token's place; more: frames of 64 x 64 patches as (time, height, width), or (height, width)
    s["pos"] = torch.stack({1: [t], 2: [t // 64, t % 64], 3: [t // 4096, t // 64 % 64, t % 64]}[A]).to(torch.int32).contiguous()
    s["inv_freq"] = 10000.0 ** (-torch.arange(case["rot"] // 2, device=DEV, dtype=torch.float64) * 2 / case["rot"])
    s["wq"] = s["wk"] = None
    if case["norm"]:
        s["wq"], s["wk"] = ((1 + 0.2 * torch.randn(d, generator=g, device=DEV)).to(torch.bfloat16) for _ in range(2))
    s["q_out"] = torch.empty((B, Hq, N, d), dtype=torch.bfloat16, device=DEV)
    s["k_out"] = torch.empty((B, Hk, N, d), dtype=torch.bfloat16, device=DEV)
    if case["op"] == "ready_bwd":
        s["dq_out"], s["dk_out"] = _randn(g, B, Hq, N, d), _randn(g, B, Hk, N, d)
    return s


# ------------------------------------------------------------------ plain forms
def _angles(s):
    """cos and sin of every token's and pair's angle, [B, 1, N, rot / 2]: 64 bits up to the angle, which is far from zero."""
    axis = torch.repeat_interleave(torch.arange(len(s["sections"]), device=DEV), torch.tensor(s["sections"], device=DEV))
    a = s["pos"].double()[axis].permute(1, 2, 0) * s["inv_freq"]
    return torch.cos(a).float()[:, None], torch.sin(a).float()[:, None]


def _pairs(x, s):
    """The first and the second members of the rotated pairs, and what is not rotated."""
    r = s["rot"]
    if s["inter"]:
        return x[..., 0:r:2], x[..., 1:r:2], x[..., r:]
    return x[..., : r // 2], x[..., r // 2: r], x[..., r:]


def _join(a, b, rest, s):
    r = torch.stack([a, b], -1).flatten(-2) if s["inter"] else torch.cat([a, b], -1)
    return torch.cat([r, rest], -1)


def _ready(x, w, cs, s):
    y = x.float()
    if w is not None:
        y = y * torch.rsqrt((y * y).mean(-1, keepdim=True) + EPS) * w.float()
    a, b, rest = _pairs(y, s)
    cos, sin = cs
    return _join(a * cos - b * sin, b * cos + a * sin, rest, s).to(torch.bfloat16)


def _ready_bwd(dy, x, w, cs, s):
    a, b, rest = _pairs(dy.float(), s)
    cos, sin = cs
    u = _join(a * cos + b * sin, b * cos - a * sin, rest, s)
    if w is None:
        return u.to(torch.bfloat16), None
    y = x.float()
    r = torch.rsqrt((y * y).mean(-1, keepdim=True) + EPS)
    h = y * r
    uw = u * w.float()
    dx = r * (uw - h * (uw * h).mean(-1, keepdim=True))
    return dx.to(torch.bfloat16), (u * h).double().sum((0, 1, 2)).float()


def _prefix(s):
    R, Hq, T, d = s["q"].shape
    Hk, P, C = s["kp"].shape[0], s["kp"].shape[1], s["ko"].shape[2]
    G = Hq // Hk
    scale = 1.0 / math.sqrt(d)
    q = s["q"].float().reshape(R, Hk, G * T, d)
    qh = q.transpose(0, 1).reshape(Hk, R * G * T, d)
    sp = torch.matmul(qh, s["kp"].float().transpose(1, 2)).reshape(Hk, R, G * T, P).transpose(0, 1) * scale
    so = torch.matmul(q, s["ko"].float().transpose(2, 3)) * scale
    last = s["lens"].view(R, 1) - (T - 1) + torch.arange(T, device=DEV)  # own keys token t sees
    seen = torch.arange(C, device=DEV) < last[..., None]  # [R, T, C]
    seen = seen[:, None, None].expand(R, 1, G, T, C).reshape(R, 1, G * T, C)
    so = so.masked_fill(~seen, -math.inf)
    m = torch.maximum(sp.amax(-1, keepdim=True), so.amax(-1, keepdim=True))
    ep, eo = torch.exp(sp - m), torch.exp(so - m)
    l = ep.sum(-1, keepdim=True) + eo.sum(-1, keepdim=True)
    o = torch.matmul(ep.transpose(0, 1).reshape(Hk, R * G * T, P), s["vp"].float()).reshape(Hk, R, G * T, d).transpose(0, 1)
    o = (o + torch.matmul(eo, s["vo"].float())) / l
    return o.reshape(R, Hq, T, d).to(torch.bfloat16), (m + torch.log(l)).reshape(R, Hq, T)


def run(s):
    if own:
        import exact_long_sequence_gb300 as ela

        if s["op"] == "prefix":
            return ela.attn_fwd_prefix(s["q"], s["kp"], s["vp"], s["ko"], s["vo"], s["lens"], out=s["out"], lse=s["lse"])
        kw = dict(q_weight=s["wq"], k_weight=s["wk"], sections=s["sections"], eps=EPS, interleaved=s["inter"])
        if s["op"] == "ready":
            return ela.qk_norm_rope(s["q"], s["k"], s["pos"], s["inv_freq"], q_out=s["q_out"], k_out=s["k_out"], **kw)
        return ela.qk_norm_rope_bwd(s["dq_out"], s["dk_out"], s["q"], s["k"], s["pos"], s["inv_freq"], dq=s["q_out"],
                                    dk=s["k_out"], **kw)
    if s["op"] == "prefix":
        return _prefix(s)
    cs = _angles(s)
    if s["op"] == "ready":
        return _ready(s["q"], s["wq"], cs, s), _ready(s["k"], s["wk"], cs, s)
    dq, dwq = _ready_bwd(s["dq_out"], s["q"], s["wq"], cs, s)
    dk, dwk = _ready_bwd(s["dk_out"], s["k"], s["wk"], cs, s)
    return dq, dk, dwq, dwk


def work(case):
    d = case["d"]
    if case["op"] == "prefix":
        R, T, Hq, Hk, P = (case[x] for x in ("R", "T", "Hq", "Hk", "P"))
        lens = _lens(case)
        kv = 2 * 2 * d * Hk * (P + sum(lens))
        rows = R * Hq * T
        seen = sum(max(0, n - t) for n in lens for t in range(T))  # own keys over all tokens
        return {"bytes": kv + rows * (2 * 2 * d + 4) + 4 * R, "flops": 4 * d * Hq * (R * T * P + seen)}
    tokens = case["B"] * case["N"]
    elements = tokens * (case["Hq"] + case["Hk"]) * d
    small = tokens * 4 * len(case["axes"].split(",")) + 8 * case["rot"] // 2 + 2 * 2 * d * case["norm"]
    if case["op"] == "ready":
        return {"bytes": 2 * 2 * elements + small, "flops": (3 + 4 * case["norm"]) * elements}
    x = 1 if case["norm"] else 0  # the inputs are read for the norm's gradient only
    return {"bytes": (2 + x) * 2 * elements + small + x * 2 * 4 * d, "flops": (3 + 12 * case["norm"]) * elements}


# ------------------------------------------------------------------ the definitions in 64 bits
def _turned(x, w, s):
    """RMS norm of each head, then each pair as a complex number times exp(i angle)."""
    y = x
    if w is not None:
        y = x / (x.pow(2).sum(-1, keepdim=True) / x.shape[-1] + EPS).sqrt() * w
    r, n = s["rot"], s["rot"] // 2
    first = torch.arange(n, device=DEV) * (2 if s["inter"] else 1)
    second = first + (1 if s["inter"] else n)
    angle = []
    for a, count in enumerate(s["sections"]):
        f = s["inv_freq"][sum(s["sections"][:a]):][:count]
        angle.append(s["pos"][a].to(torch.float64).unsqueeze(-1) * f)
    angle = torch.cat(angle, -1).unsqueeze(1)
    z = torch.complex(y[..., first], y[..., second]) * torch.polar(torch.ones_like(angle), angle)
    out = y.new_zeros(y.shape).index_copy(3, torch.cat([first, second]), torch.cat([z.real, z.imag], -1))
    return torch.cat([out[..., :r], y[..., r:]], -1)


def exact(case, seed):
    s = prepare(case, seed)
    wide = lambda x: None if x is None else x.to(torch.float64)  # noqa: E731
    if case["op"] == "ready":
        return _turned(wide(s["q"]), wide(s["wq"]), s), _turned(wide(s["k"]), wide(s["wk"]), s)
    if case["op"] == "ready_bwd":
        grads = []
        for x, w, dy in ((s["q"], s["wq"], s["dq_out"]), (s["k"], s["wk"], s["dk_out"])):
            x, w = wide(x).requires_grad_(), (None if w is None else wide(w).requires_grad_())
            y = _turned(x, w, s)
            got = torch.autograd.grad(y, [x] if w is None else [x, w], wide(dy))
            grads.append((got[0], got[1] if w is not None else None))
            del y, got
        return grads[0][0], grads[1][0], grads[0][1], grads[1][1]
    R, T, Hq, Hk, P = (case[x] for x in ("R", "T", "Hq", "Hk", "P"))
    G, d = Hq // Hk, case["d"]
    out = torch.zeros(R, Hq, T, d, dtype=torch.float64, device=DEV)
    lse = torch.zeros(R, Hq, T, dtype=torch.float64, device=DEV)
    lens = s["lens"].tolist()
    for h in range(Hk):
        kp, vp = wide(s["kp"][h]), wide(s["vp"][h])
        qs = wide(s["q"][:, h * G:(h + 1) * G]) / d ** 0.5  # [R, G, T, d]
        shared = (qs.reshape(-1, d) @ kp.T).reshape(R, G, T, P)
        for r in range(R):
            for t in range(T):
                n = max(0, lens[r] - (T - 1 - t))
                z = torch.cat([shared[r, :, t], qs[r, :, t] @ wide(s["ko"][r, h, :n]).T], -1)
                lse[r, h * G:(h + 1) * G, t] = torch.logsumexp(z, -1)
                p = torch.softmax(z, -1)
                out[r, h * G:(h + 1) * G, t] = p[:, :P] @ vp + p[:, P:] @ wide(s["vo"][r, h, :n])
        del shared
    return out, lse
