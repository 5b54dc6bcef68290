"""What lies between a layer's projections and its attention, and the attention over a latent cache, as measured cases.

Five operators of one engine step.  "rope": queries and keys normed head by head, rotated by their positions, keys and
values written to the paged cache.  "latent": the same for a latent cache -- one 512-dim latent and one 64-dim rotated
key a token, shared by all heads.  "absorbed": attention over the paged latent cache by queries that took the key
expansion into them.  "expand": a request's cached latents expanded to keys and values of every head.  "expanded":
causal attention of prefill chunks over such keys and values.  ``run`` computes them in plain torch, or, with ``own``
set, through the framework's entry points.
"""
import math
import random

import torch

own = False

BS, D = 16, 128            # tokens a block; head dim of the grouped-query cache
LAT, ROPE = 512, 64        # a cached row: latent and rotated key
NOPE, VAL = 128, 128       # an expanded head: unrotated key and value
EPS = 1e-6


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # the benchmark's decode batch, one token a request: latency only
        dict(name="rope 64 decode", op="rope", reqs=64, chunks=0, chunk=1, lo=512, hi=512, hq=12, hkv=2, rot=128,
             norm=True, inter=False),
        # a prefill step: 8 chunks of 512 after odd prefixes
        dict(name="rope 8x512", op="rope", reqs=8, chunks=8, chunk=512, lo=517, hi=4601, hq=32, hkv=8, rot=128,
             norm=True, inter=False),
        # a decode batch over a latent cache, few heads
        dict(name="latent 64 decode", op="latent", reqs=64, chunks=0, chunk=1, lo=100, hi=2000, hq=16, inter=True,
             norm=True),
        # a prefill step's latents, and the rotated part of 128 heads' queries
        dict(name="latent 8x512", op="latent", reqs=8, chunks=8, chunk=512, lo=517, hi=4601, hq=128, inter=True,
             norm=True),
        # a handful of short chats: the smallest decode step
        dict(name="absorbed 4 short", op="absorbed", reqs=4, chunks=0, chunk=1, lo=17, hi=128, hq=16),
        # ragged requests that check four draft tokens each
        dict(name="absorbed 32 drafts", op="absorbed", reqs=32, chunks=32, chunk=4, lo=100, hi=3001, hq=32),
        # a large batch with many heads: tensor core and memory nearly in balance
        dict(name="absorbed 64x4096", op="absorbed", reqs=64, chunks=0, chunk=1, lo=4096, hi=4096, hq=128),
        # few requests with long documents, few heads: memory
        dict(name="absorbed 8x32768", op="absorbed", reqs=8, chunks=0, chunk=1, lo=32768, hi=32768, hq=16),
        # one odd context expanded
        dict(name="expand 701", op="expand", reqs=1, chunks=0, chunk=1, lo=701, hi=701, hq=16),
        # the contexts of a prefill step expanded
        dict(name="expand 8x", op="expand", reqs=8, chunks=0, chunk=1, lo=512, hi=4608, hq=32),
        # small odd chunks, one request only decoding
        dict(name="expanded 3 odd", op="expanded", reqs=4, chunks=3, chunk=61, lo=33, hi=701, hq=16),
        # chunked prefill after prefixes of up to 4096 tokens: tensor core
        dict(name="expanded 8x512", op="expanded", reqs=8, chunks=8, chunk=512, lo=512, hi=4608, hq=32),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "latent", "absorbed", "absorbed", "expand", "expanded", "expanded"])
    kind = rng.choice(["decode", "draft", "prefill", "mixed"])
    if op in ("rope", "latent"):
        n = _log(rng, 1, 256 if kind in ("decode", "draft") else 16)
        chunk = {"decode": 1, "draft": rng.randint(2, 9)}.get(kind) or _log(rng, 10, max(10, 4096 // n))
        chunks = 0 if kind == "decode" else rng.randint(1, n) if kind == "mixed" else n
        lo = _log(rng, 1, 1000)
        case = dict(op=op, reqs=n, chunks=chunks, chunk=chunk, lo=lo, hi=lo + _log(rng, 1, 30000),
                    inter=rng.random() < 0.5, norm=rng.random() < 0.8)
        if op == "latent":
            return dict(case, hq=_log(rng, 1, 128))
        hkv = rng.randint(1, 8)
        return dict(case, hkv=hkv, hq=hkv * rng.randint(1, 4), rot=rng.choice([32, 64, 96, 128, 128]))
    if op == "expand":
        hq = _log(rng, 1, 64)
        n = _log(rng, 1, 32)
        hi = _log(rng, 1, max(1, min(8192, 440000 // (hq * n))))
        return dict(op=op, reqs=n, chunks=0, chunk=1, lo=_log(rng, max(1, hi // 16), hi), hi=hi, hq=hq)
    if op == "absorbed":
        hq = _log(rng, 1, 128)
        n = _log(rng, 1, 128 if kind in ("decode", "draft") else 8)
        hi = _log(rng, 20, max(20, min(32768, 260000 // n)))
        chunk = {"decode": 1, "draft": rng.randint(2, 9)}.get(kind) or _log(rng, 10, max(10, min(hi, 256)))
        # rows times keys within the largest listed case's
        while n * chunk * hq * hi > 64 * 128 * 4096:
            hi = max(20, hi // 2)
            chunk = max(1, min(chunk, hi) * 3 // 4)
            if hi == 20 and chunk == 1:
                break
    else:
        hq = _log(rng, 1, 64)
        n = _log(rng, 1, 24)
        hi = _log(rng, 20, max(20, min(8192, 500000 // (n * hq))))
        chunk = _log(rng, 1, min(hi, 2048))
        while n * chunk * hq * hi > 8 * 512 * 32 * 1800:
            hi = max(20, hi // 2)
            chunk = max(1, min(chunk, hi) * 3 // 4)
            if hi == 20 and chunk == 1:
                break
    chunks = 0 if kind == "decode" else rng.randint(1, n) if kind == "mixed" else n
    return dict(op=op, reqs=n, chunks=chunks, chunk=chunk, lo=_log(rng, max(1, hi // 16), hi), hi=hi, hq=hq)


def _shape(case):
    """The requests of a case, as a batch of that kind has them: (new tokens, length with them) of each."""
    rng = random.Random(repr(sorted((k, v) for k, v in case.items() if k != "name")))
    n, lo, hi = case["reqs"], case["lo"], case["hi"]
    lens = [int(round(lo * (hi / lo) ** ((i + 0.5) / n))) for i in range(n)]
    rng.shuffle(lens)
    long = set(rng.sample(range(n), case["chunks"]))
    return [(min(case["chunk"] if i in long else 1, b), b) for i, b in enumerate(lens)]


def _cdiv(a, b):
    return -(-a // b)


def work(case):
    shape = _shape(case)
    rows, keys, hq = sum(q for q, _ in shape), sum(n for _, n in shape), case["hq"]
    seen = sum(q * (n - q) + q * (q + 1) // 2 for q, n in shape)
    blocks = sum(_cdiv(n, BS) for _, n in shape)
    if case["op"] == "rope":
        hkv, rot = case["hkv"], case["rot"]
        return {"bytes": rows * ((hq + 2 * hkv) * D * 4 + rot * 4 + 16), "flops": rows * (hq + hkv) * (4.0 * D + 3 * rot)}
    if case["op"] == "latent":
        return {"bytes": rows * ((LAT + ROPE + hq * ROPE) * 4 + ROPE * 4 + 16),
                "flops": rows * (4.0 * LAT + 3.0 * ROPE * (hq + 1))}
    if case["op"] == "absorbed":
        return {"bytes": keys * (LAT + ROPE) * 2 + rows * hq * (2 * LAT + ROPE) * 2 + blocks * 4 + len(shape) * 8,
                "flops": 2.0 * hq * seen * (2 * LAT + ROPE)}
    if case["op"] == "expand":
        return {"bytes": keys * (LAT + 2 * ROPE + hq * (NOPE + VAL)) * 2 + hq * (NOPE + VAL) * LAT * 2 + blocks * 4,
                "flops": 2.0 * keys * hq * (NOPE + VAL) * LAT}
    return {"bytes": rows * hq * (NOPE + ROPE + VAL) * 2 + keys * (hq * (NOPE + VAL) + ROPE) * 2 + len(shape) * 12,
            "flops": 2.0 * hq * seen * (NOPE + ROPE + VAL)}


# ------------------------------------------------------------------- the inputs
def _ints(v, dtype=torch.int32):
    return torch.tensor(v, dtype=dtype).cuda()


def _starts(v):
    s = [0]
    for a in v:
        s.append(s[-1] + a)
    return s


def _table(n, rot):
    """cos | sin of n positions, as a model's start makes them once."""
    f = 10000.0 ** (-torch.arange(0, rot, 2, device="cuda", dtype=torch.float64) / rot)
    a = torch.arange(n, device="cuda", dtype=torch.float64)[:, None] * f
    return torch.cat([a.cos(), a.sin()], 1).float()


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    host = torch.Generator().manual_seed(seed)
    shape = _shape(case)
    q, lens = [a for a, _ in shape], [b for _, b in shape]
    op, hq, rows = case["op"], case["hq"], sum(q)
    st = dict(case, rows=rows, qmax=max(q), kmax=max(lens))

    def normal(*size, of=1.0):
        return (torch.randn(*size, device="cuda", generator=gen) * of).bfloat16()

    st["lens"], st["qsl"] = _ints(lens), _ints(_starts(q))
    # the physical blocks of every request, in no order
    cols = _cdiv(max(lens), BS)
    need = sum(_cdiv(a, BS) for a in lens)
    nb = need + need // 4 + 4
    table = torch.full((len(q), cols), -1, dtype=torch.int32)
    table[torch.arange(cols)[None, :] < torch.tensor([_cdiv(a, BS) for a in lens])[:, None]] = \
        torch.randperm(nb, generator=host).to(torch.int32)[:need]
    st["table"] = table.cuda()
    if op in ("rope", "latent"):
        pos = torch.cat([torch.arange(b - a, b) for a, b in shape])
        req = torch.repeat_interleave(torch.arange(len(q)), torch.tensor(q))
        st["pos"] = pos.cuda()
        st["slots"] = (table[req, pos // BS].long() * BS + pos % BS).cuda()
    if op == "rope":
        # queries, keys and values side by side, as one projection leaves them
        hkv = case["hkv"]
        st["cos_sin"] = _table(max(lens), case["rot"])
        qkv = normal(rows, hq + 2 * hkv, D, of=2.0)
        st["q"], st["k"], st["v"] = qkv.split([hq, hkv, hkv], 1)
        st["wq"], st["wk"] = [(1 + 0.2 * torch.randn(D, device="cuda", generator=gen)).bfloat16() if case["norm"] else None
                              for _ in range(2)]
        st["k_pool"], st["v_pool"] = normal(nb, hkv, BS, D), normal(nb, hkv, BS, D)
        st["out"] = torch.empty(rows, hq, D, device="cuda", dtype=torch.bfloat16)
        return st
    if op == "latent":
        st["cos_sin"] = _table(max(lens), ROPE)
        st["kv"] = normal(rows, LAT + ROPE, of=2.0)
        st["w"] = (1 + 0.2 * torch.randn(LAT, device="cuda", generator=gen)).bfloat16() if case["norm"] else None
        # the queries' projection, [unrotated | to be rotated] a head, and the absorbed queries' buffer
        st["q_rope"] = normal(rows, hq, NOPE + ROPE)[:, :, NOPE:]
        st["q"] = normal(rows, hq, LAT + ROPE)
        st["pool"] = normal(nb, BS, LAT + ROPE)
        return st
    st["scale"] = (NOPE + ROPE) ** -0.5
    if op in ("absorbed", "expand"):
        st["pool"] = normal(nb, BS, LAT + ROPE)
    if op in ("expand", "expanded"):
        st["ksl"] = _ints(_starts(lens))
    if op == "expand":
        st["w"] = normal(hq, NOPE + VAL, LAT, of=LAT ** -0.5)
        st["kv"] = torch.empty(sum(lens), hq, NOPE + VAL, device="cuda", dtype=torch.bfloat16)
        st["k_rope"] = torch.empty(sum(lens), ROPE, device="cuda", dtype=torch.bfloat16)
        return st
    if op == "absorbed":
        st["q"] = normal(rows, hq, LAT + ROPE)
        st["out"] = torch.empty(rows, hq, LAT, device="cuda", dtype=torch.bfloat16)
    else:
        st["q"] = normal(rows, hq, NOPE + ROPE)
        st["kv"], st["k_rope"] = normal(sum(lens), hq, NOPE + VAL), normal(sum(lens), ROPE)
        st["out"] = torch.empty(rows, hq, VAL, device="cuda", dtype=torch.bfloat16)
    if own:
        import paged_kv_cache_195_gb300 as pkv

        st["ws"] = pkv.LatentWorkspace(rows, hq, len(q))
    return st


# ------------------------------------------------------------------- the plain forms
def _norm(x, w):
    x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
    return x * w.float()


def _rotate(x, cos, sin, inter):
    """The leading dims of x, as many as cos and sin have together, rotated in pairs."""
    r = cos.shape[-1]
    if inter:
        a, b = x[..., 0:2 * r:2], x[..., 1:2 * r:2]
    else:
        a, b = x[..., :r], x[..., r:2 * r]
    u, v = a * cos - b * sin, b * cos + a * sin
    y = torch.stack([u, v], -1).flatten(-2) if inter else torch.cat([u, v], -1)
    return torch.cat([y, x[..., 2 * r:]], -1)


def _rope(s):
    cos, sin = s["cos_sin"][s["pos"]].chunk(2, 1)
    out = []
    for x, w in ((s["q"], s["wq"]), (s["k"], s["wk"])):
        x = x.float()
        out.append(_rotate(x if w is None else _norm(x, w), cos[:, None], sin[:, None], s["inter"]).bfloat16())
    s["out"].copy_(out[0])
    s["k_pool"][s["slots"] // BS, :, s["slots"] % BS] = out[1]
    s["v_pool"][s["slots"] // BS, :, s["slots"] % BS] = s["v"]


def _latent(s):
    cos, sin = s["cos_sin"][s["pos"]].chunk(2, 1)
    c, k = s["kv"].float().split([LAT, ROPE], 1)
    c = c if s["w"] is None else _norm(c, s["w"])
    row = torch.cat([c, _rotate(k, cos, sin, s["inter"])], 1).bfloat16()
    s["pool"].view(-1, LAT + ROPE)[s["slots"]] = row
    s["q"][:, :, LAT:] = _rotate(s["q_rope"].float(), cos[:, None], sin[:, None], s["inter"]).bfloat16()


def _softmax(s, x, k, v, last):
    """Causal attention of padded query rows x [n, heads, rows, d] over k, v [n, heads, keys, d]; row i of request r sees
    the keys up to last[r, i]."""
    j = torch.arange(k.shape[2], device=x.device)
    p = torch.matmul(x, k.transpose(2, 3)).mul_(s["scale"])
    p.masked_fill_(j > last[:, None, :, None], -math.inf)
    p.sub_(p.amax(3, keepdim=True)).exp_()
    return torch.matmul(p, v).div_(p.sum(3, keepdim=True))


def _rows(s):
    """Of each query row: its request and its place among the request's new tokens."""
    i = torch.arange(s["rows"], device=s["qsl"].device)
    r = torch.searchsorted(s["qsl"][1:].long(), i, right=True)
    return r, i - s["qsl"].long()[r]


def _padded(s):
    """The query rows in 32 bits, [n, qmax, heads, d], and the last key that each sees, [n, qmax]."""
    r, i = _rows(s)
    q = s["q"].float()
    x = torch.zeros(s["lens"].numel(), s["qmax"], *q.shape[1:], device=q.device)
    x[r, i] = q
    new = s["qsl"][1:] - s["qsl"][:-1]
    return x, (s["lens"] - new)[:, None] + torch.arange(s["qmax"], device=q.device)


def _absorbed(s):
    n, hq = s["lens"].numel(), s["hq"]
    c = s["pool"][s["table"].long().clamp(min=0)].float().reshape(n, 1, -1, LAT + ROPE)
    x, last = _padded(s)
    # the heads share the keys: (token, head) pairs are the rows of one product
    o = _softmax(s, x.reshape(n, 1, -1, LAT + ROPE), c, c[..., :LAT], last.repeat_interleave(hq, 1))
    r, i = _rows(s)
    s["out"].copy_(o.reshape(n, s["qmax"], hq, LAT)[r, i].bfloat16())


def _cached(s):
    """The cached rows of all requests, one after the other."""
    i = torch.arange(s["kv"].shape[0], device="cuda")
    r = torch.searchsorted(s["ksl"][1:].long(), i, right=True)
    j = i - s["ksl"].long()[r]
    return s["pool"][s["table"][r, j // BS].long(), j % BS]


def _expand(s):
    c = _cached(s)
    s["kv"].copy_(torch.matmul(c[:, :LAT].float(), s["w"].float().reshape(-1, LAT).T).view(s["kv"].shape).bfloat16())
    s["k_rope"].copy_(c[:, LAT:])


def _expanded(s):
    n = s["lens"].numel()
    j = torch.arange(s["kmax"], device="cuda")
    at = (s["ksl"][:-1].long()[:, None] + j).clamp(max=s["kv"].shape[0] - 1)
    kv = s["kv"][at].float().transpose(1, 2)
    rope = s["k_rope"][at].float()[:, None].expand(n, s["hq"], s["kmax"], ROPE)
    x, last = _padded(s)
    o = _softmax(s, x.transpose(1, 2), torch.cat([kv[..., :NOPE], rope], 3), kv[..., NOPE:], last)
    r, i = _rows(s)
    s["out"].copy_(o.transpose(1, 2)[r, i].bfloat16())


def run(s):
    op = s["op"]
    if own:
        import paged_kv_cache_195_gb300 as pkv

        if op == "rope":
            pkv.pkv_norm_rope_append(s["q"], s["k"], s["v"], s["pos"], s["cos_sin"], s["slots"], s["k_pool"], s["v_pool"],
                                     q_weight=s["wq"], k_weight=s["wk"], eps=EPS, interleaved=s["inter"], q_out=s["out"])
        elif op == "latent":
            pkv.pkv_append_latent(s["kv"], s["pos"], s["cos_sin"], s["slots"], s["pool"], weight=s["w"], eps=EPS,
                                  interleaved=s["inter"], q_rope=s["q_rope"], q_rope_out=s["q"][:, :, LAT:])
        elif op == "absorbed":
            pkv.pkv_attention_latent(s["q"], s["pool"], s["table"], s["lens"], s["qsl"], s["scale"], out=s["out"],
                                     workspace=s["ws"])
        elif op == "expand":
            pkv.pkv_expand_latent(s["pool"], s["w"], s["table"], s["lens"], s["ksl"], s["kv"], s["k_rope"])
        else:
            pkv.pkv_attention_expanded(s["q"], s["kv"], s["k_rope"], s["lens"], s["qsl"], s["ksl"], s["scale"],
                                       out=s["out"], workspace=s["ws"])
    else:
        {"rope": _rope, "latent": _latent, "absorbed": _absorbed, "expand": _expand, "expanded": _expanded}[op](s)
    if op == "rope":
        return [s["out"], s["k_pool"], s["v_pool"]]
    if op == "latent":
        return [s["pool"], s["q"]]
    if op == "expand":
        return [s["kv"], s["k_rope"]]
    return s["out"]


# ------------------------------------------------------------------- the definitions, in 64 bits
def _turned(x, w, table, pos, inter):
    """x [tokens, heads, dims] normed by w over its dims, then turned, pair by pair, by the angle of its position."""
    x = x.double()
    if w is not None:
        x = w.double() * x / torch.sqrt(x.square().sum(2, keepdim=True) / x.shape[2] + EPS)
    y = x.clone()
    half = table.shape[1] // 2
    for i in range(half):
        a, b = (2 * i, 2 * i + 1) if inter else (i, i + half)
        c, t = table[pos, i].double()[:, None], table[pos, half + i].double()[:, None]
        y[:, :, a], y[:, :, b] = x[:, :, a] * c - x[:, :, b] * t, x[:, :, a] * t + x[:, :, b] * c
    return y


def exact(case, seed):
    s = prepare(case, seed)
    op, hq = case["op"], case["hq"]
    if op == "rope":
        k_pool, v_pool = s["k_pool"].double(), s["v_pool"].double()
        k = _turned(s["k"], s["wk"], s["cos_sin"], s["pos"], case["inter"])
        b, o = torch.div(s["slots"], BS, rounding_mode="floor"), torch.remainder(s["slots"], BS)
        k_pool[b, :, o], v_pool[b, :, o] = k, s["v"].double()
        return [_turned(s["q"], s["wq"], s["cos_sin"], s["pos"], case["inter"]), k_pool, v_pool]
    if op == "latent":
        pool, q = s["pool"].double(), s["q"].double()
        c = s["kv"][:, None, :LAT].double()
        if s["w"] is not None:
            c = s["w"].double() * c / torch.sqrt(c.square().sum(2, keepdim=True) / LAT + EPS)
        k = _turned(s["kv"][:, None, LAT:], None, s["cos_sin"], s["pos"], case["inter"])
        flat = pool.reshape(-1, LAT + ROPE)
        flat[s["slots"]] = torch.cat([c, k], 2)[:, 0]
        q[:, :, LAT:] = _turned(s["q_rope"], None, s["cos_sin"], s["pos"], case["inter"])
        return [flat.reshape(pool.shape), q]
    lens, new = [b for _, b in _shape(case)], [a for a, _ in _shape(case)]
    qsl, ksl = _starts(new), _starts(lens)
    out = torch.zeros(s["kv" if op == "expand" else "out"].shape, dtype=torch.float64, device="cuda")
    tail = torch.zeros(sum(lens), ROPE, dtype=torch.float64, device="cuda")
    for r, n in enumerate(lens):
        if op != "expanded":
            c = s["pool"][s["table"][r, :_cdiv(n, BS)].long()].double().reshape(-1, LAT + ROPE)[:n]
        if op == "expand":
            tail[ksl[r]:ksl[r + 1]] = c[:, LAT:]
            for h in range(hq):
                out[ksl[r]:ksl[r + 1], h] = c[:, :LAT] @ s["w"][h].double().T
            continue
        m = new[r]
        sees = torch.arange(n, device="cuda")[None, :] <= torch.arange(n - m, n, device="cuda")[:, None]
        for h in range(hq):
            if op == "absorbed":
                k, v = c, c[:, :LAT]
            else:
                e = s["kv"][ksl[r]:ksl[r + 1], h].double()
                k, v = torch.cat([e[:, :NOPE], s["k_rope"][ksl[r]:ksl[r + 1]].double()], 1), e[:, NOPE:]
            w = (s["q"][qsl[r]:qsl[r + 1], h].double() @ k.T) * s["scale"]
            out[qsl[r]:qsl[r + 1], h] = torch.softmax(w.masked_fill(~sees, -math.inf), 1) @ v
    return [out, tail] if op == "expand" else out
