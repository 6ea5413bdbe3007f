"""Rotary positions and the paged cache: cases, inputs, plain forms and exact values.

Four operators that a prompt passes through before its keys are scored and evicted:

* ``rotate``  rotary positions of queries and keys (first ``rot`` dimensions of a head);
* ``append``  new tokens' rotated keys and their values into a paged cache, and
              their rotated queries;
* ``attend``  causal attention of the new tokens over the paged cache;
* ``gather``  rows of given positions out of the pages into contiguous arrays.

``run`` computes them in elementary torch operations, or, where ``own`` is
true, through the framework's layer. Sizes are those of the repository's
workloads (a 32-head, 8-KV-head layer of dimension 128 in bf16, contexts of
4096 to 131072, batches of 1, 4 and 64, and the tiny fp32 layer).
"""
import math

import numpy as np
import torch

own = False

TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
BASE = 500000.0
ORIG = 8192          # context length that the scaled rotations start from
FACTOR = 8.0
BAND = (1.0, 4.0)    # turns over ORIG: below the first stretched, above the second kept
RAMP = (1.0, 32.0)   # the same two borders for the ramp over the dimension's index


def _case(name, op, dtype="bf16", batch=1, new=1, kv=1, hq=32, hkv=8, d=128, page=64, ragged=False,
          rot=128, layout="half", scaling="plain", n=0):
    return {"name": name, "op": op, "dtype": dtype, "batch": batch, "new": new, "kv": kv, "hq": hq,
            "hkv": hkv, "d": d, "page": page, "ragged": ragged, "rot": rot, "layout": layout,
            "scaling": scaling, "n": n}


def listed():
    return [
        # one decode step of 64 sequences: queries and keys of 64 tokens at far positions
        _case("rotate-step", "rotate", batch=64, new=1, kv=32768),
        # the whole prompt of four 16K sequences, half of each head rotated
        _case("rotate-prompt", "rotate", batch=4, new=16384, kv=16384, rot=64, layout="interleaved",
              scaling="band"),
        # one decode step into the pages of 64 sequences
        _case("append-step", "append", batch=64, new=1, kv=2048),
        # a chunk of a ragged batch of prompts
        _case("append-chunk", "append", batch=4, new=8192, kv=16384, ragged=True, page=128,
              scaling="ramp"),
        # the smallest call: one token of one sequence
        _case("attend-one", "attend", batch=1, new=1, kv=4096),
        # a full serving batch, one token each, ragged contexts
        _case("attend-step", "attend", batch=64, new=1, kv=32768, ragged=True),
        # a few tokens each (drafted tokens checked at once), small pages
        _case("attend-few", "attend", batch=4, new=5, kv=16384, ragged=True, page=16),
        # whole prompts of a ragged batch, nothing cached before
        _case("attend-prompt", "attend", batch=4, new=4096, kv=4096, ragged=True),
        # the last chunk of a 128K prompt
        _case("attend-chunk", "attend", batch=1, new=8192, kv=131072, page=128),
        # the tiny fp32 layer's prompt
        _case("attend-fp32", "attend", dtype="fp32", batch=1, new=1024, kv=1024, hq=8, hkv=2, d=64,
              rot=64, page=16),
        # the retained tokens of four 16K sequences
        _case("gather-kept", "gather", batch=4, kv=16384, n=1024),
        # all that leaves a 128K sequence
        _case("gather-left", "gather", batch=1, kv=131072, n=117965, page=16),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """One more case of the same ranges; it costs no more than the largest listed one."""
    op = rng.choice(["rotate", "append", "attend", "attend", "attend", "gather"])
    d = rng.choice([64, 128, 128])
    hkv = rng.choice([1, 2, 4, 8, 8])
    hq = hkv * rng.choice([g for g in (1, 2, 4, 4, 8) if g * hkv <= 32])
    dtype = rng.choice(["bf16", "bf16", "bf16", "fp32"])
    page = rng.choice([16, 32, 64, 128, 256])
    rot = rng.choice([r for r in (16, 32, 64, 96, 128) if r <= d] + [d])
    while True:
        batch = _log(rng, 1, 64)
        new = 1 if op == "attend" and rng.random() < 0.3 else _log(rng, 1, 8192)
        kv = max(new, _log(rng, 64, 131072))
        n = _log(rng, 1, kv)
        pairs = batch * new * kv * (1 if dtype == "bf16" else 8)
        rows = batch * (kv if op != "rotate" else new)
        if rows > 1 << 20 or (op == "attend" and (pairs > 1 << 30 or pairs * (hq // hkv) > 1 << 32)):
            continue
        if op != "attend" and (batch * new > 1 << 16 or (op == "append" and rows > 1 << 18)):
            continue
        return {k: v for k, v in _case("", op, dtype=dtype, batch=batch, new=new, kv=kv, hq=hq, hkv=hkv,
                                       d=d, page=page, ragged=rng.random() < 0.7, rot=rot,
                                       layout=rng.choice(["half", "interleaved"]),
                                       scaling=rng.choice(["plain", "linear", "band", "ramp"]),
                                       n=n if op == "gather" else 0).items() if k != "name"}


def _lengths(c):
    """Per sequence the new tokens and the cached tokens with them."""
    b, new, past = c["batch"], c["new"], c["kv"] - c["new"]
    if not c["ragged"]:
        return [new] * b, [c["kv"]] * b
    news = [max(1, new - new * ((37 * s) % 64) // 128) for s in range(b)]
    return news, [n + past - past * ((29 * s) % 64) // 128 for s, n in enumerate(news)]


def _turns(c):
    """Radians per position of each rotated pair, in 64 bits."""
    half = c["rot"] // 2
    i = torch.arange(half, dtype=torch.float64)
    theta = torch.pow(torch.tensor(BASE, dtype=torch.float64), -2.0 * i / c["rot"])
    if c["scaling"] == "plain":
        return theta
    if c["scaling"] == "linear":
        return theta / FACTOR
    if c["scaling"] == "band":
        keep = ((ORIG * theta / (2 * math.pi) - BAND[0]) / (BAND[1] - BAND[0])).clamp(0, 1)
    else:
        at = [c["rot"] * math.log(ORIG / (2 * math.pi * t)) / (2 * math.log(BASE)) for t in RAMP]
        lo = min(max(math.floor(at[1]), 0), half - 1)
        hi = min(max(math.ceil(at[0]), 0), half - 1)
        keep = 1 - ((i - lo) / max(hi - lo, 1e-3)).clamp(0, 1)
    return theta * (keep + (1 - keep) / FACTOR)


def _magnitude(c):
    return 0.1 * math.log(FACTOR) + 1.0 if c["scaling"] == "ramp" else 1.0


_layers = {}


def _layer(c):
    """The program's layer: one handle for a shape and a rotation."""
    from learned_kv_cache_indexmem_b200 import synth
    from learned_kv_cache_indexmem_b200.layer import IndexMemLayer
    key = tuple(c[k] for k in ("dtype", "hq", "hkv", "d", "rot", "layout", "scaling"))
    if key not in _layers:
        shape = synth.LayerShape(hidden=512, n_q_heads=c["hq"], n_kv_heads=c["hkv"], head_dim=c["d"],
                                 idx_dim=32, mem_r=32, lam=0.99, dtype=c["dtype"])
        lay = IndexMemLayer.from_shape(shape, synth.make_weights(shape, 0, "cuda"))
        low, high = RAMP if c["scaling"] == "ramp" else BAND
        lay.set_rope(rot_dim=c["rot"], base=BASE, layout=c["layout"], scaling=c["scaling"], factor=FACTOR,
                     low=low, high=high, orig_len=ORIG, magnitude=_magnitude(c))
        _layers[key] = lay
    return _layers[key]


def prepare(case, seed):
    c, dev = case, torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    dt, b, d, hq, hkv, page = TYPES[c["dtype"]], c["batch"], c["d"], c["hq"], c["hkv"], c["page"]
    news, lens = _lengths(c)
    s = {"case": c}

    def ints(v):
        return torch.tensor(v, dtype=torch.int32, device=dev)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=dev, dtype=dt)

    if c["op"] in ("rotate", "append", "attend"):
        T = sum(news)
        starts = np.concatenate([[0], np.cumsum(news)])
        # one row per token of the joint projection: queries, keys and values side by side
        qkv = normal(T, (hq + 2 * hkv) * d)
        s["q"] = qkv[:, :hq * d].view(T, hq, d)
        s["k"] = qkv[:, hq * d:(hq + hkv) * d].view(T, hkv, d)
        s["v"] = qkv[:, (hq + hkv) * d:].view(T, hkv, d)
        s["start"] = ints(starts)
        s["theta"], s["magnitude"] = _turns(c).to(dev), _magnitude(c)
        s["positions"] = ints(np.concatenate([np.arange(l - n, l) for n, l in zip(news, lens)]))
    if c["op"] != "rotate":
        # the cache: the sequences' pages in any order among a few free ones
        per = -(-c["kv"] // page)
        pages = b * per + 7
        s["K"], s["V"] = normal(pages, page, hkv, d), normal(pages, page, hkv, d)
        order = torch.randperm(pages, generator=g, device=dev)[:b * per]
        s["table"] = order.to(torch.int32).view(b, per).contiguous()
        s["len"] = ints(lens)
        if c["op"] != "append":
            # heavy hitters: 1 % of the rows with three times the key
            s["K"] *= 1 + 2 * (torch.rand(pages, page, 1, 1, generator=g, device=dev) < 0.01).to(dt)
    if c["op"] == "gather":
        at = [torch.randperm(l, generator=g, device=dev)[:min(c["n"], l)].sort().values for l in lens]
        n = min(len(a) for a in at)
        s["idx"] = torch.stack([a[:n] for a in at]).to(torch.int32).contiguous()
    s["max_new"], s["max_len"] = max(news), max(lens)
    if own:
        s["layer"] = _layer(c)
        if c["op"] != "rotate":
            from learned_kv_cache_indexmem_b200.layer import PagedCache
            s["cache"] = PagedCache(s["K"], s["V"], s["table"], s["len"])
    return s


# ------------------------------------------------------------------ plain forms

def _rotated(x, s, c):
    a = s["positions"].double()[:, None] * s["theta"][None]
    cos = (a.cos() * s["magnitude"]).float()[:, None]
    sin = (a.sin() * s["magnitude"]).float()[:, None]
    half, x32 = c["rot"] // 2, x.float()
    y = x32.clone()
    if c["layout"] == "half":
        x1, x2 = x32[..., :half], x32[..., half:2 * half]
        y[..., :half], y[..., half:2 * half] = x1 * cos - x2 * sin, x2 * cos + x1 * sin
    else:
        x1, x2 = x32[..., 0:2 * half:2], x32[..., 1:2 * half:2]
        y[..., 0:2 * half:2], y[..., 1:2 * half:2] = x1 * cos - x2 * sin, x2 * cos + x1 * sin
    return y.to(x.dtype)


def _token_of(s, T):
    """The sequence of each token, and its place among that sequence's new tokens."""
    t = torch.arange(T, device=s["start"].device, dtype=torch.int32)
    seq = torch.searchsorted(s["start"], t, right=True) - 1
    return seq, t - s["start"][seq]


def _append_plain(s, c):
    seq, i = _token_of(s, s["k"].shape[0])
    pos = (s["len"] - (s["start"][1:] - s["start"][:-1]))[seq] + i
    row = s["table"][seq, (pos // c["page"]).long()].long() * c["page"] + pos % c["page"]
    s["K"].view(-1, c["hkv"], c["d"])[row] = _rotated(s["k"], s, c)
    s["V"].view(-1, c["hkv"], c["d"])[row] = s["v"]
    return {"q": _rotated(s["q"], s, c), "K": s["K"], "V": s["V"]}


def _attend_plain(s, c):
    T, b, G, L, N = s["q"].shape[0], c["batch"], c["hq"] // c["hkv"], s["max_len"], s["max_new"]
    n = s["start"][1:] - s["start"][:-1]
    i = torch.arange(N, device=n.device)
    padded = s["q"][(s["start"][:-1, None] + i).clamp(max=T - 1).long()].float()     # [b, N, hq, d]
    seen = torch.arange(L, device=n.device) <= ((s["len"] - n)[:, None] + i)[..., None]  # [b, N, L]
    outs, lses = [], []
    for h in range(c["hkv"]):
        k = s["K"][:, :, h][s["table"].long()].flatten(1, 2)[:, :L].float()
        v = s["V"][:, :, h][s["table"].long()].flatten(1, 2)[:, :L].float()
        x = padded[:, :, h * G:(h + 1) * G].reshape(b, N * G, -1) @ k.transpose(1, 2)
        x = x.mul_(1 / math.sqrt(c["d"])).view(b, N, G, L).masked_fill_(~seen[:, :, None], -math.inf)
        m = x.amax(-1, keepdim=True)
        x = x.sub_(m).exp_()
        total = x.sum(-1, keepdim=True)
        outs.append((x.view(b, N * G, L) @ v).view(b, N, G, -1) / total)
        lses.append((m + total.log())[..., 0])
    seq, i = _token_of(s, T)
    return {"out": torch.cat(outs, 2)[seq, i.long()].to(s["q"].dtype), "lse": torch.cat(lses, 2)[seq, i.long()]}


def _gather_plain(s, c):
    at = s["idx"].long()
    row = s["table"].long().gather(1, at // c["page"]) * c["page"] + at % c["page"]
    return {"K": s["K"].view(-1, c["hkv"], c["d"])[row], "V": s["V"].view(-1, c["hkv"], c["d"])[row]}


def run(state):
    s, c = state, state["case"]
    if own:
        lay = s["layer"]
        if c["op"] == "rotate":
            q, k = lay.rotate(s["q"], s["k"], s["positions"])
            return {"q": q, "k": k}
        if c["op"] == "append":
            q = lay.append_paged(s["k"], s["v"], s["cache"], tok_start=s["start"], q=s["q"])
            return {"q": q, "K": s["K"], "V": s["V"]}
        if c["op"] == "attend":
            out, lse = lay.attend_paged(s["q"], s["cache"], tok_start=s["start"], max_new=s["max_new"],
                                        max_len=s["max_len"], return_lse=True)
            return {"out": out, "lse": lse}
        K, V = lay.gather_paged(s["cache"], s["idx"])
        return {"K": K, "V": V}
    if c["op"] == "rotate":
        return {"q": _rotated(s["q"], s, c), "k": _rotated(s["k"], s, c)}
    return {"append": _append_plain, "attend": _attend_plain, "gather": _gather_plain}[c["op"]](s, c)


# ------------------------------------------------------------------------- work

def work(case):
    c, e = case, 2 if case["dtype"] == "bf16" else 4
    news, lens = _lengths(c)
    T, row = sum(news), c["d"] * e
    q, kv = c["hq"] * row, c["hkv"] * row
    if c["op"] == "rotate":
        return {"bytes": T * (2 * (q + kv) + 4), "flops": 3 * T * (c["hq"] + c["hkv"]) * c["rot"]}
    if c["op"] == "append":
        return {"bytes": T * (2 * (q + 2 * kv) + 4), "flops": 3 * T * (c["hq"] + c["hkv"]) * c["rot"]}
    if c["op"] == "gather":
        return {"bytes": c["batch"] * min([c["n"]] + lens) * (4 * kv + 4), "flops": 0}
    pairs = sum(n * l - n * (n - 1) // 2 for n, l in zip(news, lens))
    return {"bytes": T * (2 * q + 4 * c["hq"]) + sum(lens) * (2 * kv) + 4 * sum(-(-l // c["page"]) for l in lens),
            "flops": 4 * c["d"] * c["hq"] * pairs}


# ------------------------------------------------------------------------ exact

def _exact_turn(x, positions, c):
    """The rotation as a product of complex numbers."""
    r = c["rot"]
    z = x[..., :r].double()
    z = z.unflatten(-1, (2, r // 2)).transpose(-1, -2) if c["layout"] == "half" else z.unflatten(-1, (r // 2, 2))
    w = []
    for i in range(r // 2):
        f = BASE ** (-2.0 * i / r)
        if c["scaling"] == "linear":
            f /= FACTOR
        elif c["scaling"] == "band":
            keep = (ORIG * f / (2 * math.pi) - BAND[0]) / (BAND[1] - BAND[0])
            keep = min(1.0, max(0.0, keep))
            f = keep * f + (1 - keep) * f / FACTOR
        elif c["scaling"] == "ramp":
            def index(turns):
                return r * math.log(ORIG / (turns * 2 * math.pi)) / (2 * math.log(BASE))
            first = min(max(math.floor(index(RAMP[1])), 0), r // 2 - 1)
            last = min(max(math.ceil(index(RAMP[0])), 0), r // 2 - 1)
            slow = min(1.0, max(0.0, (i - first) / max(last - first, 1e-3)))
            f = slow * f / FACTOR + (1 - slow) * f
        w.append(f)
    angle = positions.double()[:, None] * torch.tensor(w, dtype=torch.float64, device=x.device)
    size = torch.full_like(angle, 0.1 * math.log(FACTOR) + 1 if c["scaling"] == "ramp" else 1.0)
    z = torch.view_as_real(torch.view_as_complex(z.contiguous()) * torch.polar(size, angle)[:, None])
    z = z.transpose(-1, -2).flatten(-2) if c["layout"] == "half" else z.flatten(-2)
    return torch.cat([z, x[..., r:].double()], -1)


def exact(case, seed):
    global own
    c, was, own = case, own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    news, lens = _lengths(c)
    first = [sum(news[:i]) for i in range(len(news))]
    if c["op"] == "rotate":
        return {"q": _exact_turn(s["q"], s["positions"], c), "k": _exact_turn(s["k"], s["positions"], c)}
    table = s["table"].tolist()
    slots = [(torch.tensor(t, device="cuda")[:, None] * c["page"] + torch.arange(c["page"], device="cuda")).flatten()
             for t in table]
    flat_K, flat_V = s["K"].flatten(0, 1), s["V"].flatten(0, 1)
    if c["op"] == "append":
        K, V = flat_K.double(), flat_V.double()
        turned = _exact_turn(s["k"], s["positions"], c)
        for i, (a, n, l) in enumerate(zip(first, news, lens)):
            K[slots[i][l - n:l]], V[slots[i][l - n:l]] = turned[a:a + n], s["v"][a:a + n].double()
        return {"q": _exact_turn(s["q"], s["positions"], c), "K": K.view(s["K"].shape), "V": V.view(s["V"].shape)}
    if c["op"] == "gather":
        at = [slots[i][s["idx"][i].long()] for i in range(c["batch"])]
        return {"K": torch.stack([flat_K[a].double() for a in at]), "V": torch.stack([flat_V[a].double() for a in at])}
    if sum(n * l for n, l in zip(news, lens)) * c["hq"] * c["d"] > 1 << 43:
        return None
    G = c["hq"] // c["hkv"]
    out = torch.empty(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.empty(s["q"].shape[:2], dtype=torch.float64, device="cuda")
    for i, (a, n, l) in enumerate(zip(first, news, lens)):
        K, V = flat_K[slots[i][:l]].double(), flat_V[slots[i][:l]].double()
        step = max(1, (1 << 28) // (l * G))
        for lo in range(0, n, step):
            hi = min(n, lo + step)
            hidden = torch.arange(l, device="cuda")[None] > torch.arange(l - n + lo, l - n + hi, device="cuda")[:, None]
            for h in range(c["hkv"]):
                q = s["q"][a + lo:a + hi, h * G:(h + 1) * G].double().transpose(0, 1)
                x = torch.matmul(q, K[:, h].T) / c["d"] ** 0.5
                x = torch.where(hidden, torch.full((), -math.inf, dtype=torch.float64, device="cuda"), x)
                lse[a + lo:a + hi, h * G:(h + 1) * G] = torch.logsumexp(x, -1).T
                out[a + lo:a + hi, h * G:(h + 1) * G] = torch.matmul(torch.softmax(x, -1), V[:, h]).transpose(0, 1)
    return {"out": out, "lse": lse}
