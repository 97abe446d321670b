"""Cases of the rotary-position, paged-cache append and paged-attention operators.

A case is a plain dict; ``prepare`` makes its inputs on the GPU from a seed,
``run`` makes one pass (the plain torch form, or the framework's calls when
``own`` is set) and ``exact`` gives the definition in float64.

Three operators, named by a case's ``op``:
  rope    rotation of q and k by their positions (``dir`` "fwd" or "bwd")
  append  new keys (rotated) and values into a paged cache, queries rotated on the way
  attend  attention of a ragged batch of new tokens over a paged cache

Tensors: q [B, H, N, D] (rope) or [H, T, D] (packed rows of a ragged batch), the
caches [pages, Hkv, page, D]; ``tokens`` says that the storage behind them is
token-major ([B, N, H, D], [T, H, D], [pages, page, Hkv, D]), the tensor being a
transposed view, as a projection or another program's cache leaves it.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16}


# ---------------------------------------------------------------- the cases
def _rope(name=None, **kw):
    c = dict(op="rope", dir="fwd", B=1, H=32, Hkv=8, N=1, D=128, rot=128, inter=False, dtype="bf16",
             base=500000.0, factor=1.0, far=0, tokens=False)
    c.update(kw)
    return c if name is None else dict(c, name=name)


def _append(name=None, **kw):
    c = dict(op="append", B=1, H=32, Hkv=8, D=128, page=64, new_hi=1, new_lo=1, len_hi=1024, len_lo=1024,
             rot=128, inter=False, dtype="bf16", base=500000.0, factor=1.0, tokens=False)
    c.update(kw)
    return c if name is None else dict(c, name=name)


def _attend(name=None, **kw):
    c = dict(op="attend", B=1, H=32, Hkv=8, D=128, page=64, new_hi=1, new_lo=1, len_hi=1024, len_lo=1024,
             singles=0, dtype="bf16", tokens=False)
    c.update(kw)
    return c if name is None else dict(c, name=name)


def listed():
    return [
        # a training step's q and k of the Llama layer the benchmark runs (H=32, N=8192), grouped kv heads
        _rope("rope llama fwd", N=8192),
        # gradients of a two-sequence batch straight from a token-major projection, interleaved pairs, half the head
        _rope("rope bwd part f16", dir="bwd", B=2, N=4096, rot=64, inter=True, dtype="f16", base=10000.0, tokens=True),
        # a short odd sequence of small heads far into a scaled context: the call's latency
        _rope("rope short far", B=3, H=8, Hkv=8, N=37, D=64, rot=32, base=10000.0, factor=8.0, far=1 << 20),
        # one decoding step of a full batch: 64 tokens into their sequences' pages
        _append("append decode 64", B=64, page=16, len_hi=2048, len_lo=256),
        # prompts of uneven lengths entering the cache of another program (token-major pages)
        _append("append prompts", B=6, new_hi=4000, new_lo=700, len_hi=4000, len_lo=4000, page=64, tokens=True),
        # a single user's token: the smallest call
        _append("append one f16", H=16, Hkv=16, D=64, rot=64, page=32, len_hi=777, len_lo=777, dtype="f16", base=10000.0),
        # a single user's token over a short context: latency
        _attend("attend one", len_hi=1000, len_lo=1000, page=16),
        # one decoding step of a full batch with uneven contexts
        _attend("attend decode 64", B=64, len_hi=8192, len_lo=512, page=16),
        # one token over the benchmark's 65536-key decoding context, as many kv heads as heads
        _attend("attend long f16", H=8, Hkv=8, len_hi=65536, len_lo=65536, page=128, dtype="f16"),
        # a few drafted tokens of several sequences, small heads, token-major pages
        _attend("attend draft", B=16, H=16, Hkv=2, D=64, new_hi=7, new_lo=3, len_hi=6000, len_lo=900, page=32, tokens=True),
        # chunks of prompts and single tokens in one batch
        _attend("attend mixed", B=20, new_hi=1000, new_lo=300, singles=5, len_hi=7000, len_lo=1000, page=32),
        # a long prompt's chunk over what is cached already: the largest call
        _attend("attend chunk", B=2, new_hi=2048, new_lo=2048, len_hi=16384, len_lo=12001, page=64),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    while True:
        op = rng.choice(["rope", "append", "attend", "attend"])
        D = rng.choice([64, 128])
        Hkv = rng.choice([1, 2, 4, 8, 8])
        H = Hkv * rng.choice([1, 2, 3, 4, 4, 5, 8])
        common = dict(D=D, H=H, Hkv=Hkv, dtype=rng.choice(["bf16", "bf16", "f16"]), tokens=rng.random() < 0.4)
        rope = dict(rot=rng.choice([D, D, D // 2, D // 4]), inter=rng.random() < 0.4, base=rng.choice([10000.0, 500000.0]),
                    factor=rng.choice([1.0, 1.0, 8.0]))
        if op == "rope":
            c = _rope(dir=rng.choice(["fwd", "bwd"]), B=rng.randint(1, 4), N=_log(rng, 1, 8192),
                      far=rng.choice([0, 0, 1 << 17, 1 << 20]), **common, **rope)
        elif op == "append":
            new = _log(rng, 1, 4096)
            length = new + _log(rng, 1, 4096)
            c = _append(B=_log(rng, 1, 64), new_hi=new, new_lo=max(1, new // 3), len_hi=length, len_lo=new + (length - new) // 4,
                        page=rng.choice([16, 32, 48, 64, 128]), **common, **rope)
        else:
            new = _log(rng, 1, 2048) if rng.random() < 0.6 else 1
            length = new + _log(rng, 1, 30000)
            c = _attend(B=_log(rng, 1, 64), new_hi=new, new_lo=rng.choice([1, new]), len_hi=length,
                        len_lo=new + (length - new) // rng.choice([1, 2, 8]), page=rng.choice([16, 32, 48, 64, 128]), singles=rng.choice([0, 0, 4]), **common)
        w, big = work(c), max((work(x) for x in listed() if x["op"] == op), key=lambda w: w["bytes"] + w["flops"] / 50)
        if w["bytes"] + w["flops"] / 50 <= big["bytes"] + big["flops"] / 50 and _padded(c) <= 3e9:
            return c


def _padded(c):
    """Elements that the plain form of the attention holds: caches (gathered, in 32 bits and transposed) and scores, padded to the longest."""
    return 0 if c["op"] != "attend" else c["B"] * c["len_hi"] * (5 * c["Hkv"] * c["D"] + c["H"] * c["new_hi"])


def _lengths(c):
    """(total lengths, new tokens) of the sequences: spread between the case's bounds, the first the longest."""
    b = np.arange(c["B"])
    spread = lambda hi, lo, g: hi - np.floor((hi - lo + 0.999) * (b * g % 1.0)).astype(np.int64)  # noqa: E731
    new = spread(c["new_hi"], c["new_lo"], 0.7548776662)
    if c.get("singles"):        # all but one in so many sequences have a single new token
        new = np.where(b % c["singles"] == 0, new, 1)
    return spread(c["len_hi"], c["len_lo"], 0.6180339887), new


def work(c):
    H, Hkv, D = c["H"], c["Hkv"], c["D"]
    if c["op"] == "rope":
        rows = c["B"] * c["N"] * (H + Hkv)
        return {"bytes": 4.0 * rows * D, "flops": 3.0 * rows * c["rot"]}
    lens, new = _lengths(c)
    T = int(new.sum())
    if c["op"] == "append":
        return {"bytes": 4.0 * T * (H + 2 * Hkv) * D, "flops": 3.0 * T * (H + Hkv) * c["rot"]}
    seen = float((new * (lens - new) + new * (new + 1) // 2).sum())
    return {"bytes": 4.0 * float(lens.sum()) * Hkv * D + 4.0 * T * H * D + 4.0 * T * H, "flops": 4.0 * seen * H * D}


# ---------------------------------------------------------------- the inputs
def _inv_freq(c):
    """base^(-2i/rot); with a factor, low frequencies divided by it, high ones kept and those between blended."""
    i = np.arange(0, c["rot"], 2, dtype=np.float64)
    f = c["base"] ** (-i / c["rot"])
    if c["factor"] != 1.0:
        turns = 8192 * f / (2 * math.pi)
        keep = np.clip((turns - 1.0) / (4.0 - 1.0), 0.0, 1.0)
        f = f * keep + f / c["factor"] * (1.0 - keep)
    return f


def prepare(case, seed):
    c = case
    g = torch.Generator("cuda").manual_seed(seed)
    rng = np.random.default_rng(seed)
    dt, tok = DTYPES[c["dtype"]], c["tokens"]
    H, Hkv, D = c["H"], c["Hkv"], c["D"]

    def rows(h, *lead):     # [B, h, N, D] or [h, T, D]
        shape = (*lead[:-1], lead[-1], h, D) if tok else (*lead[:-1], h, lead[-1], D)
        x = torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(dt)
        return x.transpose(-2, -3) if tok else x

    s = dict(case=c)
    if c["op"] != "attend":
        s["inv_freq"] = torch.from_numpy(_inv_freq(c)).cuda()
    if c["op"] == "rope":
        s["q"], s["k"] = rows(H, c["B"], c["N"]), rows(Hkv, c["B"], c["N"])
        start = rng.integers(0, max(1, c["far"]), size=(c["B"], 1))
        s["positions"] = torch.from_numpy((start + np.arange(c["N"])).astype(np.int32)).cuda()
        return s
    lens, new = _lengths(c)
    T, B, S = int(new.sum()), c["B"], c["page"]
    need = (lens + S - 1) // S
    pages = int(need.sum()) + 3
    table = np.zeros((B, int(need.max())), dtype=np.int32)
    order, at = rng.permutation(pages), 0
    for b in range(B):
        table[b, :need[b]] = order[at:at + need[b]]
        at += need[b]
    shape = (pages, S, Hkv, D) if tok else (pages, Hkv, S, D)
    for name in ("k_cache", "v_cache"):
        x = torch.empty(shape, device="cuda", dtype=dt).normal_(generator=g)
        s[name] = x.transpose(1, 2) if tok else x
    cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    s.update(page_table=torch.from_numpy(table).cuda(), seq_lens=torch.from_numpy(lens.astype(np.int32)).cuda(),
             cu=torch.from_numpy(cu).cuda(), max_new=int(new.max()), q=rows(H, T))
    if c["op"] == "append":
        s["k"], s["v"] = rows(Hkv, T), rows(Hkv, T)
    # the buffers and the host's own copy of the batch's bookkeeping that such a program keeps
    s["out"] = torch.empty_like(s["q"])
    if c["op"] == "attend":
        s["lse"] = torch.empty((H, T), dtype=torch.float32, device="cuda")
    seq = np.repeat(np.arange(B), new)
    s["seq"] = torch.from_numpy(seq).cuda()
    s["row"] = torch.from_numpy(np.arange(T) - cu[seq]).cuda()
    s["pos"] = torch.from_numpy(lens[seq] - new[seq] + np.arange(T) - cu[seq]).cuda()
    return s


# ---------------------------------------------------------------- one pass
def run(s):
    c = s["case"]
    if own:
        return _run_own(s)
    if c["op"] == "rope":
        sign = -1.0 if c["dir"] == "bwd" else 1.0
        cos, sin = _angles(s["positions"], s["inv_freq"], sign)
        return _rotated(s["q"], cos[:, None], sin[:, None], c), _rotated(s["k"], cos[:, None], sin[:, None], c)
    if c["op"] == "append":
        cos, sin = _angles(s["pos"], s["inv_freq"], 1.0)
        page, off = s["page_table"][s["seq"], s["pos"] // c["page"]], s["pos"] % c["page"]
        s["k_cache"][page, :, off] = _rotated(s["k"], cos, sin, c).transpose(0, 1)
        s["v_cache"][page, :, off] = s["v"].transpose(0, 1)
        return s["k_cache"], s["v_cache"], _rotated(s["q"], cos, sin, c)
    return _attention(s)


def _angles(pos, inv_freq, sign):
    theta = pos.double()[..., None] * inv_freq      # far positions need 64 bits
    return theta.cos().float(), (sign * theta.sin()).float()


def _rotated(x, cos, sin, c):
    r, y = c["rot"], x.float()
    a, b = (y[..., 0:r:2], y[..., 1:r:2]) if c["inter"] else (y[..., :r // 2], y[..., r // 2:r])
    u, v = a * cos - b * sin, b * cos + a * sin
    uv = torch.stack((u, v), -1).flatten(-2) if c["inter"] else torch.cat((u, v), -1)
    return torch.cat((uv, y[..., r:]), -1).to(x.dtype)


def _attention(s):
    c = s["case"]
    H, Hkv, D, B, S = c["H"], c["Hkv"], c["D"], c["B"], c["page"]
    G, M, L, T = H // Hkv, s["max_new"], c["len_hi"], s["q"].shape[1]
    j = torch.arange(L, device="cuda")
    page = s["page_table"][:, j // S].long()                                         # [B, L]
    k = s["k_cache"][page, :, (j % S)[None]].permute(0, 2, 1, 3).float()             # [B, Hkv, L, D]
    v = s["v_cache"][page, :, (j % S)[None]].permute(0, 2, 1, 3).float()
    q = torch.zeros((B, M, H, D), device="cuda")
    q[s["seq"], s["row"]] = s["q"].transpose(0, 1).float()
    q = q.view(B, M, Hkv, G, D).permute(0, 2, 3, 1, 4).reshape(B, Hkv, G * M, D)
    x = torch.matmul(q, k.transpose(-1, -2)).mul_(1.0 / math.sqrt(D)).view(B, Hkv, G, M, L)
    lens, new = s["seq_lens"].long(), (s["cu"][1:] - s["cu"][:-1]).long()
    last = torch.arange(M, device="cuda")[None] + (lens - new)[:, None]               # [B, M]
    seen = (j[None, None] <= last[..., None]) & (j[None, None] < lens[:, None, None])
    x.masked_fill_(~seen[:, None, None], -math.inf)
    m = x.amax(-1, keepdim=True)
    x.sub_(m).exp_()
    l = x.sum(-1, keepdim=True)
    o = torch.matmul(x.view(B, Hkv, G * M, L), v).view(B, Hkv, G, M, D) / l
    lse = (m + l.log())[..., 0]
    o = o.permute(0, 3, 1, 2, 4).reshape(B, M, H, D)[s["seq"], s["row"]]              # [T, H, D]
    lse = lse.permute(0, 3, 1, 2).reshape(B, M, H)[s["seq"], s["row"]]
    return o.transpose(0, 1).to(s["q"].dtype), lse.transpose(0, 1)


def _run_own(s):
    import exact_attention_112_b200 as fa
    c = s["case"]
    # the handles a program makes once for its model and its cache
    if "rope" not in s and c["op"] != "attend":
        s["rope"] = fa.Rope(s["inv_freq"], interleaved=c["inter"])
    if "kv" not in s and c["op"] != "rope":
        s["kv"] = fa.PagedKV(s["k_cache"], s["v_cache"], s["page_table"], s["seq_lens"])
    if c["op"] == "rope":
        f = fa.rope_backward if c["dir"] == "bwd" else fa.rope_forward
        return f(s["q"], s["k"], s["rope"], positions=s["positions"])
    if c["op"] == "append":
        fa.fa_paged_append(s["kv"], s["k"], s["v"], s["cu"], rope=s["rope"], q=s["q"], q_out=s["out"])
        return s["k_cache"], s["v_cache"], s["out"]
    if "workspace" not in s:
        s["workspace"] = torch.empty(fa.fa_paged_fwd_workspace_bytes(s["kv"], c["H"], s["max_new"]), dtype=torch.uint8, device="cuda")
    fa.fa_paged_fwd(s["kv"], s["q"], s["out"], s["lse"], s["cu"], s["max_new"], s["workspace"], causal=True)
    return s["out"], s["lse"]


# ---------------------------------------------------------------- the definition in 64 bits
def exact(case, seed):
    c, s = case, prepare(case, seed)

    def turn(x, pos, sign):     # the pair (a, b) as the complex number a + ib, times e^(i theta)
        x, r = x.double(), c["rot"]
        pairs = x[..., :r].unflatten(-1, (r // 2, 2)) if c["inter"] else x[..., :r].unflatten(-1, (2, r // 2)).transpose(-1, -2)
        w = torch.polar(torch.ones((), dtype=torch.float64, device=x.device), sign * pos[..., None].double() * s["inv_freq"])
        y = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * w)
        return torch.cat((y.flatten(-2) if c["inter"] else y.transpose(-1, -2).flatten(-2), x[..., r:]), -1)

    if c["op"] == "rope":
        sign = -1.0 if c["dir"] == "bwd" else 1.0
        return turn(s["q"], s["positions"][:, None], sign), turn(s["k"], s["positions"][:, None], sign)
    lens, new = _lengths(c)
    S, cu, table = c["page"], s["cu"].tolist(), s["page_table"].long()
    if c["op"] == "append":
        kc, vc, qo = s["k_cache"].double(), s["v_cache"].double(), s["q"].double()
        for b in range(c["B"]):
            p = torch.arange(int(lens[b] - new[b]), int(lens[b]), device="cuda")
            rows = slice(cu[b], cu[b + 1])
            kc[table[b, p // S], :, p % S] = turn(s["k"][:, rows], p[None], 1.0).transpose(0, 1)
            vc[table[b, p // S], :, p % S] = s["v"][:, rows].double().transpose(0, 1)
            qo[:, rows] = turn(s["q"][:, rows], p[None], 1.0)
        return kc, vc, qo
    H, Hkv, D = c["H"], c["Hkv"], c["D"]
    o = torch.empty((H, cu[-1], D), dtype=torch.float64, device="cuda")
    lse = torch.empty((H, cu[-1]), dtype=torch.float64, device="cuda")
    for b in range(c["B"]):
        n, t = int(lens[b]), int(new[b])
        past = torch.ones((t, n), dtype=torch.bool, device="cuda").tril(n - t)
        for h in range(Hkv):
            own_pages = table[b, :(n + S - 1) // S]
            k = s["k_cache"][own_pages, h].reshape(-1, D)[:n].double()
            v = s["v_cache"][own_pages, h].reshape(-1, D)[:n].double()
            for g in range(h * H // Hkv, (h + 1) * H // Hkv):
                z = (s["q"][g, cu[b]:cu[b + 1]].double() @ k.T / math.sqrt(D)).where(past, -math.inf)
                lse[g, cu[b]:cu[b + 1]] = z.logsumexp(-1)
                o[g, cu[b]:cu[b + 1]] = z.softmax(-1) @ v
    return o, lse
