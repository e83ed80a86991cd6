"""Cases of the softmax attention of the network in front of a conditional (LowRank) circuit: the heads' norm with the
rotation by position, causal attention over whole sequences and its gradients, and attention of new tokens over a cache
in pages.

The network that gives a circuit its per-sample factors mixes its features along a sequence.  Linear attention with a
decay forgets at a fixed rate; causal softmax attention looks anything up.  A run of it is: heads of queries and keys
normalised and rotated, attended, and for training their gradients; for answering, a chunk of the prompt or one token at
a time against what is kept of the tokens before.
"""
import math

import torch

own = False

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
BYTES = {"f32": 4, "bf16": 2, "f16": 2}
EPS = 1e-6
BASE = 10000.0
FAR = 131072          # positions of a context stretched by FACTOR from FAR / FACTOR
FACTOR = 8.0
LOW, HIGH = 1.0, 32.0


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # the heads of one new token of one stream: launch latency
        {"name": "rotate_one", "op": "rotate", "dir": "fwd", "type": "bf16", "tokens": 1, "heads": 16, "kv_heads": 4, "dim": 64,
         "part": 64, "layout": "half", "norm": True},
        # part of each head, neighbours as pairs, no norm, an odd number of tokens
        {"name": "rotate_part", "op": "rotate", "dir": "fwd", "type": "f16", "tokens": 5001, "heads": 6, "kv_heads": 3, "dim": 80,
         "part": 40, "layout": "pairs", "norm": False},
        # a long prompt, 32 heads of queries and 8 of keys
        {"name": "rotate_long", "op": "rotate", "dir": "fwd", "type": "bf16", "tokens": 16384, "heads": 32, "kv_heads": 8, "dim": 128,
         "part": 128, "layout": "half", "norm": True},
        # gradients of a training batch of 8 x 2048 positions
        {"name": "rotate_bwd", "op": "rotate", "dir": "bwd", "type": "bf16", "tokens": 16384, "heads": 16, "kv_heads": 16, "dim": 128,
         "part": 128, "layout": "half", "norm": True},
        # one long prompt, key and value heads shared by four
        {"name": "attend_long", "op": "attend", "dir": "fwd", "type": "bf16", "seqs": 1, "tokens": 16384, "lens": "same", "heads": 16,
         "kv_heads": 4, "dk": 128, "dv": 128},
        # prompts of mixed length (one token and empty ones among them)
        {"name": "attend_ragged", "op": "attend", "dir": "fwd", "type": "f16", "seqs": 24, "tokens": 1500, "lens": "ragged", "heads": 16,
         "kv_heads": 4, "dk": 64, "dv": 64},
        # a training batch
        {"name": "attend_bwd", "op": "attend", "dir": "bwd", "type": "bf16", "seqs": 8, "tokens": 2048, "lens": "same", "heads": 16,
         "kv_heads": 16, "dk": 128, "dv": 128},
        # float32 training, ragged, shared heads, odd head sizes
        {"name": "attend_bwd_ragged", "op": "attend", "dir": "bwd", "type": "f32", "seqs": 7, "tokens": 900, "lens": "ragged", "heads": 6,
         "kv_heads": 3, "dk": 48, "dv": 80},
        # one stream, one token: latency
        {"name": "cache_one", "op": "cache", "type": "bf16", "seqs": 1, "tokens": 1, "past": 1000, "lens": "same", "page": 16, "heads": 16,
         "kv_heads": 4, "dk": 64, "dv": 64},
        # many streams of mixed length, one token each: the cache is read
        {"name": "cache_many", "op": "cache", "type": "bf16", "seqs": 64, "tokens": 1, "past": 8192, "lens": "ragged", "page": 16, "heads": 32,
         "kv_heads": 8, "dk": 128, "dv": 128},
        # chunks of four prompts behind what is cached of them
        {"name": "cache_chunk", "op": "cache", "type": "bf16", "seqs": 4, "tokens": 512, "past": 8192, "lens": "same", "page": 64, "heads": 32,
         "kv_heads": 8, "dk": 128, "dv": 128},
        # short chunks of mixed length in float32, odd pages and head sizes
        {"name": "cache_ragged", "op": "cache", "type": "f32", "seqs": 13, "tokens": 17, "past": 700, "lens": "ragged", "page": 24, "heads": 6,
         "kv_heads": 3, "dk": 48, "dv": 80},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rotate", "attend", "attend", "cache", "cache"])
    kv = rng.choice([1, 2, 3, 4, 8])
    heads = kv * rng.choice([1, 1, 2, 4])
    c = {"op": op, "type": rng.choice(sorted(TYPES)), "heads": heads, "kv_heads": kv}
    if op == "rotate":
        dim = rng.choice([16, 24, 32, 48, 64, 80, 96, 128])
        return {**c, "dir": rng.choice(["fwd", "bwd"]), "tokens": _log(rng, 1, 16384), "dim": dim,
                "part": rng.choice([dim, dim, dim // 2, dim // 8 * 2]), "layout": rng.choice(["half", "pairs"]), "norm": rng.random() < 0.7}
    c["dk"], c["dv"] = (rng.choice([16, 24, 32, 48, 64, 80, 96, 128]) for _ in range(2))
    if rng.random() < 0.5:
        c["dv"] = c["dk"]
    c["lens"] = rng.choice(["same", "ragged"])
    if op == "attend":
        c["dir"] = rng.choice(["fwd", "bwd"])
        c["seqs"] = _log(rng, 1, 24)
        most = math.sqrt((1 << (30 if c["dir"] == "fwd" else 28)) / (c["seqs"] * heads))
        # (a single token's weight is 1 whatever q and k are: their gradients are 0, and nothing but rounding is left)
        least = 1 if c["dir"] == "fwd" else 2
        c["tokens"] = _log(rng, least, max(least, min(8192, most)))
        return c
    c["page"] = rng.choice([1, 8, 16, 24, 32, 64, 100, 256])
    c["tokens"] = rng.choice([1, 1, _log(rng, 2, 512)])
    c["seqs"] = _log(rng, 1, 64 if c["tokens"] == 1 else 8)
    c["past"] = _log(rng, 1, max(1, min(16384, (1 << 28) // (c["seqs"] * heads * c["tokens"]))))
    return c


def lengths(case):
    """(new tokens, tokens in the cache) of each sequence: all the same, or from none to the most in a fixed order."""
    n, most, past = case["seqs"], case["tokens"], case.get("past", 0)
    if case["lens"] == "same":
        return [most] * n, [past] * n
    new = [most] + [(0, 1, most // 2 + i, most // 3, most // 7 + 2 * i, most // 5, most - i)[(i - 1) % 7] for i in range(1, n)]
    old = [past] + [(past // 2 + 3 * i, 0, past // 3, 1, past - i, past // 5, past // 4 * 3)[(i - 1) % 7] for i in range(1, n)]
    if most == 1:
        new = [1] * n      # one token of every stream
    return [max(0, min(most, x)) for x in new], [max(0, min(past, x)) for x in old]


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    t = TYPES[case["type"]]

    def normal(*shape, dtype=t, scale=1.0, shift=0.0):
        return (torch.randn(shape, generator=g, device="cuda") * scale + shift).to(dtype)

    s = {"case": dict(case)}
    H, K = case["heads"], case["kv_heads"]
    if case["op"] == "rotate":
        T, d, half = case["tokens"], case["dim"], case["part"] // 2
        s["q"], s["k"] = normal(T, H, d, scale=1.5), normal(T, K, d, scale=1.5)
        # tokens of one prompt, from anywhere in a long context
        start = torch.randint(0, FAR - T, (1,), generator=g, device="cuda")
        s["positions"] = (start + torch.arange(T, device="cuda")).to(torch.int32)
        # slow pairs are stretched, fast ones kept, by their turns over the context before it was stretched
        f = BASE ** (-torch.arange(half, device="cuda", dtype=torch.float64) / half)
        ramp = ((FAR / FACTOR * f / (2 * math.pi) - LOW) / (HIGH - LOW)).clamp(0, 1)
        s["freq"] = f * (ramp + (1 - ramp) / FACTOR)
        s["magnitude"] = 0.1 * math.log(FACTOR) + 1.0
        if case["norm"]:
            s["q_weight"], s["k_weight"] = (normal(d, dtype=torch.float32, scale=0.2, shift=1.0) for _ in range(2))
        if case["dir"] == "bwd":
            s["dq"], s["dk"] = normal(T, H, d), normal(T, K, d)
        if own:
            import log_space_sum_amd as L
            s["q_out"], s["k_out"] = torch.empty_like(s["q"]), torch.empty_like(s["k"])
            if case["dir"] == "bwd" and case["norm"]:
                s["dq_weight"], s["dk_weight"] = torch.empty_like(s["q_weight"]), torch.empty_like(s["k_weight"])
                s["ws"] = L.rotary_workspace(s["q"], s["k"])
        return s
    dk, dv = case["dk"], case["dv"]
    new, old = lengths(case)
    n, T = len(new), sum(new)
    s["new"], s["longest"] = new, max(new)
    s["q"], s["k"], s["v"] = normal(T, H, dk), normal(T, K, dk), normal(T, K, dv)
    s["cu"] = torch.tensor([sum(new[:i]) for i in range(n + 1)], dtype=torch.int32, device="cuda")
    # where each token lies in a batch padded to the longest sequence: the plan that the plain form gathers by
    at = torch.repeat_interleave(torch.arange(n, device="cuda"), s["cu"].diff().long())
    s["row"], s["col"] = at, torch.arange(T, device="cuda") - s["cu"].long()[at]
    if case["op"] == "attend":
        if case["dir"] == "bwd":
            s["do"] = normal(T, H, dv)
            s |= _attend_forward(s)      # what the forward pass kept
        if own:
            import log_space_sum_amd as L
            s["ws"] = L.attention_workspace(s["q"], s["k"], s["v"], s["cu"], s["longest"], backward=case["dir"] == "bwd")
            if case["dir"] == "bwd":
                s["dq"], s["dk"], s["dv"] = (torch.empty_like(s[x]) for x in ("q", "k", "v"))
            else:
                s["o"], s["lse"] = torch.empty((T, H, dv), dtype=t, device="cuda"), torch.empty((T, H), device="cuda")
        return s
    page = case["page"]
    s["most"] = max(a + b for a, b in zip(new, old))
    each = -(-s["most"] // page)
    pages = n * each + 3
    s["k_cache"], s["v_cache"] = normal(pages, page, K, dk), normal(pages, page, K, dv)
    s["table"] = torch.randperm(pages, generator=g, device="cuda")[:n * each].view(n, each).to(torch.int32)
    s["past"] = torch.tensor(old, dtype=torch.int32, device="cuda")
    if own:
        import log_space_sum_amd as L
        s["o"] = torch.empty((T, H, dv), dtype=t, device="cuda")
        s["ws"] = L.attention_cached_workspace(s["q"], s["k_cache"], s["v_cache"], s["table"], s["cu"], s["longest"], s["most"])
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(s):
    case = s["case"]
    if own:
        return _run_own(s, case)
    if case["op"] == "rotate":
        return _rotate_forward(s) if case["dir"] == "fwd" else _rotate_backward(s)
    if case["op"] == "attend":
        return _attend_forward(s) if case["dir"] == "fwd" else _attend_backward(s)
    return _cached(s)


def _run_own(s, case):
    import log_space_sum_amd as L
    if case["op"] == "rotate":
        how = {"interleaved": case["layout"] == "pairs", "magnitude": s["magnitude"], "norm": case["norm"], "eps": EPS,
               "q_weight": s.get("q_weight"), "k_weight": s.get("k_weight")}
        if case["dir"] == "fwd":
            L.pc_rotary_forward(s["q"], s["k"], s["q_out"], s["k_out"], s["positions"], s["freq"], **how)
            return {"q": s["q_out"], "k": s["k_out"]}
        L.pc_rotary_backward(s["dq"], s["dk"], s["q_out"], s["k_out"], s["positions"], s["freq"], q=s["q"], k=s["k"],
                             dq_weight=s.get("dq_weight"), dk_weight=s.get("dk_weight"), ws=s.get("ws"), **how)
        out = {"dq": s["q_out"], "dk": s["k_out"]}
        return {**out, "dq_weight": s["dq_weight"], "dk_weight": s["dk_weight"]} if case["norm"] else out
    if case["op"] == "cache":
        L.pc_attention_cached(s["q"], s["k"], s["v"], s["k_cache"], s["v_cache"], s["table"], s["past"], s["o"], cu_seqlens=s["cu"],
                              max_seqlen=s["longest"], max_length=s["most"], ws=s["ws"])
        return {"o": s["o"], "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
    if case["dir"] == "fwd":
        L.pc_attention_forward(s["q"], s["k"], s["v"], s["o"], s["lse"], cu_seqlens=s["cu"], max_seqlen=s["longest"], ws=s["ws"])
        return {"o": s["o"], "lse": s["lse"]}
    L.pc_attention_backward(s["do"], s["q"], s["k"], s["v"], s["o"], s["lse"], s["dq"], s["dk"], s["dv"], cu_seqlens=s["cu"],
                            max_seqlen=s["longest"], ws=s["ws"])
    return {"dq": s["dq"], "dk": s["dk"], "dv": s["dv"]}


# ---- plain forms: elementary operations in float32 (angles in 64 bits) ----

def _turn(s, x, way):
    """The first `part` elements of each head turned by way * position * freq, times the magnitude."""
    part, pairs = s["case"]["part"], s["case"]["layout"] == "pairs"
    angle = s["positions"].double()[:, None] * s["freq"]
    cos, sin = ((f(angle) * s["magnitude"]).float()[:, None] for f in (torch.cos, torch.sin))
    a, b = (x[..., 0:part:2], x[..., 1:part:2]) if pairs else (x[..., :part // 2], x[..., part // 2:part])
    y, z = a * cos - way * b * sin, b * cos + way * a * sin
    y = torch.stack((y, z), -1).flatten(-2) if pairs else torch.cat((y, z), -1)
    return torch.cat((y, x[..., part:]), -1)


def _rotate_forward(s):
    out = {}
    for name in ("q", "k"):
        x = s[name].float()
        if s["case"]["norm"]:
            x = x * (x.square().mean(-1, keepdim=True) + EPS).rsqrt() * s[name + "_weight"]
        out[name] = _turn(s, x, 1.0).to(s[name].dtype)
    return out


def _rotate_backward(s):
    out = {}
    for name in ("q", "k"):
        g = _turn(s, s["d" + name].float(), -1.0)
        if s["case"]["norm"]:
            x = s[name].float()
            r = (x.square().mean(-1, keepdim=True) + EPS).rsqrt()
            n = x * r
            out["d%s_weight" % name] = (g * n).sum((0, 1))
            g = g * s[name + "_weight"]
            g = r * (g - n * (g * n).mean(-1, keepdim=True))
        out["d" + name] = g.to(s[name].dtype)
    return out


def _padded(s, x, kv):
    """[T, h, d] tokens as a padded float32 batch [n, kv, h / kv, longest, d]."""
    out = torch.zeros((len(s["new"]), max(1, s["longest"]), x.shape[1], x.shape[2]), device=x.device)
    out[s["row"], s["col"]] = x.float()
    return out.transpose(1, 2).unflatten(1, (kv, x.shape[1] // kv))


def _flat(s, x):
    return x.flatten(1, 2).transpose(1, 2)[s["row"], s["col"]]


def _weights(q, k, scale, first):
    """Scores of padded queries [n, K, g, T, d] and keys [n, K, 1, S, d], -inf where key j lies behind position first + i."""
    n, K, g, T, d = q.shape
    x = ((q * scale).reshape(n, K, g * T, d) @ k[:, :, 0].mT).reshape(n, K, g, T, k.shape[3])
    i, j = torch.arange(T, device=q.device), torch.arange(k.shape[3], device=q.device)
    return x.masked_fill_((j > first[:, None, None] + i[:, None])[:, None, None], -math.inf)


def _softmax_of(x, v):
    """(outputs, log of the sums) for scores x [n, K, g, T, S] and values v [n, K, 1, S, d]."""
    n, K, g, T, S = x.shape
    top = x.amax(-1, keepdim=True)
    p = x.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    o = (p.reshape(n, K, g * T, S) @ v[:, :, 0]).reshape(n, K, g, T, v.shape[4]) / total
    return o, (top + total.log())[..., 0]


def _attend_forward(s):
    K, scale = s["case"]["kv_heads"], s["q"].shape[2] ** -0.5
    q, k, v = (_padded(s, s[x], K) for x in ("q", "k", "v"))
    o, lse = _softmax_of(_weights(q, k, scale, s["cu"][:-1] * 0), v)
    return {"o": _flat(s, o).to(s["q"].dtype), "lse": _flat(s, lse[..., None])[..., 0]}


def _attend_backward(s):
    K, scale, t = s["case"]["kv_heads"], s["q"].shape[2] ** -0.5, s["q"].dtype
    q, k, v, o, do, lse = (_padded(s, x, K) for x in (s["q"], s["k"], s["v"], s["o"], s["do"], s["lse"][..., None]))
    n, _, g, T, _ = q.shape
    p = _weights(q, k, scale, s["cu"][:-1] * 0).sub_(lse).exp_()
    dp = (do.reshape(n, K, g * T, -1) @ v[:, :, 0].mT).reshape(n, K, g, T, T)
    ds = dp.sub_((do * o).sum(-1, keepdim=True)).mul_(p).reshape(n, K, g * T, T)
    p = p.reshape(n, K, g * T, T)
    dq = (ds @ k[:, :, 0]).reshape(q.shape) * scale
    dk = (ds.mT @ q.reshape(n, K, g * T, -1))[:, :, None] * scale
    dv = (p.mT @ do.reshape(n, K, g * T, -1))[:, :, None]
    return {"dq": _flat(s, dq).to(t), "dk": _flat(s, dk).to(t), "dv": _flat(s, dv).to(t)}


def _cached(s):
    K, page, scale = s["case"]["kv_heads"], s["case"]["page"], s["q"].shape[2] ** -0.5
    where = s["past"].long()[s["row"]] + s["col"]      # the new tokens' positions
    at = s["table"].long()[s["row"], where // page]
    s["k_cache"][at, where % page] = s["k"]
    s["v_cache"][at, where % page] = s["v"]
    q = _padded(s, s["q"], K)
    k, v = (c[s["table"].long()].flatten(1, 2).transpose(1, 2)[:, :, None].float() for c in (s["k_cache"], s["v_cache"]))
    # keys behind a sequence's last token are another one's, or nobody's: not to be met even with weight 0
    v = v.masked_fill((torch.arange(v.shape[3], device=v.device) >= (s["past"] + s["cu"].diff())[:, None])[:, None, None, :, None], 0.0)
    o, _ = _softmax_of(_weights(q, k, scale, s["past"]), v)
    return {"o": _flat(s, o).to(s["q"].dtype), "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


# ---------------------------------------------------------------------------
# the least work of one pass, and the definitions in 64 bits
# ---------------------------------------------------------------------------

def work(case):
    e, H, K = BYTES[case["type"]], case["heads"], case["kv_heads"]
    if case["op"] == "rotate":
        n, d = case["tokens"] * (H + K) * case["dim"], case["dim"]
        small = 4 * case["tokens"] + 4 * case["part"] + (8 * d if case["norm"] else 0)
        if case["dir"] == "fwd":
            return {"bytes": 2 * n * e + small, "flops": (9 if case["norm"] else 6) * n}
        return {"bytes": (3 if case["norm"] else 2) * n * e + small + (8 * d if case["norm"] else 0), "flops": (16 if case["norm"] else 6) * n}
    new, old = lengths(case)
    T, dk, dv = sum(new), case["dk"], case["dv"]
    pairs = sum(a * b + a * (a + 1) // 2 for a, b in zip(new, old))
    tokens = T * (H * dk + K * dk + K * dv + H * dv) * e
    if case["op"] == "cache":
        kept = (sum(b for a, b in zip(new, old) if a) + T) * K * (dk + dv) * e      # what is read, and the new tokens written
        return {"bytes": tokens + kept, "flops": 2 * pairs * H * (dk + dv)}
    if case["dir"] == "fwd":
        return {"bytes": tokens + 4 * T * H, "flops": 2 * pairs * H * (dk + dv)}
    return {"bytes": 2 * tokens + 4 * T * H + T * H * dv * e, "flops": 2 * pairs * H * (3 * dk + 2 * dv)}


def _exact_rotate(s, case):
    angle = s["positions"].double()[:, None] * s["freq"].double()
    z = torch.polar(torch.full_like(angle, s["magnitude"]), angle)[:, None]
    out, part, half = {}, case["part"], case["part"] // 2

    def rotated(x, z):
        y = x.clone()
        first, second = (slice(0, part, 2), slice(1, part, 2)) if case["layout"] == "pairs" else (slice(0, half), slice(half, part))
        turned = torch.complex(x[..., first], x[..., second]) * z
        y[..., first], y[..., second] = turned.real, turned.imag
        return y

    for name in ("q", "k"):
        x = s[name].double()
        r = 1.0 / torch.sqrt((x * x).sum(-1, keepdim=True) / case["dim"] + EPS)
        w = s[name + "_weight"].double() if case["norm"] else None
        if case["dir"] == "fwd":
            out[name] = rotated(x if w is None else w * (x * r), z)
            continue
        g = rotated(s["d" + name].double(), z.conj())
        if w is not None:
            out["d%s_weight" % name] = (g * x * r).sum(0).sum(0)
            h = g * w
            g = r * h - x * r ** 3 * (h * x).sum(-1, keepdim=True) / case["dim"]
        out["d" + name] = g
    return out


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rotate":
        return _exact_rotate(s, case)
    H, K, scale = case["heads"], case["kv_heads"], case["dk"] ** -0.5
    new, old = lengths(case)
    grp = H // K
    names = ["o"] + (["lse"] if case.get("dir") == "fwd" else [])
    out = {x: [] for x in (names if case.get("dir") != "bwd" else ("dq", "dk", "dv"))}
    if case["op"] == "cache":
        kc, vc = s["k_cache"].clone(), s["v_cache"].clone()
    at = 0
    for i, (n, past) in enumerate(zip(new, old)):
        q, k, v = (s[x][at:at + n].double() for x in ("q", "k", "v"))
        if case["op"] == "cache":
            where = torch.arange(past + n, device="cuda")
            pages, inside = s["table"][i].long()[where // case["page"]], where % case["page"]
            kc[pages[past:], inside[past:]], vc[pages[past:], inside[past:]] = s["k"][at:at + n], s["v"][at:at + n]
            k, v = kc[pages, inside].double(), vc[pages, inside].double()
        parts = {x: [] for x in out}
        behind = torch.arange(past + n, device="cuda")[None] > past + torch.arange(n, device="cuda")[:, None]
        for h in range(H):
            qh, kh, vh = q[:, h], k[:, h // grp], v[:, h // grp]
            x = torch.matmul(qh, kh.t().contiguous()) * scale
            x[behind] = -math.inf
            if case.get("dir") != "bwd":
                lse = torch.logsumexp(x, 1) if n else x.sum(1)
                parts["o"].append(torch.matmul(torch.exp(x - lse[:, None]), vh))
                if "lse" in parts:
                    parts["lse"].append(lse)
                continue
            # of the outputs and sums that are given, as the pass defines its gradient
            go = s["do"][at:at + n, h].double()
            w = torch.exp(x - s["lse"][at:at + n, h].double()[:, None])
            c = (go * s["o"][at:at + n, h].double()).sum(1, keepdim=True)
            e = scale * w * (torch.matmul(go, vh.t().contiguous()) - c)
            parts["dq"].append(torch.matmul(e, kh))
            dkh, dvh = torch.matmul(e.t().contiguous(), qh), torch.matmul(w.t().contiguous(), go)
            if h % grp == 0:
                parts["dk"].append(dkh)
                parts["dv"].append(dvh)
            else:
                parts["dk"][-1] += dkh
                parts["dv"][-1] += dvh
        for x in out:
            out[x].append(torch.stack(parts[x], 1))
        at += n
    out = {x: torch.cat(v) for x, v in out.items()}
    return {**out, "k_cache": kc.double(), "v_cache": vc.double()} if case["op"] == "cache" else out
