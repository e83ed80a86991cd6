"""Cases of the operators around conditional (LowRank) circuits: layer norm, linear attention with a decay for each
head, and the orthogonalised update.

A LowRank circuit takes per-sample factors A_b [M, k] and B_b [k, N] from a sequence network and gives back dLL/dA and
dLL/dB.  These operators are what such a network is made of: it normalises its features, mixes them along the
sequence, and its matrices are updated from the gradients that the circuit returns.
"""
import math

import torch

own = False

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
BYTES = {"f32": 4, "bf16": 2, "f16": 2}
QUINTIC = (3.4445, -4.7750, 2.0315)
STEPS = 5
LN_EPS = 1e-5
NS_EPS = 1e-7


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # one position's features of a small encoder at a small batch: launch latency
        {"name": "norm_fwd_small", "op": "norm", "dir": "fwd", "type": "f32", "rows": 32, "cols": 768},
        # odd sizes, rows that are not aligned to a vector load
        {"name": "norm_fwd_odd", "op": "norm", "dir": "fwd", "type": "f16", "rows": 9001, "cols": 1001},
        # a training batch of 512 x 32 positions, 4096 features: both directions
        {"name": "norm_bwd_large", "op": "norm", "dir": "bwd", "type": "bf16", "rows": 16384, "cols": 4096},
        # one long prompt, 32 heads
        {"name": "mix_fwd_long", "op": "mix", "dir": "fwd", "type": "bf16", "seqs": 1, "tokens": 16384, "lens": "same",
         "heads": 32, "kv_heads": 32, "dk": 128, "dv": 128},
        # prompts of mixed length (one token and empty ones among them), key and value heads shared by four
        {"name": "mix_fwd_ragged", "op": "mix", "dir": "fwd", "type": "bf16", "seqs": 24, "tokens": 1500, "lens": "ragged",
         "heads": 16, "kv_heads": 4, "dk": 64, "dv": 64},
        # a training batch
        {"name": "mix_bwd_batch", "op": "mix", "dir": "bwd", "type": "bf16", "seqs": 8, "tokens": 2048, "lens": "same",
         "heads": 16, "kv_heads": 16, "dk": 128, "dv": 128},
        # float32 training, ragged, shared heads, odd head sizes
        {"name": "mix_bwd_ragged", "op": "mix", "dir": "bwd", "type": "f32", "seqs": 7, "tokens": 900, "lens": "ragged",
         "heads": 6, "kv_heads": 3, "dk": 48, "dv": 80},
        # one stream, one token: latency
        {"name": "mix_step_one", "op": "mix", "dir": "step", "type": "bf16", "seqs": 1, "tokens": 1, "lens": "same",
         "heads": 16, "kv_heads": 16, "dk": 64, "dv": 64},
        # many streams, one token each: the states are read and written
        {"name": "mix_step_batch", "op": "mix", "dir": "step", "type": "bf16", "seqs": 256, "tokens": 1, "lens": "same",
         "heads": 32, "kv_heads": 8, "dk": 128, "dv": 128},
        # the factor gradients dLL/dA of one LowRank slot: 64 samples, 1024 states, rank 16
        {"name": "orth_factors", "op": "orth", "type": "f32", "batch": 64, "rows": 1024, "cols": 16},
        # a few weight matrices of odd shape
        {"name": "orth_ragged", "op": "orth", "type": "f32", "batch": 3, "rows": 333, "cols": 1000},
        # a square weight matrix of 4096
        {"name": "orth_large", "op": "orth", "type": "bf16", "batch": 1, "rows": 4096, "cols": 4096},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "mix", "mix", "orth"])
    if op == "norm":
        cols = _log(rng, 16, 8192)
        rows = _log(rng, 1, max(1, min(16384, (1 << 26) // cols)))
        return {"op": op, "dir": rng.choice(["fwd", "bwd"]), "type": rng.choice(sorted(TYPES)), "rows": rows, "cols": cols}
    if op == "mix":
        way = rng.choice(["fwd", "bwd", "step"])
        kv = rng.choice([1, 2, 3, 4, 8])
        heads = kv * rng.choice([1, 1, 2, 4])
        dk, dv = (rng.choice([16, 24, 32, 48, 64, 80, 96, 128]) for _ in range(2))
        seqs = _log(rng, 1, 256 if way == "step" else 24)
        tokens = 1 if way == "step" else _log(rng, 1, max(1, min(8192, (1 << 17) // (heads * seqs))))
        return {"op": op, "dir": way, "type": rng.choice(sorted(TYPES)), "seqs": seqs, "tokens": tokens,
                "lens": rng.choice(["same", "ragged"]), "heads": heads, "kv_heads": kv, "dk": dk, "dv": dv}
    kind = rng.choice(["factors", "factors", "matrix", "matrix"])
    typ = rng.choice(sorted(TYPES))
    if kind == "factors":
        k, long, batch = rng.choice([1, 4, 5, 8, 16, 32, 64]), _log(rng, 130, 4096), _log(rng, 1, 256)
    else:
        k, batch = _log(rng, 65, 500), rng.choice([1, 1, 2, 3, 5])
        long = _log(rng, 2 * k, 2500)
    rows, cols = (k, long) if rng.random() < 0.5 else (long, k)
    return {"op": op, "type": typ, "batch": batch, "rows": rows, "cols": cols}


def lengths(case):
    """Tokens of each sequence: all the same, or from none to the most, in a fixed order."""
    n, most = case["seqs"], case["tokens"]
    if case["lens"] == "same" or case["dir"] == "step":
        return [most] * n
    out = [most]
    for i in range(1, n):
        out.append((0, 1, most // 2 + i, most // 3, most // 7 + 2 * i, most // 5, most - i)[(i - 1) % 7])
    return [max(0, min(most, x)) for x in out]


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
    if case["op"] == "norm":
        r, c = case["rows"], case["cols"]
        s["x"] = (torch.randn((r, c), generator=g, device="cuda") *
                  (0.5 + torch.rand((r, 1), generator=g, device="cuda") * 2) + 0.3).to(t)
        s["weight"] = normal(c, dtype=torch.float32, scale=0.2, shift=1.0)
        s["bias"] = normal(c, dtype=torch.float32, scale=0.1)
        if case["dir"] == "bwd":
            s["dy"] = normal(r, c)
            xd = s["x"].double()      # what the forward pass kept
            s["mean"] = xd.mean(1).float()
            s["rstd"] = (xd.var(1, unbiased=False) + LN_EPS).rsqrt().float()
            del xd
        if own:
            import log_space_sum_amd as L
            if case["dir"] == "bwd":
                s["dx"] = torch.empty_like(s["x"])
                s["dweight"], s["dbias"] = torch.empty_like(s["weight"]), torch.empty_like(s["bias"])
                s["ws"] = L.layer_norm_workspace(r, c, s["x"].device)
            else:
                s["y"] = torch.empty_like(s["x"])
                s["mean"], s["rstd"] = (torch.empty(r, device="cuda") for _ in range(2))
        return s
    if case["op"] == "orth":
        s["g"] = normal(case["batch"], case["rows"], case["cols"], scale=1e-3)
        if own:
            import log_space_sum_amd as L
            s["out"] = torch.empty_like(s["g"])
            s["ws"] = L.orthogonalize_workspace(s["g"])
        return s
    H, K, dk, dv = case["heads"], case["kv_heads"], case["dk"], case["dv"]
    lens = lengths(case)
    T = sum(lens)
    s["log_decay"] = -torch.exp2(-8.0 * torch.arange(H, device="cuda", dtype=torch.float32) / H)
    s["q"], s["k"], s["v"] = normal(T, H, dk), normal(T, K, dk), normal(T, K, dv)
    s["state"] = normal(len(lens), H, dk, dv, dtype=torch.float32, scale=0.5)
    if case["dir"] == "step":
        s["o"] = torch.empty((T, H, dv), dtype=t, device="cuda")
        return s
    s["lens"], s["longest"] = lens, max(lens)
    s["cu"] = torch.tensor([sum(lens[:i]) for i in range(len(lens) + 1)], dtype=torch.int32, device="cuda")
    # where each token lies in a batch padded to the longest sequence: the plan that the plain form gathers by
    at = torch.tensor([i for i, n in enumerate(lens) for _ in range(n)], device="cuda", dtype=torch.int64)
    s["row"] = at
    s["col"] = torch.arange(T, device="cuda") - s["cu"].long()[at]
    s["len"] = torch.tensor(lens, device="cuda", dtype=torch.int64)
    if case["dir"] == "bwd":
        s["do"] = normal(T, H, dv)
        s["dstate"] = normal(len(lens), H, dk, dv, dtype=torch.float32, scale=0.1)
    if own:
        import log_space_sum_amd as L
        s["ws"] = L.linear_attention_workspace(s["q"], s["k"], s["v"], s["cu"], s["longest"],
                                                  backward=case["dir"] == "bwd")
        if case["dir"] == "fwd":
            s["o"], s["state_out"] = torch.empty((T, H, dv), dtype=t, device="cuda"), torch.empty_like(s["state"])
        else:
            s["dq"], s["dk"], s["dv"] = (torch.empty_like(s[x]) for x in ("q", "k", "v"))
            s["dstate_in"] = torch.empty_like(s["state"])
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(s):
    case = s["case"]
    if own:
        return _run_own(s, case)
    if case["op"] == "norm":
        return _norm_forward(s) if case["dir"] == "fwd" else _norm_backward(s)
    if case["op"] == "orth":
        return _orth(s)
    return {"fwd": _mix_forward, "bwd": _mix_backward, "step": _mix_step}[case["dir"]](s)


def _run_own(s, case):
    import log_space_sum_amd as L
    if case["op"] == "norm":
        if case["dir"] == "fwd":
            L.pc_layer_norm_forward(s["x"], s["weight"], s["bias"], s["y"], s["mean"], s["rstd"], eps=LN_EPS)
            return {"y": s["y"], "mean": s["mean"], "rstd": s["rstd"]}
        L.pc_layer_norm_backward(s["dy"], s["x"], s["weight"], s["mean"], s["rstd"], s["dx"], s["dweight"], s["dbias"],
                                 ws=s["ws"])
        return {"dx": s["dx"], "dweight": s["dweight"], "dbias": s["dbias"]}
    if case["op"] == "orth":
        L.pc_orthogonalize(s["g"], s["out"], steps=STEPS, coefficients=QUINTIC, eps=NS_EPS, ws=s["ws"])
        return {"out": s["out"]}
    if case["dir"] == "step":
        L.pc_linear_attention_step(s["q"], s["k"], s["v"], s["log_decay"], s["state"], s["o"])
        return {"o": s["o"], "state": s["state"]}
    if case["dir"] == "fwd":
        L.pc_linear_attention_forward(s["q"], s["k"], s["v"], s["log_decay"], s["o"], cu_seqlens=s["cu"],
                                      max_seqlen=s["longest"], state_in=s["state"], state_out=s["state_out"], ws=s["ws"])
        return {"o": s["o"], "state": s["state_out"]}
    L.pc_linear_attention_backward(s["do"], s["q"], s["k"], s["v"], s["log_decay"], s["dq"], s["dk"], s["dv"],
                                   cu_seqlens=s["cu"], max_seqlen=s["longest"], state_in=s["state"],
                                   dstate_out=s["dstate"], dstate_in=s["dstate_in"], ws=s["ws"])
    return {"dq": s["dq"], "dk": s["dk"], "dv": s["dv"], "dstate": s["dstate_in"]}


# ---- plain forms: elementary operations in float32 ----

def _norm_forward(s):
    x = s["x"].float()
    mean = x.mean(1, keepdim=True)
    c = x - mean
    rstd = (c.square().mean(1, keepdim=True) + LN_EPS).rsqrt()
    y = c * rstd * s["weight"] + s["bias"]
    return {"y": y.to(s["x"].dtype), "mean": mean[:, 0], "rstd": rstd[:, 0]}


def _norm_backward(s):
    x, dy, rstd = s["x"].float(), s["dy"].float(), s["rstd"][:, None]
    n = (x - s["mean"][:, None]) * rstd
    g = dy * s["weight"]
    dx = rstd * (g - g.mean(1, keepdim=True) - n * (g * n).mean(1, keepdim=True))
    return {"dx": dx.to(s["x"].dtype), "dweight": (dy * n).sum(0), "dbias": dy.sum(0)}


def _orth(s):
    g = s["g"].float()
    a, b, c = QUINTIC
    tall = g.shape[1] > g.shape[2]
    x = g.mT.contiguous() if tall else g
    x = x / (x.square().sum((1, 2), keepdim=True).sqrt() + NS_EPS)
    for _ in range(STEPS):
        m = x @ x.mT
        x = a * x + (b * m + c * (m @ m)) @ x
    return {"out": (x.mT if tall else x).to(s["g"].dtype).contiguous()}


CHUNK = 128


def _mix(q, k, v, gamma, state, length):
    """o_t = q_t^T S_t with S_t = exp(gamma) S_{t-1} + k_t v_t^T, and the state after `length` tokens, of padded
    float32 batches [n, H, T, d]: within chunks as a masked product, between chunks through their states.
    Tokens behind a sequence's length have k = v = 0."""
    n, H, T, dk = q.shape
    dv, C = v.shape[3], min(CHUNK, max(1, T))
    N = -(-T // C)
    if N * C != T:
        q, k, v = (torch.nn.functional.pad(x, (0, 0, 0, N * C - T)) for x in (q, k, v))
    q, k, v = (x.reshape(n, H, N, C, x.shape[3]) for x in (q, k, v))
    i = torch.arange(C, device=q.device, dtype=torch.float32)
    gap = i[:, None] - i[None, :]
    g = gamma[:, None, None]
    mask = torch.where(gap >= 0, torch.exp(g * gap.clamp(min=0)), 0.0)          # [H, C, C]
    inside = ((q @ k.mT) * mask[:, None]) @ v
    part = (k * torch.exp(g * (C - 1 - i)[:, None])[:, None]).mT @ v            # [n, H, N, dk, dv]
    j = torch.arange(N + 1, device=q.device, dtype=torch.float32)
    far = j[:, None] - 1 - j[None, :N]
    carry = torch.where(far >= 0, torch.exp(g * C * far.clamp(min=0)), 0.0)     # [H, N + 1, N]
    start = (carry @ part.reshape(n, H, N, dk * dv)).reshape(n, H, N + 1, dk, dv)
    start = start + torch.exp(g * C * j[:, None])[..., None] * state[:, :, None]
    o = inside + (q * torch.exp(g * (i + 1)[:, None])[:, None]) @ start[:, :, :N]
    # the state after `length` tokens: that of the chunk's start, decayed, and the chunk's own tokens
    at = length // C
    first = start[torch.arange(n, device=q.device), :, at]                      # [n, H, dk, dv]
    used = (length - at * C).float()[:, None, None]
    kk, vv = (x[torch.arange(n, device=q.device), :, at.clamp(max=N - 1)] for x in (k, v))
    w = torch.where(i < used, torch.exp(gamma[None, :, None] * (used - 1 - i).clamp(min=0)), 0.0)
    last = torch.exp(gamma[None, :, None] * used)[..., None] * first + (kk * w[..., None]).mT @ vv
    return o.reshape(n, H, N * C, dv)[:, :, :T], last


def _padded(s, x, heads):
    """[T, h, d] tokens as a padded float32 batch [n, heads, longest, d]; shared heads are repeated."""
    out = torch.zeros((len(s["lens"]), max(1, s["longest"]), x.shape[1], x.shape[2]), device=x.device)
    out[s["row"], s["col"]] = x.float()
    return out.transpose(1, 2).repeat_interleave(heads // x.shape[1], 1)


def _flat(s, x):
    return x.transpose(1, 2)[s["row"], s["col"]]


def _turned(s, x):
    """Each sequence of a padded batch back to front."""
    t = torch.arange(x.shape[2], device=x.device)
    back = s["len"][:, None] - 1 - t[None, :]
    y = torch.gather(x, 2, back.clamp(min=0)[:, None, :, None].expand_as(x))
    return torch.where((back >= 0)[:, None, :, None], y, 0.0)


def _mix_forward(s):
    H = s["case"]["heads"]
    q, k, v = (_padded(s, s[x], H) for x in ("q", "k", "v"))
    o, last = _mix(q, k, v, s["log_decay"], s["state"], s["len"])
    return {"o": (_flat(s, o) * s["q"].shape[2] ** -0.5).to(s["q"].dtype), "state": last}


def _mix_backward(s):
    H, K, gamma, scale = s["case"]["heads"], s["case"]["kv_heads"], s["log_decay"], s["q"].shape[2] ** -0.5
    q, k, v, do = (_padded(s, s[x], H) for x in ("q", "k", "v", "do"))
    t = s["q"].dtype
    dq, _ = _mix(do, v, k, gamma, s["state"].mT.contiguous(), s["len"])
    # the adjoint state D_t = exp(gamma) D_{t+1} + scale q_t do_t^T runs from the sequence's end: at the first token
    # met it is exp(gamma) dstate / exp(gamma), so the walk starts from dstate / exp(gamma)
    q, k, v, do = (_turned(s, x) for x in (q * scale, k, v, do))
    d0 = s["dstate"] * torch.exp(-gamma)[:, None, None]
    dv, d1 = _mix(k, q, do, gamma, d0, s["len"])
    dk, _ = _mix(v, do, q, gamma, d0.mT.contiguous(), s["len"])
    grouped = [_flat(s, _turned(s, x)) for x in (dk, dv)]
    dk, dv = (x.reshape(x.shape[0], K, H // K, x.shape[2]).sum(2) for x in grouped)
    return {"dq": (_flat(s, dq) * scale).to(t), "dk": dk.to(t), "dv": dv.to(t),
            "dstate": d1 * torch.exp(gamma)[:, None, None]}


def _mix_step(s):
    H = s["case"]["heads"]
    q = s["q"].float() * s["q"].shape[2] ** -0.5
    k, v = (s[x].float().repeat_interleave(H // s["case"]["kv_heads"], 1) for x in ("k", "v"))
    s["state"].mul_(torch.exp(s["log_decay"])[None, :, None, None]).add_(k[..., None] * v[..., None, :])
    s["o"].copy_((q[..., None, :] @ s["state"])[..., 0, :])
    return {"o": s["o"], "state": s["state"]}


# ---------------------------------------------------------------------------
# the least work of one pass, and the definitions in 64 bits
# ---------------------------------------------------------------------------

def work(case):
    e = BYTES[case["type"]]
    if case["op"] == "norm":
        n, c = case["rows"] * case["cols"], case["cols"]
        if case["dir"] == "fwd":
            return {"bytes": 2 * n * e + 8 * c + 8 * case["rows"], "flops": 8 * n}
        return {"bytes": 3 * n * e + 12 * c + 8 * case["rows"], "flops": 14 * n}
    if case["op"] == "orth":
        m, n = sorted((case["rows"], case["cols"]))
        # symmetric products count half; either every step on the matrix itself, or all steps on its Gram matrix
        direct = STEPS * (3 * m * m * n + m ** 3)
        gram = 3 * m * m * n + (4 * STEPS - 3) * m ** 3
        return {"bytes": 2 * case["batch"] * m * n * e, "flops": case["batch"] * min(direct, gram)}
    T, H, K, dk, dv = sum(lengths(case)), case["heads"], case["kv_heads"], case["dk"], case["dv"]
    state = case["seqs"] * H * dk * dv * 4
    tokens = T * (H * dk + K * dk + K * dv + H * dv) * e
    if case["dir"] == "bwd":
        return {"bytes": tokens + T * (H * dk + K * dk + K * dv) * e + 3 * state + 4 * H, "flops": 10 * T * H * dk * dv}
    return {"bytes": tokens + 2 * state + 4 * H, "flops": 4 * T * H * dk * dv}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        x, w, b = s["x"].double(), s["weight"].double(), s["bias"].double()
        mu = x.sum(1) / case["cols"]
        var = ((x - mu[:, None]) ** 2).sum(1) / case["cols"]
        r = 1.0 / torch.sqrt(var + LN_EPS)
        if case["dir"] == "fwd":
            return {"y": (x - mu[:, None]) * r[:, None] * w + b, "mean": mu, "rstd": r}
        # of the statistics that are given, as the pass defines its gradient
        mu, r, dy = s["mean"].double(), s["rstd"].double(), s["dy"].double()
        h = (x - mu[:, None]) * r[:, None]
        p = dy * w
        dx = r[:, None] * (p - (p.sum(1) / case["cols"])[:, None] - h * ((p * h).sum(1) / case["cols"])[:, None])
        return {"dx": dx, "dweight": (dy * h).sum(0), "dbias": dy.sum(0)}
    if case["op"] == "orth":
        g = s["g"].double()
        if case["rows"] > case["cols"]:
            g = g.transpose(1, 2).contiguous()
        a, b, c = QUINTIC
        g = g / (torch.linalg.vector_norm(g, dim=(1, 2), keepdim=True) + NS_EPS)
        for _ in range(STEPS):
            m = torch.matmul(g, g.transpose(1, 2).contiguous())
            p = torch.matmul(m, g)
            g = a * g + b * p + c * torch.matmul(m, p)
        return {"out": g.transpose(1, 2).contiguous() if case["rows"] > case["cols"] else g}
    H, K, scale = case["heads"], case["kv_heads"], case["dk"] ** -0.5
    lam = torch.exp(s["log_decay"].double())[:, None, None]
    head = torch.arange(H, device="cuda") // (H // K)
    q, k, v = s["q"].double(), s["k"].double()[:, head], s["v"].double()[:, head]
    S = s["state"].double()
    if case["dir"] == "step":
        S = lam * S + k[:, :, :, None] * v[:, :, None, :]
        return {"o": scale * (q[:, :, :, None] * S).sum(2), "state": S}
    # token by token, all sequences that have such a token at once
    lens = s["lens"]
    cu = [sum(lens[:i]) for i in range(len(lens) + 1)]
    live = []
    for t in range(s["longest"]):
        if t == 0 or any(n == t for n in lens):
            ids = [i for i, n in enumerate(lens) if n > t]
            seq = torch.tensor(ids, device="cuda")
            base = torch.tensor([cu[i] for i in ids], device="cuda")
        live.append((seq, base))
    o = torch.zeros_like(s["q"].double()[:, :, :1]).repeat(1, 1, case["dv"])
    if case["dir"] == "fwd":
        for t in range(s["longest"]):
            seq, at = live[t][0], live[t][1] + t
            S[seq] = lam * S[seq] + k[at][..., :, None] * v[at][..., None, :]
            o[at] = scale * torch.matmul(q[at][..., None, :], S[seq])[..., 0, :]
        return {"o": o, "state": S}
    do, D = s["do"].double(), s["dstate"].double()
    dq, dk, dv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    for t in range(s["longest"]):
        seq, at = live[t][0], live[t][1] + t
        S[seq] = lam * S[seq] + k[at][..., :, None] * v[at][..., None, :]
        dq[at] = scale * torch.matmul(S[seq], do[at][..., :, None])[..., 0]
    for t in range(s["longest"] - 1, -1, -1):
        seq, at = live[t][0], live[t][1] + t
        now = D[seq] + scale * q[at][..., :, None] * do[at][..., None, :]
        dk[at] = torch.matmul(now, v[at][..., :, None])[..., 0]
        dv[at] = torch.matmul(k[at][..., None, :], now)[..., 0, :]
        D[seq] = lam * now
    dk, dv = (x.reshape(x.shape[0], K, H // K, x.shape[2]).sum(2) for x in (dk, dv))
    return {"dq": dq, "dk": dk, "dv": dv, "dstate": D}
