"""Softmax attention and the heads' rotation on the GPU against their float64 definitions.

Tolerances.  u: half a step of the output's type (2^-24, 2^-8, 2^-11 of the value); E = 2^-24.  A float32 sum of n
products in any order is off by at most (n + 2) E times the sum of their magnitudes.  So a score is off by (dk + 4) E times
scale sum |q k|, and the exponential of x by that and (|x| + 4) E of itself: together `e` of a weight, relative.  Sums over keys or rows add
(n + 16) E of the magnitudes.  What is computed and multiplied again keeps 2^-21 of itself (three bfloat16 planes 2^-24, products of planes
that are left out for float32 2^-22, two float16 planes 2^-21).  Magnitudes are the definition's on absolute values."""
import math

import numpy as np
import pytest

from oracle import ops_oracle as R

pytestmark = pytest.mark.gpu
U = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}
TINY = {"f32": 2.0 ** -126, "bf16": 2.0 ** -126, "f16": 2.0 ** -25}
E = 2.0 ** -24
KEPT = 2.0 ** -21
DEV = "cuda:0"


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import log_space_sum_amd as L
    L.lib()


def T():
    import torch
    return torch, {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def put(a, typ="f32"):
    torch, types = T()
    return torch.tensor(np.ascontiguousarray(a, dtype=np.float32), device=DEV).to(types[typ])


def ints(a):
    torch, _ = T()
    return torch.tensor(np.asarray(a, np.int32), device=DEV)


def get(t):
    return t.detach().double().cpu().numpy()


def near(got, want, tol, what):
    got = get(got)
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), (what, int(bad.sum()), float(np.nanmax(np.abs(got - want)[bad])), np.argwhere(bad)[:3].tolist())


# ---------------------------------------------------------------------------
# norm and rotation
# ---------------------------------------------------------------------------

ROT = [(1, 1, 1, 2, 2), (1, 16, 4, 64, 64), (7, 3, 0, 128, 128), (33, 5, 2, 80, 40), (130, 2, 7, 48, 6), (3, 1, 1, 9, 4), (5, 4, 4, 256, 256),
       (2500, 3, 1, 24, 24), (4, 6, 3, 31, 0), (9, 70, 70, 16, 8)]


@pytest.mark.parametrize("typ", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("n,H,K,d,part", ROT)
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("norm", [False, True])
def test_rotary(n, H, K, d, part, inter, norm, typ):
    """y and dx: a norm's sums of d products, two products a pair, angles exact in float32: (d / 4 + 16) E of the pair's size;
    the weights' gradients: sums over n heads' rows."""
    import log_space_sum_amd as L
    torch, types = T()
    rng = np.random.default_rng(n + d + part)
    # heads at odd strides inside wider rows
    whole = put(rng.normal(size=(n, H + K, d + 3)) * 1.5, typ)
    q, k = whole[:, :H, 1:1 + d], whole[:, H:, 1:1 + d]
    pos = rng.integers(-5, 10 ** 6, n)
    freq = L.rotary_frequencies(part, 10000.0, "parts" if part else None, 8.0, 16384.0, device=DEV)
    w = [put(rng.normal(size=d) * 0.2 + 1) if norm else None for _ in range(2)]
    mag = 1.25
    how = dict(interleaved=inter, magnitude=mag, norm=norm)
    out = torch.full((n, H + K, d + 5), 7.0, device=DEV, dtype=types[typ])
    qo, ko = out[:, :H, 2:2 + d], out[:, H:, 2:2 + d]
    L.pc_rotary_forward(q, k if K else None, qo, ko if K else None, ints(pos), freq, q_weight=w[0], k_weight=w[1], **how)
    dy = put(rng.normal(size=(n, H + K, d)), typ)
    dx = torch.full_like(dy, 7.0)
    dw = [torch.full((d,), 7.0, device=DEV) if norm else None for _ in range(2)]
    ws = L.rotary_workspace(q, k if K else None)
    both = dict(q=q, k=k if K else None, q_weight=w[0], k_weight=w[1], dq_weight=dw[0], dk_weight=dw[1], ws=ws, **how) if norm else how
    L.pc_rotary_backward(dy[:, :H], dy[:, H:] if K else None, dx[:, :H], dx[:, H:] if K else None, ints(pos), freq, **both)
    f = get(freq)
    for x, y, g, gx, wt, gw, heads in ((q, qo, dy[:, :H], dx[:, :H], w[0], dw[0], H), (k, ko, dy[:, H:], dx[:, H:], w[1], dw[1], K)):
        if not heads:
            if norm:
                assert not gw.any()
            continue
        xs, gs, wv = get(x), get(g), get(wt) if norm else None
        args = dict(interleaved=inter, norm=norm, w=wv)
        want = R.rotary(xs, pos, f, magnitude=mag, **args)
        size = np.abs(R.rotary(xs, pos * 0, f, **args))       # before it is turned
        pair = mag * np.maximum(size, R.rotary(size, pos * 0 + 0, f * 0, interleaved=inter)) + mag * _partner(size, part, inter)
        near(y, want, TINY[typ] + U[typ] * np.abs(want) + (d / 4 + 16) * E * pair, "y")
        ref, rw = R.rotary_grad(gs, xs, pos, f, inter, mag, norm, wv)
        turned = mag * (np.abs(gs) + _partner(np.abs(gs), part, inter))
        if norm:
            r = 1 / np.sqrt((xs * xs).mean(-1, keepdims=True) + 1e-6)
            nn, big = np.abs(xs) * r, turned * np.abs(wv)
            turned_dx = r * (big + nn * (big * nn).mean(-1, keepdims=True))
            near(gw, rw, (n * heads + d / 4 + 16) * E * (turned * nn).sum((0, 1)), "dw")
        else:
            turned_dx = turned
        near(gx, ref, TINY[typ] + U[typ] * np.abs(ref) + (d / 4 + 24) * E * turned_dx, "dx")
    assert (out[..., :2] == 7).all() and (out[..., 2 + d:] == 7).all()
    # in place: the same bits
    a = whole.clone()
    qa, ka = a[:, :H, 1:1 + d], a[:, H:, 1:1 + d]
    L.pc_rotary_forward(qa, ka if K else None, qa, ka if K else None, ints(pos), freq, q_weight=w[0], k_weight=w[1], **how)
    assert torch.equal(qa, qo) and torch.equal(ka, ko)
    b = dy.clone()
    L.pc_rotary_backward(b[:, :H], b[:, H:] if K else None, b[:, :H], b[:, H:] if K else None, ints(pos), freq, **both)
    assert torch.equal(b, dx)


def _partner(x, part, inter):
    y = np.zeros_like(x)
    n = part // 2
    a, b = (np.arange(0, part, 2), np.arange(1, part, 2)) if inter else (np.arange(n), np.arange(n, part))
    y[..., a], y[..., b] = x[..., b], x[..., a]
    return y


@pytest.mark.parametrize("typ", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("n,H,K,d,part", [(9001, 3, 1, 24, 24), (4099, 6, 2, 128, 64)])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("norm", [False, True])
def test_rotary_of_more_tokens_than_waves(n, H, K, d, part, inter, norm, typ):
    """The backward pass has 4096 waves at most: each takes a second token, its angles anew, its sums carried on."""
    test_rotary(n, H, K, d, part, inter, norm, typ)


def test_rotary_of_far_positions():
    """Positions up to 2^31 - 1 and below 0 with pairs of a radian a position: 64-bit angles."""
    import log_space_sum_amd as L
    torch, _ = T()
    pos = np.array([0, 1, -1, 131071, 10 ** 6 + 7, 2 ** 31 - 1, -2 ** 31])
    q = put(np.ones((7, 1, 4)))
    freq = torch.tensor([1.0, 0.7], dtype=torch.float64, device=DEV)
    out = torch.empty_like(q)
    L.pc_rotary_forward(q, None, out, None, ints(pos), freq)
    near(out, R.rotary(get(q), pos, get(freq)), 2.0 ** -21, "far")


def test_rotary_edges():
    import log_space_sum_amd as L
    torch, _ = T()
    freq = L.rotary_frequencies(8, device=DEV)
    # no tokens: the weights' gradients are 0
    e, z = torch.empty((0, 3, 8), device=DEV), ints([])
    w, dw = put(np.ones(8)), torch.full((8,), 5.0, device=DEV)
    L.pc_rotary_forward(e, e, e, e, z, freq)
    L.pc_rotary_backward(e, e, e, e, z, freq, norm=True, q=e, k=e, q_weight=w, k_weight=w, dq_weight=dw, dk_weight=dw.clone(), ws=L.rotary_workspace(e, e))
    assert not dw.any()
    # a head that is not finite reaches no other; a head of zeros stays zeros
    x = put(np.random.default_rng(0).normal(size=(4, 3, 8)))
    x[1, 1, 2], x[2, 0] = math.nan, 0
    y = torch.empty_like(x)
    L.pc_rotary_forward(x, None, y, None, ints(range(4)), freq, norm=True)
    bad = torch.isnan(y).any(-1)
    assert bad[1, 1] and bad.sum() == 1 and not y[2, 0].any()
    with pytest.raises(ValueError):
        L.pc_rotary_forward(x, None, y, None, ints(range(4)), freq, q_weight=w)
    with pytest.raises(TypeError):
        L.pc_rotary_forward(x, None, y, None, ints(range(4)), freq.float())
    with pytest.raises(L.PCError):
        L.pc_rotary_backward(x, None, y, None, ints(range(4)), freq, norm=True, q=x, q_weight=w, dq_weight=dw)
    # gradients of the weights are the same bits at every run
    big = put(np.random.default_rng(1).normal(size=(5000, 4, 8)), "bf16")
    ws, first = L.rotary_workspace(big), None
    for _ in range(3):
        L.pc_rotary_backward(big, None, torch.empty_like(big), None, ints(range(5000)), freq, norm=True, q=big, dq_weight=dw, ws=ws)
        assert first is None or torch.equal(first, dw)
        first = dw.clone()


# ---------------------------------------------------------------------------
# whole sequences
# ---------------------------------------------------------------------------

def _cu(lens, start=0):
    return [start + sum(lens[:i]) for i in range(len(lens) + 1)]


def _qkv(rng, T_, H, K, dk, dv, typ, size=1.0):
    return (put(rng.normal(size=(T_, H, dk)) * size, typ), put(rng.normal(size=(T_, K, dk)) * size, typ), put(rng.normal(size=(T_, K, dv)), typ),
            put(rng.normal(size=(T_, H, dv)), typ))


def _errors(q, k, v, scale, past=0):
    """(tolerance of o without its rounding, of lse, `e` [H, n, m], weights) of one sequence, all of float64 values."""
    x, g = R._scores(q, k, scale, past), q.shape[1] // k.shape[1]
    size = R._scores(np.abs(q), np.abs(k), abs(scale), past)
    lse = np.log(np.exp(x - x.max(-1, keepdims=True)).sum(-1, keepdims=True)) + x.max(-1, keepdims=True)
    w = np.exp(x - lse)
    m, dk = x.shape[2], q.shape[2]
    live = np.isfinite(x)
    far = np.where(live, np.abs(np.where(live, x, 0) - x.max(-1, keepdims=True)) + np.abs(x.max(-1, keepdims=True)), 0)
    e = np.where(live, (dk + 4) * E * np.where(live, size, 0) + (far + 4) * E + KEPT, 0)
    row = (w * e).sum(-1)
    vv = np.abs(np.repeat(v, g, 1))
    o = np.einsum("hij,jhd->ihd", w * e, vv) + (row.T[..., None] + (m + 16) * E) * np.einsum("hij,jhd->ihd", w, vv)
    return o, row.T + (m + 16) * E + 2 * E * np.abs(lse[..., 0].T), e, w


def _check_forward(q, k, v, o, lse, cu, scale, typ):
    Q, K, V = get(q), get(k), get(v)
    ro, rl = R.softmax_attention(Q, K, V, cu, scale)
    to, tl = np.zeros_like(ro), np.zeros_like(rl)
    for a, b in zip(cu[:-1], cu[1:]):
        if b > a:
            to[a:b], tl[a:b] = _errors(Q[a:b], K[a:b], V[a:b], scale)[:2]
    i = slice(cu[0], cu[-1])
    near(o[i], ro[i], TINY[typ] + U[typ] * np.abs(ro[i]) + to[i], "o")
    if lse is not None:
        near(lse[i], rl[i], tl[i], "lse")
    return ro, rl


def _check_backward(do, q, k, v, o, lse, grads, cu, scale, typ):
    Q, K, V, DO, O, LSE = (get(t) for t in (q, k, v, do, o, lse))
    ref = R.softmax_attention_grad(DO, Q, K, V, O, LSE, cu, scale)
    g = Q.shape[1] // K.shape[1]
    for a, b in zip(cu[:-1], cu[1:]):
        if b == a:
            continue
        n = b - a
        x = R._scores(Q[a:b], K[a:b], scale, 0)
        p = np.exp(x - LSE[a:b].T[..., None])
        _, _, e, _ = _errors(Q[a:b], K[a:b], V[a:b], scale)
        # the exponent's constant is lse in units of log 2, rounded once more
        e = np.where(p > 0, e + 2 * E * np.abs(LSE[a:b].T[..., None]), 0)
        vv, kk = np.abs(np.repeat(V[a:b], g, 1)), np.abs(np.repeat(K[a:b], g, 1))
        qq, gg = np.abs(Q[a:b]), np.abs(DO[a:b])
        size = np.einsum("ihd,jhd->hij", gg, vv) + (gg * np.abs(O[a:b])).sum(-1).T[..., None]     # of dP - delta
        dS = p * size
        eS = dS * (e + (V.shape[2] + 8) * E + KEPT) + dS * (n + 16) * E
        tq = abs(scale) * np.einsum("hij,jhd->ihd", eS, kk)
        rows = n * g
        tk = abs(scale) * np.einsum("hij,ihd->jhd", eS + dS * (rows + 16) * E, qq)
        tv = np.einsum("hij,ihd->jhd", p * (e + (rows + 16) * E), gg)
        tk, tv = (t.reshape(n, K.shape[1], g, -1).sum(2) for t in (tk, tv))
        for got, want, tol, name in zip(grads, ref, (tq, tk, tv), ("dq", "dk", "dv")):
            near(got[a:b], want[a:b], TINY[typ] + U[typ] * np.abs(want[a:b]) + tol, name)
    return ref


SHAPES = [([1], 1, 1, 64, 64), ([130], 2, 1, 64, 64), ([5, 0, 200, 33], 4, 2, 128, 128), ([70, 300], 6, 3, 48, 80), ([129, 1, 1], 3, 1, 7, 33),
          ([31, 32, 33, 64, 65, 127, 128], 2, 2, 16, 128), ([20] * 70, 5, 1, 24, 40), ([257], 33, 1, 32, 8), ([40], 160, 1, 8, 1), ([600], 1, 1, 1, 128), ([600, 5, 400], 2, 1, 64, 64),
          ([520, 256], 3, 1, 128, 96)]


@pytest.mark.parametrize("typ", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("lens,H,K,dk,dv", SHAPES)
def test_attention(lens, H, K, dk, dv, typ):
    """Outputs, sums and gradients; tokens in front of the first and behind the last sequence are left as they were."""
    import log_space_sum_amd as L
    torch, _ = T()
    rng = np.random.default_rng(len(lens) + dk)
    cu = _cu(lens, 3)
    n = cu[-1] + 2
    q, k, v, do = _qkv(rng, n, H, K, dk, dv, typ)
    for t in (q, k, v, do):                 # nobody's tokens: not to be read
        t[:3], t[cu[-1]:] = math.nan, math.nan
    o, lse = torch.full_like(do, 7.0), torch.full((n, H), 7.0, device=DEV)
    L.pc_attention_forward(q, k, v, o, lse, ints(cu), max(lens))
    _check_forward(q, k, v, o, lse, cu, dk ** -0.5, typ)
    grads = [torch.full_like(t, 7.0) for t in (q, k, v)]
    ws = L.attention_workspace(q, k, v, ints(cu), backward=True)
    L.pc_attention_backward(do, q, k, v, o, lse, *grads, ints(cu), ws=ws)
    _check_backward(do, q, k, v, o, lse, grads, cu, dk ** -0.5, typ)
    for t in (o, lse, *grads):
        assert (t[:3] == 7).all() and (t[cu[-1]:] == 7).all()
    # the same bits again, and without lse
    first = [t.clone() for t in (o, *grads)]
    L.pc_attention_forward(q, k, v, o, None, ints(cu))
    L.pc_attention_backward(do, q, k, v, o, lse, *grads, ints(cu), ws=ws)
    assert all(torch.equal(a, b) for a, b in zip(first, (o, *grads)))
    # keys in parts where there is a workspace, and not cut where the bound of the lengths says so
    o.fill_(7.0), lse.fill_(7.0)
    L.pc_attention_forward(q, k, v, o, lse, ints(cu), ws=L.attention_workspace(q, k, v, ints(cu)))
    _check_forward(q, k, v, o, lse, cu, dk ** -0.5, typ)
    for t in grads:
        t.fill_(7.0)
    L.pc_attention_backward(do, q, k, v, o, lse, *grads, ints(cu), 1, ws=ws)
    _check_backward(do, q, k, v, o, lse, grads, cu, dk ** -0.5, typ)
    for t in (o, lse, *grads):
        assert (t[:3] == 7).all() and (t[cu[-1]:] == 7).all()


@pytest.mark.parametrize("typ", ["bf16", "f16"])
@pytest.mark.parametrize("lens,H,K,dk,dv", [([700, 300], 4, 2, 64, 64), ([400, 513], 2, 1, 128, 128), ([450], 3, 3, 96, 40)])
def test_attention_rounds_a_float32_exact_result(lens, H, K, dk, dv, typ):
    """Normwise, results before their rounding are off by what float32 leaves: scores by sqrt(dk) 2^-25 of their terms (below 2^-22
    here), exponents of a few units by 2^-23, sums of n terms by sqrt(n) 2^-25: 2e-6 in all, 4e-6 allowed.  An element whose value
    lies d from the definition's rounds differently in a share d / step of the cases, then by a step, at most 2 u of the value: the squares of
    the differences from the rounded definition sum to 2 u 4e-6 of the result's.  (Weights rounded to one plane would leave 1e-3 of a result.)"""
    import log_space_sum_amd as L
    torch, _ = T()
    cu = _cu(lens)
    q, k, v, do = _qkv(np.random.default_rng(dk), cu[-1], H, K, dk, dv, typ)
    o, lse = torch.empty_like(do), torch.empty((cu[-1], H), device=DEV)
    L.pc_attention_forward(q, k, v, o, lse, ints(cu))
    dq, dk_, dv_ = (torch.empty_like(t) for t in (q, k, v))
    L.pc_attention_backward(do, q, k, v, o, lse, dq, dk_, dv_, ints(cu), ws=L.attention_workspace(q, k, v, ints(cu), backward=True))
    ref = R.softmax_attention(get(q), get(k), get(v), cu, dk ** -0.5)[:1] + R.softmax_attention_grad(
        get(do), get(q), get(k), get(v), get(o), get(lse), cu, dk ** -0.5)
    for got, want, name in zip((o, dq, dk_, dv_), ref, ("o", "dq", "dk", "dv")):
        off = np.linalg.norm(get(got) - get(put(want, typ)))
        assert off <= np.sqrt(2 * U[typ] * 4e-6) * np.linalg.norm(want), (name, off / np.linalg.norm(want))


@pytest.mark.parametrize("typ", ["f32", "bf16", "f16"])
def test_attention_strides(typ):
    """q, k, v as parts of one packed tensor, outputs head by head, one sequence without cu_seqlens, scales of either sign."""
    import log_space_sum_amd as L
    torch, types = T()
    rng = np.random.default_rng(9)
    n, H, K, d = 150, 4, 2, 64
    packed = put(rng.normal(size=(n, H + 2 * K, d + 1)), typ)
    q, k, v = packed[:, :H, 1:], packed[:, H:H + K, 1:], packed[:, H + K:, :d]
    do = put(rng.normal(size=(H, n, d)), typ).transpose(0, 1)
    o = torch.empty((H, n, d), device=DEV, dtype=types[typ]).transpose(0, 1)
    lse = torch.empty((n, H), device=DEV)
    grads = [torch.empty((t.shape[1], n, d + 3), device=DEV, dtype=types[typ])[..., 3:].transpose(0, 1) for t in (q, k, v)]
    ws = L.attention_workspace(q, k, v, backward=True)
    for scale in (0.3, -0.2):
        L.pc_attention_forward(q, k, v, o, lse, scale=scale)
        _check_forward(q, k, v, o, lse, [0, n], scale, typ)
        L.pc_attention_backward(do, q, k, v, o, lse, *grads, scale=scale, ws=ws)
        _check_backward(do, q, k, v, o, lse, grads, [0, n], scale, typ)


@pytest.mark.parametrize("typ", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("off", ["q", "o", "qo"])
def test_attention_of_rows_that_are_aligned_in_part(off, typ):
    """Aligned keys and values, and queries or outputs an element off."""
    import log_space_sum_amd as L
    torch, _ = T()
    rng = np.random.default_rng(19)
    cu, H, K, d = [0, 130, 200], 4, 2, 64
    q, k, v, do = _qkv(rng, 200, H, K, d, d, typ)

    def moved(t):
        wide = torch.zeros((*t.shape[:2], t.shape[2] + 9), device=DEV, dtype=t.dtype)[..., 1:d + 1]
        wide.copy_(t)
        return wide
    o, lse, dq = torch.empty_like(do), torch.empty((200, H), device=DEV), torch.empty_like(q)
    if "q" in off:
        q, dq = moved(q), moved(dq)
    if "o" in off:
        o, do = moved(o), moved(do)
    L.pc_attention_forward(q, k, v, o, lse, ints(cu), ws=L.attention_workspace(q, k, v, ints(cu)))
    _check_forward(q, k, v, o, lse, cu, d ** -0.5, typ)
    dk, dv = torch.empty_like(k), torch.empty_like(v)
    L.pc_attention_backward(do, q, k, v, o, lse, dq, dk, dv, ints(cu), ws=L.attention_workspace(q, k, v, ints(cu), backward=True))
    _check_backward(do, q, k, v, o, lse, (dq, dk, dv), cu, d ** -0.5, typ)


@pytest.mark.parametrize("typ", ["f32", "bf16", "f16"])
def test_attention_of_large_scores(typ):
    """Scores of hundreds: weights of 1 and 0, sums that move their maximum often."""
    import log_space_sum_amd as L
    torch, _ = T()
    rng = np.random.default_rng(4)
    n, H, d = 300, 2, 64
    q, k, v, do = _qkv(rng, n, H, H, d, d, typ, 5.0)
    k *= put(np.linspace(0.1, 4, n)[:, None, None], typ)
    o, lse = torch.empty_like(do), torch.empty((n, H), device=DEV)
    L.pc_attention_forward(q, k, v, o, lse)
    _check_forward(q, k, v, o, lse, [0, n], d ** -0.5, typ)
    grads = [torch.empty_like(t) for t in (q, k, v)]
    L.pc_attention_backward(do, q, k, v, o, lse, *grads, ws=L.attention_workspace(q, k, v, backward=True))
    _check_backward(do, q, k, v, o, lse, grads, [0, n], d ** -0.5, typ)


@pytest.mark.parametrize("size", [1e-6, 10.0, 1e3])
@pytest.mark.parametrize("typ", ["f32", "bf16", "f16"])
def test_attention_gradients_of_small_and_large_values(typ, size):
    """do of any size: gradients scale with it (float16: as far as its outputs reach)."""
    import log_space_sum_amd as L
    torch, _ = T()
    rng = np.random.default_rng(5)
    n, H, d = 200, 2, 32
    q, k, v, do = _qkv(rng, n, H, 1, d, d, typ)
    do = (do.float() * size * put(np.exp(rng.normal(size=(n, 1, 1)) * 2))).to(do.dtype)
    if not torch.isfinite(do).all():
        pytest.skip("beyond float16")
    o, lse = torch.empty_like(do), torch.empty((n, H), device=DEV)
    L.pc_attention_forward(q, k, v, o, lse)
    grads = [torch.empty_like(t) for t in (q, k, v)]
    L.pc_attention_backward(do, q, k, v, o, lse, *grads, ws=L.attention_workspace(q, k, v, backward=True))
    ref = R.softmax_attention_grad(*(get(t) for t in (do, q, k, v, o, lse)), [0, n], d ** -0.5)
    if typ == "f16" and max(np.abs(r).max() for r in ref) > 60000:
        pytest.skip("beyond float16")
    _check_backward(do, q, k, v, o, lse, grads, [0, n], d ** -0.5, typ)


@pytest.mark.parametrize("typ", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("dk,dv", [(32, 32), (64, 40), (33, 7)])
def test_attention_gradients_of_large_values(dk, dv, typ):
    """do of thousands with small queries, keys and values: gradients up to the end of float16's range, none beyond it."""
    import log_space_sum_amd as L
    torch, _ = T()
    rng = np.random.default_rng(25)
    n, H = 200, 2
    q, k, v, do = _qkv(rng, n, H, 1, dk, dv, typ)
    q, k, v = q * 0.25, k * 0.25, v * 2.0 ** -4
    do.copy_(put(rng.normal(size=(n, H, dv)) * np.exp(rng.normal(size=(n, 1, 1)) * 0.5) * 1500, typ))
    o, lse = torch.empty_like(do), torch.empty((n, H), device=DEV)
    L.pc_attention_forward(q, k, v, o, lse)
    grads = [torch.empty_like(t) for t in (q, k, v)]
    L.pc_attention_backward(do, q, k, v, o, lse, *grads, ws=L.attention_workspace(q, k, v, backward=True))
    ref = _check_backward(do, q, k, v, o, lse, grads, [0, n], dk ** -0.5, typ)
    assert 3000 < max(np.abs(r).max() for r in ref) < 60000


@pytest.mark.parametrize("typ", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("n,H,dk,dv", [(400, 1, 32, 32), (900, 4, 64, 40), (200, 3, 33, 7)])
def test_attention_gradients_of_values_with_small_weights(n, H, dk, dv, typ):
    """A key that no row looks at, of weights of 2^-37 and less, under gradients of a scaled loss (2^13 / H): sums of many rows that a
    float16 holds again, to the bits of their weights."""
    import log_space_sum_amd as L
    torch, _ = T()
    rng = np.random.default_rng(n)
    q, k, v, do = _qkv(rng, n, H, 1, dk, dv, typ)
    q[:], k[:] = 0, 0
    q[..., 0], k[5, 0, 0] = 1, -24
    v *= 2.0 ** -8
    do.copy_(put(rng.uniform(0.5, 1, size=(n, H, dv)) * 2.0 ** 13 / H, typ))
    o, lse = torch.empty_like(do), torch.empty((n, H), device=DEV)
    L.pc_attention_forward(q, k, v, o, lse, scale=1.0)
    grads = [torch.empty_like(t) for t in (q, k, v)]
    L.pc_attention_backward(do, q, k, v, o, lse, *grads, scale=1.0, ws=L.attention_workspace(q, k, v, backward=True))
    ref = _check_backward(do, q, k, v, o, lse, grads, [0, n], 1.0, typ)
    assert np.abs(ref[2][5]).min() > 2.0 ** -21


@pytest.mark.parametrize("typ", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("what", ["q", "k", "v", "do"])
@pytest.mark.parametrize("value", [math.inf, -math.inf, math.nan])
def test_attention_keeps_what_is_not_finite_in_its_place(typ, what, value):
    """An infinity or NaN at one token of one head reaches its own and later rows (gradients of keys: its own and earlier ones) of
    its sequence and head alone; everything else is what it is without it."""
    import log_space_sum_amd as L
    torch, _ = T()
    rng = np.random.default_rng(6)
    cu, H, d, at, head = [0, 90, 260, 300], 2, 64, 150, 1
    q, k, v, do = _qkv(rng, 300, H, H, d, d, typ)

    def run():
        o, lse = torch.empty_like(do), torch.empty((300, H), device=DEV)
        L.pc_attention_forward(q, k, v, o, lse, ints(cu), ws=L.attention_workspace(q, k, v, ints(cu)))
        grads = [torch.empty_like(t) for t in (q, k, v)]
        L.pc_attention_backward(do, q, k, v, o, lse, *grads, ints(cu), ws=L.attention_workspace(q, k, v, ints(cu), backward=True))
        return [get(t) for t in (o, lse[..., None], *grads)]
    clean = run()
    {"q": q, "k": k, "v": v, "do": do}[what][at, head, 5] = value
    dirty = run()
    reach = {"q": [(at, at + 1)] * 3 + [(90, at + 1)] * 2,
             "k": [(at, 260)] * 3 + [(90, 260)] * 2,
             "v": [(at, 260), (0, 0), (at, 260), (90, 260), (90, 260)],
             "do": [(0, 0), (0, 0), (at, at + 1), (90, at + 1), (90, at + 1)]}[what]
    for a, b, (lo, hi), name in zip(clean, dirty, reach, ("o", "lse", "dq", "dk", "dv")):
        free = np.ones(a.shape[:2], bool)
        free[lo:hi, head] = False
        # (rows that a tile takes again in plain float32 round by themselves: a few units of the last place)
        rms = np.sqrt((a * a).mean())
        assert (np.abs(a - b)[free] <= 2 * U[typ] * np.abs(a[free]) + 1e-5 * rms).all(), name
    # of the rows that it reaches, finite where the definition is: a score of -inf has weight 0, one of +inf or NaN none
    with np.errstate(invalid="ignore"):
        ro, rl = R.softmax_attention(get(q), get(k), get(v), cu, d ** -0.5)
    i = slice(at, 260)
    assert (np.isfinite(dirty[0][i]) == np.isfinite(ro[i])).all() and (np.isfinite(dirty[1][i, :, 0]) == np.isfinite(rl[i])).all()
    if what == "v":      # the column of v alone: a weight times the value
        own = dirty[0][at:260, head, 5]
        with np.errstate(invalid="ignore"):
            assert (own == value).all() or (np.isnan(value) and np.isnan(own).all())


def test_attention_edges():
    import log_space_sum_amd as L
    torch, _ = T()
    e = torch.empty((0, 2, 8), device=DEV)
    ws = L.attention_workspace(e, e, e, ints([0, 0]), backward=True)
    L.pc_attention_forward(e, e, e, e, torch.empty((0, 2), device=DEV), ints([0, 0]))
    L.pc_attention_backward(e, e, e, e, e, torch.empty((0, 2), device=DEV), e, e, e, ints([0, 0]), ws=ws)
    x = put(np.ones((4, 2, 8)))
    for bad in (ints([0, 4])[None], ints([])):
        with pytest.raises(ValueError):
            L.pc_attention_forward(x, x, x, x.clone(), None, bad)
    with pytest.raises(TypeError):
        L.pc_attention_forward(x, x.bfloat16(), x, x.clone())
    with pytest.raises(ValueError):
        L.pc_attention_forward(x, x, x, torch.empty((4, 2, 9), device=DEV))
    with pytest.raises(ValueError):
        L.pc_attention_forward(x.cpu(), x, x, x.clone())
    with pytest.raises(L.PCError):
        L.pc_attention_backward(x, x, x, x, x, torch.zeros((4, 2), device=DEV), *(x.clone() for _ in range(3)))
    # offsets that lie outside the tokens are clamped
    o = torch.full_like(x, 7.0)
    L.pc_attention_forward(x, x, x, o, None, ints([-3, 2, 9]))
    assert (o == 1).all()


@pytest.mark.parametrize("typ", ["f32", "bf16"])
@pytest.mark.parametrize("cu", [[0, 600, 10, 610], [-4, 30, 20, 50, 2000], [590, 3, 3, 610, 0], [2000, 600, 500, 0], "random"])
def test_attention_of_offsets_that_fall_stays_inside_its_tensors(cu, typ):
    """Which rows are computed is not defined then, but nothing around the tensors is touched, whole sequences, their gradients and
    over a cache; the next call is right."""
    import log_space_sum_amd as L
    torch, types = T()
    rng = np.random.default_rng(24)
    n, H, K, d, edge = 610, 4, 2, 64, 700
    if cu == "random":
        cu = rng.integers(-10, n + 10, 150).tolist()

    def inside(*shape, dtype=types[typ], fill=7.0):
        whole.append(torch.full((edge + n + edge, *shape), fill, device=DEV, dtype=dtype))
        return whole[-1][edge:edge + n]
    whole = []
    o, dq, dk, dv, lse = inside(H, d), inside(H, d), inside(K, d), inside(K, d), inside(H, dtype=torch.float32)
    q, k, v, do = _qkv(rng, n, H, K, d, d, typ)
    bad, good = ints(cu), ints([0, n])
    seqs = len(cu) - 1
    table = ints(np.arange(seqs * 70).reshape(seqs, 70) + 5)
    kc, vc = (torch.full((seqs * 70 + 10, 16, K, d), 7.0, device=DEV, dtype=types[typ]) for _ in range(2))
    for at in (bad, good):
        past = ints([30] * (at.numel() - 1))
        for most in (n, 40):
            for ws in (None, L.attention_workspace(q, k, v, at, most)):
                L.pc_attention_forward(q, k, v, o, lse, at, most, ws=ws)
                if at is good and most == n:
                    _check_forward(q, k, v, o, lse, [0, n], d ** -0.5, typ)
            L.pc_attention_backward(do, q, k, v, o, lse, dq, dk, dv, at, most, ws=L.attention_workspace(q, k, v, at, most, backward=True))
            if at is good and most == n:
                _check_backward(do, q, k, v, o, lse, (dq, dk, dv), [0, n], d ** -0.5, typ)
            for m in (n, 3):
                t = table[:at.numel() - 1]
                ws = L.attention_cached_workspace(q, kc, vc, t, at, m, most)
                L.pc_attention_cached(q, k, v, kc, vc, t, past, o, at, m, most, ws=ws)
        torch.cuda.synchronize()
        for x in whole:
            assert (x[:edge] == 7).all() and (x[edge + n:] == 7).all()
        for x in (kc, vc):
            assert (x[:5] == 7).all() and (x[seqs * 70 + 5:] == 7).all()


def test_attention_of_many_sequences():
    """More sequences than a search step of 64 x 64 tells apart, none, one or two tokens each."""
    import log_space_sum_amd as L
    torch, _ = T()
    rng = np.random.default_rng(8)
    lens = rng.integers(0, 3, 5000)
    cu = np.concatenate([[0], np.cumsum(lens)])
    n = int(cu[-1])
    q, k, v, _ = _qkv(rng, n, 2, 1, 8, 8, "f32")
    o = torch.empty_like(q)
    L.pc_attention_forward(q, k, v, o, None, ints(cu))
    # with one token o = v; with two a sigmoid of the scores' difference
    Q, K, V = get(q), get(k), get(v)
    want = np.repeat(V, 2, 1)
    second = np.nonzero(np.concatenate([[0], np.repeat(np.arange(5000), lens)[1:] == np.repeat(np.arange(5000), lens)[:-1]]))[0]
    s = np.einsum("ihd,id->ih", Q[second], K[second, 0] - K[second - 1, 0]) * 8 ** -0.5
    w = 1 / (1 + np.exp(-s))[..., None]
    want[second] = w * V[second] + (1 - w) * V[second - 1]
    near(o, want, 2e-6 * (1 + np.abs(want)), "o")


# ---------------------------------------------------------------------------
# over a cache
# ---------------------------------------------------------------------------

class Cache:
    """A cache in pages with sequences of `past` tokens in shuffled pages, their new tokens, and the definition of a call on them."""
    gap = 1     # elements in front of each row: 8 leaves the rows of 16-bit types aligned

    def __init__(self, rng, past, new, H, K, dk, dv, page, typ, spare=2, order="token"):
        torch, types = T()
        self.past, self.new, self.typ, self.page = past, new, typ, page
        self.cu = _cu(new)
        each = max(1, max(-(-(a + b) // page) for a, b in zip(past, new)))
        pages = len(past) * each + spare
        self.table = rng.permutation(pages)[:len(past) * each].reshape(len(past), each)
        shape = {"token": (pages, page, K), "head": (pages, K, page)}[order]
        self.k_cache, self.v_cache = (put(rng.normal(size=(*shape, d + self.gap)), typ)[..., self.gap:] for d in (dk, dv))
        if order == "head":
            self.k_cache, self.v_cache = self.k_cache.transpose(1, 2), self.v_cache.transpose(1, 2)
        self.q, self.k, self.v, self.o = _qkv(rng, self.cu[-1], H, K, dk, dv, typ)

    def rows(self, cache, i, n):
        at = np.arange(n)
        return get(cache)[self.table[i][at // self.page], at % self.page]

    def want(self, scale):
        """(o, tolerance) from the caches before the call."""
        Q, K, V = get(self.q), get(self.k), get(self.v)
        o, tol = np.zeros((self.cu[-1], Q.shape[1], V.shape[2])), np.zeros((self.cu[-1], Q.shape[1], V.shape[2]))
        for i, (p, n) in enumerate(zip(self.past, self.new)):
            a, b = self.cu[i], self.cu[i + 1]
            if n:
                k, v = np.concatenate([self.rows(self.k_cache, i, p), K[a:b]]), np.concatenate([self.rows(self.v_cache, i, p), V[a:b]])
                o[a:b] = R.attend(Q[a:b], k, v, scale, p)[0]
                tol[a:b] = _errors(Q[a:b], k, v, scale, p)[0]
        return o, tol

    def run(self, scale=None, single=False, **kw):
        import log_space_sum_amd as L
        table = ints(self.table)
        cu = None if single else ints(self.cu)
        most = dict(max_seqlen=max(self.new), max_length=max(a + b for a, b in zip(self.past, self.new)))
        most.update(kw)
        ws = L.attention_cached_workspace(self.q, self.k_cache, self.v_cache, table, cu, **most)
        self.o.fill_(7.0)
        L.pc_attention_cached(self.q, self.k, self.v, self.k_cache, self.v_cache, table, ints(self.past), self.o, cu, scale=scale, ws=ws, **most)
        return ws.numel()

    def check(self, scale=None, **kw):
        scale_ = self.q.shape[2] ** -0.5 if scale is None else scale
        want, tol = self.want(scale_)
        before = [self.k_cache.clone(), self.v_cache.clone()]
        n = self.run(scale, **kw)
        near(self.o, want, TINY[self.typ] + U[self.typ] * np.abs(want) + tol, "o")
        # the caches hold the new tokens at their places, and what they held elsewhere
        for cache, was, new in zip((self.k_cache, self.v_cache), before, (self.k, self.v)):
            for i, (p, m) in enumerate(zip(self.past, self.new)):
                for x in range(m):
                    was[self.table[i][(p + x) // self.page], (p + x) % self.page] = new[self.cu[i] + x]
            assert cache.equal(was)
        return n


CACHES = [([0], [1], 1, 1, 64, 64, 16), ([1000], [1], 16, 4, 64, 64, 16), ([700, 0, 3, 64], [1, 1, 1, 1], 8, 2, 128, 128, 24),
          ([100, 0, 517, 33, 0], [5, 17, 0, 1, 40], 6, 3, 48, 80, 24), ([300], [200], 4, 4, 128, 128, 64), ([129, 1], [70, 300], 6, 2, 64, 64, 1),
          ([2000, 90], [9, 64], 3, 1, 7, 33, 100), ([50] * 70, [1] * 70, 2, 1, 32, 16, 7), ([400], [3], 33, 1, 16, 24, 8), ([64], [64], 160, 2, 24, 8, 256)]


@pytest.mark.parametrize("typ", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("past,new,H,K,dk,dv,page", CACHES)
def test_attention_cached(past, new, H, K, dk, dv, page, typ):
    c = Cache(np.random.default_rng(page + dk), past, new, H, K, dk, dv, page, typ)
    c.check()


@pytest.mark.parametrize("typ", ["f32", "bf16", "f16"])
def test_attention_cached_single_tokens_and_orders(typ):
    """One token each without cu_seqlens; pages that lie head by head; a scale below 0; bounds that are not given or too small."""
    rng = np.random.default_rng(11)
    for order in ("token", "head"):
        c = Cache(rng, [30, 0, 900, 257], [1] * 4, 8, 2, 64, 64, 16, typ, order=order)
        c.check(-0.2, single=True)
        first = c.o.clone()
        c.run(-0.2, single=True)
        assert c.o.equal(first)
        c.check(single=True, max_seqlen=None, max_length=None)
        c.check(max_seqlen=1, max_length=1)
        c.check(max_seqlen=900, max_length=10 ** 9)
    c = Cache(rng, [500], [3], 4, 2, 128, 128, 16, typ)
    c.check(single=True)      # one sequence: all tokens are its


@pytest.mark.parametrize("typ", ["f32", "bf16"])
@pytest.mark.parametrize("new", [1, 40])
def test_attention_cached_in_parts(new, typ):
    """Long caches of few streams are cut; streams that end before a part, and bounds far above the lengths."""
    c = Cache(np.random.default_rng(12), [5000, 10, 300], [new] * 3, 4, 2, 64, 64, 32, typ)
    assert c.check() > 0
    c.check(max_length=100000)
    c.check(max_length=600)      # too small a bound: the last part is long


@pytest.mark.parametrize("typ", ["f32", "bf16"])
@pytest.mark.parametrize("total", [128, 129, 256, 257, 511, 512, 513, 640, 769])
def test_attention_cached_of_lengths_around_a_part(total, typ):
    """Lengths where calls begin to be cut, and where parts end."""
    rng = np.random.default_rng(total)
    Cache(rng, [total - 1, total - 3, total - 2], [1, 3, 1], 4, 2, 64, 40, 16, typ).check()


@pytest.mark.parametrize("typ", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("new", [1, 90])
def test_attention_cached_pages_that_are_none(new, typ):
    """Pages outside the cache: their cached positions are not attended, new tokens are attended but not stored; lengths below 0
    and above what the table holds are clamped."""
    import log_space_sum_amd as L
    torch, _ = T()
    rng = np.random.default_rng(13)
    c = Cache(rng, [100, 40], [new] * 2, 4, 2, 64, 64, 16, typ)
    pages = c.k_cache.shape[0]
    c.table[0][1], c.table[0][3], c.table[1][0:2] = -1, pages, 2 ** 31 - 1
    last = (100 + new - 1) // 16
    c.table[0][last] = -7
    Q, K, V = get(c.q), get(c.k), get(c.v)
    before, bv = c.k_cache.clone(), c.v_cache.clone()
    kc, vc = get(before), get(bv)
    c.run()
    for i, p in enumerate(c.past):
        a, b = c.cu[i], c.cu[i + 1]
        there = [j for j in range(p) if 0 <= c.table[i][j // 16] < pages]
        k = np.concatenate([kc[[c.table[i][j // 16] for j in there], [j % 16 for j in there]].reshape(-1, 2, 64), K[a:b]])
        v = np.concatenate([vc[[c.table[i][j // 16] for j in there], [j % 16 for j in there]].reshape(-1, 2, 64), V[a:b]])
        want, tol = R.attend(Q[a:b], k, v, 0.125, len(there))[0], _errors(Q[a:b], k, v, 0.125, len(there))[0]
        near(c.o[a:b], want, TINY[typ] + U[typ] * np.abs(want) + tol, "o")
        for x in range(new):
            t = c.table[i][(p + x) // 16]
            if 0 <= t < pages:
                before[t, (p + x) % 16], bv[t, (p + x) % 16] = c.k[a + x], c.v[a + x]
    assert c.k_cache.equal(before) and c.v_cache.equal(bv)
    # lengths outside the table: nothing of the cache, and all of it (new tokens have no place then)
    c = Cache(rng, [0, 64], [new] * 2, 4, 2, 64, 64, 16, typ)
    c.table = c.table[:, :4]
    want, tol = c.want(0.125)
    before = c.k_cache.clone()
    c.past = [-5, 10 ** 6]
    c.run(max_length=64 + new)
    near(c.o, want, TINY[typ] + U[typ] * np.abs(want) + tol, "o")
    for x in range(min(new, 64)):
        before[c.table[0][x // 16], x % 16] = c.k[x]
    assert c.k_cache.equal(before)
    # an empty cache: new tokens alone
    e = torch.empty((0, 16, 2, 64), device=DEV, dtype=c.k.dtype)
    ws = L.attention_cached_workspace(c.q, e, e, ints(c.table), ints(c.cu))
    L.pc_attention_cached(c.q, c.k, c.v, e, e, ints(c.table), ints([0, 0]), c.o, ints(c.cu), ws=ws)
    _check_forward(c.q, c.k, c.v, c.o, None, c.cu, 0.125, typ)


@pytest.mark.parametrize("typ", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("past,new", [([64, 40], 90), ([100, 64], 1), ([100, 64], 40), ([5000, 200], 200), ([5000, 200], 2)])
@pytest.mark.parametrize("gap", [1, 8])
def test_attention_cached_without_pages(gap, past, new, typ, monkeypatch):
    """A cache that has no pages at all: whatever the lengths and the table say, new tokens attend new tokens alone."""
    import log_space_sum_amd as L
    torch, _ = T()
    monkeypatch.setattr(Cache, "gap", gap)
    c = Cache(np.random.default_rng(18), past, [new] * 2, 4, 2, 64, 64, 16, typ)
    c.table[0][:2] = -1, 2 ** 31 - 1
    e = torch.empty((0, 16, 2, 64), device=DEV, dtype=c.k.dtype)
    ws = L.attention_cached_workspace(c.q, e, e, ints(c.table), ints(c.cu))
    L.pc_attention_cached(c.q, c.k, c.v, e, e, ints(c.table), ints(past), c.o, ints(c.cu), ws=ws)
    _check_forward(c.q, c.k, c.v, c.o, None, c.cu, 0.125, typ)


@pytest.mark.parametrize("typ", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("dk,dv", [(24, 40), (88, 16), (7, 33)])
@pytest.mark.parametrize("value", [math.inf, math.nan])
def test_attention_of_narrow_heads_keeps_what_is_not_finite_in_its_place(value, dk, dv, typ):
    """The same where a head is narrower than the tile that it lies in, whole sequences and their gradients: the first elements of a row
    stand there in the place of those behind it."""
    import log_space_sum_amd as L
    torch, _ = T()
    rng = np.random.default_rng(15)
    cu, at = [0, 150], 70
    for what in range(4):
        q, k, v, do = _qkv(rng, 150, 2, 2, dk, dv, typ)

        def run():
            o, lse = torch.empty_like(do), torch.empty((150, 2), device=DEV)
            L.pc_attention_forward(q, k, v, o, lse, ints(cu))
            grads = [torch.empty_like(t) for t in (q, k, v)]
            L.pc_attention_backward(do, q, k, v, o, lse, *grads, ints(cu), ws=L.attention_workspace(q, k, v, ints(cu), backward=True))
            return [get(t) for t in (o, lse[..., None], *grads)]
        clean = run()
        (q, k, v, do)[what][at, 1, 2] = value
        dirty = run()
        reach = [[(at, at + 1)] * 3 + [(0, at + 1)] * 2, [(at, 150)] * 3 + [(0, 150)] * 2,
                 [(at, 150), (0, 0), (at, 150), (0, 150), (0, 150)], [(0, 0), (0, 0), (at, at + 1), (0, at + 1), (0, at + 1)]][what]
        # An element of o that a tile taken again rounds the other way moves delta_i = do_i . o_i, so dq_i by
        # scale sum_j P_ij k_j of that, at most scale max |k|, and dk_j by scale P_ij q_i, at most scale max |q|.
        known = lambda x: np.where(np.isfinite(x), np.abs(x), 0.0)  # noqa: E731
        with np.errstate(invalid="ignore"):
            moved = (known(get(do)) * known(clean[0] - dirty[0])).sum(-1)
        moved[reach[0][0]:reach[0][1], 1] = 0.0
        more = [0.0, 0.0, dk ** -0.5 * known(get(k)).max() * moved[..., None],
                dk ** -0.5 * known(get(q)).max() * np.broadcast_to(moved.sum(0)[None, :, None], (150, 2, 1)), 0.0]
        for a, b, (lo, hi), extra, name in zip(clean, dirty, reach, more, ("o", "lse", "dq", "dk", "dv")):
            free = np.ones(a.shape[:2], bool)
            free[lo:hi, 1] = False
            rms = np.sqrt((a * a).mean())
            assert (np.abs(a - b) <= 2 * U[typ] * np.abs(a) + 1e-5 * rms + extra)[free].all(), name
        with np.errstate(invalid="ignore"):
            ro, rl = R.softmax_attention(get(q), get(k), get(v), cu, dk ** -0.5)
        assert (np.isfinite(dirty[0][at:]) == np.isfinite(ro[at:])).all() and (np.isfinite(dirty[1][at:, :, 0]) == np.isfinite(rl[at:])).all()


@pytest.mark.parametrize("typ", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("new", [2, 100])
def test_attention_cached_keeps_what_is_not_finite_in_its_place(new, typ):
    """Nobody's rows of the cache hold NaN (also behind the last token of a page), and a new token's value is infinite: rows before
    it, and other streams, do not see it."""
    c = Cache(np.random.default_rng(14), [70, 30], [new] * 2, 4, 2, 64, 64, 16, typ)
    keep_k, keep_v = c.k_cache.clone(), c.v_cache.clone()
    c.k_cache.fill_(math.nan)
    c.v_cache.fill_(math.nan)
    for i, p in enumerate(c.past):
        for j in range(p):
            at = (c.table[i][j // 16], j % 16)
            c.k_cache[at], c.v_cache[at] = keep_k[at], keep_v[at]
    want, tol = c.want(0.125)
    c.run()
    near(c.o, want, TINY[typ] + U[typ] * np.abs(want) + tol, "o")
    c.v[new - 1, 0, 3] = math.inf
    c.run()
    got = get(c.o)
    assert (got[new - 1, :2, 3] == math.inf).all()
    want[new - 1, :2, 3] = got[new - 1, :2, 3] = 0
    assert (np.abs(got - want) <= TINY[typ] + U[typ] * np.abs(want) + tol).all()


@pytest.mark.parametrize("typ", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("past,new,H,K,dk,dv,page", CACHES)
def test_attention_cached_of_aligned_rows(past, new, H, K, dk, dv, page, typ, monkeypatch):
    monkeypatch.setattr(Cache, "gap", 8)
    Cache(np.random.default_rng(page + dk), past, new, H, K, dk, dv, page, typ).check()


@pytest.mark.parametrize("typ", ["bf16", "f16"])
def test_attention_cached_of_aligned_rows_at_the_edges(typ, monkeypatch):
    monkeypatch.setattr(Cache, "gap", 8)
    test_attention_cached_single_tokens_and_orders(typ)
    for new in (1, 40, 200):
        test_attention_cached_in_parts(new, typ)
    for new in (1, 90):
        test_attention_cached_pages_that_are_none(new, typ)
    for new in (2, 100):
        test_attention_cached_keeps_what_is_not_finite_in_its_place(new, typ)
    for total in (128, 257, 512, 513, 769):
        test_attention_cached_of_lengths_around_a_part(total, typ)


@pytest.mark.parametrize("typ", ["f32", "bf16"])
@pytest.mark.parametrize("new,page,index,rest", [(new, *at) for new in (1, 40) for at in (
    (1, 999, 1), (3, 333, 2), (7, 1000, 7), (100, 60, 99), (1000, 77, 5), (65536, 300, 9), (65537, 300, 9), (1000003, 20, 6))] + [
    (1, 65521, 32700, 11)])
def test_attention_cached_finds_pages_of_any_size(new, page, index, rest, typ):
    """All pages are none but the one that the last `rest` cached positions lie in, from its first row on, and the next: a position
    that were divided by the page's size to another page, or row, would miss them."""
    import log_space_sum_amd as L
    torch, types = T()
    rng = np.random.default_rng(page % 1000 + new)
    H, d, past, behind = 4, 16, page * index + rest, -(-new // page) + 1
    q, k, v, o = _qkv(rng, new, H, 1, d, d, typ)
    kc, vc = (torch.full((1 + behind, page, 1, d), 7.0, device=DEV, dtype=types[typ]) for _ in range(2))
    ck, cv = (put(rng.normal(size=(rest, 1, d)), typ) for _ in range(2))
    kc[0, :rest], vc[0, :rest] = ck, cv
    table = np.full((1, index + 1 + behind), -1)
    table[0, index:] = np.arange(1 + behind)
    cu = ints([0, new])
    ws = L.attention_cached_workspace(q, kc, vc, ints(table), cu)
    L.pc_attention_cached(q, k, v, kc, vc, ints(table), ints([past]), o, cu, ws=ws)
    kk, vv = np.concatenate([get(ck), get(k)]), np.concatenate([get(cv), get(v)])
    want = R.attend(get(q), kk, vv, d ** -0.5, rest)[0]
    near(o, want, TINY[typ] + U[typ] * np.abs(want) + _errors(get(q), kk, vv, d ** -0.5, rest)[0], "o")
    for cache, first, then in ((kc, ck, k), (vc, cv, v)):
        rows = cache.view(-1, 1, d)
        assert rows[:rest].equal(first) and rows[rest:rest + new].equal(then) and (rows[rest + new:] == 7).all()


@pytest.mark.parametrize("n", [3, 130])
def test_attention_cached_chunks_in_far_pages(n):
    """The same for a chunk: few rows, and many."""
    import log_space_sum_amd as L
    torch, _ = T()
    pages, page, K, d = 70000, 64, 4, 128
    if torch.cuda.mem_get_info()[0] < pages * page * K * d * 2 * 2.5:
        pytest.skip("memory")
    kc, vc = (torch.zeros((pages, page, K, d), device=DEV, dtype=torch.bfloat16) for _ in range(2))
    rng = np.random.default_rng(17)
    q, k, v, o = _qkv(rng, n, 4, K, d, d, "bf16")
    pk, pv = put(rng.normal(size=(2, page, K, d)), "bf16"), put(rng.normal(size=(2, page, K, d)), "bf16")
    kc[pages - 2:], vc[pages - 2:] = pk, pv
    table = ints([[pages - 2, pages - 1, 1, pages - 3, 2]])
    cu = ints([0, n])
    ws = L.attention_cached_workspace(q, kc, vc, table, cu)
    L.pc_attention_cached(q, k, v, kc, vc, table, ints([2 * page]), o, cu, ws=ws)
    kk, vv = (np.concatenate([get(p).reshape(2 * page, K, d), get(x)]) for p, x in ((pk, k), (pv, v)))
    want = R.attend(get(q), kk, vv, d ** -0.5, 2 * page)[0]
    near(o, want, U["bf16"] * np.abs(want) + _errors(get(q), kk, vv, d ** -0.5, 2 * page)[0], "o")
    m = min(n, page)
    assert kc[1, :m].equal(k[:m]) and vc[1, :m].equal(v[:m]) and (n <= page or kc[pages - 3, :page].equal(k[page:2 * page]))


def test_attention_cached_far_pages():
    """Pages whose offsets in the cache pass 2^32 bytes and 2^31 elements."""
    import log_space_sum_amd as L
    torch, _ = T()
    free = torch.cuda.mem_get_info()[0]
    pages, page, K, d = 70000, 64, 4, 128         # 2.3 x 10^9 elements
    if free < pages * page * K * d * 2 * 2.5:
        pytest.skip("memory")
    kc, vc = (torch.zeros((pages, page, K, d), device=DEV, dtype=torch.bfloat16) for _ in range(2))
    rng = np.random.default_rng(15)
    q, k, v, o = _qkv(rng, 1, 4, K, d, d, "bf16")
    pk, pv = put(rng.normal(size=(page, K, d)), "bf16"), put(rng.normal(size=(page, K, d)), "bf16")
    kc[pages - 1], vc[pages - 1] = pk, pv
    table = ints([[pages - 1, pages - 2]])
    ws = L.attention_cached_workspace(q, kc, vc, table)
    L.pc_attention_cached(q, k, v, kc, vc, table, ints([page]), o, ws=ws)
    kk, vv = np.concatenate([get(pk), get(k)]), np.concatenate([get(pv), get(v)])
    want = R.attend(get(q), kk, vv, d ** -0.5, page)[0]
    near(o, want, U["bf16"] * np.abs(want) + _errors(get(q), kk, vv, d ** -0.5, page)[0], "o")
    assert kc[pages - 2, 0].equal(k[0]) and vc[pages - 2, 0].equal(v[0]) and not kc[0].any() and not kc[pages - 2, 1:].any()


@pytest.mark.parametrize("d", [128, 124])
def test_attention_of_tensors_beyond_32_bits(d):
    """Rows whose offsets pass 2^32 bytes and 2^31 elements, loaded directly and through registers: norm and rotation in place, whole
    sequences, gradients and new tokens over a cache; the last sequences against the definition."""
    import log_space_sum_amd as L
    torch, _ = T()
    H, K, each, last = 64, 8, 250, 40
    lens = [each] * 1120 + [last, 1, last]
    cu = _cu(lens)
    n = cu[-1]
    if torch.cuda.mem_get_info()[0] < 7 * n * H * d * 2:
        pytest.skip("memory")
    assert n * H * d > 1 << 31
    g = torch.Generator(device=DEV)
    g.manual_seed(26)
    q, do = (torch.randn((n, H, d), generator=g, device=DEV, dtype=torch.bfloat16) for _ in range(2))
    k, v = (torch.randn((n, K, d), generator=g, device=DEV, dtype=torch.bfloat16) for _ in range(2))
    end = slice(cu[-4], n)
    near_end = [c - cu[-4] for c in cu[-4:]]
    pos, freq = torch.arange(n, dtype=torch.int32, device=DEV), L.rotary_frequencies(32, device=DEV)
    before = get(q[end])
    L.pc_rotary_forward(q, k, q, k, pos, freq, norm=True)
    want = R.rotary(before, np.arange(end.start, n), get(freq), norm=True)
    size = np.abs(R.rotary(before, np.zeros(n - end.start), get(freq), norm=True))
    near(q[end], want, U["bf16"] * np.abs(want) + (d / 4 + 16) * E * (size + _partner(size, 32, False)), "rotated")
    o, lse, dq, dk, dv = torch.empty_like(do), torch.empty((n, H), device=DEV), torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    L.pc_attention_forward(q, k, v, o, lse, ints(cu), each, ws=L.attention_workspace(q, k, v, ints(cu), each))
    L.pc_attention_backward(do, q, k, v, o, lse, dq, dk, dv, ints(cu), each, ws=L.attention_workspace(q, k, v, ints(cu), each, backward=True))
    _check_forward(q[end], k[end], v[end], o[end], lse[end], near_end, d ** -0.5, "bf16")
    _check_backward(*(t[end] for t in (do, q, k, v, o, lse)), [t[end] for t in (dq, dk, dv)], near_end, d ** -0.5, "bf16")
    # new tokens of every sequence with nothing cached: outputs, and their rows in the cache
    table = ints(np.arange(len(lens)))[:, None]
    kc, vc = (torch.zeros((len(lens), each, K, d), device=DEV, dtype=torch.bfloat16) for _ in range(2))
    o.fill_(0)
    ws = L.attention_cached_workspace(q, kc, vc, table, ints(cu), each, each)
    L.pc_attention_cached(q, k, v, kc, vc, table, ints([0] * len(lens)), o, ints(cu), each, each, ws=ws)
    _check_forward(q[end], k[end], v[end], o[end], None, near_end, d ** -0.5, "bf16")
    assert kc[-1, :last].equal(k[-last:]) and vc[-1, :last].equal(v[-last:]) and not kc[-1, last:].any()


@pytest.mark.parametrize("typ", ["f32", "bf16"])
def test_attention_of_the_most_heads(typ):
    """65535 heads that share one: rows of a token on many tiles."""
    import log_space_sum_amd as L
    torch, _ = T()
    rng = np.random.default_rng(27)
    n, H, d = 3, 65535, 8
    q, k, v, do = _qkv(rng, n, H, 1, d, d, typ)
    o, lse = torch.empty_like(do), torch.empty((n, H), device=DEV)
    L.pc_attention_forward(q, k, v, o, lse, ws=L.attention_workspace(q, k, v))
    _check_forward(q, k, v, o, lse, [0, n], d ** -0.5, typ)
    grads = [torch.empty_like(t) for t in (q, k, v)]
    L.pc_attention_backward(do, q, k, v, o, lse, *grads, ws=L.attention_workspace(q, k, v, backward=True))
    _check_backward(do, q, k, v, o, lse, grads, [0, n], d ** -0.5, typ)
    c = Cache(rng, [20], [n], H, 1, d, d, 16, typ)
    c.check()


# ---------------------------------------------------------------------------
# together
# ---------------------------------------------------------------------------

def _layer(seed, typ, lens, H=4, K=2, d=64):
    """Heads of a layer, their norm's weights, positions and frequencies."""
    import log_space_sum_amd as L
    rng = np.random.default_rng(seed)
    cu = _cu(lens)
    q, k, v, do = _qkv(rng, cu[-1], H, K, d, d, typ)
    pos = ints(np.concatenate([np.arange(n) for n in lens]))
    return q, k, v, do, cu, pos, L.rotary_frequencies(d // 2, device=DEV), put(rng.normal(size=d) * 0.2 + 1), put(rng.normal(size=d) * 0.2 + 1)


@pytest.mark.parametrize("typ", ["f32", "bf16", "f16"])
def test_a_prompt_in_chunks_and_single_tokens_is_the_prompt(typ):
    """Rotated heads attended as whole prompts, and the same prompts in chunks and single tokens over a cache: the same outputs within
    the tolerance of both, with every row of a call for chunks of its own length."""
    import log_space_sum_amd as L
    torch, _ = T()
    lens = [75, 40, 130]
    q, k, v, _, cu, pos, freq, wq, wk = _layer(21, typ, lens)
    L.pc_rotary_forward(q, k, q, k, pos, freq, norm=True, q_weight=wq, k_weight=wk)
    whole = torch.empty_like(q)
    L.pc_attention_forward(q, k, v, whole, None, ints(cu), max(lens))
    want, _ = _check_forward(q, k, v, whole, None, cu, 0.125, typ)
    kc, vc = (torch.full((60, 16, 2, 64), math.nan, device=DEV, dtype=q.dtype) for _ in range(2))
    table = ints(np.random.default_rng(22).permutation(60)[:27].reshape(3, 9))
    done, got = [0, 0, 0], torch.empty_like(q)
    steps = [[60, 1, 33], [1, 20, 0], [1, 1, 1], [13, 18, 96]]
    assert [sum(s[i] for s in steps) for i in range(3)] == lens
    for step in steps:
        rows = torch.cat([torch.arange(cu[i] + done[i], cu[i] + done[i] + n) for i, n in enumerate(step)]).to(DEV)
        o = torch.empty((len(rows), 4, 64), device=DEV, dtype=q.dtype)
        at = ints(_cu(step))
        ws = L.attention_cached_workspace(q[rows], kc, vc, table, at)
        L.pc_attention_cached(q[rows], k[rows], v[rows], kc, vc, table, ints(done), o, at, ws=ws)
        got[rows] = o
        done = [a + b for a, b in zip(done, step)]
    _check_forward(q, k, v, got, None, cu, 0.125, typ)


def test_a_layer_learns_from_a_conditional_circuit():
    """Heads normalised, rotated and attended give the factor A of a LowRank HMM; dLL/dA goes back through the operators to the
    inputs, and every gradient agrees with slopes of the circuit's log-likelihood along it: float32 operators and a
    float32-level circuit (batch below 16), so a central difference of a step h is off by about 2^-22 |LL| / h and h^2."""
    import log_space_sum_amd as L
    from workloads import make_config
    torch, _ = T()
    cfg = make_config("lowrank", H=32, T=3, V=5, rank=4, B=8)
    circ, B = cfg["circuit"], cfg["B"]
    h = L.pc_compile_layout(circ, device=0)
    L.pc_set_precision(h, "fp32")
    params, tokens = torch.tensor(cfg["params"], device=DEV), torch.tensor(cfg["tokens"], device=DEV)
    vals, flows = (torch.empty((circ.num_nodes, B), device=DEV) for _ in range(2))
    pflows, ll, ws = torch.zeros(circ.num_params, device=DEV), torch.empty(B, device=DEV), L.workspace(h, B, DEV)
    fixed = [(torch.tensor(a, device=DEV), torch.tensor(b, device=DEV)) for a, b in cfg["lowrank"]]
    M, r = fixed[0][0].shape[1:]
    # a sample is a sequence of M positions (the states), 2 heads of width 2 give its rows of the rank 4 factor
    n, H, d = B * M, 2, 2
    lens = [M] * B
    cu, pos = ints(_cu(lens)), ints(np.tile(np.arange(M), B))
    rng = np.random.default_rng(23)
    q, k, v = (put(rng.normal(size=(n, H, d))) for _ in range(3))
    wq, wk = put(rng.normal(size=d) * 0.2 + 1), put(rng.normal(size=d) * 0.2 + 1)
    freq = L.rotary_frequencies(d, device=DEV)
    aws, rws = L.attention_workspace(q, k, v, cu, backward=True), L.rotary_workspace(q, k)

    def forward(q, k, v, wq, wk):
        qr, kr, o, lse = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v), torch.empty((n, H), device=DEV)
        L.pc_rotary_forward(q, k, qr, kr, pos, freq, norm=True, q_weight=wq, k_weight=wk)
        L.pc_attention_forward(qr, kr, v, o, lse, cu, M)
        lr = [(o.view(B, M, r), fixed[0][1])] + fixed[1:]
        L.pc_forward(h, B, tokens, params, vals, ll, lr, ws)
        return qr, kr, o, lse, lr

    qr, kr, o, lse, lr = forward(q, k, v, wq, wk)
    grads = [(torch.empty_like(a), torch.empty_like(b)) for a, b in lr]
    L.pc_backward(h, B, tokens, params, vals, flows, pflows, 0, lr, grads, ws)
    do = grads[0][0].view(n, H, d)
    dq, dk, dv, dwq, dwk = (torch.empty_like(t) for t in (q, k, v, wq, wk))
    L.pc_attention_backward(do, qr, kr, v, o, lse, dq, dk, dv, cu, M, ws=aws)
    L.pc_rotary_backward(dq, dk, dq, dk, pos, freq, norm=True, q=q, k=k, q_weight=wq, k_weight=wk, dq_weight=dwq, dk_weight=dwk, ws=rws)
    # the operators' part of the chain exactly, from the circuit's dLL/dA
    Q, K, V, WQ, WK, DO, F = (get(t) for t in (q, k, v, wq, wk, do, freq))
    P = np.tile(np.arange(M), B)
    rq, rk = R.rotary(Q, P, F, norm=True, w=WQ), R.rotary(K, P, F, norm=True, w=WK)
    ro, rl = R.softmax_attention(rq, rk, V, _cu(lens), d ** -0.5)
    gq, gk, gv = R.softmax_attention_grad(DO, rq, rk, V, ro, rl, _cu(lens), d ** -0.5)
    xq, xwq = R.rotary_grad(gq, Q, P, F, norm=True, w=WQ)
    xk, xwk = R.rotary_grad(gk, K, P, F, norm=True, w=WK)
    # (sums over M rows of terms that cancel; float32 throughout: (M + 64) E of their size, here at most 100 times the results')
    for got, want, name in ((dq, xq, "dq"), (dk, xk, "dk"), (dv, gv, "dv"), (dwq, xwq, "dwq"), (dwk, xwk, "dwk")):
        assert np.linalg.norm(get(got) - want) <= 100 * (M + 64) * E * np.linalg.norm(want), name
    # and slopes of the log-likelihood
    inputs, g = [q, k, v, wq, wk], [dq, dk, dv, dwq, dwk]
    for i in range(5):
        step = 2.0 ** -5 / float(g[i].norm())

        def at(sign):
            args = list(inputs)
            args[i] = args[i] + sign * step * g[i]
            forward(*args)
            return float(ll.double().sum())
        slope, want = (at(1) - at(-1)) / (2 * step), float(g[i].double().square().sum())
        noise = 2.0 ** -20 * abs(float(ll.double().sum())) / step
        assert abs(slope - want) <= 0.02 * want + noise, (i, slope, want)


def test_two_calls_at_once_and_captured():
    """Calls on two streams with workspaces of their own, and all calls of a layer captured into a graph that is replayed between
    eager work: the same bits as alone."""
    import log_space_sum_amd as L
    torch, _ = T()
    q, k, v, do, cu, pos, freq, wq, wk = _layer(31, "bf16", [300, 0, 77, 500])
    n = cu[-1]
    dcu = ints(cu)
    kc, vc = (put(np.random.default_rng(32).normal(size=(80, 16, 2, 64)), "bf16") for _ in range(2))
    table, past = ints(np.arange(80).reshape(4, 20)), ints([310, 5, 0, 200])
    one = [t[:4].contiguous() for t in (q, k, v)]

    class Run:
        def __init__(self):
            self.qr, self.kr, self.o, self.lse = torch.empty_like(q), torch.empty_like(k), torch.empty_like(do), torch.empty((n, 4), device=DEV)
            self.g = [torch.empty_like(t) for t in (q, k, v, wq, wk)]
            self.aws, self.rws = L.attention_workspace(q, k, v, dcu, backward=True), L.rotary_workspace(q, k)
            self.kc, self.vc, self.co = kc.clone(), vc.clone(), torch.empty_like(one[0])
            self.cws = L.attention_cached_workspace(one[0], kc, vc, table, max_length=100000)

        def __call__(self):
            dq, dk, dv, dwq, dwk = self.g
            L.pc_rotary_forward(q, k, self.qr, self.kr, pos, freq, norm=True, q_weight=wq, k_weight=wk)
            L.pc_attention_forward(self.qr, self.kr, v, self.o, self.lse, dcu)
            L.pc_attention_backward(do, self.qr, self.kr, v, self.o, self.lse, dq, dk, dv, dcu, ws=self.aws)
            L.pc_rotary_backward(dq, dk, dq, dk, pos, freq, norm=True, q=q, k=k, q_weight=wq, k_weight=wk, dq_weight=dwq, dk_weight=dwk, ws=self.rws)
            L.pc_attention_cached(*one, self.kc, self.vc, table, past, self.co, max_length=100000, ws=self.cws)

        def results(self):
            return [self.o, self.lse, *self.g, self.co, self.kc, self.vc]

        def clear(self):
            for t in [self.o, self.lse, *self.g, self.co]:
                t.zero_()
    first = Run()
    first()
    torch.cuda.synchronize()
    want = [t.clone() for t in first.results()]
    runs, streams = [Run(), Run()], [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(3):
        for r, s in zip(runs, streams):
            with torch.cuda.stream(s):
                r()
    torch.cuda.synchronize()
    for r in runs:
        assert all(torch.equal(a, b) for a, b in zip(want, r.results()))
    graph, captured = torch.cuda.CUDAGraph(), Run()
    with torch.cuda.graph(graph):
        captured()
    for _ in range(3):
        captured.clear()
        first()                       # eager work of the program's own between replays
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, captured.results()))
