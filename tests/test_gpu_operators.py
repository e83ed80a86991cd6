"""The operators in front of a conditional circuit on the GPU against their float64 definitions.

Tolerances.  u is half a step of the output's type (2^-24, 2^-8, 2^-11 of the value for float32, bfloat16, float16).
A sum of n products taken in float32 in any order differs from the exact one by at most (n + 2) 2^-24 times the sum
of the products' magnitudes; the magnitudes are the definition run on absolute values.  Below a
type's normal numbers half a step is absolute: 2^-25 for float16, and float32 results below 2^-126 may be 0.  bfloat16
linear attention splits the products inside a chunk and the state into two planes each, which leaves 2^-17 of the magnitudes at each
of the two places."""
import numpy as np
import pytest

from oracle import ops_oracle as R

pytestmark = pytest.mark.gpu
U = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}
E32 = 2.0 ** -24
TINY = {"f32": 2.0 ** -126, "bf16": 2.0 ** -126, "f16": 2.0 ** -25}
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


def get(t):
    return t.detach().double().cpu().numpy()


def near(got, want, tol, what):
    got = get(got)
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), (what, int(bad.sum()), float(np.abs(got - want)[bad].max()), np.argwhere(bad)[:3].tolist())


# ---------------------------------------------------------------------------
# layer norm
# ---------------------------------------------------------------------------

def _norm_tol(x, w, b, mean, rstd, y, u):
    # mean, variance and the centred values: (cols + 2) roundings of sums, relative to the row's spread and mean
    n = x.shape[1]
    spread = np.abs(x).max(1, keepdims=True) * rstd[:, None]
    return (2.0 ** -25 if u == U["f16"] else 0) + u * np.abs(y) + (n / 8 + 16) * E32 * (spread * (1 + np.abs(y)) * (1 if w is None else np.abs(w).max()) +
                                                (0 if b is None else np.abs(b).max()))


SHAPES = [(1, 1), (3, 7), (65, 129), (7, 1001), (37, 512), (5, 4096), (2, 16384), (3, 5000), (300, 40)]


@pytest.mark.parametrize("typ", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_layer_norm(rows, cols, typ):
    import log_space_sum_amd as L
    torch, types = T()
    rng = np.random.default_rng(rows * 7 + cols)
    # rows at a stride and an offset that are not multiples of a vector
    whole = put(rng.normal(size=(rows, cols + 3)) * 2 + 0.5, typ)
    x = whole[:, 1:1 + cols]
    w, b = put(rng.normal(size=cols) + 1), put(rng.normal(size=cols))
    out = torch.full((rows, cols + 5), 7.0, device=DEV, dtype=types[typ])
    y, mean, rstd = out[:, 3:3 + cols], torch.empty(rows, device=DEV), torch.empty(rows, device=DEV)
    L.pc_layer_norm_forward(x, w, b, y, mean, rstd)
    xs, ws, bs = get(x), get(w), get(b)
    ry, rm, rr = R.layer_norm(xs, ws, bs)
    near(mean, rm, (cols / 8 + 8) * E32 * np.abs(xs).max(1), "mean")
    near(rstd, rr, (cols / 8 + 16) * E32 * rr * (1 + (np.abs(xs).max(1) * rr) ** 2 / max(1, cols / 64)), "rstd")
    near(y, ry, _norm_tol(xs, ws, bs, rm, rr, ry, U[typ]), "y")
    assert (out[:, :3] == 7).all() and (out[:, 3 + cols:] == 7).all()
    # without weight and bias, in place
    y0, _, _ = R.layer_norm(xs)
    L.pc_layer_norm_forward(x, None, None, x)
    near(x, y0, _norm_tol(xs, None, None, rm, rr, y0, U[typ]), "in place")


@pytest.mark.parametrize("typ", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("rows,cols", SHAPES + [(5000, 65)])
def test_layer_norm_backward(rows, cols, typ):
    import log_space_sum_amd as L
    torch, types = T()
    rng = np.random.default_rng(rows + cols)
    x, dy = put(rng.normal(size=(rows, cols + 1)), typ)[:, 1:], put(rng.normal(size=(rows, cols + 2)), typ)[:, :cols]
    w = put(rng.normal(size=cols) + 1)
    _, m, r = R.layer_norm(get(x))
    mean, rstd = put(m), put(r)
    rx, rw, rb = R.layer_norm_grad(get(dy), get(x), get(mean), get(rstd), get(w))
    n = np.abs((get(x) - get(mean)[:, None]) * get(rstd)[:, None])
    g = np.abs(get(dy) * get(w))
    dx, dw, db = torch.empty((rows, cols), device=DEV, dtype=types[typ]), torch.empty(cols, device=DEV), torch.empty(cols, device=DEV)
    ws = L.layer_norm_workspace(rows, cols, DEV)
    L.pc_layer_norm_backward(dy, x, w, mean, rstd, dx, dw, db, ws)
    size = get(rstd)[:, None] * (g + g.mean(1, keepdims=True) + n * (g * n).mean(1, keepdims=True))
    near(dx, rx, TINY[typ] + U[typ] * np.abs(rx) + (cols / 8 + 16) * E32 * size, "dx")
    near(dw, rw, (rows + 8) * E32 * (np.abs(get(dy)) * n).sum(0), "dweight")
    near(db, rb, (rows + 8) * E32 * np.abs(get(dy)).sum(0), "dbias")
    first = [t.clone() for t in (dx, dw, db)]
    L.pc_layer_norm_backward(dy, x, w, mean, rstd, dx, dw, db, ws)
    assert all(torch.equal(a, b) for a, b in zip(first, (dx, dw, db)))
    # one of the two gradients alone, and neither
    L.pc_layer_norm_backward(dy, x, w, mean, rstd, dx, None, db.zero_(), ws)
    assert torch.equal(db, first[2])
    L.pc_layer_norm_backward(dy, x, w, mean, rstd, dx.zero_())
    assert torch.equal(dx, first[0])


@pytest.mark.parametrize("typ", ["f32", "bf16"])
@pytest.mark.parametrize("rows,cols", [(37, 512), (3, 5000), (5000, 65), (70, 9)])
def test_layer_norm_backward_in_place(rows, cols, typ):
    """dx over dy and over x gives the bits of a dx of its own."""
    import log_space_sum_amd as L
    torch, types = T()
    rng = np.random.default_rng(rows)
    x, dy = put(rng.normal(size=(rows, cols)), typ), put(rng.normal(size=(rows, cols)), typ)
    w, mean, rstd = put(rng.normal(size=cols)), put(rng.normal(size=rows) * 0.1), put(np.exp(rng.normal(size=rows) * 0.1))
    ws, out = L.layer_norm_workspace(rows, cols, DEV), []
    for place in (None, "dy", "x"):
        a, b = dy.clone(), x.clone()
        dx = {None: torch.empty_like(x), "dy": a, "x": b}[place]
        dw, db = torch.empty(cols, device=DEV), torch.empty(cols, device=DEV)
        L.pc_layer_norm_backward(a, b, w, mean, rstd, dx, dw, db, ws)
        out.append((dx, dw, db))
    for other in out[1:]:
        assert all(torch.equal(p, q) for p, q in zip(out[0], other))


def test_layer_norm_edges():
    import log_space_sum_amd as L
    torch, _ = T()
    # no rows: the gradients of the parameters are 0
    e = torch.empty((0, 12), device=DEV)
    dw, db = torch.full((12,), 5.0, device=DEV), torch.full((12,), 5.0, device=DEV)
    z = torch.empty(0, device=DEV)
    L.pc_layer_norm_forward(e, None, None, e, z, z)
    L.pc_layer_norm_backward(e, e, None, z, z, e, dw, db, L.layer_norm_workspace(0, 12, DEV))
    assert not dw.any() and not db.any()
    # a constant row, a far offset, a row with NaN and one with infinities beside finite ones
    x = torch.randn(5, 300, device=DEV)
    x[1] = 3.0
    x[2] += 4096.0
    x[3, 17] = float("nan")
    x[4, 5] = float("inf")
    y = torch.empty_like(x)
    L.pc_layer_norm_forward(x, None, None, y)
    ry, _, rr = R.layer_norm(get(x)[:3])
    assert torch.isnan(y[3]).all() and not torch.isfinite(y[4]).any()
    assert (y[1] == 0).all()
    near(y[:3], ry, 64 * E32 * (1 + np.abs(get(x)[:3]).max(1, keepdims=True) * rr[:, None]), "rows")


# ---------------------------------------------------------------------------
# linear attention
# ---------------------------------------------------------------------------

def _att(rng, lens, H, K, dk, dv, typ, tail=0):
    n = sum(lens) + tail
    q, k, v, do = (rng.normal(size=s) for s in ((n, H, dk), (n, K, dk), (n, K, dv), (n, H, dv)))
    q, k, v, do = (put(a, typ) for a in (q, k, v, do))
    cu = np.cumsum([0] + list(lens))
    torch, _ = T()
    return q, k, v, do, cu, torch.tensor(cu, dtype=torch.int32, device=DEV)


def _bound(typ, n, size, ref):
    return TINY[typ] + U[typ] * np.abs(ref) + ((2.0 ** -16 if typ == "bf16" else 0) + n * E32) * size


DECAYS = np.array([-0.02, 0.0, -np.inf, -1.0, -30.0, -0.5, -3e-3, -200.0], dtype=np.float32)
CASES = [
    ([1], 1, 1, 1, 1), ([0, 1, 0], 2, 1, 4, 6), ([63, 64, 65, 31, 32, 33], 2, 2, 16, 16), ([130, 0, 7], 4, 2, 33, 65),
    ([200, 129], 3, 1, 64, 128), ([600], 2, 2, 128, 64), ([1100, 3, 700], 2, 1, 40, 20), ([0, 0], 2, 2, 8, 8),
    ([300], 8, 4, 128, 128),
]


@pytest.mark.parametrize("typ", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("lens,H,K,dk,dv", CASES)
def test_linear_attention(lens, H, K, dk, dv, typ):
    import log_space_sum_amd as L
    torch, types = T()
    rng = np.random.default_rng(sum(lens) + H + dk)
    q, k, v, do, cu, dcu = _att(rng, lens, H, K, dk, dv, typ, tail=5)
    n, ns = q.shape[0], len(lens)
    g = put(DECAYS[:H])
    s0, ds = put(rng.normal(size=(ns, H, dk, dv))), put(rng.normal(size=(ns, H, dk, dv)))
    scale = 0.3
    o, s1 = torch.full((n, H, dv), 9.0, device=DEV, dtype=types[typ]), torch.empty_like(s0)
    top = max(lens)
    L.pc_linear_attention_forward(q, k, v, g, o, dcu, top, s0, s1, scale, L.linear_attention_workspace(q, k, v, dcu, top))
    A = [get(t) for t in (q, k, v, g, s0, do, ds)]
    ro, rs = R.linear_attention(*A[:4], cu, scale, A[4])
    mo, ms = R.linear_attention(np.abs(A[0]), np.abs(A[1]), np.abs(A[2]), A[3], cu, scale, np.abs(A[4]))
    live, terms = cu[-1], dk + top + 40
    near(o[:live], ro[:live], _bound(typ, terms, mo, ro)[:live], "o")
    near(s1, rs, TINY['f32'] + E32 * np.abs(rs) + (top + 40) * E32 * ms, "state")
    assert (o[live:] == 9).all()
    # without states
    L.pc_linear_attention_forward(q, k, v, g, o, dcu, top, None, None, scale, L.linear_attention_workspace(q, k, v, dcu, top))
    zo, _ = R.linear_attention(*A[:4], cu, scale)
    near(o[:live], zo[:live], _bound(typ, terms, mo, zo)[:live], "o without states")
    # in place, and with a bound of the lengths that is too small
    s2, o2 = s0.clone(), torch.empty_like(o)
    L.pc_linear_attention_forward(q, k, v, g, o2, dcu, 1, s2, s2, scale, L.linear_attention_workspace(q, k, v, dcu, 1))
    near(s2, rs, TINY['f32'] + E32 * np.abs(rs) + (top + 40) * E32 * ms, "state in place")
    near(o2[:live], ro[:live], _bound(typ, terms, mo, ro)[:live], "o, one segment")

    dq, dk_, dv_ = (torch.full_like(t, 9.0) for t in (q, k, v))
    d0 = torch.empty_like(s0)
    ws = L.linear_attention_workspace(q, k, v, dcu, top, backward=True)
    L.pc_linear_attention_backward(do, q, k, v, g, dq, dk_, dv_, dcu, top, s0, ds, d0, scale, ws)
    want = R.linear_attention_grad(A[5], *A[:4], cu, scale, A[4], A[6])
    size = R.linear_attention_grad(np.abs(A[5]), *[np.abs(a) for a in A[:3]], A[3], cu, scale, np.abs(A[4]), np.abs(A[6]))
    terms = max(dk, dv) + top + H + 40
    for got, ref, mag, name in zip((dq, dk_, dv_), want, size, ("dq", "dk", "dv")):
        near(got[:live], ref[:live], _bound(typ, terms, mag, ref)[:live], name)
        assert (got[live:] == 9).all(), name
    near(d0, want[3], TINY['f32'] + E32 * np.abs(want[3]) + (top + 40) * E32 * size[3], "dstate")
    # no states, the gradient of the state in place
    dz = ds.clone()
    L.pc_linear_attention_backward(do, q, k, v, g, dq, dk_, dv_, dcu, top, None, dz, dz, scale, ws)
    want = R.linear_attention_grad(A[5], *A[:4], cu, scale, None, A[6])
    for got, ref, mag, name in zip((dq, dk_, dv_), want, size, ("dq", "dk", "dv")):
        near(got[:live], ref[:live], _bound(typ, terms, mag, ref)[:live], name + " without state_in")
    assert torch.equal(dz, d0)


@pytest.mark.parametrize("typ", ["bf16", "f16"])
@pytest.mark.parametrize("lens,H,K,dk,dv", [([700, 300], 4, 4, 64, 64), ([400, 513], 2, 1, 128, 128), ([450], 3, 3, 96, 40)])
def test_linear_attention_rounds_a_float32_exact_result(lens, H, K, dk, dv, typ):
    """Outputs and gradients before their rounding are off by the roundings of float32 sums of a chunk's and the state's
    terms, sqrt(terms) 2^-25 of the result (roundings of partial sums that average out).  An element whose value lies d
    from the definition's rounds differently in a share d / step of the cases, then by a step, at most 2 u of the value:
    the squares of the differences from the rounded definition sum to 2 u sqrt(terms) 2^-25 of the result's."""
    import log_space_sum_amd as L
    torch, types = T()
    rng = np.random.default_rng(dk + dv)
    q, k, v, do, cu, dcu = _att(rng, lens, H, K, dk, dv, typ)
    g = put(np.array([-0.02, 0.0, -0.5, -3e-3])[:H])
    s0, ds = (put(rng.normal(size=(len(lens), H, dk, dv))) for _ in range(2))
    o, dq, dk_, dv_ = torch.empty_like(do), *(torch.empty_like(t) for t in (q, k, v))
    L.pc_linear_attention_forward(q, k, v, g, o, dcu, max(lens), s0, ws=L.linear_attention_workspace(q, k, v, dcu, max(lens)))
    L.pc_linear_attention_backward(do, q, k, v, g, dq, dk_, dv_, dcu, max(lens), s0, ds,
                                   ws=L.linear_attention_workspace(q, k, v, dcu, max(lens), backward=True))
    A = [get(t) for t in (q, k, v, g)]
    ref = (R.linear_attention(*A, cu, dk ** -0.5, get(s0))[0],
           *R.linear_attention_grad(get(do), *A, cu, dk ** -0.5, get(s0), get(ds))[:3])
    for got, want, name in zip((o, dq, dk_, dv_), ref, ("o", "dq", "dk", "dv")):
        off = np.linalg.norm(get(got) - get(put(want, typ)))
        assert off <= np.sqrt(2 * U[typ] * np.sqrt(max(dk, dv) + 64) / 2 * E32) * np.linalg.norm(want), name


@pytest.mark.parametrize("typ", ["f32", "bf16"])
def test_linear_attention_strides(typ):
    """q, k, v as parts of one packed tensor, outputs head by head, one sequence without cu_seqlens."""
    import log_space_sum_amd as L
    torch, types = T()
    rng = np.random.default_rng(3)
    n, H, dk, dv = 150, 3, 20, 36
    packed = put(rng.normal(size=(n, H, 2 * dk + dv + 1)), typ)
    q, k, v = packed[..., :dk], packed[..., dk:2 * dk], packed[..., 2 * dk:2 * dk + dv]
    g = put(DECAYS[:H])
    o = torch.empty((H, n, dv), device=DEV, dtype=types[typ]).transpose(0, 1)
    L.pc_linear_attention_forward(q, k, v, g, o, scale=0.2, ws=L.linear_attention_workspace(q, k, v))
    A = [get(t) for t in (q, k, v, g)]
    ro, _ = R.linear_attention(*A, [0, n], 0.2)
    mo, _ = R.linear_attention(*[np.abs(a) for a in A[:3]], A[3], [0, n], 0.2)
    near(o, ro, _bound(typ, dk + n + 40, mo, ro), "o")
    do = put(rng.normal(size=(H, n, dv)), typ).transpose(0, 1)
    grads = torch.full_like(packed, 4.0)
    L.pc_linear_attention_backward(do, q, k, v, g, grads[..., :dk], grads[..., dk:2 * dk], grads[..., 2 * dk:2 * dk + dv], scale=0.2,
                                   ws=L.linear_attention_workspace(q, k, v, backward=True))
    want = R.linear_attention_grad(get(do), *A, [0, n], 0.2)
    size = R.linear_attention_grad(np.abs(get(do)), *[np.abs(a) for a in A[:3]], A[3], [0, n], 0.2)
    for got, ref, mag, name in zip((grads[..., :dk], grads[..., dk:2 * dk], grads[..., 2 * dk:2 * dk + dv]), want, size, ("dq", "dk", "dv")):
        near(got, ref, _bound(typ, dv + n + 40, mag, ref), name)
    assert (grads[..., -1] == 4).all()


@pytest.mark.parametrize("typ", ["f32", "bf16", "f16"])
def test_linear_attention_values_that_are_not_finite(typ):
    """They reach their own and later tokens of their sequence, and nothing else."""
    import log_space_sum_amd as L
    torch, types = T()
    rng = np.random.default_rng(4)
    lens = [100, 90, 40]
    q, k, v, do, cu, dcu = _att(rng, lens, 2, 2, 32, 48, typ)
    g = put(np.array([-0.1, -0.01]))
    clean = torch.empty((230, 2, 48), device=DEV, dtype=types[typ])
    ws = L.linear_attention_workspace(q, k, v, dcu)
    L.pc_linear_attention_forward(q, k, v, g, clean, dcu, ws=ws)
    k2, v2, q2 = k.clone(), v.clone(), q.clone()
    v2[130, 0, 5] = float("nan")     # sequence 1, head 0, one column
    k2[150, 1, 3] = float("inf")     # sequence 1, head 1
    q2[10, 0] = float("nan")         # its own output
    o = torch.empty_like(clean)
    L.pc_linear_attention_forward(q2, k2, v2, g, o, dcu, ws=ws)
    bad = torch.zeros_like(o, dtype=torch.bool)
    bad[130:190, 0, 5] = True
    bad[150:190, 1] = True
    bad[10, 0] = True
    assert (~torch.isfinite(o[bad])).all()
    # (tokens of a chunk that holds such a value are taken one by one: equal up to the order of sums)
    ro, _ = R.linear_attention(get(q), get(k), get(v), get(g), cu, 32 ** -0.5)
    mo, _ = R.linear_attention(np.abs(get(q)), np.abs(get(k)), np.abs(get(v)), get(g), cu, 32 ** -0.5)
    ok = ~bad.cpu().numpy()
    tol = _bound(typ, 32 + 100 + 40, mo, ro)
    assert (np.abs(get(o) - ro) <= tol)[ok].all()


def test_linear_attention_clamps_bad_offsets():
    import log_space_sum_amd as L
    torch, _ = T()
    rng = np.random.default_rng(5)
    q, k, v, do, _, _ = _att(rng, [70], 2, 2, 16, 16, "f32")
    cu = torch.tensor([-4, 30, 20, 50, 1000], dtype=torch.int32, device=DEV)   # -> 0..30, (none), 20..50, 50..70
    g = put(np.array([-0.1, -0.2]))
    o, s1 = torch.full((70, 2, 16), 3.0, device=DEV), torch.empty((4, 2, 16, 16), device=DEV)
    L.pc_linear_attention_forward(q, k, v, g, o, cu, state_out=s1, ws=L.linear_attention_workspace(q, k, v, cu))
    _, rs = R.linear_attention(*[get(t) for t in (q, k, v, g)], [50, 70], 0.25)
    near(s1[3:], rs, 200 * E32 * 70, "the last sequence's state")
    assert not s1[1].any()


@pytest.mark.parametrize("typ", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("rows,H,K,dk,dv", [(1, 1, 1, 1, 1), (5, 4, 2, 64, 64), (3, 6, 3, 48, 80), (2, 2, 1, 128, 128), (4, 3, 3, 7, 5)])
def test_linear_attention_step(rows, H, K, dk, dv, typ):
    import log_space_sum_amd as L
    torch, types = T()
    rng = np.random.default_rng(rows + dk)
    q, k, v = (put(rng.normal(size=(rows, h, d)), typ) for h, d in ((H, dk), (K, dk), (K, dv)))
    g = put(DECAYS[:H])
    state = put(rng.normal(size=(rows + 2, H, dk, dv)))
    before = get(state)
    o = torch.empty((rows, H, dv), device=DEV, dtype=types[typ])
    L.pc_linear_attention_step(q, k, v, g, state, o, scale=0.5)
    A = [get(t) for t in (q, k, v, g)]
    ro, rs = R.linear_attention(*A, list(range(rows + 1)), 0.5, before[:rows])
    mo, ms = R.linear_attention(*[np.abs(a) for a in A[:3]], A[3], list(range(rows + 1)), 0.5, np.abs(before[:rows]))
    near(o, ro, TINY[typ] + U[typ] * np.abs(ro) + (dk + 8) * E32 * mo, "o")
    near(state[:rows], rs, TINY["f32"] + 4 * E32 * ms, "state")
    assert (get(state)[rows:] == before[rows:]).all()


def test_linear_attention_step_slots():
    """Rows of one slot are successive tokens; slots out of range are padding."""
    import log_space_sum_amd as L
    torch, _ = T()
    rng = np.random.default_rng(6)
    slots = [3, -1, 0, 3, 7, 3, 2 ** 31 - 1, 0]
    n, H, dk, dv = len(slots), 2, 24, 32
    q, k, v = (put(rng.normal(size=(n, H, d))) for d in (dk, dk, dv))
    g, state = put(np.array([-0.3, 0.0])), put(rng.normal(size=(5, H, dk, dv)))
    before = get(state)
    o = torch.full((n, H, dv), 8.0, device=DEV)
    L.pc_linear_attention_step(q, k, v, g, state, o, torch.tensor(slots, dtype=torch.int32, device=DEV), scale=1.0)
    want = before.copy()
    for slot in (0, 3):
        rows = [i for i, s in enumerate(slots) if s == slot]
        ro, rs = R.linear_attention(*[get(t)[rows] for t in (q, k, v)], get(g), [0, len(rows)], 1.0, before[slot:slot + 1])
        near(o[rows], ro, 60 * E32 * dk * 8, f"rows of slot {slot}")
        want[slot] = rs[0]
    near(state, want, 20 * E32 * 8, "states")
    assert (get(state)[[1, 2, 4]] == before[[1, 2, 4]]).all()
    for i in (1, 4, 6):
        assert (o[i] == 8).all()


def test_linear_attention_of_single_tokens_far_apart():
    """Rows at one position of a padded batch, more than 2^23 elements apart: as single tokens, and one of them as a
    sequence of one token."""
    import log_space_sum_amd as L
    torch, _ = T()
    rng = np.random.default_rng(10)
    n, H, dk, dv, far = 3, 2, 16, 24, 2 ** 23 + 40
    buf = torch.zeros(n * far, device=DEV)
    rows = [torch.as_strided(buf, (n, H, d), (far, d, 1), at) for d, at in ((dk, 0), (dk, 100), (dv, 200), (dv, 300))]
    q, k, v, o = rows
    for t in (q, k, v):
        t.copy_(put(rng.normal(size=t.shape)))
    g, state = put(DECAYS[:H]), put(rng.normal(size=(n, H, dk, dv)))
    before = get(state)
    L.pc_linear_attention_step(q, k, v, g, state, o, scale=0.5)
    A = [get(t) for t in (q, k, v, g)]
    cu = list(range(n + 1))
    ro, rs = R.linear_attention(*A, cu, 0.5, before)
    mo, ms = R.linear_attention(*[np.abs(a) for a in A[:3]], A[3], cu, 0.5, np.abs(before))
    near(o, ro, _bound("f32", dk + 8, mo, ro), "o")
    near(state, rs, TINY["f32"] + 4 * E32 * ms, "state")
    o.zero_()
    one = [t[1:2] for t in rows]
    L.pc_linear_attention_forward(*one[:3], g, one[3], state_in=put(before[1:2]), scale=0.5, ws=L.linear_attention_workspace(*one[:3]))
    near(one[3], ro[1:2], _bound("f32", dk + 40, mo, ro)[1:2], "one token")
    dq, dk_, dv_ = (torch.empty(1, *t.shape[1:], device=DEV) for t in one[:3])
    L.pc_linear_attention_backward(one[3], *one[:3], g, dq, dk_, dv_, state_in=put(before[1:2]), scale=0.5,
                                   ws=L.linear_attention_workspace(*one[:3], backward=True))
    B = [get(t) for t in one] + [before[1:2]]
    want = R.linear_attention_grad(B[3], *B[:3], A[3], [0, 1], 0.5, B[4])
    size = R.linear_attention_grad(np.abs(B[3]), *[np.abs(a) for a in B[:3]], A[3], [0, 1], 0.5, np.abs(B[4]))
    for got, ref, mag in zip((dq, dk_, dv_), want, size):
        near(got, ref, _bound("f32", dv + 40, mag, ref), "gradients of one token")


def test_linear_attention_steps_continue_a_prompt():
    import log_space_sum_amd as L
    torch, types = T()
    rng = np.random.default_rng(7)
    lens, H, K, d = [70, 33], 4, 2, 64
    q, k, v, _, cu, dcu = _att(rng, lens, H, K, d, d, "bf16")
    g = put(DECAYS[[0, 1, 3, 5]])
    o, s = torch.empty_like(q), torch.empty((2, H, d, d), device=DEV)
    L.pc_linear_attention_forward(q, k, v, g, o, dcu, state_out=s, ws=L.linear_attention_workspace(q, k, v, dcu))
    more = [put(rng.normal(size=(2, 3, h, d)), "bf16") for h in (H, K, K)]   # three tokens more of each
    got = torch.empty((2, 3, H, d), device=DEV, dtype=types["bf16"])
    for t in range(3):
        row = torch.empty((2, H, d), device=DEV, dtype=types["bf16"])
        L.pc_linear_attention_step(*[m[:, t] for m in more], g, s, row)
        got[:, t] = row
    for i in range(2):
        A = [np.concatenate([get(t)[cu[i]:cu[i + 1]], get(m)[i]]) for t, m in zip((q, k, v), more)]
        n = len(A[0])
        ro, rs = R.linear_attention(*A, get(g), [0, n], d ** -0.5)
        mo, ms = R.linear_attention(*[np.abs(a) for a in A], get(g), [0, n], d ** -0.5)
        near(got[i], ro[-3:], (U["bf16"] * np.abs(ro) + (d + n + 40) * E32 * mo)[-3:], "tokens")
        near(s[i:i + 1], rs, (n + 40) * E32 * ms, "state")


# ---------------------------------------------------------------------------
# orthogonalised update
# ---------------------------------------------------------------------------

QUINTIC = (3.4445, -4.7750, 2.0315)


def _orth_tol(coefficients, m, n, typ):
    """A perturbation of X grows at most by |p'| <= 3.5 a step where singular values are small (|p'| of the quintic on
    [0, 1.2] is at most its value a at 0); float32-level steps add (two planes: 2^-22 an operand, float32 sums of n
    terms that average out: sqrt(n) 2^-24) to each of the three products, in the Frobenius norm of X, at most
    1.2 sqrt(m)."""
    grow = max(abs(c[0]) for c in coefficients)
    one = 6 * 2.0 ** -22 + 3 * np.sqrt(n) * E32
    return one * sum(grow ** k for k in range(len(coefficients) + 1)) * 1.2 * np.sqrt(m)


def _operands(typ, m, steps):
    """What the products see: for bfloat16 matrices too large for the Gram form the operands of A are rounded to
    float16 of a scaled value (11 bits), and so is everything in the first two of five or more steps."""
    exact = lambda x: x  # noqa: E731
    if typ != "bf16" or m <= 64:
        return lambda step: (exact,) * 3
    short = lambda x: (x * 2.0 ** 13).astype(np.float16).astype(np.float64) / 2.0 ** 13  # noqa: E731
    return lambda step: (short,) * 3 if step < 2 and step + 3 < steps else (short, exact, exact)


@pytest.mark.parametrize("typ", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("batch,rows,cols", [(1, 1, 1), (2, 1, 37), (3, 50, 4), (5, 16, 300), (2, 17, 17), (3, 33, 500), (2, 200, 64),
                                             (1, 64, 65), (2, 65, 65), (1, 70, 400), (2, 300, 129), (1, 256, 128)])
def test_orthogonalize(batch, rows, cols, typ):
    import log_space_sum_amd as L
    torch, types = T()
    rng = np.random.default_rng(rows * 3 + cols)
    whole = put(rng.normal(size=(batch, rows + 2, cols + 3)) * 0.01, typ)
    g = whole[:, 1:1 + rows, 2:2 + cols]
    out = torch.full((batch, rows + 1, cols + 1), 6.0, device=DEV, dtype=types[typ])
    y = out[:, :rows, :cols]
    L.pc_orthogonalize(g, y, ws=L.orthogonalize_workspace(g))
    co = [QUINTIC] * 5
    m, n = sorted((rows, cols))
    tol = _orth_tol(co, m, n, typ)
    for b in range(batch):
        ref = R.orthogonalize(get(g)[b], co, 1e-7, _operands(typ, m, 5))
        d = get(y)[b] - ref
        assert np.linalg.norm(d) <= tol + U[typ] * np.linalg.norm(ref), (b, np.linalg.norm(d), tol)
        # element by element: no place is off by what a wrong or missing element would be
        assert np.abs(d).max() <= tol + U[typ] * np.abs(ref).max()
    assert (out[:, rows] == 6).all() and (out[:, :, cols] == 6).all()
    # in place, same bits
    L.pc_orthogonalize(g, g, ws=L.orthogonalize_workspace(g))
    assert torch.equal(g, y)


@pytest.mark.parametrize("rows,cols", [(40, 90), (90, 130)])
def test_orthogonalize_edges(rows, cols):
    import log_space_sum_amd as L
    torch, _ = T()
    rng = np.random.default_rng(8)
    g = put(rng.normal(size=(5, rows, cols)))
    g[1] = 0                                             # zeros stay zeros
    g[2, 3, 4] = float("nan")                            # reaches its own matrix only
    g[3] = put(np.outer(rng.normal(size=rows), rng.normal(size=cols)) * 1e-18)   # rank 1, squares below float32's range
    g[4] = g[4] * 1e25                                   # squares above it
    out = torch.empty_like(g)
    # one triple for each step
    co = [(2.0, -1.5, 0.5), QUINTIC, (1.5, -0.5, 0.0)]
    L.pc_orthogonalize(g, out, steps=3, coefficients=co, eps=1e-20, ws=L.orthogonalize_workspace(g))
    assert not out[1].any() and not torch.isfinite(out[2]).any()
    for b in (0, 3, 4):
        ref = R.orthogonalize(get(g)[b], co, 1e-20)
        assert np.linalg.norm(get(out)[b] - ref) <= _orth_tol(co, rows, cols, "f32")
    with pytest.raises(L.PCError, match="grow past"):
        L.pc_orthogonalize(g, out, steps=4, coefficients=(20.0, 1.0, 1.0), ws=L.orthogonalize_workspace(g))


@pytest.mark.parametrize("typ", ["f32", "bf16"])
@pytest.mark.parametrize("rows,cols", [(2100, 2100), (25600, 300), (1100, 4200)])
def test_orthogonalize_many_tiles(rows, cols, typ):
    """Sizes with whole rounds of tiles and some left over, with a long and a short K; the steps in float64 on the GPU."""
    import log_space_sum_amd as L
    torch, types = T()
    gen = torch.Generator(device=DEV)
    gen.manual_seed(rows)
    g = (torch.randn((rows, cols), generator=gen, device=DEV) * 0.1).to(types[typ])
    out = torch.empty_like(g)
    L.pc_orthogonalize(g, out, ws=L.orthogonalize_workspace(g))
    m, n = sorted((rows, cols))
    x = g.double().t() if rows > cols else g.double()
    x = x / (x.square().sum().sqrt() + 1e-7)
    short = lambda v: (v * 2.0 ** 13).half().double() / 2.0 ** 13  # noqa: E731
    for step, (a, b, c) in enumerate([QUINTIC] * 5):
        r = [short] * 3 if typ == "bf16" and step < 2 else [short if typ == "bf16" else (lambda v: v)] + [lambda v: v] * 2
        A = r[0](x) @ r[0](x).t().contiguous()
        x = a * x + r[2](b * A + c * (r[1](A) @ r[1](A))) @ r[2](x)
    ref = x.t() if rows > cols else x
    tol = _orth_tol([QUINTIC] * 5, m, n, typ)
    d = out.double() - ref
    assert float(d.norm()) <= tol + U[typ] * float(ref.norm())
    assert float(d.abs().max()) <= tol / 10 + U[typ] * float(ref.abs().max())
    first = out.clone()
    L.pc_orthogonalize(g, out, ws=L.orthogonalize_workspace(g))
    assert torch.equal(first, out)


def test_orthogonalize_tiny_values():
    """Matrices whose norm's inverse is past float32, without eps."""
    import log_space_sum_amd as L
    torch, _ = T()
    rng = np.random.default_rng(11)
    for rows, cols in ((20, 40), (70, 140)):
        g = put(rng.normal(size=(rows, cols)) * 1e-37)
        out = torch.empty_like(g)
        L.pc_orthogonalize(g, out, eps=0.0, ws=L.orthogonalize_workspace(g))
        ref = R.orthogonalize(get(g), [QUINTIC] * 5, 0.0)
        assert np.linalg.norm(get(out) - ref) <= _orth_tol([QUINTIC] * 5, rows, cols, "f32")


@pytest.mark.parametrize("rows,cols", [(128, 256), (333, 1000), (700, 700)])
def test_orthogonalize_has_no_element_that_stands_out(rows, cols):
    """The two planes of every value belong together.  Errors of many small roundings are nearly normal: the largest
    of 10^6 lies at 5 of their deviations, 7.4 of the median size, 24 with rows and columns that differ by a factor
    of 3.  One value whose planes do not match is off by 2^-11, 2^11 of a rounding to two planes."""
    import log_space_sum_amd as L
    torch, _ = T()
    g = put(np.random.default_rng(13).normal(size=(rows, cols)) * 1e-3)
    out = torch.empty_like(g)
    L.pc_orthogonalize(g, out, ws=L.orthogonalize_workspace(g))
    d = np.abs(get(out) - R.orthogonalize(get(g), [QUINTIC] * 5, 1e-7))
    assert d.max() <= 24 * np.median(d)


@pytest.mark.parametrize("batch,rows,cols,typ", [(3, 333, 1000, "f32"), (2, 700, 700, "f16"), (1, 1100, 1300, "bf16")])
def test_orthogonalize_gives_the_same_bits_every_time(batch, rows, cols, typ):
    """Sums have a fixed order: every call, whatever its workspace held before, gives the first one's bits."""
    import log_space_sum_amd as L
    torch, _ = T()
    g = put(np.random.default_rng(12).normal(size=(batch, rows, cols)), typ)
    ws = L.orthogonalize_workspace(g)
    first, out = torch.empty_like(g), torch.empty_like(g)
    L.pc_orthogonalize(g, first, ws=ws)
    wrong = torch.zeros((), device=DEV, dtype=torch.int64)
    for k in range(400):
        ws.fill_(127 if k % 2 else 60)
        L.pc_orthogonalize(g, out, ws=ws)
        wrong += (out != first).sum()
    assert int(wrong) == 0


# Accuracy of the planes.  A value in two float16 planes is off by at most 2^-23 of itself, the product of the two
# small planes that is left out by 2^-24 of the product's terms, and a float32 sum of n terms by about sqrt(n) 2^-25 of
# its terms' norm: each of a step's three products is off by less than 1e-6 of its norm for n <= 1300, and the steps on
# random matrices, whose singular values and perturbations grow alike, add them up to 2e-6 of the result (the steps
# with rounded operands: tests/test_operators.py).  Ten times that is allowed; one plane anywhere costs 4e-4 or more.
PLANES = 2e-5


@pytest.mark.parametrize("typ", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("batch,rows,cols", [(2, 65, 65), (1, 70, 400), (2, 300, 129), (1, 256, 128), (3, 333, 1000), (1, 700, 700),
                                             (1, 1100, 1300)])
def test_orthogonalize_is_float32_exact_in_every_type(batch, rows, cols, typ):
    """The result before its rounding is within PLANES of the definition.  float32: that, normwise and element by
    element (nearly normal errors: the largest of 10^6 below 24 deviations).  16-bit types: an element whose value lies
    d from the definition's rounds differently in a share d / step of the cases, then by a step, at most 2 u of the
    value: the squares of the differences from the rounded definition sum to at most 2 u PLANES of the result's."""
    import log_space_sum_amd as L
    torch, types = T()
    g = put(np.random.default_rng(rows + 3 * cols).normal(size=(batch, rows, cols)) * 1e-3, typ)
    out = torch.empty_like(g)
    L.pc_orthogonalize(g, out, ws=L.orthogonalize_workspace(g))
    for b in range(batch):
        ref = R.orthogonalize(get(g)[b], [QUINTIC] * 5, 1e-7)
        size, rms = np.linalg.norm(ref), np.sqrt((ref * ref).mean())
        d = get(out)[b] - ref
        assert (np.abs(d) <= U[typ] * np.abs(ref) + 24 * PLANES * rms + TINY[typ]).all()
        if typ == "f32":
            assert np.linalg.norm(d) <= (PLANES + E32) * size
        else:
            off = get(out)[b] - get(put(ref, typ))
            assert np.linalg.norm(off) <= np.sqrt(2 * U[typ] * PLANES) * size


CUBIC = (1.5, -0.5, 0.0)
TUNED = [(8.287, -23.596, 17.300), (4.107, -2.948, 0.545), (3.949, -2.909, 0.552), (3.318, -2.488, 0.510), (2.301, -1.669, 0.419)]


def _exact_rank(rng, m, n, rank):
    """A matrix of small whole numbers of exactly this rank (or less), in every type."""
    return rng.integers(-4, 5, size=(m, rank)).astype(float) @ rng.integers(-4, 5, size=(rank, n))


def _by_singular_values(g, co):
    """The steps on the singular values with the coefficients that the library takes, float32; the values that should
    be 0 kept there; the largest growth of a relative error of one; the smallest one at the start."""
    u, s, v = np.linalg.svd(g, full_matrices=False)
    t = s / np.linalg.norm(g)
    t[t < 1e-12] = 0
    live, grow, least = t > 0, np.ones(len(t)), t[t > 0].min()
    for a, b, c in np.float32(co).astype(np.float64):
        grow = grow * np.maximum(1, np.abs(a + 3 * b * t ** 2 + 5 * c * t ** 4))
        t = a * t + b * t ** 3 + c * t ** 5
    return (u * t) @ v, grow[live].max(), least


@pytest.mark.parametrize("typ", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("m,n", [(16, 1024), (4, 37), (33, 500), (64, 300), (20, 20)])
def test_orthogonalize_many_steps_of_thin_matrices(m, n, typ):
    """Matrices without full rank, whose missing singular values must stay out of the result however many the steps.
    What the m x m form may add: Q's rounding in 64 bits, m 2^-53 of the largest Q, 2 / sqrt(d) (a few times), and the
    shift d, relative to the smallest singular value's square, times the growth of a relative error over the steps.
    Up to a growth of Q of 2048 the steps run on A itself, whose rounding grows as Q's square."""
    import log_space_sum_amd as L
    torch, types = T()
    rng = np.random.default_rng(m * n)
    for rank in (1, 4):
        g = np.stack([_exact_rank(rng, m, n, rank) for _ in range(2)])
        x = put(g, typ)
        assert (get(x) == g).all()
        for co in ([QUINTIC] * 6, [QUINTIC] * 8, [QUINTIC] * 10, [QUINTIC] * 16, [QUINTIC] * 20, [QUINTIC] * 32, [CUBIC] * 32):
            out = torch.empty_like(x)
            L.pc_orthogonalize(x, out, steps=len(co), coefficients=co, eps=0.0, ws=L.orthogonalize_workspace(x))
            growth = np.prod([a for a, _, _ in co])
            for b in range(2):
                ref, grow, least = _by_singular_values(g[b], co)
                d = 4 * (n / 8 + 16 + m) * 2.0 ** -53
                tol = 8 * m * 2.0 ** -53 / np.sqrt(d) + d / least ** 2 * grow + (8 * m * 2.0 ** -53 * growth ** 2 if growth <= 2048 else 0)
                e = np.linalg.norm(get(out)[b] - ref)
                assert e <= (tol + U[typ]) * np.linalg.norm(ref), (rank, len(co), co[0], e / np.linalg.norm(ref), tol)


@pytest.mark.parametrize("rows,cols", [(20, 300), (64, 64), (130, 90), (300, 300)])
def test_orthogonalize_with_a_triple_for_each_step(rows, cols):
    """Triples tuned step by step, which rise steeply behind their interval.  A step's roundings, 3 2^-22 of X, grow by at
    most the largest |p'| between 0 and the largest singular value in each later step."""
    import log_space_sum_amd as L
    torch, _ = T()
    rng = np.random.default_rng(rows)
    for g in (rng.normal(size=(rows, cols)), rng.integers(-4, 5, size=(rows, 1)) @ rng.integers(-4, 5, size=(1, cols))):
        x = put(g)
        out = torch.empty_like(x)
        co = [(a / 1.01, b / 1.01 ** 3, c / 1.01 ** 5) for a, b, c in TUNED[:-1]] + TUNED[-1:] + [(1.875, -1.25, 0.375)] * 2
        L.pc_orthogonalize(x, out, steps=len(co), coefficients=co, ws=L.orthogonalize_workspace(x))
        co = np.float32(co).astype(np.float64)
        ref = R.orthogonalize(get(x), co, 1e-7)
        t = np.linalg.svd(get(x), compute_uv=False)
        t, tol = t / np.linalg.norm(t), 0.0
        for a, b, c in co:
            z = np.linspace(0, t.max(), 2001)
            tol = (tol + 3 * 2.0 ** -22 * np.linalg.norm(t)) * np.abs(a + 3 * b * z ** 2 + 5 * c * z ** 4).max()
            t = a * t + b * t ** 3 + c * t ** 5
        assert np.linalg.norm(get(out) - ref) <= tol + E32 * np.linalg.norm(ref)


@pytest.mark.parametrize("m,n", [(4, 37), (33, 500), (64, 130)])
def test_orthogonalize_at_the_ends_of_float32(m, n):
    """Rank 1 and 4 matrices scaled by a power of two, which changes nothing: subnormal elements whose norm's inverse, times
    the growth of Q, is far past float32, and elements near its largest."""
    import log_space_sum_amd as L
    torch, _ = T()
    rng = np.random.default_rng(m + n)
    for rank in (1, 4):
        g = _exact_rank(rng, m, n, rank)
        outs = []
        for e in (0, -140, 118):
            x = put(np.ldexp(g, e))
            assert (get(x) == np.ldexp(g, e)).all()
            outs.append(torch.empty_like(x))
            L.pc_orthogonalize(x, outs[-1], eps=0.0, ws=L.orthogonalize_workspace(x))
        ref, _, _ = _by_singular_values(g, [QUINTIC] * 5)
        for out in outs:
            assert np.linalg.norm(get(out) - ref) <= (E32 + 8 * m * 2.0 ** -53 * 485.0 ** 2) * np.linalg.norm(ref)


@pytest.mark.parametrize("rows,cols", [(16, 1024), (500, 48), (90, 130)])
def test_orthogonalize_many_steps_stay_bounded(rows, cols):
    """Rank 1 up to float32's rounding of its elements, whose small singular values the steps raise to the others' size;
    a matrix of zeros and one with a NaN beside it.  The quintic's values stay below 1.2 (float32 steps for more than
    64 rows: their roundings join, each below 1e-6 of the value)."""
    import log_space_sum_amd as L
    torch, _ = T()
    rng = np.random.default_rng(15)
    g = torch.stack([put(rng.normal(size=(rows, 1)) @ rng.normal(size=(1, cols))) for _ in range(4)])
    g[1] = 0
    g[2, 3, 4] = float("nan")
    for steps in (7, 12, 16, 20, 32):
        out = torch.empty_like(g)
        L.pc_orthogonalize(g, out, steps=steps, ws=L.orthogonalize_workspace(g))
        assert not out[1].any() and not torch.isfinite(out[2]).any()
        for b in (0, 3):
            s = np.linalg.svd(get(out)[b], compute_uv=False)
            assert np.isfinite(s).all() and s.max() <= 1.21, (steps, s.max())
            assert s.max() >= 0.6


# ---------------------------------------------------------------------------
# together
# ---------------------------------------------------------------------------

def test_offsets_past_32_bits():
    """Rows, tokens, slots and matrices that lie more than 2^31 elements into their buffers."""
    import log_space_sum_amd as L
    torch, types = T()
    rng = np.random.default_rng(12)
    far = 2 ** 31 + 64
    buf = torch.empty(far + 2 ** 22, dtype=types["bf16"], device=DEV)
    # layer norm: two rows 2^31 apart
    x = torch.as_strided(buf, (2, 100), (far, 1))
    x.copy_(put(rng.normal(size=(2, 100)), "bf16"))
    y = torch.empty((2, 100), device=DEV, dtype=types["bf16"])
    L.pc_layer_norm_forward(x, None, None, y)
    ry, _, _ = R.layer_norm(get(x))
    near(y, ry, U["bf16"] * np.abs(ry) + 100 * E32 * 8, "norm")
    # orthogonalise: two matrices 2^31 apart, thin and wide
    for rows, cols in ((8, 50), (70, 90)):
        g = torch.as_strided(buf, (2, rows, cols), (far, cols, 1))
        g.copy_(put(rng.normal(size=(2, rows, cols)), "bf16"))
        out = torch.empty((2, rows, cols), device=DEV, dtype=types["bf16"])
        L.pc_orthogonalize(g, out, ws=L.orthogonalize_workspace(g))
        for b in range(2):
            ref = R.orthogonalize(get(g)[b], [QUINTIC] * 5, 1e-7, _operands("bf16", min(rows, cols), 5))
            assert np.linalg.norm(get(out)[b] - ref) <= _orth_tol([QUINTIC] * 5, *sorted((rows, cols)), "bf16") + U["bf16"] * np.linalg.norm(ref)
    # linear attention: the last tokens of a long buffer
    H, d = 4, 64
    n = buf.numel() // (H * d)
    t = buf[:n * H * d].view(n, H, d)
    t[-90:] = put(rng.normal(size=(90, H, d)), "bf16")
    cu = torch.tensor([n - 90, n - 20, n], dtype=torch.int32, device=DEV)
    g = put(np.array([-0.1, 0.0, -1.0, -0.01]))
    s = torch.empty((2, H, d, d), device=DEV)
    o = torch.empty_like(t)
    L.pc_linear_attention_forward(t, t, t, g, o, cu, 70, state_out=s, ws=L.linear_attention_workspace(t, t, t, cu, 70))
    z = get(t[-90:])
    ro, rs = R.linear_attention(z, z, z, get(g), [0, 70, 90], d ** -0.5)
    mo, ms = R.linear_attention(*[np.abs(z)] * 3, get(g), [0, 70, 90], d ** -0.5)
    near(o[-90:], ro, _bound("bf16", 200, mo, ro), "o")
    near(s, rs, 200 * E32 * ms, "state")
    del o, t, buf, x, g
    torch.cuda.empty_cache()
    # a pool of states with more than 2^31 elements
    slots, H, d = 131075, 4, 64
    pool = torch.empty((slots, H, d, d), device=DEV)
    last = torch.tensor([slots - 1, slots, slots - 2], dtype=torch.int32, device=DEV)
    pool[-2:] = 0
    q = put(rng.normal(size=(3, H, d)))
    o, g = torch.zeros_like(q), put(np.zeros(4))
    L.pc_linear_attention_step(q, q, q, g, pool, o, last, scale=1.0)
    z = get(q)
    want = np.einsum("bhk,bhk->bh", z, z)[..., None] * z
    want[1] = 0
    near(o, want, 80 * E32 * np.einsum("bhk,bhk->bh", z, z)[..., None] * np.abs(z), "step")


def test_linear_attention_step_of_more_rows_than_a_launch_has_blocks():
    """2^24 rows and some: as many blocks of 256 threads along one dimension are 2^32, which no launch takes."""
    import log_space_sum_amd as L
    torch, _ = T()
    n = 2 ** 24 + 5
    gen = torch.Generator(device=DEV)
    gen.manual_seed(3)
    q, k, v = (torch.randn((n, 1, 1), generator=gen, device=DEV) for _ in range(3))
    state, o = torch.randn((n, 1, 1, 1), generator=gen, device=DEV), torch.empty((n, 1, 1), device=DEV)
    before = state.double()
    L.pc_linear_attention_step(q, k, v, put(np.array([-0.5])), state, o, scale=1.0)
    left = np.exp(-0.5) * before[..., 0]
    want = left + k.double() * v.double()
    size = left.abs() + (k * v).abs()
    # the decay's, two products' and the sum's roundings, and one more of the output's product
    assert ((state[..., 0].double() - want).abs() <= 4 * E32 * size + TINY["f32"]).all()
    assert ((o.double() - q.double() * want).abs() <= 5 * E32 * size * q.abs() + TINY["f32"]).all()


def test_linear_attention_gradients_of_more_elements_than_a_launch_has_threads():
    """Shared heads, 2^20 + 256 tokens x 32 key heads x 128: 2^32 sums of two heads and some.  Inputs are one token
    repeated (stride 0); the sequences are the first and the last tokens, the ones between stay as they were."""
    import log_space_sum_amd as L
    torch, types = T()
    n, K, dk, few = 2 ** 20 + 256, 32, 128, 40
    rng = np.random.default_rng(21)
    one = [put(rng.normal(size=(1, h, d)), "bf16") for h, d in ((2 * K, dk), (K, dk), (K, 1), (2 * K, 1))]
    q, k, v, do = (t.expand(n, -1, -1) for t in one)
    dq, dk_, dv_ = (torch.empty((n, h, d), device=DEV, dtype=types["bf16"]) for h, d in ((2 * K, dk), (K, dk), (K, 1)))
    dk_[few:few + 10] = 5
    dk_[n - few - 10:n - few] = 5
    g = put(np.full(2 * K, -0.1))
    for start, end in ((0, few), (n - few, n)):
        cu = torch.tensor([start, end], dtype=torch.int32, device=DEV)
        L.pc_linear_attention_backward(do, q, k, v, g, dq, dk_, dv_, cu, few, scale=1.0,
                                       ws=L.linear_attention_workspace(q, k, v, cu, few, backward=True))
        A = [np.repeat(get(t), few, 0) for t in one]
        want = R.linear_attention_grad(A[3], *A[:3], get(g), [0, few], 1.0)
        size = R.linear_attention_grad(np.abs(A[3]), *[np.abs(a) for a in A[:3]], get(g), [0, few], 1.0)
        for got, ref, mag, name in zip((dq, dk_, dv_), want, size, ("dq", "dk", "dv")):
            near(got[start:end], ref, _bound("bf16", dk + few + 40, mag, ref), name)
    assert (dk_[few:few + 10] == 5).all() and (dk_[n - few - 10:n - few] == 5).all()
    del dq, dk_, dv_
    torch.cuda.empty_cache()


@pytest.mark.parametrize("typ", ["f32", "bf16"])
def test_linear_attention_of_many_sequences_without_a_bound_of_the_lengths(typ):
    """Short, empty and a few long sequences with max_seqlen left out: few of them have segments, whose states are packed.
    States in place, and a workspace that holds NaN before."""
    import log_space_sum_amd as L
    torch, types = T()
    rng = np.random.default_rng(17)
    lens = [int(x) for x in rng.integers(0, 30, size=150)]
    lens[0], lens[40], lens[41], lens[42], lens[90], lens[-1] = 700, 129, 0, 300, 257, 400
    H, K, dk, dv = 4, 2, 16, 24
    q, k, v, do, cu, dcu = _att(rng, lens, H, K, dk, dv, typ, tail=3)
    g = put(DECAYS[[0, 1, 5, 6]])
    s0, ds = (put(rng.normal(size=(len(lens), H, dk, dv))) for _ in range(2))
    o, s1, d0 = torch.empty_like(do), s0.clone(), ds.clone()
    dq, dk_, dv_ = (torch.empty_like(t) for t in (q, k, v))
    ws = L.linear_attention_workspace(q, k, v, dcu)
    assert 0 < ws.numel() < len(lens) * H * dk * dv * 4 * 2
    L.pc_linear_attention_forward(q, k, v, g, o, dcu, None, s1, s1, 0.3, ws.fill_(255))
    L.pc_linear_attention_backward(do, q, k, v, g, dq, dk_, dv_, dcu, None, s0, d0, d0, 0.3,
                                   L.linear_attention_workspace(q, k, v, dcu, backward=True).fill_(255))
    A = [get(t) for t in (q, k, v, g, s0, do, ds)]
    B = [np.abs(a) for a in A]
    ro, rs = R.linear_attention(*A[:4], cu, 0.3, A[4])
    mo, ms = R.linear_attention(*B[:3], A[3], cu, 0.3, B[4])
    live, terms = cu[-1], dk + max(lens) + 40
    near(o[:live], ro[:live], _bound(typ, terms, mo, ro)[:live], "o")
    near(s1, rs, TINY["f32"] + E32 * np.abs(rs) + terms * E32 * ms, "state")
    want = R.linear_attention_grad(A[5], *A[:4], cu, 0.3, A[4], A[6])
    size = R.linear_attention_grad(B[5], *B[:3], A[3], cu, 0.3, B[4], B[6])
    for got, ref, mag, name in zip((dq, dk_, dv_), want, size, ("dq", "dk", "dv")):
        near(got[:live], ref[:live], _bound(typ, terms + H, mag, ref)[:live], name)
    near(d0, want[3], TINY["f32"] + E32 * np.abs(want[3]) + terms * E32 * size[3], "dstate")


def test_linear_attention_many_short_sequences():
    """More sequences than one grid takes three times over; one token each."""
    import log_space_sum_amd as L
    torch, _ = T()
    rng = np.random.default_rng(13)
    n, H, d = 30000, 1, 4
    q, k, v, do = (put(rng.normal(size=(n, H, d))) for _ in range(4))
    cu = torch.arange(n + 1, dtype=torch.int32, device=DEV)
    s0, ds = put(rng.normal(size=(n, H, d, d))), put(rng.normal(size=(n, H, d, d)))
    g, lam = put(np.array([-0.5])), np.exp(-0.5)
    o, s1, d0 = torch.empty_like(q), torch.empty_like(s0), torch.empty_like(s0)
    dq, dk, dv = (torch.empty_like(q) for _ in range(3))
    L.pc_linear_attention_forward(q, k, v, g, o, cu, 1, s0, s1, 1.0, L.linear_attention_workspace(q, k, v, cu, 1))
    L.pc_linear_attention_backward(do, q, k, v, g, dq, dk, dv, cu, 1, s0, ds, d0, 1.0,
                                   L.linear_attention_workspace(q, k, v, cu, 1, backward=True))
    Q, K, V, G, S, D = (get(x) for x in (q, k, v, do, s0, ds))
    S = lam * S + K[..., :, None] * V[..., None, :]
    D = D + Q[..., :, None] * G[..., None, :]
    tol = 64 * E32 * 200   # sums of four products of normal values, at most about 6^3
    for got, want in ((s1, S), (o, np.einsum("thk,thkv->thv", Q, S)), (dq, np.einsum("thkv,thv->thk", S, G)),
                      (dk, np.einsum("thkv,thv->thk", D, V)), (dv, np.einsum("thkv,thk->thv", D, K)), (d0, lam * D)):
        near(got, want, tol, "one token")


def test_calls_on_two_streams_at_once():
    """Two calls of each operator at the same time, on their own streams and workspaces, give the results of one alone."""
    import log_space_sum_amd as L
    torch, types = T()
    rng = np.random.default_rng(14)
    data = []
    for _ in range(2):
        q, k, v, do, cu, dcu = _att(rng, [900, 500], 4, 2, 64, 64, "bf16")
        m = put(rng.normal(size=(1400, 256)), "bf16")
        data.append(dict(q=q, k=k, v=v, do=do, cu=dcu, m=m, g=put(DECAYS[:4]), o=torch.empty_like(q), dq=torch.empty_like(q),
                         dk=torch.empty_like(k), dv=torch.empty_like(v), up=torch.empty_like(m), dx=torch.empty_like(m),
                         w=torch.empty(256, device=DEV), mean=torch.zeros(1400, device=DEV), rstd=torch.ones(1400, device=DEV),
                         w1=L.linear_attention_workspace(q, k, v, dcu), w2=L.linear_attention_workspace(q, k, v, dcu, backward=True),
                         w3=L.orthogonalize_workspace(m), w4=L.layer_norm_workspace(1400, 256, DEV)))
    names = ("o", "dq", "dk", "dv", "up", "dx", "w")

    def calls(s):
        L.pc_linear_attention_forward(s["q"], s["k"], s["v"], s["g"], s["o"], s["cu"], ws=s["w1"])
        L.pc_linear_attention_backward(s["do"], s["q"], s["k"], s["v"], s["g"], s["dq"], s["dk"], s["dv"], s["cu"], ws=s["w2"])
        L.pc_orthogonalize(s["m"], s["up"], ws=s["w3"])
        L.pc_layer_norm_backward(s["m"], s["m"], None, s["mean"], s["rstd"], s["dx"], s["w"], None, s["w4"])

    for s in data:
        calls(s)
    torch.cuda.synchronize()
    want = [{n: s[n].clone() for n in names} for s in data]
    streams = [torch.cuda.Stream() for _ in data]
    for _ in range(5):
        for s in data:
            for n in names:
                s[n].fill_(3)
        torch.cuda.synchronize()
        for s, st in zip(data, streams):
            with torch.cuda.stream(st):
                calls(s)
        torch.cuda.synchronize()
        for s, w in zip(data, want):
            assert all(torch.equal(s[n], w[n]) for n in names)


def test_captured_calls_replay():
    """All calls in one captured graph on a stream of its own; every replay equals the eager results on new inputs,
    with eager work and synchronizations between."""
    import log_space_sum_amd as L
    torch, types = T()
    bf = types["bf16"]
    n, H, d = 700, 2, 64
    x, y = torch.empty((n, H * d), device=DEV, dtype=bf), torch.empty((n, H * d), device=DEV, dtype=bf)
    mean, rstd = torch.empty(n, device=DEV), torch.empty(n, device=DEV)
    g = put(np.array([-0.1, -0.01]))
    k, v, do = (torch.empty((n, H, d), device=DEV, dtype=bf) for _ in range(3))
    cu = torch.tensor([0, 650, n], dtype=torch.int32, device=DEV)
    o, dq, dk, dv, dx = (torch.empty((n, H, d), device=DEV, dtype=bf) for _ in range(5))
    dw, db = torch.empty(H * d, device=DEV), torch.empty(H * d, device=DEV)
    state = torch.zeros((2, H, d, d), device=DEV)
    upd, thin = torch.empty((n, H * d), device=DEV, dtype=bf), torch.empty((n, d), device=DEV, dtype=bf)
    w1, w2 = L.linear_attention_workspace(x.view(n, H, d), k, v, cu), L.linear_attention_workspace(x.view(n, H, d), k, v, cu, backward=True)
    w3, w4, w5 = L.layer_norm_workspace(n, H * d, DEV), L.orthogonalize_workspace(x), L.orthogonalize_workspace(thin)
    outs = [y, mean, rstd, o, state, dq, dk, dv, dx, dw, db, upd, thin]

    def calls():
        L.pc_layer_norm_forward(x, None, None, y, mean, rstd)
        q = y.view(n, H, d)
        L.pc_linear_attention_forward(q, k, v, g, o, cu, state_out=state, ws=w1)
        L.pc_linear_attention_step(q[:2], k[:2], v[:2], g, state, o[:2])
        L.pc_linear_attention_backward(do, q, k, v, g, dq, dk, dv, cu, ws=w2)
        L.pc_layer_norm_backward(dq.view(n, H * d), x, None, mean, rstd, dx.view(n, H * d), dw, db, w3)
        L.pc_orthogonalize(dx.view(n, H * d), upd, ws=w4)
        L.pc_orthogonalize(dx[:, 0], thin, ws=w5)

    def fill(seed):
        gen = torch.Generator(device=DEV)
        gen.manual_seed(seed)
        for t in (x, k, v, do):
            t.copy_(torch.randn(t.shape, generator=gen, device=DEV))

    fill(0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        calls()
        side.synchronize()
        with torch.cuda.graph(graph, stream=side):
            calls()
    torch.cuda.synchronize()
    for seed in (1, 2, 3):
        fill(seed)
        calls()
        torch.cuda.synchronize()
        want = [t.clone() for t in outs]
        for t in outs:
            t.fill_(7)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(outs, want):
            assert torch.equal(a, b)


def test_factors_of_a_conditional_circuit_learn():
    """What the operators are for: a context is normalised and mixed along the sequence, a product makes the LowRank
    factors of an HMM's transitions from it, the circuit's backward gives dLL/dA and dLL/dB, and the gradients walk
    back through the operators to a matrix, whose update is orthogonalised.  Against the same chain in float64."""
    import log_space_sum_amd as L
    import oracle
    from workloads import make_config
    torch, _ = T()
    cfg = make_config("lowrank", H=24, T=4, V=6, rank=3, B=16)
    circ, B = cfg["circuit"], cfg["B"]
    M, k = cfg["lowrank"][0][0].shape[1:]
    N, slots = cfg["lowrank"][0][1].shape[2], len(cfg["lowrank"])
    rng = np.random.default_rng(9)
    heads, d, F = 2, 8, 16
    x = put(rng.normal(size=(B * slots, F)) + 0.2)                  # a context of one vector a slot and sample
    w, b, g = put(1 + 0.1 * rng.normal(size=F)), put(0.1 * rng.normal(size=F)), put(np.array([-0.2, -0.05]))
    Wa, Wb = put(rng.normal(size=(F, M * k)) * 0.1), put(rng.normal(size=(F, k * N)) * 0.1)
    cu = torch.tensor([i * slots for i in range(B + 1)], dtype=torch.int32, device=DEV)
    h = L.pc_compile_layout(circ, device=0)
    L.pc_set_precision(h, "fp32")
    params, tokens = put(cfg["params"]), torch.tensor(cfg["tokens"], device=DEV)

    # forward: normalise, mix (q = k = v), factors
    y, mean, rstd = torch.empty_like(x), torch.empty(B * slots, device=DEV), torch.empty(B * slots, device=DEV)
    L.pc_layer_norm_forward(x, w, b, y, mean, rstd)
    q = y.view(-1, heads, d)
    o = torch.empty_like(q)
    L.pc_linear_attention_forward(q, q, q, g, o, cu, max_seqlen=slots, ws=L.linear_attention_workspace(q, q, q, cu, slots))
    feat = o.view(B, slots, F)
    lr = [((feat[:, s] @ Wa).view(B, M, k).contiguous(), (feat[:, s] @ Wb).view(B, k, N).contiguous()) for s in range(slots)]
    vals, flows = torch.empty((circ.num_nodes, B), device=DEV), torch.empty((circ.num_nodes, B), device=DEV)
    pflows, ll, ws = torch.zeros(circ.num_params, device=DEV), torch.empty(B, device=DEV), L.workspace(h, B, DEV)
    grads = [(torch.empty_like(a), torch.empty_like(c)) for a, c in lr]
    L.pc_forward(h, B, tokens, params, vals, ll, lr, ws)
    L.pc_backward(h, B, tokens, params, vals, flows, pflows, 0, lr, grads, ws)
    # backward
    dfeat = torch.stack([ga.view(B, -1) @ Wa.t() + gb.view(B, -1) @ Wb.t() for ga, gb in grads], 1)
    dWa = sum(feat[:, s].t() @ grads[s][0].view(B, -1) for s in range(slots))
    dq, dk, dv = (torch.empty_like(q) for _ in range(3))
    L.pc_linear_attention_backward(dfeat.reshape(-1, heads, d), q, q, q, g, dq, dk, dv, cu, max_seqlen=slots,
                                   ws=L.linear_attention_workspace(q, q, q, cu, slots, backward=True))
    dy = (dq + dk + dv).view(-1, F)
    dx, dw, db = torch.empty_like(x), torch.empty_like(w), torch.empty_like(b)
    L.pc_layer_norm_backward(dy, x, w, mean, rstd, dx, dw, db, L.layer_norm_workspace(B * slots, F, DEV))
    up = torch.empty_like(dWa)
    L.pc_orthogonalize(dWa, up, ws=L.orthogonalize_workspace(dWa))
    torch.cuda.synchronize()

    # the same in float64
    ry, rm, rr = R.layer_norm(get(x), get(w), get(b))
    rq = ry.reshape(-1, heads, d)
    lens = [i * slots for i in range(B + 1)]
    rf = R.linear_attention(rq, rq, rq, get(g), lens, d ** -0.5)[0].reshape(B, slots, F)
    rlr = [((rf[:, s] @ get(Wa)).reshape(B, M, k), (rf[:, s] @ get(Wb)).reshape(B, k, N)) for s in range(slots)]
    p64 = cfg["params"].astype(np.float64)
    V, rll = oracle.forward(circ, p64, B, tokens=cfg["tokens"], lowrank=rlr)
    r = oracle.backward(circ, p64, V, tokens=cfg["tokens"], lowrank=rlr)
    rdf = np.stack([a.reshape(B, -1) @ get(Wa).T + c.reshape(B, -1) @ get(Wb).T for a, c in ((r["dA"][s], r["dB"][s]) for s in range(slots))], 1)
    rdWa = sum(rf[:, s].T @ r["dA"][s].reshape(B, -1) for s in range(slots))
    gq, gk, gv, _ = R.linear_attention_grad(rdf.reshape(-1, heads, d), rq, rq, rq, get(g), lens, d ** -0.5)
    rdx, rdw, rdb = R.layer_norm_grad((gq + gk + gv).reshape(-1, F), get(x), rm, rr, get(w))
    rup = R.orthogonalize(rdWa, [QUINTIC] * 5, 1e-7)
    near(ll, rll, 4e-6 * np.abs(rll), "log-likelihood")   # the library's 2e-6, and as much from factors off by float32 roundings
    # gradients normwise: the circuit's own 1e-5 (of dLL/dA, dLL/dB), carried through linear maps
    for got, ref, name in ((dWa, rdWa, "dWa"), (dx, rdx, "dx"), (dw, rdw, "dweight"), (db, rdb, "dbias")):
        e = np.linalg.norm(get(got) - ref) / np.linalg.norm(ref)
        assert e <= 1e-4, (name, e)
    # the update: the gradient's error (measured above, at most 1e-4 of its norm) grows at most 3.4445-fold a step
    assert np.linalg.norm(get(up) - rup) <= 1e-4 * 3.4445 ** 5 + _orth_tol([QUINTIC] * 5, F, M * k, "f32")
    # a small step along dx raises the log-likelihood by its square, to first order
    eps = 1e-3 / float(np.linalg.norm(rdx))
    y2, _, _ = R.layer_norm(get(x) + eps * get(dx), get(w), get(b))
    q2 = y2.reshape(-1, heads, d)
    f2 = R.linear_attention(q2, q2, q2, get(g), lens, d ** -0.5)[0].reshape(B, slots, F)
    lr2 = [((f2[:, s] @ get(Wa)).reshape(B, M, k), (f2[:, s] @ get(Wb)).reshape(B, k, N)) for s in range(slots)]
    _, ll2 = oracle.forward(circ, p64, B, tokens=cfg["tokens"], lowrank=lr2)
    gain, want = (ll2 - rll).sum(), eps * (rdx * get(dx)).sum()
    assert abs(gain - want) <= 0.05 * abs(want), (gain, want)
