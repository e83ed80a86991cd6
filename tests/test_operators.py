"""The operators in front of a conditional circuit on the CPU: the float64 definitions against differences and
against each other, and every refusal of the C ABI (refused before any device work)."""
import ctypes as C
import re

import numpy as np
import pytest

import log_space_sum_amd as L
from oracle import ops_oracle as R


def _difference(f, x, d, h=1e-6):
    return (f(x + h * d) - f(x - h * d)) / (2 * h)


def test_layer_norm_gradient_is_the_difference():
    rng = np.random.default_rng(0)
    x, dy, w, b = rng.normal(size=(5, 7)), rng.normal(size=(5, 7)), rng.normal(size=7), rng.normal(size=7)
    _, mean, rstd = R.layer_norm(x, w, b)
    dx, dw, db = R.layer_norm_grad(dy, x, mean, rstd, w)
    for value, grad, f in ((x, dx, lambda z: (R.layer_norm(z, w, b)[0] * dy).sum()),
                           (w, dw, lambda z: (R.layer_norm(x, z, b)[0] * dy).sum()),
                           (b, db, lambda z: (R.layer_norm(x, w, z)[0] * dy).sum())):
        d = rng.normal(size=value.shape)
        # central differences: truncation h^2, rounding eps / h
        np.testing.assert_allclose((grad * d).sum(), _difference(f, value, d), rtol=1e-7, atol=1e-7)


def test_linear_attention_gradient_is_the_difference():
    rng = np.random.default_rng(1)
    cu = [0, 3, 3, 4, 9]
    q, k, v = rng.normal(size=(9, 4, 3)), rng.normal(size=(9, 2, 3)), rng.normal(size=(9, 2, 5))
    g, s = -np.array([0.0, 0.1, 1.0, np.inf]), rng.normal(size=(4, 4, 3, 5))
    do, ds = rng.normal(size=(9, 4, 5)), rng.normal(size=(4, 4, 3, 5))

    def loss(q, k, v, s):
        o, e = R.linear_attention(q, k, v, g, cu, 0.7, s)
        return (o * do).sum() + (e * ds).sum()

    grads = R.linear_attention_grad(do, q, k, v, g, cu, 0.7, s, ds)
    args = [q, k, v, s]
    for i, grad in enumerate(grads):
        d = rng.normal(size=args[i].shape)
        f = lambda z: loss(*[z if j == i else a for j, a in enumerate(args)])  # noqa: E731
        np.testing.assert_allclose((grad * d).sum(), _difference(f, args[i], d), rtol=1e-6, atol=1e-6)


def test_orthogonalize_moves_the_singular_values():
    rng = np.random.default_rng(2)
    g = rng.normal(size=(6, 4))
    co = [(3.4445, -4.7750, 2.0315)] * 5
    x = R.orthogonalize(g, co, 0.0)
    u, s, vt = np.linalg.svd(g, full_matrices=False)
    t = s / np.sqrt((s * s).sum())
    for a, b, c in co:
        t = a * t + b * t ** 3 + c * t ** 5
    np.testing.assert_allclose(x, (u * t) @ vt, rtol=1e-10, atol=1e-12)


def _rounded_steps(g, planes, steps=5):
    """Newton-Schulz steps in float32 whose operands are `planes` float16 planes of a scaled value."""
    scale = np.float32(2.0 ** 13)

    def product(a, b):
        hi, lo = [], []
        for x in (a, b):
            x = x * scale
            h = x.astype(np.float16).astype(np.float32)
            hi.append(h)
            lo.append((x - h).astype(np.float16).astype(np.float32) if planes == 2 else 0 * h)
        return (hi[0] @ lo[1] + lo[0] @ hi[1] + hi[0] @ hi[1]) / (scale * scale)

    x = (g / np.linalg.norm(g)).astype(np.float32)
    a, b, c = (np.float32(v) for v in (3.4445, -4.7750, 2.0315))
    for _ in range(steps):
        A = product(x, x.T)
        x = product(a * np.eye(len(A), dtype=np.float32) + b * A + c * product(A, A), x)
    return x.astype(np.float64)


@pytest.mark.parametrize("m,n", [(65, 65), (70, 400), (129, 300), (333, 1000)])
def test_the_bounds_of_the_update_tell_one_plane_from_two(m, n):
    """2e-5 of the result normwise and 24 times that of its root mean square for an element (what the GPU tests allow a
    float32 result): two planes stay ten times below, one plane is far beyond both."""
    g = np.random.default_rng(m).normal(size=(m, n))
    ref = R.orthogonalize(g, [(3.4445, -4.7750, 2.0315)] * 5, 0.0)
    size, rms = np.linalg.norm(ref), np.sqrt((ref * ref).mean())
    two, one = (_rounded_steps(g, p) - ref for p in (2, 1))
    assert np.linalg.norm(two) <= 4e-6 * size and np.abs(two).max() <= 24 * 4e-6 * rms
    assert np.linalg.norm(one) > 20 * 2e-5 * size and np.abs(one).max() > 5 * 24 * 2e-5 * rms


# ---- refusals: host-side checks, nothing reaches a device -------------------

P = 4096   # an address that is never read
FLOATS = (C.c_float * 96)(*([3.4445, -4.7750, 2.0315] * 32))


def _refuses(code, rc):
    assert rc == code, (rc, L.pc_last_error())
    assert L.pc_last_error()


NORM = dict(device=0, dtype=0, rows=4, cols=8, x=P, xs=8, w=None, b=None, eps=1e-5, y=P, ys=8, mean=None, rstd=None)


@pytest.mark.parametrize("code,change", [
    (L.PC_ERR_NO_DEVICE, dict(device=-1)), (L.PC_ERR_UNSUPPORTED, dict(dtype=3)),
    (L.PC_ERR_INVALID_ARG, dict(rows=-1)), (L.PC_ERR_INVALID_ARG, dict(rows=2 ** 31)),
    (L.PC_ERR_INVALID_ARG, dict(cols=0)), (L.PC_ERR_UNSUPPORTED, dict(cols=16385, xs=16385, ys=16385)),
    (L.PC_ERR_INVALID_ARG, dict(x=None)), (L.PC_ERR_INVALID_ARG, dict(y=None)),
    (L.PC_ERR_INVALID_ARG, dict(xs=7)), (L.PC_ERR_INVALID_ARG, dict(ys=7)),
    (L.PC_ERR_INVALID_ARG, dict(eps=-1.0)), (L.PC_ERR_INVALID_ARG, dict(eps=float("nan"))),
])
def test_layer_norm_forward_refuses(code, change):
    a = {**NORM, **change}
    _refuses(code, L.lib().pc_layer_norm_forward(a["device"], a["dtype"], a["rows"], a["cols"], a["x"], a["xs"], a["w"],
                                                 a["b"], a["eps"], a["y"], a["ys"], a["mean"], a["rstd"], None))


def _norm_ws(rows, cols):
    n = C.c_size_t()
    assert L.lib().pc_layer_norm_workspace_bytes(rows, cols, C.byref(n)) == L.PC_OK
    return n.value


NBWD = dict(device=0, dtype=1, rows=4, cols=8, dy=P, dys=8, x=P, xs=8, w=None, mean=P, rstd=P, dx=P, dxs=8, dw=P, db=P,
            ws=P, nws=1 << 30)


@pytest.mark.parametrize("code,change", [
    (L.PC_ERR_INVALID_ARG, dict(dy=None)), (L.PC_ERR_INVALID_ARG, dict(mean=None)), (L.PC_ERR_INVALID_ARG, dict(rstd=None)),
    (L.PC_ERR_INVALID_ARG, dict(dx=None)), (L.PC_ERR_INVALID_ARG, dict(dys=3)), (L.PC_ERR_INVALID_ARG, dict(dxs=3)),
    (L.PC_ERR_WORKSPACE, dict(ws=None)), (L.PC_ERR_WORKSPACE, dict(nws=8)), (L.PC_ERR_INVALID_ARG, dict(ws=P + 4)),
    (L.PC_ERR_UNSUPPORTED, dict(cols=20000)),
])
def test_layer_norm_backward_refuses(code, change):
    a = {**NBWD, **change}
    _refuses(code, L.lib().pc_layer_norm_backward(*[a[k] for k in ("device", "dtype", "rows", "cols", "dy", "dys", "x", "xs",
                                                                   "w", "mean", "rstd", "dx", "dxs", "dw", "db", "ws",
                                                                   "nws")], None))


def test_layer_norm_workspace():
    assert _norm_ws(0, 8) == 0
    assert 0 < _norm_ws(4, 8) <= _norm_ws(4096, 8)
    # the partial sums stay a small part of what the pass moves
    assert _norm_ws(1 << 20, 4096) < (1 << 20) * 4096 * 4 // 64


def _attention(**change):
    d = L.pc_linear_attention(dtype=1, heads=4, kv_heads=2, dim_k=16, dim_v=24, num_seqs=2, num_tokens=10, max_seqlen=10,
                              cu_seqlens=P, log_decay=P, scale=0.25, state=P, num_slots=16)
    for n, h, w in (("q", 4, 16), ("k", 2, 16), ("v", 2, 24), ("o", 4, 24), ("d_o", 4, 24), ("d_q", 4, 16), ("d_k", 2, 16),
                    ("d_v", 2, 24)):
        setattr(d, n, L.pc_heads(P, h * w, w))
    for k, v in change.items():
        setattr(d, k, v)
    return d


BOTH = [
    (L.PC_ERR_UNSUPPORTED, dict(dtype=7)), (L.PC_ERR_INVALID_ARG, dict(heads=0)), (L.PC_ERR_INVALID_ARG, dict(kv_heads=3)),
    (L.PC_ERR_INVALID_ARG, dict(dim_k=0)), (L.PC_ERR_UNSUPPORTED, dict(dim_k=129)), (L.PC_ERR_UNSUPPORTED, dict(dim_v=256)),
    (L.PC_ERR_INVALID_ARG, dict(num_tokens=-1)), (L.PC_ERR_INVALID_ARG, dict(log_decay=None)),
    (L.PC_ERR_INVALID_ARG, dict(scale=0.0)), (L.PC_ERR_INVALID_ARG, dict(scale=float("inf"))),
    (L.PC_ERR_INVALID_ARG, dict(q=L.pc_heads(None, 64, 16))), (L.PC_ERR_INVALID_ARG, dict(k=L.pc_heads(P, -1, 16))),
]
SEQS = [
    (L.PC_ERR_INVALID_ARG, dict(num_seqs=-1)), (L.PC_ERR_UNSUPPORTED, dict(num_seqs=65536)),
    (L.PC_ERR_INVALID_ARG, dict(max_seqlen=-1)), (L.PC_ERR_INVALID_ARG, dict(cu_seqlens=None)),
]


@pytest.mark.parametrize("code,change", BOTH + SEQS + [(L.PC_ERR_INVALID_ARG, dict(o=L.pc_heads(P, 95, 24))),
                                                       (L.PC_ERR_INVALID_ARG, dict(o=L.pc_heads(P, 96, 23)))])
def test_linear_attention_forward_refuses(code, change):
    _refuses(code, L.lib().pc_linear_attention_forward(0, C.byref(_attention(**change)), P, 1 << 40, None))


@pytest.mark.parametrize("code,change", BOTH + SEQS + [(L.PC_ERR_INVALID_ARG, dict(d_o=L.pc_heads(None, 96, 24))),
                                                       (L.PC_ERR_INVALID_ARG, dict(d_q=L.pc_heads(P, 0, 0))),
                                                       (L.PC_ERR_INVALID_ARG, dict(d_k=L.pc_heads(P, 32, 15))),
                                                       (L.PC_ERR_INVALID_ARG, dict(d_v=L.pc_heads(P, 0, 24)))])
def test_linear_attention_backward_refuses(code, change):
    _refuses(code, L.lib().pc_linear_attention_backward(0, C.byref(_attention(**change)), P, 1 << 40, None))


@pytest.mark.parametrize("code,change", BOTH + [(L.PC_ERR_INVALID_ARG, dict(state=None)),
                                                (L.PC_ERR_INVALID_ARG, dict(num_slots=-1)),
                                                (L.PC_ERR_INVALID_ARG, dict(num_slots=9)),   # fewer than rows, no slots
                                                (L.PC_ERR_INVALID_ARG, dict(o=L.pc_heads(P, 20, 24)))])
def test_linear_attention_step_refuses(code, change):
    _refuses(code, L.lib().pc_linear_attention_step(0, C.byref(_attention(**change)), None))


def test_linear_attention_strides_that_are_taken():
    """Rows of single tokens may lie anywhere (positions of a padded batch); chunks of whole sequences hold offsets of
    32 bits.  (No slots, or no sequences: nothing reaches a device.)"""
    far = dict(q=L.pc_heads(P, 1 << 24, 16), k=L.pc_heads(P, 1 << 40, 16), v=L.pc_heads(P, 1 << 30, 24), o=L.pc_heads(P, 1 << 25, 24))
    step, whole = L.lib().pc_linear_attention_step, L.lib().pc_linear_attention_forward
    assert step(0, C.byref(_attention(**far, num_slots=0, slots=P)), None) == L.PC_OK, L.pc_last_error()
    _refuses(L.PC_ERR_UNSUPPORTED, whole(0, C.byref(_attention(**far, num_seqs=0)), P, 1 << 40, None))
    # a single token's stride is not used
    assert whole(0, C.byref(_attention(**far, num_seqs=0, num_tokens=1)), P, 1 << 40, None) == L.PC_OK, L.pc_last_error()
    _refuses(L.PC_ERR_INVALID_ARG, step(0, C.byref(_attention(q=L.pc_heads(P, -1, 16), num_slots=0, slots=P)), None))


def test_linear_attention_workspace():
    n = C.c_size_t()
    f = L.lib().pc_linear_attention_workspace_bytes
    # many heads and short sequences: no split, no workspace; gradients of shared heads are summed from it
    d = _attention(num_seqs=256, num_tokens=256 * 10)
    assert f(C.byref(d), 0, C.byref(n)) == L.PC_OK and n.value == 0
    assert f(C.byref(d), 1, C.byref(n)) == L.PC_OK and n.value >= 2560 * 4 * (16 + 24) * 4
    long = _attention(num_seqs=1, num_tokens=1 << 15, max_seqlen=1 << 15)
    assert f(C.byref(long), 0, C.byref(n)) == L.PC_OK and n.value > 0
    _refuses(L.PC_ERR_WORKSPACE, L.lib().pc_linear_attention_forward(0, C.byref(long), P, n.value - 1, None))
    _refuses(L.PC_ERR_WORKSPACE, L.lib().pc_linear_attention_backward(0, C.byref(long), P, n.value, None))
    _refuses(L.PC_ERR_INVALID_ARG, f(None, 0, C.byref(n)))
    _refuses(L.PC_ERR_INVALID_ARG, f(C.byref(d), 0, None))


@pytest.mark.parametrize("seqs,tokens,heads,dim", [(4096, 512, 16, 128), (1000, 100, 8, 128), (65535, 30, 4, 64), (300, 700, 32, 32)])
@pytest.mark.parametrize("dtype", [0, 1])
def test_linear_attention_workspace_without_a_bound_of_the_lengths(seqs, tokens, heads, dim, dtype):
    """Many sequences whose longest is not given (max_seqlen: all tokens): the segments' states take no more than the
    tokens themselves, for each direction."""
    n, f = C.c_size_t(), L.lib().pc_linear_attention_workspace_bytes
    d = _attention(dtype=dtype, heads=heads, kv_heads=heads, dim_k=dim, dim_v=dim, num_seqs=seqs, num_tokens=seqs * tokens,
                   max_seqlen=seqs * tokens)
    own = 4 * seqs * tokens * heads * dim * (2 if dtype else 4)     # q, k, v, o
    assert f(C.byref(d), 0, C.byref(n)) == L.PC_OK and n.value <= own
    assert f(C.byref(d), 1, C.byref(n)) == L.PC_OK and n.value <= 2 * own


def _segments(lens, total, seglen, nsegs):
    """The packed places of every sequence's segments, as the kernels take them."""
    places, t0 = [], 0
    for n in lens:
        live = min(max(-(-n // seglen), 1), nsegs)
        if live > 1:
            places += [2 * t0 // seglen + s for s in range(live)]
        t0 += n
    assert t0 <= total
    return places


def test_segments_places_are_distinct():
    rng = np.random.default_rng(5)
    for trial in range(400):
        seglen = int(rng.choice([64, 128, 192, 1000]))
        lens = [int(x) for x in rng.choice([0, 1, seglen - 1, seglen, seglen + 1, 2 * seglen, 2 * seglen + 1, 5 * seglen + 3, 7], size=30)]
        total = sum(lens) + int(rng.integers(0, 9))
        for nsegs in (2, 3, 40):
            p = _segments(lens, total, seglen, nsegs)
            assert len(set(p)) == len(p) and all(0 <= x < 2 * total // seglen + 1 for x in p)


ORTH = dict(device=0, dtype=0, batch=2, rows=96, cols=80, g=P, gb=7680, gr=80, out=P, ob=7680, orow=80, steps=5, co=FLOATS,
            eps=1e-7, ws=P, nws=1 << 40)
DIVERGES = (C.c_float * 96)(*([8.0, 0.0, 0.0] * 32))
NOT_FINITE = (C.c_float * 96)(*([3.0, float("nan"), 0.0] * 32))


@pytest.mark.parametrize("code,change", [
    (L.PC_ERR_NO_DEVICE, dict(device=-1)), (L.PC_ERR_UNSUPPORTED, dict(dtype=-1)), (L.PC_ERR_INVALID_ARG, dict(batch=-1)),
    (L.PC_ERR_UNSUPPORTED, dict(batch=65536)), (L.PC_ERR_INVALID_ARG, dict(rows=0)),
    (L.PC_ERR_UNSUPPORTED, dict(rows=32769)), (L.PC_ERR_INVALID_ARG, dict(g=None)), (L.PC_ERR_INVALID_ARG, dict(gr=79)),
    (L.PC_ERR_INVALID_ARG, dict(orow=79)), (L.PC_ERR_INVALID_ARG, dict(ob=7679)), (L.PC_ERR_INVALID_ARG, dict(gb=-1)),
    (L.PC_ERR_INVALID_ARG, dict(steps=0)), (L.PC_ERR_INVALID_ARG, dict(steps=33)), (L.PC_ERR_INVALID_ARG, dict(co=None)),
    (L.PC_ERR_INVALID_ARG, dict(co=DIVERGES)), (L.PC_ERR_INVALID_ARG, dict(co=NOT_FINITE)),
    (L.PC_ERR_INVALID_ARG, dict(eps=-1e-9)), (L.PC_ERR_WORKSPACE, dict(nws=100)), (L.PC_ERR_WORKSPACE, dict(ws=None)),
])
def test_orthogonalize_refuses(code, change):
    a = {**ORTH, **change}
    _refuses(code, L.lib().pc_orthogonalize(*[a[k] for k in ("device", "dtype", "batch", "rows", "cols", "g", "gb", "gr", "out",
                                                             "ob", "orow", "steps", "co", "eps", "ws", "nws")], None))


TUNED = [(8.287, -23.596, 17.300), (4.107, -2.948, 0.545), (3.949, -2.909, 0.552), (3.318, -2.488, 0.510), (2.301, -1.669, 0.419)]


SAFE = [(a / 1.01, b / 1.01 ** 3, c / 1.01 ** 5) for a, b, c in TUNED[:-1]] + TUNED[-1:]
POLAR = (1.875, -1.25, 0.375)


def _largest(triples):
    """The largest singular value that steps from [0, 1] reach: the image of an interval from 0 is one (up to the sign)."""
    x, top = 1.0, 0.0
    for a, b, c in triples:
        z = np.linspace(0, x, 200001)
        x = np.abs(a * z + b * z ** 3 + c * z ** 5).max()
        top = max(top, x)
        if top > 1e6:
            break
    return top


@pytest.mark.parametrize("triples,accepted", [
    (TUNED, True),                                                              # each tuned for the interval before it
    (SAFE, True), (SAFE + [POLAR] * 20, True),
    (TUNED + [POLAR] * 20, False),                                              # 2.97 after TUNED, which POLAR raises
    ([(1.5, -0.5, 0.0)] * 32, True), ([(3.4445, -4.7750, 2.0315)] * 32, True),
    ([(3.9, 0.0, 0.0)] * 5, True), ([(4.1, 0.0, 0.0)] * 5, False), ([(1.6, 0.2, 0.0)] * 12, False),
    (TUNED[:1] * 5, False)])
def test_orthogonalize_takes_the_schedules_that_stay_bounded(triples, accepted):
    """A schedule is refused where singular values from [0, 1] can pass 1024, and only there; one that is taken is
    refused here for its missing workspace, before any device work."""
    assert (_largest(triples) <= 1024) == accepted
    flat = (C.c_float * (3 * len(triples)))(*[v for t in triples for v in t])
    a = {**ORTH, "steps": len(triples), "co": flat, "ws": None, "nws": 0}
    rc = L.lib().pc_orthogonalize(*[a[k] for k in ("device", "dtype", "batch", "rows", "cols", "g", "gb", "gr", "out", "ob",
                                                   "orow", "steps", "co", "eps", "ws", "nws")], None)
    assert rc == (L.PC_ERR_WORKSPACE if accepted else L.PC_ERR_INVALID_ARG), L.pc_last_error()


def test_calls_in_place_keep_the_strides():
    """An output that is the input at other strides would be overwritten while it is read."""
    a = {**NORM, "ys": 9}
    fwd = lambda a: L.lib().pc_layer_norm_forward(*[a[k] for k in ("device", "dtype", "rows", "cols", "x", "xs", "w", "b", "eps", "y",  # noqa: E731
                                                                   "ys", "mean", "rstd")], None)
    _refuses(L.PC_ERR_INVALID_ARG, fwd(a))
    for change in (dict(dxs=9, dys=9), dict(dxs=9, xs=9), dict(dxs=9, x=2 * P)):
        a = {**NBWD, **change}
        _refuses(L.PC_ERR_INVALID_ARG, L.lib().pc_layer_norm_backward(*[a[k] for k in ("device", "dtype", "rows", "cols", "dy", "dys",
                                                                                       "x", "xs", "w", "mean", "rstd", "dx", "dxs", "dw",
                                                                                       "db", "ws", "nws")], None))
    for change in (dict(orow=81, ob=8000), dict(ob=7681), dict(batch=1, orow=81), dict(rows=1, batch=2, ob=90, gb=80)):
        a = {**ORTH, **change}
        _refuses(L.PC_ERR_INVALID_ARG, L.lib().pc_orthogonalize(*[a[k] for k in ("device", "dtype", "batch", "rows", "cols", "g", "gb",
                                                                                 "gr", "out", "ob", "orow", "steps", "co", "eps", "ws",
                                                                                 "nws")], None))


def test_binding_refuses_host_tensors_and_wrong_shapes():
    torch = pytest.importorskip("torch")
    x = torch.zeros(3, 4)
    with pytest.raises(ValueError, match="GPU"):
        L.pc_layer_norm_forward(x, None, None, torch.empty_like(x))
    with pytest.raises(ValueError, match="two dimensions"):
        L.pc_layer_norm_forward(x[0], None, None, x[0])
    q = torch.zeros(5, 2, 4)
    with pytest.raises(ValueError, match="GPU"):
        L.pc_linear_attention_forward(q, q, q, None, q)
    with pytest.raises(ValueError, match="three dimensions"):
        L.pc_linear_attention_step(q[0], q, q, None, q, q)
    with pytest.raises(ValueError, match="dimensions"):
        L.pc_orthogonalize(x[0], x[0])


@pytest.mark.parametrize("load", ["global_load_lds_dwordx4", "global_load_lds_dword "])
def test_ring_loads_wait_for_their_base(load):
    """Inline assembly gets no wait states from the compiler: five between the VALU's write of the base's scalar
    registers, which may be the instruction in front, and the vector load that reads them."""
    import pathlib
    text = (pathlib.Path(L.__file__).parent / "csrc" / "pc_ring.h").read_text()
    found = [a for a in re.findall(r'asm volatile\("([^"]*)"', text) if load in a]
    assert len(found) == 1
    before = found[0].replace("\\t", "").split("\\n")
    at = next(i for i, op in enumerate(before) if op.startswith(load))
    assert sum(int(op.split()[1]) + 1 if op.startswith("s_nop") else 1 for op in before[:at]) >= 5
