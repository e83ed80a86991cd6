"""Softmax attention and the heads' rotation on the CPU: definitions against differences, frequencies, every refusal of
the calls (host-side checks: nothing reaches a device) and workspace sizes."""
import ctypes as C

import numpy as np
import pytest

import log_space_sum_amd as L
from oracle import ops_oracle as R

P = 4096   # an address that is never read


def _refuses(code, rc):
    assert rc == code, (rc, L.pc_last_error())
    assert L.pc_last_error()


def _slope(f, x, d, h=1e-5):
    return (f(x + h * d) - f(x - h * d)) / (2 * h)


# ---- definitions ---------------------------------------------------------------

@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("norm", [False, True])
def test_rotary_gradients_are_slopes(interleaved, norm):
    rng = np.random.default_rng(1)
    x, dy, w = rng.normal(size=(5, 3, 10)), rng.normal(size=(5, 3, 10)), rng.normal(size=10) + 1
    pos, freq = rng.integers(0, 10 ** 6, 5), L_frequencies(6)
    how = dict(interleaved=interleaved, magnitude=1.2, norm=norm)
    dx, dw = R.rotary_grad(dy, x, pos, freq, w=w, **how)
    d = rng.normal(size=x.shape)
    assert np.isclose((dx * d).sum(), _slope(lambda t: (R.rotary(t, pos, freq, w=w, **how) * dy).sum(), x, d), rtol=1e-7)
    if norm:
        d = rng.normal(size=10)
        assert np.isclose((dw * d).sum(), _slope(lambda t: (R.rotary(x, pos, freq, w=t, **how) * dy).sum(), w, d), rtol=1e-7)


def test_rotary_scores_depend_on_distances():
    rng = np.random.default_rng(2)
    q, k = rng.normal(size=(2, 1, 1, 8))
    f = L_frequencies(8)
    for inter in (False, True):
        s = [(R.rotary(q, [p + 3], f, inter) * R.rotary(k, [p], f, inter)).sum() for p in (0, 17, 9000)]
        np.testing.assert_allclose(s, s[0], rtol=1e-9)


def test_softmax_attention_gradients_are_slopes():
    rng = np.random.default_rng(3)
    cu = [0, 4, 4, 5, 11]
    q, k, v, do = rng.normal(size=(12, 4, 5)), rng.normal(size=(12, 2, 5)), rng.normal(size=(12, 2, 3)), rng.normal(size=(12, 4, 3))
    do[11] = 0   # outside every sequence
    o, lse = R.softmax_attention(q, k, v, cu, 0.6)
    assert not o[11].any()
    grads = R.softmax_attention_grad(do, q, k, v, o, lse, cu, 0.6)
    for i, g in enumerate(grads):
        d = rng.normal(size=g.shape)

        def f(t):
            a = [q, k, v]
            a[i] = t
            return (R.softmax_attention(*a, cu, 0.6)[0] * do).sum()
        assert np.isclose((g * d).sum(), _slope(f, (q, k, v)[i], d), rtol=1e-7)


# ---- frequencies ----------------------------------------------------------------

def L_frequencies(n, *args, **kw):
    return L.rotary_frequencies(n, *args, device="cpu", **kw).numpy()


def test_rotary_frequencies():
    f = L_frequencies(64)
    np.testing.assert_allclose(f, 10000.0 ** (-np.arange(32) / 32), rtol=1e-14)
    np.testing.assert_allclose(L_frequencies(64, scaling="linear", factor=4.0), f / 4, rtol=1e-14)
    g = L_frequencies(64, scaling="base", factor=4.0)
    assert g[0] == 1.0 and np.isclose(g[-1], f[-1] / 4, rtol=1e-12) and (np.diff(g / f) < 0).all()
    h = L_frequencies(64, scaling="parts", factor=4.0, original=8192, low=1, high=32)
    turns = 8192 * f / (2 * np.pi)
    assert (h[turns >= 32] == f[turns >= 32]).all() and (turns < 1).any()
    np.testing.assert_allclose(h[turns <= 1], f[turns <= 1] / 4, rtol=1e-14)
    mid = (turns > 1) & (turns < 32)
    t = (turns[mid] - 1) / 31
    np.testing.assert_allclose(h[mid], f[mid] * (t + (1 - t) / 4), rtol=1e-13)
    assert len(L_frequencies(0)) == 0


@pytest.mark.parametrize("bad", [dict(rotary_dim=7), dict(rotary_dim=-2), dict(base=0.0), dict(base=float("inf")),
                                 dict(scaling="linear", factor=0.0), dict(scaling="parts", factor=2.0),
                                 dict(scaling="parts", factor=2.0, original=100.0, low=3.0, high=3.0),
                                 dict(rotary_dim=2, scaling="base", factor=2.0)])
def test_rotary_frequencies_refuse(bad):
    with pytest.raises(L.PCError):
        L.rotary_frequencies(**{"rotary_dim": 8, "device": "cpu", **bad})


def test_rotary_frequencies_refuse_a_name():
    with pytest.raises(ValueError):
        L.rotary_frequencies(8, scaling="other", device="cpu")


# ---- refusals --------------------------------------------------------------------

def _rotary(**change):
    d = L.pc_rotary(dtype=1, heads=4, kv_heads=2, dim=16, num_tokens=10, rotary_dim=16, norm=1, eps=1e-6, magnitude=1.0,
                    positions=P, freq=P, d_q_weight=P, d_k_weight=P)
    for n, h, at in (("q", 4, 0), ("k", 2, 0), ("q_out", 4, 1 << 20), ("k_out", 2, 1 << 20), ("d_q_out", 4, 0), ("d_k_out", 2, 0),
                     ("d_q", 4, 1 << 20), ("d_k", 2, 1 << 20)):
        setattr(d, n, L.pc_heads(P + at, h * 16, 16))
    for k, v in change.items():
        setattr(d, k, v)
    return d


ROTARY = [
    (L.PC_ERR_UNSUPPORTED, dict(dtype=3)), (L.PC_ERR_INVALID_ARG, dict(num_tokens=-1)), (L.PC_ERR_INVALID_ARG, dict(heads=-1)),
    (L.PC_ERR_INVALID_ARG, dict(kv_heads=70000)), (L.PC_ERR_INVALID_ARG, dict(dim=0)), (L.PC_ERR_UNSUPPORTED, dict(dim=257)),
    (L.PC_ERR_INVALID_ARG, dict(rotary_dim=15)), (L.PC_ERR_INVALID_ARG, dict(rotary_dim=18)), (L.PC_ERR_INVALID_ARG, dict(interleaved=2)),
    (L.PC_ERR_INVALID_ARG, dict(norm=-1)), (L.PC_ERR_INVALID_ARG, dict(eps=-1.0)), (L.PC_ERR_INVALID_ARG, dict(eps=float("nan"))),
    (L.PC_ERR_INVALID_ARG, dict(magnitude=float("inf"))), (L.PC_ERR_INVALID_ARG, dict(positions=None)), (L.PC_ERR_INVALID_ARG, dict(freq=None)),
]


@pytest.mark.parametrize("code,change", ROTARY + [(L.PC_ERR_INVALID_ARG, dict(q=L.pc_heads(None, 64, 16))),
                                                  (L.PC_ERR_INVALID_ARG, dict(k=L.pc_heads(P, -1, 16))),
                                                  (L.PC_ERR_INVALID_ARG, dict(q_out=L.pc_heads(P + 64, 63, 16))),
                                                  (L.PC_ERR_INVALID_ARG, dict(q_out=L.pc_heads(P, 128, 16))),
                                                  (L.PC_ERR_INVALID_ARG, dict(k_out=L.pc_heads(None, 32, 16)))])
def test_rotary_forward_refuses(code, change):
    _refuses(code, L.lib().pc_rotary_forward(0, C.byref(_rotary(**change)), None))


@pytest.mark.parametrize("code,change", ROTARY + [(L.PC_ERR_INVALID_ARG, dict(d_q_out=L.pc_heads(None, 64, 16))),
                                                  (L.PC_ERR_INVALID_ARG, dict(q=L.pc_heads(None, 64, 16))),
                                                  (L.PC_ERR_INVALID_ARG, dict(d_k=L.pc_heads(P + 64, 32, 15))),
                                                  (L.PC_ERR_INVALID_ARG, dict(d_q=L.pc_heads(P, 128, 16)))])
def test_rotary_backward_refuses(code, change):
    _refuses(code, L.lib().pc_rotary_backward(0, C.byref(_rotary(**change)), P, 1 << 30, None))


def test_rotary_workspace():
    n = C.c_size_t()
    assert L.lib().pc_rotary_workspace_bytes(C.byref(_rotary()), C.byref(n)) == L.PC_OK and n.value > 0
    _refuses(L.PC_ERR_WORKSPACE, L.lib().pc_rotary_backward(0, C.byref(_rotary()), P, n.value - 1, None))
    _refuses(L.PC_ERR_WORKSPACE, L.lib().pc_rotary_backward(0, C.byref(_rotary()), None, n.value, None))
    _refuses(L.PC_ERR_INVALID_ARG, L.lib().pc_rotary_backward(0, C.byref(_rotary()), P + 8, n.value, None))
    assert L.lib().pc_rotary_workspace_bytes(C.byref(_rotary(num_tokens=1 << 20, dim=256, rotary_dim=256)), C.byref(n)) == L.PC_OK
    assert n.value < (1 << 20) * 256 * 6 * 2 // 64
    _refuses(L.PC_ERR_INVALID_ARG, L.lib().pc_rotary_workspace_bytes(None, C.byref(n)))
    _refuses(L.PC_ERR_NO_DEVICE, L.lib().pc_rotary_forward(-1, C.byref(_rotary()), None))
    # nothing to do reaches no device
    none = _rotary(num_tokens=0, d_q_weight=None, d_k_weight=None)
    assert L.lib().pc_rotary_forward(0, C.byref(none), None) == L.PC_OK
    assert L.lib().pc_rotary_backward(0, C.byref(none), None, 0, None) == L.PC_OK


def test_rotary_of_no_heads_reads_nothing_of_them():
    """What is said of heads that are not there is no error: null pointers at any strides."""
    some, other = L.pc_heads(None, 32, 16), L.pc_heads(None, 0, 0)
    none = _rotary(heads=0, kv_heads=0, norm=0, d_q_weight=None, d_k_weight=None, q=some, k=some, q_out=other, k_out=other, d_q_out=some,
                   d_k_out=some, d_q=other, d_k=other)
    assert L.lib().pc_rotary_forward(0, C.byref(none), None) == L.PC_OK, L.pc_last_error()
    assert L.lib().pc_rotary_backward(0, C.byref(none), None, 0, None) == L.PC_OK, L.pc_last_error()


def _attention(**change):
    d = L.pc_attention(dtype=1, heads=4, kv_heads=2, dim_k=16, dim_v=24, num_seqs=2, num_tokens=10, cu_seqlens=P, scale=0.25, lse=P,
                       num_pages=8, page_size=5, max_pages=3, page_table=P, page_table_stride=3, cached=P, max_seqlen=10, max_length=15)
    for n, h, w in (("q", 4, 16), ("k", 2, 16), ("v", 2, 24), ("o", 4, 24), ("d_o", 4, 24), ("d_q", 4, 16), ("d_k", 2, 16),
                    ("d_v", 2, 24)):
        setattr(d, n, L.pc_heads(P, h * w, w))
    d.k_cache, d.v_cache = L.pc_pages(P, 160, 32, 16), L.pc_pages(P, 240, 48, 24)
    for k, v in change.items():
        setattr(d, k, v)
    return d


BOTH = [
    (L.PC_ERR_UNSUPPORTED, dict(dtype=7)), (L.PC_ERR_INVALID_ARG, dict(heads=0)), (L.PC_ERR_INVALID_ARG, dict(kv_heads=3)),
    (L.PC_ERR_INVALID_ARG, dict(heads=65536, kv_heads=1)), (L.PC_ERR_INVALID_ARG, dict(dim_k=0)), (L.PC_ERR_UNSUPPORTED, dict(dim_k=129)),
    (L.PC_ERR_UNSUPPORTED, dict(dim_v=256)), (L.PC_ERR_INVALID_ARG, dict(num_tokens=-1)), (L.PC_ERR_INVALID_ARG, dict(num_tokens=2 ** 31)),
    (L.PC_ERR_INVALID_ARG, dict(num_seqs=-1)), (L.PC_ERR_INVALID_ARG, dict(num_seqs=1 << 25)), (L.PC_ERR_INVALID_ARG, dict(cu_seqlens=None)),
    (L.PC_ERR_INVALID_ARG, dict(scale=0.0)), (L.PC_ERR_INVALID_ARG, dict(scale=float("inf"))), (L.PC_ERR_INVALID_ARG, dict(scale=float("nan"))),
    (L.PC_ERR_INVALID_ARG, dict(q=L.pc_heads(None, 64, 16))), (L.PC_ERR_INVALID_ARG, dict(k=L.pc_heads(P, -1, 16))),
    (L.PC_ERR_INVALID_ARG, dict(v=L.pc_heads(P, 48, -1))),
]
OUT = [(L.PC_ERR_INVALID_ARG, dict(o=L.pc_heads(P, 95, 24))), (L.PC_ERR_INVALID_ARG, dict(o=L.pc_heads(P, 96, 23))),
       (L.PC_ERR_INVALID_ARG, dict(o=L.pc_heads(None, 96, 24)))]


@pytest.mark.parametrize("code,change", BOTH + OUT)
def test_attention_forward_refuses(code, change):
    _refuses(code, L.lib().pc_attention_forward(0, C.byref(_attention(**change)), P, 1 << 40, None))


@pytest.mark.parametrize("code,change", BOTH + [(L.PC_ERR_INVALID_ARG, dict(d_o=L.pc_heads(None, 96, 24))),
                                                (L.PC_ERR_INVALID_ARG, dict(o=L.pc_heads(None, 96, 24))),
                                                (L.PC_ERR_INVALID_ARG, dict(lse=None)),
                                                (L.PC_ERR_INVALID_ARG, dict(d_q=L.pc_heads(P, 0, 0))),
                                                (L.PC_ERR_INVALID_ARG, dict(d_k=L.pc_heads(P, 32, 15))),
                                                (L.PC_ERR_INVALID_ARG, dict(d_v=L.pc_heads(P, 0, 24)))])
def test_attention_backward_refuses(code, change):
    _refuses(code, L.lib().pc_attention_backward(0, C.byref(_attention(**change)), P, 1 << 40, None))


@pytest.mark.parametrize("code,change", BOTH + OUT + [
    (L.PC_ERR_INVALID_ARG, dict(page_size=0)), (L.PC_ERR_INVALID_ARG, dict(num_pages=-1)), (L.PC_ERR_INVALID_ARG, dict(max_pages=-1)),
    (L.PC_ERR_INVALID_ARG, dict(max_pages=1 << 20, page_size=1 << 11)), (L.PC_ERR_INVALID_ARG, dict(max_seqlen=-1)),
    (L.PC_ERR_INVALID_ARG, dict(max_length=-1)), (L.PC_ERR_INVALID_ARG, dict(cached=None)), (L.PC_ERR_INVALID_ARG, dict(page_table=None)),
    (L.PC_ERR_INVALID_ARG, dict(page_table_stride=2)), (L.PC_ERR_INVALID_ARG, dict(k_cache=L.pc_pages(None, 160, 32, 16))),
    (L.PC_ERR_INVALID_ARG, dict(k_cache=L.pc_pages(P, 159, 32, 16))), (L.PC_ERR_INVALID_ARG, dict(v_cache=L.pc_pages(P, 240, 40, 24))),
    (L.PC_ERR_INVALID_ARG, dict(v_cache=L.pc_pages(P, 240, -48, 24))), (L.PC_ERR_INVALID_ARG, dict(k_cache=L.pc_pages(P, 160, 32, 15))),
])
def test_attention_cached_refuses(code, change):
    _refuses(code, L.lib().pc_attention_cached(0, C.byref(_attention(**change)), P, 1 << 40, None))


def test_attention_takes_what_is_documented():
    """Nothing to do reaches no device: no sequences, no tokens; head-major and token-major caches."""
    f = L.lib()
    for none in (dict(num_seqs=0), dict(num_tokens=0)):
        for k in (L.pc_pages(P, 160, 32, 16), L.pc_pages(P, 160, 16, 80), L.pc_pages(P, 16, 256, 128)):
            d = _attention(k_cache=k, **none)
            assert f.pc_attention_cached(0, C.byref(d), P, 1 << 40, None) == L.PC_OK, L.pc_last_error()
        assert f.pc_attention_forward(0, C.byref(d), None, 0, None) == L.PC_OK
        assert f.pc_attention_backward(0, C.byref(d), P, 1 << 20, None) == L.PC_OK
    _refuses(L.PC_ERR_NO_DEVICE, f.pc_attention_forward(-1, C.byref(_attention()), None, 0, None))
    _refuses(L.PC_ERR_INVALID_ARG, f.pc_attention_forward(0, None, None, 0, None))


def test_attention_workspaces():
    n, f = C.c_size_t(), L.lib()
    assert f.pc_attention_workspace_bytes(C.byref(_attention()), 0, C.byref(n)) == L.PC_OK and n.value == 0
    assert f.pc_attention_workspace_bytes(C.byref(_attention()), 1, C.byref(n)) == L.PC_OK and n.value >= 10 * 4 * 4
    _refuses(L.PC_ERR_WORKSPACE, f.pc_attention_backward(0, C.byref(_attention()), P, n.value - 1, None))
    _refuses(L.PC_ERR_INVALID_ARG, f.pc_attention_backward(0, C.byref(_attention()), P + 4, n.value, None))
    # a short cache is not cut; a long one of few streams is, into parts whose results stay a small share of what is read
    assert f.pc_attention_cached_workspace_bytes(C.byref(_attention()), C.byref(n)) == L.PC_OK and n.value == 0
    long = _attention(num_seqs=1, num_tokens=1, max_seqlen=1, max_pages=1 << 14, page_table_stride=1 << 14, page_size=16, max_length=1 << 18,
                      k_cache=L.pc_pages(P, 512, 32, 16), v_cache=L.pc_pages(P, 768, 48, 24))
    assert f.pc_attention_cached_workspace_bytes(C.byref(long), C.byref(n)) == L.PC_OK
    assert 0 < n.value < (1 << 18) * 2 * 40 * 2 // 64
    _refuses(L.PC_ERR_WORKSPACE, f.pc_attention_cached(0, C.byref(long), P, n.value - 1, None))
    _refuses(L.PC_ERR_INVALID_ARG, f.pc_attention_cached_workspace_bytes(None, C.byref(n)))


@pytest.mark.parametrize("call", ["forward", "backward", "cached"])
def test_attention_workspaces_are_of_one_shape(call):
    """Sizes do not grow with the shapes: few rows are cut into parts, many are not.  What is asked for a call is what it takes: a
    byte less is refused, whichever shape it was made for."""
    f, n = L.lib(), C.c_size_t()

    def bytes_of(d):
        rc = (f.pc_attention_cached_workspace_bytes(C.byref(d), C.byref(n)) if call == "cached"
              else f.pc_attention_workspace_bytes(C.byref(d), int(call == "backward"), C.byref(n)))
        assert rc == L.PC_OK
        return n.value

    def shape(tokens, seqs):
        pages = 4096
        return _attention(num_tokens=tokens, num_seqs=seqs, max_seqlen=tokens // seqs, max_pages=pages, page_table_stride=pages, page_size=16,
                          max_length=pages * 16, k_cache=L.pc_pages(P, 512, 32, 16), v_cache=L.pc_pages(P, 768, 48, 24))
    shapes = [(1, 1), (64, 1), (512, 1), (700, 1), (2048, 1), (2048, 2), (4096, 1), (64, 64), (512, 64), (16384, 1), (65536, 8)]
    sizes = [bytes_of(shape(*x)) for x in shapes]
    assert any(a > b for a, b in zip(sizes, sizes[1:]))
    assert sizes == [bytes_of(shape(*x)) for x in shapes]
    run = getattr(f, "pc_attention_" + call)
    for x, size in zip(shapes, sizes):
        if size:
            _refuses(L.PC_ERR_WORKSPACE, run(0, C.byref(shape(*x)), P, size - 1, None))


@pytest.mark.parametrize("size", [1, 2, 3, 5, 7, 16, 24, 100, 1000, 65536, 65537, 2 ** 31 - 1])
def test_the_division_by_a_page_size(size):
    """What the kernels divide positions by: j magic >> (31 + s) with s = ceil(log2 size)."""
    s = (size - 1).bit_length()
    magic = -(-(1 << (31 + s)) // size)
    assert magic < 1 << 32
    rng = np.random.default_rng(size % 1000)
    j = np.unique(np.concatenate([np.arange(300), rng.integers(0, 2 ** 31 - 1, 2000), 2 ** 31 - 1 - np.arange(300),
                                  np.minimum(size * rng.integers(0, max(1, (2 ** 31 - 2) // size) + 1, 2000), 2 ** 31 - 1)]))
    for x in j.tolist():
        assert x * magic >> (31 + s) == x // size
        assert x * magic < 1 << 64
