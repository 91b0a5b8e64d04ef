"""The sequence operators without a GPU: their fp64 definitions against
differences and closed forms, and the argument checks of their entry points."""
import ctypes

import numpy as np
import pytest

from oracle import sequence_ops as S
from test_rnn_layer_b200 import build as B
from test_rnn_layer_b200 import tttmlp as L

RNG = np.random.default_rng


# ---------------------------------------------------------------- definitions
def _differences(loss, arrays, h=1e-5):
    out = []
    for a in arrays:
        g = np.zeros_like(a)
        for i in np.ndindex(a.shape):
            keep = a[i]
            a[i] = keep + h
            up = loss()
            a[i] = keep - h
            g[i] = (up - loss()) / (2 * h)
            a[i] = keep
        out.append(g)
    return out


@pytest.mark.parametrize("left,right,sinks", [(3, 0, 0), (1, 0, 2), (2, 2, 1), (99, 0, 0), (0, 0, 0)])
def test_window_gradient_equals_differences(left, right, sinks):
    r = RNG(0)
    cu_q, cu_k = [0, 4, 4, 9], [0, 6, 8, 11]      # cached prefix, no queries, fewer keys than queries
    q, k, v, g = r.normal(size=(9, 2, 3)), r.normal(size=(11, 1, 3)), r.normal(size=(11, 1, 3)), r.normal(size=(9, 2, 3))

    def loss():
        return float((S.window_attention(q, k, v, left, right, sinks, cu_q, cu_k)["out"] * g).sum())

    ref = S.window_attention(q, k, v, left, right, sinks, cu_q, cu_k, grad_out=g)
    for name, d in zip(("dq", "dk", "dv"), _differences(loss, (q, k, v))):
        assert np.abs(ref[name] - d).max() < 1e-8, name


def test_window_rows_that_see_nothing():
    r = RNG(1)
    q, k, v = r.normal(size=(5, 1, 3)), r.normal(size=(2, 1, 3)), r.normal(size=(2, 1, 3))
    ref = S.window_attention(q, k, v, 10, 0, 0, grad_out=np.ones_like(q))
    assert np.all(ref["out"][:3] == 0) and np.all(np.isneginf(ref["lse"][0, :3])) and np.all(ref["dq"][:3] == 0)
    assert np.allclose(ref["out"][3, 0], v[0, 0])


@pytest.mark.parametrize("form", ["sum", "convex", "unit"])
@pytest.mark.parametrize("reverse", [False, True])
def test_scan_gradient_equals_differences(form, reverse):
    r = RNG(2)
    cu = [0, 5, 5, 6, 9]
    f, x, h0 = r.normal(size=(9, 2)), r.normal(size=(9, 2)), r.normal(size=(4, 2))
    gy, gh = r.normal(size=(9, 2)), r.normal(size=(4, 2))

    def loss():
        o = S.gated_scan(f, x, form, reverse, cu, h0)
        return float((o["y"] * gy).sum() + (o["hT"] * gh).sum())

    ref = S.gated_scan(f, x, form, reverse, cu, h0, gy, gh)
    for name, d in zip(("df", "dx", "dh0"), _differences(loss, (f, x, h0))):
        assert np.abs(ref[name] - d).max() < 1e-8, name


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_rope_keeps_relative_angles_and_its_inverse_is_the_transpose(layout):
    r = RNG(3)
    q, k = r.normal(size=(1, 1, 8)), r.normal(size=(1, 1, 8))

    def score(pq, pk):
        a, b = S.rope(q, [pq], 6, layout)[0], S.rope(k, [pk], 6, layout)[0]
        return float((a * b).sum())

    assert abs(score(7, 3) - score(1007, 1003)) < 1e-9
    sc = {"kind": "ramp", "factor": 8.0, "length": 64, "low": 1.0, "high": 4.0, "amplitude": 1.5}
    y, g = S.rope(q, [11], 6, layout, scaling=sc)[0], r.normal(size=(1, 1, 8))
    back = S.rope(g, [11], 6, layout, scaling=sc, inverse=True)[0]
    assert abs((y * g).sum() - (q * back).sum()) < 1e-12


# ---------------------------------------------------------------- refusals
@pytest.fixture(scope="module")
def no_gpu():
    """Fake device addresses are only passed where no GPU exists; every call below is refused before its use."""
    import torch
    if torch.cuda.is_available():
        pytest.skip("fake device addresses are only used where no GPU exists")
    B.build()


A = 0x10000000     # 16- and 256-byte aligned fake addresses, 256 MB apart
P = [A * (i + 1) for i in range(12)]


def _rope(**kw):
    q = dict(T=16, H=2, d=64, rot=64, layout=0, x_dtype=L.TTT_BF16, scaling=0, base=1e4, factor=1.0, length=0.0, low=0.0,
             high=0.0, amplitude=1.0)
    c = dict(X=P[0], ld_x=128, Y=P[1], ld_y=128, pos=None)
    for k, v in kw.items():
        (q if k in q else c)[k] = v
    return L.ttt_rope(L.ttt_rope_desc(*q.values()), c["X"], c["ld_x"], c["Y"], c["ld_y"], c["pos"], 0, 0, 0)


@pytest.mark.parametrize("bad", [
    dict(T=-1), dict(H=0), dict(d=60), dict(d=0), dict(rot=3), dict(rot=0), dict(rot=66), dict(layout=2), dict(x_dtype=2),
    dict(scaling=4), dict(base=1.0), dict(base=float("nan")), dict(scaling=1, factor=0.5), dict(scaling=1, factor=float("inf")),
    dict(scaling=2, factor=2.0, rot=2), dict(scaling=3, factor=2.0), dict(scaling=3, factor=2.0, length=64.0, low=2.0, high=2.0),
    dict(amplitude=float("inf")), dict(X=None), dict(Y=None), dict(X=P[0] + 8), dict(ld_x=120), dict(ld_x=132), dict(ld_y=64),
    dict(pos=P[2] + 2), dict(Y=P[0] + 64), dict(Y=P[0], ld_y=256)])
def test_rope_refusals(no_gpu, bad):
    assert _rope(**bad) == L.TTT_ERR_INVALID_ARG and L.ttt_last_error()


def test_rope_accepts_an_empty_call_and_refuses_wide_heads(no_gpu):
    assert _rope(T=0, X=None, Y=None) == L.TTT_OK
    assert _rope(d=264, ld_x=528, ld_y=528) == L.TTT_ERR_UNSUPPORTED


def _window(backward=False, **kw):
    q = dict(Tq=100, Tk=120, n_seq=1, Hq=4, Hk=2, d=64, left=10, right=0, sinks=2, scale=0.125)
    c = dict(cu_q=None, cu_k=None, Q=P[0], ld_q=256, K=P[1], ld_k=128, V=P[2], ld_v=128, Xres=None, Out=P[3], ld_out=256,
             Lse=P[4], dOut=P[5], ld_do=256, dQ=P[6], ld_dq=256, dK=P[7], ld_dk=128, dV=P[8], ld_dv=128, ws=P[9], n=1 << 20)
    for k, v in kw.items():
        (q if k in q else c)[k] = v
    d = L.ttt_window_desc(*q.values())
    a = [c[k] for k in ("cu_q", "cu_k", "Q", "ld_q", "K", "ld_k", "V", "ld_v")]
    if backward:
        a += [c[k] for k in ("Out", "ld_out", "Lse", "dOut", "ld_do", "dQ", "ld_dq", "dK", "ld_dk", "dV", "ld_dv", "ws", "n")]
        return L.ttt_window_attention_backward(d, *a, 0)
    return L.ttt_window_attention(d, *a, *[c[k] for k in ("Xres", "Out", "ld_out", "Lse", "ws", "n")], 0)


WINDOW_BAD = [dict(Tq=-1), dict(Tk=-1), dict(Tq=(1 << 30) + 1), dict(n_seq=0), dict(n_seq=2), dict(Hq=3), dict(Hk=0), dict(Hq=0),
              dict(left=-1), dict(right=-1), dict(sinks=-1), dict(scale=0.0), dict(scale=float("nan")), dict(scale=float("inf")),
              dict(cu_q=P[10]), dict(cu_k=P[10]), dict(cu_q=P[10] + 2, cu_k=P[11]), dict(Q=None), dict(K=None), dict(V=P[2] + 8),
              dict(ld_q=248), dict(ld_k=132), dict(Out=None), dict(ws=None), dict(ws=P[9] + 16), dict(n=128)]


@pytest.mark.parametrize("bad", WINDOW_BAD + [dict(Xres=P[3] + 2), dict(Lse=P[4] + 4), dict(Out=P[0]), dict(Out=P[1] + 512)])
def test_window_refusals(no_gpu, bad):
    assert _window(**bad) == L.TTT_ERR_INVALID_ARG and L.ttt_last_error()


@pytest.mark.parametrize("bad", WINDOW_BAD + [dict(Lse=None), dict(dOut=None), dict(dQ=None), dict(dK=P[7] + 4), dict(ld_dv=64),
                                              dict(dQ=P[0]), dict(dK=P[1]), dict(dV=P[7]), dict(n=1024)])
def test_window_backward_refusals(no_gpu, bad):
    assert _window(True, **bad) == L.TTT_ERR_INVALID_ARG and L.ttt_last_error()


def test_window_unsupported_head_dim_and_sizes(no_gpu):
    assert _window(d=128) == L.TTT_ERR_UNSUPPORTED and _window(True, d=32) == L.TTT_ERR_UNSUPPORTED
    d = L.ttt_window_desc(100, 120, 1, 4, 2, 64, 10, 0, 2, 0.125)
    assert L.ttt_window_attention_workspace_size(d) >= 16 and L.ttt_window_attention_backward_workspace_size(d) >= 1600
    d.Hq = 3
    assert L.ttt_window_attention_workspace_size(d) == 0 and L.ttt_last_error()


def _decode(**kw):
    q = dict(B=3, Hq=4, Hk=2, d=64, slots=32, left=20, sinks=4, scale=0.125, ld_request=4096, ld_slot=128, ld_head=64)
    c = dict(Q=P[0], ld_q=256, K_new=P[1], V_new=P[2], ld_new=128, K=P[3], V=P[4], lens=P[5], Out=P[6], ld_out=256, ws=P[7], n=256)
    for k, v in kw.items():
        (q if k in q else c)[k] = v
    return L.ttt_window_attention_decode(L.ttt_window_decode_desc(*q.values()), *c.values(), 0)


@pytest.mark.parametrize("bad", [
    dict(B=-1), dict(Hq=3), dict(Hk=0), dict(slots=-4), dict(slots=0), dict(left=-1), dict(sinks=-1), dict(scale=-1.0),
    dict(ld_request=4100), dict(ld_slot=32), dict(ld_slot=130), dict(ld_head=-64), dict(Q=None), dict(ld_q=128), dict(K_new=None),
    dict(V_new=None), dict(ld_new=64), dict(K=None), dict(V=P[4] + 2), dict(lens=None), dict(lens=P[5] + 1), dict(Out=None),
    dict(Out=P[0]), dict(ws=None), dict(ws=P[7] + 64), dict(n=0)])
def test_decode_refusals(no_gpu, bad):
    assert _decode(**bad) == L.TTT_ERR_INVALID_ARG and L.ttt_last_error()


def test_decode_empty_batch(no_gpu):
    assert _decode(B=0) == L.TTT_OK and _decode(d=128) == L.TTT_ERR_UNSUPPORTED


def _scan(backward=False, **kw):
    q = dict(T=100, D=64, n_seq=1, form=1, dir=L.TTT_FWD, x_dtype=L.TTT_BF16)
    c = dict(cu=None, F=P[0], ld_f=64, X=P[1], ld_x=64, H_0=None, Y=P[2], ld_y=64, H_T=None, states=P[3], dY=P[4], ld_dy=64,
             dH_T=None, dF=P[5], ld_df=64, dX=P[6], ld_dx=64, dH_0=None, ws=P[7], n=1 << 24)
    for k, v in kw.items():
        (q if k in q else c)[k] = v
    d = L.ttt_gated_scan_desc(*q.values())
    a = [c[k] for k in ("cu", "F", "ld_f", "X", "ld_x", "H_0")]
    if backward:
        return L.ttt_gated_scan_backward(d, *a, *[c[k] for k in ("states", "dY", "ld_dy", "dH_T", "dF", "ld_df", "dX", "ld_dx",
                                                                   "dH_0", "ws", "n")], 0)
    return L.ttt_gated_scan(d, *a, *[c[k] for k in ("Y", "ld_y", "H_T", "states", "ws", "n")], 0)


SCAN_BAD = [dict(T=-1), dict(D=0), dict(D=12), dict(n_seq=0), dict(n_seq=3), dict(form=3), dict(form=-1), dict(dir=L.TTT_BIDIR),
            dict(x_dtype=2), dict(cu=P[8] + 2), dict(F=None), dict(X=P[1] + 4), dict(ld_f=56), dict(ld_x=68), dict(H_0=P[8] + 4),
            dict(ws=None), dict(ws=P[7] + 8), dict(n=0)]


@pytest.mark.parametrize("bad", SCAN_BAD + [dict(Y=None), dict(Y=P[0]), dict(H_T=P[8] + 4), dict(H_0=P[8], H_T=P[8]),
                                            dict(states=P[3] + 4)])
def test_scan_refusals(no_gpu, bad):
    assert _scan(**bad) == L.TTT_ERR_INVALID_ARG and L.ttt_last_error()


@pytest.mark.parametrize("bad", SCAN_BAD + [dict(states=None), dict(dY=None), dict(dF=P[0]), dict(dX=P[5]), dict(dH_0=P[8], dH_T=P[8])])
def test_scan_backward_refusals(no_gpu, bad):
    assert _scan(True, **bad) == L.TTT_ERR_INVALID_ARG and L.ttt_last_error()


@pytest.mark.parametrize("bad", [dict(B=-1), dict(D=4), dict(form=9), dict(F=None), dict(H=None), dict(H_out=P[3] + 4), dict(Y=P[0]),
                                 dict(H_out=P[2] + 256), dict(ld_x=32)])
def test_step_refusals(no_gpu, bad):
    c = dict(B=4, D=64, form=0, dt=L.TTT_F32, F=P[0], ld_f=64, X=P[1], ld_x=64, H=P[2], H_out=P[3], Y=P[4], ld_y=64)
    c.update(bad)
    assert L.ttt_gated_scan_step(*c.values(), 0) == L.TTT_ERR_INVALID_ARG and L.ttt_last_error()


def test_outputs_that_overlap_other_arrays_are_refused(no_gpu):
    bad = L.TTT_ERR_INVALID_ARG
    assert _window(Xres=P[3] + 512) == bad            # a residual one row off in Out
    assert _window(Xres=P[3] - 16) == bad
    assert _decode(Out=P[1]) == bad and _decode(Out=P[2] - 256) == bad
    assert _decode(ld_request=0) == bad               # every request would store into the same slots
    c = dict(B=4, D=64, form=0, dt=L.TTT_BF16, F=P[0], ld_f=64, X=P[1], ld_x=64, H=P[2], H_out=P[3], Y=P[4], ld_y=64)
    for kw in (dict(Y=P[2]), dict(Y=P[3] + 512), dict(H_out=P[0]), dict(H_out=P[1])):
        assert L.ttt_gated_scan_step(*{**c, **kw}.values(), 0) == bad, kw


def test_struct_layouts_match_the_header():
    """Sizes of the descriptors as a C compiler lays them out (natural alignment, no packing)."""
    assert ctypes.sizeof(L.ttt_rope_desc) == 7 * 4 + 4 + 6 * 8
    assert ctypes.sizeof(L.ttt_window_desc) == 10 * 4
    assert ctypes.sizeof(L.ttt_window_decode_desc) == 8 * 4 + 3 * 8
    assert ctypes.sizeof(L.ttt_gated_scan_desc) == 6 * 4


# ---------------------------------------------------------------- tensor-level functions
class _Like:
    """What the checks look at of a tensor on a GPU."""
    is_cuda = True

    def __init__(self, *shape):
        self.shape = shape

    def dim(self):
        return len(self.shape)

    def stride(self, k=None):
        s = tuple(int(np.prod(self.shape[i + 1:], dtype=np.int64)) for i in range(len(self.shape)))
        return s if k is None else s[k]


def test_descriptors_hold_the_numbers_of_the_call():
    """A number given as a tensor of one element that changes between calls."""
    import torch
    q, k, cache = _Like(8, 4, 64), _Like(8, 2, 64), _Like(8, 16, 2, 64)
    scale, left = torch.tensor(0.125), torch.tensor(5)
    for s, n in ((0.125, 5), (0.5, 2)):
        scale.fill_(s), left.fill_(n)
        for d in (L._window_desc(q, k, 1, left, 0, 0, scale), L._decode_desc(q, cache, left, 0, scale)):
            assert (d.scale, d.left) == (s, n)


def test_numbers_past_32_bits_are_refused():
    """A descriptor's integers have 32 bits: neither sizes nor windows may lose their upper ones."""
    q, k = _Like(8, 4, 64), _Like(8, 2, 64)
    for n in (2 ** 31, 2 ** 32 + 5, -2 ** 31 - 1):
        for call in (lambda: L._window_desc(q, k, 1, n, 0, 0, None), lambda: L._window_desc(q, k, 1, 3, n, 0, None),
                     lambda: L._window_desc(q, _Like(n, 2, 64), 1, 3, 0, 0, None),
                     lambda: L._decode_desc(q, _Like(8, n, 2, 64), 3, 0, None), lambda: L._gated_sizes(n, 8, 1, 0, 0, 0)):
            with pytest.raises(ValueError):
                call()


@pytest.mark.parametrize("d", [32, 128])
def test_keys_of_another_head_width_are_refused(d):
    with pytest.raises(ValueError):
        L._window_desc(_Like(8, 4, 64), _Like(8, 2, d), 1, 3, 0, 0, None)


@pytest.mark.parametrize("bad", [
    dict(ld_head=0), dict(ld_head=32),                              # one place for both heads, half of one
    dict(ld_slot=64, ld_head=64), dict(ld_slot=64, ld_head=128),    # a slot's second head is a later slot's first
    dict(ld_slot=64, ld_head=64 * 31),                              # heads of 32 slots, one too near
    dict(ld_slot=120), dict(V=P[3])])
def test_decode_refuses_new_keys_that_overwrite_each_other(no_gpu, bad):
    assert _decode(**bad) == L.TTT_ERR_INVALID_ARG and L.ttt_last_error()


@pytest.mark.parametrize("good", [
    dict(), dict(ld_slot=64, ld_head=64 * 32, ld_request=64 * 64), dict(Hk=1, Hq=4, ld_head=0, ld_slot=64),
    dict(K_new=None, V_new=None, ld_head=0), dict(K_new=None, V_new=None, V=P[3]), dict(ld_slot=136, ld_head=72),
    dict(V=P[3], V_new=P[1])])
def test_decode_accepts_its_cache_layouts(no_gpu, good):
    """Without a GPU the launch fails, behind the checks."""
    assert _decode(**good) == L.TTT_ERR_CUDA
