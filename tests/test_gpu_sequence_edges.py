"""The sequence operators where their kernels' tiles, strips, chunks and shares end, and what must not reach from
one row, sequence, call or stream into another.  Bounds as in oracle/sequence_ops.py."""
import math

import numpy as np
import pytest
import torch

from oracle import sequence_ops as S
from test_rnn_layer_b200 import tttmlp as L

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
NAN = float("nan")


def _rand(seed, *shape, dtype=torch.float32):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(*shape, generator=g, device="cuda").to(dtype)


def _np(t):
    return t.detach().double().cpu().numpy()


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _within(got, want, tol, name):
    g = _np(got)
    has = ~np.isnan(want)
    with np.errstate(invalid="ignore"):
        off = np.where(has & (g != want), np.abs(g - want), 0.0)
    over = float(np.where(has, off - tol, 0.0).max(initial=0.0))
    assert np.all(np.isfinite(g[has & np.isfinite(want)])), f"{name}: non-finite values"
    assert over <= 0, f"{name}: {over} beyond the bound"


# ---------------------------------------------------------------- rotary positions
@pytest.mark.parametrize("T,H,d,rot,layout,dtype", [
    (9, 3, 64, 24, "interleaved", "bf16"),      # three 16-byte pieces: the last has no second
    (9, 3, 64, 12, "interleaved", "f32"),
    (5, 2, 64, 4, "interleaved", "bf16"),       # no whole piece: pair by pair
    (5, 2, 24, 8, "interleaved", "bf16"),       # one piece
    (2000, 1, 64, 32, "half", "bf16"),          # several rows a block, part of the head
    (1999, 2, 128, 64, "half", "f32"),
    (700, 40, 64, 64, "half", "f32"),
    (1, 200, 64, 64, "interleaved", "bf16"),    # one row, more heads than one batch of loads
    (3, 300, 256, 256, "half", "bf16"),
])
@pytest.mark.parametrize("place", ["new", "in place", "strided"])
def test_rope_pieces(T, H, d, rot, layout, dtype, place):
    dt = BF if dtype == "bf16" else torch.float32
    wide = _rand(T + rot, T, H + 2, d, dtype=dt)
    x = wide[:, 1:H + 1] if place == "strided" else wide[:, :H].contiguous()
    want, tol = S.rope(_np(x), 5 + np.arange(T), rot, layout, dtype=dtype)
    keep = wide.clone()
    y = L.rope(x, pos0=5, rot=rot, layout=layout, out=x if place != "new" else None)
    _within(y, want, tol, "rope")
    if place == "strided":      # the heads on both sides were left alone
        assert torch.equal(wide[:, 0], keep[:, 0]) and torch.equal(wide[:, H + 1], keep[:, H + 1])


# ---------------------------------------------------------------- window attention
LONG = [   # cu_q, cu_k, Hq, Hk, left, right, sinks
    ([0, 5000], [0, 5000], 4, 2, 100, 0, 130),                 # sinks in two key blocks, their queries in three chunks
    ([0, 2048, 4097, 4099], [0, 2048, 4097, 4099], 2, 1, 50, 0, 1),   # chunks that end with a sequence
    ([0, 300, 4600], [0, 2500, 7000], 2, 2, 64, 10, 20),       # behind cached tokens, both sides
    ([0, 3000], [0, 3000], 1, 1, 3000, 0, 4),                  # causal: nothing behind the window
    ([0, 2600], [0, 2600], 1, 1, 20, 0, 300),                  # more sinks than are cut up
    ([0, 2500], [0, 40], 2, 1, 10, 0, 3),                      # fewer keys than queries
]


@pytest.mark.parametrize("cu_q,cu_k,Hq,Hk,left,right,sinks", LONG)
def test_window_long_lists_of_queries(cu_q, cu_k, Hq, Hk, left, right, sinks):
    Tq, Tk = cu_q[-1], cu_k[-1]
    q, k, v, g = (_rand(i, T, H, 64, dtype=BF) for i, (T, H) in enumerate(((Tq, Hq), (Tk, Hk), (Tk, Hk), (Tq, Hq))))
    mask = dict(left=left, right=right, sinks=sinks, cu_q=_ints(cu_q), cu_k=_ints(cu_k))
    ref = S.window_attention(_np(q), _np(k), _np(v), left, right, sinks, cu_q, cu_k, grad_out=_np(g))
    r = L.window_attention(q, k, v, want_lse=True, **mask)
    _within(r["out"], ref["out"], ref["out_tol"], "out")
    _within(r["lse"], ref["lse"], 2.0 ** -16 + 2.0 ** -17 * np.abs(np.nan_to_num(ref["lse"], neginf=0.0)), "lse")
    b = L.window_attention_backward(q, k, v, r["out"], r["lse"], g, **mask)
    for n in ("dq", "dk", "dv"):
        _within(b[n], ref[n], ref[n + "_tol"] + 1e-7, n)
    again = L.window_attention_backward(q, k, v, r["out"], r["lse"], g, **mask)
    assert all(torch.equal(again[n], b[n]) for n in ("dq", "dk", "dv"))


@pytest.mark.parametrize("left", [0, 1, 40])
def test_window_log_sum_exp_of_few_keys(left):
    """The sum is held in fp32: with one key its logarithm is the score, to fp32's last bits."""
    T = 300
    q, k, v = (_rand(7 + i, T, 1, 64, dtype=BF) for i in range(3))
    r = L.window_attention(q, k, v, left=left, want_lse=True)
    ref = S.window_attention(_np(q), _np(k), _np(v), left, 0, 0)["lse"]
    # 64 additions in fp32 (64 2^-24 of the sum of the products' sizes, which times the scale is below 16 here), an
    # exponential good to 2^-18
    assert np.abs(_np(r["lse"]) - ref).max() < 2.0 ** -18 * 16 + 2.0 ** -18


@pytest.mark.parametrize("left,right,sinks", [(0, 0, 1), (1, 0, 0), (2, 1, 1), (7, 0, 4), (0, 0, 16)])
def test_window_gradients_of_few_keys_do_not_lean_on_the_rounded_output(left, right, sinks):
    """dP - delta of a row with few keys is small beside dP, so delta must not come from Out's bf16 values there: the
    bound has dS's own rounding (2^-8 in all with the exponential's 2^-10) and fp32's, and no part of Out's."""
    T = 300
    q, k, v, g = (_rand(50 + i, T, 1, 64, dtype=BF) for i in range(4))
    r = L.window_attention(q, k, v, left=left, right=right, sinks=sinks, want_lse=True)
    b = L.window_attention_backward(q, k, v, r["out"], r["lse"], g, left=left, right=right, sinks=sinks)
    Q, K, V, G = (_np(t[:, 0]) for t in (q, k, v, g))
    see = S.visible(T, T, left, right, sinks)
    assert see.sum(1).max() <= 17
    s = np.where(see, Q @ K.T / 8, -np.inf)
    P = np.exp(s - s.max(1, keepdims=True))
    P /= P.sum(1, keepdims=True)
    dP = G @ V.T
    dS = P * (dP - (P * dP).sum(1, keepdims=True))
    # 2^-17: 64 products in fp32 (2^-18 of the sum of their sizes), in dP and in delta
    off = (2.0 ** -8 + 2.0 ** -10) * abs(dS) + P * 2.0 ** -17 * (abs(G) @ abs(V).T).max(1, keepdims=True)
    rows = see.sum(1) <= 20
    for n, want, tol, at in (("dq", dS @ K / 8, off @ abs(K) / 8, rows), ("dk", dS.T @ Q / 8, off.T @ abs(Q) / 8, slice(sinks, None))):
        _within(b[n][:, 0][torch.as_tensor(np.arange(T)[at], device="cuda")], want[at], (tol + 2.0 ** -8 * abs(want))[at], n)


def test_window_of_one_key_has_no_gradient_but_the_values():
    """A softmax of one score is constant."""
    T = 500
    q, k, v, g = (_rand(60 + i, T, 2, 64, dtype=BF) for i in range(4))
    r = L.window_attention(q, k, v, left=0, want_lse=True)
    b = L.window_attention_backward(q, k, v, r["out"], r["lse"], g, left=0)
    assert torch.equal(r["out"], v) and torch.all(b["dq"] == 0) and torch.all(b["dk"] == 0)
    _within(b["dv"], _np(g), 2.0 ** -8 * np.abs(_np(g)) * 1.25, "dv")


@pytest.mark.parametrize("value", [NAN, math.inf])
@pytest.mark.parametrize("which", ["q", "k", "v", "g"])
def test_window_backward_keeps_non_finite_values_to_those_that_meet_them(which, value):
    T, left, sinks, at = 700, 90, 2, 333
    q, k, v, g = (_rand(30 + i, T, 2, 64, dtype=BF) for i in range(4))
    r = L.window_attention(q, k, v, left=left, sinks=sinks, want_lse=True)
    clean = L.window_attention_backward(q, k, v, r["out"], r["lse"], g, left=left, sinks=sinks)
    t = dict(q=q, k=k, v=v, g=g)
    t[which][at, 0, 9] = value
    f = L.window_attention(q, k, v, left=left, sinks=sinks, want_lse=True, check_status=False)
    b = L.window_attention_backward(q, k, v, f["out"], f["lse"], g, left=left, sinks=sinks, check_status=False)
    assert L.ttt_mlp_status(b["workspace"]) == L.TTT_ERR_NONFINITE
    i = torch.arange(T, device="cuda")
    # query rows that meet it, and the keys that those rows see
    rows = (i >= at) & (i <= at + left) if which in "kv" else i == at
    first, last = int(rows.nonzero().min()), int(rows.nonzero().max())
    keys = ((i >= first - left) & (i <= last)) | (i < sinks)
    for n, touched in (("dq", rows), ("dk", keys), ("dv", keys)):
        assert torch.equal(b[n][~touched], clean[n][~touched]), n
        assert torch.equal(b[n][:, 1], clean[n][:, 1]), n          # the other head
    assert not torch.isfinite(b["dq"][rows, 0].float()).all()


def test_window_unseen_keys_get_zeros_whatever_they_hold():
    Tq, Tk, left = 50, 600, 30
    q, k, v, g = _rand(1, Tq, 1, 64, dtype=BF), _rand(2, Tk, 1, 64, dtype=BF), _rand(3, Tk, 1, 64, dtype=BF), _rand(4, Tq, 1, 64, dtype=BF)
    k[:400], v[:400] = NAN, math.inf
    r = L.window_attention(q, k, v, left=left, want_lse=True)
    b = L.window_attention_backward(q, k, v, r["out"], r["lse"], g, left=left)
    assert torch.all(b["dk"][:520] == 0) and torch.all(b["dv"][:520] == 0) and torch.isfinite(b["dq"].float()).all()


def test_two_window_calls_at_once():
    """Two streams, a workspace each, many items: the calls share nothing."""
    T = 3000
    a = [_rand(i, T, 4, 64, dtype=BF) for i in range(4)]
    c = [_rand(10 + i, T, 4, 64, dtype=BF) for i in range(4)]

    def step(q, k, v, g, ws=None, stream=None):
        r = L.window_attention(q, k, v, left=200, sinks=3, want_lse=True, workspace=ws, check_status=False, stream=stream)
        return r["out"], L.window_attention_backward(q, k, v, r["out"], r["lse"], g, left=200, sinks=3, workspace=ws,
                                                     check_status=False, stream=stream)

    alone = [step(*t) for t in (a, c)]
    torch.cuda.synchronize()
    ws = [L.window_attention_workspace(t[0], t[1], 1, backward=True) for t in (a, c)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(5):
        both = [step(*t, ws=w, stream=s) for t, w, s in zip((a, c), ws, streams)]
        torch.cuda.synchronize()
        for (o, b), (o1, b1) in zip(both, alone):
            assert torch.equal(o, o1) and all(torch.equal(b[n], b1[n]) for n in ("dq", "dk", "dv"))


# ---------------------------------------------------------------- decode
def test_decode_one_token_at_every_length_around_tiles_and_the_ring():
    Hq, Hk, sinks, left = 6, 2, 3, 130
    slots = sinks + left + 1
    lens = list(range(0, 140)) + [slots - 1, slots, slots + 1, 2 * slots, 1000, 2 ** 30]
    B = len(lens)
    ck, cv, q = (_rand(i, B, n, h, 64, dtype=BF) for i, (n, h) in enumerate(((slots, Hk), (slots, Hk), (1, Hq))))
    r = L.window_attention_decode(q[:, 0], ck, cv, _ints(lens), left=left, sinks=sinks)
    K, V = _np(ck), _np(cv)
    small = [i for i, n in enumerate(lens) if n < 2 ** 20]
    want, tol = S.window_decode(_np(q[:, 0])[small], lambda b, u: K[small[b], S.cache_slot(u, slots, sinks)],
                                lambda b, u: V[small[b], S.cache_slot(u, slots, sinks)], [lens[i] for i in small], left, sinks, slots)
    _within(r["out"][small], want, tol, "decode")
    # a far position sees every slot of a ring of exactly its window, whatever their order
    s = torch.einsum("hd,chd->hc", q[-1, 0].double(), ck[-1].double().repeat_interleave(Hq // Hk, 1)) / 8
    far = torch.einsum("hc,chd->hd", s.softmax(-1), cv[-1].double().repeat_interleave(Hq // Hk, 1))
    assert (r["out"][-1].double() - far).abs().max() < 2.0 ** -6


# ---------------------------------------------------------------- gated recurrence
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dirs", ["fwd", "rev"])
@pytest.mark.parametrize("T,D", [
    (1, 8), (7, 16), (8, 40), (56, 8), (57, 72), (449, 200),     # narrow strips, less than a tile, a tile and a row
    (3000, 8), (2000, 520), (900, 1000), (700, 2048), (300, 5000),
])
def test_scan_strips_and_tiles(T, D, dirs, dtype):
    dt = BF if dtype == "bf16" else torch.float32
    f, x, dy = (_rand(1, T, D) + 3).to(dt), _rand(2, T, D, dtype=dt), _rand(3, T, D, dtype=dt)
    h0, dhT = _rand(4, 1, D), _rand(5, 1, D)
    ref = S.gated_scan(_np(f), _np(x), "unit", dirs == "rev", None, _np(h0), _np(dy), _np(dhT), dtype)
    r = L.gated_scan(f, x, form="unit", dirs=dirs, h0=h0, want_state=True, want_chunk_states=True)
    _within(r["y"], ref["y"], ref["y_tol"], "y")
    _within(r["h_T"], ref["hT"], ref["hT_tol"], "h_T")
    b = L.gated_scan_backward(f, x, dy, r["chunk_states"], form="unit", dirs=dirs, h0=h0, dh_T=dhT, want_dh0=True)
    for n in ("df", "dx", "dh0"):
        _within(b[n], ref[n], ref[n + "_tol"] + 1e-30, n)


@pytest.mark.parametrize("dirs", ["fwd", "rev"])
@pytest.mark.parametrize("D", [8, 24, 264])
def test_scan_of_many_short_sequences(D, dirs):
    lens = [(5 * i) % 7 for i in range(800)]
    cu = np.concatenate([[0], np.cumsum(lens)]).tolist()
    T = cu[-1]
    f, x, dy = _rand(1, T, D) + 1, _rand(2, T, D), _rand(3, T, D)
    h0, dhT = _rand(4, 800, D), _rand(5, 800, D)
    ref = S.gated_scan(_np(f), _np(x), "convex", dirs == "rev", cu, _np(h0), _np(dy), _np(dhT))
    how = dict(dirs=dirs, cu=_ints(cu), h0=h0)
    r = L.gated_scan(f, x, want_state=True, want_chunk_states=True, **how)
    _within(r["y"], ref["y"], ref["y_tol"], "y")
    _within(r["h_T"], ref["hT"], ref["hT_tol"], "h_T")
    b = L.gated_scan_backward(f, x, dy, r["chunk_states"], dh_T=dhT, want_dh0=True, **how)
    for n in ("df", "dx", "dh0"):
        _within(b[n], ref[n], ref[n + "_tol"] + 1e-30, n)


@pytest.mark.parametrize("dirs", ["fwd", "rev"])
@pytest.mark.parametrize("which", ["f", "x", "dy", "h0"])
@pytest.mark.parametrize("value", [NAN, math.inf])
def test_scan_keeps_non_finite_values_to_their_sequence_and_channel(which, value, dirs):
    cu, D = [0, 300, 700, 1500], 72
    T = cu[-1]
    f, x, dy, h0 = _rand(1, T, D) + 4, _rand(2, T, D), _rand(3, T, D), _rand(4, 3, D)
    how = dict(form="sum", dirs=dirs, cu=_ints(cu))

    def both():
        r = L.gated_scan(f, x, h0=h0, want_state=True, want_chunk_states=True, check_status=False, **how)
        b = L.gated_scan_backward(f, x, dy, r["chunk_states"], h0=h0, want_dh0=True, check_status=False, **how)
        return [r["y"], b["df"], b["dx"]], [r["h_T"], b["dh0"]], r["workspace"], b["workspace"]

    rows0, states0, _, _ = both()
    t = dict(f=f, x=x, dy=dy, h0=h0)[which]
    t[1 if which == "h0" else 500, 5] = NAN if which == "f" else value
    rows, states, w1, w2 = both()
    assert L.TTT_ERR_NONFINITE in (L.ttt_mlp_status(w1), L.ttt_mlp_status(w2))
    other = torch.ones(T, D, dtype=torch.bool, device="cuda")
    other[cu[1]:cu[2], 5] = False
    for a, c in zip(rows, rows0):
        assert torch.equal(a[other], c[other])
    keep = torch.ones(3, D, dtype=torch.bool, device="cuda")
    keep[1, 5] = False
    for a, c in zip(states, states0):
        assert torch.equal(a[keep], c[keep])
    if which != "dy":
        assert not torch.isfinite(rows[0][cu[1]:cu[2], 5]).all()


def test_two_scans_at_once():
    T, D = 5000, 512
    sets = [[_rand(10 * j + i, T, D, dtype=BF) for i in range(2)] for j in range(2)]
    alone = [L.gated_scan(*s, want_state=True) for s in sets]
    ws, streams = [L.gated_scan_workspace(s[1]) for s in sets], [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(5):
        both = [L.gated_scan(*s, want_state=True, workspace=w, stream=st, check_status=False) for s, w, st in zip(sets, ws, streams)]
        torch.cuda.synchronize()
        for a, b in zip(both, alone):
            assert torch.equal(a["y"], b["y"]) and torch.equal(a["h_T"], b["h_T"])


def test_operators_refuse_tensors_of_the_wrong_place_or_size():
    x = _rand(1, 16, 64)
    r = L.gated_scan(x, x.clone(), want_chunk_states=True)
    for call in (lambda: L.gated_scan_backward(x, x, x, r["chunk_states"][:-8]),
                 lambda: L.gated_scan(x, x.cpu()),
                 lambda: L.gated_scan(x, x.half()),
                 lambda: L.gated_scan(x, x, h0=_rand(2, 2, 64)),
                 lambda: L.rope(x.view(16, 1, 64), positions=torch.zeros(15, dtype=torch.int32, device="cuda"))):
        with pytest.raises(ValueError):
            call()
    q = _rand(3, 8, 1, 64, dtype=BF)
    with pytest.raises(L.TTTError):     # a workspace of the forward pass is too small for the backward pass
        f = L.window_attention(q, q.clone(), q.clone(), left=3, want_lse=True)
        L.window_attention_backward(q, q.clone(), q.clone(), f["out"], f["lse"], q.clone(), left=3, workspace=f["workspace"])


def test_row_strides_past_32_bits():
    """Rows 2^30 elements apart: every offset of the last rows needs 64 bits."""
    T, ld = 3, 2 ** 30
    big = torch.empty((T - 1) * ld + 4096, dtype=BF, device="cuda")

    def far(col, *shape):       # [T, *shape] at columns col...
        n = math.prod(shape)
        t = big.as_strided((T, *shape), (ld, 64, 1) if len(shape) == 2 else (ld, 1), col)
        return t.copy_(_rand(col + n, T, *shape, dtype=BF))

    q, k, v, g = (far(512 * i, 2, 64) for i in range(4))
    near = [t.contiguous() for t in (q, k, v, g)]
    out, dq, dk, dv = (far(512 * i, 2, 64) for i in range(4, 8))
    r = L.window_attention(q, k, v, left=5, want_lse=True, out=out)
    b = L.window_attention_backward(q, k, v, out, r["lse"], g, left=5, dq=dq, dk=dk, dv=dv)
    r1 = L.window_attention(*near[:3], left=5, want_lse=True)
    b1 = L.window_attention_backward(*near[:3], r1["out"], r1["lse"], near[3], left=5)
    assert torch.equal(out, r1["out"]) and torch.equal(r["lse"], r1["lse"])
    assert all(torch.equal(b[n], b1[n]) for n in ("dq", "dk", "dv"))
    assert torch.equal(L.rope(q, out=out), L.rope(near[0]))
    f, x, dy = (far(512 * i, 128) for i in range(3))
    near = [t.contiguous() for t in (f, x, dy)]
    y, df, dx = (far(512 * i, 128) for i in range(3, 6))
    s = L.gated_scan(f, x, y=y, want_chunk_states=True)
    c = L.gated_scan_backward(f, x, dy, s["chunk_states"], df=df, dx=dx)
    s1 = L.gated_scan(*near[:2], want_chunk_states=True)
    c1 = L.gated_scan_backward(*near, s1["chunk_states"])
    assert torch.equal(y, s1["y"]) and torch.equal(df, c1["df"]) and torch.equal(dx, c1["dx"])
    h = _rand(9, T, 128)
    y1, h1 = L.gated_scan_step(f, x, h, y=y)
    y2, h2 = L.gated_scan_step(*near[:2], h)
    assert torch.equal(y1, y2) and torch.equal(h1, h2)


def test_a_training_block_in_one_graph():
    """rotary positions, attention and recurrence, forward and backward, captured together and replayed on new inputs."""
    T, Hq, Hk = 900, 4, 2
    W = Hq * 64
    cu = _ints([0, 400, 401, 850])
    ins = [_rand(1, T, Hq + 2 * Hk, 64, dtype=BF), _rand(2, T, W, dtype=BF), _rand(3, T, W, dtype=BF)]
    mask = dict(left=100, sinks=2, cu_q=cu, cu_k=cu, check_status=False)
    like = torch.zeros(T, Hq + Hk, 64, dtype=BF, device="cuda")
    ws = L.window_attention_workspace(like[:, :Hq], like[:, Hq:], 3, backward=True)
    sw = L.gated_scan_workspace(ins[1], 3)

    def step():
        qkv, f, dy = ins
        turned = L.rope(qkv[:, :Hq + Hk])
        q, k, v = turned[:, :Hq], turned[:, Hq:], qkv[:, Hq + Hk:]
        a = L.window_attention(q, k, v, want_lse=True, workspace=ws, **mask)
        x = a["out"].view(T, W)
        s = L.gated_scan(f, x, cu=cu, want_chunk_states=True, workspace=sw, check_status=False)
        sb = L.gated_scan_backward(f, x, dy, s["chunk_states"], cu=cu, workspace=sw, check_status=False)
        ab = L.window_attention_backward(q, k, v, a["out"], a["lse"], sb["dx"].view(T, Hq, 64), workspace=ws, **mask)
        back = L.rope(torch.cat([ab["dq"], ab["dk"]], 1), inverse=True)
        return [a["out"], a["lse"], s["y"], sb["df"], sb["dx"], ab["dv"], back]

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            out = step()
    s.synchronize()
    for i, t in enumerate(ins):
        t.copy_(_rand(20 + i, *t.shape, dtype=BF))
    torch.cuda.synchronize()
    graph.replay()
    torch.cuda.synchronize()
    got = [t.clone() for t in out]
    for a, b in zip(got, step()):
        assert torch.equal(a, b)
    assert L.ttt_mlp_status(ws) == L.TTT_OK and L.ttt_mlp_status(sw) == L.TTT_OK


@pytest.mark.parametrize("default", [torch.bfloat16, torch.float64])
def test_buffers_keep_their_type_under_another_default(default):
    """What the wrappers allocate is fp32 where the kernels write fp32, whatever torch's default type."""
    f, x, dy = (_rand(i, 40, 64, dtype=BF) for i in range(3))
    q, k, v, g = (_rand(9 + i, 40, 2, 64, dtype=BF) for i in range(4))
    cache = torch.stack([k[:8], v[:8]])

    def run():
        s = L.gated_scan(f, x, want_state=True, want_chunk_states=True)
        b = L.gated_scan_backward(f, x, dy, s["chunk_states"], want_dh0=True)
        r = L.window_attention(q, k, v, left=7, want_lse=True)
        w = L.window_attention_backward(q, k, v, r["out"], r["lse"], g, left=7)
        d = L.window_attention_decode(q[:1], cache[:1], cache[1:], _ints([5]), left=7)
        y, h = L.gated_scan_step(f[:1], x[:1], s["h_T"])
        return [s["y"], s["h_T"], s["chunk_states"], b["df"], b["dx"], b["dh0"], r["out"], r["lse"], w["dq"], w["dk"],
                w["dv"], d["out"], y, h, L.rope(q)]

    want = run()
    before = torch.get_default_dtype()
    try:
        torch.set_default_dtype(default)
        got = run()
    finally:
        torch.set_default_dtype(before)
    for a, b in zip(got, want):
        assert a.dtype is b.dtype and torch.equal(a, b)


@pytest.mark.parametrize("left,right,sinks", [(1023, 0, 4), (500, 400, 0), (5000, 0, 130)])
def test_few_blocks_are_drawn_by_their_work(left, right, sinks):
    """Sequences of unequal lengths, more items than CTAs: every row's result, and none behind the last one's, whatever
    the order in which the blocks are drawn (a sequence alone gives the same bits)."""
    Hq, Hk = 12, 4
    nq, nk = [700, 0, 1, 129, 256, 257, 900], [1500, 300, 800, 100, 256, 1300, 900]
    cq, ck = np.cumsum([0] + nq).tolist(), np.cumsum([0] + nk).tolist()
    Tq, Tk = cq[-1] + 9, ck[-1] + 5
    q, k, v, g = (_rand(60 + i, T, H, 64, dtype=BF) for i, (T, H) in enumerate([(Tq, Hq), (Tk, Hk), (Tk, Hk), (Tq, Hq)]))
    mask = dict(left=left, right=right, sinks=sinks)
    both = dict(mask, cu_q=_ints(cq), cu_k=_ints(ck))
    r = L.window_attention(q, k, v, want_lse=True, **both)
    b = L.window_attention_backward(q, k, v, r["out"], r["lse"], g, **both)
    assert not r["out"][cq[-1]:].any() and not b["dq"][cq[-1]:].any()
    for s in range(len(nq)):
        if not nq[s]:
            continue
        i, u = slice(cq[s], cq[s + 1]), slice(ck[s], ck[s + 1])
        r1 = L.window_attention(q[i], k[u], v[u], want_lse=True, **mask)
        b1 = L.window_attention_backward(q[i], k[u], v[u], r1["out"], r1["lse"], g[i], **mask)
        assert torch.equal(r["out"][i], r1["out"]) and torch.equal(r["lse"][:, i], r1["lse"])
        assert torch.equal(b["dq"][i], b1["dq"])


def test_query_gradients_of_rows_with_few_keys():
    """Rows of 1 to 30 keys: dQ is one rounding from the formula's where the delta pass makes it (up to 20 keys), and a row
    whose upstream gradient is not finite is NaN while the others keep their bits."""
    T, Hq, Hk = 400, 4, 2
    q, k, v, g = (_rand(80 + i, T, H, 64, dtype=BF) for i, H in enumerate([Hq, Hk, Hk, Hq]))
    cu = list(range(0, 400, 30)) + [400]
    both = dict(left=200, sinks=1, cu_q=_ints(cu), cu_k=_ints(cu))
    r = L.window_attention(q, k, v, want_lse=True, **both)
    b = L.window_attention_backward(q, k, v, r["out"], r["lse"], g, **both)
    want = S.window_attention(*map(_np, (q, k, v)), 200, 0, 1, cu, cu, grad_out=_np(g))["dq"]
    few = np.concatenate([np.arange(a, min(a + 20, e)) for a, e in zip(cu, cu[1:])])
    got = _np(b["dq"])
    # a rounding of bf16 is off by at most 2^-8 of the value; 2^-12 of the row's largest value covers fp32 and the log-sum-exp
    tol = 2.0 ** -8 * np.abs(want) + 2.0 ** -12 * np.abs(want).max(axis=(1, 2), keepdims=True)
    single = np.isin(np.arange(T), cu[:-1])
    assert not got[single].any()
    assert (np.abs(got - want) <= tol)[few][~single[few]].all()
    g2 = g.clone()
    g2[7, 1, 3] = NAN
    b2 = L.window_attention_backward(q, k, v, r["out"], r["lse"], g2, check_status=False, **both)
    assert b2["dq"][7, 1].isnan().all() and L.ttt_mlp_status(b2["workspace"]) == L.TTT_ERR_NONFINITE
    keep = torch.ones(T, Hq, dtype=torch.bool, device="cuda")
    keep[7, 1] = False
    assert torch.equal(b2["dq"][keep], b["dq"][keep])
