"""The sequence operators on the GPU against their fp64 definitions, element
by element within the bounds oracle/sequence_ops.py derives (a rounding is off
by at most half a step; the softmax weights and dS enter their products as
bf16; everything else is fp32)."""
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


def _within(got, want, tol, name="", slack=0.0):
    """|got - want| <= tol wherever the definition has a value (NaN: rows of no sequence)."""
    g = _np(got) if isinstance(got, torch.Tensor) else got
    has = ~np.isnan(want)
    same_inf = np.isinf(want) & (g == want)
    with np.errstate(invalid="ignore"):
        off = np.where(has & ~same_inf, np.abs(g - want), 0.0)
    over = np.where(has, off - tol, 0.0)
    assert np.all(np.isfinite(g[has & ~np.isinf(want)])), f"{name}: non-finite values"
    worst = float(over.max(initial=0.0))
    print(f"{name}: worst excess {worst:.2e}, worst share of the bound "
          f"{float(np.max(off / (tol + 1e-30), initial=0.0)):.2f}")
    assert worst <= slack, f"{name}: {worst} beyond the bound"


# ---------------------------------------------------------------- rotary positions
RAMP = {"kind": "ramp", "factor": 8.0, "length": 4096, "low": 1.0, "high": 4.0, "amplitude": 1.2}


@pytest.mark.parametrize("T,H,d,rot,layout,scaling,dtype,inverse", [
    (1, 1, 64, 64, "half", None, "bf16", False),
    (1, 1, 8, 2, "interleaved", None, "f32", False),
    (37, 5, 64, 32, "half", {"kind": "linear", "factor": 4.0}, "f32", False),
    (130, 3, 80, 80, "interleaved", {"kind": "base", "factor": 4.0}, "bf16", True),
    (61, 7, 80, 20, "half", RAMP, "bf16", False),          # rot / 2 = 10: pairs at no vector boundary
    (33, 2, 24, 6, "half", RAMP, "f32", True),
    (1000, 12, 64, 64, "half", RAMP, "bf16", False),
    (77, 2, 256, 256, "interleaved", None, "f32", False),
    (3001, 1, 128, 64, "interleaved", None, "bf16", False),
])
@pytest.mark.parametrize("where", ["near", "far"])
def test_rope(T, H, d, rot, layout, scaling, dtype, inverse, where):
    x = _rand(T + rot, T, H, d, dtype=BF if dtype == "bf16" else torch.float32)
    pos = torch.arange(T) * 3 if where == "near" else torch.randint(-2 ** 31, 2 ** 31 - 1, (T,), generator=torch.Generator().manual_seed(T))
    y = L.rope(x, pos.to(torch.int32).cuda(), rot=rot, layout=layout, scaling=scaling, inverse=inverse)
    want, tol = S.rope(_np(x), pos.numpy(), rot, layout, scaling=scaling, inverse=inverse, dtype=dtype)
    _within(y, want, tol, "rope")
    again = L.rope(x.clone(), pos.to(torch.int32).cuda(), rot=rot, layout=layout, scaling=scaling, inverse=inverse, out=None)
    assert torch.equal(again, y)


def test_rope_in_place_on_the_queries_and_keys_of_a_fused_array():
    T, Hq, Hk = 203, 4, 2
    qkv = _rand(1, T, Hq + 2 * Hk, 64, dtype=BF)
    keep = qkv.clone()
    part = qkv[:, :Hq + Hk]
    L.rope(part, pos0=2 ** 31 - 100, out=part)
    want, tol = S.rope(_np(keep[:, :Hq + Hk]), 2 ** 31 - 100 + np.arange(T), 64, "half", dtype="bf16")
    _within(part, want, tol, "rope")
    assert torch.equal(qkv[:, Hq + Hk:], keep[:, Hq + Hk:])


def test_rope_of_no_rows():
    assert L.rope(torch.empty(0, 2, 64, device="cuda", dtype=BF)).shape == (0, 2, 64)


# ---------------------------------------------------------------- window attention
# (cu_q, cu_k, Hq, Hk, left, right, sinks, padding rows)
WINDOW = [
    ([0, 1], [0, 1], 1, 1, 0, 0, 0, 0),
    ([0, 1], [0, 300], 2, 1, 99, 0, 3, 0),                     # one query behind a cached prefix
    ([0, 129], [0, 129], 1, 1, 2 ** 31 - 1, 0, 0, 0),          # causal, one row past a tile
    ([0, 256], [0, 256], 3, 3, 63, 0, 0, 0),
    ([0, 700], [0, 700], 4, 2, 127, 0, 5, 0),                  # window of exactly a tile
    ([0, 1000], [0, 1000], 2, 2, 300, 0, 130, 0),              # more sinks than a tile
    ([0, 513], [0, 513], 2, 1, 50, 50, 4, 0),                  # both sides
    ([0, 300], [0, 300], 1, 1, 0, 2 ** 31 - 1, 0, 0),          # everything ahead
    ([0, 400], [0, 400], 1, 1, 2 ** 31 - 1, 2 ** 31 - 1, 7, 0),  # full
    ([0, 300], [0, 170], 2, 1, 40, 0, 2, 0),                   # fewer keys than queries: empty rows
    ([0, 200], [0, 0], 2, 2, 40, 40, 2, 0),                    # no keys at all
    ([0, 0], [0, 77], 2, 2, 40, 40, 2, 0),                     # no queries
    ([0, 5, 5, 6, 260, 389, 640], [0, 9, 20, 21, 275, 404, 400 + 300], 6, 2, 90, 0, 4, 37),
    ([0, 100, 201, 202, 330], [0, 100, 201, 202, 330], 5, 5, 20, 20, 0, 3),
    ([0, 128, 256, 512], [0, 128, 256, 512], 8, 1, 200, 0, 1, 0),
    ([0, 900], [0, 2300], 3, 1, 1500, 0, 0, 5),
    ([0, 50, 700], [0, 3, 1500], 4, 4, 10, 3, 900, 0),         # sinks overlap the window
]


def _window_inputs(case, seed=0, pad_value=NAN):
    cu_q, cu_k, Hq, Hk, left, right, sinks, pad = case
    Tq, Tk = cu_q[-1] + pad, cu_k[-1] + pad
    q, kv, g = _rand(seed, Tq, Hq, 64, dtype=BF), _rand(seed + 1, Tk, 2 * Hk, 64, dtype=BF), _rand(seed + 2, Tq, Hq, 64, dtype=BF)
    q = (q.float() * 2).to(BF)
    q[cu_q[-1]:], kv[cu_k[-1]:], g[cu_q[-1]:] = pad_value, pad_value, pad_value
    packed = len(cu_q) > 2 or pad
    mask = dict(left=left, right=right, sinks=sinks, cu_q=_ints(cu_q) if packed else None, cu_k=_ints(cu_k) if packed else None)
    return q, kv[:, :Hk], kv[:, Hk:], g, mask


def _reference(case, q, k, v, g=None):
    cu_q, cu_k, _, _, left, right, sinks, _ = case
    return S.window_attention(_np(q), _np(k), _np(v), left, right, sinks, cu_q, cu_k, grad_out=None if g is None else _np(g))


def _check_forward(r, ref):
    _within(r["out"], ref["out"], ref["out_tol"], "out")
    # exponentials good to 2^-13, logits to 2^-17 of their size (64 products of bf16 values summed in fp32)
    _within(r["lse"], ref["lse"], 2.0 ** -12 + 2.0 ** -17 * np.abs(np.nan_to_num(ref["lse"], neginf=0.0)), "lse")


@pytest.mark.parametrize("case", WINDOW, ids=str)
def test_window_attention(case):
    q, k, v, _, mask = _window_inputs(case)
    cu_q, pad = case[0], case[-1]
    out, lse = torch.full_like(q, 7.0), torch.full((q.shape[1], q.shape[0]), 7.0, device="cuda")
    r = L.window_attention(q, k, v, out=out, lse=lse, **mask)
    _check_forward(r, _reference(case, q, k, v))
    if pad:   # rows behind the last sequence stay as they were
        assert torch.all(out[cu_q[-1]:] == 7.0) and torch.all(lse[:, cu_q[-1]:] == 7.0)
    again = L.window_attention(q, k, v, want_lse=True, **mask)
    n = cu_q[-1]
    assert torch.equal(again["out"][:n], out[:n]) and torch.equal(again["lse"][:, :n], lse[:, :n])


@pytest.mark.parametrize("case", WINDOW, ids=str)
def test_window_attention_backward(case):
    q, k, v, g, mask = _window_inputs(case, seed=5)
    cu_q, cu_k, pad = case[0], case[1], case[-1]
    ref = _reference(case, q, k, v, g)
    r = L.window_attention(q, k, v, want_lse=True, **mask)
    grads = [torch.full_like(q, 7.0)] + [torch.full(k.shape, 7.0, dtype=BF, device="cuda") for _ in range(2)]
    b = L.window_attention_backward(q, k, v, r["out"], r["lse"], g, dq=grads[0], dk=grads[1], dv=grads[2], **mask)
    for n in ("dq", "dk", "dv"):
        _within(b[n], ref[n], ref[n + "_tol"] + 1e-7, n)
    if pad:
        assert torch.all(b["dq"][cu_q[-1]:] == 7.0) and torch.all(b["dk"][cu_k[-1]:] == 7.0) and torch.all(b["dv"][cu_k[-1]:] == 7.0)
    again = L.window_attention_backward(q, k, v, r["out"], r["lse"], g, **mask)
    for n, end in (("dq", cu_q[-1]), ("dk", cu_k[-1]), ("dv", cu_k[-1])):
        assert torch.equal(again[n][:end], b[n][:end]), n


def test_window_scale_and_residual():
    case = WINDOW[4]
    q, k, v, _, mask = _window_inputs(case)
    x = _rand(9, *q.shape, dtype=BF)
    ref = S.window_attention(_np(q), _np(k), _np(v), *case[4:7], scale=0.31)
    out = x.clone()
    L.window_attention(q, k, v, scale=0.31, residual=out, out=out, **mask)
    want = ref["out"] + _np(x)
    _within(out, want, ref["out_tol"] + 2.0 ** -8 * np.abs(want), "out + residual")
    # a row that sees nothing passes its residual through
    q2, k2, v2, _, mask2 = _window_inputs(WINDOW[9])
    x2 = _rand(10, *q2.shape, dtype=BF)
    r2 = L.window_attention(q2, k2, v2, residual=x2, **mask2)
    assert torch.equal(r2["out"][:130], x2[:130])


def test_window_large_logits():
    """Logits of some hundreds and a maximum that rises late: the running maximum must follow it."""
    T = 600
    q, k, v = (_rand(20 + i, T, 1, 64, dtype=BF) for i in range(3))
    q = (q.float() * 6).to(BF)
    k = (k.float() * torch.linspace(0.1, 9.0, T, device="cuda")[:, None, None]).to(BF)
    r = L.window_attention(q, k, v, left=T, sinks=3, want_lse=True)
    _check_forward(r, S.window_attention(_np(q), _np(k), _np(v), T, 0, 3))


@pytest.mark.parametrize("value", [NAN, math.inf, -math.inf])
@pytest.mark.parametrize("which", ["k", "v", "q"])
def test_window_non_finite_values_stay_with_the_rows_that_see_them(which, value):
    T, left, sinks, at = 700, 100, 2, 333
    q, k, v = (_rand(30 + i, T, 1, 64, dtype=BF) for i in range(3))
    clean = L.window_attention(q, k, v, left=left, sinks=sinks)["out"]
    dict(q=q, k=k, v=v)[which][at, 0, 5] = value
    r = L.window_attention(q, k, v, left=left, sinks=sinks, check_status=False)
    i = torch.arange(T, device="cuda")
    sees = (i >= at) & (i <= at + left) if which != "q" else i == at
    assert torch.equal(r["out"][~sees], clean[~sees])
    assert L.ttt_mlp_status(r["workspace"]) == L.TTT_ERR_NONFINITE
    if which != "k":      # a key's infinity may also end as a weight of zero
        assert not torch.isfinite(r["out"][sees].float()).all(dim=(1, 2)).any()


def test_window_on_strided_arrays_and_another_stream():
    T, H = 300, 2
    wide = _rand(40, T, 3 * H + 1, 64, dtype=BF)
    q, k, v = wide[:, :H], wide[:, H:2 * H], wide[:, 2 * H:3 * H]
    out = torch.full((T, H + 2, 64), 7.0, dtype=BF, device="cuda")
    want = L.window_attention(q.contiguous(), k.contiguous(), v.contiguous(), left=40, sinks=1)["out"]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    r = L.window_attention(q, k, v, left=40, sinks=1, out=out[:, 1:H + 1], stream=s)
    assert torch.equal(r["out"], want)
    assert torch.all(out[:, 0] == 7.0) and torch.all(out[:, H + 1:] == 7.0)


def test_window_bad_offsets_are_reported():
    q, k, v = (_rand(50 + i, 200, 1, 64, dtype=BF) for i in range(3))
    for bad in ([0, 150, 100, 200], [0, 100, 150, 5000], [-7, 10, 20, 200], [0, 10, 20, -5], [3, 10, 20, 200]):
        with pytest.raises(L.TTTError) as e:
            L.window_attention(q, k, v, left=10, cu_q=_ints(bad), cu_k=_ints(bad))
        assert e.value.status == L.TTT_ERR_INVALID_ARG
        ok = _ints([0, 50, 60, 200])
        r = L.window_attention(q, k, v, left=10, cu_q=ok, cu_k=ok, want_lse=True)
        with pytest.raises(L.TTTError) as e:
            L.window_attention_backward(q, k, v, r["out"], r["lse"], q, left=10, cu_q=ok, cu_k=_ints(bad))
        assert e.value.status == L.TTT_ERR_INVALID_ARG


def test_window_many_sequences():
    n = 700
    lens = [(7 * i) % 5 for i in range(n)]
    cu = np.concatenate([[0], np.cumsum(lens)]).tolist()
    case = (cu, cu, 2, 1, 3, 1, 1, 4)
    q, k, v, g, mask = _window_inputs(case)
    ref = _reference(case, q, k, v, g)
    r = L.window_attention(q, k, v, want_lse=True, **mask)
    _check_forward(r, ref)
    b = L.window_attention_backward(q, k, v, r["out"], r["lse"], g, **mask)
    for m in ("dq", "dk", "dv"):
        _within(b[m], ref[m], ref[m + "_tol"] + 1e-7, m)


def test_window_training_step_in_a_graph():
    case = WINDOW[12]
    q, k, v, g, mask = _window_inputs(case)
    ws = L.window_attention_workspace(q, k, len(case[0]) - 1, backward=True)
    out, lse = torch.zeros_like(q), torch.zeros(q.shape[1], q.shape[0], device="cuda")
    dq, dk, dv = torch.zeros_like(q), torch.zeros(k.shape, dtype=BF, device="cuda"), torch.zeros(k.shape, dtype=BF, device="cuda")

    def step():
        L.window_attention(q, k, v, out=out, lse=lse, workspace=ws, check_status=False, **mask)
        L.window_attention_backward(q, k, v, out, lse, g, dq=dq, dk=dk, dv=dv, workspace=ws, check_status=False, **mask)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    q2, k2, v2, g2, _ = _window_inputs(case, seed=60)
    for a, b in ((q, q2), (k, k2), (v, v2), (g, g2)):
        a.copy_(b)
    for t in (out, lse, dq, dk, dv):
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    got = [t.clone() for t in (out, lse, dq, dk, dv)]
    for t in (out, lse, dq, dk, dv):
        t.zero_()
    step()
    for a, b in zip(got, (out, lse, dq, dk, dv)):
        assert torch.equal(a, b)
    assert float(dq[:5].float().abs().max()) > 0


# ---------------------------------------------------------------- decode
def _decode_case(B, Hq, Hk, slots, left, sinks, lens, layout="slots", seed=0, new=True, scale=None):
    """Fills a cache as a server would: token after token, in its slot."""
    shape = (B, slots, Hk, 64)
    if layout == "heads":       # [B, Hk, slots, 64] in memory
        ck = torch.full((B, Hk, slots, 64), NAN, dtype=BF, device="cuda").transpose(1, 2)
        cv = torch.full((B, Hk, slots, 64), NAN, dtype=BF, device="cuda").transpose(1, 2)
    else:
        ck, cv = torch.full(shape, NAN, dtype=BF, device="cuda"), torch.full(shape, NAN, dtype=BF, device="cuda")
    n = max(1, max(lens))
    K, V = _rand(seed, B, n, Hk, 64, dtype=BF), _rand(seed + 1, B, n, Hk, 64, dtype=BF)
    q = (_rand(seed + 2, B, Hq, 64) * 2).to(BF)
    for b, ln in enumerate(lens):
        last = ln - (1 if new else 0)
        us = [u for u in range(max(last, 0)) if u < sinks or last - u <= slots - sinks or last <= slots]
        if us:
            at = torch.tensor([S.cache_slot(u, slots, sinks) for u in us], device="cuda")
            ck[b, at], cv[b, at] = K[b, us], V[b, us]
    idx = torch.tensor([max(ln - 1, 0) for ln in lens], device="cuda")
    rows = torch.arange(B, device="cuda")
    k_new, v_new = (K[rows, idx].contiguous(), V[rows, idx].contiguous()) if new else (None, None)
    before = ck.clone(), cv.clone()
    r = L.window_attention_decode(q, ck, cv, _ints(lens), left=left, sinks=sinks, k_new=k_new, v_new=v_new, scale=scale)
    Kn, Vn = _np(K), _np(V)
    want, tol = S.window_decode(_np(q), lambda b, u: Kn[b, u], lambda b, u: Vn[b, u], lens, left, sinks, slots, scale)
    _within(r["out"], want, tol, "decode")
    if new:                     # the new token and nothing else was stored
        for c, src, old in ((ck, K, before[0]), (cv, V, before[1])):
            for b, ln in enumerate(lens):
                if ln > 0:
                    old[b, S.cache_slot(ln - 1, slots, sinks)] = src[b, ln - 1]
            assert torch.equal(c.view(torch.int16) if c.is_contiguous() else c.contiguous().view(torch.int16),
                               old.contiguous().view(torch.int16))
    return r


@pytest.mark.parametrize("B,Hq,Hk,slots,left,sinks,lens", [
    (1, 1, 1, 2, 0, 1, [1]),
    (1, 8, 1, 40, 30, 4, [29]),
    (3, 4, 2, 68, 63, 4, [1, 68, 500]),             # ring of exactly the window: not full, full, wrapped
    (4, 6, 6, 300, 2 ** 31 - 1, 0, [0, 1, 299, 300]),  # a slot per token, an idle request
    (2, 10, 2, 200, 50, 3, [150, 1000]),            # a ring wider than the window
    (2, 4, 4, 50, 200, 10, [60, 49]),               # a window wider than the ring: what is stored is seen
    (5, 16, 1, 1100, 1023, 64, [5000, 3, 64, 65, 1087]),
    (1, 48, 48, 700, 600, 4, [700]),
    (2, 24, 2, 3000, 2 ** 31 - 1, 4, [2999, 1777]),
    (1, 5, 1, 9000, 8999, 0, [8765]),
    (1, 64, 1, 513, 400, 2, [777]),                 # 64 query heads on one key head
])
@pytest.mark.parametrize("layout", ["slots", "heads"])
def test_decode(B, Hq, Hk, slots, left, sinks, lens, layout):
    _decode_case(B, Hq, Hk, slots, left, sinks, lens, layout)


def test_decode_without_new_tokens_and_with_a_scale():
    _decode_case(2, 4, 2, 100, 60, 4, [30, 90], new=False, scale=0.4)


def test_decode_negative_length_is_reported():
    q, c = _rand(1, 2, 2, 64, dtype=BF), _rand(2, 2, 8, 1, 64, dtype=BF)
    ws = L.window_attention_decode_workspace(q, c)
    r = L.window_attention_decode(q, c, c.clone(), _ints([-3, 4]), left=9, workspace=ws, check_status=False)
    assert torch.all(r["out"][0] == 0)
    assert L.ttt_mlp_status(ws) == L.TTT_ERR_INVALID_ARG and L.ttt_mlp_status(ws) == L.TTT_OK


def test_decode_with_fewer_slots_than_sinks():
    _decode_case(2, 2, 1, 3, 5, 8, [3, 2])
    q, c = _rand(1, 2, 2, 64, dtype=BF), _rand(2, 2, 8, 1, 64, dtype=BF)
    ws = L.window_attention_decode_workspace(q, c)
    r = L.window_attention_decode(q, c, c.clone(), _ints([9, 8]), left=9, sinks=8, workspace=ws, check_status=False)
    assert torch.all(r["out"][0] == 0) and torch.any(r["out"][1] != 0)
    assert L.ttt_mlp_status(ws) == L.TTT_ERR_INVALID_ARG


def test_decode_offsets_past_32_bits():
    """A cache whose last slots lie past 2^31 elements (a strided view: little of it is ever touched)."""
    slots, B = 5, 2
    big = torch.empty(2 ** 31 + 4096, dtype=BF, device="cuda")
    ck = big.as_strided((B, slots, 1, 64), (2 ** 31, 64, 64, 1))
    ck[:] = _rand(3, B, slots, 1, 64, dtype=BF)
    cv = ck                                    # keys as values
    q = _rand(4, B, 2, 64, dtype=BF)
    r = L.window_attention_decode(q, ck, cv, _ints([5, 4]), left=10)
    c = _np(ck)
    want, tol = S.window_decode(_np(q), lambda b, u: c[b, u], lambda b, u: c[b, u], [5, 4], 10, 0, slots)
    _within(r["out"], want, tol, "decode")


def test_decode_in_a_graph_grows_with_its_lengths():
    B, Hq, Hk, slots, left, sinks = 3, 4, 2, 20, 15, 4
    ck, cv = (torch.full((B, slots, Hk, 64), NAN, dtype=BF, device="cuda") for _ in range(2))
    q, kn, vn, out = (torch.zeros(B, h, 64, dtype=BF, device="cuda") for h in (Hq, Hk, Hk, Hq))
    lens, ws = _ints([1, 1, 1]), L.window_attention_decode_workspace(q, ck)

    def step():
        L.window_attention_decode(q, ck, cv, lens, left=left, sinks=sinks, k_new=kn, v_new=vn, out=out, workspace=ws,
                                  check_status=False)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    K, V, Q = _rand(1, 50, B, Hk, 64, dtype=BF), _rand(2, 50, B, Hk, 64, dtype=BF), _rand(3, 50, B, Hq, 64, dtype=BF)
    full = []
    for t in range(50):
        lens.fill_(t + 1)
        q.copy_(Q[t]), kn.copy_(K[t]), vn.copy_(V[t])
        graph.replay()
        full.append(out.clone())
    assert L.ttt_mlp_status(ws) == L.TTT_OK
    for b in range(B):          # the prefill form over the whole sequence sees the same keys
        ref = S.window_attention(_np(Q[:, b]), _np(K[:, b]), _np(V[:, b]), left, 0, sinks)
        _within(torch.stack(full)[:, b], ref["out"], ref["out_tol"], "token by token")


# ---------------------------------------------------------------- gated recurrence
SCAN = [   # cu, D, padding rows
    ([0, 1], 8, 0),
    ([0, 2], 24, 0),
    ([0, 63], 64, 0),
    ([0, 64], 40, 0),
    ([0, 65], 128, 0),
    ([0, 1000], 72, 0),
    ([0, 5000], 16, 0),
    ([0, 0], 16, 0),
    ([0, 0, 3, 3, 70, 71, 200, 200], 56, 19),
    ([0, 64, 128, 192, 256], 64, 0),
    ([0, 900, 1000, 2500], 136, 1),
]


def _scan_inputs(cu, D, pad, dtype, seed=0, bias=3.0):
    dt = BF if dtype == "bf16" else torch.float32
    T, n = cu[-1] + pad, len(cu) - 1
    f = (_rand(seed, T, D) * 1.5 + torch.linspace(0, 2 * bias, D, device="cuda")).to(dt)
    x, dy = _rand(seed + 1, T, D, dtype=dt), _rand(seed + 2, T, D, dtype=dt)
    for t in (f, x, dy):
        t[cu[-1]:] = NAN
    return f, x, dy, _rand(seed + 3, n, D), _rand(seed + 4, n, D), (_ints(cu) if n > 1 or pad else None)


@pytest.mark.parametrize("cu,D,pad", SCAN, ids=str)
@pytest.mark.parametrize("form,dtype,dirs", [("sum", "f32", "fwd"), ("convex", "bf16", "rev"), ("unit", "f32", "rev"),
                                             ("unit", "bf16", "fwd"), ("convex", "f32", "fwd"), ("sum", "bf16", "rev")])
def test_gated_scan(cu, D, pad, form, dtype, dirs):
    f, x, dy, h0, dhT, dcu = _scan_inputs(cu, D, pad, dtype)
    ref = S.gated_scan(_np(f), _np(x), form, dirs == "rev", cu, _np(h0), _np(dy), _np(dhT), dtype)
    how = dict(form=form, dirs=dirs, cu=dcu, h0=h0)
    y = torch.full_like(x, 7.0)
    r = L.gated_scan(f, x, y=y, want_state=True, want_chunk_states=True, **how)
    _within(r["y"], ref["y"], ref["y_tol"], "y")
    _within(r["h_T"], ref["hT"], ref["hT_tol"], "h_T")
    df, dx = torch.full_like(x, 7.0), torch.full_like(x, 7.0)
    b = L.gated_scan_backward(f, x, dy, r["chunk_states"], dh_T=dhT, df=df, dx=dx, want_dh0=True, **how)
    for n in ("df", "dx", "dh0"):
        _within(b[n], ref[n], ref[n + "_tol"] + 1e-30, n)
    if pad:
        assert all(torch.all(t[cu[-1]:] == 7.0) for t in (y, df, dx))
    r2 = L.gated_scan(f, x, want_state=True, want_chunk_states=True, **how)
    b2 = L.gated_scan_backward(f, x, dy, r2["chunk_states"], dh_T=dhT, want_dh0=True, **how)
    n = cu[-1]
    assert torch.equal(r2["y"][:n], y[:n]) and torch.equal(r2["h_T"], r["h_T"])
    assert torch.equal(b2["df"][:n], df[:n]) and torch.equal(b2["dx"][:n], dx[:n]) and torch.equal(b2["dh0"], b["dh0"])


@pytest.mark.parametrize("dirs", ["fwd", "rev"])
def test_gated_scan_without_optional_states(dirs):
    cu = [0, 40, 40, 300]
    f, x, dy, _, _, dcu = _scan_inputs(cu, 32, 0, "f32")
    ref = S.gated_scan(_np(f), _np(x), "convex", dirs == "rev", cu, None, _np(dy))
    r = L.gated_scan(f, x, dirs=dirs, cu=dcu, want_chunk_states=True)
    b = L.gated_scan_backward(f, x, dy, r["chunk_states"], dirs=dirs, cu=dcu)
    _within(r["y"], ref["y"], ref["y_tol"], "y")
    for n in ("df", "dx"):
        _within(b[n], ref[n], ref[n + "_tol"] + 1e-30, n)


@pytest.mark.parametrize("form", ["sum", "convex", "unit"])
def test_gated_scan_extreme_gates(form):
    """Gates that never forget, forget at once, and infinite logits: no NaN, and 1 - a keeps its scale."""
    T, D = 300, 16
    f = torch.tensor([-math.inf, -100.0, -30.0, -5.0, 0.0, 5.0, 17.0, 30.0, 60.0, 88.0, 100.0, math.inf, 1e30, -1e30, 3.0, -3.0],
                     device="cuda").expand(T, D).contiguous()
    x, dy = _rand(1, T, D), _rand(2, T, D)
    ref = S.gated_scan(_np(f), _np(x), form, False, None, None, _np(dy))
    r = L.gated_scan(f, x, form=form, want_chunk_states=True)
    b = L.gated_scan_backward(f, x, dy, r["chunk_states"], form=form)
    # In fp32, 1 - a below 2^-126 (f above 87) may become zero: an absolute error of 2^-126 in 1 - a and of
    # sqrt(2 * 2^-126) < 2^-62 in sqrt(1 - a^2) and in ds/df.  y sums at most T such errors times |x|, a
    # gradient one of them times l (at most T |dy|) and x, beside l times an error of y times 1 - a.
    under = T * 2.0 ** -62 * float(x.abs().max())
    _within(r["y"], ref["y"], ref["y_tol"] + under, "y")
    for n in ("df", "dx"):
        _within(b[n], ref[n], ref[n + "_tol"] + T * float(dy.abs().max()) * (2.0 ** -62 * (1 + float(x.abs().max())) + under), n)


def test_gated_scan_strided_and_in_a_graph_on_another_stream():
    T, D = 700, 48
    wide = _rand(3, T, 3 * D, dtype=BF)
    f, x = wide[:, :D], wide[:, D:2 * D]
    want = L.gated_scan(f.contiguous(), x.contiguous(), want_state=True)
    ws, out, hT = L.gated_scan_workspace(x), torch.zeros(T, 2 * D, dtype=BF, device="cuda"), torch.zeros(1, D, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        L.gated_scan(f, x, y=out[:, D:], h_T=hT, workspace=ws, check_status=False)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            L.gated_scan(f, x, y=out[:, D:], h_T=hT, workspace=ws, check_status=False)
        out.zero_(), hT.zero_()
        for _ in range(3):
            graph.replay()
    s.synchronize()
    assert torch.equal(out[:, D:], want["y"]) and torch.equal(hT, want["h_T"]) and torch.all(out[:, :D] == 0)
    assert L.ttt_mlp_status(ws) == L.TTT_OK


def test_gated_scan_bad_offsets_and_non_finite_inputs_are_reported():
    f, x = _rand(1, 100, 16), _rand(2, 100, 16)
    for bad in ([0, 60, 50, 100], [0, 10, 20, 101], [-1, 10, 20, 100], [5, 10, 20, 100]):
        with pytest.raises(L.TTTError) as e:
            L.gated_scan(f, x, cu=_ints(bad))
        assert e.value.status == L.TTT_ERR_INVALID_ARG
    x[50, 3] = NAN
    r = L.gated_scan(f, x, check_status=False)
    assert L.ttt_mlp_status(r["workspace"]) == L.TTT_ERR_NONFINITE
    assert torch.isfinite(r["y"][:50]).all() and torch.isfinite(r["y"][:, 4:]).all()


@pytest.mark.parametrize("form", ["sum", "convex", "unit"])
@pytest.mark.parametrize("B,D,dtype", [(1, 8, "f32"), (3, 1000, "bf16"), (70, 520, "f32")])
def test_step_walks_the_scan(form, B, D, dtype):
    dt = BF if dtype == "bf16" else torch.float32
    T = 12
    f, x, h0 = _rand(1, B, T, D, dtype=dt), _rand(2, B, T, D, dtype=dt), _rand(3, B, D)
    h = h0.clone()
    ys = []
    for t in range(T):
        y, _ = L.gated_scan_step(f[:, t], x[:, t], h, form=form, h_out=h)
        ys.append(y)
    cu = [T * i for i in range(B + 1)]
    ref = S.gated_scan(_np(f).reshape(B * T, D), _np(x).reshape(B * T, D), form, False, cu, _np(h0), dtype=dtype)
    _within(torch.stack(ys, 1).reshape(B * T, D), ref["y"], ref["y_tol"], "y")
    _within(h, ref["hT"], ref["hT_tol"], "h")


# ---------------------------------------------------------------- arguments seen from Python
def test_python_checks():
    q, k = _rand(1, 10, 2, 64, dtype=BF), _rand(2, 10, 2, 64, dtype=BF)
    for call in (lambda: L.window_attention(q.float(), k, k, left=3),
                 lambda: L.window_attention(q, k, k[:9], left=3),
                 lambda: L.window_attention(q, k, k.cpu(), left=3),
                 lambda: L.window_attention(q, k, k, left=3, cu_q=_ints([0, 10])),
                 lambda: L.window_attention(q, k, k, left=3, cu_q=_ints([0, 10]).long(), cu_k=_ints([0, 10]).long()),
                 lambda: L.window_attention(q.transpose(0, 1), k, k, left=3),
                 lambda: L.gated_scan(q[:, 0], k[:, 0].float()),
                 lambda: L.gated_scan_step(q[:, 0], k[:, 0], k[:, 0]),
                 lambda: L.rope(q, torch.arange(10, device="cuda")),
                 lambda: L.rope(q, scaling={"factor": 2.0, "kind": "other"}),
                 lambda: L.window_attention_decode(q, k[None], k[None], _ints([3] * 10), left=3)):
        with pytest.raises(ValueError):
            call()


# ---------------------------------------------------------------- together
def test_a_block_of_the_operators_as_it_is_used():
    """rotary positions on a fused projection, window attention with the residual, the gated recurrence on its
    output; then the same tokens one at a time through the single-token forms."""
    T, Hq, Hk, left, sinks = 150, 4, 2, 40, 3
    W = Hq * 64
    qkv, x, f = _rand(1, T, Hq + 2 * Hk, 64, dtype=BF), _rand(2, T, W, dtype=BF), (_rand(3, T, W) + 2).to(BF)
    turned = L.rope(qkv[:, :Hq + Hk])
    q, k, v = turned[:, :Hq], turned[:, Hq:], qkv[:, Hq + Hk:]
    a = L.window_attention(q, k, v, left=left, sinks=sinks, residual=x.view(T, Hq, 64))
    whole = L.gated_scan(f, a["out"].view(T, W), want_state=True)

    ck, cv = (torch.full((1, sinks + left + 1, Hk, 64), NAN, dtype=BF, device="cuda") for _ in range(2))
    h, rows, ws = torch.zeros(1, W, device="cuda"), [], None
    att = []
    for t in range(T):
        row = L.rope(qkv[t:t + 1, :Hq + Hk], pos0=t)
        assert torch.equal(row, turned[t:t + 1])
        d = L.window_attention_decode(row[:, :Hq], ck, cv, _ints([t + 1]), left=left, sinks=sinks, k_new=row[:, Hq:],
                                      v_new=qkv[t:t + 1, Hq + Hk:],
                                      workspace=ws)
        ws = d["workspace"]
        att.append(d["out"])
        y, _ = L.gated_scan_step(f[t:t + 1], a["out"][t:t + 1].view(1, W), h, h_out=h)
        rows.append(y)
    ref = S.window_attention(_np(q), _np(k), _np(v), left, 0, sinks)
    _within(torch.cat(att), ref["out"], ref["out_tol"], "token by token")
    want = ref["out"] + _np(x).reshape(T, Hq, 64)
    _within(a["out"], want, ref["out_tol"] + 2.0 ** -8 * np.abs(want), "block")
    scan = S.gated_scan(_np(f), _np(a["out"]).reshape(T, W), "convex", dtype="bf16")
    _within(whole["y"], scan["y"], scan["y_tol"], "scan")
    _within(torch.cat(rows), scan["y"], scan["y_tol"], "scan, token by token")
