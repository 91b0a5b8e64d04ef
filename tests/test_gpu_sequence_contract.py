"""What the sequence operators promise beyond their formulas: unseen places may hold anything, values that are not finite
are reported where they take part, numbers and streams are taken as they are at the call."""
import math

import pytest
import torch

from test_rnn_layer_b200 import tttmlp as L

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
NAN, INF = float("nan"), math.inf


def _rand(seed, *shape, dtype=torch.float32):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(*shape, generator=g, device="cuda").to(dtype)


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


# ---------------------------------------------------------------- unseen places
def _garbage(kind, like):
    """Finite values of about 3e38 of both signs, or any 16 bits (NaN and infinities among them)."""
    g = torch.Generator(device="cuda").manual_seed(17)
    if kind == "huge":
        return torch.where(torch.rand(like.shape, generator=g, device="cuda") < 0.5, -3e38, 3e38).to(BF)
    return torch.randint(-2 ** 15, 2 ** 15, like.shape, generator=g, device="cuda", dtype=torch.int32).to(torch.int16).view(BF)


LENGTHS = list(range(1, 49)) + [127, 128, 129, 200]     # ends at every place of sixteen keys, and about a tile's end


@pytest.mark.parametrize("kind", ["huge", "bits"])
@pytest.mark.parametrize("left,right,sinks", [(1000, 0, 0), (20, 0, 3), (9, 9, 0)])
@pytest.mark.parametrize("place", ["padding", "neighbour"])
def test_other_sequences_and_padding_change_no_bit(place, left, right, sinks, kind):
    """A sequence's results do not depend on what lies behind the last one, nor on its neighbours."""
    lens = LENGTHS if place == "neighbour" else [70, 45]
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    T = cu[-1] + 150
    q, k, v, g = (_rand(i, T, H, 64, dtype=BF) for i, H in enumerate((4, 2, 2, 4)))
    mask = dict(left=left, right=right, sinks=sinks, cu_q=_ints(cu), cu_k=_ints(cu), check_status=False)

    def run():
        r = L.window_attention(q, k, v, want_lse=True, **mask)
        b = L.window_attention_backward(q, k, v, r["out"], r["lse"], g, **mask)
        return [r["out"], r["lse"].t(), b["dq"], b["dk"], b["dv"]], r["workspace"]

    want, _ = run()
    mine = torch.zeros(T, dtype=torch.bool, device="cuda")
    for s in range(0, len(lens), 2 if place == "neighbour" else 1):
        mine[cu[s]:cu[s + 1]] = True
    for t in (q, k, v, g):
        t[~mine] = _garbage(kind, t)[~mine]
    got, ws = run()
    for n, a, b in zip(("out", "lse", "dq", "dk", "dv"), got, want):
        assert torch.equal(a[mine], b[mine]), n
    if place == "padding":
        assert L.ttt_mlp_status(ws) == L.TTT_OK


@pytest.mark.parametrize("kind", ["huge", "bits"])
@pytest.mark.parametrize("at", range(130, 146))
def test_a_value_changes_only_the_rows_that_see_it(at, kind):
    T, left, sinks = 300, 20, 3
    q, k, v = (_rand(i, T, 2, 64, dtype=BF) for i in range(3))
    want = L.window_attention(q, k, v, left=left, sinks=sinks, want_lse=True)
    k[at], v[at] = _garbage(kind, k)[at], _garbage(kind, v)[at]
    got = L.window_attention(q, k, v, left=left, sinks=sinks, want_lse=True, check_status=False)
    rest = torch.ones(T, dtype=torch.bool, device="cuda")
    rest[at:at + left + 1] = False
    assert torch.equal(got["out"][rest], want["out"][rest]) and torch.equal(got["lse"][:, rest], want["lse"][:, rest])


@pytest.mark.parametrize("seg", [9, 16, 100, 130, 143])
def test_segment_attention_takes_no_part_of_the_next_segment(seg):
    T, H = 3 * seg, 2
    q, k, v = (_rand(i, T, H * 64, dtype=BF) for i in range(3))

    def run():
        out = torch.empty(T, H * 64, dtype=BF, device="cuda")
        ws = torch.empty(L.ttt_seg_attention_workspace_size(), dtype=torch.uint8, device="cuda")
        L.check(L.ttt_seg_attention(T, H, 64, seg, q, k, v, H * 64, None, out, H * 64, 0, T, ws, ws.numel()), "ttt_seg_attention")
        torch.cuda.synchronize()
        return out

    want = run()
    v[seg:2 * seg] = _garbage("huge", v)[seg:2 * seg]
    got = run()
    rest = torch.ones(T, dtype=torch.bool, device="cuda")
    rest[seg:2 * seg] = False
    assert torch.equal(got[rest], want[rest])


# ---------------------------------------------------------------- values that are not finite
@pytest.mark.parametrize("at", range(64, 81))
@pytest.mark.parametrize("left", [0, 3])
def test_a_key_that_is_nan_makes_its_rows_nan_at_every_place_of_a_tile(left, at):
    T = 150
    q, k, v = (_rand(i, T, 1, 64, dtype=BF) for i in range(3))
    want = L.window_attention(q, k, v, left=left, want_lse=True)
    k[at, 0, 5] = NAN
    got = L.window_attention(q, k, v, left=left, want_lse=True, check_status=False)
    assert L.ttt_mlp_status(got["workspace"]) == L.TTT_ERR_NONFINITE
    rows = torch.zeros(T, dtype=torch.bool, device="cuda")
    rows[at:at + left + 1] = True
    assert got["out"][rows].isnan().all() and got["lse"][:, rows].isnan().all()
    assert torch.equal(got["out"][~rows], want["out"][~rows]) and torch.equal(got["lse"][:, ~rows], want["lse"][:, ~rows])


@pytest.mark.parametrize("at", range(128, 144))
def test_query_gradients_of_rows_that_see_an_infinite_key_are_nan(at):
    """Also where its score is -infinity (a weight of zero: 0 times infinity), at every place of a tile."""
    T, left = 400, 60
    q, k, v, g = (_rand(i, T, 1, 64, dtype=BF) for i in range(4))
    q[:, 0, 9] = -q[:, 0, 9].abs() - 0.125
    g *= 2.0 ** -10
    k[at, 0, 9] = INF
    r = L.window_attention(q, k, v, left=left, want_lse=True, check_status=False)
    b = L.window_attention_backward(q, k, v, r["out"], r["lse"], g, left=left, check_status=False)
    assert L.ttt_mlp_status(b["workspace"]) == L.TTT_ERR_NONFINITE
    rows = torch.zeros(T, dtype=torch.bool, device="cuda")
    rows[at:at + left + 1] = True
    assert b["dq"][rows].isnan().all() and torch.isfinite(b["dq"][~rows]).all()


@pytest.mark.parametrize("at", [8, 78, 79])
@pytest.mark.parametrize("which", ["q", "k"])
@pytest.mark.parametrize("residual", [False, True])
def test_rows_whose_only_scores_are_minus_infinity_are_nan(which, at, residual):
    """Such a row sees keys: it is not an empty one."""
    T = 150
    q, k, v, x = (_rand(i, T, 1, 64, dtype=BF) for i in range(4))
    q[at, 0, 9], k[at, 0, 9] = -1.5, 1.5
    how = dict(left=0, want_lse=True, residual=x if residual else None)
    want = L.window_attention(q, k, v, **how)
    (q if which == "q" else k)[at, 0, 9] *= INF
    got = L.window_attention(q, k, v, check_status=False, **how)
    assert L.ttt_mlp_status(got["workspace"]) == L.TTT_ERR_NONFINITE
    rest = torch.arange(T, device="cuda") != at
    assert got["out"][at].isnan().all() and got["lse"][0, at].isnan()
    assert torch.equal(got["out"][rest], want["out"][rest]) and torch.equal(got["lse"][:, rest], want["lse"][:, rest])


@pytest.mark.parametrize("left", [0, 40])
def test_rows_that_see_no_key_stay_empty(left):
    """More queries than keys: rows in front of the first key, with queries that are not finite among them."""
    Tq, Tk = 300, 100
    q, k, v = _rand(0, Tq, 2, 64, dtype=BF), _rand(1, Tk, 1, 64, dtype=BF), _rand(2, Tk, 1, 64, dtype=BF)
    q[7, 1, 3], q[150, 0, 0] = NAN, -INF
    r = L.window_attention(q, k, v, left=left, want_lse=True)
    assert not r["out"][:200].any() and (r["lse"][:, :200] == -INF).all() and torch.isfinite(r["lse"][:, 200:]).all()


@pytest.mark.parametrize("at", [1, 14, 15, 33])
def test_a_score_of_minus_infinity_beside_others_is_a_weight_of_zero(at):
    """As in the formula: the same bits as a score that is very low."""
    T = 60
    q, k, v = (_rand(i, T, 1, 64, dtype=BF) for i in range(3))
    q[:, 0, 9] = -q[:, 0, 9].abs() - 0.125
    how = dict(left=100, want_lse=True)
    k[at, 0, 9] = 1e30
    want = L.window_attention(q, k, v, **how)
    k[at, 0, 9] = INF
    got = L.window_attention(q, k, v, check_status=False, **how)
    assert torch.equal(got["out"], want["out"]) and torch.equal(got["lse"], want["lse"])


@pytest.mark.parametrize("which", ["q", "k"])
def test_decode_of_scores_of_minus_infinity(which):
    """One visible key: NaN and reported, beside an idle request; among others: a weight of zero."""
    B, slots, Hq = 4, 40, 2
    q, ck, cv = _rand(0, B, Hq, 64, dtype=BF), _rand(1, B, slots, 1, 64, dtype=BF), _rand(2, B, slots, 1, 64, dtype=BF)
    lens = _ints([0, 1, 30, 40])
    q[:, 0, 9], ck[:, 0, 0, 9] = -1.5, 1.5
    ck[2, 0, 0, 9] = 1e30
    want = L.window_attention_decode(q, ck, cv, lens, left=100)
    (q[1, 0] if which == "q" else ck[1, 0, 0])[9] *= INF
    ck[2, 0, 0, 9] = INF if which == "k" else 1e30
    got = L.window_attention_decode(q, ck, cv, lens, left=100, check_status=False)
    assert L.ttt_mlp_status(got["workspace"]) == L.TTT_ERR_NONFINITE
    assert got["out"][1, 0].isnan().all() and not got["out"][0].any()
    assert torch.equal(got["out"][2, 0], want["out"][2, 0]) and torch.equal(got["out"][3], want["out"][3])


# ---------------------------------------------------------------- streams and numbers
def test_a_raw_stream_handle_orders_every_fill():
    """Buffers that the functions make and fill themselves are filled on the stream that the kernels run on."""
    T, D = 500, 64
    cu = _ints([0, 200, 450])
    q, k, v, g = (_rand(i, T, 2, 64, dtype=BF) for i in range(4))
    f, x, dy = (_rand(9 + i, T, D, dtype=BF) for i in range(3))
    mask = dict(left=60, cu_q=cu, cu_k=cu)
    cache = torch.stack([k[:8], v[:8]])
    lens = _ints([5])
    w0 = L.window_attention(q, k, v, want_lse=True, **mask)
    s0 = L.gated_scan(f, x, cu=cu, want_chunk_states=True)

    def run(stream):
        how = dict(check_status=False, stream=stream)
        w = L.window_attention(q, k, v, want_lse=True, **mask, **how)
        b = L.window_attention_backward(q, k, v, w0["out"], w0["lse"], g, **mask, **how)
        s = L.gated_scan(f, x, cu=cu, **how)
        t = L.gated_scan_backward(f, x, dy, s0["chunk_states"], cu=cu, **how)
        d = L.window_attention_decode(q[:1], cache[:1], cache[1:], lens, left=9, **how)
        return [w["out"], w["lse"], b["dq"], b["dk"], b["dv"], s["y"], t["df"], t["dx"], d["out"]]

    want = run(None)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    torch.cuda._sleep(400_000_000)      # a fifth of a second on the current stream
    got = run(side.cuda_stream)
    assert not torch.cuda.current_stream().query()
    torch.cuda.synchronize()
    for i, (a, b) in enumerate(zip(got, want)):
        assert torch.equal(a, b), i


@pytest.mark.parametrize("handle", [0, 1, 2])   # the default stream's two names, this thread's
def test_streams_by_their_fixed_handles(handle):
    q = _rand(0, 40, 1, 64, dtype=BF)
    cu = _ints([0, 30])
    a, b = (L.window_attention(q, q, q, left=3, cu_q=cu, cu_k=cu, stream=s)["out"] for s in (handle, None))
    torch.cuda.synchronize()
    assert torch.equal(a, b)


def test_the_capturing_stream_by_its_handle():
    """Inside a capture: fills and outputs belong to the graph, and a replay on new inputs gives what a call gives."""
    q, k, v, g = (_rand(i, 300, 2, 64, dtype=BF) for i in range(4))
    cu = _ints([0, 120, 290])
    ws = L.window_attention_workspace(q, k, 2, backward=True)
    mask = dict(left=50, cu_q=cu, cu_k=cu, check_status=False)

    def run(ws, stream):
        r = L.window_attention(q, k, v, want_lse=True, workspace=ws, stream=stream, **mask)
        b = L.window_attention_backward(q, k, v, r["out"], r["lse"], g, workspace=ws, stream=stream, **mask)
        return [r["out"], r["lse"], b["dq"], b["dk"], b["dv"]]

    run(ws, None)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run(ws, torch.cuda.current_stream().cuda_stream)
    for t in (q, k, v, g):
        t.copy_(_rand(9, *t.shape, dtype=BF) * (1 + t.float().mean()))
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    got = [t.clone() for t in out]
    for a, b in zip(got, run(None, None)):
        assert torch.equal(a, b)


def test_numbers_are_taken_at_the_call():
    """A number given as a tensor of one element that changes between calls."""
    q, k, v = (_rand(i, 50, 2, 64, dtype=BF) for i in range(3))
    cache, lens = torch.stack([k[:8], v[:8]]), _ints([6])
    scale, base, factor, left = torch.tensor(0.125), torch.tensor(100.0), torch.tensor(1.0), torch.tensor(5)

    def run(scale, base, factor, left):
        return [L.window_attention(q, k, v, left=left, scale=scale)["out"],
                L.window_attention_decode(q[:1], cache[:1], cache[1:], lens, left=left, scale=scale)["out"],
                L.rope(q, base=base, scaling={"kind": "linear", "factor": factor})]

    for s, b, f, n in ((0.125, 100.0, 1.0, 5), (0.5, 1000.0, 4.0, 2)):
        scale.fill_(s), base.fill_(b), factor.fill_(f), left.fill_(n)
        for x, y in zip(run(scale, base, factor, left), run(s, b, f, n)):
            assert torch.equal(x, y), (s, b, f, n)


def test_numbers_past_32_bits_are_refused():
    """The interface's integers have 32 bits: a larger number must not lose its upper ones."""
    q = _rand(0, 30, 1, 64, dtype=BF)
    cache, lens = q[:16][None], _ints([6])
    for n in (2 ** 32, 2 ** 32 + 5, 2 ** 31, -2 ** 32 + 1):
        for call in (lambda: L.window_attention(q, q, q, left=n), lambda: L.window_attention(q, q, q, left=3, right=n),
                     lambda: L.window_attention(q, q, q, left=3, sinks=n), lambda: L.rope(q, pos0=n), lambda: L.rope(q, rot=n),
                     lambda: L.window_attention_decode(q[:1], cache, cache, lens, left=n),
                     lambda: L.window_attention_decode(q[:1], cache, cache, lens, left=3, sinks=n)):
            with pytest.raises((ValueError, L.TTTError)):
                call()


def test_keys_of_another_head_width_are_refused():
    q, k = _rand(0, 30, 2, 64, dtype=BF), _rand(1, 30, 2, 128, dtype=BF)
    r = L.window_attention(q, q, q, left=3, want_lse=True)
    with pytest.raises(ValueError):
        L.window_attention(q, k, k, left=3)
    with pytest.raises(ValueError):
        L.window_attention_backward(q, k, k, r["out"], r["lse"], q.clone(), left=3)


def test_status_waits_for_its_own_stream_only():
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    ws.view(torch.int32)[0] = 1
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(400_000_000)      # a fifth of a second on the default stream
    assert L.ttt_mlp_status(ws, side) == L.TTT_ERR_NONFINITE
    assert not torch.cuda.current_stream().query()
    assert L.ttt_mlp_status(ws, side) == L.TTT_OK
    torch.cuda.synchronize()
    assert not ws.any()


# ---------------------------------------------------------------- gated recurrence
@pytest.mark.parametrize("dirs", ["fwd", "rev"])
@pytest.mark.parametrize("form", ["sum", "convex", "unit"])
@pytest.mark.parametrize("value", [INF, -INF])
def test_scan_takes_infinite_logits_as_open_and_closed_gates(value, form, dirs):
    """a = 1 or 0: every output stays finite, and what no such gate touches keeps its bits."""
    cu, D, at = [0, 300, 700, 1500], 72, 500
    T = cu[-1]
    f, x, dy, h0 = _rand(1, T, D) + 2, _rand(2, T, D), _rand(3, T, D), _rand(4, 3, D)
    how = dict(form=form, dirs=dirs, cu=_ints(cu))

    def both():
        r = L.gated_scan(f, x, h0=h0, want_state=True, want_chunk_states=True, **how)
        b = L.gated_scan_backward(f, x, dy, r["chunk_states"], h0=h0, want_dh0=True, **how)
        return [r["y"], b["df"], b["dx"]], [r["h_T"], b["dh0"]]

    f[at, 5] = 200.0 if value > 0 else -200.0
    rows0, states0 = both()
    f[at, 5] = value
    rows, states = both()           # (the status is looked at: nothing is reported)
    for a, b in zip(rows + states, rows0 + states0):
        assert torch.equal(a, b) and torch.isfinite(a).all()
    y, df, dx = rows
    prev = y[at - 1, 5] if dirs == "fwd" else y[at + 1, 5]
    gain = {"sum": 1.0, "convex": 0.0, "unit": 0.0}[form] if value > 0 else 1.0
    # gates: a and s(a) to 2^-20; the closed gate's a is below 2^-115
    want = (prev if value > 0 else 0.0) + gain * x[at, 5]
    assert abs(float(y[at, 5] - want)) <= 2.0 ** -20 * (abs(float(prev)) + abs(float(x[at, 5])))
    assert abs(float(df[at, 5])) <= 2.0 ** -100
