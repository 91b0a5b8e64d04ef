"""What is measured of the sequence operators beside the TTT layer: rotary positions, attention with a
sliding window and first tokens that stay visible (training, prefill and single-token form), and the gated
linear recurrence (training, prefill and single-token form).

`run` computes an operator in its plain form (elementary torch operations in 32 bits, angles in 64) or, where
`own` is true, through the library's calls.  `exact` computes the definition in 64 bits.

Definitions.
  rope: pair (x, y) of frequency i of a head turns by pos * freq_i:  (x cos - y sin, x sin + y cos); the
    pairs are (j, j + rot/2) ("half") or (2 j, 2 j + 1) ("interleaved") of the head's first `rot` columns.
  window attention: query i of a sequence with nq queries and nk keys has position p = nk - nq + i and sees
    key u where u <= p + right and (u >= p - left or u < sinks); a row that sees nothing is zero, its
    log-sum-exp minus infinity.  Query head h reads key head h // (Hq / Hk).
  gated recurrence: a = sigmoid(f), h_t = a_t h_{t-1} + s(a_t) x_t with s = 1 ("sum"), 1 - a ("convex") or
    sqrt(1 - a^2) ("unit"), per channel, over each sequence of the packed rows, forward or in reverse.
Rows behind the last sequence are not read and stay as they were.
"""
import math

import torch

own = False

D = 64                      # head width of this library's attention
INF = float("inf")


# ------------------------------------------------------------------------------------------------ cases
def listed():
    return [
        # rotary positions of a long training sequence's queries or keys, every column of 48 heads
        dict(name="rope-train", op="rope", T=32768, heads=48, d=64, rot=64, layout="half", scaling="none",
             dtype="bf16", inverse=False, far=False),
        # one token of each of 64 requests, 32 query and 8 key heads in one array, far positions, long-context scaling
        dict(name="rope-step", op="rope", T=64, heads=40, d=64, rot=32, layout="interleaved", scaling="ramp",
             dtype="f32", inverse=False, far=True),
        # prefill of one long document
        dict(name="attn-prefill", op="attn", seqs=1, rows=32768, prefix=0, Hq=32, Hk=8, left=4095, right=0, sinks=4,
             train=False, pad=0),
        # prefill of several requests of odd lengths whose first parts are cached already, padding rows behind them
        dict(name="attn-prefill-ragged", op="attn", seqs=13, rows=5003, prefix=700, Hq=12, Hk=4, left=1023, right=0,
             sinks=4, train=False, pad=93),
        # training on one long sequence, shared key heads
        dict(name="attn-train", op="attn", seqs=1, rows=16384, prefix=0, Hq=16, Hk=4, left=1023, right=0, sinks=16,
             train=True, pad=0),
        # training on packed sequences with a window to both sides, as the segment-local backbone has it
        dict(name="attn-train-both-sides", op="attn", seqs=5, rows=7777, prefix=0, Hq=8, Hk=8, left=255, right=255,
             sinks=1, train=True, pad=31),
        # one token of one request, its cache a ring
        dict(name="decode-one", op="decode", B=1, Hq=32, Hk=8, left=1023, sinks=4, slots=1028, longest=4100),
        # one token of each of 64 requests over long caches
        dict(name="decode-batch", op="decode", B=64, Hq=32, Hk=8, left=16383, sinks=4, slots=32768, longest=32768),
        # training on one long sequence
        dict(name="scan-train", op="scan", seqs=1, rows=102400, D=2048, form="convex", reverse=False, dtype="bf16",
             train=True, pad=0),
        # training in 32 bits on packed sequences of odd lengths, the reverse direction of a bidirectional layer
        dict(name="scan-train-ragged", op="scan", seqs=7, rows=9001, D=776, form="unit", reverse=True, dtype="f32",
             train=True, pad=55),
        # prefill of the longest sequence this library is measured on
        dict(name="scan-prefill", op="scan", seqs=1, rows=313344, D=1024, form="sum", reverse=False, dtype="bf16",
             train=False, pad=0),
        # one token of each of 32 requests
        dict(name="scan-step", op="step", B=32, D=4096, form="unit", dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["rope", "attn", "attn", "attn-train", "decode", "scan", "scan-train", "step"])
    if kind == "rope":
        d = rng.choice([64, 64, 128, 80])
        return dict(op="rope", T=_log(rng, 1, 20000), heads=rng.randint(1, 40), d=d, rot=rng.choice([d, d // 2, 16]),
                    layout=rng.choice(["half", "interleaved"]), scaling=rng.choice(["none", "linear", "base", "ramp"]),
                    dtype=rng.choice(["bf16", "f32"]), inverse=rng.random() < 0.4, far=rng.random() < 0.5)
    if kind in ("attn", "attn-train"):
        train = kind == "attn-train"
        Hk = rng.randint(1, 6)
        left = _log(rng, 1, 4096) - 1
        return dict(op="attn", seqs=rng.randint(1, 9), rows=_log(rng, 40, 12000 if not train else 7000),
                    prefix=0 if rng.random() < 0.5 else _log(rng, 1, 1500), Hq=Hk * rng.choice([1, 1, 2, 3, 4]), Hk=Hk,
                    left=left, right=0 if rng.random() < 0.6 else rng.randint(0, left), sinks=rng.choice([0, 1, 4, 130]),
                    train=train, pad=rng.randint(0, 70))
    if kind == "decode":
        Hk = rng.randint(1, 8)
        longest, sinks, left = _log(rng, 1, 20000), rng.choice([0, 1, 4, 64]), _log(rng, 1, 20000) - 1
        ring = rng.random() < 0.5
        return dict(op="decode", B=_log(rng, 1, 40), Hq=Hk * rng.choice([1, 2, 4, 5, 8]), Hk=Hk, left=left, sinks=sinks,
                    slots=sinks + left + 1 if ring else longest + rng.randint(0, 9), longest=longest)
    if kind in ("scan", "scan-train"):
        train = kind == "scan-train"
        return dict(op="scan", seqs=rng.randint(1, 9), rows=_log(rng, 40, 60000 if train else 100000),
                    D=8 * _log(rng, 1, 200), form=rng.choice(["sum", "convex", "unit"]), reverse=rng.random() < 0.5,
                    dtype=rng.choice(["bf16", "f32"]), train=train, pad=rng.randint(0, 70))
    return dict(op="step", B=_log(rng, 1, 500), D=8 * _log(rng, 1, 1000), form=rng.choice(["sum", "convex", "unit"]),
                dtype=rng.choice(["bf16", "f32"]))


# ------------------------------------------------------------------------------------------------ inputs
def _lengths(total, n, gen):
    """n lengths with sum `total`, uneven; one of them zero and one of them one where there is room for it."""
    if n == 1:
        return [total]
    cuts = sorted(torch.randint(0, total + 1, (n - 1,), generator=gen).tolist())
    out = [b - a for a, b in zip([0] + cuts, cuts + [total])]
    if n >= 4:
        for i, want in ((1, 0), (2, 1)):
            if out[0] + out[i] >= want:
                out[0] += out[i] - want
                out[i] = want
    return out


def _cu(lens):
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    return cu


def _split(case):
    """The sequences' lengths (queries, keys): a part of the case, the same for every seed."""
    gen = torch.Generator().manual_seed(1000 + case["rows"] + 7 * case["seqs"])
    lq = _lengths(case["rows"], case["seqs"], gen)
    if not case.get("prefix"):
        return lq, list(lq)
    more = torch.randint(0, 2 * case["prefix"] + 1, (case["seqs"],), generator=gen).tolist()
    lk = [q + m for q, m in zip(lq, more)]
    if case["seqs"] >= 5:
        lk[3] = max(0, lq[3] - 3)      # fewer keys than queries: the first rows see nothing
    return lq, lk


def _dtype(name):
    return torch.bfloat16 if name == "bf16" else torch.float32


ROPE_BASE, ROPE_FACTOR, ROPE_LEN, ROPE_LOW, ROPE_HIGH = 10000.0, 8.0, 4096, 1.0, 4.0


def _rope_scaling(kind):
    if kind == "none":
        return None
    if kind == "ramp":
        return dict(kind="ramp", factor=ROPE_FACTOR, length=ROPE_LEN, low=ROPE_LOW, high=ROPE_HIGH, amplitude=1.25)
    return dict(kind=kind, factor=ROPE_FACTOR)


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)

    def randn(*shape, dtype=torch.float32):
        return torch.randn(*shape, generator=g, device=dev, dtype=torch.float32).to(dtype)

    st = dict(case=case)
    if case["op"] == "rope":
        dt = _dtype(case["dtype"])
        st["x"] = randn(case["T"], case["heads"], case["d"], dtype=dt)
        if case["far"]:
            st["pos"] = torch.randint(0, 1 << 20, (case["T"],), generator=g, device=dev, dtype=torch.int32)
        else:
            st["pos"] = torch.arange(case["T"], device=dev, dtype=torch.int32) + (seed % 1000)
        st["out"] = torch.empty_like(st["x"])
    elif case["op"] == "attn":
        lq, lk = _split(case)
        st["cu_q_host"], st["cu_k_host"] = _cu(lq), _cu(lk)
        st["cu_q"] = torch.tensor(st["cu_q_host"], dtype=torch.int32, device=dev)
        st["cu_k"] = torch.tensor(st["cu_k_host"], dtype=torch.int32, device=dev)
        Tq, Tk = sum(lq) + case["pad"], sum(lk) + case["pad"]
        st["q"] = randn(Tq, case["Hq"], D, dtype=torch.bfloat16)
        kv = randn(Tk, 2 * case["Hk"], D)
        for c, n in zip(st["cu_k_host"], lk):      # the first tokens draw attention
            kv[c:c + min(4, n), :case["Hk"], 0] += 6.0
        st["q"][:, :, 0] += 2.0
        kv = kv.to(torch.bfloat16)                 # keys and values side by side, as one projection leaves them
        st["k"], st["v"] = kv[:, :case["Hk"]], kv[:, case["Hk"]:]
        st["out"] = torch.zeros_like(st["q"])
        st["lse"] = torch.zeros(case["Hq"], Tq, device=dev)
        if case["train"]:
            st["dout"] = randn(Tq, case["Hq"], D, dtype=torch.bfloat16)
            st["dq"] = torch.zeros_like(st["q"])
            st["dk"] = torch.zeros(Tk, case["Hk"], D, dtype=torch.bfloat16, device=dev)
            st["dv"] = torch.zeros(Tk, case["Hk"], D, dtype=torch.bfloat16, device=dev)
        if case["pad"]:                            # what lies behind the last sequence was never written
            for name, t in (("q", sum(lq)), ("k", sum(lk)), ("v", sum(lk)), ("dout", sum(lq))):
                if name in st:
                    st[name][t:] = float("nan")
    elif case["op"] == "decode":
        B, Hk = case["B"], case["Hk"]
        st["q"] = randn(B, case["Hq"], D, dtype=torch.bfloat16)
        lens = torch.randint(max(1, case["longest"] // 2), case["longest"] + 1, (B,), generator=g, device=dev)
        lens[0] = case["longest"]
        st["lens"] = lens.to(torch.int32)
        st["k_new"], st["v_new"] = randn(B, Hk, D, dtype=torch.bfloat16), randn(B, Hk, D, dtype=torch.bfloat16)
        st["cache_k"] = torch.empty(B, case["slots"], Hk, D, dtype=torch.bfloat16, device=dev)
        st["cache_v"] = torch.empty(B, case["slots"], Hk, D, dtype=torch.bfloat16, device=dev)
        for b in range(B):
            st["cache_k"][b] = randn(case["slots"], Hk, D)
            st["cache_v"][b] = randn(case["slots"], Hk, D)
        st["out"] = torch.empty_like(st["q"])
    elif case["op"] == "scan":
        dt = _dtype(case["dtype"])
        lens, _ = _split(case)
        st["cu_host"] = _cu(lens)
        st["cu"] = torch.tensor(st["cu_host"], dtype=torch.int32, device=dev)
        T, W = case["rows"] + case["pad"], case["D"]
        memory = torch.rand(W, generator=g, device=dev) * 6.0      # from a few tokens to several hundred
        st["f"], st["x"] = (randn(T, W) + memory).to(dt), randn(T, W, dtype=dt)
        st["h0"] = randn(case["seqs"], W)
        st["y"] = torch.zeros_like(st["x"])
        st["hT"] = torch.zeros_like(st["h0"])
        if case["train"]:
            st["dy"], st["dhT"] = randn(T, W, dtype=dt), randn(case["seqs"], W)
            st["df"], st["dx"], st["dh0"] = torch.zeros_like(st["x"]), torch.zeros_like(st["x"]), torch.zeros_like(st["h0"])
        if case["pad"]:
            for name in ("f", "x", "dy"):
                if name in st:
                    st[name][case["rows"]:] = float("nan")
    else:
        dt = _dtype(case["dtype"])
        st["f"] = (randn(case["B"], case["D"]) + 3.0).to(dt)
        st["x"], st["h"] = randn(case["B"], case["D"], dtype=dt), randn(case["B"], case["D"])
        st["y"], st["h_out"] = torch.empty_like(st["x"]), torch.empty_like(st["h"])
    return st


# ------------------------------------------------------------------------------------------------ the calls
def run(st):
    return (_run_own if own else _run_plain)(st)


def _run_own(st):
    from test_rnn_layer_b200 import tttmlp as L
    c = st["case"]
    if c["op"] == "rope":
        return L.rope(st["x"], st["pos"], rot=c["rot"], layout=c["layout"], base=ROPE_BASE,
                      scaling=_rope_scaling(c["scaling"]), inverse=c["inverse"], out=st["out"])
    if c["op"] == "attn":
        mask = dict(left=c["left"], right=c["right"], sinks=c["sinks"], cu_q=st["cu_q"], cu_k=st["cu_k"])
        if "ws" not in st:
            st["ws"] = L.window_attention_workspace(st["q"], st["k"], len(st["cu_q_host"]) - 1, backward=c["train"])
        r = L.window_attention(st["q"], st["k"], st["v"], out=st["out"], lse=st["lse"], workspace=st["ws"],
                               check_status=False, **mask)
        if not c["train"]:
            return r["out"], r["lse"]
        b = L.window_attention_backward(st["q"], st["k"], st["v"], r["out"], r["lse"], st["dout"], dq=st["dq"],
                                        dk=st["dk"], dv=st["dv"], workspace=st["ws"], check_status=False, **mask)
        return r["out"], r["lse"], b["dq"], b["dk"], b["dv"]
    if c["op"] == "decode":
        if "ws" not in st:
            st["ws"] = L.window_attention_decode_workspace(st["q"], st["cache_k"])
        L.window_attention_decode(st["q"], st["cache_k"], st["cache_v"], st["lens"], left=c["left"], sinks=c["sinks"],
                                  k_new=st["k_new"], v_new=st["v_new"], out=st["out"], workspace=st["ws"],
                                  check_status=False)
        return st["out"], st["cache_k"], st["cache_v"]
    if c["op"] == "scan":
        how = dict(form=c["form"], dirs="rev" if c["reverse"] else "fwd", cu=st["cu"], h0=st["h0"], check_status=False)
        if "ws" not in st:
            st["ws"] = L.gated_scan_workspace(st["x"], c["seqs"])
        r = L.gated_scan(st["f"], st["x"], y=st["y"], h_T=st["hT"], want_chunk_states=c["train"], workspace=st["ws"],
                         **how)
        if not c["train"]:
            return r["y"], r["h_T"]
        b = L.gated_scan_backward(st["f"], st["x"], st["dy"], r["chunk_states"], dh_T=st["dhT"], df=st["df"],
                                  dx=st["dx"], dh0=st["dh0"], workspace=st["ws"], **how)
        return r["y"], r["h_T"], b["df"], b["dx"], b["dh0"]
    return L.gated_scan_step(st["f"], st["x"], st["h"], form=c["form"], y=st["y"], h_out=st["h_out"])


# ------------------------------------------------------------------------------------------------ plain forms
def _run_plain(st):
    return dict(rope=_rope_plain, attn=_attn_plain, decode=_decode_plain, scan=_scan_plain, step=_step_plain)[
        st["case"]["op"]](st)


def _freqs(c, device):
    """Radians per position of each pair, in 64 bits."""
    i = torch.arange(c["rot"] // 2, dtype=torch.float64, device=device)
    base = ROPE_BASE
    if c["scaling"] == "base":
        base = base * ROPE_FACTOR ** (c["rot"] / (c["rot"] - 2))
    f = base ** (-2.0 * i / c["rot"])
    if c["scaling"] == "linear":
        f = f / ROPE_FACTOR
    if c["scaling"] == "ramp":
        turns = ROPE_LEN * f / (2 * math.pi)
        keep = ((turns - ROPE_LOW) / (ROPE_HIGH - ROPE_LOW)).clamp(0, 1)
        f = f * (keep + (1 - keep) / ROPE_FACTOR)
    return f


def _rope_plain(st):
    c, x = st["case"], st["x"]
    amp = 1.25 if c["scaling"] == "ramp" else 1.0
    ang = st["pos"].double()[:, None] * _freqs(c, x.device)
    cos, sin = (amp * ang.cos()).float()[:, None], (amp * ang.sin()).float()[:, None]
    if c["inverse"]:
        sin = -sin
    r, out = c["rot"], st["out"]
    v = x[..., :r].float()
    out[..., r:] = x[..., r:]
    if c["layout"] == "half":
        a, b = v[..., :r // 2], v[..., r // 2:]
        out[..., :r // 2] = (a * cos - b * sin).to(x.dtype)
        out[..., r // 2:r] = (a * sin + b * cos).to(x.dtype)
    else:
        a, b = v[..., 0::2], v[..., 1::2]
        out[..., 0:r:2] = (a * cos - b * sin).to(x.dtype)
        out[..., 1:r:2] = (a * sin + b * cos).to(x.dtype)
    return out


def _blocks(st, rows):
    """Blocks of at most `rows` query rows: (first query row, rows, first key row, key columns, mask)."""
    c, dev = st["case"], st["q"].device
    for s in range(c["seqs"]):
        q0, nq = st["cu_q_host"][s], st["cu_q_host"][s + 1] - st["cu_q_host"][s]
        k0, nk = st["cu_k_host"][s], st["cu_k_host"][s + 1] - st["cu_k_host"][s]
        for i in range(0, nq, rows):
            n = min(rows, nq - i)
            p = torch.arange(i, i + n, device=dev) + (nk - nq)
            lo = max(0, min(nk, nk - nq + i - c["left"]))
            hi = max(lo, min(nk, nk - nq + i + n + c["right"]))
            first = min(c["sinks"], lo)
            u = torch.cat([torch.arange(0, first, device=dev), torch.arange(lo, hi, device=dev)])
            seen = (u[None] <= p[:, None] + c["right"]) & ((u[None] >= p[:, None] - c["left"]) | (u[None] < c["sinks"]))
            yield q0 + i, n, k0, u, seen


def _attn_plain(st):
    c = st["case"]
    G, sc = c["Hq"] // c["Hk"], 1.0 / math.sqrt(D)
    out, lse = st["out"], st["lse"]
    if c["train"]:
        dk = torch.zeros(st["k"].shape, device=out.device)
        dv = torch.zeros(st["k"].shape, device=out.device)
    for q0, n, k0, u, seen in _blocks(st, 512):
        q = st["q"][q0:q0 + n].float().view(n, c["Hk"], G, D).permute(1, 2, 0, 3)      # Hk G n D
        k = st["k"][k0 + u].float().transpose(0, 1)[:, None]                          # Hk 1 m D
        v = st["v"][k0 + u].float().transpose(0, 1)[:, None]
        s = (q @ k.transpose(-1, -2)) * sc
        s = torch.where(seen, s, torch.full_like(s, -INF))
        if len(u):
            m = s.amax(-1, keepdim=True)
        else:
            m = torch.full((c["Hk"], G, n, 1), -INF, device=out.device)
        m0 = torch.where(m == -INF, torch.zeros_like(m), m)
        e = (s - m0).exp()
        l = e.sum(-1, keepdim=True)
        p = e / torch.where(l == 0, torch.ones_like(l), l)
        o = p @ v
        out[q0:q0 + n] = o.permute(2, 0, 1, 3).reshape(n, c["Hq"], D).to(out.dtype)
        lse[:, q0:q0 + n] = (m0 + l.log()).reshape(c["Hq"], n)
        if c["train"]:
            do = st["dout"][q0:q0 + n].float().view(n, c["Hk"], G, D).permute(1, 2, 0, 3)
            dp = do @ v.transpose(-1, -2)
            ds = p * (dp - (p * dp).sum(-1, keepdim=True)) * sc
            st["dq"][q0:q0 + n] = (ds @ k).permute(2, 0, 1, 3).reshape(n, c["Hq"], D).to(out.dtype)
            dk.index_add_(0, k0 + u, (ds.transpose(-1, -2) @ q).sum(1).transpose(0, 1))
            dv.index_add_(0, k0 + u, (p.transpose(-1, -2) @ do).sum(1).transpose(0, 1))
    if not c["train"]:
        return out, lse
    total = st["cu_k_host"][-1]
    st["dk"][:total], st["dv"][:total] = dk[:total].to(out.dtype), dv[:total].to(out.dtype)
    return out, lse, st["dq"], st["dk"], st["dv"]


def _decode_plain(st):
    c = st["case"]
    B, G, ring = c["B"], c["Hq"] // c["Hk"], c["slots"] - c["sinks"]
    pos = st["lens"].long() - 1
    here = torch.where(pos < c["slots"], pos, c["sinks"] + (pos - c["sinks"]) % max(ring, 1))
    at = torch.arange(B, device=pos.device)
    st["cache_k"][at, here], st["cache_v"][at, here] = st["k_new"], st["v_new"]
    slot = torch.arange(c["slots"], device=pos.device)
    for b0 in range(0, B, 8):
        p = pos[b0:b0 + 8, None]
        # the position that each slot holds: the last one up to p that falls on it
        u = torch.where(p < c["slots"], slot[None], torch.where(slot[None] < c["sinks"], slot[None],
                        p - (p - slot[None]) % max(ring, 1)))
        seen = (u <= p) & ((u >= p - c["left"]) | (u < c["sinks"]))
        n = p.shape[0]
        q = st["q"][b0:b0 + 8].float().view(n, c["Hk"], G, D)
        k = st["cache_k"][b0:b0 + 8].float().transpose(1, 2)
        v = st["cache_v"][b0:b0 + 8].float().transpose(1, 2)
        s = (q @ k.transpose(-1, -2)) / math.sqrt(D)
        s = torch.where(seen[:, None, None], s, torch.full_like(s, -INF))
        e = (s - s.amax(-1, keepdim=True)).exp()
        st["out"][b0:b0 + 8] = ((e / e.sum(-1, keepdim=True)) @ v).reshape(n, c["Hq"], D).to(st["out"].dtype)
    return st["out"], st["cache_k"], st["cache_v"]


def _gate(form, f):
    """(a, s, ds/da * da/df) of the logits f, elementwise."""
    a, b = torch.sigmoid(f), torch.sigmoid(-f)
    if form == "sum":
        return a, torch.ones_like(a), torch.zeros_like(a)
    if form == "convex":
        return a, b, -a * b
    return a, (b * (1 + a)).sqrt(), -a * a * (b / (1 + a)).sqrt()


def _doubling(a, b):
    """h_t = a_t h_{t-1} + b_t from h_{-1} = 0, by doubling the span that each row covers."""
    n, step = a.shape[0], 1
    while step < n:
        b2, a2 = b.clone(), a.clone()
        b2[step:] += a[step:] * b[:-step]
        a2[step:] *= a[:-step]
        a, b, step = a2, b2, 2 * step
    return b


def _scan_plain(st):
    c = st["case"]
    for s in range(c["seqs"]):
        t0, t1 = st["cu_host"][s], st["cu_host"][s + 1]
        if t0 == t1:
            st["hT"][s] = st["h0"][s]
            if c["train"]:
                st["dh0"][s] = st["dhT"][s]
            continue
        part = min(c["D"], max(8, (1 << 27) // (t1 - t0) // 8 * 8))      # columns at a time, to bound the memory
        for j in range(0, c["D"], part):
            cols = slice(j, j + part)
            walk = (lambda t: t.flip(0)) if c["reverse"] else (lambda t: t)
            f, x, h0 = walk(st["f"][t0:t1, cols].float()), walk(st["x"][t0:t1, cols].float()), st["h0"][s, cols]
            a, sc, dsc = _gate(c["form"], f)
            b = sc * x
            b[0] += a[0] * h0
            h = _doubling(a, b)
            st["y"][t0:t1, cols] = walk(h).to(st["y"].dtype)
            st["hT"][s, cols] = h[-1]
            if not c["train"]:
                continue
            g = walk(st["dy"][t0:t1, cols].float()).clone()
            g[-1] += st["dhT"][s, cols]
            nxt = torch.cat([a[1:], torch.zeros_like(a[:1])])
            lam = _doubling(nxt.flip(0), g.flip(0)).flip(0)
            before = torch.cat([h0[None], h[:-1]])
            st["df"][t0:t1, cols] = walk(lam * (before * a * torch.sigmoid(-f) + x * dsc)).to(st["df"].dtype)
            st["dx"][t0:t1, cols] = walk(lam * sc).to(st["dx"].dtype)
            st["dh0"][s, cols] = a[0] * lam[0]
    if not c["train"]:
        return st["y"], st["hT"]
    return st["y"], st["hT"], st["df"], st["dx"], st["dh0"]


def _step_plain(st):
    a, sc, _ = _gate(st["case"]["form"], st["f"].float())
    h = a * st["h"] + sc * st["x"].float()
    st["h_out"].copy_(h)
    st["y"].copy_(h)
    return st["y"], st["h_out"]


# ------------------------------------------------------------------------------------------------ 64 bits
def exact(case, seed):
    st = prepare(case, seed)
    return dict(rope=_rope_exact, attn=_attn_exact, decode=_decode_exact, scan=_scan_exact, step=_step_exact)[
        case["op"]](case, st)


def _rope_exact(c, st):
    x, pos = st["x"].double(), st["pos"].double()
    r = c["rot"]
    out = x.clone()
    base = ROPE_BASE * (ROPE_FACTOR ** (r / (r - 2)) if c["scaling"] == "base" else 1.0)
    for i in range(r // 2):
        w = math.pow(base, -2.0 * i / r)
        if c["scaling"] == "linear":
            w /= ROPE_FACTOR
        if c["scaling"] == "ramp":
            keep = min(1.0, max(0.0, (ROPE_LEN * w / (2 * math.pi) - ROPE_LOW) / (ROPE_HIGH - ROPE_LOW)))
            w = keep * w + (1.0 - keep) * w / ROPE_FACTOR
        z = torch.polar(torch.full_like(pos, 1.25 if c["scaling"] == "ramp" else 1.0), -pos * w if c["inverse"] else pos * w)
        j0, j1 = (i, i + r // 2) if c["layout"] == "half" else (2 * i, 2 * i + 1)
        turned = torch.complex(x[..., j0], x[..., j1]) * z[:, None]
        out[..., j0], out[..., j1] = turned.real, turned.imag
    return out


def _attn_exact(c, st):
    out, lse = torch.zeros(st["q"].shape, dtype=torch.float64, device="cuda"), st["lse"].double()
    out += st["out"].double()
    if c["train"]:
        dq, dk, dv = st["dq"].double(), st["dk"].double(), st["dv"].double()
    for s in range(c["seqs"]):
        q0, q1 = st["cu_q_host"][s:s + 2]
        k0, k1 = st["cu_k_host"][s:s + 2]
        nq, nk = q1 - q0, k1 - k0
        for h in range(c["Hq"]):
            hk = h * c["Hk"] // c["Hq"]
            K, V = st["k"][k0:k1, hk].double(), st["v"][k0:k1, hk].double()
            for i in range(0, nq, 2048):
                j = min(nq, i + 2048)
                # keys from the window of the block's first row to that of its last, the sinks in front
                a = min(nk, max(0, nk - nq + i - c["left"]))
                b = max(a, min(nk, nk - nq + j + c["right"]))
                z = min(a, c["sinks"])
                Kb, Vb = torch.cat([K[:z], K[a:b]]), torch.cat([V[:z], V[a:b]])
                u = torch.cat([torch.arange(z), torch.arange(a, b)]).cuda()
                back = (torch.arange(i, j).cuda() + nk - nq)[:, None] - u[None]      # how far the key lies behind
                hidden = (back < -c["right"]) | ((back > c["left"]) & (u >= c["sinks"])[None])
                Q = st["q"][q0 + i:q0 + j, h].double()
                w = (Q @ Kb.T / 8.0).masked_fill(hidden, -INF)
                L = torch.logsumexp(w, 1) if len(u) else torch.full((j - i,), -INF, dtype=torch.float64, device="cuda")
                P = torch.exp(w - L[:, None]).masked_fill(hidden, 0.0)
                lse[h, q0 + i:q0 + j] = L
                out[q0 + i:q0 + j, h] = P @ Vb
                if c["train"]:
                    dO = st["dout"][q0 + i:q0 + j, h].double()
                    dP = dO @ Vb.T
                    dS = P * (dP - (dO * (P @ Vb)).sum(1)[:, None]) / 8.0
                    dq[q0 + i:q0 + j, h] = dS @ Kb
                    gk, gv = dS.T @ Q, P.T @ dO
                    dk[k0:k0 + z, hk] += gk[:z]
                    dk[k0 + a:k0 + b, hk] += gk[z:]
                    dv[k0:k0 + z, hk] += gv[:z]
                    dv[k0 + a:k0 + b, hk] += gv[z:]
    return (out, lse, dq, dk, dv) if c["train"] else (out, lse)


def _decode_exact(c, st):
    out = torch.zeros(st["q"].shape, dtype=torch.float64, device="cuda")
    for b, n in enumerate(st["lens"].tolist()):
        u = torch.cat([torch.arange(min(c["sinks"], n)), torch.arange(max(c["sinks"], n - 1 - c["left"]), n)])
        u = u[u < n].unique()
        slot = torch.where(u < c["slots"], u, c["sinks"] + (u - c["sinks"]) % max(1, c["slots"] - c["sinks"])).cuda()
        K, V = st["cache_k"][b, slot].double(), st["cache_v"][b, slot].double()
        K[-1], V[-1] = st["k_new"][b].double(), st["v_new"][b].double()
        for h in range(c["Hq"]):
            hk = h * c["Hk"] // c["Hq"]
            out[b, h] = torch.softmax(K[:, hk] @ st["q"][b, h].double() / 8.0, 0) @ V[:, hk]
    return out, None, None      # the caches' rows are copies, not computed numbers


def _recurrence(a, b, h):
    """h_t = a_t h_{t-1} + b_t in 64 bits: spans side by side, then their carries one after the other."""
    n, w = a.shape
    span = max(1, int(math.isqrt(n)))
    m = -(-n // span)
    A, Bb = torch.ones(m * span, w, dtype=torch.float64, device=a.device), torch.zeros(m * span, w, dtype=torch.float64, device=a.device)
    A[:n], Bb[:n] = a, b
    A, Bb = A.view(m, span, w), Bb.view(m, span, w)
    for t in range(1, span):
        Bb[:, t] += A[:, t] * Bb[:, t - 1]
        A[:, t] *= A[:, t - 1]
    for j in range(m):
        Bb[j] += A[j] * h
        h = Bb[j, -1].clone()
    return Bb.view(m * span, w)[:n]


def _gate64(form, f):
    a, rest = 1.0 / (1.0 + torch.exp(-f)), 1.0 / (1.0 + torch.exp(f))      # a and 1 - a
    if form == "sum":
        return a, rest, torch.ones_like(a), torch.zeros_like(a)
    if form == "convex":
        return a, rest, rest, -torch.ones_like(a)
    s = torch.sqrt(rest * (1.0 + a))
    return a, rest, s, -a / s


def _scan_exact(c, st):
    res = {k: st[k].double() for k in ("y", "hT")}
    if c["train"]:
        res.update({k: st[k].double() for k in ("df", "dx", "dh0")})
    for s in range(c["seqs"]):
        t0, t1 = st["cu_host"][s], st["cu_host"][s + 1]
        if t1 == t0:
            res["hT"][s] = st["h0"][s].double()
            if c["train"]:
                res["dh0"][s] = st["dhT"][s].double()
            continue
        rows = torch.arange(t0, t1, device="cuda")
        if c["reverse"]:
            rows = rows.flip(0)
        for j in range(0, c["D"], 512):
            cols = slice(j, min(c["D"], j + 512))
            f, x = st["f"][:, cols][rows].double(), st["x"][:, cols][rows].double()
            h0 = st["h0"][s, cols].double()
            a, rest, g, slope = _gate64(c["form"], f)
            h = _recurrence(a, g * x, h0)
            res["y"][rows, cols] = h
            res["hT"][s, cols] = h[-1]
            if not c["train"]:
                continue
            dy = st["dy"][:, cols][rows].double()
            ahead = torch.ones_like(a)
            ahead[:-1] = a[1:]
            lam = _recurrence(ahead.flip(0), dy.flip(0), st["dhT"][s, cols].double()).flip(0)
            prev = torch.cat([h0[None], h[:-1]])
            res["df"][rows, cols] = lam * (prev + slope * x) * a * rest
            res["dx"][rows, cols] = lam * g
            res["dh0"][s, cols] = lam[0] * a[0]
    return tuple(res[k] for k in (("y", "hT", "df", "dx", "dh0") if c["train"] else ("y", "hT")))


def _step_exact(c, st):
    a, _, g, _ = _gate64(c["form"], st["f"].double())
    h = a * st["h"].double() + g * st["x"].double()
    return h, h


# ------------------------------------------------------------------------------------------------ work
def _pairs(c):
    """Visible (query, key) pairs of one head."""
    lq, lk = _split(c)
    n = 0
    for q, k in zip(lq, lk):
        p = torch.arange(q) + (k - q)
        hi = (p + c["right"] + 1).clamp(0, k)
        lo = torch.minimum((p - c["left"]).clamp(0, k), hi)
        n += int((hi - lo + torch.minimum(lo, torch.tensor(c["sinks"]))).sum())
    return n


def work(case):
    c = case
    if c["op"] == "rope":
        e = 2 if c["dtype"] == "bf16" else 4
        n = c["T"] * c["heads"]
        return dict(bytes=2 * n * c["d"] * e + 4 * c["T"], flops=3 * n * c["rot"])
    if c["op"] == "attn":
        lq, lk = _split(c)
        q, kv = sum(lq) * c["Hq"] * D * 2, sum(lk) * c["Hk"] * D * 2
        lse = 4 * c["Hq"] * sum(lq)
        pairs = _pairs(c) * c["Hq"]
        if c["train"]:      # q, k, v, dout in; out, log-sum-exp, dq, dk, dv out
            return dict(bytes=4 * q + 4 * kv + lse, flops=14 * D * pairs)
        return dict(bytes=2 * q + 2 * kv + lse, flops=4 * D * pairs)
    if c["op"] == "decode":      # lengths lie between half of the longest and the longest
        n = c["longest"] * 0.75 if c["B"] > 1 else c["longest"]
        n = min(n, c["left"] + 1 + c["sinks"])
        return dict(bytes=int(c["B"] * (n * c["Hk"] * D * 4 + 4 * c["Hq"] * D)), flops=int(4 * c["B"] * n * c["Hq"] * D))
    e = 2 if c["dtype"] == "bf16" else 4
    if c["op"] == "scan":
        n, s = c["rows"] * c["D"], 4 * c["seqs"] * c["D"]
        if c["train"]:      # f, x, dy in; y, df, dx out
            return dict(bytes=6 * n * e + 4 * s, flops=20 * n)
        return dict(bytes=3 * n * e + 2 * s, flops=6 * n)
    n = c["B"] * c["D"]
    return dict(bytes=n * (3 * e + 8), flops=6 * n)
