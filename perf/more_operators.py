"""What is measured of the selective state space scan, of the short causal
convolution in front of it and of the residual layer norm.

Kinds of case:

  scan        the selective scan over packed sequences (prompts),
  scan_train  the same with its backward pass (one training step's share),
  scan_step   one token per sequence on a pool of states (decode),
  conv, conv_train, conv_step   the same three of the short convolution,
  norm        residual addition + layer norm, output in the input's type or
              in 8 bits with scales,
  norm_train  the same with its backward pass.

The scan, per channel c of D, state n of N and row t of a sequence, with one B
and C for the channels of a group:

  delta = softplus(dt + bias_c),  h[c,n] = exp(-A[c,n] delta) h[c,n] + delta x B[n],
  y = (sum_n C[n] h[c,n] + skip_c x) * silu(z).

The convolution, per channel, over the last `taps` rows (what comes before a
sequence is part of its state):

  y[t] = silu(bias + sum_k w[taps-1-k] x[t-k]).

`own` selects the framework's kernels; otherwise `run` computes the same with
elementary torch operations in 32 bits (column sums over all rows in 64).
"""
import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
E4M3_MAX = 448.0
SCALE_MIN = 2.0 ** -126
EPS = 1e-5
MOST_ELEMENTS = 1 << 29                # rows x D x N of a training case


def listed():
    return [
        # A chunk of a serving batch: 16 sequences of a few tokens each (some
        # of none or one), carried states.
        {"name": "conv_chunk", "kind": "conv", "dtype": "bf16", "n_seq": 16, "rows": 600, "D": 1920, "taps": 4, "ragged": True, "start": True},
        {"name": "scan_chunk", "kind": "scan", "dtype": "bf16", "n_seq": 16, "rows": 600, "D": 1920, "N": 16, "groups": 1, "z": True, "ragged": True, "start": True},
        # One long document: 131072 tokens, 8 heads of 128.
        {"name": "scan_long", "kind": "scan", "dtype": "bf16", "n_seq": 1, "rows": 131072, "D": 1024, "N": 16, "groups": 1, "z": True, "ragged": False, "start": False},
        # Training, batch x length uniform (8 heads of 128).
        {"name": "conv_train_large", "kind": "conv_train", "dtype": "bf16", "n_seq": 8, "rows": 32768, "D": 2048, "taps": 4, "ragged": False, "start": False},
        {"name": "scan_train_large", "kind": "scan_train", "dtype": "bf16", "n_seq": 8, "rows": 32768, "D": 1024, "N": 16, "groups": 1, "z": True, "ragged": False, "start": False},
        # Training on packed documents in 32 bits, odd sizes, learned starts;
        # fewer taps, more states and several groups.
        {"name": "conv_train_ragged_f32", "kind": "conv_train", "dtype": "f32", "n_seq": 11, "rows": 10007, "D": 1000, "taps": 3, "ragged": True, "start": True},
        {"name": "scan_train_ragged_f32", "kind": "scan_train", "dtype": "f32", "n_seq": 11, "rows": 5003, "D": 960, "N": 32, "groups": 2, "z": False, "ragged": True, "start": True},
        # Decode: 64 sequences.
        {"name": "conv_step_64", "kind": "conv_step", "dtype": "bf16", "rows": 64, "D": 1920, "taps": 4, "n_slots": 96},
        {"name": "scan_step_64", "kind": "scan_step", "dtype": "bf16", "rows": 64, "D": 1920, "N": 16, "groups": 1, "z": True, "n_slots": 96},
        # The norm before a projection in 8 bits, at prefill (a scale per 128 channels).
        {"name": "norm_prefill_e4m3", "kind": "norm", "dtype": "bf16", "rows": 16384, "D": 3840, "out": "e4m3", "group": 128},
        # Training: forward and backward of the norm on the residual stream.
        {"name": "norm_train_large", "kind": "norm_train", "dtype": "bf16", "rows": 32768, "D": 1024},
        {"name": "norm_train_f32", "kind": "norm_train", "dtype": "f32", "rows": 4999, "D": 1920},
    ]


def _log_uniform(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def draw(rng):
    kind = rng.choice(["scan", "scan", "scan_train", "scan_train", "scan_step", "conv", "conv_train", "conv_step", "norm", "norm_train"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    D = 8 * _log_uniform(rng, 16, 512)                      # 128 .. 4096
    if kind in ("norm", "norm_train"):
        rows = _log_uniform(rng, 1, (1 << 25) // D)
        if kind == "norm_train":
            return {"kind": kind, "dtype": dtype, "rows": rows, "D": D}
        out = rng.choice(["same", "e4m3"])
        group = 0 if out == "same" else rng.choice([0, 32, 64, 128])
        if group:
            D = max(1, D // group) * group
        return {"kind": kind, "dtype": dtype, "rows": rows, "D": D, "out": out, "group": group}
    case = {"kind": kind, "dtype": dtype}
    scan = kind.startswith("scan")
    if scan:
        N = rng.choice([8, 16, 16, 16, 32, 64])
        groups = rng.choice([1, 1, 2, 4])
        D = max(1, D // (8 * groups)) * 8 * groups
        case.update(N=N, groups=groups, z=rng.random() < 0.7)
    else:
        N = 1
        case.update(taps=rng.choice([2, 3, 4, 4]))
    if kind.endswith("_step"):
        rows = _log_uniform(rng, 1, 1024)
        case.update(rows=rows, D=D, n_slots=rows + rng.randrange(rows + 1))
        return case
    most = min(65536, MOST_ELEMENTS // (D * N)) if scan else (1 << 25) // D
    rows = _log_uniform(rng, 65, most)
    n_seq = _log_uniform(rng, 1, 32)
    ragged = rng.random() < 0.6
    if not ragged:
        rows = max(1, rows // n_seq) * n_seq
    case.update(n_seq=n_seq, rows=rows, D=D, ragged=ragged, start=rng.random() < 0.5)
    return case


# ------------------------------------------------------------------- inputs

def _offsets(case, seed):
    """Where each sequence begins (n_seq + 1 numbers): equal lengths, or a
    random partition of the rows in which some sequences have no or one row."""
    n, rows = case["n_seq"], case["rows"]
    if not case["ragged"]:
        return np.arange(n + 1, dtype=np.int64) * (rows // n)
    r = np.random.RandomState(seed % (1 << 31))
    lens = np.floor(r.dirichlet(np.ones(n)) * rows).astype(np.int64)
    if n >= 4:
        k = r.permutation(n)[:2]
        lens[k[0]], lens[k[1]] = 0, 1
    lens[int(np.argmax(lens))] += rows - int(lens.sum())
    return np.concatenate([[0], np.cumsum(lens)])


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed))
    dt, rows, D, kind = DTYPES[case["dtype"]], case["rows"], case["D"], case["kind"]

    def normal(*shape, mean=0.0, std=1.0, dtype=dt):
        t = torch.empty(shape, dtype=torch.float32, device=dev).normal_(mean, std, generator=g)
        return t.to(dtype)

    def uniform(*shape, lo=0.0, hi=1.0):
        return torch.empty(shape, dtype=torch.float32, device=dev).uniform_(lo, hi, generator=g)

    st = {"case": dict(case)}
    if kind in ("norm", "norm_train"):
        # A residual stream a few times wider than the branch added to it, with
        # a mean of its own.
        st.update(x=normal(rows, D), residual=normal(rows, D, mean=0.5, std=3.0), gamma=uniform(D, lo=0.5, hi=1.5),
                  beta=normal(D, std=0.2, dtype=torch.float32))
        if kind == "norm_train":
            st.update(dout=normal(rows, D), ds=normal(rows, D, std=0.5))
        return st
    st["x"] = normal(rows, D)
    if kind.startswith("conv"):
        # Uniform in +- 1 / sqrt(taps), as such a convolution is initialised.
        lim = case["taps"] ** -0.5
        st.update(w=uniform(D, case["taps"], lo=-lim, hi=lim), bias=uniform(D, lo=-lim, hi=lim))
        per_state, state_type = (case["taps"] - 1, D), dt
    else:
        # Time steps log-uniform in [1e-3, 0.1] around which dt moves, rates
        # near 1, 2, .. N: memories from a few to about a thousand tokens.
        G, N = case["groups"], case["N"]
        step = torch.exp(uniform(D, lo=float(np.log(1e-3)), hi=float(np.log(0.1))))
        rate = torch.arange(1, N + 1, dtype=torch.float32, device=dev) * torch.exp(normal(D, N, std=0.1, dtype=torch.float32))
        st.update(dt=normal(rows, D, std=0.7), B=normal(rows, G, N), C=normal(rows, G, N), A=rate,
                  skip=normal(D, mean=1.0, std=0.1, dtype=torch.float32), bias=torch.log(torch.expm1(step)),
                  z=normal(rows, D) if case["z"] else None)
        per_state, state_type = (D, N), torch.float32
    if kind.endswith("_step"):
        st["state"] = normal(case["n_slots"], *per_state, std=0.5, dtype=state_type)
        st["slots"] = torch.randperm(case["n_slots"], generator=g, device=dev)[:rows].to(torch.int32)
        return st
    off = _offsets(case, int(seed))
    st["n_seq"] = case["n_seq"]
    st["longest"] = int(np.max(np.diff(off)))
    st["offsets"] = torch.from_numpy(off.astype(np.int32)).to(dev) if case["ragged"] else None
    st["start"] = normal(case["n_seq"], *per_state, std=0.5, dtype=state_type) if case["start"] else None
    if kind.endswith("_train"):
        st.update(dy=normal(rows, D), dend=normal(case["n_seq"], *per_state, dtype=state_type))
    return st


# --------------------------------------------------------------- plain forms

def _silu(x):
    return x * torch.sigmoid(x)


def _dsilu(x):
    s = torch.sigmoid(x)
    return s * (1 + x * (1 - s))


def _softplus(x):
    return torch.clamp(x, min=0) + torch.log1p(torch.exp(-x.abs()))


def _layout(st):
    """Of every row its sequence and its position there; of every sequence its
    first row and its length."""
    rows, n = st["x"].shape[0], st["n_seq"]
    off = st["offsets"].long() if st["offsets"] is not None else torch.arange(n + 1, device="cuda") * (rows // n)
    r = torch.arange(rows, device="cuda")
    seq = torch.searchsorted(off[1:].contiguous(), r, right=True)
    return seq, r - off[seq], off[:-1], off[1:] - off[:-1]


def _plain_conv(st, train):
    dt, D = st["x"].dtype, st["x"].shape[1]
    taps = st["w"].shape[1]
    seq, pos, first, length = _layout(st)
    x, w = st["x"].float(), st["w"]
    x0 = st["start"].float() if st["start"] is not None else torch.zeros(st["n_seq"], taps - 1, D, device="cuda")
    r = torch.arange(x.shape[0], device="cuda")
    past = [x]                                             # past[k][t] = x[t - k]
    for k in range(1, taps):
        inside = (pos >= k)[:, None]
        past.append(torch.where(inside, x[(r - k).clamp(min=0)], x0[seq, (taps - 1 + pos - k).clamp(0, taps - 2)]))
    pre = st["bias"].expand_as(x)
    for k in range(taps):
        pre = pre + w[:, taps - 1 - k] * past[k]
    # The last taps - 1 rows of a sequence, of its start where it is shorter.
    at = length[:, None] - (taps - 1) + torch.arange(taps - 1, device="cuda")
    own_row = at >= 0
    last = torch.where(own_row[:, :, None], x[(first[:, None] + at).clamp(0, x.shape[0] - 1)],
                       x0[torch.arange(st["n_seq"], device="cuda")[:, None], (taps - 1 + at).clamp(0, taps - 2)])
    out = {"y": _silu(pre).to(dt), "end": last.to(dt)}
    if not train:
        return out
    dpre = st["dy"].float() * _dsilu(pre)
    dx, dx0 = torch.zeros_like(x), torch.zeros_like(x0)
    for k in range(taps):
        term = w[:, taps - 1 - k] * dpre
        here = pos >= k
        dx[r[here] - k] += term[here]                      # a row is hit once for each k
        dx0.index_put_((seq[~here], (taps - 1 + pos - k)[~here]), term[~here], accumulate=True)
    dend = st["dend"].float()
    dx[(first[:, None] + at)[own_row]] += dend[own_row]
    s, j = torch.nonzero(~own_row, as_tuple=True)
    dx0[s, taps - 1 + at[s, j]] += dend[s, j]
    dw = torch.stack([(dpre * past[taps - 1 - j]).sum(0, dtype=torch.float64).float() for j in range(taps)], 1)
    out.update(dx=dx.to(dt), dw=dw, dbias=dpre.sum(0, dtype=torch.float64).float(), dstart=dx0.to(dt))
    return out


def _doubling(a, b, longest):
    """h[t] = a[t] h[t-1] + b[t] along the rows (a is 0 where a sequence
    begins); in place."""
    d = 1
    while d < longest:
        b[d:] += a[d:] * b[:-d]
        a[d:] = a[d:] * a[:-d]
        d *= 2
    return b


def _to_channels(t, D):
    """[rows, groups, N] for every channel: [rows, D, N]."""
    rows, G, N = t.shape
    return t.float()[:, :, None, :].expand(rows, G, D // G, N).reshape(rows, D, N)


def _plain_scan(st, train):
    dt, D = st["x"].dtype, st["x"].shape[1]
    x, A, N = st["x"].float(), st["A"], st["A"].shape[1]
    G = st["B"].shape[1]
    seq, pos, first, length = _layout(st)
    some = torch.nonzero(length > 0).flatten()
    begin, last = first[some], (first + length - 1)[some]
    h0 = st["start"] if st["start"] is not None else torch.zeros(st["n_seq"], D, N, device="cuda")
    raw = st["dt"].float() + st["bias"]
    delta = _softplus(raw)
    a = torch.exp(-A * delta[:, :, None])
    h = _to_channels(st["B"], D) * (delta * x)[:, :, None]
    h[begin] += a[begin] * h0[some]
    carry = a.clone() if train else a
    carry[begin] = 0
    h = _doubling(carry, h, st["longest"])
    del carry
    C = st["C"].float()
    inner = (h.view(-1, G, D // G, N) * C[:, :, None, :]).sum(3).view(-1, D) + st["skip"] * x
    z = st["z"].float() if st["z"] is not None else None
    gate = _silu(z) if z is not None else torch.ones_like(x)
    end = h0.clone()
    end[some] = h[last]
    out = {"y": (inner * gate).to(dt), "end": end}
    if not train:
        return out
    dy = st["dy"].float()
    dinner = dy * gate
    g = _to_channels(C, D) * dinner[:, :, None]
    g[last] += st["dend"][some]
    following = torch.cat([a[1:], a[:1]])                  # a[t+1], nothing after a sequence's end
    following[last] = 0
    g = _doubling(following.flip(0), g.flip(0), st["longest"]).flip(0)
    del following
    dstart = st["dend"].clone()
    dstart[some] = (a * g)[begin]
    dC = (h.view(-1, G, D // G, N) * dinner.view(-1, G, D // G, 1)).sum(2)
    before = torch.cat([h[:1], h[:-1]])
    before[begin] = h0[some]
    del h
    dlog = a.mul_(g).mul_(before)                          # d loss / d ln a
    del before
    B = _to_channels(st["B"], D)
    du = (g * B).sum(2)
    del B
    dB = (g.view(-1, G, D // G, N) * (delta * x).view(-1, G, D // G, 1)).sum(2)
    ddelta = du * x - (dlog * A).sum(2)
    dA = torch.zeros(D, N, dtype=torch.float64, device="cuda")
    for r in range(0, x.shape[0], 4096):                   # in 64 bits, a piece at a time
        dA -= (dlog[r:r + 4096] * delta[r:r + 4096, :, None]).sum(0, dtype=torch.float64)
    draw_ = ddelta * torch.sigmoid(raw)
    out.update(dx=(du * delta + dinner * st["skip"]).to(dt), ddt=draw_.to(dt), dA=dA.float(), dB=dB.to(dt), dC=dC.to(dt),
               dskip=(dinner * x).sum(0, dtype=torch.float64).float(), dbias=draw_.sum(0, dtype=torch.float64).float(), dstart=dstart)
    if z is not None:
        out["dz"] = (dy * inner * _dsilu(z)).to(dt)
    return out


def _plain_conv_step(st):
    x, w, slots = st["x"], st["w"], st["slots"].long()
    window = torch.cat([st["state"][slots], x[:, None]], 1)
    pre = st["bias"] + (window.float() * w.t()).sum(1)
    st["state"][slots] = window[:, 1:]
    return {"y": _silu(pre).to(x.dtype), "state": st["state"]}


def _plain_scan_step(st):
    x, slots, D = st["x"].float(), st["slots"].long(), st["x"].shape[1]
    delta = _softplus(st["dt"].float() + st["bias"])
    h = torch.exp(-st["A"] * delta[:, :, None]) * st["state"][slots] + _to_channels(st["B"], D) * (delta * x)[:, :, None]
    st["state"][slots] = h
    y = (h * _to_channels(st["C"], D)).sum(2) + st["skip"] * x
    if st["z"] is not None:
        y = y * _silu(st["z"].float())
    return {"y": y.to(st["x"].dtype), "state": st["state"]}


def _plain_norm(st, train):
    case, dt = st["case"], st["x"].dtype
    s = (st["x"].float() + st["residual"].float()).to(dt)
    f = s.float()
    f = f - f.mean(1, keepdim=True)
    inv = torch.rsqrt((f * f).mean(1, keepdim=True) + EPS)
    hat = f * inv
    y = hat * st["gamma"] + st["beta"]
    if not train:
        if case["out"] == "same":
            return {"s": s, "out": y.to(dt)}
        per = y.view(y.shape[0], -1, case["group"] or y.shape[1])
        scale = torch.clamp(per.abs().amax(2) / E4M3_MAX, min=SCALE_MIN)
        q = torch.clamp(per / scale[:, :, None], -E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
        return {"s": s, "out": q.view(y.shape), "scale": scale if case["group"] else scale[:, 0]}
    dout = st["dout"].float()
    w = dout * st["gamma"]
    dx = st["ds"].float() + inv * (w - w.mean(1, keepdim=True) - hat * (w * hat).mean(1, keepdim=True))
    return {"s": s, "out": y.to(dt), "dx": dx.to(dt), "dgamma": (dout * hat).sum(0, dtype=torch.float64).float(),
            "dbeta": dout.sum(0, dtype=torch.float64).float()}


# ------------------------------------------------------- the framework's calls

def _own(st):
    import sparse_state_linear_gb300 as sdm
    case = st["case"]
    kind, rows, D = case["kind"], case["rows"], case["D"]
    dt = sdm.SDM_BF16 if case["dtype"] == "bf16" else sdm.SDM_F32
    train = kind.endswith("_train")
    if kind in ("norm", "norm_train"):
        sh = sdm.make_norm(rows, D, dtype=dt)
        if kind == "norm" and case["out"] == "e4m3":
            r = sdm.sdm_add_layernorm(sh, st["x"], st["residual"], st["gamma"], st["beta"], eps=EPS, out_dtype=sdm.SDM_E4M3, group=case["group"])
            return {"s": r["s"], "out": r["out"], "scale": r["scale"]}
        r = sdm.sdm_add_layernorm(sh, st["x"], st["residual"], st["gamma"], st["beta"], eps=EPS, out_dtype=dt)
        out = {"s": r["s"], "out": r["out"]}
        if train:
            b = sdm.sdm_add_layernorm_backward(sh, r["s"], st["dout"], st["gamma"], ds=st["ds"], eps=EPS)
            out.update(dx=b["dx"], dgamma=b["dgamma"], dbeta=b["dbeta"])
        return out
    n_seq = case.get("n_seq", 1)
    if kind.startswith("conv"):
        sh = sdm.make_conv(n_seq, rows, D, taps=case["taps"], dtype=dt)
        if kind == "conv_step":
            y = sdm.sdm_short_conv_step(sh, st["x"], st["w"], st["state"], bias=st["bias"], slots=st["slots"])
            return {"y": y, "state": st["state"]}
        r = sdm.sdm_short_conv_forward(sh, st["x"], st["w"], bias=st["bias"], offsets=st["offsets"], x0=st["start"])
        out = {"y": r["y"], "end": r["xT"]}
        if train:
            b = sdm.sdm_short_conv_backward(sh, st["x"], st["w"], st["dy"], bias=st["bias"], offsets=st["offsets"], x0=st["start"], dxT=st["dend"])
            out.update(dx=b["dx"], dw=b["dw"], dbias=b["dbias"], dstart=b["dx0"])
        return out
    sh = sdm.make_selective(n_seq, rows, D, case["N"], groups=case["groups"], dtype=dt)
    ins = (st["x"], st["dt"], st["A"], st["B"], st["C"])
    kw = dict(skip=st["skip"], bias=st["bias"], z=st["z"])
    if kind == "scan_step":
        y = sdm.sdm_selective_scan_step(sh, *ins, st["state"], slots=st["slots"], **kw)
        return {"y": y, "state": st["state"]}
    r = sdm.sdm_selective_scan_forward(sh, *ins, offsets=st["offsets"], h0=st["start"], save_states=train, **kw)
    out = {"y": r["y"], "end": r["hT"]}
    if train:
        b = sdm.sdm_selective_scan_backward(sh, *ins, r["states"], st["dy"], offsets=st["offsets"], dhT=st["dend"], **kw)
        out.update({k: b[k] for k in ("dx", "ddt", "dA", "dB", "dC", "dskip", "dbias")}, dstart=b["dh0"])
        if st["z"] is not None:
            out["dz"] = b["dz"]
    return out


def run(state):
    if own:
        return _own(state)
    kind = state["case"]["kind"]
    train = kind.endswith("_train")
    if kind == "conv_step":
        return _plain_conv_step(state)
    if kind == "scan_step":
        return _plain_scan_step(state)
    if kind in ("norm", "norm_train"):
        return _plain_norm(state, train)
    return (_plain_conv if kind.startswith("conv") else _plain_scan)(state, train)


# ---------------------------------------------------------------------- work

def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    rows, D, kind = case["rows"], case["D"], case["kind"]
    n = rows * D
    if kind in ("norm", "norm_train"):      # x, residual, s, out (+ dout, s, ds, dx)
        if kind == "norm_train":
            return {"bytes": n * 8 * e + 16 * D, "flops": 20 * n}
        if case["out"] == "same":
            return {"bytes": n * 4 * e + 8 * D, "flops": 8 * n}
        scales = rows * (D // case["group"] if case["group"] else 1)
        return {"bytes": n * (3 * e + 1) + 8 * D + 4 * scales, "flops": 10 * n}
    if kind.startswith("conv"):
        taps = case["taps"]
        params = 4 * D * (taps + 1)
        if kind == "conv_step":             # x, y, the state in and out
            return {"bytes": n * e * (2 + 2 * (taps - 1)) + params + 4 * rows, "flops": n * (2 * taps + 5)}
        ends = case["n_seq"] * (taps - 1) * D * e
        if kind == "conv":                  # x, y
            return {"bytes": n * 2 * e + params + ends * (2 if case["start"] else 1), "flops": n * (2 * taps + 5)}
        # and x, dy, dx; of the ends, the start twice, what comes out, its gradient and the start's
        return {"bytes": n * 5 * e + 3 * params + ends * (5 if case["start"] else 3), "flops": n * (6 * taps + 15)}
    N, G, z = case["N"], case["groups"], int(case["z"])
    bc, params = rows * 2 * G * N * e, 4 * D * (N + 2)
    if kind == "scan_step":                 # x, dt, z, y, the state in and out
        return {"bytes": n * (e * (3 + z) + 8 * N) + bc + params + 4 * rows, "flops": n * (7 * N + 20)}
    ends = case["n_seq"] * D * N * 4
    if kind == "scan":
        return {"bytes": n * e * (3 + z) + bc + params + ends * (2 if case["start"] else 1), "flops": n * (7 * N + 20)}
    # and x, dt, z, dy, dx, ddt, dz; B, C and their gradients
    return {"bytes": n * e * (8 + 3 * z) + 3 * bc + 3 * params + ends * (4 if case["start"] else 3), "flops": n * (28 * N + 70)}


# --------------------------------------------------------------------- exact

def exact(case, seed):
    """The definition in 64 bits, one row after the other."""
    st = prepare(case, seed)
    kind, D, rows = case["kind"], case["D"], case["rows"]
    R = {k: t.double() for k, t in st.items() if torch.is_tensor(t) and t.is_floating_point()}
    if kind in ("norm", "norm_train"):
        return _exact_norm(case, st, R)
    if kind == "conv_step":
        y, new = torch.empty_like(R["x"]), R["state"].clone()
        slots, taps = st["slots"].long(), case["taps"]
        pre = R["bias"] + R["w"][:, taps - 1] * R["x"]
        for j in range(taps - 1):
            pre = pre + R["w"][:, j] * R["state"][slots, j]
            new[slots, j] = R["state"][slots, j + 1] if j + 1 < taps - 1 else R["x"]
        y = pre / (1 + torch.exp(-pre))
        return {"y": y, "state": new}
    if kind == "scan_step":
        slots, per = st["slots"].long(), D // case["groups"]
        delta = torch.logaddexp(R["dt"] + R["bias"], torch.zeros_like(R["x"]))
        h = R["state"][slots] * torch.exp(-(delta.unsqueeze(2) * R["A"]))
        h += (delta * R["x"]).unsqueeze(2) * R["B"].repeat_interleave(per, 1)
        new = R["state"].clone()
        new[slots] = h
        y = torch.einsum("rdn,rdn->rd", h, R["C"].repeat_interleave(per, 1)) + R["skip"] * R["x"]
        if case["z"]:
            y = y * R["z"] / (1 + torch.exp(-R["z"]))
        return {"y": y, "state": new}
    off = _offsets(case, seed)
    return (_exact_conv if kind.startswith("conv") else _exact_scan)(case, R, off)


def _exact_norm(case, st, R):
    D, rows = case["D"], case["rows"]
    s = (R["x"] + R["residual"]).to(st["x"].dtype).double()
    mean = s.sum(1, keepdim=True) / D
    norm = torch.sqrt((s - mean).square().sum(1, keepdim=True) / D + EPS)
    hat = (s - mean) / norm
    y = hat * R["gamma"] + R["beta"]
    if case["kind"] == "norm":
        if case["out"] == "same":
            return {"s": s, "out": y}
        per = y.reshape(rows, -1, case["group"] or D)
        scale = (per.abs().max(2).values / E4M3_MAX).clamp(min=SCALE_MIN)
        q = (per / scale.unsqueeze(2)).float().to(torch.float8_e4m3fn).double().reshape(y.shape)
        return {"s": s, "out": q, "scale": scale if case["group"] else scale.squeeze(1)}
    dhat = R["dout"] * R["gamma"]
    dnorm = -(dhat * (s - mean)).sum(1, keepdim=True) / norm.square()
    dcentred = dhat / norm + dnorm * (s - mean) / (D * norm)
    dx = R["ds"] + dcentred - dcentred.sum(1, keepdim=True) / D
    return {"s": s, "out": y, "dx": dx, "dgamma": (R["dout"] * hat).sum(0), "dbeta": R["dout"].sum(0)}


def _exact_conv(case, R, off):
    """Sequence by sequence, with its start in front of it."""
    taps, D = case["taps"], case["D"]
    train = case["kind"] == "conv_train"
    y, dx = torch.empty_like(R["x"]), torch.empty_like(R["x"])
    end, dstart = (torch.zeros(case["n_seq"], taps - 1, D, dtype=torch.float64, device="cuda") for _ in range(2))
    dw, dbias = torch.zeros_like(R["w"]), torch.zeros_like(R["bias"])
    for s in range(case["n_seq"]):
        a, b = int(off[s]), int(off[s + 1])
        head = R["start"][s] if "start" in R else torch.zeros(taps - 1, D, dtype=torch.float64, device="cuda")
        seq = torch.cat([head, R["x"][a:b]])
        T = b - a
        pre = R["bias"] + sum(R["w"][:, j] * seq[j:j + T] for j in range(taps))
        y[a:b] = pre / (1 + torch.exp(-pre))
        end[s] = seq[T:]
        if train:
            sig = 1 / (1 + torch.exp(-pre))
            dpre = R["dy"][a:b] * (sig + pre * sig * (1 - sig))
            dseq = torch.zeros_like(seq)
            dseq[T:] = R["dend"][s]
            for j in range(taps):
                dseq[j:j + T] += R["w"][:, j] * dpre
                dw[:, j] += (dpre * seq[j:j + T]).sum(0)
            dbias += dpre.sum(0)
            dstart[s], dx[a:b] = dseq[:taps - 1], dseq[taps - 1:]
    if not train:
        return {"y": y, "end": end}
    return {"y": y, "end": end, "dx": dx, "dw": dw, "dbias": dbias, "dstart": dstart}


def _exact_scan(case, R, off):
    D, N, G, n_seq, rows = case["D"], case["N"], case["groups"], case["n_seq"], case["rows"]
    per, train = D // G, case["kind"] == "scan_train"
    raw = R["dt"] + R["bias"]
    delta = torch.logaddexp(raw, torch.zeros_like(raw))
    u = delta * R["x"]
    wide = lambda t: t.repeat_interleave(per, -2)           # groups -> channels
    # Sequences side by side, longest first, so that those still running at
    # row t are the leading ones.
    lens = np.diff(off)
    order = np.argsort(-lens, kind="stable")
    starts = torch.from_numpy(off[:-1][order].copy()).cuda()
    seqs = torch.from_numpy(order.copy()).cuda()
    running = [int(k) for k in np.searchsorted(-lens[order], -np.arange(int(lens.max())), side="left")]
    end = R["start"].clone() if "start" in R else torch.zeros(n_seq, D, N, dtype=torch.float64, device="cuda")
    h = end[seqs]
    inner = torch.empty_like(u)
    states = torch.empty(rows, D, N, dtype=torch.float64, device="cuda") if train else None     # before each row
    minus_A = -R["A"]
    for t, k in enumerate(running):
        at = slice(int(starts[0]) + t, int(starts[0]) + t + 1) if n_seq == 1 else starts[:k] + t
        if train:
            states[at] = h[:k]
        h[:k] *= torch.exp(minus_A * delta[at].unsqueeze(2))
        h[:k] += u[at].unsqueeze(2) * (R["B"][at] if G == 1 else wide(R["B"][at]))
        inner[at] = (h[:k] * (R["C"][at] if G == 1 else wide(R["C"][at]))).sum(2)
    end[seqs] = h
    inner += R["skip"] * R["x"]
    sig = 1 / (1 + torch.exp(-R["z"])) if case["z"] else None
    y = inner * R["z"] * sig if case["z"] else inner
    out = {"y": y, "end": end}
    if not train:
        return out
    dinner = R["dy"] * R["z"] * sig if case["z"] else R["dy"]
    dB, dC = torch.empty_like(R["B"]), torch.empty_like(R["C"])
    du, ddelta = torch.empty_like(u), torch.empty_like(u)
    dA = torch.zeros_like(R["A"])
    dh = R["dend"][seqs]
    for t in range(len(running) - 1, -1, -1):
        k = running[t]
        at = slice(int(starts[0]) + t, int(starts[0]) + t + 1) if n_seq == 1 else starts[:k] + t
        a = torch.exp(minus_A * delta[at].unsqueeze(2))
        kept = a * states[at]
        B = wide(R["B"][at])
        now = kept + u[at].unsqueeze(2) * B
        g = dh[:k] + dinner[at].unsqueeze(2) * wide(R["C"][at])
        dC[at] = (dinner[at].unsqueeze(2) * now).view(k, G, per, N).sum(2)
        dB[at] = (g * u[at].unsqueeze(2)).view(k, G, per, N).sum(2)
        du[at] = (g * B).sum(2)
        dlog = g * kept
        ddelta[at] = (dlog * minus_A).sum(2)
        dA -= (dlog * delta[at].unsqueeze(2)).sum(0)
        dh[:k] = a * g
    dstart = torch.empty_like(dh)
    dstart[seqs] = dh
    ddt = (ddelta + du * R["x"]) / (1 + torch.exp(-raw))
    out.update(dx=du * delta + dinner * R["skip"], ddt=ddt, dA=dA, dB=dB, dC=dC, dskip=(dinner * R["x"]).sum(0), dbias=ddt.sum(0), dstart=dstart)
    if case["z"]:
        out["dz"] = R["dy"] * inner * (sig + R["z"] * sig * (1 - sig))
    return out
