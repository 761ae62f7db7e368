"""What is measured of the gated recurrence and of the residual RMS-Norm.

Five entry points in four kinds of case:

  forward     the gated delta recurrence over packed sequences (prefill),
  train       the same with its backward pass (one training step's share),
  step        one token per sequence on a pool of states (decode),
  norm        residual addition + RMS-Norm, output in the input's type or in
              8 bits with scales,
  norm_train  the same with its backward pass.

The recurrence, per channel c of D and row t of a sequence:

  alpha = exp(-A_c * softplus(za + bias_c)),  beta = sigmoid(zb),
  h~ = alpha * h[t-1],  h[t] = h~ + beta * (v - h~),  y[t] = h[t].

`own` selects the framework's kernels; otherwise `run` computes the same with
elementary torch operations in 32 bits (column sums over all rows in 64).
"""
import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
E4M3_MAX = 448.0
SCALE_MIN = 2.0 ** -126
EPS = 1e-6


def listed():
    return [
        # A chunk of a serving batch: 16 sequences of a few tokens each (some
        # of none or one), carried states, the width of two heads of 960.
        {"name": "forward_chunk", "kind": "forward", "dtype": "bf16", "n_seq": 16, "rows": 600, "D": 1920, "ragged": True, "h0": True},
        # A packed prefill in 32 bits, odd total.
        {"name": "forward_ragged_f32", "kind": "forward", "dtype": "f32", "n_seq": 13, "rows": 9001, "D": 1920, "ragged": True, "h0": True},
        # One long document: 131072 tokens, 16 heads of 128.
        {"name": "forward_long", "kind": "forward", "dtype": "bf16", "n_seq": 1, "rows": 131072, "D": 2048, "ragged": False, "h0": False},
        # Training at the mid and the large training shapes (4 heads of 128
        # and 8 of 128), batch x length uniform.
        {"name": "train_mid", "kind": "train", "dtype": "bf16", "n_seq": 4, "rows": 8192, "D": 512, "ragged": False, "h0": False},
        {"name": "train_large", "kind": "train", "dtype": "bf16", "n_seq": 8, "rows": 32768, "D": 1024, "ragged": False, "h0": False},
        # Training on packed documents in 32 bits, odd sizes, learned starts.
        {"name": "train_ragged_f32", "kind": "train", "dtype": "f32", "n_seq": 11, "rows": 10007, "D": 1000, "ragged": True, "h0": True},
        # Decode: 64 sequences; and a very large batch in 32 bits.
        {"name": "step_64", "kind": "step", "dtype": "bf16", "rows": 64, "D": 1920, "n_slots": 96},
        {"name": "step_1024_f32", "kind": "step", "dtype": "f32", "rows": 1024, "D": 3840, "n_slots": 1500},
        # The norm before a projection in 8 bits, at decode (a scale per row)
        # and at prefill (a scale per 128 channels).
        {"name": "norm_decode_e4m3", "kind": "norm", "dtype": "bf16", "rows": 64, "D": 1920, "out": "e4m3", "group": 0},
        {"name": "norm_prefill_e4m3", "kind": "norm", "dtype": "bf16", "rows": 16384, "D": 3840, "out": "e4m3", "group": 128},
        # Training: forward and backward of the norm on the residual stream.
        {"name": "norm_train_large", "kind": "norm_train", "dtype": "bf16", "rows": 32768, "D": 1024},
        {"name": "norm_train_f32", "kind": "norm_train", "dtype": "f32", "rows": 4999, "D": 1920},
    ]


def _log_uniform(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def draw(rng):
    kind = rng.choice(["forward", "train", "step", "norm", "norm_train"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    D = 8 * _log_uniform(rng, 16, 512)                      # 128 .. 4096
    if kind in ("forward", "train"):
        rows = _log_uniform(rng, 65, min(131072, (1 << 25) // D))
        n_seq = _log_uniform(rng, 1, 32)
        ragged = rng.random() < 0.6
        if not ragged:
            rows = max(1, rows // n_seq) * n_seq
        return {"kind": kind, "dtype": dtype, "n_seq": n_seq, "rows": rows, "D": D, "ragged": ragged, "h0": rng.random() < 0.5}
    if kind == "step":
        rows = _log_uniform(rng, 1, 1024)
        return {"kind": kind, "dtype": dtype, "rows": rows, "D": D, "n_slots": rows + rng.randrange(rows + 1)}
    rows = _log_uniform(rng, 1, (1 << 25) // D)
    if kind == "norm_train":
        return {"kind": kind, "dtype": dtype, "rows": rows, "D": D}
    out = rng.choice(["same", "e4m3", "e4m3"])
    group = 0 if out == "same" else rng.choice([0, 32, 64, 128])
    if group:
        D = max(1, D // group) * group
    return {"kind": kind, "dtype": dtype, "rows": rows, "D": D, "out": out, "group": group}


# ------------------------------------------------------------------- inputs

def _offsets(case, seed):
    """Where each sequence begins (n_seq + 1 numbers): equal lengths, or a
    random partition of the rows in which some sequences have no or one row."""
    n, rows = case["n_seq"], case["rows"]
    if not case["ragged"]:
        return np.arange(n + 1, dtype=np.int64) * (rows // n)
    r = np.random.RandomState(seed % (1 << 31))
    lens = r.dirichlet(np.ones(n)) * rows
    lens = np.floor(lens).astype(np.int64)
    if n >= 4:
        k = r.permutation(n)[:2]
        lens[k[0]], lens[k[1]] = 0, 1
    lens[int(np.argmax(lens))] += rows - int(lens.sum())
    return np.concatenate([[0], np.cumsum(lens)])


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed))
    dt, rows, D = DTYPES[case["dtype"]], case["rows"], case["D"]

    def normal(*shape, mean=0.0, std=1.0, dtype=dt):
        t = torch.empty(shape, dtype=torch.float32, device=dev).normal_(mean, std, generator=g)
        return t.to(dtype)

    def uniform(*shape, lo=0.0, hi=1.0):
        return torch.empty(shape, dtype=torch.float32, device=dev).uniform_(lo, hi, generator=g)

    st = {"case": dict(case)}
    if case["kind"] in ("norm", "norm_train"):
        # A residual stream a few times wider than the branch added to it.
        st.update(x=normal(rows, D), residual=normal(rows, D, std=3.0), gamma=uniform(D, lo=0.5, hi=1.5))
        if case["kind"] == "norm_train":
            st.update(dout=normal(rows, D), ds=normal(rows, D, std=0.5))
        return st
    # Time steps softplus(bias) log-uniform in [1e-3, 0.1] and rates A in
    # [1, 16]: memories from a few to about a thousand tokens.
    step = torch.exp(uniform(D, lo=float(np.log(1e-3)), hi=float(np.log(0.1))))
    st.update(za=normal(rows, D, std=0.7), zb=normal(rows, D, mean=-3.0, std=2.0), v=normal(rows, D),
              A=uniform(D, lo=1.0, hi=16.0), bias=torch.log(torch.expm1(step)))
    if case["kind"] == "step":
        st["state"] = normal(case["n_slots"], D, dtype=torch.float32)
        perm = torch.randperm(case["n_slots"], generator=g, device=dev)
        st["slots"] = perm[:rows].to(torch.int32)
        return st
    off = _offsets(case, int(seed))
    st["n_seq"] = case["n_seq"]
    st["longest"] = int(np.max(np.diff(off)))
    st["offsets"] = torch.from_numpy(off.astype(np.int32)).to(dev) if case["ragged"] else None
    st["h0"] = normal(case["n_seq"], D, std=0.5, dtype=torch.float32) if case["h0"] else None
    if case["kind"] == "train":
        st.update(dy=normal(rows, D), dhT=normal(case["n_seq"], D, dtype=torch.float32))
    return st


# --------------------------------------------------------------- plain forms

def _gates(st):
    x = st["za"].float() + st["bias"]
    sp = torch.clamp(x, min=0) + torch.log1p(torch.exp(-x.abs()))
    alpha = torch.exp(-st["A"] * sp)
    zb = st["zb"].float()
    return x, sp, alpha, torch.sigmoid(zb), torch.sigmoid(-zb)


def _scan(a, b, longest):
    """h[t] = a[t] h[t-1] + b[t] along the rows by doubling (a is 0 where a
    sequence begins)."""
    d = 1
    a, b = a.clone(), b.clone()
    while d < longest:
        b[d:] += a[d:] * b[:-d]
        a[d:] = a[d:] * a[:-d]
        d *= 2
    return b


def _bounds(st):
    """First and last row of every sequence that has rows, those sequences'
    numbers, and whether a row begins a sequence."""
    rows, n = st["za"].shape[0], st["n_seq"]
    off = st["offsets"].long() if st["offsets"] is not None else torch.arange(n + 1, device="cuda") * (rows // n)
    some = torch.nonzero(off[1:] > off[:-1]).flatten()
    first, last = off[:-1][some], off[1:][some] - 1
    begins = torch.zeros(rows, 1, dtype=torch.bool, device="cuda")
    begins[first] = True
    return first, last, some, begins


def _plain_recurrence(st, train):
    x, sp, alpha, beta, keep = _gates(st)
    dt, D = st["za"].dtype, st["za"].shape[1]
    first, last, some, begins = _bounds(st)
    h0 = st["h0"] if st["h0"] is not None else torch.zeros(st["n_seq"], D, device="cuda")
    v = st["v"].float()
    a, b = keep * alpha, beta * v
    b[first] += a[first] * h0[some]
    h = _scan(torch.where(begins, torch.zeros_like(a), a), b, st["longest"])
    hT = h0.clone()
    hT[some] = h[last]
    out = {"y": h.to(dt), "hT": hT}
    if not train:
        return out
    prev = torch.cat([h[:1], h[:-1]])
    prev[first] = h0[some]
    dy = st["dy"].float()
    dy[last] += st["dhT"][some]
    following = torch.cat([a[1:], a[:1]])          # a[t+1], nothing after a sequence's end
    following[last] = 0
    g = _scan(following.flip(0), dy.flip(0), st["longest"]).flip(0)
    dbeta = g * (v - alpha * prev)
    dlog = g * a * prev                            # d loss / d ln alpha
    dx = -st["A"] * dlog * torch.sigmoid(x)
    dh0 = st["dhT"].clone()
    dh0[some] = (a * g)[first]
    out.update(dza=dx.to(dt), dzb=(dbeta * beta * keep).to(dt), dv=(beta * g).to(dt),
               dA=(-sp * dlog).sum(0, dtype=torch.float64).float(), dbias=dx.sum(0, dtype=torch.float64).float(), dh0=dh0)
    return out


def _plain_step(st):
    _, _, alpha, beta, keep = _gates(st)
    slots = st["slots"].long()
    h = keep * alpha * st["state"][slots] + beta * st["v"].float()
    st["state"][slots] = h
    return {"y": h.to(st["za"].dtype), "state": st["state"]}


def _plain_norm(st, train):
    case, dt = st["case"], st["x"].dtype
    s = (st["x"].float() + st["residual"].float()).to(dt)
    f = s.float()
    inv = torch.rsqrt((f * f).mean(1, keepdim=True) + EPS)
    hat = f * inv
    y = hat * st["gamma"]
    if not train:
        if case["out"] == "same":
            return {"s": s, "out": y.to(dt)}
        per = y.view(y.shape[0], -1, case["group"] or y.shape[1])
        scale = torch.clamp(per.abs().amax(2) / E4M3_MAX, min=SCALE_MIN)
        q = torch.clamp(per / scale[:, :, None], -E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
        return {"s": s, "out": q.view(y.shape), "scale": scale if case["group"] else scale[:, 0]}
    dout = st["dout"].float()
    w = dout * st["gamma"]
    dx = st["ds"].float() + inv * (w - hat * (w * hat).mean(1, keepdim=True))
    return {"s": s, "out": y.to(dt), "dx": dx.to(dt), "dgamma": (dout * hat).sum(0, dtype=torch.float64).float()}


def _own(st):
    import sparse_state_linear_gb300 as sdm
    case = st["case"]
    dt = sdm.SDM_BF16 if case["dtype"] == "bf16" else sdm.SDM_F32
    if case["kind"] in ("norm", "norm_train"):
        sh = sdm.make_norm(case["rows"], case["D"], dtype=dt)
        if case["kind"] == "norm" and case["out"] == "e4m3":
            r = sdm.sdm_add_rmsnorm(sh, st["x"], st["residual"], st["gamma"], eps=EPS, out_dtype=sdm.SDM_E4M3, group=case["group"])
            return {"s": r["s"], "out": r["out"], "scale": r["scale"]}
        r = sdm.sdm_add_rmsnorm(sh, st["x"], st["residual"], st["gamma"], eps=EPS, out_dtype=dt)
        out = {"s": r["s"], "out": r["out"]}
        if case["kind"] == "norm_train":
            b = sdm.sdm_add_rmsnorm_backward(sh, r["s"], st["dout"], st["gamma"], ds=st["ds"], eps=EPS)
            out.update(dx=b["dx"], dgamma=b["dgamma"])
        return out
    if case["kind"] == "step":
        sh = sdm.make_recurrence(1, case["rows"], case["D"], dtype=dt)
        y = sdm.sdm_recurrence_step(sh, st["za"], st["zb"], st["v"], st["state"], A=st["A"], bias=st["bias"], slots=st["slots"])
        return {"y": y, "state": st["state"]}
    train = case["kind"] == "train"
    sh = sdm.make_recurrence(case["n_seq"], case["rows"], case["D"], dtype=dt)
    r = sdm.sdm_recurrence_forward(sh, st["za"], st["zb"], st["v"], A=st["A"], bias=st["bias"], offsets=st["offsets"], h0=st["h0"],
                                   save_states=train)
    out = {"y": r["y"], "hT": r["hT"]}
    if train:
        b = sdm.sdm_recurrence_backward(sh, st["za"], st["zb"], st["v"], r["states"], st["dy"], A=st["A"], bias=st["bias"],
                                        offsets=st["offsets"], dhT=st["dhT"])
        out.update({k: b[k] for k in ("dza", "dzb", "dv", "dA", "dbias", "dh0")})
        _leave_dy_as_the_plain_form_does(st)
    return out


def _leave_dy_as_the_plain_form_does(st):
    """The plain form adds the final states' gradient to the last rows of dy,
    and where dy is in 32 bits that is the state's own dy: a further pass on
    the same state starts from the sum.  So it does here."""
    dy, dhT, off = st["dy"], st["dhT"], st["offsets"]
    if dy.dtype != torch.float32:
        return
    if off is None:
        dy.view(dhT.shape[0], -1, dy.shape[1])[:, -1] += dhT
        return
    some = off[1:] > off[:-1]                      # an empty sequence adds nothing
    dy.index_add_(0, (off[1:] - 1).clamp_(min=0), dhT * some[:, None])


def run(state):
    if own:
        return _own(state)
    kind = state["case"]["kind"]
    if kind == "step":
        return _plain_step(state)
    if kind in ("norm", "norm_train"):
        return _plain_norm(state, kind == "norm_train")
    return _plain_recurrence(state, kind == "train")


# ---------------------------------------------------------------------- work

def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    n = case["rows"] * case["D"]
    D, kind = case["D"], case["kind"]
    if kind == "step":                      # za, zb, v, the state in and out, y
        return {"bytes": n * (4 * e + 8) + 8 * D + 4 * case["rows"], "flops": 12 * n}
    if kind in ("norm", "norm_train"):      # x, residual, s, out (+ dout, s, ds, dx)
        if kind == "norm_train":
            return {"bytes": n * 8 * e + 12 * D, "flops": 16 * n}
        if case["out"] == "same":
            return {"bytes": n * 4 * e + 4 * D, "flops": 6 * n}
        scales = case["rows"] * (D // case["group"] if case["group"] else 1)
        return {"bytes": n * (3 * e + 1) + 4 * D + 4 * scales, "flops": 8 * n}
    ends = case["n_seq"] * D * 4 * (2 if case["h0"] else 1)
    if kind == "forward":                   # za, zb, v, y
        return {"bytes": n * 4 * e + 8 * D + ends, "flops": 12 * n}
    # and za, zb, v, dy, dza, dzb, dv
    return {"bytes": n * 11 * e + 24 * D + ends + 2 * case["n_seq"] * D * 4, "flops": 40 * n}


# --------------------------------------------------------------------- exact

def exact(case, seed):
    """The definition in 64 bits, one row after the other."""
    st = prepare(case, seed)
    D = case["D"]
    R = {k: t.double() for k, t in st.items() if torch.is_tensor(t) and t.is_floating_point()}
    if case["kind"] in ("norm", "norm_train"):
        s = (R["x"] + R["residual"]).to(st["x"].dtype).double()
        norm = torch.sqrt(s.square().sum(1, keepdim=True) / D + EPS)
        y = s / norm * R["gamma"]
        if case["kind"] == "norm":
            if case["out"] == "same":
                return {"s": s, "out": y}
            per = y.reshape(case["rows"], -1, case["group"] or D)
            scale = (per.abs().max(2).values / E4M3_MAX).clamp(min=SCALE_MIN)
            q = (per / scale.unsqueeze(2)).float().to(torch.float8_e4m3fn).double().reshape(y.shape)
            return {"s": s, "out": q, "scale": scale if case["group"] else scale.squeeze(1)}
        dn = R["dout"] * R["gamma"]                                     # gradient at s / norm
        dnorm = -(dn * s).sum(1, keepdim=True) / norm.square()
        return {"s": s, "out": y, "dx": R["ds"] + dn / norm + dnorm * s / (D * norm), "dgamma": (R["dout"] * s / norm).sum(0)}
    x = R["za"] + R["bias"]
    softplus = torch.logaddexp(x, torch.zeros_like(x))
    alpha = torch.exp(-R["A"] * softplus)
    beta = 1.0 / (1.0 + torch.exp(-R["zb"]))
    drop = 1.0 / (1.0 + torch.exp(R["zb"]))                             # 1 - beta
    if case["kind"] == "step":
        state, i = R["state"], st["slots"].long()
        h = alpha * state[i]
        h = drop * h + beta * R["v"]
        state[i] = h
        return {"y": h, "state": state}
    off = _offsets(case, seed)
    a, b = drop * alpha, beta * R["v"]
    h0 = R.get("h0", torch.zeros(case["n_seq"], D, dtype=torch.float64, device="cuda"))
    y, before, hT = torch.empty_like(b), torch.empty_like(b), h0.clone()
    # Sequences side by side, longest first, so that those still running at
    # row t are the leading ones.
    lens = np.diff(off)
    order = np.argsort(-lens, kind="stable")
    starts = torch.from_numpy(off[:-1][order].copy()).cuda()
    seqs = torch.from_numpy(order.copy()).cuda()
    running = [int(k) for k in np.searchsorted(-lens[order], -np.arange(int(lens.max())), side="left")]
    h = h0[seqs]
    single = case["n_seq"] == 1
    for t, k in enumerate(running):
        if single:
            before[t] = h[0]
            torch.addcmul(b[t], a[t], h[0], out=y[t])
            h = y[t:t + 1]
            continue
        at = starts[:k] + t
        before[at] = h[:k]
        h = a[at] * h[:k] + b[at]
        y[at] = h
    ends = torch.from_numpy(np.flatnonzero(lens > 0)).cuda()
    lasts = torch.from_numpy((off[1:] - 1)[lens > 0].copy()).cuda()
    hT[ends] = y[lasts]
    out = {"y": y, "hT": hT}
    if case["kind"] == "forward":
        return out
    g, dh = torch.empty_like(y), R["dhT"][seqs]
    for t in range(len(running) - 1, -1, -1):
        k = running[t]
        at = starts[:k] + t
        grad = R["dy"][at] + dh[:k]
        g[at] = grad
        dh[:k] = a[at] * grad
    dh0 = torch.empty_like(dh)
    dh0[seqs] = dh
    dalpha = g * drop * before
    dx = dalpha * alpha * -R["A"] / (1.0 + torch.exp(-x))
    out.update(dza=dx, dzb=g * (R["v"] - alpha * before) * beta * drop, dv=g * beta, dA=(dalpha * alpha * -softplus).sum(0),
               dbias=dx.sum(0), dh0=dh0)
    return out
