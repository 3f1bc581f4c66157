"""Cases for the operators of recurrent sequence models and their training:

- the gated linear recurrence  h_t = a_t h_{t-1} + u_t  along time, one
  independent recurrence per channel (a unit lower bidiagonal solve per
  channel), its backward pass, and its single-token form over a table of
  states;
- the orthogonalisation of an update matrix by Newton-Schulz products.

Each case is one call on synthetic inputs.  ``run`` makes the call of this
library where ``own`` is true, and otherwise computes the same from the
formulas with elementary torch operations in 32 bits.
"""
import math
import random

import torch

own = False

# the quintic polynomial a + b s^2 + c s^4 of each Newton-Schulz step
COEFFICIENTS = (3.4445, -4.7750, 2.0315)
STEPS = 5
EPS = 1e-7

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


# ------------------------------------------------------------------ cases
def listed():
    """The cases of the record."""
    return [
        # a first short prompt in single precision: launch latency
        scan("scan_short", "forward", "f32", "sigmoid", 1, 19, 256),
        # a layer's prefill / training forward; gate and input are the two
        # halves of one projection, so rows are strided
        scan("scan_layer", "forward", "bf16", "sigmoid", 4, 2048, 2048, fused=True),
        # one long document, the recurrence's memory is what counts; state
        # carried in from an earlier part
        scan("scan_long", "forward", "bf16", "log", 1, 65536, 2048, state=True),
        # packed documents of uneven length (empty ones and single tokens
        # among them), a width that is no multiple of a vector
        scan("scan_packed", "forward", "f16", "decay", 37, 10007, 1001, packed=True, state=True),
        # a small odd training batch in single precision
        scan("grad_small", "backward", "f32", "log", 3, 301, 130, state=True),
        # the training batch of a layer
        scan("grad_layer", "backward", "bf16", "sigmoid", 8, 4096, 2048),
        # one request generating, and a full batch of them out of a larger
        # table of states
        step("step_one", "f32", "log", 1, 2048, 1),
        step("step_batch", "bf16", "sigmoid", 256, 4096, 512),
        # per-head blocks of 64 x 64, one call for the heads of many layers
        orth("orth_heads", "bf16", 64, 64, 1024),
        # a tall single-precision momentum of an odd shape
        orth("orth_odd", "f32", 1500, 1000, 1),
        # the square projections of several layers
        orth("orth_layers", "bf16", 1024, 1024, 16),
        # a wide feed-forward matrix
        orth("orth_wide", "bf16", 4096, 16384, 1),
    ]


def scan(name, direction, dtype, form, batch, steps, width, fused=False, packed=False, state=False):
    """``batch`` sequences of ``steps`` tokens (packed: ``steps`` tokens in
    all) of ``width`` channels; state: an initial state, and in the backward
    pass the gradient of the last state, are given."""
    return {"name": name, "op": "scan", "direction": direction, "dtype": dtype, "form": form, "batch": batch,
            "steps": steps, "width": width, "fused": fused, "packed": packed, "state": state}


def step(name, dtype, form, batch, width, slots):
    return {"name": name, "op": "step", "dtype": dtype, "form": form, "batch": batch, "width": width, "slots": slots}


def orth(name, dtype, rows, cols, batch):
    return {"name": name, "op": "orth", "dtype": dtype, "rows": rows, "cols": cols, "batch": batch}


def draw(rng: random.Random):
    def spread(lo, hi):
        return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))

    def size(lo, hi):
        """Half of them odd, half round: a power of two times 1, 5/4 or 7/4."""
        v = spread(lo, hi)
        if rng.random() < 0.5:
            return v if v % 2 else max(lo, v - 1)
        two = 1 << (v.bit_length() - 1)
        return max(lo, [f * two // 4 for f in (4, 5, 7) if f * two // 4 <= v][-1])

    kind = rng.choice(("forward", "forward", "backward", "backward", "step", "orth", "orth"))
    dtype = rng.choice(("f32", "f16", "bf16", "bf16"))
    form = rng.choice(("decay", "log", "sigmoid"))
    if kind in ("forward", "backward"):
        most = 1 << (25 if kind == "forward" else 24)
        w = size(1, 4096)
        packed = rng.random() < 0.3
        t = size(1, max(1, min(131071 if packed else 65536, most // w)))
        b = spread(1, 64 if packed else max(1, min(64, most // (w * t))))
        c = scan("", kind, dtype, form, b, t, w, fused=rng.random() < 0.3, packed=packed, state=rng.random() < 0.5)
    elif kind == "step":
        b = spread(1, 512)
        c = step("", dtype, form, b, size(1, 8192), b + spread(1, 512) - 1)
    else:
        r, k = size(8, 3000), size(8, 6000)
        if rng.random() < 0.5:
            r, k = k, r
        one = work(orth("", dtype, r, k, 1))
        most = max(1, int(min(2e12 / one["flops"], 4e8 / one["bytes"], 512)))
        c = orth("", dtype, r, k, spread(1, most))
    del c["name"]
    return c


def work(case):
    """Bytes and operations that a pass cannot do without: each input read
    once and each output written once.  Recurrence: a multiply and an add per
    element (the backward pass: those of the reverse recurrence and the
    products of the two gradients).  Orthogonalisation: of each step's three
    products two are symmetric and need half."""
    if case["op"] == "orth":
        r, k = min(case["rows"], case["cols"]), max(case["rows"], case["cols"])
        size = 4 if case["dtype"] == "f32" else 2
        return {"bytes": case["batch"] * r * k * (size + 2.0),
                "flops": case["batch"] * STEPS * (3.0 * r * r * k + 1.0 * r * r * r)}
    size = 4 if case["dtype"] == "f32" else 2
    if case["op"] == "step":
        n = case["batch"] * case["width"]
        return {"bytes": n * (3.0 * size + 8), "flops": 3.0 * n}
    n = case["steps"] * case["width"] * (1 if case["packed"] else case["batch"])
    last = 4.0 * case["batch"] * case["width"]
    if case["direction"] == "forward":
        return {"bytes": n * 3.0 * size + last * (2 if case["state"] else 1), "flops": 2.0 * n}
    tensors = 6.0 if case["form"] == "sigmoid" else 5.0
    return {"bytes": n * tensors * size + last * (3 if case["state"] else 1), "flops": 4.0 * n}


# ------------------------------------------------------------------ inputs
def gates(form, shape, gen, dtype):
    """Gates of channels that forget within a few tokens up to ones that
    remember over a thousand."""
    dev = gen.device
    memory = torch.exp(torch.rand(shape[-1], generator=gen, device=dev) * math.log(1000.0) + 0.7)
    noise = torch.randn(shape, generator=gen, device=dev)
    rate = torch.exp(0.5 * noise) / memory  # -log a
    if form == "log":
        return (-rate).to(dtype)
    if form == "sigmoid":
        return (-torch.log(torch.expm1(rate.clamp(min=1e-4)))).to(dtype)
    return torch.exp(-rate).to(dtype)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    dt = DTYPES[case["dtype"]]
    s = {"case": dict(case)}

    def normal(shape, dtype=dt):
        return torch.randn(shape, generator=gen, device="cuda").to(dtype)

    if case["op"] == "orth":
        # a gradient: a few strong directions over noise
        b, m, n = case["batch"], case["rows"], case["cols"]
        k = max(1, min(m, n) // 16)
        strength = torch.exp(-torch.arange(k, device="cuda") / 4.0)
        g = normal((b, m, k), torch.float32) * strength @ normal((b, k, n), torch.float32)
        g = (g + 0.05 * normal((b, m, n), torch.float32)) * 1e-3
        s["g"] = g.to(dt)
        return s
    w = case["width"]
    if case["op"] == "step":
        b = case["batch"]
        s["gate"] = gates(case["form"], (b, w), gen, dt)
        s["x"] = normal((b, w))
        s["state"] = normal((case["slots"], w), torch.float32)
        s["slots"] = torch.randperm(case["slots"], generator=gen, device="cuda")[:b].to(torch.int32)
        s["next"] = torch.zeros_like(s["state"])
        return s
    b, t = case["batch"], case["steps"]
    shape = (t, w) if case["packed"] else (b, t, w)
    s["gate"] = gates(case["form"], shape, gen, dt)
    s["x"] = normal(shape)
    if case["fused"]:  # one projection's output, gate first
        both = torch.cat([s["gate"], s["x"]], dim=-1)
        s["gate"], s["x"] = both[..., :w], both[..., w:]
    s["h0"] = normal((b, w), torch.float32) if case["state"] else None
    s["offsets"] = None
    if case["packed"]:
        cuts = sorted(random.Random(int(seed)).randint(0, t) for _ in range(b - 1))
        s["offsets"] = torch.tensor([0] + cuts + [t], dtype=torch.int32, device="cuda")
    if case["direction"] == "backward":
        s["h"] = plain_forward(s)[0]
        s["dh"] = normal(shape)
        s["dh_last"] = normal((b, w), torch.float32) if case["state"] else None
    return s


# ------------------------------------------------------------------ the calls
def run(state):
    case = state["case"]
    if own:
        import triangular_solve_gb300 as tg
        if case["op"] == "orth":
            return tg.orthogonalize(state["g"], steps=STEPS, coefficients=COEFFICIENTS, eps=EPS)
        if case["op"] == "step":
            y = tg.linear_recurrence_step(state["gate"], state["x"], state["state"], form=case["form"],
                                          slots=state["slots"], out_state=state["next"])
            return [y, state["next"]]
        if case["direction"] == "forward":
            return list(tg.linear_recurrence(state["gate"], state["x"], state["h0"], form=case["form"],
                                             offsets=state["offsets"]))
        return list(tg.linear_recurrence_backward(state["gate"], state["x"], state["h"], state["dh"], state["h0"],
                                                  state["dh_last"], form=case["form"], offsets=state["offsets"]))
    if case["op"] == "orth":
        return plain_orth(state["g"])
    if case["op"] == "step":
        return plain_step(state)
    return plain_forward(state) if case["direction"] == "forward" else plain_backward(state)


# ------------------------------------------------------------------ plain forms
def decay_and_input(form, gate, x):
    """a_t and u_t in 32 bits."""
    g, x = gate.float(), x.float()
    if form == "decay":
        return g, x
    if form == "log":
        return torch.exp(g), x
    return torch.sigmoid(g), torch.sigmoid(-g) * x


def inclusive_scan(a, u):
    """h_t = a_t h_{t-1} + u_t along dimension -2 from h = 0: after the pass
    with distance d each (a, u) stands for 2 d tokens."""
    d = 1
    while d < u.shape[-2]:
        u = torch.cat([u[..., :d, :], u[..., d:, :] + a[..., d:, :] * u[..., :-d, :]], dim=-2)
        a = torch.cat([a[..., :d, :], a[..., d:, :] * a[..., :-d, :]], dim=-2)
        d *= 2
    return u


def flat(state, t):
    """Batched tensors as one packed list of rows."""
    return t.reshape(-1, t.shape[-1])


def bounds(state):
    """First row and row count of each sequence in the packed list, and the
    sequences that have a row."""
    case = state["case"]
    if case["packed"]:
        o = state["offsets"].long()
    else:
        o = torch.arange(case["batch"] + 1, device="cuda") * case["steps"]
    return o[:-1], o[1:] - o[:-1]


def keep_apart(state, a):
    """The decay with a zero at the first row of each sequence."""
    first, count = bounds(state)
    cut = torch.ones(a.shape[0] + 1, 1, device=a.device)
    cut[first] = 0.0  # an empty sequence at the end points past the list
    return a * cut[:-1]


def previous(state, h):
    """h_{t-1} of each row: the row above, the initial state at a first row."""
    first, count = bounds(state)
    prev = torch.cat([torch.zeros_like(h[:1]), h[:-1]]).float()
    some = count > 0
    h0 = state["h0"] if state["h0"] is not None else torch.zeros(first.shape[0], h.shape[1], device=h.device)
    prev[first[some]] = h0[some]
    return prev


def plain_forward(state):
    case = state["case"]
    a, u = decay_and_input(case["form"], flat(state, state["gate"]), flat(state, state["x"]))
    first, count = bounds(state)
    some = count > 0
    start = state["h0"] if state["h0"] is not None else torch.zeros(first.shape[0], u.shape[1], device=u.device)
    u = u.clone()
    u[first[some]] += a[first[some]] * start[some]
    if case["packed"]:
        h = inclusive_scan(keep_apart(state, a), u)
    else:
        shape = (case["batch"], case["steps"], case["width"])
        h = inclusive_scan(a.view(shape), u.view(shape)).reshape(-1, case["width"])
    last = start.clone()
    last[some] = h[(first + count - 1)[some]]
    return [h.to(state["x"].dtype).view(state["x"].shape), last]


def plain_backward(state):
    case = state["case"]
    shape = state["gate"].shape
    gate, x = flat(state, state["gate"]), flat(state, state["x"])
    a, _ = decay_and_input(case["form"], gate, x)
    first, count = bounds(state)
    some = count > 0
    final = (first + count - 1)[some]
    dh = flat(state, state["dh"]).float()
    if state["dh_last"] is not None:
        dh = dh.clone()
        dh[final] += state["dh_last"][some]
    # dh_t += a_{t+1} dh_{t+1}: the same scan from the last row up
    back = torch.cat([keep_apart(state, a)[1:], torch.zeros_like(a[:1])])
    if case["packed"]:
        dh = inclusive_scan(back.flip(0), dh.flip(0)).flip(0)
    else:
        cube = (case["batch"], case["steps"], case["width"])
        dh = inclusive_scan(back.view(cube).flip(1), dh.view(cube).flip(1)).flip(1).reshape(-1, case["width"])
    prev = previous(state, flat(state, state["h"]))
    if case["form"] == "decay":
        dgate, dx = dh * prev, dh
    elif case["form"] == "log":
        dgate, dx = dh * prev * a, dh
    else:
        rest = torch.sigmoid(-gate.float())
        dgate, dx = dh * (prev - x.float()) * a * rest, dh * rest
    zero = torch.zeros(first.shape[0], a.shape[1], device=a.device)
    dh0 = zero if state["dh_last"] is None else state["dh_last"].clone()
    dh0[some] = a[first[some]] * dh[first[some]]
    return [dgate.to(gate.dtype).view(shape), dx.to(gate.dtype).view(shape), dh0]


def plain_step(state):
    rows = state["slots"].long()
    a, u = decay_and_input(state["case"]["form"], state["gate"], state["x"])
    h = a * state["state"][rows] + u
    state["next"][rows] = h
    return [h.to(state["x"].dtype), state["next"]]


def plain_orth(g):
    a, b, c = COEFFICIENTS
    x = g.float()
    if x.shape[-2] > x.shape[-1]:
        x = x.transpose(-1, -2)
    x = x / (x.square().sum((-1, -2), keepdim=True).sqrt() + EPS)
    for _ in range(STEPS):
        s = x @ x.transpose(-1, -2)
        x = a * x + (b * s + c * (s @ s)) @ x
    if g.shape[-2] > g.shape[-1]:
        x = x.transpose(-1, -2)
    return x.to(torch.float16 if g.dtype == torch.float16 else torch.bfloat16).contiguous()


# ------------------------------------------------------------------ 64 bits
def exact(case, seed):
    if case["op"] == "scan" and case["steps"] > 200000 or work(case)["flops"] > 8e12:
        return None  # too long in 64 bits
    s = prepare(case, seed)
    if case["op"] == "orth":
        return exact_orth(s["g"].double())
    form = case["form"]

    def open_gate(g):
        g = g.double()
        return g if form == "decay" else g.exp() if form == "log" else 1 / (1 + (-g).exp())

    def shut_gate(g):
        return 1 / (1 + g.double().exp())

    if case["op"] == "step":
        rows = s["slots"].long()
        u = s["x"].double() * (shut_gate(s["gate"]) if form == "sigmoid" else 1.0)
        h = open_gate(s["gate"]) * s["state"].double()[rows] + u
        nxt = torch.zeros(s["next"].shape, dtype=torch.float64, device="cuda")
        nxt[rows] = h
        return [h, nxt]

    # token by token; a packed list goes sequence by sequence
    b, w = case["batch"], case["width"]
    if case["packed"]:
        o = s["offsets"].tolist()
        parts = [(slice(o[i], o[i + 1]), slice(i, i + 1)) for i in range(b)]
    else:
        parts = [(slice(None), slice(None))]
    start = s["h0"].double() if s["h0"] is not None else torch.zeros(b, w, dtype=torch.float64, device="cuda")

    def rows(t, part):
        return t[part].unsqueeze(0) if case["packed"] else t

    if case["direction"] == "forward":
        h = torch.empty(s["x"].shape, dtype=torch.float64, device="cuda")
        last = start.clone()
        for part, seq in parts:
            gate, x, out = rows(s["gate"], part), rows(s["x"], part), rows(h, part)
            cur = start[seq]
            for t in range(gate.shape[1]):
                u = x[:, t].double()
                if form == "sigmoid":
                    u = shut_gate(gate[:, t]) * u
                cur = open_gate(gate[:, t]) * cur + u
                out[:, t] = cur
            last[seq] = cur
        return [h, last]
    dgate = torch.empty(s["x"].shape, dtype=torch.float64, device="cuda")
    dx = torch.empty_like(dgate)
    dh0 = s["dh_last"].double() if s["dh_last"] is not None else torch.zeros_like(start)
    for part, seq in parts:
        gate, x, h, dh = (rows(s[k], part) for k in ("gate", "x", "h", "dh"))
        dg, du = rows(dgate, part), rows(dx, part)
        carry = dh0[seq].clone()
        for t in range(gate.shape[1] - 1, -1, -1):
            a = open_gate(gate[:, t])
            d = dh[:, t].double() + carry
            prev = h[:, t - 1].double() if t else start[seq]
            if form == "sigmoid":
                r = shut_gate(gate[:, t])
                dg[:, t] = d * (prev - x[:, t].double()) * a * r
                du[:, t] = d * r
            else:
                dg[:, t] = d * prev * (a if form == "log" else 1.0)
                du[:, t] = d
            carry = a * d
        dh0[seq] = carry
    return [dgate, dx, dh0]


def exact_orth(g):
    tall = g.shape[-2] > g.shape[-1]
    x = g.mT if tall else g
    x = x / (torch.linalg.matrix_norm(x, keepdim=True) + EPS)
    a, b, c = COEFFICIENTS
    one = torch.eye(x.shape[-2], dtype=torch.float64, device=x.device)
    for _ in range(STEPS):
        s = x @ x.mT
        x = (a * one + s @ (b * one + c * s)) @ x
    return (x.mT if tall else x).contiguous()
