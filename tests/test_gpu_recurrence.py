"""The gated linear recurrence on the GPU against a token-by-token
evaluation in 64 bits.

Tolerance.  A token does at most: the gate's value (exponential and
reciprocal, up to 4 roundings of 2^-24 relative), a product and a sum, and
once more each where runs of tokens are composed.  So the error of the state
obeys  e_t <= |a_t| e_{t-1} + 8 * 2^-24 (|a_t| s_{t-1} + |u_t|)  with s the
recurrence of the magnitudes, and the test carries that bound along; 16-bit
gates are opened with the hardware's exponential (2^-22 relative), so c is
four times larger there.  The output adds its own rounding (half a unit in
the last place), and for half the smallest step of its subnormals.
"""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

UNIT = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}  # bf16: 2^-9, doubled for ties of the bound itself
TINY = {"f32": 2.0 ** -149, "f16": 2.0 ** -25, "bf16": 2.0 ** -133}


@pytest.fixture(scope="module")
def env():
    import torch

    import triangular_solve_gb300 as tg
    from triangular_solve_gb300 import build
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    build.build()
    return torch, tg


def dtype_of(torch, name):
    return {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}[name]


def gate_values(rng, form, shape):
    if form == "decay":
        return rng.uniform(-0.3, 1.0, shape)
    if form == "log":
        return -np.exp(rng.uniform(-7, 1, shape))
    return rng.normal(2.0, 3.0, shape)


def opened(form, g):
    if form == "decay":
        return g, np.ones_like(g)
    if form == "log":
        return np.exp(g), np.ones_like(g)
    t = np.exp(-np.abs(g))
    big, small = 1 / (1 + t), t / (1 + t)
    return np.where(g >= 0, big, small), np.where(g >= 0, small, big)


def reference_forward(form, g, x, h0, c):
    """States (T, D), last state, and the bound on the float error of both."""
    T, D = g.shape
    a, r = opened(form, g)
    u = r * x if form == "sigmoid" else x
    h, s, e = h0.copy(), np.abs(h0), np.zeros(D)
    H, E = np.zeros((T, D)), np.zeros((T, D))
    for t in range(T):
        e = np.abs(a[t]) * e + c * (np.abs(a[t]) * s + np.abs(u[t]))
        s = np.abs(a[t]) * s + np.abs(u[t])
        h = a[t] * h + u[t]
        H[t], E[t] = h, e
    return H, h, E, e


def reference_backward(form, g, x, h, h0, dh, dlast, c):
    T, D = g.shape
    a, r = opened(form, g)
    carry, s, e = dlast.copy(), np.abs(dlast), np.zeros(D)
    dg, dx = np.zeros((T, D)), np.zeros((T, D))
    Eg, Ex = np.zeros((T, D)), np.zeros((T, D))
    for t in range(T - 1, -1, -1):
        d = dh[t] + carry
        ds, de = np.abs(dh[t]) + s, e + c * (np.abs(dh[t]) + s)
        prev = h[t - 1] if t else h0
        if form == "sigmoid":
            w, f = (prev - x[t]) * a[t] * r[t], r[t]
            m = (np.abs(prev) + np.abs(x[t])) * a[t] * r[t]
        else:
            f = np.ones(D)
            w = prev * (a[t] if form == "log" else 1.0)
            m = np.abs(w)
        dg[t], dx[t] = d * w, d * f
        Eg[t], Ex[t] = de * np.abs(w) + c * ds * m, de * f + c * ds * f
        carry, s, e = a[t] * d, np.abs(a[t]) * ds, np.abs(a[t]) * (de + c * ds)
    return dg, dx, carry, Eg, Ex, e


def factor(name):
    return (8 if name == "f32" else 32) * 2.0 ** -24


def near(got, want, bound, name, what):
    got = got.double().cpu().numpy()
    slack = bound + UNIT[name] * (np.abs(want) + bound) + TINY[name]
    over = np.abs(got - want) - slack
    assert np.all(over <= 0), f"{what}: {over.max():.3e} over its bound"


class Case:
    def __init__(self, torch, name, form, lengths, D, state, seed=0):
        rng = np.random.default_rng(seed)
        n = sum(lengths)
        self.torch, self.name, self.form, self.lengths, self.D = torch, name, form, lengths, D
        dt = dtype_of(torch, name)

        def dev(v, t):
            return torch.from_numpy(v).to(t).cuda()

        self.gate, self.x = dev(gate_values(rng, form, (n, D)), dt), dev(rng.normal(size=(n, D)), dt)
        self.dh = dev(rng.normal(size=(n, D)), dt)
        b = len(lengths)
        self.h0 = dev(rng.normal(size=(b, D)), torch.float32) if state else None
        self.dlast = dev(rng.normal(size=(b, D)), torch.float32) if state else None
        self.offsets = torch.tensor(np.concatenate([[0], np.cumsum(lengths)]), dtype=torch.int32, device="cuda")

    def sequences(self):
        r0 = 0
        for i, n in enumerate(self.lengths):
            yield i, slice(r0, r0 + n)
            r0 += n

    def arr(self, t, part):
        return t[part].double().cpu().numpy()

    def state(self, t, i):
        return np.zeros(self.D) if t is None else t[i].double().cpu().numpy()

    def check_forward(self, h, last):
        c = factor(self.name)
        for i, part in self.sequences():
            H, hl, E, e = reference_forward(self.form, self.arr(self.gate, part), self.arr(self.x, part),
                                            self.state(self.h0, i), c)
            near(h[part], H, E, self.name, f"h of sequence {i}")
            near(last[i], hl, e, "f32", f"last state of sequence {i}")

    def check_backward(self, h, dgate, dx, dh0):
        c = factor(self.name)
        for i, part in self.sequences():
            dg, du, d0, Eg, Ex, e0 = reference_backward(
                self.form, self.arr(self.gate, part), self.arr(self.x, part), self.arr(h, part),
                self.state(self.h0, i), self.arr(self.dh, part), self.state(self.dlast, i), c)
            near(dgate[part], dg, Eg, self.name, f"dgate of sequence {i}")
            near(dx[part], du, Ex, self.name, f"dx of sequence {i}")
            near(dh0[i], d0, e0, "f32", f"dh0 of sequence {i}")


SHAPES = [(1, 1, 1), (2, 1, 64), (3, 2, 33), (1, 127, 24), (2, 129, 130), (2, 300, 64), (1, 700, 72), (1, 2500, 8),
          (5, 33, 257), (1, 4100, 3)]


@pytest.mark.parametrize("name", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("form", ["decay", "log", "sigmoid"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_batched_forward_and_backward(env, name, form, shape):
    torch, tg = env
    b, T, D = shape
    c = Case(torch, name, form, [T] * b, D, state=T % 2 == 1, seed=T + D)
    g, x, dh = (t.view(b, T, D) for t in (c.gate, c.x, c.dh))
    h, last = tg.linear_recurrence(g, x, c.h0, form=form)
    assert h.dtype == g.dtype and last.dtype == torch.float32
    c.check_forward(h.view(-1, D), last)
    grads = tg.linear_recurrence_backward(g, x, h, dh, c.h0, c.dlast, form=form)
    c.check_backward(h.view(-1, D), grads[0].view(-1, D), grads[1].view(-1, D), grads[2])


@pytest.mark.parametrize("name", ["f32", "bf16"])
@pytest.mark.parametrize("form", ["decay", "sigmoid"])
@pytest.mark.parametrize("lengths", [[0], [1], [0, 0, 3], [5, 0, 1, 1, 130, 0], [257, 1, 1024, 64], [3, 2000, 2],
                                     [7] * 45 + [600, 0] + [2] * 30 + [513, 1500, 1]], ids=str)
@pytest.mark.parametrize("D", [40, 61])
def test_packed_sequences(env, name, form, lengths, D):
    torch, tg = env
    c = Case(torch, name, form, lengths, D, state=True, seed=len(lengths))
    h, last = tg.linear_recurrence(c.gate, c.x, c.h0, form=form, offsets=c.offsets)
    c.check_forward(h, last)
    grads = tg.linear_recurrence_backward(c.gate, c.x, h, c.dh, c.h0, c.dlast, form=form, offsets=c.offsets)
    c.check_backward(h, *grads)


# Each number of lanes and threads that the number of channels selects, over
# more than one step of a cluster.
@pytest.mark.parametrize("name", ["f32", "bf16"])
@pytest.mark.parametrize("shape", [(1, 2500, 57), (1, 2500, 327), (1, 2500, 1025), (1, 2500, 640), (2, 1100, 1024),
                                   (7, 600, 648), (1, 9000, 5), (40, 130, 8), (40, 130, 16), (70, 90, 24)], ids=str)
def test_plans_of_batched_sequences(env, name, shape):
    torch, tg = env
    b, T, D = shape
    c = Case(torch, name, "sigmoid", [T] * b, D, state=True, seed=T + D)
    g, x, dh = (t.view(b, T, D) for t in (c.gate, c.x, c.dh))
    h, last = tg.linear_recurrence(g, x, c.h0, form="sigmoid")
    c.check_forward(h.view(-1, D), last)
    grads = tg.linear_recurrence_backward(g, x, h, dh, c.h0, c.dlast, form="sigmoid")
    c.check_backward(h.view(-1, D), grads[0].view(-1, D), grads[1].view(-1, D), grads[2])


@pytest.mark.parametrize("name", ["f32", "bf16"])
@pytest.mark.parametrize("D", [5, 8, 57, 327, 1025, 320, 648])
def test_plans_of_packed_sequences(env, name, D):
    torch, tg = env
    c = Case(torch, name, "log", [3, 0, 2300, 40, 600], D, state=True, seed=D)
    h, last = tg.linear_recurrence(c.gate, c.x, c.h0, form="log", offsets=c.offsets)
    c.check_forward(h, last)
    grads = tg.linear_recurrence_backward(c.gate, c.x, h, c.dh, c.h0, c.dlast, form="log", offsets=c.offsets)
    c.check_backward(h, *grads)


def test_empty_sequences_pass_their_state_on(env):
    torch, tg = env
    h0 = torch.randn(4, 24, device="cuda")
    g = torch.zeros(4, 0, 24, device="cuda")
    h, last = tg.linear_recurrence(g, g, h0)
    assert h.shape == (4, 0, 24) and torch.equal(last, h0)
    assert torch.equal(tg.linear_recurrence_backward(g, None, g, g, None, h0)[2], h0)
    assert torch.equal(tg.linear_recurrence(g, g)[1], torch.zeros_like(h0))
    for shape in ((0, 5, 24), (3, 5, 0)):
        e = torch.zeros(shape, device="cuda")
        h, last = tg.linear_recurrence(e, e)
        assert h.shape == shape and last.shape == (shape[0], shape[2])


def test_offsets_outside_the_list_are_held_inside(env):
    """Row numbers past either end count as the nearest row, a decreasing
    pair as an empty sequence, and rows of no sequence stay as they were."""
    torch, tg = env
    T, D = 50, 32
    g = torch.rand(T, D, device="cuda")
    x = torch.randn(T, D, device="cuda")
    off = torch.tensor([-7, 10, 30, 20, 1000], dtype=torch.int32, device="cuda")
    h = torch.full((T, D), 7.0, device="cuda")
    last = torch.empty(4, D, device="cuda")
    tg.trsm_linrec_forward("f32", "decay", 4, T, D, g, 0, D, x, 0, D, None, 0, off, h, 0, D, last)
    want, wl = tg.linear_recurrence(g, x, offsets=torch.tensor([0, 10, 30], dtype=torch.int32, device="cuda"))
    assert torch.equal(last[:2], wl) and torch.equal(last[2], torch.zeros(D, device="cuda"))
    assert torch.equal(h[:20], want[:20])
    tail, tl = tg.linear_recurrence(g[20:], x[20:], offsets=torch.tensor([0, 30], dtype=torch.int32, device="cuda"))
    assert torch.equal(h[30:], tail[10:])  # rows 20 .. 29 belong to two sequences
    assert torch.equal(last[3], tl[0])
    off = torch.tensor([10, 20], dtype=torch.int32, device="cuda")
    h.fill_(7.0)
    tg.trsm_linrec_forward("f32", "decay", 1, T, D, g, 0, D, x, 0, D, None, 0, off, h, 0, D, None)
    assert torch.all(h[:10] == 7) and torch.all(h[20:] == 7)


@pytest.mark.parametrize("name", ["f32", "bf16"])
@pytest.mark.parametrize("layout", ["halves", "time_major", "odd_offset", "shared_gate", "reversed_batch"])
def test_strides(env, name, layout):
    torch, tg = env
    b, T, D = 3, 70, 48
    dt = dtype_of(torch, name)
    gen = torch.Generator("cuda").manual_seed(3)

    def rnd(*s):
        return torch.rand(s, generator=gen, device="cuda").to(dt)

    if layout == "halves":
        both = rnd(b, T, 2 * D)
        g, x = both[..., :D], both[..., D:]
    elif layout == "time_major":
        g, x = rnd(T, b, D).transpose(0, 1), rnd(T, b, D).transpose(0, 1)
    elif layout == "odd_offset":
        g, x = rnd(b, T, D + 1)[..., 1:], rnd(b, T, D + 3)[..., 2:D + 2]
    elif layout == "shared_gate":
        g, x = rnd(1, 1, D).expand(b, T, D), rnd(b, T, D)
    else:
        g, x = rnd(b + 1, T, D)[1:], rnd(b, 2 * T, D)[:, ::2]
    h, last = tg.linear_recurrence(g, x)
    hc, lc = tg.linear_recurrence(g.contiguous(), x.contiguous())
    assert torch.allclose(h.float(), hc.float(), rtol=2 * UNIT[name], atol=1e-6)
    assert torch.allclose(last, lc, rtol=1e-5, atol=1e-6)
    dh = rnd(1, T, 2 * D)[..., :D].expand(b, T, D)
    got = tg.linear_recurrence_backward(g, x, h, dh, form="sigmoid")
    want = tg.linear_recurrence_backward(g.contiguous(), x.contiguous(), h.contiguous(), dh.contiguous(),
                                         form="sigmoid")
    for a, w in zip(got, want):
        assert torch.allclose(a.float(), w.float(), rtol=2 * UNIT[name], atol=1e-5)


def test_rows_further_apart_than_32_bits_reach(env):
    torch, tg = env
    T, D, far = 35, 40, 1 << 27  # the last row starts past 2^32 elements
    buf = torch.empty((T - 1) * far + 2 * D, dtype=torch.bfloat16, device="cuda")
    g, x = (buf.as_strided((1, T, D), (0, far, 1), k * D) for k in (0, 1))
    g.copy_(torch.rand(1, T, D, device="cuda"))
    x.copy_(torch.randn(1, T, D, device="cuda"))
    h, last = tg.linear_recurrence(g, x)
    hc, lc = tg.linear_recurrence(g.contiguous(), x.contiguous())
    assert torch.equal(h, hc) and torch.equal(last, lc)
    got = tg.linear_recurrence_backward(g, None, h, x)
    want = tg.linear_recurrence_backward(g.contiguous(), None, h, x.contiguous())
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_equals_the_bidiagonal_solve(env):
    """The recurrence is the solve with the unit lower bidiagonal matrix."""
    torch, tg = env
    T, D = 96, 5
    a = torch.rand(1, T, 1, device="cuda").expand(1, T, D).contiguous()
    x = torch.randn(1, T, D, device="cuda")
    h, _ = tg.linear_recurrence(a, x)
    L = torch.eye(T, device="cuda") - torch.diag(a[0, 1:, 0], -1)
    X = x[0].clone()
    tg.solve(L, X)
    assert torch.allclose(h[0], X, rtol=1e-5, atol=1e-5)


def test_resets_and_values_that_are_not_finite(env):
    """A zero decay starts anew; a NaN or infinity stays in its channel, in
    its sequence, and after its token (before it, in the backward pass)."""
    torch, tg = env
    b, T, D = 2, 600, 16
    g = torch.full((b, T, D), 0.999, device="cuda")
    x = torch.randn(b, T, D, device="cuda")
    clean, _ = tg.linear_recurrence(g, x)
    g2 = g.clone()
    g2[:, 300] = 0
    h, _ = tg.linear_recurrence(g2, x)
    fresh, _ = tg.linear_recurrence(g[:, 300:].contiguous(), x[:, 300:].contiguous())
    assert torch.allclose(h[:, 300:], fresh, rtol=1e-4, atol=1e-4) and torch.equal(h[:, :128], clean[:, :128])
    for bad in (float("nan"), float("inf"), -float("inf")):
        x2 = x.clone()
        x2[1, 200, 3] = bad
        h, last = tg.linear_recurrence(g, x2)
        assert not torch.isfinite(h[1, 200:, 3]).any() and not torch.isfinite(last[1, 3])
        h[1, 200:, 3] = clean[1, 200:, 3]
        assert torch.isfinite(h).all() and torch.allclose(h, clean, rtol=1e-5, atol=1e-4)
        dh = x.clone()
        dh[0, 100, 7] = bad
        base = tg.linear_recurrence_backward(g, None, clean, x)
        got = tg.linear_recurrence_backward(g, None, clean, dh)
        assert not torch.isfinite(got[1][0, :101, 7]).any() and not torch.isfinite(got[2][0, 7])
        got[1][0, :101, 7] = base[1][0, :101, 7]
        assert torch.isfinite(got[1]).all() and torch.allclose(got[1], base[1], rtol=1e-5, atol=1e-4)


@pytest.mark.parametrize("form", ["log", "sigmoid"])
@pytest.mark.parametrize("name", ["f32", "f16", "bf16"])
def test_extreme_gates(env, name, form):
    """Gates far out close or open fully, without infinities or NaN."""
    torch, tg = env
    dt = dtype_of(torch, name)
    low = torch.finfo(dt).min
    g = torch.tensor([low, -float("inf"), -90.0, -20.0, 0.0], device="cuda", dtype=dt)
    if form == "sigmoid":
        g = torch.cat([g, torch.tensor([20.0, 90.0, float("inf"), -low], device="cuda", dtype=dt)])
    n = g.numel()
    gate = g.view(1, n, 1).expand(1, n, 4).contiguous()
    x = torch.ones(1, n, 4, device="cuda", dtype=dt)
    h, last = tg.linear_recurrence(gate, x, form=form)
    a, r = opened(form, np.nan_to_num(g.double().cpu().numpy(), neginf=-1e4, posinf=1e4))
    cur, want = 0.0, []
    for t in range(n):
        cur = a[t] * cur + (r[t] if form == "sigmoid" else 1.0)
        want.append(cur)
    assert np.allclose(h[0, :, 0].double().cpu().numpy(), want, rtol=2 * UNIT[name], atol=1e-6)
    grads = tg.linear_recurrence_backward(gate, x, h, x, form=form)
    assert all(torch.isfinite(t).all() for t in grads)


def test_runs_are_identical(env):
    torch, tg = env
    g = torch.rand(2, 3000, 200, device="cuda")
    x = torch.randn(2, 3000, 200, device="cuda")
    h, last = tg.linear_recurrence(g, x)
    grads = tg.linear_recurrence_backward(g, x, h, x, form="sigmoid")
    for _ in range(5):
        again = tg.linear_recurrence(g, x) + tg.linear_recurrence_backward(g, x, h, x, form="sigmoid")
        assert all(torch.equal(a, b) for a, b in zip((h, last) + grads, again))


def test_runs_on_the_current_stream(env):
    torch, tg = env
    g = torch.rand(4, 2000, 256, device="cuda")
    x = torch.randn(4, 2000, 256, device="cuda")
    want, _ = tg.linear_recurrence(g, x)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        y = x
        for _ in range(4):
            y = y * 2 / 2  # queued work the call has to come after
        h, _ = tg.linear_recurrence(g, y)
    s.synchronize()
    assert torch.equal(h, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        h, last = tg.linear_recurrence(g, x)
    x.mul_(2)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(h, 2 * want)


@pytest.mark.parametrize("name", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("form", ["decay", "log", "sigmoid"])
@pytest.mark.parametrize("b,D,slots", [(1, 1, 1), (1, 128, 4), (7, 61, 9), (33, 264, 40)])
def test_single_tokens(env, name, form, b, D, slots):
    torch, tg = env
    dt = dtype_of(torch, name)
    rng = np.random.default_rng(b + D)
    g = torch.from_numpy(gate_values(rng, form, (b, D))).to(dt).cuda()
    x = torch.from_numpy(rng.normal(size=(b, D))).to(dt).cuda()
    state = torch.from_numpy(rng.normal(size=(slots, D))).float().cuda()
    where = rng.permutation(slots)[:b]
    idx = torch.tensor(where, dtype=torch.int32, device="cuda")
    before = state.clone()
    out = torch.full_like(state, 7.0)
    y = tg.linear_recurrence_step(g, x, state, form=form, slots=idx, out_state=out)
    assert torch.equal(state, before)
    rest = [s for s in range(slots) if s not in set(where)]
    assert torch.all(out[rest] == 7.0)
    for i in range(b):
        H, last, E, e = reference_forward(form, g[i:i + 1].double().cpu().numpy(), x[i:i + 1].double().cpu().numpy(),
                                          before[where[i]].double().cpu().numpy(), factor(name))
        near(y[i], H[0], E[0], name, "y")
        near(out[where[i]], last, e, "f32", "state")
    y2 = tg.linear_recurrence_step(g, x, state, form=form, slots=idx)  # in place
    assert torch.equal(y2, y) and torch.equal(state[where], out[where]) and torch.equal(state[rest], before[rest])
    if slots > b:
        idx = torch.tensor([-1] + list(range(1, b)), dtype=torch.int32, device="cuda")
        idx[b // 2] = slots if b > 1 else -5
        keep = state.clone()
        y = tg.linear_recurrence_step(g, x, state, form=form, slots=idx)
        assert torch.all(y[0] == 0) and torch.all(y[b // 2] == 0) and torch.equal(state[0], keep[0])


def test_single_tokens_continue_a_sequence(env):
    torch, tg = env
    g = torch.rand(3, 40, 72, device="cuda")
    x = torch.randn(3, 40, 72, device="cuda")
    h, last = tg.linear_recurrence(g, x, form="sigmoid")
    _, state = tg.linear_recurrence(g[:, :30].contiguous(), x[:, :30].contiguous(), form="sigmoid")
    for t in range(30, 40):
        y = tg.linear_recurrence_step(g[:, t], x[:, t], state, form="sigmoid")
        assert torch.allclose(y, h[:, t], rtol=1e-5, atol=1e-6)
    assert torch.allclose(state, last, rtol=1e-5, atol=1e-6)


@pytest.mark.parametrize("form", ["decay", "log", "sigmoid"])
def test_gradients_against_differences(env, form):
    """Central differences of the kernel's own float forward along random
    directions.  With step 2^-6 the truncation is about 2^-12 of the third
    derivative's scale and the rounding 2^-24 / 2^-6 of the function's, so
    1e-2 of the directional derivative's scale has a wide margin."""
    torch, tg = env
    gen = torch.Generator("cuda").manual_seed(5)

    def rnd(*s):
        return torch.randn(s, generator=gen, device="cuda")

    b, T, D = 2, 37, 12
    g = rnd(b, T, D) * 0.3 + (0.5 if form == "decay" else -0.7)
    x, h0, w, wl = rnd(b, T, D), rnd(b, D), rnd(b, T, D), rnd(b, D)
    args = [t.clone().requires_grad_() for t in (g, x, h0)]
    h, last = tg.linear_recurrence(*args, form=form)
    ((h * w).sum() + (last * wl).sum()).backward()

    def f(*v):
        h, last = tg.linear_recurrence(*v, form=form)
        return ((h.double() * w).sum() + (last.double() * wl).sum()).item()

    for k in range(3):
        v = rnd(*args[k].shape)
        step = 2.0 ** -6
        up = [t.detach() + (step * v if i == k else 0) for i, t in enumerate(args)]
        down = [t.detach() - (step * v if i == k else 0) for i, t in enumerate(args)]
        slope = (f(*up) - f(*down)) / (2 * step)
        scale = (args[k].grad.double().norm() * v.double().norm()).item()
        assert abs(slope - (args[k].grad.double() * v).sum().item()) <= 1e-2 * scale, k


def test_autograd_matches_the_backward_call(env):
    torch, tg = env
    g = torch.randn(2, 50, 24, device="cuda").bfloat16().requires_grad_()
    x = torch.randn(2, 50, 24, device="cuda").bfloat16().requires_grad_()
    h, last = tg.linear_recurrence(g, x, form="sigmoid")
    h.sum().backward()  # a broadcast gradient, and none for the last state
    want = tg.linear_recurrence_backward(g.detach(), x.detach(), h.detach(), torch.ones_like(h), form="sigmoid")
    assert torch.equal(g.grad, want[0]) and torch.equal(x.grad, want[1])
    shared = torch.full((24,), 0.5, device="cuda", requires_grad=True)
    y = torch.randn(2, 50, 24, device="cuda")
    h, last = tg.linear_recurrence(shared.expand(2, 50, 24), y)
    last.sum().backward()
    dgate = tg.linear_recurrence_backward(shared.detach().expand(2, 50, 24), None, h.detach(), torch.zeros_like(h),
                                          None, torch.ones(2, 24, device="cuda"))[0]
    assert torch.allclose(shared.grad, dgate.sum((0, 1)), rtol=1e-5)


def test_refusals(env):
    torch, tg = env
    g = torch.rand(2, 5, 8, device="cuda")
    for bad in (g[:, :4], g.half(), g.cpu()):
        with pytest.raises((ValueError, TypeError)):
            tg.linear_recurrence(g, bad)
    with pytest.raises(ValueError, match="contiguous"):
        tg.linear_recurrence(g, torch.rand(2, 8, 5, device="cuda").transpose(1, 2))
    with pytest.raises(ValueError, match="contiguous"):
        tg.linear_recurrence(torch.rand(2, 8, 5, device="cuda").transpose(1, 2), g)
    with pytest.raises(TypeError):
        tg.linear_recurrence(g.double(), g.double())
    with pytest.raises(ValueError):
        tg.linear_recurrence(g, g, form="tanh")
    with pytest.raises(ValueError):
        tg.linear_recurrence(g[0], g[0])
    with pytest.raises(TypeError):
        tg.linear_recurrence(g, g, torch.zeros(2, 8, device="cuda").half())
    with pytest.raises(ValueError):
        tg.linear_recurrence(g, g, torch.zeros(2, 7, device="cuda"))
    with pytest.raises(ValueError):
        tg.linear_recurrence(g[0], g[0], offsets=torch.tensor([0, 5], device="cuda"))  # int64
    with pytest.raises(ValueError):
        tg.linear_recurrence(g[0], g[0], offsets=torch.tensor([0, 5], dtype=torch.int32))  # on the CPU
    with pytest.raises(ValueError, match="sigmoid"):
        tg.linear_recurrence_backward(g, None, g, g, form="sigmoid")
    with pytest.raises(ValueError):
        tg.linear_recurrence_step(g[0], g[0], torch.zeros(5, 7, device="cuda"))
    with pytest.raises(ValueError):
        tg.linear_recurrence_step(g[0], g[0], torch.zeros(5, 8, device="cuda"),
                                  slots=torch.zeros(4, dtype=torch.int32, device="cuda"))
    # fewer states than rows: the rows without one are padding
    y = tg.linear_recurrence_step(g[0], g[0], torch.zeros(3, 8, device="cuda"))
    assert torch.all(y[3:] == 0) and torch.equal(y[:3], g[0][:3])


def test_expired_wait_is_reported_and_leaves_the_device_usable(env):
    """A sequence long enough for a cluster, with a wait limit of zero polls:
    the exchange between the CTAs gives up, the status word says so, and the
    next call is right again."""
    torch, tg = env
    g = torch.rand(1, 5000, 64, device="cuda")
    x = torch.randn(1, 5000, 64, device="cuda")
    want, last = tg.linear_recurrence(g, x)
    assert tg.trsm_device_status() == 0
    tg.trsm_set_wait_limit(0)
    try:
        tg.linear_recurrence(g, x)
        assert tg.trsm_device_status() == tg.ERR_DEVICE_TIMEOUT
    finally:
        tg.trsm_set_wait_limit(-1)
    h, l2 = tg.linear_recurrence(g, x)
    assert torch.equal(h, want) and torch.equal(l2, last) and tg.trsm_device_status() == 0


def test_marshalled_calls_equal_the_python_ones(env, monkeypatch):
    """The calls' C half takes plain calls and leaves everything else to the
    Python half, with the same results."""
    import sysconfig
    import os
    torch, tg = env
    from triangular_solve_gb300 import model
    model._load_torch()
    if not os.path.exists(os.path.join(sysconfig.get_paths()["include"], "Python.h")):
        pytest.skip("Python's headers are not here")
    m = model._marshal
    assert m is not None
    gen = torch.Generator("cuda").manual_seed(1)

    def rnd(*s, dtype=torch.bfloat16):
        return torch.randn(s, generator=gen, device="cuda").to(dtype)

    both = rnd(3, 40, 64)
    g, x = both[..., :32], both[..., 32:]
    h0, dl = rnd(3, 32, dtype=torch.float32), rnd(3, 32, dtype=torch.float32)
    off = torch.tensor([0, 3, 40], dtype=torch.int32, device="cuda")
    slots = torch.tensor([4, 0, 2], dtype=torch.int32, device="cuda")
    table = rnd(5, 32, dtype=torch.float32)

    def calls(out):
        h, last = tg.linear_recurrence(g, x, h0, form="sigmoid")
        r = [h, last, *tg.linear_recurrence(g[0], x[0], form="decay", offsets=off)]
        r += tg.linear_recurrence_backward(g, x, h, x, h0, dl, form="sigmoid")
        r += tg.linear_recurrence_backward(g[0], None, h[0], x[0], offsets=off)
        return r + [tg.linear_recurrence_step(g[:, 0], x[:, 0], table, form="log", slots=slots, out_state=out), out]

    assert m.forward(g, x, h0, "sigmoid", None) is not None
    fast = calls(torch.zeros_like(table))
    monkeypatch.setattr(model, "_marshal", None)
    slow = calls(torch.zeros_like(table))
    assert len(fast) == len(slow) and all(torch.equal(a, b) for a, b in zip(fast, slow))
    for bad in ((g.cpu(), x, None, "decay", None), (g, x.float(), None, "decay", None), (g, x, h0[:2], "decay", None),
                (g, x, None, "tanh", None), (g[0], x[0], None, "decay", None), (g, x, None, 0, None),
                (g.transpose(1, 2), x, None, "decay", None), (None, x, None, "decay", None), (g, x, None, "decay", off)):
        assert m.forward(*bad) is None
    assert m.step(g[:, 0], x[:, 0], table, "log", slots[:2], None) is None
    assert m.step(g[:, 0], x[:, 0], table[:, :8], "log", slots, None) is None
    assert m.backward(g, None, g, x, None, None, "sigmoid", None) is None
