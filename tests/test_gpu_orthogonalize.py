"""Newton-Schulz orthogonalisation on the GPU against the same steps in 64
bits.

Tolerance, relative to |O|_F.  A rounding to f16 moves a matrix by
2^-12 / sqrt(3) = 1.4e-4 of its Frobenius norm.  X's rounding is amplified at
most 16 times by the steps to come, 24 times with the steps after it; S and C
are rounded once a step each and enter with a factor up to |b| + 2 |c| = 9,
independently from step to step: 24 * 1.4e-4 + 9 * sqrt(2 * 5) * 1.4e-4 = 7.4e-3.
The result adds its own rounding, 2^-9 or 2^-12.
"""
import ctypes

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

DEFAULT = (3.4445, -4.7750, 2.0315)
TOL = {"bf16": 7.4e-3 + 2.0 ** -9, "f16": 7.4e-3 + 2.0 ** -12}


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


def matrices(kind, b, m, n, seed=0):
    rng = np.random.default_rng(seed)
    r = min(m, n)
    if kind == "noise":
        return rng.normal(size=(b, m, n))
    if kind == "low_rank":
        k = max(1, r // 16)
        return rng.normal(size=(b, m, k)) * np.exp(-np.arange(k) / 4) @ rng.normal(size=(b, k, n)) + \
            0.01 * rng.normal(size=(b, m, n))
    if kind == "rank_one":
        return rng.normal(size=(b, m, 1)) @ rng.normal(size=(b, 1, n))
    if kind == "spike":
        g = 1e-3 * rng.normal(size=(b, m, n))
        g[:, -1, -1] = 50.0
        return g
    u = np.linalg.qr(rng.normal(size=(b, m, r)))[0]
    v = np.linalg.qr(rng.normal(size=(b, n, r)))[0]
    s = np.ones(r) if kind == "orthonormal" else np.arange(1, r + 1.0) ** -1.5  # or "power_law"
    return u * s @ v.transpose(0, 2, 1)


def reference(g, steps=5, coef=DEFAULT, eps=1e-7):
    coef = [coef] * steps if np.ndim(coef[0]) == 0 else coef
    x = g if g.shape[-2] <= g.shape[-1] else g.transpose(0, 2, 1)
    x = x / (np.sqrt((x * x).sum((1, 2), keepdims=True)) + eps)
    for a, b, c in coef:
        s = x @ x.transpose(0, 2, 1)
        x = a * x + b * (s @ x) + c * (s @ (s @ x))
    return x if g.shape[-2] <= g.shape[-1] else x.transpose(0, 2, 1)


def errors(got, want):
    got = got.double().cpu().numpy()
    return np.linalg.norm((got - want).reshape(len(want), -1), axis=1) / np.linalg.norm(
        want.reshape(len(want), -1), axis=1)


SHAPES = [(1, 1, 1), (2, 1, 500), (2, 500, 1), (3, 2, 3), (4, 17, 5), (5, 64, 64), (3, 65, 64), (2, 100, 1001),
          (1, 256, 257), (2, 300, 130), (1, 513, 700), (1, 1000, 384), (40, 32, 48), (3, 128, 128), (2, 129, 128),
          (2, 31, 1200), (2, 33, 600), (2, 65, 240), (1, 128, 300), (1, 120, 320), (2, 1600, 20),
          (3, 25, 4023), (1, 9, 65), (2, 2000, 61), (1, 127, 2111), (90, 60, 900), (1, 128, 5000), (80, 100, 700)]


@pytest.mark.parametrize("name", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("kind", ["noise", "low_rank"])
def test_parity(env, name, shape, kind):
    torch, tg = env
    G = torch.from_numpy(matrices(kind, *shape)).to(dtype_of(torch, name)).cuda()
    O = tg.orthogonalize(G)
    assert O.dtype == (torch.float16 if name == "f16" else torch.bfloat16) and O.shape == G.shape
    e = errors(O, reference(G.double().cpu().numpy()))
    assert e.max() <= TOL["f16" if name == "f16" else "bf16"], e.max()


@pytest.mark.parametrize("kind", ["rank_one", "spike", "orthonormal", "power_law"])
@pytest.mark.parametrize("name,out", [("f32", "bf16"), ("f32", "f16"), ("bf16", "f16"), ("f16", "bf16")])
@pytest.mark.parametrize("shape", [(2, 96, 96), (1, 200, 520), (1, 520, 200)], ids=str)
def test_spectra_and_output_types(env, kind, name, out, shape):
    torch, tg = env
    G = torch.from_numpy(matrices(kind, *shape)).to(dtype_of(torch, name)).cuda()
    O = torch.empty(G.shape, dtype=dtype_of(torch, out), device="cuda")
    assert tg.orthogonalize(G, out=O) is O
    e = errors(O, reference(G.double().cpu().numpy()))
    assert e.max() <= TOL[out], e.max()


def test_singular_values_come_near_one(env):
    torch, tg = env
    G = torch.randn(300, 900, device="cuda")
    s = torch.linalg.svdvals(tg.orthogonalize(G).float())
    assert s.min() > 0.65 and s.max() < 1.25
    # a convergent polynomial takes them all the way
    cubic = (1.5, -0.5, 0.0)
    s = torch.linalg.svdvals(tg.orthogonalize(G, steps=20, coefficients=cubic).float())
    assert (s - 1).abs().max() < 2e-2


@pytest.mark.parametrize("steps,coef", [(0, None), (1, None), (2, (1.5, -0.5, 0.0)),
                                        (3, [(4.0, -6.0, 3.0), (3.0, -4.0, 2.0), (1.875, -1.25, 0.375)])])
@pytest.mark.parametrize("shape", [(2, 70, 90), (2, 90, 70)], ids=str)
def test_steps_and_coefficients(env, steps, coef, shape):
    torch, tg = env
    G = torch.from_numpy(matrices("noise", *shape)).float().cuda()
    O = tg.orthogonalize(G, steps=steps, coefficients=coef)
    e = errors(O, reference(G.double().cpu().numpy(), steps, coef or DEFAULT))
    assert e.max() <= TOL["bf16"]


@pytest.mark.parametrize("shape", [(3, 40, 72), (3, 72, 41), (2, 150, 150)], ids=str)
@pytest.mark.parametrize("layout", ["padded", "odd_padding", "column_major", "odd_offset", "one_matrix"])
def test_layouts(env, shape, layout):
    torch, tg = env
    b, m, n = shape
    g = torch.from_numpy(matrices("noise", *shape)).bfloat16().cuda()
    want = reference(g.double().cpu().numpy())
    if layout in ("padded", "odd_padding"):
        p = 8 if layout == "padded" else 3
        G = torch.zeros(b, m + 2, n + p, dtype=g.dtype, device="cuda")[:, :m, :n]
        full = torch.full((b, m + 2, n + p), 7.0, dtype=torch.bfloat16, device="cuda")
        G.copy_(g)
        tg.orthogonalize(G, out=full[:, :m, :n])
        O = full[:, :m, :n].clone()
        full[:, :m, :n] = 7.0
        assert torch.all(full == 7.0), "wrote outside the matrices"
    elif layout == "column_major":
        G = g.mT.contiguous().mT
        O = tg.orthogonalize(G)
        assert O.stride() == G.stride()
    elif layout == "odd_offset":
        G = torch.zeros(b * m * n + 1, dtype=g.dtype, device="cuda")[1:].view(b, m, n)
        out = torch.zeros(b * m * n + 1, dtype=g.dtype, device="cuda")[1:].view(b, m, n)
        G.copy_(g)
        O = tg.orthogonalize(G, out=out)
    else:
        O = torch.stack([tg.orthogonalize(x) for x in g])
    assert errors(O, want).max() <= TOL["bf16"]


@pytest.mark.parametrize("scale", [1e-38, 1e-30, 1e-3, 1e18, 1e30, 1e36])
def test_scale_of_the_input_does_not_matter(env, scale):
    torch, tg = env
    g = torch.from_numpy(matrices("low_rank", 1, 60, 90)).float().cuda() * scale
    O = tg.orthogonalize(g, eps=0.0)
    x = g.double().cpu().numpy()
    assert errors(O, reference(x, eps=0.0)).max() <= TOL["bf16"]


def test_zero_and_non_finite_matrices(env):
    """Zero stays zero (eps), a NaN or infinity makes its own matrix NaN and
    leaves the others of the batch alone."""
    torch, tg = env
    for shape in ((6, 50, 70), (6, 300, 200)):
        g = torch.from_numpy(matrices("noise", *shape)).float().cuda()
        want = tg.orthogonalize(g)
        g[1] = 0
        g[2, 3, 4] = float("nan")
        g[4, -1, -1] = float("inf")
        O = tg.orthogonalize(g)
        assert torch.all(O[1] == 0) and torch.isnan(O[2]).all() and torch.isnan(O[4]).all()
        for k in (0, 3, 5):
            assert torch.equal(O[k], want[k])
        assert torch.isnan(tg.orthogonalize(g[2], steps=0)).all()


def test_empty(env):
    torch, tg = env
    for shape in ((0, 4, 5), (3, 0, 5), (3, 5, 0), (0, 5)):
        assert tg.orthogonalize(torch.empty(shape, device="cuda")).shape == shape


def test_own_workspace(env):
    torch, tg = env
    b, m, n = 2, 190, 230
    G = torch.randn(b, m, n, device="cuda")
    want = tg.orthogonalize(G)
    need = tg.trsm_orthogonalize_workspace_bytes("f32", m, n, b)
    ws = torch.full((need + 256,), 255, dtype=torch.uint8, device="cuda")  # NaN patterns
    O = torch.empty(b, m, n, dtype=torch.bfloat16, device="cuda")

    def call(p, size):
        tg.trsm_orthogonalize("f32", "bf16", m, n, G, n, m * n, O, n, m * n, b, workspace=p, ws_bytes=size)

    call(ws, need)
    assert torch.equal(O, want) and torch.all(ws[need:] == 255)
    for p, size in ((ws.data_ptr(), need - 1), (ws.data_ptr() + 8, need)):
        with pytest.raises(tg.TrsmError) as e:
            call(p, size)
        assert e.value.status == tg.ERR_WORKSPACE


def test_runs_are_identical_and_follow_the_stream(env):
    torch, tg = env
    G = torch.randn(3, 400, 300, device="cuda")
    want = tg.orthogonalize(G)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        H = G
        for _ in range(4):
            H = H * 2 / 2
        O = tg.orthogonalize(H)
    s.synchronize()
    assert torch.equal(O, want)
    graph = torch.cuda.CUDAGraph()
    out = torch.empty_like(want)
    need = tg.trsm_orthogonalize_workspace_bytes("f32", 400, 300, 3)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    with torch.cuda.graph(graph):
        tg.trsm_orthogonalize("f32", "bf16", 400, 300, G, 300, 120000, out, 300, 120000, 3, workspace=ws, ws_bytes=need)
    G.mul_(4)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)  # the scale of G does not matter, a power of two exactly
    assert tg.trsm_device_status() == 0


def test_refusals(env):
    torch, tg = env
    g = torch.randn(4, 6, device="cuda")
    with pytest.raises(TypeError):
        tg.orthogonalize(g.double())
    with pytest.raises(ValueError):
        tg.orthogonalize(g[0])
    with pytest.raises(ValueError):
        tg.orthogonalize(torch.randn(4, 12, device="cuda")[:, ::2])
    with pytest.raises(TypeError):
        tg.orthogonalize(g, out=torch.empty(4, 6, device="cuda"))
    with pytest.raises(ValueError):
        tg.orthogonalize(g, out=torch.empty(6, 4, device="cuda").bfloat16())
    with pytest.raises(ValueError):
        tg.orthogonalize(g, out=torch.empty(6, 4, device="cuda").bfloat16().T)  # column-major
    with pytest.raises(ValueError):
        tg.orthogonalize(g, steps=3, coefficients=[(1, 2, 3), (1, 2, 3)])
    with pytest.raises(ValueError):
        tg.orthogonalize(g, steps=-1)
    with pytest.raises(tg.TrsmError) as e:
        tg.orthogonalize(g, eps=-1.0)
    assert e.value.status == -14
    with pytest.raises(ctypes.ArgumentError):
        tg.orthogonalize(g, eps="x")
