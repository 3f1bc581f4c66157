"""The operators of include/trsm_model.h: the header's symbols are exported,
argument checking and quick returns work without a GPU (no call here reaches
a kernel launch), and the tensor functions refuse what they cannot take."""
import os
import re

import pytest

import triangular_solve_gb300 as tg
from triangular_solve_gb300 import model

HEADER = os.path.join(os.path.dirname(tg.HEADER), "trsm_model.h")
FAKE = 1 << 20  # an aligned address that is never dereferenced


@pytest.fixture(scope="module")
def lib():
    from triangular_solve_gb300 import build
    build.build()
    return model._library()


def test_every_declared_symbol_is_exported_and_bound(lib):
    text = open(HEADER).read()
    names = set(re.findall(r"^\w+\s*\*?\s*(trsm_\w+)\s*\(", text, re.M))
    assert {"trsm_linrec_forward", "trsm_linrec_backward", "trsm_linrec_step"} <= names
    for name in names:
        assert hasattr(lib, name) and hasattr(tg, name) and name in tg.__all__, name
    assert "torch" not in text.lower() and 'extern "C"' in text


# name: (position, bad value) pairs against a valid call
FORWARD = [1, 2, 2, 5, 6, FAKE, 30, 6, FAKE, 30, 6, FAKE, 6, None, FAKE, 30, 6, FAKE, None]
BACKWARD = [1, 2, 2, 5, 6, FAKE, 30, 6, FAKE, 30, 6, FAKE, 30, 6, FAKE, 6, FAKE, 30, 6, FAKE, None, FAKE, 30, 6, FAKE,
            30, 6, FAKE, None]
STEP = [1, 2, 2, 6, FAKE, 6, FAKE, 6, FAKE, 9, FAKE, 6, FAKE, 6, FAKE, 6, None]


@pytest.mark.parametrize("pos,bad", [
    (1, 3), (1, -1), (2, 3), (2, -1), (3, -1), (4, -1), (4, 1 << 31), (5, -1), (6, None), (6, FAKE + 1), (9, None),
    (9, FAKE + 1), (12, FAKE + 2), (14, FAKE + 2), (15, None), (15, FAKE + 1), (16, 5), (17, 5), (17, -5),
    (18, FAKE + 2)])
def test_forward_argument_errors_report_position(lib, pos, bad):
    args = list(FORWARD)
    args[pos - 1] = bad
    assert lib.trsm_linrec_forward(*args) == -pos


@pytest.mark.parametrize("pos,bad", [
    (1, 3), (2, 7), (3, -1), (4, -1), (4, 1 << 31), (5, -1), (6, None), (9, None), (9, FAKE + 1), (12, None),
    (12, FAKE + 1), (15, FAKE + 2), (17, None), (20, FAKE + 2), (21, FAKE + 2), (22, None), (22, FAKE + 1), (23, 5),
    (24, 5), (25, None), (25, FAKE + 1), (26, 5), (27, -5), (28, FAKE + 2)])
def test_backward_argument_errors_report_position(lib, pos, bad):
    args = list(BACKWARD)
    args[pos - 1] = bad
    assert lib.trsm_linrec_backward(*args) == -pos


@pytest.mark.parametrize("pos,bad", [
    (1, 3), (2, 7), (3, -1), (4, -1), (5, None), (5, FAKE + 1), (7, None), (9, FAKE + 2), (10, -1), (11, None),
    (11, FAKE + 2), (12, 5), (13, None), (14, 5), (15, None), (16, 5)])
def test_step_argument_errors_report_position(lib, pos, bad):
    args = list(STEP)
    args[pos - 1] = bad
    assert lib.trsm_linrec_step(*args) == -pos


def test_quick_returns_touch_nothing(lib):
    for pos in (3, 5):  # no sequences, no channels
        args = list(FORWARD)
        args[pos - 1] = 0
        args[5] = args[8] = args[14] = None
        assert lib.trsm_linrec_forward(*args) == 0
    args = list(FORWARD)  # no tokens and no one asks for the last states
    args[3], args[5], args[8], args[14], args[17] = 0, None, None, None, None
    assert lib.trsm_linrec_forward(*args) == 0
    args = list(BACKWARD)
    args[2] = 0
    args[5] = args[11] = args[16] = args[21] = args[24] = None
    assert lib.trsm_linrec_backward(*args) == 0
    args = list(STEP)
    args[3] = 0
    assert lib.trsm_linrec_step(*args) == 0


def test_cpu_tensors_are_refused():
    torch = pytest.importorskip("torch")
    g = torch.zeros(2, 3, 4)
    with pytest.raises(ValueError, match="CPU tensor"):
        tg.linear_recurrence(g, g)
    with pytest.raises(ValueError, match="CPU tensor"):
        tg.linear_recurrence_backward(g, g, g, g)
    with pytest.raises(ValueError, match="CPU tensor"):
        tg.linear_recurrence_step(g[0], g[0], g[0])
    with pytest.raises(ValueError, match="CPU tensor"):
        tg.linear_recurrence(g.requires_grad_(), g)


ORTH = [2, 2, 4, 6, FAKE, 6, 24, FAKE, 6, 24, 2, 5, None, 1e-7, FAKE, 1 << 30, None]


@pytest.mark.parametrize("pos,bad", [
    (1, 3), (2, 0), (2, 3), (3, -1), (3, 65537), (4, -1), (4, 65537), (5, None), (5, FAKE + 1), (6, 5), (7, -1),
    (8, None), (8, FAKE + 1), (9, 5), (10, 23), (11, -1), (11, 65536), (12, -1), (12, 65), (14, -1.0),
    (14, float("nan"))])
def test_orthogonalize_argument_errors_report_position(lib, pos, bad):
    args = list(ORTH)
    args[pos - 1] = bad
    assert lib.trsm_orthogonalize(*args) == -pos


def test_orthogonalize_workspace(lib):
    args = list(ORTH)
    args[2:4], args[5], args[6], args[8], args[9] = (300, 200), 200, 60000, 200, 60000
    args[15] = tg.trsm_orthogonalize_workspace_bytes("bf16", 300, 200, 2) - 1
    assert args[15] > 4 * 2 * 300 * 200 * 2  # X twice, head and tail
    assert lib.trsm_orthogonalize(*args) == tg.ERR_WORKSPACE
    args[14], args[15] = FAKE + 8, 1 << 30
    assert lib.trsm_orthogonalize(*args) == tg.ERR_WORKSPACE
    size = tg.trsm_orthogonalize_workspace_bytes
    assert size("f32", 0, 300, 2) == 0 and size("f32", 64, 64, 1024) == 0  # nothing to do, on chip
    assert size("f32", 300, 200, 2) == size("f32", 200, 300, 2)
    for bad in (dict(m=-1), dict(n=65537), dict(batch=-1), dict(steps=65)):
        with pytest.raises(ValueError):
            tg.trsm_orthogonalize_workspace_bytes(**(dict(in_dtype="f32", m=4, n=6, batch=1) | bad))
    for pos in (3, 4, 11):  # nothing to do
        args = list(ORTH)
        args[pos - 1], args[4], args[7] = 0, None, None
        assert lib.trsm_orthogonalize(*args) == 0


def test_coefficients():
    assert list(model._coefficients(2, (1, 2, 3))) == [1, 2, 3, 1, 2, 3]
    assert list(model._coefficients(2, [(1, 2, 3), (4, 5, 6)])) == [1, 2, 3, 4, 5, 6]
    assert model._coefficients(5, None) is None and list(model._coefficients(0, None) or []) == []
    for bad in ((1, 2), [(1, 2, 3), (4, 5)]):
        with pytest.raises(ValueError):
            model._coefficients(2, bad)
