"""Truncated sampling, top logits and distillation on the host: bad sizes and
settings are refused before the GPU is touched, host tensors by the binding
(no GPU needed), and the references agree with small cases worked by hand."""
import math

import numpy as np
import pytest
import torch

import draft_verification_row_gb300 as sdv
from tests import row_reference as R


@pytest.fixture(scope="module")
def lib():
    from draft_verification_row_gb300 import build
    build.build()
    return sdv.lib()


BAD_ROWS = [dict(n=-1), dict(V=0), dict(V=262145, stride=262152), dict(stride=15), dict(dtype=2), dict(dtype=-1)]
BAD_SETTINGS = [dict(T=-1.0), dict(T=float("nan")), dict(T=float("inf")), dict(T=1e-39), dict(k=-1), dict(p=0.0),
                dict(p=-0.5), dict(p=1.5), dict(p=float("nan")), dict(m=-0.1), dict(m=1.1), dict(m=float("nan"))]


def _rows(over):
    a = dict(n=2, V=16, stride=16, dtype=0, T=1.0, k=0, p=1.0, m=0.0)
    a.update(over)
    return a


@pytest.mark.parametrize("over", BAD_ROWS + BAD_SETTINGS)
def test_truncation_refusals(lib, over):
    a = _rows(over)
    head = (a["n"], a["V"], a["stride"], a["dtype"], a["T"], a["k"], a["p"], a["m"], None, None, None, None, None)
    assert lib.sdv_sample_truncated(*head, 1, None, None, None, None) == 1
    assert lib.sdv_truncate_rows(*head, None, max(a["V"], 1), None, None) == 1


@pytest.mark.parametrize("draws", [0, -1, 65])
def test_draw_count_refusals(lib, draws):
    assert lib.sdv_sample_truncated(0, 16, 16, 0, 1.0, 0, 1.0, 0.0, None, None, None, None, None, draws, None, None,
                                    None, None) == 1


def test_missing_pointers_are_refused(lib):
    assert lib.sdv_sample_truncated(2, 16, 16, 0, 1.0, 0, 1.0, 0.0, None, None, None, None, None, 1, None, None,
                                    None, None) == 1
    assert lib.sdv_truncate_rows(2, 16, 16, 0, 1.0, 0, 1.0, 0.0, None, None, None, None, None, None, 16, None,
                                 None) == 1
    assert lib.sdv_truncate_rows(0, 16, 16, 0, 1.0, 0, 1.0, 0.0, None, None, None, None, None, None, 15, None,
                                 None) == 1
    assert lib.sdv_top_logits(2, 16, 16, 0, 1.0, None, 4, None, None, None, None, None) == 1


@pytest.mark.parametrize("over", BAD_ROWS + [dict(T=0.0), dict(T=-1.0), dict(T=float("nan")), dict(T=float("inf")),
                                             dict(T=1e-39), dict(k=-1), dict(k=1025)])
def test_top_and_distill_refusals(lib, over):
    a = _rows(dict(k=4))
    a.update(over)
    head = (a["n"], a["V"], a["stride"], a["dtype"], a["T"], None, a["k"])
    assert lib.sdv_top_logits(*head, None, None, None, None, None) == 1
    assert lib.sdv_distill_forward(*head, 0, None, None, None, None, None, None, None, None) == 1
    assert lib.sdv_distill_backward(*head, 0, None, None, None, None, None, None, 1, None, a["V"], None) == 1
    assert lib.sdv_distill_loss_grad(*head, 0, None, None, None, None, None, None, a["V"], None, None) == 1


def test_empty_batches_are_no_ops(lib):
    head = (0, 16, 17, 1, 1.0, 0, 1.0, 0.0, None, None, None, None, None)
    assert lib.sdv_sample_truncated(*head, 1, None, None, None, None) == 0
    assert lib.sdv_truncate_rows(*head, None, 16, None, None) == 0
    assert lib.sdv_top_logits(0, 16, 16, 1, 1.0, None, 4, None, None, None, None, None) == 0
    assert lib.sdv_distill_forward(0, 16, 16, 0, 1.0, None, 4, 0, None, None, None, None, None, None, None, None) == 0
    assert lib.sdv_distill_loss_grad(0, 16, 16, 0, 1.0, None, 4, 0, None, None, None, None, None, None, 16, None,
                                     None) == 0
    assert lib.sdv_distill_forward(0, 16, 16, 0, 1.0, None, 4, 2, None, None, None, None, None, None, None, None) == 1


def test_binding_refuses_host_tensors():
    x = torch.zeros((2, 16))
    with pytest.raises(ValueError, match="CUDA"):
        sdv.sample_truncated(x, 1, torch.zeros((2, 1)), 1.0)
    with pytest.raises(ValueError, match="CUDA"):
        sdv.truncate_rows(x, 1.0)
    with pytest.raises(ValueError, match="CUDA"):
        sdv.top_logits(x, 4)
    with pytest.raises(ValueError, match="CUDA"):
        sdv.distill_loss(x, x[:, :4], torch.zeros((2, 4), dtype=torch.int32))


def test_reference_by_hand():
    x = np.log([0.1, 0.4, 0.2, 0.2, 0.1])
    assert list(R.kept_tokens(x, 1.0)) == [1, 2, 3, 0, 4]
    assert list(R.kept_tokens(x, 1.0, k=2)) == [1, 2]
    assert list(R.kept_tokens(x, 1.0, p=0.7)) == [1, 2, 3]
    assert list(R.kept_tokens(x, 1.0, k=2, p=0.6)) == [1]   # 0.4 of 0.6 is over 0.6
    assert list(R.kept_tokens(x, 1.0, m=0.4)) == [1, 2, 3]
    assert list(R.kept_tokens(x, 0.0)) == [1]
    kept = R.kept_tokens(x, 1.0, k=3)
    assert [R.draw(x, kept, 1.0, u) for u in (0.0, 0.49, 0.51, 0.74, 0.76)] == [1, 1, 2, 2, 3]
    values, index, rest = R.top(x, 2, 1.0)
    assert list(index) == [1, 2] and math.isclose(rest, math.log(0.4))
    # the student is the teacher: no loss, no gradient
    loss, grad = R.distill(x, values, index, rest, 1.0)
    assert abs(loss) < 1e-12 and np.abs(grad).max() < 1e-12
    # renormalised over two tokens: 2/3 and 1/3 against 0.4 and 0.2
    loss, grad = R.distill(x, values, index, -np.inf, 1.0)
    assert math.isclose(loss, math.log(1 / 0.6), rel_tol=1e-12)
    assert np.allclose(grad, [0.1, 0.4 - 2 / 3, 0.2 - 1 / 3, 0.2, 0.1], atol=1e-12)


@pytest.mark.parametrize("T", [1.0, 2.0])
def test_reference_gradient_against_differences(T):
    rng = np.random.default_rng(5)
    t, s, h = rng.normal(size=30) * 2, rng.normal(size=30) * 2, 1e-5
    values, index, rest = R.top(t, 6, T)
    for r in (rest, -np.inf):
        _, grad = R.distill(s, values, index, r, T, 0.5)
        for i in range(30):
            d = np.eye(30)[i] * h
            up, down = (R.distill(s + e, values, index, r, T, 0.5)[0] for e in (d, -d))
            assert abs((up - down) / (2 * h) - grad[i]) < 1e-8
