"""GPU top logits and the distillation loss against the 64-bit reference.

Tolerances.  A fp32 exponential exp((x - m) / T) is off by at most 2^-22
(ex2.approx) plus |x - m| / T log2(e) 2^-23 from its argument (two roundings
of half a step): below 2^-17.5 for the ranges used here (up to 64 in log2),
and a sum of them, with at most 12 levels of partial sums and 2^9 terms in
a thread, by a further 2^-15 at worst; logarithms and probabilities follow
these.  TOL = 2^-14 covers a logarithm (absolute) and a probability
(relative).  A gradient is q - p times the scale: TOL (q + p) and half a step
of its type, torch.finfo(t).eps / 2 relative (for bf16 2^-8 is one half step
in this measure).
"""
import numpy as np
import pytest
import torch

import draft_verification_row_gb300 as sdv
from tests import row_reference as R

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
TOL = 2.0 ** -14


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()


def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _rows(n, V, dtype, seed, std=3.0):
    return (torch.randn((n, V), generator=_gen(seed), device=DEV) * std).to(DT[dtype])


def _check_top(x, k, T, V=None):
    V = x.shape[1] if V is None else V
    values, index, rest, status = sdv.top_logits(x, k, T, V=V)
    torch.cuda.synchronize()
    assert int(status.item()) == 0 and values.dtype == x.dtype
    xx = x[:, :V].double().cpu().numpy()
    values, index, rest = values.double().cpu().numpy(), index.cpu().numpy(), rest.double().cpu().numpy()
    for r in range(x.shape[0]):
        v, i, s = R.top(xx[r], k, T)
        assert np.array_equal(index[r], i), (r, np.flatnonzero(index[r] != i)[:5])
        assert np.array_equal(values[r], v)
        if np.isfinite(s):
            assert abs(rest[r] - s) <= TOL + abs(s) * 2.0 ** -22, (r, rest[r], s)
        else:
            assert rest[r] == s


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V,k", [(1, 1), (2, 1), (7, 7), (7, 9), (8, 3), (33, 32), (1000, 20), (1000, 1000),
                                 (4097, 1024), (20011, 64), (40007, 1), (40007, 1024), (151936, 128),
                                 (262144, 257)])
def test_top_logits(dtype, V, k):
    _check_top(_rows(3, V, dtype, 3 + V), k, 1.0)
    _check_top(_rows(2, V, dtype, 4 + V, std=0.5), k, 0.7)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_top_logits_ties_masks_alignment(dtype):
    V = 5003
    x = torch.randint(0, 4, (3, V), generator=_gen(5), device=DEV).to(DT[dtype])
    for k in (1, 7, 500, 1024):
        _check_top(x, k, 1.0)
    _check_top(torch.zeros((2, V), dtype=DT[dtype], device=DEV), 100, 1.0)
    x = _rows(4, V, dtype, 6)
    x[0, 5:] = float("-inf")
    x[1, :] = float("-inf")
    x[1, 77] = 1.0
    x[2, 10:] = torch.finfo(DT[dtype]).min
    _check_top(x, 16, 1.0)
    x = _rows(3, V + 6, dtype, 7)
    _check_top(x[:, 3:], 50, 2.0, V=V)
    _check_top(torch.sort(x.float(), dim=1).values.to(DT[dtype]), 50, 2.0)  # all of them in one place
    peaked = _rows(2, V, dtype, 8, std=1.0)
    peaked[:, 11] = 30.0  # the others hold 1e-9 of the mass
    _check_top(peaked, 1, 1.0)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V", [4097, 40007, 151936])
def test_top_logits_of_mostly_masked_rows(dtype, V):
    """Few tokens left, spread over the row or side by side, fewer and more than k."""
    for left in (1, 3, 60, 1000, 1500):
        x = _rows(2, V, dtype, 75 + V + left)
        place = torch.rand((2, V), generator=_gen(76), device=DEV).argsort(1)
        place[0] = (torch.arange(V, device=DEV) + V // 3) % V
        x.scatter_(1, place[:, left:], float("-inf"))
        for k in (1, 50, 1024):
            _check_top(x, k, 0.8)


def test_top_logits_unusable_rows():
    x = _rows(4, 3000, "bf16", 9)
    x[1, 5] = float("nan")
    x[2, 5] = float("inf")
    x[3] = float("-inf")
    values, index, rest, status = sdv.top_logits(x, 8, 1.0)
    torch.cuda.synchronize()
    assert int(status.item()) == 4
    assert (index[1:] == -1).all() and values[1:].isnan().all() and rest[1:].isnan().all()
    assert (index[0] >= 0).all() and rest[0].isfinite()


def _record(teacher, k, T):
    return sdv.top_logits(teacher, k, T)[:3]


def _check(student, values, index, rest, T, weight=None, V=None, grad_loss=None):
    """Forward, backward and the one call against the reference; returns the loss."""
    n = student.shape[0]
    V = student.shape[1] if V is None else V
    kw = dict(temperature=T, row_weight=weight, V=V)
    stats = torch.empty((n, 4), device=DEV)
    loss, st1 = sdv.distill_forward(student, values, index, rest, stats=stats, **kw)
    grad = sdv.distill_backward(student, values, index, rest, stats, grad_loss, **kw)
    loss2, grad2, st2 = sdv.distill_loss_grad(student, values, index, rest, **kw)
    torch.cuda.synchronize()
    assert int(st1.item()) == 0 and int(st2.item()) == 0
    s = student[:, :V].detach().double().cpu().numpy()
    v, i = values.double().cpu().numpy(), index.cpu().numpy()
    half = torch.finfo(student.dtype).eps / 2
    for r in range(n):
        w = 1.0 if weight is None else float(weight[r])
        g = 1.0 if grad_loss is None else float(grad_loss[r])
        rr = -np.inf if rest is None else float(rest[r])
        want, dwant = R.distill(s[r], v[r], i[r], rr, T, w)
        for got in (float(loss[r]), float(loss2[r])):
            if np.isfinite(want):
                assert abs(got - want) <= abs(w) * TOL * 2 + abs(want) * 2.0 ** -20, (r, got, want)
            else:
                assert got == want
        z = s[r] / T
        q = np.exp(z - z.max())
        q /= q.sum()
        p = np.zeros(V)
        here = i[r] >= 0
        _, pull = R.distill(s[r], v[r], i[r], rr, T, 1.0)
        p = np.abs(q - pull * T)  # what the teacher asks of each token
        for got, scale in ((grad, g), (grad2, 1.0)):
            x = got[r, :V].double().cpu().numpy()
            tol = abs(scale * w) / T * TOL * (q + p) + half * 1.01 * np.abs(dwant * scale) + 1e-38
            bad = np.abs(x - dwant * scale) > tol
            assert not bad.any(), (r, np.flatnonzero(bad)[:5], x[bad][:5], (dwant * scale)[bad][:5], here.sum())
    return loss


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V,k", [(2, 1), (9, 4), (33, 33), (1000, 20), (4097, 1024), (20011, 64), (151936, 128)])
@pytest.mark.parametrize("T", [1.0, 2.0])
def test_loss_and_gradient(dtype, V, k, T):
    teacher = _rows(3, V, dtype, 11 + V)
    student = (teacher.float() + torch.randn((3, V), generator=_gen(12), device=DEV)).to(DT[dtype])
    values, index, rest = _record(teacher, k, T)
    weight = torch.tensor([0.5, 1.0, 0.0], device=DEV)
    up = torch.tensor([1.0, -2.0, 3.0], device=DEV)
    _check(student, values, index, rest, T, weight, grad_loss=up)
    _check(student, values, index, None, T)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_small_losses_keep_their_digits(dtype):
    """Where the k tokens hold little of either mass, the loss is a small part of its terms: it is off by TOL of what
    the k tokens hold, not of 1."""
    teacher = _rows(6, 9576, dtype, 41)
    student = (teacher.float() + 0.3 * torch.randn((6, 9576), generator=_gen(42), device=DEV)).to(DT[dtype])
    for k in (1, 3):
        values, index, rest = _record(teacher, k, 2.0)
        loss = _check(student, values, index, rest, 2.0)
        for r in range(6):
            want, _ = R.distill(student[r].double().cpu().numpy(), values[r].double().cpu().numpy(),
                                index[r].cpu().numpy(), float(rest[r]), 2.0)
            t = np.append(values[r].double().cpu().numpy() / 2.0, float(rest[r]))
            held = 1.0 - np.exp(t[-1] - t.max()) / np.exp(t - t.max()).sum()
            assert held < 0.1 and abs(float(loss[r]) - want) <= TOL * held, (k, r, float(loss[r]), want)


def test_teacher_of_another_type_and_alignment():
    teacher = _rows(4, 5003, "f32", 13)
    values, index, rest = _record(teacher, 30, 1.0)
    for dtype in DT:
        for off in (0, 1, 3):
            wide = _rows(4, 5003 + 7, dtype, 14)
            _check(wide[:, off:], values, index, rest, 1.0, V=5003)
            _check(wide[:, off:], values.bfloat16(), index, rest, 1.0, V=5003)


def test_absent_entries_and_empty_records():
    teacher, student = _rows(4, 1000, "f32", 15), _rows(4, 1000, "f32", 16)
    values, index, rest = _record(teacher, 8, 1.0)
    index = index.clone()
    index[0, 3:] = -1
    index[1, :] = -1
    values = values.clone()
    values[0, 5] = float("nan")  # an absent entry's value is not used
    v = torch.where(index < 0, torch.zeros_like(values), values)
    _check(student, v, index, rest, 1.0)
    loss = _check(student, v, index, None, 1.0)
    assert float(loss[1]) == 0.0
    got, _ = sdv.distill_forward(student, values, index, rest)
    assert got.isfinite().all()
    empty = torch.empty((4, 0), device=DEV), torch.empty((4, 0), dtype=torch.int32, device=DEV)
    loss = _check(student, *empty, rest, 1.0)  # one outcome: nothing to learn
    assert (loss.abs() <= TOL).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_extreme_rows(dtype):
    """A student sure of the teacher's tokens (the others hold 1e-12), sure of others, with masked tokens."""
    V = 2000
    teacher = _rows(5, V, dtype, 17)
    values, index, rest = _record(teacher, 16, 1.0)
    s = _rows(5, V, dtype, 18, std=1.0)
    s[0].scatter_(0, index[0].long(), 35.0)
    s[1].scatter_(0, index[1].long(), -60.0)
    out = torch.ones(V, dtype=torch.bool, device=DEV)
    out[index[2].long()] = False
    s[2, out.nonzero()[5:, 0]] = float("-inf")
    s[3] *= 0
    _check(s, values, index, rest, 1.0)
    _check(s, values, index, None, 1.0)
    low = s.clone()  # masks of the type's lowest value, around the teacher's tokens and over whole stretches
    low[:, 1000:] = torch.finfo(DT[dtype]).min
    low[1, 30:] = torch.finfo(DT[dtype]).min
    _check(low, values, index, rest, 1.0)
    _check(low, values, index, None, 2.0)
    masked = torch.full_like(teacher, torch.finfo(DT[dtype]).min)  # teachers whose listed logits are masks, too
    masked[:3, 5] = 1.0
    mv, mi, mr = _record(masked, 4, 1.0)
    small = s.float().clamp(min=-50.0).to(DT[dtype])
    _check(small, mv, mi, None, 0.5)
    _check(small, mv, mi, torch.zeros(5, device=DEV), 0.5)
    s[4, int(index[4, 0])] = float("-inf")  # a token the teacher wants and the student rules out
    loss = _check(s, values, index, rest, 1.0)
    assert float(loss[4]) == float("inf")


def test_unusable_rows_and_masked_rows():
    teacher, s = _rows(7, 1000, "f32", 19), _rows(7, 1000, "f32", 20)
    values, index, rest = _record(teacher, 8, 1.0)
    index = index.clone()
    s[0, 3] = float("nan")
    s[1, 3] = float("inf")
    s[2] = float("-inf")
    index[3, 2] = 1000
    index[4, 2] = index[4, 1]
    s[5] = float("nan")
    weight = torch.ones(7, device=DEV)
    weight[5] = 0.0
    stats = torch.empty((7, 4), device=DEV)
    loss, status = sdv.distill_forward(s, values, index, rest, row_weight=weight, stats=stats)
    grad = sdv.distill_backward(s, values, index, rest, stats, row_weight=weight)
    loss2, grad2, status2 = sdv.distill_loss_grad(s, values, index, rest, row_weight=weight)
    torch.cuda.synchronize()
    assert int(status.item()) == 2 | 4 and int(status2.item()) == 2 | 4
    for l, g in ((loss, grad), (loss2, grad2)):
        assert l[:5].isnan().all() and g[:5].isnan().all()
        assert float(l[5]) == 0.0 and (g[5] == 0).all()
        assert l[6].isfinite() and g[6].isfinite().all()
    assert torch.equal(loss[6], loss2[6])


def test_gradient_against_differences():
    """Central differences of the loss itself: h = 1/16 leaves h^2 / 6 times a
    third derivative (below 1 at T = 1, so below 7e-4), and rounding of the
    loss (2^-20) over 2h."""
    V, k, h = 40, 5, 1.0 / 16
    teacher, s = _rows(1, V, "f32", 21, std=1.5), _rows(1, V, "f32", 22, std=1.5)
    values, index, rest = _record(teacher, k, 1.0)
    step = torch.eye(V, device=DEV) * h
    both = torch.cat([s + step, s - step]).contiguous()
    rec = [t.expand(2 * V, *t.shape[1:]).contiguous() for t in (values, index, rest)]
    for r in (rec[2], None):
        loss, _ = sdv.distill_forward(both, rec[0], rec[1], r)
        diff = (loss[:V] - loss[V:]) / (2 * h)
        _, grad, _ = sdv.distill_loss_grad(s, values, index, None if r is None else rest)
        torch.cuda.synchronize()
        assert (diff - grad[0]).abs().max() <= h * h / 6 + 2.0 ** -20 / h


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_autograd(dtype):
    teacher = _rows(6, 3001, dtype, 23)
    student = _rows(6, 3008, dtype, 24).requires_grad_()
    values, index, rest = _record(teacher, 12, 2.0)
    weight = torch.rand(6, generator=_gen(25), device=DEV)
    loss = sdv.distill_loss(student, values, index, rest, temperature=2.0, row_weight=weight, V=3001)
    up = torch.rand(6, generator=_gen(26), device=DEV)
    loss.backward(up, retain_graph=True)
    once = student.grad.clone()
    loss.backward(up)
    torch.cuda.synchronize()
    assert torch.equal(student.grad, once * 2)
    assert (once[:, 3001:] == 0).all()  # columns past V
    _check(student.detach(), values, index, rest, 2.0, weight, V=3001, grad_loss=up)
    # an expanded upstream gradient, and a student that needs none
    student.grad = None
    sdv.distill_loss(student, values, index, rest, temperature=2.0, row_weight=weight, V=3001).sum().backward()
    _, want, _ = sdv.distill_loss_grad(student.detach(), values, index, rest, temperature=2.0, row_weight=weight,
                                       V=3001)
    half = torch.finfo(DT[dtype]).eps / 2
    assert ((student.grad - want).float().abs() <= want.float().abs() * (2 * half + TOL) + 1e-7).all()
    assert not sdv.distill_loss(student.detach(), values, index, rest, V=3001).requires_grad
    with torch.no_grad():
        assert not sdv.distill_loss(student, values, index, rest, V=3001).requires_grad
    loss = sdv.distill_loss(student, values, index, rest, V=3001).sum()
    with pytest.raises(RuntimeError, match="differentiated again"):
        torch.autograd.grad(loss, student, create_graph=True)


def test_in_place_repeat_and_graph():
    teacher, s = _rows(16, 32000, "bf16", 27), _rows(16, 32000, "bf16", 28)
    values, index, rest = _record(teacher, 64, 1.0)
    loss, grad, _ = sdv.distill_loss_grad(s, values, index, rest)
    again, grad2, _ = sdv.distill_loss_grad(s, values, index, rest)
    t = s.clone()
    loss3, grad3, _ = sdv.distill_loss_grad(t, values, index, rest, grad=t)
    torch.cuda.synchronize()
    assert torch.equal(loss, again) and torch.equal(grad, grad2)
    assert torch.equal(loss, loss3) and torch.equal(grad, t) and grad3 is t
    # an autograd step captured into a graph and replayed on other logits
    leaf = s.clone().requires_grad_()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        torch.autograd.grad(sdv.distill_loss(leaf, values, index, rest).sum(), leaf)
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = sdv.distill_loss(leaf, values, index, rest)
        dout, = torch.autograd.grad(out.sum(), leaf)
    other = _rows(16, 32000, "bf16", 29)
    with torch.no_grad():
        leaf.copy_(other)
    g.replay()
    torch.cuda.synchronize()
    want, dwant, _ = sdv.distill_loss_grad(other, values, index, rest)
    assert torch.equal(out, want)
    assert ((dout - dwant).float().abs() <= dwant.float().abs() * (2.0 ** -7 + TOL) + 1e-7).all()


def test_rejects_bad_arguments():
    s = _rows(2, 100, "f32", 31)
    values, index, rest = _record(s, 4, 1.0)
    for T in (0.0, -1.0, float("nan"), float("inf")):
        with pytest.raises(sdv.SDVError):
            sdv.distill_forward(s, values, index, rest, temperature=T)
        with pytest.raises(sdv.SDVError):
            sdv.top_logits(s, 4, T)
    with pytest.raises(sdv.SDVError):
        sdv.top_logits(s, 1025, 1.0)
    with pytest.raises(ValueError):
        sdv.top_logits(s, 0, 1.0)
    with pytest.raises(ValueError):
        sdv.distill_forward(s, values, index.long(), rest)
    with pytest.raises(ValueError):
        sdv.distill_forward(s, values, index[:, :3].contiguous(), rest)
    with pytest.raises(ValueError):
        sdv.distill_forward(s, values, index, rest.double())
    with pytest.raises(ValueError):
        sdv.distill_loss_grad(s, values, index, rest, grad=torch.empty((2, 99), device=DEV))
    with pytest.raises(TypeError):
        sdv.distill_forward(s.double(), values, index, rest)
    assert sdv.distill_forward(s[:0], values[:0], index[:0], rest[:0])[0].shape == (0,)
