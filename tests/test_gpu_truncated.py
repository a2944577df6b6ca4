"""GPU truncated sampling and truncated rows against the 64-bit reference.

Kept sets and drawn tokens are whole decisions and have to be equal: the
library's sums are fixed-point integers that agree with 64-bit arithmetic to
about 1e-12 (relative), and with the seeds used here no border or uniform
lies that close to another outcome (a run of 10^4 decisions meets one with a
probability of about 1e-6).
"""
import numpy as np
import pytest
import torch

import draft_verification_row_gb300 as sdv
from draft_verification_row_gb300 import workloads as W
from tests import row_reference as R

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()


def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _rows(n, V, dtype, seed, std=3.0):
    return (torch.randn((n, V), generator=_gen(seed), device=DEV) * std).to(DT[dtype])


def _check(logits, T, k=0, p=1.0, m=0.0, draws=3, V=None, seed=0):
    """Kept sets and draws of every row; settings are numbers or per-row lists."""
    n = logits.shape[0]
    V = logits.shape[1] if V is None else V
    u = torch.rand((n, draws), generator=_gen(seed + 1000), device=DEV)
    u[0, 0] = 0.0
    u[-1, -1] = 1.0 - 2.0 ** -24

    def arg(x, dtype):
        return torch.tensor(x, dtype=dtype, device=DEV) if isinstance(x, list) else x

    args = (arg(T, torch.float32),)
    kw = dict(top_k=arg(k, torch.int32), top_p=arg(p, torch.float32), min_p=arg(m, torch.float32), V=V)
    tokens, st1 = sdv.sample_truncated(logits, draws, u, *args, **kw)
    rows, st2 = sdv.truncate_rows(logits, *args, **kw)
    torch.cuda.synchronize()
    assert int(st1.item()) == 0 and int(st2.item()) == 0
    x = logits[:, :V].double().cpu().numpy()
    got, out, uu = tokens.cpu().numpy(), rows[:, :V].double().cpu().numpy(), u.cpu().numpy()
    for r in range(n):
        s = [v[r] if isinstance(v, list) else v for v in (T, k, p, m)]
        kept = R.kept_tokens(x[r], *s)
        want = np.full(V, -np.inf)
        want[kept] = x[r, kept]
        assert np.array_equal(out[r], want), (r, s, kept.size, int(np.isfinite(out[r]).sum()))
        for d in range(draws):
            assert got[r, d] == R.draw(x[r], kept, s[0], uu[r, d]), (r, d, s)


SETTINGS = [dict(T=0.7, k=50, p=0.9), dict(T=1.0, p=0.95), dict(T=0.8, k=20), dict(T=1.0, m=0.05), dict(T=0.0),
            dict(T=1.2), dict(T=0.7, k=1000, p=0.8, m=0.02), dict(T=0.1, p=0.99)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V", [1, 2, 7, 8, 9, 33, 1000, 4097])
@pytest.mark.parametrize("s", range(len(SETTINGS)))
def test_vocabulary_edges(V, dtype, s):
    _check(_rows(4, V, dtype, 11 + V), **SETTINGS[s], seed=V)


# group, segment and step boundaries of both types, and the longest row
@pytest.mark.parametrize("V,dtype", [(2047, "bf16"), (2048, "bf16"), (2049, "bf16"), (32768, "bf16"),
                                     (32769, "bf16"), (151936, "bf16"), (16385, "f32"), (40007, "f32"),
                                     (262144, "f32"), (262144, "bf16")])
@pytest.mark.parametrize("s", [0, 1, 3, 6])
def test_long_rows(V, dtype, s):
    _check(_rows(3, V, dtype, 5), **SETTINGS[s], seed=6)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_rows_of_any_alignment(dtype):
    """Odd strides and bases that are not on a 16-byte boundary."""
    for off, V, width in ((1, 1001, 1003), (3, 5003, 5007), (0, 999, 1001), (5, 2048, 2061)):
        base = _rows(5, width + off, dtype, 21 + off)
        _check(base[:, off:off + V], 0.8, k=100, p=0.9, seed=off)
        _check(base[:, off:], 1.0, p=0.9, V=V, seed=off)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_wide_kept_sets(dtype):
    """Flat rows, whose nucleus is most of the vocabulary, and large top-k."""
    x = _rows(2, 151936, dtype, 31, std=0.5)
    _check(x, 1.0, p=0.95)
    _check(x, 1.0, k=100000, p=0.9)
    _check(x, 1.0, k=30000)
    _check(x, 1.0, m=0.001)
    _check(_rows(2, 151936, dtype, 32, std=3.0), 1.0, p=0.99)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V,head,tail", [(5003, 0.0, -10.0), (40007, 0.0, -11.0), (5003, -4.0, -5.0),
                                         (40007, -4.0, -5.5), (151936, -8.0, -10.0), (151936, 0.0, -12.0)])
def test_borders_that_fp32_sums_leave_open(dtype, V, head, tail):
    """top_p is the fp32 number just below, at and above the share of the tokens up to a border: p Z and the sum there
    differ by 1e-8 to 1e-7 of Z, less than the error of the fp32 mass of the tail."""
    g = _gen(V)
    x = torch.full((3, V), tail, device=DEV)
    where = torch.randperm(V, generator=g, device=DEV)
    x[:, where[:1]] = 0.0
    x[:, where[1:41]] = head
    x += (torch.rand((3, V), generator=g, device=DEV) < 0.5) * 0.125 * (x == tail)  # two levels of the tail
    x = x.to(DT[dtype])
    for r in range(3):
        w = torch.exp(x[r].double()).sort(descending=True).values
        share = (w.cumsum(0) / w.sum())[[0, 20, 40][r]].item()
        p = np.float32(share)
        for q in (np.nextafter(p, np.float32(0)), p, np.nextafter(p, np.float32(1))):
            _check(x[r:r + 1], 1.0, p=float(q))
            _check(x, 1.0, p=float(q), m=1e-6)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V", [2048, 2049, 8191, 50021, 151936])
def test_flat_rows(dtype, V):
    """Kept sets from a few hundred tokens to most of the row, where lists end and whole-row passes begin."""
    for std, T, p in ((3.0, 1.0, 0.9), (2.0, 1.0, 0.9), (3.0, 1.2, 0.95), (2.0, 0.6, 0.8), (1.0, 1.0, 0.99)):
        x = _rows(2, V, dtype, 33 + V, std=std)
        _check(x, T, p=p, draws=5)
        _check(x, T, p=p, m=0.01, draws=5)
    _check(_rows(2, V, dtype, 34 + V, std=2.0)[:, 3:], 1.0, p=0.9, draws=5)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("n,V", [(2, 2049), (2, 40007), (310, 5003), (2, 151936)])
def test_mostly_masked_rows(dtype, n, V):
    """Rows with few tokens left, fewer than top_k among them, spread over the row or side by side."""
    for left in (1, 3, 60, 1000, 1500):
        x = _rows(n, V, dtype, 71 + V + left)
        place = torch.rand((n, V), generator=_gen(72), device=DEV).argsort(1)
        place[0] = (torch.arange(V, device=DEV) + V // 3) % V
        x.scatter_(1, place[:, left:], float("-inf"))
        for kw in ({"k": 50}, {"k": 1200, "p": 0.9}, {"p": 0.95}, {"k": 2000, "m": 1e-4}, {"m": 1e-30}):
            _check(x, 0.8, draws=3, **kw)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V", [1000, 40007])
def test_ties(dtype, V):
    """Few distinct values: borders inside ties go by index."""
    x = torch.randint(0, 4, (4, V), generator=_gen(41), device=DEV).to(DT[dtype])
    for k in (1, 7, V // 5, V // 2, V - 1, V, V + 5):
        _check(x, 1.0, k=k, draws=2)
    for p in (0.25, 0.5, 0.9):
        _check(x, 1.0, p=p, draws=2)
        _check(x, 1.0, k=V // 3, p=p, draws=2)
    _check(x, 1.0, m=float(np.exp(np.float32(-1.5))), draws=2)
    _check(torch.zeros((2, V), dtype=DT[dtype], device=DEV), 0.7, p=0.5)  # the sums are exact: half of the row
    _check(torch.zeros((2, V), dtype=DT[dtype], device=DEV), 0.7, k=3)
    z = torch.zeros((2, V), dtype=DT[dtype], device=DEV)  # -0 and +0 are one value
    z[:, ::2] = -0.0
    _check(z, 0.7, k=11)
    _check(z, 0.0)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_masked_rows(dtype):
    """-inf and the type's lowest value in masked places, down to one token."""
    V = 5003
    x = _rows(6, V, dtype, 51)
    low = torch.finfo(DT[dtype]).min
    x[0, torch.randperm(V, generator=_gen(52), device=DEV)[:V - 3]] = float("-inf")
    x[1, :] = float("-inf")
    x[1, 4711] = -2.0
    x[2, torch.randperm(V, generator=_gen(53), device=DEV)[:V - 10]] = low
    x[3, :] = low
    x[4, 100:] = float("-inf")
    x[5, 0] = 3e38
    for s in SETTINGS:
        _check(x, **s)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_settings_by_row(dtype):
    n = 12
    _check(_rows(n, 32000, dtype, 61), [0.0, 0.6, 0.7, 1.0] * 3, k=[0, 20, 50, 1000, 1, 0] * 2,
           p=[1.0, 0.9, 0.5] * 4, m=[0.0, 0.05] * 6)


def test_unusable_rows_are_isolated():
    x = _rows(7, 5000, "f32", 71)
    x[1, 17] = float("nan")
    x[2, 4000] = float("inf")
    x[3, :] = float("-inf")
    T = torch.tensor([0.7, 0.7, 0.7, 0.7, -1.0, float("nan"), 0.7], device=DEV)
    u = torch.rand((7, 2), generator=_gen(72), device=DEV)
    tokens, status = sdv.sample_truncated(x, 2, u, T, top_k=5)
    rows, status2 = sdv.truncate_rows(x, T, top_k=5)
    torch.cuda.synchronize()
    t = tokens.cpu().numpy()
    assert (t[1:6] == -1).all() and (t[[0, 6]] >= 0).all()
    assert int(status.item()) == 4 | 16 and int(status2.item()) == 4 | 16
    assert torch.equal(rows[1:6].view(torch.int32), x[1:6].view(torch.int32))  # as they were
    assert (rows[[0, 6]].isfinite().sum(dim=1) == 5).all()
    for kw, bad in ((dict(top_k=torch.tensor([-1, 3], dtype=torch.int32, device=DEV)), 0),
                    (dict(top_p=torch.tensor([0.0, 0.5], device=DEV)), 0),
                    (dict(top_p=torch.tensor([1.5, 0.5], device=DEV)), 0),
                    (dict(min_p=torch.tensor([0.1, float("nan")], device=DEV)), 1)):
        tokens, status = sdv.sample_truncated(x[[0, 6]].contiguous(), 1, u[:2, :1].contiguous(), 0.7, **kw)
        torch.cuda.synchronize()
        assert int(status.item()) == 16 and int(tokens[bad]) == -1 and int(tokens[1 - bad]) >= 0


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_in_place_and_padding(dtype):
    V, width = 3001, 3016
    x = _rows(5, width, dtype, 81)
    x[:, V:] = float("nan")  # padding is neither read nor written
    want, _ = sdv.truncate_rows(x, 0.7, top_p=0.9, V=V)
    y = x.clone()
    got, _ = sdv.truncate_rows(y, 0.7, top_p=0.9, V=V, out=y)
    torch.cuda.synchronize()
    assert got is y and torch.equal(y[:, :V], want) and y[:, V:].isnan().all()
    odd = torch.full((5, width + 1), 7.0, dtype=DT[dtype], device=DEV)  # rows aligned otherwise than the logits'
    sdv.truncate_rows(x, 0.7, top_p=0.9, V=V, out=odd[:, 1:])
    torch.cuda.synchronize()
    assert torch.equal(odd[:, 1:V + 1], want) and (odd[:, V + 1:] == 7.0).all() and (odd[:, 0] == 7.0).all()


def test_offsets_past_32_bits():
    stride, V = 1 << 30, 1000
    base = torch.empty(4 * stride, dtype=torch.bfloat16, device=DEV).view(4, stride)
    base[:, :V] = _rows(4, V, "bf16", 91)
    _check(base[:, :V], 0.7, k=50, p=0.9)


def test_repeated_streams_and_graph():
    """The same call on other streams, and replayed from a graph, gives the same tokens."""
    x = _rows(64, 32000, "bf16", 101)
    u = torch.rand((64, 4), generator=_gen(102), device=DEV)
    want, _ = sdv.sample_truncated(x, 4, u, 0.7, top_p=0.9)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    got = [sdv.sample_truncated(x, 4, u, 0.7, top_p=0.9, stream=s)[0] for s in streams]
    torch.cuda.synchronize()
    assert all(torch.equal(g, want) for g in got)
    out = torch.empty_like(want)
    rows = torch.empty_like(x)
    status = torch.empty(1, dtype=torch.int32, device=DEV)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        sdv.sample_truncated(x, 4, u, 0.7, top_p=0.9, tokens=out, device_status=status)
        sdv.truncate_rows(x, 0.7, top_p=0.9, out=rows, device_status=status)
    y = _rows(64, 32000, "bf16", 103)
    x.copy_(y)
    g.replay()
    torch.cuda.synchronize()
    want, _ = sdv.sample_truncated(y, 4, u, 0.7, top_p=0.9)
    assert torch.equal(out, want) and torch.equal(rows, sdv.truncate_rows(y, 0.7, top_p=0.9)[0])


def test_verification_reads_truncated_rows():
    """Drafts drawn from truncated rows, verified on truncated rows: every
    emitted token lies in the target's kept set, and a draft equal to the
    target is accepted whole."""
    b = W.make("multidraft-B32-K4-L4-V32000-f32", DEV)
    shape = b.target.shape
    kw = dict(top_k=40, top_p=0.9, V=b.V)
    target = sdv.truncate_rows(b.target.view(-1, shape[3]), b.temperature, **kw)[0]
    draft_rows = b.target[:, :, :b.L].reshape(-1, shape[3])  # a draft model that is the target
    draft, _ = sdv.truncate_rows(draft_rows, b.temperature, **kw)
    # one shared prefix: all drafts take request 0's draft-0 rows' order of tokens
    u = torch.rand((draft_rows.shape[0], 1), generator=_gen(111), device=DEV)
    tokens = sdv.sample_truncated(draft_rows, 1, u, b.temperature, **kw)[0].view(b.B, b.K, b.L)
    k1 = slice(0, 1)
    out = sdv.verify("token", target.view(*shape[:3], -1)[:, k1].contiguous(),
                     draft.view(b.B, b.K, b.L, -1)[:, k1].contiguous(), tokens[:, k1].contiguous(), None,
                     b.accept_u[:, k1].contiguous(), b.sample_u[:, k1].contiguous(), b.temperature, V=b.V)
    torch.cuda.synchronize()
    assert int(out["device_status"].item()) == 0
    assert (out["accept_len"] == b.L).all()
    last = target.view(*shape[:3], -1)[:, 0, b.L]
    assert last.gather(1, out["out_token"].long()[:, None]).isfinite().all()


def test_rejects_bad_arguments():
    x = _rows(2, 100, "f32", 121)
    u = torch.rand((2, 2), device=DEV)
    for kw in (dict(top_k=-1), dict(top_p=0.0), dict(top_p=1.01), dict(min_p=-0.1), dict(min_p=1.5),
               dict(top_p=float("nan"))):
        with pytest.raises(sdv.SDVError):
            sdv.sample_truncated(x, 2, u, 1.0, **kw)
        with pytest.raises(sdv.SDVError):
            sdv.truncate_rows(x, 1.0, **kw)
    for T in (-0.5, float("nan"), float("inf"), 1e-39):
        with pytest.raises(sdv.SDVError):
            sdv.sample_truncated(x, 2, u, T)
    with pytest.raises(sdv.SDVError):
        sdv.sample_truncated(x, 2, None, 1.0)  # uniforms are needed for T > 0
    with pytest.raises(sdv.SDVError):
        sdv.sample_truncated(x, 65, torch.rand((2, 65), device=DEV), 1.0)
    with pytest.raises(TypeError):
        sdv.truncate_rows(x.half(), 1.0)
    with pytest.raises(ValueError):
        sdv.sample_truncated(x, 2, u, torch.ones(3, device=DEV))
    with pytest.raises(ValueError):
        sdv.truncate_rows(x, 1.0, out=torch.empty((2, 99), device=DEV))
    assert sdv.sample_truncated(x[:0], 2, u[:0], 1.0)[0].shape == (0, 2)
