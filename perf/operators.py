"""The operators around verification, as they are timed: truncated sampling, truncated rows, a teacher's top logits and
the distillation loss with its gradient.

Each case names its operator in "op".  With ``own`` false, run() computes it from elementary torch operations; with
``own`` true, it makes the calls of this repository's package.  Logits are the synthetic rows of the repository's
workloads: normal noise, a Zipf(1.1) bias by a random rank and, in some cases, a few spikes, as a language model's rows
have a few likely tokens and a long tail.
"""
import math

import torch

own = False

DEV = "cuda:0"
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
ELEM = {"bf16": 2, "f32": 4}


def listed():
    return [
        # one decoding step of four requests: one draw each, the usual server settings; latency counts
        dict(name="sample-B4-V32000", op="sample", n=4, V=32000, dtype="bf16", draws=1, T=0.7, k=50, p=0.9, m=0.0,
             mixed=False, std=3.0, zipf=True, spikes=20),
        # min-p alone on fp32 rows, several drafts drawn from one row
        dict(name="sample-minp-64-V128256-f32", op="sample", n=64, V=128256, dtype="f32", draws=4, T=1.0, k=0, p=1.0,
             m=0.05, mixed=False, std=2.0, zipf=True, spikes=0),
        # a batch of requests that each bring their own settings, eight drafts a row
        dict(name="sample-mixed-256-V151936", op="sample", n=256, V=151936, dtype="bf16", draws=8, T=0.7, k=0, p=1.0,
             m=0.0, mixed=True, std=3.0, zipf=True, spikes=20),
        # every draft row of one depth of the largest batch, top-p alone
        dict(name="sample-topp-2048-V151936", op="sample", n=2048, V=151936, dtype="bf16", draws=1, T=0.7, k=0, p=0.9,
             m=0.0, mixed=False, std=3.0, zipf=True, spikes=0),
        # the target rows of 32 requests with 4 drafts of 4 tokens, fp32, top-p with min-p
        dict(name="truncate-640-V32000-f32", op="truncate", n=640, V=32000, dtype="f32", T=0.7, k=0, p=0.95, m=0.02,
             mixed=False, std=2.0, zipf=False, spikes=20),
        # target rows of the largest vocabulary under top-k and top-p
        dict(name="truncate-2048-V151936", op="truncate", n=2048, V=151936, dtype="bf16", T=0.7, k=200, p=0.9, m=0.0,
             mixed=False, std=3.0, zipf=True, spikes=0),
        # a short teacher record of a few fp32 rows of odd length
        dict(name="top-64-V40007-f32", op="top", n=64, V=40007, dtype="f32", k=20, T=2.0, std=3.0, zipf=True, spikes=0),
        # the teacher's records of a training batch
        dict(name="top-2048-V151936", op="top", n=2048, V=151936, dtype="bf16", k=128, T=1.0, std=3.0, zipf=True,
             spikes=0),
        # the loss alone, as an evaluation takes it
        dict(name="distill-eval-512-V128256", op="distill", call="forward", n=512, V=128256, dtype="bf16", k=64, T=1.0,
             rest=True, std=3.0, zipf=True, spikes=0),
        # a training step through autograd: loss, then the gradient with respect to the draft's logits
        dict(name="distill-train-4096-V32000", op="distill", call="autograd", n=4096, V=32000, dtype="bf16", k=64,
             T=1.0, rest=True, std=3.0, zipf=True, spikes=20),
        # loss and gradient in one call: fp32, odd rows, a teacher renormalised over its top logits, a high temperature
        dict(name="distill-step-1000-V20011-f32", op="distill", call="both", n=1000, V=20011, dtype="f32", k=32, T=2.0,
             rest=False, std=2.0, zipf=False, spikes=0),
        # the same for a long batch of the largest vocabulary
        dict(name="distill-step-8192-V151936", op="distill", call="both", n=8192, V=151936, dtype="bf16", k=128, T=1.0,
             rest=True, std=3.0, zipf=True, spikes=0),
    ]


def draw(rng):
    def log_int(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["sample", "sample", "truncate", "top", "distill", "distill"])
    V = log_int(500, 151936)
    dtype = rng.choice(["bf16", "bf16", "f32"])
    most = (2048 if op != "distill" else 8192) * 151936 * 2 // (V * ELEM[dtype])
    n = log_int(1, max(1, min(most, 2048 if op != "distill" else 8192)))
    case = dict(op=op, n=n, V=V, dtype=dtype, std=rng.choice([2.0, 3.0]), zipf=rng.random() < 0.6,
                spikes=rng.choice([0, 0, 20]))
    if op in ("sample", "truncate"):
        case.update(T=rng.choice([0.5, 0.7, 0.8, 1.0, 1.2]), k=rng.choice([0, 0, 1, 20, 50, 200, 1000]),
                    p=rng.choice([1.0, 0.8, 0.9, 0.95]), m=rng.choice([0.0, 0.0, 0.02, 0.1]), mixed=rng.random() < 0.3)
        if case["k"] == 0 and case["p"] == 1.0 and case["m"] == 0.0:
            case["p"] = 0.9
        if op == "sample":
            case["draws"] = rng.choice([1, 1, 2, 5, 8])
    elif op == "top":
        case.update(k=min(V, log_int(1, 256)), T=rng.choice([0.7, 1.0, 2.0]))
    else:
        case.update(k=min(V // 2, log_int(1, 256)), T=rng.choice([0.7, 1.0, 2.0]), rest=rng.random() < 0.6,
                    call=rng.choice(["forward", "autograd", "both", "both"]))
    return case


def _rows(g, n, case):
    """n rows of logits in fp32."""
    V = case["V"]
    x = torch.randn((n, V), generator=g, device=DEV) * case["std"]
    if case["zipf"]:
        x -= 1.1 * torch.log1p(torch.rand((n, V), generator=g, device=DEV) * (V - 1))
    if case["spikes"]:
        at = torch.randint(0, V, (n, case["spikes"]), generator=g, device=DEV)
        x.scatter_add_(1, at, torch.full(at.shape, 8.0, device=DEV))
    return x


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    n, V, dt = case["n"], case["V"], DTYPES[case["dtype"]]
    state = dict(case)
    if case["op"] != "distill":
        state["logits"] = _rows(g, n, case).to(dt)
    if case["op"] in ("sample", "truncate"):
        if case["mixed"]:  # each row is one of a few kinds of request

            def pick(values, dtype):
                which = torch.randint(0, len(values), (n,), generator=g, device=DEV)
                return torch.tensor(values, dtype=dtype, device=DEV)[which]

            state["T"] = pick([0.0, 0.6, 0.7, 1.0], torch.float32)
            state["k"] = pick([20, 50, 200, 1000], torch.int32)
            state["p"] = pick([0.8, 0.9, 0.95, 1.0], torch.float32)
            state["m"] = pick([0.0, 0.0, 0.02, 0.05], torch.float32)
        if case["op"] == "sample":
            state["u"] = torch.rand((n, case["draws"]), generator=g, device=DEV)
    if case["op"] == "distill":
        k = case["k"]
        student = torch.empty((n, V), dtype=dt, device=DEV)
        values = torch.empty((n, k), dtype=dt, device=DEV)
        index = torch.empty((n, k), dtype=torch.int32, device=DEV)
        rest = torch.empty(n, dtype=torch.float32, device=DEV)
        step = max(1, (1 << 28) // V)
        for r in range(0, n, step):  # the teacher's whole rows are not kept
            t = _rows(g, min(step, n - r), case)
            student[r:r + step] = (t + torch.randn(t.shape, generator=g, device=DEV)).to(dt)
            t = t.to(dt).float()
            v, i = torch.topk(t, k, dim=1)
            values[r:r + step], index[r:r + step] = v.to(dt), i.int()
            t.scatter_(1, i, -math.inf)
            rest[r:r + step] = torch.logsumexp(t / case["T"], dim=1)
        state.update(student=student.requires_grad_(case["call"] == "autograd"), values=values, index=index,
                     rest=rest if case["rest"] else None)
        # a tenth of the positions are masked; the others share the mean
        used = (torch.rand(n, generator=g, device=DEV) >= 0.1).float()
        state["weight"] = used / n
    return state


def _column(v, n, dtype):
    return torch.full((n, 1), v, dtype=dtype, device=DEV) if not torch.is_tensor(v) else v.to(dtype).view(n, 1)


def _kept(state, x):
    """The kept set as a mask, and the weights exp((x - max) / T), in 64 bits: a token next to the border of the set must
    not change sides."""
    n, V = x.shape
    x = x.float()
    # the settings as the fp32 numbers that the calls take
    T = _column(state["T"], n, torch.float32).double()
    p = _column(state["p"], n, torch.float32).double()
    m = _column(state["m"], n, torch.float32).double()
    k = _column(state["k"], n, torch.int64)
    s, order = torch.sort(x, dim=1, descending=True, stable=True)
    greedy = T == 0
    z = (s.double() - s[:, :1].double()) / torch.where(greedy, torch.ones_like(T), T)
    w = torch.exp(z)
    n_k = torch.where(k > 0, k.clamp(max=V), torch.full_like(k, V))
    place = torch.arange(V, device=DEV)
    cum = torch.cumsum(torch.where(place < n_k, w, torch.zeros_like(w)), dim=1)
    n_p = torch.where(p < 1, (cum < p * cum[:, -1:]).sum(dim=1, keepdim=True) + 1, n_k)
    n_m = torch.where(m > 0, (z >= torch.log(m)).sum(dim=1, keepdim=True), torch.full_like(k, V))
    count = torch.minimum(torch.minimum(n_k, n_p), n_m).clamp(min=1)
    count = torch.where(greedy, torch.ones_like(count), count)
    mask = torch.zeros((n, V), dtype=torch.bool, device=DEV).scatter_(1, order, place < count)
    del order, cum, s, z
    return mask, torch.exp((x.double() - x.amax(dim=1, keepdim=True).double()) / torch.where(greedy, torch.ones_like(T), T))


def _plain_distill(state):
    T, k = state["T"], state["k"]
    s = state["student"].detach().float() / T
    index = state["index"].long()
    t = state["values"].float() / T
    rest = state["rest"]
    t = torch.cat([t, torch.full_like(t[:, :1], -math.inf) if rest is None else rest[:, None]], dim=1)
    t = t - t.amax(dim=1, keepdim=True)
    lp = t - torch.log(torch.exp(t).sum(dim=1, keepdim=True))
    p = torch.exp(lp)
    s = s - s.amax(dim=1, keepdim=True)
    q = torch.exp(s)
    top = torch.gather(q, 1, index)
    others = q.scatter(1, index, torch.zeros_like(top)).sum(dim=1, keepdim=True)
    total = others + top.sum(dim=1, keepdim=True)
    lq = torch.cat([torch.gather(s, 1, index) - torch.log(total), torch.log(others) - torch.log(total)], dim=1)
    loss = torch.where(p > 0, p * (lp - lq), torch.zeros_like(p)).sum(dim=1) * state["weight"]
    if state["call"] == "forward":
        return loss
    scale = state["weight"][:, None] / T
    grad = q * (scale * (1 - p[:, k:] * total / others) / total)
    grad.scatter_(1, index, scale * (top / total - p[:, :k]))
    return loss, grad.to(state["student"].dtype)


def _plain(state):
    op = state["op"]
    if op == "distill":
        return _plain_distill(state)
    x = state["logits"]
    if op == "top":
        k = state["k"]
        s, order = torch.sort(x.float(), dim=1, descending=True, stable=True)
        s = s / state["T"]
        others = torch.exp(s[:, k:] - s[:, :1]).sum(dim=1)
        index = order[:, :k]
        return torch.gather(x, 1, index), index.int(), torch.log(others) + s[:, 0]
    mask, w = _kept(state, x)
    if op == "truncate":
        return torch.where(mask, x, torch.full_like(x, -math.inf))
    w = torch.where(mask, w, torch.zeros_like(w)).cumsum(dim=1)
    return torch.searchsorted(w, state["u"].double() * w[:, -1:], right=True).int()


def run(state):
    if not own:
        return _plain(state)
    import draft_verification_row_gb300 as sdv

    op = state["op"]
    if op == "sample":
        return sdv.sample_truncated(state["logits"], state["draws"], state["u"], state["T"], top_k=state["k"],
                                    top_p=state["p"], min_p=state["m"])[0]
    if op == "truncate":
        return sdv.truncate_rows(state["logits"], state["T"], top_k=state["k"], top_p=state["p"], min_p=state["m"])[0]
    if op == "top":
        return sdv.top_logits(state["logits"], state["k"], state["T"])[:3]
    student, teacher = state["student"], (state["values"], state["index"], state["rest"])
    if state["call"] == "both":
        return sdv.distill_loss_grad(student, *teacher, temperature=state["T"], row_weight=state["weight"])[:2]
    loss = sdv.distill_loss(student, *teacher, temperature=state["T"], row_weight=state["weight"])
    if state["call"] == "forward":
        return loss
    return loss.detach(), torch.autograd.grad(loss.sum(), student)[0]


def work(case):
    """Each logit read once, each output written once; about four operations a logit for its exponential and sums."""
    n, V, e = case["n"], case["V"], ELEM[case["dtype"]]
    rows = n * V * e
    if case["op"] == "sample":
        return {"bytes": rows + n * case["draws"] * 8, "flops": 4 * n * V}
    if case["op"] == "truncate":
        return {"bytes": 2 * rows, "flops": 4 * n * V}
    if case["op"] == "top":
        return {"bytes": rows + n * case["k"] * (e + 4) + 4 * n, "flops": 4 * n * V}
    record = n * (case["k"] * (e + 4) + 12)
    if case["call"] == "forward":
        return {"bytes": rows + record, "flops": 4 * n * V}
    return {"bytes": 2 * rows + record, "flops": 8 * n * V}


def exact(case, seed):
    """The computed numbers of top and distill in 64 bits, some rows at a time, from the definitions: a teacher's
    distribution over its k tokens and one outcome for all others, and the derivative of the cross entropy.  The other
    operators return tokens and copies of logits, which have no such values."""
    if case["op"] in ("sample", "truncate"):
        return None
    state = prepare(case, seed)
    n, V, k, T = case["n"], case["V"], case["k"], float(case["T"])
    step = max(1, (1 << 27) // V)
    if case["op"] == "top":
        rest = []
        for r in range(0, n, step):
            x = state["logits"][r:r + step].double() / T
            x = torch.sort(x, dim=1).values[:, :V - k]
            rest.append(torch.logsumexp(x, dim=1))
        return None, None, torch.cat(rest)
    losses, grads = [], []
    for r in range(0, n, step):
        s = state["student"][r:r + step].detach().double()
        lq = torch.log_softmax(s / T, dim=1)
        i = state["index"][r:r + step].long()
        outcome = state["values"][r:r + step].double() / T
        if state["rest"] is not None:
            outcome = torch.cat([outcome, state["rest"][r:r + step, None].double()], dim=1)
        p = torch.softmax(outcome, dim=1)
        weight = state["weight"][r:r + step].double()
        inside = torch.zeros_like(s, dtype=torch.bool).scatter_(1, i, True)
        # log of the mass of all other tokens, from those tokens
        lr = torch.logsumexp(torch.where(inside, torch.full_like(lq, -math.inf), lq), dim=1, keepdim=True)
        lq_outcome = torch.cat([lq.gather(1, i), lr], dim=1)[:, :p.shape[1]]
        losses.append(weight * (p * (torch.log(p) - lq_outcome)).nan_to_num(nan=0.0, posinf=math.inf).sum(dim=1))
        if case["call"] != "forward":
            # softmax minus the target distribution; the others' part of it is spread like the student's own tail
            want = torch.zeros_like(s).scatter_(1, i, p[:, :k])
            if state["rest"] is not None:
                want += torch.where(inside, torch.zeros_like(lq), torch.exp(lq - lr)) * p[:, k:]
            grads.append((weight[:, None] * (torch.exp(lq) - want) / T).float())
    loss = torch.cat(losses)
    if case["call"] == "forward":
        return loss
    return loss, torch.cat(grads)
