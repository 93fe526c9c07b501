"""What the operators around a binarized projection are measured on.

Two groups of operators that a binarized language model needs next to its
packed projections:

- low-rank adapters of many requests beside one shared projection: the
  forward (serving: a few tokens of many adapters; training: long runs of few)
  and its backward;
- distillation from a float teacher's stored top logits, the loss such
  adapters are trained with: forward, backward, and both in one pass over the
  logits.

Every case is a dict; ``op`` names the operator. ``run`` computes it either in
its plain form (elementary torch operations in 32 bits, rounded once) or, with
``own`` set, through the library's entry points. ``exact`` is the definition
in 64 bits.
"""
import math

import torch

own = False

DEV = "cuda"
_DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
_SIZE = {"bf16": 2, "f16": 2, "f32": 4}


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # one request generating one token: nothing but latency
        {"name": "adapter_token", "op": "adapter", "T": 1, "K": 4096, "N": 4096, "R": 16, "L": 8, "mix": "decode",
         "none": 0.0, "dtype": "bf16", "out": "bf16", "want_u": False},
        # a decode step of 64 requests over 48 adapters, some requests without one, the wide MLP projection
        {"name": "adapter_decode64", "op": "adapter", "T": 64, "K": 4096, "N": 11008, "R": 32, "L": 48, "mix": "decode",
         "none": 0.125, "dtype": "bf16", "out": "bf16", "want_u": False},
        # prompts of several requests beside decoding ones in one batch, ragged sizes, half precision, f32 results
        {"name": "adapter_mixed_ragged", "op": "adapter", "T": 777, "K": 4100, "N": 4093, "R": 24, "L": 12, "mix": "mixed",
         "none": 0.1, "dtype": "f16", "out": "f32", "want_u": False},
        # the training forward of four tenants' adapters on the long-K projection, u kept for the backward
        {"name": "adapter_train", "op": "adapter", "T": 8192, "K": 11008, "N": 4096, "R": 64, "L": 4, "mix": "runs",
         "none": 0.0, "dtype": "bf16", "out": "bf16", "want_u": True},
        # the backward of a small layer with short sequences of three adapters, ragged sizes
        {"name": "adapter_bwd_ragged", "op": "adapter_bwd", "T": 1500, "K": 4100, "N": 4093, "R": 24, "L": 3, "mix": "runs",
         "none": 0.05, "gbase": False},
        # a training step's backward on the square projection, the projection's own input gradient added in
        {"name": "adapter_bwd", "op": "adapter_bwd", "T": 4096, "K": 4096, "N": 4096, "R": 16, "L": 8, "mix": "runs",
         "none": 0.0, "gbase": True},
        # the loss alone while a short sequence is evaluated
        {"name": "distill_eval_small", "op": "distill", "T": 8, "V": 32000, "S": 32, "dtype": "bf16", "rest": False,
         "tau": 1.0, "pad_rows": 0.0, "pad_cols": 0},
        # evaluation over a batch: odd vocabulary with masked padding columns, f32 logits, the teacher's rest counted
        {"name": "distill_eval_odd", "op": "distill", "T": 512, "V": 50001, "S": 50, "dtype": "f32", "rest": True,
         "tau": 2.0, "pad_rows": 0.1, "pad_cols": 37},
        # the loss's gradient for logits that another loss reads as well: half precision, odd vocabulary
        {"name": "distill_bwd_odd", "op": "distill_bwd", "T": 300, "V": 50001, "S": 100, "dtype": "f16", "rest": True,
         "tau": 1.5, "pad_rows": 0.0, "pad_cols": 0},
        {"name": "distill_bwd", "op": "distill_bwd", "T": 2048, "V": 32000, "S": 64, "dtype": "bf16", "rest": False,
         "tau": 2.0, "pad_rows": 0.2, "pad_cols": 0},
        # a training step on a few sequences' last tokens, f32 logits
        {"name": "distill_step_small", "op": "distill_step", "T": 16, "V": 131072, "S": 64, "dtype": "f32", "rest": False,
         "tau": 1.0, "pad_rows": 0.0, "pad_cols": 0},
        # a training step over a full batch of a large vocabulary
        {"name": "distill_step", "op": "distill_step", "T": 4096, "V": 131072, "S": 64, "dtype": "bf16", "rest": True,
         "tau": 2.0, "pad_rows": 0.1, "pad_cols": 0},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _width(rng):
    """A projection's width: mostly whole 64s, now and then odd."""
    w = _log_int(rng, 256, 11008)
    return max(64, w // 64 * 64) if rng.random() < 0.7 else w


def draw(rng):
    op = rng.choice(["adapter", "adapter", "adapter_bwd", "distill", "distill_bwd", "distill_step"])
    if op.startswith("adapter"):
        K, N = _width(rng), _width(rng)
        R = rng.choice([4, 8, 16, 16, 24, 32, 64]) if rng.random() < 0.9 else rng.randint(1, 64)
        if op == "adapter":
            mix = rng.choice(["decode", "decode", "mixed", "runs"])
            T = _log_int(rng, 1, 256) if mix == "decode" else _log_int(rng, 16, 8192)
            return {"op": op, "T": T, "K": K, "N": N, "R": R, "L": _log_int(rng, 1, 64), "mix": mix,
                    "none": rng.choice([0.0, 0.1, 0.5]), "dtype": rng.choice(["bf16", "bf16", "f16"]),
                    "out": rng.choice(["same", "same", "f32"]), "want_u": rng.random() < 0.3}
        return {"op": op, "T": _log_int(rng, 16, 8192), "K": K, "N": N, "R": R, "L": _log_int(rng, 1, 16),
                "mix": rng.choice(["runs", "runs", "mixed"]), "none": rng.choice([0.0, 0.0, 0.2]),
                "gbase": rng.random() < 0.5}
    V = rng.choice([32000, 65536, 131072]) if rng.random() < 0.4 else _log_int(rng, 1000, 150000)
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    most = max(1, min(8192, 4096 * 131072 * 2 // (V * _SIZE[dtype])))
    return {"op": op, "T": _log_int(rng, 1, most), "V": V, "S": _log_int(rng, 1, 256), "dtype": dtype,
            "rest": rng.random() < 0.5, "tau": rng.choice([1.0, 1.5, 2.0, 4.0]), "pad_rows": rng.choice([0.0, 0.1, 0.3]),
            "pad_cols": rng.choice([0, 0, 17, 64])}


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------
def _adapter_ids(case, gen):
    """The adapter of every token (-1: none), as the scheduler of a batch has it on the host."""
    T, L, mix, none = case["T"], case["L"], case["mix"], case["none"]

    def rnd(n, hi):
        return torch.randint(0, hi, (n,), generator=gen)

    def pick(n):
        ids = rnd(n, L)
        ids[torch.rand(n, generator=gen) < none] = -1
        return ids

    if mix == "decode":                        # one token of every request, in any order
        return pick(T).tolist()
    if mix == "runs":                          # a few long sequences
        n = max(1, min(T, 2 * L))
    else:                                      # some prompts, then requests that decode
        n = max(1, min(6, T // 64))
    body = T if mix == "runs" else max(1, T - T // 10)
    cuts = sorted(rnd(n - 1, body).tolist()) if n > 1 else []
    cuts = [0] + cuts + [body]
    ids = []
    for (a, b), i in zip(zip(cuts[:-1], cuts[1:]), pick(n).tolist()):
        ids += [i] * (b - a)
    return ids + pick(T - body).tolist()


def _prepare_adapter(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    ids = _adapter_ids(case, torch.Generator().manual_seed(seed))
    T, K, N, R, L = (case[k] for k in "TKNRL")
    bwd = case["op"] == "adapter_bwd"
    dt = _DT["bf16" if bwd else case["dtype"]]

    def normal(*shape, std=1.0, dtype=dt):
        return (torch.randn(*shape, generator=gen, device=DEV) * std).to(dtype)

    st = {"case": case, "ids": ids, "x": normal(T, K), "a": normal(L, R, K, std=K ** -0.5),
          "b": normal(L, N, R, std=0.5 * R ** -0.5),
          "scale": torch.rand(L, generator=gen, device=DEV) + 0.5}
    if bwd:
        st["g"] = normal(T, N, std=0.01)
        st["gbase"] = normal(T, K, std=0.01) if case["gbase"] else None
        u = torch.zeros(T, R, device=DEV)      # what the forward kept
        for i, rows in _groups(ids):
            u[rows] = st["x"][rows].float() @ st["a"][i].float().t()
        st["u"] = u
    else:
        st["base"] = normal(T, N)              # the shared projection's result
    if own:
        import xnor_popcount_gemm_gb300 as bt
        st["bt"] = bt
        st["plan"] = bt.bt_adapter_plan(ids, L, device=DEV)
    else:
        st["groups"] = _groups(ids)
    return st


def _groups(ids):
    """(adapter, its tokens) of every adapter in use, tokens without one left out."""
    t = torch.tensor(ids)
    return [(int(i), (t == i).nonzero().flatten().to(DEV)) for i in t.unique().tolist() if i >= 0]


def _prepare_distill(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    T, V, S, tau = case["T"], case["V"], min(case["S"], case["V"] - case["pad_cols"]), case["tau"]
    dt = _DT[case["dtype"]]
    logits = torch.empty(T, V, dtype=dt, device=DEV)
    ids = torch.empty(T, S, dtype=torch.int32, device=DEV)
    top = torch.empty(T, S, device=DEV)
    tlse = torch.empty(T, device=DEV)
    rows = max(1, (1 << 27) // V)
    for r in range(0, T, rows):                # the teacher agrees with the student in part
        n = min(rows, T - r)
        z = torch.randn(n, V, generator=gen, device=DEV).mul_(2.0)
        t = z + torch.randn(n, V, generator=gen, device=DEV).mul_(1.5)
        t += 6.0 * (torch.rand(n, V, generator=gen, device=DEV) < 4.0 / V)
        if case["pad_cols"]:
            z[:, V - case["pad_cols"]:] = -math.inf
            t[:, V - case["pad_cols"]:] = -math.inf
        logits[r:r + n] = z.to(dt)
        v, i = t.topk(S, dim=1)
        top[r:r + n], ids[r:r + n] = v, i.int()
        tlse[r:r + n] = torch.logsumexp(t / tau, dim=1)
    pad = torch.rand(T, generator=gen, device=DEV) < case["pad_rows"]
    ids[pad] = -1                              # padding tokens: no teacher
    st = {"case": case, "logits": logits, "ids": ids, "top": top, "tlse": tlse if case["rest"] else None,
          # the mean over the tokens, tau^2 for the gradients' size, a loss scale for half precision
          "weight": (torch.rand(T, generator=gen, device=DEV) + 0.5) *
                    (tau * tau / T * (65536.0 if dt == torch.float16 else 1.0))}
    if case["op"] == "distill_bwd":
        st["stats"] = _stats(logits, ids, tau)
    if own:
        import xnor_popcount_gemm_gb300 as bt
        st["bt"] = bt
    return st


def prepare(case, seed):
    return _prepare_adapter(case, seed) if case["op"].startswith("adapter") else _prepare_distill(case, seed)


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------
def run(state):
    return {"adapter": _run_adapter, "adapter_bwd": _run_adapter_bwd, "distill": _run_distill,
            "distill_bwd": _run_distill_bwd, "distill_step": _run_distill_step}[state["case"]["op"]](state)


def _out_dtype(case):
    return _DT[case["dtype"] if case["out"] == "same" else case["out"]]


def _run_adapter(st):
    case, x, a, b = st["case"], st["x"], st["a"], st["b"]
    if own:
        u = torch.empty(case["T"], case["R"], device=x.device) if case["want_u"] else None
        y = st["bt"].bt_adapter_linear(x, a, b, st["scale"], st["plan"], base=st["base"], out_dtype=_out_dtype(case), u=u)
        return [y, u] if case["want_u"] else y
    y = st["base"].float()
    u = torch.zeros(case["T"], case["R"], device=x.device)
    for i, rows in st["groups"]:
        ui = x[rows].float() @ a[i].float().t()
        u[rows] = ui
        y[rows] += st["scale"][i] * (ui @ b[i].float().t())
    y = y.to(_out_dtype(case))
    return [y, u] if case["want_u"] else y


def _run_adapter_bwd(st):
    x, g, u, a, b = st["x"], st["g"], st["u"], st["a"], st["b"]
    if own:
        return list(st["bt"].bt_adapter_linear_backward(x, g, u, a, b, st["scale"], st["plan"], grad_base=st["gbase"]))
    gx = torch.zeros(x.shape, device=x.device) if st["gbase"] is None else st["gbase"].float()
    ga = torch.zeros(a.shape, device=x.device)
    gb = torch.zeros(b.shape, device=x.device)
    for i, rows in st["groups"]:
        gi = st["scale"][i] * g[rows].float()
        du = gi @ b[i].float()
        gx[rows] += du @ a[i].float()
        ga[i] = du.t() @ x[rows].float()
        gb[i] = gi.t() @ u[rows]
    return [gx.to(x.dtype), ga, gb]


def _in_slots(ids, V):
    """Which vocabulary entries are among a row's teacher slots."""
    m = torch.zeros(ids.shape[0], V + 1, dtype=torch.bool, device=ids.device)
    m.scatter_(1, torch.where(ids >= 0, ids, V).long(), True)
    return m[:, :V]


def _log_sum(a):
    m = a.amax(dim=1, keepdim=True)
    m = torch.where(m > -math.inf, m, 0.0)
    return m.squeeze(1) + (a - m).exp().sum(dim=1).log()


def _stats(logits, ids, tau):
    """(log sum of exp(z / tau), the same outside the teacher's slots) of every row; zeros for rows without a slot."""
    a = logits.float() / tau
    s = torch.stack([_log_sum(a), _log_sum(a.masked_fill(_in_slots(ids, logits.shape[1]), -math.inf))], dim=1)
    return torch.where((ids >= 0).any(dim=1, keepdim=True), s, 0.0)


def _teacher(top, ids, tlse, tau):
    """q over the slots and the rest's q, of every row."""
    t = torch.where(ids >= 0, top.float() / tau, -math.inf)
    if tlse is None:
        m = t.amax(dim=1, keepdim=True)
        e = (t - torch.where(m > -math.inf, m, 0.0)).exp()
        s = e.sum(dim=1, keepdim=True)
        return e / torch.where(s > 0, s, 1.0), None
    q = (t - tlse[:, None]).exp()
    return q, (1.0 - q.sum(dim=1)).clamp(min=0.0)


def _xlogy(q, lp):
    return torch.where(q > 0, q * lp, 0.0)


def _plain_loss(a, ids, q, qr, stats):
    lp = a.gather(1, ids.clamp(min=0).long()) - stats[:, :1]
    loss = _xlogy(q, q.log() - lp).sum(dim=1)
    if qr is not None:
        loss = loss + torch.where(stats[:, 1] > -math.inf, _xlogy(qr, qr.log() - (stats[:, 1] - stats[:, 0])), 0.0)
    return torch.where((ids >= 0).any(dim=1), loss, 0.0)


def _plain_grad(a, ids, q, qr, stats, weight, tau):
    has = (ids >= 0).any(dim=1)
    c = torch.where(has, weight / tau, 0.0)[:, None]
    if qr is None:
        grad = (a - stats[:, :1]).exp()
    else:
        pr = (stats[:, 1] - stats[:, 0]).exp()
        grad = torch.where(_in_slots(ids, a.shape[1]), (a - stats[:, :1]).exp(),
                           (pr - qr)[:, None] * (a - stats[:, 1:]).exp())
    grad.scatter_add_(1, ids.clamp(min=0).long(), -q)
    return torch.where(has[:, None], c * grad, 0.0)


def _run_distill(st):
    case, z, ids = st["case"], st["logits"], st["ids"]
    if own:
        return list(st["bt"].bt_distill_topk(z, ids, st["top"], st["tlse"], case["tau"]))
    stats = _stats(z, ids, case["tau"])
    q, qr = _teacher(st["top"], ids, st["tlse"], case["tau"])
    return [_plain_loss(z.float() / case["tau"], ids, q, qr, stats), stats]


def _run_distill_bwd(st):
    case, z, ids = st["case"], st["logits"], st["ids"]
    if own:
        return st["bt"].bt_distill_topk_backward(st["weight"], z, ids, st["top"], st["stats"], st["tlse"], case["tau"])
    q, qr = _teacher(st["top"], ids, st["tlse"], case["tau"])
    return _plain_grad(z.float() / case["tau"], ids, q, qr, st["stats"], st["weight"], case["tau"]).to(z.dtype)


def _run_distill_step(st):
    case, z, ids = st["case"], st["logits"], st["ids"]
    if own:
        return list(st["bt"].bt_distill_topk_step(st["weight"], z, ids, st["top"], st["tlse"], case["tau"]))
    stats = _stats(z, ids, case["tau"])
    q, qr = _teacher(st["top"], ids, st["tlse"], case["tau"])
    a = z.float() / case["tau"]
    return [_plain_loss(a, ids, q, qr, stats), _plain_grad(a, ids, q, qr, stats, st["weight"], case["tau"]).to(z.dtype)]


# ---------------------------------------------------------------------------
# What a pass cannot do without
# ---------------------------------------------------------------------------
def work(case):
    if case["op"].startswith("adapter"):
        T, K, N, R, L = (case[k] for k in "TKNRL")
        # adapters in use: at most every one, and one for each token
        used = min(L, T) if case["mix"] == "decode" else min(L, max(1, T // 16))
        if case["op"] == "adapter":
            out = _SIZE[case["dtype"] if case["out"] == "same" else case["out"]]
            moved = T * K * 2 + T * N * (2 + out) + used * R * (K + N) * 2 + (4 * T * R if case["want_u"] else 0)
            return {"bytes": moved, "flops": 2.0 * T * R * (K + N)}
        moved = T * (N + 2 * K) * 2 + (T * K * 2 if case["gbase"] else 0) + 4 * T * R + used * R * (K + N) * 2 + \
            4 * L * R * (K + N)
        return {"bytes": moved, "flops": 4.0 * T * R * (K + N)}
    T, V, S, e = case["T"], case["V"], case["S"], _SIZE[case["dtype"]]
    live = T * (1.0 - case["pad_rows"])        # rows without a teacher need no reading
    read = live * (V * e + 8 * S) + 16 * T
    written = 0 if case["op"] == "distill" else T * V * e
    return {"bytes": int(read + written), "flops": live * V * (5.0 if case["op"] != "distill_step" else 9.0)}


# ---------------------------------------------------------------------------
# The definition in 64 bits
# ---------------------------------------------------------------------------
def exact(case, seed):
    st = prepare(case, seed)
    if case["op"].startswith("adapter"):
        return _exact_adapter(case, st)
    return _exact_distill(case, st)


def _exact_adapter(case, st):
    x, a, b, s = (st[k].double() for k in ("x", "a", "b", "scale"))
    ids = torch.tensor(st["ids"], device=DEV)
    if case["op"] == "adapter":
        y = st["base"].double()
        u = torch.zeros(case["T"], case["R"], dtype=torch.float64, device=DEV)
        for i in range(case["L"]):
            rows = ids == i
            if rows.any():
                u[rows] = torch.einsum("tk,rk->tr", x[rows], a[i])
                y[rows] += torch.einsum("tr,nr->tn", u[rows], b[i]) * s[i]
        return [y, u] if case["want_u"] else y
    g, u = st["g"].double(), st["u"].double()
    gx = torch.zeros_like(x) if st["gbase"] is None else st["gbase"].double()
    ga, gb = torch.zeros_like(a), torch.zeros_like(b)
    for i in range(case["L"]):
        rows = ids == i
        if rows.any():
            du = torch.einsum("tn,nr->tr", g[rows], b[i]) * s[i]
            gx[rows] += torch.einsum("tr,rk->tk", du, a[i])
            ga[i] = torch.einsum("tr,tk->rk", du, x[rows])
            gb[i] = torch.einsum("tn,tr->nr", g[rows], u[rows]) * s[i]
    return [gx, ga, gb]


def _exact_distill(case, st):
    tau, T, V, op = case["tau"], case["T"], case["V"], case["op"]
    losses, stats, grads = [], [], []
    rows = max(1, (1 << 25) // V)
    for r in range(0, T, rows):
        ids = st["ids"][r:r + rows].long()
        a = st["logits"][r:r + rows].double() / tau
        live = ids >= 0
        some = live.any(dim=1)
        q = torch.zeros_like(a)                # the teacher's probabilities over the vocabulary
        t = torch.where(live, st["top"][r:r + rows].double() / tau, -math.inf)
        if st["tlse"] is None:
            w = torch.where(some[:, None], torch.softmax(torch.where(some[:, None], t, 0.0), dim=1), 0.0)
        else:
            w = (t - st["tlse"][r:r + rows, None].double()).exp()
        inside = torch.zeros_like(a, dtype=torch.int32)
        q.scatter_add_(1, ids.clamp(min=0), torch.where(live, w, 0.0))
        inside.scatter_add_(1, ids.clamp(min=0), live.int())
        inside = inside > 0
        lse = torch.logsumexp(a, dim=1)
        out = torch.logsumexp(a.masked_fill(inside, -math.inf), dim=1)
        logp = a - lse[:, None]
        term = torch.where(q > 0, q * (q.log() - logp), 0.0).sum(dim=1)
        d = logp.exp() - q
        if st["tlse"] is not None:
            rest = (1.0 - q.sum(dim=1)).clamp(min=0.0)
            term += torch.where((rest > 0) & (out > -math.inf), rest * (rest.log() - (out - lse)), 0.0)
            d = torch.where(inside, d, ((out - lse).exp() - rest)[:, None] * (a - out[:, None]).exp())
        losses.append(torch.where(some, term, 0.0))
        stats.append(torch.where(some[:, None], torch.stack([lse, out], dim=1), 0.0))
        if op != "distill":
            w = st["weight"][r:r + rows, None].double() / tau
            grads.append(torch.where(some[:, None], w * d, 0.0))
    if op == "distill":
        return [torch.cat(losses), torch.cat(stats)]
    return torch.cat(grads) if op == "distill_bwd" else [torch.cat(losses), torch.cat(grads)]
