"""Cases for timing the operators of a policy's recurrent core and of its head's loss.

Three operators: layer norm of a residual stream (forward, and backward with the
gradients of its weights), the gated linear recurrence over a rollout's steps
(forward, one step at a time or a whole sequence, and backward), and the
distillation of a head from a teacher's top logits (forward, backward, and both at once).
``run`` computes them in elementary torch operations, or, with ``own`` set,
through ``backward_implicit_gemm_amd.binding``; ``exact`` gives the definitions'
values in 64 bits.
"""
import math

import torch

own = False

DEV = "cuda"
EPS = 1e-5
TYPES = {"float32": torch.float32, "bfloat16": torch.bfloat16}
FEATURES = 128 * 1 * 2 + 47 * 32      # the encoder's feature row: conv2's outputs and the embedded features
MOST_NORM = 32768 * FEATURES          # elements of the largest listed cases
MOST_RECUR = 32768 * 1024
MOST_DISTILL = 4096 * 40960


# ---------------------------------------------------------------------------
# The cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # an agent acting alone: the feature row of one observation
        norm("norm fwd one observation", "norm_fwd", 1, FEATURES, "float32", residual=True),
        # the features of a whole rollout, the residual stream passed on beside the normed rows
        norm("norm fwd rollout", "norm_fwd", 32768, FEATURES, "bfloat16", residual=True),
        # one minibatch's gradient, fp32, no residual
        norm("norm bwd minibatch", "norm_bwd", 1024, FEATURES, "float32"),
        # a wide model's gradient, rows that are parts of wider ones
        norm("norm bwd wide", "norm_bwd", 8191, 4096, "bfloat16", residual=True, extra=256),
        # 64 agents acting: one step from their kept states
        recur("recurrence step", "recur_fwd", 64, 1, 512, "float32", h0=True),
        # a rollout's 64 steps of 512 environments, time first, episodes that end inside
        recur("recurrence fwd rollout", "recur_fwd", 512, 64, 512, "bfloat16", order="tb", reset=0.02, h0=True, joined=True),
        # one long text
        recur("recurrence fwd long", "recur_fwd", 1, 32768, 1024, "bfloat16"),
        # the rollout's gradient
        recur("recurrence bwd rollout", "recur_bwd", 512, 64, 512, "float32", order="tb", reset=0.02, h0=True, joined=True),
        # a few long texts of different lengths, an odd width
        recur("recurrence bwd long", "recur_bwd", 3, 12001, 777, "bfloat16", ragged=True, h0=True),
        # a minibatch's action heads: 300 actions, a tenth of them not allowed, the teacher's best 8;
        # loss and gradient at once
        distill("distillation step actions", "distill_step", 1024, 300, 8, "float32", masked=0.1),
        # a text vocabulary's gradient behind a loss taken before, of odd size, with some padded rows
        distill("distillation bwd vocabulary", "distill_bwd", 2048, 40961, 64, "bfloat16", temperature=2.0, empty=0.1),
        # loss and gradient of a larger batch at once
        distill("distillation step vocabulary", "distill_step", 4096, 40960, 64, "bfloat16", temperature=2.0, empty=0.1),
    ]


def norm(name, op, rows, dim, dtype, residual=False, extra=0, params="float32"):
    return {"name": name, "op": op, "rows": rows, "dim": dim, "dtype": dtype, "residual": residual, "extra": extra,
            "params": params}


def recur(name, op, batch, length, dim, dtype, order="bt", reset=0.0, h0=False, ragged=False, joined=False, coupled=True):
    return {"name": name, "op": op, "batch": batch, "length": length, "dim": dim, "dtype": dtype, "order": order,
            "reset": reset, "h0": h0, "ragged": ragged, "joined": joined, "coupled": coupled}


def distill(name, op, rows, vocab, top, dtype, temperature=1.0, masked=0.0, empty=0.0, index="int32", extra=0):
    return {"name": name, "op": op, "rows": rows, "vocab": vocab, "top": top, "dtype": dtype, "temperature": temperature,
            "masked": masked, "empty": empty, "index": index, "extra": extra}


def spread(rng, low, high):
    """A whole number of [low, high], spread over its logarithm."""
    return max(low, min(high, round(math.exp(rng.uniform(math.log(low), math.log(high))))))


def draw(rng):
    op = rng.choice(("norm_fwd", "norm_bwd", "recur_fwd", "recur_bwd", "distill_fwd", "distill_bwd", "distill_step"))
    dtype = rng.choice(("float32", "bfloat16"))
    if op.startswith("norm"):
        dim = spread(rng, 2, 12000)
        rows = spread(rng, 1, min(65536, MOST_NORM // 2 // dim))
        case = norm("", op, rows, dim, dtype, rng.random() < 0.6, rng.choice((0, 0, 1, 64)), rng.choice(("float32", dtype)))
    elif op.startswith("recur"):
        batch = spread(rng, 1, 1024)
        dim = spread(rng, 1, min(4096, MOST_RECUR // 2 // batch))
        length = spread(rng, 1, min(32768, MOST_RECUR // 2 // (batch * dim)))
        case = recur("", op, batch, length, dim, dtype, rng.choice(("bt", "tb")), rng.choice((0.0, 0.001, 0.05)),
                     rng.random() < 0.5, rng.random() < 0.3, rng.random() < 0.5, rng.random() < 0.8)
    else:
        vocab = spread(rng, 2, 150000)
        rows = spread(rng, 1, min(32768, MOST_DISTILL // 2 // vocab))
        case = distill("", op, rows, vocab, spread(rng, 1, min(vocab, 256)), dtype, rng.choice((1.0, 2.0, 0.7)),
                       rng.choice((0.0, 0.1)), rng.choice((0.0, 0.1)), rng.choice(("int32", "int64")), rng.choice((0, 0, 7)))
    del case["name"]
    return case


# ---------------------------------------------------------------------------
# What a program has in hand
# ---------------------------------------------------------------------------
def prepare(case, seed):
    gen = torch.Generator(DEV).manual_seed(int(seed))
    op = case["op"]
    if op.startswith("norm"):
        return _prepare_norm(case, gen)
    if op.startswith("recur"):
        return _prepare_recur(case, gen)
    return _prepare_distill(case, gen)


def _normal(gen, *shape):
    return torch.randn(shape, generator=gen, device=DEV)


def _rows(case, values, dtype=None):
    """Rows of `values` as parts of rows that are `extra` columns wider."""
    wide = torch.empty((values.shape[0], values.shape[1] + case["extra"]), dtype=dtype or TYPES[case["dtype"]], device=DEV)
    part = wide[:, :values.shape[1]]
    part.copy_(values)
    return part


def _prepare_norm(case, gen):
    rows, dim = case["rows"], case["dim"]
    pt = TYPES[case["params"]]
    # columns with their own offsets and widths, as a trained stream has them
    offset, width = 0.5 * _normal(gen, 1, dim), 0.3 + torch.rand((1, dim), generator=gen, device=DEV)
    state = {"case": case, "x": _rows(case, _normal(gen, rows, dim) * width + offset),
             "gamma": (1 + 0.2 * _normal(gen, dim)).to(pt), "beta": (0.2 * _normal(gen, dim)).to(pt)}
    if case["op"] == "norm_fwd":
        if case["residual"]:
            state["residual"] = _rows(case, 2 * _normal(gen, rows, dim))
    else:
        state["dy"] = _rows(case, _normal(gen, rows, dim))
        if case["residual"]:
            state["dtotal"] = _rows(case, _normal(gen, rows, dim))
        v = state["x"].double()
        mean = v.mean(1)
        state["mean"], state["rstd"] = mean.float(), ((v - mean[:, None]).square().mean(1) + EPS).rsqrt().float()
        del v
    if own:
        from backward_implicit_gemm_amd import binding as gb
        state["handle"] = gb.LayerNorm(rows, dim, TYPES[case["dtype"]], EPS, pt, DEV)
        state["out"] = _rows(case, torch.empty_like(state["x"]))
        if case["op"] == "norm_fwd":
            state["mean"], state["rstd"] = (torch.empty(rows, device=DEV) for _ in range(2))
            if case["residual"]:
                state["total"] = _rows(case, torch.empty_like(state["x"]))
        else:
            state["dgamma"], state["dbeta"] = (torch.empty(dim, dtype=pt, device=DEV) for _ in range(2))
    return state


def _lengths(case):
    """Valid steps of each sequence: all of them, or from all down to half, and one sequence without any."""
    batch, length = case["batch"], case["length"]
    if not case["ragged"]:
        return [length] * batch
    lengths = [length - (i * 7919) % (length // 2 + 1) for i in range(batch)]
    if batch > 3:
        lengths[-1] = 0
    return lengths


def _sequences(case, count):
    """`count` buffers of (batch, length, dim), time first in memory if the order says so; side by
    side in one buffer where they are joined."""
    batch, length, dim = case["batch"], case["length"], case["dim"]
    t = TYPES[case["dtype"]]
    outer = (batch, length) if case["order"] == "bt" else (length, batch)

    def view(w):
        return w if case["order"] == "bt" else w.transpose(0, 1)

    if case["joined"] and count == 2:
        both = torch.empty(outer + (2 * dim,), dtype=t, device=DEV)
        return [view(both[..., :dim]), view(both[..., dim:])]
    return [view(torch.empty(outer + (dim,), dtype=t, device=DEV)) for _ in range(count)]


def _prepare_recur(case, gen):
    batch, length, dim = case["batch"], case["length"], case["dim"]
    shape = (batch, length, dim)
    gate, value = _sequences(case, 2)
    # channels that forget within steps beside others that keep for hundreds
    gate.copy_(_normal(gen, *shape) + 6 * torch.rand(dim, generator=gen, device=DEV))
    value.copy_(_normal(gen, *shape))
    state = {"case": case, "gate": gate, "value": value, "h0": None, "reset": None, "lengths": None}
    if case["h0"]:
        state["h0"] = _normal(gen, batch, dim)
    if case["reset"]:
        reset = torch.rand((batch, length), generator=gen, device=DEV) < case["reset"]
        state["reset"] = reset if case["order"] == "bt" else reset.t().contiguous().t()
    if case["ragged"]:
        state["lengths"] = torch.tensor(_lengths(case), dtype=torch.int32, device=DEV)
    if case["op"] == "recur_bwd":
        state["dout"], = _sequences(case, 1)
        state["dout"].copy_(_normal(gen, *shape))
        state["dlast"] = _normal(gen, batch, dim)
    if own:
        from backward_implicit_gemm_amd import binding as gb
        h = state["handle"] = gb.Recurrence(batch, length, dim, TYPES[case["dtype"]], case["coupled"], DEV)
        state["out"], = _sequences(case, 1)
        state["last"] = torch.empty((batch, dim), device=DEV)
        # a single step is not trained on: nothing is kept for a backward pass
        state["states"] = torch.empty(h.states_shape, device=DEV) if length > 1 or case["op"] == "recur_bwd" else None
        if case["op"] == "recur_bwd":
            # the forward pass that a training step has behind it
            h.fwd(gate, value, state["out"], state["h0"], state["last"], state["states"], state["reset"], state["lengths"])
            state["dgate"], state["dvalue"] = _sequences(case, 2)
            state["dh0"] = torch.empty((batch, dim), device=DEV) if case["h0"] else None
    return state


def _has_gradient(case):
    return case["op"] in ("distill_bwd", "distill_step")


def _prepare_distill(case, gen):
    rows, vocab, top = case["rows"], case["vocab"], case["top"]
    t = TYPES[case["dtype"]]
    # a skewed student and a teacher that agrees with it in part
    shared = 2 * _normal(gen, rows, vocab)
    if case["masked"]:
        barred = torch.rand((rows, vocab), generator=gen, device=DEV) < case["masked"]
        barred[:, 0] = False
        shared.masked_fill_(barred, float("-inf"))
        del barred
    teacher, index = (shared + _normal(gen, rows, vocab)).topk(top, 1)
    logits = _rows(case, shared + 0.5 * _normal(gen, rows, vocab))
    del shared
    if case["empty"]:
        # rows of padding, and rows for which the teacher gave fewer entries
        index[torch.rand(rows, generator=gen, device=DEV) < case["empty"]] = -1
        short = torch.rand(rows, generator=gen, device=DEV) < case["empty"]
        index[:, top // 2 + 1:] = torch.where(short[:, None], -1, index[:, top // 2 + 1:])
    state = {"case": case, "logits": logits, "index": index.to(getattr(torch, case["index"])), "teacher": teacher}
    if case["op"] == "distill_bwd":
        v = logits.double() / case["temperature"]
        state["peak"] = logits.float().amax(1)
        state["mass"] = torch.exp(v - (state["peak"].double() / case["temperature"])[:, None]).sum(1).float()
        del v
    if _has_gradient(case):
        # the mean over the rows, some of them weighing less
        state["dloss"] = torch.rand(rows, generator=gen, device=DEV) / rows
    if own:
        from backward_implicit_gemm_amd import binding as gb
        state["handle"] = gb.Distill(rows, vocab, top, t, case["temperature"], torch.float32, DEV)
        if case["op"] != "distill_bwd":
            state["loss"], state["peak"], state["mass"] = (torch.empty(rows, device=DEV) for _ in range(3))
        if _has_gradient(case):
            state["out"] = _rows(case, torch.empty((rows, vocab), dtype=t, device=DEV))
    return state


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------
def run(state):
    s, op = state, state["case"]["op"]
    if own:
        h = s["handle"]
        if op == "norm_fwd":
            return h.fwd(s["x"], s["gamma"], s["beta"], s["out"], s["mean"], s["rstd"], s.get("residual"), s.get("total"))
        if op == "norm_bwd":
            return h.bwd(s["x"], s["gamma"], s["dy"], s["mean"], s["rstd"], s["out"], s["dgamma"], s["dbeta"],
                         s.get("dtotal"))
        if op == "recur_fwd":
            return h.fwd(s["gate"], s["value"], s["out"], s["h0"], s["last"], s["states"], s["reset"], s["lengths"])
        if op == "recur_bwd":
            return h.bwd(s["gate"], s["value"], s["states"], s["dout"], s["dgate"], s["dvalue"], s["dlast"], s["dh0"],
                         s["reset"], s["lengths"])
        if op == "distill_fwd":
            return h.fwd(s["logits"], s["index"], s["teacher"], s["loss"], s["peak"], s["mass"])
        if op == "distill_step":
            return h.step(s["logits"], s["index"], s["teacher"], s["dloss"], s["loss"], s["out"])
        return h.bwd(s["logits"], s["index"], s["teacher"], s["peak"], s["mass"], s["dloss"], s["out"])
    return {"norm_fwd": _norm_fwd, "norm_bwd": _norm_bwd, "recur_fwd": _recur_fwd, "recur_bwd": _recur_bwd,
            "distill_fwd": _distill_fwd, "distill_bwd": _distill_bwd, "distill_step": _distill_step}[op](s)


def _norm_fwd(s):
    t, x = s["x"].dtype, s["x"].float()
    if "residual" in s:
        x = x + s["residual"].float()
    mean = x.mean(1, keepdim=True)
    off = x - mean
    rstd = 1 / torch.sqrt((off * off).mean(1, keepdim=True) + EPS)
    y = (off * rstd * s["gamma"].float() + s["beta"].float()).to(t)
    return y, mean[:, 0], rstd[:, 0], x.to(t) if "residual" in s else None


def _norm_bwd(s):
    t, dy = s["x"].dtype, s["dy"].float()
    rstd = s["rstd"][:, None]
    hat = (s["x"].float() - s["mean"][:, None]) * rstd
    w = dy * s["gamma"].float()
    dx = rstd * (w - w.mean(1, keepdim=True) - hat * (w * hat).mean(1, keepdim=True))
    if "dtotal" in s:
        dx = dx + s["dtotal"].float()
    return dx.to(t), (dy * hat).sum(0).to(s["gamma"].dtype), dy.sum(0).to(s["gamma"].dtype)


def _gates(s):
    """The valid steps, the share a step keeps of the state before it and takes of its value, and its values."""
    c = s["case"]
    f, v = s["gate"].float(), s["value"].float()
    e = torch.exp(-f.abs())
    small, large = e / (1 + e), 1 / (1 + e)
    a, i = torch.where(f >= 0, large, small), torch.where(f >= 0, small, large)
    ok = None
    if s["lengths"] is not None:
        ok = (torch.arange(c["length"], device=DEV) < s["lengths"][:, None])[..., None]
    return ok, a, i, v


def _scan(a, b, first):
    """h_t = a_t h_{t-1} + b_t along the steps, h before them `first`; by doubling distances."""
    a, b = a.clone(), b.clone()
    if first is not None:
        b[:, 0] += a[:, 0] * first
    step = 1
    while step < a.shape[1]:
        b[:, step:] = b[:, step:] + a[:, step:] * b[:, :-step]
        a[:, step:] = a[:, step:] * a[:, :-step]
        step *= 2
    return b


def _kept(s, ok, a):
    """The share of the state before a step that goes on: none at a reset, all of it behind the end."""
    if s["reset"] is not None:
        a = torch.where(s["reset"][..., None], 0.0, a)
    return a if ok is None else torch.where(ok, a, 1.0)


def _recur_fwd(s):
    ok, a, i, v = _gates(s)
    b = i * v if s["case"]["coupled"] else v
    if ok is not None:
        b = torch.where(ok, b, 0.0)
    h = _scan(_kept(s, ok, a), b, s["h0"])
    last = h[:, -1].clone()
    return (h if ok is None else torch.where(ok, h, 0.0)).to(s["gate"].dtype), last


def _recur_bwd(s):
    coupled, t = s["case"]["coupled"], s["gate"].dtype
    ok, a, i, v = _gates(s)
    kept = _kept(s, ok, a)
    b, dout = i * v if coupled else v, s["dout"].float()
    if ok is not None:
        b, dout = torch.where(ok, b, 0.0), torch.where(ok, dout, 0.0)
    h = _scan(kept, b, s["h0"])
    first = torch.zeros_like(h[:, :1]) if s["h0"] is None else s["h0"][:, None]
    before = torch.cat([first, h[:, :-1]], 1)
    if s["reset"] is not None:
        before = torch.where(s["reset"][..., None], 0.0, before)
    after = torch.cat([kept[:, 1:], torch.ones_like(kept[:, :1])], 1)
    g = _scan(after.flip(1), dout.flip(1), s["dlast"]).flip(1)
    dgate = a * i * (before - v if coupled else before) * g
    dvalue = i * g if coupled else g
    if ok is not None:
        dgate, dvalue = torch.where(ok, dgate, 0.0), torch.where(ok, dvalue, 0.0)
    dh0 = None if s["h0"] is None else kept[:, 0] * g[:, 0]
    return dgate.to(t), dvalue.to(t), dh0


def _shares(s):
    """The teacher's shares of its entries, and log of them; entries outside the vocabulary have none."""
    tau = s["case"]["temperature"]
    index = s["index"].long()
    ok = (index >= 0) & (index < s["case"]["vocab"])
    t = torch.where(ok, s["teacher"].float() / tau, -math.inf)
    peak = t.amax(1, keepdim=True)
    t = t - torch.where(peak == -math.inf, 0.0, peak)
    e = torch.exp(t)
    total = e.sum(1, keepdim=True)
    total = torch.where(total == 0, 1.0, total)
    return index.clamp(min=0), e / total, t - torch.log(total)


def _distill_fwd(s):
    tau = s["case"]["temperature"]
    z = s["logits"].float()
    peak = z.amax(1)
    mass = torch.exp((z - peak[:, None]) / tau).sum(1)
    index, p, logp = _shares(s)
    logq = (z.gather(1, index) - peak[:, None]) / tau - torch.log(mass)[:, None]
    loss = tau * tau * torch.where(p > 0, p * (logp - logq), 0.0).sum(1)
    return loss, peak, mass


def _distill_step(s):
    loss, peak, mass = _distill_fwd(s)
    return loss, _distill_bwd({**s, "peak": peak, "mass": mass})


def _distill_bwd(s):
    tau = s["case"]["temperature"]
    q = torch.exp((s["logits"].float() - s["peak"][:, None]) / tau) / s["mass"][:, None]
    index, p, _ = _shares(s)
    some = (p > 0).any(1, keepdim=True)
    dz = torch.where(some, q, 0.0).scatter_add(1, index, -p) * (s["dloss"] * tau)[:, None]
    return dz.to(s["logits"].dtype)


# ---------------------------------------------------------------------------
# What a pass cannot do without, and the definitions' values
# ---------------------------------------------------------------------------
def work(case):
    op = case["op"]
    size = 4 if case["dtype"] == "float32" else 2
    if op.startswith("norm"):
        n, params = case["rows"] * case["dim"], case["dim"] * (4 if case["params"] == "float32" else 2)
        more = 1 if case["residual"] else 0
        if op == "norm_fwd":
            return {"bytes": n * size * (2 + 2 * more) + 8 * case["rows"] + 2 * params, "flops": 8 * n}
        return {"bytes": n * size * (3 + more) + 8 * case["rows"] + 3 * params, "flops": 14 * n}
    if op.startswith("recur"):
        cells = case["batch"] * case["length"] * case["dim"]
        valid = sum(_lengths(case)) * case["dim"]
        flags = case["batch"] * case["length"] if case["reset"] else 0
        ends = 4 * case["batch"] * case["dim"]
        # read where valid, written everywhere; the state before the first step and the one after the last
        if op == "recur_fwd":
            return {"bytes": size * (2 * valid + cells) + flags + ends * (2 if case["h0"] else 1), "flops": 8 * valid}
        return {"bytes": size * (3 * valid + 2 * cells) + flags + ends * (3 if case["h0"] else 1), "flops": 20 * valid}
    n, k = case["rows"] * case["vocab"], case["rows"] * case["top"]
    entries = k * (4 + (4 if case["index"] == "int32" else 8))
    if op == "distill_fwd":
        return {"bytes": n * size + entries + 12 * case["rows"], "flops": 5 * n}
    return {"bytes": 2 * n * size + entries + 12 * case["rows"], "flops": (6 if op == "distill_bwd" else 9) * n}


def exact(case, seed):
    s = prepare(case, seed)
    return {"norm_fwd": _exact_norm_fwd, "norm_bwd": _exact_norm_bwd, "recur_fwd": _exact_recur_fwd,
            "recur_bwd": _exact_recur_bwd, "distill_fwd": _exact_distill_fwd, "distill_bwd": _exact_distill_bwd,
            "distill_step": _exact_distill_step}[case["op"]](s)


def _exact_norm_fwd(s):
    total = s["x"].double()
    if "residual" in s:
        total = total + s["residual"].double()
    var, mean = torch.var_mean(total, 1, correction=0)
    rstd = (var + EPS).pow(-0.5)
    y = torch.addcmul(s["beta"].double(), (total - mean[:, None]) * rstd[:, None], s["gamma"].double())
    return y, mean, rstd, total if "residual" in s else None


def _exact_norm_bwd(s):
    n, dy = s["case"]["dim"], s["dy"].double()
    hat = s["x"].double().sub_(s["mean"].double()[:, None]).mul_(s["rstd"].double()[:, None])
    dgamma, dbeta = torch.einsum("rd,rd->d", dy, hat), dy.sum(0)
    w = dy.mul_(s["gamma"].double())
    along = torch.einsum("rd,rd->r", w, hat) / n
    dx = (w - w.sum(1, keepdim=True) / n - along[:, None] * hat) * s["rstd"].double()[:, None]
    if "dtotal" in s:
        dx += s["dtotal"].double()
    return dx, dgamma, dbeta


def _exact_steps(s):
    """The recurrence one step at a time; yields (step, valid, goes on, keep, take, value, state before)."""
    c = s["case"]
    h = torch.zeros((c["batch"], c["dim"]), dtype=torch.float64, device=DEV) if s["h0"] is None else s["h0"].double()
    lengths = torch.tensor(_lengths(c), device=DEV)[:, None]
    for t in range(c["length"]):
        f = s["gate"][:, t].double()
        keep, v = torch.sigmoid(f), s["value"][:, t].double()
        take = torch.sigmoid(-f) if c["coupled"] else 1.0
        valid = t < lengths if c["ragged"] else None
        on = h if s["reset"] is None else h.masked_fill(s["reset"][:, t, None], 0.0)
        yield t, valid, keep, take, v, on
        new = keep * on + take * v
        h = new if valid is None else torch.where(valid, new, h)
    yield None, None, None, None, None, h


def _exact_recur_fwd(s):
    c = s["case"]
    out = torch.zeros((c["batch"], c["length"], c["dim"]), dtype=torch.float64, device=DEV)
    for t, valid, keep, take, v, before in _exact_steps(s):
        if t is None:
            return out, before
        h = keep * before + take * v
        out[:, t] = h if valid is None else h * valid
    return None


def _exact_recur_bwd(s):
    c = s["case"]
    befores = torch.empty((c["length"], c["batch"], c["dim"]), dtype=torch.float64, device=DEV)
    for t, *_, before in _exact_steps(s):
        if t is not None:
            befores[t] = before
    dgate, dvalue = (torch.zeros((c["batch"], c["length"], c["dim"]), dtype=torch.float64, device=DEV) for _ in range(2))
    lengths = torch.tensor(_lengths(c), device=DEV)[:, None]
    back = s["dlast"].double()          # gradient of the state behind step t
    for t in range(c["length"] - 1, -1, -1):
        f = s["gate"][:, t].double()
        keep, left = torch.sigmoid(f), torch.sigmoid(-f)
        g = back + s["dout"][:, t].double()
        v = s["value"][:, t].double()
        dg = g * keep * left * (befores[t] - v if c["coupled"] else befores[t])
        dv = g * left if c["coupled"] else g
        through = g * keep
        if s["reset"] is not None:
            through = through.masked_fill(s["reset"][:, t, None], 0.0)
        if c["ragged"]:
            valid = t < lengths
            dg, dv, through = dg * valid, dv * valid, torch.where(valid, through, back)
        dgate[:, t], dvalue[:, t], back = dg, dv, through
    return dgate, dvalue, None if s["h0"] is None else back


def _exact_shares(s):
    c = s["case"]
    ok = (s["index"] >= 0) & (s["index"] < c["vocab"])
    t = (s["teacher"].double() / c["temperature"]).masked_fill(~ok, -math.inf)
    logp = torch.log_softmax(t, 1)
    return s["index"].long().clamp(0, c["vocab"] - 1), logp.exp().nan_to_num(nan=0.0), logp


def _exact_distill_fwd(s):
    tau = s["case"]["temperature"]
    z = s["logits"].double()
    peak = z.max(1).values
    z.sub_(peak[:, None]).div_(tau)
    lse = torch.logsumexp(z, 1)
    index, p, logp = _exact_shares(s)
    kl = torch.xlogy(p, p) - p * (z.gather(1, index) - lse[:, None])
    return tau ** 2 * kl.masked_fill(p == 0, 0.0).sum(1), peak, lse.exp()


def _exact_gradient(s, q):
    index, p, _ = _exact_shares(s)
    q.mul_((p.sum(1, keepdim=True) > 0).double())
    for k in range(p.shape[1]):
        q.scatter_add_(1, index[:, k:k + 1], -p[:, k:k + 1])
    return q.mul_(s["dloss"].double()[:, None] * s["case"]["temperature"])


def _exact_distill_bwd(s):
    z = s["logits"].double()
    z.sub_(s["peak"].double()[:, None]).div_(s["case"]["temperature"]).exp_().div_(s["mass"].double()[:, None])
    return _exact_gradient(s, z)


def _exact_distill_step(s):
    return _exact_distill_fwd(s)[0], _exact_gradient(s, torch.softmax(s["logits"].double() / s["case"]["temperature"], 1))
