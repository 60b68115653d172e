"""More operators of large language models that are measured: the token embedding, the layer norm and
the gated linear recurrence, each with its gradient.

Each case names its operator and sizes.  ``run`` computes it in elementary
torch operations, or with ``own`` through the library's own calls.
"""
import math

import torch

own = False

_DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
_SIZE = {"f32": 4, "bf16": 2, "f16": 2}
_BLOCK = 1 << 26          # elements that inputs are made and plain forms are taken at a time
_EPS = 1e-5
_KEEP = 128               # the recurrence's states are kept for its gradient before every 128th step


# ---------------------------------------------------------------------------
# cases


def listed():
    return [
        # the newest token of each sequence of a decoding batch: latency
        dict(name="embed_step", op="embedding", tokens=64, vocab=32768, dim=4096, table="bf16", dtype="bf16", skipped=0.0),
        # a training batch with some padding, master weights in 32 bits, activations in 16
        dict(name="embed_train", op="embedding", tokens=16384, vocab=65536, dim=2048, table="f32", dtype="bf16",
             skipped=0.05),
        # the table's gradient for a training batch: most of the vocabulary is not met, a few tokens very often
        dict(name="embed_grad", op="embedding_grad", tokens=16384, vocab=65536, dim=2048, table="bf16", dtype="bf16",
             skipped=0.05),
        # a small batch in 32 bits, odd in every size
        dict(name="embed_grad_odd", op="embedding_grad", tokens=3001, vocab=10007, dim=1001, table="f32", dtype="f32",
             skipped=0.0),
        # the norm of a few new tokens: latency
        dict(name="norm_step", op="norm", rows=8, cols=4096, params="bf16", dtype="bf16"),
        # the norm of a training batch
        dict(name="norm_train", op="norm", rows=16384, cols=4096, params="f32", dtype="bf16"),
        # its gradients, the weight's and the bias's among them
        dict(name="norm_grad", op="norm_grad", rows=16384, cols=4096, params="f32", dtype="bf16"),
        # a ragged batch in 32 bits with rows at odd addresses
        dict(name="norm_grad_odd", op="norm_grad", rows=4099, cols=1021, params="f32", dtype="f32"),
        # one step of a decoding batch with its states
        dict(name="rec_step", op="recurrence", batch=64, time=1, channels=4096, form="sigmoid", ragged=False, dtype="bf16"),
        # one very long document
        dict(name="rec_long", op="recurrence", batch=1, time=65536, channels=2048, form="sigmoid", ragged=False,
             dtype="bf16"),
        # the gradients of a training batch
        dict(name="rec_grad", op="recurrence_grad", batch=8, time=4096, channels=2048, form="sigmoid", ragged=False,
             dtype="bf16"),
        # a padded batch of ragged lengths in 32 bits with decays as they are, odd in every size
        dict(name="rec_grad_odd", op="recurrence_grad", batch=5, time=1531, channels=509, form="decay", ragged=True,
             dtype="f32"),
    ]


_MOST_BYTES = 806_000_000        # no drawn case costs more than the largest listed one


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    while True:
        op = rng.choice(["embedding", "embedding_grad", "norm", "norm_grad", "recurrence", "recurrence_grad"])
        dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
        if op in ("embedding", "embedding_grad"):
            case = dict(op=op, tokens=_log(rng, 1, 32768), vocab=_log(rng, 1000, 262144), dim=_log(rng, 64, 8192),
                        table=rng.choice([dtype, "f32"]), dtype=dtype, skipped=rng.choice([0.0, 0.05, 0.5]))
            wide = "dim"
        elif op in ("norm", "norm_grad"):
            case = dict(op=op, rows=_log(rng, 1, 32768), cols=_log(rng, 32, 16384), params=rng.choice([dtype, "f32"]),
                        dtype=dtype)
            wide = "cols"
        else:
            case = dict(op=op, batch=_log(rng, 1, 64), time=rng.choice([1, _log(rng, 1, 65536), _log(rng, 64, 65536)]),
                        channels=_log(rng, 16, 8192), form=rng.choice(["sigmoid", "decay"]), ragged=rng.random() < 0.3,
                        dtype=dtype)
            wide = "channels"
        if rng.random() < 0.6:
            case[wide] = (case[wide] + 31) // 32 * 32
        if work(case)["bytes"] <= _MOST_BYTES:
            return case


# ---------------------------------------------------------------------------
# inputs


def _normal(shape, dtype, gen, spread=1.0, offset=0.0):
    out = torch.empty(shape, device="cuda", dtype=dtype)
    flat = out.view(-1)
    for at in range(0, flat.numel(), _BLOCK):
        part = flat[at:at + _BLOCK]
        part.copy_(torch.randn(part.shape, device="cuda", generator=gen) * spread + offset)
    return out


def _tokens(case, gen):
    """Tokens whose frequency falls as one over their rank; the ranks are spread over the table."""
    n, vocab = case["tokens"], case["vocab"]
    u = torch.rand(n, device="cuda", generator=gen, dtype=torch.float64)
    rank = (torch.exp(u * math.log(vocab + 1)) - 1).long().clamp(0, vocab - 1)
    order = torch.randperm(vocab, device="cuda", generator=gen)
    tokens = order[rank].to(torch.int32)
    skip = torch.rand(n, device="cuda", generator=gen) < case["skipped"]
    return torch.where(skip, torch.full_like(tokens, -1), tokens)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dt = _DTYPES[case["dtype"]]
    s = {"case": case}
    if case["op"] in ("embedding", "embedding_grad"):
        s["tokens"] = _tokens(case, gen)
        s["scale"] = math.sqrt(case["dim"])
        if case["op"] == "embedding":
            s["table"] = _normal((case["vocab"], case["dim"]), _DTYPES[case["table"]], gen, case["dim"] ** -0.5)
        else:
            s["grad"] = _normal((case["tokens"], case["dim"]), dt, gen, 1e-2)
    elif case["op"] in ("norm", "norm_grad"):
        rows, cols = case["rows"], case["cols"]
        x = _normal((rows, cols), dt, gen, 1.5)
        x += torch.randn(rows, 1, device="cuda", generator=gen).to(dt)           # rows have means of their own,
        x[:, torch.randint(0, cols, (2,), device="cuda", generator=gen)] *= 20   # and a few columns stand out
        s["x"] = x
        s["weight"] = _normal((cols,), _DTYPES[case["params"]], gen, 0.2, 1.0)
        s["bias"] = _normal((cols,), _DTYPES[case["params"]], gen, 0.2)
        if case["op"] == "norm_grad":
            _, s["mean"], s["rstd"] = _plain_norm(x, s["weight"], s["bias"])
            s["grad"] = _normal((rows, cols), dt, gen, 1e-2)
    else:
        batch, time, channels = case["batch"], case["time"], case["channels"]
        shape = (batch, time, channels)
        s["x"] = _normal(shape, dt, gen)
        if case["form"] == "sigmoid":
            s["gate"] = _normal(shape, dt, gen, 2.0, 2.0)
        else:
            s["gate"] = torch.empty(shape, device="cuda", dtype=dt)
            flat = s["gate"].view(-1)
            for at in range(0, flat.numel(), _BLOCK):
                part = flat[at:at + _BLOCK]
                part.copy_(1 - torch.rand(part.shape, device="cuda", generator=gen) ** 2 * 0.5)
        s["initial"] = _normal((batch, channels), torch.float32, gen)
        s["lengths"] = None
        if case["ragged"]:
            n = (torch.rand(batch, generator=torch.Generator().manual_seed(seed)) * (time + 1)).long()
            n[0] = time
            if batch > 2:
                n[1] = 0                                    # a slot of the batch that holds no sequence
            s["lengths"] = n.to(torch.int32).cuda()
            for b in range(batch):                          # memory past a sequence's end has never been written
                s["x"][b, n[b]:] = math.nan
                s["gate"][b, n[b]:] = math.nan
        if case["op"] == "recurrence_grad":
            s["grad"] = _normal(shape, dt, gen)
            s["grad_final"] = _normal((batch, channels), torch.float32, gen)
            if case["ragged"]:
                for b in range(batch):
                    s["grad"][b, n[b]:] = math.nan
            a, u, _ = _gated(s)
            h = _scan(a, u, s["initial"])
            s["states"] = torch.cat([s["initial"][:, None], h[:, _KEEP - 1:time - 1:_KEEP]], 1).contiguous()
    return s


# ---------------------------------------------------------------------------
# one pass


def run(state):
    return (_run_own if own else _run_plain)(state["case"], state)


def _run_own(case, s):
    from deterministic_floating_point_gb300 import det
    op = case["op"]
    if op == "embedding":
        return det.det_embedding(s["table"], s["tokens"], scale=s["scale"], dtype=_DTYPES[case["dtype"]])
    if op == "embedding_grad":
        return det.det_embedding_backward(s["grad"], s["tokens"], case["vocab"], scale=s["scale"],
                                          dtype=_DTYPES[case["table"]])
    if op == "norm":
        r = det.det_layer_norm(s["x"], s["weight"], s["bias"], eps=_EPS)
        return {"out": r.out, "mean": r.mean, "rstd": r.rstd}
    if op == "norm_grad":
        r = det.det_layer_norm_backward(s["grad"], s["x"], s["mean"], s["rstd"], s["weight"])
        return {"x": r.x, "weight": r.weight, "bias": r.bias}
    if op == "recurrence":
        r = det.det_linear_recurrence(s["x"], s["gate"], s["initial"], form=case["form"], lengths=s["lengths"])
        return {"out": r.out, "final": r.final}
    r = det.det_linear_recurrence_backward(s["grad"], s["x"], s["gate"], s["states"], grad_final=s["grad_final"],
                                           form=case["form"], lengths=s["lengths"])
    return {"x": r.x, "gate": r.gate, "initial": r.initial}


def _plain_norm(x, weight, bias):
    x32 = x.float()
    mean = x32.mean(1)
    d = x32 - mean[:, None]
    rstd = 1 / torch.sqrt((d * d).mean(1) + _EPS)
    return (d * rstd[:, None] * weight.float() + bias.float()).to(x.dtype), mean, rstd


def _valid(s):
    if s["lengths"] is None:
        return None
    return (torch.arange(s["case"]["time"], device="cuda")[None, :] < s["lengths"][:, None])[:, :, None]


def _gated(s):
    """(decay, input, 1 - decay) of every step in 32 bits; steps past a sequence's end change nothing."""
    x, gate = s["x"].float(), s["gate"].float()
    if s["case"]["form"] == "sigmoid":
        a, rest = 1 / (1 + torch.exp(-gate)), 1 / (1 + torch.exp(gate))
        u = rest * x
    else:
        a, u, rest = gate, x, None
    valid = _valid(s)
    if valid is not None:
        a, u = torch.where(valid, a, torch.ones_like(a)), torch.where(valid, u, torch.zeros_like(u))
    return a, u, rest


def _scan(a, u, initial):
    """h[t] = a[t] h[t-1] + u[t] along the second dimension, by doubling distances."""
    a, h = a.clone(), u.clone()
    h[:, 0] += a[:, 0] * initial
    step, time = 1, a.shape[1]
    while step < time:
        more = a[:, step:] * h[:, :-step]
        h[:, step:] += more
        del more
        a[:, step:] = a[:, step:] * a[:, :-step]
        step *= 2
    return h


def _run_plain(case, s):
    op = case["op"]
    if op == "embedding":
        tok = s["tokens"].long()
        rows = s["table"][tok.clamp(0, case["vocab"] - 1)].float() * s["scale"]
        return torch.where((tok >= 0)[:, None], rows, torch.zeros_like(rows)).to(_DTYPES[case["dtype"]])
    if op == "embedding_grad":
        tok = s["tokens"].long()
        total = torch.zeros(case["vocab"] + 1, case["dim"], device="cuda")
        total.index_add_(0, torch.where(tok >= 0, tok, torch.full_like(tok, case["vocab"])), s["grad"].float())
        return (total[:-1] * s["scale"]).to(_DTYPES[case["table"]])
    if op == "norm":
        out, mean, rstd = _plain_norm(s["x"], s["weight"], s["bias"])
        return {"out": out, "mean": mean, "rstd": rstd}
    if op == "norm_grad":
        xh = (s["x"].float() - s["mean"][:, None]) * s["rstd"][:, None]
        g = s["grad"].float()
        gw = g * s["weight"].float()
        gx = (gw - gw.mean(1, keepdim=True) - xh * (gw * xh).mean(1, keepdim=True)) * s["rstd"][:, None]
        dt = s["weight"].dtype
        return {"x": gx.to(s["x"].dtype), "weight": (g * xh).sum(0).to(dt), "bias": g.sum(0).to(dt)}
    dt, valid = s["x"].dtype, _valid(s)
    a, u, rest = _gated(s)
    h = _scan(a, u, s["initial"])
    if op == "recurrence":
        final = h[:, -1].clone()
        if valid is not None:
            h = torch.where(valid, h, torch.zeros_like(h))
        return {"out": h.to(dt), "final": final}
    before = torch.cat([s["initial"][:, None], h[:, :-1]], 1)
    g = s["grad"].float()
    if valid is not None:
        g = torch.where(valid, g, torch.zeros_like(g))
    # the state's gradient runs backwards: that of step t takes step t + 1's, decayed
    later = torch.cat([a[:, 1:], torch.ones_like(a[:, :1])], 1)
    back = _scan(later.flip(1), g.flip(1), s["grad_final"]).flip(1)
    initial = a[:, 0] * back[:, 0]
    if case["form"] == "sigmoid":
        gate, x = back * (before - s["x"].float()) * a * rest, back * rest
    else:
        gate, x = back * before, back
    if valid is not None:
        gate, x = torch.where(valid, gate, torch.zeros_like(gate)), torch.where(valid, x, torch.zeros_like(x))
    return {"x": x.to(dt), "gate": gate.to(dt), "initial": initial}


# ---------------------------------------------------------------------------
# what a pass cannot do without


def work(case):
    size, op = _SIZE[case["dtype"]], case["op"]
    if op in ("embedding", "embedding_grad"):
        used, dim, vocab, table = case["tokens"] * (1 - case["skipped"]), case["dim"], case["vocab"], _SIZE[case["table"]]
        if op == "embedding":
            rank = torch.arange(vocab, dtype=torch.float64)
            p = torch.log((rank + 2) / (rank + 1)) / math.log(vocab + 1)
            met = float((1 - (1 - p) ** used).sum())                # rows of the table that are needed
            return {"bytes": int(met * dim * table + case["tokens"] * (dim * size + 4)),
                    "flops": int(used * dim)}
        return {"bytes": int(used * dim * size + vocab * dim * table + case["tokens"] * 4), "flops": int(used * dim)}
    if op in ("norm", "norm_grad"):
        n, small = case["rows"] * case["cols"], case["cols"] * _SIZE[case["params"]]
        if op == "norm":
            return {"bytes": 2 * n * size + 8 * case["rows"] + 2 * small, "flops": 7 * n}
        return {"bytes": 3 * n * size + 8 * case["rows"] + 3 * small, "flops": 13 * n}
    batch, time = case["batch"], case["time"]
    steps = batch * time
    if case["ragged"]:          # the first sequence is whole, the second empty, the others half as long on average
        steps = time + int(time / 2 * max(0, batch - 2 if batch > 2 else batch - 1))
    rows, c = batch * time, case["channels"]
    kept = -(-time // _KEEP)
    if op == "recurrence":
        return {"bytes": (2 * steps + rows) * c * size + 8 * batch * c, "flops": 2 * steps * c}
    return {"bytes": (3 * steps + 2 * rows) * c * size + (4 * kept + 8) * batch * c, "flops": 6 * steps * c}


# ---------------------------------------------------------------------------
# the definitions in 64 bits


def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    if op == "embedding":
        out = torch.nn.functional.embedding(s["tokens"].long().clamp(min=0), s["table"]).double()
        return out.mul_(s["scale"]).masked_fill_((s["tokens"] < 0)[:, None], 0.0)
    if op == "embedding_grad":
        # the tokens in order of their row, each row's run summed
        order = torch.argsort(s["tokens"], stable=True)
        row, count = torch.unique_consecutive(s["tokens"][order], return_counts=True)
        out = torch.zeros(case["vocab"], case["dim"], dtype=torch.float64, device="cuda")
        start = 0
        for r, n in zip(row.tolist(), count.tolist()):
            if r >= 0:
                out[r] = s["grad"][order[start:start + n]].double().sum(0)
            start += n
        return out.mul_(s["scale"])
    if op == "norm":
        out = torch.empty(s["x"].shape, dtype=torch.float64, device="cuda")
        mean, rstd = (torch.empty(case["rows"], dtype=torch.float64, device="cuda") for _ in range(2))
        step = max(1, _BLOCK // case["cols"])
        for r in range(0, case["rows"], step):
            x = s["x"][r:r + step].double()
            var, mu = torch.var_mean(x, 1, correction=0)
            mean[r:r + step], rstd[r:r + step] = mu, torch.rsqrt(var + _EPS)
            out[r:r + step] = torch.addcmul(s["bias"].double(), (x - mu[:, None]) * rstd[r:r + step, None],
                                            s["weight"].double())
        return {"out": out, "mean": mean, "rstd": rstd}
    if op == "norm_grad":
        gx = torch.empty(s["x"].shape, dtype=torch.float64, device="cuda")
        weight, bias = (torch.zeros(case["cols"], dtype=torch.float64, device="cuda") for _ in range(2))
        step = max(1, _BLOCK // case["cols"])
        w, n = s["weight"].double(), case["cols"]
        for r in range(0, case["rows"], step):
            rstd = s["rstd"][r:r + step].double()[:, None]
            xh = (s["x"][r:r + step].double() - s["mean"][r:r + step].double()[:, None]) * rstd
            g = s["grad"][r:r + step].double()
            one, two = (g @ w)[:, None] / n, ((g * xh) @ w)[:, None] / n
            gx[r:r + step] = rstd * (torch.addcmul(-one, g, w) - xh * two)
            weight += torch.einsum("rc,rc->c", g, xh)
            bias += g.sum(0)
        return {"x": gx, "weight": weight, "bias": bias}
    # one step after the other, each sequence to its own end
    batch, time, channels = case["batch"], case["time"], case["channels"]
    length = torch.full((batch,), time, device="cuda") if s["lengths"] is None else s["lengths"].long()
    out = torch.zeros(batch, time, channels, dtype=torch.float64, device="cuda")
    h = s["initial"].double()
    states = [h]

    def step(t):
        gate, x = s["gate"][:, t].double(), s["x"][:, t].double()
        if case["form"] == "decay":
            return gate, x, torch.ones_like(gate)
        return torch.sigmoid(gate), x, torch.sigmoid(-gate)
    for t in range(time):
        a, x, rest = step(t)
        here = torch.addcmul(rest * x, a, h)
        if s["lengths"] is not None:
            here = torch.where((t < length)[:, None], here, h)
            out[:, t] = torch.where((t < length)[:, None], here, out[:, t])
        else:
            out[:, t] = here
        h = here
        if op == "recurrence_grad":
            states.append(h)
    if op == "recurrence":
        return {"out": out, "final": h}
    gx, ggate = torch.zeros_like(out), torch.zeros_like(out)
    carry = s["grad_final"].double()
    for t in reversed(range(time)):
        a, x, rest = step(t)
        inside = (t < length)[:, None]
        total = torch.where(inside, carry + s["grad"][:, t].double(), torch.zeros_like(carry))
        if case["form"] == "decay":
            gx[:, t], ggate[:, t] = total, torch.where(inside, total * states[t], gx[:, t])
        else:
            gx[:, t] = torch.where(inside, total * rest, gx[:, t])
            ggate[:, t] = torch.where(inside, total * (states[t] - x) * a * rest, ggate[:, t])
        carry = torch.where(inside, a * total, carry)
    return {"x": gx, "gate": ggate, "initial": carry}
