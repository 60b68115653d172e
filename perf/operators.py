"""Operators of large language models that are measured: token log probabilities
(with their gradient), the learned relative position bias (with its gradient)
and the attention of one new token over a paged key-value cache.

Each case names its operator and sizes.  ``run`` computes it in elementary
torch operations, or with ``own`` through the library's own calls.
"""
import bisect
import math

import torch

own = False

_DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
_SIZE = {"f32": 4, "bf16": 2, "f16": 2}
_BLOCK = 1 << 26          # elements that the plain forms take at a time


# ---------------------------------------------------------------------------
# cases


def listed():
    return [
        # one new token of one sequence: the smallest call a server makes, with a few alternatives
        dict(name="logprobs_step", op="logprobs", rows=1, vocab=32768, dtype="bf16", top=5, masked=0.0, skipped=0.0),
        # a decoding batch under a grammar: half of each row is masked, 20 alternatives are reported
        dict(name="logprobs_batch", op="logprobs", rows=256, vocab=131072, dtype="bf16", top=20, masked=0.5, skipped=0.0),
        # scoring a training batch whose vocabulary is not padded: rows start at odd addresses, some tokens are padding
        dict(name="logprobs_train", op="logprobs", rows=4096, vocab=100003, dtype="bf16", top=0, masked=0.0, skipped=0.1),
        # the gradient of a loss over such log probabilities and the entropy, padded vocabulary
        dict(name="logprobs_grad", op="logprobs_grad", rows=4096, vocab=65536, dtype="bf16", masked=0.0, skipped=0.1),
        # the same in 32 bits with a ragged number of rows and an odd vocabulary
        dict(name="logprobs_grad_odd", op="logprobs_grad", rows=1021, vocab=100003, dtype="f32", masked=0.1, skipped=0.0),
        # the bias of one new token against its cache: latency
        dict(name="bias_step", op="bias", heads=32, q_len=1, k_len=4097, q_offset=4096, buckets=32, reach=128,
             both=False, dtype="f32"),
        # the bias of a whole sequence, made once per step and shared by the layers
        dict(name="bias_full", op="bias", heads=16, q_len=4096, k_len=4096, q_offset=0, buckets=32, reach=128,
             both=True, dtype="bf16"),
        # its gradient from the scores' gradient of a training batch
        dict(name="bias_grad", op="bias_grad", batch=8, heads=16, q_len=2048, k_len=2048, q_offset=0, buckets=32,
             reach=128, both=True, dtype="bf16"),
        # a small ragged batch in 32 bits: odd lengths, more keys than queries
        dict(name="bias_grad_odd", op="bias_grad", batch=3, heads=12, q_len=509, k_len=1531, q_offset=1022, buckets=64,
             reach=1024, both=False, dtype="f32"),
        # one sequence of ordinary length: latency
        dict(name="decode_one", op="decode", batch=1, heads=32, kv_heads=8, dim=128, longest=1000, page=16,
             dtype="bf16", bias=False),
        # few sequences with a long cache
        dict(name="decode_long", op="decode", batch=2, heads=32, kv_heads=8, dim=128, longest=131072, page=64,
             dtype="bf16", bias=False),
        # a serving batch of ragged lengths (one of them empty) with the learned bias
        dict(name="decode_batch", op="decode", batch=64, heads=32, kv_heads=4, dim=64, longest=8191, page=16,
             dtype="f16", bias=True),
    ]


_MOST_BYTES = 1_070_000_000      # no drawn case costs more than the largest listed ones


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    while True:
        op = rng.choice(["logprobs", "logprobs", "logprobs_grad", "bias", "bias_grad", "decode", "decode"])
        if op in ("logprobs", "logprobs_grad"):
            case = dict(op=op, rows=_log(rng, 1, 4096), vocab=_log(rng, 1000, 262144),
                        dtype=rng.choice(["bf16", "bf16", "f16", "f32"]), masked=rng.choice([0.0, 0.0, 0.1, 0.9]),
                        skipped=rng.choice([0.0, 0.1]))
            if rng.random() < 0.5:
                case["vocab"] = (case["vocab"] + 127) // 128 * 128
            if op == "logprobs":
                case["top"] = rng.choice([0, 1, 5, 20, 32])
        elif op in ("bias", "bias_grad"):
            q_len = rng.choice([1, _log(rng, 1, 4096), _log(rng, 64, 4096)])
            k_len = _log(rng, 16, 8192)
            if rng.random() < 0.5:
                q_len, k_len = (q_len + 7) // 8 * 8, (k_len + 7) // 8 * 8
            buckets = rng.choice([32, 64, 128])
            case = dict(op=op, heads=rng.choice([1, 8, 12, 16, 32]), q_len=q_len, k_len=k_len,
                        q_offset=max(0, k_len - q_len), buckets=buckets, reach=rng.choice([128, 500, 1024]),
                        both=rng.random() < 0.5, dtype=rng.choice(["bf16", "f16", "f32"]))
            if op == "bias_grad":
                case["batch"] = _log(rng, 1, 16)
        else:
            kv_heads = rng.choice([1, 2, 4, 8])
            case = dict(op=op, batch=_log(rng, 1, 128), heads=kv_heads * rng.choice([1, 2, 4, 7, 8, 16]),
                        kv_heads=kv_heads, dim=rng.choice([64, 128, 128, 256]), longest=_log(rng, 1, 131072),
                        page=rng.choice([8, 16, 24, 64, 256]), dtype=rng.choice(["bf16", "bf16", "f16"]),
                        bias=rng.random() < 0.3)
        if work(case)["bytes"] <= _MOST_BYTES:
            return case


# ---------------------------------------------------------------------------
# inputs


def _bounds(buckets, reach, both):
    """The least distance of each bucket after the first: single distances up to half of
    the buckets, then logarithmic steps up to ``reach``; from the integers alone."""
    n = buckets // 2 if both else buckets
    exact = max(n // 2, 1)
    steps = n - exact
    out = list(range(1, exact + 1))[: n - 1]
    for j in range(1, steps):
        # least d with log(d / exact) / log(reach / exact) * steps >= j
        goal = reach ** j * exact ** (steps - j)
        lo, hi = exact, max(reach, exact)
        while lo < hi:
            mid = (lo + hi) // 2
            lo, hi = (lo, mid) if mid ** steps >= goal else (mid + 1, hi)
        out.append(lo)
    return out


def _lengths(case, gen):
    if case["batch"] == 1:
        return [case["longest"]]
    n = (torch.rand(case["batch"], generator=gen) * case["longest"]).long().tolist()
    n[0] = case["longest"]
    if case["batch"] > 2:
        n[1] = 0                                    # a slot of the batch that holds no sequence
    return n


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)
    host = torch.Generator().manual_seed(seed)
    dt = _DTYPES[case["dtype"]]
    state = {"case": case}
    if case["op"] in ("logprobs", "logprobs_grad"):
        rows, vocab = case["rows"], case["vocab"]
        logits = torch.empty(rows, vocab, device=dev, dtype=dt)
        step = max(1, _BLOCK // vocab)
        for r in range(0, rows, step):
            x = torch.randn(min(step, rows - r), vocab, device=dev, generator=gen) * 2.5
            if case["masked"]:
                x.masked_fill_(torch.rand(x.shape, device=dev, generator=gen) < case["masked"], -math.inf)
            logits[r:r + step] = x.to(dt)
        tokens = torch.randint(0, vocab, (rows,), device=dev, generator=gen).to(torch.int32)
        logits[torch.arange(rows, device=dev), tokens.long()] = torch.randn(rows, device=dev, generator=gen).abs().to(dt) * 4
        skip = torch.rand(rows, device=dev, generator=gen) < case["skipped"]
        state.update(logits=logits, tokens=torch.where(skip, torch.full_like(tokens, -1), tokens))
        if case["op"] == "logprobs_grad":
            _, state["entropy"], state["lse"] = _plain_logprobs(logits, state["tokens"])
            state["g_logprob"] = torch.randn(rows, device=dev, generator=gen) / rows
            state["g_entropy"] = torch.randn(rows, device=dev, generator=gen) * (0.01 / rows)
    elif case["op"] in ("bias", "bias_grad"):
        bounds = _bounds(case["buckets"], case["reach"], case["both"])
        state["bounds"] = torch.tensor(bounds, dtype=torch.int32, device=dev)
        if case["op"] == "bias":
            state["table"] = torch.randn(case["buckets"], case["heads"], device=dev, generator=gen).to(dt)
        else:
            g = torch.empty(case["batch"], case["heads"], case["q_len"], case["k_len"], device=dev, dtype=dt)
            for b in range(case["batch"]):
                g[b] = (torch.randn(g.shape[1:], device=dev, generator=gen) * 1e-2).to(dt)
            state["grad"] = g
    else:
        page, hk, d = case["page"], case["kv_heads"], case["dim"]
        lengths = _lengths(case, host)
        used = [-(-n // page) for n in lengths]
        pages = sum(used) + 3
        order = torch.randperm(pages, generator=host)
        table = torch.full((case["batch"], max(1, max(used))), -1, dtype=torch.int32)
        at = 0
        for b, u in enumerate(used):
            table[b, :u] = order[at:at + u].int()
            at += u
        k = torch.randn(pages, page, hk, d, device=dev, generator=gen).to(dt)
        v = torch.randn(pages, page, hk, d, device=dev, generator=gen).to(dt)
        for b, (n, u) in enumerate(zip(lengths, used)):
            if n % page:                            # memory past a sequence's end has never been written
                k[int(table[b, u - 1]), n % page:] = math.nan
                v[int(table[b, u - 1]), n % page:] = math.nan
        state.update(k=k, v=v, table=table.to(dev), longest=max(lengths),
                     lengths=torch.tensor(lengths, dtype=torch.int32, device=dev),
                     host_lengths=lengths, q=torch.randn(case["batch"], case["heads"], d, device=dev, generator=gen).to(dt))
        if case["bias"]:
            state["bias_bounds"] = torch.tensor(_bounds(32, 128, False), dtype=torch.int32, device=dev)
            state["bias_table"] = torch.randn(32, case["heads"], device=dev, generator=gen)
    return state


# ---------------------------------------------------------------------------
# one pass


def run(state):
    case = state["case"]
    return (_run_own if own else _run_plain)(case["op"], case, state)


def _run_own(op, case, s):
    from deterministic_floating_point_gb300 import det
    if op == "logprobs":
        r = det.det_token_logprobs(s["logits"], s["tokens"], top_k=case["top"])
        out = {"logprob": r.logprob, "entropy": r.entropy, "lse": r.lse}
        if case["top"]:
            out.update(top_logprob=r.top_logprob, top_index=r.top_index)
        return out
    if op == "logprobs_grad":
        return det.det_token_logprobs_backward(s["logits"], s["tokens"], s["lse"], s["entropy"],
                                               grad_logprob=s["g_logprob"], grad_entropy=s["g_entropy"])
    if op == "bias":
        return det.det_relative_bias(s["table"], s["bounds"], case["q_len"], case["k_len"],
                                     q_offset=case["q_offset"], bidirectional=case["both"])
    if op == "bias_grad":
        return det.det_relative_bias_backward(s["grad"], s["bounds"], q_offset=case["q_offset"],
                                              bidirectional=case["both"])
    r = det.det_paged_attention(s["q"], s["k"], s["v"], s["table"], s["lengths"], max_len=s["longest"],
                                bias_table=s.get("bias_table"), bias_bounds=s.get("bias_bounds"))
    return {"out": r.out, "lse": r.lse}


def _plain_logprobs(logits, tokens):
    rows, vocab = logits.shape
    logprob, entropy, lse = (torch.empty(rows, device=logits.device) for _ in range(3))
    step = max(1, _BLOCK // vocab)
    for r in range(0, rows, step):
        x = logits[r:r + step].float()
        m = x.amax(1, keepdim=True)
        m = torch.where(m == -math.inf, torch.zeros_like(m), m)
        d = x - m
        e = torch.exp(d)
        z = e.sum(1)
        t = torch.where(e > 0, e * d, torch.zeros_like(e)).sum(1)
        lse[r:r + step] = m[:, 0] + torch.log(z)
        entropy[r:r + step] = torch.where(z > 0, torch.log(z) - t / z, torch.zeros_like(z))
        tok = tokens[r:r + step].long()
        ok = (tok >= 0) & (tok < vocab)
        at = x.gather(1, tok.clamp(0, vocab - 1)[:, None])[:, 0]
        logprob[r:r + step] = torch.where(ok, (at - m[:, 0]) - torch.log(z), torch.zeros_like(at))
    return logprob, entropy, lse


def _top(logits, k):
    """The k largest of each row, the lowest index first among equals."""
    rows, vocab = logits.shape
    index = torch.empty(rows, k, device=logits.device, dtype=torch.int32)
    behind = (vocab - 1) - torch.arange(vocab, device=logits.device)
    step = max(1, _BLOCK // vocab)
    for r in range(0, rows, step):
        bits = (logits[r:r + step].float() + 0.0).view(torch.int32).long()
        key = torch.where(bits >= 0, bits, -(bits & 0x7FFFFFFF)) * (1 << 32) + behind
        index[r:r + step] = (vocab - 1 - (key.topk(k, dim=1).values & 0xFFFFFFFF)).int()
    return index


def _buckets(case, bounds, dev):
    """The bucket of each (query, key) distance key - query, from the most negative one up."""
    rel = torch.arange(case["q_len"] + case["k_len"] - 1, device=dev) - (case["q_len"] - 1) - case["q_offset"]
    dist = rel.abs() if case["both"] else (-rel).clamp(min=0)
    bucket = (dist[:, None] >= bounds[None, :]).sum(1)
    return torch.where(rel > 0, bucket + bounds.numel() + 1, bucket) if case["both"] else bucket


def _run_plain(op, case, s):
    if op == "logprobs":
        logprob, entropy, lse = _plain_logprobs(s["logits"], s["tokens"])
        out = {"logprob": logprob, "entropy": entropy, "lse": lse}
        if case["top"]:
            out["top_index"] = _top(s["logits"], case["top"])
            out["top_logprob"] = s["logits"].gather(1, out["top_index"].long()).float() - lse[:, None]
        return out
    if op == "logprobs_grad":
        x, tok, vocab = s["logits"], s["tokens"].long(), case["vocab"]
        ok = (tok >= 0) & (tok < vocab)
        g = torch.where(ok, s["g_logprob"], torch.zeros_like(s["g_logprob"]))
        out = torch.empty_like(x)
        step = max(1, _BLOCK // vocab)
        for r in range(0, x.shape[0], step):
            sl = slice(r, r + step)
            lp = x[sl].float() - s["lse"][sl, None]
            p = torch.exp(lp)
            w = g[sl, None] + s["g_entropy"][sl, None] * (lp + s["entropy"][sl, None])
            d = torch.where(p > 0, -p * w, torch.zeros_like(p))
            d.scatter_add_(1, tok[sl, None].clamp(0, vocab - 1), g[sl, None])
            out[sl] = d.to(out.dtype)
        return out
    if op == "bias":
        bucket = _buckets(case, s["bounds"], s["table"].device)
        dev = s["table"].device
        at = torch.arange(case["k_len"], device=dev)[None, :] - torch.arange(case["q_len"], device=dev)[:, None]
        return s["table"].t()[:, bucket[at + case["q_len"] - 1]]
    if op == "bias_grad":
        g = s["grad"]
        dev, heads, q_len, k_len = g.device, case["heads"], case["q_len"], case["k_len"]
        bucket = _buckets(case, s["bounds"], dev)
        hot = (bucket[:, None] == torch.arange(case["buckets"], device=dev)).float()
        total = torch.zeros(heads, case["buckets"], device=dev)
        step = max(1, (_BLOCK >> 3) // (k_len * max(heads, case["buckets"])))
        for i in range(0, q_len, step):
            n = min(step, q_len - i)
            part = g[:, :, i:i + n].float().sum(0).reshape(heads, n * k_len)
            at = torch.arange(k_len, device=dev)[None, :] - torch.arange(i, i + n, device=dev)[:, None] + q_len - 1
            total += part @ hot[at.reshape(-1)]
        return total.t().contiguous()
    return _plain_decode(case, s)


def _plain_decode(case, s):
    group, page = case["heads"] // case["kv_heads"], case["page"]
    out = torch.zeros_like(s["q"])
    lse = torch.full(s["q"].shape[:2], -math.inf, device=out.device)
    for b, n in enumerate(s["host_lengths"]):
        if n == 0:
            continue
        pages = s["table"][b, : -(-n // page)].long()
        k = s["k"][pages].flatten(0, 1)[:n].float().transpose(0, 1)          # heads, tokens, dim
        v = s["v"][pages].flatten(0, 1)[:n].float().transpose(0, 1)
        q = s["q"][b].float().view(case["kv_heads"], group, case["dim"]) * case["dim"] ** -0.5
        x = q @ k.transpose(1, 2)
        if case["bias"]:
            dist = torch.arange(n - 1, -1, -1, device=out.device)
            bucket = (dist[:, None] >= s["bias_bounds"][None, :]).sum(1)
            x = x + s["bias_table"][bucket].t().reshape(case["kv_heads"], group, n)
        m = x.amax(2, keepdim=True)
        e = torch.exp(x - m)
        z = e.sum(2, keepdim=True)
        out[b] = ((e @ v) / z).to(out.dtype).flatten(0, 1)
        lse[b] = (m + torch.log(z)).flatten()
    return {"out": out, "lse": lse}


# ---------------------------------------------------------------------------
# what a pass cannot do without


def work(case):
    size = _SIZE[case["dtype"]]
    if case["op"] == "logprobs":
        n = case["rows"] * case["vocab"]
        return {"bytes": n * size + case["rows"] * (16 + 8 * case["top"]), "flops": 6 * n}
    if case["op"] == "logprobs_grad":
        n = case["rows"] * case["vocab"]
        return {"bytes": 2 * n * size + case["rows"] * 20, "flops": 6 * n}
    if case["op"] == "bias":
        n = case["heads"] * case["q_len"] * case["k_len"]
        return {"bytes": n * size + case["heads"] * case["buckets"] * size, "flops": 0}
    if case["op"] == "bias_grad":
        n = case["batch"] * case["heads"] * case["q_len"] * case["k_len"]
        return {"bytes": n * size + case["heads"] * case["buckets"] * 4, "flops": n}
    mean = case["longest"] if case["batch"] == 1 else (case["longest"] + case["longest"] / 2 * max(0, case["batch"] - 2))
    tokens = int(mean)
    return {"bytes": 2 * tokens * case["kv_heads"] * case["dim"] * size
            + 2 * case["batch"] * case["heads"] * case["dim"] * size,
            "flops": 4 * tokens * case["heads"] * case["dim"]}


# ---------------------------------------------------------------------------
# the definitions in 64 bits


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "logprobs":
        rows = []
        for r in range(case["rows"]):
            x = s["logits"][r].double()
            lse = torch.logsumexp(x, 0)
            lp = x - lse
            p = torch.exp(lp)
            tok = int(s["tokens"][r])
            none = torch.zeros((), dtype=torch.float64, device=x.device)
            row = [lp[tok] if tok >= 0 else none, torch.special.entr(p).sum(), lse]
            if case["top"]:
                order = torch.sort(x, descending=True, stable=True).indices[: case["top"]]
                row += [lp[order], order.int()]
            rows.append(row)
        names = ["logprob", "entropy", "lse", "top_logprob", "top_index"][: len(rows[0])]
        return {name: torch.stack(col) for name, col in zip(names, zip(*rows))}
    if case["op"] == "logprobs_grad":
        out = torch.empty(s["logits"].shape, dtype=torch.float64, device=s["logits"].device)
        for r in range(case["rows"]):
            lp = s["logits"][r].double() - s["lse"][r].double()
            p = torch.exp(lp)
            # p * lp has the limit 0 where p is 0
            out[r] = s["g_entropy"][r].double() * (torch.special.entr(p) - p * s["entropy"][r].double())
            tok = int(s["tokens"][r])
            if tok >= 0:
                out[r] -= s["g_logprob"][r].double() * p
                out[r, tok] += s["g_logprob"][r].double()
        return out
    if case["op"] in ("bias", "bias_grad"):
        bounds, q_len, k_len = s["bounds"].tolist(), case["q_len"], case["k_len"]

        def bucket(rel):
            if case["both"]:
                return bisect.bisect_right(bounds, abs(rel)) + (len(bounds) + 1 if rel > 0 else 0)
            return bisect.bisect_right(bounds, max(-rel, 0))

        of = torch.tensor([bucket(d - (q_len - 1) - case["q_offset"]) for d in range(q_len + k_len - 1)],
                          device=s["bounds"].device)
        if case["op"] == "bias":
            strip = s["table"].double()[of].t().contiguous()                 # heads, distances
            # row i of the result is the window of the strip that starts at q_len - 1 - i
            out = strip.unfold(1, k_len, 1).flip(1)
            return out.contiguous() if out.numel() <= 1 << 29 else None
        total = torch.zeros(case["buckets"], case["heads"], dtype=torch.float64, device=of.device)
        for h in range(case["heads"]):
            g = s["grad"][:, h].double().sum(0).flip(0)
            # row i of the flipped gradient moves i places to the right: its diagonals become columns
            g = torch.nn.functional.pad(g, (0, q_len)).flatten()[: q_len * (k_len + q_len - 1)]
            total[:, h].index_add_(0, of, g.view(q_len, k_len + q_len - 1).sum(0))
        return total
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=s["q"].device)
    lse = torch.full(s["q"].shape[:2], -math.inf, dtype=torch.float64, device=s["q"].device)
    group = case["heads"] // case["kv_heads"]
    for b, n in enumerate(s["host_lengths"]):
        at = torch.arange(n, device=out.device)
        page, slot = s["table"][b].long()[at // case["page"]], at % case["page"]
        for h in range(case["kv_heads"] if n else 0):
            hs = slice(h * group, (h + 1) * group)
            x = s["k"][page, slot, h].double() @ s["q"][b, hs].double().t() / math.sqrt(case["dim"])
            if case["bias"]:
                bucket = torch.bucketize(n - 1 - at, s["bias_bounds"].long(), right=True)
                x = x + s["bias_table"][:, hs].double()[bucket]
            lse[b, hs] = torch.logsumexp(x, 0)
            out[b, hs] = torch.softmax(x, 0).t() @ s["v"][page, slot, h].double()
    return {"out": out, "lse": lse}
