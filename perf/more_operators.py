"""Cases of the operators around a rounded layer's products: tokens sorted by expert and back with weights and
gradients, low-rank adapters of many requests beside a shared projection with their gradients, and the verification
of drafted tokens.

`own = False` computes the plain forms with elementary torch operations; `own = True` makes the calls of
`two_sided_gptq_amd.bakron`.  Weights are N(0, 0.02^2), activations N(0, 1) with a few channels of 20 times the size.
"""
import math

import torch

own = False

BLOCK = 128
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"f32": 4, "bf16": 2, "f16": 2}


def listed():
    return [
        # decoding a batch of 32 tokens, two experts of 64 each: the tokens sorted and copied by expert
        {"name": "dispatch_tokens", "op": "dispatch", "tokens": 32, "k": 2, "groups": 64, "cols": 1024, "skew": 0.5, "dropped": 0.0, "dtype": "bf16", "fp8": False},
        # prompts on their way into fp8 experts: sorted, rounded and copied 8 times
        {"name": "dispatch_prompt", "op": "dispatch", "tokens": 8192, "k": 8, "groups": 128, "cols": 4096, "skew": 0.5, "dropped": 0.0, "dtype": "bf16", "fp8": True},
        # a training batch in 16 bits, odd sizes, some of the tokens dropped by their experts
        {"name": "dispatch_train", "op": "dispatch", "tokens": 4099, "k": 4, "groups": 33, "cols": 2050, "skew": 1.0, "dropped": 0.1, "dtype": "f16", "fp8": False},
        # the way back of the decoded batch
        {"name": "combine_tokens", "op": "combine", "tokens": 32, "k": 2, "groups": 64, "cols": 2048, "skew": 0.5, "dropped": 0.0, "dtype": "bf16", "weighted": True, "grad": False},
        # the way back of prompts
        {"name": "combine_prompt", "op": "combine", "tokens": 8192, "k": 8, "groups": 128, "cols": 4096, "skew": 0.5, "dropped": 0.0, "dtype": "bf16", "weighted": True, "grad": False},
        # backward through a training batch's way back: gradients of the experts' outputs and of the weights
        {"name": "combine_grad", "op": "combine", "tokens": 4096, "k": 4, "groups": 16, "cols": 4096, "skew": 0.5, "dropped": 0.1, "dtype": "bf16", "weighted": True, "grad": True},
        # decoding one token each of 64 requests with adapters of their own, some without
        {"name": "adapter_tokens", "op": "adapter", "rows": 64, "n": 4096, "k": 4096, "rank": 16, "adapters": 64, "run": 1, "dtype": "bf16", "out": "same", "grad": False},
        # prompts of several requests through a wide projection with larger adapters
        {"name": "adapter_prompt", "op": "adapter", "rows": 8192, "n": 14336, "k": 4096, "rank": 64, "adapters": 8, "run": 1024, "dtype": "bf16", "out": "same", "grad": False},
        # training adapters beside a rounded layer
        {"name": "adapter_grad", "op": "adapter", "rows": 8192, "n": 4096, "k": 4096, "rank": 16, "adapters": 4, "run": 512, "dtype": "bf16", "out": "same", "grad": True},
        # small odd layers, an odd rank
        {"name": "adapter_grad_odd", "op": "adapter", "rows": 515, "n": 1000, "k": 520, "rank": 12, "adapters": 5, "run": 37, "dtype": "f16", "out": "same", "grad": True},
        # one request with 4 drafted tokens of a small vocabulary of odd size
        {"name": "verify_one", "op": "verify", "batch": 1, "drafts": 4, "vocab": 50001, "dtype": "f32", "draft": "model", "ragged": False},
        # a batch of requests with up to 5 drafted tokens each
        {"name": "verify_batch", "op": "verify", "batch": 128, "drafts": 5, "vocab": 131072, "dtype": "f32", "draft": "model", "ragged": True},
    ]


def _spread(rng, low, high, step=1):
    """A size spread over its logarithm, a multiple of `step`."""
    v = math.exp(rng.uniform(math.log(low), math.log(high)))
    return max(step, int(round(v / step)) * step)


def draw(rng):
    op = rng.choice(["dispatch", "combine", "combine", "adapter", "adapter", "verify"])
    if op in ("dispatch", "combine"):
        k = rng.choice([1, 2, 4, 6, 8])
        cols = _spread(rng, 64, 14336, rng.choice([16, 16, 16, 1]))
        dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
        grad = op == "combine" and rng.random() < 0.5
        tokens = _spread(rng, 1, min(16384, (1 << (27 if grad else 28)) // (k * cols * SIZE[dtype])))
        case = {"op": op, "tokens": tokens, "k": k, "groups": _spread(rng, k + 1, 512), "cols": cols, "skew": round(rng.uniform(0, 1.5), 2),
                "dropped": rng.choice([0.0, 0.0, 0.05, 0.3]), "dtype": dtype}
        if op == "dispatch":
            return case | {"fp8": rng.random() < 0.5}
        # without weights the way back is the gradient of the copies
        return case | {"weighted": grad or rng.random() < 0.7, "grad": grad}
    if op == "adapter":
        step = rng.choice([16, 16, 16, 1])
        n, k = _spread(rng, 64, 14336, step), _spread(rng, 64, 14336, step)
        rank = rng.choice([4, 8, 16, 16, 32, 64, 128, _spread(rng, 1, 128)])
        rows = _spread(rng, 1, min(16384, (1 << 26) // (n + k)))
        adapters = max(1, min(_spread(rng, 1, 128), (1 << 26) // (rank * (n + k))))
        return {"op": op, "rows": rows, "n": n, "k": k, "rank": rank, "adapters": adapters, "run": _spread(rng, 1, max(2, rows // 2)),
                "dtype": rng.choice(["bf16", "bf16", "f16"]), "out": rng.choice(["same", "same", "f32"]), "grad": rng.random() < 0.4}
    drafts, vocab = rng.choice([1, 2, 3, 4, 5, 8]), _spread(rng, 1000, 131072, rng.choice([1, 64]))
    return {"op": op, "batch": _spread(rng, 1, min(256, (1 << 27) // (vocab * (2 * drafts + 1)))), "drafts": drafts, "vocab": vocab,
            "dtype": rng.choice(["f32", "f32", "bf16", "f16"]), "draft": rng.choice(["model", "model", "none"]), "ragged": rng.random() < 0.5}


def _activations(rows, cols, gen):
    x = torch.randn(rows, cols, device="cuda", generator=gen)
    loud = torch.randint(0, cols, (max(1, cols // 128),), device="cuda", generator=gen)
    x[:, loud] *= 20.0
    return x


def _routing(case, gen):
    """Each token's k experts, all different: the largest of random scores around shares that fall as 1 / rank^skew.
    A dropped choice has the number -1."""
    groups, tokens = case["groups"], case["tokens"]
    share = torch.arange(1, groups + 1, device="cuda").float().log_().mul_(-case["skew"])
    share = share[torch.randperm(groups, device="cuda", generator=gen)]
    noise = torch.rand(tokens, groups, device="cuda", generator=gen).clamp_(min=1e-9)
    ids = torch.topk(share - (-noise.log()).log(), case["k"], dim=1).indices
    if case["dropped"]:
        ids[torch.rand(tokens, case["k"], device="cuda", generator=gen) < case["dropped"]] = -1
    return ids


def _by_group(ids, groups):
    """(offsets, order, slots) of group numbers, as group_sort gives them: a stable sort, rows of no group last."""
    key = torch.where(ids.flatten() < 0, groups, ids.flatten())
    order = torch.sort(key, stable=True).indices
    slots = torch.empty_like(order)
    slots[order] = torch.arange(order.numel(), device=order.device)
    offsets = torch.zeros(groups + 1, dtype=torch.int32, device=order.device)
    offsets[1:] = torch.bincount(key, minlength=groups + 1)[:groups].cumsum(0)
    return offsets, order.to(torch.int32), slots.to(torch.int32).view(ids.shape)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op = case["op"]
    if op == "dispatch":
        ids = _routing(case, gen)
        return {"case": case, "ids": ids, "x": _activations(case["tokens"], case["cols"], gen).to(DTYPES[case["dtype"]])}
    if op == "combine":
        t = DTYPES[case["dtype"]]
        ids = _routing(case, gen)
        offsets, _, slots = _by_group(ids, case["groups"])
        y = torch.randn(ids.numel(), case["cols"], device="cuda", generator=gen).to(t)
        state = {"case": case, "offsets": offsets, "slots": slots, "y": y, "weights": None, "kept": ids >= 0}
        if case["weighted"]:
            state["weights"] = torch.randn(ids.shape, device="cuda", generator=gen).softmax(1)
        if case["grad"]:
            state["dout"] = torch.randn(case["tokens"], case["cols"], device="cuda", generator=gen).mul_(0.1).to(t)
        return state
    if op == "adapter":
        t, rows, n, k, rank, adapters = DTYPES[case["dtype"]], case["rows"], case["n"], case["k"], case["rank"], case["adapters"]
        out = t if case["out"] == "same" else torch.float32
        # requests of `run` rows each; about one in eight has no adapter
        runs = -(-rows // case["run"])
        of = torch.randint(0, adapters, (runs,), device="cuda", generator=gen)
        of[torch.rand(runs, device="cuda", generator=gen) < 0.125] = -1
        ids = of.repeat_interleave(case["run"])[:rows]
        offsets, order, _ = _by_group(ids, adapters)
        state = {"case": case, "ids": ids, "offsets": offsets, "order": order, "x": _activations(rows, k, gen).to(t),
                 "a": torch.randn(adapters, rank, k, device="cuda", generator=gen).mul_(k ** -0.5).to(t),
                 "b": torch.randn(adapters, n, rank, device="cuda", generator=gen).mul_(0.02).to(t),
                 "scale": torch.rand(adapters, device="cuda", generator=gen).add_(0.5)}
        if case["grad"]:
            state["dy"] = torch.randn(rows, n, device="cuda", generator=gen).mul_(0.1).to(t)
            state["base"] = torch.randn(rows, k, device="cuda", generator=gen).mul_(0.1).to(out)
        else:
            state["base"] = torch.randn(rows, n, device="cuda", generator=gen).to(out)
        state["counts"] = torch.diff(offsets).tolist()
        return state
    batch, drafts, vocab, t = case["batch"], case["drafts"], case["vocab"], DTYPES[case["dtype"]]
    x = torch.randn(batch, drafts + 1, vocab, device="cuda", generator=gen).mul_(2.0)
    # a few likely tokens in each row
    likely = torch.randint(0, vocab, (batch, drafts + 1, 8), device="cuda", generator=gen)
    x.scatter_add_(2, likely, torch.rand(likely.shape, device="cuda", generator=gen).mul_(12.0))
    p = x.softmax(2)
    if case["draft"] == "model":  # a draft whose logits differ a little from the target's
        y = x[:, :drafts].add_(torch.randn(batch, drafts, vocab, device="cuda", generator=gen), alpha=0.4)
        q = y.softmax(2)
        chosen = torch.multinomial(q.reshape(-1, vocab), 1, generator=gen).view(batch, drafts)
        q = q.to(t)
    else:  # drafts looked up in the text: no distribution
        q, chosen = None, likely[:, :drafts, 0].clone()
    if case["ragged"]:
        count = torch.randint(0, drafts + 1, (batch,), device="cuda", generator=gen)
        chosen[torch.arange(drafts, device="cuda") >= count[:, None]] = -1
    return {"case": case, "p": p.to(t), "q": q, "drafts": chosen,
            "u": torch.rand(batch, drafts, device="cuda", generator=gen), "v": torch.rand(batch, device="cuda", generator=gen)}


def _plain_dispatch(state):
    case, x = state["case"], state["x"]
    offsets, order, slots = _by_group(state["ids"], case["groups"])
    out = {"offsets": offsets, "order": order, "slots": slots}
    kept = (torch.arange(order.numel(), device=order.device) < offsets[-1])[:, None]
    token = order.long() // case["k"]
    if not case["fp8"]:
        return out | {"rows": torch.where(kept, x[token], 0.0)}
    rows, cols = x.shape
    kb = -(-cols // BLOCK)
    full = torch.zeros(rows, kb * BLOCK, device=x.device)
    full[:, :cols] = x
    full = full.view(rows, kb, BLOCK)
    amax = full.abs().amax(2)
    amax = torch.where(amax > 0, amax.clamp(min=2.0 ** -100), 448.0)  # a block of zeros has the scale 1
    q = (full * (448.0 / amax)[:, :, None]).clamp(-448.0, 448.0).view(rows, -1)[:, :cols].to(torch.float8_e4m3fn)
    q = torch.where(kept, q.view(torch.uint8)[token], 0).view(torch.float8_e4m3fn)
    scales = torch.where(kept, (amax / 448.0)[token], 1.0)
    return out | {"rows": q, "scales": scales.t().contiguous()}


def _plain_combine(state):
    y, slots, kept = state["y"].float(), state["slots"].long(), state["kept"]
    if not state["case"]["grad"]:
        rows = torch.where(kept[:, :, None], y[slots], 0.0)
        if state["weights"] is not None:
            rows = rows * state["weights"][:, :, None]
        return rows.sum(1).to(state["y"].dtype)
    dout, w = state["dout"].float(), torch.where(kept, state["weights"], 0.0)
    dy = torch.empty_like(y)
    dy[slots.flatten()] = (w[:, :, None] * dout[:, None, :]).flatten(0, 1)
    dw = torch.where(kept, (dout[:, None, :] * y[slots]).sum(2), 0.0)
    return {"dy": dy.to(state["y"].dtype), "dw": dw}


def _plain_adapter(state):
    case = state["case"]
    x, order, counts, base = state["x"].float(), state["order"].long(), state["counts"], state["base"]
    out = base.float()
    if case["grad"]:
        dy, da, db = state["dy"].float(), torch.zeros_like(state["a"]), torch.zeros_like(state["b"])
    at = 0
    for g, count in enumerate(counts):
        if count == 0:
            continue
        rows, at = order[at:at + count], at + count
        a, b, s = state["a"][g].float(), state["b"][g].float(), state["scale"][g]
        if not case["grad"]:
            out[rows] += s * ((x[rows] @ a.t()) @ b.t())
            continue
        u, p = s * (dy[rows] @ b), s * (x[rows] @ a.t())
        out[rows] += u @ a
        da[g] = u.t() @ x[rows]
        db[g] = dy[rows].t() @ p
    out = out.to(base.dtype)
    return {"dx": out, "da": da, "db": db} if case["grad"] else out


def _plain_verify(state):
    case, p, q, d = state["case"], state["p"], state["q"], state["drafts"]
    batch, drafts, vocab = case["batch"], case["drafts"], case["vocab"]
    # in 64 bits: the product of two 32-bit numbers and the sums over a vocabulary lie next to borders
    at = d.clamp(min=0)[:, :, None]
    pd = p[:, :drafts].gather(2, at).squeeze(2).double()
    qd = 1.0 if q is None else q.gather(2, at).squeeze(2).double()
    good = (d >= 0) & (state["u"].double() * qd < pd)
    accepted = good.long().cumprod(1).sum(1)
    each = torch.arange(batch, device=p.device)
    last = accepted.clamp(max=max(drafts - 1, 0))
    refused = (accepted < drafts) & (d[each, last] >= 0)
    row = p[each, accepted].double()
    if q is None:
        rest = row.scatter(1, d[each, last].clamp(min=0)[:, None], 0.0)
    else:
        rest = (row - q[each, last].double()).clamp(min=0.0)
    rest = torch.where(refused[:, None], rest, row)
    rest = torch.where(rest.sum(1, keepdim=True) > 0, rest, row)
    sums = rest.cumsum(1)
    token = (sums <= state["v"].double()[:, None] * sums[:, -1:]).sum(1).clamp(max=vocab - 1)
    place = torch.arange(drafts + 1, device=p.device)
    tokens = torch.cat([d, d.new_full((batch, 1), -1)], 1)
    tokens = torch.where(place < accepted[:, None], tokens, -1)
    tokens[each, accepted] = token
    return {"accepted": accepted.to(torch.int32), "tokens": tokens}


def run(state):
    case, op = state["case"], state["case"]["op"]
    if own:
        from two_sided_gptq_amd import bakron
        if op == "dispatch":
            offsets, order, slots = bakron.group_sort(state["ids"], case["groups"])
            out = {"offsets": offsets, "order": order, "slots": slots}
            if case["fp8"]:
                rows, scales = bakron.group_gather_fp8(state["x"], slots, offsets)
                return out | {"rows": rows, "scales": scales}
            return out | {"rows": bakron.group_gather(state["x"], slots, offsets)}
        if op == "combine":
            if case["grad"]:
                dy, dw = bakron.group_combine_grad(state["dout"], state["y"], state["slots"], state["offsets"], state["weights"])
                return {"dy": dy, "dw": dw}
            return bakron.group_combine(state["y"], state["slots"], state["offsets"], state["weights"])
        if op == "adapter":
            if case["grad"]:
                dx, da, db = bakron.adapter_matmul_grad(state["dy"], state["x"], state["a"], state["b"], state["offsets"],
                                                        state["order"], state["scale"], base=state["base"])
                return {"dx": dx, "da": da, "db": db}
            return bakron.adapter_matmul(state["x"], state["a"], state["b"], state["offsets"], state["order"], state["scale"],
                                         base=state["base"])
        accepted, tokens = bakron.verify_drafts(state["p"], state["q"], state["drafts"], state["u"], state["v"])
        return {"accepted": accepted, "tokens": tokens}
    return {"dispatch": _plain_dispatch, "combine": _plain_combine, "adapter": _plain_adapter, "verify": _plain_verify}[op](state)


def work(case):
    op = case["op"]
    if op in ("dispatch", "combine"):
        e, b, pairs = case["tokens"] * case["cols"], SIZE[case["dtype"]], case["tokens"] * case["k"]
        if op == "dispatch":
            copies = pairs * case["cols"] * (1 if case["fp8"] else b) + (4 * pairs * -(-case["cols"] // BLOCK) if case["fp8"] else 0)
            return {"bytes": 16 * pairs + 4 * case["groups"] + e * b + copies, "flops": 3 * e if case["fp8"] else 0}
        kept = pairs * (1 - case["dropped"]) * case["cols"]
        if case["grad"]:  # dout and Y read, all of dY written
            return {"bytes": 12 * pairs + b * (e + kept + pairs * case["cols"]), "flops": 3 * kept}
        return {"bytes": (8 if case["weighted"] else 4) * pairs + b * (e + kept), "flops": 2 * kept}
    if op == "adapter":
        rows, n, k, rank, b = case["rows"], case["n"], case["k"], case["rank"], SIZE[case["dtype"]]
        o = b if case["out"] == "same" else 4
        with_one = 0.875 * rows
        used = case["adapters"] * (1 - (1 - 0.875 / case["adapters"]) ** -(-rows // case["run"]))
        weights = used * rank * (n + k) * b
        if case["grad"]:
            return {"bytes": with_one * (n + k) * b + 2 * rows * k * o + weights + case["adapters"] * rank * (n + k) * b,
                    "flops": 2 * with_one * rank * (3 * k + 2 * n)}
        return {"bytes": with_one * k * b + 2 * rows * n * o + weights, "flops": 2 * with_one * rank * (n + k)}
    # one row of the target's probabilities a request, and the draft's where one was refused
    rows = 1 + (0.7 if case["draft"] == "model" else 0)
    e = case["batch"] * case["vocab"] * rows
    return {"bytes": e * SIZE[case["dtype"]] + case["batch"] * (16 + 28 * case["drafts"]), "flops": 2 * e}


def exact(case, seed):
    """The same outputs from their definitions in 64 bits."""
    state, op = prepare(case, seed), case["op"]
    if op == "dispatch":
        x, ids, groups = state["x"].double(), state["ids"].flatten(), case["groups"]
        members = [(ids == g).nonzero().squeeze(1) for g in range(groups)]
        offsets = [0]
        for m in members:
            offsets.append(offsets[-1] + m.numel())
        order = torch.cat([*members, (ids < 0).nonzero().squeeze(1)])
        slots = torch.argsort(order).view(state["ids"].shape)
        out = {"offsets": torch.tensor(offsets, device="cuda", dtype=torch.int32), "order": order.to(torch.int32), "slots": slots.to(torch.int32)}
        n, end = order.numel(), offsets[-1]
        source = order[:end] // case["k"]
        rows = torch.zeros(n, case["cols"], device="cuda", dtype=torch.float64)
        if not case["fp8"]:
            rows[:end] = x[source]
            return out | {"rows": rows}
        scales = torch.ones(-(-case["cols"] // BLOCK), n, device="cuda", dtype=torch.float64)
        for b in range(scales.shape[0]):
            part = x[:, b * BLOCK:(b + 1) * BLOCK]
            amax = part.abs().max(1).values
            s = torch.where(amax == 0, 1.0, amax.clamp(min=2.0 ** -100) / 448)
            scales[b, :end] = s[source]
            rows[:end, b * BLOCK:(b + 1) * BLOCK] = (part / s[:, None])[source]
        return out | {"rows": rows, "scales": scales}
    if op == "combine":
        y, slots, kept = state["y"], state["slots"].long(), state["kept"]
        if not case["grad"]:
            total = torch.zeros(case["tokens"], case["cols"], device="cuda", dtype=torch.float64)
            for j in range(case["k"]):
                w = kept[:, j].double() if state["weights"] is None else kept[:, j] * state["weights"][:, j].double()
                total += w[:, None] * y[slots[:, j]].double()
            return total
        dout = state["dout"].double()
        dy = torch.zeros(y.shape, device="cuda", dtype=torch.float64)
        dw = torch.zeros(slots.shape, device="cuda", dtype=torch.float64)
        for j in range(case["k"]):
            token = kept[:, j].nonzero().squeeze(1)
            at = slots[token, j]
            dy[at] = state["weights"][token, j].double()[:, None] * dout[token]
            dw[token, j] = (dout[token] * y[at].double()).sum(1)
        return {"dy": dy, "dw": dw}
    if op == "adapter":
        x, a, b, s = state["x"].double(), state["a"].double(), state["b"].double(), state["scale"].double()
        out = state["base"].double()
        da, db = torch.zeros_like(a), torch.zeros_like(b)
        for g in range(case["adapters"]):
            mine = (state["ids"] == g).nonzero().squeeze(1)
            if mine.numel() == 0:
                continue
            whole = s[g] * (b[g] @ a[g]) if not case["grad"] and mine.numel() > case["n"] else None
            if not case["grad"]:
                out[mine] += x[mine] @ whole.t() if whole is not None else x[mine] @ a[g].t() @ (s[g] * b[g]).t()
                continue
            dy = state["dy"][mine].double() * s[g]
            out[mine] += dy @ b[g] @ a[g]
            da[g] = (dy @ b[g]).t() @ x[mine]
            db[g] = dy.t() @ (x[mine] @ a[g].t())
        return {"dx": out, "da": da, "db": db} if case["grad"] else out
    p, q, d, u, v = (t.cpu() if t is not None else None for t in (state["p"], state["q"], state["drafts"], state["u"].double(), state["v"].double()))
    accepted, tokens = [], torch.full((case["batch"], case["drafts"] + 1), -1, dtype=torch.int64)
    for r in range(case["batch"]):
        n, rest = 0, None
        while n < case["drafts"] and d[r, n] >= 0:
            t = int(d[r, n])
            if not float(u[r, n]) * (1.0 if q is None else float(q[r, n, t])) < float(p[r, n, t]):
                rest = p[r, n].double()
                if q is None:
                    rest[t] = 0.0
                else:
                    rest = torch.maximum(rest - q[r, n].double(), torch.zeros((), dtype=torch.float64))
                break
            tokens[r, n] = t
            n += 1
        if rest is None or not float(rest.sum()) > 0:
            rest = p[r, n].double()
        sums = rest.cumsum(0)
        tokens[r, n] = torch.searchsorted(sums, v[r] * sums[-1], right=True).clamp(max=case["vocab"] - 1)
        accepted.append(n)
    return {"accepted": torch.tensor(accepted, dtype=torch.int32, device="cuda"), "tokens": tokens.cuda()}
