"""Cases of a layer's other parts as calls: products with 4-bit matrices, tokens sorted by expert and back, and the norms
around a block with its gate and residual.

``run`` computes a case in plain torch operations, or with ``own`` through the library's binding.
"""
import math
import types

import numpy as np
import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "f16": 2, "bf16": 2}
BLOCK = 32  # weights to a scale and a min


# --- cases ---------------------------------------------------------------------------------------------------


def listed():
    return [
        # one token through a query projection
        {"name": "linear token", "op": "linear", "rows": 1, "n": 1, "in": 2048, "out": 4096, "glu": False,
         "spread": 0.0, "dtype": "bf16"},
        # the output projection of a verify window's rows
        {"name": "linear window", "op": "linear", "rows": 8, "n": 1, "in": 4096, "out": 2048, "glu": False,
         "spread": 0.0, "dtype": "f32"},
        # a chunk of a prompt between decode steps, gate and up of a dense block
        {"name": "linear chunk", "op": "linear", "rows": 203, "n": 1, "in": 2048, "out": 4096, "glu": True,
         "spread": 0.0, "dtype": "f16"},
        # a prompt's q, k and v in one product
        {"name": "linear prompt", "op": "linear", "rows": 8191, "n": 1, "in": 2048, "out": 5120, "glu": False,
         "spread": 0.0, "dtype": "bf16"},
        # a shorter prompt's output projection on the f32 residual stream
        {"name": "linear prompt f32", "op": "linear", "rows": 2041, "n": 1, "in": 4096, "out": 2048, "glu": False,
         "spread": 0.0, "dtype": "f32"},
        # gate and up of 128 experts for a prompt's rows sorted by expert, some experts asked for far more than others
        {"name": "linear experts", "op": "linear", "rows": 32760, "n": 128, "in": 2048, "out": 768, "glu": True,
         "spread": 0.5, "dtype": "bf16"},
        # a batch of decode rows: the router's choice, then the rows in the experts' order
        {"name": "sort batch", "op": "sort", "rows": 64, "experts": 128, "top_k": 8, "hidden": 2048, "renorm": True,
         "out": 0.0, "dtype": "f32"},
        # a prompt, padded: some rows are no one's
        {"name": "sort prompt", "op": "sort", "rows": 8191, "experts": 128, "top_k": 8, "hidden": 2048,
         "renorm": False, "out": 0.03, "dtype": "bf16"},
        # the experts' results back to their rows, weighted, on top of the shared expert's
        {"name": "back prompt", "op": "back", "rows": 8191, "experts": 128, "top_k": 8, "hidden": 2048, "base": True,
         "out": 0.03, "dtype": "bf16"},
        # its gradient for the experts' results and the weights
        {"name": "back gradient", "op": "back_grad", "rows": 2047, "experts": 160, "top_k": 8, "hidden": 4096,
         "base": False, "out": 0.0, "dtype": "f32"},
        # between a window's attention and its MoE half
        {"name": "norm window", "op": "norm", "rows": 8, "hidden": 2048, "after": False, "gate": "none",
         "sigmoid": False, "before": True, "dtype": "f32"},
        # a prompt between two blocks: normed after the block, gated by channel, added, normed before the next
        {"name": "norm prompt", "op": "norm", "rows": 8191, "hidden": 4096, "after": True, "gate": "channel",
         "sigmoid": False, "before": True, "dtype": "bf16"},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["linear", "linear", "linear", "sort", "back", "back_grad", "norm"])
    dtype = rng.choice(["f32", "f16", "bf16"])
    if op == "linear":
        n = rng.choice([1, 1, 1, 8, 40, 128])
        d, out = 64 * _log(rng, 1, 64), 16 * _log(rng, 1, 256)
        glu = rng.random() < 0.4
        most = 30e9 if dtype == "f32" else 100e9  # multiplications of a call
        rows = _log(rng, 1, max(1, min(20000, int(most / (d * out * (2 if glu else 1))))))
        while n * d * out > 2.0e8:
            n = max(1, n // 4)
        return {"op": op, "rows": rows, "n": n, "in": d, "out": out, "glu": glu,
                "spread": round(rng.uniform(0, 1), 2) if n > 1 else 0.0, "dtype": dtype}
    if op == "norm":
        return {"op": op, "rows": _log(rng, 1, 6000), "hidden": 8 * _log(rng, 1, 1024), "after": rng.random() < 0.5,
                "gate": rng.choice(["none", "channel", "row", "element"]), "sigmoid": rng.random() < 0.4,
                "before": rng.random() < 0.8, "dtype": dtype}
    experts = rng.choice([4, 8, 60, 128, 160, 256, 384])
    case = {"op": op, "experts": experts, "top_k": rng.choice([k for k in (1, 2, 3, 4, 6, 8) if k <= experts]),
            "hidden": 8 * _log(rng, 8, 512), "out": rng.choice([0.0, 0.0, 0.1, 0.9]), "dtype": dtype}
    case["rows"] = _log(rng, 1, max(1, min(12000, 60000000 // (case["top_k"] * case["hidden"]))))
    if op == "sort":
        return {**case, "renorm": rng.random() < 0.5}
    return {**case, "base": op == "back" and rng.random() < 0.5}


def _counts(case):
    """Rows of each matrix, from the case alone: they fall off as rank ** -spread, in a scattered order; the last of many
    rows are no one's."""
    n, live = case["n"], case["rows"] - (case["rows"] // 50 if case["n"] > 1 else 0)
    share = np.array([(1.0 + (i * 37) % n) ** -case["spread"] for i in range(n)])
    upto = np.rint(live * np.cumsum(share) / share.sum()).astype(int)
    return np.diff(upto, prepend=0).tolist()


def work(case):
    z, T = SIZE[case["dtype"]], case["rows"]
    if case["op"] == "linear":
        counts, mats = _counts(case), 2 if case["glu"] else 1
        live = sum(counts)
        weights = sum(c > 0 for c in counts) * mats * case["in"] * case["out"]
        return {"bytes": weights * 5 // 8 + live * (case["in"] + case["out"]) * z,
                "flops": 2 * live * mats * case["in"] * case["out"]}
    if case["op"] == "norm":
        n = T * case["hidden"]
        arrays = 3 + case["before"] + (case["gate"] == "element")
        return {"bytes": arrays * n * z, "flops": 12 * n}
    d, E, live = case["hidden"], case["experts"], max(1, int(T * (1 - case["out"])))
    entries = live * case["top_k"]
    if case["op"] == "sort":
        return {"bytes": T * E * 4 + T * case["top_k"] * 16 + E * 8 + (live + entries) * d * z, "flops": 4 * T * E}
    if case["op"] == "back":
        return {"bytes": T * case["top_k"] * 8 + (entries + T * (2 if case["base"] else 1)) * d * z,
                "flops": 2 * entries * d}
    return {"bytes": T * case["top_k"] * 12 + (2 * entries + T) * d * z, "flops": 3 * entries * d}


# --- inputs --------------------------------------------------------------------------------------------------


def _values(g, shape, dtype, spread):
    """Normal values whose size varies from row to row and from channel to channel, as activations do."""
    x = torch.randn(shape, generator=g, device="cuda")
    x *= torch.exp2(spread * torch.randn(shape[:-1] + (1,), generator=g, device="cuda"))
    x *= torch.exp2(0.5 * torch.randn(shape[-1], generator=g, device="cuda"))
    return x.to(dtype)


def _quantized(g, n, rows, cols):
    """A stack of N(0, 0.02) matrices in blocks of 32: 4-bit codes, the even element in the low nibble, an f16 scale and
    an f16 min (bit patterns)."""
    codes = torch.empty(n, rows, cols // 2, dtype=torch.uint8, device="cuda")
    scale, low = (torch.empty(n, rows, cols // BLOCK, dtype=torch.float16, device="cuda") for _ in range(2))
    step = max(1, 50000000 // (rows * cols))
    for i in range(0, n, step):
        w = 0.02 * torch.randn(min(step, n - i), rows, cols // BLOCK, BLOCK, generator=g, device="cuda")
        m = w.amin(-1).half()
        s = ((w.amax(-1) - m) / 15).half()
        q = torch.round((w - m.float()[..., None]) / s.float()[..., None]).clamp_(0, 15).to(torch.uint8)
        q = q.view(-1, rows, cols // 2, 2)
        codes[i:i + step] = q[..., 0] | q[..., 1] << 4
        scale[i:i + step], low[i:i + step] = s, m
    return types.SimpleNamespace(codes=codes, scale=scale.view(torch.int16), min=low.view(torch.int16), rows=rows,
                                 cols=cols, bits=4, block=BLOCK)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed * 2654435761 % (1 << 62))
    dt, T = DTYPES[case["dtype"]], case["rows"]
    s = {"case": case}
    if case["op"] == "linear":
        n = case["n"]
        s["w"] = _quantized(g, n, case["out"], case["in"])
        s["up"] = _quantized(g, n, case["out"], case["in"]) if case["glu"] else None
        s["x"] = _values(g, (T, case["in"]), dt, 0.7)
        counts = _counts(case)
        s["most"], s["live"] = max(counts), sum(counts)
        s["offsets"] = torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32, device="cuda")
        s["y"] = torch.zeros(T, case["out"], dtype=dt, device="cuda")
        if own:
            from slot_decode_window_gb300 import binding
            s["handle"] = binding.Linear(s["w"], up=s["up"], max_rows=T)
        return s
    if case["op"] == "norm":
        d = case["hidden"]
        s["x"], s["y"] = _values(g, (T, d), dt, 0.3), _values(g, (T, d), dt, 1.0)
        s["after"] = 1 + 0.3 * torch.randn(d, generator=g, device="cuda") if case["after"] else None
        s["before"] = 1 + 0.3 * torch.randn(d, generator=g, device="cuda") if case["before"] else None
        s["gate"] = {"none": lambda: None, "channel": lambda: torch.randn(d, generator=g, device="cuda"),
                     "row": lambda: torch.randn(T, generator=g, device="cuda"),
                     "element": lambda: torch.randn(T, d, generator=g, device="cuda").to(dt)}[case["gate"]]()
        if own:
            from slot_decode_window_gb300 import binding
            s["handle"] = binding.BlockNorm(d, after=s["after"], before=s["before"], gate=case["gate"],
                                            channel_gate=s["gate"] if case["gate"] == "channel" else None,
                                            sigmoid=case["sigmoid"], residual_scale=0.9, block_scale=1.25, eps=1e-6)
        return s
    E, k, d = case["experts"], case["top_k"], case["hidden"]
    gone = torch.rand(T, generator=g, device="cuda") < case["out"]  # rows that are no one's
    logits = 1.5 * torch.randn(T, E, generator=g, device="cuda") + torch.randn(E, generator=g, device="cuda")
    # a grid of values that a softmax's sum keeps exactly apart, so that equal logits are met and must go to the lower expert
    s["logits"] = torch.where(gone[:, None], -math.inf, torch.round(logits * 4096) / 4096)
    if own:
        from slot_decode_window_gb300 import binding
        s["handle"] = binding.ExpertSort(E, k, renorm=case.get("renorm", False))
    if case["op"] == "sort":
        s["x"] = _values(g, (T, d), dt, 0.7)
        s["xs"] = torch.zeros(T * k, d, dtype=dt, device="cuda")  # rows behind the last expert's stay
        return s
    idx, w = _plain_route(s["logits"], k, False)
    s["w"] = w
    s["offsets"], s["entries"], s["place"] = _plain_plan(idx, E)
    s["z"] = _values(g, (T * k, d), dt, 0.7)
    if case["base"]:
        s["base"] = _values(g, (T, d), dt, 0.7)
    if case["op"] == "back_grad":
        s["dy"] = _values(g, (T, d), dt, 0.7)
        s["dz"] = torch.zeros(T * k, d, dtype=dt, device="cuda")
    if own:
        s["plan"] = s["handle"].plan(idx)
    return s


# --- plain forms ---------------------------------------------------------------------------------------------


def _dequantized(w):
    """[n][rows][cols] in f32."""
    q = torch.stack((w.codes & 15, w.codes >> 4), -1).view(*w.codes.shape[:2], -1, BLOCK).float()
    q = q * w.scale.view(torch.float16).float()[..., None] + w.min.view(torch.float16).float()[..., None]
    return q.flatten(-2)


def _plain_linear(s):
    case, n, y = s["case"], s["case"]["n"], s["y"]
    x = s["x"].float()
    if n > 1:  # each matrix's rows, padded to the most that one has
        i = torch.arange(s["most"], device="cuda")
        at = s["offsets"][:-1, None] + i
        mine = at < s["offsets"][1:, None]
        at = at.clamp(max=case["rows"] - 1).long()
        x = x[at]
    else:
        x = x[None]
    out = torch.matmul(x, _dequantized(s["w"]).transpose(1, 2))
    if case["glu"]:
        out = out * torch.sigmoid(out) * torch.matmul(x, _dequantized(s["up"]).transpose(1, 2))
    out = out.to(y.dtype)
    if n > 1:
        y[at[mine]] = out[mine]
    else:
        y.copy_(out[0])
    return y


def _plain_norm(s):
    case, x, u = s["case"], s["x"].float(), s["y"].float()
    if case["after"]:
        u = u * torch.rsqrt((u * u).mean(-1, keepdim=True) + 1e-6) * s["after"]
    if s["gate"] is not None:
        gate = s["gate"].float()
        gate = torch.sigmoid(gate) if case["sigmoid"] else gate
        u = u * (gate[:, None] if case["gate"] == "row" else gate)
    h = 0.9 * x + 1.25 * u
    out = [h.to(s["x"].dtype)]
    if case["before"]:
        out.append((h * torch.rsqrt((h * h).mean(-1, keepdim=True) + 1e-6) * s["before"]).to(s["x"].dtype))
    return out


def _plain_route(logits, k, renorm):
    """The k largest logits of each row, equal ones by the lower expert; -1 and weight 0 where only -inf is left."""
    value, idx = torch.sort(logits, dim=-1, descending=True, stable=True)
    value, idx = value[:, :k], idx[:, :k]
    top = value[:, :1].clamp(min=-1e30)
    part = (value - top).exp()
    total = part.sum(-1, keepdim=True) if renorm else (logits - top).exp().sum(-1, keepdim=True)
    none = value == -math.inf
    return torch.where(none, -1, idx).to(torch.int32), torch.where(none, 0.0, part / total)


def _plain_plan(idx, E):
    """offsets [E + 1], entries [T k] by expert, and each entry's place among them (-1: no expert's)."""
    e = idx.flatten()
    key = torch.where((e >= 0) & (e < E), e, E)
    order = torch.argsort(key, stable=True)
    count = torch.bincount(key, minlength=E + 1)[:E]
    offsets = torch.cat((torch.zeros_like(count[:1]), count.cumsum(0))).to(torch.int32)
    place = torch.empty_like(e)
    place[order] = torch.arange(e.numel(), dtype=torch.int32, device="cuda")
    live = key < E
    entries = torch.where(live[order], order, -1).to(torch.int32)
    return offsets, entries, torch.where(live, place, -1)


def _plain_sort(s):
    case = s["case"]
    idx, w = _plain_route(s["logits"], case["top_k"], case["renorm"])
    offsets, entries, place = _plain_plan(idx, case["experts"])
    live = entries >= 0
    token = entries.clamp(min=0).long() // case["top_k"]
    torch.where(live[:, None], s["x"][token], s["xs"], out=s["xs"])
    return [idx, w, offsets, entries, place, s["xs"]]


def _plain_back(s):
    case, k = s["case"], s["case"]["top_k"]
    live = (s["place"] >= 0).view(-1, k)
    rows = s["z"].float()[s["place"].clamp(min=0).long()].view(-1, k, case["hidden"])
    y = (torch.where(live, s["w"], 0.0)[..., None] * rows).sum(1)
    if case["base"]:
        y = y + s["base"].float()
    return y.to(s["z"].dtype)


def _plain_back_grad(s):
    case, k = s["case"], s["case"]["top_k"]
    live = s["place"] >= 0
    at = s["place"].clamp(min=0).long()
    rows = s["z"].float()[at].view(-1, k, case["hidden"])
    dy = s["dy"].float()
    dw = torch.where(live.view(-1, k), (rows * dy[:, None]).sum(-1), 0.0)
    dz = (s["w"][..., None] * dy[:, None]).to(s["z"].dtype).flatten(0, 1)
    s["dz"][at[live]] = dz[live]
    return [s["dz"], dw]


def run(state):
    s, op = state, state["case"]["op"]
    if own:
        h = s["handle"]
        if op == "linear":
            return h.forward(s["x"], y=s["y"], offsets=s["offsets"] if s["case"]["n"] > 1 else None)
        if op == "norm":
            hn = h.forward(s["x"], s["y"], gate=s["gate"] if s["case"]["gate"] in ("row", "element") else None)
            return [t for t in hn if t is not None]
        if op == "sort":
            idx, w = h.route(s["logits"])
            plan = h.plan(idx)
            h.gather(plan, s["x"], out=s["xs"])
            return [idx, w, plan.offsets, plan.entries, plan.place, s["xs"]]
        if op == "back":
            return h.combine(s["plan"], s["z"], w=s["w"], base=s.get("base"))
        return list(h.combine_backward(s["plan"], s["dy"], s["z"], s["w"], dz=s["dz"]))
    return {"linear": _plain_linear, "norm": _plain_norm, "sort": _plain_sort, "back": _plain_back,
            "back_grad": _plain_back_grad}[op](s)


# --- 64 bits -------------------------------------------------------------------------------------------------


def _weight(w, i):
    """Matrix i in 64 bits, from the format's bits."""
    byte = w.codes[i].repeat_interleave(2, -1)
    odd = torch.arange(w.cols, device="cuda") % 2 == 1
    q = torch.where(odd, byte // 16, byte % 16).double()
    s, m = (t[i].view(torch.float16).double().repeat_interleave(BLOCK, -1) for t in (w.scale, w.min))
    return q * s + m


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "linear":
        y, off = s["y"].double(), s["offsets"].tolist()
        for i in range(case["n"]):
            if off[i] < off[i + 1]:
                x = s["x"][off[i]:off[i + 1]].double()
                p = x @ _weight(s["w"], i).T
                if case["glu"]:
                    p = p / (1 + torch.exp(-p)) * (x @ _weight(s["up"], i).T)
                y[off[i]:off[i + 1]] = p
        return y
    if op == "norm":
        x, u = s["x"].double(), s["y"].double()
        if case["after"]:
            u = u / (u.square().mean(-1, keepdim=True) + 1e-6).sqrt() * s["after"].double()
        gate = 1.0 if s["gate"] is None else s["gate"].double()
        if case["gate"] == "row":
            gate = gate[:, None]
        if case["sigmoid"] and s["gate"] is not None:
            gate = 1 / (1 + torch.exp(-gate))
        h = 0.9 * x + 1.25 * u * gate
        out = [h]
        if case["before"]:
            out.append(h / (h.square().mean(-1, keepdim=True) + 1e-6).sqrt() * s["before"].double())
        return out
    k, E, T = case["top_k"], case["experts"], case["rows"]
    if op == "sort":
        logits = s["logits"].double().cpu().numpy()
        idx, w = np.full((T, k), -1, np.int32), np.zeros((T, k))
        order = np.lexsort((np.broadcast_to(np.arange(E), (T, E)), -logits))[:, :k]
        kept = np.isfinite(np.take_along_axis(logits, order, 1))
        idx[kept] = order[kept]
        e = np.exp(logits - np.maximum(logits.max(1, keepdims=True), -1e300))
        part = np.take_along_axis(e, order, 1)
        total = (part if case["renorm"] else e).sum(1, keepdims=True)
        w = np.where(kept, part / np.where(total > 0, total, 1), 0.0)
        groups = [np.flatnonzero(idx.ravel() == i) for i in range(E)]
        offsets = np.concatenate([[0], np.cumsum([len(x) for x in groups])]).astype(np.int32)
        live = np.concatenate(groups)
        entries, place = np.full(T * k, -1, np.int32), np.full(T * k, -1, np.int32)
        entries[:len(live)] = live
        place[live] = np.arange(len(live))
        xs = s["xs"].double()
        xs[:len(live)] = s["x"].double()[torch.from_numpy(live // k).cuda()]
        return [idx, w, offsets, entries, place, xs]
    place, w = s["place"].view(T, k).long(), s["w"].double()
    if op == "back":
        y = s["base"].double() if case["base"] else torch.zeros(T, case["hidden"], dtype=torch.float64, device="cuda")
        for j in range(k):
            y += torch.where(place[:, j] >= 0, w[:, j], 0.0)[:, None] * s["z"][place[:, j].clamp(min=0)].double()
        return y
    dz, dw, dy = s["dz"].double(), torch.zeros(T, k, dtype=torch.float64, device="cuda"), s["dy"].double()
    for j in range(k):
        mine = place[:, j] >= 0
        at = place[mine, j]
        dw[mine, j] = (dy[mine] * s["z"][at].double()).sum(-1)
        dz[at] = w[mine, j, None] * dy[mine]
    return [dz, dw]
