"""Cases of the attention-side operators: the per-head norms of q and k with the position rotation, and the 8-bit
KV caches of the slots (written from a call's rows, read back, attended over).

``run`` computes a case in plain torch operations, or with ``own`` through the library's binding.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "f16": 2, "bf16": 2}
QMAX = {"e4m3": 448.0, "int8": 127.0}
E_MIN, E_MAX, BIAS = -48, 47, 127


# --- cases ---------------------------------------------------------------------------------------------------


def listed():
    return [
        # one verify window of the 48-layer stack: 4 slots, each a token and a proposal, f32 rows
        {"name": "qknorm window", "op": "qknorm", "rows": 8, "heads": 32, "kv_heads": 4, "head_dim": 128,
         "rotary": 128, "interleaved": False, "gain": True, "far": 1002, "dtype": "f32"},
        # a long prompt's rows, far into a conversation, a part of each head rotated
        {"name": "qknorm prompt", "op": "qknorm", "rows": 8191, "heads": 32, "kv_heads": 8, "head_dim": 128,
         "rotary": 64, "interleaved": True, "gain": True, "far": 900001, "dtype": "bf16"},
        # the same window's k and v into the slots' caches, blocks partly held
        {"name": "append window", "op": "append", "seqs": 4, "rows": 2, "ctx": 1002, "max_ctx": 1024, "heads": 32,
         "kv_heads": 4, "head_dim": 128, "block": 16, "format": "int8", "dtype": "f32", "ragged": 0.3},
        # several prompts of other lengths, written at once
        {"name": "append prompts", "op": "append", "seqs": 6, "rows": 5003, "ctx": 6001, "max_ctx": 8192,
         "heads": 32, "kv_heads": 8, "head_dim": 128, "block": 64, "format": "e4m3", "dtype": "bf16", "ragged": 0.5},
        # one slot's conversation read back, to move it elsewhere
        {"name": "read slot", "op": "read", "seqs": 1, "rows": 1002, "ctx": 1002, "max_ctx": 1024, "heads": 32,
         "kv_heads": 4, "head_dim": 128, "block": 32, "format": "int8", "dtype": "f32", "ragged": 0.0},
        # many slots' long conversations
        {"name": "read slots", "op": "read", "seqs": 8, "rows": 16383, "ctx": 16383, "max_ctx": 16384, "heads": 32,
         "kv_heads": 8, "head_dim": 128, "block": 64, "format": "e4m3", "dtype": "bf16", "ragged": 0.6},
        # the window's attention at the 48-layer stack's shapes
        {"name": "attend window", "op": "attend", "seqs": 4, "rows": 2, "ctx": 1002, "max_ctx": 1024, "heads": 32,
         "kv_heads": 4, "head_dim": 128, "block": 32, "format": "e4m3", "dtype": "f32", "ragged": 0.0},
        # one conversation, one token, a long cache
        {"name": "attend long", "op": "attend", "seqs": 1, "rows": 1, "ctx": 131071, "max_ctx": 131072, "heads": 32,
         "kv_heads": 8, "head_dim": 128, "block": 64, "format": "e4m3", "dtype": "bf16", "ragged": 0.0},
        # many conversations of other lengths, one token each
        {"name": "attend batch", "op": "attend", "seqs": 64, "rows": 1, "ctx": 8191, "max_ctx": 8192, "heads": 32,
         "kv_heads": 8, "head_dim": 128, "block": 64, "format": "e4m3", "dtype": "bf16", "ragged": 0.8},
        # no shared heads, short heads, two rows a slot
        {"name": "attend heads of 64", "op": "attend", "seqs": 24, "rows": 2, "ctx": 2047, "max_ctx": 2100,
         "heads": 16, "kv_heads": 16, "head_dim": 64, "block": 16, "format": "int8", "dtype": "f16", "ragged": 0.5},
        # a prompt from its first token
        {"name": "attend prompt", "op": "attend", "seqs": 1, "rows": 8191, "ctx": 8191, "max_ctx": 8192, "heads": 32,
         "kv_heads": 8, "head_dim": 128, "block": 64, "format": "e4m3", "dtype": "bf16", "ragged": 0.0},
        # chunks of two prompts on what their slots hold already, f32 rows
        {"name": "attend chunks", "op": "attend", "seqs": 2, "rows": 1531, "ctx": 9001, "max_ctx": 9008, "heads": 32,
         "kv_heads": 4, "head_dim": 128, "block": 32, "format": "int8", "dtype": "f32", "ragged": 0.4},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["qknorm", "append", "read", "attend", "attend", "attend"])
    heads, kv_heads = rng.choice([(32, 4), (32, 8), (16, 16), (28, 4), (64, 8), (8, 1), (5, 5), (20, 4)])
    head_dim = rng.choice([64, 128, 128])
    dtype = rng.choice(["f32", "f16", "bf16"])
    if op == "qknorm":
        return {"op": op, "rows": _log(rng, 1, 6000), "heads": heads, "kv_heads": kv_heads, "head_dim": head_dim,
                "rotary": rng.choice([head_dim, head_dim // 2]), "interleaved": rng.random() < 0.5,
                "gain": rng.random() < 0.7, "far": _log(rng, 1, 1000000), "dtype": dtype}
    case = {"op": op, "heads": heads, "kv_heads": kv_heads, "head_dim": head_dim, "dtype": dtype,
            "block": rng.choice([16, 32, 64, 128]), "format": rng.choice(["e4m3", "int8"]),
            "ragged": round(rng.uniform(0.0, 0.8), 2)}
    if op == "attend" and rng.random() < 0.4:  # prompts: the pairs of row and position stay below the listed one's
        ctx = _log(rng, 17, 5600)
        rows = _log(rng, 9, ctx) if ctx > 9 else ctx
        seqs = max(1, min(_log(rng, 1, 6), 30000000 // (rows * ctx * (1 + heads // 40))))
    elif op == "attend":
        rows = rng.choice([1, 1, 2, 3, 8])
        ctx = _log(rng, rows, 60000)
        seqs = max(1, min(_log(rng, 1, 96), 2000000 // (ctx * kv_heads)))
    else:
        ctx = _log(rng, 1, 16000)
        rows = ctx if op == "read" else _log(rng, 1, ctx)
        seqs = max(1, min(_log(rng, 1, 64), 400000 // (ctx * kv_heads)))
    return {**case, "seqs": seqs, "rows": rows, "ctx": ctx, "max_ctx": ctx + rng.randrange(0, 40)}


def _plan(case):
    """(rows, length) of each sequence, from the case alone: the first is the longest, the others spread below it."""
    frac = [1.0 - case["ragged"] * ((i * 0.6180339887) % 1.0) for i in range(case["seqs"])]
    length = [max(1, int(case["ctx"] * f)) for f in frac]
    rows = [min(n, max(1, int(case["rows"] * f))) if case["rows"] > 8 else min(n, case["rows"])
            for n, f in zip(length, frac)]
    return rows, length


def work(case):
    z, hd = SIZE[case["dtype"]], case["head_dim"]
    if case["op"] == "qknorm":
        n = case["rows"] * (case["heads"] + case["kv_heads"]) * hd
        return {"bytes": 2 * n * z + 4 * case["rows"], "flops": 10 * n}
    rows, length = _plan(case)
    kv = case["kv_heads"] * hd
    if case["op"] in ("append", "read"):
        n = 2 * sum(rows) * kv
        return {"bytes": n * (z + 1) + n // (hd * case["block"]), "flops": 2 * n}
    seen = sum(r * n - r * (r - 1) // 2 for r, n in zip(rows, length))
    codes = 2 * sum(length) * kv
    return {"bytes": codes + codes // (hd * case["block"]) + 2 * sum(rows) * case["heads"] * hd * z,
            "flops": 4 * seen * case["heads"] * hd}


# --- inputs --------------------------------------------------------------------------------------------------


def _values(g, shape, dtype, spread):
    """Normal values whose size varies from token to token and from channel to channel, as keys and values do."""
    x = torch.randn(shape, generator=g, device="cuda")
    x *= torch.exp2(spread * torch.randn(shape[:-1] + (1,), generator=g, device="cuda"))
    x *= torch.exp2(0.5 * torch.randn(shape[-1], generator=g, device="cuda"))
    return x.to(dtype)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed * 2654435761 % (1 << 62))
    dt, hd, kvh = DTYPES[case["dtype"]], case["head_dim"], case["kv_heads"]
    s = {"case": case}
    if case["op"] == "qknorm":
        T = case["rows"]
        qkv = _values(g, (T, case["heads"] + 2 * kvh, hd), dt, 1.0)  # one product's rows: q, k, v side by side
        s["q"], s["k"] = qkv[:, :case["heads"]], qkv[:, case["heads"]:case["heads"] + kvh]
        far = torch.randint(0, max(1, case["far"] - T) + 1, (1,), generator=g, device="cuda")
        s["position"] = (far + torch.arange(T, device="cuda")).to(torch.int32)
        s["freq"] = [1e6 ** (-2.0 * i / case["rotary"]) for i in range(case["rotary"] // 2)]
        s["freqs"] = torch.tensor(s["freq"], dtype=torch.float64, device="cuda")
        s["q_gain"] = 1 + 0.3 * torch.randn(hd, generator=g, device="cuda") if case["gain"] else None
        s["k_gain"] = 1 + 0.3 * torch.randn(hd, generator=g, device="cuda") if case["gain"] else None
        if own:
            from slot_decode_window_gb300 import binding
            s["handle"] = binding.QkNorm(case["heads"], kvh, hd, rotary_dim=case["rotary"], freqs=s["freq"],
                                         interleaved=case["interleaved"], eps=1e-6, q_gain=s["q_gain"],
                                         k_gain=s["k_gain"])
        return s
    rows, length = _plan(case)
    n, B, ctx = case["seqs"], case["block"], case["max_ctx"]
    slots = n + 1
    start = np.concatenate([[0], np.cumsum(rows)])
    T, fmt = int(start[-1]), case["format"]
    dev = dict(dtype=torch.int32, device="cuda")
    s.update(T=T, max_rows=max(rows), max_len=max(length), start=torch.tensor(start, **dev),
             length=torch.tensor(length, **dev),
             slot=torch.randperm(slots, generator=torch.Generator().manual_seed(seed))[:n].to(**dev))
    for name in ("k", "v"):
        held = _values(g, (slots, kvh, ctx, hd), torch.float32, 0.7)
        pad = -ctx % B
        e = _exponent(torch.nn.functional.pad(held.abs().amax(-1), (0, pad)).view(slots, kvh, -1, B).amax(-1),
                      fmt)
        s[name + "_codes"] = _encode(held, e.repeat_interleave(B, -1)[..., :ctx, None], fmt)
        s[name + "_exp"] = (e + BIAS).to(torch.uint8)
        del held
        if case["op"] == "append":
            s[name] = _values(g, (T, kvh, hd), dt, 0.7)
    if case["op"] == "attend":
        s["q"] = _values(g, (T, case["heads"], hd), dt, 0.5)
        s["scale"] = 1 / math.sqrt(hd)
    if own:
        from slot_decode_window_gb300 import binding
        s["handle"] = binding.KvCache8(1, slots, case["heads"], kvh, hd, ctx, block=B, format=fmt,
                                       buffers=(s["k_codes"], s["v_codes"], s["k_exp"], s["v_exp"]))
        s["rows"] = binding.KvRows(s["start"], s["slot"], s["length"], n_rows=T, max_rows=s["max_rows"])
    return s


# --- plain forms ---------------------------------------------------------------------------------------------


def _exponent(a, fmt):
    """The least e with a <= qmax 2^e, within the format's range."""
    m, x = torch.frexp(a)  # a = m 2^x, m in [0.5, 1)
    qm, qx = math.frexp(QMAX[fmt])
    e = x - qx + (m > qm).to(x.dtype)
    return torch.where(a > 0, e, torch.full_like(e, E_MIN)).clamp(E_MIN, E_MAX)


def _pow2(e):
    """2^e in f32 for whole e in [-126, 127], by its bits."""
    return ((e.int() + 127) << 23).view(torch.float32)


def _encode(x, e, fmt):
    v = (x.float() * _pow2(-e)).clamp(-QMAX[fmt], QMAX[fmt])
    if fmt == "e4m3":
        return v.to(torch.float8_e4m3fn).view(torch.uint8)
    return torch.round(v).to(torch.int8).view(torch.uint8)


def _decode(codes, e, fmt):
    v = codes.view(torch.float8_e4m3fn if fmt == "e4m3" else torch.int8).float()
    return v * _pow2(e)


def _plain_qknorm(s):
    case = s["case"]
    rd, half = case["rotary"], case["rotary"] // 2
    turn = s["position"].double()[:, None] * s["freqs"]
    cos, sin = torch.cos(turn).float()[:, None], torch.sin(turn).float()[:, None]
    out = []
    for x, gain in ((s["q"], s["q_gain"]), (s["k"], s["k_gain"])):
        y = x.float()
        y = y * torch.rsqrt((y * y).mean(-1, keepdim=True) + 1e-6)
        if gain is not None:
            y = y * gain
        r = y[..., :rd]
        a, b = (r[..., 0::2], r[..., 1::2]) if case["interleaved"] else (r[..., :half], r[..., half:])
        p, q = a * cos - b * sin, a * sin + b * cos
        r = torch.stack((p, q), -1).flatten(-2) if case["interleaved"] else torch.cat((p, q), -1)
        out.append(torch.cat((r, y[..., rd:]), -1).to(x.dtype))
    return out


def _where(s):
    """Each row's sequence, slot and position."""
    seq = torch.bucketize(torch.arange(s["T"], device="cuda", dtype=torch.int32), s["start"][1:], right=True)
    pos = s["length"][seq] - s["start"][seq + 1] + torch.arange(s["T"], device="cuda")
    return seq, s["slot"][seq].long(), pos.long()


def _plain_append(s):
    case = s["case"]
    fmt, B, kvh = case["format"], case["block"], case["kv_heads"]
    seq, slot, pos = _where(s)
    first = (s["length"] - (s["start"][1:] - s["start"][:-1])).long()  # each sequence's first new position
    own_slot, blk0 = s["slot"].long(), first // B
    held = first % B != 0
    out = []
    for name in ("k", "v"):
        x, codes, exps = s[name], s[name + "_codes"], s[name + "_exp"]
        nblk = exps.shape[2]
        a = torch.zeros(exps.shape[0] * nblk, kvh, device="cuda")
        at = slot * nblk + pos // B
        a.scatter_reduce_(0, at[:, None].expand(-1, kvh), x.abs().amax(-1).float(), "amax")
        e = _exponent(a, fmt)
        e_held = exps[own_slot, :, blk0].int() - BIAS
        at0 = own_slot * nblk + blk0
        e0 = torch.where(held[:, None], torch.maximum(e_held, e[at0]), e[at0])
        e[at0] = e0
        # what the sequences' first blocks hold before the new rows
        p = blk0[:, None] * B + torch.arange(B, device="cuda")
        keep = p < first[:, None]
        p = p.clamp(max=codes.shape[2] - 1)
        old = codes[own_slot[:, None], :, p]
        new = _encode(_decode(old, (e_held - e0)[:, None, :, None], fmt), torch.zeros_like(e0)[:, None, :, None], fmt)
        codes[own_slot[:, None], :, p] = torch.where(keep[..., None, None], new, old)
        codes[slot, :, pos] = _encode(x, e[at][..., None], fmt)
        exps[slot, :, pos // B] = (e[at] + BIAS).to(torch.uint8)
        out += [codes.view(torch.float8_e4m3fn if fmt == "e4m3" else torch.int8), exps]
    return out


def _plain_read(s):
    case = s["case"]
    _, slot, pos = _where(s)
    return [_decode(s[n + "_codes"][slot, :, pos], (s[n + "_exp"][slot, :, pos // case["block"]].int() - BIAS)[..., None],
                    case["format"]).to(DTYPES[case["dtype"]]) for n in ("k", "v")]


def _plain_attend(s):
    case = s["case"]
    L, R, B, hd, kvh = s["max_len"], s["max_rows"], case["block"], case["head_dim"], case["kv_heads"]
    group = case["heads"] // kvh
    n = case["seqs"]
    j = torch.arange(L, device="cuda")
    k, v = (_decode(s[x + "_codes"][s["slot"].long(), :, :L],
                    (s[x + "_exp"][s["slot"].long()].int() - BIAS).repeat_interleave(B, -1)[..., :L, None],
                    case["format"]) for x in ("k", "v"))
    # each sequence's rows, padded to the most that one has
    count = s["start"][1:] - s["start"][:-1]
    i = torch.arange(R, device="cuda")
    at = (s["start"][:-1, None] + i).clamp(max=s["T"] - 1).long()
    q = s["q"].float()[at].view(n, R, kvh, group, hd).permute(0, 2, 3, 1, 4).reshape(n, kvh, group * R, hd)
    pos = (s["length"] - count)[:, None] + i  # [n][R]
    sees = (j <= pos[..., None]) & (j < s["length"][:, None, None])  # [n][R][L]
    score = torch.matmul(q, k.transpose(-1, -2)).view(n, kvh, group, R, L) * s["scale"]
    score = score.masked_fill_(~sees[:, None, None], -math.inf)
    score -= score.amax(-1, keepdim=True).clamp(min=-1e30)
    p = score.exp_()
    o = torch.matmul(p.view(n, kvh, group * R, L), v).view(n, kvh, group, R, hd)
    total = p.sum(-1, keepdim=True)
    o = torch.where(total > 0, o / total, torch.zeros_like(o)).permute(0, 3, 1, 2, 4).reshape(n, R, case["heads"], hd)
    seq, _, _ = _where(s)
    row = torch.arange(s["T"], device="cuda") - s["start"][seq]
    return o[seq, row].to(DTYPES[case["dtype"]])


def run(state):
    s, op = state, state["case"]["op"]
    if own:
        if op == "qknorm":
            return s["handle"].forward(s["q"], s["k"], s["position"])
        if op == "append":
            s["handle"].append(0, s["k"], s["v"], s["rows"])
            as_type = torch.float8_e4m3fn if s["case"]["format"] == "e4m3" else torch.int8
            return [s["k_codes"].view(as_type), s["k_exp"], s["v_codes"].view(as_type), s["v_exp"]]
        if op == "read":
            return s["handle"].read(0, s["rows"], DTYPES[s["case"]["dtype"]])
        return s["handle"].attend(0, s["q"], s["rows"])
    return {"qknorm": _plain_qknorm, "append": _plain_append, "read": _plain_read, "attend": _plain_attend}[op](s)


# --- 64 bits -------------------------------------------------------------------------------------------------


def _stands_for(codes, fmt):
    """The numbers that the codes are, from the formats' bits."""
    c = codes.astype(np.int64)
    if fmt == "int8":
        return np.where(c > 127, c - 256, c).astype(np.float64)
    m, x = c & 7, (c >> 3) & 15
    mag = np.where(x > 0, (8 + m) * np.exp2(x - 10.0), m * np.exp2(-9.0))
    return np.where(c > 127, -mag, mag)


def _nearest(v, fmt):
    """The format's number nearest to v, ties to the even one."""
    v = np.clip(v, -QMAX[fmt], QMAX[fmt])
    if fmt == "int8":
        return np.rint(v)
    size = np.floor(np.log2(np.maximum(np.abs(v), 2.0 ** -6)))
    step = np.exp2(np.maximum(size, -6.0) - 3.0)
    return np.rint(v / step) * step


def _least(a, fmt):
    """The least exponent whose range holds a, by trying them in turn."""
    e = np.full(a.shape, E_MAX)
    for x in range(E_MAX, E_MIN - 1, -1):
        e = np.where(a <= QMAX[fmt] * 2.0 ** x, x, e)
    return e


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "qknorm":
        pos = s["position"].cpu().numpy().astype(np.longdouble)
        angle = np.fmod(pos[:, None] * np.array(s["freq"], np.longdouble), 2 * np.arccos(np.longdouble(-1)))
        z = np.exp(1j * angle.astype(np.float64))[:, None]
        rd, out = case["rotary"], []
        for x, gain in ((s["q"], s["q_gain"]), (s["k"], s["k_gain"])):
            y = x.double().cpu().numpy()
            y = y / np.sqrt(np.square(y).mean(-1, keepdims=True) + 1e-6)
            if gain is not None:
                y = y * gain.double().cpu().numpy()
            one = slice(0, rd, 2) if case["interleaved"] else slice(0, rd // 2)
            two = slice(1, rd, 2) if case["interleaved"] else slice(rd // 2, rd)
            w = (y[..., one] + 1j * y[..., two]) * z
            y[..., one], y[..., two] = w.real, w.imag
            out.append(y)
        return out
    fmt, B = case["format"], case["block"]
    start, length, slot = (s[x].cpu().numpy() for x in ("start", "length", "slot"))
    if case["op"] == "append":
        out = []
        for name in ("k", "v"):
            x, codes, exps = (s[n].float().cpu().numpy() if n == name else s[n].cpu().numpy()
                              for n in (name, name + "_codes", name + "_exp"))
            value, exps = _stands_for(codes, fmt), exps.copy()
            for i in range(case["seqs"]):
                new = x[start[i]:start[i + 1]].astype(np.float64).transpose(1, 0, 2)
                p0, p1 = length[i] - new.shape[1], length[i]
                for b in range(p0 // B, (p1 - 1) // B + 1):
                    lo, hi = max(p0, b * B), min(p1, b * B + B)
                    part = new[:, lo - p0:hi - p0]
                    e = _least(np.abs(part).max((1, 2)), fmt)
                    if lo > b * B:
                        held = exps[slot[i], :, b].astype(np.int64) - BIAS
                        e = np.maximum(e, held)
                        old = value[slot[i], :, b * B:lo]
                        value[slot[i], :, b * B:lo] = _nearest(old * np.exp2(held - e)[:, None, None], fmt)
                    value[slot[i], :, lo:hi] = _nearest(part * np.exp2(-e.astype(np.float64))[:, None, None], fmt)
                    exps[slot[i], :, b] = e + BIAS
            out += [value if fmt == "e4m3" else value.astype(np.int8), exps]
        return out
    table = torch.from_numpy(_stands_for(np.arange(256), fmt)).cuda()
    held = {}
    for name in ("k", "v"):
        held[name] = []
        for i in range(case["seqs"]):
            step = torch.exp2(s[name + "_exp"][slot[i]].double() - BIAS).repeat_interleave(B, 1)[:, :length[i], None]
            held[name].append(table[s[name + "_codes"][slot[i], :, :length[i]].int()] * step)
    if case["op"] == "read":
        return [torch.cat([held[n][i][:, length[i] - (start[i + 1] - start[i]):].transpose(0, 1)
                           for i in range(case["seqs"])]) for n in ("k", "v")]
    group, out = case["heads"] // case["kv_heads"], []
    for i in range(case["seqs"]):
        q = s["q"][start[i]:start[i + 1]].double().transpose(0, 1)
        n, r = int(length[i]), q.shape[1]
        k, v = held["k"][i], held["v"][i]
        at = torch.arange(n - r, n, device="cuda")
        late = torch.arange(n, device="cuda") > at[:, None]
        o = []
        for h in range(case["heads"]):
            w = (q[h] @ k[h // group].T) / math.sqrt(case["head_dim"])
            w = torch.softmax(w.masked_fill(late, -math.inf), -1)
            o.append(w @ v[h // group])
        out.append(torch.stack(o, 1))
    return torch.cat(out)
