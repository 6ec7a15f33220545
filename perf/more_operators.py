"""Workloads of the position rotation and of linear attention with a decay for each head: the table of cosines and sines
(scaled for long contexts), the rotation and its backward pass, the chunked linear attention and its backward pass, and
its recurrent step for single tokens, each as a plain torch form and as the library's call.

A case names its operator (`op`), the number of sequences (`seqs`), the tokens of the longest (`length`), whether the
sequences are packed with lengths of their own (`packed`), the heads of queries and of keys and values (`hq`, `hkv`) and
the head dimension (`d`).  For the rotation also the rotated dims (`rot`), the first of them (`offset`) and whether a
pair is adjacent (`interleaved`); for the table the scaling and its factor, `length` being its positions; for linear
attention whether it starts from and returns states (`states`).
"""
import math

import torch

own = False

CHUNK = 256                  # tokens of a step of the plain chunked form


def _case(name, op, seqs, length, packed, hq, hkv, d, rot=0, offset=0, interleaved=False, scaling="none", factor=1.0,
          states=False):
    c = dict(op=op, seqs=seqs, length=length, packed=packed, hq=hq, hkv=hkv, d=d, rot=rot, offset=offset,
             interleaved=interleaved, scaling=scaling, factor=factor, states=states)
    return dict(name=name, **c) if name else c


def listed():
    return [
        # the table of a short-context model that rotates half of a head of 128
        _case("table_short", "table", 1, 4096, False, 1, 1, 64, rot=64),
        # a model taken to sixteen times its length, the frequencies scaled by parts
        _case("table_long", "table", 1, 131072, False, 1, 1, 128, rot=128, scaling="parts", factor=16.0),
        # the training batch of the benchmark's headline shape, shared key heads
        _case("rotary_fwd_dense", "rotary_fwd", 4, 4096, False, 32, 8, 128, rot=128),
        # packed sequences, adjacent pairs, half of the head rotated: the gradients of q and k
        _case("rotary_bwd_packed", "rotary_bwd", 16, 2000, True, 16, 16, 64, rot=32, interleaved=True),
        # a decoding batch: one token of each sequence at a position of its own
        _case("rotary_fwd_step", "rotary_fwd", 64, 1, False, 32, 8, 128, rot=128),
        # training, as many key heads as query heads
        _case("linear_fwd_dense", "linear_fwd", 4, 4096, False, 32, 32, 128),
        # packed sequences with shared key heads of 64
        _case("linear_fwd_packed", "linear_fwd", 12, 8192, True, 16, 4, 64),
        # one user's chunk of a prompt, from the state that the chunk before left: few tokens, latency counts
        _case("linear_fwd_prompt", "linear_fwd", 1, 500, False, 32, 32, 128, states=True),
        # the training step's other half, two long sequences with shared key heads
        _case("linear_bwd_dense", "linear_bwd", 2, 8192, False, 32, 8, 128),
        # packed sequences continued from states: the gradients of the first states too
        _case("linear_bwd_packed", "linear_bwd", 12, 2500, True, 16, 16, 64, states=True),
        # a decoding batch: every state is read and written once
        _case("step_batch", "step", 64, 1, False, 32, 32, 128),
        # one user generating, shared key heads
        _case("step_one", "step", 1, 1, False, 32, 8, 128),
    ]


def lengths(case):
    """The tokens of each sequence: the longest first, then, where packed, spread over the logarithm."""
    n, top = case["seqs"], case["length"]
    if not case["packed"]:
        return [top] * n
    return [max(1, round(top ** (1.0 - 0.5 * ((i * 0.6180339887498949) % 1.0)))) for i in range(n)]


def work(case):
    T, n, hq, hkv, d = sum(lengths(case)), case["seqs"], case["hq"], case["hkv"], case["d"]
    op = case["op"]
    index = 4 * (n + 1) if case["packed"] else 0
    if op == "table":
        # a multiplication and two functions for a pair of outputs
        return {"bytes": 4 * case["length"] * case["rot"], "flops": 3 * case["length"] * case["rot"] // 2}
    if op.startswith("rotary"):
        positions = n if case["length"] == 1 else max(lengths(case))
        nbytes = 2 * 2 * T * (hq + hkv) * d + 4 * positions * case["rot"] + index + (4 * T if case["length"] == 1 else 0)
        return {"bytes": nbytes, "flops": 3 * T * (hq + hkv) * case["rot"]}
    # the recurrent form's products, the least there are: an outer product and a product with the state, 2 d^2 each
    state = 4 * n * hkv * d * d
    if op == "step":
        return {"bytes": 2 * n * (2 * hq + 2 * hkv) * d + 2 * state + 4 * hkv + 4 * n, "flops": 2 * n * d * d * (hq + 2 * hkv)}
    if op == "linear_fwd":
        return {"bytes": 2 * T * (2 * hq + 2 * hkv) * d + 4 * hkv + index + (2 * state if case["states"] else 0),
                "flops": 2 * T * d * d * (hq + hkv)}
    return {"bytes": 2 * T * (3 * hq + 4 * hkv) * d + 4 * hkv + index + (3 * state if case["states"] else 0),
            "flops": 2 * T * d * d * (2 * hq + 3 * hkv)}


def _cost(case):
    w = work(case)
    return max(w["bytes"] / 6.8e12, w["flops"] / 1.9e15)


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    top = {}
    for c in listed():
        top[c["op"]] = max(top.get(c["op"], 0.0), _cost(c))
    top["rotary_fwd"] = top["rotary_bwd"] = max(top["rotary_fwd"], top["rotary_bwd"])
    while True:
        op = rng.choice(("table", "rotary_fwd", "rotary_bwd", "linear_fwd", "linear_bwd", "step"))
        d = rng.choice((64, 128))
        hkv = rng.choice((1, 2, 3, 4, 5, 8, 16, 32))
        hq = hkv * rng.choice((1, 1, 2, 3, 4, 6, 8))
        if op == "table":
            rot = 16 * rng.randint(1, 8)
            scaling = rng.choice(("none", "linear", "base", "parts"))
            c = _case("", op, 1, log(256, 131072), False, 1, 1, rot, rot=rot, scaling=scaling,
                      factor=1.0 if scaling == "none" else round(2.0 ** rng.uniform(0.5, 5.0), 2))
        elif op.startswith("rotary"):
            # heads of 576 carry the rotated dims behind 512 others, as the sparse attention's do
            d = rng.choice((64, 128, 128, 576))
            rot = 64 if d == 576 else rng.choice((d, d // 2, 16 * rng.randint(1, d // 16)))
            if d == 576:
                hkv = 1
                hq = rng.choice((16, 24, 64))
            single = op == "rotary_fwd" and rng.random() < 0.3
            c = _case("", op, log(1, 256) if single else log(1, 32), 1 if single else log(16, 16384),
                      not single and rng.random() < 0.5, hq, hkv, d, rot=rot, offset=512 if d == 576 else 0,
                      interleaved=rng.random() < 0.5)
        elif op == "step":
            c = _case("", op, log(1, 256), 1, False, hq, hkv, d)
        else:
            seqs = log(1, 24)
            c = _case("", op, seqs, log(1, 16384), seqs > 1 and rng.random() < 0.6, hq, hkv, d, states=rng.random() < 0.4)
        if _cost(c) <= top[op]:
            return c


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)
    op, n, hq, hkv, d = case["op"], case["seqs"], case["hq"], case["hkv"], case["d"]
    lens = lengths(case)
    T = sum(lens)
    s = dict(case=case)
    if op == "table":
        # another base for each seed: models differ in it
        s["base"] = 10000.0 * (1.0 + (seed % 97))
        return s
    lead = (n, case["length"]) if not case["packed"] and case["length"] > 1 else (T,)

    def rows(heads):
        return torch.randn(*lead, heads, d, generator=g, device=dev, dtype=torch.bfloat16)

    if case["packed"]:
        s["cu_seqlens"] = torch.tensor([0] + lens, dtype=torch.int64).cumsum(0).to(torch.int32).to(dev)
    s["q"], s["k"] = rows(hq), rows(hkv)
    if op.startswith("rotary"):
        r, top = case["rot"], 8192 if case["length"] == 1 else max(lens)
        freq = 10000.0 ** (-torch.arange(0, r, 2, dtype=torch.float64, device=dev) / r)
        angle = torch.arange(top, dtype=torch.float64, device=dev)[:, None] * freq
        s["cos_sin"] = torch.cat([angle.cos(), angle.sin()], 1).to(torch.float32)
        if case["length"] == 1:
            s["positions"] = torch.randint(0, top, (T,), generator=g, device=dev, dtype=torch.int32)
        return s
    s["v"] = rows(hkv)
    # memories from one or two tokens to some thousands, in another order for each seed
    u = torch.rand(hkv, generator=g, device=dev)
    s["log_decay"] = -torch.exp2(-11.0 * u)
    if op == "step":
        slots = n + 3
        s["state"] = torch.randn(slots, hkv, d, d, generator=g, device=dev)
        s["slots"] = torch.randperm(slots, generator=g, device=dev)[:n].to(torch.int32)
        return s
    if op == "linear_bwd":
        s["dout"] = rows(hq)
    if case["states"]:
        s["initial_state"] = 3.0 * torch.randn(n, hkv, d, d, generator=g, device=dev)
        if op == "linear_bwd":
            s["dfinal_state"] = torch.randn(n, hkv, d, d, generator=g, device=dev)
    return s


# ---------------------------------------------------------------------------------------------------------------------
# Plain forms
# ---------------------------------------------------------------------------------------------------------------------
ORIGINAL, FAST, SLOW = 8192, 32.0, 1.0    # of the scaling by parts: positions trained on, turns that bound the ramp


def _magnitude(case):
    return 0.1 * math.log(case["factor"]) + 1.0 if case["scaling"] == "parts" else 1.0


def _table_plain(s):
    case = s["case"]
    r, factor, base = case["rot"], case["factor"], s["base"]
    if case["scaling"] == "base":
        base = base * factor ** (r / (r - 2))
    freq = base ** (-torch.arange(0, r, 2, dtype=torch.float64, device="cuda") / r)
    if case["scaling"] == "linear":
        freq = freq / factor
    if case["scaling"] == "parts":
        keep = ((ORIGINAL * freq / (2.0 * math.pi) - SLOW) / (FAST - SLOW)).clamp(0.0, 1.0)
        freq = freq * (keep + (1.0 - keep) / factor)
    angle = torch.arange(case["length"], dtype=torch.float64, device="cuda")[:, None] * freq
    return (torch.cat([angle.cos(), angle.sin()], 1) * _magnitude(case)).to(torch.float32)


def _positions(s):
    """The position of each token, tokens in one row."""
    case = s["case"]
    if case["length"] == 1 and "positions" in s:
        return s["positions"].long()
    if not case["packed"]:
        return torch.arange(case["length"], device="cuda").repeat(case["seqs"])
    cu = s["cu_seqlens"].long()
    t = torch.arange(s["q"].shape[0], device="cuda")
    return t - cu[torch.searchsorted(cu[1:], t, right=True)]


def _rotary_plain(s):
    case, pos = s["case"], _positions(s)
    r, lo = case["rot"], case["offset"]
    c, sn = s["cos_sin"][pos, None, :r // 2], s["cos_sin"][pos, None, r // 2:]
    if case["op"] == "rotary_bwd":
        sn = -sn
    out = []
    for x in (s["q"], s["k"]):
        x = x.view(-1, *x.shape[-2:])
        p = x[..., lo:lo + r].float()
        if case["interleaved"]:
            a, b = p[..., 0::2], p[..., 1::2]
            y = torch.stack([a * c - b * sn, b * c + a * sn], -1).flatten(-2)
        else:
            a, b = p[..., :r // 2], p[..., r // 2:]
            y = torch.cat([a * c - b * sn, b * c + a * sn], -1)
        out.append(torch.cat([x[..., :lo], y.to(torch.bfloat16), x[..., lo + r:]], -1))
    return dict(q=out[0].view(s["q"].shape), k=out[1].view(s["k"].shape))


def _padded(s):
    """What gathers the packed rows into [n, longest] and back, and the lengths."""
    case = s["case"]
    n, dev = case["seqs"], torch.device("cuda")
    if not case["packed"]:
        return (lambda x: x.view(n, case["length"], *x.shape[-2:]).float(), lambda x, like: x.reshape(like.shape),
                torch.full((n,), case["length"], device=dev))
    cu = s["cu_seqlens"].long()
    count = cu[1:] - cu[:-1]
    i = torch.arange(case["length"], device=dev)
    live = i[None] < count[:, None]
    row = (cu[:-1, None] + i).clamp(max=s["q"].shape[0] - 1)
    return (lambda x: torch.where(live[:, :, None, None], x[row].float(), torch.zeros((), device=dev)),
            lambda x, like: x[live].view(like.shape), count)


def _walk(x, y, z, count, g, scale, state, backwards):
    """out_i = scale sum_j exp(g |i - j|) <x_i, y_j> z_j over j up to i (or, backwards, from i on) and what `state`
    holds, chunk by chunk; x, y, z [n, H, L, d], g [H].  Forwards, a state reaches its first token decayed once and
    scaled; backwards it arrives as it is, and leaves decayed and scaled."""
    n, H, L, d = x.shape
    dev = x.device
    out = torch.empty_like(x)
    steps = list(range(0, L, CHUNK))
    for lo in (reversed(steps) if backwards else steps):
        hi = min(L, lo + CHUNK)
        i = torch.arange(hi - lo, device=dev)
        m = (count - lo).clamp(0, hi - lo)                                      # tokens of each sequence in the chunk
        far = (i[:, None] - i[None]) * (-1 if backwards else 1)
        near = torch.where(far >= 0, torch.exp(g[:, None, None] * far.clamp(min=0)), torch.zeros((), device=dev))
        p = x[:, :, lo:hi] @ y[:, :, lo:hi].transpose(-1, -2) * (scale * near)
        if backwards:
            reach = (m[:, None] - 1 - i).clamp(min=0)                           # decays from the chunk's end
            into = scale * torch.exp(g[:, None] * (i + 1))[None].expand(n, -1, -1)
            seen = torch.exp(g[None, :, None] * reach[:, None])
        else:
            seen = scale * torch.exp(g[:, None] * (i + 1))[None].expand(n, -1, -1)
            into = torch.exp(g[None, :, None] * (m[:, None] - 1 - i).clamp(min=0)[:, None])
        out[:, :, lo:hi] = p @ z[:, :, lo:hi] + seen[..., None] * (x[:, :, lo:hi] @ state)
        grown = (y[:, :, lo:hi] * into[..., None]).transpose(-1, -2) @ z[:, :, lo:hi]
        state = state * torch.exp(g[None] * m[:, None])[..., None, None] + grown
    return out, state


def _linear_plain(s):
    case = s["case"]
    n, hq, hkv, d = case["seqs"], case["hq"], case["hkv"], case["d"]
    group = hq // hkv
    pad, unpad, count = _padded(s)
    scale = 1.0 / math.sqrt(d)
    g = s["log_decay"].repeat_interleave(group)

    def heads(x):
        x = pad(x).transpose(1, 2)
        return x.repeat_interleave(hq // x.shape[1], 1)

    q, k, v = (heads(s[t]) for t in ("q", "k", "v"))
    zero = torch.zeros(n, hkv, d, d, device=q.device)
    start = s.get("initial_state", zero).repeat_interleave(group, 1)

    def rows(x, like):
        return unpad(x.transpose(1, 2).contiguous(), like).to(torch.bfloat16)

    if case["op"] == "linear_fwd":
        o, final = _walk(q, k, v, count, g, scale, start, False)
        out = dict(o=rows(o, s["q"]))
        if case["states"]:
            out["final_state"] = final[:, ::group].contiguous()
        return out
    do = heads(s["dout"])
    end = s.get("dfinal_state", zero).repeat_interleave(group, 1) / group       # shared among the group's heads
    dq, _ = _walk(do, v, k, count, g, scale, start.transpose(-1, -2), False)
    dv, dstart = _walk(k, q, do, count, g, scale, end, True)
    dk, _ = _walk(v, do, q, count, g, scale, end.transpose(-1, -2), True)
    dk, dv = (t.view(n, hkv, group, -1, d).sum(2) for t in (dk, dv))
    out = dict(dq=rows(dq, s["q"]), dk=rows(dk, s["k"]), dv=rows(dv, s["v"]))
    if case["states"]:
        out["dinitial_state"] = dstart.view(n, hkv, group, d, d).sum(2)
    return out


def _step_plain(s):
    case, at = s["case"], s["slots"].long()
    group = case["hq"] // case["hkv"]
    h = s["state"][at] * torch.exp(s["log_decay"])[:, None, None]
    h = h + s["k"].float()[..., :, None] * s["v"].float()[..., None, :]
    s["state"][at] = h
    q = s["q"].float().view(-1, case["hkv"], group, case["d"])
    o = (q @ h) * (1.0 / math.sqrt(case["d"]))
    return dict(o=o.view(s["q"].shape).to(torch.bfloat16), state=s["state"])


# ---------------------------------------------------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------------------------------------------------
def run(s):
    case = s["case"]
    op = case["op"]
    if not own:
        if op == "table":
            return _table_plain(s)
        if op.startswith("rotary"):
            return _rotary_plain(s)
        return _step_plain(s) if op == "step" else _linear_plain(s)
    import softmax_attention_backward_gb300 as A
    if op == "table":
        return A.attn_rotary_table(case["length"], case["rot"], base=s["base"], scaling=case["scaling"],
                                   factor=case["factor"], original=ORIGINAL, fast=FAST, slow=SLOW,
                                   magnitude=_magnitude(case))
    if op.startswith("rotary"):
        call = A.attn_rotary_fwd if op == "rotary_fwd" else A.attn_rotary_bwd
        q, k = call(s["q"], s["k"], s["cos_sin"], positions=s.get("positions"), cu_seqlens=s.get("cu_seqlens"),
                    interleaved=case["interleaved"], rot_offset=case["offset"])
        return dict(q=q, k=k)
    if op == "step":
        o = A.linear_attn_step(s["q"], s["k"], s["v"], s["log_decay"], s["state"], slots=s["slots"])
        return dict(o=o, state=s["state"])
    kw = dict(cu_seqlens=s.get("cu_seqlens"), initial_state=s.get("initial_state"))
    lead = (s["q"], s["k"], s["v"])
    if op == "linear_fwd":
        if case["length"] == 1 and not case["packed"]:
            lead = tuple(x[:, None] for x in lead)
        o, final = A.linear_attn_fwd(*lead, s["log_decay"], want_final_state=case["states"], **kw)
        out = dict(o=o.view(s["q"].shape))
        if case["states"]:
            out["final_state"] = final
        return out
    lead = (*lead, s["dout"])
    if case["length"] == 1 and not case["packed"]:
        lead = tuple(x[:, None] for x in lead)
    dq, dk, dv, dstart = A.linear_attn_bwd(*lead, s["log_decay"], dfinal_state=s.get("dfinal_state"),
                                           want_dinitial_state=case["states"], **kw)
    out = dict(dq=dq.view(s["q"].shape), dk=dk.view(s["k"].shape), dv=dv.view(s["v"].shape))
    if case["states"]:
        out["dinitial_state"] = dstart
    return out


# ---------------------------------------------------------------------------------------------------------------------
# The definition in 64 bits
# ---------------------------------------------------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    F = torch.float64
    op, n, hq, hkv, d = case["op"], case["seqs"], case["hq"], case["hkv"], case["d"]
    lens = lengths(case)
    if op == "table":
        r, pairs = case["rot"], []
        for a in range(r // 2):
            f = (s["base"] * (case["factor"] ** (r / (r - 2.0)) if case["scaling"] == "base" else 1.0)) ** (-2.0 * a / r)
            if case["scaling"] == "linear":
                f /= case["factor"]
            if case["scaling"] == "parts":
                w = min(1.0, max(0.0, (ORIGINAL * f / (2 * math.pi) - SLOW) / (FAST - SLOW)))
                f = w * f + (1 - w) * f / case["factor"]
            pairs.append(f)
        angle = torch.outer(torch.arange(case["length"], dtype=F, device="cuda"), torch.tensor(pairs, dtype=F, device="cuda"))
        turned = torch.polar(torch.full_like(angle, _magnitude(case)), angle)
        return torch.cat([turned.real, turned.imag], 1)
    if op.startswith("rotary"):
        r, lo = case["rot"], case["offset"]
        sign = -1.0 if op == "rotary_bwd" else 1.0
        if case["length"] == 1:
            at = s["positions"].cpu()
        else:
            at = torch.cat([torch.arange(m) for m in lens])
        cs = s["cos_sin"].to(F)[at.to("cuda").long()]
        turn = torch.complex(cs[:, :r // 2], sign * cs[:, r // 2:])[:, None]
        out = {}
        for name in ("q", "k"):
            x = s[name].reshape(-1, *s[name].shape[-2:]).to(F)
            ia = slice(lo, lo + r, 2) if case["interleaved"] else slice(lo, lo + r // 2)
            ib = slice(lo + 1, lo + r, 2) if case["interleaved"] else slice(lo + r // 2, lo + r)
            z = torch.complex(x[..., ia].contiguous(), x[..., ib].contiguous()) * turn
            x[..., ia], x[..., ib] = z.real, z.imag
            out[name] = x.view(s[name].shape)
        return out
    decay, scale, group = s["log_decay"].to(F), d ** -0.5, hq // hkv
    if op == "step":
        state, o = s["state"].to(F), torch.empty(s["q"].shape, dtype=F, device="cuda")
        for i, at in enumerate(s["slots"].cpu().tolist()):
            for h in range(hkv):
                state[at, h] = state[at, h] * torch.exp(decay[h]) + torch.outer(s["k"][i, h].to(F), s["v"][i, h].to(F))
                o[i, h * group:(h + 1) * group] = scale * (s["q"][i, h * group:(h + 1) * group].to(F) @ state[at, h])
        return dict(o=o, state=state)
    if sum(m * m for m in lens) * hq * d * (4.0 if op == "linear_fwd" else 14.0) > 6e12:
        return None
    flat = {t: s[t].reshape(-1, *s[t].shape[-2:]) for t in ("q", "k", "v", "dout") if t in s}
    names = ("q",) if op == "linear_fwd" else ("q", "k", "v")
    out = {t: torch.zeros(flat[t].shape, dtype=F, device="cuda") for t in names}
    states = torch.zeros(n, hkv, d, d, dtype=F, device="cuda")
    t0 = 0
    for b, m in enumerate(lens):
        rows = slice(t0, t0 + m)
        i = torch.arange(m, dtype=F, device="cuda")
        for h in range(hkv):
            k, v = flat["k"][rows, h].to(F), flat["v"][rows, h].to(F)
            first = s["initial_state"][b, h].to(F) if case["states"] else torch.zeros(d, d, dtype=F, device="cuda")
            w = torch.exp(decay[h] * (i[:, None] - i)).tril() * scale
            reach = torch.exp(decay[h] * (i + 1))[:, None]              # of the first state in each token's
            left = torch.exp(decay[h] * (m - 1 - i))[:, None]           # of each token in the last state
            if op == "linear_fwd":
                for hh in range(h * group, (h + 1) * group):
                    q = flat["q"][rows, hh].to(F)
                    out["q"][rows, hh] = ((q @ k.T) * w) @ v + scale * (reach * q) @ first
                states[b, h] = torch.exp(decay[h] * m) * first + (left * k).T @ v
                continue
            last = s["dfinal_state"][b, h].to(F) if case["states"] else torch.zeros(d, d, dtype=F, device="cuda")
            states[b, h] = torch.exp(decay[h] * m) * last
            out["k"][rows, h] = left * (v @ last.T)
            out["v"][rows, h] = left * (k @ last)
            for hh in range(h * group, (h + 1) * group):
                q, do = flat["q"][rows, hh].to(F), flat["dout"][rows, hh].to(F)
                pv = (do @ v.T) * w
                out["q"][rows, hh] = pv @ k + scale * reach * (do @ first.T)
                out["k"][rows, h] += pv.T @ q
                out["v"][rows, h] += ((q @ k.T) * w).T @ do
                states[b, h] += scale * (reach * q).T @ do
        t0 += m
    if op == "linear_fwd":
        return dict(o=out["q"].view(s["q"].shape), **(dict(final_state=states) if case["states"] else {}))
    return dict(dq=out["q"].view(s["q"].shape), dk=out["k"].view(s["k"].shape), dv=out["v"].view(s["v"].shape),
                **(dict(dinitial_state=states) if case["states"] else {}))
