"""Workloads of the paged key/value cache operators: the append (with the position rotation) and the attention over
the cache, each as a plain torch form and as the library's call.

A case names its operator (`op`: "append" or "fwd"), the cache's type (`cache`: "bf16" or "e4m3", the latter with one
power-of-two scale for each page and KV head), the number of sequences, the tokens already cached (`ctx`) and the new
tokens (`new`) of the longest sequence, whether the others are shorter (`ragged`), the heads, the head dimension and
the tokens of a page; for the append also the rotated dimensions (`rot`) and whether a pair is adjacent
(`interleaved`).
"""
import math

import torch

own = False

E4M3_MAX = 448.0
MIN_EXPONENT = -100          # the scale of a page of zeros is 2^-100


def _case(name, op, cache, seqs, ctx, new, ragged, hq, hkv, d, page, rot=0, interleaved=False):
    c = dict(op=op, cache=cache, seqs=seqs, ctx=ctx, new=new, ragged=ragged, hq=hq, hkv=hkv, d=d, page=page, rot=rot,
             interleaved=interleaved)
    return dict(name=name, **c) if name else c


def listed():
    return [
        # one user generating: a single token, where only latency counts
        _case("append_bf16_one", "append", "bf16", 1, 4095, 1, False, 32, 8, 128, 64, rot=128),
        # a decoding batch with sequences of every length
        _case("append_e4m3_step", "append", "e4m3", 64, 8191, 1, True, 32, 8, 128, 64, rot=128),
        # four fresh prompts packed one after another, as the library's THD workload packs them
        _case("append_e4m3_prompts", "append", "e4m3", 4, 0, 8192, True, 16, 16, 128, 128, rot=128),
        # chunks of prompts whose beginnings are cached; half the dimensions rotated, adjacent pairs
        _case("append_bf16_chunks", "append", "bf16", 8, 1500, 1000, True, 32, 32, 64, 16, rot=32, interleaved=True),
        # one user, a short conversation: the smallest attention
        _case("fwd_bf16_one", "fwd", "bf16", 1, 1000, 1, False, 32, 8, 128, 64),
        # a decoding batch, bf16 and 8-bit
        _case("fwd_bf16_step", "fwd", "bf16", 64, 8191, 1, True, 32, 8, 128, 64),
        _case("fwd_e4m3_step", "fwd", "e4m3", 64, 8191, 1, True, 32, 8, 128, 64),
        # one user with a long document: few rows, a long key axis
        _case("fwd_e4m3_long", "fwd", "e4m3", 1, 262143, 1, False, 32, 8, 128, 128),
        # no shared heads, small pages
        _case("fwd_bf16_heads64", "fwd", "bf16", 24, 4000, 1, True, 32, 32, 64, 16),
        # five drafted tokens to verify in each sequence
        _case("fwd_e4m3_draft", "fwd", "e4m3", 16, 4000, 5, True, 16, 2, 64, 32),
        # a chunk of a prompt over its cached beginning
        _case("fwd_bf16_chunk", "fwd", "bf16", 2, 8192, 2048, False, 32, 8, 128, 64),
        # prompts' chunks and decoding sequences in one batch
        _case("fwd_e4m3_mixed", "fwd", "e4m3", 12, 4000, 700, True, 16, 4, 128, 64),
    ]


def lengths(case):
    """(cached tokens, new tokens) of each sequence: the longest first, then, where ragged, spread over the logarithm."""
    n = case["seqs"]
    if not case["ragged"]:
        return [case["ctx"]] * n, [case["new"]] * n
    ctx, new = [], []
    for i in range(n):
        u, w = (i * 0.6180339887498949) % 1.0, (i * 0.7548776662466927) % 1.0
        ctx.append(round(case["ctx"] ** (1.0 - 0.7 * u)) if case["ctx"] else 0)
        new.append(max(1, round(case["new"] ** (1.0 - (0.35 if case["ctx"] == 0 else 1.0) * w))))
    return ctx, new


def _pairs(case):
    """Visible (query, key) pairs of one head, over all sequences."""
    return sum(m * c + m * (m + 1) // 2 for c, m in zip(*lengths(case)))


def work(case):
    ctx, new = lengths(case)
    T, n = sum(new), case["seqs"]
    hq, hkv, d, ps = case["hq"], case["hkv"], case["d"], case["page"]
    el = 2 if case["cache"] == "bf16" else 1
    if case["op"] == "append":
        touched = sum((c + m - 1) // ps - c // ps + 1 for c, m in zip(ctx, new))
        positions = len(set().union(*(range(c, c + m) for c, m in set(zip(ctx, new))))) if T else 0
        nbytes = 2 * T * (2 * hq + 2 * hkv) * d + 2 * T * hkv * d * el + 4 * positions * case["rot"]
        nbytes += 4 * touched + 4 * 2 * n + (8 * touched * hkv if el == 1 else 0)
        return {"bytes": nbytes, "flops": 3 * T * (hq + hkv) * case["rot"]}
    keys = sum(c + m for c, m in zip(ctx, new))
    pages = sum(-(-(c + m) // ps) for c, m in zip(ctx, new))
    nbytes = 2 * keys * hkv * d * el + 4 * T * hq * d + 4 * T * hq + 4 * pages + 4 * 2 * n
    nbytes += 8 * pages * hkv if el == 1 else 0
    return {"bytes": nbytes, "flops": 4 * d * hq * _pairs(case)}


def _cost(case):
    w = work(case)
    return max(w["bytes"] / 6.8e12, w["flops"] / 1.9e15)


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    top = {op: max(_cost(c) for c in listed() if c["op"] == op) for op in ("append", "fwd")}
    while True:
        op = rng.choice(("append", "fwd"))
        d = rng.choice((64, 128))
        hkv = rng.choice((1, 2, 4, 5, 8, 16))
        group = rng.choice((1, 2, 3, 4, 6, 8))
        kind = rng.choice(("one", "step", "draft", "chunk"))
        seqs = log(1, 96)
        ctx = log(16, 65536) if kind != "chunk" else rng.choice((0, log(16, 16384)))
        new = {"one": 1, "step": 1, "draft": rng.randint(2, 9), "chunk": log(17, 4096)}[kind]
        if kind == "one":
            seqs = 1
        rot = rng.choice((d, d // 2)) if op == "append" else 0
        c = _case("", op, rng.choice(("bf16", "e4m3")), seqs, ctx, new, rng.random() < 0.7 and seqs > 1, hkv * group,
                  hkv, d, rng.choice((16, 32, 64, 128)), rot, op == "append" and rng.random() < 0.5)
        # the plain form pads every sequence to the longest: its scores have to fit
        scores = seqs * c["hq"] * new * (ctx + new) * 4 if op == "fwd" else 0
        padded = seqs * hkv * (ctx + new) * d * 4
        if _cost(c) <= top[op] and scores < 6e9 and padded < 6e9:
            return c


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)
    ctx, new = lengths(case)
    n, T, ps = case["seqs"], sum(new), case["page"]
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    total = [c + m for c, m in zip(ctx, new)]
    width = max(-(-t // ps) for t in total)
    pages = sum(-(-t // ps) for t in total) + 3
    order = torch.randperm(pages, generator=g, device=dev).to(torch.int32)
    table = torch.full((n, width), -1, dtype=torch.int32)
    order, at = order.cpu(), 0
    for i, t in enumerate(total):
        k = -(-t // ps)
        table[i, :k] = order[at:at + k]
        at += k
    cu = torch.tensor([0] + new, dtype=torch.int64).cumsum(0).to(torch.int32)

    def randn(*shape):
        return torch.randn(*shape, generator=g, device=dev, dtype=torch.float32)

    def filled():
        """A pool whose pages hold N(0, 1) values; in 8 bits under scales of 2^-7 to 2^-5."""
        if case["cache"] == "bf16":
            return torch.randn(pages, hkv, ps, d, generator=g, device=dev, dtype=torch.bfloat16), None
        scale = torch.exp2(torch.randint(-7, -4, (pages, hkv), generator=g, device=dev).float())
        codes = torch.empty(pages, hkv, ps, d, dtype=torch.float8_e4m3fn, device=dev)
        for lo in range(0, pages, 4096):
            part = randn(min(4096, pages - lo), hkv, ps, d)
            codes[lo:lo + 4096] = (part / scale[lo:lo + 4096, :, None, None]).clamp(-E4M3_MAX, E4M3_MAX).to(codes.dtype)
        return codes, scale

    (kc, ks), (vc, vs) = filled(), filled()
    s = dict(case=case, q=randn(T, hq, d).to(torch.bfloat16), k_cache=kc, v_cache=vc, k_scale=ks, v_scale=vs,
             page_table=table.to(dev), cu_seqlens=cu.to(dev), longest=max(total), max_new=max(new),
             seqlens_kv=torch.tensor(total, dtype=torch.int32, device=dev))
    if case["op"] == "append":
        s["k"] = randn(T, hkv, d).to(torch.bfloat16)
        s["v"] = randn(T, hkv, d).to(torch.bfloat16)
        r = case["rot"]
        freq = 10000.0 ** (-torch.arange(0, r, 2, dtype=torch.float64, device=dev) / r)
        angle = torch.arange(max(total), dtype=torch.float64, device=dev)[:, None] * freq
        s["cos_sin"] = torch.cat([angle.cos(), angle.sin()], 1).to(torch.float32)
    return s


# ---------------------------------------------------------------------------------------------------------------------
# Plain forms
# ---------------------------------------------------------------------------------------------------------------------
def _rotate(x, cos, sin, interleaved):
    r = 2 * cos.shape[-1]
    x = x.float()
    c, s = cos[:, None], sin[:, None]
    if interleaved:
        a, b = x[..., 0:r:2], x[..., 1:r:2]
        y = torch.stack([a * c - b * s, b * c + a * s], -1).flatten(-2)
    else:
        a, b = x[..., :r // 2], x[..., r // 2:r]
        y = torch.cat([a * c - b * s, b * c + a * s], -1)
    return torch.cat([y, x[..., r:]], -1)


def _append_plain(s):
    case = s["case"]
    cu, total, table, ps = s["cu_seqlens"].long(), s["seqlens_kv"].long(), s["page_table"].long(), case["page"]
    token = torch.arange(s["q"].shape[0], device=cu.device)
    seq = torch.searchsorted(cu[1:], token, right=True)
    pos = total[seq] - cu[seq + 1] + token
    page, slot = table[seq, pos // ps], pos % ps
    r = case["rot"]
    cos, sin = s["cos_sin"][pos, :r // 2], s["cos_sin"][pos, r // 2:]
    q_out = _rotate(s["q"], cos, sin, case["interleaved"]).to(torch.bfloat16)
    for new, cache, scale in ((_rotate(s["k"], cos, sin, case["interleaved"]), s["k_cache"], s["k_scale"]),
                              (s["v"].float(), s["v_cache"], s["v_scale"])):
        if scale is None:
            cache[page, :, slot] = new.to(torch.bfloat16)
            continue
        # the largest magnitude that this call brings to each page and head, and the first row it writes there
        amax = torch.zeros_like(scale).scatter_reduce_(0, page[:, None].expand(-1, case["hkv"]), new.abs().amax(-1), "amax")
        first = torch.full_like(scale[:, 0], ps).scatter_reduce_(0, page, slot.float(), "amin")
        part, e = torch.frexp(amax)                       # amax = part 2^e, part in [1/2, 1); 448 = 7/8 2^9
        e = torch.where(part <= 0.875, e - 9, e - 8)
        e = torch.where(amax > 0, e, torch.full_like(e, MIN_EXPONENT)).clamp(min=MIN_EXPONENT)
        want = torch.exp2(e.float())
        grown = torch.where(first[:, None] > 0, torch.maximum(scale, want), want)
        grown = torch.where(first[:, None] < ps, grown, scale)
        # pages that held tokens before: their codes again under the grown scale (a sequence's first page at most)
        start = total - (cu[1:] - cu[:-1])
        old = table.gather(1, (start // ps)[:, None])[:, 0]
        codes = cache[old]
        again = (codes.float() * (scale[old] / grown[old])[..., None, None]).to(codes.dtype)
        keep = torch.arange(ps, device=cu.device)[None, None, :, None] < (start % ps)[:, None, None, None]
        cache.view(torch.uint8)[old] = torch.where(keep, again.view(torch.uint8), codes.view(torch.uint8))
        scale.copy_(grown)
        cache.view(torch.uint8)[page, :, slot] = (new / grown[page][..., None]).to(cache.dtype).view(torch.uint8)
    return _outputs(s, q_out)


def _outputs(s, q_out):
    out = dict(q=q_out, k_cache=s["k_cache"], v_cache=s["v_cache"])
    if s["k_scale"] is not None:
        out.update(k_scale=s["k_scale"], v_scale=s["v_scale"])
    return out


def _gathered(s, cache, scale, pages, live):
    """[n, hkv, keys, d] in 32 bits, zeros where no key is."""
    x = cache[pages].float()
    if scale is not None:
        x = x * scale[pages][..., None, None]
    x = x.permute(0, 2, 1, 3, 4).flatten(2, 3)
    return torch.where(live[:, None, :, None], x, torch.zeros((), device=x.device))


def _fwd_plain(s):
    case = s["case"]
    cu, total, ps = s["cu_seqlens"].long(), s["seqlens_kv"].long(), case["page"]
    hq, hkv, d, n = case["hq"], case["hkv"], case["d"], case["seqs"]
    T, m, dev = s["q"].shape[0], s["max_new"], cu.device
    pages = s["page_table"].long().clamp(min=0)
    key = torch.arange(pages.shape[1] * ps, device=dev)
    live = key[None] < total[:, None]
    k, v = (_gathered(s, s[c], s[x], pages, live) for c, x in (("k_cache", "k_scale"), ("v_cache", "v_scale")))
    row = torch.arange(m, device=dev)
    count = cu[1:] - cu[:-1]
    token = (cu[:-1, None] + row).clamp(max=T - 1)
    q = s["q"][token].float().view(n, m, hkv, hq // hkv, d).permute(0, 2, 3, 1, 4).flatten(2, 3)
    x = q @ k.transpose(-1, -2) * (1.0 / math.sqrt(d))
    seen = live[:, None] & (key[None, None] <= (total - count)[:, None, None] + row[None, :, None])
    x = x.view(n, hkv, hq // hkv, m, -1).masked_fill_(~seen[:, None, None], -math.inf)
    top = x.amax(-1, keepdim=True)
    top = torch.where(torch.isinf(top), torch.zeros_like(top), top)
    p = torch.exp(x - top)
    norm = p.sum(-1)
    o = (p.flatten(2, 3) @ v).view(n, hkv, hq // hkv, m, d)
    o = torch.where(norm[..., None] > 0, o / norm[..., None], torch.zeros_like(o))
    lse = top[..., 0] + torch.log(norm)
    t = torch.arange(T, device=dev)
    seq = torch.searchsorted(cu[1:], t, right=True)
    i = t - cu[seq]
    o = o.permute(0, 3, 1, 2, 4).flatten(2, 3)[seq, i]
    lse = lse.permute(0, 3, 1, 2).flatten(2, 3)[seq, i]
    return dict(o=o.to(torch.bfloat16), lse=lse.t().contiguous())


# ---------------------------------------------------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------------------------------------------------
def run(s):
    if not own:
        return _append_plain(s) if s["case"]["op"] == "append" else _fwd_plain(s)
    import softmax_attention_backward_gb300 as A
    kw = dict(page_table=s["page_table"], seqlens_kv=s["seqlens_kv"], cu_seqlens=s["cu_seqlens"], max_new=s["max_new"],
              k_scale=s["k_scale"], v_scale=s["v_scale"])
    if s["case"]["op"] == "append":
        q_out = A.attn_cache_append(s["q"], s["k"], s["v"], s["k_cache"], s["v_cache"], cos_sin=s["cos_sin"],
                                    interleaved=s["case"]["interleaved"], **kw)
        return _outputs(s, q_out)
    o, lse = A.attn_cache_fwd(s["q"], s["k_cache"], s["v_cache"], **kw)
    return dict(o=o, lse=lse)


# ---------------------------------------------------------------------------------------------------------------------
# The definition in 64 bits
# ---------------------------------------------------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    ctx, new = lengths(case)
    ps, hq, hkv, d = case["page"], case["hq"], case["hkv"], case["d"]
    F = torch.float64
    table = s["page_table"].cpu().tolist()
    if case["op"] == "append":
        r = case["rot"]
        cs = s["cos_sin"].to(F)

        def turned(x, lo):
            x = x.to(F).clone()
            c, sn = cs[lo:lo + x.shape[0], None, :r // 2], cs[lo:lo + x.shape[0], None, r // 2:]
            ia = slice(0, r, 2) if case["interleaved"] else slice(0, r // 2)
            ib = slice(1, r, 2) if case["interleaved"] else slice(r // 2, r)
            a, b = x[..., ia].clone(), x[..., ib].clone()
            x[..., ia], x[..., ib] = a * c - b * sn, a * sn + b * c
            return x

        out = dict(q=torch.empty(s["q"].shape, dtype=F, device="cuda"), k_cache=s["k_cache"].to(F), v_cache=s["v_cache"].to(F))
        if s["k_scale"] is not None:
            out.update(k_scale=s["k_scale"].to(F), v_scale=s["v_scale"].to(F))
        t0 = 0
        for i, (c, m) in enumerate(zip(ctx, new)):
            rows = slice(t0, t0 + m)
            out["q"][rows] = turned(s["q"][rows], c)
            for name, x in (("k", turned(s["k"][rows], c)), ("v", s["v"][rows].to(F))):
                cache, scale = out[name + "_cache"], out.get(name + "_scale")
                lo = c
                while lo < c + m:
                    hi = min(c + m, (lo // ps + 1) * ps)
                    page, part = table[i][lo // ps], x[lo - c:hi - c].transpose(0, 1)
                    if scale is not None:
                        least = torch.ceil(torch.log2(part.abs().amax((1, 2)) / E4M3_MAX)).clamp(min=MIN_EXPONENT)
                        wide = torch.exp2(least)
                        if lo % ps:
                            wide = torch.maximum(wide, scale[page])
                            cache[page, :, :lo % ps] *= (scale[page] / wide)[:, None, None]
                        scale[page] = wide
                        part = part / wide[:, None, None]
                    cache[page, :, lo % ps:lo % ps + hi - lo] = part
                    lo = hi
            t0 += m
        return out
    if 4.0 * d * hq * _pairs(case) > 4e12:
        return None
    o = torch.zeros(s["q"].shape, dtype=F, device="cuda")
    lse = torch.zeros(hq, s["q"].shape[0], dtype=F, device="cuda")
    t0 = 0
    for i, (c, m) in enumerate(zip(ctx, new)):
        L = c + m
        pages = torch.tensor(table[i][:-(-L // ps)], device="cuda")
        k, v = s["k_cache"][pages].to(F), s["v_cache"][pages].to(F)
        if s["k_scale"] is not None:
            k, v = k * s["k_scale"][pages].to(F)[..., None, None], v * s["v_scale"][pages].to(F)[..., None, None]
        k, v = (x.transpose(0, 1).reshape(hkv, -1, d)[:, :L] for x in (k, v))
        ahead = torch.ones(m, L, dtype=torch.bool, device="cuda").triu(c + 1)
        for h in range(hq):
            x = s["q"][t0:t0 + m, h].to(F) @ k[h * hkv // hq].T / math.sqrt(d)
            x[ahead] = -math.inf
            lse[h, t0:t0 + m] = torch.logsumexp(x, -1)
            o[t0:t0 + m, h] = torch.softmax(x, -1) @ v[h * hkv // hq]
        t0 += m
    return dict(o=o, lse=lse)
