"""The paged-cache operators as workloads: what they compute in plain torch, and the library's calls.

Three operators of one serving step over a paged, group-quantized KV cache:

  qk      RMS norm of each query and key head and the position rotation, one pass
  append  new K and V rows into the pages, K rotated on the way; the tokens of the touched groups are then read back
          as the values their codes stand for
  attend  attention of each sequence's new tokens over its pages (one token, drafted tokens, chunks, whole prompts)

A cache of pages: k_codes [pages, H_kv, P * D * bits / 8], k_scales [pages, H_kv, P / g, D], v_codes the same as k_codes,
v_scales [pages, H_kv, P, D / g]; 4-bit codes two to a byte, the even feature in the low half; a code stands for
(code - qmax) * scale, qmax 7 or 127. K groups are g tokens of one channel, V groups g features of one token. The rows of
a sequence's unfinished K group are kept unquantized in tail [slots, H_kv, g, D].
"""

import math
import random

import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def attend_case(**kw):
    c = dict(op="attend", S=1, new_lo=1, new_hi=1, ctx_lo=1024, ctx_hi=1024, H=8, G=4, D=128, bits=4, group=32, page=64,
             dtype="bf16", causal=True)
    c.update(kw)
    return c


def append_case(**kw):
    c = dict(op="append", S=1, new_lo=1, new_hi=1, ctx_hi=4096, H=8, D=128, bits=4, group=32, page=64, dtype="bf16",
             rot=128, interleaved=False)
    c.update(kw)
    return c


def qk_case(**kw):
    c = dict(op="qk", T=64, H=8, G=4, D=128, dtype="bf16", rot=128, interleaved=False, norm=True, fused=True)
    c.update(kw)
    return c


def listed():
    return [
        # one user, one token, a short context: latency
        attend_case(name="attend_one", ctx_lo=1000, ctx_hi=1000),
        # the decode workload of the benchmark, in pages
        attend_case(name="attend_decode", S=32, ctx_lo=4096, ctx_hi=4096),
        # the long-context workload's lengths at 8 bits
        attend_case(name="attend_long_8bit", S=8, ctx_lo=1000, ctx_hi=32768, bits=8, page=256),
        # drafted tokens checked by the target: five rows a sequence, eight query heads a KV head
        attend_case(name="attend_draft", S=24, new_lo=5, new_hi=5, ctx_lo=300, ctx_hi=6000, G=8, page=32),
        # the chunk workload: 64 rows over 16k tokens
        attend_case(name="attend_chunk", S=4, new_lo=64, new_hi=64, ctx_lo=16384, ctx_hi=16384, page=128),
        # a ragged batch of prompts, some after a cached prefix
        attend_case(name="attend_prompts", S=5, new_lo=200, new_hi=2500, ctx_lo=1800, ctx_hi=3000, bits=8),
        # float32 activations, a small model's heads, an odd head ratio
        attend_case(name="attend_f32", S=7, ctx_lo=50, ctx_hi=2777, H=4, G=3, D=64, dtype="f32", page=32),
        # one decode step's append
        append_case(name="append_step", S=64),
        # prompts arriving: 8k tokens
        append_case(name="append_prompts", S=4, new_lo=1500, new_hi=2600, ctx_hi=8192, page=128),
        # float32 rows, groups of 8, a partial interleaved rotation, sizes off the powers of two
        append_case(name="append_odd", S=9, new_lo=1, new_hi=301, ctx_hi=2000, H=3, D=80, bits=8, group=8, page=40,
                    dtype="f32", rot=40, interleaved=True),
        # q and k of a decode step, and of 8k prompt tokens
        qk_case(name="qk_step"),
        qk_case(name="qk_prompts", T=8192),
    ]


def spread(rng, lo, hi):
    """A whole number of lo..hi, even in its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["attend", "attend", "append", "qk"])
    H, G, D = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 3, 4, 7, 8]), rng.choice([64, 128, 128])
    bits = rng.choice([4, 8])
    if op == "attend":
        kind = rng.choice(["step", "step", "draft", "chunk", "prompt"])
        page = rng.choice([32, 64, 128, 256, 96])
        dtype = rng.choice(["bf16", "bf16", "f32"]) if kind in ("step", "draft") else "bf16"
        if kind == "step":
            S, hi, new = spread(rng, 1, 64), spread(rng, 40, 32768), (1, 1)
        elif kind == "draft":
            S, hi = spread(rng, 1, 32), spread(rng, 100, 16384)
            n = rng.randint(2, 8)
            new = (n if rng.random() < 0.5 else 1, n)
        elif kind == "chunk":
            S, hi = spread(rng, 1, 8), spread(rng, 600, 16384)
            n = spread(rng, 16, 512)
            new = (spread(rng, 1, n), n)
        else:
            S, hi = spread(rng, 1, 6), spread(rng, 100, 2500)
            new = (max(1, hi // 4), hi)
        lo = hi if rng.random() < 0.3 else max(new[1], spread(rng, max(1, hi // 20), hi))
        # at most the keys and the products of the largest listed cases
        while S > 1 and (S * hi * H * D * bits > 32 * 4096 * 8 * 128 * 4 or S * new[1] * hi * H * G * D > 2**38 // 4):
            S -= 1
        return attend_case(S=S, new_lo=new[0], new_hi=new[1], ctx_lo=lo, ctx_hi=max(hi, new[1]), H=H, G=G, D=D, bits=bits,
                           page=page, dtype=dtype, causal=rng.random() < 0.85)
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op == "append":
        group = rng.choice([8, 32, 32])
        if group == 8 and rng.random() < 0.4:
            D = rng.choice([40, 72, 80, 96])
        page = group * rng.choice([1, 2, 4, 5, 8])
        if rng.random() < 0.5:
            S, new = spread(rng, 1, 256), (1, 1)
        else:
            S = spread(rng, 1, 16)
            n = spread(rng, 2, max(2, min(2048, 8192 // S)))
            new = (spread(rng, 1, n), n)
        rot = rng.choice([0, D, D, D // 2])
        return append_case(S=S, new_lo=new[0], new_hi=new[1], ctx_hi=new[1] + spread(rng, 64, 8192), H=H, D=D, bits=bits,
                           group=group, page=page, dtype=dtype, rot=rot, interleaved=rng.random() < 0.3)
    D = rng.choice([64, 80, 96, 128, 128, 256])
    rot = rng.choice([D, D, D // 2, 0])
    T = spread(rng, 1, 8192 * 8 * 5 * 128 // (H * (G + 1) * max(D, 128)) // 2)
    return qk_case(T=min(T, 16384), H=H, G=G, D=D, dtype=dtype, rot=rot, interleaved=rng.random() < 0.3,
                   norm=rot == 0 or rng.random() < 0.8, fused=rng.random() < 0.6)


def extents(c):
    """Each sequence's (length, new tokens): the case's own, the same for every seed."""
    rng = random.Random(repr(sorted((k, v) for k, v in c.items() if k != "name")))
    got = []
    for i in range(c["S"]):
        n = rng.randint(c["new_lo"], c["new_hi"]) if i else c["new_hi"]
        if c["op"] == "attend":
            got.append((max(n, rng.randint(c["ctx_lo"], c["ctx_hi"]) if i else c["ctx_hi"]), n))
        elif c["new_hi"] == 1:
            got.append((rng.randint(1, c["ctx_hi"]), 1))
        else:
            # a chunk starts where the last one ended, on a group's border: then a pass can be run again on its own result
            start = rng.randint(0, max(0, c["ctx_hi"] - n)) // c["group"] * c["group"]
            got.append((start + n, n))
    return got


def work(case):
    c = case
    es = 2 if c["dtype"] == "bf16" else 4
    if c["op"] == "qk":
        heads = c["T"] * c["H"] * (c["G"] + 1)
        return {"bytes": 2 * heads * c["D"] * es + c["T"] * (c["rot"] * 4 + 4), "flops": heads * (4 * c["D"] + 3 * c["rot"])}
    D, H, g, ext = c["D"], c["H"], c["group"], extents(c)
    token = H * (2 * D * c["bits"] // 8 + 2 * 4 * D // g)          # codes and scales of K and V
    if c["op"] == "attend":
        seen = sum(n * L - (n * (n - 1) // 2 if c["causal"] else 0) for L, n in ext)
        rows = sum(n for _, n in ext) * H * c["G"] * D
        return {"bytes": sum(L for L, _ in ext) * token + 2 * rows * es, "flops": 4 * seen * H * c["G"] * D}
    new = sum(n for _, n in ext)
    back = sum(L - (L - n) // g * g for L, n in ext)              # tokens from the first touched group's start
    kept = sum((L - n) % g + min(n, L % g) for L, n in ext)       # tail rows read and written
    return {"bytes": 2 * new * H * D * es + new * c["rot"] * 4 + kept * H * D * 4 + 2 * back * token + 2 * back * H * D * 4,
            "flops": new * H * (3 * c["rot"] + 6 * D) + 2 * back * H * D}


# ---------------------------------------------------------------------------
# what a program has in hand
# ---------------------------------------------------------------------------
def rope_table(n_pos, rot):
    """[n_pos, rot] float32: cos of each pair's angle, then sin; angles in 64 bits."""
    inv = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=DEV) / rot)
    a = torch.arange(n_pos, dtype=torch.float64, device=DEV)[:, None] * inv
    return torch.cat([a.cos(), a.sin()], 1).float().contiguous()


def quantize(x, bits, dim):
    """Codes (0..2 qmax, uint8) and scales of x grouped whole along `dim`. Both quotients are rounded once (torch multiplies by
    an inverse where the divisor is a Python number): a code next to a border is decided by that."""
    qmax = 7 if bits == 4 else 127
    top = x.abs().amax(dim, keepdim=True)
    s = torch.where(top == 0, torch.ones_like(top), top / torch.full_like(top, qmax))
    return (torch.round(x / s) + qmax).to(torch.uint8), s


def packed(codes, bits):
    """Codes [..., n] two to a byte."""
    return codes[..., 0::2] | (codes[..., 1::2] << 4) if bits == 4 else codes


def prepare(case, seed):
    c = case
    gen = torch.Generator(device=DEV).manual_seed(seed)
    dt = TYPES[c["dtype"]]

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device=DEV)

    if c["op"] == "qk":
        T, H, Hq, D = c["T"], c["H"], c["H"] * c["G"], c["D"]
        n_pos = 8192
        qkv = (1.5 * normal(T, (Hq + 2 * H) * D)).to(dt)           # a fused projection's output
        Q = qkv[:, :Hq * D].unflatten(1, (Hq, D))
        K = qkv[:, Hq * D:(Hq + H) * D].unflatten(1, (H, D))
        if not c["fused"]:
            Q, K = Q.contiguous(), K.contiguous()
        w = [(1 + 0.2 * normal(D)).to(dt) if c["norm"] else None for _ in range(2)]
        pos = torch.randint(0, n_pos, (T,), generator=gen, device=DEV, dtype=torch.int32)
        return {"case": c, "Q": Q, "K": K, "qw": w[0], "kw": w[1], "pos": pos, "eps": 1e-6,
                "rope": rope_table(n_pos, c["rot"]) if c["rot"] else None}

    S, H, D, g, P, bits = c["S"], c["H"], c["D"], c["group"], c["page"], c["bits"]
    ext = extents(c)
    cols = max(-(-L // P) for L, _ in ext)
    used = sum(-(-L // P) for L, _ in ext)
    pages = used + 3
    order = torch.randperm(pages, generator=gen, device=DEV, dtype=torch.int32)[:used].tolist()
    table = torch.full((S, cols), -1, dtype=torch.int32)           # past a sequence's last page: nothing
    for b, (L, _) in enumerate(ext):
        n = -(-L // P)
        table[b, :n] = torch.tensor(order[:n], dtype=torch.int32)
        del order[:n]
    cu = torch.tensor([0] + [n for _, n in ext]).cumsum(0).to(torch.int32)
    T = int(cu[-1])
    lengths = torch.tensor([L for L, _ in ext], dtype=torch.int32)
    st = {"case": c, "table": table.to(DEV), "lengths": lengths.to(DEV), "cu": cu.to(DEV), "T": T, "pages": pages,
          "max_new": max(n for _, n in ext), "cols": cols}

    # what the pages hold: normal keys and values, a hundredth of the channels eight times as large
    big = torch.where(torch.rand(2, H, 1, D, generator=gen, device=DEV) < 0.01, 8.0, 1.0)
    kc, ks = quantize((normal(pages, H, P, D) * big[0]).view(pages, H, P // g, g, D), bits, 3)
    vc, vs = quantize((normal(pages, H, P, D) * big[1]).view(pages, H, P, D // g, g), bits, 4)
    st["k_codes"] = packed(kc.view(pages, H, P * D), bits).contiguous().flatten()
    st["k_scales"] = ks.contiguous().flatten()
    st["v_codes"] = packed(vc.view(pages, H, P * D), bits).contiguous().flatten()
    st["v_scales"] = vs.contiguous().flatten()
    if c["op"] == "attend":
        st["tail"] = torch.zeros(S, H, g, D, device=DEV)
        st["scale"] = 1.0 / math.sqrt(D)
        st["Q"] = normal(T, H * c["G"], D).to(dt)
    else:
        st["tail"] = normal(S, H, g, D)
        kv = normal(T, 2 * H * D).to(dt)                           # a fused projection's output
        st["K"], st["V"] = kv[:, :H * D].unflatten(1, (H, D)), kv[:, H * D:].unflatten(1, (H, D))
        st["rope"] = rope_table(cols * P, c["rot"]) if c["rot"] else None
        start = [(L - n) // g * g for L, n in ext]
        st["start"] = torch.tensor(start, dtype=torch.int32, device=DEV)
        st["cu_back"] = torch.tensor([0] + [L - s for (L, _), s in zip(ext, start)]).cumsum(0).to(torch.int32).to(DEV)
        st["n_back"] = sum(L - s for (L, _), s in zip(ext, start))
        st["max_back"] = max(L - s for (L, _), s in zip(ext, start))
    return st


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def handle(st):
    """The library's cache over the state's buffers: made once, as a program keeps it."""
    if "cache" not in st:
        import sm_b200 as sm
        c = st["case"]
        st["cache"] = sm.PagedCache(st["pages"], c["H"], c["page"], c["D"], c["bits"], c["group"], slots=c["S"], device=DEV,
                                    buffers=(st["k_codes"], st["k_scales"], st["v_codes"], st["v_scales"], st["tail"]))
    return st["cache"]


def run(state):
    st, c = state, state["case"]
    if own:
        import sm_b200 as sm
        if c["op"] == "qk":
            return sm.qk_norm_rope(st["Q"], st["K"], st["pos"], st["rope"], st["qw"], st["kw"], eps=st["eps"],
                                   interleaved=c["interleaved"])
        cache = handle(st)
        if c["op"] == "attend":
            return sm.paged_attend(st["Q"], cache, st["table"], st["lengths"], st["cu"], st["max_new"], st["scale"],
                                   causal=c["causal"])
        sm.paged_append(st["K"], st["V"], cache, st["table"], st["lengths"], st["cu"], st["max_new"], rope=st["rope"],
                        interleaved=c["interleaved"])
        k, v = sm.paged_gather(cache, st["table"], st["start"], st["cu_back"], st["n_back"], st["max_back"])
        return {"k": k, "v": v, "tail": cache.k_tail}
    return {"qk": plain_qk, "append": plain_append, "attend": plain_attend}[c["op"]](st, c)


def halves(x, rot, interleaved):
    return (x[..., 0:rot:2], x[..., 1:rot:2]) if interleaved else (x[..., :rot // 2], x[..., rot // 2:rot])


def rotated(x, cs, rot, interleaved):
    """x [T, heads, D] with its first `rot` features turned by the angles of cs [T, rot]."""
    c, s = cs[:, None, :rot // 2], cs[:, None, rot // 2:]
    a, b = halves(x, rot, interleaved)
    y, z = a * c - b * s, b * c + a * s
    turned = torch.stack([y, z], -1).flatten(-2) if interleaved else torch.cat([y, z], -1)
    return torch.cat([turned, x[..., rot:]], -1)


def plain_qk(st, c):
    got = []
    for x, w in ((st["Q"], st["qw"]), (st["K"], st["kw"])):
        y = x.float()
        if w is not None:
            y = y * torch.rsqrt(y.square().mean(-1, keepdim=True) + st["eps"]) * w.float()
        if c["rot"]:
            y = rotated(y, st["rope"][st["pos"].long()], c["rot"], c["interleaved"])
        got.append(y.to(x.dtype))
    return tuple(got)


def decoded(codes, bits):
    """Bytes [..., n] to their codes less qmax, float32, in order."""
    if bits == 8:
        return codes.float() - 127
    return torch.stack([codes & 15, codes >> 4], -1).flatten(-2).float() - 7


def plain_attend(st, c):
    S, H, G, D, P, g, bits = c["S"], c["H"], c["G"], c["D"], c["page"], c["group"], c["bits"]
    n = st["max_new"]
    idx = st["table"].clamp_min(0).long()
    N = st["cols"] * P

    def paged(buf, *tail):                                         # [S, H, cols, ...]
        return buf.view(st["pages"], H, *tail)[idx].transpose(1, 2)

    k = decoded(paged(st["k_codes"], P * D * bits // 8), bits).reshape(S, H, N // g, g, D)
    k = (k * paged(st["k_scales"], P // g, D).reshape(S, H, N // g, 1, D)).view(S, H, N, D)
    v = decoded(paged(st["v_codes"], P * D * bits // 8), bits).reshape(S, H, N, D // g, g)
    v = (v * paged(st["v_scales"], P, D // g).reshape(S, H, N, D // g, 1)).view(S, H, N, D)
    cu, L = st["cu"].long(), st["lengths"].long()
    new = cu[1:] - cu[:-1]
    i = torch.arange(n, device=DEV)
    there = i < new[:, None]                                       # [S, n]: query i of sequence b exists
    row = torch.where(there, cu[:-1, None] + i, 0)
    q = st["Q"].float()[row].view(S, n, H, G, D).permute(0, 2, 3, 1, 4).reshape(S, H, G * n, D)
    s = (q @ k.transpose(-1, -2)).view(S, H, G, n, N) * st["scale"]
    t = torch.arange(N, device=DEV)
    last = (L - new)[:, None] + i if c["causal"] else (L - 1)[:, None].expand(S, n)
    seen = t <= torch.minimum(last, (L - 1)[:, None])[..., None]    # [S, n, N]
    s = s.masked_fill_(~seen[:, None, None], float("-inf"))
    p = torch.exp_(s - s.amax(-1, keepdim=True))
    o = (p.view(S, H, G * n, N) @ v).view(S, H, G, n, D) / p.sum(-1, keepdim=True)
    out = o.permute(0, 3, 1, 2, 4).reshape(S, n, H * G, D)
    return out[there].to(st["Q"].dtype)


def plain_append(st, c):
    S, H, D, g, bits, T = c["S"], c["H"], c["D"], c["group"], c["bits"], st["T"]
    cu, L = st["cu"].long(), st["lengths"].long()
    tok = torch.arange(T, device=DEV)
    b = torch.searchsorted(cu, tok, right=True) - 1                # each new row's sequence and position
    first = L - (cu[1:] - cu[:-1])
    pos = first[b] + tok - cu[b]
    k = st["K"].float()
    if c["rot"]:
        k = rotated(k, st["rope"][pos], c["rot"], c["interleaved"])
    # rows [S, n, H, D] from each sequence's first touched group on, the unfinished group's kept rows before the new ones
    n = -(-st["max_back"] // g) * g
    base = first // g * g
    rows = torch.zeros(S, n, H, D, device=DEV)
    keep = torch.arange(g, device=DEV)[None] < (first - base)[:, None]
    rows[:, :g] = torch.where(keep[..., None, None], st["tail"].transpose(1, 2), rows[:, :g])
    rows[b, pos - base[b]] = k
    codes, s = quantize(rows.view(S, n // g, g, H, D), bits, 2)
    qmax = 7 if bits == 4 else 127
    kd = ((codes.float() - qmax) * s).view(S, n, H, D)
    # V of the new rows; the group's earlier rows as the pages hold them
    vcode, vs = quantize(st["V"].float().unflatten(-1, (D // g, g)), bits, 3)
    P = c["page"]
    i = torch.arange(n, device=DEV)
    at = base[:, None] + i
    there = at < L[:, None]
    page = st["table"].gather(1, torch.where(there, at // P, 0)).clamp_min(0).long()
    old = decoded(st["v_codes"].view(st["pages"], H, P, D * bits // 8)[page, :, at % P], bits).view(S, n, H, D // g, g)
    vd = old * st["v_scales"].view(st["pages"], H, P, D // g)[page, :, at % P][..., None]
    vd[b, pos - base[b]] = (vcode.float() - qmax) * vs
    # the rows of the group that is now unfinished
    left = L // g * g
    kept = torch.arange(g, device=DEV)
    src = (left - base)[:, None] + kept
    live = (left[:, None] + kept < L[:, None]) & (left[:, None] + kept >= first[:, None])
    fresh = rows[torch.arange(S, device=DEV)[:, None], torch.where(live, src, 0)].transpose(1, 2)
    tail = torch.where(live[:, None, :, None], fresh, st["tail"])
    return {"k": kd[there], "v": vd.flatten(-2)[there], "tail": tail}


# ---------------------------------------------------------------------------
# in 64 bits, from the definition
# ---------------------------------------------------------------------------
def exact(case, seed):
    st, c = prepare(case, seed), case
    D, H = c["D"], c["H"]

    def turn(x, pos, r32=lambda x: x):
        """The rotation of x [n, heads, D] (64 bits) at the positions; r32 rounds each product and each sum."""
        r, h = c["rot"], c["rot"] // 2
        if not r:
            return x
        cs = st["rope"].double()[pos][:, None]
        lo, hi = (list(range(0, r, 2)), list(range(1, r, 2))) if c["interleaved"] else (list(range(h)), list(range(h, r)))
        y = x.clone()
        for to, sign, (u, w) in ((lo, -1, (lo, hi)), (hi, 1, (hi, lo))):
            y[..., to] = r32(r32(x[..., u] * cs[..., :h]) + sign * r32(x[..., w] * cs[..., h:]))
        return y

    def held(x):
        """Rounded once to float32, as the cache's definition has it for a key's rotation, a scale and a quotient: a code
        next to a border is decided by these."""
        return x.float().double()

    if c["op"] == "qk":
        got = []
        for x, w in ((st["Q"], st["qw"]), (st["K"], st["kw"])):
            y = x.double()
            if w is not None:
                y = y / (y.pow(2).sum(-1, keepdim=True) / D + st["eps"]).sqrt() * w.double()
            got.append(turn(y, st["pos"].long()))
        return tuple(got)

    g, P, bits, ext = c["group"], c["page"], c["bits"], extents(case)
    qmax, per = (7, 2) if bits == 4 else (127, 1)

    def row_codes(buf, b, L):
        """Codes less qmax of the first L tokens, [H, L, D], in 64 bits."""
        x = buf.view(-1, H, P, D // per)[st["table"][b, :-(-L // P)].long()]
        x = x.permute(1, 0, 2, 3).reshape(H, -1, D // per)[:, :L]
        y = torch.empty(H, L, D, dtype=torch.float64, device=DEV)
        if bits == 4:
            y[..., 0::2], y[..., 1::2] = x % 16, x // 16
        else:
            y[:] = x
        return y - qmax

    def scales(name, b, n, rows, width):
        x = st[name].view(-1, H, rows, width)[st["table"][b, :-(-n // P)].long()]
        return x.permute(1, 0, 2, 3).reshape(H, -1, width).double()

    outs, cu = [], st["cu"].tolist()
    if c["op"] == "attend":
        for b, (L, n) in enumerate(ext):
            k = row_codes(st["k_codes"], b, L) * scales("k_scales", b, L, P // g, D).repeat_interleave(g, 1)[:, :L]
            v = row_codes(st["v_codes"], b, L) * scales("v_scales", b, L, P, D // g)[:, :L].repeat_interleave(g, 2)
            q = st["Q"][cu[b]:cu[b + 1]].double().view(n, H, c["G"], D)
            o = torch.empty(n, H, c["G"], D, dtype=torch.float64, device=DEV)
            for i in range(0, n, 256):                             # a few rows at a time
                s = torch.einsum("ihgd,htd->higt", q[i:i + 256], k) * st["scale"]
                if c["causal"]:
                    at = torch.arange(L - n + i, L - n + min(n, i + 256), device=DEV)
                    s = s - torch.where(torch.arange(L, device=DEV) > at[:, None], math.inf, 0.0)[None, :, None]
                o[i:i + 256] = torch.einsum("higt,htd->ihgd", torch.softmax(s, -1), v)
            outs.append(o.reshape(n, H * c["G"], D))
        return torch.cat(outs)

    ks, vs, tail = [], [], st["tail"].double().clone()
    for b, (L, n) in enumerate(ext):
        first = L - n
        base = first // g * g
        new = turn(st["K"][cu[b]:cu[b + 1]].double(), torch.arange(first, L, device=DEV), held)
        rows = torch.cat([st["tail"][b].double().transpose(0, 1)[:first - base], new])
        for j in range(0, L - base, g):
            x = rows[j:j + g]
            s = held(x.abs().amax(0) / qmax)
            s[s == 0] = 1
            ks.append(torch.round(held(x / s)) * s)
        left = max(first, L // g * g)
        if left < L:
            tail[b, :, left % g:left % g + L - left] = rows[left - base:].transpose(0, 1)
        if first > base:
            old = row_codes(st["v_codes"], b, first) * scales("v_scales", b, first, P, D // g)[:, :first].repeat_interleave(g, 2)
            vs.append(old[:, base:].transpose(0, 1))
        x = st["V"][cu[b]:cu[b + 1]].double().unflatten(-1, (D // g, g))
        s = held(x.abs().amax(-1, keepdim=True) / qmax)
        s[s == 0] = 1
        vs.append((torch.round(held(x / s)) * s).flatten(-2))
    return {"k": torch.cat(ks), "v": torch.cat(vs), "tail": tail}
