"""The operators between the qkv site and the o site of a block, as workloads that can be timed and checked.

Four operators, each in a plain form (elementary torch operations) and as the call that a user makes:

heads    norm of every query and key head, rotary positions on them, value heads copied, in one pass
cache    tokens' keys and values into a paged cache, as bf16 or as 8-bit floating point (e4m3) codes with one float32
         scale for a token's head; and rows of the cache read back as bf16
prompt   attention of whole prompts, packed one behind another, with grouped heads; causal or not, and over keys
         of their own lengths (a prefix that was cached before)
decode   attention of one new token of each sequence over the paged cache

`own` selects the framework's calls.
"""
import math

import torch

own = False

E4M3_MAX = 448.0
F32, F64 = torch.float32, torch.float64
BF16, E4M3 = torch.bfloat16, torch.float8_e4m3fn


# ---------------------------------------------------------------------------------------------------------------- cases
def _ragged(n, low, high, step):
    """n lengths between low and high, spread over their logarithm in a fixed order."""
    return " ".join(str(int(round(low * (high / low) ** ((i * step % n) / max(n - 1, 1))))) for i in range(n))


def listed():
    return [
        # one token's q and k heads of a decode step, far into a context
        dict(name="heads token", op="heads", M=1, q=8, k=2, v=2, D=256, rot=256, inter=False, far=100003, layout="rows"),
        # the qkv site's output of a long ragged prompt
        dict(name="heads prompt 4571", op="heads", M=4571, q=28, k=4, v=4, D=128, rot=128, inter=False, far=0, layout="heads"),
        # the new tokens of a decode batch into an 8-bit cache
        dict(name="cache write 23", op="cache", way="write", M=23, kv=4, D=128, bits=8, page=64, pad=0),
        # a padded batch of prompts into an 8-bit cache of small pages
        dict(name="cache write 4580", op="cache", way="write", M=4580, kv=4, D=128, bits=8, page=16, pad=120),
        # a cached prefix read back for a prompt that continues it
        dict(name="cache read 4571", op="cache", way="read", M=4571, kv=8, D=128, bits=8, page=64, pad=0),
        # 50 tokens of an action chunk that see each other and an 816-token prefix
        dict(name="prompt chunk 50", op="prompt", lens="50", more=816, q=8, kv=1, D=256, causal=False, layout="rows"),
        # one prefill chunk, straight from the qkv site
        dict(name="prompt 1024", op="prompt", lens="1024", more=0, q=28, kv=4, D=128, causal=True, layout="heads"),
        # a batch of ragged prompts of 4580 tokens, packed
        dict(name="prompt packed 4580", op="prompt", lens="1 811 50 2047 3 640 1024 4", more=0, q=28, kv=4, D=128, causal=True,
             layout="heads"),
        # a long context
        dict(name="prompt long 16384", op="prompt", lens="16384", more=0, q=28, kv=4, D=128, causal=True, layout="heads"),
        # one sequence's decode step after 1024 tokens
        dict(name="decode 1 x 1024", op="decode", lens="1024", q=28, kv=4, D=128, bits=16, page=64),
        # a serving batch of very different lengths, some of its places idle, 8-bit cache
        dict(name="decode 64 ragged", op="decode", lens=_ragged(61, 17, 8191, 23) + " 0 0 1", q=28, kv=4, D=128, bits=8, page=64),
        # one sequence with a very long cache
        dict(name="decode 1 x 131071", op="decode", lens="131071", q=32, kv=8, D=128, bits=16, page=256),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _lens(c):
    return [int(x) for x in c["lens"].split()]


def draw(rng):
    op = rng.choice(["heads", "cache", "prompt", "decode"])
    D = rng.choice([64, 80, 96, 128, 256])
    if op == "heads":
        while True:
            M, q, k = _log(rng, 1, 24571), rng.randint(1, 32), rng.randint(1, 8)
            if M * (q + 2 * k) * D <= 4571 * 36 * 128:
                break
        return dict(op=op, M=M, q=q, k=k, v=rng.choice([0, k]), D=D, rot=2 * rng.choice([D // 2, D // 4, D // 8]),
                    inter=rng.random() < 0.5, far=_log(rng, 1, 1000000), layout=rng.choice(["rows", "heads"]))
    kv = rng.choice([1, 2, 4, 5, 8])
    if op == "cache":
        while True:
            M = _log(rng, 1, 36571)
            if M * kv * D <= 4571 * 8 * 128:
                break
        return dict(op=op, way=rng.choice(["write", "read"]), M=M, kv=kv, D=D, bits=rng.choice([8, 16]),
                    page=16 * _log(rng, 1, 16), pad=rng.choice([0, _log(rng, 1, max(2, M // 4))]))
    q = kv * rng.choice([1, 2, 3, 4, 7, 8])
    if op == "prompt":
        while True:
            n = _log(rng, 1, 32)
            lens = [_log(rng, 1, 16384) for _ in range(n)]
            more = rng.choice([0, 0, _log(rng, 1, 4096)])
            if sum(x * (x + more) for x in lens) * q * D <= 16384 * 16384 * 14 * 128 and sum(lens) * q * D <= 1 << 28:
                break
        return dict(op=op, lens=" ".join(map(str, lens)), more=more, q=q, kv=kv, D=D, causal=rng.random() < 0.7,
                    layout=rng.choice(["rows", "heads"]))
    bits = rng.choice([8, 16])
    while True:
        n = _log(rng, 1, 128)
        top = _log(rng, 16, 131072)
        lens = [_log(rng, 1, top) if rng.random() < 0.95 else 0 for _ in range(n)]
        # (the padded batch too: the plain form reads every sequence up to the longest)
        if n * max(lens) * kv * D * bits <= 131071 * 8 * 128 * 16 and sum(lens) > 0:
            break
    return dict(op=op, lens=" ".join(map(str, lens)), q=q, kv=kv, D=D, bits=bits, page=16 * _log(rng, 1, 16))


def _seen(c):
    """Pairs of a query and a key that it sees, of one head."""
    return sum(n * (n + 1) // 2 + n * c["more"] if c["causal"] else n * (n + c["more"]) for n in _lens(c))


def _row_bytes(D, bits):
    """A token's key (or value) of one head in the cache."""
    return 2 * D if bits == 16 else D + 4


def work(case):
    c = case
    if c["op"] == "heads":
        n = c["M"] * (c["q"] + c["k"] + c["v"]) * c["D"]
        return {"bytes": 4 * n + 4 * c["M"] + 4 * c["rot"] + 8 * c["D"], "flops": 8 * n}
    if c["op"] == "cache":
        n = (c["M"] - c["pad"] * (c["way"] == "write")) * c["kv"] * 2
        return {"bytes": n * (2 * c["D"] + _row_bytes(c["D"], c["bits"])) + 4 * c["M"], "flops": 3 * n * c["D"]}
    if c["op"] == "prompt":
        n = sum(_lens(c))
        keys = n + c["more"] * len(_lens(c))
        return {"bytes": 2 * c["D"] * (2 * n * c["q"] + 2 * keys * c["kv"]), "flops": 4 * c["D"] * c["q"] * _seen(c)}
    n, keys = len(_lens(c)), sum(_lens(c))
    return {"bytes": 4 * n * c["q"] * c["D"] + 2 * keys * c["kv"] * _row_bytes(c["D"], c["bits"]) + 4 * n,
            "flops": 4 * c["D"] * c["q"] * keys}


# --------------------------------------------------------------------------------------------------------------- inputs
def _randn(g, *shape, scale=1.0):
    return (torch.randn(*shape, generator=g, device="cuda", dtype=F32) * scale).to(BF16)


def _cache(g, pages, kv, page, D, bits):
    """(rows or codes, scales) [pages][kv][page]... of a cache that is in use."""
    x = _randn(g, pages, kv, page, D)
    if bits == 16:
        return x, None
    s = x.abs().amax(-1).to(F32) / torch.tensor(E4M3_MAX, device="cuda")
    return (x.to(F32) / s.clamp_min(1e-30)[..., None]).clamp(-E4M3_MAX, E4M3_MAX).to(E4M3), s


def _offsets(lens):
    at = [0]
    for n in lens:
        at.append(at[-1] + n)
    return torch.tensor(at, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device="cuda").manual_seed(seed)
    D = c["D"]
    if c["op"] == "heads":
        M, H = c["M"], c["q"] + c["k"] + c["v"]
        x = _randn(g, H, M, D)
        x[: c["q"] + c["k"], :, ::16] *= 8.0  # q and k heads have a few large channels
        c["x"] = x if c["layout"] == "heads" else x.transpose(0, 1).contiguous()
        c["gq"] = torch.rand(D, generator=g, device="cuda") + 0.5
        c["gk"] = torch.rand(D, generator=g, device="cuda") + 0.5
        first = torch.randint(0, c["far"] + 1, (-(-M // 64),), generator=g, device="cuda")
        at = torch.arange(M, device="cuda")
        # one prompt counts from 0; the rows of a batch are runs that begin anywhere up to `far`
        c["pos"] = (first[at // 64] + at % 64 if c["far"] else at).to(torch.int32)
    elif c["op"] == "cache":
        M, kv, page = c["M"], c["kv"], c["page"]
        pages = -(-M // page) + 3
        c["pages"] = pages
        c["kc"], c["ks"] = _cache(g, pages, kv, page, D, c["bits"])
        c["vc"], c["vs"] = _cache(g, pages, kv, page, D, c["bits"])
        c["k"], c["v"] = _randn(g, kv, M, D), _randn(g, kv, M, D, scale=0.5)
        # consecutive tokens in pages that lie in any order; the tokens that only pad the batch have no slot
        order = torch.randperm(pages, generator=g, device="cuda")
        at = torch.arange(M, device="cuda")
        slots = order[at // page] * page + at % page
        if c["pad"]:
            slots[torch.randperm(M, generator=g, device="cuda")[: c["pad"]]] = -1
        c["slots"] = slots.to(torch.int32)
    elif c["op"] == "prompt":
        lens = _lens(c)
        n, keys = sum(lens), sum(lens) + c["more"] * len(lens)
        q, k, v = _randn(g, c["q"], n, D, scale=2.0), _randn(g, c["kv"], keys, D), _randn(g, c["kv"], keys, D)
        if c["layout"] == "rows":
            q, k, v = (t.transpose(0, 1).contiguous() for t in (q, k, v))
        c["qs"], c["ks"], c["vs"] = q, k, v
        c["cu"] = _offsets(lens)
        c["cuk"] = _offsets([x + c["more"] for x in lens]) if c["more"] else None
    else:
        lens, page = _lens(c), c["page"]
        width = -(-max(lens) // page)
        need = [-(-x // page) for x in lens]
        pages = sum(need) + 2
        c["pages"] = pages
        c["kc"], c["ks"] = _cache(g, pages, c["kv"], page, D, c["bits"])
        c["vc"], c["vs"] = _cache(g, pages, c["kv"], page, D, c["bits"])
        c["x"] = _randn(g, len(lens), c["q"], D, scale=2.0)
        order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
        table = torch.full((len(lens), width), -1, dtype=torch.int32, device="cuda")  # no page past a sequence's end
        at = 0
        for i, x in enumerate(need):
            table[i, :x] = order[at:at + x]
            at += x
        c["table"], c["lens_dev"] = table, torch.tensor(lens, dtype=torch.int32, device="cuda")
    return c


ROPE_BASE = 10000.0


# ---------------------------------------------------------------------------------------------------------- plain forms
def _by_head(t, layout):
    """[heads][M][D] view of heads in either layout."""
    return t if layout == "heads" else t.transpose(0, 1)


def _plain_heads(c):
    q, k, rot = c["q"], c["k"], c["rot"]
    x = _by_head(c["x"], c["layout"])
    f = x[: q + k].to(F32)
    r = 1.0 / torch.sqrt(f.to(F64).square().mean(-1, keepdim=True).to(F32) + 1e-6)
    gain = torch.cat((c["gq"].expand(q, 1, -1), c["gk"].expand(k, 1, -1)))
    f = f * r * gain
    i = torch.arange(rot // 2, dtype=F64, device="cuda")
    a = c["pos"].to(F64)[:, None] * ROPE_BASE ** (-2.0 * i / rot)
    cs, sn = torch.cos(a).to(F32), torch.sin(a).to(F32)
    part = f[..., :rot]
    if c["inter"]:
        u, w = part[..., 0::2], part[..., 1::2]
        new = torch.stack((u * cs - w * sn, w * cs + u * sn), -1).flatten(-2)
    else:
        u, w = part[..., : rot // 2], part[..., rot // 2:]
        new = torch.cat((u * cs - w * sn, w * cs + u * sn), -1)
    return torch.cat((torch.cat((new, f[..., rot:]), -1).to(BF16), x[q + k:]))  # [heads][M][D]


def _codes(h):
    s = h.abs().amax(-1) / torch.tensor(E4M3_MAX, device="cuda")
    v = torch.where(s[..., None] > 0, h / s[..., None], torch.zeros_like(h))
    return v.clamp(-E4M3_MAX, E4M3_MAX).to(E4M3), s


def _plain_cache(c):
    page = c["page"]
    if c["way"] == "write":
        at = c["slots"].to(torch.int64)
        ok = at >= 0
        at = at[ok]
        for x, rows, scales in ((c["k"], c["kc"], c["ks"]), (c["v"], c["vc"], c["vs"])):
            x = x.transpose(0, 1)[ok]  # [M][kv][D]
            if c["bits"] == 16:
                rows[at // page, :, at % page] = x
            else:
                codes, s = _codes(x.to(F32))
                rows.view(torch.uint8)[at // page, :, at % page] = codes.view(torch.uint8)
                scales[at // page, :, at % page] = s
        return {"k": c["kc"], "v": c["vc"], "k_scale": c["ks"], "v_scale": c["vs"]} if c["bits"] == 8 else \
            {"k": c["kc"], "v": c["vc"]}
    ok = (c["slots"] >= 0)[:, None, None]
    at = c["slots"].to(torch.int64).clamp_min(0)
    out = []
    for rows, scales in ((c["kc"], c["ks"]), (c["vc"], c["vs"])):
        bits8 = c["bits"] == 8
        x = (rows.view(torch.uint8) if bits8 else rows)[at // page, :, at % page]
        if bits8:
            x = (x.view(E4M3).to(F32) * scales[at // page, :, at % page][..., None]).to(BF16)
        out.append(torch.where(ok, x, torch.zeros_like(x)))
    return {"k": out[0], "v": out[1]}


def _plain_prompt(c):
    D, H, kv = c["D"], c["q"], c["kv"]
    q, k, v = (_by_head(c[n], c["layout"]) for n in ("qs", "ks", "vs"))
    out = torch.empty(q.shape[1], H, D, dtype=BF16, device="cuda")
    G = H // kv
    a = b = 0
    for n in _lens(c):
        m = n + c["more"]
        for h in range(kv):
            kk, vv = k[h, b:b + m].to(F32), v[h, b:b + m].to(F32)
            for i in range(0, n, 4096):  # rows at a time, for the room of their scores
                e = min(n, i + 4096)
                top = e + c["more"] if c["causal"] else m  # keys that any of these rows sees
                s = torch.matmul(q[h * G:(h + 1) * G, a + i:a + e].to(F32), kk[:top].t()) * D ** -0.5
                if c["causal"]:
                    row = torch.arange(i, e, device="cuda")[:, None] + c["more"]
                    s = s.masked_fill(torch.arange(top, device="cuda") > row, -math.inf)
                s = torch.exp(s - s.amax(-1, keepdim=True))
                o = torch.matmul(s, vv[:top]) / s.sum(-1, keepdim=True)
                out[a + i:a + e, h * G:(h + 1) * G] = o.transpose(0, 1).to(BF16)
        a, b = a + n, b + m
    return out


def _plain_decode(c):
    D, H, kv, page = c["D"], c["q"], c["kv"], c["page"]
    n, width = c["table"].shape
    at = c["table"].to(torch.int64).clamp_min(0)

    def rows(t, s):
        x = t.view(torch.uint8)[at].view(E4M3).to(F32) * s[at][..., None] if c["bits"] == 8 else t[at].to(F32)
        return x.transpose(1, 2).reshape(n, kv, width * page, D)

    hidden = (torch.arange(width * page, device="cuda") >= c["lens_dev"][:, None])[:, None, None]
    s = torch.matmul(c["x"].to(F32).view(n, kv, H // kv, D), rows(c["kc"], c["ks"]).transpose(2, 3)) * D ** -0.5
    s = s.masked_fill(hidden, -math.inf)
    s = torch.exp(s - s.amax(-1, keepdim=True).clamp_min(-1e30))
    o = torch.matmul(s, rows(c["vc"], c["vs"]))
    total = s.sum(-1, keepdim=True)
    return torch.where(total > 0, o / total, torch.zeros_like(o)).view(n, H, D).to(BF16)


# ------------------------------------------------------------------------------------------------- the framework's calls
def _strides(t, layout, D):
    """(elements from token to token, from head to head)"""
    return (D, t.shape[1] * D) if layout == "heads" else (t.shape[1] * D, D)


def _own_heads(c):
    import w4a4_integer_gemm_amd as fq
    M, H, D = c["M"], c["q"] + c["k"] + c["v"], c["D"]
    plan = c.get("plan")
    if plan is None:  # made once per model
        freq, grow = fq.fq_rope_freqs(c["rot"], ROPE_BASE)
        plan = c["plan"] = (torch.from_numpy(freq.view("int64")).cuda(), grow)
    y = torch.empty(H, M, D, dtype=BF16, device="cuda")
    token, head = _strides(c["x"], c["layout"], D)
    fq.fq_qk_norm_rope(c["x"], token, head, M, H, c["q"], c["k"], D, c["gq"], c["gk"], 1e-6, c["rot"], c["inter"], plan[0],
                       plan[1], c["pos"], 0, y, D, M * D)
    return y


def _own_cache(c):
    import w4a4_integer_gemm_amd as fq
    M, kv, D = c["M"], c["kv"], c["D"]
    if c["way"] == "write":
        fq.fq_kv_write(c["k"], D, M * D, c["v"], D, M * D, c["slots"], M, kv, D, c["bits"], c["pages"], c["page"], c["kc"],
                       c["vc"], c["ks"], c["vs"])
        return {"k": c["kc"], "v": c["vc"], "k_scale": c["ks"], "v_scale": c["vs"]} if c["bits"] == 8 else \
            {"k": c["kc"], "v": c["vc"]}
    k, v = (torch.empty(M, kv, D, dtype=BF16, device="cuda") for _ in range(2))
    fq.fq_kv_read(c["kc"], c["vc"], c["ks"], c["vs"], c["bits"], c["pages"], c["page"], c["slots"], M, kv, D, k, kv * D, D,
                  v, kv * D, D)
    return {"k": k, "v": v}


def _own_prompt(c):
    import w4a4_integer_gemm_amd as fq
    D, H, kv, lay = c["D"], c["q"], c["kv"], c["layout"]
    q, k, v = c["qs"], c["ks"], c["vs"]
    n, m = (t.shape[1 if lay == "heads" else 0] for t in (q, k))
    o = torch.empty(n, H, D, dtype=BF16, device="cuda")
    fq.fq_attn_prefill(q, *_strides(q, lay, D), k, *_strides(k, lay, D), v, *_strides(v, lay, D), n, m, c["cu"], c["cuk"],
                       c["cu"].numel() - 1, H, kv, D, D ** -0.5, c["causal"], o, H * D, D)
    return o


def _own_decode(c):
    import w4a4_integer_gemm_amd as fq
    D, H, kv, page = c["D"], c["q"], c["kv"], c["page"]
    n, width = c["table"].shape
    ws = c.get("ws")
    if ws is None:  # kept by the program, like the cache
        ws = c["ws"] = torch.empty(fq.fq_attn_decode_workspace_bytes(n, H, kv, D, width * page), dtype=torch.uint8, device="cuda")
    o = torch.empty(n, H, D, dtype=BF16, device="cuda")
    fq.fq_attn_decode(c["x"], H * D, D, n, H, kv, D, D ** -0.5, c["kc"], c["vc"], c["ks"], c["vs"], c["bits"], c["pages"], page,
                      c["table"], width, c["lens_dev"], o, H * D, D, ws, ws.numel())
    return o


def run(state):
    if own:
        return {"heads": _own_heads, "cache": _own_cache, "prompt": _own_prompt, "decode": _own_decode}[state["op"]](state)
    return {"heads": _plain_heads, "cache": _plain_cache, "prompt": _plain_prompt, "decode": _plain_decode}[state["op"]](state)


# ---------------------------------------------------------------------------------------------------- 64-bit definition
def _exact_heads(c):
    q, k, v, rot, D = c["q"], c["k"], c["v"], c["rot"], c["D"]
    x = c["x"].to(F64)
    x = x.clone() if c["layout"] == "heads" else x.permute(1, 0, 2).contiguous()
    n = x[: q + k]
    n /= (n.pow(2).sum(-1, keepdim=True) / D + 1e-6).sqrt()
    n[:q] *= c["gq"].to(F64)
    n[q:] *= c["gk"].to(F64)
    theta = ROPE_BASE ** (torch.arange(0, rot, 2, dtype=F64, device="cuda") / -rot)
    turn = torch.exp(1j * torch.outer(c["pos"].to(F64), theta))
    if c["inter"]:
        z = torch.view_as_complex(n[..., :rot].unflatten(-1, (-1, 2)).contiguous()) * turn
        n[..., :rot] = torch.view_as_real(z).flatten(-2)
    else:
        z = torch.complex(n[..., : rot // 2].contiguous(), n[..., rot // 2: rot].contiguous()) * turn
        n[..., : rot // 2], n[..., rot // 2: rot] = z.real, z.imag
    return x


def _exact_cache(c):
    page, out = c["page"], {}
    slots = c["slots"].tolist()
    if c["way"] == "read":
        keep = torch.tensor([s >= 0 for s in slots], device="cuda")
        flat = torch.tensor([max(s, 0) for s in slots], device="cuda")
        for name in ("k", "v"):
            t = c[name + "c"].to(F64)
            if c["bits"] == 8:
                t = t * c[name + "s"].to(F64).unsqueeze(-1)
            t = t.permute(0, 2, 1, 3).reshape(-1, c["kv"], c["D"])  # token after token
            out[name] = t.index_select(0, flat) * keep[:, None, None]
        return out
    src = torch.tensor([i for i, s in enumerate(slots) if s >= 0], device="cuda")
    dst = torch.tensor([s for s in slots if s >= 0], device="cuda")
    for name in ("k", "v"):
        t, s = c[name + "c"], c[name + "s"]
        all_rows = t.to(F64).permute(0, 2, 1, 3).reshape(-1, c["kv"], c["D"]).clone()
        new = c[name].to(F64).permute(1, 0, 2).index_select(0, src)
        if c["bits"] == 8:
            # the scale and the quotient are float32 values by definition
            scale = (new.abs().max(-1).values / 448).to(F32).to(F64)
            each = scale.unsqueeze(-1)
            new = torch.where(each > 0, new / each, 0.0).to(F32).clamp(-448, 448).to(E4M3).to(F64)
            flat = s.to(F64).permute(0, 2, 1).reshape(-1, c["kv"]).clone()
            flat[dst] = scale
            out[name + "_scale"] = flat.view(-1, page, c["kv"]).permute(0, 2, 1).contiguous()
        all_rows[dst] = new
        out[name] = all_rows.view(-1, page, c["kv"], c["D"]).permute(0, 2, 1, 3).contiguous()
    return {n: out[n] for n in ("k", "v", "k_scale", "v_scale") if n in out}


def _attend64(q, k, v, last):
    """Rows q [n][D] over keys 0 .. last[i] (inclusive) of k and v [m][D], 64 bits."""
    w = torch.mm(q, k.t()) / math.sqrt(q.shape[1])
    w.masked_fill_(last[:, None] < torch.arange(k.shape[0], device="cuda"), -math.inf)
    w -= torch.logsumexp(w, 1, keepdim=True)
    return torch.mm(w.exp_(), v)


def _exact_prompt(c):
    lay, G = c["layout"], c["q"] // c["kv"]
    q, k, v = (c[n].to(F64) if lay == "heads" else c[n].to(F64).permute(1, 0, 2) for n in ("qs", "ks", "vs"))
    o = torch.zeros_like(q)
    starts, at = [], 0
    for n in _lens(c):
        starts.append((at, n))
        at += n
    for j, (a, n) in enumerate(starts):
        b, m = a + j * c["more"], n + c["more"]
        see = torch.arange(n, device="cuda") + c["more"] if c["causal"] else torch.full((n,), m - 1, device="cuda")
        for h in range(c["q"]):
            for i in range(0, n, 2048):
                part = slice(i, min(i + 2048, n))
                end = min(m, part.stop + c["more"]) if c["causal"] else m
                o[h, a:a + n][part] = _attend64(q[h, a:a + n][part], k[h // G, b:b + end], v[h // G, b:b + end], see[part])
    return o.permute(1, 0, 2).contiguous()


def _exact_decode(c):
    G, D = c["q"] // c["kv"], c["D"]
    o = torch.zeros(len(_lens(c)), c["q"], D, dtype=F64, device="cuda")
    for i, n in enumerate(_lens(c)):
        if n == 0:
            continue
        pages = c["table"][i, : -(-n // c["page"])].long()
        kv = []
        for name in ("k", "v"):
            t = (c[name + "c"].view(torch.uint8)[pages].view(E4M3) if c["bits"] == 8 else c[name + "c"][pages]).to(F64)
            if c["bits"] == 8:
                t *= c[name + "s"][pages].to(F64).unsqueeze(-1)
            kv.append(t.permute(1, 0, 2, 3).reshape(c["kv"], -1, D)[:, :n])
        for h in range(c["kv"]):
            last = torch.full((G,), n - 1, device="cuda")
            o[i, h * G:(h + 1) * G] = _attend64(c["x"][i, h * G:(h + 1) * G].to(F64), kv[0][h], kv[1][h], last)
    return o


def exact(case, seed):
    c = prepare(case, seed)
    return {"heads": _exact_heads, "cache": _exact_cache, "prompt": _exact_prompt, "decode": _exact_decode}[c["op"]](c)
