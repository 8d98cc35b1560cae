"""The operators of a transformer block next to the quantised linear sites, as workloads that can be timed and checked.

Three operators, each in a plain form (elementary torch operations) and as the call that a user makes:

fp8_linear   y = deq(quant(norm(x))) . deq(W)^T [+ bias] [+ residual], 8-bit floating point (e4m3) codes with one float32
             scale for every 128 consecutive k of a token and every 128 x 128 block of the weight
block_norm   the stream r' = r + c * gate * norm(x; g_post), and the next block's input norm(r'; g_pre) * (1 + scale) + shift
             as bf16 or as e4m3 codes with their scales
rope         rotary positions on the q and k heads of a qkv output, v heads copied

`own` selects the framework's calls.
"""
import math

import torch

own = False

E4M3_MAX = 448.0
GROUP = 128
F32, F64 = torch.float32, torch.float64


# ---------------------------------------------------------------------------------------------------------------- cases
def listed():
    return [
        # one token through the wide gate+up layer of a decode step: 136 MB of weights for one row
        dict(name="fp8 decode 1 wide", op="fp8_linear", M=1, K=3584, N=37888, norm=True, residual=False, bias=False, head_dim=0),
        # a small layer on a few tokens (the smallest site of the tests): latency counts
        dict(name="fp8 tiny 16", op="fp8_linear", M=16, K=256, N=512, norm=True, residual=False, bias=True, head_dim=0),
        # a decode batch through a down projection with the residual
        dict(name="fp8 decode 23 down", op="fp8_linear", M=23, K=16384, N=2048, norm=False, residual=True, bias=False, head_dim=0),
        # a prefill chunk through the fused qkv layer, written in the head layout
        dict(name="fp8 qkv 1024", op="fp8_linear", M=1024, K=3584, N=4608, norm=True, residual=False, bias=True, head_dim=128),
        # a ragged prefill through the down projection with the residual
        dict(name="fp8 down 811", op="fp8_linear", M=811, K=16384, N=2048, norm=False, residual=True, bias=False, head_dim=0),
        # a long prompt through the gate+up layer
        dict(name="fp8 gateup 4096", op="fp8_linear", M=4096, K=3584, N=37888, norm=True, residual=False, bias=False, head_dim=0),
        # one token between two blocks: norms on both sides, gated
        dict(name="norm token", op="block_norm", M=1, K=2048, post=True, gate=True, mod=True, f32=False, out="bf16", per=1, scale=1.0),
        # a prefill chunk between two blocks of a model that norms on both sides, into e4m3 codes for the next site
        dict(name="norm prefill fp8", op="block_norm", M=1024, K=3584, post=True, gate=False, mod=False, f32=False, out="fp8", per=1, scale=1.0),
        # a conditioned block over a padded batch of 50 tokens a sequence, the stream held in float32
        dict(name="norm gated batch f32", op="block_norm", M=12800, K=2048, post=False, gate=True, mod=True, f32=True, out="bf16", per=50, scale=0.5),
        # one token's q and k heads far into a context
        dict(name="rope token", op="rope", M=1, heads=12, rot_heads=10, D=256, rot=256, inter=False, kind="plain", far=100003, inverse=False),
        # a prefill chunk's qkv rows into the head layout, positions scaled for a long context
        dict(name="rope prefill 1024", op="rope", M=1024, heads=36, rot_heads=32, D=128, rot=128, inter=False, kind="ramp", far=70001, inverse=False),
        # a long ragged batch, interleaved pairs on part of the head, undone again
        dict(name="rope part 24571", op="rope", M=24571, heads=18, rot_heads=17, D=80, rot=32, inter=True, kind="linear", far=500000, inverse=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["fp8_linear", "block_norm", "rope"])
    if op == "fp8_linear":
        while True:
            M, K, N = _log(rng, 1, 4096), GROUP * _log(rng, 2, 148), 8 * _log(rng, 32, 4736)
            if M * K * N <= 4096 * 3584 * 37888:
                break
        heads = rng.random() < 0.25
        if heads:
            N = max(GROUP, N // GROUP * GROUP)
        return dict(op=op, M=M, K=K, N=N, norm=rng.random() < 0.5, residual=rng.random() < 0.5, bias=rng.random() < 0.5,
                    head_dim=rng.choice([64, 128]) if heads else 0)
    if op == "block_norm":
        while True:
            M, fp8 = _log(rng, 1, 12800), rng.random() < 0.4
            K = GROUP * _log(rng, 1, 148) if fp8 else 8 * _log(rng, 8, 2368)
            if M * K <= 12800 * 2048:
                break
        return dict(op=op, M=M, K=K, post=rng.random() < 0.6, gate=rng.random() < 0.5, mod=rng.random() < 0.5,
                    f32=rng.random() < 0.4, out="fp8" if fp8 else "bf16", per=_log(rng, 1, max(1, M)), scale=rng.choice([1.0, 0.5, 0.1]))
    D = rng.choice([64, 80, 96, 128, 192, 256])
    rot_heads = rng.randint(1, 40)
    heads = rot_heads + rng.randint(0, 8)
    while True:
        M = _log(rng, 1, 24571)
        if M * heads * D <= 24571 * 18 * 80:
            break
    return dict(op=op, M=M, heads=heads, rot_heads=rot_heads, D=D, rot=2 * rng.choice([D // 2, D // 4, D // 8]),
                inter=rng.random() < 0.5, kind=rng.choice(["plain", "linear", "base", "bands", "ramp"]), far=_log(rng, 1, 1000000),
                inverse=rng.random() < 0.3)


def work(case):
    c = case
    if c["op"] == "fp8_linear":
        M, K, N = c["M"], c["K"], c["N"]
        b = 2 * M * K + N * K + 4 * (-(-N // GROUP)) * (K // GROUP) + 2 * M * N
        b += 4 * K * c["norm"] + 2 * M * N * c["residual"] + 4 * N * c["bias"]
        return {"bytes": b, "flops": 2 * M * N * K}
    if c["op"] == "block_norm":
        M, K = c["M"], c["K"]
        conds = -(-M // c["per"])
        b = 2 * M * K + 2 * (4 if c["f32"] else 2) * M * K + 4 * K * (1 + c["post"]) + 2 * K * conds * (c["gate"] + 2 * c["mod"])
        b += M * K + 4 * M * K // GROUP if c["out"] == "fp8" else 2 * M * K
        return {"bytes": b, "flops": 12 * M * K}
    n = c["M"] * c["heads"] * c["D"]
    return {"bytes": 4 * n + 4 * c["M"] + 4 * c["rot"], "flops": 3 * c["M"] * c["rot_heads"] * c["rot"]}


# --------------------------------------------------------------------------------------------------------------- inputs
def _randn(g, *shape, dtype=F32):
    return torch.randn(*shape, generator=g, device="cuda", dtype=F32).to(dtype)


def _block_scaled(w):
    """Weight rows as e4m3 codes with a float32 scale for each 128 x 128 block, as a stored checkpoint holds them."""
    N, K = w.shape
    nb = -(-N // GROUP)
    full = torch.zeros(nb * GROUP, K, device=w.device)
    full[:N] = w
    blocks = full.view(nb, GROUP, K // GROUP, GROUP)
    s = blocks.abs().amax((1, 3)) / torch.tensor(E4M3_MAX, device=w.device)
    q = (blocks / s.clamp_min(1e-30)[:, None, :, None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
    return q.view(nb * GROUP, K)[:N].contiguous(), s.contiguous()


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device="cuda").manual_seed(seed)
    if c["op"] == "fp8_linear":
        M, K, N = c["M"], c["K"], c["N"]
        x = _randn(g, M, K)
        hot = torch.randint(0, K, (max(1, K // 100),), generator=g, device="cuda")
        x[:, hot] *= 20.0  # activations of such layers have a few large channels
        c["x"] = x.to(torch.bfloat16)
        c["codes"], c["wscale"] = _block_scaled(_randn(g, N, K) * 0.02)
        c["gamma"] = torch.rand(K, generator=g, device="cuda") + 0.5 if c["norm"] else None
        c["b"] = _randn(g, N) * 0.1 if c["bias"] else None
        c["res"] = _randn(g, M, N, dtype=torch.bfloat16) if c["residual"] else None
    elif c["op"] == "block_norm":
        M, K = c["M"], c["K"]
        conds = -(-M // c["per"])
        c["x"] = _randn(g, M, K, dtype=torch.bfloat16)
        c["r"] = (_randn(g, M, K) * 3.0).to(F32 if c["f32"] else torch.bfloat16)
        c["g_post"] = torch.rand(K, generator=g, device="cuda") + 0.5 if c["post"] else None
        c["g_pre"] = torch.rand(K, generator=g, device="cuda") + 0.5
        cond = (_randn(g, conds, 3 * K) * 0.3).to(torch.bfloat16)  # one projection of the condition: [scale | shift | gate]
        c["s"], c["t"] = (cond[:, :K], cond[:, K:2 * K]) if c["mod"] else (None, None)
        c["g"] = cond[:, 2 * K:] if c["gate"] else None
    else:
        M, H, D = c["M"], c["heads"], c["D"]
        c["x"] = _randn(g, M, H * D, dtype=torch.bfloat16)
        # the rows of a batch sit at positions of their own: runs that begin anywhere up to `far`
        first = torch.randint(0, c["far"] + 1, (-(-M // 64),), generator=g, device="cuda")
        at = torch.arange(M, device="cuda")
        c["pos"] = (first[at // 64] + at % 64).to(torch.int32)
    return c


# ------------------------------------------------------------------------------------------------ rotary frequencies
ROPE_BASE, ROPE_FACTOR, ROPE_LEN = 10000.0, 8.0, 8192  # base, context factor and trained length of the scaled forms


def _angles_per_position(kind, rot):
    """(float64 radians per position of each pair, factor on cos and sin) of a scaling rule."""
    i = torch.arange(rot // 2, dtype=F64, device="cuda")
    th = ROPE_BASE ** (-2.0 * i / rot)
    if kind == "linear":
        return th / ROPE_FACTOR, 1.0
    if kind == "base":
        return (ROPE_BASE * ROPE_FACTOR ** (rot / (rot - 2.0))) ** (-2.0 * i / rot), 1.0
    if kind == "bands":  # long waves stretched, short ones kept, a linear blend between
        turns = ROPE_LEN * th / (2 * math.pi)  # over the trained length
        keep = ((turns - 1.0) / (4.0 - 1.0)).clamp(0.0, 1.0)
        return th * (keep + (1.0 - keep) / ROPE_FACTOR), 1.0
    if kind == "ramp":  # a ramp over the pair index between the pairs of 32 and of 1 turns; cos and sin grow with log(factor)
        at = [rot * math.log(ROPE_LEN / (n * 2 * math.pi)) / (2 * math.log(ROPE_BASE)) for n in (32.0, 1.0)]
        lo, hi = max(math.floor(at[0]), 0), min(math.ceil(at[1]), rot - 1)
        ramp = ((i - lo) / max(hi - lo, 0.001)).clamp(0.0, 1.0)
        return th * (1.0 - ramp) + th / ROPE_FACTOR * ramp, 0.1 * math.log(ROPE_FACTOR) + 1.0
    return th, 1.0


# ---------------------------------------------------------------------------------------------------------- plain forms
def _rms(x, eps):
    """1 / rms of each row in float32, from a float64 sum of squares."""
    ms = x.to(F64).square().mean(-1, keepdim=True).to(F32)
    return 1.0 / torch.sqrt(ms + eps)


def _group_codes(h):
    """(e4m3 codes [M][K], scales [M][K / 128]) of float32 rows."""
    M, K = h.shape
    v = h.view(M, K // GROUP, GROUP)
    s = v.abs().amax(-1) / torch.tensor(E4M3_MAX, device=h.device)
    q = torch.where(s[..., None] > 0, v / s[..., None], torch.zeros_like(v))
    return q.clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).view(M, K), s


def _plain_fp8(c):
    M, K, N = c["M"], c["K"], c["N"]
    h = c["x"].to(F32)
    if c["norm"]:
        h = h * _rms(h, 1e-6) * c["gamma"]
    q, s = _group_codes(h)
    a = (q.to(F32).view(M, K // GROUP, GROUP) * s[..., None]).view(M, K)
    w = c["codes"].to(F32) * c["wscale"].repeat_interleave(GROUP, 0)[:N].repeat_interleave(GROUP, 1)
    y = a @ w.t()
    if c["bias"]:
        y = y + c["b"]
    if c["residual"]:
        y = y + c["res"].to(F32)
    y = y.to(torch.bfloat16)
    return y.view(M, N // c["head_dim"], c["head_dim"]).transpose(0, 1).contiguous() if c["head_dim"] else y


def _plain_norm(c):
    M, per = c["M"], c["per"]
    row = torch.arange(M, device="cuda") // per
    p = c["x"].to(F32)
    if c["post"]:
        p = p * _rms(p, 1e-6) * c["g_post"]
    if c["gate"]:
        p = p * c["g"][row].to(F32)
    r = (c["r"].to(F32) + c["scale"] * p).to(c["r"].dtype)
    h = r.to(F32)
    h = h * _rms(h, 1e-6) * c["g_pre"]
    if c["mod"]:
        h = h * (1.0 + c["s"][row].to(F32)) + c["t"][row].to(F32)
    if c["out"] == "fp8":
        q, s = _group_codes(h)
        return {"stream": r, "codes": q, "scales": s.t().contiguous()}
    return {"stream": r, "h": h.to(torch.bfloat16)}


def _rotate(x, c, cs, sn):
    """x [M][heads][D] rotated by cos and sin [M][1][rot / 2]."""
    rot = c["rot"]
    part = x[..., :rot]
    if c["inverse"]:
        sn = -sn
    if c["inter"]:
        a, b = part[..., 0::2], part[..., 1::2]
        new = torch.stack((a * cs - b * sn, b * cs + a * sn), -1).flatten(-2)
    else:
        a, b = part[..., :rot // 2], part[..., rot // 2:]
        new = torch.cat((a * cs - b * sn, b * cs + a * sn), -1)
    return torch.cat((new, x[..., rot:]), -1)


def _plain_rope(c):
    M, H, D, R = c["M"], c["heads"], c["D"], c["rot_heads"]
    th, grow = _angles_per_position(c["kind"], c["rot"])
    a = c["pos"].to(F64)[:, None] * th
    cs, sn = (torch.cos(a) * grow).to(F32)[:, None], (torch.sin(a) * grow).to(F32)[:, None]
    x = c["x"].view(M, H, D)
    y = torch.cat((_rotate(x[:, :R].to(F32), c, cs, sn).to(torch.bfloat16), x[:, R:]), 1)
    return y.transpose(0, 1).contiguous()  # [heads][M][D]


# ------------------------------------------------------------------------------------------------- the framework's calls
def _own_fp8(c):
    import w4a4_integer_gemm_amd as fq
    M, K, N, hd = c["M"], c["K"], c["N"], c["head_dim"]
    ws = c.get("ws")
    if ws is None:  # kept by the program, like the weights
        ws = c["ws"] = torch.empty(fq.fq_fp8_linear_workspace_bytes(M, K), dtype=torch.uint8, device="cuda")
    x, res = c["x"], c["res"]
    y = torch.empty((N // hd, M, hd) if hd else (M, N), dtype=torch.bfloat16, device="cuda")
    fq.fq_fp8_linear(x, M, K, K, c["gamma"], 1e-6, c["codes"], c["wscale"], N, c["b"], res, N, hd, y, N, ws, ws.numel())
    return y


def _own_norm(c):
    import w4a4_integer_gemm_amd as fq
    M, K = c["M"], c["K"]
    r = torch.empty_like(c["r"])
    h = q = s = None
    if c["out"] == "fp8":
        ld = (M + 3) // 4 * 4
        q = torch.empty(M, K, dtype=torch.float8_e4m3fn, device="cuda")
        s = torch.empty(K // GROUP, ld, device="cuda")
    else:
        h = torch.empty(M, K, dtype=torch.bfloat16, device="cuda")
    fq.fq_block_norm(M, K, c["x"], K, c["g_post"], 1e-6, c["g"], 3 * K, c["scale"], c["r"], K, r, K, c["f32"],
                     c["g_pre"], 1e-6, c["s"], c["t"], 3 * K, c["per"], h, K, q, s)
    return {"stream": r, "codes": q, "scales": s[:, :M]} if h is None else {"stream": r, "h": h}


def _own_rope(c):
    import w4a4_integer_gemm_amd as fq
    M, H, D = c["M"], c["heads"], c["D"]
    plan = c.get("plan")
    if plan is None:  # made once per model
        kind = {"plain": fq.ROPE_PLAIN, "linear": fq.ROPE_LINEAR, "base": fq.ROPE_BASE, "bands": fq.ROPE_BANDS,
                "ramp": fq.ROPE_RAMP}[c["kind"]]
        low, high = (1.0, 4.0) if c["kind"] == "bands" else (1.0, 32.0)
        freq, grow = fq.fq_rope_freqs(c["rot"], ROPE_BASE, kind, ROPE_FACTOR, ROPE_LEN, low, high)
        plan = c["plan"] = (torch.from_numpy(freq.view("int64")).cuda(), grow)
    y = torch.empty(H, M, D, dtype=torch.bfloat16, device="cuda")
    fq.fq_rope(c["x"], H * D, D, M, H, c["rot_heads"], D, c["rot"], c["inter"], plan[0], plan[1], c["pos"], 0,
               c["inverse"], y, D, M * D)
    return y


def run(state):
    if own:
        return {"fp8_linear": _own_fp8, "block_norm": _own_norm, "rope": _own_rope}[state["op"]](state)
    return {"fp8_linear": _plain_fp8, "block_norm": _plain_norm, "rope": _plain_rope}[state["op"]](state)


# ---------------------------------------------------------------------------------------------------- 64-bit definition
def _unit64(v, eps):
    return v / (v.pow(2).sum(-1, keepdim=True) / v.shape[-1] + eps).sqrt()


def _scaled64(h):
    """(codes, scales) by the definition: the scale is the float32 nearest max / 448, the code the e4m3 nearest h / scale."""
    top = h.unflatten(-1, (-1, GROUP)).abs().max(-1).values
    s = (top / 448).to(F32).to(F64)
    each = s.repeat_interleave(GROUP, -1)
    return torch.where(each > 0, h / each, 0.0).clamp(-448, 448).to(torch.float8_e4m3fn), s


def exact(case, seed):
    c = prepare(case, seed)
    if c["op"] == "fp8_linear":
        h = c["x"].to(F64)
        if c["norm"]:
            h = _unit64(h, 1e-6) * c["gamma"].to(F64)
        q, s = _scaled64(h)
        w = c["codes"].to(F64)
        w *= c["wscale"].to(F64).repeat_interleave(GROUP, 1).repeat_interleave(GROUP, 0)[: c["N"]]
        y = torch.mm(q.to(F64) * s.repeat_interleave(GROUP, 1), w.t())
        y = y + (c["b"].to(F64) if c["bias"] else 0.0) + (c["res"].to(F64) if c["residual"] else 0.0)
        return y.unflatten(1, (-1, c["head_dim"])).permute(1, 0, 2).contiguous() if c["head_dim"] else y
    if c["op"] == "block_norm":
        at = torch.div(torch.arange(c["M"], device="cuda"), c["per"], rounding_mode="floor")
        v = c["x"].to(F64)
        v = _unit64(v, 1e-6) * c["g_post"].to(F64) if c["post"] else v
        v = v * c["g"].to(F64).index_select(0, at) if c["gate"] else v
        r = c["r"].to(F64) + c["scale"] * v
        # the norm reads the stream as it is stored
        h = _unit64(r.to(c["r"].dtype).to(F64), 1e-6) * c["g_pre"].to(F64)
        if c["mod"]:
            h = h + h * c["s"].to(F64).index_select(0, at) + c["t"].to(F64).index_select(0, at)
        if c["out"] == "fp8":
            q, s = _scaled64(h)
            return {"stream": r, "codes": q, "scales": s.t().contiguous()}
        return {"stream": r, "h": h}
    M, H, D, rot = c["M"], c["heads"], c["D"], c["rot"]
    th, grow = _angles_per_position(c["kind"], rot)
    turn = torch.polar(torch.full((M, rot // 2), grow, dtype=F64, device="cuda"), torch.outer(c["pos"].to(F64), th))
    turn = (turn.conj() if c["inverse"] else turn)[None]
    y = c["x"].to(F64).view(M, H, D).permute(1, 0, 2).contiguous()
    part = y[: c["rot_heads"], :, :rot].clone()
    if c["inter"]:
        z = torch.view_as_complex(part.unflatten(-1, (-1, 2)).contiguous()) * turn
        new = torch.view_as_real(z).flatten(-2)
    else:
        z = torch.complex(part[..., : rot // 2], part[..., rot // 2:]) * turn
        new = torch.cat((z.real, z.imag), -1)
    y[: c["rot_heads"], :, :rot] = new
    return y
