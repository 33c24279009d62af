"""Measured cases of the 4-bit operators and of gradient clipping: rows and
weights rounded to MXFP4 (E2M1 codes, one E8M0 scale per 32 columns) and read
back, the experts' products with such weights and bf16 or MXFP4 rows, the rows'
gradient through them, and a whole set of gradients clipped by its norm.

With ``own`` false every operator runs in its plain form, elementary torch
operations in float32 (64-bit sums where they are long); with ``own`` true it
runs through this package's entry points.  Both take the same state.
"""

import math

import torch

own = False

MX = 32            # columns that share one scale byte
MAX_NORM = 1.0


# ------------------------------------------------------------------- cases --

def listed():
    return [
        # rows of a decode batch rounded to 4 bits on their way to their experts
        dict(name="quantize_decode", op="quantize", src="bf16", M=8, H=2048, E=128, k=8, BS=16, skew=0.0, drop=0.0, pitch=0),
        # rows of a prefill chunk, each to its eight experts
        dict(name="quantize_prefill", op="quantize", src="bf16", M=4096, H=2048, E=128, k=8, BS=16, skew=0.5, drop=0.0, pitch=0),
        # float32 master weights of one projection rounded again after an optimizer's step, with the values the step's
        # gradient is taken at
        dict(name="quantize_weights_train", op="quantize", src="f32", M=128 * 768, H=2048, E=0, k=1, BS=1, skew=0.0, drop=0.0, pitch=0),
        # a decode batch through the experts' gate and up weights in 4 bits, bf16 rows
        dict(name="linear_decode", op="linear", M=8, E=128, k=8, BS=16, K=2048, N=768, act="swiglu", bias=False, residual=False,
             rows4=False, save=False, skew=0.0, drop=0.0),
        # few tokens over experts of awkward sizes, some experts without a token
        dict(name="linear_ragged", op="linear", M=777, E=12, k=2, BS=1, K=992, N=520, act="gelu", bias=True, residual=False,
             rows4=False, save=True, skew=2.0, drop=0.05),
        # gate and up of a training step on 4-bit weights, pre-activations kept for the gradient
        dict(name="linear_train", op="linear", M=4096, E=128, k=8, BS=16, K=2048, N=768, act="swiglu", bias=False, residual=False,
             rows4=False, save=True, skew=0.5, drop=0.0),
        # the same products of a prefill chunk with 4-bit rows as well
        dict(name="linear_rows4_prefill", op="linear", M=4096, E=128, k=8, BS=16, K=2048, N=768, act="swiglu", bias=False,
             residual=False, rows4=True, save=False, skew=0.5, drop=0.0),
        # a dense projection of a wide model, rows and weights in 4 bits, the residual stream added
        dict(name="linear_rows4_dense", op="linear", M=8192, E=0, k=1, BS=1, K=7168, N=2048, act="none", bias=True, residual=True,
             rows4=True, save=False, skew=0.0, drop=0.0),
        # a few tokens' rows' gradient through 4-bit weights (fine-tuning on short texts)
        dict(name="backward_short", op="backward", M=300, E=8, k=2, BS=16, K=1056, N=264, gated=False, skew=1.0, drop=0.05),
        # the rows' gradient of the gate and up products of a training step
        dict(name="backward_train", op="backward", M=4096, E=128, k=8, BS=16, K=2048, N=768, gated=True, skew=0.5, drop=0.0),
        # the small gradients of a few layers: routers, norms, biases and two small experts each
        dict(name="clip_small", op="clip", layers=8, E=2, H=256, N=128, dw="bf16", flat=False, clip=True),
        # a whole expert block's gradients
        dict(name="clip_block", op="clip", layers=1, E=128, H=2048, N=768, dw="bf16", flat=False, clip=True),
    ]


def _log(rng, lo, hi):
    """A whole number from lo to hi, spread over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["quantize", "quantize", "linear", "linear", "linear", "linear", "backward", "backward", "clip", "clip"])
    if op == "clip":
        layers, E = rng.randint(1, 8), _log(rng, 1, 64)
        H = _log(rng, 32, 2048)
        N = _log(rng, 16, max(16, min(1024, 100_000_000 // (layers * E * H))))
        return dict(op=op, layers=layers, E=E, H=H, N=N, dw=rng.choice(["bf16", "f32"]), flat=rng.random() < 0.4,
                    clip=rng.random() < 0.7)
    E = rng.choice([0, 1, _log(rng, 2, 128), _log(rng, 2, 128)])
    k = 1 if E <= 1 else rng.randint(1, min(8, E))
    M = _log(rng, 1, max(1, 32768 // k))
    case = dict(op=op, M=M, E=E, k=k, BS=1 if E == 0 else rng.choice([1, 16, 64]), skew=rng.choice([0.0, 0.5, 1.0]),
                drop=0.0 if E <= 1 else rng.choice([0.0, 0.1]))
    if op == "quantize":
        case.update(src=rng.choice(["bf16", "f32"]), H=MX * _log(rng, 1, 128), pitch=rng.choice([0, 0, 8, 5]))
        return case
    case.update(K=MX * _log(rng, 2, 64), N=8 * _log(rng, 8, 128))
    if op == "backward":
        case.update(gated=rng.random() < 0.5)
        return case
    act = rng.choice(["none", "silu", "gelu", "swiglu", "swiglu"])
    case.update(act=act, bias=rng.random() < 0.5, residual=rng.random() < 0.4, rows4=rng.random() < 0.5,
                save=act != "none" and rng.random() < 0.4)
    return case


# ------------------------------------------------------------------ inputs --

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(g, *shape, scale=1.0, dtype=torch.bfloat16):
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)


def _max_total(n, E, BS):
    bound = min(n * BS, n + E * (BS - 1))
    return -(-bound // BS) * BS


def _route(case, g):
    """What the router and the alignment hand over: each slot's sorted position
    (-1: dropped), the experts' first rows and row counts."""
    M, E, k, BS = case["M"], case["E"], case["k"], case["BS"]
    if E == 0:  # a dense projection: no experts, every row
        return dict(rows=M, cap=M, offsets=None, counts=None, perm=None)
    logits = torch.randn(M, E, generator=g, device="cuda") + case["skew"] * torch.randn(E, generator=g, device="cuda")
    ids = torch.topk(logits, k, dim=1).indices
    gone = torch.rand(M, k, generator=g, device="cuda") < case["drop"]
    key = torch.where(gone, E, ids).reshape(-1)
    n = M * k
    order = torch.argsort(key, stable=True)
    counts = torch.bincount(key, minlength=E + 1)
    first = torch.cumsum(counts, 0) - counts
    padded = (counts[:E] + BS - 1) // BS * BS
    offsets = torch.zeros(E + 1, dtype=torch.int64, device="cuda")
    offsets[1:] = torch.cumsum(padded, 0)
    skey = key[order]
    pos = torch.where(skey < E, offsets[skey] + torch.arange(n, device="cuda") - first[skey], -1)
    perm = torch.empty(n, dtype=torch.int32, device="cuda")
    perm[order] = pos.to(torch.int32)
    return dict(rows=_max_total(n, E, BS), cap=max(1, int(counts[:E].max())), offsets=offsets.to(torch.int32),
                counts=counts[:E].to(torch.int32), perm=perm)


def _codes(v):
    """Float rows as MXFP4: packed codes [..., C/2], scale bytes [..., C/32]."""
    b = v.float().reshape(*v.shape[:-1], -1, MX)
    amax = b.abs().amax(-1)
    # the exponent field less 2, the exponent of the largest code: the block's maximum lands in [4, 8)
    field = amax.view(torch.int32) >> 23
    byte = torch.where(field == 255, 255, torch.where(amax == 0, 127, torch.clamp(field - 2, min=2)))
    m = b.abs() / torch.exp2((byte - 127).float())[..., None]
    # nearest code, ties to the even one
    code = ((m > 0.25).to(torch.uint8) + (m >= 0.75) + (m > 1.25) + (m >= 1.75) + (m > 2.5) + (m >= 3.5) + (m > 5)).to(torch.uint8)
    code = (code | ((b < 0).to(torch.uint8) << 3)).reshape(v.shape)
    return code[..., 0::2] | (code[..., 1::2] << 4), byte.to(torch.uint8)


def _values(codes, scales):
    """What packed codes and scale bytes stand for, float32."""
    table = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0], device="cuda")
    v = torch.stack([table[(codes & 15).int()], table[(codes >> 4).int()]], -1).reshape(*codes.shape[:-1], -1, MX)
    return (v * torch.exp2(scales.float() - 127)[..., None]).reshape(*codes.shape[:-1], -1)


def _weight4(g, E, N, K):
    return _codes(torch.randn(E, N, K, generator=g, device="cuda") * (K ** -0.5))


def _gradients(case, g):
    """A block's gradients, layer by layer: the experts' three weights (of the type
    the products return), the router's, the experts' bias and the norm's."""
    E, H, N = case["E"], case["H"], case["N"]
    kind = torch.float32 if case["dw"] == "f32" else torch.bfloat16
    shapes = [((E, N, H), kind), ((E, N, H), kind), ((E, H, N), kind), ((E, H), torch.bfloat16), ((E, N), torch.float32),
              ((H,), torch.float32)] * case["layers"]
    total = sum(math.prod(s) for s, _ in shapes)
    scale = (20.0 if case["clip"] else 0.5) * MAX_NORM / math.sqrt(total)
    if not case["flat"]:
        return [_randn(g, *s, scale=scale, dtype=t) for s, t in shapes]
    # slices of one buffer per type, as a bucket of gradients holds them, at any element
    pools = {t: _randn(g, 1 + sum(math.prod(s) for s, u in shapes if u == t), scale=scale, dtype=t) for t in {u for _, u in shapes}}
    at, grads = {t: 1 for t in pools}, []
    for s, t in shapes:
        n = math.prod(s)
        grads.append(pools[t][at[t]:at[t] + n].view(s))
        at[t] += n
    return grads


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    if op == "clip":
        grads = _gradients(case, g)
        return dict(case=case, grads=grads, out=[torch.empty_like(t) for t in grads])
    r = _route(case, g)
    s = dict(case=case, **r)
    P = r["rows"]
    if op == "quantize":
        M, H = case["M"], case["H"]
        kind = torch.float32 if case["src"] == "f32" else torch.bfloat16
        # rows with a few columns much larger than the rest
        loud = 1.0 + 8.0 * (torch.rand(H + case["pitch"], generator=g, device="cuda") < 0.01)
        s["x"] = (torch.randn(M, H + case["pitch"], generator=g, device="cuda") * loud).to(kind)[:, :H]
        s["codes"] = torch.zeros(P, H // 2, dtype=torch.uint8, device="cuda")
        s["scales"] = torch.zeros(P, H // MX, dtype=torch.uint8, device="cuda")
        return s
    E, N, K = max(1, case["E"]), case["N"], case["K"]
    gated = case["act"] == "swiglu" if op == "linear" else case["gated"]
    s["w"], s["up"] = _weight4(g, E, N, K), _weight4(g, E, N, K) if gated else None
    if op == "backward":
        s["dz"] = _randn(g, P, (2 if gated else 1) * N)
        s["dx"] = torch.zeros(P, K, dtype=torch.bfloat16, device="cuda")
        return s
    x = _randn(g, P, K)
    s["x"], s["x_scale"] = _codes(x) if case["rows4"] else (x, None)
    s["bias"] = _randn(g, E, N, scale=0.2) if case["bias"] else None
    s["up_bias"] = _randn(g, E, N, scale=0.2) if case["bias"] and gated else None
    s["residual"] = _randn(g, P, N) if case["residual"] else None
    s["out"] = torch.zeros(P, N, dtype=torch.bfloat16, device="cuda")
    s["pre"] = torch.zeros(P, (2 if gated else 1) * N, dtype=torch.bfloat16, device="cuda") if case["save"] else None
    return s


# ------------------------------------------------------------- plain forms --

def _quantize(s):
    c = s["case"]
    v = _values(*_codes(s["x"])).bfloat16()  # four-bit values times a power of two: exact in bf16
    if s["perm"] is None:
        return v
    p = s["perm"].long()
    out = torch.zeros(s["rows"] + 1, c["H"], dtype=torch.bfloat16, device="cuda")
    out[torch.where(p < 0, s["rows"], p)] = v.repeat_interleave(c["k"], 0)
    return out[:-1]


def _where(s):
    """[E, cap] rows of each expert (clamped) with their mask, and for each row
    its place in [E * cap] with its mask."""
    P, cap = s["rows"], s["cap"]
    if s["offsets"] is None:
        p = torch.arange(P, device="cuda")
        return p[None], torch.ones(1, P, dtype=torch.bool, device="cuda"), p, torch.ones(P, dtype=torch.bool, device="cuda")
    off, cnt = s["offsets"].long(), s["counts"].long()
    E = cnt.numel()
    j = torch.arange(cap, device="cuda")
    mask = j[None] < cnt[:, None]
    idx = torch.where(mask, off[:E, None] + j[None], 0)
    p = torch.arange(P, device="cuda")
    e = torch.searchsorted(off[1:].contiguous(), p, right=True)
    rank = p - off[e]
    e = e.clamp(max=E - 1)
    return idx, mask, e * cap + rank.clamp(0, cap - 1), (p < off[E]) & (rank < cnt[e])


def _padded(v, idx, mask):
    return torch.where(mask[..., None], v[idx].float(), 0.0)


def _act(name, z):
    if name == "silu":
        return z / (1 + torch.exp(-z))
    if name == "gelu":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)))
    return z


def _linear(s):
    c = s["case"]
    x = _values(s["x"], s["x_scale"]) if c["rows4"] else s["x"].float()
    idx, mask, back, kept = _where(s)
    xp = _padded(x, idx, mask)

    def product(w, b):
        z = torch.bmm(xp, _values(*w).transpose(1, 2).contiguous())
        z = z if b is None else z + b.float()[:, None]
        return z.reshape(-1, z.shape[2])[back]

    z = product(s["w"], s["bias"])
    if s["up"] is not None:
        u = product(s["up"], s["up_bias"])
        y, pre = _act("silu", z) * u, torch.cat([z, u], 1)
    else:
        y, pre = _act(c["act"], z), z
    if s["residual"] is not None:
        y = y + s["residual"].float()
    out = dict(y=torch.where(kept[:, None], y, 0.0).bfloat16())
    if c["save"]:
        out["pre"] = torch.where(kept[:, None], pre, 0.0).bfloat16()
    return out


def _backward(s):
    N = s["case"]["N"]
    idx, mask, back, kept = _where(s)
    dz = _padded(s["dz"], idx, mask)
    dx = torch.bmm(dz[..., :N].contiguous(), _values(*s["w"]))
    if s["up"] is not None:
        dx = dx + torch.bmm(dz[..., N:].contiguous(), _values(*s["up"]))
    return torch.where(kept[:, None], dx.reshape(-1, dx.shape[2])[back], 0.0).bfloat16()


def _clip(s):
    # sums over up to 600 million squares: in 64 bits
    norm = torch.stack([g.float().square().sum(dtype=torch.float64) for g in s["grads"]]).sum().sqrt()
    scale = torch.clamp(MAX_NORM / norm, max=1.0).float()
    return dict(norm=norm.float().reshape(1), grads=[(g.float() * scale).to(g.dtype) for g in s["grads"]])


# --------------------------------------------------- the framework's calls --

def _own(s):
    import mixture_experts_routing_align_amd as moe

    c = s["case"]
    if c["op"] == "quantize":
        codes, scales = moe.moe_mxfp4_quantize(s["x"], s["perm"], c["k"], s["rows"], codes=s["codes"], scales=s["scales"])
        return moe.moe_mxfp4_dequantize(codes, scales)
    if c["op"] == "linear":
        y, _, pre = moe.moe_grouped_linear_mxfp4(
            s["x"], s["w"], s["offsets"], s["counts"], act=c["act"], up=s["up"], bias=s["bias"], up_bias=s["up_bias"],
            residual=s["residual"], x_scale=s["x_scale"], out=s["out"], preact=s["pre"])
        return dict(y=y) if pre is None else dict(y=y, pre=pre)
    if c["op"] == "backward":
        return moe.moe_grouped_linear_mxfp4_backward_x(s["dz"], s["w"], s["offsets"], s["counts"], up=s["up"], dx=s["dx"])
    norm = moe.moe_clip_grad_norm(s["grads"], MAX_NORM, out=s["out"])
    return dict(norm=norm, grads=s["out"])


_PLAIN = dict(quantize=_quantize, linear=_linear, backward=_backward, clip=_clip)


def run(state):
    if own:
        return _own(state)
    return _PLAIN[state["case"]["op"]](state)


# -------------------------------------------------------------------- work --

FOUR = 0.5 + 1 / MX  # bytes of an MXFP4 value with its share of a scale


def work(case):
    op = case["op"]
    if op == "clip":  # the gradients in, the clipped ones out
        E, H, N, L = case["E"], case["H"], case["N"], case["layers"]
        big, router, rest = 3 * E * N * H * L, E * H * L, (E * N + H) * L
        item = 4 if case["dw"] == "f32" else 2
        return {"bytes": 2 * (big * item + router * 2 + rest * 4) + 4, "flops": 3 * (big + router + rest)}
    M, E = case["M"], max(1, case["E"])
    n = M * case["k"] * (1 - case["drop"])
    if op == "quantize":  # rows in, codes out; codes in, values out
        H = case["H"]
        return {"bytes": M * H * (4 if case["src"] == "f32" else 2) + 2 * n * H * FOUR + 2 * n * H
                + (0 if case["E"] == 0 else 4 * M * case["k"]), "flops": 4 * (M + n) * H}
    K, N = case["K"], case["N"]
    # an expert without a row needs no weight
    active = E * (1 - (1 - 1 / E) ** n) if E > 1 else 1
    wide = 2 if case.get("act") == "swiglu" or case.get("gated") else 1
    weights = active * wide * N * K * FOUR
    if op == "backward":
        return {"bytes": weights + n * (2 * wide * N + 2 * K), "flops": 2 * n * wide * N * K}
    x = n * K * (FOUR if case["rows4"] else 2)
    y = n * N * (2 + (2 if case["residual"] else 0) + (2 * wide if case["save"] else 0))
    return {"bytes": weights + x + y + (2 * active * wide * N if case["bias"] else 0), "flops": 2 * n * wide * N * K}


# ------------------------------------------------- the definitions, 64 bits --

def _exact_round(v):
    """Rows of doubles rounded to MXFP4: to the nearest of the scale's multiples."""
    b = v.reshape(-1, MX)
    amax = b.abs().amax(1)
    e = torch.clamp(torch.frexp(amax).exponent - 3, min=-125)  # amax in [2^(e+2), 2^(e+3))
    scale = torch.ldexp(torch.ones_like(amax), torch.where(amax > 0, e, torch.zeros_like(e)))[:, None]
    m = (b.abs() / scale).clamp(max=6.0)
    step = torch.where(m < 2, 0.5, torch.where(m < 4, 1.0, 2.0))
    return (torch.round(m / step) * step * torch.sign(b) * scale).reshape(v.shape)


def _exact_read(pair, at):
    """float64 values of codes and scales from index `at` on."""
    codes, scales = pair[0][at].int(), pair[1][at].double()
    nibbles = torch.stack([codes % 16, codes // 16], -1).reshape(*codes.shape[:-1], -1)
    low = nibbles % 8
    mag = torch.where(low < 2, low.double() / 2, torch.ldexp(1 + (low % 2).double() / 2, low // 2 - 1))
    return torch.where(nibbles < 8, mag, -mag) * torch.pow(2.0, scales - 127).repeat_interleave(MX, -1)


def _exact_rows(s):
    """(expert, first row, rows) of each expert that has one."""
    if s["offsets"] is None:
        return [(0, 0, s["rows"])]
    off, cnt = s["offsets"].tolist(), s["counts"].tolist()
    return [(e, off[e], cnt[e]) for e in range(len(cnt)) if cnt[e]]


def _exact_act(name, z):
    if name == "silu":
        return z * torch.sigmoid(z)
    if name == "gelu":
        return 0.5 * z * (1 + torch.tanh((2 / math.pi) ** 0.5 * (z + 0.044715 * z ** 3)))
    return z


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "clip":
        total = 0.0
        for g in s["grads"]:
            total += float((g.double() ** 2).sum())
        scale = min(1.0, MAX_NORM / math.sqrt(total))
        return dict(norm=torch.tensor([math.sqrt(total)], dtype=torch.float64), grads=[g.double() * scale for g in s["grads"]])
    if op == "quantize":
        v = _exact_round(s["x"].double())
        if s["perm"] is None:
            return v
        M, k = case["M"], case["k"]
        perm = s["perm"].long().reshape(M, k)
        out = torch.zeros(s["rows"], case["H"], dtype=torch.float64, device="cuda")
        for j in range(k):
            t = torch.nonzero(perm[:, j] >= 0)[:, 0]
            out[perm[t, j]] = v[t]
        return out
    P, N, K = s["rows"], case["N"], case["K"]
    if op == "backward":
        dx = torch.zeros(P, K, dtype=torch.float64, device="cuda")
        for e, at, c in _exact_rows(s):
            dx[at:at + c] = s["dz"][at:at + c, :N].double() @ _exact_read(s["w"], e)
            if s["up"] is not None:
                dx[at:at + c] += s["dz"][at:at + c, N:].double() @ _exact_read(s["up"], e)
        return dx
    gated = case["act"] == "swiglu"
    y = torch.zeros(P, N, dtype=torch.float64, device="cuda")
    pre = torch.zeros(P, (2 if gated else 1) * N, dtype=torch.float64, device="cuda")
    for e, at, c in _exact_rows(s):
        x = _exact_read((s["x"], s["x_scale"]), slice(at, at + c)) if case["rows4"] else s["x"][at:at + c].double()
        z = x @ _exact_read(s["w"], e).T
        if s["bias"] is not None:
            z = z + s["bias"][e].double()
        pre[at:at + c, :N] = z
        v = _exact_act("silu" if gated else case["act"], z)
        if gated:
            u = x @ _exact_read(s["up"], e).T
            if s["up_bias"] is not None:
                u = u + s["up_bias"][e].double()
            pre[at:at + c, N:] = u
            v = v * u
        if s["residual"] is not None:
            v = v + s["residual"][at:at + c].double()
        y[at:at + c] = v
    return dict(y=y, pre=pre) if case["save"] else dict(y=y)
