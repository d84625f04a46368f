"""Workloads of the attention-layer operators: rotary positions and
differential attention.

``run`` makes one pass through an operator on the inputs of ``prepare``:
with ``own`` false in its plain form (elementary torch operations in 32 or 64
bits, rounded once at the end), with ``own`` true through this package.  The
cases cover single tokens and short sequences, where latency counts, up to the
longest attention the plain form can hold; bf16 and fp32; forward alone and
forward with backward.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
#: bound on B*H*N*N of an attention case: the plain form holds several such tensors
MOST_SCORES = 8 * 16384 * 16384


def listed():
    return [
        # one decoding step of eight sequences at far positions: the smallest call
        _rotary("rotary_token", 8, 16, 1, 128, 128, "bf16", "bf16", "bhnd", True, False, "plain",
                False),
        # queries of a training step, straight from an fp32 projection [B, N, H, d] into the
        # bf16 [B, H, N, d] that attention reads; positions scaled by frequency bands
        _rotary("rotary_heads", 2, 16, 4096, 128, 128, "fp32", "bf16", "bnhd", False, False,
                "yarn", True),
        # half of each head turned, interleaved pairs, an odd length, fp32
        _rotary("rotary_part", 1, 8, 4097, 64, 32, "fp32", "fp32", "bhnd", False, True, "plain",
                True),
        # a long context with interpolated positions, interleaved pairs
        _rotary("rotary_long", 1, 8, 65536, 128, 128, "bf16", "bf16", "bhnd", False, True,
                "linear", True),
        # a short prompt
        _diff("diff_short", 1, 8, 8, 37, 64, 128, "bf16", True, "head", False),
        # a layer's forward at an ordinary training length
        _diff("diff_forward", 2, 8, 8, 4096, 64, 128, "bf16", True, "head", False),
        # a long document
        _diff("diff_forward_long", 1, 8, 8, 16384, 64, 128, "bf16", True, "head", False),
        # the fp32 configuration of the library, forward and backward
        _diff("diff_fp32_train", 1, 4, 4, 256, 64, 64, "fp32", False, "head", True),
        # fp32 at a ragged ordinary length
        _diff("diff_fp32_forward", 1, 4, 4, 2049, 64, 128, "fp32", True, "query", False),
        # key heads shared by four query heads, no mask, one weight for all, an uneven length
        _diff("diff_shared_train", 2, 8, 2, 1000, 64, 64, "bf16", False, "one", True),
        # a training step at an ordinary length
        _diff("diff_train", 2, 8, 8, 4096, 64, 128, "bf16", True, "head", True),
        # a training step on a long document, one weight per query
        _diff("diff_train_long", 1, 8, 8, 16384, 64, 128, "bf16", True, "query", True),
    ]


def _rotary(name, B, H, N, d, turned, dtype, out, layout, far, interleaved, scaling, train):
    return {"name": name, "op": "rotary", "B": B, "H": H, "N": N, "d": d, "turned": turned,
            "dtype": dtype, "out": out, "layout": layout, "far": far, "interleaved": interleaved,
            "scaling": scaling, "train": train}


def _diff(name, B, H, Hk, N, d, dv, dtype, causal, weight, train):
    return {"name": name, "op": "diff", "B": B, "H": H, "Hk": Hk, "N": N, "d": d, "dv": dv,
            "dtype": dtype, "causal": causal, "weight": weight, "train": train}


def _spread(rng, low, high):
    """An integer between the two, spread evenly over its logarithm."""
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    train = rng.random() < 0.5
    if rng.random() < 0.4:
        d = rng.choice([40, 64, 64, 96, 128, 128])
        turned = rng.choice([d, d, d // 2])
        B, H = _spread(rng, 1, 8), _spread(rng, 1, 32)
        N = _spread(rng, 1, min(65536, 8 * 65536 * 128 // (B * H * d)))
        dtype = rng.choice(["bf16", "bf16", "fp32"])
        case = _rotary("", B, H, N, d, turned, dtype, rng.choice([dtype, "bf16"]),
                       rng.choice(["bhnd", "bnhd"]), rng.random() < 0.5, rng.random() < 0.5,
                       rng.choice(["plain", "linear", "yarn"]), train)
    else:
        B, Hk = _spread(rng, 1, 4), _spread(rng, 1, 8)
        H = Hk * rng.choice([1, 1, 2, 4])
        kind = rng.choice(["bf16", "bf16", "bf16", "odd", "fp32"])
        if kind == "bf16":
            dtype, d, dv, most = "bf16", 64, rng.choice([64, 128, 128]), MOST_SCORES
        elif kind == "odd":
            dtype, d, dv, most = "bf16", rng.choice([24, 40, 96, 128]), rng.choice([40, 80, 128]), 1 << 24
        else:
            dtype, d, dv, most = "fp32", rng.choice([32, 40, 64]), rng.choice([64, 72, 128]), 1 << 26
        # with very few keys the gradients of queries and keys are differences that cancel (at one
        # key they are zero), so training lengths begin at 8
        N = _spread(rng, 8 if train else 1, min(16384, math.isqrt(most // (B * H))))
        case = _diff("", B, H, Hk, N, d, dv, dtype, rng.random() < 0.6,
                     rng.choice(["one", "head", "query"]), train)
    del case["name"]
    return case


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))

    def normal(*shape, std=1.0, dtype=torch.float32):
        return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)

    dtype = DTYPES[case["dtype"]]
    train = case["train"]
    state = dict(case)
    if case["op"] == "rotary":
        B, H, N, d = case["B"], case["H"], case["N"], case["d"]
        if case["layout"] == "bnhd":  # a projection's output, seen head by head
            base = normal(B, N, H, d, dtype=dtype)
            x = base.transpose(1, 2)
        else:
            x = normal(B, H, N, d, dtype=dtype)
        state["x"] = x.detach().requires_grad_(train)
        if case["far"]:  # every sequence at a place of its own in a long context
            at = torch.randint(0, 262144 - N + 1, (B, 1), generator=g, device="cuda")
            state["positions"] = at + torch.arange(N, device="cuda")
        else:
            state["positions"] = None
        state["inv_freq"], state["magnitude"] = _frequencies(case["turned"], case["scaling"])
        if train:
            state["dy"] = normal(B, H, N, d, std=0.1, dtype=DTYPES[case["out"]])
        return state
    B, H, Hk, N, d, dv = (case[n] for n in ("B", "H", "Hk", "N", "d", "dv"))
    for name, heads, width in (("q", 2 * H, d), ("k", 2 * Hk, d), ("v", Hk, dv)):
        state[name] = normal(B, heads, N, width, dtype=dtype).requires_grad_(train)
    shape = {"one": (), "head": (H,), "query": (B, H, N)}[case["weight"]]
    lam = torch.rand(shape, generator=g, device="cuda") * 0.6 + 0.2
    state["lam"] = lam.to(dtype).requires_grad_(train)
    if train:
        state["do"] = normal(B, H, N, dv, std=0.1, dtype=dtype)
    return state


def _frequencies(turned, scaling):
    """Angles a position adds to each pair, in 64 bits, and the factor on the
    result: 10000^(-2i/r); "linear" divides every one by 4; "yarn" divides by
    4 those with less than one turn in 4096 positions, leaves those with more
    than 32 turns, and blends in between."""
    i = torch.arange(turned // 2, dtype=torch.float64, device="cuda")
    f = 10000.0 ** (-2.0 * i / turned)
    if scaling == "linear":
        return f / 4.0, 1.0
    if scaling == "yarn":
        keep = ((4096 * f / (2 * math.pi) - 1.0) / 31.0).clamp(0.0, 1.0)
        return f / 4.0 * (1.0 - keep) + f * keep, 0.1 * math.log(4.0) + 1.0
    return f, 1.0


def run(state):
    if state["op"] == "rotary":
        return _rotary_own(state) if own else _rotary_plain(state)
    return _diff_own(state) if own else _diff_plain(state)


# ---- the package's operators, called as a user's program calls them ----------
def _rotary_own(s):
    import exact_second_order_two_gb300 as fbob

    y = fbob.rotary(s["x"], s["inv_freq"], s["positions"], interleaved=s["interleaved"],
                    magnitude=s["magnitude"], dtype=DTYPES[s["out"]])
    if not s["train"]:
        return y
    return y.detach(), torch.autograd.grad(y, s["x"], s["dy"])[0]


def _diff_own(s):
    import exact_second_order_two_gb300 as fbob

    o = fbob.diff_attention(s["q"], s["k"], s["v"], s["lam"], causal=s["causal"])
    if not s["train"]:
        return o
    leaves = (s["q"], s["k"], s["v"], s["lam"])
    return (o.detach(),) + torch.autograd.grad(o, leaves, s["do"])


# ---- the plain forms ---------------------------------------------------------
def _turn_plain(x, cos, sin, turned, interleaved):
    a = x[..., 0:turned:2] if interleaved else x[..., : turned // 2]
    b = x[..., 1:turned:2] if interleaved else x[..., turned // 2: turned]
    u, w = a * cos - b * sin, a * sin + b * cos
    turned_part = torch.stack((u, w), -1).flatten(-2) if interleaved else torch.cat((u, w), -1)
    return torch.cat((turned_part, x[..., turned:]), -1)


def _rotary_plain(s):
    x = s["x"].detach()
    N = x.shape[2]
    at = s["positions"] if s["positions"] is not None else torch.arange(N, device=x.device)[None]
    angle = at[:, None, :, None].double() * s["inv_freq"]
    cos = (angle.cos() * s["magnitude"]).float()
    sin = (angle.sin() * s["magnitude"]).float()
    y = _turn_plain(x.float(), cos, sin, s["turned"], s["interleaved"]).to(DTYPES[s["out"]])
    if not s["train"]:
        return y
    dx = _turn_plain(s["dy"].float(), cos, -sin, s["turned"], s["interleaved"])
    return y, dx.to(x.dtype)


def _diff_plain(s):
    q, k, v, lam = (s[n].detach() for n in ("q", "k", "v", "lam"))
    B, H, Hk, N, d, dv = (s[n] for n in ("B", "H", "Hk", "N", "d", "dv"))
    G, scale = H // Hk, s["d"] ** -0.5
    dtype = q.dtype
    # [B, key head, query head of it, map, N, ...]; keys and values are shared by G query heads
    q = q.float().view(B, Hk, G, 2, N, d)
    k = k.float().view(B, Hk, 1, 2, N, d)
    v = v.float().view(B, Hk, 1, N, dv)
    row = lam.float()
    row = row.view(1, H, 1).expand(B, H, N) if s["weight"] == "head" else row.expand(B, H, N)
    row = row.reshape(B, Hk, G, N, 1)
    p = scale * (q @ k.transpose(-1, -2))
    if s["causal"]:
        p.masked_fill_(torch.ones(N, N, dtype=torch.bool, device=q.device).triu(1), -math.inf)
    p = torch.exp(p - p.amax(-1, keepdim=True))
    p = p / p.sum(-1, keepdim=True)
    both = p @ v.unsqueeze(3)
    o = both[:, :, :, 0] - row * both[:, :, :, 1]
    out = o.reshape(B, H, N, dv).to(dtype)
    if not s["train"]:
        return out
    do = s["do"].float().view(B, Hk, G, N, dv)
    dot = (do.unsqueeze(3) * both).sum(-1, keepdim=True)
    dlam = -dot[:, :, :, 1, :, 0].reshape(B, H, N)
    dlam = dlam.sum() if s["weight"] == "one" else dlam.sum((0, 2)) if s["weight"] == "head" else dlam
    w = p[:, :, :, 0] - row * p[:, :, :, 1]
    dv_ = (w.transpose(-1, -2) @ do).sum(2)
    del w
    dp = do @ v.transpose(-1, -2)
    ds = p.mul_(dp.unsqueeze(3) - dot)
    ds[:, :, :, 1].mul_(-row)
    dq = scale * (ds @ k)
    dk = scale * (ds.transpose(-1, -2) @ q).sum(2)
    return (out, dq.reshape(B, 2 * H, N, d).to(dtype), dk.reshape(B, 2 * Hk, N, d).to(dtype),
            dv_.to(dtype), dlam.to(dtype))


# ---- work --------------------------------------------------------------------
def work(case):
    size = {"bf16": 2, "fp32": 4}
    if case["op"] == "rotary":
        n = case["B"] * case["H"] * case["N"]
        pairs = n * case["turned"] // 2
        passes = 2 if case["train"] else 1
        elems = n * case["d"]
        at = case["B"] * case["N"] * 8 if case["far"] else 0
        return {"bytes": passes * elems * (size[case["dtype"]] + size[case["out"]]) + at,
                "flops": passes * 6 * pairs}
    B, H, Hk, N, d, dv = (case[n] for n in ("B", "H", "Hk", "N", "d", "dv"))
    e = size[case["dtype"]]
    weights = {"one": 1, "head": H, "query": B * H * N}[case["weight"]]
    pairs = B * H * (N * (N + 1) // 2 if case["causal"] else N * N)
    reads = 2 * H * N * d + 2 * Hk * N * d + Hk * N * dv
    bytes_ = e * (B * (reads + H * N * dv) + weights)
    flops = pairs * (4 * d + 4 * dv)
    if case["train"]:
        # the output gradient in, a gradient of each input out; two score maps again, the
        # products for the gradients of the probabilities, values, queries and keys
        bytes_ += e * (B * (H * N * dv + reads) + weights)
        flops += pairs * (12 * d + 4 * dv)
    return {"bytes": bytes_, "flops": flops}


# ---- the definitions in 64 bits ----------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    return _rotary_exact(s) if case["op"] == "rotary" else _diff_exact(s)


def _rotary_exact(s):
    """Each pair (a, b) is the number a + ib; a position multiplies it by
    magnitude * exp(i position inv_freq), and the gradient by the conjugate."""
    r = s["turned"]
    N = s["x"].shape[2]
    at = torch.arange(N, device="cuda").view(1, N) if s["positions"] is None else s["positions"]
    phase = torch.polar(torch.full((), s["magnitude"], dtype=torch.float64, device="cuda"),
                        at.double()[:, None, :, None] * s["inv_freq"])

    def turned(x, factor):
        x = x.detach().double()
        head, tail = x[..., :r], x[..., r:]
        if s["interleaved"]:
            z = torch.view_as_complex(head.unflatten(-1, (r // 2, 2)).contiguous())
            back = torch.view_as_real(z * factor).flatten(-2)
        else:
            z = torch.complex(*head.chunk(2, -1)) * factor
            back = torch.cat((z.real, z.imag), -1)
        return torch.cat((back, tail), -1)

    y = turned(s["x"], phase)
    return (y, turned(s["dy"], phase.conj())) if s["train"] else y


def _diff_exact(s):
    """Head by head through torch's softmax and autograd in 64 bits."""
    B, H, Hk, N = (s[n] for n in ("B", "H", "Hk", "N"))
    if B * H * N * N > MOST_SCORES:
        return None
    q, k, v = (s[n].detach().double() for n in ("q", "k", "v"))
    lam = s["lam"].detach().double()
    out = torch.empty(B, H, N, s["dv"], dtype=torch.float64, device="cuda")
    dq, dk, dv, dlam = (torch.zeros_like(t) for t in (q, k, v, lam))
    hidden = torch.ones(N, N, dtype=torch.bool, device="cuda").triu(1) if s["causal"] else None

    def softmax_map(a, b):
        x = a @ b.T / math.sqrt(s["d"])
        return torch.softmax(x if hidden is None else x.masked_fill(hidden, -math.inf), -1)

    for b in range(B):
        for h in range(H):
            n = h // (H // Hk)
            part = [q[b, 2 * h], q[b, 2 * h + 1], k[b, 2 * n], k[b, 2 * n + 1], v[b, n],
                    lam if lam.dim() == 0 else lam[h] if lam.dim() == 1 else lam[b, h][:, None]]
            part = [t.clone().requires_grad_(s["train"]) for t in part]
            q1, q2, k1, k2, vv, w = part
            o = softmax_map(q1, k1) @ vv - w * (softmax_map(q2, k2) @ vv)
            out[b, h] = o.detach()
            if s["train"]:
                g = torch.autograd.grad(o, part, s["do"][b, h].double())
                dq[b, 2 * h], dq[b, 2 * h + 1] = g[0], g[1]
                dk[b, 2 * n] += g[2]
                dk[b, 2 * n + 1] += g[3]
                dv[b, n] += g[4]
                if lam.dim() == 0:
                    dlam += g[5]
                elif lam.dim() == 1:
                    dlam[h] += g[5]
                else:
                    dlam[b, h] = g[5][:, 0]
    return (out, dq, dk, dv, dlam) if s["train"] else out
