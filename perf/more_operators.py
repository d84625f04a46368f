"""Workloads of the operators of a meta-learned attention layer: norms of
queries and keys for each head with their rotary positions, and orthogonalised
updates by Newton-Schulz products.

``run`` makes one pass through an operator on the inputs of ``prepare``:
with ``own`` false in its plain form (elementary torch operations in 32 or 64
bits, rounded once at the end), with ``own`` true through this package.  The
cases go from single tokens and stacks of small matrices, where latency counts,
to long contexts and the largest weight matrices; bf16 and fp32; forward, first
and second derivatives.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
#: the steps' polynomials a x + b x^3 + c x^5: one for all steps, which lifts small
#: singular values quickly, or two more of another kind at the end, which bring them to 1
ONE = (3.4445, -4.7750, 2.0315)
SCHEDULE = (ONE,) * 3 + ((1.875, -1.25, 0.375),) * 2
#: bound on the multiplications of an orthogonalisation (forward, all steps): the largest listed one
MOST_PRODUCTS = 5 * (2 * 4096 * 4096 * 16384 + 4096 ** 3)


def listed():
    return [
        # one decoding step of eight sequences at far positions: the smallest call
        _norm("norm_token", 8, 16, 4, 1, 128, 128, "bf16", "bf16", "fused", True, False, "plain",
              "forward"),
        # a short prompt through the same layer
        _norm("norm_prompt", 1, 16, 4, 37, 128, 128, "bf16", "bf16", "fused", False, False, "plain",
              "forward"),
        # a training step, from one fused fp32 projection to the bf16 heads that attention reads
        _norm("norm_train", 2, 16, 16, 4096, 128, 128, "fp32", "bf16", "fused", False, False,
              "yarn", "train"),
        # half of each head turned, interleaved pairs, an odd length, fp32
        _norm("norm_part_train", 1, 8, 2, 4097, 64, 32, "fp32", "fp32", "bhnd", False, True, "plain",
              "train"),
        # a long context, shared key heads
        _norm("norm_long_train", 1, 8, 2, 65536, 128, 128, "bf16", "bf16", "bnhd", False, False,
              "linear", "train"),
        # a meta-learning step: the derivative of the first derivative
        _norm("norm_second", 2, 16, 16, 4096, 128, 128, "bf16", "bf16", "bnhd", False, False,
              "plain", "second"),
        # fast weights of sixteen heads, updated within a sequence
        _orth("orth_heads", 16, 64, 64, "bf16", "one", False),
        # the four projections of a small layer in fp32, whose update a meta-gradient passes
        _orth("orth_layer_fp32_train", 4, 128, 128, "fp32", "one", True),
        # a ragged tall matrix
        _orth("orth_ragged", 1, 1000, 333, "bf16", "schedule", False),
        # the four projections of a layer of 16 heads of 128
        _orth("orth_layer", 4, 2048, 2048, "bf16", "one", False),
        # an update with a meta-gradient through it, at an ordinary width
        _orth("orth_train", 2, 1024, 4096, "bf16", "one", True),
        # the largest: a wide feed-forward weight
        _orth("orth_wide", 1, 4096, 16384, "bf16", "one", False),
    ]


def _norm(name, B, H, Hk, N, d, turned, dtype, out, layout, far, interleaved, scaling, order):
    return {"name": name, "op": "norm", "B": B, "H": H, "Hk": Hk, "N": N, "d": d, "turned": turned,
            "dtype": dtype, "out": out, "layout": layout, "far": far, "interleaved": interleaved,
            "scaling": scaling, "order": order}


def _orth(name, L, m, n, dtype, polynomial, train):
    return {"name": name, "op": "orth", "L": L, "m": m, "n": n, "dtype": dtype,
            "polynomial": polynomial, "train": train}


def _spread(rng, low, high):
    """An integer between the two, spread evenly over its logarithm."""
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    if rng.random() < 0.5:
        d = rng.choice([40, 64, 64, 80, 96, 128, 128, 256])
        turned = rng.choice([d, d, d // 2])
        B, Hk = _spread(rng, 1, 8), _spread(rng, 1, 16)
        H = Hk * rng.choice([1, 1, 2, 4])
        order = rng.choice(["forward", "train", "train", "second"])
        N = _spread(rng, 1, min(65536, 10 * 65536 * 128 // (B * (H + Hk) * d)))
        dtype = rng.choice(["bf16", "bf16", "fp32"])
        case = _norm("", B, H, Hk, N, d, turned, dtype, rng.choice([dtype, "bf16"]),
                     rng.choice(["bhnd", "bnhd", "fused"]), rng.random() < 0.5, rng.random() < 0.5,
                     rng.choice(["plain", "linear", "yarn"]), order)
    else:
        train = rng.random() < 0.5
        dtype = rng.choice(["bf16", "bf16", "fp32"])
        small = _spread(rng, 16, 1024 << ((dtype == "bf16") + (not train)))
        large = min(16384, _spread(rng, small, 8 * small))
        # a training pass multiplies about three times as much as the forward alone
        most = MOST_PRODUCTS // (3 if train else 1)
        one = 5 * (2 * small * small * large + small ** 3)
        L = _spread(rng, 1, max(1, min(64, most // one, (1 << 26) // (small * large))))
        m, n = rng.choice([(small, large), (small, large), (large, small)])
        case = _orth("", L, m, n, dtype, rng.choice(["one", "one", "schedule"]), train)
    del case["name"]
    return case


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))

    def normal(*shape, std=1.0, dtype=torch.float32):
        return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)

    dtype = DTYPES[case["dtype"]]
    state = dict(case)
    if case["op"] == "orth":
        L, m, n = case["L"], case["m"], case["n"]
        # a gradient: a few strong directions, and noise in all of them
        r = max(1, min(m, n) // 8)
        strong = normal(L, m, r, std=r ** -0.5) @ normal(L, r, n)
        G = 1e-3 * (strong + normal(L, m, n, std=0.3))
        state["G"] = G.to(dtype).requires_grad_(case["train"])
        if case["train"]:
            state["dX"] = normal(L, m, n, std=0.1, dtype=dtype)
        return state
    B, H, Hk, N, d = (case[n] for n in ("B", "H", "Hk", "N", "d"))
    order = case["order"]
    if case["layout"] == "fused":  # one projection to queries, keys and values
        base = normal(B, N, H + 2 * Hk, d, dtype=dtype).transpose(1, 2)
        q, k = base[:, :H], base[:, H:H + Hk]
    elif case["layout"] == "bnhd":
        q, k = (normal(B, N, h, d, dtype=dtype).transpose(1, 2) for h in (H, Hk))
    else:
        q, k = (normal(B, h, N, d, dtype=dtype) for h in (H, Hk))
    wq, wk = (1.0 + normal(d, std=0.2) for _ in range(2))
    for name, t in (("q", q), ("k", k), ("wq", wq), ("wk", wk)):
        state[name] = t.detach().requires_grad_(order != "forward")
    if case["far"]:  # every sequence at a place of its own in a long context
        at = torch.randint(0, 262144 - N + 1, (B, 1), generator=g, device="cuda")
        state["positions"] = at + torch.arange(N, device="cuda")
    else:
        state["positions"] = None
    state["inv_freq"], state["magnitude"] = _frequencies(case["turned"], case["scaling"])
    if order != "forward":
        for name, h in (("dyq", H), ("dyk", Hk)):
            dy = normal(B, h, N, d, std=0.1, dtype=DTYPES[case["out"]])
            state[name] = dy.requires_grad_(order == "second")
    if order == "second":  # cotangents of the gradients
        state["aq"], state["ak"] = (normal(B, h, N, d, std=0.1, dtype=dtype) for h in (H, Hk))
        state["cq"], state["ck"] = normal(d, std=0.1), normal(d, std=0.1)
    return state


EPS = 1e-6       # of the norms' mean square
ORTH_EPS = 1e-7  # beside the norm of an update


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


def _polynomials(case):
    return [ONE] * 5 if case["polynomial"] == "one" else list(SCHEDULE)


def run(state):
    if state["op"] == "norm":
        return _norm_own(state) if own else _norm_plain(state)
    return _orth_own(state) if own else _orth_plain(state)


# ---- the package's operators, called as a user's program calls them ----------
def _norm_own(s):
    import exact_second_order_two_gb300 as fbob

    leaves = (s["q"], s["k"], s["wq"], s["wk"])
    y = fbob.qk_norm_rotary(*leaves, s["inv_freq"], s["positions"], eps=EPS,
                            interleaved=s["interleaved"], magnitude=s["magnitude"],
                            dtype=DTYPES[s["out"]])
    if s["order"] == "forward":
        return y
    dy = (s["dyq"], s["dyk"])
    second = s["order"] == "second"
    grads = torch.autograd.grad(y, leaves, dy, create_graph=second)
    out = tuple(t.detach() for t in y + grads)
    if second:
        out += torch.autograd.grad(grads, leaves + dy, (s["aq"], s["ak"], s["cq"], s["ck"]))
    return out


def _orth_own(s):
    import exact_second_order_two_gb300 as fbob

    X = fbob.orthogonalize(s["G"], 5, ONE if s["polynomial"] == "one" else SCHEDULE, eps=ORTH_EPS)
    if not s["train"]:
        return X
    return X.detach(), torch.autograd.grad(X, s["G"], s["dX"])[0]


# ---- the plain forms ---------------------------------------------------------
def _turn_plain(x, cos, sin, turned, interleaved):
    a = x[..., 0:turned:2] if interleaved else x[..., : turned // 2]
    b = x[..., 1:turned:2] if interleaved else x[..., turned // 2: turned]
    u, w = a * cos - b * sin, a * sin + b * cos
    turned_part = torch.stack((u, w), -1).flatten(-2) if interleaved else torch.cat((u, w), -1)
    return torch.cat((turned_part, x[..., turned:]), -1)


def _norm_plain(s):
    d, m, r = s["d"], s["magnitude"], s["turned"]
    N = s["q"].shape[2]
    at = s["positions"] if s["positions"] is not None else torch.arange(N, device="cuda")[None]
    angle = at[:, None, :, None].double() * s["inv_freq"]
    cos, sin = (angle.cos() * m).float(), (angle.sin() * m).float()

    def turn(x, sign=1.0):
        return _turn_plain(x, cos, sign * sin, r, s["interleaved"])

    def dot(a, b):
        return (a * b).sum(-1, keepdim=True)

    outs, grads, seconds, ddys = [], [], [], []
    for x, w, dy, a, c in (("q", "wq", "dyq", "aq", "cq"), ("k", "wk", "dyk", "ak", "ck")):
        dtype, x, w = s[x].dtype, s[x].detach().float(), s[w].detach()
        rs = 1.0 / torch.sqrt(dot(x, x) / d + EPS)
        n = x * rs
        outs.append(turn(w * n).to(DTYPES[s["out"]]))
        if s["order"] == "forward":
            continue
        dout = s[dy].dtype
        g = turn(s[dy].detach().float(), -1.0)
        h = g * w
        hn = dot(h, n)
        grads.append(((rs * (h - n * (hn / d))).to(dtype), (g * n).sum((0, 1, 2))))
        if s["order"] == "train":
            continue
        a, c = s[a].float(), s[c]
        an = dot(a, n)
        t = rs * (a - n * (an / d))
        u = c * g - (rs / d) * (an * h + hn * a)
        gx = -(rs / d) * dot(h, t) * n + rs * (u - n * (dot(u, n) / d))
        seconds.append((gx.to(dtype), (g * t).sum((0, 1, 2))))
        ddys.append(turn(w * t + c * n).to(dout))
    out = tuple(outs)
    for pair in (grads, seconds):  # both inputs, then both weights
        if pair:
            out += (pair[0][0], pair[1][0], pair[0][1], pair[1][1])
    return out + tuple(ddys)


def _orth_plain(s):
    G = s["G"].detach()
    dtype, G = G.dtype, G.float()
    tall = s["m"] > s["n"]
    if tall:
        G = G.transpose(-1, -2)
    norm = torch.sqrt((G * G).sum((-1, -2), keepdim=True))
    scale = 1.0 / (norm + ORTH_EPS)
    X, kept = G * scale, []
    for a, b, c in _polynomials(s):
        A = X @ X.transpose(-1, -2)
        P = b * A + c * (A @ A)
        kept.append((X, A, P))
        X = a * X + P @ X
    out = (X.transpose(-1, -2) if tall else X).to(dtype).contiguous()
    if not s["train"]:
        return out
    H = s["dX"].float()
    H = H.transpose(-1, -2) if tall else H
    for (a, b, c), (X, A, P) in zip(reversed(_polynomials(s)), reversed(kept)):
        S = H @ X.transpose(-1, -2)
        S = S + S.transpose(-1, -2)
        T = A @ S
        T = b * S + c * (T + T.transpose(-1, -2))
        H = a * H + P @ H + T @ X
    H = scale * (H - (H * G).sum((-1, -2), keepdim=True) * (scale / norm) * G)
    return out, (H.transpose(-1, -2) if tall else H).to(dtype).contiguous()


# ---- work --------------------------------------------------------------------
def work(case):
    size = {"bf16": 2, "fp32": 4}
    if case["op"] == "orth":
        p, q = sorted((case["m"], case["n"]))
        elems = case["L"] * p * q
        # a step: the Gram matrix and its square, half of each by symmetry, and the product
        flops = 5 * (3 * p * p * q + p ** 3)
        if case["train"]:  # two symmetric sums of two products each, two products for the result
            flops += 5 * (6 * p * p * q + 2 * p ** 3)
        return {"bytes": elems * size[case["dtype"]] * (4 if case["train"] else 2),
                "flops": case["L"] * flops}
    n = case["B"] * (case["H"] + case["Hk"]) * case["N"] * case["d"]
    i, o = size[case["dtype"]], size[case["out"]]
    bytes_ = n * (i + o) + (case["B"] * case["N"] * 8 if case["far"] else 0)
    flops = n * 6
    if case["order"] != "forward":  # x and the output's gradient in, x's gradient out
        bytes_ += n * (2 * i + o)
        flops += n * 13
    if case["order"] == "second":  # x, dy and a in, two gradients out
        bytes_ += n * (3 * i + 2 * o)
        flops += n * 30
    return {"bytes": bytes_, "flops": flops}


# ---- the definitions in 64 bits ----------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    return _norm_exact(s) if case["op"] == "norm" else _orth_exact(s)


def _norm_exact(s):
    """The forward from its definition, pairs as complex numbers; derivatives
    by torch's autograd in 64 bits."""
    r, N, order = s["turned"], s["N"], s["order"]
    at = torch.arange(N, device="cuda").view(1, N) if s["positions"] is None else s["positions"]
    phase = torch.polar(torch.full((), s["magnitude"], dtype=torch.float64, device="cuda"),
                        at.double()[:, None, :, None] * s["inv_freq"])

    def forward(x, w):
        n = x / torch.sqrt(x.square().mean(-1, keepdim=True) + EPS) * w
        head, tail = n[..., :r], n[..., r:]
        if s["interleaved"]:
            z = torch.view_as_complex(head.unflatten(-1, (r // 2, 2)).contiguous())
            back = torch.view_as_real(z * phase).flatten(-2)
        else:
            z = torch.complex(*(t.contiguous() for t in head.chunk(2, -1))) * phase
            back = torch.cat((z.real, z.imag), -1)
        return torch.cat((back, tail), -1)

    outs, grads, seconds, ddys = [], [], [], []
    for x, w, dy, a, c in (("q", "wq", "dyq", "aq", "cq"), ("k", "wk", "dyk", "ak", "ck")):
        x, w = (s[t].detach().double().requires_grad_(order != "forward") for t in (x, w))
        y = forward(x, w)
        outs.append(y.detach())
        if order == "forward":
            continue
        dy = s[dy].detach().double().requires_grad_(order == "second")
        g = torch.autograd.grad(y, (x, w), dy, create_graph=order == "second")
        grads.append(tuple(t.detach() for t in g))
        if order == "second":
            gg = torch.autograd.grad(g, (x, w, dy), (s[a].double(), s[c].double()))
            seconds.append(gg[:2])
            ddys.append(gg[2])
    out = tuple(outs)
    for pair in (grads, seconds):
        if pair:
            out += (pair[0][0], pair[1][0], pair[0][1], pair[1][1])
    return out + tuple(ddys)


def _orth_exact(s):
    """Matrix by matrix, the shorter side first, gradients by torch's autograd
    in 64 bits."""
    p, q = sorted((s["m"], s["n"]))
    if s["L"] * (2 * p * p * q + p ** 3) * (3 if s["train"] else 1) > 1.2e12:
        return None
    out = torch.empty(s["G"].shape, dtype=torch.float64, device="cuda")
    grad = torch.empty_like(out) if s["train"] else None
    for i in range(s["L"]):
        G = s["G"][i].detach().double().requires_grad_(s["train"])
        X = G / (torch.linalg.matrix_norm(G) + ORTH_EPS)
        if s["m"] > s["n"]:
            X = X.mT
        for a, b, c in _polynomials(s):
            A = X @ X.mT
            X = a * X + b * (A @ X) + c * (A @ (A @ X))
        X = X.mT if s["m"] > s["n"] else X
        out[i] = X.detach()
        if s["train"]:
            (grad[i],) = torch.autograd.grad(X, G, s["dX"][i].double())
    return (out, grad) if s["train"] else out
