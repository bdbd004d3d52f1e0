"""Cases of the gated feed-forward block and of the products with 4-bit weights.

Four operators, row-major throughout (``M`` rows of activations):

glu         H = act(G) * U with G = X Wg and U = X Wu (M x F), float32; a
            training step keeps G and U as well.
backward    from dH: dG = dH U act'(G), dU = dH act(G), then dX = dG Wg^T +
            dU Wu^T, dWg = X^T dG, dWu = X^T dU, float32.
q4          Y[m, n] = sum_k X[m, k] s[n, k / group] (q[n, k] - z[n, k / group])
            with 4-bit q, two to a byte along K, low half first; z is 8 where
            no zero points are given.
q4_glu      H = act(G) * U with G and U products of the form above.

``linear`` weights are stored F x K (the layout of a linear layer), otherwise
K x F.  Gate and up weights are the two halves of one allocation, as model
checkpoints hold them.
"""
import math

import torch

own = False

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
ACTS = ("silu", "gelu", "gelu_tanh", "relu", "sigmoid")


def listed():
    return [
        # One token of a decoding step through a block of a mid-size model
        # whose weights are float32: the weights are read once.
        {"name": "glu_one_token", "op": "glu", "M": 1, "K": 4096, "F": 8192, "act": "silu",
         "linear": True, "save": False},
        # A handful of rows with nothing aligned: weights K x F.
        {"name": "glu_few_rows_odd", "op": "glu", "M": 7, "K": 2047, "F": 4099,
         "act": "gelu_tanh", "linear": False, "save": False},
        # The forward pass of a training step over 4096 tokens.
        {"name": "glu_train", "op": "glu", "M": 4096, "K": 4096, "F": 8192, "act": "silu",
         "linear": True, "save": True},
        # The same over a batch whose sizes fit no tile.
        {"name": "glu_ragged", "op": "glu", "M": 3001, "K": 2047, "F": 4099, "act": "gelu",
         "linear": False, "save": False},
        # The backward pass of that training step.
        {"name": "backward_train", "op": "backward", "M": 4096, "K": 4096, "F": 8192,
         "act": "silu", "linear": True},
        # Fine-tuning a small block on a short batch, odd sizes, weights K x F.
        {"name": "backward_small_odd", "op": "backward", "M": 257, "K": 1023, "F": 1027,
         "act": "gelu", "linear": False},
        # One token of a served model, half precision, weights quantised in
        # groups of 128 without zero points.
        {"name": "q4_one_token", "op": "q4", "M": 1, "N": 8192, "K": 8192, "x": "f16", "s": "f16",
         "group": 128, "zeros": False},
        # Eight sequences decoded together in float32, small groups with zero
        # points.
        {"name": "q4_eight_rows", "op": "q4", "M": 8, "N": 4096, "K": 4096, "x": "f32", "s": "f16",
         "group": 32, "zeros": True},
        # The prompt of a served model.
        {"name": "q4_prompt", "op": "q4", "M": 2048, "N": 8192, "K": 4096, "x": "bf16",
         "s": "bf16", "group": 128, "zeros": False},
        # A short prompt in float32 with nothing aligned.
        {"name": "q4_odd", "op": "q4", "M": 67, "N": 1025, "K": 2047, "x": "f32", "s": "f32",
         "group": 64, "zeros": True},
        # One token through a served feed-forward block.
        {"name": "q4_glu_one_token", "op": "q4_glu", "M": 1, "N": 8192, "K": 4096, "x": "bf16",
         "s": "bf16", "group": 128, "zeros": False, "act": "silu"},
        # A prompt of float32 activations through the same block.
        {"name": "q4_glu_prompt", "op": "q4_glu", "M": 1024, "N": 8192, "K": 4096, "x": "f32",
         "s": "f16", "group": 64, "zeros": True, "act": "gelu_tanh"},
    ]


def draw(rng):
    """A case of the same ranges: 1 to 4096 rows, widths of 64 to 8192."""
    def size(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    def width(lo, hi):
        n = size(lo, hi)
        # Half of the widths are multiples of 64, as most models' are.
        return max(lo, n // 64 * 64) if rng.random() < 0.5 else n

    op = rng.choice(["glu", "backward", "q4", "q4_glu"])
    case = {"op": op, "M": size(1, 4096)}
    if rng.random() < 0.25:
        case["M"] = rng.randint(1, 16)  # decoding steps
    if op in ("glu", "backward"):
        case.update(K=width(64, 4096), F=width(64, 8192), act=rng.choice(ACTS),
                    linear=rng.random() < 0.5)
        if op == "glu":
            case["save"] = rng.random() < 0.5
    else:
        case.update(N=width(64, 8192), K=width(64, 8192), x=rng.choice(list(TYPES)),
                    s=rng.choice(list(TYPES)), group=rng.choice([32, 64, 128]),
                    zeros=rng.random() < 0.5)
        if op == "q4_glu":
            case["act"] = rng.choice(ACTS)
    return case


# ---- inputs -----------------------------------------------------------------

def _q4_weight(gen, N, K, group, stype, zeros):
    """An N x K weight quantised the usual way: per group of K, a scale from
    the largest magnitude (or the range, with zero points); packed bytes,
    scales and zero points."""
    groups = -(-K // group)
    w = torch.randn((N, groups * group), generator=gen, device="cuda") / math.sqrt(K)
    w = w.view(N, groups, group)
    if zeros:
        lo, hi = w.amin(2), w.amax(2)
        s = ((hi - lo) / 15).to(stype)
        z = torch.clamp(torch.round(-lo / s.float()), 0, 15)
    else:
        s = (w.abs().amax(2) / 8).to(stype)
        z = torch.full_like(s, 8, dtype=torch.float32)
    q = torch.clamp(torch.round(w / s.float()[..., None]) + z[..., None], 0, 15).to(torch.uint8)
    q = q.view(N, groups * group)[:, :K]
    if K % 2:
        q = torch.cat([q, torch.zeros((N, 1), dtype=torch.uint8, device="cuda")], 1)
    packed = (q[:, 0::2] | (q[:, 1::2] << 4)).contiguous()
    return packed, s.contiguous(), z.to(torch.uint8).contiguous() if zeros else None


def _activations(gen, M, K):
    """Normal activations with a few channels ten times larger, as residual
    streams have them."""
    x = torch.randn((M, K), generator=gen, device="cuda")
    big = torch.rand((K,), generator=gen, device="cuda") < 0.01
    return torch.where(big, 10 * x, x)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    M, K = case["M"], case["K"]
    st = {"case": case}
    if case["op"] in ("glu", "backward"):
        F = case["F"]
        st["X"] = torch.randn((M, K), generator=gen, device="cuda")
        shape = (2 * F, K) if case["linear"] else (K, 2 * F)
        W = torch.randn(shape, generator=gen, device="cuda") / math.sqrt(K)
        st["Wg"], st["Wu"] = (W[:F], W[F:]) if case["linear"] else (W[:, :F], W[:, F:])
        if case["op"] == "backward":
            # The forward pass left G and U (here: of the same distribution).
            GU = torch.randn((M, 2 * F), generator=gen, device="cuda")
            st["G"], st["U"] = GU[:, :F], GU[:, F:]
            st["dH"] = torch.randn((M, F), generator=gen, device="cuda") / math.sqrt(M)
        return st
    N, group, stype = case["N"], case["group"], TYPES[case["s"]]
    st["X"] = _activations(gen, M, K).to(TYPES[case["x"]])
    st["W"] = [_q4_weight(gen, N, K, group, stype, case["zeros"])
               for _ in range(2 if case["op"] == "q4_glu" else 1)]
    return st


# ---- one pass ---------------------------------------------------------------

def _act(name, g):
    """act(g) and its derivative, from elementary operations."""
    if name == "relu":
        return torch.where(g > 0, g, torch.zeros_like(g)), (g > 0).to(g.dtype)
    if name in ("silu", "sigmoid"):
        s = 1 / (1 + torch.exp(-g))
        if name == "sigmoid":
            return s, s * (1 - s)
        return g * s, s * (1 + g * (1 - s))
    if name == "gelu":
        c = 0.5 * (1 + torch.erf(g * math.sqrt(0.5)))
        return g * c, c + g * torch.exp(-0.5 * g * g) / math.sqrt(2 * math.pi)
    c = math.sqrt(2 / math.pi)
    t = torch.tanh(c * (g + 0.044715 * g * g * g))
    return 0.5 * g * (1 + t), 0.5 * (1 + t) + 0.5 * g * (1 - t * t) * c * (1 + 3 * 0.044715 * g * g)


def _dequantise(packed, s, z, K, group):
    q = torch.stack([packed & 15, packed >> 4], 2).flatten(1)[:, :K].float()
    s = s.float().repeat_interleave(group, 1)[:, :K]
    zf = z.float().repeat_interleave(group, 1)[:, :K] if z is not None else 8.0
    return (q - zf) * s


def run(state):
    c = state["case"]
    op, X = c["op"], state["X"]
    if own:
        import roofline_sgemm_f32_amd as rs
        if op == "glu":
            return rs.glu(X, state["Wg"], state["Wu"], act=c["act"], transw=c["linear"],
                          save=c["save"])
        if op == "backward":
            return rs.glu_backward(state["dH"], X, state["Wg"], state["Wu"], state["G"],
                                   state["U"], act=c["act"], transw=c["linear"])
        if op == "q4":
            w, s, z = state["W"][0]
            return rs.q4_matmul(X, w, s, zeros=z, group=c["group"])
        (wg, sg, zg), (wu, su, zu) = state["W"]
        return rs.q4_glu(X, wg, sg, wu, su, gate_zeros=zg, up_zeros=zu, group=c["group"],
                         act=c["act"])
    if op == "glu":
        Wg, Wu = state["Wg"], state["Wu"]
        G, U = (X @ Wg.t(), X @ Wu.t()) if c["linear"] else (X @ Wg, X @ Wu)
        H = _act(c["act"], G)[0] * U
        return (H, G, U) if c["save"] else H
    if op == "backward":
        Wg, Wu, dH = state["Wg"], state["Wu"], state["dH"]
        a, da = _act(c["act"], state["G"])
        dG, dU = dH * state["U"] * da, dH * a
        if c["linear"]:
            return dG @ Wg + dU @ Wu, dG.t() @ X, dU.t() @ X
        return dG @ Wg.t() + dU @ Wu.t(), X.t() @ dG, X.t() @ dU
    ys = [X.float() @ _dequantise(w, s, z, c["K"], c["group"]).t() for w, s, z in state["W"]]
    y = ys[0] if op == "q4" else _act(c["act"], ys[0])[0] * ys[1]
    return y.to(X.dtype)


def work(case):
    M, K = case["M"], case["K"]
    if case["op"] == "glu":
        F = case["F"]
        out = 3 * M * F if case["save"] else M * F
        return {"bytes": 4 * (M * K + 2 * K * F + out), "flops": 4 * M * K * F}
    if case["op"] == "backward":
        F = case["F"]
        return {"bytes": 4 * (2 * M * K + 4 * K * F + 3 * M * F), "flops": 8 * M * K * F}
    N, groups = case["N"], -(-K // case["group"])
    size = {"f32": 4, "f16": 2, "bf16": 2}
    weight = N * ((K + 1) // 2) + N * groups * (size[case["s"]] + (1 if case["zeros"] else 0))
    n = 2 if case["op"] == "q4_glu" else 1
    return {"bytes": n * weight + size[case["x"]] * M * (K + N), "flops": n * 2 * M * N * K}


# ---- the definition in 64 bits ----------------------------------------------

def _exact_act(name, g):
    if name == "relu":
        return g.clamp_min(0), torch.heaviside(g, torch.zeros((), dtype=g.dtype, device=g.device))
    if name == "sigmoid":
        return torch.sigmoid(g), torch.sigmoid(g) * torch.sigmoid(-g)
    if name == "silu":
        return g * torch.sigmoid(g), torch.sigmoid(g) + g * torch.sigmoid(g) * torch.sigmoid(-g)
    if name == "gelu":
        phi = torch.special.ndtr(g)
        return g * phi, phi + g * torch.exp(-g.square() / 2) * 0.39894228040143267794
    # 0.5 (1 + tanh v) = sigmoid(2 v)
    v2 = 2 * 0.79788456080286535588 * (g + 0.044715 * g.pow(3))
    s = torch.sigmoid(v2)
    return g * s, s + g * s * torch.sigmoid(-v2) * 2 * 0.79788456080286535588 * (1 + 0.134145 * g.square())


def _exact_q4(X, weight, K, group):
    """Sum over groups of (X_g (q_g - z_g)^T) s_g."""
    packed, s, z = weight
    b = packed.to(torch.int64)
    k = torch.arange(K, device=X.device)
    q = ((b[:, k // 2] >> (4 * (k % 2))) & 15).double()
    y = torch.zeros((X.shape[0], packed.shape[0]), dtype=torch.float64, device=X.device)
    for g in range(s.shape[1]):
        lo, hi = g * group, min(K, (g + 1) * group)
        zg = z[:, g:g + 1].double() if z is not None else 8.0
        y += (X[:, lo:hi] @ (q[:, lo:hi] - zg).t()) * s[:, g].double()
    return y


def exact(case, seed):
    st = prepare(case, seed)
    op, act, X = case["op"], case.get("act"), st["X"].double()
    if op in ("glu", "backward"):
        # Weights as K x F whatever their storage.
        Wg, Wu = (st[n].double().t() if case["linear"] else st[n].double() for n in ("Wg", "Wu"))
        if op == "glu":
            G, U = torch.mm(X, Wg), torch.mm(X, Wu)
            H = torch.mul(_exact_act(act, G)[0], U)
            return (H, G, U) if case["save"] else H
        a, da = _exact_act(act, st["G"].double())
        dU = a * st["dH"].double()
        dG = da * st["U"].double() * st["dH"].double()
        dX = torch.mm(dG, Wg.t()) + torch.mm(dU, Wu.t())
        dW = [torch.mm(X.t(), d) for d in (dG, dU)]
        return (dX, *((d.t() for d in dW) if case["linear"] else dW))
    ys = [_exact_q4(X, w, case["K"], case["group"]) for w in st["W"]]
    return ys[0] if op == "q4" else _exact_act(act, ys[0])[0] * ys[1]
