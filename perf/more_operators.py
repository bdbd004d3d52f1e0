"""Cases of low-rank adapters beside a projection, their gradients, and
orthogonalised updates.

Three operators, row-major throughout:

lora      Y[m] = base[m] + s_l (X[m] A_l^T) B_l^T with l = ids[m]: each row of
          the batch has the adapter of its own request, or none (an id of -1:
          Y[m] = base[m]).  A is L x R x K, B is L x N x R, s float32.  base is
          what the shared projection gave.  A training step keeps H = X A_l^T
          in float32 (zero for a row without adapter).
backward  from dY, X and H: dH[m] = s_l dY[m] B_l, dX[m] = base[m] + dH[m] A_l
          (base: the gradient through the projection), dA_l = sum dH[m]^T X[m]
          and dB_l = s_l sum dY[m]^T H[m] over the rows m of adapter l.
ortho     X = G / (|G| + eps), then per step X <- a X + (b S + c S S) X with
          S = X X^T (of the smaller side): an update whose singular values are
          all near one.  G is one matrix or a stack of them.
"""
import math

import torch

own = False

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
COEFFICIENTS = (3.4445, -4.7750, 2.0315)
EPS = 1e-7


def listed():
    return [
        # One token of one request: latency.
        {"name": "lora_one_token", "op": "lora", "M": 1, "K": 4096, "N": 4096, "R": 16, "L": 8,
         "type": "bf16", "rows": "mixed", "save": False},
        # 64 sequences decoded together, the adapters in no order.
        {"name": "lora_decode", "op": "lora", "M": 64, "K": 4096, "N": 8192, "R": 16, "L": 32,
         "type": "f16", "rows": "mixed", "save": False},
        # The prompts of some requests in one batch, each a run of rows.
        {"name": "lora_prompts", "op": "lora", "M": 8192, "K": 4096, "N": 8192, "R": 64, "L": 8,
         "type": "bf16", "rows": "runs", "save": False},
        # A float32 training batch over a few adapters, nothing aligned.
        {"name": "lora_odd", "op": "lora", "M": 1025, "K": 1023, "N": 2049, "R": 12, "L": 5,
         "type": "f32", "rows": "mixed", "save": True},
        # The backward pass of fine-tuning four adapters on one batch.
        {"name": "backward_train", "op": "backward", "M": 8192, "K": 4096, "N": 4096, "R": 16,
         "L": 4, "type": "bf16", "rows": "runs"},
        # The same in float32 at a larger rank, one adapter.
        {"name": "backward_f32", "op": "backward", "M": 2048, "K": 4096, "N": 2048, "R": 64, "L": 1,
         "type": "f32", "rows": "runs"},
        # A short odd batch whose rows are of many adapters.
        {"name": "backward_odd", "op": "backward", "M": 257, "K": 1023, "N": 1027, "R": 8, "L": 6,
         "type": "f16", "rows": "mixed"},
        # The updates of 16 adapters' A factors.
        {"name": "ortho_factors", "op": "ortho", "batch": 16, "M": 16, "N": 4096, "type": "f32"},
        # A small weight.
        {"name": "ortho_small", "op": "ortho", "batch": 1, "M": 256, "N": 256, "type": "f32"},
        # A wide weight's half-precision gradient.
        {"name": "ortho_wide", "op": "ortho", "batch": 1, "M": 1024, "N": 4096, "type": "bf16"},
        # A stack of tall odd weights.
        {"name": "ortho_odd", "op": "ortho", "batch": 3, "M": 1027, "N": 509, "type": "f32"},
        # A square weight of a mid-size model.
        {"name": "ortho_square", "op": "ortho", "batch": 1, "M": 4096, "N": 4096, "type": "f32"},
    ]


def draw(rng):
    """A case of the same ranges: 1 to 8192 rows of 64 to 8192, adapters of ranks 4
    to 128, updates of sides 16 to 4096."""
    def size(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    def width(lo, hi):
        n = size(lo, hi)
        # Half of the widths are multiples of 64, as most models' are.
        return max(lo, n // 64 * 64) if rng.random() < 0.5 else n

    op = rng.choice(["lora", "backward", "ortho"])
    case = {"op": op, "type": rng.choice(list(TYPES))}
    if op == "ortho":
        m, n = width(16, 4096), width(16, 4096)
        case.update(M=m, N=n, batch=rng.randint(1, max(1, min(16, 2 ** 24 // (m * n)))))
        return case
    R = rng.choice([4, 8, 16, 32, 64, 128]) if rng.random() < 0.7 else rng.randint(4, 128)
    case.update(M=size(1, 8192), K=width(64, 8192), N=width(64, 8192), R=R, L=size(1, 32),
                rows=rng.choice(["mixed", "runs"]))
    if rng.random() < 0.3:
        case["M"] = rng.randint(1, 64)  # decoding steps
    if op == "lora":
        case["save"] = rng.random() < 0.3
    return case


# ---- inputs -----------------------------------------------------------------

def _ids(gen, M, L, rows):
    """Adapters of M rows: mixed (any order) or in runs of one request each;
    about one request in eight has none."""
    if rows == "mixed":
        n = M
    else:
        n = min(M, max(L, 1) + 2)  # requests
    of = torch.randint(0, L, (n,), generator=gen, device="cuda", dtype=torch.int32)
    none = torch.rand((n,), generator=gen, device="cuda") < 0.125
    if n == 1 or L == 1:
        none[0] = False
    of = torch.where(none, torch.full_like(of, -1), of)
    if rows == "mixed":
        return of
    ends = torch.sort(torch.randint(0, M, (n - 1,), generator=gen, device="cuda"))[0]
    return of[torch.searchsorted(ends, torch.arange(M, device="cuda"), right=True)].contiguous()


def _activations(gen, M, K):
    """Normal activations with a few channels ten times larger, as residual
    streams have them."""
    x = torch.randn((M, K), generator=gen, device="cuda")
    big = torch.rand((K,), generator=gen, device="cuda") < 0.01
    return torch.where(big, 10 * x, x)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    t = TYPES[case["type"]]
    st = {"case": case}
    if case["op"] == "ortho":
        b, m, n = case["batch"], case["M"], case["N"]
        # A gradient: noise, and a part of low rank that is larger.
        g = torch.randn((b, m, n), generator=gen, device="cuda")
        u = torch.randn((b, m, 4), generator=gen, device="cuda")
        v = torch.randn((b, 4, n), generator=gen, device="cuda")
        g = (1e-3 * (g + 0.5 * torch.bmm(u, v))).to(t)
        st["G"] = g if b > 1 else g[0]
        return st
    M, K, N, R, L = (case[k] for k in "MKNRL")
    st["ids"] = _ids(gen, M, L, case["rows"])
    st["scale"] = 0.5 + torch.rand((L,), generator=gen, device="cuda")
    st["A"] = (torch.randn((L, R, K), generator=gen, device="cuda") / math.sqrt(K)).to(t)
    st["B"] = (torch.randn((L, N, R), generator=gen, device="cuda") / math.sqrt(R)).to(t)
    X = _activations(gen, M, K)
    st["X"] = X.to(t)
    if case["op"] == "lora":
        st["base"] = torch.randn((M, N), generator=gen, device="cuda").to(t)
        return st
    st["dY"] = (torch.randn((M, N), generator=gen, device="cuda") / math.sqrt(M)).to(t)
    st["base"] = (torch.randn((M, K), generator=gen, device="cuda") / math.sqrt(M)).to(t)
    # H as the forward pass left it.
    H = torch.zeros((M, R), device="cuda")
    for l in range(L):
        rows = (st["ids"] == l).nonzero()[:, 0]
        H[rows] = st["X"][rows].float() @ st["A"][l].float().t()
    st["H"] = H
    return st


# ---- one pass ---------------------------------------------------------------

def _plain_lora(X, A, B, ids, scale, base):
    M, R = X.shape[0], A.shape[1]
    Y = base.float()
    H = torch.zeros((M, R), device=X.device)
    if M * R * (A.shape[2] + B.shape[1]) <= 1 << 24:  # few rows: every row's own adapter
        has, l = ids >= 0, ids.clamp_min(0).long()
        H = torch.where(has[:, None], (A[l].float() * X.float()[:, None, :]).sum(2), H)
        D = (B[l].float() * H[:, None, :]).sum(2) * scale[l][:, None]
        return torch.where(has[:, None], Y + D, Y).to(X.dtype), H
    for l in range(A.shape[0]):
        rows = (ids == l).nonzero()[:, 0]
        if rows.numel():
            h = X[rows].float() @ A[l].float().t()
            H[rows] = h
            Y = Y.index_add(0, rows, h @ B[l].float().t() * scale[l]) if Y is base else \
                Y.index_add_(0, rows, h @ B[l].float().t() * scale[l])
    return Y.to(X.dtype), H


def _plain_backward(dY, X, A, B, H, ids, scale, base):
    dX = base.to(torch.float32, copy=True)
    dA = torch.zeros(A.shape, device=X.device)
    dB = torch.zeros(B.shape, device=X.device)
    for l in range(A.shape[0]):
        rows = (ids == l).nonzero()[:, 0]
        if rows.numel():
            dy = dY[rows].float() * scale[l]
            dh = dy @ B[l].float()
            dX.index_add_(0, rows, dh @ A[l].float())
            dA[l] = dh.t() @ X[rows].float()
            dB[l] = dy.t() @ H[rows]
    return dX.to(X.dtype), dA.to(X.dtype), dB.to(X.dtype)


def _plain_ortho(G):
    x = G.float()
    if G.dim() == 2:
        x = x[None]
    tall = x.shape[1] > x.shape[2]
    if tall:
        x = x.transpose(1, 2).contiguous()
    a, b, c = COEFFICIENTS
    norm = x.double().square().sum((1, 2), keepdim=True).sqrt()  # a long sum
    x = x / (norm + EPS).float()
    for _ in range(5):
        s = torch.bmm(x, x.transpose(1, 2))
        x = a * x + torch.bmm(b * s + c * torch.bmm(s, s), x)
    if tall:
        x = x.transpose(1, 2)
    return x.reshape(G.shape).to(G.dtype)


def run(state):
    c = state["case"]
    if own:
        import roofline_sgemm_f32_amd as rs
        if c["op"] == "ortho":
            return rs.orthogonalize(state["G"], steps=5, coefficients=COEFFICIENTS, eps=EPS)
        X, A, B, ids, scale, base = (state[k] for k in ("X", "A", "B", "ids", "scale", "base"))
        if c["op"] == "lora":
            return rs.lora(X, A, B, ids, scale=scale, base=base, save=c["save"])
        return rs.lora_backward(state["dY"], X, A, B, state["H"], ids, scale=scale, base=base)
    if c["op"] == "ortho":
        return _plain_ortho(state["G"])
    args = [state[k] for k in ("X", "A", "B")]
    rest = [state[k] for k in ("ids", "scale", "base")]
    if c["op"] == "lora":
        Y, H = _plain_lora(*args, *rest)
        return (Y, H) if c["save"] else Y
    return _plain_backward(state["dY"], *args, state["H"], *rest)


def work(case):
    """Adapters count as far as rows can be of them; of the symmetric products
    one half counts."""
    size = 4 if case["type"] == "f32" else 2
    if case["op"] == "ortho":
        m, n = sorted((case["M"], case["N"]))
        return {"bytes": 2 * case["batch"] * m * n * size,
                "flops": case["batch"] * 5 * (3 * m * m * n + m * m * m)}
    M, K, N, R, L = (case[k] for k in "MKNRL")
    used = min(L, M) * R * (K + N) * size
    flops = 2 * M * R * (K + N)
    if case["op"] == "lora":
        rows = M * (K + 2 * N) * size + (4 * M * R if case["save"] else 0)
        return {"bytes": rows + used + 4 * M + 4 * L, "flops": flops}
    rows = M * (3 * K + N) * size + 4 * M * R
    return {"bytes": rows + used + L * R * (K + N) * size + 4 * M + 4 * L, "flops": 2 * flops}


# ---- the definition in 64 bits ----------------------------------------------

def _of_adapter(st):
    """M x L: the scale where the row has the adapter, else zero, and the mask
    itself, in 64 bits."""
    L = st["A"].shape[0]
    mask = (st["ids"].long()[:, None] == torch.arange(L, device="cuda")[None, :]).double()
    return mask, mask * st["scale"].double()[None, :]


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "ortho":
        out = []
        for g in (st["G"][None] if st["G"].dim() == 2 else st["G"]):
            x = g.double()
            x = torch.div(x, torch.linalg.vector_norm(x) + EPS)
            left = x.shape[0] <= x.shape[1]
            eye = torch.eye(min(x.shape), dtype=torch.float64, device=x.device)
            a, b, c = COEFFICIENTS
            for _ in range(5):
                s = torch.mm(x, x.t()) if left else torch.mm(x.t(), x)
                p = a * eye + torch.mm(s, b * eye + c * s)
                x = torch.mm(p, x) if left else torch.mm(x, p)
            out.append(x)
        return out[0] if st["G"].dim() == 2 else torch.stack(out)
    mask, scaled = _of_adapter(st)
    X, A, B = st["X"].double(), st["A"].double(), st["B"].double()
    L = A.shape[0]
    if case["op"] == "lora":
        Y, H = st["base"].double(), torch.zeros((X.shape[0], A.shape[1]), dtype=torch.float64, device="cuda")
        for l in range(L):
            h = torch.mm(X, A[l].t())
            H += mask[:, l:l + 1] * h
            Y = Y + torch.mm(scaled[:, l:l + 1] * h, B[l].t())
        return (Y, H) if case["save"] else Y
    dY, H, dX = st["dY"].double(), st["H"].double(), st["base"].double()
    dA, dB = torch.empty_like(A), torch.empty_like(B)
    for l in range(L):
        d = scaled[:, l:l + 1] * dY
        dH = torch.mm(d, B[l])
        dX = dX + torch.mm(dH, A[l])
        dA[l] = torch.mm(dH.t(), X)
        dB[l] = torch.mm(d.t(), H)
    return dX, dA, dB
