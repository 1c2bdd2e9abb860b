"""Cases of the operators on a model's hidden matrices, next to a rank's
sharded optimizer step: their products, forward and backward, and the step by
orthogonalised momentum (Muon) that trains them.

  linear         y = act(x W^T + b) + residual; W and b are tensors of the
                 rank's flat 16-bit parameter buffer.  A training pass also
                 keeps the sum before act.  The tied output table is such a W.
  linear_grad    its backward pass from dz = dloss / d(x W^T + b):
                 dx = (dz W) * act'(pre), where x = act(pre) came out of the
                 layer before, and dW = scale dz^T x, db = scale colsum(dz),
                 into the rank's flat gradient buffer or one owner's slice
  orthogonalize  each matrix G of a flat 16-bit buffer by Newton-Schulz
                 products: X = G / (|G| + eps), then `steps` times
                 X <- a X + (b A + c A A) X with A = X X^T, times a factor
  muon_momentum  g = grad_scale * sum over the ranks' slices, in rank order,
                 M <- mu M + g, U = g + mu M rounded into the flat buffer that
                 orthogonalize reads
  muon_apply     w <- (1 - lr decay) w - lr O, and the 16-bit parameters

Where ``own`` is false the operators are elementary torch operations in 32
bits, rounded once; where it is true they are the library's calls.
"""
import math

import torch

own = False

DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16}
CODES = {"f32": 0, "f16": 1, "bf16": 2}
ACTS = {"none": 0, "relu": 1, "gelu": 2, "gelu_tanh": 3, "silu": 4}
NS_STEPS, NS_A, NS_B, NS_C, NS_EPS = 5, 3.4445, -4.7750, 2.0315, 1e-7
MU, LR, DECAY = 0.95, 0.02, 0.1
ALIGN = 64                    # shard alignment of the flat buffers, elements


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------

def _linear(rows, inner, outer, dt, act, bias, residual, train):
    return {"op": "linear", "rows": rows, "in": inner, "out": outer, "dtype": dt, "act": act, "bias": bias,
            "residual": residual, "train": train}


def _linear_grad(rows, inner, outer, dt, act, bias, ranks=1, rank=-1):
    return {"op": "linear_grad", "rows": rows, "in": inner, "out": outer, "dtype": dt, "act": act, "bias": bias,
            "ranks": ranks, "rank": rank}


def _ortho(count, rows, cols, dt):
    return {"op": "orthogonalize", "count": count, "rows": rows, "cols": cols, "dtype": dt}


def _momentum(n, ranks, dt, full):
    return {"op": "muon_momentum", "n": n, "ranks": ranks, "dtype": dt, "full": full}


def _apply(n, ranks, dt):
    return {"op": "muon_apply", "n": n, "ranks": ranks, "dtype": dt}


def listed():
    cases = {
        # One token through a square projection of GPT-2-small: latency alone.
        "linear one row": _linear(1, 768, 768, "bf16", "none", True, True, False),
        # The tied output table of GPT-2-small: logits of 2048 tokens, whose rows are odd.
        "linear odd head": _linear(2048, 768, 50257, "bf16", "none", False, False, False),
        # The widening product of an 8192-wide layer on 4096 tokens, kept for the backward pass.
        "linear wide": _linear(4096, 8192, 32768, "bf16", "gelu", True, False, True),
        # The backward pass of a square GPT-2-small projection, one owner's slice of eight.
        "linear_grad owner slice": _linear_grad(8191, 768, 768, "f16", "none", True, ranks=8, rank=3),
        # The backward pass of a square 8192-wide product behind an activation.
        "linear_grad wide": _linear_grad(8192, 8192, 8192, "bf16", "gelu_tanh", True),
        # One small odd matrix.
        "orthogonalize small odd": _ortho(1, 65, 33, "bf16"),
        # The attention weights of GPT-2-small: 12 layers of four.
        "orthogonalize gpt2": _ortho(48, 768, 768, "bf16"),
        # One square weight of an 8192-wide layer.
        "orthogonalize wide": _ortho(1, 8192, 8192, "bf16"),
        # A small odd matrix's share, two ranks.
        "muon_momentum small": _momentum(65 * 33, 2, "f16", True),
        # The hidden matrices of GPT-2-small (12 layers of 12 * 768^2) over eight ranks.
        "muon_momentum gpt2": _momentum(12 * 12 * 768 * 768, 8, "bf16", True),
        # A small odd matrix, one rank.
        "muon_apply small": _apply(65 * 33, 1, "bf16"),
        # The matrices of one 8192-wide layer (12 * 8192^2) over eight ranks.
        "muon_apply wide": _apply(12 * 8192 * 8192, 8, "f16"),
    }
    return [{"name": k, **v} for k, v in cases.items()]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng):
    n = _log(rng, 32, 16384)
    return max(64, n // 64 * 64) if rng.random() < 0.6 else n


def draw(rng):
    op = rng.choice(["linear", "linear", "linear_grad", "linear_grad", "orthogonalize", "orthogonalize",
                     "muon_momentum", "muon_apply"])
    dt = rng.choice(["bf16", "f16"])
    if op in ("linear", "linear_grad"):
        rows, inner, outer = _log(rng, 1, 16384), _width(rng), _width(rng)
        while rows * inner * outer > 1 << 39:
            rows = max(1, rows // 2)
        act, bias = rng.choice(list(ACTS)), rng.random() < 0.7
        if op == "linear":
            return _linear(rows, inner, outer, dt, act, bias, rng.random() < 0.5, rng.random() < 0.5)
        ranks = rng.choice([1, 1, 4, 8])
        return _linear_grad(rows, inner, outer, dt, act, bias, ranks, -1 if ranks == 1 else rng.randrange(ranks))
    if op == "orthogonalize":
        rows, cols, count = _log(rng, 16, 8192), _log(rng, 16, 8192), _log(rng, 1, 64)
        if rng.random() < 0.6:
            rows, cols = max(64, rows // 64 * 64), max(64, cols // 64 * 64)
        while count > 1 and count * rows * cols > 1 << 25:
            count //= 2
        return _ortho(count, rows, cols, dt)
    n = _log(rng, 1000, 1 << 28)
    if op == "muon_momentum":
        ranks = rng.choice([1, 2, 4, 8, 16, 24])
        return _momentum(n, ranks, dt, rng.random() < 0.5)
    return _apply(n, rng.choice([1, 2, 4, 8, 16]), dt)


# ---------------------------------------------------------------------------
# What a program has in hand
# ---------------------------------------------------------------------------

def _padded(n, ranks):
    return -(-n // (ranks * ALIGN)) * ranks * ALIGN


def _slice(case):
    """(elements of the flat gradient buffer, first, last + 1) of the part returned."""
    padded = _padded(case["in"] * case["out"] + case["out"] * case["bias"], case["ranks"])
    if case["rank"] < 0:
        return padded, 0, padded
    share = padded // case["ranks"]
    return padded, case["rank"] * share, (case["rank"] + 1) * share


def _owner(case):
    return case["ranks"] // 2      # the rank whose share a muon case takes


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = dict(case)
    dt = DTYPES[case["dtype"]]

    def normal(shape, sigma, dtype=dt):
        return torch.empty(shape, device="cuda", dtype=dtype).normal_(0, sigma, generator=g)

    op = case["op"]
    if op in ("linear", "linear_grad"):
        rows, inner, outer = case["rows"], case["in"], case["out"]
        s["params"] = normal(_padded(inner * outer + outer * case["bias"], case.get("ranks", 1)), 0.02)
        if op == "linear":
            s["x"] = normal((rows, inner), 1.0)
            s["residual"] = normal((rows, outer), 1.0) if case["residual"] else None
            s["y"] = torch.empty((rows, outer), device="cuda", dtype=dt)
            s["pre"] = torch.empty_like(s["y"]) if case["train"] else None
        else:
            s["dz"] = normal((rows, outer), 1.0)
            s["pre"] = normal((rows, inner), 1.0)
            s["x"] = torch.empty_like(s["pre"])
            for a in range(0, rows, 4096):
                s["x"][a:a + 4096] = _act(case["act"], s["pre"][a:a + 4096].float()).to(dt)
            s["scale"] = 1.0 / rows
            _, lo, hi = _slice(case)
            s["dx"] = torch.empty_like(s["x"])
            s["grad"] = torch.zeros(hi - lo, device="cuda", dtype=dt)
    elif op == "orthogonalize":
        # A few strong directions over noise, as an update's matrices have.
        count, rows, cols = case["count"], case["rows"], case["cols"]
        s["src"] = torch.zeros(_padded(count * rows * cols, 1), device="cuda", dtype=dt)
        rank = min(16, rows, cols)
        fade = 1.0 / torch.arange(1, rank + 1, device="cuda")
        for m in s["src"][:count * rows * cols].view(count, rows, cols):
            left, right = normal((rows, rank), 1.0, torch.float32), normal((rank, cols), 1.0, torch.float32)
            m.copy_(1e-3 * (normal((rows, cols), 0.5, torch.float32) + (left * fade) @ right))
        s["dst"] = torch.zeros(s["src"].numel(), device="cuda", dtype=torch.bfloat16)
        s["scale"] = 0.2 * math.sqrt(max(rows, cols))
    else:
        padded = _padded(case["n"], case["ranks"])
        share = padded // case["ranks"]
        if op == "muon_momentum":
            # Each slice starts on its own 256-byte boundary, as received slices do.
            s["slices"] = [normal(share, 1e-3) for _ in range(case["ranks"])]
            s["momentum"] = normal(share, 1e-2, torch.float32)
            s["update"] = torch.zeros(padded if case["full"] else share, device="cuda", dtype=torch.bfloat16)
        else:
            s["direction"] = normal(padded, 0.2, torch.bfloat16)
            s["master"] = normal(share, 0.02, torch.float32)
            s["params"] = torch.zeros(padded, device="cuda", dtype=dt)
    if own:
        _handles(s)
    return s


def work(case):
    op = case["op"]
    if op == "linear":
        r, i, o = case["rows"], case["in"], case["out"]
        outs = 1 + case["residual"] + case["train"]
        return {"bytes": 2 * (r * i + i * o + o * case["bias"] + r * o * outs), "flops": 2 * r * i * o}
    if op == "linear_grad":
        r, i, o = case["rows"], case["in"], case["out"]
        _, lo, hi = _slice(case)
        share = max(0, min(hi, i * o) - lo) / (i * o)          # of the weight's gradient
        read = r * o + r * i + r * i * (case["act"] != "none") + i * o
        return {"bytes": 2 * (read + r * i + hi - lo), "flops": 2 * r * i * o * (1 + share)}
    if op == "orthogonalize":
        n, m = sorted((case["rows"], case["cols"]))
        # A and A A are symmetric: half of their products.
        return {"bytes": 4 * case["count"] * n * m, "flops": case["count"] * NS_STEPS * (n * n * m + n ** 3 + 2 * n * n * m)}
    share = _padded(case["n"], case["ranks"]) // case["ranks"]
    if op == "muon_momentum":
        return {"bytes": share * (2 * case["ranks"] + 8 + 2), "flops": share * (case["ranks"] + 5)}
    return {"bytes": share * (2 + 8 + 2), "flops": share * 3}


# ---------------------------------------------------------------------------
# The library's calls
# ---------------------------------------------------------------------------

def _handles(s):
    import zero_sharded_mixed_02_amd as Z
    op, code, need = s["op"], CODES[s["dtype"]], 0
    if op in ("linear", "linear_grad"):
        sizes = [s["in"] * s["out"]] + ([s["out"]] if s["bias"] else [])
        s["plan"] = Z.zero_plan(sum(sizes), s.get("ranks", 1), sizes, 0, ALIGN)
        if op == "linear":
            need = Z.zero_linear_workspace_bytes(s["plan"], 0, s["in"], s["rows"])
        else:
            need = max(Z.zero_linear_input_grad_workspace_bytes(s["plan"], 0, s["in"], s["rows"]),
                       Z.zero_linear_weight_grad_workspace_bytes(s["plan"], 0, s["in"], s["rows"], s["rank"]))
    elif op == "orthogonalize":
        n = s["rows"] * s["cols"]
        s["plan"] = Z.zero_plan(s["count"] * n, 1, [n] * s["count"], 0, ALIGN)
        s["matrices"] = Z.Matrices([(t, s["rows"], s["cols"], s["scale"]) for t in range(s["count"])])
        need = Z.zero_orthogonalize_workspace_bytes(s["plan"], s["matrices"])
    else:
        s["plan"] = Z.zero_plan(s["n"], s["ranks"], [s["n"]], 0, ALIGN)
        s["hyper"] = Z.MuonHyper(lr=LR, momentum=MU, weight_decay=DECAY, grad_scale=1.0 / s["ranks"], nesterov=True)
        if op == "muon_momentum":
            s["src"] = Z.GradSrc(code, s["slices"])
    s["ws"] = torch.empty(max(1, need), device="cuda", dtype=torch.uint8)
    s["Z"], s["code"] = Z, code


def _run_own(s):
    Z, op, code = s["Z"], s["op"], s["code"]
    if op == "linear":
        Z.zero_linear(s["plan"], 0, s["in"], s["params"], code, s["x"], s["y"], bias=1 if s["bias"] else -1,
                      act=ACTS[s["act"]], residual=s["residual"], pre=s["pre"], workspace=s["ws"])
        return {"y": s["y"], "pre": s["pre"]}
    if op == "linear_grad":
        Z.zero_linear_input_grad(s["plan"], 0, s["in"], s["params"], code, s["dz"], s["dx"], act=ACTS[s["act"]],
                                 pre=s["pre"] if s["act"] != "none" else None, workspace=s["ws"])
        Z.zero_linear_weight_grad(s["plan"], 0, s["in"], s["dz"], s["x"], code, s["scale"], s["grad"], code,
                                  bias=1 if s["bias"] else -1, rank=s["rank"], workspace=s["ws"])
        return {"dx": s["dx"], "grad": s["grad"]}
    if op == "orthogonalize":
        Z.zero_orthogonalize(s["plan"], s["matrices"], s["src"], code, s["dst"], Z.ZERO_BF16, workspace=s["ws"])
        return s["dst"]
    if op == "muon_momentum":
        Z.zero_muon_momentum(s["plan"], _owner(s), s["hyper"], s["src"], None, s["momentum"], s["update"], Z.ZERO_BF16,
                             s["full"])
        return {"momentum": s["momentum"], "update": s["update"]}
    Z.zero_muon_apply(s["plan"], _owner(s), s["hyper"], s["direction"], Z.ZERO_BF16, True, s["master"], s["params"],
                      code, True)
    return {"master": s["master"], "params": s["params"]}


# ---------------------------------------------------------------------------
# The plain forms
# ---------------------------------------------------------------------------

def _act(name, z):
    if name == "relu":
        return torch.clamp(z, min=0)
    if name == "gelu":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    if name == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)))
    if name == "silu":
        return z / (1 + torch.exp(-z))
    return z


def _act_slope(name, z):
    if name == "relu":
        return (z > 0).to(z.dtype)
    if name == "gelu":
        return 0.5 * (1 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    if name == "gelu_tanh":
        k = math.sqrt(2 / math.pi)
        t = torch.tanh(k * (z + 0.044715 * z * z * z))
        return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * k * (1 + 3 * 0.044715 * z * z)
    if name == "silu":
        e = 1 / (1 + torch.exp(-z))
        return e * (1 + z * (1 - e))
    return torch.ones_like(z)


def _run_plain(s):
    op, dt = s["op"], DTYPES[s["dtype"]]
    if op in ("linear", "linear_grad"):
        inner, outer = s["in"], s["out"]
        weight = s["params"][:inner * outer].view(outer, inner).float()
    if op == "linear":
        z = s["x"].float() @ weight.t()
        if s["bias"]:
            z += s["params"][inner * outer:inner * outer + outer].float()
        pre = z.to(dt) if s["train"] else None
        y = _act(s["act"], z)
        if s["residual"] is not None:
            y = y + s["residual"].float()
        return {"y": y.to(dt), "pre": pre}
    if op == "linear_grad":
        dz = s["dz"].float()
        dx = dz @ weight
        if s["act"] != "none":
            dx = dx * _act_slope(s["act"], s["pre"].float())
        padded, lo, hi = _slice(s)
        flat = torch.zeros(padded, device="cuda")
        flat[:inner * outer] = (dz.t() @ s["x"].float()).view(-1) * s["scale"]
        if s["bias"]:
            flat[inner * outer:inner * outer + outer] = dz.sum(0) * s["scale"]
        return {"dx": dx.to(dt), "grad": flat[lo:hi].to(dt)}
    if op == "orthogonalize":
        count, rows, cols = s["count"], s["rows"], s["cols"]
        x = s["src"][:count * rows * cols].view(count, rows, cols).float()
        x = x / (torch.sqrt((x * x).sum((1, 2), keepdim=True)) + NS_EPS)
        if rows > cols:
            x = x.transpose(1, 2).contiguous()
        for _ in range(NS_STEPS):
            a = torch.bmm(x, x.transpose(1, 2).contiguous())
            x = NS_A * x + torch.bmm(NS_B * a + NS_C * torch.bmm(a, a), x)
        if rows > cols:
            x = x.transpose(1, 2)
        out = torch.zeros(s["src"].numel(), device="cuda", dtype=torch.bfloat16)
        out[:count * rows * cols] = (x * s["scale"]).to(torch.bfloat16).reshape(-1)
        return out
    rank = _owner(s)
    if op == "muon_momentum":
        total = s["slices"][0].float()
        for q in range(1, s["ranks"]):
            total = total + s["slices"][q].float()
        total = total * (1.0 / s["ranks"])
        s["momentum"].mul_(MU).add_(total)
        update = (total + MU * s["momentum"]).to(torch.bfloat16)
        if not s["full"]:
            return {"momentum": s["momentum"], "update": update}
        s["update"][rank * update.numel():(rank + 1) * update.numel()] = update
        return {"momentum": s["momentum"], "update": s["update"]}
    share = s["master"].numel()
    mine = slice(rank * share, (rank + 1) * share)
    s["master"].mul_(1 - LR * DECAY).sub_(LR * s["direction"][mine].float())
    s["params"][mine] = s["master"].to(dt)
    return {"master": s["master"], "params": s["params"]}


def run(s):
    return _run_own(s) if own else _run_plain(s)


# ---------------------------------------------------------------------------
# In 64 bits
# ---------------------------------------------------------------------------

def _phi(z):
    return torch.special.erfc(-z / math.sqrt(2.0)) / 2


def _act64(name, z):
    return {"none": lambda: z, "relu": lambda: torch.where(z > 0, z, 0.0), "gelu": lambda: z * _phi(z),
            "gelu_tanh": lambda: z * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)),
            "silu": lambda: z * torch.sigmoid(z)}[name]()


def _slope64(name, z):
    with torch.enable_grad():
        z = z.detach().requires_grad_(True)
        return torch.autograd.grad(_act64(name, z).sum(), z)[0]


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("linear", "linear_grad"):
        rows, inner, outer = case["rows"], case["in"], case["out"]
        weight = s["params"][:inner * outer].double().view(outer, inner)
        bias = s["params"][inner * outer:inner * outer + outer].double() if case["bias"] else None
        step = max(1, (1 << 27) // max(inner, outer))
    if op == "linear":
        y = torch.empty((rows, outer), device="cuda", dtype=torch.float64)
        pre = torch.empty_like(y) if case["train"] else None
        for a in range(0, rows, step):
            z = torch.nn.functional.linear(s["x"][a:a + step].double(), weight, bias)
            y[a:a + step] = _act64(case["act"], z)
            if pre is not None:
                pre[a:a + step] = z
            if s["residual"] is not None:
                y[a:a + step] += s["residual"][a:a + step].double()
        return {"y": y, "pre": pre}
    if op == "linear_grad":
        padded, lo, hi = _slice(case)
        dx = torch.empty((rows, inner), device="cuda", dtype=torch.float64)
        flat = torch.zeros(padded, device="cuda", dtype=torch.float64)
        wide = flat[:inner * outer].view(outer, inner)
        for a in range(0, rows, step):
            dz = s["dz"][a:a + step].double()
            dx[a:a + step] = torch.mm(dz, weight) * _slope64(case["act"], s["pre"][a:a + step].double())
            wide.addmm_(dz.t(), s["x"][a:a + step].double(), alpha=1.0 / rows)
            if case["bias"]:
                flat[inner * outer:inner * outer + outer] += dz.sum(0) / rows
        return {"dx": dx, "grad": flat[lo:hi]}
    if op == "orthogonalize":
        rows, cols, size = case["rows"], case["cols"], case["rows"] * case["cols"]
        out = torch.zeros(s["src"].numel(), device="cuda", dtype=torch.float64)
        for k in range(case["count"]):
            x = s["src"][k * size:(k + 1) * size].double().view(rows, cols)
            x = x / (torch.linalg.vector_norm(x) + NS_EPS)
            for _ in range(NS_STEPS):
                if rows <= cols:
                    gram = x @ x.mT
                    x = NS_A * x + NS_B * (gram @ x) + NS_C * (gram @ (gram @ x))
                else:
                    gram = x.mT @ x
                    x = NS_A * x + NS_B * (x @ gram) + NS_C * ((x @ gram) @ gram)
            out[k * size:(k + 1) * size] = x.reshape(-1) * s["scale"]
        return out
    rank, ranks = _owner(case), case["ranks"]
    if op == "muon_momentum":
        g = torch.zeros(s["momentum"].numel(), device="cuda", dtype=torch.float64)
        for q in s["slices"]:
            g += q
        g /= ranks
        m = MU * s["momentum"].double() + g
        out = torch.zeros(s["update"].numel(), device="cuda", dtype=torch.float64)
        lo = rank * g.numel() if case["full"] else 0
        out[lo:lo + g.numel()] = g + MU * m
        return {"momentum": m, "update": out}
    n = s["master"].numel()
    w = s["master"].double()
    w = w - LR * (DECAY * w + s["direction"][rank * n:(rank + 1) * n].double())
    out = torch.zeros(s["params"].numel(), device="cuda", dtype=torch.float64)
    out[rank * n:(rank + 1) * n] = w
    return {"master": w, "params": out}
