"""What is measured of the operators of a transformer block: three of them,
each in plain torch (``own`` false) and through this package (``own`` true).

  gated    H = act(X Wg^T) * (X Wu^T), and as a training step with the
           gradients of X, Wg and Wu;
  lora     Y = X W^T + b + scale_i (X A_i^T) B_i^T, adapter i = index[token]
           (-1: none), the low-rank adapters of many requests at once;
  qknorm   RMS norm of each query and key head, times a weight, then the
           position rotation, and as a training step with its gradients.
"""
import math

import torch

own = False

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
EPS = 1e-6


# ------------------------------------------------------------------ cases --

def listed():
    return [
        # serving: the next token of one sequence, where the weights' bytes are all there is
        dict(name="gated 1 token", op="gated", M=1, K=2048, F=8192, act="silu", train=False),
        # serving: the next tokens of two dozen sequences
        dict(name="gated 24 tokens", op="gated", M=24, K=4096, F=8192, act="silu", train=False),
        # serving: a prompt of odd length, the width no power of two
        dict(name="gated prompt 777", op="gated", M=777, K=2048, F=5504, act="gelu_tanh", train=False),
        # training: the 192-atom water box, 64 edge tokens per atom, 256 -> 1024
        dict(name="gated train 192 atoms", op="gated", M=12288, K=256, F=1024, act="silu", train=True),
        # training: a batch of 8192 tokens, the largest
        dict(name="gated train 8192", op="gated", M=8192, K=2048, F=8192, act="silu", train=True),
        # serving: 16 sequences' next tokens, each with an adapter of its own choice
        dict(name="lora 16 tokens", op="lora", M=16, K=2048, N=2048, R=16, n=64, run=1, bias=False),
        # serving: an odd number of sequences, some tokens each, a wide projection (q, k and v)
        dict(name="lora 131 tokens", op="lora", M=131, K=4096, N=6144, R=32, n=40, run=3, bias=True),
        # serving: a dozen prompts at once, some without an adapter
        dict(name="lora prompts 6000", op="lora", M=6000, K=4096, N=4096, R=16, n=12, run=500, bias=False),
        # serving: eight sequences' next tokens
        dict(name="qknorm 8 tokens", op="qknorm", T=8, Hq=32, Hk=8, D=128, rot=128, type="bf16",
             pairs=False, train=False),
        # serving: prompts
        dict(name="qknorm 16384 tokens", op="qknorm", T=16384, Hq=32, Hk=8, D=128, rot=128, type="bf16",
             pairs=False, train=False),
        # training in FP32, as many key heads as query heads, odd length
        dict(name="qknorm train 4099", op="qknorm", T=4099, Hq=16, Hk=16, D=64, rot=64, type="f32",
             pairs=False, train=True),
        # training, neighbouring pairs, a part of each head rotated, head width no power of two
        dict(name="qknorm train 12001", op="qknorm", T=12001, Hq=24, Hk=4, D=96, rot=64, type="f16",
             pairs=True, train=True),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _width(rng, lo, hi):
    """A width: mostly a multiple of 64, some of 8, a few odd."""
    w = _log(rng, lo, hi)
    step = rng.choice([64, 64, 64, 8, 1])
    return max(step, w // step * step)


def draw(rng):
    op = rng.choice(["gated", "gated", "lora", "qknorm", "qknorm"])
    if op == "gated":
        train = rng.random() < 0.5
        M = _log(rng, 16 if train else 1, 16384)
        K = _width(rng, 128, 4096)
        F = _width(rng, 256, 8192)
        while M * K * F > (1 << 37):                 # the largest listed one's work
            M = M * 2 // 3
        return dict(op=op, M=M, K=K, F=F, act=rng.choice(["silu", "gelu", "gelu_tanh", "relu", "sigmoid"]),
                    train=train)
    if op == "lora":
        M = _log(rng, 1, 8192)
        return dict(op=op, M=M, K=_width(rng, 256, 4096), N=_width(rng, 256, 6144),
                    R=rng.choice([4, 8, 16, 16, 32, 64]), n=_log(rng, 1, 64),
                    run=rng.choice([1, 1, 7, 200, 1500]), bias=rng.random() < 0.5)
    D = rng.choice([64, 64, 80, 96, 128, 128, 128, 192, 256, 33 * 2])
    return dict(op=op, T=_log(rng, 1, 16384), Hq=rng.choice([4, 8, 12, 16, 32]), Hk=rng.choice([1, 2, 4, 8]), D=D,
                rot=rng.choice([D, D, D // 4 * 2]), type=rng.choice(["f32", "bf16", "f16"]),
                pairs=rng.random() < 0.4, train=rng.random() < 0.5)


# ----------------------------------------------------------------- inputs --

def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, std=1.0):
        return torch.randn(*shape, generator=g, device="cuda") * std

    c = dict(case)
    s = {"case": c}
    if c["op"] == "gated":
        M, K, F = c["M"], c["K"], c["F"]
        s["X"] = normal(M, K)
        s["Wg"], s["Wu"] = normal(F, K, std=K ** -0.5), normal(F, K, std=K ** -0.5)
        if c["train"]:
            s["dH"] = normal(M, F)
        elif own:
            # a serving program lays its weights out once; a training step does it each time (in run)
            import fp32_emulated_gemm_split_gb300 as emu
            s["w"] = emu.emu_gated_pack(s["Wg"], s["Wu"])
    elif c["op"] == "lora":
        M, K, N, R, n = c["M"], c["K"], c["N"], c["R"], c["n"]
        s["X"] = normal(M, K)
        s["W"] = normal(N, K, std=K ** -0.5)
        s["bias"] = normal(N, std=0.1) if c["bias"] else None
        s["A"], s["B"] = normal(n, R, K, std=K ** -0.5), normal(n, N, R, std=R ** -0.5)
        s["scale"] = torch.rand(n, generator=g, device="cuda") * 1.5 + 0.5
        # requests of `run` tokens each; one in ten has no adapter
        req = (M + c["run"] - 1) // c["run"]
        i = torch.randint(0, n, (req,), generator=g, device="cuda")
        i = torch.where(torch.rand(req, generator=g, device="cuda") < 0.1, -1, i)
        s["index"] = i.repeat_interleave(c["run"])[:M].to(torch.int32)
        if own:
            import fp32_emulated_gemm_split_gb300 as emu
            s["w"] = emu.emu_lora_pack(s["W"], s["bias"])
    else:
        T, Hq, Hk, D, rot = c["T"], c["Hq"], c["Hk"], c["D"], c["rot"]
        t = TYPES[c["type"]]
        # queries, keys and values as one projection writes them
        qkv = (normal(T, (Hq + 2 * Hk) * D) * (0.5 + torch.rand(T, 1, generator=g, device="cuda"))).to(t)
        s["q"] = qkv[:, : Hq * D].view(T, Hq, D)
        s["k"] = qkv[:, Hq * D: (Hq + Hk) * D].view(T, Hk, D)
        s["wq"], s["wk"] = 1 + normal(D, std=0.2), 1 + normal(D, std=0.2)
        most = 32768
        at = torch.arange(most, device="cuda", dtype=torch.float64)[:, None]
        f = 10000.0 ** (-torch.arange(rot // 2, device="cuda", dtype=torch.float64) * 2 / rot)
        s["cos"], s["sin"] = (at * f).cos().float(), (at * f).sin().float()
        start = torch.randint(0, most - T, (1,), generator=g, device="cuda")
        s["positions"] = (start + torch.arange(T, device="cuda")).to(torch.int32)
        if T < 64:                                   # next tokens of as many sequences
            s["positions"] = torch.randint(0, most, (T,), generator=g, device="cuda", dtype=torch.int32)
        if c["train"]:
            s["dq"], s["dk"] = normal(T, Hq, D).to(t), normal(T, Hk, D).to(t)
    return s


# ------------------------------------------------------------ plain forms --

def _act(g, act):
    """act(g) and its derivative."""
    if act == "silu":
        e = 1 / (1 + torch.exp(-g))
        return g * e, e * (1 + g * (1 - e))
    if act == "sigmoid":
        e = 1 / (1 + torch.exp(-g))
        return e, e * (1 - e)
    if act == "relu":
        on = (g > 0).to(g.dtype)
        return g * on, on
    if act == "gelu":
        p = 0.5 * (1 + torch.erf(g * math.sqrt(0.5)))
        return g * p, p + g * torch.exp(-0.5 * g * g) * (1 / math.sqrt(2 * math.pi))
    c = math.sqrt(2 / math.pi)
    t = torch.tanh(c * (g + 0.044715 * g * g * g))
    return 0.5 * g * (1 + t), 0.5 * (1 + t) + 0.5 * g * (1 - t * t) * c * (1 + 3 * 0.044715 * g * g)


def _gated(s):
    c, X, Wg, Wu = s["case"], s["X"], s["Wg"], s["Wu"]
    G, U = X @ Wg.t(), X @ Wu.t()
    a, d = _act(G, c["act"])
    H = a * U
    if not c["train"]:
        return H
    dU = s["dH"] * a
    dG = s["dH"] * U * d
    return H, dG @ Wg + dU @ Wu, dG.t() @ X, dU.t() @ X


def _lora(s):
    c, X = s["case"], s["X"]
    n, R, M = c["n"], c["R"], c["M"]
    # every adapter on every token, then each token's own
    mine = (s["index"][:, None] == torch.arange(n, device=X.device)).float() * s["scale"]
    S = (X @ s["A"].reshape(n * R, -1).t()).view(M, n, R) * mine[:, :, None]
    Y = X @ s["W"].t() + S.view(M, n * R) @ s["B"].permute(0, 2, 1).reshape(n * R, -1)
    return Y if s["bias"] is None else Y + s["bias"]


def _turn(a, b, cos, sin):
    return a * cos - b * sin, a * sin + b * cos


def _pairs(x, rot, pairs):
    return (x[..., 0:rot:2], x[..., 1:rot:2]) if pairs else (x[..., : rot // 2], x[..., rot // 2: rot])


def _joined(a, b, rest, pairs):
    y = torch.stack((a, b), -1).flatten(-2) if pairs else torch.cat((a, b), -1)
    return torch.cat((y, rest), -1)


def _head(x, w, cos, sin, rot, pairs):
    v = x.float()
    v = v * torch.rsqrt((v * v).mean(-1, keepdim=True) + EPS) * w
    a, b = _turn(*_pairs(v, rot, pairs), cos, sin)
    return _joined(a, b, v[..., rot:], pairs).to(x.dtype)


def _head_grad(dy, x, w, cos, sin, rot, pairs):
    d, v = dy.float(), x.float()
    a, b = _turn(*_pairs(d, rot, pairs), cos, -sin)
    dn = _joined(a, b, d[..., rot:], pairs)
    r = torch.rsqrt((v * v).mean(-1, keepdim=True) + EPS)
    dw = (dn * v * r).sum((0, 1))
    dv = dn * w
    dx = r * (dv - v * (r * r * (dv * v).mean(-1, keepdim=True)))
    return dx.to(x.dtype), dw


def _qknorm(s):
    c = s["case"]
    at = s["positions"].long()
    cos, sin = s["cos"][at][:, None, :], s["sin"][at][:, None, :]
    far = (cos, sin, c["rot"], c["pairs"])
    q, k = _head(s["q"], s["wq"], *far), _head(s["k"], s["wk"], *far)
    if not c["train"]:
        return q, k
    return (q, k, *_head_grad(s["dq"], s["q"], s["wq"], *far), *_head_grad(s["dk"], s["k"], s["wk"], *far))


# -------------------------------------------------------------- one pass --

def run(state):
    s, c = state, state["case"]
    if not own:
        return {"gated": _gated, "lora": _lora, "qknorm": _qknorm}[c["op"]](s)
    import fp32_emulated_gemm_split_gb300 as emu
    if c["op"] == "gated":
        if not c["train"]:
            return emu.emu_gated(s["X"], s["w"], act=c["act"])
        w = emu.emu_gated_pack(s["Wg"], s["Wu"])     # the weights changed with the last step
        H, G, U = emu.emu_gated(s["X"], w, act=c["act"], save=True)
        return (H, *emu.emu_gated_bwd(s["dH"], s["X"], w, G, U, act=c["act"]))
    if c["op"] == "lora":
        return emu.emu_lora(s["X"], s["w"], s["A"], s["B"], s["index"], s["scale"])
    far = dict(eps=EPS, interleaved=c["pairs"])
    at = (s["wq"], s["wk"], s["cos"], s["sin"], s["positions"])
    q, k = emu.emu_qk_norm_rope(s["q"], s["k"], *at, **far)
    if not c["train"]:
        return q, k
    dq, dk, dwq, dwk = emu.emu_qk_norm_rope_bwd(s["dq"], s["dk"], s["q"], s["k"], *at, **far)
    return q, k, dq, dwq, dk, dwk


def work(case):
    """Each input read once, each output written once; FP32 multiplications
    and additions of the products (nine times as many on the BF16 tensor cores)."""
    c = case
    if c["op"] == "gated":
        M, K, F = c["M"], c["K"], c["F"]
        values, flops = M * K + 2 * F * K + M * F, 4 * M * K * F
        if c["train"]:
            values, flops = values + M * F + M * K + 2 * F * K, 3 * flops
        return {"bytes": 4 * values, "flops": flops}
    if c["op"] == "lora":
        M, K, N, R = c["M"], c["K"], c["N"], c["R"]
        used = min(c["n"], -(-M // c["run"]))        # adapters that a request asks for, at most
        return {"bytes": 4 * (M * K + N * K + M * N + used * R * (K + N) + M),
                "flops": 2 * M * N * K + 2 * M * R * (K + N)}
    size = 4 if c["type"] == "f32" else 2
    n = c["T"] * (c["Hq"] + c["Hk"]) * c["D"]
    table = 4 * c["T"] * (c["rot"] + 1)
    # a training step reads q, k and the gradients, and writes the outputs and the gradients
    return {"bytes": (4 if c["train"] else 2) * n * size + table, "flops": (20 if c["train"] else 7) * n}


# --------------------------------------------------------- in 64 bits --

def _exact_gated(s, c):
    X, Wg, Wu = s["X"].double(), s["Wg"].double(), s["Wu"].double()
    leaf = torch.einsum("mk,fk->mf", X, Wg).requires_grad_(c["train"])
    U = torch.einsum("mk,fk->mf", X, Wu)
    f = torch.nn.functional
    a = {"silu": f.silu, "gelu": f.gelu, "relu": f.relu, "sigmoid": torch.sigmoid,
         "gelu_tanh": lambda g: f.gelu(g, approximate="tanh")}[c["act"]](leaf)
    H = (a * U).detach()
    if not c["train"]:
        return H
    dH = s["dH"].double()
    dG, = torch.autograd.grad(a, leaf, dH * U)
    a = a.detach()
    dU = dH * a
    dX = torch.einsum("mf,fk->mk", dG, Wg) + torch.einsum("mf,fk->mk", dU, Wu)
    return H, dX, torch.einsum("mf,mk->fk", dG, X), torch.einsum("mf,mk->fk", dU, X)


def _exact_lora(s, c):
    X = s["X"].double()
    Y = torch.einsum("mk,nk->mn", X, s["W"].double())
    if s["bias"] is not None:
        Y += s["bias"].double()
    for i in range(c["n"]):
        rows = (s["index"] == i).nonzero()[:, 0]
        if rows.numel():
            down = torch.einsum("mk,rk->mr", X[rows], s["A"][i].double())
            Y[rows] += s["scale"][i].double() * torch.einsum("mr,nr->mn", down, s["B"][i].double())
    return Y


def _exact_qknorm(s, c):
    rot, half = c["rot"], c["rot"] // 2
    # the rotation as complex products of the pairs
    at = s["positions"].long()
    z = torch.complex(s["cos"].double()[at], s["sin"].double()[at])[:, None, :]
    order = torch.arange(c["D"], device=z.device)
    if c["pairs"]:                                   # to the (j, j + rot/2) order and back
        order[:rot] = torch.cat((order[0:rot:2], order[1:rot:2]))
    back = order.argsort()

    def forward(x, w):
        v = (x / (x.square().sum(-1, keepdim=True) / c["D"] + EPS).sqrt() * w)[..., order]
        y = torch.complex(v[..., :half], v[..., half:rot]) * z
        return torch.cat((y.real, y.imag, v[..., rot:]), -1)[..., back]

    outs, grads = [], []
    for x, w, d in ((s["q"], s["wq"], s.get("dq")), (s["k"], s["wk"], s.get("dk"))):
        x, w = x.double().requires_grad_(c["train"]), w.double().requires_grad_(c["train"])
        y = forward(x, w)
        outs.append(y.detach())
        if c["train"]:
            grads += torch.autograd.grad(y, (x, w), d.double())
    return (*outs, *grads)


def exact(case, seed):
    s = prepare(case, seed)
    # about 1 TFLOP/s in 64 bits
    if work(case)["flops"] > 8e12:
        return None
    return {"gated": _exact_gated, "lora": _exact_lora, "qknorm": _exact_qknorm}[case["op"]](s, case)
