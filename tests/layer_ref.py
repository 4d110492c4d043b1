"""Plain 64-bit implementations of the block operators and the error bounds
that their tests use.

Every function takes the FP32 (or 16-bit) tensors that the kernels get and
computes in float64.  The bounds count roundings: EPS = 2^-24 is half an FP32
unit in the last place, `terms` the number of FP32 operations a value went
through, and the magnitudes are sums of absolute values, so that cancellation
is allowed for.
"""
import math

import torch

EPS = 2.0 ** -24
ACT_ROUNDINGS = 16          # of an activation or its derivative: exp or erfc (a few ulp), divide, two products
# the final rounding to a 16-bit type: half of the type's spacing (finfo.eps) relative to the value
HALF_ULP = {torch.float32: 0.0, torch.bfloat16: torch.finfo(torch.bfloat16).eps / 2,
            torch.float16: torch.finfo(torch.float16).eps / 2}
LEAST = {torch.float32: 0.0, torch.bfloat16: 0.0, torch.float16: 2.0 ** -25}


def act(name, g):
    """act(g) and act'(g)."""
    if name == "silu":
        s = torch.sigmoid(g)
        return g * s, s * (1 + g * torch.sigmoid(-g))
    if name == "gelu":
        c = 0.5 * torch.erfc(-g / math.sqrt(2))
        return g * c, c + g * torch.exp(-0.5 * g * g) / math.sqrt(2 * math.pi)
    if name == "gelu_tanh":
        z = math.sqrt(2 / math.pi) * (g + 0.044715 * g ** 3)
        s = torch.sigmoid(2 * z)
        dz = math.sqrt(2 / math.pi) * (1 + 3 * 0.044715 * g * g)
        return g * s, s + g * 2 * s * torch.sigmoid(-2 * z) * dz
    if name == "relu":
        return g.clamp(min=0), (g > 0).double()
    s = torch.sigmoid(g)
    return s, s * torch.sigmoid(-g)


def gated(name, X, Wg, Wu):
    """(H, G, U) and their bounds (bH, bG, bU).  Derivatives of the
    activations are at most 1.13 in size."""
    X, Wg, Wu = X.double(), Wg.double(), Wu.double()
    K = X.size(1)
    G, U = X @ Wg.t(), X @ Wu.t()
    bG = (2 * K + 2) * EPS * (X.abs() @ Wg.abs().t())
    bU = (2 * K + 2) * EPS * (X.abs() @ Wu.abs().t())
    a, _ = act(name, G)
    H = a * U
    bH = 1.13 * bG * (U.abs() + bU) + a.abs() * bU + ACT_ROUNDINGS * EPS * (H.abs() + bG * bU) + 1e-37
    return (H, G, U), (bH, bG, bU)


def gated_bwd(name, dH, X, Wg, Wu, G, U):
    """(dX, dWg, dWu) and their bounds, from given G and U."""
    dH, X, Wg, Wu, G, U = (t.double() for t in (dH, X, Wg, Wu, G, U))
    a, d = act(name, G)
    dG, dU = dH * U * d, dH * a
    # the derivative's terms are at most 1.3 in size, the activation is accurate relative to itself
    bdG = ACT_ROUNDINGS * EPS * 1.3 * (dH * U).abs() + 1e-37
    bdU = ACT_ROUNDINGS * EPS * dU.abs() + 1e-37
    M, F = dH.shape
    dX, dWg, dWu = dG @ Wg + dU @ Wu, dG.t() @ X, dU.t() @ X
    mG, mU = dG.abs() + bdG, dU.abs() + bdU
    rows = 2 * ((F + 31) // 32 * 32)
    bX = (2 * rows + 2) * EPS * (mG @ Wg.abs() + mU @ Wu.abs()) + bdG @ Wg.abs() + bdU @ Wu.abs()
    bWg = (2 * M + 2) * EPS * (mG.t() @ X.abs()) + bdG.t() @ X.abs()
    bWu = (2 * M + 2) * EPS * (mU.t() @ X.abs()) + bdU.t() @ X.abs()
    return (dX, dWg, dWu), (bX, bWg, bWu)


def lora(X, W, bias, A, B, index, scale):
    """Y and its bound."""
    n, R, K = A.shape
    Xd, Wd = X.double(), W.double()
    Y = Xd @ Wd.t()
    bound = (2 * K + 4) * EPS * (Xd.abs() @ Wd.abs().t())
    if bias is not None:
        Y = Y + bias.double()
        bound = bound + 4 * EPS * bias.double().abs()
    for i in range(n):
        rows = (index == i).nonzero()[:, 0]
        if rows.numel() == 0:
            continue
        x, a, b = X[rows].double(), A[i].double(), B[i].double()
        s = 1.0 if scale is None else float(scale[i])
        Y[rows] += s * ((x @ a.t()) @ b.t())
        bound[rows] += (K + 2 * R + 6) * EPS * abs(s) * ((x.abs() @ a.abs().t()) @ b.abs().t())
    return Y, bound + 4 * EPS * Y.abs() + 1e-37


def _split(x, rot, interleaved):
    if interleaved:
        return x[..., 0:rot:2], x[..., 1:rot:2]
    return x[..., :rot // 2], x[..., rot // 2:rot]


def _join(a, b, rest, interleaved):
    if interleaved:
        return torch.cat((torch.stack((a, b), -1).flatten(-2), rest), -1)
    return torch.cat((a, b, rest), -1)


def turn(x, cos, sin, rot, interleaved):
    if rot == 0:
        return x
    a, b = _split(x, rot, interleaved)
    return _join(a * cos - b * sin, a * sin + b * cos, x[..., rot:], interleaved)


def qk(x, w, cos, sin, positions, eps, interleaved):
    """y and its bound for one side (tokens x heads x D)."""
    kind, D = x.dtype, x.size(-1)
    rot = 0 if cos is None else 2 * cos.size(1)
    c = s = None
    if rot:
        c, s = cos.double()[positions.long()][:, None], sin.double()[positions.long()][:, None]
    x = x.double()
    n = x / (x.square().mean(-1, keepdim=True) + eps).sqrt() * (1.0 if w is None else w.double())
    y = turn(n, c, s, rot, interleaved)
    # sum of D squares: half of D + 2 roundings survive the square root; 8 for the rest
    m = turn(n.abs(), c.abs(), -s.abs(), rot, interleaved) if rot else n.abs()
    if rot:                                        # |a c| + |b s| in both places of a pair
        a, b = _split(n.abs(), rot, interleaved)
        m = _join(a * c.abs() + b * s.abs(), a * s.abs() + b * c.abs(), n.abs()[..., rot:], interleaved)
    return y, (D / 2 + 10) * EPS * m + HALF_ULP[kind] * (1 + 1e-4) * y.abs() + LEAST[kind]


def qk_bwd(dy, x, w, cos, sin, positions, eps, interleaved):
    """(dx, dw) and their bounds for one side."""
    kind, D = x.dtype, x.size(-1)
    rot = 0 if cos is None else 2 * cos.size(1)
    x, d = x.double(), dy.double()
    w = torch.ones(D, dtype=torch.float64, device=x.device) if w is None else w.double()
    m = d.abs()
    if rot:
        c, s = cos.double()[positions.long()][:, None], sin.double()[positions.long()][:, None]
        a, b = _split(d.abs(), rot, interleaved)
        m = _join(a * c.abs() + b * s.abs(), a * s.abs() + b * c.abs(), d.abs()[..., rot:], interleaved)
        d = turn(d, c, -s, rot, interleaved)
    r = (x.square().mean(-1, keepdim=True) + eps).rsqrt()
    dn = d * w
    dx = r * (dn - x * r * r * (dn * x).mean(-1, keepdim=True))
    mx = r * (m * w.abs() + x.abs() * r * r * (m * w.abs() * x.abs()).mean(-1, keepdim=True))
    dw = (d * x * r).sum((0, 1))
    mw = (m * x.abs() * r).sum((0, 1))
    n = x.size(0) * x.size(1)
    bx = (2.5 * D + 20) * EPS * mx + HALF_ULP[kind] * (1 + 1e-4) * dx.abs() + LEAST[kind]
    return (dx, dw), (bx, (n + D / 2 + 20) * EPS * mw + 1e-37)


def ratio(got, want, bound):
    """Largest |got - want| / bound; NaNs and infinities have to agree."""
    got = got.double()
    fine = torch.isfinite(want)
    assert torch.equal(torch.isfinite(got), fine), "finite in different places"
    if not bool(fine.any()):
        return 0.0
    off = (got - want).abs()[fine]
    return float((off / bound[fine].clamp(min=1e-300)).max()) if float(off.max()) > 0 else 0.0


def rel(got, want):
    """Relative error in the 2-norm."""
    return float((got.double() - want).norm() / want.norm().clamp(min=1e-300))
