"""Plain 64-bit forms of the feed-forward operators and elementwise error
bounds derived from them (no code of the package).

Bounds, with u = eps / 2 of the 16-bit type (half a step relative to the
value) and `tiny` half its smallest subnormal:
  sums     binary32 accumulation of n exact products p_i in any order:
           |error| <= (n + 8) 2^-23 sum |p_i| (one unit in the last place an
           addition, whatever the matrix core's rounding)
  act      silu: 2^-22 (1 + |x|) |silu(x)|; gelu: 2.5e-7 |x| + 2.4e-7 |gelu(x)|
           (the device functions' stated errors); the derivatives' terms
           s (1 + x (1 - s)) and cdf + x pdf are off by at most
           2^-19 (1 + |x|) absolutely
  output   u |y| + tiny
Errors of factors are propagated by their products; |act'| <= 1.13.
"""
import math

import torch

TORCH = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}


def half_step(dt):
    return torch.finfo(dt).eps / 2


def tiny(dt):
    f = torch.finfo(dt)
    return f.tiny * f.eps / 2


def kept(W, N, M):
    """Mask of the N largest magnitudes per group of M, ties to the lower position."""
    a = W.double().abs().unflatten(1, (-1, M))
    order = a.sort(dim=2, descending=True, stable=True).indices
    keep = torch.zeros(a.shape, dtype=torch.bool, device=W.device)
    keep.scatter_(2, order[..., :N], True)
    return keep.flatten(1)


def act64(x, act):
    cdf = torch.sigmoid(x) if act == "silu" else 0.5 * torch.erfc(-x / math.sqrt(2.0))
    return x * cdf


def slope64(x, act):
    if act == "silu":
        s = torch.sigmoid(x)
        return s * (1 + x * (1 - s))
    return 0.5 * torch.erfc(-x / math.sqrt(2.0)) + x * torch.exp(-x * x / 2) / math.sqrt(2 * math.pi)


def act_err(x, act):
    y = act64(x, act).abs()
    return 2.0 ** -22 * (1 + x.abs()) * y if act == "silu" else 2.5e-7 * x.abs() + 2.4e-7 * y


def sum_err(n, s):
    return (n + 8) * 2.0 ** -23 * s


def glu64(X, Wg, Wu, act):
    """(H, G, U, bounds of each before output rounding) in 64 bits."""
    x, wg, wu = X.double(), Wg.double(), Wu.double()
    g, u = x @ wg.t(), x @ wu.t()
    eg = sum_err(x.shape[1], x.abs() @ wg.abs().t())
    eu = sum_err(x.shape[1], x.abs() @ wu.abs().t())
    a = act64(g, act)
    ea = 1.13 * eg + act_err(g, act) + 2.0 ** -22 * (1 + eg) * (a.abs() + eg)
    h = a * u
    eh = ea * (u.abs() + eu) + a.abs() * eu + 2.0 ** -23 * h.abs()
    return h, g, u, eh, eg, eu


def glu_grad64(X, Wg, Wu, kg, ku, pre, dH, act):
    """Gradients from the products in `pre`, and their bounds before output
    rounding: (dX, dWg, dWu), (their bounds)."""
    dt = X.dtype
    x, wg, wu, dh = X.double(), Wg.double(), Wu.double(), dH.double()
    g, u = pre[0].double(), pre[1].double()
    a, sl = act64(g, act), slope64(g, act)
    dg, du = dh * u * sl, dh * a
    es = 2.0 ** -19 * (1 + g.abs())
    eg = (dh * u).abs() * es + 2.0 ** -22 * dg.abs()
    eu = dh.abs() * act_err(g, act) + 2.0 ** -22 * du.abs()
    h = half_step(dt)
    eg = eg + h * (dg.abs() + eg) + tiny(dt)          # dG, dU as 16-bit operands
    eu = eu + h * (du.abs() + eu) + tiny(dt)
    T, R = g.shape
    dx = dg @ wg + du @ wu
    ex = eg @ wg.abs() + eu @ wu.abs() + sum_err(2 * R, (dg.abs() + eg) @ wg.abs() + (du.abs() + eu) @ wu.abs())
    dwg, dwu = (dg.t() @ x) * kg, (du.t() @ x) * ku
    xa = x.abs()
    ewg = eg.t() @ xa + sum_err(T, (dg.abs() + eg).t() @ xa)
    ewu = eu.t() @ xa + sum_err(T, (du.abs() + eu).t() @ xa)
    return (dx, dwg, dwu), (ex, ewg, ewu)


def check(got, want, bound, what):
    """|got - want| <= bound + output rounding of got's type, elementwise."""
    dt = got.dtype
    g = got.double()
    lim = bound + half_step(dt) * (want.abs() + bound) + tiny(dt)
    bad = ~((g - want).abs() <= lim)
    n = int(bad.sum())
    if n:
        i = tuple(int(v) for v in bad.nonzero()[0])
        raise AssertionError(f"{what}: {n} of {bad.numel()} elements off, first at {i}: got {float(g[i])}, "
                             f"want {float(want[i])} +- {float(lim[i])}")


# ---------------------------------------------------------------- microscaled 4-bit format
GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def mx_exponent(top):
    """Scale exponent of a block's largest magnitude (float64, finite)."""
    m, e = torch.frexp(torch.where(top > 0, top, torch.ones_like(top)))
    return torch.where(top > 0, (e - 3).clamp(-127, 127), torch.full_like(e, -127))


def mx64(x):
    """(values, codes, scale bytes) of x [rows, K], from the definition: the
    nearest grid magnitude, on a tie the even code; codes [rows, K], scale
    bytes [rows, ceil(K / 32)] (255 where the block is not finite)."""
    rows, K = x.shape
    nb = -(-K // 32)
    v = torch.zeros(rows, nb * 32, dtype=torch.float64, device=x.device)
    v[:, :K] = x.double()
    v = v.view(rows, nb, 32)
    bad = ~torch.isfinite(v).all(dim=2)
    f = torch.where(bad[..., None], torch.zeros_like(v), v)
    e = mx_exponent(f.abs().amax(dim=2))
    m = torch.ldexp(f.abs(), -e[..., None])
    grid = torch.tensor(GRID, dtype=torch.float64, device=x.device)
    d = (m[..., None] - grid).abs()
    # nearest; of two equally near the even index
    d = d + torch.where(torch.arange(8, device=x.device) % 2 == 1, 1e-12, 0.0)
    code = d.argmin(dim=3)
    val = torch.ldexp(grid[code], e[..., None])
    neg = torch.signbit(f)
    val = torch.where(neg, -val, val)
    code = code + 8 * neg
    byte = torch.where(bad, torch.full_like(e, 255), e + 127)
    val = torch.where(bad[..., None], torch.full_like(val, float("nan")), val)
    return val.reshape(rows, -1)[:, :K], code.reshape(rows, -1)[:, :K], byte


def mx_read(m):
    """An independent reader of the documented layout: (codes, scale bytes)
    of an Mx's two buffers, laid out as mx64's."""
    Kp = -(-m.K // 256) * 256
    c = m.codes.cpu().reshape(m.rows, Kp // 2).to(torch.int64)
    codes = torch.stack((c & 15, c >> 4), dim=2).reshape(m.rows, Kp)
    s = m.scales.cpu().to(torch.int64)
    r = torch.arange(m.rows)[:, None]
    k = torch.arange(0, Kp, 32)[None, :]
    b = (k % 256) // 32
    at = ((r // 32) * (Kp // 256) + k // 256) * 256 + 4 * (16 * (b % 4) + r % 16) + 2 * ((r % 32) // 16) + b // 4
    return codes, s[at]
