"""Plain 64-bit forms of the 8-bit rows and of the products of rows grouped by
expert, and elementwise error bounds derived from them (no code of the
package).

Bounds, in the notation of _ffn.py: 16-bit sums (n + 8) 2^-23 sum |p_i| before
the output's rounding.  8-bit sums are exact; conversion, the two scales and
the bias are four binary32 roundings of at most 2^-24 each, (1 + 2^-24)^3 - 1
< 3.01 2^-24 for the first three; numbers below binary32's normal range are off
by half its smallest, 2^-150, a step.
"""
import torch

from tests._ffn import act64, act_err, kept, sum_err


def i8_64(x):
    """(elements, scales) of x's rows from the definition, int64 and float32:
    the scale amax times binary32's 1 / 127, rounded to binary32, at least 2^-126;
    the nearest whole number of the exact quotient, the even one on a tie; rows
    that are not finite: NaN and zeros."""
    x = x.double()
    fin = torch.isfinite(x).all(dim=1)
    f = torch.where(fin[:, None], x, torch.zeros_like(x))
    # (a product of two binary32 numbers is exact in binary64)
    s = (f.abs().amax(dim=1) * float.fromhex("0x1.020408p-7")).float().clamp(min=2.0 ** -126)
    u = f / s.double()[:, None]
    # a binary32 value over another is no closer than 2^-25 to a half without
    # being one, far beyond binary64's error of the quotient
    low = torch.floor(u)
    up = (u - low > 0.5) | ((u - low == 0.5) & (low.remainder(2) == 1))
    q = (low + up).clamp(-127, 127).to(torch.int64)
    return q, torch.where(fin, s, torch.full_like(s, float("nan")))


def experts_of(offsets, T):
    """[(first, end)] of each expert, and the rows of none, as the calls read
    offsets: into [0, T], each at least the one before it."""
    at = []
    for o in offsets.tolist():
        at.append(max(at[-1] if at else 0, min(max(o, 0), T)))
    return list(zip(at, at[1:])), [r for r in range(T) if r < at[0] or r >= at[-1]]


def i8_product64(q, sx, w, sw, bias, act):
    """(Y, bound before output rounding) of one weight: q [T, K], w [R, K] whole
    numbers, sx [T], sw [R] float32."""
    y = (q.double() @ w.double().t()) * sx.double()[:, None] * sw.double()[None, :]
    e = 3.01 * 2.0 ** -24 * y.abs() + 2.0 ** -149
    if bias is not None:
        y = y + bias.double()
        e = e + 2.0 ** -24 * (y.abs() + e)
    if act == "gelu":
        a = act64(y, act)
        # the activation's error at the computed argument, itself off by e
        return a, 1.13 * e + act_err(y.abs() + e, act) + 2.0 ** -22 * a.abs()
    return y, e


def expert64(X, W, offsets):
    """(Y, bound) of expert_linear on pruned dense weights W [E, R, K]; rows of
    no expert are zeros."""
    T, R = X.shape[0], W.shape[1]
    Y = torch.zeros(T, R, dtype=torch.float64, device=X.device)
    B = torch.zeros_like(Y)
    for e, (a, b) in enumerate(experts_of(offsets, T)[0]):
        x, w = X[a:b].double(), W[e].double()
        Y[a:b] = x @ w.t()
        B[a:b] = sum_err(X.shape[1], x.abs() @ w.abs().t())
    return Y, B


def expert_grad64(X, W, keep, dY, offsets):
    """((dX, dW), (their bounds))."""
    T, K = X.shape
    E, R = W.shape[:2]
    dX = torch.zeros(T, K, dtype=torch.float64, device=X.device)
    dW = torch.zeros(E, R, K, dtype=torch.float64, device=X.device)
    bX, bW = torch.zeros_like(dX), torch.zeros_like(dW)
    for e, (a, b) in enumerate(experts_of(offsets, T)[0]):
        x, w, g = X[a:b].double(), W[e].double(), dY[a:b].double()
        dX[a:b] = g @ w
        bX[a:b] = sum_err(R, g.abs() @ w.abs())
        dW[e] = (g.t() @ x) * keep[e]
        bW[e] = sum_err(b - a, g.abs().t() @ x.abs()) * keep[e]
    return (dX, dW), (bX, bW)


def i8_expert64(q, sx, w, sw, bias, act, offsets):
    """(Y, bound) of i8_expert_linear: w [E, R, K] whole numbers, sw, bias [E, R]."""
    T, R = q.shape[0], w.shape[1]
    Y = torch.zeros(T, R, dtype=torch.float64, device=q.device)
    B = torch.zeros_like(Y)
    for e, (a, b) in enumerate(experts_of(offsets, T)[0]):
        if b > a:
            Y[a:b], B[a:b] = i8_product64(q[a:b], sx[a:b], w[e], sw[e], None if bias is None else bias[e], act)
    return Y, B


def pruned(W, N, M):
    """(W with zeros where pruned, mask) for [..., R, K] weights."""
    k = kept(W.reshape(-1, W.shape[-1]), N, M).reshape(W.shape)
    return torch.where(k, W, torch.zeros_like(W)), k
