"""Operands in 8 bits with one FP32 scale per 128, in float64: the rules of the section on products in
include/moe.h, written out with torch on whatever device the tensors are on."""
import torch

F64 = torch.float64


def pow2(e):
    """2^e in float64, exactly (torch.ldexp goes by way of pow, which is not)."""
    return (e.long() + 1023 << 52).view(F64)


def e4m3(q):
    """The nearest E4M3 values to q (float64), ties to even; exact."""
    _, e = torch.frexp(q)
    step = pow2((e - 1).clamp(min=-6) - 3)
    return ((q / step).round() * step).clamp(-448, 448)


def scale(top):
    """max(top / 448, 2^-100), the quotient rounded once to 32 bits; NaN for infinities and NaN."""
    s = (top.to(F64) / 448).float().to(F64).clamp(min=2.0 ** -100)
    return torch.where(torch.isfinite(top.to(F64)), s, torch.full_like(s, float("nan")))


def rows(v):
    """v [R, K] as (values on the E4M3 grid, scales [R, K/128]), float64."""
    b = v.to(F64).unflatten(-1, (-1, 128))
    s = scale(b.abs().amax(-1, keepdim=True))
    return e4m3(b / s).flatten(-2), s.squeeze(-1)


def rows_value(v):
    q, s = rows(v)
    return q * s.repeat_interleave(128, -1)


def squares(w):
    """w [E, N, K] as (values on the grid, scales [E, N/128, K/128])."""
    E, N, K = w.shape
    b = w.to(F64).view(E, N // 128, 128, K // 128, 128)
    s = scale(b.abs().amax((2, 4), keepdim=True))
    return e4m3(b / s).view(E, N, K), s[:, :, 0, :, 0]


def matrix(codes, s):
    """The float64 values of codes (uint8) [E, N, K] with scales [E, N/128, K/128]."""
    v = codes.view(torch.float8_e4m3fn).to(F64)
    return v * s.to(F64).repeat_interleave(128, 1).repeat_interleave(128, 2)


def mx_columns(v):
    """v [rows, N] in MXFP8 along its rows, as float64 values."""
    n = v.shape[0]
    b = torch.nn.functional.pad(v.to(F64), (0, 0, 0, -n % 32)).unflatten(0, (-1, 32))
    top = b.abs().amax(1, keepdim=True)
    m, e = torch.frexp(top)
    s = torch.where(top > 0, e - 9 + (m > 0.875).int(), -127).clamp(-127, 127)
    return (e4m3(b * pow2(-s)) * pow2(s)).flatten(0, 1)[:n]


def act(kind, g):
    if kind == 1:
        return 0.5 * g * (1 + torch.erf(g * 0.5 ** 0.5))
    return g.clamp(min=0) if kind == 2 else g * torch.sigmoid(g)


def layer(x, ids, scores, w13, w2, kind=0):
    """The expert layer in float64: x BF16 [T, d], ids [T, k], w13 and w2 float64 values; a quantized along I."""
    T, k = ids.shape
    I = w2.shape[2]
    xv = rows_value(x)
    y = torch.zeros(T, w2.shape[1], dtype=F64, device=x.device)
    for e in ids.unique().tolist():
        t, j = (ids == e).nonzero(as_tuple=True)
        gu = xv[t] @ w13[e].T
        a = rows_value(act(kind, gu[:, :I]) * gu[:, I:])
        y.index_add_(0, t, a @ w2[e].T * scores[t, j].to(F64)[:, None])
    return y
