"""Plain 64-bit norm and rotation of heads, for the tests (torch on the CPU; no
code of the library), with bounds that count the kernels' roundings."""
import torch


def split(x, r, pairs):
    if pairs:
        return x[..., 0:r:2], x[..., 1:r:2], x[..., r:]
    return x[..., :r // 2], x[..., r // 2:r], x[..., r:]


def join(a, b, rest, pairs):
    ab = torch.stack([a, b], -1).flatten(-2) if pairs else torch.cat([a, b], -1)
    return torch.cat([ab, rest], -1)


def angles(table, pos):
    """Cosines and sines [.., N, r / 2] of positions, taken as within the table."""
    rows = table.double()[pos.long().clamp(0, table.shape[0] - 1)]
    return rows.chunk(2, -1)


def turn(x, cs, pairs, back=False, size=False):
    """R(p) x, or R(p)^T x; size: the sum of the magnitudes that each element is formed of."""
    c, s = cs
    a, b, rest = split(x, 2 * c.shape[-1], pairs)
    if size:
        a, b, rest, c, s = (t.abs() for t in (a, b, rest, c, s))
        return join(a * c + b * s, b * c + a * s, rest, pairs)
    if back:
        s = -s
    return join(a * c - b * s, b * c + a * s, rest, pairs)


def forward(x, w, cs, eps, pairs):
    """x [B, H, N, d] float64, w [d] float64, cs broadcast against [B, 1, N, r / 2]."""
    n = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    return turn(n * w, cs, pairs)


def forward_tolerance(x, w, cs, eps, pairs, half):
    """Bound on the kernel's error. In fp32 (u = 2^-24): the squares' sum is off by
    (d + 1) u of itself, its root's reciprocal by half of that and 3 u, two products
    and the rotation's three operations by u each, of the magnitudes that a result
    is formed of; then one rounding, `half` a step (fp16: 2^-25 below its normal range)."""
    d = x.shape[-1]
    n = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    size = turn(n * w, cs, pairs, size=True)
    err = size * (d / 2 + 12) * 2.0 ** -24
    y = forward(x, w, cs, eps, pairs)
    return err + (y.abs() + err) * half + (2.0 ** -25 if half == 2.0 ** -11 else 1e-37)


def backward(x, dy, w, cs, eps, pairs):
    """(dx, dw) by the formula."""
    inv = 1 / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    t, n = turn(dy, cs, pairs, back=True), x * inv
    dx = inv * (t * w - n * (t * w * n).mean(-1, keepdim=True))
    return dx, (t * n).sum((0, 1, 2))


def backward_tolerance(x, dy, w, cs, eps, pairs, half):
    """Bounds on dx and dw: 1 / rms as in the forward, (d / 2 + 4) u; t 3 u of its
    magnitudes; the mean's sum d u; products u each. dw's sum: u for each of its terms."""
    d = x.shape[-1]
    inv = 1 / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    n, size = (x * inv).abs(), turn(dy, cs, pairs, size=True)
    u = 2.0 ** -24
    err = inv * (size * w.abs() * (d / 2 + 12)
                 + n * (size * w.abs() * n).mean(-1, keepdim=True) * (2.5 * d + 24)) * u
    dx, _ = backward(x, dy, w, cs, eps, pairs)
    tol_x = err + (dx.abs() + err) * half + (2.0 ** -25 if half == 2.0 ** -11 else 1e-37)
    rows = x.numel() // d
    return tol_x, (size * n).sum((0, 1, 2)) * (d / 2 + 12 + rows) * u + 1e-37
