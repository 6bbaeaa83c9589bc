"""Plain references, in 64 bits and without the library, of the operators around a layer's products:
head norms with the position rotation and their gradient."""
import torch


def rope_table(rows, rotary, base=10000.0):
    i = torch.arange(rotary // 2, dtype=torch.float64)
    a = torch.arange(rows, dtype=torch.float64)[:, None] / base ** (2 * i / rotary)
    return torch.cat([a.cos(), a.sin()], 1).float()


def _angles(positions, table, T, D):
    """cos, sin [T, 1, pairs] in FP64 and which tokens have a position ([T, 1, 1])."""
    p = torch.arange(T) if positions is None else positions.long()
    there = p >= 0
    n = 0 if table is None else table.shape[1] // 2
    if n == 0:
        z = torch.zeros(T, 1, 0, dtype=torch.float64)
        return z, z, there[:, None, None]
    there = there & (p < table.shape[0])
    row = table.double()[p.clamp(0, table.shape[0] - 1)][:, None]
    return row[..., :n], row[..., n:], there[:, None, None]


def _pairs(D, n, interleaved):
    i = torch.arange(n)
    return (2 * i, 2 * i + 1) if interleaved else (i, i + n)


def turn(y, cos, sin, interleaved):
    a, b = _pairs(y.shape[-1], cos.shape[-1], interleaved)
    z = y.clone()
    z[..., a] = y[..., a] * cos - y[..., b] * sin
    z[..., b] = y[..., b] * cos + y[..., a] * sin
    return z


def turn_bound(y, cos, sin, interleaved):
    """|a cos| + |b sin| and the like: what the rounding of the turned values goes by."""
    return turn(y.abs(), cos.abs(), -sin.abs(), interleaved).abs().maximum(
        turn(y.abs(), cos.abs(), sin.abs(), interleaved).abs())


def qk(x, w, eps, positions, table, interleaved):
    """(z, bound): the heads after, and the sums of magnitudes behind each value."""
    x = x.double()
    T, H, D = x.shape
    w = torch.ones(D, dtype=torch.float64) if w is None else w.double()
    cos, sin, there = _angles(positions, table, T, D)
    y = x / (x.square().mean(-1, keepdim=True) + eps).sqrt() * w
    zero = torch.zeros((), dtype=torch.float64)
    return (torch.where(there, turn(y, cos, sin, interleaved), zero),
            torch.where(there, turn_bound(y, cos, sin, interleaved), zero))


def qk_backward(d, x, w, eps, positions, table, interleaved):
    """(dx, dw, terms): terms are the magnitudes behind the two parts of dx and behind dw."""
    x, d = x.double(), d.double()
    T, H, D = x.shape
    w = torch.ones(D, dtype=torch.float64) if w is None else w.double()
    cos, sin, there = _angles(positions, table, T, D)
    zero = torch.zeros((), dtype=torch.float64)
    d = torch.where(there, d, zero)
    x = torch.where(there, x, zero)
    r = 1 / (x.square().mean(-1, keepdim=True) + eps).sqrt()
    n = r * x
    dy, size = turn(d, cos, -sin, interleaved), turn_bound(d, cos, sin, interleaved)
    dn = dy * w
    dx = r * (dn - n * (dn * n).mean(-1, keepdim=True))
    first = r * size * w.abs()
    second = r * n.abs() * (size * w.abs() * n.abs()).mean(-1, keepdim=True)
    return dx, (dy * n).sum((0, 1)), (first, second, (size * n.abs()).sum((0, 1)))


MUON = (3.4445, -4.7750, 2.0315)


def orthogonalize(g, steps=5, coefficients=MUON, eps=1e-7):
    """X after the steps, FP64, from the side with fewer rows."""
    x = g.double()
    turned = x.shape[-2] > x.shape[-1]
    x = x.mT if turned else x
    x = x / (x.square().sum((-2, -1), keepdim=True).sqrt() + eps)
    for i in range(steps):
        a, b, c = coefficients[i] if hasattr(coefficients[0], "__len__") else coefficients
        gram = x @ x.mT
        x = a * x + (b * gram + c * gram @ gram) @ x
    return x.mT if turned else x


def orthogonalize_rounded(g, steps=5, coefficients=MUON, eps=1e-7, seed=0):
    """The same with every operand of a product (values that the kernels round to FP16, 11 significant bits: X's copy,
    A and B without their diagonals) moved up or down, at random, by the most that rounding can: half a step,
    2^-11 relative."""
    gen = torch.Generator(device=g.device).manual_seed(seed)

    def off(t):
        up = torch.rand(t.shape, generator=gen, device=t.device) < 0.5
        return t * torch.where(up, 1 + 2.0 ** -11, 1 - 2.0 ** -11).to(t.dtype)

    def off_symmetric(t):
        low = off(t).tril()
        return low + low.tril(-1).mT
    x = g.double()
    x = x.mT if x.shape[-2] > x.shape[-1] else x
    x = x / (x.square().sum((-2, -1), keepdim=True).sqrt() + eps)

    def apart(t):  # the diagonal stays as it is
        d = torch.diag_embed(t.diagonal(dim1=-2, dim2=-1))
        return d, off_symmetric(t - d)
    for i in range(steps):
        a, b, c = coefficients[i] if hasattr(coefficients[0], "__len__") else coefficients
        copy = off(x)
        d, h = apart(copy @ copy.mT)
        f, e = apart(b * (d + h) + c * (d + h) @ (d + h))
        x = a * x + f @ x + e @ copy
    return x.mT if g.shape[-2] > g.shape[-1] else x
