"""Plain 64-bit forms of the 4-bit expert operators, from the format's definition (include/moe.h, moe_w4_t)."""
import torch

NIBBLE = [0, 4, 1, 5, 2, 6, 3, 7]  # nibble of a word that holds column j


def pack(codes):
    """[..., k] codes -> [..., k / 2] bytes, one word of eight columns at a time."""
    c = codes.reshape(*codes.shape[:-1], -1, 8).long()
    word = sum(c[..., j] << (4 * NIBBLE[j]) for j in range(8))
    return torch.stack([(word >> (8 * i)) & 255 for i in range(4)], -1).to(torch.uint8).reshape(*codes.shape[:-1], -1)


def unpack(q):
    b = q.reshape(*q.shape[:-1], -1, 4).long()
    word = sum(b[..., i] << (8 * i) for i in range(4))
    return torch.stack([(word >> (4 * NIBBLE[j])) & 15 for j in range(8)], -1).reshape(*q.shape[:-1], -1)


def dequant(q, s, z, group, rounded=True):
    """fp64 [E][n][k]; rounded: to bf16, as the products take the weights."""
    codes = unpack(q).double()
    k = codes.shape[-1]
    at = torch.arange(k) // group
    zz = z.double() if z is not None else torch.full(s.shape, 8.0, dtype=torch.float64)
    w = (codes - zz.transpose(1, 2)[..., at]) * s.double().transpose(1, 2)[..., at]
    return w.float().to(torch.bfloat16).double() if rounded else w


def quantize(x, group, zero):
    """codes, scales (fp64), zero points of x [E][n][k], by the definition: scales by search, quotients in fractions of 64 bits."""
    E, n, k = x.shape
    G = -(-k // group)
    codes = torch.empty((E, n, k), dtype=torch.int64)
    s = torch.empty((E, G, n), dtype=torch.float64)
    z = torch.full((E, G, n), 8, dtype=torch.int64)
    bits, steps = (4, 15.0) if zero else (5, 7.0)
    for g in range(G):
        v = x[..., g * group:(g + 1) * group].double()
        lo, hi = v.amin(-1).clamp(max=0), v.amax(-1).clamp(min=0)
        rng = hi - lo if zero else v.abs().amax(-1)
        # the least m 2^e (2^(bits-1) <= m < 2^bits) with steps * m 2^e >= rng: products are exact here
        e = torch.floor(torch.log2(torch.where(rng > 0, rng, torch.ones_like(rng)) / steps)) - bits
        best = torch.full_like(rng, float("inf"))
        for de in range(-1, 4):
            unit = torch.exp2(e + de)
            for m in range(2 ** (bits - 1), 2 ** bits):
                c = m * unit
                best = torch.where((steps * c >= rng) & (c < best), c, best)
        best = torch.where(rng > 0, best.clamp(min=2.0 ** -100), torch.ones_like(best))
        s[:, g] = best
        zp = (-lo / best).round().clamp(0, 15) if zero else torch.full_like(best, 8.0)
        z[:, g] = zp.long()
        codes[..., g * group:(g + 1) * group] = ((v / best[..., None]).round() + zp[..., None]).clamp(0, 15).long()
    return codes, s, z


def silu(g):
    return g / (1 + torch.exp(-g))


def acc_bound(x, w, k):
    """How far a sum of k products x w^T may be off: K / 16 MMA steps and 16 products inside each, every addition
    off by at most one fp32 step (2^-23) of the magnitudes summed so far."""
    return (k / 16 + 16) * 2.0 ** -23 * (x.abs() @ w.abs().T)


def row_bound(x, w, group, bits):
    """The share of rows that enter the products rounded to 2^-bits of the largest value of their group."""
    k = x.shape[1]
    G = -(-k // group)
    padded = torch.zeros((x.shape[0], G * group), dtype=x.dtype)
    padded[:, :k] = x.abs()
    top = padded.reshape(-1, G, group).amax(-1)
    return 2.0 ** -bits * (top.repeat_interleave(group, 1)[:, :k] @ w.abs().T)


def product_bound(x, w, group, bits=15):
    return acc_bound(x, w, x.shape[1]) + row_bound(x, w, group, bits)


def gate_up(x, wg, wu, group, bits=15):
    """fp64 h and its bound before h is rounded: silu' is below 1.1, |silu(a) - silu(b)| <= 1.1 |a - b|."""
    g, u = x @ wg.T, x @ wu.T
    dg, du = product_bound(x, wg, group, bits), product_bound(x, wu, group, bits)
    h = silu(g) * u
    return h, 1.1 * dg * u.abs() + silu(g).abs() * du + 1.1 * dg * du + 2.0 ** -20 * h.abs()


def readings(*weights):
    """The matrices' fp64 weights in the two readings that a call may take: exact, and rounded to bf16."""
    for rounded in (False, True):
        yield [dequant(*w, rounded=rounded) for w in weights]


def within(got, want, tol, half):
    """got is want up to tol before it was rounded by at most half of its value."""
    return bool(((got - want).abs() <= tol + half * (want.abs() + tol) + 1e-30).all())
