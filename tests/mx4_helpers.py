"""The microscaled 4-bit formats in 64 bits, for the tests: written from the
formulas in include/egopq.h, with torch's elementary operations."""
import torch

BLOCK = {0: 32, 1: 16}
GRID = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64)
# half way between neighbours, and whether that goes up (to the even code)
MIDS = ((0.25, False), (0.75, True), (1.25, False), (1.75, True), (2.5, False), (3.5, True),
        (5.0, False))
HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
# the smallest step of a type near zero, halved
TINY = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25, torch.float32: 2.0 ** -150}


def power(e):
    """2^e in 64 bits, exactly (torch.pow is off by a last place on a GPU)."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def e4m3_table():
    """The 127 numbers e4m3 bytes 0..126 stand for."""
    b = torch.arange(127)
    e, m = b >> 3, (b & 7).double()
    return torch.where(e == 0, m * 2.0 ** -9, (1 + m / 8) * power(e - 7))


def magnitude(v):
    m = torch.zeros_like(v, dtype=torch.uint8)
    for mid, up in MIDS:
        m += ((v >= mid) if up else (v > mid)).to(torch.uint8)
    return m


def gated64(x, K):
    g, u = x[:, :K].double(), x[:, K:].double()
    return g / (1.0 + torch.exp(-g)) * u


def values_in(x, K, fmt, g, gated):
    """u of the formulas: in fp32's numbers unless gated."""
    r = None if g is None else torch.reciprocal(g.float()).double()
    u = gated64(x, K) if gated else x.double()
    if r is not None:
        u = u * r
    return u if gated or r is None else u.float().double()


def quant(u, fmt):
    """codes uint8 [M, K/2], scales uint8 [M, K/block] of u [M, K] (64 bits)."""
    M, K = u.shape
    b = u.reshape(M, -1, BLOCK[fmt])
    top = b.abs().amax(dim=2)  # (a NaN is the largest)
    bad = ~(top < 2.0 ** 128 * (1 - 2.0 ** -25))
    if fmt == 0:
        e = torch.frexp(torch.where(bad, 1.0, top))[1].long() - 3
        e = torch.where(top == 0, -127, e).clamp(min=-127)
        scale, byte = power(e), e + 127
        byte = torch.where(bad, 255, byte)
    else:
        table = e4m3_table().to(u.device)
        want = torch.where(bad, 0.0, top / torch.full_like(top, 6.0))
        hi = torch.searchsorted(table, want.contiguous()).clamp(max=126)
        lo = (hi - 1).clamp(min=0)
        dl, dh = want - table[lo], table[hi] - want
        byte = torch.where((dh < dl) | ((dh == dl) & (hi % 2 == 0)), hi, lo)
        byte = torch.where(want >= 448.0, 126, byte)
        scale, byte = table[byte], torch.where(bad, 127, byte)
    q = torch.where(scale[..., None] > 0, b.abs() / torch.where(scale == 0, 1.0, scale)[..., None],
                    torch.zeros_like(b))
    code = torch.where(bad[..., None], 0, magnitude(q) + 8 * torch.signbit(b).to(torch.uint8))
    code = code.to(torch.uint8).reshape(M, K)
    return code[:, 0::2] | (code[:, 1::2] << 4), byte.to(torch.uint8)


def dequant(codes, scales, fmt):
    """64-bit values [..., K] (without a tensor's scale)."""
    code = torch.stack((codes & 15, codes >> 4), dim=-1).flatten(-2).long()
    v = GRID.to(codes.device)[code & 7]
    v = torch.where(code >= 8, -v, v)
    if fmt == 0:
        s = torch.where(scales == 255, float("nan"), power(scales.long() - 127))
    else:
        t = torch.cat((e4m3_table(), torch.tensor([float("nan")], dtype=torch.float64)))
        s = t.to(codes.device)[scales.long() & 127]
    return (v.unflatten(-1, (-1, BLOCK[fmt])) * s[..., None]).flatten(-2)


def same_codes(got, want):
    """Equal but for the sign of zeros."""
    for shift in (0, 4):
        a, b = (got >> shift) & 15, (want >> shift) & 15
        if not torch.equal(torch.where(a == 8, 0, a), torch.where(b == 8, 0, b)):
            return False
    return True


def tolerance(y64, size, K, dtype):
    """What a product may be off: its rounding to dtype, the tensors' scales (two
    products of fp32, two half steps each at most), and the sums. `size` is
    sum |a w| (times the scales). An instruction adds 64 products to the sum: those
    are cut off at 2^-23 of the largest of them, 64 times at most, and the sum of
    each of the K / 64 instructions is off by 2^-23 of what it holds."""
    sums = (64 + (K + 63) // 64) * 2.0 ** -23 * size
    off = sums + 4 * 2.0 ** -24 * y64.abs()
    return off + HALF_STEP[dtype] * (y64.abs() + off) + TINY[dtype]
