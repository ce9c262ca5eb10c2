"""Plain forms of the 4-bit floating-point operators for the tests: the quantizers as they are defined, operation by operation in
fp32, products in 64 bits. CPU tensors; no code of the package."""
import torch

from .fp8_reference import EPS, cdiv, tokens  # noqa: F401

LEVELS = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0])
SCALE = {16: torch.float8_e4m3fn, 32: torch.float8_e8m0fnu}


def pitch(K, block):
    return cdiv(K, 256) * (256 // block)


def e2m1(t):
    """Codes of fp32 values: nearest level, halfway to the even code, past 6 to 6; NaN is not looked at."""
    a = t.abs()
    code = ((a > 0.25).int() + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0)).to(torch.uint8)
    return code | (torch.signbit(t).to(torch.uint8) << 3)


def quantize(x, block):
    """Codes uint8 [rows, K], block scales as bytes [rows, K / block], row scales (None for blocks of 32) of fp32 x."""
    rows, K = x.shape
    parts = x.view(rows, K // block, block)
    b = parts.abs().amax(2)                                            # propagates NaN
    if block == 16:
        a = b.amax(1)
        a = torch.where(torch.isfinite(a), a, torch.tensor(float("nan")))
        a = torch.where(a < 1e-30, torch.tensor(1e-30), a)
        s = a / torch.tensor(2688.0)
        c = (b * (torch.tensor(448.0) / a)[:, None]).to(torch.float8_e4m3fn)
        f = c.float()
        up = torch.where(f > 0, (torch.tensor(2688.0) / a)[:, None] / f, torch.tensor(0.0))
        sf = c.view(torch.uint8)
    else:
        s = None
        sf = torch.zeros(b.shape, dtype=torch.int64)
        for e in range(253, -1, -1):                                   # the smallest 2^(e - 127) with b <= 6 2^(e - 127)
            sf[b.double() <= 6.0 * 2.0 ** (e - 127)] = e
        sf[~torch.isfinite(b)] = 255
        up = (2.0 ** (127.0 - sf.double())).float()
        sf = sf.to(torch.uint8)
    codes = e2m1((parts * up[:, :, None]).view(rows, K))
    return codes, sf, s


def pack(codes):
    return codes[..., 0::2] | (codes[..., 1::2] << 4)


def unpack(q):
    return torch.stack([q & 15, q >> 4], -1).flatten(-2)


def scale_values(sf, block):
    return sf.view(SCALE[block]).double()


def pad(sf, K, block):
    """Rows of block scales with the zeros behind them."""
    return torch.cat([sf, sf.new_zeros((*sf.shape[:-1], pitch(K, block) - sf.shape[-1]))], -1)


def tile(sf, K, block):
    """Bytes [N, K / block] in the weights' order, entry by entry."""
    N, groups = sf.shape
    out = torch.zeros((cdiv(N, 128), pitch(K, block) // 4, 32, 4, 4), dtype=torch.uint8)
    n, b = torch.arange(N)[:, None], torch.arange(groups)
    out[n // 128, b // 4, n % 32, n % 128 // 32, b % 4] = sf
    return out


def values(codes, sf, s, block):
    """What codes [rows, K] stand for, in 64 bits."""
    v = LEVELS.double()[codes.long()] * scale_values(sf, block).repeat_interleave(block, -1)
    return v if s is None else v * s.double()[:, None]


def product(a, w):
    """(y, sum of the products' magnitudes) in 64 bits of values."""
    return a @ w.T, a.abs() @ w.abs().T


def product_tolerance(y, mag, K, dtype):
    """The tensor core adds the blocks' sums of 64 K (at most four of them, exact in themselves: 16 or 32 products of multiples of 1/4 up
    to 36, times a product of two scales of four bits each) to an fp32 sum. However it rounds those additions, each loses at
    most a step of the sum, 2^-23 of the magnitudes: 5 for each 64 K. Then two fp32 products, and one rounding to dtype."""
    sums = (5 * cdiv(K, 64) + 2) * 2.0 ** -23 * mag
    floor = 2.0 ** -25 if dtype == torch.float16 else 2.0 ** -149      # half a step of the subnormals
    return sums + EPS[dtype] * (y.abs() + sums) + floor


def operand(rows, K, block, seed, outliers=True, scale=1.0):
    """(values in 64 bits, q, padded rows of block scales as bytes, tiled ones, row scales) of random rows."""
    codes, sf, s = quantize(tokens(rows, K, seed, outliers) * scale, block)
    return values(codes, sf, s, block), pack(codes), pad(sf, K, block), tile(sf, K, block), s
