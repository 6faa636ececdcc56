"""Plain MXFP4 reference for the tests: numpy, 64 bits, a block at a time,
written from the format's definition and sharing nothing with the library.

  scale exponent e = clamp(floor(log2 A) - 2, -127, 127) of a block's largest
  magnitude A (0 for none: code 0), code byte e + 127, 255 where the block has
  an infinity or a NaN; element = the E2M1 value nearest to v / 2^e, ties to
  the even code, at most 6.
"""
import numpy as np
import torch

GRID = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def up(n, m):
    return -(-n // m) * m


def scale_codes(amax):
    """E8M0 codes of largest magnitudes (float64)."""
    m, e = np.frexp(np.where(np.isfinite(amax), amax, 1.0))   # amax = m 2^e, m in [0.5, 1)
    code = np.clip(e - 1 - 2 + 127, 0, 254)
    code = np.where(amax == 0, 0, code)
    return np.where(np.isfinite(amax), code, 255).astype(np.uint8)


def nearest_code(a):
    """E2M1 magnitude codes of non-negative values, by distance."""
    best = np.zeros(a.shape, np.uint8)
    far = np.abs(a - GRID[0])
    for c in range(1, 8):
        d = np.abs(a - GRID[c])
        take = (d < far) | ((d == far) & (c % 2 == 0))
        best = np.where(take, np.uint8(c), best)
        far = np.where(take, d, far)
    return best


def quantize(x):
    """x float64 [R, K] -> (codes uint8 [R, Kp], scale codes uint8 [R, Kp/32])
    with Kp = K rounded up to 128."""
    x = np.asarray(x, np.float64)
    R, K = x.shape
    v = np.zeros((R, up(K, 128)))
    v[:, :K] = x
    b = v.reshape(R, -1, 32)
    bad = ~np.isfinite(b).all(-1)
    amax = np.where(bad, np.inf, np.max(np.abs(np.where(np.isfinite(b), b, 0.0)), axis=-1, initial=0.0))
    s = scale_codes(amax)
    scale = np.exp2(np.where(s == 255, 127, s).astype(np.float64) - 127)
    with np.errstate(invalid="ignore"):
        c = nearest_code(np.where(bad[..., None], 0.0, np.abs(b)) / scale[..., None])
    c = c | (np.signbit(b).astype(np.uint8) << 3)
    c = np.where(bad[..., None], 0, c).astype(np.uint8)
    return c.reshape(R, -1), s


def values(codes, s):
    """float64 values of codes [R, Kp] and scale codes [R, Kp/32]."""
    g = GRID[codes & 7] * np.where(codes & 8, -1.0, 1.0)
    scale = np.where(s == 255, np.nan, np.exp2(s.astype(np.float64) - 127))
    return (g.reshape(*s.shape, 32) * scale[..., None]).reshape(codes.shape)


def fake(x):
    """The values that x's codes along its last dimension stand for."""
    x = np.asarray(x, np.float64)
    return values(*quantize(x))[:, :x.shape[1]]


def pack_codes(codes):
    return (codes[:, 0::2] | (codes[:, 1::2] << 4)).astype(np.uint8)


def pack_scales(s):
    """[R, Kp/32] -> [cdiv(R, 128), Kp/128, 128, 4], zeros past R, element by element."""
    R, nb = s.shape
    out = np.zeros((up(R, 128) // 128, nb // 4, 128, 4), np.uint8)
    r, b = np.meshgrid(np.arange(R), np.arange(nb), indexing="ij")
    out[r // 128, b // 4, r % 128, b % 4] = s
    return out


def operand(x):
    """(q, sf) device tensors of x's rows."""
    c, s = quantize(x)
    return torch.from_numpy(pack_codes(c)).cuda(), torch.from_numpy(pack_scales(s)).cuda()


def host64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


# half a unit in the last place of an output type, relative
UNIT = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}


def check_product(got, a, b, factor=None):
    """got (device) against a b^T in 64 bits.  Every product of two codes and
    their scales is exact in fp32 (4 significant bits and a power of two), and
    adding K of them in any order in fp32 is off by at most K 2^-24 of the sum
    of magnitudes, to first order; the factor adds a rounding and the output
    type half a unit (fp16's below 2^-14: half its least subnormal)."""
    K = a.shape[1]
    want, mag = a @ b.T, np.abs(a) @ np.abs(b).T
    if factor is not None:
        want, mag = want * factor[:, None], mag * np.abs(factor)[:, None]
    unit = UNIT[got.dtype]
    tol = (K + 2) * 2.0 ** -24 * 1.01 * mag + unit * np.abs(want) * 1.01
    tol += 2.0 ** -25 if got.dtype == torch.float16 else 2.0 ** -133
    assert got.shape == want.shape
    got64 = host64(got)
    if got.dtype == torch.float16:
        # a sum from 65520 on rounds to fp16's infinity: it has to where it is
        # past that for certain, and may where it is within the tolerance
        inf = np.isinf(got64) & (np.abs(want) + tol >= 65520) & (np.sign(got64) == np.sign(want))
        assert (inf | (np.abs(want) - tol < 65520)).all()
        got64 = np.where(inf, want, got64)
    # NaN where, and only where, a block of either operand stands for NaN
    nan = np.isnan(want)
    assert np.array_equal(nan, np.isnan(got64))
    got64, want, tol = (np.where(nan, 0.0, v) for v in (got64, want, tol))
    err = np.abs(got64 - want)
    worst = np.unravel_index(np.argmax(err - tol), err.shape) if err.size else None
    assert err.size == 0 or (err <= tol).all(), (worst, err[worst], tol[worst], want[worst])
