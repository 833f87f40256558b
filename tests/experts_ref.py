"""The experts' operators in 64 bits, for the tests: E4M3 codes and scales are decoded
by a table, everything else follows the formulas of include/moe_route.h."""
import torch

BLK = 128
EPS = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}   # half a step, relative


def e4m3_table():
    code = torch.arange(256)
    e, m = (code >> 3) & 15, (code & 7).double()
    v = torch.where(e == 0, m * 2.0 ** -9, (8 + m) * torch.pow(2.0, e.double() - 10))
    v = torch.where(code >= 128, -v, v)
    v[(code & 127) == 127] = float("nan")
    return v


def two_to(n):
    """2^n in 64 bits, exactly."""
    return ((n.long() + 1023) << 52).view(torch.float64)


def scale_values(s):
    """float32 scales, or UE8M0 bytes (255 is a NaN), in 64 bits."""
    if s.dtype == torch.uint8:
        return torch.where(s == 255, float("nan"), two_to(s.long() - 127))
    return s.double()


def decode(codes, scale, rows):
    """[..., r, c] codes with a scale for each rows x 128 block."""
    v = e4m3_table().to(codes.device)[codes.long()]
    s = scale_values(scale)
    i = torch.arange(v.shape[-2], device=v.device) // rows
    j = torch.arange(v.shape[-1], device=v.device) // BLK
    return v * s[..., i, :][..., j]


def pow2ceil(t):
    m, e = torch.frexp(t)
    return two_to(e - (m == 0.5).to(e.dtype))


def block_scale(amax):
    """The scale of a block with this largest magnitude; the rule is one of 32-bit arithmetic."""
    t = amax.clamp_min(1e-4).float() * torch.tensor(1.0, dtype=torch.float32).div(448.0).to(amax.device)
    return pow2ceil(t.double())


def round_e4m3(v):
    """To the nearest E4M3 value (ties to even) within 448, and the step there."""
    e = torch.floor(torch.log2(v.abs().clamp_min(2.0 ** -30))).clamp(-6, 8)
    step = two_to(e.nan_to_num(0) - 3)
    return (torch.round(v / step) * step).clamp(-448, 448), step


def quant_rows(x):
    """-> (value after rounding, scale per element, step per element)"""
    b = x.unflatten(-1, (-1, BLK))
    s = block_scale(b.abs().amax(-1))[..., None]
    q, step = round_e4m3(b / s)
    return (q * s).flatten(-2), s.expand_as(b).flatten(-2), (step * s).flatten(-2)


def encode_rows(x, fmt):
    """float rows -> codes uint8, scales; the codes by torch's own cast of exactly scaled values."""
    b = x.double().unflatten(-1, (-1, BLK))
    s = block_scale(b.abs().amax(-1))
    q = (b / s[..., None]).float().to(torch.float8_e4m3fn).view(torch.uint8).flatten(-2)
    return q.contiguous(), encode_scale(s, fmt)


def encode_scale(s, fmt):
    if fmt == "fp32":
        return s.float()
    return (torch.frexp(s)[1] - 1 + 127).to(torch.uint8)


def encode_weight(W, fmt):
    E, n, k = W.shape
    nb, kb = -(-n // BLK), -(-k // BLK)
    pad = torch.nn.functional.pad(W.double().abs(), (0, kb * BLK - k, 0, nb * BLK - n))
    s = block_scale(pad.view(E, nb, BLK, kb, BLK).amax((2, 4)))
    per = s.repeat_interleave(BLK, 1)[:, :n].repeat_interleave(BLK, 2)[:, :, :k]
    q = (W.double() / per).float().to(torch.float8_e4m3fn).view(torch.uint8)
    return q.contiguous(), encode_scale(s, fmt)


def offsets_of(counts, device):
    off = torch.zeros(len(counts) + 1, dtype=torch.int64)
    off[1:] = torch.tensor(counts).cumsum(0)
    return off.to(torch.int32).to(device)


def swiglu(gu):
    g, u = gu.chunk(2, -1)
    return g / (1 + torch.exp(-g)) * u


def swiglu_grad(da, gu):
    g, u = gu.chunk(2, -1)
    s = 1 / (1 + torch.exp(-g))
    return torch.cat([da * u * s * (1 + g * (1 - s)), da * g * s], -1)
