"""Plain forms of the norm and the backward pass from 8-bit checkpoints, for the tests: torch in float64, or in the fp32 steps
that the definitions name, on any device."""
import torch


def e4m3(v):
    """fp32 values to E4M3 codes, nearest even, saturating."""
    return v.clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8)


def decode(q, s):
    """fp32 values of a 1x128 checkpoint [M, K]."""
    M, K = q.shape
    return (q.view(torch.float8_e4m3fn).float().view(M, K // 128, 128) * s.t()[:, :, None]).reshape(M, K)


def power_byte(amax):
    """E8M0 byte of the least power of two p >= 2^-127 with amax <= 448 p; 0 for 0."""
    a = amax.double()
    m, e = torch.frexp(a)
    byte = (e - 9 + (m > 0.875).int() + 127).clamp(min=0)
    return torch.where(a > 0, byte, torch.zeros_like(byte)).to(torch.uint8)


def power(byte):
    """2^(byte - 127) in float64, exact (torch's ldexp of float64 on the GPU is not)."""
    return ((byte.long() - 127 + 1023) << 52).view(torch.float64)


def backward_copy(v):
    """The transposed copy of fp32 values [M, C]: codes [C, Mp], bytes [Mp/128, C].  Exact: the definition's only rounding is
    E4M3's."""
    M, C = v.shape
    nb = (M + 127) // 128
    v = torch.cat([v, torch.zeros((nb * 128 - M, C), device=v.device)]).view(nb, 128, C)
    et = power_byte(v.abs().amax(1) if nb else torch.zeros((0, C), device=v.device))
    q = e4m3((v.double() / power(et)[:, None, :]).float())
    return q.view(nb * 128, C).t().contiguous(), et


def copy_values(qt, et):
    """float64 values [C, Mp] of a transposed copy."""
    C, cols = qt.shape
    return (qt.view(torch.float8_e4m3fn).double().view(C, cols // 128, 128) * power(et).t()[:, :, None]).reshape(C, cols)


def rows_of(q, row_token, T):
    """Rows [rows, K] of a layout; a token outside [0, T) is a row of zeros."""
    t = row_token.long()
    t = torch.where((t < 0) | (t >= T), T, t)
    return torch.cat([q, torch.zeros_like(q[:1]) if T else torch.zeros((1, q.shape[1]), dtype=q.dtype, device=q.device)])[t]


def norm64(h, w, eps):
    h = h.double()
    return h * (h.pow(2).mean(1, keepdim=True) + eps).rsqrt() * w.double()


def swiglu_grad64(x, u, gh):
    x, u, gh = x.double(), u.double(), gh.double()
    p = torch.sigmoid(x)
    return gh * u * (p + x * p * (1 - p)), gh * x * p, x * p * u
