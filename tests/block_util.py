"""Plain 64-bit forms of the block-scaled 8-bit operators, and their inputs."""
import torch

from mlx_grouped_affine_gb300 import qmm

TYPES = {"f32": (torch.float32, qmm.QMM_F32), "bf16": (torch.bfloat16, qmm.QMM_BF16),
         "f16": (torch.float16, qmm.QMM_F16)}


def blocks(n):
    return -(-n // 128)


def values(codes):
    return codes.view(torch.float8_e4m3fn).double()


def spread(scales, block_rows, rows, cols):
    """Scales in 64 bits at every element."""
    return scales.double().repeat_interleave(block_rows, 0)[:rows].repeat_interleave(128, 1)[:, :cols]


def grid():
    """The 127 values of e4m3 from 0 to 448."""
    return values(torch.arange(127, dtype=torch.uint8))


def quantized(x, block_rows):
    """(values of the codes in 64 bits, fp32 scales) of a CPU tensor: the definition, each
    quotient compared with the borders between codes (a 64-bit quotient of numbers of 24
    bits is on a border of 5 bits only where the exact one is)."""
    rows, cols = x.shape
    d = x.double()
    pad = torch.zeros(-(-rows // block_rows) * block_rows, blocks(cols) * 128, dtype=torch.float64)
    pad[:rows, :cols] = d
    top = pad.abs().reshape(-1, block_rows, blocks(cols), 128).amax((1, 3))
    scales = (top / torch.full_like(top, 448.0)).float()
    scales = torch.where(scales < 2.0 ** -126, torch.full_like(scales, 2.0 ** -126), scales)
    q = d / spread(scales, block_rows, rows, cols)
    g = grid()
    border = (g[1:] + g[:-1]) / 2
    at = torch.searchsorted(border, q.abs())
    on = border[at.clamp(max=125)] == q.abs()
    at = torch.where(on & (at % 2 == 1), at + 1, at).clamp(max=126)
    got = torch.copysign(g[at], q)
    return torch.where(q.isnan(), q, got), scales


def operands(m, n, k, seed, spread_bits=0.5):
    g = torch.Generator().manual_seed(seed)
    code = lambda r: (torch.randn(r, k, generator=g) * 100).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    scale = lambda r: torch.exp(torch.randn(r, blocks(k), generator=g) * spread_bits) / 100
    return code(m), scale(m), code(n), scale(blocks(n))


def product(a, a_scales, w, w_scales):
    """(A . W^T, the sum of the magnitudes of its terms) in 64 bits."""
    x = values(a) * spread(a_scales, 1, *a.shape)
    v = values(w) * spread(w_scales, 128, *w.shape)
    return x @ v.T, x.abs() @ v.abs().T


def bound(size, k, dtype):
    """Of |y|, the sum of magnitudes: k additions and 4 roundings of scales and blocks in
    fp32 (a tensor core may cut instead of rounding: 2^-23 each), and y's own rounding."""
    y, terms = size
    return terms * (k + 4) * 2.0 ** -23 + y.abs() * torch.finfo(dtype).eps / 2 + 2.0 ** -140
