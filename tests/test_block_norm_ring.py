"""The norms around a block where there are many rows (GPU): the kernel whose rows
come through a ring, by warps and by blocks, on its rare paths, against the plain
64-bit definition."""
import pytest
import torch

import layer_oracle as ref
from bit_weight_delta_bd_gb300 import bitdelta as bd
from test_block_norm import definition, dev, gen, within  # noqa: F401  (dev is a fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,d", [(300, 1000), (700, 256), (700, 504), (700, 1000), (400, 5120), (400, 8192), (400, 16384)])
@pytest.mark.parametrize("small,gain_size,eps", [
    (2.0 ** -60, 2.0 ** -62, 2.0 ** -70),   # |h gain| near 2^-122: 448 over it is past fp32's range
    (2.0 ** -62, 2.0 ** -60, 0.0),          # the same without eps: the factor is near 2^62
    (2.0 ** -60, 2.0 ** -62, 2.0 ** -40),   # |y| near 2^-102: it counts as 1e-30
    (2.0 ** -60, 2.0 ** -60, 2.0 ** -47),   # near 2^-96, next to that border
    (1.0, 1.0, 1e-5)])
def test_e4m3_of_tiny_rows(dev, T, d, small, gain_size, eps):  # noqa: F811
    """Codes and scale are the definition's wherever |h gain| is a normal number (elements below 2^-126 may be off by
    2^-149, the step of numbers there)."""
    g = gen(9)
    r = (small * torch.randn(T, d, generator=g)).to(torch.bfloat16)
    gain = (gain_size * (1 + 0.2 * torch.randn(d, generator=g))).to(torch.bfloat16)
    x = torch.zeros_like(r)
    out, sc = torch.empty(T, d, device=dev, dtype=torch.float8_e4m3fn), torch.empty(T, device=dev)
    ws = bd.new_workspace(256, dev)
    bd.bd_block_norm(x.to(dev), r.to(dev), gain.to(dev), eps, out, ws, scale=sc)
    assert bd.bd_check_async(ws) == bd.BD_OK
    h, y, size = definition(x, r, None, None, gain.expand(T, d), 1.0, 1.0, eps)
    amax = y.abs().amax(1)
    s = amax.clamp_min(1e-30) / 448
    rel = ref.norm_rel(d) + 8 * ref.U32
    mult = (h.pow(2).mean(1, keepdim=True) + eps).rsqrt()  # of h gain, whose last bit may be 2^-149
    within(sc, s, s * rel + mult[:, 0] * 2.0 ** -149 / 448, "scale")
    z = (y / s[:, None]).abs()
    half_step = torch.where(z >= 2.0 ** -6, torch.pow(2.0, torch.floor(torch.log2((z * 1.001).clamp_min(2.0 ** -6))) - 4),
                            torch.full_like(z, 2.0 ** -10))
    step = mult * 2.0 ** -149
    within(out.float().cpu().double(), y / s[:, None],
           half_step * (1 + 2.0 ** -10) + z * 3 * rel + (1 + z / 448) * step / s[:, None], "codes")
