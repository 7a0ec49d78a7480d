"""GPU: the norm rounds y once.  Every element equals the float64 product rounded to bf16
(nearest, ties to even), zeros with their sign, and the codes those of that y.

The kernel's product is float64, 3 roundings of 2^-53 and a's few: it differs from the
reference's only for a product within 2^-49 of halfway between two bf16, a chance of
2^-40 an element."""
import pytest
import torch

from test_norm_gpu import DEV, randn, same_code
from weight_shared_rank_amd import binding

pytestmark = pytest.mark.gpu


def to_bf16_once(x):
    _, e = torch.frexp(x)
    step = torch.exp2((e.double() - 8).clamp_min(-133))
    y = torch.where(x == 0, x, torch.round(x / step) * step)
    return torch.copysign(y, x).to(torch.bfloat16)


# a shape of each row layout, enough elements that a second rounding shows (some 2^-17 of them)
@pytest.mark.parametrize("T,K", [(9000, 256), (4000, 1000), (2000, 2048), (500, 4096), (500, 8192), (900, 4096), (900, 5376), (600, 8192),
                                 (300, 12000), (150, 24000), (120, 32768)])
@pytest.mark.parametrize("f32,offset", [(False, 1.0), (True, 1.0), (True, 0.0)])
def test_y_is_rounded_once(gpu_lib, T, K, f32, offset):
    x, r = randn(1, T, K, std=3.0), randn(2, T, K)
    w = randn(3, K, std=0.5, dtype=torch.float32 if f32 else torch.bfloat16)
    w[5] = -offset                        # a weight of zero: y is a zero with h's sign
    o = binding.norm_act(x, w, residual=r, offset=offset, want=("y", "h", "code"))
    h = o.h.double()
    a = (h.square().mean(1, keepdim=True) + float(torch.tensor(1e-6, dtype=torch.float32))) ** -0.5
    want = to_bf16_once(h * a * (offset + w.double()))
    off = int((o.y.view(torch.int16) != want.view(torch.int16)).sum())
    assert off == 0, off
    same_code(o.code, binding.encode_act(want))
