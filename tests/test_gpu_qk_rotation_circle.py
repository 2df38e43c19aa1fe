"""The rotation's cosines and sines around the whole circle."""
import pytest
import torch

from gpu_helpers import ensure_built
from resident_decoder_trainer_gb300 import rdt

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    ensure_built()


@pytest.mark.parametrize("start", [0, -(1 << 16)])
def test_every_part_of_the_circle(start):
    """65,536 positions of a radian each, 1e-4 of a radian apart on the circle: rounding the angle
    to fp32 changes it by at most 2 2^-24 pi / 4 and its unit, the polynomials are off by 2^-28.7
    and their evaluation by a few 2^-25: below 2^-22."""
    n, d = 1 << 16, 16
    q = torch.zeros(n, 1, d, device="cuda")
    q[..., :d // 2] = 1  # turned: cosines, then sines
    positions = torch.arange(start, start + n, device="cuda", dtype=torch.int32)
    out = torch.empty_like(q)
    rdt.qk_norm_rope(q, None, out, None, positions=positions, theta=1.0)
    angle = positions.double()[:, None, None]
    assert (out[..., :d // 2].double() - angle.cos()).abs().max() < 2.0 ** -22
    assert (out[..., d // 2:].double() - angle.sin()).abs().max() < 2.0 ** -22
    eighths = ((angle / (torch.pi / 4)) % 8).floor().unique()
    assert len(eighths) == 8
