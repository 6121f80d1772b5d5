"""The norm of the residual stream where a kernel takes row after row: more rows than a round of CTAs, in each of its kernels."""
import pytest

from tests.step_testutil import TYPES
from tests.test_gpu_norm import backward, forward

pytestmark = pytest.mark.gpu

# Rows of a warp with 1, 2 and 4 pieces of 8 values a lane: a round is 4,864 rows on 152 SMs (rows of 520 to 1,024 values only
# where their CTAs' last round would be far from full, or in FP32); of a CTA: 152 to 1,520; rows of any kind: 608.
WARP = [(6000, 64, dict(group=64)), (6000, 256, dict(group=0, same="x")), (6000, 512, dict(group=128, same="r")), (5000, 40, dict(residual=False)),
        (6000, 520, dict(residual=False, group=0)), (6000, 1000, dict(group=0, pad=8)), (6000, 1024, dict(group=128, plain=False)),
        (3000, 1024, dict(group=32))]
CTA = [(4000, 1096, dict(pad=8)), (2000, 2048, dict(group=32, same="x")), (1300, 4096, dict(group=0, plain=False)), (700, 8192, dict(group=64, same="r")),
       (400, 12288, dict(group=128)), (320, 16384, dict(group=0, residual=False))]
ANY = [(1500, 77, dict(group=0)), (1500, 1001, dict(same="r")), (1300, 96, dict(group=32, shift=1)), (1300, 512, dict(group=0, pad=3)),
       (700, 16416, dict(group=32, plain=False)), (700, 3, dict(residual=False))]


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("T,C,kw", WARP + CTA + ANY)
def test_forward_of_more_rows_than_a_round(T, C, kw, dtype):
    forward(T, C, dtype, seed=T + C, **kw)


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("T,C,kw", [
    (6000, 64, {}), (6000, 256, dict(same="dy")), (6000, 512, dict(same="dres")), (5000, 40, dict(along=False)), (3000, 1000, dict(pad=8)),
    (2600, 1024, dict(same="dy")), (3000, 520, dict(along=False)), (3000, 1024, dict(want_dw=False)), (6000, 520, {}), (6000, 1024, dict(same="dres")),
    (1500, 77, {}), (1500, 1001, dict(same="dy")), (1300, 96, dict(shift=1, along=False)), (700, 16400, dict(pad=3)), (700, 3, dict(same="dres"))])
def test_backward_of_more_rows_than_a_round(T, C, kw, dtype):
    backward(T, C, dtype, seed=T + C, **kw)
