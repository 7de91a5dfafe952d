"""Microscaled layers at the borders of their kernels' routes: few output columns at every number of
tokens where the route changes, long contractions, grids around one and two CTAs per SM, ranks of
the K split with unequal shares.  Same oracle and bounds as the other tests of these layers."""
import pytest

from test_mx_gpu import check_backward, check_forward, q  # noqa: F401 (q: fixture)

pytestmark = pytest.mark.gpu

ROUTES = [1, 4, 5, 8, 9, 16, 17, 64, 65, 128, 129, 384, 385, 512, 513]


@pytest.mark.parametrize("d_out", [1, 2, 3, 7])
@pytest.mark.parametrize("T", ROUTES)
def test_few_output_columns(q, T, d_out):  # noqa: F811
    check_forward(q, T, d_out, 192, 3, seed=T)
    for base, ckpt in (("mx", True), ("mx", False), ("nf4", True)):
        check_backward(q, T, d_out, 192, 3, base, ckpt, T % 2 == 0, seed=T + d_out)


# ring lengths of up to 11 stages of 256, split over 1, 2 and 4 ranks: shares from one stage to many turns of the ring
@pytest.mark.parametrize("T,d_out,d_in,r", [
    (2, 130, 28672, 4), (8, 100, 28672, 128), (16, 128, 14336, 16), (20, 130, 28672, 4), (66, 130, 14336, 9), (200, 260, 11008, 16),
    (3, 60, 2880, 4), (6, 60, 2816, 4), (11, 60, 2752, 4), (33, 60, 1088, 65), (70, 60, 832, 70), (130, 60, 576, 1),
    # one CTA per SM is 148 tiles of 128 rows
    (1, 9472, 512, 2), (3, 9480, 1088, 2), (5, 18944, 320, 2), (5, 18950, 320, 2), (5, 37900, 128, 2),
    (40, 18944, 192, 2), (40, 18950, 1088, 2), (100, 9472, 1088, 2), (100, 9480, 1088, 2), (512, 4736, 1088, 2),
    (500, 4740, 1152, 8)])
def test_forward_schedules(q, T, d_out, d_in, r):  # noqa: F811
    check_forward(q, T, d_out, d_in, r, seed=d_in + T)


@pytest.mark.parametrize("T,d_out,d_in,r", [(2, 11008, 192, 4), (20, 100, 9600, 8), (100, 5000, 448, 128), (128, 37, 2048, 127),
                                            (129, 4100, 128, 2), (700, 130, 128, 128), (1, 1, 64, 128)])
@pytest.mark.parametrize("base,ckpt", [("mx", True), ("mx", False), ("nf4", True)])
def test_backward_schedules(q, T, d_out, d_in, r, base, ckpt):  # noqa: F811
    check_backward(q, T, d_out, d_in, r, base, ckpt, False, seed=d_in + T)
