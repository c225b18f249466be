"""Host-side checks of the 8-bit binding at empty axes: no GPU needed."""
import torch

from evoformer_pair_bias_b200 import fp8


def test_rows_counts_the_rows_of_an_empty_last_axis():
    for shape, rows in (((2, 3, 0), 6), ((5, 0), 5), ((0,), 1), ((2, 0, 0), 0), ((4, 0, 7), 0), ((0, 7), 0)):
        r, c, v, ld = fp8._rows(torch.zeros(shape))
        assert (r, c, tuple(v.shape)) == (rows, shape[-1], (rows, shape[-1])), shape
