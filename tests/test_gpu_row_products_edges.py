"""Products whose weights differ by rows, at the ends of what their arguments may be."""
import numpy as np
import pytest
import torch

from host_offloaded_weight_gb300 import lstream as L
from test_gpu_grouped_mxfp4 import Case as Grouped
from test_gpu_grouped_mxfp4 import _dev

pytestmark = pytest.mark.gpu
LOW, HIGH = -2 ** 31, 2 ** 31 - 1


@pytest.mark.parametrize("epi", ["store", "swiglu", "scale"])
@pytest.mark.parametrize("M", [60, 300])          # single CTAs and pairs
@pytest.mark.parametrize("bounds", [[20, LOW, 0, 40, HIGH], [30, LOW, -7, HIGH, LOW], [LOW, 40, 41, HIGH, 45], [HIGH, 5, 50, LOW, LOW + 3],
                                    [16, LOW, LOW, LOW, LOW]], ids=lambda b: "_".join(map(str, b)))
def test_bounds_of_any_value_are_cut_to_the_rows(bounds, M, epi):
    """Row i is group g's where bounds[g] <= i < bounds[g + 1], and nothing else is written."""
    n = len(bounds) - 1
    wants = []
    for g in range(n):
        c = Grouped([0] * g + [M] + [0] * (n - 1 - g), 72, 128, epi)
        if g:
            c.codes, c.scales, c.values = first.codes, first.scales, first.values
        else:
            first = c
        want, tol = c.exact()
        wants.append((want, tol if epi == "scale" else tol + 2.0 ** -8 * (want.abs() + tol) + 1e-38))
    first.bounds = _dev(np.array(bounds, np.int32))
    first.run()
    torch.cuda.synchronize()
    assert L.lsk_device_error() == 0
    rows = torch.arange(M, device="cuda")
    place = first.table.long() if epi == "scale" else rows
    got = first.out[:M].double()
    assert bool((first.out[M] == 77.0).all())
    for g, (want, tol) in enumerate(wants):
        at = place[(rows >= bounds[g]) & (rows < bounds[g + 1])]
        assert bool(((got[at] - want[at]).abs() <= tol[at]).all()), g
    none = torch.ones(M, dtype=torch.bool, device="cuda")
    for g in range(n):
        none &= ~((rows >= bounds[g]) & (rows < bounds[g + 1]))
    assert bool((got[place[none]] == 77.0).all())
