"""The check of single elements that the GPU tests of orthogonalising use, on the CPU: it lets
the simulated roundings pass and sees one wrong element."""
import pytest
import torch

from test_gpu_ortho import FAST, check_elements, simulate


@pytest.mark.parametrize("plant", ["nothing", "zero", "sign", "corner"])
@pytest.mark.parametrize("rows,cols", [(130, 200), (200, 130)])
def test_one_wrong_element_is_seen(rows, cols, plant):
    torch.manual_seed(0)
    G = torch.randn(rows, cols)
    got = simulate(G, 5, FAST).bfloat16()
    rms = float(got.double().square().mean().sqrt())
    i, j = (got[100:, 100:].abs() > 0.5 * rms).nonzero()[0].tolist()
    if plant == "zero":
        got[100 + i, 100 + j] = 0
    elif plant == "sign":
        got[100 + i, 100 + j] *= -1
    elif plant == "corner":
        got[-4:, -4:] = got[:4, :4].clone()
    if plant == "nothing":
        check_elements(got, G, 5, FAST)
    else:
        with pytest.raises(AssertionError):
            check_elements(got, G, 5, FAST)
