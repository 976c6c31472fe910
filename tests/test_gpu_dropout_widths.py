"""GPU tests of the residual add with RMSNorm and dropout at the widths between those of test_gpu_dropout.py, so that
every number of lanes that a row may take is run with a mask."""
import pytest

import test_gpu_dropout as dropout

pytestmark = pytest.mark.gpu
B = dropout.B

@pytest.mark.parametrize("rows,D", [(40, 12), (33, 200), (70, 515), (9, 1000), (3, 1029)])
@pytest.mark.parametrize("dtype,rdtype,scaled,p", [("bf16", "f32", True, 0.1), ("f16", "f16", True, 0.5),
                                                   ("f32", "f32", False, 0.3), ("bf16", "bf16", False, 0.9),
                                                   ("f16", "f32", False, 0.2), ("f32", "f32", True, 0.6)])
def test_widths(B, rows, D, dtype, rdtype, scaled, p):
    dropout.test_dropout_add_norm(B, rows, D, dtype, rdtype, scaled, p)
