"""The mixture-of-experts example end to end (GPU), against its unquantized float32 form."""
import pytest

from examples import moe_layer
from tests._util import ensure_built

pytestmark = pytest.mark.gpu


# A bf16 layer rounds its inner values and output to 2^-9: below 2 % of its contribution beside the
# residual stream's own rounding. Rounding a value to 4 bits (3 significant bits at best, 2 at the
# least) leaves an error of about a tenth of its size on random data; four such operands (inputs
# and weights of two projections) and the gate's slope add up to less than a half.
@pytest.mark.parametrize("fmt,bound", [("bf16", 0.02), ("mxfp4", 0.5), ("nvfp4", 0.5)])
@pytest.mark.parametrize("tokens,experts,topk,hidden,inner", [(1, 8, 2, 512, 256), (37, 16, 4, 1024, 640), (600, 8, 3, 512, 512)])
def test_example(tokens, experts, topk, hidden, inner, fmt, bound):
    ensure_built()
    args = ["--tokens", tokens, "--experts", experts, "--topk", topk, "--hidden", hidden, "--inner", inner, "--format", fmt]
    assert moe_layer.main([str(v) for v in args]) < bound
