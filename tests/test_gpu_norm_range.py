"""The norms and their gradients of rows far from the usual sizes: the squares of a row's values, and
their sum, are in fp32's range, and so is every result, whatever the powers of rms(out) between."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import block_refs as refs  # noqa: E402
import operator_refs  # noqa: E402
import lora_moe_expert_gb300 as mlg  # noqa: E402
from test_gpu_block_norm import _backward, _case, _forward, _np  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    mlg.lib()
    yield
    torch.cuda.synchronize()


@pytest.mark.parametrize("gate", ["row", "full"])
@pytest.mark.parametrize("n,width,dtype", [(5, 264, "bf16"), (9, 2048, "bf16"), (4, 4104, "bf16"),
                                           (7, 1036, "f32"), (40, 64, "f32")])
@pytest.mark.parametrize("size", [1e-16, 1e-13, 1e-6, 1e10, 1e14, 1e15, 1e16, 1e17])
@pytest.mark.parametrize("eps", [0.0, 1e-6])
def test_rows_of_any_size(size, eps, n, width, dtype, gate):
    """x and y of the size; gradients of out of its inverse, so that both of d's terms count."""
    if eps > 0 and size < 1e-3:
        size = size ** 0.25  # (rows below sqrt(eps) do not come near the range's ends)
    rs, bs, bf16 = 0.75, 0.5, dtype == "bf16"
    c = _case(n, width, dtype, gate, True, True, n + width)
    c["x"], c["y"] = c["x"] * size, c["y"] * size
    c["dout"] = c["dout"] / size
    out, z = _forward(c, rs, bs, eps)
    h = {k: _np(v) for k, v in c.items()}
    eps = float(np.float32(eps))
    ref, err = refs.norm_out(h["x"], h["y"], h["gate"], h["post"], rs, bs, eps)
    operator_refs.assert_within(_np(out), ref, err, bf16, "out")
    ref, err = refs.norm_z(_np(out), h["pre"], eps)
    operator_refs.assert_within(_np(z), ref, err, bf16, "z")
    got = _backward(c, out, rs, bs, eps)
    want = refs.norm_grad(h["dout"], h["dz"], _np(out), h["y"], h["gate"], h["post"], h["pre"], rs,
                          bs, eps)
    assert set(got) == set(want)
    for k, (ref, err) in want.items():
        operator_refs.assert_within(_np(got[k]), ref, err, bf16 and k in ("dx", "dy", "dgate"), k)
