"""The quantiser bit for bit in the format and group pairs that test_q4.py's
own parametrisation leaves out."""
import pytest

import test_q4
from test_q4 import dev, m  # noqa: F401

torch = pytest.importorskip("torch")


@pytest.mark.gpu
@pytest.mark.parametrize("fmt,group", [("int4", 64), ("e2m1", 32), ("e2m1", 128)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("H,Im", [(128, 128), (384, 256), (2176, 128)])
def test_quantize_formats(m, dev, H, Im, dtype, fmt, group):  # noqa: F811
    test_q4.test_quantize(m, dev, H, Im, dtype, fmt, group)
