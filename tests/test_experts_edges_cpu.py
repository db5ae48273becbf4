"""Host side of the expert-layer calls, corners: what the package needs of torch when it is
imported, and what its calls refuse."""
import os
import subprocess
import sys

import pytest
import torch

import table_embedding_amd as te

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_import_needs_no_gpu_functions_of_torch():
    """A torch built without them imports the package and uses the host-side checks."""
    code = ("import torch\n"
            "for n in ('_cuda_getDevice', '_cuda_getCurrentRawStream'):\n"
            "    if hasattr(torch._C, n): delattr(torch._C, n)\n"
            "import table_embedding_amd as te\n"
            "assert te.tbe_expert_rows(4, 2, 8, 16) == 128\n"
            "try:\n"
            "    te.quantize_f8(torch.zeros(4, 4))\n"
            "except ValueError as e:\n"
            "    assert 'device tensors' in str(e)\n"
            "else:\n"
            "    raise SystemExit('a host tensor was taken')\n")
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0, r.stderr


class _On(torch.Tensor):
    """A host tensor that says it is on a given device (its memory is never read)."""

    @staticmethod
    def on(t, device):
        t = torch.Tensor._make_subclass(_On, t)
        t.says = device
        return t

    is_cuda = property(lambda self: True)

    def get_device(self):
        return self.says


def _f8(rows, cols, values_on, scales_on, square=False):
    vs, ss = te.F8Matrix.shapes(rows, cols, square)
    m = te.F8Matrix.__new__(te.F8Matrix)
    m.values = _On.on(torch.zeros(vs, dtype=torch.float8_e4m3fn), values_on)
    m.scales = _On.on(torch.zeros(ss, dtype=torch.uint8), scales_on)
    m.rows, m.cols, m.square = rows, cols, square
    return m


def test_8_bit_matrix_has_values_and_scales_on_one_device():
    vs, ss = te.F8Matrix.shapes(4, 128)
    values = _On.on(torch.zeros(vs, dtype=torch.float8_e4m3fn), 0)
    te.F8Matrix(values, _On.on(torch.zeros(ss, dtype=torch.uint8), 0), 4, 128)
    with pytest.raises(ValueError, match="one device"):
        te.F8Matrix(values, _On.on(torch.zeros(ss, dtype=torch.uint8), 1), 4, 128)


@pytest.mark.parametrize("which", [0, 1])
def test_products_look_at_the_devices_of_scales(which):
    """Scales of another device than everything else are refused before the launch."""
    a, b = _f8(4, 128, 0, which ^ 1), _f8(8, 128, 0, which)
    offsets = _On.on(torch.tensor([0, 4], dtype=torch.int32), 0)
    with pytest.raises(ValueError, match="one device"):
        te.tbe_matmul_f8(a, b, offsets, _On.on(torch.zeros(4, 8, dtype=torch.bfloat16), 0))
    with pytest.raises(ValueError, match="one device"):
        te.tbe_matmul_f8_segments(a, b, offsets,
                                  _On.on(torch.zeros(1, 4, 8, dtype=torch.bfloat16), 0))
