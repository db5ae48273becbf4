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


@pytest.mark.parametrize("big", [(1 << 32) + 2, -(1 << 32) + 2, 1 << 31])
def test_counts_past_32_bits_are_refused(big):
    """Counts travel to the library in 32 bits: none is taken modulo 2^32."""
    x, ids = torch.zeros(0, 4), torch.zeros(0, 2, dtype=torch.int32)
    for call in (lambda: te.tbe_expert_rows(4, big, 8, 1), lambda: te.tbe_expert_rows(4, 2, big, 1),
                 lambda: te.tbe_expert_rows(4, 2, 8, big),
                 lambda: te.tbe_expert_sort_workspace_size(4, big, 8, 1),
                 lambda: te.tbe_expert_sort_workspace_size(4, 2, big, 1),
                 lambda: te.tbe_expert_sort_workspace_size(4, 2, 8, big),
                 lambda: te.ExpertRows(ids, big), lambda: te.ExpertRows(ids, 4, align=big),
                 lambda: te.tbe_route(x, big, None, 0, ids, torch.zeros(0, 2)),
                 lambda: te.route(x, big)):
        with pytest.raises(ValueError, match="32 bits"):
            call()
    if big > 0:  # experts that a row is wide: a view of one element
        wide = torch.empty(1).expand(0, big)
        some = torch.zeros(0, 2)
        for call in (lambda: te.route(wide, 2), lambda: te.route_backward(wide, ids, some),
                     lambda: te.tbe_route(wide, 2, None, 0, ids, some),
                     lambda: te.tbe_route_backward(wide, ids, some, 0, wide)):
            with pytest.raises(ValueError, match="32 bits"):
                call()
        slots, row = torch.empty(1, dtype=torch.int32).expand(0, big), torch.zeros(0, 8)
        source, f8 = torch.zeros(0, dtype=torch.int32), _f8(4, 128, 0, 0)
        many = torch.empty(1, dtype=torch.int32).expand(big + 1)
        each = _f8(4, 128, 0, 0)
        each.values = each.values.as_subclass(torch.Tensor)[None].expand(big, 4, 128)
        for call in (lambda: te.tbe_expert_dispatch(row, slots, source, row),
                     lambda: te.tbe_expert_dispatch_f8(row, slots, source, row, row),
                     lambda: te.tbe_expert_combine(row, slots, None, row),
                     lambda: te.tbe_expert_combine_backward(row, row, slots, source, row, row, row),
                     lambda: te.tbe_matmul_f8(f8, each, many, row),
                     lambda: te.tbe_matmul_f8_segments(f8, f8, many, row.bfloat16())):
            with pytest.raises(ValueError, match="32 bits"):
                call()


def test_clip_limits_are_those_of_the_header():
    import ctypes as C
    n, size = (1 << 20) + 1, C.c_size_t()
    f = te.lib().tbe_clip_workspace_size
    assert f(n, (C.c_int64 * n)(), C.byref(size)) == te.TBE_E_UNSUPPORTED
    assert f(n - 1, (C.c_int64 * n)(), C.byref(size)) == te.TBE_OK
    assert f(1, (C.c_int64 * 1)((1 << 36) + 1), C.byref(size)) == te.TBE_E_RANGE
    assert f(1, (C.c_int64 * 1)(1 << 36), C.byref(size)) == te.TBE_OK
