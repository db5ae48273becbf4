"""Host side of the expert-layer calls, corners: what the package needs of torch when it is
imported, and what its calls refuse."""
import os
import subprocess
import sys

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
