"""The attention kernels that the library has are those that a call can reach (no GPU)."""
import re
import subprocess

from mlx_grouped_affine_gb300 import qmm


def test_each_type_and_head_size_has_one_home():
    """Heads up to 128 of 16-bit types have the tensor cores, everything else the CUDA cores."""
    names = subprocess.run(["nm", "-C", qmm.lib()._name], capture_output=True, text=True, check=True).stdout
    got = {}
    for kernel, element, size in re.findall(r"::(decode|prefill|tiles)_kernel<qmm::(?:paged::)?Elem(\w+), (\d+)>\(", names):
        got.setdefault(kernel, set()).add((element, int(size)))
    tensor = {(e, d) for e in ("BF16", "F16") for d in (64, 128)}
    assert got["decode"] == tensor and got["prefill"] == tensor
    assert got["tiles"] == {("F32", 64), ("F32", 128), ("F32", 256), ("BF16", 256), ("F16", 256)}
