"""A workspace is any 16-byte aligned memory of the stated size (no GPU): the part of
it that the kernels use begins where their widest store, 32 bytes, may go."""
from mlx_grouped_affine_gb300 import qmm
from paged_host import workspace_bases


def test_the_kernels_part_is_aligned_and_inside(tmp_path):
    size, at = qmm.QMM_ATTENTION_WORKSPACE_BYTES, [(1 << 40) + 16 * i for i in range(17)]
    for p, (base, room) in zip(at, workspace_bases(tmp_path, at, size)):
        assert base % 32 == 0 and base % 128 == 0
        assert p <= base < p + 128 and base + room == p + size
    # Less memory than the way to the boundary holds nothing.
    assert workspace_bases(tmp_path, [16, 112, 128], 32) == [(128, 0), (128, 16), (128, 32)]
