"""Host functions of the library that need no CUDA, compiled on their own."""
import os
import subprocess

from mlx_grouped_affine_gb300 import build


def workspace_bases(folder, addresses, size):
    """(base, bytes) of the part of [address, address + size) that the kernels use."""
    source, program = os.path.join(str(folder), "base.cpp"), os.path.join(str(folder), "base")
    with open(source, "w") as f:
        f.write('#include <cstdio>\n#include <cstdlib>\n#include "workspace.h"\n'
                'int main(int n, char **v) {\n'
                '  for (int i = 2; i < n; ++i) {\n'
                '    void *p = reinterpret_cast<void *>(strtoull(v[i], nullptr, 10));\n'
                '    qmm::Workspace w = qmm::aligned_workspace(p, strtoull(v[1], nullptr, 10));\n'
                '    printf("%llu %llu\\n", (unsigned long long)(uintptr_t)w.base, (unsigned long long)w.bytes);\n'
                '  }\n}\n')
    subprocess.run(["g++", "-std=c++17", "-I", build.CSRC, source, "-o", program], check=True)
    r = subprocess.run([program, str(size)] + [str(a) for a in addresses], check=True, capture_output=True, text=True)
    return [tuple(int(x) for x in line.split()) for line in r.stdout.splitlines()]
