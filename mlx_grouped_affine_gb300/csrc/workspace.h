// Where the kernels begin in a caller's workspace.  Host code without CUDA headers.
#pragma once
#include <cstddef>
#include <cstdint>

namespace qmm {

// Callers give 16-byte aligned memory; the widest stores into it are 32 bytes, and
// whole 128-byte lines are what the memory system moves.
constexpr size_t kWorkspaceAlign = 128;

struct Workspace {
  char *base;
  size_t bytes;
};

// The part of `bytes` bytes at p that begins on a kWorkspaceAlign boundary.
inline Workspace aligned_workspace(void *p, size_t bytes) {
  const size_t skip = (kWorkspaceAlign - reinterpret_cast<uintptr_t>(p) % kWorkspaceAlign) % kWorkspaceAlign;
  return Workspace{static_cast<char *>(p) + skip, bytes < skip ? 0 : bytes - skip};
}

}  // namespace qmm
