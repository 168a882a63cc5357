"""The offsets that the panel kernel's loads of weight codes and the tiles' copies are made
of, run through on the host: every one that the lanes' own parts leave unmasked lies within
the matrix, no scalar part passes its end, and every block that the product wants is among
them.  Small C++ programs over the kernels' header; no GPU work is issued."""
import os
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "bit_nf4_quantized_10_amd", "csrc")
PROGRAM = r"""
#include <cstdio>
#include <vector>
#include "mx_offsets.hpp"
// rows of a 64 RW-row workgroup's lanes, its chunks, steps and lane groups, as mx_panel_kernel's
int main() {
  const int sizes[][2] = {{8, 40}, {16384, 1280}, {200, 8}, {72, 520}, {64, 512}, {264, 2056}, {1336, 4104}, {1000, 32}, {8, 8}, {8, 32}, {8, 1032}};
  for (auto& size : sizes) {
    const int rows = size[0], cols = size[1], nb = (cols + 31) / 32, chunks = (cols + 511) / 512;
    const long long bytes = 16LL * rows * nb;
    std::vector<char> seen(static_cast<size_t>(rows) * nb, 0);
    for (int row = 0; row < (rows + 127) / 128 * 128; ++row)
      for (int c = 0; c < chunks; ++c)
        for (int s = 0; s < 4; ++s)
          for (int g = 0; g < 4; ++g) {
            const qn::MxOffset o = qn::mx_code_offset(row, rows, nb, c, s, g);
            if (o.scalar >= bytes) return std::printf("%d x %d: scalar part %u of %lld\n", rows, cols, o.scalar, bytes), 1;
            if (o.lane >= bytes) continue;            // the range check sees the lane's part
            const long long at = static_cast<long long>(o.lane) + o.scalar;
            if (at + 16 > bytes || at % 16) return std::printf("%d x %d: row %d chunk %d step %d group %d reads %lld of %lld\n", rows, cols, row, c, s, g, at, bytes), 1;
            if (at / 16 != static_cast<long long>(row) * nb + 16 * c + 4 * s + g) return std::printf("%d x %d: the wrong block\n", rows, cols), 1;
            seen[at / 16] = 1;
          }
    for (char x : seen)
      if (!x) return std::printf("%d x %d: a block is never read\n", rows, cols), 1;
  }
  return 0;
}
"""


STAGES = r"""
#include <cstdio>
#include "mx_offsets.hpp"
// the stages that CoreMx copies for shares of chunks_per chunks, two of them past the end; a
// matrix of one row is the smallest
int main() {
  for (int nb = 1; nb < 200; ++nb) {
    const int chunks = (nb + 15) / 16;
    for (int per = 1; per <= chunks; ++per)
      for (int beg = 0; beg < chunks; beg += per) {
        const int end = beg + per < chunks ? beg + per : chunks, last = 16 * end < nb ? 16 * end : nb;
        for (int stage = 2 * beg; stage < 2 * end + 2; ++stage) {
          const unsigned so = qn::mx_stage_offset(stage, last);
          if (so >= 16u * nb) return std::printf("%d blocks, stage %d: scalar part %u\n", nb, stage, so), 1;
          // where the stage holds a block of the share, it is that stage's
          if (8 * stage < last && so != 128u * stage) return std::printf("%d blocks, stage %d at %u\n", nb, stage, so), 1;
        }
      }
  }
  return 0;
}
"""


@pytest.mark.parametrize("text", [PROGRAM, STAGES], ids=["panels", "tiles"])
def test_no_load_of_codes_leaves_the_matrix(tmp_path, text):
    compiler = shutil.which("g++") or shutil.which("clang++") or shutil.which("hipcc")
    if compiler is None:
        pytest.skip("no C++ compiler")
    source, program = tmp_path / "offsets.cpp", tmp_path / "offsets"
    source.write_text(text)
    subprocess.run([compiler, "-std=c++17", "-O1", "-I", CSRC, str(source), "-o", str(program)], check=True, timeout=120)
    done = subprocess.run([str(program)], capture_output=True, text=True, timeout=60)
    assert done.returncode == 0, done.stdout


def _source(name):
    with open(os.path.join(CSRC, name)) as f:
        return f.read()


def test_the_kernels_load_by_them():
    """The panels' weight codes and the tiles' copies come through these offsets alone."""
    assert _source("mx_core.hpp").count(" so = ") == 1 and "so = mx_stage_offset(" in _source("mx_core.hpp")
    text = _source("mx_gemv.hip")
    body = text[text.index("void mx_panel_kernel"):text.index("void mx_decode_kernel")]
    loads = [line for line in body.splitlines() if "ld128s(rw" in line]
    assert len(loads) == 1 and "mx_code_offset(" in body and "vw[" not in body
