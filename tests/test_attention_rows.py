"""Whatever a sequence's offsets hold, the rows that the attention takes lie inside the queries.

The arithmetic is compiled for the host from the header that the kernels include.
"""
import os
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PROGRAM = r"""
#include <cstdio>
#include "qg_attention_rows.h"
using namespace qg;
int main() {
  const int32_t least = -2147483647 - 1, most = 2147483647;
  const int32_t offsets[] = {least, least + 1, -16777217, -5, -1, 0, 1, 3, 7, 8, 9, 100, 16777216, 16777217, most - 1, most};
  const long long counts[] = {1, 8, 100, 16777216};
  const int limits[] = {1, 2, 8, 65535};
  for (long long tokens : counts)
    for (int max_q : limits)
      for (int32_t begin : offsets)
        for (int32_t end : offsets) {
          const Queries q = sequence_queries(begin, end, tokens, max_q);
          bool ok = q.count >= 0 && q.count <= max_q && (q.count == 0 || (q.first >= 0 && q.first + q.count <= tokens));
          if (begin >= end && q.count != 0 && begin >= 0) ok = false;                 // nothing lies between
          if (begin >= 0 && begin <= end && end <= tokens)                            // offsets as they should be
            ok = ok && q.first == begin && q.count == (end - begin < max_q ? end - begin : max_q);
          if (!ok) {
            std::printf("offsets %d %d of %lld tokens, at most %d: %lld + %d\n", begin, end, tokens, max_q, (long long)q.first, q.count);
            return 1;
          }
        }
  return 0;
}
"""


def test_rows_of_any_offsets_lie_inside(tmp_path):
    src, exe = tmp_path / "rows.cpp", tmp_path / "rows"
    src.write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-I", os.path.join(ROOT, "quantized_gemm_amd", "csrc"), str(src), "-o", str(exe)],
                   check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout
