"""Every weight load of the few-rows int8 kernel, those past a wave's last step too, has a scalar offset inside the weights.

The kernel keeps loads past a wave's steps out of range by the lane's offset; the scalar offset that goes with
it still has to lie inside the buffer, or a range check that subtracts it from the buffer's size wraps.  The
arithmetic is compiled for the host from the header that the kernel includes.
"""
import os
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PROGRAM = r"""
#include <cstdio>
#include "qg_int8_steps.h"
using namespace qg;
int main() {
  for (int nsteps = 1; nsteps <= 1023; ++nsteps) {       // k = 128 * nsteps < 2^17
    long long bytes = 64LL * 128 * nsteps;               // the narrowest layer: 64 columns
    int total = 0;
    for (int wave = 0; wave < kParts; ++wave) {
      int cnt = wave_steps(nsteps, wave);
      total += cnt;
      for (int i = 0; i < cnt + kAhead; ++i) {           // the loads that the kernel issues
        if (i < cnt && (wave_step(wave, i) < 0 || wave_step(wave, i) >= nsteps)) {
          std::printf("step: nsteps %d wave %d load %d\n", nsteps, wave, i);
          return 1;
        }
        for (int chunk = 0; chunk < 8; ++chunk) {        // a step's eight 16-byte chunks of K
          long long so = weight_step_offset(wave, i, cnt, chunk);
          if (i < cnt && so != wave_step(wave, i) * 2048LL + 256 * chunk) {
            std::printf("offset: nsteps %d wave %d load %d\n", nsteps, wave, i);
            return 1;
          }
          // the last lane of the last column block of 16 reads 16 bytes from here (k / 16 units of 256 bytes per block)
          long long lane = 3LL * nsteps * 8 * 256 + 15 * 16;
          if (so < 0 || so + 16 > bytes || (i < cnt && lane + so + 16 > bytes)) {
            std::printf("range: nsteps %d wave %d load %d of %d chunk %d: %lld of %lld bytes\n", nsteps, wave, i, cnt, chunk, so,
                        bytes);
            return 1;
          }
        }
      }
    }
    if (total != nsteps) {
      std::printf("waves take %d of %d steps\n", total, nsteps);
      return 1;
    }
  }
  return 0;
}
"""


def test_scalar_offsets_lie_inside_the_weights(tmp_path):
    src, exe = tmp_path / "steps.cpp", tmp_path / "steps"
    src.write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-I", os.path.join(ROOT, "quantized_gemm_amd", "csrc"), str(src), "-o", str(exe)],
                   check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout
