// K steps of the few-rows int8 kernel: which step a wave's i-th load is for and where in the weights it
// lies.  Plain arithmetic, without HIP, so that host code can check it against the buffers' sizes.
#pragma once

namespace qg {

constexpr int kParts = 4;             // waves (8: N = K = 4096, 16 rows 4.6 -> 4.7 us, N = K = 7168 10.3 -> 10.9)
constexpr int kAhead = 4;             // steps loaded ahead

// A wave's steps: wave, wave + kParts, ...
constexpr int wave_steps(int nsteps, int wave) { return (nsteps - wave + kParts - 1) / kParts; }
constexpr int wave_step(int wave, int i) { return wave + kParts * i; }

// Scalar part of the weight offset of a wave's i-th step, chunk `chunk` (256 bytes of 16 columns each).  A
// load past the wave's steps is put out of range by its lanes' offset alone: its scalar part stays at the
// first step, inside the weights, so that neither a check of the lane's offset nor one that subtracts the
// scalar part from the buffer's size lets it through.
constexpr int weight_step_offset(int wave, int i, int cnt, int chunk) {
  return (i < cnt ? wave_step(wave, i) : 0) * 2048 + 256 * chunk;
}

}  // namespace qg
