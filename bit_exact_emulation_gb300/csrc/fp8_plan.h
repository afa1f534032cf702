// fp8_plan.h -- which form an FP8 product takes.
#pragma once
#include "fp8.h"

namespace mcemu {

struct Fp8Plan {
  bool few;                  // fp8_few.cuh, else fp8_pair.cuh
  int width;                 // few: tokens to a tile; pair: rows of b to a tile
  int64_t units;             // tiles at most (a group's rows are known on the device alone)
  int parts, per;            // few: CTAs that share K, blocks of 128 to each
  int64_t clusters;          // and how many such clusters run at a time
  bool turned;               // pair: with the operands exchanged
};
int launch_fp8_pair(const Fp8Product &p, const Fp8Plan &plan, void *stream);
int launch_fp8_few(const Fp8Product &p, const Fp8Plan &plan, void *stream);

}  // namespace mcemu
