// Rows of values to and from 8-bit checkpoints: arguments and launchers.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace moe {
namespace checkpoint {

struct Args {
  uint8_t* x;            // [rows][cols] BF16 or FP32, rows ld elements apart
  int64_t ld;
  int64_t rows, cols;
  uint8_t* codes;        // [rows][cols]
  uint8_t* scales;       // [rows][ceil(cols / 32)]
};

// whether a launch of these sizes exists (a launch holds 2^32 threads)
bool fits(int64_t rows, int64_t cols);
void launch_store(hipStream_t st, const Args& a, bool fp32);
void launch_load(hipStream_t st, const Args& a, bool fp32);

}  // namespace checkpoint
}  // namespace moe
