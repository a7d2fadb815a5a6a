// What the parts of the linear layer on 8-bit integers share.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

namespace sgemm {
namespace i8 {

struct Operand {       // int8, k contiguous
  const int8_t *q;
  long long ld;        // bytes, a multiple of 16
  const float *scale;  // of each row
};

struct Result {        // D(i, j) = y + beta D(i, j)
  void *ptr;
  int type;
  long long ld;
  const float *bias;
  float beta;
  int vec;             // no beta, and 16-byte stores to rows are aligned
};

// Few rows of x (M <= kFewRows), without tensor cores. (dp4a runs at 16 per cycle and SM: 4 x 4096 x 14336
// took 18.7 us so, 17 on the tensor cores; 2 x 4096 x 4096 4.4 and 7.7.)
constexpr int kFewRows = 2;
cudaError_t launch_few(int M, int N, int K, const Operand &x, const Operand &w, const Result &d, int sms,
                       cudaStream_t stream);

// out (rows x K FP16 numbers, leading dimension ldo elements, 16-byte aligned rows) = q.
cudaError_t launch_unpack(int rows, int K, const Operand &q, void *out, long long ldo, int sms,
                          cudaStream_t stream);

}  // namespace i8
}  // namespace sgemm
