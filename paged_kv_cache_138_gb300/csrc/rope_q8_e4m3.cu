#include "rope_q8.cuh"

namespace pkv {
namespace rope {

int launch_q8_e4m3(const Q8Params& p, bool step, bool adjacent, int block_size, dim3 grid,
                   void* stream) {
  return launch_q8_of<E4m3Near>(p, step, adjacent, block_size, grid, stream);
}

}  // namespace rope
}  // namespace pkv
