// Weight-streaming GEMM instantiations: int8 weights with int8 activations (MoE blocks).
#include "qg_stream_kernel.h"

namespace qg {

bool stream_int8(const StreamArgs& a, const StreamTile& t, int wp, int af, int of, int stype, bool zero, bool moe,
                 hipStream_t st) {
  if (wp == WP_INT8 && af == A_INT8 && of == O_BF16 && stype == S_F32 && zero == false)
    return launch_stream_variant<WP_INT8, A_INT8, O_BF16, S_F32, false>(a, t, moe, st);
  if (wp == WP_INT8 && af == A_INT8 && of == O_F16 && stype == S_F32 && zero == false)
    return launch_stream_variant<WP_INT8, A_INT8, O_F16, S_F32, false>(a, t, moe, st);
  return false;
}

}  // namespace qg
