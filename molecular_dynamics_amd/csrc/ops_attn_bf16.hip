// bf16 instantiations of the structure attention kernels.
#include "ops_attn.hpp"

namespace mdmp {
namespace ops {
int launch_attn_bf16(const AttnArgs& A, int C, int dh, bool split, int what, hipStream_t st) {
  switch (1000 * C + dh) {
    case 32016: return launch_attn_c<uint16_t, 32, 16>(A, split, what, st);
    case 32032: return launch_attn_c<uint16_t, 32, 32>(A, split, what, st);
    case 64016: return launch_attn_c<uint16_t, 64, 16>(A, split, what, st);
    case 64032: return launch_attn_c<uint16_t, 64, 32>(A, split, what, st);
    case 64064: return launch_attn_c<uint16_t, 64, 64>(A, split, what, st);
    case 128016: return launch_attn_c<uint16_t, 128, 16>(A, split, what, st);
    case 128032: return launch_attn_c<uint16_t, 128, 32>(A, split, what, st);
    case 128064: return launch_attn_c<uint16_t, 128, 64>(A, split, what, st);
  }
  return arg_error("structure attention: no kernel for these channels and heads");
}
}  // namespace ops
}  // namespace mdmp
