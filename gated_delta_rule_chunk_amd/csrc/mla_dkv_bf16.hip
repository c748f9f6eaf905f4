// The bf16 dk, dv kernels (mla_dkv.hpp), compiled with their accumulators in the
// second half of the register file: the 160 accumulators of Dn = 128, Dr = 64
// and the operands do not fit the first half, and copies between the halves
// cost 7% of the whole backward. float32 is the other way round (13%).
#include "mla_dkv.hpp"

namespace kda {

hipError_t launch_mla_dkv_bf16(const MlaArgs& a, hipStream_t s) { return mla::launch_dkv_dims<__bf16>(a, s); }

}  // namespace kda
