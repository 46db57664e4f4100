// The orthogonalised step of bf16 parameters.
#include "muon_apply.hpp"

namespace salr {

hipError_t launch_muon_apply_bf16(const MuonArgs& a, int cls, int64_t c0, int64_t chunks, hipStream_t s) {
  return launch_apply<false, false>(a, cls, c0, chunks, s);
}

}  // namespace salr
