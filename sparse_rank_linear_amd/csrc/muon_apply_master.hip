// The orthogonalised step of bf16 parameters with float master copies.
#include "muon_apply.hpp"

namespace salr {

hipError_t launch_muon_apply_master(const MuonArgs& a, int cls, int64_t c0, int64_t chunks, hipStream_t s) {
  return launch_apply<false, true>(a, cls, c0, chunks, s);
}

}  // namespace salr
