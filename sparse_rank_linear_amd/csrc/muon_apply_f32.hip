// The orthogonalised step of float parameters.
#include "muon_apply.hpp"

namespace salr {

hipError_t launch_muon_apply_f32(const MuonArgs& a, int cls, int64_t c0, int64_t chunks, hipStream_t s) {
  return launch_apply<true, false>(a, cls, c0, chunks, s);
}

}  // namespace salr
