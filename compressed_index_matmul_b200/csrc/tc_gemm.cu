// The tensor-core forward without a fused epilogue, and its plan (the kernel: tc_gemm.cuh).
#include "tc_gemm.cuh"

namespace vq {

bool plan_tc(const vq_linear_desc& d, const DeviceInfo& dev, int M, Plan* p) {
  if (M < 1 || dev.smem_optin < (int)kTcSmemMax) return false;
  const TcGeom g = tc_geom(d.fmt, d.n16, d.n8, M, d.N, d.K, dev.num_sms);
  p->path = VQ_PATH_TC;
  p->splits = g.S;
  p->k_per_split = g.kps;
  p->launches = 1;
  const bool partials = g.S > 1 && g.epi == kEpiGlobal;
  p->scratch_bytes = partials ? (size_t)g.S * M * d.N * sizeof(float) : 0;
  p->tickets = partials ? g.RT * g.TT : 0;
  p->ctas = g.RT * g.TT * g.S;
  return true;
}

cudaError_t launch_tc(const LayerArgs& a, const Plan& pl, float* scratch, uint32_t* tickets, uint32_t* err,
                      cudaStream_t s) {
  return a.epi ? launch_tc_fused(a, pl, scratch, tickets, err, s)
               : launch_tc_f<false>(a, pl, scratch, tickets, err, s);
}

}  // namespace vq
