// fa_paged4.cu -- attention over a paged key/value cache held in 4 bits: the kernel
// for few query rows (fa_paged4_decode.cuh), and the choice of kernels for a call.
#include "fa_internal.h"
#include "fa_kv4.cuh"
#include "fa_paged.cuh"
#include "fa_paged4_decode.cuh"
#include "fa_paged_launch.h"
#include "sm100_ptx.cuh"

namespace fa {
namespace {

template <int D, int R>
__global__ void __launch_bounds__(Decode4Cfg<D, R>::kThreads, Decode4Cfg<D, R>::kCtas)
    fa_paged4_decode_kernel(const Paged4Params p, const PagedPhase ph, int subs) {
  extern __shared__ uint8_t smem_raw[];
  decode4_cta<D, R>(p, ph, subs, blockIdx.x, gridDim.x, smem_raw);
}

template <int D, int R>
int launch_decode(const Paged4Params& p, const PagedPhase& ph, int subs,
                  const cudaLaunchConfig_t& base) {
  static_assert((sizeof(Decode4Smem<D, R>) + 128 + 1024) * Decode4Cfg<D, R>::kCtas <= 233472,
                "shared memory above the 228 KB of an SM, of which a CTA takes 1 KB more");
  cudaLaunchConfig_t c = base;
  c.blockDim = dim3(Decode4Cfg<D, R>::kThreads, 1, 1);
  c.dynamicSmemBytes = sizeof(Decode4Smem<D, R>) + 128;
  if (paged_kernel_ready<fa_paged4_decode_kernel<D, R>, 0>(c.dynamicSmemBytes) != FA_OK)
    return FA_ERR_LAUNCH;
  if (cudaLaunchKernelEx(&c, fa_paged4_decode_kernel<D, R>, p, ph, subs) != cudaSuccess) {
    cudaGetLastError();
    return FA_ERR_LAUNCH;
  }
  return FA_OK;
}

template <int D>
int launch_paged4_d(const Paged4Params& p, cudaStream_t stream) {
  cudaLaunchAttribute pdl[1];
  pdl[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  pdl[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t c = {};
  c.stream = stream;
  c.attrs = pdl;
  c.numAttrs = 1;
  const Paged4Form f = paged4_form(p.T, p.B, p.G, p.max_q, p.v_scale);
  const Paged4Workspace w = paged4_workspace_layout(D, f);
  auto at = [&](size_t offset) { return reinterpret_cast<float*>(p.workspace + offset); };
  int rc;
  c.gridDim = dim3((unsigned)p.ctas, 1, 1);
  if (f.prompt) {
    PagedPhase ph = {};
    ph.rec = p.workspace + w.rec[1];
    ph.slot_o = at(w.slot_o[1]);
    ph.slot_lse = at(w.slot_lse[1]);
    ph.n_min = f.small_tokens + 1;
    ph.n_max = 0x7fffffff;
    if ((rc = launch_paged4_prompt(p, ph, D, c)) != FA_OK) return rc;
    if ((rc = launch_paged_merge(p, ph, D, 0, c)) != FA_OK) return rc;
  }
  if (f.rows > 0) {
    Paged4Params q = p;  // its heads are runs of a token's
    q.G = f.heads;
    q.Hkv = p.Hkv * f.subs;
    q.ctas = p.ctas * kPaged4CtasPerSm;
    c.gridDim.x = (unsigned)q.ctas;
    PagedPhase ph = {};
    ph.rec = p.workspace + w.rec[0];
    ph.slot_o = at(w.slot_o[0]);
    ph.slot_lse = at(w.slot_lse[0]);
    ph.n_max = f.prompt ? f.small_tokens : 0x7fffffff;
    ph.unit_tokens = ph.tile_tokens = f.rows / f.heads;
    ph.slot_rows = f.rows;
    rc = f.rows == 8 ? launch_decode<D, 8>(q, ph, f.subs, c) : launch_decode<D, 16>(q, ph, f.subs, c);
    if (rc != FA_OK) return rc;
    if ((rc = launch_paged_merge(q, ph, D, 4, c)) != FA_OK) return rc;
  }
  return FA_OK;
}

}  // namespace

int launch_fwd_paged4(const Paged4Params& p, int d, cudaStream_t stream) {
  return d == 128 ? launch_paged4_d<128>(p, stream) : launch_paged4_d<64>(p, stream);
}

}  // namespace fa
