// fa_paged_duo.cu -- two phases of a paged call side by side: some CTAs run the
// kernel for many query rows (fa_paged_prompt.cuh), the others the one for few
// (fa_paged_decode.cuh).  The first is bound by the tensor core and, when there
// is little of it, by its own latencies, the second by memory, so together they
// take little longer than the longer one: the prompt chunks and the decoding
// sequences of a mixed batch, or a shared prefix and the sequences' own keys.
//
// Every CTA works out the same split of the CTAs, in proportion to the time the
// two lists take: a step of the prompt kernel (two Q tiles, a key tile) 1.6 us
// and the end of a unit 6 us, a tile of the decode kernel 1.0 us on half of the
// SMs (76 CTAs read 5.1 of the 5.4 TB/s that 152 read) and a unit's end 1.5 us.
// These were measured at d = 128 with units of 8 rows, a unit's end behind shared
// prefixes of 2K and 16K keys, and serve d = 64 and units of 16 rows too, where
// they have not been measured apart: they decide how well the two kinds end
// together, never the result, and a list with work has CTAs whatever they say.
//
// Clusters of two CTAs have one kind of work: two neighbouring SMs that run
// both kinds, whose loops together do not fit what they share of the
// instruction cache, take 4 us instead of 1.5 for a step of the prompt kernel
// (a call behind a shared prefix of 16K keys 67 us instead of 58).
//
// With 32 query and 8 key/value heads, d = 128, the merge or join included: two
// chunks of 500 rows among 30 single ones, up to 2,500 keys each, 60 us; 64
// sequences of up to 500 own keys behind 16K shared ones 50 us.
#include "fa_paged_decode.cuh"
#include "fa_paged_launch.h"
#include "fa_paged_prompt.cuh"

namespace fa {
namespace {

constexpr PagedWeight kPromptWeight = {16, 60}, kDecodeWeight = {10, 15};  // 0.1 us

template <int D, int R, bool kNeg>
__global__ void __launch_bounds__(kPagedThreads, 1)
    fa_paged_duo_kernel(const __grid_constant__ CUtensorMap tqa,
                        const __grid_constant__ CUtensorMap tqb,
                        const __grid_constant__ CUtensorMap tk,
                        const __grid_constant__ CUtensorMap tv,
                        const __grid_constant__ CUtensorMap to, const PagedParams p,
                        const PagedPhase pa, const PagedPhase pb) {
  extern __shared__ uint8_t smem_raw[];
  launch_dependents();
  wait_prior_grid();
  long long wa, wb;
  paged_weights(p, pa, kPromptWeight, pb, kDecodeWeight, wa, wb);
  const int ctas = gridDim.x;
  const int na = paged_duo_split(wa, wb, ctas, paged_groups(p, pa, ctas - 2));
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    *pa.ctas = na;
    *pb.ctas = ctas - na;
  }
  if ((int)blockIdx.x < na)
    prompt_cta<D, kNeg, true>(&tqa, &tk, &tv, &to, p, pa, blockIdx.x, na, smem_raw);
  else
    decode_cta<D, R, true>(&tqb, &tk, &tv, p, pb, blockIdx.x - na, ctas - na, smem_raw);
}

template <int D, int R, bool kNeg>
int launch(const PagedMaps& t, const CUtensorMap& tq_b, const PagedParams& p,
           const PagedPhase& pa, const PagedPhase& pb, const cudaLaunchConfig_t& base) {
  cudaLaunchConfig_t c = base;
  c.blockDim = dim3(kPagedThreads, 1, 1);
  c.gridDim.x &= ~1u;
  cudaLaunchAttribute attrs[2];
  attrs[0] = base.attrs[0];
  attrs[1].id = cudaLaunchAttributeClusterDimension;
  attrs[1].val.clusterDim.x = 2;
  attrs[1].val.clusterDim.y = attrs[1].val.clusterDim.z = 1;
  c.attrs = attrs;
  c.numAttrs = 2;
  const size_t a = sizeof(PromptSmem<D>), b = sizeof(DecodeSmem<D, R>);
  c.dynamicSmemBytes = (a > b ? a : b) + 1024;
  if (paged_kernel_ready<fa_paged_duo_kernel<D, R, kNeg>>(c.dynamicSmemBytes) != FA_OK)
    return FA_ERR_LAUNCH;
  if (cudaLaunchKernelEx(&c, fa_paged_duo_kernel<D, R, kNeg>, t.q, tq_b, t.k, t.v, t.o, p, pa,
                         pb) != cudaSuccess) {
    cudaGetLastError();
    return FA_ERR_LAUNCH;
  }
  return FA_OK;
}

template <int D, bool kNeg>
int launch_rows(const PagedMaps& t, const CUtensorMap& tq_b, const PagedParams& p,
                const PagedPhase& pa, const PagedPhase& pb, const cudaLaunchConfig_t& c) {
  if (pb.slot_rows == 8) return launch<D, 8, kNeg>(t, tq_b, p, pa, pb, c);
  if (pb.slot_rows == 16) return launch<D, 16, kNeg>(t, tq_b, p, pa, pb, c);
  return FA_ERR_LAUNCH;
}

}  // namespace

int launch_paged_duo(const PagedMaps& t, const CUtensorMap& tq_b, const PagedParams& params,
                     const PagedPhase& pa, const PagedPhase& pb, int d,
                     const cudaLaunchConfig_t& c) {
  PagedParams p = params;
  if (p.scale_log2 == 0.f) p.scale_log2 = 1.17549435e-38f;  // as the prompt kernel takes it
  if (p.scale_log2 < 0.f)
    return d == 128 ? launch_rows<128, true>(t, tq_b, p, pa, pb, c)
                    : launch_rows<64, true>(t, tq_b, p, pa, pb, c);
  return d == 128 ? launch_rows<128, false>(t, tq_b, p, pa, pb, c)
                  : launch_rows<64, false>(t, tq_b, p, pa, pb, c);
}

}  // namespace fa
