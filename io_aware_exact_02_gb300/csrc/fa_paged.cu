// fa_paged.cu -- attention over a paged key/value cache on sm_103a: the kernel
// for few query rows (fa_paged_decode.cuh) on all CTAs, the kernels that join
// what was computed in parts, and the choice of kernels for a call.
#include "fa_internal.h"
#include "fa_paged.cuh"
#include "fa_paged_decode.cuh"
#include "fa_paged_launch.h"
#include "sm100_ptx.cuh"

namespace fa {
namespace {

template <int D, int R>
__global__ void __launch_bounds__(kPagedThreads, 1)
    fa_paged_decode_kernel(const __grid_constant__ CUtensorMap tq,
                           const __grid_constant__ CUtensorMap tk,
                           const __grid_constant__ CUtensorMap tv, const PagedParams p,
                           const PagedPhase ph) {
  extern __shared__ uint8_t smem_raw[];
  decode_cta<D, R, false>(&tq, &tk, &tv, p, ph, blockIdx.x, gridDim.x, smem_raw);
}

// Joins the parts of the units that were shared between CTAs.  The blocks of
// a column of the grid look at one boundary between CTAs; the columns of the
// boundaries inside a unit share its rows, several warps to a row when the
// rows are few; parts are added in list order within a warp and the warps'
// sums in order, so the result does not depend on timing.
//
// Bound by latency (2.6 us after the attention kernel for 8 units of 4 rows in
// 8 parts each), or by memory: 10 us for the 40 MB of parts that prompt chunks
// of 4,096 rows leave, most of it in L2.
constexpr int kMergeWarps = 8;

template <int D>
__global__ void __launch_bounds__(32 * kMergeWarps) fa_paged_merge_kernel(const PagedParams p,
                                                                          const PagedPhase ph0,
                                                                          const PagedPhase ph1) {
  const PagedPhase& ph = blockIdx.z == 0 ? ph0 : ph1;
  launch_dependents();
  wait_prior_grid();
  constexpr int kPer = D / 32;
  __shared__ float part_o[kMergeWarps][D], part_l[kMergeWarps], part_m[kMergeWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int ctas = ph.ctas ? *ph.ctas : p.ctas;
  const PagedRec rec = *reinterpret_cast<const PagedRec*>(ph.rec + blockIdx.x * kPagedRecBytes);
  if ((int)blockIdx.x >= ctas || !rec.split) return;
  const int c0 = rec.slot >> 1, n = rec.n;
  // Block `y` of the unit's `ny`.
  const int ny = (n - 1) * (int)gridDim.y;
  const int y = ((int)blockIdx.x - c0 - 1) * (int)gridDim.y + (int)blockIdx.y;
  const float ninf = __int_as_float(0xff800000);
  const int rows = rec.ntok * p.G;
  int share = 1;  // warps to a row
  while (share < kMergeWarps && 2 * share * rows <= ny * kMergeWarps && 2 * share <= n) share *= 2;
  // Row r's place in a slot: two Q tiles at most, 128 rows apart.
  const int tile_rows = ph.tile_tokens * p.G;
  auto place = [&](int r) { return r < tile_rows ? r : kTile + r - tile_rows; };
  auto load = [&](long long slot_row, float (&v)[kPer]) {
    const float* src = ph.slot_o + slot_row * D + lane * kPer;
    if constexpr (kPer == 4) {
      const float4 x = *reinterpret_cast<const float4*>(src);
      v[0] = x.x, v[1] = x.y, v[kPer - 2] = x.z, v[kPer - 1] = x.w;
    } else {
      const float2 x = *reinterpret_cast<const float2*>(src);
      v[0] = x.x, v[1] = x.y;
    }
  };
  auto store = [&](int r, const float (&acc)[kPer], float m, float sum) {
    const int tok = (int)((unsigned)r / (unsigned)p.G), head = r - tok * p.G;
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    const long long out = (long long)(rec.tok0 + tok) * p.Hq + rec.h * p.G + head;
    const float lse2 = sum == 0.f ? ninf : m + log2f(sum);
    int no_abort = 0;
    if (!bound_ok(rec.tok0 + tok < p.T && rec.h < p.Hkv, p.status, &no_abort, kChkPgRow)) return;
    if (ph.out_o) {
      float* dst = ph.out_o + out * D + lane * kPer;
#pragma unroll
      for (int e = 0; e < kPer; ++e) dst[e] = acc[e] * inv;
      if (lane == 0) ph.out_lse[out] = lse2;
    } else {
      __nv_bfloat16* dst = p.o + out * D + lane * kPer;
#pragma unroll
      for (int e = 0; e < kPer; e += 2)
        *reinterpret_cast<uint32_t*>(dst + e) = pack_bf16x2(acc[e] * inv, acc[e + 1] * inv);
      if (lane == 0) p.lse[out] = lse2 == ninf ? ninf : lse2 * kLn2;
    }
  };
  if (n == 2 && share == 1) {
    // Many rows of two parts (a prompt's): two rows of a warp in flight.  (Four
    // were slower, by the longer code: prompt chunks of 4,096 rows 177 us
    // instead of 174.)
    constexpr int kRows = 2;
    const int step = ny * kMergeWarps;
    for (int r0 = y * kMergeWarps + warp; r0 < rows; r0 += kRows * step) {
      float v[kRows][2][kPer], w[kRows][2];
#pragma unroll
      for (int k = 0; k < kRows; ++k) {
        const int row = place(min(r0 + k * step, rows - 1));
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const long long s = (long long)(i == 0 ? rec.slot : 2 * (c0 + 1)) * ph.slot_rows + row;
          w[k][i] = ph.slot_lse[s];
          load(s, v[k][i]);
        }
      }
#pragma unroll
      for (int k = 0; k < kRows; ++k) {
        if (r0 + k * step >= rows) break;
        const float m = fmaxf(w[k][0], w[k][1]);
        const bool none = w[k][0] == ninf && w[k][1] == ninf;
        const float a = none ? 0.f : exp2f(w[k][0] - m), b = none ? 0.f : exp2f(w[k][1] - m);
        float acc[kPer];
#pragma unroll
        for (int x = 0; x < kPer; ++x)
          acc[x] = (a != 0.f ? a * v[k][0][x] : 0.f) + (b != 0.f ? b * v[k][1][x] : 0.f);
        store(r0 + k * step, acc, m, a + b);
      }
    }
    return;
  }
  const int per_block = kMergeWarps / share, sub = warp % share;
  for (int r0 = y * per_block; r0 < rows; r0 += ny * per_block) {
    const int r = r0 + warp / share;
    const bool valid = r < rows;
    const int row = place(valid ? r : 0);
    auto slot_of = [&](int i) -> long long {
      return (long long)(i == 0 ? rec.slot : 2 * (c0 + i)) * ph.slot_rows + row;
    };
    // One pass over the parts, kBatch of them in flight, with the running
    // maximum of their logsumexp.
    constexpr int kBatch = 4;
    float m = ninf, acc[kPer], sum = 0.f;
#pragma unroll
    for (int i = 0; i < kPer; ++i) acc[i] = 0.f;
    for (int i0 = sub; i0 < n; i0 += kBatch * share) {
      float v[kBatch][kPer], w[kBatch], top = m;
#pragma unroll
      for (int b = 0; b < kBatch; ++b) {
        const int i = i0 + b * share;
        w[b] = ninf;
#pragma unroll
        for (int e = 0; e < kPer; ++e) v[b][e] = 0.f;
        if (i < n) {
          const long long s = slot_of(i);
          w[b] = ph.slot_lse[s];
          load(s, v[b]);
        }
      }
      bool none = true;  // (of a NaN, `top` would not tell)
#pragma unroll
      for (int b = 0; b < kBatch; ++b) {
        top = fmaxf(top, w[b]);
        none = none && w[b] == ninf;
      }
      if (none) continue;
      const float old = exp2f(m - top);
      m = top;
      sum *= old;
#pragma unroll
      for (int x = 0; x < kPer; ++x) acc[x] *= old;
#pragma unroll
      for (int b = 0; b < kBatch; ++b) {
        const float e = exp2f(w[b] - m);
        sum += e;
        if (e != 0.f) {
#pragma unroll
          for (int x = 0; x < kPer; ++x) acc[x] += e * v[b][x];
        }
      }
    }
    if (share > 1) {  // the same for the whole block
      __syncthreads();  // the last rows' parts were read
#pragma unroll
      for (int e = 0; e < kPer; ++e) part_o[warp][lane * kPer + e] = acc[e];
      if (lane == 0) part_l[warp] = sum, part_m[warp] = m;
      __syncthreads();
      if (sub == 0) {
        float top = m;
        for (int w = 1; w < share; ++w) top = fmaxf(top, part_m[warp + w]);
        if (top == ninf) {
          for (int w = 1; w < share; ++w) sum += part_l[warp + w];  // 0, or NaN
        } else {
          const float own = exp2f(m - top);
          m = top;
          sum *= own;
#pragma unroll
          for (int e = 0; e < kPer; ++e) acc[e] *= own;
          for (int w = 1; w < share; ++w) {
            const float f = exp2f(part_m[warp + w] - top);
            sum += f * part_l[warp + w];
#pragma unroll
            for (int e = 0; e < kPer; ++e) acc[e] += f * part_o[warp + w][lane * kPer + e];
          }
        }
      }
    }
    if (valid && sub == 0) store(r, acc, m, sum);
  }
}

// Joins each row's parts of the shared prefix (pa) and of its sequence's own
// keys (pb), which one launch computed side by side: a warp per row adds them
// up as the merge kernel does.  The attention kernels left word of each unit's
// slots; to find them again from the tables took the row's warp 6 us, most of
// it divisions and the fetching of their code.  The join now ends 4 us after the
// attention for 360 rows of a few parts, 6 us for 2,048 of eleven.
template <int D>
__global__ void __launch_bounds__(256) fa_paged_join_kernel(const PagedParams p,
                                                            const PagedPhase pa,
                                                            const PagedPhase pb) {
  launch_dependents();
  constexpr int kPer = D / 32;
  const int lane = threadIdx.x & 31;
  const int r = (int)((blockIdx.x * blockDim.x + threadIdx.x) >> 5);  // T * Hq rows: some ten thousand
  const int t = r / p.Hq, hq = r - t * p.Hq;
  if (t >= p.T) return;
  const int h = hq / p.G, gh = hq - h * p.G;
  const int tok0 = t / pa.unit_tokens * pa.unit_tokens, tile = (t - tok0) / pa.tile_tokens;
  wait_prior_grid();
  const int first = p.cu_q[0], end = p.cu_q[p.B], ctas_a = *pa.ctas, ctas_b = *pb.ctas;
  const uint2 ua = pa.parts[(long long)tok0 * p.Hkv + h], ub = pb.parts[(long long)t * p.Hkv + h];
  if (t < first || t >= end) return;  // a padding row
  struct Parts {
    int slot, n, row;
  };
  const Parts A = {(int)(ua.x & 0xffff), (int)(ua.x >> 16),
                   tile * kTile + (t - tok0 - tile * pa.tile_tokens) * p.G + gh};
  const Parts B = {(int)(ub.x & 0xffff), (int)(ub.x >> 16), (int)ub.y + gh};
  // A word that cannot be was not written: the row gets no result but an error
  // (already recorded where bad tables or a failed wait are the reason).  Words
  // left by an earlier call in the same workspace may pass; they point into it.
  if (!paged_parts_ok(A.slot, A.n, A.row, ctas_a, pa.slot_rows) ||
      !paged_parts_ok(B.slot, B.n, B.row, ctas_b, pb.slot_rows)) {
    int abort_flag = 0;
    if (lane == 0) report_status(p.status, &abort_flag, FA_ERR_BOUNDS, kChkPgParts);
    return;
  }
  auto src = [&](int k, const float*& o) -> float {
    const bool own = k >= A.n;
    const PagedPhase& ph = own ? pb : pa;
    const Parts& x = own ? B : A;
    const int c = own ? k - A.n : k;
    if (x.n == 1) {  // the whole unit
      o = ph.out_o + (long long)r * D;
      return ph.out_lse[r];
    }
    const long long row =
        (long long)(c == 0 ? x.slot : (x.slot & ~1) + 2 * c) * ph.slot_rows + x.row;
    o = ph.slot_o + row * D;
    return ph.slot_lse[row];
  };
  const int n = A.n + B.n;
  const float ninf = __int_as_float(0xff800000);
  float m = ninf, acc[kPer], sum = 0.f;
#pragma unroll
  for (int e = 0; e < kPer; ++e) acc[e] = 0.f;
  // 32 parts at a time: a lane finds one and weighs it, then all lanes add up
  // the parts, kBatch of them in flight (the first before their weights).
  constexpr int kBatch = 12;
#pragma unroll 1
  for (int k0 = 0; k0 < n; k0 += 32) {
    const float* o = pa.out_o;
    float w = ninf;
    if (k0 + lane < n) w = src(k0 + lane, o);
    const int cnt = min(32, n - k0);
    float f = 0.f;
#pragma unroll 1
    for (int j0 = 0; j0 < cnt; j0 += kBatch) {
      float v[kBatch][kPer];
#pragma unroll
      for (int b = 0; b < kBatch; ++b) {
        const float* from = reinterpret_cast<const float*>(
            __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(o), min(j0 + b, cnt - 1)));
        if constexpr (kPer == 4) {
          const float4 x = *reinterpret_cast<const float4*>(from + lane * kPer);
          v[b][0] = x.x, v[b][1] = x.y, v[b][kPer - 2] = x.z, v[b][kPer - 1] = x.w;
        } else {
          const float2 x = *reinterpret_cast<const float2*>(from + lane * kPer);
          v[b][0] = x.x, v[b][1] = x.y;
        }
      }
      if (j0 == 0) {
        float top = w;
#pragma unroll 1
        for (int x = 16; x > 0; x >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
        top = fmaxf(top, m);
        // (of a NaN, `top` would not tell)
        if (__all_sync(0xffffffffu, w == ninf)) break;
        const float old = exp2f(m - top);
        m = top;
        f = exp2f(w - m);
        float fs = f;
#pragma unroll 1
        for (int x = 16; x > 0; x >>= 1) fs += __shfl_xor_sync(0xffffffffu, fs, x);
        sum = sum * old + fs;
#pragma unroll
        for (int e = 0; e < kPer; ++e) acc[e] *= old;
      }
#pragma unroll
      for (int b = 0; b < kBatch; ++b) {
        const float fb = __shfl_sync(0xffffffffu, f, min(j0 + b, 31));
        if (j0 + b < cnt && fb != 0.f) {
#pragma unroll
          for (int e = 0; e < kPer; ++e) acc[e] += fb * v[b][e];
        }
      }
    }
  }
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  __nv_bfloat16* dst = p.o + (long long)r * D + lane * kPer;
#pragma unroll
  for (int e = 0; e < kPer; e += 2)
    *reinterpret_cast<uint32_t*>(dst + e) = pack_bf16x2(acc[e] * inv, acc[e + 1] * inv);
  if (lane == 0) p.lse[r] = sum == 0.f ? ninf : (m + log2f(sum)) * kLn2;
}

template <int D, int R>
int launch_decode(const PagedMaps& t, const PagedParams& p, const PagedPhase& ph,
                  const cudaLaunchConfig_t& base) {
  static_assert(sizeof(DecodeSmem<D, R>) + 1024 <= 232448,
                "decode shared memory above the 227 KB a CTA may have");
  cudaLaunchConfig_t c = base;
  c.blockDim = dim3(kPagedThreads, 1, 1);
  c.dynamicSmemBytes = sizeof(DecodeSmem<D, R>) + 1024;
  if (paged_kernel_ready<fa_paged_decode_kernel<D, R>>(c.dynamicSmemBytes) != FA_OK)
    return FA_ERR_LAUNCH;
  if (cudaLaunchKernelEx(&c, fa_paged_decode_kernel<D, R>, t.q, t.k, t.v, p, ph) != cudaSuccess) {
    cudaGetLastError();
    return FA_ERR_LAUNCH;
  }
  return FA_OK;
}

// The merge of one phase's split units, or of two phases' (ph1 not null).
template <int D>
int launch_merge(const PagedParams& p, const PagedPhase& ph0, const PagedPhase* ph1,
                 const cudaLaunchConfig_t& base) {
  cudaLaunchConfig_t c = base;
  c.blockDim = dim3(32 * kMergeWarps, 1, 1);
  c.dynamicSmemBytes = 0;
  c.gridDim = dim3((unsigned)p.ctas, ph0.slot_rows <= kPagedDecodeRows ? 4 : 8, ph1 ? 2 : 1);
  if (cudaLaunchKernelEx(&c, fa_paged_merge_kernel<D>, p, ph0, ph1 ? *ph1 : ph0) != cudaSuccess) {
    cudaGetLastError();
    return FA_ERR_LAUNCH;
  }
  return FA_OK;
}

// The units of a phase of `rows` rows, and the tensor maps of their Q tiles and
// of the prompt kernel's results.
template <int D>
int phase_units(const PagedParams& p, PagedPhase& ph, int rows, PagedMaps& t, CUtensorMap* tq) {
  const int tile_rows = rows <= kPagedDecodeRows ? rows : kTile;
  ph.tile_tokens = tile_rows / p.G;
  ph.unit_tokens = rows <= kPagedDecodeRows ? ph.tile_tokens : 2 * ph.tile_tokens;
  ph.slot_rows = rows;
  if (rows > kPagedDecodeRows) {
    ph.box_out = 32 % p.G == 0 && ph.out_o == nullptr;
    const int rc = make_tmap_rows(p.o, p.Hq, p.T, (long long)p.Hq * D, D, p.G,
                                  ph.box_out ? 32 / p.G : 1, &t.o);
    if (rc != FA_OK) return rc;
  }
  return make_tmap_rows(p.q, p.Hq, p.T, p.q_stride, D, p.G, ph.tile_tokens, tq);
}

// One phase's attention kernel on all CTAs.
template <int D>
int launch_phase(const PagedParams& p, PagedPhase& ph, int rows, PagedMaps& t,
                 const cudaLaunchConfig_t& c) {
  const int rc = phase_units<D>(p, ph, rows, t, &t.q);
  if (rc != FA_OK) return rc;
  switch (rows) {
    case 8: return launch_decode<D, 8>(t, p, ph, c);
    case 16: return launch_decode<D, 16>(t, p, ph, c);
    case 32: return launch_decode<D, 32>(t, p, ph, c);
    case 64: return launch_decode<D, 64>(t, p, ph, c);
    default: return launch_paged_prompt(t, p, ph, D, c);
  }
}

template <int D>
int launch_paged_d(const PagedParams& p, cudaStream_t stream) {
  cudaLaunchAttribute pdl[1];
  pdl[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  pdl[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t c = {};
  c.gridDim = dim3((unsigned)p.ctas, 1, 1);
  c.stream = stream;
  c.attrs = pdl;
  c.numAttrs = 1;
  const PagedForm f = paged_form(p.T, p.B, p.Hq, p.G, p.max_q, p.prefix_len);
  const PagedWorkspace w = paged_workspace_layout(p.T, p.Hq, p.Hkv, D, f);
  const int box = p.page_size < kTile ? p.page_size : kTile;
  PagedMaps t;
  int rc;
  if ((rc = make_tmap_bhnd_rows(p.k_pages, p.num_pages * p.Hkv, p.page_size, D, box, &t.k)) != FA_OK ||
      (rc = make_tmap_bhnd_rows(p.v_pages, p.num_pages * p.Hkv, p.page_size, D, box, &t.v)) != FA_OK)
    return rc;
  auto at = [&](size_t offset) { return reinterpret_cast<float*>(p.workspace + offset); };
  PagedPhase ph[2] = {};
  for (int k = 0; k < 2; ++k) {
    ph[k].rec = p.workspace + w.rec[k];
    ph[k].slot_o = at(w.slot_o[k]);
    ph[k].slot_lse = at(w.slot_lse[k]);
    ph[k].n_max = 0x7fffffff;
    if (f.duo) ph[k].ctas = reinterpret_cast<int*>(p.workspace + w.ctas) + k;
  }
  if (f.share) {
    PagedPhase pre = ph[0];
    pre.whole_batch = 1;
    pre.out_o = at(w.pre_o);
    pre.out_lse = at(w.pre_lse);
    if (f.duo) {
      // The prefix beside the sequences' own keys, then their join.
      PagedPhase own = ph[1];
      own.key0 = p.prefix_len;
      own.out_o = at(w.own_o);
      own.out_lse = at(w.own_lse);
      pre.parts = reinterpret_cast<uint2*>(p.workspace + w.parts[0]);
      own.parts = reinterpret_cast<uint2*>(p.workspace + w.parts[1]);
      CUtensorMap tq_own;
      if ((rc = phase_units<D>(p, pre, f.prefix_rows, t, &t.q)) != FA_OK ||
          (rc = phase_units<D>(p, own, f.rows, t, &tq_own)) != FA_OK ||
          (rc = launch_paged_duo(t, tq_own, p, pre, own, D, c)) != FA_OK)
        return rc;
      c.blockDim = dim3(256, 1, 1);
      c.gridDim = dim3((unsigned)(((long long)p.T * p.Hq + 7) / 8), 1, 1);
      if (cudaLaunchKernelEx(&c, fa_paged_join_kernel<D>, p, pre, own) != cudaSuccess) {
        cudaGetLastError();
        return FA_ERR_LAUNCH;
      }
      return FA_OK;
    }
    if ((rc = launch_phase<D>(p, pre, f.prefix_rows, t, c)) != FA_OK) return rc;
    if ((rc = launch_merge<D>(p, pre, nullptr, c)) != FA_OK) return rc;
    for (int k = 0; k < 2; ++k) {
      ph[k].key0 = p.prefix_len;
      ph[k].pre_o = pre.out_o;
      ph[k].pre_lse = pre.out_lse;
    }
  }
  const bool mixed = f.small_rows > 0;
  if (mixed) {
    ph[1].n_max = f.small_rows / p.G;
    ph[0].n_min = ph[1].n_max + 1;
  }
  if (f.duo) {
    CUtensorMap tq_small;
    if ((rc = phase_units<D>(p, ph[0], f.rows, t, &t.q)) != FA_OK ||
        (rc = phase_units<D>(p, ph[1], f.small_rows, t, &tq_small)) != FA_OK ||
        (rc = launch_paged_duo(t, tq_small, p, ph[0], ph[1], D, c)) != FA_OK)
      return rc;
  } else {
    if (mixed && (rc = launch_phase<D>(p, ph[1], f.small_rows, t, c)) != FA_OK) return rc;
    if ((rc = launch_phase<D>(p, ph[0], f.rows, t, c)) != FA_OK) return rc;
  }
  return launch_merge<D>(p, ph[0], mixed ? &ph[1] : nullptr, c);
}

}  // namespace

int launch_fwd_paged(const PagedParams& p, int d, cudaStream_t stream) {
  return d == 128 ? launch_paged_d<128>(p, stream) : launch_paged_d<64>(p, stream);
}

}  // namespace fa
