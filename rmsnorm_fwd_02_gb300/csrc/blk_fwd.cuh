// blk_fwd.cuh -- the forward of a block's boundary for sm_103a (include/block_train.h), and of
// the norm that keeps its input in 8 bits (include/act8_train.h).  Included by the translation
// units of the two activation types.
//
// HBM-bound: 8 bytes an element (x, residual; h, y) and 1.03 for each tensor kept in 8 bits, for
// some 16 thread instructions.  Two row sums follow one another, of x^2 and, through rstd, of h^2,
// so a row cannot be streamed; it waits in shared memory, h between the sums in registers.
//
// Measured, both norms and a gate, 65536 rows: of 4096 352 us (92 % of a plain copy's rate over the 8
// bytes), of 1536 137 (88 %), of 512 52 (78 %); keeping 8 bits 425 (95 % of 10), 172, 65.  The norm
// alone keeping 8 bits: of 4096 214 us (95 %), with a residual 398 (92 %).
#pragma once

#include "blk_common.cuh"

namespace blk {

// One 16-byte vector, packed into its row; every lane of the warp takes part, with zeros where the
// vector is not there (`live`).
template <typename T>
__device__ __forceinline__ void keep8(unsigned char* packed_row, int first_scale, int c, bool live,
                                      const uint4& u) {
  const uint4 one[1] = {u};
  const uint32_t amax = act8_max_block(act8_max8<T>(one));
  if (!live) return;
  const uint32_t s = act8_scale_byte(amax);
  *reinterpret_cast<uint2*>(packed_row + 8 * c) = act8_pack8<T>(u, amax, s);
  if ((c & 3) == 0) packed_row[first_scale + (c >> 2)] = static_cast<unsigned char>(s);
}
// A packed row's padding, by the first threads of its row (at least four).
__device__ __forceinline__ void keep8_padding(const Args& a, int lt, unsigned char* p) {
  const int first = static_cast<int>(act8_scale_offset(a.H));
  if (lt == 3 && a.H < first) *reinterpret_cast<uint2*>(p + a.H) = make_uint2(0u, 0u);
  if (lt < 3) act8_pad_scales(p + first, (a.H + kAct8Block - 1) / kAct8Block, lt);
}

template <typename T, int VPT, int kForm, bool kPack, bool kEven>
__global__ void __launch_bounds__(fwd_threads(kForm), 1) blk_fwd_kernel(const FwdArgs a) {
  constexpr bool kPostN = kForm == kBoth || kForm == kPost, kPreN = kForm != kPost;
  extern __shared__ __align__(128) unsigned char smem[];
  const uint64_t pol = l2_evict_first_policy();
  Team t = team_begin<2>(a, smem, pol, true);
  const int NV = a.H >> 3;
  f2 w[VPT][4];   // w_pre
  f2 k1[VPT][4];  // scale * gate * w_post
  if constexpr (kPreN) {
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      const int c = t.lt + v * a.ntg;
#pragma unroll
      for (int q = 0; q < 4; ++q) w[v][q] = f2_splat(0.f);
      if (kEven || c < NV) load8(a.w_pre, a.w_dtype, c, w[v]);
    }
  }
  int32_t next_sample = 0;  // the row from which k1 is another sample's
  const float inv_h = 1.f / static_cast<float>(a.H);
  const f2 rscale = f2_splat(a.residual_scale);
  const int step = a.ntg < 32 ? 32 / a.ntg : 1;
  const int64_t packed_row = act8_row_size(a.H);
  const int first_scale = static_cast<int>(act8_scale_offset(a.H));
  const bool padded = a.H % 512 != 0;  // numbers and scales are not both whole 16 bytes
  int s = 0;
  uint32_t parity = 0;
  for (int32_t j = 0; j < t.nslots; ++j) {
    wait_slot(a, t, s, parity);
    const int32_t ra = t.r0 + j * t.stride;
    const int32_t n = min(a.rows, t.r1 - ra);
    for (int32_t i = 0; i < n; i += step) {
      const int32_t row = ra + i + t.sub;
      const bool valid = kEven || i + t.sub < n;
      const uint32_t slot = t.ring + static_cast<uint32_t>(s) * a.slot +
                            static_cast<uint32_t>(i + t.sub) * (static_cast<uint32_t>(a.H) * 2u);
      const uint32_t xs = slot + a.in[0].off, rs = slot + a.in[1].off;
      if constexpr (kForm != kKeep) {
        if (valid && row >= next_sample) {
          const int32_t sample = row / a.L;
          load_factor<VPT, kPostN>(a, sample, t.lt, k1);
          next_sample = (sample + 1) * a.L;
        }
      }
      f2 r1 = f2_splat(1.f);
      if constexpr (kPostN) {
        f2 ss = f2_splat(0.f);
#pragma unroll
        for (int v = 0; v < VPT; ++v) {
          const int c = t.lt + v * a.ntg;
          const uint4 xw = lds128_at(kEven || (valid && c < NV) ? xs + 16u * c : t.zero);
#pragma unroll
          for (int q = 0; q < 4; ++q) ss = square_onto<T>(u4_get(xw, q), ss);
        }
        const float sum = row_sum(a, t, f2_lo(ss) + f2_hi(ss));
        if (i == 0 && t.warps > 1 && t.leader && j >= 1 && j - 1 + a.stages < t.nslots)
          issue<2>(a, t, j - 1 + a.stages, pol);
        const float r = row_rstd(sum, inv_h, a.eps);
        if (valid && t.lt == 0) a.rstd_post[row] = r;
        r1 = f2_splat(r);
      }
      f2 h[VPT][4];
      f2 ss = f2_splat(0.f);
#pragma unroll
      for (int v = 0; v < VPT; ++v) {
        const int c = t.lt + v * a.ntg;
        const bool live = kEven || (valid && c < NV);
        const bool add = kForm != kKeep || a.in[1].p != nullptr;
        const uint4 xw = lds128_at(live ? xs + 16u * c : t.zero);
        uint4 o = xw;
        if constexpr (kForm == kKeep) {
          VecOf<T>::unpack(xw, h[v]);
          if (add) {
            f2 res[4];
            VecOf<T>::unpack(lds128_at(live ? rs + 16u * c : t.zero), res);
#pragma unroll
            for (int q = 0; q < 4; ++q) h[v][q] = f2_add(h[v][q], res[q]);
            o = VecOf<T>::pack(h[v]);
            VecOf<T>::unpack(o, h[v]);  // the norm of h as it is written
          }
        } else {
          f2 x[4], res[4];
          VecOf<T>::unpack(xw, x);
          VecOf<T>::unpack(lds128_at(live ? rs + 16u * c : t.zero), res);
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const f2 p = kPostN ? f2_mul(x[q], r1) : x[q];
            h[v][q] = f2_fma(p, k1[v][q], f2_mul(res[q], rscale));
          }
          o = VecOf<T>::pack(h[v]);
        }
        if constexpr (kPreN) {
#pragma unroll
          for (int q = 0; q < 4; ++q) ss = f2_fma(h[v][q], h[v][q], ss);
        }
        if (live && (kForm != kKeep || add))
          stg128(static_cast<T*>(a.h) + static_cast<size_t>(row) * a.H + 8 * c, o);
        if constexpr (kPack) {
          if (kForm != kKeep && a.x8 != nullptr)
            keep8<T>(a.x8 + row * packed_row, first_scale, c, live, xw);
          if constexpr (kPreN) keep8<T>(a.h8 + row * packed_row, first_scale, c, live, o);
        }
      }
      if constexpr (kPack) {
        if (padded && valid) {
          if (kForm != kKeep && a.x8 != nullptr) keep8_padding(a, t.lt, a.x8 + row * packed_row);
          if (kPreN) keep8_padding(a, t.lt, a.h8 + row * packed_row);
        }
      }
      if constexpr (kPreN) {
        const float sum = row_sum(a, t, f2_lo(ss) + f2_hi(ss));
        if (!kPostN && i == 0 && t.warps > 1 && t.leader && j >= 1 && j - 1 + a.stages < t.nslots)
          issue<2>(a, t, j - 1 + a.stages, pol);
        const float r = row_rstd(sum, inv_h, a.eps);
        if (valid && t.lt == 0) a.rstd_pre[row] = r;
        const f2 r2 = f2_splat(r);
#pragma unroll
        for (int v = 0; v < VPT; ++v) {
          const int c = t.lt + v * a.ntg;
          f2 y[4];
#pragma unroll
          for (int q = 0; q < 4; ++q) y[q] = f2_mul(f2_mul(h[v][q], r2), w[v][q]);
          if (kEven || (valid && c < NV))
            stg128(static_cast<T*>(a.y) + static_cast<size_t>(row) * a.H + 8 * c, VecOf<T>::pack(y));
        }
      }
    }
    if (t.warps == 1) {
      __syncwarp();
      if (t.leader && j + a.stages < t.nslots) issue<2>(a, t, j + a.stages, pol);
    }
    if (++s == a.stages) {
      s = 0;
      parity ^= 1u;
    }
  }
  drain(a, t);
}

template <typename T, int VPT, bool kEven>
const void* pick_fwd(int form, bool pack) {
  auto fn = [](auto k) { return reinterpret_cast<const void*>(k); };
#define BLK_PICK(F)                                            \
  (pack ? fn(&blk_fwd_kernel<T, VPT, F, true, kEven>)          \
        : fn(&blk_fwd_kernel<T, VPT, F, false, kEven>))
  switch (form) {
    case kKeep: return fn(&blk_fwd_kernel<T, VPT, kKeep, true, kEven>);
    case kPre: return BLK_PICK(kPre);
    case kBoth: return BLK_PICK(kBoth);
    default: return BLK_PICK(kPost);
  }
#undef BLK_PICK
}

template <typename T>
cudaError_t launch_fwd_t(const FwdArgs& a, const Shape& s, int form, bool pack, cudaStream_t st) {
  const bool even = even_rows(a.H, s.vpt, s.ntg);
  const void* fn = s.vpt == 1   ? pick_fwd<T, 1, false>(form, pack)
                   : s.vpt == 2 ? pick_fwd<T, 2, false>(form, pack)
                   : s.vpt == 3 ? (even ? pick_fwd<T, 3, true>(form, pack)
                                        : pick_fwd<T, 3, false>(form, pack))
                                : (even ? pick_fwd<T, 4, true>(form, pack)
                                        : pick_fwd<T, 4, false>(form, pack));
  const cudaError_t e = prepare_kernel(fn, s.smem);
  if (e != cudaSuccess) return e;
  FwdArgs copy = a;
  void* args[] = {&copy};
  return launch_pdl(fn, dim3(static_cast<unsigned>(s.P)), dim3(static_cast<unsigned>(s.threads)),
                    s.smem, st, args);
}

}  // namespace blk
