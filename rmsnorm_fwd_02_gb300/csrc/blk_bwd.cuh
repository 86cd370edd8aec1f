// blk_bwd.cuh -- the backward of a block's boundary for sm_103a (include/block_train.h), and of
// the norm that keeps its input in 8 bits (include/act8_train.h).  Included by the translation
// units of the two activation types.
//
// HBM-bound: up to 12 bytes an element (h, dy, dh, x; dx, dresidual; h and x 1.03 each where they
// are kept in 8 bits) for some 26 to 29 (32) thread instructions where rows are even, 31 (39) where
// a thread's last vector may be missing and each vector has a predicate.  Two row sums follow one
// another: of dy w_pre h for the gradient t of h, then of the branch's gradient times x for dx; t
// waits between them in registers.  One column sum serves both dw_post and the gate's gradient: S =
// sum of t * xhat over a sample's rows, of which dgate is scale * w_post * S and dw_post the sum over
// samples of scale * gate * S.
//
// A team sums its columns in FP32 over its rows (in registers, or in tensor memory: uses_tmem), a CTA
// its teams' sums, which it writes as one row of partials; the finish adds these in a fixed order.
// Both carry the additions' errors along; a team's own sums are plain.  Past 64 rows they have two
// levels (kFold): every f rows the sums are added to those in tensor memory and start again, which
// of the error after n rows of either sign leaves sqrt(f / n + 1 / f), so f is about the root of n.  (dw of
// 65536 x 8192, where n is 431: at most 1.14 of 1e-4 + 1e-4 |dw| off with one level, 0.41 with two.)
// With a gate for each of several samples, a team writes its S whenever its rows pass into another
// sample (row k + n for team k and sample n: teams and samples both go forward, so no two share one).
//
// Measured, both norms, a gate and dh, 65536 rows: of 4096 521 us (93 % of a plain copy's rate over
// the 12 bytes), of 1536 205 (89 %), of 512 81 (75 %); from 8 bits 445 (91 % of its 10), 175 and 82.
// The norm alone from 8 bits, of 4096 with dh 296 us (96 %), without 245 (83 %).  Past bandwidth the
// threads' own dependencies bound it: two to four warps a scheduler issue in 33 to 57 % of cycles.
#pragma once

#include "blk_common.cuh"

namespace blk {

// Vector c of a staged row: 16-bit values, or 8-bit numbers; their values are v * the unit that is
// returned (a vector lies in one block, so the unit can go to what the numbers are multiplied by).
template <typename T, bool kPacked>
__device__ __forceinline__ float load_saved(const Args& a, const Team& t, uint32_t at, int c,
                                            bool live, f2 (&v)[4]) {
  if constexpr (kPacked) {
    act8_numbers8(lds64_at(live ? at + 8u * c : t.zero), v);
    const uint32_t scale = at + ((static_cast<uint32_t>(a.H) + 15u) & ~15u) + (c >> 2);
    return act8_unit(lds8_at(live ? scale : t.zero));
  } else {
    VecOf<T>::unpack(lds128_at(live ? at + 16u * c : t.zero), v);
    return 1.f;
  }
}

// A team's sums of its columns to row `out` (rows side by side in a warp are added), and back to
// zero.
template <int VPT>
__device__ __forceinline__ void write_sums(const Args& a, const Team& t, float* out,
                                           f2 (&acc)[VPT][4]) {
#pragma unroll
  for (int v = 0; v < VPT; ++v) {
    const int c = t.lt + v * a.ntg;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      for (int o = a.ntg; o < 32; o <<= 1) {
        const float lo = __shfl_xor_sync(0xffffffffu, f2_lo(acc[v][q]), o);
        const float hi = __shfl_xor_sync(0xffffffffu, f2_hi(acc[v][q]), o);
        acc[v][q] = f2_add(acc[v][q], f2_make(lo, hi));
      }
    }
    if (8 * c < a.H && t.sub == 0) {
      float4* p = reinterpret_cast<float4*>(out) + 2 * c;
      p[0] = make_float4(f2_lo(acc[v][0]), f2_hi(acc[v][0]), f2_lo(acc[v][1]), f2_hi(acc[v][1]));
      p[1] = make_float4(f2_lo(acc[v][2]), f2_hi(acc[v][2]), f2_lo(acc[v][3]), f2_hi(acc[v][3]));
    }
#pragma unroll
    for (int q = 0; q < 4; ++q) acc[v][q] = f2_splat(0.f);
  }
}

// The teams' rows of sums in shared memory to one row of the CTA, in the teams' order, the additions'
// errors carried along.
__device__ __forceinline__ void join_teams(const Args& a, const float* rows, float* out) {
  for (int col = static_cast<int>(threadIdx.x); col < a.H; col += static_cast<int>(blockDim.x)) {
    float s = 0.f, e = 0.f;
    for (int k = 0; k < a.teams; ++k) {
      float err;
      s = add_exact(s, rows[k * a.H + col], err);
      e = __fadd_rn(e, err);
    }
    out[col] = isfinite(s) ? __fadd_rn(s, e) : s;
  }
}

template <typename T, int VPT, int kForm, bool kPacked, bool kEven, int kLong, bool kTmem,
          bool kMore = false>
__global__ void __launch_bounds__(bwd_threads(kForm, kTmem, kMore), 1) blk_bwd_kernel(const BwdArgs a) {
  constexpr bool kPostN = kForm == kBoth || kForm == kPost, kPreN = kForm != kPost;
  constexpr bool kX = kForm != kKeep, kFold = kLong != kShort;
  extern __shared__ __align__(128) unsigned char smem[];
  const uint64_t pol = l2_evict_first_policy();
  // Sums in tensor memory (kTm), then their second level (kFold): of each for each vector 8 columns of
  // dw_pre's, then 8 of S; the warps that share a quarter of its lanes side by side.
  constexpr bool kTm = kTmem && VPT >= 3;
  constexpr int kTmVec = kX ? 16 : 8, kTmLevel = kTmVec * VPT, kTmWarp = (kTm + kFold) * kTmLevel;
  constexpr int kTmCols =
      kTmWarp > 0
          ? static_cast<int>(tmem_alloc_cols(bwd_threads(kForm, kTmem, kMore) / 128 * kTmWarp))
          : 0;
  static_assert(kTmCols <= 512);
  Team t = team_begin<4, kTmCols>(a, smem, pol, a.samples == 1);
  uint32_t tm = 0u;
  if constexpr (kTmCols > 0) {
    const uint32_t warp = threadIdx.x >> 5;
    tm = tmem_warp_addr(*t.tmem, warp, (warp >> 2) * kTmWarp);
  }
  const int NV = a.H >> 3;
  // (a factor in shared memory: each thread's part is its own, the rows of a warp share theirs)
  constexpr bool kFactorMem = factor_in_smem(kForm, kPacked);
  f2 w[VPT][4], k1[kFactorMem ? 1 : VPT][4];
  f2 sum_pre[VPT][4], sum_s[VPT][4];  // (kTm: filled from tensor memory where they are written)
  float4* const k1_mem =
      reinterpret_cast<float4*>(smem + a.factor_at) + t.team * (2 * VPT * a.ntg) + t.lt;
  auto set_factor = [&](int32_t n) {
    if constexpr (kFactorMem) {
      f2 f[VPT][4];
      load_factor<VPT, kPostN>(a, n, t.lt, f);
      __syncwarp();
#pragma unroll
      for (int v = 0; v < VPT; ++v) {
        if (t.sub != 0) continue;  // (the rows of a warp have one sample)
        k1_mem[(2 * v) * a.ntg] =
            make_float4(f2_lo(f[v][0]), f2_hi(f[v][0]), f2_lo(f[v][1]), f2_hi(f[v][1]));
        k1_mem[(2 * v + 1) * a.ntg] =
            make_float4(f2_lo(f[v][2]), f2_hi(f[v][2]), f2_lo(f[v][3]), f2_hi(f[v][3]));
      }
      __syncwarp();
    } else {
      load_factor<VPT, kPostN>(a, n, t.lt, k1);
    }
  };
  auto get_factor = [&](int v, f2 (&f)[4]) {
    if constexpr (kFactorMem) {
      const float4 p = k1_mem[(2 * v) * a.ntg], q = k1_mem[(2 * v + 1) * a.ntg];
      f[0] = f2_make(p.x, p.y);
      f[1] = f2_make(p.z, p.w);
      f[2] = f2_make(q.x, q.y);
      f[3] = f2_make(q.z, q.w);
    } else {
#pragma unroll
      for (int q = 0; q < 4; ++q) f[q] = k1[v][q];
    }
  };
#pragma unroll
  for (int v = 0; v < VPT; ++v) {
    const int c = t.lt + v * a.ntg;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      sum_pre[v][q] = f2_splat(0.f);
      sum_s[v][q] = f2_splat(0.f);
    }
    if constexpr (kPreN) {
#pragma unroll
      for (int q = 0; q < 4; ++q) w[v][q] = f2_splat(0.f);
      if (kEven || c < NV) load8(a.w_pre, a.w_dtype, c, w[v]);
    }
  }
  const f2 zero[4] = {f2_splat(0.f), f2_splat(0.f), f2_splat(0.f), f2_splat(0.f)};
  auto load_cells = [&](uint32_t at, float (&to)[VPT][8]) {
#pragma unroll
    for (int v = 0; v < VPT; ++v) tmem_ld8(at + kTmVec * v, to[v]);
  };
  // (after a wait for them)
  auto add_cells = [&](float (&cells)[VPT][8], f2 (&sum)[VPT][4]) {
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      tmem_loaded(cells[v]);
#pragma unroll
      for (int q = 0; q < 4; ++q)
        sum[v][q] = f2_add(sum[v][q], f2_make(cells[v][2 * q], cells[v][2 * q + 1]));
    }
  };
  auto clear = [&](f2 (&sum)[VPT][4]) {
#pragma unroll
    for (int v = 0; v < VPT; ++v)
#pragma unroll
      for (int q = 0; q < 4; ++q) sum[v][q] = f2_splat(0.f);
  };
  // what tensor memory has of one kind's sums (at `from`) added to those in registers, and zeros in
  // its place
  auto take_sums = [&](int from, f2 (&sum)[VPT][4]) {
    if constexpr (kTm || kFold) {
      __syncwarp();
      tmem_wait_st();
#pragma unroll
      for (int o = 0; o < kTmWarp; o += kTmLevel) {
        float cells[VPT][8];
        load_cells(tm + o + from, cells);
        tmem_wait_ld(cells[0]);
        add_cells(cells, sum);
#pragma unroll
        for (int v = 0; v < VPT; ++v) tmem_st8(tm + o + kTmVec * v + from, zero);
      }
    }
  };
  // every sum to its second level, and zeros in its place; few waits: the team does nothing else
  auto fold_sums = [&] {
    const uint32_t second = tm + kTmWarp - kTmLevel;
    __syncwarp();
    tmem_wait_st();
    if constexpr (kTm) {
#pragma unroll
      for (int from = kPreN ? 0 : 8; from < kTmVec; from += 8) {
        float one[VPT][8], two[VPT][8];
        f2 sum[VPT][4];
        load_cells(tm + from, one);
        load_cells(second + from, two);
        tmem_wait_ld(one[0]);
        clear(sum);
        add_cells(one, sum);
        add_cells(two, sum);
#pragma unroll
        for (int v = 0; v < VPT; ++v) {
          tmem_st8(second + kTmVec * v + from, sum[v]);
          tmem_st8(tm + kTmVec * v + from, zero);
        }
      }
    } else {
      float pre[VPT][8], s[VPT][8];
      if constexpr (kPreN) load_cells(second, pre);
      if constexpr (kX) load_cells(second + 8, s);
      if constexpr (kPreN) tmem_wait_ld(pre[0]);
      if constexpr (!kPreN) tmem_wait_ld(s[0]);
      if constexpr (kPreN) add_cells(pre, sum_pre);
      if constexpr (kX) add_cells(s, sum_s);
#pragma unroll
      for (int v = 0; v < VPT; ++v) {
        if constexpr (kPreN) tmem_st8(second + kTmVec * v, sum_pre[v]);
        if constexpr (kX) tmem_st8(second + kTmVec * v + 8, sum_s[v]);
      }
      if constexpr (kPreN) clear(sum_pre);
      if constexpr (kX) clear(sum_s);
    }
  };
  if constexpr (kTmCols > 0) {
    __syncwarp();
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
#pragma unroll
      for (int o = 0; o < kTmWarp; o += kTmLevel) {
        tmem_st8(tm + o + kTmVec * v, sum_pre[v]);
        if constexpr (kX) tmem_st8(tm + o + kTmVec * v + 8, sum_s[v]);
      }
    }
  }
  const float inv_h = 1.f / static_cast<float>(a.H);
  const f2 rscale = f2_splat(a.residual_scale);
  const int side = a.ntg < 32 ? 32 / a.ntg : 1;  // rows side by side
  const bool has_dh = kFold ? kLong == kLongDh : a.in[2].p != nullptr;
  int32_t sample = kX ? t.r0 / a.L : 0;
  int32_t next_sample = (sample + 1) * a.L;  // the row from which k1 and S are another sample's
  if constexpr (kX) {
    if (t.r0 < t.r1) set_factor(sample);
  }
  // the r's of the row ahead, so that no row waits for them
  float r1_next = 0.f, r2_next = 0.f;
  auto fetch = [&](int32_t row) {
    if (row < t.r1) {
      if constexpr (kPreN) r2_next = __ldg(a.rstd_pre + row);
      if constexpr (kPostN) r1_next = __ldg(a.rstd_post + row);
    }
  };
  fetch(t.r0 + t.sub);
  // the rows of one sample that are taken together from row on, of n
  auto take = [&](int32_t row, int32_t n) {
    int32_t k = kEven ? 1 : min(side, n);
    if (kX && !kEven && a.samples > 1) k = min(k, next_sample - row);
    return k;
  };
  int s = 0;
  uint32_t parity = 0;
  int32_t j = 0, until = kFold ? min(a.fold, t.nslots) : t.nslots;
  for (;;) {
    for (; j < until; ++j) {
      wait_slot(a, t, s, parity);
      const int32_t ra = t.r0 + j * t.stride;
      const int32_t n = min(a.rows, t.r1 - ra);
      for (int32_t i = 0; i < n;) {
        if constexpr (kX) {
          if (a.samples > 1 && ra + i >= next_sample) {
            take_sums(8, sum_s);
            write_sums<VPT>(a, t, a.part_s + (t.k + sample) * a.H, sum_s);
            sample = (ra + i) / a.L;
            next_sample = (sample + 1) * a.L;
            set_factor(sample);
          }
        }
        const int32_t together = take(ra + i, n - i);
        const int32_t row = ra + i + t.sub;
        const bool valid = kEven || t.sub < together;
        const uint32_t base = t.ring + static_cast<uint32_t>(s) * a.slot;
        const uint32_t at = static_cast<uint32_t>(i + t.sub);  // (lanes without a row read zeros)
        const uint32_t hs = base + a.in[0].off + at * a.in[0].bytes;
        const uint32_t dys = base + a.in[1].off + at * a.in[1].bytes;
        const uint32_t dhs = base + a.in[2].off + at * a.in[2].bytes;
        const uint32_t xs = base + a.in[3].off + at * a.in[3].bytes;
        // (a lane without a row has zeros throughout, and adds zeros to its columns' sums)
        const float r1 = valid ? r1_next : 0.f, r2 = valid ? r2_next : 0.f;
        fetch(i + together < n ? row + together : ra + t.stride + t.sub);
        const bool first = i == 0;
        i += together;
        // Packed vectors stay in registers between the passes over a row, times rstd (h, then x in its
        // place): their unpacking is three times that of 16-bit values, which are read again.
        f2 kept[kPacked ? VPT : 1][4];
        f2 nc2 = f2_splat(0.f);
        if constexpr (kPreN) {
          f2 dot0 = f2_splat(0.f), dot1 = f2_splat(0.f);
#pragma unroll
          for (int v = 0; v < VPT; ++v) {
            const int c = t.lt + v * a.ntg;
            const bool live = kEven || (valid && c < NV);
            const uint4 dyw = lds128_at(live ? dys + 16u * c : t.zero);
            if constexpr (kPacked) {
              f2 dy[4];
              const f2 rh = f2_splat(load_saved<T, kPacked>(a, t, hs, c, live, kept[v]) * r2);
              VecOf<T>::unpack(dyw, dy);
#pragma unroll
              for (int q = 0; q < 4; q += 2) {
                kept[v][q] = f2_mul(kept[v][q], rh);
                kept[v][q + 1] = f2_mul(kept[v][q + 1], rh);
                dot0 = f2_fma(f2_mul(dy[q], w[v][q]), kept[v][q], dot0);
                dot1 = f2_fma(f2_mul(dy[q + 1], w[v][q + 1]), kept[v][q + 1], dot1);
              }
            } else {
              const uint4 hw = lds128_at(live ? hs + 16u * c : t.zero);
#pragma unroll
              for (int q = 0; q < 4; q += 2) {
                dot0 = f2_fma(mul_exact<T>(u4_get(dyw, q), u4_get(hw, q)), w[v][q], dot0);
                dot1 = f2_fma(mul_exact<T>(u4_get(dyw, q + 1), u4_get(hw, q + 1)), w[v][q + 1], dot1);
              }
            }
          }
          const f2 d = f2_add(dot0, dot1);
          const float dot = row_sum(a, t, f2_lo(d) + f2_hi(d));
          if (first && t.warps > 1 && t.leader && j >= 1 && j - 1 + a.stages < t.nslots)
            issue<4>(a, t, j - 1 + a.stages, pol);
          // t = r2 (dy w - hhat mean(dy w hhat)); from 16 bits the sum is of dy w h
          nc2 = f2_splat(-(kPacked ? dot * inv_h : dot * (r2 * inv_h)));
        }
        const f2 r2v = f2_splat(r2), r1v = f2_splat(r1);
        // without dh the 8-bit norm's t has no use but its outputs: its factor r2 goes to theirs
        const bool late = kForm == kKeep && !has_dh;
        const f2 ro = late ? f2_splat(a.residual_scale * r2) : rscale;
        f2 m[VPT][4];
        f2 dot0 = f2_splat(0.f), dot1 = f2_splat(0.f);
        const size_t out_row = static_cast<size_t>(row) * a.H;
        if constexpr (kTm) {
          __syncwarp();
          tmem_wait_st();  // the row before's sums are stored before they are loaded
        }
#pragma unroll
        for (int v = 0; v < VPT; ++v) {
          const int c = t.lt + v * a.ntg;
          const bool live = kEven || (valid && c < NV);
          f2 g[4], ap[4], as[4];
          float tp[8], ts[8];  // sums from tensor memory, to be read after the wait
          if constexpr (kTm) {
            tmem_ld8(tm + kTmVec * v, tp);
            if constexpr (kX) tmem_ld8(tm + kTmVec * v + 8, ts);
          }
          if constexpr (kPreN) {
            f2 h[4], dy[4];
            if constexpr (!kPacked) {
              load_saved<T, kPacked>(a, t, hs, c, live, h);
#pragma unroll
              for (int q = 0; q < 4; ++q) h[q] = f2_mul(h[q], r2v);
            }
            VecOf<T>::unpack(lds128_at(live ? dys + 16u * c : t.zero), dy);
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const f2 hhat = kPacked ? kept[kPacked ? v : 0][q] : h[q];
              g[q] = f2_fma(hhat, nc2, f2_mul(dy[q], w[v][q]));
              if constexpr (kTm)
                ap[q] = f2_mul(dy[q], hhat);
              else
                sum_pre[v][q] = f2_fma(dy[q], hhat, sum_pre[v][q]);
            }
          }
          f2 dh[4] = {f2_splat(0.f), f2_splat(0.f), f2_splat(0.f), f2_splat(0.f)};
          if (!kPreN || has_dh) VecOf<T>::unpack(lds128_at(live ? dhs + 16u * c : t.zero), dh);
          if (!late) {
#pragma unroll
            for (int q = 0; q < 4; ++q) g[q] = kPreN ? f2_fma(g[q], r2v, dh[q]) : dh[q];
          }
          f2 o[4];
#pragma unroll
          for (int q = 0; q < 4; ++q) o[q] = f2_mul(g[q], ro);
          if (live) stg128(static_cast<T*>(a.dres) + out_row + 8 * c, VecOf<T>::pack(o));
          if constexpr (kX) {
            f2 x[4];
            const float u = load_saved<T, kPacked>(a, t, xs, c, live, x);
            const f2 rx = f2_splat(kPostN ? r1 * u : u);
            f2 f[4];
            get_factor(v, f);
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const f2 xh = kPostN || kPacked ? f2_mul(x[q], rx) : x[q];
              if constexpr (kPostN && kPacked) kept[v][q] = xh;
              if constexpr (kTm)
                as[q] = f2_mul(g[q], xh);
              else
                sum_s[v][q] = f2_fma(g[q], xh, sum_s[v][q]);
              m[v][q] = f2_mul(g[q], f[q]);
            }
            if constexpr (kPostN) {
#pragma unroll
              for (int q = 0; q < 4; q += 2) {
                dot0 = f2_fma(m[v][q], kPacked ? kept[kPacked ? v : 0][q] : x[q], dot0);
                dot1 = f2_fma(m[v][q + 1], kPacked ? kept[kPacked ? v : 0][q + 1] : x[q + 1], dot1);
              }
            }
            if (!kPostN && live)
              stg128(static_cast<T*>(a.dx) + out_row + 8 * c, VecOf<T>::pack(m[v]));
          } else if (live && a.dx != nullptr) {
            f2 d[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) d[q] = f2_mul(g[q], f2_splat(late ? a.scale * r2 : a.scale));
            stg128(static_cast<T*>(a.dx) + out_row + 8 * c, VecOf<T>::pack(d));
          }
          if constexpr (kTm) {
            __syncwarp();
            tmem_wait_ld(tp);
            if constexpr (kX) tmem_loaded(ts);
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              ap[q] = f2_add(f2_make(tp[2 * q], tp[2 * q + 1]), ap[q]);
              if constexpr (kX) as[q] = f2_add(f2_make(ts[2 * q], ts[2 * q + 1]), as[q]);
            }
            tmem_st8(tm + kTmVec * v, ap);
            if constexpr (kX) tmem_st8(tm + kTmVec * v + 8, as);
          }
        }
        if constexpr (kPostN) {
          const f2 d = f2_add(dot0, dot1);
          const float dot = row_sum(a, t, f2_lo(d) + f2_hi(d));
          if (!kPreN && first && t.warps > 1 && t.leader && j >= 1 && j - 1 + a.stages < t.nslots)
            issue<4>(a, t, j - 1 + a.stages, pol);
          const f2 nc1 = f2_splat(-(kPacked ? dot * inv_h : dot * (r1 * inv_h) * r1));
#pragma unroll
          for (int v = 0; v < VPT; ++v) {
            const int c = t.lt + v * a.ntg;
            const bool live = kEven || (valid && c < NV);
            f2 x[4], o[4];
            if constexpr (kPacked) {
#pragma unroll
              for (int q = 0; q < 4; ++q) x[q] = kept[v][q];
            } else {
              load_saved<T, kPacked>(a, t, xs, c, live, x);
            }
#pragma unroll
            for (int q = 0; q < 4; ++q) o[q] = f2_mul(f2_fma(x[q], nc1, m[v][q]), r1v);
            if (live) stg128(static_cast<T*>(a.dx) + out_row + 8 * c, VecOf<T>::pack(o));
          }
        }
      }
      if (t.warps == 1) {
        __syncwarp();
        if (t.leader && j + a.stages < t.nslots) issue<4>(a, t, j + a.stages, pol);
      }
      if (++s == a.stages) {
        s = 0;
        parity ^= 1u;
      }
    }
    if (until == t.nslots) break;
    if constexpr (kFold) fold_sums();
    until = t.nslots - until > a.fold ? until + a.fold : t.nslots;
  }
  drain(a, t);
  if constexpr (kTmCols > 0) {
    if constexpr (kPreN) take_sums(0, sum_pre);
    if constexpr (kX) take_sums(8, sum_s);
    __syncwarp();
    tmem_wait_st();
    tmem_fence_before_sync();
    __syncthreads();
    if (threadIdx.x < 32) {
      __syncwarp();
      tmem_fence_after_sync();
      tmem_dealloc_warp(*t.tmem, kTmCols);
    }
  }
  if (kX && a.samples > 1) {
    // (a team without rows writes zeros: it lies among the teams of its first row's sample)
    write_sums<VPT>(a, t, a.part_s + (t.k + sample) * a.H, sum_s);
  }
  const int64_t cta = static_cast<int64_t>(blockIdx.x) * a.H;
  if (a.teams == 1) {
    if constexpr (kPreN) write_sums<VPT>(a, t, a.part_pre + cta, sum_pre);
    if (kX && a.samples == 1) write_sums<VPT>(a, t, a.part_s + cta, sum_s);
    return;
  }
  __syncthreads();  // every team is done with its ring
  float* rows = reinterpret_cast<float*>(smem);
  if constexpr (kPreN) write_sums<VPT>(a, t, rows + t.team * a.H, sum_pre);
  float* rows_s = rows + (kPreN ? a.teams * a.H : 0);
  if (kX && a.samples == 1) write_sums<VPT>(a, t, rows_s + t.team * a.H, sum_s);
  __syncthreads();
  if constexpr (kPreN) join_teams(a, rows, a.part_pre + cta);
  if (kX && a.samples == 1) join_teams(a, rows_s, a.part_s + cta);
}

// The build for a shape.  (Few vectors a thread are a matter of narrow rows or of few, which keep no
// sums in tensor memory but have its builds' threads.)
template <typename T, int VPT, bool kEven, int kLong>
const void* pick_bwd(int form, bool packed, bool tmem, bool more) {
  auto fn = [](auto k) { return reinterpret_cast<const void*>(k); };
#define BLK_PICK(F)                                                     \
  (packed ? fn(&blk_bwd_kernel<T, VPT, F, true, kEven, kLong, false>)          \
          : fn(&blk_bwd_kernel<T, VPT, F, false, kEven, kLong, false>))
  if (form == kBoth && tmem) return fn(&blk_bwd_kernel<T, VPT, kBoth, true, kEven, kLong, true>);
  if constexpr (VPT == 4) {
    if (form == kKeep && tmem) return fn(&blk_bwd_kernel<T, VPT, kKeep, true, kEven, kLong, true>);
    if (form == kBoth && packed) return fn(&blk_bwd_kernel<T, VPT, kBoth, true, kEven, kLong, false>);
  }
  if constexpr (VPT == 3 && kEven) {  // (more_rows' rows are even)
    if (more) return fn(&blk_bwd_kernel<T, VPT, kKeep, true, kEven, kLong, false, true>);
  }
  switch (form) {
    case kKeep: return BLK_PICK(kKeep);
    case kPre: return BLK_PICK(kPre);
    case kBoth: return fn(&blk_bwd_kernel<T, VPT, kBoth, false, kEven, kLong, false>);
    default:
      if constexpr (kLong == kLongNoDh)
        return nullptr;  // (dh is all there is)
      else
        return BLK_PICK(kPost);
  }
#undef BLK_PICK
}

template <typename T, int kLong>
cudaError_t launch_bwd_t(const BwdArgs& a, const Shape& s, int form, bool packed, cudaStream_t st) {
  const bool even = even_rows(a.H, s.vpt, s.ntg), tmem = uses_tmem(form, packed, a.H),
             more = more_rows(form, packed, s.vpt, s.ntg);
  const void* fn = s.vpt == 1   ? pick_bwd<T, 1, false, kLong>(form, packed, tmem, more)
                   : s.vpt == 2 ? pick_bwd<T, 2, false, kLong>(form, packed, tmem, more)
                   : s.vpt == 3 ? (even ? pick_bwd<T, 3, true, kLong>(form, packed, tmem, more)
                                        : pick_bwd<T, 3, false, kLong>(form, packed, tmem, more))
                                : (even ? pick_bwd<T, 4, true, kLong>(form, packed, tmem, more)
                                        : pick_bwd<T, 4, false, kLong>(form, packed, tmem, more));
  const cudaError_t e = prepare_kernel(fn, s.smem);
  if (e != cudaSuccess) return e;
  BwdArgs copy = a;
  void* args[] = {&copy};
  return launch_pdl(fn, dim3(static_cast<unsigned>(s.P)), dim3(static_cast<unsigned>(s.threads)),
                    s.smem, st, args);
}

}  // namespace blk
