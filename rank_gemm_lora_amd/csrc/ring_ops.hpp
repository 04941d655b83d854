// Operands of the ring GEMMs of a fine-tuning step (ring16.hpp runs the loop), and what their epilogues share.
#pragma once

#include "ring16.hpp"
#include "step.hpp"

namespace lora {
namespace {
using namespace pipe;

// NT: rows of outputs. DUAL: the tile's rows are blocks of 16 gate rows and 16 up rows in turn, so that a lane holds the
// gate and the up value of the same four outputs in acc[2 i] and acc[2 i + 1]; a copy instruction's 8 rows then belong
// to one projection, the same for all of a wave's (waves 0 and 1 copy gate rows, 2 and 3 up rows).
template <class P, bool DUAL>
struct NtOp {
  __amdgpu_buffer_rsrc_t xr, wr, xm, tr, wm, br;
  uint32_t ldx_b, ldw_b, ldt_b, ldb_b, ax, aw, c16;
  int NE, hi, seg, kb_total, rows_m, rows_n, per, ph0, ph1, lo;
  NtRows<P> vx, vw;
  __device__ __forceinline__ void init(const RingArgs& p, int64_t m0, int64_t n0, int s_lo, int s_hi) {
    const int side = DUAL ? ring_wave() >> 1 : 0;
    rows_m = static_cast<int>(min<int64_t>(P::BM, p.T - m0));
    rows_n = static_cast<int>(min<int64_t>(DUAL ? P::BN / 2 : P::BN, p.N - n0));
    kb_total = static_cast<int>(p.K[0] * 2);
    ldx_b = static_cast<uint32_t>(p.ldx * 2);
    ldw_b = static_cast<uint32_t>(p.K[0] * 2);
    ldt_b = static_cast<uint32_t>(p.ldt * 2);
    ldb_b = static_cast<uint32_t>(p.re[side] * 2);
    xm = make_rsrc(p.x[0] + m0 * p.ldx, static_cast<uint32_t>(rows_m) * ldx_b);
    wm = make_rsrc(p.W[side] + n0 * p.K[0], static_cast<uint32_t>(rows_n) * ldw_b);
    tr = make_rsrc(p.tt + m0 * p.ldt, static_cast<uint32_t>(rows_m) * ldt_b);
    br = make_rsrc(p.E[side] + n0 * p.re[side], static_cast<uint32_t>(rows_n) * ldb_b);
    NE = p.tt != nullptr ? static_cast<int>(p.ldt / 64) : 0;
    per = (p.re[0] + p.re[1]) * 2;  // bytes of a term's columns; this side's are [ph0, ph1) of them
    ph0 = side ? p.re[0] * 2 : 0;
    ph1 = ph0 + p.re[side] * 2;
    c16 = ring_chunk<P>();
    lo = s_lo;
    hi = s_hi;
    seg = -1;
  }
  __device__ __forceinline__ void w_rows(uint32_t ld) {
    if constexpr (!DUAL) vw.init(ld);
    else vw.init(ld, 16, (ring_wave() & 1) * 8);
  }
  __device__ __forceinline__ void seek(int t) {
    const int s = lo + t;
    if (s < NE && s < hi) {
      if (seg != 0) {
        seg = 0;
        xr = tr;
        wr = br;
        vx.init(ldt_b);
        w_rows(ldb_b);
      }
      ax = static_cast<uint32_t>(s) * 128u;
      const int b = s * 128 + static_cast<int>(c16), ph = b < per ? b : b - per;
      aw = b < 2 * per && ph >= ph0 && ph < ph1 ? static_cast<uint32_t>(ph - ph0) - c16 : kMissing;
    } else {
      if (seg != 1) {
        seg = 1;
        xr = xm;
        wr = wm;
        vx.init(ldx_b);
        w_rows(ldw_b);
      }
      const int kb = (s - NE) * 128;
      ax = aw = s < hi && kb + static_cast<int>(c16) < kb_total ? static_cast<uint32_t>(kb) : kMissing;
    }
  }
  __device__ __forceinline__ void load_x(int l, char* d) const { ring_copy<P>(l, d, xr, vx.at(l, ax)); }
  __device__ __forceinline__ void load_w(int l, char* d) const { ring_copy<P>(l, d, wr, vw.at(l, aw)); }
};

// NN: rows of the contraction: NSEG segments x_i . W_i behind an extension of NEXT adapters. Extension rows are the
// adapters' A rows, once for each term; a copy instruction's rows (2 or 4 of 8 consecutive ones) belong to one adapter.
// (What a form does not have is no member of it: scalar registers run out otherwise, and spill into vector ones.)
template <class P, int NSEG, int NEXT>
struct NnOp {
  const uint16_t *x0, *x1, *W0, *W1;
  const uint16_t* tt;
  __amdgpu_buffer_rsrc_t xr, wr, wr2, er0, er1;
  uint32_t ldx_b, ldw_b, ldt_b, ax, c16;
  int K0, K1, re0, per, NE, n0s, hi, seg, rows_m, cols, lo;
  bool inited = false;
  uint32_t second;  // bit l: copy instruction l takes the second adapter's rows (wr2)
  NtRows<P> vx;
  NnRows<P> vw;
  uint32_t first[NEXT > 0 ? ring_loads<P>() : 1];  // with an extension: where the rows of each instruction start
  __device__ __forceinline__ __amdgpu_buffer_rsrc_t rows_of(const uint16_t* base, int rows) const {
    return make_rsrc(base, rows > 0 ? static_cast<uint32_t>(rows - 1) * ldw_b + static_cast<uint32_t>(cols) * 2 : 0u);
  }
  // x_i [T, K_i] (from row m0 on), W_i [K_i, N], E_i [re_i, N] (columns from n0 on)
  __device__ __forceinline__ void init(const uint16_t* const* xs, int64_t ldx, const uint16_t* const* Ws, const int64_t* Ks,
                                       int64_t T, int64_t N, int64_t m0, int64_t n0, int s_lo, int s_hi) {
    rows_m = static_cast<int>(min<int64_t>(P::BM, T - m0));
    cols = static_cast<int>(min<int64_t>(P::BN, N - n0));
    x0 = xs[0] + m0 * ldx;
    W0 = Ws[0] + n0;
    K0 = static_cast<int>(Ks[0]);
    if constexpr (NSEG > 1) {
      x1 = xs[1] + m0 * ldx;
      W1 = Ws[1] + n0;
      K1 = static_cast<int>(Ks[1]);
    }
    ldx_b = static_cast<uint32_t>(ldx * 2);
    ldw_b = static_cast<uint32_t>(N * 2);
    n0s = (K0 + 63) / 64;
    c16 = ring_chunk<P>();
    NE = 0;
    lo = s_lo;
    hi = s_hi;
    seg = -1;
    second = 0;
  }
  __device__ __forceinline__ void extend(const RingArgs& p, int64_t m0, int64_t n0) {
    if (p.tt == nullptr) return;
    tt = p.tt + m0 * p.ldt;
    ldt_b = static_cast<uint32_t>(p.ldt * 2);
    NE = static_cast<int>(p.ldt / 64);
    re0 = p.re[0];
    per = p.re[0] + (NEXT > 1 ? p.re[1] : 0);
    er0 = rows_of(p.E[0] + n0, p.re[0]);
    if constexpr (NEXT > 1) er1 = rows_of(p.E[1] + n0, p.re[1]);
  }
  __device__ __forceinline__ void seek(int t) {
    const int s = lo + t;
    if (NEXT > 0 && s < NE && s < hi) {
      if (seg != 0) {
        xr = make_rsrc(tt, static_cast<uint32_t>(rows_m) * ldt_b);
        vx.init(ldt_b);
        wr = er0;
        if constexpr (NEXT > 1) wr2 = er1;
      }
      seg = 0;
      ax = static_cast<uint32_t>(s) * 128u;
      if (!inited) vw.init(ldw_b, cols);
      inited = true;
      second = 0;
#pragma unroll
      for (int l = 0; l < ring_loads<P>(); ++l) {  // (groups of eight rows: ranks are multiples of 8)
        const int gr = s * 8 + NnRows<P>::group(l), ph = gr < per / 8 ? gr : gr - per / 8;
        const bool is2 = NEXT > 1 && ph >= re0 / 8;
        first[NEXT > 0 ? l : 0] = gr < per / 4 ? static_cast<uint32_t>(is2 ? ph - re0 / 8 : ph) * 8u * ldw_b : kMissingRow;
        if (NEXT > 1) second |= static_cast<uint32_t>(is2 ? 1 : 0) << l;
      }
    } else {
      const int ms = s - NE;
      const int sg = NSEG == 1 || ms < n0s ? 1 : 2;
      if (seg != sg) {
        if (seg < 1) {
          vx.init(ldx_b);
          if (!inited) vw.init(ldw_b, cols);
          inited = true;
          if constexpr (NEXT > 0) {
#pragma unroll
            for (int l = 0; l < ring_loads<P>(); ++l) first[l] = static_cast<uint32_t>(NnRows<P>::group(l)) * 8u * ldw_b;
          }
        }
        seg = sg;
        xr = make_rsrc(NSEG > 1 && sg == 2 ? x1 : x0, static_cast<uint32_t>(rows_m) * ldx_b);
        second = 0;
      }
      const int k0 = (sg == 1 ? ms : ms - n0s) * 64;
      const int left = s < hi ? min(64, (NSEG > 1 && sg == 2 ? K1 : K0) - k0) : 0;
      ax = static_cast<int>(c16) < left * 2 ? static_cast<uint32_t>(k0) * 2u : kMissing;
      wr = rows_of((NSEG > 1 && sg == 2 ? W1 : W0) + (left > 0 ? static_cast<int64_t>(k0) * (ldw_b / 2) : 0), left);
    }
  }
  __device__ __forceinline__ void load_x(int l, char* d) const { ring_copy<P>(l, d, xr, vx.at(l, ax)); }
  __device__ __forceinline__ void load_w(int l, char* d) const {
    const uint32_t off = vw.at(l, NEXT > 0 ? first[NEXT > 0 ? l : 0] : static_cast<uint32_t>(NnRows<P>::group(l)) * 8u * ldw_b);
    if constexpr (NEXT > 1) ring_copy<P>(l, d, (second >> l) & 1 ? wr2 : wr, off);
    else ring_copy<P>(l, d, wr, off);
  }
};

// Partial sums of a wave's block.
template <class P>
__device__ __forceinline__ void store_part(const f32x4 (&acc)[P::NI][P::NJ], float* part, int64_t ld, int64_t m0,
                                           int64_t n0, int64_t T, int64_t N) {
  const int lane = opaque_int(threadIdx.x & 63), r = lane & 15, q = lane >> 4;
#pragma unroll
  for (int j = 0; j < P::NJ; ++j) {
    const int64_t m = m0 + j * 16 + r;
    if (m >= T) continue;
#pragma unroll
    for (int i = 0; i < P::NI; ++i) {
      const int64_t n = n0 + i * 16 + q * 4;
      float* dst = part + m * ld + n;
      if (ld % 4 == 0 && n + 3 < N) {
        *reinterpret_cast<f32x4*>(dst) = acc[i][j];
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (n + e < N) dst[e] = acc[i][j][e];
      }
    }
  }
}

__device__ __forceinline__ void load_bias4(float (&bv)[4], const uint16_t* bias, int64_t n, int64_t N) {
#pragma unroll
  for (int e = 0; e < 4; ++e) bv[e] = bias != nullptr && n + e < N ? bf16_to_f32(bias[n + e]) : 0.f;
}

}  // namespace
}  // namespace lora
