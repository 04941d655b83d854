// The 16 x 16 x 32 MFMA ring of the hot GEMM (five LDS slots, x and W units of 64 contraction indices, copies and
// fragment reads spread over the MFMA bundles) as a loop over stages whose operands an `Op` names, for the kernels of a
// training step: their operands come from several places (gate and up weights, adapters behind a base weight) and
// their epilogues differ.
//
// acc[i][j] += W-side block i . x-side block j over NS stages. x units are always rows of tokens, contiguous along the
// contraction. W units come in two forms:
//   NT  rows of outputs, contiguous along the contraction (a weight as the forward reads it)
//   NN  rows of the contraction, contiguous along the outputs (the same weight as its input gradient reads it): staged
//       as [64 k][BN] and read with the transposing LDS read, so no transposed copy of the weight is made.
//       (The hot backward's copy of W^T costs a read and a write of the weight in every call.)
//
// An Op has
//   void seek(int s)               makes the copies below those of stage s (called in ascending order from 0; stages past
//                                  the last must read as zeros: they are copied all the same, so that the loop has one
//                                  form and its wait counts are constant)
//   void load_x(int l, char* dst)  copy instruction l of NL of the x unit, and of the W unit
//   void load_w(int l, char* dst)
//   void between(acc)              (with SPLIT) runs once, before a named stage
//   void fetch(int t), next()      (with TOUCH) begins to load what stage t's fragments are changed with, at most one stage
//   void touch(bf16x8& b, int j)   ahead; makes it current; changes fragment j of the x side before it is multiplied
#pragma once

#include "pipe_dev.hpp"

namespace lora {
namespace {
namespace pipe {

// 256 x 256 tiles, one workgroup on a compute unit, and 128 x 128 tiles, two (as the hot GEMM's).
using Ring256 = QCfg<256, 256, 128, 128, 128, 5>;
using Ring128 = QCfg<128, 128, 64, 64, 128, 5, 2>;

typedef __attribute__((__vector_size__(4 * sizeof(short)))) short s16x4;
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;

// A chunk that does not exist gets this added to its offset: past a tile's resource (at most 2^30 bytes: 256 rows of 4 MB),
// with no wrap around behind it.
constexpr uint32_t kMissing = 0x40000000u;
// A row that does not exist of a resource of up to 2^31 bytes (all rows of an adapter: 1024 of 2 MB). The columns that do
// not exist keep kMissing and may lie inside such a resource: what they read reaches outputs that do not exist.
constexpr uint32_t kMissingRow = 0x80000000u;

template <class P>
constexpr int ring_loads() { return P::BM * P::CPR / 64 / P::WAVES; }

__device__ __forceinline__ int ring_wave() { return __builtin_amdgcn_readfirstlane(threadIdx.x >> 6); }

template <class P>
__device__ __forceinline__ void ring_copy(int l, char* dst, __amdgpu_buffer_rsrc_t r, uint32_t off) {
  const int slot0 = (l * P::WAVES + ring_wave()) * 64;
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void*)(dst + slot0 * 16), 16, off, 0, 0, 0);
}

// This lane's 16-byte chunk of a 128-byte row, in bytes (the same in every copy instruction of a unit).
template <class P>
__device__ __forceinline__ uint32_t ring_chunk() {
  const int lane = threadIdx.x & 63;
  return static_cast<uint32_t>(((lane & 7) ^ (((ring_wave() * 8 + (lane >> 3)) >> 1) & 7)) * 16);
}

// A lane's offsets in a unit whose tile row R is source row R: `base` in copy instruction 0, `step` more in each after it.
// (A row behind the last lies behind the resource, whose size is a whole number of row strides: it reads as zeros.)
template <class P>
struct NtRows {
  uint32_t base, step;
  __device__ __forceinline__ void init(uint32_t ld_bytes, int rows_per_copy = P::WAVES * 8, int first = -1) {
    const int lane = opaque_int(threadIdx.x & 63);
    base = static_cast<uint32_t>((first < 0 ? ring_wave() * 8 : first) + (lane >> 3)) * ld_bytes + ring_chunk<P>();
    step = static_cast<uint32_t>(rows_per_copy) * ld_bytes;
  }
  __device__ __forceinline__ uint32_t at(int l, uint32_t add) const { return base + add + static_cast<uint32_t>(l) * step; }
};

// A lane's offsets in an NN unit: tile row k is source row k of the stage (the resource ends behind its last row), and
// 32-byte granule g of it sits at g ^ f(k), f(k) = (k & 3) | (k >> 3 & 1) << 2: the eight rows that half a wave's
// transposing read touches then lie in eight different granules of the 256 bytes of the banks. A wave's rows in one copy
// instruction lie in one group of eight: `base` is the offset within the group (its columns by the group's last bit),
// the rest the same for the whole wave.
template <class P>
struct NnRows {
  static constexpr int LPR = P::BN * 2 / 16, ROWS = 64 / LPR;  // lanes (16-byte pieces) per row; rows per wave
  static constexpr int GPC = P::WAVES * ROWS / 8;              // groups per copy instruction
  uint32_t base[2];
  static_assert(GPC == 1 || GPC == 2, "two or four rows per wave");
  __device__ __forceinline__ static int group(int l) { return GPC == 1 ? l : 2 * l + (ring_wave() >> 1); }
  __device__ __forceinline__ void init(uint32_t ld_bytes, int cols_valid) {
    const int lane = opaque_int(threadIdx.x & 63), p = lane % LPR;
    const int in = (ring_wave() * ROWS + lane / LPR) & 7;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int col = (((p >> 1) ^ ((in & 3) | h << 2)) * 2 + (p & 1)) * 8;
      base[h] = col < cols_valid ? static_cast<uint32_t>(in) * ld_bytes + static_cast<uint32_t>(col) * 2 : kMissing;
    }
  }
  // (a group starts at `rows`, counted from the resource's first)
  __device__ __forceinline__ uint32_t at(int l, uint32_t rows) const {
    return (GPC == 1 ? base[l & 1] : (ring_wave() >> 1) ? base[1] : base[0]) + rows;
  }
};

template <class P, bool NN>
struct RingFrags {
  uint32_t x, w;  // byte offsets of this lane's first fragment in an x / a W unit
  __device__ __forceinline__ void init(int wm0, int wn0) {
    const int lane = threadIdx.x & 63, r = lane & 15, q = lane >> 4;
    const FragOffsets o = frag_offsets<P>(wn0, wm0, lane);
    x = o.x;
    if (NN) {
      // a transposing read gives lane (r, q) rows 8 q .. + 3 of column r where it names row 8 q + r / 4, columns 4 (r % 4)
      const int f = (r >> 2) | ((q & 1) << 2);
      w = static_cast<uint32_t>((8 * q + (r >> 2)) * P::BN * 2 + (((wn0 / 16) ^ f) * 32) + (r & 3) * 8);
    } else {
      w = o.w;
    }
  }
  __device__ __forceinline__ bf16x8 read_x(const char* xs, int j, int kk) const {
    return *(const bf16x8*)(xs + (x ^ (kk ? 64u : 0u)) + j * 2048);
  }
  __device__ __forceinline__ bf16x8 read_w(const char* ws, int i, int kk) const {
    if constexpr (!NN) return *(const bf16x8*)(ws + (w ^ (kk ? 64u : 0u)) + i * 2048);
    else {
      const char* at = ws + (w ^ static_cast<uint32_t>(i << 5)) + kk * 32 * P::BN * 2;
      const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)at);
      const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(at + 4 * P::BN * 2));
      return __builtin_bit_cast(bf16x8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
    }
  }
  // fragment f of k-step kk, in order of first use: a0, b0 .. b(NJ-1), a1 .. a(NI-1)
  __device__ __forceinline__ void read(Frags16<P>& d, int f, const char* xs, const char* ws, int kk) const {
    if (f == 0 || f > P::NJ) {
      const int ia = f == 0 ? 0 : f - P::NJ;
      d.a[ia] = read_w(ws, ia, kk);
    } else {
      d.b[f - 1] = read_x(xs, f - 1, kk);
    }
  }
};

// One stage: its MFMAs, the fragment reads of its second k-step and of the next stage's first, the copies of stage t + 2.
// (ws and ws2 are restrict: nothing copies into the W slots that are read here, and without the compiler's knowing so it
// waits for every copy in flight before each transposing read.)
template <class P, bool NN, bool TOUCH, class Op>
__device__ __forceinline__ void ring_stage(f32x4 (&acc)[P::NI][P::NJ], Frags16<P> (&fr)[2], const Op& op,
                                           const RingFrags<P, NN>& rf, const char* xs, const char* __restrict__ ws,
                                           const char* xs2, const char* __restrict__ ws2, char* xdst, char* wdst) {
  constexpr int NL = ring_loads<P>(), NB = P::NI * P::NJ, RS = NB / (P::NI + P::NJ), LS = NB / NL;
  static_assert(NB % (P::NI + P::NJ) == 0 && NB % NL == 0 && LS % 2 == 0 && RS >= 2, "bundle schedule");
  __builtin_amdgcn_sched_barrier(0);
#pragma unroll
  for (int m = 0; m < NB; ++m) {
    const int i = m / P::NJ, j = m % P::NJ;
    if constexpr (TOUCH) {
      if (i == 0) op.touch(fr[0].b[j], j);
    }
    acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fr[0].a[i], fr[0].b[j], acc[i][j], 0, 0, 0);
    // (twice as dense as those of the next stage: they have all come before the barrier waits for them; 1.5% at 4096 inputs)
    if (m % (RS / 2) == 0 && m / (RS / 2) < P::NI + P::NJ) rf.read(fr[1], m / (RS / 2), xs, ws, 1);
    if (m % LS == LS / 2) op.load_x(m / LS, xdst);
    __builtin_amdgcn_sched_barrier(0);
  }
#pragma unroll
  for (int m = 0; m < NB; ++m) {
    const int i = m / P::NJ, j = m % P::NJ;
    if constexpr (TOUCH) {
      if (i == 0) op.touch(fr[1].b[j], j);
    }
    acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fr[1].a[i], fr[1].b[j], acc[i][j], 0, 0, 0);
    if (m == 0) {
      __builtin_amdgcn_sched_barrier(0);
      __builtin_amdgcn_s_waitcnt(waitcnt_vm(NL));
      stage_barrier();  // stage t + 1 landed and visible; every wave is done reading stage t
    } else if (m % RS == 1) {
      rf.read(fr[0], m / RS, xs2, ws2, 0);
    }
    if (m % LS == LS / 2) op.load_w(m / LS, wdst);
    __builtin_amdgcn_sched_barrier(0);
  }
}

// The larger tile's accumulators fill the accumulation registers, all of them: what reads them behind the loop (an
// epilogue with more values of its own) else moves some to others within it.
template <class P>
__device__ __forceinline__ void keep_acc(f32x4 (&acc)[P::NI][P::NJ]) {
#if defined(__HIP_DEVICE_COMPILE__)
  if constexpr (P::BM == 256) {
#pragma unroll
    for (int i = 0; i < P::NI; ++i)
#pragma unroll
      for (int j = 0; j < P::NJ; ++j) asm volatile("" : "+a"(acc[i][j]));
  }
#endif
}

// The loop. Behind it the LDS is free (every copy has landed, every wave has read its last fragments). With SPLIT,
// op.between(acc) runs before stage `at` (0 < at; not at all where at >= NS).
// (Schedule as the hot GEMM's: x of stage t + 2 is copied beside k-step 0, W beside k-step 1, into the slots that the
// barriers of stages t - 1 and t release; the wait of stage t leaves the x copies of stage t + 2 in flight.)
template <class P, bool NN, bool SPLIT = false, bool TOUCH = false, class Op>
__device__ __forceinline__ void ring_run(f32x4 (&acc)[P::NI][P::NJ], Op& op, int NS, char* smem, int wm0, int wn0,
                                         int at = 0) {
  static_assert(P::WAVES == 4, "schedule written for 4 waves");
  constexpr int NL = ring_loads<P>();
#pragma unroll
  for (int i = 0; i < P::NI; ++i)
#pragma unroll
    for (int j = 0; j < P::NJ; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[i][j][e] = 0.f;
  if constexpr (TOUCH) op.fetch(0);
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    op.seek(s);
#pragma unroll
    for (int l = 0; l < NL; ++l) op.load_x(l, smem + 2 * s * P::SLOT_BYTES);
#pragma unroll
    for (int l = 0; l < NL; ++l) op.load_w(l, smem + (2 * s + 1) * P::SLOT_BYTES);
  }
  __builtin_amdgcn_s_waitcnt(waitcnt_vm(2 * NL));  // stage 0 landed
  stage_barrier();
  RingFrags<P, NN> rf;
  rf.init(wm0, wn0);
  Frags16<P> fr[2];
  int a = 0;  // slot of x of stage t
  int t = 0;
  auto after = [](int slot) { return slot == 4 ? 0 : slot + 1; };
  auto run = [&](int end) {
#pragma unroll
    for (int f = 0; f < P::NI + P::NJ; ++f)
      rf.read(fr[0], f, smem + a * P::SLOT_BYTES, smem + after(a) * P::SLOT_BYTES, 0);
    for (; t < end; ++t) {
      op.seek(t + 2);
      if constexpr (TOUCH) {
        op.next();
        op.fetch(t + 1);
      }
      const int b1 = after(a), a2 = after(b1), b2 = after(a2), a3 = after(b2);  // W of t; x, W of t + 1; x of t + 2
      ring_stage<P, NN, TOUCH>(acc, fr, op, rf, smem + a * P::SLOT_BYTES, smem + b1 * P::SLOT_BYTES, smem + a2 * P::SLOT_BYTES,
                        smem + b2 * P::SLOT_BYTES, smem + a3 * P::SLOT_BYTES, smem + a * P::SLOT_BYTES);
      a = a2;
    }
    keep_acc<P>(acc);
  };
  if constexpr (SPLIT) {
    if (at > 0 && at < NS) {
      run(at);
      op.between(acc);
    }
  }
  run(NS);
  __builtin_amdgcn_s_waitcnt(waitcnt_vm(0));
  __syncthreads();
}

// Tile L of mt x nt: m-tiles in groups of `group` over all n-tiles.
struct RingTile {
  int m, n;
  __device__ __forceinline__ RingTile(int L, int mt, int nt, int group) {
    const int gsize = group * nt;
    const int grp = L / gsize, first = grp * group;
    const int gm = min(group, mt - first), within = L - grp * gsize;
    m = first + within % gm;
    n = within / gm;
  }
};

// A workgroup's work: a whole tile, or part `unit` of the tiles behind the first `full`, stages [lo, hi) of it. A run of
// neighbours to each XCD.
struct RingWork {
  int tile, unit, lo, hi;
  __device__ __forceinline__ RingWork(int b, int full, int tiles, int S, int ks, int NS) {
    if (b < full) {
      tile = xcd_remap(b, full);
      unit = -1;
      lo = 0;
      hi = NS;
    } else {
      const int rem = tiles - full, r = xcd_remap(b - full, rem * S), z = r / rem;
      tile = full + r - z * rem;
      unit = (r - z * rem) * S + z;
      lo = z * ks;
      hi = min(NS, lo + ks);
    }
  }
};

// A part's sums as the registers hold them, [unit][wave][j][i][lane] of four, and the sum of a tile's parts in order for
// column block j (16 tokens) of a wave.
template <class P>
__device__ __forceinline__ f32x4* part_at(float* part, int unit, int j, int i, int other = 0) {  // (of wave + other)
  return reinterpret_cast<f32x4*>(part) +
         (((static_cast<int64_t>(unit) * P::WAVES + ring_wave() + other) * P::NJ + j) * P::NI + i) * 64;
}
template <class P>
__device__ __forceinline__ void put_part(const f32x4 (&acc)[P::NI][P::NJ], float* part, int unit) {
  const int lane = opaque_int(threadIdx.x & 63);
#pragma unroll
  for (int j = 0; j < P::NJ; ++j)
#pragma unroll
    for (int i = 0; i < P::NI; ++i) part_at<P>(part, unit, j, i)[lane] = acc[i][j];
}
template <class P>
__device__ __forceinline__ void sum_parts(f32x4 (&acc)[P::NI][1], float* part, int rem_tile, int S, int j, int other = 0) {
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int i = 0; i < P::NI; ++i) acc[i][0] = part_at<P>(part, rem_tile * S, j, i, other)[lane];
  for (int z = 1; z < S; ++z)
#pragma unroll
    for (int i = 0; i < P::NI; ++i) acc[i][0] += part_at<P>(part, rem_tile * S + z, j, i, other)[lane];
}

// The kernel's first argument read again, for what comes behind the loop: its fields are then not kept in scalar registers
// (and, where those run out, in vector ones) through it.
template <class A>
__device__ __forceinline__ A late_args() {
  A v;
#if defined(__HIP_DEVICE_COMPILE__)
  auto* at = __builtin_amdgcn_kernarg_segment_ptr();
  asm volatile("" : "+s"(at));
  __builtin_memcpy(&v, (const void*)at, sizeof(A));
#endif
  return v;
}

// bf16 outputs of a wave's block through LDS: `put` 4 consecutive columns of a row, then `store` the block as whole
// rows of 16-byte pieces. COLS columns, 16-byte chunks XOR-swizzled by row.
template <int ROWS, int COLS>
struct BlockOut {
  static constexpr int RBY = COLS * 2, CH = RBY / 16, RPL = 256 / RBY > 0 ? 256 / RBY : 1;
  char* st;  // ROWS * RBY bytes of this wave's own
  __device__ __forceinline__ static int at(int row, int chunk) {
    return row * RBY + ((chunk ^ ((row / RPL) & (CH - 1))) * 16);
  }
  __device__ __forceinline__ void put(int row, int col, uint32_t lo, uint32_t hi) const {
    *reinterpret_cast<uint2*>(st + at(row, col >> 3) + (col & 4) * 2) = uint2{lo, hi};
  }
  // rows [0, rows) and columns [0, cols) of the block exist; y is its first element
  __device__ __forceinline__ void store(bf16_bits* y, int64_t ldy, int rows, int cols) const {
    const int lane = threadIdx.x & 63, c = lane % CH, r0 = lane / CH;
    const bool wide = reinterpret_cast<uintptr_t>(y) % 16 == 0 && ldy % 8 == 0 && cols >= COLS;
#pragma unroll 4
    for (int it = 0; it < ROWS * CH / 64; ++it) {
      const int row = it * (64 / CH) + r0;
      const u32x4 v = *reinterpret_cast<const u32x4*>(st + at(row, c));
      if (row >= rows) continue;
      bf16_bits* dst = y + row * ldy + c * 8;
      if (wide) {
        __builtin_nontemporal_store(v, reinterpret_cast<u32x4*>(dst));
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (c * 8 + e < cols) dst[e] = static_cast<bf16_bits>(v[e >> 1] >> (16 * (e & 1)));
      }
    }
  }
};

}  // namespace pipe
}  // namespace
}  // namespace lora
