// Device code that the pipelined kernels share: tiles copied global -> LDS by buffer_load ... lds into rings of
// stages, their swizzles, fragment reads, waits and the rank-wide producer's loop (gemm.hip, and the kernels of a
// training step built on the same rings). Everything sits in an unnamed namespace: each source keeps its own copy.
#pragma once

#include "common.hpp"

namespace lora {
namespace {

typedef __attribute__((address_space(3))) void lds_void;

// Physical workgroup ids are dealt round-robin to the 8 XCDs. Remap so each XCD
// receives a contiguous run of logical tiles (tiles sharing x rows / W rows then
// share that XCD's L2).
__device__ __forceinline__ int xcd_remap(int pid, int G) {
  const int q = G / 8, rem = G % 8;
  const int xcd = pid % 8, idx = pid / 8;
  return (xcd < rem) ? xcd * (q + 1) + idx : rem * (q + 1) + (xcd - rem) * q + idx;
}

namespace pipe {

template <int BM_, int BN_, int WM_, int WN_, int RB_, int S_>
struct PCfg {
  static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_, RB = RB_, S = S_;
  static constexpr int WAVES_M = BM / WM, WAVES_N = BN / WN, WAVES = WAVES_M * WAVES_N;
  static constexpr int THREADS = 64 * WAVES;
  static constexpr int NI = WN / 32, NJ = WM / 32;
  static constexpr int CPR = RB / 16;      // 16-byte chunks per staged row
  static constexpr int RPL = 256 / RB;     // staged rows per 256-byte line of the 64 LDS banks
  static constexpr int KK = RB / 32;       // 16-k MFMA steps per stage
  static constexpr int X_BYTES = BM * RB, STAGE_BYTES = (BM + BN) * RB;
  static constexpr int LPS = (BM + BN) * CPR / THREADS;  // buffer loads per thread per stage
  static constexpr int GROUP_M = 4;
  static_assert(KK % 2 == 0, "fragment sets alternate across stages");
  static_assert((BM * CPR / 64) % WAVES == 0 && (BN * CPR / 64) % WAVES == 0, "uneven load split");
  static_assert(S * STAGE_BYTES <= 160 * 1024, "LDS");
  static_assert((S - 2) * LPS <= 63, "vmcnt range");
};

// Chunk index XORed with (row / RPL) % CPR: the 16-byte reads of 16 consecutive
// rows at one chunk (one quarter of a wave's ds_read_b128) hit distinct banks.
template <class P>
__device__ __forceinline__ int swz(int row, int chunk) {
  return row * P::CPR + (chunk ^ ((row / P::RPL) % P::CPR));
}

// Tile rows [row_lo, row_hi) come from source row (row + shift), bytes
// [kb0, kb0 + RB) of it; other rows and bytes >= kb_valid read as zero.
template <class P, int ROWS>
__device__ __forceinline__ void dma(char* lds, __amdgpu_buffer_rsrc_t rsrc, uint32_t ld_bytes, int row_lo,
                                    int row_hi, int shift, int kb0, int kb_valid) {
  constexpr int INSTR = ROWS * P::CPR / 64;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
  for (int it = 0; it < INSTR / P::WAVES; ++it) {
    const int slot0 = (it * P::WAVES + wave) * 64;  // wave-uniform LDS destination
    const int sl = slot0 + lane;
    const int row = sl / P::CPR;
    const int c = (sl % P::CPR) ^ ((row / P::RPL) % P::CPR);
    const int kb = kb0 + c * 16;
    const uint32_t voff = (row >= row_lo && row < row_hi && kb < kb_valid)
                              ? static_cast<uint32_t>(row + shift) * ld_bytes + static_cast<uint32_t>(kb)
                              : 0x80000000u;
    __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc, (lds_void*)(lds + slot0 * 16), 16, voff, 0, 0, 0);
  }
}

template <class P>
struct Frags {
  bf16x8 a[P::NI], b[P::NJ];
};

template <class P>
__device__ __forceinline__ void load_frags(Frags<P>& f, const char* stage, int kk, int wn0, int wm0, int lane) {
  const int r = lane & 31, h = lane >> 5;
  const char* lx = stage;
  const char* lw = stage + P::X_BYTES;
#pragma unroll
  for (int i = 0; i < P::NI; ++i) f.a[i] = *(const bf16x8*)(lw + swz<P>(wn0 + i * 32 + r, kk * 2 + h) * 16);
#pragma unroll
  for (int j = 0; j < P::NJ; ++j) f.b[j] = *(const bf16x8*)(lx + swz<P>(wm0 + j * 32 + r, kk * 2 + h) * 16);
}

template <class P>
__device__ __forceinline__ void mfma_frags(f32x16 (&acc)[P::NI][P::NJ], const Frags<P>& f) {
#pragma unroll
  for (int i = 0; i < P::NI; ++i)
#pragma unroll
    for (int j = 0; j < P::NJ; ++j)
      acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(f.a[i], f.b[j], acc[i][j], 0, 0, 0);
}

// Scheduling hint for a block "NI + NJ fragment reads + NI * NJ MFMAs": the reads
// go out two at a time behind the first MFMAs and complete while the rest run.
template <class P>
__device__ __forceinline__ void interleave_reads_with_mfma() {
  constexpr int R = P::NI + P::NJ, M = P::NI * P::NJ;
#pragma unroll
  for (int i = 0; i < R / 2; ++i) {
    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);  // 1 MFMA
    __builtin_amdgcn_sched_group_barrier(0x100, 2, 0);  // 2 DS reads
  }
  __builtin_amdgcn_sched_group_barrier(0x008, M - R / 2, 0);
}

// Cache-policy operand of the buffer intrinsics on gfx950: bit 1 = nt (streaming).
constexpr int kCachePolicyNT = 2;

// s_waitcnt immediates (gfx9 encoding: vmcnt[3:0] bits 3:0, expcnt bits 6:4,
// lgkmcnt bits 11:8, vmcnt[5:4] bits 15:14); counters not named stay at their
// maximum, i.e. are not waited for. Using the builtin (not inline asm) lets the
// compiler's own wait insertion see these waits.
constexpr int waitcnt_vm(int n) { return (n & 0xf) | ((n >> 4) << 14) | 0x70 | 0xf00; }
constexpr int kWaitLgkm0 = 0xc07f;

// Wait until at most `n` stages of this thread's buffer loads are outstanding.
template <int LPS>
__device__ __forceinline__ void wait_stages(int n) {
  if (n >= 4) __builtin_amdgcn_s_waitcnt(waitcnt_vm(4 * LPS > 63 ? 63 : 4 * LPS));
  else if (n == 3) __builtin_amdgcn_s_waitcnt(waitcnt_vm(3 * LPS > 63 ? 63 : 3 * LPS));
  else if (n == 2) __builtin_amdgcn_s_waitcnt(waitcnt_vm(2 * LPS));
  else if (n == 1) __builtin_amdgcn_s_waitcnt(waitcnt_vm(LPS));
  else __builtin_amdgcn_s_waitcnt(waitcnt_vm(0));
}

// Workgroup barrier without the release/acquire fences of __syncthreads (those
// would also wait for the loads of later stages). LDS reads of this wave are
// complete before it arrives.
__device__ __forceinline__ void stage_barrier() {
  __builtin_amdgcn_s_waitcnt(kWaitLgkm0);
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// v unchanged, through an empty asm: values computed from it stay where they
// are written instead of being hoisted out of loops into long-lived registers.
// (The asm exists only in the device pass; the host pass has no such operand.)
__device__ __forceinline__ int opaque_int(int v) {
#if defined(__HIP_DEVICE_COMPILE__)
  asm volatile("" : "+v"(v));
#endif
  return v;
}

// Per-lane byte offsets of one operand tile's rows for the buffer_load ... lds
// copies (k offset 0); rows outside [row_lo, row_hi) get an offset past the
// resource range. The k offset of a stage travels in the scalar soffset.
template <class P, int ROWS>
struct TileOffsets {
  static constexpr int N = ROWS * P::CPR / 64 / P::WAVES;
  uint32_t v[N];
  __device__ __forceinline__ void init(uint32_t ld_bytes, int row_lo, int row_hi, int shift) {
    const int lane = opaque_int(threadIdx.x & 63);
    const int wave = threadIdx.x >> 6;
#pragma unroll
    for (int it = 0; it < N; ++it) {
      const int sl = (it * P::WAVES + wave) * 64 + lane;
      const int row = sl / P::CPR;
      const int c = (sl % P::CPR) ^ ((row / P::RPL) % P::CPR);
      v[it] = (row >= row_lo && row < row_hi) ? static_cast<uint32_t>(row + shift) * ld_bytes + c * 16
                                              : 0x80000000u;
    }
  }
  // One of the N copy instructions of a stage (no K tail).
  __device__ __forceinline__ void load_one(int it, char* lds, __amdgpu_buffer_rsrc_t rsrc, int kb0) const {
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int slot0 = (it * P::WAVES + wave) * 64;
    __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc, (lds_void*)(lds + slot0 * 16), 16, v[it], kb0, 0, 0);
  }
  // Copy the stage at byte offset kb0 into lds. With a K tail, chunks at or past
  // kb_valid are redirected out of range as well.
  __device__ __forceinline__ void load(char* lds, __amdgpu_buffer_rsrc_t rsrc, int kb0, bool tail, int kb_valid) const {
    const int lane = opaque_int(threadIdx.x & 63);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    // When each copy instruction covers a whole number of swizzle periods of rows
    // the lane's chunk is the same in all of them.
    constexpr bool same_chunk = (P::WAVES * 64 / P::CPR / P::RPL) % P::CPR == 0;
    const int c0 = (lane % P::CPR) ^ (((wave * 64 + lane) / P::CPR / P::RPL) % P::CPR);
#pragma unroll
    for (int it = 0; it < N; ++it) {
      const int slot0 = (it * P::WAVES + wave) * 64;
      uint32_t voff = v[it];
      if (tail) {
        int c = c0;
        if (!same_chunk) {
          const int sl = slot0 + lane;
          const int row = sl / P::CPR;
          c = (sl % P::CPR) ^ ((row / P::RPL) % P::CPR);
        }
        if (kb0 + c * 16 >= kb_valid) voff = 0x80000000u;
      }
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc, (lds_void*)(lds + slot0 * 16), 16, voff, kb0, 0, 0);
    }
  }
};

// One copy instruction `it` of a staged tile whose rows come from source row
// (row + shift) for rows in [row_lo, row_hi), bytes [kb0, kb_valid); other
// lanes read as zero (K-extension units: t~ rows and LoRA B rows).
template <class P, int ROWS>
__device__ __forceinline__ void dma_one(int it, char* lds, __amdgpu_buffer_rsrc_t rsrc, uint32_t ld_bytes,
                                        int row_lo, int row_hi, int shift, int kb0, int kb_valid) {
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int slot0 = (it * P::WAVES + wave) * 64;
  const int sl = slot0 + lane;
  const int row = sl / P::CPR;
  const int c = (sl % P::CPR) ^ ((row / P::RPL) % P::CPR);
  const int kb = kb0 + c * 16;
  const uint32_t voff = (row >= row_lo && row < row_hi && kb < kb_valid)
                            ? static_cast<uint32_t>(row + shift) * ld_bytes + static_cast<uint32_t>(kb)
                            : 0x80000000u;
  __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc, (lds_void*)(lds + slot0 * 16), 16, voff, 0, 0, 0);
}

// ---------------------------------------------------------------------------
// The hot kernel on v_mfma_f32_16x16x32_bf16: 256 x 256 tile, 4 waves of
// 128 x 128; the x part and the W part of a 64-k stage are separate units of a
// ring of five 32 KB LDS slots (unit 2s = x rows of stage s, 2s + 1 = W rows,
// slot = unit mod 5), 128-byte rows; each wave holds 8 x 8 blocks of 16 x 16
// (4 accumulators per lane each) and a 64-k stage is two 32-k steps of 64 MFMAs.
// Under a sustained MFMA load this instruction runs at a clearly higher clock
// than the 32 x 32 x 16 one for the same work per cycle (measured on MI355X:
// about 2.05 against 1.77 GHz with LDS operand reads), which is where the
// kernel's throughput is decided once the copies are hidden.
template <int BM_, int BN_, int WM_, int WN_, int RB_, int SLOTS_, int OCC_ = 1>
struct QCfg {
  static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_, RB = RB_, SLOTS = SLOTS_;
  static constexpr int OCC = OCC_;                    // workgroups resident per CU (waves per SIMD)
  static constexpr int WAVES_M = BM / WM, WAVES_N = BN / WN, WAVES = WAVES_M * WAVES_N;
  static constexpr int THREADS = 64 * WAVES;
  static constexpr int NI = WN / 16, NJ = WM / 16;   // 16 x 16 blocks per wave
  static constexpr int CPR = RB / 16, RPL = 256 / RB;
  static constexpr int KK = RB / 64;                  // 32-k MFMA steps per stage
  static constexpr int SLOT_BYTES = BM * RB;
  static constexpr int GROUP_M = 4;
  static_assert(BM == BN && RB == 128 && KK == 2, "x and W units share one slot size; two k-steps per stage");
  static_assert((BM * CPR / 64) % WAVES == 0, "uneven load split");
  static_assert(SLOTS == 5 && OCC * SLOTS * SLOT_BYTES <= 160 * 1024, "LDS");
};

template <class P>
struct Frags16 {
  bf16x8 a[P::NI], b[P::NJ];
};

// Operand fragments of 32-k step kk: lane (r = lane % 16, q = lane / 16) holds
// k = 8q .. 8q + 7 of row r of each 16-row block, i.e. 16-byte chunk 4 kk + q.
// With 128-byte rows the swizzle term (row / 2) % 8 is the same for every
// 16-row block, so block i sits at a fixed 2048-byte offset from the lane's
// block-0 address, and k-step 1 is k-step 0's address with byte bit 6 flipped.
struct FragOffsets {
  uint32_t x, w;  // byte offsets of this lane's k-step-0 chunk in block 0 of an x / W slot
};

template <class P>
__device__ __forceinline__ FragOffsets frag_offsets(int wn0, int wm0, int lane) {
  const int r = lane & 15, q = lane >> 4;
  const int c = q ^ ((r >> 1) & 7);
  return FragOffsets{static_cast<uint32_t>(((wm0 + r) * P::CPR + c) * 16),
                     static_cast<uint32_t>(((wn0 + r) * P::CPR + c) * 16)};
}

template <class P>
__device__ __forceinline__ void ring_frags16(Frags16<P>& f, const char* xs, const char* ws, int kk,
                                             FragOffsets o) {
  const uint32_t flip = kk ? 64u : 0u;
#pragma unroll
  for (int i = 0; i < P::NI; ++i) f.a[i] = *(const bf16x8*)(ws + (o.w ^ flip) + i * 2048);
#pragma unroll
  for (int j = 0; j < P::NJ; ++j) f.b[j] = *(const bf16x8*)(xs + (o.x ^ flip) + j * 2048);
}

template <class P>
__device__ __forceinline__ void mfma_frags16(f32x4 (&acc)[P::NI][P::NJ], const Frags16<P>& f) {
#pragma unroll
  for (int i = 0; i < P::NI; ++i)
#pragma unroll
    for (int j = 0; j < P::NJ; ++j)
      acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(f.a[i], f.b[j], acc[i][j], 0, 0, 0);
}

// A staged 16-byte chunk with its two 8-byte halves back in column order (swapped when sw).
__device__ __forceinline__ u32x4 unswap_halves(u32x4 v, int sw) {
  return sw ? u32x4{v[2], v[3], v[0], v[1]} : v;
}

struct NoTouch {
  template <class F>
  __device__ __forceinline__ void operator()(F&, int, int) const {}
};

// One pipelined K loop over NS stages for config P; issue(s) fills ring slot s % S. touch(f, s, kk) may change the
// fragments of k-step kk of stage s before they are multiplied.
template <class P, class Issue, class Touch = NoTouch>
__device__ __forceinline__ void pipe_loop(f32x16 (&acc)[P::NI][P::NJ], char* smem, int NS, Issue&& issue,
                                          int wn0, int wm0, int lane, Touch touch = Touch{}) {
#pragma unroll
  for (int i = 0; i < P::NI; ++i)
#pragma unroll
    for (int j = 0; j < P::NJ; ++j)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.f;
  for (int s = 0; s < P::S && s < NS; ++s) issue(s);
  wait_stages<P::LPS>(min(NS, P::S) - 1);
  stage_barrier();
  Frags<P> fr[2];
  load_frags<P>(fr[0], smem, 0, wn0, wm0, lane);
  auto run_stage = [&](int j, bool steady) {
    const char* st = smem + (j % P::S) * P::STAGE_BYTES;
#pragma unroll
    for (int kk = 0; kk < P::KK; ++kk) {
      if (kk + 1 < P::KK) {
        load_frags<P>(fr[(kk + 1) & 1], st, kk + 1, wn0, wm0, lane);
      } else {
        if (steady) wait_stages<P::LPS>(P::S - 2);
        else wait_stages<P::LPS>(min(NS - j - 2, P::S - 2));
        stage_barrier();
        if (steady) issue(j + P::S);
        load_frags<P>(fr[(kk + 1) & 1], smem + ((j + 1) % P::S) * P::STAGE_BYTES, 0, wn0, wm0, lane);
      }
      touch(fr[kk & 1], j, kk);
      mfma_frags<P>(acc, fr[kk & 1]);
      interleave_reads_with_mfma<P>();
    }
  };
  int j = 0;
  for (; j + P::S < NS; ++j) run_stage(j, true);
  for (; j + 1 < NS; ++j) run_stage(j, false);
  const char* st = smem + ((NS - 1) % P::S) * P::STAGE_BYTES;
#pragma unroll
  for (int kk = 0; kk < P::KK; ++kk) {
    if (kk + 1 < P::KK) load_frags<P>(fr[(kk + 1) & 1], st, kk + 1, wn0, wm0, lane);
    touch(fr[kk & 1], NS - 1, kk);
    mfma_frags<P>(acc, fr[kk & 1]);
  }
}

}  // namespace pipe
}  // namespace
}  // namespace lora
