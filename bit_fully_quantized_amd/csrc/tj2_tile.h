// Tile product of two row-major operands along their contiguous axis, shared by
// the MXFP4 products (mx.hip) and the head's cross entropy (loss.hip):
//
//   D[q, p] = sum_k Q[q, k] P[p, k]
//
// for bf16 operands (v_mfma_f32_16x16x32_bf16) or MXFP4 operands (E2M1 codes
// with one power-of-two scale per 32; v_mfma_scale_f32_16x16x128_f8f6f4 applies
// the scales itself).  Both instructions take 16 bytes of each operand per lane
// and run in 16 cycles, so one loop serves both: a chunk is 128 bytes of every
// row (64 bf16 or 256 E2M1), two instruction steps.
//
// Work of a workgroup: BM = 16 WM TM rows of P by BN = 16 WN TN rows of Q; wave
// (wm, wn) owns 16 TM by 16 TN of it in registers.  P is the side whose rows are
// contiguous in the output, so a lane's four results of one instruction lie next
// to each other in memory.  Which 16 rows make up an instruction tile is free, so
// the rows are dealt out such that the results of PB = min(TM, 4) tiles are 4 PB
// neighbours in one lane (16-byte stores, whole lines over a wave), and such that
// lane n's TN tiles are TN neighbouring rows of Q.
//
// LDS: two stages of (BM + BN) rows of 128 bytes, filled by buffer loads straight
// into LDS (no registers, and out-of-range lanes read zero: rows past the
// operand's end and 16-byte pieces past the row's end get an offset beyond the
// buffer's size).  Such a load writes lane after lane, so a row's eight pieces
// are permuted by permuting what each lane fetches: piece g of row r sits in slot
// g ^ key(r), with key so chosen that 8 lanes reading the same piece of their
// tile's rows touch all 32 banks once.
//
// One barrier a chunk, placed between its two steps: the loads of the next chunk
// were issued a whole chunk earlier and must have landed, every wave has read
// this chunk's last fragments (so its stage may be refilled), and the second
// step's instructions cover the reads of the next chunk's first fragments.
#pragma once
#include "tj2_device.h"
#include "tj2_internal.h"

namespace tj2 {

typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));
typedef int i32x4_t __attribute__((ext_vector_type(4)));
typedef int i32x8_t __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2v_t __attribute__((ext_vector_type(2)));
typedef float f32x2v_t __attribute__((ext_vector_type(2)));

enum { EL_BF16 = 0, EL_MX = 1 };

// Two fp32 values rounded to the nearest even bf16, a in the low half.
__device__ __forceinline__ uint32_t bf16_pair(float a, float b) {
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2v_t{a, b}, bf16x2v_t));
}

// An operand of a tile product: rows of `kb` bytes (a multiple of 16) at a pitch
// of `ld` bytes; MXFP4: `sb` scale bytes (a multiple of 4) per row at a pitch of
// `lds` bytes.
struct TileOp {
  const uint8_t* p;
  const uint8_t* s;
  int64_t rows, ld, lds;
  int32_t kb, sb;
};

constexpr uint32_t kOutside = 0x80000000u;  // lane offset beyond every buffer below

// Raw buffer at `base` (same for all lanes) of 2^31 - 1 bytes: lane offsets of
// kOutside and above read zero; the others are the caller's to keep in range.
__device__ __forceinline__ u32x4_t raw_buffer(const uint8_t* base) {
  const uint64_t a = (uint64_t)(uintptr_t)base;
  u32x4_t d;
  d.x = __builtin_amdgcn_readfirstlane((uint32_t)a);
  d.y = __builtin_amdgcn_readfirstlane((uint32_t)(a >> 32) & 0xFFFFu);
  d.z = 0x7FFFFFFFu;
  d.w = 0x00020000u;
  return d;
}

// Descriptors written by vector instructions (readfirstlane) may be read by a
// load five cycles later at the earliest; the loads below are assembly, which the
// compiler does not pad.
__device__ __forceinline__ void settle(u32x4_t& a, u32x4_t& b) { asm volatile("s_nop 4" : "+s"(a), "+s"(b)); }

// 16 (or 4) bytes per lane from buffer d at lane offset v into LDS at byte
// address m (of the wave's first lane), lane after lane.  In assembly because
// the compiler's own form waits for every such load before the next LDS read;
// here the chunk's barrier carries the wait.  m0, which holds the LDS address, is
// left changed: nothing else in these kernels reads it.
__device__ __forceinline__ void load_lds16(u32x4_t d, uint32_t v, uint32_t m) {
  asm volatile(
      "s_mov_b32 m0, %2\n\t"
      "s_nop 0\n\t"
      "buffer_load_dwordx4 %0, %1, 0 offen lds"
      :
      : "v"(v), "s"(d), "s"(m)
      : "memory");
}
__device__ __forceinline__ void load_lds4(u32x4_t d, uint32_t v, uint32_t m) {
  asm volatile(
      "s_mov_b32 m0, %2\n\t"
      "s_nop 0\n\t"
      "buffer_load_dword %0, %1, 0 offen lds"
      :
      : "v"(v), "s"(d), "s"(m)
      : "memory");
}

__device__ __forceinline__ uint32_t lds_address(const void* p) {
  return (uint32_t)(uintptr_t)(const __attribute__((address_space(3))) char*)p;
}

template <class T>
__device__ __forceinline__ T lds_read(uint32_t a) {
  return *reinterpret_cast<const __attribute__((address_space(3))) T*>(a);
}

// All of this wave's loads (those into LDS too) and LDS accesses are done, then
// the workgroup's barrier.
__device__ __forceinline__ void tile_barrier() {
  asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
}

template <int EL, int WM, int WN, int TM, int TN>
struct Tile {
  static constexpr int kWN = WN, kTM = TM, kTN = TN;
  static constexpr int NT = 64 * WM * WN;           // threads
  static constexpr int BM = 16 * WM * TM, BN = 16 * WN * TN;
  static constexpr int ROWS = BM + BN;
  static constexpr int PB = TM < 4 ? TM : 4;        // tiles whose rows interleave
  static constexpr int RPI = NT / 8;                // rows one load instruction of all threads covers
  static constexpr int LP = BM / RPI, LQ = BN / RPI;
  static constexpr int SCALE_DW = EL == EL_MX ? ROWS * 2 : 0;  // scale words of a chunk
  static_assert(BM % RPI == 0 && BN % RPI == 0, "whole load instructions");
  static_assert(8 * PB <= RPI && 8 * TN <= RPI, "a thread's key is the same in all its rows");
  static_assert(TM % PB == 0, "whole row blocks");

  struct Smem {
    uint8_t stage[2][ROWS * 128];
    uint32_t scale[2][EL == EL_MX ? SCALE_DW : 1];
  };

  typedef float4_t Acc[TM][TN];

  // row of the wave's P rows that lane quad g (0..3), result r (0..3) of tile tm holds
  static __device__ __forceinline__ constexpr int p_row(int tm, int g, int r) {
    return (tm / PB) * 16 * PB + g * 4 * PB + (tm % PB) * 4 + r;
  }
  // row of the wave's Q rows that lane n (0..15) of tile tn holds
  static __device__ __forceinline__ constexpr int q_row(int tn, int n) { return n * TN + tn; }
  static __device__ __forceinline__ constexpr int p_key(int row) { return (row & 3) | (((row / (4 * PB)) & 1) << 2); }
  static __device__ __forceinline__ constexpr int q_key(int row) { return (row / TN) & 7; }

  // Chunks [c0, c1) of the product of P rows p0.. and Q rows q0.., added to acc.
  // Every thread of the workgroup calls it with the same arguments.
  static __device__ __forceinline__ void run(const TileOp& P, int64_t p0, const TileOp& Q, int64_t q0, int c0, int c1,
                                             Smem& sm, Acc& acc) {
    const int t = threadIdx.x, lane = t & 63, w = __builtin_amdgcn_readfirstlane(t >> 6);
    const int wm = w / WN, wn = w % WN, n = lane & 15, g = lane >> 4;

    // what this thread loads: row i * RPI + t / 8, slot t % 8
    const int lr = t >> 3;
    const int np = (int)min(P.rows - p0, (int64_t)BM), nq = (int)min(Q.rows - q0, (int64_t)BN);
    const uint32_t gp = (uint32_t)((t & 7) ^ p_key(lr)) * 16, gq = (uint32_t)((t & 7) ^ q_key(lr)) * 16;
    uint32_t vp[LP], vq[LQ];
#pragma unroll
    for (int i = 0; i < LP; ++i) vp[i] = i * RPI + lr < np ? (uint32_t)(i * RPI + lr) * (uint32_t)P.ld + gp : kOutside;
#pragma unroll
    for (int i = 0; i < LQ; ++i) vq[i] = i * RPI + lr < nq ? (uint32_t)(i * RPI + lr) * (uint32_t)Q.ld + gq : kOutside;
    const uint8_t* pb = P.p + p0 * P.ld;
    const uint8_t* qb = Q.p + q0 * Q.ld;
    const uint32_t lds_w = lds_address(sm.stage[0]) + (uint32_t)w * 1024u;
    constexpr uint32_t kStage = ROWS * 128;

    // scales: [row][2] words of a chunk, a wave 32 rows at a time (all of P or all
    // of Q: BM is a multiple of 32)
    constexpr int SJ = EL == EL_MX ? SCALE_DW / NT : 1;
    static_assert(SCALE_DW % NT == 0 && BM % 32 == 0, "whole scale loads");
    uint32_t vs[SJ];
    if constexpr (EL == EL_MX) {
#pragma unroll
      for (int j = 0; j < SJ; ++j) {
        const int r0 = w * 32 + j * (NT / 2), r = r0 + (lane >> 1);
        const bool isp = r0 < BM;
        const uint32_t pitch = (uint32_t)(isp ? P.lds : Q.lds);
        vs[j] = (isp ? r < np : r - BM < nq) ? (uint32_t)(isp ? r : r - BM) * pitch + (lane & 1) * 4 : kOutside;
      }
    }

    auto load = [&](int c, uint32_t stage) __attribute__((always_inline)) {
      const uint32_t at = (uint32_t)c * 128u;
      u32x4_t dp = raw_buffer(pb + at), dq = raw_buffer(qb + at);
      settle(dp, dq);
      const uint32_t badp = at + gp >= (uint32_t)P.kb ? kOutside : 0u;
      const uint32_t badq = at + gq >= (uint32_t)Q.kb ? kOutside : 0u;
      const uint32_t dst = lds_w + stage * kStage;
#pragma unroll
      for (int i = 0; i < LP; ++i) load_lds16(dp, vp[i] | badp, dst + i * (RPI * 128));
#pragma unroll
      for (int i = 0; i < LQ; ++i) load_lds16(dq, vq[i] | badq, dst + (LP + i) * (RPI * 128));
      if constexpr (EL == EL_MX) {
        const uint32_t ats = (uint32_t)c * 8u;
        u32x4_t sp = raw_buffer(P.s + p0 * P.lds + ats), sq = raw_buffer(Q.s + q0 * Q.lds + ats);
        settle(sp, sq);
        const uint32_t bad = ats + (lane & 1) * 4 >= (uint32_t)P.sb ? kOutside : 0u;
        const uint32_t sd = lds_address(sm.scale[0]) + stage * (SCALE_DW * 4) + (uint32_t)w * 256u;
#pragma unroll
        for (int j = 0; j < SJ; ++j) {
          const bool isp = w * 32 + j * (NT / 2) < BM;
          u32x4_t d;
          d.x = isp ? sp.x : sq.x;
          d.y = isp ? sp.y : sq.y;
          d.z = sp.z;
          d.w = sp.w;
          load_lds4(d, vs[j] | bad, sd + j * (NT * 4));
        }
      }
    };

    // Fragments of step s of a chunk: piece 2 g + s of the lane's rows.  P's are
    // kept once: those of the next step are read into a tile's registers as soon
    // as its instructions have issued.  Q's, which every tile needs, twice.
    i32x4_t fp[TM], fq[2][TN];
    uint32_t sp[TM], sq[TN], sqn[TN];
    const int pr0 = wm * TM * 16, qr0 = BM + wn * TN * 16;
    const int pk = p_key((n >> 2) * 4 * PB + (n & 3)), qk = q_key(n * TN);
    // LDS byte addresses; the two steps' pieces are neighbours, 16 bytes apart
    const uint32_t lp = lds_address(sm.stage[0]) + (uint32_t)(pr0 + p_row(0, n >> 2, n & 3)) * 128u + ((2 * g) ^ pk) * 16;
    const uint32_t lq = lds_address(sm.stage[0]) + (uint32_t)(qr0 + q_row(0, n)) * 128u + ((2 * g) ^ qk) * 16;
    const uint32_t lsp = lds_address(sm.scale[0]) + (uint32_t)(pr0 + p_row(0, n >> 2, n & 3)) * 8u + 2 * g;
    const uint32_t lsq = lds_address(sm.scale[0]) + (uint32_t)(qr0 + q_row(0, n)) * 8u + 2 * g;
    auto read_p = [&](uint32_t stage, int s, int tm) __attribute__((always_inline)) {
      fp[tm] = lds_read<i32x4_t>(((lp ^ (s * 16)) + stage * kStage) + p_row(tm, 0, 0) * 128);
    };
    auto read_q = [&](uint32_t stage, int s, int tn) __attribute__((always_inline)) {
      fq[s][tn] = lds_read<i32x4_t>(((lq ^ (s * 16)) + stage * kStage) + q_row(tn, 0) * 128);
    };
    auto read_sp = [&](uint32_t stage, int tm) __attribute__((always_inline)) {
      if constexpr (EL == EL_MX) sp[tm] = lds_read<uint16_t>(lsp + stage * (SCALE_DW * 4) + p_row(tm, 0, 0) * 8);
    };
    auto read_sq = [&](uint32_t stage, int tn) __attribute__((always_inline)) {
      if constexpr (EL == EL_MX) sqn[tn] = lds_read<uint16_t>(lsq + stage * (SCALE_DW * 4) + q_row(tn, 0) * 8);
    };
    auto mma = [&](auto sc, int tm) __attribute__((always_inline)) {
      constexpr int s = decltype(sc)::value;
#pragma unroll
      for (int tn = 0; tn < TN; ++tn) {
        if constexpr (EL == EL_BF16) {
          acc[tm][tn] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, fp[tm]),
                                                                __builtin_bit_cast(bf16x8_t, fq[s][tn]), acc[tm][tn], 0, 0, 0);
        } else {
          const i32x8_t a = __builtin_shufflevector(fp[tm], i32x4_t{0, 0, 0, 0}, 0, 1, 2, 3, 4, 5, 6, 7);
          const i32x8_t b = __builtin_shufflevector(fq[s][tn], i32x4_t{0, 0, 0, 0}, 0, 1, 2, 3, 4, 5, 6, 7);
          acc[tm][tn] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, acc[tm][tn], 4, 4, s, (int)sp[tm], s, (int)sq[tn]);
        }
      }
    };
    using S0 = std::integral_constant<int, 0>;
    using S1 = std::integral_constant<int, 1>;
    // the tiles of the second step before which the barrier is crossed
    constexpr int LEAD = TM >= 4 ? 2 : 1;
    load(c0, 0);
    tile_barrier();
    load(c0 + 1, 1);
#pragma unroll
    for (int tn = 0; tn < TN; ++tn) {
      read_q(0, 0, tn);
      read_sq(0, tn);
    }
#pragma unroll
    for (int tm = 0; tm < TM; ++tm) {
      read_p(0, 0, tm);
      read_sp(0, tm);
    }
#pragma unroll
    for (int tn = 0; tn < TN; ++tn) sq[tn] = sqn[tn];
    // Every chunk runs the same straight line: past the last one the loads bring
    // zeros (or the next split's chunks) and the fragments read then are not used.
    uint32_t st = 0;
#pragma nounroll
    for (int c = c0; c < c1; ++c) {
#pragma unroll
      for (int tn = 0; tn < TN; ++tn) read_q(st, 1, tn);
#pragma unroll
      for (int tm = 0; tm < TM; ++tm) {
        mma(S0{}, tm);
        __builtin_amdgcn_sched_barrier(0);
        read_p(st, 1, tm);
      }
#pragma unroll
      for (int tm = 0; tm < TM; ++tm) {
        mma(S1{}, tm);
        __builtin_amdgcn_sched_barrier(0);
        if (tm == LEAD - 1) {
          tile_barrier();
          load(c + 2, st);
#pragma unroll
          for (int tn = 0; tn < TN; ++tn) {
            read_q(st ^ 1u, 0, tn);
            read_sq(st ^ 1u, tn);
          }
#pragma unroll
          for (int k = 0; k < LEAD; ++k) {
            read_p(st ^ 1u, 0, k);
            read_sp(st ^ 1u, k);
          }
        } else if (tm >= LEAD) {
          read_p(st ^ 1u, 0, tm);
          read_sp(st ^ 1u, tm);
        }
      }
      if constexpr (EL == EL_MX) {
#pragma unroll
        for (int tn = 0; tn < TN; ++tn) sq[tn] = sqn[tn];
      }
      st ^= 1u;
    }
    tile_barrier();  // nothing is in flight into LDS when the caller goes on
  }
};

// Tile number -> (tm, tn), XCD by XCD (workgroups go to the 8 XCDs in turn, each
// with its own L2): an XCD takes a contiguous range of the tiles, in groups of 8
// along the first axis, that axis fastest, so the tiles it runs at one time share
// few row blocks of both operands.
__device__ __forceinline__ void tile_of(uint32_t id, uint32_t nwg, uint32_t tiles_m, uint32_t tiles_n, uint32_t& tm,
                                        uint32_t& tn) {
  const uint32_t per = nwg / 8;
  if (id < per * 8) id = (id % 8) * per + id / 8;
  const uint32_t group = 8 * tiles_n, gi = id / group, first = gi * 8;
  const uint32_t rows = min(tiles_m - first, 8u), in = id - gi * group;
  tm = __builtin_amdgcn_readfirstlane(first + in % rows);
  tn = __builtin_amdgcn_readfirstlane(in / rows);
}

}  // namespace tj2
