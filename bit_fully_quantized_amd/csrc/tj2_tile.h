// Tile product of two row-major operands along their contiguous axis, shared by
// the MXFP4 and FP8 products (mx.hip, fp8.hip), the head's cross entropy (loss.hip)
// and the gated feed-forward block (ffn.hip):
//
//   D[q, p] = sum_k Q[q, k] P[p, k]
//
// for bf16 operands (v_mfma_f32_16x16x32_bf16) or MXFP4 operands (E2M1 codes
// with one power-of-two scale per 32; v_mfma_scale_f32_16x16x128_f8f6f4 applies
// the scales itself).  Both instructions take 16 bytes of each operand per lane
// and run in 16 cycles, so one loop serves both: a chunk is 128 bytes of every
// row (64 bf16 or 256 E2M1), two instruction steps.  FP8 operands (E4M3 codes, an
// fp32 scale per 128) have a loop of their own: a chunk is one instruction of 128
// elements, and its result is scaled as it is added to the sums.  That instruction keeps
// some 14 bits of what neighbouring products add to the largest of them (1.4e-5 of a
// result of normal operands, 1e-5 of the sum of magnitudes at most, measured), which is
// less than half a step of a bf16 result but not of an fp32 one: EL_FP8X and EL_FP8BX
// decode the codes to f16, which holds them, and use v_mfma_f32_16x16x32_f16 at half the
// rate, whose products are exact and whose sums are fp32.
//
// EL_PAIR: bf16, with P's rows taken from two matrices of the same shape in turn, so
// that a lane holds the results of a row of both (first: tiles 0 to PB - 1 of a wave's
// P rows, second: the next PB, ...); a tile then has BM / 2 rows of each.
//
// Workgroups go to the 8 XCDs in turn, each with its own L2, so an XCD takes a
// contiguous range of the tiles.
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
// g ^ key(r), with key so chosen that the lanes which a read serves together touch
// all 64 banks once.
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

// FP8B: P's scales are those of 128 rows; FP8X, FP8BX: the same with exact products
enum { EL_BF16 = 0, EL_MX = 1, EL_FP8 = 2, EL_FP8B = 3, EL_PAIR = 4, EL_FP8X = 5, EL_FP8BX = 6 };

// Two fp32 values rounded to the nearest even bf16, a in the low half.
__device__ __forceinline__ uint32_t bf16_pair(float a, float b) {
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2v_t{a, b}, bf16x2v_t));
}

// The values of 8 E4M3 codes, which f16 holds, the k-th of 32 in a and b.
__device__ __forceinline__ half8_t fp8_to_f16(i32x4_t a, i32x4_t b, int k) {
  half2_t h[4];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t u = (uint32_t)(k < 2 ? a : b)[k % 2 * 2 + i];
    h[2 * i] = __builtin_bit_cast(half2_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(u, 1.0f, false));
    h[2 * i + 1] = __builtin_bit_cast(half2_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(u, 1.0f, true));
  }
  return half8_t{h[0].x, h[0].y, h[1].x, h[1].y, h[2].x, h[2].y, h[3].x, h[3].y};
}

// An operand of a tile product: rows of `kb` bytes (a multiple of 16).  Row r's
// bytes [128 c, 128 c + 128) start at (r / 128) bs + (r % 128) ld + c cs:
//   row-major:  ld the pitch, cs 128, bs 128 ld;
//   blocked:    ld 128, cs the 16 KB of 128 rows' chunk, bs all chunks of 128 rows,
// the latter for operands that a pass of this library writes: a chunk of a tile is
// contiguous, where a long pitch spreads its rows over as many pages and, if it is a
// power of two, over few memory channels.  MXFP4: the scale bytes, one for 16 of codes,
// lie as the codes do.  FP8: the scale of row r (EL_FP8B's P: of rows r to r + 127) and
// chunk c lies at s + r srs (r / 128 srs) + c scs.
struct TileOp {
  const uint8_t* p;
  const uint8_t* s;
  int64_t rows, ld, bs;
  int32_t kb, cs;
  const uint8_t* p2;  // EL_PAIR: the second matrix
  int64_t srs, scs;
};

constexpr uint32_t kOutside = 0x80000000u;  // lane offset beyond every buffer below

// Raw buffer at `base` (same for all lanes) of 2^31 - 1 bytes: lane offsets of
// kOutside and above read zero (with or without the scalar offset, which is below
// 2^31); the others are the caller's to keep in range.
__device__ __forceinline__ u32x4_t raw_buffer(const uint8_t* base) {
  const uint64_t a = (uint64_t)(uintptr_t)base;
  u32x4_t d;
  d.x = __builtin_amdgcn_readfirstlane((uint32_t)a);
  d.y = __builtin_amdgcn_readfirstlane((uint32_t)(a >> 32) & 0xFFFFu);
  d.z = 0x7FFFFFFFu;
  d.w = 0x00020000u;
  return d;
}

// A value the same for all lanes, kept in a scalar register: the compiler would rather
// read a kernel argument again, in the middle of a loop and waiting for it.
__device__ __forceinline__ uint32_t pinned(uint32_t x) {
  x = __builtin_amdgcn_readfirstlane(x);
  asm volatile("" : "+s"(x));
  return x;
}

// Descriptors written by vector instructions (readfirstlane) may be read by a
// load five cycles later at the earliest; the loads below are assembly, which the
// compiler does not pad.
__device__ __forceinline__ void settle(u32x4_t& a, u32x4_t& b) { asm volatile("s_nop 4" : "+s"(a), "+s"(b)); }

// 16 (or 4) bytes per lane from buffer d at lane offset v + s into LDS at byte
// address m (of the wave's first lane), lane after lane.  In assembly because
// the compiler's own form waits for every such load before the next LDS read;
// here the chunk's barrier carries the wait.  m0, which holds the LDS address, is
// left changed: nothing else in these kernels reads it.
__device__ __forceinline__ void load_lds16(u32x4_t d, uint32_t v, uint32_t s, uint32_t m) {
  asm volatile(
      "s_mov_b32 m0, %3\n\t"
      "s_nop 0\n\t"
      "buffer_load_dwordx4 %0, %1, %2 offen lds"
      :
      : "v"(v), "s"(d), "s"(s), "s"(m)
      : "memory");
}
__device__ __forceinline__ void load_lds4(u32x4_t d, uint32_t v, uint32_t s, uint32_t m) {
  asm volatile(
      "s_mov_b32 m0, %3\n\t"
      "s_nop 0\n\t"
      "buffer_load_dword %0, %1, %2 offen lds"
      :
      : "v"(v), "s"(d), "s"(s), "s"(m)
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

// Tile number -> (tm, tn): in groups of 8 along the first axis, that axis fastest,
// so that neighbours share few row blocks of both operands.
__device__ __forceinline__ void tile_of(uint32_t id, uint32_t tiles_m, uint32_t tiles_n, uint32_t& tm, uint32_t& tn) {
  const uint32_t group = 8 * tiles_n, gi = id / group, first = gi * 8;
  const uint32_t rows = min(tiles_m - first, 8u), in = id - gi * group;
  tm = __builtin_amdgcn_readfirstlane(first + in % rows);
  tn = __builtin_amdgcn_readfirstlane(in / rows);
}

constexpr uint32_t kCus = 256;

// Arguments of a launch that does two jobs: `first` workgroups take x[0], the others
// x[1].  (Indexed, so that what differs is read from the arguments as scalars.)
template <class A>
struct Pair {
  A x[2];
  uint32_t first;
};
// This workgroup's job, its number there and the job's workgroups.
struct Share {
  uint32_t job, block, blocks;
  __device__ __forceinline__ explicit Share(uint32_t first)
      : job(blockIdx.x < first ? 0 : 1), block(job ? blockIdx.x - first : blockIdx.x), blocks(job ? gridDim.x - first : first) {}
};

template <int EL, int WM, int WN, int TM, int TN>
struct Tile {
  static constexpr int kWN = WN, kTM = TM, kTN = TN;
  static constexpr int NT = 64 * WM * WN;           // threads
  static constexpr int BM = 16 * WM * TM, BN = 16 * WN * TN;
  static constexpr int ROWS = BM + BN;
  static constexpr bool kExact = EL == EL_FP8X || EL == EL_FP8BX, kBlockP = EL == EL_FP8B || EL == EL_FP8BX;
  static constexpr bool kFp8 = EL == EL_FP8 || EL == EL_FP8B || kExact, kPair = EL == EL_PAIR;
  static constexpr int RPI = NT / 8;                // rows one load instruction of all threads covers
  static constexpr int PB = kPair ? RPI / 16 : TM < 4 ? TM : 4;  // tiles whose rows interleave
  static constexpr int LP = BM / RPI, LQ = BN / RPI;
  static constexpr int SCALE_DW = EL == EL_MX ? ROWS * 2 : kFp8 ? ROWS : 0;  // scale words of a chunk
  static constexpr int PROWS = kPair ? BM / 2 : BM;  // rows of P('s matrices) in a tile
  static_assert(!kPair || (TM % (2 * PB) == 0 && PB <= 4), "a wave holds as many rows of either matrix");
  static_assert(BM % RPI == 0 && BN % RPI == 0, "whole load instructions");
  static_assert(RPI >= 2 * TN && RPI % 32 == 0, "a thread's rows i * RPI + r differ from r by bits of the key above its own");
  static_assert(TN == 1 || TN % 2 == 0, "q_place pairs rows");
  static_assert(TM % PB == 0, "whole row blocks");

  // Workgroups a CU holds at once (by LDS; at most 16 waves, which then have 128
  // registers each), and those of a launch over `items` tiles: as many as run at once,
  // each going on to further tiles itself.
  static constexpr int kLds = (ROWS * 128 + SCALE_DW * 4) * 2;
  static constexpr int PER_CU = 160 * 1024 / kLds < 1024 / NT ? 160 * 1024 / kLds : 1024 / NT;
  static constexpr int WAVES = PER_CU * NT / 256;  // waves a SIMD then holds
  static uint32_t grid(uint64_t items) { return (uint32_t)(items < kCus * PER_CU ? items : kCus * PER_CU); }

  struct Smem {
    uint8_t stage[2][ROWS * 128];
    uint32_t scale[2][SCALE_DW ? SCALE_DW : 1];
  };

  typedef float4_t Acc[TM][TN];

  // row of the wave's P rows that lane quad g (0..3), result r (0..3) of tile tm holds
  static __device__ __forceinline__ constexpr int p_row(int tm, int g, int r) {
    return (tm / PB) * 16 * PB + g * 4 * PB + (tm % PB) * 4 + r;
  }
  // row of the wave's Q rows that lane n (0..15) of tile tn holds
  static __device__ __forceinline__ constexpr int q_row(int tn, int n) { return n * TN + tn; }
  // A 16-byte read serves 16 lanes in a pass if they touch all 64 banks (256 bytes)
  // once.  The lanes of a pass are not neighbours: of 32, {0-3, 12-15, 20-27} go
  // first, then the others, so half of them read the piece 2 further (g odd) in rows
  // that differ from the others' in (n / 4) & 1 ^ n / 8, the bit which the key's top
  // bit therefore is.  (With n / 4 for the key's top bits every read took two passes;
  // head forward of 16384 x 50304 over 1024: 676 million busy cycles of all CUs, 662 so.)
  // P: rows of one tile differ in their low two bits and in row / (4 PB), of which
  // the lowest picks the half of 256 bytes by itself.  Q: rows of one tile are TN
  // apart, so for even TN every other of them trades places with its neighbour.
  static __device__ __forceinline__ constexpr int spread(int k) { return (k & 1) | ((k >> 1) & 2) | (((k << 1) ^ k) & 4); }
  static __device__ __forceinline__ constexpr int p_key(int row) { return spread(((row >> 1) & 1) | (((row / (4 * PB)) & 3) << 1)); }
  static __device__ __forceinline__ constexpr int q_key(int row) { return spread((row / (2 * TN)) & 7); }
  static __device__ __forceinline__ constexpr int q_place(int row) { return TN % 2 ? row : row ^ ((row / TN) & 1); }

  // The launch's tiles (times the splits of their reduction) in the order of
  // tile_of; a workgroup takes every step-th of its XCD's range.
  struct Items {
    uint32_t tiles_p, tiles_q, nch, splits;
    uint32_t at, end, step;
    // of workgroup b of n
    __device__ __forceinline__ Items(uint32_t tp, uint32_t tq, uint32_t chunks, uint32_t z, uint32_t b = blockIdx.x,
                                     uint32_t n = gridDim.x)
        : tiles_p(tp), tiles_q(tq), nch(chunks), splits(z) {
      // XCD x has the workgroups b = x modulo 8; its range is in proportion to their
      // number, so that no workgroup has two more items than another
      const uint32_t total = tp * tq * z, x = b % 8;
      const uint32_t before = x * (n / 8) + min(x, n % 8), count = n / 8 + (x < n % 8 ? 1 : 0);
      at = (uint32_t)((uint64_t)total * before / n) + b / 8;
      end = (uint32_t)((uint64_t)total * (before + count) / n);
      step = count;
    }
  };
  struct Item {
    uint32_t tp, tq, z;
    int c, c1;
    __device__ __forceinline__ void set(const Items& s, uint32_t at) {
      const uint32_t tiles = s.tiles_p * s.tiles_q;
      z = __builtin_amdgcn_readfirstlane(at / tiles);
      tile_of(at - z * tiles, s.tiles_q, s.tiles_p, tq, tp);
      c = __builtin_amdgcn_readfirstlane((int)(s.nch * z / s.splits));
      c1 = __builtin_amdgcn_readfirstlane((int)(s.nch * (z + 1) / s.splits));
    }
  };

  // All items of this workgroup as one sequence of chunks: the loads run two chunks
  // ahead, across the items' borders, so that an item's first chunks arrive while
  // the last one's results are stored.  epilogue(p0, q0, z, acc) takes an item's sums.
  template <class Epilogue>
  static __device__ __forceinline__ void run(const TileOp& P, const TileOp& Q, const Items& items, Smem& sm,
                                             Epilogue&& epilogue) {
    if (items.at >= items.end) return;
    const int t = threadIdx.x, lane = t & 63, w = __builtin_amdgcn_readfirstlane(t >> 6);
    const int wm = w / WN, wn = w % WN, n = lane & 15, g = lane >> 4;
    Acc acc = {};
    Item now;
    now.set(items, items.at);

    // what this thread loads: row i * RPI + t / 8, slot t % 8
    const int lr = t >> 3;
    const int lrq = q_place(lr);
    // byte in the row of what it fetches for row i * RPI + lr
    auto gp = [&](int i) __attribute__((always_inline)) { return (uint32_t)((t & 7) ^ p_key(lr) ^ p_key(i * RPI)) * 16u; };
    auto gq = [&](int i) __attribute__((always_inline)) { return (uint32_t)((t & 7) ^ q_key(lr) ^ q_key(i * RPI)) * 16u; };
    // (MXFP4 operands of a product have one layout, and their scales the same in 1/16)
    constexpr bool kMx = EL == EL_MX;
    const uint32_t ldp = pinned((uint32_t)P.ld), ldq = kMx ? ldp : pinned((uint32_t)Q.ld);
    const uint32_t bsp = pinned((uint32_t)P.bs), bsq = kMx ? bsp : pinned((uint32_t)Q.bs);
    const uint32_t csp = pinned((uint32_t)P.cs), csq = kMx ? csp : pinned((uint32_t)Q.cs);
    const int kbp = (int)pinned((uint32_t)P.kb), kbq = kMx ? kbp : (int)pinned((uint32_t)Q.kb);
    const uint32_t vp = (uint32_t)lr * ldp, vq = (uint32_t)lrq * ldq;
    // and the uniform offset of its row i * RPI
    static_assert(128 % RPI == 0 && (BM < 128 || BM % 128 == 0) && (BN < 128 || BN % 128 == 0), "rows of a block");
    auto far_p = [&](int i) __attribute__((always_inline)) {
      return (uint32_t)(i * RPI / 128) * bsp + (uint32_t)(i * RPI % 128) * ldp;
    };
    auto far_q = [&](int i) __attribute__((always_inline)) {
      return (uint32_t)(i * RPI / 128) * bsq + (uint32_t)(i * RPI % 128) * ldq;
    };
    const uint32_t lds_w = lds_address(sm.stage[0]) + (uint32_t)w * 1024u;
    constexpr uint32_t kStage = ROWS * 128;

    // scales: MXFP4 [row][2] words of a chunk, a wave 32 rows at a time (all of P or all
    // of Q: BM is a multiple of 32); FP8 a word a row, 64 rows at a time
    constexpr int SJ = EL == EL_MX ? SCALE_DW / NT : kFp8 ? (SCALE_DW + NT - 1) / NT : 1;
    static_assert(kFp8 ? BM % 64 == 0 && BN % 64 == 0 : SCALE_DW % NT == 0 && BM % 32 == 0, "whole scale loads");
    const uint32_t vs = (uint32_t)(lane >> 1) * (ldp / 16) + (lane & 1) * 4;
    const uint32_t srp = kFp8 ? pinned((uint32_t)P.srs) : 0, srq = kFp8 ? pinned((uint32_t)Q.srs) : 0;

    // The load cursor: its item, the item's rows (none once the items are done), where
    // its chunk starts and the bytes of a row from there on.
    Item ahead = now;
    uint32_t ahead_at = items.at;
    const uint8_t *pb, *qb, *psb = nullptr, *qsb = nullptr, *pb2 = nullptr;
    int np, nq, leftp, leftq;
    auto enter = [&]() __attribute__((always_inline)) {
      const int64_t p0 = (int64_t)ahead.tp * PROWS, q0 = (int64_t)ahead.tq * BN;
      if constexpr (kPair) pb2 = P.p2 + (p0 >> 7) * P.bs + (p0 & 127) * P.ld + mul32(ahead.c, csp);
      if constexpr (kFp8) {
        psb = P.s + (kBlockP ? p0 >> 7 : p0) * P.srs + (int64_t)ahead.c * P.scs;
        qsb = Q.s + q0 * Q.srs + (int64_t)ahead.c * Q.scs;
      }
      pb = P.p + (p0 >> 7) * P.bs + (p0 & 127) * P.ld + mul32(ahead.c, csp);
      qb = Q.p + (q0 >> 7) * Q.bs + (q0 & 127) * Q.ld + mul32(ahead.c, csq);
      leftp = kbp - ahead.c * 128;
      leftq = kbq - ahead.c * 128;
      if constexpr (EL == EL_MX) {
        psb = P.s + ((p0 >> 7) * P.bs + (p0 & 127) * P.ld + mul32(ahead.c, csp)) / 16;
        qsb = Q.s + ((q0 >> 7) * Q.bs + (q0 & 127) * Q.ld + mul32(ahead.c, csq)) / 16;
      }
      np = __builtin_amdgcn_readfirstlane((int)min(P.rows - p0, (int64_t)PROWS));
      nq = __builtin_amdgcn_readfirstlane((int)min(Q.rows - q0, (int64_t)BN));
    };
    enter();
    // The loads of the cursor's chunk into `stage`, one at a time: begin() sets them up.
    u32x4_t dp, dq, dsp, dsq, dp2;
    uint32_t bads = 0, dst = 0, sdst = 0;
    // (FP8: the cursor's rows and bytes as they were then; it goes on before the last load,
    // where its branch does not part a chunk's instructions)
    int np1 = 0, nq1 = 0, leftp1 = 0, leftq1 = 0;
    auto begin = [&](uint32_t stage) __attribute__((always_inline)) {
      np1 = np;
      nq1 = nq;
      leftp1 = leftp;
      leftq1 = leftq;
      dp = raw_buffer(pb);
      dq = raw_buffer(qb);
      settle(dp, dq);
      dst = lds_w + stage * kStage;
      if constexpr (kPair) {
        dp2 = raw_buffer(pb2);
        settle(dp, dp2);
      }
      if constexpr (kFp8) {
        dsp = raw_buffer(psb);
        dsq = raw_buffer(qsb);
        settle(dsp, dsq);
        sdst = lds_address(sm.scale[0]) + stage * (SCALE_DW * 4) + (uint32_t)w * 256u;
      }
      if constexpr (EL == EL_MX) {
        dsp = raw_buffer(psb);
        dsq = raw_buffer(qsb);
        settle(dsp, dsq);
        bads = (lane & 1) * 64 >= leftp ? kOutside : 0u;  // 4 scale bytes stand for 64 of codes
        sdst = lds_address(sm.scale[0]) + stage * (SCALE_DW * 4) + (uint32_t)w * 256u;
      }
    };
    // after the chunk's last load: on to the next one
    auto advance = [&]() __attribute__((always_inline)) {
      if (++ahead.c == ahead.c1) {
        ahead_at += items.step;
        if (ahead_at < items.end) {
          ahead.set(items, ahead_at);
          enter();
        } else {
          np = nq = 0;
          ahead.c1 = 1 << 30;
        }
      } else {
        pb += csp;
        qb += csq;
        leftp -= 128;
        leftq -= 128;
        if constexpr (kPair) pb2 += csp;
        if constexpr (kMx) {
          psb += csp / 16;
          qsb += csq / 16;
        }
        if constexpr (kFp8) {
          psb += P.scs;
          qsb += Q.scs;
        }
      }
    };
    constexpr int LOADS = LP + LQ + (EL == EL_MX || kFp8 ? SJ : 0);
    auto load = [&](int i) __attribute__((always_inline)) {
      const int np_ = kFp8 ? np1 : np, nq_ = kFp8 ? nq1 : nq, leftp_ = kFp8 ? leftp1 : leftp, leftq_ = kFp8 ? leftq1 : leftq;
      if (kPair && i < LP) {
        load_lds16(i & 1 ? dp2 : dp, lr < np_ - (i >> 1) * RPI && (int)gp(i) < leftp_ ? vp + gp(i) : kOutside, far_p(i >> 1), dst + i * (RPI * 128));
      } else if (i < LP) {
        load_lds16(dp, lr < np_ - i * RPI && (int)gp(i) < leftp_ ? vp + gp(i) : kOutside, far_p(i), dst + i * (RPI * 128));
      } else if (i < LP + LQ) {
        load_lds16(dq, lrq < nq_ - (i - LP) * RPI && (int)gq(i - LP) < leftq_ ? vq + gq(i - LP) : kOutside, far_q(i - LP), dst + i * (RPI * 128));
      } else if constexpr (EL == EL_MX) {
        const int j = i - LP - LQ, r0 = w * 32 + j * (NT / 2);
        const bool isp = r0 < BM;
        const int first = isp ? r0 : r0 - BM;
        u32x4_t d;
        d.x = isp ? dsp.x : dsq.x;
        d.y = isp ? dsp.y : dsq.y;
        d.z = dsp.z;
        d.w = dsp.w;
        load_lds4(d, (lane >> 1) < (isp ? np_ : nq_) - first ? vs | bads : kOutside, (uint32_t)(first >> 7) * (bsp / 16) + (uint32_t)(first & 127) * (ldp / 16),
                  sdst + j * (NT * 4));
      } else if constexpr (kFp8) {
        const int j = i - LP - LQ, r0 = w * 64 + j * NT;
        if (ROWS % NT && r0 >= ROWS) return;
        const bool isp = r0 < BM;
        const int first = isp ? r0 : r0 - BM;
        const bool block = kBlockP && isp;
        u32x4_t d;
        d.x = isp ? dsp.x : dsq.x;
        d.y = isp ? dsp.y : dsq.y;
        d.z = dsp.z;
        d.w = dsp.w;
        const uint32_t sr = isp ? srp : srq;
        load_lds4(d, lane < (isp ? np_ : nq_) - first ? (block ? 0u : (uint32_t)lane * sr) : kOutside, (uint32_t)(block ? first >> 7 : first) * sr,
                  sdst + j * (NT * 4));
      }
    };

    const int pr0 = wm * TM * 16, qr0 = BM + wn * TN * 16;
    const int pk = p_key(p_row(0, n >> 2, n & 3)), qk = q_key(q_row(0, n));
    // LDS byte addresses; the two steps' pieces are neighbours, 16 bytes apart
    const uint32_t lp = lds_address(sm.stage[0]) + (uint32_t)(pr0 + p_row(0, n >> 2, n & 3)) * 128u + ((2 * g) ^ pk) * 16;
    // even and odd tiles of Q: a lane's rows trade places in pairs
    const uint32_t lq0 = lds_address(sm.stage[0]) + (uint32_t)(qr0 + q_place(q_row(0, n))) * 128u + ((2 * g) ^ qk) * 16;
    const uint32_t lq1 = lds_address(sm.stage[0]) + (uint32_t)(qr0 + q_place(q_row(TN > 1 ? 1 : 0, n))) * 128u + ((2 * g) ^ qk) * 16;
    if constexpr (kFp8) {
      // A chunk: TM rows of TN instructions.  The result of one waits in registers until the
      // next row's has its turn there and is scaled and added to the sums then, so that the
      // wave's arithmetic fills the instructions' time (the chunk's last row among the
      // next chunk's first).  P's fragments are read two rows ahead; Q's, which every row
      // needs, as the last row's instructions let go of them.  The barrier comes before the
      // last row, all of whose operands are in registers: the stage is refilled from there on.
      constexpr int PR = 2;
      i32x4_t fp[PR][2], fq[TN][2];
      float4_t part[TN];
      float sq[TN], sb = 0.0f;
      float4_t sp[kBlockP ? 1 : PR];
      // exact: the codes as f16, two rows of P's (the next one's is decoded while one runs)
      half8_t xp[kExact ? 2 : 1][4], xq[kExact ? TN : 1][4];
      const uint32_t lsp = lds_address(sm.scale[0]) + (uint32_t)(pr0 + (kBlockP ? 0 : p_row(0, g, 0))) * 4u;
      const uint32_t lsq = lds_address(sm.scale[0]) + (uint32_t)(qr0 + q_row(0, n)) * 4u;
      auto read_p = [&](uint32_t stage, int tm) __attribute__((always_inline)) {
#pragma unroll
        for (int h = 0; h < 2; ++h) fp[tm % PR][h] = lds_read<i32x4_t>(((lp ^ (h * 16)) + stage * kStage) + p_row(tm, 0, 0) * 128);
      };
      auto read_q1 = [&](uint32_t stage, int tn) __attribute__((always_inline)) {
#pragma unroll
        for (int h = 0; h < 2; ++h) fq[tn][h] = lds_read<i32x4_t>((((tn & 1 ? lq1 : lq0) ^ (h * 16)) + stage * kStage) + (tn & ~1) * 128);
      };
      auto read_scales = [&](uint32_t stage) __attribute__((always_inline)) {
        if constexpr (TN == 4) {
          const float4_t v = lds_read<float4_t>(lsq + stage * (SCALE_DW * 4));
          sq[0] = v.x; sq[1] = v.y; sq[2] = v.z; sq[3] = v.w;
        } else {
#pragma unroll
          for (int tn = 0; tn < TN; ++tn) sq[tn] = lds_read<float>(lsq + stage * (SCALE_DW * 4) + tn * 4);
        }
        if constexpr (kBlockP) sb = lds_read<float>(lsp + stage * (SCALE_DW * 4));
      };
      auto read_sp = [&](uint32_t stage, int tm) __attribute__((always_inline)) {
        if constexpr (!kBlockP) sp[tm % PR] = lds_read<float4_t>(lsp + stage * (SCALE_DW * 4) + p_row(tm, 0, 0) * 4);
      };
      auto decode_p = [&](int tm) __attribute__((always_inline)) {
        if constexpr (kExact)
#pragma unroll
          for (int k = 0; k < 4; ++k) xp[tm % 2][k] = fp8_to_f16(fp[tm % PR][0], fp[tm % PR][1], k);
      };
      auto decode_q = [&]() __attribute__((always_inline)) {
        if constexpr (kExact)
#pragma unroll
          for (int i = 0; i < TN * 4; ++i) xq[i / 4][i % 4] = fp8_to_f16(fq[i / 4][0], fq[i / 4][1], i % 4);
      };
      // instruction k of tile (tm, tn) (exact: four of 32 elements, k by k so that none waits
      // for the one before it)
      constexpr int KS = kExact ? 4 : 1;
      auto mma = [&](auto tmc, auto tnc, auto kc) __attribute__((always_inline)) {
        constexpr int tm = decltype(tmc)::value, tn = decltype(tnc)::value, k = decltype(kc)::value;
        const float4_t z = {0.0f, 0.0f, 0.0f, 0.0f};
        if constexpr (kExact) {
          part[tn] = __builtin_amdgcn_mfma_f32_16x16x32_f16(xp[tm % 2][k], xq[tn][k], k ? part[tn] : z, 0, 0, 0);
        } else {
          const i32x8_t a = __builtin_shufflevector(fp[tm % PR][0], fp[tm % PR][1], 0, 1, 2, 3, 4, 5, 6, 7);
          const i32x8_t b = __builtin_shufflevector(fq[tn][0], fq[tn][1], 0, 1, 2, 3, 4, 5, 6, 7);
          part[tn] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, z, 0, 0, 0, 0, 0, 0);
        }
      };
      // the result of tile (tm, tn)
      auto add = [&](auto tmc, auto tnc) __attribute__((always_inline)) {
        constexpr int tm = decltype(tmc)::value, tn = decltype(tnc)::value;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          if constexpr (kBlockP) acc[tm][tn][r] = fmaf(part[tn][r], sq[tn], acc[tm][tn][r]);
          else acc[tm][tn][r] = fmaf(part[tn][r] * sq[tn], sp[tm % PR][r], acc[tm][tn][r]);
        }
      };
      auto scale_q = [&]() __attribute__((always_inline)) {
        if constexpr (kBlockP) {
#pragma unroll
          for (int tn = 0; tn < TN; ++tn) sq[tn] *= sb;
        }
      };
      // the next chunk's loads: EARLY of them in the last row, the others in the next SPAN
      constexpr int EARLY = TM >= 4 ? 2 : 1, SPAN = TM >= 4 ? TM / 2 : 1;
      begin(0);
#pragma unroll
      for (int i = 0; i < LOADS; ++i) load(i);
      advance();
      tile_barrier();
      begin(1);
#pragma unroll
      for (int i = 0; i < EARLY; ++i) load(i);
      uint32_t st = 0, at = items.at;
      for (;;) {
        // the item's first fragments (read again after an epilogue, which has the registers
        // to itself), and nothing of a chunk before
#pragma unroll
        for (int tn = 0; tn < TN; ++tn) read_q1(st, tn);
        read_p(st, 0);
        read_sp(st, 0);
        read_p(st, 1);
#pragma unroll
        for (int tn = 0; tn < TN; ++tn) {
          part[tn] = float4_t{0.0f, 0.0f, 0.0f, 0.0f};
          sq[tn] = 0.0f;
        }
        if constexpr (!kBlockP) sp[(TM - 1) % PR] = float4_t{0.0f, 0.0f, 0.0f, 0.0f};
#pragma nounroll
        for (; now.c < now.c1; ++now.c) {
          advance();
          decode_q();
          decode_p(0);
          static_for<TM>([&](auto tmc) __attribute__((always_inline)) {
            constexpr int tm = decltype(tmc)::value;
            using Before = std::integral_constant<int, (tm + TM - 1) % TM>;
            static_for<KS * TN>([&](auto ic) __attribute__((always_inline)) {
              constexpr int tn = decltype(ic)::value % TN, k = decltype(ic)::value / TN;
              using Tn = std::integral_constant<int, tn>;
              if constexpr (k == 0) add(Before{}, Tn{});
              mma(tmc, Tn{}, std::integral_constant<int, k>{});
              __builtin_amdgcn_sched_barrier(0);
              if constexpr (tm == TM - 1 && k == KS - 1) read_q1(st, tn);
            });
            if constexpr (tm + 1 < TM) decode_p(tm + 1);
            if constexpr (tm == 0) {  // (the last chunk's scales have been used)
              read_scales(st);
              scale_q();
            }
            if constexpr (tm < SPAN) {
#pragma unroll
              for (int i = EARLY; i < LOADS; ++i)
                if ((i - EARLY) * SPAN / (LOADS - EARLY) == tm) load(i);
            }
            if constexpr (tm + 1 < TM) read_sp(st, tm + 1);
            if constexpr (tm + 2 < TM) read_p(st, tm + 2);
            if constexpr (tm == TM - 2) {
              tile_barrier();
              begin(st);
              st ^= 1u;
              read_p(st, 0);
            }
            if constexpr (tm == TM - 1) {
              read_p(st, 1);
              read_sp(st, 0);
#pragma unroll
              for (int i = 0; i < EARLY; ++i) load(i);
            }
          });
        }
        static_for<TN>([&](auto tnc) __attribute__((always_inline)) { add(std::integral_constant<int, TM - 1>{}, tnc); });
        epilogue((int64_t)now.tp * BM, (int64_t)now.tq * BN, now.z, acc);
        at += items.step;
        if (at >= items.end) break;
        now.set(items, at);
#pragma unroll
        for (int tm = 0; tm < TM; ++tm)
#pragma unroll
          for (int tn = 0; tn < TN; ++tn) acc[tm][tn] = float4_t{0.0f, 0.0f, 0.0f, 0.0f};
      }
      tile_barrier();  // nothing is in flight into LDS when the caller goes on
      return;
    }
    // Fragments of step s of a chunk: piece 2 g + s of the lane's rows.  P's are
    // kept once: those of the next step are read into a tile's registers as soon
    // as its instructions have issued.  Q's, which every tile needs, twice.
    i32x4_t fp[TM], fq[2][TN];
    // scale bytes of both steps, two tiles a register; as read (two bytes) they wait a
    // while in rp, rq before they are paired, which would wait for the read
    constexpr int NSP = (TM + 1) / 2, NSQ = (TN + 1) / 2;
    uint32_t sp[NSP], sq[NSQ], rp[TM], rq[TN];
    const uint32_t lsp = lds_address(sm.scale[0]) + (uint32_t)(pr0 + p_row(0, n >> 2, n & 3)) * 8u + 2 * g;
    const uint32_t lsq = lds_address(sm.scale[0]) + (uint32_t)(qr0 + q_row(0, n)) * 8u + 2 * g;
    auto read_p = [&](uint32_t stage, int s, int tm) __attribute__((always_inline)) {
      fp[tm] = lds_read<i32x4_t>(((lp ^ (s * 16)) + stage * kStage) + p_row(tm, 0, 0) * 128);
    };
    auto read_q = [&](uint32_t stage, int s, int tn) __attribute__((always_inline)) {
      fq[s][tn] = lds_read<i32x4_t>((((tn & 1 ? lq1 : lq0) ^ (s * 16)) + stage * kStage) + (tn & ~1) * 128);
    };
    auto read_sp = [&](uint32_t stage, int tm) __attribute__((always_inline)) {
      if constexpr (EL == EL_MX) rp[tm] = lds_read<uint16_t>(lsp + stage * (SCALE_DW * 4) + p_row(tm, 0, 0) * 8);
    };
    auto read_sq = [&](uint32_t stage, int tn) __attribute__((always_inline)) {
      if constexpr (EL == EL_MX) rq[tn] = lds_read<uint16_t>(lsq + stage * (SCALE_DW * 4) + q_row(tn, 0) * 8);
    };
    auto pair_sp = [&](int k) __attribute__((always_inline)) {
      if constexpr (EL == EL_MX) sp[k] = 2 * k + 1 < TM ? rp[2 * k] | rp[2 * k + 1] << 16 : rp[2 * k];
    };
    auto pair_sq = [&]() __attribute__((always_inline)) {
      if constexpr (EL == EL_MX) {
#pragma unroll
        for (int k = 0; k < NSQ; ++k) sq[k] = 2 * k + 1 < TN ? rq[2 * k] | rq[2 * k + 1] << 16 : rq[2 * k];
      }
    };
    auto mma = [&](auto sc, auto tmc) __attribute__((always_inline)) {
      constexpr int s = decltype(sc)::value, tm = decltype(tmc)::value;
      static_for<TN>([&](auto tnc) __attribute__((always_inline)) {
        constexpr int tn = decltype(tnc)::value;
        if constexpr (EL != EL_MX) {
          acc[tm][tn] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, fp[tm]),
                                                                __builtin_bit_cast(bf16x8_t, fq[s][tn]), acc[tm][tn], 0, 0, 0);
        } else {
          const i32x8_t a = __builtin_shufflevector(fp[tm], i32x4_t{0, 0, 0, 0}, 0, 1, 2, 3, 4, 5, 6, 7);
          const i32x8_t b = __builtin_shufflevector(fq[s][tn], i32x4_t{0, 0, 0, 0}, 0, 1, 2, 3, 4, 5, 6, 7);
          acc[tm][tn] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
              a, b, acc[tm][tn], 4, 4, s + 2 * (tm % 2), (int)sp[tm / 2], s + 2 * (tn % 2), (int)sq[tn / 2]);
        }
      });
    };
    using S0 = std::integral_constant<int, 0>;
    using S1 = std::integral_constant<int, 1>;
    // the tiles of the second step before which the barrier is crossed
    constexpr int LEAD = TM >= 4 ? 2 : 1;
    // the next chunk's loads are dealt out over the instruction tiles after it, so that
    // no burst of them keeps the waves from issuing; in large tiles, whose chunks take
    // longest, two are left for the next step (forward of 16384 x 50304 over 1024: 1483
    // us without, 1452 with; with four 1507; 128 x 128 tiles lose by it)
    constexpr int SLOTS = TM - LEAD + 1, LATE = TM >= 8 ? 2 : 0;
    // the last pair of P's scales is made up in the next chunk, before its tiles
    constexpr int LAZY = TM >= 8 ? 1 : 0;
    begin(0);
#pragma unroll
    for (int i = 0; i < LOADS; ++i) load(i);
    advance();
    tile_barrier();
    begin(1);
#pragma unroll
    for (int i = 0; i < LOADS - LATE; ++i) load(i);
    // Every chunk runs the same straight line: past the last item the loads bring
    // zeros, and the fragments read then are not used.
    uint32_t st = 0, at = items.at;
    for (;;) {
      // the item's first fragments (read again after an epilogue, which has the
      // registers to itself)
#pragma unroll
      for (int tn = 0; tn < TN; ++tn) {
        read_q(st, 0, tn);
        read_sq(st, tn);
      }
#pragma unroll
      for (int tm = 0; tm < TM; ++tm) {
        read_p(st, 0, tm);
        read_sp(st, tm);
      }
      pair_sq();
#pragma unroll
      for (int k = 0; k < NSP - LAZY; ++k) pair_sp(k);
#pragma nounroll
      for (; now.c < now.c1; ++now.c) {
#pragma unroll
        for (int tn = 0; tn < TN; ++tn) read_q(st, 1, tn);
        static_for<TM>([&](auto tmc) __attribute__((always_inline)) {
          constexpr int tm = decltype(tmc)::value;
          mma(S0{}, tmc);
          __builtin_amdgcn_sched_barrier(0);
          read_p(st, 1, tm);
          if constexpr (LAZY && tm == TM - 4) pair_sp(NSP - 1);
#pragma unroll
          for (int i = LOADS - LATE; i < LOADS; ++i)
            if ((i - (LOADS - LATE)) * TM / 2 == tm) load(i);
        });
        advance();
        static_for<TM>([&](auto tmc) __attribute__((always_inline)) {
          constexpr int tm = decltype(tmc)::value;
          mma(S1{}, tmc);
          __builtin_amdgcn_sched_barrier(0);
          if constexpr (tm == LEAD - 1) {
            tile_barrier();
            begin(st);
#pragma unroll
            for (int tn = 0; tn < TN; ++tn) {
              read_q(st ^ 1u, 0, tn);
              read_sq(st ^ 1u, tn);
            }
#pragma unroll
            for (int k = 0; k < LEAD; ++k) read_p(st ^ 1u, 0, k);
          } else if constexpr (tm >= LEAD) {
            read_p(st ^ 1u, 0, tm);
          }
          // (a register of two tiles' scales is free after the second; none before the barrier)
          if constexpr (tm >= LEAD - 1 && (tm % 2 == 1 || tm == TM - 1)) {
            constexpr int from = tm == (LEAD - 1) / 2 * 2 + 1 || tm == LEAD - 1 ? 0 : tm / 2 * 2;
#pragma unroll
            for (int k = from; k <= tm; ++k) read_sp(st ^ 1u, k);
            if constexpr (from > 0) pair_sp(from / 2 - 1);
          }
          if constexpr (tm >= LEAD - 1) {
#pragma unroll
            for (int i = 0; i < LOADS - LATE; ++i)
              if (i * SLOTS / (LOADS - LATE) == tm - (LEAD - 1)) load(i);
          }
        });
        if constexpr (!LAZY) pair_sp(NSP - 1);
        pair_sq();
        st ^= 1u;
      }
      epilogue((int64_t)now.tp * BM, (int64_t)now.tq * BN, now.z, acc);
      at += items.step;
      if (at >= items.end) break;
      now.set(items, at);
#pragma unroll
      for (int tm = 0; tm < TM; ++tm)
#pragma unroll
        for (int tn = 0; tn < TN; ++tn) acc[tm][tn] = float4_t{0.0f, 0.0f, 0.0f, 0.0f};
    }
    tile_barrier();  // nothing is in flight into LDS when the caller goes on
  }
};

}  // namespace tj2
