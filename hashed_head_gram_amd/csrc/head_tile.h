// Products of the head's losses on the matrix cores: tiles of P Q^T with both
// operands walked through an LDS ring, and what the losses do with a tile's
// accumulators (maxima and sums, gradients of the logits, products). gfx950.
//
// A tile is 256 x 256 by 8 waves of 128 x 64, or 128 x 128 by 4 of 64 x 64. K
// advances 32 at a time through a ring of four slots filled by direct
// global-to-LDS loads, two steps of v_mfma_f32_32x32x16 a slot, fragments read
// one step ahead, one barrier a slot; three slots of loads stay in flight. An
// operand lies in memory with K contiguous in a row (plain) or with a row for
// each K (transposed: read by ds_read_b64_tr_b16, 16 columns by 4 rows of K at a
// time, so no transposed copy of h, T or dz is ever made).
//
// What bounds it: power. The large products run at 1,070 to 1,290 TFLOP/s (a
// large library product: 1,155), the clock at 1.4 to 1.7 GHz with the matrix
// units busy 53 to 75 % of the time; with zeros for dz the same launch is 12 %
// faster. Four waves of 128 x 128, which read a third less from LDS, were 4 %
// slower (nothing runs through barriers and epilogues), K walks a slot apart on
// neighbouring tiles within 1 % either way.
#pragma once

#include <type_traits>

#include "train.h"

namespace pg {
namespace {

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8_t __attribute__((ext_vector_type(8)));
typedef _Float16 f16v2_t __attribute__((ext_vector_type(2)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));
typedef float f32x16_t __attribute__((ext_vector_type(16)));
typedef short s16x4_t __attribute__((ext_vector_type(4)));
typedef short s16x8_t __attribute__((ext_vector_type(8)));
typedef __attribute__((address_space(3))) void lds_void_t;
typedef __attribute__((address_space(3))) s16x4_t lds_s16x4_t;

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr int kCUs = 256;
constexpr int kRing = 4;                  // slots in the LDS ring
// halves of the two operands by segment of K, small products first
constexpr int kSegs = 3;
__device__ __forceinline__ int seg_a(int s) { return s == 1; }
__device__ __forceinline__ int seg_b(int s) { return s == 0; }
constexpr int kTop = 14;                  // exponent that placements bring the largest value to
constexpr int kNone = -4096;              // exponent of nothing

// Two floats to packed fp16, nearest even.
__device__ __forceinline__ uint32_t pack2_f16(float a, float b) {
  const f32v2_t v = {a, b};
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, f16v2_t));
}
__device__ __forceinline__ float lo_f16(uint32_t w) {
  return (float)__builtin_bit_cast(_Float16, (uint16_t)w);
}
__device__ __forceinline__ float hi_f16(uint32_t w) {
  return (float)__builtin_bit_cast(_Float16, (uint16_t)(w >> 16));
}
// The type that dz is held in: fp16, or bf16.
template <bool F16>
struct Half {
  static __device__ __forceinline__ uint32_t pack(float a, float b) {
    return F16 ? pack2_f16(a, b) : pack2_bf16(a, b);
  }
  static __device__ __forceinline__ float lo(uint32_t w) {
    return F16 ? lo_f16(w) : __uint_as_float(w << 16);
  }
  static __device__ __forceinline__ float hi(uint32_t w) {
    return F16 ? hi_f16(w) : __uint_as_float(w & 0xFFFF0000u);
  }
};
// x with 2^e: floor(log2 |x|); nothing for zeros, infinities and NaN.
__device__ __forceinline__ int exponent_of(float x) {
  const float a = fabsf(x);
  return a > 0.f && a < INFINITY ? ilogbf(a) : kNone;
}

// Levels of dz. A row of dz in fp16 is placed by its own bound, which leaves 28
// bits above fp16's smallest normal number; a vocabulary row that no token finds
// likely lies below them. Its column is then lifted by a power of two, the level:
// by the largest |dz| of a group of rows, kFlat where that is 2^kRare or more (fp16
// steps are 2^-19 of it at most), else in steps of kLift, so that the groups of a
// column mostly agree; kEmpty for zeros alone. One byte a group and column. Later
// all groups of a column come to its lowest level, dT undoes it, and T's copy for
// dh carries its inverse.
constexpr int kFlat = 0, kEmpty = 255;
constexpr int kRare = -6;                 // against bounds of 2^kTop
constexpr int kLift = 20;                 // a lifted column's largest: 2^kRare to 2^(kRare + kLift)
static_assert(kRare + kLift <= kTop && 126 + kLift < kEmpty, "in fp16, and in a byte");
// of the upper 16 bits of the largest |dz| in fp32
__device__ __forceinline__ uint32_t level_of(uint32_t top16) {
  if (top16 == 0) return kEmpty;
  const int e = (int)(top16 >> 7) - 127;             // NaN and infinity: 128
  return e < kRare ? (uint32_t)((kRare - (e < -126 ? -126 : e) + kLift - 1) / kLift * kLift) : kFlat;
}
__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) {
  typedef uint16_t u16v2_t __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(u16v2_t, a),
                                                                __builtin_bit_cast(u16v2_t, b)));
}
// x of another lane of the 16, by a DPP control word.
template <int CTRL>
__device__ __forceinline__ uint32_t dpp(uint32_t x) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, CTRL, 0xF, 0xF, false);
}

// s_waitcnt with only a vmcnt limit (vmcnt[3:0], expcnt[6:4], lgkmcnt[11:8],
// vmcnt[5:4] in bits [15:14]).
template <int N>
__device__ __forceinline__ void wait_loads() {
  static_assert(N >= 0 && N < 64, "vmcnt range");
  __builtin_amdgcn_s_waitcnt((N & 15) | (7 << 4) | (15 << 8) | ((N >> 4) << 14));
}
__device__ __forceinline__ void wait_lds() {
  __builtin_amdgcn_s_waitcnt(0xF | (7 << 4) | (0 << 8) | (3 << 14));
}
__device__ __forceinline__ void barrier() {
  __builtin_amdgcn_sched_barrier(0);
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
  __builtin_amdgcn_sched_barrier(0);
}

// Direct global-to-LDS loads: each lane moves 16 (4) bytes from base + off, the
// wave 1 KiB (256 bytes) to LDS address lds + 16 (4) lane. No memory clobber:
// the ring orders them with counted waits and barriers. s_nop: the wait state
// between the write of M0 and a load that reads it.
__device__ __forceinline__ void load_to_lds(const void* base, uint32_t off, uint32_t lds) {
  asm volatile("s_nop 0\n\tglobal_load_lds_dwordx4 %0, %1" : : "v"(off), "s"(base), "{m0}"(lds));
}
__device__ __forceinline__ void load_to_lds4(const void* base, uint32_t off, uint32_t lds) {
  asm volatile("s_nop 0\n\tglobal_load_lds_dword %0, %1" : : "v"(off), "s"(base), "{m0}"(lds));
}

// One operand of a product. Plain: `outer` rows of K contiguous elements.
// Transposed: K rows of `outer` contiguous elements.
struct Side {
  const uint8_t* p;
  int64_t ld;          // bytes between rows
  int64_t plane;       // bytes between planes
  int64_t outer;       // valid rows (plain) or columns, a multiple of 8 (transposed)
  // transposed: slots of K from tail_slot on lie tail bytes further (elsewhere:
  // the last rows of T, copied to whole slots); 0: none
  int64_t tail;
  int tail_slot;
};

struct TileArgs {
  Side A, B;           // A: the index that lies over lanes, B: over accumulators
  int nseg;            // 1, 2 (dz alone in halves) or 3 products of halves
  int slots;           // slots of 32 of K in all
  int splits;          // K is shared by this many tiles, each with a result of its own
  int nbm, nbn;        // tiles
  float c2;            // scale log2(e) / tau
  // running maximum and sum
  float2* part;        // [nbn][M]
  int64_t M, V;        // valid rows, valid columns
  // the logits that the targets name, by tile (EPI_PICK): entries of row tile r
  // and column tile c are list[r cap + starts[r (cols + 1) + c]] .. the next start
  const uint32_t* list;    // row in the tile, column in it, entry of the row: 8 bits each
  const int* starts;
  int64_t cap;
  int tiles, tile0;        // column tiles in all, of them before this launch
  float* logits;           // [M][k]
  int k;
  float zf;                // base-2 logits to logits
  const float* rowf;       // fp16 operands: c2 with the placements undone, by row
  // gradient of the logits
  const float *a, *lse2;   // [rows padded to whole tiles]
  uint16_t* dz;
  int64_t ldz, dz_plane;   // elements
  int64_t Mpad, Vpad;      // rows and columns of dz that exist
  const uint32_t* stop;    // largest |dz| at the sparse positions by column, as bits of fp32
  uint8_t* level;          // [groups of rows of a wave's tiles][ldz]
  int* any;                // set where a level is neither kFlat nor kEmpty
  // products
  void* out;
  int64_t ld_out, split_out;   // elements; between the results of two splits
  int out_bf16;
  const float* prev;   // added (nullable); may be out
  int64_t ld_prev;
  const int* row_exp;  // results times 2^(row_exp[row] + *all_exp); each nullable
  const int* row_any;  // row_exp counts where this is not 0 (nullable: always)
  const int* all_exp;
};

// EPI_DZB: dz as two bf16 halves, unplaced
enum { EPI_LSE, EPI_DZ, EPI_OUT, EPI_PICK, EPI_DZB };
constexpr int kPicks = 256;               // entries of a tile that wait in LDS

// One side's walk over K: this wave's part of every slot.
template <int BX, bool TR, int NW>
struct Walk {
  static constexpr int DMA = BX / 16 / NW;           // loads of 1 KiB a wave and slot
  static_assert(DMA >= 1 && BX % (16 * NW) == 0, "whole loads");
  static_assert(BX >= 128, "the places of a transposed slot's units");
  const uint8_t* base;
  uint32_t off[DMA];
  int64_t step;

  // A slot's row is 64 bytes of K (plain; four 16-byte chunks, chunk c of row r
  // at c ^ (r / 4) % 4) or BX elements (transposed; 64-byte units, unit u of
  // row k at u ^ k % 4): a fragment read then meets every bank of a 256-byte
  // line once.
  __device__ __forceinline__ void start(const Side& s, int64_t outer0, int slot0, int wave,
                                        int lane) {
    if constexpr (!TR) {
      const int dr = lane >> 2;
      const uint32_t chunk = (uint32_t)(((lane & 3) ^ ((dr >> 2) & 3)) * 16);
      const int64_t r0 = outer0 + wave * DMA * 16;
      const int64_t rb = r0 < s.outer ? r0 : s.outer - 1;
#pragma unroll
      for (int q = 0; q < DMA; ++q) {
        const int64_t r = r0 + q * 16 + dr;
        const int64_t rc = r < s.outer ? r : s.outer - 1;
        off[q] = (uint32_t)((rc - rb) * s.ld) + chunk;
      }
      step = 64;
      base = s.p + rb * s.ld + slot0 * 64;
    } else {
      constexpr int kChunks = BX / 8, RPI = 64 / kChunks;
      const int kr = lane / kChunks, cp = lane % kChunks;
#pragma unroll
      for (int q = 0; q < DMA; ++q) {
        const int k = (wave * DMA + q) * RPI + kr;
        int64_t col = outer0 + (cp ^ ((k & 3) * 4)) * 8;
        if (col > s.outer - 8) col = s.outer - 8;
        off[q] = (uint32_t)(k * s.ld + (col - outer0) * 2);
      }
      step = 32 * s.ld;
      base = s.p + outer0 * 2 + slot0 * step;
    }
  }
  __device__ __forceinline__ void issue(uint32_t lds, int wave) const {
#pragma unroll
    for (int q = 0; q < DMA; ++q) load_to_lds(base, off[q], lds + (wave * DMA + q) * 1024);
  }
  // fragment of 32 of the outer index from w0 on, K elements 16 t + 8 (lane / 32) ..
  __device__ __forceinline__ static bf16x8_t frag(const uint8_t* slot, int w0, int t, int lane) {
    if constexpr (!TR) {
      const int fr = lane & 31, c = t * 2 + (lane >> 5);
      return __builtin_bit_cast(
          bf16x8_t, *reinterpret_cast<const uint4*>(slot + (w0 + fr) * 64 +
                                                    ((c ^ ((fr >> 2) & 3)) * 16)));
    } else {
      // a transposing read gives lane i of 16 the i-th of 16 columns, four rows of K
      const int k = t * 16 + 8 * (lane >> 5) + ((lane & 15) >> 2);
      const uint8_t* p = slot + k * BX * 2 + (((w0 >> 5) ^ ((lane & 15) >> 2)) * 64) +
                         ((lane >> 4) & 1) * 32 + (lane & 3) * 8;
      const s16x4_t lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4_t*)p);
      const s16x4_t hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4_t*)(p + 4 * BX * 2));
      const s16x8_t v = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
      return __builtin_bit_cast(bf16x8_t, v);
    }
  }
};

// Geometry of a tile kernel: BM x BN by WGM x WGN waves of (BM / WGM) x 64.
template <int BM, int BN, int WGM, int WGN>
struct Geo {
  static constexpr int NW = WGM * WGN, NT = 64 * NW;
  static constexpr int WTM = BM / WGM, WTN = BN / WGN, FM = WTM / 32, FN = WTN / 32;
  static_assert(WTN == 64 && WTM % 32 == 0, "a wave's part");
  static constexpr int kA = BM * 64, kB = BN * 64;   // bytes of a slot
  static constexpr int kRingBytes = kRing * (kA + kB);
  // row vectors (two tiles' up to three), the waves' maxima and sums, two tiles'
  // first entries
  static constexpr int kRows = 2 * 3 * BM * 4;
  static constexpr int kRed = BM * 8 * WGN;
  static constexpr int kExtra = kRows + kRed + 2 * kPicks * 4;
  static constexpr int kLds = kRingBytes + kExtra;
  static_assert(kA + kB >= NW * 4096 || kRing * (kA + kB) >= NW * 4096, "patches");
};

// The tile of a product's numbering: groups of 8 M tiles, N-major inside, so
// that tiles running together share their panels.
__device__ __forceinline__ void tile_at(uint32_t id, uint32_t nbm, uint32_t nbn, uint32_t& bm,
                                        uint32_t& bn) {
  const uint32_t per_group = 8 * nbn, g = id / per_group, local = id - g * per_group;
  const uint32_t rows = nbm - g * 8 < 8 ? nbm - g * 8 : 8;
  bn = local / rows;
  bm = g * 8 + (local - bn * rows);
}

// Walks the tiles next(0), next(1), ... of one block (0xFFFFFFFF: none). The
// ring of four slots runs on from tile to tile: the last slots of a tile
// request the first ones of the next, all but the fourth, whose place the
// epilogue uses as scratch.
template <int EPI, bool F16, int BM, int BN, int WGM, int WGN, bool TA, bool TB, typename Next>
__device__ __forceinline__ void walk_tiles(const TileArgs& g, uint8_t* smem, Next next) {
  using G = Geo<BM, BN, WGM, WGN>;
  constexpr int NW = G::NW, FM = G::FM, FN = G::FN;
  using WA = Walk<BM, TA, NW>;
  using WB = Walk<BN, TB, NW>;
  constexpr int LS = WA::DMA + WB::DMA;
  static_assert(3 * LS < 60, "vmcnt");

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave / WGN, wn = wave % WGN;
  const int fr = lane & 31, half = lane >> 5;
  const uint32_t lds0 = (uint32_t)(uintptr_t)(const lds_void_t*)smem;
  uint8_t* const smemB = smem + kRing * G::kA;
  uint8_t* const extra = smem + G::kRingBytes;

  struct Tile { uint32_t bm, bn, split; };
  auto decode = [&](uint32_t id) {
    Tile t;
    const uint32_t mn = (uint32_t)g.nbm * g.nbn;
    t.split = g.splits > 1 ? id / mn : 0;
    tile_at(id - t.split * mn, g.nbm, g.nbn, t.bm, t.bn);
    return t;
  };
  auto slot_range = [&](uint32_t split, int& s0, int& n) {
    if (g.splits == 1) {
      s0 = 0;
      n = g.slots;
      return;
    }
    s0 = (int)((int64_t)g.slots * split / g.splits);
    n = (int)((int64_t)g.slots * (split + 1) / g.splits) - s0;
  };

  // the walk: where the next slot to request lies
  WA wa;
  WB wb;
  const uint8_t *a00 = nullptr, *b00 = nullptr;
  int seg_slots = 0, seg_at = 0, seg = 0;
  constexpr bool kTail = EPI == EPI_OUT && !TA && TB;
  int first_slot = 0;
  auto set_seg = [&] {
    wa.base = a00 + seg_a(seg) * g.A.plane;
    wb.base = b00 + seg_b(seg) * g.B.plane;
    if (kTail && g.B.tail && first_slot >= g.B.tail_slot) wb.base += g.B.tail;
    seg_at = 0;
  };
  auto start_walk = [&](const Tile& t) {
    int s0;
    slot_range(t.split, s0, seg_slots);
    first_slot = s0;
    wa.start(g.A, (int64_t)t.bm * BM, s0, wave, lane);
    wb.start(g.B, (int64_t)t.bn * BN, s0, wave, lane);
    a00 = wa.base;
    b00 = wb.base;
    seg = kSegs - g.nseg;
    set_seg();
  };
  auto issue_a = [&](int ring) { wa.issue(lds0 + ring * G::kA, wave); };
  auto issue_b = [&](int ring) {
    wb.issue(lds0 + kRing * G::kA + ring * G::kB, wave);
    wa.base += wa.step;
    wb.base += wb.step;
    ++seg_at;
    if (kTail && first_slot + seg_at == g.B.tail_slot) wb.base += g.B.tail;
    if (seg_at == seg_slots) {
      ++seg;
      if (seg < kSegs) set_seg();
    }
  };
  // a tile's row vectors into the half of its parity
  constexpr bool LSE = EPI == EPI_LSE || EPI == EPI_PICK;
  constexpr bool DZ = EPI == EPI_DZ || EPI == EPI_DZB;
  constexpr int NV = (DZ ? 2 : 0) + (EPI != EPI_OUT && F16 ? 1 : 0);
  constexpr int NC = EPI == EPI_DZ ? BN / 64 : 0;    // loads of a vector along the columns
  static_assert(2 * NC * 256 <= G::kRed, "it lies where maxima and sums do");
  auto picks_of = [&](const Tile& t, int& count) -> const uint32_t* {
    // by the scalar cache (written by an earlier launch): a vector load's wait
    // would drain the ring
    const int at = __builtin_amdgcn_readfirstlane((int)(g.tile0 + t.bn));
    const int row = __builtin_amdgcn_readfirstlane((int)t.bm);
    const int* first = g.starts + (int64_t)row * (g.tiles + 1) + at;
    const auto* s = (const __attribute__((address_space(4))) int*)first;
    const int a = s[0];
    count = s[1] - a;
    return g.list + t.bm * g.cap + a;
  };
  // and its entries, behind which the list has room for a whole load
  auto issue_rows = [&](const Tile& t, int parity) {
    if constexpr (EPI == EPI_PICK) {
      int count;
      const uint32_t* src = picks_of(t, count);
#pragma unroll
      for (int x = 0; x < kPicks / 64; ++x)
        if (x % NW == wave && x * 64 < count)
          load_to_lds4(src + x * 64, (uint32_t)lane * 4,
                       lds0 + G::kRingBytes + G::kRows + G::kRed + parity * (kPicks * 4) + x * 256);
    }
    constexpr int per = BM / 64;                     // loads of 64 rows
    if constexpr (NV > 0)
#pragma unroll
      for (int q = 0; q < (NV * per + NC + NW - 1) / NW; ++q) {
        const int x = q * NW + wave, v = x / per;
        if (NC > 0 && x >= NV * per && x < NV * per + NC) {
          const int y = x - NV * per;
          load_to_lds4(g.stop + (int64_t)t.bn * BN + y * 64, (uint32_t)lane * 4,
                       lds0 + G::kRingBytes + G::kRows + parity * (BN * 4) + y * 256);
        }
        if (x < NV * per) {
          const float* src = NV == 1 || v == 2 ? g.rowf : v == 0 ? g.a : g.lse2;
          load_to_lds4(src + (int64_t)t.bm * BM + (x % per) * 64, (uint32_t)lane * 4,
                       lds0 + G::kRingBytes + parity * (NV * BM * 4) + x * 256);
        }
      }
  };

  uint32_t id = next(0);
  if (id == 0xFFFFFFFFu) return;
  Tile cur = decode(id);
  f32x16_t acc[FM][FN];
  bf16x8_t fa[2][FM], fb[2][FN];

  issue_rows(cur, 0);
  start_walk(cur);
#pragma unroll
  for (int p = 0; p < kRing; ++p) {
    issue_a(p);
    if (p < kRing - 1) issue_b(p);
  }
  wait_loads<2 * LS + WA::DMA>();
  barrier();
  int ring0 = 0;                                     // ring place of the tile's first slot

  for (int jt = 0;; ++jt) {
    int s0, KS;
    slot_range(cur.split, s0, KS);
    KS *= g.nseg;
    const uint32_t nid = next(jt + 1);
    const bool more = nid != 0xFFFFFFFFu;
    Tile nxt = cur;
    if (more) nxt = decode(nid);

    auto read_step = [&](int s, int t, bf16x8_t (&af)[FM], bf16x8_t (&bf)[FN]) {
      const int b = (ring0 + s) & (kRing - 1);
      const uint8_t* sa = smem + b * G::kA;
      const uint8_t* sb = smemB + b * G::kB;
#pragma unroll
      for (int i = 0; i < FM; ++i) af[i] = WA::frag(sa, wm * G::WTM + i * 32, t, lane);
#pragma unroll
      for (int j = 0; j < FN; ++j) bf[j] = WB::frag(sb, wn * 64 + j * 32, t, lane);
    };
    constexpr int kReads = FM * (TA ? 2 : 1) + FN * (TB ? 2 : 1);
    constexpr int kMma = FM * FN;
    // MFMAs of a step, its fragment reads (kReads, when reads) spread between them
    auto mma = [&](int i, int j, const bf16x8_t (&af)[FM], const bf16x8_t (&bf)[FN]) {
      if constexpr (F16)
        acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8_t, bf[j]),
                                                           __builtin_bit_cast(f16x8_t, af[i]),
                                                           acc[i][j], 0, 0, 0);
      else
        acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(bf[j], af[i], acc[i][j], 0, 0, 0);
    };
    auto spread = [&](auto first) {                  // first: MFMAs already issued
      constexpr int kF = decltype(first)::value, kM = kMma - kF;
      constexpr int per = (kReads + kM - 1) / kM;
#pragma unroll
      for (int x = 0; x < kM; ++x) {
        if (x * per < kReads)
          __builtin_amdgcn_sched_group_barrier(0x100, per, 0);
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
      }
    };

#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
      for (int j = 0; j < FN; ++j)
#pragma unroll
        for (int q = 0; q < 16; ++q) acc[i][j][q] = 0.f;
    read_step(0, 0, fa[0], fb[0]);

    // Slot s: the second half of the request for slot s + 3 goes out, step 0
    // reads step 1's fragments; at the barrier slot s + 1 has landed everywhere
    // and slot s is read; step 1 starts the request of slot s + 4 into slot s's
    // place and reads slot s + 1's first fragments. From slot KS - 4 on the
    // requests are the next tile's first slots, or, behind the last tile, the
    // same tile's again, which nothing reads.
    auto step0 = [&](int s) {
      read_step(s, 1, fa[1], fb[1]);
#pragma unroll
      for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j) mma(i, j, fa[0], fb[0]);
      spread(std::integral_constant<int, 0>{});
      __builtin_amdgcn_sched_barrier(0);
      wait_loads<2 * LS>();
      wait_lds();
      barrier();
    };
    auto rest = [&] {
#pragma unroll
      for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j)
          if (i + j > 0) mma(i, j, fa[1], fb[1]);
    };
    for (int s = 0; s < KS - 1; ++s) {
      __builtin_amdgcn_sched_barrier(0);
      issue_b((ring0 + s + 3) & (kRing - 1));
      if (s == KS - 4) {
        issue_rows(nxt, (jt + 1) & 1);
        start_walk(nxt);
      }
      __builtin_amdgcn_sched_barrier(0);
      step0(s);
      mma(0, 0, fa[1], fb[1]);
      __builtin_amdgcn_sched_barrier(0);
      issue_a((ring0 + s) & (kRing - 1));
      __builtin_amdgcn_sched_barrier(0);
      read_step(s + 1, 0, fa[0], fb[0]);
      rest();
      spread(std::integral_constant<int, 1>{});
      __builtin_amdgcn_sched_barrier(0);
    }
    issue_b((ring0 + KS + 2) & (kRing - 1));
    __builtin_amdgcn_sched_barrier(0);
    step0(KS - 1);
    mma(0, 0, fa[1], fb[1]);
    rest();

    // ---- epilogue: a lane has, of each 32 x 32 block, row fr of A's index and
    // 4 of B's from 8 q + 4 half on, q = 0 .. 3
    const int free_slot = (ring0 + KS - 1) & (kRing - 1);
    uint8_t* patch;                                  // 4 KiB of the wave's own
    {
      constexpr int inA = G::kA / 4096 < NW ? G::kA / 4096 : NW;
      static_assert(inA + G::kB / 4096 >= NW, "patches");
      patch = wave < inA ? smem + free_slot * G::kA + wave * 4096
                         : smemB + free_slot * G::kB + (wave - inA) * 4096;
    }
    const int64_t m0 = (int64_t)cur.bm * BM + wm * G::WTM;
    const int64_t n0 = (int64_t)cur.bn * BN + wn * 64;

    const float* rows = reinterpret_cast<const float*>(extra) + (jt & 1) * NV * BM;
    const int live = (int)(g.V - n0 < 64 ? g.V - n0 : 64);     // columns of this wave's 64
    const bool edge = live < 64;
    if constexpr (LSE) {
      float2* red = reinterpret_cast<float2*>(extra + G::kRows);          // [WGN][BM]
      float flip = 1.f;
      if (g.c2 < 0.f) {                              // the largest logit is the smallest product
        flip = -1.f;
#pragma unroll
        for (int i = 0; i < FM; ++i)
#pragma unroll
          for (int j = 0; j < FN; ++j) acc[i][j] = -acc[i][j];
      }
#pragma unroll
      for (int i = 0; i < FM; ++i) {
        if (edge) {
          int past = live - 4 * half;
          asm volatile("" : "+v"(past));             // compared here, not held in masks all along
#pragma unroll
          for (int j = 0; j < FN; ++j)
#pragma unroll
            for (int q = 0; q < 16; ++q)
              if (j * 32 + 8 * (q >> 2) + (q & 3) >= past) acc[i][j][q] = -INFINITY;
        }
        // (never 0, so that masked columns stay -infinity under it)
        const float c2 = fmaxf(flip * (F16 ? rows[wm * G::WTM + i * 32 + fr] : g.c2), 1.2e-38f);
        float m = -INFINITY;
#pragma unroll
        for (int j = 0; j < FN; ++j)
#pragma unroll
          for (int q = 0; q < 16; ++q) m = fmaxf(m, acc[i][j][q]);
        m = fmaxf(m, __shfl_xor(m, 32));
        m *= c2;
        const float ref = m == -INFINITY ? 0.f : m;
        float sum = 0.f;
#pragma unroll
        for (int j = 0; j < FN; ++j)
#pragma unroll
          for (int q = 0; q < 16; ++q)
            sum += __builtin_amdgcn_exp2f(fmaf(acc[i][j][q], c2, -ref));
        sum += __shfl_xor(sum, 32);
        if (half == 0) red[wn * BM + wm * G::WTM + i * 32 + fr] = make_float2(m, sum);
      }
      if constexpr (EPI == EPI_PICK) {
        int count;
        const uint32_t* src = picks_of(cur, count);
        const auto* near = reinterpret_cast<const uint32_t*>(extra + G::kRows + G::kRed) +
                           (jt & 1) * kPicks;
        // block by block through the wave's scratch, 64 entries at a time
        auto entry = [&](int x) -> uint32_t {
          const uint32_t e = x + lane >= count ? 0xFFFFFFFFu
                             : x < kPicks ? near[x + lane] : src[x + lane];
          return (e & 255) / G::WTM == (uint32_t)wm && ((e >> 8) & 255) / 64 == (uint32_t)wn
                     ? e : 0xFFFFFFFFu;
        };
        uint64_t blocks = 0;                         // of this wave's, those with entries
        for (int x = 0; x < count; x += 64) {
          const uint32_t e = entry(x);
          const int at = (int)(e & 255) % G::WTM / 32 * FN + (int)((e >> 8) & 63) / 32;
#pragma unroll
          for (int t = 0; t < FM * FN; ++t)
            if (__any(e != 0xFFFFFFFFu && at == t)) blocks |= 1ull << t;
        }
        float* z = reinterpret_cast<float*>(patch);
#pragma unroll
        for (int i = 0; i < FM; ++i)
#pragma unroll
          for (int j = 0; j < FN; ++j)
            if (blocks >> (i * FN + j) & 1) {
              const float f = flip * (F16 ? rows[wm * G::WTM + i * 32 + fr] : g.c2) * g.zf;
              wave_sync();
              // 16-byte chunk c of row r at c ^ r % 8
#pragma unroll
              for (int q = 0; q < 4; ++q)
                *reinterpret_cast<float4*>(z + fr * 32 + (((2 * q + half) ^ (fr & 7)) * 4)) =
                    make_float4(acc[i][j][4 * q] * f, acc[i][j][4 * q + 1] * f,
                                acc[i][j][4 * q + 2] * f, acc[i][j][4 * q + 3] * f);
              wave_sync();
              for (int x = 0; x < count; x += 64) {
                const uint32_t e = entry(x);
                const int r = e & 255, c = (e >> 8) & 63;
                if (e != 0xFFFFFFFFu && r % G::WTM / 32 == i && c / 32 == j)
                  g.logits[((int64_t)cur.bm * BM + r) * g.k + (e >> 16)] =
                      z[(r & 31) * 32 + ((((c & 31) >> 2) ^ (r & 7)) * 4) + (c & 3)];
              }
            }
      }
      wait_lds();
      barrier();
      for (int r = tid; r < BM; r += G::NT) {
        float m = -INFINITY, sum = 0.f;
#pragma unroll
        for (int w = 0; w < WGN; ++w) m = fmaxf(m, red[w * BM + r].x);
        const float ref = m == -INFINITY ? 0.f : m;
#pragma unroll
        for (int w = 0; w < WGN; ++w)
          sum += red[w * BM + r].y * __builtin_amdgcn_exp2f(red[w * BM + r].x - ref);
        const int64_t row = (int64_t)cur.bm * BM + r;
        if (row < g.M) g.part[(int64_t)cur.bn * g.M + row] = make_float2(m, sum);
      }
    } else if constexpr (DZ) {
      constexpr bool kApart = F16 || EPI == EPI_DZB;  // stored in halves
#pragma unroll
      for (int i = 0; i < FM; ++i) {
        const float a = rows[wm * G::WTM + i * 32 + fr];
        const float l = rows[BM + wm * G::WTM + i * 32 + fr];
        const float c2 = F16 ? rows[2 * BM + wm * G::WTM + i * 32 + fr] : g.c2;
#pragma unroll
        for (int j = 0; j < FN; ++j)
#pragma unroll
          for (int q = 0; q < 16; ++q)
            acc[i][j][q] = a * __builtin_amdgcn_exp2f(fmaf(acc[i][j][q], c2, -l));
        // columns behind the last row of T, and rows without weight, give zeros
        // whatever their logits are
        if (edge || __any(a == 0.f)) {
          int past = a == 0.f ? 0 : live - 4 * half;
          asm volatile("" : "+v"(past));             // compared here, not held in masks all along
#pragma unroll
          for (int j = 0; j < FN; ++j)
#pragma unroll
            for (int q = 0; q < 16; ++q)
              if (j * 32 + 8 * (q >> 2) + (q & 3) >= past) acc[i][j][q] = 0.f;
        }
      }
      if constexpr (EPI == EPI_DZ) {
        // largest |dz| of each of the wave's columns: two columns' upper 16 bits a
        // word, halved over the lanes' rows until a pair of lanes has one word,
        // columns (fr / 16) 32 + (fr / 4 % 4) 8 + 4 half + fr / 2 % 2 2 and the next
        uint32_t w[16];
#pragma unroll
        for (int t = 0; t < 16; ++t) {
          float m[2] = {0.f, 0.f};
#pragma unroll
          for (int i = 0; i < FM; ++i)
#pragma unroll
            for (int u = 0; u < 2; ++u) m[u] = fmaxf(m[u], fabsf(acc[i][t >> 3][(t & 7) * 2 + u]));
          w[t] = (__float_as_uint(m[0]) >> 16) | (__float_as_uint(m[1]) & 0xFFFF0000u);
        }
#pragma unroll
        for (int t = 0; t < 8; ++t) {                // lanes 16 apart
          const auto x = __builtin_amdgcn_permlane16_swap(w[t], w[t + 8], false, false);
          w[t] = max_u16x2(x[0], x[1]);
        }
        auto halve = [&](auto n, auto ctrl, int bit) {
          const bool up = (fr >> bit) & 1;
#pragma unroll
          for (int t = 0; t < decltype(n)::value; ++t) {
            const uint32_t x = w[t], y = w[t + decltype(n)::value];
            w[t] = max_u16x2(up ? y : x, dpp<decltype(ctrl)::value>(up ? x : y));
          }
        };
        halve(std::integral_constant<int, 4>{}, std::integral_constant<int, 0x128>{}, 3);  // 8 apart
        halve(std::integral_constant<int, 2>{}, std::integral_constant<int, 0x141>{}, 2);  // 8 mirrored
        halve(std::integral_constant<int, 1>{}, std::integral_constant<int, 0x4E>{}, 1);   // 2 apart
        w[0] = max_u16x2(w[0], dpp<0xB1>(w[0]));                                           // next
        const int col = (fr >> 4) * 32 + ((fr >> 2) & 3) * 8 + half * 4 + ((fr >> 1) & 1) * 2;
        const auto* stop = reinterpret_cast<const uint32_t*>(extra + G::kRows) + (jt & 1) * BN +
                           wn * 64 + col;
        w[0] = max_u16x2(w[0], (stop[0] >> 16) | (stop[1] & 0xFFFF0000u));
        const uint32_t l0 = level_of(w[0] & 0xFFFFu), l1 = level_of(w[0] >> 16);
        const uint16_t both = (uint16_t)(l0 | l1 << 8);
        if ((fr & 1) == 0 && n0 < g.Vpad)
          *reinterpret_cast<uint16_t*>(g.level + ((int64_t)cur.bm * WGM + wm) * g.ldz + n0 + col) =
              both;
        if (__any((l0 != kFlat && l0 != kEmpty) || (l1 != kFlat && l1 != kEmpty))) {
          if (lane == 0) *g.any = 1;
          wave_sync();
          *reinterpret_cast<uint16_t*>(patch + col) = both;
          wave_sync();
#pragma unroll
          for (int j = 0; j < FN; ++j)
#pragma unroll
            for (int q = 0; q < 16; ++q) {
              const uint32_t l = patch[j * 32 + 8 * (q >> 2) + 4 * half + (q & 3)];
              const float f = __uint_as_float((127u + (l == kEmpty ? 0u : l)) << 23);
#pragma unroll
              for (int i = 0; i < FM; ++i) acc[i][j][q] *= f;
            }
        }
      }
#pragma unroll
      for (int i = 0; i < FM; ++i) {
#pragma unroll
        for (int p = 0; p < (kApart ? 2 : 1); ++p) {
          wave_sync();
          // rows of 128 bytes, 16-byte chunk c of row r at c ^ r % 8
#pragma unroll
          for (int j = 0; j < FN; ++j)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              using H = Half<EPI != EPI_DZB>;
              const uint32_t lo = H::pack(acc[i][j][4 * q], acc[i][j][4 * q + 1]);
              const uint32_t hi = H::pack(acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]);
              if (kApart) {           // what the high half leaves
                acc[i][j][4 * q] -= H::lo(lo);
                acc[i][j][4 * q + 1] -= H::hi(lo);
                acc[i][j][4 * q + 2] -= H::lo(hi);
                acc[i][j][4 * q + 3] -= H::hi(hi);
              }
              *reinterpret_cast<uint2*>(patch + fr * 128 + (((j * 4 + q) ^ (fr & 7)) * 16) +
                                        half * 8) = make_uint2(lo, hi);
            }
          wave_sync();
          if (n0 < g.Vpad) {
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              const int r = x * 8 + (lane >> 3), c = lane & 7;
              const uint4 v =
                  *reinterpret_cast<const uint4*>(patch + r * 128 + ((c ^ (r & 7)) * 16));
              const int64_t row = m0 + i * 32 + r;
              if (row < g.Mpad)
                store16<true>(g.dz + p * g.dz_plane + row * g.ldz + n0 + c * 8, v.x, v.y, v.z, v.w);
            }
          }
        }
      }
    } else {
      const int64_t so = (int64_t)cur.split * g.split_out;
      const int all_exp = g.all_exp ? *g.all_exp : 0;
      const bool by_row = g.row_exp && !(g.row_any && *g.row_any == 0);
#pragma unroll
      for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j) {
          if (i + j > 0) wave_sync();
#pragma unroll
          for (int q = 0; q < 4; ++q)
            *reinterpret_cast<float4*>(patch + fr * 128 + (((2 * q + half) ^ (fr & 7)) * 16)) =
                make_float4(acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2],
                            acc[i][j][4 * q + 3]);
          wave_sync();
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const int r = x * 8 + (lane >> 3), c = lane & 7;
            const float4 f =
                *reinterpret_cast<const float4*>(patch + r * 128 + ((c ^ (r & 7)) * 16));
            const int64_t row = m0 + i * 32 + r, col = n0 + j * 32 + c * 4;
            const int left = (int)(g.V - col < 4 ? g.V - col : 4);
            if (row >= g.M || left <= 0) continue;
            const int e = all_exp + (by_row ? g.row_exp[row] : 0);
            float v[4] = {ldexpf(f.x, e), ldexpf(f.y, e), ldexpf(f.z, e), ldexpf(f.w, e)};
            if (g.prev) {
              const float* pv = g.prev + row * g.ld_prev + col;
              if (left == 4) {
                float t[4];
                __builtin_memcpy(t, pv, 16);
#pragma unroll
                for (int u = 0; u < 4; ++u) v[u] += t[u];
              } else {
#pragma unroll
                for (int u = 0; u < 4; ++u)
                  if (u < left) v[u] += pv[u];
              }
            }
            if (g.out_bf16) {
              uint16_t* o = static_cast<uint16_t*>(g.out) + so + row * g.ld_out + col;
              const uint2 w = make_uint2(pack2_bf16(v[0], v[1]), pack2_bf16(v[2], v[3]));
              if (left == 4) {
                __builtin_memcpy(o, &w, 8);
              } else {
#pragma unroll
                for (int u = 0; u < 4; ++u)
                  if (u < left) o[u] = (uint16_t)(((u & 2) ? w.y : w.x) >> (16 * (u & 1)));
              }
            } else {
              float* o = static_cast<float*>(g.out) + so + row * g.ld_out + col;
              if (left == 4) {
                __builtin_memcpy(o, v, 16);
              } else {
#pragma unroll
                for (int u = 0; u < 4; ++u)
                  if (u < left) o[u] = v[u];
              }
            }
          }
        }
    }
    if (!more) {
      wait_loads<0>();                               // no load lands behind the block's end
      return;
    }
    // every wave is done with the scratch: the next tile's fourth slot may land there
    wait_lds();
    barrier();
    ring0 = (ring0 + KS) & (kRing - 1);
    cur = nxt;
    issue_a((ring0 + 3) & (kRing - 1));
  }
}

// One product's tiles. Consecutive tile numbers run on one of the 8 XCDs and
// share panels in its L2; a block walks every 1/8 grid-th of its XCD's range.
template <int EPI, bool F16, int BM, int BN, int WGM, int WGN>
__global__ __launch_bounds__(64 * WGM * WGN, 2) void head_tile_kernel(TileArgs g) {
  __shared__ __attribute__((aligned(1024))) uint8_t smem[Geo<BM, BN, WGM, WGN>::kLds];
  const uint32_t total = (uint32_t)g.nbm * g.nbn * g.splits, per = total / 8;
  const uint32_t grid = gridDim.x;
  auto next = [&](int j) -> uint32_t {
    if (grid == total) {                             // a tile each
      if (j > 0) return 0xFFFFFFFFu;
      const uint32_t b = blockIdx.x;
      return b < per * 8 ? (b & 7) * per + (b >> 3) : b;
    }
    const uint32_t g8 = grid / 8, xcd = blockIdx.x & 7, c = blockIdx.x >> 3;
    const uint32_t n_main = c < per ? (per - c + g8 - 1) / g8 : 0;
    if ((uint32_t)j < n_main) return xcd * per + c + g8 * j;
    if ((uint32_t)j == n_main && blockIdx.x < total - 8 * per) return 8 * per + blockIdx.x;
    return 0xFFFFFFFFu;
  };
  walk_tiles<EPI, F16, BM, BN, WGM, WGN, false, false>(g, smem, next);
}

// Both gradients' products of a piece in one launch: nw blocks of dT = dz^T h
// (both operands transposed) and nh of dh = dz T, whichever has the longer K
// first. Where K is short a block takes `per` tiles in a row, the next one's
// first slots under way in the last one's epilogue (MANY; 185 tokens of 105,456
// x 545: 181 us, 211 a tile each; the walk itself costs a long product 1 %).
template <bool F16, bool MANY, int BM, int BN, int WGM, int WGN>
__global__ __launch_bounds__(64 * WGM * WGN, 2) void head_grad_kernel(TileArgs w, TileArgs h,
                                                                   uint32_t nw, uint32_t nh,
                                                                   uint32_t per_w, uint32_t per_h) {
  __shared__ __attribute__((aligned(1024))) uint8_t smem[Geo<BM, BN, WGM, WGN>::kLds];
  auto one = [](uint32_t b, uint32_t total) {
    const uint32_t per = total / 8;
    return b < per * 8 ? (b & 7) * per + (b >> 3) : b;
  };
  const bool w_first = w.slots / w.splits > h.slots / h.splits;
  const uint32_t b = blockIdx.x;
  const bool is_w = w_first ? b < nw : b >= nh;
  const uint32_t id = (is_w ? one(w_first ? b : b - nh, nw) : one(w_first ? b - nw : b, nh)) *
                      (is_w ? per_w : per_h);
  const TileArgs& g = is_w ? w : h;
  const uint32_t total = (uint32_t)g.nbm * g.nbn * g.splits, per = is_w ? per_w : per_h;
  auto next = [&](int j) -> uint32_t {
    if constexpr (!MANY) return j ? 0xFFFFFFFFu : id;
    return (uint32_t)j < per && id + j < total ? id + j : 0xFFFFFFFFu;
  };
  if (is_w)
    walk_tiles<EPI_OUT, F16, BM, BN, WGM, WGN, true, true>(w, smem, next);
  else
    walk_tiles<EPI_OUT, F16, BM, BN, WGM, WGN, false, true>(h, smem, next);
}

}  // namespace
}  // namespace pg
