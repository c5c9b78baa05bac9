// Losses of the head over a large vocabulary (gfx950): cross entropy and
// distillation from a teacher's largest logits, forward and backward.
//
//   z_nv = scale h_n . T_v            (T: the token table, tied)
//   lse_n = log sum_v exp(z_nv / tau)
//   dz_nv = a_n exp(z_nv / tau - lse_n) - (sparse part)
//   dh = dz T,  dT = dz^T h
//
// The logits are never kept. Forward: tiles of 256 tokens x 256 rows of the
// table on the matrix cores; a tile leaves one running maximum and sum a
// token, a second kernel joins them along the vocabulary and takes the few
// logits that the targets name as dot products of their own. Backward, piece
// by piece of the vocabulary: the tiles again, now with the softmax's
// statistics known, leave dz of the piece; the sparse positions are written
// over it with values rounded once; then one launch forms both products of the
// piece, dh adding up in fp32 from piece to piece.
//
// Number formats. bf16 operands enter the logits as they are. dz is held in
// fp16, not bf16: it is the sum's dominant rounding (bf16 took dh from 1.7e-3
// to 2.6e-3 off in the 2-norm, of which 1.65e-3 is the result's own rounding;
// fp16 leaves it there). Powers of two keep it in range: each row of dz is
// placed by its own bound, which dh's rows undo; h for dT carries the inverse of
// its row's placement, T is placed by its largest element. So a product's
// second operands are fp16 copies of h and T, exact for bf16 values down to
// 2^-31 of the largest. fp32 operands, and dz with them, are two fp16 halves
// (22 bits), multiplied as hi lo, lo hi and hi hi, one K three times as long;
// h for the logits is placed row by row.
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
  int nseg;            // 1, or 3 products of halves
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
  // products
  void* out;
  int64_t ld_out, split_out;   // elements; between the results of two splits
  int out_bf16;
  const float* prev;   // added (nullable); may be out
  int64_t ld_prev;
  const int* row_exp;  // results times 2^(row_exp[row] + *all_exp); each nullable
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
  const uint8_t* base;
  uint32_t off[DMA];
  int64_t step;

  // A slot's row is 64 bytes of K (plain; four 16-byte chunks, chunk c of row r
  // at c ^ (r / 4) % 4) or BX elements (transposed; 64-byte units, unit u of
  // row k at u ^ k % 4, or u ^ (k / 2) % 2 where a row has only two): a
  // fragment read then meets every bank of a 256-byte line once.
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
        const int f = BX >= 128 ? (k & 3) : ((k >> 1) & 1);
        int64_t col = outer0 + (cp ^ (f * 4)) * 8;
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
      const int f = BX >= 128 ? ((lane & 15) >> 2) : ((lane & 15) >> 3);
      const uint8_t* p = slot + k * BX * 2 + (((w0 >> 5) ^ f) * 64) + ((lane >> 4) & 1) * 32 +
                         (lane & 3) * 8;
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
  auto picks_of = [&](const Tile& t, int& count) -> const uint32_t* {
    const int* s = g.starts + (int64_t)t.bm * (g.tiles + 1) + g.tile0 + t.bn;
    const int a = __builtin_amdgcn_readfirstlane(s[0]);
    count = __builtin_amdgcn_readfirstlane(s[1]) - a;
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
      for (int q = 0; q < (NV * per + NW - 1) / NW; ++q) {
        const int x = q * NW + wave, v = x / per;
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
#pragma unroll
        for (int p = 0; p < (F16 || EPI == EPI_DZB ? 2 : 1); ++p) {
          if (i + p > 0) wave_sync();
          // rows of 128 bytes, 16-byte chunk c of row r at c ^ r % 8
#pragma unroll
          for (int j = 0; j < FN; ++j)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              using H = Half<EPI != EPI_DZB>;
              const uint32_t lo = H::pack(acc[i][j][4 * q], acc[i][j][4 * q + 1]);
              const uint32_t hi = H::pack(acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]);
              if (F16 || EPI == EPI_DZB) {           // what the high half leaves
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
              const uint4 v = *reinterpret_cast<const uint4*>(patch + r * 128 + ((c ^ (r & 7)) * 16));
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
            const int e = all_exp + (g.row_exp ? g.row_exp[row] : 0);
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

// ---------------------------------------------------------------------------
// Few tokens

// Maxima and sums of few tokens over 128 rows of the table: what counts is
// reading the table once, from where it lies and whatever its width. Blocks of
// up to 64 tokens, those of one tile of the table next to each other. A wave has
// 32 rows to itself and takes the fragments of 16 x 16 x 32 products straight
// from memory, 16 rows by 64 bytes a load; the next 128 of K are under way
// while the last are multiplied. No barrier until the end. (Fragments of
// 32 x 32 x 16, 32 bytes a row, read at 4.0 TB/s, 64 bytes at 6.1, as whole
// rows would.) fp32 operands are split in registers into three bf16 planes (24
// bits), six products for one, so nothing has to be placed or copied.
struct FewArgs {
  const void *h, *table;
  int64_t ld, n, V;
  int d, groups;           // of 64 tokens
  float c2;
  float2* part;            // [tiles of 128 rows][n]
};

// dz instead of maxima and sums: rows_pad rows, zeros behind the tokens and
// behind the table.
struct FewDz {
  const float *a, *lse2;
  uint16_t* dz;
  int64_t ldz, plane;      // elements
  int rows_pad;
};
// dz of token tok at four columns from col on, from their logits in base 2; MODE
// 1: fp16, two halves where F32; 2: two bf16 halves.
template <int MODE, bool F32>
__device__ __forceinline__ void few_dz(const FewDz& z, int64_t tok, int64_t n, int64_t col,
                                       const float (&v)[4]) {
  using H = Half<MODE == 1>;
  const float a = tok < n ? z.a[tok] : 0.f, l = tok < n ? z.lse2[tok] : 0.f;
  float f[4];
#pragma unroll
  for (int q = 0; q < 4; ++q) f[q] = a == 0.f ? 0.f : a * __builtin_amdgcn_exp2f(v[q] - l);
  const uint2 w = make_uint2(H::pack(f[0], f[1]), H::pack(f[2], f[3]));
  uint16_t* to = z.dz + tok * z.ldz + col;
  *reinterpret_cast<uint2*>(to) = w;
  if constexpr (F32 || MODE == 2)
    *reinterpret_cast<uint2*>(to + z.plane) =
        make_uint2(H::pack(f[0] - H::lo(w.x), f[1] - H::hi(w.x)),
                   H::pack(f[2] - H::lo(w.y), f[3] - H::hi(w.y)));
}
// Zeros in dz's rows from `from` on, `cols` (a multiple of 4) from col on; by the block.
template <int MODE, bool F32>
__device__ __forceinline__ void few_dz_zero(const FewDz& z, int from, int64_t col, int cols) {
  const int per = cols / 4;
  for (int i = threadIdx.x; i < (z.rows_pad - from) * per; i += 256) {
    uint16_t* to = z.dz + (from + i / per) * z.ldz + col + i % per * 4;
    *reinterpret_cast<uint2*>(to) = make_uint2(0, 0);
    if constexpr (F32 || MODE == 2) *reinterpret_cast<uint2*>(to + z.plane) = make_uint2(0, 0);
  }
}

// A fragment of 8 elements as bf16 (fp32: its three planes).
template <typename T>
__device__ __forceinline__ void planes_of(const Raw8<T>& v, uint4 (&f)[sizeof(T) == 4 ? 3 : 1]) {
  if constexpr (sizeof(T) == 4) {
    float x[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) x[u] = v.v[u];
#pragma unroll
    for (int p = 0; p < 3; ++p) {
      uint32_t w[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        w[u] = pack2_bf16(x[2 * u], x[2 * u + 1]);
        x[2 * u] -= __uint_as_float(w[u] << 16);
        x[2 * u + 1] -= __uint_as_float(w[u] & 0xFFFF0000u);
      }
      f[p] = make_uint4(w[0], w[1], w[2], w[3]);
    }
  } else {
    f[0] = make_uint4(v.w[0], v.w[1], v.w[2], v.w[3]);
  }
}
// acc += w h of two fragments' planes, small products first.
template <int P>
__device__ __forceinline__ void mma_planes(const uint4 (&w)[P], const uint4 (&h)[P], f32x4_t& acc) {
  auto mma = [&](int a, int b) {
    acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, w[a]),
                                                  __builtin_bit_cast(bf16x8_t, h[b]), acc, 0, 0, 0);
  };
  if constexpr (P == 3) {
    mma(2, 0);
    mma(0, 2);
    mma(1, 1);
    mma(1, 0);
    mma(0, 1);
  }
  mma(0, 0);
}

template <typename T, int TB, int DZ>
__global__ __launch_bounds__(256, 2) void head_few_kernel(FewArgs g, FewDz dz) {
  constexpr bool F32 = sizeof(T) == 4;
  constexpr int ST = F32 ? 2 : 4;                    // steps of 32 of K under way
  constexpr int P = F32 ? 3 : 1, KC = 32 * ST;
  constexpr int RB = KC * 2;                         // bytes of a token's row in LDS
  constexpr int CH = 16 * TB * KC / 8;               // its 8-element chunks in all
  constexpr int HL = (CH + 255) / 256;               // of them a thread
  __shared__ __attribute__((aligned(256))) uint8_t hs[2][P][16 * TB * RB];
  __shared__ float2 red[4][16 * TB];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, fr = lane & 15, kq = lane >> 4;
  // a tile's groups run 8 blocks apart: on one XCD, where they share its L2
  const uint32_t id = blockIdx.x;
  const uint32_t grp = g.groups == 1 ? 0 : (id >> 3) % g.groups;
  const uint32_t tile = g.groups == 1 ? id : (id >> 3) / g.groups * 8 + (id & 7);
  if (DZ == 0 && (int64_t)tile * 128 >= g.V) return;
  const int64_t v0 = (int64_t)tile * 128 + wave * 32, x0 = (int64_t)grp * 64;
  const T* wp[2];
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    const int64_t v = v0 + r * 16 + fr;
    wp[r] = static_cast<const T*>(g.table) + (v < g.V ? v : g.V - 1) * g.d + kq * 8;
  }
  // 16-byte chunk c of token x in LDS: the 16 tokens a read serves together
  // meet every bank once
  auto place = [](int x, int c) {
    return RB == 256 ? x * 256 + ((c ^ (x & 15)) * 16) : x * 128 + ((c ^ ((x >> 1) & 7)) * 16);
  };
  const T* hp[HL];
  int hc[HL];
#pragma unroll
  for (int u = 0; u < HL; ++u) {
    const int i = u * 256 + threadIdx.x, x = i / (KC / 8);
    hc[u] = i % (KC / 8) * 8;
    hp[u] = static_cast<const T*>(g.h) + (x0 + x < g.n ? x0 + x : g.n - 1) * g.ld + hc[u];
  }
  f32x4_t acc[TB][2] = {};
  Raw8<T> hr[HL], wr[2][ST][2];
  auto load = [&](int k, Raw8<T> (&w)[ST][2]) {
    const bool all = k + KC <= g.d;
#pragma unroll
    for (int u = 0; u < HL; ++u)
      if (HL * 256 == CH || u * 256 + (int)threadIdx.x < CH)
        hr[u] = load8(hp[u] + k, all ? 8 : g.d - k - hc[u]);
#pragma unroll
    for (int s = 0; s < ST; ++s)
#pragma unroll
      for (int r = 0; r < 2; ++r)
        w[s][r] = load8(wp[r] + k + s * 32, all ? 8 : g.d - k - s * 32 - kq * 8);
  };
  auto stage = [&](int buf) {
#pragma unroll
    for (int u = 0; u < HL; ++u) {
      const int i = u * 256 + threadIdx.x;
      if (HL * 256 == CH || i < CH) {
        uint4 f[P];
        planes_of(hr[u], f);
#pragma unroll
        for (int p = 0; p < P; ++p)
          *reinterpret_cast<uint4*>(hs[buf][p] + place(i / (KC / 8), i % (KC / 8))) = f[p];
      }
    }
  };
  auto multiply = [&](int buf, const Raw8<T> (&w)[ST][2]) {
#pragma unroll
    for (int s = 0; s < ST; ++s) {
      uint4 wf[2][P];
#pragma unroll
      for (int r = 0; r < 2; ++r) planes_of(w[s][r], wf[r]);
#pragma unroll
      for (int t = 0; t < TB; ++t) {
        uint4 hf[P];
#pragma unroll
        for (int p = 0; p < P; ++p)
          hf[p] = *reinterpret_cast<const uint4*>(hs[buf][p] + place(t * 16 + fr, s * 4 + kq));
#pragma unroll
        for (int r = 0; r < 2; ++r) mma_planes(wf[r], hf, acc[t][r]);
      }
    }
  };
  // One barrier a chunk: a buffer is written again two chunks on, behind the
  // barrier that every wave reaches with its reads of it done.
  const int chunks = (g.d + KC - 1) / KC;
  int at = (int)(tile % chunks);                     // tiles start apart
  auto chunk = [&](int c, int buf, const Raw8<T> (&w)[ST][2], Raw8<T> (&next)[ST][2]) {
    stage(buf);
    at = at + 1 == chunks ? 0 : at + 1;
    if (c + 1 < chunks) load(at * KC, next);
    wait_lds();
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    multiply(buf, w);
  };
  load(at * KC, wr[0]);
  for (int c = 0; c < chunks; c += 2) {
    chunk(c, 0, wr[0], wr[1]);
    if (c + 1 < chunks) chunk(c + 1, 1, wr[1], wr[0]);
  }

  // a lane has rows 16 r + 4 kq + q of the wave's 32, token 16 t + fr
#pragma unroll
  for (int t = 0; t < TB; ++t) {
    float z[2][4], m = -INFINITY;
    if constexpr (DZ != 0) {
#pragma unroll
      for (int r = 0; r < 2; ++r) {
#pragma unroll
        for (int q = 0; q < 4; ++q)
          z[r][q] = v0 + r * 16 + 4 * kq + q < g.V ? acc[t][r][q] * g.c2 : -INFINITY;
        few_dz<DZ, F32>(dz, t * 16 + fr, g.n, v0 + r * 16 + 4 * kq, z[r]);
      }
      continue;
    }
#pragma unroll
    for (int r = 0; r < 2; ++r)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        z[r][q] = v0 + r * 16 + 4 * kq + q < g.V ? acc[t][r][q] * g.c2 : -INFINITY;
        m = fmaxf(m, z[r][q]);
      }
    m = fmaxf(m, __shfl_xor(m, 16));
    m = fmaxf(m, __shfl_xor(m, 32));
    const float ref = m == -INFINITY ? 0.f : m;
    float s = 0.f;
#pragma unroll
    for (int r = 0; r < 2; ++r)
#pragma unroll
      for (int q = 0; q < 4; ++q) s += __builtin_amdgcn_exp2f(z[r][q] - ref);
    s += __shfl_xor(s, 16);
    s += __shfl_xor(s, 32);
    if (kq == 0) red[wave][t * 16 + fr] = make_float2(m, s);
  }
  if constexpr (DZ != 0) {
    few_dz_zero<DZ, F32>(dz, 16 * TB, (int64_t)tile * 128, 128);
    return;
  }
  __syncthreads();
  const int x = threadIdx.x;
  if (x < 16 * TB && x0 + x < g.n) {
    float m = -INFINITY, s = 0.f;
#pragma unroll
    for (int w = 0; w < 4; ++w) m = fmaxf(m, red[w][x].x);
    const float ref = m == -INFINITY ? 0.f : m;
#pragma unroll
    for (int w = 0; w < 4; ++w) s += red[w][x].y * __builtin_amdgcn_exp2f(red[w][x].x - ref);
    g.part[(int64_t)tile * g.n + x0 + x] = make_float2(m, s);
  }
}

// The same where the table is short too and blocks of 128 rows would leave most
// of the chip idle: a block has 32 rows, its four waves share K and their sums
// meet in LDS, so a chain of loads is a quarter as long. Fragments of the tokens
// come straight from memory here. DZ: leaves dz (rows_pad rows, zeros behind the
// tokens and behind the table) instead of maxima and sums.
template <typename T, int TB, int DZ>
__global__ __launch_bounds__(256, sizeof(T) == 4 && TB == 4 ? 1 : 2) void head_few_split_kernel(FewArgs g, FewDz z) {
  constexpr bool F32 = sizeof(T) == 4;
  constexpr int ST = F32 ? 2 : 4, P = F32 ? 3 : 1, KC = 32 * ST;
  __shared__ f32x4_t join[4][TB * 2][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, fr = lane & 15, kq = lane >> 4;
  const int64_t v0 = (int64_t)blockIdx.x * 32;
  const T *wp[2], *hp[TB];
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    const int64_t v = v0 + r * 16 + fr;
    wp[r] = static_cast<const T*>(g.table) + (v < g.V ? v : g.V - 1) * g.d + kq * 8;
  }
#pragma unroll
  for (int t = 0; t < TB; ++t) {
    const int64_t x = t * 16 + fr;
    hp[t] = static_cast<const T*>(g.h) + (x < g.n ? x : g.n - 1) * g.ld + kq * 8;
  }
  f32x4_t acc[TB][2] = {};
  struct Step {
    Raw8<T> w[2], h[TB];
  };
  auto load = [&](int k, Step (&to)[ST]) {
    const bool all = k + KC <= g.d;
#pragma unroll
    for (int s = 0; s < ST; ++s) {
      const int left = all ? 8 : g.d - k - s * 32 - kq * 8;
#pragma unroll
      for (int r = 0; r < 2; ++r) to[s].w[r] = load8(wp[r] + k + s * 32, left);
#pragma unroll
      for (int t = 0; t < TB; ++t) to[s].h[t] = load8(hp[t] + k + s * 32, left);
    }
  };
  auto multiply = [&](const Step (&x)[ST]) {
#pragma unroll
    for (int s = 0; s < ST; ++s) {
      uint4 wf[2][P];
#pragma unroll
      for (int r = 0; r < 2; ++r) planes_of(x[s].w[r], wf[r]);
#pragma unroll
      for (int t = 0; t < TB; ++t) {
        uint4 hf[P];
        planes_of(x[s].h[t], hf);
#pragma unroll
        for (int r = 0; r < 2; ++r) mma_planes(wf[r], hf, acc[t][r]);
      }
    }
  };
  Step x[2][ST];
  int k = wave * KC;
  if (k < g.d) load(k, x[0]);
  for (; k < g.d; k += 8 * KC) {
    if (k + 4 * KC < g.d) load(k + 4 * KC, x[1]);
    multiply(x[0]);
    if (k + 4 * KC < g.d) {
      if (k + 8 * KC < g.d) load(k + 8 * KC, x[0]);
      multiply(x[1]);
    }
  }
#pragma unroll
  for (int t = 0; t < TB; ++t)
#pragma unroll
    for (int r = 0; r < 2; ++r) join[wave][t * 2 + r][lane] = acc[t][r];
  __syncthreads();
  // wave t has token block t from here on: rows 16 r + 4 kq + q, token 16 t + fr
  if (wave < TB) {
    const int64_t tok = wave * 16 + fr;
    float v[2][4], m = -INFINITY;
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const f32x4_t sum = (join[0][wave * 2 + r][lane] + join[1][wave * 2 + r][lane]) +
                          (join[2][wave * 2 + r][lane] + join[3][wave * 2 + r][lane]);
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        v[r][q] = v0 + r * 16 + 4 * kq + q < g.V ? sum[q] * g.c2 : -INFINITY;
        m = fmaxf(m, v[r][q]);
      }
    }
    if constexpr (DZ == 0) {
      m = fmaxf(m, __shfl_xor(m, 16));
      m = fmaxf(m, __shfl_xor(m, 32));
      const float ref = m == -INFINITY ? 0.f : m;
      float s = 0.f;
#pragma unroll
      for (int r = 0; r < 2; ++r)
#pragma unroll
        for (int q = 0; q < 4; ++q) s += __builtin_amdgcn_exp2f(v[r][q] - ref);
      s += __shfl_xor(s, 16);
      s += __shfl_xor(s, 32);
      if (kq == 0 && tok < g.n) g.part[(int64_t)blockIdx.x * g.n + tok] = make_float2(m, s);
    } else {
#pragma unroll
      for (int r = 0; r < 2; ++r) few_dz<DZ, F32>(z, tok, g.n, v0 + r * 16 + 4 * kq, v[r]);
    }
  }
  if constexpr (DZ != 0) few_dz_zero<DZ, F32>(z, 16 * TB, v0, 32);
}

// ---------------------------------------------------------------------------
// Rows

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) v += __shfl_xor(v, o);
  return v;
}
__device__ __forceinline__ float wave_max(float v) {
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) v = fmaxf(v, __shfl_xor(v, o));
  return v;
}

// Dot product of two rows of d elements by one wave, in every lane.
template <typename T>
__device__ __forceinline__ float row_dot(const T* x, const T* y, int d, int lane) {
  float s = 0.f;
  int c = lane * 8;
#pragma unroll 4
  for (; c + 8 <= d; c += 512) {
    const Raw8<T> a = load8(x + c, 8), b = load8(y + c, 8);
#pragma unroll
    for (int u = 0; u < 8; ++u) s = fmaf(a.get(u), b.get(u), s);
  }
  if (c < d) {
    const Raw8<T> a = load8(x + c, d - c), b = load8(y + c, d - c);
#pragma unroll
    for (int u = 0; u < 8; ++u) s = fmaf(a.get(u), b.get(u), s);
  }
  return wave_sum(s);
}

constexpr int kMaxK = 256;                 // teacher's entries a token
constexpr int kPer = kMaxK / 64;           // of them a lane

// The teacher's shares of a row by one wave: q[u] belongs to entry lane + 64 u,
// 0 where there is none. Returns the sum of q log q; any: an entry has weight.
__device__ __forceinline__ float teacher_shares(const int32_t* ids, const float* t, int k,
                                                int64_t V, float inv_tau, int lane, int (&id)[kPer],
                                                float (&q)[kPer], bool& any) {
  float m = -INFINITY, x[kPer];
#pragma unroll
  for (int u = 0; u < kPer; ++u) {
    const int j = lane + 64 * u;
    id[u] = j < k ? ids[j] : -1;
    if (id[u] < 0 || id[u] >= V) id[u] = -1;
    x[u] = id[u] >= 0 ? t[j] * inv_tau : -INFINITY;
    m = fmaxf(m, x[u]);
  }
  m = wave_max(m);
  const float ref = m == -INFINITY ? 0.f : m;
  float s = 0.f;
#pragma unroll
  for (int u = 0; u < kPer; ++u) {
    q[u] = id[u] >= 0 ? expf(x[u] - ref) : 0.f;
    s += q[u];
  }
  s = wave_sum(s);
  any = !(s == 0.f);
  float e = 0.f;
#pragma unroll
  for (int u = 0; u < kPer; ++u) {
    if (any) q[u] /= s;
    if (q[u] != 0.f) e += q[u] * logf(q[u]);
  }
  return wave_sum(e);
}

// Joins the tiles' maxima and sums along the vocabulary and forms the losses:
// blocks of R rows by NT threads, NT / R threads a row for the join, whole waves
// a row for the dot products that its targets name. Eight rows by 1024 threads,
// or, where there are few, one by 256.
struct JoinArgs {
  const float2* part;
  int64_t parts;
  int64_t n;
  int d;
  const void* h;
  int64_t ld;
  const void* table;
  int64_t V;
  float scale, inv_tau;
  const int32_t* ids;      // [n][k] (cross entropy: k = 1)
  const float* teacher;    // nullable: cross entropy
  int k;
  int picked;              // logits holds z already
  float *loss, *lse, *logits;
};
template <typename T, int kJoinRows, int NT>
__global__ __launch_bounds__(NT) void head_join_kernel(JoinArgs g) {
  constexpr int NW = NT / 64, WR = NW / kJoinRows;   // waves, and of them a row
  __shared__ float2 red[NW][kJoinRows];
  __shared__ float lse_s[kJoinRows];
  __shared__ float zs[kJoinRows][kMaxK];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int64_t r0 = (int64_t)blockIdx.x * kJoinRows;
  // dot products
  const int r = wave / WR;
  const int64_t row = r0 + r;
  if (row < g.n && g.picked) {
    for (int j = wave % WR * 64 + lane; j < g.k; j += WR * 64) {
      const int id = g.ids[row * g.k + j];
      zs[r][j] = id >= 0 && id < g.V ? g.logits[row * g.k + j] : 0.f;
    }
  } else if (row < g.n) {
    const T* hr = static_cast<const T*>(g.h) + row * g.ld;
    const T* tab = static_cast<const T*>(g.table);
    for (int j = wave % WR; j < g.k; j += WR) {
      const int id = g.ids[row * g.k + j];
      float z = 0.f;
      if (id >= 0 && id < g.V) z = g.scale * row_dot(hr, tab + (int64_t)id * g.d, g.d, lane);
      if (lane == 0) zs[r][j] = z;
    }
  }
  {
    const int rr = tid % kJoinRows;
    const int64_t jr = r0 + rr < g.n ? r0 + rr : g.n - 1;
    float m = -INFINITY, s = 0.f;
#pragma unroll 4
    for (int64_t p = tid / kJoinRows; p < g.parts; p += NT / kJoinRows) {
      const float2 v = g.part[p * g.n + jr];
      const float hi = fmaxf(m, v.x), ref = hi == -INFINITY ? 0.f : hi;
      s = s * __builtin_amdgcn_exp2f(m - ref) + v.y * __builtin_amdgcn_exp2f(v.x - ref);
      m = hi;
    }
#pragma unroll
    for (int o = kJoinRows; o < 64; o <<= 1) {
      const float om = __shfl_xor(m, o), os = __shfl_xor(s, o);
      const float hi = fmaxf(m, om), ref = hi == -INFINITY ? 0.f : hi;
      s = s * __builtin_amdgcn_exp2f(m - ref) + os * __builtin_amdgcn_exp2f(om - ref);
      m = hi;
    }
    if (lane < kJoinRows) red[wave][lane] = make_float2(m, s);
  }
  __syncthreads();
  if (tid < kJoinRows) {
    float m = -INFINITY, s = 0.f;
#pragma unroll
    for (int w = 0; w < NW; ++w) m = fmaxf(m, red[w][tid].x);
    const float ref = m == -INFINITY ? 0.f : m;
#pragma unroll
    for (int w = 0; w < NW; ++w) s += red[w][tid].y * __builtin_amdgcn_exp2f(red[w][tid].x - ref);
    // log(s 2^m)
    const float l = (m + log2f(s)) * kLn2;
    lse_s[tid] = l;
    if (r0 + tid < g.n) g.lse[r0 + tid] = l;
  }
  __syncthreads();
  if (wave % WR || row >= g.n) return;
  const float l = lse_s[r];
  if (!g.teacher) {
    const int id = g.ids[row];
    if (lane == 0) g.loss[row] = id >= 0 && id < g.V ? l - zs[r][0] : 0.f;
    return;
  }
  int id[kPer];
  float q[kPer];
  bool any;
  const float ent = teacher_shares(g.ids + row * g.k, g.teacher + row * g.k, g.k, g.V, g.inv_tau,
                                   lane, id, q, any);
  float x = 0.f;
#pragma unroll
  for (int u = 0; u < kPer; ++u) {
    const int j = lane + 64 * u;
    if (j < g.k) {
      g.logits[row * g.k + j] = zs[r][j];
      if (q[u] != 0.f) x += q[u] * (l - zs[r][j] * g.inv_tau);
    }
  }
  x = wave_sum(x);
  if (lane == 0) g.loss[row] = any ? (ent + x) / (g.inv_tau * g.inv_tau) : 0.f;
}

// Sorts the entries of each row tile by column tile: a block a row tile, counts,
// a running sum, places. The order inside a tile is free: every entry has a
// place of its own to write to. Fetched as dot products of their own, 8,192
// tokens' 64 entries at width 2,560 took 520 of 5,200 us; sorted, and picked
// from the tiles' accumulators, 30.
constexpr int kMostTiles = 8192;
__global__ __launch_bounds__(1024) void head_bin_kernel(const int32_t* ids, int64_t n, int k, int64_t V,
                                                        int b, int tiles, int64_t cap,
                                                        uint32_t* list, int* starts) {
  __shared__ int count[kMostTiles];
  __shared__ int part[16];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int64_t r0 = (int64_t)blockIdx.x * b;
  const int total = (int)((n - r0 < b ? n - r0 : b) * k);
  const int shift = b == 256 ? 8 : 7;
  for (int i = tid; i < tiles; i += 1024) count[i] = 0;
  __syncthreads();
  const int32_t* src = ids + r0 * k;
  for (int i = tid; i < total; i += 1024) {
    const int id = src[i];
    if (id >= 0 && id < V) atomicAdd(&count[id >> shift], 1);
  }
  __syncthreads();
  int* out = starts + (int64_t)blockIdx.x * (tiles + 1);
  int base = 0;
  for (int t0 = 0; t0 < tiles; t0 += 1024) {         // exclusive running sum
    const int v = t0 + tid < tiles ? count[t0 + tid] : 0;
    int x = v;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const int y = __shfl_up(x, o);
      if (lane >= o) x += y;
    }
    if (lane == 63) part[wave] = x;
    __syncthreads();
    int before = base, all = 0;
#pragma unroll
    for (int w = 0; w < 16; ++w) {
      if (w < wave) before += part[w];
      all += part[w];
    }
    if (t0 + tid < tiles) {
      count[t0 + tid] = before + x - v;
      out[t0 + tid] = before + x - v;
    }
    base += all;
    __syncthreads();
  }
  if (tid == 0) out[tiles] = base;
  for (int i = tid; i < total; i += 1024) {
    const int id = src[i];
    if (id >= 0 && id < V) {
      const int row = i / k;
      list[blockIdx.x * cap + atomicAdd(&count[id >> shift], 1)] =
          (uint32_t)row | ((uint32_t)(id & (b - 1)) << 8) | ((uint32_t)(i - row * k) << 16);
    }
  }
}

// ---------------------------------------------------------------------------
// Operand copies

__device__ __forceinline__ int wave_imax(int v) {
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) v = max(v, __shfl_xor(v, o));
  return v;
}
// Largest of n exponents, in every thread of a block of 256.
__device__ __forceinline__ int block_exponent(const int* part, int n, int* sh) {
  int e = kNone;
  for (int i = threadIdx.x; i < n; i += 256) e = max(e, part[i]);
  e = wave_imax(e);
  if ((threadIdx.x & 63) == 0) sh[threadIdx.x >> 6] = e;
  __syncthreads();
  e = max(max(sh[0], sh[1]), max(sh[2], sh[3]));
  __syncthreads();
  return e;
}
// 2^this brings a value of exponent e to 2^kTop.
__device__ __forceinline__ int placement(int e) { return e == kNone ? 0 : kTop - e; }

template <typename T>
__device__ __forceinline__ int exponent_of8(const T* p, int left) {
  const Raw8<T> v = load8(p, left);
  float m = 0.f;
#pragma unroll
  for (int u = 0; u < 8; ++u) {
    const float a = fabsf(v.get(u));
    if (a < INFINITY) m = fmaxf(m, a);               // NaN and infinity aside
  }
  return exponent_of(m);
}

// src[c .. c + 8) times 2^e as fp16 halves (zeros behind d, or all zeros).
template <typename T>
__device__ __forceinline__ void put_halves(const T* src, int d, int c, bool keep, int e,
                                           uint16_t* dst, int64_t plane) {
  float x[8];
#pragma unroll
  for (int u = 0; u < 8; ++u) x[u] = 0.f;
  if (keep && c < d) {
    const Raw8<T> v = load8(src + c, d - c);
#pragma unroll
    for (int u = 0; u < 8; ++u) x[u] = ldexpf(v.get(u), e);
  }
  uint32_t w[4];
#pragma unroll
  for (int u = 0; u < 4; ++u) w[u] = pack2_f16(x[2 * u], x[2 * u + 1]);
  *reinterpret_cast<uint4*>(dst + c) = make_uint4(w[0], w[1], w[2], w[3]);
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int u = 0; u < 4; ++u) w[u] = pack2_f16(x[2 * u] - lo_f16(w[u]), x[2 * u + 1] - hi_f16(w[u]));
    *reinterpret_cast<uint4*>(dst + plane + c) = make_uint4(w[0], w[1], w[2], w[3]);
  }
}
__device__ __forceinline__ void put_raw(const uint16_t* src, int d, int c, bool keep, uint16_t* dst) {
  Raw8<uint16_t> v{};
  if (keep && c < d) v = load8(src + c, d - c);
  *reinterpret_cast<uint4*>(dst + c) = make_uint4(v.w[0], v.w[1], v.w[2], v.w[3]);
}

// tokens up to which the table's reading is all that counts: read in place, or
// where tiles would need a copy of it
constexpr int kFew = 64, kFewCopied = 256;
// and rows of the table up to which they are read 32 a block, one block a compute
// unit (2048 wide, 32 tokens: 15 us for 23 at 8,192 rows, 26 for 24 at 16,384)
constexpr int64_t kFewShort = 8192;
// Tokens up to which bf16 tables are used as they are for dh too: dz is then two
// bf16 halves (16 bits), two products for one, and the fp16 copies, three more
// passes over the table, fall away (65,536 rows of 2048, 8 tokens: 354 us, 430).
constexpr int kWide = 256;
constexpr int kScanBlocks = 512;
constexpr int kRowBlocks = 512;           // most blocks over rows, four waves each

// What all row kernels know of a call's rows (row pieces: of the piece).
struct RowArgs {
  const void* h;
  int64_t ld;
  int64_t n, rows_pad, vec_pad;
  int d, dp;
  const void* table;
  int64_t V;
  float scale, inv_tau;
  const int32_t* ids;
  const float *teacher, *logits;    // distillation
  int k;
  const float *lse, *dloss, *dlse;
  float *a, *lse2, *rowf;
  int* row_exp;                     // dz's rows hold 2^-row_exp times their values; kNone: zeros
  int32_t* sidx;
  float* sval;
  int *part_h, *part_w;             // exponents by block: of 2^row_exp h, of T
  int *all_h, *all_w;               // what dT and dh undo: minus their placements
  int nparts_h, nparts_w;
  int placed;                       // dz in fp16, placed by powers of two; 0: two bf16 halves
  uint16_t *hp, *hz;                // fp16 h for dT; h for the logits (NULL: read in place)
  float c2;
};

// First kernel of the backward pass. The first `row_blocks` blocks, a wave a
// row: the weight a of the row's softmax (with scale), its lse in base 2, the
// gradient at its sparse positions, and the placement of its dz. The others:
// the exponent of T's largest element.
template <typename T>
__global__ __launch_bounds__(256) void head_stats_kernel(RowArgs g, int row_blocks) {
  __shared__ int sh[4];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int top = kNone;
  if ((int)blockIdx.x >= row_blocks) {
    const int64_t count = g.V * g.d, step = (int64_t)(gridDim.x - row_blocks) * 2048;
    const T* t = static_cast<const T*>(g.table);
#pragma unroll 4
    for (int64_t i = ((int64_t)blockIdx.x - row_blocks) * 2048 + threadIdx.x * 8; i < count; i += step)
      top = max(top, exponent_of8(t + i, (int)(count - i < 8 ? count - i : 8)));
  } else {
    for (int64_t row = (int64_t)blockIdx.x * 4 + wave; row < g.vec_pad; row += row_blocks * 4) {
      const T* hr = static_cast<const T*>(g.h) + row * g.ld;
      float a = 0.f, l2 = 0.f, w = 0.f;
      int e = kNone, re = kNone;
      if (row < g.n) {
        const float l = g.lse[row], dl = g.dloss[row];
        l2 = l * kLog2e;
        float z = 0.f;
        int id[kPer];
        float q[kPer];
        bool valid;
        if (!g.teacher) {
          id[0] = g.ids[row];
          valid = id[0] >= 0 && id[0] < g.V;
          w = valid ? g.scale * dl : 0.f;
          a = w + (g.dlse ? g.scale * g.dlse[row] : 0.f);
        } else {
          teacher_shares(g.ids + row * g.k, g.teacher + row * g.k, g.k, g.V, g.inv_tau, lane, id,
                         q, valid);
          a = w = valid ? dl * g.scale / g.inv_tau : 0.f;
        }
        // a NaN weight stays one
        const bool keep = !(a == 0.f && w == 0.f);
        if (keep) {
          const float bound = fabsf(a) + fabsf(w);
          re = g.placed && exponent_of(bound) != kNone ? exponent_of(bound) - kTop : 0;
          if (g.placed) {
            for (int c = lane * 8; c < g.d; c += 512) e = max(e, exponent_of8(hr + c, g.d - c));
            e = wave_imax(e);
            if (e != kNone) top = max(top, e + re);
          }
        }
        const int place = keep ? -re : 0;
        if (!g.teacher) {
          float val = 0.f;
          if (valid && keep) {
            z = g.scale * row_dot(hr, static_cast<const T*>(g.table) + (int64_t)id[0] * g.d, g.d, lane);
            val = ldexpf(a, place) * __builtin_amdgcn_exp2f((z - l) * kLog2e);
            val = (a == 0.f ? 0.f : val) - ldexpf(w, place);
          }
          if (lane == 0) {
            g.sidx[row] = valid && keep ? id[0] : -1;
            g.sval[row] = val;
          }
        } else {
          // an id named more than once: its first entry carries the sum
          float sum[kPer];
          bool first[kPer];
#pragma unroll
          for (int u = 0; u < kPer; ++u) {
            sum[u] = 0.f;
            first[u] = id[u] >= 0;
          }
          for (int j = 0; j < g.k; ++j) {
            int oid = 0;
            float oq = 0.f;
#pragma unroll
            for (int u = 0; u < kPer; ++u)
              if ((j >> 6) == u) {
                oid = __shfl(id[u], j & 63);
                oq = __shfl(q[u], j & 63);
              }
#pragma unroll
            for (int u = 0; u < kPer; ++u)
              if (oid >= 0 && id[u] == oid) {
                sum[u] += oq;
                if (j < lane + 64 * u) first[u] = false;
              }
          }
#pragma unroll
          for (int u = 0; u < kPer; ++u) {
            const int j = lane + 64 * u;
            if (j < g.k) {
              const bool put = first[u] && keep;
              const float p = __builtin_amdgcn_exp2f(
                  (g.logits[row * g.k + j] * g.inv_tau - l) * kLog2e);
              g.sidx[row * g.k + j] = put ? id[u] : -1;
              g.sval[row * g.k + j] = put ? ldexpf(w, place) * (p - sum[u]) : 0.f;
            }
          }
        }
        a = ldexpf(a, place);
      }
      if (lane == 0) {
        g.a[row] = a;
        g.lse2[row] = l2;
        g.row_exp[row] = re;
      }
      if constexpr (sizeof(T) == 2)
        if (!g.placed && row < g.rows_pad)           // all that dT needs of h: rows without weight are zeros
          for (int c = lane * 8; c < g.dp; c += 512)
            put_raw(row < g.n ? hr : static_cast<const T*>(g.h), g.d, c, re != kNone, g.hp + row * g.dp);
    }
  }
  top = wave_imax(top);
  if (lane == 0) sh[wave] = top;
  __syncthreads();
  if (threadIdx.x == 0) {
    top = max(max(sh[0], sh[1]), max(sh[2], sh[3]));
    if ((int)blockIdx.x < row_blocks) g.part_h[blockIdx.x] = top;
    else g.part_w[blockIdx.x - row_blocks] = top;
  }
}

// Exponent of the largest element, for the forward pass of fp32 operands.
template <typename T>
__global__ __launch_bounds__(256) void head_scan_kernel(const T* t, int64_t count, int* part) {
  __shared__ int sh[4];
  int top = kNone;
#pragma unroll 4
  for (int64_t i = (int64_t)blockIdx.x * 2048 + threadIdx.x * 8; i < count; i += (int64_t)gridDim.x * 2048)
    top = max(top, exponent_of8(t + i, (int)(count - i < 8 ? count - i : 8)));
  top = wave_imax(top);
  if ((threadIdx.x & 63) == 0) sh[threadIdx.x >> 6] = top;
  __syncthreads();
  if (threadIdx.x == 0) part[blockIdx.x] = max(max(sh[0], sh[1]), max(sh[2], sh[3]));
}

// Copies of the operands. The first `row_blocks` blocks, a wave a row of h: for
// the logits (hz: fp16 halves placed by the row's own largest element, or bf16
// as it is) and for dT (hp). The others: rows of a piece of T, as fp16 (wp) and,
// where the logits cannot read it in place, as bf16 (wz). Zeros behind d and
// behind the rows.
struct PieceArgs {
  const void* src;
  int64_t rows, rows_pad;
  uint16_t *wp, *wz;
};

template <typename T>
__global__ __launch_bounds__(256) void head_copy_kernel(RowArgs g, PieceArgs w, int row_blocks) {
  __shared__ int sh[4];
  constexpr bool F32 = sizeof(T) == 4;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const bool scaled = g.nparts_w > 0;
  const int pw = scaled ? placement(block_exponent(g.part_w, g.nparts_w, sh)) : 0;
  if ((int)blockIdx.x >= row_blocks) {
    const int per = g.dp / 8;
    const int64_t total = w.rows_pad * per, step = (int64_t)(gridDim.x - row_blocks) * 256;
    for (int64_t i = ((int64_t)blockIdx.x - row_blocks) * 256 + threadIdx.x; i < total; i += step) {
      const int64_t r = i / per;
      const int c = (int)(i - r * per) * 8;
      const bool in = r < w.rows;
      const T* src = static_cast<const T*>(w.src) + (in ? r : 0) * g.d;
      if (w.wp) put_halves(src, g.d, c, in, pw, w.wp + r * g.dp, w.rows_pad * g.dp);
      if constexpr (!F32)
        if (w.wz) put_raw(src, g.d, c, in, w.wz + r * g.dp);
    }
    return;
  }
  int ph = 0;
  if (g.hp) ph = placement(block_exponent(g.part_h, g.nparts_h, sh));
  if (blockIdx.x == 0 && threadIdx.x == 0 && g.hp) {
    *g.all_h = -ph;
    *g.all_w = -pw;
  }
  for (int64_t row = (int64_t)blockIdx.x * 4 + wave; row < g.vec_pad; row += row_blocks * 4) {
    const bool in = row < g.n;
    const T* src = static_cast<const T*>(g.h) + (in ? row : 0) * g.ld;
    if constexpr (F32) {
      // the logits' copy, and the factor that undoes its placement
      int e = kNone;
      if (in) {
        for (int c = lane * 8; c < g.d; c += 512) e = max(e, exponent_of8(src + c, g.d - c));
        e = wave_imax(e);
      }
      const int p = placement(e);
      if (lane == 0) g.rowf[row] = ldexpf(g.c2, min(-p - pw, 100));
      if (row < g.rows_pad)
        for (int c = lane * 8; c < g.dp; c += 512)
          put_halves(src, g.d, c, in, p, g.hz + row * g.dp, g.rows_pad * g.dp);
    } else {
      if (g.hz && row < g.rows_pad)
        for (int c = lane * 8; c < g.dp; c += 512) put_raw(src, g.d, c, in, g.hz + row * g.dp);
    }
    if (g.hp && row < g.rows_pad) {
      const int re = in ? g.row_exp[row] : kNone;
      const bool keep = re != kNone;                 // rows without weight add zeros
      for (int c = lane * 8; c < g.dp; c += 512)
        put_halves(src, g.d, c, keep, keep ? ph + re : 0, g.hp + row * g.dp, g.rows_pad * g.dp);
    }
  }
}

// Writes the sparse positions of a piece over its dz.
__global__ __launch_bounds__(256) void head_sparse_kernel(const int32_t* sidx, const float* sval,
                                                          int64_t n, int k, int64_t v0, int64_t cols,
                                                          uint16_t* dz, int64_t ldz,
                                                          int64_t plane, int planes, int f16) {
  const int64_t total = n * k;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
    const int64_t v = (int64_t)sidx[i] - v0;
    if (v < 0 || v >= cols) continue;
    const float x = sval[i];
    uint16_t* p = dz + i / k * ldz + v;
    const uint32_t w = f16 ? pack2_f16(x, 0.f) : pack2_bf16(x, 0.f);
    *p = (uint16_t)w;
    const float left = x - (f16 ? lo_f16(w) : __uint_as_float(w << 16));
    if (planes > 1) p[plane] = (uint16_t)(f16 ? pack2_f16(left, 0.f) : pack2_bf16(left, 0.f));
  }
}

// Sums the results of K's splits in order, adds prev, and stores: two products.
struct SumArgs {
  const float* part;
  int splits;
  int64_t stride, ld_part;             // elements
  int64_t M, N;
  const float* prev;
  int64_t ld_prev;
  void* out;
  int64_t ld_out;
  int out_bf16;
};
__global__ __launch_bounds__(256) void head_sum_kernel(SumArgs a, SumArgs b, int na) {
  // 32 groups of four columns a block; eight threads a group take every eighth
  // split (one thread took 66 us for 180 splits of 32 x 59)
  __shared__ float4 sh[8][32];
  const bool first = (int)blockIdx.x < na;
  const SumArgs& g = first ? a : b;
  const int x = threadIdx.x & 31, y = threadIdx.x >> 5;
  const int64_t per = (g.N + 3) / 4, total = g.M * per;
  const int64_t step = (int64_t)(first ? na : (int)gridDim.x - na) * 32;
  for (int64_t i0 = ((int64_t)blockIdx.x - (first ? 0 : na)) * 32; i0 < total; i0 += step) {
    const int64_t i = i0 + x;
    const int64_t row = i / per, col = (i - row * per) * 4;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    if (i < total) {
      const float* p = g.part + row * g.ld_part + col;   // rows of whole tiles
#pragma unroll 4
      for (int s = y; s < g.splits; s += 8) {
        const float4 t = *reinterpret_cast<const float4*>(p + s * g.stride);
        v.x += t.x;
        v.y += t.y;
        v.z += t.z;
        v.w += t.w;
      }
    }
    sh[y][x] = v;
    __syncthreads();
    if (y == 0 && i < total) {
#pragma unroll
      for (int s = 1; s < 8; ++s) {
        const float4 t = sh[s][x];
        v.x += t.x;
        v.y += t.y;
        v.z += t.z;
        v.w += t.w;
      }
      const float f[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int u = 0; u < 4; ++u)
        if (col + u < g.N) {
          const float r = g.prev ? f[u] + g.prev[row * g.ld_prev + col + u] : f[u];
          if (g.out_bf16)
            static_cast<uint16_t*>(g.out)[row * g.ld_out + col + u] = (uint16_t)pack2_bf16(r, 0.f);
          else
            static_cast<float*>(g.out)[row * g.ld_out + col + u] = r;
        }
    }
    __syncthreads();
  }
}

__global__ __launch_bounds__(256) void head_zero_kernel(uint16_t* out, int64_t count) {
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < count; i += (int64_t)gridDim.x * 256)
    out[i] = 0;
}

int64_t pad(int64_t x, int64_t a) { return (x + a - 1) / a * a; }
int64_t tiles_of(int64_t x, int64_t b) { return (x + b - 1) / b; }
int blocks_for(int64_t items, int most) {
  const int64_t b = (items + 255) / 256;
  return (int)(b < 1 ? 1 : b > most ? most : b);
}
int elt_size(int32_t dtype) { return dtype == PG_F32 ? 4 : 2; }

// An operand that the logits' tiles can read where it lies: bf16 rows of whole
// slots at 16-byte alignment.
bool in_place(int32_t dtype, int d, int64_t ld, const void* p) {
  return dtype == PG_BF16 && d % 32 == 0 && d >= 128 && ld % 8 == 0 && ld < (1 << 24) &&
         (uintptr_t)p % 16 == 0;
}

bool big_tiles(int64_t M, int64_t N) {
  return tiles_of(M, 256) * tiles_of(N, 256) >= kCUs / 2 && M > 128;
}

template <int EPI>
hipError_t launch_tiles(TileArgs& g, int64_t M, int64_t N, bool big, bool f16, hipStream_t s) {
  const int b = big ? 256 : 128;
  g.splits = 1;
  g.nbm = (int)tiles_of(M, b);
  g.nbn = (int)tiles_of(N, b);
  const int64_t total = (int64_t)g.nbm * g.nbn;
  const int64_t most = big ? kCUs : 2 * kCUs;
  const unsigned grid = (unsigned)(total < most ? total : most);
  constexpr bool H = EPI != EPI_DZB;                 // its dz is bf16, as its operands
  auto* kernel = big ? (H && f16 ? head_tile_kernel<EPI, H, 256, 256, 2, 4>
                                 : head_tile_kernel<EPI, false, 256, 256, 2, 4>)
                     : (H && f16 ? head_tile_kernel<EPI, H, 128, 128, 2, 2>
                                 : head_tile_kernel<EPI, false, 128, 128, 2, 2>);
  hipLaunchKernelGGL(kernel, dim3(grid), dim3(big ? 512 : 256), 0, s, g);
  return hipGetLastError();
}

void launch_copy(bool f32, const RowArgs& r, const PieceArgs& w, bool rows, hipStream_t s) {
  const int rb = rows ? (int)(tiles_of(r.vec_pad, 4) < kRowBlocks ? tiles_of(r.vec_pad, 4) : kRowBlocks) : 0;
  const int wb = w.rows ? blocks_for(w.rows_pad * r.dp / 8, 2048) : 0;
  if (rb + wb == 0) return;
  if (f32)
    hipLaunchKernelGGL((head_copy_kernel<float>), dim3(rb + wb), dim3(256), 0, s, r, w, rb);
  else
    hipLaunchKernelGGL((head_copy_kernel<uint16_t>), dim3(rb + wb), dim3(256), 0, s, r, w, rb);
}

}  // namespace

// ---------------------------------------------------------------------------
// Workspace geometry

HeadPlan head_plan(int64_t n, int d, int64_t V, int32_t dtype, int k, bool backward) {
  HeadPlan p{};
  p.planes = dtype == PG_F32 ? 2 : 1;
  p.dp = (int)pad(d < 128 ? 128 : d, 32);
  int64_t at = 0;
  auto take = [&](int64_t bytes) {
    const int64_t o = at;
    at += pad(bytes, 256);
    return o;
  };
  const int64_t row = (int64_t)p.dp * 2 * p.planes;
  p.off_parts = take((kScanBlocks + kRowBlocks + 2) * 4);
  if (!backward) {
    p.rows = n;
    // rows of the table are copied a piece at a time, about 256 MB of them
    p.cols = pad(V, 256);
    const int64_t most = ((int64_t)1 << 28) / row / 256 * 256;
    if (p.cols > most) p.cols = most > 256 ? most : 256;
    p.off_rowf = take(pad(n, 256) * 4);
    p.off_hz = take(n * row);
    p.off_wz = take(p.cols * row);
    const int64_t few = tiles_of(V < kFewShort ? V : kFewShort, 32) * (n < kFew ? n : kFew);
    const int64_t parts = tiles_of(V, 128) * n;
    p.off_part = take((parts > few ? parts : few) * 8);
    // entries by tile: whole row tiles, and room for a load behind the last
    p.off_list = take((pad(n, 256) * k + kPicks) * 4);
    p.off_starts = take(tiles_of(n, 128) * (tiles_of(V, 128) + 1) * 4);
  } else {
    // dz of a piece: at most 2^29 elements (1 GiB) of both halves
    const int halves = n <= kWide ? 2 : p.planes;
    p.rows = pad(n < 1 ? 1 : n, 128);
    if (p.rows > 32768) p.rows = 32768;
    const int64_t elems = ((int64_t)1 << 29) / halves;
    int64_t c = elems / p.rows / 256 * 256;
    if (c > pad(V, 256)) c = pad(V, 256);
    const int64_t pieces = (V + c - 1) / c;
    p.cols = pad((V + pieces - 1) / pieces, 256);
    const int64_t vec = pad(p.rows, 256);
    p.off_a = take(vec * 4);
    p.off_lse = take(vec * 4);
    p.off_rowf = take(vec * 4);
    p.off_exp = take(vec * 4);
    p.off_sidx = take(p.rows * k * 4);
    p.off_sval = take(p.rows * k * 4);
    p.off_h = take(p.rows * row);
    p.off_hz = take(p.rows * row);
    p.off_w = take(p.cols * row);
    // bf16 rows that cannot be read in place: all, or the last ones
    p.off_wz = p.planes == 2 ? at : take((d % 32 == 0 && d >= 128 ? 128 : p.cols) * row);
    p.off_dz = take(p.rows * p.cols * 2 * halves);
    p.off_dh = take(p.rows * d * 4);
    p.off_dw = n > 32768 ? take(V * d * 4) : at;
    p.off_split = take((int64_t)kCUs * 256 * 256 * 4);   // most tiles at once
  }
  p.bytes = at;
  return p;
}

hipError_t launch_head_forward(const HeadPlan& p, const HeadArgs& g, void* workspace,
                               hipStream_t s) {
  auto* ws = static_cast<uint8_t*>(workspace);
  const int es = elt_size(g.dtype);
  const bool f32 = g.dtype == PG_F32;
  const int64_t dp2 = (int64_t)p.dp * 2;
  auto* parts_w = reinterpret_cast<int*>(ws + p.off_parts);
  TileArgs t{};
  t.nseg = f32 ? kSegs : 1;
  t.c2 = (float)((double)g.scale * (double)g.inv_tau * 1.4426950408889634);
  t.M = g.n;
  t.rowf = reinterpret_cast<const float*>(ws + p.off_rowf);
  t.slots = p.dp / 32;
  int64_t parts = 0;
  bool picked = false;
  const bool h_here = in_place(g.dtype, g.d, g.ld_h, g.h);
  const bool w_here = in_place(g.dtype, g.d, g.d, g.table);
  if (g.n <= (w_here ? kFew : kFewCopied)) {
    const int groups = (int)tiles_of(g.n, 64);
    const FewArgs f{g.h, g.table, g.ld_h, g.n, g.V, g.d, groups, t.c2,
                    reinterpret_cast<float2*>(ws + p.off_part)};
    if (groups == 1 && g.V <= kFewShort) {
      parts = tiles_of(g.V, 32);
      auto* kernel = f32 ? (g.n <= 16   ? head_few_split_kernel<float, 1, 0>
                            : g.n <= 32 ? head_few_split_kernel<float, 2, 0>
                                        : head_few_split_kernel<float, 4, 0>)
                         : (g.n <= 16   ? head_few_split_kernel<uint16_t, 1, 0>
                            : g.n <= 32 ? head_few_split_kernel<uint16_t, 2, 0>
                                        : head_few_split_kernel<uint16_t, 4, 0>);
      hipLaunchKernelGGL(kernel, dim3((unsigned)parts), dim3(256), 0, s, f, FewDz{});
    } else {
    parts = tiles_of(g.V, 128);
    const int64_t blocks = groups == 1 ? parts : pad(parts, 8) * groups;
    auto* kernel = f32 ? (g.n <= 16 ? head_few_kernel<float, 1, 0> : g.n <= 32 ? head_few_kernel<float, 2, 0>
                                                                            : head_few_kernel<float, 4, 0>)
                       : (g.n <= 16   ? head_few_kernel<uint16_t, 1, 0>
                          : g.n <= 32 ? head_few_kernel<uint16_t, 2, 0>
                                      : head_few_kernel<uint16_t, 4, 0>);
    hipLaunchKernelGGL(kernel, dim3((unsigned)blocks), dim3(256), 0, s, f, FewDz{});
    }
  } else {
    RowArgs r{};
    r.h = g.h;
    r.ld = g.ld_h;
    r.n = r.rows_pad = g.n;
    r.vec_pad = pad(g.n, 256);
    r.d = g.d;
    r.dp = p.dp;
    r.rowf = reinterpret_cast<float*>(ws + p.off_rowf);
    r.part_w = parts_w;
    r.c2 = t.c2;
    if (f32) {
      r.nparts_w = blocks_for((g.V * g.d + 7) / 8, kScanBlocks);
      hipLaunchKernelGGL((head_scan_kernel<float>), dim3(r.nparts_w), dim3(256), 0, s,
                         static_cast<const float*>(g.table), g.V * g.d, parts_w);
    }
    if (h_here) {
      t.A = Side{static_cast<const uint8_t*>(g.h), g.ld_h * 2, 0, g.n};
    } else {
      r.hz = reinterpret_cast<uint16_t*>(ws + p.off_hz);
      t.A = Side{ws + p.off_hz, dp2, g.n * dp2, g.n};
    }
    const int64_t piece = w_here ? g.V : p.cols;       // all but the last of whole tiles
    const bool big = big_tiles(g.n, g.V < piece ? g.V : piece);
    const int b = big ? 256 : 128;
    picked = g.teacher && tiles_of(g.V, b) <= kMostTiles;
    if (picked) {
      auto* list = reinterpret_cast<uint32_t*>(ws + p.off_list);
      auto* starts = reinterpret_cast<int*>(ws + p.off_starts);
      t.list = list;
      t.starts = starts;
      t.cap = (int64_t)b * g.k;
      t.tiles = (int)tiles_of(g.V, b);
      t.logits = g.logits;
      t.k = g.k;
      t.zf = (float)(0.6931471805599453 / (double)g.inv_tau);
      hipLaunchKernelGGL(head_bin_kernel, dim3((unsigned)tiles_of(g.n, b)), dim3(1024), 0, s, g.ids,
                         g.n, g.k, g.V, b, t.tiles, t.cap, list, starts);
    }
    for (int64_t v0 = 0; v0 < g.V; v0 += piece) {
      const int64_t c = g.V - v0 < piece ? g.V - v0 : piece;
      PieceArgs w{};
      w.src = static_cast<const uint8_t*>(g.table) + v0 * g.d * es;
      if (w_here) {
        t.B = Side{static_cast<const uint8_t*>(w.src), (int64_t)g.d * 2, 0, c};
      } else {
        w.rows = w.rows_pad = c;
        (f32 ? w.wp : w.wz) = reinterpret_cast<uint16_t*>(ws + p.off_wz);
        t.B = Side{ws + p.off_wz, dp2, c * dp2, c};
      }
      launch_copy(f32, r, w, v0 == 0 && !h_here, s);
      t.V = c;
      t.part = reinterpret_cast<float2*>(ws + p.off_part) + parts * g.n;
      t.tile0 = (int)parts;
      const hipError_t e = picked ? launch_tiles<EPI_PICK>(t, g.n, c, big, f32, s)
                                  : launch_tiles<EPI_LSE>(t, g.n, c, big, f32, s);
      if (e != hipSuccess) return e;
      parts += t.nbn;
    }
  }
  JoinArgs j{};
  j.part = reinterpret_cast<const float2*>(ws + p.off_part);
  j.parts = parts;
  j.n = g.n;
  j.d = g.d;
  j.h = g.h;
  j.ld = g.ld_h;
  j.table = g.table;
  j.V = g.V;
  j.scale = g.scale;
  j.inv_tau = g.inv_tau;
  j.ids = g.ids;
  j.teacher = g.teacher;
  j.k = g.k;
  j.picked = picked;
  j.loss = g.loss;
  j.lse = g.lse;
  j.logits = g.logits;
  const bool alone = g.n <= 2 * kCUs;
  const unsigned grid = (unsigned)(alone ? g.n : tiles_of(g.n, 8)), nt = alone ? 256 : 1024;
  auto* join = f32 ? (alone ? head_join_kernel<float, 1, 256> : head_join_kernel<float, 8, 1024>)
                   : (alone ? head_join_kernel<uint16_t, 1, 256> : head_join_kernel<uint16_t, 8, 1024>);
  hipLaunchKernelGGL(join, dim3(grid), dim3(nt), 0, s, j);
  return hipGetLastError();
}

// Time until na tiles of length la, then nb of length lb <= la, have run on m
// units, each taking the next tile as it gets free.
static double makespan(int64_t na, double la, int64_t nb, double lb, int m) {
  const int64_t full = na / m, rest = na % m;
  const double t0 = full * la, t1 = t0 + (rest ? la : 0);
  if (nb == 0) return t1;
  // m - rest units are free from t0 on, the others from t1
  const int64_t early = lb > 0 && rest ? (int64_t)((t1 - t0) / lb) : 0;
  const int64_t before = (m - rest) * early;
  if (rest && nb <= before) return t1;
  const int64_t left = nb - before;
  const double te = t0 + early * lb;                 // the early units' next start
  if (!rest) return t0 + (double)((left + m - 1) / m) * lb;
  const int64_t rounds = left / m, more = left % m;
  if (more == 0) return t1 + rounds * lb;
  return more <= m - rest ? (te + (rounds + 1) * lb > t1 + rounds * lb ? te + (rounds + 1) * lb
                                                                     : t1 + rounds * lb)
                          : t1 + (rounds + 1) * lb;
}

// The products of a piece: both in one launch; where their tiles are few, K is
// split and a second launch joins the splits.
static hipError_t launch_grads(TileArgs tw, TileArgs th, bool f16, float* split, hipStream_t s) {
  const bool w = tw.out != nullptr, h = th.out != nullptr;
  tw.splits = th.splits = 1;
  // Tile size and K's splits: tiles run longest first, a large one to a compute
  // unit or two small ones; splitting evens out their end, but writes and reads a
  // result more. Times in us: 0.95 a slot of a large tile, 0.6 of a small one
  // (4 more for its start and end; twice as many run at once), 5 MB/us for partial results.
  double best = 1e30;
  bool big = false;
  int kw = 1, kh = 1;
  for (int large = 0; large < 2; ++large) {
    const int b = large ? 256 : 128, at_once = large ? kCUs : 2 * kCUs;
    const double slot = (large ? 0.95 : 0.6) * tw.nseg;
    const int64_t nw = w ? tiles_of(tw.M, b) * tiles_of(tw.V, b) : 0;
    const int64_t nh = h ? tiles_of(th.M, b) * tiles_of(th.V, b) : 0;
    auto splits_up_to = [&](const TileArgs& t, int64_t n) {
      int64_t most = (int64_t)t.slots * t.nseg / 8;    // 8 slots a tile at least
      if (most > t.slots / 2) most = t.slots / 2;
      if (n == 0 || most > at_once / n) most = n == 0 ? 1 : at_once / n;
      return most < 1 ? 1 : (int)most;
    };
    const int mw = splits_up_to(tw, nw), mh = splits_up_to(th, nh);
    // at most at_once split tiles in all: what the workspace holds
    for (int i = 1; i <= mw; i = i < 16 ? i + 1 : i * 5 / 4)
      for (int j = 1; j <= mh; j = j < 16 ? j + 1 : j * 5 / 4) {
        const int64_t split_tiles = (i > 1 ? nw * i : 0) + (j > 1 ? nh * j : 0);
        if (split_tiles > at_once) continue;
        const double lw = nw ? (double)tw.slots / i + 4 : 0, lh = nh ? (double)th.slots / j + 4 : 0;
        double t = slot * (lw > lh ? makespan(nw * i, lw, nh * j, lh, at_once)
                                   : makespan(nh * j, lh, nw * i, lw, at_once));
        if (split_tiles) t += 6 + (double)split_tiles * b * b * 8 / 5e6;
        if (t < best) {
          best = t;
          big = large;
          kw = i;
          kh = j;
        }
      }
  }
  const int b = big ? 256 : 128;
  auto tiles = [&](TileArgs& t) {
    t.nbm = (int)tiles_of(t.M, b);
    t.nbn = (int)tiles_of(t.V, b);
    return (int64_t)t.nbm * t.nbn;
  };
  const int64_t nw = w ? tiles(tw) : 0, nh = h ? tiles(th) : 0;
  SumArgs sums[2] = {};
  int64_t used = 0;
  auto share = [&](TileArgs& t, int k, SumArgs& sa) {
    if (k < 2) return;
    sa = SumArgs{split + used, k, 0, (int64_t)t.nbn * b, t.M, t.V, t.prev, t.ld_prev,
                 t.out, t.ld_out, t.out_bf16};
    sa.stride = (int64_t)t.nbm * b * sa.ld_part;
    t.splits = k;
    t.out = split + used;
    t.ld_out = sa.ld_part;
    t.split_out = sa.stride;
    t.out_bf16 = 0;
    t.prev = nullptr;
    used += k * sa.stride;
  };
  share(tw, kw, sums[0]);
  share(th, kh, sums[1]);
  // short tiles: about 64 slots a block, while that leaves blocks enough
  const int at_once = big ? kCUs : 2 * kCUs;
  auto per_block = [&](const TileArgs& t, int64_t n) {
    int64_t per = 64 / ((int64_t)t.slots * t.nseg / t.splits);
    if (per > n / (4 * at_once)) per = n / (4 * at_once);
    return (uint32_t)(per < 1 ? 1 : per);
  };
  const uint32_t per_w = per_block(tw, nw * tw.splits), per_h = per_block(th, nh * th.splits);
  const uint32_t gw = (uint32_t)tiles_of(nw * tw.splits, per_w);
  const uint32_t gh = (uint32_t)tiles_of(nh * th.splits, per_h);
  const bool many = per_w > 1 || per_h > 1;
  auto pick = [&](auto* f, auto* b, auto* fm, auto* bm) { return many ? (f16 ? fm : bm) : f16 ? f : b; };
  auto* kernel = big ? pick(head_grad_kernel<true, false, 256, 256, 2, 4>,
                            head_grad_kernel<false, false, 256, 256, 2, 4>,
                            head_grad_kernel<true, true, 256, 256, 2, 4>,
                            head_grad_kernel<false, true, 256, 256, 2, 4>)
                     : pick(head_grad_kernel<true, false, 128, 128, 2, 2>,
                            head_grad_kernel<false, false, 128, 128, 2, 2>,
                            head_grad_kernel<true, true, 128, 128, 2, 2>,
                            head_grad_kernel<false, true, 128, 128, 2, 2>);
  hipLaunchKernelGGL(kernel, dim3(gw + gh), dim3(big ? 512 : 256), 0, s, tw, th, gw, gh,
                     per_w, per_h);
  const int sw = sums[0].splits ? blocks_for(sums[0].M * ((sums[0].N + 3) / 4) * 8, 2048) : 0;
  const int sh = sums[1].splits ? blocks_for(sums[1].M * ((sums[1].N + 3) / 4) * 8, 2048) : 0;
  if (sw + sh)
    hipLaunchKernelGGL(head_sum_kernel, dim3(sw + sh), dim3(256), 0, s, sums[0], sums[1], sw);
  return hipGetLastError();
}

hipError_t launch_head_backward(const HeadPlan& p, const HeadArgs& g, void* workspace,
                                hipStream_t s) {
  auto* ws = static_cast<uint8_t*>(workspace);
  const int es = elt_size(g.dtype);
  const int64_t dp2 = (int64_t)p.dp * 2;
  const bool f32 = g.dtype == PG_F32;
  const bool wide = !f32 && g.n <= kWide;
  const int nseg = f32 ? kSegs : 1, nseg_grad = wide ? 2 : nseg;
  auto* dz = reinterpret_cast<uint16_t*>(ws + p.off_dz);
  if (g.n == 0) {
    const int64_t count = g.V * g.d * elt_size(g.dw_dtype) / 2;
    if (!g.dw || g.accumulate) return hipSuccess;
    hipLaunchKernelGGL(head_zero_kernel, dim3(blocks_for(count, 8192)), dim3(256), 0, s,
                       static_cast<uint16_t*>(g.dw), count);
    return hipGetLastError();
  }
  const bool w_here = in_place(g.dtype, g.d, g.d, g.table);
  for (int64_t r0 = 0; r0 < g.n; r0 += p.rows) {
    const int64_t n = g.n - r0 < p.rows ? g.n - r0 : p.rows;
    const int64_t rows = pad(n, nseg_grad > 1 ? 64 : 128);   // four slots of K at least
    const bool first_rows = r0 == 0, last_rows = r0 + n == g.n;
    RowArgs r{};
    r.h = static_cast<const uint8_t*>(g.h) + r0 * g.ld_h * es;
    r.ld = g.ld_h;
    r.n = n;
    r.rows_pad = rows;
    r.vec_pad = pad(n, 256);
    r.d = g.d;
    r.dp = p.dp;
    r.table = g.table;
    r.V = g.V;
    r.scale = g.scale;
    r.inv_tau = g.inv_tau;
    r.ids = g.ids + r0 * g.k;
    r.teacher = g.teacher ? g.teacher + r0 * g.k : nullptr;
    r.logits = g.logits ? g.logits + r0 * g.k : nullptr;
    r.k = g.k;
    r.lse = g.lse + r0;
    r.dloss = g.dloss + r0;
    r.dlse = g.dlse ? g.dlse + r0 : nullptr;
    r.a = reinterpret_cast<float*>(ws + p.off_a);
    r.lse2 = reinterpret_cast<float*>(ws + p.off_lse);
    r.rowf = reinterpret_cast<float*>(ws + p.off_rowf);
    r.row_exp = reinterpret_cast<int*>(ws + p.off_exp);
    r.sidx = reinterpret_cast<int32_t*>(ws + p.off_sidx);
    r.sval = reinterpret_cast<float*>(ws + p.off_sval);
    r.part_w = reinterpret_cast<int*>(ws + p.off_parts);
    r.part_h = r.part_w + kScanBlocks;
    r.all_h = r.part_h + kRowBlocks;
    r.all_w = r.all_h + 1;
    r.placed = !wide;
    r.nparts_w = wide ? 0 : blocks_for((g.V * g.d + 7) / 8, kScanBlocks);
    r.nparts_h = (int)(tiles_of(r.vec_pad, 4) < kRowBlocks ? tiles_of(r.vec_pad, 4) : kRowBlocks);
    r.hp = reinterpret_cast<uint16_t*>(ws + p.off_h);
    const bool h_here = in_place(g.dtype, g.d, g.ld_h, r.h);
    r.hz = h_here ? nullptr : reinterpret_cast<uint16_t*>(ws + p.off_hz);
    r.c2 = (float)((double)g.scale * (double)g.inv_tau * 1.4426950408889634);
    // T's exponent is the same for every piece of the rows
    const unsigned grid = r.nparts_h + (first_rows ? r.nparts_w : 0);
    if (f32)
      hipLaunchKernelGGL((head_stats_kernel<float>), dim3(grid), dim3(256), 0, s, r, r.nparts_h);
    else
      hipLaunchKernelGGL((head_stats_kernel<uint16_t>), dim3(grid), dim3(256), 0, s, r, r.nparts_h);

    for (int64_t v0 = 0; v0 < g.V; v0 += p.cols) {
      const int64_t c = g.V - v0 < p.cols ? g.V - v0 : p.cols;
      const int64_t cols = pad(c, 128);
      const bool first = v0 == 0, last = v0 + c == g.V;
      PieceArgs w{};
      w.src = static_cast<const uint8_t*>(g.table) + v0 * g.d * es;
      auto* wz = reinterpret_cast<uint16_t*>(ws + p.off_wz);
      w.rows = c;
      w.rows_pad = cols;
      if (!wide) w.wp = reinterpret_cast<uint16_t*>(ws + p.off_w);
      if (!f32 && !w_here) w.wz = wz;
      PieceArgs copies = w;
      const int64_t odd = c % 128;
      if (wide && w_here) {                          // only the last rows, to whole slots
        copies.src = static_cast<const uint8_t*>(w.src) + (c - odd) * g.d * es;
        copies.rows = odd;
        copies.rows_pad = odd ? 128 : 0;
        copies.wz = wz;
      }
      launch_copy(f32, r, copies, first && !wide, s);
      const int64_t ldz = cols, plane = rows * cols;

      TileArgs t{};
      t.A = h_here ? Side{static_cast<const uint8_t*>(r.h), g.ld_h * 2, 0, n}
                   : Side{ws + (wide ? p.off_h : p.off_hz), dp2, rows * dp2, n};
      t.B = f32 ? Side{ws + p.off_w, dp2, cols * dp2, c}
                : w_here ? Side{static_cast<const uint8_t*>(w.src), (int64_t)g.d * 2, 0, c}
                         : Side{ws + p.off_wz, dp2, 0, c};
      t.nseg = nseg;
      t.slots = p.dp / 32;
      t.c2 = r.c2;
      t.M = n;
      t.V = c;
      t.rowf = r.rowf;
      t.a = r.a;
      t.lse2 = r.lse2;
      t.dz = dz;
      t.ldz = ldz;
      t.dz_plane = plane;
      t.Mpad = rows;
      t.Vpad = cols;
      hipError_t e = hipSuccess;
      if (n <= kFew) {
        const FewArgs f{r.h, w.src, g.ld_h, n, c, g.d, 1, r.c2, nullptr};
        const FewDz z{r.a, r.lse2, dz, ldz, plane, (int)rows};
        const bool one = c <= kFewShort;             // 32 rows of T a block
        auto pick = [&](auto* split, auto* whole) { return one ? split : whole; };
        auto* kernel =
            f32 ? (n <= 16   ? pick(head_few_split_kernel<float, 1, 1>, head_few_kernel<float, 1, 1>)
                   : n <= 32 ? pick(head_few_split_kernel<float, 2, 1>, head_few_kernel<float, 2, 1>)
                             : pick(head_few_split_kernel<float, 4, 1>, head_few_kernel<float, 4, 1>))
                : (n <= 16   ? pick(head_few_split_kernel<uint16_t, 1, 2>, head_few_kernel<uint16_t, 1, 2>)
                   : n <= 32 ? pick(head_few_split_kernel<uint16_t, 2, 2>, head_few_kernel<uint16_t, 2, 2>)
                             : pick(head_few_split_kernel<uint16_t, 4, 2>, head_few_kernel<uint16_t, 4, 2>));
        hipLaunchKernelGGL(kernel, dim3((unsigned)(cols / (one ? 32 : 128))), dim3(256), 0, s, f, z);
      } else {
        const bool big = big_tiles(rows, cols);
        e = wide ? launch_tiles<EPI_DZB>(t, rows, cols, big, false, s)
                 : launch_tiles<EPI_DZ>(t, rows, cols, big, f32, s);
      }
      if (e != hipSuccess) return e;
      hipLaunchKernelGGL(head_sparse_kernel, dim3(blocks_for(n * g.k, 8192)), dim3(256), 0, s,
                         r.sidx, r.sval, n, g.k, v0, c, dz, ldz, plane, wide ? 2 : p.planes, !wide);

      // dT of the piece: [c x d], K over the rows
      TileArgs tw{}, th{};
      tw.A = Side{ws + p.off_dz, ldz * 2, plane * 2, cols};
      tw.B = Side{ws + p.off_h, dp2, rows * dp2, p.dp};
      tw.nseg = nseg_grad;
      tw.slots = (int)(rows / 32);
      tw.M = c;
      tw.V = g.d;
      if (!wide) tw.all_exp = r.all_h;
      if (g.dw) {
        auto* acc = reinterpret_cast<float*>(ws + p.off_dw) + v0 * g.d;
        auto* dw32 = static_cast<float*>(g.dw) + v0 * g.d;
        const bool to16 = g.dw_dtype == PG_BF16;
        tw.ld_out = tw.ld_prev = g.d;
        if (to16) {
          tw.out = last_rows ? static_cast<void*>(static_cast<uint16_t*>(g.dw) + v0 * g.d) : acc;
          tw.out_bf16 = last_rows;
          tw.prev = first_rows ? nullptr : acc;
        } else {
          tw.out = dw32;
          tw.prev = first_rows && !g.accumulate ? nullptr : dw32;
        }
      }
      // dh: [n x d], K over the piece's columns
      th.A = Side{ws + p.off_dz, ldz * 2, plane * 2, rows};
      th.B = Side{ws + (wide ? p.off_wz : p.off_w), dp2, cols * dp2, p.dp};
      if (wide && w_here) {
        th.B.p = static_cast<const uint8_t*>(w.src);
        if (odd) {
          th.B.tail_slot = (int)((c - odd) / 32);
          th.B.tail = (int64_t)((uintptr_t)wz - ((uintptr_t)w.src + (c - odd) * dp2));
        }
      }
      th.nseg = nseg_grad;
      th.slots = (int)(cols / 32);
      th.M = n;
      th.V = g.d;
      if (!wide) {
        th.row_exp = r.row_exp;
        th.all_exp = r.all_w;
      }
      if (g.dh) {
        auto* acc = reinterpret_cast<float*>(ws + p.off_dh);
        auto* out = static_cast<uint8_t*>(g.dh) + r0 * g.ld_dh * es;
        if (f32) {
          th.out = out;
          th.ld_out = th.ld_prev = g.ld_dh;
          th.prev = first ? nullptr : reinterpret_cast<const float*>(out);
        } else {
          th.out = last ? static_cast<void*>(out) : acc;
          th.ld_out = last ? g.ld_dh : g.d;
          th.out_bf16 = last;
          th.prev = first ? nullptr : acc;
          th.ld_prev = g.d;
        }
      }
      e = launch_grads(tw, th, !wide, reinterpret_cast<float*>(ws + p.off_split), s);
      if (e != hipSuccess) return e;
    }
  }
  return hipGetLastError();
}

}  // namespace pg
