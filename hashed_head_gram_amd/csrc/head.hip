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
// 2^-31 of the largest. Columns of dz that lie below fp16's normal numbers in every
// row (tokens that no position finds likely, whose rows of dT are as small) are
// lifted by powers of two of their own, which dT undoes and T's copy takes back:
// 1 % of a call where there are none (16,384 x 768 of 50,304: 3,740 us, 3,700
// without; 16,384 x 2,560 of 128,000: 28.86 ms, 28.76), up to a quarter where most
// columns change from one group of rows to the next. fp32 operands, and dz with
// them, are two fp16 halves (22 bits), multiplied as hi lo, lo hi and hi hi, one K
// three times as long; h for the logits is placed row by row.
#include <math.h>

#include "head_few.h"
#include "head_rows.h"
#include "head_tile.h"

namespace pg {
namespace {

int64_t pad(int64_t x, int64_t a) { return (x + a - 1) / a * a; }
int64_t tiles_of(int64_t x, int64_t b) { return (x + b - 1) / b; }
int blocks_for(int64_t items, int most) {
  const int64_t b = (items + 255) / 256;
  return (int)(b < 1 ? 1 : b > most ? most : b);
}
// Blocks of the row kernels, four waves each.
int row_blocks(int64_t rows) { return blocks_for(rows * 64, kRowBlocks); }
int elt_size(int32_t dtype) { return dtype == PG_F32 ? 4 : 2; }

// An operand that the logits' tiles can read where it lies: bf16 rows of whole
// slots at 16-byte alignment.
bool in_place(int32_t dtype, int d, int64_t ld, const void* p) {
  return dtype == PG_BF16 && d % 32 == 0 && d >= 128 && ld % 8 == 0 && ld < (1 << 24) &&
         (uintptr_t)p % 16 == 0;
}

// The same of a table, whose rows are packed and aligned.
bool table_in_place(int32_t dtype, int d) { return in_place(dtype, d, d, nullptr); }

// Whether M x N of K's slots go by large tiles: rounds of tiles over the chip (a
// large one to a compute unit, or two small ones) times a tile's us, 0.95 or 0.6
// a slot and its epilogue.
bool big_tiles(int64_t M, int64_t N, int slots, double epilogue) {
  const double large = (double)tiles_of(tiles_of(M, 256) * tiles_of(N, 256), kCUs) *
                       (0.95 * slots + epilogue);
  const double small = (double)tiles_of(tiles_of(M, 128) * tiles_of(N, 128), 2 * kCUs) *
                       (0.6 * slots + epilogue / 2);
  return large <= small;
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

// The few-token kernels of type T: dz (DZ) or maxima and sums of all of f's rows.
template <typename T, int DZ>
void launch_few(const FewArgs& f, const FewDz& z, unsigned blocks, bool short_table,
                hipStream_t s) {
  void (*kernel)(FewArgs, FewDz);
  if (short_table)
    kernel = f.n <= 16   ? head_few_split_kernel<T, 1, DZ>
             : f.n <= 32 ? head_few_split_kernel<T, 2, DZ>
                         : head_few_split_kernel<T, 4, DZ>;
  else
    kernel = f.n <= 16   ? head_few_kernel<T, 1, DZ>
             : f.n <= 32 ? head_few_kernel<T, 2, DZ>
                         : head_few_kernel<T, 4, DZ>;
  hipLaunchKernelGGL(kernel, dim3(blocks), dim3(256), 0, s, f, z);
}

void launch_copy(bool f32, const RowArgs& r, const PieceArgs& w, bool rows, hipStream_t s) {
  const int rb = rows ? row_blocks(r.vec_pad) : 0;
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
    p.off_wz = take(table_in_place(dtype, d) ? 0 : p.cols * row);
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
    const bool wide = p.planes == 1 && n <= kWide;       // dz in bf16, T as it is
    p.off_w = take(wide ? 0 : p.cols * row);
    // bf16 rows that cannot be read in place: all, or the last ones
    p.off_wz = p.planes == 2 ? at : take((table_in_place(dtype, d) ? 128 : p.cols) * row);
    p.off_dz = take(p.rows * p.cols * 2 * halves);
    p.off_dh = take(p.planes == 2 ? 0 : p.rows * d * 4);  // fp32 adds up in dh
    p.off_dw = n > 32768 ? take(V * d * 4) : at;
    p.off_split = take((int64_t)kCUs * 256 * 256 * 4);   // most tiles at once
    if (!wide) {
      p.pieces = (V + p.cols - 1) / p.cols;
      p.off_stop = take((pad(V, 256) + p.pieces) * 4);
      p.off_level = take(p.rows / 64 * p.cols);
      p.off_cexp = take(p.cols * 4);
    }
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
  if (g.n <= (w_here ? kFew : f32 ? kFewF32 : kFewOdd)) {
    const int groups = (int)tiles_of(g.n, 64);
    const FewArgs f{g.h, g.table, g.ld_h, g.n, g.V, g.d, groups, t.c2,
                    reinterpret_cast<float2*>(ws + p.off_part)};
    const bool short_table = groups == 1 && g.V <= kFewShort;
    parts = tiles_of(g.V, short_table ? 32 : 128);
    const int64_t blocks = groups == 1 ? parts : pad(parts, 8) * groups;
    if (f32) launch_few<float, 0>(f, FewDz{}, (unsigned)blocks, short_table, s);
    else launch_few<uint16_t, 0>(f, FewDz{}, (unsigned)blocks, short_table, s);
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
    const bool big = big_tiles(g.n, g.V < piece ? g.V : piece, t.slots * t.nseg, 6);
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
  const unsigned grid = (unsigned)(alone ? g.n : tiles_of(g.n, 16)), nt = alone ? 256 : 1024;
  auto* join = f32 ? head_join_kernel<float, 16, 1024> : head_join_kernel<uint16_t, 16, 1024>;
  if (alone) join = f32 ? head_join_kernel<float, 1, 256> : head_join_kernel<uint16_t, 1, 256>;
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
  if (more > m - rest) return t1 + (rounds + 1) * lb;
  return fmax(te + (rounds + 1) * lb, t1 + rounds * lb);
}

// The products of a piece: both in one launch; where their tiles are few, K is
// split and a second launch joins the splits.
static hipError_t launch_grads(TileArgs tw, TileArgs th, bool f16, float* split, hipStream_t s) {
  const bool w = tw.out != nullptr, h = th.out != nullptr;
  tw.splits = th.splits = 1;
  // Tile size and K's splits: tiles run longest first, a large one to a compute
  // unit or two small ones; splitting evens out their end, but writes and reads a
  // result more. Times in us: 0.95 a slot of a large tile, 0.6 of a small one
  // (4 more for its start and end; twice as many run at once), 5 MB/us for partial
  // results. (One large product, its tiles two to three rounds: 7 % of the time.)
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
        const double lw = nw ? (double)tw.slots / i + 4 : 0;
        const double lh = nh ? (double)th.slots / j + 4 : 0;
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
  auto pick = [&](auto* one16, auto* one, auto* many16, auto* many_) {
    return many ? (f16 ? many16 : many_) : (f16 ? one16 : one);
  };
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
    // by vocabulary row, and behind them a flag a piece
    auto* stop = reinterpret_cast<int*>(ws + p.off_stop);
    int* any = stop + pad(g.V, 256);
    r.nparts_w = wide ? 0 : blocks_for((g.V * g.d + 7) / 8, kScanBlocks);
    r.nparts_h = row_blocks(r.vec_pad);
    r.hp = reinterpret_cast<uint16_t*>(ws + p.off_h);
    const bool h_here = in_place(g.dtype, g.d, g.ld_h, r.h);
    r.hz = h_here ? nullptr : reinterpret_cast<uint16_t*>(ws + p.off_hz);
    // dz by fragments (of 128 fp32 tokens two groups of 64 took longer than the
    // tiles: 2,048 rows of 2048, 111 us and 95); in fp32 that pass finds T's
    // largest element too, unless other pieces need it first
    const bool few = n <= kFew && (f32 || wide);
    if (few && f32) r.hz = nullptr;
    if (few && f32 && g.n == n && g.V <= p.cols) {
      r.nparts_w = kTops;
      r.clear_w = 1;
    }
    if (!wide) {
      r.clear = few ? any : stop;
      r.nclear = (few ? 0 : pad(g.V, 256)) + p.pieces;
      r.stop = few ? nullptr : reinterpret_cast<uint32_t*>(stop);
    }
    r.c2 = (float)((double)g.scale * (double)g.inv_tau * 1.4426950408889634);
    // T's exponent is the same for every piece of the rows
    const unsigned grid = r.nparts_h + (first_rows && !r.clear_w ? r.nparts_w : 0);
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
      const int64_t ldz = cols, plane = rows * cols;
      auto* level = reinterpret_cast<uint8_t*>(ws + p.off_level);
      int group = (int)rows;                         // rows with levels of their own
      if (few) {
        const FewArgs f{r.h, w.src, g.ld_h, n, c, g.d, 1, r.c2, nullptr};
        const FewDz z{r.a, r.lse2, dz, ldz, plane, (int)rows, r.clear_w ? r.part_w : nullptr,
                      r.sidx, r.sval, (int)(n * g.k), v0, level, any};
        const bool short_table = c <= kFewShort;
        const unsigned blocks = (unsigned)(cols / (short_table ? 32 : 128));
        if (f32) launch_few<float, 1>(f, z, blocks, short_table, s);
        else launch_few<uint16_t, 2>(f, z, blocks, short_table, s);
        if (!wide) {
          copies.level = level;
          copies.any = any;
        }
      }
      launch_copy(f32, r, copies, first && !wide, s);

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
      t.stop = reinterpret_cast<uint32_t*>(stop) + v0;
      t.level = level;
      t.any = any;
      hipError_t e = hipSuccess;
      if (!few) {
        const bool big = big_tiles(rows, cols, t.slots * t.nseg, 9);
        group = big ? 128 : 64;
        e = wide ? launch_tiles<EPI_DZB>(t, rows, cols, big, false, s)
                 : launch_tiles<EPI_DZ>(t, rows, cols, big, f32, s);
      }
      if (e != hipSuccess) return e;
      DzArgs z{r.sidx, r.sval, n, rows, g.k, v0, c, dz, ldz, plane, wide ? 2 : p.planes, !wide};
      z.level = level;
      z.group = group;
      z.groups = (int)tiles_of(rows, group);
      z.any = any;
      z.col_exp = reinterpret_cast<int*>(ws + p.off_cexp);
      z.wp = w.wp;
      z.dp = p.dp;
      z.wplane = cols * p.dp;
      const int cb = wide ? 0 : blocks_for(cols, 2048);
      hipLaunchKernelGGL(head_sparse_kernel, dim3(cb + blocks_for(n * g.k, 8192)), dim3(256), 0, s,
                         z, cb);
      ++any;
      if (!wide && !few) {
        const int db = blocks_for(z.groups * tiles_of(cols, 256) * 256, 1024);
        const int tb = blocks_for(cols * p.dp / 8, 2048);
        hipLaunchKernelGGL(head_level_kernel, dim3(db + tb), dim3(256), 0, s, z, db);
      }

      // dT of the piece: [c x d], K over the rows
      TileArgs tw{}, th{};
      tw.A = Side{ws + p.off_dz, ldz * 2, plane * 2, cols};
      tw.B = Side{ws + p.off_h, dp2, rows * dp2, p.dp};
      tw.nseg = nseg_grad;
      tw.slots = (int)(rows / 32);
      tw.M = c;
      tw.V = g.d;
      if (!wide) {
        tw.row_exp = z.col_exp;
        tw.row_any = z.any;
        tw.all_exp = r.all_h;
      }
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
