// Token embedding and the gradient of its table (gfx950).
//
// Forward: out[t] = scale * T[tokens[t]], one fp32 product rounded once.
// Backward: dT[v] = scale * sum over t with tokens[t] = v of dout[t].
//
// The gradient groups the tokens by row with a stable LSD radix sort (up to
// 9-bit digits: two passes for vocabularies below 2^18), so a row's tokens are
// summed in token order. Up to 4,096 tokens one block sorts in LDS, in one
// launch. Up to 65,536 a digit pass is one launch too: every block counts the
// digits of all tokens itself (at most 256 KiB, from L2) rather than wait for
// the others' counts. Beyond, a pass is three launches: count, scan, scatter.
//
// The sorted positions are cut into chunks of equal length; a wave (or part
// of one, for narrow rows) owns one chunk and a slab of columns, walks its
// positions with the running sum in registers and writes it out where the row
// changes. Rows inside one chunk go straight to the result; a row cut by a
// chunk border leaves its parts in the workspace and a second kernel adds
// them in order. Every wave reads the same number of gradient rows whatever
// the distribution of the tokens, each gradient row is read once, and no
// floating-point atomics are used, so results repeat bit for bit.
#include <type_traits>

#include "train.h"
#include "scan.h"

namespace pg {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxDigitBits = 9;
constexpr int kMaxDigits = 1 << kMaxDigitBits;
// Items a thread of a three-launch sort pass takes: two fill the chip up to
// 2^18 items (a pass over 131,072: 16 us against 21), eight keep the count
// matrix small beyond.
constexpr int kFewItems = 2, kManyItems = 8;
constexpr int64_t kFewLimit = 1 << 18;
constexpr int kSortThreads = 1024;
constexpr int kSmall = 4096;                 // most tokens the one-block sort takes
constexpr int kEmbedBlocks = 4;              // forward blocks a compute unit
// LDS a reduction block asks for without using it: three blocks, twelve waves
// a compute unit, whose eight rows in flight are enough; 268 us at 32 waves,
// 260 at 12 (131,072 rows of 2,560 bf16).
constexpr unsigned kReduceLds = 53 * 1024;
constexpr int64_t kOneLaunch = 65536;        // most tokens a one-launch pass takes

// ---------------------------------------------------------------------------
// Forward

// A group of L lanes covers one row, U vectors of 8 columns a lane at a time:
// the loads of a whole pass are out before the first store. Blocks walk rows
// with the next token in hand, four blocks a compute unit. The output is
// written past the caches, which the table's hot rows keep to themselves.
// 131,072 rows of 2,560 bf16: 208 us with one vector a pass and 32 waves a
// unit, 192 with streaming stores, 180 with the whole pass in flight, 171 with
// 16 waves (180, 175 and 187 with 12, 20 and 32).
template <typename TI, typename TO, int L, int U>
__global__ __launch_bounds__(kThreads) void embed_kernel(
    const TI* __restrict__ table, int64_t V, int d, float scale,
    const int32_t* __restrict__ tokens, int64_t n, TO* __restrict__ out, int64_t ld,
    int32_t* __restrict__ status) {
  const int ln = threadIdx.x & (L - 1);
  const int64_t stride = (int64_t)gridDim.x * (kThreads / L);
  int64_t t = (int64_t)blockIdx.x * (kThreads / L) + threadIdx.x / L;
  int32_t tok = t < n ? tokens[t] : 0;
  for (; t < n; t += stride) {
    const int32_t next = t + stride < n ? tokens[t + stride] : 0;
    const bool ok = tok >= 0 && (int64_t)tok < V;
    if (!ok && ln == 0 && status) atomicOr(status, 1);
    const TI* src = table + (int64_t)(ok ? tok : 0) * d;
    TO* dst = out + t * ld;
    for (int c0 = ln * 8; c0 < d; c0 += U * L * 8) {
      Raw8<TI> r[U];
#pragma unroll
      for (int u = 0; u < U; ++u) r[u] = load8(src + c0 + u * L * 8, ok ? d - c0 - u * L * 8 : 0);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int c = c0 + u * L * 8;
        if (c >= d) continue;
        float y[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = ok ? scale * r[u].get(i) : 0.f;
        store8<true>(dst + c, y, d - c);
      }
    }
    tok = next;
  }
}

// ---------------------------------------------------------------------------
// Sort

// Key of token i: its row, or V (sorted last, no gradient) outside [0, V).
__device__ __forceinline__ uint32_t token_key(int32_t tok, int64_t V) {
  return tok >= 0 && (int64_t)tok < V ? (uint32_t)tok : (uint32_t)V;
}

// Blocks b = 0 .. nb - 1 of NT threads clear the `count` floats at p. The
// dense gradient clears its whole table beside the sort and writes touched
// rows over it: with Zipf tokens few rows are touched, and a flat fill runs
// at 6.8 TB/s where one that skips rows made 2.8 (50,304 rows of 385).
template <int NT>
__device__ __forceinline__ void fill_zero(float* __restrict__ p, int64_t count, int64_t b,
                                          int64_t nb) {
  const float4 z = make_float4(0.f, 0.f, 0.f, 0.f);
  const int64_t vecs = count / 4;
  for (int64_t i = b * NT + threadIdx.x; i < vecs; i += nb * NT) __builtin_memcpy(p + 4 * i, &z, 16);
  if (b == 0 && threadIdx.x < (count & 3)) p[4 * vecs + threadIdx.x] = 0.f;
}

// counts[digit * nblk + b] = keys of block b's tile with that digit. The
// first pass reads the tokens themselves and clears the join lists' counters;
// blocks behind the nblk tiles clear the dense gradient.
template <int kItems>
__global__ __launch_bounds__(kThreads) void embed_hist_kernel(
    const int32_t* __restrict__ tokens, const uint32_t* __restrict__ keys, int64_t n, int64_t V,
    int shift, int digits, int64_t nblk, int32_t* __restrict__ counts, int32_t* __restrict__ list,
    float* __restrict__ fill, int64_t fill_count) {
  __shared__ int32_t c[kMaxDigits];
  if ((int64_t)blockIdx.x >= nblk) {
    fill_zero<kThreads>(fill, fill_count, blockIdx.x - nblk, gridDim.x - nblk);
    return;
  }
  for (int q = threadIdx.x; q < digits; q += kThreads) c[q] = 0;
  if (tokens && blockIdx.x == 0 && threadIdx.x < 2) list[threadIdx.x] = 0;
  __syncthreads();
  const int64_t base = (int64_t)blockIdx.x * (kThreads * kItems);
#pragma unroll
  for (int q = 0; q < kItems; ++q) {
    const int64_t i = base + q * kThreads + threadIdx.x;
    if (i < n) {
      const uint32_t k = tokens ? token_key(tokens[i], V) : keys[i];
      atomicAdd(&c[(k >> shift) & (digits - 1)], 1);
    }
  }
  __syncthreads();
  for (int q = threadIdx.x; q < digits; q += kThreads)
    counts[(int64_t)q * nblk + blockIdx.x] = c[q];
}

// Exclusive scan of the m counts of row blockIdx.x, in place; the row's sum
// goes to totals[blockIdx.x], and as n_unique to a caller who wants it.
template <int NT>
__global__ __launch_bounds__(NT) void embed_scan_kernel(int32_t* __restrict__ a, int64_t m,
                                                        int32_t* __restrict__ totals,
                                                        int64_t* __restrict__ n_unique) {
  __shared__ int32_t sh[NT / 64];
  int32_t* row = a + (int64_t)blockIdx.x * m;
  int32_t run = 0;
  for (int64_t base = 0; base < m; base += NT) {
    const int64_t i = base + threadIdx.x;
    const int32_t x = i < m ? row[i] : 0;
    int32_t tot;
    const int32_t e = block_exclusive_scan<NT>(x, sh, &tot);
    if (i < m) row[i] = run + e;
    run += tot;
  }
  if (threadIdx.x == 0) {
    totals[blockIdx.x] = run;
    if (n_unique) *n_unique = run;
  }
}

// Mask of the wave's live lanes whose digit equals the lane's own.
__device__ __forceinline__ uint64_t same_digit(bool live, int dg, int rb) {
  uint64_t same = __ballot(live);
  for (int bit = 0; bit < rb; ++bit) {
    const uint64_t b = __ballot((dg >> bit) & 1);
    same &= ((dg >> bit) & 1) ? b : ~b;
  }
  return same;
}

// Stable scatter of one digit pass. Items are ranked in order: a wave takes
// 64 consecutive items at a time; lanes of equal digit find each other with
// one ballot per digit bit, and per-wave digit counters in LDS carry the
// order from one step to the next.
template <int kItems>
__global__ __launch_bounds__(kThreads) void embed_scatter_kernel(
    const int32_t* __restrict__ tokens, const uint32_t* __restrict__ kin,
    const int32_t* __restrict__ vin, int64_t n, int64_t V, int shift, int rb,
    const int32_t* __restrict__ counts, const int32_t* __restrict__ totals,
    uint32_t* __restrict__ kout, int32_t* __restrict__ vout) {
  constexpr int kWaves = kThreads / 64;
  __shared__ int32_t wcnt[kWaves][kMaxDigits];   // then the wave's first output position
  __shared__ int32_t sh[kWaves];
  const int digits = 1 << rb;
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  for (int q = threadIdx.x; q < kWaves * kMaxDigits; q += kThreads)
    (&wcnt[0][0])[q] = 0;
  __syncthreads();
  // wave w owns the tile's items [64 w kItems, 64 (w + 1) kItems)
  const int64_t base = ((int64_t)blockIdx.x * kThreads + wave * 64) * kItems;
  uint32_t key[kItems];
  int32_t val[kItems];
  int rank[kItems];                 // rank among the wave's earlier equal digits
#pragma unroll
  for (int q = 0; q < kItems; ++q) {
    const int64_t i = base + q * 64 + lane;
    const bool live = i < n;
    key[q] = live ? (tokens ? token_key(tokens[i], V) : kin[i]) : 0u;
    val[q] = live ? (tokens ? (int32_t)i : vin[i]) : 0;
  }
#pragma unroll
  for (int q = 0; q < kItems; ++q) {
    const bool live = base + q * 64 + lane < n;
    const int dg = (key[q] >> shift) & (digits - 1);
    const uint64_t same = same_digit(live, dg, rb);
    const uint64_t below = same & ((1ull << lane) - 1);
    int before = 0;
    if (live) before = wcnt[wave][dg];
    rank[q] = before + __popcll(below);
    wave_sync();
    if (live && below == 0) wcnt[wave][dg] = before + __popcll(same);
    wave_sync();
  }
  __syncthreads();
  // first output position of (digit, wave): digit base + block offset + the
  // earlier waves' counts
  int32_t run = 0;
  for (int d0 = 0; d0 < digits; d0 += kThreads) {
    const int dg = d0 + threadIdx.x;
    const int32_t x = dg < digits ? totals[dg] : 0;
    int32_t tot;
    const int32_t e = block_exclusive_scan<kThreads>(x, sh, &tot);
    if (dg < digits) {
      int32_t p = run + e + counts[(int64_t)dg * gridDim.x + blockIdx.x];
#pragma unroll
      for (int w = 0; w < kWaves; ++w) {
        const int32_t c = wcnt[w][dg];
        wcnt[w][dg] = p;
        p += c;
      }
    }
    run += tot;
  }
  __syncthreads();
#pragma unroll
  for (int q = 0; q < kItems; ++q) {
    if (base + q * 64 + lane >= n) continue;
    const int dg = (key[q] >> shift) & (digits - 1);
    const int32_t pos = wcnt[wave][dg] + rank[q];
    kout[pos] = key[q];
    vout[pos] = val[q];
  }
}

// ---------------------------------------------------------------------------
// Rows of the sorted order

// heads[c] = sorted positions of chunk c where a new valid row starts.
__global__ __launch_bounds__(kThreads) void embed_heads_kernel(
    const uint32_t* __restrict__ keys, int64_t n, int64_t V, int chunk, int64_t nchunk,
    int32_t* __restrict__ heads) {
  const int lane = threadIdx.x & 63;
  const int64_t c = (int64_t)blockIdx.x * (kThreads / 64) + (threadIdx.x >> 6);
  if (c >= nchunk) return;
  const int64_t i = c * chunk + lane;
  bool head = false;
  if (lane < chunk && i < n) {
    const uint32_t k = keys[i];
    head = (int64_t)k < V && (i == 0 || keys[i - 1] != k);
  }
  const uint64_t m = __ballot(head);
  if (lane == 0) heads[c] = __popcll(m);
}

// The whole sort for n <= kSmall by block 0: digit passes in LDS, then the
// sorted keys and values, the rank first[c] of the first row that starts in
// chunk c, and the number of rows. The other blocks clear the dense gradient.
// R: 64-item rounds of a wave, n <= 1024 R.
template <int R>
__global__ __launch_bounds__(kSortThreads) void embed_sort_kernel(
    const int32_t* __restrict__ tokens, int n, int64_t V, int rb, int passes, int chunk,
    uint32_t* __restrict__ keys, int32_t* __restrict__ vals, int32_t* __restrict__ first,
    int32_t* __restrict__ total, int64_t* __restrict__ n_unique, int32_t* __restrict__ list,
    float* __restrict__ fill, int64_t fill_count) {
  constexpr int kWaves = kSortThreads / 64;
  __shared__ uint32_t kbuf[R * kSortThreads];
  __shared__ uint16_t vbuf[R * kSortThreads];           // positions below 2^12
  __shared__ uint16_t wcnt[kWaves][kMaxDigits];          // counts, then first positions
  __shared__ int32_t sh[kWaves];
  __shared__ int32_t groups[kWaves * R];
  if (blockIdx.x > 0) {
    fill_zero<kSortThreads>(fill, fill_count, blockIdx.x - 1, gridDim.x - 1);
    return;
  }
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int base = wave * R * 64 + lane;                 // wave w owns R * 64 items in a row
  const int digits = 1 << rb;
  uint32_t key[R];
  int val[R], rank[R];
#pragma unroll
  for (int q = 0; q < R; ++q) {
    const int i = base + q * 64;
    key[q] = i < n ? token_key(tokens[i], V) : 0u;
    val[q] = i;
  }
  for (int p = 0; p < passes; ++p) {
    const int shift = p * rb;
    for (int q = threadIdx.x; q < kWaves * kMaxDigits; q += kSortThreads) (&wcnt[0][0])[q] = 0;
    __syncthreads();
#pragma unroll
    for (int q = 0; q < R; ++q) {
      const bool live = base + q * 64 < n;
      const int dg = (key[q] >> shift) & (digits - 1);
      const uint64_t same = same_digit(live, dg, rb);
      const uint64_t below = same & ((1ull << lane) - 1);
      int before = 0;
      if (live) before = wcnt[wave][dg];
      rank[q] = before + __popcll(below);
      wave_sync();
      if (live && below == 0) wcnt[wave][dg] = (uint16_t)(before + __popcll(same));
      wave_sync();
    }
    __syncthreads();
    int sum = 0;
    if ((int)threadIdx.x < digits)
      for (int w = 0; w < kWaves; ++w) sum += wcnt[w][threadIdx.x];
    int32_t tot;
    int pos = block_exclusive_scan<kSortThreads>(sum, sh, &tot);
    if ((int)threadIdx.x < digits)
      for (int w = 0; w < kWaves; ++w) {
        const int c = wcnt[w][threadIdx.x];
        wcnt[w][threadIdx.x] = (uint16_t)pos;            // below n
        pos += c;
      }
    __syncthreads();
#pragma unroll
    for (int q = 0; q < R; ++q) {
      if (base + q * 64 >= n) continue;
      const int at = wcnt[wave][(key[q] >> shift) & (digits - 1)] + rank[q];
      kbuf[at] = key[q];
      vbuf[at] = (uint16_t)val[q];
    }
    __syncthreads();
#pragma unroll
    for (int q = 0; q < R; ++q) {
      const int i = base + q * 64;
      if (i >= n) continue;
      key[q] = kbuf[i];
      val[q] = vbuf[i];
    }
  }
  // rows: heads of each 64-item group, then the ranks at chunk starts
  uint64_t hm[R];
#pragma unroll
  for (int q = 0; q < R; ++q) {
    const int i = base + q * 64;
    bool head = false;
    if (i < n) {
      keys[i] = key[q];
      vals[i] = val[q];
      head = (int64_t)key[q] < V && (i == 0 || kbuf[i - 1] != key[q]);
    }
    hm[q] = __ballot(head);
    if (lane == 0) groups[wave * R + q] = __popcll(hm[q]);
  }
  __syncthreads();
  constexpr int ng = kWaves * R;
  int32_t tot;
  const int g = block_exclusive_scan<kSortThreads>((int)threadIdx.x < ng ? groups[threadIdx.x] : 0,
                                                    sh, &tot);
  if ((int)threadIdx.x < ng) groups[threadIdx.x] = g;
  if (threadIdx.x == 0) {
    *total = tot;
    list[0] = list[1] = 0;
    if (n_unique) *n_unique = tot;
  }
  __syncthreads();
#pragma unroll
  for (int q = 0; q < R; ++q) {
    const int i = base + q * 64;
    if (i < n && (i & (chunk - 1)) == 0)
      first[i / chunk] = groups[wave * R + q] + __popcll(hm[q] & ((1ull << lane) - 1));
  }
}

// One digit pass in one launch for n <= kOneLaunch: the block of tile b counts
// the digits of the tokens before its tile and of all others, which gives
// every output position without the other blocks. A tile is 1,024 items,
// one a thread.
__global__ __launch_bounds__(kSortThreads) void embed_pass_kernel(
    const int32_t* __restrict__ tokens, const uint32_t* __restrict__ kin,
    const int32_t* __restrict__ vin, int n, int64_t V, int shift, int rb, int nblk,
    uint32_t* __restrict__ kout, int32_t* __restrict__ vout, int32_t* __restrict__ list,
    float* __restrict__ fill, int64_t fill_count) {
  constexpr int kWaves = kSortThreads / 64;
  __shared__ int32_t cnt[2][kMaxDigits];                 // before the tile; in it and behind
  __shared__ int32_t wcnt[kWaves][kMaxDigits];           // then the wave's first position
  __shared__ int32_t sh[kWaves];
  if ((int)blockIdx.x >= nblk) {
    fill_zero<kSortThreads>(fill, fill_count, blockIdx.x - nblk, gridDim.x - nblk);
    return;
  }
  const int digits = 1 << rb;
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  for (int q = threadIdx.x; q < kWaves * kMaxDigits; q += kSortThreads) (&wcnt[0][0])[q] = 0;
  if (threadIdx.x < 2 * kMaxDigits) (&cnt[0][0])[threadIdx.x] = 0;
  if (tokens && blockIdx.x == 0 && threadIdx.x < 2) list[threadIdx.x] = 0;
  __syncthreads();
  const auto* src = tokens ? reinterpret_cast<const uint32_t*>(tokens) : kin;
  auto to_key = [&](uint32_t x) { return tokens ? token_key((int32_t)x, V) : x; };
  auto key_at = [&](int i) { return to_key(src[i]); };
  const int t0 = blockIdx.x * kSortThreads;
  // four tokens a load (t0 is a multiple of 4), eight loads in flight
  for (int i0 = 0; i0 < n; i0 += 32 * kSortThreads) {
    uint4 x[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const int i = i0 + 4 * (u * kSortThreads + (int)threadIdx.x);
      x[u] = make_uint4(0, 0, 0, 0);
      if (i + 4 <= n) __builtin_memcpy(&x[u], src + i, 16);
    }
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const int i = i0 + 4 * (u * kSortThreads + (int)threadIdx.x);
      if (i + 4 > n) continue;
      int32_t* c = cnt[i < t0 ? 0 : 1];
      const int m = digits - 1;
      const int da = (to_key(x[u].x) >> shift) & m, db = (to_key(x[u].y) >> shift) & m;
      const int dc = (to_key(x[u].z) >> shift) & m, dd = (to_key(x[u].w) >> shift) & m;
      // a hot token fills most of a wave, whose adds would queue on one
      // address: the digit of the first lane is counted by ballots and added
      // once (the wave lies on one side of t0)
      const int d0 = __builtin_amdgcn_readfirstlane(da);
      const int peeled = __popcll(__ballot(da == d0)) + __popcll(__ballot(db == d0)) +
                         __popcll(__ballot(dc == d0)) + __popcll(__ballot(dd == d0));
      if (lane == __ffsll((unsigned long long)__ballot(true)) - 1) atomicAdd(&c[d0], peeled);
      if (da != d0) atomicAdd(&c[da], 1);
      if (db != d0) atomicAdd(&c[db], 1);
      if (dc != d0) atomicAdd(&c[dc], 1);
      if (dd != d0) atomicAdd(&c[dd], 1);
    }
  }
  if ((int)threadIdx.x < (n & 3))                        // the last tile's or behind it
    atomicAdd(&cnt[1][(key_at((n & ~3) + threadIdx.x) >> shift) & (digits - 1)], 1);
  const int base = t0 + (int)threadIdx.x;
  const bool live = base < n;
  const uint32_t key = live ? key_at(base) : 0u;
  const int32_t val = live ? (tokens ? base : vin[base]) : 0;
  const int dg = (key >> shift) & (digits - 1);
  const uint64_t same = same_digit(live, dg, rb);
  const uint64_t below = same & ((1ull << lane) - 1);
  if (live && below == 0) wcnt[wave][dg] = __popcll(same);
  __syncthreads();
  const bool mine = (int)threadIdx.x < digits;
  int32_t tot;
  const int32_t e = block_exclusive_scan<kSortThreads>(
      mine ? cnt[0][threadIdx.x] + cnt[1][threadIdx.x] : 0, sh, &tot);
  if (mine) {
    int32_t p = e + cnt[0][threadIdx.x];
    for (int w = 0; w < kWaves; ++w) {
      const int32_t c = wcnt[w][threadIdx.x];
      wcnt[w][threadIdx.x] = p;
      p += c;
    }
  }
  __syncthreads();
  if (!live) return;
  const int32_t pos = wcnt[wave][dg] + __popcll(below);
  kout[pos] = key;
  vout[pos] = val;
}

// Ranks of rows in one launch for n <= kOneLaunch: the block of tile b counts
// the heads before its tile itself. first[c]: rank of the first row that
// starts in chunk c; *total, *n_unique: the number of rows.
__global__ __launch_bounds__(kSortThreads) void embed_rank_kernel(
    const uint32_t* __restrict__ keys, int n, int64_t V, int chunk, int32_t* __restrict__ first,
    int32_t* __restrict__ total, int64_t* __restrict__ n_unique) {
  constexpr int kWaves = kSortThreads / 64;
  __shared__ int32_t before[kWaves], groups[kWaves];
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  auto head_at = [&](int i) {
    const uint32_t k = keys[i];
    return (int64_t)k < V && (i == 0 || keys[i - 1] != k);
  };
  const int t0 = blockIdx.x * kSortThreads;
  int c = 0;
  for (int i0 = 0; i0 < t0; i0 += 32 * kSortThreads) {   // t0 is a multiple of 4
    uint4 x[8];
    uint32_t prev[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const int i = i0 + 4 * (u * kSortThreads + (int)threadIdx.x);
      x[u] = make_uint4((uint32_t)V, (uint32_t)V, (uint32_t)V, (uint32_t)V);
      prev[u] = (uint32_t)V;
      if (i < t0) {
        __builtin_memcpy(&x[u], keys + i, 16);
        if (i > 0) prev[u] = keys[i - 1];
      }
    }
#pragma unroll
    for (int u = 0; u < 8; ++u) {                        // V marks no row
      const uint32_t none = (uint32_t)V;
      c += (x[u].x != none && x[u].x != prev[u]) + (x[u].y != none && x[u].y != x[u].x) +
           (x[u].z != none && x[u].z != x[u].y) + (x[u].w != none && x[u].w != x[u].z);
    }
  }
  for (int s = 32; s >= 1; s >>= 1) c += __shfl_xor(c, s, 64);
  if (lane == 0) before[wave] = c;
  const int base = t0 + (int)threadIdx.x;
  const uint64_t hm = __ballot(base < n && head_at(base));
  if (lane == 0) groups[wave] = __popcll(hm);
  __syncthreads();
  int32_t start = 0, mine = 0, all = 0;                  // before the tile, the wave; the tile's
  for (int w = 0; w < kWaves; ++w) {
    start += before[w];
    mine += w < wave ? groups[w] : 0;
    all += groups[w];
  }
  if (threadIdx.x == 0 && t0 + kSortThreads >= n) {      // the last tile
    *total = start + all;
    if (n_unique) *n_unique = start + all;
  }
  if (base < n && (base & (chunk - 1)) == 0)
    first[base / chunk] = start + mine + __popcll(hm & ((1ull << lane) - 1));
}

// Where a finished row goes: rank `seg` of the sparse form, or its row of the
// dense one.
enum { EMBED_SPARSE, EMBED_DENSE, EMBED_ADD };
struct RowOut {
  int64_t* urows;
  float* ugrad;
  float* dtable;
  float scale;
};

// The 8 columns a lane covers start at `col`. A lane whose columns would pass
// the row's end covers its last 8 instead: it computes and writes what its
// neighbour does, and no code for part vectors is needed. Only where that
// cannot be (PARTS: rows of fewer than 8 columns, and the adding form at every
// width, which must read and write an element once) the last lane moves single
// elements (131,072 x 2,560 bf16 of 128,000, added: 276 us, touched rows alone
// 218, with one set of inputs).
template <bool PARTS>
__device__ __forceinline__ int lane_col(int col, int d) {
  return !PARTS && col > d - 8 ? d - 8 : col;
}

// dst[0 .. 8) = f * acc, after dst's old values in the adding form.
template <int MODE, bool PARTS>
__device__ __forceinline__ void put8(float* dst, const float (&acc)[8], float f, bool row,
                                     int cols) {
  const int left = PARTS ? cols : 8;
  float y[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) y[i] = f * acc[i];
  if (MODE == EMBED_ADD && row) {
    const Raw8<float> old = load8(dst, left);
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] += old.get(i);
  }
  store8(dst, y, left);
}

template <int MODE>
__device__ __forceinline__ float* row_dst(const RowOut& o, int64_t seg, uint32_t row, int d) {
  return MODE == EMBED_SPARSE ? o.ugrad + seg * d : o.dtable + (int64_t)row * d;
}

constexpr int kShortParts = 8;

// One group of L lanes per (chunk, slab of 8 L columns; L < 64: the whole
// row). first[c] = rank of the first row that starts in chunk c. part[2 c]:
// the sum of the row that entered chunk c from an earlier one; part[2 c + 1]:
// of the row that starts in c and goes on; such a chunk joins a list of the
// second kernel: rows that reach chunk c + kShortParts (list[0] of them, from
// list[2] on) or shorter ones (list[1], from the list's end back), each in any
// order, for every entry is a row summed by itself. keys and vals are readable
// to a multiple of 8 entries.
template <typename T, int L, int MODE, bool PARTS>
__global__ __launch_bounds__(kThreads) void embed_reduce_kernel(
    const T* __restrict__ dout, int64_t ld, const uint32_t* __restrict__ keys,
    const int32_t* __restrict__ vals, int64_t n, int64_t V, int d, int chunk, int64_t nchunk,
    int slabs, const int32_t* __restrict__ first, float* __restrict__ part, int dpad,
    int32_t* __restrict__ list, RowOut out) {
  const int ln = threadIdx.x & (L - 1);
  int grp = threadIdx.x / L;
  if constexpr (L == 64) grp = __builtin_amdgcn_readfirstlane(grp);   // scalar index loads
  const int64_t w = (int64_t)blockIdx.x * (kThreads / L) + grp;
  const int64_t c = w / slabs;
  if (c >= nchunk) return;
  int col = (int)(w - c * slabs) * 512 + ln * 8;
  if (col >= d) return;
  const bool lead = col == 0;                        // one lane speaks for the row
  col = lane_col<PARTS>(col, d);
  const int left = PARTS ? d - col : 8;
  const int64_t base = c * chunk;
  const int len = (int)(n - base < chunk ? n - base : chunk);
  const uint32_t none = (uint32_t)V;                 // no row: sentinels and the end
  uint32_t prev = base > 0 ? keys[base - 1] : none;  // row of the position before
  int64_t seg = (int64_t)first[c] - 1;               // rank of the row being summed
  bool started = false, any = false;                 // it started here; there is one
  float acc[8] = {};
  float* entered = part + (2 * c) * (int64_t)dpad;
  const T* src = dout + col;
  struct Index {
    uint32_t k[8];
    int32_t v[8];
  };
  auto fetch = [&](int p0) {
    Index x;
    __builtin_memcpy(x.k, keys + base + p0, 32);
    __builtin_memcpy(x.v, vals + base + p0, 32);
    return x;
  };
  // the row that ends at a head, or its part that ends with the chunk
  auto flush = [&](float* part_row) {
    float* dst = part_row ? part_row : row_dst<MODE>(out, seg, prev, d);
    put8<MODE, PARTS>(dst + col, acc, part_row ? 1.0f : out.scale, !part_row, left);
    if (MODE == EMBED_SPARSE && lead && !part_row) out.urows[seg] = (int64_t)prev;
  };
  Index now = fetch(0);
  for (int p0 = 0; p0 < len; p0 += 8) {
    Raw8<T> x[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const bool live = p0 + u < len && now.k[u] != none;
      if (!live) now.k[u] = none;
      x[u] = load8<true>(src + (int64_t)(live ? now.v[u] : 0) * ld, live ? left : 0);
    }
    const Index next = p0 + 8 < len ? fetch(p0 + 8) : now;
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      if (now.k[u] == none) continue;                // only sentinels follow
      if (now.k[u] != prev || base + p0 + u == 0) {
        if (any) flush(started ? nullptr : entered);
        ++seg;
        started = true;
        prev = now.k[u];
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[e] = 0.f;
      }
      any = true;
#pragma unroll
      for (int e = 0; e < 8; ++e) acc[e] += x[u].get(e);
    }
    now = next;
  }
  if (!any) return;
  // does the last row go on in the next chunk?
  const bool goes_on = base + chunk < n && keys[base + chunk] == prev;
  if (started && goes_on && lead) {
    const int64_t far = base + (int64_t)kShortParts * chunk;
    if (far < n && keys[far] == prev)
      list[2 + atomicAdd(list, 1)] = (int32_t)c;
    else
      list[1 + nchunk - atomicAdd(list + 1, 1)] = (int32_t)c;
  }
  flush(!started ? entered : goes_on ? entered + dpad : nullptr);
}

// Rows cut by chunk borders, from the lists: the parts of the row that starts
// in chunk c are part[2 c + 1], part[2 (c + 1)], ... up to the chunk where it
// ends. Blocks below `longs` take the long rows, a block each, split over its
// sixteen waves in order (the hottest row of 131,072 Zipf tokens has about 350
// parts); the others the short ones, a wave each.
constexpr int kJoinThreads = 1024;
template <int MODE, bool PARTS>
__global__ __launch_bounds__(kJoinThreads) void embed_join_kernel(
    const uint32_t* __restrict__ keys, int d, int chunk, int64_t nchunk,
    const int32_t* __restrict__ first, const float* __restrict__ part, int dpad,
    const int32_t* __restrict__ list, int longs, RowOut out) {
  constexpr int kWaves = kJoinThreads / 64;
  __shared__ float red[kWaves][64][8];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const bool act = blockIdx.y * 512 + lane * 8 < d;
  const int col = lane_col<PARTS>(blockIdx.y * 512 + lane * 8, d);
  // parts [lo, hi) of the row that starts in chunk c, added in order
  auto add = [&](int64_t c, int64_t lo, int64_t hi, float (&acc)[8]) {
#pragma unroll 8
    for (int64_t q = lo; q < hi; ++q) {
      const int64_t slot = q == 0 ? 2 * c + 1 : 2 * (c + q);
      const Raw8<float> x = load8(part + slot * dpad + col, act ? 8 : 0);
#pragma unroll
      for (int i = 0; i < 8; ++i) acc[i] += x.get(i);
    }
  };
  auto finish = [&](int64_t c, uint32_t key, const float (&acc)[8]) {
    if (!act) return;
    const int64_t seg = (int64_t)first[c + 1] - 1;
    put8<MODE, PARTS>(row_dst<MODE>(out, seg, key, d) + col, acc, out.scale, true, d - col);
    if (MODE == EMBED_SPARSE && blockIdx.y == 0 && lane == 0) out.urows[seg] = (int64_t)key;
  };
  // the row's parts: up to the chunk behind which another row starts
  auto count_parts = [&](int64_t c, uint32_t key) {
    int64_t e = c + 1;
    for (;;) {
      const int64_t q = e + lane;
      const uint64_t m = __ballot(q + 1 >= nchunk || keys[(q + 1) * chunk] != key);
      if (m) return e + __ffsll((unsigned long long)m) - c;
      e += 64;
    }
  };
  if ((int)blockIdx.x >= longs) {
    const int count = list[1];
    for (int li = (blockIdx.x - longs) * kWaves + wave; li < count;
         li += (gridDim.x - longs) * kWaves) {
      const int64_t c = list[1 + nchunk - li];
      const uint32_t key = keys[(c + 1) * chunk];
      float acc[8] = {};
      add(c, 0, count_parts(c, key), acc);
      finish(c, key, acc);
    }
    return;
  }
  const int count = list[0];
  for (int li = blockIdx.x; li < count; li += longs) {
    const int64_t c = list[2 + li];
    const uint32_t key = keys[(c + 1) * chunk];
    const int64_t parts = count_parts(c, key);
    const int64_t per = (parts + kWaves - 1) / kWaves;
    const int64_t lo = wave * per, hi = lo + per < parts ? lo + per : parts;
    float acc[8] = {};
    add(c, lo, hi, acc);
#pragma unroll
    for (int i = 0; i < 8; ++i) red[wave][lane][i] = acc[i];
    __syncthreads();
    if (wave == 0) {
      const int used = (int)((parts + per - 1) / per);   // waves that had parts
      for (int w = 1; w < used; ++w)
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[i] += red[w][lane][i];
      finish(c, key, acc);
    }
    __syncthreads();
  }
}

// The dense gradient of no tokens.
__global__ __launch_bounds__(kThreads) void embed_zero_kernel(float* __restrict__ p,
                                                              int64_t count) {
  fill_zero<kThreads>(p, count, blockIdx.x, gridDim.x);
}

int64_t al(int64_t x) { return (x + 255) / 256 * 256; }

template <int N>
using IC = std::integral_constant<int, N>;

}  // namespace

hipError_t launch_embed(int32_t table_dtype, const void* table, int64_t V, int d, float scale,
                        const int32_t* tokens, int64_t n, int32_t out_dtype, void* out,
                        int64_t ld, int32_t* status, hipStream_t s) {
  auto go = [&](auto* tab, auto* o) {
    using TI = std::remove_const_t<std::remove_pointer_t<decltype(tab)>>;
    using TO = std::remove_pointer_t<decltype(o)>;
    auto launch = [&](auto L, auto U) {
      const int64_t rows = kThreads / L(), need = (n + rows - 1) / rows, cap = 256 * kEmbedBlocks;
      hipLaunchKernelGGL((embed_kernel<TI, TO, L(), U()>), dim3((unsigned)std::min(need, cap)),
                         dim3(kThreads), 0, s, tab, V, d, scale, tokens, n, o, ld, status);
    };
    if (d <= 64) return launch(IC<8>{}, IC<1>{});
    if (d <= 128) return launch(IC<16>{}, IC<1>{});
    if (d <= 256) return launch(IC<32>{}, IC<1>{});
    switch ((d + 511) / 512) {
      case 1: return launch(IC<64>{}, IC<1>{});
      case 2: return launch(IC<64>{}, IC<2>{});
      case 3: return launch(IC<64>{}, IC<3>{});
      case 4: return launch(IC<64>{}, IC<4>{});
      case 5: return launch(IC<64>{}, IC<5>{});
      default: return launch(IC<64>{}, IC<4>{});
    }
  };
  const auto* tf = static_cast<const float*>(table);
  const auto* tb = static_cast<const uint16_t*>(table);
  if (table_dtype == PG_F32 && out_dtype == PG_F32) go(tf, static_cast<float*>(out));
  else if (table_dtype == PG_F32) go(tf, static_cast<uint16_t*>(out));
  else if (out_dtype == PG_F32) go(tb, static_cast<float*>(out));
  else go(tb, static_cast<uint16_t*>(out));
  return hipGetLastError();
}

namespace {

// Lanes of a reduction group for width d, and the padded width of its parts.
int embed_lanes(int d) { return d <= 64 ? 8 : d <= 128 ? 16 : d <= 256 ? 32 : 64; }
int64_t embed_dpad(int64_t d) { return d <= 256 ? 8 * embed_lanes((int)d) : (d + 511) / 512 * 512; }

}  // namespace

EmbedPlan embed_plan(int64_t n, int64_t V, int d) {
  EmbedPlan p{};
  p.bits = 1;
  while (((int64_t)1 << p.bits) <= V) ++p.bits;      // keys 0 .. V
  p.passes = (p.bits + kMaxDigitBits - 1) / kMaxDigitBits;
  p.rb = (p.bits + p.passes - 1) / p.passes;
  const int64_t few = kThreads * kFewItems, tile = n <= kFewLimit ? few : kThreads * kManyItems;
  p.nblk = (n + tile - 1) / tile;
  const int64_t slabs = ((int64_t)d + 511) / 512;
  p.chunk = 64;
  const int64_t groups = 64 / embed_lanes(d);        // a wave's
  while (p.chunk > 8 && n / p.chunk * slabs < 2048 * groups) p.chunk /= 2;
  p.nchunk = (n + p.chunk - 1) / p.chunk;
  // Room for what any smaller batch needs, whose tiles and chunks may be
  // shorter and more: one workspace serves every batch up to the largest. A
  // chunk of c < 64 is taken up to n / 2c = q - 1, so there are at most 2 q.
  const int64_t q = (2048 * groups + slabs - 1) / slabs;
  const int64_t chunks = std::max(p.nchunk, std::min((n + 7) / 8, 2 * q));
  const int64_t tiles = std::max(p.nblk, (std::min(n, kFewLimit) + few - 1) / few);
  int64_t off = 0;
  for (int i = 0; i < 2; ++i) { p.off_keys[i] = off; off += al((n + 8) * 4); }
  for (int i = 0; i < 2; ++i) { p.off_vals[i] = off; off += al((n + 8) * 4); }
  p.off_counts = off; off += al(((int64_t)1 << p.rb) * tiles * 4);
  p.off_totals = off; off += al((kMaxDigits + 1) * 4);
  p.off_heads = off; off += al((chunks + 1) * 4);
  p.off_list = off; off += al((chunks + 2) * 4);
  p.off_part = off; off += al(2 * chunks * embed_dpad(d) * 4);
  p.bytes = off;
  return p;
}

hipError_t launch_embed_backward(const EmbedPlan& p, const void* dout, int32_t dtype, int64_t ld,
                                 const int32_t* tokens, int64_t n, int64_t V, int d, float scale,
                                 int64_t* urows, float* ugrad, int64_t* n_unique, float* dtable,
                                 int accumulate, void* workspace, hipStream_t s) {
  const int64_t fill_count = dtable && !accumulate ? V * d : 0;
  const int64_t fill_need = (fill_count + 16383) / 16384;
  const int64_t fill_blocks = fill_need < 2048 ? fill_need : 2048;
  const dim3 block(kThreads);
  if (n == 0) {                                      // dense, not accumulating
    hipLaunchKernelGGL(embed_zero_kernel, dim3((unsigned)fill_blocks), block, 0, s, dtable,
                       fill_count);
    return hipGetLastError();
  }
  auto* ws = static_cast<uint8_t*>(workspace);
  uint32_t* keys[2];
  int32_t* vals[2];
  for (int i = 0; i < 2; ++i) {
    keys[i] = reinterpret_cast<uint32_t*>(ws + p.off_keys[i]);
    vals[i] = reinterpret_cast<int32_t*>(ws + p.off_vals[i]);
  }
  auto* counts = reinterpret_cast<int32_t*>(ws + p.off_counts);
  auto* totals = reinterpret_cast<int32_t*>(ws + p.off_totals);
  auto* heads = reinterpret_cast<int32_t*>(ws + p.off_heads);
  auto* list = reinterpret_cast<int32_t*>(ws + p.off_list);
  auto* part = reinterpret_cast<float*>(ws + p.off_part);
  const int slabs = (d + 511) / 512, dpad = (int)embed_dpad(d), lanes = embed_lanes(d);
  const int digits = 1 << p.rb;
  int32_t* total = totals + kMaxDigits;
  const uint32_t* k = keys[0];
  const int32_t* v = vals[0];

  if (n <= kSmall) {
    const int64_t fb = (fill_blocks + 3) / 4;        // blocks four times as wide
    auto sort = [&](auto R) {
      hipLaunchKernelGGL(embed_sort_kernel<R()>, dim3((unsigned)(1 + fb)), dim3(kSortThreads), 0,
                         s, tokens, (int)n, V, p.rb, p.passes, p.chunk, keys[0], vals[0], heads,
                         total, n_unique, list, dtable, fill_count);
    };
    if (n <= kSortThreads) sort(IC<1>{});
    else sort(IC<kSmall / kSortThreads>{});
  } else if (n <= kOneLaunch) {
    const int nblk = (int)((n + kSortThreads - 1) / kSortThreads);
    for (int q = 0; q < p.passes; ++q) {
      const int64_t fb = q == 0 ? (fill_blocks + 3) / 4 : 0;
      hipLaunchKernelGGL(embed_pass_kernel, dim3((unsigned)(nblk + fb)), dim3(kSortThreads), 0, s,
                         q == 0 ? tokens : nullptr, keys[(q + 1) & 1], vals[(q + 1) & 1], (int)n,
                         V, q * p.rb, p.rb, nblk, keys[q & 1], vals[q & 1], list, dtable,
                         fill_count);
    }
    k = keys[(p.passes - 1) & 1];
    v = vals[(p.passes - 1) & 1];
    hipLaunchKernelGGL(embed_rank_kernel, dim3((unsigned)nblk), dim3(kSortThreads), 0, s, k,
                       (int)n, V, p.chunk, heads, total, n_unique);
  } else {
    auto sort = [&](auto ITEMS) {
      for (int q = 0; q < p.passes; ++q) {
        const int shift = q * p.rb;
        const int32_t* tk = q == 0 ? tokens : nullptr;
        const uint32_t* kin = keys[(q + 1) & 1];
        const int32_t* vin = vals[(q + 1) & 1];
        const int64_t fb = q == 0 ? fill_blocks : 0;
        hipLaunchKernelGGL(embed_hist_kernel<ITEMS()>, dim3((unsigned)(p.nblk + fb)), block, 0, s,
                           tk, kin, n, V, shift, digits, p.nblk, counts, list, dtable, fill_count);
        hipLaunchKernelGGL(embed_scan_kernel<kThreads>, dim3((unsigned)digits), block, 0, s,
                           counts, p.nblk, totals, nullptr);
        hipLaunchKernelGGL(embed_scatter_kernel<ITEMS()>, dim3((unsigned)p.nblk), block, 0, s, tk,
                           kin, vin, n, V, shift, p.rb, counts, totals, keys[q & 1], vals[q & 1]);
      }
    };
    if (n <= kFewLimit) sort(IC<kFewItems>{});
    else sort(IC<kManyItems>{});
    k = keys[(p.passes - 1) & 1];
    v = vals[(p.passes - 1) & 1];
    hipLaunchKernelGGL(embed_heads_kernel, dim3((unsigned)((p.nchunk + 3) / 4)), block, 0, s, k, n,
                       V, p.chunk, p.nchunk, heads);
    hipLaunchKernelGGL(embed_scan_kernel<kSortThreads>, dim3(1), dim3(kSortThreads), 0, s, heads,
                       p.nchunk, total, n_unique);
  }
  const RowOut out{urows, ugrad, dtable, scale};
  auto finish = [&](auto MODE, auto PARTS) {
    auto reduce = [&](auto* src, auto L) {
      using T = std::remove_const_t<std::remove_pointer_t<decltype(src)>>;
      const int64_t per = kThreads / L(), groups = p.nchunk * slabs;
      hipLaunchKernelGGL((embed_reduce_kernel<T, L(), MODE(), PARTS()>),
                         dim3((unsigned)((groups + per - 1) / per)), block, kReduceLds, s, src, ld, k, v, n,
                         V, d, p.chunk, p.nchunk, slabs, heads, part, dpad, list, out);
    };
    auto by_lanes = [&](auto* src) {
      if (lanes == 8) reduce(src, IC<8>{});
      else if (lanes == 16) reduce(src, IC<16>{});
      else if (lanes == 32) reduce(src, IC<32>{});
      else reduce(src, IC<64>{});
    };
    if (dtype == PG_F32) by_lanes(static_cast<const float*>(dout));
    else by_lanes(static_cast<const uint16_t*>(dout));
    if (p.nchunk > 1) {
      const int64_t longs = std::min<int64_t>(p.nchunk / kShortParts + 1, 128);
      const int64_t shorts = std::min<int64_t>((p.nchunk + 15) / 16, 256);
      hipLaunchKernelGGL((embed_join_kernel<MODE(), PARTS()>),
                         dim3((unsigned)(longs + shorts), (unsigned)slabs), dim3(kJoinThreads), 0,
                         s, k, d, p.chunk, p.nchunk, heads, part, dpad, list, (int)longs, out);
    }
  };
  auto by_width = [&](auto MODE) {
    if (d < 8) finish(MODE, std::true_type{});
    else finish(MODE, std::false_type{});
  };
  if (!dtable) by_width(IC<EMBED_SPARSE>{});
  else if (!accumulate) by_width(IC<EMBED_DENSE>{});
  else finish(IC<EMBED_ADD>{}, std::true_type{});
  return hipGetLastError();
}

}  // namespace pg
