// Token embedding and the gradient of its table (gfx950).
//
// Forward: out[t] = scale * T[tokens[t]], one fp32 product rounded once.
// Backward: dT[v] = scale * sum over t with tokens[t] = v of dout[t].
//
// The gradient groups the tokens by row with a stable LSD radix sort (up to
// 9-bit digits: two passes for vocabularies below 2^18), so a row's tokens are
// summed in token order. The sorted positions are cut into chunks of equal
// length; a wave owns one chunk and a slab of columns, walks its positions
// with the running sum in registers and writes it out where the row changes.
// Rows inside one chunk go straight to the result; a row cut by a chunk
// border leaves its parts in the workspace and a second kernel adds them in
// order. Every wave reads the same number of gradient rows whatever the
// distribution of the tokens, each gradient row is read once, and no
// floating-point atomics are used, so results repeat bit for bit.
#include "train.h"
#include "scan.h"

namespace pg {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxDigitBits = 9;
constexpr int kMaxDigits = 1 << kMaxDigitBits;
constexpr int kItems = 8;
constexpr int kTile = kThreads * kItems;     // items per block of a sort pass

// ---------------------------------------------------------------------------
// Forward

// A group of 2^lg threads covers one row, 8 elements a thread at a time.
template <typename TI, typename TO>
__global__ __launch_bounds__(kThreads) void embed_kernel(
    const TI* __restrict__ table, int64_t V, int d, float scale,
    const int32_t* __restrict__ tokens, int64_t n, TO* __restrict__ out, int64_t ld, int lg,
    int32_t* __restrict__ status) {
  const int tpr = 1 << lg;
  const int ln = threadIdx.x & (tpr - 1);
  const int64_t t = (int64_t)blockIdx.x * (kThreads >> lg) + (threadIdx.x >> lg);
  if (t >= n) return;
  const int32_t tok = tokens[t];
  const bool ok = tok >= 0 && (int64_t)tok < V;
  if (!ok && ln == 0 && status) atomicOr(status, 1);
  const TI* src = table + (int64_t)(ok ? tok : 0) * d;
  TO* dst = out + t * ld;
  for (int c = ln * 8; c < d; c += tpr * 8) {
    const Raw8<TI> r = load8(src + c, ok ? d - c : 0);
    float y[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = ok ? scale * r.get(i) : 0.f;
    store8(dst + c, y, d - c);
  }
}

// ---------------------------------------------------------------------------
// Sort

// Key of token i: its row, or V (sorted last, no gradient) outside [0, V).
__device__ __forceinline__ uint32_t token_key(int32_t tok, int64_t V) {
  return tok >= 0 && (int64_t)tok < V ? (uint32_t)tok : (uint32_t)V;
}

// counts[digit * nblk + b] = keys of block b's tile with that digit. The
// first pass reads the tokens themselves; it also clears present[].
__global__ __launch_bounds__(kThreads) void embed_hist_kernel(
    const int32_t* __restrict__ tokens, const uint32_t* __restrict__ keys, int64_t n, int64_t V,
    int shift, int digits, int32_t* __restrict__ counts, uint8_t* __restrict__ present) {
  __shared__ int32_t c[kMaxDigits];
  for (int q = threadIdx.x; q < digits; q += kThreads) c[q] = 0;
  if (present)
    for (int64_t v = (int64_t)blockIdx.x * kThreads + threadIdx.x; v < V;
         v += (int64_t)gridDim.x * kThreads)
      present[v] = 0;
  __syncthreads();
  const int64_t base = (int64_t)blockIdx.x * kTile;
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
    counts[(int64_t)q * gridDim.x + blockIdx.x] = c[q];
}

// Exclusive scan of the m counts of row blockIdx.x, in place; the row's sum
// goes to totals[blockIdx.x].
__global__ __launch_bounds__(kThreads) void embed_scan_kernel(int32_t* __restrict__ a, int64_t m,
                                                              int32_t* __restrict__ totals) {
  __shared__ int32_t sh[kThreads / 64];
  int32_t* row = a + (int64_t)blockIdx.x * m;
  int32_t run = 0;
  for (int64_t base = 0; base < m; base += kThreads) {
    const int64_t i = base + threadIdx.x;
    const int32_t x = i < m ? row[i] : 0;
    int32_t tot;
    const int32_t e = block_exclusive_scan<kThreads>(x, sh, &tot);
    if (i < m) row[i] = run + e;
    run += tot;
  }
  if (threadIdx.x == 0) totals[blockIdx.x] = run;
}

// Stable scatter of one digit pass. Items are ranked in order: a wave takes
// 64 consecutive items at a time; lanes of equal digit find each other with
// one ballot per digit bit, and per-wave digit counters in LDS carry the
// order from one step to the next.
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
  // wave w owns items [base + w * 512, base + (w + 1) * 512) of the tile
  const int64_t base = (int64_t)blockIdx.x * kTile + (int64_t)wave * (kItems * 64);
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
    uint64_t same = __ballot(live);
    for (int bit = 0; bit < rb; ++bit) {
      const uint64_t b = __ballot((dg >> bit) & 1);
      same &= ((dg >> bit) & 1) ? b : ~b;
    }
    const uint64_t below = same & ((1ull << lane) - 1);
    int before = 0;
    if (live) before = wcnt[wave][dg];
    rank[q] = before + __popcll(below);
    __builtin_amdgcn_wave_barrier();
    if (live && below == 0) wcnt[wave][dg] = before + __popcll(same);
    __builtin_amdgcn_wave_barrier();
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

// heads[c] = sorted positions of chunk c where a new valid row starts; marks
// the rows in present[] (dense form).
__global__ __launch_bounds__(kThreads) void embed_heads_kernel(
    const uint32_t* __restrict__ keys, int64_t n, int64_t V, int chunk, int64_t nchunk,
    int32_t* __restrict__ heads, uint8_t* __restrict__ present) {
  const int lane = threadIdx.x & 63;
  const int64_t c = (int64_t)blockIdx.x * (kThreads / 64) + (threadIdx.x >> 6);
  if (c >= nchunk) return;
  const int64_t i = c * chunk + lane;
  bool head = false;
  if (lane < chunk && i < n) {
    const uint32_t k = keys[i];
    head = (int64_t)k < V && (i == 0 || keys[i - 1] != k);
    if (head && present) present[k] = 1;
  }
  const uint64_t m = __ballot(head);
  if (lane == 0) heads[c] = __popcll(m);
}

__global__ void embed_count_kernel(const int32_t* __restrict__ total,
                                   int64_t* __restrict__ n_unique) {
  *n_unique = *total;
}

// Where a finished row goes.
struct RowOut {
  int64_t* urows;      // sparse: row ids and sums by rank of the row
  float* ugrad;
  float* dtable;       // dense: sums by row (NULL: sparse)
  int accumulate;
  float scale;
};

// 8 columns of a finished row: rank `seg`, table row `row`.
__device__ __forceinline__ void put_row(const RowOut& o, int64_t seg, uint32_t row, int d, int col,
                                        const float (&acc)[8]) {
  float y[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) y[i] = o.scale * acc[i];
  float* p = o.dtable ? o.dtable + (int64_t)row * d + col : o.ugrad + seg * d + col;
  if (o.dtable && o.accumulate) {
    const Raw8<float> old = load8(p, d - col);
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] += old.get(i);
  }
  store8(p, y, d - col);
  if (!o.dtable && col == 0) o.urows[seg] = (int64_t)row;
}

// One wave per (chunk, slab of 512 columns). first[c] = rank of the first row
// that starts in chunk c. part[(2 c) ..]: the sum of the row that entered
// chunk c from an earlier one; part[2 c + 1]: of the row that starts in c and
// goes on.
template <typename T>
__global__ __launch_bounds__(kThreads) void embed_reduce_kernel(
    const T* __restrict__ dout, int64_t ld, const uint32_t* __restrict__ keys,
    const int32_t* __restrict__ vals, int64_t n, int64_t V, int d, int chunk, int64_t nchunk,
    int slabs, const int32_t* __restrict__ first, float* __restrict__ part, int dpad, RowOut out) {
  const int lane = threadIdx.x & 63;
  const int64_t w = (int64_t)blockIdx.x * (kThreads / 64) + (threadIdx.x >> 6);
  const int64_t c = w / slabs;
  if (c >= nchunk) return;
  const int col = (int)(w - c * slabs) * 512 + lane * 8;
  const int64_t base = c * chunk;
  const int64_t i = base + lane;
  const bool in = lane < chunk && i < n;
  const uint32_t key = in ? keys[i] : (uint32_t)V;
  const int32_t val = in ? vals[i] : 0;
  const bool valid = (int64_t)key < V;               // sentinels and the end sort last
  const uint32_t prev = in && i > 0 ? keys[i - 1] : (uint32_t)V;
  const uint64_t headmask = __ballot(valid && (i == 0 || prev != key));
  const int cnt = __popcll(__ballot(valid));         // valid positions of the chunk
  if (cnt == 0) return;
  // does the chunk's last valid row go on in the next chunk?
  const uint32_t last_key = __shfl(key, cnt - 1, 64);
  const bool goes_on = cnt == chunk && base + chunk < n && keys[base + chunk] == last_key;
  const int left = d - col;
  int64_t seg = first[c] - 1;                        // rank of the row being summed
  bool started = false;                              // it started in this chunk
  float acc[8] = {};
  float* entered = part + (2 * c) * (int64_t)dpad + col;
  for (int p0 = 0; p0 < cnt; p0 += 8) {
    Raw8<T> x[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const int p = p0 + u;
      const int32_t tok = __builtin_amdgcn_readlane(val, p & 63);
      x[u] = load8(dout + (int64_t)tok * ld + col, p < cnt ? left : 0);
    }
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const int p = p0 + u;
      if (p >= cnt) break;
      if ((headmask >> p) & 1) {
        if (p > 0) {
          if (started) {
            if (left > 0)
              put_row(out, seg, __builtin_amdgcn_readlane(key, (p - 1) & 63), d, col, acc);
          } else {
            store8(entered, acc, 8);
          }
        }
        ++seg;
        started = true;
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[e] = 0.f;
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) acc[e] += x[u].get(e);
    }
  }
  if (!started)
    store8(entered, acc, 8);
  else if (goes_on)
    store8(entered + dpad, acc, 8);
  else if (left > 0)
    put_row(out, seg, last_key, d, col, acc);
}

// Rows cut by chunk borders: block (c, slab) acts if the last row of chunk c
// starts in it and goes on; its parts are part[2 c + 1], part[2 (c + 1)], ...
// up to the chunk where the row ends, split over the block's waves in order.
__global__ __launch_bounds__(kThreads) void embed_join_kernel(
    const uint32_t* __restrict__ keys, int64_t n, int64_t V, int d, int chunk, int64_t nchunk,
    const int32_t* __restrict__ first, const int32_t* __restrict__ total,
    const float* __restrict__ part, int dpad, RowOut out) {
  constexpr int kWaves = kThreads / 64;
  __shared__ float red[kWaves][64][8];
  const int64_t c = blockIdx.x;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int col = blockIdx.y * 512 + lane * 8;
  const int64_t end = (c + 1) * chunk;               // first position of chunk c + 1
  if (end >= n) return;
  const int32_t next_first = c + 1 < nchunk ? first[c + 1] : *total;
  if (next_first == first[c]) return;                // no row starts in chunk c
  const uint32_t key = keys[end - 1];
  if ((int64_t)key >= V || keys[end] != key) return; // the last row ends here
  // last chunk of the row: the first one after c that does not consist of
  // it alone, or the last chunk
  int64_t e = c + 1;
  for (;;) {
    const int64_t q = e + lane;
    const bool stop = q + 1 >= nchunk || keys[(q + 1) * chunk] != key;
    const uint64_t m = __ballot(stop);
    if (m) {
      e += __ffsll((unsigned long long)m) - 1;
      break;
    }
    e += 64;
  }
  const int64_t parts = e - c + 1;
  const int64_t per = (parts + kWaves - 1) / kWaves;
  const int64_t lo = wave * per, hi = lo + per < parts ? lo + per : parts;
  float acc[8] = {};
#pragma unroll 8
  for (int64_t q = lo; q < hi; ++q) {
    const int64_t slot = q == 0 ? 2 * c + 1 : 2 * (c + q);
    const Raw8<float> x = load8(part + slot * dpad + col, 8);
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[i] += x.get(i);
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) red[wave][lane][i] = acc[i];
  __syncthreads();
  if (wave != 0 || col >= d) return;
#pragma unroll
  for (int w = 1; w < kWaves; ++w)
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[i] += red[w][lane][i];
  put_row(out, (int64_t)next_first - 1, key, d, col, acc);
}

// dtable rows that no token touched (every row without present) = 0.
__global__ __launch_bounds__(kThreads) void embed_zero_kernel(
    const uint8_t* __restrict__ present, int64_t V, int d, float* __restrict__ dtable) {
  const float zero[8] = {};
  const int lane = threadIdx.x & 63;
  for (int64_t v = (int64_t)blockIdx.x * (kThreads / 64) + (threadIdx.x >> 6); v < V;
       v += (int64_t)gridDim.x * (kThreads / 64)) {
    if (present && present[v]) continue;
    for (int c = lane * 8; c < d; c += 512) store8(dtable + v * d + c, zero, d - c);
  }
}

int64_t al(int64_t x) { return (x + 255) / 256 * 256; }

}  // namespace

hipError_t launch_embed(int32_t table_dtype, const void* table, int64_t V, int d, float scale,
                        const int32_t* tokens, int64_t n, int32_t out_dtype, void* out,
                        int64_t ld, int32_t* status, hipStream_t s) {
  const int64_t vecs = ((int64_t)d + 7) / 8;
  int lg = 0;
  while (lg < 6 && ((int64_t)1 << lg) < vecs) ++lg;
  const int64_t rows = kThreads >> lg;
  const dim3 grid((unsigned)((n + rows - 1) / rows));
  auto go = [&](auto* tab, auto* o) {
    hipLaunchKernelGGL(embed_kernel, grid, dim3(kThreads), 0, s, tab, V, d, scale, tokens, n, o,
                       ld, lg, status);
  };
  const auto* tf = static_cast<const float*>(table);
  const auto* tb = static_cast<const uint16_t*>(table);
  if (table_dtype == PG_F32 && out_dtype == PG_F32) go(tf, static_cast<float*>(out));
  else if (table_dtype == PG_F32) go(tf, static_cast<uint16_t*>(out));
  else if (out_dtype == PG_F32) go(tb, static_cast<float*>(out));
  else go(tb, static_cast<uint16_t*>(out));
  return hipGetLastError();
}

EmbedPlan embed_plan(int64_t n, int64_t V, int d) {
  EmbedPlan p{};
  p.bits = 1;
  while (((int64_t)1 << p.bits) <= V) ++p.bits;      // keys 0 .. V
  p.passes = (p.bits + kMaxDigitBits - 1) / kMaxDigitBits;
  p.rb = (p.bits + p.passes - 1) / p.passes;
  p.nblk = (n + kTile - 1) / kTile;
  const int64_t slabs = ((int64_t)d + 511) / 512;
  p.chunk = 64;
  while (p.chunk > 8 && (n / p.chunk) * slabs < 4096) p.chunk /= 2;
  p.nchunk = (n + p.chunk - 1) / p.chunk;
  int64_t off = 0;
  for (int i = 0; i < 2; ++i) { p.off_keys[i] = off; off += al(n * 4); }
  for (int i = 0; i < 2; ++i) { p.off_vals[i] = off; off += al(n * 4); }
  p.off_counts = off; off += al(((int64_t)1 << p.rb) * p.nblk * 4);
  p.off_totals = off; off += al((kMaxDigits + 1) * 4);
  p.off_heads = off; off += al((p.nchunk + 1) * 4);
  p.off_present = off; off += al(V);
  p.off_part = off; off += al(2 * p.nchunk * slabs * 512 * 4);
  p.bytes = off;
  return p;
}

hipError_t launch_embed_backward(const EmbedPlan& p, const void* dout, int32_t dtype, int64_t ld,
                                 const int32_t* tokens, int64_t n, int64_t V, int d, float scale,
                                 int64_t* urows, float* ugrad, int64_t* n_unique, float* dtable,
                                 int accumulate, void* workspace, hipStream_t s) {
  auto zero = [&](const uint8_t* present) {
    const int64_t blocks = (V + 3) / 4;
    hipLaunchKernelGGL(embed_zero_kernel, dim3((unsigned)(blocks < 65536 ? blocks : 65536)),
                       dim3(kThreads), 0, s, present, V, d, dtable);
  };
  if (n == 0) {                                      // dense, not accumulating
    zero(nullptr);
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
  auto* part = reinterpret_cast<float*>(ws + p.off_part);
  const bool fill = dtable && !accumulate;
  uint8_t* present = fill ? ws + p.off_present : nullptr;
  const int slabs = (d + 511) / 512, dpad = slabs * 512;
  const int digits = 1 << p.rb;
  const dim3 block(kThreads);

  for (int q = 0; q < p.passes; ++q) {
    const int shift = q * p.rb;
    const int32_t* tk = q == 0 ? tokens : nullptr;
    const uint32_t* kin = keys[(q + 1) & 1];
    const int32_t* vin = vals[(q + 1) & 1];
    hipLaunchKernelGGL(embed_hist_kernel, dim3((unsigned)p.nblk), block, 0, s, tk, kin, n, V,
                       shift, digits, counts, q == 0 ? present : nullptr);
    hipLaunchKernelGGL(embed_scan_kernel, dim3((unsigned)digits), block, 0, s, counts, p.nblk,
                       totals);
    hipLaunchKernelGGL(embed_scatter_kernel, dim3((unsigned)p.nblk), block, 0, s, tk, kin, vin, n,
                       V, shift, p.rb, counts, totals, keys[q & 1], vals[q & 1]);
  }
  const uint32_t* k = keys[(p.passes - 1) & 1];
  const int32_t* v = vals[(p.passes - 1) & 1];
  int32_t* total = totals + kMaxDigits;
  hipLaunchKernelGGL(embed_heads_kernel, dim3((unsigned)((p.nchunk + 3) / 4)), block, 0, s, k, n,
                     V, p.chunk, p.nchunk, heads, present);
  hipLaunchKernelGGL(embed_scan_kernel, dim3(1), block, 0, s, heads, p.nchunk, total);
  if (n_unique)
    hipLaunchKernelGGL(embed_count_kernel, dim3(1), dim3(1), 0, s, total, n_unique);
  if (fill) zero(present);
  const RowOut out{urows, ugrad, dtable, accumulate, scale};
  const int64_t waves = p.nchunk * slabs;
  const dim3 rgrid((unsigned)((waves + 3) / 4));
  if (dtype == PG_F32)
    hipLaunchKernelGGL(embed_reduce_kernel<float>, rgrid, block, 0, s,
                       static_cast<const float*>(dout), ld, k, v, n, V, d, p.chunk, p.nchunk,
                       slabs, heads, part, dpad, out);
  else
    hipLaunchKernelGGL(embed_reduce_kernel<uint16_t>, rgrid, block, 0, s,
                       static_cast<const uint16_t*>(dout), ld, k, v, n, V, d, p.chunk, p.nchunk,
                       slabs, heads, part, dpad, out);
  if (p.nchunk > 1)
    hipLaunchKernelGGL(embed_join_kernel, dim3((unsigned)p.nchunk, (unsigned)slabs), block, 0, s,
                       k, n, V, d, p.chunk, p.nchunk, heads, total, part, dpad, out);
  return hipGetLastError();
}

}  // namespace pg
