// Item-id embedding: the lookup that makes a history's feature rows, and the
// gradient of its table.
//
// Lookup: out[t] = scale * table[ids[t]], one 16-byte piece of a row per
// thread and step. It moves each looked-up row in and out once and does one
// multiplication per value, so HBM bounds it.
//
// Gradient: d_table[r] = scale * sum over {t : ids[t] = r} of d_out[t].
// Sorting the tokens by id turns the scattered sum into sums over runs, each
// in the order of the tokens, with no atomics on values: equal calls give
// equal bits. The sort moves 8 bytes per token and the sums read d_out once,
// so writing the table (every row, mostly zeros for a large vocabulary)
// bounds it; the blocks of the sort's launches that the sort does not need
// write the zeros meanwhile.
#include <algorithm>

#include "common.cuh"
#include "history.h"

namespace rest {
namespace {

// ---------------------------------------------------------------- lookup

constexpr int LOOK_THREADS = 256;
constexpr int LOOK_PIECES = 4;  // 16-byte pieces per thread, loads in flight together

template <typename T>
__device__ __forceinline__ uint4 scaled(uint4 u, float s);
template <>
__device__ __forceinline__ uint4 scaled<float>(uint4 u, float s) {
  return make_uint4(__float_as_uint(__uint_as_float(u.x) * s), __float_as_uint(__uint_as_float(u.y) * s),
                    __float_as_uint(__uint_as_float(u.z) * s), __float_as_uint(__uint_as_float(u.w) * s));
}
template <>
__device__ __forceinline__ uint4 scaled<bf16>(uint4 u, float s) {
  uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i)
    w[i] = pack_bf16x2(__uint_as_float(w[i] << 16) * s, __uint_as_float(w[i] & 0xffff0000u) * s);
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// per_row: 16-byte pieces of a row; the block's pieces are consecutive.
template <typename T>
__global__ void __launch_bounds__(LOOK_THREADS) embed_forward_kernel(const uint4* __restrict__ table,
                                                                     const int64_t* __restrict__ ids, float scale,
                                                                     uint4* __restrict__ out, long long n_tokens,
                                                                     long long n_rows, int per_row, int32_t* err) {
  pdl_wait();
  pdl_release();
  const long long base = (long long)blockIdx.x * (LOOK_THREADS * LOOK_PIECES);
  const long long row0 = base / per_row;  // the block's first row and the piece of it that it starts at
  const unsigned rem = (unsigned)(base - row0 * per_row);
  uint4 u[LOOK_PIECES];
  long long row[LOOK_PIECES];
#pragma unroll
  for (int i = 0; i < LOOK_PIECES; ++i) {
    const unsigned local = rem + threadIdx.x + i * LOOK_THREADS;
    const unsigned dr = local / (unsigned)per_row, piece = local - dr * (unsigned)per_row;
    row[i] = row0 + dr;
    u[i] = make_uint4(0, 0, 0, 0);
    if (row[i] < n_tokens) {
      const long long id = ids[row[i]];
      if (id >= 0 && id < n_rows)
        u[i] = table[id * per_row + piece];
      else if (id != -1)
        set_error(err, REST_ERR_INVALID_ARG);
    }
  }
#pragma unroll
  for (int i = 0; i < LOOK_PIECES; ++i)
    if (row[i] < n_tokens) out[base + threadIdx.x + i * LOOK_THREADS] = scaled<T>(u[i], scale);
}

// ---------------------------------------------------------------- sort by id

constexpr int SORT_THREADS = 256, SORT_WARPS = SORT_THREADS / 32;
constexpr int SORT_ITEMS = 4;                         // per thread
constexpr int SORT_TILE = SORT_THREADS * SORT_ITEMS;  // tokens per block

// One digit of a least-significant-digit-first radix sort of (key, token).
// The key is the id, or n_rows for a token that counts nowhere.
struct SortPass {
  const int64_t* ids;  // the first pass reads the ids themselves, in token order
  const uint32_t* keys;
  const uint32_t* toks;
  uint32_t* keys_out;
  uint32_t* toks_out;
  uint32_t* hist;    // [blocks, bins]: tokens per digit; then the blocks before it
  uint32_t* totals;  // [bins]
  int n, n_rows, blocks, shift, bins;
  uint32_t* named;   // first pass: one bit a row of the table, some token names it (null: not wanted)
  // blocks past `blocks` write zeros to table[fill0 .. fill1)
  float4* table;
  long long fill0, fill1;
  int32_t* err;
};

__device__ __forceinline__ uint32_t sort_key(const SortPass& p, int i) {
  if (!p.ids) return p.keys[i];
  const long long id = p.ids[i];
  return id >= 0 && id < p.n_rows ? (uint32_t)id : (uint32_t)p.n_rows;
}

__device__ __forceinline__ bool fill_zero(const SortPass& p) {
  if ((int)blockIdx.x < p.blocks) return false;
  const long long n_fill = gridDim.x - p.blocks;
  const long long stride = n_fill * SORT_THREADS;
  for (long long i = p.fill0 + (blockIdx.x - p.blocks) * (long long)SORT_THREADS + threadIdx.x; i < p.fill1;
       i += stride)
    p.table[i] = make_float4(0.f, 0.f, 0.f, 0.f);
  return true;
}

__global__ void __launch_bounds__(SORT_THREADS) sort_count_kernel(SortPass p) {
  extern __shared__ uint32_t count[];
  pdl_wait();
  pdl_release();
  if (fill_zero(p)) return;
  if (p.named)  // the first scatter sets the bits
    for (long long i = (long long)blockIdx.x * SORT_THREADS + threadIdx.x; i < (p.n_rows + 31LL) / 32;
         i += (long long)p.blocks * SORT_THREADS)
      p.named[i] = 0;
  for (int i = threadIdx.x; i < p.bins; i += SORT_THREADS) count[i] = 0;
  __syncthreads();
  for (int k = 0; k < SORT_ITEMS; ++k) {
    const int i = blockIdx.x * SORT_TILE + k * SORT_THREADS + threadIdx.x;
    if (i >= p.n) break;
    if (p.ids && (p.ids[i] < -1 || p.ids[i] >= p.n_rows)) set_error(p.err, REST_ERR_INVALID_ARG);
    atomicAdd(&count[(sort_key(p, i) >> p.shift) & (p.bins - 1)], 1u);
  }
  __syncthreads();
  for (int i = threadIdx.x; i < p.bins; i += SORT_THREADS) p.hist[(size_t)blockIdx.x * p.bins + i] = count[i];
}

// Per digit, the tokens in the blocks before each block, and all of them: 32
// digits a block, 32 threads a digit, each over a range of the blocks.
__global__ void __launch_bounds__(1024) sort_scan_kernel(SortPass p, int scan_blocks) {
  __shared__ uint32_t part[32][33];
  pdl_wait();
  pdl_release();
  if ((int)blockIdx.x >= scan_blocks) {  // these write zeros
    const long long stride = (long long)(gridDim.x - scan_blocks) * 1024;
    for (long long i = p.fill0 + (blockIdx.x - scan_blocks) * 1024LL + threadIdx.x; i < p.fill1; i += stride)
      p.table[i] = make_float4(0.f, 0.f, 0.f, 0.f);
    return;
  }
  const int x = threadIdx.x & 31, y = threadIdx.x >> 5, bin = blockIdx.x * 32 + x;
  const int per = (p.blocks + 31) / 32, b0 = min(p.blocks, y * per), b1 = min(p.blocks, b0 + per);
  uint32_t sum = 0;
  if (bin < p.bins)
    for (int b = b0; b < b1; ++b) sum += p.hist[(size_t)b * p.bins + bin];
  part[y][x] = sum;
  __syncthreads();
  if (y == 0) {
    uint32_t run = 0;
    for (int j = 0; j < 32; ++j) {
      const uint32_t v = part[j][x];
      part[j][x] = run;
      run += v;
    }
    if (bin < p.bins) p.totals[bin] = run;
  }
  __syncthreads();
  if (bin < p.bins) {
    uint32_t run = part[y][x];
    for (int b = b0; b < b1; ++b) {
      const size_t at = (size_t)b * p.bins + bin;
      const uint32_t v = p.hist[at];
      p.hist[at] = run;
      run += v;
    }
  }
}

// Moves every token behind those with a smaller digit, the blocks before it and
// the tokens before it in its block. A warp takes consecutive tokens, 32 at a
// time in order, so equal digits keep their order.
__global__ void __launch_bounds__(SORT_THREADS) sort_scatter_kernel(SortPass p) {
  extern __shared__ uint32_t smem[];
  uint32_t* base = smem;                                           // [bins]: where the block's tokens of a digit go
  uint16_t* seen = reinterpret_cast<uint16_t*>(smem + p.bins);     // [SORT_WARPS][bins]
  __shared__ uint32_t warp_sum[SORT_WARPS];
  pdl_wait();
  pdl_release();
  if (fill_zero(p)) return;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  for (int i = tid; i < p.bins * SORT_WARPS; i += SORT_THREADS) seen[i] = 0;
  // exclusive prefix of the digits' totals: a contiguous range of digits per thread
  const int per = (p.bins + SORT_THREADS - 1) / SORT_THREADS;
  const int lo = min(p.bins, tid * per), hi = min(p.bins, lo + per);
  uint32_t mine = 0;
  for (int i = lo; i < hi; ++i) mine += p.totals[i];
  uint32_t incl = mine;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const uint32_t v = __shfl_up_sync(0xffffffffu, incl, d);
    if (lane >= d) incl += v;
  }
  if (lane == 31) warp_sum[warp] = incl;
  __syncthreads();
  uint32_t run = incl - mine;
  for (int w = 0; w < warp; ++w) run += warp_sum[w];
  for (int i = lo; i < hi; ++i) {
    base[i] = run + p.hist[(size_t)blockIdx.x * p.bins + i];
    run += p.totals[i];
  }
  uint32_t key[SORT_ITEMS], tok[SORT_ITEMS], rank[SORT_ITEMS];
  uint16_t* my_seen = seen + warp * p.bins;
  const int i0 = blockIdx.x * SORT_TILE + warp * (32 * SORT_ITEMS) + lane;
#pragma unroll
  for (int k = 0; k < SORT_ITEMS; ++k) {
    const int i = i0 + 32 * k;
    const bool in = i < p.n;
    key[k] = in ? sort_key(p, i) : 0u;
    tok[k] = !in ? 0u : p.ids ? (uint32_t)i : p.toks[i];
    if (in && p.named && key[k] < (uint32_t)p.n_rows) atomicOr(&p.named[key[k] >> 5], 1u << (key[k] & 31));
  }
#pragma unroll
  for (int k = 0; k < SORT_ITEMS; ++k) {
    const bool in = i0 + 32 * k < p.n;
    const uint32_t digit = (key[k] >> p.shift) & (p.bins - 1);
    const uint32_t peers = __match_any_sync(0xffffffffu, in ? digit : 0xffffffffu);
    const uint32_t before = in ? my_seen[digit] : 0u;
    rank[k] = before + __popc(peers & ((1u << lane) - 1));
    __syncwarp();
    if (in && (peers >> lane) == 1u) my_seen[digit] = (uint16_t)(rank[k] + 1);  // the last of its peers
    __syncwarp();
  }
  __syncthreads();
  for (int i = tid; i < p.bins; i += SORT_THREADS) {  // seen: the block's tokens of a digit in earlier warps
    uint32_t r = 0;
    for (int w = 0; w < SORT_WARPS; ++w) {
      const uint32_t v = seen[w * p.bins + i];
      seen[w * p.bins + i] = (uint16_t)r;
      r += v;
    }
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < SORT_ITEMS; ++k) {
    if (i0 + 32 * k >= p.n) break;
    const uint32_t digit = (key[k] >> p.shift) & (p.bins - 1);
    const uint32_t at = base[digit] + my_seen[digit] + rank[k];
    p.keys_out[at] = key[k];
    p.toks_out[at] = tok[k];
  }
}

// ---------------------------------------------------------------- sort by id, one block
//
// Up to SMALL_MOST tokens the whole sort is one launch of one block, the tokens
// in shared memory between its passes; three launches a digit cost about 2.5 us
// each. (One cluster of eight blocks for 32k tokens took 30 us, the launches
// above 24 us: eight SMs are too few for the scattered stores.)

constexpr int SMALL_THREADS = 1024, SMALL_WARPS = SMALL_THREADS / 32, SMALL_ITEMS = 4;
constexpr int SMALL_MOST = SMALL_THREADS * SMALL_ITEMS;
constexpr int SMALL_BINS = 256;

struct SmallSort {
  const int64_t* ids;
  uint32_t* keys;
  uint32_t* toks;
  uint32_t* named;  // one bit a row of the table: some token names it (null: not wanted)
  int n, n_rows, passes, bits;
  float4* table;    // blocks past the first write zeros to table[0 .. fill)
  long long fill;
  int32_t* err;
};

__global__ void __launch_bounds__(SMALL_THREADS) sort_small_kernel(SmallSort p) {
  extern __shared__ uint32_t smem[];
  uint32_t* skey = smem;                                                    // [SMALL_MOST]
  uint32_t* stok = smem + SMALL_MOST;                                       // [SMALL_MOST]
  uint16_t* seen = reinterpret_cast<uint16_t*>(smem + 2 * SMALL_MOST);      // [SMALL_WARPS][SMALL_BINS]
  __shared__ uint32_t base[SMALL_BINS];
  __shared__ uint32_t warp_sum[SMALL_BINS / 32];
  pdl_wait();
  pdl_release();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (blockIdx.x > 0) {
    const long long stride = (long long)(gridDim.x - 1) * SMALL_THREADS;
    for (long long i = (blockIdx.x - 1) * (long long)SMALL_THREADS + tid; i < p.fill; i += stride)
      p.table[i] = make_float4(0.f, 0.f, 0.f, 0.f);
    return;
  }
  const int bins = 1 << p.bits;
  const int rounds = (p.n + SMALL_THREADS - 1) / SMALL_THREADS;  // of 32 tokens a warp, consecutive
  const int i0 = warp * 32 * rounds + lane;
  if (p.named)
    for (long long i = tid; i < (p.n_rows + 31LL) / 32; i += SMALL_THREADS) p.named[i] = 0;
  uint32_t key[SMALL_ITEMS], tok[SMALL_ITEMS], place[SMALL_ITEMS];
  __syncthreads();
#pragma unroll
  for (int k = 0; k < SMALL_ITEMS; ++k) {
    const int i = i0 + 32 * k;
    key[k] = tok[k] = 0;
    if (k < rounds && i < p.n) {
      const long long id = p.ids[i];
      const bool in = id >= 0 && id < p.n_rows;
      key[k] = in ? (uint32_t)id : (uint32_t)p.n_rows;
      tok[k] = i;
      if (!in && id != -1) set_error(p.err, REST_ERR_INVALID_ARG);
      if (in && p.named) atomicOr(&p.named[id >> 5], 1u << (id & 31));
    }
  }
  uint16_t* my_seen = seen + warp * SMALL_BINS;
  for (int pass = 0; pass < p.passes; ++pass) {
    const int shift = pass * p.bits;
    for (int i = lane; i < SMALL_BINS / 2; i += 32) reinterpret_cast<uint32_t*>(my_seen)[i] = 0;
    __syncwarp();
#pragma unroll
    for (int k = 0; k < SMALL_ITEMS; ++k) {
      if (k < rounds) {
        const bool in = i0 + 32 * k < p.n;
        const uint32_t digit = (key[k] >> shift) & (bins - 1);
        const uint32_t peers = __match_any_sync(0xffffffffu, in ? digit : 0xffffffffu);
        const uint32_t before = in ? my_seen[digit] : 0u;
        place[k] = before + __popc(peers & ((1u << lane) - 1));
        __syncwarp();
        if (in && (peers >> lane) == 1u) my_seen[digit] = (uint16_t)(place[k] + 1);  // the last of its peers
        __syncwarp();
      }
    }
    __syncthreads();
    // a digit a thread: its tokens in earlier warps, then in smaller digits
    uint32_t total = 0, incl = 0;
    if (tid < SMALL_BINS) {
      uint16_t c[SMALL_WARPS];
#pragma unroll
      for (int w = 0; w < SMALL_WARPS; ++w) c[w] = seen[w * SMALL_BINS + tid];
#pragma unroll
      for (int w = 0; w < SMALL_WARPS; ++w) {
        seen[w * SMALL_BINS + tid] = (uint16_t)total;
        total += c[w];
      }
      incl = total;
#pragma unroll
      for (int x = 1; x < 32; x <<= 1) {
        const uint32_t v = __shfl_up_sync(0xffffffffu, incl, x);
        if (lane >= x) incl += v;
      }
      if (lane == 31) warp_sum[warp] = incl;
    }
    __syncthreads();
    if (tid < SMALL_BINS) {
      uint32_t run = incl - total;
#pragma unroll
      for (int w = 0; w < SMALL_BINS / 32; ++w) run += w < warp ? warp_sum[w] : 0;
      base[tid] = run;
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < SMALL_ITEMS; ++k) {
      if (k < rounds && i0 + 32 * k < p.n) {
        const uint32_t digit = (key[k] >> shift) & (bins - 1);
        const uint32_t at = base[digit] + my_seen[digit] + place[k];
        skey[at] = key[k];
        stok[at] = tok[k];
      }
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < SMALL_ITEMS; ++k) {
      const int i = i0 + 32 * k;
      if (k < rounds && i < p.n) {
        key[k] = skey[i];
        tok[k] = stok[i];
      }
    }
  }
#pragma unroll
  for (int k = 0; k < SMALL_ITEMS; ++k) {
    const int i = i0 + 32 * k;
    if (k < rounds && i < p.n) {
      p.keys[i] = key[k];
      p.toks[i] = tok[k];
    }
  }
}

// ---------------------------------------------------------------- sums over runs

constexpr int RUN_TILE = 16;     // sorted tokens of a group of lanes
constexpr int RUN_COLS = 256;    // columns of a group at most, 8 a lane
constexpr int RUN_THREADS = 128;

struct RunArgs {
  const uint32_t* keys;
  const uint32_t* toks;
  const void* d_out;
  float* d_table;
  float* part;  // [2, tiles, d]: what a tile leaves of the run it starts inside, and of the one it ends inside
  int n, n_rows, d, tiles, accumulate;
  float scale;
  int group;        // lanes of a group
  int sum_blocks, cols;  // cols blocks side by side sum a range of tiles; the grid's other blocks write zeros
  const uint32_t* named;
  long long row0;   // zeros go to the rows from row0 on that no token names
};

template <typename T>
__device__ __forceinline__ void load8(const T* p, float v[8]) {
  load4(p, v);
  load4(p + 4, v + 4);
}
template <>
__device__ __forceinline__ void load8<bf16>(const bf16* p, float v[8]) {
  const uint4 u = *reinterpret_cast<const uint4*>(p);
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}

__device__ __forceinline__ void put_row(const RunArgs& a, uint32_t key, int col, const float acc[8]) {
  float* dst = a.d_table + (size_t)key * a.d + col;
  float v[8];
  if (a.accumulate) load8(dst, v);
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = a.accumulate ? v[i] + acc[i] * a.scale : acc[i] * a.scale;
  store4(dst, v);
  store4(dst + 4, v + 4);
}

// Block `block` of `blocks`: zeros to its share of the rows from row0 on that no
// token names. A warp takes a range of rows, whose bits it loads 32 at a time;
// short rows go several at a time.
__device__ __forceinline__ void zero_rows(const RunArgs& a, long long block, long long blocks) {
  const int quads = a.d / 4, lane = threadIdx.x & 31;
  const int rows = quads < 32 ? 32 / quads : 1;  // rows of a warp at a time
  const int sub = quads < 32 ? lane / quads : 0, q0 = quads < 32 ? lane % quads : lane;
  const long long warps = blocks * (RUN_THREADS / 32), warp = block * (RUN_THREADS / 32) + (threadIdx.x >> 5);
  const long long span = a.n_rows - a.row0, end = a.row0 + span * (warp + 1) / warps;
  for (long long r = a.row0 + span * warp / warps; r < end;) {
    const uint32_t bits = a.named[r >> 5];
    const long long stop = min(end, (r | 31) + 1);
    for (long long z = r + sub; z < stop && sub < rows; z += rows) {
      if ((bits >> (z & 31)) & 1) continue;
      float4* dst = reinterpret_cast<float4*>(a.d_table) + z * quads;
      for (int q = q0; q < quads; q += 32) dst[q] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    r = stop;
  }
}

// Group of lanes: RUN_TILE sorted tokens, 8 columns a lane. A run inside the
// tile goes to its row; one that crosses the tile's ends leaves partial sums.
// Other blocks write the zero rows meanwhile: the sums wait for their tokens'
// rows most of the time.
template <typename T>
__global__ void __launch_bounds__(RUN_THREADS) run_sum_kernel(RunArgs a) {
  pdl_wait();
  pdl_release();
  // sums and zeros take turns in the order of the blocks
  const long long sums = (long long)a.sum_blocks * a.cols, all = gridDim.x;
  const long long unit = blockIdx.x * sums / all;
  if ((blockIdx.x + 1LL) * sums / all == unit) {
    zero_rows(a, blockIdx.x - unit, all - sums);
    return;
  }
  const int per_block = RUN_THREADS / a.group;
  const int tile = (int)(unit / a.cols) * per_block + threadIdx.x / a.group;
  if (tile >= a.tiles) return;
  const int col = (int)(unit % a.cols) * RUN_COLS + (threadIdx.x % a.group) * 8;
  if (col >= a.d) return;
  const int p0 = tile * RUN_TILE, m = min(RUN_TILE, a.n - p0);
  const uint32_t none = 0xffffffffu;  // no id has this key
  const uint32_t prev = p0 > 0 ? a.keys[p0 - 1] : none;
  const uint32_t after = p0 + m < a.n ? a.keys[p0 + m] : none;
  const T* src = reinterpret_cast<const T*>(a.d_out);
  float acc[8] = {};
  constexpr int AHEAD = 8;
  bool starts_here = true;  // the current run starts in this tile
#pragma unroll
  for (int r0 = 0; r0 < RUN_TILE; r0 += AHEAD) {
    if (r0 >= m) break;
    uint32_t key[AHEAD + 1], tok[AHEAD];
#pragma unroll
    for (int j = 0; j <= AHEAD; ++j) key[j] = r0 + j < m ? a.keys[p0 + r0 + j] : after;
#pragma unroll
    for (int j = 0; j < AHEAD; ++j) tok[j] = r0 + j < m ? a.toks[p0 + r0 + j] : 0;
    float x[AHEAD][8];
#pragma unroll
    for (int j = 0; j < AHEAD; ++j)
      if (r0 + j < m) load8(src + (size_t)tok[j] * a.d + col, x[j]);
    if (r0 == 0) starts_here = key[0] != prev;
#pragma unroll
    for (int j = 0; j < AHEAD; ++j) {
      const int r = r0 + j;
      if (r >= m) break;
#pragma unroll
      for (int i = 0; i < 8; ++i) acc[i] += x[j][i];
      const bool ends = key[j + 1] != key[j];
      if (ends || r + 1 == m) {
        if (key[j] < (uint32_t)a.n_rows) {
          if (ends && starts_here) {
            put_row(a, key[j], col, acc);
          } else {
            float* dst = a.part + ((size_t)(starts_here ? a.tiles : 0) + tile) * a.d + col;
            store4(dst, acc);
            store4(dst + 4, acc + 4);
          }
        }
        starts_here = true;
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[i] = 0.f;
      }
    }
  }
}

// Block: the last runs of JOIN_TILES tiles, those that start there and go on in
// later tiles. A warp takes one, or the whole block if it goes on for more than
// JOIN_SHORT tiles, whose partial sums its warps then take in turn.
constexpr int JOIN_THREADS = 256, JOIN_WARPS = JOIN_THREADS / 32, JOIN_TILES = 8, JOIN_SHORT = 8, JOIN_AHEAD = 4;
__device__ __forceinline__ void add_parts(const RunArgs& a, float (&acc)[8], int tile, int col, int j0, int step, int last) {
  for (int j = j0; j <= last; j += step * JOIN_AHEAD) {  // j = 0: the tile's own end
    float x[JOIN_AHEAD][8];
#pragma unroll
    for (int k = 0; k < JOIN_AHEAD; ++k) {
      const int jj = j + k * step;
      if (jj <= last) load8(a.part + ((size_t)(jj == 0 ? a.tiles : 0) + tile + jj) * a.d + col, x[k]);
    }
#pragma unroll
    for (int k = 0; k < JOIN_AHEAD; ++k)
      if (j + k * step <= last)
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[i] += x[k][i];
  }
}
__global__ void __launch_bounds__(JOIN_THREADS) run_join_kernel(RunArgs a) {
  __shared__ float sum[JOIN_WARPS][RUN_COLS];
  __shared__ uint32_t keys[JOIN_TILES];
  __shared__ int longs[JOIN_TILES], n_long;
  __shared__ uint32_t owners;
  pdl_wait();
  pdl_release();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, tile0 = blockIdx.x * JOIN_TILES;
  if (warp == 0) {
    const int p0 = (tile0 + min(lane, JOIN_TILES - 1)) * RUN_TILE, end = p0 + RUN_TILE;
    bool owner = lane < JOIN_TILES && end < a.n;
    if (owner) {
      const uint32_t key = a.keys[end - 1], next = a.keys[end], start = a.keys[p0];
      const uint32_t prev = p0 > 0 ? a.keys[p0 - 1] : 0xffffffffu;
      owner = key < (uint32_t)a.n_rows && next == key && !(start == key && prev == key);  // it starts in this tile
      keys[lane] = key;
    }
    const uint32_t set = __ballot_sync(0xffffffffu, owner);
    if (lane == 0) {
      owners = set;
      n_long = 0;
    }
  }
  __syncthreads();
  const int col = blockIdx.y * RUN_COLS + lane * 8;
  const bool cols = col < a.d;
  int nth = 0;
  for (uint32_t left = owners; left; left &= left - 1, ++nth) {
    if (nth % JOIN_WARPS != warp) continue;
    const int o = __ffs(left) - 1, tile = tile0 + o, u = tile + 1 + lane;
    const uint32_t in = __ballot_sync(0xffffffffu, u < a.tiles && a.keys[(size_t)u * RUN_TILE] == keys[o]);
    const int more = in == 0xffffffffu ? 32 : __ffs(~in) - 1;  // later tiles that begin inside the run
    if (more > JOIN_SHORT) {
      if (lane == 0) longs[atomicAdd(&n_long, 1)] = o;  // in any order: each has its own row
    } else if (cols) {
      float acc[8] = {};
      add_parts(a, acc, tile, col, 0, 1, more);
      put_row(a, keys[o], col, acc);
    }
  }
  __syncthreads();
  for (int l = 0; l < n_long; ++l) {
    const int o = longs[l], tile = tile0 + o;
    int more = 0;
    for (;;) {
      const int u = tile + 1 + more + threadIdx.x;
      const int c = __syncthreads_count(u < a.tiles && a.keys[(size_t)u * RUN_TILE] == keys[o]);
      more += c;
      if (c < JOIN_THREADS) break;
    }
    float acc[8] = {};
    if (cols) add_parts(a, acc, tile, col, warp, JOIN_WARPS, more);
#pragma unroll
    for (int i = 0; i < 8; ++i) sum[warp][lane * 8 + i] = acc[i];
    __syncthreads();
    if (warp == 0 && cols) {
      for (int w = 1; w < JOIN_WARPS; ++w)
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[i] += sum[w][lane * 8 + i];
      put_row(a, keys[o], col, acc);
    }
    __syncthreads();
  }
}

// Digits of the sort: as few passes as digits of at most 11 bits allow (8 bits
// in one block, whose passes are cheap and whose counters a thread has to add
// up), of equal width.
struct Digits { int passes, bits; };
Digits sort_digits(long long n_rows, long long n_tokens) {
  int b = 1;
  while ((1LL << b) <= n_rows) ++b;  // keys 0 .. n_rows
  const int most = n_tokens <= SMALL_MOST ? 8 : 11, passes = (b + most - 1) / most;
  return {passes, (b + passes - 1) / passes};
}

struct EmbedWs {
  size_t keys[2], toks[2], hist, totals, part, named, total;
};
EmbedWs embed_ws(long long n_rows, int d, long long n) {
  EmbedWs w;
  size_t off = 0;
  auto take = [&](size_t b) { size_t o = off; off = (off + b + 255) / 256 * 256; return o; };
  const Digits dg = sort_digits(n_rows, n);
  const long long blocks = (n + SORT_TILE - 1) / SORT_TILE, tiles = (n + RUN_TILE - 1) / RUN_TILE;
  for (int i = 0; i < 2; ++i) {
    w.keys[i] = take(4 * (size_t)n);
    w.toks[i] = take(4 * (size_t)n);
  }
  w.hist = take(((size_t)4 << dg.bits) * blocks);
  w.totals = take((size_t)4 << dg.bits);
  w.part = take((size_t)8 * tiles * d);
  w.named = take((size_t)4 * ((n_rows + 31) / 32));
  w.total = off;
  return w;
}

}  // namespace

cudaError_t launch_embed_forward(bool bf, long long n_rows, int d, const void* table, long long n_tokens,
                                 const int64_t* ids, float scale, void* out, int32_t* err, cudaStream_t s) {
  const int per_row = d * (bf ? 2 : 4) / 16;
  const long long pieces = n_tokens * per_row, per_block = LOOK_THREADS * LOOK_PIECES;
  const dim3 grid((unsigned)((pieces + per_block - 1) / per_block));
  const uint4* t = (const uint4*)table;
  if (bf) return launch_k(embed_forward_kernel<bf16>, grid, dim3(LOOK_THREADS), 0, s, t, ids, scale, (uint4*)out,
                          n_tokens, n_rows, per_row, err);
  return launch_k(embed_forward_kernel<float>, grid, dim3(LOOK_THREADS), 0, s, t, ids, scale, (uint4*)out, n_tokens,
                  n_rows, per_row, err);
}

size_t embed_backward_ws_bytes(long long n_rows, int d, long long n_tokens) {
  return embed_ws(n_rows, d, n_tokens).total;
}

// Sorting launches: one for up to SMALL_MOST tokens, else three a digit.
static int sort_launches(long long n_rows, long long n_tokens) {
  return n_tokens <= SMALL_MOST ? 1 : 3 * sort_digits(n_rows, n_tokens).passes;
}

int embed_backward_launches(long long n_rows, long long n_tokens) { return sort_launches(n_rows, n_tokens) + 2; }

// Launch number `step` of the gradient.
cudaError_t launch_embed_backward(int step, bool bf, long long n_rows, int d, const void* d_out, long long n_tokens,
                                  const int64_t* ids, float scale, bool accumulate, float* d_table, void* ws,
                                  int32_t* err, cudaStream_t s) {
  const EmbedWs w = embed_ws(n_rows, d, n_tokens);
  const Digits dg = sort_digits(n_rows, n_tokens);
  char* base = (char*)ws;
  const int n = (int)n_tokens, blocks = (n + SORT_TILE - 1) / SORT_TILE;
  const int sorts = sort_launches(n_rows, n_tokens);
  // Zeros: each sorting launch writes 26 MB of them beside the sort, whichever rows
  // tokens name; the sums' launch writes the rest, without the rows that tokens
  // name. That is 4 us of stores, more than a sort of 32k tokens alone takes
  // (2.5 us) and less than one of 300k. At 8, 16, 20 and 26 MB: 32k tokens, 200k
  // rows of 512: 96, 103, 101, 103 us; 300k tokens, 1M rows of 64: 119, 109, 107,
  // 106; 5,000 and 100k tokens, 200k rows of 512 and 500k of 256: within 3 %.
  const long long early = n == 0 ? n_rows : std::min<long long>(n_rows, sorts * ((26LL << 20) / (4 * d)));
  const bool late = !accumulate && early < n_rows;
  uint32_t* named = (uint32_t*)(base + w.named);
  auto fill_blocks = [](long long span, int threads) {
    return (int)std::min<long long>((span + threads - 1) / threads, 148 * 2048 / threads);
  };
  if (step < sorts && n <= SMALL_MOST) {
    SmallSort p;
    p.ids = ids;
    p.keys = (uint32_t*)(base + w.keys[0]);
    p.toks = (uint32_t*)(base + w.toks[0]);
    p.named = late ? named : nullptr;
    p.n = n; p.n_rows = (int)n_rows; p.passes = dg.passes; p.bits = dg.bits;
    p.table = (float4*)d_table;
    p.fill = accumulate ? 0 : early * (d / 4);
    p.err = err;
    constexpr int bytes = 8 * SMALL_MOST + 2 * SMALL_WARPS * SMALL_BINS;
    cudaError_t e = cudaFuncSetAttribute(sort_small_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != cudaSuccess) return e;
    return launch_k(sort_small_kernel, dim3(1 + fill_blocks(p.fill, SMALL_THREADS)), dim3(SMALL_THREADS), bytes, s, p);
  }
  if (step < sorts) {
    const int pass = step / 3, kind = step % 3;
    SortPass p;
    p.ids = pass == 0 ? ids : nullptr;
    p.keys = (const uint32_t*)(base + w.keys[(pass + 1) & 1]);
    p.toks = (const uint32_t*)(base + w.toks[(pass + 1) & 1]);
    p.keys_out = (uint32_t*)(base + w.keys[pass & 1]);
    p.toks_out = (uint32_t*)(base + w.toks[pass & 1]);
    p.hist = (uint32_t*)(base + w.hist);
    p.totals = (uint32_t*)(base + w.totals);
    p.named = late && pass == 0 ? named : nullptr;
    p.n = n; p.n_rows = (int)n_rows; p.blocks = blocks; p.shift = pass * dg.bits; p.bins = 1 << dg.bits;
    p.table = (float4*)d_table;
    const long long quads = accumulate ? 0 : early * (d / 4);
    p.fill0 = quads * step / sorts;
    p.fill1 = quads * (step + 1) / sorts;
    p.err = err;
    const int threads = kind == 1 ? 1024 : SORT_THREADS, fill = fill_blocks(p.fill1 - p.fill0, threads);
    if (kind == 0)
      return launch_k(sort_count_kernel, dim3(blocks + fill), dim3(SORT_THREADS), 4 * (size_t)p.bins, s, p);
    if (kind == 1) {
      const int sb = (p.bins + 31) / 32;
      return launch_k(sort_scan_kernel, dim3(sb + fill), dim3(1024), 0, s, p, sb);
    }
    return launch_k(sort_scatter_kernel, dim3(blocks + fill), dim3(SORT_THREADS),
                    (4 + 2 * SORT_WARPS) * (size_t)p.bins, s, p);
  }
  RunArgs a;
  const int last = n <= SMALL_MOST ? 0 : (dg.passes - 1) & 1;
  a.keys = (const uint32_t*)(base + w.keys[last]);
  a.toks = (const uint32_t*)(base + w.toks[last]);
  a.d_out = d_out; a.d_table = d_table; a.part = (float*)(base + w.part);
  a.n = n; a.n_rows = (int)n_rows; a.d = d; a.tiles = (n + RUN_TILE - 1) / RUN_TILE; a.accumulate = accumulate;
  a.scale = scale;
  a.group = 4;
  while (a.group < 32 && a.group * 8 < d) a.group *= 2;
  const int per_block = RUN_THREADS / a.group, cols = (d + RUN_COLS - 1) / RUN_COLS;
  a.sum_blocks = (a.tiles + per_block - 1) / per_block;
  a.cols = cols;
  a.named = named;
  a.row0 = early;
  if (step == sorts) {
    const int fill = late ? fill_blocks((n_rows - early) * (d / 4), RUN_THREADS) : 0;
    const dim3 grid(std::max(1, a.sum_blocks * cols + fill));
    if (bf) return launch_k(run_sum_kernel<bf16>, grid, dim3(RUN_THREADS), 0, s, a);
    return launch_k(run_sum_kernel<float>, grid, dim3(RUN_THREADS), 0, s, a);
  }
  return launch_k(run_join_kernel, dim3(std::max(1, (a.tiles + JOIN_TILES - 1) / JOIN_TILES), cols), dim3(JOIN_THREADS), 0, s, a);
}

}  // namespace rest
