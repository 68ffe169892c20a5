// Decay attention: linear attention with a decay for each head.
#include <algorithm>

#include "common.cuh"
#include "history.h"
#include "sm100.h"
#include "sm100_common.cuh"

namespace rest {
namespace {

// Rotation index of a time head: whole buckets of tau seconds, dt seconds after
// the history's first token (rounded down before it, where only timestamps that
// decrease lead). inv = 1 / tau.
__device__ __forceinline__ long long buckets(long long dt, long long tau, double inv) {
  long long n;
  if (dt >= (1LL << 52) || dt <= -(1LL << 52)) n = dt / tau;
  else n = (long long)((double)dt * inv);  // within one of the quotient: both are below 2^52
  const long long r = dt - n * tau;
  return r < 0 ? n - 1 : r >= tau ? n + 1 : n;
}

// ---------------------------------------------------------------- prologue

// Block: one user. Finds the state it continues, checks its slot, writes the
// user's work items and parts, and moves the state's bookkeeping past the
// call's tokens; the kernels after it read the items alone.
__global__ void __launch_bounds__(128) decay_prep_kernel(DecayUsers users, const int64_t* ts, DecayState st,
                                                         DecayCut cut, DecayItem* items, DecayPart* parts,
                                                         DecayUser* heads, int32_t* err) {
  pdl_wait();
  pdl_release();
  const int u = users.u0 + blockIdx.x;
  const int row0 = users.cu[blockIdx.x], rows = users.cu[blockIdx.x + 1] - row0;
  int slot = -1;
  if (st.s) {
    slot = st.slots ? st.slots[u] : u;
    int bad = slot < -1 || slot >= st.n_slots;
    if (st.slots && slot >= 0 && !bad)
      for (int i = threadIdx.x; i < u; i += 128) bad |= st.slots[i] == slot;
    if (__syncthreads_or(bad)) {
      if (threadIdx.x == 0) set_error(err, REST_ERR_INVALID_ARG);
      slot = -1;
    }
  }
  DecayRec r;
  r.row0 = row0;
  r.slot = slot;
  r.len0 = slot >= 0 ? st.len[slot] : 0;
  r.t0 = r.tprev = 0;
  long long t_last = 0;
  if (ts && rows > 0) {
    r.t0 = r.tprev = ts[row0];
    t_last = ts[row0 + rows - 1];
    if (r.len0 > 0) {
      r.t0 = st.t_first[slot];
      r.tprev = st.t_last[slot];
    }
  }
  const int nseg = (rows + cut.rows - 1) / cut.rows, of_part = cut.rows / cut.m;
  const int np = nseg > 1 ? (rows + of_part - 1) / of_part : 0, p0 = users.part0[blockIdx.x];
  for (int i = threadIdx.x; i < nseg; i += 128)
    items[users.item0[blockIdx.x] + i] = DecayItem{r, row0 + i * cut.rows, min(cut.rows, rows - i * cut.rows), i, nseg,
                                                   p0 + i * cut.m, p0 + min((i + 1) * cut.m, np) - 1};
  for (int i = threadIdx.x; i < np; i += 128)
    parts[p0 + i] = DecayPart{r, row0 + i * of_part, min(of_part, rows - i * of_part), i, np};
  __syncthreads();  // every thread has read the bookkeeping
  if (threadIdx.x != 0) return;
  heads[u] = DecayUser{slot, p0, np, r.len0};
  if (slot >= 0 && rows > 0) {
    st.len[slot] = r.len0 + rows;
    if (ts) {
      if (r.len0 == 0) st.t_first[slot] = r.t0;
      st.t_last[slot] = t_last;
    }
  }
}

// Work item, part and user by number. Of a few users that start empty they
// follow from the row bounds in the arguments, sooner than a load would bring
// them and without the prologue's launch.
__device__ __forceinline__ int few_find(const int32_t* first, int n, int i) {
  int lo = 0, hi = n;  // the last user whose first is at most i has it (users before it may have none)
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (first[mid] <= i) lo = mid;
    else hi = mid;
  }
  return lo;
}
__device__ __forceinline__ DecayRec few_rec(const DecayArgs& a, int u) {
  const long long t0 = a.ts ? a.ts[a.few.cu[u]] : 0;
  return DecayRec{a.few.cu[u], -1, 0, t0, t0};
}
__device__ __forceinline__ int few_parts(const DecayArgs& a, int u) {
  const int rows = a.few.cu[u + 1] - a.few.cu[u], of_part = a.cut.rows / a.cut.m;
  return rows > a.cut.rows ? (rows + of_part - 1) / of_part : 0;
}
__device__ __forceinline__ DecayItem item_at(const DecayArgs& a, int i) {
  if (a.few.n == 0) return a.items[i];
  const int u = few_find(a.few.item0, a.few.n, i), seg = i - a.few.item0[u];
  const int row0 = a.few.cu[u], rows = a.few.cu[u + 1] - row0, at = seg * a.cut.rows, p0 = a.few.part0[u];
  return DecayItem{few_rec(a, u), row0 + at, min(a.cut.rows, rows - at), seg, (rows + a.cut.rows - 1) / a.cut.rows,
                   p0 + seg * a.cut.m, p0 + min((seg + 1) * a.cut.m, few_parts(a, u)) - 1};
}
__device__ __forceinline__ DecayPart part_at(const DecayArgs& a, int i) {
  if (a.few.n == 0) return a.parts[i];
  const int u = few_find(a.few.part0, a.few.n, i), part = i - a.few.part0[u], of_part = a.cut.rows / a.cut.m;
  const int row0 = a.few.cu[u], rows = a.few.cu[u + 1] - row0, at = part * of_part;
  return DecayPart{few_rec(a, u), row0 + at, min(of_part, rows - at), part, few_parts(a, u)};
}
__device__ __forceinline__ DecayUser user_at(const DecayArgs& a, int u) {
  if (a.few.n == 0) return a.users[u];
  return DecayUser{-1, a.few.part0[u], few_parts(a, u), 0};
}

// ---------------------------------------------------------------- products of 64-row blocks
//
// A history is cut into segments and a segment into blocks of 64 rows. With
// S the state at the row before a block, of index n_0, n_1 the index of the
// block's last row and D the matrix exp(g (n_i - n_j)) for j <= i inside it:
//   O = (D * (Q K^T)) V + diag(exp(g (n_i - n_0))) Q S
//   S' = exp(g (n_1 - n_0)) S + (diag(exp(g (n_1 - n_j))) K)^T V
// Every exponent that is used is <= 0, however strong the decay (over a decrease
// of the timestamps it counts as 0). Exponents are formed in 64 bits and kept as a
// pair of floats, within 2^-48 of themselves: a gap of 30 years in buckets of a
// second leaves the rows after it their distances, at g = -1 to 4e-6.
//
// The products run on mma.sync (m16n8k16, bf16 in, fp32 out), which runs at
// 545 TFLOP/s here. Of the three kernels only the segments' own states were tried
// on tcgen05, with their sums in TMEM: no faster than mma.sync (2 x 16384 rows
// 30 us against 26, gradients of 8 x 4096 40 against 42), since what decays the
// rows bounds both. The pass, two thirds of the time, was not: one warp issues a
// tcgen05.mma of M = 128 about every 107 cycles whatever its N, so it would want
// several issuing warps.
//
// An operand is one bf16 number (bf16 calls) or the exact sum of three (fp32
// calls: 8 + 8 + 8 significant bits), and a product sums the pairs of terms
// down to 2^-16 of the largest. What is computed on the way into a product (a
// weighted score into P V, S into Q S, the decayed K into S) is two bf16 terms in
// bf16 calls, within 2^-16, and three in fp32 ones. A bf16 result is then
// rounded once, at the end: its error is that rounding's own, 1.66e-3 of the
// result. With one term each it was 2.4e-3, and 27.2 us instead of 33.3 for
// 32 x 1024 rows, 148 instead of 190 for the gradients of 8 x 4096. Where the
// state is an output, which is fp32, the decayed K has three terms. The tensor
// pipe cuts its fp32 sums off instead of rounding them, which is a bias: with
// three terms each block's products are summed apart and added to the state by
// an ordinary, rounded fma.

constexpr int BLK = 64;        // rows of a block
constexpr int CH_THREADS = 128;  // of the segments' own states

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t a) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a) : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t a) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a) : "memory");
}
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
               : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// The same into c, whatever it held
__device__ __forceinline__ void mma16816_new(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}

// x and y as N bf16 terms each, every term the rest rounded to nearest: three
// hold all of an fp32 number, and a product without its pairs past 2^-16 is off
// by at most 2^-23.
template <int N>
__device__ __forceinline__ void terms2(float x, float y, uint32_t (&t)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) {
    t[i] = pack_bf16x2(x, y);
    if (i + 1 < N) {
      x -= __uint_as_float(t[i] << 16);
      y -= __uint_as_float(t[i] & 0xffff0000u);
    }
  }
}

// A [64, HD] bf16 tile in shared memory: rows of 2 HD bytes, their 16-byte
// pieces permuted as a TMA box with a swizzle of the row's length has them, so
// that ldmatrix reads eight rows without a bank conflict.
template <int HD>
struct Tile {
  static constexpr int PIECES = HD / 8, ROW = HD * 2, PER_LINE = 128 / ROW, BYTES = BLK * ROW;
  __device__ static uint32_t at(int row, int piece) {
    return row * ROW + ((piece ^ ((row / PER_LINE) & (PIECES - 1))) << 4);
  }
};
// The state as an operand: HD rows in the same arrangement.

// Terms of an operand that the call is given (N) and of one that is computed on the way, a weighted score or the
// state (MID)
template <typename T>
struct Terms { static constexpr int N = sizeof(T) == 2 ? 1 : 3, MID = sizeof(T) == 2 ? 2 : 3; };

// fp32 tiles: n rows (zeros up to 64) of a head's columns, from src on, through
// registers into the three planes of a tile. A thread takes one 16-byte column
// of the planes and every STEP-th row.
template <int HD, int THREADS>
__device__ __forceinline__ void split_tile(uint32_t dst, const float* src, int d, int n) {
  using L = Tile<HD>;
  constexpr int STEP = THREADS / L::PIECES;
  const int r0 = threadIdx.x / L::PIECES, c = threadIdx.x % L::PIECES;
  const float* p = src + (size_t)r0 * d + c * 8;
#pragma unroll
  for (int i = 0; i < BLK; i += STEP, p += (size_t)STEP * d) {
    if (BLK % STEP != 0 && r0 + i >= BLK) break;
    float x[8] = {};
    if (r0 + i < n) {
      load4(p, x);
      load4(p + 4, x + 4);
    }
    uint32_t t[4][3];
#pragma unroll
    for (int j = 0; j < 4; ++j) terms2<3>(x[2 * j], x[2 * j + 1], t[j]);
#pragma unroll
    for (int k = 0; k < 3; ++k)
      asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(dst + L::at(r0 + i, c) + k * L::BYTES), "r"(t[0][k]),
                   "r"(t[1][k]), "r"(t[2][k]), "r"(t[3][k]) : "memory");
  }
}

// bf16 tiles arrive by TMA: N boxes of 64 rows a step, `full` one barrier a
// stage. The boxes go on past a history's last row, where the next history's
// rows lie: clear_rows makes them zeros before the products read them.
struct TileMaps { CUtensorMap m[4]; };
template <int HD, int N>
__device__ __forceinline__ void tma_tiles(uint32_t dst, const TileMaps& maps, int x, int y, uint64_t* full) {
  sm100::mbar_arrive_expect_tx(full, N * Tile<HD>::BYTES);
#pragma unroll
  for (int i = 0; i < N; ++i)
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(
            dst + i * Tile<HD>::BYTES),
        "l"(reinterpret_cast<uint64_t>(&maps.m[i])), "r"(x), "r"(y), "r"(sm100::smem_u32(full)) : "memory");
}
// Bounded wait for a phase of a barrier. Unlike the library's other waits it does
// not give up once any error is on record: what these kernels report of a slot or
// a timestamp leaves the outputs as documented. A timeout elsewhere does end it,
// and takes the place of such a report, since it voids the outputs.
__device__ __forceinline__ void wait_phase(uint64_t* bar, uint32_t parity, int32_t* err, volatile int* abort,
                                           long long limit = sm100::kWaitCycles) {
  if (sm100::mbar_try_wait(bar, parity)) return;
  const long long t0 = clock64();
  for (uint32_t n = 1; !sm100::mbar_try_wait(bar, parity); ++n) {
    if ((n & 127) != 0) continue;
    if (*abort) return;
    const bool late = clock64() - t0 > limit;
    if (late && err) atomicExch(reinterpret_cast<int*>(err), REST_ERR_TIMEOUT);
    if (late || (err && *reinterpret_cast<volatile int32_t*>(err) == REST_ERR_TIMEOUT)) {
      *abort = 1;
      return;
    }
  }
}
// A wait that ran out has recorded its error and set the block's abort flag.
// Every warp goes on through its barriers (what it computes is void, and each
// later wait gives up at once), no more copies are started, and before the
// block ends their issuer waits, as long as any wait may, for those in flight.
template <int STAGES>
__device__ __noinline__ void drain(uint64_t* full, int issued, long long limit = sm100::kWaitCycles) {
  int none = 0;
  for (int i = issued > STAGES ? issued - STAGES : 0; i < issued; ++i)
    sm100::mbar_wait_for(&full[i % STAGES], (i / STAGES) & 1, nullptr, &none, limit);
}
template <int HD, int THREADS>
__device__ __forceinline__ void clear_rows(uint32_t tile, int from) {
  using L = Tile<HD>;
  for (int i = from * L::PIECES + threadIdx.x; i < BLK * L::PIECES; i += THREADS)
    asm volatile("st.shared.v4.b32 [%0], {%1,%1,%1,%1};" ::"r"(tile + i * 16), "r"(0) : "memory");
}

// Fragments, for the whole warp. A: 16 rows of the product; B: 16 of its
// columns. The permutation of a row's pieces depends on the row modulo 16, so
// a lane's offset within 16 rows and a 32-byte column pair is fixed.
template <int HD>
struct Frag {
  using L = Tile<HD>;
  static constexpr int N = HD / 16;
  uint32_t o1[N], o2[N];
  __device__ explicit Frag(int lane) {
#pragma unroll
    for (int k = 0; k < N; ++k) {
      o1[k] = L::at(lane & 15, k * 2 + (lane >> 4));
      o2[k] = L::at((lane & 7) + ((lane >> 4) << 3), k * 2 + ((lane >> 3) & 1));
    }
  }
  // A[m][k] = tile[m0 + m][16 kk + k]
  __device__ void a(uint32_t (&r)[4], uint32_t tile, int m0, int kk) const { ldsm4(r, tile + o1[kk] + m0 * L::ROW); }
  // B[k][n] = tile[n0 + n][16 kk + k]
  __device__ void b(uint32_t (&r)[4], uint32_t tile, int n0, int kk) const { ldsm4(r, tile + o2[kk] + n0 * L::ROW); }
  // B[k][n] = tile[k0 + k][16 nn + n]
  __device__ void bt(uint32_t (&r)[4], uint32_t tile, int k0, int nn) const { ldsm4t(r, tile + o1[nn] + k0 * L::ROW); }
};

// Rows (lane / 4, + 8) and columns (2 (lane % 4), + 1) of four 8 x 8 matrices, 16 x 16 of a tile
template <int HD>
__device__ __forceinline__ void stsm4(uint32_t tile, int row, int piece, int lane, const uint32_t (&r)[4]) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.shared.b16 [%0], {%1,%2,%3,%4};" ::"r"(
                   tile + Tile<HD>::at(row + (lane & 15), piece + (lane >> 4))),
               "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]) : "memory");
}

// The terms of w_j x_j for an A fragment whose k index is j: w at j, j + 1, j + 8, j + 9
template <int NT, int KT>
__device__ __forceinline__ void weigh(uint32_t (&out)[KT][4], const uint32_t (&x)[NT][4], const float (&w)[4]) {
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    float lo = 0.f, hi = 0.f;
#pragma unroll
    for (int t = NT - 1; t >= 0; --t) {
      lo += __uint_as_float(x[t][r] << 16);
      hi += __uint_as_float(x[t][r] & 0xffff0000u);
    }
    uint32_t tt[KT];
    terms2<KT>(lo * w[(r >> 1) * 2], hi * w[(r >> 1) * 2 + 1], tt);
#pragma unroll
    for (int t = 0; t < KT; ++t) out[t][r] = tt[t];
  }
}

// c0, c1 (16 x 16) += (FRESH: =) sum over the pairs of terms i + j < LIM of a[i] b[j]. The
// small pairs are summed apart: each sum on the tensor pipe cuts off up to a
// step of what it adds to.
template <int LIM, bool FRESH = false, int NA, int NB>
__device__ __forceinline__ void mma_terms(float (&c0)[4], float (&c1)[4], const uint32_t (&a)[NA][4],
                                          const uint32_t (&b)[NB][4]) {
  if (FRESH) {
    mma16816_new(c0, a[0], b[0][0], b[0][1]);
    mma16816_new(c1, a[0], b[0][2], b[0][3]);
  } else {
    mma16816(c0, a[0], b[0][0], b[0][1]);
    mma16816(c1, a[0], b[0][2], b[0][3]);
  }
  if (LIM == 1 || NA * NB == 1) return;
  float s0[4] = {}, s1[4] = {};
#pragma unroll
  for (int i = NA - 1; i >= 0; --i)
#pragma unroll
    for (int j = NB - 1; j >= 0; --j)
      if (i + j < LIM && i + j > 0) {
        mma16816(s0, a[i], b[j][0], b[j][1]);
        mma16816(s1, a[i], b[j][2], b[j][3]);
      }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    c0[i] += s0[i];
    c1[i] += s1[i];
  }
}

// Which part of the [HD, HD] state update a warp computes: 16 rows, and the
// 16-column groups [n0, n1).
template <int HD>
struct StatePart {
  static constexpr int WM = HD / 16 < 4 ? HD / 16 : 4, WN = HD == 32 ? 2 : 1, NG = HD / 16 / WN;
  __device__ static bool on(int warp) { return warp < WM * WN; }
  __device__ static int m(int warp) { return warp % WM; }
  __device__ static int g(int warp) { return warp / WM; }  // groups g * NG .. g * NG + NG - 1
};

// acc = fade acc + (diag(w) X)^T Y over a block's 64 rows: a warp's part of the state. Y's
// fragments are on their way while X's are weighed, the next X's after them.
template <typename T, int HD, int KT>
__device__ __forceinline__ void add_products(float (*acc)[4], float fade, uint32_t tx, uint32_t ty, uint32_t ox,
                                             const uint32_t* oy, int lane, const float* weight) {
  using L = Tile<HD>;
  using P = StatePart<HD>;
  constexpr int NT = Terms<T>::N;
  constexpr bool APART = KT == 3;
  float block[APART ? 2 * P::NG : 1][4] = {};
  float(*sum)[4] = APART ? block : acc;
  if (!APART) {
#pragma unroll
    for (int n = 0; n < 2 * P::NG; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[n][i] *= fade;
  }
  constexpr int XA = NT == 1 ? 2 : 1, YB = NT == 1 ? P::NG : 1;
  uint32_t xa[XA][NT][4], yb[YB][NT][4];
  auto read_x = [&](int kb) {
#pragma unroll
    for (int t = 0; t < NT; ++t) ldsm4t(xa[kb % XA][t], tx + t * L::BYTES + kb * 16 * L::ROW + ox);
  };
  auto read_y = [&](int kb, int g) {
#pragma unroll
    for (int t = 0; t < NT; ++t) ldsm4t(yb[g % YB][t], ty + t * L::BYTES + kb * 16 * L::ROW + oy[g]);
  };
  if (NT == 1) read_x(0);
#pragma unroll
  for (int kb = 0; kb < BLK / 16; ++kb) {
    if (NT == 1) {
#pragma unroll
      for (int g = 0; g < P::NG; ++g) read_y(kb, g);
      if (kb + 1 < BLK / 16) read_x(kb + 1);
    } else {
      read_x(kb);
    }
    const float2 w0 = *reinterpret_cast<const float2*>(&weight[kb * 16 + (lane & 3) * 2]);
    const float2 w1 = *reinterpret_cast<const float2*>(&weight[kb * 16 + (lane & 3) * 2 + 8]);
    uint32_t xw[KT][4];
    weigh<NT, KT>(xw, xa[kb % XA], {w0.x, w0.y, w1.x, w1.y});
    if (NT == 1) {
      // term by term over all columns, so that no product waits for the one before it
#pragma unroll
      for (int i = 0; i < KT; ++i)
#pragma unroll
        for (int g = 0; g < P::NG; ++g) {
          mma16816(sum[2 * g], xw[i], yb[g % YB][0][0], yb[g % YB][0][1]);
          mma16816(sum[2 * g + 1], xw[i], yb[g % YB][0][2], yb[g % YB][0][3]);
        }
    } else {
#pragma unroll
      for (int g = 0; g < P::NG; ++g) {
        read_y(kb, g);
        mma_terms<3>(sum[2 * g], sum[2 * g + 1], xw, yb[g % YB]);
      }
    }
  }
  if (APART) {
#pragma unroll
    for (int n = 0; n < 2 * P::NG; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[n][i] = acc[n][i] * fade + block[n][i];
  }
}

// ---------------------------------------------------------------- rotation indexes

// The head's rotation index of a row, less the one of the history's first row.
struct Index {
  long long tau, t0, len0;
  double inv;
  int row0;
  const int64_t* ts;
  __device__ long long of_time(long long t) const { return buckets(t - t0, tau, inv); }
  // of the history's last cached row; without one, of its first row
  __device__ long long before(const DecayRec& rec) const {
    return tau > 0 ? of_time(rec.tprev) : rec.len0 > 0 ? rec.len0 - 1 : 0;
  }
  __device__ long long of_row(int row) const { return tau > 0 ? of_time(ts[row]) : len0 + (row - row0); }
};
__device__ __forceinline__ Index head_index(const DecayArgs& a, const DecayRec& rec, int h) {
  Index x;
  x.tau = a.h.tau[h];
  x.inv = a.h.inv[h];
  x.t0 = rec.t0;
  x.len0 = rec.len0;
  x.row0 = rec.row0;
  x.ts = a.ts;
  return x;
}
// decay2 * steps as two floats (positive where the timestamps decrease on the way: what becomes of two such
// exponents' difference is clamped, not they, so that rows on one side of a decrease keep their distance)
__device__ __forceinline__ float2 exponent(double decay2, long long steps) {
  const double x = decay2 * (double)steps;
  const float hi = (float)x;
  return make_float2(hi, (float)(x - (double)hi));
}
// 2^min(hi + lo, 0): over a decrease of the timestamps the sum is positive. The approximation is off by 2^-22, which a state
// that is an output, or fp32 rows, show after a few factors: FINE sums the
// exponential series of the fraction (|f ln 2| <= 0.35: the eighth power's term
// is below 2^-27) and puts the whole part into the exponent.
template <bool FINE>
__device__ __forceinline__ float decay_exp2(float hi, float lo) {
  if (!FINE) return exp2_approx(fminf(hi + lo, 0.f));
  if (hi + lo >= 0.f) return 1.f;
  if (hi + lo < -126.f) return 0.f;
  const float n = rintf(hi + lo), t = ((hi - n) + lo) * 0.69314718055994531f;
  float p = 1.f / 5040;
  p = p * t + 1.f / 720;
  p = p * t + 1.f / 120;
  p = p * t + 1.f / 24;
  p = p * t + 1.f / 6;
  p = p * t + 0.5f;
  p = p * t + 1.f;
  p = p * t + 1.f;
  return fminf(p * __int_as_float(((int)n + 127) << 23), 1.f);
}
template <bool FINE>
__device__ __forceinline__ float decay_between(float2 later, float2 earlier) {
  return decay_exp2<FINE>(later.x - earlier.x, later.y - earlier.y);
}

// ---------------------------------------------------------------- a segment's own state

template <typename T>
__host__ __device__ constexpr int part_stages() { return sizeof(T) == 2 ? 3 : 1; }

// Block: one part and head (blockIdx.y = 0: sum_j exp(g (n' - n_j)) k_j v_j^T, n'
// the part's last index, for segments that have a next one; blockIdx.y = 1,
// backward: sum_i exp(g (n_i - n')) q_i do_i^T, n' the index before the part, for
// those that have a previous one). Writes the sum and the decay that a state
// takes over the part.
template <typename T, int HD, int KT>
__global__ void __launch_bounds__(CH_THREADS) decay_part_kernel(const __grid_constant__ TileMaps maps0,
                                                                   const __grid_constant__ TileMaps maps1,
                                                                   const __grid_constant__ DecayArgs a,
                                                                   const T* x0, const T* y0, const T* x1, const T* y1) {
  using L = Tile<HD>;
  using P = StatePart<HD>;
  constexpr int NT = Terms<T>::N, PLANE = NT * L::BYTES, STAGES = part_stages<T>();
  extern __shared__ __align__(1024) char smem[];
  __shared__ float wt[2][BLK];
  __shared__ uint64_t full[STAGES];
  __shared__ int abort_flag;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, d = a.d;
  if (tid == 0) {
    abort_flag = 0;
    for (int i = 0; i < STAGES; ++i) sm100::mbar_init(&full[i], 1);
    sm100::fence_mbar_init();
    if (NT == 1)
      for (int i = 0; i < 2; ++i) sm100::prefetch_tmap(blockIdx.y == 1 ? &maps1.m[i] : &maps0.m[i]);
  }
  __syncthreads();
  pdl_wait();
  pdl_release();
  const int H = a.h.n_heads, h = blockIdx.x % H;
  const DecayPart it = part_at(a, blockIdx.x / H);
  const bool rev = blockIdx.y == 1;
  const int seg = it.part / a.cut.m, last_seg = (it.parts - 1) / a.cut.m;
  if (rev ? seg == 0 : seg == last_seg) return;
  const uint32_t base = sm100::smem_u32(smem);
  const size_t off = (size_t)it.row0 * d + h * HD;
  const int blocks = (it.rows + BLK - 1) / BLK;
  int issued = 0;
  auto stopped = [&] { return *reinterpret_cast<volatile int*>(&abort_flag) != 0; };
  auto load = [&](int c) {
    const uint32_t buf = base + (c % STAGES) * 2 * PLANE;
    if constexpr (NT == 1) {
      if (tid == 0 && !stopped()) {
        tma_tiles<HD, 2>(buf, rev ? maps1 : maps0, h * HD, it.row0 + c * BLK, &full[c % STAGES]);
        issued = c + 1;
      }
    } else {
      const size_t at = off + (size_t)c * BLK * d;
      split_tile<HD, CH_THREADS>(buf, (rev ? x1 : x0) + at, d, it.rows - c * BLK);
      split_tile<HD, CH_THREADS>(buf + PLANE, (rev ? y1 : y0) + at, d, it.rows - c * BLK);
    }
  };
  if (STAGES > 1)
    for (int c = 0; c < STAGES - 1 && c < blocks; ++c) load(c);
  const DecayRec& rec = it.rec;
  const Index ix = head_index(a, rec, h);
  const double decay2 = a.h.decay2[h];
  const long long n_last = ix.of_row(it.row0 + it.rows - 1);
  const long long n_before = it.part > 0 ? ix.of_row(it.row0 - 1) : ix.before(rec);
  long long t_row = 0;
  auto read_time = [&](int c) {
    if (tid < BLK && c < blocks && ix.tau > 0) t_row = a.ts[it.row0 + min(it.rows - 1, c * BLK + tid)];
  };
  auto put_weights = [&](int c) {
    if (tid < BLK && c < blocks) {
      const long long n = ix.tau > 0 ? ix.of_time(t_row) : ix.len0 + (it.row0 + min(it.rows - 1, c * BLK + tid) - ix.row0);
      const float2 e = exponent(decay2, rev ? n - n_before : n_last - n);
      wt[c & 1][tid] = decay_exp2<KT == 3>(e.x, e.y);
    }
  };
  // x by its columns that are this warp's rows of the state, y by the state's columns
  const uint32_t ox = L::at((lane & 7) + ((lane >> 4) << 3), P::m(warp) * 2 + ((lane >> 3) & 1));
  uint32_t oy[P::NG];
#pragma unroll
  for (int g = 0; g < P::NG; ++g) oy[g] = L::at(lane & 15, (P::g(warp) * P::NG + g) * 2 + (lane >> 4));
  float acc[2 * P::NG][4] = {};
  read_time(0);
  put_weights(0);
  read_time(1);
  for (int c = 0; c < blocks; ++c) {
    __syncthreads();
    if (STAGES > 1) {
      if (c + STAGES - 1 < blocks) load(c + STAGES - 1);
      wait_phase(&full[c % STAGES], (c / STAGES) & 1, a.err, &abort_flag);
    } else {
      load(c);
      __syncthreads();
    }
    const uint32_t tx = base + (c % STAGES) * 2 * PLANE, ty = tx + PLANE;
    if (NT == 1 && it.rows - c * BLK < BLK) {
      clear_rows<HD, CH_THREADS>(tx, it.rows - c * BLK);
      clear_rows<HD, CH_THREADS>(ty, it.rows - c * BLK);
      __syncthreads();
    }
    if (P::on(warp)) add_products<T, HD, KT>(acc, 1.f, tx, ty, ox, oy, lane, wt[c & 1]);
    put_weights(c + 1);
    read_time(c + 2);
    if (STAGES == 1) __syncthreads();
  }
  if (STAGES > 1 && tid == 0 && stopped()) drain<STAGES>(full, issued);
  const size_t at = (size_t)blockIdx.x + (rev ? (size_t)gridDim.x : 0);
  if (P::on(warp)) {
    float* out = a.part_state + at * HD * HD + (P::m(warp) * 16 + (lane >> 2)) * HD + P::g(warp) * P::NG * 16 + (lane & 3) * 2;
#pragma unroll
    for (int n = 0; n < 2 * P::NG; ++n) {
      store2(out + n * 8, acc[n][0], acc[n][1]);
      store2(out + 8 * HD + n * 8, acc[n][2], acc[n][3]);
    }
  }
  if (tid == 0) {
    const float2 f = exponent(decay2, n_last - n_before);
    a.part_decay[at] = decay_exp2<KT == 3>(f.x, f.y);
  }
}

// The state before every segment (blockIdx.z = 1: after it) from the parts' own,
// for users with more than one. Thread: two state values; the parts' values do
// not depend on one another, so 16 loads go out at once, and the decays' beside
// the first of them. Waiting for these loads is all that bounds it: one value a
// thread, for twice the blocks, took 13 us instead of 9 (8 x 4096 rows backward),
// and 32 loads at once, whose registers hold an SM to four blocks, 24.
constexpr int JOIN_THREADS = 128, JOIN_AHEAD = 16, JOIN_VALUES = 2;
template <int HD>
__global__ void __launch_bounds__(JOIN_THREADS, 10) decay_join_kernel(const __grid_constant__ DecayArgs a) {
  __shared__ float decays[JOIN_THREADS];
  pdl_wait();
  pdl_release();
  const int H = a.h.n_heads, h = blockIdx.x % H, m = a.cut.m;
  const DecayUser u = user_at(a, blockIdx.x / H);
  if (u.parts == 0) return;
  const bool rev = blockIdx.z == 1;
  const int at = (blockIdx.y * JOIN_THREADS + threadIdx.x) * JOIN_VALUES, last = u.parts - 1;
  float2 S = make_float2(0.f, 0.f);
  if (!rev && u.slot >= 0 && u.len0 > 0)
    S = *reinterpret_cast<const float2*>(a.state + ((size_t)u.slot * H + h) * HD * HD + at);
  // forwards from the first part up to the last segment's, backwards from the
  // last part down to the first segment's
  const int steps = rev ? u.parts - m : last / m * m;
  const long long step = (rev ? -1LL : 1LL) * H;
  const size_t first = ((size_t)(rev ? a.n_parts : 0) + u.part0 + (rev ? last : 0)) * H + h;
  float* state = a.part_state + first * HD * HD + at;
  const long long stride = step * (HD * HD);
  // a counter of the parts left until the next store: at a segment's first part,
  // backwards at its last (the last segment may have fewer parts)
  int left = 0;
  const int after_first = rev ? last % m + 1 : m;
  for (int s0 = 0; s0 <= steps; s0 += JOIN_AHEAD) {
    const bool fresh = s0 % JOIN_THREADS == 0;  // the next parts' decays, beside their values
    float decay = 0.f;
    if (fresh && s0 + (int)threadIdx.x < steps) decay = a.part_decay[first + (s0 + threadIdx.x) * step];
    float2 own[JOIN_AHEAD];
#pragma unroll
    for (int k = 0; k < JOIN_AHEAD; ++k)
      own[k] = s0 + k < steps ? *reinterpret_cast<const float2*>(state + (s0 + k) * stride) : make_float2(0.f, 0.f);
    if (fresh) {
      __syncthreads();
      decays[threadIdx.x] = decay;
      __syncthreads();
    }
#pragma unroll
    for (int k = 0; k < JOIN_AHEAD; ++k) {
      if (left == 0) {
        if (s0 + k <= steps) *reinterpret_cast<float2*>(state + (s0 + k) * stride) = S;
        left = s0 + k == 0 ? after_first : m;
      }
      --left;
      const float w = decays[(s0 + k) % JOIN_THREADS];
      S.x = S.x * w + own[k].x;
      S.y = S.y * w + own[k].y;
    }
  }
}

// Blocks an SM holds, which their registers are cut to. One number for both types:
// bf16's, whose head_dim 32 and 64 passes have next to no spills at it. fp32 spills
// up to 72 bytes; one block less, without spills, measured 287 us instead of 272
// (forward, 8 x 4096 rows of 8 heads of 64), 271 instead of 251 (backward, 32 x
// 1024 of 8 heads of 32), but 87 instead of 103 for the forward of the latter.
template <typename T, int HD, bool BACK>
__host__ __device__ constexpr int pass_blocks() { return HD < 64 ? (BACK ? 2 : 3) : BACK ? 1 : 2; }

// State accumulators of a warp as the operand planes of the next block
template <int HD, int NT>
__device__ __forceinline__ void put_state(uint32_t dst, const float (*acc)[4], int warp, int lane) {
  using P = StatePart<HD>;
#pragma unroll
  for (int g = 0; g < P::NG; ++g) {
    uint32_t t[4][NT];
#pragma unroll
    for (int r = 0; r < 4; ++r) terms2<NT>(acc[2 * g + (r >> 1)][(r & 1) * 2], acc[2 * g + (r >> 1)][(r & 1) * 2 + 1], t[r]);
#pragma unroll
    for (int k = 0; k < NT; ++k)
      stsm4<HD>(dst + k * HD * HD * 2, P::m(warp) * 16, (P::g(warp) * P::NG + g) * 2, lane,
                {t[0][k], t[1][k], t[2][k], t[3][k]});
  }
}

// A warp's 16 rows of accumulators to rows of `out`: bf16 through the warp's
// own rows of a tile that no other warp reads, to 16-byte stores; fp32 directly.
template <typename T, int HD>
__device__ __forceinline__ void store_rows(T* out, int d, uint32_t tile, const float (*o)[4], int rows, int warp,
                                           int lane) {
  using L = Tile<HD>;
  if constexpr (sizeof(T) == 2) {
    __syncwarp();
#pragma unroll
    for (int g = 0; g < HD / 16; ++g)
      stsm4<HD>(tile, warp * 16, g * 2, lane,
                {pack_bf16x2(o[2 * g][0], o[2 * g][1]), pack_bf16x2(o[2 * g][2], o[2 * g][3]),
                 pack_bf16x2(o[2 * g + 1][0], o[2 * g + 1][1]), pack_bf16x2(o[2 * g + 1][2], o[2 * g + 1][3])});
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 16 * L::PIECES; i += 32) {
      const int r = warp * 16 + (i + lane) / L::PIECES, p = lane % L::PIECES;
      uint32_t x[4];
      asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3])
                   : "r"(tile + L::at(r, p)) : "memory");
      if (r < rows) *reinterpret_cast<uint4*>(out + (size_t)r * d + p * 8) = make_uint4(x[0], x[1], x[2], x[3]);
    }
  } else {
    const int i0 = warp * 16 + (lane >> 2);
#pragma unroll
    for (int n = 0; n < HD / 8; ++n) {
      const int col = n * 8 + (lane & 3) * 2;
      if (i0 < rows) store2(out + (size_t)i0 * d + col, o[n][0], o[n][1]);
      if (i0 + 8 < rows) store2(out + (size_t)(i0 + 8) * d + col, o[n][2], o[n][3]);
    }
  }
}

// ---------------------------------------------------------------- the pass, forward and backward
//
// Block: one segment and head, its 64-row blocks in order (BACK: from the last
// one), four warps for the state and four for each output, 16 rows a warp. The
// state's warps work out the next block's state, operand and decays while the
// output's warps use this block's, and the tiles after it are on their way.
// Barriers of three stages keep them apart; no warp waits for another's rows.
// (With operands of one term, all of it in the same four warps measured 57 us at
// 2 x 16384 rows of 8 heads of 64, one latency after the other, and 40 so.) Now 53
// us: the tensor pipe is busy 48 % of the time, shared memory's wavefronts 52 % and
// the issue slots 45 %, HBM 2.1 TB/s: the mix of products, fragment loads, weights
// and roundings bounds it, no one of them alone.
//
// Forward, and for dq with dO, V, K in the places of Q, K, V:
//   O = (D * (Q K^T)) V + diag(exp(g (n_i - n_0))) Q S,  n_0 the index before the block
// Backward, with G the sum of exp(g (n_i - n)) q_i dO_i^T over the rows i after
// a block, n the block's last index and w_j = exp(g (n - n_j)):
//   dV = (D * (Q K^T))^T dO + diag(w) K G,   dK = (D * (dO V^T))^T Q + diag(w) V G^T
// Each is a product of own rows (operand A) with the block's rows before (after)
// them, weighted, times those rows' values, plus the own rows times the state.

template <typename T, int HD, bool BACK>
struct PassShape {
  static constexpr int NT = Terms<T>::N, TILES = BACK ? 4 : 3, WARPS = BACK ? 12 : 8, THREADS = WARPS * 32;
  static constexpr int STAGES = NT == 1 ? 3 : 1;  // tiles in flight; fp32 splits its tiles on the way in
  static constexpr int STATES = NT == 1 ? 2 : 1;  // operand planes of the state: the step's and the next one's
};
template <typename T, int HD, bool BACK>
__host__ __device__ constexpr int pass_smem() {
  using Q = PassShape<T, HD, BACK>;
  return Q::STAGES * Q::TILES * Q::NT * Tile<HD>::BYTES + Q::STATES * Terms<T>::MID * HD * HD * 2;
}

// Of a block's rows: exponents from the row before the block; the decay between
// a row and the end (BACK: start) of its 16; the row's weight in the state, from
// it to the block's end (BACK: from the row before the block to it).
struct BlockDecays {
  float2 e[3][BLK];
  float w[3][BLK], u[3][BLK];
  bool quotient[3][BLK / 16];  // the decays between the rows of a 16 are quotients of their w
};

// 16 own rows against the block's rows before (BACK: after) them and the state.
// Fragments are read a product ahead: a warp's ldmatrix and its mma would
// otherwise wait for one another in turn.
template <typename T, int HD, bool BACK, bool STATE_T>
__device__ __forceinline__ void block_output(float (&o)[HD / 8][4], const Frag<HD>& f, uint32_t ta, uint32_t tb,
                                             uint32_t tw, uint32_t state, bool has_state, const float2* e,
                                             const float* wt, const bool* quotient, int warp, int lane, int rows,
                                             float scale) {
  using L = Tile<HD>;
  constexpr bool FINE = Terms<T>::N == 3;
  constexpr int NT = Terms<T>::N, MT = Terms<T>::MID, ST = HD * HD * 2, N = HD / 16, QN = NT == 1 ? N : 1;
  const int i0 = warp * 16 + (lane >> 2);
  const float2 ei0 = e[i0], ei1 = e[i0 + 8];
  uint32_t qf[QN][NT][4];  // bf16 keeps its own rows' fragments, fp32 reads them again
  uint32_t kf[QN][NT][4];  // the score operand's of 16 rows
  uint32_t vb[QN][NT][4];  // the value operand's of 16 rows
  auto read_own = [&](int kk) {
#pragma unroll
    for (int t = 0; t < NT; ++t) f.a(qf[kk % QN][t], ta + t * L::BYTES, warp * 16, kk);
  };
  auto read_keys = [&](int kb, int kk) {
#pragma unroll
    for (int t = 0; t < NT; ++t) f.b(kf[kk % QN][t], tb + t * L::BYTES, kb * 16, kk);
  };
  auto read_values = [&](int kb, int g) {
#pragma unroll
    for (int t = 0; t < NT; ++t) f.bt(vb[g % QN][t], tw + t * L::BYTES, kb * 16, g);
  };
  auto read_state = [&](uint32_t (&r)[4], int kk, int g, int t) {
    if (STATE_T) f.b(r, state + t * ST, g * 16, kk);
    else f.bt(r, state + t * ST, kk * 16, g);
  };
  if (NT == 1)
#pragma unroll
    for (int kk = 0; kk < N; ++kk) read_own(kk);
  if (!has_state) {
#pragma unroll
    for (int n = 0; n < HD / 8; ++n) o[n][0] = o[n][1] = o[n][2] = o[n][3] = 0.f;
  } else if (NT == 1) {
    // the state's small terms first, then its large ones
#pragma unroll
    for (int g = 0; g < N; ++g) read_state(vb[g % QN][0], 0, g, MT - 1);
#pragma unroll
    for (int i = 0; i < MT * N; ++i) {
      const int kk = i % N, next = i + 1;
#pragma unroll
      for (int g = 0; g < N; ++g) {
        if (i == 0) {
          mma16816_new(o[2 * g], qf[kk % QN][0], vb[g % QN][0][0], vb[g % QN][0][1]);
          mma16816_new(o[2 * g + 1], qf[kk % QN][0], vb[g % QN][0][2], vb[g % QN][0][3]);
        } else {
          mma16816(o[2 * g], qf[kk % QN][0], vb[g % QN][0][0], vb[g % QN][0][1]);
          mma16816(o[2 * g + 1], qf[kk % QN][0], vb[g % QN][0][2], vb[g % QN][0][3]);
        }
        if (next < MT * N) read_state(vb[g % QN][0], next % N, g, MT - 1 - next / N);
      }
    }
  } else {
#pragma unroll
    for (int kk = 0; kk < N; ++kk) {
      read_own(kk);
#pragma unroll
      for (int g = 0; g < N; ++g) {
#pragma unroll
        for (int t = 0; t < NT; ++t) read_state(vb[0][t], kk, g, t);
        if (kk == 0) mma_terms<NT, true>(o[2 * g], o[2 * g + 1], qf[0], vb[0]);
        else mma_terms<NT>(o[2 * g], o[2 * g + 1], qf[0], vb[0]);
      }
    }
  }
  if (NT == 1)
#pragma unroll
    for (int kk = 0; kk < N; ++kk) {
      read_keys(warp, kk);
      read_values(warp, kk);
    }
  if (has_state) {
    const float f0 = (BACK ? decay_between<FINE>(e[BLK - 1], ei0) : decay_exp2<FINE>(ei0.x, ei0.y)) * scale;
    const float f1 = (BACK ? decay_between<FINE>(e[BLK - 1], ei1) : decay_exp2<FINE>(ei1.x, ei1.y)) * scale;
#pragma unroll
    for (int n = 0; n < HD / 8; ++n) {
      o[n][0] *= f0; o[n][1] *= f0; o[n][2] *= f1; o[n][3] *= f1;
    }
  }
  auto scores = [&](float (&s)[2][4], int kb) {
#pragma unroll
    for (int kk = 0; kk < N; ++kk) {
      if (NT > 1) {
        read_own(kk);
        read_keys(kb, kk);
      }
      if (kk == 0) mma_terms<NT, true>(s[0], s[1], qf[kk % QN], kf[kk % QN]);
      else mma_terms<NT>(s[0], s[1], qf[kk % QN], kf[kk % QN]);
    }
  };
  auto values = [&](const float (&s)[2][4], int kb) {
    uint32_t pa[MT][4];
#pragma unroll
    for (int r = 0; r < 4; ++r) {  // the accumulators are the next product's A fragment
      uint32_t t[MT];
      terms2<MT>(s[r >> 1][(r & 1) * 2], s[r >> 1][(r & 1) * 2 + 1], t);
#pragma unroll
      for (int k = 0; k < MT; ++k) pa[k][r] = t[k];
    }
    if (NT == 1) {
#pragma unroll
      for (int t = MT - 1; t >= 0; --t)
#pragma unroll
        for (int g = 0; g < N; ++g) {
          mma16816(o[2 * g], pa[t], vb[g % QN][0][0], vb[g % QN][0][1]);
          mma16816(o[2 * g + 1], pa[t], vb[g % QN][0][2], vb[g % QN][0][3]);
        }
    } else {
#pragma unroll
      for (int g = 0; g < N; ++g) {
        read_values(kb, g);
        mma_terms<NT>(o[2 * g], o[2 * g + 1], pa, vb[0]);
      }
    }
  };
  // the 16 x 16 blocks, the diagonal one first; then wholly on one side
  const int first = BACK ? warp + 1 : 0, end = BACK ? (rows + 15) / 16 : warp;
  // rows i0, i0 + 8; columns j, j + 1, j + 8, j + 9 of a 16 x 16 block
  {
    const int j = warp * 16 + (lane & 3) * 2;
    float s[2][4];
    scores(s, warp);
    if (NT == 1 && first < end)
#pragma unroll
      for (int kk = 0; kk < N; ++kk) read_keys(first, kk);
    auto in = [&](int own, int other) { return BACK ? other >= own : other <= own; };
    // Within the 16 rows D is the quotient of the decays to (BACK: from) their end
    if (quotient[warp]) {
      const float x0 = scale / wt[i0], x1 = scale / wt[i0 + 8];
      const float2 w0 = *reinterpret_cast<const float2*>(&wt[j]), w1 = *reinterpret_cast<const float2*>(&wt[j + 8]);
      s[0][0] *= x0 * w0.x; s[0][1] *= x0 * w0.y; s[0][2] *= x1 * w0.x; s[0][3] *= x1 * w0.y;
      s[1][0] *= x0 * w1.x; s[1][1] *= x0 * w1.y; s[1][2] *= x1 * w1.x; s[1][3] *= x1 * w1.y;
    } else {
#pragma unroll
      for (int n = 0; n < 2; ++n) {
        const float2 e0 = e[j + 8 * n], e1 = e[j + 8 * n + 1];
        auto d = [&](float2 own, float2 other) {
          return (BACK ? decay_between<FINE>(other, own) : decay_between<FINE>(own, other)) * scale;
        };
        s[n][0] *= d(ei0, e0); s[n][1] *= d(ei0, e1); s[n][2] *= d(ei1, e0); s[n][3] *= d(ei1, e1);
      }
    }
#pragma unroll
    for (int n = 0; n < 2; ++n) {
      const int jj = j + 8 * n;
      if (!in(i0, jj)) s[n][0] = 0.f;
      if (!in(i0, jj + 1)) s[n][1] = 0.f;
      if (!in(i0 + 8, jj)) s[n][2] = 0.f;
      if (!in(i0 + 8, jj + 1)) s[n][3] = 0.f;
    }
    values(s, warp);
  }
  // On one side D is the decay from the earlier row to the end of its 16, on to
  // the start of the later 16 and to the later row, each factor at most 1.
  const float2 near = e[BACK ? warp * 16 + 15 : warp * 16];  // the end of the own 16 rows nearest the others
  const float v0 = (BACK ? decay_between<FINE>(near, ei0) : decay_between<FINE>(ei0, near)) * scale;
  const float v1 = (BACK ? decay_between<FINE>(near, ei1) : decay_between<FINE>(ei1, near)) * scale;
#pragma unroll 1
  for (int kb = first; kb < end; ++kb) {
    if (NT == 1)
#pragma unroll
      for (int g = 0; g < N; ++g) read_values(kb, g);
    const int j = kb * 16 + (lane & 3) * 2;
    const float2 far = e[BACK ? kb * 16 : kb * 16 + 15];
    const float between = BACK ? decay_between<FINE>(far, near) : decay_between<FINE>(near, far);
    const float2 w0 = *reinterpret_cast<const float2*>(&wt[j]), w1 = *reinterpret_cast<const float2*>(&wt[j + 8]);
    const float x0 = v0 * between, x1 = v1 * between;
    float s[2][4];
    scores(s, kb);
    if (NT == 1 && kb + 1 < end)
#pragma unroll
      for (int kk = 0; kk < N; ++kk) read_keys(kb + 1, kk);
    s[0][0] *= x0 * w0.x; s[0][1] *= x0 * w0.y; s[0][2] *= x1 * w0.x; s[0][3] *= x1 * w0.y;
    s[1][0] *= x0 * w1.x; s[1][1] *= x0 * w1.y; s[1][2] *= x1 * w1.x; s[1][3] *= x1 * w1.y;
    values(s, kb);
  }
}

// Barrier of the whole block, reached from either role's loop.
template <int THREADS>
__device__ __forceinline__ void block_sync() {
  asm volatile("bar.sync 1, %0;" ::"n"(THREADS) : "memory");
}

template <typename T, int HD, int KT, bool BACK>
__global__ void __launch_bounds__(PassShape<T, HD, BACK>::THREADS, pass_blocks<T, HD, BACK>())
    decay_pass_kernel(const __grid_constant__ TileMaps maps, const __grid_constant__ DecayArgs a, const T* p0, const T* p1, const T* p2,
                      const T* p3, T* out0, T* out1) {
  using Q = PassShape<T, HD, BACK>;
  using L = Tile<HD>;
  using P = StatePart<HD>;
  constexpr int NT = Q::NT, PLANE = NT * L::BYTES, STAGE = Q::TILES * PLANE, STAGES = Q::STAGES;
  constexpr int MT = Terms<T>::MID, SPLANE = MT * HD * HD * 2, DECS = NT == 1 ? STAGES : 2;
  constexpr int OUT = BACK ? 8 : 4;  // warps OUT .. OUT + 3 have the state
  constexpr int LOADER = (OUT + 3) * 32;
  extern __shared__ __align__(1024) char smem[];
  __shared__ BlockDecays dec;
  // of a step's stage: its tiles are there; its state and decays are there; every warp is done with all of it
  __shared__ uint64_t full[STAGES], ready[STAGES], done[STAGES];
  __shared__ int abort_flag;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, d = a.d;
  if (tid == 0) {
    abort_flag = 0;
    for (int i = 0; i < STAGES; ++i) {
      sm100::mbar_init(&full[i], 1);
      sm100::mbar_init(&ready[i], 4);
      sm100::mbar_init(&done[i], Q::WARPS);
    }
    sm100::fence_mbar_init();
    if (NT == 1)
      for (int i = 0; i < Q::TILES; ++i) sm100::prefetch_tmap(&maps.m[i]);
  }
  __syncthreads();
  pdl_wait();
  pdl_release();
  const int H = a.h.n_heads, h = blockIdx.x % H;
  const DecayItem it = item_at(a, blockIdx.x / H);
  const uint32_t base = sm100::smem_u32(smem), sbase = base + STAGES * STAGE;
  const size_t off = (size_t)it.row0 * d + h * HD;
  const int blocks = (it.rows + BLK - 1) / BLK;
  auto block_of = [&](int s) { return BACK ? blocks - 1 - s : s; };  // the block of step s
  int issued = 0;
  auto stopped = [&] { return *reinterpret_cast<volatile int*>(&abort_flag) != 0; };
  auto load = [&](int s) {
    const int c = block_of(s);
    const uint32_t buf = base + (s % STAGES) * STAGE;
    if constexpr (NT == 1) {
      if (tid == LOADER && !stopped()) {
        tma_tiles<HD, Q::TILES>(buf, maps, h * HD, it.row0 + c * BLK, &full[s % STAGES]);
        issued = s + 1;
      }
    } else {
      const size_t at = off + (size_t)c * BLK * d;
      const int n = it.rows - c * BLK;
      split_tile<HD, Q::THREADS>(buf, p0 + at, d, n);
      split_tile<HD, Q::THREADS>(buf + PLANE, p1 + at, d, n);
      split_tile<HD, Q::THREADS>(buf + 2 * PLANE, p2 + at, d, n);
      if (BACK) split_tile<HD, Q::THREADS>(buf + 3 * PLANE, p3 + at, d, n);
    }
  };
  if (STAGES > 1)
    for (int s = 0; s < STAGES - 1 && s < blocks; ++s) load(s);
  const DecayRec& rec = it.rec;
  const bool last = it.seg + 1 == it.nseg, keep = !BACK && last && rec.slot >= 0;
  // a state before (BACK: after) the segment: the cached one, or the joined one
  const bool starts = BACK ? !last : it.nseg > 1 || (rec.slot >= 0 && rec.len0 > 0);
  auto wait = [&](uint64_t* bars, int s) {
    wait_phase(&bars[s % STAGES], (s / STAGES) & 1, a.err, &abort_flag);
  };
  auto arrive = [&](uint64_t* bars, int s) {  // of the whole warp
    __syncwarp();
    if (lane == 0) sm100::mbar_arrive(&bars[s % STAGES]);
  };
  // bf16: the step's tiles and state are there. fp32, whose tiles and state have
  // one buffer: every warp is done with the step before, the tiles are loaded.
  auto begin = [&](int s) {
    const int rows = it.rows - block_of(s) * BLK;
    if (NT == 1) {
      wait(full, s);
      wait(ready, s);
      if (rows < BLK) {  // the operands that other rows' products read
        const uint32_t t0 = base + (s % STAGES) * STAGE;
        block_sync<Q::THREADS>();
        clear_rows<HD, Q::THREADS>(t0 + (BACK ? 0 : PLANE), rows);
        clear_rows<HD, Q::THREADS>(t0 + (BACK ? PLANE : 2 * PLANE), rows);
        if (BACK) sm100::fence_async_smem();  // every warp's zeros lie where TMA writes three steps on
        block_sync<Q::THREADS>();
      }
    } else {
      block_sync<Q::THREADS>();
      load(s);
      block_sync<Q::THREADS>();
    }
  };
  auto finish = [&](int s) {
    if (NT == 1) {
      if (warp < OUT) sm100::fence_async_smem();  // outputs went through the tiles that TMA fills next
      arrive(done, s);
    } else if (s + 1 < blocks) {
      block_sync<Q::THREADS>();
    }
  };

  // The roles run loops of their own, so that neither holds the other's registers.
  if (warp >= OUT) {
    const int sw = warp - OUT, st = tid - OUT * 32;
    // Threads 0 .. 63 keep the rows' indexes: timestamps are read a step before they are needed.
    const Index ix = head_index(a, rec, h);
    const double decay2 = a.h.decay2[h];
    auto row_of = [&](int c, int i) { return it.row0 + min(c * BLK + i, it.rows - 1); };
    // The index at the block's edge that the next step shares: the next block's
    // reference is this block's end (BACK: its end is this one's reference).
    auto edge_row = [&](int c) { return BACK ? it.row0 + c * BLK - 1 : row_of(c, BLK - 1); };
    auto time_of = [&](int row) { return row >= rec.row0 ? a.ts[row] : rec.tprev; };
    long long t_row = 0, t_edge = 0, t_before = 0, n_shared = 0;
    const bool check = !BACK && h == 0 && a.ts != nullptr;
    auto read_times = [&](int s) {
      if (s >= blocks || st >= BLK || !a.ts) return;
      const int c = block_of(s), row = row_of(c, st);
      t_row = a.ts[row];
      t_edge = time_of(edge_row(c));
      if (check) t_before = time_of(row - 1);
    };
    if (st < BLK && ix.tau > 0) {
      const int c = block_of(0);
      n_shared = ix.of_time(time_of(BACK ? row_of(c, BLK - 1) : it.row0 + c * BLK - 1));
    }
    auto put_decays = [&](int s) {
      if (s >= blocks || st >= BLK) return;
      if (check && t_row < t_before) set_error(a.err, REST_ERR_UNSORTED_TIME);
      const int c = block_of(s), ref = it.row0 + c * BLK - 1;
      long long n, n_end;
      if (ix.tau > 0) {
        const long long n_edge = ix.of_time(t_edge), n_ref = BACK ? n_edge : n_shared;
        n = ix.of_time(t_row) - n_ref;
        n_end = (BACK ? n_shared : n_edge) - n_ref;
        n_shared = n_edge;
      } else {
        // a position head's whole blocks are alike: their stage has this already
        if (s >= DECS && !(BACK && s == DECS) && it.rows - c * BLK >= BLK) return;
        n = row_of(c, st) - ref;
        n_end = row_of(c, BLK - 1) - ref;
      }
      const float2 e = exponent(decay2, n);
      dec.e[s % DECS][st] = e;
      const int end = BACK ? lane & 16 : lane | 15;
      const float2 x = make_float2(__shfl_sync(0xffffffffu, e.x, end), __shfl_sync(0xffffffffu, e.y, end));
      const float w = BACK ? decay_between<NT == 3>(e, x) : decay_between<NT == 3>(x, e);
      dec.w[s % DECS][st] = w;
      // while they are far from the smallest number and no timestamp decreases between the rows, which
      // their clamped decays would not show
      const long long before = __shfl_up_sync(0xffffffffu, n, 1);
      const uint32_t good = __ballot_sync(0xffffffffu, w >= 0x1p-60f && ((lane & 15) == 0 || n >= before));
      if ((lane & 15) == 0) dec.quotient[s % DECS][st >> 4] = ((good >> lane) & 0xffffu) == 0xffffu;
      dec.u[s % DECS][st] = BACK ? decay_exp2<KT == 3>(e.x, e.y) : decay_between<KT == 3>(exponent(decay2, n_end), e);
    };
    read_times(0);
    put_decays(0);
    read_times(1);

    float S[2 * P::NG][4] = {};
    const bool on = P::on(sw);
    const size_t part = (P::m(sw) * 16 + (lane >> 2)) * HD + P::g(sw) * P::NG * 16 + (lane & 3) * 2;
    if (starts && on) {
      const size_t joined = BACK ? (size_t)a.n_parts + it.part1 : it.part0;
      const float* src = (it.nseg > 1 ? a.part_state + (joined * H + h) * HD * HD
                                      : a.state + ((size_t)rec.slot * H + h) * HD * HD) + part;
#pragma unroll
      for (int n = 0; n < 2 * P::NG; ++n) {
        const float2 x = *reinterpret_cast<const float2*>(src + n * 8);
        const float2 y = *reinterpret_cast<const float2*>(src + 8 * HD + n * 8);
        S[n][0] = x.x; S[n][1] = x.y; S[n][2] = y.x; S[n][3] = y.y;
      }
      put_state<HD, MT>(sbase, S, sw, lane);
    }
    if (NT == 1) arrive(ready, 0);
    // x by its columns that are this warp's rows of the state, y by the state's columns
    const uint32_t ox = L::at((lane & 7) + ((lane >> 4) << 3), P::m(sw) * 2 + ((lane >> 3) & 1));
    uint32_t oy[P::NG];
#pragma unroll
    for (int g = 0; g < P::NG; ++g) oy[g] = L::at(lane & 15, (P::g(sw) * P::NG + g) * 2 + (lane >> 4));
    for (int s = 0; s < blocks; ++s) {
      begin(s);
      const uint32_t t0 = base + (s % STAGES) * STAGE;
      if (NT == 1 && warp == LOADER / 32 && s + STAGES - 1 < blocks) {
        if (s > 0) wait(done, s - 1);
        load(s + STAGES - 1);
      }
      const bool more = s + 1 < blocks;
      if ((more || keep) && on) {  // a state that nothing reads is not computed
        const float2 end = dec.e[s % DECS][BLK - 1];  // rows past the last repeat it
        const uint32_t tx = BACK ? t0 : t0 + PLANE, ty = tx + PLANE;
        add_products<T, HD, KT>(S, decay_exp2<KT == 3>(end.x, end.y), tx, ty, ox, oy, lane, dec.u[s % DECS]);
      }
      if (NT == 1) {
        if (more) {
          if (s > 0) wait(done, s - 1);  // the state's buffer of the step before, and the decays' of the one before that
          if (on) put_state<HD, MT>(sbase + ((s + 1) % Q::STATES) * SPLANE, S, sw, lane);
          put_decays(s + 1);
          arrive(ready, s + 1);
          read_times(s + 2);
        }
        finish(s);
      } else {
        put_decays(s + 1);
        read_times(s + 2);
        finish(s);
        if (more && on) put_state<HD, MT>(sbase, S, sw, lane);
      }
    }
    if (STAGES > 1 && tid == LOADER && stopped()) drain<STAGES>(full, issued);
    if (keep && on) {
      float* dst = a.state + ((size_t)rec.slot * H + h) * HD * HD + part;
#pragma unroll
      for (int n = 0; n < 2 * P::NG; ++n) {
        store2(dst + n * 8, S[n][0], S[n][1]);
        store2(dst + 8 * HD + n * 8, S[n][2], S[n][3]);
      }
    }
    return;
  }

  const Frag<HD> f(lane);
  for (int s = 0; s < blocks; ++s) {
    // the 16 rows with the most others before them move on from warp to warp
    const int w = NT == 1 ? (warp + s + blockIdx.x) & 3 : warp & 3;
    begin(s);
    const int c = block_of(s), rows = min(BLK, it.rows - c * BLK);
    const uint32_t t0 = base + (s % STAGES) * STAGE, t1 = t0 + PLANE, t2 = t1 + PLANE, t3 = t2 + PLANE;
    const uint32_t ts = sbase + (s % Q::STATES) * SPLANE;
    const float2* e = dec.e[s % DECS];
    const float* wt = dec.w[s % DECS];
    const bool* quotient = dec.quotient[s % DECS];
    const bool has_state = starts || s > 0;
    if (w * 16 < rows) {
      float o[HD / 8][4];
      const size_t at = off + (size_t)c * BLK * d;
      if (!BACK) {
        block_output<T, HD, false, false>(o, f, t0, t1, t2, ts, has_state, e, wt, quotient, w, lane, rows, a.scale);
        store_rows<T, HD>(out0 + at, d, t0, o, rows, w, lane);
      } else if (warp < 4) {  // dV from K, Q, dO and G; the rows of K are no other warp's
        block_output<T, HD, true, false>(o, f, t2, t0, t1, ts, has_state, e, wt, quotient, w, lane, rows, a.scale);
        store_rows<T, HD>(out1 + at, d, t2, o, rows, w, lane);
      } else {                // dK from V, dO, Q and G^T
        block_output<T, HD, true, true>(o, f, t3, t1, t0, ts, has_state, e, wt, quotient, w, lane, rows, a.scale);
        store_rows<T, HD>(out0 + at, d, t3, o, rows, w, lane);
      }
    }
    finish(s);
  }
}

// ---------------------------------------------------------------- one token

constexpr int STEP_THREADS = 256, STEP_STAGES = 3;
constexpr int STEP_CHUNK = 4096;  // floats of a slot's state at a time: G = 4096 / hd^2 heads, 16 KB

// Cluster: one entry; block `rank` of it takes every cluster-size-th chunk of
// the slot's states. A chunk is copied to shared memory whole, updated there
// and copied back, the next ones on their way meanwhile: the state is read and
// written once and bounds the call. Thread (g, r, c) has rows r, r + HD / 4 ..
// of head g's state, columns 4 c .. 4 c + 3.
template <typename T, int HD>
__global__ void __launch_bounds__(STEP_THREADS, 4) decay_step_kernel(DecayHeadsArg hs, const T* __restrict__ q,
                                                                     const T* __restrict__ k,
                                                                     const T* __restrict__ v, const int64_t* ts,
                                                                     DecayState st, T* o, float scale,
                                                                     DecayWait waits, int32_t* err) {
  constexpr int G = STEP_CHUNK / (HD * HD), C = HD / 4, R = HD / 4, PER = STEP_THREADS / G;  // threads per head
  constexpr int LANES_R = 32 / C < R ? 32 / C : R;  // row groups of a head within a warp
  extern __shared__ __align__(128) float chunk[];   // [STEP_STAGES][STEP_CHUNK]
  __shared__ float part[STEP_THREADS / C][HD];
  __shared__ float keep[32];
  __shared__ uint64_t full[STEP_STAGES];
  __shared__ int abort_flag;
  const int tid = threadIdx.x;
  if (tid == 0) {
    abort_flag = 0;
    for (int i = 0; i < STEP_STAGES; ++i) sm100::mbar_init(&full[i], 1 + waits.missing);
    sm100::fence_mbar_init();
  }
  pdl_wait();
  pdl_release();
  uint32_t rank, size;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
  asm volatile("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(size));
  const int b = blockIdx.x / size, H = hs.n_heads, d = H * HD;
  const int slot = st.slots ? st.slots[b] : b;
  const bool in = slot >= 0 && slot < st.n_slots;
  const int chunks = (H + G - 1) / G, mine = ((int)rank < chunks && in) ? (chunks - (int)rank + (int)size - 1) / (int)size : 0;
  float* states = st.s + (size_t)(in ? slot : 0) * H * (HD * HD);
  auto head0 = [&](int i) { return ((int)rank + i * (int)size) * G; };  // first head of the block's chunk i
  auto bytes = [&](int i) { return (uint32_t)(min(G, H - head0(i)) * HD * HD * 4); };
  auto load = [&](int i) {
    uint64_t* bar = &full[i % STEP_STAGES];
    sm100::mbar_arrive_expect_tx(bar, bytes(i));
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                     sm100::smem_u32(chunk + (i % STEP_STAGES) * STEP_CHUNK)),
                 "l"(states + (size_t)head0(i) * (HD * HD)), "r"(bytes(i)), "r"(sm100::smem_u32(bar))
                 : "memory");
  };
  // read even before it is known whether the slot holds anything: what an empty slot has is not used
  int issued = min(mine, STEP_STAGES);
  if (tid == 0)
    for (int i = 0; i < issued; ++i) load(i);
  long long len = 0, t = 0, t_first = 0, t_last = 0;
  if (in) {
    len = st.len[slot];
    if (ts) {
      t = ts[b];
      t_first = st.t_first[slot];
      t_last = st.t_last[slot];
    }
  }
  if (len == 0) t_first = t_last = t;
  if (in && tid < H) {
    const long long tau = hs.tau[tid];
    long long n = 1;
    if (tau > 0) n = max(0LL, buckets(t - t_first, tau, hs.inv[tid]) - buckets(t_last - t_first, tau, hs.inv[tid]));
    keep[tid] = (float)exp2(hs.decay2[tid] * (double)n);
  }
  int bad = slot < -1 || slot >= st.n_slots;
  if (st.slots && in)  // an earlier entry with the same slot
    for (int i = tid; i < b; i += STEP_THREADS) bad |= st.slots[i] == slot;
  bad = __syncthreads_or(bad);
  // every block of the cluster has read the bookkeeping once all have arrived
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  auto stopped = [&] { return *reinterpret_cast<volatile int*>(&abort_flag) != 0; };
  const int g = tid / PER, r = tid % PER / C, c = tid % C;
  for (int i = 0; i < mine; ++i) {
    const int h0 = head0(i), h = h0 + g;
    const bool on = h < H;
    float vv[4] = {}, kk[4] = {}, qq[4] = {};
    if (on && !bad) {
      const size_t at = (size_t)b * d + h * HD;
      load4(v + at + 4 * c, vv);
#pragma unroll
      for (int y = 0; y < 4; ++y) {
        kk[y] = to_f(k[at + r + y * R]);
        qq[y] = to_f(q[at + r + y * R]);
      }
    }
    wait_phase(&full[i % STEP_STAGES], (i / STEP_STAGES) & 1, err, &abort_flag, waits.limit);
    if (bad) {  // nothing but the loads that are on their way
      if (i + 1 == min(mine, STEP_STAGES)) break;
      continue;
    }
    float* S = chunk + (i % STEP_STAGES) * STEP_CHUNK + g * (HD * HD) + 4 * c;
    float acc[4] = {};
    if (on) {
      const float f = keep[h];
#pragma unroll
      for (int y = 0; y < 4; ++y) {
        float x[4];
        load4(S + (r + y * R) * HD, x);
#pragma unroll
        for (int z = 0; z < 4; ++z) {
          x[z] = len > 0 ? x[z] * f + kk[y] * vv[z] : kk[y] * vv[z];
          acc[z] += qq[y] * x[z];
        }
        store4(S + (r + y * R) * HD, x);
      }
    }
    // sum over the rows: lanes of a warp, then warps
#pragma unroll
    for (int m = C; m < C * LANES_R; m <<= 1)
#pragma unroll
      for (int z = 0; z < 4; ++z) acc[z] += __shfl_xor_sync(0xffffffffu, acc[z], m);
    if (r % LANES_R == 0) store4(&part[tid / C][4 * c], acc);
    sm100::fence_async_smem();
    __syncthreads();
    // A wait ran out: what the chunk holds is not the state and stays here. All
    // threads see the same, since none waits again before the next barrier.
    if (stopped()) break;
    if (tid == 0) {
      asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(
                       states + (size_t)h0 * (HD * HD)),
                   "r"(sm100::smem_u32(chunk + (i % STEP_STAGES) * STEP_CHUNK)), "r"(bytes(i))
                   : "memory");
      sm100::bulk_commit();
      if (i >= 1 && i - 1 + STEP_STAGES < mine) {  // the chunk before has left its buffer
        sm100::bulk_wait_read<1>();
        load(i - 1 + STEP_STAGES);
        issued = i + STEP_STAGES;
      }
    }
    for (int y = tid; y < G * HD; y += STEP_THREADS) {
      const int gg = y / HD, col = y % HD;
      if (h0 + gg < H) {
        float sum = 0.f;
#pragma unroll
        for (int z = 0; z < R; z += LANES_R) sum += part[gg * R + z][col];
        o[(size_t)b * d + (h0 + gg) * HD + col] = from_f<T>(sum * scale);
      }
    }
    if (i + 1 < mine) __syncthreads();  // the sums are read
  }
  if (tid == 0) {
    if (stopped()) drain<STEP_STAGES>(full, issued, waits.limit);
    sm100::bulk_wait<0>();
  }
  __syncwarp();
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
  if (rank == 0 && tid == 0) {
    if (bad) set_error(err, REST_ERR_INVALID_ARG);
    if (in && !bad && !stopped()) {
      st.len[slot] = len + 1;
      if (ts) {
        if (t < t_last) set_error(err, REST_ERR_UNSORTED_TIME);
        if (len == 0) st.t_first[slot] = t;
        st.t_last[slot] = t;
      }
    }
  }
}

// More than 48 KB a block need the kernel's attribute. Every launch sets it, to
// one number a kernel, whatever the launch takes: calls from several threads
// cannot lower one another's, and a new context of the device has it too.
template <auto KERNEL, int BYTES>
cudaError_t allow_smem() {
  return cudaFuncSetAttribute(KERNEL, cudaFuncAttributeMaxDynamicSharedMemorySize, BYTES);
}

template <typename T, int HD>
cudaError_t step_hd(const DecayHeadsArg& hs, int n, const void* q, const void* k, const void* v, const int64_t* ts,
                    const DecayState& st, void* o, float scale, const DecayWait& waits, int32_t* err, cudaStream_t s) {
  // Blocks of an entry: as many as its chunks while they do not fill the GPU
  // (four blocks an SM).
  constexpr int G = STEP_CHUNK / (HD * HD), bytes = STEP_STAGES * STEP_CHUNK * 4;
  const int chunks = (hs.n_heads + G - 1) / G;
  int size = 1;
  while (size < 8 && size < chunks && (long long)n * size < 148 * 4) size *= 2;
  cudaError_t e = allow_smem<decay_step_kernel<T, HD>, bytes>();
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg;
  memset(&cfg, 0, sizeof(cfg));
  cfg.gridDim = dim3(n * size);
  cfg.blockDim = dim3(STEP_THREADS);
  cfg.dynamicSmemBytes = bytes;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = size;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl_enabled() ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, decay_step_kernel<T, HD>, hs, (const T*)q, (const T*)k, (const T*)v, ts, st, (T*)o,
                            scale, waits, err);
}

template <typename T, int HD>
constexpr int part_smem() { return part_stages<T>() * 2 * Terms<T>::N * Tile<HD>::BYTES; }
// Boxes of 64 rows and a head's columns over [rows, d] arrays (bf16 only; null arrays have none)
template <typename T, int HD>
bool tile_maps(TileMaps* maps, const DecayArgs& a, const void* p0, const void* p1, const void* p2, const void* p3) {
  memset(maps, 0, sizeof(*maps));
  if (sizeof(T) != 2) return true;
  const void* p[4] = {p0, p1, p2, p3};
  for (int i = 0; i < 4; ++i)
    if (p[i] && !make_tmap_bf16(&maps->m[i], p[i], a.rows, a.d, a.d, HD, BLK, HD * 2)) return false;
  return true;
}

// Fewer blocks than the SMs hold are spread evenly: the hardware puts a second
// and third on some SMs and leaves others empty (256 blocks of 32 x 1024 rows: 24
// SMs had three and 32 none). Shared memory that nothing uses keeps an SM to its share.
constexpr int SPREAD_MOST = 227 * 1024, SPREAD_KERNEL = 5 * 1024;  // static arrays and the system's 1 KB
constexpr int spread_even(int share) {  // share + 1 of these do not fit
  return SPREAD_MOST / (share + 1) + 1 - SPREAD_KERNEL + 4 * 1024;
}
int spread_smem(int bytes, long long blocks) {
  constexpr int SMS = 148;
  const int share = (int)std::min<long long>(32, (blocks + SMS - 1) / SMS), even = spread_even(share);
  return (blocks + SMS - 1) / SMS > 4 || (long long)(even + SPREAD_KERNEL) * share > SPREAD_MOST ? bytes
                                                                                                 : std::max(bytes, even);
}

template <typename T, int HD, int KT>
cudaError_t part_hd(bool back, const DecayArgs& a, const void* x0, const void* y0, const void* x1, const void* y1,
                    cudaStream_t s) {
  const dim3 grid(a.n_parts * a.h.n_heads, back ? 2 : 1);
  const int bytes = spread_smem(part_smem<T, HD>(), (long long)grid.x * grid.y);
  TileMaps m0, m1;
  if (!tile_maps<T, HD>(&m0, a, x0, y0, nullptr, nullptr) || !tile_maps<T, HD>(&m1, a, x1, y1, nullptr, nullptr))
    return cudaErrorInvalidValue;
  cudaError_t e = allow_smem<decay_part_kernel<T, HD, KT>, std::max(part_smem<T, HD>(), spread_even(1))>();
  if (e != cudaSuccess) return e;
  return launch_k(decay_part_kernel<T, HD, KT>, grid, dim3(CH_THREADS), bytes, s, m0, m1, a, (const T*)x0,
                  (const T*)y0, (const T*)x1, (const T*)y1);
}

template <typename T, int HD, int KT, bool BACK>
cudaError_t pass_hd(int n_items, const DecayArgs& a, const void* p0, const void* p1, const void* p2, const void* p3,
                    void* out0, void* out1, cudaStream_t s) {
  const dim3 grid(n_items * a.h.n_heads);
  const int bytes = spread_smem(pass_smem<T, HD, BACK>(), grid.x);
  TileMaps m;
  if (!tile_maps<T, HD>(&m, a, p0, p1, p2, p3)) return cudaErrorInvalidValue;
  cudaError_t e = allow_smem<decay_pass_kernel<T, HD, KT, BACK>, std::max(pass_smem<T, HD, BACK>(), spread_even(1))>();
  if (e != cudaSuccess) return e;
  return launch_k(decay_pass_kernel<T, HD, KT, BACK>, grid, dim3(PassShape<T, HD, BACK>::THREADS), bytes, s, m, a,
                  (const T*)p0, (const T*)p1, (const T*)p2, (const T*)p3, (T*)out0, (T*)out1);
}

template <int HD>
cudaError_t join_hd(bool back, int n_users, const DecayArgs& a, cudaStream_t s) {
  return launch_k(decay_join_kernel<HD>, dim3(n_users * a.h.n_heads, HD * HD / (JOIN_THREADS * JOIN_VALUES), back ? 2 : 1),
                  dim3(JOIN_THREADS), 0, s, a);
}

// Terms of the decayed K (KT): three where the state is an output, else as many as Terms::MID
template <int HD>
cudaError_t part_any(bool bf, bool back, bool exact, const DecayArgs& a, const void* x0, const void* y0,
                     const void* x1, const void* y1, cudaStream_t s) {
  if (!bf) return part_hd<float, HD, 3>(back, a, x0, y0, x1, y1, s);
  return exact ? part_hd<bf16, HD, 3>(back, a, x0, y0, x1, y1, s) : part_hd<bf16, HD, 2>(back, a, x0, y0, x1, y1, s);
}
template <int HD>
cudaError_t pass_any(bool bf, bool exact, int n, const DecayArgs& a, const void* q, const void* k, const void* v,
                     void* o, cudaStream_t s) {
  if (!bf) return pass_hd<float, HD, 3, false>(n, a, q, k, v, nullptr, o, nullptr, s);
  return exact ? pass_hd<bf16, HD, 3, false>(n, a, q, k, v, nullptr, o, nullptr, s)
               : pass_hd<bf16, HD, 2, false>(n, a, q, k, v, nullptr, o, nullptr, s);
}
template <int HD>
cudaError_t dkdv_any(bool bf, int n, const DecayArgs& a, const void* q, const void* k, const void* v, const void* g,
                     void* dk, void* dv, cudaStream_t s) {
  return bf ? pass_hd<bf16, HD, 2, true>(n, a, q, g, k, v, dk, dv, s)
            : pass_hd<float, HD, 3, true>(n, a, q, g, k, v, dk, dv, s);
}

}  // namespace

cudaError_t launch_decay_prep(const DecayUsers& users, const int64_t* ts, const DecayState& st, const DecayArgs& a,
                              DecayItem* items, DecayPart* parts, DecayUser* heads, cudaStream_t s) {
  return launch_k(decay_prep_kernel, dim3(users.n), dim3(128), 0, s, users, ts, st, a.cut, items, parts, heads, a.err);
}

cudaError_t launch_decay_parts(bool bf, int hd, bool back, bool exact, const DecayArgs& a, const void* x0,
                               const void* y0, const void* x1, const void* y1, cudaStream_t s) {
  if (hd == 16) return part_any<16>(bf, back, exact, a, x0, y0, x1, y1, s);
  if (hd == 32) return part_any<32>(bf, back, exact, a, x0, y0, x1, y1, s);
  return part_any<64>(bf, back, exact, a, x0, y0, x1, y1, s);
}

cudaError_t launch_decay_join(int hd, bool back, int n_users, const DecayArgs& a, cudaStream_t s) {
  if (hd == 16) return join_hd<16>(back, n_users, a, s);
  if (hd == 32) return join_hd<32>(back, n_users, a, s);
  return join_hd<64>(back, n_users, a, s);
}

cudaError_t launch_decay_pass(bool bf, int hd, bool exact, int n_items, const DecayArgs& a, const void* q,
                              const void* k, const void* v, void* o, cudaStream_t s) {
  if (hd == 16) return pass_any<16>(bf, exact, n_items, a, q, k, v, o, s);
  if (hd == 32) return pass_any<32>(bf, exact, n_items, a, q, k, v, o, s);
  return pass_any<64>(bf, exact, n_items, a, q, k, v, o, s);
}

cudaError_t launch_decay_dkdv(bool bf, int hd, int n_items, const DecayArgs& a, const void* q, const void* k,
                              const void* v, const void* d_o, void* dk, void* dv, cudaStream_t s) {
  if (hd == 16) return dkdv_any<16>(bf, n_items, a, q, k, v, d_o, dk, dv, s);
  if (hd == 32) return dkdv_any<32>(bf, n_items, a, q, k, v, d_o, dk, dv, s);
  return dkdv_any<64>(bf, n_items, a, q, k, v, d_o, dk, dv, s);
}

cudaError_t launch_decay_step(bool bf, int hd, const DecayHeadsArg& hs, int n, const void* q, const void* k,
                              const void* v, const int64_t* ts, const DecayState& st, void* o, float scale,
                              const DecayWait& waits, int32_t* err, cudaStream_t s) {
  if (bf) {
    if (hd == 16) return step_hd<bf16, 16>(hs, n, q, k, v, ts, st, o, scale, waits, err, s);
    if (hd == 32) return step_hd<bf16, 32>(hs, n, q, k, v, ts, st, o, scale, waits, err, s);
    return step_hd<bf16, 64>(hs, n, q, k, v, ts, st, o, scale, waits, err, s);
  }
  if (hd == 16) return step_hd<float, 16>(hs, n, q, k, v, ts, st, o, scale, waits, err, s);
  if (hd == 32) return step_hd<float, 32>(hs, n, q, k, v, ts, st, o, scale, waits, err, s);
  return step_hd<float, 64>(hs, n, q, k, v, ts, st, o, scale, waits, err, s);
}

}  // namespace rest
