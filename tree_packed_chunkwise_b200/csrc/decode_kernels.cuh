// Kernels of token-by-token generation: the recurrent KDA step on a cache of states, the append to
// the paged cache of latents, and the rotation of the absorbed queries.
#pragma once
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <cstdint>

#include "common.cuh"
#include "tc.cuh"

namespace tpc {

constexpr int kLatDim = 512, kLatRope = 64, kLatHead = 128, kLatWidth = kLatDim + kLatRope, kLatQK = kLatHead + kLatRope;

// device view of tpc_rows
struct DecodeRows {
  int n_rows, n_seqs;
  const int32_t* row_start;  // NULL: row b is sequence b's
  const int32_t* kv_len;
};

// device view of tpc_latent_cache
struct LatentCache {
  __nv_bfloat16* data;
  int n_pages, page_size;
  const int32_t* table;
  int max_pages;
};

// Sequence that owns row t, by the whole warp: the number of sequences whose rows end at or before t,
// found by 33-way search (one probe per lane and level, so three dependent loads reach 32,768
// sequences).  In [0, n_seqs] whatever row_start holds, and the range shrinks on every level.
__device__ __forceinline__ int seq_of_row(const int32_t* row_start, int n_seqs, int t) {
  const int lane = threadIdx.x & 31;
  int lo = 0, hi = n_seqs;
  while (lo < hi) {
    const int step = (hi - lo + 31) / 32, j = lo + (lane + 1) * step - 1;
    const bool ended = j < hi && row_start[j + 1] <= t;
    lo += __popc(__ballot_sync(0xffffffffu, ended)) * step;
    hi = min(hi, lo + step - 1);
  }
  return lo;
}

struct RowAt {
  int seq;      // -1: the row belongs to no sequence
  int64_t pos;  // may be negative
};

__device__ __forceinline__ RowAt row_at(const DecodeRows& r, int t) {
  if (!r.row_start) return {t, (int64_t)r.kv_len[t] - 1};
  const int b = seq_of_row(r.row_start, r.n_seqs, t);
  if (b >= r.n_seqs || t < r.row_start[b]) return {-1, 0};
  return {b, (int64_t)r.kv_len[b] - r.row_start[b + 1] + t};
}

// cos and sin of pos * 10000^(-2 i / 64).  The angle is taken in turns in double precision and reduced
// there (2^31 positions: error below 1e-6 of a turn), so that far positions keep fp32 accuracy.
__device__ __forceinline__ void rope_angle(int64_t pos, int i, float* cs, float* sn) {
  const double turns = (double)pos * (exp2(-(double)i * (13.287712379549449 / (kLatRope / 2))) * 0.15915494309189535);
  sincospif(2.f * (float)(turns - rint(turns)), sn, cs);
}

// ------------------------------------------------------------------------------------ KDA step
struct StepArgs {
  const void *q, *k, *v, *g, *beta;
  float* state;
  const int32_t *src, *dst;  // dst NULL: in place
  void* o;
  int n_slots, H;
  DecodeRows rows;
  int* status;
};

// N consecutive elements (N * sizeof(T) a power of two up to 32 bytes, aligned to min(that, 16))
template <typename T, int N>
__device__ __forceinline__ void load_vec(const T* p, float (&x)[N]) {
  constexpr int B = N * (int)sizeof(T);
  if constexpr (B >= 16) {
    constexpr int V = 16 / sizeof(T);
#pragma unroll
    for (int j = 0; j < N / V; ++j) {
      const uint4 u = reinterpret_cast<const uint4*>(p)[j];
      const T* e = reinterpret_cast<const T*>(&u);
#pragma unroll
      for (int i = 0; i < V; ++i) x[j * V + i] = to_f(e[i]);
    }
  } else if constexpr (B == 8) {
    const uint2 u = *reinterpret_cast<const uint2*>(p);
    const T* e = reinterpret_cast<const T*>(&u);
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = to_f(e[i]);
  } else {
    static_assert(B == 4, "vector width");
    const uint32_t u = *reinterpret_cast<const uint32_t*>(p);
    const T* e = reinterpret_cast<const T*>(&u);
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = to_f(e[i]);
  }
}

template <typename T>
__device__ __forceinline__ void store4(T* p, const float (&x)[4]) {
  if constexpr (sizeof(T) == 4) {
    *reinterpret_cast<float4*>(p) = make_float4(x[0], x[1], x[2], x[3]);
  } else {
    __align__(8) T e[4] = {from_f<T>(x[0]), from_f<T>(x[1]), from_f<T>(x[2]), from_f<T>(x[3])};
    *reinterpret_cast<uint2*>(p) = *reinterpret_cast<const uint2*>(e);
  }
}

constexpr int kStepThreads = 128;

// The columns of S evolve independently: with Sd = Diag(e^g) S, u = Sd^T k and w = Sd^T q,
//   delta = beta (v - u),  S' = Sd + k delta^T,  o = S'^T q = w + (k . q) delta,
// so one pass over a column does everything: a state is read once and written once, and their bytes
// bound the step (4 flops a byte).
//
// In registers: a warp owns 256 / D groups of 4 columns, a lane 8 rows x 4 columns; sums over the rows are
// shuffles, and nothing is shared between warps (no barrier).  For small batches and runs of rows
// (launch and latency bound; 16 heads of one sequence 2.8 us against 3.4 us of the kernel below, runs of
// six rows 52 against 58 us) and for d < 128.
template <typename T, typename TO, int D>
__global__ void __launch_bounds__(kStepThreads, 6) kda_step_regs(StepArgs a) {
  constexpr int R = 8, CG = 256 / D, SL = D / (4 * CG);  // rows per lane, column groups, warps per head
  const int lane = threadIdx.x & 31, rg = lane / CG;
  const int64_t unit = (int64_t)blockIdx.x * (kStepThreads / 32) + (threadIdx.x >> 5);
  const int64_t bh = unit / SL;
  const int sl = (int)(unit % SL), h = (int)(bh % a.H);
  const int64_t b64 = bh / a.H;
  if (b64 >= a.rows.n_seqs) return;
  const int b = (int)b64;
  const int src = a.src[b], dst = a.dst ? a.dst[b] : src;
  const int t0 = a.rows.row_start ? a.rows.row_start[b] : b, t1 = a.rows.row_start ? a.rows.row_start[b + 1] : b + 1;
  if (src < 0) return;  // padding entry
  if (src >= a.n_slots || dst < 0 || dst >= a.n_slots || t0 < 0 || t1 < t0 || t1 > a.rows.n_rows) {
    if (lane == 0) set_status(a.status, kStatusCheck);
    return;
  }
  // one warp per sequence looks for another sequence that writes or reads the slot it writes
  if (a.status && h == 0 && sl == 0) {
    bool clash = false;
    for (int j = lane; j < a.rows.n_seqs; j += 32) {
      const int sj = a.src[j];
      if (j == b || sj < 0) continue;
      clash |= sj == dst || (a.dst && a.dst[j] == dst);
    }
    if (__any_sync(0xffffffffu, clash) && lane == 0) set_status(a.status, kStatusCheck);
  }
  const int r0 = rg * R, c0 = (sl * CG + lane % CG) * 4;
  const size_t at = (size_t)r0 * D + c0;
  const float* sp = a.state + ((size_t)src * a.H + h) * D * D + at;
  float S[R][4];
#pragma unroll
  for (int i = 0; i < R; ++i) load_vec<float, 4>(sp + (size_t)i * D, S[i]);
#pragma unroll 1
  for (int t = t0; t < t1; ++t) {
    const size_t row = ((size_t)t * a.H + h) * D;
    float q[R], k[R], g[R], v[4];
    load_vec<T, R>((const T*)a.q + row + r0, q);
    load_vec<T, R>((const T*)a.k + row + r0, k);
    load_vec<T, R>((const T*)a.g + row + r0, g);
    load_vec<T, 4>((const T*)a.v + row + c0, v);
    const float beta = to_f(((const T*)a.beta)[(size_t)t * a.H + h]);
    float u[4] = {}, w[4] = {}, kq = 0.f;
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const float al = expf(g[i]);
      kq = fmaf(k[i], q[i], kq);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        S[i][j] *= al;
        u[j] = fmaf(S[i][j], k[i], u[j]);
        w[j] = fmaf(S[i][j], q[i], w[j]);
      }
    }
#pragma unroll
    for (int m = CG; m < 32; m <<= 1) {
      kq += __shfl_xor_sync(0xffffffffu, kq, m);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        u[j] += __shfl_xor_sync(0xffffffffu, u[j], m);
        w[j] += __shfl_xor_sync(0xffffffffu, w[j], m);
      }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      u[j] = beta * (v[j] - u[j]);
      w[j] = fmaf(kq, u[j], w[j]);
    }
#pragma unroll
    for (int i = 0; i < R; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) S[i][j] = fmaf(k[i], u[j], S[i][j]);
    if (rg == 0) store4((TO*)a.o + row + c0, w);
  }
  float* dp = a.state + ((size_t)dst * a.H + h) * D * D + at;
#pragma unroll
  for (int i = 0; i < R; ++i) store4(dp + (size_t)i * D, S[i]);
}

constexpr int kStepCols = 32, kStepPerSm = 4;

template <int D>
struct StepSmem {
  static constexpr int stages = D == 128 ? 3 : D == 64 ? 6 : 8;
  static constexpr uint32_t tile = D * kStepCols * 4;
  static constexpr uint32_t vec = stages * tile, red = vec + 2 * D * 16, kq = red + 2 * 4 * 2 * kStepCols * 4;
  static constexpr uint32_t bars = kq + 2 * 4 * 4, total = bars + 8 * stages + 128;  // + slack to align the tiles
};

// The same through shared memory, for large batches at d = 128: a unit of work is 32 columns of one
// head's state, fetched and stored by TMA through a ring, so that the copies of the next units are in
// flight while this one is computed (four CTAs an SM, 48 KB of states each).  Lane = column, warp = a
// quarter of the rows (held in registers over a run's rows); the four partial sums of a column meet in
// shared memory.  512 sequences of 32 heads: 352 us (6.16 TB/s; fp32 rows 339 us, 6.46 TB/s), the
// kernel above 370 us (447 us).  At d = 64 a unit is 8 KB and its barriers cost more than they save
// (569 against 409 us at 2000 sequences).
template <typename T, typename TO, int D>
__global__ void __launch_bounds__(kStepThreads, kStepPerSm)
    kda_step_ring(const __grid_constant__ CUtensorMap tma_state, StepArgs a) {
  using namespace tc;
  using L = StepSmem<D>;
  constexpr int R = D / 4, SL = D / kStepCols, NS = L::stages;  // rows per warp, units per head
  extern __shared__ __align__(128) uint8_t ssm_raw[];
  uint8_t* sm = ssm_raw + ((128u - (smem_u32(ssm_raw) & 127u)) & 127u);
  float4* vec = reinterpret_cast<float4*>(sm + L::vec);  // [2][D]: e^g k, e^g q, e^g, k of a row
  float* red = reinterpret_cast<float*>(sm + L::red);    // [2][warp][u, w][column]
  float* skq = reinterpret_cast<float*>(sm + L::kq);     // [2][warp]
  uint64_t* full = reinterpret_cast<uint64_t*>(sm + L::bars);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int64_t units = (int64_t)a.rows.n_seqs * a.H * SL;
  struct Unit {
    int b, h, c0, src, dst, t0, t1;
    bool ok;
  };
  auto unit_of = [&](int64_t u) {
    Unit x{};
    if (u >= units) return x;
    x.c0 = (int)(u % SL) * kStepCols;
    const int64_t bh = u / SL;
    x.h = (int)(bh % a.H);
    x.b = (int)(bh / a.H);
    x.src = a.src[x.b];
    x.dst = a.dst ? a.dst[x.b] : x.src;
    x.t0 = a.rows.row_start ? a.rows.row_start[x.b] : x.b;
    x.t1 = a.rows.row_start ? a.rows.row_start[x.b + 1] : x.b + 1;
    x.ok = x.src >= 0;  // else a padding entry
    if (x.ok && (x.src >= a.n_slots || x.dst < 0 || x.dst >= a.n_slots || x.t0 < 0 || x.t1 < x.t0 || x.t1 > a.rows.n_rows)) {
      set_status(a.status, kStatusCheck);
      x.ok = false;
    }
    return x;
  };
  auto issue = [&](int64_t u, int st) {  // thread 0: the state of unit u into stage st
    const Unit x = unit_of(u);
    if (!x.ok) {
      mbar_arrive(&full[st]);
      return;
    }
    mbar_arrive_expect_tx(&full[st], L::tile);
    tma_load_2d(sm + st * L::tile, &tma_state, x.c0, (int)(((int64_t)x.src * a.H + x.h) * D), &full[st]);
  };
  // this thread's share of a token: row tid of q, k, g; column c0 + lane of v
  float q = 0.f, k = 0.f, g = 0.f, v = 0.f, beta = 0.f;
  auto load_row = [&](const Unit& x, int t) {
    const size_t row = (size_t)t * a.H + x.h;
    if (tid < D) {
      q = to_f(((const T*)a.q)[row * D + tid]);
      k = to_f(((const T*)a.k)[row * D + tid]);
      g = to_f(((const T*)a.g)[row * D + tid]);
    }
    v = to_f(((const T*)a.v)[row * D + x.c0 + lane]);
    beta = to_f(((const T*)a.beta)[row]);
  };
  if (tid == 0) {
    for (int i = 0; i < NS; ++i) mbar_init(&full[i], 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    for (int i = 0; i < NS - 1; ++i) {
      const int64_t u = blockIdx.x + (int64_t)i * gridDim.x;
      if (u < units) issue(u, i);
    }
  }
  __syncthreads();
  Unit cur = unit_of(blockIdx.x);
  if (cur.ok && cur.t0 < cur.t1) load_row(cur, cur.t0);
  int st = 0, buf = 0;
  uint32_t parity = 0;
#pragma unroll 1
  for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
    const Unit nxt = unit_of(u + gridDim.x);
    const bool more = nxt.ok && nxt.t0 < nxt.t1;
    // the first unit of a sequence looks for another sequence that writes or reads the slot it writes
    if (a.status && cur.ok && cur.h == 0 && cur.c0 == 0) {
      bool clash = false;
      for (int j = tid; j < a.rows.n_seqs; j += kStepThreads) {
        const int sj = a.src[j];
        if (j != cur.b && sj >= 0) clash |= sj == cur.dst || (a.dst && a.dst[j] == cur.dst);
      }
      if (clash) set_status(a.status, kStatusCheck);
    }
    const bool got = mbar_wait(&full[st], parity, 2000000000ull);
    if (!got) set_status(a.status, 8);
    if (cur.ok) {
      float* tile = reinterpret_cast<float*>(sm + st * L::tile) + (warp * R) * kStepCols + lane;
      float S[R];
#pragma unroll
      for (int i = 0; i < R; ++i) S[i] = tile[i * kStepCols];
      if (cur.t0 == cur.t1 && more) load_row(nxt, nxt.t0);
#pragma unroll 1
      for (int t = cur.t0; t < cur.t1; ++t, buf ^= 1) {
        float kq = 0.f;
        if (tid < D) {
          const float al = expf(g);
          vec[buf * D + tid] = make_float4(al * k, al * q, al, k);
          kq = k * q;
        }
#pragma unroll
        for (int m = 16; m; m >>= 1) kq += __shfl_xor_sync(0xffffffffu, kq, m);
        if (lane == 0) skq[buf * 4 + warp] = kq;
        const float v_now = v, b_now = beta;
        __syncthreads();
        if (t + 1 < cur.t1)
          load_row(cur, t + 1);
        else if (more)
          load_row(nxt, nxt.t0);
        const float4* f = vec + buf * D + warp * R;
        float p = 0.f, w = 0.f;
#pragma unroll
        for (int i = 0; i < R; ++i) {
          const float4 x = f[i];
          p = fmaf(S[i], x.x, p);
          w = fmaf(S[i], x.y, w);
        }
        float* rd = red + buf * 4 * 2 * kStepCols;
        rd[(2 * warp) * kStepCols + lane] = p;
        rd[(2 * warp + 1) * kStepCols + lane] = w;
        __syncthreads();
        p = w = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          p += rd[(2 * i) * kStepCols + lane];
          w += rd[(2 * i + 1) * kStepCols + lane];
        }
        const float delta = b_now * (v_now - p);
        if (warp == 0) {
          kq = skq[buf * 4] + skq[buf * 4 + 1] + skq[buf * 4 + 2] + skq[buf * 4 + 3];
          ((TO*)a.o)[((size_t)t * a.H + cur.h) * D + cur.c0 + lane] = from_f<TO>(fmaf(kq, delta, w));
        }
#pragma unroll
        for (int i = 0; i < R; ++i) {
          const float4 x = f[i];
          S[i] = fmaf(S[i], x.z, x.w * delta);
        }
      }
#pragma unroll
      for (int i = 0; i < R; ++i) tile[i * kStepCols] = S[i];
      fence_async_smem();
      if (__syncthreads_and(got) && tid == 0)
        tma_store_2d(sm + st * L::tile, &tma_state, cur.c0, (int)(((int64_t)cur.dst * a.H + cur.h) * D));
    } else if (more) {
      load_row(nxt, nxt.t0);
    }
    if (tid == 0) {
      bulk_commit();
      // the stage before this one is refilled once its store (all but the newest) has read it
      bulk_wait_read_1();
      const int64_t ahead = u + (int64_t)(NS - 1) * gridDim.x;
      if (ahead < units) issue(ahead, st == 0 ? NS - 1 : st - 1);
    }
    cur = nxt;
    if (++st == NS) {
      st = 0;
      parity ^= 1;
    }
  }
  if (tid == 0) bulk_wait_all();
}

// ------------------------------------------------------------------------------------ cache append
struct AppendArgs {
  LatentCache cache;
  DecodeRows rows;
  const void *c, *kr;
  int64_t ld_c, ld_kr;
  int* status;
};

constexpr int kAppendThreads = 128;

// One warp per row: 16 latent elements per lane, then lane i turns the pair (i, i + 32) of the
// rotary key.  Bound by the row's bytes; each is read and written once.
template <typename T>
__global__ void __launch_bounds__(kAppendThreads) latent_append_kernel(AppendArgs a) {
  const int lane = threadIdx.x & 31;
  const int64_t t64 = (int64_t)blockIdx.x * (kAppendThreads / 32) + (threadIdx.x >> 5);
  if (t64 >= a.rows.n_rows) return;
  const int t = (int)t64;
  const RowAt r = row_at(a.rows, t);
  if (r.seq < 0 || r.pos < 0) return;
  const int64_t pg = r.pos / a.cache.page_size;
  const int page = pg < a.cache.max_pages ? a.cache.table[(size_t)r.seq * a.cache.max_pages + pg] : -1;
  if (page < 0 || page >= a.cache.n_pages) {
    if (lane == 0) set_status(a.status, kStatusCheck);
    return;
  }
  __nv_bfloat16* dst =
      a.cache.data + ((size_t)page * a.cache.page_size + (size_t)(r.pos - pg * a.cache.page_size)) * kLatWidth;
  const T* c = (const T*)a.c + (size_t)t * a.ld_c;
  const T* kr = (const T*)a.kr + (size_t)t * a.ld_kr;
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    float x[8];
    load_vec<T, 8>(c + (j * 32 + lane) * 8, x);
    __align__(16) __nv_bfloat16 e[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) e[i] = __float2bfloat16_rn(x[i]);
    reinterpret_cast<uint4*>(dst)[j * 32 + lane] = *reinterpret_cast<const uint4*>(e);
  }
  const float x = to_f(kr[lane]), y = to_f(kr[lane + 32]);
  float cs, sn;
  rope_angle(r.pos, lane, &cs, &sn);
  dst[kLatDim + lane] = __float2bfloat16_rn(x * cs - y * sn);
  dst[kLatDim + 32 + lane] = __float2bfloat16_rn(x * sn + y * cs);
  // a page that two sequences both write: the first of this row's run in the page compares the
  // (sequence, page) pairs of the batch
  if (!a.status) return;
  const int first = a.rows.row_start ? a.rows.row_start[r.seq] : t;
  if (t != first && r.pos % a.cache.page_size) return;
  bool clash = false;
  for (int s = 0; s < a.rows.n_seqs; ++s) {
    const int m = a.rows.row_start ? a.rows.row_start[s + 1] - a.rows.row_start[s] : 1;
    const int64_t kv = a.rows.kv_len[s], p0 = max((int64_t)0, kv - m) / a.cache.page_size;
    const int64_t p1 = min((kv + a.cache.page_size - 1) / a.cache.page_size, (int64_t)a.cache.max_pages);
    if (m <= 0) continue;
    for (int64_t p = p0 + lane; p < p1; p += 32)
      clash |= !(s == r.seq && p == pg) && a.cache.table[(size_t)s * a.cache.max_pages + p] == page;
  }
  if (__any_sync(0xffffffffu, clash) && lane == 0) set_status(a.status, kStatusCheck);
}

// ------------------------------------------------------------------------------------ rotated queries
// The rotary part of the absorbed queries: a warp turns every head of one row.  Lane i takes cos and sin of
// angle i; then four lanes hold a head (8 neighbouring pairs each), eight heads at a time.
__device__ __forceinline__ void absorb_rope_row(const DecodeRows& rows, int H, const __nv_bfloat16* q, int64_t ld_q,
                                                __nv_bfloat16* qa, int t) {
  const int lane = threadIdx.x & 31, j0 = (lane & 3) * 8;
  const RowAt r = row_at(rows, t);
  if (r.seq < 0) return;
  float cs, sn, c[8], s[8];
  rope_angle(r.pos, lane, &cs, &sn);
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    c[j] = __shfl_sync(0xffffffffu, cs, j0 + j);
    s[j] = __shfl_sync(0xffffffffu, sn, j0 + j);
  }
#pragma unroll 2
  for (int h = lane >> 2; h < H; h += 8) {
    const __nv_bfloat16* src = q + (size_t)t * ld_q + (size_t)h * kLatQK + kLatHead + j0;
    __nv_bfloat16* dst = qa + ((size_t)t * H + h) * kLatWidth + kLatDim + j0;
    float x[8], y[8];
    load_vec<__nv_bfloat16, 8>(src, x);
    load_vec<__nv_bfloat16, 8>(src + 32, y);
    __align__(16) __nv_bfloat16 u[8], v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      u[j] = __float2bfloat16_rn(x[j] * c[j] - y[j] * s[j]);
      v[j] = __float2bfloat16_rn(x[j] * s[j] + y[j] * c[j]);
    }
    *reinterpret_cast<uint4*>(dst) = *reinterpret_cast<const uint4*>(u);
    *reinterpret_cast<uint4*>(dst + 32) = *reinterpret_cast<const uint4*>(v);
  }
}

}  // namespace tpc
