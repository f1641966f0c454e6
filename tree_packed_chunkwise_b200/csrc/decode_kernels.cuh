// Kernels of token-by-token generation: the recurrent KDA step on a cache of states, the append to
// the paged cache of latents, and the rotation of the absorbed queries.
#pragma once
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <cstdint>

#include "common.cuh"

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

// the rows first .. end - 1 of a sequence lie within 0 .. n_rows (a sequence whose rows do not has none)
__device__ __forceinline__ bool rows_ok(const DecodeRows& r, int first, int end) {
  return first >= 0 && end >= first && end <= r.n_rows;
}

// the sequence and position of row t, by the whole warp
__device__ __forceinline__ RowAt row_at(const DecodeRows& r, int t) {
  if (!r.row_start) return {t, (int64_t)r.kv_len[t] - 1};
  auto owns = [&](int first, int end) { return t >= first && t < end && rows_ok(r, first, end); };
  int b = seq_of_row(r.row_start, r.n_seqs, t);
  if (b >= r.n_seqs) return {-1, 0};
  int first = r.row_start[b], end = r.row_start[b + 1], kv = r.kv_len[b];
  if (!owns(first, end)) {  // no sequence's row, or the search was misled by a table that decreases somewhere
    uint32_t found = 0;
    const int lane = threadIdx.x & 31;
    for (b = lane; !found && b - lane < r.n_seqs; b += 32)
      found = __ballot_sync(0xffffffffu, b < r.n_seqs && owns(r.row_start[b], r.row_start[b + 1]));
    if (!found) return {-1, 0};
    b = b - lane - 32 + __ffs(found) - 1;
    end = r.row_start[b + 1];
    kv = r.kv_len[b];
  }
  return {b, (int64_t)kv - end + t};
}

// Whether a sequence of this thread's (every `of`-th from `at`) has rows outside 0 .. n_rows
__device__ __forceinline__ bool bad_row_starts(const DecodeRows& r, int64_t at, int64_t of) {
  bool bad = false;
  if (r.row_start)
    for (int64_t b = at; b < r.n_seqs; b += of) bad |= !rows_ok(r, r.row_start[b], r.row_start[b + 1]);
  return bad;
}

// 10000^(-2 i / 64) / (2 pi), the turns per position of the rotary pair i, as powers of 10000^(-1 / 32) (their
// relative errors, with the ratio's own, stay below (2 i + 1) 2^-53, of a value that shrinks by a quarter per i).  A table in memory:
// lane i's load takes the time of the others beside it, a power in double precision more.
struct RopeTurns {
  double t[kLatRope / 2];
  constexpr RopeTurns() : t{} {
    double x = 0.15915494309189535;
    for (int i = 0; i < kLatRope / 2; ++i) {
      t[i] = x;
      x *= 0.7498942093324559;
    }
  }
};
__device__ const RopeTurns kRopeTurns{};

// cos and sin of the angle at position pos.  The angle is taken in turns in double precision and reduced
// there (2^31 positions: error below 1e-6 of a turn), so that far positions keep fp32 accuracy.
__device__ __forceinline__ void rope_angle(int64_t pos, double per_pos, float* cs, float* sn) {
  const double turns = (double)pos * per_pos;
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
  } else {
    static_assert(B == 8, "vector width");
    const uint2 u = *reinterpret_cast<const uint2*>(p);
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
// bound the step (7 flops for the 8 bytes of an element).
//
// A lane holds R rows x 4 columns of one head's state in registers, a warp 4 CG columns; sums over the
// rows are shuffles, and nothing is shared between warps (no barrier, so runs of rows and small batches
// are as short as their loads).  CG neighbouring lanes read 16 CG consecutive bytes of a row: 64 (d = 128
// and 64) or 128.  Many bytes in flight matter most: at d = 128, 512 sequences of 32 heads, bf16 rows, 16 rows
// a lane and 4 CTAs an SM take 324 us (6.69 TB/s, of a measured copy rate of 6.56), 3 CTAs 353 us, 8 rows
// and 6 CTAs 370 us, 8 rows unbounded 439 us, and a ring of TMA copies through shared memory 352 us.
// d = 64 at 2000 sequences 329 us (6.51 TB/s), d = 32 86 us (6.36 TB/s).
template <int D>
struct StepShape {
  static constexpr int R = D == 128 ? 16 : 8, CG = 32 * R / D, warps = D / (4 * CG), per_sm = D == 128 ? 4 : 6;
};

template <typename T, typename TO, int D>
__global__ void __launch_bounds__(kStepThreads, StepShape<D>::per_sm) kda_step_kernel(StepArgs a) {
  constexpr int R = StepShape<D>::R, CG = StepShape<D>::CG, SL = StepShape<D>::warps;
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
  // one warp per sequence looks for another sequence that writes or reads the slot it writes (in place,
  // a later one: the earlier ones look themselves)
  if (a.status && h == 0 && sl == 0) {
    bool clash = false;
#pragma unroll 4
    for (int j = (a.dst ? 0 : b + 1) + lane; j < a.rows.n_seqs; j += 32) {
      const int sj = a.src[j];
      clash |= j != b && sj >= 0 && (sj == dst || (a.dst && a.dst[j] == dst));
    }
    if (clash) set_status(a.status, kStatusCheck);
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
//
// CHECK: with a status word.  A page that two sequences both write, or one twice, is then found by the
// first row of a run in the page, which compares it with the pages that its own and later sequences write
// after it: 100,000 tokens of one sequence in 16-token pages 56 us, 41 without; 4,096 sequences of one token
// 59 and 4.6 us (17 without row_start).  Without a status word the kernel has none of these instructions: 24
// runs of 512 rows take 6.3 us instead of 7.0.
template <typename T, bool CHECK>
__global__ void __launch_bounds__(kAppendThreads) latent_append_kernel(AppendArgs a) {
  const int lane = threadIdx.x & 31;
  const int64_t t64 = (int64_t)blockIdx.x * (kAppendThreads / 32) + (threadIdx.x >> 5);
  if (t64 >= a.rows.n_rows) return;
  const int t = (int)t64;
  if (CHECK && bad_row_starts(a.rows, t64 * 32 + lane, 32ll * a.rows.n_rows)) set_status(a.status, kStatusCheck);
  const T* c = (const T*)a.c + (size_t)t * a.ld_c;
  const T* kr = (const T*)a.kr + (size_t)t * a.ld_kr;
  float l[2][8];  // loaded before the search for the row's place, which is a chain of loads itself
  load_vec<T, 8>(c + lane * 8, l[0]);
  load_vec<T, 8>(c + (32 + lane) * 8, l[1]);
  const float x = to_f(kr[lane]), y = to_f(kr[lane + 32]);
  const RowAt r = row_at(a.rows, t);
  if (r.seq < 0 || r.pos < 0) return;
  const int ps = a.cache.page_size;
  const bool fits = r.pos < (int64_t)a.cache.max_pages * ps;
  const int pos = fits ? (int)r.pos : 0, pg = pos / ps;
  const int page = fits ? a.cache.table[(size_t)r.seq * a.cache.max_pages + pg] : -1;
  if (page < 0 || page >= a.cache.n_pages) {
    if (lane == 0) set_status(a.status, kStatusCheck);
    return;
  }
  __nv_bfloat16* dst = a.cache.data + ((size_t)page * ps + (pos - pg * ps)) * kLatWidth;
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    __align__(16) __nv_bfloat16 e[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) e[i] = __float2bfloat16_rn(l[j][i]);
    reinterpret_cast<uint4*>(dst)[j * 32 + lane] = *reinterpret_cast<const uint4*>(e);
  }
  float cs, sn;
  rope_angle(pos, kRopeTurns.t[lane], &cs, &sn);
  dst[kLatDim + lane] = __float2bfloat16_rn(x * cs - y * sn);
  dst[kLatDim + 32 + lane] = __float2bfloat16_rn(x * sn + y * cs);
  if (!CHECK) return;
  const int first = a.rows.row_start ? a.rows.row_start[r.seq] : t;
  if (t != first && pos % ps) return;
  bool clash = false;
  if (!a.rows.row_start) {
#pragma unroll 4
    for (int s = r.seq + 1 + lane; s < a.rows.n_seqs; s += 32) {
      const int p = max(a.rows.kv_len[s] - 1, 0) / ps;
      clash |= a.rows.kv_len[s] > 0 && p < a.cache.max_pages && a.cache.table[(size_t)s * a.cache.max_pages + p] == page;
    }
  } else {
    auto written = [&](int s, int* p0) -> int {  // pages p0 .. (result) - 1 of sequence s
      const int first = a.rows.row_start[s], end = a.rows.row_start[s + 1];
      const int kv = min(max(a.rows.kv_len[s], 0), a.cache.max_pages * ps);
      if (first == end || kv == 0 || !rows_ok(a.rows, first, end)) return *p0 = 0;
      *p0 = max(kv - (end - first), 0) / ps;
      return (kv - 1) / ps + 1;
    };
    auto pages_by_lanes = [&](int s, int p0, int p1) {
      const int32_t* row = a.cache.table + (size_t)s * a.cache.max_pages;
#pragma unroll 4
      for (int p = p0 + lane; p < p1; p += 32) clash |= row[p] == page;
    };
    int p0, p1 = written(r.seq, &p0);
    pages_by_lanes(r.seq, pg + 1, p1);
    bool put_off = false;  // long runs, which one lane would walk on its own
    for (int s = r.seq + 1 + lane; s < a.rows.n_seqs; s += 32) {
      p1 = written(s, &p0);
      put_off |= p1 - p0 > 64;
      if (p1 - p0 <= 64)
        for (int p = p0; p < p1; ++p) clash |= a.cache.table[(size_t)s * a.cache.max_pages + p] == page;
    }
    if (__any_sync(0xffffffffu, put_off))
      for (int s0 = r.seq + 1; s0 < a.rows.n_seqs; s0 += 32) {
        p1 = s0 + lane < a.rows.n_seqs ? written(s0 + lane, &p0) : p0 = 0;
        for (uint32_t left = __ballot_sync(0xffffffffu, p1 - p0 > 64); left; left &= left - 1) {
          const int l = __ffs(left) - 1;
          pages_by_lanes(s0 + l, __shfl_sync(0xffffffffu, p0, l), __shfl_sync(0xffffffffu, p1, l));
        }
      }
  }
  if (clash) set_status(a.status, kStatusCheck);
}

// ------------------------------------------------------------------------------------ rotated queries
// The rotary part of the absorbed queries: a warp turns every head of one row.  Lane i takes cos and sin of
// angle i; then four lanes hold a head (8 neighbouring pairs each), eight heads at a time.
__device__ __forceinline__ void absorb_rope_row(const DecodeRows& rows, int H,
                                                const __nv_bfloat16* q, int64_t ld_q, __nv_bfloat16* qa, int t) {
  const int lane = threadIdx.x & 31, j0 = (lane & 3) * 8;
  const __nv_bfloat16* src = q + (size_t)t * ld_q + kLatHead + j0;
  uint4 x4, y4;  // the first heads, loaded before the position is known
  int h = lane >> 2;
  auto load = [&] {
    const uint4* p = reinterpret_cast<const uint4*>(src + (size_t)h * kLatQK);
    x4 = p[0];
    y4 = p[4];
  };
  if (h < H) load();
  const RowAt r = row_at(rows, t);
  if (r.seq < 0) return;
  float cs, sn, c[8], s[8];
  rope_angle(r.pos, kRopeTurns.t[lane], &cs, &sn);
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    c[j] = __shfl_sync(0xffffffffu, cs, j0 + j);
    s[j] = __shfl_sync(0xffffffffu, sn, j0 + j);
  }
  while (h < H) {
    const __nv_bfloat16 *x = reinterpret_cast<const __nv_bfloat16*>(&x4), *y = reinterpret_cast<const __nv_bfloat16*>(&y4);
    __align__(16) __nv_bfloat16 u[8], v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float xf = to_f(x[j]), yf = to_f(y[j]);
      u[j] = __float2bfloat16_rn(xf * c[j] - yf * s[j]);
      v[j] = __float2bfloat16_rn(xf * s[j] + yf * c[j]);
    }
    __nv_bfloat16* dst = qa + ((size_t)t * H + h) * kLatWidth + kLatDim + j0;
    h += 8;
    if (h < H) load();
    *reinterpret_cast<uint4*>(dst) = *reinterpret_cast<const uint4*>(u);
    *reinterpret_cast<uint4*>(dst + 32) = *reinterpret_cast<const uint4*>(v);
  }
}

}  // namespace tpc
