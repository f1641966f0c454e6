// Absorbed latent attention over a paged cache on 5th-generation tensor cores (sm_100a).
//
// Every head of every new row of a sequence reads the same cached rows [c | kr], so the (row, head)
// pairs of a sequence are the columns of one product with the cache as its tall operand:
//   S^T [KT tokens x NT columns] = K [KT x 576] Qa^T,   O^T [512 x NT] += C^T [512 x KT] P^T [KT x NT].
// The cached tile is the MMA's A operand both times, once K-major and once (its latent part, the same
// shared memory) MN-major, and is fetched once; the few columns are N, which the tensor core takes
// in steps of 16 (rows as M would fill 16 of 128 lanes).  An MMA with few columns takes the time of reading
// its A operand from shared memory, 4 KB at 128 bytes a cycle for M = 128 (measured: 36 to 58 cycles; 64 to
// 90 when one lane of a diverged warp issues), so a tile of 128 tokens, 36 + 32 MMAs, needs 3,300 cycles of
// the tensor core against 6,200 that its 147 KB take from HBM.
//
// A weight enters its product as two bf16 values, its rounding and the rounding of what that leaves (as in
// the tree attention): one alone is off by 2^-8 at worst, more than the outputs' own rounding where tokens
// cancel.  Up to 32 columns the two parts stand side by side as 2 NT columns of one MMA, whose time is
// still that of its A operand; at 64 columns, where tensor memory has no room for that, they are two products
// one after the other, and a tile is 64 tokens (KT; otherwise 128), whose parts fit beside the cached tiles.
#pragma once
#include <cuda.h>

#include "common.cuh"
#include "decode_kernels.cuh"
#include "tc.cuh"

namespace tpc {
namespace tc {

// 1 in one lane of the (converged) warp, 0 in the others
__device__ __forceinline__ uint32_t elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}\n" : "=r"(p));
  return p;
}
// mma_bf16 and commit of the lane whose `lead` is not 0, for code that the whole warp runs
__device__ __forceinline__ void mma_bf16_if(uint32_t lead, uint32_t d_tmem, uint64_t a, uint64_t b, uint32_t idesc,
                                            uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d_tmem),
      "l"(a), "l"(b), "r"(idesc), "r"(acc), "r"(lead));
}
__device__ __forceinline__ void commit_if(uint32_t lead, uint64_t* bar) {
  asm volatile(
      "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %1, 0;\n\t"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}\n" ::"r"(smem_u32(bar)),
      "r"(lead)
      : "memory");
}

// as mbar_try_wait, which may suspend the thread for a while, but returns at once
__device__ __forceinline__ bool mbar_test_wait(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\tmbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}\n"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}

// The kernels' waits are bounded by a limit of their arguments; with 0 they give up at once, so that the ways
// out can be tested (the attention, whose waits cost time, starts as if one had run out).  What a CTA waits
// for on its way out (its copies to land, its MMAs to complete) is bounded by kWayOutNs instead, whatever the
// limit.
constexpr uint64_t kWayOutNs = 2000000000ull;
__device__ __forceinline__ bool mbar_wait_limit(uint64_t* bar, uint32_t parity, uint64_t limit_ns) {
  return limit_ns ? mbar_wait(bar, parity, limit_ns) : mbar_test_wait(bar, parity);
}

// fetches a tensor map (a __grid_constant__ parameter) ahead of its first use
__device__ __forceinline__ void prefetch_tensor_map(const void* tmap) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(tmap) : "memory");
}

}  // namespace tc

constexpr int kLatBox = 64;                         // most rows of one TMA box
constexpr int kLatChunks = kLatWidth / 64;          // 64-column chunks of a cached row (the last one rotary)
constexpr int kLatItems = 1 + kLatDim / 128;        // slots of a tile: the rotary chunk, then pairs of latent chunks
constexpr int kLatAttnThreads = 192;                // producer warp, MMA warp, four softmax warps
constexpr int kLatMaxCtas = 148;
constexpr int kLatMaxNT = 64;

// A tile goes through a ring of slots of two chunks, so that its slots are refilled one by one: the rotary
// chunk once the scores have read it, each latent pair once its 128 dimensions are summed.  At NT = 64 the
// rotary chunk has a slot of its own and the ring holds two tiles' pairs: the next tile's scores are complete
// before the weights of this one are there.
// The weights P^T stand in shared memory as two bf16 operands, high parts and what they leave (low parts):
// 64 tokens by 2 NT rows at a time, high before low.
template <int NT>
struct LatSmem {
  static constexpr int KT = NT == 64 ? 64 : 128;  // tokens per tile
  static constexpr uint32_t chunk = KT * 128, slot = 2 * chunk, slots = NT == 16 ? 6 : NT == 32 ? 5 : 8;
  static constexpr bool own_rope = NT == 64;         // slot number `slots`
  static constexpr int ring_items = kLatItems - own_rope;  // of a tile
  static constexpr uint32_t q = 0, ring = q + kLatChunks * NT * 128, p = ring + slots * slot + own_rope * chunk,
                            end = p + KT / 64 * 2 * NT * 128;
  // item e of the CTA's tile `it`: its slot, and how many items the slot held before
  static __device__ __forceinline__ uint32_t slot_of(int it, int e) {
    return own_rope && e == 0 ? slots : (uint32_t)(it * ring_items + e - own_rope) % slots;
  }
  static __device__ __forceinline__ uint32_t uses_of(int it, int e) {
    return own_rope && e == 0 ? it : (uint32_t)(it * ring_items + e - own_rope) / slots;
  }
  static constexpr uint32_t red = end, fac = red + 2 * 4 * NT * 4, lim = fac + NT * 4, bars = lim + NT * 4;
  static constexpr uint32_t total = bars + 320;
};
static_assert(LatSmem<64>::total <= 232448 && LatSmem<32>::total <= 232448 && LatSmem<16>::total <= 232448,
              "shared memory of one CTA");

// scratch: partial sums of the pieces (two per CTA), their (maximum, sum of the weights), and one record per CTA
struct LatPiece {
  int col0;  // first (row, head) pair of the split unit that starts in this CTA
  int ncols;
  int n;     // its pieces: this CTA's last one, then the first ones of the next n - 1 CTAs
};
constexpr size_t kLatPartBytes = (size_t)kLatMaxCtas * 2 * kLatMaxNT * kLatDim * 4;
constexpr size_t kLatMlBytes = (size_t)kLatMaxCtas * 2 * kLatMaxNT * 8;
constexpr size_t kLatScratch = kLatPartBytes + kLatMlBytes + ((kLatMaxCtas * sizeof(LatPiece) + 255) / 256) * 256;

struct LatAttnArgs {
  LatentCache cache;
  DecodeRows rows;
  int H;
  float scale_log2;  // scale * log2(e)
  __nv_bfloat16* o;
  float* lse;
  float* part;
  float2* ml;
  LatPiece* meta;
  int* status;
  uint64_t wait_ns;
};

struct LatSeq {
  int row0, m, kv;
};
struct LatStart {  // where a share begins
  int b, ct, tile;
  LatSeq s;
};

__device__ __forceinline__ LatSeq lat_seq(const LatAttnArgs& a, int b) {
  LatSeq s;
  s.row0 = a.rows.row_start ? a.rows.row_start[b] : b;
  const int end = a.rows.row_start ? a.rows.row_start[b + 1] : b + 1;
  s.kv = max(a.rows.kv_len[b], 0);
  s.m = end - s.row0;
  if (s.row0 < 0 || end < s.row0 || end > a.rows.n_rows) {
    set_status(a.status, kStatusCheck);
    s.row0 = s.m = 0;
  }
  const int cap = a.cache.max_pages * a.cache.page_size;
  if (s.kv > cap && s.m > 0) set_status(a.status, kStatusCheck);
  s.kv = min(s.kv, cap);
  return s;
}

// column tiles of a sequence
template <int NT>
__device__ __forceinline__ int lat_cts(const LatAttnArgs& a, const LatSeq& s) {
  return (s.m * a.H + NT - 1) / NT;
}
// token tiles that the columns of column tile ct can see (at least one: the rows are written either way)
template <int NT>
__device__ __forceinline__ int lat_tiles(const LatAttnArgs& a, const LatSeq& s, int ct) {
  constexpr int KT = LatSmem<NT>::KT;
  const int last = s.m == 1 ? 0 : min(((ct + 1) * NT - 1) / a.H, s.m - 1);
  return max(1, (s.kv - s.m + last + KT) / KT);
}

// Walks a CTA's share of the work: pieces (column tile of a sequence, range of token tiles)
template <int NT>
struct LatWalk {
  const LatAttnArgs& a;
  long long left;
  int b, ct, t0, n, tiles;
  LatSeq s;
  __device__ LatWalk(const LatAttnArgs& args, const LatStart& at, long long count)
      : a(args), left(count), b(at.b), ct(at.ct), t0(at.tile), n(0), tiles(0), s(at.s) {
    if (left > 0) size();
  }
  __device__ void size() {
    tiles = lat_tiles<NT>(a, s, ct);
    n = (int)min((long long)(tiles - t0), left);
  }
  __device__ void next() {  // the share's weights were summed from the same numbers, so b stays in range
    left -= n;
    if (left <= 0) return;
    t0 = 0;
    if (++ct < lat_cts<NT>(a, s)) {
      size();
      return;
    }
    ct = 0;
    do {
      if (++b >= a.rows.n_seqs) {
        left = 0;
        return;
      }
      s = lat_seq(a, b);
    } while (s.m <= 0);
    size();
  }
};

// 8 * R columns of 16 TMEM lanes, spread over the warp: x[4 j + e] is lane l / 4 + 8 (e / 2), column
// 8 j + 2 (l % 4) + e % 2
template <int R>
__device__ __forceinline__ void tmem_ld_16x256(uint32_t taddr, float (&x)[4 * R]) {
  uint32_t r[4 * R];
  if constexpr (R == 2) {
    asm volatile("tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(taddr));
  } else if constexpr (R == 4) {
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
  } else {
    static_assert(R == 8, "16, 32 or 64 columns");
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
          "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
          "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr));
  }
  tc::tmem_wait_ld();
#pragma unroll
  for (int i = 0; i < 4 * R; ++i) {
    asm volatile("" : "+r"(r[i]));
    x[i] = __uint_as_float(r[i]);
  }
}

// four 8 x 8 bf16 matrices in MMA accumulator order, each stored transposed: lane l gives the address of
// stored row l % 8 (16 bytes) of matrix l / 8
__device__ __forceinline__ void stmatrix4_trans(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(a), "r"(b), "r"(c),
               "r"(d)
               : "memory");
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// 32 fp32 accumulator values (as tmem_ld32_nowait gives them) rounded to bf16 at p (16-byte aligned)
__device__ __forceinline__ void round_to_smem(const uint32_t (&r)[32], uint8_t* p) {
#pragma unroll
  for (int i = 0; i < 32; i += 8) {
    uint32_t e[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) e[j] = pack_bf16(__uint_as_float(r[i + 2 * j]), __uint_as_float(r[i + 2 * j + 1]));
    *reinterpret_cast<uint4*>(p + 2 * i) = make_uint4(e[0], e[1], e[2], e[3]);
  }
}

// Persistent: the token tiles of all (sequence, column tile) units are one list, cut into equal
// shares, one CTA each, so ragged lengths balance and one long context uses every SM.  The shares are
// found on the device from kv_len (no host copy, graphs replay with new lengths).  A unit that is cut
// leaves partial sums for latent_combine_kernel.
//
// Warp 0 fetches tiles by TMA (64-column boxes, one per page and column chunk) into the ring (a prefetch
// of the next tile into L2 beside it measured 2 % slower).  Warp 1 issues the MMAs: the scores of tile i + 1
// as far as its slots have arrived, and the weighted sum of tile i as soon as the weights are there.  Warps
// 2-5 run the softmax: a warp holds KT / 4 tokens x NT columns of S^T in the 16x256b register layout, maxima
// over tokens are 3 shuffles and one exchange between the four warps.  Running sums stay per lane until the piece ends.  A column's maximum is only
// raised when it grew by more than 8 (base 2): until then its weights are at most 2^8 and the sums of
// the old maximum stay valid, which saves the pass over O^T.
//
// 64 contexts of 16,384 tokens, 16 heads: 213 us (5.67 TB/s of cache, 86 % of the copy rate; copies alone
// 186 us), 32 heads (NT = 32, half the tokens) 130 us.  Runs of 300 rows over 4,096 tokens (NT = 64): 440
// TFLOP/s (without the low parts 490, the rows' bound being the chain of scores, softmax and weighted sum).
// Kernel times of 64 contexts of 4,000 tokens with 16, 32 and 64 columns a tile: one row of 16 heads (16
// columns used) 65, 73 and 92 us; 2 rows 105, 75 and 92; 4 rows 214, 126 and 94.
template <int NT>
__global__ void __launch_bounds__(kLatAttnThreads, 1)
    latent_attn_tc(const __grid_constant__ CUtensorMap tma_kv, const __grid_constant__ CUtensorMap tma_q, LatAttnArgs a) {
  using namespace tc;
  using L = LatSmem<NT>;
  constexpr int R = NT / 8, U = L::slots, KT = L::KT, G = KT / 64;  // G: 16-token groups of a softmax warp
  // columns of an accumulator of O^T: products with the high and the low parts side by side where they fit
  constexpr int W = NT == 64 ? NT : 2 * NT;
  constexpr uint32_t kTmem = NT == 16 ? 256 : 512, kScores = 4 * W;
  extern __shared__ __align__(1024) uint8_t lsm_raw[];
  uint8_t* sm = lsm_raw;
  const uint32_t sb = smem_u32(sm);
  if (sb & 1023u) {  // the tiles need the alignment that the array asks for (there is no room to correct it)
    set_status(a.status, kStatusCheck);
    if (threadIdx.x == 0) a.meta[blockIdx.x].n = 0;
    return;
  }
  float* red = reinterpret_cast<float*>(sm + L::red);
  float* fac = reinterpret_cast<float*>(sm + L::fac);
  int* lim = reinterpret_cast<int*>(sm + L::lim);
  uint64_t* bars = reinterpret_cast<uint64_t*>(sm + L::bars);
  uint64_t *full = bars, *empty = bars + 9, *s_full = bars + 18, *p_full = bars + 20, *o_done = bars + 22,
           *q_full = bars + 24, *q_empty = bars + 25, *done = bars + 26;
  uint32_t* tslot = reinterpret_cast<uint32_t*>(bars + 27);
  int* abort_flag = reinterpret_cast<int*>(bars + 27) + 1;
  LatStart* where = reinterpret_cast<LatStart*>(bars + 28);
  long long* sums = reinterpret_cast<long long*>(bars + 31);  // per warp
  const int tid = threadIdx.x, w = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    prefetch_tensor_map(&tma_kv);
    prefetch_tensor_map(&tma_q);
  }

  // ---- this CTA's share: every thread sums the tiles of consecutive sequences
  const int lo = (int)((long long)a.rows.n_seqs * tid / kLatAttnThreads);
  const int hi = (int)((long long)a.rows.n_seqs * (tid + 1) / kLatAttnThreads);
  long long mine = 0;
#pragma unroll 1
  for (int b = lo; b < hi; ++b) {
    const LatSeq s = lat_seq(a, b);
    const int n = lat_cts<NT>(a, s);
#pragma unroll 1
    for (int c = 0; c < n; ++c) mine += lat_tiles<NT>(a, s, c);
  }
  long long incl = mine;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, incl, d);
    if (lane >= d) incl += y;
  }
  if (lane == 31) sums[w] = incl;
  if (w == 1) tmem_alloc(tslot, kTmem);
  if (tid == 0) {
    for (int i = 0; i < U + L::own_rope; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&p_full[i], 4);
      mbar_init(&o_done[i], 1);
    }
    for (uint64_t* b : {q_full, q_empty, done}) mbar_init(b, 1);
    *abort_flag = a.wait_ns == 0;
    if (a.wait_ns == 0) set_status(a.status, 8);
    where->b = -1;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  fence_before_sync();
  __syncthreads();
  fence_after_sync();
  long long total = 0;
  for (int i = 0; i < kLatAttnThreads / 32; ++i) {
    if (i < w) incl += sums[i];
    total += sums[i];
  }
  const long long per = total <= INT32_MAX ? ((unsigned)total + gridDim.x - 1) / gridDim.x : (total + gridDim.x - 1) / gridDim.x;
  const long long start = per * blockIdx.x, share = max(0ll, min(per, total - start));
  if (share > 0 && start >= incl - mine && start < incl) {
    long long at = start - (incl - mine);
#pragma unroll 1
    for (int b = lo; b < hi; ++b) {
      const LatSeq s = lat_seq(a, b);
      const int n = lat_cts<NT>(a, s);
#pragma unroll 1
      for (int c = 0; c < n; ++c) {
        const int t = lat_tiles<NT>(a, s, c);
        if (at >= 0 && at < t) *where = {b, c, (int)at, s};
        at -= t;
      }
    }
  }
  __syncthreads();
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // latent_combine_kernel waits for this grid's end itself
  const uint32_t tb = *tslot;
  LatWalk<NT> walk(a, *where, where->b < 0 ? 0 : share);  // (< 0: no start was found: lengths changed, which they must not)
  auto aborted = [&] { return *((volatile int*)abort_flag) != 0; };
  // Every wait is bounded.  After the first that runs out no role waits any more; the producer stops, the
  // others walk on to the end of their loops, so the barriers between the softmax warps match.
  auto give_up = [&] {
    set_status(a.status, 8);
    atomicExch(abort_flag, 1);
  };
  auto wait = [&](uint64_t* bar, uint32_t parity) -> bool {
    if (aborted()) return false;
    if (mbar_wait(bar, parity, a.wait_ns)) return true;
    give_up();
    return false;
  };

  if (w == 0) {  // ---- producer
    const int ps = a.cache.page_size, box = min(ps, kLatBox);
    struct Tile {
      bool valid, first;
      int segs, page, off, q_row;  // page of segment `lane` as the table holds it, first row inside it
    };
    int ahead = 0;                 // tile of the walk's piece that fetch() returns next
    auto fetch = [&]() -> Tile {   // only loads the page number: it is looked at a tile later
      Tile t{walk.left > 0, ahead == 0, 0, 0, 0, 0};
      if (!t.valid) return t;
      const int t0 = (walk.t0 + ahead) * KT;
      t.segs = (min(max(walk.s.kv - t0, 0), KT) + box - 1) / box;
      t.q_row = walk.s.row0 * a.H + walk.ct * NT;
      if (lane < t.segs) {
        const int tok = t0 + lane * box;
        t.page = a.cache.table[(size_t)walk.b * a.cache.max_pages + tok / ps];
        t.off = tok % ps;
      }
      if (++ahead == walk.n) {
        ahead = 0;
        walk.next();
      }
      return t;
    };
    int it = 0, pieces = 0, ring_sent = 0, rope_sent = 0;  // tiles, and copies issued to each kind of slot
    bool ok = true;
    Tile cur = fetch(), nxt = cur;
    while (cur.valid && ok) {
      if (cur.page < 0 || cur.page >= a.cache.n_pages) {
        set_status(a.status, kStatusCheck);
        cur.page = a.cache.n_pages;  // past the tensor map's end: the copies read zeros, no other sequence's tokens
        cur.off = 0;
      }
      const int my_row = cur.page * ps + cur.off;
      if (cur.first) {
        ok = __all_sync(0xffffffffu, pieces == 0 || wait(q_empty, (pieces - 1) & 1));
        if (!ok) break;
        if (lane == 0) mbar_arrive_expect_tx(q_full, kLatChunks * NT * 128);
        __syncwarp();
        if (lane < kLatChunks) tma_load_2d(sm + L::q + lane * NT * 128, &tma_q, 64 * lane, cur.q_row, q_full);
        ++pieces;
      }
      for (int e = 0; e < kLatItems; ++e) {
        const uint32_t st = L::slot_of(it, e), uses = L::uses_of(it, e);
        const int nc = e == 0 ? 1 : 2;  // chunks of the item: 8, then 0 1, 2 3, 4 5, 6 7
        if (e == 1) nxt = fetch();
        ok = __all_sync(0xffffffffu, uses == 0 || wait(&empty[st], (uses - 1) & 1));
        if (!ok) break;
        ++(L::own_rope && e == 0 ? rope_sent : ring_sent);
        if (lane == 0) {
          if (cur.segs)
            mbar_arrive_expect_tx(&full[st], cur.segs * nc * box * 128);
          else
            mbar_arrive(&full[st]);
        }
        __syncwarp();
        const int seg = lane / nc, c = lane % nc;
        const int row = __shfl_sync(0xffffffffu, my_row, seg);
        if (seg < cur.segs)
          tma_load_2d(sm + L::ring + st * L::slot + c * L::chunk + seg * box * 128, &tma_kv,
                      64 * (e == 0 ? kLatChunks - 1 : 2 * (e - 1) + c), row, &full[st]);
      }
      cur = nxt;
      ++it;
    }
    if (lane == 0) {  // every copy lands before the CTA ends, whoever gave up (at once if no one did)
      for (int i = max(0, ring_sent - U); i < ring_sent; ++i) mbar_wait(&full[i % U], (i / U) & 1, kWayOutNs);
      if (rope_sent > 0) mbar_wait(&full[U], (rope_sent - 1) & 1, kWayOutNs);
      if (pieces > 0) mbar_wait(q_full, (pieces - 1) & 1, kWayOutNs);
    }
  } else if (w == 1) {  // ---- MMA
    // The whole warp walks the loops and one elected lane issues, so that descriptors stay in uniform
    // registers.
    const uint32_t lead = elect_one();
    constexpr uint32_t id_s = idesc_bf16(KT, NT, false, false), id_o = idesc_bf16(128, W, true, false);
    // descriptors of slot 0 and of step 0; the low word holds address / 16
    const uint64_t d_kv_k = sw_desc_k(sb + L::ring, KT, 0), d_kv_mn = sw_desc_mn(sb + L::ring, KT, 0);
    const uint64_t d_q = sw_desc_k(sb + L::q, NT, 0), d_p = sw_desc_k(sb + L::p, 2 * NT, 0);
    auto k_step = [](int rows, int ks) { return (uint64_t)(((ks >> 2) * rows * 128 + (ks & 3) * 32) >> 4); };
    int it = 0, piece = 0, slot = 0, pend = -1;  // slot: of the next item in the ring; pend: tile whose weighted sum is not issued yet
    int pend_slot = 0;                           // slot of its first latent pair
    uint32_t pend_acc = 0;
    auto weighted_sum = [&] {  // O^T (+)= C^T P^T of the pending tile
      fence_after_sync();
      int st = pend_slot;
#pragma unroll
      for (int mb = 0; mb < 4; ++mb) {
        const uint64_t d = d_kv_mn + (uint64_t)(st * (L::slot >> 4));
#pragma unroll
        for (int part = 0; part < 2 * NT / W; ++part)
#pragma unroll
          for (int ks = 0; ks < KT / 16; ++ks)
            mma_bf16_if(lead, tb + mb * W, d + (uint64_t)(ks * (2048 >> 4)), d_p + (uint64_t)(part * (W * 128 >> 4)) + k_step(2 * NT, ks),
                        id_o, part || ks ? 1u : pend_acc);
        if (mb == 3) commit_if(lead, &o_done[pend & 1]);
        commit_if(lead, &empty[st]);
        st = st + 1 == U ? 0 : st + 1;
      }
      pend = -1;
    };
    // Waits for item e of tile `it` (ready: bits of items known to be there) and, with it, for the piece's
    // queries, and issues the pending sum meanwhile, on which they may depend.
    uint32_t ready = 0;
    auto wait_item = [&](int e) -> bool {
      const uint32_t queries = 1u << (kLatItems + 1), need = 1u << e | queries;
      uint64_t t0 = 0;
      while ((ready & need) != need) {
        if constexpr (NT == 64) {
          // One look at a barrier takes 200 to 400 cycles of the warp that also issues the MMAs, so every lane
          // looks at another one: the items of the tile (their slots' earlier copies have been waited for), the
          // pending weights, the queries.  Runs of 300 rows over 4,096 tokens 361 us, one look after the other 414.
          bool up = false;
          if (lane < kLatItems)
            up = mbar_test_wait(&full[L::slot_of(it, lane)], L::uses_of(it, lane) & 1);
          else if (lane == kLatItems)
            up = pend >= 0 && mbar_test_wait(&p_full[pend & 1], (pend >> 1) & 1);
          else if (lane == kLatItems + 1)
            up = mbar_test_wait(q_full, piece & 1);
          ready = __ballot_sync(0xffffffffu, up);
          __syncwarp();
          if (ready >> kLatItems & 1) weighted_sum();
        } else {
          // (bound by the copies: looks that suspend the warp, 64 x 16,384 tokens 210 us, otherwise 219)
          if (pend >= 0 && __all_sync(0xffffffffu, mbar_try_wait(&p_full[pend & 1], (pend >> 1) & 1))) weighted_sum();
          if (!(ready & queries) && __all_sync(0xffffffffu, mbar_try_wait(q_full, piece & 1))) ready |= queries;
          if (__all_sync(0xffffffffu, mbar_try_wait(&full[L::slot_of(it, e)], L::uses_of(it, e) & 1))) ready |= 1u << e;
        }
        if ((ready & need) == need) break;
        if (__any_sync(0xffffffffu, aborted())) return false;
        const uint64_t t = globaltimer();
        if (t0 == 0) t0 = t;
        if (t - t0 > a.wait_ns) give_up();
      }
      return true;
    };
    auto sum_now = [&] {
      if (pend >= 0 && __all_sync(0xffffffffu, wait(&p_full[pend & 1], (pend >> 1) & 1))) weighted_sum();
    };
    // (loop bounds read from one lane: the compiler then knows that the warp agrees on them)
    for (; __shfl_sync(0xffffffffu, walk.left > 0, 0); walk.next(), ++piece) {
      const int n = __shfl_sync(0xffffffffu, walk.n, 0);
      for (int i = 0; i < n; ++i, ++it) {
        const uint32_t acc = tb + kScores + (it & 1) * NT;
#pragma unroll
        for (int e = 0; e < kLatItems; ++e) {
          const int st = L::own_rope && e == 0 ? U : slot;
          if (st == slot) slot = slot + 1 == U ? 0 : slot + 1;
          if (e == 0) ready = NT == 64 || i == 0 ? 0u : 1u << (kLatItems + 1);
          if (!wait_item(e)) continue;
          fence_after_sync();
          const uint64_t d = d_kv_k + (uint64_t)(st * (L::slot >> 4));
          if (e == 0) {
#pragma unroll
            for (int ks = 0; ks < 4; ++ks)
              mma_bf16_if(lead, acc, d + k_step(KT, ks), d_q + k_step(NT, 4 * (kLatChunks - 1) + ks), id_s, ks ? 1u : 0u);
            commit_if(lead, &empty[st]);
          } else {
#pragma unroll
            for (int ks = 0; ks < 8; ++ks)
              mma_bf16_if(lead, acc, d + k_step(KT, ks), d_q + k_step(NT, 8 * (e - 1) + ks), id_s, 1u);
          }
        }
        if (!__any_sync(0xffffffffu, aborted())) {
          commit_if(lead, &s_full[it & 1]);
          if (i == n - 1) commit_if(lead, q_empty);
        }
        sum_now();  // the previous tile's sum before this one becomes the pending one
        pend = it;
        pend_acc = i > 0 ? 1u : 0u;
        pend_slot = slot >= 4 ? slot - 4 : slot - 4 + U;
      }
    }
    sum_now();
    commit_if(lead, done);  // the MMAs are complete before TMEM is freed, whoever gave up
    if (!mbar_wait(done, 0, kWayOutNs)) set_status(a.status, 8);
    __syncwarp();
  } else {  // ---- softmax warps: sub-partition sp holds tokens 16 G sp .. 16 G sp + 16 G - 1 of a tile, and
            //      latent dimensions 32 sp .. 32 sp + 31 of each 128-row block of O^T
    const int sp = w & 3, k0 = 16 * G * sp + (lane >> 2), st = tid - 64;
    const uint32_t la = tb + ((uint32_t)(32 * sp) << 16);
    auto meet = [] { asm volatile("bar.sync 1, 128;" ::: "memory"); };
    int it = 0;
    if (st == 0) a.meta[blockIdx.x].n = 0;
    for (; walk.left > 0; walk.next()) {
      const LatSeq s = walk.s;
      const int col0 = s.row0 * a.H + walk.ct * NT, ncols = min(NT, s.m * a.H - walk.ct * NT);
      // last visible position of every column (columns past the run's end take its last row's)
      if (st < NT) lim[st] = s.kv - s.m + min((walk.ct * NT + st) / a.H, s.m - 1);
      const int lim0 = s.kv - s.m + walk.ct * NT / a.H;
      float mx[2 * R], sum[2 * R];
#pragma unroll
      for (int c = 0; c < 2 * R; ++c) {
        // columns past the unit's own hold queries of other sequences, or of rows outside every one: with
        // this maximum they never ask for a pass over O^T
        mx[c] = 8 * (c >> 1) + 2 * (lane & 3) + (c & 1) < ncols ? -INFINITY : INFINITY;
        sum[c] = 0.f;
      }
      meet();  // lim is set; the last piece's reads of red and fac are over
      for (int i = 0; i < walk.n; ++i, ++it) {
        const int t0 = (walk.t0 + i) * KT;
        wait(&s_full[it & 1], (it >> 1) & 1);
        __syncwarp();
        fence_after_sync();
        float x[G][4 * R];  // [16-token group][...]; the rows of an M = 64 accumulator are lanes 0 .. 15 of a sub-partition
#pragma unroll
        for (int g = 0; g < G; ++g) tmem_ld_16x256<R>(la + ((uint32_t)(16 * g) << 16) + kScores + (it & 1) * NT, x[g]);
        const bool mask = t0 + KT - 1 > lim0;
        // Tokens of the tile that some of the rows do not see: with a weight of 0 a latent that is not finite would
        // still make their sums NaN.  Its scores are not finite either, so only then the latents are looked
        // at, those that are not finite leave the product, and the rows that see them become NaN here.
        const int part0 = max(max(lim0 + 1 - t0, 0), 16 * G * sp), part1 = min(min(s.kv - t0, KT), 16 * G * (sp + 1));
        if (part0 < part1) {  // (of this warp's tokens)
          bool odd = false;
#pragma unroll
          for (int g = 0; g < G; ++g)
#pragma unroll
            for (int j = 0; j < 4 * R; ++j) odd |= !(fabsf(x[g][j]) <= 3.4028235e38f);
          if (__any_sync(0xffffffffu, odd)) {
            uint32_t gone = 0;
#pragma unroll 1
            for (int r = part0; r < part1; ++r) {
              uint4 v[2];
              bool bad = false;
#pragma unroll
              for (int h = 0; h < 2; ++h) {  // 16-byte unit lane + 32 h of the row: chunk 4 h + lane / 8
                const int c = 4 * h + (lane >> 3);
                uint8_t* p = sm + L::ring + L::slot_of(it, 1 + (c >> 1)) * L::slot + (c & 1) * L::chunk + r * 128 + (lane & 7) * 16;
                v[h] = *reinterpret_cast<const uint4*>(p);
                for (uint32_t u : {v[h].x, v[h].y, v[h].z, v[h].w}) bad |= (u & 0x7f80u) == 0x7f80u || (u & 0x7f800000u) == 0x7f800000u;
              }
              if (!__any_sync(0xffffffffu, bad)) continue;
              gone |= 1u << (r - 16 * G * sp);
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                const int c = 4 * h + (lane >> 3);
                uint8_t* p = sm + L::ring + L::slot_of(it, 1 + (c >> 1)) * L::slot + (c & 1) * L::chunk + r * 128 + (lane & 7) * 16;
                *reinterpret_cast<uint4*>(p) = make_uint4(0, 0, 0, 0);
              }
            }
#pragma unroll
            for (int g = 0; g < G; ++g)
#pragma unroll
              for (int j = 0; j < 4 * R; ++j)
                if (gone >> (16 * g + 8 * (j >> 1 & 1) + (lane >> 2)) & 1) x[g][j] = __int_as_float(0x7fffffff);
          }
        }
        float tm[2 * R];
#pragma unroll
        for (int c = 0; c < 2 * R; ++c) {  // maximum of each column over the tile
          float v = -INFINITY;
          const int last = mask ? lim[8 * (c >> 1) + 2 * (lane & 3) + (c & 1)] : 0;
#pragma unroll
          for (int g = 0; g < 2 * G; ++g) {
            float& y = x[g >> 1][4 * (c >> 1) + 2 * (g & 1) + (c & 1)];
            y = mask && t0 + k0 + 8 * g > last ? -INFINITY : y * a.scale_log2;
            v = fmaxf(v, y);
          }
          v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 4));
          v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 8));
          tm[c] = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 16));
        }
        float* rd = red + (it & 1) * 4 * NT;
        if (lane < 4) {
#pragma unroll
          for (int j = 0; j < R; ++j)
            *reinterpret_cast<float2*>(rd + sp * NT + 8 * j + 2 * lane) = make_float2(tm[2 * j], tm[2 * j + 1]);
        }
        meet();
        bool grew = false;
#pragma unroll
        for (int j = 0; j < R; ++j) {
          float2 v = make_float2(-INFINITY, -INFINITY);
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const float2 u = *reinterpret_cast<const float2*>(rd + q * NT + 8 * j + 2 * (lane & 3));
            v.x = fmaxf(v.x, u.x);
            v.y = fmaxf(v.y, u.y);
          }
          tm[2 * j] = v.x;
          tm[2 * j + 1] = v.y;
          grew |= v.x > mx[2 * j] + 8.f || v.y > mx[2 * j + 1] + 8.f;
        }
        // the same data in every warp, so the four agree
        grew = __any_sync(0xffffffffu, grew);
        if (grew) {
#pragma unroll
          for (int c = 0; c < 2 * R; ++c) {  // (only columns that grew: a column's results depend on itself alone)
            const bool up = tm[c] > mx[c] + 8.f;
            const float f = up ? ex2(mx[c] - tm[c]) : 1.f;
            if (up) mx[c] = tm[c];
            sum[c] *= f;
            tm[c] = f;
          }
        }
        if (i > 0) {  // the last tile's weights have been read, and its sum is complete
          wait(&o_done[(it - 1) & 1], ((it - 1) >> 1) & 1);
          __syncwarp();
          fence_after_sync();
          if (grew) {
            if (sp == 0 && lane < 4) {
#pragma unroll
              for (int j = 0; j < R; ++j)
                *reinterpret_cast<float2*>(fac + 8 * j + 2 * lane) = make_float2(tm[2 * j], tm[2 * j + 1]);
            }
            meet();
#pragma unroll 1
            for (int c0 = 0; c0 < 4 * W; c0 += 16) {
              float v[16];
              tmem_ld16(la + c0, v);
#pragma unroll
              for (int c = 0; c < 16; ++c) v[c] *= fac[(c0 % NT) + c];
              tmem_st16(la + c0, v);
            }
          }
        }
        // weights: fp32 into their sum; into the product as two bf16 values (the tensor core's operand type),
        // the second holding what the first leaves, so that a weight is off by less than 2^-16 of itself
#pragma unroll
        for (int c = 0; c < 2 * R; ++c) {
          const float m = mx[c] == -INFINITY ? 0.f : mx[c];
#pragma unroll
          for (int g = 0; g < 2 * G; ++g) {
            float& y = x[g >> 1][4 * (c >> 1) + 2 * (g & 1) + (c & 1)];
            y = ex2(y - m);
            sum[c] += y;
          }
        }
        const uint32_t ph = sb + L::p + (16 * G * sp / 64) * 2 * NT * 128;
#pragma unroll
        for (int g = 0; g < G; ++g)
#pragma unroll
          for (int j = 0; j < R; j += 2) {
            const int n = 8 * (j + (lane >> 4)) + (lane & 7), unit = 2 * ((G * sp + g) & 3) + ((lane >> 3) & 1);
            const uint32_t at = ph + n * 128 + ((unit ^ (lane & 7)) << 4);
            uint32_t hi[4], lo[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float y0 = x[g][4 * j + 2 * e], y1 = x[g][4 * j + 2 * e + 1];
              hi[e] = pack_bf16(y0, y1);
              lo[e] = pack_bf16(y0 - __uint_as_float(hi[e] << 16), y1 - __uint_as_float(hi[e] & 0xffff0000u));
            }
            stmatrix4_trans(at, hi[0], hi[1], hi[2], hi[3]);
            stmatrix4_trans(at + NT * 128, lo[0], lo[1], lo[2], lo[3]);
          }
        // rows of the tile that hold no token of the sequence: their weights are 0, but whatever the
        // page holds there (NaN among it) must not meet them
        const int have = max(s.kv - t0, 0);
        if (have < KT) {
          const int per_chunk = (KT - have) * 8;
          for (int c = 0; c < kLatDim / 64; ++c) {
            uint8_t* row = sm + L::ring + L::slot_of(it, 1 + (c >> 1)) * L::slot + (c & 1) * L::chunk + have * 128;
            for (int u = st; u < per_chunk; u += 128) *reinterpret_cast<uint4*>(row + u * 16) = make_uint4(0, 0, 0, 0);
          }
        }
        fence_async_smem();
        fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[it & 1]);
      }
      // ---- end of the piece: sums over the tokens, then O^T out of tensor memory
#pragma unroll
      for (int c = 0; c < 2 * R; ++c) {
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) sum[c] += __shfl_xor_sync(0xffffffffu, sum[c], d);
      }
      meet();  // red and fac have been read
      if (lane < 4) {
#pragma unroll
        for (int j = 0; j < R; ++j) {
          *reinterpret_cast<float2*>(red + sp * NT + 8 * j + 2 * lane) = make_float2(sum[2 * j], sum[2 * j + 1]);
          if (sp == 0) *reinterpret_cast<float2*>(fac + 8 * j + 2 * lane) = make_float2(mx[2 * j], mx[2 * j + 1]);
        }
      }
      meet();
      const bool whole = walk.t0 == 0 && walk.n == walk.tiles;
      const int slot = 2 * blockIdx.x + (walk.t0 == 0 ? 1 : 0);
      float l = 0.f;
      if (st < NT)
        for (int i = 0; i < 4; ++i) l += red[i * NT + st];
      if (st < ncols) {
        if (whole)
          a.lse[col0 + st] = l == 0.f ? -INFINITY : (fac[st] + log2f(l)) * 0.6931471805599453f;
        else
          a.ml[slot * kLatMaxNT + st] = make_float2(fac[st], l);
      }
      if (!whole && walk.t0 == 0 && st == 0) {
        const long long rest = walk.tiles - walk.n;
        a.meta[blockIdx.x] = {col0, ncols, 1 + (int)((rest + per - 1) / per)};
      }
      meet();
      if (st < NT) fac[st] = !whole ? 1.f : l == 0.f ? 0.f : 1.f / l;
      meet();
      wait(&o_done[(it - 1) & 1], ((it - 1) >> 1) & 1);
      __syncwarp();
      fence_after_sync();
#pragma unroll 1
      for (int c0 = 0; c0 < 4 * NT; c0 += 16) {
        const int cc = c0 % NT;
        float v[16];
        tmem_ld16(la + c0 / NT * W + cc, v);
        if constexpr (W == 2 * NT) {
          float v2[16];
          tmem_ld16(la + c0 / NT * W + NT + cc, v2);
#pragma unroll
          for (int c = 0; c < 16; ++c) v[c] += v2[c];
        }
        const int dim = c0 / NT * 128 + 32 * sp + lane;
        if (whole) {
#pragma unroll
          for (int c = 0; c < 16; ++c)
            if (cc + c < ncols) a.o[((size_t)col0 + cc + c) * kLatDim + dim] = __float2bfloat16_rn(v[c] * fac[cc + c]);
        } else {
#pragma unroll
          for (int c = 0; c < 16; ++c)
            if (cc + c < ncols) a.part[((size_t)slot * kLatMaxNT + cc + c) * kLatDim + dim] = v[c];
        }
      }
      fence_before_sync();
    }
  }
  fence_before_sync();
  __syncthreads();
  if (w == 1) tmem_dealloc(tb, kTmem);
}

// Joins the pieces of every unit that starts in one share and ends in a later one:
//   o = sum_i e^{m_i - m} O_i / sum_i e^{m_i - m} l_i,
// in an order that depends on the number of pieces alone.  Launched while the attention kernel still
// runs (it waits for that grid's end).  Its time is that of a chain of loads, so a thread takes at most
// 4 to 10 pieces, mostly loaded at once, and the CTAs share a list of work items of three kinds:
//   up to 4 pieces (ragged batches, most units): four columns, 128 threads x 4 dimensions each;
//   up to 32 (a few contexts): one column, a group of 128 threads for every fourth piece;
//   more (one context over all CTAs): 128 dimensions of a column, a warp for every 16th piece.
// Whole calls of 8 contexts of 4000 tokens with 64 columns, while single bf16 weights went into 128-token
// tiles: 25.2 us; with up to 8 pieces a thread (one CTA an SM for its registers) 30.4, with the last kind
// for all above 8 pieces 46.  One context of 6000
// tokens: 14 us, and 34 with one CTA per column.
constexpr int kLatCombThreads = 512, kLatCombFew = 4, kLatCombSome = 32;

struct LatJoin {  // running sum of pieces for 4 dimensions of a column
  float4 o;
  __device__ __forceinline__ void add(float e, const float4& x) {
    o.x = fmaf(e, x.x, o.x);
    o.y = fmaf(e, x.y, o.y);
    o.z = fmaf(e, x.z, o.z);
    o.w = fmaf(e, x.w, o.w);
  }
  __device__ __forceinline__ void store(const LatAttnArgs& a, size_t col, int d, float m, float l) const {
    const float inv = l == 0.f ? 0.f : 1.f / l;
    const float v[4] = {o.x * inv, o.y * inv, o.z * inv, o.w * inv};
    store4(a.o + col * kLatDim + d, v);
    if (d == 0) a.lse[col] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
  }
};

__global__ void __launch_bounds__(kLatCombThreads, 2) latent_combine_kernel(LatAttnArgs a, int shares) {
  __shared__ LatPiece unit[kLatMaxCtas];
  __shared__ int ends[kLatMaxCtas];  // items of units 0 .. i
  __shared__ int part_sum[kLatCombThreads / 32];
  __shared__ float f[kLatMaxCtas];
  __shared__ float4 acc_s[kLatCombThreads];
  const int tid = threadIdx.x, w = tid >> 5, lane = tid & 31;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  int cnt = 0;
  if (tid < shares) {
    const LatPiece u = a.meta[tid];
    unit[tid] = u;
    cnt = u.n == 0 ? 0 : u.n <= kLatCombFew ? (u.ncols + 3) / 4 : u.n <= kLatCombSome ? u.ncols : 4 * u.ncols;
  }
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, cnt, d);
    if (lane >= d) cnt += y;
  }
  if (lane == 31) part_sum[w] = cnt;
  __syncthreads();
  for (int i = 0; i < w; ++i) cnt += part_sum[i];
  if (tid < shares) ends[tid] = cnt;
  __syncthreads();
  const int items = ends[shares - 1];
  for (int item = blockIdx.x; item < items; item += gridDim.x) {
    int s = 0;  // the unit: as many as end at or before the item
    for (int i = lane; i < kLatMaxCtas; i += 32) s += i < shares && ends[i] <= item;
    s = __reduce_add_sync(0xffffffffu, s);
    const LatPiece u = unit[s];
    const int k = item - (s ? ends[s - 1] : 0);
    auto slot = [&](int i) { return (size_t)(i == 0 ? 2 * s + 1 : 2 * (s + i)) * kLatMaxNT; };
    LatJoin join{make_float4(0.f, 0.f, 0.f, 0.f)};
    if (u.n <= kLatCombFew) {
      const int c = 4 * k + (tid >> 7), d = 4 * (tid & 127);
      if (c >= u.ncols) continue;
      float m = -INFINITY, l = 0.f;
      float2 ml[kLatCombFew];
      float4 x[kLatCombFew];
#pragma unroll
      for (int i = 0; i < kLatCombFew; ++i)
        if (i < u.n) {
          ml[i] = a.ml[slot(i) + c];
          x[i] = *reinterpret_cast<const float4*>(a.part + (slot(i) + c) * kLatDim + d);
          m = fmaxf(m, ml[i].x);
        }
      if (m == -INFINITY) m = 0.f;  // no token is visible: every piece's sums are 0
#pragma unroll
      for (int i = 0; i < kLatCombFew; ++i)
        if (i < u.n) {
          const float e = tc::ex2(ml[i].x - m);
          l = fmaf(e, ml[i].y, l);
          join.add(e, x[i]);
        }
      join.store(a, (size_t)u.col0 + c, d, m, l);
      continue;
    }
    // G groups of threads, group g takes pieces g, g + G, ...; d: the thread's dimensions
    const bool some = u.n <= kLatCombSome;
    const int c = some ? k : k >> 2, d = some ? 4 * (tid & 127) : 128 * (k & 3) + 4 * lane;
    const int G = some ? kLatCombThreads / 128 : kLatCombThreads / 32, g = some ? tid >> 7 : w;
    float m = -INFINITY, l = 0.f;
    for (int i = lane; i < u.n; i += 32) m = fmaxf(m, a.ml[slot(i) + c].x);
#pragma unroll
    for (int e = 16; e; e >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, e));
    if (m == -INFINITY) m = 0.f;
    for (int i = lane; i < u.n; i += 32) {
      const float2 ml = a.ml[slot(i) + c];
      const float e = tc::ex2(ml.x - m);
      if (w == 0) f[i] = e;
      l = fmaf(e, ml.y, l);
    }
#pragma unroll
    for (int e = 16; e; e >>= 1) l += __shfl_xor_sync(0xffffffffu, l, e);
    __syncthreads();
#pragma unroll 5
    for (int i = g; i < u.n; i += G)
      join.add(f[i], *reinterpret_cast<const float4*>(a.part + (slot(i) + c) * kLatDim + d));
    acc_s[tid] = join.o;
    __syncthreads();
    if (g == 0) {
      const int step = kLatCombThreads / G;
#pragma unroll 3
      for (int i = 1; i < G; ++i) join.add(1.f, acc_s[step * i + tid]);
      join.store(a, (size_t)u.col0 + c, d, m, l);
    }
    __syncthreads();  // f and acc_s are free again
  }
}

// ------------------------------------------------------------------------------------ per-head products
// The absorbed queries qa[t][h][l] = sum_i q[t][h][i] W_k[h][i][l] (K = 128, 512 outputs) and their rotary
// part.  Bound by writing qa (the weights and q are read from L2 after their first use).  The work is one
// list of blocks (128 rows, head, 128 outputs), outputs fastest, and a CTA takes `blocks` consecutive ones:
// the rows stay in shared memory while their four output blocks go by, the weights (stored [i][l],
// MN-major) follow in steps of 64 i, and two accumulators alternate, so that rounding and writing a block
// overlaps the loads and MMAs of the next one.  Two CTAs share an SM, one block each while that is
// all there is.  The rotary parts of all rows are spread over the CTAs' writing warps, between blocks.
// 4096 rows of 16 heads: 24.5 us (4.2 TB/s; without the stores 11.6, without the rotary parts 20.8); every
// CTA a tile of its own 26.6 (four output blocks) and 37.8 us (one); one CTA an SM with its head's weights
// resident and sixteen writing warps 28.0 us: the chains of loads of a single CTA are not hidden.
constexpr int kAbsorbThreads = 320;  // producer warp, MMA warp, eight writing warps
constexpr int kAbsorbPerSm = 2;

struct AbsorbSmem {
  static constexpr int w_slots = 3;
  static constexpr uint32_t x = 2 * 128 * 128, w = 64 * 256, out_ld = 32 * 2 + 16;
  static constexpr uint32_t out = x + w_slots * w, total = out + 8 * 32 * out_ld + 1024;  // + slack to align the tiles
};

struct AbsorbArgs {
  DecodeRows rows;
  int H;
  const __nv_bfloat16* q;
  int64_t ld_q;
  __nv_bfloat16* qa;
  int* status;
  uint64_t wait_ns;
  int64_t total;  // blocks in all, and of one CTA
  int blocks;
};

__global__ void __launch_bounds__(kAbsorbThreads, kAbsorbPerSm)
    latent_absorb_tc(const __grid_constant__ CUtensorMap tma_x, const __grid_constant__ CUtensorMap tma_w, AbsorbArgs a) {
  using namespace tc;
  using L = AbsorbSmem;
  extern __shared__ __align__(1024) uint8_t hsm_raw[];
  uint8_t* sm = hsm_raw + ((1024u - (smem_u32(hsm_raw) & 1023u)) & 1023u);
  __shared__ __align__(8) uint64_t x_full, x_empty, w_full[L::w_slots], w_empty[L::w_slots], acc_full[2], acc_empty[2], done;
  __shared__ uint32_t tslot;
  __shared__ int sound;  // 0: a sequence's rows are not within 0 .. n_rows
  const int tid = threadIdx.x, w = tid >> 5, lane = tid & 31;
  constexpr int kOut = kLatDim / 128;  // output blocks of a (rows, head) pair
  const int64_t first = (int64_t)blockIdx.x * a.blocks;
  const int count = (int)min((int64_t)a.blocks, a.total - first);
  struct Block {
    int h, t0, n0;
    bool fresh;  // its rows are not those of the CTA's block before it
  };
  auto block = [&](int j) -> Block {
    const int g = (int)(first + j), pair = g / kOut;
    return {pair % a.H, pair / a.H * 128, g % kOut * 128, j == 0 || g % kOut == 0};
  };
  if (tid == 0) {
    sound = 1;
    prefetch_tensor_map(&tma_x);
    prefetch_tensor_map(&tma_w);
    for (int i = 0; i < L::w_slots; ++i) {
      mbar_init(&w_full[i], 1);
      mbar_init(&w_empty[i], 1);
    }
    mbar_init(&x_full, 1);
    mbar_init(&x_empty, 1);
    mbar_init(&done, 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&acc_full[i], 1);
      mbar_init(&acc_empty[i], 8);
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (w == 1) tmem_alloc(&tslot, 256);
  fence_before_sync();
  __syncthreads();
  fence_after_sync();
  const uint32_t tb = tslot;
  // every wait is bounded; a role whose wait ran out records it and stops
  auto wait = [&](uint64_t* bar, uint32_t parity) -> bool {
    if (mbar_wait_limit(bar, parity, a.wait_ns)) return true;
    set_status(a.status, 8);
    return false;
  };
  if (w == 0) {
    if (lane == 0) {
      int item = 0, xs = 0;  // weight steps and row tiles issued
      bool ok = true;
      for (int j = 0; j < count && ok; ++j) {
        const Block b = block(j);
        if (b.fresh) {
          ok = xs == 0 || wait(&x_empty, (xs - 1) & 1);
          if (!ok) break;
          mbar_arrive_expect_tx(&x_full, L::x);
          tma_load_3d(sm, &tma_x, 0, b.h, b.t0, &x_full);
          tma_load_3d(sm + L::x / 2, &tma_x, 64, b.h, b.t0, &x_full);
          ++xs;
        }
        for (int kc = 0; kc < 2; ++kc, ++item) {
          const int st = item % L::w_slots;
          ok = item < L::w_slots || wait(&w_empty[st], (item / L::w_slots - 1) & 1);
          if (!ok) break;
          uint8_t* ws = sm + L::x + st * L::w;
          mbar_arrive_expect_tx(&w_full[st], L::w);
          tma_load_2d(ws, &tma_w, b.n0, b.h * kLatHead + 64 * kc, &w_full[st]);
          tma_load_2d(ws + L::w / 2, &tma_w, b.n0 + 64, b.h * kLatHead + 64 * kc, &w_full[st]);
        }
      }
      // every copy lands before the CTA ends, whoever gave up (at once if no one did)
      for (int i = max(0, item - L::w_slots); i < item; ++i) mbar_wait(&w_full[i % L::w_slots], (i / L::w_slots) & 1, kWayOutNs);
      if (xs) mbar_wait(&x_full, (xs - 1) & 1, kWayOutNs);
    }
  } else if (w == 1) {
    const uint32_t lead = elect_one();
    constexpr uint32_t id = idesc_bf16(128, 128, false, true);
    bool ok = true;
    int st = 0, parity = 0, xs = 0, j = 0;
    for (; j < count; ++j) {
      const bool fresh = j == 0 || (first + j) % kOut == 0, leaves = j + 1 == count || (first + j + 1) % kOut == 0;
      if (fresh) ok = __all_sync(0xffffffffu, wait(&x_full, xs++ & 1));
      if (ok && j >= 2) ok = __all_sync(0xffffffffu, wait(&acc_empty[j & 1], ((j >> 1) - 1) & 1));
      const uint32_t acc = tb + (j & 1) * 128;
#pragma unroll
      for (int kc = 0; kc < 2; ++kc) {
        ok = ok && __all_sync(0xffffffffu, wait(&w_full[st], parity));
        if (!ok) break;
        fence_after_sync();
        const uint32_t x = smem_u32(sm) + kc * (L::x / 2), ws = smem_u32(sm) + L::x + st * L::w;
#pragma unroll
        for (int ks = 0; ks < 4; ++ks)
          mma_bf16_if(lead, acc, sw_desc_k(x, 128, ks), sw_desc_mn(ws, 64, ks), id, kc || ks ? 1u : 0u);
        commit_if(lead, &w_empty[st]);
        if (++st == L::w_slots) {
          st = 0;
          parity ^= 1;
        }
      }
      if (!ok) break;
      commit_if(lead, &acc_full[j & 1]);
      if (leaves) commit_if(lead, &x_empty);
    }
    commit_if(lead, &done);  // the MMAs are complete before TMEM is freed, whoever gave up
    if (!mbar_wait(&done, 0, kWayOutNs)) set_status(a.status, 8);
    __syncwarp();
  } else {
    const int sp = w & 3;
    int row0 = 0, row1 = a.rows.n_rows;  // rows that belong to a sequence, if the table is sound
    bool all_sound = true;
    if (a.rows.row_start) {
      row0 = a.rows.row_start[0];
      row1 = min(row1, a.rows.row_start[a.rows.n_seqs]);
      // the writing warps look through the table together, while the first copies and MMAs run
      if (bad_row_starts(a.rows, tid - 64, kAbsorbThreads - 64)) sound = 0;
      asm volatile("bar.sync 1, %0;" ::"n"(kAbsorbThreads - 64) : "memory");
      all_sound = sound != 0;
      if (!all_sound && lane == 0) set_status(a.status, kStatusCheck);
    }
    // this CTA's share of the rotary parts: a row per warp and block, while copies and MMAs run
    int64_t rope = (int64_t)a.rows.n_rows * blockIdx.x / gridDim.x + w - 2;
    const int64_t rope_end = (int64_t)a.rows.n_rows * (blockIdx.x + 1) / gridDim.x;
    auto turn = [&] {
      absorb_rope_row(a.rows, a.H, a.q, a.ld_q, a.qa, (int)rope);
      rope += 8;
    };
    // rows 32 sp .. of the tile, one half of a block's columns in steps of 32
    uint8_t* out = sm + L::out + 32 * (w - 2) * L::out_ld;
    const int half = 64 * ((w - 2) >> 2);
    for (int j = 0; j < count; ++j) {
      if (rope < rope_end) turn();
      const Block b = block(j);
      if (!__all_sync(0xffffffffu, wait(&acc_full[j & 1], (j >> 1) & 1))) break;
      fence_after_sync();
      const int mine = b.t0 + 32 * sp + lane;  // rows of this warp that belong to a sequence
      uint32_t owned = __ballot_sync(0xffffffffu, mine >= row0 && mine < row1);
      if (!all_sound) {
        owned = 0;
        for (int i = 0; i < 32 && b.t0 + 32 * sp + i < a.rows.n_rows; ++i)
          if (row_at(a.rows, b.t0 + 32 * sp + i).seq >= 0) owned |= 1u << i;
      }
#pragma unroll
      for (int c0 = half; c0 < half + 64; c0 += 32) {
        uint32_t r[32];
        tmem_ld32_nowait(tb + ((uint32_t)(32 * sp) << 16) + (j & 1) * 128 + c0, r);
        tmem_wait_ld();
#pragma unroll
        for (int i = 0; i < 32; ++i) asm volatile("" : "+r"(r[i]));
        round_to_smem(r, out + lane * L::out_ld);
        __syncwarp();
#pragma unroll
        for (int i = lane >> 2; i < 32; i += 8) {
          const int t = b.t0 + 32 * sp + i;
          if (owned >> i & 1)
            *reinterpret_cast<uint4*>(a.qa + ((size_t)t * a.H + b.h) * kLatWidth + b.n0 + c0 + (lane & 3) * 8) =
                *reinterpret_cast<const uint4*>(out + i * L::out_ld + (lane & 3) * 16);
        }
        __syncwarp();
      }
      fence_before_sync();
      if (lane == 0) mbar_arrive(&acc_empty[j & 1]);
    }
    while (rope < rope_end) turn();
  }
  __syncthreads();
  if (w == 1) tmem_dealloc(tb, 256);
}

// The head outputs out[t][h][i] = sum_l W_v[h][i][l] o[t][h][l] (K = 512, 128 outputs), one CTA per 128 rows,
// head and BN outputs.  Bound by reading o.  K steps of 64 through three stages (both operands K-major),
// M = 128 MMAs, the outputs written in whole row pieces through the stages' memory.  Two CTAs share an SM
// and hide one another's epilogue (2047 rows of 32 heads: 14.6 us, 6.0 TB/s, inputs partly in L2; 20.5 us
// from memory.  Equal shares of consecutive tiles with two accumulators a CTA: 14.3 and 20.7 us).  A few
// rows are a chain of fetching a head's weights, which BN = 32 cuts to a quarter (96
// rows of 16 heads 4.2 against 5.3 us, 500 rows 5.5 against 5.6; 96 rows of 128 heads 8.5 against 5.6 us).
constexpr int kExpandThreads = 192;
template <int BN>
struct ExpandSmem {
  static constexpr int stages = 3, steps = kLatDim / 64;
  static constexpr uint32_t x = 128 * 128, stage = x + BN * 128, out_ld = BN * 2 + 16;
  static constexpr uint32_t total = stages * stage + 1024;  // + slack to align the stages
  static_assert(128 * out_ld <= stages * stage, "the output tile takes the stages' place");
};

struct ExpandArgs {
  int H, n_rows;
  __nv_bfloat16* out;
  int* status;
  uint64_t wait_ns;
};

template <int BN>
__global__ void __launch_bounds__(kExpandThreads)
    latent_expand_tc(const __grid_constant__ CUtensorMap tma_x, const __grid_constant__ CUtensorMap tma_w, ExpandArgs a) {
  using namespace tc;
  using L = ExpandSmem<BN>;
  extern __shared__ __align__(1024) uint8_t hsm_raw[];
  uint8_t* sm = hsm_raw + ((1024u - (smem_u32(hsm_raw) & 1023u)) & 1023u);
  __shared__ __align__(8) uint64_t full[L::stages], empty[L::stages], acc_full, done;
  __shared__ uint32_t tslot;
  const int tid = threadIdx.x, w = tid >> 5, lane = tid & 31;
  const int n0 = (int)(blockIdx.x % (kLatHead / BN)) * BN, pair = (int)(blockIdx.x / (kLatHead / BN));
  const int h = pair % a.H, t0 = pair / a.H * 128;
  if (tid == 0) {
    prefetch_tensor_map(&tma_x);
    prefetch_tensor_map(&tma_w);
    for (int i = 0; i < L::stages; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    mbar_init(&acc_full, 1);
    mbar_init(&done, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (w == 1) tmem_alloc(&tslot, BN);
  fence_before_sync();
  __syncthreads();
  fence_after_sync();
  const uint32_t tb = tslot;
  // every wait is bounded; a role whose wait ran out records it and stops
  auto wait = [&](uint64_t* bar, uint32_t parity) -> bool {
    if (mbar_wait_limit(bar, parity, a.wait_ns)) return true;
    set_status(a.status, 8);
    return false;
  };
  if (w == 0) {
    if (lane == 0) {
      int issued = 0;
      for (; issued < L::steps; ++issued) {
        const int st = issued % L::stages, k0 = 64 * issued;
        if (issued >= L::stages && !wait(&empty[st], (issued / L::stages - 1) & 1)) break;
        uint8_t* xs = sm + st * L::stage;
        mbar_arrive_expect_tx(&full[st], L::stage);
        tma_load_3d(xs, &tma_x, k0, h, t0, &full[st]);
        tma_load_2d(xs + L::x, &tma_w, k0, (a.H + h) * kLatHead + n0, &full[st]);
      }
      // every copy lands before the CTA ends, whoever gave up (at once if no one did)
      for (int i = max(0, issued - L::stages); i < issued; ++i) mbar_wait(&full[i % L::stages], (i / L::stages) & 1, kWayOutNs);
    }
  } else if (w == 1) {
    const uint32_t lead = elect_one();
    constexpr uint32_t id = idesc_bf16(128, BN, false, false);
    bool ok = true;
#pragma unroll
    for (int i = 0; i < L::steps; ++i) {
      const int st = i % L::stages;
      ok = ok && __all_sync(0xffffffffu, wait(&full[st], (i / L::stages) & 1));
      if (!ok) break;
      fence_after_sync();
      const uint32_t xs = smem_u32(sm) + st * L::stage;
#pragma unroll
      for (int ks = 0; ks < 4; ++ks) mma_bf16_if(lead, tb, sw_desc_k(xs, 128, ks), sw_desc_k(xs + L::x, BN, ks), id, i || ks ? 1u : 0u);
      commit_if(lead, &empty[st]);
    }
    if (ok) commit_if(lead, &acc_full);  // (otherwise the accumulator is not whole)
    commit_if(lead, &done);              // the MMAs are complete before TMEM is freed, whoever gave up
    if (!mbar_wait(&done, 0, kWayOutNs)) set_status(a.status, 8);
    __syncwarp();
  } else {
    const int sp = w & 3;
    const bool got = __all_sync(0xffffffffu, wait(&acc_full, 0));
    fence_after_sync();
    uint8_t* out = sm + 32 * sp * L::out_ld;  // this warp's rows; every copy has landed and been read
    if (got) {
#pragma unroll
      for (int c0 = 0; c0 < BN; c0 += 32) {
        uint32_t r[32];
        tmem_ld32_nowait(tb + ((uint32_t)(32 * sp) << 16) + c0, r);
        tmem_wait_ld();
#pragma unroll
        for (int i = 0; i < 32; ++i) asm volatile("" : "+r"(r[i]));
        round_to_smem(r, out + lane * L::out_ld + c0 * 2);
      }
      __syncwarp();
      constexpr int lanes = BN / 8;  // of a row piece
#pragma unroll 4
      for (int i = lane / lanes; i < 32; i += 32 / lanes) {
        const int t = t0 + 32 * sp + i;
        if (t < a.n_rows)
          *reinterpret_cast<uint4*>(a.out + ((size_t)t * a.H + h) * kLatHead + n0 + lane % lanes * 8) =
              *reinterpret_cast<const uint4*>(out + i * L::out_ld + lane % lanes * 16);
      }
    }
    fence_before_sync();
  }
  __syncthreads();
  if (w == 1) tmem_dealloc(tb, BN);
}

}  // namespace tpc
