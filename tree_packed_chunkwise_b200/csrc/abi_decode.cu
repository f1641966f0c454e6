// C ABI of the tree-packed chunkwise KDA library: token-by-token generation (recurrent KDA step,
// paged latent cache, absorbed latent attention).  Declarations and contracts in include/tpc.h.
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <string>

#include "../../include/tpc.h"
#include "abi_internal.h"
#include "decode_kernels.cuh"
#include "latent_tc.cuh"

namespace {
using tpc_abi::fail;
using tpc_abi::g_prof;
using tpc_abi::set_smem;
using tpc_abi::tensor_map;
using tpc_abi::tensor_map_rows;
using tpc_abi::tensor_map_rows_ld;
using bf = __nv_bfloat16;

static_assert(TPC_LATENT_DIM == tpc::kLatDim && TPC_LATENT_ROPE == tpc::kLatRope && TPC_LATENT_HEAD == tpc::kLatHead &&
                  TPC_LATENT_WIDTH == tpc::kLatWidth,
              "cache layout");

constexpr int kLatMaxH = 128;

std::atomic<int64_t> g_wait_ns{2000000000};  // limit of the tensor-core kernels' waits

bool misaligned(const void* p, size_t to = 16) { return reinterpret_cast<uintptr_t>(p) % to != 0; }

int rows_check(const char* call, const tpc_rows* r, bool kv, tpc::DecodeRows* out) {
  if (!r) return fail(TPC_ERR_NULL, std::string(call) + ": rows is NULL");
  if (r->n_rows < 0 || r->n_seqs < 0) return fail(TPC_ERR_BAD_SHAPE, std::string(call) + ": negative n_rows or n_seqs");
  if (!r->row_start && r->n_rows != r->n_seqs)
    return fail(TPC_ERR_BAD_SHAPE, std::string(call) + ": without row_start n_rows must equal n_seqs");
  if (kv && r->n_seqs > 0 && !r->kv_len) return fail(TPC_ERR_NULL, std::string(call) + ": kv_len is NULL");
  *out = {r->n_rows, r->n_seqs, r->row_start, r->kv_len};
  return TPC_OK;
}

// (a batch without a row or a sequence reads no table)
int cache_check(const char* call, const tpc_latent_cache* c, bool empty, tpc::LatentCache* out) {
  if (!c || !c->data || (!empty && !c->block_table))
    return fail(TPC_ERR_NULL, std::string(call) + ": cache, its data or its block table is NULL");
  if (c->n_pages < 1 || c->max_pages < (empty ? 0 : 1))
    return fail(TPC_ERR_BAD_SHAPE, std::string(call) + ": n_pages and max_pages must be >= 1");
  if (!(c->page_size == 16 || c->page_size == 32 || (c->page_size >= 64 && c->page_size % 64 == 0)))
    return fail(TPC_ERR_UNSUPPORTED, std::string(call) + ": page_size must be 16, 32 or a multiple of 64");
  // (room for a tile past the end)
  if (std::max(c->n_pages, c->max_pages) > (INT32_MAX - 256) / c->page_size)
    return fail(TPC_ERR_BAD_SHAPE, std::string(call) + ": more than 2^31 - 257 cached tokens");
  if (misaligned(c->data)) return fail(TPC_ERR_BAD_SHAPE, std::string(call) + ": the cache must be 16-byte aligned");
  *out = {(bf*)c->data, c->n_pages, c->page_size, c->block_table, c->max_pages};
  return TPC_OK;
}

int heads_check(const char* call, int32_t H, int64_t n_rows) {
  if (H < 1 || H > kLatMaxH) return fail(TPC_ERR_UNSUPPORTED, std::string(call) + ": 1 <= H <= 128");
  // (room for a column tile past the end)
  if (n_rows * H > INT32_MAX - 256) return fail(TPC_ERR_BAD_SHAPE, std::string(call) + ": more than 2^31 - 257 (row, head) pairs");
  return TPC_OK;
}
}  // namespace

extern "C" {

int tpc_kda_step(const tpc_kda_shape* shape, const tpc_rows* rows, const tpc_kda_step_io* io, int32_t* status,
                 tpc_stream_t stream) {
  if (!shape || !io) return fail(TPC_ERR_NULL, "kda step: shape or io is NULL");
  tpc::DecodeRows r;
  if (int rc = rows_check("kda step", rows, false, &r)) return rc;
  if (shape->H < 1 || shape->dk != shape->dv) return fail(TPC_ERR_BAD_SHAPE, "kda step: H >= 1 and dk == dv");
  if (shape->dk != 32 && shape->dk != 64 && shape->dk != 128) return fail(TPC_ERR_UNSUPPORTED, "kda step: head size 32, 64 or 128");
  if ((shape->in_dtype != TPC_F32 && shape->in_dtype != TPC_BF16) || (shape->out_dtype != TPC_F32 && shape->out_dtype != TPC_BF16))
    return fail(TPC_ERR_UNSUPPORTED, "kda step: dtypes are TPC_F32 or TPC_BF16");
  if (io->n_slots < 1) return fail(TPC_ERR_BAD_SHAPE, "kda step: n_slots must be >= 1");
  if (r.n_seqs == 0) return TPC_OK;
  if (!io->src || !io->state) return fail(TPC_ERR_NULL, "kda step: state or src is NULL");
  if (r.n_rows > 0 && (!io->q || !io->k || !io->v || !io->g || !io->beta || !io->o))
    return fail(TPC_ERR_NULL, "kda step: NULL tensor");
  for (const void* p : {io->q, io->k, io->v, io->g, (const void*)io->state, (const void*)io->o})
    if (misaligned(p)) return fail(TPC_ERR_BAD_SHAPE, "kda step: tensors must be 16-byte aligned");
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const tpc::StepArgs a{io->q, io->k, io->v, io->g, io->beta, io->state, io->src, io->dst, io->o, io->n_slots, shape->H, r, status};
  constexpr int per = tpc::kStepThreads / 32;
  if ((int64_t)r.n_seqs * shape->H > INT32_MAX / per) return fail(TPC_ERR_BAD_SHAPE, "kda step: too many sequences and heads");
  tpc_abi::NvtxRange nvtx_call("tpc_kda_step");
  auto go = [&](auto tin, auto tout, auto d) -> int {
    using T = decltype(tin);
    using TO = decltype(tout);
    constexpr int D = decltype(d)::value;
    const int64_t warps = (int64_t)r.n_seqs * shape->H * tpc::StepShape<D>::warps;
    TPC_LAUNCH("kda_step", st,
               (tpc::kda_step_kernel<T, TO, D><<<(unsigned)((warps + per - 1) / per), tpc::kStepThreads, 0, st>>>(a)));
    return TPC_OK;
  };
  auto with_d = [&](auto tin, auto tout) -> int {
    if (shape->dk == 128) return go(tin, tout, std::integral_constant<int, 128>{});
    if (shape->dk == 64) return go(tin, tout, std::integral_constant<int, 64>{});
    return go(tin, tout, std::integral_constant<int, 32>{});
  };
  if (shape->in_dtype == TPC_BF16) return shape->out_dtype == TPC_BF16 ? with_d(bf{}, bf{}) : with_d(bf{}, float{});
  return shape->out_dtype == TPC_BF16 ? with_d(float{}, bf{}) : with_d(float{}, float{});
}

int tpc_latent_append(const tpc_latent_cache* cache, const tpc_rows* rows, const void* c, int64_t ld_c, const void* kr,
                      int64_t ld_kr, int32_t in_dtype, int32_t* status, tpc_stream_t stream) {
  tpc::LatentCache lc;
  tpc::DecodeRows r;
  if (int rc = rows_check("latent append", rows, true, &r)) return rc;
  const bool empty = r.n_rows == 0 || r.n_seqs == 0;
  if (int rc = cache_check("latent append", cache, empty, &lc)) return rc;
  if (in_dtype != TPC_F32 && in_dtype != TPC_BF16) return fail(TPC_ERR_UNSUPPORTED, "latent append: in_dtype is TPC_F32 or TPC_BF16");
  if (empty) return TPC_OK;
  if (!c || !kr) return fail(TPC_ERR_NULL, "latent append: NULL tensor");
  const int unit = in_dtype == TPC_BF16 ? 8 : 4;
  if (ld_c < tpc::kLatDim || ld_kr < tpc::kLatRope || ld_c % unit || ld_kr % unit || misaligned(c) || misaligned(kr))
    return fail(TPC_ERR_BAD_SHAPE, "latent append: rows of 512 and 64 elements, 16-byte aligned, leading dimensions multiples of 16 bytes");
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  tpc_abi::NvtxRange nvtx_call("tpc_latent_append");
  const tpc::AppendArgs a{lc, r, c, kr, ld_c, ld_kr, status};
  constexpr int per = tpc::kAppendThreads / 32;
  const unsigned grid = (unsigned)(((int64_t)r.n_rows + per - 1) / per);
  auto go = [&](auto tin, auto check) -> int {
    TPC_LAUNCH("latent_append", st,
               (tpc::latent_append_kernel<decltype(tin), decltype(check)::value><<<grid, tpc::kAppendThreads, 0, st>>>(a)));
    return TPC_OK;
  };
  auto with_check = [&](auto tin) { return status ? go(tin, std::true_type{}) : go(tin, std::false_type{}); };
  return in_dtype == TPC_BF16 ? with_check(bf{}) : with_check(float{});
}

int tpc_latent_absorb(const tpc_rows* rows, int32_t H, const void* q, int64_t ld_q, const void* w_b, void* qa,
                      int32_t* status, tpc_stream_t stream) {
  tpc::DecodeRows r;
  if (int rc = rows_check("latent absorb", rows, true, &r)) return rc;
  if (int rc = heads_check("latent absorb", H, r.n_rows)) return rc;
  if (r.n_rows == 0 || r.n_seqs == 0) return TPC_OK;
  if (!q || !w_b || !qa) return fail(TPC_ERR_NULL, "latent absorb: NULL tensor");
  if (ld_q < (int64_t)H * tpc::kLatQK || ld_q % 8 || misaligned(q) || misaligned(w_b) || misaligned(qa))
    return fail(TPC_ERR_BAD_SHAPE, "latent absorb: 16-byte aligned tensors, ld_q >= 192 H and a multiple of 8");
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  tpc_abi::NvtxRange nvtx_call("tpc_latent_absorb");
  CUtensorMap tx, tw;
  if (!tensor_map_rows_ld(&tx, q, tpc::kLatQK, H, r.n_rows, ld_q, 128) ||
      !tensor_map(&tw, w_b, tpc::kLatDim, (uint64_t)2 * tpc::kLatHead * H, tpc::kLatDim, 64))
    return fail(TPC_ERR_CUDA, "latent absorb: cuTensorMapEncodeTiled failed");
  const int64_t total = (int64_t)((r.n_rows + 127) / 128) * H * (tpc::kLatDim / 128);
  const int64_t slots = (int64_t)tpc::kAbsorbPerSm * tpc_abi::sm_count(), blocks = (total + slots - 1) / slots;
  const int64_t grid = (total + blocks - 1) / blocks;
  const tpc::AbsorbArgs a{r, H, (const bf*)q, ld_q, (bf*)qa, status, (uint64_t)g_wait_ns, total, (int)blocks};
  constexpr size_t smem = tpc::AbsorbSmem::total;
  TPC_CUDA(set_smem(tpc::latent_absorb_tc, smem));
  TPC_LAUNCH("latent_absorb_tc", st, (tpc::latent_absorb_tc<<<(unsigned)grid, tpc::kAbsorbThreads, smem, st>>>(tx, tw, a)));
  return TPC_OK;
}

size_t tpc_latent_attn_scratch_bytes(int32_t H) { return H < 1 || H > kLatMaxH ? 0 : tpc::kLatScratch; }

int tpc_latent_attn(const tpc_latent_cache* cache, const tpc_rows* rows, int32_t H, float scale, const void* qa,
                    void* o, float* lse, void* scratch, size_t scratch_bytes, int32_t* status, tpc_stream_t stream) {
  tpc::LatentCache lc;
  tpc::DecodeRows r;
  if (int rc = rows_check("latent attention", rows, true, &r)) return rc;
  const bool empty = r.n_rows == 0 || r.n_seqs == 0;
  if (int rc = cache_check("latent attention", cache, empty, &lc)) return rc;
  if (int rc = heads_check("latent attention", H, r.n_rows)) return rc;
  if (empty) return TPC_OK;
  if (!qa || !o || !lse || !scratch) return fail(TPC_ERR_NULL, "latent attention: NULL tensor");
  if (misaligned(qa) || misaligned(o)) return fail(TPC_ERR_BAD_SHAPE, "latent attention: qa and o must be 16-byte aligned");
  if (scratch_bytes < tpc_latent_attn_scratch_bytes(H) || misaligned(scratch, 256))
    return fail(TPC_ERR_WORKSPACE, "latent attention: scratch too small or not 256-byte aligned");
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  tpc_abi::NvtxRange nvtx_call("tpc_latent_attn");
  CUtensorMap tkv, tq;
  // columns of a tile: the (row, head) pairs that an average sequence has (times at the kernel)
  const int64_t cols = ((int64_t)r.n_rows * H + r.n_seqs - 1) / r.n_seqs;
  const int NT = cols <= 16 ? 16 : cols <= 32 ? 32 : 64;
  if (!tensor_map(&tkv, lc.data, tpc::kLatWidth, (uint64_t)lc.n_pages * lc.page_size, tpc::kLatWidth, std::min(lc.page_size, tpc::kLatBox)) ||
      !tensor_map(&tq, qa, tpc::kLatWidth, (uint64_t)r.n_rows * H, tpc::kLatWidth, NT))
    return fail(TPC_ERR_CUDA, "latent attention: cuTensorMapEncodeTiled failed");
  char* sc = static_cast<char*>(scratch);
  const tpc::LatAttnArgs a{lc, r, H, scale * 1.4426950408889634f, (bf*)o, lse, (float*)sc, (float2*)(sc + tpc::kLatPartBytes),
                           (tpc::LatPiece*)(sc + tpc::kLatPartBytes + tpc::kLatMlBytes), status, (uint64_t)g_wait_ns};
  const int grid = std::min(tpc_abi::sm_count(), tpc::kLatMaxCtas);
  auto go = [&](auto nt) -> int {
    constexpr int N = decltype(nt)::value;
    constexpr size_t smem = tpc::LatSmem<N>::total;
    TPC_CUDA(set_smem(tpc::latent_attn_tc<N>, smem));
    TPC_LAUNCH("latent_attn_tc", st, (tpc::latent_attn_tc<N><<<grid, tpc::kLatAttnThreads, smem, st>>>(tkv, tq, a)));
    // contexts of one tile are never cut into pieces
    if ((int64_t)lc.max_pages * lc.page_size <= tpc::LatSmem<N>::KT) return TPC_OK;
    cudaLaunchAttribute early{};
    early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    early.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(2 * grid);
    cfg.blockDim = dim3(tpc::kLatCombThreads);
    cfg.stream = st;
    cfg.attrs = &early;
    cfg.numAttrs = 1;
    TPC_LAUNCH("latent_combine", st, TPC_CUDA(cudaLaunchKernelEx(&cfg, tpc::latent_combine_kernel, a, grid)));
    return TPC_OK;
  };
  if (NT == 16) return go(std::integral_constant<int, 16>{});
  if (NT == 32) return go(std::integral_constant<int, 32>{});
  return go(std::integral_constant<int, 64>{});
}

int tpc_latent_expand(int32_t n_rows, int32_t H, const void* o, const void* w_b, void* out, int32_t* status,
                      tpc_stream_t stream) {
  if (n_rows < 0) return fail(TPC_ERR_BAD_SHAPE, "latent expand: negative n_rows");
  if (int rc = heads_check("latent expand", H, n_rows)) return rc;
  if (n_rows == 0) return TPC_OK;
  if (!o || !w_b || !out) return fail(TPC_ERR_NULL, "latent expand: NULL tensor");
  if (misaligned(o) || misaligned(w_b) || misaligned(out)) return fail(TPC_ERR_BAD_SHAPE, "latent expand: tensors must be 16-byte aligned");
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  tpc_abi::NvtxRange nvtx_call("tpc_latent_expand");
  const tpc::ExpandArgs a{H, n_rows, (bf*)out, status, (uint64_t)g_wait_ns};
  const int64_t pairs = (int64_t)((n_rows + 127) / 128) * H;
  auto go = [&](auto bn) -> int {
    constexpr int BN = decltype(bn)::value;
    CUtensorMap tx, tw;
    if (!tensor_map_rows(&tx, o, tpc::kLatDim, H, n_rows, 128) ||
        !tensor_map(&tw, w_b, tpc::kLatDim, (uint64_t)2 * tpc::kLatHead * H, tpc::kLatDim, BN))
      return fail(TPC_ERR_CUDA, "latent expand: cuTensorMapEncodeTiled failed");
    const unsigned grid = (unsigned)(pairs * (tpc::kLatHead / BN));
    constexpr size_t smem = tpc::ExpandSmem<BN>::total;
    TPC_CUDA(set_smem(tpc::latent_expand_tc<BN>, smem));
    TPC_LAUNCH("latent_expand_tc", st, (tpc::latent_expand_tc<BN><<<grid, tpc::kExpandThreads, smem, st>>>(tx, tw, a)));
    return TPC_OK;
  };
  // narrow output blocks while their CTAs fit the SMs twice (both sides at the kernel)
  if (pairs * (tpc::kLatHead / 32) <= 2 * tpc_abi::sm_count()) return go(std::integral_constant<int, 32>{});
  return go(std::integral_constant<int, 128>{});
}

int64_t tpc_debug_wait_limit(int64_t ns) { return ns < 0 ? g_wait_ns.load() : g_wait_ns.exchange(std::min<int64_t>(ns, 2000000000)); }

}  // extern "C"
