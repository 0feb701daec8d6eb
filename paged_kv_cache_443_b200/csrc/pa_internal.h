// pa_internal.h -- declarations shared by the library's translation units
// (host side only; nothing here is part of the public ABI).
#pragma once

#include <cstddef>
#include <cstdint>
#include <utility>

#include <cuda_runtime.h>

#include "pagedkv.h"

namespace pa {

// Records a message for pa_last_error() and returns `st`.
pa_status fail(pa_status st, const char* fmt, ...)
#if defined(__GNUC__)
    __attribute__((format(printf, 2, 3)))
#endif
    ;

// Counts successful kernel launches (pa_launch_count).
void count_launch(uint64_t n = 1);

// Device address of the current device's status word (cached per device).
// Returns nullptr (and records a message) if CUDA fails.
unsigned int* device_status_word();

// Element size of a dtype, 0 if invalid.
inline int elem_size(pa_dtype dt) {
  switch (dt) {
    case PA_F32: return 4;
    case PA_F16: return 2;
    case PA_BF16: return 2;
    case PA_FP8_E4M3: return 1;
    default: return 0;
  }
}

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

constexpr int kDefaultPartition = 512;  // tokens per split-K partition
constexpr int kStageTokens = 32;        // tokens per pipeline stage of the decode kernel

// ---- decode launch description (validated on the host) ----
struct DecodeArgs {
  void* out;
  const void* q;
  const void* k_cache;
  const void* v_cache;
  const int32_t* block_tables;
  const int32_t* context_lens;
  float* workspace;  // may be null when num_partitions == 1
  int64_t max_blocks;
  int num_seqs, Hq, Hkv, D, block_size, num_blocks;
  int partition_size, num_partitions;
  int max_context_len = 0;
  float scale;
  pa_dtype dtype;      // q and out (and the caches unless kv_dtype says otherwise)
  pa_dtype kv_dtype;   // the caches: dtype, or PA_FP8_E4M3
  float k_scale = 1.f, v_scale = 1.f;  // per-cache scales of E4M3 codes
  // Shared-prefix groups (pa_decode_grouped).  num_partitions is then the
  // workspace's slots per (sequence, head): the groups' span partitions first,
  // then the rest of each sequence's from slot_base.  seq_shift[b] (device,
  // nullable) is the number of leading tokens of sequence b its group serves.
  const int32_t* seq_shift = nullptr;
  int slot_base = 0;          // first slot of the partition launch (and rest of the reduce)
  // the group launch: members group_start[i] .. group_start[i+1]-1 (device)
  const int32_t* group_start = nullptr;
  int num_groups = 0, max_group_size = 0;
  // An E4M3 cache with a scale per (block, kv head) (pa_decode_fp8_block):
  // [NB][Hkv] (device); k_scale = v_scale = 1 then
  const float* k_scales = nullptr;
  const float* v_scales = nullptr;
  // pa_decode_scored; num_partitions then counts from a sequence's first
  // visible block (rule_span_bound)
  bool has_rule = false;
  pa_score_rule rule = {};
};

// The scales that the kernels take a block of codes to have: a stored value
// outside is read as the nearer bound (their 1 / scale stays finite, and the
// weights of two blocks stay within the range of an fp32).
constexpr float kScaleMin = 9.094947017729282e-13f;  // 2^-40
constexpr float kScaleMax = 1.2089258196146292e+24f; // 2^80

// Most tokens from the first visible block to the last visible key of a run of
// run_len query tokens under a rule, for contexts up to max_context_len.
inline int rule_span_bound(const pa_score_rule& r, int max_context_len, int run_len,
                           int block_size) {
  if (r.window <= 0 || r.prefix_lens != nullptr) return max_context_len;
  const int64_t n = static_cast<int64_t>(r.window) + run_len + block_size;
  return n < max_context_len ? static_cast<int>(n) : max_context_len;
}

// Kernel launchers (kernels.cu).  They return cudaError_t as int.
int launch_decode_partitions(const DecodeArgs& a, unsigned int* status, void* stream);
int launch_decode_reduce(const DecodeArgs& a, unsigned int* status, void* stream);
// Tensor-core partition kernel (decode_tc.cu): fp16/bf16, head size 128, 4 or 8
// query heads per kv head, partition length a multiple of 128.
bool decode_tc_supported(const DecodeArgs& a);
int launch_decode_partitions_tc(const DecodeArgs& a, unsigned int* status, void* stream);
// Consecutive partitions one CTA of a tensor-core decode kernel streams (1, 2,
// 4 or 8) when ctas_without CTAs would each serve one partition of n_parts.
int tc_parts_per_cta(const DecodeArgs& a);
// rows: CTAs per partition index (sequences x kv heads); other_ctas: CTAs of
// other work in the same grid.
int tc_parts_per_cta(int64_t rows, int partition_size, int n_parts, int64_t other_ctas);
// pa_decode_grouped's partition phase on the tcgen05 kernel in one launch (f16
// / bf16, head size 128, G in {1, 2, 4, 8}): the groups' shared spans
// (partials into slots [0, a.slot_base) of every member's row) and the rest of
// every sequence (slots from a.slot_base).
bool decode_group_tc_supported(const DecodeArgs& a);
int launch_decode_group_tc(const DecodeArgs& a, unsigned int* status, void* stream);
// Tensor-core partition kernel over an E4M3 cache (decode_tc8.cu): f16/bf16
// queries, head size 128, 4 or 8 query heads per kv head, partition length a
// multiple of 128.
bool decode_tc8_supported(const DecodeArgs& a);  // needs tmap_available()
bool decode_block_on_tc(pa_dtype dtype, int G, int max_context_len);  // over block scales, head size 128
int launch_decode_partitions_tc8(const DecodeArgs& a, unsigned int* status, void* stream);
// The groups' shared spans over an E4M3 cache (pa_decode_grouped_fp8), G = 1, 2, 4, 8.
bool decode_group_tc8_supported(const DecodeArgs& a);  // needs tmap_available()
int launch_decode_group_tc8(const DecodeArgs& a, unsigned int* status, void* stream);
// A TMA tensor map of 16-bit elements (bytes for PA_FP8_E4M3) with the 128-byte swizzle: `rank` dims
// (innermost first), byte strides of dims 1..rank-1, a box; `map` points at a
// CUtensorMap.  False if encoding fails.
bool make_tmap(void* map, const void* base, int rank, const int64_t* dims,
               const int64_t* strides_bytes, const int* box, pa_dtype dt);
// Whether the driver entry point that encodes tensor maps could be found.
bool tmap_available();

// ---- several query tokens per sequence (decode_mq.cu) ----
struct MqArgs {
  void* out;
  const void* q;
  const void* k_cache;
  const void* v_cache;
  const int32_t* block_tables;
  const int32_t* context_lens;
  const int32_t* query_start;
  float* workspace;  // may be null when num_partitions == 1
  int64_t max_blocks;
  int num_seqs, total_q, max_query_len, Hq, Hkv, D, block_size, num_blocks;
  int partition_size, num_partitions;
  float scale;
  pa_dtype dtype;
  // Set by the partition launcher for the reduce: the partition kernel groups a
  // sequence's query tokens in runs of this many (from the first) and writes a
  // run's outputs directly, with no partials, when its last query token's last
  // key lies in the first partition.
  int direct_qblock = 0;
  // pa_decode_multi_scored: partitions then count from the first visible block
  // of each run of direct_qblock query tokens (set before the launches)
  bool has_rule = false;
  pa_score_rule rule = {};
};
constexpr int kMqRows = 128;  // (query token, head) rows per query tile of the multi-query kernel
constexpr int kMqTiles = 2;   // query tiles per CTA of the multi-query kernel
int launch_decode_mq(const MqArgs& a, unsigned int* status, void* stream);
// Its form under a score rule (decode_mq_rule.cu).
int launch_decode_mq_rule(const MqArgs& a, unsigned int* status, void* stream);
// Few query tokens per sequence (max_query_len * G <= 64, G = 4 or 8): the
// token-major tcgen05 decode kernel with per-column causal limits, 16 / G query
// tokens per CTA (decode_tc.cu).
bool decode_mq_tc_supported(const MqArgs& a);
// Whether a call's query tokens are few enough for the token-major kernel: up to
// 64 (query token, head) columns at G = 4 and 8; under a rule also up to 32 at
// G = 1 and 2, where the query-major kernel leaves its 128-row blocks nearly
// empty (178 sequences of 57-102 tokens, 16/8 heads, one query each: 82 -> 40 us).
inline bool mq_token_major(int G, int max_query_len, bool rule) {
  if (G == 4 || G == 8) return max_query_len <= 64 / G;
  return rule && (G == 1 || G == 2) && max_query_len <= 32 / G;
}
// Query tokens one CTA of the token-major kernel serves for G query heads per kv
// head: 2 (G * 2 <= 16 columns), 4 at G = 4 (16 columns), else 32 / G (the
// N = 32 variant: 4 at G = 8, 8 at G = 4).
inline int tc_query_tokens_per_cta(int G, int max_query_len) {
  if (G <= 2) return max_query_len * G <= 8 ? 8 / G : 16 / G;   // under a rule
  if (max_query_len <= 2) return 2;
  if (G == 4 && max_query_len <= 4) return 4;
  return 32 / G;
}
int launch_decode_mq_tc(const MqArgs& a, unsigned int* status, void* stream);
int launch_decode_mq_reduce(const MqArgs& a, void* stream);

int launch_reshape_and_cache(const void* key, const void* value, void* k_cache, void* v_cache,
                             const int64_t* slot_mapping, int num_tokens, int Hkv, int D,
                             int block_size, int num_blocks, int esize, unsigned int* status,
                             void* stream);
// Append into an E4M3 cache; key/value of `dtype` (f32 / f16 / bf16).
int launch_reshape_and_cache_fp8(const void* key, const void* value, void* k_cache,
                                 void* v_cache, const int64_t* slot_mapping, int num_tokens,
                                 int Hkv, int D, int block_size, int num_blocks, pa_dtype dtype,
                                 float k_scale, float v_scale, unsigned int* status, void* stream);
// Append into an E4M3 cache with a scale per (block, kv head) (cache_block.cu).
int launch_append_block(const void* key, const void* value, void* k_cache, void* v_cache,
                        float* k_scales, float* v_scales, const int64_t* slot_mapping,
                        int num_tokens, int Hkv, int D, int block_size, int num_blocks,
                        pa_dtype dtype, unsigned int* status, void* stream);
// Block copies of such a cache, codes and scales ([0]: keys, [1]: values).
struct CopyScaled {
  void* dst[2];
  const void* src[2];
  float* dst_scales[2];
  const float* src_scales[2];
  const int64_t* pairs;
  int num_pairs, src_blocks, dst_blocks, Hkv, D, block_size;
  bool device;   // one pool in device memory (copy-on-write, compaction)
};
int launch_copy_block_scaled(const CopyScaled& c, unsigned int* status, void* stream);
int launch_copy_blocks(void* dst_k, void* dst_v, const void* src_k, const void* src_v,
                       const int64_t* pairs, int num_pairs, int Hkv, int D, int block_size,
                       int src_blocks, int dst_blocks, int esize, unsigned int* status,
                       void* stream);

// Launches `kernel` on `stream` allowing it to overlap the tail of the previous
// kernel on the stream (programmatic stream serialisation); the kernel must
// call grid_dependency_wait() before it reads anything an earlier launch wrote.
template <typename... KArgs, typename... Args>
inline cudaError_t launch_overlapped(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem,
                                     cudaStream_t stream, Args&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...);
}

}  // namespace pa
