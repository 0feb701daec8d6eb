// decode_mq_rule.cu -- attention under a score rule for several new query tokens
// per sequence (prompt chunks), query-major on the tensor cores: fp16/bf16, head
// size 128, G = Hq/Hkv in {1, 2, 4, 8}.  What pa_rule.cuh says of the scores,
// with the products, tiles and partials of decode_mq.cu.
//
// A CTA serves a run of two query blocks of 128 / G query tokens (128 rows of
// (token, head) pairs each) and one kv head over a partition of the run's keys:
// positions count from the block of the first key that any token of the run
// sees, up to the last one.  Per tile of 128 keys and block X
//
//   S_X [128 x 128] = Q_X . K^T;  P_X = 2^(rule(S_X) - m);  O_X += P_X . V
//
// The two blocks take turns on the tensor core (S_X and O_X fill all 512 TMEM
// columns; P_X goes back into S_X's), so a block's softmax has to be done in the
// time of the other's two products.  Tiles are taken from the last key to the
// first: a bias that grows with distance then puts the largest scores first,
// and the running maximum, set by the first tiles, hardly rises again (from the
// first key on, 72 % of the tiles of the chunks below raised it and rescaled O).
// Each row has ONE softmax thread, which reads its 128 scores from TMEM once and
// keeps them in registers: maximum, rule, exponentials and sum touch nothing
// else, and no two threads have to agree on a row's maximum (decode_mq.cu's two
// threads per row read S twice and meet at a barrier every tile; with the rule's
// work added that took 805 us on 512-token chunks of 8 sequences, 332 GFLOP,
// where this kernel takes 383: 0.53 of the bf16 peak).  P goes to the tensor
// core in two halves.  The commit of S_X (i) also covers O_X (i - 1), which was
// issued before it, so a raised maximum rescales O without another wait.
//
// Roles (12 warps): warps 0-3 the first block's softmax and epilogue, warps 4-7
// the second's, warp 8 TMA producer (Q, then the K/V tiles), warp 9 TMEM owner
// and MMA issuer (its warpgroup hands its registers to the softmax).  A ring of
// four K/V tiles and the two Q blocks, 193 KB of shared memory: one CTA per SM.
// The CTAs of one kv head's runs are neighbours in the grid and read its K/V
// from L2.  Every wait is bounded; block ids outside the pool are skipped and
// flagged; inconsistent query offsets are flagged (PA_DEVERR_CONTEXT) and their
// sequence skipped.
#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "mq_common.cuh"
#include "pa_device.cuh"
#include "pa_internal.h"
#include "pa_rule.cuh"
#include "tc_common.cuh"

namespace pa {

namespace {

using namespace tc;
using namespace mq;

constexpr unsigned FULL = 0xffffffffu;
constexpr int NT = kMqTiles;                    // query blocks per CTA
constexpr int SLOTS = 4;
constexpr int THREADS = NT * 128 + 128;       // two softmax warpgroups; producer, MMA, two idle
constexpr int OFF_Q = SLOTS * SLOT_BYTES;
constexpr int OFF_BAR = OFF_Q + NT * OPA_BYTES;
// ring full/empty; s_full, p_half, p_full, o_full per block; q_ready
constexpr int NBARS = 2 * SLOTS + 4 * NT + 1;
constexpr int OFF_TMEM = OFF_BAR + NBARS * 8;
constexpr int SMEM_BYTES = OFF_TMEM + 16 + 1024;
static_assert(SMEM_BYTES <= 227 * 1024, "shared memory");
static_assert(NT == 2, "TMEM holds (S, O) of two blocks");

struct Params {
  void* out;
  const int32_t* block_tables;
  const int32_t* context_lens;
  const int32_t* query_start;
  float* ws_o;
  float* ws_m;
  float* ws_l;
  unsigned int* status;
  int64_t max_blocks;
  int total_q, Hq, Hkv, G, num_blocks, block_size, partition_size, num_partitions, n_pairs;
  RuleParams rule;
};

// Pairs of fp32 in one instruction.
__device__ __forceinline__ void add2(float& x, float& y, float a, float b, float c, float d) {
  asm("{\n\t.reg .b64 u, v;\n\tmov.b64 u, {%2, %3};\n\tmov.b64 v, {%4, %5};\n\t"
      "add.rn.f32x2 u, u, v;\n\tmov.b64 {%0, %1}, u;\n\t}"
      : "=f"(x), "=f"(y)
      : "f"(a), "f"(b), "f"(c), "f"(d));
}
// (x, y) = (x, y) * m + (c, d)
__device__ __forceinline__ void fma2(float& x, float& y, float m, float c, float d) {
  asm("{\n\t.reg .b64 u, v, w;\n\tmov.b64 u, {%0, %1};\n\tmov.b64 v, {%2, %2};\n\t"
      "mov.b64 w, {%3, %4};\n\tfma.rn.f32x2 u, u, v, w;\n\tmov.b64 {%0, %1}, u;\n\t}"
      : "+f"(x), "+f"(y)
      : "f"(m), "f"(c), "f"(d));
}

// Register shares: the softmax warpgroups take what the producer's and the MMA
// issuer's give up (launch: 384 threads of 168; 2 * 128 * 224 + 128 * 40 = 62464
// of its 64512).
constexpr int REGS_SOFTMAX = 224, REGS_OTHER = 40;
constexpr int REGS_LAUNCH = 168;               // per thread, checked before a launch
static_assert(NT * 128 * REGS_SOFTMAX + 128 * REGS_OTHER <= REGS_LAUNCH * THREADS, "register shares");
template <int N>
__device__ __forceinline__ void more_registers() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void fewer_registers() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// 32 TMEM columns of this thread's lane, without waiting for them.
__device__ __forceinline__ void tmem_ld32_async(uint32_t taddr, float* v) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,"
      "%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]),
        "=f"(v[7]), "=f"(v[8]), "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]),
        "=f"(v[14]), "=f"(v[15]), "=f"(v[16]), "=f"(v[17]), "=f"(v[18]), "=f"(v[19]),
        "=f"(v[20]), "=f"(v[21]), "=f"(v[22]), "=f"(v[23]), "=f"(v[24]), "=f"(v[25]),
        "=f"(v[26]), "=f"(v[27]), "=f"(v[28]), "=f"(v[29]), "=f"(v[30]), "=f"(v[31])
      : "r"(taddr)
      : "memory");
}
// Waits for them; the values pass through, so that no use of them moves ahead.
__device__ __forceinline__ void tmem_wait_ld() {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void hold(float* v, int n) {
#pragma unroll
  for (int i = 0; i < n; ++i) asm volatile("" : "+f"(v[i]));
}

// The 128 raw scores of a row to finished ones (base 2) plus `add`.  open: the
// row sees every key of the tile; left: none lies behind the row's own position,
// so that the bias is linear in the key (8 keys share a base; one add and one
// FMA per two scores).
template <int RULE, bool SLOPES>
__device__ __forceinline__ void finish_scores(const Params& p, float* s, float add, bool open,
                                              bool left, int pos_c, int lo_c, int hi_c,
                                              float slope) {
  if constexpr (RULE == kRuleCapped) {
#pragma unroll
    for (int j = 0; j < TOK; ++j) s[j] = rule_cap<RULE>(p.rule.cap_log2, s[j] * p.rule.scale);
  }
  const float scale = RULE == kRuleCapped ? 1.f : p.rule.scale;
  if constexpr (SLOPES) {
    const float d0 = static_cast<float>(pos_c);          // the row's own column
    if (left) {
      float step[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) step[e] = slope * static_cast<float>(e);
#pragma unroll
      for (int j = 0; j < TOK; j += 8) {
        const float base = fmaf(slope, static_cast<float>(j) - d0, add);
#pragma unroll
        for (int e = 0; e < 8; e += 2) {
          float b0, b1;
          add2(b0, b1, step[e], step[e + 1], base, base);
          fma2(s[j + e], s[j + e + 1], scale, b0, b1);
        }
      }
    } else {
#pragma unroll
      for (int j = 0; j < TOK; ++j)
        s[j] = fmaf(-slope, fabsf(d0 - static_cast<float>(j)), fmaf(s[j], scale, add));
    }
  } else {
#pragma unroll
    for (int j = 0; j < TOK; j += 2) fma2(s[j], s[j + 1], scale, add, add);
  }
  if (!open) {
#pragma unroll
    for (int w = 0; w < TOK / 32; ++w) {
      // bit j: the row sees column 32 w + j
      const int a = lo_c - 32 * w, b = hi_c - 32 * w;
      const unsigned from = a <= 0 ? FULL : a > 31 ? 0u : FULL << a;
      const unsigned to = b < 0 ? 0u : b >= 31 ? FULL : FULL >> (31 - b);
      const unsigned see = from & to;
#pragma unroll
      for (int j = 0; j < 32; ++j)
        if (((see >> j) & 1u) == 0) s[32 * w + j] = -INFINITY;
    }
  }
}

template <typename T, int RULE, bool SLOPES>
__global__ void __launch_bounds__(THREADS, 1)
    decode_mq_rule_kernel(const Params p, const __grid_constant__ CUtensorMap tmap_k,
                          const __grid_constant__ CUtensorMap tmap_v,
                          const __grid_constant__ CUtensorMap tmap_q) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint8_t* ring = smem;
  uint8_t* qop = smem + OFF_Q;                      // NT blocks of OPA_BYTES
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + OFF_BAR);
  uint64_t* ring_full = bars;
  uint64_t* ring_empty = bars + SLOTS;
  uint64_t* s_full = bars + 2 * SLOTS;              // [NT]
  uint64_t* p_half = s_full + NT;                   // [NT] P of the tile's first 64 keys
  uint64_t* p_full = p_half + NT;                   // [NT] and of the rest
  uint64_t* o_full = p_full + NT;                   // [NT]
  uint64_t* q_ready = o_full + NT;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + OFF_TMEM);

  // the runs of one kv head are neighbours
  const int pair = blockIdx.x % p.n_pairs;
  int rest = blockIdx.x / p.n_pairs;
  const int part = rest % p.num_partitions;
  rest /= p.num_partitions;
  const int g = rest % p.Hkv, b = rest / p.Hkv;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int G = p.G, QB = MR / G;

  grid_dependency_wait();
  allow_dependents();
  // ---- this CTA's query rows and key range (validated) ----
  const int q0 = p.query_start[b];
  const int Qb = p.query_start[b + 1] - q0;
  const int L = p.context_lens[b];
  const int P = p.partition_size;
  if (L < 0 || L > p.max_blocks * p.block_size || Qb < 0 || Qb > L || q0 < 0 ||
      q0 + Qb > p.total_q) {
    if (threadIdx.x == 0 && pair == 0 && part == 0 && g == 0) atomicOr(p.status, PA_DEVERR_CONTEXT);
    return;
  }
  if (pair == 0 && part == 0 && g == 0 && threadIdx.x == 0 && Qb > p.n_pairs * NT * QB)
    atomicOr(p.status, PA_DEVERR_CONTEXT);          // max_query_len below this Q_b
  const int i0 = pair * NT * QB;                    // the run's query tokens i0 .. i1 - 1
  if (i0 >= Qb) return;
  const int i1 = min(Qb, i0 + NT * QB);
  int lo, hi;
  rule_span(p.rule, b, q0, L - Qb, L, i0, i1, lo, hi);
  if (lo > hi) {                                    // nothing is seen: zero rows
    if (part == 0) {
      for (int i = threadIdx.x; i < (i1 - i0) * G * DH; i += THREADS) {
        const int64_t hq = (static_cast<int64_t>(q0) + i0 + i / (G * DH)) * p.Hq + g * G + i / DH % G;
        static_cast<T*>(p.out)[hq * DH + i % DH] = Elem<T>::from_float(0.f);
      }
    }
    return;
  }
  const int bs = p.block_size;
  const int shift = lo / bs * bs;                   // positions count from here on
  const int first = lo - shift;                     // the first one seen
  const int pmax = hi - shift;                      // the last one
  if (pmax >= static_cast<int64_t>(p.num_partitions) * P) {   // a context beyond max_context_len
    if (threadIdx.x == 0 && part == 0 && g == 0) atomicOr(p.status, PA_DEVERR_CONTEXT);
    return;
  }
  const int kstart = part * P;
  if (kstart > pmax) return;
  const int kend = min(kstart + P, pmax + 1);
  const int n_tiles = (kend - kstart + TOK - 1) / TOK;
  const bool single = pmax < P;

  const int bpt = TOK / bs;
  const int first_blk = kstart / bs;
  const int last_blk = (kend + bs - 1) / bs;
  const int32_t* trow = p.block_tables + static_cast<int64_t>(b) * p.max_blocks + shift / bs;
  if (warp == 4 * NT && lane == 0) {                // the producer
    for (int s = 0; s < SLOTS; ++s) {
      mbar_init(&ring_full[s], 1);
      mbar_init(&ring_empty[s], 1);
    }
    for (int x = 0; x < NT; ++x) {
      mbar_init(&s_full[x], 1);
      mbar_init(&p_half[x], 4);
      mbar_init(&p_full[x], 4);
      mbar_init(&o_full[x], 1);
    }
    mbar_init(q_ready, 1);
    fence_mbar_init();
    // Q of both blocks: row r = (token r / G, head r % G), 64 columns a box.
    // Rows past the run's tokens hold other tokens' queries or zeros; what
    // becomes of them is not written.
    mbar_arrive_expect_tx(q_ready, NT * OPA_BYTES);
#pragma unroll
    for (int c = 0; c < 2 * NT; ++c)
      tma_load_4d(qop + c * OPA_HALF, &tmap_q, 0, g * G, c & 1, q0 + i0 + (c >> 1) * QB, q_ready);
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tmap_k)) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tmap_v)) : "memory");
  }
  if (warp == 4 * NT + 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_addr(tmem_slot)),
                 "r"(TMEM_COLS)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  if (warp >= 4 * NT) {
    fewer_registers<REGS_OTHER>();
    if (warp == 4 * NT) {
      // ================= producer =================
      const int row_stride = p.Hkv * bs;
      bool ok = true;
      int issued = 0;
      auto table = [&](int i) {
        const int b0 = first_blk + (n_tiles - 1 - i) * bpt;
        return (i < n_tiles && lane < min(bpt, last_blk - b0)) ? __ldg(trow + b0 + lane) : -1;
      };
      int pb_next = table(0);
      for (int i = 0; i < n_tiles && ok; ++i) {
        const int b0 = first_blk + (n_tiles - 1 - i) * bpt;
        const int nb = min(bpt, last_blk - b0);
        const int pb = pb_next;
        pb_next = table(i + 1);
        const bool mine = lane < nb;
        const bool valid = mine && pb >= 0 && pb < p.num_blocks;
        if (mine && !valid) atomicOr(p.status, PA_DEVERR_TABLE);
        const unsigned vmask = __ballot_sync(FULL, valid);
        const uint32_t bytes = __popc(vmask) * 2u * static_cast<uint32_t>(bs) * 128u;
        const int grp = valid ? (pb * row_stride + g * bs) / 8 : 0;
        for (int kv = 0; kv < 2; ++kv) {
          const int u = 2 * i + kv;
          const int s = u % SLOTS;
          if (u >= SLOTS && !mbar_wait(&ring_empty[s], ((u / SLOTS) - 1) & 1, p.status)) {
            ok = false;
            break;
          }
          if (lane == 0) mbar_arrive_expect_tx(&ring_full[s], bytes);
          __syncwarp();
          if (valid)
            tma_load_4d(ring + s * SLOT_BYTES + lane * bs * 256, kv == 0 ? &tmap_k : &tmap_v, 0, 0,
                        0, grp, &ring_full[s]);
          issued = u + 1;
        }
      }
      if (!ok) {
        for (int u = issued - SLOTS < 0 ? 0 : issued - SLOTS; u < issued; ++u)
          mbar_wait(&ring_full[u % SLOTS], (u / SLOTS) & 1, p.status);
      }
    } else if (warp == 4 * NT + 1) {
      // ================= MMA issuer =================
      if (lane == 0) {
        const uint32_t id_s = idesc_mq<T>(false);
        const uint32_t id_o = idesc_mq<T>(true);
        const uint32_t ring_a = smem_addr(ring), q_a = smem_addr(qop);
        auto issue_s = [&](int x, int i) {           // S_x = Q_x . K_i^T
          const int s = (2 * i) % SLOTS;
          const uint32_t d = tmem + x * 128;
#pragma unroll
          for (int k = 0; k < DH / 16; ++k) {
            const uint64_t a =
                smem_desc(q_a + x * OPA_BYTES + (k >> 2) * OPA_HALF + (k & 3) * 32, 16, 1024);
            const uint64_t bk =
                smem_desc(ring_a + s * SLOT_BYTES + (k >> 2) * HALF_OFF + (k & 3) * 32, 16, GROUP_BYTES);
            mma_f16(d, a, bk, id_s, k > 0);
          }
          mma_commit(&s_full[x]);
        };
        auto issue_pv = [&](int x, int i, int h) {   // O_x += P_x . V_i over half h's keys, P_x in TMEM
          const int s = (2 * i + 1) % SLOTS;
          const uint32_t d = tmem + 256 + x * 128;
#pragma unroll
          for (int k = 4 * h; k < 4 * h + 4; ++k) {
            const uint64_t bv =
                smem_desc(ring_a + s * SLOT_BYTES + k * 2 * GROUP_BYTES, HALF_OFF, GROUP_BYTES);
            mma_f16_ts(d, tmem + x * 128 + k * 8, bv, id_o, (i > 0 || k > 0) ? 1u : 0u);
          }
        };
        auto ring_wait = [&](int u) { return mbar_wait(&ring_full[u % SLOTS], (u / SLOTS) & 1, p.status); };
        bool ok = mbar_wait(q_ready, 0, p.status) && ring_wait(0);
        if (ok) {
          tc_fence_after();
          issue_s(0, 0);
          issue_s(1, 0);
          mma_commit(&ring_empty[0]);
        }
        for (int i = 0; i < n_tiles && ok; ++i) {
          const bool more = i + 1 < n_tiles;
          ok = ring_wait(2 * i + 1) && mbar_wait(&p_half[0], i & 1, p.status);
          if (!ok) break;
          tc_fence_after();
          issue_pv(0, i, 0);
          ok = mbar_wait(&p_full[0], i & 1, p.status);
          if (!ok) break;
          tc_fence_after();
          issue_pv(0, i, 1);
          if (more) {
            ok = ring_wait(2 * i + 2);
            if (!ok) break;
            tc_fence_after();
            issue_s(0, i + 1);                       // over P_0, which O_0 has read by then
          } else {
            mma_commit(&o_full[0]);
          }
          ok = mbar_wait(&p_half[1], i & 1, p.status);
          if (!ok) break;
          tc_fence_after();
          issue_pv(1, i, 0);
          ok = mbar_wait(&p_full[1], i & 1, p.status);
          if (!ok) break;
          tc_fence_after();
          issue_pv(1, i, 1);
          mma_commit(&ring_empty[(2 * i + 1) % SLOTS]);
          if (more) {
            issue_s(1, i + 1);
            mma_commit(&ring_empty[(2 * i + 2) % SLOTS]);
          } else {
            mma_commit(&o_full[1]);
          }
        }
      }
      __syncwarp();
      // every softmax warp is done with TMEM
      named_sync(1, NT * 128 + 32);
      tc_fence_after();
      asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem),
                   "r"(TMEM_COLS)
                   : "memory");
    }
  } else {
    more_registers<REGS_SOFTMAX>();
    // ================= softmax: thread of block X, row r (its TMEM lane) =================
    const int X = warp >> 2;
    const int r = (warp & 3) * 32 + lane;
    const int qtok = i0 + X * QB + r / G;
    const int head = g * G + r % G;
    const bool row_valid = qtok < Qb;
    const int64_t t = static_cast<int64_t>(q0) + qtok;
    const int pos = L - Qb + qtok - shift;          // its own position, and what it sees
    int row_lo = 0, row_hi = -1;
    float slope = 0.f;
    if (row_valid) {
      rule_limits(p.rule, b, t, L - Qb + qtok, L, row_lo, row_hi);
      row_lo -= shift;
      row_hi -= shift;
      if (SLOPES && p.rule.slopes != nullptr) slope = __ldcg(p.rule.slopes + head) * kLog2e;
    }
    const bool warp_active = __any_sync(FULL, row_valid);
    const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t s_col = tmem + lane_base + X * 128;
    const uint32_t o_col = tmem + lane_base + 256 + X * 128;
    float m_run = -INFINITY, l_sum = 0.f;
    bool ok = true;
    auto wait = [&](uint64_t* bar, uint32_t parity) {
      if (ok) ok = mbar_wait(bar, parity, p.status);
      ok = __all_sync(FULL, ok);
      return ok;
    };
    auto first_half = [&]() {                       // P of the tile's first 64 keys is there
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&p_half[X]);
    };
    for (int i = 0; i < n_tiles; ++i) {
      const int tile0 = kstart + (n_tiles - 1 - i) * TOK;
      const int n_valid = min(TOK, kend - tile0);
      const int n_first = first - tile0;           // > 0 in the sequence's first tile only
      if (X == 0 && (n_valid < TOK || n_first > 0)) {
        // zero the V rows of keys that no token of the run sees, so that
        // whatever they hold adds 0 to O (PV of both blocks waits for this)
        const int u = 2 * i + 1, s_ = u % SLOTS;
        if (wait(&ring_full[s_], (u / SLOTS) & 1) && (r >= n_valid || r < n_first)) {
          uint8_t* row = ring + s_ * SLOT_BYTES + (r >> 3) * GROUP_BYTES + (r & 7) * 128;
#pragma unroll
          for (int c = 0; c < 8; ++c) {
            *reinterpret_cast<uint4*>(row + c * 16) = make_uint4(0, 0, 0, 0);
            *reinterpret_cast<uint4*>(row + HALF_OFF + c * 16) = make_uint4(0, 0, 0, 0);
          }
        }
        fence_async_smem();
      }
      const bool have = wait(&s_full[X], i & 1);
      tc_fence_after();
      if (warp_active && have) {
        float s[TOK];
#pragma unroll
        for (int c = 0; c < TOK / 32; ++c) tmem_ld32_async(s_col + c * 32, s + c * 32);
        tmem_wait_ld();
        hold(s, TOK);
        const int lo_c = row_lo - tile0, hi_c = min(row_hi - tile0, n_valid - 1);
        const bool open = __all_sync(FULL, lo_c <= 0 && hi_c >= TOK - 1);
        const bool left = __all_sync(FULL, pos - tile0 >= TOK - 1);
        // scores relative to the running maximum (0 before the first): with no
        // raise, which is rare, they are the exponents as they stand
        const float m_old = m_run == -INFINITY ? 0.f : m_run;
        finish_scores<RULE, SLOPES>(p, s, -m_old, open, left, pos - tile0, lo_c, hi_c, slope);
        float pm[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
        for (int j = 4; j + 1 < TOK; j += 2)
          pm[(j >> 1) & 3] = fmaxf(fmaxf(pm[(j >> 1) & 3], s[j]), s[j + 1]);
        const float rise = fmaxf(fmaxf(pm[0], pm[1]), fmaxf(pm[2], pm[3]));
        if (__any_sync(FULL, m_run == -INFINITY ? rise > -INFINITY : rise > RESCALE_THRESHOLD)) {
          // every row of the warp to its maximum so far
          const float up = m_run == -INFINITY ? (rise == -INFINITY ? 0.f : rise) : fmaxf(rise, 0.f);
          const float alpha = m_run == -INFINITY ? 0.f : ex2_approx(-up);
          if (m_run != -INFINITY || rise > -INFINITY) m_run = m_old + up;
          l_sum *= alpha;
#pragma unroll
          for (int j = 0; j < TOK; j += 2) add2(s[j], s[j + 1], s[j], s[j + 1], -up, -up);
          if (i > 0) {                             // O of tiles before i is complete (see above)
#pragma unroll 1
            for (int c = 0; c < DH / 16; ++c) {
              float o[16];
              tmem_ld16(o_col + c * 16, o);
#pragma unroll
              for (int j = 0; j < 16; ++j) o[j] *= alpha;
              tmem_st16(o_col + c * 16, o);
            }
          }
        }
        float ps[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int c = 0; c < TOK / 32; ++c) {
          uint32_t w[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const float a = ex2_approx(s[32 * c + 2 * e]);   // masked: 2^-inf = 0
            const float d = ex2_approx(s[32 * c + 2 * e + 1]);
            add2(ps[(2 * e) & 3], ps[(2 * e + 1) & 3], ps[(2 * e) & 3], ps[(2 * e + 1) & 3], a, d);
            w[e] = pack2<T>(a, d);
          }
          tmem_st16u(s_col + c * 16, w);
          if (c == 1) first_half();
        }
        l_sum += (ps[0] + ps[1]) + (ps[2] + ps[3]);
      } else {
        // no query row in this warp: its P rows are 0
        uint32_t z[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) z[e] = 0u;
#pragma unroll
        for (int c = 0; c < TOK / 32; ++c) tmem_st16u(s_col + c * 16, z);
        first_half();
      }
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&p_full[X]);
    }
    // ---- epilogue: row r of O_X ----
    wait(&o_full[X], 0);
    tc_fence_after();
    const int64_t hq = t * p.Hq + head;
    const float inv = l_sum == 0.f ? 0.f : 1.f / l_sum;
#pragma unroll 1
    for (int c = 0; c < (warp_active && ok ? DH / 32 : 0); ++c) {
      float o[32];
      tmem_ld32(o_col + c * 32, o);
      if (!row_valid) continue;
      if (single) {
        T* dst = static_cast<T*>(p.out) + hq * DH + c * 32;
#pragma unroll
        for (int j = 0; j < 32; j += 8) {
          uint32_t w[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) w[e] = pack2<T>(o[j + 2 * e] * inv, o[j + 2 * e + 1] * inv);
          *reinterpret_cast<uint4*>(dst + j) = make_uint4(w[0], w[1], w[2], w[3]);
        }
      } else {
        const int64_t slot = hq * p.num_partitions + part;
        float* dst = p.ws_o + slot * DH + c * 32;
#pragma unroll
        for (int j = 0; j < 32; j += 4)
          *reinterpret_cast<float4*>(dst + j) = make_float4(o[j], o[j + 1], o[j + 2], o[j + 3]);
        if (c == 0) {
          p.ws_m[slot] = m_run;
          p.ws_l[slot] = l_sum;
        }
      }
    }
    tc_fence_before();
    named_sync(1, NT * 128 + 32);
  }
}

template <typename T, int RULE, bool SLOPES>
cudaError_t launch_t(const MqArgs& a, unsigned int* status, cudaStream_t stream) {
  auto kern = decode_mq_rule_kernel<T, RULE, SLOPES>;
  // the register shares count on what the kernel was compiled to (a property of
  // the code, read once); a smaller pool would leave a warpgroup waiting
  static const int regs = [&] {
    cudaFuncAttributes at;
    return cudaFuncGetAttributes(&at, kern) == cudaSuccess ? at.numRegs : 0;
  }();
  if (regs < REGS_LAUNCH) return cudaErrorInvalidConfiguration;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM_BYTES);
  if (e != cudaSuccess) return e;
  CUtensorMap mk, mv, mq;
  const int64_t groups = static_cast<int64_t>(a.num_blocks) * a.Hkv * a.block_size / 8;
  const int64_t dims[4] = {64, 8, 2, groups};
  const int64_t strides[3] = {DH * 2, 128, 8 * DH * 2};
  const int box[4] = {64, 8, 2, a.block_size / 8};
  if (!make_tmap(&mk, a.k_cache, 4, dims, strides, box, a.dtype) ||
      !make_tmap(&mv, a.v_cache, 4, dims, strides, box, a.dtype))
    return cudaErrorInvalidValue;
  // the queries [total_q][Hq][128] as 64 columns, heads, column halves, tokens; a
  // box is 128 / G tokens of a kv head's G query heads
  const int G = a.Hq / a.Hkv;
  const int64_t qdims[4] = {64, a.Hq, 2, a.total_q};
  const int64_t qstrides[3] = {DH * 2, 128, static_cast<int64_t>(a.Hq) * DH * 2};
  const int qbox[4] = {64, G, 1, MR / G};
  if (!make_tmap(&mq, a.q, 4, qdims, qstrides, qbox, a.dtype)) return cudaErrorInvalidValue;
  Params p;
  p.out = a.out;
  p.block_tables = a.block_tables;
  p.context_lens = a.context_lens;
  p.query_start = a.query_start;
  const int64_t nrows = static_cast<int64_t>(a.total_q) * a.Hq * a.num_partitions;
  p.ws_o = a.workspace;
  p.ws_m = a.workspace ? a.workspace + nrows * DH : nullptr;
  p.ws_l = a.workspace ? a.workspace + nrows * (DH + 1) : nullptr;
  p.status = status;
  p.max_blocks = a.max_blocks;
  p.total_q = a.total_q;
  p.Hq = a.Hq;
  p.Hkv = a.Hkv;
  p.G = G;
  p.num_blocks = a.num_blocks;
  p.block_size = a.block_size;
  p.partition_size = a.partition_size;
  p.num_partitions = a.num_partitions;
  const int qblocks = (a.max_query_len + MR / p.G - 1) / (MR / p.G);
  p.n_pairs = (qblocks + NT - 1) / NT;
  p.rule = make_rule(a.rule, a.scale);
  const int64_t ctas = static_cast<int64_t>(a.num_seqs) * a.Hkv * p.n_pairs * a.num_partitions;
  if (ctas > 0x7fffffff) return cudaErrorInvalidValue;
  return launch_overlapped(kern, dim3(static_cast<unsigned>(ctas)), dim3(THREADS), SMEM_BYTES,
                           stream, p, mk, mv, mq);
}

template <typename T>
cudaError_t launch_rule(const MqArgs& a, unsigned int* status, cudaStream_t stream) {
  const bool slopes = a.rule.alibi_slopes != nullptr;
  if (rule_kind(a.has_rule, a.rule) == kRuleCapped)
    return slopes ? launch_t<T, kRuleCapped, true>(a, status, stream)
                  : launch_t<T, kRuleCapped, false>(a, status, stream);
  return slopes ? launch_t<T, kRuleOpen, true>(a, status, stream)
                : launch_t<T, kRuleOpen, false>(a, status, stream);
}

}  // namespace

int launch_decode_mq_rule(const MqArgs& a, unsigned int* status, void* stream) {
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return a.dtype == PA_BF16 ? launch_rule<__nv_bfloat16>(a, status, st)
                            : launch_rule<__half>(a, status, st);
}

}  // namespace pa
