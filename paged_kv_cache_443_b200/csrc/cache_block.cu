// cache_block.cu -- updates of an E4M3 KV cache that keeps one scale per
// (physical block, kv head): the quantising append and the block copy.
//
// A cache with two scales in all has to be calibrated before the first token
// and either saturates or wastes codes when layers, heads or texts differ.
// With a scale per block and head ("quantization" in "4. 이 밖의 기법들",
// blog.aqudi.me, read per block; block sharing and copy-on-write as in
// "블록 공유", supersilo.blog) the append finds it:
//
//   a    = max |x| over the call's tokens of the block and head (NaNs aside)
//   need = the smallest 2^e with a <= 448 * 2^e, -40 <= e <= 80
//   old  = the stored scale; 0 if the call writes offset 0 of the block, which
//          starts the block anew
//   new  = max(old, need);  code = E4M3(x / new), saturating at 448
//   if new > old > 0: the block's other slots, code := E4M3(code * old / new)
//
// E4M3 is a floating format: the relative step of a code is the same wherever
// its scale puts it, so a power of two costs no precision and makes the
// rescaling of the older codes exact except where it reaches the subnormals.
#include <cuda_runtime.h>

#include <cstdint>

#include "pa_device.cuh"
#include "pa_internal.h"

namespace pa {

namespace {

constexpr unsigned FULL = 0xffffffffu;
constexpr int kWarps = 8;          // warps per CTA of the append
constexpr int kChunk = 16;         // most tokens whose elements a warp keeps in registers

// The smallest 2^e, -40 <= e <= 80, with most <= 448 * 2^e = 1.75 * 2^(e + 8).
__device__ __forceinline__ float scale_for(float most) {
  const uint32_t u = __float_as_uint(most);
  int e = static_cast<int>(u >> 23) - 127 - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
  e = max(-40, min(80, e));
  return __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
}

__device__ __forceinline__ uint32_t codes2(float a, float b) {
  return static_cast<uint32_t>(
      __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3));
}

// Codes of 4 floats, the first in the low byte.
__device__ __forceinline__ uint32_t codes4(const float* f) {
  return codes2(f[0], f[1]) | (codes2(f[2], f[3]) << 16);
}

struct AppendParams {
  const void* x[2];        // key, value [N][Hkv][D]
  uint8_t* cache[2];       // [NB][Hkv][bs][D]
  float* scales[2];        // [NB][Hkv]
  const int64_t* slots;    // [N]
  unsigned int* status;
  int64_t num_slots;
  int num_tokens, Hkv, log2_bs;
  int positions;           // list positions a warp looks after
};

// One warp per (run of positions of slot_mapping, kv head, K or V).  A block's
// tokens stand next to each other in slot_mapping; the warp that looks after
// the first of them does them all: it loads up to 16 tokens' elements into
// registers (16 bytes per lane and load, all loads in flight together), finds
// the largest, settles the scale, rescales the older codes if it grew, and
// writes the codes.  Longer runs (blocks of 32; a slot given several times)
// are read a second time, from L2.
template <typename T, int D>
__global__ void __launch_bounds__(32 * kWarps) append_block_kernel(const AppendParams p) {
  allow_dependents();   // the decode kernels may start launching (they wait for us)
  constexpr int EPL = Elem<T>::EPL;          // elements per lane and load
  constexpr int LPR = D / EPL;               // lanes per token row
  constexpr int RPW = 32 / LPR;              // token rows per load
  constexpr int IT = kChunk / RPW;           // loads of a full chunk
  const int lane = threadIdx.x & 31;
  const int64_t item = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  const int kv = static_cast<int>(item & 1);
  const int64_t rest = item >> 1;
  const int h = static_cast<int>(rest % p.Hkv);
  const int64_t c0 = rest / p.Hkv * p.positions;
  if (c0 >= p.num_tokens) return;
  const int n_pos = static_cast<int>(min(static_cast<int64_t>(p.positions), p.num_tokens - c0));
  const int bs = 1 << p.log2_bs;
  const T* x = static_cast<const T*>(p.x[kv]) + static_cast<int64_t>(h) * D;
  const int64_t x_stride = static_cast<int64_t>(p.Hkv) * D;

  // lane i: the block of position c0 - 1 + i (-1: no slot)
  auto block_at = [&](int64_t i) -> int64_t {
    if (i < 0 || i >= p.num_tokens) return -1;
    const int64_t s = __ldg(p.slots + i);
    return s >= 0 && s < p.num_slots ? s >> p.log2_bs : -1;
  };
  const int64_t mine = block_at(c0 + lane), before = block_at(c0 + lane - 1);
  if (lane < n_pos && h == 0 && kv == 0 && __ldg(p.slots + c0 + lane) >= p.num_slots)
    atomicOr(p.status, PA_DEVERR_SLOT);
  unsigned leaders = __ballot_sync(FULL, lane < n_pos && mine >= 0 && mine != before);

  while (leaders) {                          // warp-uniform
    const int at = __ffs(leaders) - 1;
    leaders &= leaders - 1;
    const int64_t first = c0 + at;
    const int64_t blk = __shfl_sync(FULL, mine, at);
    // ---- the run of positions in this block, and the offsets it writes ----
    int64_t n = 0;
    unsigned written = 0;
    for (;;) {
      const int64_t i = first + n + lane;
      const bool in = block_at(i) == blk;
      const unsigned same = __ballot_sync(FULL, in);
      const int add = same == FULL ? 32 : __ffs(~same) - 1;
      unsigned bit = 0;
      if (lane < add) bit = 1u << static_cast<int>(__ldg(p.slots + i) & (bs - 1));
      written |= __reduce_or_sync(FULL, bit);
      n += add;
      if (add < 32) break;
    }
    const bool fresh = (written & 1u) != 0;
    uint8_t* rows = p.cache[kv] + ((blk * p.Hkv + h) << p.log2_bs) * D;
    float* scale_at = p.scales[kv] + blk * p.Hkv + h;
    const float old = fresh ? 0.f : fmaxf(*scale_at, 0.f);

    const int sub = lane / LPR, col = lane % LPR * EPL;
    uint4 v[IT];
    auto load = [&](int64_t t0) {            // tokens first + t0 ..
#pragma unroll
      for (int k = 0; k < IT; ++k) {
        const int64_t t = t0 + k * RPW + sub;
        v[k] = t < n ? __ldg(reinterpret_cast<const uint4*>(x + (first + t) * x_stride + col))
                     : make_uint4(0, 0, 0, 0);
      }
    };
    float most = 0.f;
    for (int64_t t0 = 0; t0 < n; t0 += kChunk) {
      load(t0);
#pragma unroll
      for (int k = 0; k < IT; ++k) {
        float f[EPL];
        Elem<T>::unpack(v[k], f);
#pragma unroll
        for (int e = 0; e < EPL; ++e) most = fmaxf(most, fabsf(f[e]));
      }
    }
    most = __uint_as_float(__reduce_max_sync(FULL, __float_as_uint(most)));   // >= 0: ordered as bits
    const float now = fmaxf(old, scale_for(most));
    // x / now; a power of two divides exactly as its reciprocal multiplies
    const bool power = (__float_as_uint(now) & 0x7fffffu) == 0;
    const float inv = __frcp_rn(now);

    if (now > old && !fresh) {
      // the scale grew: the block's other codes, a row of D bytes per D / 16 lanes
      const float keep = __fdiv_rn(old, now);
      constexpr int CPR = D / 16;
      for (int r = lane / CPR; r < bs; r += 32 / CPR) {
        if ((written >> r) & 1u) continue;
        uint4* q = reinterpret_cast<uint4*>(rows + r * D) + lane % CPR;
        float f[16];
        Elem<__nv_fp8_e4m3>::load(q, f);
        Elem<__nv_fp8_e4m3>::load(reinterpret_cast<uint2*>(q) + 1, f + 8);
#pragma unroll
        for (int e = 0; e < 16; ++e) f[e] *= keep;
        *q = make_uint4(codes4(f), codes4(f + 4), codes4(f + 8), codes4(f + 12));
      }
    }
    if (lane == 0) *scale_at = now;
    for (int64_t t0 = 0; t0 < n; t0 += kChunk) {
      if (n > kChunk) load(t0);
#pragma unroll
      for (int k = 0; k < IT; ++k) {
        const int64_t t = t0 + k * RPW + sub;
        if (t >= n) continue;
        float f[EPL];
        Elem<T>::unpack(v[k], f);
#pragma unroll
        for (int e = 0; e < EPL; ++e) f[e] = power ? f[e] * inv : __fdiv_rn(f[e], now);
        const int off = static_cast<int>(__ldg(p.slots + first + t) & (bs - 1));
        uint8_t* dst = rows + off * D + col;
        if constexpr (EPL == 8)
          *reinterpret_cast<uint2*>(dst) = make_uint2(codes4(f), codes4(f + 4));
        else
          *reinterpret_cast<uint32_t*>(dst) = codes4(f);
      }
    }
  }
}

struct CopyParams {
  uint4* dst[2];
  const uint4* src[2];
  float* dst_scales[2];
  const float* src_scales[2];
  const int64_t* pairs;
  unsigned int* status;
  int64_t src_blocks, dst_blocks, chunks;   // chunks of 16 bytes per block and cache
  int num_pairs, Hkv;
};

// Block pairs[p][1] of the destination := block pairs[p][0] of the source, codes
// and scales; blockIdx.z selects K or V, a thread moves four 16-byte chunks
// with all four loads in flight.
__global__ void __launch_bounds__(256) copy_block_scaled_kernel(const CopyParams p) {
  allow_dependents();
  const int kv = blockIdx.z;
  for (int pr = blockIdx.y; pr < p.num_pairs; pr += gridDim.y) {
    const int64_t src = __ldg(p.pairs + 2 * pr);
    const int64_t dst = __ldg(p.pairs + 2 * pr + 1);
    if (src < 0 || src >= p.src_blocks || dst < 0 || dst >= p.dst_blocks) {
      if (threadIdx.x == 0 && blockIdx.x == 0 && kv == 0) atomicOr(p.status, PA_DEVERR_PAIR);
      continue;
    }
    const uint4* s = p.src[kv] + src * p.chunks;
    uint4* d = p.dst[kv] + dst * p.chunks;
    for (int64_t i0 = static_cast<int64_t>(blockIdx.x) * 1024; i0 < p.chunks;
         i0 += static_cast<int64_t>(gridDim.x) * 1024) {
      const int64_t i = i0 + threadIdx.x;
      uint4 v[4];
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (i + k * 256 < p.chunks) v[k] = s[i + k * 256];
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (i + k * 256 < p.chunks) d[i + k * 256] = v[k];
    }
    if (blockIdx.x == 0) {
      for (int h = threadIdx.x; h < p.Hkv; h += 256)
        p.dst_scales[kv][dst * p.Hkv + h] = p.src_scales[kv][src * p.Hkv + h];
    }
  }
}

int log2_of(int x) {
  int r = 0;
  while ((1 << r) < x) ++r;
  return r;
}

// List positions a warp looks after: one when the launch is small enough that
// the warps which find nothing to do cost nothing (a decode step: every
// position starts a block's run of its own), else a block's worth.
int positions_per_warp(int num_tokens, int Hkv, int block_size) {
  return static_cast<int64_t>(num_tokens) * Hkv <= 16384 ? 1 : block_size;
}

template <typename T>
int launch_append_t(const AppendParams& p, int D, cudaStream_t st) {
  const int64_t runs = (static_cast<int64_t>(p.num_tokens) + p.positions - 1) / p.positions;
  const int64_t items = runs * p.Hkv * 2;
  const int64_t ctas = (items + kWarps - 1) / kWarps;
  if (ctas > 0x7fffffff) return cudaErrorInvalidValue;
  if (D == 64)
    append_block_kernel<T, 64><<<static_cast<unsigned>(ctas), 32 * kWarps, 0, st>>>(p);
  else
    append_block_kernel<T, 128><<<static_cast<unsigned>(ctas), 32 * kWarps, 0, st>>>(p);
  return cudaGetLastError();
}

}  // namespace

int launch_append_block(const void* key, const void* value, void* k_cache, void* v_cache,
                        float* k_scales, float* v_scales, const int64_t* slot_mapping,
                        int num_tokens, int Hkv, int D, int block_size, int num_blocks,
                        pa_dtype dtype, unsigned int* status, void* stream) {
  AppendParams p;
  p.x[0] = key;
  p.x[1] = value;
  p.cache[0] = static_cast<uint8_t*>(k_cache);
  p.cache[1] = static_cast<uint8_t*>(v_cache);
  p.scales[0] = k_scales;
  p.scales[1] = v_scales;
  p.slots = slot_mapping;
  p.status = status;
  p.num_slots = static_cast<int64_t>(num_blocks) * block_size;
  p.num_tokens = num_tokens;
  p.Hkv = Hkv;
  p.log2_bs = log2_of(block_size);
  p.positions = positions_per_warp(num_tokens, Hkv, block_size);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  switch (dtype) {
    case PA_F32: return launch_append_t<float>(p, D, st);
    case PA_F16: return launch_append_t<__half>(p, D, st);
    case PA_BF16: return launch_append_t<__nv_bfloat16>(p, D, st);
    default: return cudaErrorInvalidValue;
  }
}

int launch_copy_block_scaled(const CopyScaled& c, unsigned int* status, void* stream) {
  CopyParams p;
  for (int i = 0; i < 2; ++i) {
    p.dst[i] = static_cast<uint4*>(c.dst[i]);
    p.src[i] = static_cast<const uint4*>(c.src[i]);
    p.dst_scales[i] = c.dst_scales[i];
    p.src_scales[i] = c.src_scales[i];
  }
  p.pairs = c.pairs;
  p.status = status;
  p.src_blocks = c.src_blocks;
  p.dst_blocks = c.dst_blocks;
  p.chunks = static_cast<int64_t>(c.Hkv) * c.block_size * c.D / 16;
  p.num_pairs = c.num_pairs;
  p.Hkv = c.Hkv;
  int64_t gx = (p.chunks + 1023) / 1024;
  if (gx > 1024) gx = 1024;
  const int gy = c.num_pairs < 65535 ? c.num_pairs : 65535;
  copy_block_scaled_kernel<<<dim3(static_cast<unsigned>(gx), static_cast<unsigned>(gy), 2), 256, 0,
                             static_cast<cudaStream_t>(stream)>>>(p);
  return cudaGetLastError();
}

}  // namespace pa
