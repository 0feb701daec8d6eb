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
//   old  = the stored scale, as the decode reads it; 0 if the call writes offset 0
//          of the block, which starts the block anew
//   new  = max(old, need);  code = E4M3(x / new), saturating at 448
//   if new > old > 0: the block's other slots, code := E4M3(code * old / new)
//
// E4M3 is a floating format: the relative step of a code is the same wherever
// its scale puts it, so a power of two costs no precision and makes the
// rescaling of the older codes exact except where it reaches the subnormals.
#include <cuda_runtime.h>

#include <cstdint>
#include <type_traits>

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

// A stored scale (negative and NaN taken as 0) as the decode kernels read it; 0
// stays 0, its codes are no tokens yet.  What the append stores is at least the
// stored one, so one above the bound stays as the caller set it, and its codes are
// relative to the bound.
__device__ __forceinline__ float as_read(float stored) {
  return stored > 0.f ? fminf(fmaxf(stored, kScaleMin), kScaleMax) : 0.f;
}

__device__ __forceinline__ uint32_t codes2(float a, float b) {
  return static_cast<uint32_t>(
      __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3));
}

// Codes of 4 floats, the first in the low byte.
__device__ __forceinline__ uint32_t codes4(const float* f) {
  return codes2(f[0], f[1]) | (codes2(f[2], f[3]) << 16);
}

// max |x| over 16-byte chunks, NaNs aside, gathered as bits.  16-bit types:
// magnitudes compare as integers, two at a time, without widening (which would
// take registers for all the widened elements); a NaN's bits are above
// infinity's, and bits_max() then says so by NaN.  32-bit: fmax drops NaNs.
template <typename T>
__device__ __forceinline__ void gather_max(uint32_t& m, const uint4& v) {
  if constexpr (sizeof(T) == 2) {
    m = __vmaxu2(m, __vmaxu2(__vmaxu2(v.x & 0x7fff7fffu, v.y & 0x7fff7fffu),
                             __vmaxu2(v.z & 0x7fff7fffu, v.w & 0x7fff7fffu)));
  } else {
    const float a = fmaxf(fabsf(__uint_as_float(v.x)), fabsf(__uint_as_float(v.y)));
    const float b = fmaxf(fabsf(__uint_as_float(v.z)), fabsf(__uint_as_float(v.w)));
    m = __float_as_uint(fmaxf(__uint_as_float(m), fmaxf(a, b)));
  }
}
template <typename T>
__device__ __forceinline__ float bits_max(uint32_t m) {
  if constexpr (sizeof(T) == 4) return __uint_as_float(m);
  const uint32_t most = max(m & 0xffffu, m >> 16);
  return std::is_same<T, __nv_bfloat16>::value
             ? __uint_as_float(most << 16)
             : __half2float(__ushort_as_half(static_cast<unsigned short>(most)));
}
// The same of one chunk where there are NaNs.
template <typename T>
__device__ __forceinline__ float plain_max(const uint4& v) {
  float f[Elem<T>::EPL], m = 0.f;
  Elem<T>::unpack(v, f);
#pragma unroll
  for (int e = 0; e < Elem<T>::EPL; ++e) m = fmaxf(m, fabsf(f[e]));
  return m;
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

// How the elements are divided by a scale: a power of two divides exactly as its
// reciprocal multiplies; f16 elements by one that f16 holds as a normal number
// stay f16 pairs (a product that f16 cannot hold exactly is below 2^-14, far
// inside the half step below E4M3's smallest code).
struct Divide {
  float by, inv;
  uint32_t inv2;       // the reciprocal as an f16 pair, 0: not that way
};
template <typename T>
__device__ __forceinline__ Divide divide_by(float scale) {
  Divide d{scale, 0.f, 0u};
  if ((__float_as_uint(scale) & 0x7fffffu) == 0) {
    d.inv = __frcp_rn(scale);
    if (std::is_same<T, __half>::value && scale >= 0.000030517578125f && scale <= 16384.f) {
      const __half2 h = __float2half2_rn(d.inv);
      d.inv2 = *reinterpret_cast<const uint32_t*>(&h);
    }
  }
  return d;
}
__device__ __forceinline__ uint32_t codes2_h(uint32_t x, uint32_t inv2) {
  const __half2 p = __hmul2(*reinterpret_cast<const __half2*>(&x), *reinterpret_cast<const __half2*>(&inv2));
  return static_cast<uint32_t>(
      __nv_cvt_halfraw2_to_fp8x2(static_cast<__half2_raw>(p), __NV_SATFINITE, __NV_E4M3));
}
// The codes of a chunk's elements at dst.
template <typename T>
__device__ __forceinline__ void store_codes(const uint4& v, const Divide& d, uint8_t* dst) {
  constexpr int EPL = Elem<T>::EPL;
  if (std::is_same<T, __half>::value && d.inv2 != 0) {
    *reinterpret_cast<uint2*>(dst) =
        make_uint2(codes2_h(v.x, d.inv2) | (codes2_h(v.y, d.inv2) << 16),
                   codes2_h(v.z, d.inv2) | (codes2_h(v.w, d.inv2) << 16));
    return;
  }
  float f[EPL];
  Elem<T>::unpack(v, f);
  if (d.inv != 0.f) {
#pragma unroll
    for (int e = 0; e < EPL; ++e) f[e] *= d.inv;
  } else {
#pragma unroll
    for (int e = 0; e < EPL; ++e) f[e] = __fdiv_rn(f[e], d.by);
  }
  if constexpr (EPL == 8)
    *reinterpret_cast<uint2*>(dst) = make_uint2(codes4(f), codes4(f + 4));
  else
    *reinterpret_cast<uint32_t*>(dst) = codes4(f);
}

// The scale of a block grew: its codes at offsets outside `written`, a row of D
// bytes per D / 16 lanes.
template <int D>
__device__ __forceinline__ void rescale(uint8_t* rows, int bs, unsigned written, float old,
                                        float now) {
  const int lane = threadIdx.x & 31;
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

// One warp per (up to 16 positions of slot_mapping, kv head, K or V).  A block's
// tokens form a run of positions, skipped slots among them; the warp that looks
// after the first of them does them all.  One read of 32 slots tells where the
// runs begin and end and which offsets they write, except next to skipped slots:
// the block of the last slot in use before them, and of the next one behind them,
// is then looked for, the latter while the elements are loaded.
//   Several runs that end among the positions (a decode or verification step):
//   all the positions' rows are loaded at once, a row per D / EPL lanes, and a
//   run's first lane settles its scale.
//   A run that goes on, or a single one: up to 16 positions' elements are loaded
//   into registers (16 bytes per lane and load, all loads in flight together),
//   their largest found, the scale settled, the codes written.  A run that
//   goes on past the 32 slots (blocks of 32; a slot given several times) is
//   followed further, and what is past 16 positions is read again, from L2.
// Bound by memory latency, not bandwidth, until the call has a few thousand
// tokens: three dependent accesses (slots; elements and scale; codes).
// Measured (8 kv heads, head size 128, bf16 / f16): 256 tokens 4 us; 24 x 512
// tokens 21 us (75.7 MB, 3.6 TB/s).  Padding behind a batch costs its last warps a
// scan: 100 tokens and 156 skipped slots 4.4 us, 8 and 1000 8.0 us (where skipped
// slots ended a run, 4.6 and 4.1; tokens behind them were then another warp's, and
// the two raced on the block's scale and codes).
template <typename T, int D>
__global__ void __launch_bounds__(32 * kWarps, sizeof(T) == 4 ? 2 : 3)
    append_block_kernel(const AppendParams p) {
  allow_dependents();   // the decode kernels may start launching (they wait for us)
  constexpr int EPL = Elem<T>::EPL;          // elements per lane and load
  constexpr int LPR = D / EPL;               // lanes per token row
  constexpr int RPW = 32 / LPR;              // token rows per load
  constexpr int IT = kChunk / RPW;           // loads of a full chunk
  const int lane = threadIdx.x & 31;
  const uint32_t item = blockIdx.x * kWarps + (threadIdx.x >> 5);
  const int kv = static_cast<int>(item & 1);
  const int h = static_cast<int>((item >> 1) % static_cast<uint32_t>(p.Hkv));
  const int64_t at0 = static_cast<int64_t>((item >> 1) / static_cast<uint32_t>(p.Hkv)) * p.positions;
  if (at0 >= p.num_tokens) return;
  const int c0 = static_cast<int>(at0);
  const int bs = 1 << p.log2_bs;
  const int64_t x_stride = static_cast<int64_t>(p.Hkv) * D;
  const int sub = lane / LPR, col = lane % LPR * EPL;
  const T* x = static_cast<const T*>(p.x[kv]) + static_cast<int64_t>(h) * D + col;
  uint8_t* cache = p.cache[kv];
  float* scales = p.scales[kv];

  // lane i: position c0 + i, its block (-1: no slot) and offset
  auto slot_at = [&](int64_t i) -> int64_t {
    return i >= 0 && i < p.num_tokens ? __ldg(p.slots + i) : -1;
  };
  auto block_of = [&](int64_t s) -> int {
    return s >= 0 && s < p.num_slots ? static_cast<int>(s >> p.log2_bs) : -1;
  };
  const int64_t slot = slot_at(at0 + lane);
  const int64_t slot_ahead = __ldg(p.slots + (at0 > 0 ? at0 - 1 : 0));
  const int mine = block_of(slot);
  const int offset = static_cast<int>(slot) & (bs - 1);
  const bool here = lane < p.positions;
  if (here && h == 0 && kv == 0 && slot >= p.num_slots) atomicOr(p.status, PA_DEVERR_SLOT);
  // A run starts where the last slot in use before it is of another block: skipped
  // slots do not end one.  `before` is that block for the window's first slot in use.
  const unsigned used = __ballot_sync(FULL, mine >= 0);
  int before = at0 > 0 ? block_of(slot_ahead) : -1;
  if (before < 0 && at0 > 1 && (used & ((1u << p.positions) - 1u)) != 0) {
#pragma unroll 1
    for (int64_t i = at0 - 2; before < 0 && i >= 0; i -= 32) {
      const int b = block_of(slot_at(i - lane));
      const unsigned in = __ballot_sync(FULL, b >= 0);
      if (in != 0) before = __shfl_sync(FULL, b, __ffs(in) - 1);
    }
  }
  const unsigned below = used & ((1u << lane) - 1u);
  int prev = __shfl_sync(FULL, mine, below != 0 ? 31 - __clz(below) : 0);
  if (below == 0) prev = before;
  unsigned leaders = __ballot_sync(FULL, here && mine >= 0 && mine != prev);
  uint4 v[IT];

  // the first position from i on whose slot is in use (num_tokens: none); 128 slots
  // in flight (four loads a lane: eight cost the registers of the paths below)
  auto next_used = [&](int64_t i) -> int64_t {
#pragma unroll 1
    for (; i < p.num_tokens; i += 128) {
      unsigned m = 0;                        // bit k: position i + 32 k + lane
#pragma unroll
      for (int k = 0; k < 4; ++k) m |= block_of(slot_at(i + 32 * k + lane)) >= 0 ? 1u << k : 0u;
      const unsigned any = __reduce_or_sync(FULL, m);
      if (any != 0) {
        const int k = __ffs(any) - 1;
        return i + 32 * k + __ffs(__ballot_sync(FULL, (m >> k) & 1u)) - 1;
      }
    }
    return p.num_tokens;
  };
  // The runs that end among the positions, if there are several: all but the
  // last one where that goes on behind them.
  const int last = 31 - __clz(leaders);
  const unsigned later = used >> p.positions;
  const int next = __shfl_sync(FULL, mine, later != 0 ? p.positions + __ffs(later) - 1 : 0);
  const int last_block = __shfl_sync(FULL, mine, last & 31);
  const bool cross = later != 0 && next == last_block;
  unsigned many = cross && leaders != 0 ? leaders & ~(1u << last) : leaders;
  if ((many & (many - 1)) != 0) {
    // ---- row r = position c0 + r, a member of the run of the leader before it ----
    const int end = cross ? last : p.positions;
    const unsigned upto = many & (0xffffffffu >> (31 - lane));
    const bool member = lane < end && upto != 0;   // or a skipped slot between two
    const bool in = member && mine >= 0;
    unsigned rows_in = __ballot_sync(FULL, in);
    const int lead = member ? 31 - __clz(upto) : lane;
    const int64_t srow = static_cast<int64_t>(in ? mine : 0) * p.Hkv + h;
    float stored = in ? fmaxf(__ldcg(scales + srow), 0.f) : 0.f;
    {
      const T* src = x + (static_cast<int64_t>(c0) + sub) * x_stride;
#pragma unroll
      for (int k = 0; k < IT; ++k, src += RPW * x_stride)
        v[k] = (rows_in >> (k * RPW + sub)) & 1u ? __ldg(reinterpret_cast<const uint4*>(src))
                                                 : make_uint4(0, 0, 0, 0);
    }
    // nothing but skipped slots in the rest of the window: the last run may go on
    // behind them and is then not for here
    if (later == 0 && at0 + 32 < p.num_tokens &&
        block_of(slot_at(next_used(at0 + 32))) == last_block) {
      many &= ~(1u << last);
      rows_in &= (1u << last) - 1u;
    }
    float most = 0.f;                        // of position `lane`
#pragma unroll
    for (int k = 0; k < IT; ++k) {
      uint32_t bits = 0;
      gather_max<T>(bits, v[k]);
      float m = bits_max<T>(bits);
      if (isnan(m)) m = plain_max<T>(v[k]);
#pragma unroll
      for (int o = LPR / 2; o >= 1; o >>= 1) m = fmaxf(m, __shfl_xor_sync(FULL, m, o));
      m = __shfl_sync(FULL, m, (lane % RPW) * LPR);
      if (lane / RPW == k) most = m;
    }
    // the run's largest and the offsets it writes, at its leader's lane
    unsigned written = in ? 1u << offset : 0u;
#pragma unroll
    for (int o = 1; o < kChunk; o <<= 1) {
      const float m = __shfl_down_sync(FULL, most, o);
      const unsigned w = __shfl_down_sync(FULL, written, o);
      const int l = __shfl_down_sync(FULL, lead, o);
      if (lane + o < 32 && l == lead) {
        most = fmaxf(most, m);
        written |= w;
      }
    }
    if (written & 1u) stored = 0.f;
    const float old = as_read(stored);
    float now = fmaxf(old, scale_for(most));
    const bool is_lead = (many >> lane) & 1u;
    unsigned grown = __ballot_sync(FULL, is_lead && !(written & 1u) && now > old);
    if (is_lead) scales[srow] = fmaxf(stored, now);
    while (grown) {
      const int at = __ffs(grown) - 1;
      grown &= grown - 1;
      const int64_t row = __shfl_sync(FULL, srow, at);
      rescale<D>(cache + (row << p.log2_bs) * D, bs, __shfl_sync(FULL, written, at),
                 __shfl_sync(FULL, old, at), __shfl_sync(FULL, now, at));
    }
    now = __shfl_sync(FULL, now, lead);
#pragma unroll
    for (int k = 0; k < IT; ++k) {
      const int r = k * RPW + sub;
      const int b = __shfl_sync(FULL, mine, r);
      const int off = __shfl_sync(FULL, offset, r);
      const float by = __shfl_sync(FULL, now, r);
      if (((rows_in >> r) & 1u) == 0) continue;
      store_codes<T>(v[k], divide_by<T>(by), cache + (((static_cast<int64_t>(b) * p.Hkv + h) << p.log2_bs) + off) * D + col);
    }
    leaders &= ~many;
  }

  while (leaders) {                          // warp-uniform
    const int at = __ffs(leaders) - 1;
    leaders &= leaders - 1;
    const int blk = __shfl_sync(FULL, mine, at);
    // ---- the run's n positions (skipped slots among them), which of the window's and
    // of the next 32 are its tokens, and the offsets it writes ----
    const int64_t first = static_cast<int64_t>(c0) + at;
    unsigned written = 0, other = 0;
    int n = 0, offset1 = 0;                  // offset1: of position c0 + 32 + lane
    // its tokens among 32 positions from c0 + from on, up to the next one of another block
    auto take = [&](int64_t from, int b, int off, unsigned keep) -> unsigned {
      other = __ballot_sync(FULL, b >= 0 && b != blk) & keep;
      unsigned m = __ballot_sync(FULL, b == blk) & keep;
      if (other != 0) m &= (other & (0u - other)) - 1u;
      written |= __reduce_or_sync(FULL, (m >> lane) & 1u ? 1u << off : 0u);
      if (m != 0) n = static_cast<int>(from) + 32 - __clz(m) - at;
      return m;
    };
    const int64_t row0 = static_cast<int64_t>(blk) * p.Hkv + h;
    const float stored = fmaxf(__ldcg(scales + row0), 0.f);
    const unsigned tokens0 = take(0, mine, offset, FULL << at);
    unsigned tokens1 = 0;
    // lane l < kChunk: whether position first + t0 + l is a token of the run, its offset
    unsigned rows_in = 0;
    int off_in = 0;
    auto look = [&](int t0) {
      const int w = at + t0 + lane;
      off_in = __shfl_sync(FULL, offset, w & 31);
      bool in = w < 32 && ((tokens0 >> (w & 31)) & 1u) != 0;
      if (at + t0 + kChunk > 32) {
        const int o = __shfl_sync(FULL, offset1, w & 31);
        if (w >= 32) {
          off_in = o;
          in = w < 64 && ((tokens1 >> (w & 31)) & 1u) != 0;
          if (w >= 64 && t0 + lane < n) {    // read again, from L1 or L2
            const int64_t s = __ldg(p.slots + first + t0 + lane);
            in = block_of(s) == blk;
            off_in = static_cast<int>(s) & (bs - 1);
          }
        }
      }
      rows_in = __ballot_sync(FULL, lane < kChunk && in);
    };
    auto load = [&](int t0) {                // the tokens among first + t0 ..
      look(t0);
      const T* src = x + (first + t0 + sub) * x_stride;
#pragma unroll
      for (int k = 0; k < IT; ++k, src += RPW * x_stride)
        v[k] = (rows_in >> (k * RPW + sub)) & 1u ? __ldg(reinterpret_cast<const uint4*>(src))
                                                 : make_uint4(0, 0, 0, 0);
    };
    load(0);                                 // in flight while the rest of the run is found
    if (other == 0 && at0 + 32 < p.num_tokens) {
      const int64_t s = slot_at(at0 + 32 + lane);
      offset1 = static_cast<int>(s) & (bs - 1);
      tokens1 = take(32, block_of(s), offset1, FULL);
#pragma unroll 1
      for (int64_t i = at0 + 64; other == 0 && (i = next_used(i)) < p.num_tokens; i += 32) {
        const int64_t t = slot_at(i + lane);
        take(i - at0, block_of(t), static_cast<int>(t) & (bs - 1), FULL);
      }
    }
    const bool fresh = (written & 1u) != 0;
    uint8_t* rows = cache + (row0 << p.log2_bs) * D;
    const float old = fresh ? 0.f : as_read(stored);

    float most = 0.f;
    for (int t0 = 0; t0 < n; t0 += kChunk) {
      if (t0 > 0) load(t0);
      uint32_t bits = 0;
#pragma unroll
      for (int k = 0; k < IT; ++k) gather_max<T>(bits, v[k]);
      float m = bits_max<T>(bits);
      if (isnan(m)) {
        m = 0.f;
#pragma unroll
        for (int k = 0; k < IT; ++k) m = fmaxf(m, plain_max<T>(v[k]));
      }
      most = fmaxf(most, m);
    }
    most = __uint_as_float(__reduce_max_sync(FULL, __float_as_uint(most)));   // >= 0: ordered as bits
    const float now = fmaxf(old, scale_for(most));
    if (now > old && !fresh) rescale<D>(rows, bs, written, old, now);
    if (lane == 0) scales[row0] = fresh ? now : fmaxf(stored, now);
    const Divide div = divide_by<T>(now);
    for (int t0 = 0; t0 < n; t0 += kChunk) {
      if (n > kChunk) load(t0);
#pragma unroll
      for (int k = 0; k < IT; ++k) {
        const int r = k * RPW + sub;
        const int off = __shfl_sync(FULL, off_in, r);
        if (((rows_in >> r) & 1u) == 0) continue;
        store_codes<T>(v[k], div, rows + off * D + col);
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
// and scales, between any memories that the GPU addresses (swap); blockIdx.z
// selects K or V, a thread moves four 16-byte chunks with all four loads in flight.
__global__ void __launch_bounds__(256) copy_block_scaled_kernel(const CopyParams p) {
  allow_dependents();
  const int kv = blockIdx.z;
  for (int64_t pr = blockIdx.y; pr < p.num_pairs; pr += gridDim.y) {
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

// The same within device memory, through shared memory with bulk copies: a warp
// keeps kStages pieces of up to 16 KB in flight, each loaded by one instruction
// and stored by another as soon as it has landed, so that no register or issue
// slot carries the data.  A second warp copies the scales.
// Bound by HBM: 8192 blocks of 32 KB (538 MB read and written) in 92 us, 5.8
// TB/s (107 us with four 16-byte loads and stores per thread).
constexpr int kPiece = 16384;
constexpr int kStages = 6;

__device__ __forceinline__ void bulk_store(void* gmem_dst, const void* smem_src, uint32_t bytes) {
  asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(gmem_dst),
               "r"(smem_addr(smem_src)), "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void bulk_commit() {
  asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}
// Until at most N of this thread's latest store groups still read shared memory.
template <int N>
__device__ __forceinline__ void bulk_wait_read() {
  asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(N) : "memory");
}

__global__ void __launch_bounds__(64) copy_block_bulk_kernel(const CopyParams p) {
  allow_dependents();
  extern __shared__ __align__(128) uint8_t ring[];
  __shared__ uint64_t full[kStages];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (warp == 1) {
    const int64_t n = static_cast<int64_t>(p.num_pairs) * p.Hkv;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * 32 + lane; i < n;
         i += static_cast<int64_t>(gridDim.x) * 32) {
      const int64_t pr = i / p.Hkv, h = i - pr * p.Hkv;
      const int64_t src = __ldg(p.pairs + 2 * pr), dst = __ldg(p.pairs + 2 * pr + 1);
      if (src < 0 || src >= p.src_blocks || dst < 0 || dst >= p.dst_blocks) {
        if (h == 0) atomicOr(p.status, PA_DEVERR_PAIR);
        continue;
      }
      const float k = p.src_scales[0][src * p.Hkv + h], v = p.src_scales[1][src * p.Hkv + h];
      p.dst_scales[0][dst * p.Hkv + h] = k;
      p.dst_scales[1][dst * p.Hkv + h] = v;
    }
    return;
  }
  if (lane == 0) {
    for (int s = 0; s < kStages; ++s) mbar_init(&full[s], 1);
    fence_mbar_init();
  }
  __syncwarp();
  // item i of this CTA: piece c of pair pr of cache kv, in that order from slow to fast
  const int64_t block_bytes = p.chunks * 16;
  const int pieces = static_cast<int>((block_bytes + kPiece - 1) / kPiece);
  const int64_t total = static_cast<int64_t>(p.num_pairs) * 2 * pieces;
  const int64_t mine =
      total > blockIdx.x ? (total - blockIdx.x + gridDim.x - 1) / gridDim.x : 0;
  int64_t src_at = 0, dst_at = 0;      // lane l: item 32 g + l of the group last looked up
  uint32_t bytes_at = 0;               // 0: nothing to copy (a bad pair)
  const char* from = nullptr;
  char* to = nullptr;
  auto look_up = [&](int64_t i) {      // every lane its item of the group that i begins
    const int64_t item = (i + lane) * gridDim.x + blockIdx.x;
    bytes_at = 0;
    if (item >= total) return;
    const int64_t pr = item / (2 * pieces);
    const int rest = static_cast<int>(item - pr * 2 * pieces), kv = rest / pieces, c = rest % pieces;
    const int64_t src = __ldg(p.pairs + 2 * pr), dst = __ldg(p.pairs + 2 * pr + 1);
    if (src < 0 || src >= p.src_blocks || dst < 0 || dst >= p.dst_blocks) return;
    src_at = src * block_bytes + static_cast<int64_t>(c) * kPiece;
    dst_at = dst * block_bytes + static_cast<int64_t>(c) * kPiece;
    from = reinterpret_cast<const char*>(p.src[kv]);
    to = reinterpret_cast<char*>(p.dst[kv]);
    bytes_at = static_cast<uint32_t>(min(block_bytes - static_cast<int64_t>(c) * kPiece,
                                         static_cast<int64_t>(kPiece)));
  };
  // what each stage holds, known to lane 0
  char* target[kStages];
  uint32_t size[kStages];
  auto load = [&](int64_t i, int s) {  // item i into stage s (i ascends over the calls)
    if ((i & 31) == 0) look_up(i);
    const int l = static_cast<int>(i & 31);
    const uint32_t n = __shfl_sync(FULL, bytes_at, l);
    const char* f = reinterpret_cast<const char*>(
        __shfl_sync(FULL, reinterpret_cast<unsigned long long>(from + src_at), l));
    char* t = reinterpret_cast<char*>(
        __shfl_sync(FULL, reinterpret_cast<unsigned long long>(to + dst_at), l));
    target[s] = t;
    size[s] = n;
    if (lane == 0) {
      mbar_arrive_expect_tx(&full[s], n);
      if (n > 0) bulk_load(ring + s * kPiece, f, n, &full[s]);
    }
  };
  bool ok = true;
  for (int s = 0; s < kStages; ++s)
    if (s < mine) load(s, s);
  for (int64_t i0 = 0; i0 < mine && ok; i0 += kStages) {
#pragma unroll
    for (int s = 0; s < kStages; ++s) {
      const int64_t i = i0 + s;
      if (i >= mine || !ok) break;
      if (lane == 0) {
        ok = mbar_wait(&full[s], static_cast<uint32_t>(i0 / kStages) & 1, p.status);
        if (ok && size[s] > 0) bulk_store(target[s], ring + s * kPiece, size[s]);
        bulk_commit();
      }
      ok = __all_sync(FULL, ok);
      // the stage of the item before: its store has read it; refill it
      if (ok && i >= 1 && i - 1 + kStages < mine) {
        if (lane == 0) bulk_wait_read<1>();
        __syncwarp();
        load(i - 1 + kStages, (s + kStages - 1) % kStages);
      }
    }
  }
  if (lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
  if (!ok && lane == 0) {   // wait (bounded) for copies still in flight
    for (int s = 0; s < kStages; ++s) {
      mbar_wait(&full[s], 0, p.status, 1000000);
      mbar_wait(&full[s], 1, p.status, 1000000);
    }
  }
}

int num_sms() {
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0)
    return 148;
  return n;
}

int log2_of(int x) {
  int r = 0;
  while ((1 << r) < x) ++r;
  return r;
}

// List positions a warp looks after (1 .. 16): as many as still give the SMs six
// warps each: enough to have the loads of a short call in flight at once, and
// fewer warps that read the same slots.  Decode steps of 256 / 512 / 1024 / 2048
// tokens (8 kv heads) take 4.0 / 4.4 / 5.2 / 6.4 us so, 5.9 / 7.7 / 8.2 / 9.0 with
// sixteen warps each; 4096 tokens 12.0 / 11.7.
int positions_per_warp(int num_tokens, int Hkv) {
  const int64_t items = static_cast<int64_t>(num_tokens) * Hkv * 2;
  const int64_t least = 6ll * num_sms();
  int n = 1;
  while (n < kChunk && items / (2 * n) >= least) n *= 2;
  return n;
}

template <typename T>
int launch_append_t(const AppendParams& p, int D, cudaStream_t st) {
  const int64_t runs = (static_cast<int64_t>(p.num_tokens) + p.positions - 1) / p.positions;
  const int64_t items = runs * p.Hkv * 2;      // below 2^31 (num_tokens * Hkv < 2^30)
  const int64_t ctas = (items + kWarps - 1) / kWarps;
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
  p.positions = positions_per_warp(num_tokens, Hkv);
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
  if (c.device) {
    constexpr int smem = kStages * kPiece;
    const cudaError_t e =
        cudaFuncSetAttribute(copy_block_bulk_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    const int64_t items = static_cast<int64_t>(c.num_pairs) * 2 * ((p.chunks * 16 + kPiece - 1) / kPiece);
    const int64_t most = 2ll * num_sms();
    copy_block_bulk_kernel<<<static_cast<unsigned>(items < most ? items : most), 64, smem,
                             static_cast<cudaStream_t>(stream)>>>(p);
    return cudaGetLastError();
  }
  int64_t gx = (p.chunks + 1023) / 1024;
  if (gx > 1024) gx = 1024;
  const int gy = c.num_pairs < 65535 ? c.num_pairs : 65535;
  copy_block_scaled_kernel<<<dim3(static_cast<unsigned>(gx), static_cast<unsigned>(gy), 2), 256, 0,
                             static_cast<cudaStream_t>(stream)>>>(p);
  return cudaGetLastError();
}

}  // namespace pa
