// paged_decode.cu -- xattn_paged_decode: attention of one new token per request
// over a paged key-value cache.
//
// For a request of n tokens and a KV head with its g query heads:
//   s[h, t] = q_h . k_t / sqrt(d),  o_h = sum_t e^(s - lse_h) v_t,  lse_h = log sum_t e^s.
// K and V are read once, which bounds the call: 2 * d * esize bytes a token
// against 4 * g * d flops, g flops a byte in bf16 (26 TFLOP/s at the measured
// copy rate for g = 4). Measured, 32 query and 8 KV heads of 128 in bf16: one
// request of 131072 tokens 87.0 us (6.2 TB/s, 94 % of the copy rate), 64 of up to
// 8192 161 us (95 %), one of 517 8.6 us.
//
// Work split. A unit is a request's KV head; its tokens are cut into tiles of
// kWarps * kChunk. Three ways, chosen on the host by what the table can hold:
//  * Ranges. The tiles of all units are numbered in a row (and each unit counts
//    two more, for what it costs beyond them), and each CTA takes an equal range,
//    whatever the lengths: one long request and many ragged ones load the GPU
//    alike. A unit inside one CTA's range is written
//    straight to O; one that several CTAs share leaves a partial result
//    (the weights' reference, their sum, unnormalised o) in the workspace, at most two a
//    CTA, and a second kernel, launched with programmatic stream
//    serialization, joins them in CTA order.
//  * Units. Each unit goes to a CTA, or to a cluster of CTAs whose results meet
//    through distributed shared memory: one launch, no scan of the lengths and
//    no workspace. For tables of so few tokens that latency is all (one request
//    of 517 tokens: 8.6 us, 9.8 in ranges), and for many more units than the GPU
//    has room for, which the block scheduler balances (256 requests of up to 500
//    tokens, 8 KV heads: 49.4 us, 55.2 in ranges; of up to 2000: 161.6 and 168.8);
//    the latter only where no unit can be long, as one CTA would be left with it
//    (60000 tokens among 255 x 200: 632 us by units, 84 in ranges).
//  * Warps. Each unit goes to one warp, whose tiles are single chunks: the warps
//    share nothing, and the four units of a CTA overlap. For many units of few
//    tokens, which a CTA would start, join and end for too little (1024 requests of
//    up to 100 tokens: 47.0 us, 86.1 with a CTA a unit; 512 of up to 250: 50.0 and
//    58.6, in fp32 93 and 111; but 512 of up to 500: 92 and 88, and of up to 1000,
//    d = 64: 96 and 88, as the warps that are left at the end load little). Where the
//    table could hold long requests and there are as many units, the split by ranges
//    looks at the lengths and gives each warp the units that begin in its own equal
//    range (1024 of up to 100: 60 us, 90 by CTAs' ranges; 512 of up to 130: 45 and 53;
//    512 of up to 60 in fp32: 41 and 75; at the bound 800 of up to 250: 96 and 94, 512 of
//    up to 250 with d = 64: 37 and 41).
// All work the bounds out on the device from lens, so a captured graph follows
// the lengths.
//
// Inside a CTA with a unit the warps take the tile's chunks, each with its own running
// maximum, sum and o; they meet once at the end of a unit. A warp's K and V come
// by TMA through a ring of stages in shared memory of its own, so a stage
// passes between a warp's lanes only: no CTA-wide barrier in the loop, and the
// copies run ahead across unit boundaries.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <type_traits>

#include "host.cuh"
#include "paged.cuh"
#include "ptx.cuh"

namespace xattn {
namespace {

using host::make_pages_map;

constexpr int kWarps = 4;
constexpr int kMaxCtas = 640;  // of the split by ranges (bounds the workspace)
// What a unit costs a CTA beyond its tiles (Q, the join of the warps, the result),
// in tiles. Ranges of equal tiles alone end far apart where short requests lie
// together (256 requests of up to 500 tokens in a wide table: 66 us; with a cost of
// 1, 2, 3 tiles a unit 57.6, 55.3, 55.9; 8 of up to 2500: 18.6; 18.0, 17.6, 17.1).
constexpr int kUnitCost = 2;
// By warps: no unit of more tokens than this, and so many units a CTA at least.
constexpr int kAloneTokens = 288, kAloneWaves = 2;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kLead = 8.0f;  // of a weight's reference over the maximum, in powers of two

// What the join has to know of a unit: its first CTA and how many CTAs follow
// it. One entry per unit, or one per first CTA where there are more units.
struct Split {
  int request, head, first, more;
};

struct DecodeArgs {
  PagedDims D;
  int hc, per;  // chunks the group's heads are cut into, and heads in a chunk
  bool by_unit;  // Split entries are indexed by unit
  int cluster;   // CTAs a unit (the split by units)
  int sms;
  const void *Q, *k_pages, *v_pages;
  const int32_t *table, *lens;
  void* O;
  float* lse;
  int* status;
  // workspace: per CTA a Split and two partial results of `per` heads
  Split* split;
  float2* part_ml;  // [CTA][2][per]: reference of the weights (base 2) and sum
  float* part_o;    // [CTA][2][per][d]
};

__device__ __forceinline__ int clamped(const DecodeArgs& a, int len) {
  return min(max(len, 0), a.D.max_pages << a.D.page_shift);
}
__device__ __forceinline__ Split* split_of(const DecodeArgs& a, int request, int head, int part) {
  return a.split +
         (a.by_unit ? (request * a.D.hkv + head) * a.hc + part : static_cast<int>(blockIdx.x));
}

__device__ __forceinline__ void read16(uint32_t src, uint32_t* r) {
  asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(src)
               : "memory");
}

__device__ __forceinline__ void ldmatrix(uint32_t src, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(src)
               : "memory");
}
__device__ __forceinline__ void ldmatrix_trans(uint32_t src, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(src)
               : "memory");
}

__device__ __forceinline__ void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// Transposes an 8 x 8 matrix of 16-bit values held by the warp.
__device__ __forceinline__ uint32_t transpose8x8(uint32_t v) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}

// ------------------------------------------------------------ bf16 core
// A warp's chunk is 16 tokens, NT * 8 heads. Tokens are the rows of both
// products, so that no matrix row is padding when the group is small:
//   S^T [16 tokens, 8 heads] = K Q^T  and  O^T [d, 8 heads] += V^T P^T
// with mma.sync m16n8k16 (d / 16 instructions each per 8 heads). tcgen05
// would want 64 or 128 rows behind descriptors to feed a product that needs
// 2 % of its rate, and its result back from tensor memory every chunk.
// ldmatrix brings both operands from TMA's 128-byte swizzle without bank
// conflicts, V transposed on the way; P goes from the accumulator's layout to an
// operand's with an 8x8 transpose per 8 tokens and term. A weight is the sum of two
// bf16 numbers, so V^T P^T is two products: with one, O of 64 requests of up to 8192
// tokens is off by 0.0022 of it, with two by 0.0017, which is its rounding to bf16. The
// second costs up to 16 heads a pass 0 to 4 %, 17 to 32 heads 8 to 17 % (16 requests of
// up to 65536 tokens, 2 KV heads of 32: 119.6 us and 139).
// A lane is (r, c) = (lane / 4, lane % 4): tokens r and r + 8 and heads 2c, 2c + 1 of
// S^T, features r and r + 8 of every 16 of O^T.
template <int kD, int NT>
struct CoreBf16 {
  static constexpr int kDim = kD;
  static constexpr int kChunk = 16;          // tokens of a warp's step
  static constexpr int kBox = 64;            // features of a TMA box: 128 bytes
  // CTAs an SM, and bytes of a warp's ring: 96 or 128 KB of copies under way an
  // SM. With 192 KB every page id and Q row queues 4 us behind them, and DRAM is
  // no faster (24 KB rings against 16: one 128K request 91.4 against 86.9 us, two
  // of 76800 tokens without shared heads 200.4 against 193.6).
  static constexpr int kCtas = kD == 128 ? 2 : 3, kRing = kD == 128 ? 16384 : 8192;
  static constexpr int kStage = 2 * kChunk * kD * 2;   // K, then V, box after box
  static constexpr int kParts = NT;                  // a warp's result is joined in parts,
  static constexpr bool kSpread = true;              // each in another warp,
  static constexpr int kBuf = (kD / 16 + 1) * 512;   // of this size
  using T = __nv_bfloat16;

  // Q: in registers for up to 8 heads. For more it would take half of them, and
  // sits in shared memory, swizzled like K.
  static constexpr bool kQShared = NT > 1;
  static constexpr int kQBytes = kQShared ? 8 * NT * kD * 2 : 0;
  static constexpr int kQEach = kQShared ? kQBytes / 16 / (kWarps * 32) : 1;
  uint4 fetched[kQEach];
  uint32_t q[NT][kQShared ? 1 : kD / 8], q_at, p[NT][2], p_low[NT][2];
  float o[NT][kD / 16][4], m[NT][2], base[NT][2], l[NT][2];
  int r, c;
  // This lane's row of the four 8x8 matrices of an ldmatrix, at the first 16
  // features; the next 16 are a xor with 32 further.
  uint32_t k_at, v_at;

  __device__ __forceinline__ void init() {
    const uint32_t lane = threadIdx.x % 32;
    r = lane / 4;
    c = lane % 4;
    // K: (tokens 0-7, 8-15) x (features 0-7, 8-15); V: features vary first
    k_at = lane % 16 * 128 + ((lane / 16 ^ lane % 8) << 4);
    v_at = (lane % 8 + lane / 16 * 8) * 128 + ((lane / 8 % 2 ^ lane % 8) << 4);
  }

  // Reads the unit's Q (rows past the chunk's heads are zero); `settle` puts it
  // where the products take it from, and begins the sums.
  __device__ __forceinline__ void fetch(const DecodeArgs& a, long long q_row, int heads) {
    if constexpr (kQShared) {  // shared out over the CTA's threads
#pragma unroll
      for (int x = 0; x < kQEach; ++x) {
        const int h = (x * kWarps * 32 + threadIdx.x) / (kD / 8), piece = threadIdx.x % (kD / 8);
        fetched[x] = h < heads ? static_cast<const uint4*>(a.Q)[(q_row + h) * (kD / 8) + piece]
                               : make_uint4(0, 0, 0, 0);
      }
    } else {
      const uint32_t* x = static_cast<const uint32_t*>(a.Q) + (q_row + r) * (kD / 2) + c;
#pragma unroll
      for (int j = 0; j < kD / 8; ++j) q[0][j] = r < heads ? x[4 * j] : 0;
    }
  }
  __device__ __forceinline__ void settle(char* q_shared) {
    if constexpr (kQShared) {
#pragma unroll
      for (int x = 0; x < kQEach; ++x) {
        const int h = (x * kWarps * 32 + threadIdx.x) / (kD / 8), piece = threadIdx.x % (kD / 8);
        *reinterpret_cast<uint4*>(q_shared + h * (kD * 2) + ((piece ^ h % 8) << 4)) = fetched[x];
      }
      point_at(q_shared);
    }
    clear();
  }
  // ldmatrix of Q: features vary over all four matrices, 32 at a time
  __device__ __forceinline__ void point_at(const char* q_shared) {
    const uint32_t lane = threadIdx.x % 32;
    q_at = smem_u32(q_shared) + lane % 8 * (kD * 2) + ((lane / 8 ^ lane % 8) << 4);
  }
  // For one warp by itself, whose Q, where kQShared, has a place of its own (1024
  // requests of up to 100 tokens, 2 KV heads of 16: 26.8 us, 41.1 by CTAs).
  __device__ __forceinline__ void settle_alone(const DecodeArgs& a, long long q_row, int heads,
                                               char* q_own) {
    if constexpr (kQShared) {
      const int lane = threadIdx.x % 32;
      __syncwarp();  // every lane is done with the last unit's
#pragma unroll 8
      for (int x = lane; x < kQBytes / 16; x += 32) {
        const int h = x / (kD / 8), piece = x % (kD / 8);
        const uint4 y = h < heads ? static_cast<const uint4*>(a.Q)[(q_row + h) * (kD / 8) + piece]
                                  : make_uint4(0, 0, 0, 0);
        *reinterpret_cast<uint4*>(q_own + h * (kD * 2) + ((piece ^ h % 8) << 4)) = y;
      }
      __syncwarp();
      point_at(q_own);
      clear();
    } else {
      settle(nullptr);
    }
  }
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int t = 0; t < NT; ++t) {
#pragma unroll
      for (int i = 0; i < kD / 16; ++i)
#pragma unroll
        for (int x = 0; x < 4; ++x) o[t][i][x] = 0.0f;
#pragma unroll
      for (int x = 0; x < 2; ++x) m[t][x] = -INFINITY, base[t][x] = 0.0f, l[t][x] = 0.0f;
    }
  }

  __device__ __forceinline__ void scores(uint32_t stage, int valid) {
    const float scale = kLog2e * (kD == 64 ? 0.125f : 0.08838834764831845f);  // log2(e) / sqrt(d)
    // with few heads, even and odd steps of 16 features sum apart: chains half as long
    float s[NT][4], s1[1][4];
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int j = 0; j < 4; ++j) s[t][j] = s1[0][j] = 0.0f;
#pragma unroll
    for (int i = 0; i < kD / 16; i += 2) {
      uint32_t k0[4], k1[4];
      ldmatrix(stage + i / 4 * (kChunk * 128) + (k_at ^ i % 4 * 32), k0);
      ldmatrix(stage + i / 4 * (kChunk * 128) + (k_at ^ (i + 1) % 4 * 32), k1);
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        uint32_t y[4];
        if constexpr (kQShared) {
          // features 16 i .. + 31: pieces 2 i .. + 3, xor'ed with the head in their low 3 bits
          ldmatrix((q_at ^ i % 4 * 32) + i / 4 * 128 + t * (8 * kD * 2), y);
        } else {
#pragma unroll
          for (int j = 0; j < 4; ++j) y[j] = q[t][2 * i + j];
        }
        mma_bf16(s[t], k0[0], k0[1], k0[2], k0[3], y[0], y[1]);
        mma_bf16(NT == 1 ? s1[0] : s[t], k1[0], k1[1], k1[2], k1[3], y[2], y[3]);
      }
    }
#pragma unroll
    for (int t = 0; t < NT; ++t) {
#pragma unroll
      for (int j = 0; j < 4; ++j) s[t][j] = (NT == 1 ? s[t][j] + s1[0][j] : s[t][j]) * scale;
      if (valid < kChunk) {
        if (r >= valid) s[t][0] = s[t][1] = -INFINITY;
        if (r + 8 >= valid) s[t][2] = s[t][3] = -INFINITY;
      }
    }
    // The reference m that a weight is taken against is set to kLead above the
    // maximum so far, and set again (o and l are rescaled) only when a logit passes
    // it, which after a few chunks hardly happens. So no weight is above the one
    // against the maximum itself, 1 at most, and products with large values overflow
    // no earlier than with those; the largest is 2^-kLead at least, fp32 holds weights
    // down to 2^-118 of it, and their rounding is relative.
    bool grow = false;
#pragma unroll
    for (int t = 0; t < NT; ++t)
      grow = grow || fmaxf(s[t][0], s[t][2]) > m[t][0] || fmaxf(s[t][1], s[t][3]) > m[t][1];
    if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
      for (int t = 0; t < NT; ++t) {
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          float top = fmaxf(s[t][x], s[t][x + 2]);
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 4));
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 8));
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 16));
          rescale(t, x, top + kLead);
        }
      }
    }
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      float w[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) w[j] = ex2(s[t][j] - base[t][j & 1]);
      l[t][0] += w[0] + w[2];
      l[t][1] += w[1] + w[3];
      // The tensor cores take bf16: a weight goes to them cut to 8 bits, and what
      // that leaves, rounded, as a second term; together off by 2^-16 of it at
      // most. The sum keeps the fp32 one. The second term of a weight above zero is
      // above zero (where nothing is left 2^-17 of it and the smallest weight, 2^-126),
      // so that a value of infinity stays one: times 0 or times a negative term it
      // would make a NaN.
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        float low[2];
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          const float u = w[2 * x + y];
          const float cut = __uint_as_float(__float_as_uint(u) & 0xffff0000u);
          low[y] = fmaxf(u - cut, fminf(u, fmaf(u, 0x1p-17f, 0x1p-126f)));
        }
        p[t][x] = transpose8x8(
            __byte_perm(__float_as_uint(w[2 * x]), __float_as_uint(w[2 * x + 1]), 0x7632));
        p_low[t][x] = transpose8x8(pack_bf16x2(low[0], low[1]));
      }
    }
  }

  // Takes the reference of head (t, x) up to `top`.
  __device__ __forceinline__ void rescale(int t, int x, float top) {
    top = fmaxf(top, m[t][x]);
    base[t][x] = top == -INFINITY ? 0.0f : top;
    const float f = ex2(m[t][x] - base[t][x]);
    m[t][x] = top;
    l[t][x] *= f;
#pragma unroll
    for (int i = 0; i < kD / 16; ++i) {
      o[t][i][x] *= f;
      o[t][i][x + 2] *= f;
    }
  }

  __device__ __forceinline__ void values(uint32_t stage, int valid) {
#pragma unroll
    for (int i = 0; i < kD / 16; ++i) {
      uint32_t v[4];
      ldmatrix_trans(stage + kStage / 2 + i / 4 * (kChunk * 128) + (v_at ^ i % 4 * 32), v);
      if (valid < kChunk) {  // a weight of 0 does not undo a NaN or infinity
        const uint32_t low = 2 * c < valid ? (2 * c + 1 < valid ? ~0u : 0xffffu) : 0;
        const uint32_t high = 2 * c + 8 < valid ? (2 * c + 9 < valid ? ~0u : 0xffffu) : 0;
        v[0] &= low, v[1] &= low, v[2] &= high, v[3] &= high;
      }
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        mma_bf16(o[t][i], v[0], v[1], v[2], v[3], p_low[t][0], p_low[t][1]);
        mma_bf16(o[t][i], v[0], v[1], v[2], v[3], p[t][0], p[t][1]);
      }
    }
  }

  // Part t of a warp's result to and from a buffer; each lane's share is its own.
  __device__ __forceinline__ void put(float4* buf, int t) const {
    buf += threadIdx.x % 32;
#pragma unroll
    for (int i = 0; i < kD / 16; ++i)
      buf[i * 32] = make_float4(o[t][i][0], o[t][i][1], o[t][i][2], o[t][i][3]);
    buf[kD / 16 * 32] = make_float4(m[t][0], m[t][1], l[t][0], l[t][1]);
  }
  __device__ __forceinline__ void merge(const float4* buf, int t, int) {
    buf += threadIdx.x % 32;
    const float4 ml = buf[kD / 16 * 32];
    rescale(t, 0, ml.x);
    rescale(t, 1, ml.y);
    const float f0 = ex2(ml.x - base[t][0]), f1 = ex2(ml.y - base[t][1]);
    l[t][0] += ml.z * f0;
    l[t][1] += ml.w * f1;
#pragma unroll
    for (int i = 0; i < kD / 16; ++i) {
      const float4 y = buf[i * 32];
      o[t][i][0] += y.x * f0;
      o[t][i][1] += y.y * f1;
      o[t][i][2] += y.z * f0;
      o[t][i][3] += y.w * f1;
    }
  }

  // Part t of the unit's result: to O and lse, or as the partial result at `slot`.
  __device__ __forceinline__ void emit(const DecodeArgs& a, long long q_row, int heads, bool whole,
                                       long long slot, int t) {
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      float sum = l[t][x];
      sum += __shfl_xor_sync(0xffffffffu, sum, 4);
      sum += __shfl_xor_sync(0xffffffffu, sum, 8);
      sum += __shfl_xor_sync(0xffffffffu, sum, 16);
      const int h = 8 * t + 2 * c + x;
      if (h >= heads) continue;
      if (whole) {
        const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
        T* out = static_cast<T*>(a.O) + (q_row + h) * kD + r;
#pragma unroll
        for (int i = 0; i < kD / 16; ++i) {
          out[16 * i] = __float2bfloat16_rn(o[t][i][x] * inv);
          out[16 * i + 8] = __float2bfloat16_rn(o[t][i][x + 2] * inv);
        }
        if (r == 0 && a.lse != nullptr)
          a.lse[q_row + h] = sum == 0.0f ? -INFINITY : base[t][x] * kLn2 + logf(sum);
      } else {
        float* out = a.part_o + (slot * a.per + h) * kD + r;
#pragma unroll
        for (int i = 0; i < kD / 16; ++i) {
          out[16 * i] = o[t][i][x];
          out[16 * i + 8] = o[t][i][x + 2];
        }
        if (r == 0) a.part_ml[slot * a.per + h] = make_float2(m[t][x], sum);
      }
    }
  }
};

// ------------------------------------------------------------ fp32 core
// CUDA cores: no tensor-core type keeps fp32's mantissa. A warp's chunk is 8
// tokens, two (g, g + 4) to each group g of 8 lanes; of every 32 features lane c
// of a group holds 4 c .. + 3, so a group reads 128 contiguous bytes at a time,
// and multiplies two features an instruction (f32x2). The 2 H dot products of a
// group are summed over its lanes by halves (a lane keeps one half of the
// values at each step and hands on the other), which takes 14 exchanges in
// place of 48 for 8 heads and leaves each logit with one owner: of head h and
// token g + 4 t it is lane (2 h + t) * 8 / (2 H) of the group, or the lane of the
// head for 8 heads, with both tokens. So a weight's exponential is taken once, and
// handed to the group. (16 requests of up to 16384 tokens, 16 heads a KV head of 64:
// 69.9 us; with a sum for every lane, FMAs of one feature and passes of 4 heads 88.7.)
template <int kD, int H>
struct CoreF32 {
  static constexpr int kDim = kD;
  static constexpr int kChunk = 8;
  static constexpr int kBox = kD;
  static constexpr int kCtas = kD * H >= 512 || kD == 128 ? 2 : 3, kRing = kD == 128 ? 16384 : 8192;
  static constexpr int kPieces = kD / 32;
  static constexpr int kStage = 2 * kChunk * kD * 4;
  static constexpr int kPart = H < 2 ? 1 : 2;  // heads joined at a time
  static constexpr int kParts = H / kPart;
  static constexpr bool kSpread = false;       // (all heads' maxima come with the first)
  static constexpr int kBuf = (kPart * kPieces + 1) * 512;
  static constexpr bool kQShared = false;
  static constexpr int kQBytes = 0;
  using T = float;
  using F2 = unsigned long long;               // two floats
  static constexpr int kPairs = kD / 16;       // a lane's of one row
  static constexpr int kOwn = H == 8 ? 2 : 1;  // logits a lane owns, of one head

  F2 q[H][kPairs], o[H][kPairs];
  float m, base, l;         // of the lane's head (l: its own weights only)
  float w[kOwn], fs[2], fo[2];
  int g, c;

  __device__ __forceinline__ void init() {
    g = threadIdx.x % 32 / 8;
    c = threadIdx.x % 8;
  }
  // This group's lane that owns the logit of head h and its token t.
  __device__ __forceinline__ int owner(int h, int t) const {
    return g * 8 + (H == 8 ? h : (2 * h + t) * (4 / H));
  }
  // The sum of a value over the lanes that own logits of one head.
  __device__ __forceinline__ float over_tokens(float x) const {
    if (H < 8) x += __shfl_xor_sync(0xffffffffu, x, 4 / H);
    x += __shfl_xor_sync(0xffffffffu, x, 8);
    return x + __shfl_xor_sync(0xffffffffu, x, 16);
  }

  __device__ __forceinline__ void fetch(const DecodeArgs& a, long long q_row, int heads) {
#pragma unroll
    for (int h = 0; h < H; ++h) {
      const ulonglong2* p = reinterpret_cast<const ulonglong2*>(
                                static_cast<const float*>(a.Q) + (q_row + h) * kD) + c;
#pragma unroll
      for (int j = 0; j < kPieces; ++j) {
        const ulonglong2 y = h < heads ? p[8 * j] : make_ulonglong2(0, 0);
        q[h][2 * j] = y.x;
        q[h][2 * j + 1] = y.y;
      }
    }
  }
  __device__ __forceinline__ void settle(char*) {
    const float scale = kLog2e / sqrtf(static_cast<float>(kD));
#pragma unroll
    for (int h = 0; h < H; ++h)
#pragma unroll
      for (int j = 0; j < kPairs; ++j) q[h][j] = f2_fma(q[h][j], f2_pack(scale, scale), 0);
    clear();
  }
  __device__ __forceinline__ void settle_alone(const DecodeArgs&, long long, int, char*) {
    settle(nullptr);
  }
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int h = 0; h < H; ++h)
#pragma unroll
      for (int j = 0; j < kPairs; ++j) o[h][j] = 0;
    m = -INFINITY;
    base = 0.0f;
    l = 0.0f;
  }
  __device__ __forceinline__ void read_rows(uint32_t rows, F2 (&x)[2][kPairs]) const {
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int j = 0; j < kPieces; ++j)
        read16(rows + (g + 4 * t) * (kD * 4) + j * 128 + c * 16,
               reinterpret_cast<uint32_t*>(&x[t][2 * j]));
  }
  __device__ __forceinline__ void scores(uint32_t stage, int valid) {
    F2 k[2][kPairs];
    float s[2 * H];  // of head h and token t at 2 h + t
    read_rows(stage, k);
#pragma unroll
    for (int h = 0; h < H; ++h)
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        F2 x = 0;
#pragma unroll
        for (int j = 0; j < kPairs; ++j) x = f2_fma(q[h][j], k[t][j], x);
        float lo, hi;
        f2_unpack(x, lo, hi);
        s[2 * h + t] = lo + hi;
      }
    int n = 2 * H;
#pragma unroll
    for (int mask = 4; mask > 0; mask /= 2) {
      if (n > 1) {
        n /= 2;
        const bool upper = (c & mask) != 0;
#pragma unroll
        for (int i = 0; i < H; ++i) {
          if (i >= n) break;
          const float keep = upper ? s[i + n] : s[i], pass = upper ? s[i] : s[i + n];
          s[i] = keep + __shfl_xor_sync(0xffffffffu, pass, mask);
        }
      } else {
        s[0] += __shfl_xor_sync(0xffffffffu, s[0], mask);
      }
    }
    // the lane's tokens: both of the group, or that of its place
    if (valid < kChunk) {
      const int t = H == 8 ? 0 : c / (4 / H) % 2;
      if (g + 4 * t >= valid) s[0] = -INFINITY;
      if (kOwn == 2 && g + 4 >= valid) s[kOwn - 1] = -INFINITY;
    }
    float top = kOwn == 2 ? fmaxf(s[0], s[kOwn - 1]) : s[0];
    if (__any_sync(0xffffffffu, top > m)) {  // as in the bf16 core
      if (H < 8) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 4 / H));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 8));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 16));
      top = fmaxf(top + kLead, m);
      base = top == -INFINITY ? 0.0f : top;
      const float f = ex2(m - base);
      m = top;
      l *= f;
#pragma unroll
      for (int h = 0; h < H; ++h) scale_head(h, __shfl_sync(0xffffffffu, f, owner(h, 0)));
    }
#pragma unroll
    for (int i = 0; i < kOwn; ++i) {
      w[i] = ex2(s[i] - base);
      l += w[i];
    }
  }
  __device__ __forceinline__ void scale_head(int h, float f) {
#pragma unroll
    for (int j = 0; j < kPairs; ++j) o[h][j] = f2_fma(o[h][j], f2_pack(f, f), 0);
  }
  __device__ __forceinline__ void values(uint32_t stage, int valid) {
    F2 v[2][kPairs];
    read_rows(stage + kStage / 2, v);
    if (valid < kChunk) {  // a weight of 0 does not undo a NaN or infinity
#pragma unroll
      for (int t = 0; t < 2; ++t)
        if (g + 4 * t >= valid)
#pragma unroll
          for (int j = 0; j < kPairs; ++j) v[t][j] = 0;
    }
#pragma unroll
    for (int h = 0; h < H; ++h)
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        const float x = __shfl_sync(0xffffffffu, w[H == 8 ? t : 0], owner(h, t));
        const F2 xx = f2_pack(x, x);
#pragma unroll
        for (int j = 0; j < kPairs; ++j) o[h][j] = f2_fma(xx, v[t][j], o[h][j]);
      }
  }
  __device__ __forceinline__ void put(float4* buf, int part) const {
    buf += threadIdx.x % 32;
#pragma unroll
    for (int x = 0; x < kPart; ++x)
#pragma unroll
      for (int j = 0; j < kPieces; ++j)
        *reinterpret_cast<ulonglong2*>(&buf[(x * kPieces + j) * 32]) =
            make_ulonglong2(o[part * kPart + x][2 * j], o[part * kPart + x][2 * j + 1]);
    buf[kPart * kPieces * 32] = make_float4(m, l, 0.0f, 0.0f);
  }
  // `which` of the join's two merges (their factors serve all parts).
  __device__ __forceinline__ void merge(const float4* buf, int part, int which) {
    buf += threadIdx.x % 32;
    if (part == 0) {  // the heads' maxima and sums, all at once
      const float4 ml = buf[kPart * kPieces * 32];
      const float top = fmaxf(m, ml.x);
      base = top == -INFINITY ? 0.0f : top;
      fs[which] = ex2(m - base);
      fo[which] = ex2(ml.x - base);
      m = top;
      l = l * fs[which] + ml.y * fo[which];
    }
#pragma unroll
    for (int x = 0; x < kPart; ++x) {
      const int h = part * kPart + x;
      scale_head(h, __shfl_sync(0xffffffffu, fs[which], owner(h, 0)));
      const float f = __shfl_sync(0xffffffffu, fo[which], owner(h, 0));
#pragma unroll
      for (int j = 0; j < kPieces; ++j) {
        const ulonglong2 y = *reinterpret_cast<const ulonglong2*>(&buf[(x * kPieces + j) * 32]);
        o[h][2 * j] = f2_fma(y.x, f2_pack(f, f), o[h][2 * j]);
        o[h][2 * j + 1] = f2_fma(y.y, f2_pack(f, f), o[h][2 * j + 1]);
      }
    }
  }
  __device__ __forceinline__ void emit(const DecodeArgs& a, long long q_row, int heads, bool whole,
                                       long long slot, int part) {
    const float all = over_tokens(l);
#pragma unroll
    for (int h = part * kPart; h < (part + 1) * kPart; ++h) {
      const float sum = __shfl_sync(0xffffffffu, all, owner(h, 0));
      const float top = __shfl_sync(0xffffffffu, m, owner(h, 0));
      if (h >= heads) continue;
      const float inv = !whole ? 1.0f : sum == 0.0f ? 0.0f : 1.0f / sum;
      float* out = whole ? static_cast<float*>(a.O) + (q_row + h) * kD
                         : a.part_o + (slot * a.per + h) * kD;
#pragma unroll
      for (int j = 0; j < kPieces; ++j) {
        float x[4];
        f2_unpack(o[h][2 * j], x[0], x[1]);
        f2_unpack(o[h][2 * j + 1], x[2], x[3]);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          x[i] += __shfl_xor_sync(0xffffffffu, x[i], 8);
          x[i] += __shfl_xor_sync(0xffffffffu, x[i], 16);
        }
        if (g == j % 4)
          *reinterpret_cast<float4*>(out + j * 32 + c * 4) =
              make_float4(x[0] * inv, x[1] * inv, x[2] * inv, x[3] * inv);
      }
      if (threadIdx.x % 32 == 0) {
        if (!whole) a.part_ml[slot * a.per + h] = make_float2(top, sum);
        else if (a.lse != nullptr)
          a.lse[q_row + h] =
              sum == 0.0f ? -INFINITY : (top == -INFINITY ? 0.0f : top) * kLn2 + logf(sum);
      }
    }
  }
};

// Stages of a warp's ring.
template <class Core>
constexpr int stages_of() {
  return Core::kRing / Core::kStage < 6 ? Core::kRing / Core::kStage : 6;
}
// Shared memory of a CTA: the warps' rings (on 1024-byte boundaries, as the
// swizzle wants them), then two buffers of the join; the second is also Q's.
// By warps there is no join, and each has a Q of its own.
template <class Core, bool kAlone>
constexpr int smem_of() {
  constexpr int kJoin = Core::kBuf + (Core::kBuf > Core::kQBytes ? Core::kBuf : Core::kQBytes);
  constexpr int kOwn = kAlone ? kWarps * Core::kQBytes : 0;
  return 1024 + kWarps * stages_of<Core>() * Core::kStage + (kJoin > kOwn ? kJoin : kOwn);
}

// ------------------------------------------------------------ both kernels

// A chunk's rows, all slices (see make_pages_map).
__device__ __forceinline__ void tma_load_5d(void* dst, const CUtensorMap* map, uint64_t* bar,
                                            int token, int head, int page) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %3, %5, %6}], [%2];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(0), "r"(token), "r"(head),
      "r"(page)
      : "memory");
}

__device__ __forceinline__ void store_pair(float* p, float x, float y) {
  *reinterpret_cast<float2*>(p) = make_float2(x, y);
}
__device__ __forceinline__ void store_pair(__nv_bfloat16* p, float x, float y) {
  *reinterpret_cast<uint32_t*>(p) = pack_bf16x2(x, y);
}

// Part of a unit that a CTA has.
struct Unit {
  int left;  // of the range from this unit's first tile on
  int request, len, head, t0, steps;  // t0: its first tile here; steps: tiles here
};

// A cluster's shared memory: this address in CTA `rank` of it.
__device__ __forceinline__ const float4* in_cluster(const float4* p, int rank) {
  unsigned long long r;
  asm volatile("mapa.u64 %0, %1, %2;" : "=l"(r) : "l"(p), "r"(rank));
  return reinterpret_cast<const float4*>(r);
}

// The first request behind x that holds tokens (there is one), and its length; by a
// whole warp. Rows that wait lie between busy ones by the thousand, so a lane reads
// kRows at once (9 requests of up to 5600 tokens spread over 65536 rows, fp32: 1020 us
// row by row, 280 so, 197 side by side; among 4096 64, 39, 40). Not inlined, the
// neighbour's length too: 8 fp32 heads a pass of 64 keep their 69.8 us so, 72 with any
// part of it in the loop; 4 of 128 take 125 in place of 121 either way.
struct Busy {
  int request, len;
};
__device__ __noinline__ Busy next_busy(const int32_t* lens, int nseq, int x) {
  constexpr int kRows = 4;
  int len = lens[++x];
  if (len > 0) return {x, len};
  const int lane = threadIdx.x % 32;
#pragma unroll 1
  for (++x; x < nseq; x += 32 * kRows) {
    int y[kRows];
#pragma unroll
    for (int j = 0; j < kRows; ++j) {
      const int i = x + j * 32 + lane;
      y[j] = i < nseq ? lens[i] : 0;
    }
#pragma unroll
    for (int j = 0; j < kRows; ++j) {
      const unsigned any = __ballot_sync(0xffffffffu, y[j] > 0);
      const int first = __ffs(static_cast<int>(any)) - 1;
      if (any != 0) return {x + j * 32 + first, __shfl_sync(0xffffffffu, y[j], first)};
    }
  }
  return {nseq - 1, 1};
}

// O = 0 and lse = -inf for a request that holds nothing, by `threads` threads of
// which this is number t; and for all such requests.
template <class Core>
__device__ __forceinline__ void empty_row(const DecodeArgs& a, int request, int head, int head0,
                                          int heads, int t, int threads) {
  constexpr int kHalf = Core::kDim / 2;
  const long long row = static_cast<long long>(request) * a.D.hq + head * a.D.group + head0;
  for (int x = t; x < heads * kHalf; x += threads) {
    store_pair(static_cast<typename Core::T*>(a.O) + row * Core::kDim + 2 * x, 0.0f, 0.0f);
    if (x % kHalf == 0 && a.lse != nullptr) a.lse[row + x / kHalf] = -INFINITY;
  }
}
template <class Core>
__device__ void empty_rows(const DecodeArgs& a, int group, int groups, int part, int head0,
                           int heads) {
  for (int i = group; i < a.D.nseq; i += groups) {
    if (clamped(a, a.lens[i]) != 0) continue;
    for (int head = 0; head < a.D.hkv; ++head) {
      empty_row<Core>(a, i, head, head0, heads, threadIdx.x, kWarps * 32);
      if (a.by_unit && threadIdx.x == 0) split_of(a, i, head, part)->more = 0;
    }
  }
}

// How the work is cut (see above). kByRangesOrWarps chooses on the device; it is a
// kernel of its own since its size costs long units of 8 fp32 heads a pass, or 32 in
// bf16, registers (200 of up to 4000 tokens, 8 KV heads of 8: 362 us, 360 without the walk
// by warps; 800 of up to 4000, one of 32: 197 and 193; where the units are short, 512 of
// up to 50, 8 of 8: 38 and 93).
enum Way { kByRanges, kByRangesOrWarps, kByUnits, kByWarps };

template <class Core, Way kWay>
__global__ void __launch_bounds__(kWarps * 32, Core::kCtas) decode_kernel(
    const DecodeArgs a, const __grid_constant__ CUtensorMap k_map,
    const __grid_constant__ CUtensorMap v_map) {
  using T = typename Core::T;
  constexpr bool kUnits = kWay == kByUnits || kWay == kByWarps;
  constexpr int kTile = kWarps * Core::kChunk, kThreads = kWarps * 32;
  constexpr int kStages = stages_of<Core>();
  constexpr bool kMaybeAlone = kWay == kByRangesOrWarps;
  const PagedDims& D = a.D;
  const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
  // CTAs (clusters) b * hc .. b * hc + hc - 1 take the same tiles for different
  // heads of the group, at about the same time: the second to read a row finds
  // it in L2.
  const int block = kWay == kByWarps   ? blockIdx.x * kWarps + warp
                    : kWay == kByUnits ? blockIdx.x / a.cluster
                                       : blockIdx.x;
  const int part = block % a.hc, group = block / a.hc;
  const int head0 = part * a.per, heads = min(a.per, D.group - head0);

  extern __shared__ char s_dynamic[];
  __shared__ uint64_t s_full[kWarps][kStages];
  __shared__ int s_abort;

  if (lane < kStages) mbar_init(&s_full[warp][lane], 1);
  if (tid == 0) s_abort = 0;
  fence_barrier_init();  // a warp's barriers are used by its own lanes and the TMA unit

  // The part of the first unit that is this CTA's.
  Unit use;
  bool bad = false;
  [[maybe_unused]] unsigned total = 0, end = 0, groups = 0;  // of the split into ranges
  bool alone = kWay == kByWarps;  // a unit is a warp's, all of it
  auto tiles_of = [](int len) { return (len + kTile - 1) / kTile; };
  // The range goes on into another unit's tiles, or, alone, to another unit's start.
  auto goes_on = [&](auto alone_c, const Unit& u) {
    return alone_c() ? u.left > tiles_of(u.len) : u.left > u.steps + kUnitCost;
  };
  auto next_unit = [&](auto alone_c, Unit& u) {
    u.left -= (alone_c() ? tiles_of(u.len) : u.steps) + kUnitCost;
    u.t0 = 0;
    if (++u.head == D.hkv) {
      u.head = 0;
      const Busy to = next_busy(a.lens, D.nseq, u.request);
      u.request = to.request;
      u.len = clamped(a, to.len);
    }
    u.steps = alone_c() ? (u.len + Core::kChunk - 1) / Core::kChunk : min(tiles_of(u.len), u.left);
  };
  if constexpr (kUnits) {
    __syncthreads();  // s_abort
    const int rank = alone ? 0 : blockIdx.x % a.cluster;
    if (alone && group >= D.nseq * D.hkv) return;
    use.request = group / D.hkv;
    use.head = group % D.hkv;
    const int raw = a.lens[use.request];
    use.len = clamped(a, raw);
    if (use.len != raw && rank == 0 && lane == 0) atomicExch(a.status, kStatusBadCache);
    if (use.len == 0) {  // so for the whole cluster
      if (rank == 0)
        empty_row<Core>(a, use.request, use.head, head0, heads, alone ? lane : tid,
                        alone ? 32 : kThreads);
      return;
    }
    const unsigned tiles =
        alone ? (use.len + Core::kChunk - 1) / Core::kChunk : tiles_of(use.len);
    use.t0 = static_cast<int>(static_cast<unsigned long long>(tiles) * rank / a.cluster);
    use.steps =
        static_cast<int>(static_cast<unsigned long long>(tiles) * (rank + 1) / a.cluster) - use.t0;
    use.left = 0;
  } else {
    __shared__ unsigned s_sum[kWarps], s_before[kWarps];
    __shared__ int s_request[kWarps], s_len[kWarps], s_longest[kWarps], s_held[kWarps];
    asm volatile("griddepcontrol.launch_dependents;");
    // Where the range begins: a scan of the requests' tile counts, a run of
    // requests to each thread. (The host has made sure of fewer than 2^31 tiles.)
    auto cost_of = [&](int len) {  // in tiles; the unit's own cost comes first
      return len == 0 ? 0 : tiles_of(len) + kUnitCost;
    };
    const int launched = gridDim.x / a.hc;
    const int run = (D.nseq + kThreads - 1) / kThreads;
    const int i0 = min(tid * run, D.nseq), i1 = min(i0 + run, D.nseq);
    unsigned mine = 0;
    int len = 0;
    int longest = 0, held = 0;  // of these requests; those that hold tokens
    for (int i = i0; i < i1; ++i) {
      const int raw = a.lens[i];
      len = clamped(a, raw);
      bad = bad || len != raw;
      longest = max(longest, len);
      held += len > 0;
      mine += cost_of(len);
    }
    const bool none = held < i1 - i0;
    if (bad && blockIdx.x == 0) atomicExch(a.status, kStatusBadCache);
    bad = false;
    unsigned upto = mine;
#pragma unroll
    for (int x = 1; x < 32; x *= 2) {
      const unsigned y = __shfl_up_sync(0xffffffffu, upto, x);
      if (lane >= x) upto += y;
    }
    if (lane == 31) s_sum[warp] = upto;
    if (kMaybeAlone) {
      longest = __reduce_max_sync(0xffffffffu, longest);
      held = __reduce_add_sync(0xffffffffu, held);
      if (lane == 0) s_longest[warp] = longest, s_held[warp] = held;
    }
    const bool empty = __syncthreads_or(none);
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) upto += s_sum[w];
      total += s_sum[w];
    }
    total *= D.hkv;
    if (kMaybeAlone) {
      longest = held = 0;
      for (int w = 0; w < kWarps; ++w) longest = max(longest, s_longest[w]), held += s_held[w];
      alone = longest <= kAloneTokens && held * D.hkv >= kAloneWaves * launched;
    }
    if (empty) empty_rows<Core>(a, group, launched, part, head0, heads);
    if (!a.by_unit && tid == 0) a.split[blockIdx.x].more = 0;
    // as many ranges as there are tiles, at most: none is empty, so a unit's
    // partial results are those of consecutive CTAs; and where there are few
    // tiles, four to a CTA rather than fewer to more of them, with more results
    // to join (one request of 8192 tokens: 18.5 us with 444 CTAs, 15.5 with 256);
    // alone, one to a warp, some of which may hold no unit's start
    groups = alone ? launched * kWarps
                   : min(static_cast<unsigned>(launched),
                         max(total / 4, min(total, static_cast<unsigned>(a.sms))));
    if (!alone && group >= static_cast<int>(groups)) return;
    // range b begins at total * b / groups
    const unsigned each = total / groups, over = total % groups;
    auto begin = [&](unsigned b) { return b * each + b * over / groups; };
    const unsigned mine0 = (upto - mine) * D.hkv, mine1 = upto * D.hkv;
    for (int w = 0; w < (alone ? kWarps : 1); ++w) {
      const unsigned pos = begin(alone ? group * kWarps + w : group);
      if (pos < mine0 || pos >= mine1) continue;
      unsigned before = mine0;
      for (int i = i0; i < i1; ++i) {
        if (run > 1) len = clamped(a, a.lens[i]);
        const unsigned next = before + cost_of(len) * D.hkv;
        if (pos < next) {
          s_request[w] = i;
          s_len[w] = len;
          s_before[w] = before;
          break;
        }
        before = next;
      }
    }
    __syncthreads();
    const int w = alone ? warp : 0, range = alone ? group * kWarps + warp : group;
    const unsigned pos = begin(range);
    end = begin(range + 1);
    use.request = s_request[w];
    use.len = s_len[w];
    const unsigned cost = cost_of(use.len), at = (pos - s_before[w]) % cost;
    use.head = static_cast<int>((pos - s_before[w]) / cost);
    use.left = end - pos;
    if (alone) {  // from the first unit that begins in the range
      use.t0 = 0;
      use.left += static_cast<int>(at) - static_cast<int>(kUnitCost);
      use.steps = (use.len + Core::kChunk - 1) / Core::kChunk;
      if (pos == end) return;
      if (at > 0) {
        if (!goes_on(std::true_type(), use)) return;
        next_unit(std::true_type(), use);
      }
    } else {
      use.t0 = static_cast<int>(max(at, static_cast<unsigned>(kUnitCost)) - kUnitCost);
      const int skip = max(at, static_cast<unsigned>(kUnitCost)) - at;
      if (use.left <= skip) return;  // it ends before the unit's first tile
      use.left -= skip;
      use.steps = min(static_cast<int>(cost - kUnitCost) - use.t0, use.left);
    }
  }
  // The units from `use` on: the CTA's warps take each together, or, alone, a warp
  // the units that begin in its range.
  auto walk = [&](auto alone_c) {
    constexpr bool kAlone = decltype(alone_c)::value;
    // Two of these walk the range's units: one issues copies, the other, some
    // stages behind, uses them.
    Unit ahead = use;

    Core core;
    core.init();
    char* rings = s_dynamic + (1024 - smem_u32(s_dynamic) % 1024) % 1024;
    char* ring = rings + warp * kStages * Core::kStage;
    float4* bufs = reinterpret_cast<float4*>(rings + kWarps * kStages * Core::kStage);

    // Q before the copies, whose bytes it would queue behind
    auto q_row_of = [&](const Unit& u) {
      return static_cast<long long>(u.request) * D.hq + u.head * D.group + head0;
    };
    if (!kAlone || !Core::kQShared) core.fetch(a, q_row_of(use), heads);

    // lane x of a warp holds the page of the warp's step 32 q + x of the unit ahead
    const int per_step = kAlone ? Core::kChunk : kTile;
    const int in_step = kAlone ? 0 : warp * Core::kChunk;  // the warp's place in a step
    int step = 0, pages = -1, pages_next = -1;
    auto page_batch = [&](const Unit& u, int step0) {
      const int t = (u.t0 + step0 + lane) * per_step + in_step;
      if (step0 + lane >= u.steps || t >= u.len) return -1;
      const int page = a.table[static_cast<long long>(u.request) * D.max_pages +
                               (t >> D.page_shift)];
      if (page >= 0 && page < D.num_pages) return page;
      bad = true;
      return -1;
    };
    pages = page_batch(ahead, 0);
    pages_next = page_batch(ahead, 32);
    uint32_t valids = 0;  // rows of the chunks under way, 5 bits each, the newest lowest
    bool done = use.steps == 0;  // (a CTA of a cluster may have none)
    // Copies the warp's next chunk to a stage.
    auto issue = [&](int stage) {
      int valid = 0;
      if (!done) {
        const int page = __shfl_sync(0xffffffffu, pages, step % 32);
        const int t = (ahead.t0 + step) * per_step + in_step;
        if (page >= 0) {
          valid = min(Core::kChunk, ahead.len - t);
          __syncwarp();  // every lane is done with the stage
          if (elect_one()) {
            uint64_t* full = &s_full[warp][stage];
            char* to = ring + stage * Core::kStage;
            mbar_arrive_expect_tx(full, Core::kStage);
            tma_load_5d(to, &k_map, full, t & (D.page - 1), ahead.head, page);
            tma_load_5d(to + Core::kStage / 2, &v_map, full, t & (D.page - 1), ahead.head, page);
          }
        }
        if (++step == ahead.steps) {
          done = kUnits || !goes_on(alone_c, ahead);
          if (!done) {
            next_unit(alone_c, ahead);
            step = 0;
            pages = page_batch(ahead, 0);
            pages_next = page_batch(ahead, 32);
          }
        } else if (step % 32 == 0) {
          pages = pages_next;
          pages_next = page_batch(ahead, step + 32);
        }
      }
      valids = valids << 5 | static_cast<unsigned>(valid);
    };
    for (int x = 0; x < kStages; ++x) issue(x);

    // The warps' results of a unit, joined in a fixed order. Part x ends up in warp
    // root_of(x), so that several warps can write a unit's heads out: it takes warp
    // root ^ 2's, warp root ^ 1 takes root ^ 3's, and then root root ^ 1's.
    // (bufs[0] is read last, and is not the one that takes the next unit's Q)
    auto root_of = [](int x) { return Core::kSpread ? x % kWarps : 0; };
    auto join_warps = [&]() {
#pragma unroll
      for (int x = 0; x < Core::kParts; ++x) {
        const int to_root = warp ^ root_of(x);
        float4* buf = bufs + (1 - to_root % 2) * (Core::kBuf / 16);
        __syncthreads();
        if (to_root >= 2) core.put(buf, x);
        __syncthreads();
        if (to_root < 2) core.merge(buf, x, 0);
        if (to_root == 1) core.put(buf, x);
        __syncthreads();
        if (to_root == 0) core.merge(bufs, x, 1);
      }
    };
    int stage = 0;
    uint32_t phases = 0;  // parity of each stage's next wait
    bool lost = false;    // a wait ran out
    while (true) {
      if constexpr (kAlone) {
        core.settle_alone(a, q_row_of(use), heads,
                          reinterpret_cast<char*>(bufs) + warp * Core::kQBytes);
      } else {
        core.settle(reinterpret_cast<char*>(bufs + Core::kBuf / 16));
        if constexpr (Core::kQShared) __syncthreads();
      }
#pragma unroll 1
      for (int x = 0; x < use.steps; ++x) {
        const int valid = static_cast<int>(valids >> (5 * (kStages - 1)) & 31);
        if (valid > 0) {
          uint64_t* full = &s_full[warp][stage];
          const uint32_t phase = phases >> stage & 1;
          if (!warp_wait(full, phase, &s_abort)) {
            // this or another warp's wait ran out: issue no more, and wait once
            // more, bounded again, for what is in flight; the status tells
            lost = done = true;
            volatile int own = 0;
            warp_wait(full, phase, &own);
          }
          phases ^= 1u << stage;
          const uint32_t at = smem_u32(ring + stage * Core::kStage);
          core.scores(at, valid);
          core.values(at, valid);
        }
        issue(stage);
        stage = stage + 1 == kStages ? 0 : stage + 1;
      }

      const Unit was = use;
      const long long q_row = q_row_of(was);
      const bool last = kUnits || !goes_on(alone_c, was);
      if (!last) {  // the next unit's Q, while this one's results are joined
        next_unit(alone_c, use);
        if (!kAlone || !Core::kQShared) core.fetch(a, q_row_of(use), heads);
      }

      if constexpr (kAlone) {
#pragma unroll
        for (int x = 0; x < Core::kParts; ++x) core.emit(a, q_row, heads, true, 0, x);
        if (last) break;
        continue;
      }
      join_warps();
      if constexpr (kUnits) {
        if (a.cluster > 1) {
          // the CTAs' results: the first CTA's warps take those of up to two CTAs
          // each, in order of rank, and join theirs
          const int rank = blockIdx.x % a.cluster;
          static_assert(Core::kParts * Core::kBuf <= kWarps * kStages * Core::kStage, "ring");
          float4* all = reinterpret_cast<float4*>(rings);  // every copy has been used
#pragma unroll
          for (int x = 0; x < Core::kParts; ++x)
            if (warp == root_of(x)) core.put(all + x * (Core::kBuf / 16), x);
          cluster_sync();
          if (rank == 0) {
            core.clear();
#pragma unroll 1
            for (int src = warp; src < a.cluster; src += kWarps)
#pragma unroll
              for (int x = 0; x < Core::kParts; ++x)
                core.merge(in_cluster(all + x * (Core::kBuf / 16), src), x, 0);
            join_warps();
          }
          cluster_sync();  // no CTA ends while its buffers are read
          if (rank > 0) break;
        }
#pragma unroll
        for (int x = 0; x < Core::kParts; ++x)
          if (warp == root_of(x)) core.emit(a, q_row, heads, true, 0, x);
        break;
      } else {
        const int tiles = (was.len + kTile - 1) / kTile;
#pragma unroll
        for (int x = 0; x < Core::kParts; ++x)
          if (warp == root_of(x))
            core.emit(a, q_row, heads, was.steps == tiles, blockIdx.x * 2ll + (was.t0 == 0 ? 1 : 0),
                      x);
        if (warp == 0) {
          if (lane == 0 && was.t0 == 0 && (a.by_unit || was.steps < tiles)) {
            // the group of CTAs whose range holds the unit's last tile
            const unsigned long long past = end - was.left + tiles;
            const int to = static_cast<int>((past * groups - 1) / total);
            *split_of(a, was.request, was.head, part) = {was.request, was.head,
                                                         static_cast<int>(blockIdx.x), to - group};
          }
        }
        if (last) break;
      }
    }
    if (bad) atomicExch(a.status, kStatusBadCache);
    if (lost && lane == 0) atomicExch(a.status, kStatusTimeout);
  };
  if constexpr (kWay == kByWarps) {
    walk(std::true_type());
  } else {
    if constexpr (kMaybeAlone)
      if (alone) return walk(std::true_type());
    walk(std::false_type());
  }
}

constexpr int kJoinWarps = 4;

__device__ __forceinline__ void store_row(float* p, const float (&x)[4]) {
  *reinterpret_cast<float4*>(p) = make_float4(x[0], x[1], x[2], x[3]);
}
__device__ __forceinline__ void store_row(float* p, const float (&x)[2]) { store_pair(p, x[0], x[1]); }
__device__ __forceinline__ void store_row(float* p, const float (&x)[1]) { *p = x[0]; }
__device__ __forceinline__ void load_row(const float* p, float (&x)[4]) {
  const float4 y = *reinterpret_cast<const float4*>(p);
  x[0] = y.x, x[1] = y.y, x[2] = y.z, x[3] = y.w;
}
__device__ __forceinline__ void load_row(const float* p, float (&x)[2]) {
  const float2 y = *reinterpret_cast<const float2*>(p);
  x[0] = y.x, x[1] = y.y;
}
__device__ __forceinline__ void load_row(const float* p, float (&x)[1]) { x[0] = *p; }

// Joins the partial results of a unit for one query head (blockIdx.y). A warp adds
// every kJoinWarps-th partial's row, in that order; the first rows are read
// together with the references and sums their weights 2^(m - max) come from.
template <typename T, int kD>
__global__ void __launch_bounds__(kJoinWarps * 32) join_kernel(const DecodeArgs a) {
  constexpr int kPer = kD / 32;  // features a lane
  constexpr int kAtOnce = 8;     // rows
  __shared__ float s_o[kJoinWarps][kD], s_w[kMaxCtas], s_max[kJoinWarps], s_sum[kJoinWarps];
  const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32, h = blockIdx.y;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const Split s = a.split[blockIdx.x];
  if (s.more == 0) return;
  const int head0 = s.first % a.hc * a.per;
  if (head0 + h >= a.D.group) return;
  const long long step = 2ll * a.hc * a.per;  // partial results between two CTAs of a unit
  const long long at0 = (2ll * s.first + 1) * a.per + h, at1 = (2ll * s.first) * a.per + h;
  auto slot_of = [&](int p) { return p == 0 ? at0 : at1 + p * step; };
  const int parts = s.more + 1;
  float y[kAtOnce][kPer];
#pragma unroll
  for (int x = 0; x < kAtOnce; ++x) {
    const int p = warp + x * kJoinWarps;
    if (p < parts) load_row(a.part_o + slot_of(p) * kD + lane * kPer, y[x]);
  }
  float2 ml = make_float2(-INFINITY, 0.0f);
  if (tid < parts) ml = a.part_ml[slot_of(tid)];
  float m = ml.x;
  for (int p = tid + kJoinWarps * 32; p < parts; p += kJoinWarps * 32)
    m = fmaxf(m, a.part_ml[slot_of(p)].x);
#pragma unroll
  for (int x = 16; x > 0; x /= 2) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, x));
  if (lane == 0) s_max[warp] = m;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kJoinWarps; ++w) m = fmaxf(m, s_max[w]);
  const float base = m == -INFINITY ? 0.0f : m;
  float sum = 0.0f;
  for (int p = tid; p < parts; p += kJoinWarps * 32) {
    if (p != tid) ml = a.part_ml[slot_of(p)];
    const float w = ex2(ml.x - base);
    s_w[p] = w;
    sum += ml.y * w;
  }
#pragma unroll
  for (int x = 16; x > 0; x /= 2) sum += __shfl_xor_sync(0xffffffffu, sum, x);
  if (lane == 0) s_sum[warp] = sum;
  __syncthreads();
  float o[kPer];
#pragma unroll
  for (int j = 0; j < kPer; ++j) o[j] = 0.0f;
  for (int p0 = warp; p0 < parts; p0 += kAtOnce * kJoinWarps) {
#pragma unroll
    for (int x = 0; x < kAtOnce; ++x) {
      const int p = p0 + x * kJoinWarps;
      if (p >= parts) continue;
      if (p0 != warp) load_row(a.part_o + slot_of(p) * kD + lane * kPer, y[x]);
      const float w = s_w[p];
#pragma unroll
      for (int j = 0; j < kPer; ++j) o[j] += y[x][j] * w;
    }
  }
  store_row(&s_o[warp][lane * kPer], o);
  __syncthreads();
  const long long row =
      static_cast<long long>(s.request) * a.D.hq + s.head * a.D.group + head0 + h;
  if (tid >= kD / 2) return;
  sum = 0.0f;
  float2 z = make_float2(0.0f, 0.0f);
#pragma unroll
  for (int w = 0; w < kJoinWarps; ++w) {
    sum += s_sum[w];
    z.x += s_o[w][2 * tid];
    z.y += s_o[w][2 * tid + 1];
  }
  const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
  store_pair(static_cast<T*>(a.O) + row * kD + 2 * tid, z.x * inv, z.y * inv);
  if (tid == 0 && a.lse != nullptr)
    a.lse[row] = sum == 0.0f ? -INFINITY : base * kLn2 + logf(sum);
}

// ------------------------------------------------------------ host

// How the group's heads are cut: chunks, heads a chunk (at most `most`).
struct Cut {
  int hc, per;
};
Cut cut_of(const PagedDims& D) {
  const int most = D.dtype == XATTN_BF16 ? 32 : D.d == 128 ? 4 : 8;
  const int hc = (D.group + most - 1) / most;
  return {hc, (D.group + hc - 1) / hc};
}

size_t align256(size_t x) { return (x + 255) / 256 * 256; }

template <class Core>
cudaError_t launch_decode(DecodeArgs a, int num_sms, cudaStream_t st) {
  constexpr int kTile = kWarps * Core::kChunk;
  const PagedDims& D = a.D;
  a.sms = num_sms;
  const long long slots = min(num_sms * Core::kCtas, kMaxCtas);  // CTAs the GPU holds
  const long long units = static_cast<long long>(D.nseq) * D.hkv * a.hc;
  const long long row_tokens = static_cast<long long>(D.max_pages) << D.page_shift;
  const long long row_tiles = (row_tokens + kTile - 1) / kTile;
  const long long tiles = row_tiles * D.nseq * D.hkv;
  CUtensorMap k_map, v_map;
  if (make_pages_map(&k_map, a.k_pages, D, Core::kBox, Core::kChunk) != XATTN_OK ||
      make_pages_map(&v_map, a.v_pages, D, Core::kBox, Core::kChunk) != XATTN_OK)
    return cudaErrorInvalidValue;
  cudaLaunchAttribute attr;
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(kWarps * 32);
  cfg.stream = st;
  cfg.attrs = &attr;

  // By warps: many short units.
  // By units: four waves of them, of 32 tiles at most, balance themselves; fewer
  // where the table holds so little that a unit's CTA, or each of its cluster, has
  // eight tiles at most; and where the tiles of all cannot be numbered.
  a.cluster = 1;
  while (a.cluster < 8 && a.cluster < row_tiles && 2 * a.cluster * units <= slots) a.cluster *= 2;
  const bool waves = units >= 4 * slots && row_tiles <= 32;
  const bool numbered = tiles + kUnitCost * D.nseq * static_cast<long long>(D.hkv) < 1ll << 31;
  if (units >= kAloneWaves * slots && row_tokens <= kAloneTokens) {
    constexpr int kSmem = smem_of<Core, true>();
    cudaError_t e = cudaFuncSetAttribute(decode_kernel<Core, kByWarps>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e != cudaSuccess) return e;
    const unsigned grid = static_cast<unsigned>((units + kWarps - 1) / kWarps);
    decode_kernel<Core, kByWarps><<<grid, kWarps * 32, kSmem, st>>>(a, k_map, v_map);
    return cudaGetLastError();
  }
  if (waves || row_tiles <= 8 * a.cluster || !numbered) {
    cudaError_t e = cudaFuncSetAttribute(decode_kernel<Core, kByUnits>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         smem_of<Core, false>());
    if (e != cudaSuccess) return e;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = a.cluster;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cfg.gridDim = dim3(static_cast<unsigned>(units * a.cluster));
    cfg.dynamicSmemBytes = smem_of<Core, false>();
    cfg.numAttrs = a.cluster > 1 ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, decode_kernel<Core, kByUnits>, a, k_map, v_map);
  }

  // By ranges, no more than there can be tiles.
  const unsigned grid = static_cast<unsigned>(max(1ll, min(slots / a.hc, tiles)) * a.hc);
  a.by_unit = units < grid;
  auto launch = [&](auto* kernel, int smem) {
    const cudaError_t e =
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    kernel<<<grid, kWarps * 32, smem, st>>>(a, k_map, v_map);
    return cudaGetLastError();
  };
  cudaError_t e = units >= kAloneWaves * grid
                      ? launch(&decode_kernel<Core, kByRangesOrWarps>, smem_of<Core, true>())
                      : launch(&decode_kernel<Core, kByRanges>, smem_of<Core, false>());
  if (e != cudaSuccess) return e;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3(a.by_unit ? static_cast<unsigned>(units) : grid, a.per);
  cfg.blockDim = dim3(kJoinWarps * 32);
  cfg.dynamicSmemBytes = 0;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, join_kernel<typename Core::T, Core::kDim>, a);
}

template <int kD>
cudaError_t launch_bf16(const DecodeArgs& a, int num_sms, cudaStream_t st) {
  return a.per <= 8    ? launch_decode<CoreBf16<kD, 1>>(a, num_sms, st)
         : a.per <= 16 ? launch_decode<CoreBf16<kD, 2>>(a, num_sms, st)
                       : launch_decode<CoreBf16<kD, 4>>(a, num_sms, st);
}

template <int kD>
cudaError_t launch_f32(const DecodeArgs& a, int num_sms, cudaStream_t st) {
  if (a.per == 1) return launch_decode<CoreF32<kD, 1>>(a, num_sms, st);
  if (a.per == 2) return launch_decode<CoreF32<kD, 2>>(a, num_sms, st);
  if constexpr (kD < 128)
    if (a.per > 4) return launch_decode<CoreF32<kD, 8>>(a, num_sms, st);
  return launch_decode<CoreF32<kD, 4>>(a, num_sms, st);
}

}  // namespace
}  // namespace xattn

using namespace xattn;
using namespace xattn::host;

extern "C" {

size_t xattn_paged_decode_workspace_bytes(const xattn_paged* cache) {
  PagedDims D;
  if (check_paged(cache, true, &D) != XATTN_OK) return 0;
  const size_t rows = static_cast<size_t>(kMaxCtas) * 2 * cut_of(D).per;
  return align256(kMaxCtas * sizeof(Split)) + align256(rows * sizeof(float2)) +
         align256(rows * D.d * sizeof(float));
}

int xattn_paged_decode(const void* Q, const void* k_pages, const void* v_pages,
                       const xattn_paged* cache, const int32_t* table, const int32_t* lens,
                       void* O, float* lse, void* ws, size_t ws_bytes, void* stream) {
  PagedDims D;
  int rc = check_paged(cache, true, &D);
  if (rc != XATTN_OK) return rc;
  if (!Q || !k_pages || !v_pages || !table || !lens || !O) return XATTN_ERR_INVALID_ARG;
  if (!aligned16(Q) || !aligned16(k_pages) || !aligned16(v_pages) || !aligned16(O) ||
      (reinterpret_cast<uintptr_t>(lse) & 3u) != 0)
    return XATTN_ERR_INVALID_ARG;
  if (!ws || ws_bytes < xattn_paged_decode_workspace_bytes(cache)) return XATTN_ERR_WORKSPACE;
  if (!aligned16(ws)) return XATTN_ERR_INVALID_ARG;
  DeviceState* ds = nullptr;
  if ((rc = device_state(&ds)) != XATTN_OK) return rc;
  const Cut cut = cut_of(D);
  const size_t rows = static_cast<size_t>(kMaxCtas) * 2 * cut.per;
  char* w = static_cast<char*>(ws);
  DecodeArgs a = {D, cut.hc, cut.per, false, 1, 0, Q, k_pages, v_pages, table, lens, O, lse, ds->status};
  a.split = reinterpret_cast<Split*>(w);
  a.part_ml = reinterpret_cast<float2*>(w + align256(kMaxCtas * sizeof(Split)));
  a.part_o = reinterpret_cast<float*>(w + align256(kMaxCtas * sizeof(Split)) +
                                      align256(rows * sizeof(float2)));
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (D.dtype == XATTN_BF16) {
    return cuda_status(D.d == 64 ? launch_bf16<64>(a, ds->num_sms, st)
                                 : launch_bf16<128>(a, ds->num_sms, st));
  }
  return cuda_status(D.d == 32   ? launch_f32<32>(a, ds->num_sms, st)
                     : D.d == 64 ? launch_f32<64>(a, ds->num_sms, st)
                                 : launch_f32<128>(a, ds->num_sms, st));
}

}  // extern "C"
