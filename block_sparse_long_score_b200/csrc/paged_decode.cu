// paged_decode.cu -- xattn_paged_decode: attention of one new token per request
// over a paged key-value cache.
//
// For a request of n tokens and a KV head with its g query heads:
//   s[h, t] = q_h . k_t / sqrt(d),  o_h = sum_t e^(s - lse_h) v_t,  lse_h = log sum_t e^s.
// K and V are read once, which bounds the call: 2 * d * esize bytes a token
// against 4 * g * d flops, g flops a byte in bf16 (26 TFLOP/s at the measured
// copy rate for g = 4).
//
// Work split. The tokens of every (request, KV head) are cut into tiles of
// kWarps * kChunk tokens, all tiles are numbered in a row, and each CTA takes an
// equal range of them, whatever the lengths: one long request and many ragged
// ones load the GPU alike. A CTA walks the (request, head) units of its
// range. A unit inside one CTA's range is written straight to O; one that
// several CTAs share leaves a partial result (running maximum, sum,
// unnormalised o) in the workspace, at most two a CTA, and a second kernel,
// launched with programmatic stream serialization, joins them in CTA order.
// The ranges are worked out on the device from lens, so a captured graph
// follows the lengths.
//
// Inside a CTA the warps take the tile's chunks, each with its own running
// maximum, sum and o; they meet once at the end of a unit. K and V go from
// global memory straight into the registers of the warp that uses them: nothing
// is shared between warps, so a stage in shared memory would only add a trip.
// Loads of the next chunk's K are issued when the products with this chunk's
// are done, V likewise, so a warp has about two chunks' halves in flight and
// 16 warps an SM cover the memory's latency.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "host.cuh"
#include "paged.cuh"
#include "ptx.cuh"

namespace xattn {
namespace {

constexpr int kWarps = 4;
constexpr int kMaxCtas = 1024;  // CTAs of the first kernel (bounds the workspace)
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// What the join has to know of a unit: its first CTA and how many CTAs follow
// it. One entry per unit, or one per first CTA where there are more units.
struct Split {
  int request, head, first, more;
};

struct DecodeArgs {
  PagedDims D;
  int hc, per;  // chunks the group's heads are cut into, and heads in a chunk
  bool by_unit; // Split entries are indexed by unit
  const void *Q, *k_pages, *v_pages;
  const int32_t *table, *lens;
  void* O;
  float* lse;
  int* status;
  // workspace: per CTA a Split and two partial results of `per` heads
  Split* split;
  float2* part_ml;  // [CTA][2][per]: maximum (base 2) and sum
  float* part_o;    // [CTA][2][per][d], features in the warps' order
};

__device__ __forceinline__ int clamped(const DecodeArgs& a, int len) {
  return min(max(len, 0), a.D.max_pages << a.D.page_shift);
}
__device__ __forceinline__ Split* split_of(const DecodeArgs& a, int request, int head, int part) {
  return a.split +
         (a.by_unit ? (request * a.D.hkv + head) * a.hc + part : static_cast<int>(blockIdx.x));
}

// ------------------------------------------------------------ loads
// 32 bytes a lane. K and V are read once: they are not kept in L1.
template <bool kWide>
__device__ __forceinline__ void load32(const char* p, uint32_t* r) {
  if constexpr (kWide) {
    asm volatile("ld.global.nc.L1::no_allocate.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]),
                   "=r"(r[6]), "=r"(r[7])
                 : "l"(p));
  } else {
    asm volatile("ld.global.nc.L1::no_allocate.v4.b32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "l"(p));
    asm volatile("ld.global.nc.L1::no_allocate.v4.b32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "l"(p + 16));
  }
}
__device__ __forceinline__ void load16(const char* p, uint32_t* r) {
  asm volatile("ld.global.nc.L1::no_allocate.v4.b32 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "l"(p));
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
// would want 64 or 128 rows staged in shared memory to feed a product that
// needs 2 % of its rate; here the operands are in registers already.
// The order of the features inside a product is free, as long as both
// operands agree: lane (r = lane / 4, c = lane % 4) holds the 16 contiguous
// features 64 j + 16 c .. + 15 of tokens r and r + 8 (K) and of head r (Q),
// which makes every load 32 contiguous bytes. For V the lane holds features
// r * d/8 .. of tokens 2c, 2c+1, 2c+8, 2c+9; a byte permutation pairs two
// tokens' values of a feature. P goes from the accumulator's layout to an
// operand's with one 8x8 transpose per 8 tokens.
template <int kD, int NT, bool kWide>
struct CoreBf16 {
  static constexpr int kDim = kD;
  static constexpr int kChunk = 16;          // tokens of a warp's step
  static constexpr int kHeads = 8 * NT;      // heads it serves
  static constexpr int kCtas = (kD == 64 ? 4 : 3) - (NT - 1);  // without spills
  using T = __nv_bfloat16;
  static constexpr int kKRegs = kD / 8, kVPer = kD / 16;  // a row's registers a lane: K, V

  uint32_t q[NT][kKRegs], k[2][kKRegs], v[4][kVPer];
  float o[NT][kD / 16][4], m[NT][2], base[NT][2], l[NT][2];
  int r, c;

  __device__ __forceinline__ void init() {
    r = threadIdx.x % 32 / 4;
    c = threadIdx.x % 4;
  }

  // Heads of the unit; rows past the chunk's heads are zero.
  __device__ __forceinline__ void start(const DecodeArgs& a, long long q_row, int heads) {
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const char* p = static_cast<const char*>(a.Q) + (q_row + 8 * t + r) * kD * 2 + c * 32;
#pragma unroll
      for (int j = 0; j < kD / 64; ++j) {
        if (8 * t + r < heads) {
          load16(p + j * 128, &q[t][8 * j]);
          load16(p + j * 128 + 16, &q[t][8 * j + 4]);
        } else {
#pragma unroll
          for (int x = 0; x < 8; ++x) q[t][8 * j + x] = 0;
        }
      }
#pragma unroll
      for (int i = 0; i < kD / 16; ++i)
#pragma unroll
        for (int x = 0; x < 4; ++x) o[t][i][x] = 0.0f;
#pragma unroll
      for (int x = 0; x < 2; ++x) m[t][x] = -INFINITY, base[t][x] = 0.0f, l[t][x] = 0.0f;
    }
  }

  // Rows past `valid` (< kChunk) take the last valid one's address.
  __device__ __forceinline__ void load_k(const char* row0, long long stride, int valid) {
    const int t0 = min(r, valid - 1), t1 = min(r + 8, valid - 1);
#pragma unroll
    for (int j = 0; j < kD / 64; ++j) {
      load32<kWide>(row0 + t0 * stride + j * 128 + c * 32, &k[0][8 * j]);
      load32<kWide>(row0 + t1 * stride + j * 128 + c * 32, &k[1][8 * j]);
    }
  }
  __device__ __forceinline__ void load_v(const char* row0, long long stride, int valid) {
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      const int t = min(2 * c + (x & 1) + (x & 2) * 4, valid - 1);
      const char* p = row0 + t * stride + r * (kD / 4);
      if constexpr (kD == 128) load32<kWide>(p, v[x]);
      else load16(p, v[x]);
    }
  }
  __device__ __forceinline__ void zero_k() {
#pragma unroll
    for (int x = 0; x < 2; ++x)
#pragma unroll
      for (int j = 0; j < kKRegs; ++j) k[x][j] = 0;
  }
  __device__ __forceinline__ void zero_v() {
#pragma unroll
    for (int x = 0; x < 4; ++x)
#pragma unroll
      for (int j = 0; j < kVPer; ++j) v[x][j] = 0;
  }

  // Weights of the chunk as operands of the second product.
  uint32_t p[NT][2];

  __device__ __forceinline__ void scores(int valid) {
    const float scale = kLog2e * (kD == 64 ? 0.125f : 0.08838834764831845f);  // log2(e) / sqrt(d)
    float s[NT][4];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      float x[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int i = 0; i < kKRegs / 2; ++i)
        mma_bf16(x, k[0][2 * i], k[1][2 * i], k[0][2 * i + 1], k[1][2 * i + 1], q[t][2 * i],
                 q[t][2 * i + 1]);
#pragma unroll
      for (int j = 0; j < 4; ++j) s[t][j] = x[j] * scale;
      if (valid < kChunk) {
        if (r >= valid) s[t][0] = s[t][1] = -INFINITY;
        if (r + 8 >= valid) s[t][2] = s[t][3] = -INFINITY;
      }
    }
    // The reference a weight is taken against lags the true maximum by at most
    // 2^8: o and l are rescaled only when a logit passes that, which after a
    // few chunks hardly happens. Weights stay below 2^8, sums in fp32 far from
    // overflow, and a weight's rounding is relative, so nothing is lost.
    bool grow = false;
#pragma unroll
    for (int t = 0; t < NT; ++t)
      grow = grow || fmaxf(s[t][0], s[t][2]) > m[t][0] + 8.0f ||
             fmaxf(s[t][1], s[t][3]) > m[t][1] + 8.0f;
    if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
      for (int t = 0; t < NT; ++t) {
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          float top = fmaxf(s[t][x], s[t][x + 2]);
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 4));
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 8));
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 16));
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
      }
    }
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      float w[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) w[j] = ex2(s[t][j] - base[t][j & 1]);
      l[t][0] += w[0] + w[2];
      l[t][1] += w[1] + w[3];
      // bf16 weights (half a step, 2^-8, relative): what the tensor cores take,
      // as in the prefill's attention; the sum keeps the fp32 ones
      p[t][0] = transpose8x8(pack_bf16x2(w[0], w[1]));
      p[t][1] = transpose8x8(pack_bf16x2(w[2], w[3]));
    }
  }

  __device__ __forceinline__ void values(int valid) {
    if (valid < kChunk) {  // a weight of 0 does not undo a NaN or infinity
#pragma unroll
      for (int x = 0; x < 4; ++x)
        if (2 * c + (x & 1) + (x & 2) * 4 >= valid)
#pragma unroll
          for (int j = 0; j < kVPer; ++j) v[x][j] = 0;
    }
#pragma unroll
    for (int i = 0; i < kD / 16; ++i) {
      const uint32_t a0 = __byte_perm(v[0][i], v[1][i], 0x5410);
      const uint32_t a1 = __byte_perm(v[0][i], v[1][i], 0x7632);
      const uint32_t a2 = __byte_perm(v[2][i], v[3][i], 0x5410);
      const uint32_t a3 = __byte_perm(v[2][i], v[3][i], 0x7632);
#pragma unroll
      for (int t = 0; t < NT; ++t) mma_bf16(o[t][i], a0, a1, a2, a3, p[t][0], p[t][1]);
    }
  }

  // Feature j of a head is at place_of(j) in the joined rows: the lanes' order,
  // which keeps the stores below free of bank conflicts.
  __device__ static __forceinline__ int place_of(int j) {
    return j % (kD / 8) / 2 * 16 + j / (kD / 8) * 2 + j % 2;
  }
  static constexpr int kRow = kD + 4;  // a head's row in shared memory, padded likewise

  __device__ __forceinline__ void finish(float2* ml, float* rows) {
#pragma unroll
    for (int t = 0; t < NT; ++t) {
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        float sum = l[t][x];
        sum += __shfl_xor_sync(0xffffffffu, sum, 4);
        sum += __shfl_xor_sync(0xffffffffu, sum, 8);
        sum += __shfl_xor_sync(0xffffffffu, sum, 16);
        if (r == 0) ml[8 * t + 2 * c + x] = make_float2(m[t][x], sum);
#pragma unroll
        for (int i = 0; i < kD / 16; ++i)
          *reinterpret_cast<float2*>(rows + (8 * t + 2 * c + x) * kRow + i * 16 + r * 2) =
              make_float2(o[t][i][x], o[t][i][x + 2]);
      }
    }
  }
};

// ------------------------------------------------------------ fp32 core
// CUDA cores: no tensor-core type keeps fp32's mantissa. A warp's chunk is 8
// tokens, two to each group of 8 lanes; a lane holds d / 8 features of its two
// tokens, 16 bytes at a time. The 2 * H dot products of a group are summed
// over its lanes by halving (one exchange less each step), which leaves one
// (token, head) logit a lane, so each exponential is taken once.
template <int kD, int H>
struct CoreF32 {
  static constexpr int kDim = kD;
  static constexpr int kChunk = 8;
  static constexpr int kHeads = H;
  static constexpr int kCtas = H == 4 ? (kD == 128 ? 2 : 3) : kD == 128 ? 3 : 4;
  using T = float;
  static constexpr int kPer = kD / 8;

  float q[H][kPer], k[2][kPer], v[2][kPer], o[H][kPer], m[H], base[H], l[H], w[2][H];
  int g, c;  // the lane's group (tokens g and g + 4) and place in it

  __device__ __forceinline__ void init() {
    g = threadIdx.x % 32 / 8;
    c = threadIdx.x % 8;
  }
  __device__ __forceinline__ void start(const DecodeArgs& a, long long q_row, int heads) {
    const float scale = kLog2e / sqrtf(static_cast<float>(kD));
#pragma unroll
    for (int h = 0; h < H; ++h) {
      const float* p = static_cast<const float*>(a.Q) + (q_row + h) * kD + c * 4;
#pragma unroll
      for (int j = 0; j < kPer; ++j) {
        q[h][j] = h < heads ? p[j / 4 * 32 + j % 4] * scale : 0.0f;
        o[h][j] = 0.0f;
      }
      m[h] = -INFINITY;
      base[h] = 0.0f;
      l[h] = 0.0f;
    }
  }
  __device__ __forceinline__ void load(const char* row0, long long stride, int valid,
                                       float (&x)[2][kPer]) {
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int j = 0; j < kPer / 4; ++j)
        load16(row0 + min(g + 4 * t, valid - 1) * stride + j * 128 + c * 16,
               reinterpret_cast<uint32_t*>(&x[t][4 * j]));
  }
  __device__ __forceinline__ void load_k(const char* row0, long long stride, int valid) {
    load(row0, stride, valid, k);
  }
  __device__ __forceinline__ void load_v(const char* row0, long long stride, int valid) {
    load(row0, stride, valid, v);
  }
  __device__ __forceinline__ void zero_k() {
#pragma unroll
    for (int j = 0; j < kPer; ++j) k[0][j] = k[1][j] = 0.0f;
  }
  __device__ __forceinline__ void zero_v() {
#pragma unroll
    for (int j = 0; j < kPer; ++j) v[0][j] = v[1][j] = 0.0f;
  }
  __device__ __forceinline__ void scores(int valid) {
    float s[2][H];
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int h = 0; h < H; ++h) {
        float x = 0.0f;
#pragma unroll
        for (int j = 0; j < kPer; ++j) x = fmaf(q[h][j], k[t][j], x);
        s[t][h] = x;
      }
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int h = 0; h < H; ++h) {
        s[t][h] += __shfl_xor_sync(0xffffffffu, s[t][h], 1);
        s[t][h] += __shfl_xor_sync(0xffffffffu, s[t][h], 2);
        s[t][h] += __shfl_xor_sync(0xffffffffu, s[t][h], 4);
        if (g + 4 * t >= valid) s[t][h] = -INFINITY;
      }
    bool grow = false;  // as in the bf16 core
#pragma unroll
    for (int h = 0; h < H; ++h) grow = grow || fmaxf(s[0][h], s[1][h]) > m[h] + 8.0f;
    if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
      for (int h = 0; h < H; ++h) {
        float top = fmaxf(s[0][h], s[1][h]);
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 8));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 16));
        top = fmaxf(top, m[h]);
        base[h] = top == -INFINITY ? 0.0f : top;
        const float f = ex2(m[h] - base[h]);
        m[h] = top;
        l[h] *= f;
#pragma unroll
        for (int j = 0; j < kPer; ++j) o[h][j] *= f;
      }
    }
#pragma unroll
    for (int h = 0; h < H; ++h) {
      w[0][h] = ex2(s[0][h] - base[h]);
      w[1][h] = ex2(s[1][h] - base[h]);
      l[h] += w[0][h] + w[1][h];
    }
  }
  __device__ __forceinline__ void values(int valid) {
    if (valid < kChunk) {  // a weight of 0 does not undo a NaN or infinity
#pragma unroll
      for (int t = 0; t < 2; ++t)
        if (g + 4 * t >= valid)
#pragma unroll
          for (int j = 0; j < kPer; ++j) v[t][j] = 0.0f;
    }
#pragma unroll
    for (int h = 0; h < H; ++h)
#pragma unroll
      for (int j = 0; j < kPer; ++j)
        o[h][j] = fmaf(w[1][h], v[1][j], fmaf(w[0][h], v[0][j], o[h][j]));
  }
  __device__ static __forceinline__ int place_of(int j) { return j; }
  static constexpr int kRow = kD + 4;
  __device__ __forceinline__ void finish(float2* ml, float* rows) {
#pragma unroll
    for (int h = 0; h < H; ++h) {
      float sum = l[h];
      sum += __shfl_xor_sync(0xffffffffu, sum, 8);
      sum += __shfl_xor_sync(0xffffffffu, sum, 16);
      if (g == 0 && c == 0) ml[h] = make_float2(m[h], sum);
#pragma unroll
      for (int j = 0; j < kPer; ++j) {
        float x = o[h][j];
        x += __shfl_xor_sync(0xffffffffu, x, 8);
        x += __shfl_xor_sync(0xffffffffu, x, 16);
        if (g == 0) rows[h * kRow + j / 4 * 32 + c * 4 + j % 4] = x;
      }
    }
  }
};

// ------------------------------------------------------------ both kernels

__device__ __forceinline__ void store_pair(float* p, float x, float y) {
  *reinterpret_cast<float2*>(p) = make_float2(x, y);
}
__device__ __forceinline__ void store_pair(__nv_bfloat16* p, float x, float y) {
  *reinterpret_cast<uint32_t*>(p) = pack_bf16x2(x, y);
}

// First tile of CTA group b's range: total * b / groups.
__device__ __forceinline__ unsigned long long range_of(unsigned long long total, int b,
                                                       int groups) {
  return total * static_cast<unsigned>(b) / static_cast<unsigned>(groups);
}

// O = 0 and lse = -inf for the requests that hold nothing.
template <class Core>
__device__ void empty_rows(const DecodeArgs& a, int group, int groups, int part, int head0,
                           int heads) {
  constexpr int kHalf = Core::kDim / 2;
  const PagedDims& D = a.D;
  for (int i = group; i < D.nseq; i += groups) {
    if (clamped(a, a.lens[i]) != 0) continue;
    for (int x = threadIdx.x; x < D.hkv * heads * kHalf; x += kWarps * 32) {
      const int h = x / kHalf, head = h / heads;
      const long long row =
          static_cast<long long>(i) * D.hq + head * D.group + head0 + h % heads;
      store_pair(static_cast<typename Core::T*>(a.O) + row * Core::kDim + x % kHalf * 2, 0.0f,
                 0.0f);
      if (x % kHalf == 0 && a.lse != nullptr) a.lse[row] = -INFINITY;
      if (a.by_unit && x % (heads * kHalf) == 0) split_of(a, i, head, part)->more = 0;
    }
  }
}

template <class Core>
__global__ void __launch_bounds__(kWarps * 32, Core::kCtas) decode_kernel(const DecodeArgs a) {
  using T = typename Core::T;
  constexpr int kD = Core::kDim, kTile = kWarps * Core::kChunk, kThreads = kWarps * 32;
  const PagedDims& D = a.D;
  const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
  // CTAs b * hc .. b * hc + hc - 1 take the same tiles for different heads of
  // the group, at about the same time: the second to read a row finds it in L2.
  const int part = blockIdx.x % a.hc, group = blockIdx.x / a.hc;
  int groups = gridDim.x / a.hc;
  const int head0 = part * a.per, heads = min(a.per, D.group - head0);

  __shared__ float2 s_ml[kWarps][Core::kHeads];
  __shared__ float s_o[kWarps][Core::kHeads * Core::kRow];
  __shared__ unsigned long long s_sum[kWarps], s_before;
  __shared__ int s_request, s_len;

  asm volatile("griddepcontrol.launch_dependents;");

  // Where this CTA's range begins: a scan of the requests' tile counts, a run
  // of requests to each thread.
  const int run = (D.nseq + kThreads - 1) / kThreads;
  const int i0 = min(tid * run, D.nseq), i1 = min(i0 + run, D.nseq);
  unsigned long long mine = 0;
  bool bad = false, empty = false;
  for (int i = i0; i < i1; ++i) {
    const int raw = a.lens[i], n = clamped(a, raw);
    bad = bad || n != raw;
    empty = empty || n == 0;
    mine += (n + kTile - 1) / kTile;
  }
  if (bad && blockIdx.x == 0) atomicExch(a.status, kStatusBadCache);
  unsigned long long upto = mine;
  for (int x = 1; x < 32; x *= 2) {
    const unsigned long long y = __shfl_up_sync(0xffffffffu, upto, x);
    if (lane >= x) upto += y;
  }
  if (lane == 31) s_sum[warp] = upto;
  empty = __syncthreads_or(empty);
  unsigned long long total = 0;
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) upto += s_sum[w];
    total += s_sum[w];
  }
  total *= D.hkv;
  if (empty) empty_rows<Core>(a, group, groups, part, head0, heads);
  if (!a.by_unit && tid == 0) a.split[blockIdx.x].more = 0;
  // as many ranges as there are tiles, at most: none is empty, so a unit's
  // partial results are those of consecutive CTAs
  groups = static_cast<int>(min(static_cast<unsigned long long>(groups), total));
  if (group >= groups) return;
  unsigned long long pos = range_of(total, group, groups);
  const unsigned long long end = range_of(total, group + 1, groups);
  unsigned long long before = (upto - mine) * D.hkv;
  if (pos >= before && pos < upto * D.hkv) {
    for (int i = i0; i < i1; ++i) {
      const int n = clamped(a, a.lens[i]);
      const unsigned long long next =
          before + static_cast<unsigned long long>((n + kTile - 1) / kTile) * D.hkv;
      if (pos < next) {
        s_request = i;
        s_len = n;
        s_before = before;
        break;
      }
      before = next;
    }
  }
  __syncthreads();
  int request = s_request, len = s_len;
  before = s_before;

  Core core;
  core.init();
  bad = false;
  while (pos < end) {
    // the unit at pos, and this CTA's tiles of it
    const int tiles = (len + kTile - 1) / kTile;
    if (pos >= before + static_cast<unsigned long long>(tiles) * D.hkv) {
      before += static_cast<unsigned long long>(tiles) * D.hkv;
      len = clamped(a, a.lens[++request]);
      continue;
    }
    const int head = static_cast<int>((pos - before) / tiles);
    const int t0 = static_cast<int>((pos - before) % tiles);
    const int steps = static_cast<int>(min(static_cast<unsigned long long>(tiles - t0), end - pos));
    const long long q_row = static_cast<long long>(request) * D.hq + head * D.group + head0;
    const int32_t* pages = a.table + static_cast<long long>(request) * D.max_pages;
    const long long head_at = head * D.head_stride;
    const char* k_head = static_cast<const char*>(a.k_pages) + head_at * sizeof(T);
    const char* v_head = static_cast<const char*>(a.v_pages) + head_at * sizeof(T);
    const long long stride = D.token_stride * sizeof(T);

    // lane x of a warp holds the page of the warp's step 32 q + x
    const int first = t0 * kTile + warp * Core::kChunk;  // the warp's first token
    auto page_batch = [&](int step0) {
      const int t = first + (step0 + lane) * kTile;
      if (step0 + lane >= steps || t >= len) return -1;
      const int page = pages[t >> D.page_shift];
      if (page >= 0 && page < D.num_pages) return page;
      bad = true;
      return -1;
    };
    int now = page_batch(0), next = page_batch(32);
    core.start(a, q_row, heads);

    // a step's tokens: how many are there, and where its rows begin
    auto rows_of = [&](int step, int* valid) {
      const int page = __shfl_sync(0xffffffffu, now, step % 32);
      const int t = first + step * kTile;
      *valid = page < 0 ? 0 : min(Core::kChunk, len - t);
      return (page * D.page_stride + (t & (D.page - 1)) * D.token_stride) *
             static_cast<long long>(sizeof(T));
    };
    int valid;
    long long at = rows_of(0, &valid);
    if (valid > 0) {
      core.load_k(k_head + at, stride, valid);
      core.load_v(v_head + at, stride, valid);
    } else {
      core.zero_k();
      core.zero_v();
    }
#pragma unroll 1
    for (int step = 0; step < steps; ++step) {
      const int valid_now = valid;
      core.scores(valid_now);
      const bool more = step + 1 < steps;
      if (more) {
        if ((step + 1) % 32 == 0) {
          now = next;
          next = page_batch(step + 33);
        }
        at = rows_of(step + 1, &valid);
        if (valid > 0) core.load_k(k_head + at, stride, valid);
        else core.zero_k();
      }
      core.values(valid_now);
      if (more) {
        if (valid > 0) core.load_v(v_head + at, stride, valid);
        else core.zero_v();
      }
    }

    // the warps' results of this unit, joined
    core.finish(s_ml[warp], s_o[warp]);
    __syncthreads();
    const bool whole = t0 == 0 && steps == tiles;
    const long long slot = blockIdx.x * 2ll + (t0 == 0 ? 1 : 0);
    for (int x = tid; x < heads * (kD / 2); x += kThreads) {
      const int h = x / (kD / 2), j = x % (kD / 2) * 2;
      float top = s_ml[0][h].x;
#pragma unroll
      for (int w = 1; w < kWarps; ++w) top = fmaxf(top, s_ml[w][h].x);
      const float base = top == -INFINITY ? 0.0f : top;
      float sum = 0.0f;
      float2 o = make_float2(0.0f, 0.0f);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float f = ex2(s_ml[w][h].x - base);
        const float2 y =
            *reinterpret_cast<const float2*>(&s_o[w][h * Core::kRow + Core::place_of(j)]);
        sum += s_ml[w][h].y * f;
        o.x += y.x * f;
        o.y += y.y * f;
      }
      if (whole) {
        const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
        store_pair(static_cast<T*>(a.O) + (q_row + h) * kD + j, o.x * inv, o.y * inv);
        if (j == 0 && a.lse != nullptr)
          a.lse[q_row + h] = sum == 0.0f ? -INFINITY : base * kLn2 + logf(sum);
      } else {
        *reinterpret_cast<float2*>(&a.part_o[(slot * a.per + h) * kD + j]) = o;
        if (j == 0) a.part_ml[slot * a.per + h] = make_float2(top, sum);
      }
    }
    if (tid == 0 && t0 == 0 && (a.by_unit || !whole)) {
      // the group of CTAs whose range holds the unit's last tile
      const unsigned long long last = pos + tiles - 1;
      const int to = static_cast<int>(((last + 1) * groups - 1) / total);
      *split_of(a, request, head, part) = {request, head, static_cast<int>(blockIdx.x),
                                           to - group};
    }
    __syncthreads();
    pos += steps;
  }
  if (bad) atomicExch(a.status, kStatusBadCache);
}

constexpr int kJoinWarps = 8;

// Joins the partial results of a unit for one query head (blockIdx.y). The
// weights 2^(m - max) are worked out for 32 partials at a time, a lane each;
// then a warp adds every kJoinWarps-th partial's row, in that order.
template <typename T, int kD>
__global__ void __launch_bounds__(kJoinWarps * 32) join_kernel(const DecodeArgs a) {
  constexpr int kPer = kD / 32;  // features a lane
  __shared__ float s_o[kJoinWarps][kD], s_w[kMaxCtas], s_max[kJoinWarps], s_sum[kJoinWarps];
  const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32, h = blockIdx.y;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const Split s = a.split[blockIdx.x];
  if (s.more == 0) return;
  const int head0 = s.first % a.hc * a.per;
  if (head0 + h >= a.D.group) return;
  auto slot_of = [&](int p) {
    return ((s.first + static_cast<long long>(p) * a.hc) * 2 + (p == 0 ? 1 : 0)) * a.per + h;
  };
  const int parts = s.more + 1;
  float m = -INFINITY;
  for (int p = tid; p < parts; p += kJoinWarps * 32) m = fmaxf(m, a.part_ml[slot_of(p)].x);
  for (int x = 16; x > 0; x /= 2) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, x));
  if (lane == 0) s_max[warp] = m;
  __syncthreads();
  for (int w = 0; w < kJoinWarps; ++w) m = fmaxf(m, s_max[w]);
  const float base = m == -INFINITY ? 0.0f : m;
  float sum = 0.0f;
  for (int p = tid; p < parts; p += kJoinWarps * 32) {
    const float2 ml = a.part_ml[slot_of(p)];
    const float w = ex2(ml.x - base);
    s_w[p] = w;
    sum += ml.y * w;
  }
  for (int x = 16; x > 0; x /= 2) sum += __shfl_xor_sync(0xffffffffu, sum, x);
  if (lane == 0) s_sum[warp] = sum;
  __syncthreads();
  float o[kPer];
#pragma unroll
  for (int j = 0; j < kPer; ++j) o[j] = 0.0f;
#pragma unroll 4
  for (int p = warp; p < parts; p += kJoinWarps) {
    const float* row = a.part_o + slot_of(p) * kD + lane;
    const float w = s_w[p];
#pragma unroll
    for (int j = 0; j < kPer; ++j) o[j] += row[j * 32] * w;
  }
#pragma unroll
  for (int j = 0; j < kPer; ++j) s_o[warp][j * 32 + lane] = o[j];
  __syncthreads();
  const long long row =
      static_cast<long long>(s.request) * a.D.hq + s.head * a.D.group + head0 + h;
  if (tid >= kD / 2) return;
  sum = 0.0f;
  float2 y = make_float2(0.0f, 0.0f);
  for (int w = 0; w < kJoinWarps; ++w) {
    sum += s_sum[w];
    y.x += s_o[w][2 * tid];
    y.y += s_o[w][2 * tid + 1];
  }
  const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
  store_pair(static_cast<T*>(a.O) + row * kD + 2 * tid, y.x * inv, y.y * inv);
  if (tid == 0 && a.lse != nullptr)
    a.lse[row] = sum == 0.0f ? -INFINITY : base * kLn2 + logf(sum);
}

// ------------------------------------------------------------ host

// How the group's heads are cut: chunks, heads a chunk (at most `most`).
struct Cut {
  int hc, per;
};
Cut cut_of(const PagedDims& D) {
  const int most = D.dtype == XATTN_BF16 ? 16 : 4;
  const int hc = (D.group + most - 1) / most;
  return {hc, (D.group + hc - 1) / hc};
}

size_t align256(size_t x) { return (x + 255) / 256 * 256; }

template <class Core>
cudaError_t launch_decode(DecodeArgs a, int num_sms, cudaStream_t st) {
  constexpr int kTile = kWarps * Core::kChunk;
  const PagedDims& D = a.D;
  // no more groups than tiles there can be
  const long long row_tiles = ((static_cast<long long>(D.max_pages) << D.page_shift) + kTile - 1) / kTile;
  const long long tiles = row_tiles * D.nseq * D.hkv;
  long long groups = min(static_cast<long long>(num_sms) * Core::kCtas, static_cast<long long>(kMaxCtas)) / a.hc;
  groups = max(1ll, min(groups, tiles));
  const unsigned grid = static_cast<unsigned>(groups * a.hc);
  const long long units = static_cast<long long>(D.nseq) * D.hkv * a.hc;
  a.by_unit = units < grid;
  decode_kernel<Core><<<grid, kWarps * 32, 0, st>>>(a);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || row_tiles == 1) return e;  // a unit of one tile is never shared
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(a.by_unit ? static_cast<unsigned>(units) : grid, a.per);
  cfg.blockDim = dim3(kJoinWarps * 32);
  cfg.stream = st;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, join_kernel<typename Core::T, Core::kDim>, a);
}

template <int kD>
cudaError_t launch_bf16(const DecodeArgs& a, bool wide, int num_sms, cudaStream_t st) {
  if (a.per <= 8)
    return wide ? launch_decode<CoreBf16<kD, 1, true>>(a, num_sms, st)
                : launch_decode<CoreBf16<kD, 1, false>>(a, num_sms, st);
  return wide ? launch_decode<CoreBf16<kD, 2, true>>(a, num_sms, st)
              : launch_decode<CoreBf16<kD, 2, false>>(a, num_sms, st);
}

template <int kD>
cudaError_t launch_f32(const DecodeArgs& a, int num_sms, cudaStream_t st) {
  if (a.per == 1) return launch_decode<CoreF32<kD, 1>>(a, num_sms, st);
  if (a.per == 2) return launch_decode<CoreF32<kD, 2>>(a, num_sms, st);
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
  DecodeArgs a = {D, cut.hc, cut.per, false, Q, k_pages, v_pages, table, lens, O, lse, ds->status};
  a.split = reinterpret_cast<Split*>(w);
  a.part_ml = reinterpret_cast<float2*>(w + align256(kMaxCtas * sizeof(Split)));
  a.part_o = reinterpret_cast<float*>(w + align256(kMaxCtas * sizeof(Split)) +
                                      align256(rows * sizeof(float2)));
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (D.dtype == XATTN_BF16) {
    // 32-byte loads need every row on a 32-byte boundary
    const uintptr_t bits = reinterpret_cast<uintptr_t>(k_pages) |
                           reinterpret_cast<uintptr_t>(v_pages) |
                           static_cast<uintptr_t>(
                               (D.page_stride | D.head_stride | D.token_stride) * D.esize);
    const bool wide = (bits & 31u) == 0;
    return cuda_status(D.d == 64 ? launch_bf16<64>(a, wide, ds->num_sms, st)
                                 : launch_bf16<128>(a, wide, ds->num_sms, st));
  }
  return cuda_status(D.d == 32   ? launch_f32<32>(a, ds->num_sms, st)
                     : D.d == 64 ? launch_f32<64>(a, ds->num_sms, st)
                                 : launch_f32<128>(a, ds->num_sms, st));
}

}  // extern "C"
