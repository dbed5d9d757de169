// adamw.cu -- AdamW over many tensors at once, with 32-bit or 8-bit states,
// and the global norm of the gradients with the factor that clips it.
//
// The list of tensors travels as a kernel parameter, so a step needs no
// device copy of it and keeps nothing between calls.  Work is cut into chunks
// of kChunk elements that never span two tensors; one block takes one chunk.
#include <math.h>

#include <cuda_fp8.h>

#include "common.cuh"
#include "internal.h"

namespace tw {

namespace {

constexpr int kBlock = 256;          // elements per scale of an 8-bit state
constexpr int kMaxTensors = 400;     // per launch (their descriptions fill a kernel's parameters)
constexpr float kE4m3Max = 448.0f;
constexpr float kTinyMax = 7.888609052210118e-31f;  // 2^-100: smallest maximum that a scale is made for

struct Entry {
  void* param;
  uint16_t* copy;
  const void* grad;
  void* m;
  void* v;
  float* m_scale;
  float* v_scale;
  long long n;
  long long number;  // of the tensor's first element within the list
  int chunk;         // the tensor's first chunk within the launch
  int wide;          // every pointer is aligned to 4 of its elements
};
template <int MAX>
struct List {
  Entry e[MAX];
  int count;
};

struct Hyper {
  float beta1, one_beta1, beta2, one_beta2;
  float one;       // 1
  float decay;     // 1 - lr weight_decay
  float size;      // lr / (1 - beta1^step)
  float inv_root;  // 1 / sqrt(1 - beta2^step)
  float eps;
  uint32_t key;
  const float* grad_scale;
  int* skipped;
  int count_skip;  // this launch adds a skipped step to the count
  // of the corrections where steps were skipped
  float step, lr, ln_beta1, ln_beta2;
};

// What follows from the step: lr / (1 - beta1^t) and 1 / sqrt(1 - beta2^t).  The
// host has them for t = step; where steps were skipped they are made here,
// 1 - beta^t = -expm1(t ln beta), right to a few units of fp32's last place for any t.
// (COUNTED, in kernels of their own: as constants they cost the others no registers.  100.7 M
// elements, without a count, with one of 0 and with one of 1: fp32 398, 401, 400 us, 8 bits with
// bf16 parameters and gradients, which instructions bound, 209, 211, 232 us.)
struct Corrections {
  float size, inv_root;
};
TW_DEV Corrections corrections(const Hyper& H, int skipped) {
  if (skipped == 0) return Corrections{H.size, H.inv_root};
  const float t = fmaxf(H.step - (float)skipped, 1.0f);
  return Corrections{H.lr / -expm1f(t * H.ln_beta1), 1.0f / sqrtf(-expm1f(t * H.ln_beta2))};
}

// The tensor that holds a chunk: the last one whose first chunk is not past it.
template <class L_>
TW_DEV int find_entry(const L_& L, int chunk) {
  int lo = 0, hi = L.count - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (L.e[mid].chunk <= chunk)
      lo = mid;
    else
      hi = mid - 1;
  }
  return lo;
}

// 16 + 16 random bits from x = the element's number spread by a multiplication:
// the halves of murmur3's 32-bit finalizer, whose last step x ^ (x >> 16)
// leaves the high half as it is.
constexpr uint32_t kSpreadLo = 0x9E3779B1u, kSpreadHi = 0x85EBCA77u;
struct Random {
  uint32_t lo, hi;
};
TW_DEV Random hash_bits(uint32_t x) {
  x = (x ^ (x >> 16)) * 0x85EBCA6Bu;
  x = (x ^ (x >> 13)) * 0xC2B2AE35u;
  const uint32_t hi = x >> 16;
  return Random{(x ^ hi) & 0xFFFFu, hi};
}

// Codes of a pair of moments scaled to |x| <= 448 (give or take a rounding) and
// then by 2^-120, stochastically rounded: x moves up to the next code with
// probability (remainder / spacing).  Times 2^-120 e4m3's exponent range,
// subnormals included, is that of the lowest fp32 exponents, so the bits of
// the value without the last 20 are the code; 16 random bits are added below.
// Only the low 8 bits of the result count.  ODD: the block holds a NaN or an infinity.
constexpr float kE4m3Shift = 7.52316384526264e-37f;  // 2^-120
template <bool ODD>
TW_DEV uint32_t signed_code(uint32_t b, uint32_t r16) {
  if (ODD && (b & 0x7FFFFFFFu) > 0x7F800000u) return 0x7Fu;
  const uint32_t t = b + r16 * 16u;
  return ((t >> 24) & 0x80u) | ((t >> 20) & ~0x80u);  // the sign is bit 11 of t >> 20
}
template <bool ODD>
TW_DEV uint32_t positive_code(uint32_t b, uint32_t r16, uint32_t least) {
  const uint32_t c = max((b + r16 * 16u) >> 20, least);
  return ODD ? min(c, 0x7Fu) : c;
}
TW_DEV uint32_t bytes4(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  return __byte_perm(__byte_perm(a, b, 0x0040), __byte_perm(c, d, 0x0040), 0x5410);
}

// Four consecutive elements as two fp32 pairs: read as one vector (WIDE), or
// one by one, those at or past `n` being 0 and not touched.
struct Quad {
  uint64_t v[2];
  TW_DEV float get(int j) const { return j & 1 ? f2_hi(v[j >> 1]) : f2_lo(v[j >> 1]); }
};
TW_DEV Quad quad(const float (&x)[4]) { return Quad{{f2_pack(x[0], x[1]), f2_pack(x[2], x[3])}}; }
template <bool WIDE>
TW_DEV Quad load4(const float* p, int n) {
  if (WIDE) {
    const ulonglong2 v = *reinterpret_cast<const ulonglong2*>(p);
    return Quad{{v.x, v.y}};
  }
  float x[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) x[j] = j < n ? p[j] : 0.0f;
  return quad(x);
}
template <bool WIDE>
TW_DEV Quad load4(const uint16_t* p, int n) {
  if (WIDE) {
    const uint2 v = *reinterpret_cast<const uint2*>(p);
    return Quad{{bf2_to_f2(v.x), bf2_to_f2(v.y)}};
  }
  float x[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) x[j] = j < n ? bf16_bits_to_float(p[j]) : 0.0f;
  return quad(x);
}
template <bool WIDE>
TW_DEV void store4(float* p, int n, const Quad& x) {
  if (WIDE) {
    *reinterpret_cast<ulonglong2*>(p) = make_ulonglong2(x.v[0], x.v[1]);
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (j < n) p[j] = x.get(j);
  }
}
template <bool WIDE>
TW_DEV void store4(uint16_t* p, int n, const Quad& x) {
  if (WIDE) {
    *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16x2(f2_lo(x.v[0]), f2_hi(x.v[0])),
                                              pack_bf16x2(f2_lo(x.v[1]), f2_hi(x.v[1])));
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (j < n) p[j] = __bfloat16_as_ushort(__float2bfloat16_rn(x.get(j)));
  }
}
template <bool WIDE>
TW_DEV uint32_t load_codes(const uint8_t* p, int n) {
  if (WIDE) return *reinterpret_cast<const uint32_t*>(p);
  uint32_t v = 0;
#pragma unroll
  for (int j = 0; j < 4; ++j)
    if (j < n) v |= (uint32_t)p[j] << (8 * j);
  return v;
}
template <bool WIDE>
TW_DEV void store_codes(uint8_t* p, int n, uint32_t v) {
  if (WIDE) {
    *reinterpret_cast<uint32_t*>(p) = v;
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (j < n) p[j] = (uint8_t)(v >> (8 * j));
  }
}
TW_DEV uint64_t e4m3_pair(uint32_t codes) {
  const float2 f = __half22float2(
      __half2(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)codes, __NV_E4M3)));
  return f2_pack(f.x, f.y);
}
TW_DEV Quad decode4(uint32_t codes, float scale) {
  const uint64_t s2 = f2_splat(scale);
  return Quad{{f2_mul(e4m3_pair(codes & 0xFFFFu), s2), f2_mul(e4m3_pair(codes >> 16), s2)}};
}

TW_DEV float warp_max(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}
TW_DEV float rcp_approx(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// The 8-bit form of a block's m and r = sqrt(v): scales from the maxima over
// the warp, codes for this lane's 8 elements.
template <bool WIDE, bool ODD>
TW_DEV void store_block(const Entry& e, const Hyper& H, long long blk, int lane, int n,
                        const Quad (&m)[2], const Quad (&r)[2], float m_max, float r_max) {
  m_max = fmaxf(m_max, kTinyMax);
  r_max = fmaxf(r_max, kTinyMax);
  const uint64_t mi = f2_splat(__fmul_rn(__frcp_rn(m_max), kE4m3Max));
  const uint64_t ri = f2_splat(__fmul_rn(__frcp_rn(r_max), kE4m3Max));
  const uint64_t shift = f2_splat(kE4m3Shift);
  const long long i0 = blk * kBlock + 4 * lane;
  // a block's numbers differ in the low 8 bits alone: one high word for all
  const unsigned long long number = (unsigned long long)(e.number + i0);
  const uint32_t x0 = (uint32_t)number * kSpreadLo + (uint32_t)(number >> 32) * kSpreadHi + H.key;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint32_t mc[4], vc[4];
#pragma unroll
    for (int j = 0; j < 4; j += 2) {
      const uint64_t mb = f2_mul(f2_mul(m[h].v[j >> 1], mi), shift);
      const uint64_t rb = f2_mul(f2_mul(r[h].v[j >> 1], ri), shift);
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const Random rnd = hash_bits(x0 + (uint32_t)(128 * h + j + q) * kSpreadLo);
        mc[j + q] = signed_code<ODD>((uint32_t)(mb >> (32 * q)), rnd.lo);
        // v > 0 stays above zero
        const uint32_t least = min((uint32_t)(r[h].v[j >> 1] >> (32 * q)), 1u);
        vc[j + q] = positive_code<ODD>((uint32_t)(rb >> (32 * q)), rnd.hi, least);
      }
    }
    store_codes<WIDE>(reinterpret_cast<uint8_t*>(e.m) + i0 + 128 * h, n - 128 * h,
                      bytes4(mc[0], mc[1], mc[2], mc[3]));
    store_codes<WIDE>(reinterpret_cast<uint8_t*>(e.v) + i0 + 128 * h, n - 128 * h,
                      bytes4(vc[0], vc[1], vc[2], vc[3]));
  }
  if (lane == 0) {
    e.m_scale[blk] = __fmul_rn(m_max, 1.0f / kE4m3Max);
    e.v_scale[blk] = __fmul_rn(r_max, 1.0f / kE4m3Max);
  }
}

// A warp's step over U blocks of 256 elements, kWarps blocks apart, all loaded
// before the first is worked on.  Lane l takes the elements 4 l .. 4 l + 3 of a block
// and the same from 128 on: with aligned tensors (WIDE) every access of a warp is
// one contiguous stretch, and the maxima behind the scales are a warp's.
// fp32 arithmetic runs on pairs.  The moments' products and sums are rounded
// one by one, so that 8-bit codes do not depend on what is contracted: as pairs
// even mul.rn and add.rn are fused into one FMA (18 % of random sums came out
// fused), so the sum is an FMA with a factor of 1 that only the host knows.
constexpr int kWarps = 8;
template <typename P, typename G, int BITS, bool WIDE, int U>
TW_DEV void step_blocks(const Entry& e, const Hyper& H, const Corrections& C, float gs, long long blk0,
                        int lane) {
  Quad g[U][2], p[U][2], m[U][2], r[U][2];
  uint32_t mc[U][2], vc[U][2];
  float ms[U], vs[U];
  int left[U];  // elements from this lane's first one to the block's or the tensor's end
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const long long blk = blk0 + u * kWarps, i0 = blk * kBlock + 4 * lane;
    left[u] = WIDE ? kBlock : (int)min(max(e.n - i0, 0ll), (long long)kBlock);
    if (BITS == 8) {
      const bool any = WIDE || blk * kBlock < e.n;
      ms[u] = any ? e.m_scale[blk] : 0.0f;
      vs[u] = any ? e.v_scale[blk] : 0.0f;
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const long long i = i0 + 128 * h;
      const int n = left[u] - 128 * h;
      g[u][h] = load4<WIDE>(reinterpret_cast<const G*>(e.grad) + i, n);
      p[u][h] = load4<WIDE>(reinterpret_cast<const P*>(e.param) + i, n);
      if (BITS == 32) {
        m[u][h] = load4<WIDE>(reinterpret_cast<const float*>(e.m) + i, n);
        r[u][h] = load4<WIDE>(reinterpret_cast<const float*>(e.v) + i, n);
      } else {
        mc[u][h] = load_codes<WIDE>(reinterpret_cast<const uint8_t*>(e.m) + i, n);
        vc[u][h] = load_codes<WIDE>(reinterpret_cast<const uint8_t*>(e.v) + i, n);
      }
    }
  }
  const uint64_t gs2 = f2_splat(gs), b1 = f2_splat(H.beta1), c1 = f2_splat(H.one_beta1);
  const uint64_t b2 = f2_splat(H.beta2), c2 = f2_splat(H.one_beta2), decay = f2_splat(H.decay);
  const uint64_t one = f2_splat(H.one), size = f2_splat(-C.size), inv = f2_splat(C.inv_root), eps = f2_splat(H.eps);
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const long long blk = blk0 + u * kWarps, i0 = blk * kBlock + 4 * lane;
    if (!WIDE && blk * kBlock >= e.n) return;  // the whole warp
    uint32_t m_bits = 0, r_bits = 0;  // largest magnitudes as bits: NaN is above all
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const long long i = i0 + 128 * h;
      const int n = left[u] - 128 * h;
      if (BITS == 8) {
        m[u][h] = decode4(mc[u][h], ms[u]);
        r[u][h] = decode4(vc[u][h], vs[u]);
      }
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const uint64_t x = f2_mul(g[u][h].v[q], gs2);
        uint64_t& mm = m[u][h].v[q];
        uint64_t& vv = r[u][h].v[q];
        if (BITS == 8) vv = f2_mul(vv, vv);
        mm = f2_fma(f2_mul(b1, mm), one, f2_mul(c1, x));
        vv = f2_fma(f2_mul(b2, vv), one, f2_mul(c2, f2_mul(x, x)));
      }
      if (BITS == 32) {
        store4<WIDE>(reinterpret_cast<float*>(e.m) + i, n, m[u][h]);
        store4<WIDE>(reinterpret_cast<float*>(e.v) + i, n, r[u][h]);
      }
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        uint64_t& vv = r[u][h].v[q];
        vv = f2_pack(__fsqrt_rn(f2_lo(vv)), __fsqrt_rn(f2_hi(vv)));
        const uint64_t den = f2_fma(vv, inv, eps);
        const uint64_t quot = f2_pack(rcp_approx(f2_lo(den)), rcp_approx(f2_hi(den)));
        p[u][h].v[q] = f2_fma(p[u][h].v[q], decay, f2_mul(f2_mul(size, m[u][h].v[q]), quot));
        if (BITS == 8) {
          m_bits = max(m_bits, max((uint32_t)m[u][h].v[q] & 0x7FFFFFFFu,
                                   (uint32_t)(m[u][h].v[q] >> 32) & 0x7FFFFFFFu));
          r_bits = max(r_bits, max((uint32_t)vv, (uint32_t)(vv >> 32)));  // roots have no sign
        }
      }
      store4<WIDE>(reinterpret_cast<P*>(e.param) + i, n, p[u][h]);
      if (e.copy) store4<WIDE>(e.copy + i, n, p[u][h]);
    }
    if (BITS == 32) continue;
    m_bits = __reduce_max_sync(0xffffffffu, m_bits);
    r_bits = __reduce_max_sync(0xffffffffu, r_bits);
    if (max(m_bits, r_bits) < 0x7F800000u) {
      store_block<WIDE, false>(e, H, blk, lane, left[u], m[u], r[u], __uint_as_float(m_bits),
                               __uint_as_float(r_bits));
    } else {  // a NaN does not count for the scales
      float m_max = 0.0f, r_max = 0.0f;
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          m_max = fmaxf(m_max, fabsf(m[u][h].get(j)));
          r_max = fmaxf(r_max, r[u][h].get(j));
        }
      store_block<WIDE, true>(e, H, blk, lane, left[u], m[u], r[u], warp_max(m_max),
                              warp_max(r_max));
    }
  }
}

// Blocks of 256 that a warp takes at once.  32-bit states keep the memory busy
// with one (101 M parameters, 22 to 28 bytes each: 103 to 104 % of the copy rate); 8-bit
// ones move 10 to 18 bytes and need two, with four thread blocks to an SM (fp32
// parameters and gradients 231 us; one block of 256 and six thread blocks 238 us, two
// and three 248 us, four and two 266 us, all in one run; 231 to 247 us from run to run).
__host__ __device__ constexpr int blocks_of(int bits) { return bits == 32 ? 1 : 2; }

template <typename P, typename G, int BITS, int MAX, bool COUNTED>
__global__ void __launch_bounds__(32 * kWarps, BITS == 8 ? 4 : 5)
    adamw_kernel(const __grid_constant__ List<MAX> L, const Hyper H) {
  constexpr int U = blocks_of(BITS);
  const float gs = H.grad_scale ? *H.grad_scale : 1.0f;
  const int skipped = COUNTED ? *reinterpret_cast<volatile const int*>(H.skipped) : 0;
  if (!(fabsf(gs) <= 3.402823466e38f)) {  // NaN or infinite: the step changes nothing
    // (and no block uses the count that this one changes)
    if (COUNTED && H.count_skip && blockIdx.x == 0 && threadIdx.x == 0) atomicAdd(H.skipped, 1);
    return;
  }
  const Corrections C = COUNTED ? corrections(H, skipped) : Corrections{H.size, H.inv_root};
  // last chunks first: those whose gradients the norm read last are still in L2
  const int chunk = (int)(gridDim.x - 1 - blockIdx.x);
  const Entry& e = L.e[find_entry(L, chunk)];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long long blk0 = (long long)(chunk - e.chunk) * (U * kWarps) + warp;
  if (e.wide && (blk0 + (U - 1) * kWarps + 1) * kBlock <= e.n)
    step_blocks<P, G, BITS, true, U>(e, H, C, gs, blk0, lane);
  else
    step_blocks<P, G, BITS, false, U>(e, H, C, gs, blk0, lane);
}

// ------------------------------------------------------------------ norm
constexpr int kNormBlocks = 1024;  // most partial sums (fp64) in the workspace

struct GradEntry {
  const void* grad;
  long long n;
  int chunk;
  int wide;
};
template <int MAX>
struct GradList {
  GradEntry e[MAX];
  int count, chunks, first;  // first launch of the norm: partials start at zero
};

// A block takes chunks of kNormChunk elements gridDim.x apart; a thread sums
// 32 squares of each in fp32, then adds them to its fp64 sum.
constexpr int kNormChunk = 8192;
template <typename G, int MAX>
__global__ void __launch_bounds__(256)
    grad_norm_kernel(const __grid_constant__ GradList<MAX> L, double* part) {
  launch_dependents();
  double acc = 0.0;
  for (int c = blockIdx.x; c < L.chunks; c += gridDim.x) {
    const GradEntry& e = L.e[find_entry(L, c)];
    const long long base = (long long)(c - e.chunk) * kNormChunk;
    const G* g = reinterpret_cast<const G*>(e.grad) + base + 4 * threadIdx.x;
    const bool wide = e.wide && base + kNormChunk <= e.n;
    const int left = (int)min(e.n - base, (long long)kNormChunk) - 4 * (int)threadIdx.x;
    float s = 0.0f;
    Quad x[8];
    if (wide) {
#pragma unroll
      for (int h = 0; h < 8; ++h) x[h] = load4<true>(g + 1024 * h, 4);
    } else {
#pragma unroll
      for (int h = 0; h < 8; ++h) x[h] = load4<false>(g + 1024 * h, left - 1024 * h);
    }
    uint64_t s2 = 0;
#pragma unroll
    for (int h = 0; h < 8; ++h)
#pragma unroll
      for (int q = 0; q < 2; ++q) s2 = f2_fma(x[h].v[q], x[h].v[q], s2);
    s = f2_sum(s2);
    acc += (double)s;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, o);
  __shared__ double sh[8];
  if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = acc;
  __syncthreads();
  if (threadIdx.x == 0) {
    acc = L.first ? 0.0 : part[blockIdx.x];
    for (int i = 0; i < 8; ++i) acc += sh[i];
    part[blockIdx.x] = acc;
  }
}

// (fp64 additions are scarce: 256 threads with up to four partial sums each take
// less of them than 1024 with one.)
constexpr int kJoinThreads = 256;
__global__ void __launch_bounds__(kJoinThreads)
    grad_norm_join_kernel(const double* part, int n, float max_norm, float* out) {
  wait_for_previous();
  double d = 0.0;
#pragma unroll
  for (int i = 0; i < kNormBlocks / kJoinThreads; ++i) {
    const int k = i * kJoinThreads + (int)threadIdx.x;
    d += k < n ? part[k] : 0.0;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) d += __shfl_xor_sync(0xffffffffu, d, o);
  __shared__ double sh[kJoinThreads / 32];
  if ((threadIdx.x & 31) == 0) sh[threadIdx.x >> 5] = d;
  __syncthreads();
  if (threadIdx.x != 0) return;
  for (int i = 1; i < kJoinThreads / 32; ++i) d += sh[i];
  const float norm = (float)sqrt(d);
  out[0] = norm;
  out[1] = !(norm <= 3.402823466e38f) ? __int_as_float(0x7FC00000) : norm > max_norm ? max_norm / norm : 1.0f;
}

// ------------------------------------------------------------------ host side
bool off(const void* p, uintptr_t bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) != 0; }
uintptr_t bytes_of(int dtype) { return dtype == TWELL_F32 ? 4 : 2; }
bool is_dtype(int d) { return d == TWELL_BF16 || d == TWELL_F32; }

// Most elements of one tensor: chunk numbers are 32-bit.
constexpr long long kMaxElements = 1ll << 40;

twell_status check_list(const twell_param* p, int count, int grad_dtype) {
  if (count < 0 || (count > 0 && !p) || !is_dtype(grad_dtype)) return TWELL_ERR_INVALID_ARG;
  for (int i = 0; i < count; ++i) {
    if (p[i].n < 0 || (p[i].n > 0 && !p[i].grad)) return TWELL_ERR_INVALID_ARG;
    if (p[i].n > kMaxElements) return TWELL_ERR_UNSUPPORTED;
    if (p[i].n > 0 && off(p[i].grad, bytes_of(grad_dtype))) return TWELL_ERR_ALIGNMENT;
  }
  return TWELL_OK;
}

long long chunks_of(long long n, long long size) { return (n + size - 1) / size; }

uint32_t step_key(uint64_t seed, int64_t step) {
  uint64_t x = seed + (uint64_t)step * 0x9E3779B97F4A7C15ull;
  x = (x ^ (x >> 30)) * 0xBF58476D1CE4E5B9ull;
  x = (x ^ (x >> 27)) * 0x94D049BB133111EBull;
  return (uint32_t)((x ^ (x >> 31)) >> 32);
}

// Shorter lists travel in smaller parameter blocks: a full one of 32 KB costs a
// launch about 4 us to submit (120 tensors: 8 us, one tensor 4 us).
constexpr int kFewTensors = 24, kSomeTensors = 128;

template <template <int> class L_, int MAX>
L_<MAX> shorter(const L_<kMaxTensors>& L) {
  L_<MAX> f;
  f.count = L.count;
  for (int i = 0; i < L.count; ++i) f.e[i] = L.e[i];
  return f;
}

template <typename P, typename G, int BITS, bool COUNTED>
void adamw_run(int grid, const List<kMaxTensors>& L, const Hyper& H, cudaStream_t s) {
  if (L.count <= kFewTensors)
    adamw_kernel<P, G, BITS, kFewTensors, COUNTED>
        <<<grid, 32 * kWarps, 0, s>>>(shorter<List, kFewTensors>(L), H);
  else if (L.count <= kSomeTensors)
    adamw_kernel<P, G, BITS, kSomeTensors, COUNTED>
        <<<grid, 32 * kWarps, 0, s>>>(shorter<List, kSomeTensors>(L), H);
  else
    adamw_kernel<P, G, BITS, kMaxTensors, COUNTED><<<grid, 32 * kWarps, 0, s>>>(L, H);
}

template <typename P, typename G>
void adamw_run(int bits, int grid, const List<kMaxTensors>& L, const Hyper& H, cudaStream_t s) {
  if (bits == 8)
    H.skipped ? adamw_run<P, G, 8, true>(grid, L, H, s) : adamw_run<P, G, 8, false>(grid, L, H, s);
  else
    H.skipped ? adamw_run<P, G, 32, true>(grid, L, H, s) : adamw_run<P, G, 32, false>(grid, L, H, s);
}

// Elements per thread block.
long long chunk_size(const twell_adamw* a) {
  return (long long)blocks_of(a->state_bits) * kWarps * kBlock;
}

cudaError_t adamw_launch(const twell_adamw* a, int grid, const List<kMaxTensors>& L,
                         const Hyper& H, cudaStream_t s) {
  ProfScope prof("adamw", s);
  const bool pf = a->param_dtype == TWELL_F32, gf = a->grad_dtype == TWELL_F32;
  if (pf && gf)
    adamw_run<float, float>(a->state_bits, grid, L, H, s);
  else if (pf)
    adamw_run<float, uint16_t>(a->state_bits, grid, L, H, s);
  else if (gf)
    adamw_run<uint16_t, float>(a->state_bits, grid, L, H, s);
  else
    adamw_run<uint16_t, uint16_t>(a->state_bits, grid, L, H, s);
  count_launch();
  return cudaGetLastError();
}

template <typename G, int MAX>
void grad_norm_shorter(int grid, const GradList<kMaxTensors>& L, double* part, cudaStream_t s) {
  GradList<MAX> f = shorter<GradList, MAX>(L);
  f.chunks = L.chunks;
  f.first = L.first;
  grad_norm_kernel<G, MAX><<<grid, 256, 0, s>>>(f, part);
}
template <typename G>
void grad_norm_run(int grid, const GradList<kMaxTensors>& L, double* part, cudaStream_t s) {
  if (L.count <= kFewTensors)
    grad_norm_shorter<G, kFewTensors>(grid, L, part, s);
  else if (L.count <= kSomeTensors)
    grad_norm_shorter<G, kSomeTensors>(grid, L, part, s);
  else
    grad_norm_kernel<G, kMaxTensors><<<grid, 256, 0, s>>>(L, part);
}

// Whether every pointer of an entry is aligned to four of its elements.
bool is_wide(const twell_param& p, const twell_adamw* a) {
  const uintptr_t st = a->state_bits == 8 ? 4 : 16;
  return !off(p.param, 4 * bytes_of(a->param_dtype)) && !off(p.grad, 4 * bytes_of(a->grad_dtype)) &&
         !off(p.copy, 8) && !off(p.m, st) && !off(p.v, st);
}

}  // namespace

}  // namespace tw

using namespace tw;

extern "C" {

size_t twell_grad_norm_workspace_bytes(void) { return kNormBlocks * sizeof(double); }

twell_status twell_grad_norm(const twell_param* params, int32_t count, int32_t grad_dtype,
                             float max_norm, float* out, void* ws, size_t ws_bytes, void* stream) {
  NvtxRange nvtx("twell_grad_norm");
  twell_status st = check_list(params, count, grad_dtype);
  if (st != TWELL_OK) return st;
  if (!out || !(max_norm > 0.0f)) return TWELL_ERR_INVALID_ARG;
  if (!ws || ws_bytes < twell_grad_norm_workspace_bytes()) return TWELL_ERR_WORKSPACE;
  if (off(out, 4) || off(ws, 16)) return TWELL_ERR_ALIGNMENT;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  double* part = reinterpret_cast<double*>(ws);
  GradList<kMaxTensors> L;
  L.count = L.chunks = 0;
  L.first = 1;
  // The first launch's grid writes every partial sum that the join reads; more
  // launches add to them.  4 blocks an SM that loop beat one block a chunk.
  long long all = 0, chunks = 0;
  for (int i = 0; i < count; ++i) all += chunks_of(params[i].n, kNormChunk);
  const int most = 4 * num_sms() < kNormBlocks ? 4 * num_sms() : kNormBlocks;
  const int grid = all < 1 ? 1 : all < most ? (int)all : most;
  auto flush = [&]() -> cudaError_t {
    L.chunks = (int)chunks;
    ProfScope prof("grad_norm", s);
    if (grad_dtype == TWELL_F32)
      grad_norm_run<float>(grid, L, part, s);
    else
      grad_norm_run<uint16_t>(grid, L, part, s);
    count_launch();
    L.first = L.count = 0;
    chunks = 0;
    return cudaGetLastError();
  };
  for (int i = 0; i < count; ++i) {
    if (params[i].n == 0) continue;
    const long long c = chunks_of(params[i].n, kNormChunk);
    if ((L.count == kMaxTensors || chunks + c > 0x7FFFFFFF) && flush() != cudaSuccess)
      return TWELL_ERR_CUDA;
    L.e[L.count++] = GradEntry{params[i].grad, params[i].n, (int)chunks,
                               !off(params[i].grad, 4 * bytes_of(grad_dtype))};
    chunks += c;
  }
  if ((L.count > 0 || L.first) && flush() != cudaSuccess) return TWELL_ERR_CUDA;
  ProfScope prof("grad_norm_join", s);
  const cudaError_t e = launch_after(grad_norm_join_kernel, 1, kJoinThreads, s, (const double*)part, grid,
                                     max_norm, out);
  count_launch();
  return e == cudaSuccess && cudaGetLastError() == cudaSuccess ? TWELL_OK : TWELL_ERR_CUDA;
}

twell_status twell_adamw_step(const twell_param* params, int32_t count, const twell_adamw* hyper,
                              void* stream) {
  NvtxRange nvtx("twell_adamw_step");
  const twell_adamw* a = hyper;
  if (!a || !is_dtype(a->param_dtype)) return TWELL_ERR_INVALID_ARG;
  if (a->state_bits != 8 && a->state_bits != 32) return TWELL_ERR_INVALID_ARG;
  if (a->step < 1) return TWELL_ERR_INVALID_ARG;
  if (!(a->lr >= 0.0) || !(a->eps >= 0.0) || !(a->weight_decay >= 0.0) || !isfinite(a->lr) ||
      !isfinite(a->eps) || !isfinite(a->weight_decay) || !(a->beta1 >= 0.0 && a->beta1 < 1.0) ||
      !(a->beta2 >= 0.0 && a->beta2 < 1.0))
    return TWELL_ERR_INVALID_ARG;
  twell_status st = check_list(params, count, a->grad_dtype);
  if (st != TWELL_OK) return st;
  if (off(a->grad_scale, 4) || off(a->skipped, 4)) return TWELL_ERR_ALIGNMENT;
  for (int i = 0; i < count; ++i) {
    const twell_param& p = params[i];
    if (p.n == 0) continue;
    if (!p.param || !p.m || !p.v) return TWELL_ERR_INVALID_ARG;
    if (a->state_bits == 8 && (!p.m_scale || !p.v_scale)) return TWELL_ERR_INVALID_ARG;
    if (off(p.param, bytes_of(a->param_dtype)) || off(p.copy, 2)) return TWELL_ERR_ALIGNMENT;
    if (a->state_bits == 32 ? off(p.m, 4) || off(p.v, 4) : off(p.m_scale, 4) || off(p.v_scale, 4))
      return TWELL_ERR_ALIGNMENT;
  }
  Hyper H;
  H.one = 1.0f;
  H.beta1 = (float)a->beta1;
  H.one_beta1 = (float)(1.0 - a->beta1);
  H.beta2 = (float)a->beta2;
  H.one_beta2 = (float)(1.0 - a->beta2);
  H.decay = (float)(1.0 - a->lr * a->weight_decay);
  H.size = (float)(a->lr / (1.0 - pow(a->beta1, (double)a->step)));
  H.inv_root = (float)(1.0 / sqrt(1.0 - pow(a->beta2, (double)a->step)));
  H.eps = (float)a->eps;
  H.key = step_key(a->seed, a->step);
  H.grad_scale = a->grad_scale;
  H.skipped = a->skipped;
  H.count_skip = a->skipped != nullptr;
  H.step = (float)a->step;
  H.lr = (float)a->lr;
  H.ln_beta1 = (float)log(a->beta1);  // -inf at 0: no correction
  H.ln_beta2 = (float)log(a->beta2);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  List<kMaxTensors> L;
  L.count = 0;
  const long long size = chunk_size(a);
  long long chunks = 0, number = 0;
  for (int i = 0; i < count; ++i) {
    const twell_param& p = params[i];
    if (p.n == 0) continue;
    const long long c = chunks_of(p.n, size);
    if (L.count == kMaxTensors || chunks + c > 0x7FFFFFFF) {
      if (adamw_launch(a, (int)chunks, L, H, s) != cudaSuccess) return TWELL_ERR_CUDA;
      L.count = 0;
      chunks = 0;
      H.count_skip = 0;
    }
    L.e[L.count++] = Entry{p.param, reinterpret_cast<uint16_t*>(p.copy), p.grad, p.m, p.v,
                           p.m_scale, p.v_scale, p.n, number, (int)chunks,
                           is_wide(p, a)};
    chunks += c;
    number += (p.n + kBlock - 1) / kBlock * kBlock;
  }
  if (L.count > 0 && adamw_launch(a, (int)chunks, L, H, s) != cudaSuccess) return TWELL_ERR_CUDA;
  return TWELL_OK;
}

}  // extern "C"
