// logits_loss.cu -- losses over logits and their gradients: token
// log-probabilities, the clipped policy loss with its KL term, the preference
// loss on pairs of answers, and the gradient through log-probabilities.
//
// With z = scale * x (x a row of logits) and X = max x:
//   s = sum_v exp(scale (x_v - X)),  lse = scale X + ln s,
//   logp = scale (x_y - X) - ln s,  softmax_v = exp(scale (x_v - X)) / s.
// The difference is taken first, so neither a large offset of the logits nor
// a mask of the type's lowest value loses or overflows anything.
//
// Times below are of whole calls in a row, by events, with no row ignored, inputs
// that do not fit L2 or alternate, and the SMs at 2070 MHz.
#include <math.h>

#include "common.cuh"
#include "internal.h"

namespace tw {

namespace {

// exp(scale d) = 2^(k d), k = scale log2(e) as the sum of two floats: with k
// rounded to one, every exponent would be off by the same 2^-25 of itself, an
// error that does not average out over a sequence's tokens.  lo > 0, so that
// d = -inf stays -inf.
struct ExpK {
  float hi, lo;
};
TW_DEV float ex2(float t) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(t));
  return r;
}
// ex2.approx is low by 5e-8 of its value on average for arguments below -1
// (-4.9e-8 to -5.2e-8 over 4 M random arguments in each of several octaves;
// 3e-8 rms around that) and by 2e-8 between -1 and 0.  A row's sum keeps the
// mean and averages the rest away, and a sequence's log-probability adds it up
// over the tokens, so sums are raised by it; a sum of 1 (one entry) stays 1.
// (The mean error of a log-probability at 128000 entries goes from 1e-7 to 1e-8.)
TW_DEV float raise(float s) { return fmaf(s, 5e-8f, s); }
TW_DEV float exp_k(float d, const ExpK& k) { return ex2(fmaf(d, k.hi, d * k.lo)); }
ExpK make_exp_k(double scale) {
  const double k = scale * 1.4426950408889634074;
  float hi = (float)k;
  if ((double)hi >= k) hi = nextafterf(hi, 0.0f);
  const float lo = (float)(k - (double)hi);
  return ExpK{hi, lo > 0.0f ? lo : nextafterf(0.0f, 1.0f)};  // it underflows only below 2^-97
}

struct Rows {
  const void* x;
  const void* target;
  long long stride;
  int rows, vocab;
  int target_i64;
  float scale;
  ExpK k;  // of scale
  int* status;
};

// Above this magnitude a log-sum-exp in fp32 no longer holds ln s to 2^-17.
constexpr float kLseExact = 128.0f;

struct Policy {
  const float *adv, *weight, *old_logp, *ref_logp;
  float lo, hi, kl;
};

TW_DEV float load1(const uint16_t* p) { return bf16_bits_to_float(*p); }
TW_DEV float load1(const float* p) { return *p; }
TW_DEV void store1(uint16_t* p, float v) { *p = __bfloat16_as_ushort(__float2bfloat16_rn(v)); }
TW_DEV void store1(float* p, float v) { *p = v; }

// The row's target as it stands in memory, and as the kernels use it: -1 for an ignored row.
TW_DEV long long raw_target(const Rows& R, int t) {
  return R.target_i64 ? reinterpret_cast<const long long*>(R.target)[t]
                      : (long long)reinterpret_cast<const int*>(R.target)[t];
}
TW_DEV int check_target(const Rows& R, long long y) {
  if (y >= R.vocab) set_status(R.status, TWELL_ERR_INDEX);
  return y < 0 || y >= R.vocab ? -1 : (int)y;
}
TW_DEV int row_target(const Rows& R, int t) { return check_target(R, raw_target(R, t)); }

template <bool B>
struct Bool {
  static constexpr bool value = B;
};

// ---- rows as 16-byte chunks
// Chunk c of a row holds the elements at bytes 16 c .. 16 c + 15 from the
// 16-byte boundary at or before the row's start.  Whole chunks are read and
// written as vectors whatever the row's alignment; the row's first and last
// one may be partial and are taken element by element, with -inf (probability
// zero) in the places outside the row.
template <typename E>
struct Vec;
template <>
struct Vec<uint16_t> {
  static constexpr int kN = 8;
  static constexpr uint32_t kFill = 0xFF80FF80u;  // -inf, -inf
  // running maxima of the even and the odd elements, as bf16
  using Max = __nv_bfloat162;
  TW_DEV static Max max_none() { return __float2bfloat162_rn(-INFINITY); }
  TW_DEV static Max max_with(Max m, const uint4& v) {
    const __nv_bfloat162* w = reinterpret_cast<const __nv_bfloat162*>(&v);
    return __hmax2(m, __hmax2(__hmax2(w[0], w[1]), __hmax2(w[2], w[3])));
  }
  TW_DEV static float max_of(Max m) { return fmaxf(__low2float(m), __high2float(m)); }
  TW_DEV static void pairs(const uint4& v, uint64_t (&o)[4]) { bf8_to_f2(v, o); }
  // x - m: as x * 1 + (-m) the FMA takes the bf16 halves as they are
  TW_DEV static void minus(const uint4& v, float m, uint64_t (&o)[4]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float lo = -m, hi = -m;
      bf16_fma(lo, w[i], 0x3F803F80u, false);
      bf16_fma(hi, w[i], 0x3F803F80u, true);
      o[i] = f2_pack(lo, hi);
    }
  }
};
template <>
struct Vec<float> {
  static constexpr int kN = 4;
  static constexpr uint32_t kFill = 0xFF800000u;
  using Max = float;
  TW_DEV static Max max_none() { return -INFINITY; }
  TW_DEV static Max max_with(Max m, const uint4& v) {
    return fmaxf(m, fmaxf(fmaxf(__uint_as_float(v.x), __uint_as_float(v.y)),
                          fmaxf(__uint_as_float(v.z), __uint_as_float(v.w))));
  }
  TW_DEV static float max_of(Max m) { return m; }
  TW_DEV static void pairs(const uint4& v, uint64_t (&o)[2]) {
    o[0] = f2_make(v.x, v.y);
    o[1] = f2_make(v.z, v.w);
  }
  TW_DEV static void minus(const uint4& v, float m, uint64_t (&o)[2]) {
    const uint64_t neg = f2_splat(-m);
    o[0] = f2_add(f2_make(v.x, v.y), neg);
    o[1] = f2_add(f2_make(v.z, v.w), neg);
  }
};

template <typename E>
struct Row {
  const E* x;     // the row's first element
  int head;       // elements of chunk 0 that lie before it
  int vocab, chunks;
  TW_DEV Row(const void* data, long long offset, int vocab_) {
    x = reinterpret_cast<const E*>(data) + offset;
    head = (int)((reinterpret_cast<uintptr_t>(x) & 15u) / sizeof(E));
    vocab = vocab_;
    chunks = (int)(((long long)head + vocab + Vec<E>::kN - 1) / Vec<E>::kN);
  }
  // first element of chunk c; negative in a partial first chunk
  TW_DEV int first(int c) const { return c * Vec<E>::kN - head; }
  TW_DEV bool whole(int c) const { return first(c) >= 0 && first(c) <= vocab - Vec<E>::kN; }
  // whether the chunks c, c + step, .. c + (count - 1) step of each lane of a warp
  // are whole, c being its first lane's
  TW_DEV bool plain(int c, int step, int count) const {
    return c >= (head ? 1 : 0) &&
           c + (count - 1) * step + 32 <= (head + vocab) / Vec<E>::kN;
  }
  // LAST: nothing reads the chunk again
  template <bool LAST>
  TW_DEV uint4 load_whole(int c) const {
    const uint4* p = reinterpret_cast<const uint4*>(x + first(c));
    return LAST ? __ldcs(p) : *p;
  }
  template <bool LAST>
  TW_DEV uint4 load(int c) const {
    const int v0 = first(c);
    if (whole(c)) return load_whole<LAST>(c);
    uint4 r = make_uint4(Vec<E>::kFill, Vec<E>::kFill, Vec<E>::kFill, Vec<E>::kFill);
    E* e = reinterpret_cast<E*>(&r);
#pragma unroll
    for (int i = 0; i < Vec<E>::kN; ++i)
      if (v0 + i >= 0 && v0 + i < vocab) e[i] = x[v0 + i];
    return r;
  }
  // Whether a gradient row's chunks are aligned as the row's own are.
  TW_DEV bool even(const E* d) const {
    return ((reinterpret_cast<uintptr_t>(d) - reinterpret_cast<uintptr_t>(x)) & 15u) == 0;
  }
  TW_DEV void store_whole(E* d, int c, const uint4& r) const {
    __stcs(reinterpret_cast<uint4*>(d + first(c)), r);
  }
  // Writes the chunk's elements of a gradient row d.
  TW_DEV void store(E* d, int c, const uint4& r) const {
    const int v0 = first(c);
    const uint32_t off = (uint32_t)(reinterpret_cast<uintptr_t>(d + v0) & 15u);
    if (whole(c) && off == 0) {
      __stcs(reinterpret_cast<uint4*>(d + v0), r);
    } else if (whole(c) && off == 8) {
      __stcs(reinterpret_cast<uint2*>(d + v0), make_uint2(r.x, r.y));
      __stcs(reinterpret_cast<uint2*>(d + v0) + 1, make_uint2(r.z, r.w));
    } else if (whole(c) && (off & 3) == 0) {
      uint32_t* p = reinterpret_cast<uint32_t*>(d + v0);
      p[0] = r.x;
      p[1] = r.y;
      p[2] = r.z;
      p[3] = r.w;
    } else {
      const E* e = reinterpret_cast<const E*>(&r);
#pragma unroll
      for (int i = 0; i < Vec<E>::kN; ++i)
        if (v0 + i >= 0 && v0 + i < vocab) d[v0 + i] = e[i];
    }
  }
};

// sum + the chunk's exp(scale (x - m)), pairwise
template <typename E>
TW_DEV uint64_t sum_exp(const uint4& v, float m, const ExpK& k, uint64_t acc) {
  uint64_t p[Vec<E>::kN / 2];
  Vec<E>::minus(v, m, p);
  const uint64_t hi = f2_splat(k.hi), lo = f2_splat(k.lo);
#pragma unroll
  for (int i = 0; i < Vec<E>::kN / 2; ++i) {
    const uint64_t t = f2_fma(p[i], hi, f2_mul(p[i], lo));
    acc = f2_add(acc, f2_pack(ex2(f2_lo(t)), ex2(f2_hi(t))));
  }
  return acc;
}

// q exp(scale (x - m)) as 2^(k x + b) q2, one FMA for the exponent: b = fl(-k m),
// and what that rounding leaves out of k m goes into q2, as 2^-rest = 1 - rest ln 2:
// good to 6e-8 while |k m| < 2^14, where |rest| <= 2^-11.  From there on (logits
// with a large offset, rows of nothing but a mask value, large scales) the
// difference is taken first: `far`.
constexpr float kNearExponent = 16384.0f;
struct Scaled {
  float k, b, q, m;
  bool far;
};
TW_DEV Scaled make_scaled(const ExpK& k, float m, float q) {
  const float mk = __fmul_rn(m, k.hi);
  if (!(fabsf(mk) < kNearExponent)) return Scaled{k.hi, 0.0f, q, m, true};
  const float rest = fmaf(m, k.hi, -mk);
  return Scaled{k.hi, -mk, q * fmaf(rest, -0.69314718f, 1.0f), m, false};
}
// ... of a chunk, rounded to E
template <typename E>
TW_DEV uint4 scaled_exp(const uint4& v, const Scaled& S) {
  uint64_t p[Vec<E>::kN / 2];
  if (S.far) {
    Vec<E>::minus(v, S.m, p);
  } else {
    Vec<E>::pairs(v, p);
  }
  const uint64_t k2 = f2_splat(S.k), b2 = f2_splat(S.b), q2 = f2_splat(S.q);
  uint32_t o[4];
#pragma unroll
  for (int i = 0; i < Vec<E>::kN / 2; ++i) {
    const uint64_t t = f2_fma(p[i], k2, b2);
    const uint64_t g = f2_mul(f2_pack(ex2(f2_lo(t)), ex2(f2_hi(t))), q2);
    if (sizeof(E) == 2) {
      o[i] = pack_bf16x2(f2_lo(g), f2_hi(g));
    } else {
      o[2 * i] = __float_as_uint(f2_lo(g));
      o[2 * i + 1] = __float_as_uint(f2_hi(g));
    }
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
}

// Running maximum m and s = sum of exp(scale (x - m)); (-inf, 0) is empty.
struct __align__(8) MaxSum {
  float m, s;
};
// a's sum over the maximum m of several parts: each part is rescaled once, to
// the last maximum, as every rescaling adds the error of an exponential.  An
// empty part (m = -inf) adds its s, 0 or NaN.
TW_DEV float rescaled(const MaxSum& a, float m, const ExpK& k) {
  if (a.m == m) return a.s;
  // maxima lie near each other, where ex2 is low by half of what raise() makes up for
  const float e = exp_k(a.m - m, k);
  return fmaf(a.s, e, a.s * e * 2.5e-8f);
}
// ln s; NaN for a row without a finite maximum (nothing but -inf, or a +inf).
TW_DEV float ln_sum(const MaxSum& a) { return fabsf(a.m) == INFINITY ? a.m - a.m : logf(a.s); }

// Adds NV chunks (those of `r` that are set) to a thread's statistics.
template <typename E, int NV>
TW_DEV void add_chunks(MaxSum& a, const uint4 (&r)[NV], int n, const ExpK& k) {
  typename Vec<E>::Max top = Vec<E>::max_none();
#pragma unroll
  for (int i = 0; i < NV; ++i)
    if (i < n) top = Vec<E>::max_with(top, r[i]);
  const float m = fmaxf(a.m, Vec<E>::max_of(top));
  a.s = rescaled(a, m, k);
  a.m = m;
  // an all -inf part keeps its 0: the difference of two -inf would be NaN
  const float ref = m == -INFINITY ? 0.0f : m;
  uint64_t acc = 0;
#pragma unroll
  for (int i = 0; i < NV; ++i)
    if (i < n) acc = sum_exp<E>(r[i], ref, k, acc);
  a.s += raise(f2_sum(acc));
}

TW_DEV float warp_max(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

// ---- thread-block clusters
TW_DEV uint32_t cluster_size() {
  uint32_t n;
  asm("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(n));
  return n;
}
TW_DEV uint32_t cluster_rank() {
  uint32_t n;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(n));
  return n;
}
// Every thread of every block of the cluster arrives and waits, in pairs.
TW_DEV void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
TW_DEV void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
// 8 bytes into the shared memory of block `rank` of the cluster, at the
// address `p` has in this block.
TW_DEV void st_cluster_b64(void* p, uint32_t rank, uint64_t v) {
  asm volatile(
      "{\n\t.reg .u32 a;\n\t"
      "mapa.shared::cluster.u32 a, %0, %1;\n\t"
      "st.shared::cluster.u64 [a], %2;\n\t}" ::"r"(smem_u32(p)),
      "r"(rank), "l"(v)
      : "memory");
}

constexpr int kMaxCluster = 8;

// G threads of a block take a row: a warp, some warps with a named barrier of
// their own, or the whole block.
template <int G>
TW_DEV void group_sync() {
  if (G == 32)
    __syncwarp();
  else
    named_barrier(1 + threadIdx.x / G, G);
}
// Statistics of the group's threads' parts; every thread of it gets them.
template <int G, int NT>
TW_DEV MaxSum group_stats(const MaxSum& a, const ExpK& k) {
  float m = warp_max(a.m);
  float s = warp_sum(rescaled(a, m, k));
  if (G == 32) return MaxSum{m, s};
  constexpr int kWarps = G / 32;
  __shared__ MaxSum parts[NT / 32];
  MaxSum* part = parts + threadIdx.x / G * kWarps;
  if ((threadIdx.x & 31) == 0) part[threadIdx.x % G / 32] = MaxSum{m, s};
  group_sync<G>();
  m = part[0].m;
#pragma unroll
  for (int i = 1; i < kWarps; ++i) m = fmaxf(m, part[i].m);
  s = 0.0f;
#pragma unroll
  for (int i = 0; i < kWarps; ++i) s += rescaled(part[i], m, k);
  return MaxSum{m, s};
}

// What the loss of one token takes beside its log-probability.
struct PolicyRow {
  float w, A, old_logp, ref_logp;
};
TW_DEV PolicyRow load_policy(const Policy& P, int t) {
  return PolicyRow{P.weight ? P.weight[t] : 1.0f, P.adv[t], P.old_logp ? P.old_logp[t] : 0.0f,
                   P.kl != 0.0f ? P.ref_logp[t] : 0.0f};
}
// Loss term of one token and its derivative by logp.  `over` and `under`: the
// ratio is past the clip on the side where min() takes the clipped, constant branch.
// Without an advantage r A is 0, also where r overflows (a NaN stays one).
TW_DEV void policy_terms(const Policy& P, const PolicyRow& x, float logp, float& tok, float& coef) {
  tok = coef = 0.0f;
  if (x.w == 0.0f) return;
  const float r = P.old_logp ? expf(logp - x.old_logp) : 1.0f;
  const bool over = x.A > 0.0f && r > P.hi, under = x.A < 0.0f && r < P.lo;
  const float rA = x.A == 0.0f && r == INFINITY ? 0.0f : r * x.A;
  tok = over ? -P.hi * x.A : under ? -P.lo * x.A : -rA;
  coef = over || under ? 0.0f : -rA;
  if (P.kl != 0.0f) {
    const float q = x.ref_logp - logp;
    const float e = expm1f(q);  // exp(q) - 1 - q without the cancellation of exp(q) - 1
    tok += P.kl * (e - q);
    coef -= P.kl * e;
  }
  tok *= x.w;
  coef *= x.w;
}

enum Mode { kLogp = 0, kPolicy = 1, kPref = 2 };

struct Outs {
  float *logp, *lse, *tok_loss, *coef;
  unsigned* zero;  // kPref: a count that the next kernel starts from 0
};
template <int MODE>
TW_DEV void write_ignored(const Outs& o, int t) {
  o.logp[t] = 0.0f;
  if (o.lse) o.lse[t] = 0.0f;
  if (MODE == kPolicy) o.tok_loss[t] = 0.0f;
  if (MODE != kLogp) o.coef[t] = 0.0f;
}

// Statistics of the blocks' parts of a row; every thread of the cluster gets
// them.  The caller has arrived at the cluster's barrier once: a block writes into
// another's shared memory only when all have started.
TW_DEV MaxSum cluster_stats(const MaxSum& a, int CL, const ExpK& k) {
  __shared__ MaxSum parts[kMaxCluster];
  cluster_wait();
  if ((int)threadIdx.x < CL)
    st_cluster_b64(&parts[cluster_rank()], threadIdx.x, f2_pack(a.m, a.s));
  cluster_arrive();
  cluster_wait();
  float m = parts[0].m, s = 0.0f;
  for (int i = 1; i < CL; ++i) m = fmaxf(m, parts[i].m);
  for (int i = 0; i < CL; ++i) s += rescaled(parts[i], m, k);
  return MaxSum{m, s};
}

// Statistics, log-probability and loss term of each row, and with GRAD its
// gradient.  Without GRAD it is bound by the reads (8192 x 65536 bf16 150 us,
// 105 % of the copy rate), with it by what the head of policy_ring_kernel says.
// A row is taken by G threads of a block of NT, or (G = NT) by the
// blocks of a cluster (gridDim.x = rows * cluster), a contiguous share of its
// chunks each.  With GRAD the first NV chunks of every thread stay in registers between
// the statistics and the gradient; what is beyond them is read again, from L2.
template <typename E, int MODE, bool GRAD, int G, int NV, int NT, int MINB>
__global__ void __launch_bounds__(NT, MINB)
    rows_kernel(Rows R, Policy P, Outs o, E* dx, long long dstride) {
  if (MODE != kLogp) launch_dependents();
  const int lane = threadIdx.x % G, warp0 = lane & ~31;
  const int CL = G == NT ? (int)cluster_size() : 1;
  const int rank = G == NT ? (int)cluster_rank() : 0;
  const int t = G == NT ? (int)(blockIdx.x / CL) : (int)blockIdx.x * (NT / G) + threadIdx.x / G;
  if (t >= R.rows) return;  // whole groups, and never within a cluster
  if (MODE == kPref && t == 0 && rank == 0 && lane == 0 && o.zero) *o.zero = 0;
  const Row<E> row(R.x, (long long)t * R.stride, R.vocab);
  E* d = GRAD ? dx + (long long)t * dstride : nullptr;
  const int per = (row.chunks + CL - 1) / CL;
  const int begin = rank * per, end = min(row.chunks, begin + per);
  const int y = row_target(R, t);
  if (y < 0) {
    if (rank == 0 && lane == 0) write_ignored<MODE>(o, t);
    if (GRAD)
      for (int c = begin + lane; c < end; c += G) row.store(d, c, make_uint4(0, 0, 0, 0));
    return;
  }
  if (G == NT && CL > 1) cluster_arrive();
  // NV chunks from c on, G apart; the number of those there are.  What nothing here reads
  // again is first to leave L2, also for the preference loss, whose gradient comes
  // back to it a kernel later (kept, 14 % of those reads hit L2, but the two
  // passes took 277 us instead of 269 us at 2048 x 128000).
  auto read = [&](int c, uint4 (&r)[NV], auto last) {
    constexpr bool kLast = decltype(last)::value;
    int n = 0;
    if (c - lane + warp0 + (NV - 1) * G + 32 <= end && row.plain(c - lane + warp0, G, NV)) {
#pragma unroll
      for (int i = 0; i < NV; ++i) r[i] = row.template load_whole<kLast>(c + i * G);
      return NV;
    }
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (c + i * G < end) {
        r[i] = row.template load<kLast>(c + i * G);
        n = i + 1;
      }
    return n;
  };
  uint4 r[NV];
  const int held = read(begin + lane, r, Bool<true>{});
  const float xy = load1(row.x + y);
  const PolicyRow pr = MODE == kPolicy ? load_policy(P, t) : PolicyRow{};
  MaxSum a{-INFINITY, 0.0f};
  if (held == NV)
    add_chunks<E, NV>(a, r, NV, R.k);
  else
    add_chunks<E, NV>(a, r, held, R.k);
  for (int c = begin + lane + NV * G; c < end; c += NV * G) {
    uint4 q[NV];
    const int n = read(c, q, Bool<!GRAD>{});
    if (n == NV)
      add_chunks<E, NV>(a, q, NV, R.k);
    else
      add_chunks<E, NV>(a, q, n, R.k);
  }
  a = group_stats<G, NT>(a, R.k);
  if (G == NT && CL > 1) a = cluster_stats(a, CL, R.k);

  __shared__ float coef_sh[NT / G];
  float c = 0.0f;
  if (lane == 0) {
    const float ln_s = ln_sum(a);
    const float logp = R.scale * (xy - a.m) - ln_s;
    float tok = 0.0f;
    if (MODE == kPolicy) policy_terms(P, pr, logp, tok, c);
    if (rank == 0) {
      o.logp[t] = logp;
      if (o.lse) o.lse[t] = fmaf(R.scale, a.m, ln_s);
      if (MODE == kPolicy) o.tok_loss[t] = tok;
      if (MODE != kLogp) o.coef[t] = c;
    }
    if (GRAD) coef_sh[threadIdx.x / G] = c * R.scale;
  }
  if (!GRAD) return;
  group_sync<G>();
  c = coef_sh[threadIdx.x / G];
  if (c == 0.0f) {
    for (int i = begin + lane; i < end; i += G) row.store(d, i, make_uint4(0, 0, 0, 0));
    return;
  }
  const float q = fabsf(a.m) == INFINITY ? a.m - a.m : -c / a.s;  // NaN as in ln_sum
  const Scaled S = make_scaled(R.k, a.m, q);
  const bool even = row.even(d);
  auto write = [&](int at, const uint4 (&w)[NV], int n) {
    if (n == NV && even && row.plain(at - lane + warp0, G, NV)) {
#pragma unroll
      for (int i = 0; i < NV; ++i) row.store_whole(d, at + i * G, scaled_exp<E>(w[i], S));
    } else {
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (i < n) row.store(d, at + i * G, scaled_exp<E>(w[i], S));
    }
  };
  write(begin + lane, r, held);
  for (int i0 = begin + lane + NV * G; i0 < end; i0 += NV * G) {
    uint4 w[NV];
    const int n = read(i0, w, Bool<true>{});
    write(i0, w, n);
  }
  // the target's entry, by the thread that wrote its chunk
  const int cy = (y + row.head) / Vec<E>::kN;
  if (cy >= begin && cy < end && (cy - begin) % G == lane)
    store1(d + y, fmaf(q, exp_k(xy - a.m, R.k), c));
}

// ---- long rows, many of them: a persistent kernel over a ring of row pieces
//
// What bounds it: a row moves 2 (bf16) or 4 bytes an entry in and out, and
// takes 13.7 warp instructions per 32 entries, of which the SM has 23 to spend
// at the memory's rate.  A kernel with a block to a row (rows_kernel) leaves the
// memory idle while blocks start, wait for their first loads and join their sums: 72 %
// of the copy rate at 4096 x 131072 bf16 (442 us), 17.8 instructions.  Here one producer
// warp copies the block's rows into a ring of kRing slots in shared memory
// (cp.async.bulk), ahead of NCW consumer warps and across row boundaries:
// 94 % there (337 us), 98 % at 8192 x 131072 (646 us).  A slot takes kSlotPass chunks a
// consumer thread: with two, and a check of every chunk's bounds, a kernel of
// this form took 22.7 instructions and was slower than rows_kernel.
// A row is read twice: for its statistics, then for its gradient.  Its last
// kKeep slots stay in the ring in between; what is before them is copied again,
// from L2 (152 rows of 256 KiB are 39 MB: DRAM reads measured 268.6 MB for
// 268.4 MB of logits).  1 to 4 kept slots measure the same.
// Rows go to blocks as they ask for them (ignored rows make the work uneven):
// `next` counts, from 0 at launch, the rows taken beyond the first of each block.
//
// Every wait is bounded.  One that gives up records TWELL_ERR_DEVICE_TIMEOUT
// and raises the block's abort flag, on which all its warps leave; the
// producer waits (again bounded) for its copies in flight before it does.
constexpr int kRing = 6;
constexpr int kKeep = 3;
constexpr int kSlotPass = 4;  // chunks of a slot that one consumer thread takes
constexpr int kQueue = 4;     // rows the producer may be ahead by

template <int NCW>
struct __align__(128) Ring {
  uint4 slot[kRing][NCW * 32 * kSlotPass];
  uint64_t full[kRing], empty[kRing];
  uint64_t q_full[kQueue], q_empty[kQueue];
  uint64_t stats;
  MaxSum part[2][NCW];
  int row[kQueue], target[kQueue];  // row -1 ends the list
  int abort;
};

TW_DEV void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1], %2, [%3], %4;" ::"r"(smem_u32(dst)),
      "l"(src), "r"(bytes), "r"(smem_u32(bar)), "l"(policy)
      : "memory");
}
TW_DEV uint64_t l2_normal_policy() {
  uint64_t pol;
  asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(pol));
  return pol;
}

// A place in the sequence of fills: the slot and the parity of its lap.
struct Cursor {
  uint32_t slot, lap;
  TW_DEV void step() {
    if (++slot == kRing) {
      slot = 0;
      lap ^= 1;
    }
  }
};

template <typename E, int NCW>
TW_DEV void ring_producer(Ring<NCW>& S, const Rows& R, int* next) {
  constexpr int kSlot = NCW * 32 * kSlotPass;  // chunks
  const uint64_t keep = l2_normal_policy(), last = l2_evict_first_policy();
  volatile int* stop = &S.abort;
  uint32_t fills = 0;  // slots filled so far
  bool ok = true;
  auto fill = [&](const Row<E>& row, int piece, uint64_t policy) {
    const uint32_t s = fills % kRing, lap = fills / kRing;
    if (lap > 0 && !mbar_wait(&S.empty[s], (lap - 1) & 1, stop)) return false;
    // the whole chunks among [c0, c1)
    int c0 = piece * kSlot, c1 = min(row.chunks, c0 + kSlot);
    const int at = c0;
    if (c0 < c1 && !row.whole(c0)) ++c0;
    if (c0 < c1 && !row.whole(c1 - 1)) --c1;
    const uint32_t bytes = (uint32_t)(c1 - c0) * 16u;
    mbar_arrive_expect_tx(&S.full[s], bytes);
    if (bytes) bulk_load(&S.slot[s][c0 - at], row.x + row.first(c0), bytes, &S.full[s], policy);
    ++fills;
    return true;
  };
  int t = blockIdx.x;
  int y = t < R.rows ? row_target(R, t) : -1;
  int t1 = t < R.rows ? (int)gridDim.x + atomicAdd(next, 1) : t;
  uint32_t k = 0;
  for (;; ++k) {
    const uint32_t q = k % kQueue;
    if (k >= kQueue && !(ok = mbar_wait(&S.q_empty[q], (k / kQueue - 1) & 1, stop))) break;
    const bool more = t < R.rows;
    S.row[q] = more ? t : -1;
    S.target[q] = y;
    mbar_arrive(&S.q_full[q]);
    if (!more) break;
    // the next row's target and the row after it, in flight behind this row's copies
    const long long y1 = t1 < R.rows ? raw_target(R, t1) : -1;
    const int t2 = t1 < R.rows ? (int)gridDim.x + atomicAdd(next, 1) : t1;
    if (y >= 0) {
      const Row<E> row(R.x, (long long)t * R.stride, R.vocab);
      const int n = (row.chunks + kSlot - 1) / kSlot, again = max(0, n - kKeep);
      for (int i = 0; ok && i < n; ++i) ok = fill(row, i, i < again ? keep : last);
      for (int i = 0; ok && i < again; ++i) ok = fill(row, i, last);
      if (!ok) break;
    }
    t = t1;
    y = check_target(R, y1);
    t1 = t2;
  }
  if (ok) return;
  set_status(R.status, TWELL_ERR_DEVICE_TIMEOUT);
  *stop = 1;
  // copies in flight must land before the block's shared memory is given up
  for (uint32_t f = fills > kRing ? fills - kRing : 0; f < fills; ++f)
    mbar_wait(&S.full[f % kRing], (f / kRing) & 1, nullptr);
}

template <typename E, int NCW>
__global__ void __launch_bounds__((NCW + 1) * 32)
    policy_ring_kernel(Rows R, Policy P, Outs o, E* dx, long long dstride, int* next) {
  constexpr int NT = NCW * 32, kSlot = NT * kSlotPass;
  extern __shared__ __align__(128) unsigned char smem[];
  Ring<NCW>& S = *reinterpret_cast<Ring<NCW>*>(smem);
  launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kRing; ++i) {
      mbar_init(&S.full[i], 1);
      mbar_init(&S.empty[i], NCW);
    }
    for (int i = 0; i < kQueue; ++i) {
      mbar_init(&S.q_full[i], 1);
      mbar_init(&S.q_empty[i], NCW);
    }
    mbar_init(&S.stats, NCW);
    S.abort = 0;
    fence_mbar_init();
  }
  __syncthreads();
  if (warp == NCW) {
    if (lane == 0) ring_producer<E, NCW>(S, R, next);
    return;
  }
  volatile int* stop = &S.abort;
  auto give_up = [&]() {
    set_status(R.status, TWELL_ERR_DEVICE_TIMEOUT);
    *stop = 1;
  };
  const int tid = threadIdx.x;
  // Gives a slot back.  Only when what was read from it has been used: a warp that
  // arrived with its reads still under way saw the next copy in them (at 4 blocks an
  // SM, in one row of 5000).  The fence orders the reads before that copy, which is the async proxy's.
  auto release = [&](uint32_t slot) {
    fence_proxy_async();
    __syncwarp();
    if (lane == 0) mbar_arrive(&S.empty[slot]);
  };
  Cursor head{0, 0}, kept{0, 0};  // the next slot, the row's first kept one
  uint32_t live = 0;              // rows with a target
  for (uint32_t k = 0;; ++k) {
    const uint32_t q = k % kQueue;
    if (!mbar_wait(&S.q_full[q], (k / kQueue) & 1, stop)) return give_up();
    const int t = S.row[q], y = S.target[q];
    __syncwarp();
    if (lane == 0) mbar_arrive(&S.q_empty[q]);
    if (t < 0) return;
    const Row<E> row(R.x, (long long)t * R.stride, R.vocab);
    E* d = dx + (long long)t * dstride;
    if (y < 0) {
      if (tid == 0) write_ignored<kPolicy>(o, t);
      for (int c = tid; c < row.chunks; c += NT) row.store(d, c, make_uint4(0, 0, 0, 0));
      continue;
    }
    const int n = (row.chunks + kSlot - 1) / kSlot, again = max(0, n - kKeep);
    const float xy = load1(row.x + y);
    const PolicyRow pr = load_policy(P, t);
    // whether all of this warp's chunks of a piece are whole: read from the slot as they are
    auto plain = [&](int piece) { return row.plain(piece * kSlot + warp * 32, NT, kSlotPass); };
    auto read = [&](uint32_t s, int piece, uint4 (&r)[kSlotPass]) {
      int m = 0;
#pragma unroll
      for (int j = 0; j < kSlotPass; ++j) {
        const int c = piece * kSlot + j * NT + tid;
        if (c < row.chunks) {
          r[j] = row.whole(c) ? S.slot[s][j * NT + tid] : row.template load<true>(c);
          m = j + 1;
        }
      }
      return m;
    };
    MaxSum a{-INFINITY, 0.0f};
    Cursor at = head;
    for (int i = 0; i < n; ++i, at.step()) {
      if (!mbar_wait(&S.full[at.slot], at.lap, stop)) return give_up();
      uint4 r[kSlotPass];
      const bool all = plain(i);
      int m = kSlotPass;
      if (all) {
#pragma unroll
        for (int j = 0; j < kSlotPass; ++j) r[j] = S.slot[at.slot][j * NT + tid];
      } else {
        m = read(at.slot, i, r);
      }
      if (all)
        add_chunks<E, kSlotPass>(a, r, kSlotPass, R.k);
      else
        add_chunks<E, kSlotPass>(a, r, m, R.k);
      if (i < again)
        release(at.slot);
      else if (i == again)
        kept = at;
    }
    // join over the block, without a barrier that would outlive an abort
    MaxSum* part = S.part[live & 1];
    {
      const float m = warp_max(a.m), sum = warp_sum(rescaled(a, m, R.k));
      if (lane == 0) {
        part[warp] = MaxSum{m, sum};
        mbar_arrive(&S.stats);
      }
      if (!mbar_wait(&S.stats, live & 1, stop)) return give_up();
      const MaxSum p = lane < NCW ? part[lane] : MaxSum{-INFINITY, 0.0f};
      a.m = warp_max(p.m);
      a.s = warp_sum(rescaled(p, a.m, R.k));
      ++live;
    }
    const float ln_s = ln_sum(a), logp = R.scale * (xy - a.m) - ln_s;
    float tok, coef;
    policy_terms(P, pr, logp, tok, coef);
    if (tid == 0) {
      o.logp[t] = logp;
      if (o.lse) o.lse[t] = fmaf(R.scale, a.m, ln_s);
      o.tok_loss[t] = tok;
      o.coef[t] = coef;
    }
    const float c = coef * R.scale;
    const float g = fabsf(a.m) == INFINITY ? a.m - a.m : -c / a.s;
    // the kept slots, then the ones copied again
    const Scaled sc = make_scaled(R.k, a.m, g);
    const bool even = row.even(d);
    for (int i = 0; i < n; ++i) {
      const int piece = i < n - again ? again + i : i - (n - again);
      Cursor& from = i < n - again ? kept : at;
      if (!mbar_wait(&S.full[from.slot], from.lap, stop)) return give_up();
      uint4 r[kSlotPass];
      const bool all = plain(piece) && even && c != 0.0f;
      if (all) {
#pragma unroll
        for (int j = 0; j < kSlotPass; ++j) r[j] = S.slot[from.slot][j * NT + tid];
      } else {
        read(from.slot, piece, r);
      }
      if (all) {
        uint4* out = reinterpret_cast<uint4*>(d + row.first(piece * kSlot + tid));
#pragma unroll
        for (int j = 0; j < kSlotPass; ++j) __stcs(out + j * NT, scaled_exp<E>(r[j], sc));
      } else {
#pragma unroll
        for (int j = 0; j < kSlotPass; ++j) {
          const int b = piece * kSlot + j * NT + tid;
          if (b < row.chunks)
            row.store(d, b, c == 0.0f ? make_uint4(0, 0, 0, 0) : scaled_exp<E>(r[j], sc));
        }
      }
      release(from.slot);
      from.step();
    }
    head = at;
    const int cy = (y + row.head) / Vec<E>::kN;
    if (c != 0.0f && cy % NT == tid) store1(d + y, fmaf(g, exp_k(xy - a.m, R.k), c));
  }
}

constexpr int kBwdThreads = 256;

// dlogits = c (onehot - exp(z - lse)), c = scale * coef * dloss.  G threads take
// a row, or (G = the block) one of its `slices`; the last rows first: what the
// forward read last is what L2 still holds.
template <typename E, int G, int NV>
__global__ void __launch_bounds__(kBwdThreads)
    logp_bwd_kernel(Rows R, const float* lse, const float* coef, const float* dloss, E* dx,
                    long long dstride, int slices) {
  const unsigned idx = gridDim.x - 1 - blockIdx.x;
  const int lane = threadIdx.x % G, warp0 = lane & ~31;
  const int t = G == kBwdThreads ? (int)(idx / slices)
                                 : (int)(idx * (kBwdThreads / G) + threadIdx.x / G);
  const int slice = G == kBwdThreads ? (int)(idx % slices) : 0;
  if (t >= R.rows) return;  // whole groups
  const Row<E> row(R.x, (long long)t * R.stride, R.vocab);
  E* d = dx + (long long)t * dstride;
  const int per = (row.chunks + slices - 1) / slices;
  const int begin = slice * per, end = min(row.chunks, begin + per);
  const int y = row_target(R, t);
  const float c = y < 0 ? 0.0f : R.scale * coef[t] * (dloss ? dloss[0] : 1.0f);
  if (c == 0.0f) {
    for (int i = begin + lane; i < end; i += G) row.store(d, i, make_uint4(0, 0, 0, 0));
    return;
  }
  const int cy = (y + row.head) / Vec<E>::kN;
  const bool mine = cy >= begin && cy < end && (cy - begin) % G == lane;
  const float xy = mine ? load1(row.x + y) : 0.0f;  // before this thread writes its chunk in place
  // exp(scale (x - m)) times q: m = lse / scale and q = -c, but where lse is
  // too large to hold ln s to 2^-17 the row's own statistics
  float m = lse[t] / R.scale, q = -c;
  if (fabsf(lse[t]) > kLseExact) {
    MaxSum a{-INFINITY, 0.0f};
    for (int i = lane; i < row.chunks; i += G) {
      const uint4 one[1] = {row.template load<false>(i)};
      add_chunks<E, 1>(a, one, 1, R.k);
    }
    a = group_stats<G, kBwdThreads>(a, R.k);
    m = a.m;
    q = fabsf(m) == INFINITY ? m - m : -c / a.s;
  }
  const Scaled S = make_scaled(R.k, m, q);
  const bool even = row.even(d);
  for (int i0 = begin + lane; i0 < end; i0 += NV * G) {
    uint4 r[NV];
    const int w = i0 - lane + warp0;
    if (even && w + (NV - 1) * G + 32 <= end && row.plain(w, G, NV)) {
#pragma unroll
      for (int i = 0; i < NV; ++i) r[i] = row.template load_whole<true>(i0 + i * G);
#pragma unroll
      for (int i = 0; i < NV; ++i) row.store_whole(d, i0 + i * G, scaled_exp<E>(r[i], S));
    } else {
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (i0 + i * G < end) r[i] = row.template load<true>(i0 + i * G);
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (i0 + i * G < end) row.store(d, i0 + i * G, scaled_exp<E>(r[i], S));
    }
  }
  if (mine) store1(d + y, fmaf(q, exp_k(xy - m, R.k), c));
}

// scale * sum of v[0..n) by a block of NT, in a fixed order: each thread a
// compensated fp32 sum, the threads' sums in fp64.  Thread 0 gets it.
template <int NT>
TW_DEV float block_sum(const float* v, int n, float scale) {
  float s = 0.0f, c = 0.0f;
  for (int i0 = threadIdx.x; i0 < n; i0 += 8 * NT) {
    float a[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) a[i] = i0 + i * NT < n ? __ldcg(v + i0 + i * NT) : 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float sum = s + a[i];
      c += fabsf(s) >= fabsf(a[i]) ? (s - sum) + a[i] : (a[i] - sum) + s;
      s = sum;
    }
  }
  // an infinite sum has a NaN compensation that must not replace it
  double d = isfinite(s) ? (double)s + (double)c : (double)s;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) d += __shfl_xor_sync(0xffffffffu, d, o);
  __shared__ double part[NT / 32];
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = d;
  __syncthreads();
  if (threadIdx.x >= 32) return 0.0f;
  d = threadIdx.x < NT / 32 ? part[threadIdx.x] : 0.0;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) d += __shfl_xor_sync(0xffffffffu, d, o);
  return (float)(d * scale);
}
// NT: few threads for few rows, as fp64 additions are scarce.
template <int NT>
__global__ void __launch_bounds__(NT) loss_sum_kernel(const float* v, int n, float* out) {
  wait_for_previous();
  const float sum = block_sum<NT>(v, n, 1.0f);
  if (threadIdx.x == 0) out[0] = sum;
}

TW_DEV float softplus(float x) { return (x > 0.0f ? x : 0.0f) + log1pf(expf(-fabsf(x))); }

// One block per pair: both sequences' gains (logp - ref rounded once, then
// fp64 sums over the tokens, in a fixed order), the pair's loss and every
// token's coefficient.  Few threads, as fp64 additions are scarce; four tokens
// of each sequence a thread in flight.  `loss` counts the blocks that are done,
// from 0; the last one replaces it by the pairs' mean.
constexpr int kPairThreads = 128;
__global__ void __launch_bounds__(kPairThreads)
    preference_kernel(Rows R, const long long* start, const float* ref, int pairs, float beta,
                      float smooth, const float* logp, float* pair_loss, float* seq_gain,
                      float* coef, float* loss) {
  wait_for_previous();
  const int p = blockIdx.x;
  __shared__ double part[2][kPairThreads / 32];
  __shared__ float slope_sh;
  __shared__ bool last_sh;
  int lo[2], hi[2];
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    const long long a = start[2 * p + q], b = start[2 * p + q + 1];
    if (a < 0 || b > R.rows || a > b) set_status(R.status, TWELL_ERR_INDEX);
    const long long a1 = a < 0 ? 0 : a > R.rows ? R.rows : a;
    const long long b1 = b < a1 ? a1 : b > R.rows ? R.rows : b;
    lo[q] = (int)a1;
    hi[q] = (int)b1;
  }
  double gain[2] = {0.0, 0.0};
  const int most = max(hi[0] - lo[0], hi[1] - lo[1]);
  for (int i0 = threadIdx.x; i0 < most; i0 += 4 * kPairThreads) {
    float over[2][4];  // logp - ref of eight tokens, their loads together
    long long y[2][4];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int q = k & 1, t = lo[q] + i0 + (k >> 1) * kPairThreads;
      const bool in = t < hi[q];
      y[q][k >> 1] = in ? raw_target(R, t) : -1;
      over[q][k >> 1] = in ? logp[t] : 0.0f;
      if (in && ref) over[q][k >> 1] -= ref[t];
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int q = k & 1;
      if (y[q][k >> 1] >= 0 && y[q][k >> 1] < R.vocab) gain[q] += (double)over[q][k >> 1];
    }
  }
#pragma unroll
  for (int q = 0; q < 2; ++q) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) gain[q] += __shfl_xor_sync(0xffffffffu, gain[q], o);
    if ((threadIdx.x & 31) == 0) part[q][threadIdx.x >> 5] = gain[q];
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int i = 1; i < kPairThreads / 32; ++i) {
      gain[0] += part[0][i];
      gain[1] += part[1][i];
    }
    const float d = (float)(beta * (gain[0] - gain[1]));
    seq_gain[2 * p] = (float)gain[0];
    seq_gain[2 * p + 1] = (float)gain[1];
    // without smoothing its term is 0, also at an infinite margin
    pair_loss[p] = (1.0f - smooth) * softplus(-d) + (smooth > 0.0f ? smooth * softplus(d) : 0.0f);
    // d pair_loss / d delta = -(1 - e) sigmoid(-delta) + e sigmoid(delta)
    const float s = smooth / (1.0f + expf(-d)) - (1.0f - smooth) / (1.0f + expf(d));
    slope_sh = s * (beta / (float)pairs);
    __threadfence();  // the pair's loss before the count
    last_sh = atomicAdd(reinterpret_cast<unsigned*>(loss), 1u) == (unsigned)pairs - 1;
  }
  __syncthreads();
#pragma unroll
  for (int q = 0; q < 2; ++q)
    for (int t = lo[q] + threadIdx.x; t < hi[q]; t += kPairThreads)
      coef[t] = row_target(R, t) < 0 ? 0.0f : q ? -slope_sh : slope_sh;
  if (!last_sh) return;
  __threadfence();
  const float mean = block_sum<kPairThreads>(pair_loss, pairs, 1.0f / (float)pairs);
  if (threadIdx.x == 0) loss[0] = mean;
}

// ------------------------------------------------------------------ host side
// Rows, and elements of a row: both are numbered in 32 bits, with room to spare
// for the last block's.
constexpr int kMaxCount = 1 << 30;

bool off(const void* p, uintptr_t bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) != 0; }

twell_status check_logits(const twell_logits* L) {
  if (!L || L->rows < 0 || L->vocab < 1 || L->stride < L->vocab) return TWELL_ERR_INVALID_ARG;
  if (L->dtype != TWELL_BF16 && L->dtype != TWELL_F32) return TWELL_ERR_INVALID_ARG;
  if (L->target_dtype != TWELL_I32 && L->target_dtype != TWELL_I64) return TWELL_ERR_INVALID_ARG;
  if (!(L->scale > 0.0f) || !isfinite(L->scale)) return TWELL_ERR_INVALID_ARG;
  if (L->vocab > kMaxCount || L->rows > kMaxCount) return TWELL_ERR_UNSUPPORTED;
  if (L->rows == 0) return TWELL_OK;
  if (!L->data || !L->target) return TWELL_ERR_INVALID_ARG;
  if (off(L->data, L->dtype == TWELL_F32 ? 4 : 2)) return TWELL_ERR_ALIGNMENT;
  if (off(L->target, L->target_dtype == TWELL_I64 ? 8 : 4)) return TWELL_ERR_ALIGNMENT;
  return TWELL_OK;
}

// fp32 arrays that must be there (unless `rows` is 0) and 4-byte aligned
twell_status check_f32(int rows, std::initializer_list<const void*> must,
                       std::initializer_list<const void*> may = {}) {
  if (rows == 0) return TWELL_OK;
  for (const void* p : must)
    if (!p) return TWELL_ERR_INVALID_ARG;
  for (const void* p : must)
    if (off(p, 4)) return TWELL_ERR_ALIGNMENT;
  for (const void* p : may)
    if (off(p, 4)) return TWELL_ERR_ALIGNMENT;
  return TWELL_OK;
}

twell_status check_grad(const twell_logits* L, const void* d, long long stride) {
  if (stride < L->vocab) return TWELL_ERR_INVALID_ARG;
  if (L->rows == 0) return TWELL_OK;
  if (!d) return TWELL_ERR_INVALID_ARG;
  if (d == L->data && stride != L->stride) return TWELL_ERR_INVALID_ARG;
  return off(d, L->dtype == TWELL_F32 ? 4 : 2) ? TWELL_ERR_ALIGNMENT : TWELL_OK;
}

bool make_rows(const twell_logits* L, Rows& R) {
  R = Rows{L->data, L->target, L->stride, L->rows, L->vocab, L->target_dtype == TWELL_I64,
           L->scale, make_exp_k(L->scale), device_status_ptr()};
  return R.status != nullptr;
}

twell_status launched() {
  return cudaGetLastError() == cudaSuccess ? TWELL_OK : TWELL_ERR_CUDA;
}

// Launches rows_kernel over clusters of `cl` blocks (cl = 1: plain blocks).
template <typename E, int MODE, bool GRAD, int G, int NV, int NT, int MINB>
twell_status launch_rows_as(const Rows& R, const Policy& P, const Outs& o, void* d,
                            long long dstride, unsigned blocks, int cl, cudaStream_t s) {
  auto kernel = rows_kernel<E, MODE, GRAD, G, NV, NT, MINB>;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(blocks);
  cfg.blockDim = dim3(NT);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)cl;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cl > 1 ? 1 : 0;
  const cudaError_t e =
      cudaLaunchKernelEx(&cfg, kernel, R, P, o, reinterpret_cast<E*>(d), dstride);
  count_launch();
  return e == cudaSuccess ? launched() : TWELL_ERR_CUDA;
}

// Most 16-byte chunks of a row: one more than its bytes need, unless every
// row starts on a boundary.
long long chunks_of(const Rows& R, int es) {
  const bool even = !off(R.x, 16) && R.stride * es % 16 == 0;
  return ((long long)R.vocab * es + 15) / 16 + (even ? 0 : 1);
}

template <typename E, int MODE, bool GRAD>
twell_status launch_rows(const char* name, const Rows& R, const Policy& P, const Outs& o, void* d,
                         long long dstride, cudaStream_t s) {
  if (R.rows == 0) return TWELL_OK;
  ProfScope prof(name, s);
  const long long chunks = chunks_of(R, sizeof(E));
  const long long bytes = chunks * 16, sms = num_sms();
  auto groups = [&](int per_block) { return (unsigned)((R.rows + per_block - 1) / per_block); };
  // Few rows: as many blocks to each as fill the GPU, while each has a chunk
  // for every thread; long rows up to three blocks to an SM.  (In a graph, one, two and
  // three blocks: 100 x 128000 bf16 policy 27.5, 20.0 and 15.6 us, logp 11.8, 9.8 and 8.4;
  // 100 x 32000 logp 5.0, 5.6 and 5.4, but policy 10.0, 9.2 and 8.4.)
  const long long places = (bytes > 128 * 1024 ? 3 : 1) * sms;
  int cl = 1;
  while (cl < 8 && R.rows * cl * 2 <= places && chunks > (long long)cl * 2 * 256) cl *= 2;
  // A warp to a row where rows are short, or many and not long: warps wait for
  // nobody but themselves.  (Against a block to a row, logp: 16384 x 4000 bf16
  // 26 us to 76 us, 4000 x 16000 24 us to 32 us; policy: 62 us to 106 us, 57 us to 61 us;
  // in a graph 311 x 2048 logp 2.7 to 3.2, policy 6.1 to 5.3.)
  const bool many = R.rows >= 16 * sms;
  if constexpr (GRAD) {
    if (bytes <= 4096 || (many && bytes <= 12288))
      return launch_rows_as<E, MODE, GRAD, 32, 4, 256, 5>(R, P, o, d, dstride, groups(8), 1, s);
    if (many && bytes <= 32768)
      return launch_rows_as<E, MODE, GRAD, 32, 8, 256, 2>(R, P, o, d, dstride, groups(8), 1, s);
    return launch_rows_as<E, MODE, GRAD, 256, 4, 256, 4>(R, P, o, d, dstride,
                                                         (unsigned)(R.rows * cl), cl, s);
  } else {
    if (bytes <= 4096 || (many && bytes <= 16384))
      return launch_rows_as<E, MODE, GRAD, 32, 4, 256, 5>(R, P, o, d, dstride, groups(8), 1, s);
    if (many && bytes <= 65536)
      return launch_rows_as<E, MODE, GRAD, 32, 8, 256, 4>(R, P, o, d, dstride, groups(8), 1, s);
    // Times by one (of 8 chunks), two and four warps and a block to a row, bf16.  64 KiB: 2439
    // rows 30, 32, 29 and 29 us, 9735 rows 94, 91, 90 and 93.  96 KiB: 1223 rows 32, 25, 26
    // and 24, 2047 rows of 98 KiB 39, 35, 37 and 41, 2439 rows 41, 45, 41 and 40, 4871 rows 77,
    // 74, 70 and 71.  128 KiB: 615 rows 34, 25, 18 and 19, 1223 rows 40, 31, 32 and 30, 8192
    // rows 155, 159, 150 and 151.  160 KiB: 1223 rows 49, 37, 40 and 36, 8192 rows 197, 201, 189
    // and 188.  256 KiB: 4096 rows 160, 155, 157 and 151.
    if (R.rows >= 8 * sms && bytes <= 112 * 1024)
      return launch_rows_as<E, MODE, GRAD, 64, 8, 256, 4>(R, P, o, d, dstride, groups(4), 1, s);
    if (R.rows >= 4 * sms && bytes <= 160 * 1024)
      return launch_rows_as<E, MODE, GRAD, 128, 8, 256, 4>(R, P, o, d, dstride, groups(2), 1, s);
    return launch_rows_as<E, MODE, GRAD, 256, 8, 256, 4>(R, P, o, d, dstride,
                                                         (unsigned)(R.rows * cl), cl, s);
  }
}

template <typename E, int NCW>
twell_status launch_ring_as(const Rows& R, const Policy& P, const Outs& o, void* d, long long dstride,
                            int* next, cudaStream_t s) {
  auto kernel = policy_ring_kernel<E, NCW>;
  const int smem = (int)sizeof(Ring<NCW>);
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
    return TWELL_ERR_CUDA;
  const int most = num_sms() * (16 / NCW);
  const int grid = R.rows < most ? R.rows : most;
  if (cudaMemsetAsync(next, 0, sizeof(int), s) != cudaSuccess) return TWELL_ERR_CUDA;
  ProfScope prof("policy_loss", s);
  kernel<<<grid, (NCW + 1) * 32, smem, s>>>(R, P, o, reinterpret_cast<E*>(d), dstride, next);
  count_launch();
  return launched();
}

// Gradient in the same call.  `next`: 4 bytes that are free until the kernel ends.
template <typename E>
twell_status launch_policy_grad(const Rows& R, const Policy& P, const Outs& o, void* d,
                                long long dstride, int* next, cudaStream_t s) {
  if (R.rows == 0) return TWELL_OK;
  // Long rows, one at least for every block: the ring, one block of 16 warps to an SM, up
  // to 160 KiB two of 8, up to 112 KiB four of 4 where each block gets some rows.  Times by
  // rows_kernel and by the rings of 4, 8 and 16 warps, bf16 but where it says fp32:
  // 47 KiB, 4096 rows 82, 79, 84, 119 us, 8192 rows 152, 137, 153, 225; 98 KiB, 2047 rows 87,
  // 90, 93, 109, 4096 rows 151, 148, 164, 201, 8192 rows 291, 268, 304, 388; 128 KiB, 1223 rows
  // 73, 77, 68, 68, 8192 rows 377, 360, 330, 360; 176 KiB, 2439 rows 184, 180, 153, 164; 256 KiB,
  // 1223 rows 159, 160, 123, 117, 8192 rows 877, 885, 694, 646; fp32 391 KiB, 1536 rows 286, 290,
  // 254, 204.  With one to four rows to a block it does not gain yet: 117 KiB, 310 rows 25, 27,
  // 34, 33, 620 rows 45, 52, 50, 49; 176 KiB, 160 rows 22, 29, 25, 30, 620 rows 65, 71, 64, 64.
  const long long bytes = chunks_of(R, sizeof(E)) * 16, sms = num_sms();
  if (bytes > 160 * 1024 && R.rows >= sms)
    return launch_ring_as<E, 16>(R, P, o, d, dstride, next, s);
  if (bytes > 112 * 1024 && R.rows >= 2 * sms)
    return launch_ring_as<E, 8>(R, P, o, d, dstride, next, s);
  if (bytes > 40 * 1024 && bytes <= 112 * 1024 && R.rows >= 24 * sms)
    return launch_ring_as<E, 4>(R, P, o, d, dstride, next, s);
  return launch_rows<E, kPolicy, true>("policy_loss", R, P, o, d, dstride, s);
}

template <int MODE>
twell_status launch_stats(const char* name, const twell_logits* L, const Rows& R, const Policy& P,
                          const Outs& o, cudaStream_t s) {
  return L->dtype == TWELL_F32 ? launch_rows<float, MODE, false>(name, R, P, o, nullptr, 0, s)
                               : launch_rows<uint16_t, MODE, false>(name, R, P, o, nullptr, 0, s);
}

template <typename E>
twell_status launch_bwd_as(const Rows& R, const float* lse, const float* coef, const float* dloss,
                           void* d, long long dstride, cudaStream_t s) {
  ProfScope prof("logp_bwd", s);
  const long long bytes = chunks_of(R, sizeof(E)) * 16;
  E* out = reinterpret_cast<E*>(d);
  if (bytes <= 4096 || (bytes <= 16384 && R.rows >= 16 * num_sms())) {
    logp_bwd_kernel<E, 32, 4><<<(unsigned)((R.rows + 7) / 8), kBwdThreads, 0, s>>>(
        R, lse, coef, dloss, out, dstride, 1);
  } else {
    // 16 KiB of a row to a block; in place a row stays with one block, which
    // may need the whole of it before it writes
    long long slices = (bytes + 16383) / 16384;
    if (d == R.x || slices * R.rows > 0x7FFFFFFF) slices = 1;
    logp_bwd_kernel<E, kBwdThreads, 4><<<(unsigned)(slices * R.rows), kBwdThreads, 0, s>>>(
        R, lse, coef, dloss, out, dstride, (int)slices);
  }
  count_launch();
  return launched();
}

twell_status launch_bwd(const twell_logits* L, const Rows& R, const float* lse, const float* coef,
                        const float* dloss, void* d, long long dstride, cudaStream_t s) {
  if (R.rows == 0) return TWELL_OK;
  return L->dtype == TWELL_F32 ? launch_bwd_as<float>(R, lse, coef, dloss, d, dstride, s)
                               : launch_bwd_as<uint16_t>(R, lse, coef, dloss, d, dstride, s);
}

twell_status launch_sum(const float* v, int n, float* out, cudaStream_t s) {
  ProfScope prof("loss_sum", s);
  const cudaError_t e = n <= 512 ? launch_after(loss_sum_kernel<128>, 1, 128, s, v, n, out)
                                 : launch_after(loss_sum_kernel<1024>, 1, 1024, s, v, n, out);
  count_launch();
  return e == cudaSuccess ? launched() : TWELL_ERR_CUDA;
}

}  // namespace

}  // namespace tw

using namespace tw;

extern "C" {

twell_status twell_token_logp(const twell_logits* logits, float* logp, float* lse, void* stream) {
  NvtxRange nvtx("twell_token_logp");
  twell_status st = check_logits(logits);
  if (st != TWELL_OK) return st;
  if ((st = check_f32(logits->rows, {logp}, {lse})) != TWELL_OK) return st;
  Rows R;
  if (!make_rows(logits, R)) return TWELL_ERR_CUDA;
  return launch_stats<kLogp>("token_logp", logits, R, Policy{}, Outs{logp, lse, nullptr, nullptr, nullptr},
                             reinterpret_cast<cudaStream_t>(stream));
}

twell_status twell_policy_loss(const twell_logits* logits, const twell_policy* policy, float* loss,
                               float* tok_loss, float* logp, float* lse, float* coef,
                               void* dlogits, int64_t dlogits_stride, void* stream) {
  NvtxRange nvtx("twell_policy_loss");
  twell_status st = check_logits(logits);
  if (st != TWELL_OK) return st;
  if (!policy || !loss) return TWELL_ERR_INVALID_ARG;
  if (!(policy->clip_low >= 0.0f && policy->clip_low <= 1.0f) || !(policy->clip_high >= 0.0f) ||
      !(policy->kl_coeff >= 0.0f) || !isfinite(policy->kl_coeff))
    return TWELL_ERR_INVALID_ARG;
  if (policy->kl_coeff > 0.0f && logits->rows > 0 && !policy->ref_logp) return TWELL_ERR_INVALID_ARG;
  st = check_f32(logits->rows, {policy->advantage, tok_loss, logp, lse, coef},
                 {policy->weight, policy->old_logp, policy->ref_logp});
  if (st != TWELL_OK) return st;
  if (off(loss, 4)) return TWELL_ERR_ALIGNMENT;
  if (dlogits && (st = check_grad(logits, dlogits, dlogits_stride)) != TWELL_OK) return st;
  Rows R;
  if (!make_rows(logits, R)) return TWELL_ERR_CUDA;
  const Policy P{policy->advantage, policy->weight, policy->old_logp, policy->ref_logp,
                 1.0f - policy->clip_low, 1.0f + policy->clip_high, policy->kl_coeff};
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const Outs o{logp, lse, tok_loss, coef, nullptr};
  int* next = reinterpret_cast<int*>(loss);  // written last, by the sum
  if (!dlogits)
    st = launch_stats<kPolicy>("policy_loss", logits, R, P, o, s);
  else if (logits->dtype == TWELL_F32)
    st = launch_policy_grad<float>(R, P, o, dlogits, dlogits_stride, next, s);
  else
    st = launch_policy_grad<uint16_t>(R, P, o, dlogits, dlogits_stride, next, s);
  if (st != TWELL_OK) return st;
  return launch_sum(tok_loss, R.rows, loss, s);
}

twell_status twell_preference_loss(const twell_logits* logits, const twell_preference* preference,
                                   float* loss, float* pair_loss, float* seq_gain, float* logp,
                                   float* lse, float* coef, void* stream) {
  NvtxRange nvtx("twell_preference_loss");
  twell_status st = check_logits(logits);
  if (st != TWELL_OK) return st;
  const twell_preference* p = preference;
  if (!p || !loss || p->pairs < 0) return TWELL_ERR_INVALID_ARG;
  if (!(p->beta >= 0.0f) || !isfinite(p->beta) ||
      !(p->label_smoothing >= 0.0f && p->label_smoothing <= 0.5f))
    return TWELL_ERR_INVALID_ARG;
  if (p->pairs > kMaxCount / 2) return TWELL_ERR_UNSUPPORTED;
  if (p->pairs > 0 && !p->seq_start) return TWELL_ERR_INVALID_ARG;
  if ((st = check_f32(p->pairs, {pair_loss, seq_gain})) != TWELL_OK) return st;
  if ((st = check_f32(logits->rows, {logp, lse, coef}, {p->ref_logp})) != TWELL_OK) return st;
  if (off(loss, 4) || off(p->seq_start, 8)) return TWELL_ERR_ALIGNMENT;
  Rows R;
  if (!make_rows(logits, R)) return TWELL_ERR_CUDA;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  // without rows or pairs the loss starts from 0 by itself, and stays 0 without pairs
  if ((R.rows == 0 || p->pairs == 0) && cudaMemsetAsync(loss, 0, sizeof(float), s) != cudaSuccess)
    return TWELL_ERR_CUDA;
  unsigned* count = p->pairs > 0 ? reinterpret_cast<unsigned*>(loss) : nullptr;
  st = launch_stats<kPref>("token_logp", logits, R, Policy{}, Outs{logp, lse, nullptr, coef, count}, s);
  if (st != TWELL_OK || p->pairs == 0) return st;
  ProfScope prof("preference_loss", s);
  const cudaError_t e = launch_after(
      preference_kernel, (unsigned)p->pairs, (unsigned)kPairThreads, s, R,
      reinterpret_cast<const long long*>(p->seq_start), p->ref_logp, (int)p->pairs, p->beta,
      p->label_smoothing, (const float*)logp, pair_loss, seq_gain, coef, loss);
  count_launch();
  return e == cudaSuccess ? launched() : TWELL_ERR_CUDA;
}

twell_status twell_logp_bwd(const twell_logits* logits, const float* lse, const float* coef,
                            const float* dloss, void* dlogits, int64_t dlogits_stride,
                            void* stream) {
  NvtxRange nvtx("twell_logp_bwd");
  twell_status st = check_logits(logits);
  if (st != TWELL_OK) return st;
  if ((st = check_f32(logits->rows, {lse, coef}, {dloss})) != TWELL_OK) return st;
  if ((st = check_grad(logits, dlogits, dlogits_stride)) != TWELL_OK) return st;
  Rows R;
  if (!make_rows(logits, R)) return TWELL_ERR_CUDA;
  return launch_bwd(logits, R, lse, coef, dloss, dlogits, dlogits_stride,
                    reinterpret_cast<cudaStream_t>(stream));
}

}  // extern "C"
