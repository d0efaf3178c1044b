// Scored routing: the k experts of each token from its E logits by softmax or sigmoid scores, with a
// bias that only chooses, groups of experts, and renormalised, scaled weights.
//
//   s = softmax(l) or sigmoid(l);  c = s + b;  v_g = the sum of the group_top largest c of group g;
//   the topk_group groups of the largest v;  the k largest c in them;  w = scale s (/ sum s).
//
// One warp a token. The lanes are dealt to the groups, P = 32 / (n_group rounded up to a power of two)
// lanes each, so a group's value is a scan of a lane's own experts and log2 P exchanges, and a group
// that is not kept just stops offering experts. Each of the k rounds takes the warp's largest key;
// without a bias the key is the logit itself, whose order is that of its score.
//
// Choices next to a border. With a bias (and for sums of two scores) fp32 values may be ordered
// otherwise than the formulas' values. Each fp32 c lies within delta + 2^-23 |c| of its formula:
// sigmoid as e / (1 + e) or 1 / (1 + e), e = expf(-|l|) to 2 ulp: relative 2^-22 + 2 * 2^-24, s <= 1, so
// delta = 2^-21; softmax: the rounding of l - max (2^-24 |l - max|, and x exp(-x) < 0.37), expf, and a
// sum of at most 69 roundings: below 2^-17 of the largest score, 1 / Z. Neighbours in the order whose
// difference is not above the sum of their bounds are computed in 64 bits and ordered again: about one
// token in a thousand at 256 experts with normal logits. Equal logits with equal biases
// (logits that were rounded to few bits) are exact ties and need no 64 bits.
#include "internal.h"
#include "router_gate.h"
#include "topk.cuh"

namespace moe {
namespace {

constexpr unsigned kAll = 0xFFFFFFFFu;

// Keys: 0 no expert, 1 a NaN, else logit_key's order.
__device__ __forceinline__ uint32_t rank_key(float v) { return v != v ? 1u : logit_key(v); }
__device__ __forceinline__ float rank_value(uint32_t key) {
  return key == 1u ? __uint_as_float(0x7FC00000u) : key_logit(key);
}
__device__ __forceinline__ uint64_t rank_key64(double v) {
  if (v != v) return 1ull;
  if (v == 0.0) v = 0.0;  // -0 as +0
  const uint64_t u = (uint64_t)__double_as_longlong(v);
  return (u >> 63) ? ~u : (u | 0x8000000000000000ull);
}
__device__ __forceinline__ double rank_value64(uint64_t key) {
  if (key == 1ull) return __longlong_as_double(0x7FF8000000000000ll);
  return __longlong_as_double((long long)((key >> 63) ? (key & 0x7FFFFFFFFFFFFFFFull) : ~key));
}

__device__ __forceinline__ float sigmoid32(float l) {
  const float e = expf(-fabsf(l));
  return (l < 0.f ? e : 1.f) / (1.f + e);
}
__device__ __forceinline__ double sigmoid64(double l) {
  const double e = exp(-fabs(l));
  return (l < 0.0 ? e : 1.0) / (1.0 + e);
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
  return v;
}
__device__ __forceinline__ double warp_sum64(double v) {
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
  return v;
}

// A lane's experts of its group: element m is expert first + at(m), if at(m) < per.
template <bool VEC>
struct Lane {
  int g, p, P, per, first;
  bool in;  // the lane has a group
  __device__ __forceinline__ int at(int m) const {
    return VEC ? 4 * (p + P * (m >> 2)) + (m & 3) : p + P * m;
  }
};

// What the 64-bit paths need of a token.
template <int MAXM, bool VEC>
struct Token {
  const float* l;
  const float* b;
  Lane<VEC> la;
  bool sigmoid;
  float lmax;

  __device__ __forceinline__ double score(int e, double Z) const {
    const double v = (double)l[e];
    return sigmoid ? sigmoid64(v) : exp(v - (double)lmax) / Z;
  }
  __device__ __forceinline__ double choice(int e, double Z) const {
    return score(e, Z) + (b ? (double)b[e] : 0.0);
  }
  __device__ double Z64() const {
    if (sigmoid) return 1.0;
    double z = 0.0;
    for (int m = 0; m < MAXM; ++m)
      if (la.in && la.at(m) < la.per) z += exp((double)l[la.first + la.at(m)] - (double)lmax);
    return warp_sum64(z);
  }
};

// Is the lane's group among the `keep` of the largest values? Lanes of a group hold its value's key.
template <typename K>
__device__ __forceinline__ bool group_kept(K key, int g, bool in, int G, int P, int keep) {
  int before = 0;
  for (int h = 0; h < G; ++h) {
    const K o = __shfl_sync(kAll, key, h * P);
    before += (o > key || (o == key && h < g)) ? 1 : 0;
  }
  return in && before < keep;
}

// The largest two keys of the P lanes of a group.
template <typename K>
__device__ __forceinline__ void group_top2(K& t1, K& t2, int P) {
  for (int o = P >> 1; o >= 1; o >>= 1) {
    const K u1 = __shfl_xor_sync(kAll, t1, o), u2 = __shfl_xor_sync(kAll, t2, o);
    const K lo = t1 < u1 ? t1 : u1, hi2 = t2 > u2 ? t2 : u2;
    t1 = t1 > u1 ? t1 : u1;
    t2 = lo > hi2 ? lo : hi2;
  }
}

template <int MAXM, bool VEC>
__device__ __noinline__ bool kept_in_64(const Token<MAXM, VEC>& t, int G, int keep, int group_top) {
  const double Z = t.Z64();
  uint64_t t1 = 0, t2 = 0;
  for (int m = 0; m < MAXM; ++m)
    if (t.la.in && t.la.at(m) < t.la.per) {
      const uint64_t key = rank_key64(t.choice(t.la.first + t.la.at(m), Z));
      if (key > t1) { t2 = t1; t1 = key; }
      else if (key > t2) t2 = key;
    }
  __syncwarp();
  group_top2(t1, t2, t.la.P);
  uint64_t v = t1;
  if (group_top == 2 && t.la.in) v = rank_key64(rank_value64(t1) + rank_value64(t2));
  return group_kept(v, t.la.g, t.la.in, G, t.la.P, keep);
}

// The order of the n candidates that lanes 0 .. n-1 hold, in 64 bits: lane r gets the one of rank r.
template <int MAXM, bool VEC>
__device__ __noinline__ int ordered_in_64(const Token<MAXM, VEC>& t, int e, int n) {
  const int lane = threadIdx.x & 31;
  const double Z = t.Z64();
  const uint64_t key = lane < n ? rank_key64(t.choice(e, Z)) : 0ull;
  int rank = 0;
  for (int i = 0; i < n; ++i) {
    const uint64_t ki = __shfl_sync(kAll, key, i);
    const int ei = __shfl_sync(kAll, e, i);
    rank += (ki > key || (ki == key && ei < e)) ? 1 : 0;
  }
  int mine = e;
  for (int i = 0; i < n; ++i) {
    const int ri = __shfl_sync(kAll, rank, i), ei = __shfl_sync(kAll, e, i);
    if (ri == lane) mine = ei;
  }
  return mine;
}

// All k rounds in 64 bits: for tokens with more than 32 candidates that fp32 does not tell apart.
template <int MAXM, bool VEC>
__device__ __noinline__ int chosen_in_64(const Token<MAXM, VEC>& t, bool kept, int k) {
  const int lane = threadIdx.x & 31;
  const double Z = t.Z64();
  uint64_t taken = 0;
  int mine = 0;
  for (int j = 0; j < k; ++j) {
    uint64_t bk = 0;
    int be = 0x7FFFFFFF, bm = 0;
    for (int m = 0; m < MAXM; ++m)
      if (kept && t.la.at(m) < t.la.per && !((taken >> m) & 1)) {
        const int e = t.la.first + t.la.at(m);
        const uint64_t key = rank_key64(t.choice(e, Z));
        if (key > bk || (key == bk && e < be)) { bk = key; be = e; bm = m; }
      }
    __syncwarp();
    uint64_t wk = bk;
    int we = be;
    for (int o = 16; o >= 1; o >>= 1) {
      const uint64_t ok = __shfl_xor_sync(kAll, wk, o);
      const int oe = __shfl_xor_sync(kAll, we, o);
      if (ok > wk || (ok == wk && oe < we)) { wk = ok; we = oe; }
    }
    if (lane == j) mine = we;
    if (be == we && bk) taken |= 1ull << bm;
  }
  return mine;
}

// A lane's experts still to be taken. Up to 8: sorted once as key << 32 | ~expert by a 19-comparator
// network. More: the keys as they are, the best found again after each win.
template <int MAXM, bool VEC>
struct Offers {
  uint64_t v[8];
  __device__ __forceinline__ void make(const uint32_t (&key)[MAXM], const Lane<VEC>& la) {
#pragma unroll
    for (int m = 0; m < 8; ++m)
      v[m] = m < MAXM && key[m < MAXM ? m : 0]
                 ? ((uint64_t)key[m < MAXM ? m : 0] << 32) | (uint32_t)~(la.first + la.at(m))
                 : 0ull;
    auto cx = [&](int a, int b) {
      const uint64_t hi = v[a] > v[b] ? v[a] : v[b];
      const uint64_t lo = v[a] > v[b] ? v[b] : v[a];
      v[a] = hi;
      v[b] = lo;
    };
    cx(0, 2); cx(1, 3); cx(4, 6); cx(5, 7);
    cx(0, 4); cx(1, 5); cx(2, 6); cx(3, 7);
    cx(0, 1); cx(2, 3); cx(4, 5); cx(6, 7);
    cx(2, 4); cx(3, 5);
    cx(1, 4); cx(3, 6);
    cx(1, 2); cx(3, 4); cx(5, 6);
  }
  __device__ __forceinline__ uint32_t best_key() const { return (uint32_t)(v[0] >> 32); }
  __device__ __forceinline__ int best() const { return (int)~(uint32_t)v[0]; }
  __device__ __forceinline__ void pop(bool mine, const Lane<VEC>&) {
#pragma unroll
    for (int m = 0; m < 7; ++m) v[m] = mine ? v[m + 1] : v[m];
    v[7] = mine ? 0ull : v[7];
  }
};

template <int MAXM, bool VEC>
struct OffersScan {
  uint32_t key[MAXM];
  uint32_t bk;
  int bm, be;
  __device__ __forceinline__ void find(const Lane<VEC>& la) {
    bk = 0;
    bm = 0;
#pragma unroll
    for (int m = 0; m < MAXM; ++m)
      if (key[m] > bk) { bk = key[m]; bm = m; }  // of equals the first: a lane's experts ascend
    be = la.first + la.at(bm);
  }
  __device__ __forceinline__ void make(const uint32_t (&k)[MAXM], const Lane<VEC>& la) {
#pragma unroll
    for (int m = 0; m < MAXM; ++m) key[m] = k[m];
    find(la);
  }
  __device__ __forceinline__ uint32_t best_key() const { return bk; }
  __device__ __forceinline__ int best() const { return be; }
  __device__ __forceinline__ void pop(bool mine, const Lane<VEC>& la) {
    if (mine) {
#pragma unroll
      for (int m = 0; m < MAXM; ++m) key[m] = m == bm ? 0u : key[m];
      find(la);
    }
    __syncwarp();
  }
};

template <bool SMALL, int MAXM, bool VEC>
struct Pick { using type = OffersScan<MAXM, VEC>; };
template <int MAXM, bool VEC>
struct Pick<true, MAXM, VEC> { using type = Offers<MAXM, VEC>; };

// The warp's largest key and its expert (the lowest of equal keys), taken from its lane.
template <typename O, bool VEC>
__device__ __forceinline__ void take(O& o, const Lane<VEC>& la, uint32_t& key, int& e) {
  const uint32_t hk = o.best_key();
  key = __reduce_max_sync(kAll, hk);
  const bool top = hk == key && key != 0u;
  const unsigned who = __ballot_sync(kAll, top);
  if (__popc(who) == 1)
    e = __shfl_sync(kAll, o.best(), __ffs(who) - 1);
  else
    e = (int)__reduce_min_sync(kAll, top ? (uint32_t)o.best() : 0x7FFFFFFFu);
  o.pop(top && o.best() == e, la);
}

__device__ __forceinline__ float finite_abs(float v) {
  const float a = fabsf(v);
  return a < INFINITY ? a : 0.f;  // infinities are exact, and NaNs never far enough apart
}

template <int MAXM, bool VEC>
__global__ void __launch_bounds__(256) k_route_select(const GateParams q) {
  pdl_wait_then_release();
  const int lane = threadIdx.x & 31;
  const long tok = (long)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
  if (tok >= q.T) return;
  const float* lt = q.logits + tok * q.E;
  Lane<VEC> la;
  la.P = q.P;
  la.g = lane / q.P;
  la.p = lane - la.g * q.P;
  la.per = q.per;
  la.in = la.g < q.G;
  la.first = la.g * q.per;

  float l[MAXM];
#pragma unroll
  for (int m = 0; m < MAXM; m += VEC ? 4 : 1) {
    const bool there = la.in && la.at(m) < q.per;
    if (VEC) {
      float4 f = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
      if (there) f = *reinterpret_cast<const float4*>(lt + la.first + la.at(m));
      l[m] = f.x;
      l[m + 1] = f.y;
      l[m + 2] = f.z;
      l[m + 3] = f.w;
    } else {
      l[m] = there ? lt[la.first + la.at(m)] : -INFINITY;
    }
  }
  const bool sums = q.keep < q.G && q.group_top == 2;  // group values are sums of scores
  const bool need_c = q.bias || sums;
  float lmax = 0.f, Z = 1.f, delta = 4.76837158e-7f;  // 2^-21
  if (!q.sigmoid && (need_c || !q.renorm)) {
    float mx = -INFINITY;
#pragma unroll
    for (int m = 0; m < MAXM; ++m) mx = fmaxf(mx, l[m]);
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(kAll, mx, o));
    lmax = mx;
    float z = 0.f;
#pragma unroll
    for (int m = 0; m < MAXM; ++m)
      if (la.in && la.at(m) < q.per) z += expf(l[m] - lmax);
    Z = warp_sum(z);
    delta = 7.62939453e-6f / Z;  // 2^-17 of the largest score
  }

  // keys: of c with a bias, else of the logit; t1, t2: the lane's largest two c
  uint32_t key[MAXM], t1 = 0, t2 = 0;
#pragma unroll
  for (int m = 0; m < MAXM; ++m) {
    const bool there = la.in && la.at(m) < q.per;
    key[m] = there ? rank_key(l[m]) : 0u;
    uint32_t ck = key[m];
    if (need_c) {
      float c = q.sigmoid ? sigmoid32(l[m]) : expf(l[m] - lmax) / Z;
      if (q.bias) c += there ? __ldg(q.bias + la.first + la.at(m)) : 0.f;
      ck = there ? rank_key(c) : 0u;
      if (q.bias) key[m] = ck;
    }
    t2 = max(t2, min(t1, ck));
    t1 = max(t1, ck);
  }

  Token<MAXM, VEC> t{lt, q.bias, la, q.sigmoid != 0, lmax};
  bool kept = la.in;
  if (q.keep < q.G) {
    group_top2(t1, t2, q.P);
    uint32_t gv = t1;
    float err = 0.f;
    if (q.group_top == 2 && la.in) {
      const float a = rank_value(t1), b = rank_value(t2), v = a + b;
      gv = rank_key(v);
      err = 2.f * delta + 1.1920929e-7f * (finite_abs(a) + finite_abs(b) + finite_abs(v));
    } else if (la.in) {
      err = delta + 1.1920929e-7f * finite_abs(rank_value(t1));
    }
    if (!la.in) gv = 0u;
    kept = group_kept(gv, la.g, la.in, q.G, q.P, q.keep);
    if (need_c) {
      const float lo = rank_value(__reduce_min_sync(kAll, kept ? gv : kAll));
      const float hi = rank_value(__reduce_max_sync(kAll, !kept ? gv : 0u));
      const float e2 = 2.f * __uint_as_float(__reduce_max_sync(kAll, __float_as_uint(err)));
      if (!(lo - hi > e2)) kept = kept_in_64(t, q.G, q.keep, q.group_top);
    }
  }
  if (!kept) {
#pragma unroll
    for (int m = 0; m < MAXM; ++m) key[m] = 0u;
  }

  typename Pick<MAXM <= 8, MAXM, VEC>::type offers;
  offers.make(key, la);
  uint32_t my_key = 0, nk = 0;
  int my_e = 0, ne = 0;
  for (int j = 0; j < q.k; ++j) {
    uint32_t wk;
    int we;
    take(offers, la, wk, we);
    if (lane == j) {
      my_key = wk;
      my_e = we;
    }
  }
  if (q.bias) {
    // neighbours in the order, the first that was not chosen among them
    take(offers, la, nk, ne);
    const bool more = nk != 0u;
    uint32_t next_key = __shfl_down_sync(kAll, my_key, 1);
    int next_e = __shfl_down_sync(kAll, my_e, 1);
    if (lane == q.k - 1) {
      next_key = nk;
      next_e = ne;
    }
    const float a = rank_value(my_key), b = rank_value(next_key);
    const float apart = 2.f * delta + 1.1920929e-7f * (finite_abs(a) + finite_abs(b));
    const bool has_next = lane < q.k - 1 || (lane == q.k - 1 && more);
    bool near = has_next && !(a - b > apart) && !(a == b && fabsf(a) == INFINITY);
    if (near) near = !(lt[my_e] == lt[next_e] && q.bias[my_e] == q.bias[next_e]);
    if (__any_sync(kAll, near)) {
      // every expert that may belong among the k: those within the bounds of the k-th's c
      const float ck = __shfl_sync(kAll, a, q.k - 1);
      int n = q.k;
      bool whole = false;
      while (nk != 0u) {
        const float v = rank_value(nk);
        if (ck - v > 2.f * delta + 1.1920929e-7f * (finite_abs(ck) + finite_abs(v))) break;
        if (n == 32) {
          whole = true;
          break;
        }
        if (lane == n) my_e = ne;
        ++n;
        take(offers, la, nk, ne);
      }
      my_e = whole ? chosen_in_64(t, kept, q.k) : ordered_in_64(t, my_e, n);
    }
  }

  // weights, lane j choice j's
  const bool mine = lane < q.k;
  const float le = mine ? lt[my_e] : -INFINITY;
  float mx = -INFINITY, s;
  if (q.renorm) {
    mx = le;
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(kAll, mx, o));
  }
  // divided by their sum, scores that are exp(l) to fp32 (softmax's other terms cancel; sigmoids of
  // logits below -60) are taken relative to the largest, so that none vanishes against 1
  if (q.renorm && (!q.sigmoid || (mx < -60.f && mx > -INFINITY))) {
    s = mine ? expf(le - mx) : 0.f;
  } else if (q.sigmoid) {
    s = mine ? sigmoid32(le) : 0.f;
  } else {
    s = mine ? expf(le - lmax) / Z : 0.f;
  }
  if (q.renorm) {
    const float sum = warp_sum(s);
    s = sum == 0.f ? 0.f : s / sum;
  }
  if (mine) {
    q.idx[tok * q.k + lane] = my_e;
    q.w[tok * q.k + lane] = s * q.scale;
  }
}

template <int MAXM, bool VEC>
cudaError_t launch_one(const GateParams& q, cudaStream_t st) {
  const int warps = 8;
  return launch_pdl(k_route_select<MAXM, VEC>, dim3((unsigned)((q.T + warps - 1) / warps)),
                    dim3(32 * warps), 0, st, q);
}

}  // namespace

cudaError_t launch_route_select(const moe_shape& s, const moe_gate& gate, const float* logits,
                                const float* bias, int32_t* idx, float* w, cudaStream_t st) {
  if (s.T == 0) return cudaSuccess;
  GateParams q{};
  q.logits = logits;
  q.bias = bias;
  q.idx = idx;
  q.w = w;
  q.T = s.T;
  q.E = s.E;
  q.k = s.k;
  q.keep = gate.topk_group;
  q.group_top = gate.group_top;
  // kept whole, groups do not choose: all experts as one group
  q.G = gate.topk_group < gate.n_group ? gate.n_group : 1;
  if (q.G == 1) q.keep = 1;
  q.per = s.E / q.G;
  q.sigmoid = gate.score == MOE_SCORE_SIGMOID;
  q.renorm = gate.renorm != 0;
  q.scale = gate.scale;
  int lanes = 1;
  while (lanes < q.G) lanes *= 2;
  q.P = 32 / lanes;
  // groups of whole quads of experts are read 16 bytes at a time
  const bool vec = q.per % 4 == 0;
  const int v = vec ? 4 : 1;
  const int m = (q.per + q.P * v - 1) / (q.P * v) * v;
  count_launches(1);
  if (vec) {
    if (m <= 4) return launch_one<4, true>(q, st);
    if (m <= 8) return launch_one<8, true>(q, st);
    if (m <= 16) return launch_one<16, true>(q, st);
    if (m <= 32) return launch_one<32, true>(q, st);
    return launch_one<64, true>(q, st);
  }
  if (m <= 4) return launch_one<4, false>(q, st);
  if (m <= 8) return launch_one<8, false>(q, st);
  if (m <= 16) return launch_one<16, false>(q, st);
  if (m <= 32) return launch_one<32, false>(q, st);
  return launch_one<64, false>(q, st);
}

}  // namespace moe
