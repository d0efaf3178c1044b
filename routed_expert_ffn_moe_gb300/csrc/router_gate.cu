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
// What bounds it: instructions and their latency. One token takes 4.1 us, most of it one warp's chain; 16384 tokens
// of 256 experts in 8 groups 19.4 us (2.6 us of reads), 16.8 MB in 4096 warps of 1900 instructions, and 5 us of
// them the tokens that are done again.
//
// Choices next to a border. With a bias (and for sums of two scores) fp32 values may be ordered
// otherwise than the formulas' values. Each fp32 c lies within delta + 2^-23 |c| of its formula: delta = 2^-20
// for a sigmoid (order_score and its 1 + e); for softmax the rounding of l - max (2^-24 |l - max|), the
// exponential, and a sum of at most 69 roundings: below 2^-17 of the largest score, 1 / Z. Neighbours in the order
// whose difference is not above the sum of their bounds are computed in 64 bits and ordered again: about two
// tokens in a thousand at 256 experts with normal logits. Equal logits with equal biases (logits that were
// rounded to few bits) are exact ties and need no 64 bits; where the k-th and the first left tie, all experts that
// do not tie with them are compared with the k-th.
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

__device__ __forceinline__ float rcp_approx(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// Scores for the order alone, without branches: __expf is off by 2 + 1.173 |x| ulp (and x exp(-x) < 0.37), the
// reciprocal by one: a sigmoid by less than 2^-21.
__device__ __forceinline__ float order_score(bool sigmoid, float l, float lmax, float rZ) {
  return sigmoid ? rcp_approx(1.f + __expf(-l)) : __expf(l - lmax) * rZ;
}

// Scores for the weights.
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
  // Has the lane an expert within the bounds of ck, the c of expert e, that does not tie with e exactly?
  __device__ bool others_near(bool kept, int e, float ck, float delta, float rZ) const {
    const float le = l[e], be = b[e];
    bool found = false;
    for (int m0 = 0; m0 < MAXM; m0 += 4) {  // four experts' loads at a time
      float lo[4], bo[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int at = la.at(m0 + i);
        const bool there = kept && at < la.per;
        lo[i] = there ? l[la.first + at] : le;
        bo[i] = there ? b[la.first + at] : be;
      }
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (lo[i] != le || bo[i] != be) {
          const float c = order_score(sigmoid, lo[i], lmax, rZ) + bo[i];
          found |= fabsf(ck - c) <= 2.f * delta + 1.1920929e-7f * (fabsf(ck) + fabsf(c));
        }
    }
    return found;
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

// The groups kept, in 64 bits. `least`: what an expert's c in 32 bits has to reach to be one of those that
// make its group's value; only these are computed again (a lane has one or two of them, as a rule).
template <int MAXM, bool VEC>
__device__ __forceinline__ bool kept_in_64(const Token<MAXM, VEC>& t, int G, int keep, int group_top,
                                        float least, float Z32) {
  const double Z = t.Z64();
  uint64_t todo = 0;
#pragma unroll
  for (int m = 0; m < MAXM; ++m)
    if (t.la.in && t.la.at(m) < t.la.per) {
      const int e = t.la.first + t.la.at(m);
      const float c = (t.sigmoid ? sigmoid32(t.l[e]) : expf(t.l[e] - t.lmax) / Z32) + (t.b ? t.b[e] : 0.f);
      if (!(c < least)) todo |= 1ull << m;
    }
  uint64_t t1 = 0, t2 = 0;
  while (__any_sync(kAll, todo != 0)) {
    if (todo) {
      const int m = __ffsll((long long)todo) - 1;
      todo &= todo - 1;
      const uint64_t key = rank_key64(t.choice(t.la.first + t.la.at(m), Z));
      if (key > t1) { t2 = t1; t1 = key; }
      else if (key > t2) t2 = key;
    }
    __syncwarp();
  }
  group_top2(t1, t2, t.la.P);
  uint64_t v = t1;
  if (group_top == 2 && t.la.in) v = rank_key64(rank_value64(t1) + rank_value64(t2));
  return group_kept(v, t.la.g, t.la.in, G, t.la.P, keep);
}

// The order of the n candidates that lanes 0 .. n-1 hold, in 64 bits: lane r gets the one of rank r.
template <int MAXM, bool VEC>
__device__ __forceinline__ int ordered_in_64(const Token<MAXM, VEC>& t, int e, int n) {
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
__device__ __forceinline__ int chosen_in_64(const Token<MAXM, VEC>& t, bool kept, int k) {
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
// network. More than 16: the keys as they are, the best found again after each win.
template <int MAXM, bool VEC>
struct Offers {
  uint64_t v[8];
  __device__ __forceinline__ void make(const uint32_t (&key)[MAXM], const Lane<VEC>& la, int m0 = 0) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int m = m0 + i < MAXM ? m0 + i : 0;
      v[i] = m0 + i < MAXM && key[m] ? ((uint64_t)key[m] << 32) | (uint32_t)~(la.first + la.at(m)) : 0ull;
    }
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
  static constexpr int kBlocks = MAXM / 8;  // each with its own best: a win looks through one of them again
  uint32_t key[MAXM];
  uint32_t block_key[kBlocks];
  int block_at[kBlocks];
  uint32_t bk;
  int bm, be;
  __device__ __forceinline__ void look(int b) {
    block_key[b] = 0;
    block_at[b] = 8 * b;
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (key[8 * b + i] > block_key[b]) {  // of equals the first: a lane's experts ascend
        block_key[b] = key[8 * b + i];
        block_at[b] = 8 * b + i;
      }
  }
  __device__ __forceinline__ void find(const Lane<VEC>& la) {
    bk = block_key[0];
    bm = block_at[0];
#pragma unroll
    for (int b = 1; b < kBlocks; ++b)
      if (block_key[b] > bk) { bk = block_key[b]; bm = block_at[b]; }
    be = la.first + la.at(bm);
  }
  __device__ __forceinline__ void make(const uint32_t (&k)[MAXM], const Lane<VEC>& la) {
#pragma unroll
    for (int m = 0; m < MAXM; ++m) key[m] = k[m];
#pragma unroll
    for (int b = 0; b < kBlocks; ++b) look(b);
    find(la);
  }
  __device__ __forceinline__ uint32_t best_key() const { return bk; }
  __device__ __forceinline__ int best() const { return be; }
  __device__ __forceinline__ void pop(bool mine, const Lane<VEC>& la) {
    if (mine) {
#pragma unroll
      for (int b = 0; b < kBlocks; ++b)
        if (bm >> 3 == b) {
#pragma unroll
          for (int i = 0; i < 8; ++i) key[8 * b + i] = 8 * b + i == bm ? 0u : key[8 * b + i];
          look(b);
        }
      find(la);
    }
    __syncwarp();
  }
};

// Up to 16: two sorted lists, the larger head of which is offered.
template <int MAXM, bool VEC>
struct OffersTwo {
  Offers<MAXM, VEC> a, b;
  __device__ __forceinline__ void make(const uint32_t (&key)[MAXM], const Lane<VEC>& la) {
    a.make(key, la, 0);
    b.make(key, la, 8);
  }
  __device__ __forceinline__ bool first() const { return a.v[0] >= b.v[0]; }
  __device__ __forceinline__ uint32_t best_key() const { return first() ? a.best_key() : b.best_key(); }
  __device__ __forceinline__ int best() const { return first() ? a.best() : b.best(); }
  __device__ __forceinline__ void pop(bool mine, const Lane<VEC>& la) {
    const bool f = first();
    a.pop(mine && f, la);
    b.pop(mine && !f, la);
  }
};

template <int LISTS, int MAXM, bool VEC>
struct Pick { using type = OffersScan<MAXM, VEC>; };
template <int MAXM, bool VEC>
struct Pick<1, MAXM, VEC> { using type = Offers<MAXM, VEC>; };
template <int MAXM, bool VEC>
struct Pick<2, MAXM, VEC> { using type = OffersTwo<MAXM, VEC>; };

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

// A lane's place among the `lanes` lanes of a token.
template <bool VEC>
__device__ __forceinline__ Lane<VEC> lane_of(const GateParams& q, int lane, int P) {
  Lane<VEC> la;
  la.P = P;
  la.g = lane / P;
  la.p = lane - la.g * P;
  la.per = q.per;
  la.in = la.g < q.G;
  la.first = la.g * q.per;
  return la;
}

// One token by a warp.
template <int MAXM, bool VEC>
__device__ __forceinline__ void select_token(const GateParams& q, long tok) {
  const int lane = threadIdx.x & 31;
  const float* lt = q.logits + tok * q.E;
  const Lane<VEC> la = lane_of<VEC>(q, lane, q.P);

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
  float bias[MAXM];  // loaded with the logits: one by one where they are used, each would wait for its own
#pragma unroll
  for (int m = 0; m < MAXM; m += VEC ? 4 : 1) {
    const bool there = q.bias && la.in && la.at(m) < q.per;
    if (VEC) {
      float4 f = make_float4(0.f, 0.f, 0.f, 0.f);
      if (there) f = __ldg(reinterpret_cast<const float4*>(q.bias + la.first + la.at(m)));
      bias[m] = f.x;
      bias[m + 1] = f.y;
      bias[m + 2] = f.z;
      bias[m + 3] = f.w;
    } else {
      bias[m] = there ? __ldg(q.bias + la.first + la.at(m)) : 0.f;
    }
  }
  const bool sums = q.keep < q.G && q.group_top == 2;  // group values are sums of scores
  const bool need_c = q.bias || sums;
  float lmax = 0.f, Z = 1.f, delta = 9.53674316e-7f;  // 2^-20
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

  const float rZ = rcp_approx(Z);
  // keys: of c with a bias, else of the logit; t1, t2: the lane's largest two c
  uint32_t key[MAXM], t1 = 0, t2 = 0;
#pragma unroll
  for (int m = 0; m < MAXM; ++m) {
    const bool there = la.in && la.at(m) < q.per;
    key[m] = there ? rank_key(l[m]) : 0u;
    uint32_t ck = key[m];
    if (need_c) {
      float c = order_score(q.sigmoid, l[m], lmax, rZ);
      if (q.bias) c += bias[m];
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
      if (!(lo - hi > e2)) {
        // (a NaN or an infinity among the two: nothing is below it, and all are computed)
        const float last = q.group_top == 2 ? rank_value(t2) : rank_value(t1);
        kept = kept_in_64(t, q.G, q.keep, q.group_top,
                          last - 2.f * (delta + 1.1920929e-7f * finite_abs(last)), Z);
      }
    }
  }
  if (!kept) {
#pragma unroll
    for (int m = 0; m < MAXM; ++m) key[m] = 0u;
  }

  typename Pick<(MAXM + 7) / 8, MAXM, VEC>::type offers;
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
    const bool close = has_next && !(a - b > apart) && !(a == b && fabsf(a) == INFINITY);
    bool near = close;
    if (close) near = !(lt[my_e] == lt[next_e] && q.bias[my_e] == q.bias[next_e]);
    const float ck = __shfl_sync(kAll, a, q.k - 1);
    // a tie of the k-th and the first left: the neighbours that are left stand behind all that tie with them
    if (__any_sync(kAll, lane == q.k - 1 && close && !near))
      near |= t.others_near(kept, __shfl_sync(kAll, my_e, q.k - 1), ck, delta, rZ);
    if (__any_sync(kAll, near)) {
      // every expert that may belong among the k: those within the bounds of the k-th's c
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
__global__ void __launch_bounds__(256) k_route_select(const GateParams q) {
  pdl_wait_then_release();
  const long tok = (long)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
  if (tok < q.T) select_token<MAXM, VEC>(q, tok);
}

// ---- large batches: eight lanes a token ------------------------------------------------------------
//
// A warp takes four tokens, M experts a lane, so that what the selection costs beside the scores is shared by
// four. A key is the value's order-preserving bits with the expert's number within the lane in the last
// B = log2 M of them: one maximum then finds value and expert. A lane keeps its eight largest keys sorted
// (networks of compare-exchanges on single words); then, with the lane's number in three more bits, the eight
// lists of a token are merged to its eight largest in three exchanges. Keys leave values a relative
// 2^-(23 - B) or 2^-(20 - B), so the eight are ranked in full precision, and the k-th is compared with the
// largest value that the rest may have. Where those are not apart by their bounds, where group values are
// not, where a lane's eight end among those looked at (what it has beside them is in no list), and where a value is
// NaN or +infinity, the whole warp selects for that token again as above (a few tokens in a thousand at 256 experts;
// in a second kernel, with a mark in the first's output, that took longer: 24.1 us for 21.4).

__device__ __forceinline__ void order(uint32_t& a, uint32_t& b) {
  const uint32_t hi = max(a, b), lo = min(a, b);
  a = hi;
  b = lo;
}

// Descending sort of eight words.
__device__ __forceinline__ void sort8(uint32_t (&v)[8]) {
  order(v[0], v[2]); order(v[1], v[3]); order(v[4], v[6]); order(v[5], v[7]);
  order(v[0], v[4]); order(v[1], v[5]); order(v[2], v[6]); order(v[3], v[7]);
  order(v[0], v[1]); order(v[2], v[3]); order(v[4], v[5]); order(v[6], v[7]);
  order(v[2], v[4]); order(v[3], v[5]);
  order(v[1], v[4]); order(v[3], v[6]);
  order(v[1], v[2]); order(v[3], v[4]); order(v[5], v[6]);
}

// The eight largest of two descending lists, descending, into a: the larger of a[i] and b[7 - i] are they, in
// an order that rises and falls once, which three steps sort.
__device__ __forceinline__ void merge8(uint32_t (&a)[8], const uint32_t (&b)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) a[i] = max(a[i], b[7 - i]);
#pragma unroll
  for (int d = 4; d >= 1; d >>= 1)
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if ((i & d) == 0) order(a[i], a[i + d]);
}

template <typename V>
__device__ __forceinline__ V max8(V v) {  // over the eight lanes of a token
#pragma unroll
  for (int o = 4; o >= 1; o >>= 1) v = max(v, __shfl_xor_sync(kAll, v, o));
  return v;
}
__device__ __forceinline__ float sum8(float v) {
#pragma unroll
  for (int o = 4; o >= 1; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
  return v;
}

// Order-preserving bits of a number that is no NaN, -0 below +0.
__device__ __forceinline__ uint32_t bits_key(float v) {
  const uint32_t u = __float_as_uint(v);
  return u ^ ((uint32_t)((int)u >> 31) | 0x80000000u);
}

template <int M>
__global__ void __launch_bounds__(128, 7) k_route_select_many(const GateParams q) {
  constexpr int B = M <= 8 ? 3 : M <= 16 ? 4 : M <= 32 ? 5 : 6;
  constexpr uint32_t kLow = (1u << B) - 1u, kLow8 = (8u << B) - 1u;
  constexpr float kRel = 2.f / (float)(1u << (23 - B));    // twice what the last bits stand for
  constexpr float kRel8 = 2.f / (float)(1u << (20 - B));
  constexpr float kRel32 = 1.1920929e-7f;
  pdl_wait_then_release();
  const int lane = threadIdx.x & 31, j = lane & 7, base = lane & 24;
  const long tok0 = 4 * ((long)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5));
  if (tok0 >= q.T) return;
  const long tok = min(tok0 + (lane >> 3), (long)q.T - 1);  // the last warp's spare lanes repeat it
  const float* lt = q.logits + tok * q.E;
  const Lane<true> la = lane_of<true>(q, j, q.P >> 2);
  const bool sums = q.keep < q.G && q.group_top == 2;

  // A lane that has a group of its own would read every 16 bytes of another line than its neighbours: its
  // experts come through shared memory instead (rows padded by 16 bytes: no bank twice), quads of experts
  // read in a row by the eight lanes (16384 tokens: 21.4 us for 22.3).
  float l[M];
  __shared__ float4 rows[4][32][M / 4 + 1];
  const bool staged = la.P == 1;
  if (staged) {
    float4 (*mine)[M / 4 + 1] = rows[threadIdx.x >> 5];
    const uint32_t quads = (uint32_t)q.per >> 2, inv = 65536u / quads + 1;  // n / quads, n < 128
    float4 f[M / 4];
#pragma unroll
    for (int i = 0; i < M / 4; ++i) {
      const uint32_t n = 8 * i + j;
      if (4 * n < (uint32_t)q.E) f[i] = *reinterpret_cast<const float4*>(lt + 4 * n);
    }
#pragma unroll
    for (int i = 0; i < M / 4; ++i) {
      const uint32_t n = 8 * i + j, g = (n * inv) >> 16;
      if (4 * n < (uint32_t)q.E) mine[base + g][n - g * quads] = f[i];
    }
    __syncwarp();
  }
#pragma unroll
  for (int m = 0; m < M; m += 4) {
    float4 f = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
    if (la.in && la.at(m) < q.per)
      f = staged ? rows[threadIdx.x >> 5][lane][m >> 2]
                 : *reinterpret_cast<const float4*>(lt + la.first + la.at(m));
    l[m] = f.x;
    l[m + 1] = f.y;
    l[m + 2] = f.z;
    l[m + 3] = f.w;
  }
  bool again = false;
  float lmax = 0.f, Z = 1.f, delta = 9.53674316e-7f;  // 2^-20
  if (!q.sigmoid && (q.bias || sums || !q.renorm)) {
    float mx = l[0];
#pragma unroll
    for (int m = 1; m < M; ++m) mx = fmaxf(mx, l[m]);
    lmax = max8(mx);
    float z = 0.f;
#pragma unroll
    for (int m = 0; m < M; ++m)
      if (la.in && la.at(m) < q.per) z += expf(l[m] - lmax);
    Z = sum8(z);
    delta = 7.62939453e-6f / Z;  // 2^-17 of the largest score
  }
  const float rZ = rcp_approx(Z);
  const auto score = [&](float x) { return order_score(q.sigmoid, x, lmax, rZ); };
  uint32_t top[8];
#pragma unroll
  for (int m0 = 0; m0 < M; m0 += 8) {
    uint32_t part[8];
#pragma unroll
    for (int i0 = 0; i0 < 8; i0 += 4) {
      const int m = m0 + i0;
      const bool there = m < M && la.in && la.at(m) < q.per;  // all four, or none
      float4 b = make_float4(0.f, 0.f, 0.f, 0.f);
      if (q.bias && there) b = __ldg(reinterpret_cast<const float4*>(q.bias + la.first + la.at(m)));
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float v = l[m + i < M ? m + i : 0];
        v = q.bias ? score(v) + (i == 0 ? b.x : i == 1 ? b.y : i == 2 ? b.z : b.w) : v + 0.f;
        again |= there && !(v < INFINITY);
        part[i0 + i] = there ? (bits_key(v) & ~kLow) | (kLow - (uint32_t)(m + i)) : 0u;
      }
    }
    sort8(part);
    if (m0 == 0) {
#pragma unroll
      for (int i = 0; i < 8; ++i) top[i] = part[i];
    } else {
      merge8(top, part);
    }
  }

  if (q.keep < q.G) {
    // not below the true value. Where softmax scores of logits are summed it is cut to the largest logit: a logit
    // of some millions may be rounded up by more than one, and e^x grows faster than the bound in err
    const float most = !q.sigmoid && !q.bias && sums ? lmax : INFINITY;
    const auto val = [most](uint32_t key) { return fminf(key_logit(key | kLow), most); };
    uint32_t t1 = top[0], t2 = top[1];
    group_top2(t1, t2, la.P);
    // v: not below the group's value but for the scores' bounds, nor above it by more than what the last
    // bits stand for (a sigmoid moves by at most a quarter of what its logit does, a softmax score by at most 1 / Z of
    // it, as e^x <= 1 between the true logit and the cut one). One side's bits and both sides' bounds are in err.
    float v = -INFINITY, err = 0.f;
    if (la.in) {
      const float a = val(t1), b = val(t2), bits = 0.5f * kRel;
      v = a;
      err = q.bias ? 2.f * delta + bits * finite_abs(a) : 0.f;  // logits' keys that differ are in order
      if (q.group_top == 2) {
        v = q.bias ? a + b : score(a) + score(b);
        err = 4.f * delta + kRel32 * finite_abs(v) +
              bits * (finite_abs(a) + finite_abs(b)) * (q.bias ? 1.f : q.sigmoid ? 0.25f : rZ);
      }
    }
    int before = 0;
    for (int h = 0; h < q.G; ++h) {
      const float o = __shfl_sync(kAll, v, base + h * la.P);
      before += (o > v || (o == v && h < la.g)) ? 1 : 0;
    }
    const bool kept = la.in && before < q.keep;
    const float lo = -max8(kept ? -v : -INFINITY), hi = max8(la.in && !kept ? v : -INFINITY);
    again |= !(lo - hi > max8(err));
    if (!kept) {
#pragma unroll
      for (int i = 0; i < 8; ++i) top[i] = 0u;
    }
  }

  // the token's eight largest, in every lane of it
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (top[i]) top[i] = (top[i] & ~kLow8) | (uint32_t)(j << B) | (top[i] & kLow);
  sort8(top);
  uint32_t best[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) best[i] = top[i];
#pragma unroll
  for (int o = 1; o <= 4; o <<= 1) {
    uint32_t other[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) other[i] = __shfl_xor_sync(kAll, best[i], o);
    merge8(best, other);
  }
  again |= M > 8 && top[7] != 0u && top[7] >= best[7];  // a lane whose eight are all among them has more
  // below the eight: the ninth, and the largest that the others may be
  uint32_t mine = best[0], ninth = 0, rest = 0;
#pragma unroll
  for (int i = 1; i < 8; ++i) mine = j == i ? best[i] : mine;
#pragma unroll
  for (int i = 7; i >= 0; --i) ninth = top[i] < best[7] ? max(ninth, top[i]) : ninth;
  ninth = max8(ninth);
  again |= M > 8 && q.k == 8 && top[7] != 0u && top[7] >= ninth;  // as one whose list ends with the ninth
#pragma unroll
  for (int i = 7; i >= 0; --i) rest = top[i] < ninth ? max(rest, top[i]) : rest;
  rest = max8(rest);

  // the eight, and the ninth if all eight are chosen, in full precision
  const auto expert = [&](uint32_t key) {
    const Lane<true> lf = lane_of<true>(q, (int)(key >> B) & 7, la.P);
    return lf.first + lf.at((int)(kLow - (key & kLow)));
  };
  const auto exact = [&](int e, float x) {
    return q.bias ? (q.sigmoid ? sigmoid32(x) : expf(x - lmax) / Z) + __ldg(q.bias + e) : x;
  };
  const bool there = mine != 0u;
  int e = there ? expert(mine) : 0;
  float le = there ? lt[e] : -INFINITY;
  const float v = there ? exact(e, le) : -INFINITY;
  // bounds of the difference of two: sigmoid32 within 2^-21, softmax as above
  const float d = !q.bias ? 0.f : q.sigmoid ? 9.53674316e-7f : 2.f * delta, rel = q.bias ? kRel32 : 0.f;
  int rank = 0;
  bool close = false;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float o = __shfl_sync(kAll, v, base + i);
    const uint32_t key = __shfl_sync(kAll, mine, base + i);
    const bool other = i != j && key != 0u;
    rank += other && o > v ? 1 : 0;
    close |= other && !(fabsf(o - v) > d + rel * (finite_abs(o) + finite_abs(v)));
  }
  if (!there) rank = 8;
  const bool in = rank < q.k;
  again |= in && close;
  if (q.k == 8 && ninth != 0u) {
    const int e9 = expert(ninth);
    const float v9 = exact(e9, lt[e9]);
    again |= !(v - v9 > d + rel * (finite_abs(v) + finite_abs(v9)));
  }
  // what the rest may be: below the keys that were given out, up to what their last bits stand for
  const uint32_t bound = q.k == 8 ? rest : ninth;
  if (bound != 0u) {
    const float r = key_logit(bound | kLow8);
    again |= in && !(v - r > 2.f * d + (q.bias ? kRel8 : 0.f) * (finite_abs(v) + finite_abs(r)));
  }
  const unsigned redo = __ballot_sync(kAll, again);
  if (__any_sync(kAll, there && rank != j)) {  // lane r takes the one of rank r
    int place = j;
    for (int i = 0; i < 8; ++i)
      if (__shfl_sync(kAll, rank, base + i) == j) place = i;
    e = __shfl_sync(kAll, e, base + place);
    le = __shfl_sync(kAll, le, base + place);
  }
  if (j >= q.k) le = -INFINITY;
  float s, mx = -INFINITY;
  if (q.renorm) mx = max8(le);
  if (q.renorm && (!q.sigmoid || (mx < -60.f && mx > -INFINITY)))
    s = j < q.k ? expf(le - mx) : 0.f;
  else if (q.sigmoid)
    s = j < q.k ? sigmoid32(le) : 0.f;
  else
    s = j < q.k ? expf(le - lmax) / Z : 0.f;
  if (q.renorm) {
    const float sum = sum8(s);
    s = sum == 0.f ? 0.f : s / sum;
  }
  if (j < q.k && tok0 + (lane >> 3) < q.T) {
    q.idx[tok * q.k + j] = e;
    q.w[tok * q.k + j] = s * q.scale;
  }
  __syncwarp();
  for (int t = 0; t < 4; ++t)
    if (((redo >> (8 * t)) & 0xFFu) && tok0 + t < q.T)
      select_token<M <= 16 ? 4 : M <= 32 ? 8 : 16, true>(q, tok0 + t);
}

template <int M>
cudaError_t launch_many(const GateParams& q, cudaStream_t st) {
  return launch_pdl(k_route_select_many<M>, dim3((unsigned)((q.T + 15) / 16)), dim3(128), 0, st, q);
}

template <int MAXM, bool VEC>
cudaError_t launch_one(const GateParams& q, cudaStream_t st) {
  // small batches: warps on SMs of their own rather than eight to a block
  const int per_sm = (q.T + num_sms() - 1) / num_sms();
  const int warps = per_sm < 8 ? per_sm : 8;
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
  // Eight lanes a token: up to 8 groups and 8 choices, and so many tokens that the warps' share of work counts
  // and not one warp's latency (with a bias a launch as a rule has tokens that are done again, 5 us; measured
  // at 256 experts in 8 groups: 4096 tokens 11.6 us by warps and 14.9, 6144 tokens 15.6 and 14.0, 16384 tokens 30.9
  // and 19.4; without a bias 4099 tokens of 160 experts 7.3 and 6.0).
  const int m8 = vec && lanes <= 8 ? (q.per + q.P - 1) / q.P * 4 : 0;  // experts of a lane
  if (m8 && m8 <= 48 && q.k <= 8 && q.T >= (bias ? 6144 : 2048)) {
    if (m8 <= 8) return launch_many<8>(q, st);
    if (m8 <= 16) return launch_many<16>(q, st);
    if (m8 <= 32) return launch_many<32>(q, st);
    return launch_many<48>(q, st);
  }
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
