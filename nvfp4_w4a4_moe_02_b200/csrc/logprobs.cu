// Log probabilities of given tokens, with the entropy of the distribution and its top
// alternatives, and their gradient: the two sides of the rollout-trainer log-prob gap.
//
// With z = l / temperature over a row l of V logits, m = max l, c = log2(e) / temperature:
//   y_v = l_v c - M with M = RN(m c),  s = sum 2^y_v,  u = sum 2^y_v y_v   (one pass, running maximum)
//   logprob = ln2 (y_id - log2 s),  entropy = ln2 (log2 s - u / s)
//   d l_v = ( g_lp (1[v = id] - p_v) - g_H p_v (ln p_v + H) ) / temperature,  p_v = 2^y_v / s
// M is the reference itself, not an approximation of one: its rounding changes nothing, and y is
// rounded once.  All sums and statistics are binary32.
//
// The forward pass reads the logits once and the backward pass reads and writes once, both bound by
// memory; on the way there the exponentials (16 a clock and SM against 11.6 bf16 logits) and the
// instructions come next, so sums and products go in pairs (fma.rn.f32x2) and masks cost one packed
// maximum: logits below kLow count as kLow, 2^y = 0 then, and y stays finite.  A row whose largest
// logit is not above kLow (masked by the type's lowest value, or all -inf) is done again exactly.
#include "common.cuh"
#include "kernels.h"
#include "logprobs_index.h"

namespace nvfp4 {

namespace {

constexpr float kLn2 = 0.6931471805599453f;
constexpr float kLog2e = 1.4426950408889634f;
// -2^100, a bf16: for c in [2^-26, 2^27] kLow c is finite, and 2^(kLow c - M) is 0 for every M above it
constexpr float kLow = -1.2676506002282294e30f;
// A row that the fast form cannot hold: nothing above kLow, or |M| so large that its rounding (y at the
// maximum, up to 2^-25 |M|) would no longer be a small power of two
__device__ __forceinline__ bool needs_exact(float m, float M) { return !(m > kLow && fabsf(M) < 268435456.0f); }

__device__ __forceinline__ float ex2(float y) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(y));  // 2 ulp; 0 below 2^-126, where it adds nothing to s >= 1
  return r;
}

template <typename L>
struct Vec;  // 16 bytes of logits
template <>
struct Vec<float> {
  static constexpr int N = 4;
  static __device__ __forceinline__ void unpack(const uint4& r, float* x) {
    x[0] = __uint_as_float(r.x);
    x[1] = __uint_as_float(r.y);
    x[2] = __uint_as_float(r.z);
    x[3] = __uint_as_float(r.w);
  }
  // A lower bound as clamp() takes it, not above `low`
  static __device__ __forceinline__ uint32_t bound(float low) { return __float_as_uint(low); }
  // x_i = max(l_i, low), NaN kept; returns the largest l, NaN skipped
  static __device__ __forceinline__ float clamp(uint4& r, uint32_t low) {
    uint32_t* w = &r.x;
    const float m = fmaxf(fmaxf(__uint_as_float(r.x), __uint_as_float(r.y)), fmaxf(__uint_as_float(r.z), __uint_as_float(r.w)));
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float v;
      asm("max.NaN.f32 %0, %1, %2;" : "=f"(v) : "f"(__uint_as_float(w[i])), "f"(__uint_as_float(low)));
      w[i] = __float_as_uint(v);
    }
    return m;
  }
  static __device__ __forceinline__ float get(const float* p) { return *p; }
  static __device__ __forceinline__ uint4 pack(const float* x) {
    return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
  }
  static __device__ __forceinline__ void put(float* p, float v) { *p = v; }
};
template <>
struct Vec<uint16_t> {  // bf16 bit patterns
  static constexpr int N = 8;
  static __device__ __forceinline__ void unpack(const uint4& r, float* x) {
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  }
  static __device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
    uint32_t v;
    asm("max.bf16x2 %0, %1, %2;" : "=r"(v) : "r"(a), "r"(b));
    return v;
  }
  static __device__ __forceinline__ uint32_t bound(float low) {
    const __nv_bfloat16 b = __float2bfloat16_rd(low);
    return (uint32_t)*reinterpret_cast<const uint16_t*>(&b) * 0x10001u;
  }
  static __device__ __forceinline__ float clamp(uint4& r, uint32_t low) {
    const uint32_t m = max2(max2(r.x, r.y), max2(r.z, r.w));
    uint32_t* w = &r.x;
#pragma unroll
    for (int i = 0; i < 4; ++i) asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(w[i]) : "r"(w[i]), "r"(low));
    return fmaxf(__uint_as_float(m << 16), __uint_as_float(m & 0xFFFF0000u));
  }
  static __device__ __forceinline__ float get(const uint16_t* p) { return bf16_bits_to_f32(*p); }
  static __device__ __forceinline__ uint4 pack(const float* x) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 b = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&b);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
  static __device__ __forceinline__ void put(uint16_t* p, float v) {
    const __nv_bfloat16 b = __float2bfloat16_rn(v);
    *p = *reinterpret_cast<const uint16_t*>(&b);
  }
};

constexpr int64_t kWarpRow = 1024;   // rows up to this length go to a warp each
constexpr int64_t kPairRow = 32768;  // and up to this one to two, where there are many

// Running statistics of a part of a row against the reference M = RN(m c), m the largest logit seen.
// Nothing above kLow yet: m is what it is, M = -inf, s = u = 0.  A NaN or +inf ends as s = NaN.
struct __align__(16) Stat {
  float m, M, s, u;
};

// Scales a part to the reference M (>= its own).
__device__ __forceinline__ void rebase(Stat& a, float M) {
  const float d = a.M - M;
  const float f = ex2(d);
  if (f == 0.0f) {
    // a part 2^-126 below adds nothing; its sums may even be infinite (a thread that saw only a mask's
    // -1e15 has an M whose rounding is large), but NaN stays NaN
    if (a.s == a.s) a.s = 0.0f;
    a.u = a.s;
  } else {
    a.u = f * fmaf(d, a.s, a.u);
    a.s *= f;
  }
  a.M = M;
}

// Joins the parts of n (a power of two) consecutive lanes; every lane gets the result, the same bits.
template <int n>
__device__ __forceinline__ void join_lanes(Stat& a) {
  float m = a.m, M = a.M;
#pragma unroll
  for (int o = n / 2; o > 0; o >>= 1) {
    m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
  }
  if (M > -INFINITY) rebase(a, M);  // else every s is 0 or NaN
  a.m = m;
#pragma unroll
  for (int o = n / 2; o > 0; o >>= 1) {
    a.s += __shfl_xor_sync(0xffffffffu, a.s, o);
    a.u += __shfl_xor_sync(0xffffffffu, a.u, o);
  }
}

// Adds U x N logits to a part.
template <typename L, int U>
__device__ __forceinline__ void add_vectors(Stat& a, uint4 (&r)[U], float c) {
  constexpr int N = Vec<L>::N;
  const uint32_t low = Vec<L>::bound(kLow);
  float bm = Vec<L>::clamp(r[0], low);
#pragma unroll
  for (int i = 1; i < U; ++i) bm = fmaxf(bm, Vec<L>::clamp(r[i], low));
  if (!(bm <= a.m)) {
    a.m = fmaxf(a.m, bm);
    if (a.m > kLow) rebase(a, __fmul_rn(a.m, c));
  }
  // while nothing is above kLow the elements are skipped: they add nothing to a row that has more, and
  // the others are done again; a NaN must not be lost
  const float M = a.M > -INFINITY ? a.M : 0.0f;
  const float2 c2 = make_float2(c, c), M2 = make_float2(-M, -M);
  float2 s = make_float2(0.0f, 0.0f), u = s;
#pragma unroll
  for (int i = 0; i < U; ++i) {
    float x[N];
    Vec<L>::unpack(r[i], x);
#pragma unroll
    for (int j = 0; j < N; j += 2) {
      const float2 y = __ffma2_rn(make_float2(x[j], x[j + 1]), c2, M2);
      const float2 e = make_float2(ex2(y.x), ex2(y.y));
      s = __fadd2_rn(s, e);
      u = __ffma2_rn(e, y, u);
    }
  }
  a.s += s.x + s.y;
  a.u += u.x + u.y;
}

// A row's edges go element by element.
__device__ __forceinline__ void add_element(Stat& a, float x, float c) {
  if (x != x) a.s = x;
  if (x > a.m) {
    a.m = x;
    if (x > kLow) rebase(a, __fmul_rn(x, c));
  }
  if (a.M > -INFINITY) {
    const float y = fmaf(fmaxf(x, kLow), c, -a.M);
    const float e = ex2(y);
    a.s += e;
    a.u = fmaf(e, y, a.u);
  }
}
// The exact form: m is the row's largest logit.
__device__ __forceinline__ void add_exact(float& s, float& u, float x, float m, float c) {
  const float y = (x - m) * c;
  const float e = ex2(y);
  s += e;
  u = fmaf(e, fmaxf(y, -1000.0f), u);
}

// Order of the alternatives: value descending, index ascending, as one unsigned key (0 = none).
__device__ __forceinline__ uint32_t order_bits(float v) {
  const uint32_t b = __float_as_uint(v + 0.0f);  // -0 ties with +0
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}
__device__ __forceinline__ uint64_t order_key(float v, uint32_t idx) {
  return ((uint64_t)order_bits(v) << 32) | (0xFFFFFFFFu - idx);
}
__device__ __forceinline__ float key_value(uint64_t key) {
  const uint32_t k = (uint32_t)(key >> 32);
  return __uint_as_float((k & 0x80000000u) ? (k & 0x7FFFFFFFu) : ~k);
}
__device__ __forceinline__ int32_t key_index(uint64_t key) { return (int32_t)(0xFFFFFFFFu - (uint32_t)key); }

// A warp's best 32 keys, lane i holding the i-th; thr: a key is taken if it is above.
__device__ __forceinline__ void insert_key(uint64_t& mine, uint64_t& thr, uint64_t key, int k) {
  const int lane = threadIdx.x & 31;
  const int pos = __popc(__ballot_sync(0xffffffffu, mine > key));
  const uint64_t up = __shfl_up_sync(0xffffffffu, mine, 1);
  if (lane == pos) mine = key;
  if (lane > pos) mine = up;
  const uint64_t kth = __shfl_sync(0xffffffffu, mine, k - 1);
  thr = kth > thr ? kth : thr;
}

// One logit per lane (`has` false: none).
__device__ __forceinline__ void offer(uint64_t& mine, uint64_t& thr, float x, uint32_t idx, bool has, int k) {
  const uint64_t key = has ? order_key(x, idx) : 0;
  uint32_t mask = __ballot_sync(0xffffffffu, key > thr);
  while (mask) {
    const uint64_t q = __shfl_sync(0xffffffffu, key, __ffs(mask) - 1);
    if (q > thr) insert_key(mine, thr, q, k);
    mask &= mask - 1;
  }
}

// Sorts one value per lane, descending.
__device__ __forceinline__ float sort_lanes(float v) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int size = 2; size <= 32; size <<= 1) {
#pragma unroll
    for (int o = size / 2; o > 0; o >>= 1) {
      const float w = __shfl_xor_sync(0xffffffffu, v, o);
      const bool keep_max = ((lane & o) == 0) == ((lane & size) == 0);
      v = keep_max ? fmaxf(v, w) : fminf(v, w);
    }
  }
  return v;
}
// The k-th largest of one value per lane: for a few, as many arg-max rounds; else the sorted list.
__device__ __forceinline__ float kth_lane(float v, int k) {
  if (k > 8) return __shfl_sync(0xffffffffu, sort_lanes(v), k - 1);
  uint32_t o = order_bits(v), m = 0;
  for (int r = 0; r < k; ++r) {
    m = __reduce_max_sync(0xffffffffu, o);
    if ((__ffs(__ballot_sync(0xffffffffu, o == m)) - 1) == (int)(threadIdx.x & 31)) o = 0;
  }
  return key_value((uint64_t)m << 32);
}
// Two descending lists -> their best 32, descending: the element-wise maximum of one and the other
// reversed is bitonic and holds them; five exchanges sort it.
__device__ __forceinline__ float merge_lanes(float a, float b) {
  const int lane = threadIdx.x & 31;
  float v = fmaxf(a, __shfl_xor_sync(0xffffffffu, b, 31));
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const float w = __shfl_xor_sync(0xffffffffu, v, o);
    v = (lane & o) == 0 ? fmaxf(v, w) : fminf(v, w);
  }
  return v;
}

__device__ __forceinline__ int64_t read_id(const void* ids, int id_bytes, int64_t t) {
  return id_bytes == 8 ? __ldg(reinterpret_cast<const long long*>(ids) + t)
                       : (int64_t)__ldg(reinterpret_cast<const int*>(ids) + t);
}

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.aligned;" ::: "memory"); }
// Stores to the same variable of the cluster's first block.
__device__ __forceinline__ uint32_t first_block(const void* p) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(r) : "r"((uint32_t)__cvta_generic_to_shared(p)));
  return r;
}
__device__ __forceinline__ void store_remote(Stat* p, const Stat& v) {
  asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};"
               :
               : "r"(first_block(p)), "f"(v.m), "f"(v.M), "f"(v.s), "f"(v.u)
               : "memory");
}
__device__ __forceinline__ void store_remote(uint64_t* p, uint64_t v) {
  asm volatile("st.shared::cluster.u64 [%0], %1;" : : "r"(first_block(p)), "l"(v) : "memory");
}

// A row, or a block's share of one: elements before the first 16-byte boundary and after the last one
// go one by one (at most 14, all to the share that has any).
template <typename L>
struct Span {
  const L* row;
  int lo, hi;        // this share's vectors
  int head, V;
  int edge;          // elements that go one by one here
  __device__ __forceinline__ Span(const L* r, int v, int part, int parts) : row(r), V(v) {
    constexpr int N = Vec<L>::N;
    head = min(v, (int)((16 - (reinterpret_cast<uintptr_t>(r) & 15)) & 15) / (int)sizeof(L));
    const int nvec = (v - head) / N;
    lo = (int)((int64_t)nvec * part / parts);
    hi = (int)((int64_t)nvec * (part + 1) / parts);
    edge = part == 0 ? v - nvec * N : 0;
  }
  __device__ __forceinline__ int edge_index(int i) const { return i < head ? i : V - edge + i; }
  __device__ __forceinline__ const uint4* vec() const { return reinterpret_cast<const uint4*>(row + head); }
};

}  // namespace

// One row per team.  W = 8: a team is a cluster of `parts` blocks, each with its share of the row, joined
// through the cluster's shared memory; W = 2: a block of two warps; W = 1: a block holds eight one-warp
// teams.
//
// Alternatives: every thread knows the largest of its logits; the k-th largest of these, tau, is a
// lower bound of the k-th alternative, and only threads whose largest is not below it can hold one.
// Their logits (k threads' worth unless logits tie) are read again, those not below tau are listed, and
// a listed one's place is the number of larger ones.  A list that would overflow (many ties at tau) is
// replaced by one sorted list per warp.
template <typename L, int W, bool TOP>
__global__ void __launch_bounds__(W > 1 ? W * 32 : 256) logprobs_kernel(LogprobArgs a, int parts) {
  constexpr int N = Vec<L>::N;
  constexpr int kTeam = W * 32;
  constexpr int kMaxParts = 8;
  constexpr int kCap = W == 1 ? 128 : W == 2 ? 256 : 512;
  __shared__ Stat part_stat[W > 1 ? W : 1];
  __shared__ float maxima[TOP && W > 1 ? W : 1][32];
  __shared__ uint64_t listed[W > 1 ? 1 : 8][TOP ? kCap : 1];  // per block, or per warp
  __shared__ int list_size[8];
  __shared__ uint8_t holder[8][32];
  __shared__ uint64_t best[TOP && W == 1 ? 8 : 1][32];         // the team's best k, in order
  // of the cluster's blocks, in the first one
  __shared__ Stat team_stat[kMaxParts];
  __shared__ uint64_t team_best[TOP && W == 8 ? kMaxParts * 32 : 1];
  const int lane = threadIdx.x & 31;
  const int warp = threadIdx.x >> 5;
  const int tid = W > 1 ? threadIdx.x : lane;
  const int part = W > 1 ? (int)(blockIdx.x % parts) : 0;
  const int64_t t = W > 1 ? (int64_t)(blockIdx.x / parts) : (int64_t)blockIdx.x * 8 + warp;
  if (t >= a.T) return;
  const int k = a.k_top;
  int64_t id = read_id(a.ids, a.id_bytes, t);
  const bool first = part == 0 && tid == 0;
  if (id >= a.V) {
    if (first) report_status(a.status, kErrInvalid);
    id = -1;
  }
  if (id < 0) {  // padding: the row is not read (all of a cluster leave here)
    if (first) {
      a.logprob[t] = 0.0f;
      if (a.entropy) a.entropy[t] = 0.0f;
      if (a.stats) reinterpret_cast<float4*>(a.stats)[t] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    }
    if (TOP && part == 0 && tid < k) {
      a.top_ids[t * k + tid] = -1;
      a.top_lp[t * k + tid] = 0.0f;
    }
    return;
  }
  const float c = a.inv_temp * kLog2e;
  const L* row = reinterpret_cast<const L*>(a.logits) + t * a.ld;
  const Span<L> sp(row, (int)a.V, part, parts);
  if (W == 8 && parts > 1) {
    __syncwarp();
    cluster_arrive();
  }
  float l_id = 0.0f;
  if (first) l_id = Vec<L>::get(row + id);

  Stat st{-INFINITY, -INFINITY, 0.0f, 0.0f};
  int v = sp.lo + tid;
  auto add_full = [&](auto& r) {
    constexpr int n = sizeof(r) / sizeof(r[0]);
#pragma unroll
    for (int i = 0; i < n; ++i) r[i] = __ldg(sp.vec() + v + i * kTeam);
    add_vectors<L, n>(st, r, c);
    v += n * kTeam;
  };
  // eight vectors on the way per thread (4096 x 131072 bf16: 162 us, four: 167 us; 1023 x 32000 f32: 24 us,
  // 27 us); a warp's short row has no use for them
  while (W > 1 && v + 7 * kTeam < sp.hi) {
    uint4 r[8];
    add_full(r);
  }
  while (v + 3 * kTeam < sp.hi) {
    uint4 r[4];
    add_full(r);
  }
  if (v < sp.hi) {
    uint4 r[3];
#pragma unroll
    for (int i = 0; i < 3; ++i) {
      // absent vectors: -inf, which adds nothing
      r[i] = sizeof(L) == 4 ? make_uint4(0xFF800000u, 0xFF800000u, 0xFF800000u, 0xFF800000u)
                            : make_uint4(0xFF80FF80u, 0xFF80FF80u, 0xFF80FF80u, 0xFF80FF80u);
      if (v + i * kTeam < sp.hi) r[i] = __ldg(sp.vec() + v + i * kTeam);
    }
    add_vectors<L, 3>(st, r, c);
  }
  if (tid < sp.edge) add_element(st, Vec<L>::get(row + sp.edge_index(tid)), c);
  // the largest logit of this thread: where it is not above kLow, the maximum was taken all the same
  const float own_max = st.m;

  join_lanes<32>(st);
  float tau = -INFINITY;
  const int team_list = W > 1 ? 0 : warp;
  if (W > 1) {
    float sorted = 0.0f;
    if (lane == 0) part_stat[warp] = st;
    if (TOP) {
      sorted = sort_lanes(own_max);
      maxima[warp][lane] = sorted;
      if (tid == 0) list_size[0] = 0;
      if (tid < 32) best[0][tid] = 0;
    }
    __syncthreads();
    st = part_stat[lane & (W - 1)];
    join_lanes<W>(st);
    if (TOP) {
#pragma unroll
      for (int o = 1; o < W; o <<= 1) {  // lists of 2 o warps meet in the first of them
        if ((warp & (2 * o - 1)) == 0) {
          sorted = merge_lanes(sorted, maxima[warp + o][lane]);
          maxima[warp][lane] = sorted;
        }
        __syncthreads();
      }
      tau = maxima[0][k - 1];
    }
  } else if (TOP) {
    tau = kth_lane(own_max, k);
    if (lane == 0) list_size[warp] = 0;
    best[warp][lane] = 0;
  }
  uint64_t key = 0;
  int place = 32;
  if (TOP) {
    uint64_t* list = listed[team_list];
    const uint64_t floor_key = (uint64_t)order_bits(tau) << 32;  // below every logit that is not below tau
    auto put = [&](float x, uint32_t idx) {
      const uint64_t q = order_key(x, idx);
      if (q > floor_key) {
        const int at = atomicAdd(&list_size[team_list], 1);
        if (at < kCap) list[at] = q;
      }
    };
    const uint32_t holders = __ballot_sync(0xffffffffu, !(own_max < tau));
    if (!(own_max < tau)) holder[warp][__popc(holders & ((1u << lane) - 1u))] = (uint8_t)lane;
    __syncwarp();
    const int per = (sp.hi - sp.lo + kTeam - 1) / kTeam;  // vectors of a thread
    const int todo = per * __popc(holders);
    const volatile int* listed_now = &list_size[team_list];
    for (int m = lane; m < todo && *listed_now <= kCap; m += 32) {
      const int h = m / per;
      const int w = sp.lo + (m - h * per) * kTeam + (W > 1 ? warp * 32 : 0) + holder[warp][h];
      if (w < sp.hi) {
        const uint4 r = __ldg(sp.vec() + w);
        float x[N];
        Vec<L>::unpack(r, x);
#pragma unroll
        for (int i = 0; i < N; ++i) put(x[i], (uint32_t)(sp.head + w * N + i));
      }
    }
    if (tid < sp.edge) {
      const int i = sp.edge_index(tid);
      put(Vec<L>::get(row + i), (uint32_t)i);
    }
    if (W > 1)
      __syncthreads();
    else
      __syncwarp();
    int size = list_size[team_list];
    if (size > kCap) {
      // too many: a sorted list of k per warp, of the warp's share of the row
      uint64_t mine = 0, thr = 0;
      for (int b = sp.lo + (W > 1 ? warp * 32 : 0); b < sp.hi; b += kTeam) {
        const int w = b + lane;
        const bool has = w < sp.hi;
        float x[N];
        Vec<L>::unpack(has ? __ldg(sp.vec() + w) : make_uint4(0, 0, 0, 0), x);
#pragma unroll
        for (int i = 0; i < N; ++i) offer(mine, thr, x[i], (uint32_t)(sp.head + w * N + i), has, k);
      }
      if (W == 1 || warp == 0) {
        const bool has = lane < sp.edge;
        const int i = has ? sp.edge_index(lane) : 0;
        offer(mine, thr, has ? Vec<L>::get(row + i) : 0.0f, (uint32_t)i, has, k);
      }
      if (W > 1) {
        __syncthreads();
        list[32 * warp + lane] = lane < k ? mine : 0;
        __syncthreads();
        size = 32 * W;
      } else {
        list[lane] = mine;
        __syncwarp();
        size = 32;
      }
    }
    // the place of each listed logit among them (zeros are none)
    for (int i = tid; i < size; i += kTeam) {
      const uint64_t q = list[i];
      int larger = 0;
      for (int j = 0; j < size; ++j) larger += list[j] > q;
      if (q != 0 && larger < k) best[team_list][larger] = q;
    }
    if (W > 1)
      __syncthreads();
    else
      __syncwarp();
  }
  if (W == 8 && parts > 1) {
    cluster_wait();  // every block of the cluster runs: the first one's shared memory may be written
    if (tid == 0) store_remote(&team_stat[part], st);
    if (TOP && tid < 32) store_remote(&team_best[32 * part + tid], best[0][tid]);
    __syncwarp();
    cluster_arrive();
    cluster_wait();
    if (part != 0) return;
    st = Stat{-INFINITY, -INFINITY, 0.0f, 0.0f};
    if ((lane & (kMaxParts - 1)) < parts) st = team_stat[lane & (kMaxParts - 1)];
    join_lanes<kMaxParts>(st);
    if (TOP && tid < 32 * parts) {
      key = team_best[tid];
      if (key != 0) {
        place = 0;
        for (int i = 0; i < parts; ++i)
          for (int j = 0; place < k && j < k && team_best[32 * i + j] > key; ++j) ++place;
      }
    }
  } else if (TOP && tid < 32) {
    key = best[team_list][tid];
    place = tid;
  }

  // m = -inf and no NaN: no distribution
  const bool empty = st.m == -INFINITY && st.s == 0.0f;
  if (st.m > -INFINITY && needs_exact(st.m, st.M)) {
    float s = 0.0f, u = 0.0f;
    for (int64_t i = tid; i < a.V; i += kTeam) add_exact(s, u, Vec<L>::get(row + i), st.m, c);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      s += __shfl_xor_sync(0xffffffffu, s, o);
      u += __shfl_xor_sync(0xffffffffu, u, o);
    }
    if (W > 1) {
      __syncthreads();
      if (lane == 0) part_stat[warp] = Stat{0.0f, 0.0f, s, u};
      __syncthreads();
      s = u = 0.0f;
      for (int w = 0; w < W; ++w) {
        s += part_stat[w].s;
        u += part_stat[w].u;
      }
    }
    st.s = s;
    st.u = u;
  }
  const float ls = empty ? 0.0f : log2f(st.s);
  const bool exact = needs_exact(st.m, st.M);
  auto log_prob = [&](float l) {
    // in nats where the pairs' form could overflow on the way to a finite result
    if (empty) return -INFINITY;
    if (exact || !(l > kLow)) return fmaf(ls, -kLn2, (l - st.m) * a.inv_temp);
    return (fmaf(l, c, -st.M) - ls) * kLn2;
  };
  if (tid == 0) {
    const bool bad = !empty && !(st.s < INFINITY);
    if (bad) report_status(a.status, kErrRange);
    const float h = empty ? 0.0f : bad ? NAN : fmaxf((ls - st.u / st.s) * kLn2, 0.0f);
    a.logprob[t] = bad ? NAN : log_prob(l_id);
    if (a.entropy) a.entropy[t] = h;
    if (a.stats) reinterpret_cast<float4*>(a.stats)[t] = make_float4(bad ? NAN : st.m, empty ? 0.0f : 1.0f / st.s, ls, h);
  }
  if (TOP && place < k && key != 0) {
    a.top_ids[t * k + place] = key_index(key);
    a.top_lp[t * k + place] = !empty && !(st.s < INFINITY) ? NAN : log_prob(key_value(key));
  }
}

// dlogits = 2^y (A + B y) + [v = id] g_lp / temperature, with the row's factors A, B.  W > 1: a block
// takes a stretch of a row, W = 1: a warp takes a row.  16-byte accesses where the row of the logits and
// of the gradient have the same phase.
// Eight blocks a SM keep enough bytes on the way for reads and writes together (4096 x 131072 bf16: 397 us
// at four, 347 us at six, 334 us at eight; with 32-bit indices in a row 327 us, 6.56 TB/s).
template <typename L, int W>
__global__ void __launch_bounds__(256, W > 1 ? 8 : 4) logprobs_backward_kernel(LogprobBwdArgs a, int64_t stretches) {
  constexpr int N = Vec<L>::N;
  constexpr int kTeam = W * 32;
  constexpr int U = 4;
  const int tid = W > 1 ? threadIdx.x : threadIdx.x & 31;
  const int64_t unit = W > 1 ? blockIdx.x : (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  const int64_t t = W > 1 ? unit / stretches : unit;
  const int64_t at = W > 1 ? unit % stretches : 0;
  if (t >= a.T) return;
  const L* row = reinterpret_cast<const L*>(a.logits) + t * a.ld;
  L* grow = reinterpret_cast<L*>(a.grad) + t * a.ldg;
  int64_t id = read_id(a.ids, a.id_bytes, t);
  const float4 st = __ldg(reinterpret_cast<const float4*>(a.stats) + t);  // m, 1 / s, log2 s, entropy
  if (id >= a.V) {
    if (tid == 0 && at == 0) report_status(a.status, kErrInvalid);
    id = -1;
  }
  const float c = a.inv_temp * kLog2e;
  const bool zero = id < 0 || st.x == -INFINITY;
  const float M = __fmul_rn(st.x, c);  // as the forward pass took it
  const bool exact = needs_exact(st.x, M);
  float ga = 0.0f, gb = 0.0f;
  if (!zero) {
    if (a.g_lp) ga = __ldg(a.g_lp + t) * a.inv_temp;
    if (a.g_ent) gb = __ldg(a.g_ent + t) * a.inv_temp;
  }
  const float rs = st.y;  // 2^-log2(s) would carry log2's rounding, 7e-7 of p at 100000 logits
  const float A = -rs * fmaf(gb, fmaf(st.z, -kLn2, st.w), ga), B = -rs * gb * kLn2;
  // logits whose 2^y is 0 many times over count as this: A + B y stays finite
  const float floor_l = (M - 16384.0f) / c;
  const uint32_t low = Vec<L>::bound(floor_l);
  const int at_id = (int)id;
  auto element = [&](float l, int v) {
    float g;
    if (exact) {
      const float y = fmaxf((l - st.x) * c, -1000.0f);
      g = -rs * ex2(y) * fmaf(gb, fmaf(y - st.z, kLn2, st.w), ga) + (st.x - st.x);
    } else {
      const float y = fmaf(l < floor_l ? floor_l : l, c, -M);
      g = ex2(y) * fmaf(B, y, A);
    }
    return v == at_id ? g + ga : g;
  };
  const Span<L> sp(row, (int)a.V, 0, 1);
  if (((reinterpret_cast<uintptr_t>(row) ^ reinterpret_cast<uintptr_t>(grow)) & 15) != 0) {
    const ElementRange r = stretch_elements(a.V, at, stretches);
    for (auto v = r.first + tid; v < r.end; v += kTeam) Vec<L>::put(grow + v, zero ? 0.0f : element(Vec<L>::get(row + v), (int)v));
    return;
  }
  uint4* gvec = reinterpret_cast<uint4*>(grow + sp.head);
  const int lo = (int)(sp.hi * at / stretches), hi = (int)(sp.hi * (at + 1) / stretches);
  const float2 c2 = make_float2(c, c), M2 = make_float2(-M, -M);
  const float2 A2 = make_float2(A, A), B2 = make_float2(B, B);
  for (int v0 = lo + tid; v0 < hi; v0 += U * kTeam) {
    uint4 r[U];
#pragma unroll
    for (int i = 0; i < U; ++i) r[i] = v0 + i * kTeam < hi && !zero ? sp.vec()[v0 + i * kTeam] : make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int v = v0 + i * kTeam;
      if (v >= hi) break;
      const int e0 = sp.head + v * N;
      float x[N];
      if (zero) {
#pragma unroll
        for (int j = 0; j < N; ++j) x[j] = 0.0f;
      } else if (exact) {
        Vec<L>::unpack(r[i], x);
#pragma unroll
        for (int j = 0; j < N; ++j) x[j] = element(x[j], e0 + j);
      } else {
        Vec<L>::clamp(r[i], low);
        Vec<L>::unpack(r[i], x);
#pragma unroll
        for (int j = 0; j < N; j += 2) {
          const float2 y = __ffma2_rn(make_float2(x[j], x[j + 1]), c2, M2);
          const float2 g = __fmul2_rn(make_float2(ex2(y.x), ex2(y.y)), __ffma2_rn(B2, y, A2));
          x[j] = g.x;
          x[j + 1] = g.y;
        }
        if ((uint32_t)(at_id - e0) < (uint32_t)N) {
#pragma unroll
          for (int j = 0; j < N; ++j)
            if (e0 + j == at_id) x[j] += ga;
        }
      }
      gvec[v] = Vec<L>::pack(x);
    }
  }
  if (at == 0 && tid < sp.edge) {
    const int v = sp.edge_index(tid);
    Vec<L>::put(grow + v, zero ? 0.0f : element(Vec<L>::get(row + v), v));
  }
}

namespace {

// Blocks per row: one, or as many as it takes to give every SM two blocks, while a block keeps 4096
// logits to itself.
int row_parts(int64_t T, int64_t V, int num_sms) {
  int parts = 1;
  while (parts < 8 && T * parts < 2 * (int64_t)num_sms && V >= 8192 * (int64_t)parts) parts *= 2;
  return parts;
}

template <typename L, bool TOP>
cudaError_t launch_forward(const LogprobArgs& a, int num_sms, cudaStream_t st) {
  if (a.V <= kWarpRow) {
    logprobs_kernel<L, 1, TOP><<<(unsigned)((a.T + 7) / 8), 256, 0, st>>>(a, 1);
    return cudaGetLastError();
  }
  // Eight warps that meet for a short row wait for one another (us, two warps against eight: 2000 x 2000
  // bf16 5.1, 11.1; 4000 x 8000 19.6, 29.6; 2000 x 32000 27.7, 28.7); rows that do not fill the card with
  // eight each are done sooner so (20 x 8000 f32 5.0, 3.8; 300 x 16000 6.9, 5.4)
  if (a.V <= kPairRow && a.T >= 4 * (int64_t)num_sms) {
    logprobs_kernel<L, 2, TOP><<<(unsigned)a.T, 64, 0, st>>>(a, 1);
    return cudaGetLastError();
  }
  const int parts = row_parts(a.T, a.V, num_sms);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(a.T * parts));
  cfg.blockDim = dim3(256);
  cfg.stream = st;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = (unsigned)parts;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = parts > 1 ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, logprobs_kernel<L, 8, TOP>, a, parts);
}

template <typename L>
cudaError_t launch_backward(const LogprobBwdArgs& a, int num_sms, cudaStream_t st) {
  // a warp a row where a block would not fill its stretch and the rows fill the card (us, warp against
  // block: 4000 x 1500 bf16 5.1, 12.6; 4000 x 8000 21.3, 24.0; 300 x 3000 f32 5.1, 3.2)
  if (a.V <= kWarpRow || (a.V <= 8 * kWarpRow && a.T >= 8 * (int64_t)num_sms)) {
    logprobs_backward_kernel<L, 1><<<(unsigned)((a.T + 7) / 8), 256, 0, st>>>(a, 1);
    return cudaGetLastError();
  }
  const int64_t stretches = logprob_stretches(a.T, a.V, Vec<L>::N);
  logprobs_backward_kernel<L, 8><<<(unsigned)(a.T * stretches), 256, 0, st>>>(a, stretches);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_logprobs(const LogprobArgs& a, int num_sms, cudaStream_t st) {
  if (a.bf16)
    return a.k_top > 0 ? launch_forward<uint16_t, true>(a, num_sms, st) : launch_forward<uint16_t, false>(a, num_sms, st);
  return a.k_top > 0 ? launch_forward<float, true>(a, num_sms, st) : launch_forward<float, false>(a, num_sms, st);
}

cudaError_t launch_logprobs_backward(const LogprobBwdArgs& a, int num_sms, cudaStream_t st) {
  return a.bf16 ? launch_backward<uint16_t>(a, num_sms, st) : launch_backward<float>(a, num_sms, st);
}

}  // namespace nvfp4
