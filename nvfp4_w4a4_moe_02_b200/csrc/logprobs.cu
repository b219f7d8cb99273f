// Log probabilities of given tokens, with the entropy of the distribution and its top
// alternatives, and their gradient: the two sides of the rollout-trainer log-prob gap.
//
// With z = l / temperature over a row l of V logits, m = max l, c = log2(e) / temperature:
//   y_v = (l_v - m) c,  s = sum 2^y_v,  u = sum 2^y_v y_v        (one pass, running maximum)
//   logprob = (l_id - m) / temperature - ln s,  entropy = ln2 (log2 s - u / s)
//   d l_v = ( g_lp (1[v = id] - p_v) - g_H p_v (ln p_v + H) ) / temperature,  p_v = 2^(y_v - log2 s)
// The difference l - m is taken before the product with c: it is exact at the maximum, and a row
// held at the type's lowest value stays finite.  All sums and statistics are binary32.
#include "common.cuh"
#include "kernels.h"

namespace nvfp4 {

namespace {

constexpr float kLn2 = 0.6931471805599453f;
constexpr float kLog2e = 1.4426950408889634f;

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
  static __device__ __forceinline__ float get(const float* p) { return __ldg(p); }
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
  static __device__ __forceinline__ float get(const uint16_t* p) { return bf16_bits_to_f32(__ldg(p)); }
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

// Running statistics of a part of a row.  No element yet, or only -inf: m = -inf, s = u = 0.
// A NaN or +inf among the elements ends as s = NaN.
struct Stat {
  float m, s, u;
};

__device__ __forceinline__ Stat combine(const Stat& a, const Stat& b, float c) {
  Stat r;
  r.m = fmaxf(a.m, b.m);
  r.s = 0.0f;
  r.u = 0.0f;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const Stat& q = i ? b : a;
    if (q.m == -INFINITY) {
      r.s += q.s;  // 0, or NaN
    } else {
      const float d = (q.m - r.m) * c;
      const float f = ex2(d);
      r.s += f * q.s;
      // a part 2^-150 below the maximum adds nothing; its d times s could be -inf times 0
      if (f > 0.0f || !(d <= 0.0f)) r.u += f * (q.u + d * q.s);
    }
  }
  return r;
}

// Adds n elements to a part: one rescale per call, when its maximum rises.
template <int N>
__device__ __forceinline__ void add_elements(Stat& a, const float* x, float c) {
  float bm = x[0];
#pragma unroll
  for (int i = 1; i < N; ++i) bm = fmaxf(bm, x[i]);  // skips NaN
  if (!(bm <= a.m)) {
    if (a.m > -INFINITY) {
      const float d = (a.m - bm) * c;
      const float f = ex2(d);
      a.u = f > 0.0f ? f * (a.u + d * a.s) : 0.0f;
      a.s *= f;
    }
    a.m = fmaxf(a.m, bm);
  }
  if (a.m == -INFINITY) {
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (x[i] != x[i]) a.s = x[i];
    return;
  }
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const float y = (x[i] - a.m) * c;
    const float e = ex2(y);
    a.s += e;
    a.u = fmaf(e, fmaxf(y, -1000.0f), a.u);  // -inf: e = 0 times a finite number
  }
  // fmaxf drops a NaN, but s keeps it
}

// Order of the alternatives: value descending, index ascending, as one unsigned key (0 = none).
__device__ __forceinline__ uint64_t order_key(float v, uint32_t idx) {
  const uint32_t b = __float_as_uint(v + 0.0f);  // -0 ties with +0
  const uint32_t k = (b & 0x80000000u) ? ~b : (b | 0x80000000u);
  return ((uint64_t)k << 32) | (0xFFFFFFFFu - idx);
}
__device__ __forceinline__ float key_value(uint64_t key) {
  const uint32_t k = (uint32_t)(key >> 32);
  return __uint_as_float((k & 0x80000000u) ? (k & 0x7FFFFFFFu) : ~k);
}
__device__ __forceinline__ int32_t key_index(uint64_t key) { return (int32_t)(0xFFFFFFFFu - (uint32_t)key); }

// A warp's best 32 keys, lane i holding the i-th; thr is the k-th.
__device__ __forceinline__ void insert_key(uint64_t& mine, uint64_t& thr, uint64_t key, int k) {
  const int lane = threadIdx.x & 31;
  const int pos = __popc(__ballot_sync(0xffffffffu, mine > key));
  const uint64_t up = __shfl_up_sync(0xffffffffu, mine, 1);
  if (lane == pos) mine = key;
  if (lane > pos) mine = up;
  thr = __shfl_sync(0xffffffffu, mine, k - 1);
}

template <int N>
__device__ __forceinline__ void offer(uint64_t& mine, uint64_t& thr, const float* x, uint32_t idx0, int n, int k) {
  // one key per lane first: its largest element stands for the others
  uint64_t best = 0;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const uint64_t q = i < n ? order_key(x[i], idx0 + i) : 0;
    best = q > best ? q : best;
  }
  uint32_t mask = __ballot_sync(0xffffffffu, best > thr);
  while (mask) {
    const int src = __ffs(mask) - 1;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const uint64_t q = __shfl_sync(0xffffffffu, i < n ? order_key(x[i], idx0 + i) : 0ull, src);
      if (q > thr) insert_key(mine, thr, q, k);
    }
    mask &= __ballot_sync(0xffffffffu, best > thr) & ~((2u << src) - 1u);
  }
}

// Two descending lists -> their best 32, descending: the element-wise maximum of one and the other
// reversed is bitonic and holds them; five exchanges sort it.
__device__ __forceinline__ uint64_t merge_lists(uint64_t a, uint64_t b) {
  const int lane = threadIdx.x & 31;
  const uint64_t r = __shfl_xor_sync(0xffffffffu, b, 31);
  uint64_t v = a > r ? a : r;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const uint64_t w = __shfl_xor_sync(0xffffffffu, v, o);
    const bool keep_max = (lane & o) == 0;
    v = keep_max == (v > w) ? v : w;
  }
  return v;
}

__device__ __forceinline__ int64_t read_id(const void* ids, int id_bytes, int64_t t) {
  return id_bytes == 8 ? __ldg(reinterpret_cast<const long long*>(ids) + t)
                       : (int64_t)__ldg(reinterpret_cast<const int*>(ids) + t);
}

}  // namespace

// One row per team of W warps; a block holds one team (W > 1) or eight one-warp teams.
template <typename L, int W, bool TOP>
__global__ void __launch_bounds__(W > 1 ? W * 32 : 256) logprobs_kernel(LogprobArgs a) {
  constexpr int N = Vec<L>::N;
  constexpr int kTeam = W * 32;
  __shared__ Stat part[W];
  __shared__ uint64_t lists[TOP ? W : 1][32];
  const int lane = threadIdx.x & 31;
  const int tid = W > 1 ? threadIdx.x : lane;
  const int warp = W > 1 ? threadIdx.x >> 5 : 0;
  const int64_t t = W > 1 ? blockIdx.x : (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  if (t >= a.T) return;
  const int k = a.k_top;
  int64_t id = read_id(a.ids, a.id_bytes, t);
  if (id >= a.V) {
    if (tid == 0) report_status(a.status, kErrInvalid);
    id = -1;
  }
  if (id < 0) {  // padding: the row is not read
    if (tid == 0) {
      a.logprob[t] = 0.0f;
      if (a.entropy) a.entropy[t] = 0.0f;
      if (a.stats) reinterpret_cast<float4*>(a.stats)[t] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    }
    if (TOP && tid < k) {
      a.top_ids[t * k + tid] = -1;
      a.top_lp[t * k + tid] = 0.0f;
    }
    return;
  }
  const float c = a.inv_temp * kLog2e;
  const L* row = reinterpret_cast<const L*>(a.logits) + t * a.ld;
  const int64_t V = a.V;

  Stat st{-INFINITY, 0.0f, 0.0f};
  uint64_t mine = 0, thr = 0;
  // the elements before the first 16-byte boundary and those after the last one go one by one
  const int64_t head = min(V, (int64_t)((16 - (reinterpret_cast<uintptr_t>(row) & 15)) & 15) / (int64_t)sizeof(L));
  const int64_t nvec = (V - head) / N;
  const int64_t tail0 = head + nvec * N;
  const int edge = (int)(head + (V - tail0));
  {
    float x = -INFINITY;
    const int64_t v = lane < head ? lane : tail0 + (lane - head);
    const bool has = warp == 0 && lane < edge;
    if (has) {
      x = Vec<L>::get(row + v);
      add_elements<1>(st, &x, c);
    }
    if (TOP && warp == 0) offer<1>(mine, thr, &x, (uint32_t)v, has ? 1 : 0, k);
  }
  const uint4* vrow = reinterpret_cast<const uint4*>(row + head);
  constexpr int U = 4;
  for (int64_t v0 = 0; v0 < nvec; v0 += kTeam * U) {
    uint4 r[U];
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int64_t v = v0 + i * kTeam + tid;
      if (v < nvec) r[i] = __ldg(vrow + v);
    }
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int64_t v = v0 + i * kTeam + tid;
      const bool has = v < nvec;
      float x[N];
      if (has) {
        Vec<L>::unpack(r[i], x);
        add_elements<N>(st, x, c);
      }
      if (TOP) offer<N>(mine, thr, x, (uint32_t)(head + v * N), has ? N : 0, k);
    }
  }
  // join the lanes, then the warps
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    Stat q;
    q.m = __shfl_xor_sync(0xffffffffu, st.m, o);
    q.s = __shfl_xor_sync(0xffffffffu, st.s, o);
    q.u = __shfl_xor_sync(0xffffffffu, st.u, o);
    // the same order of the two in both lanes: the sums come out equal
    st = (lane & o) ? combine(q, st, c) : combine(st, q, c);
  }
  if (W > 1) {
    if (lane == 0) part[warp] = st;
    if (TOP) lists[warp][lane] = mine;
    __syncthreads();
    if (warp != 0) return;
    st = part[0];
    for (int w = 1; w < W; ++w) st = combine(st, part[w], c);
    if (TOP)
      for (int w = 1; w < W; ++w) mine = merge_lists(mine, lists[w][lane]);
  }
  const bool empty = st.m == -INFINITY && st.s == 0.0f;  // every logit is -inf: no distribution
  const float ls = empty ? 0.0f : log2f(st.s);
  if (lane == 0) {
    if (!empty && !(st.s < INFINITY)) report_status(a.status, kErrRange);
    // in nats from here: a finite log prob near the type's lowest value does not overflow on the way
    const float y = (Vec<L>::get(row + id) - st.m) * a.inv_temp;
    const float h = empty ? 0.0f : fmaxf((ls - st.u / st.s) * kLn2, 0.0f) + (st.s - st.s);
    a.logprob[t] = empty ? -INFINITY : fmaf(ls, -kLn2, y);
    if (a.entropy) a.entropy[t] = h;
    // m = -inf marks the row without a distribution: its gradient is zero
    const float m = !empty && st.m == -INFINITY ? st.s : st.m;
    if (a.stats) reinterpret_cast<float4*>(a.stats)[t] = make_float4(m, ls, h, 0.0f);
  }
  if (TOP && lane < k) {
    a.top_ids[t * k + lane] = key_index(mine);
    a.top_lp[t * k + lane] = empty ? -INFINITY : fmaf(ls, -kLn2, (key_value(mine) - st.m) * a.inv_temp);
  }
}

// dlogits of one stretch of a row; 16-byte loads where the row allows, 16-byte stores where the
// gradient's row has the same phase.
template <typename L>
__global__ void __launch_bounds__(256) logprobs_backward_kernel(LogprobBwdArgs a) {
  constexpr int N = Vec<L>::N;
  const int64_t t = blockIdx.x;
  const L* row = reinterpret_cast<const L*>(a.logits) + t * a.ld;
  L* grow = reinterpret_cast<L*>(a.grad) + t * a.ldg;
  int64_t id = read_id(a.ids, a.id_bytes, t);
  if (id >= a.V) {
    if (threadIdx.x == 0) report_status(a.status, kErrInvalid);
    id = -1;
  }
  const float4 stt = __ldg(reinterpret_cast<const float4*>(a.stats) + t);
  const float c = a.inv_temp * kLog2e;
  float ga = 0.0f, gb = 0.0f;
  const bool zero = id < 0 || stt.x == -INFINITY;
  if (!zero) {
    if (a.g_lp) ga = __ldg(a.g_lp + t) * a.inv_temp;
    if (a.g_ent) gb = __ldg(a.g_ent + t) * a.inv_temp;
  }
  auto grad = [&](float l, int64_t v) {
    const float q = fmaxf((l - stt.x) * c - stt.y, -1000.0f);  // log2 p; p = 0 below
    const float p = ex2(q);
    const float w = fmaf(gb, fmaf(q, kLn2, stt.z), ga);
    return (v == id ? ga : 0.0f) - p * w;
  };
  for (int64_t v = threadIdx.x; v < a.V; v += 256)
    Vec<L>::put(grow + v, zero ? 0.0f : grad(Vec<L>::get(row + v), v));
  (void)N;
}

cudaError_t launch_logprobs(const LogprobArgs& a, int num_sms, cudaStream_t st) {
  (void)num_sms;
#define NVFP4_LP(L, W, TOP) logprobs_kernel<L, W, TOP><<<(unsigned)(W > 1 ? a.T : (a.T + 7) / 8), W > 1 ? W * 32 : 256, 0, st>>>(a)
#define NVFP4_LP_W(L)                                                     \
  do {                                                                    \
    if (a.V <= 1024) {                                                    \
      if (a.k_top > 0) NVFP4_LP(L, 1, true); else NVFP4_LP(L, 1, false);  \
    } else {                                                              \
      if (a.k_top > 0) NVFP4_LP(L, 8, true); else NVFP4_LP(L, 8, false);  \
    }                                                                     \
  } while (0)
  if (a.bf16)
    NVFP4_LP_W(uint16_t);
  else
    NVFP4_LP_W(float);
#undef NVFP4_LP_W
#undef NVFP4_LP
  return cudaGetLastError();
}

cudaError_t launch_logprobs_backward(const LogprobBwdArgs& a, int num_sms, cudaStream_t st) {
  (void)num_sms;
  if (a.bf16)
    logprobs_backward_kernel<uint16_t><<<(unsigned)a.T, 256, 0, st>>>(a);
  else
    logprobs_backward_kernel<float><<<(unsigned)a.T, 256, 0, st>>>(a);
  return cudaGetLastError();
}

}  // namespace nvfp4
