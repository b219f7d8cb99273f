// A whole mixture-of-experts layer for a few tokens in four kernels: routing and layout, gate_up with
// SwiGLU, down, and the weighted combine.  Activations stay bf16 (the trainer's side of
// the method: weights fake-quantised, activations not), weights are the packed NVFP4 ones.
//
//   ids_t, w_t = the k largest logits of token t and their renormalised softmax
//   h_tj = silu(G_e x_t) * (U_e x_t),  out_t = sum_j w_tj D_e h_tj,   e = ids_tj
//
// The weights of the experts that are touched bound it.  Up to eight tokens of one expert make a slot;
// a unit of work is a slot times four 16-row tiles of the expert's matrix, streamed by one warp (or by
// S warps that split K, where there are few units) through a ring in shared memory and decoded into the
// A operand of mma.m16n8k16 (f16, binary32 sums); the slot's tokens are the eight columns.
//   - E2M1 x E4M3 has at most six significant bits and lies in [2^-10, 2688]: exact in f16.
//   - The sum over k may take its elements in any order, so a lane keeps the 32 consecutive codes
//     of its 16-byte load: instruction i of a chunk contracts elements 4i .. 4i+3 of every lane.
//   - The activations lie in that order: of each 128, element 32 t + 8 i + e at 32 i + 8 t + e, so that a copy
//     by a quad takes 64 bytes together (64 tokens in each of 4 experts: 73.1 -> 70.7 us).
//   - Activations are f16 with a power of two per token and stretch that brings the stretch's largest
//     to [2^14, 2^15): x per 128 elements, which keeps every bf16 down to 2^-31 of the largest exact;
//     h, kept with 11 bits (an eighth of the output's own rounding; binary32 would be three f16 products
//     in the place of one), per 32.  The powers are taken out of a chunk's sum; where those of h lie far
//     apart, the chunk takes a product for each magnitude.
//   - A scale atom's 16 bytes j hold the scales of rows j, 32 + j, 64 + j, 96 + j of its 128.  Tiles go in
//     pairs over eight j: the first takes rows j and 64 + j, the second rows 32 + j and 96 + j, so that one
//     16-byte load brings a lane the scales of both tiles.  In the gate/up interleaved pack rows 0 .. 63
//     are gate rows and 64 .. 127 the matching up rows, which land in one lane.
//   - The ring is filled by asynchronous copies, three steps ahead: a warp has six scoreboards for its
//     loads, and a ring in registers waits for its youngest load with its oldest (measured: 3.6 TB/s
//     without any arithmetic, at any depth).
#include <atomic>
#include <type_traits>

#include "common.cuh"
#include "kernels.h"
#include "moe_few_split.h"

namespace nvfp4 {

namespace {

constexpr int kSlot = 8;                        // tokens of a slot
constexpr int kWarps = kFewWarps;               // warps of a block, one block a SM
constexpr int kTiles = 4;                       // 16-row tiles of a unit: two pairs
constexpr int kSteps = 3;                       // depth of the ring; a step is a pair's 128 columns
constexpr int kStepBytes = 4 * 512 + 256;       // codes: [4][32 lanes] x 16 bytes, scales: [16] x 16 bytes
constexpr int kActBytes = 4 * 512 + 256;        // activations of a chunk: [4][32] x 16 bytes, scales [32] x 8
constexpr int kWarpBytes = kSteps * kStepBytes + 2 * kActBytes;
constexpr int kRedBytes = kTiles * 512;         // a warp's sums, for the warps that split K with it
constexpr int kRingBytes = kWarps * (kWarpBytes + kRedBytes);

// Workspace words: [0] slots n; a word per slot from kListHead on (expert, first pair << 10, count << 21);
// token of each pair in slot order (bytes); place in slot order of pair t * k + j (-1: none).
constexpr int kListHead = 16;
__host__ __device__ inline int token_words(int P) { return (P + 3) / 4; }
__host__ __device__ inline int list_tokens(int P) { return kListHead + P; }
__host__ __device__ inline int list_places(int P) { return list_tokens(P) + token_words(P); }
__host__ __device__ inline int list_words(int P) { return list_places(P) + P; }

__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma16816_first(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                               uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
}

// Asynchronous copies of 16, 8 or 4 bytes to smem + OFF; weights past L1, activations through it.
template <int OFF>
__device__ __forceinline__ void copy16_stream(uint32_t smem, const void* gmem) {
  asm volatile("cp.async.cg.shared.global [%0 + %2], [%1], 16;" ::"r"(smem), "l"(gmem), "n"(OFF) : "memory");
}
template <int OFF, int BYTES>
__device__ __forceinline__ void copy_act(uint32_t smem, const void* gmem) {
  asm volatile("cp.async.ca.shared.global [%0 + %2], [%1], %3;" ::"r"(smem), "l"(gmem), "n"(OFF), "n"(BYTES) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
template <int OFF>
__device__ __forceinline__ uint4 lds16(uint32_t smem) {
  uint4 r;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4 + %5];"
               : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
               : "r"(smem), "n"(OFF)
               : "memory");
  return r;
}
template <int OFF>
__device__ __forceinline__ float2 lds8(uint32_t smem) {
  float2 r;
  asm volatile("ld.shared.v2.f32 {%0,%1}, [%2 + %3];" : "=f"(r.x), "=f"(r.y) : "r"(smem), "n"(OFF) : "memory");
  return r;
}

__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
  const __half2 r = __hmul2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ uint32_t pack_f16(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

__device__ __forceinline__ void load_b(uint32_t (&b)[16], const uint4& p, const uint4& q, const uint4& r, const uint4& s) {
  const uint4 v[4] = {p, q, r, s};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    b[4 * i] = v[i].x;
    b[4 * i + 1] = v[i].y;
    b[4 * i + 2] = v[i].z;
    b[4 * i + 3] = v[i].w;
  }
}

// The byte `I` of a word of codes -> two halves.  The conversion reads its register's low byte.
template <int I>
__device__ __forceinline__ uint32_t decode_byte(uint32_t w) {
  uint32_t r;
  asm("{\n\t.reg .b8 t;\n\t"
      "cvt.u8.u32 t, %1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, t;\n\t}"
      : "=r"(r)
      : "r"(w >> (8 * I)));
  return r;
}
__device__ __forceinline__ uint32_t scale_low(uint32_t a, __half2 s) {
  const __half2 r = __hmul2(*reinterpret_cast<const __half2*>(&a), __low2half2(s));
  return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ uint32_t scale_high(uint32_t a, __half2 s) {
  const __half2 r = __hmul2(*reinterpret_cast<const __half2*>(&a), __high2half2(s));
  return *reinterpret_cast<const uint32_t*>(&r);
}
// The scales of the lane's two 16-blocks among the four of a word.
__device__ __forceinline__ __half2 lane_scales(uint32_t w) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"((uint16_t)(w >> (16 * (threadIdx.x & 1)))));
  return *reinterpret_cast<const __half2*>(&r);
}

// acc += d x (16 x 128 codes of a tile) x (B fragments b of the same 128 elements): lo, hi are the
// lane's 32 codes of its low and high row, d0, d1 the scales taken out of the lane's two columns.
__device__ __forceinline__ void mma_tile(float (&acc)[4], const uint4& klo, const uint4& khi, uint32_t sf_lo,
                                         uint32_t sf_hi, const uint32_t (&b)[16], float d0, float d1) {
  const __half2 sl = lane_scales(sf_lo), sh = lane_scales(sf_hi);
  const uint32_t lo[4] = {klo.x, klo.y, klo.z, klo.w}, hi[4] = {khi.x, khi.y, khi.z, khi.w};
  float part[4];
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    // a word is 8 codes: the first two words belong to the lane's first 16-block
    auto sc = [&](uint32_t a, __half2 s) { return w < 2 ? scale_low(a, s) : scale_high(a, s); };
    const uint32_t a0 = sc(decode_byte<0>(lo[w]), sl), a1 = sc(decode_byte<0>(hi[w]), sh);
    const uint32_t a2 = sc(decode_byte<1>(lo[w]), sl), a3 = sc(decode_byte<1>(hi[w]), sh);
    if (w == 0)
      mma16816_first(part, a0, a1, a2, a3, b[0], b[1]);
    else
      mma16816(part, a0, a1, a2, a3, b[4 * w], b[4 * w + 1]);
    mma16816(part, sc(decode_byte<2>(lo[w]), sl), sc(decode_byte<2>(hi[w]), sh), sc(decode_byte<3>(lo[w]), sl),
             sc(decode_byte<3>(hi[w]), sh), b[4 * w + 2], b[4 * w + 3]);
  }
  acc[0] = fmaf(part[0], d0, acc[0]);
  acc[1] = fmaf(part[1], d1, acc[1]);
  acc[2] = fmaf(part[2], d0, acc[2]);
  acc[3] = fmaf(part[3], d1, acc[3]);
}

// The same for one or two tokens, without scaling the codes: the lane's column holds token g % 2 for lanes
// t = g / 2 of the quad and zero for the others, so that a lane's sums c0 .. c3 are those of its own 16
// codes per row, one scale block, for either token, and take the block's scale as sums.  acc: the lane's
// low row for the tokens 0, 1, then its high row, over its own codes only; d0, d1: the scales taken out of
// the tokens' elements (first and second 16).  4 products on halves instead of 32.
__device__ __forceinline__ void mma_tile_blocks(float (&acc)[4], const uint4& klo, const uint4& khi, uint32_t sf_lo,
                                                uint32_t sf_hi, const uint32_t (&b)[16], float2 d0, float2 d1) {
  const float2 sl = __half22float2(lane_scales(sf_lo)), sh = __half22float2(lane_scales(sf_hi));
  const uint32_t lo[4] = {klo.x, klo.y, klo.z, klo.w}, hi[4] = {khi.x, khi.y, khi.z, khi.w};
#pragma unroll
  for (int blk = 0; blk < 2; ++blk) {
    float part[4];
#pragma unroll
    for (int w = 2 * blk; w < 2 * blk + 2; ++w) {
      const uint32_t a0 = decode_byte<0>(lo[w]), a1 = decode_byte<0>(hi[w]);
      const uint32_t a2 = decode_byte<1>(lo[w]), a3 = decode_byte<1>(hi[w]);
      if (w == 2 * blk)
        mma16816_first(part, a0, a1, a2, a3, b[4 * w], b[4 * w + 1]);
      else
        mma16816(part, a0, a1, a2, a3, b[4 * w], b[4 * w + 1]);
      mma16816(part, decode_byte<2>(lo[w]), decode_byte<2>(hi[w]), decode_byte<3>(lo[w]), decode_byte<3>(hi[w]),
               b[4 * w + 2], b[4 * w + 3]);
    }
    const float l = blk ? sl.y : sl.x, h = blk ? sh.y : sh.x;
    const float e0 = blk ? d0.y : d0.x, e1 = blk ? d1.y : d1.x;
    acc[0] = fmaf(part[0], l * e0, acc[0]);
    acc[1] = fmaf(part[1], l * e1, acc[1]);
    acc[2] = fmaf(part[2], h * e0, acc[2]);
    acc[3] = fmaf(part[3], h * e1, acc[3]);
  }
}

// The power of two that brings a magnitude of binary32 exponent field e to [2^14, 2^15), and its
// inverse times 2^-12: sums of weights in units of their tensor scale are up to 2^12 times the
// result's size, and would overflow first.  2^12 comes back with the tensor scale.  Below 2^-100 the
// largest power is taken; an infinity or NaN counts as 2^127.
constexpr float kSumUnit = 4096.0f;
__device__ __forceinline__ void stretch_scale(int e, float* up, float* down) {
  e = min(max(e, 27), 254);
  *up = __uint_as_float((uint32_t)(268 - e) << 23);
  *down = __uint_as_float((uint32_t)(e - 26) << 23);
}

// Stretches of a chunk whose scale is not below kNear of the largest are brought to it by an f16 quotient; the
// others go in further products of their own, so that an element keeps its 11 bits down to 2^-15 of the largest
// of its 32.  (Replayed, every chunk with one block far below, or three magnitudes apart: 64 tokens in each of
// 4 experts of hidden 4096 69.5 -> 84.8 us, 48 skewed of 2048 69.7 -> 81.9; ordinary calls as before, to 0.6 %.)
constexpr float kNear = 1.220703125e-4f;  // 2^-13
// The largest scale of a column's chunk, from the two of each lane of the quad.
__device__ __forceinline__ float quad_max(float2 f) {
  float d = fmaxf(f.x, f.y);
  d = fmaxf(d, __shfl_xor_sync(0xffffffffu, d, 1));
  return fmaxf(d, __shfl_xor_sync(0xffffffffu, d, 2));
}

// The kernels of a call overlap their launches: a kernel lets the next one start early, and that
// one waits for its results.  Every thread waits before it returns, so that a kernel's end means the
// end of those before it.
__device__ __forceinline__ void let_next_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void wait_for_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// ----------------------------------------------------------------------------------------
// routing and layout
// ----------------------------------------------------------------------------------------
struct ListScratch {
  alignas(16) uint16_t id[kFewMaxPairs];  // expert of pair t * k + j (0xFFFF: none)
  int cursor[kMaxRouteExperts];
};

// The same choice and weights as moe_route_topk: k rounds of a warp arg-max over ordered keys.
__device__ void route_token(const MoeFewArgs& a, int t, uint16_t* id) {
  const int lane = threadIdx.x & 31;
  const int nb = (a.E + 255) / 256;
  uint32_t key[8];
  uint32_t taken[4] = {0, 0, 0, 0};  // bit i of word b: the lane's element i of block b is chosen
  auto load = [&](int b) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int e = 256 * b + 32 * i + lane;
      key[i] = 0;
      if (e < a.E && !((taken[b] >> i) & 1u)) {
        const uint32_t u = __float_as_uint(__ldg(a.logits + (int64_t)t * a.E + e) + 0.0f);
        key[i] = (u & 0x7FFFFFFFu) >= 0x7F800000u ? 0xFFFFFFFFu : (u & 0x80000000u) ? ~u : (u | 0x80000000u);
      }
    }
  };
  load(0);
  uint32_t mine_key = 0;  // lane j keeps the j-th choice
  int mine_e = -1;
  bool bad = false;
  for (int j = 0; j < a.k; ++j) {
    uint32_t best = 0;
    int be = 0x7FFFFFFF;
    for (int b = 0; b < nb; ++b) {
      if (nb > 1) load(b);
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (key[i] > best) {
          best = key[i];
          be = 256 * b + 32 * i + lane;
        }
    }
    const uint32_t top = __reduce_max_sync(0xffffffffu, best);
    if (top == 0xFFFFFFFFu) {  // an infinity or NaN sorts first
      bad = true;
      break;
    }
    const uint32_t have = __ballot_sync(0xffffffffu, best == top);
    int e = __shfl_sync(0xffffffffu, be, __ffs(have) - 1);
    if (have & (have - 1)) e = (int)__reduce_min_sync(0xffffffffu, best == top ? (uint32_t)be : 0x7FFFFFFFu);
    if ((e & 31) == lane) {
      const int i = (e >> 5) & 7;
      if (nb > 1) {
#pragma unroll
        for (int b = 0; b < 4; ++b)
          if (b == e >> 8) taken[b] |= 1u << i;
      } else {
#pragma unroll
        for (int q = 0; q < 8; ++q)
          if (q == i) key[q] = 0;
      }
    }
    if (lane == j) {
      mine_key = top;
      mine_e = e;
    }
  }
  const float l = __uint_as_float((mine_key & 0x80000000u) ? (mine_key & 0x7FFFFFFFu) : ~mine_key);
  const float p = expf(__fsub_rn(l, __shfl_sync(0xffffffffu, l, 0)));
  float sum = 0.0f;
  for (int j = 0; j < a.k; ++j) sum = __fadd_rn(sum, __shfl_sync(0xffffffffu, p, j));
  if (lane < a.k) {
    const int i = t * a.k + lane;
    id[i] = bad ? 0xFFFFu : (uint16_t)mine_e;
    a.ids[i] = bad ? -1 : mine_e;
    a.topk_w[i] = bad ? 0.0f : __fdiv_rn(p, sum);
  }
  if (bad && lane == 0) report_status(a.status, kErrRange);
}

__device__ __forceinline__ uint32_t slot_word(int e, int first, int count) {
  return (uint32_t)e | (uint32_t)first << 10 | (uint32_t)count << 21;
}

__device__ void build_lists(const MoeFewArgs& a, ListScratch& B) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int P = a.T * a.k;
  uint32_t* slots = reinterpret_cast<uint32_t*>(a.lists + kListHead);
  uint8_t* token = reinterpret_cast<uint8_t*>(a.lists + list_tokens(P));
  int32_t* places = a.lists + list_places(P);
  if (P > 32)
    for (int e = threadIdx.x; e < a.E; e += blockDim.x) B.cursor[e] = 0;
  for (int t = warp; t < a.T; t += blockDim.x / 32) route_token(a, t, B.id);
  __syncthreads();
  if (P <= 32) {
    // one warp sorts the pairs by expert: a pair's place is the number of those before it
    if (warp != 0) return;
    const uint32_t e = lane < P ? B.id[lane] : 0xFFFFu;
    int place = 0, rank = 0;
    for (int j = 0; j < P; ++j) {
      const uint32_t ej = __shfl_sync(0xffffffffu, e, j);
      const bool before = ej == e && j < lane;
      rank += before;
      place += before || ej < e;
    }
    const int cnt = __popc(__match_any_sync(0xffffffffu, e));
    if (e != 0xFFFFu) token[place] = (uint8_t)(lane / a.k);
    if (lane < P) places[lane] = e != 0xFFFFu ? place : -1;
    // slots in the order of places: a slot's first pair has a rank that is a multiple of its size
    const bool first = e != 0xFFFFu && rank % kSlot == 0;
    int i = 0;
    for (int j = 0; j < P; ++j) i += __shfl_sync(0xffffffffu, first ? place : 64, j) < place;
    if (first) slots[i] = slot_word((int)e, place, min(kSlot, cnt - rank));
    const int n = __popc(__ballot_sync(0xffffffffu, first));
    if (lane == 0) a.lists[0] = n;
    return;
  }
  for (int p = threadIdx.x; p < P; p += blockDim.x)
    if (B.id[p] != 0xFFFFu) atomicAdd(&B.cursor[B.id[p]], 1);
  __syncthreads();
  if (warp == 0) {
    int n = 0, at = 0;  // slots and pairs before this group of experts
    for (int e0 = 0; e0 < a.E; e0 += 32) {
      const int e = e0 + lane;
      const int cnt = e < a.E ? B.cursor[e] : 0;
      if (__ballot_sync(0xffffffffu, cnt > 0) == 0) continue;
      int run = cnt | (cnt + kSlot - 1) / kSlot << 16;  // pairs low, slots high
      const int own = run;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, run, o);
        if (lane >= o) run += v;
      }
      const int first = at + ((run - own) & 0xFFFF);
      int i = n + ((run - own) >> 16);
      for (int c = 0; c < cnt; c += kSlot, ++i) slots[i] = slot_word(e, first + c, min(kSlot, cnt - c));
      if (cnt > 0) B.cursor[e] = first;
      const int all = __shfl_sync(0xffffffffu, run, 31);
      at += all & 0xFFFF;
      n += all >> 16;
    }
    if (lane == 0) a.lists[0] = n;
  }
  __syncthreads();
  // a pair's place: its expert's first, and the pairs of that expert before it (eight ids a read)
  for (int p = threadIdx.x; p < P; p += blockDim.x) {
    const uint32_t e = B.id[p], e2 = e | e << 16;
    int place = -1;
    if (e != 0xFFFFu) {
      int twice = 0;
      for (int q = 0; q < p >> 3; ++q) {
        const uint4 v = reinterpret_cast<const uint4*>(B.id)[q];
        twice += __popc(__vcmpeq2(v.x, e2)) + __popc(__vcmpeq2(v.y, e2)) + __popc(__vcmpeq2(v.z, e2)) +
                 __popc(__vcmpeq2(v.w, e2));
      }
      place = B.cursor[e] + (twice >> 4);  // sixteen bits a match
      for (int q = p & ~7; q < p; ++q) place += B.id[q] == e;
      token[place] = (uint8_t)(p / a.k);
    }
    places[p] = place;
  }
}

}  // namespace

// The last block routes and lays out the slots; block t converts row t of x to f16, a warp per chunk.
__global__ void __launch_bounds__(1024) moe_few_prepare_kernel(MoeFewArgs a) {
  __shared__ ListScratch scratch;
  let_next_start();
  if ((int)blockIdx.x == a.T) {
    build_lists(a, scratch);
    return;
  }
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t t = blockIdx.x;
  for (int c = warp; c < a.H / 128; c += 32) {
    const uint2 r = __ldg(reinterpret_cast<const uint2*>(a.x + t * a.ldx + 128 * c) + lane);
    const uint32_t m2 = __vmaxu2(r.x & 0x7FFF7FFFu, r.y & 0x7FFF7FFFu);
    const uint32_t m = __reduce_max_sync(0xffffffffu, max(m2 & 0xFFFFu, m2 >> 16));
    float up, down;
    stretch_scale((int)(m >> 7), &up, &down);
    uint2 o;
    o.x = pack_f16(__uint_as_float(r.x << 16) * up, __uint_as_float(r.x & 0xFFFF0000u) * up);
    o.y = pack_f16(__uint_as_float(r.y << 16) * up, __uint_as_float(r.y & 0xFFFF0000u) * up);
    reinterpret_cast<uint2*>(a.xh + t * a.H + 128 * c)[8 * (lane >> 1 & 3) + 2 * (lane >> 3) + (lane & 1)] = o;
    if (lane == 0) a.x_scale[t * (a.H / 128) + c] = down;
  }
}

// UP: gate_up + SwiGLU -> h.  Otherwise down: the products of each slot, in binary32, -> y.
//
// Units are split evenly over the teams of S warps, in one contiguous run each, slots outermost; a team's
// warps take every S-th chunk and join in shared memory.  S is the power of two that leaves the busiest warp
// the fewest chunks, a join counted as one; the least of equals.  (Against the least S that gives three quarters
// of the warps a unit, us replayed from a graph: 32 tokens, hidden 2048, 2 of 16 experts 32.0 -> 27.2; 64 tokens, 8 of 128
// 117.5 -> 109.1; one token, 8 of 128 21.5 -> 20.5; 64 tokens, hidden 7168, 8 of 256 1100 -> 1086; the smallest
// calls 13.9 -> 14.0.)
template <bool UP>
__global__ void __launch_bounds__(kWarps * 32, 1) moe_few_stream_kernel(MoeFewArgs a) {
  extern __shared__ __align__(128) uint8_t smem[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
  const int P = a.T * a.k;
  const int cols = UP ? a.H : a.I;                          // of the matrix
  const int groups = UP ? a.I / 32 : a.H / 64;              // units per slot
  const int nch = (cols + 127) / 128;
  const int64_t cb = (int64_t)a.H * a.I / (UP ? 1 : 2), sb = cb / 8;  // bytes of one expert's codes / scales
  const uint8_t* codes = UP ? a.gu_codes : a.dn_codes;
  const uint8_t* sfs = UP ? a.gu_sf : a.dn_sf;
  const float* s_gs = UP ? a.gu_sg : a.dn_sg;

  // gate_up lets down start once the lists are complete, so that down can read them, and fill its ring with
  // weights, while gate_up's last blocks run; h it reads after its wait (us replayed, one token of hidden
  // 7168 59.8 -> 58.0, seven of 2048 46.3 -> 44.2; the smallest 14.1 -> 14.4, for gate_up lets go later)
  if (UP) wait_for_previous();
  let_next_start();
  uint32_t* slots = reinterpret_cast<uint32_t*>(smem + kRingBytes);
  uint8_t* token = reinterpret_cast<uint8_t*>(slots + P);
  const int n = __ldcg(a.lists);
  for (int i = threadIdx.x; i < P; i += kWarps * 32) slots[i] = (uint32_t)__ldcg(a.lists + kListHead + i);
  if (UP)
    for (int i = threadIdx.x; i < token_words(P); i += kWarps * 32)
      reinterpret_cast<uint32_t*>(token)[i] = (uint32_t)__ldcg(a.lists + list_tokens(P) + i);
  __syncthreads();

  const int units = n * groups;
  const int warps = gridDim.x * kWarps;
  const uint32_t rank = few_split_cost(lane, units, warps, nch);  // lane i weighs S = 2^i
  const int S = 1 << (__reduce_min_sync(0xffffffffu, rank) & 7u);
  const int team = (blockIdx.x * kWarps + warp) / S, teams = warps / S, part = warp & (S - 1);
  int u = (int)((int64_t)units * team / teams);
  const int u_end = (int)((int64_t)units * (team + 1) / teams);
  if (u >= u_end) {  // a team's warps agree
    if (!UP) wait_for_previous();
    return;
  }

  const uint32_t base = (uint32_t)__cvta_generic_to_shared(smem) + warp * kWarpBytes;
  const uint32_t acts = base + kSteps * kStepBytes;
  const int my_chunks = (nch - part + S - 1) / S;  // at least one: S <= nch

  // ---- the copying side, kSteps steps ahead
  const int64_t row32 = 16 * (int64_t)cols;  // bytes of 32 rows
  const uint32_t sf_to = 2048 + 32 * g + 8 * t - 16 * lane;
  int cu = u, cc = 0;             // unit, chunk (of this warp's)
  uint32_t cstep = base + 16 * lane, cact = acts + 16 * lane;  // the lane's places in the ring
  const uint8_t *pc = nullptr, *ps = nullptr;
  const uint8_t *pa = nullptr, *pas = nullptr;  // the lane's activations of the chunk, their scales
  bool col = false;
  auto enter = [&](int unit) {
    const int slot = unit / groups, grp = unit % groups;
    const uint32_t w = slots[slot];
    const int64_t e = w & 1023u;
    const int first = (int)(w >> 10 & 2047u), cnt = (int)(w >> 21);
    // pairs of tiles 2 grp, 2 grp + 1 of the matrix's, four to 128 rows: rows j, j + 8 .. of each 32
    const int j = 16 * (grp & 1) + g;
    pc = codes + e * cb + (128 * (int64_t)(grp >> 1) + j) * (cols / 2) + 16 * t + 64 * part;
    ps = sfs + e * sb + ((int64_t)(grp >> 1) * (cols / 64) + (t >> 1)) * 512 + j * 16 + 1024 * part;
    col = g < cnt;
    const int64_t r = UP ? (col ? token[first + g] : 0) : first + (col ? g : 0);
    pa = reinterpret_cast<const uint8_t*>(UP ? a.xh : a.h) + (r * (128 * nch) + 8 * t + 128 * part) * 2;
    pas = reinterpret_cast<const uint8_t*>(UP ? a.x_scale + r * (cols / 128) + part
                                              : a.h_scale + r * (cols / 32) + 2 * (t >> 1) + 4 * part);
  };
  // the first pair of a chunk brings the activations with it
  auto copy_step = [&](auto second, auto with_codes, auto with_acts) {
    if (cu < u_end) {
      // past the last 64 columns the lane reads those before them, against activations of zero
      const bool in = UP || 128 * (part + S * cc) + 32 * t < cols;
      const uint8_t* q = pc + (in ? 0 : -32);
      if constexpr (with_codes.value) {
        copy16_stream<0>(cstep, q);
        copy16_stream<512>(cstep, q += row32);
        copy16_stream<1024>(cstep, q += row32);
        copy16_stream<1536>(cstep, q += row32);
        if ((t & 1) == 0) copy16_stream<0>(cstep + sf_to, ps + (in ? 0 : -512));
      }
      if constexpr (!second.value) {
        if (with_acts.value && col && in) {
          copy_act<0, 16>(cact, pa);
          copy_act<512, 16>(cact, pa + 64);
          copy_act<1024, 16>(cact, pa + 128);
          copy_act<1536, 16>(cact, pa + 192);
          copy_act<2048, UP ? 4 : 8>(cact - 8 * lane, pas);
        }
        cact = cact >= acts + kActBytes ? cact - kActBytes : cact + kActBytes;
        pc += row32 / 4;
        ps += 128;
      } else {
        ++cc;
        pc += 64 * S - row32 / 4;
        ps += 1024 * S - 128;
        pa += 256 * S;
        pas += (UP ? 4 : 16) * S;
        if (cc == my_chunks) {
          cc = 0;
          if (++cu < u_end) enter(cu);
        }
      }
      cstep = cstep >= base + (kSteps - 1) * kStepBytes ? cstep - (kSteps - 1) * kStepBytes : cstep + kStepBytes;
    }
    if (with_acts.value) copies_commit();
  };
  static_assert(kSteps == 3, "a chunk's first step is read as a second one is copied");
  constexpr std::false_type pair0{}, no{};
  constexpr std::true_type pair1{}, yes{};
  enter(u);
  if constexpr (!UP) {
    copy_step(pair0, yes, no);
    copy_step(pair1, yes, no);
    copy_step(pair0, yes, no);
    wait_for_previous();
    // again from the start, with the activations
    cu = u;
    cc = 0;
    cstep = base + 16 * lane;
    cact = acts + 16 * lane;
    enter(u);
  }
  copy_step(pair0, std::bool_constant<UP>{}, yes);
  copy_step(pair1, std::bool_constant<UP>{}, yes);
  copy_step(pair0, std::bool_constant<UP>{}, yes);

  uint32_t step = base + 16 * lane, act = acts;
  const uint32_t sf_from = 2048 + 32 * g + 16 * (t >> 1) - 16 * lane;
  float* red = reinterpret_cast<float*>(smem + kWarps * kWarpBytes);
  for (; u < u_end; ++u) {
    const int slot = u / groups, grp = u % groups;
    const uint32_t w = slots[slot];
    const int first = (int)(w >> 10 & 2047u), cnt = (int)(w >> 21);
    const float s_g = __ldg(s_gs + (w & 1023u)) * kSumUnit;
    float acc[kTiles][4] = {};
    auto stream = [&](auto few) {
      for (int i = 0; i < my_chunks; ++i) {
        uint32_t b[16] = {};
        float2 d0 = make_float2(0.0f, 0.0f), d1 = d0;
        bool rest = false;  // stretches far below their chunk's largest are left
        auto pair = [&](auto which) {
          constexpr int pr = which.value;
          copies_wait<kSteps - 1>();
          __syncwarp();  // the scales of a row are copied by one lane and read by two
          const uint4 lo0 = lds16<0>(step), lo1 = lds16<512>(step);
          const uint4 hi0 = lds16<1024>(step), hi1 = lds16<1536>(step);
          const uint4 sf = lds16<0>(step + sf_from);
          if (pr == 0) {
            const bool in = UP || 128 * (part + S * i) + 32 * t < cols;
            if constexpr (few.value) {
              if (in) {
                const int tok = g & 1;
                if (t == g >> 1 && tok < cnt) {
                  const uint32_t from = act + 64 * tok + 16 * t;
                  load_b(b, lds16<0>(from), lds16<512>(from), lds16<1024>(from), lds16<1536>(from));
                }
                d0 = lds8<2048>(act + 8 * t);
                if (cnt > 1) d1 = lds8<2048 + 32>(act + 8 * t);
                if (UP) {  // one scale per chunk
                  d0.y = d0.x;
                  d1.y = d1.x;
                }
              }
            } else {
              float2 f = make_float2(0.0f, 0.0f);
              if (g < cnt && in) {
                const uint32_t from = act + 16 * lane;
                load_b(b, lds16<0>(from), lds16<512>(from), lds16<1024>(from), lds16<1536>(from));
                f = lds8<2048>(act + 8 * lane);
              }
              float d = f.x;
              if (!UP) {
                // one scale per column and chunk: the largest; the others' elements take the quotient (a
                // power of two).  Of the lane's 32 elements the first and the second 16 have a scale each.
                d = quad_max(f);
                const float inv = __uint_as_float(0x7F000000u - __float_as_uint(fmaxf(d, 1.17549435e-38f)));
                const bool late0 = f.x < d * kNear, late1 = f.y < d * kNear;
                const uint32_t q0 = late0 ? 0u : pack_f16(f.x * inv, f.x * inv);
                const uint32_t q1 = late1 ? 0u : pack_f16(f.y * inv, f.y * inv);
                rest = __any_sync(0xffffffffu, (late0 && f.x > 0.0f) || (late1 && f.y > 0.0f));
#pragma unroll
                for (int q = 0; q < 16; ++q) b[q] = hmul2(b[q], q < 8 ? q0 : q1);
              }
              d0.x = __shfl_sync(0xffffffffu, d, 8 * t);
              d1.x = __shfl_sync(0xffffffffu, d, 8 * t + 4);
            }
            act = act == acts ? acts + kActBytes : acts;
          }
          if constexpr (few.value) {
            mma_tile_blocks(acc[2 * pr], lo0, hi0, sf.x, sf.z, b, d0, d1);
            mma_tile_blocks(acc[2 * pr + 1], lo1, hi1, sf.y, sf.w, b, d0, d1);
          } else {
            mma_tile(acc[2 * pr], lo0, hi0, sf.x, sf.z, b, d0.x, d1.x);
            mma_tile(acc[2 * pr + 1], lo1, hi1, sf.y, sf.w, b, d0.x, d1.x);
            if constexpr (!UP) {
              if (rest) {
                // the chunk's activations are still where they were; act has gone on to the next
                const uint32_t from = (act == acts ? acts + kActBytes : acts) + 16 * lane;
                float2 f = make_float2(0.0f, 0.0f);
                if (g < cnt && 128 * (part + S * i) + 32 * t < cols) f = lds8<2048>(from - 8 * lane);
                float d = quad_max(f);
#pragma unroll 1
                while (true) {
                  // those taken so far are out; the next ones are those near the largest that is left
                  if (f.x >= d * kNear) f.x = 0.0f;
                  if (f.y >= d * kNear) f.y = 0.0f;
                  if (!__any_sync(0xffffffffu, f.x + f.y > 0.0f)) break;
                  d = quad_max(f);
                  const float inv = __uint_as_float(0x7F000000u - __float_as_uint(fmaxf(d, 1.17549435e-38f)));
                  const float qx = f.x < d * kNear ? 0.0f : f.x * inv, qy = f.y < d * kNear ? 0.0f : f.y * inv;
                  const uint32_t q0 = pack_f16(qx, qx), q1 = pack_f16(qy, qy);
                  uint32_t c[16] = {};
                  if (f.x + f.y > 0.0f) {
                    load_b(c, lds16<0>(from), lds16<512>(from), lds16<1024>(from), lds16<1536>(from));
#pragma unroll
                    for (int q = 0; q < 8; ++q) {  // a taken block may hold an infinity
                      c[q] = q0 != 0 ? hmul2(c[q], q0) : 0u;
                      c[8 + q] = q1 != 0 ? hmul2(c[8 + q], q1) : 0u;
                    }
                  }
                  const float e0 = __shfl_sync(0xffffffffu, d, 8 * t), e1 = __shfl_sync(0xffffffffu, d, 8 * t + 4);
                  // the codes are read again, so that nothing is kept in registers for this
                  const uint4 s4 = lds16<0>(step + sf_from);
                  mma_tile(acc[2 * pr], lds16<0>(step), lds16<1024>(step), s4.x, s4.z, c, e0, e1);
                  mma_tile(acc[2 * pr + 1], lds16<512>(step), lds16<1536>(step), s4.y, s4.w, c, e0, e1);
                }
              }
            }
          }
          step = step >= base + (kSteps - 1) * kStepBytes ? step - (kSteps - 1) * kStepBytes : step + kStepBytes;
          __syncwarp();  // every lane has read the place that is filled next
          copy_step(std::bool_constant<pr == 0>{}, yes, yes);
        };
        pair(std::integral_constant<int, 0>{});
        pair(std::integral_constant<int, 1>{});
      }
    };
    if (cnt <= 2) {
      stream(std::true_type{});
      // the quad's codes together, in the columns 0 and 1
#pragma unroll
      for (int r = 0; r < kTiles; ++r) {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          acc[r][q] += __shfl_xor_sync(0xffffffffu, acc[r][q], 1);
          acc[r][q] += __shfl_xor_sync(0xffffffffu, acc[r][q], 2);
        }
      }
    } else {
      stream(std::false_type{});
    }
    if (S > 1) {
      float4* mine = reinterpret_cast<float4*>(red + warp * (kRedBytes / 4)) + lane;
      const int id = 1 + warp / S;
      if (part != 0) {
#pragma unroll
        for (int r = 0; r < kTiles; ++r) mine[32 * r] = make_float4(acc[r][0], acc[r][1], acc[r][2], acc[r][3]);
      }
      asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(32 * S) : "memory");
      if (part == 0) {
        for (int q = 1; q < S; ++q) {
#pragma unroll
          for (int r = 0; r < kTiles; ++r) {
            const float4 v = mine[q * (kRedBytes / 16) + 32 * r];
            acc[r][0] += v.x;
            acc[r][1] += v.y;
            acc[r][2] += v.z;
            acc[r][3] += v.w;
          }
        }
      }
      asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(32 * S) : "memory");
      if (part != 0) continue;
    }
    if (UP) {
      // a unit's 32 rows of h are one scale stretch of each column
      float h[kTiles][2], m[2] = {0.0f, 0.0f};
#pragma unroll
      for (int r = 0; r < kTiles; ++r) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const float gate = acc[r][j] * s_g, up = acc[r][2 + j] * s_g;
          h[r][j] = gate / (1.0f + expf(-gate)) * up;
          // as integers, magnitudes keep their order and NaN is the largest
          m[j] = __uint_as_float(max(__float_as_uint(m[j]), __float_as_uint(h[r][j]) & 0x7FFFFFFFu));
        }
      }
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        uint32_t top = __float_as_uint(m[j]);
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
        float up, down;
        stretch_scale((int)(top >> 23), &up, &down);
        if (2 * t + j < cnt) {
          const int64_t p = first + 2 * t + j;
          // row 64 (grp >> 1) + 16 (grp & 1) + 32 (r & 1) + 8 (r >> 1) + g, in the order of the activations
          uint16_t* o = a.h + p * ((a.I + 127) / 128 * 128) + 128 * (grp >> 2) + 16 * (grp >> 1 & 1) + 64 * (grp & 1) + g;
#pragma unroll
          for (int r = 0; r < kTiles; ++r)
            o[8 * (r & 1) + 32 * (r >> 1)] = __half_as_ushort(__float2half_rn(h[r][j] * up));
          if (g == 0) a.h_scale[p * (a.I / 32) + grp] = top == 0 ? 0.0f : down;
        }
      }
    } else {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        if (2 * t + j < cnt) {
          float* o = a.y + (int64_t)(first + 2 * t + j) * a.H + 128 * (grp >> 1) + 16 * (grp & 1) + g;
#pragma unroll
          for (int r = 0; r < kTiles; ++r) {
            o[32 * (r & 1) + 8 * (r >> 1)] = acc[r][j] * s_g;
            o[64 + 32 * (r & 1) + 8 * (r >> 1)] = acc[r][2 + j] * s_g;
          }
        }
      }
    }
  }
}

// out[t] = sum_j w_tj y[place of (t, j)], j ascending; four columns a thread.
__global__ void __launch_bounds__(128) moe_few_combine_kernel(MoeFewArgs a) {
  const int64_t t = blockIdx.y;
  const int c = 4 * (blockIdx.x * 128 + threadIdx.x);
  wait_for_previous();
  if (c >= a.H) return;
  const int32_t* place = a.lists + list_places(a.T * a.k) + t * a.k;
  const float* w = a.topk_w + t * a.k;
  float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 8
  for (int j = 0; j < a.k; ++j) {
    const int p = place[j];
    if (p >= 0) {
      const float4 y = *reinterpret_cast<const float4*>(a.y + (int64_t)p * a.H + c);
      const float f = w[j];
      v.x = fmaf(f, y.x, v.x);
      v.y = fmaf(f, y.y, v.y);
      v.z = fmaf(f, y.z, v.z);
      v.w = fmaf(f, y.w, v.w);
    }
  }
  const __nv_bfloat162 lo = __floats2bfloat162_rn(v.x, v.y), hi = __floats2bfloat162_rn(v.z, v.w);
  *reinterpret_cast<uint2*>(a.out + t * a.ldo + c) =
      make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
}

size_t moe_few_list_words(int64_t T, int32_t k) { return (size_t)list_words((int)(T * k)); }

// Once per device and kernel: the most shared memory that a call can need.
static cudaError_t allow_shared_memory() {
  static std::atomic<uint64_t> done{0};
  constexpr int kMost = kRingBytes + kFewMaxPairs * 5;
  static_assert(kMost <= 227 * 1024, "the most pairs fit");
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = dev < 64 ? 1ull << dev : 0;
  if (done.load() & bit) return cudaSuccess;
  for (const void* f : {reinterpret_cast<const void*>(moe_few_stream_kernel<true>),
                        reinterpret_cast<const void*>(moe_few_stream_kernel<false>)}) {
    e = cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, kMost);
    if (e != cudaSuccess) return e;
  }
  done.fetch_or(bit);
  return cudaSuccess;
}

cudaError_t launch_moe_few(const MoeFewArgs& a, int num_sms, cudaStream_t st) {
  const int P = a.T * a.k;
  const int smem = kRingBytes + P * 4 + token_words(P) * 4;
  cudaError_t e = allow_shared_memory();
  if (e != cudaSuccess) return e;
  moe_few_prepare_kernel<<<a.T + 1, 1024, 0, st>>>(a);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)num_sms);
  cfg.blockDim = dim3(kWarps * 32);
  cfg.dynamicSmemBytes = (size_t)smem;
  cfg.stream = st;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, moe_few_stream_kernel<true>, a);
  if (e != cudaSuccess) return e;
  e = cudaLaunchKernelEx(&cfg, moe_few_stream_kernel<false>, a);
  if (e != cudaSuccess) return e;
  cfg.gridDim = dim3((unsigned)((a.H + 511) / 512), (unsigned)a.T);
  cfg.blockDim = dim3(128);
  cfg.dynamicSmemBytes = 0;
  return cudaLaunchKernelEx(&cfg, moe_few_combine_kernel, a);
}

}  // namespace nvfp4
