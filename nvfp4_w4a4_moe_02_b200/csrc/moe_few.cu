// A whole mixture-of-experts layer for a few tokens in two kernels: routing and gate_up with
// SwiGLU, then down with the weighted combine.  Activations stay bf16 (the trainer's side of the
// method: weights fake-quantised, activations not), weights are the packed NVFP4 ones.
//
//   ids_t, w_t = the k largest logits of token t and their renormalised softmax
//   h_tj = silu(G_e x_t) * (U_e x_t),  out_t = sum_j w_tj D_e h_tj,   e = ids_tj
//
// The weights of the experts that are touched bound it: each 16 x 128 tile of codes goes from
// memory straight into registers and is decoded there into the A operand of mma.m16n8k16 (f16,
// binary32 sums), the expert's tokens are its eight columns.
//   - E2M1 x E4M3 has at most six significant bits and lies in [2^-10, 2688]: exact in f16.
//   - The sum over k may take its elements in any order, so a lane keeps the 32 consecutive codes
//     of its 16-byte load: instruction i of a chunk contracts elements 4i .. 4i+3 of every lane.
//   - Activations are scaled per token and 128-element chunk by a power of two that brings the
//     chunk's largest to [2^14, 2^15), which keeps every bf16 down to 2^-31 of it exact in f16;
//     the power is taken out of the chunk's sum.
//   - A tile's 16 rows are rows 4jj .. 4jj+3 of each of the four 32-row groups of a scale atom's 128:
//     their scales are 64 consecutive bytes per 64 columns, and in the gate/up interleaved pack
//     groups 0, 1 are gate rows and groups 2, 3 the matching up rows, which land in one lane.
#include "common.cuh"
#include "kernels.h"

namespace nvfp4 {

namespace {

constexpr int kWarps = 4;       // warps of a gate_up block: they split K
constexpr int kTiles = 4;       // 16-row tiles per gate_up block
constexpr int kDnWarps = 8;     // warps of a down block: they split the (expert, K) list
constexpr int kDnTiles = 2;

// workspace lists: [0] touched experts n, then (expert, first pair) x n, one closing (-, pairs),
// then the pairs t * k + j in expert order
constexpr int kListHead = 16;

__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint4 ldg_stream(const uint8_t* p) {  // weights are read once
  uint4 r;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
               : "l"(p));
  return r;
}

// One 16 x 128 chunk of a tile as it is loaded: 32 codes of each of the lane's two rows and the
// scales of their two 16-blocks.
struct Chunk {
  uint4 lo, hi;
  uint16_t sl, sh;
};

// The lane's part of a tile of a packed matrix.
struct TileRef {
  const uint8_t* codes;  // the lane's low row, its 16 bytes of chunk 0
  const uint8_t* sf;     // the lane's two scales of the low row, chunk 0; the high row's follow 8 bytes on
};

__device__ __forceinline__ TileRef tile_ref(const uint8_t* codes, const uint8_t* sf, int tile, int cols) {
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int q = tile >> 3, jj = tile & 7, j = 4 * jj + (g & 3);
  const int64_t row = 128 * (int64_t)q + 32 * (g >> 2) + j;
  TileRef r;
  r.codes = codes + row * (cols / 2) + 16 * t;
  r.sf = sf + ((int64_t)q * (cols / 64) + (t >> 1)) * 512 + j * 16 + (g >> 2) * 4 + (t & 1) * 2;
  return r;
}

__device__ __forceinline__ uint16_t ldg_u16(const uint8_t* p) {
  uint16_t r;
  asm volatile("ld.global.nc.u16 %0, [%1];" : "=h"(r) : "l"(p));
  return r;
}

// hi: bytes from the low row to the high row (64 rows).  A chunk past the last 64 columns reads
// zeros (scale 0).
template <bool TAIL>
__device__ __forceinline__ Chunk load_chunk(const TileRef& r, int64_t hi, int c, int cols) {
  Chunk k;
  if (!TAIL || 128 * c + 32 * (int)(threadIdx.x & 3) < cols) {
    const uint8_t* p = r.codes + 64 * (int64_t)c;
    k.lo = ldg_stream(p);
    k.hi = ldg_stream(p + hi);
    k.sl = ldg_u16(r.sf + 1024 * (int64_t)c);
    k.sh = ldg_u16(r.sf + 1024 * (int64_t)c + 8);
  } else {
    k.lo = k.hi = make_uint4(0, 0, 0, 0);
    k.sl = k.sh = 0;
  }
  return k;
}

// The byte `i` of a word of codes -> two halves.  The conversion reads its register's low byte.
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

__device__ __forceinline__ __half2 e4m3x2(uint16_t c) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(c));
  return *reinterpret_cast<const __half2*>(&r);
}

// acc += (chunk of weights) x (B fragments b of the same 128 elements), in units of the weights'
// tensor scale and of the activations' scale.
__device__ __forceinline__ void mma_chunk(float (&acc)[4], const Chunk& k, const uint32_t (&b)[16]) {
  const __half2 sl = e4m3x2(k.sl), sh = e4m3x2(k.sh);
  const uint32_t lo[4] = {k.lo.x, k.lo.y, k.lo.z, k.lo.w}, hi[4] = {k.hi.x, k.hi.y, k.hi.z, k.hi.w};
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    // a word is 8 codes: the first two words belong to the lane's first 16-block
    auto sc = [&](uint32_t a, __half2 s) { return w < 2 ? scale_low(a, s) : scale_high(a, s); };
    mma16816(acc, sc(decode_byte<0>(lo[w]), sl), sc(decode_byte<0>(hi[w]), sh), sc(decode_byte<1>(lo[w]), sl),
             sc(decode_byte<1>(hi[w]), sh), b[4 * w], b[4 * w + 1]);
    mma16816(acc, sc(decode_byte<2>(lo[w]), sl), sc(decode_byte<2>(hi[w]), sh), sc(decode_byte<3>(lo[w]), sl),
             sc(decode_byte<3>(hi[w]), sh), b[4 * w + 2], b[4 * w + 3]);
  }
}

__device__ __forceinline__ uint32_t pack_f16(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// The power of two for a chunk whose largest magnitude is amax, and its inverse.
__device__ __forceinline__ void chunk_scale(float amax, float* up, float* down) {
  const int e = min(max((int)(__float_as_uint(amax) >> 23), 15), 254);
  *up = __uint_as_float((uint32_t)(268 - e) << 23);
  *down = __uint_as_float((uint32_t)(e - 14) << 23);
}

__device__ __forceinline__ float quad_max(float v) {
  v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 1));
  return fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 2));
}

// B fragments of 128 elements of the lane's column (token), and the scale taken out.
__device__ __forceinline__ float scale_to_f16(const float (&v)[32], uint32_t (&b)[16]) {
  float m = 0.0f;
#pragma unroll
  for (int i = 0; i < 32; ++i) m = fmaxf(m, fabsf(v[i]));
  float up, down;
  chunk_scale(quad_max(m), &up, &down);
#pragma unroll
  for (int i = 0; i < 16; ++i) b[i] = pack_f16(v[2 * i] * up, v[2 * i + 1] * up);
  return down;
}

__device__ __forceinline__ float load_b_bf16(const uint16_t* row, bool has, int c, int cols, uint32_t (&b)[16]) {
  const int t = threadIdx.x & 3;
  float v[32];
  const bool in = has && 128 * c + 32 * t < cols;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint4 r = make_uint4(0, 0, 0, 0);
    if (in) r = __ldg(reinterpret_cast<const uint4*>(row + 128 * c + 32 * t) + i);
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[8 * i + 2 * j] = __uint_as_float(w[j] << 16);
      v[8 * i + 2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
    }
  }
  return scale_to_f16(v, b);
}

__device__ __forceinline__ float load_b_f32(const float* row, bool has, int c, int cols, uint32_t (&b)[16]) {
  const int t = threadIdx.x & 3;
  float v[32];
  const bool in = has && 128 * c + 32 * t < cols;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float4 r = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (in) r = __ldg(reinterpret_cast<const float4*>(row + 128 * c + 32 * t) + i);
    v[4 * i] = r.x;
    v[4 * i + 1] = r.y;
    v[4 * i + 2] = r.z;
    v[4 * i + 3] = r.w;
  }
  return scale_to_f16(v, b);
}

struct Lists {
  uint16_t id[kFewMaxPairs];             // expert of pair t * k + j (0xFFFF: none)
  uint16_t order[kFewMaxPairs];          // pairs in expert order, tokens ascending
  int cursor[kMaxRouteExperts];
  uint16_t expert[kMaxRouteExperts];     // touched experts, ascending
  uint16_t start[kMaxRouteExperts + 1];  // first pair of each
  int n;
};

// The same choice and weights as moe_route_topk: k rounds of a warp arg-max over ordered keys.
__device__ void route_token(const MoeFewArgs& a, int t, uint16_t* id, bool write) {
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
  if (nb == 1) load(0);
  float lmax = 0.0f, sum = 0.0f, mine_p = 0.0f;
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
    const int e = (int)__reduce_min_sync(0xffffffffu, best == top ? (uint32_t)be : 0x7FFFFFFFu);
    if ((e & 31) == lane) {
      const int i = (e >> 5) & 7;
#pragma unroll
      for (int b = 0; b < 4; ++b)
        if (b == e >> 8) taken[b] |= 1u << i;
#pragma unroll
      for (int q = 0; q < 8; ++q)
        if (q == i && nb == 1) key[q] = 0;
    }
    const float l = __uint_as_float((top & 0x80000000u) ? (top & 0x7FFFFFFFu) : ~top);
    if (j == 0) lmax = l;
    const float p = expf(__fsub_rn(l, lmax));
    sum = __fadd_rn(sum, p);
    if (lane == j) {
      mine_p = p;
      mine_e = e;
    }
  }
  if (lane < a.k) {
    const int p = t * a.k + lane;
    id[p] = bad ? 0xFFFFu : (uint16_t)mine_e;
    if (write) {
      a.ids[p] = bad ? -1 : mine_e;
      a.topk_w[p] = bad ? 0.0f : __fdiv_rn(mine_p, sum);
    }
  }
  if (bad && write && lane == 0) report_status(a.status, kErrRange);
}

// Every block routes all tokens itself: T k rounds of ~100 cycles over its warps against a launch
// and a pass over memory.  Block 0 also writes the choice and the lists for the down kernel.
__device__ void build_lists(const MoeFewArgs& a, Lists& L) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int P = a.T * a.k;
  const bool write = blockIdx.x == 0;
  for (int e = threadIdx.x; e < a.E; e += blockDim.x) L.cursor[e] = 0;
  for (int t = warp; t < a.T; t += blockDim.x / 32) route_token(a, t, L.id, write);
  __syncthreads();
  for (int p = threadIdx.x; p < P; p += blockDim.x)
    if (L.id[p] != 0xFFFFu) atomicAdd(&L.cursor[L.id[p]], 1);
  __syncthreads();
  if (warp == 0) {
    int n = 0, at = 0;
    for (int e0 = 0; e0 < a.E; e0 += 32) {
      const int e = e0 + lane;
      const int cnt = e < a.E ? L.cursor[e] : 0;
      const uint32_t m = __ballot_sync(0xffffffffu, cnt > 0);
      int run = cnt;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, run, o);
        if (lane >= o) run += v;
      }
      if (cnt > 0) {
        const int i = n + __popc(m & ((1u << lane) - 1u));
        L.expert[i] = (uint16_t)e;
        L.start[i] = (uint16_t)(at + run - cnt);
        L.cursor[e] = at + run - cnt;
      }
      n += __popc(m);
      at += __shfl_sync(0xffffffffu, run, 31);
    }
    if (lane == 0) {
      L.n = n;
      L.start[n] = (uint16_t)at;
    }
    __syncwarp();
    // ranks in pair order, 32 at a time
    for (int p0 = 0; p0 < P; p0 += 32) {
      const int p = p0 + lane;
      const uint32_t e = p < P ? L.id[p] : 0xFFFFu;
      const uint32_t same = __match_any_sync(0xffffffffu, e);
      const uint32_t before = __popc(same & ((1u << lane) - 1u));
      int base = 0;
      if (e != 0xFFFFu) base = L.cursor[e];
      __syncwarp();
      if (e != 0xFFFFu) {
        L.order[base + before] = (uint16_t)p;
        if (before == 0) L.cursor[e] = base + __popc(same);
      }
      __syncwarp();
    }
  }
  __syncthreads();
  if (write) {
    const int n = L.n;
    int32_t* o = a.lists;
    if (threadIdx.x == 0) o[0] = n;
    for (int i = threadIdx.x; i <= n; i += blockDim.x) {
      o[kListHead + 2 * i] = i < n ? L.expert[i] : -1;
      o[kListHead + 2 * i + 1] = L.start[i];
    }
    int32_t* ord = o + kListHead + 2 * (min(P, a.E) + 1);
    for (int p = threadIdx.x; p < L.start[n]; p += blockDim.x) ord[p] = L.order[p];
  }
}

}  // namespace

// gate_up + SwiGLU.  An item is (touched expert, kTiles tiles); a block's warps split its K in
// interleaved chunks and join their sums in shared memory, in warp order.
__global__ void __launch_bounds__(kWarps * 32, 4) moe_few_gate_up_kernel(MoeFewArgs a) {
  __shared__ Lists L;
  __shared__ float red[kWarps][kTiles][16][8];
  build_lists(a, L);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
  const int groups = a.I / 8 / kTiles;
  const int nch = (a.H + 127) / 128;
  const int items = L.n * groups;
  const int64_t cb = (int64_t)a.I * a.H, sb = (int64_t)a.I * a.H / 8;  // bytes of one expert's codes / scales
  for (int it = blockIdx.x; it < items; it += gridDim.x) {
    const int ei = it / groups, grp = it % groups;
    const int e = L.expert[ei];
    const float s_g = __ldg(a.gu_sg + e);
    TileRef ref[kTiles];
#pragma unroll
    for (int r = 0; r < kTiles; ++r) ref[r] = tile_ref(a.gu_codes + e * cb, a.gu_sf + e * sb, grp * kTiles + r, a.H);
    for (int p0 = L.start[ei]; p0 < L.start[ei + 1]; p0 += 8) {
      const int cnt = min(8, L.start[ei + 1] - p0);
      const bool has = g < cnt;
      const uint16_t* xr = a.x + (has ? (int64_t)(L.order[p0 + g] / a.k) * a.ldx : 0);
      float acc[kTiles][4] = {};
      for (int c = warp; c < nch; c += kWarps) {
        Chunk ck[kTiles];
#pragma unroll
        for (int r = 0; r < kTiles; ++r) ck[r] = load_chunk<false>(ref[r], 32 * (int64_t)a.H, c, a.H);
        uint32_t b[16];
        const float down = load_b_bf16(xr, has, c, a.H, b) * s_g;
        const float d0 = __shfl_sync(0xffffffffu, down, 8 * t), d1 = __shfl_sync(0xffffffffu, down, 8 * t + 4);
#pragma unroll
        for (int r = 0; r < kTiles; ++r) {
          float part[4] = {0.0f, 0.0f, 0.0f, 0.0f};
          mma_chunk(part, ck[r], b);
          acc[r][0] = fmaf(part[0], d0, acc[r][0]);
          acc[r][1] = fmaf(part[1], d1, acc[r][1]);
          acc[r][2] = fmaf(part[2], d0, acc[r][2]);
          acc[r][3] = fmaf(part[3], d1, acc[r][3]);
        }
      }
#pragma unroll
      for (int r = 0; r < kTiles; ++r) {
        *reinterpret_cast<float2*>(&red[warp][r][g][2 * t]) = make_float2(acc[r][0], acc[r][1]);
        *reinterpret_cast<float2*>(&red[warp][r][g + 8][2 * t]) = make_float2(acc[r][2], acc[r][3]);
      }
      __syncthreads();
      for (int o = threadIdx.x; o < kTiles * 64; o += kWarps * 32) {
        const int col = o >> 5, r = (o >> 3) & 3, row = o & 7;
        if (col < cnt) {
          float gate = 0.0f, up = 0.0f;
#pragma unroll
          for (int w = 0; w < kWarps; ++w) {
            gate += red[w][r][row][col];
            up += red[w][r][row + 8][col];
          }
          const int tile = grp * kTiles + r;
          const int hi = 64 * (tile >> 3) + 32 * (row >> 2) + 4 * (tile & 7) + (row & 3);
          a.h[(int64_t)(p0 + col) * a.I + hi] = gate / (1.0f + expf(-gate)) * up;
        }
      }
      __syncthreads();
    }
  }
}

// down + combine.  A block owns kDnTiles tiles of output columns for all tokens; its warps take
// equal stretches of the (touched expert, chunk) list, each adding w_tj * sum into a private
// [T][rows] array; the arrays are summed in warp order, so the result does not depend on timing.
__global__ void __launch_bounds__(kDnWarps * 32, 2) moe_few_down_kernel(MoeFewArgs a) {
  extern __shared__ float accw[];  // [kDnWarps][T][16 kDnTiles]
  constexpr int kRows = 16 * kDnTiles;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
  const int P = a.T * a.k;
  const int n = __ldg(a.lists);
  const int32_t* list = a.lists + kListHead;
  const int32_t* order = list + 2 * (min(P, a.E) + 1);
  const int nch = (a.I + 127) / 128;
  const int64_t cb = (int64_t)a.H * a.I / 2, sb = (int64_t)a.H * a.I / 16;
  float* mine = accw + warp * a.T * kRows;
  for (int i = lane; i < a.T * kRows; i += 32) mine[i] = 0.0f;
  __syncwarp();
  const int units = n * nch;
  int u = (int)((int64_t)units * warp / kDnWarps);
  const int u_end = (int)((int64_t)units * (warp + 1) / kDnWarps);
  while (u < u_end) {
    const int ei = u / nch, c0 = u % nch;
    const int c1 = min(nch, c0 + (u_end - u));
    const int e = __ldg(list + 2 * ei);
    const int s0 = __ldg(list + 2 * ei + 1), s1 = __ldg(list + 2 * ei + 3);
    const float s_g = __ldg(a.dn_sg + e);
    TileRef ref[kDnTiles];
#pragma unroll
    for (int r = 0; r < kDnTiles; ++r)
      ref[r] = tile_ref(a.dn_codes + e * cb, a.dn_sf + e * sb, blockIdx.x * kDnTiles + r, a.I);
    for (int p0 = s0; p0 < s1; p0 += 8) {
      const int cnt = min(8, s1 - p0);
      const bool has = g < cnt;
      const float* hr = a.h + (int64_t)(has ? p0 + g : 0) * a.I;
      float acc[kDnTiles][4] = {};
      for (int c = c0; c < c1; ++c) {
        Chunk ck[kDnTiles];
#pragma unroll
        for (int r = 0; r < kDnTiles; ++r) ck[r] = load_chunk<true>(ref[r], 32 * (int64_t)a.I, c, a.I);
        uint32_t b[16];
        const float down = load_b_f32(hr, has, c, a.I, b) * s_g;
        const float d0 = __shfl_sync(0xffffffffu, down, 8 * t), d1 = __shfl_sync(0xffffffffu, down, 8 * t + 4);
#pragma unroll
        for (int r = 0; r < kDnTiles; ++r) {
          float part[4] = {0.0f, 0.0f, 0.0f, 0.0f};
          mma_chunk(part, ck[r], b);
          acc[r][0] = fmaf(part[0], d0, acc[r][0]);
          acc[r][1] = fmaf(part[1], d1, acc[r][1]);
          acc[r][2] = fmaf(part[2], d0, acc[r][2]);
          acc[r][3] = fmaf(part[3], d1, acc[r][3]);
        }
      }
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int col = 2 * t + j;
        if (col < cnt) {
          const int p = __ldg(order + p0 + col);
          const float w = __ldg(a.topk_w + p);
          float* o = mine + (p / a.k) * kRows;  // an expert's tokens are distinct: no two lanes meet
#pragma unroll
          for (int r = 0; r < kDnTiles; ++r) {
            o[16 * r + g] = fmaf(w, acc[r][j], o[16 * r + g]);
            o[16 * r + g + 8] = fmaf(w, acc[r][2 + j], o[16 * r + g + 8]);
          }
        }
      }
      __syncwarp();
    }
    u += c1 - c0;
  }
  __syncthreads();
  for (int i = threadIdx.x; i < a.T * kRows; i += kDnWarps * 32) {
    float s = 0.0f;
    for (int w = 0; w < kDnWarps; ++w) s += accw[w * a.T * kRows + i];
    const int tok = i / kRows, row = i % 16, tile = blockIdx.x * kDnTiles + (i % kRows) / 16;
    const int col = 128 * (tile >> 3) + 32 * (row >> 2) + 4 * (tile & 7) + (row & 3);
    const __nv_bfloat16 b = __float2bfloat16_rn(s);
    a.out[(int64_t)tok * a.ldo + col] = *reinterpret_cast<const uint16_t*>(&b);
  }
}

size_t moe_few_list_words(int64_t T, int32_t k, int32_t E) {
  const int64_t P = T * k;
  return (size_t)(kListHead + 2 * ((P < E ? P : E) + 1) + P);
}

cudaError_t launch_moe_few(const MoeFewArgs& a, int num_sms, cudaStream_t st) {
  const int64_t P = (int64_t)a.T * a.k;
  const int64_t items = (P < a.E ? P : a.E) * (a.I / 8 / kTiles);
  const int64_t slots = 4 * (int64_t)num_sms;
  moe_few_gate_up_kernel<<<(unsigned)(items < slots ? items : slots), kWarps * 32, 0, st>>>(a);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  const int smem = kDnWarps * a.T * 16 * kDnTiles * (int)sizeof(float);
  if (smem > 48 * 1024) {
    e = cudaFuncSetAttribute(moe_few_down_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
  }
  moe_few_down_kernel<<<(unsigned)(a.H / 16 / kDnTiles), kDnWarps * 32, smem, st>>>(a);
  return cudaGetLastError();
}

}  // namespace nvfp4
