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
constexpr int kTiles = 4;       // 16-row tiles per gate_up item
constexpr int kDnWarps = 8;     // warps of a down block: they split the (slot, K) list
constexpr int kDnTiles = 4;
constexpr int kDnRows = 16 * kDnTiles;

// A slot is up to eight tokens (pairs) of one expert.  Workspace words: [0] slots n, then (expert,
// first pair, end) x n from kListHead on, the pairs t * k + j in slot order, and one arrival count
// per kDnRows output columns (zeroed by the gate_up kernel).
constexpr int kListHead = 16;
constexpr int kFewMaxSlots = kMaxRouteExperts + kFewMaxPairs / 8;
__host__ __device__ inline int max_slots(int P, int E) { return P < E + P / 8 ? P : E + P / 8; }

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

// Of a tile whose index is a multiple of 4; the three after it lie 4 rows and 64 scale bytes apart.
__device__ __forceinline__ TileRef tile_ref(const uint8_t* codes, const uint8_t* sf, int tile, int cols) {
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int q = tile >> 3, j = 4 * (tile & 7) + (g & 3);
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

// Tile `r` after the reference; `in` false (past the last 64 columns): zeros.
__device__ __forceinline__ Chunk load_chunk(const TileRef& ref, int r, int cols, bool in) {
  Chunk k;
  if (in) {
    const uint8_t* p = ref.codes + r * (2 * cols);
    k.lo = ldg_stream(p);
    k.hi = ldg_stream(p + 32 * (int64_t)cols);
    k.sl = ldg_u16(ref.sf + 64 * r);
    k.sh = ldg_u16(ref.sf + 64 * r + 8);
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

__device__ __forceinline__ float max3_abs(float m, float a, float b) {
  return fmaxf(m, fmaxf(fabsf(a), fabsf(b)));
}

// B fragments of 128 elements of the lane's column (token), and the scale taken out.
__device__ __forceinline__ float scale_to_f16(const float (&v)[32], uint32_t (&b)[16]) {
  float m0 = 0.0f, m1 = 0.0f;
#pragma unroll
  for (int i = 0; i < 32; i += 4) {
    m0 = max3_abs(m0, v[i], v[i + 1]);
    m1 = max3_abs(m1, v[i + 2], v[i + 3]);
  }
  float up, down;
  chunk_scale(quad_max(fmaxf(m0, m1)), &up, &down);
#pragma unroll
  for (int i = 0; i < 16; ++i) b[i] = pack_f16(v[2 * i] * up, v[2 * i + 1] * up);
  return down;
}

// row: the lane's 32 elements of the chunk; `in` false: zeros
__device__ __forceinline__ float load_b_bf16(const uint16_t* row, bool in, uint32_t (&b)[16]) {
  float v[32];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint4 r = make_uint4(0, 0, 0, 0);
    if (in) r = __ldg(reinterpret_cast<const uint4*>(row) + i);
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[8 * i + 2 * j] = __uint_as_float(w[j] << 16);
      v[8 * i + 2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
    }
  }
  return scale_to_f16(v, b);
}

__device__ __forceinline__ float load_b_f32(const float* row, bool in, uint32_t (&b)[16]) {
  float v[32];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float4 r = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (in) r = __ldg(reinterpret_cast<const float4*>(row) + i);
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
  uint16_t expert[kFewMaxSlots];         // slots, experts ascending
  uint16_t start[kFewMaxSlots];          // first pair of each
  uint8_t count[kFewMaxSlots];
  int n, pairs;
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
    int n = 0, at = 0;  // slots and pairs before this group of experts
    for (int e0 = 0; e0 < a.E; e0 += 32) {
      const int e = e0 + lane;
      const int cnt = e < a.E ? L.cursor[e] : 0;
      if (__ballot_sync(0xffffffffu, cnt > 0) == 0) continue;
      int run = cnt | (cnt + 7) / 8 << 16;  // pairs low, slots high
      const int own = run;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, run, o);
        if (lane >= o) run += v;
      }
      const int first = at + ((run - own) & 0xFFFF);
      int i = n + ((run - own) >> 16);
      for (int c = 0; c < cnt; c += 8, ++i) {
        L.expert[i] = (uint16_t)e;
        L.start[i] = (uint16_t)(first + c);
        L.count[i] = (uint8_t)min(8, cnt - c);
      }
      if (cnt > 0) L.cursor[e] = first;
      const int all = __shfl_sync(0xffffffffu, run, 31);
      at += all & 0xFFFF;
      n += all >> 16;
    }
    if (lane == 0) {
      L.n = n;
      L.pairs = at;
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
    o += kListHead;
    for (int i = threadIdx.x; i < n; i += blockDim.x) {
      o[3 * i] = L.expert[i];
      o[3 * i + 1] = L.start[i];
      o[3 * i + 2] = L.start[i] + L.count[i];
    }
    o += 3 * max_slots(P, a.E);
    for (int p = threadIdx.x; p < L.pairs; p += blockDim.x) o[p] = L.order[p];
    o += P;
    for (int i = threadIdx.x; i < a.H / kDnRows; i += blockDim.x) o[i] = 0;
  }
}

}  // namespace

// gate_up + SwiGLU.  An item is (slot, kTiles tiles); a block's warps split its K in interleaved
// chunks and join their sums in shared memory, in warp order.  Each warp keeps the next chunk of
// every tile in flight, across the end of an item too.
__global__ void __launch_bounds__(kWarps * 32, 4) moe_few_gate_up_kernel(MoeFewArgs a) {
  __shared__ Lists L;
  __shared__ float red[kWarps][kTiles][16][8];
  build_lists(a, L);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
  const int groups = a.I / 8 / kTiles;
  const int nch = a.H / 128;
  const int items = L.n * groups;
  const int64_t cb = (int64_t)a.I * a.H, sb = (int64_t)a.I * a.H / 8;  // bytes of one expert's codes / scales
  auto item_ref = [&](int it) {
    const int64_t e = L.expert[it / groups];
    TileRef r = tile_ref(a.gu_codes + e * cb, a.gu_sf + e * sb, it % groups * kTiles, a.H);
    r.codes += 64 * warp;
    r.sf += 1024 * warp;
    return r;
  };
  int it = blockIdx.x;
  if (it >= items) return;
  TileRef next = item_ref(it);  // what the ring holds or is about to
  Chunk ring[kTiles];
  const bool any = warp < nch;
#pragma unroll
  for (int r = 0; r < kTiles; ++r) ring[r] = load_chunk(next, r, a.H, any);
  for (; it < items; it += gridDim.x) {
    const int slot = it / groups;
    const int p0 = L.start[slot], cnt = L.count[slot];
    const float s_g = __ldg(a.gu_sg + L.expert[slot]);
    const bool has = g < cnt;
    const uint16_t* xr = a.x + (has ? (int64_t)(L.order[p0 + g] / a.k) * a.ldx : 0) + 32 * t;
    float acc[kTiles][4] = {};
    for (int c = warp; c < nch; c += kWarps) {
      bool more = true;
      if (c + kWarps < nch) {
        next.codes += 64 * kWarps;
        next.sf += 1024 * kWarps;
      } else if (it + gridDim.x < items) {
        next = item_ref(it + gridDim.x);
      } else {
        more = false;
      }
      uint32_t b[16];
      const float down = load_b_bf16(xr + 128 * c, has, b) * s_g;
      const float d0 = __shfl_sync(0xffffffffu, down, 8 * t), d1 = __shfl_sync(0xffffffffu, down, 8 * t + 4);
#pragma unroll
      for (int r = 0; r < kTiles; ++r) {
        const Chunk k = ring[r];
        if (more) ring[r] = load_chunk(next, r, a.H, true);
        float part[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        mma_chunk(part, k, b);
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
        const int tile = it % groups * kTiles + r;
        const int hi = 64 * (tile >> 3) + 32 * (row >> 2) + 4 * (tile & 7) + (row & 3);
        a.h[(int64_t)(p0 + col) * a.I + hi] = gate / (1.0f + expf(-gate)) * up;
      }
    }
    __syncthreads();
  }
}

// down + combine.  The units (kDnRows output columns, slot), columns outermost, are split evenly over
// the blocks, so that few tokens still fill the card and many leave no last wave; a block's warps
// split the (slot, chunk) list of each stretch, each adding w_tj * sum into a private [T][kDnRows]
// array, joined in warp order.  Columns that several blocks share go through the workspace: the last
// of these blocks to arrive adds their parts, in block order, so the result does not depend on timing.
__global__ void __launch_bounds__(kDnWarps * 32, 2) moe_few_down_kernel(MoeFewArgs a) {
  extern __shared__ float accw[];  // [kDnWarps][T][kDnRows]
  __shared__ int last;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
  const int P = a.T * a.k;
  const int n = a.lists[0];
  const int32_t* list = a.lists + kListHead;
  const int32_t* order = list + 3 * max_slots(P, a.E);
  int32_t* arrived = a.lists + kListHead + 3 * max_slots(P, a.E) + P;
  const int nch = (a.I + 127) / 128;
  const int64_t cb = (int64_t)a.H * a.I / 2, sb = (int64_t)a.H * a.I / 16;
  const int elems = a.T * kDnRows;
  const int groups = a.H / kDnRows;
  auto store = [&](int grp, int i, float v) {
    const int row = i % 16, tile = grp * kDnTiles + i % kDnRows / 16;
    const int col = 128 * (tile >> 3) + 32 * (row >> 2) + 4 * (tile & 7) + (row & 3);
    const __nv_bfloat16 b = __float2bfloat16_rn(v);
    a.out[(int64_t)(i / kDnRows) * a.ldo + col] = *reinterpret_cast<const uint16_t*>(&b);
  };
  if (n == 0) {  // no token could be routed
    for (int grp = blockIdx.x; grp < groups; grp += gridDim.x)
      for (int i = threadIdx.x; i < elems; i += kDnWarps * 32) store(grp, i, 0.0f);
    return;
  }
  const int64_t units = (int64_t)groups * n;
  const int64_t G = min((int64_t)gridDim.x, units);
  if (blockIdx.x >= G) return;
  auto bound = [&](int64_t b) { return units * b / G; };                       // first unit of block b
  auto block_of = [&](int64_t u) { return ((u + 1) * G - 1) / units; };        // the block that holds unit u
  int64_t u = bound(blockIdx.x);
  const int64_t u_end = bound(blockIdx.x + 1);
  float* mine = accw + warp * elems;
  for (int part = 0; u < u_end; ++part) {
    const int grp = (int)(u / n);
    const int s_lo = (int)(u - (int64_t)grp * n);
    const int s_hi = (int)min((int64_t)n, s_lo + (u_end - u));
    u += s_hi - s_lo;
    for (int i = lane; i < elems; i += 32) mine[i] = 0.0f;
    __syncwarp();
    const int todo = (s_hi - s_lo) * nch;
    int w0 = todo * warp / kDnWarps;
    const int w1 = todo * (warp + 1) / kDnWarps;
    int slot = s_lo + w0 / nch, c = w0 % nch;
    auto slot_ref = [&](int sl, int ch) {
      const int64_t e = __ldg(list + 3 * sl);
      TileRef r = tile_ref(a.dn_codes + e * cb, a.dn_sf + e * sb, grp * kDnTiles, a.I);
      r.codes += 64 * ch;
      r.sf += 1024 * ch;
      return r;
    };
    TileRef next;
    Chunk ring[kDnTiles];
    if (w0 < w1) {
      next = slot_ref(slot, c);
#pragma unroll
      for (int r = 0; r < kDnTiles; ++r) ring[r] = load_chunk(next, r, a.I, 128 * c + 32 * t < a.I);
    }
    while (w0 < w1) {
      const int c_end = min(nch, c + (w1 - w0));
      const int p0 = __ldg(list + 3 * slot + 1), cnt = __ldg(list + 3 * slot + 2) - p0;
      const float s_g = __ldg(a.dn_sg + __ldg(list + 3 * slot));
      const bool has = g < cnt;
      const float* hr = a.h + (int64_t)(has ? p0 + g : 0) * a.I + 32 * t;
      float acc[kDnTiles][4] = {};
      w0 += c_end - c;
      for (; c < c_end; ++c) {
        bool more = true;
        int cn = c + 1;
        if (cn < c_end) {
          next.codes += 64;
          next.sf += 1024;
        } else if (w0 < w1) {
          next = slot_ref(slot + 1, 0);
          cn = 0;
        } else {
          more = false;
        }
        const bool in = 128 * c + 32 * t < a.I, in_next = more && 128 * cn + 32 * t < a.I;
        uint32_t b[16];
        const float down = load_b_f32(hr + 128 * c, has && in, b) * s_g;
        const float d0 = __shfl_sync(0xffffffffu, down, 8 * t), d1 = __shfl_sync(0xffffffffu, down, 8 * t + 4);
#pragma unroll
        for (int r = 0; r < kDnTiles; ++r) {
          const Chunk k = ring[r];
          ring[r] = load_chunk(next, r, a.I, in_next);
          float pt[4] = {0.0f, 0.0f, 0.0f, 0.0f};
          mma_chunk(pt, k, b);
          acc[r][0] = fmaf(pt[0], d0, acc[r][0]);
          acc[r][1] = fmaf(pt[1], d1, acc[r][1]);
          acc[r][2] = fmaf(pt[2], d0, acc[r][2]);
          acc[r][3] = fmaf(pt[3], d1, acc[r][3]);
        }
      }
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int col = 2 * t + j;
        if (col < cnt) {
          const int p = __ldg(order + p0 + col);
          const float w = __ldg(a.topk_w + p);
          float* o = mine + (p / a.k) * kDnRows + g;  // a slot's tokens are distinct: no two lanes meet
#pragma unroll
          for (int r = 0; r < kDnTiles; ++r) {
            o[16 * r] = fmaf(w, acc[r][j], o[16 * r]);
            o[16 * r + 8] = fmaf(w, acc[r][2 + j], o[16 * r + 8]);
          }
        }
      }
      __syncwarp();
      ++slot;
      c = 0;
    }
    __syncthreads();
    const int64_t b0 = block_of((int64_t)grp * n), b1 = block_of((int64_t)grp * n + n - 1);
    if (b0 == b1) {
      for (int i = threadIdx.x; i < elems; i += kDnWarps * 32) {
        float v = 0.0f;
        for (int w = 0; w < kDnWarps; ++w) v += accw[w * elems + i];
        store(grp, i, v);
      }
    } else {
      // a block shares at most two groups of columns: the one that it enters in the middle (or
      // before its end) and the one that it leaves unfinished
      float* slot_out = a.partial + ((int64_t)blockIdx.x * 2 + (part > 0)) * elems;
      for (int i = threadIdx.x; i < elems; i += kDnWarps * 32) {
        float v = 0.0f;
        for (int w = 0; w < kDnWarps; ++w) v += accw[w * elems + i];
        __stcg(slot_out + i, v);
      }
      __threadfence();
      __syncthreads();
      if (threadIdx.x == 0) last = atomicAdd(arrived + grp, 1) == (int)(b1 - b0);
      __syncthreads();
      if (last) {
        __threadfence();
        for (int i = threadIdx.x; i < elems; i += kDnWarps * 32) {
          float v = 0.0f;
          for (int64_t b = b0; b <= b1; ++b) {
            // block b's part of this group: its first stretch, or its second where it began before
            const bool second = bound(b) < (int64_t)grp * n;
            v += __ldcg(a.partial + (b * 2 + second) * elems + i);
          }
          store(grp, i, v);
        }
      }
    }
    __syncthreads();
  }
}

size_t moe_few_list_words(int64_t T, int32_t k, int32_t E, int64_t H) {
  const int P = (int)(T * k);
  return (size_t)(kListHead + 3 * max_slots(P, E) + P + H / kDnRows);
}

constexpr int kDnMaxBlocks = 2 * 160;
size_t moe_few_partial_floats(int64_t T) { return (size_t)kDnMaxBlocks * 2 * (size_t)T * kDnRows; }

cudaError_t launch_moe_few(const MoeFewArgs& a, int num_sms, cudaStream_t st) {
  const int P = a.T * a.k;
  const int64_t slots = max_slots(P, a.E);
  const int64_t items = slots * (a.I / 8 / kTiles), room = 4 * (int64_t)num_sms;
  moe_few_gate_up_kernel<<<(unsigned)(items < room ? items : room), kWarps * 32, 0, st>>>(a);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  const int smem = kDnWarps * a.T * kDnRows * (int)sizeof(float);
  if (smem > 48 * 1024) {
    e = cudaFuncSetAttribute(moe_few_down_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
  }
  int64_t blocks = slots * (a.H / kDnRows);
  if (blocks > 2 * (int64_t)num_sms) blocks = 2 * (int64_t)num_sms;
  if (blocks > kDnMaxBlocks) blocks = kDnMaxBlocks;
  moe_few_down_kernel<<<(unsigned)blocks, kDnWarps * 32, smem, st>>>(a);
  return cudaGetLastError();
}

}  // namespace nvfp4
