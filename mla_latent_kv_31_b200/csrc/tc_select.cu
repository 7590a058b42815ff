// Scores of the choice of blocks (mla_paged_select) at the DeepSeek-V3 sizes on the tensor cores: for token t and
// block g, max_i s_i (x_i . y_g) with int8 codes x_i of the 128 query rows [q~_i | q^R_i] and y_g of the block's
// summary, times the summary's scale. The products are whole numbers (kind::i8, int32 accumulation): exact.
//
// A CTA takes tokens t, t + gridDim.y, ... and of each every gridDim.x-th tile of 128 blocks. Half of its warps take the
// token's tiles: they gather 128 summary rows (cp.async; the rows of a tile lie anywhere) and multiply, M = 128 blocks,
// N = 128 heads, K = 576 in 18 MMAs of K = 32; with the blocks on the lanes the maximum over the heads stays in a
// thread, and it is taken while the next tile is fetched. The other half quantise the next token's queries into
// the other of two buffers meanwhile (the first token's by all), so queries are read from HBM once per CTA.
// Bounds: a tile takes about 2.3 us, of which the gather's latency is 1.6; a token's codes take 5 us. With one token
// a CTA the chain lookup - queries - codes - tile - score.
#include <cuda_bf16.h>

#include "paged.cuh"
#include "sm100.cuh"
#include "tc_paged.cuh"

namespace mla {
namespace {

using namespace sm100;

constexpr int H = 128, DC = 512, DR = 64, W = DC + DR;
constexpr int TILE = 128;                       // blocks per tile
constexpr int kThreads = 512;                   // 8 warps for the tiles, 8 for the next token's codes
constexpr uint32_t KBOX = 128 * 128;            // [128 rows x 128 codes], 128-byte swizzle
// A row is 4.5 boxes wide: the two query buffers share a ninth box (codes 512 .. 575 in its left or right half).
constexpr uint32_t OFF_Q = 0;                                  // 2 x 4 boxes, then the shared one
constexpr uint32_t OFF_QH = OFF_Q + 8 * KBOX;
constexpr uint32_t OFF_Y = OFF_QH + KBOX;                      // 5 boxes
constexpr uint32_t OFF_SQ = OFF_Y + 5 * KBOX;                  // [2][128] scales of the queries
constexpr uint32_t OFF_BAR = OFF_SQ + 2 * H * 4;               // a barrier, TMEM address
constexpr uint32_t SMEM_BYTES = OFF_BAR + 32 + 1024;
static_assert(SMEM_BYTES <= 232448, "shared memory budget");
// The right half of the summaries' fifth box is free: chunk c (4 .. 7) of row r holds 16 bytes of what goes with block r
// of a tile: the summary's scale (4), the maximum over the upper 64 heads (5).
__device__ __forceinline__ uint32_t row_chunk(int r, int c) {
  return OFF_Y + 4 * KBOX + r * 128 + ((c ^ (r & 7)) << 4);
}

// kind::i8: signed 8-bit A and B, 32-bit integer D, both K-major.
constexpr uint32_t idesc_i8(int M, int N) {
  return (2u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}
__device__ __forceinline__ void mma_i8(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::i8 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}
// 16 bytes from global to shared memory, or zeros.
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool zero) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(zero ? 0 : 16) : "memory");
}

// x / s to the nearest whole number (ties to even) for 8 elements, as an IEEE division gives it: x * (1 / s) is within
// 3e-5 of the quotient for |x / s| <= 127, so only chunks with a value within 1e-4 of a tie (`rare`), or a scale whose
// reciprocal overflows, are divided (about every second row of bf16 numbers has such a value, half of its
// largest magnitude at 63.5). Adding 1.5 * 2^23 rounds to the nearest even whole number and leaves it, as two's
// complement, in the low byte.
__device__ __forceinline__ uint2 codes8(uint4 u, float inv, bool* rare) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
  uint32_t t[8];
  const uint64_t inv2 = f2_pack(inv, inv), magic = f2_pack(12582912.f, 12582912.f), unmagic = f2_pack(-12582912.f, -12582912.f);
  const uint64_t minus = f2_pack(-1.f, -1.f);
  float off = 0.f;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const uint64_t r = f2_mul(f2_pack(bf16_lo(w[e]), bf16_hi(w[e])), inv2);
    const uint64_t m = f2_add(r, magic);
    float m0, m1, d0, d1;
    f2_unpack(m, m0, m1);
    f2_unpack(f2_fma(f2_add(m, unmagic), minus, r), d0, d1);
    t[2 * e] = __float_as_uint(m0);
    t[2 * e + 1] = __float_as_uint(m1);
    off = fmaxf(off, fmaxf(fabsf(d0), fabsf(d1)));
  }
  *rare = off > 0.4999f;
  return make_uint2(__byte_perm(__byte_perm(t[0], t[1], 0x0040), __byte_perm(t[2], t[3], 0x0040), 0x5410),
                    __byte_perm(__byte_perm(t[4], t[5], 0x0040), __byte_perm(t[6], t[7], 0x0040), 0x5410));
}
// One code by IEEE division.
__device__ __forceinline__ uint8_t code_exact(float x, float s) {
  return (uint8_t)(int)fminf(fmaxf(rintf(__fdiv_rn(x, s)), -127.f), 127.f);
}
// The largest magnitude of 8 elements as the bits of a bf16, which order like the magnitudes, a NaN above all: the scale
// of a row with a NaN or an infinity is not finite, and its codes are zeros.
__device__ __forceinline__ uint32_t max8(uint4 u) {
  const uint32_t m = __vmaxu2(__vmaxu2(u.x & 0x7fff7fffu, u.y & 0x7fff7fffu), __vmaxu2(u.z & 0x7fff7fffu, u.w & 0x7fff7fffu));
  return max(m & 0xffffu, m >> 16);
}

// Where the 8 codes of chunk c (0 .. 71) of query row i go in buffer b.
__device__ __forceinline__ uint32_t place(int b, int i, int c) {
  return (c < 64 ? OFF_Q + (4 * b + (c >> 4)) * KBOX + i * 128 + ((((c & 15) >> 1) ^ (i & 7)) << 4)
                 : OFF_QH + i * 128 + (((4 * b + ((c & 15) >> 1)) ^ (i & 7)) << 4)) + (c & 1) * 8;
}
// Quantises ROWS query rows, the warp's own, of token t into buffer b: loads, then codes. Lane: the chunks of 8 elements
// lane and lane + 32 of each row, and q^R's chunk lane % 8 of rows lane / 8 and 4 + lane / 8.
constexpr int ROWS = 8;
struct QueryRows {
  uint4 u[ROWS][2], ur[2];
  __device__ __forceinline__ void load(const __nv_bfloat16* q_abs, const __nv_bfloat16* q_rope, int64_t t, int i0, int lane) {
    const uint4* qa = reinterpret_cast<const uint4*>(q_abs + (t * H + i0) * DC) + lane;
    const uint4* qr = reinterpret_cast<const uint4*>(q_rope + (t * H + i0) * DR) + lane;
#pragma unroll
    for (int j = 0; j < ROWS; ++j) {
      u[j][0] = qa[j * (DC / 8)];
      u[j][1] = qa[j * (DC / 8) + 32];
    }
    ur[0] = qr[0];
    ur[1] = qr[32];
  }
  __device__ __forceinline__ void codes(uint8_t* smem, const __nv_bfloat16* q_abs, const __nv_bfloat16* q_rope, int64_t t,
                                        int b, int i0, int lane) const {
    float* sq = reinterpret_cast<float*>(smem + OFF_SQ) + b * H;
    auto put = [&](int i, int c, uint2 x) { *reinterpret_cast<uint2*>(smem + place(b, i, c)) = x; };
    // the rows' largest magnitudes, all at once
    uint32_t big[ROWS];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint32_t mr = max8(ur[h]);
#pragma unroll
      for (int o = 1; o < 8; o <<= 1) mr = max(mr, __shfl_xor_sync(0xffffffffu, mr, o));
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int j = 4 * h + k;
        big[j] = max(__reduce_max_sync(0xffffffffu, max(max8(u[j][0]), max8(u[j][1]))), __shfl_sync(0xffffffffu, mr, 8 * k));
      }
    }
    float s[ROWS], inv[ROWS];
#pragma unroll
    for (int j = 0; j < ROWS; ++j) {
      s[j] = __fdiv_rn(__uint_as_float(big[j] << 16), 127.f);
      if (!(s[j] > 0.f && s[j] < INFINITY)) s[j] = 0.f;
      inv[j] = 1.f / s[j];
      if (lane == 0) sq[i0 + j] = s[j];
    }
    // chunk k of row j: bit 2 j + k; q^R's chunk of half h: bit 16 + h
    uint32_t again = 0;
#pragma unroll
    for (int j = 0; j < ROWS; ++j)
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        bool rare;
        const uint2 x = codes8(u[j][k], inv[j], &rare);
        put(i0 + j, lane + 32 * k, s[j] == 0.f ? make_uint2(0u, 0u) : x);
        if (rare || !(inv[j] < INFINITY)) again |= 1u << (2 * j + k);
      }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float sr = s[4 * h], ir = inv[4 * h];
#pragma unroll
      for (int k = 1; k < 4; ++k) {
        sr = (lane >> 3) == k ? s[4 * h + k] : sr;
        ir = (lane >> 3) == k ? inv[4 * h + k] : ir;
      }
      bool rare;
      const uint2 x = codes8(ur[h], ir, &rare);
      put(i0 + 4 * h + (lane >> 3), 64 + (lane & 7), sr == 0.f ? make_uint2(0u, 0u) : x);
      if (rare || !(ir < INFINITY)) again |= 1u << (16 + h);
    }
    __syncwarp();
    // the rare chunks: their elements near a tie once more, from the loads' cache
    while (again) {
      const int bit = __ffs(again) - 1;
      again &= again - 1;
      const int i = bit < 16 ? i0 + (bit >> 1) : i0 + 4 * (bit - 16) + (lane >> 3), c = bit < 16 ? lane + 32 * (bit & 1) : 64 + (lane & 7);
      const float si = sq[i];
      if (si == 0.f) continue;
      const __nv_bfloat16* src = c < 64 ? q_abs + (t * H + i) * DC + 8 * c : q_rope + (t * H + i) * DR + 8 * (c - 64);
      const uint4 v4 = *reinterpret_cast<const uint4*>(src);
      const uint32_t w[4] = {v4.x, v4.y, v4.z, v4.w};
      uint8_t* dst = smem + place(b, i, c);
#pragma unroll 1
      for (int e = 0; e < 8; ++e) {
        const uint32_t we = e < 4 ? (e < 2 ? w[0] : w[1]) : (e < 6 ? w[2] : w[3]);
        dst[e] = code_exact(e & 1 ? bf16_hi(we) : bf16_lo(we), si);
      }
    }
  }
};

__global__ void __launch_bounds__(kThreads, 1)
    select_score_kernel(PagedView v, const __nv_bfloat16* q_abs, const __nv_bfloat16* q_rope, const uint8_t* summaries,
                        int64_t pitch, int32_t top_k, float* scores, uint32_t* err) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = smem_addr(smem), bar = sbase + OFF_BAR;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const bool tiles_half = warp < 8;
  const int stride = gridDim.x, first = blockIdx.x;
  int64_t t = blockIdx.y;
  let_next_start();

  // blocks of a token, 0 when there is nothing to score for this CTA
  auto blocks_of = [&](const PagedToken& k) -> int {
    const int nb = k.pos < 0 ? 0 : (int)(k.pos / v.page) + 1;
    return nb > top_k && first * TILE < nb ? nb : 0;
  };
  {
    // the first token: all loads are in flight while it is looked up
    QueryRows q;
    q.load(q_abs, q_rope, t, ROWS * warp, lane);
    if (blockIdx.x == 0 && t == 0) paged_check(v, err);
    if (tid == 0) {
      mbar_init(bar, 1);
      fence_mbar_init();
    }
    if (warp == 0) {
      tmem_alloc(bar + 16, 128);
      tmem_relinquish();
    }
    q.codes(smem, q_abs, q_rope, t, 0, ROWS * warp, lane);
    fence_proxy_async_smem();
  }
  PagedToken tok = paged_token(v, t);
  int nb = blocks_of(tok);
  // The page of row 16 warp + lane % 16 of tile i of a token, -1 for none.
  auto page_of = [&](const PagedToken& k, int n_blocks, int i) -> int {
    const int g = (first + i * stride) * TILE + 16 * warp + (lane & 15);
    if (g >= n_blocks) return -1;
    const int p = v.table[(int64_t)k.seq * v.stride + g];
    if (p < 0 || p >= v.num_pages) {
      flag_error(err, DEVERR_PAGE);
      return -1;
    }
    return p;
  };
  // A tile's summary rows, 16 a warp: the first 512 bytes of a row by 32 lanes (contiguous: four times fewer L1 requests
  // than a few lanes a row), then the last 64 of eight rows at a time, then the scales.
  auto fetch = [&](int page) {
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      const int p = __shfl_sync(0xffffffffu, page, j), r = 16 * warp + j;
      copy16(sbase + OFF_Y + (lane >> 3) * KBOX + r * 128 + (((lane & 7) ^ (j & 7)) << 4),
             summaries + (int64_t)(p < 0 ? 0 : p) * pitch + 16 * lane, p < 0);
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int j = 8 * h + (lane >> 2), p = __shfl_sync(0xffffffffu, page, j), r = 16 * warp + j, c = lane & 3;
      copy16(sbase + OFF_Y + 4 * KBOX + r * 128 + ((c ^ (j & 7)) << 4),
             summaries + (int64_t)(p < 0 ? 0 : p) * pitch + 512 + 16 * c, p < 0);
    }
    if (lane < 16)
      asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(sbase + row_chunk(16 * warp + lane, 4)),
                   "l"(summaries + (int64_t)(page < 0 ? 0 : page) * pitch + W), "r"(page < 0 ? 0 : 4)
                   : "memory");
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  auto tiles_barrier = [&]() { asm volatile("bar.sync 1, 256;" ::: "memory"); };
  if (tiles_half && nb > 0) fetch(page_of(tok, nb, 0));
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<const uint32_t*>(smem + OFF_BAR + 16);
  const int quarter = warp & 3, cg = (warp >> 2) & 1;         // lanes 32 quarter .., heads 64 cg ..
  const int row = 32 * quarter + lane;
  constexpr uint32_t idesc = idesc_i8(TILE, H);
  uint32_t done = 0;                                          // tiles multiplied by this CTA
  bool ok = true;
  for (int b = 0; t < v.total_q; b ^= 1) {
    const int64_t t_next = t + gridDim.y;
    PagedToken tok_next;
    tok_next.seq = -1;
    tok_next.pos = -1;
    int nb_next = 0;
    if (!tiles_half) {
      // ---- the next token's codes, 16 rows a warp
      if (t_next < v.total_q) {
#pragma unroll 1
        for (int h = 0; h < 2; ++h) {
          QueryRows q;
          const int i0 = 2 * ROWS * (warp - 8) + ROWS * h;
          q.load(q_abs, q_rope, t_next, i0, lane);
          q.codes(smem, q_abs, q_rope, t_next, b ^ 1, i0, lane);
        }
        fence_proxy_async_smem();
      }
    } else {
      const int n = nb > 0 ? ((nb + TILE - 1) / TILE - first + stride - 1) / stride : 0;
      const float* sq = reinterpret_cast<const float*>(smem + OFF_SQ) + b * H + 64 * cg;
      int page_next = n > 1 ? page_of(tok, nb, 1) : -1;
      for (int i = 0; i < n && ok; ++i, ++done) {
        // the tile has landed and is visible to the MMAs; the maxima of the tile before are taken
        asm volatile("cp.async.wait_group 0;" ::: "memory");
        fence_proxy_async_smem();
        tc_fence_before();
        tiles_barrier();
        if (tid == 0) {
          tc_fence_after();
#pragma unroll
          for (int k = 0; k < 18; ++k) {
            const uint32_t q = k < 16 ? OFF_Q + (4 * b + (k >> 2)) * KBOX : OFF_QH;
            const int qo = k < 16 ? 2 * (k & 3) : 4 * b + 2 * (k - 16);
            mma_i8(tmem, sw128_desc(sbase + OFF_Y + (k >> 2) * KBOX, 0, 1024) + 2 * (k & 3),
                   sw128_desc(sbase + q, 0, 1024) + qo, idesc, k > 0 ? 1u : 0u);
          }
          mma_commit(bar);
        }
        const float scale = *reinterpret_cast<const float*>(smem + row_chunk(row, 4));
        if (i == 0 && t_next < v.total_q) {
          tok_next = paged_token(v, t_next);
          nb_next = blocks_of(tok_next);
        }
        const int page_after = i + 2 < n ? page_of(tok, nb, i + 2) : i + 1 == n && nb_next > 0 ? page_of(tok_next, nb_next, 0) : -1;
        // multiplied, and the scales are read: the buffer takes the next tile (or a wait gave up, for all of them)
        ok = !bar_sync_or(1, 256, !mbar_wait(bar, done & 1));
        tc_fence_after();
        if (!ok) break;
        if (i + 1 < n) fetch(page_next);
        else if (nb_next > 0) fetch(page_after);
        page_next = page_after;
        float mx = -INFINITY;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t x[32];
          tmem_ld32(tmem + ((uint32_t)(32 * quarter) << 16) + 64 * cg + 32 * h, x);
          tmem_wait_ld();
#pragma unroll
          for (int c = 0; c < 32; c += 4) {
            const float4 s4 = *reinterpret_cast<const float4*>(sq + 32 * h + c);
            mx = fmaxf(mx, fmaxf(fmaxf((float)(int)x[c] * s4.x, (float)(int)x[c + 1] * s4.y),
                                 fmaxf((float)(int)x[c + 2] * s4.z, (float)(int)x[c + 3] * s4.w)));
          }
        }
        float* upper = reinterpret_cast<float*>(smem + row_chunk(row, 5));
        if (cg == 1) *upper = mx;
        tc_fence_before();
        tiles_barrier();
        const int g = (first + i * stride) * TILE + row;
        if (cg == 0 && g < nb) scores[t * v.max_pages + g] = fmaxf(mx, *upper) * scale + 0.f;   // + 0: a -0 ties with a 0
      }
      if (n == 0 && t_next < v.total_q) {
        tok_next = paged_token(v, t_next);
        nb_next = blocks_of(tok_next);
        if (nb_next > 0) fetch(page_of(tok_next, nb_next, 0));
      }
    }
    // the codes are written, the tiles multiplied
    if (!__syncthreads_and(ok)) {
      if (tid == 0) flag_error(err, DEVERR_TIMEOUT);
      break;
    }
    t = t_next;
    tok = tok_next;
    nb = nb_next;
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");
  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, 128);
  }
}

}  // namespace

cudaError_t tc_select_scores(const PagedView& v, const void* q_abs, const void* q_rope, const void* summaries,
                             int32_t top_k, float* scores, int num_sms, uint32_t* err, cudaStream_t st) {
  // per device, so set at every call
  cudaError_t e = cudaFuncSetAttribute(select_score_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)SMEM_BYTES);
  if (e != cudaSuccess) return e;
  // one CTA an SM: a token's tiles are split over several where tokens are few, else a CTA takes several tokens
  const int64_t tiles = (v.max_pages + TILE - 1) / TILE;
  int64_t split = num_sms / v.total_q;
  split = split < 1 ? 1 : split > tiles ? tiles : split;
  const int64_t rows = v.total_q < num_sms ? v.total_q : num_sms;
  select_score_kernel<<<dim3((unsigned)split, (unsigned)rows), kThreads, SMEM_BYTES, st>>>(
      v, (const __nv_bfloat16*)q_abs, (const __nv_bfloat16*)q_rope, (const uint8_t*)summaries,
      (int64_t)summary_pitch(DC, DR), top_k, scores, err);
  note_launch();
  return cudaGetLastError();
}

}  // namespace mla
