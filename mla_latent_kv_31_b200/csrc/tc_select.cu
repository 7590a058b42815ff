// Scores of the choice of blocks (mla_paged_select) at the DeepSeek-V3 sizes on the tensor cores: for token t and
// block g, max_i s_i (x_i . y_g) with int8 codes x_i of the 128 query rows [q~_i | q^R_i] and y_g of the block's
// summary, times the summary's scale. The products are whole numbers (kind::i8, int32 accumulation): exact.
//
// Two kernels. select_codes_kernel quantises the query rows, a warp eight rows (their bytes bound it). In
// select_score_kernel a CTA keeps one tile of 128 blocks of a sequence in shared memory (gathered by cp.async: its rows lie
// anywhere) and runs over the sequence's tokens, whose codes stream in by TMA (80 KB each): M = 128 blocks, N = 128
// heads, K = 576 in 18 MMAs of K = 32. With the blocks on the lanes the maximum over the heads stays in a thread.
// A token and tile is 1152 cycles of MMAs (64 each, measured), 1300 of copies and 1024 of the XU's conversions of the
// sums to fp32, of which no two overlap wholly: 512 tokens over 2048 blocks take 60 us, 36 of them MMAs. (100 us with an
// elected lane and a wait of all lanes for each box of codes: 128 cycles an MMA.) 512 tokens over 512 blocks: codes 27 us
// (110 MB), scores 25, choice 14; 66 in one call.
// 4 tokens over 2048 blocks: 19 us, the latency of the three launches.
// (Quantising inside the scoring kernel, a token's codes kept and the tiles streamed past, took 94 us there: 5 us of
// arithmetic a token, and a gather's latency for every tile.)
#include <cuda_bf16.h>
#include <string.h>

#include "paged.cuh"
#include "sm100.cuh"
#include "tc_gemm.cuh"
#include "tc_paged.cuh"

namespace mla {
namespace {

using namespace sm100;

constexpr int H = 128, DC = 512, DR = 64, W = DC + DR;
constexpr int TILE = 128;                       // blocks per tile
constexpr int kThreads = 384;                   // warp 0: TMA, warp 1: MMAs, warps 4-11: maxima; all: the gather
constexpr int kBoxes = 5;                       // [128 rows x 128 codes] boxes of a row (the last one half full)
constexpr int RING = 8;                         // boxes of query codes in flight
constexpr uint32_t KBOX = 128 * 128;            // 128-byte swizzle
constexpr uint32_t OFF_Y = 0;
constexpr uint32_t OFF_RING = OFF_Y + kBoxes * KBOX;
constexpr uint32_t OFF_SY = OFF_RING + RING * KBOX;            // [128] scales of the summaries
constexpr uint32_t OFF_SQ = OFF_SY + TILE * 4;                 // [8 warps][2][64] scales of the queries
constexpr uint32_t OFF_PART = OFF_SQ + 8 * 2 * 64 * 4;         // [2][128] maxima over the upper 64 heads
constexpr uint32_t OFF_BAR = OFF_PART + 2 * TILE * 4;
enum : int { B_FULL = 0, B_EMPTY = B_FULL + RING, B_DFULL = B_EMPTY + RING, B_DFREE = B_DFULL + 2, NBAR = B_DFREE + 2 };
constexpr uint32_t SMEM_BYTES = OFF_BAR + 8 * NBAR + 16 + 1024;
static_assert(SMEM_BYTES <= 232448, "shared memory budget");

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

// Codes [T * 128][576] and scales [T * 128] of the query rows, 8 rows a warp, of the tokens with more than top_k blocks
// (2048 tokens with fewer: 26 us where quantising them all took 134). Four CTAs an SM hide the look at the token (3 us
// of 80 against three CTAs; the 8 bytes that spill cost less). Lane: the chunks of 8 elements lane and
// lane + 32 of each row, and q^R's chunk lane % 8 of rows lane / 8 and 4 + lane / 8.
constexpr int ROWS = 8, CODE_WARPS = 4;
__global__ void __launch_bounds__(32 * CODE_WARPS, 4)
    select_codes_kernel(PagedView v, const __nv_bfloat16* q_abs, const __nv_bfloat16* q_rope, int32_t top_k, int8_t* codes,
                        float* scales, uint32_t* err) {
  const int lane = threadIdx.x & 31;
  const int64_t r0 = ((int64_t)blockIdx.x * CODE_WARPS + (threadIdx.x >> 5)) * ROWS;
  let_next_start();
  if (blockIdx.x == 0) paged_check(v, err);
  if (paged_token(v, r0 / H).pos < (int64_t)top_k * v.page) return;      // every block that it sees is chosen
  uint4 u[ROWS][2], ur[2];
  const uint4* qa = reinterpret_cast<const uint4*>(q_abs + r0 * DC) + lane;
  const uint4* qr = reinterpret_cast<const uint4*>(q_rope + r0 * DR) + lane;
#pragma unroll
  for (int j = 0; j < ROWS; ++j) {
    u[j][0] = qa[j * (DC / 8)];
    u[j][1] = qa[j * (DC / 8) + 32];
  }
  ur[0] = qr[0];
  ur[1] = qr[32];
  auto put = [&](int j, int c, uint2 x) { *reinterpret_cast<uint2*>(codes + (r0 + j) * W + 8 * c) = x; };
  // the rows' largest magnitudes and scales, all at once
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
    if (lane == 0) scales[r0 + j] = s[j];
  }
  // chunk k of row j: bit 2 j + k; q^R's chunk of half h: bit 16 + h
  uint32_t again = 0;
#pragma unroll
  for (int j = 0; j < ROWS; ++j)
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      bool rare;
      const uint2 x = codes8(u[j][k], inv[j], &rare);
      put(j, lane + 32 * k, s[j] == 0.f ? make_uint2(0u, 0u) : x);
      if (s[j] != 0.f && (rare || !(inv[j] < INFINITY))) again |= 1u << (2 * j + k);
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
    put(4 * h + (lane >> 3), 64 + (lane & 7), sr == 0.f ? make_uint2(0u, 0u) : x);
    if (sr != 0.f && (rare || !(ir < INFINITY))) again |= 1u << (16 + h);
  }
  // the rare chunks by division
  while (again) {
    const int bit = __ffs(again) - 1;
    again &= again - 1;
    const int j = bit < 16 ? bit >> 1 : 4 * (bit - 16) + (lane >> 3), c = bit < 16 ? lane + 32 * (bit & 1) : 64 + (lane & 7);
    const __nv_bfloat16* src = c < 64 ? q_abs + (r0 + j) * DC + 8 * c : q_rope + (r0 + j) * DR + 8 * (c - 64);
    const uint4 x = *reinterpret_cast<const uint4*>(src);
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
    float sj = s[0];
#pragma unroll
    for (int k = 1; k < ROWS; ++k) sj = j == k ? s[k] : sj;
    uint8_t* dst = reinterpret_cast<uint8_t*>(codes) + (r0 + j) * W + 8 * c;
#pragma unroll 1
    for (int e = 0; e < 8; ++e) {
      const uint32_t we = e < 4 ? (e < 2 ? w[0] : w[1]) : (e < 6 ? w[2] : w[3]);
      dst[e] = code_exact(e & 1 ? bf16_hi(we) : bf16_lo(we), sj);
    }
  }
}

struct ScoreParams {
  CUtensorMap qmap;           // codes as [T * 128, 576] bytes, box {128, 128}
  PagedView v;
  const float* scales;        // [T * 128]
  const uint8_t* summaries;
  int64_t pitch;
  int32_t top_k, group;       // tokens per CTA
  float* scores;              // [T, max_pages]
  uint32_t* err;
  int32_t stall;              // test hook: the first CTA leaves out its first box of codes
};

__global__ void __launch_bounds__(kThreads, 1) select_score_kernel(const __grid_constant__ ScoreParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = smem_addr(smem);
  const PagedView& v = p.v;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int tile = blockIdx.x;
  auto bar = [&](int i) { return sbase + OFF_BAR + 8u * (uint32_t)i; };
  const uint32_t tmem_slot = bar(NBAR);
  if (tid == 0) {
    for (int i = 0; i < NBAR; ++i) mbar_init(bar(i), i >= B_DFREE ? 8 : 1);
    fence_mbar_init();
    prefetch_tmap(&p.qmap);
  }
  if (warp == 0) {
    tmem_alloc(tmem_slot, 256);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<const uint32_t*>(smem + OFF_BAR + 8 * NBAR);
  let_next_start();

  float* sy = reinterpret_cast<float*>(smem + OFF_SY);
  const int quarter = warp & 3, cg = warp >= 8 ? 1 : 0;       // lanes 32 quarter .., heads 64 cg .. (warps 4-11)
  const int row = 32 * quarter + lane;
  bool ok = true, waited = false;
  uint32_t n = 0, done = 0;                                   // ring boxes and tokens so far, the same in every role
  const int64_t t_end = min((int64_t)(blockIdx.y + 1) * p.group, v.total_q);
  for (int64_t t = (int64_t)blockIdx.y * p.group; t < t_end;) {
    // a run: this CTA's tokens of one sequence, from the first with more than top_k blocks, some of them in this tile
    const PagedToken tok = paged_token(v, t);
    if (tok.seq < 0) break;
    const int64_t stop = tok.pos < 0 ? t + 1 : min(t_end, min(v.cu_q[tok.seq + 1], v.total_q));
    const int64_t need = (int64_t)max(p.top_k, tile * TILE) * v.page;      // the smallest position that is scored here
    const int64_t from = tok.pos < 0 ? stop : t + max((int64_t)0, need - tok.pos);
    const int64_t pos_from = tok.pos + (from - t);
    t = stop;
    if (from >= stop) continue;
    const int nb = (int)((pos_from + (stop - 1 - from)) / v.page) + 1;     // blocks of the run's last token
    // ---- the tile's summary rows: the first 512 bytes of a row by 32 lanes, then the last 64 of eight rows at a time,
    // then the scales; rows behind the last block and of pages outside the pool are zeros
    for (int r0 = 16 * warp; r0 < TILE; r0 += 16 * (kThreads / 32)) {
      const int g = tile * TILE + r0 + (lane & 15);
      int page = -1;
      if (g < nb) {
        page = v.table[(int64_t)tok.seq * v.stride + g];
        if (page < 0 || page >= v.num_pages) {
          flag_error(p.err, DEVERR_PAGE);
          page = -1;
        }
      }
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        const int q = __shfl_sync(0xffffffffu, page, j);
        copy16(sbase + OFF_Y + (lane >> 3) * KBOX + (r0 + j) * 128 + (((lane & 7) ^ (j & 7)) << 4),
               p.summaries + (int64_t)(q < 0 ? 0 : q) * p.pitch + 16 * lane, q < 0);
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int j = 8 * h + (lane >> 2), q = __shfl_sync(0xffffffffu, page, j), c = lane & 3;
        copy16(sbase + OFF_Y + 4 * KBOX + (r0 + j) * 128 + ((c ^ (j & 7)) << 4),
               p.summaries + (int64_t)(q < 0 ? 0 : q) * p.pitch + 512 + 16 * c, q < 0);
      }
      if (lane < 16) sy[r0 + lane] = page < 0 ? 0.f : *reinterpret_cast<const float*>(p.summaries + (int64_t)page * p.pitch + W);
    }
    asm volatile("cp.async.commit_group;\n\tcp.async.wait_group 0;" ::: "memory");
    fence_proxy_async_smem();
    if (!waited) wait_for_previous();                         // the codes
    waited = true;
    __syncthreads();
    const int cnt = (int)(stop - from);
    if (warp == 0) {
      // ---- codes
      for (int k = 0; ok && k < cnt; ++k)
        for (int e = 0; e < kBoxes; ++e, ++n) {
          const uint32_t slot = n % RING;
          ok = __all_sync(0xffffffffu, mbar_wait(bar(B_EMPTY + slot), ((n / RING) & 1) ^ 1)) != 0;
          if (!ok) break;
          if (elect_one()) {
            mbar_expect_tx(bar(B_FULL + slot), KBOX);
            if (!(p.stall && n == 0 && blockIdx.x == 0 && blockIdx.y == 0))
              tma_load_2d(sbase + OFF_RING + slot * KBOX, &p.qmap, 128 * e, (int32_t)((from + k) * H), bar(B_FULL + slot));
          }
          __syncwarp();
        }
    } else if (warp == 1) {
      // ---- products
      constexpr uint32_t idesc = idesc_i8(TILE, H);
      for (int k = 0; ok && k < cnt; ++k, ++done) {
        const uint32_t d = tmem + 128 * (done & 1);
        ok = __all_sync(0xffffffffu, mbar_wait(bar(B_DFREE + (done & 1)), ((done >> 1) & 1) ^ 1)) != 0;
        if (!ok) break;
        tc_fence_after();
        // one lane runs through the token's boxes, unrolled
        bool good = true;
        if (elect_one()) {
#pragma unroll
          for (int e = 0; e < kBoxes; ++e) {
            const uint32_t slot = (n + e) % RING;
            good = mbar_wait(bar(B_FULL + slot), ((n + e) / RING) & 1);
            if (!good) break;
            const uint64_t a = sw128_desc(sbase + OFF_Y + e * KBOX, 0, 1024), b = sw128_desc(sbase + OFF_RING + slot * KBOX, 0, 1024);
#pragma unroll
            for (int i = 0; i < (e < 4 ? 4 : 2); ++i) mma_i8(d, a + 2 * i, b + 2 * i, idesc, (e | i) ? 1u : 0u);
            mma_commit(bar(B_EMPTY + slot));
          }
          if (good) mma_commit(bar(B_DFULL + (done & 1)));
        }
        n += kBoxes;
        ok = __all_sync(0xffffffffu, good) != 0;
      }
    } else if (warp >= 4) {
      // ---- maxima: thread = block, 64 heads; the two warps of a block of 32 lanes meet once a token
      float* part = reinterpret_cast<float*>(smem + OFF_PART);
      float* sq = reinterpret_cast<float*>(smem + OFF_SQ) + 128 * (warp - 4);
      const float scale = sy[row];
      const float2* src = reinterpret_cast<const float2*>(p.scales + from * H + 64 * cg) + lane;
      float2 s_next = *src;
      for (int k = 0; ok && k < cnt; ++k, ++done) {
        float* sqb = sq + 64 * (done & 1);
        reinterpret_cast<float2*>(sqb)[lane] = s_next;
        if (k + 1 < cnt) s_next = src[(k + 1) * (H / 2)];
        __syncwarp();
        const bool full = __all_sync(0xffffffffu, mbar_wait(bar(B_DFULL + (done & 1)), (done >> 1) & 1)) != 0;
        float mx = -INFINITY;
        if (full) {
          tc_fence_after();
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            uint32_t x[32];
            tmem_ld32(tmem + ((uint32_t)(32 * quarter) << 16) + 128 * (done & 1) + 64 * cg + 32 * h, x);
            tmem_wait_ld();
#pragma unroll
            for (int c = 0; c < 32; c += 4) {
              const float4 s4 = *reinterpret_cast<const float4*>(sqb + 32 * h + c);
              mx = fmaxf(mx, fmaxf(fmaxf((float)(int)x[c] * s4.x, (float)(int)x[c + 1] * s4.y),
                                   fmaxf((float)(int)x[c + 2] * s4.z, (float)(int)x[c + 3] * s4.w)));
            }
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(B_DFREE + (done & 1)));
        }
        float* pb = part + TILE * (done & 1);
        if (cg == 1) pb[row] = mx;
        ok = !bar_sync_or(1 + quarter, 64, !full);
        const int64_t g = (int64_t)tile * TILE + row;
        if (ok && cg == 0 && g <= (pos_from + k) / v.page)
          p.scores[(from + k) * v.max_pages + g] = fmaxf(mx, pb[row]) * scale + 0.f;   // + 0: a -0 ties with a 0
      }
    }
    // the roles agree on what went by; the tile's buffer takes the next run's
    if (warp == 0) done += cnt;
    if (warp >= 2) n += kBoxes * cnt;
    if (warp == 2 || warp == 3) done += cnt;
    if (!__syncthreads_and(ok)) {
      ok = false;
      break;
    }
  }
  if (!waited) wait_for_previous();                           // not complete before the codes are
  if (!ok && tid == 0) {
    flag_error(p.err, DEVERR_TIMEOUT);
    for (uint32_t i = n > RING ? n - RING : 0; i < n; ++i) mbar_wait(bar(B_FULL + i % RING), (i / RING) & 1);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, 256);
  }
}

size_t align1k(size_t x) { return (x + 1023) / 1024 * 1024; }

}  // namespace

size_t tc_select_bytes(int64_t total_q, int64_t max_pages) {
  return align1k((size_t)total_q * max_pages * 4) + align1k((size_t)total_q * H * W) + align1k((size_t)total_q * H * 4);
}

cudaError_t tc_select_scores(const PagedView& v, const void* q_abs, const void* q_rope, const void* summaries,
                             int32_t top_k, void* ws, int num_sms, uint32_t* err, cudaStream_t st) {
  ScoreParams p;
  memset(&p, 0, sizeof(p));
  p.scores = (float*)ws;
  int8_t* codes = (int8_t*)ws + align1k((size_t)v.total_q * v.max_pages * 4);
  float* scales = (float*)(codes + align1k((size_t)v.total_q * H * W));
  cudaError_t e = make_tmap_u8(&p.qmap, codes, W, v.total_q * H, W, 128, 128);
  if (e != cudaSuccess) return e;
  // per device, so set at every call
  e = cudaFuncSetAttribute(select_score_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)SMEM_BYTES);
  if (e != cudaSuccess) return e;
  select_codes_kernel<<<(unsigned)(v.total_q * H / (ROWS * CODE_WARPS)), 32 * CODE_WARPS, 0, st>>>(
      v, (const __nv_bfloat16*)q_abs, (const __nv_bfloat16*)q_rope, top_k, codes, scales, err);
  note_launch();
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  p.v = v;
  p.scales = scales;
  p.summaries = (const uint8_t*)summaries;
  p.pitch = (int64_t)summary_pitch(DC, DR);
  p.top_k = top_k;
  p.err = err;
  p.stall = take_paged_stall();
  // one CTA an SM and about two rounds of them: more tokens a CTA gather a tile's summaries less often (512 tokens x 512
  // blocks: 3 rounds 89 us, 2 rounds 80, 1 round 79), fewer balance tiles behind a sequence's end and single tokens of
  // many sequences (64 x 1 over 512 blocks: 2 rounds 37, 1 round 41)
  const int64_t tiles = (v.max_pages + TILE - 1) / TILE;
  const int64_t group = (v.total_q * tiles + 2 * num_sms - 1) / (2 * num_sms);
  p.group = (int32_t)(group < 1 ? 1 : group);
  return launch_next(select_score_kernel, dim3((unsigned)tiles, (unsigned)((v.total_q + p.group - 1) / p.group)), kThreads,
                     SMEM_BYTES, st, p);
}

}  // namespace mla
