// Kernels of the paged latent cache that need no matrix unit: the append with the position rotation on the
// way, the pages' summaries, the choice of blocks, and the attention of the fp32 configuration.
#include <cuda_bf16.h>
#include <math.h>

#include "paged.cuh"
#include "tc_paged.cuh"

namespace mla {
namespace {

__device__ __forceinline__ void rope_angle(const RopeTable& rt, const LayerOpts& o, int64_t pos, int m, int d_r,
                                           float* c, float* s) {
  // the angle in double: a position of 2^17 turns the first pair by 2^17 radians
  const double theta = m < kRopeTablePairs ? rt.theta[m] : rope_theta(o.rope, m, d_r);
  double sd, cd;
  sincos((double)pos * theta, &sd, &cd);
  *c = (float)cd;
  *s = (float)sd;
}

// ---- append -----------------------------------------------------------------------------------------------
// One block per new token: its row [c | R_pos k] into its page and, with q, its n_h rotated queries. The bytes bound it
// for long chunks (a token's 2 x 1152 + 2 x 16384 at the DeepSeek-V3 sizes), the chain lookup - sine - store else,
// so every load is issued before the lookup and the angles (in double) are taken by one warp. With the summaries, 16
// tokens take 8.5 us; five chunks of 2703 tokens together 25 us (95 MB: 3.8 TB/s).
__device__ __forceinline__ uint4 rotate8(uint4 u, const float2* cs, float mul) {       // 4 pairs of bf16
  uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float x0 = __uint_as_float(w[e] << 16), x1 = __uint_as_float(w[e] & 0xffff0000u);
    const __nv_bfloat162 y = __floats2bfloat162_rn((x0 * cs[e].x - x1 * cs[e].y) * mul, (x0 * cs[e].y + x1 * cs[e].x) * mul);
    w[e] = *reinterpret_cast<const uint32_t*>(&y);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

constexpr int AP_THREADS = 256;
constexpr int AP_H = 128, AP_DC = 512, AP_DR = 64;
__global__ void __launch_bounds__(AP_THREADS)
    append_bf16_kernel(PagedView v, const __nv_bfloat16* kv, int64_t kv_stride, const __nv_bfloat16* q,
                       __nv_bfloat16* q_out, LayerOpts o, RopeTable rt, uint32_t* err) {
  __shared__ float2 cs[AP_DR / 2];
  __shared__ float red[32];
  constexpr int QC = AP_H * AP_DR / 8 / AP_THREADS;          // 16-byte chunks of the queries per thread
  let_next_start();
  const int tid = threadIdx.x;
  const int64_t t = blockIdx.x;
  uint4 uq[QC], uk = make_uint4(0u, 0u, 0u, 0u);
  const uint4* qs = reinterpret_cast<const uint4*>(q + t * AP_H * AP_DR);
  if (q) {
#pragma unroll
    for (int k = 0; k < QC; ++k) uq[k] = qs[tid + k * AP_THREADS];
  }
  const bool has_row = tid < (AP_DC + AP_DR) / 8;
  if (has_row) uk = reinterpret_cast<const uint4*>(kv + t * kv_stride)[tid];
  if (t == 0) paged_check(v, err);
  const PagedToken tok = paged_token(v, t);
  if (tok.pos < 0) {
    if (q && tok.seq >= 0) {                                 // an empty row
      uint4* qd = reinterpret_cast<uint4*>(q_out + t * AP_H * AP_DR);
#pragma unroll
      for (int k = 0; k < QC; ++k) qd[tid + k * AP_THREADS] = make_uint4(0u, 0u, 0u, 0u);
    }
    return;
  }
  const int64_t page = paged_page(v, tok.seq, tok.pos / v.page, err);
  if (tid < AP_DR / 2) rope_angle(rt, o, tok.pos, tid, AP_DR, &cs[tid].x, &cs[tid].y);
  float inv = 1.f;
  if (o.g_kv) {
    float ss = 0.f;
    if (tid < AP_DC / 8) {
      const uint32_t w[4] = {uk.x, uk.y, uk.z, uk.w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float x0 = __uint_as_float(w[e] << 16), x1 = __uint_as_float(w[e] & 0xffff0000u);
        ss = fmaf(x0, x0, fmaf(x1, x1, ss));
      }
    }
    inv = 1.f / sqrtf(block_sum(ss, red) / (float)AP_DC + o.eps);
  }
  __syncthreads();
  if (has_row && page >= 0) {
    uint4* row = reinterpret_cast<uint4*>(reinterpret_cast<__nv_bfloat16*>(v.cache) +
                                          (page * v.page + tok.pos % v.page) * (AP_DC + AP_DR));
    if (tid >= AP_DC / 8) {
      uk = rotate8(uk, cs + 4 * (tid - AP_DC / 8), rt.mul);
    } else if (o.g_kv) {
      const uint4 g = reinterpret_cast<const uint4*>(o.g_kv)[tid];
      uint32_t w[4] = {uk.x, uk.y, uk.z, uk.w};
      const uint32_t gw[4] = {g.x, g.y, g.z, g.w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const __nv_bfloat162 y = __floats2bfloat162_rn(
            __uint_as_float(w[e] << 16) * inv * __uint_as_float(gw[e] << 16),
            __uint_as_float(w[e] & 0xffff0000u) * inv * __uint_as_float(gw[e] & 0xffff0000u));
        w[e] = *reinterpret_cast<const uint32_t*>(&y);
      }
      uk = make_uint4(w[0], w[1], w[2], w[3]);
    }
    row[tid] = uk;
  }
  if (q) {
    uint4* qd = reinterpret_cast<uint4*>(q_out + t * AP_H * AP_DR);
    const float2* c = cs + 4 * (tid & 7);                    // AP_THREADS is a multiple of a head's 8 chunks
#pragma unroll
    for (int k = 0; k < QC; ++k) qd[tid + k * AP_THREADS] = rotate8(uq[k], c, rt.mul);
  }
}

// The fp32 configuration, any sizes.
__global__ void __launch_bounds__(128)
    append_kernel(PagedView v, const float* kv, int64_t kv_stride, const float* q, float* q_out, LayerOpts o,
                  RopeTable rt, uint32_t* err) {
  extern __shared__ float2 cs[];      // [d_r / 2] cos, sin
  __shared__ float red[32];
  let_next_start();
  const int tid = threadIdx.x;
  const int64_t t = blockIdx.x;
  if (t == 0) paged_check(v, err);
  const PagedToken tok = paged_token(v, t);
  if (tok.pos < 0) {
    if (q && tok.seq >= 0)                                   // an empty row
      for (int i = tid; i < v.n_h * v.d_r; i += blockDim.x) q_out[t * v.n_h * v.d_r + i] = 0.f;
    return;
  }
  const int64_t page = paged_page(v, tok.seq, tok.pos / v.page, err);
  for (int m = tid; m < v.d_r / 2; m += blockDim.x) rope_angle(rt, o, tok.pos, m, v.d_r, &cs[m].x, &cs[m].y);
  __syncthreads();
  const float* src = kv + t * kv_stride;
  if (page >= 0) {
    float* row = reinterpret_cast<float*>(v.cache) + (page * v.page + tok.pos % v.page) * (v.d_c + v.d_r);
    float inv = 1.f;
    if (o.g_kv) {
      float ss = 0.f;
      for (int c = tid; c < v.d_c; c += blockDim.x) ss = fmaf(src[c], src[c], ss);
      inv = 1.f / sqrtf(block_sum(ss, red) / (float)v.d_c + o.eps);
    }
    for (int c = tid; c < v.d_c; c += blockDim.x)
      row[c] = o.g_kv ? src[c] * inv * reinterpret_cast<const float*>(o.g_kv)[c] : src[c];
    for (int m = tid; m < v.d_r / 2; m += blockDim.x) {
      const float x0 = src[v.d_c + 2 * m], x1 = src[v.d_c + 2 * m + 1];
      row[v.d_c + 2 * m] = (x0 * cs[m].x - x1 * cs[m].y) * rt.mul;
      row[v.d_c + 2 * m + 1] = (x0 * cs[m].y + x1 * cs[m].x) * rt.mul;
    }
  }
  if (!q) return;
  const int64_t base = t * v.n_h * v.d_r;
  for (int i = tid; i < v.n_h * (v.d_r / 2); i += blockDim.x) {
    const float2 w = cs[i % (v.d_r / 2)];
    const float x0 = q[base + 2 * i], x1 = q[base + 2 * i + 1];
    q_out[base + 2 * i] = (x0 * w.x - x1 * w.y) * rt.mul;
    q_out[base + 2 * i + 1] = (x0 * w.y + x1 * w.x) * rt.mul;
  }
}

// The scale and one code of a row: x / scale to the nearest whole number. The largest magnitude is taken over the bits, so
// that a NaN or an infinity wins: such a row, and one of zeros, has scale 0 and codes 0.
__device__ __forceinline__ uint32_t magnitude(float x) { return __float_as_uint(x) & 0x7fffffffu; }
__device__ __forceinline__ float code_scale(uint32_t largest) {
  const float s = __fdiv_rn(__uint_as_float(largest), 127.f);
  return s > 0.f && s < INFINITY ? s : 0.f;
}
__device__ __forceinline__ int code_of(float x, float s) {
  return s > 0.f ? (int)fminf(fmaxf(rintf(__fdiv_rn(x, s)), -127.f), 127.f) : 0;
}

// Summaries of the pages that the new tokens complete. Block i looks at `group` <= 32 tokens, a lane each; a token that is
// its page's last row stands for the page. The lookups come before the wait for the append's rows. Four groups of
// threads take a quarter of the rows each (page sizes are multiples of 16), 16 of them in flight; their sums meet in
// shared memory. The sums are in double and in a fixed order: a quarter's rows one after the other, then the quarters. Of
// bf16 values they are exact, and so free of the order, where a column's values span fewer than 45 - log2(page size)
// binades (53 bits of a double, 8 of a value), which rows of a latent cache do.
constexpr int SUM_GROUPS = 4;
template <typename T>
__global__ void __launch_bounds__(512) summarise_kernel(PagedView v, int group, uint8_t* summaries, int64_t pitch) {
  extern __shared__ double part[];    // [SUM_GROUPS][W]
  __shared__ uint32_t largest;
  const int tid = threadIdx.x, W = v.d_c + v.d_r;
  int32_t own = -1;                   // the page that this lane's token completes
  {
    const int64_t t = (int64_t)blockIdx.x * group + (tid & 31);
    if ((tid & 31) < group && t < v.total_q && t < v.cu_q[v.B]) {
      const int64_t b = seq_of_token(v.cu_q, v.B, t), q0 = v.cu_q[b], n = v.cu_q[b + 1] - q0, len = v.kv_lens[b];
      const int64_t pos = len - n + (t - q0);
      if (t >= q0 && t - q0 < n && n <= len && len <= v.max_pages * v.page && pos >= 0 && (pos + 1) % v.page == 0) {
        own = v.table[b * v.stride + pos / v.page];
        if (own >= v.num_pages) own = -1;                     // flagged by the append
      }
    }
  }
  uint32_t pages = __ballot_sync(0xffffffffu, own >= 0);      // the same in every warp
  wait_for_previous();
  for (; pages; pages &= pages - 1) {
    const int32_t p = __shfl_sync(0xffffffffu, own, __ffs(pages) - 1);
    const T* rows = reinterpret_cast<const T*>(v.cache) + (int64_t)p * v.page * W;
    constexpr int E = sizeof(T) == 2 ? 8 : 1;     // columns per thread: 16 bytes of bf16 (W is a multiple of 8 there)
    const int cols = W / E, per = v.page / SUM_GROUPS;
    for (int i = tid; i < cols * SUM_GROUPS; i += blockDim.x) {
      const int g = i / cols, c = i % cols;
      const T* src = rows + (int64_t)g * per * W + c * E;
      double sum[E] = {};
      if constexpr (E == 8) {
        for (int r0 = 0; r0 < per; r0 += 16) {
          uint4 u[16];
#pragma unroll
          for (int r = 0; r < 16; ++r)
            if (r0 + r < per) u[r] = *reinterpret_cast<const uint4*>(src + (int64_t)(r0 + r) * W);
#pragma unroll
          for (int r = 0; r < 16; ++r)
            if (r0 + r < per) {
              const uint32_t w[4] = {u[r].x, u[r].y, u[r].z, u[r].w};
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                sum[2 * e] += (double)__uint_as_float(w[e] << 16);
                sum[2 * e + 1] += (double)__uint_as_float(w[e] & 0xffff0000u);
              }
            }
        }
      } else {
#pragma unroll 8
        for (int r = 0; r < per; ++r) sum[0] += (double)to_f(src[(int64_t)r * W]);
      }
#pragma unroll
      for (int e = 0; e < E; ++e) part[g * W + c * E + e] = sum[e];
    }
    if (tid == 0) largest = 0;
    __syncthreads();
    uint32_t own_max = 0;
    for (int c = tid; c < W; c += blockDim.x) {
      double sum = 0.0;
#pragma unroll
      for (int g = 0; g < SUM_GROUPS; ++g) sum += part[g * W + c];
      const float mean = (float)(sum / v.page);
      reinterpret_cast<float*>(part)[2 * c] = mean;          // in place of group 0's sum
      own_max = max(own_max, magnitude(mean));
    }
    own_max = __reduce_max_sync(0xffffffffu, own_max);
    if ((tid & 31) == 0) atomicMax(&largest, own_max);
    __syncthreads();
    const float s = code_scale(largest);
    uint8_t* out = summaries + (int64_t)p * pitch;
    for (int c = tid; c < pitch; c += blockDim.x)
      if (c < W) out[c] = (uint8_t)(int8_t)code_of(reinterpret_cast<float*>(part)[2 * c], s);
      else if (c >= W + 4) out[c] = 0;
    if (tid == 0) *reinterpret_cast<float*>(out + W) = s;
    __syncthreads();
  }
}

// ---- attention by CUDA cores --------------------------------------------------------------------------------
// The fp32 configuration (tcgen05 has no fp32 product): one block per (token, head). Rows come through shared memory,
// `chunk` at a time (what fits 64 KB), so that global reads are contiguous; two threads share a key's product, and
// the 256 threads split into groups of d_c threads that share the chunk's keys in P.V. Latency bounds it at small sizes:
// 9 sequences of 33 to 700 rows, 1 to 5 tokens each, d_c = 64 and 4 heads take 25 us.
constexpr int ATT = 256;
constexpr int ATT_SMEM = 65536;
__global__ void __launch_bounds__(ATT)
    paged_attention_kernel(PagedView v, const float* q_abs, const float* q_rope, const int32_t* blocks, int32_t top_k,
                           float scale, int32_t chunk, float* o_lat, float* lse, uint32_t* err) {
  extern __shared__ float rows[];     // [chunk][W | 1]
  __shared__ float qs[1024];
  __shared__ float ps[ATT / 2];
  __shared__ int64_t row_of[ATT / 2];
  __shared__ float acc_sh[ATT];
  __shared__ float red[32];
  __shared__ int list_scratch[2];
  const int64_t t = blockIdx.x;
  const int head = blockIdx.y, tid = threadIdx.x, W = v.d_c + v.d_r, ld = W | 1;
  if (t == 0 && head == 0) paged_check(v, err);
  const PagedToken tok = paged_token(v, t);
  if (tok.seq < 0) return;
  const int32_t* list = blocks ? blocks + t * top_k : nullptr;
  int64_t n = tok.pos + 1;
  if (list) n = tok.pos < 0 ? 0 : paged_list_rows(list, top_k, tok.pos, v.page, list_scratch, err);
  const int64_t oq = t * v.n_h + head;
  for (int c = tid; c < W; c += ATT) qs[c] = c < v.d_c ? q_abs[oq * v.d_c + c] : q_rope[oq * v.d_r + c - v.d_c];
  const float* cache = reinterpret_cast<const float*>(v.cache);
  const bool vec = W % 4 == 0;        // rows start on 16 bytes
  // P.V: group kg of G takes the keys kg, kg + G, ...; with d_c > ATT a thread takes columns col, col + ATT
  const int width = min(v.d_c, ATT), G = ATT / width, kg = tid / width, col = tid % width;
  float m = -INFINITY, l = 0.f, acc[2] = {0.f, 0.f};
  for (int64_t c0 = 0; c0 < n; c0 += chunk) {
    const int cnt = (int)min((int64_t)chunk, n - c0);
    for (int j = tid; j < cnt; j += ATT) {
      const int64_t k = c0 + j;
      const int64_t page = paged_page(v, tok.seq, list ? list[k / v.page] : k / v.page, err);
      row_of[j] = page < 0 ? -1 : page * v.page + k % v.page;
    }
    __syncthreads();
    // a warp a row, four rows in flight; a page outside the pool counts as rows of zeros
    const int lane = tid & 31;
    for (int j0 = tid >> 5; j0 < cnt; j0 += 4 * (ATT / 32)) {
      if (vec) {
        for (int c = lane; c < W / 4; c += 32) {
          float4 u[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int j = j0 + k * (ATT / 32);
            u[k] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (j < cnt && row_of[j] >= 0) u[k] = reinterpret_cast<const float4*>(cache + row_of[j] * W)[c];
          }
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int j = j0 + k * (ATT / 32);
            if (j >= cnt) break;
            float* dst = rows + j * ld + 4 * c;
            dst[0] = u[k].x; dst[1] = u[k].y; dst[2] = u[k].z; dst[3] = u[k].w;
          }
        }
      } else {
        for (int k = 0; k < 4; ++k) {
          const int j = j0 + k * (ATT / 32);
          if (j >= cnt) break;
          for (int c = lane; c < W; c += 32) rows[j * ld + c] = row_of[j] < 0 ? 0.f : cache[row_of[j] * W + c];
        }
      }
    }
    __syncthreads();
    const int j = tid >> 1;
    float s = -INFINITY;
    {
      // four chains of sums per thread, then the neighbour's half
      const int half = (W + 1) / 2, lo = (tid & 1) * half, hi = min(W, lo + half);
      const float* k = rows + min(j, cnt - 1) * ld;
      float d[4] = {0.f, 0.f, 0.f, 0.f};
      int c = lo;
#pragma unroll 4
      for (; c + 3 < hi; c += 4) {
#pragma unroll
        for (int e = 0; e < 4; ++e) d[e] = fmaf(qs[c + e], k[c + e], d[e]);
      }
      for (; c < hi; ++c) d[0] = fmaf(qs[c], k[c], d[0]);
      float d0 = (d[0] + d[1]) + (d[2] + d[3]);
      d0 += __shfl_xor_sync(0xffffffffu, d0, 1);
      if (j < cnt) s = d0 * scale;
    }
    const float m_new = fmaxf(m, block_max(s, red));
    const float base = m_new == -INFINITY ? 0.f : m_new;        // (no score above -inf so far: weights of 0, a NaN stays)
    const float alpha = m == -INFINITY ? 0.f : __expf(m - m_new);
    const float p = j < cnt ? __expf(s - base) : 0.f;
    if ((tid & 1) == 0 && j < cnt) ps[j] = p;
    l = l * alpha + block_sum((tid & 1) == 0 ? p : 0.f, red);
    acc[0] *= alpha;
    acc[1] *= alpha;
    __syncthreads();
    if (kg < G) {
#pragma unroll 8
      for (int jj = kg; jj < cnt; jj += G) {
        const float pj = ps[jj];
        acc[0] = fmaf(pj, rows[jj * ld + col], acc[0]);
        if (col + ATT < v.d_c) acc[1] = fmaf(pj, rows[jj * ld + col + ATT], acc[1]);
      }
    }
    m = m_new;
    __syncthreads();
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;                   // (l = 0: no rows, or every score -inf)
  acc_sh[tid] = acc[0];
  __syncthreads();
  if (kg == 0) {
    float sum = acc[0];
    for (int g = 1; g < G; ++g) sum += acc_sh[g * width + col];
    o_lat[oq * v.d_c + col] = sum * inv;
    if (col + ATT < v.d_c) o_lat[oq * v.d_c + col + ATT] = acc[1] * inv;
  }
  if (tid == 0) lse[oq] = l == 0.f ? -INFINITY : m + logf(l);
}

// ---- selection ----------------------------------------------------------------------------------------------
// Codes and scale of each fp32 query row [q~_i | q^R_i] (one warp per row); bf16 takes tc_select.cu.
__global__ void __launch_bounds__(256)
    query_codes_kernel(PagedView v, const float* q_abs, const float* q_rope, int8_t* codes, float* scales, uint32_t* err) {
  if (blockIdx.x == 0) paged_check(v, err);
  const int64_t r = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31, W = v.d_c + v.d_r;
  if (r >= v.total_q * v.n_h || r / v.n_h >= v.cu_q[v.B]) return;
  auto at = [&](int c) { return c < v.d_c ? q_abs[r * v.d_c + c] : q_rope[r * v.d_r + c - v.d_c]; };
  uint32_t largest = 0;
  for (int c = lane; c < W; c += 32) largest = max(largest, magnitude(at(c)));
  const float s = code_scale(__reduce_max_sync(0xffffffffu, largest));
  for (int c = lane; c < W; c += 32) codes[r * W + c] = (int8_t)code_of(at(c), s);
  if (lane == 0) scales[r] = s;
}

// Scores of 32 blocks for one token: lane = block, the warps share the heads.
constexpr int SCORE_WARPS = 8;
__global__ void __launch_bounds__(32 * SCORE_WARPS)
    score_kernel(PagedView v, const int8_t* codes, const float* scales, const uint8_t* summaries, int64_t pitch,
                 int32_t top_k, float* scores, uint32_t* err) {
  extern __shared__ int32_t ksh[];    // [32][W / 4 | 1]
  let_next_start();
  __shared__ float best[SCORE_WARPS][32];
  const int64_t t = blockIdx.y;
  const PagedToken tok = paged_token(v, t);
  if (tok.pos < 0) return;
  const int64_t nb = tok.pos / v.page + 1, g0 = (int64_t)blockIdx.x * 32;
  if (nb <= top_k || g0 >= nb) return;
  const int W4 = (v.d_c + v.d_r) / 4, ld = W4 | 1, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (int i = warp; i < 32; i += SCORE_WARPS) {
    const int64_t g = g0 + i;
    const int64_t p = g < nb ? paged_page(v, tok.seq, g, err) : -1;
    const int32_t* src = reinterpret_cast<const int32_t*>(summaries + (p < 0 ? 0 : p) * pitch);
    for (int c = lane; c < W4; c += 32) ksh[i * ld + c] = p < 0 ? 0 : src[c];
  }
  __syncthreads();
  float mx = -INFINITY;
  for (int h = warp; h < v.n_h; h += SCORE_WARPS) {
    const int32_t* q = reinterpret_cast<const int32_t*>(codes + (t * v.n_h + h) * 4 * W4);
    int d = 0;
    for (int c = 0; c < W4; ++c) d = __dp4a(q[c], ksh[lane * ld + c], d);
    mx = fmaxf(mx, (float)d * scales[t * v.n_h + h]);
  }
  best[warp][lane] = mx;
  __syncthreads();
  if (warp == 0 && g0 + lane < nb) {
#pragma unroll
    for (int w = 1; w < SCORE_WARPS; ++w) mx = fmaxf(mx, best[w][lane]);
    const int64_t g = g0 + lane;
    const int32_t p = v.table[(int64_t)tok.seq * v.stride + g];
    const float s = p < 0 || p >= v.num_pages ? 0.f : *reinterpret_cast<const float*>(summaries + p * pitch + 4 * W4);
    scores[t * v.max_pages + g] = mx * s + 0.f;       // + 0: a -0 ties with a 0
  }
}

// Order-preserving key of a float.
__device__ __forceinline__ uint32_t key_of(float x) {
  const uint32_t u = __float_as_uint(x);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// The chosen blocks of one token: the threshold two bits at a time (the largest key that more than `want` keys reach; the
// keys above three candidates are counted at once, until exactly `want` are), then an ordered write, each thread's
// stretch of blocks after one scan of the counts. (A histogram's atomics would serialise: the keys share their leading
// bits.) Latency bounds it, a pass costs about 0.3 us for 2048 blocks: with one bit a pass and a scan for every 512
// blocks the whole call took 22 us against 19 for 4 tokens over 2048 blocks, 44 against 36 for 2 over 8192.
// Up to kSelectKeys keys are kept in shared memory, more are read from L2 at every pass.
constexpr int kSelectThreads = 512, kSelectKeys = 8192;
__global__ void __launch_bounds__(kSelectThreads)
    select_kernel(PagedView v, const float* scores, int32_t top_k, int32_t n_first, int32_t n_last, int32_t* blocks) {
  __shared__ uint32_t keys[kSelectKeys];
  __shared__ uint32_t red[2][kSelectThreads / 32];
  __shared__ int4 wsum[2][kSelectThreads / 32];
  const int64_t t = blockIdx.x;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  constexpr int NW = kSelectThreads / 32;
  const PagedToken tok = paged_token(v, t);
  wait_for_previous();
  if (tok.seq < 0) return;
  int32_t* out = blocks + t * top_k;
  const int nb = tok.pos < 0 ? 0 : (int)(tok.pos / v.page) + 1;
  if (nb <= top_k) {
    for (int i = tid; i < top_k; i += kSelectThreads) out[i] = i < nb ? i : -1;
    return;
  }
  const int lo = n_first, hi = nb - n_last;           // candidates
  const int want = top_k - n_first - n_last;
  for (int i = tid; i < n_first; i += kSelectThreads) out[i] = i;
  for (int i = tid; i < n_last; i += kSelectThreads) out[top_k - n_last + i] = hi + i;
  if (want == 0) return;
  const float* sc = scores + t * v.max_pages;
  const bool held = hi - lo <= kSelectKeys;
  auto key = [&](int g) { return held ? keys[g - lo] : key_of(sc[g]); };
  uint32_t mn = 0xffffffffu, mx = 0;
  for (int g = lo + tid; g < hi; g += kSelectThreads) {
    const uint32_t k = key_of(sc[g]);
    if (held) keys[g - lo] = k;
    mn = min(mn, k);
    mx = max(mx, k);
  }
  mn = __reduce_min_sync(0xffffffffu, mn);
  mx = __reduce_max_sync(0xffffffffu, mx);
  if (lane == 0) {
    red[0][warp] = mn;
    red[1][warp] = mx;
  }
  __syncthreads();
  mn = __reduce_min_sync(0xffffffffu, red[0][lane & (NW - 1)]);
  mx = __reduce_max_sync(0xffffffffu, red[1][lane & (NW - 1)]);
  // keys agree above bit `top`
  const int top = mn == mx ? -1 : 31 - __clz(mn ^ mx);
  uint32_t thr = top < 0 ? mx : top == 31 ? 0u : mx & ~((2u << top) - 1u);
  int par = 0;
  auto count = [&](uint32_t c1, uint32_t c2, uint32_t c3) -> int3 {        // keys >= each of them
    int n1 = 0, n2 = 0, n3 = 0;
    for (int g = lo + tid; g < hi; g += kSelectThreads) {
      const uint32_t k = key(g);
      n1 += k >= c1;
      n2 += k >= c2;
      n3 += k >= c3;
    }
    n1 = __reduce_add_sync(0xffffffffu, n1);
    n2 = __reduce_add_sync(0xffffffffu, n2);
    n3 = __reduce_add_sync(0xffffffffu, n3);
    if (lane == 0) wsum[par][warp] = make_int4(n1, n2, n3, 0);
    __syncthreads();
    const int4 x = lane < NW ? wsum[par][lane] : make_int4(0, 0, 0, 0);
    par ^= 1;                                          // the next count writes the other row
    return make_int3(__reduce_add_sync(0xffffffffu, x.x), __reduce_add_sync(0xffffffffu, x.y),
                     __reduce_add_sync(0xffffffffu, x.z));
  };
  int left = -1;                                       // of the keys equal to thr, the first `left` are taken
  for (int bit = top | 1; bit > 0 && left < 0; bit -= 2) {     // (top even: bit top + 1 is the same in all keys)
    const uint32_t c1 = thr | (1u << (bit - 1)), c2 = thr | (1u << bit), c3 = c1 | c2;
    const int3 c = count(c1, c2, c3);
    if (c.x == want || c.y == want || c.z == want) {   // exactly the keys above a candidate - 1
      thr = (c.x == want ? c1 : c.y == want ? c2 : c3) - 1;
      left = 0;
    } else if (c.y > want) {
      thr = c.z > want ? c3 : c2;
    } else if (c.x > want) {
      thr = c1;
    }
  }
  if (left < 0) left = want - (thr == 0xffffffffu ? 0 : count(thr + 1, thr + 1, thr + 1).x);
  const int per = (hi - lo + kSelectThreads - 1) / kSelectThreads, g0 = min(hi, lo + tid * per), g1 = min(hi, g0 + per);
  int above = 0, equal = 0;                            // of this thread, then before it
  for (int g = g0; g < g1; ++g) {
    const uint32_t k = key(g);
    above += k > thr;
    equal += k == thr;
  }
  int a_sum = above, e_sum = equal;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int a = __shfl_up_sync(0xffffffffu, a_sum, o), e = __shfl_up_sync(0xffffffffu, e_sum, o);
    if (lane >= o) {
      a_sum += a;
      e_sum += e;
    }
  }
  if (lane == 31) wsum[par][warp] = make_int4(a_sum, e_sum, 0, 0);
  __syncthreads();
  const int4 x = wsum[par][lane & (NW - 1)];
  above = a_sum - above + __reduce_add_sync(0xffffffffu, lane < warp ? x.x : 0);
  equal = e_sum - equal + __reduce_add_sync(0xffffffffu, lane < warp ? x.y : 0);
  for (int g = g0; g < g1; ++g) {
    const uint32_t k = key(g);
    if (k > thr) out[n_first + above++ + min(equal, left)] = g;
    else if (k == thr && equal++ < left) out[n_first + above + equal - 1] = g;
  }
}

size_t align16(size_t x) { return (x + 15) / 16 * 16; }
size_t align1k(size_t x) { return (x + 1023) / 1024 * 1024; }

}  // namespace

size_t summary_pitch(int32_t d_c, int32_t d_r) { return align16((size_t)d_c + d_r + 4); }

cudaError_t paged_append(const PagedView& v, bool bf16, const void* kv, int64_t kv_stride, const void* q_rope,
                         void* q_out, void* summaries, const LayerOpts& o, const RopeTable& rope, uint32_t* err,
                         cudaStream_t st) {
  if (bf16)
    append_bf16_kernel<<<(unsigned)v.total_q, AP_THREADS, 0, st>>>(
        v, (const __nv_bfloat16*)kv, kv_stride, (const __nv_bfloat16*)q_rope, (__nv_bfloat16*)q_out, o, rope, err);
  else
    append_kernel<<<(unsigned)v.total_q, 128, (size_t)v.d_r * 4, st>>>(v, (const float*)kv, kv_stride, (const float*)q_rope,
                                                                      (float*)q_out, o, rope, err);
  note_launch();
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || !summaries) return e;
  // a token a block where they are few (each may complete a page), else about two blocks an SM
  const int group = (int)(v.total_q <= 296 ? 1 : v.total_q >= 32 * 296 ? 32 : (v.total_q + 295) / 296);
  const dim3 grid((unsigned)((v.total_q + group - 1) / group));
  const size_t smem = (size_t)SUM_GROUPS * (v.d_c + v.d_r) * sizeof(double);
  const int64_t pitch = (int64_t)summary_pitch(v.d_c, v.d_r);
  return bf16 ? launch_next(summarise_kernel<__nv_bfloat16>, grid, 288, smem, st, v, group, (uint8_t*)summaries, pitch)
              : launch_next(summarise_kernel<float>, grid, 512, smem, st, v, group, (uint8_t*)summaries, pitch);
}

cudaError_t paged_attention_simt(const PagedView& v, const void* q_abs, const void* q_rope, const int32_t* blocks,
                                 int32_t top_k, float scale, void* o_lat, float* lse, uint32_t* err, cudaStream_t st) {
  const size_t row = (size_t)((v.d_c + v.d_r) | 1) * 4;
  const int chunk = (int)(ATT_SMEM / row < ATT / 2 ? ATT_SMEM / row : ATT / 2);
  cudaError_t e = cudaFuncSetAttribute(paged_attention_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, ATT_SMEM);
  if (e != cudaSuccess) return e;
  paged_attention_kernel<<<dim3((unsigned)v.total_q, (unsigned)v.n_h), ATT, chunk * row, st>>>(
      v, (const float*)q_abs, (const float*)q_rope, blocks, top_k, scale, chunk, (float*)o_lat, lse, err);
  note_launch();
  return cudaGetLastError();
}

size_t paged_select_bytes(bool bf16, int32_t n_h, int32_t d_c, int32_t d_r, int64_t total_q, int64_t max_pages) {
  const size_t rows = (size_t)total_q * n_h, scores = align1k((size_t)total_q * max_pages * 4);
  return bf16 ? tc_select_bytes(total_q, max_pages) : scores + align1k(rows * (d_c + d_r)) + align1k(rows * 4);
}

cudaError_t paged_select(const PagedView& v, bool bf16, const void* q_abs, const void* q_rope, const void* summaries,
                         int32_t top_k, int32_t n_first, int32_t n_last, int32_t* blocks, void* ws, int num_sms,
                         uint32_t* err, cudaStream_t st) {
  float* scores = (float*)ws;
  cudaError_t e;
  if (bf16) {
    if ((e = tc_select_scores(v, q_abs, q_rope, summaries, top_k, ws, num_sms, err, st)) != cudaSuccess) return e;
  } else {
    const size_t rows = (size_t)v.total_q * v.n_h, W = (size_t)v.d_c + v.d_r;
    int8_t* codes = (int8_t*)ws + align1k((size_t)v.total_q * v.max_pages * 4);
    float* scales = (float*)(codes + align1k(rows * W));
    query_codes_kernel<<<(unsigned)((rows + 7) / 8), 256, 0, st>>>(v, (const float*)q_abs, (const float*)q_rope, codes,
                                                                   scales, err);
    note_launch();
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    score_kernel<<<dim3((unsigned)((v.max_pages + 31) / 32), (unsigned)v.total_q), 32 * SCORE_WARPS,
                   32 * ((W / 4) | 1) * 4, st>>>(v, codes, scales, (const uint8_t*)summaries,
                                                 (int64_t)summary_pitch(v.d_c, v.d_r), top_k, scores, err);
    note_launch();
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
  }
  return launch_next(select_kernel, dim3((unsigned)v.total_q), kSelectThreads, 0, st, v, (const float*)scores, top_k,
                     n_first, n_last, blocks);
}

}  // namespace mla
