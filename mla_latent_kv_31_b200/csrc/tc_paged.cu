// Attention over the paged latent cache at the DeepSeek-V3 sizes (n_h = 128, d_c = 512, d_h^R = 64): bf16,
// fp32 accumulation, tcgen05 + TMA. For new token t of sequence b and head i, over the rows j that t sees
// (0 .. pos, or those of its chosen blocks):
//   s_j = (q~_t,i . c_j + q^R_t,i . k^R_j) / sqrt(d_h + d_r),  o_t,i = sum_j softmax(s)_j c_j,  lse = log sum_j e^{s_j}.
//
// Shape of the work. One token's 128 heads against 256 keys at a time, by a pair of CTAs (cta_group::2, M = 128:
// 64 heads in each SM). O = P.C for 64 heads x 512 latent columns is 256 TMEM columns of each SM (an
// M = 128 pair accumulator keeps columns [0, N/2) in lanes 0-63 and [N/2, N) in lanes 64-127), which leaves
// 256 columns for two score buffers of 64 heads x 256 keys. So softmax, P and O of a head stay in one SM
// and nothing but the shared B operands crosses between the two: each CTA loads half of the keys for QK^T
// (128 keys x 576) and half of the latent columns for P.V (256 keys x 256): 272 KB per 256 keys, against
// 36 and 32 MMAs of N = 256. (An M = 128 pair MMA of K = 16 takes 64 cycles at N = 256, 32 at N = 128, measured: 4357 a
// step. The loads take about 4200 of 66 bytes a cycle and SM. With both under way a step takes 7000 to 8000.)
//
// What it reaches, in bursts of ten calls at 1965 MHz (a graph; under the power cap of a long row 8 to 20 % less). 512
// tokens of one sequence behind 32768 rows: 1520 TFLOP/s; 8 x 64 behind 16384 rows 1470 (1.59 ms), 64 x 4 behind 8192 rows
// 1200, 64 x 2 behind 16896 1155 (0.52 ms), the rows read once from HBM; 4 single tokens over 131072 rows 4.1 TB/s
// (148 us), 16 over 4096 rows 38 us: there the chain plan - first rows - last partial - merge takes half of the time.
// Where rows come from L2 a step takes 4600 cycles, MMAs and loads both near their rates. Where they come from HBM it
// takes 6500 to 8000. Single tokens share no rows, so there the bytes bound a step: 74 pairs x 256 rows x 1152 B at the
// 6.46 TB/s of a copy are 3.4 us, 6500 cycles at 1.92 GHz. Rows that several pairs share need fewer bytes a step and no
// unit is at its limit; how much of either is time in which a pair has too few rows on their way (its ring of 112 KB, and
// the fetches to L2, which go out beside the values only) has not been measured step by step.
// Measured and not kept: a ring and an issuing warp each for K and V (1184 -> 1041 TFLOP/s), waits for several entries at
// once (0 to 8 % slower), P handed over 64 keys at a time (5 % slower: each wait and commit of the MMA warp counts),
// 64 score columns a thread in registers (the same time, 128 registers instead of 94).
//
// Work split. Tokens are cut into units of a step's 256 keys; all units of all tokens, plus a fixed cost per token,
// are dealt to the pairs in equal contiguous ranges of at least kMinRange. A token that lies in one range is written by
// its pair; one that crosses ranges leaves an unnormalised fp32 partial per range, merged exactly by
// paged_combine_kernel. (The order in which tokens are dealt: order_of().)
//
// Pages. A step's 256 keys are 16 groups of 16 keys; each group's row in the pool comes from the block table (and
// the token's block list). TMA boxes are 64, 32 or 16 rows high, the largest that divides the page size, so a
// box never crosses a page; boxes past the last visible key read out of range, which fills zeros. Rows between the
// last visible key and its box's end may hold anything, even NaN: their scores are masked, and their value
// rows (at most two ring entries of a token's last step) are zeroed in shared memory before P.V.
//
// Roles (512 threads): warps 0, 2 and 3 fill the ring of 16 KB entries, every third entry each, in the order the
// MMAs take them (K of step j + 1 before V of step j; one thread issues a copy every 500 cycles or so, the copies
// take 270), and warp 2 loads a token's queries, in warp-uniform code with one elected lane at each copy; warp 1 of the
// leader CTA issues the MMAs, one elected lane a product (a lane-0 branch around the whole loop cost 650 cycles a
// ring entry, three times what the copies take); warps 4-11 are the softmax (thread = TMEM
// lane, two warps per lane quarter, 64 keys each) and rescale O when the running maximum has grown by 2^8; warps 12-15
// write O out while the next token's first step runs.
// Every wait is bounded (a timeout sets the error word and the role returns); that of the output warps, which lasts as
// long as a token's steps, by the steps' progress.
#include <cuda_bf16.h>
#include <string.h>

#include "paged.cuh"
#include "sm100.cuh"
#include "tc_gemm.cuh"
#include "tc_paged.cuh"

namespace mla {
namespace {

using namespace sm100;

constexpr int H = 128, DC = 512, DR = 64;
constexpr int HC = H / 2;                      // heads per CTA
constexpr int NK = 256;                        // keys per step
constexpr int UNIT = NK;                       // keys per unit of the work split
constexpr int GROUPS = NK / 16;                // a step's rows are looked up in groups of 16 keys
constexpr int kThreads = 512;
constexpr int kMaxPairs = 74;
constexpr int kStartUnits = 1;                 // a token's fixed cost (query load, epilogue), in units
// A pair's smallest range, in units and start costs: one token over 4096 rows takes 25 us with 2, 28 with 3, 31 with 4
// (49 when its 64-key quarters were dealt to 64 pairs); 16 over 512 rows take 22, 20 and 28.
constexpr int kMinRange = 2;
constexpr int64_t kPlanTokens = 64;            // tokens looked up in the plan's own launch
constexpr float kRescaleLog2 = 8.f;            // keep the running maximum until it grows by 2^8
constexpr int kEntriesK = 9, kEntriesV = 8;    // ring entries of a step: [128 keys x 64], 2 x [64 keys x 64]
constexpr int RING = 7;
constexpr uint32_t ENTRY = 16384, BOX = 8192;
constexpr uint32_t Q_BYTES = HC * (DC + DR) * 2;
constexpr uint32_t P_BYTES = HC * NK * 2;

constexpr uint32_t OFF_RED = 512;                                  // [2][4][64] floats: maxima of the four key blocks
constexpr uint32_t OFF_STAT = OFF_RED + 2 * 4 * HC * 4;            // [5][64] floats: sums of the four key blocks, maximum
constexpr uint32_t OFF_STEPS = OFF_STAT + 5 * HC * 4;              // steps whose scores warp 4 has taken
constexpr uint32_t OFF_Q = 4096;
constexpr uint32_t OFF_P = OFF_Q + Q_BYTES;
constexpr uint32_t OFF_RING = OFF_P + P_BYTES;
constexpr uint32_t SMEM_BYTES = OFF_RING + RING * ENTRY + 1024;
static_assert(OFF_STEPS + 4 <= OFF_Q, "statistics block");
static_assert(OFF_Q % 1024 == 0 && OFF_P % 1024 == 0 && OFF_RING % 1024 == 0, "swizzle atom alignment");
static_assert(SMEM_BYTES <= 232448, "shared memory budget");

enum : int {
  B_FULL = 0,                 // [RING] entry landed in both CTAs (leader; 1 + bytes)
  B_EMPTY = B_FULL + RING,    // [RING] entry's MMAs done (both CTAs)
  B_SFULL = B_EMPTY + RING,   // [2] scores ready (both CTAs)
  B_SFREE = B_SFULL + 2,      // [2] scores read (leader; 16 warps)
  B_PRDY = B_SFREE + 2,       // P written, O rescaled (leader; 16 warps)
  B_PVD = B_PRDY + 1,         // P.V of a step done (both CTAs)
  B_QFULL = B_PVD + 1,        // a token's queries landed in both CTAs (leader; 1 + bytes)
  B_QEMPTY = B_QFULL + 1,     // a token's last QK^T done (both CTAs)
  B_TMAX = B_QEMPTY + 1,      // [2] the four softmax warps of a block of 32 heads
  B_TAIL = B_TMAX + 2,        // the two entries with the last visible key landed in this CTA (2 + bytes)
  B_TRDY = B_TAIL + 1,        // ... and their rows behind it zeroed (leader; 16 warps)
  B_ODONE = B_TRDY + 1,       // a token's last P.V done (both CTAs)
  B_OFREE = B_ODONE + 1,      // O read out (leader; 8 warps)
  B_LRDY = B_OFREE + 1,       // a token's sums and maxima written (8 warps)
  B_LFREE = B_LRDY + 1,       // ... and read (4 warps)
  NBAR = B_LFREE + 1
};
static_assert(NBAR * 8 + 16 <= OFF_RED, "barrier block");

struct CoreParams {
  CUtensorMap kmap;           // the pool as [rows, 576], box {64, gran}
  CUtensorMap vmap;           // the pool as [9, rows, 64], box {64, gran, 2} (gran 64) or {64, gran, 1}
  CUtensorMap qmap, qrmap;    // q~ [T * 128, 512], q^R [T * 128, 64], box {64, 64}
  PagedView v;
  const int32_t* blocks;      // [T, top_k] chosen blocks; nullptr: all rows
  int32_t top_k, pairs;
  const int4* tinfo;          // [T] in the order of the walk: sequence, visible rows, token
  const int4* pinfo;          // [pairs]: first token, its first unit, last token, its end unit
  const int4* pfirst;         // [pairs]: the first token's tinfo
  __nv_bfloat16* o_lat;
  float* lse;
  float4* part_o;             // [2 * pairs][DC / 4][H]
  float2* part_ml;            // [2 * pairs][H]: maximum (natural units), sum
  float scale_log2;
  uint32_t* err;
  int32_t stall;              // test hook: the first pair's leader leaves out its first token's queries
};

// ---- pairs of CTAs ------------------------------------------------------------------------------------------
__device__ __forceinline__ void pair_alloc(uint32_t dst_smem, uint32_t ncols) {
  asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(dst_smem), "r"(ncols)
               : "memory");
}
__device__ __forceinline__ void pair_relinquish() {
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void pair_dealloc(uint32_t taddr, uint32_t ncols) {
  asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
}
// Low word of a 128-byte-swizzle descriptor (start address, distance of 64-wide MN blocks); the high word is the
// same for every operand here (8-row atoms 1024 bytes apart).
__device__ __forceinline__ uint32_t desc_lo(uint32_t saddr, uint32_t lbo) {
  return ((saddr & 0x3FFFFu) >> 4) | ((lbo >> 4) << 16);
}
constexpr uint32_t kDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);
// D (+)= A . B^T over both CTAs; the descriptors hold the same offsets in both.
__device__ __forceinline__ void pair_mma(uint32_t d, uint32_t a_lo, uint32_t b_lo, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\t"
      "mov.b64 a, {%1, %5};\n\t"
      "mov.b64 b, {%2, %5};\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], a, b, %3, p;\n\t}" ::"r"(d),
      "r"(a_lo), "r"(b_lo), "r"(idesc), "r"(accumulate), "n"(kDescHi)
      : "memory");
}
// One arrival on the barrier at this offset in both CTAs once the MMAs issued so far are done.
__device__ __forceinline__ void pair_commit(uint32_t bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
      "h"((uint16_t)3)
      : "memory");
}
// Contiguous bytes on their way to L2 (a multiple of 16).
__device__ __forceinline__ void prefetch_l2(const void* src, uint32_t bytes) {
  asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(src), "r"(bytes) : "memory");
}
// A TMA load into this CTA that counts its bytes on `bar`, a barrier of either CTA (cluster address).
__device__ __forceinline__ void pair_load(uint32_t dst, const CUtensorMap* map, int32_t x, int32_t y, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2 [%0], "
      "[%1, {%2, %3}], [%4];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void pair_load_3d(uint32_t dst, const CUtensorMap* map, int32_t x, int32_t y, int32_t z,
                                             uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2 [%0], "
      "[%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar)
      : "memory");
}
// One arrival on a barrier of either CTA. What it announces are tensor-memory reads (ordered by the tcgen05 fence
// before it) and writes to this CTA's own shared memory (handed to the async proxy by the fence before it), so
// the arrival itself needs no release at cluster scope, which costs 2000-3400 cycles here.
__device__ __forceinline__ void arrive_pair(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
// Bounded waits on the SM's own clock (about a second; reading the global timer at each miss is slower).
constexpr long long kWaitCycles = 2000000000ll;
__device__ __forceinline__ bool test_bar(uint32_t bar, uint32_t parity) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(r)
      : "r"(bar), "r"(parity)
      : "memory");
  return r != 0;
}
__device__ __forceinline__ bool wait_own(uint32_t bar, uint32_t parity) {
  if (test_bar(bar, parity)) return true;      // (try_wait costs about 60 cycles more when there is nothing to wait for)
  long long t0 = 0;
  for (uint32_t i = 1;; ++i) {
    if (mbar_try_wait(bar, parity)) return true;
    if ((i & 63) == 0) {
      const long long t = clock64();
      if (t0 == 0) t0 = t;
      else if (t - t0 > kWaitCycles) return false;
    }
  }
}

// The same for a wait that lasts as long as many steps do: the limit counts from the last change of *steps, the count of
// them that another warp keeps in shared memory.
__device__ __forceinline__ bool wait_following(uint32_t bar, uint32_t parity, const volatile uint32_t* steps) {
  uint32_t seen = *steps;
  long long t0 = clock64();
  for (uint32_t i = 1;; ++i) {
    if (mbar_try_wait(bar, parity)) return true;
    if ((i & 63) == 0) {
      const uint32_t now = *steps;
      const long long t = clock64();
      if (now != seen) {
        seen = now;
        t0 = t;
      } else if (t - t0 > kWaitCycles) {
        return false;
      }
    }
  }
}

// The slow half of a wait that is unrolled many times: one copy, a call away.
__device__ __noinline__ bool wait_slow(uint32_t bar, uint32_t parity) { return wait_own(bar, parity); }
__device__ __forceinline__ bool wait_short(uint32_t bar, uint32_t parity) { return test_bar(bar, parity) || wait_slow(bar, parity); }

// The tokens of a pair's range, and of each the keys [k0, k1) that fall into it.
struct Walk {
  const int4* tinfo;
  int tok, tok1, e1;          // in the order of the walk
  int id, seq, vis, k0, k1;   // id: the token
  __device__ void set(int4 ti, int u) {
    seq = ti.x;
    vis = ti.y;
    id = ti.z;
    k0 = u * UNIT;
    k1 = tok == tok1 ? min(vis, e1 * UNIT) : vis;
  }
  __device__ void init(const CoreParams& p, int pair) {
    const int4 pi = p.pinfo[pair];
    const int4 first = p.pfirst[pair];
    tinfo = p.tinfo;
    tok = pi.x; tok1 = pi.z; e1 = pi.w;
    if (valid()) set(first, pi.y);
  }
  __device__ bool valid() const { return tok >= 0 && tok <= tok1; }
  __device__ void next() {
    do {
      ++tok;
      if (tok > tok1) return;
      set(tinfo[tok], 0);
    } while (vis <= 0);
  }
  __device__ int steps() const { return (k1 - k0 + NK - 1) / NK; }
  __device__ bool whole() const { return k0 == 0 && k1 == vis; }
};

// The steps of a pair's range, one after the other, across its tokens.
struct Steps {
  Walk w;
  int k;                      // first key of the step
  __device__ bool valid() const { return w.valid(); }
  __device__ void next() {
    k += NK;
    if (k >= w.k1) {
      w.next();
      k = w.k0;
    }
  }
};

// Pool rows of the steps' groups of 16 keys, one group a lane (lanes 16-31 repeat): the block list is read two steps
// ahead and the block table one, so that a step finds its rows in registers.
struct Rows {
  Steps s1, s2;               // the next step, the one behind it
  int raw1, off1, blk2;       // table entry and offset for s1, block for s2 (-1: no visible key)
  int g;
  __device__ void block(const CoreParams& p) {
    blk2 = -1;
    const int j = s2.k + 16 * g;
    if (s2.valid() && j < s2.w.k1) {
      const int i = j / p.v.page;
      blk2 = p.blocks ? p.blocks[(int64_t)s2.w.id * p.top_k + i] : i;
    }
  }
  __device__ void entry(const CoreParams& p) {
    raw1 = -1;
    off1 = blk2 < 0 ? -1 : (s1.k + 16 * g) % p.v.page;
    if (blk2 >= 0) raw1 = p.v.table[(int64_t)s1.w.seq * p.v.stride + blk2];
  }
  __device__ void init(const CoreParams& p, const Walk& w, int lane) {
    g = lane & (GROUPS - 1);
    s2.w = w;
    s2.k = w.valid() ? w.k0 : 0;
    block(p);
    s1 = s2;
    entry(p);
    if (s2.valid()) s2.next();
    block(p);
  }
  // The first of this lane's rows of step s1, -1 if there are none.
  __device__ int ahead(const CoreParams& p) const {
    return off1 < 0 || raw1 < 0 || raw1 >= p.v.num_pages ? -1 : raw1 * p.v.page + off1;
  }
  // The rows of step s1 (this lane's group), and on to the next: a group behind the last visible key, or in a page
  // outside the pool (flagged), is read out of range, which gives zeros.
  __device__ int take(const CoreParams& p) {
    const int raw = raw1, off = off1;
    s1 = s2;
    entry(p);
    if (s2.valid()) s2.next();
    block(p);
    if (off < 0) return -4096;
    if (raw < 0 || raw >= p.v.num_pages) {
      flag_error(p.err, DEVERR_PAGE);
      return -4096;
    }
    return raw * p.v.page + off;
  }
};

// GRAN: rows of a TMA box, the largest of 64, 32, 16 that divides the page size.
template <int GRAN>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    paged_core_kernel(const __grid_constant__ CoreParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = smem_addr(smem);
  auto bar = [&](int i) { return sbase + 8u * (uint32_t)i; };
  const uint32_t tmem_slot = sbase + 8 * NBAR;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t r = cluster_rank();
  const int pair = blockIdx.x >> 1;
  const uint32_t lead0 = map_peer(sbase, 0);
  auto lead = [&](int i) { return lead0 + 8u * (uint32_t)i; };

  if (threadIdx.x == 0) {
    for (int i = 0; i < NBAR; ++i) {
      uint32_t cnt = 1;
      if (i == B_SFREE || i == B_SFREE + 1 || i == B_PRDY || i == B_TRDY) cnt = 16;
      else if (i == B_TMAX || i == B_TMAX + 1 || i == B_LFREE) cnt = 4;
      else if (i == B_TAIL) cnt = 2;
      else if (i == B_OFREE || i == B_LRDY) cnt = 8;
      mbar_init(bar(i), cnt);
    }
    *reinterpret_cast<volatile uint32_t*>(smem + OFF_STEPS) = 0;
    fence_mbar_init();
    prefetch_tmap(&p.kmap);
    prefetch_tmap(&p.vmap);
    prefetch_tmap(&p.qmap);
    prefetch_tmap(&p.qrmap);
  }
  if (warp == 1) {
    pair_alloc(tmem_slot, 512);
    pair_relinquish();
  }
  tc_fence_before();
  cluster_sync();
  tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<const uint32_t*>(smem + 8 * NBAR);
  let_next_start();
  wait_for_previous();
  Walk w;
  w.init(p, pair);
  bool ok = true;

  if (warp == 0 || warp == 2 || warp == 3) {
    // -------------------------------------------------------------- ring producers
    // The three warps take every third entry. (A barrier's parity tells two consecutive phases apart: a warp's own
    // entries are 3 apart, so it never looks at a slot that is more than one lap behind.)
    const int me = warp == 0 ? 0 : warp - 1;
    auto load_q = [&](int g) {
      // the token's queries, once the last QK^T of the token before is done with the buffer
      ok = __all_sync(0xffffffffu, wait_own(bar(B_QEMPTY), (g & 1) ^ 1)) != 0;
      if (ok && elect_one()) {
        if (r == 0) mbar_expect_tx(bar(B_QFULL), 2 * Q_BYTES);
        const int32_t y = w.id * H + HC * (int)r;
        if (!(p.stall && pair == 0 && r == 0 && g == 0)) {
          for (int c = 0; c < 8; ++c) pair_load(sbase + OFF_Q + c * BOX, &p.qmap, 64 * c, y, lead(B_QFULL));
          pair_load(sbase + OFF_Q + 8 * BOX, &p.qrmap, 0, y, lead(B_QFULL));
        }
      }
      __syncwarp();
    };
    if (me == 1 && w.valid()) load_q(0);      // ahead of the block table's latency
    Rows rows;
    rows.init(p, w, lane);
    int base = 0, bph = 1, turn = me;         // slot and parity of the block of entries at hand, this warp's first of it
    uint32_t n = 0, end = 0;                  // ring index of the block, behind this warp's last entry (2^32: 250 million steps)
    int gpc = 0;
    // waits for the slot of entry e of the block; false when it gave up
    auto ready = [&](int e, int* slot) -> bool {
      int s = base + e, ph = bph;
      if (s >= RING) { s -= RING; ph ^= 1; }
      if (s >= RING) { s -= RING; ph ^= 1; }
      *slot = s;
      ok = __all_sync(0xffffffffu, wait_own(bar(B_EMPTY + s), ph)) != 0;
      return ok;
    };
    auto leave = [&](int count) {
      n += count;
      base += count;
      if (base >= RING) { base -= RING; bph ^= 1; }
      if (base >= RING) { base -= RING; bph ^= 1; }
      turn = (turn + 9 - count) % 3;          // count is 8 or 9
    };
    auto keys_of = [&](int row) {             // K of a step: this CTA's 128 keys, 64 columns an entry
      int y[128 / GRAN];
#pragma unroll
      for (int s = 0; s < 128 / GRAN; ++s) y[s] = __shfl_sync(0xffffffffu, row, 8 * (int)r + s * (GRAN / 16));
      for (int e = turn, slot; e < kEntriesK && ready(e, &slot); e += 3) {
        if (elect_one()) {
          const uint32_t dst = sbase + OFF_RING + slot * ENTRY, b = lead(B_FULL + slot);
          if (r == 0) mbar_expect_tx(bar(B_FULL + slot), 2 * ENTRY);
#pragma unroll
          for (int s = 0; s < 128 / GRAN; ++s) pair_load(dst + s * GRAN * 128, &p.kmap, 64 * e, y[s], b);
        }
        __syncwarp();
        end = n + e + 1;
      }
      leave(kEntriesK);
    };
    auto values_of = [&](int row, int tail_kq) {   // V of a step: 64 keys x 128 of this CTA's columns an entry
      // ... and the next step's keys on their way to L2, 16 rows an entry: 4 x 131072 rows 164 -> 151 us, 64 x 2 behind
      // 16896 542 -> 521. (All at once, or alongside the keys, they hold the keys' own copies up: 3 to 5 % slower than
      // without. Rows that L2 has already cost 0 to 4 %: 8 x 64 behind 16384.)
      const int later = rows.ahead(p);
      for (int e = turn, slot; e < kEntriesV && ready(e, &slot); e += 3) {
        const int kq = e >> 1;
        int y[64 / GRAN];
#pragma unroll
        for (int s = 0; s < 64 / GRAN; ++s) y[s] = __shfl_sync(0xffffffffu, row, 4 * kq + s * (GRAN / 16));
        if (elect_one()) {
          const uint32_t dst = sbase + OFF_RING + slot * ENTRY;
          uint32_t b = lead(B_FULL + slot);
          if (kq == tail_kq) {
            // counted in this CTA, whose softmax warps zero rows of it before P.V takes it
            mbar_expect_tx(bar(B_TAIL), ENTRY);
            if (r == 0) mbar_arrive(bar(B_FULL + slot));
            b = bar(B_TAIL);
          } else if (r == 0) {
            mbar_expect_tx(bar(B_FULL + slot), 2 * ENTRY);
          }
          const int z = 4 * (e & 1) + 2 * (int)r;  // 64-column blocks z, z + 1
#pragma unroll
          for (int s = 0; s < 64 / GRAN; ++s) {
            pair_load_3d(dst + s * GRAN * 128, &p.vmap, 0, y[s], z, b);
            if (GRAN < 64) pair_load_3d(dst + BOX + s * GRAN * 128, &p.vmap, 0, y[s], z + 1, b);
          }
        }
        const int to_l2 = __shfl_sync(0xffffffffu, later, 8 * (int)r + e);
        if (to_l2 >= 0 && elect_one())
          prefetch_l2(reinterpret_cast<const __nv_bfloat16*>(p.v.cache) + (int64_t)to_l2 * (DC + DR), 16 * (DC + DR) * 2);
        __syncwarp();
        end = n + e + 1;
      }
      leave(kEntriesV);
    };
    for (; ok && w.valid(); w.next(), ++gpc) {
      if (me == 1 && gpc > 0) load_q(gpc);
      // the token's entries: K0 K1 V0 K2 V1 ... K(ns-1) V(ns-2) V(ns-1)
      const int ns = w.steps(), rem = w.k1 - (w.k0 + (ns - 1) * NK);
      int row = -4096;
      for (int j = 0; ok && j < ns; ++j) {
        const int before = row;
        row = rows.take(p);
        keys_of(row);
        if (ok && j > 0) values_of(before, -1);
        if (ok && j == ns - 1) values_of(row, rem % 64 ? rem / 64 : -1);
      }
    }
    if (!ok) {
      if (lane == 0) flag_error(p.err, DEVERR_TIMEOUT);
      // copies still in flight, those of the peer too (seen at the leader's barriers; a tail entry's bytes land
      // within the same waits)
      if (r == 0) {
        for (uint32_t i = end > RING ? end - RING : 0; i < end; ++i) wait_own(bar(B_FULL + i % RING), (i / RING) & 1);
        if (me == 1 && gpc > 0) wait_own(bar(B_QFULL), (gpc - 1) & 1);
      }
    }
  } else if (warp == 1) {
    // -------------------------------------------------------------- MMA issuer (leader CTA)
    if (r == 0) {
      constexpr uint32_t id_qk = idesc_bf16(128, NK, 0, 0), id_pv = idesc_bf16(128, 256, 0, 1);
      const uint32_t q_lo = desc_lo(sbase + OFF_Q, 0), p_lo = desc_lo(sbase + OFF_P, 0);
      const uint32_t k_lo = desc_lo(sbase + OFF_RING, 0), v_lo = desc_lo(sbase + OFF_RING, BOX);
      auto wait_all = [&](uint32_t b, uint32_t par) { return __all_sync(0xffffffffu, wait_own(b, par)) != 0; };
      int js = 0, gpc = 0, tails = 0;         // step, token, tokens that end inside 64 keys
      int slot = 0, ph = 0;
      auto advance = [&](int count) {         // 7 < count < 14
        slot += count - RING;
        ph ^= 1;
        if (slot >= RING) { slot -= RING; ph ^= 1; }
      };
      // One lane runs through the entries of a product, unrolled: with a wait of all lanes and an elected lane for each entry
      // a step took 6900 cycles instead of 4600 where the rows lie in L2. (The warp's own path bounds it then, 380 cycles
      // an entry of which the MMAs take 256: each instruction more adds to the step.)
      auto qk = [&](int j) -> bool {
        const int sb = j & 1;
        if (!wait_all(bar(B_SFREE + sb), ((j >> 1) & 1) ^ 1)) return false;
        if (!wait_all(bar(B_FULL + slot), ph)) return false;       // (by all lanes: 4 % faster than in the loop)
        tc_fence_after();
        const uint32_t d = tmem + 256 + 128 * sb;
        bool good = true;
        if (elect_one()) {
          int s = slot, par = ph;
#pragma unroll
          for (int e = 0; e < kEntriesK; ++e) {
            good = wait_short(bar(B_FULL + s), par);
            if (!good) break;
            const uint32_t a = q_lo + e * (BOX >> 4), b = k_lo + s * (ENTRY >> 4);
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) pair_mma(d, a + 2 * kk, b + 2 * kk, id_qk, (e | kk) ? 1u : 0u);
            pair_commit(bar(B_EMPTY + s));
            if (++s == RING) { s = 0; par ^= 1; }
          }
          if (good) pair_commit(bar(B_SFULL + sb));
        }
        advance(kEntriesK);
        return __all_sync(0xffffffffu, good) != 0;
      };
      auto pv = [&](int j, bool first, int tail_kq) -> bool {
        if (!wait_all(bar(B_PRDY), j & 1)) return false;
        if (first && !wait_all(bar(B_OFREE), (gpc & 1) ^ 1)) return false;
        tc_fence_after();
        bool good = true;
        if (elect_one()) {
          int s = slot, par = ph;
#pragma unroll
          for (int e = 0; e < kEntriesV; ++e) {
            const int kq = e >> 1;
            good = wait_short(bar(B_FULL + s), par);
            if (good && kq == tail_kq && (e & 1) == 0) good = wait_short(bar(B_TRDY), tails & 1);
            if (!good) break;
            const uint32_t a = p_lo + kq * (BOX >> 4), b = v_lo + s * (ENTRY >> 4);
            const uint32_t keep = first && kq == 0 ? 0u : 1u;
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              pair_mma(tmem + 128 * (e & 1), a + 2 * kk, b + 128 * kk, id_pv, kk ? 1u : keep);
            pair_commit(bar(B_EMPTY + s));
            if (++s == RING) { s = 0; par ^= 1; }
          }
          if (good) pair_commit(bar(B_PVD));
        }
        if (tail_kq >= 0) ++tails;
        advance(kEntriesV);
        return __all_sync(0xffffffffu, good) != 0;
      };
      for (; ok && w.valid(); w.next(), ++gpc) {
        const int ns = w.steps(), rem = w.k1 - (w.k0 + (ns - 1) * NK);
        ok = wait_all(bar(B_QFULL), gpc & 1);
        for (int j = 0; ok && j < ns; ++j) {
          ok = qk(js + j);
          if (ok && j == ns - 1 && elect_one()) pair_commit(bar(B_QEMPTY));
          __syncwarp();
          if (ok && j > 0) ok = pv(js + j - 1, j == 1, -1);
        }
        if (ok) ok = pv(js + ns - 1, ns == 1, rem % 64 ? rem / 64 : -1);
        if (ok && elect_one()) pair_commit(bar(B_ODONE));
        __syncwarp();
        js += ns;
      }
      if (!ok && lane == 0) flag_error(p.err, DEVERR_TIMEOUT);
    }
  } else if (warp >= 4 && warp < 12) {
    // -------------------------------------------------------------- softmax
    const int quarter = warp & 3, half = (warp - 4) >> 2;
    const int i = (32 * quarter + lane) & (HC - 1);          // head of this CTA
    const int kq = 2 * (quarter >> 1) + half;                // this warp's block of 64 keys
    const int rb = quarter & 1;                              // block of 32 heads
    const uint32_t trow = tmem + ((uint32_t)(32 * quarter) << 16);
    float* red = reinterpret_cast<float*>(smem + OFF_RED);
    float* stat = reinterpret_cast<float*>(smem + OFF_STAT);
    const float c2 = p.scale_log2, thr = kRescaleLog2 / c2;
    const uint32_t sfree = lead(B_SFREE), prdy = lead(B_PRDY), trdy = lead(B_TRDY);
    auto wait_u = [&](uint32_t b, uint32_t par) { return __all_sync(0xffffffffu, wait_own(b, par)) != 0; };
    int js = 0, gpc = 0, tails = 0, nbase = 0;               // nbase: slot of the token's first entry
    for (; ok && w.valid(); w.next(), ++gpc) {
      const int ns = w.steps();
      float m = -INFINITY, l = 0.f;
      for (int j = 0; j < ns; ++j, ++js) {
        const int sb = js & 1;
        const int rem = w.k1 - (w.k0 + j * NK);              // visible keys from the step's first on
        if (!wait_u(bar(B_SFULL + sb), (js >> 1) & 1)) { ok = false; break; }
        tc_fence_after();
        if (threadIdx.x == 128) *reinterpret_cast<volatile uint32_t*>(smem + OFF_STEPS) = (uint32_t)js + 1;
        // Two passes over the scores, 32 columns at a time from tensor memory (64 columns held in registers take the
        // same time, but 128 registers with spills instead of 94)
        const uint32_t scol = trow + 256 + 128 * sb + 64 * half;
        const int nvis = rem - 64 * kq;
        auto load = [&](int h, float* s) {
          tmem_ld32(scol + 32 * h, reinterpret_cast<uint32_t*>(s));
          tmem_wait_ld();
          if (nvis < 32 * h + 32) {
#pragma unroll
            for (int c = 0; c < 32; ++c) s[c] = 32 * h + c < nvis ? s[c] : -INFINITY;
          }
        };
        float own = -INFINITY;
#pragma unroll 1
        for (int h = 0; h < 2; ++h) {
          float s[32];
          load(h, s);
#pragma unroll
          for (int k = 16; k > 0; k >>= 1)
#pragma unroll
            for (int c = 0; c < k; ++c) s[c] = fmaxf(s[c], s[c + k]);
          own = fmaxf(own, s[0]);
        }
        float* rbuf = red + sb * 4 * HC;
        rbuf[kq * HC + i] = own;
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(B_TMAX + rb));
        if (!wait_u(bar(B_TMAX + rb), js & 1)) { ok = false; break; }
        const float top = fmaxf(fmaxf(rbuf[i], rbuf[HC + i]), fmaxf(rbuf[2 * HC + i], rbuf[3 * HC + i]));
        // the four threads of a head see the same maxima, so they take the same decision
        float alpha = 1.f;
        if (top > -INFINITY && (m == -INFINITY || top > m + thr)) {
          alpha = m == -INFINITY ? 0.f : ex2_approx((m - top) * c2);
          l *= alpha;
          m = top;
        }
        // P.V of the step before is done: P may be overwritten and O rescaled
        if (js > 0 && !wait_u(bar(B_PVD), (js - 1) & 1)) { ok = false; break; }
        if (j > 0 && __any_sync(0xffffffffu, alpha != 1.f)) {
          tc_fence_after();
#pragma unroll 1
          for (int c = 128 * half; c < 128 * half + 128; c += 32) {
            uint32_t v[32];
            tmem_ld32(trow + c, v);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 32; ++e) v[e] = __float_as_uint(__uint_as_float(v[e]) * alpha);
            tmem_st32(trow + c, v);
          }
          tmem_wait_st();
          tc_fence_before();
        }
        // P = 2^((s - m) c2) in bf16 for the MMA (2^-8 of each weight); the sum takes the unrounded weights
        const float moff = m > -INFINITY ? -m * c2 : 0.f;       // (no finite score: all weights are 2^-inf)
        const uint64_t cc = f2_pack(c2, c2), off = f2_pack(moff, moff);
        uint8_t* prow = smem + OFF_P + kq * BOX + i * 128;
        uint64_t acc[4] = {0ull, 0ull, 0ull, 0ull};
#pragma unroll 1
        for (int h = 0; h < 2; ++h) {
          float s[32];
          load(h, s);
          uint32_t pk[16];
#pragma unroll
          for (int c = 0; c < 16; ++c) {
            float a0, a1;
            f2_unpack(f2_fma(f2_pack(s[2 * c], s[2 * c + 1]), cc, off), a0, a1);
            const float e0 = ex2_approx(a0), e1 = ex2_approx(a1);
            pk[c] = pack_bf16(e0, e1);
            acc[c & 3] = f2_add(acc[c & 3], f2_pack(e0, e1));
          }
#pragma unroll
          for (int c = 0; c < 4; ++c)
            *reinterpret_cast<uint4*>(prow + (((4 * h + c) ^ (i & 7)) << 4)) =
                make_uint4(pk[4 * c], pk[4 * c + 1], pk[4 * c + 2], pk[4 * c + 3]);
        }
        {
          float l0, l1;
          f2_unpack(f2_add(f2_add(acc[0], acc[1]), f2_add(acc[2], acc[3])), l0, l1);
          l += l0 + l1;
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) arrive_pair(sfree + 8 * sb);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) arrive_pair(prdy);
        if (j == ns - 1 && rem % 64) {
          // value rows behind the last visible key: zeros, since 0 * NaN is not 0
          if (!wait_u(bar(B_TAIL), tails & 1)) { ok = false; break; }
          ++tails;
          const int tail_kq = rem / 64, row0 = rem % 64;
          const int e0 = nbase + kEntriesK * ns + kEntriesV * (ns - 1) + 2 * tail_kq;
          for (int q = threadIdx.x - 128; q < 2 * 64 * 16; q += 256) {
            const int e = q >> 10, row = (q >> 4) & 63, c16 = q & 15;
            if (row < row0) continue;
            uint8_t* ent = smem + OFF_RING + ((e0 + e) % RING) * ENTRY + (c16 >> 3) * BOX;
            *reinterpret_cast<uint4*>(ent + row * 128 + (c16 & 7) * 16) = make_uint4(0u, 0u, 0u, 0u);
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) arrive_pair(trdy);
        }
      }
      if (!ok) break;
      nbase = (nbase + (kEntriesK + kEntriesV) * ns) % RING;
      if (!wait_u(bar(B_LFREE), (gpc & 1) ^ 1)) { ok = false; break; }
      stat[kq * HC + i] = l;
      if (kq == 0) stat[4 * HC + i] = m;
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(B_LRDY));
    }
    if (!ok && lane == 0) flag_error(p.err, DEVERR_TIMEOUT);
  } else if (warp >= 12) {
    // -------------------------------------------------------------- outputs
    const int quarter = warp & 3;
    const int i = (32 * quarter + lane) & (HC - 1), head = HC * (int)r + i;
    const int col0 = 128 * (quarter >> 1);
    const uint32_t trow = tmem + ((uint32_t)(32 * quarter) << 16);
    const float* stat = reinterpret_cast<const float*>(smem + OFF_STAT);
    const volatile uint32_t* steps = reinterpret_cast<const volatile uint32_t*>(smem + OFF_STEPS);
    const uint32_t ofree = lead(B_OFREE);
    auto wait_u = [&](uint32_t b, uint32_t par) { return __all_sync(0xffffffffu, wait_own(b, par)) != 0; };
    int gpc = 0;
    for (; ok && w.valid(); w.next(), ++gpc) {
      // (all steps of the token's piece: 2^22 of them at the most, more than 10 s)
      if (!__all_sync(0xffffffffu, wait_following(bar(B_LRDY), gpc & 1, steps))) { ok = false; break; }
      const float l = (stat[i] + stat[HC + i]) + (stat[2 * HC + i] + stat[3 * HC + i]);
      const float m = stat[4 * HC + i] * p.scale_log2 * 0.69314718055994531f;
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(B_LFREE));
      if (!wait_u(bar(B_ODONE), gpc & 1)) { ok = false; break; }
      tc_fence_after();
      const bool whole = w.whole();
      const int64_t row = (int64_t)w.id * H + head;
      const int slot = 2 * pair + (gpc > 0 ? 1 : 0);
      if (quarter < 2) {
        if (whole) p.lse[row] = l == 0.f ? -INFINITY : m + logf(l);
        // (a maximum of -inf stands for a piece without weight; one of NaN scores alone, whose sum is NaN, gives it a 0)
        else p.part_ml[(int64_t)slot * H + head] = make_float2(l == 0.f ? -INFINITY : m == -INFINITY ? 0.f : m, l);
      }
      const float inv = l == 0.f ? 0.f : 1.f / l;
      uint4* dst = reinterpret_cast<uint4*>(p.o_lat + row * DC + col0);
      float4* part = p.part_o + ((int64_t)slot * (DC / 4) + col0 / 4) * H + head;
#pragma unroll 1
      for (int c = 0; c < 256; c += 32) {
        uint32_t v[32];
        tmem_ld32(trow + c, v);
        tmem_wait_ld();
        const int lat = (c & 127) + 256 * (c >> 7);          // latent column - col0
        if (whole) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            uint32_t u[4];
#pragma unroll
            for (int k = 0; k < 4; ++k)
              u[k] = pack_bf16(__uint_as_float(v[8 * e + 2 * k]) * inv, __uint_as_float(v[8 * e + 2 * k + 1]) * inv);
            dst[lat / 8 + e] = make_uint4(u[0], u[1], u[2], u[3]);
          }
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e)
            part[(int64_t)(lat / 4 + e) * H] =
                make_float4(__uint_as_float(v[4 * e]), __uint_as_float(v[4 * e + 1]), __uint_as_float(v[4 * e + 2]),
                            __uint_as_float(v[4 * e + 3]));
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) arrive_pair(ofree);
    }
    if (!ok && lane == 0) flag_error(p.err, DEVERR_TIMEOUT);
  }
  __syncwarp();
  tc_fence_before();
  cluster_sync();
  if (warp == 1) {
    tc_fence_after();
    pair_dealloc(tmem, 512);
  }
}

// ---- plan ---------------------------------------------------------------------------------------------------
struct PlanParams {
  PagedView v;
  const int32_t* blocks;
  int32_t top_k, pairs;
  bool reorder;               // whether order_of() may change the order of the walk
  int4* tinfo;
  int64_t* cost;
  int4* pinfo;
  int4* pfirst;
  int4* splits;               // [pairs]: the tokens that cross ranges (token, first slot, first pair, last pair), then -1
  __nv_bfloat16* o_lat;
  float* lse;
  uint32_t* err;
};

// The order of the walk. Rows that several pairs read at the same time come from HBM once, so where sequences have several
// new tokens each, these are not taken one after the other by one pair:
// - Waves, from two tokens a pair on: pair i of n takes tokens i, n + i, 2 n + i, ..., so that all pairs are at the same
//   few sequences at any time. For rows of two waves' sequences that L2 holds (kWaveRows). Measured, the tokens' own
//   order or gangs against waves: 8 ragged chunks, 225 tokens, behind 15000 to 16300 rows 850 -> 803 us, 8 x 64 behind
//   16384 1745 -> 1610 (gangs), 4 x 128 1880 -> 1680; with too many rows: 2 x 80 behind 65536 2400 -> 2680, 64 x 8 behind
//   8192 1000 -> 1110, 16 x 16 behind 16384 the same.
// - Gangs, where every sequence has n new tokens: these are cut into g groups of n / g, and the walk takes the first
//   group of every sequence, then the second of every sequence, and so on. With a multiple of g pairs each group falls to
//   as many pairs, and the i-th pairs of the g groups walk the same sequences over the same keys, side by side. g:
//   the largest divisor of n up to 12 that leaves at most 4 of 74 pairs idle. Measured, the tokens' own order against
//   gangs: 64 x 2 behind 16896 rows 579 -> 521 us, 64 x 4 1143 -> 993, 64 x 16 behind 4096 1340 -> 1135, 16 x 2
//   behind 4096 85 -> 75.
constexpr int64_t kWaveRows = 100000000 / ((DC + DR) * 2);
struct Order {
  int n, g;                   // g > 1: gangs
  int64_t waves;              // > 0: waves of this many tokens in all
};
// The same in all threads of the block (and in all blocks).
__device__ inline Order order_of(const PlanParams& p) {
  __shared__ unsigned long long rows_sh;
  Order o = {0, 1, 0};
  const PagedView& v = p.v;
  if (!p.reorder) return o;
  const int64_t T = v.cu_q[v.B], n = T / v.B;
  if (T <= v.B || T > v.total_q) return o;
  if (threadIdx.x == 0) rows_sh = 0;
  bool even = n * v.B == T;
  unsigned long long rows = 0;
  for (int64_t b = threadIdx.x; b < v.B; b += blockDim.x) {
    const int64_t q0 = v.cu_q[b];
    even = even && q0 == b * n;
    if (v.cu_q[b + 1] > q0) rows += (unsigned long long)min(max(v.kv_lens[b], (int64_t)0), v.max_pages * v.page);
  }
  even = __syncthreads_and(even);
  if (rows) atomicAdd(&rows_sh, rows);
  __syncthreads();
  const int64_t all = (int64_t)rows_sh;
  if (T >= 2 * p.pairs && all / T * (2 * p.pairs) <= kWaveRows) {
    o.waves = T;
  } else if (even) {
    o.n = (int)n;
    o.g = (int)min(n, (int64_t)12);
    while (o.g > 1 && (n % o.g != 0 || p.pairs % o.g > p.pairs / 18)) --o.g;
  }
  return o;
}
// Where token t of sequence seq stands in it: a permutation of [0, T) for any contents of cu_q.
__device__ inline int64_t place_of(const PlanParams& p, const Order& o, int64_t t, int64_t seq) {
  if (o.waves > t) {
    // pair i's column begins at i T / pairs and holds T / pairs tokens or one more; those come last
    const int64_t T = o.waves, n = p.pairs, depth = T / n, rest = T % n, i = t % n;
    if (t < n * depth) return i * T / n + t / n;
    const int64_t c = ((t - n * depth + 1) * n + rest - 1) / rest - 1;
    return c * T / n + depth;
  }
  if (o.g > 1 && t < (int64_t)o.n * p.v.B) {
    const int64_t per = o.n / o.g, k = t - seq * o.n;
    return (k / per * p.v.B + seq) * per + k % per;
  }
  return t;
}

// Sequence and visible rows of new token t, by one warp; an empty row is written here.
__device__ __forceinline__ void plan_token(const PlanParams& p, int64_t t, const Order& order, int lane, int4* also = nullptr) {
  const PagedView& v = p.v;
  const PagedToken tok = paged_token(v, t);
  int64_t vis = tok.pos + 1;
  if (p.blocks && vis > 0) {
    const int top_k = p.top_k;
    const int32_t* list = p.blocks + t * top_k;
    const int64_t own = tok.pos / v.page;
    int n = top_k, bad = 0, at = -1;          // first -1, a fault, the last block
    for (int i0 = 0; i0 < n; i0 += 32) {
      const int g = i0 + lane < top_k ? list[i0 + lane] : -1;
      int before = __shfl_up_sync(0xffffffffu, g, 1);
      if (lane == 0) before = at;
      const uint32_t end = __ballot_sync(0xffffffffu, g < 0);
      const int cnt = end ? __ffs(end) - 1 : 32;
      if (lane < cnt && (g > own || g <= before)) bad = 1;
      if (cnt > 0) at = __shfl_sync(0xffffffffu, g, cnt - 1);
      if (cnt < 32) n = i0 + cnt;
    }
    if (__any_sync(0xffffffffu, bad)) {
      if (lane == 0) flag_error(p.err, DEVERR_BLOCKS);
      n = 0;
    }
    vis = n == 0 ? 0 : (int64_t)(n - 1) * v.page + (at == own ? tok.pos % v.page + 1 : v.page);
  }
  if (lane == 0) {
    const int64_t at = place_of(p, order, t, tok.seq);
    const int4 info = make_int4(tok.seq, (int32_t)(tok.seq < 0 ? 0 : vis), (int32_t)t, 0);
    p.tinfo[at] = info;
    if (also) also[at] = info;
  }
  if (tok.seq >= 0 && vis <= 0) {
    uint4* o = reinterpret_cast<uint4*>(p.o_lat + t * H * DC);
    for (int i = lane; i < H * DC / 8; i += 32) o[i] = make_uint4(0u, 0u, 0u, 0u);
    for (int i = lane; i < H; i += 32) p.lse[t * H + i] = -INFINITY;
  }
}

// The tokens of a large batch, one warp each, and the checks of the batch.
__global__ void __launch_bounds__(256) paged_tokens_kernel(const __grid_constant__ PlanParams p) {
  let_next_start();
  if (blockIdx.x == 0) paged_check(p.v, p.err);
  const Order order = order_of(p);
  const int64_t t = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  if (t < p.v.total_q) plan_token(p, t, order, threadIdx.x & 31);
}

// Dealing the tokens' units to the pairs. In cost, token t with u_t > 0 units is kStartUnits + u_t long; of
// n = min(pairs, total / kMinRange) pairs, pair pp's range begins at the first unit whose cost starts at or after
// pp * total / n, give or take a unit of a short token. (A unit never starts two costs behind the one before, so the
// middle pieces of a token are not empty.) Each pair's range is written as (first token, its first unit, last token, its
// end unit), (-1, ...) if it has none.
__device__ __forceinline__ int units_of(const int4& info) { return (max(info.y, 0) + UNIT - 1) / UNIT; }
__device__ __forceinline__ int weight_of(int units) { return units > 0 ? units + kStartUnits : 0; }
__device__ __forceinline__ int pairs_used(const PlanParams& p, const Order& order, int64_t total) {
  const int used = (int)max((int64_t)1, min((int64_t)p.pairs, total / kMinRange));
  return used >= order.g ? used - used % order.g : used;
}
// Boundary pp: the first token whose end lies behind the boundary's cost, and the unit in it.
template <typename Cost>
__device__ __forceinline__ void deal_boundary(int pp, int used, int pairs, int64_t total, int64_t T, const int4* tinfo, const Cost* cost,
                                              int32_t* tok, int32_t* unit) {
  const int64_t q = total / used, c = q * pp + (int)(total - q * used) * pp / used;      // total * pp / used
  int64_t a = 0, b = T;                     // the last token with cost <= c
  while (b - a > 1) {
    const int64_t mid = (a + b) >> 1;
    if (cost[mid] <= c) a = mid; else b = mid;
  }
  int u = (int)max((int64_t)0, c - cost[a] - kStartUnits);
  // Short tokens are not cut for the sake of one unit: those of two units never (16 x 1 over 512 rows 21.6 -> 19.4 us), of
  // up to four not when all pairs have work (64 x 1 over 300 rows 33 -> 25, 40 x 1 over 700 34 -> 26; but one token over
  // 600 rows takes 20.0 in two ranges and 22.5 in one, and 16 over 4096, of 16 units, 40 and 43).
  const int n = units_of(tinfo[a]);
  if (n <= (used == pairs ? 4 : 2)) u = u < 2 ? 0 : u + 1 >= n ? n : u;
  if (pp == used || u >= n) {               // behind its last unit: the next token
    ++a;
    u = 0;
    if (pp == used) a = T;
  }
  *tok = (int32_t)a;
  *unit = u;
}
// Pair pp's range from the boundaries; returns its entry of splits, (-1, ...) if no token that goes on begins in it.
template <typename Cost>
__device__ __forceinline__ int4 deal_pair(const PlanParams& p, int pp, int used, int64_t total, int64_t T, const int4* tinfo,
                                          const Cost* cost, const int32_t* btok, const int32_t* bunit) {
  int4 split = make_int4(-1, 0, 0, 0), info = make_int4(-1, 0, -2, 0);
  if (pp < used) {
    int a = btok[pp], ua = bunit[pp], e = btok[pp + 1], ue = bunit[pp + 1];
    while (a < T && units_of(tinfo[a]) == 0) { ++a; ua = 0; }       // tokens without units
    if (ue == 0) {                                                  // ends with the token before
      do --e; while (e >= 0 && units_of(tinfo[e]) == 0);
      ue = e >= 0 ? units_of(tinfo[e]) : 0;
    }
    if (a < T && (a < e || (a == e && ua < ue))) {
      info = make_int4(a, ua, e, ue);
      p.pfirst[pp] = tinfo[a];
      const int ne = units_of(tinfo[e]);
      if (ue < ne && !(a == e && ua > 0)) {                         // e begins here and goes on: to its last unit's pair
        int last = (int)(((int64_t)(cost[e] + kStartUnits + ne) * used - 1) / total);
        while (btok[last] > e) --last;                              // (whose first unit went to the pair before)
        split = make_int4(tinfo[e].z, 2 * pp + (a == e ? 0 : 1), pp, last);
      }
    }
  }
  p.pinfo[pp] = info;
  return split;
}
// The pairs' entries to p.splits, the empty ones last, by one warp.
__device__ __forceinline__ void write_splits(const PlanParams& p, int lane, const int4* begins) {
  int n = 0;
  for (int p0 = 0; p0 < p.pairs; p0 += 32) {
    const int4 it = p0 + lane < p.pairs ? begins[p0 + lane] : make_int4(-1, 0, 0, 0);
    const uint32_t m = __ballot_sync(0xffffffffu, it.x >= 0);
    if (it.x >= 0) p.splits[n + __popc(m & ((1u << lane) - 1u))] = it;
    n += __popc(m);
  }
  for (int k = n + lane; k < p.pairs; k += 32) p.splits[k] = make_int4(-1, 0, 0, 0);
}

// Few tokens: one block looks them up and deals them, from shared memory and without further trips to L2; a second block
// checks the batch. (It stands in front of the whole chain. Through global memory, as below, it took 1.3 us more.)
__global__ void __launch_bounds__(1024) paged_small_plan_kernel(const __grid_constant__ PlanParams p) {
  __shared__ int4 tinfo[kPlanTokens];
  __shared__ int32_t cost[kPlanTokens];
  __shared__ int32_t btok[kMaxPairs + 1], bunit[kMaxPairs + 1];
  __shared__ int4 begins[kMaxPairs];
  constexpr int DEAL = (kMaxPairs + 1 + 31) / 32 * 32;          // threads that deal, a boundary or a pair each
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, T = (int)p.v.total_q;
  let_next_start();
  if (blockIdx.x == 1) {
    paged_check(p.v, p.err);
    return;
  }
  const Order order = order_of(p);
  for (int t = warp; t < T; t += 32) plan_token(p, t, order, lane, tinfo);
  __syncthreads();
  if (tid >= DEAL) return;
  int total = 0;                                                // (each of the warps finds the costs itself)
  for (int t0 = 0; t0 < T; t0 += 32) {
    const int w = t0 + lane < T ? weight_of(units_of(tinfo[t0 + lane])) : 0;
    int x = w;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    if (warp == 0 && t0 + lane < T) cost[t0 + lane] = total + x - w;
    total += __shfl_sync(0xffffffffu, x, 31);
  }
  const int used = pairs_used(p, order, total);
  auto sync = [&]() { asm volatile("bar.sync 1, %0;" ::"n"(DEAL) : "memory"); };
  sync();
  if (tid <= used) deal_boundary(tid, used, p.pairs, total, T, tinfo, cost, &btok[tid], &bunit[tid]);
  sync();
  if (tid < p.pairs) begins[tid] = deal_pair(p, tid, used, total, T, tinfo, cost, btok, bunit);
  sync();
  if (warp == 0) write_splits(p, lane, begins);
}

__global__ void __launch_bounds__(1024) paged_plan_kernel(const __grid_constant__ PlanParams p) {
  __shared__ int64_t warp_tot[32];
  __shared__ int64_t total;
  __shared__ int32_t btok[kMaxPairs + 1], bunit[kMaxPairs + 1];
  __shared__ int4 begins[kMaxPairs];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t T = p.v.total_q;
  const int4* tinfo = p.tinfo;
  int64_t* cost = p.cost;
  let_next_start();
  const Order order = order_of(p);
  wait_for_previous();
  const int64_t per = (T + 1023) / 1024;
  const int64_t lo = min(T, tid * per), hi = min(T, lo + per);
  int64_t sum = 0;
  for (int64_t t = lo; t < hi; ++t) sum += weight_of(units_of(tinfo[t]));
  int64_t x = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) warp_tot[warp] = x;
  __syncthreads();
  if (warp == 0) {
    int64_t y = warp_tot[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t z = __shfl_up_sync(0xffffffffu, y, o);
      if (lane >= o) y += z;
    }
    warp_tot[lane] = y;
    if (lane == 31) total = y;
  }
  __syncthreads();
  int64_t at = x - sum + (warp > 0 ? warp_tot[warp - 1] : 0);
  for (int64_t t = lo; t < hi; ++t) {
    cost[t] = at;
    at += weight_of(units_of(tinfo[t]));
  }
  __syncthreads();
  const int used = pairs_used(p, order, total);
  for (int pp = tid; pp <= used; pp += blockDim.x) deal_boundary(pp, used, p.pairs, total, T, tinfo, cost, &btok[pp], &bunit[pp]);
  __syncthreads();
  for (int pp = tid; pp < p.pairs; pp += blockDim.x) begins[pp] = deal_pair(p, pp, used, total, T, tinfo, cost, btok, bunit);
  __syncthreads();
  if (warp == 0) write_splits(p, lane, begins);
}

// Exact merge of the tokens that cross ranges. Block (k, heads, columns) takes the k-th of them:
// o = sum_s e^{m_s - M} O_s / sum_s e^{m_s - M} l_s over its pieces, in order: its first slot, then the first slots of
// the pairs behind. The first kCombEarly pieces are loaded along with the maxima.
constexpr int kCombHeads = 32, kCombCols = 32, kCombEarly = 8;
__global__ void __launch_bounds__(256)
    paged_combine_kernel(const int4* splits, const float4* part_o, const float2* part_ml, __nv_bfloat16* o_lat, float* lse) {
  __shared__ float2 ml[kMaxPairs][kCombHeads];     // maximum and sum of each piece, then its weight
  __shared__ __align__(16) float tile[kCombHeads][kCombCols + 4];   // written as float4
  const int tid = threadIdx.x, lane = tid & 31, grp = tid >> 5;
  wait_for_previous();
  const int4 sp = splits[blockIdx.x];
  const int tok = sp.x;
  if (tok < 0) return;
  const int ns = sp.w - sp.z + 1, h0 = kCombHeads * blockIdx.y, c0 = kCombCols * blockIdx.z;
  auto slot = [&](int s) -> int64_t { return s == 0 ? sp.y : 2 * (sp.z + s); };
  const float4* src = part_o + (int64_t)(c0 / 4 + grp) * H + h0 + lane;
  float4 early[kCombEarly];
#pragma unroll
  for (int s = 0; s < kCombEarly; ++s)
    if (s < ns) early[s] = src[slot(s) * (DC / 4) * H];
  for (int s = grp; s < ns; s += 8) ml[s][lane] = part_ml[slot(s) * H + h0 + lane];
  __syncthreads();
  // weights e^{m_s - M} / L of the pieces (lane = head; the warps share the pieces, each finds M and L itself)
  float M = -INFINITY, L = 0.f;
  for (int s = 0; s < ns; ++s) M = fmaxf(M, ml[s][lane].x);
  for (int s = 0; s < ns; ++s)
    if (ml[s][lane].x > -INFINITY) L += __expf(ml[s][lane].x - M) * ml[s][lane].y;
  const float inv = L == 0.f ? 0.f : 1.f / L;
  __syncthreads();
  for (int s = grp; s < ns; s += 8) ml[s][lane].x = ml[s][lane].x > -INFINITY ? __expf(ml[s][lane].x - M) * inv : 0.f;
  if (grp == 0 && blockIdx.z == 0) lse[(int64_t)tok * H + h0 + lane] = L == 0.f ? -INFINITY : M + logf(L);
  __syncthreads();
  // thread (lane = head, grp): the column quad grp of this block's 8
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  auto add = [&](int s, float4 x) {
    const float e = ml[s][lane].x;
    acc.x += e * x.x; acc.y += e * x.y; acc.z += e * x.z; acc.w += e * x.w;
  };
#pragma unroll
  for (int s = 0; s < kCombEarly; ++s)
    if (s < ns) add(s, early[s]);
#pragma unroll 8
  for (int s = kCombEarly; s < ns; ++s) add(s, src[slot(s) * (DC / 4) * H]);
  *reinterpret_cast<float4*>(&tile[lane][4 * grp]) = acc;
  __syncthreads();
  // head tid / 8, 4 columns each
  const int h = tid >> 3, cc = 4 * (tid & 7);
  const float* x = &tile[h][cc];
  *reinterpret_cast<uint2*>(o_lat + ((int64_t)tok * H + h0 + h) * DC + c0 + cc) =
      make_uint2(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]));
}

template <int GRAN>
cudaError_t launch_core(const CoreParams& p, cudaStream_t st) {
  // per device, so set at every call
  cudaError_t e = cudaFuncSetAttribute(paged_core_kernel<GRAN>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)SMEM_BYTES);
  if (e != cudaSuccess) return e;
  return launch_next(paged_core_kernel<GRAN>, dim3(2 * p.pairs), kThreads, SMEM_BYTES, st, p);
}

size_t align1k(size_t x) { return (x + 1023) / 1024 * 1024; }

struct Scratch {
  int4* tinfo;
  int64_t* cost;
  int4* pinfo;
  int4* pfirst;
  int4* splits;
  float2* part_ml;
  float4* part_o;
  size_t bytes;
};

Scratch carve(void* ws, int64_t T) {
  Scratch s;
  char* p = (char*)ws;
  s.tinfo = (int4*)p;
  p += align1k((size_t)T * sizeof(int4));
  s.cost = (int64_t*)p;
  p += align1k((size_t)T * sizeof(int64_t));
  s.pinfo = (int4*)p;
  p += align1k(kMaxPairs * sizeof(int4));
  s.pfirst = (int4*)p;
  p += align1k(kMaxPairs * sizeof(int4));
  s.splits = (int4*)p;
  p += align1k(kMaxPairs * sizeof(int4));
  s.part_ml = (float2*)p;
  p += align1k((size_t)2 * kMaxPairs * H * sizeof(float2));
  s.part_o = (float4*)p;
  p += (size_t)2 * kMaxPairs * H * DC * sizeof(float);
  s.bytes = (size_t)(p - (char*)ws);
  return s;
}

}  // namespace

size_t tc_paged_attention_bytes(int64_t total_q) { return carve(nullptr, total_q).bytes; }

cudaError_t tc_paged_attention(const PagedView& v, const void* q_abs, const void* q_rope, const int32_t* blocks,
                               int32_t top_k, float scale, void* o_lat, float* lse, void* ws, int num_sms, uint32_t* err,
                               cudaStream_t st) {
  const Scratch s = carve(ws, v.total_q);
  CoreParams p;
  memset(&p, 0, sizeof(p));
  const int gran = v.page % 64 == 0 ? 64 : v.page % 32 == 0 ? 32 : 16;
  cudaError_t e;
  const int64_t rows = v.num_pages * v.page, TH = v.total_q * H;
  if ((e = make_tmap_bf16(&p.kmap, v.cache, DC + DR, rows, DC + DR, 64, gran)) != cudaSuccess) return e;
  if ((e = make_tmap_bf16_blocks(&p.vmap, v.cache, DC + DR, rows, gran, gran == 64 ? 2 : 1)) != cudaSuccess) return e;
  if ((e = make_tmap_bf16(&p.qmap, q_abs, DC, TH, DC, 64, HC)) != cudaSuccess) return e;
  if ((e = make_tmap_bf16(&p.qrmap, q_rope, DR, TH, DR, 64, HC)) != cudaSuccess) return e;
  p.v = v;
  p.blocks = blocks;
  p.top_k = top_k;
  p.pairs = num_sms / 2 < kMaxPairs ? num_sms / 2 : kMaxPairs;
  p.tinfo = s.tinfo;
  p.pinfo = s.pinfo;
  p.pfirst = s.pfirst;
  p.o_lat = (__nv_bfloat16*)o_lat;
  p.lse = lse;
  p.part_o = s.part_o;
  p.part_ml = s.part_ml;
  p.scale_log2 = scale * 1.4426950408889634f;
  p.err = err;
  p.stall = take_paged_stall();
  PlanParams pp;
  pp.v = v;
  pp.blocks = blocks;
  pp.top_k = top_k;
  pp.pairs = p.pairs;
  // (one sequence: its pairs all walk it already, and 512 tokens behind 32768 rows lose 0-2 % to the idle pairs; lists of
  // blocks differ from token to token; the look at every cu_q in every block is for batches, not for millions)
  pp.reorder = !blocks && v.B > 1 && v.total_q > v.B && v.B <= 4096;
  pp.tinfo = s.tinfo;
  pp.cost = s.cost;
  pp.pinfo = s.pinfo;
  pp.pfirst = s.pfirst;
  pp.splits = s.splits;
  pp.o_lat = p.o_lat;
  pp.lse = lse;
  pp.err = err;
  // One block looks up few tokens in the plan's own launch; each of its 32 warps takes a token in about 1 us (a list of
  // blocks is read for it), so more than kPlanTokens of them get a launch of their own.
  if (v.total_q <= kPlanTokens) {
    paged_small_plan_kernel<<<2, 1024, 0, st>>>(pp);
    note_launch();
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
  } else {
    paged_tokens_kernel<<<(unsigned)((v.total_q + 7) / 8), 256, 0, st>>>(pp);
    note_launch();
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    if ((e = launch_next(paged_plan_kernel, dim3(1), 1024, 0, st, pp)) != cudaSuccess) return e;
  }
  e = gran == 64 ? launch_core<64>(p, st) : gran == 32 ? launch_core<32>(p, st) : launch_core<16>(p, st);
  if (e != cudaSuccess) return e;
  // at most one token per boundary, and no more than there are, goes on in the next pair's range
  const int64_t most = p.pairs - 1 < v.total_q ? p.pairs - 1 : v.total_q;
  if (most > 0)
    e = launch_next(paged_combine_kernel, dim3((unsigned)most, H / kCombHeads, DC / kCombCols), 256, 0, st,
                    (const int4*)s.splits, (const float4*)s.part_o, (const float2*)s.part_ml, p.o_lat, lse);
  return e;
}

}  // namespace mla
