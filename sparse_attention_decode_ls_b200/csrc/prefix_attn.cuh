// Decode attention of a batch over its whole paged contexts, the pages that all requests share
// (a common prefix) computed once for every row.
//
//   s_j = scale * q_h . K_j,  o_h = sum_j softmax(s)_j V_j,  lse_h = log sum_j exp(s_j)
//
// over the positions j < lens[b] of each request: 576-wide latent rows, V = their first 512 dims.
//
// * A unit of work is a block of at most 128 query rows against a range of positions: for the
//   shared pages 128 rows out of all batch * heads rows (whichever requests they belong to), for
//   a request's own pages its heads.  Partial outputs of a row's units meet in
//   prefix_attn_combine by their running maxima and sums.
// * attn_prefix_tc: a pair of CTAs (2-CTA cluster) runs a unit with tcgen05.mma cta_group::2,
//   M = 128: each CTA holds 64 query rows in all of its 128 TMEM lanes (lanes 64-127 hold the
//   second half of the columns), so O (64 x 512 float32) takes 256 columns and two S tiles of
//   256 positions the other 256.
//   Why this shape (clocks per MMA of K = 16, measured on every SM at once, A and B in shared
//   memory): cta_group::1 M 128: N 64 65, N 128 65, N 256 128; cta_group::2 M 128: N 128 65,
//   N 256 65; M 64 N 256 128.  An MMA takes at least 65 clocks, so N = 64 tiles run at half
//   rate.  One CTA with 128 rows would need all of TMEM for O; splitting O's columns over two
//   CTAs makes them either swap S or compute it twice.  With M 128 over the pair and N 256 all
//   MMAs run at full rate, S is computed once and only row maxima cross lanes.
//   The price is shared-memory fill: K (half of the tile's rows, 576 dims) and V (all rows,
//   half of the 512 dims) are loaded separately, 278,528 bytes per SM and tile: 63 bytes per clock at
//   full MMA rate.  Eight 16 KB slots in flight, each held about 2,400 clocks from its load to its
//   reuse, allow 54.6, or 5,100 clocks per tile.  A page's P goes to PV as soon as it is written, into a
//   ring of three pages, which left room for the eighth slot (without the softmax 277 -> 220 us).
//   What the issuing thread does between two MMAs (75 clocks for a wait that has already completed,
//   32 for a commit) leaves the tensor cores idle, so one warp issues S, another PV, and each fills
//   the other's gaps (two issuers: 64 clocks per MMA, commits and waits included; one: 100).
// Measured, 8 requests x 128 heads over 131,072 shared positions and up to 1,024 of their own: 284 us,
// 1,030 TFLOP/s, 0.63 of the measured cuBLAS bf16 burst; back to back for seconds, at the 1,000 W
// power cap and 1.7 GHz, 323 us (0.65 of cuBLAS under the same cap).  Tensor pipe 51 % active, DRAM
// 7 %, L2 hit rate 81 %.
// What bounds it: no part alone.  A tile takes 8,400 clocks (at 1.67 GHz): its MMAs need 4,400, the loads without
// MMAs 4,600 (158 us), loads and MMAs without the softmax 6,400 (220 us: MMAs wait for slots and slots
// for MMAs).  The other 2,000 are softmax and hand-over of P that nothing hides: PV of a tile waits
// for its P, and S is ahead by two tiles at most.  For seconds, power.
// One request of 128 heads (device time of a call): 7.4 us for a length of 0 (launch, set-up and exit of the
// pair), 12.9 for 1 to 64 (page ids -> Q, K, V -> S -> softmax -> PV -> store), 13.7 for a whole tile of
// 256, 15.7 for 200: the rows of V on the last page come one request for four rows then.
#pragma once
#include "common.cuh"

namespace ls {

namespace pfx {
constexpr int DK = 576, DV = 512;
constexpr int kRows = 128;                    // query rows of a unit, 64 per CTA
constexpr int kTile = 256;                    // positions per tile: four pages
constexpr int kPanels = DK / 64;              // 9 K panels of 64 dims (128 bytes a row)
constexpr int kSlotBytes = 16384;
constexpr int kKSlots = 4, kVSlots = 4;       // rings: K slot = 128 positions x 64 dims, V slot = 64 x 128
constexpr int kVItems = 8;                    // V slots per tile: two 256-dim halves of O x four pages
constexpr int kOffQ = 0;                      // 9 panels x 64 rows x 128 bytes
constexpr int kQBytes = kPanels * 64 * 128;
constexpr int kOffP = kOffQ + kQBytes;        // ring of 3 panels (a page's positions) x 64 rows x 128 bytes
constexpr int kPSlots = 3;
constexpr int kOffK = kOffP + kPSlots * 8192;
constexpr int kOffV = kOffK + kKSlots * kSlotBytes;
constexpr int kOffBar = kOffV + kVSlots * kSlotBytes;
// k_full[kKSlots] k_empty[kKSlots] v_full[kVSlots] v_empty[kVSlots] q_full q_free s_full[2]
// s_free[2] p_full[4] p_free[4] o_ready o_ready_peer pv_done[2]
constexpr int kNumBars = 2 * (kKSlots + kVSlots) + 18;
constexpr int kOffRed = kOffBar + kNumBars * 8;      // row maxima (sums at the end): [2][4][64] float
constexpr int kOffTmem = kOffRed + 2 * 256 * 4;
constexpr int kSmem = kOffTmem + 16;
static_assert(kOffP % 1024 == 0 && kOffK % 1024 == 0, "128-byte swizzled operands need 1024-byte alignment");
static_assert(kSmem <= 227 * 1024, "shared memory budget");
// warps 0-7 softmax (warp w: TMEM lanes 32 (w % 4) .. + 31, columns 64 (w / 4) .. + 63), 8 and 9 the
// MMAs of S and PV, 10 loads Q and K, 11 V
constexpr int kSoftWarps = 8, kSWarp = 8, kPvWarp = 9, kLoadK = 10, kLoadV = 11;
constexpr int kThreads = (kLoadV + 1) * 32;
constexpr int kTmemS = 256;                          // O in columns [0, 256), S tiles behind it
constexpr uint32_t kIdescS = make_idesc(1 /*bf16*/, 128, kTile, false, false);
constexpr uint32_t kIdescO = make_idesc(1 /*bf16*/, 128, 256, false, true);
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
}  // namespace pfx

struct PrefixParams {
  int B, H, max_pages;
  int shared_pages;        // pages that every request's table begins with
  float scale;
  long long num_rows;      // rows of the pool
  long long num_pages;
  const int* page_table;   // [B, max_pages]
  const int* lens;         // [B]
  void* o;                 // [B, H, 512]
  float* lse;              // [B, H]
  int o_f32;
  int blocks;              // 128-row blocks of the B * H rows (shared part; 0 without one)
  int np, no;              // splits of the shared part and of each request's own part
  int direct;              // a row has one unit: it writes o and lse itself
  float* part_o;           // unit partials, unnormalised: [64 groups of 8 dims][rows][8]
  float* part_ml;          // [rows of all units][2]: running max (log2 domain) and sum
};

// One unit of work.  Units run in order of their split, so that the CTA pairs working at the same
// time read the same shared pages (from L2 for all but the first).
struct PrefixUnit {
  int row0, nrows;      // query rows [row0, row0 + nrows) of B * H
  int table;            // request whose page table is used
  int begin, end;       // positions (begin at a page)
  int tiles;
  long long part;       // first of its rows among the partials
};

__device__ __forceinline__ int prefix_len_of(const PrefixParams& p, int b) {
  return max(0, min(p.lens[b], p.max_pages * LS_PAGE));
}

__device__ __forceinline__ PrefixUnit prefix_unit(const PrefixParams& p, int u) {
  using namespace pfx;
  PrefixUnit w;
  const int npre = p.blocks * p.np;
  int first, last, i, n;
  if (u < npre) {
    i = (int)((unsigned)u / (unsigned)p.blocks);
    n = p.np;
    const int m = u - i * p.blocks;
    w.row0 = m * kRows;
    w.nrows = min(kRows, p.B * p.H - w.row0);
    w.table = 0;
    w.part = (long long)u * kRows;
    first = 0;
    last = p.shared_pages * LS_PAGE;
  } else {
    const int v = u - npre;
    i = (int)((unsigned)v / (unsigned)p.B);
    n = p.no;
    const int b = v - i * p.B;
    w.row0 = b * p.H;
    w.nrows = p.H;
    w.table = b;
    w.part = (long long)npre * kRows + (long long)v * p.H;
    first = p.shared_pages * LS_PAGE;
    last = max(first, prefix_len_of(p, b));
  }
  // (at most 2^23 tiles in 74 splits: 32 bits hold the products)
  const unsigned tiles = (unsigned)(last - first + kTile - 1) / kTile;
  const int t0 = (int)(tiles * (unsigned)i / (unsigned)n), t1 = (int)(tiles * (unsigned)(i + 1) / (unsigned)n);
  w.begin = first + t0 * kTile;
  w.end = min(last, first + t1 * kTile);
  w.tiles = t1 - t0;
  return w;
}

// Pages of a unit's last tile that hold any of its positions.
__device__ __forceinline__ int prefix_last_pages(const PrefixUnit& w) {
  return (w.end - (w.begin + (w.tiles - 1) * pfx::kTile) + LS_PAGE - 1) / LS_PAGE;
}

// 32 bytes in one access.
__device__ __forceinline__ void st_global_v8(float* p, const float* v) {
  asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "f"(v[0]), "f"(v[1]), "f"(v[2]),
               "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7])
               : "memory");
}
__device__ __forceinline__ void ld_global_v8(const float* p, float* v) {
  asm volatile("ld.global.v8.f32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7])
               : "l"(p));
}

// ---- the cta_group::2 forms ---------------------------------------------------------------
__device__ __forceinline__ void tma_load_2d_pair(uint32_t dst_smem, const CUtensorMap* map, uint32_t cluster_bar,
                                                 int x, int y) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2 [%0], [%1, "
      "{%3, %4}], [%2];" ::"r"(dst_smem),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(cluster_bar), "r"(x), "r"(y)
      : "memory");
}
__device__ __forceinline__ void tma_load_3d_pair(uint32_t dst_smem, const CUtensorMap* map, uint32_t cluster_bar,
                                                 int x, int y, int z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2 [%0], [%1, "
      "{%3, %4, %5}], [%2];" ::"r"(dst_smem),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(cluster_bar), "r"(x), "r"(y), "r"(z)
      : "memory");
}
__device__ __forceinline__ void tma_gather4_pair(uint32_t dst_smem, const CUtensorMap* map, uint32_t cluster_bar,
                                                 int x, int r0, int r1, int r2, int r3) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile::gather4.mbarrier::complete_tx::bytes.cta_group::2 [%0], "
      "[%1, {%2, %3, %4, %5, %6}], [%7];" ::"r"(dst_smem),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(r0), "r"(r1), "r"(r2), "r"(r3), "r"(cluster_bar)
      : "memory");
}
__device__ __forceinline__ void mma_bf16_pair(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}
// Arrive on the barrier at this offset in both CTAs once this thread's MMAs so far are done.
__device__ __forceinline__ void tc_commit_pair(uint64_t* bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
          smem_u32(bar)),
      "h"((uint16_t)3)
      : "memory");
}
__device__ __forceinline__ void tmem_alloc_pair(uint32_t* dst, uint32_t ncols) {
  asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(dst)), "r"(ncols)
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_dealloc_pair(uint32_t taddr, uint32_t ncols) {
  asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
}

// True in one lane of the (converged) warp, always the same.
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
  return r != 0;
}
// Barrier of the softmax warps that also ands a flag over them, so that they leave a loop together
// when one of them gave up on a wait.
__device__ __forceinline__ bool softmax_sync_and(bool v) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred a, b;\n\tsetp.ne.u32 a, %1, 0;\n\tbarrier.cta.red.and.pred b, 1, 256, a;\n\t"
      "selp.u32 %0, 1, 0, b;\n\t}"
      : "=r"(r)
      : "r"((uint32_t)v)
      : "memory");
  return r != 0;
}

// Rank 0 of the pair issues every MMA; the barriers that count loads (full, q_full) live in its
// shared memory and take both CTAs' bytes, those it signals (empty, q_free, s_full, p_free, pv_done)
// exist in both.  S runs up to two tiles ahead of PV, so that the softmax of a tile has the MMAs of
// others to hide behind.  The softmax warps arrive on barriers of their own CTA: an arrival in the
// other CTA with cluster scope costs each of them about a thousand clocks, so in rank 1 the two warps
// that have no MMAs to issue pass the news on (305 -> 289 us at 8 x 128 heads, 131,072 positions).
__global__ void __launch_bounds__(pfx::kThreads, 1)
    attn_prefix_tc(const PrefixParams p, const __grid_constant__ CUtensorMap kv_map,
                   const __grid_constant__ CUtensorMap v_map, const __grid_constant__ CUtensorMap row_map,
                   const __grid_constant__ CUtensorMap q_map) {
  using namespace pfx;
  extern __shared__ __align__(1024) uint8_t sm[];
  uint64_t* k_full = (uint64_t*)(sm + kOffBar);
  uint64_t* k_empty = k_full + kKSlots;
  uint64_t* v_full = k_empty + kKSlots;
  uint64_t* v_empty = v_full + kVSlots;
  uint64_t* q_full = v_empty + kVSlots;
  uint64_t* q_free = q_full + 1;
  uint64_t* s_full = q_full + 2;   // S tile of buffer g % 2 is in TMEM
  uint64_t* s_free = q_full + 4;   // ... and has been read by the softmax
  uint64_t* p_full = q_full + 6;    // P of the tile's page k is in shared memory
  uint64_t* p_free = q_full + 10;   // ... and has been read by PV
  // this CTA's O needs no rescaling for the tile, or has been rescaled; and rank 1's, as rank 0 hears of
  // it.  (Two barriers: a warp of rank 0 may come to the next tile before rank 1's news of this one, and
  // must not be counted in its place.  It cannot on s_free and p_full, whose next arrival waits for
  // MMAs that waited for the news.)
  uint64_t* o_ready = q_full + 14;
  uint64_t* o_ready_peer = q_full + 15;
  // PV of a tile of this parity has finished.  (A wait tells a phase only from the next one.  A softmax
  // warp that has written P(g - 1) knows from p_free that PV(g - 3) is done, and nothing about PV(g - 2):
  // so tile g - 1 is waited for on a barrier whose phase before is tile g - 3.)
  uint64_t* pv_done = q_full + 16;
  float* red = (float*)(sm + kOffRed);
  uint32_t* tmem_slot = (uint32_t*)(sm + kOffTmem);

  const int warp = __shfl_sync(0xffffffffu, warp_id(), 0), lane = lane_id();  // (the same for all lanes)
  const int rank = (int)cluster_rank();
  const int pair = blockIdx.x >> 1, npairs = gridDim.x >> 1;
  const int units = p.blocks * p.np + p.B * p.no;
  const uint32_t sbase = smem_u32(sm);
  PrefixUnit w = prefix_unit(p, pair);  // (every pair has one) while the set-up runs

  if (threadIdx.x == 0) {
    for (int s = 0; s < kKSlots; ++s) {
      mbar_init(&k_full[s], 1);   // rank 0's loader, with both CTAs' bytes
      mbar_init(&k_empty[s], 1);  // the MMAs that read the slot
    }
    for (int s = 0; s < kVSlots; ++s) {
      mbar_init(&v_full[s], 1);
      mbar_init(&v_empty[s], 1);
    }
    mbar_init(q_full, 1);
    mbar_init(q_free, 1);
    for (int s = 0; s < 2; ++s) {
      mbar_init(&s_full[s], 1);
      mbar_init(&s_free[s], kSoftWarps + (rank == 0));  // (rank 0: and the news from rank 1)
    }
    for (int k = 0; k < 4; ++k) {
      mbar_init(&p_full[k], 2 + (rank == 0));  // two warps hold a page's positions
      mbar_init(&p_free[k], 1);
    }
    mbar_init(o_ready, kSoftWarps);
    mbar_init(o_ready_peer, 1);
    mbar_init(&pv_done[0], 1);
    mbar_init(&pv_done[1], 1);
    fence_mbar_init();
  } else if (threadIdx.x == kLoadK * 32) {
    prefetch_tmap(&kv_map);
    prefetch_tmap(&q_map);
    prefetch_tmap(&v_map);
  }
  if (warp == kSWarp) tmem_alloc_pair(tmem_slot, 512);
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();  // both CTAs' barriers exist before either signals the other
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  griddep_launch_dependents();

  if (warp >= kLoadK) {
    // ================= loads: item e of a ring goes to slot e % slots =============================
    const bool is_v = warp == kLoadV;
    const int slots = is_v ? kVSlots : kKSlots;
    uint64_t* full = is_v ? v_full : k_full;
    uint64_t* empty = is_v ? v_empty : k_empty;
    const uint32_t full0 = dsmem_map(smem_u32(full), 0), qfull0 = dsmem_map(smem_u32(q_full), 0);
    const uint32_t ring = sbase + (is_v ? kOffV : kOffK);
    const int oob = (int)p.num_rows;  // one row past the pool: reads as zeros
    int nu = 0, e = 0;                // units and items so far
    int s = 0, ph = 1;                // the next slot; the parity of the wait for it to be empty (1: at once)
    bool ok = true;
    // the next item: wait for its slot, announce both CTAs' bytes (rank 0); one lane
    auto open_slot = [&]() {
      const bool go = mbar_wait(&empty[s], ph);
      if (go && rank == 0) mbar_arrive_expect_tx(&full[s], 2 * kSlotBytes);
      return go;
    };
    auto next_slot = [&]() {
      ++e;
      if (++s == slots) {
        s = 0;
        ph ^= 1;
      }
    };
    for (int u = pair; ok && u < units; u += npairs) {
      if (u != pair) w = prefix_unit(p, u);
      if (w.tiles == 0) continue;
      if (!is_v) {
        int go = 1;
        if (lane == 0) {
          if (nu > 0) go = mbar_wait(q_free, (nu - 1) & 1);
          if (go) {
            if (rank == 0) mbar_arrive_expect_tx(q_full, 2 * kQBytes);
            for (int c = 0; c < kPanels; ++c)
              tma_load_2d_pair(sbase + kOffQ + c * 8192, &q_map, qfull0, c * 64, w.row0 + rank * 64);
          }
        }
        ok = __shfl_sync(0xffffffffu, go, 0) != 0;
        if (!ok) break;
      }
      ++nu;
      const int* table = p.page_table + (size_t)w.table * p.max_pages;
      const int page_end = (w.end + LS_PAGE - 1) / LS_PAGE;
      // page id of page `lane` (< 4) of tile t, -1 behind the unit's end; and its first pool row, or
      // the row past the pool
      auto page_id = [&](int t) {
        const int pg = w.begin / LS_PAGE + t * 4 + lane;
        return lane < 4 && t < w.tiles && pg < page_end ? table[pg] : -1;
      };
      auto page_row = [&](int t, int id) {
        const bool in = id >= 0 && id < p.num_pages;
        if (!in && lane < 4 && w.begin / LS_PAGE + t * 4 + lane < page_end) flag(LS_DEV_BOUNDS);
        return in ? id * LS_PAGE : oob;
      };
      int id = page_id(0);
      for (int t = 0; ok && t < w.tiles; ++t) {
        const int rk = page_row(t, id);
        id = page_id(t + 1);  // (looked at a tile later)
        int go = 1;
        if (!is_v) {
          // panel c of this CTA's 128 positions (pages 2 * rank, 2 * rank + 1 of the tile)
          const int ra = __shfl_sync(0xffffffffu, rk, 2 * rank), rb = __shfl_sync(0xffffffffu, rk, 2 * rank + 1);
          if (lane == 0) {
            for (int c = 0; c < kPanels; ++c) {
              if (!open_slot()) { go = 0; break; }
              const uint32_t dst = ring + s * kSlotBytes, bar = full0 + s * 8;
              tma_load_2d_pair(dst, &kv_map, bar, c * 64, ra);
              tma_load_2d_pair(dst + 8192, &kv_map, bar, c * 64, rb);
              next_slot();
            }
          }
        } else if (t == w.tiles - 1) {
          // the tile with the last page, up to it.  What lies behind the last position may be anything, and
          // 0 * NaN would reach O: its rows are read as zeros
          const int items = 2 * prefix_last_pages(w);
          for (int v = 0; v < items; ++v) {
            const int panel = 4 * (v & 1) + 2 * rank;
            const int r = __shfl_sync(0xffffffffu, rk, v >> 1);
            const int nv = w.end - (w.begin + t * kTile + (v >> 1) * LS_PAGE);  // valid rows of the page
            if (lane == 0) go = open_slot();
            go = __shfl_sync(0xffffffffu, go, 0);
            if (!go) break;
            const uint32_t dst = ring + s * kSlotBytes, bar = full0 + s * 8;
            if (nv > 0 && nv < LS_PAGE && r != oob) {
              const int l4 = (lane & 15) * 4;
              tma_gather4_pair(dst + (lane >> 4) * 8192 + l4 * 128, &row_map, bar, (panel + (lane >> 4)) * 64,
                               l4 < nv ? r + l4 : oob, l4 + 1 < nv ? r + l4 + 1 : oob, l4 + 2 < nv ? r + l4 + 2 : oob,
                               l4 + 3 < nv ? r + l4 + 3 : oob);
            } else if (lane == 0) {
              tma_load_3d_pair(dst, &v_map, bar, 0, r, panel);
            }
            next_slot();  // (every lane keeps count: this tile is the unit's last)
          }
        } else {
          // item v: page v / 2, this CTA's 128 of the 256 dims of half v % 2 of O
          int r[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) r[k] = __shfl_sync(0xffffffffu, rk, k);
          if (lane == 0) {
#pragma unroll
            for (int v = 0; v < kVItems; ++v) {
              if (!open_slot()) { go = 0; break; }
              tma_load_3d_pair(ring + s * kSlotBytes, &v_map, full0 + s * 8, 0, r[v >> 1], 4 * (v & 1) + 2 * rank);
              next_slot();
            }
          }
        }
        ok = __shfl_sync(0xffffffffu, go, 0) != 0;
        // lane 0 has kept count
        s = __shfl_sync(0xffffffffu, s, 0);
        ph = __shfl_sync(0xffffffffu, ph, 0);
        e = __shfl_sync(0xffffffffu, e, 0);
      }
    }
    // never leave with copies in flight: rank 0 holds the barriers that count them
    if (rank == 0 && lane == 0)
      for (int it = max(0, e - slots); it < e; ++it) mbar_wait(&full[it % slots], (it / slots) & 1);
    __syncwarp();
  } else if (warp == kSWarp) {
    if (rank == 0) {
      // The whole warp runs the loop and one elected lane issues: then the compiler sees that the
      // descriptors are the same for all lanes and keeps them in uniform registers, where the MMA
      // wants them (a loop inside `lane == 0` moves each one over first: 115 to 130 clocks per MMA
      // from one warp instead of the tensor cores' 65).  They advance by their address field (16-byte
      // units).  What TMA has written needs no tcgen05 fence: only TMEM, shared with the softmax, does.
      const bool issue = elect_one();
      const uint64_t q0 = make_sdesc(sbase + kOffQ, 16, 1024, kSwizzle128);
      const uint64_t k0 = make_sdesc(sbase + kOffK, 16, 1024, kSwizzle128);
      int s = 0, ph = 0, g = 0, nu = 0;  // ring slot and its phase; tiles and units so far
      bool ok = true;                    // (after a wait has given up nothing is waited for any more)
      for (int u = pair; u < units; u += npairs) {
        if (u != pair) w = prefix_unit(p, u);
        const int tiles = __shfl_sync(0xffffffffu, w.tiles, 0);
        if (tiles == 0) continue;
        ok = ok && mbar_wait(q_full, nu & 1);
        ++nu;
        for (int t = 0; t < tiles; ++t, ++g) {
          if (g >= 2) ok = ok && mbar_wait_cluster(&s_free[g & 1], ((g >> 1) - 1) & 1);
          if (!__all_sync(0xffffffffu, ok)) break;
          tc_fence_after();
          const uint32_t d = tmem + kTmemS + (g & 1) * 128;
#pragma unroll 1
          for (int c = 0; c < kPanels; ++c) {
            ok = ok && mbar_wait(&k_full[s], ph);
            const uint64_t a = q0 + c * 512, b = k0 + s * 1024;
            if (issue) {
#pragma unroll
              for (int kk = 0; kk < 4; ++kk) mma_bf16_pair(d, a + kk * 2, b + kk * 2, kIdescS, (c | kk) != 0);
              tc_commit_pair(&k_empty[s]);
            }
            if (++s == kKSlots) {
              s = 0;
              ph ^= 1;
            }
          }
          if (issue) {
            tc_commit_pair(&s_full[g & 1]);
            if (t == tiles - 1) tc_commit_pair(q_free);
          }
        }
      }
    } else if (lane == 0) {
      // rank 1: pass on that its softmax has read an S tile
      const uint32_t peer = dsmem_map(smem_u32(s_free), 0);
      int g = 0;
      bool ok = true;
      for (int u = pair; ok && u < units; u += npairs) {
        if (u != pair) w = prefix_unit(p, u);
        const int tiles = w.tiles;
        for (int t = 0; ok && t < tiles; ++t, ++g) {
          ok = mbar_wait(&s_free[g & 1], (g >> 1) & 1);
          if (ok) mbar_arrive_remote(peer + (g & 1) * 8);
        }
      }
    }
    __syncwarp();
  } else if (warp == kPvWarp) {
    if (rank == 0) {
      const bool issue = elect_one();
      const uint64_t p0 = make_sdesc(sbase + kOffP, 16, 1024, kSwizzle128);
      const uint64_t v0 = make_sdesc(sbase + kOffV, 8192, 1024, kSwizzle128);
      int s = 0, ph = 0, ps = 0, g = 0;  // V ring, P ring; tiles so far
      bool ok = true;
      for (int u = pair; u < units; u += npairs) {
        if (u != pair) w = prefix_unit(p, u);
        const int tiles = __shfl_sync(0xffffffffu, w.tiles, 0);
        const int last_pages = __shfl_sync(0xffffffffu, prefix_last_pages(w), 0);
        for (int t = 0; t < tiles; ++t, ++g) {
          ok = ok && mbar_wait(o_ready, g & 1) && mbar_wait_cluster(o_ready_peer, g & 1);
          if (!__all_sync(0xffffffffu, ok)) break;
          const int pages = t == tiles - 1 ? last_pages : 4;
#pragma unroll 1
          for (int k = 0; k < 4; ++k) {
            ok = ok && mbar_wait_cluster(&p_full[k], g & 1);
            tc_fence_after();
            const uint64_t a = p0 + ps * 512;
            if (k >= pages) {  // a page behind the unit's end: P is zero, and V was not loaded
              if (issue) tc_commit_pair(&p_free[k]);
              if (++ps == kPSlots) ps = 0;
              continue;
            }
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              ok = ok && mbar_wait(&v_full[s], ph);
              const uint64_t b = v0 + s * 1024;
              if (issue) {
#pragma unroll
                for (int kk = 0; kk < 4; ++kk)
                  mma_bf16_pair(tmem + j * 128, a + kk * 2, b + kk * 128, kIdescO, (t > 0 || k > 0 || kk > 0));
                tc_commit_pair(&v_empty[s]);
                if (j == 1) tc_commit_pair(&p_free[k]);
              }
              if (++s == kVSlots) {
                s = 0;
                ph ^= 1;
              }
            }
            if (++ps == kPSlots) ps = 0;
          }
          if (issue) tc_commit_pair(&pv_done[g & 1]);
        }
      }
    } else if (lane == 0) {
      // rank 1: pass on that its O is ready and its pages of P are written
      const uint32_t opeer = dsmem_map(smem_u32(o_ready_peer), 0), ppeer = dsmem_map(smem_u32(p_full), 0);
      int g = 0;
      bool ok = true;
      for (int u = pair; ok && u < units; u += npairs) {
        if (u != pair) w = prefix_unit(p, u);
        const int tiles = w.tiles;
        for (int t = 0; ok && t < tiles; ++t, ++g) {
          ok = mbar_wait(o_ready, g & 1);
          if (ok) mbar_arrive_remote(opeer);
          for (int k = 0; ok && k < 4; ++k) {
            ok = mbar_wait(&p_full[k], g & 1);
            if (ok) mbar_arrive_remote(ppeer + k * 8);
          }
        }
      }
    }
    __syncwarp();
  } else {
    // ========= softmax: TMEM lane l = query row l % 64, position half l / 64; columns 64 cg .. =====
    const int l = threadIdx.x & 127, half = l >> 6, r64 = l & 63, cg = warp >> 2;
    const int page = 2 * half + cg;  // this thread's page of every tile
    const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
    const float sl2 = p.scale * kLog2e;
    int g = 0;  // tiles so far
    // good: none of this warp's waits gave up.  ok: nobody's had at the last barrier, the same for all
    // softmax warps; only ok decides what barriers follow.
    bool ok = true, good = true;
    for (int u = pair; ok && u < units; u += npairs) {
      if (u != pair) w = prefix_unit(p, u);
      const int rr = rank * 64 + r64;  // row of the unit
      const bool live = rr < w.nrows;
      // positions this row sees: below its own request's length
      int lim = 0;
      if (live) {
        const int b = (w.row0 + rr) / p.H, n = p.lens[b];
        if (n < 0 || n > p.max_pages * LS_PAGE) flag(LS_DEV_BOUNDS);
        lim = min(w.end, prefix_len_of(p, b));
      }
      const int* table = p.page_table + (size_t)w.table * p.max_pages;
      float m_run = -INFINITY, l_run = 0.f;
      // page id of this thread's page of tile t (-1: behind the unit's end), one tile ahead
      auto page_id = [&](int t) {
        const int at = w.begin + t * kTile + page * LS_PAGE;
        return at < w.end ? table[at / LS_PAGE] : -1;
      };
      int id_next = page_id(0);
      float s[64];
      float mt = -INFINITY;
      // S tile of tile t (the gt-th of all) into registers, its buffer given back, the invalid positions
      // masked, the row maxima exchanged
      auto take_s = [&](int t, int gt) {
        const int id = id_next;
        const int nv = id < 0 || id >= p.num_pages ? 0 : max(0, min(LS_PAGE, lim - (w.begin + t * kTile + page * LS_PAGE)));
        id_next = page_id(t + 1);
        good = __all_sync(0xffffffffu, mbar_wait(&s_full[gt & 1], (gt >> 1) & 1)) && good;
        tc_fence_after();
        tmem_ld64(tmem + kTmemS + (gt & 1) * 128 + cg * 64 + lane_off, s);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&s_free[gt & 1]);
        if (nv < 64) {
#pragma unroll
          for (int c = 0; c < 64; ++c) s[c] = c < nv ? s[c] : -INFINITY;
        }
        float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int c = 0; c < 64; ++c) m4[c & 3] = fmaxf(m4[c & 3], s[c]);
        // the other three quarters of the row are other warps'
        float* mx = red + (gt & 1) * 256;
        mx[page * 64 + r64] = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3]));
        ok = softmax_sync_and(good);
        mt = fmaxf(fmaxf(mx[r64], mx[64 + r64]), fmaxf(mx[128 + r64], mx[192 + r64])) * sl2;
      };
      if (w.tiles > 0) take_s(0, g);
      for (int t = 0; ok && t < w.tiles; ++t, ++g) {
        float factor = 1.f;
        bool rescale = false;
        // O is rescaled only when the running maximum has grown by more than 2^8
        if (mt > m_run + 8.f) {  // also true for the first tile with data
          if (m_run != -INFINITY) {
            factor = exp2f(m_run - mt);
            rescale = true;
          }
          m_run = mt;
        }
        if (__any_sync(0xffffffffu, rescale)) {  // (never at a unit's first tile)
          // once PV of the tile before has added into O
          good = __all_sync(0xffffffffu, mbar_wait(&pv_done[(g - 1) & 1], ((g - 1) >> 1) & 1)) && good;
          tc_fence_after();
#pragma unroll 1
          for (int c0 = cg * 128; c0 < cg * 128 + 128; c0 += 32) {
            float v[32];
            tmem_ld32(tmem + lane_off + c0, v);
#pragma unroll
            for (int c = 0; c < 32; ++c) v[c] *= factor;
            tmem_st32(tmem + lane_off + c0, v);
          }
          tmem_wait_st();
          tc_fence_before();
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(o_ready);
        // a row without any valid position so far: exp2(-inf - 0) = 0
        const float mm = m_run == -INFINITY ? 0.f : m_run;
        float p4[4] = {0.f, 0.f, 0.f, 0.f};
        uint32_t pw[32];  // P rounded to bf16, the type of the MMA's operands; its sum is not
#pragma unroll
        for (int c = 0; c < 64; c += 2) {
          const float a = ex2_ftz(fmaf(s[c], sl2, -mm)), b = ex2_ftz(fmaf(s[c + 1], sl2, -mm));
          p4[c & 3] += a;
          p4[(c + 1) & 3] += b;
          __nv_bfloat162 two = __floats2bfloat162_rn(a, b);
          pw[c / 2] = *(uint32_t*)&two;
        }
        l_run = l_run * factor + ((p4[0] + p4[1]) + (p4[2] + p4[3]));
        // the next S tile is taken before this one's P goes out, which has to wait for PV: so S runs on,
        // two tiles ahead of PV (but PV of a unit's first tile is not kept waiting for the second S)
        const bool early = t > 0 && t + 1 < w.tiles;
        if (early) take_s(t + 1, g + 1);
        // the P slot's last content, three pages ago, has been read by PV: page k + 1 of the tile before,
        // or for page 3 page 0 of this one (whose earlier phases this warp has waited for itself, a
        // tile ago: the parity is enough)
        const int ps = (4 * g + page) % kPSlots;
        if (page == 3 || g > 0)
          good = __all_sync(0xffffffffu, mbar_wait(&p_free[(page + 1) & 3], (page == 3 ? g : g - 1) & 1)) && good;
        if (good) {
          uint8_t* row = sm + kOffP + ps * 8192 + r64 * 128;
#pragma unroll
          for (int c = 0; c < 8; ++c)
            *(uint4*)(row + ((c ^ (r64 & 7)) << 4)) = make_uint4(pw[4 * c], pw[4 * c + 1], pw[4 * c + 2], pw[4 * c + 3]);
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(&p_full[page]);
        }
        if (!early && t + 1 < w.tiles) take_s(t + 1, g + 1);
      }
      // ---- this unit's rows out
      float* sums = red + (g & 1) * 256;  // the next tile's maxima: nobody reads them yet
      if (ok && w.tiles > 0) good = __all_sync(0xffffffffu, mbar_wait(&pv_done[(g - 1) & 1], ((g - 1) >> 1) & 1)) && good;
      sums[page * 64 + r64] = l_run;
      ok = softmax_sync_and(good && ok);
      if (!ok) break;
      const float total = (sums[r64] + sums[64 + r64]) + (sums[128 + r64] + sums[192 + r64]);
      __syncwarp();  // (bar.sync and tcgen05.ld are .aligned: the warp has to be whole before them)
      asm volatile("bar.sync 1, 256;" ::: "memory");
      // zero: nothing to see (else at least the weight of the maximum, 1).  A NaN or +inf among the scores
      // makes the sum NaN, and o and lse with it
      const bool some = total != 0.f;
      const float inv = 1.f / total;
      const int row = w.row0 + rr;
      if (w.tiles > 0) {
        tc_fence_after();
#pragma unroll 1
        for (int c0 = cg * 128; c0 < cg * 128 + 128; c0 += 64) {
          float v[64];
          __syncwarp();  // lanes without a row come here ahead of those that store
          tmem_ld64(tmem + lane_off + c0, v);
          const int d0 = cg * 256 + half * 128 + (c0 & 127);  // column 128 j + c: dim 256 j + 128 half + c
          if (!live) continue;
          if (!p.direct) {
            const size_t step = 8 * (size_t)(u < p.blocks * p.np ? kRows : p.H);
            float* o = p.part_o + w.part * DV + (size_t)(d0 / 8) * step + 8 * rr;
#pragma unroll
            for (int c = 0; c < 64; c += 8) st_global_v8(o + (c / 8) * step, v + c);
          } else if (p.o_f32) {
            float* o = (float*)p.o + (size_t)row * DV + d0;
#pragma unroll
            for (int c = 0; c < 64; ++c) v[c] = some ? v[c] * inv : 0.f;
#pragma unroll
            for (int c = 0; c < 64; c += 4) *(float4*)(o + c) = make_float4(v[c], v[c + 1], v[c + 2], v[c + 3]);
          } else {
            uint4* o = (uint4*)((__nv_bfloat16*)p.o + (size_t)row * DV + d0);
#pragma unroll
            for (int c = 0; c < 64; c += 8) {
              uint32_t x[4];
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                __nv_bfloat162 two = __floats2bfloat162_rn(v[c + 2 * k] * inv, v[c + 2 * k + 1] * inv);
                x[k] = some ? *(uint32_t*)&two : 0u;
              }
              o[c / 8] = make_uint4(x[0], x[1], x[2], x[3]);
            }
          }
        }
        tc_fence_before();
      } else if (live && p.direct) {  // a row with nothing to see
        if (p.o_f32) {
          float4* o = (float4*)((float*)p.o + (size_t)row * DV) + page * 32;
          for (int c = 0; c < 32; ++c) o[c] = make_float4(0.f, 0.f, 0.f, 0.f);
        } else {
          uint4* o = (uint4*)((__nv_bfloat16*)p.o + (size_t)row * DV) + page * 16;
          for (int c = 0; c < 16; ++c) o[c] = make_uint4(0u, 0u, 0u, 0u);
        }
      }
      if (live && page == 0) {
        if (p.direct) {
          p.lse[row] = some ? (m_run + log2f(total)) * kLn2 : -INFINITY;
        } else {
          float2* ml = (float2*)p.part_ml + w.part + rr;
          *ml = some ? make_float2(m_run, total) : make_float2(-INFINITY, 0.f);
        }
      }
      __syncwarp();
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();  // neither CTA leaves while the other may still signal it or its MMAs run
  if (warp == kSWarp) tmem_dealloc_pair(tmem, 512);
}

// Partials of a row's units -> o and lse: weights exp2(m_i - max m), float32 sums in unit order.
// A block takes 32 rows x 64 dims.  All (max, sum) pairs are fetched first, so that the loads of the
// parts' values depend on nothing but shared memory and go out together (one part after the other,
// 9 parts took 9 us, now 4).  Bound by the partials, 2 KB per row and unit, that attn_prefix_tc has just
// left in L2.
constexpr int kCombineRows = 32;
__global__ void __launch_bounds__(256) prefix_attn_combine(const PrefixParams p) {
  using namespace pfx;
  extern __shared__ float2 ml_all[];  // [parts][kCombineRows]
  griddep_wait();
  const int lane = lane_id(), warp = warp_id();
  const int rows = p.B * p.H, row = (int)(blockIdx.x >> 3) * kCombineRows + lane;
  const int d8 = (blockIdx.x & 7) * 8 + warp;  // this warp's group of 8 dims
  const int npp = p.blocks > 0 ? p.np : 0, n = npp + p.no;
  const int r = min(row, rows - 1), b = r / p.H;
  // part i of row r: the first row of its unit among the partials, its own place there, the unit's rows
  auto part = [&](int i, long long& unit0, int& at, int& nr) {
    if (i < npp) {
      unit0 = ((long long)i * p.blocks + r / kRows) * kRows;
      at = r % kRows;
      nr = kRows;
    } else {
      unit0 = (long long)p.blocks * p.np * kRows + ((long long)(i - npp) * p.B + b) * p.H;
      at = r - b * p.H;
      nr = p.H;
    }
  };
  for (int i = warp; i < n; i += 8) {
    long long u0;
    int at, nr;
    part(i, u0, at, nr);
    ml_all[i * kCombineRows + lane] = ((const float2*)p.part_ml)[u0 + at];
  }
  __syncthreads();
  float M = -INFINITY;
  for (int i = 0; i < n; ++i) M = fmaxf(M, ml_all[i * kCombineRows + lane].x);
  float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f}, total = 0.f;
  constexpr int kBatch = 6;  // parts whose values are in flight at once
  for (int i0 = 0; i0 < n; i0 += kBatch) {
    float x[kBatch][8], wgt[kBatch];
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      wgt[j] = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) x[j][e] = 0.f;
      if (i0 + j < n) {
        const float2 v = ml_all[(i0 + j) * kCombineRows + lane];
        if (v.y != 0.f) {  // (a unit without positions has written no values)
          long long u0;
          int at, nr;
          part(i0 + j, u0, at, nr);
          ld_global_v8(p.part_o + u0 * DV + ((size_t)d8 * nr + at) * 8, x[j]);
          wgt[j] = exp2f(v.x - M);
          total = fmaf(wgt[j], v.y, total);
        }
      }
    }
#pragma unroll
    for (int j = 0; j < kBatch; ++j)
#pragma unroll
      for (int e = 0; e < 8; ++e) acc[e] = fmaf(wgt[j], x[j][e], acc[e]);
  }
  if (row >= rows) return;
  const float inv = total != 0.f ? 1.f / total : 0.f;  // (NaN stays NaN)
  if (p.o_f32) {
    float4* o = (float4*)((float*)p.o + (size_t)row * DV + d8 * 8);
    o[0] = make_float4(acc[0] * inv, acc[1] * inv, acc[2] * inv, acc[3] * inv);
    o[1] = make_float4(acc[4] * inv, acc[5] * inv, acc[6] * inv, acc[7] * inv);
  } else {
    uint32_t x[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      __nv_bfloat162 two = __floats2bfloat162_rn(acc[2 * k] * inv, acc[2 * k + 1] * inv);
      x[k] = *(uint32_t*)&two;
    }
    *(uint4*)((__nv_bfloat16*)p.o + (size_t)row * DV + d8 * 8) = make_uint4(x[0], x[1], x[2], x[3]);
  }
  if (d8 == 0) p.lse[row] = total != 0.f ? (M + log2f(total)) * kLn2 : -INFINITY;
}

}  // namespace ls
