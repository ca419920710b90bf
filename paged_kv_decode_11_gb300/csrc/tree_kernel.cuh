// tree_kernel.cuh — attention of a tree of drafted tokens over a paged cache, on the
// fifth-generation tensor cores (tcgen05). Instantiated by tree_16bit.cu, tree_e4m3_head.cu and
// tree_e4m3_block.cu.
//
// The mathematics: sequence n has L new tokens, the nodes of a tree, whose keys and values
// lie behind the P tokens before them, node m at position P + m. Row (node i, head) sees
// the keys j < P and those nodes m whose bit is set in the node's mask (a chain, without
// masks: m <= i); out = softmax(scale q K^T) V over what it sees.
//
// Few rows, long contexts: the keys are read once and bound it, so that every SM has to
// read its share of them, whatever the batch. An item is a row tile (up to 128 (node, head)
// rows, the MMA's M) of one sequence and KV head; its keys are tiles of 128 (64 at D =
// 256). The items' key tiles are laid end to end, each item's behind a few places for what its
// beginning costs, and cut into as many equal ranges as there are SMs; a CTA walks through its
// range, segment by segment (the part of one item that lies in it). Where a cut falls inside an
// item each side writes its rows' normalised O and log2 sum to the workspace, and a second, small
// kernel merges them (tree_merge.cu). The ranges follow from the lengths alone, so results do not
// depend on timing.
//
// In a CTA: seven producer warps (four of K, three of V) copy tiles into two rings and run ahead
// of the segments; an E4M3 cache goes through a staging ring and is converted to f16 on the
// way (exact); the K producers also bring each segment's queries, as soon as the last S product
// of the one before is done. One MMA warp issues
//   S[128 x KEYS]  = Q . K_tile^T      and      O[128 x D] += P . V_tile,
// S, P and O in tensor memory, P written over its own S, up to three tiles of S ahead. Two
// softmax groups of four warps (one at D = 256) each take 64 keys of every tile, a row per
// thread, in chunks of 16 that are read twice, for the maximum and for P. The two threads of a
// row tell each other their maxima and keep one reference for P and O.
//   A tile of 64 rows or fewer is held 2 or 4 times in the 128 rows of the MMA, and each
// copy takes another part of its group's keys (its P is 0 in the others), so that the
// softmax still has all its threads where there are 16 rows to a KV head.
//   Block scales: a code stands for code * 2^e of its block and KV head; the codes go
// through the MMAs as they are, 2^ek joins a score as a factor and P carries 2^ev as an
// addend of its exponent, with a reference of its own for P and O.
//   Scores that a row does not see are -inf before anything is done with them. A weight of 0
// does not mask V (0 times NaN), so V of the tree goes into the product with 0 in place of what
// is no number; the merge adds that to the rows that see it.
//
// What bounds it (GB300, 32 query heads on 8 KV heads of 128): 16-bit caches, the bandwidth:
// another tile costs an SM 1.5 us, 6.6 TB/s over all; eight contexts of 16,384 with trees of 16
// take 97 us (5.5 TB/s), 32 of 4,096 104 us (5.2), 128 of 1,024 121 us (4.5). 8-bit caches, the
// conversion: 1.25 to 1.4 us a tile (1.75 with block scales and 128 rows, whose softmax has most
// to do), where the bandwidth alone would take 0.75; of that 1,800 cycles are traffic of shared
// memory (staged, read, written as f16, read by the MMAs): the same three shapes take 85, 98 and
// 132 us with a scale per head, 91, 104 and 139 with block scales. Beside the tiles a call costs
// some 12 us of latencies that follow one another (17 with an 8-bit cache), and a segment 3 us
// and more.
#pragma once
#include "block_scale.cuh"
#include "tc.cuh"
#include "tree_work.cuh"

namespace pkv {

template <int D, bool KV8>
struct TreeCfg {
  static constexpr int NG = D <= 128 ? 2 : 1;              // softmax groups
  static constexpr int HALF = 64;                          // keys of a tile that a group takes
  static constexpr int KEYS = tree_keys(D);                // keys per tile
  static constexpr int PAGES = KEYS / kBS;
  static constexpr int NSB = 3;                            // S buffers
  static constexpr int PK = 4, PV = 3;                     // producer warps of K and of V
  static constexpr int W_K = 4 * NG, W_MMA = W_K + PK, W_V = W_MMA + 1;
  static constexpr int WARPS = W_V + PV, THREADS = 32 * WARPS;
  static constexpr int SOFT = NG * 128;                    // softmax threads
  static constexpr int NBOX = D / 64;                      // 128-byte column blocks per row
  static constexpr int Q_BOX = kTreeRows * 128;
  static constexpr int Q_BYTES = NBOX * Q_BOX;
  static constexpr int KV_BOX = PAGES * kBS * 128;
  static constexpr int KV_BYTES = NBOX * KV_BOX;           // one K (or V) tile
  static constexpr int NST = D == 64 ? (KV8 ? 4 : 6) : D == 128 ? (KV8 ? 2 : 3) : 2;
  static constexpr int NSS = !KV8 ? 0 : D <= 128 ? 2 : 1;  // staging stages per operand
  static constexpr int STG_PAGE = kBS * D;
  static constexpr int STG_BYTES = PAGES * STG_PAGE;
  static constexpr int SMEM_BYTES = Q_BYTES + 2 * NST * KV_BYTES + 2 * NSS * STG_BYTES;
  static constexpr uint32_t TMEM_COLS = 512;
  // What a segment costs beside its tiles, in tiles, for the ranges' lengths. (0, 2, 3, 4, 6 and 8
  // tiles: 114, 75, 66, 66, 67 and 70 us on 64 contexts of 100 to 1,500 tokens; 231, 212, 209, 208,
  // 209 and 209 us on 64 of 1,024 to 8,192; with block scales 135, 88, 77, 74, 76 and 80 us and 244,
  // 218, 214, 208, 204 and 205 us. D = 128; at 256, where a tile is 64 keys, it was not measured.)
  static constexpr int COST = 4;
  static_assert(KEYS == NG * HALF, "a half of a tile to each group");
  static_assert(NSB * KEYS + D <= (int)TMEM_COLS, "tensor memory");
};

// What the CTA's warps share beside the tiles, which begin at the next KB behind it.
template <int D, bool KV8, bool QBF16>
struct TreeShared {
  using Cfg = TreeCfg<D, KV8>;
  uint64_t full_k[Cfg::NST], empty_k[Cfg::NST], full_v[Cfg::NST], empty_v[Cfg::NST];
  uint64_t s_bar[Cfg::NSB], o_bar[Cfg::NSB], p_bar[Cfg::NSB];   // S ready, P.V done, P written
  uint64_t q_bar;                                       // a segment's queries are in place
  TreeStart begin, end;                                 // of the range, and of the next one
  uint32_t tmem_base;
  // KV8, bf16 q: the shift of each row, of four segments (S runs three tiles ahead at most)
  int8_t shift[KV8 && QBF16 ? 4 : 1][kTreeRows];
  union {
    int64_t sum[2][Cfg::WARPS];                         // the plan's
    // what a row's threads tell each other: of a tile's maximum (two tiles), and at a
    // segment's end their log2 sums
    float top[Cfg::NG > 1 ? 2 : 1][Cfg::NG][kTreeRows];
    float lse[Cfg::NG][kTreeRows];
  };
  uint32_t odd_v;                     // not 0: V of some tree has had elements that are no numbers
};

// The item and key tile at place `at` of a sequence, `ahead` key tiles behind the first one's.
// An item's places are COST that stand for no tile, then its tiles.
template <int COST>
__device__ __forceinline__ TreeStart tree_start(const TreeSeq& s, int n, int64_t at,
                                                int64_t ahead) {
  TreeStart b;
  b.s = s;
  b.n = n;
  const int places = s.kt + COST;
  const int64_t item =
      at >> 31 == 0 ? (int64_t)((uint32_t)at / (uint32_t)places) : at / places;
  b.t0 = max((int)(at - item * places) - COST, 0);
  b.h = (int)((uint32_t)item / (uint32_t)s.rt);
  b.r = (int)item - b.h * s.rt;
  b.ahead = ahead + item * s.kt + b.t0;
  return b;
}

// Copies of a tile's rows in the MMA's 128: the softmax's part of a tile is 64 keys for each
// thread, 32 or 16.
__device__ __forceinline__ int tree_copies(int rows) { return rows <= 32 ? 4 : rows <= 64 ? 2 : 1; }

// Elements of eight 16-bit values that are no numbers (exponent all ones) to 0. True: there were
// some.
template <bool BF16>
__device__ __forceinline__ bool tree_only_numbers(uint4& v) {
  constexpr uint32_t EXP = BF16 ? 0x7F807F80u : 0x7C007C00u, ONE = BF16 ? 0x00800080u : 0x04000400u;
  auto odd = [](uint32_t w) { return ((w & EXP) + ONE) & 0x80008000u; };   // of each, the sign bit
  const uint32_t a = odd(v.x), b = odd(v.y), c = odd(v.z), d = odd(v.w);
  if ((a | b | c | d) == 0u) return false;
  auto clear = [](uint32_t w, uint32_t o) { return w & ~((o >> 15) * 0xFFFFu); };
  v = make_uint4(clear(v.x, a), clear(v.y, b), clear(v.z, c), clear(v.w, d));
  return true;
}

// The same for sixteen E4M3 codes (NaN is all that is no number).
__device__ __forceinline__ bool tree_only_numbers_e4m3(uint4& v) {
  auto odd = [](uint32_t w) { return __vcmpeq4(w & 0x7F7F7F7Fu, 0x7F7F7F7Fu); };
  const uint32_t a = odd(v.x), b = odd(v.y), c = odd(v.z), d = odd(v.w);
  if ((a | b | c | d) == 0u) return false;
  v = make_uint4(v.x & ~a, v.y & ~b, v.z & ~c, v.w & ~d);
  return true;
}

__device__ __forceinline__ uint32_t tree_swz(uint32_t r, uint32_t chunk) {
  return r * 128u + ((chunk ^ (r & 7u)) << 4);
}

// 2^x by the SFU's approximation (flushes subnormal results to 0; 2^-inf = 0).
__device__ __forceinline__ float tree_ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// log2 of a normal x, by the SFU: off by 2^-22 at most where x is in [0.5, 2], else by that much
// of the result.
__device__ __forceinline__ float tree_lg2(float x) {
  float y;
  asm("lg2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// A lane's chunks of a staged page of codes (of each pass one, from address `at` and tile row `row`
// on): rows from `valid` on, which may be of a page not loaded, to 0, NaN in rows from `tree` on
// too. True: there was such a NaN.
template <int D>
static __device__ __noinline__ bool tree_clean_page(uint32_t at, int row, int valid, int tree) {
  bool odd = false;
#pragma unroll
  for (int k = 0; k < kBS * D / 512; ++k, at += 512, row += 512 / D) {
    uint4 x = make_uint4(0u, 0u, 0u, 0u);
    if (row < valid) {
      if (row < tree) continue;
      x = lds128(at);
      if (!tree_only_numbers_e4m3(x)) continue;
      odd = true;
    }
    sts128(at, x);
  }
  return odd;
}

// The rest of a bounded wait: false once it ran out. (Out of line, as what else is not on the
// tile's path: the kernel's loops are at their fastest while they stay in the instruction
// caches.)
static __device__ __noinline__ bool tree_wait(uint64_t* bar, uint32_t parity, unsigned int* err) {
  if (mbar_wait_bounded(bar, parity)) return true;
  atomicOr(err, PKV_DEVERR_TIMEOUT);
  return false;
}

constexpr float kTreeSlack = 8.f;     // a reference moves when the maximum outgrows it by 2^8

// KV: the cache type; the MMAs take bf16 operands for a bf16 cache and f16 ones otherwise.
// QBF16: the query and output type. BSC: E4M3 with block scales.
template <int D, int KV, bool QBF16, bool BSC>
__global__ void __launch_bounds__(TreeCfg<D, KV == KV_E4M3>::THREADS, 1)
    tree_kernel(const __grid_constant__ TreeParams p) {
  constexpr bool KV8 = KV == KV_E4M3, BF16 = KV == KV_BF16;
  static_assert(!BSC || KV8, "block scales are for E4M3 codes");
  using Cfg = TreeCfg<D, KV8>;
  using Work = TreeWork<Cfg::KEYS, KV8>;
  constexpr int NG = Cfg::NG, NST = Cfg::NST, NSB = Cfg::NSB, KEYS = Cfg::KEYS;
  constexpr int PAGES = Cfg::PAGES, NSS = KV8 ? Cfg::NSS : 1;
  using Shared = TreeShared<D, KV8, QBF16>;
  static_assert((sizeof(Shared) + 1023) / 1024 * 1024 + Cfg::SMEM_BYTES <= 227 * 1024,
                "shared memory (static + dynamic)");
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  __shared__ Shared shared;
  auto &full_k = shared.full_k, &empty_k = shared.empty_k;
  auto &full_v = shared.full_v, &empty_v = shared.empty_v;
  auto &s_bar = shared.s_bar, &o_bar = shared.o_bar, &p_bar = shared.p_bar;
  auto& q_bar = shared.q_bar;
  auto &s_begin = shared.begin, &s_end = shared.end;

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t base = smem_u32(smem_raw);
  uint8_t* pK = smem_raw + Cfg::Q_BYTES;
  uint8_t* pV = pK + NST * Cfg::KV_BYTES;
  uint8_t* pStg = pV + NST * Cfg::KV_BYTES;
  const uint32_t sQ = base, sK = sQ + Cfg::Q_BYTES, sV = sK + NST * Cfg::KV_BYTES;

  bool failed = false;                                  // a wait ran out: stop waiting
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    if (!failed && !mbar_try_wait(bar, parity)) failed = !tree_wait(bar, parity, p.err);
  };

  if (warp == Cfg::W_MMA && lane == 0) {
    for (int s = 0; s < NST; ++s) {
      // the lanes that load; KV8: the warps that convert
      mbar_init(&full_k[s], KV8 ? Cfg::PK : 32 * Cfg::PK);
      mbar_init(&empty_k[s], 1);
      mbar_init(&full_v[s], KV8 ? Cfg::PV : 32 * Cfg::PV);
      mbar_init(&empty_v[s], 1);
    }
    for (int b = 0; b < NSB; ++b) {
      mbar_init(&s_bar[b], 1);
      mbar_init(&o_bar[b], 1);
      mbar_init(&p_bar[b], Cfg::SOFT / 32);
    }
    mbar_init(&q_bar, KV8 ? Cfg::PK : 32 * Cfg::PK);
    shared.odd_v = 0u;
    fence_barrier_init();
  }
  if (warp == 0) tc::alloc(&shared.tmem_base, Cfg::TMEM_COLS);
  // the merge behind this kernel may become resident now; it waits for this grid
  if (tid == 0) griddep_launch_dependents();
  // launched as a programmatic dependent: nothing is read before the grids ahead are done
  griddep_wait();

  // ---- the plan: this CTA's range of the key tiles of all items. Up to 32 sequences each warp
  // makes it by itself, a lane to a sequence; more by the whole CTA ----------------------------
  const int cta = blockIdx.x;
  int64_t places, tiles, per;                           // of all items; places of a range
  {
    const bool alone = p.num_seqs <= 32;
    const int who = alone ? lane : tid;
    const int each = alone ? 1 : (p.num_seqs + Cfg::THREADS - 1) / Cfg::THREADS;
    const int n0 = min(who * each, p.num_seqs), n1 = min(n0 + each, p.num_seqs);
    TreeSeq one{};
    auto items = [&](int n) {
      bool bad;
      one = tree_seq<KEYS>(p, p.cu_q_lens[n], p.cu_q_lens[n + 1], p.seq_lens[n], &bad);
      if (bad && cta == 0) atomicOr(p.err, PKV_DEVERR_QLEN);
      return (int64_t)one.rt * p.Hkv;
    };
    int64_t my_places = 0, my_tiles = 0;
#pragma unroll 1
    for (int n = n0; n < n1; ++n) {
      const int64_t i = items(n);
      my_places += i * (one.kt + Cfg::COST);
      my_tiles += i * one.kt;
    }
    int64_t a = my_places, b = my_tiles;                // of the warp's lanes so far
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t x = __shfl_up_sync(0xFFFFFFFFu, a, o), y = __shfl_up_sync(0xFFFFFFFFu, b, o);
      if (lane >= o) {
        a += x;
        b += y;
      }
    }
    places = __shfl_sync(0xFFFFFFFFu, a, 31);
    tiles = __shfl_sync(0xFFFFFFFFu, b, 31);
    int64_t ahead_p = a - my_places, ahead_t = b - my_tiles;
    if (!alone) {
      if (lane == 31) {
        shared.sum[0][warp] = a;
        shared.sum[1][warp] = b;
      }
      __syncthreads();
      places = tiles = 0;
#pragma unroll 1
      for (int w = 0; w < Cfg::WARPS; ++w) {
        if (w < warp) {
          ahead_p += shared.sum[0][w];
          ahead_t += shared.sum[1][w];
        }
        places += shared.sum[0][w];
        tiles += shared.sum[1][w];
      }
    }
    per = max((places + p.ctas - 1) / p.ctas, (int64_t)1);
    // this range's begin and the next one's, by the thread that has their sequence
#pragma unroll 1
    for (int e = 0; e < 2; ++e) {
      int64_t at = (cta + e) * per - ahead_p, ahead = ahead_t;
      if (at < 0 || at >= my_places || (alone && warp != 0)) continue;
      int n = n0;
#pragma unroll 1
      for (; n < n1 - 1; ++n) {
        const int64_t i = items(n), x = i * (one.kt + Cfg::COST);
        if (at < x) break;
        at -= x;
        ahead += i * one.kt;
      }
      if (n1 - n0 > 1) (void)items(n);
      (e == 0 ? s_begin : s_end) = tree_start<Cfg::COST>(one, n, at, ahead);
    }
  }
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  const int64_t begin = cta * per;
  const int n_tiles = begin >= places ? 0 : (int)((begin + per >= places ? tiles : s_end.ahead) -
                                                  s_begin.ahead);
  const uint32_t tm = shared.tmem_base;
  const uint32_t tS = tm;                               // S buffer b at KEYS b, group g's half at 64 g
  const uint32_t tO = tm + NSB * KEYS;

  const bool k_warp = warp >= Cfg::W_K && warp < Cfg::W_K + Cfg::PK;
  if (k_warp || warp >= Cfg::W_V) {
    // ---- producers: of the np warps of an operand, warp pw copies units pw, pw + np, .. of each
    // tile: eight rows of a page, or (KV8) a page, both contiguous in the cache, 16 bytes a lane.
    // (Copies by the lanes, because a page of 16 tokens is a box of 2 KB to a tensor map: some
    // 300 cycles of its warp for each TMA load, 2,000 a tile for three V warps, were what a tile
    // took.) Block ids are read 32 pages at a time, a chunk (the tiles of 32 pages of one segment)
    // ahead.
    if (tid == Cfg::THREADS - 1) {
      // where the range begins inside an item: the item's CTAs, for the merge
      TreeSplit d{};
      const TreeStart& b = s_begin;
      if (n_tiles > 0 && b.t0 > 0) {
        const int64_t item = begin - b.t0;              // its first key tile
        d.first = (int)(item / per);
        d.last = (int)((item + b.s.kt - 1) / per);
        d.row = b.s.q0 + b.r * p.q_tile;
        d.nodes = min(p.q_tile, b.s.L - b.r * p.q_tile);
        d.head = b.h;
        d.seq = b.n;
        d.node0 = b.r * p.q_tile;
      }
      p.splits[cta] = d;
      if (cta + 1 == p.ctas) p.splits[p.ctas] = TreeSplit{};
    }
    __syncwarp();
    const int np = k_warp ? Cfg::PK : Cfg::PV, pw = k_warp ? warp - Cfg::W_K : warp - Cfg::W_V;
    uint64_t* full_x = k_warp ? full_k : full_v;
    uint64_t* empty_x = k_warp ? empty_k : empty_v;
    // KV8: a lane's chunk (16 codes) and first row of a page. Eight lanes of a store have the four
    // chunks of a 64-element column block in an even and an odd row: different banks
    constexpr int CPC = D / 16, RP8 = 32 / CPC, PASSES = kBS / RP8;
    const int x = (lane & 3) | (((lane >> 3) & (CPC / 4 - 1)) << 2);
    const int rsub = ((lane >> 2) & 1) | ((lane / (2 * CPC)) << 1);
    const int lane_at = KV8 ? rsub * D + 16 * x : 16 * lane;
    const uint8_t* cache = static_cast<const uint8_t*>(k_warp ? p.k_cache : p.v_cache) + lane_at;
    const uint32_t ring = k_warp ? sK : sV;
    constexpr int CHUNK = 32 / PAGES;                   // tiles of a chunk
    Work ahead(p, s_begin, n_tiles);                  // the segment of the next chunk
    int c_t = ahead.t0;                                 // and where in it that begins
    struct Chunk { int t, cnt, pages, h, raw; };        // raw: this lane's page's block id
    auto next_chunk = [&]() {
      Chunk c{0, 0, 0, 0, 0};
      if (ahead.cnt == 0) return c;
      c.t = c_t;
      c.cnt = min(CHUNK, ahead.t0 + ahead.cnt - c_t);
      c.pages = (ahead.s.ctx + kBS - 1) / kBS;
      c.h = ahead.h;
      const int lp = c_t * PAGES + lane;
      if (lp < c.pages && lane < c.cnt * PAGES)
        c.raw = p.block_tables[(int64_t)ahead.n * p.max_blocks + (lp >> p.ppb_shift)];
      c_t += c.cnt;
      if (c_t == ahead.t0 + ahead.cnt) {
        ahead.next();
        c_t = ahead.t0;
      }
      return c;
    };
    Chunk cur = next_chunk(), nxt{0, 0, 0, 0, 0};
    bool want_next = true;                              // nxt is to be read
    int z = 0, done = -1;                               // page rows of cur (none: -1), tiles issued
    auto rows_of = [&](const Chunk& c) {
      int id = c.raw;
      if (id < 0 || id >= p.num_blocks) {
        atomicOr(p.err, PKV_DEVERR_BLOCK_ID);
        id = 0;
      }
      const int lp = c.t * PAGES + lane;
      return ((id * p.Hkv + c.h) << p.ppb_shift) + (lp & ((1 << p.ppb_shift) - 1));
    };
    // 16-bit: a lane's place in a unit, less the part that depends on the pass alone
    constexpr int CPR = D / 8, RPI = CPR >= 32 ? 1 : 32 / CPR;   // 16-byte chunks a row; rows a pass
    const int u_row = lane / CPR, u_ch = lane % CPR;
    const uint32_t u_at = (u_ch / 8) * Cfg::KV_BOX + u_row * 128 + (((u_ch & 7) ^ u_row) << 4);
    const uint32_t stage = smem_u32(pStg) + (k_warp ? 0 : NSS * Cfg::STG_BYTES) + 16 * lane;
    // copies of the range's tile u: into ring stage u % NST or (KV8) staging stage u % NSS
    auto issue = [&](int u) {
      if (done < 0) {
        z = rows_of(cur);
        done = 0;
      } else if (done == cur.cnt) {
        if (want_next) nxt = next_chunk();
        cur = nxt;
        done = 0;
        z = rows_of(cur);
        want_next = true;
      }
      const int npg = min(PAGES, cur.pages - (cur.t + done) * PAGES);
      if constexpr (KV8) {
        const uint32_t dst = stage + (u % NSS) * Cfg::STG_BYTES;
#pragma unroll 1
        for (int pg = pw; pg < npg; pg += np) {
          const int zz = __shfl_sync(0xFFFFFFFFu, z, done * PAGES + pg);
          const uint8_t* src = cache + (int64_t)zz * Cfg::STG_PAGE;   // (its lane's chunk)
#pragma unroll
          for (int k = 0; k < Cfg::STG_PAGE / 512; ++k)
            cp_async16_l2(dst + pg * Cfg::STG_PAGE + k * 512, src + k * 512);
        }
        cp_async_commit();
      } else {
        const uint32_t dst = ring + (u % NST) * Cfg::KV_BYTES + u_at;
#pragma unroll 1
        for (int un = pw; un < 2 * npg; un += np) {
          const int zz = __shfl_sync(0xFFFFFFFFu, z, done * PAGES + un / 2);
          const uint8_t* src = cache + (int64_t)zz * (kBS * D * 2) + (un & 1) * (8 * D * 2);
#pragma unroll
          for (int k = 0; k < 8 / RPI; ++k)
            cp_async16_l2((dst + un * 1024 + k * RPI * 128) ^ ((k * RPI) << 4), src + k * 512);
        }
        cp_async_mbar_arrive_noinc(&full_x[u % NST]);
      }
      ++done;
      if (want_next) {                                  // behind the copies, whose turn is sooner
        nxt = next_chunk();
        want_next = false;
      }
    };
    // the K producers: a segment's queries into every copy's rows (rows past the last hold the
    // last one's); with an E4M3 cache each lane then scales what it has copied to f16
    constexpr int RPP = 32 * Cfg::PK / CPR;             // rows a pass of the four warps
    Work qw(p, s_begin, n_tiles);
    int q_seg = 0, q_end = 0;                           // segments brought; where theirs ends
    const int q_row0 = (tid - 32 * Cfg::W_K) / CPR, q_chunk = (tid - 32 * Cfg::W_K) % CPR;
    const uint32_t inv_G = 65536u / p.G + 1u;           // x / G = x inv_G >> 16 for x < 128, G <= 16
    auto bring_queries = [&]() {
      const int used = qw.nodes() * p.G, reps = tree_copies(used), RP = kTreeRows / reps;
      const uint16_t* src = static_cast<const uint16_t*>(p.q) + 8 * q_chunk +
                            ((int64_t)(qw.s.q0 + qw.node0()) * p.Hq + (int64_t)qw.h * p.G) * D;
      const uint32_t dst = sQ + (q_chunk / 8) * Cfg::Q_BOX;
#pragma unroll 1
      for (int qr = q_row0; qr < RP; qr += RPP) {
        const int r = min(qr, used - 1), node = (int)(r * inv_G >> 16);
        const uint16_t* from = src + ((int64_t)node * p.Hq + r - node * p.G) * D;
#pragma unroll 1
        for (int m = qr; m < (KV8 ? qr + 1 : kTreeRows); m += RP)
          cp_async16_l2(dst + tree_swz(m, q_chunk % 8), from);
      }
      if constexpr (!KV8) {
        cp_async_mbar_arrive_noinc(&q_bar);
      } else {
        cp_async_wait_all();
#pragma unroll 1
        for (int qr = q_row0; qr < RP; qr += RPP) {     // (the same passes for a row's lanes)
          uint4 x = lds128(dst + tree_swz(qr, q_chunk % 8));
          if constexpr (QBF16) {
            uint32_t mx = max(max(bf16x2_max_abs(x.x), bf16x2_max_abs(x.y)),
                              max(bf16x2_max_abs(x.z), bf16x2_max_abs(x.w)));
#pragma unroll
            for (int o = 1; o < CPR; o <<= 1) mx = max(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, o));
            const int sh = q_f16_shift(mx);
            const float inv = pow2f(-sh);
            x = make_uint4(bf16x2_to_f16x2_scaled(x.x, inv), bf16x2_to_f16x2_scaled(x.y, inv),
                           bf16x2_to_f16x2_scaled(x.z, inv), bf16x2_to_f16x2_scaled(x.w, inv));
            if (q_chunk == 0)
#pragma unroll 1
              for (int m = qr; m < kTreeRows; m += RP) shared.shift[q_seg & 3][m] = (int8_t)sh;
          }
#pragma unroll 1
          for (int m = qr; m < kTreeRows; m += RP) sts128(dst + tree_swz(m, q_chunk % 8), x);
        }
        fence_proxy_async_smem();                       // the tensor cores read these stores
        __syncwarp();
        if (lane == 0) mbar_arrive(&q_bar);
      }
      ++q_seg;
      q_end += qw.cnt;
      qw.next();
    };
    // before tile u takes its ring stage: the product that read tile u - NST there is done,
    // and with it, where that was its segment's last, those that read its queries
    auto stage_free = [&](int u) {
      if (u >= NST) wait(&empty_x[u % NST], ((u / NST) - 1) & 1);
      if (k_warp && qw.cnt > 0 && (u == 0 || u - NST + 1 == q_end)) bring_queries();
    };
    const int u_end = k_warp ? n_tiles + NST : n_tiles;   // (K: to the last segment's queries)
    if constexpr (!KV8) {
      for (int u = 0; u < u_end; ++u) {
        stage_free(u);
        if (u < n_tiles) issue(u);
      }
    } else {
      Work w(p, s_begin, n_tiles);
      int t = w.t0;
      // the warp turns its pages of staged tile u into f16 in ring stage u % NST, NaN in the V of
      // the tree into zeros, and refills the staging stage. A lane has the chunk of every
      // RP8-th row that it has copied
      uint32_t into[PASSES];
#pragma unroll
      for (int k = 0; k < PASSES; ++k)
        into[k] = (x / 4) * Cfg::KV_BOX + tree_swz(k * RP8 + rsub, 2 * (x % 4));
#pragma unroll 1
      for (int u = -NSS; u < u_end; ++u) {
        cp_async_wait_group<NSS - 1>();                 // staged: tile u
        if (u >= 0) stage_free(u);
        if (u >= 0 && u < n_tiles) {
          const int st = u % NST, valid = w.s.ctx - t * KEYS;
          // V: the tile's first row of the tree, where NaN has to go (of K, scores are masked)
          const int tree = k_warp ? KEYS : w.before() - t * KEYS;
          const uint32_t src = stage + (u % NSS) * Cfg::STG_BYTES;
          const uint32_t dst = ring + st * Cfg::KV_BYTES;
#pragma unroll 1
          for (int pg = pw; pg < PAGES; pg += np) {
            if ((pg + 1) * kBS > tree && tree_clean_page<D>(src + pg * Cfg::STG_PAGE, pg * kBS + rsub, valid, tree))
              shared.odd_v = 1u;
            uint4 e[PASSES];
#pragma unroll
            for (int k = 0; k < PASSES; ++k) e[k] = lds128(src + pg * Cfg::STG_PAGE + k * 512);
#pragma unroll
            for (int k = 0; k < PASSES; ++k) {
              const uint32_t to = dst + pg * (kBS * 128) + into[k];
              const uint4 c = e[k];
              sts128(to, make_uint4(e4m3x2_to_f16x2(c.x & 0xFFFFu), e4m3x2_to_f16x2(c.x >> 16),
                                    e4m3x2_to_f16x2(c.y & 0xFFFFu), e4m3x2_to_f16x2(c.y >> 16)));
              sts128(to ^ 16u, make_uint4(e4m3x2_to_f16x2(c.z & 0xFFFFu), e4m3x2_to_f16x2(c.z >> 16),
                                          e4m3x2_to_f16x2(c.w & 0xFFFFu), e4m3x2_to_f16x2(c.w >> 16)));
            }
          }
          fence_proxy_async_smem();                       // the tensor cores read these stores
          __syncwarp();
          if (lane == 0) mbar_arrive(&full_x[st]);
          if (++t == w.t0 + w.cnt) {
            w.next();
            t = w.t0;
          }
        }
        if (u + NSS < n_tiles) issue(u + NSS);
        else cp_async_commit();
      }
    }
  } else if (warp == Cfg::W_MMA) {
    // ---- MMA warp: whatever is ready, S products first. Tile u of the range is in S buffer
    // u % NSB. The whole warp walks through it and one lane issues, so that descriptors and
    // counters stay in uniform registers (issued by a lane by itself, each block of eight
    // products took 1,280 cycles of a tile's 3,100, and bound the kernel).
    constexpr uint32_t ID_S = tc::idesc_f16(kTreeRows, KEYS, BF16, false);
    constexpr uint32_t ID_O = tc::idesc_f16(kTreeRows, D, BF16, true);
    const uint64_t dQ = tc::sdesc(sQ, 16, 1024), dK = tc::sdesc(sK, 16, 1024);
    const uint64_t dV = tc::sdesc(sV, Cfg::KV_BOX, 1024);
    const bool elected = elect_lane();
    auto ready = [&](uint64_t* bar, uint32_t parity) {
      return __any_sync(0xFFFFFFFFu, mbar_test_wait(bar, parity)) != 0;
    };
    Work ws(p, s_begin, n_tiles), wp(p, s_begin, n_tiles);
    int us = 0, up = 0;                                 // next S, next P.V
    int s_end = ws.cnt, p_end = wp.cnt;                 // their segments' ends
    // the ring stages, S buffers and phases of both
    uint32_t s_st = 0, s_ph = 0, sb = 0, sb_ph = 1, p_st = 0, p_ph = 0, pb = 0, pb_ph = 0;
    uint32_t seg = 0, idle = 0;
    bool s_first = true, p_first = true;                // the first tile of its segment
    while (up < n_tiles) {
      bool did = false;
      if (us < n_tiles && us < up + NSB && ready(&full_k[s_st], s_ph) &&
          (!s_first || ready(&q_bar, seg & 1))) {
        // the P.V that read P from this S buffer, the last issued but two, is complete
        if (us >= NSB) wait(&o_bar[sb], sb_ph);
        if (!KV8) fence_proxy_async_smem();             // the lanes' copies, for the tensor cores
        tc::fence_after();
        const uint64_t kd = dK + s_st * (Cfg::KV_BYTES / 16);
        if (elected) {
#pragma unroll
          for (int k = 0; k < D / 16; ++k)
            tc::mma(tS + sb * KEYS, dQ + ((k / 4) * Cfg::Q_BOX + (k % 4) * 32) / 16,
                    kd + ((k / 4) * Cfg::KV_BOX + (k % 4) * 32) / 16, ID_S, k > 0 ? 1u : 0u);
          tc::commit(&s_bar[sb]);
          tc::commit(&empty_k[s_st]);
        }
        __syncwarp();
        if (++s_st == NST) {
          s_st = 0;
          s_ph ^= 1;
        }
        if (++sb == NSB) {
          sb = 0;
          sb_ph ^= 1;
        }
        s_first = false;
        if (++us == s_end) {
          ws.next();
          s_end = us + ws.cnt;
          ++seg;
          s_first = true;
        }
        did = true;
      } else if (up < us && ready(&p_bar[pb], pb_ph)) {
        wait(&full_v[p_st], p_ph);
        if (!KV8) fence_proxy_async_smem();
        tc::fence_after();
        const uint64_t vd = dV + p_st * (Cfg::KV_BYTES / 16);
        if (elected) {
#pragma unroll
          for (int k = 0; k < KEYS / 16; ++k)
            // 16 keys of P: 8 columns, a half's P at the start of its S columns
            tc::mma_ts(tO, tS + pb * KEYS + 64 * (k / 4) + 8 * (k % 4), vd + k * 2 * 1024 / 16, ID_O,
                       (!p_first || k > 0) ? 1u : 0u);
          tc::commit(&o_bar[pb]);
          tc::commit(&empty_v[p_st]);
        }
        __syncwarp();
        if (++p_st == NST) {
          p_st = 0;
          p_ph ^= 1;
        }
        if (++pb == NSB) {
          pb = 0;
          pb_ph ^= 1;
        }
        p_first = false;
        if (++up == p_end) {
          wp.next();
          p_end = up + wp.cnt;
          p_first = true;
        }
        did = true;
      }
      if (did) {
        idle = 0;
      } else if (++idle > (1u << 26)) {
        if (elected) atomicOr(p.err, PKV_DEVERR_TIMEOUT);   // nothing became ready: give up
        break;
      }
    }
    __syncwarp();
  } else {
    // ---- softmax groups -------------------------------------------------------------------
    const int grp = warp >> 2, r = tid & (kTreeRows - 1);
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    constexpr int COLS = D / NG;                        // columns of O that a group rescales and writes
    const uint32_t tOg = tO + grp * COLS + lanes;
    Work w(p, s_begin, n_tiles);
    uint32_t seg = 0;
    // BSC: of the tile's pages, one to a lane, the scale bytes, read a tile ahead by block ids
    // read two ahead; a segment's first ones while the one before ends
    uint32_t k_byte = 0u, v_byte = 0u;
    int next_id = 0;
    auto read_id = [&](const Work& x, int t) {
      const int lp = t * PAGES + lane;
      if (lane >= PAGES || t >= x.t0 + x.cnt || lp * kBS >= x.s.ctx) return 0;
      return p.block_tables[(int64_t)x.n * p.max_blocks + (lp >> p.ppb_shift)];
    };
    auto read_bytes = [&](const Work& x, int id) {      // (the page loads flag a bad id)
      const int64_t i = (int64_t)(id < 0 || id >= p.num_blocks ? 0 : id) * p.Hkv + x.h;
      k_byte = static_cast<const uint8_t*>(p.k_scales)[i];
      v_byte = static_cast<const uint8_t*>(p.v_scales)[i];
    };
    auto first_bytes = [&](const Work& x) {
      read_bytes(x, read_id(x, x.t0));
      next_id = read_id(x, x.t0 + 1);
    };
    if (BSC && w.cnt > 0) first_bytes(w);
    for (int u0 = 0; w.cnt > 0; ++seg) {
      const int used = w.nodes() * p.G;                 // rows of the tile
      const int reps = tree_copies(used);                 // copies of them in the 128 rows
      const int RP = kTreeRows / reps, copy = r / RP, row = r % RP;
      const bool mine = row < used;
      const int node = w.node0() + row / p.G;           // (of a row that is none: unused)
      const int q_row = w.s.q0 + node;
      const int P = w.before();
      // the references of the probabilities and their sum, and (BSC) of P and O
      float m_ref = -INFINITY, w_ref = -INFINITY, l = 0.f;
      float sl2 = 0.f;
      // A row's part of a tile is chunks c0 .. c1-1 of 16 keys (a page) of the group's half. They
      // are read twice, for the maximum and for P, by loops that are not unrolled: straight-line
      // code for 64 keys does not stay in the instruction caches beside the producers' loops.
      constexpr int CHUNKS = Cfg::HALF / kBS;
      const int each = CHUNKS / reps, c0 = copy * each, c1 = c0 + each;
      for (int u = u0; u < u0 + w.cnt; ++u) {
        const int t = w.t0 + (u - u0), b = u % NSB;
        const bool tail = (t + 1) * KEYS > P;           // keys of the tree, or behind it
        [[maybe_unused]] const uint32_t scale_bytes = k_byte | (v_byte << 8);
        if constexpr (BSC) {
          read_bytes(w, next_id);
          next_id = read_id(w, t + 2);
        }
        uint64_t see = ~(uint64_t)0;                    // the keys of the half that this row sees
        if (tail) {
          see = tree_sees(p, mine ? q_row : w.s.q0, mine ? node : 0,
                          t * KEYS + Cfg::HALF * grp - P, w.s.L);
          if constexpr (!KV8) {
            // V of the tree and of what lies behind it: zeros for what is no number, as a weight
            // of 0 does not keep it from a row (the rows that see it get it at the end)
            const int st = u % NST, from = max(P - t * KEYS, 0);
            // The stage's tile before, u - NST, first: a barrier tells only the last phase from the
            // one under way, and tile u - NST may not have landed, let alone been multiplied, when a
            // warp comes here (S(u - 1) waited for P.V of u - 4 alone, and NST may be 2)
            static_assert(NSB == 3 && NST >= 2, "P.V of u - 2 NST is done");
            if (u >= NST) wait(&empty_v[st], ((u / NST) - 1) & 1);
            wait(&full_v[st], (u / NST) & 1);
#pragma unroll 1
            for (int i = tid; i < (KEYS - from) * Cfg::NBOX * 8; i += Cfg::SOFT) {
              const int vr = from + i / (Cfg::NBOX * 8), rest = i % (Cfg::NBOX * 8);
              uint4* at = reinterpret_cast<uint4*>(
                  pV + st * Cfg::KV_BYTES + (rest / 8) * Cfg::KV_BOX + vr * 128 + (rest % 8) * 16);
              if (t * KEYS + vr >= w.s.ctx) {
                *at = make_uint4(0u, 0u, 0u, 0u);
              } else {
                uint4 x = *at;
                if (tree_only_numbers<BF16>(x)) {
                  *at = x;
                  shared.odd_v = 1u;
                }
              }
            }
            fence_proxy_async_smem();
          }
        }
        wait(&s_bar[b], (u / NSB) & 1);
        __syncwarp();
        tc::fence_after();
        if (u == u0) {
          sl2 = p.qk_scale_log2;                        // undoes the row's q scaling
          if constexpr (KV8 && QBF16) sl2 *= pow2f(shared.shift[seg & 3][r]);
          if constexpr (KV8 && !BSC) sl2 *= static_cast<const float*>(p.k_scales)[w.h];
          if (sl2 == 0.f) sl2 = 0x1p-126f;              // (a scale of 0: -inf stays -inf)
        }
        const uint32_t half = tS + b * KEYS + Cfg::HALF * grp + lanes;
        float x[kBS], kf = sl2, ev = 0.f;
        uint32_t bytes = 0u, seen = 0xFFFFu;            // of a chunk: scale bytes, keys seen
        auto load = [&](int i) {
          uint32_t v[kBS];
          tc::ld16(half + kBS * i, v);
          if constexpr (BSC) {
            bytes = __shfl_sync(0xFFFFFFFFu, scale_bytes, CHUNKS * grp + i);
            kf = fmaxf(sl2 * pow2_any(min((int)(bytes & 0xFFu), 254) - kE8M0Bias), 0x1p-126f);
            ev = (float)((int)(bytes >> 8) - kE8M0Bias);
          }
          tc::wait_ld();
#pragma unroll
          for (int c = 0; c < kBS; ++c) x[c] = __uint_as_float(v[c]);
          if (tail) {
            seen = (uint32_t)(see >> (kBS * i)) & 0xFFFFu;
#pragma unroll
            for (int c = 0; c < kBS; ++c)
              if (!((seen >> c) & 1u)) x[c] = -INFINITY;
          }
        };
        float mx = -INFINITY, mxw = -INFINITY;          // largest score, largest score + ev
#pragma unroll 1
        for (int i = c0; i < c1; ++i) {
          load(i);
          float m4[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
          for (int c = 4; c < kBS; ++c) m4[c % 4] = fmaxf(m4[c % 4], x[c]);
          // (a positive factor: max commutes)
          const float top = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3])) * kf;
          mx = fmaxf(mx, top);
          if constexpr (BSC) {
            mxw = fmaxf(mxw, top + ev);
            // a NaN K scale that the row sees makes its sum NaN, a V scale its P (below)
            if ((bytes & 0xFFu) == 255u && seen != 0u) l = __int_as_float(0x7FFFFFFF);
            __syncwarp();
          }
        }
        // the row's maximum over the groups, as both its threads see it
        float o_top = BSC ? mxw : mx;
        if constexpr (NG > 1) {
          shared.top[u & 1][grp][r] = o_top;
          named_barrier(1, Cfg::SOFT);
          o_top = fmaxf(shared.top[u & 1][0][r], shared.top[u & 1][1][r]);
        }
        // O's reference moves when P would pass 2^15, then to 2^7 below the row's maximum
        float& o_ref = BSC ? w_ref : m_ref;
        const float o_new = o_top - kWeightHeadLog2;
        const bool move = o_new > o_ref + kTreeSlack;
        const bool scales_o = move && o_ref != -INFINITY;
        const float alpha = scales_o ? tree_ex2(o_ref - o_new) : 1.f;
        float l_alpha = alpha;
        if constexpr (BSC) {
          const bool moves = mx > m_ref + kTreeSlack;
          l_alpha = moves && m_ref != -INFINITY ? tree_ex2(m_ref - mx) : 1.f;
          if (moves) m_ref = mx;
        }
        if (move) o_ref = o_new;
        if (u > u0 && __any_sync(0xFFFFFFFFu, scales_o)) {
          // O must hold every earlier tile before it is scaled, by each group its columns
          wait(&o_bar[(u - 1) % NSB], ((u - 1) / NSB) & 1);
          __syncwarp();
          tc::fence_after();
#pragma unroll 1
          for (int k = 0; k < COLS; k += 16) {
            uint32_t ov[16];
            tc::ld16(tOg + k, ov);
            tc::wait_ld();
#pragma unroll
            for (int c = 0; c < 16; ++c) ov[c] = __float_as_uint(__uint_as_float(ov[c]) * alpha);
            tc::st16(tOg + k, ov);
          }
          tc::wait_st();
        }
        // P over the half's scores already read: chunk i at columns 8 i .., 0 in the other copies'
        // chunks. P is rounded to the MMAs' 16-bit type, by half a step at most (bf16 2^-8, f16
        // 2^-11 of a weight); the sum takes the weights unrounded. BSC: P of a page is its
        // probabilities times 2^-back, back = w_ref - ev - m_ref; one whose V scale is so small
        // that P would leave fp32 (back above 80) keeps 2^-80 times them, 0 in f16, so that its
        // sum stays exact.
        const float ms = m_ref == -INFINITY ? 0.f : m_ref;
        [[maybe_unused]] const float wr = w_ref == -INFINITY ? 0.f : w_ref;
        float sum = 0.f;
#pragma unroll 1
        for (int i = c0; i < c1; ++i) {
          load(i);
          uint32_t pv[kBS / 2];
          float back = 0.f;
          if constexpr (BSC) back = fminf(wr - ev - ms, 80.f);
          const float sub = ms + back;
          float s4[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int c = 0; c < kBS; c += 2) {
            const float e0 = tree_ex2(fmaf(x[c], kf, -sub)), e1 = tree_ex2(fmaf(x[c + 1], kf, -sub));
            s4[c % 4] += e0;
            s4[c % 4 + 1] += e1;
            pv[c / 2] = pack2<BF16>(e0, e1);
          }
          const float ps = (s4[0] + s4[1]) + (s4[2] + s4[3]);
          sum = BSC ? fmaf(ps, tree_ex2(back), sum) : sum + ps;
          if (BSC && bytes >> 8 == 255u && seen != 0u) {
#pragma unroll
            for (int c = 0; c < kBS / 2; ++c) pv[c] = 0x7FFF7FFFu;
          }
          if constexpr (BSC) __syncwarp();
          tc::st8(half + 8 * i, pv);
        }
        l = l * l_alpha + sum;
        if (reps > 1) {
          const uint32_t zero[8] = {};
#pragma unroll 1
          for (int i = 0; i < CHUNKS; ++i)
            if (i < c0 || i >= c1) tc::st8(half + 8 * i, zero);
        }
        tc::wait_st();
        tc::fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_bar[b]);
      }

      // ---- the segment's end: O normalised by the row's sum, over its groups and for a whole
      // item over its copies (those of a part stay apart) ------------------------------------
      const int last = u0 + w.cnt - 1;
      Work then = w;
      // (not yet for a scale per head: 368 us on four contexts of 80,000, where later takes 362)
      if constexpr (!KV8 || BSC) then.next();
      if constexpr (BSC) first_bytes(then);
      wait(&o_bar[last % NSB], (last / NSB) & 1);
      __syncwarp();
      tc::fence_after();
      const bool whole = w.cnt == w.s.kt;               // else: a part, for the merge
      float lse = !(l == 0.f) ? m_ref + tree_lg2(l) : -INFINITY;
      if (NG > 1 || reps > 1) {
        shared.lse[grp][r] = lse;
        named_barrier(1, Cfg::SOFT);
        const int k0 = whole ? 0 : copy, k1 = whole ? reps : copy + 1;
        float top = -INFINITY, sum = 0.f;
#pragma unroll 1
        for (int i = NG * k0; i < NG * k1; ++i)
          top = fmaxf(top, shared.lse[i % NG][(i / NG) * RP + row]);
#pragma unroll 1
        for (int i = NG * k0; i < NG * k1; ++i) {
          const float v = shared.lse[i % NG][(i / NG) * RP + row];
          sum += v == -INFINITY ? 0.f : tree_ex2(v - top);
        }
        lse = !(sum == 0.f) ? top + tree_lg2(sum) : -INFINITY;
      }
      const float o_ref = BSC ? w_ref : m_ref;
      float f = o_ref == -INFINITY ? (lse == lse ? 0.f : lse) : tree_ex2(o_ref - lse);
      if constexpr (KV8 && !BSC)
        if (whole) f *= static_cast<const float*>(p.v_scales)[w.h];
      // a part's rows, or (whole) the copies' for their sum: [D / 4][128] float4
      const int slot = 3 * cta + (whole ? 2 : w.t0 == 0 ? 1 : 0);
      float4* po = reinterpret_cast<float4*>(p.part_o + slot * tree_part_floats(D));
      const bool direct = whole && reps == 1;
      uint16_t* orow = static_cast<uint16_t*>(p.out) +
                       ((int64_t)(mine ? q_row : 0) * p.Hq + (int64_t)w.h * p.G +
                        (mine ? row % p.G : 0)) * D;
#pragma unroll 1
      for (int c = grp * COLS; c < (grp + 1) * COLS; c += 16) {
        uint32_t v[16];
        __syncwarp();                                   // (rows that are none went on)
        tc::ld16(tO + lanes + c, v);
        tc::wait_ld();
        float o[16];
#pragma unroll
        for (int k = 0; k < 16; ++k) o[k] = f != 0.f ? __uint_as_float(v[k]) * f : 0.f;
        if (!mine) continue;
        if (direct) {
#pragma unroll
          for (int k = 0; k < 16; k += 8)
            *reinterpret_cast<uint4*>(orow + c + k) =
                make_uint4(pack2<QBF16>(o[k], o[k + 1]), pack2<QBF16>(o[k + 2], o[k + 3]),
                           pack2<QBF16>(o[k + 4], o[k + 5]), pack2<QBF16>(o[k + 6], o[k + 7]));
        } else {
#pragma unroll
          for (int k = 0; k < 16; k += 4)
            po[((c + k) / 4) * kTreeRows + r] = make_float4(o[k], o[k + 1], o[k + 2], o[k + 3]);
        }
      }
      if (grp == 0 && mine) {
        if (!whole)
          p.part_lse[slot * kTreeRows + r] = lse;
        else if (copy == 0 && p.out_lse != nullptr)
          p.out_lse[(int64_t)q_row * p.Hq + w.h * p.G + row % p.G] =
              lse == -INFINITY ? lse : lse * kLn2;
      }
      tc::fence_before();                               // O may be written again
      if (whole && reps > 1) {
        // the copies' sum: a thread takes a row's columns of group and copy, 2 or 4 copies each,
        // the loads BATCH at a time (one after the other they cost an item 3 us). 16 at a time take
        // 121 us on 128 contexts of 1,024, where 4 take 125; with a scale per head 130 and 132, but
        // with block scales 92 us on eight contexts of 16,384, where 4 at a time take 91.
        named_barrier(1, Cfg::SOFT);
        constexpr int EACH = D / 4 / NG;                // float4 of a row to load, all copies'
        constexpr int BATCH = KV8 ? 4 : EACH < 16 ? EACH : 16;
        const int two = reps >> 2;                      // log2(reps) - 1
        int k = grp * EACH + copy * (EACH / reps);
        const float4* from = po + row;
#pragma unroll 1
        for (int done = 0; done < EACH; done += BATCH, k += BATCH / reps) {
          float4 x[BATCH];
#pragma unroll
          for (int i = 0; i < BATCH; ++i)
            x[i] = from[(k + (i >> (1 + two))) * kTreeRows + (i & (reps - 1)) * RP];
#pragma unroll
          for (int i = 0; i < BATCH; i += 4) {
            float4 a = make_float4(x[i].x + x[i + 1].x, x[i].y + x[i + 1].y, x[i].z + x[i + 1].z,
                                   x[i].w + x[i + 1].w);
            float4 b = make_float4(x[i + 2].x + x[i + 3].x, x[i + 2].y + x[i + 3].y,
                                   x[i + 2].z + x[i + 3].z, x[i + 2].w + x[i + 3].w);
            if (reps == 4) a = make_float4(a.x + b.x, a.y + b.y, a.z + b.z, a.w + b.w);
            uint16_t* to = orow + 4 * (k + (i >> (1 + two)));
            if (!mine) continue;
            *reinterpret_cast<uint2*>(to) = make_uint2(pack2<QBF16>(a.x, a.y), pack2<QBF16>(a.z, a.w));
            if (reps == 2)
              *reinterpret_cast<uint2*>(to + 4) =
                  make_uint2(pack2<QBF16>(b.x, b.y), pack2<QBF16>(b.z, b.w));
          }
        }
      }
      named_barrier(1, Cfg::SOFT);                      // shared.lse, the copies' space
      u0 += w.cnt;
      if constexpr (KV8 && !BSC) then.next();
      w = then;
    }
  }
  tc::fence_before();
  __syncthreads();
  if (warp == 0) tc::dealloc(tm, Cfg::TMEM_COLS);
  // for the merge: V that was no number, and this range to find the rows that see it
  if (tid == Cfg::THREADS - 1) {
    TreeOdd* odd = p.odd + cta;
    odd->tiles = shared.odd_v != 0u ? n_tiles : 0;
    if (shared.odd_v != 0u) odd->begin = s_begin;
  }
}

// One instance and its launch, as a programmatic dependent of the kernel ahead.
template <int D, int KV, bool QBF16, bool BSC>
static pkv_status launch_tree_kernel(const TreeParams& p, cudaStream_t stream) {
  using Cfg = TreeCfg<D, KV == KV_E4M3>;
  auto kern = tree_kernel<D, KV, QBF16, BSC>;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return PKV_ERR_CUDA;
  static std::atomic<bool> attr_set[64];                // per device; the call is idempotent
  if (!attr_set[dev]) {
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg::SMEM_BYTES) !=
        cudaSuccess)
      return PKV_ERR_CUDA;
    attr_set[dev] = true;
  }
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3(p.ctas);
  cfg.blockDim = dim3(Cfg::THREADS);
  cfg.dynamicSmemBytes = Cfg::SMEM_BYTES;
  cfg.stream = stream;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, p) == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
}

}  // namespace pkv
