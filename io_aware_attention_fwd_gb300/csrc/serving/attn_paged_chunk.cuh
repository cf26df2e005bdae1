// Attention of chunks of new tokens over the pages.  Part of attn_fwd.cu: the tile
// arithmetic, the barriers and the roles are attn_varlen_sm103a's (query tiles of
// tokens x heads, two of them a work unit, four warpgroups); what differs is stated
// here.
//
//   * K and V tiles of 128 keys come page by page: a warp's lanes look up and load a
//     box of min(page, 128) rows x 64 channels each.  Boxes that no token of the unit
//     sees, and those behind the sequence's end, are read from behind the last page,
//     which gives zeros, whatever the table has for them.
//   * A unit visits the tiles of the first `sinks` keys and those from its first
//     token's window on.  Tiles that every token of a query tile sees go through
//     unmasked; the others compare each key's number with the row's limits.
//   * Work split.  Few units may have many keys (512 tokens over 32768: 64 units of
//     256 tiles for 152 SMs), so the tiles of all (unit, key head) form one list that
//     is cut into equal shares, one a CTA, a unit counting kChunkUnitCost tiles more
//     for its start and end.  A one-block kernel makes the list; units that a share's
//     end cuts leave partials (m, l, O in fp32), which a third kernel joins.  Where
//     there are few units of few keys each CTA takes one: one launch.
//
// 512 tokens over 32768 entries, 32/8 heads, D = 128: 186 to 199 us from run to run, 1370
// to 1470 TFLOP/s, of which the list takes 7, the attention 171 to 176 (its MMAs 70% of the
// tensor pipe's nominal time) and the merge 11.  A prompt of 16384 with windows of 4096: 677
// to 738 us as the power cap has it, 1320 to 1440 TFLOP/s of visible pairs, 4% more with the
// masked halves of edge tiles.

namespace {

constexpr int kChunkUnitCost = 4;  // tiles that a unit's start and end count as (2 to 7: within 2%)
constexpr int kChunkLeast = 4;     // tiles of a unit that are cut off, at least
constexpr int kChunkCtas = 152;    // shares (the workspace's size is asked for without a device)
constexpr int kChunkRows = kQTiles * kBM;

struct __align__(16) ChunkUnit {  // as the list holds it
  int64_t before;   // tiles (and costs) of the units before it, for one key head
  int32_t b, i0;    // sequence, first token
  int32_t row0, n, len, p0;  // as PagedSpan's
};
struct ChunkHead {  // the list's head
  int64_t total, share;    // tiles and costs of all key heads; of a CTA
  int32_t start[kChunkCtas];  // unit in which each share begins
};
// What the merge needs of a unit that is cut at the beginning of a share, and nowhere
// before in it: the share's CTA leaves it (first is -1 where there is none).
struct __align__(16) ChunkCut {
  int32_t first, last;  // shares that have pieces of it
  int32_t h, row0;      // key head, packed row of the sequence's first token
  int32_t i0, n;        // the unit's first token, and the sequence's number of them
  int32_t pad[2];
};

// Where a share's end cuts a unit of `tiles` tiles, `v` tiles behind its first one: not
// within kChunkLeast of its ends, where the piece would cost more than it brings.
__device__ __forceinline__ int chunk_cut(int64_t v, int tiles) {
  return v < min(kChunkLeast, tiles) ? 0 : v > tiles - kChunkLeast ? tiles : static_cast<int>(v);
}
// First float of column c (a multiple of 4) of row r in a partial's O: blocks of 32 rows
// x 32 columns, as the epilogue's staging buffer holds them, 16-byte pieces swapped.
template <int D>
__device__ __forceinline__ int chunk_part_at(int r, int c) {
  return ((r >> 5) * (D / 32) + (c >> 5)) * 1024 + (r & 31) * 32 + ((((c >> 2) & 7) ^ (r & 7)) << 2);
}

struct ChunkParams {
  PagedAttn a;
  const ChunkHead* head;  // null: CTA x takes unit x / H_kv
  const ChunkUnit* units;
  ChunkCut* cuts;         // [CTAs]
  float* o_part;          // [2 * CTAs][256][D]
  float2* ml_part;        // [2 * CTAs][256]
  int tok, rows;          // tokens and rows of a query tile
  uint32_t inv_G;         // ceil(2^16 / G)
  int box_rows, box_log2, missing;  // as TokParams
};

// A unit at hand: two query tiles of sequence b, key head h, tiles j0 .. j0 + n - 1 of
// those that it sees.
struct ChunkAt {
  PagedSpan w;       // (n, len, p0 are the sequence's; the tiles are the unit's)
  int b, h, i0, j0, n;
  bool whole;        // all of the unit's tiles
  // (one read of a list's unit: what the roles wait for where units change)
  __device__ int64_t load(const ChunkParams& p, const ChunkUnit* unit) {
    const int4 x = __ldg(reinterpret_cast<const int4*>(unit)), y = __ldg(reinterpret_cast<const int4*>(unit) + 1);
    b = x.z, i0 = x.w;
    w.row0 = y.x, w.n = y.y, w.len = y.z, w.p0 = y.w;
    tiles(p);
    return static_cast<int64_t>(static_cast<uint64_t>(static_cast<uint32_t>(x.x)) | static_cast<uint64_t>(static_cast<uint32_t>(x.y)) << 32);
  }
  __device__ void load(const ChunkParams& p, int seq, int first) {
    b = seq, i0 = first;
    w = PagedSpan::of<kBN>(p.a, b);
    tiles(p);
  }
  __device__ void tiles(const ChunkParams& p) {
    const int p0 = w.p0 + i0;
    w.visible<kBN>(p.a, p0, p0 + min(kQTiles * p.tok, w.n - i0));
    w.tiles = max(w.tiles, 1);  // (a unit that sees nothing visits one tile, masked)
  }
  // Tiles at hand that query tile t visits: up to its last token's (one at least, to have
  // its zeros).
  __device__ int nkv(const ChunkParams& p, int t) const {
    const int first = i0 + t * p.tok;
    if (first >= w.n) return 1;
    const int hi = max(0, min(w.p0 + min(first + p.tok, w.n), w.len));
    const int count = w.first_tiles + (hi + kBN - 1) / kBN - w.from;
    return min(max(count - j0, 1), n);
  }
};

// A CTA's units: its share of the list, or one.  Each warp has a walk of its own in
// shared memory, which its first lane moves on: held in registers across the MMA warp's
// loop, it took the descriptors' places (512 tokens over 32768 entries: 208 us instead
// of 190).
struct ChunkWalk {
  int64_t first, end;  // where the unit's tiles begin in the list, and the share ends
  int64_t from;        // where the share begins
  int u;
  ChunkAt at;
  bool one;
  // (the whole warp)
  __device__ void start(const ChunkParams& p) {
    if ((threadIdx.x & 31) == 0) init(p);
    __syncwarp();
  }
  __device__ void init(const ChunkParams& p) {
    first = end = from = 0;
    u = 0;
    at.h = -1;
    at.w.tiles = 0;
    one = p.head == nullptr;
    if (one) return;
    const int64_t total = __ldg(&p.head->total), share = __ldg(&p.head->share);
    from = static_cast<int64_t>(blockIdx.x) * share;
    end = min(from + share, total);
    if (from >= end) {
      end = 0;
      return;
    }
    u = __ldg(&p.head->start[blockIdx.x]);
    const int64_t unit = at.load(p, p.units + u) * p.a.s.H_kv;
    const int per = at.w.tiles + kChunkUnitCost;
    const int h = static_cast<int>((from - unit) / per);  // the key head that the share begins in
    at.h = h - 1;
    first = unit + static_cast<int64_t>(h - 1) * per + kChunkUnitCost;
  }
  // The next unit, or false (the whole warp).  own: sequence and first token of the
  // CTA's only one, or -1.
  __device__ bool next(const ChunkParams& p, const volatile int* own) {
    __syncwarp();  // the unit at hand has been read
    int more = 0;
    if ((threadIdx.x & 31) == 0) more = step(p, own);
    more = __shfl_sync(0xffffffffu, more, 0);
    __syncwarp();
    return more != 0;
  }
  __device__ bool step(const ChunkParams& p, const volatile int* own) {
    if (one) {
      if (at.h >= 0 || own[0] < 0) return false;
      at.load(p, own[0], own[1]);
      at.h = static_cast<int>(blockIdx.x) % p.a.s.H_kv;
      at.j0 = 0;
      at.n = at.w.tiles;
      at.whole = true;
      return true;
    }
    while (true) {
      first += at.w.tiles + kChunkUnitCost;
      if (first >= end) return false;  // (also where the share is empty)
      if (++at.h == p.a.s.H_kv) {
        ++u;
        at.load(p, p.units + u);
        at.h = 0;
      }
      at.j0 = chunk_cut(from - first, at.w.tiles);
      at.n = chunk_cut(end - first, at.w.tiles) - at.j0;
      at.whole = at.n == at.w.tiles;
      if (at.n > 0) return true;
    }
  }
};

// This warp's walk: behind the CTA's only unit in the room of the dense kernel's list.
template <int D>
__device__ __forceinline__ ChunkWalk& chunk_walk(const Smem<D, false>& sm) {
  static_assert(64 + (kFwdThreads / 32) * sizeof(ChunkWalk) <= 2 * kListMax, "the walks in the list's room");
  ChunkWalk* const all = reinterpret_cast<ChunkWalk*>(sm.ptr + Cfg<D, false>::kListOff + 64);
  return all[threadIdx.x >> 5];
}

// a / b, rounded up (a 64-bit division is some hundred instructions).
__device__ __forceinline__ int64_t chunk_div_up(int64_t a, int64_t b) {
  const int64_t x = a + b - 1;
  return x < (int64_t{1} << 32) ? static_cast<int64_t>(static_cast<uint32_t>(x) / static_cast<uint32_t>(b)) : x / b;
}

// The list: units in the sequences' order, what lies before each, and in which one
// every share begins.  One block; a warp walks a sequence's units, 32 at a time.
__global__ void __launch_bounds__(kPlanThreads)
    attn_paged_chunk_plan(const __grid_constant__ ChunkParams p, ChunkHead* __restrict__ head, ChunkUnit* __restrict__ units, int cap) {
  __shared__ int64_t tiles_s[kPlanThreads];
  __shared__ int count_s[kPlanThreads];
  __shared__ int64_t warp_tiles[kPlanThreads / 32];
  __shared__ int warp_count[kPlanThreads / 32];
  __shared__ int64_t total_s, end_s;
  const int tid = static_cast<int>(threadIdx.x), lane = tid & 31, warp = tid >> 5;
  const int unit_tok = kQTiles * p.tok;
  grid_dependency_wait();
  grid_launch_dependents();
  int64_t share = 1;
  // round 0 adds everything up, round 1 writes the list; 1024 sequences at a time
  for (int round = p.a.s.B > kPlanThreads ? 0 : 1; round < 2; ++round) {
    int64_t tiles0 = 0;
    int count0 = 0;
    for (int b0 = 0; b0 < p.a.s.B; b0 += kPlanThreads) {
      const int nb = min(kPlanThreads, p.a.s.B - b0);
      for (int i = warp; i < nb; i += kPlanThreads / 32) {
        const PagedSpan w = PagedSpan::of<kBN>(p.a, b0 + i);
        int64_t sum = 0;
        for (int64_t i0 = static_cast<int64_t>(lane) * unit_tok; i0 < w.n; i0 += 32 * static_cast<int64_t>(unit_tok)) {
          PagedSpan v = w;
          v.visible<kBN>(p.a, w.p0 + static_cast<int>(i0), w.p0 + static_cast<int>(min(i0 + unit_tok, static_cast<int64_t>(w.n))));
          sum += max(v.tiles, 1) + kChunkUnitCost;
        }
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
        if (lane == 0) {
          tiles_s[i] = sum;
          count_s[i] = (w.n + unit_tok - 1) / unit_tok;
        }
      }
      __syncthreads();
      // exclusive scans over these sequences
      int64_t t = tid < nb ? tiles_s[tid] : 0;
      int c = tid < nb ? count_s[tid] : 0;
      const int64_t my_t = t;
      const int my_c = c;
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, t, off);
        const int z = __shfl_up_sync(0xffffffffu, c, off);
        if (lane >= off) t += y, c += z;
      }
      if (lane == 31) warp_tiles[warp] = t, warp_count[warp] = c;
      __syncthreads();
      int64_t all_t = 0, add_t = 0;
      int all_c = 0, add_c = 0;
      for (int w = 0; w < kPlanThreads / 32; ++w) {
        if (w == warp) add_t = all_t, add_c = all_c;
        all_t += warp_tiles[w];
        all_c += warp_count[w];
      }
      tiles_s[tid] = tiles0 + add_t + t - my_t;
      count_s[tid] = count0 + add_c + c - my_c;
      if (tid == 0) total_s = tiles0 + all_t;
      __syncthreads();
      if (round == 1) {
        if (p.a.s.B <= kPlanThreads || b0 == 0) {
          // (of all sequences: known after round 0, or these are all)
          const int64_t total = (p.a.s.B <= kPlanThreads ? total_s : head->total / p.a.s.H_kv) * p.a.s.H_kv;
          share = max(static_cast<int64_t>(1), (total + kChunkCtas - 1) / kChunkCtas);
          if (tid == 0) head->total = total, head->share = share;
        }
        for (int i = warp; i < nb; i += kPlanThreads / 32) {
          const int b = b0 + i;
          const PagedSpan w = PagedSpan::of<kBN>(p.a, b);
          int64_t at = tiles_s[i];
          int u = count_s[i] + lane;
          for (int64_t base = 0; base < w.n; base += 32 * static_cast<int64_t>(unit_tok), u += 32) {
            const int64_t i0 = base + static_cast<int64_t>(lane) * unit_tok;
            int64_t mine = 0;
            if (i0 < w.n) {
              PagedSpan v = w;
              v.visible<kBN>(p.a, w.p0 + static_cast<int>(i0), w.p0 + static_cast<int>(min(i0 + unit_tok, static_cast<int64_t>(w.n))));
              mine = max(v.tiles, 1) + kChunkUnitCost;
            }
            int64_t incl = mine;
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
              const int64_t y = __shfl_up_sync(0xffffffffu, incl, off);
              if (lane >= off) incl += y;
            }
            int64_t c_lo = 0, c_hi = 0;  // shares that begin in this lane's unit
            if (mine > 0 && u < cap) {
              const int64_t before = at + incl - mine;
              units[u] = ChunkUnit{before, b, static_cast<int>(i0), w.row0, w.n, w.len, w.p0};
              if (u == cap - 1) end_s = (before + mine) * p.a.s.H_kv;
              c_lo = chunk_div_up(before * p.a.s.H_kv, share);
              c_hi = min(static_cast<int64_t>(kChunkCtas), chunk_div_up((before + mine) * p.a.s.H_kv, share));
            }
            // a unit in which few shares begin is its lane's; the others are the warp's, in turn
            if (c_hi - c_lo <= 4) {
              for (int64_t x = c_lo; x < c_hi; ++x) head->start[x] = u;
            }
            for (unsigned rest = __ballot_sync(0xffffffffu, c_hi - c_lo > 4); rest != 0; rest &= rest - 1) {
              const int from = __ffs(static_cast<int>(rest)) - 1, unit = __shfl_sync(0xffffffffu, u, from);
              const int lo = __shfl_sync(0xffffffffu, static_cast<int>(c_lo), from), hi = __shfl_sync(0xffffffffu, static_cast<int>(c_hi), from);
              for (int x = lo + lane; x < hi; x += 32) head->start[x] = unit;
            }
            at += __shfl_sync(0xffffffffu, incl, 31);
          }
        }
      }
      tiles0 += all_t;
      count0 += all_c;
      __syncthreads();
    }
    if (round == 0) {
      if (tid == 0) head->total = tiles0 * p.a.s.H_kv;
      __threadfence_block();
      __syncthreads();
    } else if (tid == 0 && count0 > cap) {
      head->total = end_s;  // sequences that overlap: as many units as there is room for
    }
  }
}

// TMA producers, as varlen_load_role: warp 0 brings Q and the K tiles (kv 0), warp 2
// the V tiles (kv 1): a tile in pages of 16 rows is 16 copies, and one warp for both took
// 930 cycles a tile where a step of the tensor core, which needs two, takes 2048 (512
// tokens over 32768 entries in pages of 16: 240 us instead of 189).
template <int D>
__device__ void chunk_load_role(const Smem<D, false>& sm, const volatile int* own, int kv, const CUtensorMap* tmQ,
                                const CUtensorMap* map, const ChunkParams& p, const WaitCtx& wc) {
  using C = Cfg<D, false>;
  static_assert(C::kSlots % 2 == 0, "a slot always has K tiles or always V tiles");
  const int lane = static_cast<int>(threadIdx.x) & 31;
  const int boxes = kBN >> p.box_log2;
  const int box = lane & (boxes - 1), panel = lane / boxes;
  const bool mine = panel < C::kPanels;
  const uint32_t dst = panel * kPanelBytes + static_cast<uint32_t>(box << p.box_log2) * 128;
  const int page_mask = (1 << p.a.s.page_log2) - 1;
  int it = kv, k = 0;
  bool ok = true, missing = false;
  const uint64_t pol_first = l2_evict_first();
  ChunkWalk& us = chunk_walk<D>(sm);
  us.start(p);
  while (ok && us.next(p, own)) {
    const ChunkAt un = us.at;  // (here in registers)
    const int p0 = un.w.p0 + un.i0, p1 = un.w.p0 + min(un.i0 + kQTiles * p.tok, un.w.n) - 1;
    const int32_t* const table = p.a.s.table + static_cast<int64_t>(un.b) * p.a.s.max_pages;
    // Whether this lane's box of the unit's tile i is needed, and its entry in the table.
    // That is asked for a tile ahead and looked at only then: an instruction that needs
    // it would hold the warp up for the time that it travels.
    const auto needed = [&](int i) {
      const int key = un.w.tile(i) * kBN + (box << p.box_log2);
      return mine && i < un.j0 + un.n && key < un.w.len && paged_seen(p.a, key, key + p.box_rows, p0, p1);
    };
    const auto entry = [&](int i) {
      const int block = (un.w.tile(i) * kBN + (box << p.box_log2)) >> p.a.s.page_log2;
      return needed(i) ? __ldg(table + block) : -1;
    };
    int pg = entry(un.j0);
    if (kv == 0) {
      if (k > 0) {
        ok = __all_sync(0xffffffffu, mbar_wait(sm.bar_qfree(0), (k - 1) & 1, wc) && mbar_wait(sm.bar_qfree(1), (k - 1) & 1, wc));
        if (!ok) break;
      }
      if (lane == 0) {
        mbar_expect_tx(sm.bar_q(), static_cast<uint32_t>(kQTiles * C::kPanels * p.rows * 128));
        for (int t = 0; t < kQTiles; ++t) {
          const int i0 = un.i0 + t * p.tok < un.w.n ? un.i0 + t * p.tok : un.i0;  // a tile past the end reloads tile 0
          for (int pn = 0; pn < C::kPanels; ++pn)
            tma_load_3d_hint(sm.q(t) + pn * kPanelBytes, tmQ, sm.bar_q(), pn * C::kBoxCols, un.h * p.a.G, un.w.row0 + i0, pol_first);
        }
      }
      __syncwarp();
    }
    ++k;
    for (int i = un.j0; i < un.j0 + un.n; ++i, it += 2) {
      const int next = entry(i + 1);
      const int y = (un.w.tile(i) * kBN + (box << p.box_log2)) & page_mask;
      const int s = it % C::kSlots, round = it / C::kSlots;
      if (round > 0) ok = __all_sync(0xffffffffu, mbar_wait(sm.bar_empty(s), (round - 1) & 1, wc));
      if (!ok) break;
      int z = p.missing;
      if (pg >= 0 && pg < p.a.s.n_pages)
        z = pg * p.a.s.H_kv + un.h;
      else
        missing |= needed(i);
      if (lane == 0) mbar_expect_tx(sm.bar_full(s), C::kTileBytes);
      __syncwarp();
      if (mine) tma_load_3d(sm.slot(s) + dst, map, sm.bar_full(s), panel * C::kBoxCols, y, z);
      pg = next;
    }
  }
  if (missing) atomicOr(&g_attn_status, kPagedNoPage);
  grid_launch_dependents();
  bool drained = kv != 0 || k == 0 || __all_sync(0xffffffffu, mbar_wait_drain(sm.bar_q(), (k - 1) & 1, wc));
  for (int i = it > C::kSlots ? it - C::kSlots : kv; i < it && drained; i += 2)
    drained = __all_sync(0xffffffffu, mbar_wait_drain(sm.bar_full(i % C::kSlots), (i / C::kSlots) & 1, wc));
}

// MMA issuer, as varlen_mma_role.
template <int D, int kType>
__device__ void chunk_mma_role(const Smem<D, false>& sm, const volatile int* own, uint32_t tmem, const ChunkParams& p, const WaitCtx& w) {
  using C = Cfg<D, false>;
  constexpr uint32_t idesc_s = make_idesc(kBM, kBN, false, false, kType == kFP16);
  constexpr uint32_t idesc_pv = make_idesc(kBM, D, false, true, kType == kFP16);
  const uint32_t leader = elect_one();
  const int lane = static_cast<int>(threadIdx.x & 31);
  const uint32_t tS[kQTiles] = {tmem, tmem + kBN};
  const uint32_t tO[kQTiles] = {tmem + C::kOCol0, tmem + C::kOCol0 + D};
  const uint64_t qd[kQTiles] = {sdesc_kmajor_sw128(sm.q(0)), sdesc_kmajor_sw128(sm.q(1))};
  const uint64_t kd0 = sdesc_kmajor_sw128(sm.slot(0));
  const uint64_t vd0 = sdesc_mnmajor_sw128(sm.slot(0), kPanelBytes);
  constexpr uint64_t kSlotStep = C::kTileBytes >> 4;
  int it = 0;
  int k = 0;
  int pc[kQTiles] = {0, 0};
  bool ok = true, issued = false;
  ChunkWalk& us = chunk_walk<D>(sm);
  us.start(p);
  while (ok && us.next(p, own)) {
    const int n = us.at.n;
    const int nkv[kQTiles] = {us.at.nkv(p, 0), us.at.nkv(p, 1)};
    // rows of the last tile at hand that lie behind the sequence
    const int past = min((us.at.w.tile(us.at.j0 + n - 1) + 1) * kBN - us.at.w.len, kBN);
    const int sk0 = it % C::kSlots;
    ok = __all_sync(0xffffffffu, mbar_wait(sm.bar_q(), k & 1, w) &&
                                     mbar_wait(sm.bar_full(sk0), (it / C::kSlots) & 1, w));
    if (!ok) break;
    tc_fence_after();
#pragma unroll
    for (int t = 0; t < kQTiles; ++t) {
      issue_qk<D, false>(leader, tS[t], qd[t], kd0 + sk0 * kSlotStep, idesc_s);
      tc_commit_if(leader, sm.bar_s(t));
      if (nkv[t] == 1) tc_commit_if(leader, sm.bar_qfree(t));
    }
    issued = true;
    tc_commit_if(leader, sm.bar_empty(sk0));
    ++it;
    for (int j = 0; j < n && ok; ++j) {
      const int iv = it, ik = it + 1;
      const int sv = iv % C::kSlots, skn = ik % C::kSlots;
      const bool has_next = j + 1 < n;
      ok = __all_sync(0xffffffffu, mbar_wait(sm.bar_full(sv), (iv / C::kSlots) & 1, w) &&
                                       (!has_next || mbar_wait(sm.bar_full(skn), (ik / C::kSlots) & 1, w)));
      if (ok && !has_next && past > 0) {
        for (int pn = 0; pn < C::kPanels; ++pn) {
          const uint32_t end = sm.slot(sv) + static_cast<uint32_t>((pn + 1) * kPanelBytes);
          for (uint32_t a = end - static_cast<uint32_t>(past * 128 - lane * 16); a < end; a += 32 * 16)
            st_shared_v4_b32(a, 0u, 0u, 0u, 0u);
        }
        fence_async_smem();
        __syncwarp();
      }
#pragma unroll
      for (int t = 0; t < kQTiles; ++t) {
        if (!ok || j >= nkv[t]) continue;
        constexpr int kH = C::kPvSteps / 2;
        ok = __all_sync(0xffffffffu, mbar_wait(sm.bar_phalf(t), pc[t] & 1, w));
        if (ok && j == 0 && k > 0) ok = __all_sync(0xffffffffu, mbar_wait(sm.bar_ofree(t), (k - 1) & 1, w));
        if (!ok) continue;
        tc_fence_after();
        issue_pv<D, false, 0, kH>(leader, tO[t], tS[t], vd0 + sv * kSlotStep, idesc_pv, j > 0);
        ok = __all_sync(0xffffffffu, mbar_wait(sm.bar_p(t), pc[t] & 1, w));
        ++pc[t];
        if (!ok) continue;
        tc_fence_after();
        issue_pv<D, false, kH, C::kPvSteps>(leader, tO[t], tS[t], vd0 + sv * kSlotStep, idesc_pv, true);
        tc_commit_if(leader, sm.bar_o(t));
        if (j + 1 < nkv[t]) {
          issue_qk<D, false>(leader, tS[t], qd[t], kd0 + skn * kSlotStep, idesc_s);
          tc_commit_if(leader, sm.bar_s(t));
          if (j + 2 == nkv[t]) tc_commit_if(leader, sm.bar_qfree(t));
        }
      }
      if (!ok) break;
      tc_commit_if(leader, sm.bar_empty(sv));
      ++it;
      if (has_next) {
        tc_commit_if(leader, sm.bar_empty(skn));
        ++it;
      }
    }
    ++k;
  }
  if (issued) {
    tc_commit_if(leader, sm.bar_drain());
    __all_sync(0xffffffffu, mbar_wait_drain(sm.bar_drain(), 0, w));
  }
}

// Softmax of query tile t, as varlen_softmax_role; what P is held in is its choice, too.
template <int D, int kType>
__device__ void chunk_softmax_role(const Smem<D, false>& sm, const volatile int* own, int t, uint32_t tmem, const ChunkParams& p,
                                   const WaitCtx& w) {
  using C = Cfg<D, false>;
  const int r = static_cast<int>(threadIdx.x) - kBM * (1 + t);
  const int qw = r >> 5;
  const uint32_t lane_off = static_cast<uint32_t>(qw * 32) << 16;
  const uint32_t tS = tmem + lane_off + t * kBN;
  const float c = p.a.scale_log2;
  const int tok = static_cast<int>((static_cast<uint32_t>(r) * p.inv_G) >> 16);
  int cnt = 0;
  int sbase = 0;
  int k = 0;
  bool ok = true;
  ChunkWalk& us = chunk_walk<D>(sm);
  us.start(p);
  while (ok && us.next(p, own)) {
    const int nkv = us.at.nkv(p, t), n_other = us.at.nkv(p, 1 - t);
    const int first = us.at.w.p0 + us.at.i0 + t * p.tok;  // positions of the tile's first and last token, and this row's
    const int last = us.at.w.p0 + min(us.at.i0 + (t + 1) * p.tok, us.at.w.n) - 1, pos = first + tok;
    // Of the tiles at hand, full0 .. full1 - 1 are seen whole by every token here: those of
    // the list's second part from the last token's window on and up to the first token.
    const int shift = us.at.w.first_tiles - us.at.w.from - us.at.j0;  // number at hand of the part's key tile k is k + shift
    const int full0 = max(us.at.w.first_tiles - us.at.j0, (max(0, last - p.a.window + 1) + kBN - 1) / kBN + shift);
    const int full1 = max(0, first + 1) / kBN + shift;
    const int steps = nkv + n_other;
    int step = sbase + t;

    float m_c = -INFINITY;
    float l = 0.f;
    for (int j = 0; j < nkv; ++j) {
      ok = __all_sync(0xffffffffu, mbar_wait(sm.bar_s(t), cnt & 1, w) &&
                                       (!C::kTurn || step == 0 || mbar_wait(sm.bar_turn(), (step - 1) & 1, w)));
      if (!ok) break;
      step += j + t < n_other ? 2 : 1;
      tc_fence_after();
      uint32_t sr[kBN];
      tmem_ld32(tS + 0, sr + 0);
      tmem_ld32(tS + 32, sr + 32);
      tmem_ld32(tS + 64, sr + 64);
      tmem_ld32(tS + 96, sr + 96);
      tmem_wait_ld();
      float s[kBN];
#pragma unroll
      for (int i = 0; i < kBN; ++i) s[i] = __uint_as_float(sr[i]);

      if (j < full0) {
        // keys i < hi of the tile that are at or behind lo, or before sinks
        const int key0 = us.at.w.tile(us.at.j0 + j) * kBN;
        const int hi = pos + 1 - key0, lo = pos - p.a.window + 1 - key0, sinks = p.a.sinks - key0;
#pragma unroll
        for (int i = 0; i < kBN; ++i) s[i] = (i < hi && (i >= lo || i < sinks)) ? s[i] : -INFINITY;
      } else if (j >= full1) {
        const int hi = pos + 1 - us.at.w.tile(us.at.j0 + j) * kBN;
#pragma unroll
        for (int i = 0; i < kBN; ++i) s[i] = i < hi ? s[i] : -INFINITY;
      }
      float mx0 = -INFINITY, mx1 = -INFINITY, mx2 = -INFINITY, mx3 = -INFINITY;
#pragma unroll
      for (int i = 0; i < kBN; i += 8) {
        mx0 = max3f(mx0, s[i], s[i + 1]);
        mx1 = max3f(mx1, s[i + 2], s[i + 3]);
        mx2 = max3f(mx2, s[i + 4], s[i + 5]);
        mx3 = max3f(mx3, s[i + 6], s[i + 7]);
      }
      const float new_mc = max3f(mx0, mx1, fmaxf(mx2, mx3)) * c;
      float alpha = 1.f;
      bool rescale_o = false;
      // (m_c lies kVarlenUp below the reference: what the exponents subtract)
      if (new_mc > m_c + (kVarlenRescale<kType> + kVarlenUp<kType>)) {
        const float to = kType == kFP16 ? new_mc - kVarlenUp<kType> : new_mc;
        alpha = ex2_approx(m_c - to);
        rescale_o = j > 0;
        m_c = to;
      }
      const float mc = (m_c == -INFINITY) ? 0.f : m_c;

      auto rescale_if_needed = [&]() {
        if (!__any_sync(0xffffffffu, rescale_o)) return;
        ok = __all_sync(0xffffffffu, mbar_wait(sm.bar_o(t), (cnt - 1) & 1, w));
        if (!ok) return;
        tc_fence_after();
        const uint32_t tO = tmem + lane_off + C::kOCol0 + t * D;
        const uint64_t a2 = pack_f32x2(alpha, alpha);
#pragma unroll 1
        for (int cc = 0; cc < D; cc += 32) {
          uint32_t o[32];
          tmem_ld32(tO + cc, o);
          tmem_wait_ld();
#pragma unroll
          for (int i = 0; i < 32; i += 2) {
            float x0, x1;
            unpack_f32x2(mul_f32x2(pack_f32x2(__uint_as_float(o[i]), __uint_as_float(o[i + 1])), a2), x0, x1);
            o[i] = __float_as_uint(x0);
            o[i + 1] = __float_as_uint(x1);
          }
          tmem_st32(tO + cc, o);
        }
        tmem_wait_st();
      };

      // P in the inputs' 16-bit type, handed over in two halves of 64 keys
      uint32_t pk[C::kPCols];
      float sum0 = 0.f, sum1 = 0.f;
#pragma unroll
      for (int i = 0; i < kBN / 4; ++i) {
        const float a = ex2_approx(fmaf(s[2 * i], c, -mc));
        const float b = ex2_approx(fmaf(s[2 * i + 1], c, -mc));
        sum0 += a;
        sum1 += b;
        pk[i] = pack_16x2<kType>(a, b);
      }
      tmem_st32(tS, pk);
      if (C::kTurn) mbar_arrive(sm.bar_turn());
      tmem_wait_st();
      rescale_if_needed();
      tc_fence_before();
      mbar_arrive(sm.bar_phalf(t));
#pragma unroll
      for (int i = kBN / 4; i < kBN / 2; ++i) {
        const float a = ex2_approx(fmaf(s[2 * i], c, -mc));
        const float b = ex2_approx(fmaf(s[2 * i + 1], c, -mc));
        sum0 += a;
        sum1 += b;
        pk[i] = pack_16x2<kType>(a, b);
      }
      tmem_st32(tS + 32, pk + 32);
      l = l * alpha + (sum0 + sum1);
      tmem_wait_st();
      tc_fence_before();
      mbar_arrive(sm.bar_p(t));
      ++cnt;
    }
    sbase += steps;
    if (!ok) break;
    if (k > 0) ok = __all_sync(0xffffffffu, mbar_wait(sm.bar_ofree(t), (k - 1) & 1, w));
    if (!ok) break;
    sm.stat(t)[r] = make_float2(m_c, l);
    mbar_arrive(sm.bar_epi(t));
    ++k;
  }
}

// log-sum-exp (natural) from a reference and a sum that carries kVarlenUp.
template <int kType>
__device__ __forceinline__ float chunk_lse(float m, float l) {
  const float l2 = kType == kFP16 ? (m + kVarlenUp<kType>) + log2f(l * 0x1p-11f) : m + log2f(l);
  return l == 0.f ? -INFINITY : l2 * kLn2;
}

// shared -> global copy of contiguous bytes (both sides 16-byte aligned)
__device__ __forceinline__ void bulk_store(void* dst, uint32_t src, uint32_t bytes) {
  asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(dst), "r"(src), "r"(bytes) : "memory");
}

// Epilogue warpgroup, as varlen_epilogue_role; a unit that a share's end cut leaves
// O in fp32, undivided, and (m, l): the staging buffer's 32 columns a turn, as they lie
// there, by one bulk copy.
template <int D, int kType>
__device__ void chunk_epilogue_role(const Smem<D, false>& sm, const volatile int* own, uint32_t tmem, const ChunkParams& p,
                                    const WaitCtx& w) {
  using C = Cfg<D, false>;
  const int qw = static_cast<int>(threadIdx.x >> 5) & 3;
  const int lane = static_cast<int>(threadIdx.x & 31);
  const int rt = qw * 32 + lane;
  const uint32_t lane_off = static_cast<uint32_t>(qw * 32) << 16;
  const uint32_t stage = sm.stage(qw);
  const uint32_t rowa = stage + static_cast<uint32_t>(lane) * 128u;
  const int tok = static_cast<int>((static_cast<uint32_t>(rt) * p.inv_G) >> 16);  // this row's token and head
  int cnt[kQTiles] = {0, 0};
  int k = 0;
  bool ok = true;
  ChunkWalk& us = chunk_walk<D>(sm);
  us.start(p);
  while (ok && us.next(p, own)) {
#pragma unroll
    for (int t = 0; t < kQTiles; ++t) {
      if (!ok) break;
      const int nkv = us.at.nkv(p, t);
      ok = __all_sync(0xffffffffu, mbar_wait_sleepy(sm.bar_epi(t), k & 1, w));
      if (!ok) break;
      const float2 ml = sm.stat(t)[rt];
      ok = __all_sync(0xffffffffu, mbar_wait(sm.bar_o(t), (cnt[t] + nkv - 1) & 1, w));
      cnt[t] += nkv;
      if (!ok) break;
      tc_fence_after();
      const uint32_t tO = tmem + lane_off + C::kOCol0 + t * D;
      // rows of this tile that exist: tokens before the sequence's end
      const int i0 = us.at.i0 + t * p.tok;
      const int rows = min(p.rows, (us.at.w.n - i0) * p.a.G);
      if (us.at.whole) {
        const float inv = ml.y == 0.f ? 0.f : 1.f / ml.y;  // (a row that sees nothing: 0)
        const uint64_t il2 = pack_f32x2(inv, inv);
        const int64_t tok0 = us.at.w.row0 + i0;
#pragma unroll 1
        for (int pn = 0; pn < C::kOPanels; ++pn) {
          __syncwarp();  // the staging panel's last rows have been read
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            uint32_t o[32];
            tmem_ld32(tO + pn * 64 + h * 32, o);
            tmem_wait_ld();
            if (pn == C::kOPanels - 1 && h == 1) {
              tc_fence_before();
              mbar_arrive(sm.bar_ofree(t));
            }
#pragma unroll
            for (int ch = 0; ch < 4; ++ch) {  // 16 bytes: 8 columns
              uint32_t pk[4];
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                float x0, x1;
                unpack_f32x2(mul_f32x2(pack_f32x2(__uint_as_float(o[8 * ch + 2 * i]), __uint_as_float(o[8 * ch + 2 * i + 1])), il2),
                             x0, x1);
                pk[i] = kType == kFP16 ? pack_f16x2_sat(x0, x1) : pack_bf16x2(x0, x1);
              }
              st_shared_v4_b32(rowa + (static_cast<uint32_t>((4 * h + ch) ^ (lane & 7)) << 4), pk[0], pk[1], pk[2], pk[3]);
            }
          }
          __syncwarp();
          // eight lanes a row: 16 bytes each
#pragma unroll 1
          for (int i = 0; i < 8; ++i) {
            const int lr = 4 * i + (lane >> 3), ch = lane & 7;
            const int row = qw * 32 + lr;
            if (row >= rows) continue;
            const int rtok = static_cast<int>((static_cast<uint32_t>(row) * p.inv_G) >> 16);
            uint32_t x[4];
            asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3])
                         : "r"(stage + static_cast<uint32_t>(lr * 128) + (static_cast<uint32_t>(ch ^ (lr & 7)) << 4))
                         : "memory");
            const int64_t at = ((tok0 + rtok) * p.a.s.H_kv + us.at.h) * p.a.G + (row - rtok * p.a.G);
            st_global_v4(p.a.o + at * D + pn * 64 + ch * 8, x[0], x[1], x[2], x[3]);
          }
        }
        if (rt < rows)
          p.a.lse[((tok0 + tok) * p.a.s.H_kv + us.at.h) * p.a.G + (rt - tok * p.a.G)] = chunk_lse<kType>(ml.x, ml.y);
      } else {
        const int64_t part = 2 * static_cast<int64_t>(blockIdx.x) + (us.at.j0 == 0 ? 1 : 0);
        float* const to = p.o_part + part * (kChunkRows * D) + (t * kBM + qw * 32) * D;
#pragma unroll 1
        for (int cc = 0; cc < D; cc += 32) {
          uint32_t o[32];
          tmem_ld32(tO + cc, o);
          tmem_wait_ld();
          if (cc == D - 32) {
            tc_fence_before();
            mbar_arrive(sm.bar_ofree(t));
          }
          if (lane == 0) bulk_wait_read_all();  // the buffer's last block is on its way
          __syncwarp();
#pragma unroll
          for (int ch = 0; ch < 8; ++ch)
            st_shared_v4_b32(rowa + (static_cast<uint32_t>(ch ^ (lane & 7)) << 4), o[4 * ch], o[4 * ch + 1], o[4 * ch + 2], o[4 * ch + 3]);
          fence_async_smem();
          __syncwarp();
          if (lane == 0) {
            bulk_store(to + cc * 32, stage, 32 * 128);
            bulk_commit();
          }
        }
        if (lane == 0) bulk_wait_read_all();
        __syncwarp();
        p.ml_part[part * kChunkRows + t * kBM + rt] = ml;
      }
    }
    ++k;
  }
  if (lane == 0) bulk_wait_all();
  if (p.head != nullptr && qw == 0 && lane == 0) {
    // the CTA's first unit: is this the first cut of it?  (chunk_cut says where cuts are)
    ChunkCut cut{-1, 0, 0, 0, 0, 0, {0, 0}};
    ChunkWalk first;
    first.init(p);
    if (first.step(p, own) && first.at.j0 > 0) {
      const int64_t share = __ldg(&p.head->share);
      const int64_t ca = (first.first + kChunkLeast + share - 1) / share - 1, cb = (first.first + first.at.w.tiles - kChunkLeast) / share;
      if (ca + 1 == static_cast<int64_t>(blockIdx.x))
        cut = ChunkCut{static_cast<int>(ca), static_cast<int>(cb), first.at.h, first.at.w.row0, first.at.i0, first.at.w.n, {0, 0}};
    }
    p.cuts[blockIdx.x] = cut;
  }
}

// The unit of this CTA where there is no list: own[0] its sequence (-1: none), own[1]
// its first token.  One warp.
__device__ __forceinline__ void chunk_own_unit(const ChunkParams& p, volatile int* own) {
  const int lane = static_cast<int>(threadIdx.x & 31);
  const int mine = static_cast<int>(blockIdx.x) / p.a.s.H_kv, unit_tok = kQTiles * p.tok;
  if (lane == 0) own[0] = -1;
  __syncwarp();
  int before = 0;
  for (int s0 = 0; s0 < p.a.s.B; s0 += 32) {
    const int s = s0 + lane;
    const int n = s < p.a.s.B ? min(p.a.s.rows_of(s), p.a.max_new) : 0;
    const int units = (n + unit_tok - 1) / unit_tok;
    int incl = units;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, incl, off);
      if (lane >= off) incl += y;
    }
    const int first = before + incl - units;
    if (first <= mine && mine < first + units) {
      own[0] = s;
      own[1] = (mine - first) * unit_tok;
    }
    before += __shfl_sync(0xffffffffu, incl, 31);
  }
}

template <int D, int kType>
__global__ void __launch_bounds__(kFwdThreads, 1)
    attn_paged_chunk_sm103a(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                            const __grid_constant__ CUtensorMap tmV, const __grid_constant__ ChunkParams p) {
  using C = Cfg<D, false>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* smem = smem_raw + (base - raw);
  const Smem<D, false> sm{base, smem};
  volatile int* const own = reinterpret_cast<volatile int*>(smem + C::kListOff);  // (the dense kernel's unit list lies here)
  volatile uint32_t* misc = reinterpret_cast<volatile uint32_t*>(smem + C::kMiscOff);

  const int warp = static_cast<int>(threadIdx.x >> 5);

  if (threadIdx.x == 0) {
    mbar_init(sm.bar_q(), 1);
    for (int s = 0; s < C::kSlots; ++s) {
      mbar_init(sm.bar_full(s), 1);
      mbar_init(sm.bar_empty(s), 1);
    }
    for (int t = 0; t < kQTiles; ++t) {
      mbar_init(sm.bar_qfree(t), 1);
      mbar_init(sm.bar_s(t), 1);
      mbar_init(sm.bar_p(t), kBM);
      mbar_init(sm.bar_o(t), 1);
      mbar_init(sm.bar_ofree(t), kBM);
      mbar_init(sm.bar_epi(t), kBM);
      mbar_init(sm.bar_phalf(t), kBM);
    }
    mbar_init(sm.bar_drain(), 1);
    mbar_init(sm.bar_turn(), kBM);
    misc[1] = 0u;
    fence_barrier_init();
  } else if (threadIdx.x == 32) {
    tma_prefetch_desc(&tmQ);
    tma_prefetch_desc(&tmK);
    tma_prefetch_desc(&tmV);
  }
  if (warp == 1) {
    tmem_alloc(base + C::kMiscOff, kTmemCols);
    tmem_relinquish();
  }
  // rows of the Q tiles that no token fills (G no divisor of 128): zero for good
  for (int i = p.rows * 8 + static_cast<int>(threadIdx.x); i < 128 * 8; i += kFwdThreads)
    for (int t = 0; t < kQTiles; ++t)
      for (int pn = 0; pn < C::kPanels; ++pn)
        st_shared_v4_b32(sm.q(t) + static_cast<uint32_t>(pn * kPanelBytes + i * 16), 0u, 0u, 0u, 0u);
  fence_async_smem();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = misc[0];
  const WaitCtx w{p.a.timeout_ns, misc + 1};
  grid_dependency_wait();  // the list, and the caller's inputs before it
  if (p.head == nullptr) {
    if (warp == 0) chunk_own_unit(p, own);
    __syncthreads();
  }

  if (warp < 4) {
    regs_set<kRegsRoles>();
    if (warp == 0 || warp == 2) {
      chunk_load_role<D>(sm, own, warp >> 1, &tmQ, warp == 0 ? &tmK : &tmV, p, w);
    } else if (warp == 1) {
      chunk_mma_role<D, kType>(sm, own, tmem, p, w);
    }
  } else if (warp < kEpiWarp0) {
    regs_set<kRegsSoftmax>();
    chunk_softmax_role<D, kType>(sm, own, (warp - 4) >> 2, tmem, p, w);
  } else {
    regs_set<kRegsEpi>();
    chunk_epilogue_role<D, kType>(sm, own, tmem, p, w);
  }
  grid_launch_dependents();

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

// Joins the partials of the units that the shares' ends cut: blocks (c, y) the y-th part
// of the rows of the one across the beginning of share c, if that is the first cut of it.
// A warp takes a row (D = 128) or two, four pieces at a time.
constexpr int kChunkMergeParts = 16;
template <int D, int kType>
__global__ void __launch_bounds__(256) attn_paged_chunk_merge(const __grid_constant__ ChunkParams p) {
  grid_dependency_wait();
  grid_launch_dependents();
  const int4 c0 = __ldg(reinterpret_cast<const int4*>(p.cuts + blockIdx.x)), c1 = __ldg(reinterpret_cast<const int4*>(p.cuts + blockIdx.x) + 1);
  const int ca = c0.x, cb = c0.y, h = c0.z, row0 = c0.w, i0 = c1.x, n = c1.y;
  if (ca < 0) return;
  constexpr int kRows = kChunkRows / kChunkMergeParts, kLanes = D / 4;
  for (int i = static_cast<int>(threadIdx.x); i < kRows * kLanes; i += 256) {
    const int rr = static_cast<int>(blockIdx.y) * kRows + i / kLanes, ch = (i % kLanes) * 4;
    const int t = rr / kBM, r = rr % kBM;
    const int tok = static_cast<int>((static_cast<uint32_t>(r) * p.inv_G) >> 16), token = i0 + t * p.tok + tok;
    if (r >= p.rows || token >= n) continue;
    const int at_o = chunk_part_at<D>(rr, ch);
    float m = -INFINITY, sum = 0.f;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int y0 = ca; y0 <= cb; y0 += 4) {
      float2 s[4];
      float4 o[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        s[e] = make_float2(-INFINITY, 0.f);
        o[e] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (y0 + e <= cb) {
          const int64_t part = 2 * (y0 + e) + (y0 + e == ca ? 1 : 0);
          s[e] = __ldg(p.ml_part + part * kChunkRows + rr);
          o[e] = __ldg(reinterpret_cast<const float4*>(p.o_part + part * (kChunkRows * D) + at_o));
        }
      }
      const float to = fmaxf(fmaxf(fmaxf(s[0].x, s[1].x), fmaxf(s[2].x, s[3].x)), m);
      const float keep = m == -INFINITY ? 1.f : ex2_approx(m - to);  // (without a reference there is nothing, or NaN)
      m = to;
      sum *= keep, v.x *= keep, v.y *= keep, v.z *= keep, v.w *= keep;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if (s[e].x == -INFINITY && s[e].y == 0.f) continue;  // it saw none of these keys
        const float f = s[e].x == -INFINITY ? 1.f : ex2_approx(s[e].x - m);
        sum = fmaf(s[e].y, f, sum);
        v.x = fmaf(o[e].x, f, v.x), v.y = fmaf(o[e].y, f, v.y), v.z = fmaf(o[e].z, f, v.z), v.w = fmaf(o[e].w, f, v.w);
      }
    }
    const int64_t at = (static_cast<int64_t>(row0 + token) * p.a.s.H_kv + h) * p.a.G + (r - tok * p.a.G);
    tok_write<kType>(p.a, at * D + ch, at, v, m, sum, ch == 0);
  }
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------

// Units that a call may have, and whether each CTA takes one.
struct ChunkPlan {
  int tok;
  int64_t cap;
  bool direct;
};
constexpr int kChunkDirectLen = 2048;  // keys up to which a CTA a unit is one launch instead of three
ChunkPlan chunk_plan(int B, int H_kv, int G, int64_t rows, int max_new, int max_len, int window, int sinks) {
  ChunkPlan c;
  c.tok = kBM / G;
  c.cap = rows / (kQTiles * c.tok) + std::min<int64_t>(B, rows);
  const int64_t keys = window > 0 ? std::min<int64_t>(max_len, static_cast<int64_t>(window) + sinks + max_new) : max_len;
  c.direct = c.cap * H_kv <= kChunkCtas && keys <= kChunkDirectLen;
  return c;
}
constexpr uint64_t kChunkHeadBytes = (sizeof(ChunkHead) + 255) / 256 * 256;
uint64_t chunk_list_bytes(const ChunkPlan& c) { return kChunkHeadBytes + (static_cast<uint64_t>(c.cap) * sizeof(ChunkUnit) + 255) / 256 * 256; }
uint64_t chunk_workspace(const ChunkPlan& c, int D) {
  return c.direct ? 16
                  : chunk_list_bytes(c) + static_cast<uint64_t>(2 * kChunkCtas) * kChunkRows * (D * sizeof(float) + sizeof(float2)) +
                        kChunkCtas * sizeof(ChunkCut);
}

template <int D, int kType>
bool chunk_limits() {
  return cudaFuncSetAttribute(reinterpret_cast<const void*>(attn_paged_chunk_sm103a<D, kType>),
                              cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg<D, false>::kSmemBytes) == cudaSuccess;
}

template <int D, int kType>
cudaError_t chunk_launch(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv, const ChunkParams& p, const ChunkPlan& c,
                         void* workspace, cudaStream_t s) {
  if (!c.direct) {
    const cudaError_t e =
        launch_pdl(attn_paged_chunk_plan, dim3(1), dim3(kPlanThreads), 0, s, p, static_cast<ChunkHead*>(workspace),
                   reinterpret_cast<ChunkUnit*>(static_cast<char*>(workspace) + kChunkHeadBytes), static_cast<int>(c.cap));
    if (e != cudaSuccess) return e;
  }
  const unsigned grid = c.direct ? static_cast<unsigned>(c.cap * p.a.s.H_kv) : kChunkCtas;
  const cudaError_t e = launch_pdl(attn_paged_chunk_sm103a<D, kType>, dim3(grid), dim3(kFwdThreads), Cfg<D, false>::kSmemBytes, s, tq,
                                   tk, tv, p);
  if (e != cudaSuccess || c.direct) return e;
  return launch_pdl(attn_paged_chunk_merge<D, kType>, dim3(kChunkCtas, kChunkMergeParts), dim3(256), 0, s, p);
}

attn_status_t chunk_run(const attn_pages_t* cache, const PagedAttn& a, const ChunkPlan& c, void* workspace, cudaStream_t s) {
  const int box = std::min(cache->page, kBN), H_q = cache->H_kv * a.G, D = cache->D;
  CUtensorMap tq, tk, tv;
  if (!encode_rows(&tq, a.q, D, H_q, a.s.rows, a.q_stride, a.G, c.tok, cache->dtype) || !encode_pages(&tk, cache->k_pages, cache, box) ||
      !encode_pages(&tv, cache->v_pages, cache, box))
    return ATTN_ERR_LAUNCH;
  ChunkParams p;
  p.a = a;
  p.head = c.direct ? nullptr : static_cast<const ChunkHead*>(workspace);
  p.units = c.direct ? nullptr : reinterpret_cast<const ChunkUnit*>(static_cast<char*>(workspace) + kChunkHeadBytes);
  p.o_part = c.direct ? nullptr : reinterpret_cast<float*>(static_cast<char*>(workspace) + chunk_list_bytes(c));
  p.ml_part = c.direct ? nullptr : reinterpret_cast<float2*>(p.o_part + static_cast<int64_t>(2 * kChunkCtas) * kChunkRows * D);
  p.cuts = c.direct ? nullptr : reinterpret_cast<ChunkCut*>(p.ml_part + static_cast<int64_t>(2 * kChunkCtas) * kChunkRows);
  p.tok = c.tok;
  p.rows = c.tok * a.G;
  p.inv_G = static_cast<uint32_t>((65536 + a.G - 1) / a.G);
  p.box_rows = box;
  p.box_log2 = 0;
  while ((1 << p.box_log2) < box) ++p.box_log2;
  p.missing = cache->n_pages * cache->H_kv;
  const bool bf = cache->dtype == ATTN_BF16;
  const cudaError_t e = D == 64 ? (bf ? chunk_launch<64, kBF16>(tq, tk, tv, p, c, workspace, s)
                                      : chunk_launch<64, kFP16>(tq, tk, tv, p, c, workspace, s))
                                : (bf ? chunk_launch<128, kBF16>(tq, tk, tv, p, c, workspace, s)
                                      : chunk_launch<128, kFP16>(tq, tk, tv, p, c, workspace, s));
  return e == cudaSuccess ? ATTN_OK : ATTN_ERR_LAUNCH;
}

}  // namespace

extern "C" {

uint64_t attn_paged_attend_workspace_bytes(int B, int H_q, int H_kv, int D, int64_t rows, int max_new, int max_len, int window,
                                           int sinks) {
  if (B < 1 || H_kv < 1 || H_q < H_kv || H_q % H_kv != 0 || H_q / H_kv > kBM || (D != 64 && D != 128) || rows < 0 || max_new < 0 ||
      max_len < 0 || window < 0 || sinks < 0)
    return 0;
  const int G = H_q / H_kv;
  max_new = static_cast<int>(std::min<int64_t>(max_new, rows));
  if (paged_is_token(max_new, G)) return tok_workspace(tok_plan(B, H_kv, G, max_new, max_len, window, sinks), D);
  return chunk_workspace(chunk_plan(B, H_kv, G, rows, max_new, max_len, window, sinks), D);
}

attn_status_t attn_paged_attend(const attn_pages_t* cache, const void* q, int64_t q_stride, void* o, float* lse, int64_t rows,
                                const int32_t* seq_start, int H_q, float scale, int window, int sinks, int max_new, int max_len,
                                void* workspace, uint64_t workspace_bytes, void* stream) {
  attn_status_t st = check_pages(cache);
  if (st != ATTN_OK) return st;
  const int D = cache->D, H_kv = cache->H_kv, B = cache->B;
  if (rows < 0 || H_q < H_kv || H_q % H_kv != 0 || (seq_start == nullptr && rows != B)) return ATTN_ERR_INVALID_ARG;
  if (rows > 0 && (q == nullptr || o == nullptr || lse == nullptr)) return ATTN_ERR_INVALID_ARG;
  if (!std::isfinite(scale) || !(scale > 0.f) || window < 0 || sinks < 0 || max_new < 0 || max_len < 0 ||
      max_len > static_cast<int64_t>(cache->max_pages) * cache->page)
    return ATTN_ERR_INVALID_ARG;
  if (H_q / H_kv > kBM || rows > INT_MAX / 2 || q_stride > (int64_t{1} << 40)) return ATTN_ERR_UNSUPPORTED;
  if (q_stride < static_cast<int64_t>(H_q) * D) return ATTN_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(o, 16) || !aligned(lse, 4) || !aligned(seq_start, 4) || !aligned(workspace, 16) || q_stride % 8 != 0)
    return ATTN_ERR_ALIGNMENT;
  const int G = H_q / H_kv;
  max_new = static_cast<int>(std::min<int64_t>(max_new, rows));
  const uint64_t need = attn_paged_attend_workspace_bytes(B, H_q, H_kv, D, rows, max_new, max_len, window, sinks);
  if (rows > 0 && need > 16 && (workspace == nullptr || workspace_bytes < need)) return ATTN_ERR_INVALID_ARG;
  if (rows == 0 || max_new == 0) return ATTN_OK;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return ATTN_ERR_DEVICE;
  st = prepare_device(dev);
  if (st != ATTN_OK) return st;
  if (g_paged_state[dev].load(std::memory_order_acquire) == 0) {
    if (!tok_limits<64, kBF16>() || !tok_limits<64, kFP16>() || !tok_limits<128, kBF16>() || !tok_limits<128, kFP16>() ||
        !chunk_limits<64, kBF16>() || !chunk_limits<64, kFP16>() || !chunk_limits<128, kBF16>() || !chunk_limits<128, kFP16>())
      return ATTN_ERR_DEVICE;
    g_paged_state[dev].store(1, std::memory_order_release);
  }
  if (!get_encoder()) return ATTN_ERR_DEVICE;
  PagedAttn a;
  a.s = paged_seqs(cache, seq_start, rows);
  a.q = static_cast<const uint16_t*>(q);
  a.o = static_cast<uint16_t*>(o);
  a.lse = lse;
  a.q_stride = q_stride;
  a.G = G;
  // beyond what positions reach, a window and a number of sinks say nothing more
  a.window = window > 0 ? std::min(window, INT_MAX / 2) : INT_MAX / 2;
  a.sinks = window > 0 ? std::min(sinks, INT_MAX / 2) : 0;
  a.most = max_len;
  a.max_new = max_new;
  a.scale_log2 = static_cast<float>(static_cast<double>(scale) * 1.4426950408889634074);
  a.timeout_ns = kDefaultTimeoutNs;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (paged_is_token(max_new, G)) return tok_run(cache, a, tok_plan(B, H_kv, G, max_new, max_len, window, sinks), workspace, s);
  const ChunkPlan c = chunk_plan(B, H_kv, G, rows, max_new, max_len, window, sinks);
  if (c.cap * H_kv > INT_MAX / 2) return ATTN_ERR_UNSUPPORTED;
  return chunk_run(cache, a, c, workspace, s);
}

}  // extern "C"
