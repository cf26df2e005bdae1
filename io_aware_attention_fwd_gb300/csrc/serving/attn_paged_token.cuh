// Attention of few query rows per sequence over the pages: one new token each, or
// as many as fit 16 rows of (token, query head) a key head.  Part of attn_fwd.cu.
//
// Every key and value row is read once and meets at most 16 query rows, so the
// pass is bound by HBM: 4 D bytes a key and key head.  What the kernel is built
// around is therefore bytes in flight and nothing that stops them:
//
//   * One CTA an SM.  Two producer warps bring tiles of 64 keys (K and V, 32 KB at
//     D = 128) into a ring of 192 KB with TMA, page by page, and never stop at the
//     end of a sequence or head: the next one's tiles are on their way while the
//     last one's results are joined.  (In pages of 16 rows a tile is 16 copies; one
//     warp for all of them held the pass up: 64 sequences of up to 16000 entries took
//     360 us instead of 328.)
//   * Eight consumer warps: four take 16 keys each of one tile, four of the next.
//     S^T = K Q^T and O^T += V^T P^T on mma.sync m16n8k16, keys and channels as the
//     M rows, 8 query rows a tile of N; ldmatrix reads both from the 128-byte
//     swizzle.  (With so few rows a product of the tensor core's own
//     width would be nine tenths padding; the pipe is idle most of the time as it is.)
//   * P enters P V as the sum of two 16-bit numbers, which leaves 16 (bf16) or 22
//     bits of it: the products are there for the taking, and O is as exact as from
//     fp32 products.
//   * Work split.  The visible tiles of all (sequence, key head) form one list, cut
//     into equal shares, one a CTA, whatever the lengths; each of its rows counts
//     kTokRowCost tiles more for its start and end.  A row within a share is
//     written at once; of a row that was cut, each share leaves a partial (m, l, O),
//     and a second kernel joins them.  Few short rows have a CTA each instead:
//     one launch.
//   * With a window the list holds the tiles of the first `sinks` keys and those
//     from the first new token's window on; no other page is looked at.
//
// 64 sequences of up to 16000 entries, 64/8 heads, D = 128: 311 us, 6.85 TB/s.  One of
// 131072, 32/8: 84 us, 6.4 TB/s (80 in the attention, then the merge).  32 windows of
// 4096 in pages of 16: 87 to 91 us, 5.8 TB/s: each CTA has one to three rows to start and end.
// One of 701, 16/16, D = 64: 6.8 us on the GPU.

namespace {

constexpr int kTokTile = 64;       // keys a tile
constexpr int kTokWarps = 8;       // consumers
constexpr int kTokThreads = 32 * (kTokWarps + 2);  // and a producer each for K and V
constexpr int kTokRowCost = 4;     // tiles that a row's start and end count as

// What a call gives its tokens.
struct PagedAttn {
  PagedSeqs s;
  const uint16_t* q;
  uint16_t* o;
  float* lse;
  int64_t q_stride;
  int G;               // query heads per key head
  int window, sinks;   // window: INT_MAX / 2 for none
  int most, max_new;   // bounds on lengths and new tokens
  float scale_log2;
  unsigned long long timeout_ns;
};

// A sequence's new tokens and the tiles of `kTile` keys that some of them see: the
// first `first_tiles`, then those from `from` on.
struct PagedSpan {
  int row0, n;   // packed row of its first new token; tokens that are looked at
  int len, p0;   // entries; position of the first new token (below 0: it sees nothing)
  int first_tiles, from, tiles;
  template <int kTile>
  __device__ static PagedSpan of(const PagedAttn& p, int b) {
    PagedSpan w;
    w.row0 = p.s.seq_start != nullptr ? p.s.start(b) : b;
    const int all = p.s.rows_of(b);
    w.n = min(all, p.max_new);
    w.len = min(p.s.held(b), p.most);
    w.p0 = w.len - all;
    w.visible<kTile>(p, w.p0, w.p0 + w.n);
    return w;
  }
  // The tiles that tokens at positions p0 .. end - 1 see.
  template <int kTile>
  __device__ void visible(const PagedAttn& p, int p0, int end) {
    const int hi = max(0, min(end, len)), lo = max(0, p0 - p.window + 1);
    from = min(lo, hi) / kTile;
    first_tiles = min((min(p.sinks, hi) + kTile - 1) / kTile, from);
    tiles = hi > 0 && n > 0 ? first_tiles + (hi + kTile - 1) / kTile - from : 0;
  }
  __device__ int tile(int i) const { return i < first_tiles ? i : from + (i - first_tiles); }
};

// Whether some token at p0 .. p1 sees some key of k0 .. k1 - 1.
__device__ __forceinline__ bool paged_seen(const PagedAttn& p, int k0, int k1, int p0, int p1) {
  return k0 <= p1 && (k1 - 1 > p0 - p.window || k0 < p.sinks);
}
// Whether every token sees all of them.
__device__ __forceinline__ bool paged_all_seen(const PagedAttn& p, int k0, int k1, int p0, int p1) {
  return k1 - 1 <= p0 && (k0 > p1 - p.window || k1 <= p.sinks);
}

// kNT: tiles of 8 query rows, which hold a sequence's (token, query head) rows of a key
// head.  With one, the two groups of four consumer warps
// take tiles of keys in turn; with two, each takes every tile for 8 of the rows: 16 rows a
// warp spilt and kept half the pace (64 sequences of up to 16000 entries with 16 query
// heads a key head: 358 us instead of 323).
template <int D, int kNT>
struct TokCfg {
  static constexpr int kRows = 8 * kNT;                    // query rows
  static constexpr bool kSplit = kNT == 2;
  static constexpr int kUsers = kSplit ? 8 : 4;            // warps that use a stage
  static constexpr int kJoin = kSplit ? 4 : 8;             // warps that have keys of a row
  static constexpr int kPanels = D / 64;                   // 128-byte panels of a row
  static constexpr int kPanel = kTokTile * 128;            // bytes of one
  static constexpr int kV = kPanels * kPanel;              // V of a stage
  static constexpr int kStage = 2 * kV;
  // 6 (D = 128) or 12.  Even, so that where the groups take turns a stage is always the
  // same four warps': a warp that did not see every phase of a barrier could take one for
  // the next but one.
  static constexpr int kStages = (192 * 1024) / kStage;
  static_assert(kStages % 2 == 0, "a stage belongs to one group of warps");
  static constexpr int kOStride = D + 4;                   // floats; 4: lanes' banks differ
  static constexpr int kSlots = kNT == 1 ? 4 : 2;          // places for warps' O as they are added up
  static constexpr int kO = kStages * kStage;              // float [kSlots][kRows][kOStride]
  static constexpr int kMl = kO + kSlots * kRows * kOStride * 4;  // float2 [2][kTokWarps][8]
  static constexpr int kBar = kMl + 2 * kTokWarps * 8 * 8;
  static constexpr int kMisc = kBar + 2 * kStages * 8;     // abort flag; int64 sums of the block's scan
  static constexpr int kBytes = kMisc + 16 + 8 * (kTokThreads / 32 + 4) + 1024;
  static_assert(kBytes <= 232448, "shared memory per CTA");
};

// What the merge needs of a row that is cut at the beginning of a share, and nowhere
// before in it: the share's CTA leaves it (first is -1 where there is none).
struct __align__(16) TokCut {
  int32_t first, last;   // shares that have pieces of it
  int32_t h, row0;       // key head, packed row of the sequence's first token
  int32_t rows;          // query rows
  int32_t pad[3];
};

struct TokParams {
  PagedAttn a;
  TokCut* cuts;     // [CTAs]
  float* o_part;    // [2 * CTAs][kRows][D]
  float2* ml_part;  // [2 * CTAs][kRows]
  int box_rows, box_log2;  // rows of a TMA box: the page's, at most a tile's
  int missing;      // third coordinate behind the pages: reads zeros
};

__device__ __forceinline__ int64_t tok_units(const PagedAttn& p, int b) {
  const PagedSpan w = PagedSpan::of<kTokTile>(p, b);
  return w.n > 0 ? static_cast<int64_t>(w.tiles + kTokRowCost) * p.s.H_kv : 0;
}

// Units of all sequences, and those before this thread's (contiguous) ones; sums: a
// block's scratch of warps + 1 words.  The whole block calls it.
template <int kThreads>
__device__ int64_t tok_total(const PagedAttn& p, volatile int64_t* sums, int64_t* before) {
  const int tid = static_cast<int>(threadIdx.x), lane = tid & 31;
  const int per = (p.s.B + kThreads - 1) / kThreads;
  int64_t mine = 0;
  for (int i = 0; i < per; ++i) {
    const int b = tid * per + i;
    if (b < p.s.B) mine += tok_units(p, b);
  }
  int64_t incl = mine;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, incl, off);
    if (lane >= off) incl += y;
  }
  if (lane == 31) sums[tid >> 5] = incl;
  __syncthreads();
  int64_t total = 0, first = 0;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) {
    if (w == (tid >> 5)) first = total;
    total += sums[w];
  }
  *before = first + incl - mine;
  return total;
}
// The sequence in whose units x lies, and the units before it, by the thread that has it.
template <int kThreads>
__device__ void tok_find(const PagedAttn& p, int64_t x, int64_t before, volatile int* b_out, volatile int64_t* before_out) {
  const int per = (p.s.B + kThreads - 1) / kThreads;
  if (x < before) return;
  for (int i = 0; i < per; ++i) {
    const int b = static_cast<int>(threadIdx.x) * per + i;
    if (b >= p.s.B) return;
    const int64_t u = tok_units(p, b);
    if (x < before + u) {
      *b_out = b;
      *before_out = before;
      return;
    }
    before += u;
  }
}

// A CTA's share, row by row.
struct TokWalk {
  int64_t x, end, before, share;
  int b, heads, per_row;  // sequence; its rows (none without tokens), and what each counts
  PagedSpan w;
  int h, t0, t1;  // key head, tiles of the list
  int64_t at;     // place of the row's first tile in the list
  __device__ void load(const PagedAttn& p) {
    w = PagedSpan::of<kTokTile>(p, b);
    heads = w.n > 0 ? p.s.H_kv : 0;
    per_row = w.tiles + kTokRowCost;
  }
  __device__ bool next(const PagedAttn& p) {
    while (x < end) {
      const int64_t row = (x - before) / per_row;
      if (row >= heads) {
        before += static_cast<int64_t>(per_row) * heads;
        if (++b >= p.s.B) return false;
        load(p);
        continue;
      }
      const int64_t x0 = before + row * per_row;
      h = static_cast<int>(row);
      const bool starts = x == x0;
      t0 = static_cast<int>(max(static_cast<int64_t>(0), x - x0 - kTokRowCost));
      t1 = static_cast<int>(max(static_cast<int64_t>(0), min(static_cast<int64_t>(w.tiles), end - x0 - kTokRowCost)));
      x = x0 + per_row;
      at = x0 + kTokRowCost;
      if (t0 < t1 || (w.tiles == 0 && starts)) return true;
    }
    return false;
  }
};

// Sets this CTA's walk up; false: there is nothing for it.  kDirect: row blockIdx.x.
template <int kThreads, bool kDirect>
__device__ __forceinline__ bool tok_start(TokWalk& k, const TokParams& p, volatile int64_t* sums) {
  if constexpr (kDirect) {
    k.b = static_cast<int>(blockIdx.x) / p.a.s.H_kv;
    k.load(p.a);
    k.h = static_cast<int>(blockIdx.x) - k.b * p.a.s.H_kv;
    k.t0 = 0, k.t1 = k.w.tiles;
    return k.h < k.heads;
  } else {
    int64_t before;
    const int64_t total = tok_total<kThreads>(p.a, sums, &before);
    const int64_t share = (total + gridDim.x - 1) / gridDim.x;
    k.share = share;
    k.x = static_cast<int64_t>(blockIdx.x) * share;
    k.end = k.x + share < total ? k.x + share : total;
    if (threadIdx.x == 0) p.cuts[blockIdx.x].first = -1;  // (the first row writes it again, behind a barrier)
    volatile int* const b_s = reinterpret_cast<volatile int*>(sums + kThreads / 32 + 1);
    if (k.x < k.end) tok_find<kThreads>(p.a, k.x, before, b_s, sums + kThreads / 32);
    __syncthreads();
    if (k.x >= k.end) return false;
    k.b = *b_s;
    k.before = sums[kThreads / 32];
    k.load(p.a);
    return true;
  }
}

template <int kType>
__device__ __forceinline__ void tok_mma(float* d, const uint32_t* a, uint32_t b0, uint32_t b1) {
  if constexpr (kType == kFP16) {
    mma_16816(d, a[0], a[1], a[2], a[3], b0, b1);
  } else {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  }
}

__device__ __forceinline__ void tok_join_sync() { asm volatile("bar.sync 1, %0;" ::"n"(kTokWarps * 32) : "memory"); }

// What P is held times, and how far a score may exceed its row's reference before
// that moves, in log2: bf16 has fp32's range; fp16 ends at 2^16 and below 2^-14 its
// bits go, so there p is 2^11 times as large and the reference moves at 2^4.
template <int kType>
constexpr float kTokUp = kType == kFP16 ? 11.f : 0.f;
template <int kType>
constexpr float kTokMove = kType == kFP16 ? 4.f : kRescaleLog2;

// Four channels of a row's O, and its LSE, from the joined sums.
template <int kType>
__device__ __forceinline__ void tok_write(const PagedAttn& p, int64_t at, int64_t row, const float4& v, float m, float sum, bool lse) {
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  // (a mean of fp16 values is one, but may be rounded up past the largest)
  const uint32_t lo = kType == kFP16 ? pack_f16x2_sat(v.x * inv, v.y * inv) : pack_bf16x2(v.x * inv, v.y * inv);
  const uint32_t hi = kType == kFP16 ? pack_f16x2_sat(v.z * inv, v.w * inv) : pack_bf16x2(v.z * inv, v.w * inv);
  *reinterpret_cast<uint2*>(p.o + at) = make_uint2(lo, hi);
  if (lse) {
    // (the factor comes off the sum first: a sum near 1 has the more exact logarithm)
    const float l2 = kType == kFP16 ? (m + kTokUp<kType>) + log2f(sum * 0x1p-11f) : m + log2f(sum);
    p.lse[row] = sum == 0.f ? -INFINITY : l2 * kLn2;
  }
}

// Producer warp of K (kv 0) or V (1).
template <int D, int kNT, bool kDirect>
__device__ void tok_load(TokWalk k, const TokParams& p, int kv, const CUtensorMap* map, uint32_t base, const WaitCtx& wc) {
  using C = TokCfg<D, kNT>;
  const int lane = static_cast<int>(threadIdx.x) & 31;
  const int boxes = kTokTile >> p.box_log2;
  const int box = lane & (boxes - 1), panel = lane / boxes;
  const bool mine = panel < C::kPanels;
  const uint32_t dst0 = base + kv * C::kV + panel * C::kPanel + (box << p.box_log2) * 128;
  const int page_mask = (1 << p.a.s.page_log2) - 1;
  int it = 0;
  bool ok = true, missing = false;
  bool more = kDirect ? true : k.next(p.a);
  while (more && ok) {
    const int p1 = k.w.p0 + k.w.n - 1;
    // Whether this lane's box of the list's tile i is needed, and its entry in the table.
    // That is asked for two tiles ahead and looked at only then: an instruction that
    // needs it would hold the warp up for the time that it travels.
    const auto needed = [&](int i) {
      const int key = k.w.tile(i) * kTokTile + (box << p.box_log2);
      return mine && i < k.t1 && key < k.w.len && paged_seen(p.a, key, key + p.box_rows, k.w.p0, p1);
    };
    const auto entry = [&](int i) {
      const int block = (k.w.tile(i) * kTokTile + (box << p.box_log2)) >> p.a.s.page_log2;
      return needed(i) ? __ldg(p.a.s.table + static_cast<int64_t>(k.b) * p.a.s.max_pages + block) : -1;
    };
    int pg = entry(k.t0), pg1 = entry(k.t0 + 1);
    for (int i = k.t0; i < k.t1 && ok; ++i, ++it) {
      const int pg2 = entry(i + 2);
      const int s = it % C::kStages;
      const uint32_t full = base + C::kBar + 8 * s;
      if (it >= C::kStages)
        ok = __all_sync(0xffffffffu, mbar_wait(full + 8 * C::kStages, (it / C::kStages - 1) & 1, wc));
      if (!ok) break;
      const int y = (k.w.tile(i) * kTokTile + (box << p.box_log2)) & page_mask;
      int z = p.missing;
      if (pg >= 0 && pg < p.a.s.n_pages)
        z = pg * p.a.s.H_kv + k.h;
      else
        missing |= needed(i);
      if (lane == 0) mbar_expect_tx(full, C::kStage / 2);
      __syncwarp();
      if (mine) tma_load_3d(dst0 + s * C::kStage, map, full, panel * 64, y, z);
      pg = pg1, pg1 = pg2;
    }
    more = kDirect ? false : k.next(p.a);
  }
  if (missing) atomicOr(&g_attn_status, kPagedNoPage);
  // what is in flight lands before the CTA leaves
  bool drained = true;
  for (int i = it > C::kStages ? it - C::kStages : 0; i < it && drained; ++i)
    drained = __all_sync(0xffffffffu, mbar_wait_drain(base + C::kBar + 8 * (i % C::kStages), (i / C::kStages) & 1, wc));
}

// Consumer warp `warp`.
template <int D, int kType, int kNT, bool kDirect>
__device__ void tok_compute(TokWalk k, const TokParams& p, uint32_t base, uint8_t* smem, int warp, const WaitCtx& wc) {
  using C = TokCfg<D, kNT>;
  constexpr int kSteps = D / 16;
  const int lane = static_cast<int>(threadIdx.x) & 31, r = lane >> 2, c = lane & 3;
  const int group = warp >> 2, key_w = (warp & 3) * 16;
  // ldmatrix addresses in a stage: K rows 0-15 by 16-byte pieces 0 and 1; V rows 0-7 and 8-15, transposed
  const int krow = key_w + (lane & 15), vrow = key_w + (lane & 7) + ((lane >> 4) << 3);
  const uint32_t kaddr = base + krow * 128, vaddr = base + C::kV + vrow * 128;
  const int kpiece = lane >> 4, vpiece = (lane >> 3) & 1;
  float* const o_s = reinterpret_cast<float*>(smem + C::kO);
  float2* const ml_s = reinterpret_cast<float2*>(smem + C::kMl);
  const int r0 = C::kSplit ? group * 8 : 0;  // this warp's query rows
  int it = 0, seg = 0;
  bool ok = true;
  const float cl = p.a.scale_log2;
  bool more = kDirect ? true : k.next(p.a);
  while (more) {
    const PagedSpan& w = k.w;
    const int rows = w.n * p.a.G;  // (at most kRows)
    // Q as B operands, and the positions of this lane's columns.  (Coherent loads, not the
    // read-only path's: the append before may have written Q since this kernel began.  They
    // may stay in the SM's cache, where the other warps find them: past it, one sequence of
    // 131072 entries took 88.7 us instead of 84.2.)
    uint32_t q[kSteps][2];
    int pos[2];
    {
      const int mine = min(r0 + r, rows - 1), tok = mine / p.a.G, g = mine - tok * p.a.G;
      const uint16_t* src = p.a.q + (w.row0 + tok) * p.a.q_stride + (k.h * p.a.G + g) * static_cast<int64_t>(D) + 2 * c;
#pragma unroll
      for (int ks = 0; ks < kSteps; ++ks)
#pragma unroll
        for (int i = 0; i < 2; ++i)
          q[ks][i] = r0 + r < rows ? __ldca(reinterpret_cast<const uint32_t*>(src + ks * 16 + i * 8)) : 0u;
#pragma unroll
      for (int e = 0; e < 2; ++e) pos[e] = w.p0 + min(r0 + 2 * c + e, rows - 1) / p.a.G;
    }
    const int p_first = w.p0, p_last = w.p0 + w.n - 1;
    float ref[2], sub[2], l[2], o[kSteps][4];
#pragma unroll
    for (int e = 0; e < 2; ++e) ref[e] = -INFINITY, sub[e] = l[e] = 0.f;
#pragma unroll
    for (int mb = 0; mb < kSteps; ++mb)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[mb][e] = 0.f;
    for (int i = k.t0; i < k.t1; ++i, ++it) {
      if (!C::kSplit && (it & 1) != group) continue;
      const int s = it % C::kStages;
      const uint32_t full = base + C::kBar + 8 * s, stage = static_cast<uint32_t>(s) * C::kStage;
      ok = ok && __all_sync(0xffffffffu, mbar_wait(full, (it / C::kStages) & 1, wc));
      if (!ok) continue;  // (the barriers below still have all warps)
      const int key0 = w.tile(i) * kTokTile + key_w;
      float d[4], d2[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) d[e] = d2[e] = 0.f;
#pragma unroll
      for (int ks = 0; ks < kSteps; ++ks) {
        uint32_t a[4];
        ldmatrix_x4(a, kaddr + stage + (ks >> 2) * C::kPanel + ((((ks & 3) * 2 + kpiece) ^ (krow & 7)) << 4));
        tok_mma<kType>((ks & 1) ? d2 : d, a, q[ks][0], q[ks][1]);
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) d[e] += d2[e];
      if (!paged_all_seen(p.a, key0, key0 + 16, p_first, p_last)) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int j = key0 + r + (e >> 1) * 8, at = pos[e & 1];
          if (!(j <= at && (j > at - p.a.window || j < p.a.sinks))) d[e] = -INFINITY;
        }
        // rows behind the sequence's end hold anything, and 0 * NaN is NaN (where both groups
        // read them, both write the same zeros)
        const int past = key0 + 16 - w.len;
        if (past > 0) {
          for (int x = lane; x < min(past, 16) * C::kPanels * 8; x += 32) {
            const int row = key_w + 15 - x / (C::kPanels * 8), piece = x % (C::kPanels * 8);
            st_shared_v4_b32(base + stage + C::kV + (piece >> 3) * C::kPanel + row * 128 + ((piece & 7) << 4), 0u, 0u, 0u, 0u);
          }
          fence_async_smem();
          __syncwarp();
        }
      }
      // New references only where a score exceeds the old one by more than kTokMove
      float top[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) top[e] = fmaxf(d[e], d[e + 2]) * cl;
      constexpr float kFar = kTokMove<kType> + kTokUp<kType>;
      if (__any_sync(0xffffffffu, (top[0] > ref[0] + kFar) | (top[1] > ref[1] + kFar))) {
        float a[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
#pragma unroll
          for (int off = 4; off < 32; off <<= 1) top[e] = fmaxf(top[e], __shfl_xor_sync(0xffffffffu, top[e], off));
          const bool moves = top[e] > ref[e] + kFar;
          const float to = moves ? top[e] - kTokUp<kType> : ref[e];
          a[e] = moves ? ex2_approx(ref[e] - to) : 1.f;
          ref[e] = to;
          sub[e] = to == -INFINITY ? 0.f : to;
          l[e] *= a[e];
        }
#pragma unroll
        for (int mb = 0; mb < kSteps; ++mb)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[mb][e] *= a[e & 1];
      }
      uint32_t hi[2], lo[2];
#pragma unroll
      for (int i2 = 0; i2 < 2; ++i2) {
        const float x0 = ex2_approx(fmaf(d[2 * i2], cl, -sub[0])), x1 = ex2_approx(fmaf(d[2 * i2 + 1], cl, -sub[1]));
        l[0] += x0;
        l[1] += x1;
        const uint32_t h2 = pack_16x2<kType>(x0, x1);
        const float2 back = unpack_16x2<kType>(h2);
        hi[i2] = movmatrix_trans(h2);
        lo[i2] = movmatrix_trans(pack_16x2<kType>(x0 - back.x, x1 - back.y));
      }
#pragma unroll
      for (int mb = 0; mb < kSteps; mb += 2) {  // two at a time: an accumulator's second product waits for its first
        uint32_t a[2][4];
#pragma unroll
        for (int x = 0; x < 2; ++x)
          ldmatrix_x4_trans(a[x], vaddr + stage + (mb >> 2) * C::kPanel + (((((mb + x) & 3) * 2 + vpiece) ^ (vrow & 7)) << 4));
#pragma unroll
        for (int x = 0; x < 2; ++x) tok_mma<kType>(o[mb + x], a[x], hi[0], hi[1]);
#pragma unroll
        for (int x = 0; x < 2; ++x) tok_mma<kType>(o[mb + x], a[x], lo[0], lo[1]);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(full + 8 * C::kStages);
    }
    // The warps' statistics and O become the row's, or the share's partial.
    float2* const ml = ml_s + (seg & 1) * kTokWarps * 8;
    ++seg;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
#pragma unroll
      for (int off = 4; off < 32; off <<= 1) l[e] += __shfl_xor_sync(0xffffffffu, l[e], off);
      if (r == 0) ml[warp * 8 + 2 * c + e] = make_float2(ref[e], l[e]);
    }
    tok_join_sync();
    const int join0 = C::kSplit ? group * 4 : 0;  // the first warp of those that have keys of this one's rows
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      float m = -INFINITY;
#pragma unroll
      for (int x = 0; x < C::kJoin; ++x) m = fmaxf(m, ml[(join0 + x) * 8 + 2 * c + e].x);
      const float f = ref[e] == -INFINITY ? 0.f : ex2_approx(ref[e] - m);
      // (a warp without keys has nothing to add, and 0 * NaN would be something)
      if (ref[e] != -INFINITY || l[e] != 0.f) {
#pragma unroll
        for (int mb = 0; mb < kSteps; ++mb) o[mb][e] *= f, o[mb][e + 2] *= f;
      }
    }
    // kSlots of a row's warps at a time, always in the same order
    const int rank = C::kSplit ? warp & 3 : warp ^ 4;
    float* const mine = o_s + ((rank % C::kSlots) * C::kRows + r0) * C::kOStride;
#pragma unroll 1
    for (int step = 0; step < C::kJoin / C::kSlots; ++step) {
      if (rank / C::kSlots == step) {
#pragma unroll
        for (int mb = 0; mb < kSteps; ++mb)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            float& to = mine[(2 * c + (e & 1)) * C::kOStride + mb * 16 + r + (e >> 1) * 8];
            to = step == 0 ? o[mb][e] : to + o[mb][e];
          }
      }
      tok_join_sync();
    }
    if constexpr (!kDirect) {
      if (warp == 0 && lane == 0 && seg == 1) {
        // the CTA's first row: is this the first cut of it?
        const int64_t share = k.share, first = k.at / share, last = (k.at + w.tiles - 1) / share;
        const bool here = k.t0 > 0 && first + 1 == static_cast<int64_t>(blockIdx.x);
        *(p.cuts + blockIdx.x) = TokCut{here ? static_cast<int>(first) : -1, static_cast<int>(last), k.h, w.row0, rows, {0, 0, 0}};
      }
    }
    const bool whole = kDirect || (k.t0 == 0 && k.t1 == w.tiles);
    const int part = 2 * static_cast<int>(blockIdx.x) + (k.t0 == 0 ? 1 : 0);
    for (int x = warp * 32 + lane; x < C::kRows * (D / 4); x += kTokWarps * 32) {
      const int n = x / (D / 4), ch = (x % (D / 4)) * 4;
      if (n >= rows || !ok) continue;
      float m = -INFINITY, sum = 0.f;
#pragma unroll
      for (int y = 0; y < C::kJoin; ++y) m = fmaxf(m, ml[((n >> 3) * C::kJoin + y) * 8 + (n & 7)].x);
#pragma unroll
      for (int y = 0; y < C::kJoin; ++y) {
        const float2 v = ml[((n >> 3) * C::kJoin + y) * 8 + (n & 7)];
        if (v.x != -INFINITY || v.y != 0.f) sum += v.x == -INFINITY ? v.y : v.y * ex2_approx(v.x - m);
      }
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int y = 0; y < C::kSlots; ++y) {
        const float4 u = *reinterpret_cast<const float4*>(o_s + (y * C::kRows + n) * C::kOStride + ch);
        v.x += u.x, v.y += u.y, v.z += u.z, v.w += u.w;
      }
      if (whole) {
        const int tok = n / p.a.G, g = n - tok * p.a.G;
        const int64_t at = static_cast<int64_t>(w.row0 + tok) * p.a.s.H_kv * p.a.G + k.h * p.a.G + g;
        tok_write<kType>(p.a, at * D + ch, at, v, m, sum, ch == 0);
      } else {
        *reinterpret_cast<float4*>(p.o_part + (static_cast<int64_t>(part) * C::kRows + n) * D + ch) = v;
        if (ch == 0) p.ml_part[static_cast<int64_t>(part) * C::kRows + n] = make_float2(m, sum);
      }
    }
    more = kDirect ? false : k.next(p.a);
  }
}

template <int D, int kType, int kNT, bool kDirect>
__global__ void __launch_bounds__(kTokThreads, 1)
    attn_paged_token_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                            const __grid_constant__ TokParams p) {
  using C = TokCfg<D, kNT>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* const smem = smem_raw + (base - raw);
  volatile uint32_t* const misc = reinterpret_cast<volatile uint32_t*>(smem + C::kMisc);
  const int warp = static_cast<int>(threadIdx.x >> 5);
  if (threadIdx.x == 0) {
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(base + C::kBar + 8 * s, 2);                 // both producers
      mbar_init(base + C::kBar + 8 * (C::kStages + s), C::kUsers);
    }
    misc[0] = 0u;
    fence_barrier_init();
  } else if (threadIdx.x == 32) {
    tma_prefetch_desc(&tmK);
    tma_prefetch_desc(&tmV);
  }
  __syncthreads();
  const WaitCtx wc{p.a.timeout_ns, misc};
  grid_dependency_wait();
  grid_launch_dependents();
  TokWalk k;
  if (!tok_start<kTokThreads, kDirect>(k, p, reinterpret_cast<volatile int64_t*>(smem + C::kMisc + 16))) return;
  if (warp >= kTokWarps)
    tok_load<D, kNT, kDirect>(k, p, warp - kTokWarps, warp == kTokWarps ? &tmK : &tmV, base, wc);
  else
    tok_compute<D, kType, kNT, kDirect>(k, p, base, smem, warp, wc);
}

// Joins the partials of the rows that the shares' ends cut: blocks (c, y) query row y of
// those across the beginning of share c, if that is the first one within them.  The
// warps (and, at D = 64, half-warps) take turns at the partials, four on their way at
// once, and join through shared memory in their order.
constexpr int kTokMergeThreads = 128;
template <int D, int kType, int kRows>
__global__ void __launch_bounds__(kTokMergeThreads) attn_paged_merge_kernel(const __grid_constant__ TokParams p) {
  constexpr int kLanes = D / 4, kGroups = kTokMergeThreads / kLanes;
  __shared__ float2 ml_s[kGroups];
  __shared__ float4 o_s[kGroups][kLanes];
  grid_dependency_wait();
  grid_launch_dependents();
  const int4 c0 = __ldg(reinterpret_cast<const int4*>(p.cuts + blockIdx.x));
  const int rows = __ldg(&p.cuts[blockIdx.x].rows);
  const int ca = c0.x, cb = c0.y, h = c0.z, row0 = c0.w;
  const int n = static_cast<int>(blockIdx.y), group = static_cast<int>(threadIdx.x) / kLanes;
  const int ch = (static_cast<int>(threadIdx.x) % kLanes) * 4;
  if (ca < 0 || n >= rows) return;
  float m = -INFINITY, sum = 0.f;
  float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
  const auto add = [&](const float2* s, const float4* o) {
    const float to = fmaxf(fmaxf(fmaxf(s[0].x, s[1].x), fmaxf(s[2].x, s[3].x)), m);
    const float keep = m == -INFINITY ? 1.f : ex2_approx(m - to);  // (without a reference there is nothing, or NaN)
    m = to;
    sum *= keep, v.x *= keep, v.y *= keep, v.z *= keep, v.w *= keep;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if (s[e].x == -INFINITY && s[e].y == 0.f) continue;  // no key of it was seen
      const float f = s[e].x == -INFINITY ? 1.f : ex2_approx(s[e].x - m);
      sum = fmaf(s[e].y, f, sum);
      v.x = fmaf(o[e].x, f, v.x), v.y = fmaf(o[e].y, f, v.y), v.z = fmaf(o[e].z, f, v.z), v.w = fmaf(o[e].w, f, v.w);
    }
  };
  float2 s[4];
  float4 o[4];
  for (int y0 = ca + group; y0 <= cb; y0 += 4 * kGroups) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int y = y0 + e * kGroups;
      s[e] = make_float2(-INFINITY, 0.f);
      o[e] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (y <= cb) {
        const int64_t part = static_cast<int64_t>(2 * y + (y == ca ? 1 : 0)) * kRows + n;
        s[e] = __ldg(p.ml_part + part);
        o[e] = __ldg(reinterpret_cast<const float4*>(p.o_part + part * D + ch));
      }
    }
    add(s, o);
  }
  o_s[group][ch / 4] = v;
  if (ch == 0) ml_s[group] = make_float2(m, sum);
  __syncthreads();
  if (group != 0) return;
  for (int g0 = 1; g0 < kGroups; g0 += 4) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const bool there = g0 + e < kGroups;
      s[e] = there ? ml_s[g0 + e] : make_float2(-INFINITY, 0.f);
      o[e] = there ? o_s[g0 + e][ch / 4] : make_float4(0.f, 0.f, 0.f, 0.f);
    }
    add(s, o);
  }
  const int tok = n / p.a.G, g = n - tok * p.a.G;
  const int64_t at = static_cast<int64_t>(row0 + tok) * p.a.s.H_kv * p.a.G + h * p.a.G + g;
  tok_write<kType>(p.a, at * D + ch, at, v, m, sum, ch == 0);
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------

// Few rows with few keys each: a CTA a row and no second kernel.  16 rows of 700 / 1500 /
// 4000 keys, D = 64, took 6.7 / 11.6 / 26 us on the GPU so and 8.2 / 8.6 / 10.4 in shares,
// 128 rows 6.9 / 12.4 / 28 and 12.3 / 17.6 / 32; a second launch is 6 us on the host.
constexpr int kTokDirectLen = 1536;
constexpr int kTokSms = 152;  // (the workspace's size is asked for without a device)

// Up to how many (token, head) rows of a key head a sequence may have here.  16 rows over
// 32260 entries of 8 key heads take 30 us, 32 rows 54 us in the chunks' kernel.
constexpr int kTokMaxRows = 16;
static_assert(kTokMaxRows <= TokCfg<64, 2>::kRows && kTokMaxRows <= TokCfg<128, 2>::kRows, "a sequence's rows are one block");
bool paged_is_token(int max_new, int G) { return static_cast<int64_t>(max_new) * G <= kTokMaxRows; }

// What an attention over pages takes: 8 or 16 query rows, and a CTA a row or shares.
struct TokPlan {
  int nt;  // tiles of 8 query rows
  bool direct;
};
TokPlan tok_plan(int B, int H_kv, int G, int max_new, int max_len, int window, int sinks) {
  TokPlan t;
  t.nt = max_new * G <= 8 ? 1 : 2;  // (paged_is_token holds)
  const int64_t keys = window > 0 ? std::min<int64_t>(max_len, static_cast<int64_t>(window) + sinks + max_new) : max_len;
  t.direct = static_cast<int64_t>(B) * H_kv <= kTokSms && keys <= kTokDirectLen;
  return t;
}
uint64_t tok_workspace(const TokPlan& t, int D) {
  return t.direct ? 16 : static_cast<uint64_t>(2 * kTokSms) * 8 * t.nt * (D * sizeof(float) + sizeof(float2)) + kTokSms * sizeof(TokCut);
}

std::atomic<int> g_paged_state[kMaxDevices];  // 1: shared-memory limits set

template <int D, int kType>
bool tok_limits() {
  const auto limit = [](const void* f, int bytes) {
    return cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) == cudaSuccess;
  };
  return limit(reinterpret_cast<const void*>(attn_paged_token_kernel<D, kType, 1, false>), TokCfg<D, 1>::kBytes) &&
         limit(reinterpret_cast<const void*>(attn_paged_token_kernel<D, kType, 1, true>), TokCfg<D, 1>::kBytes) &&
         limit(reinterpret_cast<const void*>(attn_paged_token_kernel<D, kType, 2, false>), TokCfg<D, 2>::kBytes) &&
         limit(reinterpret_cast<const void*>(attn_paged_token_kernel<D, kType, 2, true>), TokCfg<D, 2>::kBytes);
}

// Pages as a tensor map {D, page, n_pages * H_kv} with boxes of 64 channels x `rows`, 128-byte swizzle.
bool encode_pages(CUtensorMap* m, const void* ptr, const attn_pages_t* c, int rows) {
  cuuint64_t dims[3] = {static_cast<cuuint64_t>(c->D), static_cast<cuuint64_t>(c->page),
                        static_cast<cuuint64_t>(c->n_pages) * static_cast<cuuint64_t>(c->H_kv)};
  cuuint64_t strides[2] = {static_cast<cuuint64_t>(c->D) * 2, static_cast<cuuint64_t>(c->page) * c->D * 2};
  cuuint32_t box[3] = {64, static_cast<cuuint32_t>(rows), 1};
  cuuint32_t estr[3] = {1, 1, 1};
  return g_encode(m, c->dtype == ATTN_FP16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3,
                  const_cast<void*>(ptr), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, int kType, int kNT>
cudaError_t tok_launch(const CUtensorMap& tk, const CUtensorMap& tv, const TokParams& p, bool direct, int64_t rows, cudaStream_t s) {
  using C = TokCfg<D, kNT>;
  if (direct)
    return launch_pdl(attn_paged_token_kernel<D, kType, kNT, true>, dim3(static_cast<unsigned>(rows)), dim3(kTokThreads), C::kBytes,
                      s, tk, tv, p);
  const cudaError_t e = launch_pdl(attn_paged_token_kernel<D, kType, kNT, false>, dim3(kTokSms), dim3(kTokThreads), C::kBytes, s,
                                   tk, tv, p);
  return e != cudaSuccess ? e
                          : launch_pdl(attn_paged_merge_kernel<D, kType, C::kRows>, dim3(kTokSms, static_cast<unsigned>(p.a.max_new * p.a.G)),
                                       dim3(kTokMergeThreads), 0, s, p);
}

attn_status_t tok_run(const attn_pages_t* c, const PagedAttn& a, const TokPlan& t, void* workspace, cudaStream_t s) {
  const int box = std::min(c->page, kTokTile);
  CUtensorMap tk, tv;
  if (!encode_pages(&tk, c->k_pages, c, box) || !encode_pages(&tv, c->v_pages, c, box)) return ATTN_ERR_LAUNCH;
  TokParams p;
  p.a = a;
  p.o_part = static_cast<float*>(workspace);
  p.ml_part = reinterpret_cast<float2*>(p.o_part + static_cast<int64_t>(2 * kTokSms) * 8 * t.nt * c->D);
  p.cuts = reinterpret_cast<TokCut*>(p.ml_part + static_cast<int64_t>(2 * kTokSms) * 8 * t.nt);
  p.box_rows = box;
  p.box_log2 = 0;
  while ((1 << p.box_log2) < box) ++p.box_log2;
  p.missing = c->n_pages * c->H_kv;
  const int64_t rows = static_cast<int64_t>(c->B) * c->H_kv;
  const auto run = [&](auto d, auto type) {
    return t.nt == 1 ? tok_launch<d(), type(), 1>(tk, tv, p, t.direct, rows, s) : tok_launch<d(), type(), 2>(tk, tv, p, t.direct, rows, s);
  };
  using D64 = std::integral_constant<int, 64>;
  using D128 = std::integral_constant<int, 128>;
  using Bf = std::integral_constant<int, kBF16>;
  using Fp = std::integral_constant<int, kFP16>;
  const bool bf = c->dtype == ATTN_BF16;
  const cudaError_t e = c->D == 64 ? (bf ? run(D64(), Bf()) : run(D64(), Fp())) : (bf ? run(D128(), Bf()) : run(D128(), Fp()));
  return e == cudaSuccess ? ATTN_OK : ATTN_ERR_LAUNCH;
}

}  // namespace
