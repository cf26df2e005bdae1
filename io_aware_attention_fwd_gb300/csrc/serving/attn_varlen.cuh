// Attention over whole prompts of different lengths, packed one behind the
// other, with grouped query heads.  Part of attn_fwd.cu: the tile arithmetic,
// the barriers and the roles are attn_fwd_sm103a's (bf16 form); what differs is
// stated here.
//
//   * A query tile's 128 rows are floor(128 / G) tokens times the G query heads
//     that share a key head, token by token: one TMA box {64 channels, G heads,
//     tokens} lays them out so.  Every K and V tile then serves all G heads, a
//     short prompt fills G times as many rows of its tile, and a causal tile
//     ends G times closer to the diagonal.  With G no divisor of 128 the last
//     128 mod G rows stay zero and are not stored.
//   * A work unit is two such tiles of one (sequence, key head).  The lengths
//     are on the device, so a one-block kernel lists the units there, heaviest
//     (most kv tiles) first, by a counting sort; the persistent CTAs walk that
//     list in the same snake order as the dense kernel's.  Where there can be no
//     more units than SMs, no order matters: each CTA finds its one unit itself
//     and there is no list (6 prompts of up to 61 tokens: 6.3 us instead of 7.6).
//   * A kv tile that reaches past its sequence's end holds rows of the next one
//     (or behind the last): their scores are masked, and the MMA warp zeroes
//     those rows of V in shared memory, because 0 * NaN is NaN.
//   * O rows of a tile go to memory a head's 128-byte panel at a time from the
//     staging buffer, so a tile that crosses its sequence's end writes nothing
//     of the next one's.

namespace {

struct VarlenUnit {  // two query tiles of one sequence, for every key head
  int row0;  // first packed row of the sequence
  int len;
  int i0;    // first token of the unit
};

struct VarlenParams {
  uint16_t* o;              // [total][H_q][D]
  float* lse;               // [H_q][total]
  const VarlenUnit* units;  // written by the plan kernel; null: a CTA finds its unit in seq_start
  const int32_t* n_listed;
  const int32_t* seq_start;
  int n_seqs;
  int64_t total;
  int H_kv;
  int G;             // query heads per key head
  int tok;           // tokens per query tile: 128 / G
  int rows;          // tok * G
  uint32_t inv_G;    // ceil(2^16 / G): r / G = r * inv_G >> 16 for r < 128
  float scale_log2;
  int causal;
  unsigned long long timeout_ns;
};

constexpr int kPlanThreads = 1024;
constexpr int kPlanBuckets = 2048;  // by kv tiles; longer units share the last

__device__ __forceinline__ int varlen_tiles(int i0, int len, int unit_tok, int causal) {
  const int lim = causal ? min(len, i0 + unit_tok) : len;
  return (lim + kBN - 1) / kBN;
}

// First row and length of sequence s, both ends taken as the rows there are: an
// end of any value leaves the length within 0 .. most.
struct VarlenRows {
  int row0, len;
};
__device__ __forceinline__ VarlenRows varlen_rows(const int32_t* __restrict__ seq_start, int s, int most) {
  const int row0 = min(max(__ldg(seq_start + s), 0), most);
  return {row0, max(0, min(max(__ldg(seq_start + s + 1), 0), most) - row0)};
}

// Lists the work units of every sequence, most kv tiles first (in no fixed
// order among equals: each unit's result is its own).  At most `cap` entries,
// which ascending seq_start never exceeds.
__global__ void __launch_bounds__(kPlanThreads)
    attn_varlen_plan(const int32_t* __restrict__ seq_start, int n_seqs, int64_t total, int unit_tok, int causal,
                     VarlenUnit* __restrict__ units, int32_t* __restrict__ n_listed, int cap) {
  __shared__ int cnt[kPlanBuckets];
  __shared__ int warp_s[kPlanThreads / 32];
  const int tid = static_cast<int>(threadIdx.x), lane = tid & 31, warp = tid >> 5;
  for (int i = tid; i < kPlanBuckets; i += kPlanThreads) cnt[i] = 0;
  grid_dependency_wait();
  grid_launch_dependents();
  __syncthreads();
  const int most = static_cast<int>(total);
  // pass 0 counts the units of each bucket, pass 1 places them
  for (int pass = 0; pass < 2; ++pass) {
    for (int s = warp; s < n_seqs; s += kPlanThreads / 32) {
      const auto [row0, len] = varlen_rows(seq_start, s, most);
      for (int i0 = lane * unit_tok; i0 < len; i0 += 32 * unit_tok) {
        const int b = kPlanBuckets - 1 - min(varlen_tiles(i0, len, unit_tok, causal), kPlanBuckets - 1);
        const int at = atomicAdd(&cnt[b], 1);
        if (pass == 1 && static_cast<unsigned>(at) < static_cast<unsigned>(cap)) units[at] = VarlenUnit{row0, len, i0};
        if (len - i0 <= 32 * unit_tok) break;  // i0 + 32 * unit_tok may not fit an int
      }
    }
    __syncthreads();
    if (pass == 0) {  // exclusive scan, two buckets a thread
      static_assert(kPlanBuckets == 2 * kPlanThreads, "two buckets a thread");
      const int a = cnt[2 * tid], c = cnt[2 * tid + 1];
      int incl = a + c;
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, incl, off);
        if (lane >= off) incl += y;
      }
      if (lane == 31) warp_s[warp] = incl;
      __syncthreads();
      int before = incl - a - c;
      for (int w = 0; w < warp; ++w) before += warp_s[w];
      cnt[2 * tid] = before;
      cnt[2 * tid + 1] = before + a;
      if (tid == kPlanThreads - 1) *n_listed = min(before + a + c, cap);
      __syncthreads();
    }
  }
}

struct VUnit {
  int row0, len, h;
  int i0[kQTiles];   // first token of each tile (past the end: the tile is not stored)
  int nkv[kQTiles];  // kv tiles it visits (>= 1)
  int n;
};

// Unit u: from the list, or the CTA's only one from shared memory.
__device__ __forceinline__ VUnit varlen_unit(const VarlenParams& p, const volatile int* own, int u) {
  const VarlenUnit* e = p.units + u / p.H_kv;
  const bool listed = p.units != nullptr;
  VUnit w;
  w.h = u % p.H_kv;
  // (clamped once more: whatever seq_start holds, no row outside the buffers)
  const int most = static_cast<int>(p.total);
  w.row0 = min(max(listed ? __ldg(&e->row0) : own[1], 0), most);
  w.len = min(max(listed ? __ldg(&e->len) : own[2], 0), most - w.row0);
  const int i0 = max(listed ? __ldg(&e->i0) : own[3], 0);
  w.n = 1;
#pragma unroll
  for (int t = 0; t < kQTiles; ++t) {
    w.i0[t] = i0 + t * p.tok;
    w.nkv[t] = w.i0[t] < w.len ? varlen_tiles(w.i0[t], w.len, p.tok, p.causal) : 1;
    w.n = max(w.n, w.nkv[t]);
  }
  return w;
}

// The units of this CTA: the snake order over the listed ones, or its own one.
struct VarlenSeq {
  int n_units, rounds, G, cta;
  __device__ VarlenSeq(const VarlenParams& p, const volatile int* own)
      : n_units((p.units != nullptr ? __ldg(p.n_listed) : own[0]) * p.H_kv),
        G(static_cast<int>(gridDim.x)),
        cta(static_cast<int>(blockIdx.x)) {
    rounds = (n_units + G - 1) / G;
  }
  __device__ int at(int r) const { return unit_of(r, cta, G); }
};

// TMA producer (one thread), as load_role.
template <int D>
__device__ void varlen_load_role(const Smem<D, false>& sm, const volatile int* own, const CUtensorMap* tmQ, const CUtensorMap* tmK,
                                 const CUtensorMap* tmV, const VarlenParams& p, const WaitCtx& w) {
  using C = Cfg<D, false>;
  int it = 0;
  int k = 0;
  bool ok = true;
  const uint64_t pol_first = l2_evict_first();
  const VarlenSeq us(p, own);
  for (int r = 0; r < us.rounds && ok; ++r) {
    const int u = us.at(r);
    if (u >= us.n_units) continue;
    const VUnit un = varlen_unit(p, own, u);
    if (k > 0) {
      ok = mbar_wait(sm.bar_qfree(0), (k - 1) & 1, w) && mbar_wait(sm.bar_qfree(1), (k - 1) & 1, w);
      if (!ok) break;
    }
    mbar_expect_tx(sm.bar_q(), static_cast<uint32_t>(kQTiles * C::kPanels * p.rows * 128));
    for (int t = 0; t < kQTiles; ++t) {
      const int i0 = un.i0[t] < un.len ? un.i0[t] : un.i0[0];  // a tile past the end reloads tile 0
      for (int pn = 0; pn < C::kPanels; ++pn)
        tma_load_3d_hint(sm.q(t) + pn * kPanelBytes, tmQ, sm.bar_q(), pn * C::kBoxCols, un.h * p.G, un.row0 + i0,
                         pol_first);
    }
    ++k;
    for (int j = 0; j < un.n && ok; ++j) {
      for (int kv = 0; kv < 2; ++kv) {
        const int s = it % C::kSlots;
        const int round = it / C::kSlots;
        if (round > 0 && !mbar_wait(sm.bar_empty(s), (round - 1) & 1, w)) {
          ok = false;
          break;
        }
        mbar_expect_tx(sm.bar_full(s), C::kTileBytes);
        const CUtensorMap* m = kv ? tmV : tmK;
        for (int pn = 0; pn < C::kPanels; ++pn)
          tma_load_3d(sm.slot(s) + pn * kPanelBytes, m, sm.bar_full(s), pn * C::kBoxCols, un.h, un.row0 + j * kBN);
        ++it;
      }
    }
  }
  grid_launch_dependents();
  bool drained = (k == 0) || mbar_wait_drain(sm.bar_q(), (k - 1) & 1, w);
  for (int i = (it > C::kSlots ? it - C::kSlots : 0); i < it && drained; ++i)
    drained = mbar_wait_drain(sm.bar_full(i % C::kSlots), (i / C::kSlots) & 1, w);
}

// MMA issuer, as mma_role; it also zeroes the rows of V past the sequence's end.
template <int D, int kType>
__device__ void varlen_mma_role(const Smem<D, false>& sm, const volatile int* own, uint32_t tmem, const VarlenParams& p, const WaitCtx& w) {
  using C = Cfg<D, false>;
  // kind::f16: format code 0 is fp16, 1 is bf16 (make_idesc's e4m3 flag writes 0)
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
  const VarlenSeq us(p, own);
  for (int r = 0; r < us.rounds && ok; ++r) {
    const int u = us.at(r);
    if (u >= us.n_units) continue;
    const VUnit un = varlen_unit(p, own, u);
    const int sk0 = it % C::kSlots;
    ok = __all_sync(0xffffffffu, mbar_wait(sm.bar_q(), k & 1, w) &&
                                     mbar_wait(sm.bar_full(sk0), (it / C::kSlots) & 1, w));
    if (!ok) break;
    tc_fence_after();
#pragma unroll
    for (int t = 0; t < kQTiles; ++t) {
      issue_qk<D, false>(leader, tS[t], qd[t], kd0 + sk0 * kSlotStep, idesc_s);
      tc_commit_if(leader, sm.bar_s(t));
      if (un.nkv[t] == 1) tc_commit_if(leader, sm.bar_qfree(t));
    }
    issued = true;
    tc_commit_if(leader, sm.bar_empty(sk0));
    ++it;
    for (int j = 0; j < un.n && ok; ++j) {
      const int iv = it, ik = it + 1;
      const int sv = iv % C::kSlots, skn = ik % C::kSlots;
      const bool has_next = j + 1 < un.n;
      ok = __all_sync(0xffffffffu, mbar_wait(sm.bar_full(sv), (iv / C::kSlots) & 1, w) &&
                                       (!has_next || mbar_wait(sm.bar_full(skn), (ik / C::kSlots) & 1, w)));
      const int past = (j + 1) * kBN - un.len;  // rows of this tile behind the sequence
      if (ok && past > 0) {  // (at most one tile of a unit)
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
        if (!ok || j >= un.nkv[t]) continue;
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
        if (j + 1 < un.nkv[t]) {
          issue_qk<D, false>(leader, tS[t], qd[t], kd0 + skn * kSlotStep, idesc_s);
          tc_commit_if(leader, sm.bar_s(t));
          if (j + 2 == un.nkv[t]) tc_commit_if(leader, sm.bar_qfree(t));
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

// What P is held in.  bf16 has fp32's range: p is relative to the row's reference,
// which moves when the maximum exceeds it by 2^8, as in softmax_role.  fp16 ends at
// 2^16, and its bits go below 2^-14: there P is held 2^11 times as large and the
// reference moves at 2^4, so p stays at or below 2^15 and keeps its 11 bits down to
// 2^-25 of the largest (as p itself it lost them from 2^-14 on and was 0 from 2^-25
// on, while the row sum counted it: 4096 keys 18 nats below one of V = 0 gave an O
// that was off by all of itself).  The row sum carries the same factor, which leaves
// O with the division and the LSE in the epilogue.
template <int kType>
constexpr float kVarlenUp = kType == kFP16 ? 11.f : 0.f;
template <int kType>
constexpr float kVarlenRescale = kType == kFP16 ? 4.f : kRescaleLog2;

// Softmax of query tile t, as softmax_role: row r is token r / G of the tile.
template <int D, int kType>
__device__ void varlen_softmax_role(const Smem<D, false>& sm, const volatile int* own, int t, uint32_t tmem, const VarlenParams& p,
                                    const WaitCtx& w) {
  using C = Cfg<D, false>;
  const int r = static_cast<int>(threadIdx.x) - kBM * (1 + t);
  const int qw = r >> 5;
  const uint32_t lane_off = static_cast<uint32_t>(qw * 32) << 16;
  const uint32_t tS = tmem + lane_off + t * kBN;
  const float c = p.scale_log2;
  const int tok = static_cast<int>((static_cast<uint32_t>(r) * p.inv_G) >> 16);
  int cnt = 0;
  int sbase = 0;
  int k = 0;
  bool ok = true;
  const VarlenSeq us(p, own);
  for (int rr = 0; rr < us.rounds && ok; ++rr) {
    const int u = us.at(rr);
    if (u >= us.n_units) continue;
    const VUnit un = varlen_unit(p, own, u);
    const int i0 = t ? un.i0[1] : un.i0[0];
    // Keys j < lj of the kv tile at hand are allowed for this row; tiles from
    // `masked` on hold keys that some row may not see
    int lj = p.causal ? min(un.len, i0 + tok + 1) : un.len;
    const int masked = p.causal ? min(un.len, i0 + 1) / kBN : un.len / kBN;
    const int nkv = t ? un.nkv[1] : un.nkv[0], n_other = t ? un.nkv[0] : un.nkv[1];
    const int steps = nkv + n_other;  // of both query tiles
    int step = sbase + t;             // of this tile's next kv tile, in the order tile 0, tile 1

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

      if (j >= masked) {
#pragma unroll
        for (int i = 0; i < kBN; ++i) s[i] = (i < lj) ? s[i] : -INFINITY;
      }
      lj -= kBN;
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

// Epilogue warpgroup, as epilogue_role, with O written row by row.  Half a
// panel at a time and loops that are not unrolled keep it within its 72
// registers; unrolled, it spilt 250 bytes (16 prompts of up to 2500 tokens,
// D = 128: 175 us instead of 154 to 157).
template <int D, int kType>
__device__ void varlen_epilogue_role(const Smem<D, false>& sm, const volatile int* own, uint32_t tmem, const VarlenParams& p,
                                     const WaitCtx& w) {
  using C = Cfg<D, false>;
  const int qw = static_cast<int>(threadIdx.x >> 5) & 3;
  const int lane = static_cast<int>(threadIdx.x & 31);
  const int rt = qw * 32 + lane;
  const uint32_t lane_off = static_cast<uint32_t>(qw * 32) << 16;
  const uint32_t stage = sm.stage(qw);
  const int tok = static_cast<int>((static_cast<uint32_t>(rt) * p.inv_G) >> 16);  // this row's token and head
  const int g = rt - tok * p.G;
  int cnt[kQTiles] = {0, 0};
  int k = 0;
  bool ok = true;
  const VarlenSeq us(p, own);
  for (int rr = 0; rr < us.rounds && ok; ++rr) {
    const int u = us.at(rr);
    if (u >= us.n_units) continue;
    const VUnit un = varlen_unit(p, own, u);
#pragma unroll
    for (int t = 0; t < kQTiles; ++t) {
      if (!ok) break;
      const int nkv = un.nkv[t];
      ok = __all_sync(0xffffffffu, mbar_wait_sleepy(sm.bar_epi(t), k & 1, w));
      if (!ok) break;
      const float2 ml = sm.stat(t)[rt];
      ok = __all_sync(0xffffffffu, mbar_wait(sm.bar_o(t), (cnt[t] + nkv - 1) & 1, w));
      cnt[t] += nkv;
      if (!ok) break;
      tc_fence_after();
      const uint32_t tO = tmem + lane_off + C::kOCol0 + t * D;
      const uint64_t il2 = pack_f32x2(1.f / ml.y, 1.f / ml.y);
      const uint32_t rowa = stage + static_cast<uint32_t>(lane) * 128u;
      // rows of this tile that exist: tokens before the sequence's end
      const int rows = min(p.rows, (un.len - un.i0[t]) * p.G);
      const int64_t tok0 = un.row0 + un.i0[t];
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
              // A mean of fp16 values is an fp16 value, but the sum of the rounded P
              // may exceed the row's by half a step: at 65504 that is infinity.
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
          // row - rtok * G is the head in the group
          const int64_t at = ((tok0 + rtok) * p.H_kv + un.h) * p.G + (row - rtok * p.G);
          st_global_v4(p.o + at * D + pn * 64 + ch * 8, x[0], x[1], x[2], x[3]);
        }
      }
      if (rt < rows) {  // (the factor comes off the sum first: a sum near 1 has the more exact logarithm)
        const float l2 = kType == kFP16 ? (ml.x + kVarlenUp<kType>) + log2f(ml.y * 0x1p-11f) : ml.x + log2f(ml.y);
        p.lse[static_cast<int64_t>(un.h * p.G + g) * p.total + tok0 + tok] = l2 * kLn2;
      }
    }
    ++k;
  }
}

// The unit of this CTA where there is no list: own[0] the number of units per
// key head, own[1 .. 3] row0, len and i0 of unit blockIdx.x / H_kv.  One warp;
// units are numbered sequence by sequence.
__device__ __forceinline__ void varlen_own_unit(const VarlenParams& p, volatile int* own) {
  const int lane = static_cast<int>(threadIdx.x & 31);
  const int mine = static_cast<int>(blockIdx.x) / p.H_kv, unit_tok = kQTiles * p.tok, most = static_cast<int>(p.total);
  int before = 0;
  for (int s0 = 0; s0 < p.n_seqs; s0 += 32) {
    const int s = s0 + lane;
    VarlenRows r{0, 0};
    if (s < p.n_seqs) r = varlen_rows(p.seq_start, s, most);
    const auto [row0, len] = r;
    const int n = (len + unit_tok - 1) / unit_tok;
    int incl = n;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, incl, off);
      if (lane >= off) incl += y;
    }
    const int first = before + incl - n;
    if (first <= mine && mine < first + n) {
      own[1] = row0;
      own[2] = len;
      own[3] = (mine - first) * unit_tok;
    }
    before += __shfl_sync(0xffffffffu, incl, 31);
  }
  if (lane == 0) own[0] = min(before, static_cast<int>(gridDim.x) / p.H_kv);
}

template <int D, int kType>
__global__ void __launch_bounds__(kFwdThreads, 1)
    attn_varlen_sm103a(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                       const __grid_constant__ CUtensorMap tmV, const VarlenParams p) {
  using C = Cfg<D, false>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* smem = smem_raw + (base - raw);
  const Smem<D, false> sm{base, smem};
  volatile int* const own = reinterpret_cast<volatile int*>(smem + C::kListOff);  // (the dense kernel's unit list lies here)
  volatile uint32_t* misc = reinterpret_cast<volatile uint32_t*>(smem + C::kMiscOff);

  const int warp = static_cast<int>(threadIdx.x >> 5);
  const int lane = static_cast<int>(threadIdx.x & 31);

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
  const WaitCtx w{p.timeout_ns, misc + 1};
  grid_dependency_wait();  // the unit list, and the caller's inputs before it
  if (p.units == nullptr) {
    if (warp == 0) varlen_own_unit(p, own);
    __syncthreads();
  }

  if (warp < 4) {
    regs_set<kRegsRoles>();
    if (warp == 0) {
      if (lane == 0) varlen_load_role<D>(sm, own, &tmQ, &tmK, &tmV, p, w);
    } else if (warp == 1) {
      varlen_mma_role<D, kType>(sm, own, tmem, p, w);
    }
  } else if (warp < kEpiWarp0) {
    regs_set<kRegsSoftmax>();
    varlen_softmax_role<D, kType>(sm, own, (warp - 4) >> 2, tmem, p, w);
  } else {
    regs_set<kRegsEpi>();
    varlen_epilogue_role<D, kType>(sm, own, tmem, p, w);
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

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------

std::atomic<int> g_varlen_state[kMaxDevices];  // 1: shared-memory limits set

// Rows [total][H][D] (row stride in elements) as a 3-D tensor map with boxes
// of 64 channels x `heads` heads x `tokens` rows, 128-byte swizzle.
bool encode_rows(CUtensorMap* m, const void* ptr, int D, int H, int64_t total, int64_t stride, int heads, int tokens,
                 int dtype) {
  cuuint64_t dims[3] = {static_cast<cuuint64_t>(D), static_cast<cuuint64_t>(H), static_cast<cuuint64_t>(total)};
  cuuint64_t strides[2] = {static_cast<cuuint64_t>(D) * 2, static_cast<cuuint64_t>(stride) * 2};
  cuuint32_t box[3] = {64, static_cast<cuuint32_t>(heads), static_cast<cuuint32_t>(tokens)};
  cuuint32_t estr[3] = {1, 1, 1};
  return g_encode(m, dtype == ATTN_FP16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3,
                  const_cast<void*>(ptr), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Units the list can hold: one for every 2 * tok tokens and one ragged end a
// sequence.
int64_t varlen_cap(int64_t total, int n_seqs, int G) { return total / (kQTiles * (kBM / G)) + n_seqs; }

// Without a list where there are at most as many units as a GB300 has SMs.
constexpr int kVarlenDirect = 152;
bool varlen_listed(int64_t cap, int H_kv) { return cap * H_kv > kVarlenDirect; }

template <int D, int kType>
attn_status_t launch_varlen(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv, const VarlenParams& prm,
                            int grid, cudaStream_t stream) {
  return launch_pdl(attn_varlen_sm103a<D, kType>, dim3(static_cast<unsigned>(grid)), dim3(kFwdThreads),
                    Cfg<D, false>::kSmemBytes, stream, tq, tk, tv, prm) == cudaSuccess
             ? ATTN_OK
             : ATTN_ERR_LAUNCH;
}

}  // namespace

extern "C" {

uint64_t attn_fwd_varlen_workspace_bytes(int64_t total, int n_seqs, int H_q, int H_kv, int D) {
  if (total < 0 || total > INT_MAX || n_seqs < 1 || H_kv < 1 || H_q < H_kv || H_q % H_kv != 0 || H_q / H_kv > kBM ||
      (D != 64 && D != 128))
    return 0;
  const int64_t cap = varlen_cap(total, n_seqs, H_q / H_kv);
  return varlen_listed(cap, H_kv) ? 16 + static_cast<uint64_t>(cap) * sizeof(VarlenUnit) : 16;
}

attn_status_t attn_fwd_varlen(const void* q, const void* k, const void* v, void* o, float* lse, int64_t total,
                              const int32_t* seq_start, int n_seqs, int H_q, int H_kv, int D, int dtype,
                              int64_t q_stride, int64_t k_stride, int64_t v_stride, float scale, int causal,
                              void* workspace, uint64_t workspace_bytes, void* stream) {
  if (total < 0 || n_seqs < 1 || H_kv < 1 || H_q < H_kv || H_q % H_kv != 0) return ATTN_ERR_INVALID_ARG;
  if (total > 0 && (q == nullptr || k == nullptr || v == nullptr || o == nullptr || lse == nullptr ||
                    seq_start == nullptr))
    return ATTN_ERR_INVALID_ARG;
  if (causal != 0 && causal != 1) return ATTN_ERR_INVALID_ARG;
  if (!std::isfinite(scale) || !(scale > 0.f)) return ATTN_ERR_INVALID_ARG;
  if ((D != 64 && D != 128) || (dtype != ATTN_BF16 && dtype != ATTN_FP16) || H_q / H_kv > kBM || total > INT_MAX)
    return ATTN_ERR_UNSUPPORTED;
  if (q_stride < static_cast<int64_t>(H_q) * D || k_stride < static_cast<int64_t>(H_kv) * D ||
      v_stride < static_cast<int64_t>(H_kv) * D)
    return ATTN_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(o, 16) || !aligned(lse, 4) ||
      !aligned(seq_start, 4) || !aligned(workspace, 16) || q_stride % 8 != 0 || k_stride % 8 != 0 || v_stride % 8 != 0)
    return ATTN_ERR_ALIGNMENT;
  const int G = H_q / H_kv;
  const int64_t cap = varlen_cap(total, n_seqs, G);
  if (cap * H_kv > INT_MAX / 2) return ATTN_ERR_UNSUPPORTED;
  const bool listed = varlen_listed(cap, H_kv);
  if (total > 0 && listed &&
      (workspace == nullptr || workspace_bytes < attn_fwd_varlen_workspace_bytes(total, n_seqs, H_q, H_kv, D)))
    return ATTN_ERR_INVALID_ARG;
  if (total == 0) return ATTN_OK;

  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return ATTN_ERR_DEVICE;
  const attn_status_t ps = prepare_device(dev);
  if (ps != ATTN_OK) return ps;
  if (g_varlen_state[dev].load(std::memory_order_acquire) == 0) {
    const auto limit = [](const void* f, int bytes) {
      return cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) == cudaSuccess;
    };
    if (!limit(reinterpret_cast<const void*>(attn_varlen_sm103a<64, kBF16>), Cfg<64, false>::kSmemBytes) ||
        !limit(reinterpret_cast<const void*>(attn_varlen_sm103a<64, kFP16>), Cfg<64, false>::kSmemBytes) ||
        !limit(reinterpret_cast<const void*>(attn_varlen_sm103a<128, kBF16>), Cfg<128, false>::kSmemBytes) ||
        !limit(reinterpret_cast<const void*>(attn_varlen_sm103a<128, kFP16>), Cfg<128, false>::kSmemBytes))
      return ATTN_ERR_DEVICE;
    g_varlen_state[dev].store(1, std::memory_order_release);
  }
  if (!get_encoder()) return ATTN_ERR_DEVICE;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  const int tok = kBM / G;
  CUtensorMap tq, tk, tv;
  if (!encode_rows(&tq, q, D, H_q, total, q_stride, G, tok, dtype) ||
      !encode_rows(&tk, k, D, H_kv, total, k_stride, 1, kBN, dtype) ||
      !encode_rows(&tv, v, D, H_kv, total, v_stride, 1, kBN, dtype))
    return ATTN_ERR_LAUNCH;
  int32_t* n_listed = listed ? static_cast<int32_t*>(workspace) : nullptr;
  VarlenUnit* units = listed ? reinterpret_cast<VarlenUnit*>(static_cast<char*>(workspace) + 16) : nullptr;
  if (listed && launch_pdl(attn_varlen_plan, dim3(1), dim3(kPlanThreads), 0, st, seq_start, n_seqs, total, kQTiles * tok, causal,
                 units, n_listed, static_cast<int>(cap)) != cudaSuccess)
    return ATTN_ERR_LAUNCH;
  VarlenParams prm;
  prm.o = static_cast<uint16_t*>(o);
  prm.lse = lse;
  prm.units = units;
  prm.n_listed = n_listed;
  prm.seq_start = seq_start;
  prm.n_seqs = n_seqs;
  prm.total = total;
  prm.H_kv = H_kv;
  prm.G = G;
  prm.tok = tok;
  prm.rows = tok * G;
  prm.inv_G = static_cast<uint32_t>((65536 + G - 1) / G);
  prm.scale_log2 = static_cast<float>(static_cast<double>(scale) * 1.4426950408889634074);
  prm.causal = causal;
  prm.timeout_ns = kDefaultTimeoutNs;
  const int64_t n_ctas = cap * H_kv;  // without a list a CTA to each, whatever SMs there are
  const int grid = static_cast<int>(listed ? std::min<int64_t>(n_ctas, g_dev_sms[dev].load(std::memory_order_relaxed)) : n_ctas);
  if (D == 64)
    return dtype == ATTN_BF16 ? launch_varlen<64, kBF16>(tq, tk, tv, prm, grid, st)
                              : launch_varlen<64, kFP16>(tq, tk, tv, prm, grid, st);
  return dtype == ATTN_BF16 ? launch_varlen<128, kBF16>(tq, tk, tv, prm, grid, st)
                            : launch_varlen<128, kFP16>(tq, tk, tv, prm, grid, st);
}

}  // extern "C"
