// A K/V cache in pages: writing a step's new tokens (with the norm and rotation
// of attn_rotary.cuh), and attention of them over it.  Part of attn_fwd.cu.
//
// Entry j of sequence b is row j % page of page table[b][j / page]; a page holds
// `page` rows of every key head, a head's rows side by side, so 16 keys of a head
// are 4 KB (D = 128) wherever they lie.

namespace {

constexpr unsigned kPagedOverflow = 4u;  // g_attn_status: entries beyond the capacity were dropped
constexpr unsigned kPagedNoPage = 8u;    // g_attn_status: an entry's page is none of the cache's

// Sequences of a call and where their entries lie.
struct PagedSeqs {
  const int32_t* table;      // [B][max_pages]
  const int32_t* len;        // [B]
  const int32_t* seq_start;  // [B + 1], or null: row b is sequence b's one row
  int64_t rows;
  int B, max_pages, n_pages, page_log2, H_kv;
  // First row, and rows, of sequence b: what seq_start says outside the rows counts for nothing.
  __device__ int start(int b) const {
    return static_cast<int>(min(max(static_cast<int64_t>(__ldg(seq_start + b)), static_cast<int64_t>(0)), rows));
  }
  __device__ int rows_of(int b) const { return seq_start != nullptr ? max(0, start(b + 1) - start(b)) : 1; }
  // The sequence of packed row `row`, or B.
  __device__ int sequence(int row) const {
    if (seq_start == nullptr) return row;
    if (row < start(0) || row >= start(B)) return B;
    int lo = 0, hi = B;  // start[lo] <= row < start[hi]
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (start(mid) <= row)
        lo = mid;
      else
        hi = mid;
    }
    return lo;
  }
  __device__ int64_t capacity() const { return static_cast<int64_t>(max_pages) << page_log2; }
  // Entries held.  Lengths are read past the SM's own cache: a kernel's blocks may be on the SM
  // while the append before it runs, which reads starts, table and old lengths and writes new
  // ones, and a line of all of these that came to that cache meanwhile has the old ones.
  __device__ int held(int b) const { return max(__ldcg(len + b), 0); }
  // Page of a sequence's block of entries, or -1.
  __device__ int page_of(int b, int block) const {
    const int pg = __ldg(table + static_cast<int64_t>(b) * max_pages + block);
    return pg >= 0 && pg < n_pages ? pg : -1;
  }
};

// Where an append's rows go, row by row, as rot_forward_body walks them.
struct PagedPlaces {
  PagedSeqs s;
  uint16_t *k, *v;
  int64_t head_step;  // page * D: from one key head's rows in a page to the next's
  // of the row at hand:
  int64_t to;         // first element of its place in its page, for key head 0, or -1
  int b, end;         // its sequence, or B, and the row behind its sequence's (or the next to look up)
  int pos;            // its entry's number
  __device__ bool live() const { return b < s.B; }
  __device__ void find(int row) {
    b = s.sequence(row);
    to = -1;
    pos = 0;
    end = row + 1;
    if (b >= s.B) return;
    int i = 0;
    if (s.seq_start != nullptr) {
      i = row - s.start(b);
      end = s.start(b + 1);
    }
    const int64_t at = static_cast<int64_t>(s.held(b)) + i;
    pos = static_cast<int>(min(at, static_cast<int64_t>(INT_MAX)));
    place();
  }
  // The next row: nearly always the same sequence's next entry.
  __device__ void step(int row) {
    if (row >= end || b >= s.B) {
      find(row);
      return;
    }
    pos = min(pos, INT_MAX - 1) + 1;
    if (to >= 0 && (pos & ((1 << s.page_log2) - 1)) != 0)
      to += head_step >> s.page_log2;
    else
      place();
  }
  __device__ void place() {
    to = -1;
    if (pos >= s.capacity()) {
      atomicOr(&g_attn_status, kPagedOverflow);
      return;
    }
    const int pg = s.page_of(b, pos >> s.page_log2);
    if (pg < 0) {
      atomicOr(&g_attn_status, kPagedNoPage);
      return;
    }
    to = static_cast<int64_t>(pg) * s.H_kv * head_step + static_cast<int64_t>(pos & ((1 << s.page_log2) - 1)) * (head_step >> s.page_log2);
  }
};

// An append: q normed and turned to its own rows, k normed and turned and v as it
// is to their pages, and the lengths after it.
// HBM-bound, 4 bytes a channel.
template <int D, int kType>
__global__ void __launch_bounds__(kRotThreads, kRotFwdBlocks)
    attn_paged_append_kernel(const __grid_constant__ RotParams p, const __grid_constant__ PagedPlaces places, int32_t* len_out) {
  rot_forward_body<D, kType, true>(p, places);
  if (len_out == nullptr) return;
  for (int64_t b = blockIdx.x * static_cast<int64_t>(blockDim.x) + threadIdx.x; b < places.s.B;
       b += static_cast<int64_t>(gridDim.x) * blockDim.x) {
    const int64_t l = static_cast<int64_t>(places.s.held(static_cast<int>(b))) + places.s.rows_of(static_cast<int>(b));
    len_out[b] = static_cast<int32_t>(min(l, places.s.capacity()));
  }
}
// The same update where len_out is the cache's own length (a launch behind the one
// whose blocks all read it), or where there are no rows.
__global__ void attn_paged_grow_kernel(const __grid_constant__ PagedSeqs s, int32_t* len_out) {
  grid_dependency_wait();
  grid_launch_dependents();
  for (int64_t b = blockIdx.x * static_cast<int64_t>(blockDim.x) + threadIdx.x; b < s.B;
       b += static_cast<int64_t>(gridDim.x) * blockDim.x) {
    const int64_t l = static_cast<int64_t>(s.held(static_cast<int>(b))) + s.rows_of(static_cast<int>(b));
    len_out[b] = static_cast<int32_t>(min(l, s.capacity()));
  }
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------

attn_status_t check_pages(const attn_pages_t* c) {
  if (c == nullptr || c->k_pages == nullptr || c->v_pages == nullptr || c->page_table == nullptr || c->length == nullptr || c->B < 1 ||
      c->H_kv < 1 || c->n_pages < 1 || c->max_pages < 1)
    return ATTN_ERR_INVALID_ARG;
  if ((c->D != 64 && c->D != 128) || (c->dtype != ATTN_BF16 && c->dtype != ATTN_FP16) || c->page < 16 || c->page > 256 ||
      (c->page & (c->page - 1)) != 0)
    return ATTN_ERR_UNSUPPORTED;
  if (static_cast<int64_t>(c->n_pages) * c->H_kv > INT_MAX / 2 || static_cast<int64_t>(c->max_pages) * c->page > INT_MAX / 2 ||
      static_cast<int64_t>(c->B) * c->H_kv > INT_MAX / 2)
    return ATTN_ERR_UNSUPPORTED;
  if (!aligned(c->k_pages, 16) || !aligned(c->v_pages, 16) || !aligned(c->page_table, 4) || !aligned(c->length, 4)) return ATTN_ERR_ALIGNMENT;
  return ATTN_OK;
}

PagedSeqs paged_seqs(const attn_pages_t* c, const int32_t* seq_start, int64_t rows) {
  int log2 = 0;
  while ((1 << log2) < c->page) ++log2;
  return {c->page_table, c->length, seq_start, rows, c->B, c->max_pages, c->n_pages, log2, c->H_kv};
}

}  // namespace

extern "C" {

attn_status_t attn_paged_append(const attn_pages_t* cache, const void* k, const void* v, int64_t rows, int64_t k_stride,
                                int64_t v_stride, const int32_t* seq_start, const void* q, int64_t q_stride, void* q_out,
                                int H_q, const attn_rotary_t* rope, const void* q_weight, const void* k_weight,
                                int weight_dtype, float eps, int32_t* length_out, void* stream) {
  attn_status_t st = check_pages(cache);
  if (st != ATTN_OK) return st;
  const int D = cache->D, H_kv = cache->H_kv;
  RotParams p{};
  st = rot_check_turn(rope, D, &p.turn);
  if (st != ATTN_OK) return st;
  st = rot_check_norm(q_weight, k_weight, weight_dtype, cache->dtype, eps);
  if (st != ATTN_OK) return st;
  if (rows < 0 || length_out == nullptr) return ATTN_ERR_INVALID_ARG;
  if (seq_start == nullptr && rows != cache->B) return ATTN_ERR_INVALID_ARG;
  // (without rows every buffer of rows may be null, as empty tensors are)
  if (rows > 0 && (k == nullptr || v == nullptr || (q == nullptr) != (q_out == nullptr) || (q == nullptr && q_weight != nullptr)))
    return ATTN_ERR_INVALID_ARG;
  if (q != nullptr && (H_q < 1 || H_q > 65535)) return H_q < 1 ? ATTN_ERR_INVALID_ARG : ATTN_ERR_UNSUPPORTED;
  if (rows > INT_MAX || H_kv > 65535) return ATTN_ERR_UNSUPPORTED;
  if (k_stride < static_cast<int64_t>(H_kv) * D || v_stride < static_cast<int64_t>(H_kv) * D ||
      (q != nullptr && q_stride < static_cast<int64_t>(H_q) * D))
    return ATTN_ERR_INVALID_ARG;
  if (!aligned(k, 16) || !aligned(v, 16) || !aligned(q, 16) || !aligned(q_out, 16) || k_stride % 8 != 0 || v_stride % 8 != 0 ||
      (q != nullptr && q_stride % 8 != 0) || !aligned(seq_start, 4) || !aligned(length_out, 4))
    return ATTN_ERR_ALIGNMENT;
  // new lengths over the old ones of other sequences
  if (length_out != cache->length && std::less<>()(length_out, cache->length + cache->B) &&
      std::less<>()(static_cast<const int32_t*>(cache->length), length_out + cache->B))
    return ATTN_ERR_INVALID_ARG;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return ATTN_ERR_DEVICE;
  st = prepare_device(dev);
  if (st != ATTN_OK) return st;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  PagedPlaces places{paged_seqs(cache, seq_start, rows), static_cast<uint16_t*>(cache->k_pages),
                     static_cast<uint16_t*>(cache->v_pages), static_cast<int64_t>(cache->page) * D, -1, 0, 0, 0};
  const bool in_place = length_out == cache->length;
  cudaError_t e = cudaSuccess;
  if (rows > 0) {
    const auto rows_of = [&](const void* x, int64_t stride) {
      return RotRows{static_cast<uint16_t*>(const_cast<void*>(x)), 0, stride, D};
    };
    if (q != nullptr) {
      p.in[0] = rows_of(q, q_stride);
      p.out[0] = rows_of(q_out, static_cast<int64_t>(H_q) * D);
    }
    p.in[1] = rows_of(k, k_stride);
    p.in[2] = rows_of(v, v_stride);
    p.w[0] = q_weight, p.w[1] = k_weight;
    p.w_fp32 = weight_dtype == ATTN_FP32;
    p.eps = eps;
    p.S = static_cast<int>(rows);
    const RotGrid g = rot_grid(rows, rot_groups(&p, D, q != nullptr ? H_q : 0, H_kv, H_kv),
                               g_dev_sms[dev].load(std::memory_order_relaxed), kRotFwdBlocks, kRotWarps);
    p.total = g.total, p.share = g.share;
    const auto run = [&](auto kernel) {
      return launch_pdl(kernel, dim3(g.blocks), dim3(kRotThreads), 0, s, p, places, in_place ? nullptr : length_out);
    };
    const bool bf = cache->dtype == ATTN_BF16;
    e = D == 64 ? (bf ? run(attn_paged_append_kernel<64, kBF16>) : run(attn_paged_append_kernel<64, kFP16>))
                : (bf ? run(attn_paged_append_kernel<128, kBF16>) : run(attn_paged_append_kernel<128, kFP16>));
  }
  if (e == cudaSuccess && (in_place || rows == 0))
    e = launch_pdl(attn_paged_grow_kernel, dim3(static_cast<unsigned>(std::min((cache->B + 255) / 256, 64))), dim3(256), 0, s,
                   places.s, length_out);
  return e == cudaSuccess ? ATTN_OK : ATTN_ERR_LAUNCH;
}

}  // extern "C"
