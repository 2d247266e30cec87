// The paged cache's bookkeeping for a step: lengths, page tables, the free list
// and the rows' positions and slots from what sequences keep and gain
// (moe_kv_pages).
//
// Every CTA scans the sequences (at most 8192) by itself, so one launch does it
// all, and then serves its share of the rows and of the pages that move.  No CTA
// reads what another writes: pages that are taken come from entries of the list
// below its old length, or straight from the table of a sequence that shrinks;
// what is written are table entries of sequences that grow and list entries past
// the old length.
//
// What bounds it is a thread's chain of loads, scans and searches, not bytes: 256
// sequences with a token each take 3.4 us, 61 with 5 drafts 4.3, 1024 prompts of up to
// 2048 tokens 10 (16 bytes a row, 1.8 TB/s).  512 threads: 768 and 1024 took 3.6 and
// 3.8 us for the first; a second CTA an SM made all of them slower.
#include <algorithm>

#include "common.cuh"

namespace moe {
namespace {

constexpr int kPagesThreads = 512;
constexpr int kPagesMaxBatch = 8192;

struct PagesArgs {
  moe_kv_pages_desc d;
  int32_t shift;   // log2 page_size
};

// Sums over sequences that stop at 2^31 - 1, which is past all that may be asked for: below
// it they are exact, and so are the sums in front of them.
constexpr uint32_t kMost = INT32_MAX;
__device__ __forceinline__ uint32_t add(uint32_t x, uint32_t y) { return min(x + y, kMost); }
struct Sums {      // new tokens, pages taken, pages given back
  uint32_t n, take, back;
  __device__ __forceinline__ Sums operator+(const Sums& o) const { return {add(n, o.n), add(take, o.take), add(back, o.back)}; }
};

__device__ __forceinline__ Sums shfl_up(const Sums& v, int o) {
  return {__shfl_up_sync(0xffffffffu, v.n, o), __shfl_up_sync(0xffffffffu, v.take, o), __shfl_up_sync(0xffffffffu, v.back, o)};
}
__device__ __forceinline__ Sums shfl(const Sums& v, int lane) {
  return {__shfl_sync(0xffffffffu, v.n, lane), __shfl_sync(0xffffffffu, v.take, lane), __shfl_sync(0xffffffffu, v.back, lane)};
}

// The sums over the block's threads before this one; `total` gets the sum of all.
__device__ Sums block_scan(const Sums& v, Sums* part, Sums& total) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  Sums x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const Sums y = shfl_up(x, o);
    if (lane >= o) x = x + y;
  }
  __syncthreads();            // `part` of an earlier call has been read
  if (lane == 31) part[warp] = x;
  __syncthreads();
  Sums w = lane < kPagesThreads / 32 ? part[lane] : Sums{0, 0, 0};
#pragma unroll
  for (int o = 1; o < kPagesThreads / 32; o <<= 1) {
    const Sums y = shfl_up(w, o);
    if (lane >= o) w = w + y;
  }
  total = shfl(w, kPagesThreads / 32 - 1);
  Sums before = shfl_up(x, 1);
  if (lane == 0) before = Sums{0, 0, 0};
  return warp ? shfl(w, warp - 1) + before : before;
}

// The last b in [0, n) with first[b] <= x (first is not decreasing, first[0] <= x).
__device__ __forceinline__ int find_last(const int32_t* first, int n, int32_t x) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (first[mid] <= x) lo = mid; else hi = mid;
  }
  return lo;
}

__global__ void __launch_bounds__(kPagesThreads) kv_pages_kernel(const __grid_constant__ PagesArgs a) {
  extern __shared__ int32_t pages_smem[];
  __shared__ Sums part[kPagesThreads / 32];
  const moe_kv_pages_desc& d = a.d;
  const int B = d.batch;
  // by sequence: first row, first page taken, first page given back (a prefix sum each,
  // one entry more than sequences), tokens kept, pages held and pages in the end
  int32_t* row0 = pages_smem;
  int32_t* take0 = row0 + B + 1;
  int32_t* back0 = take0 + B + 1;
  int32_t* keep_of = back0 + B + 1;
  int32_t* held_of = keep_of + B;
  int32_t* need_of = held_of + B;
  grid_dependency_wait();
  grid_launch_dependents();

  const int per = (B + kPagesThreads - 1) / kPagesThreads;
  const int b0 = min(static_cast<int>(threadIdx.x) * per, B), b1 = min(b0 + per, B);
  const int64_t most = static_cast<int64_t>(d.max_pages) << a.shift;
  const int32_t f = *d.free_count;
  const bool list_ok = f >= 0 && f <= d.free_capacity;
  auto pages = [&](int64_t tokens) { return static_cast<int32_t>((tokens + d.page_size - 1) >> a.shift); };

  // What a sequence asks for, kept in its places of the arrays until it is known what it gets:
  // tokens to keep, pages held and needed, new tokens (row0) and whether it is left alone (2) or
  // needs more pages than a row of the table has (1) (take0).
  int32_t bits = 0;
  Sums mine{0, 0, 0}, total;
  for (int b = b0; b < b1; ++b) {
    const int32_t old = __ldg(d.kv_old + b), n = __ldg(d.n_new + b), keep = d.kv_keep ? __ldg(d.kv_keep + b) : old;
    const bool bad = !list_ok || old < 0 || n < 0 || old > most || keep < 0 || keep > old;
    const int64_t want = static_cast<int64_t>(keep) + n;
    const bool wide = !bad && want > most;
    const int32_t held = bad ? 0 : pages(old), need = bad || wide ? held : pages(want);
    keep_of[b] = keep;
    held_of[b] = held;
    need_of[b] = need;
    row0[b] = n;
    take0[b] = bad ? 2 : wide ? 1 : 0;
    if (bad) bits |= MOE_DEV_BAD_INDEX;
    if (wide) bits |= MOE_DEV_OVERFLOW;
    // (too wide: more than there is, so that the sums tell)
    mine = mine + Sums{bad ? 0u : wide ? kMost : static_cast<uint32_t>(n), static_cast<uint32_t>(max(0, need - held)),
                       static_cast<uint32_t>(max(0, held - need))};
  }
  Sums before = block_scan(mine, part, total);
  const uint32_t room = add(f, total.back), all_rows_u = static_cast<uint32_t>(d.rows);
  if (list_ok && (total.n > all_rows_u || total.take > room)) {
    // not all get what they ask for: by rows first, then by pages among those that pass
    Sums asks{0, 0, 0}, sum;
    for (int b = b0; b < b1; ++b) asks.n = add(asks.n, take0[b] ? 0 : row0[b]);
    uint32_t n = block_scan(asks, part, sum).n;
    asks = Sums{0, 0, 0};
    for (int b = b0; b < b1; ++b)
      if (take0[b] == 0) {
        n = add(n, row0[b]);
        if (row0[b] > 0 && n > all_rows_u) take0[b] = 1;
        else asks.take = add(asks.take, max(0, need_of[b] - held_of[b]));
      }
    uint32_t take = block_scan(asks, part, sum).take;
    mine = Sums{0, 0, 0};
    for (int b = b0; b < b1; ++b) {
      if (take0[b] == 0 && need_of[b] > held_of[b]) {
        take = add(take, need_of[b] - held_of[b]);
        if (take > room) take0[b] = 1;
      }
      if (take0[b] == 1) {             // keeps what it keeps
        bits |= MOE_DEV_OVERFLOW;
        row0[b] = 0;
        need_of[b] = pages(keep_of[b]);
      }
      if (take0[b] != 2)
        mine = mine + Sums{static_cast<uint32_t>(row0[b]), static_cast<uint32_t>(max(0, need_of[b] - held_of[b])),
                           static_cast<uint32_t>(max(0, held_of[b] - need_of[b]))};
    }
    before = block_scan(mine, part, total);
  }
  // a list that would not hold what comes back: nothing moves
  const bool whole = list_ok && add(f, total.back) <= d.free_capacity;
  if (!whole) {
    bits |= MOE_DEV_BAD_INDEX;
    before = total = Sums{0, 0, 0};
  }
  for (int b = b0; b < b1; ++b) {
    const bool stays = !whole || take0[b] == 2;
    const int32_t n = stays ? 0 : row0[b], held = held_of[b], need = stays ? held : need_of[b];
    if (blockIdx.x == 0) {
      d.cu_new[b] = static_cast<int32_t>(before.n);
      d.kv_len[b] = stays ? __ldg(d.kv_old + b) : keep_of[b] + n;
    }
    row0[b] = static_cast<int32_t>(before.n);
    take0[b] = static_cast<int32_t>(before.take);
    back0[b] = static_cast<int32_t>(before.back);
    need_of[b] = need;
    before = before + Sums{static_cast<uint32_t>(n), static_cast<uint32_t>(max(0, need - held)), static_cast<uint32_t>(max(0, held - need))};
  }
  const int32_t rows = static_cast<int32_t>(total.n), taken = static_cast<int32_t>(total.take), back = static_cast<int32_t>(total.back);
  const int32_t left = f + back - taken;
  if (threadIdx.x == 0) {
    row0[B] = rows;
    take0[B] = taken;
    back0[B] = back;
    if (blockIdx.x == 0) {
      d.cu_new[B] = rows;
      *d.free_count_out = whole ? left : f;
    }
  }
  if (blockIdx.x == 0 && bits) set_err(d.err, bits);
  __syncthreads();

  const int32_t step = static_cast<int32_t>(gridDim.x) * kPagesThreads;
  const int32_t first = static_cast<int32_t>(blockIdx.x) * kPagesThreads + threadIdx.x;
  auto entry = [&](int b, int32_t j) { return d.page_table + b * d.table_ld + j; };
  // The i-th page given back, and the i-th page taken.  Read from the L2, as a precaution: other CTAs
  // write other words of these lines, while the next launch may be on an SM already (1024 prompts 9.4
  // -> 10 us).  The wait in front makes what was written before visible, and lengths and counts, which
  // share lines in the same way and are read through the L1, were never found as they had been.
  auto given = [&](int32_t i) {
    const int b = find_last(back0, B, i);
    return __ldcg(entry(b, need_of[b] + i - back0[b]));
  };
  auto source = [&](int32_t i) {
    const int32_t at = f + back - 1 - i;
    return at < f ? __ldcg(d.free_list + at) : given(at - f);
  };
  // page j of sequence b
  auto lookup = [&](int b, int32_t j) { return j < held_of[b] ? __ldcg(entry(b, j)) : source(take0[b] + j - held_of[b]); };
  for (int64_t i = first; i < taken; i += step) {
    const int b = find_last(take0, B, static_cast<int32_t>(i));
    *entry(b, held_of[b] + static_cast<int32_t>(i) - take0[b]) = source(static_cast<int32_t>(i));
  }
  for (int64_t i = first; i < static_cast<int64_t>(left) - f; i += step) d.free_list[f + i] = given(static_cast<int32_t>(i));
  if (d.seqs == nullptr && d.positions == nullptr && d.slots == nullptr) return;
  auto one_row = [&](int r, int b) {        // b: its sequence, -1 behind the last
    int32_t pos = -1;
    int64_t slot = -1;
    if (b >= 0) {
      pos = keep_of[b] + r - row0[b];
      if (d.slots) slot = (static_cast<int64_t>(lookup(b, pos >> a.shift)) << a.shift) + (pos & (d.page_size - 1));
    }
    if (d.seqs) d.seqs[r] = b;
    if (d.positions) d.positions[r] = pos;
    if (d.slots) d.slots[r] = slot;
  };
  if (d.rows <= step) {                  // few rows, mostly a sequence each
    if (first < d.rows) one_row(first, first < rows ? find_last(row0, B, first) : -1);
    return;
  }
  // four rows a thread: the search for their sequence, and mostly the page, are shared
  const bool wide = ((reinterpret_cast<uintptr_t>(d.seqs) | reinterpret_cast<uintptr_t>(d.positions) | reinterpret_cast<uintptr_t>(d.slots)) & 15) == 0;
  const int all_rows = static_cast<int>(d.rows), in_page = d.page_size - 1;
  for (int64_t r64 = 4ll * first; r64 < all_rows; r64 += 4ll * step) {
    const int r0 = static_cast<int>(r64);
    int seq[4], pos[4];
    int64_t slot[4];
    int b = r0 < rows ? find_last(row0, B, r0) : 0, end = row0[b + 1], from = keep_of[b] - row0[b], page_of = -1, page = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = r0 + i;
      seq[i] = pos[i] = -1;
      slot[i] = -1;
      if (r < rows) {
        while (r >= end) {
          end = row0[++b + 1];
          from = keep_of[b] - row0[b];
          page_of = -1;
        }
        seq[i] = b;
        pos[i] = from + r;
        const int j = pos[i] >> a.shift;
        if (d.slots != nullptr && j != page_of) {
          page = lookup(b, j);
          page_of = j;
        }
        slot[i] = (static_cast<int64_t>(page) << a.shift) + (pos[i] & in_page);
      }
    }
    if (wide && r0 + 4 <= all_rows) {
      if (d.seqs) *reinterpret_cast<int4*>(d.seqs + r0) = make_int4(seq[0], seq[1], seq[2], seq[3]);
      if (d.positions) *reinterpret_cast<int4*>(d.positions + r0) = make_int4(pos[0], pos[1], pos[2], pos[3]);
      if (d.slots) {
        *reinterpret_cast<longlong2*>(d.slots + r0) = make_longlong2(slot[0], slot[1]);
        *reinterpret_cast<longlong2*>(d.slots + r0 + 2) = make_longlong2(slot[2], slot[3]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (r0 + i < all_rows) {
          if (d.seqs) d.seqs[r0 + i] = seq[i];
          if (d.positions) d.positions[r0 + i] = pos[i];
          if (d.slots) d.slots[r0 + i] = slot[i];
        }
    }
  }
}

// Six arrays of a sequence each, three of them with an entry more, and room for one more
// sequence, which is looked at (and not used) where there is none.
inline size_t pages_smem_bytes(int batch) { return sizeof(int32_t) * (6 * (static_cast<size_t>(batch) + 1) + 3); }

struct Range {
  const void* p;
  int64_t bytes;
};
inline bool overlap(const Range& a, const Range& b) { return memory_overlaps(a.p, a.bytes, b.p, b.bytes); }

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" int moe_kv_pages(const moe_kv_pages_desc* d, void* stream) {
  MOE_CHECK_ARG(d != nullptr && d->flags == 0);
  MOE_CHECK_ARG(d->batch >= 0 && d->max_pages >= 0 && d->rows >= 0 && d->free_capacity >= 0 && d->table_ld >= d->max_pages);
  if (d->page_size != 16 && d->page_size != 32 && d->page_size != 64 && d->page_size != 128) return MOE_ERR_UNSUPPORTED;
  if (d->batch > kPagesMaxBatch || d->max_pages > (INT32_MAX - 65535) / d->page_size || d->rows > (1 << 30) ||
      d->free_capacity > (1 << 30) || d->table_ld > INT32_MAX)
    return MOE_ERR_UNSUPPORTED;
  MOE_CHECK_ARG(d->free_count && d->free_count_out && d->cu_new && (d->free_list || d->free_capacity == 0));
  MOE_CHECK_ARG(d->batch == 0 || (d->kv_old && d->n_new && d->kv_len && (d->page_table || d->max_pages == 0)));
  const int64_t b4 = 4ll * d->batch;
  const Range in[4] = {{d->kv_old, b4}, {d->kv_keep, b4}, {d->n_new, b4}, {d->free_count, 4}};
  const Range out[8] = {{d->kv_len, b4}, {d->cu_new, b4 + 4}, {d->free_count_out, 4},
                        {d->page_table, d->batch ? 4 * ((d->batch - 1) * d->table_ld + d->max_pages) : 0},
                        {d->free_list, 4 * d->free_capacity}, {d->seqs, 4 * d->rows}, {d->positions, 4 * d->rows}, {d->slots, 8 * d->rows}};
  for (int i = 0; i < 8; ++i) {
    const uintptr_t unit = i == 7 ? 7 : 3;
    MOE_CHECK_ARG((reinterpret_cast<uintptr_t>(out[i].p) & unit) == 0);
    for (const Range& r : in) MOE_CHECK_ARG(!overlap(out[i], r) && (reinterpret_cast<uintptr_t>(r.p) & 3) == 0);
    for (int j = 0; j < i; ++j) MOE_CHECK_ARG(!overlap(out[i], out[j]));
  }
  if (int rc = check_device()) return rc;
  PagesArgs a{*d, 0};
  while ((1 << a.shift) < d->page_size) ++a.shift;
  // a CTA for every 512 rows, and for 16 sequences, whose pages may all go back
  const int64_t told = d->seqs || d->positions || d->slots ? d->rows : 0;
  const int64_t ctas = std::min<int64_t>(std::max<int64_t>({(told + kPagesThreads - 1) / kPagesThreads, (d->batch + 15) / 16, 1}),
                                         num_sms());
  const size_t smem = pages_smem_bytes(d->batch);
  if (smem > 48 * 1024)
    MOE_CUDA_TRY(cudaFuncSetAttribute(kv_pages_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                      static_cast<int>(pages_smem_bytes(kPagesMaxBatch))));
  return launch_pdl(kv_pages_kernel, dim3(static_cast<unsigned>(ctas)), dim3(kPagesThreads), smem, as_stream(stream), a);
}
