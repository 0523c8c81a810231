// Page operations of the pool: copies of pages (mkv_seq_copy), copy-on-write branches
// (mkv_seq_fork), rollback (mkv_seq_truncate), release (mkv_seq_free) and compaction of the slabs
// (mkv_pool_compact).  All are one kernel over two lists: pages to copy or to cut, and runs of
// block-table entries to copy or to unmap.
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include <cstring>

#include "device_util.cuh"
#include "mkv_internal.h"

namespace mkv {
namespace {

constexpr int kThreads = 256;
constexpr int kVecs = 4;                                // 16-byte vectors a thread holds at once
constexpr int kPieceBytes = kThreads * kVecs * 16;      // bytes of a page that one CTA copies

// CTAs [0, pages * pieces): piece (blockIdx.x % pieces) of page blockIdx.x / pieces; the rest: one
// run of table entries each.
template <class P>
__global__ void __launch_bounds__(kThreads) page_ops_kernel(const __grid_constant__ P p) {
  const int pages = p.pages * p.pieces;
  if (static_cast<int>(blockIdx.x) >= pages) {
    const RowMove r = p.row[blockIdx.x - pages];
    int32_t* dst = p.tables + r.dst;
    if (r.src < 0) {
      for (int i = threadIdx.x; i < r.count; i += kThreads) dst[i] = -1;
    } else {
      const int32_t* src = p.tables + r.src;
      for (int i = threadIdx.x; i < r.count; i += kThreads) dst[i] = src[i];
    }
    return;
  }
  const int page = blockIdx.x / p.pieces, piece = blockIdx.x % p.pieces;
  int lo = 0, hi = p.n_page - 1;  // the run that holds the page
  if (p.pages == p.n_page) lo = hi = page;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (p.page[mid].first <= page) lo = mid;
    else hi = mid - 1;
  }
  PageMove m = p.page[lo];
  m.src_slot += page - m.first;
  m.dst_slot += page - m.first;
  m.table_index += page - m.first;
  const bool tq3 = m.fmt == 1;
  const int64_t bytes = tq3 ? p.tq3_slot_bytes : p.fp8_slot_bytes;  // (BF16 pages: first slab)
  uint8_t* slab = tq3 ? p.tq3_slab : p.fp8_slab;
  const uint4* src = reinterpret_cast<const uint4*>(slab + m.src_slot * bytes);
  uint4* dst = reinterpret_cast<uint4*>(slab + m.dst_slot * bytes);
  // a cut page: rows (of a head's K and of its V) from m.kept on become zero
  const int row_bytes = m.fmt == 2 ? 2 * p.D : p.D;
  const int head_bytes = m.fmt == 2 ? 64 * p.D : 32 * p.D + 16;
  auto dropped = [&](int i) {
    const int off = (i * 16) % head_bytes;
    return off < 32 * row_bytes && (off / row_bytes) % kPageTokens >= m.kept;
  };
  const int n = static_cast<int>(bytes / 16), step = p.pieces * kThreads;
  const bool in_place = m.src_slot == m.dst_slot;
  for (int i0 = piece * kThreads + threadIdx.x; i0 < n; i0 += kVecs * step) {
    uint4 v[kVecs];
#pragma unroll
    for (int e = 0; e < kVecs; ++e)
      if (!in_place && i0 + e * step < n) v[e] = src[i0 + e * step];
#pragma unroll
    for (int e = 0; e < kVecs; ++e) {
      const int i = i0 + e * step;
      if (i >= n) continue;
      if (m.kept < kPageTokens && dropped(i)) dst[i] = make_uint4(0, 0, 0, 0);
      else if (!in_place) dst[i] = v[e];
    }
  }
  if (piece != 0 || in_place) return;
  const uint32_t tag = static_cast<uint32_t>(m.fmt) << kFmtShift;
  const int32_t entry = static_cast<int32_t>(tag | static_cast<uint32_t>(m.dst_slot));
  if (!m.shared) {
    if (threadIdx.x == 0) p.tables[m.table_index] = entry;
  } else {  // sequences that share a page hold it at the same logical page: one table column
    const int32_t old = static_cast<int32_t>(tag | static_cast<uint32_t>(m.src_slot));
    for (int r = threadIdx.x; r < p.max_seqs; r += kThreads) {
      int32_t* e = p.tables + static_cast<int64_t>(r) * p.max_pages + m.table_index;
      if (*e == old) *e = entry;
    }
  }
}

}  // namespace

cudaError_t launch_page_ops(PageOpParams& p, cudaStream_t s) {
  if (p.n_page + p.n_row <= 0) return cudaSuccess;
  const int64_t slot = p.fp8_slot_bytes > p.tq3_slot_bytes ? p.fp8_slot_bytes : p.tq3_slot_bytes;
  p.pieces = static_cast<int32_t>((slot + kPieceBytes - 1) / kPieceBytes);
  const unsigned grid = static_cast<unsigned>(p.pages * p.pieces + p.n_row);
  if (p.n_page <= kMoveFew && p.n_row <= kMoveFew) {
    PageOpFewParams f;
    std::memcpy(&f, &p, offsetof(PageOpFewParams, page));
    std::memcpy(f.page, p.page, p.n_page * sizeof(PageMove));
    std::memcpy(f.row, p.row, p.n_row * sizeof(RowMove));
    page_ops_kernel<<<grid, kThreads, 0, s>>>(f);
  } else {
    page_ops_kernel<<<grid, kThreads, 0, s>>>(p);
  }
  return cudaGetLastError();
}

}  // namespace mkv
