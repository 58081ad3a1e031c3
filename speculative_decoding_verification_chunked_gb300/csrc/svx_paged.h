// Internal interface of the paged-cache operators: head norms with rotation (svx_heads.cu), one-token
// attention (svx_decode.cu) and eviction (svx_evict.cu).  Not part of the C ABI.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <initializer_list>

#include "svx.h"
#include "svx_internal.h"

namespace svx {

// Status-word bit (beside kErrBounds of the checked build): a length, slot or page id read on the device
// lies outside its bounds.  What it names was clamped or left out; nothing outside the buffers is touched.
constexpr int kErrInput = 8;

// Sites of the bounds-checked build, after those of svx_internal.h: rows of heads, and rows of K and V pages.
enum PagedSite : int {
  kSiteHeadsIn = 9,
  kSiteHeadsOut = 10,
  kSitePool = 11,
};

// K and V pages as the kernels see them: element (page, slot, head, 0) of either pool is at
// page * page_stride + slot * tok_stride + head * head_stride elements.
struct PageView {
  void* k;
  void* v;
  const int32_t* table;  // [n_req][max_pages]
  int* status;
  int64_t page_stride, tok_stride, head_stride;
  int64_t extent;        // elements from the first to one past the last (checked build)
  int32_t n_pages, page_size, max_pages, n_kv_heads;
  int32_t n_req;
  int32_t cap;           // max_pages * page_size: slots of a request
  uint32_t div_mul, div_shift;  // t / page_size = (t + mulhi(t, div_mul)) >> div_shift for t < 2^31
};

// Page of a request's slot (an index into its row of the table).
__device__ __forceinline__ uint32_t page_of(const PageView& p, uint32_t t) {
  return (t + __umulhi(t, p.div_mul)) >> p.div_shift;
}

// Page and offset of a request's slot, 0 <= slot < cap: the element offset of (slot, head 0), or -1 where
// the table names no page of the pool.
__device__ __forceinline__ int64_t slot_offset(const PageView& p, int32_t page_id, uint32_t in_page) {
  if (static_cast<uint32_t>(page_id) >= static_cast<uint32_t>(p.n_pages)) return -1;
  return static_cast<int64_t>(page_id) * p.page_stride + static_cast<int64_t>(in_page) * p.tok_stride;
}

// svx_debug_clip_paged: the most elements that this thread's calls describe a buffer of a kind as holding.
enum PagedBuffer : int { kClipInputs = 0, kClipOutputs = 1, kClipPool = 2, kClips = 3 };
int64_t clipped(PagedBuffer kind, int64_t extent);

// Host side, shared by the entry points (svx_paged.cu).
svx_status paged_fail(svx_status st, const char* fmt, ...);
// Checks a svx_pages and fills the view (with n_req rows in the table).  SVX_OK or the failure reported.
svx_status paged_view(const svx_pages* c, int32_t n_req, PageView* out);
// For calls that write the pools: true if two slots' rows share memory, of one pool (strides that fold onto each other) or of
// K and V; same_pool_too: also if K and V are one buffer.  The pools may be interleaved.
bool pools_collide(const svx_pages* c, bool same_pool_too);
// True for device (or managed) memory of `device`.
bool on_device(const void* p, int device);
inline bool is_aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
// True if no pointer is off the 4-byte grid of its int32 or fp32 elements (NULL: none).
inline bool words_aligned(std::initializer_list<const void*> ptrs) {
  for (const void* p : ptrs)
    if (!is_aligned(p, 4)) return false;
  return true;
}
int sm_count(int device);
// A buffer of a call; p NULL: none.
struct Span {
  const void* p;
  size_t bytes;
};
// True if a written buffer meets another written one or one that is read.
inline bool any_overlap(std::initializer_list<Span> written, std::initializer_list<Span> read) {
  auto meet = [](const Span& a, const Span& b) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
    return x && y && x < y + b.bytes && y < x + a.bytes;
  };
  for (const Span* w = written.begin(); w != written.end(); ++w) {
    for (const Span* o = w + 1; o != written.end(); ++o)
      if (meet(*w, *o)) return true;
    for (const Span& r : read)
      if (meet(*w, r)) return true;
  }
  return false;
}

// Makes `device` current for the entry point's duration.
struct PagedDevice {
  int prev = -1;
  bool ok = false;
  explicit PagedDevice(int dev) {
    if (cudaGetDevice(&prev) != cudaSuccess) {
      cudaGetLastError();
      return;
    }
    ok = prev == dev || cudaSetDevice(dev) == cudaSuccess;
    if (!ok) cudaGetLastError();
    target = dev;
  }
  ~PagedDevice() {
    if (ok && prev != target) cudaSetDevice(prev);
  }
  int target = -1;
};

}  // namespace svx
