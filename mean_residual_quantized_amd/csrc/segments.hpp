// Row segments (expert groups) and segment-aligned row chunks.
//
// A tensor's rows are split into nseg segments by a device array of offsets
// (nseg + 1 non-decreasing int64, first 0, last rows); offsets == nullptr
// means one segment of all rows.  Kernels cut each segment into chunks of
// `ch` rows so that no chunk straddles two segments; chunk c of the whole
// tensor maps to (segment, row range) through a prefix sum over the
// segments' chunk counts, computed by one wavefront.  Offsets outside
// [0, rows] are clamped and a decreasing pair counts as an empty segment, so
// malformed offsets never address memory outside the tensor.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace averis {

struct SegRange {
  int seg;          // segment index (-1: chunk past the end)
  int64_t r0, r1;   // row range [r0, r1) of this chunk (or segment)
  int64_t seg_r0, seg_r1;  // the whole segment's rows
  int64_t c0, c1;   // the segment's chunk index range
};

__device__ __forceinline__ int64_t clamp_row(int64_t v, int64_t rows) {
  return v < 0 ? 0 : (v > rows ? rows : v);
}

__device__ __forceinline__ void seg_bounds(const int64_t* offs, int s, int64_t rows, int64_t& a,
                                           int64_t& b) {
  a = clamp_row(offs[s], rows);
  b = clamp_row(offs[s + 1], rows);
  if (b < a) b = a;
}

// One segment of all rows (offsets == nullptr): the range in closed form.
__device__ __forceinline__ SegRange plain_range(int64_t rows, int64_t ch, int64_t key, int mode) {
  const int64_t n = (rows + ch - 1) / ch;
  SegRange r;
  r.seg = (mode == 1) ? (key == 0 ? 0 : -1) : (key < n ? 0 : -1);
  r.seg_r0 = 0;
  r.seg_r1 = rows;
  r.c0 = 0;
  r.c1 = n;
  r.r0 = mode == 1 ? 0 : key * ch;
  r.r1 = mode == 1 ? rows : (key * ch + ch < rows ? key * ch + ch : rows);
  return r;
}

// Wave-level scan.  Must be called by all 64 lanes of one wavefront; the lane
// that finds the answer writes it to *out.  mode 0: locate chunk `key`;
// mode 1: describe segment `key`.
__device__ inline void seg_scan(const int64_t* offs, int nseg, int64_t rows, int64_t ch,
                                int64_t key, int mode, SegRange* out) {
  const int lane = threadIdx.x & 63;
  if (offs == nullptr) {
    if (lane == 0) *out = plain_range(rows, ch, key, mode);
    return;
  }
  int64_t carry = 0;
  bool found = false;
  for (int base = 0; base < nseg; base += 64) {
    const int s = base + lane;
    int64_t a = 0, b = 0;
    if (s < nseg) seg_bounds(offs, s, rows, a, b);
    const int64_t n = (b - a + ch - 1) / ch;
    int64_t incl = n;
    for (int d = 1; d < 64; d <<= 1) {
      const int64_t t = __shfl_up(incl, d, 64);
      if (lane >= d) incl += t;
    }
    const int64_t excl = carry + incl - n;
    incl += carry;
    const bool hit = s < nseg && (mode == 1 ? (s == key) : (key >= excl && key < incl));
    if (hit) {
      SegRange r;
      r.seg = s;
      r.seg_r0 = a;
      r.seg_r1 = b;
      r.c0 = excl;
      r.c1 = incl;
      if (mode == 1) {
        r.r0 = a;
        r.r1 = b;
      } else {
        r.r0 = a + (key - excl) * ch;
        r.r1 = r.r0 + ch < b ? r.r0 + ch : b;
      }
      *out = r;
    }
    found = found || __any(hit);
    carry = __shfl(incl, 63, 64);
    if (found) break;
  }
  if (!found && lane == 0) {
    SegRange r;
    r.seg = -1;
    r.r0 = r.r1 = r.seg_r0 = r.seg_r1 = 0;
    r.c0 = r.c1 = 0;
    *out = r;
  }
}

// Block-level wrappers: every thread of the block gets the result (without
// offsets in closed form, with no block synchronization).
__device__ inline SegRange locate_chunk(const int64_t* offs, int nseg, int64_t rows, int64_t ch,
                                        int64_t chunk) {
  if (offs == nullptr) return plain_range(rows, ch, chunk, 0);
  __shared__ SegRange sr;
  if (threadIdx.x < 64) seg_scan(offs, nseg, rows, ch, chunk, 0, &sr);
  __syncthreads();
  SegRange r = sr;
  __syncthreads();
  return r;
}

__device__ inline SegRange describe_segment(const int64_t* offs, int nseg, int64_t rows,
                                            int64_t ch, int seg) {
  if (offs == nullptr) return plain_range(rows, ch, seg, 1);
  __shared__ SegRange sr;
  if (threadIdx.x < 64) seg_scan(offs, nseg, rows, ch, seg, 1, &sr);
  __syncthreads();
  SegRange r = sr;
  __syncthreads();
  return r;
}

// Chunks of the segments, 64 segments at a time, one a lane: the segment of a
// chunk (of `ch` rows) or a segment's chunks come from a ballot, with no LDS
// and no barrier.  Up to 64 segments are read once for a whole kernel.  Every
// wavefront keeps its own; all its lanes call.  Rows below 2^31.
struct SegTable {
  const int64_t* offs;
  int nseg, ch;
  int64_t rows;
  int base;       // first segment of the loaded 64
  int r0, r1;     // this lane's segment's rows
  int c0, c1;     // its chunks

  __device__ __forceinline__ void load(int b, int before) {
    const int lane = threadIdx.x & 63;
    base = b;
    int64_t a = 0, e = 0;
    if (b + lane < nseg) seg_bounds(offs, b + lane, rows, a, e);
    r0 = (int)a;
    r1 = (int)e;
    const int n = (r1 - r0 + ch - 1) / ch;
    int incl = n;
    for (int d = 1; d < 64; d <<= 1) {
      const int t = __shfl_up(incl, d, 64);
      if (lane >= d) incl += t;
    }
    c1 = before + incl;
    c0 = c1 - n;
  }
  __device__ __forceinline__ void init(const int64_t* o, int ns, int64_t r, int c) {
    offs = o;
    nseg = ns;
    rows = r;
    ch = c;
    load(0, 0);
  }
  // the next 64 segments (false past the last)
  __device__ __forceinline__ bool advance() {
    if (base + 64 >= nseg) return false;
    load(base + 64, __builtin_amdgcn_readlane(c1, 63));
    return true;
  }
  // rows [a, b) of chunk c and its segment; false past the last chunk
  __device__ __forceinline__ bool chunk(int c, int& seg, int& a, int& b) {
    if (c < (int)__builtin_amdgcn_readfirstlane(c0)) load(0, 0);
    do {
      const uint64_t hit = __ballot(c >= c0 && c < c1);
      if (hit) {
        const int l = __builtin_ctzll(hit);
        seg = base + l;
        a = (int)__builtin_amdgcn_readlane(r0, l) + (c - (int)__builtin_amdgcn_readlane(c0, l)) * ch;
        b = __builtin_amdgcn_readlane(r1, l);
        b = a + ch < b ? a + ch : b;
        return true;
      }
    } while (advance());
    return false;
  }
  // chunks of all segments
  __device__ __forceinline__ int count() {
    while (advance()) {}
    const int n = __builtin_amdgcn_readlane(c1, 63);
    if (base != 0) load(0, 0);
    return n;
  }
  // the segment that is number s when the 64 around it go by length, longest
  // first (lengths within a factor of two by index)
  __device__ __forceinline__ int by_length(int s) {
    while (base > s || s >= base + 64) {
      if (base > s) load(0, 0);
      else if (!advance()) break;
    }
    int left = s - base;
    const int n = c1 - c0, cls = n > 0 ? 32 - __builtin_clz(n) : 0;   // chunks below 2^24
    for (int k = 24; k > 0; --k) {
      const uint64_t of = __ballot(cls == k);
      const int many = __builtin_popcountll(of);
      if (left < many) return base + nth_bit(of, left);
      left -= many;
    }
    return base + nth_bit(__ballot(cls == 0), left);
  }
  // the place of set bit number i
  __device__ __forceinline__ int nth_bit(uint64_t bits, int i) {
    const int below = __builtin_amdgcn_mbcnt_hi((uint32_t)(bits >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)bits, 0));
    return __builtin_ctzll(__ballot(below == i && (bits >> (threadIdx.x & 63) & 1)));
  }
  // chunks [a, b) of a segment
  __device__ __forceinline__ void segment(int s, int& a, int& b) {
    if (s < base) load(0, 0);
    while (s >= base + 64 && advance()) {}
    a = __builtin_amdgcn_readlane(c0, (s - base) & 63);
    b = __builtin_amdgcn_readlane(c1, (s - base) & 63);
  }
};

// Upper bound on the total chunk count, known on the host.
static inline int64_t chunk_upper_bound(int64_t rows, int nseg, int64_t ch) {
  return (rows + ch - 1) / ch + (nseg > 1 ? nseg : 0);
}

}  // namespace averis
