// Global gradient norm over many tensors, and clipping.
//
//   norm = sqrt(sum of squares over every element of every tensor)
//   out  = g min(1, max_norm / norm); a norm that is not finite (in fp32, as it is
//   handed out) leaves g as it is
//
// Bound by HBM: the norm needs every element before the first result can be
// written, so a clipped list is read twice and written once (300 tensors, 1.33
// GB into others: 709 us, 5.6 TB/s; the norm alone 1.07 GB in 188 us).  Squares are
// taken and summed in fp64 (fp32 squares of gradients over 1e19 or under
// 1e-19 would overflow or vanish), one partial sum per workgroup in a fixed
// partition, so the norm does not depend on the order in which workgroups run.
//
// Tensors are described by kernel arguments, kTable of them a launch: the
// caller's arrays are read on the host, nothing is copied to the device, and a
// captured graph keeps the description with its nodes.

#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>

#include "nvq.h"
#include "nvq_device.h"
#include "nvq_internal.h"

namespace nvq {
namespace {

constexpr int kTable = 128;      // tensors a launch: 3.6 KB of kernel arguments
constexpr int kThreads = 256;
// 16-byte vectors of one tensor that a workgroup takes at a time: four loads a
// thread.  1.07 GB in 300 tensors, clipped into others: 512 / 1024 / 2048 / 4096
// vectors 605 / 566 / 582 / 608 us.
constexpr int kChunk = 1024;
// Workgroups a launch at most, each with one partial sum: eight a CU, as many as
// fit (1024: 600 us, 4096: 566).
constexpr int kBlocks = 2048;
// So few partial sums (one table's) are added by every workgroup that scales,
// which saves a launch: 34 MB in 100 tensors 24 us instead of 26, 134 MB 68
// instead of 70.
constexpr int kSumParts = 2048;

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

struct Table {
  const void* in[kTable];
  void* out[kTable];
  int64_t numel[kTable];
  uint32_t first[kTable + 1];  // chunks before tensor i
  uint32_t bf16[kTable / 32];  // bit i: tensor i is bf16 (else fp32)
  int count;
  int backwards;               // the chunks of a tensor are numbered from its end
};

// One tensor as 16-byte vectors between two ragged ends.
struct Span {
  int64_t head, vecs;  // elements before the first vector; vectors
};
__host__ __device__ inline Span span_of(const void* p, int64_t numel, bool bf16) {
  const int size = bf16 ? 2 : 4;
  Span s;
  const int64_t off = (int64_t)((16 - ((uintptr_t)p & 15u)) & 15u) / size;
  s.head = off < numel ? off : numel;
  s.vecs = (numel - s.head) / (16 / size);
  return s;
}

struct Piece {  // what a workgroup has to do for one chunk
  int tensor;
  bool bf16;
  Span span;
  int64_t v0, v1;     // its vectors
  bool first, last;   // it also takes the elements before the first / after the last vector
};

__device__ __forceinline__ Piece piece_of(const Table& t, uint32_t chunk) {
  int lo = 0, hi = t.count;  // the last tensor whose first chunk is at or before this one
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (t.first[mid] <= chunk) lo = mid; else hi = mid;
  }
  Piece p;
  p.tensor = lo;
  p.bf16 = (t.bf16[lo >> 5] >> (lo & 31)) & 1u;
  p.span = span_of(t.in[lo], t.numel[lo], p.bf16);
  const int64_t c = t.backwards ? t.first[lo + 1] - 1 - chunk : chunk - t.first[lo];
  p.first = c == 0;
  p.last = c + 1 == t.first[lo + 1] - t.first[lo];
  p.v0 = c * kChunk;
  p.v1 = p.span.vecs < p.v0 + kChunk ? p.span.vecs : p.v0 + kChunk;
  return p;
}

__device__ __forceinline__ float element(const void* p, int64_t i, bool bf16) {
  return bf16 ? bf16_to_f32(static_cast<const uint16_t*>(p)[i]) : static_cast<const float*>(p)[i];
}

__device__ __forceinline__ void add_square(double& s, float v) { s = __builtin_fma((double)v, (double)v, s); }

__device__ __forceinline__ double block_sum(double v, double* s) {
#pragma unroll
  for (int m = 32; m > 0; m >>= 1) v += __shfl_xor(v, m, 64);
  if ((threadIdx.x & 63) == 0) s[threadIdx.x >> 6] = v;
  __syncthreads();
  return (s[0] + s[1]) + (s[2] + s[3]);
}

__global__ __launch_bounds__(kThreads) void k_square_sums(Table t, uint32_t chunks, double* part) {
  __shared__ double s[4];
  double sum = 0.0;
  for (uint32_t c = blockIdx.x; c < chunks; c += gridDim.x) {
    const Piece p = piece_of(t, c);
    const void* const in = t.in[p.tensor];
    const int size = p.bf16 ? 2 : 4;
    const uint4* const vec = reinterpret_cast<const uint4*>(static_cast<const char*>(in) + p.span.head * size);
    for (int64_t v = p.v0 + threadIdx.x; v < p.v1; v += kThreads) {
      const uint4 q = vec[v];
      const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (p.bf16) {
          add_square(sum, bf16_lo(w[j]));
          add_square(sum, bf16_hi(w[j]));
        } else {
          add_square(sum, __uint_as_float(w[j]));
        }
      }
    }
    if (p.first && threadIdx.x < p.span.head) add_square(sum, element(in, threadIdx.x, p.bf16));
    const int64_t tail = p.span.head + p.span.vecs * (16 / size);
    if (p.last && tail + threadIdx.x < t.numel[p.tensor]) add_square(sum, element(in, tail + threadIdx.x, p.bf16));
  }
  sum = block_sum(sum, s);
  if (threadIdx.x == 0) part[blockIdx.x] = sum;
}

// The sum of squares, in the same order wherever it is taken.
__device__ __forceinline__ double total_of(const double* part, int n) {
  __shared__ double s[4];
  double sum = 0.0;
#pragma unroll 4
  for (int i = threadIdx.x; i < n; i += kThreads) sum += part[i];
  return block_sum(sum, s);
}

// Whether the norm that the caller gets, in fp32, is a number: one past the
// largest is none, whatever fp64 still holds.
__device__ __forceinline__ bool finite_norm(double norm) { return __builtin_isfinite((float)norm); }

__device__ __forceinline__ float coef_of(double norm, float max_norm) {
  return finite_norm(norm) && norm > (double)max_norm ? (float)((double)max_norm / norm) : 1.0f;
}

__device__ __forceinline__ void report(double norm, float max_norm, float* out, float* coef, uint32_t* status) {
  *out = (float)norm;
  *coef = coef_of(norm, max_norm);
  *status = finite_norm(norm) ? 0u : (uint32_t)NVQ_STATUS_NONFINITE;
}

__global__ __launch_bounds__(kThreads) void k_norm(const double* part, int n, float max_norm, float* norm, float* coef,
                                                   uint32_t* status) {
  const double v = sqrt(total_of(part, n));
  if (threadIdx.x == 0) report(v, max_norm, norm, coef, status);
}

// kSum: every workgroup adds the (few) partial sums itself, and the first one
// reports; else the factor is in memory.  kPast: results go past the caches.
template <bool kSum, bool kPast>
__global__ __launch_bounds__(kThreads) void k_scale(Table t, uint32_t chunks, const double* part, int n, float max_norm,
                                                    float* norm, float* coef, uint32_t* status) {
  float c;
  if (kSum) {
    const double v = sqrt(total_of(part, n));
    c = coef_of(v, max_norm);
    if (blockIdx.x == 0 && threadIdx.x == 0) report(v, max_norm, norm, coef, status);
  } else {
    c = *coef;
  }
  const bool scaled = c != 1.0f;  // else bits are copied: a product would change a NaN's
  for (uint32_t k = blockIdx.x; k < chunks; k += gridDim.x) {
    const Piece p = piece_of(t, k);
    const void* const in = t.in[p.tensor];
    void* const out = t.out[p.tensor];
    if (in == out && !scaled) continue;  // nothing changes
    const int size = p.bf16 ? 2 : 4, per = 16 / size;
    const uint4* const vec = reinterpret_cast<const uint4*>(static_cast<const char*>(in) + p.span.head * size);
    char* const ov = static_cast<char*>(out) + p.span.head * size;
    const bool aligned = ((uintptr_t)ov & 15u) == 0;
    for (int64_t v = p.v0 + threadIdx.x; v < p.v1; v += kThreads) {
      const uint4 q = vec[v];
      uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
      for (int j = 0; j < 4 && scaled; ++j)
        w[j] = p.bf16 ? f32_to_bf16_any(bf16_lo(w[j]) * c) | (f32_to_bf16_any(bf16_hi(w[j]) * c) << 16)
                      : __float_as_uint(__uint_as_float(w[j]) * c);
      if (aligned) {
        u32x4* const o = reinterpret_cast<u32x4*>(ov) + v;
        const u32x4 r = {w[0], w[1], w[2], w[3]};
        if (kPast) __builtin_nontemporal_store(r, o);
        else *o = r;
      } else if (p.bf16) {
#pragma unroll
        for (int j = 0; j < 8; ++j) reinterpret_cast<uint16_t*>(ov)[8 * v + j] = (uint16_t)(w[j >> 1] >> (16 * (j & 1)));
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) reinterpret_cast<uint32_t*>(ov)[4 * v + j] = w[j];
      }
    }
    auto one = [&](int64_t i) {
      if (!scaled) {
        if (p.bf16) static_cast<uint16_t*>(out)[i] = static_cast<const uint16_t*>(in)[i];
        else static_cast<uint32_t*>(out)[i] = static_cast<const uint32_t*>(in)[i];
        return;
      }
      const float v = element(in, i, p.bf16) * c;
      if (p.bf16) static_cast<uint16_t*>(out)[i] = (uint16_t)f32_to_bf16_any(v);
      else static_cast<float*>(out)[i] = v;
    };
    if (p.first && threadIdx.x < p.span.head) one(threadIdx.x);
    const int64_t tail = p.span.head + p.span.vecs * per;
    if (p.last && tail + threadIdx.x < t.numel[p.tensor]) one(tail + threadIdx.x);
  }
}

int64_t chunks_of(const nvq_tensor_list* l, int64_t i) {
  if (l->numel[i] == 0) return 0;
  const Span s = span_of(l->data[i], l->numel[i], l->dtype[i] == NVQ_BF16);
  return std::max<int64_t>(1, (s.vecs + kChunk - 1) / kChunk);
}

// Walks the list in tables of up to kTable tensors (and 2^31 chunks), forwards
// or backwards; calls f(table, chunks) for each that has any element.
template <class F>
int each_table(const nvq_tensor_list* in, const nvq_tensor_list* out, bool backwards, F&& f) {
  Table t;
  t.backwards = backwards;
  int64_t done = 0;
  while (done < in->count) {
    t.count = 0;
    int64_t chunks = 0;
    for (uint32_t& b : t.bf16) b = 0u;
    for (; done < in->count && t.count < kTable; ++done) {
      const int64_t i = backwards ? in->count - 1 - done : done;
      const int64_t n = chunks_of(in, i);
      if (n == 0) continue;
      if (t.count > 0 && chunks + n > INT32_MAX) break;
      t.in[t.count] = in->data[i];
      t.out[t.count] = out ? out->data[i] : in->data[i];
      t.numel[t.count] = in->numel[i];
      t.first[t.count] = (uint32_t)chunks;
      if (in->dtype[i] == NVQ_BF16) t.bf16[t.count >> 5] |= 1u << (t.count & 31);
      chunks += n;
      ++t.count;
    }
    if (t.count == 0) continue;
    t.first[t.count] = (uint32_t)chunks;
    if (int rc = f(t, (uint32_t)chunks)) return rc;
  }
  return NVQ_OK;
}

int check_list(const nvq_tensor_list* l) {
  if (!l || l->struct_size < sizeof(nvq_tensor_list)) return NVQ_EINVAL;
  if (l->count < 0 || l->count > ((int64_t)1 << 20)) return NVQ_ESHAPE;
  if (l->count && (!l->data || !l->numel || !l->dtype)) return NVQ_EINVAL;
  for (int64_t i = 0; i < l->count; ++i) {
    if (l->dtype[i] != NVQ_F32 && l->dtype[i] != NVQ_BF16) return NVQ_EINVAL;
    if (l->numel[i] < 0 || l->numel[i] > ((int64_t)1 << 42)) return NVQ_ESHAPE;
    if (l->numel[i] && !l->data[i]) return NVQ_EINVAL;
    if ((uintptr_t)l->data[i] & (l->dtype[i] == NVQ_BF16 ? 1u : 3u)) return NVQ_EALIGN;
  }
  return NVQ_OK;
}

struct Extent {
  uintptr_t from, to;
  uint32_t number;  // of the tensor, twice, plus one where it is only read
  bool operator<(const Extent& o) const { return from != o.from ? from < o.from : number < o.number; }
};
// Memory in order of its addresses: each extent is held against the furthest end
// so far, of the written ones and, for a written one, of all.
struct Reach {
  uintptr_t written = 0, any = 0;
  bool meets(const Extent& e) {
    const bool w = (e.number & 1u) == 0, found = e.from < (w ? any : written);
    any = std::max(any, e.to);
    if (w) written = std::max(written, e.to);
    return found;
  }
};

bool ascending(const nvq_tensor_list* l) {
  uintptr_t at = 0;
  for (int64_t i = 0; i < l->count; ++i) {
    if (l->numel[i] == 0) continue;
    if ((uintptr_t)l->data[i] < at) return false;
    at = (uintptr_t)l->data[i];
  }
  return true;
}

// Whether a tensor that is written (of out; of in, if there is no out) lies over
// another tensor of the call.  out_i may be in_i.  Lists that ascend, as views of
// one buffer do, are merged.  Else the order is found on the stack (96 KB), without
// memory of the heap's: a list of more than kAtOnce extents is gone over several
// times, and each time gives the next ones in order, half of kAtOnce at least.
// Into others, ascending: 300 tensors 6 us, 20000 0.3 ms; in random order 18 us, 10
// ms (one sort in memory of the heap's 12 us, 3.5 ms).
bool overlaps(const nvq_tensor_list* in, const nvq_tensor_list* out) {
  constexpr int64_t kAtOnce = 4096;
  Extent next[kAtOnce];
  Extent last{0, 0, 0};  // the last of those before (no tensor is at 0)
  Reach reach;
  auto extent = [&](const nvq_tensor_list* l, int64_t i, uint32_t read) -> Extent {
    const uintptr_t from = (uintptr_t)l->data[i];
    return {from, from + (uintptr_t)l->numel[i] * (l->dtype[i] == NVQ_BF16 ? 2 : 4), (uint32_t)i << 1 | read};
  };
  if (!out) out = in;
  if (ascending(out) && ascending(in)) {
    for (int64_t i = 0, j = 0;;) {
      while (i < in->count && in->numel[i] == 0) ++i;
      while (j < in->count && (in->numel[j] == 0 || in->data[j] == out->data[j])) ++j;
      if (i == in->count && j == in->count) return false;
      const bool read = i == in->count || (j < in->count && (uintptr_t)in->data[j] < (uintptr_t)out->data[i]);
      if (reach.meets(read ? extent(in, j, 1) : extent(out, i, 0))) return true;
      ++(read ? j : i);
    }
  }
  for (;;) {
    int64_t n = 0;
    bool left = false;
    Extent end{~(uintptr_t)0, 0, 0};  // what is not before this one is left for later
    auto take = [&](const Extent& e) {
      if (!(last < e)) return;
      if (!(e < end)) {
        left = true;
        return;
      }
      if (n == kAtOnce) {
        n = kAtOnce / 2;
        std::nth_element(next, next + n, next + kAtOnce);
        end = next[n];
        left = true;
        if (!(e < end)) return;
      }
      next[n++] = e;
    };
    for (int64_t i = 0; i < in->count; ++i) {
      if (in->numel[i] == 0) continue;
      take(extent(out, i, 0));
      if (in->data[i] != out->data[i]) take(extent(in, i, 1));
    }
    std::sort(next, next + n);
    for (int64_t k = 0; k < n; ++k)
      if (reach.meets(next[k])) return true;
    if (!left) return false;
    last = next[n - 1];
  }
}

struct ClipLayout {
  float* coef;
  double* part;
  int64_t parts;
  size_t bytes;
};

ClipLayout clip_layout(void* ws, const nvq_tensor_list* l) {
  ClipLayout c;
  c.parts = 0;
  each_table(l, nullptr, false, [&](const Table&, uint32_t chunks) {
    c.parts += std::min<int64_t>(chunks, kBlocks);
    return NVQ_OK;
  });
  WsCarve w(ws);
  c.coef = w.take<float>(1);
  c.part = w.take<double>((size_t)std::max<int64_t>(1, c.parts));
  c.bytes = w.off;
  return c;
}

int norm_and_clip(const nvq_tensor_list* grads, const nvq_tensor_list* out, float max_norm, bool clip, float* norm, void* ws,
                  size_t ws_bytes, void* stream) {
  if (int rc = check_list(grads)) return rc;
  if (out) {
    if (int rc = check_list(out)) return rc;
    if (out->count != grads->count) return NVQ_ESHAPE;
    for (int64_t i = 0; i < grads->count; ++i) {
      if (out->numel[i] != grads->numel[i]) return NVQ_ESHAPE;
      if (out->dtype[i] != grads->dtype[i]) return NVQ_EINVAL;
    }
  }
  if (!norm || !(max_norm >= 0.0f)) return NVQ_EINVAL;
  if (clip && overlaps(grads, out)) return NVQ_EINVAL;
  if ((uintptr_t)norm & 3u) return NVQ_EALIGN;
  const ClipLayout L = clip_layout(ws, grads);
  if (!ws || ws_bytes < L.bytes) return NVQ_EWORKSPACE;
  if (!aligned256(ws)) return NVQ_EALIGN;
  hipStream_t s = static_cast<hipStream_t>(stream);
  double* part = L.part;
  if (int rc = each_table(grads, out, false, [&](const Table& t, uint32_t chunks) {
        const unsigned G = (unsigned)std::min<int64_t>(chunks, kBlocks);
        hipLaunchKernelGGL(k_square_sums, dim3(G), dim3(kThreads), 0, s, t, chunks, part);
        part += G;
        return last_launch();
      }))
    return rc;
  uint32_t* const status = WsCarve(ws).status();
  const int n = (int)L.parts;
  const bool sum = clip && n > 0 && n <= kSumParts;
  if (!sum) {
    hipLaunchKernelGGL(k_norm, dim3(1), dim3(kThreads), 0, s, L.part, n, max_norm, norm, L.coef, status);
    if (int rc = last_launch()) return rc;
  }
  if (!clip) return NVQ_OK;
  // Results beside their gradients that are more than the 256 MB of the
  // memory-side cache leave it to the gradients, which are read again: 1.3 GB
  // clipped in 721 us against 761; below that size the reader of the results
  // may find them there.
  int64_t bytes = 0;
  for (int64_t i = 0; i < grads->count; ++i) bytes += grads->numel[i] * (grads->dtype[i] == NVQ_BF16 ? 2 : 4);
  const bool past = out && bytes > ((int64_t)1 << 28);
  // from the end of the list to its start: what the norm read last is still in the cache
  return each_table(grads, out, true, [&](const Table& t, uint32_t chunks) {
    const dim3 G((unsigned)std::min<int64_t>(chunks, kBlocks));
    const auto scale = sum ? (past ? k_scale<true, true> : k_scale<true, false>) : past ? k_scale<false, true> : k_scale<false, false>;
    hipLaunchKernelGGL(scale, G, dim3(kThreads), 0, s, t, chunks, L.part, n, max_norm, norm,
                       L.coef, status);
    return last_launch();
  });
}

}  // namespace
}  // namespace nvq

using namespace nvq;

extern "C" size_t nvq_grad_norm_workspace_bytes(const nvq_tensor_list* grads) {
  return check_list(grads) ? kAlign : clip_layout(nullptr, grads).bytes;
}

extern "C" int nvq_grad_norm(const nvq_tensor_list* grads, float* norm, void* ws, size_t ws_bytes, void* stream) {
  return norm_and_clip(grads, nullptr, INFINITY, false, norm, ws, ws_bytes, stream);
}

extern "C" int nvq_clip_grad_norm(const nvq_tensor_list* grads, const nvq_tensor_list* out, float max_norm, float* norm,
                                  void* ws, size_t ws_bytes, void* stream) {
  return norm_and_clip(grads, out, max_norm, true, norm, ws, ws_bytes, stream);
}
