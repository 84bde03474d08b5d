// grad_clip.hip -- the global norm of many gradients and their clipping on
// gfx950.
//
//   total = sqrt(sum over all tensors of sum g^2),  c = min(1, max_norm /
//   (total + 1e-6)),  out = rn(c g)
//
// Bound by HBM: the norm reads every gradient once; clipping reads it again
// (the factor depends on all of them) and writes it.  The tensors are cut into
// chunks of one size, and workgroups walk the chunks of all tensors, so that
// the work is even whatever the tensors' sizes.  The table of tensors travels
// in the kernel's arguments: nothing is copied to the device or kept for a
// later call, and a captured graph holds its own.
#include <new>

#include <algorithm>

#include "block_common.hpp"

namespace swb {

constexpr int kTensors = 128;      // of one launch: 29 bytes each within 4 KB of arguments
constexpr int kNormGroups = 1024;  // workgroups of one launch, each with one partial sum

struct Table {
  const void* in[kTensors];
  void* out[kTensors];
  int64_t n[kTensors];
  int first[kTensors + 1];  // tensor i has chunks first[i] .. first[i + 1] - 1
  uint8_t type[kTensors];
  int count, chunk;  // tensors; elements of a chunk
};

// the tensor of chunk c: the last one whose first chunk is not past c.  Every
// lane looks at two entries; empty tensors are never the last such one.
__device__ __forceinline__ int tensor_of(const Table& t, int c) {
  const int lane = threadIdx.x & 63;
  const bool a = lane < t.count && t.first[lane] <= c;
  const bool b = lane + 64 < t.count && t.first[lane + 64] <= c;
  return __popcll(__ballot(a)) + __popcll(__ballot(b)) - 1;
}

template <class T>
__device__ __forceinline__ double square_sum(const T* p, int n) {
  constexpr int VEC = Vec<T>::N, U = 4;
  const int nvec = n / VEC;
  double s[2] = {0.0, 0.0};
  for (int v0 = threadIdx.x; v0 < nvec; v0 += 256 * U) {
    typename Vec<T>::type r[U];
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (v0 + 256 * u < nvec) r[u] = load_vec(p + (int64_t)(v0 + 256 * u) * VEC);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (v0 + 256 * u < nvec) {
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          const double g = (double)(float)r[u][e];
          s[e & 1] = __builtin_fma(g, g, s[e & 1]);
        }
      }
    }
  }
  const int tail = nvec * VEC + (int)threadIdx.x;
  if (tail < n) {
    const double g = (double)(float)p[tail];
    s[0] = __builtin_fma(g, g, s[0]);
  }
  return s[0] + s[1];
}

__device__ __forceinline__ double group_sum(double v, double* red) {
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) v += __shfl_xor(v, d, 64);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
  __syncthreads();
  return (red[0] + red[1]) + (red[2] + red[3]);
}

// part[blockIdx.x] = this workgroup's share of the sum of squares, in 64 bits:
// no finite gradient overflows it, and a long sum loses nothing.
__global__ void __launch_bounds__(256) grad_norm_kernel(const Table t, double* __restrict__ part) {
  __shared__ double red[4];
  const int total = t.first[t.count];
  double s = 0.0;
  for (int c = blockIdx.x; c < total; c += gridDim.x) {
    const int i = __builtin_amdgcn_readfirstlane(tensor_of(t, c));
    const int64_t at = (int64_t)(c - t.first[i]) * t.chunk;
    const int64_t left = t.n[i] - at;
    const int n = (int)(left < t.chunk ? left : t.chunk);
    const int type = t.type[i];
    if (type == SWIGLU_FP32) s += square_sum((const float*)t.in[i] + at, n);
    else if (type == SWIGLU_BF16) s += square_sum((const bf16_t*)t.in[i] + at, n);
    else s += square_sum((const fp16_t*)t.in[i] + at, n);
  }
  s = group_sum(s, red);
  if (threadIdx.x == 0) part[blockIdx.x] = s;
}

// total and the factor from the parts, added in a fixed order
__global__ void __launch_bounds__(256) grad_total_kernel(const double* __restrict__ part, int parts, double max_norm,
                                                         float* total, float* factor) {
  __shared__ double red[4];
  double s = 0.0;
  for (int p = threadIdx.x; p < parts; p += 256) s += part[p];
  s = group_sum(s, red);
  if (threadIdx.x == 0) {
    const double norm = __builtin_sqrt(s), q = max_norm / (norm + 1e-6);
    *total = (float)norm;
    *factor = q < 1.0 || q != q ? (float)q : 1.0f;
  }
}

template <class T>
__device__ __forceinline__ void scale(const T* p, T* o, int n, float f) {
  constexpr int VEC = Vec<T>::N, U = 4;
  const int nvec = n / VEC;
  for (int v0 = threadIdx.x; v0 < nvec; v0 += 256 * U) {
    typename Vec<T>::type r[U];
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (v0 + 256 * u < nvec) r[u] = load_vec(p + (int64_t)(v0 + 256 * u) * VEC);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (v0 + 256 * u < nvec) {
#pragma unroll
        for (int e = 0; e < VEC; ++e) r[u][e] = (T)((float)r[u][e] * f);
        stream_vec(o + (int64_t)(v0 + 256 * u) * VEC, r[u]);
      }
    }
  }
  const int tail = nvec * VEC + (int)threadIdx.x;
  if (tail < n) o[tail] = (T)((float)p[tail] * f);
}

// The chunks from the last to the first: the end of the gradients, which the
// norm read last, is still in the last-level cache.
__global__ void __launch_bounds__(256) grad_scale_kernel(const Table t, const float* __restrict__ factor) {
  const float f = *factor;
  const int total = t.first[t.count];
  for (int c = total - 1 - (int)blockIdx.x; c >= 0; c -= gridDim.x) {
    const int i = __builtin_amdgcn_readfirstlane(tensor_of(t, c));
    if (f == 1.0f && t.in[i] == t.out[i]) continue;  // in place and unchanged
    const int64_t at = (int64_t)(c - t.first[i]) * t.chunk;
    const int64_t left = t.n[i] - at;
    const int n = (int)(left < t.chunk ? left : t.chunk);
    const int type = t.type[i];
    if (type == SWIGLU_FP32) scale((const float*)t.in[i] + at, (float*)t.out[i] + at, n, f);
    else if (type == SWIGLU_BF16) scale((const bf16_t*)t.in[i] + at, (bf16_t*)t.out[i] + at, n, f);
    else scale((const fp16_t*)t.in[i] + at, (fp16_t*)t.out[i] + at, n, f);
  }
}

}  // namespace swb

// ===========================================================================
// Host side
// ===========================================================================
namespace {

using namespace swb;

constexpr int64_t kMaxElements = (int64_t)1 << 40;  // of one tensor
constexpr int64_t kMaxTensors = (int64_t)1 << 20;

int64_t launches(int64_t n) { return (n + kTensors - 1) / kTensors; }

struct Span {
  uintptr_t lo, hi;
  bool out;
};

// Outputs must not overlap one another or an input; inputs may overlap inputs.
// Sorted by start, a span conflicts if it starts before the end of an earlier
// output, or is an output and starts before the end of anything earlier.
int check_spans(Span* s, int64_t n) {
  std::sort(s, s + n, [](const Span& a, const Span& b) { return a.lo < b.lo; });
  uintptr_t any = 0, outs = 0;
  for (int64_t i = 0; i < n; ++i) {
    if (s[i].hi == s[i].lo) continue;
    if (s[i].lo < outs || (s[i].out && s[i].lo < any)) return SWIGLU_ERR_ALIAS;
    if (s[i].hi > any) any = s[i].hi;
    if (s[i].out && s[i].hi > outs) outs = s[i].hi;
  }
  return SWIGLU_OK;
}

// Elements of a chunk: small enough that a few tensors still fill the chip,
// large enough that a workgroup's loop is long.
int chunk_of(int64_t total) {
  int64_t c = 2048;
  while (c < 65536 && total / c > 2048) c *= 2;
  return (int)c;
}

}  // namespace

extern "C" {

// a partial sum for every workgroup of every launch, then the factor
size_t swiglu_clip_grad_norm_workspace(int64_t n) {
  if (n < 0 || n > kMaxTensors) return 0;
  return (size_t)launches(n) * kNormGroups * sizeof(double) + 256;
}

int swiglu_clip_grad_norm(const void* const* grads, void* const* outs, const int64_t* numels, const int* dtypes,
                          int64_t n, double max_norm, float* total, void* ws, size_t ws_bytes, void* stream) {
  if (n < 0 || !(max_norm >= 0.0)) return SWIGLU_ERR_SHAPE;
  if (n > kMaxTensors) return SWIGLU_ERR_UNSUPPORTED;
  if (n > 0 && (!grads || !numels || !dtypes)) return SWIGLU_ERR_NULL;
  int64_t elements = 0;
  for (int64_t i = 0; i < n; ++i) {
    if (numels[i] < 0) return SWIGLU_ERR_SHAPE;
    if (numels[i] > kMaxElements || !dtype_ok(dtypes[i])) return SWIGLU_ERR_UNSUPPORTED;
    elements += numels[i];
  }
  if (elements > kMaxElements) return SWIGLU_ERR_UNSUPPORTED;
  const bool norm_only = max_norm == __builtin_inf();
  if (!total) return SWIGLU_ERR_NULL;
  for (int64_t i = 0; i < n; ++i) {
    if (numels[i] > 0 && (!grads[i] || (outs && !outs[i]))) return SWIGLU_ERR_NULL;
    if (norm_only && outs && numels[i] > 0 && outs[i] != grads[i]) return SWIGLU_ERR_UNSUPPORTED;
  }
  if (!aligned_to(total, 4) || !aligned_to(ws, 16)) return SWIGLU_ERR_ALIGN;
  for (int64_t i = 0; i < n; ++i) {
    const int es = elem_size(dtypes[i]);
    if (!aligned_to(grads[i], es) || (outs && !aligned_to(outs[i], es))) return SWIGLU_ERR_ALIGN;
  }
  const size_t need = swiglu_clip_grad_norm_workspace(n);
  if (!ws || ws_bytes < need) return SWIGLU_ERR_WORKSPACE;

  Span* spans = new (std::nothrow) Span[(size_t)(2 * n + 2)];
  if (!spans) return SWIGLU_ERR_HIP;
  int64_t ns = 0;
  for (int64_t i = 0; i < n; ++i) {
    const uintptr_t bytes = (uintptr_t)numels[i] * elem_size(dtypes[i]);
    const bool in_place = !outs || outs[i] == grads[i];
    spans[ns++] = {(uintptr_t)grads[i], (uintptr_t)grads[i] + bytes, in_place && !norm_only};
    if (!in_place) spans[ns++] = {(uintptr_t)outs[i], (uintptr_t)outs[i] + bytes, true};
  }
  spans[ns++] = {(uintptr_t)total, (uintptr_t)total + 4, true};
  spans[ns++] = {(uintptr_t)ws, (uintptr_t)ws + need, true};
  const int bad = check_spans(spans, ns);
  delete[] spans;
  if (bad != SWIGLU_OK) return bad;

  hipStream_t st = as_stream(stream);
  double* part = (double*)ws;
  float* factor = (float*)((char*)ws + need - 256);
  Table t;
  t.chunk = chunk_of(elements);
  const int64_t L = launches(n);
  auto fill = [&](int64_t l) {
    const int64_t i0 = l * kTensors;
    t.count = (int)(n - i0 < kTensors ? n - i0 : kTensors);
    int64_t c = 0;
    for (int k = 0; k < t.count; ++k) {
      t.in[k] = grads[i0 + k];
      t.out[k] = outs ? outs[i0 + k] : (void*)grads[i0 + k];
      t.n[k] = numels[i0 + k];
      t.type[k] = (uint8_t)dtypes[i0 + k];
      t.first[k] = (int)c;
      c += (numels[i0 + k] + t.chunk - 1) / t.chunk;  // at most 2^40 / 65536 + 128 in all
    }
    t.first[t.count] = (int)c;
    return (int)(c < kNormGroups ? c : kNormGroups);
  };
  int parts = 0;
  for (int64_t l = 0; l < L; ++l) {
    const int groups = fill(l);
    if (groups == 0) continue;
    hipLaunchKernelGGL(grad_norm_kernel, dim3((unsigned)groups), dim3(256), 0, st, t, part + parts);
    SW_TRY(launch_status());
    parts += groups;
  }
  hipLaunchKernelGGL(grad_total_kernel, dim3(1), dim3(256), 0, st, (const double*)part, parts, max_norm, total, factor);
  SW_TRY(launch_status());
  if (norm_only) return SWIGLU_OK;
  for (int64_t l = L - 1; l >= 0; --l) {
    const int groups = fill(l);
    if (groups == 0) continue;
    hipLaunchKernelGGL(grad_scale_kernel, dim3((unsigned)groups), dim3(256), 0, st, t, (const float*)factor);
    SW_TRY(launch_status());
  }
  return SWIGLU_OK;
}

}  // extern "C"
