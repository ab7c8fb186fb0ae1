// Accepted drafts moved to the front of the drafted ones, in place, in every
// layer (sm_103a).
//
// Request b has l_b cached tokens, the last n_b drafted in this step, of which
// a_0 < a_1 < ... are accepted: slot c_b + i takes the K and V rows of slot c_b
// + a_i (c_b = l_b - n_b).  a_i >= i, so a row is read before its slot is
// written when i goes up; from the first a_i != i on every row moves.
//
// A block moves the rows of one request in one layer: a thread holds a 16-byte
// column of the tokens' rows (256 of them for 8 heads of 128 bf16 values) and
// walks the accepted tokens, kAhead loads ahead of their stores, so nothing but
// its own column is ever at stake and no barrier is needed.  The slots are
// looked up once per block.  What bounds it is the chain of look-ups before the
// first row (about 3 us), then memory: 64 requests x 32 layers, 85 MB read and
// written, 16.0 us, 5.3 TB/s (6.5 behind the look-ups); 2.7 us for one request.  Two
// and four layers a block took 16.4 and 17.1 (3.2 and 4.3 for one request), 128 and 512 threads 16.9 and 22.2, 4 and 16
// loads ahead 17.7 and 23.0; loads and stores that leave no line behind gave 0.6.
#include <cuda_runtime.h>
#include <stdint.h>

#include "pkd_internal.h"
#include "step.h"
#include "sm103_ptx.cuh"

namespace pkd {
namespace {

using namespace dev;

constexpr int kThreads = 256;
constexpr int kAhead = 8;

__global__ void __launch_bounds__(kThreads) accept_kernel(const __grid_constant__ AcceptArgs a) {
  __shared__ int64_t from[kMaxAccepted], to[kMaxAccepted];   // slots in bytes
  __shared__ int count, first;   // accepted tokens, the first that moves
  const int b = blockIdx.x, layer = blockIdx.y;
  pdl_wait();
  const int p0 = a.indptr[b], p1 = a.indptr[b + 1], last = a.last[b], drafted = a.drafted[b];
  const int64_t len = (int64_t)a.page_size * ((int64_t)p1 - p0 - 1) + last;
  bool good = p0 >= 0 && p1 > p0 && p1 <= a.num_indices && last >= 1 && last <= a.page_size &&
              drafted >= 0 && drafted <= len;
  if (threadIdx.x == 0) count = first = a.width;
  __syncthreads();
  const int32_t* path = a.accepted + (int64_t)b * a.width;
  for (int i = threadIdx.x; i < a.width; i += kThreads) {
    const int x = path[i];
    if (x < 0) atomicMin(&count, i);
    if (x != i) atomicMin(&first, i);
  }
  __syncthreads();
  const int n = count;
  for (int i = threadIdx.x; i < n && good; i += kThreads) {
    const int x = path[i];
    // (x < i cannot be where all before it increase, and keeps the slots in the table here)
    if (x >= drafted || x < i || (i > 0 && path[i - 1] >= x)) {
      good = false;
      break;
    }
    const int64_t src = len - drafted + x, dst = len - drafted + i;
    const int ps = a.indices[p0 + src / a.page_size], pd = a.indices[p0 + dst / a.page_size];
    good = ps >= 0 && ps < a.num_pages && pd >= 0 && pd < a.num_pages;
    from[i] = ps * a.page_bytes + src % a.page_size * a.token_bytes;
    to[i] = pd * a.page_bytes + dst % a.page_size * a.token_bytes;
  }
  if (__syncthreads_or(!good)) {   // the request stays as it is
    if (threadIdx.x == 0 && layer == 0 && a.err != nullptr) atomicOr(a.err, PKD_DEV_ERR_BOUNDS);
    return;
  }
  uint8_t* kv = static_cast<uint8_t*>(a.kv[layer]);
  const int row = a.hkv * a.pieces;
  for (int col = threadIdx.x; col < 2 * row; col += kThreads) {
    const int in = col % row;
    uint8_t* base = kv + (col >= row ? a.v_bytes : 0) + in / a.pieces * a.head_bytes + in % a.pieces * 16;
    for (int i = first; i < n; i += kAhead) {
      uint4 x[kAhead];
#pragma unroll
      for (int u = 0; u < kAhead; ++u)
        if (i + u < n) x[u] = __ldcs(reinterpret_cast<const uint4*>(base + from[i + u]));
#pragma unroll
      for (int u = 0; u < kAhead; ++u)
        if (i + u < n) __stcs(reinterpret_cast<uint4*>(base + to[i + u]), x[u]);
    }
  }
}

}  // namespace

cudaError_t launch_accept(const AcceptArgs& a, int layers, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)a.batch, (unsigned)layers);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, accept_kernel, a);
}

}  // namespace pkd
