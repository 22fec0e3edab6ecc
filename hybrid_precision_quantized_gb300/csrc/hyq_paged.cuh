// Shared by the paged cache's kernels: the pool as the kernels see it, launch
// declarations and the exponents of bounds and query codes.
#pragma once

#include "hyq_common.cuh"

// Device view of one layer of a pool.
struct PageView {
  uint8_t* pool;    // [n_pages][HKV][block bytes]
  uint8_t* bounds;  // [n_pages][HKV][HYQ_BOUND_BYTES]
  const int32_t* table;
  const int32_t* lens;
  int32_t* err;
  int32_t n_pages, n_seqs, max_blocks;
};

inline PageView hyq_page_view(const hyq_config* c, const hyq_pages* p, int32_t layer) {
  const size_t pages = (size_t)layer * p->n_pages * c->num_kv_heads;
  return PageView{p->pool + pages * hyq_qblock_bytes(c), p->bounds + pages * HYQ_BOUND_BYTES,
                  p->table, p->lens, p->err, p->n_pages, p->n_seqs, p->max_blocks};
}

inline size_t hyq_align256(size_t x) { return (x + 255) / 256 * 256; }

size_t hyq_paged_attention_ws_bytes(const hyq_config* c, int32_t batch, int32_t n_q);
cudaError_t hyq_launch_paged_attention(const hyq_config* c, const PageView& pv, const int32_t* seqs, int32_t batch,
                                       int32_t n_q, const void* q, int64_t ldq, const int32_t* sel, int32_t k_sel,
                                       void* out, void* ws, cudaStream_t s);
cudaError_t hyq_launch_paged_append(const hyq_config* c, const PageView& pv, const int32_t* seqs, int32_t batch,
                                    const int32_t* cu, int32_t n_rows, const void* k, const void* v, int64_t ld,
                                    void* k_hat, void* v_hat, cudaStream_t s);
size_t hyq_paged_select_ws_bytes(const hyq_config* c, const hyq_pages* p, int32_t batch, int32_t n_q);
cudaError_t hyq_launch_paged_select(const hyq_config* c, const PageView& pv, const int32_t* seqs, int32_t batch,
                                    int32_t n_q, const void* q, int64_t ldq, int32_t k, int32_t n_first,
                                    int32_t n_last, int32_t* sel, void* ws, cudaStream_t s);
size_t hyq_pages_reserve_ws_bytes(const hyq_pages* p);
cudaError_t hyq_launch_pages_reserve(const hyq_config* c, const hyq_pages* p, const int32_t* seqs, int32_t batch,
                                     const int32_t* n_new, void* ws, cudaStream_t s);
cudaError_t hyq_launch_pages_fork(const hyq_pages* p, const int32_t* src, const int32_t* dst, int32_t n,
                                  cudaStream_t s);
cudaError_t hyq_launch_pages_truncate(const hyq_pages* p, const int32_t* seqs, const int32_t* new_lens, int32_t n,
                                      cudaStream_t s);
size_t hyq_pages_compact_ws_bytes(const hyq_pages* p);
cudaError_t hyq_launch_pages_compact(const hyq_config* c, const hyq_pages* p, int32_t* table_out, int32_t* refs_out,
                                     void* ws, cudaStream_t s);

// Every kernel of the paged cache is launched as a programmatic dependent: it
// may be scheduled while the kernel before it on the stream still runs, and
// begins with chain_kernel(), which waits until all of that kernel's work is done
// and visible, before it reads or writes anything.  Only the launch overlaps (a
// kernel that lets its dependents go early; after any other kernel the order
// is the usual one).  It lets the next launch go only after its own wait, so that all
// kernels but the immediately preceding one have finished whenever a launch
// starts.  What an earlier kernel may have written is read by plain loads: one
// through the read-only path could be moved ahead of the wait.
template <class... Ks, class... As>
inline cudaError_t hyq_launch_chained(void (*k)(Ks...), dim3 grid, int threads, size_t smem, cudaStream_t s, As... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, k, args...);
}
__device__ __forceinline__ void chain_kernel() {
  asm volatile("griddepcontrol.wait;\n" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
}

// Sequence of call row i, or -1 when it is out of range.
__device__ __forceinline__ int32_t page_seq(const int32_t* seqs, int32_t i, int32_t n_seqs) {
  const int32_t s = seqs ? seqs[i] : i;
  return s >= 0 && s < n_seqs ? s : -1;
}

// Smallest integer e >= HYQ_BOUND_EXP_MIN with amax <= 127 * 2^e, for a
// finite amax >= 0: with amax = f 2^x, f in [1, 2), that is x - 6, or x - 5
// when f > 127/64.  (Zeros and subnormals lie far below the least exponent.)
__device__ __forceinline__ int bound_exp(float amax) {
  const int u = __float_as_int(amax);
  const int e = (u >> 23) - 127 - 6 + ((u & 0x7FFFFF) > 0x7E0000 ? 1 : 0);
  return e > HYQ_BOUND_EXP_MIN ? e : HYQ_BOUND_EXP_MIN;
}
// 2^k for -126 <= k <= 127.
__device__ __forceinline__ float pow2_int(int k) { return __int_as_float((k + 127) << 23); }
