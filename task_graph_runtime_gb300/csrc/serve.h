// Launch parameters and host entry points of the serving operators over the
// paged KV cache (append.cu, attend.cu, verify.cu): several new tokens a
// sequence, shared prefixes, drafted tokens.  The C ABI is in serve_api.cpp.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace mpk {

// Division of a non-negative 31-bit number by a fixed divisor.
struct FastDiv {
  uint32_t div, mul, shift;
};
inline FastDiv fast_div(uint32_t d) {
  uint32_t s = 0;
  while (s < 31 && (1u << s) < d) ++s;
  const uint64_t one = 1;
  return FastDiv{d, (uint32_t)(((one << 32) * ((one << s) - d)) / d + 1), s};
}

// A ragged batch of new tokens over one layer of the paged cache.
struct PagedArgs {
  uint16_t* k;                 // the layer's [num_pages][Hkv][page_size][d]
  uint16_t* v;
  const int32_t* page_table;   // [batch][max_pages]
  const int32_t* seq_lens;     // [batch] tokens cached before the new ones
  const int32_t* q_start;      // nullable [batch + 1]
  int tokens_per_seq;          // rows of a sequence when q_start is null
  int batch, n_tokens;
  int num_pages, page_size, max_pages;
  FastDiv page_div, grp_div;   // by page_size; by query heads per KV head
  int Hq, Hkv, d;
  uint32_t* status;            // nullable: first error found
};

struct AppendArgs {
  PagedArgs p;
  const uint16_t *q, *k, *v;   // rows of heads; strides in elements
  int64_t q_stride, k_stride, v_stride;
  const uint16_t *q_norm, *k_norm;
  float eps;
  const float* table;          // [n_pos][rot / 2][2]
  int n_pos, rot, interleaved;
  uint16_t* q_out;             // nullable
  int64_t q_out_stride;
};
cudaError_t launch_append(const AppendArgs& a, cudaStream_t s);

struct RopeTableArgs {
  float* out;
  int64_t first_pos;
  int n_pos, rot;
  int scaling;
  double theta, factor, low, high, old_ctx, attn_factor;
};
cudaError_t launch_rope_table(const RopeTableArgs& a, cudaStream_t s);

// Partial results of one launch over (row tile, KV head) units.
struct AttnSet {
  float* part;       // [slots][M][d]
  float2* ml;        // [slots][M]: running maximum (log2 domain) and sum
  int2* meta;        // per unit (at meta_of): first slot, number of segments
  int64_t units, slots;   // room in meta and in part
  int M, shift;      // rows of a tile: a power of two, and its logarithm
};

struct AttendArgs {
  PagedArgs p;
  const uint16_t* q;
  int64_t q_stride;
  const int32_t* group_start;  // [n_groups + 1]
  const int32_t* prefix_len;   // [n_groups]
  int n_groups;                // 0: no shared prefix
  float scale_log2;            // softmax scale * log2(e)
  uint16_t* out;
  int64_t out_stride;
  float* lse;                  // nullable [n_tokens][Hq]
  AttnSet own, pre;            // results of the sequences, of the groups
  int tc;                      // prefixes by the tensor-memory kernel
  int wmp, wmo;                // row tiles of attend_kernel: 16 x these, 8 for 0
  int box;                     // keys a TMA box takes; 0: no TMA
  CUtensorMap map_k, map_v;       // the layer's pools, if box > 0
};
int attend_ctas();
// the general kernel, one translation unit per head_dim
cudaError_t launch_attend_32(const AttendArgs& a, cudaStream_t s);
cudaError_t launch_attend_64(const AttendArgs& a, cudaStream_t s);
cudaError_t launch_attend_128(const AttendArgs& a, cudaStream_t s);
int attend_tc_ctas();
int attend_tc_rows();
int attend_box(const PagedArgs& p);
cudaError_t launch_attend_tc(const AttendArgs& a, cudaStream_t s);
// Workspace bytes, and the pointers of *a into it (base may be null).
size_t attend_workspace(AttendArgs* a, char* base);
cudaError_t launch_attend(AttendArgs& a, cudaStream_t s);

struct VerifyArgs {
  int batch, n_tokens, vocab, max_out;
  const int32_t* q_start;
  int tokens_per_seq;
  const int32_t* tokens;
  const float* logits;
  int64_t logits_stride;
  const float* draft;          // nullable
  int64_t draft_stride;
  int draft_is_logits;
  const float* temperature;    // nullable: 1
  const float* uniform;        // [n_tokens]
  const float* noise;          // [batch][noise_stride]
  int64_t noise_stride;
  int32_t* n_accepted;
  int32_t* out_tokens;         // [batch][max_out]
  float* logprobs;             // nullable [batch][max_out]
  int32_t* next_tokens;        // nullable [batch]
  const int32_t* seq_lens;     // nullable
  int32_t* seq_lens_out;
  uint32_t* status;
  // workspace
  float4* part;                // [2][n_tokens][slices]: target's, draft's
                               // maximum, sum, index of the maximum
  int slices;
  unsigned long long* race;    // [batch] packed (value, ~index)
  uint32_t* arrived;           // [batch]
};
size_t verify_workspace(VerifyArgs* a, char* base);
cudaError_t launch_verify(const VerifyArgs& a, cudaStream_t s);

}  // namespace mpk
