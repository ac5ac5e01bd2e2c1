// Internals shared by the linear-attention kernels.
#pragma once

#include "kv.h"

namespace rimuru {

// One call as the kernels see it.  S <- exp(g) S + k v^T, out = scale S^T q.
struct LinearArgs {
  const void *q, *k, *v;
  void* out;
  int64_t q_ts, q_hs, k_ts, k_hs, v_ts, v_hs, o_ts, o_hs;  // strides in elements
  const float* decay;
  int64_t g_ts, g_hs;
  float scale;
  int heads, per_key_head;  // heads, and how many of them share a query/key head
  int key_dim, value_dim;
  const int32_t* cu;  // row offsets [num_seqs + 1], or null: one row per sequence
  int num_seqs, num_tokens, max_new;
  const int32_t *state_in, *state_out;
  uint8_t* pool;
  uint64_t page_bytes;
  int num_pages;
  int* err;
  int sms;
};

// How the chunked form cuts a call: pieces of at most `piece` rows, cut where the row number is a
// multiple of it (0: sequences are left whole).
struct LinearCut {
  int piece = 0;
  int pieces = 0;            // of all sequences, empty ones included
  uint64_t state_bytes = 0;  // of the pieces' states, then of the sequences' first ones, then decays
};
LinearCut linear_cut(int heads, int key_dim, int value_dim, int sms, int num_seqs, int num_tokens, int max_new);
// New tokens of a sequence that the recurrent form still takes.  It costs 0.4 us a token where
// every SM has at most one state of 128 x 128, and as much for each state of an SM beyond; the
// chunked form costs 11 us, and 5 us for each further state of an SM, at any number of tokens up
// to 64.  32 heads: one sequence of 16 tokens 8.3 and 10.8 us, of 24 11.1 and 10.8; 8 sequences of
// 8 tokens 16.2 and 18.6, of 12 20.6 and 18.6; 64 of 4 58.7 and 72.6, of 8 90 and 73.  That is bf16; f16
// costs the same token by token and more in chunks, and changes over at the same numbers.
inline int steps_most(int heads, int key_dim, int value_dim, int sms, int num_seqs) {
  const double states = static_cast<double>(num_seqs) * heads * key_dim * value_dim / (128 * 128) / sms;
  return states <= 1 ? 16 : states <= 4 ? 10 : 5;
}

// Rows and pages of a sequence.  `ok` is false where the tables are bad (recorded by the
// thread that asks for it): the sequence is then left alone.
struct LinearSeq {
  int64_t row;
  int n;
  const float* in;  // state before the tokens, or null: zeros
  float* out;
  bool ok;
};
__device__ __forceinline__ LinearSeq linear_seq(const LinearArgs& a, int b, bool record) {
  LinearSeq s;
  const int r0 = a.cu ? a.cu[b] : b, r1 = a.cu ? a.cu[b + 1] : b + 1;
  const int in = a.state_in[b], out = a.state_out[b];
  s.row = r0;
  s.n = r1 - r0;
  const bool shape = r0 >= 0 && r1 >= r0 && r1 <= a.num_tokens && s.n <= a.max_new;
  const bool pages = in >= -1 && in < a.num_pages && out >= 0 && out < a.num_pages;
  s.ok = shape && pages;
  if (record && !s.ok) dev::set_error(a.err, shape ? RIMURU_DEV_BAD_PAGE : RIMURU_DEV_BAD_SHAPE);
  s.in = in >= 0 ? reinterpret_cast<const float*>(a.pool + static_cast<uint64_t>(in) * a.page_bytes) : nullptr;
  s.out = reinterpret_cast<float*>(a.pool + static_cast<uint64_t>(out) * a.page_bytes);
  return s;
}

cudaError_t launch_linear_steps(const LinearArgs& a, int dtype, cudaStream_t s);
// Makes its own message; returns a rimuru status.
int launch_linear_chunks(const LinearArgs& a, const LinearCut& cut, void* workspace, int dtype, cudaStream_t s);

}  // namespace rimuru
