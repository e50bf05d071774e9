// Internal declarations of the output head's losses (k_head.hip,
// k_head_rows.hip, sbl_head_api.hip).
#pragma once

#include "sbl_internal.h"

namespace sbl {
namespace head {

constexpr int kMaxTop = 256;              // listed teacher entries per token
constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.69314718055994530942f;

// device words at the start of a workspace
struct Header {
  int32_t count;                          // rows that take part
  float amax;                             // backward: largest |coefficient|; the stored logit gradient is
  float up;                               //   dz * up, up = kUp / amax (0 when amax is 0)
  float down;                             //   amax / kUp
};

// Logits over one range of the vocabulary, never stored: forward (softmax
// statistics and the listed logits) or backward (their gradient).
struct LogitsArgs {
  const uint16_t* h;                      // hidden states, rows of h_stride values
  int64_t h_stride;
  int64_t h_rows;                         // rows behind h (buffer bound)
  const int32_t* rows;                    // row of each taking-part token, or NULL (token i is row i)
  const Header* hdr;                      // its count, or NULL (m_tok rows)
  int32_t m_tok;                          // upper bound of the count
  const uint16_t* w;                      // head weights of this range
  int32_t n_vocab;                        // vocabulary entries of this range
  int32_t k;
  int32_t top;                            // listed entries per token
  float scale;                            // log2(e) / tau
  // forward
  const int64_t* index;                   // [row][top] listed ids of the original rows
  float* part_max;                        // [token][np] softmax statistics of 128 (or fewer) logits, base 2
  float* part_sum;
  int32_t np;
  float* zlist;                           // [token][top] scaled logits at the listed ids
  // backward
  int64_t v0;                             // first id of this range
  const float* lse2;                      // [token] lse * log2(e)
  const float* coef;                      // [token] softmax coefficient * up
  const int32_t* index32;                 // [token][top] id, or -1 (absent, or merged into an earlier entry)
  const float* sub;                       // [token][top] what to subtract at the id
  uint16_t* dz;                           // [token][ldz]
  int32_t ldz;
};

// dw[v][d] = down * sum_t dz[t][v] h[t][d] over one range of the vocabulary
struct WeightGradArgs {
  const uint16_t* dz;                     // [token][ldz]
  int32_t ldz;
  const uint16_t* h;                      // [token][k], taking-part rows
  const Header* hdr;
  int32_t m_tok;
  int32_t n_vocab, k;                     // of this range
  uint16_t* dw;                           // [n_vocab][k]
};

// part[s][t][d] (+)= sum over the s-th share of this range's vocabulary of dz[t][v] w[v][d]
struct HiddenGradArgs {
  const uint16_t* dz;
  int32_t ldz;
  const uint16_t* w;                      // [n_vocab][k] of this range
  const Header* hdr;
  int32_t m_tok;
  int32_t n_vocab, k;
  int32_t splits, split_steps;            // steps of 64 ids per share
  float* part;                            // [splits][m_tok][k]
  int32_t add;                            // add to what earlier ranges left there
};

// One loss call's rows (k_head_rows.hip).  Cross entropy: target; distillation:
// index, teacher, top.
struct RowArgs {
  const int64_t* target;
  const int64_t* index;
  const float* teacher;
  int32_t top;
  float tau, inv_tau;
  int32_t m_tok;
  int64_t n_vocab;
  int32_t k;
  const uint16_t* h;
  int64_t h_stride;
  // workspace
  Header* hdr;
  int32_t* rows;                          // [m_tok] original row of token i
  int32_t* pos;                           // [m_tok] token of an original row, or -1
  uint8_t* flag;                          // [m_tok] distillation: row takes part
  // forward
  const float* part_max;
  const float* part_sum;
  int32_t np;
  const float* zlist;
  float* loss;
  float* lse;
  // backward
  const float* lse_in;
  const float* dloss;
  const float* dlse;                      // nullable
  float up;                               // the type's kUp
  float* lse2;
  float* coef;
  int32_t* index32;
  float* sub;
  uint16_t* hc;                           // [token][k] copy of the taking-part rows
  uint16_t* dh;                           // nullable: rows that are taken out are zeroed
};

int64_t logits_tiles(int32_t m_tok, int32_t n_vocab);     // np of a forward call
hipError_t launch_logits(const LogitsArgs& a, bool fp16, bool backward, hipStream_t s);
hipError_t launch_weight_grad(const WeightGradArgs& a, bool fp16, hipStream_t s);
int hidden_splits(int32_t m_tok, int32_t n_vocab, int32_t k);
hipError_t launch_hidden_grad(const HiddenGradArgs& a, bool fp16, hipStream_t s);
// dh[rows[t]] = down * sum_s part[s][t]
hipError_t launch_hidden_final(const float* part, int splits, const Header* hdr, const int32_t* rows, int32_t m_tok,
                               int32_t k, uint16_t* dh, bool fp16, hipStream_t s);

// which rows take part (strict: ids past the vocabulary take their row out,
// as the backward needs); backward: also the header's scales
hipError_t launch_rows(const RowArgs& a, bool backward, hipStream_t s);
hipError_t launch_finish(const RowArgs& a, bool compact, hipStream_t s);
hipError_t launch_gather(const RowArgs& a, hipStream_t s);

}  // namespace head
}  // namespace sbl
