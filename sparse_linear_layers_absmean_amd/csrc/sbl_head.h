// Internal declarations of the output head's losses (k_head.hip,
// k_head_rows.hip, sbl_api.hip).
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
  float amax;                             // backward: largest finite |coefficient| (scale_base); the stored logit
  float down;                             //   gradient is dz / down, down = amax / up (RowArgs)
};

// Factor that keeps the logit gradient (at most 2 in magnitude once divided by
// the largest coefficient) in the 16-bit type's range: with 2^14 FP16 keeps its
// 11 bits down to 2^-28 and is off by 2^-39 at most below; BF16 has FP32's range.
constexpr float kUpBf16 = 1.0f, kUpFp16 = 16384.0f;

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
  int32_t tile0;                          // first tile of this launch
  const uint16_t* near;                   // per row (forward: original) the 256-id blocks of its entries, 8 to a vector,
                                          //   ~0 where there is none; or NULL
  // forward
  const int64_t* index;                   // [row][top] listed ids of the original rows
  float2* part;                           // [token][np] softmax statistics of a tile's ids: max logit, sum of
                                          //   2^((z - max) scale)
  int32_t np;
  float* zlist;                           // [token][top] logits at the listed ids
  // backward
  int64_t v0;                             // first id of this range
  const float* lse2;                      // [token] lse * log2(e)
  const float* coef;                      // [token] softmax coefficient / down
  const int32_t* index32;                 // [token][top] id, or -1 (absent, or merged into an earlier entry)
  const float* sub;                       // [token][top] what to subtract at the id
  uint16_t* dz;                           // [n_vocab / 256, rounded up][dz_rows][256]
  int32_t dz_rows;
  int32_t half;                           // 0, or (few tokens) rows of dz: half for the tokens' gradients, as many again
                                          //   for what their rounding to 16 bits left
};

// dw[v][d] = down * sum_t dz[t][v] h[t][d] over one range of the vocabulary
struct WeightGradArgs {
  const uint16_t* dz;                     // as LogitsArgs leaves it
  const uint16_t* h;                      // [token][k], taking-part rows
  const Header* hdr;
  int32_t rows;                           // tokens, or 0: the header's count
  int32_t m_tok;
  int32_t n_vocab, k;                     // of this range
  uint16_t* dw;                           // [n_vocab][k]
};

// part[s][t][d] (+)= sum over the s-th share of this range's vocabulary of dz[t][v] w[v][d]
struct HiddenGradArgs {
  const uint16_t* dz;
  const uint16_t* w;                      // [n_vocab][k] of this range
  const Header* hdr;
  int32_t rows;                           // as above
  int32_t m_tok;
  int32_t n_vocab, k;
  int32_t splits, split_steps;            // steps of 64 ids per share
  int32_t range_steps;                    // steps of a whole range
  float* part;                            // [splits][m_tok][k], or as many rows
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
  uint16_t* near;                         // [m_tok][top, rounded up to 8], or NULL (LogitsArgs)
  // forward
  const float2* part;
  int32_t np;
  const float* zlist;
  float* loss;
  float* lse;
  // backward
  const float* lse_in;
  const float* dloss;
  const float* dlse;                      // nullable
  float up;                               // kUpBf16 or kUpFp16
  float* lse2;
  float* coef;
  int32_t* index32;
  float* sub;
  uint16_t* hc;                           // [token][k] copy of the taking-part rows; with `half`, 2 half rows: zeros after
                                          //   the last token, and all of it twice
  int32_t half;
  uint16_t* dh;                           // nullable: rows that are taken out are zeroed
};

// Up to this many tokens both gradients run in one launch of narrow tiles, bound
// by reading w and writing dw.  The products cost nothing then, so the logit
// gradients are carried in two 16-bit parts (16 or more bits of precision):
// the second half of 2 few_half(m_tok) rows holds what rounding left.
constexpr int kFewTokens = 64;
inline int few_half(int64_t m_tok) { return m_tok > kFewTokens ? 0 : m_tok <= 32 ? 32 : 64; }

int64_t logits_tiles(int32_t m_tok, int32_t n_vocab, int32_t k);     // np of a forward call
hipError_t launch_logits(const LogitsArgs& a, bool fp16, bool backward, hipStream_t s);
// How dh is split over a range of n_vocab ids: shares per tile; token_tile > 0: the
// shares are that many if all m_tok rows take part, more in proportion if fewer
// do (tiles of token_tile rows), worked out on the GPU where the count is known.
struct HiddenPlan {
  int splits, token_tile;
};
HiddenPlan hidden_plan(int32_t m_tok, int32_t n_vocab, int32_t k);
// both gradients of a range (either may be absent: dw or part NULL); `range`: ids of a whole range
hipError_t launch_grads(const WeightGradArgs& w, const HiddenGradArgs& h, int32_t m_tok, int32_t range, bool fp16,
                        hipStream_t s);
// dh[rows[t]] = down * sum_s part[s][t]
hipError_t launch_hidden_final(const float* part, const HiddenPlan& plan, int32_t range_steps, const Header* hdr,
                               const int32_t* rows, int32_t m_tok, int32_t k, uint16_t* dh, bool fp16, hipStream_t s);

// which rows take part (strict: ids past the vocabulary take their row out,
// as the backward needs); backward: also the header's scales
hipError_t launch_rows(const RowArgs& a, bool backward, hipStream_t s);
hipError_t launch_finish(const RowArgs& a, bool compact, hipStream_t s);
// backward, after launch_rows: coefficients, lists and hidden states of the rows that take part.  own_rows: in place
// of launch_rows as well (few rows and list entries: gather_alone), in the same launch
bool gather_alone(int32_t m_tok, int32_t top);
hipError_t launch_gather(const RowArgs& a, bool own_rows, hipStream_t s);

// out[0 .. values) = 0 (a multiple of 8 values, 16-byte aligned)
hipError_t launch_zero(uint16_t* out, int64_t values, hipStream_t s);

}  // namespace head
}  // namespace sbl
