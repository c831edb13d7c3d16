// verify.cuh - verification of drafted tokens (declarations).
#pragma once

#include "common.cuh"

namespace smol {

// A token that stays, and its mass.
struct VerifyToken {
  unsigned long long mass;
  int x, pad;
};
constexpr int kVerifyList = 256;   // tokens of a row's list

// What the choice needs of one target row.
struct VerifyRow {
  unsigned long long z;        // mass of the tokens that stay (0: no distribution)
  unsigned long long mx;       // mass of the drafted token, 0 if it does not stay
  float lmax;
  unsigned vcut;               // order key: values above stay, and of this one
  int xcut;                    //   the tokens with index <= xcut
  int argmax;
  int listed;                  // tokens that stay, all in the row's list; -1: no list
  int pad[3];
};

struct VerifyParams {
  const uint16_t *logits;      // bf16, row b * (T + 1) + i at ld elements a row
  long long ld;
  const int *drafts;           // [B, T]
  const int *n_draft;          // [B] or nullptr
  const float *probs;          // or nullptr: row b * T + i at ldq elements a row
  long long ldq;
  int B, T, V;
  float temperature, top_p;
  float c_hi, c_lo;            // log2(e) / temperature as a sum of two floats
  int top_k, greedy;
  const float *uniform;        // [B, T + 1]
  int *n_accepted, *next;      // [B]
  float *p_draft;              // [B, T] or nullptr
  VerifyRow *rows;             // [B, T + 1], workspace
  VerifyToken *lists;          // [B, T + 1][kVerifyList], workspace
  int *status;
};
cudaError_t launch_verify(const VerifyParams &p, int sms, cudaStream_t st, int *launches);

}  // namespace smol
