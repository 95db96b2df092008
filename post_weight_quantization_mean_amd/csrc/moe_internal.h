// Internal declarations of the mixture of experts (moe.hip, moe_api.cpp).
#pragma once

#include "a8_internal.h"

namespace awq {

constexpr int kMaxExperts = 1024, kMaxChosen = 32;
constexpr int kMoePairs = 2048;  // (token, expert) pairs of one pass at most: their list is kept on chip
constexpr int kRouteHere = 256;  // experts up to which the router may run inside the products' first kernel
constexpr int kSoftmax = 0, kSigmoid = 1;

struct RouteArgs {
  const void* logits;  // [M, E], ld
  int32_t* ids;        // [M, k]
  float* weights;      // [M, k]
  int64_t M, ld;
  int E, k, score;
  bool renorm;
};
hipError_t launch_moe_route(const RouteArgs& a, int l_type, hipStream_t st);

struct ExpertWeights {  // as awq_w4a8_weight leaves them, all experts' channels one after the other
  const uint32_t* codes;
  const uint32_t* steps;
  const float* powers;
};
struct MoeArgs {
  const void* x;         // [M, H], ldx
  const float* xscale;   // [M] for codes, else null
  const int32_t* ids;    // [M, k]
  const float* weights;  // [M, k]
  ExpertWeights up, down;
  void* y;               // [M, H], ldy
  uint16_t* h;           // [terms][pairs][I]: act(gate) * up as bf16 terms
  float* o;              // [pairs][H]: the weighted experts' results
  int64_t ldx, ldy;
  int M, k, E, H, I, act, terms;
  bool ybf16, by_pair;   // by_pair: slots are pairs, not experts
};
// Whether the products' first kernel makes the routing of M tokens itself.
bool moe_routes(int64_t M, int k, int E);
// r: the routing that it makes (where a.ids and a.weights point), or null where they are given
hipError_t launch_moe(const MoeArgs& a, const RouteArgs* r, int l_type, int x_type, hipStream_t st);

}  // namespace awq
