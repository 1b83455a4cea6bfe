// Internal launchers of the kernel-level operators around a prompt: rotary positions, prompt attention, block bookkeeping.
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>

#include "kv8.cuh"

namespace eagle {

struct RopeArgs {
  const void *q, *k;
  void *qo, *ko;
  long long ldq, ldk, ldqo, ldko;      // row strides in elements
  int R, nq, nkv, d, rot;
  const int* pos;
  const unsigned long long* turns;     // [rot / 2]: angle of a position, in 2^-64 of a turn
  float factor;
  bool inverse;
  int slices;                          // set by the launcher: warps a row
};
int rope_rows(cudaStream_t st, RopeArgs a, bool in_f32, bool out_f32, bool neighbours);

struct PromptArgs {
  const void *q, *k, *v;               // bf16, row strides ldq, ldk, ldv elements
  long long ldq, ldk, ldv, ldo;
  void* out;                           // bf16
  float* lse;                          // [R][nq], nullable
  int R, Rk, nq, nkv, d, B;
  const int *start, *kstart;           // [B + 1]
  float scale;
  void* scratch;                       // of prompt_attention_scratch's size, or less: then items are not split
  size_t scratch_bytes;
  int* err;
};
int prompt_attention(cudaStream_t st, const PromptArgs& a);
size_t prompt_attention_scratch(int R, int Rk, int nq, int nkv, int d, int B);      // 0: no use for it

// Code and exponent arrays of one layer: k, v, ke, ve.
struct Kv8Layer { uint8_t* p[4]; };

int kv8_compact(cudaStream_t st, const Kv8& c, const Kv8Layer* layers, int n_layers, int B, const int* n_old,
                const int* acc_len, const int* acc_path, int Dmax, int* err);
size_t kv8_resize_scratch(const Kv8& c);
int kv8_resize(cudaStream_t st, const Kv8& c, const Kv8Layer* layers, int n_layers, int B, int* refs, const int* parent,
               const int* length, void* scratch, int* err);

}  // namespace eagle
