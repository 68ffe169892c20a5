// Launchers of item ids (embed.cu) and decay attention (decay_attn.cu), and what
// they share with the host side.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace rest {

// ---------------------------------------------------------------- item ids
cudaError_t launch_embed_forward(bool bf16, long long n_rows, int d, const void* table, long long n_tokens,
                                 const int64_t* ids, float scale, void* out, int32_t* err, cudaStream_t s);
size_t embed_backward_ws_bytes(long long n_rows, int d, long long n_tokens);
// The gradient runs as embed_backward_launches() launches, `step` counting them.
int embed_backward_launches(long long n_rows, long long n_tokens);
cudaError_t launch_embed_backward(int step, bool bf16, long long n_rows, int d, const void* d_out,
                                  long long n_tokens, const int64_t* ids, float scale, bool accumulate,
                                  float* d_table, void* ws, int32_t* err, cudaStream_t s);

// ---------------------------------------------------------------- decay attention
struct DecayHeadsArg {
  int n_heads;
  long long tau[32];   // per head, 0 = position head
  double inv[32];      // 1 / tau
  double decay2[32];   // per head, log decay in base 2 (<= 0)
};
// Cached states (rest_decay_state) and the slot of each user or entry; s null: none.
struct DecayState {
  float* s;
  int64_t* len;
  int64_t* t_first;
  int64_t* t_last;
  int n_slots;
  const int32_t* slots;  // null: slot u of user u
};
// Users u0 .. u0 + n - 1 of a call and their rows, passed to a kernel by value
// (a copy from host memory would be read again by every replay of a captured
// call, when the host array may be gone).
constexpr int DECAY_USERS = 320;
struct DecayUsers {
  int u0, n;
  int32_t cu[DECAY_USERS + 1];
  int32_t part0[DECAY_USERS];  // each user's first part
  int32_t item0[DECAY_USERS];  // and its first item
};
// What a user's rows continue: its slot (-1: none) and what the slot held before the call.
struct DecayRec {
  int row0, slot;   // the user's first row
  long long len0;
  long long t0;     // timestamp of the history's first token
  long long tprev;  // of the last cached token (t0 without one)
};
// Work item: one segment of a user's rows, segment seg of nseg. A history of
// more than one segment has states between them, summed over parts, DecayCut::m
// to a segment; part0 .. part1 are this segment's.
struct DecayItem {
  DecayRec rec;
  int row0, rows, seg, nseg, part0, part1;
};
// Part of a segment (of a history with more than one), part `part` of the user's `parts`.
struct DecayPart {
  DecayRec rec;
  int row0, rows, part, parts;
};
// A user: its parts (none without a second segment), for the join.
struct DecayUser {
  int slot, part0, parts;
  long long len0;
};
struct DecayCut {
  int rows;  // of a segment: m parts
  int m;
};
// The row bounds of a call on histories that start empty, by value: up to
// DECAY_FEW users, whose items and parts every kernel works out itself (n = 0:
// the prologue has written them).
constexpr int DECAY_FEW = 80;
struct DecayFew {
  int n;
  int32_t cu[DECAY_FEW + 1];
  int32_t item0[DECAY_FEW];
  int32_t part0[DECAY_FEW];
};
struct DecayArgs {
  DecayHeadsArg h;
  DecayFew few;
  const DecayItem* items;
  const DecayPart* parts;
  const DecayUser* users;
  int n_parts;
  DecayCut cut;
  const int64_t* ts;
  float* state;      // cached states, or null
  // [1 or 2 (backward), parts, n_heads, hd, hd]: a part's own state; after the join, at a
  // segment's first part the state before it (backward: at its last, the one after it)
  float* part_state;
  float* part_decay;  // [1 or 2, parts, n_heads]: what a state keeps over the part
  int d;
  long long rows;  // T
  float scale;     // 1 / sqrt(head_dim)
  int32_t* err;
};
// The step's bounded waits: their limit in cycles, and arrivals that never come (the self-test's).
struct DecayWait {
  long long limit;
  int missing;
};
cudaError_t launch_decay_prep(const DecayUsers& users, const int64_t* ts, const DecayState& st, const DecayArgs& a,
                              DecayItem* items, DecayPart* parts, DecayUser* heads, cudaStream_t s);
// Every part's own state sum_j decay x0_j y0_j^T; with back also sum_i decay x1_i y1_i^T from the other side.
cudaError_t launch_decay_parts(bool bf16, int hd, bool back, bool exact, const DecayArgs& a, const void* x0,
                               const void* y0, const void* x1, const void* y1, cudaStream_t s);
// The states before (back: also after) every segment.
cudaError_t launch_decay_join(int hd, bool back, int n_users, const DecayArgs& a, cudaStream_t s);
// o = decay attention of q, k, v. exact: the state is an output too.
cudaError_t launch_decay_pass(bool bf16, int hd, bool exact, int n_items, const DecayArgs& a, const void* q,
                              const void* k, const void* v, void* o, cudaStream_t s);
cudaError_t launch_decay_dkdv(bool bf16, int hd, int n_items, const DecayArgs& a, const void* q, const void* k,
                              const void* v, const void* d_o, void* dk, void* dv, cudaStream_t s);
cudaError_t launch_decay_step(bool bf16, int hd, const DecayHeadsArg& hs, int n, const void* q, const void* k,
                              const void* v, const int64_t* ts, const DecayState& st, void* o, float scale,
                              const DecayWait& waits, int32_t* err, cudaStream_t s);

}  // namespace rest
