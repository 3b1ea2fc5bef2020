// prefill_replay.cu with a tile's start counted as replay_start says, instead of as PRE_START.
#include "../mxfp4_routed_expert_latentmoe_gb300/csrc/attn/k3_prefill.cuh"

static int replay_started = k3::PRE_START;
struct StartedParams : k3::PrefillParams {
  StartedParams() : k3::PrefillParams{} { start = replay_started; }
};
#define PrefillParams StartedParams
#define PRE_START replay_started
#include "prefill_replay.cu"
#undef PrefillParams
#undef PRE_START

extern "C" void replay_start(int start) { replay_started = start; }
// what the kernel is called with
extern "C" int replay_start_of(int bf16, int two_halves) { return k3::pre_start(bf16 != 0, two_halves != 0); }
// what it counts as in a call of `total` places with `start`
extern "C" int replay_start_in(int start, int64_t total, int64_t blocks) {
  k3::PrefillParams p{};
  p.start = start;
  return k3::pre_start_in(p, total, blocks);
}
