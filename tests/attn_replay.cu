// Host entries over parts of the decode kernel that decide which thread writes and reads what,
// for tests without a GPU.
#include "../mxfp4_routed_expert_latentmoe_gb300/csrc/attn/k3_decode.cuh"

namespace {
using namespace k3;

template <typename F>
bool with_config(int fmt, int dp, int nt, F&& f) {
  switch (fmt * 1000 + dp * 2 + nt - 1) {
    case 128: f(DecCfg<CF_BF16, 64, 1>()); return true;
    case 129: f(DecCfg<CF_BF16, 64, 2>()); return true;
    case 256: f(DecCfg<CF_BF16, 128, 1>()); return true;
    case 257: f(DecCfg<CF_BF16, 128, 2>()); return true;
    case 384: f(DecCfg<CF_BF16, 192, 1>()); return true;
    case 385: f(DecCfg<CF_BF16, 192, 2>()); return true;
    case 512: f(DecCfg<CF_BF16, 256, 1>()); return true;
    case 513: f(DecCfg<CF_BF16, 256, 2>()); return true;
    case 1128: f(DecCfg<CF_E4M3, 64, 1>()); return true;
    case 1129: f(DecCfg<CF_E4M3, 64, 2>()); return true;
    case 1256: f(DecCfg<CF_E4M3, 128, 1>()); return true;
    case 1257: f(DecCfg<CF_E4M3, 128, 2>()); return true;
    case 1384: f(DecCfg<CF_E4M3, 192, 1>()); return true;
    case 1385: f(DecCfg<CF_E4M3, 192, 2>()); return true;
    case 1512: f(DecCfg<CF_E4M3, 256, 1>()); return true;
  }
  return false;
}
}  // namespace

extern "C" {

// An instance's shape: warps, bytes of all rings, tokens of a tile.  0: no such instance.
int replay_config(int fmt, int dp, int nt, int32_t* shape) {
  return with_config(fmt, dp, nt, [&](auto c) {
    using C = decltype(c);
    shape[0] = C::WARPS;
    shape[1] = C::RING;
    shape[2] = C::TW;
  });
}

// What one lane of a warp clears of the rings.
void replay_clear(int fmt, int dp, int nt, uint8_t* rings, int warp, int lane) {
  with_config(fmt, dp, nt, [&](auto c) { clear_ring<decltype(c)>(rings, warp, lane); });
}

// The token of a row of a warp's tile of a unit, for tiles of 16 or 32 tokens.
uint32_t replay_token(int32_t first, int32_t u, int W, int tw, int tile, int row) {
  DecAt at{};
  at.first = first;
  at.u = u;
  return tile == 16 ? at.token<16>(W, tw, row) : at.token<32>(W, tw, row);
}

// The units that a team takes, as (b, kvh, grp, u) each: its range begins `off` places after the
// first one of sequence b and has `end` places.  Returns their number (at most `most` are written).
int replay_team(const int32_t* lens, int B, int Hkv, int groups, int window, int longest, int tile_log, int wlog,
                int whole, int start, int b, int64_t off, int32_t end, int32_t* units, int most) {
  DecodeParams p{};
  p.B = B;
  p.Hkv = Hkv;
  p.groups = groups;
  p.window = window;
  p.lens = lens;
  p.table_width = longest;
  p.c.page_size = 1;
  DecAt at{};
  at.b = b;
  at.open(p, tile_log + wlog);
  int n = 0;
  for (at.land(p, tile_log + wlog, off, end, whole, start); at.in(end, whole, start); at.next(p, tile_log + wlog, end, start)) {
    if (n < most) {
      units[4 * n] = at.b;
      units[4 * n + 1] = at.kvh;
      units[4 * n + 2] = at.grp;
      units[4 * n + 3] = at.u;
    }
    ++n;
  }
  return n;
}

// Places of a sequence's start, and the most units of a sequence that is not cut, for teams of
// 2^wlog warps.
int replay_start(int wlog) { return dec_start(wlog); }
int replay_whole(int wlog) { return DEC_WHOLE >> wlog; }

}  // extern "C"
