// Host-only stand-ins for the launchers of seed_channels_launch.h (see
// stub_launch.cpp): they enqueue nothing and report success.  Sizes that the
// validation asks for are the library's own formulas' order of magnitude.
#include "seed_channels_launch.h"

namespace seed {

hipError_t launch_short_conv(const ConvArgs&, hipStream_t) { return hipSuccess; }
hipError_t launch_short_conv_backward(const ConvArgs&, hipStream_t) { return hipSuccess; }
hipError_t launch_short_conv_step(const ConvArgs&, hipStream_t) { return hipSuccess; }
int short_conv_parts(int n_seq, int, int tokens) { return tokens / 32 + n_seq < 128 ? tokens / 32 + n_seq : 128; }
bool short_conv_fits(int n_seq, int, int tokens) { return (long long)(tokens >> 5) + n_seq < (1LL << 24) - 1; }
SelectLayout select_layout(int n_seq, int channels, int groups, int d_state, int tokens, bool backward) {
  SelectLayout l{};
  const int states = d_state <= 16 ? 16 : d_state <= 32 ? 32 : 64;
  l.bytes = (size_t)tokens * groups * 8 * states + (backward ? (size_t)n_seq * channels * 64 : 0);
  return l;
}
bool select_fits(int n_seq, int channels, int groups, int d_state, int tokens) {
  return d_state <= 64 && (long long)groups * ((channels / groups + 63) / 64) <= 65535 &&
         (long long)(tokens >> 6) + n_seq < (1LL << 24) && (long long)tokens + 64 <= 0x7fffffffLL;
}
hipError_t launch_select(const SelectArgs&, hipStream_t) { return hipSuccess; }
hipError_t launch_select_backward(const SelectArgs&, hipStream_t) { return hipSuccess; }
hipError_t launch_select_step(const SelectArgs&, hipStream_t) { return hipSuccess; }

}  // namespace seed
