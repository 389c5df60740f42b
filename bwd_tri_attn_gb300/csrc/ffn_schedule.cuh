// Which buffer, which barrier and which phase of it belong to a feature block in the one-kernel forward (ffn_block.cu): plain
// arithmetic, so that a model of the waits can take it on the host, too.
//
// A wait by parity passes when the barrier's phase of that parity is done, and one phase before it as well: it is right only
// where the phase before is known to be done. Two groups of warps take the blocks in turn. With an odd number of buffers the
// blocks of one buffer go to the groups in turn as well, and a group would see only every second phase of its barrier: block n's
// sums could be taken for those of block n + 2 NS, while those of n + NS, the other group's, are not there yet (two warps
// issue them, each when its own weights have come). So the sums have a barrier for each buffer and group: whoever waits there
// sees every phase. All others are seen by one warp in order, or follow such a wait.
#pragma once

namespace triattn {
namespace ffn {

template <int BUFFERS, int SLOTS>  // of sums in TMEM, of weights in shared memory
struct BlockSchedule {
  static constexpr int kSums = BUFFERS % 2 ? 2 * BUFFERS : BUFFERS;  // barriers
  static constexpr int buffer(int n) { return n % BUFFERS; }
  static constexpr int slot(int n) { return n % SLOTS; }
  static constexpr int slot_phase(int n) { return n / SLOTS; }  // (weights there; free again after block n)
  static constexpr int sums(int n) { return n % kSums; }
  static constexpr int sums_phase(int n) { return n / kSums; }
  static constexpr int hidden_phase(int n) { return n / BUFFERS; }  // (h written; its barrier is the buffer's)
};

}  // namespace ffn
}  // namespace triattn
