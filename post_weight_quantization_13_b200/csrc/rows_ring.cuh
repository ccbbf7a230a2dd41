// How int8_rows.cu's blocks share out channels and shared memory, and the walk
// over their rings: plain C++ (no device code), so that host tests can go
// through every size.
//
// A block has a ring for each group of threads.  Batches alternate between the
// groups, a batch is whole slots of its group's ring, and a group waits for
// every fill of that ring in the order in which they are issued.  That is what
// makes a wait on a phase's parity safe: such a wait also passes while the
// barrier is still one phase behind, which cannot be where the same threads
// have waited for the slot's previous fill.  (In one ring for both groups that
// fill may be the other group's, and copies land in any order.)
#pragma once

#include <cstdint>

#ifdef __CUDACC__
#define GPTQ_BOTH __host__ __device__ __forceinline__
#else
#define GPTQ_BOTH inline
#endif

namespace gptq {
namespace rows {

constexpr int kThreads = 256;          // of a group, whose threads split k
constexpr int kGroups = 2;             // that take the batches in turn
constexpr int kBatch = 8;              // weight rows of a reduction
constexpr int kSlice = kThreads * 16;  // columns of one step
constexpr int kMaxSteps = 3;           // in <= 12288
constexpr int kMaxSlots = 20;          // of a ring
constexpr int kStatic = 4 * 1024;      // shared memory left to the static arrays
constexpr int kSmem = 227 * 1024 - kStatic;

// A place in a ring of `slots` slots and the parity of its current fill.
struct Cursor {
  int slot = 0;
  uint32_t phase = 0;
  GPTQ_BOTH void advance(int by, int slots) {
    slot += by;
    while (slot >= slots) {
      slot -= slots;
      phase ^= 1;
    }
  }
};

struct Plan {
  int grid;        // blocks; block b owns channels out * b / grid up to out * (b + 1) / grid
  int rows;        // the most channels a block owns
  int dense;       // rows come as they lie, padding and all, one copy a slot
  int row_bytes;   // between rows in a slot
  int group;       // channels of a slot: 1, 2, 4 or 8, so that a batch is whole slots
  int slot_bytes;
  int slots;       // of one ring, at least a batch
  int smem;        // dynamic shared memory
};

// G projections of T tokens; ldw: their row strides, the same for all or 0.
inline Plan plan(int G, int T, int in, int out, int64_t ldw, int sms) {
  Plan p = {};
  const int codes = T * ((in + kSlice - 1) / kSlice) * kThreads * 16;
  const int vectors = 4 * (2 * G + (G == 1 ? 1 : 0));  // of a channel: scales, zeros, bias
  // Slots of up to 32 KB (a copy's issue takes as long as some KB of it).  Rows
  // that lie closely one after another come in one copy, unless their padding
  // leaves a ring no room for a batch.
  for (p.dense = ldw > 0 && ldw <= in + 127;; p.dense = 0) {
    p.row_bytes = p.dense ? (int)ldw : (in + 15) / 16 * 16;
    p.group = kBatch / G;
    while (p.group > 1 && G * p.group * p.row_bytes > 32768) p.group /= 2;
    p.slot_bytes = (G * p.group * p.row_bytes + 127) / 128 * 128;
    const int batch = kBatch / G / p.group;  // slots
    // one block an SM; more where a block's channels would leave the rings no
    // room for a batch each (only with many channels on few SMs)
    const int most = (kSmem - codes - kGroups * batch * p.slot_bytes) / vectors;
    const int wide = out < sms ? out : sms;
    if (p.dense && most < (out + wide - 1) / wide) continue;  // without padding most is 448 at least
    const int least = (out + most - 1) / most;
    p.grid = wide > least ? wide : least;
    p.rows = (out + p.grid - 1) / p.grid;
    const int room = (kSmem - codes - vectors * p.rows) / p.slot_bytes / kGroups;
    p.slots = room < kMaxSlots ? room : kMaxSlots;
    p.smem = codes + vectors * p.rows + kGroups * p.slots * p.slot_bytes;
    return p;
  }
}

}  // namespace rows
}  // namespace gptq
