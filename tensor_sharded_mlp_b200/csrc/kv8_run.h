// kv8_run.h -- the order in which a CTA of the prompt append works through its run of units (also compiled for the host, by
// a test).
#pragma once

#ifdef __CUDACC__
#define TPMLP_RUN_FN __host__ __device__ __forceinline__
#else
#define TPMLP_RUN_FN inline
#endif

namespace tpmlp {

// `run` units from head `head0` of slot 0 on, heads within slots.  work(slot, head, turn) for those whose slot has
// something to write.  `turn` says which of two exchange buffers the unit may use: it alternates between the units that
// run, whatever lies between them.  A unit holds one barrier, so a warp can be one unit ahead of another, and two units
// in a row must not share a buffer.
template <typename HasWork, typename Work>
TPMLP_RUN_FN void for_units(int run, int head0, int heads, HasWork has_work, Work work) {
    int slot = 0, head = head0, turn = 0;
    for (int u = 0; u < run; ++u) {
        if (has_work(slot)) {
            work(slot, head, turn);
            turn ^= 1;
        }
        if (++head == heads) {
            head = 0;
            ++slot;
        }
    }
}

}  // namespace tpmlp
