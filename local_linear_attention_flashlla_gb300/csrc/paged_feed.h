// The order in which the feeding warp of the paged tcgen05 kernel fills its two rings of copies, of K (0) and of V (1), and
// which copies it waits for where it gives up.  Host code too, so that the order is tested without a GPU.
#pragma once

#ifdef __CUDACC__
#define LLA_FEED_FN __host__ __device__ __forceinline__
#else
#define LLA_FEED_FN inline
#endif

namespace lla {
namespace paged {

// NS stages to a ring.  Rings has wait_empty(ring, stage, parity), false where the wait gave up, copy(ring, stage), which
// starts the copies of a block, and wait_full(ring, stage, parity), which waits (with a limit) until they have landed.
template <int NS>
struct RingCount {
    int blocks = 0;        // both of whose copies were started
    bool k_ahead = false;  // K's copy of the next one was, too: the wait for V's stage gave up

    // One block; false: a wait gave up.
    template <typename Rings>
    LLA_FEED_FN bool feed_block(Rings& rings) {
        const int stage = blocks % NS, parity = ((blocks / NS) & 1) ^ 1;
        if (!rings.wait_empty(0, stage, parity)) return false;
        rings.copy(0, stage);
        if (!rings.wait_empty(1, stage, parity)) {
            k_ahead = true;
            return false;
        }
        rings.copy(1, stage);
        ++blocks;
        return true;
    }
    // Every copy that may be in flight has landed: the last NS of each ring (a stage is filled again only after its
    // copy before was consumed).
    template <typename Rings>
    LLA_FEED_FN void drain(Rings& rings) const {
        for (int kv = 0; kv < 2; ++kv) {
            const int n = blocks + (kv == 0 && k_ahead);
            for (int t = n > NS ? n - NS : 0; t < n; ++t) rings.wait_full(kv, t % NS, (t / NS) & 1);
        }
    }
};

}  // namespace paged
}  // namespace lla
