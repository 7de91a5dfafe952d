// ring.cuh -- how groups of warps take the stages of a ring in turn.  (Plain C++ too, so that a test can run
// it against a model of the barriers.)
#pragma once

#ifdef __CUDACC__
#define QL_HD __host__ __device__ __forceinline__
#else
#define QL_HD inline
#endif

namespace qlora {

// A position in a ring of S stages: the slot, and the parity of its use (use n of a slot is phase n of
// its barriers).
struct RingPos {
    int S, s, ph;
    QL_HD RingPos(int stages, int start) : S(stages), s(start), ph(0) {
        if (s >= S) s -= S, ph ^= 1;
    }
    QL_HD void skip(int n) {                 // n <= S
        s += n;
        if (s >= S) s -= S, ph ^= 1;
    }
};

// Stages that one group takes in a row before the next group's.
constexpr int kRingRun = 2;
// Fewest stages of a ring that `groups` groups share (see ring_landed).
constexpr int ring_min_stages(int groups) { return kRingRun * (groups - 1) + 1; }

// Until the load of this position's use of its slot has landed.  A wait by parity tells a barrier's last two
// phases apart only.  A group that sees every stage knows that the use before this one has landed; one that
// takes stages in turn with others does not, and loads land in any order: with the load before still in
// flight, full[s] is a phase further back, whose parity says "landed".  So such a group first waits
// until the slot's last use was released (which came after its load had landed).  That wait
// cannot be mistaken: the group has seen the load of kRingRun (groups - 1) + 1 stages ago land, the producer
// issued that one after the release of S stages earlier still, and, from ring_min_stages on, this is the use
// before the last one or a later stage; and the use waited for here is not released without this group.
template <int GROUPS, typename WaitEmpty, typename WaitFull>
QL_HD bool ring_landed(const RingPos& p, WaitEmpty wait_empty, WaitFull wait_full) {
    if (GROUPS > 1 && !wait_empty(p.s, p.ph ^ 1)) return false;
    return wait_full(p.s, p.ph);
}

}  // namespace qlora
