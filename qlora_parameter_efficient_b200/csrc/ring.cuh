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
    QL_HD RingPos(int stages, int start) : S(stages), s(start), ph(0) {     // start < 2 S
        if (s >= S) s -= S, ph ^= 1;
    }
    QL_HD void skip(int n) {                 // n <= S
        s += n;
        if (s >= S) s -= S, ph ^= 1;
    }
};

// Until the load of this position's use of its slot has landed, for one of GROUPS groups that take every
// GROUPS-th stage each (GROUPS <= S).  A wait by parity tells a barrier's last two phases apart only, so
// whoever waits for full[s] must know that the load of the slot's use before has landed: with that load
// still in flight (loads land in any order) the barrier is a phase further back, whose parity says "landed".
// Where S is a multiple of GROUPS, a slot is always the same group's, which has waited for that load itself.
// Where it is not, the use before was another group's, and the group first waits for its release (which
// came after its load had landed).  That wait cannot be mistaken: the group has seen the load of GROUPS
// stages ago land, the producer issued that one after the release of S stages earlier still, which is the use
// before the last one or a later stage; and the use waited for here is not released without this group.
// (With pairs of stages in turn and that wait at each, dA and dB of 4096 tokens, 4096 x 4096, took 26.5 us, so 25.5.)
template <int GROUPS, typename WaitEmpty, typename WaitFull>
QL_HD bool ring_landed(const RingPos& p, WaitEmpty wait_empty, WaitFull wait_full) {
    if (p.S % GROUPS != 0 && !wait_empty(p.s, p.ph ^ 1)) return false;
    return wait_full(p.s, p.ph);
}

}  // namespace qlora
