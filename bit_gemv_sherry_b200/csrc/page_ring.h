// page_ring.h -- which pages of a warp's ring are on their way (plain C++: the kernels' and the host's).
//
// Page j of a warp lies in slot j % S of its ring and completes phase (j / S) & 1 of that slot's barrier.
// A page is copied, and later taken by a wait that saw it land.  A wait that runs out takes nothing: from
// there on no page is copied or taken, and the pages in [taken, copied) may still be landing, whatever the
// warp's walk does after it.  Their waits have to end before the ring is used again or released.
#pragma once

#ifdef __CUDACC__
#define SHERRY_HD __host__ __device__ __forceinline__
#else
#define SHERRY_HD inline
#endif

namespace sherry {

template <int S>
struct PageRing {
    int copied = 0, taken = 0;
    int to = 0, at = 0;     // slots of the next copy and of the next wait
    unsigned lap = 0;       // the next wait's phase
    bool dead = false;      // a wait ran out

    SHERRY_HD void copy() {
        copied++;
        to = to + 1 == S ? 0 : to + 1;
    }
    SHERRY_HD void take(bool landed) {
        if (!landed) dead = true;
        if (dead) return;
        taken++;
        if (++at == S) at = 0, lap ^= 1;
    }
    // f(slot, phase) for each page that may still be landing.
    template <typename F>
    SHERRY_HD void drain(F f) const {
        for (int j = taken; j < copied; j++) f(j % S, (unsigned)(j / S) & 1u);
    }
};

}  // namespace sherry
