// rssm_wait.h -- a bounded wait of a whole warp, whose outcome is the same for every lane.
//
// Every lane polls (each needs the barrier's ordering for itself), and lanes may see a barrier's phase end, the
// limit pass or the failure flag rise at different times.  What follows a wait are instructions of the whole warp
// (votes, tensor-memory loads and stores), so that lanes which went different ways would leave the others waiting
// for them: all lanes go on once all have seen the phase, and all give up as soon as one does.
#pragma once

#if defined(__CUDACC__)
#define RSSM_WAIT_FN __device__ __forceinline__
#else
#define RSSM_WAIT_FN inline
#endif

namespace rssm {

// ready(): this lane sees the phase ended; expired(): it has waited too long, or another wait has failed; all(x), any(x):
// votes of the warp.  ready() is not asked again once it was true: the next phase may end meanwhile.
template <class Ready, class Expired, class All, class Any>
RSSM_WAIT_FN bool wait_together(Ready ready, Expired expired, All all, Any any) {
    bool mine = ready();
    while (!all(mine)) {
        if (any(!mine && expired())) return false;
        if (!mine) mine = ready();
    }
    return true;
}

}  // namespace rssm
