// moe_ring.h -- the way out of a block whose waits ran out: which copies into its
// shared memory may still be on their way, and the barriers that tell of them.  Host and
// device, so that tests/test_ring.py runs it without a GPU.
//
// A ring: copy n goes to stage n % stages, and phase n / stages of that stage's barrier
// is complete once it has landed.  A thread that issues copies waits for a stage's
// readers before it uses it again and issues nothing more once the block gives up, so
// the copies issued are 0 .. issued - 1 and of them only the last `stages` may not have
// landed.  (A phase whose copy was never issued must not be waited for: its parity is
// that of the phase before it, or never comes.)
#pragma once

#ifdef __CUDACC__
#define MOE_RING_FN __host__ __device__ __forceinline__
#else
#define MOE_RING_FN inline
#endif

namespace moe {

// landed(stage, parity) waits for that phase of the stage's barrier.
template <class Landed>
MOE_RING_FN void ring_drain(int issued, int stages, Landed landed)
{
    for (int n = issued > stages ? issued - stages : 0; n < issued; ++n) landed(n % stages, (n / stages) & 1);
}

// The same for copies that come in two halves by two threads (two arrivals a phase), which
// take every other copy, those with n % 2 = first.  a and b: one past the last copy whose half each
// issued (0: none).  The half that one of them did not get to is arrived for, once.
template <class Arrive, class Landed>
MOE_RING_FN void ring_drain_halves(int first, int a, int b, int stages, Arrive arrive, Landed landed)
{
    const int lo = a < b ? a : b, hi = a < b ? b : a;
    for (int n = lo + ((lo ^ first) & 1); n < hi; n += 2) arrive(n % stages);
    const int n0 = hi > stages ? hi - stages : 0;
    for (int n = n0 + ((n0 ^ first) & 1); n < hi; n += 2) landed(n % stages, (n / stages) & 1);
}

}  // namespace moe
