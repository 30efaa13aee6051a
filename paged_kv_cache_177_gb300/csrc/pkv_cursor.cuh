// pkv_cursor.cuh -- walks over a worker's units: plain integer code, compiled
// for the host as well.
#pragma once

#ifdef __CUDACC__
#define PKV_HOST_DEVICE __host__ __device__ __forceinline__
#else
#define PKV_HOST_DEVICE inline
#endif

namespace pkv {

// Calls f(s, h) for every unit that begins behind cursor c's own within the `left` positions from c on;
// advance(c, k) moves c by k positions.
template <typename C, typename Advance, typename F>
PKV_HOST_DEVICE void units_begun_later(C c, int left, Advance advance, F f) {
    while (left > c.n - c.j) {
        left -= c.n - c.j;
        advance(c, c.n - c.j);
        f(c.s, c.h);
    }
}

}  // namespace pkv
