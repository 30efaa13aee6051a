// pkv_cursor.cuh -- a worker's way along the line of all (sequence, kv head)
// units' blocks: plain integer code, compiled for the host as well.
#pragma once

#ifdef __CUDACC__
#define PKV_HOST_DEVICE __host__ __device__ __forceinline__
#else
#define PKV_HOST_DEVICE inline
#endif

namespace pkv {

// Position cursor: sequence s (with n = its blocks), kv head h, block j.
struct Cursor {
    int s, h, j, n;
};

// Moves c forward by k >= 0 positions; prefix[] holds the block-count prefix
// sums. The caller guarantees the target position exists.
PKV_HOST_DEVICE void cursor_advance(Cursor &c, int k, const int *prefix, int num_kv_heads) {
    while (c.j + k >= c.n) {
        k -= c.n - c.j;
        c.j = 0;
        if (++c.h == num_kv_heads) {
            c.h = 0;
            do {
                ++c.s;
                c.n = prefix[c.s + 1] - prefix[c.s];
            } while (c.n == 0);
        }
    }
    c.j += k;
}

// Calls f(s, h) for every unit that begins behind c's own within the `left` positions from c on.
template <typename F>
PKV_HOST_DEVICE void units_begun_later(Cursor c, int left, const int *prefix, int num_kv_heads, F f) {
    while (left > c.n - c.j) {
        left -= c.n - c.j;
        cursor_advance(c, c.n - c.j, prefix, num_kv_heads);
        f(c.s, c.h);
    }
}

}  // namespace pkv
