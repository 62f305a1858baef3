// Host arithmetic of the launches, apart from CUDA so that it can be compiled and checked by itself.
#pragma once

namespace w4g {

// ceil(n / per) for n >= 0, per >= 1; n + per - 1 may pass 31 bits.
inline unsigned blocks_for(int n, int per) {
    return (static_cast<unsigned>(n) + static_cast<unsigned>(per) - 1) / static_cast<unsigned>(per);
}

// The exponent of a power of two (v >= 1), or -1 if v is none.
inline int power_of_two(int v) {
    if ((v & (v - 1)) != 0) return -1;
    int l = 0;
    while (v >> l != 1) ++l;
    return l;
}

}  // namespace w4g
