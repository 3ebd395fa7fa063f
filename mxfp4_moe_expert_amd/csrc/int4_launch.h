// int4_launch.h -- which kernel an int4 product runs on.
#pragma once

#include "int4_tile.h"

namespace k3g {

template <int XT, int GROUP, int MODE>
int launch_int4_mode(const I4Args &a, hipStream_t st) {
    if (MODE == DENSE && a.T <= 16 && a.rows <= 16 * 256) return launch_int4_stream<XT, GROUP, MODE, 1, 1>(a, st);
    constexpr int RT = MODE == GLU ? 1 : 2;
    const int64_t n = MODE == DENSE ? a.T : (a.T + a.E - 1) / a.E;
    if (n > 32) {
        if constexpr (XT != K3G_F32)
            if (a.x_vec) return launch_int4_tile<XT, GROUP, MODE, 8, true>(a, st);
        return launch_int4_tile<XT, GROUP, MODE, 4, false>(a, st);
    }
    if (n <= 16) return launch_int4_stream<XT, GROUP, MODE, RT, 1>(a, st);
    if (n <= 32) return launch_int4_stream<XT, GROUP, MODE, RT, 2>(a, st);
    return launch_int4_stream<XT, GROUP, MODE, RT, 4>(a, st);
}

template <int XT, int GROUP>
int launch_int4_group(const I4Args &a, int mode, hipStream_t st) {
    return mode == DENSE ? launch_int4_mode<XT, GROUP, DENSE>(a, st) : mode == GROUPED ? launch_int4_mode<XT, GROUP, GROUPED>(a, st) : launch_int4_mode<XT, GROUP, GLU>(a, st);
}

template <int XT>
int launch_int4_type(const I4Args &a, int mode, int group, hipStream_t st) {
    return group == 32 ? launch_int4_group<XT, 32>(a, mode, st) : group == 64 ? launch_int4_group<XT, 64>(a, mode, st) : launch_int4_group<XT, 128>(a, mode, st);
}

}  // namespace k3g
