// int4_tile_f32.hip -- the tiled int4 kernels for fp32 activations.
#include "int4_tile.h"

namespace k3g {
int launch_int4_tile_f32(const I4Args &a, int mode, int group, int form, hipStream_t st) {
    return launch_int4_tile_type<K3G_F32>(a, mode, group, form, st);
}
}  // namespace k3g
