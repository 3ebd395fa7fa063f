// int4_tile_f16.hip -- the tiled int4 kernels for fp16 activations.
#include "int4_tile.h"

namespace k3g {
int launch_int4_tile_f16(const I4Args &a, int mode, int group, int form, hipStream_t st) {
    return launch_int4_tile_type<K3G_F16>(a, mode, group, form, st);
}
}  // namespace k3g
