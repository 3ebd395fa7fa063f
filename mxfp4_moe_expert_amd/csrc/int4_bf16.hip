// int4_bf16.hip -- the int4 product kernels for bf16 activations.
#include "int4_launch.h"

namespace k3g {
int launch_int4_bf16(const I4Args &a, int mode, int group, hipStream_t st) {
    return launch_int4_type<K3G_BF16>(a, mode, group, st);
}
}  // namespace k3g
