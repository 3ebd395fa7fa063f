// int4_stream_f32.hip -- the streaming int4 kernels for fp32 activations.
#include "int4_stream.h"

namespace k3g {
int launch_int4_stream_f32(const I4Args &a, int mode, int group, int form, hipStream_t st) {
    return launch_int4_stream_type<K3G_F32>(a, mode, group, form, st);
}
}  // namespace k3g
